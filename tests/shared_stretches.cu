// How the keys of swa_paged_attend_shared's units are cut into stretches and which sequences have rows in common
// (swa_paged_shared.cuh), for test_shared_lists_cpu.py: the kernels' own functions, run on the host.  Built by that test as a
// library of its own.
#include "swa_paged_shared.cuh"

namespace {

swa::PagedArgs args(int window, int n_sink) {
    swa::PagedArgs a{};
    a.window = window > 0 ? window : INT_MAX;
    a.n_sink = n_sink;
    return a;
}

int put(const swa::Keys &k, int *out) {
    for (int i = 0; i < k.stretches(); ++i) {
        out[2 * i] = k.begin(i);
        out[2 * i + 1] = k.close(i);
    }
    return k.stretches();
}

swa::PartResults planes_of(int planes) {
    swa::PartResults p{};
    p.planes = planes;
    return p;
}

}  // namespace

#define EXPORT extern "C" __attribute__((visibility("default")))

// out [planes][2]: the first key of each stretch and the one behind its last; returns their number.
EXPORT int own_stretches(int p0, int n, int base, int ut, int TT, int window, int n_sink, int planes, int *out) {
    return put(swa::own_keys(args(window, n_sink), swa::Seq{0, n, p0, true}, base, ut, TT, planes_of(planes)), out);
}

EXPORT int prefix_stretches(int p0, int end, int window, int n_sink, int planes, int *out) {
    return put(swa::prefix_keys(args(window, n_sink), p0, end, planes_of(planes)), out);
}

// Of a batch of B sequences with their rows q_start[b] .. q_start[b + 1] - 1 in [0, N): the stretches of all that are in
// range, and of those of them that have no row in common with another.
EXPORT void count_stretches(const int *q_start, const int *p0, int B, int N, int TT, int planes, long long *all, long long *taken) {
    *all = *taken = 0;
    const auto sequence = [&](int b) {
        const bool ok = q_start[b] >= 0 && q_start[b + 1] >= q_start[b] && q_start[b + 1] <= N;
        return swa::Seq{q_start[b], ok ? q_start[b + 1] - q_start[b] : 0, p0[b], ok};
    };
    for (int b = 0; b < B; ++b) {
        const swa::Seq s = sequence(b);
        bool alone = true;
        for (int c = 0; c < B && alone; ++c) alone = c == b || !swa::in_common(s, sequence(c));
        long long mine = 0;
        for (int ut = 0; ut * TT < s.n; ++ut)
            mine += swa::own_keys(args(0, 0), s, 0, ut, TT, planes_of(planes)).stretches();
        *all += mine;
        if (alone) *taken += mine;
    }
}
