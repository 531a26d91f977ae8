// swa_paged.cuh -- device-side geometry of a paged batch: which sequence a token belongs to,
// what is valid of it, and which page holds a position.  Everything read from the device is
// checked here, so that an index made from it stays inside its tensor.
#pragma once

#include <climits>

#include "ptx.cuh"
#include "swa_paged.h"

namespace swa {

// New tokens q0 .. q0 + n - 1 of sequence b at positions p0 ..; ok: its rows lie in [0, N) and
// its positions in its table row (otherwise n = 0 and the sequence is skipped).
struct Seq {
    int q0, n, p0;
    bool ok;
};

__device__ __forceinline__ Seq load_seq(const PagedArgs &a, int b) {
    Seq s;
    int q1;
    if (a.q_start) {
        s.q0 = __ldg(a.q_start + b);
        q1 = __ldg(a.q_start + b + 1);
    } else {
        s.q0 = b;
        q1 = b + 1;
    }
    s.p0 = __ldg(a.p0 + b);
    s.ok = s.q0 >= 0 && q1 >= s.q0 && q1 <= a.N && s.p0 >= 0 &&
           static_cast<int64_t>(s.p0) + (q1 - s.q0) <= (static_cast<int64_t>(a.width) << a.ps_log2);
    s.n = s.ok ? q1 - s.q0 : 0;
    return s;
}

// The sequence of token n, looked up by a whole warp: the last b with q_start[b] <= n (for a
// list that does not decrease); -1 if none has it.  Each step cuts the range 32-fold.
__device__ __forceinline__ int find_sequence(const PagedArgs &a, int n, int lane) {
    if (!a.q_start) return n < a.B ? n : -1;
    int lo = 0, len = a.B;  // candidates lo .. lo + len - 1
    while (len > 1) {
        const int part = (len + 31) / 32;
        const int at = lo + lane * part;
        const bool le = lane * part < len && __ldg(a.q_start + at) <= n;
        const unsigned bal = __ballot_sync(0xffffffffu, le);
        const int k = bal ? 31 - __clz(bal) : 0;
        const int end = lo + len;
        lo += k * part;
        len = min(part, end - lo);
    }
    return __ldg(a.q_start + lo) <= n && n < __ldg(a.q_start + lo + 1) ? lo : -1;
}

// The page of table entry j of sequence b; n_pages if there is none (a coordinate past the
// pool: TMA fills such rows with zeros).
__device__ __forceinline__ int page_of(const PagedArgs &a, int b, int j) {
    const int e = j < a.width ? __ldg(a.table + static_cast<int64_t>(b) * a.width + j) : -1;
    return static_cast<unsigned>(e) < static_cast<unsigned>(a.n_pages) ? e : a.n_pages;
}

}  // namespace swa
