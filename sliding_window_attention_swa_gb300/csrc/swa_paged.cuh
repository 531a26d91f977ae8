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

// Keys that the query at position t keeps.
__device__ __forceinline__ int kept_keys(const PagedArgs &a, int t) {
    const int behind = t >= a.window ? t - a.window + 1 : 0;  // positions behind the window
    return t + 1 - behind + min(behind, a.n_sink);
}

// ---------------------------------------------------------------------------------------------
// Work: a unit is (sequence, kv head, block of TT new tokens); it reads the tiles of BN keys
// that its tokens can reach -- those of the sinks, then those of the window -- as one list of
// n_tiles.  Lengths are only known on the device, so the work is shared out there: all units'
// tiles, in the order (sequence, kv head, block), form one list, and CTA c takes the tiles
// c * R .. (c + 1) * R - 1 of it.  Every CTA thus has the same number of tiles whatever the
// batch looks like; a unit that crosses a border is finished by a merge of its pieces.
// ---------------------------------------------------------------------------------------------
struct UnitTiles {
    int sink, lo, n;  // tiles 0 .. sink - 1, then lo, lo + 1, ...: n in all
    __device__ __forceinline__ int tile(int j) const { return j < sink ? j : lo + (j - sink); }
};

template <int BN>
__device__ __forceinline__ UnitTiles unit_tiles(const PagedArgs &a, const Seq &s, int ut, int TT) {
    const int t0 = s.p0 + ut * TT, t1 = s.p0 + min(s.n, (ut + 1) * TT) - 1;
    UnitTiles u;
    u.lo = t0 >= a.window ? (t0 - a.window + 1) / BN : 0;
    u.sink = a.n_sink > 0 ? min(u.lo, (min(a.n_sink, t0 + 1) + BN - 1) / BN) : 0;
    u.n = u.sink + t1 / BN - u.lo + 1;
    return u;
}

// A CTA's share: from tile j of unit (b, kvh, ut), `left` tiles in list order.
struct Share {
    int b, kvh, ut, j, left, R;
};

// One unit's part of a CTA's share: tiles j0 .. j1 - 1.
struct Piece {
    Seq s;
    UnitTiles u;
    int b, kvh, ut, j0, j1;
    __device__ __forceinline__ bool begun() const { return j0 > 0; }   // an earlier CTA has its first tiles
    __device__ __forceinline__ bool open() const { return j1 < u.n; }  // a later CTA has its last tiles
};

// Walks a share piece by piece; every role of a CTA walks it alike.
template <int BN>
struct Walk {
    const PagedArgs *args;
    int TT, b, kvh, ut, j, left;
    Seq s;
    __device__ __forceinline__ Walk(const PagedArgs &a, int tt, const Share &sh)
        : args(&a), TT(tt), b(sh.b), kvh(sh.kvh), ut(sh.ut), j(sh.j), left(sh.left) {
        if (left > 0) s = load_seq(a, b);
    }
    __device__ __forceinline__ bool next(Piece &p) {
        const PagedArgs &a = *args;
        if (left <= 0) return false;
        if (j < 0) {  // the unit after the last piece's
            j = 0;
            if ((++ut) * TT >= s.n) {
                ut = 0;
                if (++kvh >= a.H_kv) {
                    kvh = 0;
                    do {
                        if (++b >= a.B) {
                            left = 0;
                            return false;
                        }
                        s = load_seq(a, b);
                    } while (s.n == 0);
                }
            }
        }
        p.s = s;
        p.b = b;
        p.kvh = kvh;
        p.ut = ut;
        p.u = unit_tiles<BN>(a, s, ut, TT);
        p.j0 = j;
        p.j1 = min(p.u.n, j + left);
        left -= p.j1 - p.j0;
        j = -1;
        return p.j1 > p.j0;
    }
};

// A walk kept in shared memory, one per warp: warps whose registers are taken by their tiles read
// what they need of the current piece from here.
struct WalkState {
    int b, kvh, ut, j, left, q0, n, p0;  // the walk
    int sink, lo, nt, j0, j1;            // the piece (its unit is (b, kvh, ut) of the walk)
    __device__ __forceinline__ int tile(int i) const volatile { return j0 + i < sink ? j0 + i : lo + (j0 + i - sink); }
    __device__ __forceinline__ bool begun() const volatile { return j0 > 0; }
    __device__ __forceinline__ bool open() const volatile { return j1 < nt; }
};
// The warp's next piece (all lanes take part); the first call starts the share.
template <int BN>
__device__ __forceinline__ bool walk_step(const PagedArgs &a, int TT, const volatile Share *sh, bool first,
                                          volatile WalkState *w) {
    Walk<BN> walk(a, TT, Share{0, 0, 0, 0, 0, 0});
    if (first) {
        walk = Walk<BN>(a, TT, Share{sh->b, sh->kvh, sh->ut, sh->j, sh->left, 0});
    } else {
        walk.b = w->b;
        walk.kvh = w->kvh;
        walk.ut = w->ut;
        walk.j = w->j;
        walk.left = w->left;
        walk.s = Seq{w->q0, w->n, w->p0, true};
    }
    __syncwarp();
    Piece p;
    const bool more = walk.next(p);
    if (more && (threadIdx.x & 31) == 0) {
        w->b = walk.b;
        w->kvh = walk.kvh;
        w->ut = walk.ut;
        w->j = walk.j;
        w->left = walk.left;
        w->q0 = walk.s.q0;
        w->n = walk.s.n;
        w->p0 = walk.s.p0;
        w->sink = p.u.sink;
        w->lo = p.u.lo;
        w->nt = p.u.n;
        w->j0 = p.j0;
        w->j1 = p.j1;
    }
    __syncwarp();
    return more;
}

__device__ __forceinline__ int piece_slot(const Piece &p) { return 2 * static_cast<int>(blockIdx.x) + (p.begun() ? 0 : 1); }
__device__ __forceinline__ int4 open_record(const Piece &p, int R) {
    return make_int4(1 + (p.u.n - p.j1 + R - 1) / R, p.b, p.kvh, p.ut);
}

// This CTA's share, found by the whole block (kThreads threads; tiles: scratch for B sums in
// shared memory; two block barriers inside, the result valid after the last).  min_tiles: no
// CTA gets fewer, so that short work is not cut into pieces that cost more than they save.
template <int BN, int kThreads>
__device__ __forceinline__ void find_share(const PagedArgs &a, int TT, int min_tiles, long long *tiles,
                                           Share *out, unsigned int *err) {
    constexpr int kSerial = 4;  // units of a sequence that one thread counts
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    // tiles of each sequence (one kv head): by one thread where there are few units
    for (int b0 = warp * 32; b0 < a.B; b0 += kThreads) {
        const int b = b0 + lane;
        Seq s{};
        if (b < a.B) {
            s = load_seq(a, b);
            if (!s.ok && blockIdx.x == 0) atomicOr(err, SWA_DEVERR_BAD_POSITION);
        }
        const int nu = (s.n + TT - 1) / TT;
        long long sum = 0;
        if (nu <= kSerial)
            for (int ut = 0; ut < nu; ++ut) sum += unit_tiles<BN>(a, s, ut, TT).n;
        unsigned many = __ballot_sync(0xffffffffu, nu > kSerial);
        while (many) {  // ... by the warp's lanes where there are many
            const int l = __ffs(many) - 1;
            many &= many - 1;
            Seq t;
            t.n = __shfl_sync(0xffffffffu, s.n, l);
            t.p0 = __shfl_sync(0xffffffffu, s.p0, l);
            long long part = 0;
            for (int ut = lane; ut * static_cast<long long>(TT) < t.n; ut += 32) part += unit_tiles<BN>(a, t, ut, TT).n;
#pragma unroll
            for (int o = 16; o >= 1; o >>= 1) part += __shfl_xor_sync(0xffffffffu, part, o);
            if (lane == l) sum = part;
        }
        if (b < a.B) tiles[b] = sum;
    }
    __syncthreads();
    if (warp == 0) {
        long long all = 0;
        for (int b = lane; b < a.B; b += 32) all += tiles[b];
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) all += __shfl_xor_sync(0xffffffffu, all, o);
        const long long total = all * a.H_kv, grid = gridDim.x;
        const long long R = max((total + grid - 1) / grid, static_cast<long long>(min_tiles));
        const long long X = R * blockIdx.x;
        Share sh{0, 0, 0, 0, 0, 0};
        if (X < total) {
            sh.R = static_cast<int>(min(R, static_cast<long long>(INT_MAX)));
            sh.left = static_cast<int>(min(static_cast<long long>(sh.R), total - X));
            // the sequence that has tile X
            long long before = 0;
            int b0 = 0;
            while (true) {
                const long long v = b0 + lane < a.B ? tiles[b0 + lane] * a.H_kv : 0;
                long long inc = v;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const long long t = __shfl_up_sync(0xffffffffu, inc, o);
                    if (lane >= o) inc += t;
                }
                const unsigned past = __ballot_sync(0xffffffffu, before + inc > X);
                if (past) {
                    const int l = __ffs(past) - 1;
                    before += __shfl_sync(0xffffffffu, inc - v, l);
                    sh.b = b0 + l;
                    break;
                }
                before += __shfl_sync(0xffffffffu, inc, 31);
                b0 += 32;
                if (b0 >= a.B) break;  // (cannot be: X < total)
            }
            const long long per = max(tiles[sh.b], 1ll), rel = X - before;
            sh.kvh = static_cast<int>(rel / per);
            // the block of tokens that has tile rel % per of its kv head
            const Seq s = load_seq(a, sh.b);
            long long r = rel % per;
            const int nu = (s.n + TT - 1) / TT;
            for (int u0 = 0; u0 < nu; u0 += 32) {
                const int v = u0 + lane < nu ? unit_tiles<BN>(a, s, u0 + lane, TT).n : 0;
                long long inc = v;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const long long t = __shfl_up_sync(0xffffffffu, inc, o);
                    if (lane >= o) inc += t;
                }
                const unsigned past = __ballot_sync(0xffffffffu, inc > r);
                if (past) {
                    const int l = __ffs(past) - 1;
                    sh.ut = u0 + l;
                    sh.j = static_cast<int>(r - __shfl_sync(0xffffffffu, inc - v, l));
                    break;
                }
                r -= __shfl_sync(0xffffffffu, inc, 31);
            }
        }
        if (lane == 0) *out = sh;
    }
    __syncthreads();
}

}  // namespace swa
