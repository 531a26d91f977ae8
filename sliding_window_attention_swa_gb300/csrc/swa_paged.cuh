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
// n tiles.  Lengths are only known on the device, so the work is shared out there.  All units,
// in the order (sequence, kv head, block), and their tiles form one list.
//   Waves (tile kernel, from two units a CTA): whole units are dealt one a CTA in waves of
//   alternating direction, so that the CTAs work on neighbouring units, which read the same
//   keys, at the same time: with a stretch of the list for each CTA instead, their working sets
//   together (1.1 MB each for the Gemma-shape window) exceed L2 and every tile comes from HBM.
//   Tail: the tiles of the last units (between one and two waves of them, or all units of a
//   smaller batch) are cut into one stretch a CTA, of such lengths that all CTAs end up with the
//   same number of tiles, whatever the batch looks like.  A unit that crosses a border is
//   finished by a merge of its pieces.
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

// A CTA's share: `waves` whole units, then from tile j of unit (b, kvh, ut) `left` tiles in list
// order; `tiles` in all.  span: CTAs from this one to the one that has the last tile of the unit
// that this CTA's last tile belongs to (1: this one).
struct Share {
    int b, kvh, ut, j, left, waves, tiles, span;
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

__device__ __forceinline__ int piece_slot(const Piece &p) { return 2 * static_cast<int>(blockIdx.x) + (p.begun() ? 0 : 1); }

// Where a tile of the list lies: tile j of unit (b, kvh, ut), whose n tiles start at `at`.
struct Place {
    int b, kvh, ut, j, n;
    long long at;
};
// Looks up tile X (within the list) with one warp; tiles: tiles of one kv head of each sequence.
template <int BN>
__device__ __forceinline__ Place find_place(const PagedArgs &a, int TT, const long long *tiles, long long X, int lane) {
    Place r{0, 0, 0, 0, 0, 0};
    long long before = 0;
    for (int b0 = 0; b0 < a.B; b0 += 32) {
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
            r.b = b0 + l;
            break;
        }
        before += __shfl_sync(0xffffffffu, inc, 31);
    }
    const long long per = max(tiles[r.b], 1ll), rel = X - before;
    r.kvh = static_cast<int>(rel / per);
    r.at = before + r.kvh * per;
    const Seq s = load_seq(a, r.b);
    const int nu = (s.n + TT - 1) / TT;
    for (int u0 = 0; u0 < nu; u0 += 32) {
        const int v = u0 + lane < nu ? unit_tiles<BN>(a, s, u0 + lane, TT).n : 0;
        long long inc = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long t = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += t;
        }
        const unsigned past = __ballot_sync(0xffffffffu, r.at + inc > X);
        if (past) {
            const int l = __ffs(past) - 1;
            r.at += __shfl_sync(0xffffffffu, inc - v, l);
            r.ut = u0 + l;
            r.n = __shfl_sync(0xffffffffu, v, l);
            break;
        }
        r.at += __shfl_sync(0xffffffffu, inc, 31);
    }
    r.j = static_cast<int>(X - r.at);
    return r;
}

constexpr int kMaxWaveCtas = 256;
// Scratch of find_share: tiles [B] (64 bits), units [B], loads [CTAs].
constexpr int kShareScratch = kPagedMaxB * 12 + kMaxWaveCtas * 4;

// Unit u of the list goes to this CTA in wave u / grid.
__device__ __forceinline__ int dealt_to(int u, int grid) {
    const int w = u / grid, c = u - w * grid;
    return w & 1 ? grid - 1 - c : c;
}

// This CTA's share, found by the whole block (kThreads threads; scratch in shared memory; block
// barriers inside, the result valid after the last).  min_tiles: no stretch of the tail is
// shorter, so that little work is not cut into pieces that cost more than they save.
template <int BN, int kThreads, bool kWaves>
__device__ __forceinline__ void find_share(const PagedArgs &a, int TT, int min_tiles, uint8_t *scratch, Share *out,
                                           unsigned int *err) {
    constexpr int kSerial = 4;  // units of a sequence that one thread counts
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, grid = static_cast<int>(gridDim.x);
    long long *tiles = reinterpret_cast<long long *>(scratch);
    int *units = reinterpret_cast<int *>(scratch + a.B * 8), *loads = units + a.B;
    // visit(b, s, ut) for every unit of one kv head: by one thread for a sequence of few units, by
    // the warp's lanes for one of many; done(b, nu) for every sequence afterwards
    auto for_units = [&](auto visit, auto done) {
        for (int b0 = warp * 32; b0 < a.B; b0 += kThreads) {
            const int b = b0 + lane;
            Seq s{};
            if (b < a.B) s = load_seq(a, b);
            const int nu = (s.n + TT - 1) / TT;
            if (nu <= kSerial)
                for (int ut = 0; ut < nu; ++ut) visit(b, s, ut);
            unsigned many = __ballot_sync(0xffffffffu, nu > kSerial);
            while (many) {
                const int l = __ffs(many) - 1;
                many &= many - 1;
                Seq t{0, __shfl_sync(0xffffffffu, s.n, l), __shfl_sync(0xffffffffu, s.p0, l), true};
                for (int ut = lane; ut < (t.n + TT - 1) / TT; ut += 32) visit(b0 + l, t, ut);
            }
            if (b < a.B) done(b, s, nu);
        }
    };
    for (int b = tid; b < a.B; b += kThreads) tiles[b] = 0;
    __syncthreads();
    for_units(
        [&](int b, const Seq &s, int ut) {
            atomicAdd(reinterpret_cast<unsigned long long *>(tiles + b),
                      static_cast<unsigned long long>(unit_tiles<BN>(a, s, ut, TT).n));
        },
        [&](int b, const Seq &s, int nu) {
            if (!s.ok && blockIdx.x == 0) atomicOr(err, SWA_DEVERR_BAD_POSITION);
            if (kWaves) units[b] = nu * a.H_kv;
        });
    __syncthreads();
    int waves = 0;
    if constexpr (kWaves) {
        if (warp == 0) {  // first unit of each sequence
            int before = 0;
            for (int b0 = 0; b0 < a.B; b0 += 32) {
                const int v = b0 + lane < a.B ? units[b0 + lane] : 0;
                int inc = v;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int t = __shfl_up_sync(0xffffffffu, inc, o);
                    if (lane >= o) inc += t;
                }
                if (b0 + lane < a.B) units[b0 + lane] = before + inc - v;
                before += __shfl_sync(0xffffffffu, inc, 31);
            }
            if (lane == 0) out->waves = grid <= kMaxWaveCtas ? max(0, before / grid - 1) : 0;
        }
        __syncthreads();
        waves = out->waves;
        if (waves > 0) {  // tiles that the waves give each CTA
            for (int c = tid; c < grid; c += kThreads) loads[c] = 0;
            __syncthreads();
            const int bulk = waves * grid;
            for_units(
                [&](int b, const Seq &s, int ut) {
                    const int nu = (s.n + TT - 1) / TT, n = unit_tiles<BN>(a, s, ut, TT).n;
                    for (int h = 0, u = units[b] + ut; h < a.H_kv && u < bulk; ++h, u += nu)
                        atomicAdd(loads + dealt_to(u, grid), n);
                },
                [](int, const Seq &, int) {});
            __syncthreads();
        }
    }
    if (warp == 0) {
        long long all = 0;
        for (int b = lane; b < a.B; b += 32) all += tiles[b];
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) all += __shfl_xor_sync(0xffffffffu, all, o);
        const long long total = all * a.H_kv;
        const int c = static_cast<int>(blockIdx.x);
        long long X, len, R = 0;    // this CTA's stretch of the list
        int mine = 0;               // tiles from the waves
        constexpr int kPer = kMaxWaveCtas / 32;
        long long first[kPer];      // start of the stretch of CTA 32 * i + lane
        if (waves == 0) {
            R = max((total + grid - 1) / grid, static_cast<long long>(min_tiles));
            X = R * c;
            len = R;
        } else {
            // the level to which the tail fills the CTAs up: the least at which it all fits
            int ld[kPer];
            int top = 0;
            long long bulk_tiles = 0;
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                const int ci = 32 * i + lane;
                ld[i] = ci < grid ? loads[ci] : INT_MAX;
                if (ci < grid) {
                    bulk_tiles += ld[i];
                    top = max(top, ld[i]);
                }
            }
#pragma unroll
            for (int o = 16; o >= 1; o >>= 1) {
                bulk_tiles += __shfl_xor_sync(0xffffffffu, bulk_tiles, o);
                top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
            }
            const long long tail = total - bulk_tiles;
            long long lo = 0, hi = top + (tail + grid - 1) / grid;
            while (lo < hi) {
                const long long mid = (lo + hi) >> 1;
                long long room = 0;
#pragma unroll
                for (int i = 0; i < kPer; ++i) room += ld[i] < mid ? mid - ld[i] : 0;
#pragma unroll
                for (int o = 16; o >= 1; o >>= 1) room += __shfl_xor_sync(0xffffffffu, room, o);
                if (room >= tail) hi = mid;
                else lo = mid + 1;
            }
            long long at = bulk_tiles;
            X = len = 0;
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                const long long q = ld[i] < lo ? lo - ld[i] : 0;
                long long inc = q;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const long long t = __shfl_up_sync(0xffffffffu, inc, o);
                    if (lane >= o) inc += t;
                }
                first[i] = at + inc - q;
                if (i == c / 32) {
                    X = __shfl_sync(0xffffffffu, first[i], c % 32);
                    len = __shfl_sync(0xffffffffu, q, c % 32);
                    mine = __shfl_sync(0xffffffffu, ld[i], c % 32);
                }
                at += __shfl_sync(0xffffffffu, inc, 31);
            }
        }
        Share sh{0, 0, 0, 0, 0, waves, mine, 1};
        len = min(len, total - X);
        if (len > 0) {
            const Place p = find_place<BN>(a, TT, tiles, X, lane), q = find_place<BN>(a, TT, tiles, X + len - 1, lane);
            sh.b = p.b;
            sh.kvh = p.kvh;
            sh.ut = p.ut;
            sh.j = p.j;
            sh.left = static_cast<int>(len);
            sh.tiles += sh.left;
            const long long end = q.at + q.n;  // of the unit of the last tile
            if (waves == 0) {
                sh.span = 1 + static_cast<int>((end - X - len + R - 1) / R);
            } else {
#pragma unroll
                for (int i = 0; i < kPer; ++i) {
                    const int ci = 32 * i + lane;
                    sh.span += __popc(__ballot_sync(0xffffffffu, ci > c && ci < grid && first[i] < end));
                }
            }
        }
        if (lane == 0) *out = sh;
    }
    __syncthreads();
}

}  // namespace swa
