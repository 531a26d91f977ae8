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
// Of a part: kOwn: positions are counted from `base` on.  kPrefix: a group, its rows' positions between p0 and
// `top`, its keys below `base`, its pages those of sequence `row`.
struct Seq {
    int q0, n, p0;
    bool ok;
    int base = 0, row = 0, top = 0;
};

template <Part PT = Part::kAll>
__device__ __forceinline__ Seq load_seq(const PagedArgs &a, int b) {
    Seq s;
    if constexpr (PT == Part::kPrefix) {
        const int4 *g = reinterpret_cast<const int4 *>(a.groups + b);
        const int4 x = __ldcg(g), y = __ldcg(g + 1);  // (written by the kernel before this one)
        s.q0 = x.x;
        s.n = x.y;
        s.p0 = x.z;
        s.ok = true;
        s.base = x.w;
        s.row = y.x;
        s.top = y.y;
        return s;
    }
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
    if constexpr (PT == Part::kOwn) {
        s.base = s.ok ? __ldcg(a.base + b) : 0;
        s.p0 -= s.base;
    }
    return s;
}

// The sinks among a part's positions.
template <Part PT>
__device__ __forceinline__ int sinks_of(const PagedArgs &a, int base) {
    return PT == Part::kOwn ? max(a.n_sink - base, 0) : a.n_sink;
}

// The sequence of token n, looked up by a whole warp: the last b with q_start[b] <= n (for a
// list that does not decrease); -1 if none has it.  Each step cuts the range 128-fold, by four loads
// a lane that are in flight together.
__device__ __forceinline__ int find_sequence(const PagedArgs &a, int n, int lane) {
    if (!a.q_start) return n < a.B ? n : -1;
    constexpr int kProbes = 4;
    int lo = 0, len = a.B;  // candidates lo .. lo + len - 1
    while (len > 1) {
        const int part = (len + 32 * kProbes - 1) / (32 * kProbes);
        bool le[kProbes];
#pragma unroll
        for (int i = 0; i < kProbes; ++i) {
            const int x = (i * 32 + lane) * part;
            le[i] = x < len && __ldg(a.q_start + lo + x) <= n;
        }
        int k = 0;
#pragma unroll
        for (int i = 0; i < kProbes; ++i) {
            const unsigned bal = __ballot_sync(0xffffffffu, le[i]);
            if (bal) k = i * 32 + 31 - __clz(bal);
        }
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

// Stores token n's keys and values in its page, by a whole warp.
__device__ __forceinline__ void store_token(const PagedArgs &a, int n, int lane, unsigned int *err) {
    const int b = find_sequence(a, n, lane);
    if (b < 0) return;
    const Seq s = load_seq(a, b);
    if (!s.ok) {
        if (lane == 0) atomicOr(err, SWA_DEVERR_BAD_POSITION);
        return;
    }
    const int p = s.p0 + (n - s.q0);
    const int page = page_of(a, b, p >> a.ps_log2);
    if (page >= a.n_pages) {
        if (lane == 0) atomicOr(err, SWA_DEVERR_BAD_PAGE);
        return;
    }
    if (!SWA_IN_BOUNDS(b < a.B && page >= 0 && p >= 0 && p >> a.ps_log2 < a.width, err)) return;
    const int64_t row = static_cast<int64_t>(page) * a.H_kv * a.ps + (p & (a.ps - 1));
    const int P = a.D / 8;  // 16-byte pieces of one head's row
    for (int x = lane; x < 2 * a.H_kv * P; x += 32) {
        const int pc = x % P, h = (x / P) % a.H_kv;
        const bool is_v = x >= a.H_kv * P;
        const uint16_t *src = is_v ? a.vn + static_cast<int64_t>(n) * a.vn_st[0] + h * a.vn_st[1]
                                   : a.kn + static_cast<int64_t>(n) * a.kn_st[0] + h * a.kn_st[1];
        uint16_t *dst = (is_v ? a.v_pages : a.k_pages) + (row + static_cast<int64_t>(h) * a.ps) * a.D;
        reinterpret_cast<uint4 *>(dst)[pc] = reinterpret_cast<const uint4 *>(src)[pc];
    }
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
//   Waves (tile kernel): whole units are dealt one a CTA in waves of alternating direction, so that
//   the CTAs work on neighbouring units, which read the same keys, at the same time: with a
//   stretch of the list for each CTA instead, their working sets together (1.1 MB each for the
//   Gemma-shape window) exceed L2 and every tile comes from HBM.
//   Tail: the tiles of the last units (between one and two waves of them, or all units of a
//   smaller batch) are cut into one stretch a CTA, of such lengths that every CTA ends up with the
//   mean number of tiles (one whose waves alone have more gets no stretch).  The pieces of a unit that crosses a
//   border are joined at the end, which takes as long as about kJoinTiles tiles (10 us); where
//   dealing every unit whole leaves no CTA further above the mean than that, there is no tail.
// ---------------------------------------------------------------------------------------------
struct UnitTiles {
    int sink, lo, n;  // tiles 0 .. sink - 1, then lo, lo + 1, ...: n in all
    __device__ __forceinline__ int tile(int j) const { return j < sink ? j : lo + (j - sink); }
};

template <int BN, Part PT = Part::kAll>
__device__ __forceinline__ UnitTiles unit_tiles(const PagedArgs &a, const Seq &s, int ut, int TT) {
    if constexpr (PT == Part::kPrefix) {  // (the same for every block of rows)
        UnitTiles u;
        u.lo = s.p0 >= a.window ? (s.p0 - a.window + 1) / BN : 0;
        u.sink = a.n_sink > 0 ? min(u.lo, (min(a.n_sink, s.base) + BN - 1) / BN) : 0;
        u.n = u.sink + (s.base - 1) / BN - u.lo + 1;
        return u;
    }
    const int n_sink = sinks_of<PT>(a, s.base);
    const int t0 = s.p0 + ut * TT, t1 = s.p0 + min(s.n, (ut + 1) * TT) - 1;
    UnitTiles u;
    u.lo = t0 >= a.window ? (t0 - a.window + 1) / BN : 0;
    u.sink = n_sink > 0 ? min(u.lo, (min(n_sink, t0 + 1) + BN - 1) / BN) : 0;
    u.n = u.sink + t1 / BN - u.lo + 1;
    return u;
}

// A CTA's share: `waves` whole units, then from tile j of unit (b, kvh, ut), tile `first` of the
// list, `left` tiles in list order; `tiles` in all.  turn: its number among the CTAs that have a
// stretch.  owner, pieces: the turn of the CTA that begins the unit of the first tile, and the
// CTAs that share it; open_pieces: those that share the unit of the last tile.
struct Share {
    long long first;
    int b, kvh, ut, j, left, waves, tiles, turn, owner, pieces, open_pieces;
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
template <int BN, Part PT = Part::kAll>
struct Walk {
    const PagedArgs *args;
    int TT, b, kvh, ut, j, left;
    Seq s;
    __device__ __forceinline__ Walk(const PagedArgs &a, int tt, const Share &sh)
        : args(&a), TT(tt), b(sh.b), kvh(sh.kvh), ut(sh.ut), j(sh.j), left(sh.left) {
        if (left > 0) s = load_seq<PT>(a, b);
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
                        s = load_seq<PT>(a, b);
                    } while (s.n == 0);
                }
            }
        }
        p.s = s;
        p.b = b;
        p.kvh = kvh;
        p.ut = ut;
        p.u = unit_tiles<BN, PT>(a, s, ut, TT);
        p.j0 = j;
        p.j1 = min(p.u.n, j + left);
        left -= p.j1 - p.j0;
        j = -1;
        return p.j1 > p.j0;
    }
};

// A CTA's pieces one by one, found by one warp: its whole units, one a wave, then its stretch of the
// list.  The sequences are searched 32 at a time from block b0, whose first unit is u0.
template <int BN, Part PT = Part::kAll>
struct Plan {
    const PagedArgs *args;
    int TT, waves, w, b0, u0;
    Walk<BN, PT> walk;
    __device__ __forceinline__ Plan(const PagedArgs &a, int tt, const Share &sh)
        : args(&a), TT(tt), waves(sh.waves), w(0), b0(0), u0(0), walk(a, tt, sh) {}
    __device__ __forceinline__ bool next(Piece &p, int lane) {
        const PagedArgs &a = *args;
        if (w >= waves) return walk.next(p);
        const int grid = static_cast<int>(gridDim.x), c = static_cast<int>(blockIdx.x);
        const int u = w * grid + (w & 1 ? grid - 1 - c : c);
        ++w;
        while (b0 < a.B) {
            Seq s{};
            if (b0 + lane < a.B) s = load_seq<PT>(a, b0 + lane);
            const int nu = (s.n + TT - 1) / TT, v = nu * a.H_kv;
            int inc = v;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int t = __shfl_up_sync(0xffffffffu, inc, o);
                if (lane >= o) inc += t;
            }
            const unsigned past = __ballot_sync(0xffffffffu, u0 + inc > u);
            if (past) {
                const int l = __ffs(past) - 1;
                const int rel = u - u0 - __shfl_sync(0xffffffffu, inc - v, l);
                const int units = max(__shfl_sync(0xffffffffu, nu, l), 1);
                p.b = b0 + l;
                p.kvh = rel / units;
                p.ut = rel % units;
                p.s = Seq{__shfl_sync(0xffffffffu, s.q0, l), __shfl_sync(0xffffffffu, s.n, l),
                          __shfl_sync(0xffffffffu, s.p0, l), true};
                if constexpr (PT != Part::kAll) p.s.base = __shfl_sync(0xffffffffu, s.base, l);
                if constexpr (PT == Part::kPrefix) {
                    p.s.row = __shfl_sync(0xffffffffu, s.row, l);
                    p.s.top = __shfl_sync(0xffffffffu, s.top, l);
                }
                p.u = unit_tiles<BN, PT>(a, p.s, p.ut, TT);
                p.j0 = 0;
                p.j1 = p.u.n;
                return true;
            }
            u0 += __shfl_sync(0xffffffffu, inc, 31);
            b0 += 32;
        }
        return false;  // (the last wave has no unit for this CTA)
    }
};

// Element (row, col) of the partial results of a slot of `rows` rows: 8 columns of a row together,
// then the same columns of the next row, so that a warp whose lanes have a row each stores whole
// lines.
template <int D>
__device__ __forceinline__ int64_t partial_at(int64_t slot, int rows, int row, int col) {
    return ((slot * (D / 8) + col / 8) * rows + row) * 8 + col % 8;
}
// The split kernel's slot of a piece (a CTA's turn is its index).
__device__ __forceinline__ int piece_slot(const Piece &p) {
    return 2 * static_cast<int>(blockIdx.x) + (p.begun() ? 0 : 1);
}

// Tile X of the list: tile j of unit (b, kvh, ut), which has n.
struct Place {
    int b, kvh, ut, j, n;
};
// Looked up by one warp; tiles: tiles of one kv head of each sequence.
template <int BN, Part PT = Part::kAll>
__device__ __forceinline__ Place find_tile(const PagedArgs &a, int TT, const long long *tiles, long long X, int lane) {
    Place r{0, 0, 0, 0, 1};
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
    const long long per = max(tiles[r.b], 1ll);
    r.kvh = static_cast<int>((X - before) / per);
    long long rel = X - before - r.kvh * per;
    const Seq s = load_seq<PT>(a, r.b);
    const int nu = (s.n + TT - 1) / TT;
    for (int u0 = 0; u0 < nu; u0 += 32) {
        const int v = u0 + lane < nu ? unit_tiles<BN, PT>(a, s, u0 + lane, TT).n : 0;
        long long inc = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long t = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += t;
        }
        const unsigned past = __ballot_sync(0xffffffffu, inc > rel);
        if (past) {
            const int l = __ffs(past) - 1;
            r.ut = u0 + l;
            r.j = static_cast<int>(rel - __shfl_sync(0xffffffffu, inc - v, l));
            r.n = __shfl_sync(0xffffffffu, v, l);
            break;
        }
        rel -= __shfl_sync(0xffffffffu, inc, 31);
    }
    return r;
}

constexpr int kMaxWaveCtas = 256;
constexpr int kJoinTiles = 12;
// (a prefix part's pieces are not joined by its kernel, and cost little more than to be written)
template <Part PT>
__device__ __forceinline__ constexpr int join_tiles() {
    return PT == Part::kPrefix ? 2 : kJoinTiles;
}
// Scratch of find_share: tiles [B] (64 bits), first units [B + 1], and with waves loads [2][CTAs].
__host__ __device__ constexpr int share_scratch(int B) { return B * 12 + 4; }
constexpr int kShareScratch = share_scratch(kPagedMaxB) + 2 * kMaxWaveCtas * 4;

// The CTA that unit u of the list goes to, in wave u / grid.
__device__ __forceinline__ int dealt_to(int u, int grid) {
    const int w = u / grid, c = u - w * grid;
    return w & 1 ? grid - 1 - c : c;
}

// Units of one kv head, counted in 64 bits, for a batch in which some sequence is broken (by one warp; out
// of line, which costs the others nothing).  Sequences that do not overlap have at most N / TT + B
// of them.  A q_start that goes down can give each of the others all rows, more work than any
// call has and more units than 32 bits count: then there is none.
static __device__ __noinline__ int units_of_broken(const PagedArgs &a, int TT, int lane) {
    long long n = 0;
    for (int b = lane; b < a.B; b += 32) n += (load_seq(a, b).n + TT - 1) / TT;
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
    return n <= static_cast<long long>(a.N / TT) + a.B ? static_cast<int>(n) : 0;
}

// This CTA's share, found by the whole block (kThreads threads; scratch in shared memory; block
// barriers inside, the result valid after the last).  min_tiles: without waves ahead of it the list is
// cut into stretches of at least that many tiles (but for the last), so that little work is not cut
// into pieces that cost more than they save.
template <int BN, int kThreads, bool kWaves, Part PT = Part::kAll>
__device__ __forceinline__ void find_share(const PagedArgs &a, int TT, int min_tiles, uint8_t *scratch, Share *out,
                                           unsigned int *err) {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, grid = static_cast<int>(gridDim.x);
    // 0. few sequences of a few units each, and no waves: one warp finds the share in registers (the
    // latency of a small batch; 2.3 us less than the general way for one sequence of one token)
    if (a.B <= 32) {
        constexpr int kFew = 4;
        bool found = false;
        if (warp == 0) {
            Seq s{};
            if (lane < a.B) {
                s = load_seq<PT>(a, lane);
                if (!s.ok && blockIdx.x == 0) atomicOr(err, SWA_DEVERR_BAD_POSITION);
            }
            const int nu = (s.n + TT - 1) / TT;
            const bool few = __all_sync(0xffffffffu, nu <= kFew && s.p0 + s.n < (1 << 24)) && a.H_kv <= 64 &&
                             (!kWaves || __reduce_add_sync(0xffffffffu, nu <= kFew ? nu : 0) * a.H_kv <= grid);
            if (few) {  // (32 sequences of 4 units of < 2^19 tiles of 64 heads: 32 bits hold every sum but one)
                int n[kFew], sum = 0;
#pragma unroll
                for (int ut = 0; ut < kFew; ++ut) {
                    n[ut] = ut < nu ? unit_tiles<BN, PT>(a, s, ut, TT).n : 0;
                    sum += n[ut];
                }
                long long inc = static_cast<long long>(sum) * a.H_kv;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const long long t = __shfl_up_sync(0xffffffffu, inc, o);
                    if (lane >= o) inc += t;
                }
                const long long total = __shfl_sync(0xffffffffu, inc, 31);
                const long long len = max((total + grid - 1) / grid, static_cast<long long>(min_tiles));
                const int c = static_cast<int>(blockIdx.x);
                const long long first = min(len * c, total);
                const int left = static_cast<int>(min(len, total - first));
                // tile X, in the lane of its sequence
                auto place = [&](long long X) -> Place {
                    const long long rel = X - (inc - static_cast<long long>(sum) * a.H_kv);
                    Place p{lane, static_cast<int>(rel / sum), 0, 0, n[0]};
                    p.j = static_cast<int>(rel - static_cast<long long>(p.kvh) * sum);
#pragma unroll
                    for (int ut = 0; ut < kFew - 1; ++ut)
                        if (p.ut == ut && p.j >= n[ut]) {
                            p.j -= n[ut];
                            ++p.ut;
                            p.n = n[ut + 1];
                        }
                    return p;
                };
                int longest = 0;
#pragma unroll
                for (int ut = 0; ut < kFew; ++ut) longest = max(longest, n[ut]);
                longest = __reduce_max_sync(0xffffffffu, longest);
                if (kWaves && longest <= len + join_tiles<PT>()) {  // unit c whole
                    int units = nu * a.H_kv;
#pragma unroll
                    for (int o = 1; o < 32; o <<= 1) {
                        const int t = __shfl_up_sync(0xffffffffu, units, o);
                        if (lane >= o) units += t;
                    }
                    const unsigned past = __ballot_sync(0xffffffffu, units > c);
                    if (past == 0) {
                        if (lane == 0) *out = Share{total, 0, 0, 0, 0, 0, 1, 0, 0, 0, 0, 0};
                    } else if (lane == __ffs(past) - 1) {
                        const int ut = (c - (units - nu * a.H_kv)) % nu;
                        int mine = n[0];
#pragma unroll
                        for (int i = 1; i < kFew; ++i) mine = ut == i ? n[i] : mine;
                        *out = Share{total, 0, 0, 0, 0, 0, 1, mine, 0, 0, 0, 0};
                    }
                } else if (left == 0) {
                    if (lane == 0) *out = Share{first, 0, 0, 0, 0, 0, 0, 0, c, 0, 0, 0};
                } else {
                    const int l0 = __ffs(__ballot_sync(0xffffffffu, inc > first)) - 1;
                    const int l1 = __ffs(__ballot_sync(0xffffffffu, inc > first + left - 1)) - 1;
                    if (lane == l0) {
                        const Place p = place(first);
                        const long long u0 = first - p.j;  // the unit's first tile
                        out->first = first;
                        out->b = p.b;
                        out->kvh = p.kvh;
                        out->ut = p.ut;
                        out->j = p.j;
                        out->left = out->tiles = left;
                        out->waves = 0;
                        out->turn = c;
                        out->owner = static_cast<int>(u0 / len);
                        out->pieces = static_cast<int>((u0 + p.n - 1) / len) - out->owner + 1;
                    }
                    if (lane == l1) {
                        const Place p = place(first + left - 1);
                        out->open_pieces = static_cast<int>((first + left - 1 - p.j + p.n - 1) / len) - c + 1;
                    }
                }
            }
            found = few;
        }
        if (__syncthreads_or(found)) return;
    }
    long long *tiles = reinterpret_cast<long long *>(scratch);
    int *units = reinterpret_cast<int *>(scratch + a.B * 8);
    int *all_loads = units + a.B + 1, *bulk_loads = all_loads + kMaxWaveCtas;
    // 1. units of one kv head of each sequence, 2. their running sum
    bool fine = true;
    for (int b = tid; b < a.B; b += kThreads) {
        const Seq s = load_seq<PT>(a, b);
        fine = fine && s.ok;
        if (!s.ok && blockIdx.x == 0) atomicOr(err, SWA_DEVERR_BAD_POSITION);
        units[b] = (s.n + TT - 1) / TT;
        tiles[b] = 0;
    }
    if (kWaves && grid <= kMaxWaveCtas)
        for (int c = tid; c < grid; c += kThreads) all_loads[c] = bulk_loads[c] = 0;
    fine = __syncthreads_and(fine);
    if (warp == 0) {
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
        if (!fine) before = units_of_broken(a, TT, lane);
        if (lane == 0) units[a.B] = before;
    }
    __syncthreads();
    // 3. tiles of every sequence, and those that each CTA gets if all units are dealt whole, or if
    // all but the last are: a thread per unit
    const int n_units = units[a.B];  // of one kv head
    const long long all_units = static_cast<long long>(n_units) * a.H_kv;
    const bool deal = kWaves && grid <= kMaxWaveCtas && all_units < (1 << 26);
    const int bulk_waves = deal ? max(0, static_cast<int>(all_units) / grid - 1) : 0;
    for (int x0 = warp * 32; x0 < n_units; x0 += kThreads) {
        const int x = x0 + lane;
        int b = 0, len = a.B;  // the last sequence whose first unit is <= x
        while (len > 1) {
            const int half = len >> 1;
            if (units[b + half] <= x) {
                b += half;
                len -= half;
            } else {
                len = half;
            }
        }
        const bool in = x < n_units;
        int n = 0;
        if (in) {
            const Seq s = load_seq<PT>(a, b);
            const int ut = x - units[b];
            n = unit_tiles<BN, PT>(a, s, ut, TT).n;
            if (deal) {
                const int nu = (s.n + TT - 1) / TT;
                for (int h = 0, u = units[b] * a.H_kv + ut; h < a.H_kv; ++h, u += nu) {
                    const int c = dealt_to(u, grid);
                    atomicAdd(all_loads + c, n);
                    if (u < bulk_waves * grid) atomicAdd(bulk_loads + c, n);
                }
            }
        }
        // (lanes of one sequence add up first)
        const int b_first = __shfl_sync(0xffffffffu, b, 0);
        if (__all_sync(0xffffffffu, !in || b == b_first)) {
            long long sum = n;
#pragma unroll
            for (int o = 16; o >= 1; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            if (lane == 0) atomicAdd(reinterpret_cast<unsigned long long *>(tiles + b), static_cast<unsigned long long>(sum));
        } else if (in) {
            atomicAdd(reinterpret_cast<unsigned long long *>(tiles + b), static_cast<unsigned long long>(n));
        }
    }
    __syncthreads();
    // 4. this CTA's stretch of the list, by warp 0 with its first tile, by warp 1 with its last
    if (warp < 2) {
        long long all = 0;
        for (int b = lane; b < a.B; b += 32) all += tiles[b];
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) all += __shfl_xor_sync(0xffffffffu, all, o);
        const long long total = all * a.H_kv;
        const int c = static_cast<int>(blockIdx.x);
        constexpr int kPer = kMaxWaveCtas / 32;
        long long first, len, begin[kPer];  // begin, q: the stretch of CTA 32 * i + lane (waves > 0)
        int q[kPer], mine = 0, turn = c, waves = bulk_waves;
        if (deal) {  // all units whole?
            int top = 0;
            for (int i = lane; i < grid; i += 32) top = max(top, all_loads[i]);
            top = __reduce_max_sync(0xffffffffu, top);
            if (top <= max((total + grid - 1) / grid, static_cast<long long>(min_tiles)) + join_tiles<PT>()) {
                if (warp == 0 && lane == 0)
                    *out = Share{total, 0, 0, 0, 0, 0, static_cast<int>((all_units + grid - 1) / grid), all_loads[c],
                                 0, 0, 0, 0};
                waves = -1;
            }
        }
        const int *loads = bulk_loads;
        if (waves < 0) {
            first = total;
            len = 0;
        } else if (waves == 0) {
            len = max((total + grid - 1) / grid, static_cast<long long>(min_tiles));
            first = len * c;
        } else {
            // the tail fills the CTAs up to the mean; one whose waves alone are above it gets nothing
            int ld[kPer];
            long long bulk = 0;
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                ld[i] = 32 * i + lane < grid ? loads[32 * i + lane] : INT_MAX;
                if (32 * i + lane < grid) bulk += ld[i];
            }
#pragma unroll
            for (int o = 16; o >= 1; o >>= 1) bulk += __shfl_xor_sync(0xffffffffu, bulk, o);
            const int level = static_cast<int>((total + grid - 1) / grid);
            long long at = bulk;
            first = len = 0;
            turn = 0;
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                const int want = ld[i] < level ? level - ld[i] : 0;
                long long inc = want;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const long long t = __shfl_up_sync(0xffffffffu, inc, o);
                    if (lane >= o) inc += t;
                }
                begin[i] = at + inc - want;
                q[i] = static_cast<int>(max(min(static_cast<long long>(want), total - begin[i]), 0ll));
                turn += __popc(__ballot_sync(0xffffffffu, q[i] > 0 && 32 * i + lane < c));
                if (i == c / 32) {
                    first = __shfl_sync(0xffffffffu, begin[i], c % 32);
                    len = __shfl_sync(0xffffffffu, q[i], c % 32);
                    mine = __shfl_sync(0xffffffffu, ld[i], c % 32);
                }
                at += __shfl_sync(0xffffffffu, inc, 31);
            }
        }
        first = min(first, total);
        const int left = static_cast<int>(min(len, total - first));
        // the turn of the CTA that has tile X of the tail, and the CTAs that have some of [X, Y)
        auto turn_of = [&](long long X) -> int {
            if (waves == 0) return static_cast<int>(X / len);
            int n = 0;
#pragma unroll
            for (int i = 0; i < kPer; ++i) n += __popc(__ballot_sync(0xffffffffu, q[i] > 0 && begin[i] + q[i] <= X));
            return n;
        };
        if (warp == 0 && waves >= 0) {
            Share sh{first, 0, 0, 0, 0, left, waves, mine + left, turn, 0, 0, 0};
            if (left > 0) {
                const Place p = find_tile<BN, PT>(a, TT, tiles, first, lane);
                sh.b = p.b;
                sh.kvh = p.kvh;
                sh.ut = p.ut;
                sh.j = p.j;
                if (kWaves) {
                    sh.owner = turn_of(first - p.j);
                    sh.pieces = turn_of(first - p.j + p.n - 1) - sh.owner + 1;
                }
            }
            if (lane == 0) {  // (open_pieces is warp 1's)
                out->first = sh.first;
                out->b = sh.b;
                out->kvh = sh.kvh;
                out->ut = sh.ut;
                out->j = sh.j;
                out->left = sh.left;
                out->waves = sh.waves;
                out->tiles = sh.tiles;
                out->turn = sh.turn;
                out->owner = sh.owner;
                out->pieces = sh.pieces;
            }
        } else if (kWaves && warp == 1 && left > 0) {
            const long long X = first + left - 1;
            const Place p = find_tile<BN, PT>(a, TT, tiles, X, lane);
            const int n = turn_of(X - p.j + p.n - 1) - turn + 1;
            if (lane == 0) out->open_pieces = n;
        }
    }
    __syncthreads();
}

}  // namespace swa
