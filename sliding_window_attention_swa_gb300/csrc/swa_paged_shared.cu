// swa_paged_shared.cu -- attention of sequences that share leading pages: each group's prefix is read
// once for the new tokens of all its sequences.
//
// A row's softmax over its keys is that over any two parts of them, joined by their maxima:
//   1. plan (here): finds for every group how many leading positions its sequences share, and lists the
//      stretches that the kernel for few rows takes.
//   2. prefix part: the group's packed rows, of all its sequences, over the shared positions: tiles of the tensor
//      cores (paged_tile_kernel, kPrefix), or, where a group has at most 16 rows, stretches.
//   3. own part: each sequence over the positions behind those: stretches (paged_rows_kernel), or, where a
//      sequence has more than 16 rows, tiles again (paged_tile_kernel, kOwn).
//   4. join (here): the partial results of every row, all of them in fp32, are joined and rounded once.
// The kernels follow one another by programmatic dependence: the own part's blocks start where the
// prefix part's have ended, without waiting for all of them.
// With single tokens a group of R sequences reads its prefix once instead of R times, and its products go to
// the tensor cores in tiles of 128 rows instead of 16.
#include <algorithm>
#include <climits>
#include <cmath>
#include <type_traits>

#include <cooperative_groups.h>

#include "swa_paged_shared.cuh"

namespace swa {
namespace {

namespace cg = cooperative_groups;

__device__ unsigned int g_shared_err = 0;

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kFewGroups = 32;  // below it a cluster plans a group, else a block
constexpr int kCluster = 8;
// Entries that a warp compares at a time: sixteen loads a lane and row in flight.
constexpr int kWords = 16, kChunk = 32 * kWords;

// Shared positions below which a group is computed as none: a part of its own costs more than they do (64 sequences of
// 32 heads of 128, 200 tokens of their own: up to 128 shared positions 24.6 us, 22.6 without the part, up to 256 in groups of
// four 24.6 against 28.7, in groups of 64 28.7 against 33).  It is a limit against this call without the part, for many
// sequences: swa_paged_attend is faster for few (four behind 900 positions: 15.5 us, 20.6 shared).
constexpr int kLeastShared = 192;
// With many new tokens a sequence the prefix part saves what its tiles of rows are fewer than the sequences' own, and its
// parts are written and joined again. Below this many positions saved per own tile that costs more (12 sequences of 16
// tokens, 6 tiles for 12, 32 heads of 128 on 8: 6000 shared positions 60 us, 56 as none; 24000 94 against 148; 48
// sequences of 80 tokens, 120 tiles for 144: 1024 positions 222 us, 146 as none; 12 such, 24000: 304 against 361; 48 of 4
// tokens, 6 tiles for 48: 1024 positions 60 against 57, 6000 76 against 135). Measured there alone: 57 sequences of up
// to three tokens in three groups, 16 heads on one, behind 9000 are above it, and take 62 us (swa_paged_attend 41). The build that checks indices shares
// wherever there is anything to save: its tests are to reach every part.
#ifdef SWA_DEBUG
constexpr int kLeastSaved = 1;
#else
constexpr int kLeastSaved = 3500;
#endif
constexpr int kMostPlanes = 129;  // of a part in stretches
constexpr int kTileRows = 128;  // rows of a query tile of the many-row kernel
// Of the join of units, for an SM (two at a time; 22 chunks of up to 16 tokens: 72 us, 75 with two, 72 with eight).
constexpr int kJoinBlocks = 4;

// Of a group's sequences that have new tokens.
struct Members {
    unsigned long long least;  // least p0, and the first sequence with it: p0 << 13 | (b - b0)
    unsigned long long next;   // the second least
    int top, count, tiles, broken;
    long long tokens;
};
static_assert(kPagedMaxB <= 1 << 13, "the first sequence's number");

__device__ __forceinline__ Members join(const Members &x, const Members &y) {
    return Members{min(x.least, y.least),
                   min(max(x.least, y.least), min(x.next, y.next)),
                   max(x.top, y.top),
                   x.count + y.count,
                   x.tiles + y.tiles,
                   x.broken | y.broken,
                   x.tokens + y.tokens};
}
__device__ __forceinline__ Members shuffled(const Members &x, int o) {
    return Members{__shfl_xor_sync(0xffffffffu, x.least, o), __shfl_xor_sync(0xffffffffu, x.next, o),
                   __shfl_xor_sync(0xffffffffu, x.top, o),
                   __shfl_xor_sync(0xffffffffu, x.count, o), __shfl_xor_sync(0xffffffffu, x.tiles, o),
                   __shfl_xor_sync(0xffffffffu, x.broken, o), __shfl_xor_sync(0xffffffffu, x.tokens, o)};
}

// ---------------------------------------------------------------------------------------------
// plan: a cluster (of one block where there are many groups) per group.
// The group's pages are those of the sequence with the least p0, which needs every page below p0 that any
// of the others needs (its window starts first).  A position is shared if it lies below that p0 and every
// sequence has the same entry there, or has no use for it (behind its window and no sink), and all the
// positions before it that matter are shared, too.  So the result does not rest on what the caller
// says of the tables: a group that shares nothing is computed as if it were none.
// Bound by latency: the list, the sequences' lengths, then the table's rows, all of them once, then the lists: 64
// sequences of 512 shared entries 6.8 us, 31 groups 9.
// ---------------------------------------------------------------------------------------------
// Puts the stretches of a warp's units on the list: `lanes` lanes have a unit, `count` stretches of keys k; t.first: of
// the first plane.  (Tokens in planes are counted in 32 bits: each has 256 bytes at least.)
__device__ __forceinline__ void list_stretches(const SharedArgs &sa, const Keys &k, int count, Stretch t, int lanes) {
    const int lane = threadIdx.x & 31, sub = lane & (lanes - 1);
    const int mine = sub == 0 ? count : 0;
    int inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += x;
    }
    int at = 0;
    if (lane == 31 && inc > 0) at = atomicAdd(sa.counts + (t.part ? kPrefixStretches : kOwnStretches), inc);
    const PartResults &part = t.part ? sa.few_prefix : sa.part[0];
    const int first = t.first;
    at = __shfl_sync(0xffffffffu, at, 31) + __shfl_sync(0xffffffffu, inc - mine, lane - sub);
    for (int i = sub; i < count; i += lanes) {
        // (no list has more than there is room for: the units' sequences have no row in common)
        if (at + i >= (t.part ? sa.prefix_cap : sa.own_cap)) {
            atomicOr(&g_shared_err, SWA_DEVERR_BAD_POSITION);
            break;
        }
        t.k0 = k.begin(i);
        t.k1 = k.close(i);
        t.first = first + (i < k.count ? i : part.planes - 1) * part.tokens;
        int4 *dst = reinterpret_cast<int4 *>(sa.stretches + (t.part ? 0 : sa.prefix_cap) + at + i);
        dst[0] = make_int4(t.row, t.q0, t.n, t.first);
        dst[1] = make_int4(t.k0, t.k1, t.part, 0);
    }
}

// Whether another sequence has rows of sequence b (s), too, as a q_start that goes down can make it.
__device__ __forceinline__ bool rows_in_common(const PagedArgs &a, const Seq &s, int b) {
    for (int c = 0; c < a.B; ++c) {
        const Seq t = load_seq(a, c);
        if (c != b && in_common(s, t)) return true;
    }
    return false;
}

// What the other kernels need to know of sequences b0 .. b1 - 1 (of group g), by `warps` warps, of which this is
// number w; a warp has as many sequences at a time as leave none to another turn, 32 at most.
// kOrdered: q_start does not go down.
template <bool kOrdered>
__device__ __forceinline__ void put_sequences(const SharedArgs &sa, int b0, int b1, const PagedGroup &group, int g, int w,
                                              int warps) {
    const PagedArgs &a = sa.a;
    const int TT = few_tokens(a.G), base = group.end;
    int each = 1;
    while (each < 32 && each * warps < b1 - b0) each *= 2;
    const int lane = threadIdx.x & 31, lanes = 32 / each, sub = lane & (lanes - 1);
    for (int first = b0 + w * each; first < b1; first += warps * each) {
        const int b = first + lane / lanes;
        Seq s{};
        if (b < b1) {
            s = load_seq(a, b);
            if (!s.ok) atomicOr(&g_shared_err, SWA_DEVERR_BAD_POSITION);
            if (!kOrdered && sa.few && s.n > 0 && rows_in_common(a, s, b)) s.n = 0;
            if (sub == 0) {
                // (a sequence without new tokens may end inside what the others share)
                if (!sa.few) sa.base[b] = s.n > 0 ? base : 0;
                int4 *info = sa.info + 2 * static_cast<int64_t>(b);
                info[0] = s.n > 0 ? make_int4(base, group.n, group.few, group.q0) : make_int4(0, 0, 0, 0);
                info[1] = make_int4(group.p0, g, s.n > 0, 0);
            }
        }
        if (sa.few || (base > 0 && a.window != INT_MAX))  // the rows' positions
            for (int i = sub; i < s.n; i += lanes)
                if (SWA_IN_BOUNDS(s.q0 + i < a.N, &g_shared_err)) {
                    sa.pos[s.q0 + i] = s.p0 + i;
                    if (sa.few) sa.seq[s.q0 + i] = b;
                }
        if (!sa.few) continue;
        const int longest = __reduce_max_sync(0xffffffffu, s.n);
        for (int ut = 0; ut * TT < longest; ++ut) {
            const bool unit = ut * TT < s.n;
            const Keys k = unit ? own_keys(a, s, base, ut, TT, sa.part[0]) : Keys{};
            list_stretches(sa, k, unit ? k.stretches() : 0,
                           Stretch{b, s.q0 + ut * TT, min(TT, s.n - ut * TT), 0, 0, 0, 0, 0}, lanes);
        }
    }
}

// All sequences, alone.  Stretches write their results by rows, so of sequences that have rows in common, as a q_start that
// goes down can make them, none is taken: their rows stay as they were.  Thus the units are no more than the lists have
// room for, and are counted in 32 bits.  (Out of line: for broken lists alone.)
__device__ __noinline__ void put_alone(const SharedArgs &sa, bool ordered, int w, int warps) {
    if (ordered) put_sequences<true>(sa, 0, sa.a.B, PagedGroup{}, -1, w, warps);
    else put_sequences<false>(sa, 0, sa.a.B, PagedGroup{}, -1, w, warps);
}

// (two blocks an SM: the blocks that store tokens are many; with one and 222 registers the plan of 64 sequences takes 6.4
// us, 6.7 with two, and that of 5700 new tokens 23.4 instead of 16.5)
__global__ void __launch_bounds__(kThreads, 2) paged_plan_kernel(const __grid_constant__ SharedArgs sa) {
    const PagedArgs &a = sa.a;
    const cg::cluster_group cluster = cg::this_cluster();
    __shared__ Members sums[kWarps];
    __shared__ int first;  // of the group's entries in question: the first that is not shared
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = static_cast<int>(cluster.block_rank()), ranks = static_cast<int>(cluster.num_blocks());
    const int clusters = sa.clusters, c = static_cast<int>(blockIdx.x) / ranks;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (c >= clusters) {  // the blocks behind those of the plan store the new tokens, a warp a token
        const int w0 = (static_cast<int>(blockIdx.x) - clusters * ranks) * kWarps + warp;
        const int warps = (static_cast<int>(gridDim.x) - clusters * ranks) * kWarps;
        for (int n = w0; n < a.N; n += warps) store_token(a, n, lane, &g_shared_err);
        return;
    }
    if (clusters == 1 && rank == 0 && tid < kCounts) sa.counts[tid] = 0;  // (seen by the cluster behind its first barrier)
    const int first_b = __ldg(sa.group_start), end_b = __ldg(sa.group_start + sa.n_groups);
    bool fine = true, ordered = true;
    for (int i = tid; i < sa.n_groups; i += kThreads) {
        const int b0 = __ldg(sa.group_start + i), b1 = __ldg(sa.group_start + i + 1);
        fine = fine && b0 >= 0 && b1 >= b0 && b1 <= a.B;
    }
    // (A q_start that goes down can give many groups the same rows, and each of them all rows: more work than any call
    // has.  Then there is no group.)
    if (a.q_start) {
#pragma unroll 8
        for (int b = tid; b < a.B; b += kThreads) ordered = ordered && __ldg(a.q_start + b) <= __ldg(a.q_start + b + 1);
    }
    fine = __syncthreads_and(fine && ordered);
    ordered = fine || __syncthreads_and(ordered);
    if (!fine && blockIdx.x == 0 && tid == 0) atomicOr(&g_shared_err, SWA_DEVERR_BAD_POSITION);
    for (int g = c; g < sa.n_groups; g += clusters) {
        const int b0 = fine ? __ldg(sa.group_start + g) : 0, b1 = fine ? __ldg(sa.group_start + g + 1) : 0;
        Members m{~0ull, ~0ull, -1, 0, 0, 0, 0};
        for (int b = b0 + tid; b < b1; b += kThreads) {
            const Seq s = load_seq(a, b);
            if (!s.ok) m.broken = 1;
            if (s.n > 0)
                m = join(m, Members{static_cast<unsigned long long>(s.p0) << 13 | static_cast<unsigned int>(b - b0),
                                    ~0ull, s.p0 + s.n - 1, 1, sa.few ? 1 : (s.n + sa.own_tokens - 1) / sa.own_tokens, 0, s.n});
        }
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) m = join(m, shuffled(m, o));
        if (lane == 0) sums[warp] = m;
        if (tid == 0) first = INT_MAX;
        // (the words that the cluster's other blocks write to are set before any of them does)
        if (ranks > 1) cluster.barrier_arrive();
        __syncthreads();
        m = sums[0];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) m = join(m, sums[w]);
        int base = 0, leader = 0, p0 = 0;
        // A prefix part that has as many tiles of rows as the sequences alone would save nothing.
        const bool stretch = sa.few && m.tokens * a.G <= kStretchRows;
        const int64_t prefix_tiles = (m.tokens + sa.prefix_tokens - 1) / sa.prefix_tokens;
        const bool shares = !m.broken && m.count >= 2 && prefix_tiles < m.tiles && (stretch || sa.any_tiles);
        if (shares) {  // (the same for every thread of the cluster)
            leader = b0 + static_cast<int>(m.least & ((1u << 13) - 1));
            p0 = static_cast<int>(m.least >> 13);
            const int lo = p0 >= a.window ? p0 - a.window + 1 : 0;
            const int e_lo = lo >> a.ps_log2, e_end = p0 >> a.ps_log2;
            const int e_sink = static_cast<int>((static_cast<int64_t>(a.n_sink) + a.ps - 1) >> a.ps_log2);
            const int sinks = min(e_lo, e_sink);
            const int n = sinks + e_end - e_lo;  // entries in question: those of the sinks, then the window's
            const int chunks = (n + kChunk - 1) / kChunk;
            const int32_t *row0 = a.table + static_cast<int64_t>(leader) * a.width;
            // Where rows are short and there are more than warps, a warp compares several at a time (2048 sequences of 64
            // entries: the kernel takes 18 us, 40 with one; 512 of 32 9, 15 with one).
            int words = kWords;  // of a row that a lane loads
            while (words > 1 && 2 * n <= 32 * words && (b1 - b0) * words > ranks * kWarps * kWords) words /= 2;
            int differs = INT_MAX;
            auto compare = [&](auto rows) {
                constexpr bool several = decltype(rows)::value;
                const int w = several ? words : kWords, w_log2 = __ffs(w) - 1, each = kWords >> w_log2;
                const int64_t tasks = static_cast<int64_t>((b1 - b0 + each - 1) / each) * chunks;
                for (int64_t t = rank * kWarps + warp; t < tasks; t += ranks * kWarps) {
                    const int i0 = static_cast<int>(t % chunks) * kChunk, b = b0 + static_cast<int>(t / chunks) * each;
                    if (__all_sync(0xffffffffu, i0 >= differs)) continue;
                    const Seq s = load_seq(a, min(b + (lane & (each - 1)), b1 - 1));  // (the last one's several times over)
                    // (a sequence without new tokens needs nothing)
                    const int my_lo = s.n == 0 ? -1 : s.p0 >= a.window ? s.p0 - a.window + 1 : 0;
                    int x[kWords], y[kWords];
#pragma unroll
                    for (int k = 0; k < kWords; ++k) {
                        const int i = i0 + (k & (w - 1)) * 32 + lane, e = several ? min(i, n - 1) : i;
                        const int j = e < sinks ? e : e_lo + e - sinks;
                        // (several: all loads, so that they are on their way at a time; one: those there are)
                        const bool in = e < n && SWA_IN_BOUNDS(j >= 0 && j < a.width, &g_shared_err);
                        x[k] = in ? __ldg(row0 + j) : 0;
                        y[k] = in ? __ldg(a.table + static_cast<int64_t>(min(b + (k >> w_log2), b1 - 1)) * a.width + j) : 0;
                    }
#pragma unroll
                    for (int k = kWords - 1; k >= 0; --k) {
                        const int i = i0 + (k & (w - 1)) * 32 + lane, e = several ? min(i, n - 1) : i;
                        const int j = e < sinks ? e : e_lo + e - sinks;
                        const int lo_k = several ? __shfl_sync(0xffffffffu, my_lo, k >> w_log2) : my_lo;
                        // (needed: some position of the entry is in reach of the sequence's first new token, or a sink)
                        const bool needed = lo_k >= 0 && ((static_cast<int64_t>(j) + 1) << a.ps_log2 > lo_k || j < e_sink);
                        if (x[k] != y[k] && needed) differs = min(differs, e);
                    }
                }
            };
            if (words < kWords) compare(std::true_type{});
            else compare(std::false_type{});
            differs = __reduce_min_sync(0xffffffffu, differs);
            if (ranks > 1) cluster.barrier_wait();
            if (lane == 0 && differs < INT_MAX) atomicMin(ranks > 1 ? cluster.map_shared_rank(&first, 0) : &first, differs);
            if (ranks > 1) cluster.sync();
            else __syncthreads();
            const int f = min(ranks > 1 ? *cluster.map_shared_rank(&first, 0) : first, n);
            base = f < sinks ? 0 : (e_lo + f - sinks) << a.ps_log2;
            // (what two sequences at least have a use for; the others look behind it)
            const int p1 = static_cast<int>(m.next >> 13);
            const int used = base - (p1 >= a.window ? p1 - a.window + 1 : 0);
            const int64_t saved = static_cast<int64_t>(used) * (m.tiles - prefix_tiles);
            if (used < kLeastShared || (!sa.few && saved < static_cast<int64_t>(kLeastSaved) * m.tiles)) base = 0;
        } else if (ranks > 1) {
            cluster.barrier_wait();
        }
        // (read by the other blocks before it is set for the next group; the sums, too)
        if (ranks > 1) cluster.barrier_arrive();
        PagedGroup out{};
        if (base > 0) {
            out.q0 = a.q_start ? __ldg(a.q_start + b0) : b0;
            (stretch ? out.few : out.n) = static_cast<int>(m.tokens);
            out.p0 = p0;
            out.end = base;
            out.row = leader;
            out.top = m.top;
        }
        if (rank == 0 && warp == 0) {
            if (lane == 0) {
                sa.groups[g] = out;
                if (out.n > 0) atomicAdd(sa.counts + kTileGroups, 1);
            }
            if (out.few > 0) {
                const Keys k = prefix_keys(a, p0, base, sa.few_prefix);
                list_stretches(sa, k, k.stretches(), Stretch{leader, out.q0, out.few, prefix_place(sa, g, out.q0) - out.q0, 0, 0, 1, 0}, 32);
            }
        }
        put_sequences<true>(sa, b0, b1, out, g, rank * kWarps + warp, ranks * kWarps);
        if (ranks > 1) cluster.barrier_wait();
        else __syncthreads();
    }
    if (c == 0 && fine) {  // sequences of no group
        put_sequences<true>(sa, 0, first_b, PagedGroup{}, -1, rank * kWarps + warp, ranks * kWarps);
        put_sequences<true>(sa, end_b, a.B, PagedGroup{}, -1, rank * kWarps + warp, ranks * kWarps);
    } else if (c == 0) {
        put_alone(sa, ordered, rank * kWarps + warp, ranks * kWarps);
    }
}

// ---------------------------------------------------------------------------------------------
// join: `kLanes` lanes a row, a warp the rows of a few heads of one token.  A row's results (m, l, acc), of its own
// part and of its group's prefix part, each in planes or in the slots of the CTAs that share a unit, are joined:
// with M the largest m, o = sum 2^(m - M) acc / sum 2^(m - M) l.  Bound by latency -- the row's sequence, its
// units, the maxima, the values, each read from L2 or HBM behind the last --, so 8 lanes a row where warps of one row
// would fill the SMs a good part (76000 rows of 128: 105 us with 32 lanes each, 35 with 8; 14400 and 8192 rows, the whole
// call: 150 and 132 us, 137 and 125 with 8; 4160 rows the same), 32 where they would not (2048 rows with 22 results
// each: 7 us, 12 with 8).
// ---------------------------------------------------------------------------------------------
template <int E>
__device__ __forceinline__ void load_columns(float (&x)[E], const float *src) {
    if constexpr (E == 2) {
        const float2 t = __ldcg(reinterpret_cast<const float2 *>(src));
        x[0] = t.x, x[1] = t.y;
    } else {
#pragma unroll
        for (int e = 0; e < E; e += 4) {
            const float4 t = __ldcg(reinterpret_cast<const float4 *>(src + e));
            x[e] = t.x, x[e + 1] = t.y, x[e + 2] = t.z, x[e + 3] = t.w;
        }
    }
}

// Where the results of a row's part are: in planes, or in the slots of the CTAs that share its unit.
struct Where {
    const PartResults *p = nullptr;
    int count = 0, sink = -1, owner = 0;  // sink: the number of the sinks' stretch (their plane is the last)
    int row = 0;  // of the unit, or the token's place in a plane
    bool pieces = false;
};
__device__ __forceinline__ Where in_planes(const PartResults &p, const Keys &k, int place) {
    return Where{&p, k.stretches(), k.count, 0, place, false};
}
// Of a unit of the many-row kernel with owner and pieces x, a row of it, of token n.
__device__ __forceinline__ Where in_unit(const PartResults &p, int2 x, int row, int n) {
    // (a unit that was never finished, after an expired wait, has any record)
    if (x.y <= 0 || x.x < 0 || x.y > p.ctas || x.x > p.ctas - x.y) return Where{&p, 1, -1, 0, n, false};
    return Where{&p, x.y, -1, x.x, row, true};
}
// Of a row's prefix part in tiles; q0, number: of the group.
__device__ __forceinline__ Where in_prefix_tiles(const SharedArgs &sa, int q0, int number, int n, int head) {
    const PagedArgs &a = sa.a;
    const PartResults &p = sa.part[1];
    const int tok = n - q0, ut = tok / p.TT, r = tok % p.TT;
    const int2 rec = __ldcg(p.units + (static_cast<int64_t>(q0 / p.TT) + number + ut) * a.H_kv + head / a.G);
    return in_unit(p, rec, r / p.TQ * kTileRows + r % p.TQ * a.G + head % a.G, n);
}

// Joins the row of token n of sequence b (s) and a head, by kLanes lanes; row_there: whether they have one.
template <int D, int kLanes>
__device__ __forceinline__ void join_row(const SharedArgs &sa, int b, const Seq &s, int n, int head, bool row_there,
                                         const Where &own, const Where &pre) {
    // columns of a lane: kV neighbours in each of E / kV blocks of kLanes * kV
    constexpr int E = D / kLanes, kV = E < 4 ? E : 4;
    constexpr int kAtOnce = E <= 4 ? 12 : E <= 8 ? 8 : E <= 16 ? 4 : 2;  // results whose values are on their way at a time
    const PagedArgs &a = sa.a;
    const int part = threadIdx.x % kLanes;
    const int64_t row = static_cast<int64_t>(n) * a.H_q + head;
    auto result = [&](int c, const float2 *&ml, const float *&o) {
        const bool first = c < own.count;
        const Where &w = first ? own : pre;
        const int k = first ? c : c - own.count;
        const PartResults &p = *w.p;
        if (w.pieces) {
            const int64_t slot = k == 0 ? 2 * w.owner + 1 : 2 * (w.owner + k);
            ml = reinterpret_cast<const float2 *>(p.ws.ml) + slot * p.rows + w.row;
            o = p.ws.acc + (slot * p.rows + w.row) * D;
        } else {
            const int64_t at = (static_cast<int64_t>(k == w.sink ? p.planes - 1 : k) * p.tokens + w.row) * a.H_q + head;
            ml = p.ml + at;
            o = p.o + at * D;
        }
    };
    // (heads of a token have as many results each, but for those of units that several CTAs have)
    const int count = !row_there || own.count == 0 ? 0 : own.count + pre.count;
    const int most = __reduce_max_sync(0xffffffffu, count);
    float acc[E], m = -INFINITY, L = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.f;
    for (int c0 = 0; c0 < most; c0 += kLanes) {
        const int in = min(kLanes, count - c0);
        float2 v2 = make_float2(-INFINITY, 0.f);
        const float *o = nullptr;
        if (part < in) {
            const float2 *ml;
            result(c0 + part, ml, o);
            v2 = __ldcg(ml);
        }
        float val[kAtOnce][E];
        auto load = [&](int k0) {
#pragma unroll
            for (int k = 0; k < kAtOnce; ++k) {
                const auto src = reinterpret_cast<const float *>(
                    __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(o), (k0 + k) % kLanes, kLanes));
                float t[kV];
#pragma unroll
                for (int e = 0; e < E; e += kV) {
                    if (k0 + k < in) {
                        load_columns<kV>(t, src + (e / kV * kLanes + part) * kV);
                    } else {
#pragma unroll
                        for (int z = 0; z < kV; ++z) t[z] = 0.f;
                    }
#pragma unroll
                    for (int z = 0; z < kV; ++z) val[k][e + z] = t[z];
                }
            }
        };
        load(0);
        float mn = fmaxf(m, v2.x);
#pragma unroll
        for (int d = kLanes / 2; d >= 1; d >>= 1) mn = fmaxf(mn, __shfl_xor_sync(0xffffffffu, mn, d));
        // (a result that kept nothing of this row has weight 0 and finite values)
        const float ms = mn == -INFINITY ? 0.f : mn, old = ex2(m - ms), f = ex2(v2.x - ms);
        L = L * old + f * v2.y;
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] *= old;
        m = mn;
        for (int k0 = 0; k0 < min(kLanes, most - c0); k0 += kAtOnce) {
            if (k0 > 0) load(k0);
#pragma unroll
            for (int k = 0; k < kAtOnce; ++k) {
                const float fk = __shfl_sync(0xffffffffu, f, (k0 + k) % kLanes, kLanes);
#pragma unroll
                for (int e = 0; e < E; ++e) acc[e] += fk * val[k][e];
            }
        }
    }
#pragma unroll
    for (int d = kLanes / 2; d >= 1; d >>= 1) L += __shfl_xor_sync(0xffffffffu, L, d);
    if (count == 0 || !SWA_IN_BOUNDS(n < a.N && head < a.H_q && b < a.B, &g_shared_err)) return;
    const float inv = 1.f / L;  // every row keeps its own key
    uint16_t *op = a.o + n * a.o_st[0] + head * a.o_st[1];
#pragma unroll
    for (int e = 0; e < E; e += kV) {
        uint16_t *at = op + (e / kV * kLanes + part) * kV;
        if constexpr (kV == 2)
            *reinterpret_cast<uint32_t *>(at) = pack_bf16x2(acc[e] * inv, acc[e + 1] * inv);
        else
            *reinterpret_cast<uint2 *>(at) = make_uint2(pack_bf16x2(acc[e] * inv, acc[e + 1] * inv),
                                                        pack_bf16x2(acc[e + 2] * inv, acc[e + 3] * inv));
    }
    if (part == 0) {
        a.lse[row] = (m + log2f(L)) * 0.69314718055994531f;
        if (a.counts) a.counts[row] = kept_keys(a, s.p0 + n - s.q0);
    }
}

// By rows: own parts in stretches, every row is joined.
template <int D, int kLanes>
__global__ void __launch_bounds__(kThreads) paged_join_kernel(const __grid_constant__ SharedArgs sa) {
    constexpr int kHeads = 32 / kLanes;
    const PagedArgs &a = sa.a;
    const int lane = threadIdx.x & 31;
    const int64_t x = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    const int blocks = (a.H_q + kHeads - 1) / kHeads;  // of a token's heads
    const int n = static_cast<int>(x / blocks), h = static_cast<int>(x % blocks) * kHeads + lane / kLanes;
    // (the plan's: the kernels before this one have waited for it before they let this grid start; of a row of no
    // sequence any number)
    const int at = n < a.N ? __ldcg(sa.seq + n) : -1;
    const int b = at >= 0 && at < a.B ? at : -1;
    const Seq s = b >= 0 ? load_seq(a, b) : Seq{};
    const int4 *info = sa.info + 2 * static_cast<int64_t>(max(b, 0));
    // base, the group's tokens in tiles, in stretches, its first; its p0, number, whether the sequence is taken
    const int4 u = __ldcg(info), v = __ldcg(info + 1);
    // (by every warp, with a row or without, so that what waits for this grid waits for those before it)
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (b < 0 || !v.z || n < s.q0 || n >= s.q0 + s.n) return;
    const bool row_there = h < a.H_q;
    const int head = row_there ? h : 0, TT = few_tokens(a.G);
    const Where own = in_planes(sa.part[0], own_keys(a, s, u.x, (n - s.q0) / TT, TT, sa.part[0]), n);
    const Where pre = u.z > 0   ? in_planes(sa.few_prefix, prefix_keys(a, v.x, u.x, sa.few_prefix),
                                            prefix_place(sa, v.y, u.w) + n - u.w)
                      : u.y > 0 ? in_prefix_tiles(sa, u.w, v.y, n, head)
                                : Where{};
    join_row<D, kLanes>(sa, b, s, n, head, row_there, own, pre);
}

// By units: own parts in tiles of rows, whose units are on a list if their rows are not final (two chunks of 12981
// tokens that share nothing, 16 heads of 256: the call takes 198 us, 255 by rows, which find that next to none is to be
// joined; 14 chunks of up to 500 tokens 358, 376; 57 short ones about three prefixes, where all are, 62, 59).
// A block has as many rows of a unit at a time as it has lanes for.
template <int D, int kLanes>
__global__ void __launch_bounds__(kThreads, 2) paged_join_units_kernel(const __grid_constant__ SharedArgs sa) {
    constexpr int kRows = kThreads / kLanes;
    const PagedArgs &a = sa.a;
    const PartResults &p = sa.part[0];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int subs = p.TT / p.TQ * (kTileRows / kRows);
    int64_t x = blockIdx.x;
    // (an entry is on its way while the one before it is used, the first one with the list's length)
    int4 next = __ldcg(sa.own_units + x / subs * 2), next_seq = __ldcg(sa.own_units + x / subs * 2 + 1);
    const int64_t items = static_cast<int64_t>(min(__ldcg(sa.counts + kOwnUnits), sa.own_units_cap)) * subs;
    while (x < items) {
        const int4 unit = next, seq = next_seq;
        const int r = static_cast<int>(x % subs) * kRows + static_cast<int>(threadIdx.x) / kLanes, y = r % kTileRows;
        x += gridDim.x;
        if (x < items) next = __ldcg(sa.own_units + x / subs * 2), next_seq = __ldcg(sa.own_units + x / subs * 2 + 1);
        const int b = unit.z, ut = unit.w / a.H_kv, kvh = unit.w % a.H_kv;
        if (!SWA_IN_BOUNDS(b >= 0 && b < a.B && ut >= 0 && kvh >= 0 && seq.x >= 0 && seq.x + seq.y <= a.N, &g_shared_err)) continue;
        const Seq s{seq.x, seq.y, __ldg(a.p0 + b), true};
        const int i = ut * p.TT + r / kTileRows * p.TQ + y / a.G;
        const bool row_there = y < p.TQ * a.G && i < s.n;
        const int n = s.q0 + (row_there ? i : 0), head = kvh * a.G + y % a.G;
        if (__all_sync(0xffffffffu, !row_there)) continue;
        const Where pre = seq.z >= 0 ? in_prefix_tiles(sa, seq.z, seq.w, n, head) : Where{};
        join_row<D, kLanes>(sa, b, s, n, head, row_there, in_unit(p, make_int2(unit.x, unit.y), r, n), pre);
    }
}

// ---------------------------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------------------------
struct Layout {
    bool few, tiles;  // tiles: prefixes may go to the many-row kernel
    int planes, prefix_planes, prefix_tokens, own_cap, prefix_cap;
    PagedShape shape;  // of the many-row kernel
    int own_units;  // units of the own part, at most
    size_t slots[2], base, info, groups, pos, seq, count, list, units[2], ml[2], o[2], few_ml, few_o, bytes;
};

Layout layout(const PagedArgs &a, int n_groups) {
    Layout l{};
    l.few = paged_few_rows(a);
    // (no group of a batch of so few rows has more than a stretch takes)
    l.tiles = !l.few || static_cast<int64_t>(a.N) * a.G > kStretchRows;
    l.shape = paged_tile_shape(a);
    const int TT = few_tokens(a.G);
    const int64_t units = std::min<int64_t>(a.N, static_cast<int64_t>(a.N) / TT + a.B);
    // Planes: the stretches that a unit of each part has at most, and the sinks'.  So many that there are six own
    // stretches for every resident warp where all are as long as that, two of prefixes, whose results have more rows;
    // two a unit at least.  (31 groups of up to 13 rows: 1, 2, 8, 24 prefix stretches a warp 130, 108, 124, 153 us;
    // 64 histories of 4096 tokens that share nothing: 4, 6, 16 own ones 193, 194, 217 us.)
    auto planes = [&](int64_t each, int64_t n) {
        const int64_t want = (each * shared_rows_warps(a.D) + n * a.H_kv - 1) / (n * a.H_kv);
        return static_cast<int>(std::min<int64_t>(std::max<int64_t>(want, 2), kMostPlanes - 1)) + 1;
    };
    // At least planes(each, n) * n, and not less for more n, so that the size does not shrink where the call grows.
    auto room = [&](int64_t each, int64_t n) {
        const int64_t stretches = (each * shared_rows_warps(a.D) + a.H_kv - 1) / a.H_kv;
        return std::min<int64_t>(kMostPlanes * n, std::max(stretches + 2 * n, 3 * n));
    };
    // A prefix of few rows is that of two tokens at least, and of no more than a stretch takes: as many places each.
    const int64_t prefixes = std::min<int64_t>(n_groups, (static_cast<int64_t>(a.N) + 1) / 2);
    const bool few_prefixes = l.few && TT >= 2 && a.N >= 2;
    l.planes = l.few ? planes(6, units) : 1;
    l.prefix_planes = few_prefixes ? planes(2, prefixes) : 0;
    l.prefix_tokens = few_prefixes ? static_cast<int>(std::min<int64_t>(a.N, static_cast<int64_t>(n_groups) * TT)) : 0;
    const int64_t most = INT_MAX / 2 / a.H_kv;  // (the items of both, a head each, are counted in 32 bits)
    l.own_cap = l.few ? static_cast<int>(std::min(units * l.planes, most)) : 0;
    l.prefix_cap = few_prefixes ? static_cast<int>(std::min(prefixes * l.prefix_planes, most)) : 0;
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t x = at;
        at += paged_up(bytes);
        return x;
    };
    const bool tiles[2] = {!l.few, l.tiles};
    for (int p = 0; p < 2; ++p) {
        const int TU = paged_tile_tokens(a, p ? Part::kPrefix : Part::kOwn);
        const size_t n_units = (static_cast<size_t>(a.N) / TU + (p ? n_groups : a.B) + 2) * a.H_kv;
        // (tokens times planes)
        const size_t results = p || !l.few ? a.N : (static_cast<size_t>(room(6, units)) * a.N + units - 1) / units;
        l.slots[p] = take(tiles[p] ? paged_ws_bytes(l.shape, a.D) : 0);
        l.units[p] = take(tiles[p] ? n_units * (p ? sizeof(int2) : 2 * sizeof(int4)) : 0);
        if (!p) l.own_units = tiles[p] ? static_cast<int>(std::min<size_t>(n_units, INT_MAX / 2)) : 0;
        l.ml[p] = take(tiles[p] || !p ? results * a.H_q * 8 : 0);
        l.o[p] = take(tiles[p] || !p ? results * a.H_q * a.D * 4 : 0);
    }
    // (prefix_tokens * prefix_planes at least: groups * TT are all tokens or those of all groups, and fewer groups do not
    // have fewer planes)
    const int64_t groups = std::min<int64_t>(prefixes, (static_cast<int64_t>(a.N) + TT - 1) / TT);
    const size_t results = few_prefixes ? static_cast<size_t>(room(2, groups)) * TT : 0;
    l.few_ml = take(results * a.H_q * 8);
    l.few_o = take(results * a.H_q * a.D * 4);
    l.base = take(static_cast<size_t>(a.B) * 4);
    l.info = take(static_cast<size_t>(a.B) * 32);
    l.groups = take(static_cast<size_t>(n_groups) * sizeof(PagedGroup));
    l.pos = take(static_cast<size_t>(a.N) * 4);
    l.seq = take(l.few ? static_cast<size_t>(a.N) * 4 : 0);
    l.count = take(kCounts * 4);
    l.list = take(((few_prefixes ? room(2, prefixes) : 0) + (l.few ? room(6, units) : 0)) * sizeof(Stretch));
    l.bytes = at;
    return l;
}

cudaError_t launch_plan(SharedArgs &sa, cudaStream_t s) {
    const int ranks = sa.n_groups < kFewGroups ? kCluster : 1;
    sa.clusters = std::min(sa.n_groups, paged_sm_count() * 4);
    if (sa.clusters > 1) {
        const cudaError_t e = cudaMemsetAsync(sa.counts, 0, kCounts * 4, s);
        if (e != cudaSuccess) return e;
    }
    int append = 0;
    if (sa.a.kn) append = std::min((sa.a.N + kWarps - 1) / kWarps, paged_sm_count() * 8);
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(ranks * (sa.clusters + (append + ranks - 1) / ranks));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = ranks;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, paged_plan_kernel, sa);
}

template <int D>
cudaError_t launch_join_d(const SharedArgs &sa, cudaStream_t s) {
    const int64_t rows = static_cast<int64_t>(sa.a.N) * sa.a.H_q;
    const bool many = rows > static_cast<int64_t>(paged_sm_count()) * 20;
    const int heads = many ? 4 : 1;  // of a warp
    if (!sa.few) {
        const PartResults &p = sa.part[0];
        const int64_t items = static_cast<int64_t>(sa.own_units_cap) * (p.TT / p.TQ * kTileRows / (kWarps * heads));
        const int blocks = static_cast<int>(std::min<int64_t>(items, paged_sm_count() * kJoinBlocks));
        return launch_dependent(true, many ? paged_join_units_kernel<D, 8> : paged_join_units_kernel<D, 32>, dim3(blocks),
                                kThreads, 0, s, sa);
    }
    const int64_t warps = static_cast<int64_t>(sa.a.N) * ((sa.a.H_q + heads - 1) / heads);
    const int64_t blocks = (warps + kWarps - 1) / kWarps;
    if (blocks > INT_MAX) return cudaErrorInvalidValue;
    return launch_dependent(true, many ? paged_join_kernel<D, 8> : paged_join_kernel<D, 32>,
                            dim3(static_cast<unsigned int>(blocks)), kThreads, 0, s, sa);
}

cudaError_t launch_join(const SharedArgs &sa, cudaStream_t s) {
    switch (sa.a.D) {
        case 64: return launch_join_d<64>(sa, s);
        case 128: return launch_join_d<128>(sa, s);
        case 256: return launch_join_d<256>(sa, s);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace

size_t paged_shared_workspace_bytes(const PagedArgs &a, int n_groups) {
    return a.N > 0 ? layout(a, n_groups).bytes : 256;
}

cudaError_t launch_paged_shared(const PagedArgs &a, const int32_t *group_start, int n_groups, void *ws,
                                cudaStream_t s) {
    const Layout l = layout(a, n_groups);
    char *p = static_cast<char *>(ws);
    SharedArgs sa{};
    sa.a = a;
    sa.group_start = group_start;
    sa.n_groups = n_groups;
    sa.groups = reinterpret_cast<PagedGroup *>(p + l.groups);
    sa.base = reinterpret_cast<int32_t *>(p + l.base);
    sa.info = reinterpret_cast<int4 *>(p + l.info);
    sa.pos = reinterpret_cast<int32_t *>(p + l.pos);
    sa.seq = reinterpret_cast<int32_t *>(p + l.seq);
    sa.stretches = reinterpret_cast<Stretch *>(p + l.list);
    sa.counts = reinterpret_cast<int32_t *>(p + l.count);
    sa.own_cap = l.own_cap;
    sa.prefix_cap = l.prefix_cap;
    sa.own_units = reinterpret_cast<const int4 *>(p + l.units[0]);
    sa.own_units_cap = l.own_units;
    sa.few = l.few;
    sa.any_tiles = l.tiles;
    sa.prefix_tokens = sa.own_tokens = l.shape.TQ;
    for (int x = 0; x < 2; ++x) {
        PartResults &r = sa.part[x];
        r.ml = reinterpret_cast<float2 *>(p + l.ml[x]);
        r.o = reinterpret_cast<float *>(p + l.o[x]);
        r.planes = x ? 1 : l.planes;
        r.tokens = a.N;
        if (x) r.units = reinterpret_cast<const int2 *>(p + l.units[x]);
        r.ws = paged_carve(p + l.slots[x], l.shape, a.D);
        r.ctas = l.shape.ctas;
        r.rows = l.shape.tiles * l.shape.rows;
        r.TQ = l.shape.TQ;
        r.TT = paged_tile_tokens(a, x ? Part::kPrefix : Part::kOwn);
    }
    sa.few_prefix.ml = reinterpret_cast<float2 *>(p + l.few_ml);
    sa.few_prefix.o = reinterpret_cast<float *>(p + l.few_o);
    sa.few_prefix.planes = l.prefix_planes;
    sa.few_prefix.tokens = l.prefix_tokens;
    auto part_args = [&](int x) {
        PagedArgs t = sa.a;
        t.kn = t.vn = nullptr;
        t.tile_groups = sa.counts + kTileGroups;
        t.groups = sa.groups;
        t.pos = sa.pos;
        t.base = sa.base;
        t.part_ml = sa.part[x].ml;
        t.part_o = sa.part[x].o;
        if (x) {
            t.part_units = reinterpret_cast<int2 *>(p + l.units[1]);
        } else {
            t.part_list = reinterpret_cast<int4 *>(p + l.units[0]);
            t.part_count = sa.counts + kOwnUnits;
            t.part_cap = l.own_units;
            t.part_info = sa.info;
        }
        if (x) t.B = n_groups;
        return t;
    };
    cudaError_t e = launch_plan(sa, s);
    if (e != cudaSuccess) return e;
    if (l.tiles) e = launch_paged_tile(part_args(1), sa.part[1].ws, true, s, Part::kPrefix);
    if (e != cudaSuccess) return e;
    e = l.few ? launch_shared_rows(sa, l.tiles, s) : launch_paged_tile(part_args(0), sa.part[0].ws, true, s, Part::kOwn);
    return e != cudaSuccess ? e : launch_join(sa, s);
}

unsigned int paged_shared_read_clear_error() {
    unsigned int v = 0, z = 0;
    if (cudaMemcpyFromSymbol(&v, g_shared_err, sizeof v) != cudaSuccess) return 0;
    cudaMemcpyToSymbol(g_shared_err, &z, sizeof z);
    return v;
}

}  // namespace swa
