// swa_paged_shared.cu -- attention of sequences that share leading pages: each group's prefix is read
// once for the new tokens of all its sequences.
//
// A row's softmax is the same over its keys in any two parts (m, l, acc), joined by their maxima:
//   1. plan (here): finds for every group how many leading positions its sequences share.
//   2. prefix part (paged_tile_kernel, kPrefix): the group's packed rows, of all its sequences, are the rows of
//      the tensor cores' tiles; each row's mean and log2 of its sum go to the workspace in fp32.
//   3. own part (the few-row or the many-row kernel, kOwn): each sequence over the positions behind, counted
//      from there, and where a unit's rows are written the prefix part joins them as one piece more.
// With single tokens a group of R sequences reads its prefix once instead of R times, and its products go to
// the tensor cores in tiles of 128 rows instead of 16.
#include <climits>

#include <cooperative_groups.h>

#include "swa_paged.cuh"

namespace swa {
namespace {

namespace cg = cooperative_groups;

__device__ unsigned int g_shared_err = 0;

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kFewGroups = 32;  // below it a cluster plans a group, else a block
constexpr int kCluster = 8;
constexpr int kChunk = 256;  // entries that a warp compares at a time: eight loads a lane and row in flight

struct PlanArgs {
    PagedArgs a;
    const int32_t *group_start;  // [n_groups + 1]
    int n_groups;
    PagedGroup *groups;
    int32_t *base, *pos;
    int32_t *zero;  // words that the kernels behind this one want zero
    int n_zero;
    int TQ;          // tokens of a tile of the prefix part
    int own_tokens;  // tokens that the own part's kernel has in a tile (0: any sequence's)
};

// Of a group's sequences that have new tokens.
struct Members {
    unsigned long long least;  // least p0, and the first sequence with it: p0 << 13 | (b - b0)
    int top, count, tiles, broken;
    long long tokens;
};
static_assert(kPagedMaxB <= 1 << 13, "the first sequence's number");

__device__ __forceinline__ Members join(const Members &x, const Members &y) {
    return Members{min(x.least, y.least), max(x.top, y.top), x.count + y.count, x.tiles + y.tiles, x.broken | y.broken,
                   x.tokens + y.tokens};
}
__device__ __forceinline__ Members shuffled(const Members &x, int o) {
    return Members{__shfl_xor_sync(0xffffffffu, x.least, o), __shfl_xor_sync(0xffffffffu, x.top, o),
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
// Bound by latency: the list, the sequences' lengths, then the table's rows, all of them once.
// ---------------------------------------------------------------------------------------------
__global__ void __launch_bounds__(kThreads) paged_plan_kernel(const __grid_constant__ PlanArgs pa) {
    const PagedArgs &a = pa.a;
    const cg::cluster_group cluster = cg::this_cluster();
    __shared__ Members sums[kWarps];
    __shared__ int first;  // of the group's entries in question: the first that is not shared
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = static_cast<int>(cluster.block_rank()), ranks = static_cast<int>(cluster.num_blocks());
    const int clusters = static_cast<int>(gridDim.x) / ranks, c = static_cast<int>(blockIdx.x) / ranks;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    for (int i = static_cast<int>(blockIdx.x) * kThreads + tid; i < pa.n_zero; i += static_cast<int>(gridDim.x) * kThreads)
        pa.zero[i] = 0;
    bool fine = true;
    for (int i = tid; i < pa.n_groups; i += kThreads) {
        const int b0 = __ldg(pa.group_start + i), b1 = __ldg(pa.group_start + i + 1);
        fine = fine && b0 >= 0 && b1 >= b0 && b1 <= a.B;
    }
    fine = __syncthreads_and(fine);
    if (!fine && blockIdx.x == 0 && tid == 0) atomicOr(&g_shared_err, SWA_DEVERR_BAD_POSITION);
    if (c == 0) {  // sequences of no group
        const int lo = fine ? __ldg(pa.group_start) : a.B, hi = fine ? __ldg(pa.group_start + pa.n_groups) : a.B;
        for (int b = rank * kThreads + tid; b < a.B; b += ranks * kThreads)
            if (b < lo || b >= hi) pa.base[b] = 0;
    }
    for (int g = c; g < pa.n_groups; g += clusters) {
        const int b0 = fine ? __ldg(pa.group_start + g) : 0, b1 = fine ? __ldg(pa.group_start + g + 1) : 0;
        Members m{~0ull, -1, 0, 0, 0, 0};
        for (int b = b0 + tid; b < b1; b += kThreads) {
            const Seq s = load_seq(a, b);
            if (!s.ok) m.broken = 1;
            if (s.n > 0)
                m = join(m, Members{static_cast<unsigned long long>(s.p0) << 13 | static_cast<unsigned int>(b - b0),
                                    s.p0 + s.n - 1, 1, pa.own_tokens ? (s.n + pa.own_tokens - 1) / pa.own_tokens : 1, 0,
                                    s.n});
        }
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) m = join(m, shuffled(m, o));
        if (lane == 0) sums[warp] = m;
        if (tid == 0) first = INT_MAX;
        // (the words that the cluster's other blocks write to are set before any of them does)
        if (ranks > 1) cluster.sync();
        else __syncthreads();
        m = sums[0];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) m = join(m, sums[w]);
        int base = 0, leader = 0, p0 = 0;
        // A prefix part that has as many tiles of rows as the sequences alone would save nothing.
        const bool shares = !m.broken && m.count >= 2 && (m.tokens + pa.TQ - 1) / pa.TQ < m.tiles;
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
            const int64_t tasks = static_cast<int64_t>(b1 - b0) * chunks;
            int differs = INT_MAX;
            for (int64_t t = rank * kWarps + warp; t < tasks; t += ranks * kWarps) {
                const int i0 = static_cast<int>(t % chunks) * kChunk, b = b0 + static_cast<int>(t / chunks);
                if (i0 >= differs || b == leader) continue;
                const Seq s = load_seq(a, b);
                if (s.n == 0) continue;
                const int my_lo = s.p0 >= a.window ? s.p0 - a.window + 1 : 0;
                const int32_t *row = a.table + static_cast<int64_t>(b) * a.width;
                int x[kChunk / 32], y[kChunk / 32];
#pragma unroll
                for (int k = 0; k < kChunk / 32; ++k) {
                    const int i = i0 + k * 32 + lane, j = i < sinks ? i : e_lo + i - sinks;
                    // (needed: some position of the entry is in reach of the sequence's first new token, or a sink)
                    const bool needed = i < n && ((static_cast<int64_t>(j) + 1) << a.ps_log2 > my_lo || j < e_sink) &&
                                        SWA_IN_BOUNDS(j >= 0 && j < a.width, &g_shared_err);
                    x[k] = needed ? __ldg(row0 + j) : 0;
                    y[k] = needed ? __ldg(row + j) : 0;
                }
#pragma unroll
                for (int k = kChunk / 32 - 1; k >= 0; --k)
                    if (x[k] != y[k]) differs = min(differs, i0 + k * 32 + lane);
            }
            differs = __reduce_min_sync(0xffffffffu, differs);
            if (lane == 0 && differs < INT_MAX) atomicMin(ranks > 1 ? cluster.map_shared_rank(&first, 0) : &first, differs);
            if (ranks > 1) cluster.sync();
            else __syncthreads();
            const int f = min(ranks > 1 ? *cluster.map_shared_rank(&first, 0) : first, n);
            base = f < sinks ? 0 : (e_lo + f - sinks) << a.ps_log2;
            if (base <= lo) base = 0;  // nothing of a window
        }
        // (read by the other blocks before it is set for the next group; the sums, too)
        if (ranks > 1) cluster.sync();
        else __syncthreads();
        if (rank == 0 && tid == 0) {
            PagedGroup out{};
            if (base > 0) {
                out.q0 = a.q_start ? __ldg(a.q_start + b0) : b0;
                out.n = static_cast<int>(m.tokens);
                out.p0 = p0;
                out.end = base;
                out.row = leader;
                out.top = m.top;
            }
            pa.groups[g] = out;
        }
        for (int b = b0 + rank * kWarps + warp; b < b1; b += ranks * kWarps) {
            const Seq s = load_seq(a, b);
            if (lane == 0) pa.base[b] = s.n > 0 ? base : 0;
            if (base > 0 && a.window != INT_MAX)
                for (int i = lane; i < s.n; i += 32)
                    if (SWA_IN_BOUNDS(s.q0 + i < a.N, &g_shared_err)) pa.pos[s.q0 + i] = s.p0 + i;
        }
    }
    // (behind an append: what waits for this kernel waits for that, too)
    asm volatile("griddepcontrol.wait;" ::: "memory");
}

struct Layout {
    PagedShape prefix, own;
    size_t done, base, groups, pos, lse, o, bytes;
};

Layout layout(const PagedArgs &a, int n_groups) {
    Layout l{};
    l.prefix = paged_tile_shape(a);
    l.own = paged_few_rows(a) ? paged_split_shape(a) : paged_tile_shape(a);
    const size_t x = paged_ws_bytes(l.prefix, a.D), y = paged_ws_bytes(l.own, a.D);
    // (one after the other: the parts' partial results share their place)
    l.done = x > y ? x : y;
    l.base = l.done + paged_up(static_cast<size_t>(l.own.ctas) * 32);
    l.groups = l.base + paged_up(static_cast<size_t>(a.B) * 4);
    l.pos = l.groups + paged_up(static_cast<size_t>(n_groups) * sizeof(PagedGroup));
    l.lse = l.pos + paged_up(static_cast<size_t>(a.N) * 4);
    l.o = l.lse + paged_up(static_cast<size_t>(a.N) * a.H_q * 4);
    l.bytes = l.o + paged_up(static_cast<size_t>(a.N) * a.H_q * a.D * 4);
    return l;
}

cudaError_t launch_plan(const PlanArgs &pa, bool after_append, cudaStream_t s) {
    const int ranks = pa.n_groups < kFewGroups ? kCluster : 1;
    const int most = paged_sm_count() * 4;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(ranks * (pa.n_groups < most ? pa.n_groups : most));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = ranks;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = after_append ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, paged_plan_kernel, pa);
}

}  // namespace

size_t paged_shared_workspace_bytes(const PagedArgs &a, int n_groups) { return layout(a, n_groups).bytes; }

cudaError_t launch_paged_shared(const PagedArgs &args, const int32_t *group_start, int n_groups, void *ws,
                                cudaStream_t s) {
    PagedArgs a = args;
    const bool few = paged_few_rows(a);
    const Layout l = layout(a, n_groups);
    char *p = static_cast<char *>(ws);
    PagedWs w_prefix = paged_carve(ws, l.prefix, a.D), w_own = paged_carve(ws, l.own, a.D);
    // the counters of shared units: those of the prefix part lie at the partial results' end, those of the own
    // part, which the prefix part's partial results must not overwrite, in a place of their own
    if (!few) w_own.done = reinterpret_cast<int32_t *>(p + l.done);
    a.base = reinterpret_cast<const int32_t *>(p + l.base);
    a.groups = reinterpret_cast<const PagedGroup *>(p + l.groups);
    a.pos = reinterpret_cast<const int32_t *>(p + l.pos);
    a.pre_lse = reinterpret_cast<float *>(p + l.lse);
    a.pre_o = reinterpret_cast<float *>(p + l.o);
    cudaError_t e = cudaSuccess;
    const bool append = a.kn && a.q_start;  // (one token a sequence: stored by the attention kernel)
    if (append) {
        e = launch_paged_append(a, w_prefix.done, l.prefix.ctas * 8, s);
        if (e != cudaSuccess) return e;
        a.kn = a.vn = nullptr;
    } else {
        e = cudaMemsetAsync(w_prefix.done, 0, l.prefix.ctas * 32, s);
        if (e != cudaSuccess) return e;
    }
    PlanArgs pa{};
    pa.a = a;
    pa.group_start = group_start;
    pa.n_groups = n_groups;
    pa.groups = reinterpret_cast<PagedGroup *>(p + l.groups);
    pa.base = reinterpret_cast<int32_t *>(p + l.base);
    pa.pos = reinterpret_cast<int32_t *>(p + l.pos);
    pa.zero = reinterpret_cast<int32_t *>(p + l.done);
    pa.n_zero = few ? 0 : l.own.ctas * 8;
    pa.TQ = l.prefix.TQ;
    pa.own_tokens = few ? 0 : l.own.TQ;
    e = launch_plan(pa, append, s);
    if (e != cudaSuccess) return e;
    PagedArgs g = a;
    g.B = n_groups;
    e = launch_paged_tile(g, w_prefix, true, s, Part::kPrefix);
    if (e != cudaSuccess) return e;
    if (!few) return launch_paged_tile(a, w_own, true, s, Part::kOwn);
    e = launch_paged_split(a, w_own, true, s, Part::kOwn);
    return e != cudaSuccess ? e : launch_paged_merge(a, w_own, l.own, s, Part::kOwn);
}

unsigned int paged_shared_read_clear_error() {
    unsigned int v = 0, z = 0;
    if (cudaMemcpyFromSymbol(&v, g_shared_err, sizeof v) != cudaSuccess) return 0;
    cudaMemcpyToSymbol(g_shared_err, &z, sizeof z);
    return v;
}

}  // namespace swa
