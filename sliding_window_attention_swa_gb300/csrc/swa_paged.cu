// swa_paged.cu -- a paged KV cache: storing new tokens in their pages, and attention of a
// ragged batch of new tokens over it (the choice of its kernel, and the merge of shared units).
#include <atomic>
#include <climits>
#include <cmath>

#include <cudaTypedefs.h>

#include "ptx.cuh"
#include "swa_paged.cuh"

namespace swa {
namespace {

__device__ unsigned int g_paged_err = 0;

constexpr int kThreads = 256;

// ---------------------------------------------------------------------------------------------
// append: a warp per token
// ---------------------------------------------------------------------------------------------
__global__ void __launch_bounds__(kThreads) paged_append_kernel(const PagedArgs a) {
    // the attention kernel behind this one may start: it waits for this grid before it reads a page
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int lane = threadIdx.x & 31;
    const int step = gridDim.x * (kThreads / 32);
    for (int n = (blockIdx.x * kThreads + threadIdx.x) >> 5; n < a.N; n += step) {
        const int b = find_sequence(a, n, lane);
        if (b < 0) continue;
        const Seq s = load_seq(a, b);
        if (!s.ok) {
            if (lane == 0) atomicOr(&g_paged_err, SWA_DEVERR_BAD_POSITION);
            continue;
        }
        const int p = s.p0 + (n - s.q0);
        const int page = page_of(a, b, p >> a.ps_log2);
        if (page >= a.n_pages) {
            if (lane == 0) atomicOr(&g_paged_err, SWA_DEVERR_BAD_PAGE);
            continue;
        }
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
}

// ---------------------------------------------------------------------------------------------
// merge of the units that several CTAs share: block (c, y) takes eight rows of the unit that CTA
// c began and left open, a warp per row.  The pieces lie in the slots 2c + 1, 2(c+1), 2(c+2), ...
// A row's weight of a piece is 2^(m_piece - m), o = sum of weighted values / sum of weighted sums.
// Bound by the latency of a few dependent loads; launched as a programmatic dependent of the
// kernel that wrote the pieces.
// ---------------------------------------------------------------------------------------------
constexpr int kMergeRows = kThreads / 32;

template <int D>
__global__ void __launch_bounds__(kThreads) paged_merge_kernel(const PagedArgs a, const PagedWs w, const PagedShape x) {
    constexpr int E = D / 32;  // columns of a lane
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int4 rec = w.open[blockIdx.x];
    const long long start = w.first[blockIdx.x];
    const int own = w.left[blockIdx.x], c = static_cast<int>(blockIdx.x);
    if (rec.x == 0) return;
    // the unit's tiles end at `end` of the list: CTAs c + 1 .. c + np - 1 start before that
    const long long end = start + own + rec.x;
    int np = 1;
    for (int k0 = c + 1; k0 < x.ctas; k0 += 32) {
        const int n = __popc(__ballot_sync(0xffffffffu, k0 + lane < x.ctas && w.first[k0 + lane] < end));
        np += n;
        if (n < 32) break;
    }
    const int row = blockIdx.y * kMergeRows + warp;  // of the unit: tile * x.rows + token * G + head
    const int tile = row / x.rows, r = row % x.rows;
    const Seq s = load_seq(a, rec.y);
    const int i = (rec.w * x.tiles + tile) * x.TQ + r / a.G;  // token of the sequence
    if (tile >= x.tiles || r >= x.TQ * a.G || i >= s.n) return;
    const int rows = x.tiles * x.rows;
    auto slot = [&](int k) { return static_cast<int64_t>(k == 0 ? 2 * c + 1 : 2 * (c + k)); };
    // (a CTA between two of the unit's may have no tiles of it)
    auto piece = [&](int k) {
        return k == 0 || w.left[c + k] > 0 ? *reinterpret_cast<const float2 *>(w.ml + (slot(k) * rows + row) * 2)
                                               : make_float2(-INFINITY, 0.f);
    };
    float m = -INFINITY;
    for (int k = lane; k < np; k += 32) m = fmaxf(m, piece(k).x);
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    float acc[E], L = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.f;
    for (int k0 = 0; k0 < np; k0 += 32) {
        float2 ml = make_float2(-INFINITY, 0.f);
        if (k0 + lane < np) ml = piece(k0 + lane);
        const float f = ml.x == -INFINITY ? 0.f : ex2(ml.x - m);
        L += f * ml.y;
        const int n = min(32, np - k0);
#pragma unroll 4
        for (int k = 0; k < n; ++k) {
            const float fk = __shfl_sync(0xffffffffu, f, k);
            if (fk == 0.f) continue;  // (nothing kept, or nothing written)
            const float *v = w.acc + partial_at<D>(slot(k0 + k), rows, row, lane * E);
#pragma unroll
            for (int e = 0; e < E; e += 2) {
                const float2 t = *reinterpret_cast<const float2 *>(v + e);
                acc[e] += fk * t.x;
                acc[e + 1] += fk * t.y;
            }
        }
    }
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
    const int64_t tok = s.q0 + i;
    const int h = rec.z * a.G + r % a.G;
    if (!SWA_IN_BOUNDS(tok < a.N && h < a.H_q, &g_paged_err)) return;
    const float inv = 1.f / L;  // every row keeps its own key
    uint16_t *op = a.o + tok * a.o_st[0] + h * a.o_st[1] + lane * E;
#pragma unroll
    for (int e = 0; e < E; e += 2) *reinterpret_cast<uint32_t *>(op + e) = pack_bf16x2(acc[e] * inv, acc[e + 1] * inv);
    if (lane == 0) {
        a.lse[tok * a.H_q + h] = (m + log2f(L)) * 0.69314718055994531f;
        if (a.counts) a.counts[tok * a.H_q + h] = kept_keys(a, s.p0 + i);
    }
}

cudaError_t launch_merge(const PagedArgs &a, const PagedWs &w, const PagedShape &x, cudaStream_t s) {
    const dim3 grid(x.ctas, (x.tiles * x.rows + kMergeRows - 1) / kMergeRows);
    switch (a.D) {
        case 64: return launch_dependent(true, paged_merge_kernel<64>, grid, kThreads, 0, s, a, w, x);
        case 128: return launch_dependent(true, paged_merge_kernel<128>, grid, kThreads, 0, s, a, w, x);
        case 256: return launch_dependent(true, paged_merge_kernel<256>, grid, kThreads, 0, s, a, w, x);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace

int paged_sm_count() {
    static std::atomic<int> n[64];  // per device; 0 = not looked up yet
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 148;
    int v = n[dev].load(std::memory_order_relaxed);
    if (v == 0) {
        if (cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || v <= 0) v = 148;
        n[dev].store(v, std::memory_order_relaxed);
    }
    return v;
}

bool paged_map(CUtensorMap *m, const void *base, int D, int64_t n1, int64_t n2, int64_t n3, int64_t s1, int64_t s2,
               int64_t s3, int b1, int b2) {
    static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
        cudaDriverEntryPointQueryResult q;
        void *p = nullptr;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            p = nullptr;
        return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    }();
    if (!fn) return false;
    cuuint64_t dims[4] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(n1), static_cast<cuuint64_t>(n2),
                          static_cast<cuuint64_t>(n3)};
    cuuint64_t strides[3] = {static_cast<cuuint64_t>(s1) * 2, static_cast<cuuint64_t>(s2) * 2,
                             static_cast<cuuint64_t>(s3) * 2};
    cuuint32_t box[4] = {64u, static_cast<cuuint32_t>(b1), static_cast<cuuint32_t>(b2), 1u};
    cuuint32_t es[4] = {1, 1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(base), dims, strides, box, es,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Few rows: every sequence's new tokens fit one unit of the split kernel (16 rows).  With more of
// them that kernel would read the keys once per 16 rows.
static bool few_rows(const PagedArgs &a) { return !a.q_start || (a.max_q > 0 && a.max_q * a.G <= 16); }
static PagedShape shape_of(const PagedArgs &a) { return few_rows(a) ? paged_split_shape(a) : paged_tile_shape(a); }

size_t paged_workspace_bytes(const PagedArgs &a) { return paged_ws_bytes(shape_of(a), a.D); }

cudaError_t launch_paged_append(const PagedArgs &a, cudaStream_t s) {
    const int64_t blocks = (static_cast<int64_t>(a.N) * 32 + kThreads - 1) / kThreads;
    const int64_t cap = static_cast<int64_t>(paged_sm_count()) * 8;
    paged_append_kernel<<<static_cast<int>(blocks < cap ? blocks : cap), kThreads, 0, s>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_paged_attend(const PagedArgs &args, void *ws, cudaStream_t s) {
    PagedArgs a = args;
    const bool after_append = a.kn && a.q_start;  // (one token a sequence: stored by the attention kernel)
    if (after_append) {
        const cudaError_t e = launch_paged_append(a, s);
        if (e != cudaSuccess) return e;
        a.kn = a.vn = nullptr;
    }
    const PagedShape x = shape_of(a);
    const PagedWs w = paged_carve(ws, x, a.D);
    const cudaError_t e = few_rows(a) ? launch_paged_split(a, w, after_append, s) : launch_paged_tile(a, w, after_append, s);
    return e != cudaSuccess ? e : launch_merge(a, w, x, s);
}

void paged_read_clear_error(unsigned int *data, unsigned int *split, unsigned int *prefill) {
    unsigned int v = 0, z = 0;
    paged_split_read_clear_error(data, split);
    paged_tile_read_clear_error(&v, prefill);
    *data |= v;
    if (cudaMemcpyFromSymbol(&v, g_paged_err, sizeof v) != cudaSuccess) return;
    cudaMemcpyToSymbol(g_paged_err, &z, sizeof z);
    *data |= v;
}

}  // namespace swa
