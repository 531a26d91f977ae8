// swa_paged.cu -- a paged KV cache: storing new tokens in their pages, and attention of a
// ragged batch of new tokens over it (the choice of its kernel).
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
// append: a warp per token.  Up to 512 tokens (8 heads of 128) 5 us, the latency of finding the sequence,
// its page, then the rows; 16384 tokens 28.0 us, 128000 208 us, 71 and 74% of the measured copy rate.
// ---------------------------------------------------------------------------------------------
__global__ void __launch_bounds__(kThreads) paged_append_kernel(const PagedArgs a, int32_t *zero, int n_zero) {
    // the attention kernel behind this one may start: it waits for this grid before it reads a page
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    for (int i = blockIdx.x * kThreads + threadIdx.x; i < n_zero; i += gridDim.x * kThreads) zero[i] = 0;
    const int lane = threadIdx.x & 31;
    const int step = gridDim.x * (kThreads / 32);
    for (int n = (blockIdx.x * kThreads + threadIdx.x) >> 5; n < a.N; n += step) {
        store_token(a, n, lane, &g_paged_err);
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

namespace {
bool encode(CUtensorMap *m, const void *base, const int64_t (&dims)[4], const int64_t (&strides)[3],
            const int (&box)[4]) {
    static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
        cudaDriverEntryPointQueryResult q;
        void *p = nullptr;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            p = nullptr;
        return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    }();
    if (!fn) return false;
    cuuint64_t d[4], st[3];
    cuuint32_t bx[4], es[4] = {1, 1, 1, 1};
    for (int i = 0; i < 4; ++i) {
        d[i] = static_cast<cuuint64_t>(dims[i]);
        bx[i] = static_cast<cuuint32_t>(box[i]);
        if (i < 3) st[i] = static_cast<cuuint64_t>(strides[i]) * 2;
    }
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(base), d, st, bx, es,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
}  // namespace

bool paged_query_map(CUtensorMap *m, const PagedArgs &a, int heads, int tokens) {
    return encode(m, a.q, {a.D, a.H_q, a.N, 1}, {a.q_st[1], a.q_st[0], a.q_st[0]}, {64, heads, tokens, 1});
}

bool paged_pool_map(CUtensorMap *m, const PagedArgs &a, const void *pool, int rows) {
    const int64_t groups = static_cast<int64_t>(a.n_pages) * a.H_kv * (a.ps / 8);
    return encode(m, pool, {64, 8, a.D / 64, groups}, {a.D, 64, static_cast<int64_t>(8) * a.D},
                  {64, 8, a.D / 64, rows / 8});
}

// Few rows: every sequence's new tokens fit one unit of the split kernel (16 rows).  With more of
// them that kernel would read the keys once per 16 rows.
bool paged_few_rows(const PagedArgs &a) { return !a.q_start || (a.max_q > 0 && a.max_q <= 16 / a.G); }
static PagedShape shape_of(const PagedArgs &a) { return paged_few_rows(a) ? paged_split_shape(a) : paged_tile_shape(a); }

size_t paged_workspace_bytes(const PagedArgs &a) { return paged_ws_bytes(shape_of(a), a.D); }

cudaError_t launch_paged_append(const PagedArgs &a, int32_t *zero, int n_zero, cudaStream_t s) {
    const int64_t blocks = (static_cast<int64_t>(a.N) * 32 + kThreads - 1) / kThreads;
    const int64_t cap = static_cast<int64_t>(paged_sm_count()) * 8;
    paged_append_kernel<<<static_cast<int>(blocks < cap ? blocks : cap), kThreads, 0, s>>>(a, zero, n_zero);
    return cudaGetLastError();
}

cudaError_t launch_paged_attend(const PagedArgs &args, void *ws, cudaStream_t s) {
    PagedArgs a = args;
    const bool few = paged_few_rows(a);
    const PagedShape x = shape_of(a);
    const PagedWs w = paged_carve(ws, x, a.D);
    const int n_done = few ? 0 : x.ctas * 8;
    const bool after_append = a.kn && a.q_start;  // (one token a sequence: stored by the attention kernel)
    cudaError_t e = cudaSuccess;
    if (after_append) {
        e = launch_paged_append(a, w.done, n_done, s);
        a.kn = a.vn = nullptr;
    } else if (n_done) {
        e = cudaMemsetAsync(w.done, 0, n_done * sizeof(int32_t), s);
    }
    if (e != cudaSuccess) return e;
    if (!few) return launch_paged_tile(a, w, after_append, s);
    e = launch_paged_split(a, w, after_append, s);
    return e != cudaSuccess ? e : launch_paged_merge(a, w, x, s);
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
