// swa_paged.cu -- a paged KV cache: storing new tokens in their pages, and attention of a
// ragged batch of new tokens over it.
#include <atomic>
#include <climits>
#include <cmath>

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
// attention, a warp per (new token, query head): one pass over the keys with the running
// maximum and sum of the softmax
// ---------------------------------------------------------------------------------------------
template <int D>
__global__ void __launch_bounds__(kThreads) paged_attend_kernel(const PagedArgs a) {
    constexpr int E = D / 32;
    const int lane = threadIdx.x & 31;
    const int64_t rows = static_cast<int64_t>(a.N) * a.H_q;
    const int64_t step = static_cast<int64_t>(gridDim.x) * (kThreads / 32);
    for (int64_t r = (static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x) >> 5; r < rows; r += step) {
        const int n = static_cast<int>(r / a.H_q), h = static_cast<int>(r % a.H_q), kvh = h / a.G;
        const int b = find_sequence(a, n, lane);
        if (b < 0) continue;
        const Seq s = load_seq(a, b);
        if (!s.ok) {
            if (lane == 0) atomicOr(&g_paged_err, SWA_DEVERR_BAD_POSITION);
            continue;
        }
        const int t = s.p0 + (n - s.q0);
        float q[E], acc[E];
        const auto *qp = reinterpret_cast<const __nv_bfloat16 *>(a.q) + static_cast<int64_t>(n) * a.q_st[0] + h * a.q_st[1];
#pragma unroll
        for (int e = 0; e < E; ++e) {
            q[e] = __bfloat162float(qp[e * 32 + lane]) * a.scale_log2;
            acc[e] = 0.f;
        }
        float m = -INFINITY, l = 0.f;
        int count = 0;
        const int lo = t >= a.window ? t - a.window + 1 : 0;
        for (int p = lo > 0 && a.n_sink > 0 ? 0 : lo; p <= t; ++p) {
            if (p >= a.n_sink && p < lo) {
                p = lo - 1;
                continue;
            }
            const int page = page_of(a, b, p >> a.ps_log2);
            const bool there = page < a.n_pages;
            if (!there && lane == 0) atomicOr(&g_paged_err, SWA_DEVERR_BAD_PAGE);
            const int64_t row = ((static_cast<int64_t>(page) * a.H_kv + kvh) * a.ps + (p & (a.ps - 1))) * D;
            const auto *kp = reinterpret_cast<const __nv_bfloat16 *>(a.k_pages) + row;
            const auto *vp = reinterpret_cast<const __nv_bfloat16 *>(a.v_pages) + row;
            float x = 0.f;
#pragma unroll
            for (int e = 0; e < E; ++e) x += there ? q[e] * __bfloat162float(kp[e * 32 + lane]) : 0.f;
#pragma unroll
            for (int o = 16; o >= 1; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
            const float mn = fmaxf(m, x), al = ex2(m - mn), w = ex2(x - mn);
            m = mn;
            l = l * al + w;
#pragma unroll
            for (int e = 0; e < E; ++e) acc[e] = acc[e] * al + (there ? w * __bfloat162float(vp[e * 32 + lane]) : 0.f);
            ++count;
        }
        auto *op = reinterpret_cast<__nv_bfloat16 *>(a.o) + static_cast<int64_t>(n) * a.o_st[0] + h * a.o_st[1];
#pragma unroll
        for (int e = 0; e < E; ++e) op[e * 32 + lane] = __float2bfloat16_rn(acc[e] / l);
        if (lane == 0) {
            a.lse[r] = (m + log2f(l)) * 0.69314718055994531f;
            if (a.counts) a.counts[r] = count;
        }
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

size_t paged_workspace_bytes(const PagedArgs &) { return 0; }

cudaError_t launch_paged_append(const PagedArgs &a, cudaStream_t s) {
    const int64_t blocks = (static_cast<int64_t>(a.N) * 32 + kThreads - 1) / kThreads;
    const int64_t cap = static_cast<int64_t>(paged_sm_count()) * 8;
    paged_append_kernel<<<static_cast<int>(blocks < cap ? blocks : cap), kThreads, 0, s>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_paged_attend(const PagedArgs &a, void *, cudaStream_t s) {
    if (a.kn) {
        const cudaError_t e = launch_paged_append(a, s);
        if (e != cudaSuccess) return e;
    }
    const int64_t blocks = (static_cast<int64_t>(a.N) * a.H_q * 32 + kThreads - 1) / kThreads;
    const int64_t cap = static_cast<int64_t>(paged_sm_count()) * 8;
    const int grid = static_cast<int>(blocks < cap ? blocks : cap);
    switch (a.D) {
        case 64: paged_attend_kernel<64><<<grid, kThreads, 0, s>>>(a); break;
        case 128: paged_attend_kernel<128><<<grid, kThreads, 0, s>>>(a); break;
        case 256: paged_attend_kernel<256><<<grid, kThreads, 0, s>>>(a); break;
        default: return cudaErrorInvalidValue;
    }
    return cudaGetLastError();
}

void paged_read_clear_error(unsigned int *data, unsigned int *split, unsigned int *prefill) {
    unsigned int v = 0, z = 0;
    *data = *split = *prefill = 0;
    if (cudaMemcpyFromSymbol(&v, g_paged_err, sizeof v) != cudaSuccess) return;
    cudaMemcpyToSymbol(g_paged_err, &z, sizeof z);
    *data = v;
}

}  // namespace swa
