// swa_paged_rows.cu -- stretches of at most 16 query rows over a few hundred keys of a paged cache: the
// sequences' own parts of swa_paged_attend_shared with few new tokens, and prefixes of few rows.
//
// A warp takes a stretch by itself: it copies 16 or 32 keys and values at a time by TMA into a ring of its own,
// scores them (mma.sync, the rows are M), keeps the running maximum and sum, and writes the unnormalised result.  No two
// warps wait for one another, so that the latencies of a stretch -- its rows, its pages, its first copies, its end -- are
// hidden by the other warps' work and by its own copies: the next stretch's first steps are on their way
// while the last one ends.  Own parts are short (a sample's answer so far), and it is these latencies, not
// the bytes, that the kernel for long histories (a block a unit) spends its time on there: 135 sequences of 250
// tokens on average behind what they share, 141 MB, 72 us of that kernel, about 25 of this one.
// Bound by HBM: 31 prefixes of up to 13 rows and 227 own parts, head dim 64, 513 MB in 87 us (5.9 TB/s, 87% of the
// measured copy rate).  P is rounded to bf16 for the second product; the sum takes it unrounded.
// Every wait is bounded; on expiry the warp records an error word, drains its copies and returns.
#include <algorithm>
#include <atomic>
#include <climits>
#include <cmath>

#include "swa_paged_shared.cuh"

namespace swa {
namespace {

__device__ unsigned int g_rows_err = 0;   // waits and bounds
__device__ unsigned int g_rows_data = 0;  // broken device data

template <int D>
struct RowsCfg {
    static constexpr int KS = D == 64 ? 32 : 16;  // keys a step
    static constexpr int STAGE = 2 * KS * D * 2;  // keys and values of a step
    // A ring a warp: more warps or deeper rings, as shared memory allows both.  Drafts of 256-wide heads with one block of
    // four warps and three steps each 100 us, two of three warps and two steps 96, one of seven and two 95; 31 small groups of
    // 64-wide heads (three blocks of four, two steps) 102, four of four and three steps of 16 keys 112; 64 sequences of
    // 128-wide ones (two of four, three steps) 73, three of four and two 76.
    static constexpr int NST = D == 128 ? 3 : 2;
    static constexpr int WARPS = D <= 128 ? 4 : 7;
    static constexpr int CTAS_PER_SM = D <= 64 ? 3 : D <= 128 ? 2 : 1;
    static constexpr int OFF_BAR = WARPS * NST * STAGE;
    static constexpr int SMEM = OFF_BAR + WARPS * NST * 8 + 1024;
    static_assert((SMEM + 1024) * CTAS_PER_SM <= 233472, "shared memory budget");
};

// Offset of 16-byte piece `pc` of row `row` in a 128B-swizzled tile (layout of paged_pool_map).
template <int D>
__device__ __forceinline__ uint32_t sw128(int row, int pc) {
    return static_cast<uint32_t>((row >> 3) * (D * 16) + (pc >> 3) * 1024 + (row & 7) * 128 +
                                 (((pc & 7) ^ (row & 7)) << 4));
}

struct Work : Stretch {
    int kvh, key0, steps;  // key0: the first step's first key
};

template <int D>
__global__ void __launch_bounds__(RowsCfg<D>::WARPS * 32, RowsCfg<D>::CTAS_PER_SM)
    paged_rows_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                      const __grid_constant__ SharedArgs sa, const int behind_tiles, const int fault_stop) {
    using C = RowsCfg<D>;
    constexpr int NST = C::NST, KS = C::KS, kWarps = C::WARPS;
    const PagedArgs &a = sa.a;
    extern __shared__ uint8_t smem_raw[];
    __shared__ int abort_flag;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t sraw = smem_u32(smem_raw);
    const uint32_t sbase = (sraw + 1023u) & ~1023u;
    const uint32_t ring = sbase + warp * (NST * C::STAGE);
    uint8_t *ring_gen = smem_raw + (ring - sraw);
    auto bar = [&](int st) { return sbase + C::OFF_BAR + 8u * (warp * NST + st); };
    if (tid == 0) {
        abort_flag = 0;
        for (int i = 0; i < kWarps * NST; ++i) mbar_init(sbase + C::OFF_BAR + 8u * i, 1);
        fence_mbar_init();
    }
    if (tid == 0) {
        tma_prefetch_desc(&tm_k);
        tma_prefetch_desc(&tm_v);
    }
    __syncthreads();
    volatile int *abort = &abort_flag;
    // Behind the prefix part, which has waited for the plan before it let this grid start, nothing has to be waited
    // for here; else the plan has.
    if (!behind_tiles) asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    // (rows that the plan's launch has stored, ahead of their copies)
    asm volatile("fence.proxy.async.global;" ::: "memory");

    // A warp's first is its own, the next ones go to whichever warp is free (results do not depend on which).
    const int firsts = static_cast<int>(gridDim.x) * kWarps;
    auto take = [&]() -> int {
        int x = 0;
        if (lane == 0) x = atomicAdd(sa.counts + kTaken, 1);
        return firsts + __shfl_sync(0xffffffffu, x, 0);
    };
    // Neighbouring warps take the heads of one stretch, which lie side by side in its pages.
    // Prefixes first: theirs are the longer ones.
    const int n_prefix = min(__ldcg(sa.counts + kPrefixStretches), sa.prefix_cap);
    const int n_items = (n_prefix + min(__ldcg(sa.counts + kOwnStretches), sa.own_cap)) * a.H_kv;
    auto load_work = [&](int item) -> Work {
        Work w{};
        if (item < n_items) {
            const int e = item / a.H_kv;
            const int4 *p = reinterpret_cast<const int4 *>(sa.stretches + (e < n_prefix ? e : sa.prefix_cap + e - n_prefix));
            const int4 x = __ldcg(p), y = __ldcg(p + 1);
            w.row = x.x, w.q0 = x.y, w.n = x.z, w.first = x.w, w.k0 = y.x, w.k1 = y.y, w.part = y.z;
            w.kvh = item % a.H_kv;
            w.key0 = w.k0 & ~(KS - 1);
            w.steps = (w.k1 - w.key0 + KS - 1) / KS;
        }
        return w;
    };
    // A step is one box, a page of 16 half of one.  The pages of 32 boxes are looked up at a time, lane i that of
    // box i from step `from` on; -1: the box is outside the stretch, n_pages: there is none.
    const int box = min(a.ps, KS), boxes = KS / box, window = 32 / boxes;
    auto pages_of = [&](const Work &w, int from) -> int {
        const int key = w.key0 + from * KS + lane * box;
        return from < w.steps && key < w.k1 && key + box > w.k0 ? page_of(a, w.row, key >> a.ps_log2) : -1;
    };
    // what is streamed once leaves L2 before the parts' results do
    const uint64_t policy = l2_evict_first();
    int issued = 0, taken = 0;  // steps copied and used so far
    bool ok = true;
    auto issue = [&](const Work &w, int i, int pages) {
        if (issued >= fault_stop) return;  // planted fault: this step is never copied
        const int j = lane % boxes, st = issued % NST;
        const int page = __shfl_sync(0xffffffffu, pages, (i * boxes + j) & 31);
        if (lane == 0) mbar_arrive_expect_tx(bar(st), C::STAGE);
        __syncwarp();
        if (lane < 2 * boxes) {  // keys, then values, a lane each
            const int v = lane / boxes, row = (w.key0 + i * KS + j * box) & (a.ps - 1);
            if (page >= a.n_pages) atomicOr(&g_rows_data, SWA_DEVERR_BAD_PAGE);
            // debug build: the box lies in the page, the head exists
            (void)SWA_IN_BOUNDS(row + box <= a.ps && w.kvh < a.H_kv && page <= a.n_pages, &g_rows_err);
            tma_load_4d(ring + st * C::STAGE + v * (C::STAGE / 2) + j * box * D * 2, v ? &tm_v : &tm_k, bar(st), 0, 0, 0,
                        ((page < 0 ? a.n_pages : page) * a.H_kv + w.kvh) * (a.ps >> 3) + (row >> 3), policy);
        }
        __syncwarp();
        ++issued;
    };

    const int own = static_cast<int>(blockIdx.x) * kWarps + warp;
    Work w = load_work(own);
    int pages = pages_of(w, 0), at = 0;  // at: steps of w that are issued
    const int r0 = lane >> 2, r1 = r0 + 8, kq = 2 * (lane & 3);
    while (ok && w.steps > 0) {
        while (at < w.steps && at < window && issued - taken < NST) issue(w, at++, pages);
        const Work next = load_work(take());
        const int next_pages = pages_of(next, 0);
        int next_at = 0;
        // ---- the rows: fragments of rows r0, r1 of the 16-row M tile, and which keys each keeps
        const int rows = w.n * a.G;
        const bool v0 = r0 < rows, v1 = r1 < rows;
        const int tok0 = w.q0 + (v0 ? r0 / a.G : 0), tok1 = w.q0 + (v1 ? r1 / a.G : 0);
        const int h0 = w.kvh * a.G + (v0 ? r0 % a.G : 0), h1 = w.kvh * a.G + (v1 ? r1 % a.G : 0);
        (void)SWA_IN_BOUNDS(w.q0 >= 0 && w.q0 + w.n <= a.N && w.row < a.B && rows <= kStretchRows, &g_rows_err);
        uint32_t qa[D / 16][4];
        {
            const uint16_t *q0 = a.q + tok0 * a.q_st[0] + h0 * a.q_st[1], *q1 = a.q + tok1 * a.q_st[0] + h1 * a.q_st[1];
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
                qa[kk][0] = v0 ? __ldg(reinterpret_cast<const unsigned *>(q0 + kk * 16 + kq)) : 0u;
                qa[kk][1] = v1 ? __ldg(reinterpret_cast<const unsigned *>(q1 + kk * 16 + kq)) : 0u;
                qa[kk][2] = v0 ? __ldg(reinterpret_cast<const unsigned *>(q0 + kk * 16 + 8 + kq)) : 0u;
                qa[kk][3] = v1 ? __ldg(reinterpret_cast<const unsigned *>(q1 + kk * 16 + 8 + kq)) : 0u;
            }
        }
        const int t0 = __ldcg(sa.pos + tok0), t1 = __ldcg(sa.pos + tok1);
        const int lo0 = t0 >= a.window ? t0 - a.window + 1 : 0, lo1 = t1 >= a.window ? t1 - a.window + 1 : 0;
        const int hi0 = min(t0 + 1, w.k1), hi1 = min(t1 + 1, w.k1);
        float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
        float acc[D / 8][4];
#pragma unroll
        for (int n = 0; n < D / 8; ++n) acc[n][0] = acc[n][1] = acc[n][2] = acc[n][3] = 0.f;

#pragma unroll 1
        for (int i = 0; i < w.steps; ++i) {
            const int st = taken % NST;
            if (!__all_sync(0xffffffffu, mbar_wait<true>(bar(st), (taken / NST) & 1, abort, &g_rows_err))) {
                ok = false;
                break;
            }
            const uint32_t ks = ring + st * C::STAGE, vs = ks + C::STAGE / 2;
            const int key = w.key0 + i * KS;
            const bool edge = key < w.k0 || key + KS > w.k1;
            if (edge) {  // value rows outside the stretch may hold anything, even NaN
                uint8_t *vg = ring_gen + st * C::STAGE + C::STAGE / 2;
                for (int idx = lane; idx < KS * (D / 8); idx += 32) {
                    const int rr = idx / (D / 8), pc = idx % (D / 8);
                    if (key + rr < w.k0 || key + rr >= w.k1)
                        *reinterpret_cast<uint4 *>(vg + sw128<D>(rr, pc)) = make_uint4(0, 0, 0, 0);
                }
                __syncwarp();
            }
            // S = Q K^T (n-tiles of 8 keys)
            constexpr int NT = KS / 8;
            float sc[NT][4];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                sc[nt][0] = sc[nt][1] = sc[nt][2] = sc[nt][3] = 0.f;
                const int row = 8 * nt + (lane & 7);
#pragma unroll
                for (int k2 = 0; k2 < D / 32; ++k2) {
                    uint32_t b0, b1, b2, b3;
                    ldsm_x4(ks + sw128<D>(row, k2 * 4 + (lane >> 3)), b0, b1, b2, b3);
                    mma_bf16_16816(sc[nt], qa[2 * k2], b0, b1);
                    mma_bf16_16816(sc[nt], qa[2 * k2 + 1], b2, b3);
                }
            }
            // (a row keeps every key of most steps)
            const bool whole = __all_sync(0xffffffffu, !edge && key >= lo0 && key >= lo1 && key + KS <= hi0 && key + KS <= hi1);
            float mx0 = -INFINITY, mx1 = -INFINITY;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int s = key + 8 * nt + kq + (e & 1);
                    const bool keep = whole || (s >= w.k0 && s < (e < 2 ? hi0 : hi1) && (s >= (e < 2 ? lo0 : lo1) || s < a.n_sink));
                    sc[nt][e] = keep ? sc[nt][e] * a.scale_log2 : -INFINITY;
                }
                mx0 = fmaxf(mx0, fmaxf(sc[nt][0], sc[nt][1]));
                mx1 = fmaxf(mx1, fmaxf(sc[nt][2], sc[nt][3]));
            }
#pragma unroll
            for (int o = 1; o <= 2; o <<= 1) {
                mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, o));
                mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, o));
            }
            const float mn0 = fmaxf(m0, mx0), mn1 = fmaxf(m1, mx1);
            const float ms0 = mn0 == -INFINITY ? 0.f : mn0, ms1 = mn1 == -INFINITY ? 0.f : mn1;
            const float al0 = ex2(m0 - ms0), al1 = ex2(m1 - ms1);  // (of nothing yet: 0)
            if (__any_sync(0xffffffffu, mn0 > m0 || mn1 > m1)) {
#pragma unroll
                for (int n = 0; n < D / 8; ++n) {
                    acc[n][0] *= al0;
                    acc[n][1] *= al0;
                    acc[n][2] *= al1;
                    acc[n][3] *= al1;
                }
            }
            m0 = mn0;
            m1 = mn1;
            float s0 = 0.f, s1 = 0.f;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                sc[nt][0] = ex2(sc[nt][0] - ms0);
                sc[nt][1] = ex2(sc[nt][1] - ms0);
                sc[nt][2] = ex2(sc[nt][2] - ms1);
                sc[nt][3] = ex2(sc[nt][3] - ms1);
                s0 += sc[nt][0] + sc[nt][1];
                s1 += sc[nt][2] + sc[nt][3];
            }
            l0 = l0 * al0 + s0;
            l1 = l1 * al1 + s1;
            // O += P V (V^T fragments via transposing ldmatrix)
#pragma unroll
            for (int kk = 0; kk < NT / 2; ++kk) {
                const uint32_t pa[4] = {pack_bf16x2(sc[2 * kk][0], sc[2 * kk][1]), pack_bf16x2(sc[2 * kk][2], sc[2 * kk][3]),
                                        pack_bf16x2(sc[2 * kk + 1][0], sc[2 * kk + 1][1]),
                                        pack_bf16x2(sc[2 * kk + 1][2], sc[2 * kk + 1][3])};
                const int vrow = 16 * kk + 8 * ((lane >> 3) & 1) + (lane & 7);
#pragma unroll
                for (int d2 = 0; d2 < D / 16; ++d2) {
                    uint32_t b0, b1, b2, b3;
                    ldsm_x4_t(vs + sw128<D>(vrow, 2 * d2 + (lane >> 4)), b0, b1, b2, b3);
                    mma_bf16_16816(acc[2 * d2], pa, b0, b1);
                    mma_bf16_16816(acc[2 * d2 + 1], pa, b2, b3);
                }
            }
            // the stage is free: this warp's zeroed rows before the next copy into it
            if (edge) fence_proxy_async_smem();
            __syncwarp();
            ++taken;
            if (at < w.steps) {
                if ((at & (window - 1)) == 0) pages = pages_of(w, at);
                issue(w, at++, pages);
            } else if (next_at < next.steps && next_at < window) {
                issue(next, next_at++, next_pages);
            }
        }
        if (!ok) break;
        // ---- the result, unnormalised
#pragma unroll
        for (int o = 1; o <= 2; o <<= 1) {
            l0 += __shfl_xor_sync(0xffffffffu, l0, o);
            l1 += __shfl_xor_sync(0xffffffffu, l1, o);
        }
        const PartResults &pt = w.part ? sa.few_prefix : sa.part[0];
        const int64_t at0 = static_cast<int64_t>(w.first + tok0) * a.H_q + h0, at1 = static_cast<int64_t>(w.first + tok1) * a.H_q + h1;
        const bool there = SWA_IN_BOUNDS(w.first + w.q0 >= 0 && w.first + w.q0 + w.n <= pt.planes * pt.tokens && h1 < a.H_q, &g_rows_err);
        if (v0 && there) {
#pragma unroll
            for (int n = 0; n < D / 8; ++n)
                *reinterpret_cast<float2 *>(pt.o + at0 * D + 8 * n + kq) = make_float2(acc[n][0], acc[n][1]);
            if ((lane & 3) == 0) pt.ml[at0] = make_float2(m0, l0);
        }
        if (v1 && there) {
#pragma unroll
            for (int n = 0; n < D / 8; ++n)
                *reinterpret_cast<float2 *>(pt.o + at1 * D + 8 * n + kq) = make_float2(acc[n][2], acc[n][3]);
            if ((lane & 3) == 0) pt.ml[at1] = make_float2(m1, l1);
        }
        w = next;
        pages = next_pages;
        at = next_at;
    }
    if (!ok && lane == 0)
        for (int i = max(0, issued - NST); i < issued; ++i)
            if (i >= taken) mbar_drain(bar(i % NST), (i / NST) & 1, &g_rows_err);
    // (what waits for this grid waits for the prefix part, too)
    asm volatile("griddepcontrol.wait;" ::: "memory");
}

template <int D>
cudaError_t launch_d(const SharedArgs &sa, bool behind_tiles, cudaStream_t s) {
    using C = RowsCfg<D>;
    // the dynamic shared-memory limit is a per-device function attribute: set once per device
    static std::atomic<bool> configured[64];
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess || dev >= 64) dev = -1;
    if (dev < 0 || !configured[dev].load(std::memory_order_acquire)) {
        cudaError_t e = cudaFuncSetAttribute(paged_rows_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
        if (e != cudaSuccess) return e;
        if (dev >= 0) configured[dev].store(true, std::memory_order_release);
    }
    CUtensorMap mk, mv;
    const int box = std::min(sa.a.ps, C::KS);
    if (!paged_pool_map(&mk, sa.a, sa.a.k_pages, box) || !paged_pool_map(&mv, sa.a, sa.a.v_pages, box))
        return cudaErrorInvalidValue;
    return launch_dependent(true, paged_rows_kernel<D>, dim3(paged_sm_count() * C::CTAS_PER_SM), C::WARPS * 32, C::SMEM, s, mk,
                            mv, sa, static_cast<int>(behind_tiles), fault_plan().split_stop_stage);
}

}  // namespace

int shared_rows_warps(int D) {
    return paged_sm_count() * (D <= 64    ? RowsCfg<64>::CTAS_PER_SM * RowsCfg<64>::WARPS
                               : D <= 128 ? RowsCfg<128>::CTAS_PER_SM * RowsCfg<128>::WARPS
                                          : RowsCfg<256>::CTAS_PER_SM * RowsCfg<256>::WARPS);
}

cudaError_t launch_shared_rows(const SharedArgs &sa, bool behind_tiles, cudaStream_t s) {
    switch (sa.a.D) {
        case 64: return launch_d<64>(sa, behind_tiles, s);
        case 128: return launch_d<128>(sa, behind_tiles, s);
        case 256: return launch_d<256>(sa, behind_tiles, s);
        default: return cudaErrorInvalidValue;
    }
}

unsigned int shared_rows_read_clear_error(unsigned int *data) {
    unsigned int v = 0, z = 0;
    *data = 0;
    if (cudaMemcpyFromSymbol(&v, g_rows_err, sizeof v) != cudaSuccess) return 0;
    cudaMemcpyToSymbol(g_rows_err, &z, sizeof z);
    if (cudaMemcpyFromSymbol(data, g_rows_data, sizeof z) != cudaSuccess) return v;
    cudaMemcpyToSymbol(g_rows_data, &z, sizeof z);
    return v;
}

}  // namespace swa
