// swa_paged_split.cu -- attention of few new tokens a sequence over a paged cache: at most 16
// query rows (new tokens x the heads of a group) per unit, so that every key and value byte is
// read for one unit and HBM bounds the work.
//
// Persistent kernel, several CTAs per SM, five warps.  A CTA takes its share of the batch's
// tiles of 64 keys (swa_paged.cuh) and streams it:
//   warp 0     producer: looks up the pages of a tile (one tile ahead) and copies its keys and
//              values by TMA, a copy per page (or half a page of 128) into a ring of NST stages with 128B swizzle.  A page that is not there is
//              read past the pool's end, which gives zeros.
//   warps 1-4  consumers: 16 keys of every tile each, S = Q K^T and O += P V by mma.sync, with a
//              running maximum and sum per row in the log2 domain.  P is rounded to bf16 for the
//              second product (the sum takes it unrounded).  Rows of V past the sequence's end
//              are zeroed in shared memory first, since a page's unused rows may hold anything
//              (even NaN).  At the end of a piece the four warps combine through shared memory
//              and write the rows, or the piece's partial result where the unit is shared.
// Where every sequence has one new token the producer of the CTA whose tile holds it also
// stores the token's key and value in their page, before it copies that tile.
// Every wait is bounded; on expiry the CTA records an error word, drains its copies and returns.
#include <atomic>
#include <climits>
#include <cmath>

#include "swa_paged.cuh"

namespace swa {
namespace {

__device__ unsigned int g_psplit_err = 0;   // waits and bounds
__device__ unsigned int g_psplit_data = 0;  // broken device data

constexpr int CH = 64;  // keys a tile
constexpr int kThreads = 160;
constexpr int ROWS = 16;  // mma.sync M
// Least share of a CTA.  Pieces of one tile each join as fast as pieces of four, and small batches are
// done sooner: one token behind 900 13.1 -> 12.6 us, eight behind up to 500 13.9 -> 11.5 us.
constexpr int kMinTiles = 1;

template <int D>
struct SplitCfg {
    static constexpr int STAGE = 2 * CH * D * 2;  // K and V of one tile
    static constexpr int CROW = D + 8;  // padded row: float2 stores of 4 rows per half-warp hit distinct banks
    static constexpr int CBUF = 4 * ROWS * CROW * 4;  // combine buffer [4 warps][16 rows][CROW] fp32
    static constexpr int CTAS_PER_SM = D <= 64 ? 3 : D <= 128 ? 2 : 1;
    static constexpr int NST_RAW = (232448 / CTAS_PER_SM - 2048 - CBUF) / STAGE;
    static constexpr int NST = NST_RAW > 8 ? 8 : NST_RAW;
    static constexpr int OFF_RING = 0;
    static constexpr int OFF_CBUF = NST * STAGE;
    static constexpr int OFF_RED = OFF_CBUF + CBUF;  // red_m, red_l [4][16]
    static constexpr int OFF_BAR = OFF_RED + 2 * 4 * ROWS * 4;
    // full[NST], empty[NST], cmb_full, cmb_done
    static constexpr int NBAR = 2 * NST + 2;
    static constexpr int SMEM = OFF_BAR + NBAR * 8 + 1024;
    static_assert(NST >= 2, "ring too shallow");
    static_assert(SMEM * CTAS_PER_SM <= 232448, "shared memory budget");
    // The scratch of the work split lies in the ring and the combine buffer, or, for more sequences
    // than they have room for (5631 at head dim 64), behind everything else.
    static constexpr int scratch_off(int B) { return share_scratch(B) <= OFF_RED ? 0 : SMEM - 1024; }
    static constexpr int smem(int B) { return share_scratch(B) <= OFF_RED ? SMEM : SMEM + share_scratch(B); }
    static_assert(SMEM % 8 == 0 && smem(kPagedMaxB) <= 232448, "scratch of the work split");
};

// Offset of 16-byte piece `pc` of row `row` in a 128B-swizzled tile (layout of paged_pool_map).
template <int D>
__device__ __forceinline__ uint32_t sw128(int row, int pc) {
    return static_cast<uint32_t>((row >> 3) * (D * 16) + (pc >> 3) * 1024 + (row & 7) * 128 +
                                 (((pc & 7) ^ (row & 7)) << 4));
}

template <int D>
__global__ void __maxnreg__(SplitCfg<D>::CTAS_PER_SM == 3 ? 128 : SplitCfg<D>::CTAS_PER_SM == 2 ? 168 : 255)
    paged_split_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                       const PagedArgs a, const PagedWs ws, const int TT, const int min_tiles, const int scratch_off,
                       const int fault_stop) {
    using C = SplitCfg<D>;
    constexpr int NST = C::NST;
    extern __shared__ uint8_t smem_raw[];
    __shared__ int abort_flag;
    __shared__ Share share;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t sraw = smem_u32(smem_raw);
    const uint32_t sbase = (sraw + 1023u) & ~1023u;
    uint8_t *sgen = smem_raw + (sbase - sraw);
    float *cbuf = reinterpret_cast<float *>(sgen + C::OFF_CBUF);
    float *red_m = reinterpret_cast<float *>(sgen + C::OFF_RED);
    float *red_l = red_m + 4 * ROWS;
    const uint32_t bars = sbase + C::OFF_BAR;
    auto bar_full = [&](int s) { return bars + 8u * s; };
    auto bar_empty = [&](int s) { return bars + 8u * (NST + s); };
    const uint32_t bar_cf = bars + 8u * (2 * NST), bar_cd = bars + 8u * (2 * NST + 1);

    if (tid == 0) {
        abort_flag = 0;
        for (int s = 0; s < NST; ++s) {
            mbar_init(bar_full(s), 1);
            mbar_init(bar_empty(s), 4);
        }
        mbar_init(bar_cf, 4);
        mbar_init(bar_cd, 4);
        fence_mbar_init();
    }
    if (warp == 0 && lane == 0) {
        tma_prefetch_desc(&tm_k);
        tma_prefetch_desc(&tm_v);
    }
    // (its block barriers also publish the mbarriers)
    find_share<CH, kThreads, false>(a, TT, min_tiles, sgen + scratch_off, &share, &g_psplit_data);
    volatile int *abort = &abort_flag;
    // the merge grid may be scheduled from here on: its blocks wait (griddepcontrol.wait)
    // for this grid to complete before they read the partials
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const Share sh = share;
    Walk<CH> walk(a, TT, sh);
    Piece p;

    if (warp == 0) {
        // ============================ producer ============================
        // the scratch of the work split lies in the ring: order its generic accesses before the copies
        fence_proxy_async_smem();
        asm volatile("griddepcontrol.wait;" ::: "memory");  // (the append before this kernel has stored its rows)
        int4 open = make_int4(0, 0, 0, 0);
        int seq = 0;  // stages emitted so far
        bool ok = true;
        const int box = min(a.ps, CH), npg = CH / box;  // rows of a box, boxes of a tile
        const int my_pg = lane % npg;                   // lane i looks up the page of box i % npg
        while (ok && walk.next(p)) {
            if (p.open() && !p.begun()) open = make_int4(p.u.n - p.j1, p.b, p.kvh, p.ut);
            const int t0 = p.s.p0 + p.ut * TT, t1 = p.s.p0 + min(p.s.n, (p.ut + 1) * TT) - 1;
            const int lo = t0 >= a.window ? t0 - a.window + 1 : 0;
            auto entry = [&](int j) { return page_of(a, p.b, (p.u.tile(j) * CH + my_pg * box) >> a.ps_log2); };
            int page = entry(p.j0);
#pragma unroll 1
            for (int j = p.j0; j < p.j1; ++j) {
                const int ahead = j + 1 < p.j1 ? entry(j + 1) : 0;
                if (seq >= fault_stop) {  // planted fault: this stage is never emitted
                    ok = false;
                    break;
                }
                const int k0 = p.u.tile(j) * CH, kp = k0 + my_pg * box;
                // a page that some row keeps a key of has to be there
                if (page == a.n_pages && kp <= t1 && (kp + box > lo || kp < a.n_sink))
                    atomicOr(&g_psplit_data, SWA_DEVERR_BAD_PAGE);
                const int st = seq % NST;
                if (seq >= NST) {
                    ok = __all_sync(0xffffffffu, mbar_wait<true>(bar_empty(st), ((seq / NST) - 1) & 1, abort, &g_psplit_err));
                    if (!ok) break;
                }
                if (a.kn && t1 >= k0 && t1 < k0 + CH) {
                    // the one new token: its key and value rows into their page, visible to the
                    // copy of this tile (the generic-proxy stores of every lane)
                    const int pg = __shfl_sync(0xffffffffu, page, (t1 - k0) / box);
                    if (pg < a.n_pages && SWA_IN_BOUNDS(p.s.q0 < a.N && p.kvh < a.H_kv, &g_psplit_err)) {
                        const int64_t row = ((static_cast<int64_t>(pg) * a.H_kv + p.kvh) * a.ps + (t1 & (a.ps - 1))) * D;
                        const uint4 *ks = reinterpret_cast<const uint4 *>(a.kn + p.s.q0 * a.kn_st[0] + p.kvh * a.kn_st[1]);
                        const uint4 *vs = reinterpret_cast<const uint4 *>(a.vn + p.s.q0 * a.vn_st[0] + p.kvh * a.vn_st[1]);
                        for (int pc = lane; pc < 2 * (D / 8); pc += 32) {
                            if (pc < D / 8) reinterpret_cast<uint4 *>(a.k_pages + row)[pc] = __ldg(ks + pc);
                            else reinterpret_cast<uint4 *>(a.v_pages + row)[pc - D / 8] = __ldg(vs + pc - D / 8);
                        }
                    }
                    asm volatile("fence.proxy.async.global;" ::: "memory");
                    __syncwarp();
                }
                if (lane == 0) mbar_arrive_expect_tx(bar_full(st), C::STAGE);
                __syncwarp();
                const int row = npg == 1 ? k0 & (a.ps - 1) : 0;  // (a tile may be part of one page)
                // debug build: the box lies in the page, the head exists
                (void)SWA_IN_BOUNDS(row + box <= a.ps && p.kvh < a.H_kv && page <= a.n_pages, &g_psplit_err);
                if (lane < 2 * npg) {  // keys, then values, a lane each
                    const int v = lane / npg;
                    tma_load_4d(sbase + C::OFF_RING + st * C::STAGE + v * (C::STAGE / 2) + my_pg * box * D * 2,
                                v ? &tm_v : &tm_k, bar_full(st), 0, 0, 0,
                                (page * a.H_kv + p.kvh) * (a.ps >> 3) + (row >> 3));
                }
                __syncwarp();
                ++seq;
                page = ahead;
            }
        }
        if (lane == 0) {
            ws.open[blockIdx.x] = ok ? open : make_int4(0, 0, 0, 0);
            ws.first[blockIdx.x] = sh.first;
            ws.left[blockIdx.x] = sh.left;
        }
        if (!ok && lane == 0) {
            // drain the copies still in flight (at most the last NST stages)
            for (int s = max(0, seq - NST); s < seq; ++s) mbar_drain(bar_full(s % NST), (s / NST) & 1, &g_psplit_err);
        }
    } else {
        // ============================ consumers ============================
        const int w = warp - 1;  // keys [16w, 16w + 16) of every tile
        const int r0 = lane >> 2, r1 = r0 + 8;
        const int kq = 2 * (lane & 3);
        int seq = 0, n_done = 0;
        bool ok = true;
        while (ok && walk.next(p)) {
            const int n_tok = min(p.s.n - p.ut * TT, TT), rows = n_tok * a.G;
            const int tb = p.s.p0 + p.ut * TT, t1 = tb + n_tok - 1;  // first and last token's positions
            const int end = p.s.p0 + p.s.n;
            const int tr0 = tb + r0 / a.G, tr1 = tb + r1 / a.G;
            const int lo0 = tr0 >= a.window ? tr0 - a.window + 1 : 0, lo1 = tr1 >= a.window ? tr1 - a.window + 1 : 0;
            const int lo_last = t1 >= a.window ? t1 - a.window + 1 : 0;  // keys from here on are in every row's window
            const int lo_first = tb >= a.window ? tb - a.window + 1 : 0;
            // query fragments of rows r0, r1 of the 16-row M tile
            uint32_t qa[D / 16][4];
            {
                const int64_t tok = p.s.q0 + p.ut * TT;
                const bool v0 = r0 < rows, v1 = r1 < rows;
                const auto *q0 = reinterpret_cast<const __nv_bfloat16 *>(a.q) + (tok + (v0 ? r0 / a.G : 0)) * a.q_st[0] +
                                 (p.kvh * a.G + (v0 ? r0 % a.G : 0)) * a.q_st[1];
                const auto *q1 = reinterpret_cast<const __nv_bfloat16 *>(a.q) + (tok + (v1 ? r1 / a.G : 0)) * a.q_st[0] +
                                 (p.kvh * a.G + (v1 ? r1 % a.G : 0)) * a.q_st[1];
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    qa[kk][0] = v0 ? __ldg(reinterpret_cast<const unsigned *>(q0 + kk * 16 + kq)) : 0u;
                    qa[kk][1] = v1 ? __ldg(reinterpret_cast<const unsigned *>(q1 + kk * 16 + kq)) : 0u;
                    qa[kk][2] = v0 ? __ldg(reinterpret_cast<const unsigned *>(q0 + kk * 16 + 8 + kq)) : 0u;
                    qa[kk][3] = v1 ? __ldg(reinterpret_cast<const unsigned *>(q1 + kk * 16 + 8 + kq)) : 0u;
                }
            }
            float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
            float acc[D / 8][4];
#pragma unroll
            for (int n = 0; n < D / 8; ++n) acc[n][0] = acc[n][1] = acc[n][2] = acc[n][3] = 0.f;

#pragma unroll 1
            for (int j = p.j0; j < p.j1; ++j, ++seq) {
                const int st = seq % NST;
                if (!__all_sync(0xffffffffu, mbar_wait<true>(bar_full(st), (seq / NST) & 1, abort, &g_psplit_err))) {
                    ok = false;
                    break;
                }
                const int k0 = p.u.tile(j) * CH + 16 * w;  // this warp's first key
                if (k0 <= t1 && (k0 + 15 >= lo_first || k0 < a.n_sink)) {
                    const uint32_t ks = sbase + C::OFF_RING + st * C::STAGE;
                    const uint32_t vs = ks + C::STAGE / 2;
                    if (k0 + 15 >= end || (k0 < lo_first && k0 + 15 >= a.n_sink)) {
                        // zero the value rows that no row keeps: past the sequence's end, or between the
                        // sinks and the window (they may hold anything, even NaN)
                        uint8_t *vg = sgen + C::OFF_RING + st * C::STAGE + C::STAGE / 2;
                        for (int idx = lane; idx < 16 * (D / 8); idx += 32) {
                            const int rr = idx / (D / 8), pc = idx % (D / 8);
                            if (k0 + rr >= end || (k0 + rr < lo_first && k0 + rr >= a.n_sink))
                                *reinterpret_cast<uint4 *>(vg + sw128<D>(16 * w + rr, pc)) = make_uint4(0, 0, 0, 0);
                        }
                        __syncwarp();
                    }
                    // S = Q K^T over this warp's 16 keys (two n-tiles of 8)
                    float sc[2][4];
#pragma unroll
                    for (int nt = 0; nt < 2; ++nt) {
                        sc[nt][0] = sc[nt][1] = sc[nt][2] = sc[nt][3] = 0.f;
                        const int row = 16 * w + 8 * nt + (lane & 7);
#pragma unroll
                        for (int k2 = 0; k2 < D / 32; ++k2) {
                            uint32_t b0, b1, b2, b3;
                            ldsm_x4(ks + sw128<D>(row, k2 * 4 + (lane >> 3)), b0, b1, b2, b3);
                            mma_bf16_16816(sc[nt], qa[2 * k2], b0, b1);
                            mma_bf16_16816(sc[nt], qa[2 * k2 + 1], b2, b3);
                        }
                    }
                    float mx0 = -INFINITY, mx1 = -INFINITY;
                    // every row keeps every key of this warp
                    const bool whole = k0 + 15 <= tb && (k0 >= lo_last || k0 + 15 < a.n_sink);
#pragma unroll
                    for (int nt = 0; nt < 2; ++nt) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int s = k0 + 8 * nt + kq + (e & 1);
                            const int t = e < 2 ? tr0 : tr1, lo = e < 2 ? lo0 : lo1;
                            const bool keep = whole || (s <= t && (s >= lo || s < a.n_sink));
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
                    const float al0 = mn0 == -INFINITY ? 1.f : ex2(m0 - mn0);
                    const float al1 = mn1 == -INFINITY ? 1.f : ex2(m1 - mn1);
                    m0 = mn0;
                    m1 = mn1;
                    float pr[2][4];
                    float s0 = 0.f, s1 = 0.f;
#pragma unroll
                    for (int nt = 0; nt < 2; ++nt) {
                        pr[nt][0] = mn0 == -INFINITY ? 0.f : ex2(sc[nt][0] - mn0);
                        pr[nt][1] = mn0 == -INFINITY ? 0.f : ex2(sc[nt][1] - mn0);
                        pr[nt][2] = mn1 == -INFINITY ? 0.f : ex2(sc[nt][2] - mn1);
                        pr[nt][3] = mn1 == -INFINITY ? 0.f : ex2(sc[nt][3] - mn1);
                        s0 += pr[nt][0] + pr[nt][1];
                        s1 += pr[nt][2] + pr[nt][3];
                    }
                    l0 = l0 * al0 + s0;
                    l1 = l1 * al1 + s1;
#pragma unroll
                    for (int n = 0; n < D / 8; ++n) {
                        acc[n][0] *= al0;
                        acc[n][1] *= al0;
                        acc[n][2] *= al1;
                        acc[n][3] *= al1;
                    }
                    uint32_t pa[4];
                    pa[0] = pack_bf16x2(pr[0][0], pr[0][1]);
                    pa[1] = pack_bf16x2(pr[0][2], pr[0][3]);
                    pa[2] = pack_bf16x2(pr[1][0], pr[1][1]);
                    pa[3] = pack_bf16x2(pr[1][2], pr[1][3]);
                    // O += P V (V^T fragments via transposing ldmatrix)
                    const int vrow = 16 * w + 8 * ((lane >> 3) & 1) + (lane & 7);
#pragma unroll
                    for (int d2 = 0; d2 < D / 16; ++d2) {
                        uint32_t b0, b1, b2, b3;
                        ldsm_x4_t(vs + sw128<D>(vrow, 2 * d2 + (lane >> 4)), b0, b1, b2, b3);
                        mma_bf16_16816(acc[2 * d2], pa, b0, b1);
                        mma_bf16_16816(acc[2 * d2 + 1], pa, b2, b3);
                    }
                    // order this warp's generic writes (zeroed rows) before the next TMA into the stage
                    fence_proxy_async_smem();
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(bar_empty(st));
            }
            if (!ok) break;

            // ---- combine the four warps: write the unit's rows, or this piece's partial
            float ls0 = l0, ls1 = l1;
#pragma unroll
            for (int o = 1; o <= 2; o <<= 1) {
                ls0 += __shfl_xor_sync(0xffffffffu, ls0, o);
                ls1 += __shfl_xor_sync(0xffffffffu, ls1, o);
            }
            if (n_done > 0 && !__all_sync(0xffffffffu, mbar_wait<true>(bar_cd, (n_done - 1) & 1, abort, &g_psplit_err))) {
                ok = false;
                break;
            }
            if ((lane & 3) == 0) {
                red_m[w * ROWS + r0] = m0;
                red_m[w * ROWS + r1] = m1;
                red_l[w * ROWS + r0] = ls0;
                red_l[w * ROWS + r1] = ls1;
            }
            if (r0 < rows) {
#pragma unroll
                for (int n = 0; n < D / 8; ++n)
                    *reinterpret_cast<float2 *>(cbuf + (w * ROWS + r0) * C::CROW + 8 * n + kq) =
                        make_float2(acc[n][0], acc[n][1]);
            }
            if (r1 < rows) {
#pragma unroll
                for (int n = 0; n < D / 8; ++n)
                    *reinterpret_cast<float2 *>(cbuf + (w * ROWS + r1) * C::CROW + 8 * n + kq) =
                        make_float2(acc[n][2], acc[n][3]);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(bar_cf);
            if (!__all_sync(0xffffffffu, mbar_wait<true>(bar_cf, n_done & 1, abort, &g_psplit_err))) {
                ok = false;
                break;
            }
            // eight threads per row: the row's warp weights once, then float4 columns interleaved
            // so each 8-thread phase reads 128 contiguous bytes
            const int t = w * 32 + lane, r = t >> 3, part = t & 7;
            const int64_t tok = p.s.q0 + p.ut * TT + r / a.G;
            const int h = p.kvh * a.G + r % a.G;
            // (a piece's partial result: two slots a CTA)
            if (r < rows && SWA_IN_BOUNDS(tok < a.N && h < a.H_q && piece_slot(p) < 2 * static_cast<int>(gridDim.x),
                                          &g_psplit_err)) {
                float mw = -INFINITY;
#pragma unroll
                for (int ww = 0; ww < 4; ++ww) mw = fmaxf(mw, red_m[ww * ROWS + r]);
                float f[4], L = 0.f;
#pragma unroll
                for (int ww = 0; ww < 4; ++ww) {
                    f[ww] = mw == -INFINITY ? 0.f : ex2(red_m[ww * ROWS + r] - mw);
                    L += red_l[ww * ROWS + r] * f[ww];
                }
                const bool whole = !p.begun() && !p.open();
                const float inv = 1.f / L;  // (of a whole unit: every row keeps its own key)
                const int64_t slot = static_cast<int64_t>(piece_slot(p)) * ROWS + r;
                uint16_t *o = a.o + tok * a.o_st[0] + h * a.o_st[1];
#pragma unroll
                for (int k4 = 0; k4 < D / 32; ++k4) {
                    const int col = k4 * 32 + part * 4;
                    float4 acc4 = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                    for (int ww = 0; ww < 4; ++ww) {
                        const float4 c4 = *reinterpret_cast<const float4 *>(cbuf + (ww * ROWS + r) * C::CROW + col);
                        acc4.x += c4.x * f[ww];
                        acc4.y += c4.y * f[ww];
                        acc4.z += c4.z * f[ww];
                        acc4.w += c4.w * f[ww];
                    }
                    if (whole)
                        *reinterpret_cast<uint2 *>(o + col) = make_uint2(pack_bf16x2(acc4.x * inv, acc4.y * inv),
                                                                         pack_bf16x2(acc4.z * inv, acc4.w * inv));
                    else
                        *reinterpret_cast<float4 *>(ws.acc + partial_at<D>(slot / ROWS, ROWS, r, col)) = acc4;
                }
                if (part == 0) {
                    if (whole) {
                        a.lse[tok * a.H_q + h] = (mw + log2f(L)) * 0.69314718055994531f;
                        if (a.counts) a.counts[tok * a.H_q + h] = kept_keys(a, static_cast<int>(tb + r / a.G));
                    } else {
                        *reinterpret_cast<float2 *>(ws.ml + slot * 2) = make_float2(mw, L);
                    }
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(bar_cd);
            ++n_done;
        }
    }
}

// ---------------------------------------------------------------------------------------------
// merge of the units that several CTAs share: block (c, y) takes eight rows of the unit that CTA c
// began and left open, a warp per row.  The pieces lie in the slots 2c + 1, 2(c+1), 2(c+2), ...
// A row's weight of a piece is 2^(m_piece - m), o = sum of weighted values / sum of weighted sums.
// Bound by the latency of three dependent loads; launched as a programmatic dependent of the
// kernel that wrote the pieces.
// ---------------------------------------------------------------------------------------------
constexpr int kMergeThreads = 256, kMergeRows = kMergeThreads / 32;

template <int D>
__global__ void __launch_bounds__(kMergeThreads) paged_merge_kernel(const PagedArgs a, const PagedWs w, const int ctas,
                                                                    const int TT) {
    constexpr int E = D / 32;  // columns of a lane
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int c = static_cast<int>(blockIdx.x), row = blockIdx.y * kMergeRows + warp;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int4 rec = w.open[c];
    const long long start = w.first[c];
    const int own = w.left[c];
    long long later = c + 1 + lane < ctas ? w.first[c + 1 + lane] : LLONG_MAX;
    if (rec.x == 0 || row >= TT * a.G) return;
    // the unit's tiles end at `end` of the list: CTAs c + 1 .. c + np - 1 start before that
    const long long end = start + own + rec.x;
    int np = 1;
    for (int k0 = c + 1; k0 < ctas; k0 += 32) {
        if (k0 > c + 1) later = k0 + lane < ctas ? w.first[k0 + lane] : LLONG_MAX;
        const int n = __popc(__ballot_sync(0xffffffffu, later < end));
        np += n;
        if (n < 32) break;
    }
    const Seq s = load_seq(a, rec.y);
    const int i = rec.w * TT + row / a.G;  // token of the sequence
    if (i >= s.n || !SWA_IN_BOUNDS(c + np <= ctas && rec.y < a.B && rec.z < a.H_kv, &g_psplit_err)) return;
    auto slot = [&](int k) { return static_cast<int64_t>(k == 0 ? 2 * c + 1 : 2 * (c + k)); };
    auto piece = [&](int k) { return *reinterpret_cast<const float2 *>(w.ml + (slot(k) * ROWS + row) * 2); };
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
            const float *v = w.acc + partial_at<D>(slot(k0 + k), ROWS, row, lane * E);
            // (a piece that kept nothing of this row has weight 0 and finite values)
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
    const int h = rec.z * a.G + row % a.G;
    if (!SWA_IN_BOUNDS(tok < a.N && h < a.H_q, &g_psplit_err)) return;
    const float inv = 1.f / L;  // every row keeps its own key
    uint16_t *op = a.o + tok * a.o_st[0] + h * a.o_st[1] + lane * E;
#pragma unroll
    for (int e = 0; e < E; e += 2) *reinterpret_cast<uint32_t *>(op + e) = pack_bf16x2(acc[e] * inv, acc[e + 1] * inv);
    if (lane == 0) {
        a.lse[tok * a.H_q + h] = (m + log2f(L)) * 0.69314718055994531f;
        if (a.counts) a.counts[tok * a.H_q + h] = kept_keys(a, s.p0 + i);
    }
}

template <int D>
cudaError_t launch_d(const PagedArgs &a, const PagedWs &w, bool after_append, cudaStream_t s) {
    using C = SplitCfg<D>;
    // the dynamic shared-memory limit is a per-device function attribute: set once per device
    static std::atomic<bool> configured[64];
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess || dev >= 64) dev = -1;
    if (dev < 0 || !configured[dev].load(std::memory_order_acquire)) {
        cudaError_t e = cudaFuncSetAttribute(paged_split_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             C::smem(kPagedMaxB));
        if (e != cudaSuccess) return e;
        if (dev >= 0) configured[dev].store(true, std::memory_order_release);
    }
    CUtensorMap mk, mv;
    const int rows = a.ps < CH ? a.ps : CH;
    if (!paged_pool_map(&mk, a, a.k_pages, rows) || !paged_pool_map(&mv, a, a.v_pages, rows))
        return cudaErrorInvalidValue;
    const PagedShape x = paged_split_shape(a);
    return launch_dependent(after_append, paged_split_kernel<D>, dim3(x.ctas), kThreads, C::smem(a.B), s, mk, mv, a, w,
                            x.TQ, kMinTiles, C::scratch_off(a.B), fault_plan().split_stop_stage);
}

}  // namespace

PagedShape paged_split_shape(const PagedArgs &a) {
    const int per_sm = a.D <= 64    ? SplitCfg<64>::CTAS_PER_SM
                       : a.D <= 128 ? SplitCfg<128>::CTAS_PER_SM
                                    : SplitCfg<256>::CTAS_PER_SM;
    return PagedShape{paged_sm_count() * per_sm, 1, ROWS, ROWS / a.G};
}

cudaError_t launch_paged_split(const PagedArgs &a, const PagedWs &w, bool after_append, cudaStream_t s) {
    switch (a.D) {
        case 64: return launch_d<64>(a, w, after_append, s);
        case 128: return launch_d<128>(a, w, after_append, s);
        case 256: return launch_d<256>(a, w, after_append, s);
        default: return cudaErrorInvalidValue;
    }
}

cudaError_t launch_paged_merge(const PagedArgs &a, const PagedWs &w, const PagedShape &x, cudaStream_t s) {
    const dim3 grid(x.ctas, (x.TQ * a.G + kMergeRows - 1) / kMergeRows);
    switch (a.D) {
        case 64: return launch_dependent(true, paged_merge_kernel<64>, grid, kMergeThreads, 0, s, a, w, x.ctas, x.TQ);
        case 128: return launch_dependent(true, paged_merge_kernel<128>, grid, kMergeThreads, 0, s, a, w, x.ctas, x.TQ);
        case 256: return launch_dependent(true, paged_merge_kernel<256>, grid, kMergeThreads, 0, s, a, w, x.ctas, x.TQ);
        default: return cudaErrorInvalidValue;
    }
}

void paged_split_read_clear_error(unsigned int *data, unsigned int *wait) {
    unsigned int z = 0;
    *data = *wait = 0;
    if (cudaMemcpyFromSymbol(wait, g_psplit_err, sizeof z) != cudaSuccess) return;
    cudaMemcpyToSymbol(g_psplit_err, &z, sizeof z);
    if (cudaMemcpyFromSymbol(data, g_psplit_data, sizeof z) != cudaSuccess) return;
    cudaMemcpyToSymbol(g_psplit_data, &z, sizeof z);
}

}  // namespace swa
