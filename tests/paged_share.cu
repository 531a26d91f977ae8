// How the paged attention kernels share their work out (swa_paged.cuh), written down: each CTA's share and
// its pieces, for test_gpu_paged_share.py.  Built by that test as a library of its own.
#include "swa_paged.cuh"

namespace {

// share [CTAs][8]: first (two words), waves, tiles, left, turn, pieces written, unused.
// pieces [CTAs][most][10]: b, kvh, ut, j0, j1, tiles of the unit, slot, owner, pieces of the unit, unused.
template <int BN, int kThreads, bool kWaves>
__global__ void __launch_bounds__(kThreads) share_kernel(const __grid_constant__ swa::PagedArgs a, int TT, int min_tiles,
                                                         int most, int *shares, int *pieces, unsigned int *err) {
    extern __shared__ __align__(16) uint8_t scratch[];
    __shared__ swa::Share share;
    swa::find_share<BN, kThreads, kWaves>(a, TT, min_tiles, scratch, &share, err);
    __syncthreads();
    if (threadIdx.x >= 32) return;
    const int lane = threadIdx.x, c = blockIdx.x;
    swa::Share sh = share;
    if (!kWaves) sh.waves = 0;
    swa::Plan<BN> plan(a, TT, sh);
    swa::Piece p{};
    int n = 0;
    for (; n < most && plan.next(p, lane); ++n) {
        if (lane != 0) continue;
        int *o = pieces + (static_cast<int64_t>(c) * most + n) * 10;
        const int v[9] = {p.b, p.kvh, p.ut, p.j0, p.j1, p.u.n,
                          kWaves ? 2 * sh.turn + (p.begun() ? 0 : 1) : swa::piece_slot(p),
                          p.begun() ? sh.owner : sh.turn, p.begun() ? sh.pieces : p.open() ? sh.open_pieces : 0};
        for (int i = 0; i < 9; ++i) o[i] = v[i];
    }
    if (lane == 0) {
        int *o = shares + c * 8;
        o[0] = static_cast<int>(sh.first & 0x7fffffff);
        o[1] = static_cast<int>(sh.first >> 31);
        o[2] = sh.waves;
        o[3] = sh.tiles;
        o[4] = sh.left;
        o[5] = sh.turn;
        o[6] = n;
    }
}

}  // namespace

// kind 0: the few-row kernel's (tiles of 64 keys), 1 and 2: the many-row kernel's with tiles of 128 and 64.
extern "C" __attribute__((visibility("default"))) int paged_shares(int kind, int grid, int TT, int min_tiles, int most,
                                                                   const int *p0, const int *q_start, int N, int B,
                                                                   int width, int ps_log2, int H_kv, int window,
                                                                   int n_sink, int *shares, int *pieces,
                                                                   unsigned int *err) {
    swa::PagedArgs a{};
    a.p0 = p0;
    a.q_start = q_start;
    a.N = N;
    a.B = B;
    a.width = width;
    a.ps_log2 = ps_log2;
    a.ps = 1 << ps_log2;
    a.H_kv = H_kv;
    a.G = 1;
    a.window = window > 0 ? window : INT_MAX;
    a.n_sink = n_sink;
    if (B < 1 || B > swa::kPagedMaxB || grid < 1 || TT < 1 || most < 1) return -1;
    const int smem = swa::kShareScratch;
    const void *fn = kind == 0   ? reinterpret_cast<const void *>(share_kernel<64, 160, false>)
                     : kind == 1 ? reinterpret_cast<const void *>(share_kernel<128, 384, true>)
                                 : reinterpret_cast<const void *>(share_kernel<64, 384, true>);
    cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return static_cast<int>(e);
    if (kind == 0) share_kernel<64, 160, false><<<grid, 160, smem>>>(a, TT, min_tiles, most, shares, pieces, err);
    else if (kind == 1) share_kernel<128, 384, true><<<grid, 384, smem>>>(a, TT, min_tiles, most, shares, pieces, err);
    else share_kernel<64, 384, true><<<grid, 384, smem>>>(a, TT, min_tiles, most, shares, pieces, err);
    e = cudaGetLastError();
    return static_cast<int>(e != cudaSuccess ? e : cudaDeviceSynchronize());
}
