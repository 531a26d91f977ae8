// swa_paged_tile.cu -- attention of many new tokens over a paged cache on 5th-generation tensor
// cores (sm_103a).
//
// Work unit: one (sequence, kv head, block of one or two query tiles).  A query tile is 128 rows = TQ
// consecutive new tokens x the G query heads of the group (row = token * G + head), so every
// key/value tile is loaded once for the whole group.  A unit reads the tiles of BN keys that its
// tokens reach; the batch's tiles are shared out evenly over one persistent CTA per SM
// (swa_paged.cuh), a part of a unit that a CTA has is a piece.
// Roles:
//   warps 0, 2    producers of the keys and of the values: K_0, V_0, K_1, V_1, ... of every piece into
//                 a ring of NSLOT shared-memory slots by TMA, one copy per page (or part of one), one
//                 lane each; the pages are looked up 32 copies ahead.  Pages that no row keeps a key
//                 of, or that are not there, read past the pool: zeros.  Two warps, since a copy takes 77 cycles of
//                 the warp that issues it and a tile on pages of 16 is 16 of them.  Every fill has
//                 its own arrival and its own release.
//   warp 1        TMEM owner and MMA issuer (warp-uniform loop, one elected lane issues):
//                   S  = Q K_j^T (A = Q from shared memory, at head dim 256 from tensor memory)
//                   O += P V_j   (A = P from tensor memory)
//   warp 3        planner: finds the CTA's pieces, up to NP ahead of the others, and hands them over
//                 through shared memory, so that no other role spends its time on that; it also
//                 loads the query tiles (at head dim 256 they pass through the ring, by warp 0).
//   softmax WGs   NQT warpgroups; one row per thread (TMEM lane).  Running max in the log2
//                 domain; P = 2^(x - m) is rounded to bf16 over the S columns it came from, the
//                 row sum takes it unrounded; O is rescaled in TMEM only when a row's max grows by
//                 more than 2^8 (numerator and denominator share the stale max, so the result is
//                 the same either way).
// Head dim 128, a unit of two query tiles: they ping-pong -- while one warpgroup turns S_A into P_A
//   the tensor cores run S_B and P_B V -- with TMEM S_A | S_B | O_A | O_B.
// Head dim <= 128, a unit of one query tile: the warpgroups share it and take its key tiles in turn,
//   each with its own S, O, maximum and sum, which meet in the epilogue.  With one warpgroup
//   alone S(j + 1) could not start before P(j) was used up.
// NQT = 1 (head dim 256): one query tile, S double-buffered, TMEM S0 | S1 | Q | O.  The other
//   warpgroup has the epilogues, so that the next piece's first tiles need not wait for them
//   (16384 tokens, window 1024: 223 us, 272 with the epilogues in the softmax warpgroup).
// A unit that several CTAs share: each writes its piece's unnormalised result, and the last to do so
// joins them, while the others work on.  (A kernel of its own for that cost 8 to 19 us.)
// Rows of V that no query of the sequence keeps -- past its end, or between the sinks and the
// window of its first new token -- may hold anything (even NaN, which a weight of zero does not take
// out): the warpgroup that turns such a tile's scores into P zeroes them in shared memory before
// it hands P over.
// Bound by the tensor cores and the exponentials for full units over long histories, by HBM for
// units of few rows.
// Every wait is bounded; on expiry the CTA records an error word, drains its copies and MMAs,
// frees TMEM and returns.
#include <atomic>
#include <climits>
#include <cmath>

#include "swa_paged.cuh"

namespace swa {
namespace {

__device__ unsigned int g_ptile_err = 0;   // waits and bounds
__device__ unsigned int g_ptile_data = 0;  // broken device data

constexpr int BM = 128;              // query rows per tile (TMEM lanes)
constexpr float kRescaleTau = 8.0f;  // log2 units: rescale O when the max grows by > 2^8

// A piece as the planner hands it to the other roles: tiles j0 .. j1 - 1 of unit (b, kvh, ut),
// which has nt; q0, n, p0 of its sequence.  j0 == j1: there are no more.  slot: where its partial
// result goes; the unit's others lie in 2 * owner + 1, 2 * owner + 2, 2 * owner + 4, ...: `pieces`.
struct TilePiece {
    int b, kvh, ut, q0, n, p0, sink, lo, nt, j0, j1, slot, owner, pieces;
    __device__ __forceinline__ int tile(int i) const volatile { return j0 + i < sink ? j0 + i : lo + (j0 + i - sink); }
    __device__ __forceinline__ bool open() const volatile { return j1 < nt; }
};

template <int D>
struct TileCfg {
    static constexpr int NQT = D <= 128 ? 2 : 1;    // softmax warpgroups
    static constexpr bool kPairs = D == 128;        // units of two query tiles, too
    static constexpr int BN = D == 256 ? 64 : 128;  // keys per K/V tile
    // Twelve warps put three on each SM sub-partition, whose 16K-register file caps the launch at
    // 168 registers a thread; setmaxnreg then moves registers from warpgroup 0 (104) to the other
    // two (200): 128 * 104 + 256 * 200 = 64512 = 384 * 168.
    static constexpr int THREADS = 384;
    static constexpr int SOFTMAX_WARP0 = 4;
    static constexpr int REG_CTRL = 104, REG_SOFTMAX = 200;
    static_assert(128 * REG_CTRL + 256 * REG_SOFTMAX <= THREADS * 168, "register split");
    static constexpr int QBYTES = BM * D * 2;  // one query tile
    static constexpr int TBYTES = BN * D * 2;  // one K or V tile
    static constexpr int OFF_Q = 0;
    static constexpr int OFF_RING = NQT == 2 ? NQT * QBYTES : 0;
    static constexpr int XBYTES = NQT * BM * 8;  // (max, sum) of the softmax warpgroups' rows
    static constexpr int NSLOT_RAW = (232448 - 512 - XBYTES - OFF_RING) / TBYTES;
    // K/V ring.  At head dim 256 the query tile, which the MMAs read from tensor memory, passes
    // through it as two fills of its own instead of holding two slots' worth of shared memory:
    // seven slots instead of five.
    static constexpr int NSLOT = D == 64 ? 10 : NSLOT_RAW;
    static_assert(NQT == 2 || QBYTES == 2 * TBYTES, "a query tile is two fills");
    static constexpr int OFF_X = OFF_RING + NSLOT * TBYTES;
    static constexpr int OFF_BAR = OFF_X + XBYTES;
    // q_full[2], q_empty[2], kv_full[NSLOT], kv_empty[NSLOT], s_full[3], p_full[3], o_done[2],
    // o_free[2], meet, drain, piece_full[NP], piece_empty[NP]
    static constexpr int NP = 4;  // pieces planned ahead
    static constexpr int NBAR = 2 * NSLOT + 16 + 2 * NP;
    static constexpr int OFF_TMEMPTR = OFF_BAR + NBAR * 8;  // TMEM address, abort flag
    static constexpr int OFF_SHARE = OFF_TMEMPTR + 16;
    static constexpr int OFF_PIECE = OFF_SHARE + 64;
    // (all of it: the kernel has no static shared memory)
    static constexpr int SMEM = OFF_PIECE + NP * static_cast<int>(sizeof(TilePiece));
    static_assert(sizeof(Share) <= 64, "share");
    static constexpr uint32_t TMEM_COLS = 512;
    // S slots: two, or three where tensor memory has room (head dim 64), so that S(j + 2) is there
    // when the warpgroup that had tile j is done with it (8192 tokens behind 8000: 910 -> 816 us; now 704)
    static constexpr int NS = D == 64 ? 3 : 2;
    __host__ __device__ static constexpr uint32_t tm_s(int slot) { return static_cast<uint32_t>(slot * BN); }
    __host__ __device__ static constexpr uint32_t tm_o(int tile) {
        return D == 64 ? 384u + static_cast<uint32_t>(tile * 64) : 256u + static_cast<uint32_t>(tile * 128);
    }
    static constexpr bool QTM = NQT == 1;  // the query tile in tensor memory, 128 columns
    static constexpr uint32_t TM_Q = 128;
    static_assert(NSLOT >= 3, "K/V ring too shallow");
    static_assert(D == 128 || NSLOT >= (D == 64 ? 8 : 7), "a slot's next release waits for P (the rescaling's wait)");
    // Waits name a phase by its parity.  A softmax warp that zeroes value rows waits for the copy of
    // V(g) when it has seen the scores of the tile before it took (g - 2 where two warpgroups share a query
    // tile, g - 1 at head dim 256).  The fill that the slot had before, K(g - (NSLOT - 1) / 2) in an odd
    // ring, V(g - NSLOT / 2) in an even one, must have landed by then: scores come from landed keys,
    // and are issued behind P V of the tile NS before theirs, so behind its values' landing.
    static constexpr int SEEN = NQT == 2 ? 2 : 1;  // the tile whose scores were seen: g - SEEN
    static_assert(NSLOT % 2 ? (NSLOT - 1) / 2 >= SEEN : NSLOT / 2 >= SEEN + NS, "the wait before value rows are zeroed");
    static_assert(SMEM <= 232448, "shared memory budget");
    static_assert(NSLOT * TBYTES >= kShareScratch, "scratch of the work split");
    static_assert(!QTM || (tm_s(1) + BN <= TM_Q && TM_Q + D / 2 <= tm_o(0)), "query tile in tensor memory");
    static_assert(tm_o(NQT - 1) + D <= TMEM_COLS && tm_s(NS - 1) + BN <= tm_o(0), "tensor memory budget");
};

struct TileArgs {
    PagedArgs a;
    PagedWs ws;
    int TQ;             // tokens per query tile
    int TT;             // tokens per unit: TQ or (head dim 128) 2 * TQ
    int min_tiles;      // least share of a CTA
    int o_align32;      // o and its strides are 32-byte aligned: rows stored 32 bytes at a time
    int fault_stop_fill;  // planted fault: no ring fill numbered at or past this (INT_MAX: off)
};

// Every lane waits (each acquires the barrier); the warp proceeds only if all did,
// so the .sync.aligned tcgen05 instructions that follow stay convergent.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int *abort) {
    const bool ok = mbar_wait(bar, parity, abort, &g_ptile_err);
    return __all_sync(0xffffffffu, ok);
}

// 16 columns of a row of o (align32: 32-byte aligned).  32-byte stores: each lane of a
// store writes one whole sector of its row.
__device__ __forceinline__ void store_row16(uint16_t *dst, const float *f, bool align32) {
    uint32_t wv[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) wv[e] = pack_bf16x2(f[2 * e], f[2 * e + 1]);
    if (align32) {
        st_global_v8(dst, wv);
    } else {
        reinterpret_cast<uint4 *>(dst)[0] = make_uint4(wv[0], wv[1], wv[2], wv[3]);
        reinterpret_cast<uint4 *>(dst)[1] = make_uint4(wv[4], wv[5], wv[6], wv[7]);
    }
}

template <int D>
__global__ void __launch_bounds__(TileCfg<D>::THREADS, 1)
    paged_tile_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                      const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ TileArgs ta) {
    using C = TileCfg<D>;
    constexpr int BN = C::BN, NSLOT = C::NSLOT, NQT = C::NQT;
    const PagedArgs &a = ta.a;
    extern __shared__ __align__(1024) uint8_t sgen[];

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t sbase = smem_u32(sgen);
    if (sbase & 1023u) {  // (the swizzled tiles rely on it)
        if (tid == 0) atomicOr(&g_ptile_err, kErrBounds);
        return;
    }

    const uint32_t sQ = sbase + C::OFF_Q, sRing = sbase + C::OFF_RING;
    const uint32_t bars = sbase + C::OFF_BAR;
    auto bar_qf = [&](int x) { return bars + 8u * x; };
    auto bar_qe = [&](int x) { return bars + 8u * (2 + x); };
    auto bar_full = [&](int s) { return bars + 8u * (4 + s); };
    auto bar_empty = [&](int s) { return bars + 8u * (4 + NSLOT + s); };
    auto bar_sf = [&](int i) { return bars + 8u * (4 + 2 * NSLOT + i); };
    auto bar_pf = [&](int i) { return bars + 8u * (7 + 2 * NSLOT + i); };
    auto bar_od = [&](int i) { return bars + 8u * (10 + 2 * NSLOT + i); };
    auto bar_of = [&](int i) { return bars + 8u * (12 + 2 * NSLOT + i); };
    const uint32_t bar_meet = bars + 8u * (14 + 2 * NSLOT);
    const uint32_t bar_drain = bars + 8u * (15 + 2 * NSLOT);
    auto bar_piece = [&](int i) { return bars + 8u * (16 + 2 * NSLOT + i); };
    auto bar_used = [&](int i) { return bars + 8u * (16 + 2 * NSLOT + C::NP + i); };
    // Ring fills, numbered over the CTA's share; fill p lies in slot p % NSLOT, phase (p / NSLOT) & 1
    // of the slot's barriers.  A piece's query tile comes first at head dim 256 (two fills), then K
    // and V of each of its tiles: kfill is K of the share's g-th tile, in its k-th piece, V the next.
    auto fphase = [&](int p) -> uint32_t { return static_cast<uint32_t>((p / NSLOT) & 1); };
    auto kfill = [&](int k, int g) { return (NQT == 1 ? 2 * (k + 1) : 0) + 2 * g; };
    Share *share = reinterpret_cast<Share *>(sgen + C::OFF_SHARE);
    volatile int *abort = reinterpret_cast<volatile int *>(sgen + C::OFF_TMEMPTR + 4);
    volatile uint32_t *tmem_holder = reinterpret_cast<volatile uint32_t *>(sgen + C::OFF_TMEMPTR);

    // ---- setup: barriers, TMEM (once per CTA), this CTA's share
    if (tid == 0) {
        *abort = 0;
        for (int x = 0; x < 2; ++x) {
            mbar_init(bar_qf(x), 1);
            mbar_init(bar_qe(x), 4);  // the four warps of a softmax warpgroup
            mbar_init(bar_od(x), 1);
            mbar_init(bar_of(x), 4);
        }
        for (int x = 0; x < 3; ++x) {
            mbar_init(bar_sf(x), 1);
            mbar_init(bar_pf(x), 4);
        }
        for (int s = 0; s < NSLOT; ++s) {
            mbar_init(bar_full(s), 1);
            mbar_init(bar_empty(s), 1);
        }
        for (int i = 0; i < C::NP; ++i) {
            mbar_init(bar_piece(i), 1);
            // the roles' warps: producers, MMA, softmax, epilogue and (two query tiles) the query loader
            mbar_init(bar_used(i), 2 + NQT + 8);
        }
        mbar_init(bar_meet, 4 * NQT);
        mbar_init(bar_drain, 1);
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(const_cast<uint32_t *>(tmem_holder)), C::TMEM_COLS);
        tmem_relinquish();
    }
    if (warp == 0 && lane == 0) {
        tma_prefetch_desc(&tm_q);
        tma_prefetch_desc(&tm_k);
        tma_prefetch_desc(&tm_v);
    }
    const int TT = ta.TT;
    tc_fence_before();
    // (its block barriers also publish the mbarriers and the TMEM address)
    find_share<BN, C::THREADS, true>(a, TT, ta.min_tiles, sgen + C::OFF_RING, share, &g_ptile_data);
    tc_fence_after();
    const uint32_t tmem = *tmem_holder;
    const int cta_tiles = share->tiles;
    volatile TilePiece *pieces = reinterpret_cast<volatile TilePiece *>(sgen + C::OFF_PIECE);
    // This warp's k-th piece (nullptr: there are no more, or a wait ran out: then ok is false); the
    // warp gives it back once it has read all it needs of it.
    auto get_piece = [&](int k, bool &ok) -> volatile TilePiece * {
        if (!warp_wait(bar_piece(k % C::NP), (k / C::NP) & 1, abort)) {
            ok = false;
            return nullptr;
        }
        volatile TilePiece *p = pieces + k % C::NP;
        return p->j1 > p->j0 ? p : nullptr;
    };
    auto give_back = [&](int k) {
        __syncwarp();
        if (lane == 0) mbar_arrive(bar_used(k % C::NP));
    };
    // a unit of one query tile, which both warpgroups share (tokens: of its sequence)
    auto is_single = [&](int tokens, int ut) {
        return NQT == 2 && (!C::kPairs || TT == ta.TQ || tokens - ut * TT <= ta.TQ);
    };

    if (warp == 0 || warp == 2) {
        // ============================ K/V producers ============================
        regs_dec<C::REG_CTRL>();
        // the scratch of the work split lies in the ring: order its generic accesses before the copies
        fence_proxy_async_smem();
        asm volatile("griddepcontrol.wait;" ::: "memory");  // (the append before this kernel has stored its rows)
        // A tile is npg boxes (pages or a part of one).  The pages are looked up 32 boxes at a time,
        // lane i that of box i, a group ahead of their use.
        const int box = min(a.ps, BN), npg = BN / box, per_group = 32 / npg;
        const bool values = warp == 2;
        struct Group {
            int tiles, kvh, row, entry;  // row, entry: of this lane's box
            bool need;                   // some query row keeps a key of this lane's box
            int token;                   // the piece's first token if the group starts it, else -1
        };
        bool ok = true;
        int np = 0, i = 0, n = 0;  // pieces taken, next tile of the current one, its tiles
        int b = 0, kvh = 0, lo = 0, t1 = 0, end = 0, sink = 0, t_first = 0, j0 = 0, looked = 0, token = 0;
        auto look_up = [&]() -> Group {
            if (i >= n) {
                volatile TilePiece *p = get_piece(np, ok);
                if (!p) return Group{INT_MAX, 0, 0, -1, false, -1};
                i = 0;
                n = p->j1 - p->j0;
                b = p->b;
                kvh = p->kvh;
                j0 = p->j0;
                sink = p->sink;
                t_first = p->lo;
                const int t0 = p->p0 + p->ut * TT;
                t1 = p->p0 + min(p->n, (p->ut + 1) * TT) - 1;
                lo = t0 >= a.window ? t0 - a.window + 1 : 0;
                end = p->p0 + p->n;
                token = p->q0 + p->ut * TT;
                give_back(np++);
            }
            const int tiles = min(n - i, per_group), j = j0 + i + lane / npg;
            const int kp = (j < sink ? j : t_first + (j - sink)) * BN + lane % npg * box;
            const bool there = lane < tiles * npg && kp < end;
            const int head = i == 0 ? token : -1;
            i += tiles;
            looked += tiles;
            return Group{tiles, kvh, kp & (a.ps - 1),
                         there ? __ldg(a.table + static_cast<int64_t>(b) * a.width + (kp >> a.ps_log2)) : -1,
                         there && kp <= t1 && (kp + box > lo || kp < a.n_sink), head};
        };
        // The next fill: its slot and its phase.  The loop below is kept short: beside two softmax warps
        // on its sub-partition an instruction of this warp takes about ten cycles.
        int slot = 0, fills = 0;
        uint32_t phase = 0;
        auto skip_fills = [&](int c) {
            slot += c;
            fills += c;
            if (slot >= NSLOT) {
                slot -= NSLOT;
                phase ^= 1u;
            }
        };
        int q0 = -2, q1 = -2, q2 = -2;  // where the query tiles of the last three pieces lie among the fills
        // the slot is free (its last occupant released; at first it is) and `bytes` are expected on it
        auto take_slot = [&](int bytes) -> bool {
            if (fills >= ta.fault_stop_fill) return false;  // planted fault: this fill is never issued
            if (!warp_wait(bar_empty(slot), phase ^ 1u, abort)) return false;
            if (lane == 0) mbar_arrive_expect_tx(bar_full(slot), static_cast<uint32_t>(bytes));
            __syncwarp();
            return true;
        };
        // On the way out: until this warp's copies have landed (lane 0).  The other producer may have refilled a
        // slot since, so that a full barrier is a phase further than this warp's last fill of it: then that
        // fill was released, and one that was has landed, as have all of this warp's before it.  What can still
        // be in flight is among the last NSLOT + 2 fills up to this warp's last one.
        auto drain = [&]() {
            auto own = [&](int p) -> bool {
                const bool query = NQT == 1 && (static_cast<unsigned>(p - q0) < 2u || static_cast<unsigned>(p - q1) < 2u ||
                                                static_cast<unsigned>(p - q2) < 2u);
                return query ? !values : ((p & 1) != 0) == values;
            };
            int last = fills - 1;
            while (last >= 0 && !own(last)) --last;
            const uint64_t t0 = globaltimer_ns();
#pragma unroll 1
            while (true) {
                bool later = false, all = true;
#pragma unroll 1
                for (int p = last; p >= 0 && p >= last - NSLOT - 1; --p) {
                    if (!own(p)) continue;
                    const bool released = mbar_test_wait(bar_empty(p % NSLOT), fphase(p));
                    all = all && (later || released || mbar_test_wait(bar_full(p % NSLOT), fphase(p)));
                    later = later || released;
                }
                if (all) break;
                if (globaltimer_ns() - t0 > kWaitLimitNs) {
                    atomicOr(&g_ptile_err, kErrDrainTimeout);
                    break;
                }
            }
        };
        // The copies of a tile: the lanes below npg issue one each.  (Copies that the converged warp
        // issues one after the other, by elect.sync, take 43 cycles each instead of 77, and yet made
        // every case slower: with one per column block the Mistral window on pages of 16 674 -> 748 us,
        // chunks of 2048 tokens behind 30000 1017 -> 1097 us.)
        const CUtensorMap *map = values ? &tm_v : &tm_k;
        const uint32_t my_off = sRing + static_cast<uint32_t>(lane * box * D * 2);
        Group now{0, 0, 0, 0, false, -1}, then = now;
        if (cta_tiles > 0) then = look_up();
        int at = 0, group8 = 0;  // next tile of the group; this lane's box as a group of eight rows of the pool
        if (values) skip_fills(1);
#pragma unroll 1
        for (int t = 0; t < cta_tiles && ok; ++t) {
            if (at >= now.tiles) {
                now = then;
                if (looked < cta_tiles) then = look_up();
                at = 0;
                // (a box that no row keeps a key of comes as zeros)
                const bool in_pool = now.need && static_cast<unsigned>(now.entry) < static_cast<unsigned>(a.n_pages);
                if (now.need && !in_pool) atomicOr(&g_ptile_data, SWA_DEVERR_BAD_PAGE);
                // debug build: the box lies in the page, the head exists
                (void)SWA_IN_BOUNDS(now.row + box <= a.ps && now.kvh < a.H_kv, &g_ptile_err);
                group8 = ((in_pool ? now.entry : a.n_pages) * a.H_kv + now.kvh) * (a.ps >> 3) + (now.row >> 3);
                if (NQT == 1 && now.token >= 0) {
                    // a new piece: its query tile, in two halves, comes before its first key tile
                    q2 = q1;
                    q1 = q0;
                    q0 = fills - (values ? 1 : 0);
#pragma unroll 1
                    for (int hlf = 0; hlf < 2 && ok; ++hlf) {
                        if (!values) {
                            ok = take_slot(a.G * ta.TQ * D);
                            // debug build: the tile's tokens and its group's heads exist
                            (void)SWA_IN_BOUNDS(now.token < a.N && (now.kvh + 1) * a.G <= a.H_q, &g_ptile_err);
                            if (ok && lane < D / 128)
                                tma_load_4d(sRing + slot * C::TBYTES + lane * (BM * 128), &tm_q, bar_full(slot),
                                            hlf * (D / 2) + lane * 64, now.kvh * a.G, now.token, 0);
                            __syncwarp();
                        }
                        if (ok) skip_fills(1);
                    }
                    if (!ok) break;
                }
            }
            const int from = __shfl_sync(0xffffffffu, group8, (at * npg + lane) & 31);
            ++at;
            ok = ok && take_slot(C::TBYTES);
            if (ok && lane < npg) tma_load_4d(my_off + slot * C::TBYTES, map, bar_full(slot), 0, 0, 0, from);
            __syncwarp();
            if (ok) skip_fills(2);
        }
        if (!ok && lane == 0) drain();
    } else if (warp == 1) {
        // ============================ MMA issuer ============================
        regs_dec<C::REG_CTRL>();
        constexpr uint32_t idS = idesc_bf16_f32(BM, BN, false, false);
        constexpr uint32_t idPV = idesc_bf16_f32(BM, D, false, true);
        bool ok = true, was_single = false, both = false;
        int y = 1;                  // the query tile's buffer of the last unit of one
        uint32_t nq[2] = {0, 0};    // uses of each buffer so far
        int J = 0;                  // tiles of this CTA's previous pieces
        int k = 0;                  // pieces so far
        uint32_t np0 = 0, np1 = 0;  // P tiles of each slot used so far
        // The query tiles never move: the A descriptor of every K slice of each is built once, and
        // the V slice descriptors once per tile for both P V of a full unit, since the MMA warp's
        // instruction count per tile is part of the tile period.
        constexpr bool kQDesc = !C::QTM;
        uint64_t qdesc[NQT][D / 16], vd[BN / 16];
#pragma unroll
        for (int qt = 0; qt < NQT; ++qt)
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
                qdesc[qt][kk] = kQDesc ? smem_desc(sQ + qt * C::QBYTES + (kk >> 2) * (BM * 128) + (kk & 3) * 32, 16,
                                                   1024, kSwizzle128B)
                                       : 0ull;
        auto v_descs = [&](int slot) {
            const uint64_t v0 = smem_desc(sRing + slot * C::TBYTES, 1024, D * 16, kSwizzle128B);
#pragma unroll
            for (int kk = 0; kk < BN / 16; ++kk) vd[kk] = desc_offset(v0, kk * D * 32);
        };
        auto landed = [&](int f) -> bool { return warp_wait(bar_full(f % NSLOT), fphase(f), abort); };
        // S of the key tile in ring slot ks (landed) into TMEM slot `slot` from query tile qt
        auto mma_s = [&](int slot, int qt, int ks, uint32_t q_bytes = 0) {
            tc_fence_after();
            const uint64_t b0 = smem_desc(sRing + ks * C::TBYTES, 16, D * 16, kSwizzle128B);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
                const uint64_t bd = desc_offset(b0, (kk >> 2) * 1024 + (kk & 3) * 32);
                if constexpr (C::QTM)
                    tc_mma_ts_e(tmem + C::tm_s(slot), tmem + C::TM_Q + kk * 8, bd, idS, kk > 0 ? 1u : 0u);
                else tc_mma_ss_e(tmem + C::tm_s(slot), desc_offset(qdesc[qt][kk], q_bytes), bd, idS, kk > 0 ? 1u : 0u);
            }
            tc_commit_e(bar_sf(slot));
        };
        // O_ot (+)= P(slot) V (descriptors in vd) once, if wait_v >= 0, that fill is there, then P (the last
        // to come), and for a fresh O once the epilogue of the previous piece has read it
        auto mma_pv = [&](int slot, int ot, bool first, uint32_t n_used, int wait_v) -> bool {
            if (wait_v >= 0 && !landed(wait_v)) return false;
            if (!warp_wait(bar_pf(slot), n_used & 1, abort)) return false;
            if (first && k >= 1) {
                if (!warp_wait(bar_of(ot), (k - 1) & 1, abort)) return false;
                // (of a piece of one query tile both warpgroups read both accumulators, and both finish with it;
                // asked before the first product only: behind it the first warpgroup may be done with
                // this piece, too, and its barrier two phases on)
                if (NQT == 2 && both && ot == 0 && !warp_wait(bar_of(1), (k - 1) & 1, abort)) return false;
            }
            tc_fence_after();
#pragma unroll
            for (int kk = 0; kk < BN / 16; ++kk)
                tc_mma_ts_e(tmem + C::tm_o(ot), tmem + C::tm_s(slot) + kk * 8, vd[kk], idPV, (!first || kk > 0) ? 1u : 0u);
            return true;
        };
#pragma unroll 1
        for (; ok; ++k) {
            volatile TilePiece *p = get_piece(k, ok);
            if (!p) break;
            const int n = p->j1 - p->j0;
            const bool single = is_single(p->n, p->ut);
            give_back(k);
            both = was_single || single;
            if constexpr (NQT == 2) {
                if (C::kPairs && !single) {
                    ok = warp_wait(bar_qf(0), nq[0]++ & 1, abort) && landed(2 * J);
                    if (!ok) break;
                    mma_s(0, 0, (2 * J) % NSLOT);
                    ok = warp_wait(bar_qf(1), nq[1]++ & 1, abort);
                    if (!ok) break;
                    mma_s(1, NQT - 1, (2 * J) % NSLOT);
#pragma unroll 1
                    for (int i = 0; i < n; ++i) {
                        const int f = 2 * (J + i), ks = (f + 2) % NSLOT;
                        v_descs((f + 1) % NSLOT);
                        // (the next keys are waited for here, not between the two products, where a wait leaves
                        // the tensor cores idle: 2% of the Mistral window on pages of 16)
                        ok = landed(f + 1) && (i + 1 == n || landed(f + 2)) && mma_pv(0, 0, i == 0, np0 + i, -1);
                        if (!ok) break;
                        if (i + 1 < n) {
                            mma_s(0, 0, ks);
                        } else {
                            tc_commit_e(bar_od(0));
                        }
                        ok = mma_pv(1, 1, i == 0, np1 + i, -1);
                        if (!ok) break;
                        if (i + 1 < n) mma_s(1, NQT - 1, ks);
                        else tc_commit_e(bar_od(1));
                    }
                    np0 += n;
                    np1 += n;
                } else {
                    // one query tile, its key tiles in the S slots in turn, for one warpgroup and the other
                    auto s_slot = [&](int i2) { return C::NS == 3 ? (J + i2) % 3 : i2 & 1; };
                    y ^= 1;
                    const uint32_t q_bytes = y ? C::QBYTES : 0;
                    ok = warp_wait(bar_qf(y), (y ? nq[1]++ : nq[0]++) & 1, abort) && landed(2 * J);
                    if (!ok) break;
                    mma_s(s_slot(0), 0, (2 * J) % NSLOT, q_bytes);
                    if (C::NS == 3 && n > 1) {
                        ok = landed(2 * J + 2);
                        if (!ok) break;
                        mma_s(s_slot(1), 0, (2 * J + 2) % NSLOT, q_bytes);
                    }
#pragma unroll 1
                    for (int i = 0; i < n; ++i) {
                        const int f = 2 * (J + i), x = i & 1;
                        if (i + C::NS - 1 < n) {  // an S slot whose P V is issued
                            const int fk = f + 2 * (C::NS - 1);
                            ok = landed(fk);
                            if (!ok) break;
                            mma_s(s_slot(i + C::NS - 1), 0, fk % NSLOT, q_bytes);
                        }
                        v_descs((f + 1) % NSLOT);
                        const uint32_t used = C::NS == 3 ? static_cast<uint32_t>((J + i) / 3) : x ? np1++ : np0++;
                        ok = mma_pv(s_slot(i), x, i < 2, used, f + 1);
                        if (!ok) break;
                        tc_commit_e(bar_empty((f + 1) % NSLOT));
                    }
                    if (!ok) break;
                    tc_commit_e(bar_od(0));
                    tc_commit_e(bar_od(1));
                }
                if (!ok) break;
                was_single = single;
            } else {
                // the piece's query tile into tensor memory, 16 columns per copy (the previous piece's
                // last S MMA precedes the copies in the tensor pipe), which frees its two slots
                const int fq = 2 * k + 2 * J;
                ok = landed(fq) && landed(fq + 1);
                if (!ok) break;
                tc_fence_after();
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk)
                    tc_cp_128x256b_e(tmem + C::TM_Q + kk * 8,
                                     smem_desc(sRing + ((fq + kk / (D / 32)) % NSLOT) * C::TBYTES +
                                                   (kk % (D / 32) >> 2) * (BM * 128) + (kk & 3) * 32,
                                               16, 1024, kSwizzle128B));
                tc_commit_e(bar_empty(fq % NSLOT));
                tc_commit_e(bar_empty((fq + 1) % NSLOT));
                // S of tile g, whose slot is free once it is done
                auto next_s = [&](int g) -> bool {
                    const int f = kfill(k, g), slot = f % NSLOT;
                    if (!landed(f)) return false;
                    mma_s(g & 1, 0, slot);
                    tc_commit_e(bar_empty(slot));
                    return true;
                };
                ok = next_s(J);
                if (!ok) break;
#pragma unroll 1
                for (int i = 0; i < n; ++i) {
                    const int g = J + i, fv = kfill(k, g) + 1, vs = fv % NSLOT;
                    // slot (g+1) & 1 last held P of tile g-1, consumed by its P V issued earlier
                    if (i + 1 < n) ok = next_s(g + 1);
                    if (!ok) break;
                    v_descs(vs);
                    ok = mma_pv(g & 1, 0, i == 0, static_cast<uint32_t>(g >> 1), fv);
                    if (!ok) break;
                    tc_commit_e(bar_empty(vs));
                    if (i + 1 == n) tc_commit_e(bar_od(0));
                }
            }
            J += n;
        }
        if (!ok) {
            tc_commit_e(bar_drain);
            mbar_drain(bar_drain, 0, &g_ptile_err);
        }
        __syncwarp();
    } else if (warp >= C::SOFTMAX_WARP0) {
        // ============================ softmax / epilogue ============================
        regs_inc<C::REG_SOFTMAX>();
        const int wg = (warp - C::SOFTMAX_WARP0) >> 2;
        const int quarter = warp & 3;
        const int r = quarter * 32 + lane;  // row == TMEM lane
        const uint32_t lane_addr = static_cast<uint32_t>(quarter * 32) << 16;
        // head dim 256: warpgroup 0 has the softmax, warpgroup 1 the epilogues; else each has both
        const bool takes_tiles = NQT == 2 || wg == 0;
        const int ow = NQT == 2 ? wg : 0;
        const uint32_t o_addr = tmem + lane_addr + C::tm_o(ow);
        float2 *meet = reinterpret_cast<float2 *>(sgen + C::OFF_X);
        bool ok = true;
        int J = 0, k = 0, y = 1;  // y: as the MMA warp's
        uint32_t ns = 0, n_meet = 0;  // S tiles of this warpgroup's slot so far; single pieces so far
#pragma unroll 1
        for (; ok; ++k) {
            volatile TilePiece *wk = get_piece(k, ok);
            if (!wk) break;
            const int n = wk->j1 - wk->j0;
            const bool single = is_single(wk->n, wk->ut);
            const int t = wk->p0 + wk->ut * TT + (single ? 0 : ow * ta.TQ) + r / a.G;  // this row's position
            // the tile's first position, and the first key that its last row's window keeps
            const int tlo = t - r / a.G;
            const int thi = min(tlo + ta.TQ, max(wk->p0 + wk->n, tlo + 1)) - 1;
            // tiles [ia, ib) of the piece lie in every row's window; iz is the one the sequence ends in, iw
            // the first of the window if in it or in the one before are keys that no query keeps
            int ia, ib, iz, iw;
            {
                const int lo_thi = thi >= a.window ? thi - a.window + 1 : 0;
                const int first = wk->sink - wk->j0 - wk->lo;  // index of tile x of the window: first + x
                ia = max(first + wk->lo, first + (lo_thi + BN - 1) / BN);
                ib = first + (tlo + 1) / BN;
                const int lo_p0 = wk->p0 >= a.window ? wk->p0 - a.window + 1 : 0;
                iw = lo_p0 > a.n_sink && (wk->sink > 0 || wk->lo * BN < lo_p0) ? wk->sink - wk->j0 : -8;
                iz = !wk->open() && (wk->tile(n - 1) + 1) * BN > wk->p0 + wk->n ? n - 1 : -1;
            }
            // A warp without a row hands its P over as it finds it: rows of other warps do not see it,
            // and its own are not stored.  The exponentials of one sub-partition's warps are what bounds a
            // tile, so the others' (a single token has rows in one warp of four) are not spent.
            const bool idle = __all_sync(0xffffffffu, (r / a.G >= ta.TQ) || t >= wk->p0 + wk->n);
            float m = -INFINITY, l = 0.f;
#pragma unroll 1
            for (int i = takes_tiles ? (single ? wg : 0) : n; i < n; i += single ? 2 : 1) {
                const int g = J + i;
                const int slot = C::NS == 3 ? g % 3 : NQT == 2 ? wg : (g & 1);
                const uint32_t parity = C::NS == 3 ? (g / 3) & 1 : NQT == 2 ? (ns & 1) : ((g >> 1) & 1);
                if ((i == iz || static_cast<unsigned>(iw - i) <= 1u) && (NQT == 1 || single || wg == 0)) {
                    // zero the value rows that no query keeps, in boxes that also hold others (the rest came as
                    // zeros), while S is under way.  The first P V of the tile waits for this warpgroup's P, and
                    // with two query tiles the second is issued after it.
                    const int box = min(a.ps, BN), k0 = wk->tile(i) * BN, p0 = wk->p0, end = p0 + wk->n;
                    const int lo = p0 >= a.window ? p0 - a.window + 1 : 0;
                    const bool below = k0 < lo && k0 + BN > a.n_sink, past = k0 + BN > end;
                    const int fv = kfill(k, g) + 1;
                    if ((below || past) && !warp_wait(bar_full(fv % NSLOT), fphase(fv), abort)) {
                        ok = false;
                        break;
                    }
                    uint8_t *vt = sgen + C::OFF_RING + (fv % NSLOT) * C::TBYTES;
                    auto zero = [&](int from, int to) {  // positions
                        from = min(max(from - k0, 0), BN);
                        to = min(to - k0, BN);
                        for (int idx = r; idx < (to - from) * (D / 8); idx += BM) {
                            const int row = from + idx / (D / 8), pc = idx % (D / 8);
                            *reinterpret_cast<uint4 *>(vt + (row >> 3) * (D * 16) + (pc >> 3) * 1024 + (row & 7) * 128 +
                                                       (((pc & 7) ^ (row & 7)) << 4)) = make_uint4(0, 0, 0, 0);
                        }
                    };
                    if (past) zero(end, (end + box - 1) & -box);
                    if (below) {
                        zero(a.n_sink, min(lo, (a.n_sink + box - 1) & -box));
                        zero(max(a.n_sink, lo & -box), lo);
                    }
                    if (below || past) fence_proxy_async_smem();
                }
                if (!warp_wait(bar_sf(slot), parity, abort)) {
                    ok = false;
                    break;
                }
                ++ns;
                if (NQT == 2 && !single) {
                    // the piece's last S from this query tile: the next piece's rows may load
                    if (i + 1 == n && lane == 0) mbar_arrive(bar_qe(wg));
                    // S_B(g) was the last MMA issued before this commit: every reader of K_g and of
                    // V_{g-1} is done (released here, not by more commits of the MMA warp)
                    if (wg == 1 && quarter == 0 && lane == 0) {
                        mbar_arrive(bar_empty((2 * g) % NSLOT));
                        if (i > 0) mbar_arrive(bar_empty((2 * g - 1) % NSLOT));
                    }
                    __syncwarp();  // tcgen05.ld is executed by the converged warp
                } else if (NQT == 2) {
                    // S was K_g's only reader (released here, not by a commit of the MMA warp: 8192 tokens
                    // of head dim 64 behind 8000 804 -> 782 us)
                    if (quarter == 0 && lane == 0) mbar_arrive(bar_empty((2 * g) % NSLOT));
                    __syncwarp();
                }
                tc_fence_after();
                const uint32_t s_addr = tmem + lane_addr + C::tm_s(slot);
                if (!idle) {
                float x[BN];
                {
                    uint32_t raw[BN / 32][32];
#pragma unroll
                    for (int c = 0; c < BN / 32; ++c) tmem_ld32(s_addr + c * 32, raw[c]);
                    tc_wait_ld();
#pragma unroll
                    for (int c = 0; c < BN / 32; ++c)
#pragma unroll
                        for (int e = 0; e < 32; ++e) x[c * 32 + e] = __uint_as_float(raw[c][e]);
                }
                // ---- mask: columns [lo, hi) and those of sinks (only tiles that some row cuts)
                if (i < ia || i >= ib) {
                    const int k0 = wk->tile(i) * BN;
                    const int hi = min(max(t - k0 + 1, 0), BN);
                    int lo = min(max((t >= a.window ? t - a.window + 1 : 0) - k0, 0), BN);
                    const int sk = min(max(a.n_sink - k0, 0), hi);
                    if (sk >= lo) lo = 0;
                    {
                        // 32 columns at a time, as a word of bits
#pragma unroll
                        for (int wd = 0; wd < BN / 32; ++wd) {
                            auto below = [&](int n) {  // the columns below n of this word
                                const int v = min(max(n - 32 * wd, 0), 32);
                                return v == 32 ? 0xffffffffu : (1u << v) - 1u;
                            };
                            const uint32_t keep = (below(hi) & ~below(lo)) | below(sk);
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                x[32 * wd + e] = (keep >> e) & 1u ? x[32 * wd + e] : -INFINITY;
                        }
                    }
                }
                // ---- running max (log2 domain): eight chains of three-input maxima
                float mx8[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) mx8[e] = x[e];
#pragma unroll
                for (int c = 8; c + 8 < BN; c += 16)
#pragma unroll
                    for (int e = 0; e < 8; ++e) mx8[e] = fmax3(mx8[e], x[c + e], x[c + 8 + e]);
                if constexpr ((BN / 8) % 2 == 0) {  // one column block of 8 left over
#pragma unroll
                    for (int e = 0; e < 8; ++e) mx8[e] = fmaxf(mx8[e], x[BN - 8 + e]);
                }
                const float mx = fmax3(fmax3(mx8[0], mx8[1], mx8[2]), fmax3(mx8[3], mx8[4], mx8[5]),
                                       fmaxf(mx8[6], mx8[7]));
                const float mt = mx * a.scale_log2;
                const bool need = mt > m + kRescaleTau;
                const float mu = need ? mt : m;
                const float alpha = need ? ex2(m - mu) : 1.f;  // m = -inf gives 0
                if (__any_sync(0xffffffffu, need) && i >= (single ? 2 : 1)) {
                    // O holds the P V of this piece's earlier tiles (of this warpgroup) and must be
                    // complete: with two S slots and two warpgroups S(i) was issued after them; else the
                    // release of the V slot of this warpgroup's last tile is committed right after its P V.
                    // (That slot's next release cannot come before this warp's P of tile g: with ten slots
                    // and two warpgroups it is that of V of tile g + 3, with seven and one of K of g + 3.)
                    if constexpr (C::NS == 3 || NQT == 1) {
                        const int f = kfill(k, g - NQT) + 1;
                        if (!warp_wait(bar_empty(f % NSLOT), fphase(f), abort)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                    }
#pragma unroll 1
                    for (int c = 0; c < D / 32; ++c) {
                        uint32_t ov[32];
                        tmem_ld32(o_addr + c * 32, ov);
                        tc_wait_ld();
#pragma unroll
                        for (int e = 0; e < 32; ++e) ov[e] = __float_as_uint(__uint_as_float(ov[e]) * alpha);
                        tmem_st32(o_addr + c * 32, ov);
                    }
                }
                m = mu;
                const float msub = mu == -INFINITY ? 0.f : mu;
                // ---- P = 2^(x*scale_log2 - m) as bf16 pairs over the first BN/2 S columns;
                // the scale-and-shift and the row sum run on column pairs (fp32x2)
                const uint64_t sc2 = f2_pack(a.scale_log2, a.scale_log2), nm2 = f2_pack(-msub, -msub);
                uint64_t rs2[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) rs2[e] = f2_pack(0.f, 0.f);
#pragma unroll
                for (int hlf = 0; hlf < BN / 64; ++hlf) {
                    uint32_t pk[32];
#pragma unroll
                    for (int e = 0; e < 32; ++e) {
                        float t0, t1;
                        f2_unpack(f2_fma(f2_pack(x[hlf * 64 + 2 * e], x[hlf * 64 + 2 * e + 1]), sc2, nm2), t0, t1);
                        const float p0 = ex2(t0), p1 = ex2(t1);
                        rs2[e & 3] = f2_add(rs2[e & 3], f2_pack(p0, p1));
                        pk[e] = pack_bf16x2(p0, p1);
                    }
                    tmem_st32(s_addr + hlf * 32, pk);
                }
                tc_wait_st();
                float rsum;
                {
                    const uint64_t r01 = f2_add(rs2[0], rs2[1]), r23 = f2_add(rs2[2], rs2[3]);
                    float lo, hi;
                    f2_unpack(f2_add(r01, r23), lo, hi);
                    rsum = lo + hi;
                }
                l = l * alpha + rsum;
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar_pf(slot));
            }
            if (!ok) break;
            if constexpr (NQT == 1) {
                // the rows' maxima and sums to the epilogue warpgroup, once it has read the last piece's
                if (takes_tiles) {
                    if (k > 0 && !warp_wait(bar_of(0), (k - 1) & 1, abort)) {
                        ok = false;
                        break;
                    }
                    meet[r] = make_float2(m, l);
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar_meet);
                    give_back(k);
                    J += n;
                    continue;
                }
                if (!warp_wait(bar_meet, k & 1, abort)) {
                    ok = false;
                    break;
                }
                m = meet[r].x;
                l = meet[r].y;
            }

            // ---- epilogue: O is final once the piece's last P V completes
            if (!warp_wait(bar_od(ow), k & 1, abort) || (single && !warp_wait(bar_od(wg ^ 1), k & 1, abort))) {
                ok = false;
                break;
            }
            tc_fence_after();
            if (NQT == 2 && !single && wg == 1 && quarter == 0 && lane == 0)
                mbar_arrive(bar_empty((2 * (J + n) - 1) % NSLOT));  // the piece's last value tile
            // weights of this row's two accumulators (one unless the warpgroups shared the tile)
            float wa = 1.f, wb = 0.f;
            if (single) {
                // every MMA of the piece has completed: the tile may be refilled
                y ^= 1;
                if (wg == y && lane == 0) mbar_arrive(bar_qe(y));
                // (the other warpgroup has read the last meeting's values: this piece's first P V
                // waited for both epilogues)
                meet[wg * BM + r] = make_float2(m, l);
                __syncwarp();
                if (lane == 0) mbar_arrive(bar_meet);
                if (!warp_wait(bar_meet, n_meet & 1, abort)) {
                    ok = false;
                    break;
                }
                ++n_meet;
                const float2 ma = meet[r], mb = meet[BM + r];
                m = fmaxf(ma.x, mb.x);
                wa = ma.x == -INFINITY ? 0.f : ex2(ma.x - m);
                wb = mb.x == -INFINITY ? 0.f : ex2(mb.x - m);
                l = ma.y * wa + mb.y * wb;
            }
            const int unit_pieces = wk->pieces;
            const bool whole = unit_pieces == 0;
            const float inv_l = whole ? 1.f / l : 1.f;  // (of a whole unit: every row keeps its own key)
            wa *= inv_l;
            wb *= inv_l;
            const int tq = r / a.G, i0 = wk->ut * TT + (single ? 0 : ow * ta.TQ);  // the tile's first token
            const int64_t tok = static_cast<int64_t>(wk->q0) + i0 + tq;
            const int h = wk->kvh * a.G + r % a.G;
            // debug build: the row exists; a shared unit's slots do, of this piece and of all others
            const bool store =
                tq < min(wk->n - i0, ta.TQ) &&
                SWA_IN_BOUNDS(tok < a.N && h < a.H_q &&
                                  (whole || (wk->slot >= 0 && wk->slot < 2 * static_cast<int>(gridDim.x) && wk->owner >= 0 &&
                                             wk->owner + unit_pieces <= static_cast<int>(gridDim.x))),
                              &g_ptile_err);
            uint16_t *orow = a.o + tok * a.o_st[0] + h * a.o_st[1];
            const int pslot = wk->slot, prow = (single ? 0 : ow * BM) + r;
            // (a shared query tile: each warpgroup keeps the maximum and sum beside its half of the columns)
            const int mrow = ow * BM + r;
            auto ml_at = [&](int slot) {
                return reinterpret_cast<float2 *>(ta.ws.ml + (static_cast<int64_t>(slot) * (NQT * BM) + mrow) * 2);
            };
            // a shared tile's columns are read out half by each warpgroup
            const int c0 = single ? wg * (D / 64) : 0, c1 = single ? c0 + D / 64 : D / 32;
#pragma unroll 1
            for (int c = idle ? c1 : c0; c < c1; ++c) {
                __syncwarp();  // tcgen05.ld is executed by the converged warp: lanes that store come back here
                uint32_t ov[32];
                tmem_ld32(tmem + lane_addr + C::tm_o(single ? 0 : ow) + c * 32, ov);
                tc_wait_ld();
                float f[32];
#pragma unroll
                for (int e = 0; e < 32; ++e) f[e] = __uint_as_float(ov[e]) * wa;
                if (single && n > 1) {
                    tmem_ld32(tmem + lane_addr + C::tm_o(NQT - 1) + c * 32, ov);
                    tc_wait_ld();
#pragma unroll
                    for (int e = 0; e < 32; ++e) f[e] += __uint_as_float(ov[e]) * wb;
                }
                if (store && !whole) {
#pragma unroll
                    for (int q8 = 0; q8 < 4; ++q8) {
                        uint32_t wv[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e) wv[e] = __float_as_uint(f[q8 * 8 + e]);
                        st_global_v8(ta.ws.acc + partial_at<D>(pslot, NQT * BM, prow, c * 32 + q8 * 8), wv);
                    }
                } else if (store) {
                    store_row16(orow + c * 32, f, ta.o_align32);
                    store_row16(orow + c * 32 + 16, f + 16, ta.o_align32);
                }
            }
            // O has been read out: the next piece's first P V may overwrite it
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar_of(ow));
            bool joined = false;
            if (!whole) {
                // The piece is written.  Warps of the same place have the same rows and columns of it in
                // every CTA that shares the unit, so the last of them to arrive joins those: a row's
                // weight of a piece is 2^(m_piece - m), o = sum of weighted values / sum of weighted sums.
                if (store) *ml_at(pslot) = make_float2(m, l);
                __threadfence();
                __syncwarp();
                const int owner = wk->owner;
                int before = 0;
                if (lane == 0) before = atomicAdd(ta.ws.done + owner * 8 + ow * 4 + quarter, 1);
                before = __shfl_sync(0xffffffffu, before, 0);
                joined = before == unit_pieces - 1;
                if (joined) {
                    __threadfence();
                    auto slot_of = [&](int e) { return e == 0 ? 2 * owner + 1 : 2 * (owner + e); };
                    // four pieces' loads in flight at a time
                    auto four = [&](int e0, float2 (&v)[4]) {
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            v[e] = store && e0 + e < unit_pieces ? __ldcg(ml_at(slot_of(e0 + e)))
                                                                 : make_float2(-INFINITY, 0.f);
                    };
                    float2 v4[4];
                    m = -INFINITY;
                    l = 0.f;
                    for (int e0 = 0; e0 < unit_pieces; e0 += 4) {
                        four(e0, v4);
                        const float mn = fmaxf(fmaxf(m, fmaxf(v4[0].x, v4[1].x)), fmaxf(v4[2].x, v4[3].x));
                        const float ms = mn == -INFINITY ? 0.f : mn;
                        l *= ex2(m - ms);
#pragma unroll
                        for (int e = 0; e < 4; ++e) l += v4[e].y * ex2(v4[e].x - ms);
                        m = mn;
                    }
                    const float inv = 1.f / l;  // (a row keeps its own key: some piece's maximum is finite)
                    if (unit_pieces > 4) four(0, v4);
                    if (store) {
#pragma unroll 1
                        for (int c = 2 * c0; c < 2 * c1; ++c) {  // 16 columns at a time
                            float f[16];
#pragma unroll
                            for (int e = 0; e < 16; ++e) f[e] = 0.f;
#pragma unroll 1
                            for (int e0 = 0; e0 < unit_pieces; e0 += 4) {
                                if (unit_pieces > 4) four(e0, v4);
                                float4 v[4][4];
#pragma unroll
                                for (int e = 0; e < 4; ++e)
#pragma unroll
                                    for (int x = 0; x < 4; ++x)
                                        v[e][x] = e0 + e < unit_pieces
                                                      ? __ldcg(reinterpret_cast<const float4 *>(
                                                            ta.ws.acc + partial_at<D>(slot_of(e0 + e), NQT * BM, prow,
                                                                                      c * 16 + x * 4)))
                                                      : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                                for (int e = 0; e < 4; ++e) {
                                    const float wt = ex2(v4[e].x - m) * inv;  // (0 past the last piece)
#pragma unroll
                                    for (int x = 0; x < 4; ++x) {
                                        f[4 * x] += wt * v[e][x].x;
                                        f[4 * x + 1] += wt * v[e][x].y;
                                        f[4 * x + 2] += wt * v[e][x].z;
                                        f[4 * x + 3] += wt * v[e][x].w;
                                    }
                                }
                            }
                            store_row16(orow + c * 16, f, ta.o_align32);
                        }
                    }
                }
            }
            if (store && (!single || ow == 0) && (whole || joined)) {
                a.lse[tok * a.H_q + h] = (m + log2f(l)) * 0.69314718055994531f;
                if (a.counts) a.counts[tok * a.H_q + h] = kept_keys(a, t);
            }
            give_back(k);
            J += n;
        }
    } else {
        // ============================ planner ============================
        regs_dec<C::REG_CTRL>();
        const Share sh = *share;
        bool ok = true;
        Piece p{};
        Plan<BN> plan(a, TT, sh);
        int k = 0, kq = 0;  // pieces handed over, query tiles loaded
        int loads0 = 0, loads1 = 0, y = 1;  // query tiles of each buffer; y: the last unit of one took that
        bool more = true;
#pragma unroll 1
        while (ok && (more || (NQT == 2 && kq < k))) {
            // hand over while there are free places; with query tiles to load, without waiting for one
#pragma unroll 1
            while (more) {
                const int e = k % C::NP;
                if (k >= C::NP) {
                    const uint32_t parity = (k / C::NP - 1) & 1;
                    if (NQT == 2 && kq < k) {
                        if (!__all_sync(0xffffffffu, mbar_test_wait(bar_used(e), parity))) break;
                    } else {
                        ok = warp_wait(bar_used(e), parity, abort);
                        if (!ok) break;
                    }
                }
                more = plan.next(p, lane);
                if (!more) p.j0 = p.j1 = 0;  // the end of the list
                if (lane == 0) {
                    volatile TilePiece *t = pieces + e;
                    t->b = p.b;
                    t->kvh = p.kvh;
                    t->ut = p.ut;
                    t->q0 = p.s.q0;
                    t->n = p.s.n;
                    t->p0 = p.s.p0;
                    t->sink = p.u.sink;
                    t->lo = p.u.lo;
                    t->nt = p.u.n;
                    t->j0 = p.j0;
                    t->j1 = p.j1;
                    t->slot = 2 * sh.turn + (p.begun() ? 0 : 1);
                    t->owner = p.begun() ? sh.owner : sh.turn;
                    t->pieces = p.begun() ? sh.pieces : p.open() ? sh.open_pieces : 0;
                    mbar_arrive(bar_piece(e));
                }
                __syncwarp();
                if (more) ++k;
            }
            if constexpr (NQT == 2) {
                if (!ok || kq >= k) continue;
                volatile TilePiece *t = pieces + kq % C::NP;
                const int tokens = t->n, ut = t->ut, q0 = t->q0, kvh = t->kvh;
                give_back(kq);
                const bool one = is_single(tokens, ut);
                if (one) y ^= 1;
#pragma unroll 1
                for (int x = one ? y : 0; x <= (one ? y : 1); ++x) {
                    // the S MMAs of the last tile in this buffer are done with it
                    const int before = x ? loads1 : loads0;
                    if (before > 0) ok = warp_wait(bar_qe(x), (before - 1) & 1, abort);
                    if (!ok) break;
                    if (lane == 0) {
                        const int i = ut * TT + (one ? 0 : x * ta.TQ);  // the tile's first token
                        // debug build: the tile's tokens and its group's heads exist
                        (void)SWA_IN_BOUNDS(q0 + i < a.N && (kvh + 1) * a.G <= a.H_q, &g_ptile_err);
                        mbar_arrive_expect_tx(bar_qf(x), static_cast<uint32_t>(a.G * ta.TQ * D * 2));
#pragma unroll
                        for (int c = 0; c < D / 64; ++c)
                            tma_load_4d(sQ + x * C::QBYTES + c * (BM * 128), &tm_q, bar_qf(x), c * 64, kvh * a.G, q0 + i,
                                        0);
                    }
                    __syncwarp();
                    if (x) ++loads1;
                    else ++loads0;
                }
                ++kq;
            }
        }
        if (!ok && lane == 0) {
            if (loads0 > 0) mbar_drain(bar_qf(0), (loads0 - 1) & 1, &g_ptile_err);
            if (loads1 > 0) mbar_drain(bar_qf(1), (loads1 - 1) & 1, &g_ptile_err);
        }
    }

    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, C::TMEM_COLS);
}

// Query tiles of a unit.  At head dim 128 pairs take 6% less time where there are enough of them
// (chunks of 2048 tokens behind 30000: 989 against 1047 us), and single tiles, twice as many
// units, where there are not (two chunks of 100 tokens 25 against 33 us, a mixed step 78
// against 91): pairs from two units a CTA, by what the host knows of the batch.  At head dim 64
// there was nothing between them (856 and 857 us, of what is now 704), so it has no pairs.
int tiles_of_unit(const PagedArgs &a) {
    if (a.D != 128) return 1;
    const int64_t pairs = static_cast<int64_t>(a.N) / (2 * (BM / a.G)) * a.H_kv;
    return pairs >= 2 * static_cast<int64_t>(paged_sm_count()) ? 2 : 1;
}

template <int D>
cudaError_t launch_d(const PagedArgs &a, const PagedWs &w, bool after_append, cudaStream_t s) {
    using C = TileCfg<D>;
    // the dynamic shared-memory limit is a per-device function attribute: set once per device
    static std::atomic<bool> configured[64];
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess || dev >= 64) dev = -1;
    if (dev < 0 || !configured[dev].load(std::memory_order_acquire)) {
        cudaError_t e = cudaFuncSetAttribute(paged_tile_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
        if (e != cudaSuccess) return e;
        if (dev >= 0) configured[dev].store(true, std::memory_order_release);
    }
    const PagedShape x = paged_tile_shape(a);
    const int box = a.ps < C::BN ? a.ps : C::BN;
    CUtensorMap mq, mk, mv;
    if (!paged_query_map(&mq, a, a.G, x.TQ) || !paged_pool_map(&mk, a, a.k_pages, box) ||
        !paged_pool_map(&mv, a, a.v_pages, box))
        return cudaErrorInvalidValue;
    TileArgs t{};
    t.a = a;
    t.ws = w;
    t.TQ = x.TQ;
    t.TT = x.TQ * tiles_of_unit(a);
    t.min_tiles = 4;
    t.o_align32 = reinterpret_cast<uintptr_t>(a.o) % 32 == 0 && a.o_st[0] % 16 == 0 && a.o_st[1] % 16 == 0;
    t.fault_stop_fill = fault_plan().band_stop_fill;
    return launch_dependent(after_append, paged_tile_kernel<D>, dim3(x.ctas), C::THREADS, C::SMEM, s, mq, mk, mv, t);
}

}  // namespace

PagedShape paged_tile_shape(const PagedArgs &a) {
    return PagedShape{paged_sm_count(), a.D <= 128 ? 2 : 1, BM, BM / a.G};
}

cudaError_t launch_paged_tile(const PagedArgs &a, const PagedWs &w, bool after_append, cudaStream_t s) {
    switch (a.D) {
        case 64: return launch_d<64>(a, w, after_append, s);
        case 128: return launch_d<128>(a, w, after_append, s);
        case 256: return launch_d<256>(a, w, after_append, s);
        default: return cudaErrorInvalidValue;
    }
}

void paged_tile_read_clear_error(unsigned int *data, unsigned int *wait) {
    unsigned int z = 0;
    *data = *wait = 0;
    if (cudaMemcpyFromSymbol(wait, g_ptile_err, sizeof z) != cudaSuccess) return;
    cudaMemcpyToSymbol(g_ptile_err, &z, sizeof z);
    if (cudaMemcpyFromSymbol(data, g_ptile_data, sizeof z) != cudaSuccess) return;
    cudaMemcpyToSymbol(g_ptile_data, &z, sizeof z);
}

}  // namespace swa
