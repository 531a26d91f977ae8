// swa_pages.cu -- the pages of a paged KV cache: reserving, giving back, forking,
// compacting and copying them, with the page tables and the holders' counts.
//
// A page is free when its count is 0.  Free pages are always taken lowest index first, by
// rank: the r-th page wanted (in the order of rows, then entries) is the r-th free one.
// Counts change by integer atomics, whose order cannot show in a result.
//
// Rows and entries number up to 2^31 - 1: what counts them in steps is unsigned or has 64 bits.
//
// Tables and counts are small beside the pages: they are bound by launches and latency.  The
// copies of page contents are bound by HBM (2 bytes moved per byte of page).
#include <climits>

#include "ptx.cuh"
#include "swa_paged.h"

namespace swa {
namespace {

__device__ unsigned int g_pages_err = 0;
constexpr unsigned int kErrBadPosition = SWA_DEVERR_BAD_POSITION, kErrBadPage = SWA_DEVERR_BAD_PAGE,
                       kErrNoPage = SWA_DEVERR_NO_PAGE, kErrBadRef = SWA_DEVERR_BAD_REF;

constexpr int kThreads = 256;
constexpr int kScanThreads = 1024, kScanWarps = kScanThreads / 32;
constexpr int kScanItems = 16;  // counts per thread and scan step: as many loads in flight
constexpr int kUnroll = 8;      // 16-byte loads in flight per thread of the page copy
// Blocks of the page copy per SM at most: blocks that come and go even out the end better than
// few that stay (compacting 4001 pages 320 us with 8, 315 with 16, 312 with 64 or more).
constexpr int kMoveBlocks = 64;
constexpr int kForkCtas = 8;    // a cluster (the largest portable one)
// Table entries and pages up to which one cluster plans a fork: one launch instead of three, which
// a short call waits for (32 rows of 250 entries: a call 24 -> 19 us, though 13.1 -> 14.5 us on the
// GPU); above that the copies bound the call and the grids' plan is the faster one (400 rows of
// head dim 256: 95.6 against 100 us).
constexpr int kFew = 16 * 1024;

// A kernel whose successor in the stream is launched with launch_dependent lets it be scheduled
// early; the successor waits for it (and its stores) before it reads anything.
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Debug build: `x` is an index into n (release build: true).
__device__ __forceinline__ bool within(int64_t x, int64_t n) { return SWA_IN_BOUNDS(x >= 0 && x < n, &g_pages_err); }

// One page copy: the first `rows` positions of page src go to page dst (src < 0: none).
// ref: the moved page's holders (compaction).
struct Move {
    int32_t src, dst, rows, ref;
};

struct TableArgs {
    const int32_t *table, *ref;
    int32_t *out_table, *out_ref;
    int B, width, n_pages, ps;
};

// ---------------------------------------------------------------------------------------------
// ranks of the marked items of a list, one block of kScanThreads
// ---------------------------------------------------------------------------------------------
struct ScanSmem {
    int cnt[kScanItems * kScanWarps];
    int total;
};

// One step over items base .. base + kScanItems * kScanThreads - 1 (item base + k * kScanThreads
// + tid is this thread's k-th, so loads are coalesced whatever the list's alignment).  mark(p)
// tells whether item p counts; put(p, rank) is called for each that does, ranks starting at
// `before`.  Returns the number of marked items up to the end of the step.
template <class Mark, class Put>
__device__ __forceinline__ int scan_step(ScanSmem &sm, int64_t base, int64_t n, int before, Mark mark, Put put) {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    unsigned bal[kScanItems];
    bool m[kScanItems];
#pragma unroll
    for (int k = 0; k < kScanItems; ++k) {
        const int64_t p = base + static_cast<int64_t>(k) * kScanThreads + tid;
        m[k] = p < n && mark(static_cast<int>(p));
    }
#pragma unroll
    for (int k = 0; k < kScanItems; ++k) {
        bal[k] = __ballot_sync(0xffffffffu, m[k]);
        if (lane == 0) sm.cnt[k * kScanWarps + warp] = __popc(bal[k]);
    }
    __syncthreads();
    if (warp == 0) {  // exclusive prefix of the kScanItems * kScanWarps counts
        constexpr int kPer = kScanItems * kScanWarps / 32;
        int v[kPer], s = 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            v[i] = s;
            s += sm.cnt[lane * kPer + i];
        }
        int inc = s;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int t = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += t;
        }
#pragma unroll
        for (int i = 0; i < kPer; ++i) sm.cnt[lane * kPer + i] = v[i] + inc - s;
        if (lane == 31) sm.total = inc;
    }
    __syncthreads();
    const int total = sm.total;
#pragma unroll
    for (int k = 0; k < kScanItems; ++k)
        if (m[k])
            put(static_cast<int>(base + static_cast<int64_t>(k) * kScanThreads + tid),
                before + sm.cnt[k * kScanWarps + warp] + __popc(bal[k] & ((1u << lane) - 1u)));
    __syncthreads();  // the counts are rewritten by the next step
    return before + total;
}

// The `need` lowest free pages into list[0 ..]; returns how many there are (at most need).
__device__ __forceinline__ int take_free(ScanSmem &sm, const int32_t *ref, int n_pages, int need, int32_t *list) {
    int found = 0;
    for (int64_t base = 0; base < n_pages && found < need; base += kScanItems * kScanThreads)
        found = scan_step(
            sm, base, n_pages, found, [&](int p) { return ref[p] == 0; },
            [&](int p, int r) {
                if (r < need && within(r, n_pages) && within(p, n_pages)) list[r] = p;
            });
    return min(found, need);
}

// dst = src (n), and `fill` [n_fill] all INT_MAX.
__global__ void __launch_bounds__(kThreads) copy_i32_kernel(const int32_t *src, int32_t *dst, int64_t n, int32_t *fill,
                                                            int64_t n_fill) {
    let_next_start();
    const int64_t step = static_cast<int64_t>(gridDim.x) * kThreads;
    const int64_t t = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
    for (int64_t i = t; i < n; i += step) dst[i] = src[i];
    for (int64_t i = t; i < n_fill; i += step) fill[i] = INT_MAX;
}

// ---------------------------------------------------------------------------------------------
// reserve: one block.  ws_row [B]: first rank of each row; list [n_pages]: the pages taken.
// The ranks need every row's count first, and a step of a server wants few pages: 33 rows of 300 entries,
// or 64 rows that want eight pages each, 8-10 us, the latency of the passes.  A warp has B / 32 rows one
// after the other, twice: 1024 rows 52 us, 8192 rows 415 us.
// ---------------------------------------------------------------------------------------------
__global__ void __launch_bounds__(kScanThreads) reserve_kernel(const TableArgs a, const int32_t *first,
                                                               const int32_t *end, int32_t *ws_row, int32_t *list) {
    __shared__ ScanSmem sm;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int64_t cap = static_cast<int64_t>(a.width) * a.ps;
    const uint32_t B = static_cast<uint32_t>(a.B);
    // entries [j0, j1) of row b are wanted
    auto range = [&](uint32_t b, uint32_t &j0, uint32_t &j1) {
        const int64_t f = first[b], e = end[b];
        j0 = j1 = 0;
        if (e <= f) return true;
        if (f < 0 || e > cap) return false;
        j0 = static_cast<uint32_t>(f / a.ps);
        j1 = static_cast<uint32_t>((e + a.ps - 1) / a.ps);
        return true;
    };
    auto missing = [&](uint32_t b, uint32_t j) {
        const int e = a.out_table[static_cast<int64_t>(b) * a.width + j];
        return e < 0 || e >= a.n_pages;
    };
    // 1. pages that each row lacks (a warp per row)
    for (uint32_t b = warp; b < B; b += kScanWarps) {
        uint32_t j0, j1;
        int n = 0;
        if (!range(b, j0, j1) && lane == 0) atomicOr(&g_pages_err, kErrBadPosition);
        for (uint32_t j = j0 + lane; j < j1; j += 32) {
            if (!missing(b, j)) continue;
            if (a.out_table[static_cast<int64_t>(b) * a.width + j] >= a.n_pages) atomicOr(&g_pages_err, kErrBadPage);
            ++n;
        }
        n = __reduce_add_sync(0xffffffffu, n);
        if (lane == 0) ws_row[b] = n;
    }
    __syncthreads();
    // 2. each row's first rank: an exclusive prefix over the rows
    __shared__ int wsum[kScanWarps];
    int total = 0;
    for (uint32_t b0 = 0; b0 < B; b0 += kScanThreads) {
        const uint32_t b = b0 + tid;
        const int n = b < B ? ws_row[b] : 0;
        int inc = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int t = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += t;
        }
        if (lane == 31) wsum[warp] = inc;
        __syncthreads();
        int before = 0, all = 0;
        for (int w = 0; w < kScanWarps; ++w) {
            if (w < warp) before += wsum[w];
            all += wsum[w];
        }
        if (b < B) ws_row[b] = total + before + inc - n;
        total += all;
        __syncthreads();
    }
    if (total == 0) return;
    // 3. the lowest free pages, 4. dealt to the rows in order
    const int found = take_free(sm, a.out_ref, a.n_pages, min(total, a.n_pages), list);
    __syncthreads();
    for (uint32_t b = warp; b < B; b += kScanWarps) {
        uint32_t j0, j1;
        range(b, j0, j1);
        int rank = ws_row[b];
        for (uint32_t jb = j0; jb < j1; jb += 32) {
            const uint32_t j = jb + lane;
            const bool want = j < j1 && missing(b, j);
            const unsigned bal = __ballot_sync(0xffffffffu, want);
            if (want && within(j, a.width)) {
                const int r = rank + __popc(bal & ((1u << lane) - 1u));
                int page = -1;
                if (r < found) {
                    page = within(r, a.n_pages) ? list[r] : -1;
                    if (within(page, a.n_pages)) a.out_ref[page] = 1;
                } else {
                    atomicOr(&g_pages_err, kErrNoPage);
                }
                a.out_table[static_cast<int64_t>(b) * a.width + j] = page;
            }
            rank += __popc(bal);
        }
    }
}

// ---------------------------------------------------------------------------------------------
// free: every entry once.  Bound by the atomics of a large table (1024 x 4096 entries, most of which
// go: 21 us; 23 with at most 8 blocks an SM instead of 64; 18 if the
// atomics returned nothing, but a page without a holder to lose has to be seen; four entries a
// thread, with vector loads, took as long).
// ---------------------------------------------------------------------------------------------
__global__ void __launch_bounds__(kThreads) free_kernel(const TableArgs a, const int32_t *below, int n_sink) {
    wait_for_previous();
    const uint32_t n = static_cast<uint32_t>(a.B) * static_cast<uint32_t>(a.width);  // < 2^31
    for (uint32_t x = blockIdx.x * kThreads + threadIdx.x; x < n; x += gridDim.x * kThreads) {
        const int b = static_cast<int>(x / static_cast<uint32_t>(a.width));
        const int64_t j = x - static_cast<uint32_t>(b) * static_cast<uint32_t>(a.width);
        int e = a.table[x];
        const int bl = __ldg(below + b);
        if (e >= a.n_pages) {
            atomicOr(&g_pages_err, kErrBadPage);
            e = -1;
        }
        if (e >= 0 && within(b, a.B) && within(j, a.width) && (bl < 0 || ((j + 1) * a.ps <= bl && j * a.ps >= n_sink))) {
            if (atomicSub(a.out_ref + e, 1) <= 0) {
                atomicAdd(a.out_ref + e, 1);
                atomicOr(&g_pages_err, kErrBadRef);
            }
            e = -1;
        }
        a.out_table[x] = e < 0 ? -1 : e;
    }
}

// ---------------------------------------------------------------------------------------------
// fork
// ---------------------------------------------------------------------------------------------
// The row that row i continues and its tokens (-1, 0: none).
__device__ __forceinline__ bool fork_source(const TableArgs &a, const int32_t *src, const int32_t *len, int i, int &s,
                                            int &n) {
    s = src[i];
    n = 0;
    if (s < 0) return s == -1;
    if (s >= a.B) {
        s = -1;
        return false;
    }
    n = len[s];
    if (n < 0 || n > static_cast<int64_t>(a.width) * a.ps) {
        s = -1;
        n = 0;
        return false;
    }
    return true;
}

// Who keeps a last page that is not full, and so may be written to: keep[p] becomes the lowest row
// whose last page is p, or -1 if a row has p as a full page.  Both are minima, so their order cannot
// show.  (A missing page is told apart by the row that it is missing in: keep[n_pages + s].)
// last_of[i] is row i's last page if that is not full: p, or -2 - s for a missing one; -1: none.
struct ForkWs {
    int32_t *last_of, *keep;
};
__device__ __forceinline__ bool wants_own(const TableArgs &a, const ForkWs &w, int i) {
    const int p = w.last_of[i];
    return p != -1 && w.keep[p >= 0 ? p : static_cast<int64_t>(a.n_pages) + (-2 - p)] != i;
}

// Row i keeps its own holders where both tables have the same entry (no atomics); the others change.
// Every row gets its last page here; those that want one of their own lose it again in fork_alloc.
__device__ __forceinline__ void fork_entry(const TableArgs &a, const ForkWs &w, int i, int j, int s, int part, int last) {
    if (!within(i, a.B) || !within(j, a.width) || !within(s + 1, static_cast<int64_t>(a.B) + 1)) return;
    int in = a.table[static_cast<int64_t>(i) * a.width + j];
    const bool is_last = part && j == last;
    int out = s >= 0 && (j < last || is_last) ? a.table[static_cast<int64_t>(s) * a.width + j] : -1;
    if (in >= a.n_pages || out >= a.n_pages) {
        atomicOr(&g_pages_err, kErrBadPage);
        in = in >= a.n_pages ? -1 : in;
        out = out >= a.n_pages ? -1 : out;
    }
    out = out < 0 ? -1 : out;
    if (is_last) {
        w.last_of[i] = out >= 0 ? out : -2 - s;
        atomicMin(w.keep + (out >= 0 ? out : static_cast<int64_t>(a.n_pages) + s), i);
    } else {
        if (out >= 0) *static_cast<volatile int32_t *>(w.keep + out) = -1;
        if (j == 0 && !part) w.last_of[i] = -1;
    }
    a.out_table[static_cast<int64_t>(i) * a.width + j] = out;
    if (in != out) {
        if (in >= 0) atomicSub(a.out_ref + in, 1);
        if (out >= 0) atomicAdd(a.out_ref + out, 1);
    }
}

// Rows' tables and the holders of everything but the fresh pages.  Block (x, i): a stretch of
// row i.
__global__ void __launch_bounds__(kThreads) fork_table_kernel(const TableArgs a, const int32_t *src,
                                                              const int32_t *len, const ForkWs w) {
    let_next_start();
    wait_for_previous();
    for (uint32_t y = blockIdx.y; y < static_cast<uint32_t>(a.B); y += gridDim.y) {
        const int i = static_cast<int>(y);
        int s, n;
        const bool ok = fork_source(a, src, len, i, s, n);
        if (!ok && threadIdx.x == 0 && blockIdx.x == 0) atomicOr(&g_pages_err, kErrBadPosition);
        const int part = n % a.ps, last = n / a.ps;
        for (uint32_t j = blockIdx.x * kThreads + threadIdx.x; j < static_cast<uint32_t>(a.width); j += gridDim.x * kThreads)
            fork_entry(a, w, i, static_cast<int>(j), s, part, last);
    }
}

// One block: fresh pages for the rows that want one, lowest first in the order of the rows.
__device__ __forceinline__ void fork_alloc(ScanSmem &sm, const TableArgs &a, const int32_t *src, const int32_t *len,
                                           const ForkWs &w, int32_t *row_of, int32_t *list, Move *moves,
                                           int32_t *n_moves) {
    int want = 0;
    for (int64_t base = 0; base < a.B; base += kScanItems * kScanThreads)
        want = scan_step(
            sm, base, a.B, want, [&](int i) { return wants_own(a, w, i); }, [&](int i, int r) { row_of[r] = i; });
    const int found = want ? take_free(sm, a.out_ref, a.n_pages, min(want, a.n_pages), list) : 0;
    __syncthreads();
    for (uint32_t r = threadIdx.x; r < static_cast<uint32_t>(want); r += kScanThreads) {
        if (!within(r, a.B) || !within(row_of[r], a.B) || !within(src[row_of[r]], a.B)) continue;
        const int i = row_of[r], s = src[i], n = len[s], last = n / a.ps;
        if (!within(last, a.width) || !within(r < static_cast<uint32_t>(found) ? list[r] : 0, a.n_pages)) continue;
        const int old = w.last_of[i];
        // (whoever keeps the page still holds it, so it was not among the free ones)
        if (old >= 0) atomicSub(a.out_ref + old, 1);
        Move m{-1, -1, n % a.ps, 0};
        if (r < static_cast<uint32_t>(found)) {
            m.dst = list[r];
            a.out_ref[m.dst] = 1;
            if (old >= 0) m.src = old;
            else atomicOr(&g_pages_err, kErrBadPage);
        } else {
            atomicOr(&g_pages_err, kErrNoPage);
        }
        a.out_table[static_cast<int64_t>(i) * a.width + last] = m.dst;
        moves[r] = m;
    }
    if (threadIdx.x == 0) *n_moves = want;
}

__global__ void __launch_bounds__(kScanThreads) fork_alloc_kernel(const TableArgs a, const int32_t *src,
                                                                  const int32_t *len, const ForkWs w,
                                                                  int32_t *row_of, int32_t *list, Move *moves,
                                                                  int32_t *n_moves) {
    __shared__ ScanSmem sm;
    let_next_start();
    wait_for_previous();
    fork_alloc(sm, a, src, len, w, row_of, list, moves, n_moves);
}

// All of that for small tables by one cluster, whose barriers order the counts' copy, the rows and
// the fresh pages: one launch instead of three.  A warp per 32 entries of a row.
__global__ void __cluster_dims__(kForkCtas, 1, 1) __launch_bounds__(kScanThreads)
    fork_plan_kernel(const TableArgs a, const int32_t *src, const int32_t *len, const ForkWs w, int32_t *row_of,
                     int32_t *list, Move *moves, int32_t *n_moves) {
    __shared__ ScanSmem sm;
    let_next_start();
    const int lane = threadIdx.x & 31;
    const int t = static_cast<int>(blockIdx.x) * kScanThreads + static_cast<int>(threadIdx.x);
    auto cluster_sync = [] {
        asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
    };
    for (int p = t; p < a.n_pages + a.B; p += kForkCtas * kScanThreads) {
        if (p < a.n_pages && a.ref != a.out_ref) a.out_ref[p] = a.ref[p];
        w.keep[p] = INT_MAX;
    }
    cluster_sync();
    const int parts = (a.width + 31) / 32;
    for (int u = t >> 5; u < a.B * parts; u += kForkCtas * kScanWarps) {
        const int i = u / parts, j = u % parts * 32 + lane;
        int s, n;
        const bool ok = fork_source(a, src, len, i, s, n);
        if (!ok && j == 0) atomicOr(&g_pages_err, kErrBadPosition);
        if (j < a.width) fork_entry(a, w, i, j, s, n % a.ps, n / a.ps);
    }
    cluster_sync();
    if (blockIdx.x == 0) fork_alloc(sm, a, src, len, w, row_of, list, moves, n_moves);
}

// ---------------------------------------------------------------------------------------------
// compact
// ---------------------------------------------------------------------------------------------
// One block: M, the holes below it and the live pages at or above it by rank, and their pairing.
// to[p]: where live page p >= M goes.
__global__ void __launch_bounds__(kScanThreads) compact_plan_kernel(const TableArgs a, int32_t *holes, int32_t *movers,
                                                                    int32_t *to, Move *moves, int32_t *n_moves,
                                                                    int32_t *n_live) {
    __shared__ ScanSmem sm;
    let_next_start();
    int live = 0;
    for (int64_t base = 0; base < a.n_pages; base += kScanItems * kScanThreads)
        live = scan_step(sm, base, a.n_pages, live, [&](int p) { return a.ref[p] > 0; }, [](int, int) {});
    int nh = 0, nm = 0;
    for (int64_t base = 0; base < live; base += kScanItems * kScanThreads)
        nh = scan_step(
            sm, base, live, nh, [&](int p) { return a.ref[p] <= 0; },
            [&](int p, int r) {
                if (within(r, a.n_pages)) holes[r] = p;
            });
    for (int64_t base = live; base < a.n_pages; base += kScanItems * kScanThreads)
        nm = scan_step(
            sm, base, a.n_pages, nm,
            [&](int p) {
                to[p] = -1;  // (a table entry may wrongly name a free page)
                return a.ref[p] > 0;
            },
            [&](int p, int r) {
                if (within(r, a.n_pages)) movers[r] = p;
            });
    (void)within(nm, static_cast<int64_t>(nh) + 1);
    __syncthreads();
    for (int r = threadIdx.x; r < nm; r += kScanThreads) {  // nh == nm: as many holes below M as live pages above
        const int s = movers[r], d = holes[r];
        if (!within(s, a.n_pages) || !within(d, live)) continue;
        to[s] = d;
        moves[r] = Move{s, d, a.ps, a.ref[s]};
    }
    if (threadIdx.x == 0) {
        *n_moves = nm;
        *n_live = live;
    }
}

// Tables and counts after the moves.  Each count is written by one thread, from values that no
// other thread writes (a hole's from its move), so the call may be in place.
struct ApplyArgs {
    TableArgs t;
    const int32_t *to, *n_live;
};
__device__ __forceinline__ void compact_apply(const ApplyArgs &x, const Move *moves, int nm) {
    const TableArgs &a = x.t;
    const int32_t *to = x.to;
    const int live = *x.n_live;
    const int64_t step = static_cast<int64_t>(gridDim.x) * kThreads;
    const int64_t t0 = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
    for (int64_t x = t0; x < static_cast<int64_t>(a.B) * a.width; x += step) {
        int e = a.table[x];
        const bool named = e >= 0;
        if (e >= live) e = e < a.n_pages ? to[e] : -1;
        if (named && e < 0) atomicOr(&g_pages_err, kErrBadPage);
        a.out_table[x] = e < 0 ? -1 : e;
    }
    for (int64_t p = t0; p < a.n_pages; p += step) {
        if (p >= live) a.out_ref[p] = 0;
        else if (a.ref != a.out_ref && a.ref[p] > 0) a.out_ref[p] = a.ref[p];
    }
    for (int64_t r = t0; r < nm; r += step)
        if (within(moves[r].dst, live)) a.out_ref[moves[r].dst] = moves[r].ref;
}

// ---------------------------------------------------------------------------------------------
// contents
// ---------------------------------------------------------------------------------------------
struct PoolArgs {
    uint4 *pool[2];        // keys, values
    int64_t layer_stride;  // 16-byte pieces from one layer to the next
    int L, H, n_pages, ps, row;  // row: pieces of one position
};

// What a copy's moves come from: a list of pairs, or a fork's or a compaction's plan (with the latter
// the tables and counts change in the same kernel: 24 rows on 700 pages 18.7 -> 15.5 us).
enum class Moves { kPairs, kFork, kCompact };

// A warp per (move, layer, keys or values, head): rows * row consecutive pieces of both pages.  (A
// warp per 4 KB of them was no faster: forking 400 rows of head dim 256 95 against 96 us,
// compacting 4001 pages 324 against 329 us.)  Stores are marked as not to be read again, which
// leaves L2 to pages that several copies read (those 400 rows 88 -> 84 us).
template <Moves kWhich>
__global__ void __launch_bounds__(kThreads) move_kernel(const PoolArgs a, const Move *moves, const int32_t *n_moves,
                                                        const int32_t *src, const int32_t *dst, int n_pairs,
                                                        const ApplyArgs apply) {
    constexpr bool kPairs = kWhich == Moves::kPairs;
    if constexpr (!kPairs) wait_for_previous();
    const int lane = threadIdx.x & 31;
    const int n = kPairs ? n_pairs : *n_moves;
    if constexpr (kWhich == Moves::kCompact) compact_apply(apply, moves, n);
    const int inner = a.L * 2 * a.H;
    const int64_t units = static_cast<int64_t>(n) * inner;
    const int64_t step = static_cast<int64_t>(gridDim.x) * (kThreads / 32);
    for (int64_t u = (static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x) >> 5; u < units; u += step) {
        const int r = static_cast<int>(u / inner), x = static_cast<int>(u - static_cast<int64_t>(r) * inner);
        const int h = x % a.H, kv = (x / a.H) & 1, l = x / (2 * a.H);
        const Move m = kPairs ? Move{__ldg(src + r), __ldg(dst + r), a.ps, 0} : moves[r];
        const bool bad = m.src < 0 || m.src >= a.n_pages || m.dst < 0 || m.dst >= a.n_pages;
        if (bad) {
            if (kPairs && x == 0 && lane == 0) atomicOr(&g_pages_err, kErrBadPage);
            continue;
        }
        if (!within(m.rows, a.ps + 1ll) || !within(l, a.L)) continue;
        const int64_t head = static_cast<int64_t>(a.ps) * a.row, page = head * a.H;
        uint4 *base = (kv ? a.pool[1] : a.pool[0]) + l * a.layer_stride + h * head;
        const uint4 *s = base + m.src * page;
        uint4 *d = base + m.dst * page;
        const int pieces = m.rows * a.row;
        for (int i0 = lane; i0 < pieces; i0 += 32 * kUnroll) {
            uint4 v[kUnroll];
#pragma unroll
            for (int k = 0; k < kUnroll; ++k)
                if (i0 + 32 * k < pieces) v[k] = s[i0 + 32 * k];
#pragma unroll
            for (int k = 0; k < kUnroll; ++k)
                if (i0 + 32 * k < pieces) __stcs(d + i0 + 32 * k, v[k]);
        }
    }
}

TableArgs table_args(const swa_page_tables *t) {
    return TableArgs{t->table, t->ref, t->out_table, t->out_ref, t->B, t->width, t->n_pages, t->page_size};
}
PoolArgs pool_args(const swa_page_pool *p) {
    PoolArgs a{};
    a.pool[0] = static_cast<uint4 *>(p->k_pages);
    a.pool[1] = static_cast<uint4 *>(p->v_pages);
    a.layer_stride = p->layer_stride / 8;
    a.L = p->n_layers;
    a.H = p->H_kv;
    a.n_pages = p->n_pages;
    a.ps = p->page_size;
    a.row = p->d_h / 8;
    return a;
}
int grid_for(int64_t n, int per_sm) {
    const int64_t blocks = (n + kThreads - 1) / kThreads, cap = static_cast<int64_t>(paged_sm_count()) * per_sm;
    return static_cast<int>(blocks < cap ? (blocks > 0 ? blocks : 1) : cap);
}
// The workspace: ints [2 * B], [3 * n_pages], [B], moves [max(B, n_pages)], a count.  (A fork takes list1
// and what follows as one list of n_pages + B.)
struct PagesWs {
    int32_t *rows0, *rows1, *list0, *list1, *list2, *count;
    Move *moves;
};
size_t up256(size_t x) { return (x + 255) & ~size_t(255); }
size_t moves_of(const swa_page_tables *t) { return t->B > t->n_pages ? t->B : t->n_pages; }
PagesWs carve(const swa_page_tables *t, void *ws) {
    char *p = static_cast<char *>(ws);
    PagesWs w;
    w.count = reinterpret_cast<int32_t *>(p);
    p += 256;
    w.moves = reinterpret_cast<Move *>(p);
    p += up256(moves_of(t) * sizeof(Move));
    w.rows0 = reinterpret_cast<int32_t *>(p);
    w.rows1 = w.rows0 + t->B;
    w.list0 = w.rows1 + t->B;
    w.list1 = w.list0 + t->n_pages;
    w.list2 = w.list1 + t->n_pages;
    return w;
}
cudaError_t copy_ref(const TableArgs &a, cudaStream_t s, int32_t *fill = nullptr, int64_t n_fill = 0) {
    const int64_t n = a.ref == a.out_ref ? 0 : a.n_pages;
    if (n == 0 && n_fill == 0) return cudaSuccess;
    copy_i32_kernel<<<grid_for(n > n_fill ? n : n_fill, 8), kThreads, 0, s>>>(a.ref, a.out_ref, n, fill, n_fill);
    return cudaGetLastError();
}
template <Moves kWhich>
cudaError_t launch_moves(const swa_page_pool *p, const PagesWs &w, int64_t most, const ApplyArgs &apply,
                         cudaStream_t s) {
    const PoolArgs a = pool_args(p);
    const int64_t units = most * a.L * 2 * a.H;
    return launch_dependent(true, move_kernel<kWhich>, dim3(grid_for(units * 32, kMoveBlocks)), kThreads, 0, s, a, w.moves,
                            w.count, nullptr, nullptr, 0, apply);
}

}  // namespace

size_t pages_workspace_bytes(const swa_page_tables *t) {
    return 256 + up256(moves_of(t) * sizeof(Move)) +
           up256((3 * static_cast<size_t>(t->B) + 3 * static_cast<size_t>(t->n_pages)) * sizeof(int32_t));
}

cudaError_t launch_reserve(const swa_page_tables *t, const int32_t *first, const int32_t *end, void *ws,
                           cudaStream_t s) {
    const PagesWs w = carve(t, ws);
    reserve_kernel<<<1, kScanThreads, 0, s>>>(table_args(t), first, end, w.rows0, w.list0);
    return cudaGetLastError();
}

cudaError_t launch_free(const swa_page_tables *t, const int32_t *below, int n_sink, cudaStream_t s) {
    const TableArgs a = table_args(t);
    cudaError_t e = copy_ref(a, s);
    if (e != cudaSuccess) return e;
    const int64_t n = static_cast<int64_t>(a.B) * a.width;
    return launch_dependent(a.ref != a.out_ref, free_kernel, dim3(grid_for(n, 64)), kThreads, 0, s, a, below,
                            n_sink);
}

cudaError_t launch_fork(const swa_page_tables *t, const swa_page_pool *pool, const int32_t *src, const int32_t *len,
                        void *ws, cudaStream_t s) {
    const TableArgs a = table_args(t);
    const PagesWs w = carve(t, ws);
    const ForkWs f{w.rows0, w.list1};
    cudaError_t e;
    if (static_cast<int64_t>(a.B) * a.width + a.n_pages <= kFew) {
        fork_plan_kernel<<<kForkCtas, kScanThreads, 0, s>>>(a, src, len, f, w.rows1, w.list0, w.moves, w.count);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
    } else {
        if ((e = copy_ref(a, s, f.keep, static_cast<int64_t>(a.n_pages) + a.B)) != cudaSuccess) return e;
        const int gx = (a.width - 1) / kThreads + 1;
        const dim3 grid(gx < 64 ? gx : 64, a.B < 65535 ? a.B : 65535);
        if ((e = launch_dependent(true, fork_table_kernel, grid, kThreads, 0, s, a, src, len, f)) != cudaSuccess)
            return e;
        if ((e = launch_dependent(true, fork_alloc_kernel, dim3(1), kScanThreads, 0, s, a, src, len, f, w.rows1,
                                  w.list0, w.moves, w.count)) != cudaSuccess)
            return e;
    }
    return launch_moves<Moves::kFork>(pool, w, a.B, ApplyArgs{}, s);
}

cudaError_t launch_compact(const swa_page_tables *t, const swa_page_pool *pool, int32_t *n_live, void *ws,
                           cudaStream_t s) {
    const TableArgs a = table_args(t);
    const PagesWs w = carve(t, ws);
    compact_plan_kernel<<<1, kScanThreads, 0, s>>>(a, w.list0, w.list1, w.list2, w.moves, w.count, n_live);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    // (as many warps as the moves and the table's entries want)
    const int64_t entries = static_cast<int64_t>(a.B) * a.width;
    const int64_t most = a.n_pages / 2 + 1 + entries / (32 * 2 * pool->H_kv);
    return launch_moves<Moves::kCompact>(pool, w, most, ApplyArgs{a, w.list2, n_live}, s);
}

cudaError_t launch_page_copy(const swa_page_pool *pool, const int32_t *src, const int32_t *dst, int n,
                             cudaStream_t s) {
    const PoolArgs a = pool_args(pool);
    const int64_t units = static_cast<int64_t>(n) * a.L * 2 * a.H;
    move_kernel<Moves::kPairs><<<grid_for(units * 32, kMoveBlocks), kThreads, 0, s>>>(a, nullptr, nullptr, src, dst, n, ApplyArgs{});
    return cudaGetLastError();
}

unsigned int pages_read_clear_error() {
    unsigned int v = 0, z = 0;
    if (cudaMemcpyFromSymbol(&v, g_pages_err, sizeof v) != cudaSuccess) return 0;
    cudaMemcpyToSymbol(g_pages_err, &z, sizeof z);
    return v;
}

}  // namespace swa
