// swa_paged.h -- host-side interface of the paged cache's translation units
// (swa_paged.cu, swa_pages.cu) to the C ABI.  Not installed.
#pragma once

#include <cuda.h>

#include "swa_internal.h"

namespace swa {

// What a launch of an attention kernel computes.  kAll: the whole of swa_paged_attend.  Of
// swa_paged_attend_shared, kPrefix: every group's new tokens over the positions that its sequences
// share, kOwn: each sequence's new tokens over the positions behind those; the parts are joined by a
// kernel of their own (swa_paged_shared.cu).
enum class Part { kAll, kPrefix, kOwn };

// A group's prefix part: the packed rows of n tokens from q0 on, of several sequences, over the positions
// below `end` (of which those at or past the window of p0, the least position stored next of them, and
// the sinks matter) in the pages of sequence `row`; top: the largest position of a row.  n = 0: nothing
// for the many-row kernel; few: the tokens of a part that the kernel for few rows has.
struct PagedGroup {
    int32_t q0, n, p0, end, row, top, few, unused;
};

// One call of swa_paged_attend / swa_paged_append, as the kernels take it.
struct PagedArgs {
    const uint16_t *q;  // [N, H_q, D] bf16 bits; element strides of (token, head)
    int64_t q_st[2];
    const uint16_t *kn, *vn;  // [N, H_kv, D] (append) or nullptr
    int64_t kn_st[2], vn_st[2];
    uint16_t *o;
    int64_t o_st[2];
    float *lse;       // [N, H_q]
    int32_t *counts;  // [N, H_q] or nullptr
    uint16_t *k_pages, *v_pages;  // [n_pages, H_kv, ps, D]
    const int32_t *table;         // [B, width]
    const int32_t *p0;            // [B]
    const int32_t *q_start;       // [B + 1] or nullptr (one token a sequence)
    int N, B, width, n_pages, ps, ps_log2, H_q, H_kv, G, D;
    int window;  // INT_MAX: none
    int n_sink;
    int max_q;  // 0: not known
    float scale_log2;
    // parts: kPrefix reads groups (B is their number) and, with a window, the rows' positions, kOwn reads base
    const PagedGroup *groups;
    const int32_t *pos;   // [N]
    const int32_t *base;  // [B]: the positions below it are in the prefix part
    const int32_t *tile_groups;  // kPrefix: the groups with rows, 0: there are none
    // A part's results, fp32.  A unit that one CTA has whole: here; one that several have: in their slots of
    // PagedWs.  Units of kPrefix, at (q0 / TT + b + ut) * H_kv + kvh: the CTA that begins the unit, and its
    // pieces (0: whole); those of kOwn whose rows are not final, in any order, two entries each: the
    // same, b, ut * H_kv + kvh; q0, n, and of the sequence's group its first token (-1: no prefix) and number.
    float2 *part_ml;  // [N, H_q]: maximum (log2 units), sum of weights
    float *part_o;    // [N, H_q, D]: unnormalised weighted values
    int2 *part_units;
    int4 *part_list;
    int32_t *part_count, part_cap;  // of the list: units
    const int4 *part_info;  // [B][2], the plan's
};

constexpr int kPagedMaxB = 8192;

// Partial results of units that several CTAs share.  The CTAs that have a stretch of the shared-out
// list are numbered t = 0, 1, ... in its order; number t has two slots of `rows` rows: 2t for the
// unit that an earlier CTA began, 2t + 1 for one that it begins and leaves open (only its last
// unit can be).
struct PagedWs {
    float *ml;    // [2 * CTAs][rows][2]: maximum (log2 units), sum
    float *acc;   // [2 * CTAs][D / 8][rows][8]: unnormalised weighted values
    int32_t *done;  // tile kernel, [CTAs][8]: pieces of the unit that CTA t began which are written, by warp
    int4 *open;     // split kernel, [CTAs]: {tiles that the unit left open still has for later CTAs (0: none), b, kvh, ut}
    long long *first;  // split kernel, [CTAs]: where its stretch of the list starts
    int32_t *left;     // split kernel, [CTAs]: and its tiles
};
// A kernel's grid and the shape of its units: tiles of query rows (row r of a tile is token
// r / G, head r % G of the group), tokens a tile.
struct PagedShape {
    int ctas, tiles, rows, TQ;
};
inline size_t paged_up(size_t v) { return (v + 255) & ~size_t(255); }
inline size_t paged_ws_bytes(const PagedShape &x, int D) {
    const size_t rows = static_cast<size_t>(x.ctas) * 2 * x.tiles * x.rows;
    return paged_up(rows * 2 * sizeof(float)) + paged_up(rows * D * sizeof(float)) +
           paged_up(static_cast<size_t>(x.ctas) * 32);
}
inline PagedWs paged_carve(void *ws, const PagedShape &x, int D) {
    const size_t rows = static_cast<size_t>(x.ctas) * 2 * x.tiles * x.rows;
    char *p = static_cast<char *>(ws);
    PagedWs w;
    w.ml = reinterpret_cast<float *>(p);
    p += paged_up(rows * 2 * sizeof(float));
    w.acc = reinterpret_cast<float *>(p);
    p += paged_up(rows * D * sizeof(float));
    w.done = reinterpret_cast<int32_t *>(p);  // 32 bytes a CTA, one use or the other
    w.open = reinterpret_cast<int4 *>(p);
    w.first = reinterpret_cast<long long *>(p + static_cast<size_t>(x.ctas) * 16);
    w.left = reinterpret_cast<int32_t *>(p + static_cast<size_t>(x.ctas) * 24);
    return w;
}

// Few rows (swa_paged_split.cu).  It stores the new rows itself where every sequence has one
// new token (q_start null).
PagedShape paged_split_shape(const PagedArgs &a);
// Its shared units are joined by launch_paged_merge.
// after_append: launched as a programmatic dependent of the append kernel just before it on the
// stream (everything up to the first copy of a page overlaps that kernel).
cudaError_t launch_paged_split(const PagedArgs &a, const PagedWs &w, bool after_append, cudaStream_t s);
void paged_split_read_clear_error(unsigned int *data, unsigned int *wait);
cudaError_t launch_paged_merge(const PagedArgs &a, const PagedWs &w, const PagedShape &x, cudaStream_t s);
// Many rows (swa_paged_tile.cu); w.done is zero at its start.
PagedShape paged_tile_shape(const PagedArgs &a);
int paged_tile_tokens(const PagedArgs &a, Part part);  // tokens of a unit
cudaError_t launch_paged_tile(const PagedArgs &a, const PagedWs &w, bool after_append, cudaStream_t s,
                              Part part = Part::kAll);
void paged_tile_read_clear_error(unsigned int *data, unsigned int *wait);

// bf16 maps with 128-B swizzle.
// The rows q [N, H_q, D]: (64 of d, head, token), a box of 64 x heads x tokens.
bool paged_query_map(CUtensorMap *m, const PagedArgs &a, int heads, int tokens);
// A pool: (64 of d, 8 rows, column block, group of 8 rows), a box of `rows` rows of one page and
// head.  The groups of all pages and heads count through, group (page * H_kv + head) * ps / 8 being
// a page's first, so one copy brings a page's rows whole, whatever the head dim, and a tile's
// pages follow one another in shared memory without a gap: column block c of row r lies at
// (r / 8) * D / 64 * 1024 + c * 1024 + r % 8 * 128.
bool paged_pool_map(CUtensorMap *m, const PagedArgs &a, const void *pool, int rows);

int paged_sm_count();  // SMs of the current device

template <class... P, class... A>
cudaError_t launch_dependent(bool dependent, void (*kernel)(P...), dim3 grid, int threads, int smem, cudaStream_t s,
                             const A &...args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = dependent ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}
bool paged_few_rows(const PagedArgs &a);  // the few-row kernel takes the batch
size_t paged_workspace_bytes(const PagedArgs &a);
// Groups of sequences that share leading pages (swa_paged_shared.cu).
size_t paged_shared_workspace_bytes(const PagedArgs &a, int n_groups);
cudaError_t launch_paged_shared(const PagedArgs &a, const int32_t *group_start, int n_groups, void *ws, cudaStream_t s);
unsigned int paged_shared_read_clear_error();
unsigned int shared_rows_read_clear_error(unsigned int *data);
// zero, n_zero: words that the kernel sets to 0 beside its own work (n_zero may be 0).
cudaError_t launch_paged_append(const PagedArgs &a, int32_t *zero, int n_zero, cudaStream_t s);
cudaError_t launch_paged_attend(const PagedArgs &a, void *ws, cudaStream_t s);

// The table of a rotation and how it turns a head (swa_rope.cu).
struct RopeArgs {
    const float *table;  // [n_pos, rot]: cosines, then sines
    int n_pos, rot, interleaved;
};
cudaError_t launch_rope_table(const double *inv_freq, int rot, int n_pos, float scale, float *out, cudaStream_t s);
// a.q may be nullptr (keys and values only), a.kn too (queries only); rotated queries go to a.o.
cudaError_t launch_rope_append(const PagedArgs &a, const RopeArgs &r, cudaStream_t s);
unsigned int rope_read_clear_error();

// Errors of the data (cache word), of the few-row and of the many-row kernels.
void paged_read_clear_error(unsigned int *data, unsigned int *split, unsigned int *prefill);

size_t pages_workspace_bytes(const swa_page_tables *t);
cudaError_t launch_reserve(const swa_page_tables *t, const int32_t *first, const int32_t *end, void *ws,
                           cudaStream_t s);
cudaError_t launch_free(const swa_page_tables *t, const int32_t *below, int n_sink, cudaStream_t s);
cudaError_t launch_fork(const swa_page_tables *t, const swa_page_pool *pool, const int32_t *src, const int32_t *len,
                        void *ws, cudaStream_t s);
cudaError_t launch_compact(const swa_page_tables *t, const swa_page_pool *pool, int32_t *n_live, void *ws,
                           cudaStream_t s);
cudaError_t launch_page_copy(const swa_page_pool *pool, const int32_t *src, const int32_t *dst, int n,
                             cudaStream_t s);
unsigned int pages_read_clear_error();

}  // namespace swa
