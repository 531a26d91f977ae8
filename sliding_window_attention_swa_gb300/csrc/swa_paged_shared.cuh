// swa_paged_shared.cuh -- what the kernels of swa_paged_attend_shared agree on: the stretches of keys that
// the kernel for few rows takes one at a time, and where their results lie.
#pragma once

#include "swa_paged.cuh"

namespace swa {

constexpr int kStretchRows = 16;  // rows of a unit of the kernel for few rows (mma.sync M)
// Least keys of a stretch.  256 instead: 135 sequences of 250 tokens on average behind their prefixes 100 us instead of 91,
// 31 small groups 110.5 instead of 105; 64 sequences with prefixes in tiles 86 instead of 89.
constexpr int kStretchKeys = 64;

// One stretch: tokens q0 .. q0 + n - 1 (n * G <= 16 rows) over the keys k0 .. k1 - 1 in the pages of row
// `row` of the table; the result of token t goes to token first + t of the planes of part `part` (0: own, 1: prefix).
struct Stretch {
    int32_t row, q0, n, first, k0, k1, part, unused;
};

// The results of a part: rows [tokens, H_q] in each of `planes` planes (one, of the many-row kernel).  A token has its
// own number in a plane, but for prefixes of few rows where the groups are too few to have all tokens: there group g
// has the places from g * few_tokens(G) on.
struct PartResults {
    float2 *ml;
    float *o;
    int planes, tokens;
    // of the many-row kernel: its units (the prefix's), and the slots of those that several CTAs have
    const int2 *units;
    PagedWs ws;
    int ctas, rows, TQ, TT;
};

// Tokens that a stretch has at most.
__host__ __device__ __forceinline__ int few_tokens(int G) { return kStretchRows / G; }

// A unit's keys: [lo, end) in `count` stretches, stretch i the part within [first + i * keys, first + (i + 1) *
// keys), and, if sink1 > sink0, one more, [sink0, sink1), in the last plane.
struct Keys {
    int lo, end, sink0, sink1, first, keys, count;
    __host__ __device__ __forceinline__ int stretches() const { return count + (sink1 > sink0 ? 1 : 0); }
    __host__ __device__ __forceinline__ int begin(int i) const { return i < count ? max(lo, first + i * keys) : sink0; }
    __host__ __device__ __forceinline__ int close(int i) const { return i < count ? min(end, first + (i + 1) * keys) : sink1; }
};

// At most p.planes - 1 stretches, and the sinks'.
__host__ __device__ __forceinline__ Keys split_keys(int lo, int end, int sink0, int sink1, const PartResults &p) {
    Keys k;
    k.lo = lo;
    k.end = end;
    k.sink0 = sink0;
    k.sink1 = sink1;
    k.first = lo & ~15;
    const int n = end - k.first, most = p.planes - 1;
    k.keys = max(kStretchKeys, ((n + most - 1) / most + 15) & ~15);
    k.count = (n + k.keys - 1) / k.keys;
    return k;
}

// Keys at or past base of the unit of tokens ut * TT .. of sequence s.
__host__ __device__ __forceinline__ Keys own_keys(const PagedArgs &a, const Seq &s, int base, int ut, int TT,
                                         const PartResults &p) {
    const int t0 = s.p0 + ut * TT, t1 = s.p0 + min(s.n, (ut + 1) * TT) - 1;
    const int lo = max(base, t0 >= a.window ? t0 - a.window + 1 : 0);
    return split_keys(lo, t1 + 1, base, min(a.n_sink, lo), p);
}

// Keys of a prefix.
__host__ __device__ __forceinline__ Keys prefix_keys(const PagedArgs &a, int p0, int end, const PartResults &p) {
    const int lo = p0 >= a.window ? p0 - a.window + 1 : 0;
    return split_keys(lo, end, 0, min(a.n_sink, lo), p);
}

// Whether two sequences have rows in common.
__host__ __device__ __forceinline__ bool in_common(const Seq &s, const Seq &t) {
    return s.n > 0 && t.n > 0 && s.q0 < t.q0 + t.n && t.q0 < s.q0 + s.n;
}

// Stretches on the lists, groups with rows for the many-row kernel, stretches taken beyond each warp's first, own units
// of the many-row kernel to be joined.
enum { kOwnStretches, kPrefixStretches, kTileGroups, kTaken, kOwnUnits, kCounts };

struct SharedArgs {
    PagedArgs a;
    const int32_t *group_start;  // [n_groups + 1]
    int n_groups;
    PagedGroup *groups;
    int32_t *base;             // [B]
    int4 *info;                // [B][2]: base, its group's n, few, q0; p0, the group's number, whether it has rows
    int32_t *pos;              // [N]
    int32_t *seq;              // [N], with few new tokens: the sequence (rows of none: anything)
    Stretch *stretches;        // [prefix_cap + own_cap]: prefixes', then own ones
    int32_t *counts;           // [kCounts]
    int clusters;              // of the plan
    int prefix_cap, own_cap;
    const int4 *own_units;     // [own_units_cap][2]: see PagedArgs::part_list
    int own_units_cap;
    int few;                   // own parts (and prefixes of few rows) are cut into stretches
    int any_tiles;             // prefixes may go to the many-row kernel
    int prefix_tokens, own_tokens;  // tokens of a query tile of the many-row kernel
    PartResults part[2];       // own, prefix in tiles
    PartResults few_prefix;
};

// Where the prefix of group g, of few rows, from token q0 on, has its results.
__device__ __forceinline__ int prefix_place(const SharedArgs &sa, int g, int q0) {
    return sa.few_prefix.tokens < sa.a.N ? g * few_tokens(sa.a.G) : q0;
}

cudaError_t launch_shared_rows(const SharedArgs &sa, bool behind_tiles, cudaStream_t s);
int shared_rows_warps(int D);  // warps that are resident at a time

}  // namespace swa
