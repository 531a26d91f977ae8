// swa_rope.cu -- rotary positions beside the paged cache: the table of a rotation's cosines and
// sines, and the append that rotates a token's queries and keys on their way.
#include <climits>
#include <cmath>

#include "ptx.cuh"
#include "swa_paged.cuh"

namespace swa {
namespace {

__device__ unsigned int g_rope_err = 0;

constexpr int kThreads = 256;

// ---------------------------------------------------------------------------------------------
// table: out[p, i] = scale cos(p f_i), out[p, R/2 + i] = scale sin(p f_i).
// An angle is only needed modulo a turn, and f_i / (2 pi) modulo 1 is held as a 64-bit fraction G_i: p G_i mod
// 2^64 is then the angle of position p in units of 2^-64 turns, off by p 2^-64 at most, by integer
// arithmetic alone.  (An SM has two lanes for 64-bit floating point: a block uses them once a column.)
// The angle's nearest quarter turn goes into signs and a swap; the rest y, in eighths of a turn, |y| <= 1, into the
// Taylor polynomials of sin and cos at y pi/4, of degree 9 and 10 (remainders below 2e-9).
// Bound by HBM writes and, as near, by the instructions of the polynomials (about 30 a pair): 131072 x 128 12.8 us,
// 5.2 TB/s written; with 64-bit floating point for every angle it would be the two lanes, above 50 us.
// ---------------------------------------------------------------------------------------------
constexpr int kTableCols = 128;  // most columns (half a head of 256)

// frac(f / (2 pi)) in units of 2^-64, off by less than one up to |f| = 2^43 (the two numbers hold 107 bits of 1 / (2 pi))
__device__ __forceinline__ unsigned long long turn_fraction(double f) {
    // |f| / (2 pi) as an unevaluated sum hi + lo, 1 / (2 pi) being one of two 64-bit numbers
    const double x = fabs(f), inv = 0.15915494309189535, inv_lo = -9.839338337591243e-18;
    const double hi = x * inv, lo = fma(x, inv, -hi) + x * inv_lo;
    const double two64 = 18446744073709551616.0;
    // (hi - floor(hi) is exact, and so is its conversion where it is not below 2^-11)
    const unsigned long long g = static_cast<unsigned long long>((hi - floor(hi)) * two64) +
                                 static_cast<unsigned long long>(__double2ll_rn((lo - rint(lo)) * two64));
    return f < 0.0 ? 0ull - g : g;
}

// cos and sin of x 2^-64 turns
__device__ __forceinline__ void cos_sin(unsigned long long x, float &c, float &s) {
    // the angle in units of 2^-32 turns, to the nearest; q: its nearest quarter, r: the rest
    const unsigned int t = static_cast<unsigned int>((x + 0x80000000ull) >> 32);
    const unsigned int q = (t + 0x20000000u) >> 30;
    const int r = static_cast<int>(t - (q << 30));
    const float y = static_cast<float>(r) * 1.862645149230957e-9f, z = y * y;  // 2^-29
    // (-1)^k (pi/4)^n / n! for n = 2 k + 1 and n = 2 k
    const float sn = y * fmaf(z, fmaf(z, fmaf(z, fmaf(z, 3.13361681492097e-07f, -3.657620254671201e-05f), 0.002490394515916705f), -0.08074551075696945f), 0.7853981852531433f);
    const float cs = fmaf(z, fmaf(z, fmaf(z, fmaf(z, fmaf(z, -2.461136894282845e-08f, 3.5908603877032874e-06f), -0.0003259918885305524f), 0.01585434377193451f), -0.3084251284599304f), 1.0f);
    const float a = q & 1u ? sn : cs, b = q & 1u ? cs : sn;
    // quarters 1, 2 turn the cosine's sign, 2, 3 the sine's
    c = __uint_as_float(__float_as_uint(a) ^ (((q + 1u) & 2u) << 30));
    s = __uint_as_float(__float_as_uint(b) ^ ((q & 2u) << 30));
}

// A block has `steps` rows of each of its threads, which have four columns each.
__global__ void __launch_bounds__(kThreads) rope_table_kernel(const double *inv_freq, int half, int n_pos, int steps,
                                                              float scale, float *out) {
    __shared__ unsigned long long fraction[kTableCols];
    __shared__ float factor[kTableCols];  // scale, or NaN
    for (int i = threadIdx.x; i < half; i += kThreads) {
        const double f = __ldg(inv_freq + i);
        const bool finite = isfinite(f);
        fraction[i] = finite ? turn_fraction(f) : 0ull;
        factor[i] = finite ? scale : NAN;
    }
    __syncthreads();
    const int per_row = half / 4, rows = kThreads / per_row;  // (threads behind the last whole row have none)
    const int row = static_cast<int>(threadIdx.x) / per_row, col = static_cast<int>(threadIdx.x) % per_row * 4;
    if (row >= rows) return;
    int64_t p = static_cast<int64_t>(blockIdx.x) * (rows * steps) + row;
    unsigned long long x[4], step[4];
    float k[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        x[e] = fraction[col + e] * static_cast<unsigned long long>(p);
        step[e] = fraction[col + e] * static_cast<unsigned long long>(rows);
        k[e] = factor[col + e];
    }
    float *at = out + p * (2 * half) + col;
    for (int i = 0; i < steps && p < n_pos; ++i, p += rows, at += static_cast<int64_t>(rows) * (2 * half)) {
        float c[4], s[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            cos_sin(x[e], c[e], s[e]);
            x[e] += step[e];
        }
        *reinterpret_cast<float4 *>(at) = make_float4(c[0] * k[0], c[1] * k[1], c[2] * k[2], c[3] * k[3]);
        *reinterpret_cast<float4 *>(at + half) = make_float4(s[0] * k[0], s[1] * k[1], s[2] * k[2], s[3] * k[3]);
    }
}

// ---------------------------------------------------------------------------------------------
// append with rotation: pair (x, y) of a query or key becomes (x c - y s, y c + x s), in 32 bits, rounded
// once; elements past the rotated ones and values are copied.
// A lane has 16 elements of a head: the eight pairs whose cosines and sines it keeps in registers
// for all heads that it goes through (a table row is read once a warp and token, not once a head).
// A warp has kUnroll such steps of 32 lanes in flight, and its rows' loads are under way while it looks up
// its sequence, position and page.  Bound by HBM: each row is read once and written once.  12780 tokens of 16 / 8
// heads of 256 68 us (94% of the measured copy rate; two blocks an SM instead of three 75), 4102 tokens of 33
// sequences, 12 / 12 heads of 64, 8.8 us, one token 2.9.
// ---------------------------------------------------------------------------------------------
constexpr int kUnroll = 4;

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// eight pairs (x_i, y_i) turned; kPairs: neighbours in a and b, else x_i in a and y_i in b
template <bool kPairs>
__device__ __forceinline__ void turn(uint4 &a, uint4 &b, const float (&c)[8], const float (&s)[8]) {
    uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    if constexpr (kPairs) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float x = bf16_lo(w[i]), y = bf16_hi(w[i]);
            w[i] = pack_bf16x2(x * c[i] - y * s[i], y * c[i] + x * s[i]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float x0 = bf16_lo(w[i]), x1 = bf16_hi(w[i]), y0 = bf16_lo(w[4 + i]), y1 = bf16_hi(w[4 + i]);
            const int k = 2 * i;
            w[i] = pack_bf16x2(x0 * c[k] - y0 * s[k], x1 * c[k + 1] - y1 * s[k + 1]);
            w[4 + i] = pack_bf16x2(y0 * c[k] + x0 * s[k], y1 * c[k + 1] + x1 * s[k + 1]);
        }
    }
    a = make_uint4(w[0], w[1], w[2], w[3]);
    b = make_uint4(w[4], w[5], w[6], w[7]);
}

template <int D, bool kPairs>
__global__ void __launch_bounds__(kThreads, 3) rope_append_kernel(const PagedArgs a, const RopeArgs r, int chunks,
                                                               int tokens) {
    constexpr int CS = D / 16, HPI = 32 / CS;  // lanes a head, heads a step
    const int lane = threadIdx.x & 31;
    const int64_t w = (static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x) >> 5;
    const int chunk = static_cast<int>(w % chunks);
    const int64_t n_first = w / chunks * tokens;
    const int n_end = static_cast<int>(min(n_first + tokens, static_cast<int64_t>(a.N)));
    const int slot = lane % CS;
    const bool turns = slot < r.rot / 16;
    const int e0 = kPairs || !turns ? slot * 16 : slot * 8;
    const int e1 = e0 + (kPairs || !turns ? 8 : r.rot / 2);
    const int Hq = a.q ? a.H_q : 0, heads = Hq + (a.kn ? 2 * a.H_kv : 0);
    const int h_first = chunk * (HPI * kUnroll) + lane / CS;
    Seq s{};
    int b = 0;  // the sequence of the last token
    for (int n = static_cast<int>(n_first); n < n_end; ++n) {
        uint4 x[kUnroll][2];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int h = h_first + u * HPI;
            if (h >= heads) continue;
            const uint16_t *src = h < Hq            ? a.q + n * a.q_st[0] + h * a.q_st[1]
                                  : h < Hq + a.H_kv ? a.kn + n * a.kn_st[0] + (h - Hq) * a.kn_st[1]
                                                    : a.vn + n * a.vn_st[0] + (h - Hq - a.H_kv) * a.vn_st[1];
            x[u][0] = *reinterpret_cast<const uint4 *>(src + e0);
            x[u][1] = *reinterpret_cast<const uint4 *>(src + e1);
        }
        if (!s.ok || n >= s.q0 + s.n) {
            b = find_sequence(a, n, lane);
            if (b < 0) {
                s.ok = false;
                continue;
            }
            s = load_seq(a, b);
        }
        const int p = s.p0 + (n - s.q0);
        if (!s.ok || p >= r.n_pos) {
            if (lane == 0) atomicOr(&g_rope_err, SWA_DEVERR_BAD_POSITION);
            continue;
        }
        const int page = a.kn ? page_of(a, b, p >> a.ps_log2) : 0;
        float c[8], sn[8];
        if (turns) {
            const float4 *row = reinterpret_cast<const float4 *>(r.table + static_cast<int64_t>(p) * r.rot + slot * 8);
            const float4 *row2 = row + r.rot / 8;
            const float4 c0 = __ldg(row), c1 = __ldg(row + 1), s0 = __ldg(row2), s1 = __ldg(row2 + 1);
            c[0] = c0.x, c[1] = c0.y, c[2] = c0.z, c[3] = c0.w, c[4] = c1.x, c[5] = c1.y, c[6] = c1.z, c[7] = c1.w;
            sn[0] = s0.x, sn[1] = s0.y, sn[2] = s0.z, sn[3] = s0.w;
            sn[4] = s1.x, sn[5] = s1.y, sn[6] = s1.z, sn[7] = s1.w;
        }
        if (page >= a.n_pages && lane == 0) atomicOr(&g_rope_err, SWA_DEVERR_BAD_PAGE);
        if (!SWA_IN_BOUNDS(n < a.N && p >= 0 && (!a.kn || (b < a.B && page >= 0 && p >> a.ps_log2 < a.width)), &g_rope_err))
            continue;
        const int64_t at = static_cast<int64_t>(page) * a.H_kv * a.ps + (p & (a.ps - 1));
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int h = h_first + u * HPI;
            if (h >= heads || (h >= Hq && page >= a.n_pages)) continue;
            if (turns && h < Hq + a.H_kv) turn<kPairs>(x[u][0], x[u][1], c, sn);
            uint16_t *dst = h < Hq ? a.o + n * a.o_st[0] + h * a.o_st[1]
                            : h < Hq + a.H_kv ? a.k_pages + (at + static_cast<int64_t>(h - Hq) * a.ps) * D
                                              : a.v_pages + (at + static_cast<int64_t>(h - Hq - a.H_kv) * a.ps) * D;
            *reinterpret_cast<uint4 *>(dst + e0) = x[u][0];
            *reinterpret_cast<uint4 *>(dst + e1) = x[u][1];
        }
    }
}

template <int D>
cudaError_t launch_d(const PagedArgs &a, const RopeArgs &r, cudaStream_t s) {
    constexpr int kHeads = 32 / (D / 16) * kUnroll;  // of a warp
    const int heads = (a.q ? a.H_q : 0) + (a.kn ? 2 * a.H_kv : 0);
    const int chunks = (heads + kHeads - 1) / kHeads;
    // Up to four tokens of a warp, one after the other, where there are warps enough: a sequence is looked up once.
    const int64_t want = static_cast<int64_t>(a.N) * chunks / (40 * paged_sm_count());
    const int tokens = static_cast<int>(want < 1 ? 1 : want > 4 ? 4 : want);
    const int64_t warps = (static_cast<int64_t>(a.N) + tokens - 1) / tokens * chunks;
    const int64_t blocks = (warps * 32 + kThreads - 1) / kThreads;
    if (blocks > INT_MAX) return cudaErrorInvalidValue;
    const auto kernel = r.interleaved ? rope_append_kernel<D, true> : rope_append_kernel<D, false>;
    kernel<<<static_cast<int>(blocks), kThreads, 0, s>>>(a, r, chunks, tokens);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rope_table(const double *inv_freq, int rot, int n_pos, float scale, float *out, cudaStream_t s) {
    const int64_t rows = kThreads / (rot / 8);  // of a step
    // (up to sixteen steps of a block where there are blocks enough: the columns' fractions are made once a block)
    const int64_t all = (static_cast<int64_t>(n_pos) + rows - 1) / rows, want = all / (8 * paged_sm_count());
    const int steps = static_cast<int>(want < 1 ? 1 : want > 16 ? 16 : want);
    const int64_t blocks = (all + steps - 1) / steps;
    if (blocks > INT_MAX) return cudaErrorInvalidValue;
    rope_table_kernel<<<static_cast<int>(blocks), kThreads, 0, s>>>(inv_freq, rot / 2, n_pos, steps, scale, out);
    return cudaGetLastError();
}

cudaError_t launch_rope_append(const PagedArgs &a, const RopeArgs &r, cudaStream_t s) {
    switch (a.D) {
        case 64: return launch_d<64>(a, r, s);
        case 128: return launch_d<128>(a, r, s);
        case 256: return launch_d<256>(a, r, s);
        default: return cudaErrorInvalidValue;
    }
}

unsigned int rope_read_clear_error() {
    unsigned int v = 0, z = 0;
    if (cudaMemcpyFromSymbol(&v, g_rope_err, sizeof v) != cudaSuccess) return 0;
    cudaMemcpyToSymbol(g_rope_err, &z, sizeof z);
    return v;
}

}  // namespace swa
