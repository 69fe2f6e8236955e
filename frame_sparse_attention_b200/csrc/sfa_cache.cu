// New tokens of a layer: norm of every head's query and key row, rotary positions, and the
// 8-bit frame cache (writing and reading back).
//
// ("Head Forcing", §2: per-head caches of a streaming model.)  Per row x of d elements:
//   y = x / sqrt(mean(x^2) + eps) * w,  then  (y_i, y_j) -> s (y_i cos - y_j sin, y_j cos + y_i sin)
// for the pairs (i, j) of the rotated part; a cached row is cut into blocks of 32 elements,
// each stored as e4m3 codes times the smallest power of two that brings it within 448.
//
// All of it moves memory: a row is read once and written once and everything between stays
// in registers, so the floor is (bytes in + bytes out) over the HBM rate.
//   * d / 8 lanes own a row, 16 bytes each: the norm's sum and a block's maximum are shuffles;
//   * norm and rotation: a warp owns a token, or a few, so the R/2 angles (fp64, reduced to one
//     turn) and their sine and cosine are formed once for all heads and kept in shared memory,
//     then folded with the norm's weight into two coefficients per element: y = rs (x A + x_partner B);
//   * a token's head rows are loaded several at a time before any arithmetic; with few
//     tokens they are dealt out over several warps (one row group each at a single token);
//   * writing and reading alone: a warp owns consecutive rows of a head, which lie side by side
//     in the cache too.
// 12 heads, d = 128, floors at 6.53 TB/s: norm and rotation of 63960 tokens 135 us (5.8 TB/s,
// floor 120), of 4680 13.5 (8.8); append of 20280 72 (48), of 4680 19 (11); write of 20280 33
// (29); read of 60000 89 (86).  The chunks of 4680 are one wave of warps, each a chain of loads,
// angles and rows: 63 % of the issue slots with 41 % of the warps there, loads the largest stall.
// Few heads are far from their floor (20000 tokens of 1 + 1 heads, d = 128, 13.3 us for 3.1): the
// angles of a token, in fp64, are then formed for two rows instead of 24.
#include <cmath>
#include <cstdint>

#include <cuda_runtime.h>

#include "sfa.h"
#include "sfa_cache.cuh"
#include "sfa_internal.h"
#include "sfa_ptx.cuh"

namespace sfa {
namespace {

constexpr int ROW_WARPS = 4;  // warps per CTA (8: a token's append 4.3 against 4.1 us, 9000 tokens' 34.1 against 33.8)
constexpr int ROW_CTAS = 8;   // CTAs per SM: 64 registers a thread, 32 warps (24 warps with 80: 150 against 143 us
                              // on 63960 tokens of 12 + 12 heads, and 26 against 20 on the append of 4680)
// Rows of a lane under way together where a warp takes consecutive rows, D / 8 lanes to a row.
// Written, 12 heads, d = 128, 1560, 4680 and 20280 tokens: two 4.1, 11.1, 33.6 us, four 4.3, 12.0, 32.9.
constexpr int WRITE_U = 2, READ_U = 4;
template <int D>
constexpr int ROWS_AT_ONCE = 32 * 8 / D;

struct RowsArgs {
    int32_t B, H, Hk, L;
    const uint16_t *q, *k, *v;
    uint16_t *q_out, *k_out;
    int64_t qs[3], ks[3], vs[3], qo[3], ko[3];
    const float *q_weight, *k_weight;
    float eps;  // < 0: no norm
    // rotation: R / 2 pairs, those of axis a end before axis_end[a]
    const double *inv_freq;
    const int32_t *pos;
    int64_t ps0, ps1;
    int32_t axis_end[SFA_ROPE_MAX_AXES];
    int32_t n_axes, R;
    float rope_scale;
    // cache
    CacheView cache;
    const int32_t *start;
    int64_t ss0, ss1;
    const int32_t *lens;
    int32_t *status;
    int32_t n_parts;   // warps per token
    uint32_t tokens;   // B * L
    uint32_t n_warps;  // tiles of tokens * n_parts
    uint32_t rows;     // B * Hk * L
};

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// cosine and sine (times the scale) of pair p at this token.  A far position times a
// frequency loses its fraction of a turn in fp32, so the product is formed and reduced to
// [-1, 1] half turns in fp64.  What fp32 drops of that (up to 2^-25 half turns, 9e-8 of a radian,
// more than the rounding of the results) turns the pair by a first-order step.
__device__ __forceinline__ float2 rotation(const RowsArgs &a, const int32_t *pos, int p)
{
    int ax = 0;
#pragma unroll
    for (int i = 0; i < SFA_ROPE_MAX_AXES - 1; ++i) ax += (i < a.n_axes - 1 && p >= a.axis_end[i]) ? 1 : 0;
    const double t = (double)__ldg(pos + ax) * __ldg(a.inv_freq + p) * 0.31830988618379067154;
    const double r = t - 2.0 * rint(0.5 * t);
    const float near = (float)r, rest = (float)(r - near) * 3.14159265358979f;
    float s, c;
    sincospif(near, &s, &c);
    return make_float2(fmaf(-rest, s, c) * a.rope_scale, fmaf(rest, c, s) * a.rope_scale);
}

// Two fp32 numbers that one instruction works on (each rounds like a scalar).
__device__ __forceinline__ uint64_t f2(float lo, float hi)
{
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ float lo2(uint64_t v) { return __uint_as_float((uint32_t)v); }
__device__ __forceinline__ float hi2(uint64_t v) { return __uint_as_float((uint32_t)(v >> 32)); }
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

// A lane's eight elements as pairs of even ones, (0, 2) and (4, 6), and of odd ones, (1, 3) and
// (5, 7): the two elements of an interleaved rotation pair lie in the same place of e and o.
struct Eight {
    uint64_t e[2], o[2];
};
__device__ __forceinline__ Eight unpack8(const uint32_t (&w)[4])
{
    Eight x;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        x.e[i] = f2(bf_lo(w[2 * i]), bf_lo(w[2 * i + 1]));
        x.o[i] = f2(bf_hi(w[2 * i]), bf_hi(w[2 * i + 1]));
    }
    return x;
}

// y = rs * (x * A + mate * B) for this lane's elements
struct Coef {
    Eight A, B;
};

template <int D, bool HALF>
__device__ __forceinline__ void coefficients(Coef &f, const float *cosp, const float *sinp, const float *w, int e0, int R)
{
    float A[8], B[8];
    const bool first = HALF && e0 < R / 2;
    const int mate0 = !HALF ? e0 : first ? e0 + R / 2 : e0 < R ? e0 - R / 2 : e0;  // where the mates' weights lie
    float wo[8], wm[8];
    if (w) {
#pragma unroll
        for (int j = 0; j < 8; j += 4) {
            const float4 x = __ldg(reinterpret_cast<const float4 *>(w + e0 + j));
            const float4 y = HALF ? __ldg(reinterpret_cast<const float4 *>(w + mate0 + j)) : x;
            wo[j] = x.x, wo[j + 1] = x.y, wo[j + 2] = x.z, wo[j + 3] = x.w;
            wm[j] = y.x, wm[j + 1] = y.y, wm[j + 2] = y.z, wm[j + 3] = y.w;
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) wo[j] = wm[j] = 1.f;
    }
    // the lane's pairs: four (interleaved), or eight from the first half's on; past the rotated
    // part the tables hold cosine 1 and sine 0
    float c[8], t[8];
#pragma unroll
    for (int j = 0; j < (HALF ? 8 : 4); j += 4) {
        const int p = HALF ? (first || e0 >= R ? e0 % (D / 2) : mate0) + j : e0 / 2;
        const float4 x = *reinterpret_cast<const float4 *>(cosp + p), y = *reinterpret_cast<const float4 *>(sinp + p);
        c[j] = x.x, c[j + 1] = x.y, c[j + 2] = x.z, c[j + 3] = x.w;
        t[j] = y.x, t[j + 1] = y.y, t[j + 2] = y.z, t[j + 3] = y.w;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int p = HALF ? j : j >> 1;
        const bool minus = HALF ? first : (j & 1) == 0;
        A[j] = wo[j] * c[p];
        B[j] = (HALF ? wm[j] : wo[j ^ 1]) * (minus ? -t[p] : t[p]);
    }
    if (R < D) {  // elements that do not turn, whatever their neighbours' weights
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            A[j] = e0 + j < R ? A[j] : wo[j];
            B[j] = e0 + j < R ? B[j] : 0.f;
        }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        f.A.e[i] = f2(A[4 * i], A[4 * i + 2]);
        f.A.o[i] = f2(A[4 * i + 1], A[4 * i + 3]);
        f.B.e[i] = f2(B[4 * i], B[4 * i + 2]);
        f.B.o[i] = f2(B[4 * i + 1], B[4 * i + 3]);
    }
}

// Norm and rotation of one row (its eight elements of this lane): bf16 pairs in and out.
template <int D, bool HALF>
__device__ __forceinline__ uint4 norm_rotate(const uint4 raw, const Coef &f, float eps, int e0, int R)
{
    constexpr int G = D / 8;
    const uint32_t in[4] = {raw.x, raw.y, raw.z, raw.w};
    const Eight x = unpack8(in);
    float rs = 1.f;
    if (eps >= 0.f) {
        const uint64_t s = fma2(x.o[1], x.o[1], fma2(x.e[1], x.e[1], fma2(x.o[0], x.o[0], mul2(x.e[0], x.e[0]))));
        float ss = lo2(s) + hi2(s);
#pragma unroll
        for (int o = G / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        rs = rsqrtf(ss * (1.f / D) + eps);
    }
    // an interleaved mate is the other element of the pair; the mates of half a row are the
    // eight elements of the lane R/16 further on or back
    Eight m;
    if (HALF) {
        const int lane = threadIdx.x & 31;
        const int src = e0 < R / 2 ? lane + R / 16 : (e0 < R ? lane - R / 16 : lane);
        uint32_t mw[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) mw[j] = __shfl_sync(0xffffffffu, in[j], src);
        if (R < D) {  // elements that do not turn have no mate, whatever the numbers there
#pragma unroll
            for (int j = 0; j < 4; ++j) mw[j] = e0 < R ? mw[j] : 0u;
        }
        m = unpack8(mw);
    } else if (R < D) {
        uint32_t mw[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) mw[j] = e0 + 2 * j < R ? in[j] : 0u;
        const Eight z = unpack8(mw);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            m.e[i] = z.o[i];
            m.o[i] = z.e[i];
        }
    } else {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            m.e[i] = x.o[i];
            m.o[i] = x.e[i];
        }
    }
    const uint64_t r2 = f2(rs, rs);
    uint32_t out[4];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint64_t ye = mul2(r2, fma2(m.e[i], f.B.e[i], mul2(x.e[i], f.A.e[i])));
        const uint64_t yo = mul2(r2, fma2(m.o[i], f.B.o[i], mul2(x.o[i], f.A.o[i])));
        out[2 * i] = pack_bf16x2(lo2(ye), lo2(yo));
        out[2 * i + 1] = pack_bf16x2(hi2(ye), hi2(yo));
    }
    return make_uint4(out[0], out[1], out[2], out[3]);
}

// Largest magnitude (bf16 bits) of the block of 32 elements that this lane and its three
// neighbours hold.
__device__ __forceinline__ uint32_t block_amax(const uint32_t (&w)[4])
{
    const uint32_t M = 0x7fff7fffu;
    uint32_t m = __vmaxu2(__vmaxu2(w[0] & M, w[1] & M), __vmaxu2(w[2] & M, w[3] & M));
    m = max(m & 0xffffu, m >> 16);
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
    return max(m, __shfl_xor_sync(0xffffffffu, m, 2));
}

// NaN -> 0, infinity -> the largest finite value of its sign
__device__ __forceinline__ uint32_t make_finite(uint32_t w)
{
    uint32_t r = 0;
#pragma unroll
    for (int s = 0; s < 32; s += 16) {
        uint32_t h = (w >> s) & 0xffffu;
        if ((h & 0x7fffu) > 0x7f80u) h = 0;
        else if ((h & 0x7fffu) == 0x7f80u) h = (h & 0x8000u) | 0x7f7fu;
        r |= h << s;
    }
    return r;
}

// Store this lane's eight elements of a row as codes (and, one lane per block, the scale).
// row < 0: nothing is stored.  Every lane of the warp calls it.
template <int D>
__device__ __forceinline__ void store_row(uint8_t *codes, uint8_t *scales, int row, uint4 raw, int e0,
                                          int32_t *status)
{
    uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
    uint32_t top = block_amax(w);
    if (__any_sync(0xffffffffu, top >= 0x7f80u)) {
        if (row >= 0 && top >= 0x7f80u) report_status(status, SFA_ERR_INVALID_ARG);
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = make_finite(w[j]);
        top = block_amax(w);
    }
    const uint32_t t = block_exponent_bits(top);
    const float inv = __uint_as_float(((127u + 8u + 127u) << 23) - (t << 16));  // 2^-e; the products are exact
    const uint64_t inv2 = f2(inv, inv);
    const Eight x = unpack8(w);
    uint32_t c4[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint64_t ye = mul2(x.e[i], inv2), yo = mul2(x.o[i], inv2);
        c4[i] = to_e4m3x4(lo2(ye), lo2(yo), hi2(ye), hi2(yo));
    }
    const uint2 c = make_uint2(c4[0], c4[1]);
    if (row >= 0) {
        *reinterpret_cast<uint2 *>(codes + (int64_t)row * D + e0) = c;
        if ((e0 & (CACHE_BLOCK - 1)) == 0)
            scales[(int64_t)row * (D / CACHE_BLOCK) + e0 / CACHE_BLOCK] = (uint8_t)((t >> 7) - 8u);
    }
}

// The rows of a token's key or value heads that a lane visits, from head `head` on in steps of
// `hs`.  The place moves on by an addition: half of what the kernel issues are integer
// instructions, and a 64-bit product per row made 20280 tokens' append 73.9, not 72.4 us.
struct HeadRows {
    const uint16_t *p;
    int64_t inc;
    int head, hs, n;
    __device__ __forceinline__ HeadRows(const uint16_t *base, int b, int h, int i, int e0, int step,
                                        const int64_t (&s)[3], int heads)
        : p(base + (b * s[0] + h * s[1] + i * s[2] + e0)), inc(step * s[1]), head(h), hs(step), n(heads)
    {
    }
    __device__ __forceinline__ uint4 load()
    {
        const uint4 r = head < n ? *reinterpret_cast<const uint4 *>(p) : make_uint4(0u, 0u, 0u, 0u);
        p += inc;
        head += hs;
        return r;
    }
};

// A warp takes a token, or with MANY RW consecutive tokens of the (b, i) order (RW rows at a time,
// D / 8 lanes to a row); where tokens are few, n_parts warps share them.  A group is RW heads of the
// token, or one head of each of the tokens: groups [0, Gq) are the queries', [Gq, Gq + Gk) the
// keys' (and values'), and part p takes the groups g = p mod n_parts.  The angles are formed once
// for all heads.  The loads of the first U groups go out before them, and a group's registers are
// loaded again as soon as it is done, so a warp has rows under way throughout.  With the cache,
// a lane looks up the place of one of the part's key rows before any is stored.
template <int D, bool HALF, bool CACHE, bool MANY>
__global__ void __launch_bounds__(ROW_WARPS * 32, ROW_CTAS) rows_kernel(const __grid_constant__ RowsArgs a)
{
    constexpr int G = D / 8;     // lanes per row
    constexpr int RW = ROWS_AT_ONCE<D>;
    constexpr int T = MANY ? RW : 1;  // tokens
    constexpr int U = CACHE ? 2 : 4;  // query groups under way (append, U = 4: 31 against 29 us)
    __shared__ __align__(16) float cos_all[ROW_WARPS][T][D / 2], sin_all[ROW_WARPS][T][D / 2];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t w = blockIdx.x * (uint32_t)ROW_WARPS + warp;
    if (w >= a.n_warps) return;
    const uint32_t tile = a.n_parts == 1 ? w : w / (uint32_t)a.n_parts;
    const int part = (int)(w - tile * a.n_parts);
    const int sub = lane / G, e0 = (lane % G) * 8;
    // this lane's token; want: it is one, and not a padded row
    const uint32_t token = tile * T + (MANY ? sub : 0), at = MANY ? min(token, a.tokens - 1) : token;
    const int b = (int)(at / (uint32_t)a.L), i = (int)(at - b * (uint32_t)a.L);
    const bool want = token < a.tokens && !(a.lens && i >= __ldg(a.lens + b));
    if (!__any_sync(0xffffffffu, want)) return;
    auto groups = [](int heads) { return MANY ? heads : (heads + RW - 1) / RW; };
    auto head = [&](int g) { return MANY ? g : g * RW + sub; };
    const int Gq = a.q ? groups(a.H) : 0, Gk = a.k ? groups(a.Hk) : 0;
    const int Hq = want ? a.H : 0, Hk = want ? a.Hk : 0;  // this lane's heads
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
    const int step = a.n_parts;

    const uint16_t *q_src = a.q + b * a.qs[0] + i * a.qs[2] + e0;
    auto load_q = [&](int g) {
        const int h = head(g);
        return g < Gq && h < Hq ? *reinterpret_cast<const uint4 *>(q_src + h * a.qs[1]) : zero;
    };
    const uint16_t *k_src = a.k + b * a.ks[0] + i * a.ks[2] + e0;
    auto load_k = [&](int g) {
        const int h = head(g);
        return g < Gk && h < Hk ? *reinterpret_cast<const uint4 *>(k_src + h * a.ks[1]) : zero;
    };
    // this part's first key group: g + Gq = part mod n_parts
    const int first = (part + step - Gq % step) % step;
    // The cache rows of G of its groups from the m0-th on, one of their rows per lane, that of
    // the lanes of sub = lane % RW: where the sequence starts, then the row (or -1).
    const int b_row = MANY ? __shfl_sync(0xffffffffu, b, lane % RW * G) : b;
    const int i_row = MANY ? __shfl_sync(0xffffffffu, i, lane % RW * G) : i;
    const int Hk_row = MANY ? __shfl_sync(0xffffffffu, Hk, lane % RW * G) : Hk;
    auto my_head = [&](int m0) {
        const int g = first + (m0 + lane / RW) * step, h = MANY ? g : g * RW + lane % RW;
        return g < Gk && h < Hk_row ? h : -1;
    };
    auto my_start = [&](int h) { return h < 0 ? 0 : __ldg(a.start + b_row * a.ss0 + h * a.ss1); };
    auto my_row = [&](int h, int start) {
        if (h < 0) return -1;
        const int row = (int)cache_row(a.cache, b_row, h, (int64_t)start + i_row);
        if (row < 0) report_status(a.status, SFA_ERR_BAD_SET);
        return row;
    };
    uint4 x[U];
#pragma unroll
    for (int u = 0; u < U; ++u) x[u] = load_q(part + u * step);
    const int start0 = CACHE ? my_start(my_head(0)) : 0;

#pragma unroll 1
    for (int t = 0; t < T; ++t) {
        const int64_t bt = MANY ? __shfl_sync(0xffffffffu, b, t * G) : b, it = MANY ? __shfl_sync(0xffffffffu, i, t * G) : i;
        const int32_t *pos = a.R ? a.pos + bt * a.ps0 + it * a.ps1 : nullptr;
        for (int p = lane; p < D / 2; p += 32) {
            const float2 r = p < a.R / 2 ? rotation(a, pos, p) : make_float2(1.f, 0.f);
            cos_all[warp][t][p] = r.x;
            sin_all[warp][t][p] = r.y;
        }
    }
    __syncwarp();
    const float *cosp = cos_all[warp][MANY ? sub : 0], *sinp = sin_all[warp][MANY ? sub : 0];

    Coef f;
    if (part < Gq) {
        coefficients<D, HALF>(f, cosp, sinp, a.q_weight, e0, a.R);
        uint16_t *dst = a.q_out + b * a.qo[0] + i * a.qo[2] + e0;
        for (int g0 = part; g0 < Gq; g0 += U * step) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int g = g0 + u * step, h = head(g);
                if (g >= Gq) break;
                const uint4 y = norm_rotate<D, HALF>(x[u], f, a.eps, e0, a.R);
                x[u] = load_q(g + U * step);
                if (h < Hq) *reinterpret_cast<uint4 *>(dst + h * a.qo[1]) = y;
            }
        }
    }
    if (first >= Gk) return;
    if (!CACHE) {
#pragma unroll
        for (int u = 0; u < U; ++u) x[u] = load_k(first + u * step);
        coefficients<D, HALF>(f, cosp, sinp, a.k_weight, e0, a.R);
        uint16_t *dst = a.k_out + b * a.ko[0] + i * a.ko[2] + e0;
        for (int g0 = first; g0 < Gk; g0 += U * step) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int g = g0 + u * step, h = head(g);
                if (g >= Gk) break;
                const uint4 y = norm_rotate<D, HALF>(x[u], f, a.eps, e0, a.R);
                x[u] = load_k(g + U * step);
                if (h < Hk) *reinterpret_cast<uint4 *>(dst + h * a.ko[1]) = y;
            }
        }
    } else {
        coefficients<D, HALF>(f, cosp, sinp, a.k_weight, e0, a.R);
        HeadRows k(a.k, b, head(first), i, e0, MANY ? step : step * RW, a.ks, Hk);
        HeadRows v(a.v, b, head(first), i, e0, MANY ? step : step * RW, a.vs, Hk);
        uint4 kk = k.load(), vv = v.load();
        for (int m0 = 0; first + m0 * step < Gk; m0 += G) {
            const int mine = my_head(m0), row = my_row(mine, m0 ? my_start(mine) : start0);
            for (int m = m0; m < m0 + G; ++m) {
                const int g = first + m * step;
                if (g >= Gk) break;
                const int at = __shfl_sync(0xffffffffu, row, (m - m0) * RW + sub);
                const uint4 y = norm_rotate<D, HALF>(kk, f, a.eps, e0, a.R), z = vv;
                kk = k.load();
                vv = v.load();
                store_row<D>(a.cache.k, a.cache.k_scale, at, y, e0, a.status);
                store_row<D>(a.cache.v, a.cache.v_scale, at, z, e0, a.status);
            }
        }
    }
}

// Keys and values stored as they are: a warp takes consecutive rows of the (b, h, i)
// order; a lane looks up the place of one of them while they load.
template <int D>
__global__ void __launch_bounds__(ROW_WARPS * 32) cache_write_kernel(const __grid_constant__ RowsArgs a)
{
    constexpr int G = D / 8;    // lanes per row
    constexpr int RW = ROWS_AT_ONCE<D>;
    constexpr int STEP = RW * WRITE_U;
    const int lane = threadIdx.x & 31, sub = lane / G, e0 = (lane % G) * 8;
    const uint32_t first = (blockIdx.x * ROW_WARPS + (threadIdx.x >> 5)) * STEP;
    if (first >= a.rows) return;
    const uint32_t r = min(first + lane % STEP, a.rows - 1), bh = r / (uint32_t)a.L;
    const int i = (int)(r - bh * (uint32_t)a.L), b = (int)(bh / (uint32_t)a.Hk), h = (int)(bh - b * (uint32_t)a.Hk);
    const int64_t ko = b * a.ks[0] + h * a.ks[1] + i * a.ks[2], vo = b * a.vs[0] + h * a.vs[1] + i * a.vs[2];
    uint4 x[WRITE_U], y[WRITE_U];
#pragma unroll
    for (int u = 0; u < WRITE_U; ++u) {
        x[u] = *reinterpret_cast<const uint4 *>(a.k + __shfl_sync(0xffffffffu, ko, u * RW + sub) + e0);
        y[u] = *reinterpret_cast<const uint4 *>(a.v + __shfl_sync(0xffffffffu, vo, u * RW + sub) + e0);
    }
    int row = -1;
    if (lane < STEP && first + lane < a.rows && !(a.lens && i >= __ldg(a.lens + b))) {
        row = (int)cache_row(a.cache, b, h, (int64_t)__ldg(a.start + b * a.ss0 + h * a.ss1) + i);
        if (row < 0) report_status(a.status, SFA_ERR_BAD_SET);
    }
#pragma unroll
    for (int u = 0; u < WRITE_U; ++u) {
        const int p = __shfl_sync(0xffffffffu, row, u * RW + sub);
        store_row<D>(a.cache.k, a.cache.k_scale, p, x[u], e0, a.status);
        store_row<D>(a.cache.v, a.cache.v_scale, p, y[u], e0, a.status);
    }
}

// ----------------------------------------------------------------- reading back
struct ReadArgs {
    CacheView cache;
    int32_t B, Hk, L;
    const int32_t *start, *lens;
    int64_t ss0, ss1;
    uint16_t *k_out, *v_out;
    int64_t ko[3], vo[3];
    int32_t *status;
    uint32_t rows;  // B * Hk * L
};

// Eight codes and their block's scale -> eight bf16 numbers.
__device__ __forceinline__ uint4 from_codes(uint2 c, uint32_t scale_byte)
{
    const uint32_t f = scale_bits(scale_byte) * 0x10001u, g = scale_rest_bits(scale_byte) * 0x10001u;
    uint4 r;
    r.x = mul_bf16x2(mul_bf16x2(spread_codes<CODES_01>(c.x, c.x), f), g);
    r.y = mul_bf16x2(mul_bf16x2(spread_codes<CODES_23>(c.x, c.x), f), g);
    r.z = mul_bf16x2(mul_bf16x2(spread_codes<CODES_01>(c.y, c.y), f), g);
    r.w = mul_bf16x2(mul_bf16x2(spread_codes<CODES_23>(c.y, c.y), f), g);
    return r;
}

// A warp takes STEP consecutive rows of the (b, h, i) order: a lane looks up the place of one
// of them, then D / 8 lanes share a row, eight elements each, with READ_U rows of a lane under
// way together.  Consecutive rows matter most: with a warp's rows a grid apart, and each lane
// looking up its own, 20280 tokens of 12 heads, d = 128, took 43.7 us, now 33.4 (5.65 TB/s), and
// 60000 tokens 119, now 89 (6.3 TB/s).  Longer stretches a warp: 33.3 and 93 (16 CTAs per SM) to
// 37.8 and 104 (4).
template <int D>
__global__ void __launch_bounds__(ROW_WARPS * 32) cache_read_kernel(const __grid_constant__ ReadArgs a)
{
    constexpr int G = D / 8;    // lanes per row
    constexpr int RW = ROWS_AT_ONCE<D>;
    constexpr int STEP = RW * READ_U;
    const int lane = threadIdx.x & 31, sub = lane / G, e0 = (lane % G) * 8;
    const uint32_t first = (blockIdx.x * ROW_WARPS + (threadIdx.x >> 5)) * STEP;
    if (first >= a.rows) return;
    const uint32_t r = min(first + lane % STEP, a.rows - 1), bh = r / (uint32_t)a.L;
    const int i = (int)(r - bh * (uint32_t)a.L), b = (int)(bh / (uint32_t)a.Hk), h = (int)(bh - b * (uint32_t)a.Hk);
    int row = -1;
    if (lane < STEP && first + lane < a.rows && !(a.lens && i >= __ldg(a.lens + b))) {
        row = (int)cache_row(a.cache, b, h, (int64_t)__ldg(a.start + b * a.ss0 + h * a.ss1) + i);
        if (row < 0) report_status(a.status, SFA_ERR_BAD_SET);
    }
    const int64_t ko = b * a.ko[0] + h * a.ko[1] + i * a.ko[2], vo = b * a.vo[0] + h * a.vo[1] + i * a.vo[2];
    uint2 kc[READ_U], vc[READ_U];
    uint32_t ks[READ_U], vs[READ_U];
    int at[READ_U];
#pragma unroll
    for (int u = 0; u < READ_U; ++u) {
        at[u] = __shfl_sync(~0u, row, u * RW + sub);
        const int64_t p = max(at[u], 0);  // (row 0 is always there: no branch parts the loads)
        kc[u] = load_codes8(a.cache.k + p * D + e0);
        vc[u] = load_codes8(a.cache.v + p * D + e0);
        ks[u] = __ldg(a.cache.k_scale + p * (D / CACHE_BLOCK) + e0 / CACHE_BLOCK);
        vs[u] = __ldg(a.cache.v_scale + p * (D / CACHE_BLOCK) + e0 / CACHE_BLOCK);
    }
#pragma unroll
    for (int u = 0; u < READ_U; ++u) {
        const int64_t ku = __shfl_sync(~0u, ko, u * RW + sub) + e0, vu = __shfl_sync(~0u, vo, u * RW + sub) + e0;
        if (at[u] < 0) continue;
        *reinterpret_cast<uint4 *>(a.k_out + ku) = from_codes(kc[u], ks[u]);
        *reinterpret_cast<uint4 *>(a.v_out + vu) = from_codes(vc[u], vs[u]);
    }
}

// ----------------------------------------------------------------- host side
int device_sms()
{
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    return sms > 0 ? sms : 148;
}

// norm weights are read 16 bytes at a time
bool weights_ok(const float *q, const float *k)
{
    return reinterpret_cast<uintptr_t>(q) % 16 == 0 && reinterpret_cast<uintptr_t>(k) % 16 == 0;
}

bool aligned16(const void *p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

sfa_status check_rows(const sfa_rows_desc *d)
{
    if (!d || d->B < 0 || d->L < 0) return SFA_ERR_INVALID_ARG;
    if (d->d != 64 && d->d != 128) return SFA_ERR_UNSUPPORTED;
    if (!(d->eps < 0.f) && !std::isfinite(d->eps)) return SFA_ERR_INVALID_ARG;
    return SFA_OK;
}

bool heads_ok(int32_t h) { return h >= 1 && h <= SFA_MAX_HEADS; }

sfa_status check_rope(const sfa_rope *r, int32_t d)
{
    if (!r) return SFA_OK;
    if (!r->inv_freq || !r->positions || reinterpret_cast<uintptr_t>(r->inv_freq) % 8 ||
        reinterpret_cast<uintptr_t>(r->positions) % 4)
        return SFA_ERR_INVALID_ARG;
    if (r->layout != SFA_ROPE_INTERLEAVED && r->layout != SFA_ROPE_HALF) return SFA_ERR_INVALID_ARG;
    if (r->n_axes < 1 || r->n_axes > SFA_ROPE_MAX_AXES || !std::isfinite(r->scale)) return SFA_ERR_INVALID_ARG;
    if (r->pos_stride[0] < 0 || r->pos_stride[1] < 0) return SFA_ERR_INVALID_ARG;
    int pairs = 0;
    for (int i = 0; i < r->n_axes; ++i) {
        if (r->axis_pairs[i] < 0 || r->axis_pairs[i] > d / 2) return SFA_ERR_INVALID_ARG;
        pairs += r->axis_pairs[i];
    }
    if (pairs < 1 || 2 * pairs > d) return SFA_ERR_INVALID_ARG;
    if (r->layout == SFA_ROPE_HALF && pairs % 8) return SFA_ERR_UNSUPPORTED;
    return SFA_OK;
}

void copy3(int64_t (&to)[3], const int64_t *from)
{
    for (int i = 0; i < 3; ++i) to[i] = from[i];
}

void fill_rope(RowsArgs &a, const sfa_rope *r)
{
    a.R = 0;
    a.n_axes = 0;
    if (!r) return;
    a.inv_freq = r->inv_freq;
    a.pos = r->positions;
    a.ps0 = r->pos_stride[0];
    a.ps1 = r->pos_stride[1];
    a.n_axes = r->n_axes;
    a.rope_scale = r->scale;
    int pairs = 0;
    for (int i = 0; i < r->n_axes; ++i) a.axis_end[i] = pairs += r->axis_pairs[i];
    a.R = 2 * pairs;
}

template <bool CACHE, bool MANY>
sfa_status launch_rows(RowsArgs &a, int d, bool half, cudaStream_t s)
{
    const int rw = d == 128 ? ROWS_AT_ONCE<128> : ROWS_AT_ONCE<64>;
    const int heads_at_once = MANY ? 1 : rw, tokens_at_once = MANY ? rw : 1;
    const int groups = (a.q ? (a.H + heads_at_once - 1) / heads_at_once : 0) + (a.k ? (a.Hk + heads_at_once - 1) / heads_at_once : 0);
    const int64_t tokens = (int64_t)a.B * a.L, tiles = (tokens + tokens_at_once - 1) / tokens_at_once;
    // Warps per tile of tokens: one (the angles are formed once) while the tiles alone give every SM
    // 16 warps, else as many as do, at most one per row group.  (Norm and rotation of 12 + 12
    // heads with 8, 16, 32 and 64 warps an SM: 200 tokens of 8 sequences 8.2, 7.4, 9.4 and
    // 12.3 us; 1560 tokens 7.6, 6.8, 9.3 and 12.5; 4680 tokens 13.6, 13.7, 16.9 and 20.3.)
    const int64_t want = ((int64_t)device_sms() * 16 + tiles - 1) / tiles;
    a.n_parts = (int32_t)(want < 1 ? 1 : (want > groups ? groups : want));
    if (tokens >= ((int64_t)1 << 31)) return SFA_ERR_INVALID_ARG;  // (parts: only where tokens are few)
    a.tokens = (uint32_t)tokens;
    a.n_warps = (uint32_t)tiles * (uint32_t)a.n_parts;
    const int64_t grid = ((int64_t)a.n_warps + ROW_WARPS - 1) / ROW_WARPS;
    const dim3 g((unsigned)grid), t(ROW_WARPS * 32);
    if (d == 128 && half) rows_kernel<128, true, CACHE, MANY><<<g, t, 0, s>>>(a);
    else if (d == 128) rows_kernel<128, false, CACHE, MANY><<<g, t, 0, s>>>(a);
    else if (half) rows_kernel<64, true, CACHE, MANY><<<g, t, 0, s>>>(a);
    else rows_kernel<64, false, CACHE, MANY><<<g, t, 0, s>>>(a);
    return launch_status();
}

// Several tokens a warp: with few heads, whose rows would leave lanes idle and the coefficients
// unshared, once there are more tokens than warps fit on the GPU.  Norm and rotation of 20000
// tokens, one and several a warp, H + H_kv = 2, 8, 12, 24: d = 128 19.3, 26.3, 31.2, 47.4 and
// 13.3, 23.3, 29.4, 49.9 us; d = 64 16.8, 19.4, 23.3, 29.2 and 8.5, 14.4, 18.2, 30.6; 2400 tokens,
// H + H_kv = 2, 8: 4.7, 5.4 and 4.6, 6.0.  Append at d = 128 24.5, 34.4, 43.0, 70.7 and 16.8, 32.5,
// 42.8, 74.1.
template <bool CACHE>
sfa_status launch_rows(RowsArgs &a, int d, bool half, cudaStream_t s)
{
    const int heads = (a.q ? a.H : 0) + (a.k ? a.Hk : 0);
    const bool many = heads <= 12 && (int64_t)a.B * a.L > (int64_t)device_sms() * ROW_WARPS * ROW_CTAS;
    return many ? launch_rows<CACHE, true>(a, d, half, s) : launch_rows<CACHE, false>(a, d, half, s);
}

void fill_cache(RowsArgs &a, const sfa_rows_desc *d, const sfa_cache *cache, const void *k, const void *v,
                const int32_t *start, const int32_t *lens, int32_t *status)
{
    a.k = static_cast<const uint16_t *>(k);
    a.v = static_cast<const uint16_t *>(v);
    copy3(a.ks, d->k_stride);
    copy3(a.vs, d->v_stride);
    a.cache = cache_view(cache);
    a.start = start;
    a.ss0 = d->start_stride[0];
    a.ss1 = d->start_stride[1];
    a.lens = lens;
    a.status = status;
}

sfa_status check_cache_rows(const sfa_rows_desc *d, const sfa_cache *cache, const int32_t *start)
{
    if (!heads_ok(d->H_kv)) return SFA_ERR_INVALID_ARG;
    sfa_status st = check_cache(cache, d->H_kv, d->d);
    if (st != SFA_OK) return st;
    if (!start || d->start_stride[0] < 0 || d->start_stride[1] < 0) return SFA_ERR_INVALID_ARG;
    return SFA_OK;
}

// Pages of one head each, one row of them for all heads and one start: every head would be
// written to the same places.
bool heads_collide(const sfa_rows_desc *d, const sfa_cache *c)
{
    return c->heads == 1 && d->H_kv > 1 && c->table_stride[1] == 0 && d->start_stride[1] == 0;
}

}  // namespace
}  // namespace sfa

using namespace sfa;

extern "C" sfa_status sfa_qk_norm_rope(const sfa_rows_desc *d, const sfa_rope *rope, const void *q, const void *k,
                                       const float *q_weight, const float *k_weight, void *q_out, void *k_out,
                                       sfa_stream_t stream)
{
    sfa_status st = check_rows(d);
    if (st == SFA_OK) st = check_rope(rope, d->d);
    if (st != SFA_OK) return st;
    if (d->B == 0 || d->L == 0) return SFA_OK;
    if ((!q && !k) || !q != !q_out || !k != !k_out) return SFA_ERR_INVALID_ARG;
    if ((q && !heads_ok(d->H)) || (k && !heads_ok(d->H_kv))) return SFA_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k) || !aligned16(q_out) || !aligned16(k_out) || !weights_ok(q_weight, k_weight))
        return SFA_ERR_INVALID_ARG;
    if (q && (!rows_stride_ok(d->q_stride, d->B, d->H, d->L) || !rows_stride_ok(d->q_out_stride, d->B, d->H, d->L)))
        return SFA_ERR_INVALID_ARG;
    if (k && (!rows_stride_ok(d->k_stride, d->B, d->H_kv, d->L) || !rows_stride_ok(d->k_out_stride, d->B, d->H_kv, d->L)))
        return SFA_ERR_INVALID_ARG;
    if (q && k && (q_out == k || k_out == q || q_out == k_out)) return SFA_ERR_INVALID_ARG;
    if ((q && !in_place_ok(q, q_out, d->q_stride, d->q_out_stride, d->B, d->H, d->L)) ||
        (k && !in_place_ok(k, k_out, d->k_stride, d->k_out_stride, d->B, d->H_kv, d->L)))
        return SFA_ERR_INVALID_ARG;
    RowsArgs a = {};
    a.B = d->B;
    a.H = d->H;
    a.Hk = d->H_kv;
    a.L = d->L;
    a.q = static_cast<const uint16_t *>(q);
    a.k = static_cast<const uint16_t *>(k);
    a.q_out = static_cast<uint16_t *>(q_out);
    a.k_out = static_cast<uint16_t *>(k_out);
    copy3(a.qs, d->q_stride);
    copy3(a.ks, d->k_stride);
    copy3(a.qo, d->q_out_stride);
    copy3(a.ko, d->k_out_stride);
    a.q_weight = q_weight;
    a.k_weight = k_weight;
    a.eps = d->eps;
    fill_rope(a, rope);
    return launch_rows<false>(a, d->d, rope && rope->layout == SFA_ROPE_HALF, as_cuda(stream));
}

extern "C" sfa_status sfa_cache_write(const sfa_rows_desc *d, const sfa_cache *cache, const void *k, const void *v,
                                      const int32_t *start, const int32_t *lens, int32_t *dev_status,
                                      sfa_stream_t stream)
{
    sfa_status st = check_rows(d);
    if (st != SFA_OK) return st;
    if (d->B == 0 || d->L == 0) return SFA_OK;
    st = check_cache_rows(d, cache, start);
    if (st != SFA_OK) return st;
    if (!k || !v || !aligned16(k) || !aligned16(v) || heads_collide(d, cache)) return SFA_ERR_INVALID_ARG;
    if (!rows_stride_ok(d->k_stride, d->B, d->H_kv, d->L) || !rows_stride_ok(d->v_stride, d->B, d->H_kv, d->L))
        return SFA_ERR_INVALID_ARG;
    RowsArgs a = {};
    a.B = d->B;
    a.Hk = d->H_kv;
    a.L = d->L;
    a.eps = -1.f;
    fill_cache(a, d, cache, k, v, start, lens, dev_status);
    const int64_t rows = (int64_t)d->B * d->H_kv * d->L;
    if ((int64_t)d->B * d->L >= ((int64_t)1 << 31) || rows >= ((int64_t)1 << 31)) return SFA_ERR_INVALID_ARG;
    a.rows = (uint32_t)rows;
    const int per_cta = ROW_WARPS * WRITE_U * (d->d == 128 ? ROWS_AT_ONCE<128> : ROWS_AT_ONCE<64>);
    const unsigned grid = (unsigned)((rows + per_cta - 1) / per_cta);
    if (d->d == 128) cache_write_kernel<128><<<grid, ROW_WARPS * 32, 0, as_cuda(stream)>>>(a);
    else cache_write_kernel<64><<<grid, ROW_WARPS * 32, 0, as_cuda(stream)>>>(a);
    return launch_status();
}

extern "C" sfa_status sfa_cache_append(const sfa_rows_desc *d, const sfa_rope *rope, const sfa_cache *cache,
                                       const void *q, const void *k, const void *v, const float *q_weight,
                                       const float *k_weight, void *q_out, const int32_t *start, const int32_t *lens,
                                       int32_t *dev_status, sfa_stream_t stream)
{
    sfa_status st = check_rows(d);
    if (st == SFA_OK) st = check_rope(rope, d->d);
    if (st != SFA_OK) return st;
    if (d->B == 0 || d->L == 0) return SFA_OK;
    st = check_cache_rows(d, cache, start);
    if (st != SFA_OK) return st;
    if (!q || !k || !v || !q_out || !heads_ok(d->H) || heads_collide(d, cache)) return SFA_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(q_out) || !weights_ok(q_weight, k_weight))
        return SFA_ERR_INVALID_ARG;
    if (!rows_stride_ok(d->q_stride, d->B, d->H, d->L) || !rows_stride_ok(d->q_out_stride, d->B, d->H, d->L) ||
        !rows_stride_ok(d->k_stride, d->B, d->H_kv, d->L) || !rows_stride_ok(d->v_stride, d->B, d->H_kv, d->L))
        return SFA_ERR_INVALID_ARG;
    if (q_out == k || q_out == v || !in_place_ok(q, q_out, d->q_stride, d->q_out_stride, d->B, d->H, d->L))
        return SFA_ERR_INVALID_ARG;
    RowsArgs a = {};
    a.B = d->B;
    a.H = d->H;
    a.Hk = d->H_kv;
    a.L = d->L;
    a.q = static_cast<const uint16_t *>(q);
    a.q_out = static_cast<uint16_t *>(q_out);
    copy3(a.qs, d->q_stride);
    copy3(a.qo, d->q_out_stride);
    a.q_weight = q_weight;
    a.k_weight = k_weight;
    a.eps = d->eps;
    fill_rope(a, rope);
    fill_cache(a, d, cache, k, v, start, lens, dev_status);
    return launch_rows<true>(a, d->d, rope && rope->layout == SFA_ROPE_HALF, as_cuda(stream));
}

extern "C" sfa_status sfa_cache_read(const sfa_rows_desc *d, const sfa_cache *cache, const int32_t *start,
                                     const int32_t *lens, void *k_out, void *v_out, int32_t *dev_status,
                                     sfa_stream_t stream)
{
    sfa_status st = check_rows(d);
    if (st != SFA_OK) return st;
    if (d->B == 0 || d->L == 0) return SFA_OK;
    st = check_cache_rows(d, cache, start);
    if (st != SFA_OK) return st;
    if (!k_out || !v_out || k_out == v_out || !aligned16(k_out) || !aligned16(v_out)) return SFA_ERR_INVALID_ARG;
    if (!rows_stride_ok(d->k_out_stride, d->B, d->H_kv, d->L) || !rows_stride_ok(d->v_out_stride, d->B, d->H_kv, d->L))
        return SFA_ERR_INVALID_ARG;
    ReadArgs a = {};
    a.cache = cache_view(cache);
    a.B = d->B;
    a.Hk = d->H_kv;
    a.L = d->L;
    a.start = start;
    a.lens = lens;
    a.ss0 = d->start_stride[0];
    a.ss1 = d->start_stride[1];
    a.k_out = static_cast<uint16_t *>(k_out);
    a.v_out = static_cast<uint16_t *>(v_out);
    copy3(a.ko, d->k_out_stride);
    copy3(a.vo, d->v_out_stride);
    a.status = dev_status;
    const int64_t rows = (int64_t)d->B * d->H_kv * d->L;
    if ((int64_t)d->B * d->L >= ((int64_t)1 << 31) || rows >= ((int64_t)1 << 31)) return SFA_ERR_INVALID_ARG;
    a.rows = (uint32_t)rows;
    const int per_cta = ROW_WARPS * READ_U * (d->d == 128 ? ROWS_AT_ONCE<128> : ROWS_AT_ONCE<64>);
    const unsigned grid = (unsigned)((rows + per_cta - 1) / per_cta);
    if (d->d == 128) cache_read_kernel<128><<<grid, ROW_WARPS * 32, 0, as_cuda(stream)>>>(a);
    else cache_read_kernel<64><<<grid, ROW_WARPS * 32, 0, as_cuda(stream)>>>(a);
    return launch_status();
}
