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
//   * a warp owns a token, so the R/2 angles (fp64, reduced to one turn) and their sine and
//     cosine are formed once for all its heads and kept in shared memory, then folded with
//     the norm's weight into two coefficients per element: y = rs (x A + x_partner B);
//   * a token's head rows are loaded several at a time before any arithmetic; with few
//     tokens they are dealt out over several warps (one row group each at a single token).
#include <cmath>
#include <cstdint>

#include <cuda_runtime.h>

#include "sfa.h"
#include "sfa_cache.cuh"
#include "sfa_internal.h"
#include "sfa_ptx.cuh"

namespace sfa {
namespace {

constexpr int ROW_WARPS = 8;  // warps per CTA

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
    int64_t n_warps;   // B * L * n_parts
};

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// cosine and sine (times the scale) of pair p at this token.  A far position times a
// frequency loses its fraction of a turn in fp32, so the product is formed and reduced to
// [-1, 1] half turns in fp64; what is left is exact to fp32.
__device__ __forceinline__ float2 rotation(const RowsArgs &a, const int32_t *pos, int p)
{
    int ax = 0;
#pragma unroll
    for (int i = 0; i < SFA_ROPE_MAX_AXES - 1; ++i) ax += (i < a.n_axes - 1 && p >= a.axis_end[i]) ? 1 : 0;
    const double t = (double)__ldg(pos + ax) * __ldg(a.inv_freq + p) * 0.31830988618379067154;
    float s, c;
    sincospif((float)(t - 2.0 * rint(0.5 * t)), &s, &c);
    return make_float2(c * a.rope_scale, s * a.rope_scale);
}

// y = rs * (x * A + x_partner * B) for this lane's eight elements
struct Coef {
    float A[8], B[8];
};

template <int D, bool HALF>
__device__ __forceinline__ void coefficients(Coef &f, const float2 *cs, const float *w, int e0, int R)
{
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int e = e0 + j;
        const float we = w ? __ldg(w + e) : 1.f;
        f.A[j] = we;
        f.B[j] = 0.f;
        if (e < R) {
            const bool first = HALF ? e < R / 2 : (j & 1) == 0;
            const int mate = HALF ? (first ? e + R / 2 : e - R / 2) : (e ^ 1);
            const float2 r = cs[HALF ? (first ? e : mate) : e >> 1];
            const float wm = w ? __ldg(w + mate) : 1.f;
            f.A[j] = we * r.x;
            f.B[j] = first ? -wm * r.y : wm * r.y;
        }
    }
}

// Norm and rotation of one row (its eight elements of this lane): bf16 pairs in and out.
template <int D, bool HALF>
__device__ __forceinline__ uint4 norm_rotate(const uint4 raw, const Coef &f, float eps, int e0, int R)
{
    constexpr int G = D / 8;
    const uint32_t in[4] = {raw.x, raw.y, raw.z, raw.w};
    float x[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        x[2 * j] = bf_lo(in[j]);
        x[2 * j + 1] = bf_hi(in[j]);
    }
    float rs = 1.f;
    if (eps >= 0.f) {
        float ss = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) ss = fmaf(x[j], x[j], ss);
#pragma unroll
        for (int o = G / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        rs = rsqrtf(ss * (1.f / D) + eps);
    }
    float y[8];
    if (HALF) {
        // the partners are the eight elements of the lane R/16 further on or back
        const int lane = threadIdx.x & 31;
        const int src = e0 < R / 2 ? lane + R / 16 : (e0 < R ? lane - R / 16 : lane);
        uint32_t m[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) m[j] = __shfl_sync(0xffffffffu, in[j], src);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float mate = (j & 1) ? bf_hi(m[j >> 1]) : bf_lo(m[j >> 1]);
            y[j] = rs * (x[j] * f.A[j] + (e0 < R ? mate * f.B[j] : 0.f));
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = rs * (x[j] * f.A[j] + (e0 + j < R ? x[j ^ 1] * f.B[j] : 0.f));
    }
    return make_uint4(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]), pack_bf16x2(y[4], y[5]),
                      pack_bf16x2(y[6], y[7]));
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
__device__ __forceinline__ void store_row(uint8_t *codes, uint8_t *scales, int64_t row, uint4 raw, int e0,
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
    const int e = block_exponent(top);
    const float inv = __uint_as_float((uint32_t)(127 - e) << 23);  // 2^-e; the products are exact
    uint2 c;
    c.x = to_e4m3x2(bf_lo(w[0]) * inv, bf_hi(w[0]) * inv) | (to_e4m3x2(bf_lo(w[1]) * inv, bf_hi(w[1]) * inv) << 16);
    c.y = to_e4m3x2(bf_lo(w[2]) * inv, bf_hi(w[2]) * inv) | (to_e4m3x2(bf_lo(w[3]) * inv, bf_hi(w[3]) * inv) << 16);
    if (row >= 0) {
        *reinterpret_cast<uint2 *>(codes + row * D + e0) = c;
        if ((e0 & (CACHE_BLOCK - 1)) == 0) scales[row * (D / CACHE_BLOCK) + e0 / CACHE_BLOCK] = (uint8_t)(e + 127);
    }
}

// One warp per token, or one of n_parts warps that share a token's row groups: groups
// [0, Gq) are the query heads, [Gq, Gq + Gk) the key (and value) heads, RW heads a group,
// and part p takes the groups g = p mod n_parts.
template <int D, bool HALF, bool CACHE>
__global__ void __launch_bounds__(ROW_WARPS * 32) rows_kernel(const __grid_constant__ RowsArgs a)
{
    constexpr int G = D / 8;     // lanes per row
    constexpr int RW = 32 / G;   // rows of a group
    constexpr int UQ = 4;        // groups loaded before any arithmetic
    constexpr int UK = CACHE ? 2 : 4;
    __shared__ float2 cs_all[ROW_WARPS][D / 2];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t w = (int64_t)blockIdx.x * ROW_WARPS + warp;
    if (w >= a.n_warps) return;
    const int64_t token = w / a.n_parts;
    const int part = (int)(w - token * a.n_parts);
    const int b = (int)(token / a.L), i = (int)(token - (int64_t)b * a.L);
    if (a.lens && i >= __ldg(a.lens + b)) return;  // a padded row (the whole warp)
    float2 *cs = cs_all[warp];
    const int32_t *pos = a.R ? a.pos + b * a.ps0 + i * a.ps1 : nullptr;
    for (int p = lane; p < a.R / 2; p += 32) cs[p] = rotation(a, pos, p);
    __syncwarp();
    const int sub = lane / G, e0 = (lane % G) * 8;
    const int Gq = a.q ? (a.H + RW - 1) / RW : 0;
    const int Gk = (a.k || a.v) ? (a.Hk + RW - 1) / RW : 0;
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);

    Coef f;
    if (part < Gq) {
        coefficients<D, HALF>(f, cs, a.q_weight, e0, a.R);
        const uint16_t *src = a.q + b * a.qs[0] + i * a.qs[2] + e0;
        uint16_t *dst = a.q_out + b * a.qo[0] + i * a.qo[2] + e0;
        for (int g0 = part; g0 < Gq; g0 += UQ * a.n_parts) {
            uint4 x[UQ];
#pragma unroll
            for (int u = 0; u < UQ; ++u) {
                const int h = (g0 + u * a.n_parts) * RW + sub;
                x[u] = h < a.H ? *reinterpret_cast<const uint4 *>(src + h * a.qs[1]) : zero;
            }
#pragma unroll
            for (int u = 0; u < UQ; ++u) {
                const int h = (g0 + u * a.n_parts) * RW + sub;
                const uint4 y = norm_rotate<D, HALF>(x[u], f, a.eps, e0, a.R);
                if (h < a.H) *reinterpret_cast<uint4 *>(dst + h * a.qo[1]) = y;
            }
        }
    }
    // this part's first key group: g + Gq = part mod n_parts
    const int first = (part + a.n_parts - Gq % a.n_parts) % a.n_parts;
    if (first >= Gk) return;
    const bool plain = a.eps < 0.f && a.R == 0 && !a.k_weight;  // keys stored as they are
    if (!plain) coefficients<D, HALF>(f, cs, a.k_weight, e0, a.R);
    const uint16_t *k_src = a.k + b * a.ks[0] + i * a.ks[2] + e0;
    if (!CACHE) {
        uint16_t *dst = a.k_out + b * a.ko[0] + i * a.ko[2] + e0;
        for (int g0 = first; g0 < Gk; g0 += UK * a.n_parts) {
            uint4 x[UK];
#pragma unroll
            for (int u = 0; u < UK; ++u) {
                const int h = (g0 + u * a.n_parts) * RW + sub;
                x[u] = h < a.Hk ? *reinterpret_cast<const uint4 *>(k_src + h * a.ks[1]) : zero;
            }
#pragma unroll
            for (int u = 0; u < UK; ++u) {
                const int h = (g0 + u * a.n_parts) * RW + sub;
                const uint4 y = norm_rotate<D, HALF>(x[u], f, a.eps, e0, a.R);
                if (h < a.Hk) *reinterpret_cast<uint4 *>(dst + h * a.ko[1]) = y;
            }
        }
    } else {
        const uint16_t *v_src = a.v + b * a.vs[0] + i * a.vs[2] + e0;
        for (int g0 = first; g0 < Gk; g0 += UK * a.n_parts) {
            uint4 x[UK], y[UK];
            int64_t row[UK];
#pragma unroll
            for (int u = 0; u < UK; ++u) {
                const int h = (g0 + u * a.n_parts) * RW + sub;
                const bool on = h < a.Hk;
                x[u] = on ? *reinterpret_cast<const uint4 *>(k_src + h * a.ks[1]) : zero;
                y[u] = on ? *reinterpret_cast<const uint4 *>(v_src + h * a.vs[1]) : zero;
                row[u] = -1;
                if (on) {
                    row[u] = cache_row(a.cache, b, h, (int64_t)__ldg(a.start + b * a.ss0 + h * a.ss1) + i);
                    if (row[u] < 0) report_status(a.status, SFA_ERR_BAD_SET);
                }
            }
#pragma unroll
            for (int u = 0; u < UK; ++u) {
                if (!plain) x[u] = norm_rotate<D, HALF>(x[u], f, a.eps, e0, a.R);
                store_row<D>(a.cache.k, a.cache.k_scale, row[u], x[u], e0, a.status);
                store_row<D>(a.cache.v, a.cache.v_scale, row[u], y[u], e0, a.status);
            }
        }
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
    int64_t rows;  // B * Hk * L
};

// Eight codes and their block's scale -> eight bf16 numbers.
__device__ __forceinline__ uint4 from_codes(uint2 c, uint32_t scale_byte)
{
    const uint32_t f = scale_bits(scale_byte) * 0x10001u, g = scale_rest_bits(scale_byte) * 0x10001u;
    uint4 r;
    r.x = mul_bf16x2(mul_bf16x2(spread_codes(__byte_perm(c.x, 0, 0x1100)), f), g);
    r.y = mul_bf16x2(mul_bf16x2(spread_codes(__byte_perm(c.x, 0, 0x3322)), f), g);
    r.z = mul_bf16x2(mul_bf16x2(spread_codes(__byte_perm(c.y, 0, 0x1100)), f), g);
    r.w = mul_bf16x2(mul_bf16x2(spread_codes(__byte_perm(c.y, 0, 0x3322)), f), g);
    return r;
}

template <int D>
__global__ void __launch_bounds__(256) cache_read_kernel(const __grid_constant__ ReadArgs a)
{
    constexpr int G = D / 8;  // lanes per row
    constexpr int U = 4;      // rows per lane group, all their loads issued first
    const int64_t group = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) / G;
    const int64_t n_groups = (int64_t)gridDim.x * blockDim.x / G;
    const int e0 = (threadIdx.x % G) * 8;
    for (int64_t r0 = group; r0 < a.rows; r0 += n_groups * U) {
        uint2 kc[U], vc[U];
        uint32_t ks[U], vs[U];
        int64_t row[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t r = r0 + u * n_groups;
            row[u] = -1;
            if (r >= a.rows) continue;
            const int64_t bh = r / a.L;
            const int i = (int)(r - bh * a.L), b = (int)(bh / a.Hk), h = (int)(bh - (int64_t)b * a.Hk);
            if (a.lens && i >= __ldg(a.lens + b)) continue;
            row[u] = cache_row(a.cache, b, h, (int64_t)__ldg(a.start + b * a.ss0 + h * a.ss1) + i);
            if (row[u] < 0) {
                report_status(a.status, SFA_ERR_BAD_SET);
                continue;
            }
            kc[u] = *reinterpret_cast<const uint2 *>(a.cache.k + row[u] * D + e0);
            vc[u] = *reinterpret_cast<const uint2 *>(a.cache.v + row[u] * D + e0);
            ks[u] = a.cache.k_scale[row[u] * (D / CACHE_BLOCK) + e0 / CACHE_BLOCK];
            vs[u] = a.cache.v_scale[row[u] * (D / CACHE_BLOCK) + e0 / CACHE_BLOCK];
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (row[u] < 0) continue;
            const int64_t r = r0 + u * n_groups;
            const int64_t bh = r / a.L;
            const int64_t i = r - bh * a.L, b = bh / a.Hk, h = bh - b * a.Hk;
            *reinterpret_cast<uint4 *>(a.k_out + b * a.ko[0] + h * a.ko[1] + i * a.ko[2] + e0) = from_codes(kc[u], ks[u]);
            *reinterpret_cast<uint4 *>(a.v_out + b * a.vo[0] + h * a.vo[1] + i * a.vo[2] + e0) = from_codes(vc[u], vs[u]);
        }
    }
}

// ----------------------------------------------------------------- host side
int device_sms()
{
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    return sms > 0 ? sms : 148;
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

template <bool CACHE>
sfa_status launch_rows(RowsArgs &a, int d, bool half, cudaStream_t s)
{
    const int rw = 32 / (d / 8);
    const int groups = (a.q ? (a.H + rw - 1) / rw : 0) + ((a.k || a.v) ? (a.Hk + rw - 1) / rw : 0);
    const int64_t tokens = (int64_t)a.B * a.L;
    // Warps per token: one (the angles are formed once) while the tokens alone fill the SMs
    // with 32 warps each, else as many as fill them, at most one per row group.
    const int64_t want = ((int64_t)device_sms() * 32 + tokens - 1) / tokens;
    a.n_parts = (int32_t)(want < 1 ? 1 : (want > groups ? groups : want));
    a.n_warps = tokens * a.n_parts;
    const int64_t grid = (a.n_warps + ROW_WARPS - 1) / ROW_WARPS;
    if (tokens >= ((int64_t)1 << 31) || grid >= ((int64_t)1 << 31)) return SFA_ERR_INVALID_ARG;
    const dim3 g((unsigned)grid), t(ROW_WARPS * 32);
    if (d == 128 && half) rows_kernel<128, true, CACHE><<<g, t, 0, s>>>(a);
    else if (d == 128) rows_kernel<128, false, CACHE><<<g, t, 0, s>>>(a);
    else if (half) rows_kernel<64, true, CACHE><<<g, t, 0, s>>>(a);
    else rows_kernel<64, false, CACHE><<<g, t, 0, s>>>(a);
    return launch_status();
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
    if (!aligned16(q) || !aligned16(k) || !aligned16(q_out) || !aligned16(k_out)) return SFA_ERR_INVALID_ARG;
    if (q && (!rows_stride_ok(d->q_stride, d->B, d->H, d->L) || !rows_stride_ok(d->q_out_stride, d->B, d->H, d->L)))
        return SFA_ERR_INVALID_ARG;
    if (k && (!rows_stride_ok(d->k_stride, d->B, d->H_kv, d->L) || !rows_stride_ok(d->k_out_stride, d->B, d->H_kv, d->L)))
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
    if (!k || !v || !aligned16(k) || !aligned16(v)) return SFA_ERR_INVALID_ARG;
    if (!rows_stride_ok(d->k_stride, d->B, d->H_kv, d->L) || !rows_stride_ok(d->v_stride, d->B, d->H_kv, d->L))
        return SFA_ERR_INVALID_ARG;
    RowsArgs a = {};
    a.B = d->B;
    a.Hk = d->H_kv;
    a.L = d->L;
    a.eps = -1.f;
    fill_cache(a, d, cache, k, v, start, lens, dev_status);
    return launch_rows<true>(a, d->d, false, as_cuda(stream));
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
    if (!q || !k || !v || !q_out || !heads_ok(d->H)) return SFA_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(q_out)) return SFA_ERR_INVALID_ARG;
    if (!rows_stride_ok(d->q_stride, d->B, d->H, d->L) || !rows_stride_ok(d->q_out_stride, d->B, d->H, d->L) ||
        !rows_stride_ok(d->k_stride, d->B, d->H_kv, d->L) || !rows_stride_ok(d->v_stride, d->B, d->H_kv, d->L))
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
    if (!k_out || !v_out || !aligned16(k_out) || !aligned16(v_out)) return SFA_ERR_INVALID_ARG;
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
    a.rows = (int64_t)d->B * d->H_kv * d->L;
    if ((int64_t)d->B * d->L >= ((int64_t)1 << 31)) return SFA_ERR_INVALID_ARG;
    const int per_cta = 256 / (d->d / 8) * 4;
    const int64_t need = (a.rows + per_cta - 1) / per_cta;
    const int64_t grid = need < (int64_t)1 << 30 ? need : (int64_t)1 << 30;
    if (d->d == 128) cache_read_kernel<128><<<(unsigned)grid, 256, 0, as_cuda(stream)>>>(a);
    else cache_read_kernel<64><<<(unsigned)grid, 256, 0, as_cuda(stream)>>>(a);
    return launch_status();
}
