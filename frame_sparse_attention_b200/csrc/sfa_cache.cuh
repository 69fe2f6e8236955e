// The 8-bit frame cache: where a token lies, and the row format (e4m3 codes in blocks of 32
// elements, one power of two per block).
#pragma once

#include <cstdint>

#include "sfa.h"

namespace sfa {

constexpr int CACHE_BLOCK = SFA_CACHE_BLOCK;
constexpr int E_MIN = -124, E_MAX = 119;  // 2^-9 * 2^-124 is the smallest bf16 number, 448 * 2^119 is finite in bf16

// Device view of a cache (sfa_cache without its host-only checks).
struct CacheView {
    uint8_t *k, *v, *k_scale, *v_scale;
    const int32_t *table;
    int64_t ts0, ts1;  // table strides: batch, key head
    int32_t n_pages, heads, page_len, table_len;
};

inline CacheView cache_view(const sfa_cache *c)
{
    CacheView w;
    w.k = static_cast<uint8_t *>(c->k);
    w.v = static_cast<uint8_t *>(c->v);
    w.k_scale = static_cast<uint8_t *>(c->k_scale);
    w.v_scale = static_cast<uint8_t *>(c->v_scale);
    w.table = c->table;
    w.ts0 = c->table_stride[0];
    w.ts1 = c->table_stride[1];
    w.n_pages = c->n_pages;
    w.heads = c->heads;
    w.page_len = c->page_len;
    w.table_len = c->table_len;
    return w;
}

inline sfa_status check_cache(const sfa_cache *c, int32_t H_kv, int32_t d)
{
    if (!c) return SFA_ERR_INVALID_ARG;
    if (c->d != 64 && c->d != 128) return SFA_ERR_UNSUPPORTED;
    if (c->d != d || c->n_pages < 1 || c->page_len < 1 || c->table_len < 1) return SFA_ERR_INVALID_ARG;
    if (c->heads != 1 && c->heads != H_kv) return SFA_ERR_INVALID_ARG;
    if (!c->k || !c->v || !c->k_scale || !c->v_scale || !c->table) return SFA_ERR_INVALID_ARG;
    const uintptr_t sb = d / CACHE_BLOCK;
    if (reinterpret_cast<uintptr_t>(c->k) % 16 || reinterpret_cast<uintptr_t>(c->v) % 16 ||
        reinterpret_cast<uintptr_t>(c->k_scale) % sb || reinterpret_cast<uintptr_t>(c->v_scale) % sb ||
        reinterpret_cast<uintptr_t>(c->table) % 4)
        return SFA_ERR_INVALID_ARG;
    if (c->table_stride[0] < 0 || c->table_stride[1] < 0) return SFA_ERR_INVALID_ARG;
    // a logical token is an int32 with room for a tile behind it, and a pool row is an int32
    // (2^31 rows of codes are past any GPU's memory)
    if ((int64_t)c->table_len * c->page_len >= ((int64_t)1 << 30)) return SFA_ERR_INVALID_ARG;
    if ((int64_t)c->n_pages * c->heads >= ((int64_t)1 << 31) / c->page_len) return SFA_ERR_INVALID_ARG;
    return SFA_OK;
}

// Strides (batch, head, token) of a [B][heads][L][d] bf16 tensor whose rows are moved 16
// bytes at a time; the stride of a dimension of one entry is not used.
inline bool rows_stride_ok(const int64_t *s, int64_t B, int64_t heads, int64_t L)
{
    const int64_t n[3] = {B, heads, L};
    for (int i = 0; i < 3; ++i)
        if (n[i] > 1 && (s[i] <= 0 || s[i] % 8 || s[i] >= ((int64_t)1 << 38))) return false;
    return true;
}

// An output at its input's address is written as the rows there have been read, which takes the
// same rows at the same places.
inline bool in_place_ok(const void *in, const void *out, const int64_t *si, const int64_t *so, int64_t B, int64_t heads,
                        int64_t L)
{
    const int64_t n[3] = {B, heads, L};
    for (int i = 0; i < 3; ++i)
        if (in == out && n[i] > 1 && si[i] != so[i]) return false;
    return true;
}

__device__ __forceinline__ void report_status(int32_t *status, int32_t code)
{
    if (status) atomicCAS(status, 0, code);
}

// Pool row of logical token j of (b, h), or -1 where it has no valid place.
__device__ __forceinline__ int64_t cache_row(const CacheView &c, int b, int h, int64_t j)
{
    if (j < 0 || j >= (int64_t)c.table_len * c.page_len) return -1;
    const uint32_t slot = (uint32_t)j / (uint32_t)c.page_len;
    const int page = __ldg(c.table + b * c.ts0 + h * c.ts1 + slot);
    if (page < 0 || page >= c.n_pages) return -1;
    return ((int64_t)page * c.heads + (c.heads > 1 ? h : 0)) * c.page_len + ((uint32_t)j - slot * (uint32_t)c.page_len);
}

// The same in two steps, so that the page number can be on its way meanwhile: `open` reads it
// (for a token that is not wanted, the row's first entry), `row` checks it.
struct CachePlace {
    int page, off;
    bool wanted;
    __device__ __forceinline__ void open(const CacheView &c, const int32_t *table_row, int j, bool want)
    {
        const uint32_t slot = want ? (uint32_t)j / (uint32_t)c.page_len : 0u;
        wanted = want;
        off = (int)((uint32_t)j - slot * (uint32_t)c.page_len);
        page = __ldg(table_row + slot);
    }
    // pool row, or -1; a wanted token without a valid page is reported
    __device__ __forceinline__ int row(const CacheView &c, int h, int32_t *status) const
    {
        const bool ok = wanted && page >= 0 && page < c.n_pages;
        if (wanted && !ok) report_status(status, SFA_ERR_BAD_SET);
        return ok ? (page * c.heads + (c.heads > 1 ? h : 0)) * c.page_len + off : -1;
    }
};

// e of a block whose largest magnitude has the bf16 bits `amax` (finite, sign cleared): the
// smallest e with amax <= 448 * 2^e = 1.75 * 2^(e + 8).  For amax = (1 + m / 128) * 2^E that
// is E - 8, one more where m > 96; adding 31 carries into the exponent field exactly then.
// Returned as the bf16 bits of 2^(e + 8), which both the stored byte and 2^-e come from.
__device__ __forceinline__ uint32_t block_exponent_bits(uint32_t amax)
{
    const uint32_t lo = (uint32_t)(E_MIN + 8 + 127) << 7, hi = (uint32_t)(E_MAX + 8 + 127) << 7;
    return min(max((amax + 31u) & 0xff80u, lo), hi);
}

// codes of a, b, c, d from the lowest byte on: nearest even, saturated to 448
__device__ __forceinline__ uint32_t to_e4m3x4(float a, float b, float c, float d)
{
    uint32_t r;
    asm("{\n"
        ".reg .b16 lo, hi;\n"
        "cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n"
        "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n"
        "mov.b32 %0, {lo, hi};\n"
        "}"
        : "=r"(r)
        : "f"(a), "f"(b), "f"(c), "f"(d));
    return r;
}

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("mul.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// 16 or 8 bytes of codes, read once: kept out of L1, where the page tables stay
__device__ __forceinline__ uint4 load_codes16(const uint8_t *p)
{
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}
__device__ __forceinline__ uint2 load_codes8(const uint8_t *p)
{
    uint2 v;
    asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
    return v;
}

// Two codes to bf16, the byte permutation P of (a, b) naming each half's code and, with the bit
// that repeats a byte's sign, the half's upper byte.  A shift by four then brings sign, exponent
// and mantissa to bf16's places and the mask clears the other copies of the sign.  That is the
// code's value times 2^(7 - 127), e4m3 subnormals becoming bf16 subnormals, and the product
// with 2^(120 + e) is exact.
template <uint32_t P>
__device__ __forceinline__ uint32_t spread_codes(uint32_t a, uint32_t b)
{
    uint32_t x;
    asm("prmt.b32 %0, %1, %2, %3;" : "=r"(x) : "r"(a), "r"(b), "n"(P));
    return (x << 4) & 0x87f087f0u;
}
// codes 0, 1 and 2, 3 of a word; code J of each of two words
constexpr uint32_t CODES_01 = 0x9180u, CODES_23 = 0xb3a2u;
template <int J>
constexpr uint32_t CODES_OF_TWO = 0xc480u + 0x1111u * J;

// bf16 bits of 2^(120 + e); 2^127 for e > 7, the rest being scale_rest's
__device__ __forceinline__ uint32_t scale_bits(uint32_t scale_byte)
{
    return min(scale_byte + 120u, 254u) << 7;
}
// bf16 bits of 2^max(e - 7, 0)
__device__ __forceinline__ uint32_t scale_rest_bits(uint32_t scale_byte)
{
    return (scale_byte > 134u ? scale_byte - 7u : 127u) << 7;
}
// The same, twice (both halves of a word) or of two scale bytes, for bytes below 135
__device__ __forceinline__ uint32_t scale_pair(uint32_t byte) { return byte * 0x00800080u + 0x3c003c00u; }
__device__ __forceinline__ uint32_t scale_pair(uint32_t lo, uint32_t hi)
{
    return hi * 0x00800000u + (lo * 0x80u + 0x3c003c00u);
}
// Scale bytes without their top bit (e <= 0, blocks of at most 448) need no second product, and
// neither do those up to 134; the kernels look at the top bits.
constexpr uint32_t SCALE_TOP_BITS = 0x80808080u;

}  // namespace sfa
