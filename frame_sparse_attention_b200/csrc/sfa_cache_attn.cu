// Attention of a chunk of new tokens over the 8-bit frame cache.
//
//   O_i = sum_j softmax_j(scale q_i . k_j) v_j over the logical tokens j of (b, key head),
//   k_j = 2^e c_j per block of 32 elements (exactly a bf16 number), the same for v_j,
// with the log-sum-exp of every row ("ISPA", §2.1), causal or over all tokens, the query
// heads of a key head sharing its rows.
//
// Few query rows (rows_attn_kernel): every code is read once from HBM, converted and used for
// at most 16 rows, so the floor is the cache's bytes.  The codes go from global memory to
// registers in the lane layout of the m16n8k16 matrix instruction (its k index may be any
// order of the elements as long as Q has the same), are turned into bf16 there (2.5
// instructions per element) and never touch shared memory.  A warp owns 16 keys at a time;
// the loads of the next keys are issued as soon as the registers are free; the key range is
// cut over warps and CTAs so that all SMs stream, and the partial results are joined by their
// log-sum-exp.
#include <algorithm>
#include <cmath>
#include <cstdint>

#include <cuda_runtime.h>

#include "sfa.h"
#include "sfa_attn_core.cuh"
#include "sfa_cache.cuh"
#include "sfa_internal.h"
#include "sfa_ptx.cuh"

namespace sfa {
namespace {

struct ChunkArgs {
    CacheView cache;
    int32_t B, H, Hk, G, Lq;  // G = H / Hk query heads per key head
    const uint16_t *q;
    uint16_t *o;
    int64_t qs[3], os[3];
    const int32_t *kv_lens, *q_lens;
    int64_t ls0, ls1;
    int32_t causal;
    float scale_log2;  // softmax scale * log2(e)
    float *lse;
    int32_t *status;
    int32_t n_row_tiles, n_split;
    int32_t range_len;  // key steps of a range, see n_ranges
    float *part_o;    // [n_split][B * H * Lq][d], normalised, when n_split > 1
    float *part_lse;  // [n_split][B * H * Lq], log2 units
    uint64_t timeout_ns;
    uint32_t debug_flags;
};

// What a CTA works on: rows [row0, row0 + tile) of (b, hk), row r being token r / G of query
// head hk * G + r % G, and its share of the keys those rows see.
struct Unit {
    int b, hk, row0, split;
    int m, n;     // query tokens and cache tokens
    int n_rows;   // m * G
    bool bad;     // n outside the table
};

__device__ __forceinline__ Unit open_unit(const ChunkArgs &a, int tile_rows)
{
    Unit u;
    int x = blockIdx.x;
    u.split = x % a.n_split;
    x /= a.n_split;
    // causal: the last row tiles see the most keys and start first
    const int rt = x % a.n_row_tiles;
    u.row0 = (a.causal ? a.n_row_tiles - 1 - rt : rt) * tile_rows;
    x /= a.n_row_tiles;
    u.hk = x % a.Hk;
    u.b = x / a.Hk;
    u.m = a.q_lens ? min(max(__ldg(a.q_lens + u.b), 0), a.Lq) : a.Lq;
    u.n = __ldg(a.kv_lens + u.b * a.ls0 + u.hk * a.ls1);
    u.bad = u.n < 0 || u.n > a.cache.table_len * a.cache.page_len;
    if (u.bad) u.n = 0;
    u.n_rows = u.m * a.G;
    return u;
}

// keys that row r sees: [0, row_limit)
__device__ __forceinline__ int row_limit(const ChunkArgs &a, const Unit &u, int r)
{
    if (r >= u.n_rows) return 0;
    return a.causal ? max(0, min(u.n, u.n - u.m + r / a.G + 1)) : u.n;
}

// Ranges that the key steps of a unit are cut into: as many of range_len steps as it has, so
// that long and short caches give pieces of one length, but no more than the n_split CTAs
// that it was given (caches longer than the caller's bound just get longer ranges).
__device__ __forceinline__ int n_ranges(const ChunkArgs &a, int steps)
{
    return max(1, min(a.n_split, (steps + a.range_len - 1) / a.range_len));
}

// Row `id` of the outputs: (b * H + h) * Lq + i for row r of a unit.
__device__ __forceinline__ int64_t row_id(const ChunkArgs &a, const Unit &u, int r)
{
    return ((int64_t)u.b * a.H + u.hk * a.G + r % a.G) * a.Lq + r / a.G;
}

// A CTA without a range of its own leaves "nothing seen" for its rows.
__device__ __forceinline__ void skip_range(const ChunkArgs &a, const Unit &u, int tile_rows)
{
    const int64_t part_rows = (int64_t)a.B * a.H * a.Lq;
    for (int r = u.row0 + threadIdx.x; r < min(u.row0 + tile_rows, u.n_rows); r += blockDim.x)
        a.part_lse[(int64_t)u.split * part_rows + row_id(a, u, r)] = -INFINITY;
}

// ----------------------------------------------------------------- few query rows
constexpr int FR_WARPS = 4;
constexpr int FR_ROWS = 16;              // the matrix instruction's rows
constexpr int FR_KEYS = 16 * FR_WARPS;   // keys of one step of the CTA

__device__ __forceinline__ void mma_16816(float (&c)[4], const uint4 &a, uint32_t b0, uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
}

// codes j and j + 1 (j = 0 or 2) of a word -> bf16 pair times f
template <int J>
__device__ __forceinline__ uint32_t codes_in_word(uint32_t w, uint32_t f)
{
    return mul_bf16x2(spread_codes(__byte_perm(w, 0, J ? 0x3322 : 0x1100)), f);
}
// code j of words lo and hi -> bf16 pair times f
__device__ __forceinline__ uint32_t codes_of_two(uint32_t lo, uint32_t hi, int j, uint32_t f)
{
    const uint32_t sel = (uint32_t)j * 0x1111u + 0x4400u;
    return mul_bf16x2(spread_codes(__byte_perm(lo, hi, sel)), f);
}

template <int D>
struct ScaleWord;
template <>
struct ScaleWord<128> {
    typedef uint32_t type;
};
template <>
struct ScaleWord<64> {
    typedef uint16_t type;
};

// Grid: (b, key head, row tile, key range), the key range fastest.  Lane (g = lane / 4,
// t = lane % 4) holds, of 16 keys: of K the rows g and g + 8, elements c * 64 + 16 t .. + 15
// (c = 0 .. D/64 - 1); of V the rows 2t, 2t + 1, 2t + 8, 2t + 9, elements g * D/8 .. + D/8 - 1.
// Both reads touch whole 32-byte sectors.  Output column i of n-tile i' is then element
// (its lane's column) * D/8 + i', so a lane ends up with D/4 consecutive elements of two rows.
template <int D>
__global__ void __launch_bounds__(FR_WARPS * 32, 4) rows_attn_kernel(const __grid_constant__ ChunkArgs a)
{
    constexpr int KC = D / 64;          // 16-byte pieces of a K row per lane
    constexpr int VW = D / 32;          // words of a V row per lane
    constexpr int NT = D / 8;           // n-tiles of the output
    typedef typename ScaleWord<D>::type scale_t;
    __shared__ uint4 q_frag[D / 16][32];
    __shared__ float o_sh[FR_WARPS][FR_ROWS][D + 4];
    __shared__ float ml_sh[FR_WARPS][FR_ROWS][2];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, t = lane & 3;
    if (a.n_split > 1) pdl_launch_dependents();  // the joining kernel's CTAs may take their places
    const Unit u = open_unit(a, FR_ROWS);
    if (u.bad && tid == 0) report_status(a.status, SFA_ERR_BAD_SET);
    if (u.row0 >= u.n_rows) return;  // rows behind this sequence's last
    // the tile's last row sees the most keys
    const int seen = row_limit(a, u, min(u.row0 + FR_ROWS, u.n_rows) - 1);
    const int steps = (seen + FR_KEYS - 1) / FR_KEYS;
    const int ranges = n_ranges(a, steps);
    if (u.split >= ranges) return skip_range(a, u, FR_ROWS);

    // Q in the A-operand layout of every k-step: rows g and g + 8, elements
    // c * 64 + 16 t + 4 w + {0, 1} and {2, 3} of k-step 4 c + w
    for (int x = tid; x < (D / 16) * 32; x += FR_WARPS * 32) {
        const int ks = x >> 5, l = x & 31, e = (ks >> 2) * 64 + 16 * (l & 3) + 4 * (ks & 3);
        uint2 v[2];
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const int r = u.row0 + (l >> 2) + 8 * s;
            v[s] = make_uint2(0u, 0u);
            if (r < u.n_rows)
                v[s] = *reinterpret_cast<const uint2 *>(a.q + u.b * a.qs[0] + (u.hk * a.G + r % a.G) * a.qs[1] +
                                                        (r / a.G) * a.qs[2] + e);
        }
        q_frag[ks][l] = make_uint4(v[0].x, v[1].x, v[0].y, v[1].y);
    }
    __syncthreads();

    const int lim0 = row_limit(a, u, u.row0 + g), lim1 = row_limit(a, u, u.row0 + g + 8);
    const int s0 = (int)((int64_t)steps * u.split / ranges), s1 = (int)((int64_t)steps * (u.split + 1) / ranges);

    float o[NT][4];
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) o[i][j] = 0.f;
    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;  // of rows g and g + 8

    // pool row of key (16 of them: lanes 0-15, repeated in 16-31) of step s, -1 past the end
    auto rows_of = [&](int s) -> int {
        const int j = s * FR_KEYS + warp * 16 + (lane & 15);
        if (s >= s1 || j >= seen) return -1;
        const int64_t r = cache_row(a.cache, u.b, u.hk, j);
        if (r < 0) report_status(a.status, SFA_ERR_BAD_SET);
        return (int)r;
    };
    uint4 kr[2][KC];
    uint32_t vr[4][VW], ksc[2], vsc[4];
    const scale_t *k_scale = reinterpret_cast<const scale_t *>(a.cache.k_scale);
    const scale_t *v_scale = reinterpret_cast<const scale_t *>(a.cache.v_scale);
    auto load_k = [&](int rows) {
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const int r = __shfl_sync(0xffffffffu, rows, g + 8 * s);
            ksc[s] = r >= 0 ? (uint32_t)__ldg(k_scale + r) : 0u;
#pragma unroll
            for (int c = 0; c < KC; ++c)
                kr[s][c] = r >= 0 ? __ldg(reinterpret_cast<const uint4 *>(a.cache.k + (int64_t)r * D + c * 64 + t * 16))
                                  : make_uint4(0u, 0u, 0u, 0u);
        }
    };
    auto load_v = [&](int rows) {
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            const int r = __shfl_sync(0xffffffffu, rows, 2 * t + (s & 1) + (s >> 1) * 8);
            vsc[s] = r >= 0 ? (uint32_t)__ldg(v_scale + r) : 0u;
            const uint8_t *p = a.cache.v + (int64_t)r * D + g * NT;
            if (D == 128) {
                const uint4 x = r >= 0 ? __ldg(reinterpret_cast<const uint4 *>(p)) : make_uint4(0u, 0u, 0u, 0u);
                vr[s][0] = x.x, vr[s][1] = x.y, vr[s][VW - 2] = x.z, vr[s][VW - 1] = x.w;
            } else {
                const uint2 x = r >= 0 ? __ldg(reinterpret_cast<const uint2 *>(p)) : make_uint2(0u, 0u);
                vr[s][0] = x.x, vr[s][1] = x.y;
            }
        }
    };

    int rows = rows_of(s0);
    load_k(rows);
    load_v(rows);
    for (int st = s0; st < s1; ++st) {
        const int rows_next = rows_of(st + 1);
        // scales of the block each register lies in; 2^e beyond bf16's range in one step (e > 7,
        // values of 57344 and more) takes a second product
        bool two = false;
#pragma unroll
        for (int s = 0; s < 2; ++s) two |= __vcmpgtu4(ksc[s], 0x01010101u * SCALE_ONE_STEP) != 0u;
#pragma unroll
        for (int s = 0; s < 4; ++s) two |= __vcmpgtu4(vsc[s], 0x01010101u * SCALE_ONE_STEP) != 0u;
        two = __any_sync(0xffffffffu, two);

        // ---- S = Q K^T, keys 8 s + 2 t + {0, 1} of rows g, g + 8
        float sc[2][4];
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int j = 0; j < 4; ++j) sc[s][j] = 0.f;
#pragma unroll
        for (int c = 0; c < KC; ++c) {
            uint32_t f[2], r2[2];
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const uint32_t byte = (ksc[s] >> (8 * (2 * c + (t >> 1)))) & 0xffu;
                f[s] = scale_bits(byte) * 0x10001u;
                r2[s] = scale_rest_bits(byte) * 0x10001u;
            }
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                const uint4 qf = q_frag[4 * c + w][lane];
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    const uint32_t kw = w == 0 ? kr[s][c].x : w == 1 ? kr[s][c].y : w == 2 ? kr[s][c].z : kr[s][c].w;
                    uint32_t b0 = codes_in_word<0>(kw, f[s]), b1 = codes_in_word<2>(kw, f[s]);
                    if (two) {
                        b0 = mul_bf16x2(b0, r2[s]);
                        b1 = mul_bf16x2(b1, r2[s]);
                    }
                    mma_16816(sc[s], qf, b0, b1);
                }
            }
        }
        load_k(rows_next);

        // ---- softmax of this warp's 16 keys (log2 units, scale folded in)
        const int key = st * FR_KEYS + warp * 16 + 2 * t;
        float x0 = -INFINITY, x1 = -INFINITY;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                sc[s][j] = key + 8 * s + j < lim0 ? sc[s][j] * a.scale_log2 : -INFINITY;
                sc[s][2 + j] = key + 8 * s + j < lim1 ? sc[s][2 + j] * a.scale_log2 : -INFINITY;
                x0 = fmaxf(x0, sc[s][j]);
                x1 = fmaxf(x1, sc[s][2 + j]);
            }
        }
        // the running max is kept while no score exceeds it by 2^8; -inf (nothing seen) is
        // always replaced
        if (__any_sync(0xffffffffu, x0 > m0 + 8.f || x1 > m1 + 8.f)) {
#pragma unroll
            for (int d = 1; d < 4; d <<= 1) {
                x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, d));
                x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, d));
            }
            const float n0 = fmaxf(m0, x0), n1 = fmaxf(m1, x1);
            const float c0 = m0 == -INFINITY ? 0.f : ex2_approx(m0 - n0), c1 = m1 == -INFINITY ? 0.f : ex2_approx(m1 - n1);
            m0 = n0;
            m1 = n1;
            l0 *= c0;
            l1 *= c1;
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                o[i][0] *= c0;
                o[i][1] *= c0;
                o[i][2] *= c1;
                o[i][3] *= c1;
            }
        }
        const float z0 = m0 == -INFINITY ? 0.f : m0, z1 = m1 == -INFINITY ? 0.f : m1;
        uint4 p;
        {
            float e[8];
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                e[4 * s] = ex2_approx(sc[s][0] - z0);
                e[4 * s + 1] = ex2_approx(sc[s][1] - z0);
                e[4 * s + 2] = ex2_approx(sc[s][2] - z1);
                e[4 * s + 3] = ex2_approx(sc[s][3] - z1);
                l0 += e[4 * s] + e[4 * s + 1];
                l1 += e[4 * s + 2] + e[4 * s + 3];
            }
            p.x = pack_bf16x2(e[0], e[1]);
            p.y = pack_bf16x2(e[2], e[3]);
            p.z = pack_bf16x2(e[4], e[5]);
            p.w = pack_bf16x2(e[6], e[7]);
        }

        // ---- O += P V
        const int blk = (g * NT) / CACHE_BLOCK * 8;
        uint32_t f01 = scale_bits((vsc[0] >> blk) & 0xffu) | (scale_bits((vsc[1] >> blk) & 0xffu) << 16);
        uint32_t f23 = scale_bits((vsc[2] >> blk) & 0xffu) | (scale_bits((vsc[3] >> blk) & 0xffu) << 16);
        uint32_t r01 = scale_rest_bits((vsc[0] >> blk) & 0xffu) | (scale_rest_bits((vsc[1] >> blk) & 0xffu) << 16);
        uint32_t r23 = scale_rest_bits((vsc[2] >> blk) & 0xffu) | (scale_rest_bits((vsc[3] >> blk) & 0xffu) << 16);
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            uint32_t b0 = codes_of_two(vr[0][i / 4], vr[1][i / 4], i % 4, f01);
            uint32_t b1 = codes_of_two(vr[2][i / 4], vr[3][i / 4], i % 4, f23);
            if (two) {
                b0 = mul_bf16x2(b0, r01);
                b1 = mul_bf16x2(b1, r23);
            }
            mma_16816(o[i], p, b0, b1);
        }
        load_v(rows_next);
    }

    // ---- join the warps: every warp's O against the common max, then the sum of four
#pragma unroll
    for (int d = 1; d < 4; d <<= 1) {
        l0 += __shfl_xor_sync(0xffffffffu, l0, d);
        l1 += __shfl_xor_sync(0xffffffffu, l1, d);
    }
    if (t == 0) {
        ml_sh[warp][g][0] = m0;
        ml_sh[warp][g][1] = l0;
        ml_sh[warp][g + 8][0] = m1;
        ml_sh[warp][g + 8][1] = l1;
    }
#pragma unroll
    for (int i = 0; i < NT; ++i) {
        // columns 2t and 2t + 1 of n-tile i are elements 2t * NT + i and (2t + 1) * NT + i
        o_sh[warp][g][2 * t * NT + i] = o[i][0];
        o_sh[warp][g][(2 * t + 1) * NT + i] = o[i][1];
        o_sh[warp][g + 8][2 * t * NT + i] = o[i][2];
        o_sh[warp][g + 8][(2 * t + 1) * NT + i] = o[i][3];
    }
    __syncthreads();
    const int64_t part_rows = (int64_t)a.B * a.H * a.Lq;
    for (int x = tid; x < FR_ROWS * (D / 8); x += FR_WARPS * 32) {
        const int r = x / (D / 8), e0 = (x % (D / 8)) * 8, row = u.row0 + r;
        if (row >= u.n_rows) continue;
        float M = -INFINITY, l = 0.f, acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int w = 0; w < FR_WARPS; ++w) M = fmaxf(M, ml_sh[w][r][0]);
#pragma unroll
        for (int w = 0; w < FR_WARPS; ++w) {
            const float mw = ml_sh[w][r][0];
            const float c = mw == -INFINITY ? 0.f : ex2_approx(mw - M);
            l += c * ml_sh[w][r][1];
#pragma unroll
            for (int j = 0; j < 8; ++j) acc[j] = fmaf(c, o_sh[w][r][e0 + j], acc[j]);
        }
        const float inv = l > 0.f ? 1.f / l : 0.f;
        const float lse2 = l > 0.f ? M + log2f(l) : -INFINITY;
        const int h = u.hk * a.G + row % a.G, i = row / a.G;
        const int64_t id = row_id(a, u, row);
        if (a.n_split == 1) {
            uint4 v;
            v.x = pack_bf16x2(acc[0] * inv, acc[1] * inv);
            v.y = pack_bf16x2(acc[2] * inv, acc[3] * inv);
            v.z = pack_bf16x2(acc[4] * inv, acc[5] * inv);
            v.w = pack_bf16x2(acc[6] * inv, acc[7] * inv);
            *reinterpret_cast<uint4 *>(a.o + u.b * a.os[0] + h * a.os[1] + i * a.os[2] + e0) = v;
            if (e0 == 0) a.lse[id] = lse2 * 0.69314718055994530942f;
        } else {
            float4 *dst = reinterpret_cast<float4 *>(a.part_o + ((int64_t)u.split * part_rows + id) * D + e0);
            dst[0] = make_float4(acc[0] * inv, acc[1] * inv, acc[2] * inv, acc[3] * inv);
            dst[1] = make_float4(acc[4] * inv, acc[5] * inv, acc[6] * inv, acc[7] * inv);
            if (e0 == 0) a.part_lse[(int64_t)u.split * part_rows + id] = lse2;
        }
    }
}

// ----------------------------------------------------------------- many query rows
// Units of two 128-row query tiles against 128-key tiles, on the tensor cores through tensor
// memory, in the schedule of the frame-list forward kernel (S one tile ahead of the softmax,
// P V behind it; a unit with one query tile runs S two key tiles ahead).  What differs is how
// the operands arrive: four warps load the codes of a K and a V tile into registers, a tile
// ahead, look up their pages, and store them as bf16 in the 128-byte-swizzled layout that
// the matrix instruction reads, zeros behind the last key; the softmax warps bring their own
// query rows, since a unit's rows may be those of several heads.
constexpr int CT_SOFTMAX_WARPS = 8;       // warps 0-3: query tile A, 4-7: B
constexpr int CT_CONV_WARP = 8;           // 8-11: codes to bf16
constexpr int CT_CONV_WARPS = 4;
constexpr int CT_MMA_WARP = 12;
constexpr int CT_THREADS = 32 * (CT_MMA_WARP + 1);
constexpr int CT_ROWS = 2 * BM;

// byte offset of the 16-byte piece `ch` (8 elements) of row r in a swizzled tile
template <int D>
__device__ __forceinline__ uint32_t swz(int r, int ch)
{
    return (uint32_t)((ch >> 3) * Cfg<D>::BOX_BYTES + r * 128 + (((ch & 7) ^ (r & 7)) << 4));
}

// The K and V tiles of the unit, codes to bf16.  Warp w takes rows 32 w .. 32 w + 31 of every
// tile: lane l looks up row l's place, D/16 lanes then share a row, 16 codes each.
template <int D>
__device__ void convert_role(const ChunkArgs &a, const Unit &u, uint32_t sbase, int key0, int key_end, int n_tiles,
                             const Ctl &ctl)
{
    using C = Cfg<D>;
    constexpr int LR = D / 16;        // lanes per row
    constexpr int RPI = 32 / LR;      // rows per load of the warp
    constexpr int NI = 32 / RPI;      // loads per tile
    typedef typename ScaleWord<D>::type scale_t;
    const Bars<D> bar{sbase + C::SMEM_BAR};
    const int lane = threadIdx.x & 31, w = (threadIdx.x >> 5) - CT_CONV_WARP;
    const int sub = lane / LR, c = lane % LR;

    auto rows_of = [&](int j) -> int {  // pool row of key 32 w + lane of tile j
        const int key = key0 + j * BN + w * 32 + lane;
        if (j >= n_tiles || key >= key_end) return -1;
        const int64_t r = cache_row(a.cache, u.b, u.hk, key);
        if (r < 0) report_status(a.status, SFA_ERR_BAD_SET);
        return (int)r;
    };
    auto load = [&](const uint8_t *codes, const uint8_t *scales, int rows, uint4 (&x)[NI], uint32_t &sw) {
        sw = rows >= 0 ? (uint32_t)__ldg(reinterpret_cast<const scale_t *>(scales) + rows) : 0u;
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            const int r = __shfl_sync(0xffffffffu, rows, i * RPI + sub);
            x[i] = r >= 0 ? __ldg(reinterpret_cast<const uint4 *>(codes + (int64_t)r * D + c * 16))
                          : make_uint4(0u, 0u, 0u, 0u);
        }
    };
    auto store = [&](uint32_t tile, const uint4 (&x)[NI], uint32_t sw) {
        const bool two = __any_sync(0xffffffffu, __vcmpgtu4(sw, 0x01010101u * SCALE_ONE_STEP) != 0u);
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            const int r = i * RPI + sub;  // row inside this warp's 32
            const uint32_t byte = (__shfl_sync(0xffffffffu, sw, r) >> (8 * (c / 2))) & 0xffu;
            const uint32_t f = scale_bits(byte) * 0x10001u;
            const uint32_t in[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
            uint32_t y[8];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                y[2 * k] = codes_in_word<0>(in[k], f);
                y[2 * k + 1] = codes_in_word<2>(in[k], f);
            }
            if (two) {
                const uint32_t g = scale_rest_bits(byte) * 0x10001u;
#pragma unroll
                for (int k = 0; k < 8; ++k) y[k] = mul_bf16x2(y[k], g);
            }
            const uint32_t lo[4] = {y[0], y[1], y[2], y[3]}, hi[4] = {y[4], y[5], y[6], y[7]};
            // the upper half of a row's lanes store their two pieces in the other order, so that
            // the eight lanes of one access fall on all eight 16-byte bank groups
            const bool swap = D == 128 && c >= 4;
            const int row = w * 32 + r;
            st_shared_v4(tile + swz<D>(row, 2 * c + (swap ? 1 : 0)), swap ? hi : lo);
            st_shared_v4(tile + swz<D>(row, 2 * c + (swap ? 0 : 1)), swap ? lo : hi);
        }
        fence_proxy_async_smem();
        __syncwarp();
    };

    uint4 kx[NI], vx[NI];
    uint32_t ks, vs;
    int rows_k = rows_of(0), rows_v;
    load(a.cache.k, a.cache.k_scale, rows_k, kx, ks);
    load(a.cache.v, a.cache.v_scale, rows_k, vx, vs);
    // K(0) | K(j + 1) V(j) | ...
    for (int j = -1; j < n_tiles; ++j) {
        if (j + 1 < n_tiles) {
            const int s = (j + 1) % C::NSK, use = (j + 1) / C::NSK;
            if (use > 0 && !__all_sync(0xffffffffu, wait_bar(bar.k_free(s), (use - 1) & 1, ctl))) return;
            store(sbase + C::SMEM_K + s * C::TILE_BYTES, kx, ks);
            if (lane == 0) mbar_arrive(bar.k_full(s));
            rows_v = rows_k;  // of tile j + 1, for its V
            rows_k = rows_of(j + 2);
            load(a.cache.k, a.cache.k_scale, rows_k, kx, ks);
        } else {
            rows_v = -1;
        }
        if (j >= 0) {
            const int s = j % C::NSV, use = j / C::NSV;
            if (use > 0 && !__all_sync(0xffffffffu, wait_bar(bar.v_free(s), (use - 1) & 1, ctl))) return;
            store(sbase + C::SMEM_V + s * C::TILE_BYTES, vx, vs);
            if (lane == 0) mbar_arrive(bar.v_full(s));
            load(a.cache.v, a.cache.v_scale, rows_v, vx, vs);
        }
    }
}

template <int D>
__device__ void chunk_mma_pair(uint32_t sbase, uint32_t tmem, int n_tiles, const Ctl &ctl)
{
    using C = Cfg<D>;
    constexpr uint32_t idesc_s = idesc_bf16_f32(BM, BN, false);
    const Bars<D> bar{sbase + C::SMEM_BAR};
    const uint64_t dq = sdesc_sw128(sbase + C::SMEM_Q, 16, 1024), dk = sdesc_sw128(sbase + C::SMEM_K, 16, 1024);
    const uint64_t dv = sdesc_sw128(sbase + C::SMEM_V, C::BOX_BYTES, 1024), dp = sdesc_sw128(sbase + C::SMEM_P, 16, 1024);
    bool issued = false;
    if (!__all_sync(0xffffffffu, wait_bar(bar.q_full(), 0, ctl))) goto done;
    if (!__all_sync(0xffffffffu, wait_bar(bar.k_full(0), 0, ctl))) goto done;
    tc_fence_after();
    for (int x = 0; x < 2; ++x) {
        issue_s<D>(tmem + tcol_s(x), desc_add(dq, x * C::TILE_BYTES), dk, idesc_s);
        commit_one(bar.s_full(x));
    }
    commit_one(bar.k_free(0));
    issued = true;
    for (int j = 0; j < n_tiles; ++j) {
        const int sv = j % C::NSV, sk = (j + 1) % C::NSK;
        for (int x = 0; x < 2; ++x) {
            if (!__all_sync(0xffffffffu, wait_bar(bar.p_full(x), j & 1, ctl))) goto done;
            if (j + 1 < n_tiles) {
                if (x == 0 && !__all_sync(0xffffffffu, wait_bar(bar.k_full(sk), ((j + 1) / C::NSK) & 1, ctl))) goto done;
                tc_fence_after();
                issue_s<D>(tmem + tcol_s(x), desc_add(dq, x * C::TILE_BYTES), desc_add(dk, sk * C::TILE_BYTES), idesc_s);
                commit_one(bar.s_full(x));
                if (x == 1) commit_one(bar.k_free(sk));
            }
            if (x == 0 && !__all_sync(0xffffffffu, wait_bar(bar.v_full(sv), (j / C::NSV) & 1, ctl))) goto done;
            tc_fence_after();
            issue_pv<D>(tmem + tcol_o(x), desc_add(dp, x * C::P_BYTES), desc_add(dv, sv * C::TILE_BYTES), BN, j > 0);
            commit_one(bar.pv_x(x));
            if (x == 1) {
                commit_one(bar.v_free(sv));
                if (j == n_tiles - 1) commit_one(bar.o_final());
            }
        }
    }
done:
    if (__any_sync(0xffffffffu, *ctl.abort != 0) && issued) {  // the tensor cores finish before TMEM is released
        commit_one(bar.drain());
        wait_drain(bar.drain(), 0);
    }
    __syncwarp();
}

template <int D>
__device__ void chunk_mma_single(uint32_t sbase, uint32_t tmem, int n_tiles, const Ctl &ctl)
{
    using C = Cfg<D>;
    constexpr uint32_t idesc_s = idesc_bf16_f32(BM, BN, false);
    const Bars<D> bar{sbase + C::SMEM_BAR};
    const uint64_t dq = sdesc_sw128(sbase + C::SMEM_Q, 16, 1024), dk = sdesc_sw128(sbase + C::SMEM_K, 16, 1024);
    const uint64_t dv = sdesc_sw128(sbase + C::SMEM_V, C::BOX_BYTES, 1024), dp = sdesc_sw128(sbase + C::SMEM_P, 16, 1024);
    bool issued = false;
    if (!__all_sync(0xffffffffu, wait_bar(bar.q_full(), 0, ctl))) goto done;
    for (int j = 0; j < 2 && j < n_tiles; ++j) {
        const int sk = j % C::NSK;
        if (!__all_sync(0xffffffffu, wait_bar(bar.k_full(sk), (j / C::NSK) & 1, ctl))) goto done;
        tc_fence_after();
        issue_s<D>(tmem + tcol_s(j), dq, desc_add(dk, sk * C::TILE_BYTES), idesc_s);
        commit_one(bar.s_full(j));
        commit_one(bar.k_free(sk));
        issued = true;
    }
    for (int j = 0; j < n_tiles; ++j) {
        const int bj = j & 1, sv = j % C::NSV;
        if (!__all_sync(0xffffffffu, wait_bar(bar.p_full(bj), (j >> 1) & 1, ctl))) goto done;
        if (!__all_sync(0xffffffffu, wait_bar(bar.v_full(sv), (j / C::NSV) & 1, ctl))) goto done;
        tc_fence_after();
        issue_pv<D>(tmem + tcol_o(0), desc_add(dp, bj * C::P_BYTES), desc_add(dv, sv * C::TILE_BYTES), BN, j > 0);
        commit_one(bar.pv_done());
        commit_one(bar.v_free(sv));
        if (j == n_tiles - 1) commit_one(bar.o_final());
        if (j + 2 < n_tiles) {
            const int sk = (j + 2) % C::NSK;
            if (!__all_sync(0xffffffffu, wait_bar(bar.k_full(sk), ((j + 2) / C::NSK) & 1, ctl))) goto done;
            tc_fence_after();
            issue_s<D>(tmem + tcol_s(bj), dq, desc_add(dk, sk * C::TILE_BYTES), idesc_s);
            commit_one(bar.s_full(bj));
            commit_one(bar.k_free(sk));
        }
    }
done:
    if (__any_sync(0xffffffffu, *ctl.abort != 0) && issued) {
        commit_one(bar.drain());
        wait_drain(bar.drain(), 0);
    }
    __syncwarp();
}

template <bool MASK>
__device__ __forceinline__ void hide_columns(int c, int nv, uint32_t (&r)[32])
{
    if (MASK && c * 32 + 32 > nv) {
#pragma unroll
        for (int i = 0; i < 32; ++i)
            if (c * 32 + i >= nv) r[i] = __float_as_uint(-INFINITY);
    }
}

// One key tile of the online softmax, as softmax_tile of the frame-list kernel, for rows that
// see columns [0, nv) of the tile each (MASK; all of them otherwise).  m_used stays -inf, and
// the row's probabilities 0, until the row has seen a key.
template <int D, bool MASK>
__device__ __forceinline__ bool chunk_softmax_tile(uint32_t t_s, uint32_t p_row, int row, uint32_t t_o, int nv, float sl2,
                                                   float &m_used, float &l, int j, uint32_t pv_done, uint32_t pv_first,
                                                   const Ctl &ctl)
{
    if (j > 0) {  // streaming pass against the current max
        Acc8 acc;
        const float neg_m = MASK && m_used == -INFINITY ? 0.f : -m_used;
        uint32_t ra[32], rb[32];
        tmem_ld32(t_s, ra);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            uint32_t(&cur)[32] = (c & 1) ? rb : ra;
            uint32_t(&nxt)[32] = (c & 1) ? ra : rb;
            tmem_wait_ld_regs(cur);
            if (c + 1 < 4) tmem_ld32(t_s + (c + 1) * 32, nxt);
            hide_columns<MASK>(c, nv, cur);
            if (c == 0 && pv_first) {
                uint32_t pk[16];
                exp_chunk(cur, sl2, neg_m, pk, acc);
                if (!__all_sync(0xffffffffu, wait_bar(pv_first, (j - 1) & 1, ctl))) return false;
                tc_fence_after();
                store_chunk(pk, p_row, row, 0);
            } else {
                exp_store_chunk(cur, sl2, neg_m, p_row, row, c, acc);
            }
        }
        const float lt = sum8(acc);
        if (!__any_sync(0xffffffffu, lt > RESCALE_LIMIT || m_used == -INFINITY)) {
            l += lt;
            return true;
        }
    }
    float mx = -INFINITY;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        uint32_t r[32];
        tmem_ld32(t_s + c * 32, r);
        tmem_wait_ld_regs(r);
        hide_columns<MASK>(c, nv, r);
        mx = fmaxf(mx, max32(r));
    }
    const float m_cand = mx * sl2;
    const bool resc = m_cand > m_used;
    const float m_new = resc ? m_cand : m_used;
    const float neg_m = m_new == -INFINITY ? 0.f : -m_new;
    const float alpha = m_used == -INFINITY ? 0.f : ex2_approx(m_used - m_new);
    Acc8 acc;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        uint32_t r[32];
        tmem_ld32(t_s + c * 32, r);
        tmem_wait_ld_regs(r);
        hide_columns<MASK>(c, nv, r);
        exp_store_chunk(r, sl2, neg_m, p_row, row, c, acc);
    }
    if (j > 0 && __any_sync(0xffffffffu, resc)) {
        if (pv_done) {
            if (!__all_sync(0xffffffffu, wait_bar(pv_done, (j - 1) & 1, ctl))) return false;
            tc_fence_after();
        }
        const float by = resc ? alpha : 1.f;
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
            uint32_t o[32];
            tmem_ld32(t_o + c * 32, o);
            tmem_wait_ld_regs(o);
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * by);
            tmem_st32(t_o + c * 32, o);
        }
    }
    l = l * (resc ? alpha : 1.f) + sum8(acc);
    m_used = m_new;
    return true;
}

// Queries, softmax and epilogue of query tile x, one thread per row.
template <int D>
__device__ void chunk_softmax_role(const ChunkArgs &a, const Unit &u, uint8_t *smem, uint32_t sbase, uint32_t tmem, int x,
                                   int key0, int n_tiles, bool one_tile, const Ctl &ctl)
{
    using C = Cfg<D>;
    constexpr int LR = D / 8;     // lanes per 16-byte-pieced row
    constexpr int RPI = 32 / LR;  // rows per access of a warp
    const Bars<D> bar{sbase + C::SMEM_BAR};
    volatile int32_t *epi_ok = reinterpret_cast<volatile int32_t *>(smem + C::SMEM_BAR + 160) + 4 * x;
    const int row = threadIdx.x & 127, lane = threadIdx.x & 31, warp = (threadIdx.x >> 5) & 3;
    const int tile_row0 = u.row0 + x * BM;
    const uint32_t s_tile = sbase + C::SMEM_Q + x * C::TILE_BYTES;
    // this warp's 32 query rows, whole rows at a time
#pragma unroll 8
    for (int i = 0; i < 32; i += RPI) {
        const int rr = warp * 32 + i + lane / LR, ch = lane % LR, r = tile_row0 + rr;
        uint4 v = make_uint4(0u, 0u, 0u, 0u);
        if (r < u.n_rows)
            v = *reinterpret_cast<const uint4 *>(a.q + u.b * a.qs[0] + (u.hk * a.G + r % a.G) * a.qs[1] +
                                                 (r / a.G) * a.qs[2] + ch * 8);
        const uint32_t y[4] = {v.x, v.y, v.z, v.w};
        st_shared_v4(s_tile + swz<D>(rr, ch), y);
    }
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(bar.q_full());

    const uint32_t lane_base = tmem + ((uint32_t)(warp * 32) << 16);
    const uint32_t t_o = lane_base + tcol_o(x);
    const int r = tile_row0 + row;
    // keys this row sees, from the range's first on; rows that are not there see all (of zeros)
    const int lim = r < u.n_rows ? row_limit(a, u, r) - key0 : 0x7fffffff;
    // rows grow in what they see, so a tile that the warp's first row sees whole needs no mask
    const int lim_warp = __reduce_min_sync(0xffffffffu, lim);
    float m_used = -INFINITY, l = 0.f;
    bool alive = true;
    for (int j = 0; j < n_tiles; ++j) {
        const int xb = one_tile ? (j & 1) : x;
        const uint32_t par = one_tile ? (uint32_t)(j >> 1) & 1 : (uint32_t)j & 1;
        const uint32_t t_s = lane_base + tcol_s(xb);
        const uint32_t p_row = sbase + C::SMEM_P + xb * C::P_BYTES + row * 128;
        if (!__all_sync(0xffffffffu, wait_bar(bar.s_full(xb), par, ctl))) {
            alive = false;
            break;
        }
        tc_fence_after();
        const uint32_t pvw = one_tile ? bar.pv_done() : 0u;
        const uint32_t pvf = (!one_tile && j > 0) ? bar.pv_x(x) : 0u;
        const bool whole = lim_warp >= (j + 1) * BN;
        const bool ok = whole ? chunk_softmax_tile<D, false>(t_s, p_row, row, t_o, BN, a.scale_log2, m_used, l, j, pvw, pvf, ctl)
                              : chunk_softmax_tile<D, true>(t_s, p_row, row, t_o, lim - j * BN, a.scale_log2, m_used, l, j,
                                                            pvw, pvf, ctl);
        if (!ok) {
            alive = false;
            break;
        }
        tmem_wait_st();
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0 && !((a.debug_flags & SFA_DEBUG_STALL_SOFTMAX) && j == 0)) mbar_arrive(bar.p_full(xb));
    }

    bool have = alive;
    if (have && n_tiles > 0) have = __all_sync(0xffffffffu, wait_bar(bar.o_final(), 0, ctl));
    if (lane == 0) epi_ok[warp] = have ? 1 : 0;
    named_bar_sync(1 + x, BM);
    if (!(epi_ok[0] && epi_ok[1] && epi_ok[2] && epi_ok[3])) return;  // uniform over the tile's warps
    const float inv_l = l > 0.f ? 1.f / l : 0.f;
    const float lse2 = l > 0.f ? m_used + log2f(l) : -INFINITY;
    const bool there = r < u.n_rows;
    const int64_t part_rows = (int64_t)a.B * a.H * a.Lq;
    if (n_tiles > 0) tc_fence_after();
#pragma unroll
    for (int c = 0; c < D / 32; ++c) {
        uint32_t o[32];
        if (n_tiles > 0) {
            tmem_ld32(t_o + c * 32, o);
            tmem_wait_ld_regs(o);
        } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = 0u;
        }
        if (a.n_split > 1) {
            if (there) {
                float4 *dst = reinterpret_cast<float4 *>(a.part_o + (u.split * part_rows + row_id(a, u, r)) * D + c * 32);
#pragma unroll
                for (int q = 0; q < 8; ++q)
                    dst[q] = make_float4(__uint_as_float(o[4 * q]) * inv_l, __uint_as_float(o[4 * q + 1]) * inv_l,
                                         __uint_as_float(o[4 * q + 2]) * inv_l, __uint_as_float(o[4 * q + 3]) * inv_l);
            }
        } else {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                uint32_t y[4];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    y[i] = pack_bf16x2(__uint_as_float(o[q * 8 + 2 * i]) * inv_l, __uint_as_float(o[q * 8 + 2 * i + 1]) * inv_l);
                st_shared_v4(s_tile + swz<D>(row, c * 4 + q), y);
            }
        }
    }
    if (there) {
        if (a.n_split > 1) a.part_lse[u.split * part_rows + row_id(a, u, r)] = lse2;
        else a.lse[row_id(a, u, r)] = lse2 * 0.69314718055994530942f;
    }
    if (a.n_split > 1) return;
    __syncwarp();  // a warp stores the 32 rows that its lanes have staged
#pragma unroll 4
    for (int i = 0; i < 32; i += RPI) {
        const int rr = warp * 32 + i + lane / LR, ch = lane % LR, ro = tile_row0 + rr;
        if (ro < u.n_rows)
            *reinterpret_cast<uint4 *>(a.o + u.b * a.os[0] + (u.hk * a.G + ro % a.G) * a.os[1] + (ro / a.G) * a.os[2] +
                                       ch * 8) = *reinterpret_cast<const uint4 *>(smem + (s_tile - sbase) + swz<D>(rr, ch));
    }
}

template <int D>
__global__ void __launch_bounds__(CT_THREADS, 1) tile_attn_kernel(const __grid_constant__ ChunkArgs a)
{
    using C = Cfg<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = smem_u32(smem);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + C::SMEM_BAR + 240);
    volatile int32_t *abort_flag = reinterpret_cast<volatile int32_t *>(smem + C::SMEM_BAR + 244);
    volatile int32_t *skip = reinterpret_cast<volatile int32_t *>(smem + C::SMEM_BAR + 248);
    const int warp = threadIdx.x >> 5;
    if (a.n_split > 1) pdl_launch_dependents();
    const Unit u = open_unit(a, CT_ROWS);
    if (u.bad && threadIdx.x == 0) report_status(a.status, SFA_ERR_BAD_SET);
    if (u.row0 >= u.n_rows) return;
    const int seen = row_limit(a, u, min(u.row0 + CT_ROWS, u.n_rows) - 1);
    const int all = (seen + BN - 1) / BN;
    const int ranges = n_ranges(a, all);
    if (u.split >= ranges) return skip_range(a, u, CT_ROWS);
    const int t0 = (int)((int64_t)all * u.split / ranges);
    int n_tiles = (int)((int64_t)all * (u.split + 1) / ranges) - t0;
    const bool has_b = u.row0 + BM < u.n_rows;

    if (threadIdx.x == 0) {
        const Bars<D> bar{sbase + C::SMEM_BAR};
        for (int i = 0; i < Bars<D>::COUNT; ++i) mbar_init(sbase + C::SMEM_BAR + 8 * i, 1);
        for (int s = 0; s < C::NSK; ++s) mbar_init(bar.k_full(s), CT_CONV_WARPS);
        for (int s = 0; s < C::NSV; ++s) mbar_init(bar.v_full(s), CT_CONV_WARPS);
        mbar_init(bar.q_full(), has_b ? CT_SOFTMAX_WARPS : CT_SOFTMAX_WARPS / 2);
        mbar_init(bar.p_full(0), BM / 32);
        mbar_init(bar.p_full(1), BM / 32);
        *abort_flag = 0;
        // once a CTA has timed out, the ones that start later skip their work
        *skip = (a.status && *reinterpret_cast<volatile int32_t *>(a.status) == SFA_ERR_TIMEOUT) ? 1 : 0;
        fence_mbar_init();
    }
    if (warp == CT_MMA_WARP) {
        tmem_alloc(smem_u32(tmem_slot), TM_COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const Ctl ctl{abort_flag, a.status, a.timeout_ns};
    const bool skipped = *skip != 0;
    if (skipped) n_tiles = 0;

    if (warp == CT_MMA_WARP) {
        if (n_tiles > 0) {
            if (has_b) chunk_mma_pair<D>(sbase, tmem, n_tiles, ctl);
            else chunk_mma_single<D>(sbase, tmem, n_tiles, ctl);
        }
    } else if (warp >= CT_CONV_WARP) {
        if (n_tiles > 0) convert_role<D>(a, u, sbase, t0 * BN, seen, n_tiles, ctl);
    } else if (!skipped && (warp < 4 || has_b)) {
        chunk_softmax_role<D>(a, u, smem, sbase, tmem, warp >> 2, t0 * BN, n_tiles, !has_b, ctl);
    }

    tc_fence_before();
    __syncthreads();
    if (warp == CT_MMA_WARP) {
        tc_fence_after();
        tmem_dealloc(tmem, TM_COLS);
    }
}

// ----------------------------------------------------------------- joining the ranges
// O = sum_s w_s O_s, w_s = 2^(L_s - L), L = log2 sum_s 2^(L_s), over the key ranges of a row.
// D / 8 lanes own a row, eight elements each.
template <int D>
__global__ void __launch_bounds__(128) join_kernel(const __grid_constant__ ChunkArgs a)
{
    pdl_wait();  // the ranges are written by the kernel before
    constexpr int G = D / 8;
    const int64_t rows = (int64_t)a.B * a.H * a.Lq;
    const int64_t id = ((int64_t)blockIdx.x * 128 + threadIdx.x) / G;
    if (id >= rows) return;
    const int e0 = (threadIdx.x % G) * 8;
    const int64_t bh = id / a.Lq;
    const int i = (int)(id - bh * a.Lq), b = (int)(bh / a.H), h = (int)(bh - (int64_t)b * a.H);
    if (a.q_lens && i >= __ldg(a.q_lens + b)) return;
    float M = -INFINITY;
    for (int s = 0; s < a.n_split; ++s) M = fmaxf(M, a.part_lse[s * rows + id]);
    float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f}, total = 0.f;
    if (M != -INFINITY) {
        for (int s = 0; s < a.n_split; ++s) {
            const float ls = a.part_lse[s * rows + id];
            if (ls == -INFINITY) continue;  // a range that was not there, or that the row does not see
            const float w = ex2_approx(ls - M);
            const float4 *src = reinterpret_cast<const float4 *>(a.part_o + (s * rows + id) * D + e0);
            const float4 x = src[0], y = src[1];
            total += w;
            acc[0] = fmaf(w, x.x, acc[0]);
            acc[1] = fmaf(w, x.y, acc[1]);
            acc[2] = fmaf(w, x.z, acc[2]);
            acc[3] = fmaf(w, x.w, acc[3]);
            acc[4] = fmaf(w, y.x, acc[4]);
            acc[5] = fmaf(w, y.y, acc[5]);
            acc[6] = fmaf(w, y.z, acc[6]);
            acc[7] = fmaf(w, y.w, acc[7]);
        }
    }
    const float inv = total > 0.f ? 1.f / total : 0.f;
    uint4 v;
    v.x = pack_bf16x2(acc[0] * inv, acc[1] * inv);
    v.y = pack_bf16x2(acc[2] * inv, acc[3] * inv);
    v.z = pack_bf16x2(acc[4] * inv, acc[5] * inv);
    v.w = pack_bf16x2(acc[6] * inv, acc[7] * inv);
    *reinterpret_cast<uint4 *>(a.o + b * a.os[0] + h * a.os[1] + i * a.os[2] + e0) = v;
    if (e0 == 0) a.lse[id] = total > 0.f ? (M + log2f(total)) * 0.69314718055994530942f : -INFINITY;
}

// ----------------------------------------------------------------- host side
int attn_sms()
{
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    return sms > 0 ? sms : 148;
}

sfa_status check_attn(const sfa_cache_attn_desc *d)
{
    if (!d || d->B < 0 || d->Lq < 0 || d->max_kv < 0) return SFA_ERR_INVALID_ARG;
    if (d->d != 64 && d->d != 128) return SFA_ERR_UNSUPPORTED;
    if (d->H < 1 || d->H > SFA_MAX_HEADS || d->H_kv < 1 || d->H % d->H_kv) return SFA_ERR_INVALID_ARG;
    if (!(d->scale > 0.f) || !std::isfinite(d->scale)) return SFA_ERR_INVALID_ARG;
    if (d->len_stride[0] < 0 || d->len_stride[1] < 0) return SFA_ERR_INVALID_ARG;
    if ((int64_t)d->B * d->H * d->Lq >= ((int64_t)1 << 31)) return SFA_ERR_INVALID_ARG;
    return SFA_OK;
}

struct Plan {
    bool tiles;  // tile_attn_kernel, else rows_attn_kernel
    int row_tiles, n_split, range_len;
    int64_t ctas;
};

constexpr int MAX_SPLIT = 64;
constexpr int TILE_MIN_ROWS = 17;

Plan plan_of(const sfa_cache_attn_desc *d, const sfa_cache *c)
{
    Plan p;
    const int64_t rows = (int64_t)d->Lq * (d->H / d->H_kv);
    p.tiles = rows >= TILE_MIN_ROWS;
    const int tile_rows = p.tiles ? CT_ROWS : FR_ROWS, step_keys = p.tiles ? BN : FR_KEYS;
    p.row_tiles = (int)((rows + tile_rows - 1) / tile_rows);
    const int64_t units = (int64_t)d->B * d->H_kv * p.row_tiles;
    int64_t kv = (int64_t)c->table_len * c->page_len;
    if (d->max_kv > 0 && d->max_kv < kv) kv = d->max_kv;
    const int64_t steps = std::max<int64_t>(1, (kv + step_keys - 1) / step_keys);
    // Modelled as waves of equal ranges: a range costs its steps and a fixed start and end,
    // and the joining kernel the partial results' bytes (in steps of a CTA's share).
    const double slots = (double)attn_sms() * (p.tiles ? 1 : 4);
    const double fixed = p.tiles ? 4.0 : 6.0;
    const double step_us = p.tiles ? 2.4 : 1.6;
    const double join_us = (double)d->B * d->H * d->Lq * (d->d + 1) * 4.0 / 5.0e6;
    double best = 1e300;
    p.n_split = 1;
    for (int64_t k = 1; k <= MAX_SPLIT && k <= steps; ++k) {
        const double len = (double)((steps + k - 1) / k);
        const double us = std::ceil(units * k / slots) * (len + fixed) * step_us + (k > 1 ? 3.0 + (k + 1) * join_us : 0.0);
        if (us < best) {
            best = us;
            p.n_split = (int)k;
        }
    }
    p.range_len = (int)std::min<int64_t>((steps + p.n_split - 1) / p.n_split, 1 << 30);
    p.ctas = units * p.n_split;
    return p;
}

template <int D>
sfa_status launch_tiles(const ChunkArgs &a, unsigned grid, cudaStream_t s)
{
    if (cudaFuncSetAttribute(tile_attn_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<D>::SMEM_BYTES) !=
        cudaSuccess)
        return SFA_ERR_CUDA;
    tile_attn_kernel<D><<<grid, CT_THREADS, Cfg<D>::SMEM_BYTES, s>>>(a);
    return launch_status();
}

size_t part_bytes(const sfa_cache_attn_desc *d, int n_split)
{
    if (n_split == 1) return 0;
    const size_t rows = (size_t)d->B * d->H * d->Lq;
    return (n_split * rows * (d->d + 1) * sizeof(float) + 255) / 256 * 256;
}

}  // namespace
}  // namespace sfa

using namespace sfa;

extern "C" sfa_status sfa_forward_cache_workspace(const sfa_cache_attn_desc *d, const sfa_cache *cache, size_t *bytes)
{
    sfa_status st = check_attn(d);
    if (st != SFA_OK) return st;
    if (!bytes) return SFA_ERR_INVALID_ARG;
    *bytes = 0;
    if (d->B == 0 || d->Lq == 0) return SFA_OK;
    st = check_cache(cache, d->H_kv, d->d);
    if (st != SFA_OK) return st;
    *bytes = part_bytes(d, plan_of(d, cache).n_split);
    return SFA_OK;
}

extern "C" sfa_status sfa_forward_cache(const sfa_cache_attn_desc *d, const sfa_cache *cache, const void *q,
                                        const int32_t *kv_lens, const int32_t *q_lens, void *o, float *lse,
                                        void *workspace, size_t workspace_bytes, int32_t *dev_status,
                                        sfa_stream_t stream)
{
    sfa_status st = check_attn(d);
    if (st != SFA_OK) return st;
    if (d->B == 0 || d->Lq == 0) return SFA_OK;
    st = check_cache(cache, d->H_kv, d->d);
    if (st != SFA_OK) return st;
    if (!q || !o || !lse || !kv_lens || reinterpret_cast<uintptr_t>(q) % 16 || reinterpret_cast<uintptr_t>(o) % 16)
        return SFA_ERR_INVALID_ARG;
    if (!rows_stride_ok(d->q_stride, d->B, d->H, d->Lq) || !rows_stride_ok(d->o_stride, d->B, d->H, d->Lq))
        return SFA_ERR_INVALID_ARG;
    const Plan p = plan_of(d, cache);
    if (p.ctas >= ((int64_t)1 << 31)) return SFA_ERR_INVALID_ARG;
    const size_t need = part_bytes(d, p.n_split);
    if (need && (!workspace || reinterpret_cast<uintptr_t>(workspace) % 256 || workspace_bytes < need))
        return SFA_ERR_INVALID_ARG;
    ChunkArgs a = {};
    a.cache = cache_view(cache);
    a.B = d->B;
    a.H = d->H;
    a.Hk = d->H_kv;
    a.G = d->H / d->H_kv;
    a.Lq = d->Lq;
    a.q = static_cast<const uint16_t *>(q);
    a.o = static_cast<uint16_t *>(o);
    for (int i = 0; i < 3; ++i) {
        a.qs[i] = d->q_stride[i];
        a.os[i] = d->o_stride[i];
    }
    a.kv_lens = kv_lens;
    a.q_lens = q_lens;
    a.ls0 = d->len_stride[0];
    a.ls1 = d->len_stride[1];
    a.causal = d->causal != 0;
    a.scale_log2 = d->scale * 1.4426950408889634f;
    a.lse = lse;
    a.status = dev_status;
    a.n_row_tiles = p.row_tiles;
    a.n_split = p.n_split;
    const int64_t rows = (int64_t)d->B * d->H * d->Lq;
    a.part_o = static_cast<float *>(workspace);
    a.part_lse = a.part_o ? a.part_o + (int64_t)p.n_split * rows * d->d : nullptr;
    a.range_len = p.range_len;
    a.timeout_ns = (uint64_t)(d->timeout_us ? d->timeout_us : DEFAULT_TIMEOUT_US) * 1000;
    a.debug_flags = d->debug_flags;
    cudaStream_t s = as_cuda(stream);
    const unsigned grid = (unsigned)p.ctas;
    if (p.tiles) {
        st = d->d == 128 ? launch_tiles<128>(a, grid, s) : launch_tiles<64>(a, grid, s);
    } else {
        if (d->d == 128) rows_attn_kernel<128><<<grid, FR_WARPS * 32, 0, s>>>(a);
        else rows_attn_kernel<64><<<grid, FR_WARPS * 32, 0, s>>>(a);
        st = launch_status();
    }
    if (st != SFA_OK || p.n_split == 1) return st;
    cudaLaunchConfig_t cfg = {};
    const int per_cta = 128 / (d->d / 8);
    cfg.gridDim = dim3((unsigned)((rows + per_cta - 1) / per_cta));
    cfg.blockDim = dim3(128);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = d->d == 128 ? cudaLaunchKernelEx(&cfg, join_kernel<128>, a) : cudaLaunchKernelEx(&cfg, join_kernel<64>, a);
    return cuda_status(e);
}
