// Attention of a chunk of new tokens over the 8-bit frame cache.
//
//   O_i = sum_j softmax_j(scale q_i . k_j) v_j over the logical tokens j of (b, key head),
//   k_j = 2^e c_j per block of 32 elements (exactly a bf16 number), the same for v_j,
// with the log-sum-exp of every row ("ISPA", §2.1), causal or over all tokens, the query
// heads of a key head sharing its rows.
//
// Few query rows (rows_attn_kernel): every code is read once from HBM, converted and used for
// at most 16 rows, so the floor is the cache's bytes.  Many (tile_attn_kernel): 4 d operations a
// query and key on the tensor cores.  Where there are few units of work either cuts the keys
// into ranges, and join_kernel joins their results by the log-sum-exp.
#include <cuda.h>
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
    int32_t range_len;  // key steps of a range, see Unit::len
    int32_t target;     // > 0: CTAs that the ranges are dealt out to by the lengths on the device
    int32_t even_split; // ranges of a cache, at most, without a target or where all are about as long
    float *part_o;    // [n_split][B * H * Lq][d], normalised, when n_split > 1
    float *part_lse;  // [n_split][B * H * Lq], log2 units
    uint64_t timeout_ns;
    uint32_t debug_flags;
};

// A row keeps a running maximum m that later scores have outgrown while their probabilities
// 2^(s - m) stay below 2^GROWTH.  They are floating numbers (bf16 for the product with V, fp32
// in the sums), so their precision does not depend on m; what limits the growth is overflow, of
// O from values beyond 2^(127 - GROWTH).  A small limit costs time instead: with 2^8, keys of
// uneven norm sent the rows of the streaming chunk through the rescaling often enough to take
// 764 us instead of 568.
constexpr float GROWTH = 24.f;

constexpr float EQUAL_LENGTHS = 0.93f;  // mean over longest, from which the caches count as equally long

// What a CTA works on: rows [row0, row0 + tile) of (b, hk), row r being token r / G of query
// head hk * G + r % G, and its share of the keys those rows see.
struct Unit {
    int b, hk, row0, split;
    int ranges;   // that the unit's keys are cut into, at most
    int len;      // key steps of a range, at least
    int m, n;     // query tokens and cache tokens
    int n_rows;   // m * G
    bool bad;     // n outside the table
};

constexpr int MAX_DEALT = 128;  // caches (B * H_kv) whose lengths a warp goes through

// Key steps of the i-th cache, cut at 2^20: so that MAX_DEALT of them add up in 32 bits, and for
// exact quotients in fp32 below (t + len - 1/2 has 22 bits, and no multiple of len within 1/2).
__device__ __forceinline__ int steps_of(const ChunkArgs &a, int i, int step_keys)
{
    if (i >= a.B * a.Hk) return 0;
    const int b = (int)(((float)i + 0.5f) * (1.f / (float)a.Hk));
    const int n = __ldg(a.kv_lens + b * a.ls0 + (i - b * a.Hk) * a.ls1);
    return n > 0 && n <= a.cache.table_len * a.cache.page_len ? min((n + step_keys - 1) / step_keys, 1 << 20) : 0;
}

// CTA x's cache, row tile and range where the caches' lengths differ (every lane of a warp calls it;
// false: there is none).  Ranges have the shortest length that makes no more than `target` of them,
// so that all start at once and end about together, and the CTAs with a range are the first
// ones: where CTAs without one lay between, a launch of 64 two-tile units took 51 us for 37, each
// holding its SM for a few us.  The loops are short code, which runs once.
// Against ranges cut by the bound alone, us: one token, 8 x 12 caches of 16384 at most, d = 128: half to
// all of it 86, now 74, one long and the rest a quarter 49 (shares by length) and 41; 12 caches of 6,
// 7 or 13 frames under 200 and 1000 rows 53 and 159, now 45 and 132; 2 x 333 causal rows, 12 on 4
// heads, d = 64, over 4099 and less 34.8, now 30.8; 32 caches of 8192, d = 128, 100 rows, one long
// 40.4, now 29.  Where all are equal the tile kernel pays for looking: 34.9 and 36.9, 55.4 and
// 57.4, 42.9 and 47.2, one token 95.7 and 96.6.
__device__ __forceinline__ bool deal(const ChunkArgs &a, int step_keys, int total, int longest, int x, int &cache,
                                     int &tile, Unit &u)
{
    const int heads = a.B * a.Hk, lane = threadIdx.x & 31;
    const int room = a.target / a.n_row_tiles;  // ranges of one row tile of all caches; `heads` or more
    float per_len;
    int len = max(1, (total + room - 1) / room);
    auto ranges_of = [&](int i) {
        const int r = (int)(((float)(steps_of(a, i, step_keys) + len) - 0.5f) * per_len);
        return i < heads ? max(1, r) : 0;
    };
#pragma unroll 1
    for (;; len += 1 + (len >> 4)) {
        per_len = 1.f / (float)len;
        int count = 0;
#pragma unroll 1
        for (int i = lane; i < heads; i += 32) count += ranges_of(i);
        if (len >= longest || __reduce_add_sync(0xffffffffu, count) <= room) break;
    }
#pragma unroll 1
    for (int i0 = 0; i0 < heads; i0 += 32) {
        const int mine = min(a.n_split, ranges_of(i0 + lane));
        int upto = mine * a.n_row_tiles;  // CTAs of the caches up to this lane's
#pragma unroll 1
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, upto, o);
            upto += lane >= o ? y : 0;
        }
        const int all = __shfl_sync(0xffffffffu, upto, 31);
        if (x < all) {
            const int at = __ffs(__ballot_sync(0xffffffffu, x < upto)) - 1;
            u.ranges = __shfl_sync(0xffffffffu, mine, at);
            x -= __shfl_sync(0xffffffffu, upto, at) - u.ranges * a.n_row_tiles;
            cache = i0 + at;
            tile = x / u.ranges;
            u.split = x - tile * u.ranges;
            u.len = 1;
            return true;
        }
        x -= all;
    }
    return false;
}

// DEAL: the launch may have a target.  (A kernel of its own with many rows: the code above, only
// jumped over, cost the streaming chunk 571 us instead of 555.)
template <bool DEAL>
__device__ __forceinline__ Unit open_unit(const ChunkArgs &a, int tile_rows, int step_keys)
{
    Unit u;
    int x = blockIdx.x, rt = 0;
    bool even = true, there = true;
    u.ranges = a.even_split;
    u.len = a.range_len;
    if (DEAL && a.target) {
        const int heads = a.B * a.Hk;
        int total = 0, longest = 0;
#pragma unroll 1
        for (int i = threadIdx.x & 31; i < heads; i += 32) {
            const int t = steps_of(a, i, step_keys);
            total += t;
            longest = max(longest, t);
        }
        total = __reduce_add_sync(0xffffffffu, total);
        longest = __reduce_max_sync(0xffffffffu, longest);
        even = (float)total >= EQUAL_LENGTHS * longest * heads;
        if (!even) there = deal(a, step_keys, total, longest, x, x, rt, u);
    }
    if (even) {  // the host's plan for the bound, which may take several waves
        u.split = x % a.even_split;
        x /= a.even_split;
        rt = x % a.n_row_tiles;
        x /= a.n_row_tiles;
        there = x < a.B * a.Hk;
    }
    if (DEAL) {  // (in uniform registers again, as what comes of the block's number alone is)
        x = __reduce_max_sync(0xffffffffu, there ? x : -1);
        rt = __reduce_max_sync(0xffffffffu, rt);
        u.split = __reduce_max_sync(0xffffffffu, u.split);
        u.ranges = __reduce_max_sync(0xffffffffu, u.ranges);
        u.len = __reduce_max_sync(0xffffffffu, u.len);
    }
    if (DEAL && x < 0) {
        u.bad = false;
        u.row0 = u.n_rows = 0;
        return u;
    }
    // causal: the last row tiles see the most keys and start first
    u.row0 = (a.causal ? a.n_row_tiles - 1 - rt : rt) * tile_rows;
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

// Ranges that the key steps of a unit are cut into: as many of `len` steps as it has, so that long
// and short caches give pieces of one length, but never more than the CTAs that it was given
// (caches longer than the caller's bound just get longer ranges).
__device__ __forceinline__ int n_ranges(const Unit &u, int steps)
{
    return max(1, min(u.ranges, (steps + u.len - 1) / u.len));
}

// Row `id` of the outputs: (b * H + h) * Lq + i for row r of a unit.
__device__ __forceinline__ int64_t row_id(const ChunkArgs &a, const Unit &u, int r)
{
    const int tok = a.G == 1 ? r : r / a.G;
    return ((int64_t)u.b * a.H + u.hk * a.G + (r - tok * a.G)) * a.Lq + tok;
}

// Thirty-two rows of a unit, N apart from one access to the next: f(access, element offset, whether
// the row is there) under the given strides of a query head and a token.  Row r is token r / G of
// head r % G; the offset of a row that is not there is 0.
struct RowWalk {
    int r, tok, head;
    __device__ __forceinline__ RowWalk(const ChunkArgs &a, const Unit &u, int first)
    {
        r = first;
        tok = a.G == 1 ? first : first / a.G;
        head = first - tok * a.G;
    }
    template <int N, typename F>
    __device__ __forceinline__ void each(const ChunkArgs &a, const Unit &u, int64_t head_stride, int64_t tok_stride,
                                         F f) const
    {
        int64_t at = (u.hk * a.G + head) * head_stride + tok * tok_stride;
        const int n = u.n_rows - r;  // rows from the first on
        if (a.G == 1) {
            const int64_t step = N * tok_stride;
#pragma unroll 4
            for (int i = 0; i < 32 / N; ++i) {
                f(i, i * N < n ? at : 0, i * N < n);
                at += step;
            }
            return;
        }
        const int64_t next_tok = tok_stride - a.G * head_stride;
        int h = head;
#pragma unroll 4
        for (int i = 0; i < 32 / N; ++i) {
            f(i, i * N < n ? at : 0, i * N < n);
            at += N * head_stride;
            h += N;
            while (h >= a.G) {
                h -= a.G;
                at += next_tok;
            }
        }
    }
};

// Stores 16-byte pieces four at a time, so that as many reads of shared memory are under way.
template <typename T>
struct RowOut {
    T *dst;
    uint4 v[4];
    int64_t at[4];
    bool on[4];
    __device__ __forceinline__ explicit RowOut(T *d) : dst(d) {}
    __device__ __forceinline__ void put(int i, const uint4 &x, int64_t offset, bool there)
    {
        v[i & 3] = x;
        at[i & 3] = offset;
        on[i & 3] = there;
        if ((i & 3) != 3) return;
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (on[k]) *reinterpret_cast<uint4 *>(dst + at[k]) = v[k];
    }
};

// The log-sum-exp of a row in this CTA's range, and "nothing seen" in the ranges that no CTA has:
// every `ranges`-th from its own on.
template <bool DEAL>
__device__ __forceinline__ void put_part_lse(const ChunkArgs &a, int split, int ranges, int64_t id, float lse2)
{
    const int64_t part_rows = (int64_t)a.B * a.H * a.Lq;
    a.part_lse[split * part_rows + id] = lse2;
    if (!DEAL) return;
#pragma unroll 1
    for (int s = split + ranges; s < a.n_split; s += ranges) a.part_lse[s * part_rows + id] = -INFINITY;
}

// A CTA whose rows see too few keys for its range leaves "nothing seen".
template <bool DEAL>
__device__ __forceinline__ void skip_range(const ChunkArgs &a, const Unit &u, int tile_rows)
{
    for (int r = u.row0 + threadIdx.x; r < min(u.row0 + tile_rows, u.n_rows); r += blockDim.x)
        put_part_lse<DEAL>(a, u.split, u.ranges, row_id(a, u, r), -INFINITY);
}

// ----------------------------------------------------------------- few query rows
// Sixteen rows against the keys, with the m16n8k16 matrix instruction.  A warp owns every
// fourth stretch of 32 keys of the CTA's range and streams them through a ring of its own in
// shared memory, so that the next stretch is on its way while it works on one (one token of 8
// sequences, 12 heads, 8192 to 16384 tokens, d = 128: 130 us with the loads in registers, 86 with the
// ring, 74 to 76 with ranges cut by the lengths, 4.3 TB/s; HBM's time is 50, the copies alone take 57).
// The codes are turned into bf16 in the lane layout of the instruction, whose k index may be any
// order of the elements as long as Q has the same; the key range is cut over warps and CTAs,
// and the partial results are joined by their log-sum-exp.
// What bounds it is issue: of some 1000 instructions for 32 keys of 128 elements 64 are matrix
// instructions and 512 turn codes into bf16, at two warps and a half a scheduler that wait for
// one another's results (55 % of the issue slots).  Sixteen warps an SM instead of twelve, with Q in
// shared memory to get by on 128 registers: 102 us instead of 86.  17 to 32 rows are two row tiles,
// which read and convert the cache twice (24 rows, 12 heads x 4 sequences over 8192: 47 us).
constexpr int FR_WARPS = 4;
constexpr int FR_ROWS = 16;              // the matrix instruction's rows
constexpr int FR_STRETCH = 32;           // keys that a warp works on at a time
constexpr int FR_KEYS = FR_STRETCH * FR_WARPS;  // keys of one step of the CTA
constexpr int FR_STAGES = 2;             // slots of a warp's ring
constexpr int FR_CTAS = 3;               // CTAs an SM: 168 registers a thread

template <int D>
struct FCfg {
    static constexpr int CODES = FR_STRETCH * D;                // a stretch's codes
    static constexpr int SCALES = FR_STRETCH * (D / CACHE_BLOCK);
    static constexpr int RING = FR_WARPS * FR_STAGES * 2 * CODES;  // K, then V, of every slot
    static constexpr int SMEM_SCALES = RING;
    static constexpr int SMEM_BARS = SMEM_SCALES + FR_WARPS * FR_STAGES * 2 * SCALES;
    static constexpr int SMEM_FLAGS = SMEM_BARS + FR_WARPS * FR_STAGES * 8;
    static constexpr int SMEM_BYTES = SMEM_FLAGS + 16 + 1024;  // + alignment slack
    static constexpr int O_PITCH = D + 4;               // floats of a row of a warp's O, in the ring's place
    static_assert(FR_WARPS * FR_ROWS * O_PITCH * 4 <= RING, "O fits the ring");
};

__device__ __forceinline__ void mma_16816(float (&c)[4], const uint4 &a, uint32_t b0, uint32_t b1)
{
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
}

// The four codes of a word -> two bf16 pairs times f
__device__ __forceinline__ void codes_of_word(uint32_t w, uint32_t f, uint32_t &p0, uint32_t &p1)
{
    p0 = mul_bf16x2(spread_codes<CODES_01>(w, w), f);
    p1 = mul_bf16x2(spread_codes<CODES_23>(w, w), f);
}

// compile-time answers for the code paths of large scales
struct Yes {
    static constexpr bool value = true;
};
struct No {
    static constexpr bool value = false;
};

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

// byte offset of the 16-byte piece `ch` of row r in a slot: the order in which the tensor-map
// copies store rows of 128 (64) bytes, under which the reads below meet no bank twice (V at
// d = 64: twice)
template <int D>
__device__ __forceinline__ uint32_t slot_piece(int r, int ch)
{
    return (uint32_t)(r * D + ((ch ^ (D == 128 ? r & 7 : (r >> 1) & 3)) << 4));
}

__device__ __forceinline__ uint4 lds16(uint32_t addr)
{
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
    return v;
}
__device__ __forceinline__ uint2 lds8(uint32_t addr)
{
    uint2 v;
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr));
    return v;
}
__device__ __forceinline__ uint32_t lds1(uint32_t addr)
{
    uint32_t v;
    asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(addr));
    return v;
}

// Grid: (b, key head, row tile, key range), the key range fastest.  Lane (g = lane / 4,
// t = lane % 4) holds, of 32 keys: of K the rows g + 8 i, elements t * D/4 .. + D/4 - 1 (at
// d = 128 one block); of V the rows 16 h + 2t + {0, 1, 8, 9}, elements g * D/8 .. + D/8 - 1.
// Output column i of n-tile i' is then element (its lane's column) * D/8 + i', so a lane ends up
// with D/4 consecutive elements of two rows.
// BULK (pages of a multiple of 16 rows, 16-byte aligned scales): 16 keys are one piece of
// memory, and lanes 0 and 1 copy a half each with two tensor-map boxes and two bulk copies;
// otherwise the lanes look up a row each and copy 16-byte pieces.
template <int D, bool BULK>
__global__ void __launch_bounds__(FR_WARPS * 32, FR_CTAS)
    rows_attn_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                     const __grid_constant__ ChunkArgs a)
{
    using C = FCfg<D>;
    constexpr int KS = D / 16;          // k-steps of S
    constexpr int KP = D / 64;          // 16-byte pieces of a K row per lane
    constexpr int VW = D / 32;          // words of a V row per lane
    constexpr int NT = D / 8;           // n-tiles of the output
    typedef typename ScaleWord<D>::type scale_t;
    extern __shared__ uint8_t smem_raw[];
    __shared__ float ml_sh[FR_WARPS][FR_ROWS][2];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = smem_u32(smem);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, t = lane & 3;
    if (a.n_split > 1) pdl_launch_dependents();  // the joining kernel's CTAs may take their places
    const Unit u = open_unit<true>(a, FR_ROWS, FR_KEYS);
    if (u.bad && tid == 0) report_status(a.status, SFA_ERR_BAD_SET);
    if (u.row0 >= u.n_rows) return;  // rows behind this sequence's last
    // the tile's last row sees the most keys
    const int seen = row_limit(a, u, min(u.row0 + FR_ROWS, u.n_rows) - 1);
    const int steps = (seen + FR_KEYS - 1) / FR_KEYS;
    const int ranges = n_ranges(u, steps);
    if (u.split >= ranges) return skip_range<true>(a, u, FR_ROWS);
    const int s0 = (int)((int64_t)steps * u.split / ranges), s1 = (int)((int64_t)steps * (u.split + 1) / ranges);
    // this warp's stretches: keys FR_KEYS (s0 + k) + 32 warp .. + 31, those that start before the end
    const int key0 = s0 * FR_KEYS + warp * FR_STRETCH;
    const int n = max(0, min(s1 - s0, (seen - key0 + FR_KEYS - 1) / FR_KEYS));

    const uint32_t ring = sbase + warp * FR_STAGES * 2 * C::CODES;
    const uint32_t scales = sbase + C::SMEM_SCALES + warp * FR_STAGES * 2 * C::SCALES;
    const uint32_t bars = sbase + C::SMEM_BARS + warp * FR_STAGES * 8;
    volatile int32_t *abort_flag = reinterpret_cast<volatile int32_t *>(smem + C::SMEM_FLAGS);
    if (lane < FR_STAGES) mbar_init(bars + 8 * lane, BULK ? 1 : 32);
    volatile int32_t *ranges_sh = abort_flag + 1;  // (not in a register until the end)
    if (tid == 0) {
        *abort_flag = 0;
        *ranges_sh = u.ranges;
    }
    fence_mbar_init();
    __syncthreads();
    const Ctl ctl{abort_flag, a.status, a.timeout_ns};

    const int32_t *table = a.cache.table + u.b * a.cache.ts0 + u.hk * a.cache.ts1;
    CachePlace place;  // of the next stretch to copy (BULK: the first row of half lane & 1; else row `lane`)
    auto look_up = [&](int k) {
        const int j = key0 + k * FR_KEYS + (BULK ? (lane & 1) * 16 : lane);
        place.open(a.cache, table, j, k < n && j < seen);
    };
    uint32_t pend_k = 0u, pend_v = 0u;  // !BULK: the scales that the stretch before is still to get
    auto put_scales = [&](int k) {
        const uint32_t at = scales + (k % FR_STAGES) * 2 * C::SCALES + lane * (D / CACHE_BLOCK);
        if (D == 128) {
            asm volatile("st.shared.u32 [%0], %1;" ::"r"(at), "r"(pend_k) : "memory");
            asm volatile("st.shared.u32 [%0], %1;" ::"r"(at + C::SCALES), "r"(pend_v) : "memory");
        } else {
            asm volatile("st.shared.u16 [%0], %1;" ::"r"(at), "h"((uint16_t)pend_k) : "memory");
            asm volatile("st.shared.u16 [%0], %1;" ::"r"(at + C::SCALES), "h"((uint16_t)pend_v) : "memory");
        }
    };
    auto copy = [&](int k) {  // stretch k into its slot
        if (k >= n) return;
        const int s = k % FR_STAGES;
        const uint32_t slot = ring + s * 2 * C::CODES, sc = scales + s * 2 * C::SCALES, bar = bars + 8 * s;
        const int r = place.row(a.cache, u.hk, a.status), row = max(r, 0);
        if (BULK) {
            if (lane == 0)
                mbar_arrive_expect_tx(bar, (C::CODES + C::SCALES) * (key0 + k * FR_KEYS + 16 < seen ? 2 : 1));
            __syncwarp();
            if (lane < 2 && place.wanted) {
                constexpr int HC = C::CODES / 2, HS = C::SCALES / 2;
                tma_load_2d(slot + lane * HC, &tm_k, bar, 0, row);
                tma_load_2d(slot + C::CODES + lane * HC, &tm_v, bar, 0, row);
                bulk_load(sc + lane * HS, a.cache.k_scale + (int64_t)row * (D / CACHE_BLOCK), HS, bar);
                bulk_load(sc + C::SCALES + lane * HS, a.cache.v_scale + (int64_t)row * (D / CACHE_BLOCK), HS, bar);
            }
        } else {
            constexpr int PR = D / 16, RPI = 32 / PR;  // pieces of a row, rows per access of the warp
#pragma unroll
            for (int i = 0; i < FR_STRETCH / RPI; ++i) {
                const int rr = i * RPI + lane / PR, ch = lane % PR;
                const int src = __shfl_sync(0xffffffffu, r, rr);
                const int64_t at = (int64_t)max(src, 0) * D + ch * 16;
                cp_async16(slot + slot_piece<D>(rr, ch), a.cache.k + at, src >= 0);
                cp_async16(slot + C::CODES + slot_piece<D>(rr, ch), a.cache.v + at, src >= 0);
            }
            cp_async_arrive(bar);
            pend_k = (uint32_t)__ldg(reinterpret_cast<const scale_t *>(a.cache.k_scale) + row);
            pend_v = (uint32_t)__ldg(reinterpret_cast<const scale_t *>(a.cache.v_scale) + row);
        }
    };
    look_up(0);
    for (int k = 0; k < FR_STAGES - 1; ++k) {
        copy(k);
        look_up(k + 1);
    }

    // Q in the A-operand layout of every k-step: rows g and g + 8, elements t * D/4 + 4 ks
    // + {0, 1} and {2, 3}
    uint4 qf[KS];
    {
        const uint16_t *src[2];
        bool on[2];
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const int r = u.row0 + g + 8 * s;
            on[s] = r < u.n_rows;
            const int tok = on[s] ? r / a.G : 0, head = on[s] ? r - tok * a.G : 0;
            src[s] = a.q + u.b * a.qs[0] + (u.hk * a.G + head) * a.qs[1] + tok * a.qs[2] + t * (D / 4);
        }
#pragma unroll
        for (int ks = 0; ks < KS; ks += 2) {  // 8 consecutive elements: two k-steps
            uint4 v[2];
#pragma unroll
            for (int s = 0; s < 2; ++s)
                v[s] = on[s] ? __ldg(reinterpret_cast<const uint4 *>(src[s] + 4 * ks)) : make_uint4(0u, 0u, 0u, 0u);
            qf[ks] = make_uint4(v[0].x, v[1].x, v[0].y, v[1].y);
            qf[ks + 1] = make_uint4(v[0].z, v[1].z, v[0].w, v[1].w);
        }
    }
    // keys that rows g and g + 8 see; rows that are not there see all of them
    const int r0 = u.row0 + g, r1 = r0 + 8;
    const int lim0 = r0 < u.n_rows ? row_limit(a, u, r0) : seen, lim1 = r1 < u.n_rows ? row_limit(a, u, r1) : seen;
    const int lim_all = __reduce_min_sync(0xffffffffu, min(lim0, lim1));  // what every row sees
    const float sl2 = a.scale_log2;

    float o[NT][4];
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) o[i][j] = 0.f;
    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;  // of rows g and g + 8

    int k = 0;
    // TWO: a block of these rows has e > 0, whose 2^(120 + e) may pass bf16's range
    auto stretch = [&](auto two, uint32_t slot, const uint32_t (&kb)[4], const uint32_t (&vb)[8]) {
        constexpr bool TWO = decltype(two)::value;
        // ---- S = Q K^T, keys 8 i + 2 t + {0, 1} of rows g, g + 8
        float sc[4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) sc[i][j] = 0.f;
        uint32_t kf[4], kf2[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            kf[i] = TWO ? scale_bits(kb[i]) * 0x10001u : scale_pair(kb[i]);
            kf2[i] = scale_rest_bits(kb[i]) * 0x10001u;
        }
#pragma unroll
        for (int c = 0; c < KP; ++c) {
            uint4 kr[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) kr[i] = lds16(slot + slot_piece<D>(g + 8 * i, KP * t + c));
#pragma unroll
            for (int w = 0; w < 4; ++w)
#pragma unroll
                for (int i = 0; i < 4; ++i) {  // four sums in turn
                    uint32_t b0, b1;
                    codes_of_word(w == 0 ? kr[i].x : w == 1 ? kr[i].y : w == 2 ? kr[i].z : kr[i].w, kf[i], b0, b1);
                    if (TWO) {
                        b0 = mul_bf16x2(b0, kf2[i]);
                        b1 = mul_bf16x2(b1, kf2[i]);
                    }
                    mma_16816(sc[i], qf[4 * c + w], b0, b1);
                }
        }

        // ---- softmax of these keys (log2 units, the scale folded into the exponent's FMA)
        const int key = key0 + k * FR_KEYS;
        if (key + FR_STRETCH > lim_all) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int x = key + 8 * i + 2 * t + j;
                    sc[i][j] = x < lim0 ? sc[i][j] : -INFINITY;
                    sc[i][2 + j] = x < lim1 ? sc[i][2 + j] : -INFINITY;
                }
        }
        float x0 = -INFINITY, x1 = -INFINITY;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x0 = fmax3(x0, sc[i][0], sc[i][1]);
            x1 = fmax3(x1, sc[i][2], sc[i][3]);
        }
        x0 *= sl2;
        x1 *= sl2;
        // a maximum of -inf (nothing seen) is always replaced
        if (__any_sync(0xffffffffu, x0 > m0 + GROWTH || x1 > m1 + GROWTH)) {
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
        // P goes to bf16, the type of the product with V, off by 2^-8 of each probability at most, as
        // sfa_forward does; in two bf16 parts it would double that product.  O's relative error is
        // 0.0023 with it, 0.0016 where O alone is rounded.  The row sums are of the fp32 numbers.
        const float z0 = m0 == -INFINITY ? 0.f : -m0, z1 = m1 == -INFINITY ? 0.f : -m1;
        uint4 p[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float e[8];
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const float(&x)[4] = sc[2 * h + s];
                e[4 * s] = ex2_approx(fmaf(x[0], sl2, z0));
                e[4 * s + 1] = ex2_approx(fmaf(x[1], sl2, z0));
                e[4 * s + 2] = ex2_approx(fmaf(x[2], sl2, z1));
                e[4 * s + 3] = ex2_approx(fmaf(x[3], sl2, z1));
                l0 += e[4 * s] + e[4 * s + 1];
                l1 += e[4 * s + 2] + e[4 * s + 3];
            }
            p[h].x = pack_bf16x2(e[0], e[1]);
            p[h].y = pack_bf16x2(e[2], e[3]);
            p[h].z = pack_bf16x2(e[4], e[5]);
            p[h].w = pack_bf16x2(e[6], e[7]);
        }

        // ---- O += P V, 16 keys at a time: the codes of two keys are dealt into pairs, then
        // converted like K's
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            uint32_t f[2], f2[2], v[4][VW];  // keys 2t, 2t + 1 and 2t + 8, 2t + 9
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const uint32_t ba = vb[4 * h + 2 * s], bb = vb[4 * h + 2 * s + 1];
                f[s] = TWO ? scale_bits(ba) | (scale_bits(bb) << 16) : scale_pair(ba, bb);
                f2[s] = scale_rest_bits(ba) | (scale_rest_bits(bb) << 16);
            }
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                const int r = 16 * h + 2 * t + (s & 1) + (s >> 1) * 8;
                if (D == 128) {
                    const uint4 x = lds16(slot + C::CODES + slot_piece<D>(r, g));
                    v[s][0] = x.x, v[s][1] = x.y, v[s][VW - 2] = x.z, v[s][VW - 1] = x.w;
                } else {
                    const uint2 x = lds8(slot + C::CODES + slot_piece<D>(r, g >> 1) + (g & 1) * 8);
                    v[s][0] = x.x, v[s][1] = x.y;
                }
            }
#pragma unroll
            for (int w = 0; w < VW; ++w) {
                uint32_t b[2][4];
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    b[s][0] = mul_bf16x2(spread_codes<CODES_OF_TWO<0>>(v[2 * s][w], v[2 * s + 1][w]), f[s]);
                    b[s][1] = mul_bf16x2(spread_codes<CODES_OF_TWO<1>>(v[2 * s][w], v[2 * s + 1][w]), f[s]);
                    b[s][2] = mul_bf16x2(spread_codes<CODES_OF_TWO<2>>(v[2 * s][w], v[2 * s + 1][w]), f[s]);
                    b[s][3] = mul_bf16x2(spread_codes<CODES_OF_TWO<3>>(v[2 * s][w], v[2 * s + 1][w]), f[s]);
                    if (TWO) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) b[s][i] = mul_bf16x2(b[s][i], f2[s]);
                    }
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) mma_16816(o[4 * w + i], p[h], b[0][i], b[1][i]);
            }
        }
    };
    for (; k < n; ++k) {
        if (!BULK) put_scales(k);  // (asked for a stretch ago)
        copy(k + FR_STAGES - 1);   // into the slot that the stretch before has left
        look_up(k + FR_STAGES);
        const int s = k % FR_STAGES;
        if (!__all_sync(0xffffffffu, wait_bar(bars + 8 * s, (k / FR_STAGES) & 1, ctl))) break;
        __syncwarp();  // (!BULK: the scales stored by other lanes)
        const uint32_t slot = ring + s * 2 * C::CODES, sc = scales + s * 2 * C::SCALES;
        // scale bytes of this lane's blocks; a row that is not there gets 0, under which any code
        // is a finite number (its key is masked, its probability 0)
        uint32_t kb[4], vb[8];
        constexpr int SB = D / CACHE_BLOCK;
#pragma unroll
        for (int i = 0; i < 4; ++i) kb[i] = lds1(sc + (g + 8 * i) * SB + (D == 128 ? t : t >> 1));
#pragma unroll
        for (int i = 0; i < 8; ++i)
            vb[i] = lds1(sc + C::SCALES + (2 * t + (i & 1) + (i >> 1) * 8) * SB + g * NT / CACHE_BLOCK);
        const int left = seen - (key0 + k * FR_KEYS);
        if (left < FR_STRETCH) {
#pragma unroll
            for (int i = 0; i < 4; ++i) kb[i] = g + 8 * i < left ? kb[i] : 0u;
#pragma unroll
            for (int i = 0; i < 8; ++i) vb[i] = 2 * t + (i & 1) + (i >> 1) * 8 < left ? vb[i] : 0u;
        }
        uint32_t top = kb[0] | kb[1] | kb[2] | kb[3];
#pragma unroll
        for (int i = 0; i < 8; ++i) top |= vb[i];
        if (__any_sync(0xffffffffu, (top & SCALE_TOP_BITS) != 0u)) stretch(Yes{}, slot, kb, vb);
        else stretch(No{}, slot, kb, vb);
        __syncwarp();  // the slot has been read
    }
    if (*abort_flag) {  // a wait ran out: the copies still on their way land before the CTA ends
        for (int j = k; j < min(n, k + FR_STAGES); ++j) wait_drain(bars + 8 * (j % FR_STAGES), (j / FR_STAGES) & 1);
        cp_async_wait_all();
    }

    // ---- join the warps: every warp's O against the common max, then the sum of four
#pragma unroll
    for (int d = 1; d < 4; d <<= 1) {
        l0 += __shfl_xor_sync(0xffffffffu, l0, d);
        l1 += __shfl_xor_sync(0xffffffffu, l1, d);
    }
    __syncthreads();  // every ring has been read: O takes their place
    if (*abort_flag) return;
    float *o_sh = reinterpret_cast<float *>(smem) + warp * FR_ROWS * C::O_PITCH;
    if (t == 0) {
        ml_sh[warp][g][0] = m0;
        ml_sh[warp][g][1] = l0;
        ml_sh[warp][g + 8][0] = m1;
        ml_sh[warp][g + 8][1] = l1;
    }
#pragma unroll
    for (int i = 0; i < NT; ++i) {
        // columns 2t and 2t + 1 of n-tile i are elements 2t * NT + i and (2t + 1) * NT + i
        o_sh[g * C::O_PITCH + 2 * t * NT + i] = o[i][0];
        o_sh[g * C::O_PITCH + (2 * t + 1) * NT + i] = o[i][1];
        o_sh[(g + 8) * C::O_PITCH + 2 * t * NT + i] = o[i][2];
        o_sh[(g + 8) * C::O_PITCH + (2 * t + 1) * NT + i] = o[i][3];
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
            const float *src = reinterpret_cast<const float *>(smem) + (w * FR_ROWS + r) * C::O_PITCH + e0;
            l += c * ml_sh[w][r][1];
#pragma unroll
            for (int j = 0; j < 8; ++j) acc[j] = fmaf(c, src[j], acc[j]);
        }
        // (a NaN, from a query that holds one, stays a NaN)
        const float inv = l != 0.f ? 1.f / l : 0.f;
        const float lse2 = l != 0.f ? M + log2f(l) : -INFINITY;
        const int64_t id = row_id(a, u, row);
        if (a.n_split == 1) {
            const int tok = row / a.G, h = u.hk * a.G + (row - tok * a.G);
            uint4 v;
            v.x = pack_bf16x2(acc[0] * inv, acc[1] * inv);
            v.y = pack_bf16x2(acc[2] * inv, acc[3] * inv);
            v.z = pack_bf16x2(acc[4] * inv, acc[5] * inv);
            v.w = pack_bf16x2(acc[6] * inv, acc[7] * inv);
            *reinterpret_cast<uint4 *>(a.o + u.b * a.os[0] + h * a.os[1] + tok * a.os[2] + e0) = v;
            if (e0 == 0) a.lse[id] = lse2 * 0.69314718055994530942f;
        } else {
            float4 *dst = reinterpret_cast<float4 *>(a.part_o + ((int64_t)u.split * part_rows + id) * D + e0);
            dst[0] = make_float4(acc[0] * inv, acc[1] * inv, acc[2] * inv, acc[3] * inv);
            dst[1] = make_float4(acc[4] * inv, acc[5] * inv, acc[6] * inv, acc[7] * inv);
            if (e0 == 0) put_part_lse<true>(a, u.split, *ranges_sh, id, lse2);
        }
    }
}

// ----------------------------------------------------------------- many query rows
// Units of two 128-row query tiles A and B against 128-key tiles, on the tensor cores:
//   S_A(0) S_B(0) | P V_A(j) S_A(j+1) | P V_B(j) S_B(j+1) | ...
// (at d = 64, where P has columns of its own, S_x(j+1) before P V_x(j)).  While the softmax of
// one query tile runs, the tensor cores work on the other.  A unit with
// one query tile has both tiles' S buffers to itself and keeps S one key tile ahead:
//   S(0) S(1) | P V(j) S(j+2) | ...
// Seven warps load the codes of the K and V tiles into registers, look up the pages of the
// next tile meanwhile, and store them as bf16 in the 128-byte-swizzled layout that the matrix
// instruction reads, zeros behind the last key; the softmax warps bring their own query rows,
// since a unit's rows may be those of several heads.
// Shared memory is what this kernel runs short of: a 128 x 128 x 16 product with both
// operands there takes all of its bandwidth, and the converted tiles have to get in as well
// (with P in shared memory, as in the frame-list kernel, a key tile took 5600 cycles, 2200 of
// them in the issue of 11 loads behind blocked stores).  So P stays in tensor memory, in the
// columns of the S that it comes from or beside it, as the first operand of P V.
// A unit takes 2.8 us a key tile at d = 128 (900 TFLOP/s; 2.0 us at d = 64), some 5400 cycles, in
// which no pipe is full: 256 x 128 exponentials are 2048 cycles of an SM's special-function pipe,
// the four products about as many of the tensor cores, and half of the issue slots are used.
// At d = 128, P lying in the columns of its S, a query tile's S waits for its P V of the key tile
// before, and that for the softmax of 128 columns; with two query tiles under way this chain is the
// time (the largest stall is the wait for tensor memory).  A unit's start and end take as long as
// five key tiles at d = 128 (page lookups, queries, the first conversions; the last product and the
// rows' way out).  The streaming chunk, 4680 rows of 12 heads over 20280 tokens and fewer: 0.389 TFLOP
// in 552 us, 704 TFLOP/s (with bf16 keys and values in place sfa_forward takes 493).
// warps 0-3: softmax of query tile A, 4-7: of B
constexpr int CT_K_WARP = 8;              // 8-11: codes of K to bf16
constexpr int CT_V_WARP = 12;             // 12-14: of V
constexpr int CT_MMA_WARP = 15;
constexpr int CT_K_WARPS = CT_V_WARP - CT_K_WARP, CT_V_WARPS = CT_MMA_WARP - CT_V_WARP;
constexpr int CT_THREADS = 512;           // four warps to a scheduler: 128 registers a thread
constexpr int CT_ROWS = 2 * BM;

// Tensor-memory columns of P of buffer x: at d = 64 its own, beside O; at d = 128, where S and O
// take all 512, those of the S that it comes from.
template <int D>
__host__ __device__ constexpr uint32_t tcol_p(int x)
{
    return D == 64 ? tcol_o(x) + 64 : tcol_s(x);
}

template <int D>
struct CCfg {
    static constexpr int TILE_BYTES = BM * D * 2;  // one Q, K or V tile in bf16
    static constexpr int NSK = 2, NSV = 2;
    static constexpr int SMEM_Q = 0;               // query tiles A and B, then their output rows
    static constexpr int SMEM_K = 2 * TILE_BYTES;
    static constexpr int SMEM_V = SMEM_K + NSK * TILE_BYTES;
    static constexpr int SMEM_BAR = SMEM_V + NSV * TILE_BYTES;
    static constexpr int SMEM_BYTES = SMEM_BAR + 256 + 1024;  // + barriers, + alignment slack
};

// mbarriers (8 bytes each) at SMEM_BAR
template <int D>
struct CBars {
    uint32_t base;
    static constexpr int NSK = CCfg<D>::NSK, NSV = CCfg<D>::NSV;
    __device__ uint32_t k_full(int s) const { return base + 8 * s; }
    __device__ uint32_t k_free(int s) const { return base + 8 * (NSK + s); }
    __device__ uint32_t v_full(int s) const { return base + 8 * (2 * NSK + s); }
    __device__ uint32_t v_free(int s) const { return base + 8 * (2 * NSK + NSV + s); }
    __device__ uint32_t s_full(int x) const { return base + 8 * (2 * NSK + 2 * NSV + x); }      // S of tile x
    __device__ uint32_t p_full(int x) const { return base + 8 * (2 * NSK + 2 * NSV + 2 + x); }  // P of tile x
    __device__ uint32_t o_final() const { return base + 8 * (2 * NSK + 2 * NSV + 4); }  // after the last P V
    __device__ uint32_t pv_done() const { return base + 8 * (2 * NSK + 2 * NSV + 5); }  // one-tile units: a P V
    __device__ uint32_t drain() const { return base + 8 * (2 * NSK + 2 * NSV + 6); }
    __device__ uint32_t pv_x(int x) const { return base + 8 * (2 * NSK + 2 * NSV + 7 + x); }  // d = 64: P V of tile x
    static constexpr int COUNT = 2 * NSK + 2 * NSV + 9;
    static_assert(8 * COUNT <= 160, "mbarriers end before the flags at +160");
};

// byte offset of the 16-byte piece `ch` (8 elements) of row r in a swizzled tile
template <int D>
__device__ __forceinline__ uint32_t swz(int r, int ch)
{
    return (uint32_t)((ch >> 3) * Cfg<D>::BOX_BYTES + r * 128 + (((ch & 7) ^ (r & 7)) << 4));
}

// The barriers and tensor memory are there from here on.  Every warp passes it once, from its
// role's code: what it can load before, it has under way by then.
__device__ __forceinline__ void block_meets()
{
    tc_fence_before();
    named_bar_sync(0, CT_THREADS);
    tc_fence_after();
}

// The K (IS_K) or V tiles of the unit, codes to bf16.  D/16 lanes share a row, 16 codes each,
// and the tile's rows go round the warps, RPI at a time.  A lane looks up one row's place (two
// where a warp has more than 32 rows).  The next tile's codes are on their way while the warp
// waits for its slot.
template <int D, bool IS_K>
__device__ void convert_role(const ChunkArgs &a, const Unit &u, uint32_t sbase, int key0, int key_end, int n_tiles,
                             const volatile int32_t *skip, const Ctl &ctl)
{
    using C = CCfg<D>;
    constexpr int NS = IS_K ? C::NSK : C::NSV;
    constexpr int NW = IS_K ? CT_K_WARPS : CT_V_WARPS;
    constexpr int LR = D / 16;                         // lanes per row
    constexpr int RPI = 32 / LR;                       // rows per load of the warp
    constexpr int NI = (BN / RPI + NW - 1) / NW;       // loads per tile
    constexpr int LK = (NI * RPI + 31) / 32;           // places that a lane looks up
    typedef typename ScaleWord<D>::type scale_t;
    const CBars<D> bar{sbase + C::SMEM_BAR};
    const uint8_t *codes = IS_K ? a.cache.k : a.cache.v;
    const scale_t *scales = reinterpret_cast<const scale_t *>(IS_K ? a.cache.k_scale : a.cache.v_scale);
    const int lane = threadIdx.x & 31, w = (threadIdx.x >> 5) - (IS_K ? CT_K_WARP : CT_V_WARP);
    const int sub = lane / LR, c = lane % LR;
    const int32_t *table = a.cache.table + u.b * a.cache.ts0 + u.hk * a.cache.ts1;
    uint4 x[NI];
    uint32_t sw[LK], there = 0u;  // scales of this lane's rows; bit i: the row of x[i] is there
    CachePlace place[LK];         // of this lane's keys in the next tile to load
    auto look_up = [&](int j) {
#pragma unroll
        for (int k = 0; k < LK; ++k) {
            const int q = k * 32 + lane, row = (q / RPI * NW + w) * RPI + q % RPI;  // this warp's q-th row
            const int key = key0 + j * BN + row;
            place[k].open(a.cache, table, key, j < n_tiles && row < BN && key < key_end);
        }
    };
    // Rows that are not there read row 0 of the pool, and count as zeros by their factor: no
    // branch parts the loads.
    auto load = [&]() {
        int rows[LK];
#pragma unroll
        for (int k = 0; k < LK; ++k) rows[k] = place[k].row(a.cache, u.hk, a.status);
        there = 0u;
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            const int r = __shfl_sync(0xffffffffu, rows[i * RPI / 32], (i * RPI + sub) & 31);
            there |= (r >= 0 ? 1u : 0u) << i;
            x[i] = load_codes16(codes + (int64_t)max(r, 0) * D + c * 16);
        }
#pragma unroll
        for (int k = 0; k < LK; ++k) sw[k] = (uint32_t)__ldg(scales + max(rows[k], 0));
    };
    uint32_t present = 0u;  // `there` of the tile that is being converted
    // codes of x[i] -> eight bf16 pairs; TWO: exponents above 7 somewhere in the warp's rows
    auto convert = [&](auto two, int i, uint32_t byte, uint32_t (&y)[8]) {
        const uint32_t some = decltype(two)::value ? scale_bits(byte) * 0x10001u : scale_pair(byte);
        const uint32_t f = (present >> i) & 1u ? some : 0u;
        codes_of_word(x[i].x, f, y[0], y[1]);
        codes_of_word(x[i].y, f, y[2], y[3]);
        codes_of_word(x[i].z, f, y[4], y[5]);
        codes_of_word(x[i].w, f, y[6], y[7]);
        if (decltype(two)::value) {
            const uint32_t g = scale_rest_bits(byte) * 0x10001u;
#pragma unroll
            for (int k = 0; k < 8; ++k) y[k] = mul_bf16x2(y[k], g);
        }
    };
    // the upper half of a 128-element row's lanes store their two pieces in the other order, so
    // that the eight lanes of one access fall on all eight 16-byte bank groups
    const bool swap = D == 128 && c >= 4;
    auto store = [&](uint32_t tile, int i, const uint32_t (&y)[8]) {
        const int row = (i * NW + w) * RPI + sub;
        if (row < BN) {
            const uint32_t first[4] = {swap ? y[4] : y[0], swap ? y[5] : y[1], swap ? y[6] : y[2], swap ? y[7] : y[3]};
            const uint32_t second[4] = {swap ? y[0] : y[4], swap ? y[1] : y[5], swap ? y[2] : y[6], swap ? y[3] : y[7]};
            st_shared_v4(tile + swz<D>(row, 2 * c + (swap ? 1 : 0)), first);
            st_shared_v4(tile + swz<D>(row, 2 * c + (swap ? 0 : 1)), second);
        }
    };
    auto one_tile = [&](auto two, int j) -> bool {
        const int s = j % NS, use = j / NS;
        const uint32_t tile = sbase + (IS_K ? C::SMEM_K : C::SMEM_V) + s * C::TILE_BYTES;
        uint32_t byte[NI];
        present = there;
#pragma unroll
        for (int i = 0; i < NI; ++i)
            byte[i] = (__shfl_sync(0xffffffffu, sw[i * RPI / 32], (i * RPI + sub) & 31) >> (8 * (c / 2))) & 0xffu;
        if (use > 0 &&
            !__all_sync(0xffffffffu, wait_bar(IS_K ? bar.k_free(s) : bar.v_free(s), (use - 1) & 1, ctl)))
            return false;
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            uint32_t y[8];
            convert(two, i, byte[i], y);
            store(tile, i, y);
        }
        load();
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(IS_K ? bar.k_full(s) : bar.v_full(s));
        return true;
    };
    look_up(0);
    load();
    look_up(1);
    block_meets();
    if (*skip) return;
    for (int j = 0; j < n_tiles; ++j) {
        uint32_t top = sw[0];
#pragma unroll
        for (int k = 1; k < LK; ++k) top |= sw[k];
        const bool go = __any_sync(0xffffffffu, (top & SCALE_TOP_BITS) != 0u) ? one_tile(Yes{}, j) : one_tile(No{}, j);
        if (!go) return;
        look_up(j + 2);
    }
}

// O[128 x D] += P[128 x 128] V[128 x D], P in tensor memory (8 columns per 16 keys), V MN-major
template <int D>
__device__ __forceinline__ void issue_pv_tmem(uint32_t t_o, uint32_t t_p, uint64_t dv, bool accumulate)
{
    constexpr uint32_t idesc = idesc_bf16_f32(BM, D, true);
    if (elect_one()) {
#pragma unroll
        for (uint32_t kk = 0; kk < BN / 16; ++kk)
            mma_ts(t_o, t_p + 8 * kk, desc_add(dv, kk * 2048), idesc, (accumulate || kk > 0) ? 1u : 0u);
    }
    __syncwarp();
}

// The tensor-core schedule (one warp, one elected lane): see above.  With two query tiles
// (PAIR) buffer x is tile x's and takes every key tile; with one, buffer j & 1 takes key tile
// j, and a buffer's next S is two key tiles on.
template <int D, bool PAIR>
__device__ void chunk_mma(uint32_t sbase, uint32_t tmem, int n_tiles, const Ctl &ctl)
{
    using C = CCfg<D>;
    constexpr uint32_t idesc_s = idesc_bf16_f32(BM, BN, false);
    const CBars<D> bar{sbase + C::SMEM_BAR};
    const uint64_t dq = sdesc_sw128(sbase + C::SMEM_Q, 16, 1024), dk = sdesc_sw128(sbase + C::SMEM_K, 16, 1024);
    const uint64_t dv = sdesc_sw128(sbase + C::SMEM_V, Cfg<D>::BOX_BYTES, 1024);
    bool issued = false;
    // S of key tile j into buffer x (the K slot is free after its last reader)
    auto s_into = [&](int x, int j, bool last_reader) {
        const int sk = j % C::NSK;
        issue_s<D>(tmem + tcol_s(x), desc_add(dq, PAIR ? x * C::TILE_BYTES : 0), desc_add(dk, sk * C::TILE_BYTES), idesc_s);
        commit_one(bar.s_full(x));
        if (last_reader) commit_one(bar.k_free(sk));
        issued = true;
    };
    for (int x = 0; x < 2; ++x) {
        const int j = PAIR ? 0 : x;
        if (j >= n_tiles) break;
        if ((!PAIR || x == 0) && !__all_sync(0xffffffffu, wait_bar(bar.k_full(j % C::NSK), (j / C::NSK) & 1, ctl))) goto done;
        tc_fence_after();
        s_into(x, j, !PAIR || x == 1);
    }
    for (int j = 0; j < n_tiles; ++j) {
        const int sv = j % C::NSV, jn = PAIR ? j + 1 : j + 2;
        for (int i = 0; i < (PAIR ? 2 : 1); ++i) {
            const int x = PAIR ? i : j & 1;
            if (!__all_sync(0xffffffffu, wait_bar(bar.p_full(x), (PAIR ? j : j >> 1) & 1, ctl))) goto done;
            if (PAIR && D == 64 && jn < n_tiles) {  // P has left S's columns: the next S goes first
                if (i == 0 && !__all_sync(0xffffffffu, wait_bar(bar.k_full(jn % C::NSK), (jn / C::NSK) & 1, ctl))) goto done;
                tc_fence_after();
                s_into(x, jn, i == 1);
            }
            if (i == 0 && !__all_sync(0xffffffffu, wait_bar(bar.v_full(sv), (j / C::NSV) & 1, ctl))) goto done;
            tc_fence_after();
            issue_pv_tmem<D>(tmem + tcol_o(PAIR ? x : 0), tmem + tcol_p<D>(x), desc_add(dv, sv * C::TILE_BYTES), j > 0);
            if (!PAIR) commit_one(bar.pv_done());
            else if (D == 64) commit_one(bar.pv_x(x));
            if (!PAIR || i == 1) {
                commit_one(bar.v_free(sv));
                if (j == n_tiles - 1) commit_one(bar.o_final());
            }
            if (jn < n_tiles && !(PAIR && D == 64)) {
                if (i == 0 && !__all_sync(0xffffffffu, wait_bar(bar.k_full(jn % C::NSK), (jn / C::NSK) & 1, ctl))) goto done;
                tc_fence_after();
                s_into(x, jn, !PAIR || i == 1);
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

template <bool MASK>
__device__ __forceinline__ void hide_columns(int nv, uint32_t (&r)[32])
{
    if (MASK && nv < 32) {
#pragma unroll
        for (int i = 0; i < 32; ++i)
            if (i >= nv) r[i] = __float_as_uint(-INFINITY);
    }
}

// A chunk of 32 columns has outgrown the running max m of some row: the row takes the chunk's
// maximum, and what stands against the old one shrinks by alpha (by 2^-19 or more, or all of it is
// 0): O, the row sum and the probabilities of the tile's chunks before, whose second rounding
// to bf16 is 2^-8 of that little.
template <int D>
__device__ __noinline__ void outgrown(uint32_t t_p, uint32_t t_o, int chunks, bool has_o, float alpha)
{
    uint32_t r[16];
    tmem_wait_st();  // the probabilities just stored are read again
#pragma unroll 1
    for (int c = 0; c < chunks; ++c) {
        tmem_ld16_wait(t_p + c * 16, r);
#pragma unroll
        for (int i = 0; i < 16; ++i)
            r[i] = pack_bf16x2(__uint_as_float(r[i] << 16) * alpha, __uint_as_float(r[i] & 0xffff0000u) * alpha);
        tmem_st16(t_p + c * 16, r);
    }
    if (!has_o) return;
#pragma unroll 1
    for (int c = 0; c < D; c += 16) {
        tmem_ld16_wait(t_o + c, r);
#pragma unroll
        for (int i = 0; i < 16; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) * alpha);
        tmem_st16(t_o + c, r);
    }
}

// One key tile of the online softmax for this thread's row (thread = TMEM lane) that sees the
// columns [0, nv) of it (MASK; all of them otherwise), 32 columns at a time:
// P = exp2(S * scale * log2e - m) as bf16 (the type of the product with V; the row sums are of the
// fp32 numbers) over the columns that S has been read from.  The first
// tile takes its row maximum before; later a row keeps m until a chunk's probabilities sum to
// more than 2^GROWTH (one above it, or enough of them).  m is -inf, and the row's
// probabilities are 0, until the row has seen a key.  P V of the key tile before has to be
// complete before O is rescaled (one-tile units: pv_done), and with P in columns of its own before
// the first of P is stored (pv_first); otherwise S of this tile came after it.
template <int D, bool MASK>
__device__ __forceinline__ bool chunk_softmax_tile(uint32_t t_s, uint32_t t_p, uint32_t t_o, int nv, float sl2,
                                                   float &m_used, float &l, int j, uint32_t pv_done, uint32_t pv_first,
                                                   const Ctl &ctl)
{
    uint32_t ra[32], rb[32];  // the load of chunk c + 1 is in flight while chunk c is used
    if (j == 0) {
        float mx = -INFINITY;
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
            tmem_ld32(t_s + c * 32, ra);
            tmem_wait_ld_regs(ra);
            hide_columns<MASK>(nv - c * 32, ra);
            mx = fmaxf(mx, max32(ra));
        }
        m_used = mx * sl2;
    }
    float neg_m = m_used == -INFINITY ? 0.f : -m_used;
    constexpr float limit = (float)(1 << (int)GROWTH);
    bool ok = true;
    auto chunk = [&](int c, uint32_t(&cur)[32], uint32_t(&nxt)[32], bool more) {
        tmem_wait_ld_regs(cur);
        if (more) tmem_ld32(t_s + (c + 1) * 32, nxt);
        hide_columns<MASK>(nv - c * 32, cur);
        uint32_t pk[16];
        Acc8 acc;
        exp_chunk(cur, sl2, neg_m, pk, acc);
        float lt = sum8(acc);
        if (D == 64 && c == 0 && pv_first) {
            ok = __all_sync(0xffffffffu, wait_bar(pv_first, (j - 1) & 1, ctl));
            tc_fence_after();
        }
        const bool grow = lt > limit || (MASK && m_used == -INFINITY && c * 32 < nv);
        if (__any_sync(0xffffffffu, grow)) {
            const float m_new = grow ? fmaxf(m_used, max32(cur) * sl2) : m_used;
            const float alpha = m_used == -INFINITY ? 0.f : ex2_approx(m_used - m_new);
            if (j > 0 && pv_done) {
                ok = ok && __all_sync(0xffffffffu, wait_bar(pv_done, (j - 1) & 1, ctl));
                tc_fence_after();
            }
            if (more) tmem_wait_ld_regs(nxt);
            outgrown<D>(t_p, t_o, c, j > 0, alpha);
            l *= alpha;
            m_used = m_new;
            neg_m = m_used == -INFINITY ? 0.f : -m_used;
            Acc8 again;
            exp_chunk(cur, sl2, neg_m, pk, again);
            lt = sum8(again);
        }
        l += lt;
        tmem_st16(t_p + c * 16, pk);
    };
    tmem_ld32(t_s, ra);
#pragma unroll 1
    for (int c = 0; c < 4; c += 2) {
        chunk(c, ra, rb, true);
        chunk(c + 1, rb, ra, c == 0);
    }
    return ok;
}

// Queries, softmax and epilogue of query tile x, one thread per row.
template <int D, bool DEAL>
__device__ void chunk_softmax_role(const ChunkArgs &a, const Unit &u, uint8_t *smem, uint32_t sbase,
                                   const volatile uint32_t *tmem_slot, const volatile int32_t *skip, int x, int key0,
                                   int n_tiles, bool one_tile, const Ctl &ctl)
{
    using C = CCfg<D>;
    constexpr int LR = D / 8;     // lanes per 16-byte-pieced row
    constexpr int RPI = 32 / LR;  // rows per access of a warp
    const CBars<D> bar{sbase + C::SMEM_BAR};
    volatile int32_t *epi_ok = reinterpret_cast<volatile int32_t *>(smem + C::SMEM_BAR + 160) + 4 * x;
    const volatile int32_t *ranges_sh = reinterpret_cast<const volatile int32_t *>(smem + C::SMEM_BAR + 252);
    const int row = threadIdx.x & 127, lane = threadIdx.x & 31, warp = (threadIdx.x >> 5) & 3;
    const int tile_row0 = u.row0 + x * BM;
    const uint32_t s_tile = sbase + C::SMEM_Q + x * C::TILE_BYTES;
    // fp32 rows of a partial result: twice a tile's bytes, in the query tiles' and K slots' place,
    // which nothing reads any more after the last product
    const uint32_t s_part = sbase + C::SMEM_Q + x * 2 * C::TILE_BYTES;
    static_assert(C::SMEM_V >= 4 * C::TILE_BYTES, "two tiles of fp32 rows end before the V slots");
    // This warp's 32 query rows, whole rows at a time, all under way at once.  (What a CTA does
    // once is kept in short loops: unrolled, it ran at the rate that its instructions came in.)
    {
        const RowWalk w(a, u, tile_row0 + warp * 32 + lane / LR);
        const uint16_t *q = a.q + u.b * a.qs[0] + (lane % LR) * 8;
        w.each<RPI>(a, u, a.qs[1], a.qs[2], [&](int i, int64_t at, bool there) {
            cp_async16(s_tile + swz<D>(warp * 32 + i * RPI + lane / LR, lane % LR), q + at, there);
        });
    }
    cp_async_wait_all();
    fence_proxy_async_smem();  // before the block meets: Q is there for the tensor cores after it
    block_meets();
    if (*skip) return;
    const uint32_t tmem = *tmem_slot;
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
        if (!__all_sync(0xffffffffu, wait_bar(bar.s_full(xb), par, ctl))) {
            alive = false;
            break;
        }
        tc_fence_after();
        const uint32_t t_p = lane_base + tcol_p<D>(xb);
        const uint32_t pvw = one_tile ? bar.pv_done() : 0u;
        const uint32_t pvf = D == 64 && !one_tile && j > 0 ? bar.pv_x(x) : 0u;
        const bool whole = lim_warp >= (j + 1) * BN;
        const bool ok = whole ? chunk_softmax_tile<D, false>(t_s, t_p, t_o, BN, a.scale_log2, m_used, l, j, pvw, pvf, ctl)
                              : chunk_softmax_tile<D, true>(t_s, t_p, t_o, lim - j * BN, a.scale_log2, m_used, l, j, pvw,
                                                            pvf, ctl);
        if (!ok) {
            alive = false;
            break;
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0 && !((a.debug_flags & SFA_DEBUG_STALL_SOFTMAX) && j == 0)) mbar_arrive(bar.p_full(xb));
    }

    bool have = alive;
    if (have && n_tiles > 0) have = __all_sync(0xffffffffu, wait_bar(bar.o_final(), 0, ctl));
    if (lane == 0) epi_ok[warp] = have ? 1 : 0;
    named_bar_sync(1 + x, BM);
    if (!(epi_ok[0] && epi_ok[1] && epi_ok[2] && epi_ok[3])) return;  // uniform over the tile's warps
    // (a NaN, from a query that holds one, stays a NaN)
    const float inv_l = l != 0.f ? 1.f / l : 0.f;
    const float lse2 = l != 0.f ? m_used + log2f(l) : -INFINITY;
    const bool there = r < u.n_rows;
    const int64_t part_rows = (int64_t)a.B * a.H * a.Lq;
    if (n_tiles > 0) tc_fence_after();
#pragma unroll 1
    for (int c = 0; c < D / 32; ++c) {
        uint32_t o[32];
        if (n_tiles > 0) {
            tmem_ld32(t_o + c * 32, o);
            tmem_wait_ld_regs(o);
        } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = 0u;
        }
        if (a.n_split > 1) {  // fp32 rows, 16-byte pieces turned by the row against bank conflicts
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                const uint32_t y[4] = {__float_as_uint(__uint_as_float(o[4 * q]) * inv_l),
                                       __float_as_uint(__uint_as_float(o[4 * q + 1]) * inv_l),
                                       __float_as_uint(__uint_as_float(o[4 * q + 2]) * inv_l),
                                       __float_as_uint(__uint_as_float(o[4 * q + 3]) * inv_l)};
                st_shared_v4(s_part + row * D * 4 + (((c * 8 + q) ^ (row & 7)) << 4), y);
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
        if (a.n_split > 1) put_part_lse<DEAL>(a, u.split, DEAL ? *ranges_sh : 0, row_id(a, u, r), lse2);
        else a.lse[row_id(a, u, r)] = lse2 * 0.69314718055994530942f;
    }
    __syncwarp();  // a warp stores the 32 rows that its lanes have staged, whole rows at a time
    if (a.n_split > 1) {
        constexpr int PL = D / 4, PR = 32 / PL;  // lanes per fp32 row, rows per access
        const RowWalk w(a, u, tile_row0 + warp * 32 + lane / PL);
        float *dst = a.part_o + (u.split * part_rows + (int64_t)u.b * a.H * a.Lq) * D + (lane % PL) * 4;
        RowOut<float> rows(dst);
        w.each<PR>(a, u, (int64_t)a.Lq * D, D, [&](int i, int64_t at, bool on) {
            const int rr = warp * 32 + i * PR + lane / PL;
            rows.put(i, lds16(s_part + rr * D * 4 + (((lane % PL) ^ (rr & 7)) << 4)), at, on);
        });
        return;
    }
    const RowWalk w(a, u, tile_row0 + warp * 32 + lane / LR);
    uint16_t *dst = a.o + u.b * a.os[0] + (lane % LR) * 8;
    RowOut<uint16_t> rows(dst);
    w.each<RPI>(a, u, a.os[1], a.os[2], [&](int i, int64_t at, bool on) {
        rows.put(i, lds16(s_tile + swz<D>(warp * 32 + i * RPI + lane / LR, lane % LR)), at, on);
    });
}

template <int D, bool DEAL>
__global__ void __launch_bounds__(CT_THREADS, 1) tile_attn_kernel(const __grid_constant__ ChunkArgs a)
{
    using C = CCfg<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = smem_u32(smem);
    volatile uint32_t *tmem_slot = reinterpret_cast<volatile uint32_t *>(smem + C::SMEM_BAR + 240);
    volatile int32_t *abort_flag = reinterpret_cast<volatile int32_t *>(smem + C::SMEM_BAR + 244);
    volatile int32_t *skip = reinterpret_cast<volatile int32_t *>(smem + C::SMEM_BAR + 248);
    const int warp = threadIdx.x >> 5;
    if (a.n_split > 1) pdl_launch_dependents();
    const Unit u = open_unit<DEAL>(a, CT_ROWS, BN);
    if (u.bad && threadIdx.x == 0) report_status(a.status, SFA_ERR_BAD_SET);
    if (u.row0 >= u.n_rows) return;
    const int seen = row_limit(a, u, min(u.row0 + CT_ROWS, u.n_rows) - 1);
    const int all = (seen + BN - 1) / BN;
    const int ranges = n_ranges(u, all);
    if (u.split >= ranges) return skip_range<DEAL>(a, u, CT_ROWS);
    const int t0 = (int)((int64_t)all * u.split / ranges);
    const int n_tiles = (int)((int64_t)all * (u.split + 1) / ranges) - t0;
    const bool has_b = u.row0 + BM < u.n_rows;

    if (threadIdx.x == 0) {
        const CBars<D> bar{sbase + C::SMEM_BAR};
        for (int i = 0; i < CBars<D>::COUNT; ++i) mbar_init(sbase + C::SMEM_BAR + 8 * i, 1);
        for (int s = 0; s < C::NSK; ++s) mbar_init(bar.k_full(s), CT_K_WARPS);
        for (int s = 0; s < C::NSV; ++s) mbar_init(bar.v_full(s), CT_V_WARPS);
        mbar_init(bar.p_full(0), BM / 32);
        mbar_init(bar.p_full(1), BM / 32);
        *abort_flag = 0;
        if (DEAL) *reinterpret_cast<volatile int32_t *>(smem + C::SMEM_BAR + 252) = u.ranges;  // (not in a register until the end)
        // once a CTA has timed out, the ones that start later skip their work
        *skip = (a.status && *reinterpret_cast<volatile int32_t *>(a.status) == SFA_ERR_TIMEOUT) ? 1 : 0;
        fence_mbar_init();
    }
    if (warp == CT_MMA_WARP) {
        tmem_alloc(sbase + C::SMEM_BAR + 240, TM_COLS);
        tmem_relinquish();
    }
    const Ctl ctl{abort_flag, a.status, a.timeout_ns};

    if (warp == CT_MMA_WARP) {
        block_meets();
        if (n_tiles > 0 && !*skip) {
            if (has_b) chunk_mma<D, true>(sbase, *tmem_slot, n_tiles, ctl);
            else chunk_mma<D, false>(sbase, *tmem_slot, n_tiles, ctl);
        }
    } else if (warp >= CT_V_WARP) {
        convert_role<D, false>(a, u, sbase, t0 * BN, seen, n_tiles, skip, ctl);
    } else if (warp >= CT_K_WARP) {
        convert_role<D, true>(a, u, sbase, t0 * BN, seen, n_tiles, skip, ctl);
    } else if (warp < 4 || has_b) {
        chunk_softmax_role<D, DEAL>(a, u, smem, sbase, tmem_slot, skip, warp >> 2, t0 * BN, n_tiles, !has_b, ctl);
    } else {
        block_meets();
    }

    tc_fence_before();
    __syncthreads();
    if (warp == CT_MMA_WARP) {
        tc_fence_after();
        tmem_dealloc(*tmem_slot, TM_COLS);
    }
}

// ----------------------------------------------------------------- joining the ranges
// O = sum_s w_s O_s, w_s = 2^(L_s - L), L = log2 sum_s 2^(L_s), over the key ranges of a row.
// A warp owns a row: its lanes hold the ranges' L_s (so their loads and the sum take one
// round), then D / 32 elements each, several ranges' loads under way at a time.
constexpr int JOIN_THREADS = 128;
constexpr int MAX_SPLIT = 64;

template <int D>
__global__ void __launch_bounds__(JOIN_THREADS) join_kernel(const __grid_constant__ ChunkArgs a)
{
    pdl_wait();  // the ranges are written by the kernel before
    constexpr int E = D / 32;  // elements a lane
    const int64_t rows = (int64_t)a.B * a.H * a.Lq;
    const int64_t id = (int64_t)blockIdx.x * (JOIN_THREADS / 32) + (threadIdx.x >> 5);
    if (id >= rows) return;
    const int lane = threadIdx.x & 31;
    const uint32_t bh = (uint32_t)id / (uint32_t)a.Lq;
    const int i = (int)((uint32_t)id - bh * (uint32_t)a.Lq), b = (int)(bh / (uint32_t)a.H), h = (int)(bh - b * (uint32_t)a.H);
    if (a.q_lens && i >= __ldg(a.q_lens + b)) return;
    static_assert(MAX_SPLIT <= 64, "two ranges a lane");
    const float l0 = lane < a.n_split ? a.part_lse[lane * rows + id] : -INFINITY;
    const float l1 = lane + 32 < a.n_split ? a.part_lse[(lane + 32) * rows + id] : -INFINITY;
    float M = fmaxf(l0, l1);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    // a range that was not there, or that the row does not see, has L_s = -inf and weight 0
    const float w0 = l0 == -INFINITY ? 0.f : ex2_approx(l0 - M), w1 = l1 == -INFINITY ? 0.f : ex2_approx(l1 - M);
    float total = w0 + w1;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    float acc[E];
#pragma unroll
    for (int j = 0; j < E; ++j) acc[j] = 0.f;
    const float *src = a.part_o + id * D + lane * E;
    // (ranges behind the last that has anything are not gone through)
    const uint32_t on0 = __ballot_sync(0xffffffffu, w0 != 0.f), on1 = __ballot_sync(0xffffffffu, w1 != 0.f);
    const int last = on1 ? 64 - __clz(on1) : 32 - __clz(on0);
    for (int s0 = 0; s0 < last; s0 += 8) {
        float x[8][E], w[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int s = s0 + k;
            w[k] = s < last ? __shfl_sync(0xffffffffu, s0 < 32 ? w0 : w1, s & 31) : 0.f;
#pragma unroll
            for (int j = 0; j < E; ++j) x[k][j] = 0.f;
            if (w[k] != 0.f) {  // (the partial O of a range with weight 0 need not be there)
                if (E == 4) {
                    const float4 v = *reinterpret_cast<const float4 *>(src + s * rows * D);
                    x[k][0] = v.x, x[k][1] = v.y, x[k][E - 2] = v.z, x[k][E - 1] = v.w;
                } else {
                    const float2 v = *reinterpret_cast<const float2 *>(src + s * rows * D);
                    x[k][0] = v.x, x[k][1] = v.y;
                }
            }
        }
#pragma unroll
        for (int k = 0; k < 8; ++k)
#pragma unroll
            for (int j = 0; j < E; ++j) acc[j] = fmaf(w[k], x[k][j], acc[j]);
    }
    const float inv = total != 0.f ? 1.f / total : 0.f;
    uint16_t *dst = a.o + b * a.os[0] + h * a.os[1] + i * a.os[2] + lane * E;
    if (E == 4)
        *reinterpret_cast<uint2 *>(dst) =
            make_uint2(pack_bf16x2(acc[0] * inv, acc[1] * inv), pack_bf16x2(acc[E - 2] * inv, acc[E - 1] * inv));
    else
        *reinterpret_cast<uint32_t *>(dst) = pack_bf16x2(acc[0] * inv, acc[1] * inv);
    if (lane == 0) a.lse[id] = total != 0.f ? (M + log2f(total)) * 0.69314718055994530942f : -INFINITY;
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
    if (!(d->scale > 0.f) || !std::isfinite(d->scale * 1.4426950408889634f)) return SFA_ERR_INVALID_ARG;
    if (d->len_stride[0] < 0 || d->len_stride[1] < 0) return SFA_ERR_INVALID_ARG;
    if ((int64_t)d->B * d->H * d->Lq >= ((int64_t)1 << 31)) return SFA_ERR_INVALID_ARG;
    return SFA_OK;
}

struct Plan {
    bool tiles;  // tile_attn_kernel, else rows_attn_kernel
    int row_tiles, n_split, range_len, target, even_split;
    int64_t ctas;
};

// Bytes of the ranges' partial results (fp32 O and LSE of every row, n_split times).
size_t part_bytes(const sfa_cache_attn_desc *d, int n_split)
{
    if (n_split == 1) return 0;
    const size_t rows = (size_t)d->B * d->H * d->Lq;
    return (n_split * rows * (d->d + 1) * sizeof(float) + 255) / 256 * 256;
}

constexpr size_t PART_BYTES_MAX = (size_t)512 << 20;  // that a plan asks for, at most
constexpr double PART_BYTES_L2 = 96e6;                // that stay in the L2 cache (126 MB) between the kernels
constexpr int FEW_ROWS = 32;
constexpr double DEALT_STEPS = 6.0;  // key steps a CTA, below which the lengths are not dealt out

// Which kernel.  Up to 32 query rows of a key head, 16 rows a CTA read the cache at most twice
// and win (12 heads x 4 sequences over 8192 tokens, d = 128: 24 rows 47 against 54 us, 32 rows 47
// against 54, 48 rows 64 against 54; 8 x 8 over 16384, d = 64: 32 rows 73 against 104, 48 rows
// 104 against 104), and beyond that while all its steps hardly fill the SMs once, where the tile
// kernel's start and end are most of its time (12 heads over 1560 tokens: 48 rows 13.7 against
// 14.8, 64 rows 15.7 against 14.9, 96 rows 18.3 against 15.3; 4 heads over 300 tokens, d = 64:
// 128 rows 7.5 against 10.7).
bool few_rows(const sfa_cache_attn_desc *d, int64_t rows, int64_t kv)
{
    if (d->debug_flags & SFA_DEBUG_CACHE_TILES) return false;
    if (d->debug_flags & SFA_DEBUG_CACHE_ROWS) return true;
    const int64_t units = (int64_t)d->B * d->H_kv * ((rows + FR_ROWS - 1) / FR_ROWS);
    return rows <= FEW_ROWS || 2 * units * ((kv + FR_KEYS - 1) / FR_KEYS) <= 3 * (int64_t)attn_sms() * FR_CTAS;
}

Plan plan_of(const sfa_cache_attn_desc *d, const sfa_cache *c)
{
    Plan p;
    const int64_t rows = (int64_t)d->Lq * (d->H / d->H_kv);
    int64_t kv = (int64_t)c->table_len * c->page_len;
    if (d->max_kv > 0 && d->max_kv < kv) kv = d->max_kv;
    p.tiles = !few_rows(d, rows, kv);
    const int tile_rows = p.tiles ? CT_ROWS : FR_ROWS, step_keys = p.tiles ? BN : FR_KEYS;
    p.row_tiles = (int)((rows + tile_rows - 1) / tile_rows);
    const int64_t units = (int64_t)d->B * d->H_kv * p.row_tiles;
    const int64_t steps = std::max<int64_t>(1, (kv + step_keys - 1) / step_keys);
    // The number of ranges per unit, by the steps that the launch takes: a range takes its own
    // steps and a fixed start and end, the join of k ranges a little, and partial results beyond
    // the L2 cache go out to memory and come back (a step is some 2.7 us, 2.0 at d = 64).  The lengths are on
    // the device, so the mean of two cases is taken: all caches as long as the bound (whole
    // waves of equal ranges), and lengths spread between half of it and all of it (three
    // quarters of the ranges, which then even out but for the last one's end).  Measured, one
    // token, 96 units of 128 steps, k = 3, 6, 9, 12, 18: 99, 111, 92, 101, 101 us at one
    // length and 94, 100, 86, 87, 82 at uneven ones; 32 units, k = 9, 13, 18: 42, 37, 46 and 40, 37, 34.
    // Many rows are seldom worth their partial results.  d = 128, k = 1, 2, 3, ms at one length and
    // at uneven ones: 64 heads on 8, 25600 rows over 65536, 58.3, 61.5, 62.2 and 43.7, 46.0, 47.0 (1.69 GB of
    // workspace for k = 2); 12 heads, 16384 over 8192, 1.03, 1.12, 1.15 and 0.74, 0.92, 0.92, over 65536
    // 7.9, 7.5, 7.3 and 5.6, 5.6, 5.5; 4680 over 20280, 0.85, 0.87, 0.78 and 0.70, 0.60, 0.63.  Without
    // the bytes' term the first two of these took k = 2; with all bytes in it, those that stay in L2 too,
    // 1560 over 8192, 12 heads on 4, d = 64, took 3 ranges, not 5, and 107 us instead of 98.  Beyond
    // PART_BYTES_MAX, where k = 1 needs no memory at all, ranges gain 5 % at most (12 heads, 25600
    // over 65536: 11.3 and 11.9).
    const double slots = (double)attn_sms() * (p.tiles ? 1 : FR_CTAS);
    const double fixed = p.tiles ? 5.0 : 2.0;
    const double step_bytes = d->d == 128 ? 17.5e6 : 13e6;  // of HBM traffic in the time of a step
    double best = 1e300;
    p.n_split = 1;
    for (int64_t k = 1; k <= MAX_SPLIT && k <= steps; ++k) {
        if (part_bytes(d, (int)k) > PART_BYTES_MAX) break;
        const double piece = (double)((steps + k - 1) / k) + fixed, waves = units * k / slots;
        const double even = std::ceil(waves) * piece;
        const double uneven = waves <= 1.0 ? piece : (0.75 * waves + 0.5) * piece;
        const double out = std::max(0.0, (double)part_bytes(d, (int)k) - PART_BYTES_L2);
        const double join = k > 1 ? 1.5 + 0.05 * k + 2.0 * out / step_bytes : 0.0;
        const double cost = 0.5 * (even + uneven) + join;
        if (cost < best) {
            best = cost;
            p.n_split = (int)k;
        }
    }
    p.range_len = (int)std::min<int64_t>((steps + p.n_split - 1) / p.n_split, 1 << 30);
    // Uneven caches are better cut by their own lengths, into as many ranges as start at once
    // (`deal`), while that leaves a unit several ranges (64 units, many rows: 36.9 us by the bound
    // and 39.0 by the lengths) and a range enough steps (few rows, cut by
    // the bound and by the lengths: five waves and 8 steps, 32 x 8 caches of 8192, 104 and 116 us; one
    // wave and 5 steps, 4 x 12 of 8192, d = 64, 21.2 and 23.3).  n_split, the ranges that there is
    // room for, is then twice the mean number of a unit, so that lengths up to twice the mean have
    // ranges like the others; with many rows, whose partial results are larger, 1.5 times (twice:
    // 59.4 for 57.4 us at 12 equal caches of 20280, 200 rows).
    p.target = 0;
    p.even_split = p.n_split;
    p.ctas = units * p.n_split;
    const bool lengths = d->B > 1 || (d->H_kv > 1 && d->len_stride[1] != 0);  // more than one
    const bool dealt = lengths && (p.tiles ? p.n_split > 1 && 3.0 * units <= slots
                                           : 4.0 * units <= slots && 0.75 * units * steps >= DEALT_STEPS * slots);
    if (dealt && (int64_t)d->B * d->H_kv <= MAX_DEALT) {
        p.target = (int)slots;
        const int64_t mean = (p.target + units - 1) / units, room = p.tiles ? (3 * mean + 1) / 2 : 2 * mean;
        p.n_split = (int)std::max<int64_t>(std::min<int64_t>(std::min<int64_t>(MAX_SPLIT, steps), room), p.even_split);
        p.ctas = std::max<int64_t>(p.target, units * p.even_split);
    }
    return p;
}

template <int D, bool DEAL>
sfa_status launch_tiles(const ChunkArgs &a, unsigned grid, cudaStream_t s)
{
    if (cudaFuncSetAttribute(tile_attn_kernel<D, DEAL>, cudaFuncAttributeMaxDynamicSharedMemorySize, CCfg<D>::SMEM_BYTES) !=
        cudaSuccess)
        return SFA_ERR_CUDA;
    tile_attn_kernel<D, DEAL><<<grid, CT_THREADS, CCfg<D>::SMEM_BYTES, s>>>(a);
    return launch_status();
}

template <int D>
sfa_status launch_tiles(const ChunkArgs &a, unsigned grid, cudaStream_t s)
{
    return a.target ? launch_tiles<D, true>(a, grid, s) : launch_tiles<D, false>(a, grid, s);
}

typedef CUresult (*EncodeFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *, const cuuint64_t *,
                             const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                             CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// A pool's codes as rows of d bytes, copied 16 rows at a time.
bool encode_pool(CUtensorMap *m, const void *codes, int d, int64_t rows)
{
    EncodeFn fn = reinterpret_cast<EncodeFn>(tensor_map_encoder());
    if (!fn) return false;
    const cuuint64_t dims[2] = {(cuuint64_t)d, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)d};
    const cuuint32_t box[2] = {(cuuint32_t)d, 16}, ones[2] = {1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(codes), dims, strides, box, ones,
              CU_TENSOR_MAP_INTERLEAVE_NONE, d == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, bool BULK>
sfa_status launch_rows_attn(const ChunkArgs &a, const CUtensorMap &tk, const CUtensorMap &tv, unsigned grid, cudaStream_t s)
{
    if (cudaFuncSetAttribute(rows_attn_kernel<D, BULK>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             FCfg<D>::SMEM_BYTES) != cudaSuccess)
        return SFA_ERR_CUDA;
    rows_attn_kernel<D, BULK><<<grid, FR_WARPS * 32, FCfg<D>::SMEM_BYTES, s>>>(tk, tv, a);
    return launch_status();
}

sfa_status launch_few_rows(const ChunkArgs &a, const sfa_cache *c, unsigned grid, cudaStream_t s)
{
    CUtensorMap tk = {}, tv = {};
    const bool bulk = c->page_len % 16 == 0 && reinterpret_cast<uintptr_t>(c->k_scale) % 16 == 0 &&
                      reinterpret_cast<uintptr_t>(c->v_scale) % 16 == 0;
    if (bulk) {
        const int64_t rows = (int64_t)c->n_pages * c->heads * c->page_len;
        if (!encode_pool(&tk, c->k, c->d, rows) || !encode_pool(&tv, c->v, c->d, rows)) return SFA_ERR_CUDA;
        return c->d == 128 ? launch_rows_attn<128, true>(a, tk, tv, grid, s) : launch_rows_attn<64, true>(a, tk, tv, grid, s);
    }
    return c->d == 128 ? launch_rows_attn<128, false>(a, tk, tv, grid, s) : launch_rows_attn<64, false>(a, tk, tv, grid, s);
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
    if (!rows_stride_ok(d->q_stride, d->B, d->H, d->Lq) || !rows_stride_ok(d->o_stride, d->B, d->H, d->Lq) ||
        !in_place_ok(q, o, d->q_stride, d->o_stride, d->B, d->H, d->Lq))
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
    a.target = p.target;
    a.even_split = p.even_split;
    a.timeout_ns = (uint64_t)(d->timeout_us ? d->timeout_us : DEFAULT_TIMEOUT_US) * 1000;
    a.debug_flags = d->debug_flags;
    cudaStream_t s = as_cuda(stream);
    const unsigned grid = (unsigned)p.ctas;
    if (p.tiles) {
        st = d->d == 128 ? launch_tiles<128>(a, grid, s) : launch_tiles<64>(a, grid, s);
    } else {
        st = launch_few_rows(a, cache, grid, s);
    }
    if (st != SFA_OK || p.n_split == 1) return st;
    cudaLaunchConfig_t cfg = {};
    const int per_cta = JOIN_THREADS / 32;
    cfg.gridDim = dim3((unsigned)((rows + per_cta - 1) / per_cta));
    cfg.blockDim = dim3(JOIN_THREADS);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = d->d == 128 ? cudaLaunchKernelEx(&cfg, join_kernel<128>, a) : cudaLaunchKernelEx(&cfg, join_kernel<64>, a);
    return cuda_status(e);
}
