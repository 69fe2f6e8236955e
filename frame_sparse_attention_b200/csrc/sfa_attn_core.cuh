// What the attention kernels share: the query/key tile shapes and their shared-memory layout,
// bounded mbarrier waits, the S and P V products, and the pieces of the online softmax.
// (Included by translation units inside which everything here is private.)
#pragma once

#include <cstdint>

#include "sfa.h"
#include "sfa_ptx.cuh"

namespace sfa {
namespace {

constexpr int BM = 128;                 // query rows per tile = MMA M = TMEM lanes
constexpr int BN = 128;                 // keys per K/V tile (largest MMA N used)
constexpr float RESCALE_LIMIT = 256.0f;  // keep a stale row max while the tile's row sum against it stays <= 2^8
constexpr uint32_t DEFAULT_TIMEOUT_US = 2000000;  // 2 s; a healthy wait lasts microseconds
constexpr uint32_t DRAIN_TIMEOUT_US = 2000000;
constexpr uint32_t MAX_SPINS = 1u << 30;           // backstop should the timer not advance

// tensor-memory columns (512 allocated): S of tile A / B, O of tile A / B (fp32)
constexpr uint32_t TM_COLS = 512;
__host__ __device__ constexpr uint32_t tcol_s(int x) { return (uint32_t)x * 128; }
__host__ __device__ constexpr uint32_t tcol_o(int x) { return 256 + (uint32_t)x * 128; }

template <int D>
struct Cfg {
    static constexpr int KBOX = D / 64;                 // 128-byte swizzle boxes per row
    static constexpr int BOX_BYTES = 128 * 128;         // 128 rows x 64 bf16
    static constexpr int TILE_BYTES = BM * D * 2;       // one Q / K / V / O tile
    // K and V rings: a K slot frees once S of both query tiles is computed from it, a V
    // slot once P V of both is (d = 128 leaves room for one V slot only)
    static constexpr int NSK = 2;
    static constexpr int NSV = D == 128 ? 1 : 2;
    static constexpr int P_BYTES = BM * BN * 2;          // one bf16 probability tile
    static constexpr int SMEM_Q = 0;                      // Q tiles A and B
    static constexpr int SMEM_P = 2 * TILE_BYTES;         // P tiles A and B
    static constexpr int SMEM_K = SMEM_P + 2 * P_BYTES;
    static constexpr int SMEM_V = SMEM_K + NSK * TILE_BYTES;
    static constexpr int SMEM_BAR = SMEM_V + NSV * TILE_BYTES;
    static constexpr int SMEM_BYTES = SMEM_BAR + 256 + 1024;  // + barriers, + alignment slack
    static_assert(2 * NSK + 2 * NSV + 10 <= 20, "mbarriers must fit in 160 bytes");
    static_assert(SMEM_BYTES <= 232448, "shared memory per CTA");
};

// mbarrier slots (8 bytes each) at SMEM_BAR
template <int D>
struct Bars {
    uint32_t base;
    __device__ uint32_t k_full(int s) const { return base + 8 * s; }
    __device__ uint32_t k_free(int s) const { return base + 8 * (Cfg<D>::NSK + s); }
    __device__ uint32_t v_full(int s) const { return base + 8 * (2 * Cfg<D>::NSK + s); }
    __device__ uint32_t v_free(int s) const { return base + 8 * (2 * Cfg<D>::NSK + Cfg<D>::NSV + s); }
    __device__ uint32_t q_full() const { return base + 8 * (2 * Cfg<D>::NSK + 2 * Cfg<D>::NSV); }
    __device__ uint32_t s_full(int x) const { return q_full() + 8 + 8 * x; }   // S of query tile x in TMEM
    __device__ uint32_t p_full(int x) const { return q_full() + 24 + 8 * x; }  // P of query tile x in smem
    __device__ uint32_t o_final() const { return q_full() + 40; }              // after the last P V
    __device__ uint32_t drain() const { return q_full() + 48; }
    __device__ uint32_t pv_done() const { return q_full() + 56; }  // one-tile CTAs: a P V complete
    __device__ uint32_t pv_x(int x) const { return q_full() + 64 + 8 * x; }  // P V of query tile x complete
    static constexpr int COUNT = 2 * Cfg<D>::NSK + 2 * Cfg<D>::NSV + 10;
};

// ----------------------------------------------------------------- pipeline control
struct Ctl {
    volatile int32_t *abort;
    int32_t *status;
    uint64_t timeout_ns;
};

__device__ __forceinline__ uint64_t global_ns()
{
    uint64_t t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    return t;
}

__device__ __forceinline__ void report(int32_t *status, int32_t code)
{
    if (status) atomicCAS(status, 0, code);
}

// bounded wait for the phase of `bar` with parity `parity`; false on timeout or abort
__device__ __noinline__ bool wait_slow(uint32_t bar, uint32_t parity, const Ctl &c)
{
    const uint64_t t0 = global_ns();
    for (uint32_t spins = 1;; ++spins) {
        if (mbar_try_wait(bar, parity)) return true;
        if (*c.abort) return false;
        if ((spins & 63) == 0 && (global_ns() - t0 > c.timeout_ns || spins >= MAX_SPINS)) {
            *c.abort = 1;
            report(c.status, SFA_ERR_TIMEOUT);
            return false;
        }
    }
}

__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, const Ctl &c)
{
    return mbar_try_wait(bar, parity) || wait_slow(bar, parity, c);
}

// wait used only while draining after an abort: ignores the abort flag
__device__ __noinline__ void wait_drain(uint32_t bar, uint32_t parity)
{
    const uint64_t t0 = global_ns();
    for (uint32_t spins = 1; spins < MAX_SPINS; ++spins) {
        if (mbar_try_wait(bar, parity)) return;
        if ((spins & 63) == 0 && global_ns() - t0 > (uint64_t)DRAIN_TIMEOUT_US * 1000) return;
    }
}

// Smem descriptors are built once per CTA; an operand at byte offset `off` from a
// descriptor's base is that descriptor plus off >> 4 (the start address is the low 14
// bits, in 16-byte units; every operand here lies below 256 KB, so nothing carries).
__device__ __forceinline__ uint64_t desc_add(uint64_t desc, uint32_t off_bytes) { return desc + (off_bytes >> 4); }

template <int D>
__device__ __forceinline__ void issue_s(uint32_t t_s, uint64_t dq, uint64_t dk, uint32_t idesc)
{
    // S[128 x n] = Q[128 x D] K[n x D]^T, both K-major; one MMA per 16 elements of D:
    // +32 bytes inside a 128-byte swizzle row, the next 64 columns one box further on
    if (elect_one()) {
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t off = (kk >> 2) * Cfg<D>::BOX_BYTES + (kk & 3) * 32;
            mma_ss(t_s, desc_add(dq, off), desc_add(dk, off), idesc, kk > 0);
        }
    }
    __syncwarp();
}

template <int D>
__device__ __forceinline__ void issue_pv(uint32_t t_o, uint64_t dp, uint64_t dv, uint32_t n, bool accumulate)
{
    // O[128 x D] += P[128 x n] V[n x D]; P K-major in shared memory (like Q), V MN-major
    // (D contiguous): 8-key groups 1024 B apart, 64-wide D blocks one box apart
    constexpr uint32_t idesc = idesc_bf16_f32(BM, D, true);
    const uint32_t steps = n >> 4;
    if (elect_one()) {
#pragma unroll
        for (uint32_t kk = 0; kk < 8; ++kk)
            if (kk < steps)
                mma_ss(t_o, desc_add(dp, (kk >> 2) * Cfg<D>::BOX_BYTES + (kk & 3) * 32), desc_add(dv, kk * 2048),
                       idesc, (accumulate || kk > 0) ? 1u : 0u);
    }
    __syncwarp();
}

// tcgen05.commit from one elected lane of the (converged) MMA warp
__device__ __forceinline__ void commit_one(uint32_t bar)
{
    if (elect_one()) tc_commit(bar);
    __syncwarp();
}

// Max of 32 values with 3-input max in a tree (depth 4).
__device__ __forceinline__ float max32(const uint32_t (&r)[32])
{
    float t[11];
#pragma unroll
    for (int k = 0; k < 10; ++k)
        t[k] = fmax3(__uint_as_float(r[3 * k]), __uint_as_float(r[3 * k + 1]), __uint_as_float(r[3 * k + 2]));
    t[10] = fmaxf(__uint_as_float(r[30]), __uint_as_float(r[31]));
    const float u0 = fmax3(t[0], t[1], t[2]), u1 = fmax3(t[3], t[4], t[5]), u2 = fmax3(t[6], t[7], t[8]);
    return fmax3(fmax3(u0, u1, u2), t[9], t[10]);
}

// Eight fp32 partial row sums kept as four pairs, each pair added with one two-lane
// instruction (every lane rounds like a scalar fp32 add, so the sums are those of eight
// scalar accumulators).
struct Acc8 {
    uint64_t v[4] = {0, 0, 0, 0};
    __device__ __forceinline__ void add(int k, float a, float b)
    {
        asm("{\n\t.reg .b64 t;\n\tmov.b64 t, {%1, %2};\n\tadd.rn.f32x2 %0, %0, t;\n\t}"
            : "+l"(v[k])
            : "f"(a), "f"(b));
    }
    __device__ __forceinline__ float get(int i) const
    {
        return __uint_as_float((uint32_t)(v[i >> 1] >> ((i & 1) * 32)));
    }
};

// exp2(s * sl2 - m) of columns 32c..32c+31 -> bf16, stored into this thread's row of the
// P tile in shared memory (K-major, 128-byte swizzle: 64 keys per 16 KB box, 16-byte
// chunk k of row r at chunk position k ^ (r & 7)); row sum into acc
__device__ __forceinline__ void exp_store_chunk(const uint32_t (&r)[32], float sl2, float neg_m, uint32_t p_row,
                                                int row, int c, Acc8 &acc)
{
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        uint32_t pk[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int e = q * 8 + 2 * i;
            const float p0 = ex2_approx(fmaf(__uint_as_float(r[e]), sl2, neg_m));
            const float p1 = ex2_approx(fmaf(__uint_as_float(r[e + 1]), sl2, neg_m));
            acc.add(i & 3, p0, p1);
            pk[i] = pack_bf16x2(p0, p1);
        }
        const uint32_t chunk = (uint32_t)((c & 1) * 4 + q);
        st_shared_v4(p_row + (c >> 1) * 16384 + ((chunk ^ (uint32_t)(row & 7)) << 4), pk);
    }
}

// exp_store_chunk in two halves: the 16 bf16 pairs of the chunk are formed first and
// stored later, so a wait can sit between them
__device__ __forceinline__ void exp_chunk(const uint32_t (&r)[32], float sl2, float neg_m, uint32_t (&pk)[16],
                                          Acc8 &acc)
{
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const float p0 = ex2_approx(fmaf(__uint_as_float(r[2 * i]), sl2, neg_m));
        const float p1 = ex2_approx(fmaf(__uint_as_float(r[2 * i + 1]), sl2, neg_m));
        acc.add(i & 3, p0, p1);
        pk[i] = pack_bf16x2(p0, p1);
    }
}

__device__ __forceinline__ void store_chunk(const uint32_t (&pk)[16], uint32_t p_row, int row, int c)
{
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const uint32_t v[4] = {pk[4 * q], pk[4 * q + 1], pk[4 * q + 2], pk[4 * q + 3]};
        const uint32_t chunk = (uint32_t)((c & 1) * 4 + q);
        st_shared_v4(p_row + (c >> 1) * 16384 + ((chunk ^ (uint32_t)(row & 7)) << 4), v);
    }
}

__device__ __forceinline__ float sum8(const Acc8 &acc)
{
    return ((acc.get(0) + acc.get(1)) + (acc.get(2) + acc.get(3))) +
           ((acc.get(4) + acc.get(5)) + (acc.get(6) + acc.get(7)));
}

}  // namespace
}  // namespace sfa
