// kda_ssm_tc.cuh -- what the scan's tensor-core kernels share: chunk lookup and decays, the
// operand tiles and their loads, bf16 splitting, and the MMA forms.  Not part of the
// public ABI.
#pragma once

#include "kda_block.cuh"
#include "kda_tc.cuh"

namespace kda {
namespace {

constexpr int kTL = 128;          // chunk length of the tensor-core path
constexpr int kPT = 64;           // columns of a head that one CTA works on
constexpr int kSub = 16;          // rows that share a reference decay
constexpr float kLog2eTc = 1.4426950408889634f;
constexpr uint64_t kSsmWaitNs = 1000000000ull;

struct TcChunk {
    int64_t r0;
    int nr;
};
__device__ __forceinline__ bool tc_find_chunk(const SsmArgs &p, int64_t slot, TcChunk &c) {
    if (p.cu) {
        if (!p.ctrl->valid || slot >= p.ctrl->total_chunks) return false;
        const int n = upper_bound_minus_one(p.chunk_start, p.N + 1, (int)slot);
        const int s = p.cu[n] + kTL * ((int)slot - p.chunk_start[n]);
        c.r0 = s;
        c.nr = min(kTL, p.cu[n + 1] - s);
    } else {
        const int per = (p.T + kTL - 1) / kTL;
        const int seq = (int)(slot / per);
        const int k = (int)(slot % per);
        c.r0 = (int64_t)seq * p.T + (int64_t)k * kTL;
        c.nr = min(kTL, p.T - k * kTL);
    }
    return c.nr > 0;
}

// A barrier of the first `threads` threads of the block (id > 0).
__device__ __forceinline__ void bar_sync(int id, int threads) {
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// Sums of two floats: s + e exactly (Knuth), and hi + lo pairs.
__device__ __forceinline__ void pair_add(float &hi, float &lo, float bh, float bl) {
    const float s = __fadd_rn(hi, bh), v = __fsub_rn(s, hi);
    const float e = __fadd_rn(__fsub_rn(hi, __fsub_rn(s, v)), __fsub_rn(bh, v));
    const float l = __fadd_rn(__fadd_rn(lo, bl), e);
    hi = __fadd_rn(s, l);
    lo = __fsub_rn(l, __fsub_rn(hi, s));
}

// ------------------------------------------------------------------ operand tiles
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, bool take) {
    const uint32_t n = take ? 16u : 0u;  // 0: sixteen zero bytes
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() {
    asm volatile("cp.async.wait_all;" ::: "memory");
}

// A chunk state of one head and 64 columns lies in memory as the next kernel's operand:
// core-matrix tiles of [Ns][64] bf16, so that one bulk copy each brings it to shared memory.  hi
// and mid (2^-17 of the state) are what y, dB and dC are made of, rounded to bf16 themselves; with
// lo, in an array of its own, the three are the fp32 state to 2^-25, for the sums behind the
// fp32 gradients of A_log and dt_bias.  Byte offset of the 16-byte row of columns 8 g .. 8 g + 7
// of state row n in any tile:
__host__ __device__ __forceinline__ int64_t state_off(int n, int g) {
    return (int64_t)(n >> 3) * (kPT * 16) + g * 128 + (n & 7) * 16;
}
__host__ __device__ __forceinline__ int64_t state_tile_bytes(int Ns) { return (int64_t)Ns * kPT * 2; }
// Units: (slot, head, 64-column tile); a unit's state has two tiles.
__host__ __device__ __forceinline__ int tiles_of(int P) { return (P + kPT - 1) / kPT; }

// The shares of <E, S> that the reverse pass leaves per (slot, head): one per warp.
__host__ __device__ __forceinline__ int64_t ssm_tc_es_per(int Ns, int P) {
    return ((int64_t)tiles_of(P) * Ns * 8 + 127) / 128 * 4;
}

// What the chunk kernels know of a chunk's rows, per (slot, head) in the workspace: a + lo, the
// cumulative log2 decay as two floats; d, the step; fd = d 2^{ref - a} with ref the decay at
// the last row of the row's block of 16; w = d 2^{a_end - a}; and fi = 2^{a - first}, with first
// the decay at the block's first row.  For a row i past j's block, 2^{a_i - a_j} d_j =
// 2^{a_i - ref} fd_j = 2^{first - a_j} d_j fi_i: one exponential per row and block in place of
// one per element, and both factors are <= 1 however strong the decay.
struct RowDecays {
    float a[kTL], lo[kTL], d[kTL], fd[kTL], w[kTL], fi[kTL];
};

// x = hi + lo in bf16 pairs: x0, x1 to about 2^-17 of each.
__device__ __forceinline__ uint32_t pack_bf16(float x0, float x1) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x0, x1);
    return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ void split2(float x0, float x1, uint32_t &hi, uint32_t &lo) {
    hi = pack_bf16(x0, x1);
    lo = pack_bf16(x0 - __uint_as_float(hi << 16), x1 - __uint_as_float(hi & 0xffff0000u));
}
__device__ __forceinline__ void split2p(uint64_t x, uint32_t &hi, uint32_t &lo) {
    float x0, x1;
    unpack2(x, x0, x1);
    hi = pack_bf16(x0, x1);
    unpack2(sub2(x, pack2(hi << 16, hi & 0xffff0000u)), x0, x1);
    lo = pack_bf16(x0, x1);
}
// x = hi + mid + lo, to about 2^-25.
__device__ __forceinline__ void split3(float x0, float x1, uint32_t &hi, uint32_t &mid, uint32_t &lo) {
    hi = pack_bf16(x0, x1);
    const float r0 = x0 - __uint_as_float(hi << 16), r1 = x1 - __uint_as_float(hi & 0xffff0000u);
    split2(r0, r1, mid, lo);
}

// D (+)= A B with A's 128 rows in tensor memory: lane i holds row i, each 32-bit column two
// consecutive bf16 of K (eight columns per instruction).
__device__ __forceinline__ void mma_bf16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc,
                                            uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}
// `steps` products of K = 16, one after another (rolled: the kernels' warps run different code
// at the same time, and unrolled it would not fit the instruction cache; a product takes 57
// cycles or more).
__device__ __forceinline__ void mma_steps(uint32_t d_tmem, uint64_t a, uint32_t a_inc, uint64_t b,
                                          uint32_t b_inc, uint32_t idesc, int steps, uint32_t acc) {
#pragma unroll 1
    for (int k = 0; k < steps; ++k) {
        tc::mma_bf16(d_tmem, a, b, idesc, acc);
        a += a_inc;
        b += b_inc;
        acc = 1;
    }
}
__device__ __forceinline__ void tmem_st16_nowait(uint32_t taddr, const uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
        "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
        : "memory");
}
__device__ __forceinline__ void tmem_wait_st() {
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// Tensor memory for one CTA: allocated by warp 0, its address in *slot after the barrier.
__device__ __forceinline__ uint32_t tmem_open(uint32_t *slot, uint32_t cols) {
    if (threadIdx.x < 32) {
        tc::tmem_alloc(slot, cols);
        tc::tmem_relinquish();
    }
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    return *slot;
}
__device__ __forceinline__ void tmem_close(uint32_t taddr, uint32_t cols) {
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    if (threadIdx.x < 32) tc::tmem_dealloc(taddr, cols);
}

__device__ __forceinline__ void tmem_ld16_nowait(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
          "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tmem_wait_ld() {
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

// Waits of a kernel whose warps take different parts.  A wait that runs out (1 s) is reported
// and marks the CTA dead; from then on no wait waits and no product is issued, but every
// thread goes through the rest of its rounds, so that barriers match and the tensor memory
// is freed.
// The wait itself is the hardware's, for up to 20 us at a time: a warp that polled would take
// issue slots from the warps it waits for.
__device__ __forceinline__ bool suspended_wait(uint64_t *bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(tc::smem_addr(bar)), "r"(parity), "r"(20000u)
        : "memory");
    return ok != 0;
}
__device__ __forceinline__ bool wait_or_die(uint64_t *bar, uint32_t parity, volatile int *dead,
                                            int32_t *status) {
    if (suspended_wait(bar, parity)) return *dead == 0;
    const uint64_t t0 = tc::globaltimer_ns();
    while (!suspended_wait(bar, parity)) {
        if (*dead) return false;
        if (tc::globaltimer_ns() - t0 > kSsmWaitNs) {
            *dead = 1;
            report(status, KDA_DEVICE_TIMEOUT);
            return false;
        }
    }
    return *dead == 0;
}

}  // namespace
}  // namespace kda
