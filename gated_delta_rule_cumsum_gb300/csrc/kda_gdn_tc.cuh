// kda_gdn_tc.cuh -- what the gated delta rule's tensor-core kernels share.  Not part of the public
// ABI.
//
// bf16 inputs, K and V multiples of 8 up to 128; chunks of 128 rows, every product a tcgen05.mma
// with 128 rows and fp32 accumulation.  K and V are padded to 128 with zeros in the tiles; only
// whole groups of 16 contracted columns and of 32 value columns are worked on.
//
// Precision.  The inputs enter the products as they are (the norm is a factor of the row).  What the
// kernels make themselves is split into two bf16 parts, and two or three products add up in one
// accumulator: 2^-17 of each factor, so that the bf16 outputs are the exact ones rounded once.
#pragma once

#include <optional>

#include "kda_gdn.cuh"

namespace kda {
namespace {

constexpr int kGC = 128;                          // rows of a chunk
constexpr int kGD = 128;                          // padded K and V
constexpr uint32_t kTile = kGdnTile;              // bytes of a [128][128] bf16 tile
constexpr int kSV = 32;                           // value columns of a scan block
// Strides of a [128][128] core-matrix tile (kda_tc.cuh): 8 rows on, 8 columns on, in bytes; the
// descriptors' steps of 16 along the contracted side, in 16-byte units.  (With all rows of eight columns
// next to each other every kernel took 5 to 15% longer.)
constexpr uint32_t kRow8 = kGD * 16, kCol8 = 128;
constexpr uint32_t kStepK = 2 * kCol8 / 16, kStepMN = 2 * kRow8 / 16;

// A [128][128] tile as an operand whose rows are M or N (k-major), or the contracted side.
__device__ __forceinline__ uint64_t desc_k(const void *tile) { return tc::sdesc(tc::smem_addr(tile), kCol8, kRow8); }
__device__ __forceinline__ uint64_t desc_mn(const void *tile) { return tc::sdesc(tc::smem_addr(tile), kRow8, kCol8); }

// `steps` products of K = 16.  Eight, the most there are, unrolled: a product of 64 columns takes 48 cycles
// then, 58 in a loop.
__device__ __forceinline__ void gdn_mma(uint32_t d_tmem, uint64_t a, uint32_t a_inc, uint64_t b, uint32_t b_inc,
                                        uint32_t idesc, int steps, uint32_t acc) {
    if (steps == 8) {
#pragma unroll
        for (int k = 0; k < 8; ++k)
            tc::mma_bf16(d_tmem, a + (uint64_t)(k * a_inc), b + (uint64_t)(k * b_inc), idesc, k > 0 ? 1u : acc);
    } else {
        mma_steps(d_tmem, a, a_inc, b, b_inc, idesc, steps, acc);
    }
}

__device__ __forceinline__ uint32_t gtile(int r, int c) { return tc::tile_off(r, c, kGD); }

// The same of a tile of 64 columns (the scans' states and rows: 32 high and 32 low parts).
__device__ __forceinline__ uint64_t desc_mn64(const void *tile) { return tc::sdesc(tc::smem_addr(tile), 64 * 16, 128); }

// Eight values as bf16 parts: 16 bytes of the high and of the low tile.
__device__ __forceinline__ void split8(const float *x, uint4 &hi, uint4 &lo) {
    split2(x[0], x[1], hi.x, lo.x);
    split2(x[2], x[3], hi.y, lo.y);
    split2(x[4], x[5], hi.z, lo.z);
    split2(x[6], x[7], hi.w, lo.w);
}
__device__ __forceinline__ void bf16x8(const uint4 &u, float (&v)[8]) {
    load_vec<__nv_bfloat16, 8, true>(reinterpret_cast<const __nv_bfloat16 *>(&u), 8, v);
}

// Whether rows can be copied 16 bytes at a time.
inline bool rows16(const void *p, int64_t stride, int cols) { return aligned_to(p, 16) && stride % 8 == 0 && cols % 8 == 0; }

// 128 rows of bf16 into a tile by TH threads; rows past nr and columns past nc (a multiple of 8)
// are zeros.  Eight lanes take eight rows of one 16-byte column.  The copies are asynchronous
// where the rows start on 16-byte boundaries.
template <bool AL, int TH>
__device__ __forceinline__ void load_tile_rows(uint8_t *tile, const __nv_bfloat16 *src, int64_t stride, int nr, int nc,
                                               int tid) {
    constexpr int CPR = kGD / 8, IT = kGC * CPR / TH, STEP = TH / CPR;
    static_assert(STEP % 8 == 0 && IT * STEP == kGC, "whole groups of rows per round");
    const int c8 = (tid >> 3) % CPR, r0 = (tid >> 3) / CPR * 8 + (tid & 7);
    const uint32_t off = (uint32_t)((r0 >> 3) * kRow8 + c8 * kCol8 + (r0 & 7) * 16);
    const __nv_bfloat16 *s = src + r0 * stride + c8 * 8;
#pragma unroll
    for (int k = 0; k < IT; ++k) {
        const bool in = c8 * 8 < nc && r0 + k * STEP < nr;
        const uint32_t at = off + k * STEP / 8 * kRow8;
        if constexpr (AL) {
            cp_async16(tc::smem_addr(tile) + at, in ? s + k * STEP * stride : src, in);
        } else {
            alignas(16) __nv_bfloat16 v[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = in ? s[k * STEP * stride + j] : __float2bfloat16_rn(0.f);
            *reinterpret_cast<uint4 *>(tile + at) = *reinterpret_cast<const uint4 *>(v);
        }
    }
}

// What a chunk's grams are multiplied with: w[k] = 2^{a_i - a_j} rk_j for the 16 columns j of block J, 0
// past i.  Blocks wholly before the warp's rows take one exponential per row (GdnRows: fd), the
// two that hold its 32 rows one per element.
__device__ __forceinline__ void decays16(const GdnRows &rd, int i, int quad, int J, float ai, float li, float (&w)[16]) {
    if (J < 2 * quad) {
        const float t = ex2_ftz((ai - rd.a[16 * J + 15]) + (li - rd.lo[16 * J + 15]));
#pragma unroll
        for (int k = 0; k < 16; k += 4) {
            const float4 f = *reinterpret_cast<const float4 *>(rd.fd + 16 * J + k);
            w[k] = t * f.x; w[k + 1] = t * f.y; w[k + 2] = t * f.z; w[k + 3] = t * f.w;
        }
    } else if (J <= 2 * quad + 1) {
#pragma unroll
        for (int k = 0; k < 16; k += 4) {
            const float4 a = *reinterpret_cast<const float4 *>(rd.a + 16 * J + k);
            const float4 l = *reinterpret_cast<const float4 *>(rd.lo + 16 * J + k);
            const float4 r = *reinterpret_cast<const float4 *>(rd.rk + 16 * J + k);
            const int d = i - 16 * J - k;  // columns before i
            w[k] = d >= 0 ? ex2_ftz((ai - a.x) + (li - l.x)) * r.x : 0.f;
            w[k + 1] = d >= 1 ? ex2_ftz((ai - a.y) + (li - l.y)) * r.y : 0.f;
            w[k + 2] = d >= 2 ? ex2_ftz((ai - a.z) + (li - l.z)) * r.z : 0.f;
            w[k + 3] = d >= 3 ? ex2_ftz((ai - a.w) + (li - l.w)) * r.w : 0.f;
        }
    } else {
#pragma unroll
        for (int k = 0; k < 16; ++k) w[k] = 0.f;
    }
}
// A unit's rows into shared memory, by all threads.
__device__ __forceinline__ void load_rows_of(float *to, const GdnArgs &p, int64_t unit, int tid, int threads) {
    const float4 *from = reinterpret_cast<const float4 *>(p.rows + unit * kGdnRowArrays * kGC);
    for (int e = tid; e < kGdnRowArrays * kGC / 4; e += threads) reinterpret_cast<float4 *>(to)[e] = from[e];
}
// 32 bytes to memory in one store where the address allows it, as 16 bf16.
__device__ __forceinline__ void store16(__nv_bfloat16 *to, const float (&x)[16], int n, bool vec) {
    if (vec && n >= 16) {
        uint32_t u[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) u[k] = pack_bf16(x[2 * k], x[2 * k + 1]);
        asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(to), "r"(u[0]), "r"(u[1]), "r"(u[2]), "r"(u[3]),
                     "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7])
                     : "memory");
    } else {
#pragma unroll
        for (int k = 0; k < 16; ++k)
            if (k < n) to[k] = __float2bfloat16_rn(x[k]);
    }
}

// 128 rows of 16 bytes as fp32 [row][32 value columns] per scan block: float4 group g (of 8) of row r
// of value tile t, so that consecutive rows lie next to each other on both sides.
__device__ __forceinline__ int64_t wide_at(int t, int g, int r) { return ((int64_t)(t * 8 + g) * kGC + r) * 4; }

}  // namespace

cudaError_t launch_gdn_tc_fwd(const GdnArgs &a, cudaStream_t st);
// One of the library's own streams, for what runs beside a pass over chunks, and the events that order it.
struct GdnSide {
    cudaStream_t stream = nullptr;
    cudaEvent_t ev[4] = {};
    cudaEvent_t last = nullptr;    // of ev: behind all that the stream holds
    unsigned long long of = 0;     // the caller's stream that had it last
    bool taken = false;            // by a call that is enqueueing
    // `st` after all that the side stream holds
    cudaError_t join(int i, cudaStream_t st) {
        const cudaError_t e = cudaEventRecord(ev[i], stream);
        if (e == cudaSuccess) last = ev[i];
        return e != cudaSuccess ? e : cudaStreamWaitEvent(st, ev[i], 0);
    }
};
// A call's hold on a side stream that holds no other stream's work, for as long as the call enqueues; side is
// null where there is none, and the call then runs in one part.
class GdnSideHold {
  public:
    explicit GdnSideHold(cudaStream_t st);
    ~GdnSideHold();
    GdnSideHold(const GdnSideHold &) = delete;
    GdnSideHold &operator=(const GdnSideHold &) = delete;
    GdnSide *side = nullptr;
    cudaError_t error = cudaSuccess;
};
int gdn_cut(const GdnArgs &a, double unit_ns, double round_ns, int64_t least, cudaStream_t st);
// Measured: the whole card's time per unit of the prep and of the gradients, and a pass's round.
constexpr double kPrepNs = 82, kGradNs = 215, kRoundNs = 2150;
cudaError_t launch_gdn_tc_rscan(const GdnArgs &a, cudaStream_t st);
cudaError_t launch_gdn_tc_bwd(const GdnArgs &a, cudaStream_t st);

}  // namespace kda
