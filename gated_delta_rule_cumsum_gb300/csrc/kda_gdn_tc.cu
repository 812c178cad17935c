// kda_gdn_tc.cu -- the gated delta rule's forward on the tensor cores (see kda_gdn.cuh for the
// chunk form, kda_gdn_tc.cuh for tiles and precision).  Three kernels: each chunk's triangular
// inverse and what the state is multiplied with (W = M diag(beta c) K, U0 = M diag(beta) V), all
// chunks at once; the pass over a sequence's chunks, U = U0 - W S and S' = 2^{a_end} S + K^T diag(e)
// U; and the outputs, all chunks at once.
#include "kda_gdn_tc.cuh"

namespace kda {
namespace {

using bf16 = __nv_bfloat16;

// ------------------------------------------------------------------ prep
// M = (I + diag(beta) A)^-1 of a chunk: blocks of 16 rows by substitution in fp32, then merged (the
// lower left of a merged pair is -M22 (N21 M11)): to 32 and 64 rows with warp-level products, since a
// tcgen05.mma has 64 rows at least, of two tf32 parts each (2^-22), and the two halves of 64 rows with
// tcgen05 products.  W and U0 take M from tensor memory with its columns scaled, so that K and V enter as
// they were loaded.
// 8192 rows of 16 heads (1024 units, two blocks an SM): 83 us; 4 x 4096 rows of 32 heads 293 us.  A unit is a chain of
// some fifteen hand-overs; issue slots are 45% busy, HBM 29%.  Substitution in blocks of 8 in place of 16
// changed nothing.
constexpr int kPrepThreads = 256;
struct PrepSmem {
    uint8_t hi[kTile], lo[kTile];  // M's parts; the halves' fp32 blocks before (in lo)
    uint8_t x[kTile];              // K, then V
    float row[kGdnRowArrays * kGC];
    float fw[kGC];                 // beta c rk
    uint64_t done;
    uint32_t slot_addr;
    int dead;
};
// Element (r, c) of a 64 x 64 fp32 block: float4 groups permuted by row, so that a column of groups
// does not conflict.
__device__ __forceinline__ int blk(int r, int c) { return r * 64 + ((((c >> 2) ^ r) & 15) << 2) + (c & 3); }

// x as two tf32 parts.
__device__ __forceinline__ void tf32_parts(float x, uint32_t &hi, uint32_t &lo) {
    asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(hi) : "f"(x));
    asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(lo) : "f"(x - __uint_as_float(hi)));
}
__device__ __forceinline__ void mma_tf32(float (&d)[4], const uint32_t (&a)[4], const uint32_t (&b)[2]) {
    asm volatile(
        "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}
// d[n] = the product of the 16 x K block at (ar, ac) and the K x 8 NT block at (br, bc) of a 64 x 64 block,
// by a warp.
template <int K, int NT>
__device__ __forceinline__ void blk_product(const float *B, int ar, int ac, int br, int bc, float (&d)[NT][4]) {
    const int g = (threadIdx.x & 31) >> 2, t = threadIdx.x & 3;
#pragma unroll
    for (int n = 0; n < NT; ++n) d[n][0] = d[n][1] = d[n][2] = d[n][3] = 0.f;
#pragma unroll
    for (int k = 0; k < K; k += 8) {
        uint32_t ah[4], al[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
            tf32_parts(B[blk(ar + g + (e & 1) * 8, ac + k + t + (e >> 1) * 4)], ah[e], al[e]);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            uint32_t bh[2], bl[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) tf32_parts(B[blk(br + k + t + e * 4, bc + 8 * n + g)], bh[e], bl[e]);
            mma_tf32(d[n], al, bh);
            mma_tf32(d[n], ah, bl);
            mma_tf32(d[n], ah, bh);
        }
    }
}
template <int NT>
__device__ __forceinline__ void blk_put(float *B, int r, int c, const float (&d)[NT][4], float sign) {
    const int g = (threadIdx.x & 31) >> 2, t = threadIdx.x & 3;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e)
            *reinterpret_cast<float2 *>(B + blk(r + g + 8 * e, c + 8 * n + 2 * t)) =
                make_float2(sign * d[n][2 * e], sign * d[n][2 * e + 1]);
}

template <bool AL>
__global__ void __launch_bounds__(kPrepThreads, 2) gdn_tc_prep_kernel(GdnArgs p) {
    extern __shared__ __align__(1024) uint8_t raw_smem[];
    PrepSmem &s = *reinterpret_cast<PrepSmem *>(raw_smem);
    int slot, hv;
    gdn_unit(p, (int)blockIdx.x, slot, hv);
    const int64_t unit = (int64_t)slot * p.HV + hv;
    const int per = p.HV / p.H, h = hv / per;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, quad = warp & 3, hf = warp >> 2, i = quad * 32 + lane;
    GdnChunk c;
    if (!gdn_find_chunk(p, slot, c)) return;
    if (tid == 0) {
        tc::mbar_init(&s.done, 1);
        tc::mbar_fence_init();
        s.dead = 0;
    }
    const uint32_t tm = tmem_open(&s.slot_addr, 256);
    volatile int *dead = &s.dead;
    uint32_t phase = 0;
    auto all_done = [&]() {  // the products issued so far
        wait_or_die(&s.done, phase, dead, p.status);
        phase ^= 1;
        tc::tc_fence_after();
    };
    auto hand_over = [&]() {  // what the threads wrote to shared and tensor memory, to the products
        tc::fence_async_smem();
        tc::tc_fence_before();
        __syncthreads();
        tc::tc_fence_after();
    };
    load_tile_rows<AL, kPrepThreads>(s.x, static_cast<const bf16 *>(p.k) + c.r0 * p.k_stride + (int64_t)h * p.K, p.k_stride,
                                     c.nr, p.K, tid);
    load_rows_of(s.row, p, unit, tid, kPrepThreads);
    const bf16 *vrows = static_cast<const bf16 *>(p.v) + c.r0 * p.v_stride + (int64_t)hv * p.V;
    cp_async_wait_all();
    hand_over();
    const GdnRows rd(s.row, kGC);
    const int ksteps = (p.K + 15) / 16;
    if (tid == 0) {
        const uint64_t d = desc_k(s.x);
        gdn_mma(tm, d, kStepK, d, kStepK, tc::idesc_bf16(128, 128, false, false), ksteps, 0);
        tc::mma_commit(&s.done);
        if (hv % per == 0) {  // K's tile, for the kernels that follow
            tc::bulk_s2g(p.kt + ((int64_t)slot * p.H + h) * kTile, s.x, kTile);
            tc::bulk_commit();
        }
    }
    all_done();
    if (tid < kGC) s.fw[tid] = rd.b[tid] * rd.c[tid] * rd.rk[tid];
    // N = beta A: the diagonal halves as fp32 blocks, the lower left one in bf16 parts (the low part in
    // the high tile's free upper right quadrant: the low tile holds the blocks)
    float *D = reinterpret_cast<float *>(s.lo) + (i >> 6) * 64 * 64;
    if (i >= 64 || hf == 0) {
        const float f = rd.b[i] * rd.rk[i], ai = rd.a[i], li = rd.lo[i];
        const bool diag = (i >> 6) == hf;
#pragma unroll 1
        for (int J = 0; J < 4; ++J) {
            const int j0 = hf * 64 + J * 16;
            float v[16], w[16];
            tc::tmem_ld16(tc::tmem_at(tm, quad * 32, j0), v);
            decays16(rd, i, quad, j0 / 16, ai, li, w);
#pragma unroll
            for (int k = 0; k < 16; ++k) v[k] = j0 + k < i ? v[k] * (f * w[k]) : 0.f;
            if (diag) {
#pragma unroll
                for (int k = 0; k < 16; k += 4)
                    *reinterpret_cast<float4 *>(D + blk(i & 63, J * 16 + k)) = make_float4(v[k], v[k + 1], v[k + 2], v[k + 3]);
            } else {
#pragma unroll
                for (int k = 0; k < 16; k += 8) {
                    uint4 a, b;
                    split8(v + k, a, b);
                    *reinterpret_cast<uint4 *>(s.hi + gtile(i, j0 + k)) = a;
                    *reinterpret_cast<uint4 *>(s.hi + gtile(i - 64, 64 + j0 + k)) = b;
                }
            }
        }
    }
    tc::tc_fence_before();
    __syncthreads();
    float *H = reinterpret_cast<float *>(s.lo) + (warp >> 2) * 64 * 64;  // a half for four warps
    if ((warp & 3) < 2) {  // 32 rows for two of them: 16 x 16 blocks, a column per lane, and their merger
        const int b0 = (warp & 1) * 32, r0 = b0 + (lane & 16), col = lane & 15;
        float m[16];
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            float x[4] = {r == col ? 1.f : 0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int l = 0; l < r; l += 4) {
                const float4 n = *reinterpret_cast<const float4 *>(H + blk(r0 + r, r0 + l));
                x[0] = fmaf(-n.x, m[l], x[0]);
                if (l + 1 < r) x[1] = fmaf(-n.y, m[l + 1], x[1]);
                if (l + 2 < r) x[2] = fmaf(-n.z, m[l + 2], x[2]);
                if (l + 3 < r) x[3] = fmaf(-n.w, m[l + 3], x[3]);
            }
            m[r] = (x[0] + x[1]) + (x[2] + x[3]);
        }
        __syncwarp();
#pragma unroll
        for (int r = 0; r < 16; ++r) H[blk(r0 + r, r0 + col)] = m[r];
        __syncwarp();
        float d[2][4];
        blk_product<16>(H, b0 + 16, b0, b0, b0, d);
        __syncwarp();
        blk_put(H, b0 + 16, b0, d, 1.f);
        __syncwarp();
        blk_product<16>(H, b0 + 16, b0 + 16, b0 + 16, b0, d);
        __syncwarp();
        blk_put(H, b0 + 16, b0, d, -1.f);
    }
    bar_sync(1 + (warp >> 2), 128);
    {  // the two blocks of 32 of a half: 16 rows and 16 columns a warp
        const int r = 32 + (warp & 1) * 16, col = (warp >> 1 & 1) * 16;
        float d[2][4];
        blk_product<32>(H, r, 0, 0, col, d);
        bar_sync(1 + (warp >> 2), 128);
        blk_put(H, r, col, d, 1.f);
        bar_sync(1 + (warp >> 2), 128);
        blk_product<32>(H, r, 32, 32, col, d);
        bar_sync(1 + (warp >> 2), 128);
        blk_put(H, r, col, d, -1.f);
    }
    __syncthreads();
    {  // the halves' inverses into the tiles
        float v[32];
#pragma unroll
        for (int k = 0; k < 32; k += 4) {
            const float4 x = *reinterpret_cast<const float4 *>(D + blk(i & 63, hf * 32 + k));
            v[k] = x.x; v[k + 1] = x.y; v[k + 2] = x.z; v[k + 3] = x.w;
        }
        __syncthreads();
        const int col = (i & 64) + hf * 32;
#pragma unroll
        for (int k = 0; k < 32; k += 8) {
            uint4 a, b;
            split8(v + k, a, b);
            *reinterpret_cast<uint4 *>(s.hi + gtile(i, col + k)) = a;
            *reinterpret_cast<uint4 *>(s.lo + gtile(i, col + k)) = b;
        }
    }
    hand_over();
    constexpr uint32_t q21 = 8 * kRow8, q12 = 8 * kCol8, q22 = q21 + q12;  // the quadrants' offsets
    const uint32_t id64 = tc::idesc_bf16(64, 64, false, true);
    if (tid == 0 && !*dead) {  // X = N21 M11
        const uint64_t nh = desc_k(s.hi + q21), nl = desc_k(s.hi + q12), mh = desc_mn(s.hi), ml = desc_mn(s.lo);
        gdn_mma(tm, nh, kStepK, ml, kStepMN, id64, 4, 0);
        gdn_mma(tm, nl, kStepK, mh, kStepMN, id64, 4, 1);
        gdn_mma(tm, nh, kStepK, mh, kStepMN, id64, 4, 1);
        tc::mma_commit(&s.done);
    }
    all_done();
    // (a result of 64 rows: row r in lane r / 16 * 32 + r % 16)
    const int r64 = quad * 16 + lane, c64 = hf * 32;
    {
        float v[32];
        tc::tmem_ld32(tc::tmem_at(tm, quad * 32, c64), v);
        if (lane < 16) {
#pragma unroll
            for (int k = 0; k < 32; k += 8) {
                uint4 a, b;
                split8(v + k, a, b);
                *reinterpret_cast<uint4 *>(s.lo + gtile(r64, 64 + c64 + k)) = a;
                *reinterpret_cast<uint4 *>(s.lo + gtile(64 + r64, c64 + k)) = b;
            }
        }
    }
    hand_over();
    if (tid == 0 && !*dead) {  // M22 X
        const uint64_t xh = desc_mn(s.lo + q12), xl = desc_mn(s.lo + q21), mh = desc_k(s.hi + q22), ml = desc_k(s.lo + q22);
        gdn_mma(tm + 64, mh, kStepK, xl, kStepMN, id64, 4, 0);
        gdn_mma(tm + 64, ml, kStepK, xh, kStepMN, id64, 4, 1);
        gdn_mma(tm + 64, mh, kStepK, xh, kStepMN, id64, 4, 1);
        tc::mma_commit(&s.done);
    }
    all_done();
    {
        float v[32];
        tc::tmem_ld32(tc::tmem_at(tm, quad * 32, 64 + c64), v);
        if (lane < 16) {
            const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
            for (int k = 0; k < 32; ++k) v[k] = -v[k];
#pragma unroll
            for (int k = 0; k < 32; k += 8) {
                uint4 a, b;
                split8(v + k, a, b);
                *reinterpret_cast<uint4 *>(s.hi + gtile(64 + r64, c64 + k)) = a;
                *reinterpret_cast<uint4 *>(s.lo + gtile(64 + r64, c64 + k)) = b;
                *reinterpret_cast<uint4 *>(s.hi + gtile(r64, 64 + c64 + k)) = zero;
                *reinterpret_cast<uint4 *>(s.lo + gtile(r64, 64 + c64 + k)) = zero;
            }
        }
    }
    hand_over();
    if (tid == 0 && p.mt) {
        tc::bulk_s2g(p.mt + unit * 2 * (int64_t)kTile, s.hi, 2 * kTile);
        tc::bulk_commit();
    }
    // M with its columns scaled, in tensor memory: 64 columns of the high parts, 64 of the low
    const uint32_t A = tm, R = tm + 128;
    auto scaled = [&](const float *f) {
#pragma unroll 1
        for (int J = 0; J < 2; ++J) {
            const int j0 = hf * 64 + J * 32;
            uint32_t a[16], b[16];
#pragma unroll
            for (int k = 0; k < 32; k += 8) {
                float x[8], y[8];
                bf16x8(*reinterpret_cast<const uint4 *>(s.hi + gtile(i, j0 + k)), x);
                bf16x8(*reinterpret_cast<const uint4 *>(s.lo + gtile(i, j0 + k)), y);
                const float4 f0 = *reinterpret_cast<const float4 *>(f + j0 + k);
                const float4 f1 = *reinterpret_cast<const float4 *>(f + j0 + k + 4);
                const float fv[8] = {f0.x, f0.y, f0.z, f0.w, f1.x, f1.y, f1.z, f1.w};
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = (x[e] + y[e]) * fv[e];
                uint4 u, l;
                split8(x, u, l);
                a[k / 2] = u.x; a[k / 2 + 1] = u.y; a[k / 2 + 2] = u.z; a[k / 2 + 3] = u.w;
                b[k / 2] = l.x; b[k / 2 + 1] = l.y; b[k / 2 + 2] = l.z; b[k / 2 + 3] = l.w;
            }
            tmem_st16_nowait(tc::tmem_at(A, quad * 32, j0 / 2), a);
            tmem_st16_nowait(tc::tmem_at(A, quad * 32, 64 + j0 / 2), b);
        }
        tmem_wait_st();
    };
    auto product = [&](int cols) {
        const uint32_t id = tc::idesc_bf16(128, cols, false, true);
        uint64_t x = desc_mn(s.x);
#pragma unroll 1
        for (int k = 0; k < kGC / 16; ++k) {
            mma_bf16_ts(R, A + 64 + 8 * k, x, id, k > 0);
            mma_bf16_ts(R, A + 8 * k, x, id, 1);
            x += kStepMN;
        }
        tc::mma_commit(&s.done);
    };
    scaled(s.fw);
    hand_over();
    if (tid == 0 && !*dead) product(128);
    all_done();
    if (tid == 0) tc::bulk_wait_read0();  // K's tile has left x
    __syncthreads();
    load_tile_rows<AL, kPrepThreads>(s.x, vrows, p.v_stride, c.nr, p.V, tid);
    scaled(rd.b);
    uint8_t *wt = p.wt + unit * 2 * (int64_t)kTile;
#pragma unroll 1
    for (int J = 0; J < 2; ++J) {
        const int j0 = hf * 64 + J * 32;
        float v[32];
        tc::tmem_ld32(tc::tmem_at(R, quad * 32, j0), v);
#pragma unroll
        for (int k = 0; k < 32; k += 8) {
            uint4 a, b;
            split8(v + k, a, b);
            *reinterpret_cast<uint4 *>(wt + gtile(i, j0 + k)) = a;
            *reinterpret_cast<uint4 *>(wt + kTile + gtile(i, j0 + k)) = b;
        }
    }
    cp_async_wait_all();
    hand_over();
    const int cols = (p.V + kSV - 1) / kSV * kSV;
    if (tid == 0 && !*dead) product(cols);
    all_done();
    float *u0 = p.u0 + unit * kGC * kGD;
    for (int t = hf; t < cols / kSV; t += 2) {
        float v[32];
        tc::tmem_ld32(tc::tmem_at(R, quad * 32, t * kSV), v);
#pragma unroll
        for (int g = 0; g < 8; ++g)
            *reinterpret_cast<float4 *>(u0 + wide_at(t, g, i)) =
                make_float4(v[4 * g], v[4 * g + 1], v[4 * g + 2], v[4 * g + 3]);
    }
    if (tid == 0) tc::bulk_wait0();
    tmem_close(tm, 256);
}

// ------------------------------------------------------------------ the pass over chunks
// One block per (sequence, value head, 32 value columns).  Eight warps keep the state in registers
// (row = key, 16 columns a thread) and form the rows; one more fetches tiles and issues the products
// (a warp that did both would keep the others waiting for its rows).  A round is a chain: product with the
// state, rows, product with the rows, state; what does not belong to it (stores, the next rows' loads)
// stands behind each hand-over.  The two bf16 parts of a right
// operand stand side by side (64 columns), so that the left operand, which is what a product's time
// goes into, is read once for both.
//   forward  rows: U = U0 - W S;                  state: S = 2^{a_end} S + K^T (e rk U)
//   reverse  rows: dU = dU0 + e rk K E;           state: E = 2^{a_end} E + B0 - W^T dU
// The state's and the rows' tile is one: each is written when the product with the other is done.  W and K
// are fetched again as soon as the product that reads them is through, which leaves them the rest of the
// round; with one buffer each (BUFS), two blocks share an SM and fill each other's waits.  Where every block
// has an SM of its own the copies are two rounds ahead.
// Bound by the chain: 8192 rows of 16 heads (64 blocks, 64 rounds) 128 us forward and 139 in reverse, 2 us a round, of
// which the products take 0.6; 28 sequences of 32 heads (3584 blocks) 288 us, 4 x 4096 rows of 32 heads 213 and 273.
// Copies into L2 ahead of a round's own, in the reverse pass with one buffer: 312 us for those 273.
constexpr int kScanRows = 256, kScanThreads = kScanRows + 32;
template <int BUFS>
struct ScanSmem {
    uint8_t w[BUFS][2 * kTile], k[BUFS][kTile];
    uint8_t right[kGD * 64 * 2];
    uint64_t w_full[BUFS], k_full[BUFS], d1, d2;
    uint32_t slot_addr;
    int dead;
};
template <bool REV, int BUFS>
__global__ void __launch_bounds__(kScanThreads, 3 - BUFS) gdn_tc_scan_kernel(GdnArgs p) {
    extern __shared__ __align__(1024) uint8_t raw_smem[];
    ScanSmem<BUFS> &s = *reinterpret_cast<ScanSmem<BUFS> *>(raw_smem);
    const int vt = (p.V + kSV - 1) / kSV, tile = (int)(blockIdx.x % vt);
    const int64_t sh = blockIdx.x / vt;
    const int hv = (int)(sh % p.HV), seq = (int)(sh / p.HV), h = hv / (p.HV / p.H);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    int64_t first, row;
    int all, len;
    if (!gdn_sequence(p, seq, first, all, row, len)) return;
    const int lo = p.c1 > 0 ? p.c0 : 0, hi = p.c1 > 0 ? p.c1 : all, nc = hi - lo;  // the launch's chunks
    if (tid == 0) {
        for (int k = 0; k < BUFS; ++k) {
            tc::mbar_init(&s.w_full[k], 1);
            tc::mbar_init(&s.k_full[k], 1);
        }
        tc::mbar_init(&s.d1, 1);
        tc::mbar_init(&s.d2, 1);
        tc::mbar_fence_init();
        s.dead = 0;
    }
    const uint32_t tm = tmem_open(&s.slot_addr, 128), D1 = tm, D2 = tm + 64;
    volatile int *dead = &s.dead;
    auto slot_of = [&](int n) { return first + (REV ? hi - 1 - n : lo + n); };
    auto fetch_w = [&](int n) {
        tc::mbar_arrive_expect_tx(&s.w_full[n % BUFS], 2 * kTile);
        tc::bulk_g2s(s.w[n % BUFS], p.wt + (slot_of(n) * p.HV + hv) * 2 * (int64_t)kTile, 2 * kTile, &s.w_full[n % BUFS]);
    };
    auto fetch_k = [&](int n) {
        tc::mbar_arrive_expect_tx(&s.k_full[n % BUFS], kTile);
        tc::bulk_g2s(s.k[n % BUFS], p.kt + (slot_of(n) * p.H + h) * (int64_t)kTile, kTile, &s.k_full[n % BUFS]);
    };
    if (warp == kScanRows / 32) {
        // contracted over keys (K-major left operands) and over rows (MN-major)
        const uint32_t id64 = tc::idesc_bf16(128, 64, false, true), id32 = tc::idesc_bf16(128, 32, false, true);
        const uint32_t im64 = tc::idesc_bf16(128, 64, true, true), im32 = tc::idesc_bf16(128, 32, true, true);
        const int ksteps = (p.K + 15) / 16;
        constexpr uint32_t step = 2 * 64;
        constexpr uint64_t low = kTile / 16;
        const uint64_t right = desc_mn64(s.right);
        int w_due = 0, k_due = 0;
        auto next = [&](bool w, int n) {
            if (lane != 0 || n >= nc) return;
            if (w) {
                fetch_w(n);
                ++w_due;
            } else {
                fetch_k(n);
                ++k_due;
            }
        };
        for (int n = 0; n < BUFS; ++n) {
            next(true, n);
            next(false, n);
        }
        for (int n = 0; n < nc; ++n) {
            const int at = n % BUFS, turn = n / BUFS & 1;
            const uint8_t *w = s.w[at], *k = s.k[at];
            bool ok = lane != 0 || copies_or_die(p, REV ? &s.k_full[at] : &s.w_full[at], turn, dead);
            __syncwarp();
            bar_sync(1, kScanThreads);  // the state's tile is written
            tc::tc_fence_after();
            if (lane == 0 && ok) {
                if (REV) {
                    gdn_mma(D1, desc_k(k), kStepK, right, step, id64, ksteps, 0);
                } else {
                    gdn_mma(D1, desc_k(w), kStepK, right, step, id64, ksteps, 0);
                    gdn_mma(D1, desc_k(w) + low, kStepK, right, step, id32, ksteps, 1);
                }
                tc::mma_commit(&s.d1);
                ok = copies_or_die(p, REV ? &s.w_full[at] : &s.k_full[at], turn, dead);
                if (wait_or_die(&s.d1, n & 1, dead, p.status)) next(!REV, n + BUFS);
            }
            bar_sync(2, kScanThreads);  // the rows are
            tc::tc_fence_after();
            if (lane == 0 && ok && !*dead) {
                if (REV) {
                    gdn_mma(D2, desc_mn(w), kStepMN, right, step, im64, kGC / 16, 0);
                    gdn_mma(D2, desc_mn(w) + low, kStepMN, right, step, im32, kGC / 16, 1);
                } else {
                    gdn_mma(D2, desc_mn(k), kStepMN, right, step, im64, kGC / 16, 0);
                }
                tc::mma_commit(&s.d2);
                if (wait_or_die(&s.d2, n & 1, dead, p.status)) next(REV, n + BUFS);
            }
        }
        if (lane == 0 && *dead) {  // copies may still be on their way here
            for (int n = w_due > BUFS ? w_due - BUFS : 0; n < w_due; ++n)
                tc::mbar_wait(&s.w_full[n % BUFS], n / BUFS & 1, 10000000ull);
            for (int n = k_due > BUFS ? k_due - BUFS : 0; n < k_due; ++n)
                tc::mbar_wait(&s.k_full[n % BUFS], n / BUFS & 1, 10000000ull);
        }
        __syncwarp();
        tmem_close(tm, 128);
        return;
    }
    // what the warps wrote, to the products
    auto hand_over = [&](int barrier) {
        tc::fence_async_smem();
        tc::tc_fence_before();
        asm volatile("bar.arrive %0, %1;" ::"r"(barrier), "r"(kScanThreads) : "memory");
    };
    const int quad = warp & 3, hf = warp >> 2, i = quad * 32 + lane, c0 = tile * kSV + hf * 16;
    const int64_t user = sh * p.K * p.V + (int64_t)i * p.V + c0;
    const int have = i < p.K ? min(16, p.V - c0) : 0;  // columns of the user's state (a multiple of 8)
    const float *from = REV ? (hi < all ? p.dcarry : p.dht) : (lo > 0 ? p.carry : p.h0);
    float st[16];
#pragma unroll
    for (int k = 0; k < 16; ++k) st[k] = from && k < have ? from[user + k] : 0.f;
    uint8_t *keep = REV ? p.et : p.st;           // the states' tiles
    uint8_t *out = REV ? p.dut : p.ut;           // the rows' tiles
    const float *base = REV ? p.du0 : p.u0;
    // 16 columns of row i as two parts, into the right operand's tile; and into a unit's tiles, behind
    // the products that wait for the first
    struct Parts {
        uint4 hi[2], lo[2];
    };
    auto parts = [&](const float (&x)[16]) {
        Parts u;
#pragma unroll
        for (int k = 0; k < 2; ++k) split8(x + 8 * k, u.hi[k], u.lo[k]);
        return u;
    };
    auto put = [&](const Parts &u) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            *reinterpret_cast<uint4 *>(s.right + tc::tile_off(i, hf * 16 + 8 * k, 64)) = u.hi[k];
            *reinterpret_cast<uint4 *>(s.right + tc::tile_off(i, 32 + hf * 16 + 8 * k, 64)) = u.lo[k];
        }
    };
    auto store = [&](const Parts &u, uint8_t *tiles, int64_t unit) {
        uint8_t *to = tiles + unit * 2 * (int64_t)kTile;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            *reinterpret_cast<uint4 *>(to + gtile(i, c0 + 8 * k)) = u.hi[k];
            *reinterpret_cast<uint4 *>(to + kTile + gtile(i, c0 + 8 * k)) = u.lo[k];
        }
    };
    auto ld_sum = [&](uint32_t d, float (&x)[16]) {  // the two parts' products
        uint32_t a[16], b[16];
        tmem_ld16_nowait(tc::tmem_at(d, quad * 32, hf * 16), a);
        tmem_ld16_nowait(tc::tmem_at(d, quad * 32, 32 + hf * 16), b);
        tmem_wait_ld();
#pragma unroll
        for (int k = 0; k < 16; ++k) x[k] = __uint_as_float(a[k]) + __uint_as_float(b[k]);
    };
    struct Next {
        float r0[16], b0[16];
        float e, rk, keep;  // (loaded, not yet waited for: nothing is formed of them here)
    } nx;
    auto fetch_rows = [&](int n) {
        const int64_t unit = slot_of(n) * p.HV + hv;
        const float *u = base + unit * kGC * kGD;
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            const float4 x = *reinterpret_cast<const float4 *>(u + wide_at(tile, hf * 4 + g, i));
            nx.r0[4 * g] = x.x; nx.r0[4 * g + 1] = x.y; nx.r0[4 * g + 2] = x.z; nx.r0[4 * g + 3] = x.w;
            if (REV && BUFS > 1) {  // (with two blocks an SM there are no registers for it)
                const float4 y = *reinterpret_cast<const float4 *>(p.b0 + unit * kGC * kGD + wide_at(tile, hf * 4 + g, i));
                nx.b0[4 * g] = y.x; nx.b0[4 * g + 1] = y.y; nx.b0[4 * g + 2] = y.z; nx.b0[4 * g + 3] = y.w;
            }
        }
        const GdnRows rd(p, unit);
        nx.e = rd.e[i];
        nx.rk = rd.rk[i];
        nx.keep = rd.c[kGC - 1];
    };
    if (nc > 0) {
        const Parts u = parts(st);
        put(u);
        hand_over(1);
        fetch_rows(0);
        store(u, keep, slot_of(0) * p.HV + hv);
    }
    for (int n = 0; n < nc; ++n) {
        const int64_t unit = slot_of(n) * p.HV + hv;
        wait_or_die(&s.d1, n & 1, dead, p.status);
        tc::tc_fence_after();
        float x[16], y[16];
        ld_sum(D1, x);
        const float er = nx.e * nx.rk, kept = nx.keep;
#pragma unroll
        for (int k = 0; k < 16; ++k) x[k] = REV ? fmaf(er, x[k], nx.r0[k]) : nx.r0[k] - x[k];
        Parts u;
        if (REV) {
            u = parts(x);
        } else {
#pragma unroll
            for (int k = 0; k < 16; ++k) y[k] = x[k] * er;
            u = parts(y);
        }
        put(u);
        hand_over(2);
        if (REV && BUFS > 1) {
#pragma unroll
            for (int k = 0; k < 16; ++k) y[k] = nx.b0[k];
        } else if (REV) {
            const float *b0 = p.b0 + unit * kGC * kGD;
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const float4 b = *reinterpret_cast<const float4 *>(b0 + wide_at(tile, hf * 4 + g, i));
                y[4 * g] = b.x; y[4 * g + 1] = b.y; y[4 * g + 2] = b.z; y[4 * g + 3] = b.w;
            }
        }
        if (!REV) u = parts(x);
        const Parts made = u;
        if (REV || BUFS == 1) store(made, out, unit);
        if (n + 1 < nc) fetch_rows(n + 1);
        wait_or_die(&s.d2, n & 1, dead, p.status);
        tc::tc_fence_after();
        ld_sum(D2, x);
#pragma unroll
        for (int k = 0; k < 16; ++k) st[k] = fmaf(kept, st[k], REV ? y[k] - x[k] : x[k]);
        if (n + 1 < nc) {
            u = parts(st);
            put(u);
            hand_over(1);
            store(u, keep, slot_of(n + 1) * p.HV + hv);
        }
        // U's tiles: the hand-over's fence would wait for these stores (139 -> 132 us; the reverse pass, whose
        // registers are full, took 163 so, 145 with the stores ahead)
        if (!REV && BUFS > 1) store(made, out, unit);
    }
    float *to = REV ? (lo > 0 ? p.dcarry : p.dh0) : (hi < all ? p.carry : p.ht);
#pragma unroll
    for (int k = 0; k < 16; ++k)
        if (to && k < have) to[user + k] = st[k];
    tmem_close(tm, 128);
}

// ------------------------------------------------------------------ outputs
// O = diag(rq) (diag(c) Q S + P U) for a chunk, one block each, two on an SM.  P and U are two bf16
// parts: where keys are alike, U's rows nearly cancel in the sum (one part each left o off by 3% of
// its largest value for keys that are all but the same); so is the state (one part left o off by half of what
// its own rounding does, and the kernel at 132 of its 151 us).  P is a left operand in tensor memory, over the gram it is
// made of, and its products are added to the state's.  Of the seven tiles three have room at a time: each is fetched
// as soon as the product with the one before it is through.  8192 rows of 16 heads: 51 us for 230 MB, 4.5 TB/s; 4 x 4096
// rows of 32 heads 151 us.
constexpr int kOutThreads = 256;
struct OutSmem {
    uint8_t q[kTile], k[kTile], s[kTile];  // Q, then U's low part; K, then the state's low part; its high part, then U's
    float row[kGdnRowArrays * kGC];
    // a barrier for each use: a thread that has not seen a phase end yet would wait for the one two later
    uint64_t full[3], done[3];
    uint32_t slot_addr;
    int dead;
};
template <bool AL>
__global__ void __launch_bounds__(kOutThreads, 2) gdn_tc_out_kernel(GdnArgs p, int vec) {
    extern __shared__ __align__(1024) uint8_t raw_smem[];
    OutSmem &s = *reinterpret_cast<OutSmem *>(raw_smem);
    int slot, hv;
    gdn_unit(p, (int)blockIdx.x, slot, hv);
    const int64_t unit = (int64_t)slot * p.HV + hv;
    const int h = hv / (p.HV / p.H);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, quad = warp & 3, hf = warp >> 2, i = quad * 32 + lane;
    GdnChunk c;
    if (!gdn_find_chunk(p, slot, c)) return;
    if (tid == 0) {
        for (int k = 0; k < 3; ++k) {
            tc::mbar_init(&s.full[k], 1);
            tc::mbar_init(&s.done[k], 1);
        }
        tc::mbar_fence_init();
        s.dead = 0;
        tc::mbar_arrive_expect_tx(&s.full[0], 2 * kTile);
        tc::bulk_g2s(s.k, p.kt + ((int64_t)slot * p.H + h) * kTile, kTile, &s.full[0]);
        tc::bulk_g2s(s.s, p.st + unit * 2 * (int64_t)kTile, kTile, &s.full[0]);
    }
    const uint32_t tm = tmem_open(&s.slot_addr, 256), G = tm, O = tm + 128;
    volatile int *dead = &s.dead;
    load_tile_rows<AL, kOutThreads>(s.q, static_cast<const bf16 *>(p.q) + c.r0 * p.q_stride + (int64_t)h * p.K, p.q_stride,
                                    c.nr, p.K, tid);
    load_rows_of(s.row, p, unit, tid, kOutThreads);
    cp_async_wait_all();
    tc::fence_async_smem();
    __syncthreads();
    const int ksteps = (p.K + 15) / 16, cols = (p.V + kSV - 1) / kSV * kSV;
    const uint32_t id_v = tc::idesc_bf16(128, cols, false, true);
    const bool ok = copies_or_die(p, &s.full[0], 0, dead);
    if (tid == 0 && ok) {
        gdn_mma(G, desc_k(s.q), kStepK, desc_k(s.k), kStepK, tc::idesc_bf16(128, 128, false, false), ksteps, 0);
        gdn_mma(O, desc_k(s.q), kStepK, desc_mn(s.s), kStepMN, id_v, ksteps, 0);
        tc::mma_commit(&s.done[0]);
    }
    wait_or_die(&s.done[0], 0, dead, p.status);
    tc::tc_fence_after();
    int fetches = 1;
    if (tid == 0 && !*dead) {
        ++fetches;
        tc::mbar_arrive_expect_tx(&s.full[1], 2 * kTile);
        tc::bulk_g2s(s.k, p.st + unit * 2 * (int64_t)kTile + kTile, kTile, &s.full[1]);
        tc::bulk_g2s(s.s, p.ut + unit * 2 * (int64_t)kTile, kTile, &s.full[1]);
    }
    const GdnRows rd(s.row, kGC);
    const float ai = rd.a[i], li = rd.lo[i], rq = rd.rq[i], ci = rd.c[i];
    uint32_t hi[32], lo[32];
#pragma unroll
    for (int J = 0; J < 4; ++J) {
        const int j0 = hf * 64 + J * 16;
        float v[16], w[16];
        tc::tmem_ld16(tc::tmem_at(G, quad * 32, j0), v);
        decays16(rd, i, quad, j0 / 16, ai, li, w);
#pragma unroll
        for (int k = 0; k < 8; ++k) split2(v[2 * k] * w[2 * k], v[2 * k + 1] * w[2 * k + 1], hi[J * 8 + k], lo[J * 8 + k]);
        if (J == 2 && tid == 0 && copies_or_die(p, &s.full[1], 0, dead)) {
            gdn_mma(O, desc_k(s.q), kStepK, desc_mn(s.k), kStepMN, id_v, ksteps, 1);
            tc::mma_commit(&s.done[1]);
        }
    }
    wait_or_die(&s.done[1], 0, dead, p.status);
    tc::tc_fence_after();
    if (tid == 0 && !*dead) {
        ++fetches;
        tc::mbar_arrive_expect_tx(&s.full[2], kTile);
        tc::bulk_g2s(s.q, p.ut + unit * 2 * (int64_t)kTile + kTile, kTile, &s.full[2]);
    }
#pragma unroll 1
    for (int J = 0; J < 8; ++J) {
        const int j0 = hf * 64 + J * 8;
        if (j0 >= cols) break;
        float x[8];
        tc::tmem_ld8(tc::tmem_at(O, quad * 32, j0), x);
#pragma unroll
        for (int k = 0; k < 8; ++k) x[k] *= ci;
        tc::tmem_st8(tc::tmem_at(O, quad * 32, j0), x);
    }
    tc::tc_fence_before();
    __syncthreads();  // everyone has read the gram
    tc::tc_fence_after();
#pragma unroll
    for (int J = 0; J < 2; ++J) {
        tmem_st16_nowait(tc::tmem_at(G, quad * 32, hf * 32 + J * 16), *reinterpret_cast<const uint32_t(*)[16]>(hi + J * 16));
        tmem_st16_nowait(tc::tmem_at(G, quad * 32, 64 + hf * 32 + J * 16),
                         *reinterpret_cast<const uint32_t(*)[16]>(lo + J * 16));
    }
    tmem_wait_st();
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    if (tid == 0 && !*dead) {
        const uint64_t u = desc_mn(s.s), ul = desc_mn(s.q);
#pragma unroll 1
        for (int k = 0; k < kGC / 16; ++k) mma_bf16_ts(O, G + 64 + 8 * k, u + k * kStepMN, id_v, 1);
#pragma unroll 1
        for (int k = 0; k < kGC / 16; ++k) mma_bf16_ts(O, G + 8 * k, u + k * kStepMN, id_v, 1);
        if (copies_or_die(p, &s.full[2], 0, dead)) {
#pragma unroll 1
            for (int k = 0; k < kGC / 16; ++k) mma_bf16_ts(O, G + 8 * k, ul + k * kStepMN, id_v, 1);
            tc::mma_commit(&s.done[2]);
        }
    }
    wait_or_die(&s.done[2], 0, dead, p.status);
    tc::tc_fence_after();
    bf16 *o = static_cast<bf16 *>(p.o) + ((c.r0 + i) * p.HV + hv) * (int64_t)p.V;
#pragma unroll 1
    for (int J = 0; J < 4; ++J) {
        const int j0 = hf * 64 + J * 16;
        if (j0 >= p.V) break;
        float x[16];
        tc::tmem_ld16(tc::tmem_at(O, quad * 32, j0), x);
#pragma unroll
        for (int k = 0; k < 16; ++k) x[k] *= rq;
        if (i < c.nr) store16(o + j0, x, p.V - j0, vec);
    }
    if (tid == 0 && *dead)  // its copies, if still on their way
        for (int k = 0; k < fetches; ++k) tc::mbar_wait(&s.full[k], 0, 10000000ull);
    tmem_close(tm, 256);
}

cudaError_t prepare_kernels() {
    static DeviceOnce once;
    int dev;
    return once.run(&dev, [](int) {
        auto room = [](auto *k, size_t n) {
            return cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)n);
        };
        cudaError_t e = room(gdn_tc_prep_kernel<true>, sizeof(PrepSmem));
        if (e == cudaSuccess) e = room(gdn_tc_prep_kernel<false>, sizeof(PrepSmem));
        if (e == cudaSuccess) e = room(gdn_tc_scan_kernel<false, 1>, sizeof(ScanSmem<1>));
        if (e == cudaSuccess) e = room(gdn_tc_scan_kernel<true, 1>, sizeof(ScanSmem<1>));
        if (e == cudaSuccess) e = room(gdn_tc_scan_kernel<false, 2>, sizeof(ScanSmem<2>));
        if (e == cudaSuccess) e = room(gdn_tc_scan_kernel<true, 2>, sizeof(ScanSmem<2>));
        if (e == cudaSuccess) e = room(gdn_tc_out_kernel<true>, sizeof(OutSmem));
        if (e == cudaSuccess) e = room(gdn_tc_out_kernel<false>, sizeof(OutSmem));
        return e;
    });
}
static_assert(2 * (sizeof(ScanSmem<1>) + 1024) <= 233472 && sizeof(ScanSmem<2>) <= 232448 &&
                  2 * (sizeof(PrepSmem) + 1024) <= 233472 && 2 * (sizeof(OutSmem) + 1024) <= 233472,
              "an SM's shared memory");

}  // namespace

bool gdn_tc_supported(kda_dtype dt, int K, int V) {
    return dt == KDA_DTYPE_BF16 && K % 8 == 0 && V % 8 == 0 && K <= 128 && V <= 128;
}

static cudaError_t launch_prep(const GdnArgs &a, int64_t units, cudaStream_t st) {
    const bool kv = rows16(a.k, a.k_stride, a.K) && rows16(a.v, a.v_stride, a.V);
    return run("gdn_tc_prep", kv ? gdn_tc_prep_kernel<true> : gdn_tc_prep_kernel<false>, units, kPrepThreads,
               sizeof(PrepSmem), st, a);
}
static int64_t scan_blocks(const GdnArgs &a) { return (int64_t)a.N * a.HV * ((a.V + kSV - 1) / kSV); }
static cudaError_t launch_scan(const GdnArgs &a, cudaStream_t st) {
    const int64_t scans = scan_blocks(a);
    return scans <= kSms ? run("gdn_tc_scan", gdn_tc_scan_kernel<false, 2>, scans, kScanThreads, sizeof(ScanSmem<2>), st, a)
                         : run("gdn_tc_scan", gdn_tc_scan_kernel<false, 1>, scans, kScanThreads, sizeof(ScanSmem<1>), st, a);
}
static cudaError_t launch_out(const GdnArgs &a, int64_t units, cudaStream_t st) {
    const bool q = rows16(a.q, a.q_stride, a.K);
    return run("gdn_tc_out", q ? gdn_tc_out_kernel<true> : gdn_tc_out_kernel<false>, units, kOutThreads, sizeof(OutSmem), st, a,
               (int)(aligned_to(a.o, 32) && a.V % 16 == 0));
}
// The reverse pass over chunks.
cudaError_t launch_gdn_tc_rscan(const GdnArgs &a, cudaStream_t st) {
    const cudaError_t e = prepare_kernels();
    if (e != cudaSuccess) return e;
    const int64_t scans = scan_blocks(a);
    return scans <= kSms ? run("gdn_tc_rscan", gdn_tc_scan_kernel<true, 2>, scans, kScanThreads, sizeof(ScanSmem<2>), st, a)
                         : run("gdn_tc_rscan", gdn_tc_scan_kernel<true, 1>, scans, kScanThreads, sizeof(ScanSmem<1>), st, a);
}

// The library's streams for what runs beside a pass over chunks: up to four per device, each made by the
// first call that needs it.  A call takes one whose work is done, or one that its own stream had last: behind
// another stream's work, which may stand behind anything, it would wait for that stream.  A taken one
// belongs to its call alone, so that no lock is held while work is enqueued.
namespace {
constexpr int kSides = 4, kDevices = 64;
GdnSide g_sides[kDevices][kSides];
std::mutex &sides_lock() {
    static std::mutex mu;
    return mu;
}
cudaError_t make_side(GdnSide &s) {
    int least = 0, greatest = 0;
    cudaError_t e = cudaDeviceGetStreamPriorityRange(&least, &greatest);
    for (cudaEvent_t &ev : s.ev)
        if (e == cudaSuccess && !ev) e = cudaEventCreateWithFlags(&ev, cudaEventDisableTiming);
    return e == cudaSuccess ? cudaStreamCreateWithPriority(&s.stream, cudaStreamNonBlocking, least) : e;
}
}  // namespace

GdnSideHold::GdnSideHold(cudaStream_t st) {
    int dev = 0;
    unsigned long long id = 0;
    if ((error = cudaGetDevice(&dev)) != cudaSuccess || (error = cudaStreamGetId(st, &id)) != cudaSuccess) return;
    if (dev < 0 || dev >= kDevices) return;
    // (asking for an event would end another thread's capture that forbids such calls)
    cudaStreamCaptureMode mode = cudaStreamCaptureModeRelaxed;
    if ((error = cudaThreadExchangeStreamCaptureMode(&mode)) != cudaSuccess) return;
    {
        std::lock_guard<std::mutex> lock(sides_lock());
        GdnSide *idle = nullptr;
        for (GdnSide &s : g_sides[dev]) {
            if (s.taken) continue;
            if (s.last && s.of == id) {
                idle = &s;
                break;
            }
            if (!idle && (!s.last || cudaEventQuery(s.last) == cudaSuccess)) idle = &s;
        }
        if (cudaPeekAtLastError() == cudaErrorNotReady) cudaGetLastError();  // (the query's; nobody else's error)
        if (idle && !idle->stream) error = make_side(*idle);
        if (idle && error == cudaSuccess) {
            idle->taken = true;
            idle->of = id;
            side = idle;
        }
    }
    const cudaError_t e = cudaThreadExchangeStreamCaptureMode(&mode);
    if (error == cudaSuccess) error = e;
}
GdnSideHold::~GdnSideHold() {
    if (!side) return;
    std::lock_guard<std::mutex> lock(sides_lock());
    side->taken = false;
}

// Where to cut a dense sequence's chunks in two for pipelined launches, from the front; 0: not at all.  While a
// pass walks one part, the kernel that takes the other part's chunks all at once runs on the SMs it leaves
// free, at `unit_ns` of the whole card per unit; a pass's round takes `round_ns`.  Only where there are
// `least` units (launches and joins cost some 20 us) and the pass has at most two thirds of the SMs, and not
// inside a capture: a graph would hold the library's stream until it ends.  Measured, a training pass (and a
// forward) in one part and in two, B = 1, K = V = 128: 8192 rows, 24 heads 924 and 867 us (357, 330); 16 heads 704 and
// 625 (286, 260 to 286: which kernel finds the SMs first is open); 8 heads 519 and 467 (224, 220); 4 heads 399 and 390
// (181, 195: one part); 32768 rows of 4 heads 1458 and 1311 (661, 612); refused: 32 heads 1091 and 1220 (410, 427),
// 2048 rows of 16 heads 212 and 245 (89, 110).
int gdn_cut(const GdnArgs &a, double unit_ns, double round_ns, int64_t least, cudaStream_t st) {
    const int nc = (a.T + a.L - 1) / a.L;
    const int64_t scans = scan_blocks(a);
    if (a.cu || nc < 16 || a.slots * a.HV < least || 3 * scans > 2 * kSms) return 0;
    cudaStreamCaptureStatus cap = cudaStreamCaptureStatusNone;
    if (cudaStreamIsCapturing(st, &cap) != cudaSuccess || cap != cudaStreamCaptureStatusNone) {
        cudaGetLastError();
        return 0;
    }
    // the part that is walked while the other one is worked on: as long as that takes
    const double beside = unit_ns * a.B * a.HV * kSms / (kSms - scans);
    const int m = (int)(nc * beside / (beside + round_ns) + 0.5);
    return m < nc / 8 ? nc / 8 : m > nc - nc / 8 ? nc - nc / 8 : m;
}

// The chunk matrices, the pass and (with p.o) the outputs; the rows' scalars are in place.
cudaError_t launch_gdn_tc_fwd(const GdnArgs &a, cudaStream_t st) {
    cudaError_t e = prepare_kernels();
    if (e != cudaSuccess) return e;
    const int m = gdn_cut(a, kPrepNs, kRoundNs, 512, st);
    std::optional<GdnSideHold> hold;
    if (m > 0 && (e = hold.emplace(st).error) != cudaSuccess) return e;
    GdnSide *const s = hold ? hold->side : nullptr;
    if (!s) {
        const int64_t units = a.slots * a.HV;
        if ((e = launch_prep(a, units, st)) != cudaSuccess) return e;
        if ((e = launch_scan(a, st)) != cudaSuccess) return e;
        return a.o ? launch_out(a, units, st) : cudaSuccess;
    }
    // chunks [0, m) and [m, nc): the second part's matrices beside the first's pass, the first's outputs beside
    // the second's
    GdnArgs x = a, y = a;
    x.c0 = 0;
    x.c1 = y.c0 = m;
    y.c1 = (a.T + a.L - 1) / a.L;
    const int64_t heads = (int64_t)a.B * a.HV, ux = heads * (x.c1 - x.c0), uy = heads * (y.c1 - y.c0);
    if ((e = launch_prep(x, ux, st)) != cudaSuccess) return e;
    if ((e = cudaEventRecord(s->ev[0], st)) != cudaSuccess) return e;
    if ((e = launch_scan(x, st)) != cudaSuccess) return e;
    if ((e = cudaEventRecord(s->ev[1], st)) != cudaSuccess) return e;
    if ((e = cudaStreamWaitEvent(s->stream, s->ev[0], 0)) != cudaSuccess) return e;
    e = launch_prep(y, uy, s->stream);
    const cudaError_t j = s->join(2, st);  // also after a failure: nothing of the call stays behind on the side
    if (e != cudaSuccess || (e = j) != cudaSuccess) return e;
    if ((e = launch_scan(y, st)) != cudaSuccess || !a.o) return e;
    if ((e = cudaStreamWaitEvent(s->stream, s->ev[1], 0)) != cudaSuccess) return e;
    e = launch_out(x, ux, s->stream);
    if (e == cudaSuccess) e = launch_out(y, uy, st);
    const cudaError_t k = s->join(3, st);
    return e != cudaSuccess ? e : k;
}

}  // namespace kda
