// kda_gdn_tc_bwd.cu -- the gated delta rule's gradients on the tensor cores (see kda_gdn.cuh for the
// formulas, kda_gdn_tc.cuh for tiles and precision): what a chunk's outputs give its rows and its
// state (P^T dO and Q^T diag(c) dO, all chunks at once), the reverse pass over chunks (in
// kda_gdn_tc.cu), and each chunk's gradients, all at once.
#include "kda_gdn_tc.cuh"

namespace kda {
namespace {

using bf16 = __nv_bfloat16;

// ------------------------------------------------------------------ what the outputs give
// dU0 = P^T dO and B0 = Q^T diag(rq c) dO, for the reverse pass, in fp32.  P and the scaled dO are two
// bf16 parts; P's are multiplied one after the other from the same tile, so that two blocks fit
// an SM.  8192 rows of 16 heads: 57 us for 230 MB, 4.0 TB/s.
constexpr int kBaseThreads = 256;
struct BaseSmem {
    uint8_t q[kTile], k[kTile], d[kTile];  // Q; K, then P's parts and the scaled dO's low part; dO
    float row[kGdnRowArrays * kGC];
    uint64_t full, done;
    uint32_t slot_addr;
    int dead;
};
template <bool AL>
__global__ void __launch_bounds__(kBaseThreads, 2) gdn_tc_base_kernel(GdnArgs p) {
    extern __shared__ __align__(1024) uint8_t raw_smem[];
    BaseSmem &s = *reinterpret_cast<BaseSmem *>(raw_smem);
    int slot, hv;
    gdn_unit(p, (int)blockIdx.x, slot, hv);
    const int64_t unit = (int64_t)slot * p.HV + hv;
    const int h = hv / (p.HV / p.H);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, quad = warp & 3, hf = warp >> 2, i = quad * 32 + lane;
    GdnChunk c;
    if (!gdn_find_chunk(p, slot, c)) return;
    if (tid == 0) {
        tc::mbar_init(&s.full, 1);
        tc::mbar_init(&s.done, 1);
        tc::mbar_fence_init();
        s.dead = 0;
        tc::mbar_arrive_expect_tx(&s.full, kTile);
        tc::bulk_g2s(s.k, p.kt + ((int64_t)slot * p.H + h) * kTile, kTile, &s.full);
    }
    const uint32_t tm = tmem_open(&s.slot_addr, 256), G = tm, R = tm + 128;
    volatile int *dead = &s.dead;
    uint32_t phase = 0;
    auto all_done = [&]() {
        wait_or_die(&s.done, phase, dead, p.status);
        phase ^= 1;
        tc::tc_fence_after();
    };
    auto hand_over = [&]() {
        tc::fence_async_smem();
        tc::tc_fence_before();
        __syncthreads();
        tc::tc_fence_after();
    };
    load_tile_rows<AL, kBaseThreads>(s.q, static_cast<const bf16 *>(p.q) + c.r0 * p.q_stride + (int64_t)h * p.K, p.q_stride,
                                     c.nr, p.K, tid);
    load_tile_rows<AL, kBaseThreads>(s.d, static_cast<const bf16 *>(p.dout) + (c.r0 * p.HV + hv) * (int64_t)p.V,
                                     (int64_t)p.HV * p.V, c.nr, p.V, tid);
    load_rows_of(s.row, p, unit, tid, kBaseThreads);
    cp_async_wait_all();
    hand_over();
    const int cols = (p.V + kSV - 1) / kSV * kSV;
    const uint32_t id_t = tc::idesc_bf16(128, cols, true, true);
    const bool ok = copies_or_die(p, &s.full, 0, dead);
    if (tid == 0 && ok) {
        gdn_mma(G, desc_k(s.q), kStepK, desc_k(s.k), kStepK, tc::idesc_bf16(128, 128, false, false), (p.K + 15) / 16, 0);
        tc::mma_commit(&s.done);
    }
    all_done();
    const GdnRows rd(s.row, kGC);
    const float ai = rd.a[i], li = rd.lo[i], rq = rd.rq[i], ci = rd.c[i];
    uint32_t low[32];
#pragma unroll
    for (int J = 0; J < 4; ++J) {
        const int j0 = hf * 64 + J * 16;
        float v[16], w[16];
        tc::tmem_ld16(tc::tmem_at(G, quad * 32, j0), v);
        decays16(rd, i, quad, j0 / 16, ai, li, w);
#pragma unroll
        for (int k = 0; k < 16; ++k) v[k] *= w[k] * rq;
#pragma unroll
        for (int k = 0; k < 16; k += 8) {
            uint4 a, b;
            split8(v + k, a, b);
            *reinterpret_cast<uint4 *>(s.k + gtile(i, j0 + k)) = a;
            low[J * 8 + k / 2] = b.x; low[J * 8 + k / 2 + 1] = b.y;
            low[J * 8 + k / 2 + 2] = b.z; low[J * 8 + k / 2 + 3] = b.w;
        }
    }
    auto product = [&](uint32_t d, const uint8_t *a, const uint8_t *b, uint32_t acc) {
        gdn_mma(d, desc_mn(a), kStepMN, desc_mn(b), kStepMN, id_t, kGC / 16, acc);
        tc::mma_commit(&s.done);
    };
    hand_over();
    if (tid == 0 && !*dead) product(R, s.k, s.d, 0);
    all_done();
#pragma unroll
    for (int k = 0; k < 8; ++k)
        *reinterpret_cast<uint4 *>(s.k + gtile(i, hf * 64 + k * 8)) =
            make_uint4(low[4 * k], low[4 * k + 1], low[4 * k + 2], low[4 * k + 3]);
    hand_over();
    if (tid == 0 && !*dead) product(R, s.k, s.d, 1);
    all_done();
    // dO scaled, its parts over dO and P
    const float f = rq * ci;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const uint32_t at = gtile(i, hf * 64 + k * 8);
        float x[8];
        bf16x8(*reinterpret_cast<const uint4 *>(s.d + at), x);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] *= f;
        uint4 a, b;
        split8(x, a, b);
        *reinterpret_cast<uint4 *>(s.d + at) = a;
        *reinterpret_cast<uint4 *>(s.k + at) = b;
    }
    hand_over();
    if (tid == 0 && !*dead) {
        gdn_mma(G, desc_mn(s.q), kStepMN, desc_mn(s.k), kStepMN, id_t, kGC / 16, 0);
        product(G, s.q, s.d, 1);
    }
    auto store = [&](uint32_t from, float *to) {
        for (int t = hf; t < cols / kSV; t += 2) {
            float v[32];
            tc::tmem_ld32(tc::tmem_at(from, quad * 32, t * kSV), v);
#pragma unroll
            for (int g = 0; g < 8; ++g)
                *reinterpret_cast<float4 *>(to + wide_at(t, g, i)) =
                    make_float4(v[4 * g], v[4 * g + 1], v[4 * g + 2], v[4 * g + 3]);
        }
    };
    store(R, p.du0 + unit * kGC * kGD);
    all_done();
    store(G, p.b0 + unit * kGC * kGD);
    if (tid == 0 && *dead) tc::mbar_wait(&s.full, 0, 10000000ull);  // K, if still on its way here
    tmem_close(tm, 256);
}

// ------------------------------------------------------------------ a chunk's gradients
// One block per (chunk, value head) with all of an SM: seven tiles and the whole tensor memory.  The
// products, in the order in which tiles come and go (parts of the left and right operand):
//   1  Z = M^T dU (2, 2);  K K^T
//   2  Z U^T (2, 2);  dO U^T (1, 2);  Q K^T        -> X, Y and the pairs' sums
//   3  Z S^T (2, 2);  dO S^T (1, 2);  U E^T (2, 2)  -> the rows' sums
//   4  X K, X^T Q, (Y + Y^T) K (2, 1), added to the rows' shares of step 3
// X and Y carry both rows' norm factors, so that what step 4 leaves is dq and dk but for the norm's
// projection.
// Each block takes every n-th unit; the next unit's tiles are fetched as soon as this one's leave room
// (224 KB are a quarter of a unit's time), which moves the tiles' parts around: see the loop's end.
// 8192 rows of 16 heads: 219 us, 32 us a unit, of which its products take 7.  One unit an SM is a chain of
// four rounds of products and what the threads do between them; HBM is 34% busy, and no shared memory is left
// for a second unit.  X and Y with one part each (208 us) left dq and dk off by 2.5e-3 from the rounded ones; their
// low parts by bulk copies, which want a fence between the threads' writes and the copy, some 235.
constexpr int kGradThreads = 512;
struct GradSmem {
    uint8_t t[7][kTile];
    float red[4][kGC], small[32];
    // (done's next phase must not end before every thread has seen this one end: a thread that had not would wait
    // for the one after.  Two products follow each other without a barrier between, so the second has its own)
    uint64_t full[4], done, done_e;
    uint32_t slot_addr;
    int dead;
};
static_assert(sizeof(GradSmem) <= 232448, "a block's shared memory");

// The sums over a warp's lanes of 32 values each: lane l gets the sum of v[l].
__device__ __forceinline__ float lane_sums(float (&v)[32]) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
        for (int k = 0; k < o; ++k) {
            const float mine = lane & o ? v[k + o] : v[k], other = lane & o ? v[k] : v[k + o];
            v[k] = mine + __shfl_xor_sync(0xffffffffu, other, o);
        }
    return v[0];
}

// Several loads of tensor memory behind one wait, whose results pass through it.
__device__ __forceinline__ void ld8_nowait(uint32_t taddr, float (&v)[8]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7])
                 : "r"(taddr)
                 : "memory");
}
__device__ __forceinline__ void pin8(float (&v)[8]) {
    asm volatile("" : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]));
}
template <typename... V>
__device__ __forceinline__ void wait_ld(V &...v) {
    tmem_wait_ld();
    (pin8(v), ...);
}

template <bool AL>
__global__ void __launch_bounds__(kGradThreads, 1) gdn_tc_grad_kernel(GdnArgs p, int direct, int wide) {
    extern __shared__ __align__(1024) uint8_t raw_smem[];
    GradSmem &s = *reinterpret_cast<GradSmem *>(raw_smem);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, quad = warp & 3, part = warp >> 2, i = quad * 32 + lane;
    const int c0 = part * 32;  // a thread's columns of its row
    const int chunks = p.cu ? (p.ctrl->valid ? p.ctrl->total_chunks : 0) : p.c1 > 0 ? p.B * (p.c1 - p.c0) : (int)p.slots;
    const int units = chunks * p.HV;
    if ((int)blockIdx.x >= units) return;
    // the tiles by what they hold: M (A, B), then Q and dO, the state, K and X; dU (C, D), then Z, E; U (E, F), then Q;
    // K (G), then the state and Y
    uint8_t *A = s.t[0], *B = s.t[1], *E = s.t[4], *F = s.t[5], *G = s.t[6];
    uint8_t *const C = s.t[2], *const D = s.t[3];
    auto fetch = [&](int bar, uint8_t *to, const uint8_t *from, uint32_t bytes) {
        tc::bulk_g2s(to, from, bytes, &s.full[bar]);
    };
    int slot, hv;  // of the unit that the tiles asked for next belong to
    gdn_unit(p, (int)blockIdx.x, slot, hv);
    auto two_of = [&](int slot, int hv) { return ((int64_t)slot * p.HV + hv) * 2 * kTile; };
    auto k_of = [&](int slot, int hv) { return p.kt + ((int64_t)slot * p.H + hv / (p.HV / p.H)) * kTile; };
    if (tid == 0) {
        for (int k = 0; k < 4; ++k) tc::mbar_init(&s.full[k], 1);
        tc::mbar_init(&s.done, 1);
        tc::mbar_init(&s.done_e, 1);
        tc::mbar_fence_init();
        s.dead = 0;
        const int64_t two = two_of(slot, hv);
        tc::mbar_arrive_expect_tx(&s.full[0], 5 * kTile);
        fetch(0, A, p.mt + two, kTile);
        fetch(0, B, p.mt + two + kTile, kTile);
        fetch(0, C, p.dut + two, 2 * kTile);
        fetch(0, G, k_of(slot, hv), kTile);
        tc::mbar_arrive_expect_tx(&s.full[1], 2 * kTile);
        fetch(1, E, p.ut + two, kTile);
        fetch(1, F, p.ut + two + kTile, kTile);
    }
    int armed[4] = {1, 1, 0, 0};  // how often thread 0 set each of them
    const uint32_t tm = tmem_open(&s.slot_addr, 512), T0 = tm, T1 = tm + 128, T2 = tm + 256, T3 = tm + 384;
    volatile int *dead = &s.dead;
    uint32_t phase = 0;
    auto all_done = [&]() {
        wait_or_die(&s.done, phase, dead, p.status);
        phase ^= 1;
        tc::tc_fence_after();
    };
    auto hand_over = [&]() {
        tc::fence_async_smem();
        tc::tc_fence_before();
        __syncthreads();
        tc::tc_fence_after();
    };
    // the sum over a row's four threads, in all of them
    auto row_sum = [&](float x) {
        s.red[part][i] = x;
        __syncthreads();
        const float y = (s.red[0][i] + s.red[1][i]) + (s.red[2][i] + s.red[3][i]);
        __syncthreads();
        return y;
    };
    const int ksteps = (p.K + 15) / 16, vsteps = (p.V + 15) / 16, cols = (p.V + kSV - 1) / kSV * kSV;
    const uint32_t id_kk = tc::idesc_bf16(128, 128, false, false);
    // d = the product of two operands of one or two parts (low: 0 where there is one), the smallest first
    auto product = [&](uint32_t d, uint64_t a, uint64_t a_low, uint32_t as, uint64_t b, uint64_t b_low, uint32_t bs,
                       uint32_t id, int steps) {
        uint32_t acc = 0;
        if (b_low) {
            gdn_mma(d, a, as, b_low, bs, id, steps, 0);
            acc = 1;
        }
        if (a_low) {
            gdn_mma(d, a_low, as, b, bs, id, steps, acc);
            acc = 1;
        }
        gdn_mma(d, a, as, b, bs, id, steps, acc);
    };
    uint32_t turn = 0;  // parity of the unit's fetches
    for (int id = blockIdx.x; id < units; id += gridDim.x, turn ^= 1) {
        int next_slot = 0, next_hv = 0;
        const bool more = units - id > (int)gridDim.x;
        if (more) gdn_unit(p, id + (int)gridDim.x, next_slot, next_hv);
        const int64_t unit = (int64_t)slot * p.HV + hv, two = two_of(slot, hv);
        const int h = hv / (p.HV / p.H);
        GdnChunk c;
        gdn_find_chunk(p, slot, c);
        const bf16 *qrows = static_cast<const bf16 *>(p.q) + c.r0 * p.q_stride + (int64_t)h * p.K;
        const bf16 *drows = static_cast<const bf16 *>(p.dout) + (c.r0 * p.HV + hv) * (int64_t)p.V;
        const GdnRows rd(p, unit);
        const float ai = rd.a[i], li = rd.lo[i], ci = rd.c[i], ei = rd.e[i], bi = rd.b[i], rq = rd.rq[i], rk = rd.rk[i];
        uint4 vr[4];  // the thread's 32 columns of v
        {
            const bf16 *v = static_cast<const bf16 *>(p.v) + (c.r0 + i) * p.v_stride + (int64_t)hv * p.V;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                vr[k] = make_uint4(0u, 0u, 0u, 0u);
                if (c0 + 8 * k < p.V && i < c.nr) {
                    if constexpr (AL) {
                        vr[k] = *reinterpret_cast<const uint4 *>(v + c0 + 8 * k);
                    } else {
                        alignas(16) bf16 e[8];
#pragma unroll
                        for (int j = 0; j < 8; ++j) e[j] = v[c0 + 8 * k + j];
                        vr[k] = *reinterpret_cast<const uint4 *>(e);
                    }
                }
            }
        }
        // ------------------------------------------------ 1
        bool ok = copies_or_die(p, &s.full[0], turn, dead);
        if (tid == 0 && ok) {
            product(T0, desc_mn(A), desc_mn(B), kStepMN, desc_mn(C), desc_mn(D), kStepMN, tc::idesc_bf16(128, cols, true, true),
                    kGC / 16);
            product(T1, desc_k(G), 0, kStepK, desc_k(G), 0, kStepK, id_kk, ksteps);
            tc::mma_commit(&s.done);
        }
        all_done();
        load_tile_rows<AL, kGradThreads>(A, qrows, p.q_stride, c.nr, p.K, tid);
        load_tile_rows<AL, kGradThreads>(B, drows, (int64_t)p.HV * p.V, c.nr, p.V, tid);
        float beta_sum = 0.f;  // of dbeta
        {
            float z[32];
            tc::tmem_ld32(tc::tmem_at(T0, quad * 32, c0), z);
            bf16 *dv = static_cast<bf16 *>(p.dv) + ((c.r0 + i) * p.HV + hv) * (int64_t)p.V;
#pragma unroll
            for (int k = 0; k < 32; k += 8) {
                if (c0 + k < p.V) {
                    float x[8];
                    bf16x8(vr[k / 8], x);
#pragma unroll
                    for (int e = 0; e < 8; ++e) beta_sum = fmaf(z[k + e], x[e], beta_sum);
                }
                uint4 a, b;
                split8(z + k, a, b);
                *reinterpret_cast<uint4 *>(C + gtile(i, c0 + k)) = a;
                *reinterpret_cast<uint4 *>(D + gtile(i, c0 + k)) = b;
            }
#pragma unroll
            for (int k = 0; k < 32; ++k) z[k] *= bi;
            if (i < c.nr)
#pragma unroll
                for (int k = 0; k < 32; k += 16)
                    if (c0 + k < p.V) store16(dv + c0 + k, *reinterpret_cast<const float(*)[16]>(z + k), p.V - c0 - k, wide & 1);
        }
        // ------------------------------------------------ 2
        cp_async_wait_all();
        hand_over();
        ok = copies_or_die(p, &s.full[1], turn, dead);
        if (tid == 0 && ok) {
            product(T2, desc_k(C), desc_k(D), kStepK, desc_k(E), desc_k(F), kStepK, id_kk, vsteps);
            product(T3, desc_k(B), 0, kStepK, desc_k(E), desc_k(F), kStepK, id_kk, vsteps);
            product(T0, desc_k(A), 0, kStepK, desc_k(G), 0, kStepK, id_kk, ksteps);
            tc::mma_commit(&s.done);
        }
        all_done();
        if (tid == 0 && !*dead) {  // the state's parts, over Q and K
            ++armed[2];
            tc::mbar_arrive_expect_tx(&s.full[2], 2 * kTile);
            fetch(2, A, p.st + two, kTile);
            fetch(2, G, p.st + two + kTile, kTile);
        }
        float pairs = 0.f;  // thread t < 128: the sum over the pairs that row t's decay lies between
        // X's and Y's low parts wait in memory (P^T dO's place), for lack of any other room: eight columns of X,
        // then of Y, at a time; a thread reads what it wrote
        uint4 *const lows = reinterpret_cast<uint4 *>(p.du0 + unit * kGC * kGD) + tid;
        {
            uint32_t xs[16] = {}, ys[16] = {};
            float f[32];  // the pairs' shares, then their sums from the thread's first column on
            if (c0 <= quad * 32 + 31) {
                float ag = 0.f;
#pragma unroll
                for (int J = 0; J < 2; ++J) {
                    float w[16];
                    decays16(rd, i, quad, c0 / 16 + J, ai, li, w);
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        const int j0 = c0 + J * 16 + q * 8;
                        float g[8], hh[8], kk[8], qk[8];
                        ld8_nowait(tc::tmem_at(T2, quad * 32, j0), g);
                        ld8_nowait(tc::tmem_at(T3, quad * 32, j0), hh);
                        ld8_nowait(tc::tmem_at(T1, quad * 32, j0), kk);
                        ld8_nowait(tc::tmem_at(T0, quad * 32, j0), qk);
                        wait_ld(g, hh, kk, qk);
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            const float d = w[q * 8 + k];
                            const float a = j0 + k < i ? g[k] * (d * rk) : 0.f;
                            hh[k] *= d * rq;
                            ag = fmaf(a, kk[k], ag);
                            g[k] = -bi * a;
                            f[J * 16 + q * 8 + k] = fmaf(hh[k], qk[k], g[k] * kk[k]);
                        }
                        uint4 a, b;
                        split8(hh, a, b);
                        lows[(J * 2 + q) * kGradThreads] = b;
                        xs[J * 8 + q * 4] = a.x; xs[J * 8 + q * 4 + 1] = a.y;
                        xs[J * 8 + q * 4 + 2] = a.z; xs[J * 8 + q * 4 + 3] = a.w;
                        split8(g, a, b);
                        lows[(4 + J * 2 + q) * kGradThreads] = b;
                        ys[J * 8 + q * 4] = a.x; ys[J * 8 + q * 4 + 1] = a.y;
                        ys[J * 8 + q * 4 + 2] = a.z; ys[J * 8 + q * 4 + 3] = a.w;
                    }
                }
                beta_sum -= ag;
            } else {
#pragma unroll
                for (int k = 0; k < 32; ++k) f[k] = 0.f;
            }
            // f[k] = the sum of the row's shares before column c0 + k, where that column is not past i
            float run = 0.f;
#pragma unroll
            for (int k = 0; k < 32; ++k) {
                const float x = f[k];
                f[k] = run;
                run += x;
            }
            s.red[part][i] = run;
            tc::tc_fence_before();
            __syncthreads();
            tc::tc_fence_after();
            float before = 0.f;
            for (int k = 0; k < part; ++k) before += s.red[k][i];
#pragma unroll
            for (int k = 0; k < 32; ++k) f[k] = c0 + k <= i ? f[k] + before : 0.f;
            const float sum = lane_sums(f);
            __syncthreads();
            s.red[quad][c0 + lane] = sum;
            __syncthreads();
            if (tid < kGC) pairs = (s.red[0][tid] + s.red[1][tid]) + (s.red[2][tid] + s.red[3][tid]);
            // X and Y wait in tensor memory until tiles are free
            tmem_st16_nowait(tc::tmem_at(T2, quad * 32, c0 / 2), xs);
            tmem_st16_nowait(tc::tmem_at(T2, quad * 32, 64 + c0 / 2), ys);
            tmem_wait_st();
        }
        // ------------------------------------------------ 3
        hand_over();
        ok = copies_or_die(p, &s.full[2], turn, dead);
        if (tid == 0 && ok) {
            product(T0, desc_k(C), desc_k(D), kStepK, desc_k(A), desc_k(G), kStepK, id_kk, vsteps);
            product(T1, desc_k(B), 0, kStepK, desc_k(A), desc_k(G), kStepK, id_kk, vsteps);
            tc::mma_commit(&s.done);
        }
        all_done();
        if (tid == 0 && !*dead) {  // E over Z, K over dO
            ++armed[3];
            tc::mbar_arrive_expect_tx(&s.full[3], 3 * kTile);
            fetch(3, C, p.et + two, 2 * kTile);
            fetch(3, B, k_of(slot, hv), kTile);
        }
        ok = copies_or_die(p, &s.full[3], turn, dead);
        if (tid == 0 && ok) {
            product(T3, desc_k(E), desc_k(F), kStepK, desc_k(C), desc_k(D), kStepK, id_kk, vsteps);
            tc::mma_commit(&s.done_e);
        }
        float es = 0.f;  // <S, E>, a share
        for (int k = 0; k < 32; k += 8)
            if (c0 + k < p.V) {
                float a[8], b[8], x[8], y[8];
                const uint32_t at = gtile(i, c0 + k);
                bf16x8(*reinterpret_cast<const uint4 *>(A + at), a);
                bf16x8(*reinterpret_cast<const uint4 *>(G + at), b);
                bf16x8(*reinterpret_cast<const uint4 *>(C + at), x);
                bf16x8(*reinterpret_cast<const uint4 *>(D + at), y);
#pragma unroll
                for (int e = 0; e < 8; ++e) es = fmaf(a[e] + b[e], x[e] + y[e], es);
            }
        wait_or_die(&s.done_e, turn, dead, p.status);
        tc::tc_fence_after();
        // Q over U; X and Y over the state, their low parts over E
        load_tile_rows<AL, kGradThreads>(E, qrows, p.q_stride, c.nr, p.K, tid);
        uint4 low[8];
#pragma unroll
        for (int k = 0; k < 8; ++k)
            low[k] = c0 <= quad * 32 + 31 ? lows[k * kGradThreads] : make_uint4(0u, 0u, 0u, 0u);
        __syncthreads();
        if (tid == 0 && more && !*dead) {  // the next unit's K; dU and M below
            ++armed[0];
            tc::mbar_arrive_expect_tx(&s.full[0], 5 * kTile);
            fetch(0, F, k_of(next_slot, next_hv), kTile);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            *reinterpret_cast<uint4 *>(C + gtile(i, c0 + 8 * k)) = low[k];
            *reinterpret_cast<uint4 *>(D + gtile(i, c0 + 8 * k)) = low[4 + k];
        }
        {
            float v[32];
            tc::tmem_ld32(tc::tmem_at(T2, quad * 32, part * 32), v);
            uint8_t *to = part < 2 ? A : G;
#pragma unroll
            for (int k = 0; k < 32; k += 4)
                *reinterpret_cast<uint4 *>(to + gtile(i, (part & 1) * 64 + 2 * k)) =
                    make_uint4(__float_as_uint(v[k]), __float_as_uint(v[k + 1]), __float_as_uint(v[k + 2]),
                               __float_as_uint(v[k + 3]));
        }
        cp_async_wait_all();
        hand_over();
        float crow, erow;  // the row's sums: of the pairs' ends i >= t, and j < t
        {
            float zs[32], x[32];
            float kz = 0.f, qd = 0.f, ke = 0.f;
            tc::tmem_ld32(tc::tmem_at(T0, quad * 32, c0), zs);
            const float fz = -ci * bi * rk, fe = ei * rk;
            tc::tmem_ld32(tc::tmem_at(T3, quad * 32, c0), x);
#pragma unroll
            for (int k = 0; k < 32; k += 8) {
                float kv[8];
                bf16x8(*reinterpret_cast<const uint4 *>(B + gtile(i, c0 + k)), kv);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    kz = fmaf(kv[e], zs[k + e], kz);
                    ke = fmaf(kv[e], x[k + e], ke);
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) zs[k + e] = fmaf(fe, x[k + e], fz * zs[k + e]);
                tc::tmem_st8(tc::tmem_at(T0, quad * 32, c0 + k), *reinterpret_cast<const float(*)[8]>(zs + k));
            }
            tc::tmem_ld32(tc::tmem_at(T1, quad * 32, c0), x);
            const float fq = rq * ci;
#pragma unroll
            for (int k = 0; k < 32; k += 8) {
                float qv[8];
                bf16x8(*reinterpret_cast<const uint4 *>(E + gtile(i, c0 + k)), qv);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    qd = fmaf(qv[e], x[k + e], qd);
                    x[k + e] *= fq;
                }
                tc::tmem_st8(tc::tmem_at(T1, quad * 32, c0 + k), *reinterpret_cast<const float(*)[8]>(x + k));
            }
            beta_sum -= ci * rk * kz;
            crow = fmaf(fq, qd, fz * kz);
            erow = fe * ke;
        }
        // ------------------------------------------------ 4
        hand_over();
        if (tid == 0 && !*dead) {
            const uint32_t id = tc::idesc_bf16(128, 128, false, true), idt = tc::idesc_bf16(128, 128, true, true);
            gdn_mma(T1, desc_k(A), kStepK, desc_mn(B), kStepMN, id, kGC / 16, 1);
            gdn_mma(T0, desc_mn(A), kStepMN, desc_mn(E), kStepMN, idt, kGC / 16, 1);
            gdn_mma(T0, desc_k(G), kStepK, desc_mn(B), kStepMN, id, kGC / 16, 1);
            gdn_mma(T0, desc_mn(G), kStepMN, desc_mn(B), kStepMN, idt, kGC / 16, 1);
            gdn_mma(T1, desc_k(C), kStepK, desc_mn(B), kStepMN, id, kGC / 16, 1);
            gdn_mma(T0, desc_mn(C), kStepMN, desc_mn(E), kStepMN, idt, kGC / 16, 1);
            gdn_mma(T0, desc_k(D), kStepK, desc_mn(B), kStepMN, id, kGC / 16, 1);
            gdn_mma(T0, desc_mn(D), kStepMN, desc_mn(B), kStepMN, idt, kGC / 16, 1);
            tc::mma_commit(&s.done);
        }
        // dbeta and dg while they run
        beta_sum = row_sum(beta_sum);
        crow = row_sum(crow);
        erow = row_sum(erow);
        {
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) es += __shfl_xor_sync(0xffffffffu, es, o);
            if (lane == 0) s.small[warp] = es;
            if (part == 0 && i < c.nr) static_cast<bf16 *>(p.dbeta)[(c.r0 + i) * p.HV + hv] = from_f32<bf16>(beta_sum);
            __syncthreads();
            if (tid < kGC) {  // (thread t has row t)
                // suffix sums of the rows' c terms and prefix sums of their e terms, four warps of 32 rows
                float cs = crow, ep = erow;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const float x = __shfl_down_sync(0xffffffffu, cs, o), y = __shfl_up_sync(0xffffffffu, ep, o);
                    if (lane + o < 32) cs += x;
                    if (lane >= o) ep += y;
                }
                if (lane == 0) s.small[16 + warp] = cs;
                if (lane == 31) s.small[20 + warp] = ep;
                bar_sync(1, kGC);
                ep -= erow;
                for (int k = warp + 1; k < 4; ++k) cs += s.small[16 + k];
                for (int k = 0; k < warp; ++k) ep += s.small[20 + k];
                float se = 0.f;
                for (int k = 0; k < kGradThreads / 32; ++k) se += s.small[k];
                if (tid < c.nr)
                    p.dg[(c.r0 + tid) * p.HV + hv] = (pairs + cs + ep + rd.c[kGC - 1] * se) * (0.6931471805599453f * p.g_scale);
            }
        }
        all_done();
        if (tid == 0 && more && !*dead) {
            fetch(0, C, p.dut + two_of(next_slot, next_hv), 2 * kTile);
            fetch(0, A, p.mt + two_of(next_slot, next_hv), kTile);
            fetch(0, G, p.mt + two_of(next_slot, next_hv) + kTile, kTile);
        }
        const float nq = rq / p.scale;
#pragma unroll 1
        for (int m = 0; m < 2; ++m) {  // dq, dk
            const uint8_t *x = m ? B : E;
            float d[32];
            tc::tmem_ld32(tc::tmem_at(m ? T0 : T1, quad * 32, c0), d);
            if (direct) {
                if (p.l2) {
                    float dot = 0.f;
#pragma unroll
                    for (int k = 0; k < 32; k += 8) {
                        float v[8];
                        bf16x8(*reinterpret_cast<const uint4 *>(x + gtile(i, c0 + k)), v);
#pragma unroll
                        for (int e = 0; e < 8; ++e) dot = fmaf(d[k + e], v[e], dot);
                    }
                    dot = row_sum(dot);
                    const float f = -dot * (m ? rk * rk : nq * nq);
#pragma unroll
                    for (int k = 0; k < 32; k += 8) {
                        float v[8];
                        bf16x8(*reinterpret_cast<const uint4 *>(x + gtile(i, c0 + k)), v);
#pragma unroll
                        for (int e = 0; e < 8; ++e) d[k + e] = fmaf(f, v[e], d[k + e]);
                    }
                }
                bf16 *to = static_cast<bf16 *>(m ? p.dk : p.dq) + ((c.r0 + i) * p.H + h) * (int64_t)p.K;
#pragma unroll
                for (int k = 0; k < 32; k += 16)
                    if (i < c.nr && c0 + k < p.K)
                        store16(to + c0 + k, *reinterpret_cast<const float(*)[16]>(d + k), p.K - c0 - k, wide & 2);
            } else {
                float *to = (m ? p.dkh : p.dqh) + ((c.r0 + i) * p.HV + hv) * (int64_t)p.K;
#pragma unroll
                for (int k = 0; k < 32; k += 4)
                    if (i < c.nr && c0 + k < p.K)
                        *reinterpret_cast<float4 *>(to + c0 + k) = make_float4(d[k], d[k + 1], d[k + 2], d[k + 3]);
            }
        }
        // the next unit's U over K and Q; M is in (A, G), K in F
        tc::tc_fence_before();
        __syncthreads();
        tc::tc_fence_after();
        if (tid == 0 && more && !*dead) {
            ++armed[1];
            tc::mbar_arrive_expect_tx(&s.full[1], 2 * kTile);
            fetch(1, B, p.ut + two_of(next_slot, next_hv), kTile);
            fetch(1, E, p.ut + two_of(next_slot, next_hv) + kTile, kTile);
        }
        uint8_t *const old_b = B, *const old_e = E;
        B = G;
        G = F;
        E = old_b;
        F = old_e;
        slot = next_slot;
        hv = next_hv;
    }
    if (tid == 0 && *dead)  // copies may still be on their way here
        for (int k = 0; k < 4; ++k)
            if (armed[k] > 0) tc::mbar_wait(&s.full[k], (armed[k] - 1) & 1, 10000000ull);
    tmem_close(tm, 512);
}

cudaError_t prepare_kernels() {
    static DeviceOnce once;
    int dev;
    return once.run(&dev, [](int) {
        auto room = [](auto *k, size_t n) {
            return cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)n);
        };
        cudaError_t e = room(gdn_tc_base_kernel<true>, sizeof(BaseSmem));
        if (e == cudaSuccess) e = room(gdn_tc_base_kernel<false>, sizeof(BaseSmem));
        if (e == cudaSuccess) e = room(gdn_tc_grad_kernel<true>, sizeof(GradSmem));
        if (e == cudaSuccess) e = room(gdn_tc_grad_kernel<false>, sizeof(GradSmem));
        return e;
    });
}
static_assert(2 * (sizeof(BaseSmem) + 1024) <= 233472, "an SM's shared memory");

}  // namespace

// The gradients from the forward's kept states; dq and dk directly where no value heads share them.
cudaError_t launch_gdn_tc_bwd(const GdnArgs &a, cudaStream_t st) {
    cudaError_t e = prepare_kernels();
    if (e != cudaSuccess) return e;
    const bool al = rows16(a.q, a.q_stride, a.K) && rows16(a.v, a.v_stride, a.V) && aligned_to(a.dout, 16);
    const int wide = (aligned_to(a.dv, 32) && a.V % 16 == 0 ? 1 : 0) |
                     (aligned_to(a.dq, 32) && aligned_to(a.dk, 32) && a.K % 16 == 0 ? 2 : 0);
    auto base = [&](const GdnArgs &x, int64_t units, cudaStream_t on) {
        return run("gdn_tc_base", al ? gdn_tc_base_kernel<true> : gdn_tc_base_kernel<false>, units, kBaseThreads,
                   sizeof(BaseSmem), on, x);
    };
    auto grad = [&](const GdnArgs &x, int64_t units, int64_t sms, cudaStream_t on) {
        return run("gdn_tc_grad", al ? gdn_tc_grad_kernel<true> : gdn_tc_grad_kernel<false>, units < sms ? units : sms,
                   kGradThreads, sizeof(GradSmem), on, x, (int)(a.HV == a.H), wide);
    };
    const int m = gdn_cut(a, kGradNs, kRoundNs, 256, st);
    std::optional<GdnSideHold> hold;
    if (m > 0 && (e = hold.emplace(st).error) != cudaSuccess) return e;
    GdnSide *const s = hold ? hold->side : nullptr;
    if (!s) {
        const int64_t units = a.slots * a.HV;
        if ((e = base(a, units, st)) != cudaSuccess) return e;
        if ((e = launch_gdn_tc_rscan(a, st)) != cudaSuccess) return e;
        return grad(a, units, kSms, st);
    }
    // chunks [m, nc) first, then [0, m): the second's base products and the first's gradients beside the passes
    GdnArgs x = a, y = a;
    x.c0 = m;
    x.c1 = (a.T + a.L - 1) / a.L;
    y.c0 = 0;
    y.c1 = m;
    const int64_t heads = (int64_t)a.B * a.HV, ux = heads * (x.c1 - x.c0), uy = heads * (y.c1 - y.c0);
    const int64_t scans = (int64_t)a.N * a.HV * ((a.V + kSV - 1) / kSV);
    if ((e = base(x, ux, st)) != cudaSuccess) return e;
    if ((e = cudaEventRecord(s->ev[0], st)) != cudaSuccess) return e;
    if ((e = launch_gdn_tc_rscan(x, st)) != cudaSuccess) return e;
    if ((e = cudaEventRecord(s->ev[1], st)) != cudaSuccess) return e;
    if ((e = cudaStreamWaitEvent(s->stream, s->ev[0], 0)) != cudaSuccess) return e;
    e = base(y, uy, s->stream);
    const cudaError_t j = s->join(2, st);
    if (e != cudaSuccess || (e = j) != cudaSuccess) return e;
    if ((e = launch_gdn_tc_rscan(y, st)) != cudaSuccess) return e;
    if ((e = cudaStreamWaitEvent(s->stream, s->ev[1], 0)) != cudaSuccess) return e;
    e = grad(x, ux, kSms - scans, s->stream);
    if (e == cudaSuccess) e = grad(y, uy, kSms, st);
    const cudaError_t k = s->join(3, st);
    return e != cudaSuccess ? e : k;
}

}  // namespace kda
