// kda_gdn.cu -- the gated delta rule with one decay per head (see kda_gdn.cuh): the rows' decays
// and norms, the chunk form on the CUDA cores in fp32 (any K and V up to 256, fp32 or bf16
// inputs), the gradients of the norm, and the single-token step.
// Which path: bf16 with K and V multiples of 8 up to 128 takes the tensor cores (kda_gdn_tc.cuh), everything
// else the CUDA cores.  The tensor cores are at least level at the smallest sizes too (training pass, K = V = 8: 300
// rows of 4 heads 101 us against 107, 6000 rows of 8 heads 302 against 674; K = V = 64: 103 and 132, 330 and 1187).
#include "kda_gdn_tc.cuh"

namespace kda {
namespace {

using bf16 = __nv_bfloat16;
constexpr int kGL = 32;       // chunk length on the CUDA cores
constexpr int kVT = 32;       // value columns of a block
constexpr int kKT = 128;      // key columns of a round of the gradients
constexpr int kThreads = 256;

// The sum over the `width` lanes of a lane's group (a power of two), in every one of them.
template <int width>
__device__ __forceinline__ float lane_sum(float x) {
#pragma unroll
    for (int o = width / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}
// ------------------------------------------------------------------ rows
// 1 / sqrt(sum x^2 + 1e-6) of every q and k row: `lanes` lanes (a power of two) for each, 16 bytes
// apiece where rows are aligned for it.  67 MB of q and k (8192 rows of 16 heads of 128) in 19 us, 3.5 TB/s; with
// four rows for a group of lanes 24 us.
template <typename T, bool AL>
__global__ void __launch_bounds__(kThreads) gdn_norms_kernel(GdnArgs p, int log_lanes) {
    constexpr int VEC = 16 / sizeof(T);  // (of scalar loads too: the sums' order is the same)
    const int lanes = 1 << log_lanes, l = threadIdx.x & (lanes - 1);
    // rows times heads are counted in 31 bits
    const uint32_t id = blockIdx.x * (uint32_t)(kThreads >> log_lanes) + (threadIdx.x >> log_lanes);
    const bool in = id < (uint32_t)p.B * (uint32_t)p.T * (uint32_t)p.H;
    const int64_t r = in ? id / (uint32_t)p.H : 0;
    const int h = in ? (int)(id % (uint32_t)p.H) : 0;
    const T *q = static_cast<const T *>(p.q) + r * p.q_stride + (int64_t)h * p.K;
    const T *k = static_cast<const T *>(p.k) + r * p.k_stride + (int64_t)h * p.K;
    float sq = 0.f, sk = 0.f;
    for (int c = l * VEC; in && c < p.K; c += lanes * VEC) {
        float x[VEC], y[VEC];
        load_vec<T, VEC, AL>(q + c, p.K - c, x);
        load_vec<T, VEC, AL>(k + c, p.K - c, y);
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
            sq = fmaf(x[j], x[j], sq);
            sk = fmaf(y[j], y[j], sk);
        }
    }
    for (int o = lanes / 2; o > 0; o >>= 1) {
        sq += __shfl_xor_sync(0xffffffffu, sq, o);
        sk += __shfl_xor_sync(0xffffffffu, sk, o);
    }
    if (in && l == 0)
        reinterpret_cast<float2 *>(p.norms)[id] = make_float2(1.f / sqrtf(sq + 1e-6f), 1.f / sqrtf(sk + 1e-6f));
}

// A decay that leaves nothing of the state (the least fp32 is 2^-149): stronger ones, -inf among them,
// are taken as this one, so that the differences of the rows behind it keep their digits.
constexpr float kReset = -8192.f;
// The rows' decays: a block per chunk and 16 value heads, whose inputs come in whole sectors; then a
// warp per head, L / 32 consecutive rows per lane.  8192 rows of 16 heads: 7 us, the launch and one
// round of loads.
constexpr int kRowHeads = 16;
template <typename T, int PER>
__global__ void __launch_bounds__(32 * kRowHeads) gdn_rows_kernel(GdnArgs p) {
    static_assert(PER == 1 || PER == 4, "a row or a vector of them per lane");
    constexpr int L = 32 * PER;
    __shared__ float gs[kRowHeads][L + 1], bs[kRowHeads][L + 1];
    const int hb = (p.HV + kRowHeads - 1) / kRowHeads, hv0 = (int)(blockIdx.x % hb) * kRowHeads;
    const int slot = (int)(blockIdx.x / hb);
    GdnChunk c;
    if (!gdn_find_chunk(p, slot, c)) return;
    for (int e = threadIdx.x; e < L * kRowHeads; e += 32 * kRowHeads) {
        const int r = e / kRowHeads, k = e % kRowHeads;
        const bool in = r < c.nr && hv0 + k < p.HV;
        const int64_t at = (c.r0 + r) * p.HV + hv0 + k;
        gs[k][r] = in ? p.g[at] : 0.f;
        bs[k][r] = in ? to_f32(static_cast<const T *>(p.beta)[at]) : 0.f;
    }
    __syncthreads();
    const int lane = threadIdx.x & 31, hl = threadIdx.x >> 5, hv = hv0 + hl, h = hv / (p.HV / p.H);
    if (hv >= p.HV) return;
    float a[PER], lo[PER], rk[PER], rq[PER], be[PER];
    const GdnRows rd(p, (int64_t)slot * p.HV + hv);
#pragma unroll
    for (int k = 0; k < PER; ++k) {
        const int r = PER * lane + k;
        const bool in = r < c.nr;
        const float g = gs[hl][r];
        a[k] = g * p.g_scale;
        lo[k] = fmaf(g, p.g_scale, -a[k]);
        if (a[k] < kReset) {
            a[k] = kReset;
            lo[k] = 0.f;
        }
        float2 n = make_float2(1.f, 1.f);
        if (in && p.l2) n = *reinterpret_cast<const float2 *>(p.norms + ((c.r0 + r) * p.H + h) * 2);
        rk[k] = in ? n.y : 0.f;
        be[k] = bs[hl][r];
        rq[k] = in ? p.scale * n.x : 0.f;
        if (k > 0) pair_add(a[k], lo[k], a[k - 1], lo[k - 1]);
    }
    float sh = a[PER - 1], sl = lo[PER - 1];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const float uh = __shfl_up_sync(0xffffffffu, sh, o), ul = __shfl_up_sync(0xffffffffu, sl, o);
        if (lane >= o) pair_add(sh, sl, uh, ul);
    }
    const float eh = __shfl_sync(0xffffffffu, sh, 31), el = __shfl_sync(0xffffffffu, sl, 31);
    const float ph = __shfl_up_sync(0xffffffffu, sh, 1), pl = __shfl_up_sync(0xffffffffu, sl, 1);
#pragma unroll
    for (int k = 0; k < PER; ++k)
        if (lane > 0) pair_add(a[k], lo[k], ph, pl);
    // the last row of the block of 16
    constexpr int BL = 16 / PER;  // lanes of a block
    const float rh = __shfl_sync(0xffffffffu, a[PER - 1], lane | (BL - 1));
    const float rl = __shfl_sync(0xffffffffu, lo[PER - 1], lane | (BL - 1));
    float cs[PER], es[PER], fd[PER];
#pragma unroll
    for (int k = 0; k < PER; ++k) {
        cs[k] = ex2_ftz(a[k] + lo[k]);
        es[k] = ex2_ftz((eh - a[k]) + (el - lo[k]));
        fd[k] = ex2_ftz((rh - a[k]) + (rl - lo[k])) * rk[k];
    }
    auto put = [&](int array, const float (&x)[PER]) {
        float *to = rd.at + array * L + PER * lane;
        if constexpr (PER == 4)
            *reinterpret_cast<float4 *>(to) = make_float4(x[0], x[1], x[2], x[3]);
        else
            to[0] = x[0];
    };
    put(0, a);
    put(1, lo);
    put(2, cs);
    put(3, es);
    put(4, be);
    put(5, rq);
    put(6, rk);
    put(7, fd);
}

// ------------------------------------------------------- CUDA cores: a chunk's matrices
// Chunks of 32 rows, and 32 value columns at a time: what all chunks can do at once stands in kernels of its
// own (the matrices here, the outputs, the gradients), so that the pass over a sequence's chunks has two
// products to a chunk left.  Everything between the kernels is fp32: per unit W = M diag(beta c rk) K and
// diag(e rk) K, both [32][K up to a multiple of 4]; per unit and 32 columns U0 = M diag(beta) V in U's
// place, the state at the chunk's start, and in the gradients dU and E likewise.
__device__ __forceinline__ int simt_kp(const GdnArgs &p) { return (p.K + 3) & ~3; }
__device__ __forceinline__ int simt_tiles(const GdnArgs &p) { return (p.V + kVT - 1) / kVT; }
__device__ __forceinline__ int64_t simt_u(const GdnArgs &p, int64_t unit, int tile) {
    return (unit * simt_tiles(p) + tile) * (kGL * kVT);
}
__device__ __forceinline__ int64_t simt_s(const GdnArgs &p, int64_t unit, int tile) {
    return (unit * simt_tiles(p) + tile) * (int64_t)(p.K * kVT);
}
// `rows` rows (zeros past nr) of `cols` columns (past `have`: zeros) into shared memory, rows `pitch` floats
// apart, each row times f[row] (null: 1).
template <typename T>
__device__ __forceinline__ void load_tile(float *to, int pitch, const T *from, int64_t stride, int rows, int nr,
                                          int cols, int have, const float *f = nullptr) {
    for (int r = threadIdx.x >> 5; r < rows; r += blockDim.x >> 5)
#pragma unroll 4
        for (int c = threadIdx.x & 31; c < cols; c += 32) {
            const float x = r < nr && c < have ? to_f32(from[r * stride + c]) : 0.f;
            to[r * pitch + c] = f ? x * f[r] : x;
        }
}
__device__ __forceinline__ float4 f4(const float *p) { return *reinterpret_cast<const float4 *>(p); }
__device__ __forceinline__ void axpy(float (&y)[4], float a, const float4 &x) {
    y[0] = fmaf(a, x.x, y[0]);
    y[1] = fmaf(a, x.y, y[1]);
    y[2] = fmaf(a, x.z, y[2]);
    y[3] = fmaf(a, x.w, y[3]);
}

// t[m] += x[m] y.
__device__ __forceinline__ void add_tile(float (&t)[4][4], const float4 &x, const float4 &y) {
    axpy(t[0], x.x, y);
    axpy(t[1], x.y, y);
    axpy(t[2], x.z, y);
    axpy(t[3], x.w, y);
}
__device__ __forceinline__ float dot4(const float4 &a, const float4 &b, float s) {
    return fmaf(a.w, b.w, fmaf(a.z, b.z, fmaf(a.y, b.y, fmaf(a.x, b.x, s))));
}

template <typename T>
__global__ void __launch_bounds__(kThreads) gdn_simt_mats_kernel(GdnArgs p) {
    extern __shared__ __align__(16) float sm[];
    const int64_t unit = blockIdx.x;
    const int slot = (int)blockIdx.x / p.HV, hv = (int)blockIdx.x % p.HV, h = hv / (p.HV / p.H), tid = threadIdx.x;
    GdnChunk c;
    if (!gdn_find_chunk(p, slot, c)) return;
    const int kp = simt_kp(p), pitch = kp + 4;
    float *ks = sm, *qs = ks + kGL * pitch, *ns = qs + kGL * pitch;  // ns [kGL][kGL + 1]
    float *vs = ns + kGL * (kGL + 1);                                // [kGL][kVT + 4]
    load_tile(ks, pitch, static_cast<const T *>(p.k) + c.r0 * p.k_stride + (int64_t)h * p.K, p.k_stride, kGL, c.nr, kp,
              p.K);
    load_tile(qs, pitch, static_cast<const T *>(p.q) + c.r0 * p.q_stride + (int64_t)h * p.K, p.q_stride, kGL, c.nr, kp,
              p.K);
    __syncthreads();
    const GdnRows rd(p, unit);
    float *M = p.mats + unit * 3 * kGL * kGL, *A = M + kGL * kGL, *P = A + kGL * kGL;
    {  // two rows and two columns of the grams a thread
        const int i0 = tid >> 4, j0 = tid & 15;
        float kk[2][2] = {}, qk[2][2] = {};
#pragma unroll 4
        for (int d = 0; d < kp; d += 4) {
            float4 ki[2], qi[2], kj[2];
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                ki[m] = f4(ks + (i0 + 16 * m) * pitch + d);
                qi[m] = f4(qs + (i0 + 16 * m) * pitch + d);
                kj[m] = f4(ks + (j0 + 16 * m) * pitch + d);
            }
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    kk[m][n] = dot4(ki[m], kj[n], kk[m][n]);
                    qk[m][n] = dot4(qi[m], kj[n], qk[m][n]);
                }
        }
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                const int i = i0 + 16 * m, j = j0 + 16 * n;
                const float w = j <= i ? ex2_ftz((rd.a[i] - rd.a[j]) + (rd.lo[i] - rd.lo[j])) * rd.rk[j] : 0.f;
                const float x = j < i ? kk[m][n] * w * rd.rk[i] : 0.f;
                ns[i * (kGL + 1) + j] = x * rd.b[i];
                A[i * kGL + j] = x;
                P[i * kGL + j] = j <= i ? qk[m][n] * (w * rd.rq[i]) : 0.f;
            }
    }
    __syncthreads();
    if (tid < kGL) {  // column j of M by substitution, over N's rows as they are done with
        const int j = tid;
        float m[kGL];
#pragma unroll
        for (int i = 0; i < kGL; ++i) {
            float x = i == j ? 1.f : 0.f;
#pragma unroll
            for (int l = 0; l < i; ++l) x = fmaf(-ns[i * (kGL + 1) + l], m[l], x);
            m[i] = x;
            M[i * kGL + j] = x;
            __syncwarp();
            ns[i * (kGL + 1) + j] = x;
        }
    }
    float *W = p.wk + unit * 2 * kGL * kp, *Kt = W + kGL * kp;
    for (int r = tid >> 5; r < kGL; r += kThreads / 32) {  // diag(e rk) K, and beta c rk K in K's place
        const float e = rd.e[r] * rd.rk[r], f = rd.b[r] * rd.c[r] * rd.rk[r];
        for (int d = tid & 31; d < kp; d += 32) {
            const float x = ks[r * pitch + d];
            Kt[r * kp + d] = x * e;
            ks[r * pitch + d] = x * f;
        }
    }
    __syncthreads();
    for (int e = tid; e < kGL / 4 * (kp / 4); e += kThreads) {  // four rows and columns of W
        const int i = e % (kGL / 4) * 4, d = e / (kGL / 4) * 4;
        float x[4][4] = {};
#pragma unroll 8
        for (int j = 0; j < kGL; ++j) {
            const float4 y = f4(ks + j * pitch + d);
#pragma unroll
            for (int m = 0; m < 4; ++m) axpy(x[m], ns[(i + m) * (kGL + 1) + j], y);
        }
#pragma unroll
        for (int m = 0; m < 4; ++m) *reinterpret_cast<float4 *>(W + (i + m) * kp + d) = make_float4(x[m][0], x[m][1], x[m][2], x[m][3]);
    }
    const int r = tid >> 3, c4 = (tid & 7) * 4;
    for (int tile = 0; tile < simt_tiles(p); ++tile) {
        const int v0 = tile * kVT;
        __syncthreads();
        load_tile(vs, kVT + 4, static_cast<const T *>(p.v) + c.r0 * p.v_stride + (int64_t)hv * p.V + v0, p.v_stride, kGL,
                  c.nr, kVT, p.V - v0, rd.b);
        __syncthreads();
        float u[4] = {};
#pragma unroll 8
        for (int j = 0; j < kGL; ++j) axpy(u, ns[r * (kGL + 1) + j], f4(vs + j * (kVT + 4) + c4));
        *reinterpret_cast<float4 *>(p.us + simt_u(p, unit, tile) + r * kVT + c4) = make_float4(u[0], u[1], u[2], u[3]);
    }
}

// ------------------------------------------------------- CUDA cores: the pass over chunks
// One block per (sequence, value head, 32 value columns), its columns of the state in shared memory, the
// next two chunks' matrices on their way there.
//   forward  U = U0 - W S;                  S' = 2^{a_end} S + K^T diag(e rk) U
//   reverse  dU = dU0 + diag(e rk) K E;     E' = 2^{a_end} E + B0 - W^T dU
// Bound by the reads of shared memory, 4 cycles for a warp's 512 bytes: a thread has two rows and four columns
// of the first product (half of the threads) and four rows and four columns of the second.  2 x 777 rows of 6
// heads, 40 keys: 43 us and 41 us (with a row and four columns each 63 and 66).  Four chunks ahead in place of two
// changed nothing.
template <bool REV>
__global__ void __launch_bounds__(kThreads) gdn_simt_scan_kernel(GdnArgs p) {
    extern __shared__ __align__(16) float sm[];
    __shared__ uint64_t full[2];
    __shared__ int gone;
    volatile int *dead = &gone;
    const int vt = simt_tiles(p), kp = simt_kp(p), tile = (int)(blockIdx.x % vt), v0 = tile * kVT;
    const int64_t sh = blockIdx.x / vt;
    const int hv = (int)(sh % p.HV), seq = (int)(sh / p.HV);
    int64_t first, row;
    int nc, len;
    if (!gdn_sequence(p, seq, first, nc, row, len)) return;
    const int tid = threadIdx.x, r = tid >> 3, c4 = (tid & 7) * 4, nv = p.V - v0 - c4;
    const int per = 2 * kGL * kp + kGL * kVT;  // floats of a chunk
    float *S = sm, *U = S + kp * kVT, *bufs = U + kGL * kVT;
    float *rows = REV ? p.zs : p.us, *keep = REV ? p.dstates : p.states;
    auto unit_of = [&](int n) { return (first + (REV ? nc - 1 - n : n)) * p.HV + hv; };
    int last = -1;  // the chunk asked for last (thread 0)
    auto fetch = [&](int n) {
        last = n;
        float *to = bufs + (n & 1) * per;
        tc::mbar_arrive_expect_tx(&full[n & 1], per * 4);
        tc::bulk_g2s(to, p.wk + unit_of(n) * 2 * kGL * kp, 2 * kGL * kp * 4, &full[n & 1]);
        tc::bulk_g2s(to + 2 * kGL * kp, rows + simt_u(p, unit_of(n), tile), kGL * kVT * 4, &full[n & 1]);
    };
    if (tid == 0) {
        tc::mbar_init(&full[0], 1);
        tc::mbar_init(&full[1], 1);
        tc::mbar_fence_init();
        gone = p.give_up;  // (here, where it takes no time: the rounds are 1.7 us)
        if (p.give_up) report(p.status, KDA_DEVICE_TIMEOUT);
        for (int n = 0; n < 2 && n < nc; ++n) fetch(n);
    }
    // the thread's part of the state: rows 4 r + 128 m and the three after, columns c4 and the three after
    constexpr int M = 2;  // K <= 256
    const float *from = REV ? p.dht : p.h0;
    const int64_t user = sh * p.K * p.V + v0 + c4;
#pragma unroll
    for (int m = 0; m < M; ++m)
        for (int d = 4 * r + 128 * m; d < min(kp, 4 * r + 128 * m + 4); ++d)
#pragma unroll
            for (int k = 0; k < 4; ++k)
                S[d * kVT + c4 + k] = from && d < p.K && k < nv ? from[user + (int64_t)d * p.V + k] : 0.f;
    float kept = nc > 0 ? GdnRows(p, unit_of(0)).c[kGL - 1] : 0.f;
    __syncthreads();
    for (int n = 0; n < nc; ++n) {
        const int64_t unit = unit_of(n);
        const float *w = bufs + (n & 1) * per, *k = w + kGL * kp, *t0 = k + kGL * kp;
        const float kept_next = n + 1 < nc ? GdnRows(p, unit_of(n + 1)).c[kGL - 1] : 0.f;
        float *at = keep + simt_s(p, unit, tile) + c4;
        float4 b0[REV ? M : 1][4];
#pragma unroll
        for (int m = 0; m < M; ++m)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int d = 4 * r + 128 * m + i;
                if (d < p.K) {
                    if (REV) b0[m][i] = f4(at + d * kVT);
                    *reinterpret_cast<float4 *>(at + d * kVT) = f4(S + d * kVT + c4);
                }
            }
        wait_or_die(&full[n & 1], n >> 1 & 1, dead, p.status);
        if (r < kGL / 2) {
            const float *left = (REV ? k : w) + 2 * r * kp;
            float y[2][4] = {};
#pragma unroll 5
            for (int d = 0; d < kp; d += 4) {
                const float4 x0 = f4(left + d), x1 = f4(left + kp + d);
                const float *sd = S + d * kVT + c4;
                const float4 s0 = f4(sd), s1 = f4(sd + kVT), s2 = f4(sd + 2 * kVT), s3 = f4(sd + 3 * kVT);
                axpy(y[0], x0.x, s0); axpy(y[1], x1.x, s0);
                axpy(y[0], x0.y, s1); axpy(y[1], x1.y, s1);
                axpy(y[0], x0.z, s2); axpy(y[1], x1.z, s2);
                axpy(y[0], x0.w, s3); axpy(y[1], x1.w, s3);
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int e = (2 * r + i) * kVT + c4;
                float4 u = f4(t0 + e);
                u = REV ? make_float4(u.x + y[i][0], u.y + y[i][1], u.z + y[i][2], u.w + y[i][3])
                        : make_float4(u.x - y[i][0], u.y - y[i][1], u.z - y[i][2], u.w - y[i][3]);
                *reinterpret_cast<float4 *>(U + e) = u;
                *reinterpret_cast<float4 *>(rows + simt_u(p, unit, tile) + e) = u;
            }
        }
        __syncthreads();
        const float *right = REV ? w : k;
#pragma unroll
        for (int m = 0; m < M; ++m) {
            const int d = 4 * r + 128 * m;
            if (d >= kp) break;
            float z[4][4] = {};
#pragma unroll 16
            for (int j = 0; j < kGL; ++j) {
                const float4 x = f4(right + j * kp + d), u = f4(U + j * kVT + c4);
                axpy(z[0], x.x, u);
                axpy(z[1], x.y, u);
                axpy(z[2], x.z, u);
                axpy(z[3], x.w, u);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (d + i >= p.K) break;
                float4 x = f4(S + (d + i) * kVT + c4);
                float b[4] = {z[i][0], z[i][1], z[i][2], z[i][3]};
                if (REV) {
                    b[0] = b0[m][i].x - b[0]; b[1] = b0[m][i].y - b[1];
                    b[2] = b0[m][i].z - b[2]; b[3] = b0[m][i].w - b[3];
                }
                axpy(b, kept, x);
                *reinterpret_cast<float4 *>(S + (d + i) * kVT + c4) = make_float4(b[0], b[1], b[2], b[3]);
            }
        }
        kept = kept_next;
        __syncthreads();
        if (tid == 0 && n + 2 < nc && !*dead) fetch(n + 2);
    }
    float *to = REV ? p.dh0 : p.ht;
    if (to)
#pragma unroll
        for (int m = 0; m < M; ++m)
            for (int d = 4 * r + 128 * m; d < min(p.K, 4 * r + 128 * m + 4); ++d)
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (k < nv) to[user + (int64_t)d * p.V + k] = S[d * kVT + c4 + k];
    if (tid == 0 && *dead)  // copies may still be on their way here
        for (int n = last > 0 ? last - 1 : 0; n <= last; ++n) tc::mbar_wait(&full[n & 1], n >> 1 & 1, 10000000ull);
}

// ------------------------------------------------------- CUDA cores: outputs, and what they give
// O = diag(rq c) Q S + P U of a chunk and 32 value columns: all threads load, half of them have two rows and
// four columns each.
template <typename T>
__global__ void __launch_bounds__(kThreads) gdn_simt_out_kernel(GdnArgs p) {
    extern __shared__ __align__(16) float sm[];
    const int64_t unit = blockIdx.x;
    const int slot = (int)blockIdx.x / p.HV, hv = (int)blockIdx.x % p.HV, h = hv / (p.HV / p.H);
    const int tile = blockIdx.y, v0 = tile * kVT;
    GdnChunk c;
    if (!gdn_find_chunk(p, slot, c)) return;
    const int tid = threadIdx.x, r = (tid >> 3) * 2, c4 = (tid & 7) * 4, kp = simt_kp(p), pitch = kp + 4;
    float *qs = sm, *S = qs + kGL * pitch, *U = S + kp * kVT, *Ps = U + kGL * kVT;  // Ps [kGL][kGL + 1]
    load_tile(qs, pitch, static_cast<const T *>(p.q) + c.r0 * p.q_stride + (int64_t)h * p.K, p.q_stride, kGL, c.nr, kp, p.K);
    const float *st = p.states + simt_s(p, unit, tile), *us = p.us + simt_u(p, unit, tile);
    for (int e = tid * 4; e < kp * kVT; e += kThreads * 4)
        *reinterpret_cast<float4 *>(S + e) = e < p.K * kVT ? f4(st + e) : make_float4(0.f, 0.f, 0.f, 0.f);
    for (int e = tid * 4; e < kGL * kVT; e += kThreads * 4) *reinterpret_cast<float4 *>(U + e) = f4(us + e);
    for (int e = tid; e < kGL * kGL; e += kThreads)
        Ps[e / kGL * (kGL + 1) + e % kGL] = p.mats[unit * 3 * kGL * kGL + 2 * kGL * kGL + e];
    __syncthreads();
    if (r >= kGL) return;
    const GdnRows rd(p, unit);
    float o[2][4] = {};
#pragma unroll 4
    for (int d = 0; d < kp; d += 4) {
        const float4 x0 = f4(qs + r * pitch + d), x1 = f4(qs + (r + 1) * pitch + d);
        const float *sd = S + d * kVT + c4;
        const float4 s0 = f4(sd), s1 = f4(sd + kVT), s2 = f4(sd + 2 * kVT), s3 = f4(sd + 3 * kVT);
        axpy(o[0], x0.x, s0); axpy(o[1], x1.x, s0);
        axpy(o[0], x0.y, s1); axpy(o[1], x1.y, s1);
        axpy(o[0], x0.z, s2); axpy(o[1], x1.z, s2);
        axpy(o[0], x0.w, s3); axpy(o[1], x1.w, s3);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const float f = rd.c[r + i] * rd.rq[r + i];
#pragma unroll
        for (int k = 0; k < 4; ++k) o[i][k] *= f;
    }
#pragma unroll 8
    for (int j = 0; j < kGL; ++j) {
        const float4 u = f4(U + j * kVT + c4);
        axpy(o[0], Ps[r * (kGL + 1) + j], u);
        axpy(o[1], Ps[(r + 1) * (kGL + 1) + j], u);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (r + i < c.nr && v0 + c4 + k < p.V)
                static_cast<T *>(p.o)[((c.r0 + r + i) * p.HV + hv) * p.V + v0 + c4 + k] = from_f32<T>(o[i][k]);
}

// dU0 = P^T dO and B0 = Q^T diag(rq c) dO of a chunk and 32 value columns, in dU's and E's places.
template <typename T>
__global__ void __launch_bounds__(kThreads) gdn_simt_base_kernel(GdnArgs p) {
    extern __shared__ __align__(16) float sm[];
    const int64_t unit = blockIdx.x;
    const int slot = (int)blockIdx.x / p.HV, hv = (int)blockIdx.x % p.HV, h = hv / (p.HV / p.H);
    const int tile = blockIdx.y, v0 = tile * kVT;
    GdnChunk c;
    if (!gdn_find_chunk(p, slot, c)) return;
    const int tid = threadIdx.x, r = tid >> 3, c4 = (tid & 7) * 4, kp = simt_kp(p);
    float *D = sm, *Ps = D + kGL * kVT, *f = Ps + kGL * kGL, *qs = f + kGL;
    const GdnRows rd(p, unit);
    if (tid < kGL) f[tid] = rd.c[tid] * rd.rq[tid];
    for (int e = tid; e < kGL * kGL; e += kThreads) Ps[e] = p.mats[unit * 3 * kGL * kGL + 2 * kGL * kGL + e];
    load_tile(D, kVT, static_cast<const T *>(p.dout) + (c.r0 * p.HV + hv) * p.V + v0, (int64_t)p.HV * p.V, kGL, c.nr, kVT,
              p.V - v0);
    __syncthreads();
    load_tile(qs, kp, static_cast<const T *>(p.q) + c.r0 * p.q_stride + (int64_t)h * p.K, p.q_stride, kGL, c.nr, kp, p.K, f);
    __syncthreads();
    if (r < kGL / 2) {
        float y[2][4] = {};
#pragma unroll 8
        for (int i = 0; i < kGL; ++i) {
            const float4 x = f4(D + i * kVT + c4);
            axpy(y[0], Ps[i * kGL + 2 * r], x);
            axpy(y[1], Ps[i * kGL + 2 * r + 1], x);
        }
        float *to = p.zs + simt_u(p, unit, tile) + 2 * r * kVT + c4;
#pragma unroll
        for (int i = 0; i < 2; ++i)
            *reinterpret_cast<float4 *>(to + i * kVT) = make_float4(y[i][0], y[i][1], y[i][2], y[i][3]);
    }
    for (int d = 4 * r; d < kp; d += kThreads / 2) {
        float z[4][4] = {};
#pragma unroll 8
        for (int i = 0; i < kGL; ++i) {
            const float4 x = f4(qs + i * kp + d), y = f4(D + i * kVT + c4);
            axpy(z[0], x.x, y);
            axpy(z[1], x.y, y);
            axpy(z[2], x.z, y);
            axpy(z[3], x.w, y);
        }
        float *to = p.dstates + simt_s(p, unit, tile) + c4;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (d + i < p.K)
                *reinterpret_cast<float4 *>(to + (d + i) * kVT) = make_float4(z[i][0], z[i][1], z[i][2], z[i][3]);
    }
}

// ------------------------------------------------------- CUDA cores: a chunk's gradients
// A warp has four rows, a lane one column of a [32][32] product or four of a [32][128] one: a row's values are
// the same address for the whole warp, and the sums over a row's columns stay in the warp.  Operands that
// are read by row lie transposed ([contracted][row]).
constexpr int kTP = kGL + 4;  // pitch of the transposed tiles
struct GradSmem {
    float Ut[kVT][kTP], Zt[kVT][kTP], Dt[kVT][kTP];  // [value column][row]
    float dU[kGL][kVT], M[kGL][kTP];
    float X[kGL][kTP], XT[kGL][kTP], Y[kGL][kTP];    // XT: X transposed; Y with its mirror image
    float F[kGL][kGL + 1];                           // the pairs' shares of dg, summed up to each column
    float St[kVT][kKT + 4], Et[kVT][kKT + 4], qs[kGL][kKT + 4], ks[kGL][kKT + 4];
    float dots[2][kGL], wsum[kThreads / 32];
};
static_assert(2 * (sizeof(GradSmem) + 1024) <= 233472, "an SM's shared memory");
template <typename T>
__global__ void __launch_bounds__(kThreads, 2) gdn_simt_grad_kernel(GdnArgs p) {
    extern __shared__ __align__(16) float sm[];
    GradSmem &s = *reinterpret_cast<GradSmem *>(sm);
    const int64_t unit = blockIdx.x;
    const int slot = (int)blockIdx.x / p.HV, hv = (int)blockIdx.x % p.HV, h = hv / (p.HV / p.H);
    GdnChunk c;
    if (!gdn_find_chunk(p, slot, c)) return;
    const GdnRows rd(p, unit);
    const int tid = threadIdx.x, lane = tid & 31, i0 = (tid >> 5) * 4;  // the warp's first row
    const float *A = p.mats + unit * 3 * kGL * kGL + kGL * kGL, *P = A + kGL * kGL;
    const T *dout = static_cast<const T *>(p.dout) + (c.r0 * p.HV + hv) * p.V;
    const T *v = static_cast<const T *>(p.v) + c.r0 * p.v_stride + (int64_t)hv * p.V;
    auto load_ud = [&](int v0) {
        const float *from = p.us + simt_u(p, unit, v0 / kVT);
        for (int e = tid; e < kGL * kVT; e += kThreads) {
            const int r = e / kVT, j = e % kVT;
            s.Ut[j][r] = from[e];
            s.Dt[j][r] = v0 + j < p.V && r < c.nr ? to_f32(dout[(int64_t)r * p.HV * p.V + v0 + j]) : 0.f;
        }
    };
    for (int e = tid; e < kGL * kGL; e += kThreads) s.M[e / kGL][e % kGL] = p.mats[unit * 3 * kGL * kGL + e];
    float ci[4], bi[4], rq[4], rk[4];
#pragma unroll
    for (int m = 0; m < 4; ++m) {
        ci[m] = rd.c[i0 + m];
        bi[m] = rd.b[i0 + m];
        rq[m] = rd.rq[i0 + m];
        rk[m] = rd.rk[i0 + m];
    }
    float gm[4] = {}, hm[4] = {}, zv[4] = {};  // Z U^T, dO U^T at column `lane`; the rows' shares of dbeta
    for (int v0 = 0; v0 < p.V; v0 += kVT) {
        float *zs = p.zs + simt_u(p, unit, v0 / kVT);
        __syncthreads();
        load_ud(v0);
        for (int e = tid; e < kGL * kVT; e += kThreads) s.dU[e / kVT][e % kVT] = zs[e];
        __syncthreads();
        float z[4] = {};  // Z = M^T dU, over dU for the rounds below, and dv
#pragma unroll 8
        for (int r = 0; r < kGL; ++r) axpy(z, s.dU[r][lane], f4(&s.M[r][i0]));
        *reinterpret_cast<float4 *>(&s.Zt[lane][i0]) = make_float4(z[0], z[1], z[2], z[3]);
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            const int i = i0 + m;
            zs[i * kVT + lane] = z[m];
            if (i < c.nr && v0 + lane < p.V) {
                zv[m] = fmaf(z[m], to_f32(v[i * p.v_stride + v0 + lane]), zv[m]);
                static_cast<T *>(p.dv)[((c.r0 + i) * p.HV + hv) * p.V + v0 + lane] = from_f32<T>(bi[m] * z[m]);
            }
        }
        __syncthreads();
#pragma unroll 8
        for (int j = 0; j < kVT; ++j) {
            const float u = s.Ut[j][lane];
            axpy(gm, u, f4(&s.Zt[j][i0]));
            axpy(hm, u, f4(&s.Dt[j][i0]));
        }
    }
    float x[4];
#pragma unroll
    for (int m = 0; m < 4; ++m) {
        const int i = i0 + m, j = lane;
        const bool on = j <= i;
        const float w = on ? ex2_ftz((rd.a[i] - rd.a[j]) + (rd.lo[i] - rd.lo[j])) : 0.f;
        const float a = on ? A[i * kGL + j] : 0.f, pv = on ? P[i * kGL + j] : 0.f;
        x[m] = on ? hm[m] * w : 0.f;
        s.X[i][j] = x[m];
        if (on) s.Y[i][j] = s.Y[j][i] = j < i ? -bi[m] * gm[m] * w : 0.f;
        float f = on ? hm[m] * pv - bi[m] * gm[m] * a : 0.f;
        if (on) zv[m] = fmaf(-a, gm[m], zv[m]);
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const float before = __shfl_up_sync(0xffffffffu, f, o);
            if (lane >= o) f += before;
        }
        f = __shfl_up_sync(0xffffffffu, f, 1);
        s.F[i][j] = lane > 0 ? f : 0.f;
    }
    *reinterpret_cast<float4 *>(&s.XT[lane][i0]) = make_float4(x[0], x[1], x[2], x[3]);
    float crow[4] = {}, erow[4] = {}, es = 0.f;  // the rows' sums: of pairs' ends i >= t, and j < t; <S, E>
    const T *qp = static_cast<const T *>(p.q) + c.r0 * p.q_stride + (int64_t)h * p.K;
    const T *kp = static_cast<const T *>(p.k) + c.r0 * p.k_stride + (int64_t)h * p.K;
    for (int k0 = 0; k0 < p.K; k0 += kKT) {
        const int nk = min(kKT, p.K - k0), d0 = 4 * lane;
        float ds[4][4] = {}, zs[4][4] = {}, ue[4][4] = {};
        for (int v0 = 0; v0 < p.V; v0 += kVT) {
            __syncthreads();
            load_ud(v0);
            const float *z = p.zs + simt_u(p, unit, v0 / kVT);
            for (int e = tid; e < kGL * kVT; e += kThreads) s.Zt[e % kVT][e / kVT] = z[e];
            const int64_t at = simt_s(p, unit, v0 / kVT) + (int64_t)k0 * kVT;
            for (int e = tid; e < (nk + 3) / 4 * 4 * kVT; e += kThreads) {
                const bool in = e < nk * kVT;
                const float st = in ? p.states[at + e] : 0.f, y = in ? p.dstates[at + e] : 0.f;
                s.St[e % kVT][e / kVT] = st;
                s.Et[e % kVT][e / kVT] = y;
                es = fmaf(st, y, es);
            }
            __syncthreads();
            if (d0 < nk)
#pragma unroll 4
                for (int j = 0; j < kVT; ++j) {
                    const float4 st = f4(&s.St[j][d0]), y = f4(&s.Et[j][d0]);
                    add_tile(ds, f4(&s.Dt[j][i0]), st);
                    add_tile(zs, f4(&s.Zt[j][i0]), st);
                    add_tile(ue, f4(&s.Ut[j][i0]), y);
                }
        }
        load_tile(&s.qs[0][0], kKT + 4, qp + k0, p.q_stride, kGL, c.nr, (nk + 3) / 4 * 4, nk, rd.rq);
        load_tile(&s.ks[0][0], kKT + 4, kp + k0, p.k_stride, kGL, c.nr, (nk + 3) / 4 * 4, nk, rd.rk);
        __syncthreads();
        if (d0 >= nk) continue;
#pragma unroll
        for (int m = 0; m < 4; ++m) {  // dq into ds, dk into ue
            const float4 q4 = f4(&s.qs[i0 + m][d0]), k4 = f4(&s.ks[i0 + m][d0]);
            const float q[4] = {q4.x, q4.y, q4.z, q4.w}, kk[4] = {k4.x, k4.y, k4.z, k4.w};
            const float ei = rd.e[i0 + m];
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                const float cz = -ci[m] * zs[m][n], kz = bi[m] * cz, ke = ei * ue[m][n];
                ds[m][n] *= ci[m];
                ue[m][n] = kz + ke;
                crow[m] = fmaf(q[n], ds[m][n], fmaf(kk[n], kz, crow[m]));
                erow[m] = fmaf(kk[n], ke, erow[m]);
                zv[m] = fmaf(kk[n], cz, zv[m]);
            }
        }
#pragma unroll 4
        for (int j = 0; j < kGL; ++j) {
            const float4 q = f4(&s.qs[j][d0]), kk = f4(&s.ks[j][d0]);
            add_tile(ds, f4(&s.XT[j][i0]), kk);
            add_tile(ue, f4(&s.X[j][i0]), q);
            add_tile(ue, f4(&s.Y[j][i0]), kk);
        }
#pragma unroll
        for (int m = 0; m < 4; ++m)
            if (i0 + m < c.nr)
#pragma unroll
                for (int n = 0; n < 4; ++n)
                    if (d0 + n < nk) {
                        const int64_t at = ((c.r0 + i0 + m) * p.HV + hv) * p.K + k0 + d0 + n;
                        p.dqh[at] = ds[m][n] * rq[m];
                        p.dkh[at] = ue[m][n] * rk[m];
                    }
    }
    es = lane_sum<32>(es);
    if (lane == 0) s.wsum[tid >> 5] = es;
#pragma unroll
    for (int m = 0; m < 4; ++m) {
        const float cr = lane_sum<32>(crow[m]), er = lane_sum<32>(erow[m]), db = lane_sum<32>(zv[m]);
        if (lane == 0) {
            s.dots[0][i0 + m] = cr;
            s.dots[1][i0 + m] = er;
            if (i0 + m < c.nr) static_cast<T *>(p.dbeta)[(c.r0 + i0 + m) * p.HV + hv] = from_f32<T>(db);
        }
    }
    __syncthreads();
    if (tid < c.nr) {
        const int t = tid;
        float sum = 0.f;
        for (int w = 0; w < kThreads / 32; ++w) sum += s.wsum[w];
        sum *= rd.c[kGL - 1];
        for (int j = 0; j < t; ++j) sum += s.dots[1][j];
        for (int r = t; r < kGL; ++r) sum += s.dots[0][r] + s.F[r][t];
        p.dg[(c.r0 + t) * p.HV + hv] = sum * 0.6931471805599453f * p.g_scale;
    }
}

// dq and dk of a row from its value heads' shares, which have the rows' factors in them: their sum,
// less the norm's projection x (x . d) / |x|^2; zeros in rows outside every sequence.  A warp per
// (row, head).  Bound by HBM: the shares are read once in fp32.
template <typename T, int VEC>  // VEC columns at a time: 4 where K is a multiple of it
__global__ void __launch_bounds__(kThreads) gdn_finish_kernel(GdnArgs p) {
    constexpr int NV = 8 / VEC;  // K <= 256
    const uint32_t unit = blockIdx.x * (uint32_t)(kThreads / 32) + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31, per = p.HV / p.H;
    if (unit >= (uint32_t)p.B * (uint32_t)p.T * (uint32_t)p.H) return;
    const int64_t id = unit, r = unit / (uint32_t)p.H;
    const int h = (int)(unit % (uint32_t)p.H);
    const bool in = !p.cu || (p.ctrl->valid && r < p.cu[p.N]);
    const T *x[2] = {static_cast<const T *>(p.q) + r * p.q_stride + (int64_t)h * p.K,
                     static_cast<const T *>(p.k) + r * p.k_stride + (int64_t)h * p.K};
    T *to[2] = {static_cast<T *>(p.dq) + id * p.K, static_cast<T *>(p.dk) + id * p.K};
    const float *from[2] = {p.dqh + (r * p.HV + (int64_t)h * per) * p.K, p.dkh + (r * p.HV + (int64_t)h * per) * p.K};
    float d[2][NV][VEC] = {}, v[2][NV][VEC] = {}, dot[2] = {};
    if (in)
        for (int m = 0; m < per; ++m)
#pragma unroll
            for (int s = 0; s < 2; ++s)
#pragma unroll
                for (int k = 0; k < NV; ++k) {
                    const int c = (lane + 32 * k) * VEC;
                    if (c >= p.K) continue;
                    float y[VEC];
                    if constexpr (VEC == 4) {
                        const float4 f = f4(from[s] + (int64_t)m * p.K + c);
                        y[0] = f.x; y[1] = f.y; y[2] = f.z; y[3] = f.w;
                    } else {
                        y[0] = from[s][(int64_t)m * p.K + c];
                    }
#pragma unroll
                    for (int e = 0; e < VEC; ++e) d[s][k][e] += y[e];
                }
    if (in && p.l2) {
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const float n = p.norms[id * 2 + s];
#pragma unroll
            for (int k = 0; k < NV; ++k)
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    const int c = (lane + 32 * k) * VEC + e;
                    if (c < p.K) v[s][k][e] = to_f32(x[s][c]) * n;
                    dot[s] = fmaf(d[s][k][e], v[s][k][e], dot[s]);
                }
            dot[s] = lane_sum<32>(dot[s]);
        }
    }
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                const int c = (lane + 32 * k) * VEC + e;
                if (c < p.K) to[s][c] = from_f32<T>(fmaf(-dot[s], v[s][k][e], d[s][k][e]));
            }
}

// Zeros in the rows outside every sequence of dv, dg and dbeta, and of dq and dk where the finishing
// kernel did not run.
template <typename T>
__global__ void __launch_bounds__(kThreads) gdn_tail_kernel(GdnArgs p, int qk) {
    const int64_t from = p.ctrl->valid ? p.cu[p.N] : 0, rows = p.T - from;
    const int64_t step = (int64_t)gridDim.x * kThreads, at = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    T *dv = static_cast<T *>(p.dv) + from * p.HV * p.V, *db = static_cast<T *>(p.dbeta) + from * p.HV;
    for (int64_t e = at; e < rows * p.HV * p.V; e += step) dv[e] = from_f32<T>(0.f);
    if (qk)
        for (int64_t e = at; e < rows * p.H * p.K; e += step)
            static_cast<T *>(p.dq)[from * p.H * p.K + e] = static_cast<T *>(p.dk)[from * p.H * p.K + e] = from_f32<T>(0.f);
    for (int64_t e = at; e < rows * p.HV; e += step) {
        db[e] = from_f32<T>(0.f);
        p.dg[from * p.HV + e] = 0.f;
    }
}

// ------------------------------------------------------- single tokens
// One block per (batch row, value head, tile of value columns): a thread keeps four columns of every 8th (or
// 2nd, 4th, 16th, 32nd) state row in registers, so that the state is read and written once.
// o = 2^g S^T q + (q . k) u needs the old state only: one exchange between the warps.
// Bound by HBM: 256 rows of 32 heads of 128 x 128 read and write 1.07 GB in 167 us, 6.4 TB/s; 1024 rows in 642
// us, 6.7 TB/s, the copy's rate.  One row: 7 us, two dependent rounds of loads and the launch.
template <typename T, int LW, int W>  // LW lanes across the columns, W warps (32 W >= K)
__global__ void __launch_bounds__(32 * W) gdn_step_kernel(GdnStepArgs p, int vec) {
    // row groups, columns of a block, rows of a thread
    constexpr int RG = 32 / LW * W, CT = 4 * LW, R = LW;
    static_assert(RG * R == 32 * W, "a warp for every 32 rows");
    __shared__ float qs[32 * W], ks[32 * W];
    __shared__ float part[2][RG][CT + 4];
    __shared__ float wsum[3][W];
    const int vt = (p.V + CT - 1) / CT;
    const int tile = (int)(blockIdx.x % vt);
    const int64_t nh = blockIdx.x / vt;
    const int hv = (int)(nh % p.HV), n = (int)(nh / p.HV), h = hv / (p.HV / p.H);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int cl = tid % LW, rg = tid / LW, col = tile * CT + cl * 4, nc = min(4, p.V - col);
    const int slot = state_slot(p.idx, n, p.slots, p.status);
    T *o = static_cast<T *>(p.o) + nh * p.V;
    if (slot < 0) {
        if (rg == 0)
            for (int j = 0; j < nc; ++j) o[col + j] = from_f32<T>(0.f);
        return;
    }
    float *st = p.state + ((int64_t)slot * p.HV + hv) * p.K * p.V + col;
    float s[R][4];
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const int d = rg + i * RG;
        s[i][0] = s[i][1] = s[i][2] = s[i][3] = 0.f;
        if (d < p.K) {
            if (vec) {
                if (nc > 0) {
                    const float4 x = *reinterpret_cast<const float4 *>(st + (int64_t)d * p.V);
                    s[i][0] = x.x; s[i][1] = x.y; s[i][2] = x.z; s[i][3] = x.w;
                }
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (j < nc) s[i][j] = st[(int64_t)d * p.V + j];
            }
        }
    }
    float qv = 0.f, kv = 0.f;
    if (tid < p.K) {
        qv = to_f32(static_cast<const T *>(p.q)[(int64_t)n * p.q_stride + (int64_t)h * p.K + tid]);
        kv = to_f32(static_cast<const T *>(p.k)[(int64_t)n * p.k_stride + (int64_t)h * p.K + tid]);
    }
    qs[tid] = qv;
    ks[tid] = kv;
    const float qq = lane_sum<32>(qv * qv), kk = lane_sum<32>(kv * kv), qk = lane_sum<32>(qv * kv);
    if (lane == 0) {
        wsum[0][warp] = qq;
        wsum[1][warp] = kk;
        wsum[2][warp] = qk;
    }
    __syncthreads();
    float ya[4] = {}, yb[4] = {};
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const int d = rg + i * RG;
        if (d < p.K) {
            const float kd = ks[d], qd = qs[d];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                ya[j] = fmaf(kd, s[i][j], ya[j]);
                yb[j] = fmaf(qd, s[i][j], yb[j]);
            }
        }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        part[0][rg][cl * 4 + j] = ya[j];
        part[1][rg][cl * 4 + j] = yb[j];
    }
    float s3[3] = {};
#pragma unroll
    for (int w = 0; w < W; ++w)
#pragma unroll
        for (int j = 0; j < 3; ++j) s3[j] += wsum[j][w];
    const float rq = p.l2 ? p.scale / sqrtf(s3[0] + 1e-6f) : p.scale, rk = p.l2 ? 1.f / sqrtf(s3[1] + 1e-6f) : 1.f;
    const float keep = exp2f(p.g[nh] * p.g_scale), beta = to_f32(static_cast<const T *>(p.beta)[nh]);
    __syncthreads();
    float u[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        float a = 0.f, b = 0.f;
#pragma unroll
        for (int w = 0; w < RG; ++w) {
            a += part[0][w][cl * 4 + j];
            b += part[1][w][cl * 4 + j];
        }
        const float v = j < nc ? to_f32(static_cast<const T *>(p.v)[(int64_t)n * p.v_stride + (int64_t)hv * p.V + col + j]) : 0.f;
        u[j] = beta * (v - keep * rk * a);
        if (rg == 0 && j < nc) o[col + j] = from_f32<T>(rq * fmaf(keep, b, s3[2] * rk * u[j]));
        u[j] *= rk;
    }
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const int d = rg + i * RG;
        if (d < p.K) {
            const float kd = ks[d];
#pragma unroll
            for (int j = 0; j < 4; ++j) s[i][j] = fmaf(kd, u[j], keep * s[i][j]);
            if (vec) {
                if (nc > 0) *reinterpret_cast<float4 *>(st + (int64_t)d * p.V) = make_float4(s[i][0], s[i][1], s[i][2], s[i][3]);
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (j < nc) st[(int64_t)d * p.V + j] = s[i][j];
            }
        }
    }
}

size_t mats_smem(const GdnArgs &a) {
    const int kp = (a.K + 3) & ~3;
    return (size_t)(2 * kGL * (kp + 4) + kGL * (kGL + 1) + kGL * (kVT + 4)) * 4;
}
size_t scan_smem(const GdnArgs &a) {
    const int kp = (a.K + 3) & ~3;
    return (size_t)(kp * kVT + kGL * kVT + 2 * (2 * kGL * kp + kGL * kVT)) * 4;
}
size_t out_smem(const GdnArgs &a) {
    const int kp = (a.K + 3) & ~3;
    return (size_t)(kGL * (kp + 4) + kp * kVT + kGL * kVT + kGL * (kGL + 1)) * 4;
}
size_t base_smem(const GdnArgs &a) { return (size_t)(kGL * kVT + kGL * kGL + kGL + kGL * ((a.K + 3) & ~3)) * 4; }

template <typename T>
cudaError_t prepare_kernels() {
    static DeviceOnce once;
    int dev;
    return once.run(&dev, [](int) {
        const GdnArgs big = [] { GdnArgs a{}; a.K = 256; return a; }();
        auto room = [](auto *k, size_t n) {
            return cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)n);
        };
        cudaError_t e = room(gdn_simt_mats_kernel<T>, mats_smem(big));
        if (e == cudaSuccess) e = room(gdn_simt_scan_kernel<false>, scan_smem(big));
        if (e == cudaSuccess) e = room(gdn_simt_scan_kernel<true>, scan_smem(big));
        if (e == cudaSuccess) e = room(gdn_simt_out_kernel<T>, out_smem(big));
        if (e == cudaSuccess) e = room(gdn_simt_base_kernel<T>, base_smem(big));
        if (e == cudaSuccess) e = room(gdn_simt_grad_kernel<T>, sizeof(GradSmem));
        return e;
    });
}

// The offsets' check, norms and rows: what every path begins with.
template <typename T>
cudaError_t launch_rows(const GdnArgs &a, cudaStream_t st) {
    cudaError_t e = cudaSuccess;
    if (a.cu) e = launch_validate_offsets(a.cu, a.N, a.T, a.status, a.ctrl, a.chunk_start, st, a.L);
    if (e == cudaSuccess && a.l2) {
        constexpr int per = 16 / sizeof(T);
        const bool al = a.K % per == 0 && a.q_stride % per == 0 && a.k_stride % per == 0 && aligned_to(a.q, 16) &&
                        aligned_to(a.k, 16);
        int log_lanes = 0;
        while (log_lanes < 5 && (per << log_lanes) < a.K) ++log_lanes;
        e = run("gdn_norms", al ? gdn_norms_kernel<T, true> : gdn_norms_kernel<T, false>,
                (((int64_t)a.B * a.T * a.H << log_lanes) + kThreads - 1) / kThreads, kThreads, 0, st, a, log_lanes);
    }
    auto rows = gdn_rows_kernel<T, kGL / 32>;
    if constexpr (sizeof(T) == 2)  // (fp32 has chunks of 32 rows only)
        if (a.L != kGL) rows = gdn_rows_kernel<T, kGC / 32>;
    if (e == cudaSuccess)
        e = run("gdn_rows", rows, a.slots * ((a.HV + kRowHeads - 1) / kRowHeads), 32 * kRowHeads, 0, st, a);
    return e;
}

template <typename T>
cudaError_t fwd(const GdnArgs &a, cudaStream_t st) {
    if (a.L != kGL) {
        cudaError_t e = launch_rows<T>(a, st);
        return e == cudaSuccess ? launch_gdn_tc_fwd(a, st) : e;
    }
    cudaError_t e = prepare_kernels<T>();
    const int64_t units = a.slots * a.HV, scans = (int64_t)a.N * a.HV * ((a.V + kVT - 1) / kVT);
    if (e == cudaSuccess) e = launch_rows<T>(a, st);
    const dim3 tiles((unsigned)units, (unsigned)((a.V + kVT - 1) / kVT));
    if (e == cudaSuccess) e = run("gdn_simt_mats", gdn_simt_mats_kernel<T>, units, kThreads, mats_smem(a), st, a);
    if (e == cudaSuccess) e = run("gdn_simt_scan", gdn_simt_scan_kernel<false>, scans, kThreads, scan_smem(a), st, a);
    if (e == cudaSuccess && a.o) e = run("gdn_simt_out", gdn_simt_out_kernel<T>, tiles, kThreads, out_smem(a), st, a);
    return e;
}

template <typename T>
cudaError_t bwd(const GdnArgs &a, bool states_kept, cudaStream_t st) {
    cudaError_t e = cudaSuccess;
    if (!states_kept) {
        GdnArgs f = a;
        f.o = nullptr;
        f.ht = nullptr;
        e = fwd<T>(f, st);
    } else {
        e = prepare_kernels<T>();
    }
    const int64_t units = a.slots * a.HV, scans = (int64_t)a.N * a.HV * ((a.V + kVT - 1) / kVT);
    const bool tensor = a.L != kGL, direct = tensor && a.HV == a.H;
    if (tensor) {
        if (e == cudaSuccess) e = launch_gdn_tc_bwd(a, st);
    } else {
        const dim3 tiles((unsigned)units, (unsigned)((a.V + kVT - 1) / kVT));
        if (e == cudaSuccess) e = run("gdn_simt_base", gdn_simt_base_kernel<T>, tiles, kThreads, base_smem(a), st, a);
        if (e == cudaSuccess) e = run("gdn_simt_rscan", gdn_simt_scan_kernel<true>, scans, kThreads, scan_smem(a), st, a);
        if (e == cudaSuccess) e = run("gdn_simt_grad", gdn_simt_grad_kernel<T>, units, kThreads, sizeof(GradSmem), st, a);
    }
    if (e == cudaSuccess && !direct)
        e = run("gdn_finish", a.K % 4 == 0 ? gdn_finish_kernel<T, 4> : gdn_finish_kernel<T, 1>,
                ((int64_t)a.B * a.T * a.H + 7) / 8, kThreads, 0, st, a);
    if (e == cudaSuccess && a.cu)
        e = run("gdn_tail", gdn_tail_kernel<T>, a.T > 0 ? kSms : 0, kThreads, 0, st, a, (int)direct);
    return e;
}

template <typename T, int LW, int W>
cudaError_t step(const GdnStepArgs &a, cudaStream_t st) {
    const int64_t blocks = (int64_t)a.N * a.HV * ((a.V + 4 * LW - 1) / (4 * LW));
    return run("gdn_step", gdn_step_kernel<T, LW, W>, blocks, 32 * W, 0, st, a,
               (int)(a.V % 4 == 0 && aligned_to(a.state, 16)));
}
// A warp for every 32 state rows, up to 64 columns a block: small blocks of few registers, many on an SM.
// 256 rows of 32 heads, us, in blocks of eight warps and up to 128 columns, then so: 128 x 128 188 and 169, 128 x 64
// 124 and 91, 64 x 64 92 and 51, 32 x 32 34 and 20; 16 heads of 256 x 256 457 and 401 (511 with 32 columns a block).
template <typename T>
cudaError_t step_of(const GdnStepArgs &a, cudaStream_t st) {
    if (a.V > 32)
        return a.K > 128 ? step<T, 16, 8>(a, st) : a.K > 64 ? step<T, 16, 4>(a, st)
               : a.K > 32 ? step<T, 16, 2>(a, st) : step<T, 16, 1>(a, st);
    return a.K > 128 ? step<T, 8, 8>(a, st) : a.K > 64 ? step<T, 8, 4>(a, st)
           : a.K > 32 ? step<T, 8, 2>(a, st) : step<T, 8, 1>(a, st);
}

}  // namespace

int gdn_chunk_len(kda_dtype dt, int K, int V) { return gdn_tc_supported(dt, K, V) ? kGC : kGL; }
size_t gdn_rows_floats(int L) { return (size_t)kGdnRowArrays * L; }
size_t gdn_mats_floats(int L) { return (size_t)3 * L * L; }
size_t gdn_wk_floats(int L, int K) { return (size_t)2 * L * ((K + 3) & ~3); }
size_t gdn_u_floats(int L, int V) { return (size_t)L * ((V + kVT - 1) / kVT * kVT); }
size_t gdn_state_floats(int K, int V) { return (size_t)K * ((V + kVT - 1) / kVT * kVT); }

cudaError_t launch_gdn_fwd(const GdnArgs &a, kda_dtype dt, cudaStream_t st) {
    return dt == KDA_DTYPE_BF16 ? fwd<bf16>(a, st) : fwd<float>(a, st);
}
cudaError_t launch_gdn_bwd(const GdnArgs &a, kda_dtype dt, bool states_kept, cudaStream_t st) {
    return dt == KDA_DTYPE_BF16 ? bwd<bf16>(a, states_kept, st) : bwd<float>(a, states_kept, st);
}
cudaError_t launch_gdn_step(const GdnStepArgs &a, kda_dtype dt, cudaStream_t st) {
    return dt == KDA_DTYPE_BF16 ? step_of<bf16>(a, st) : step_of<float>(a, st);
}

}  // namespace kda
