// kda_ssm.cu -- the selective state-space scan: per sequence and head h (B and C from
// group g = h / (H / G)), with d_t = softplus(dt_t + dt_bias) (or dt_t as given) and
// A = -exp(A_log), an fp32 state S of [Ns, P] evolves as
//
//     S_t = e^{d_t A} S_{t-1} + d_t B_t x_t^T,      y_t = S_t^T C_t + D x_t .
//
// Chunk form.  With a_i the cumulative log2 decay from a chunk's first row on (a_i <= 0),
//     local   = sum_j 2^{a_end - a_j} d_j B_j x_j^T         (per chunk, all at once)
//     S_{c+1} = 2^{a_end} S_c + local                       (over chunks, elementwise)
//     y_i     = 2^{a_i} S_c^T C_i + sum_{j <= i} (C_i . B_j) 2^{a_i - a_j} d_j x_j + D x_i .
// Every exponent is a difference taken before the exponential and is <= 0, so no gate, however
// strong, overflows.  The three steps are three launches; only the middle one walks over
// the chunks, and it moves the states alone.
//
// Gradients run the same way: the state gradient at each chunk's end is the scan from the
// right over sum_i 2^{a_i} C_i dy_i^T, and then every chunk on its own forms dx, dB, dC and
// the gradient of its decays (see ssm_chunk_grads_kernel).
//
// This file holds the fp32 kernels on the CUDA cores, for every type and size, and the
// single-token form.  fp32 throughout, each output rounded once.  bf16 inputs whose columns and
// state rows allow it take the tensor cores instead (kda_ssm_tc.cu): forward and gradients of
// 16 sequences of 512 rows, 32 heads of 64, 128 state rows, 392 us there against 2830 us here,
// and of one sequence of one row 63 against 107.  Here the products are bound by the fp32
// pipe and by shared memory's bandwidth.
#include "kda_block.cuh"

namespace kda {
namespace {

constexpr int kL = 64;            // chunk length here
constexpr int kLD = kL + 4;       // row stride of a shared tile: 16-byte aligned, off the banks
constexpr int kTile = kL * kLD;   // floats per tile
constexpr float kLog2e = 1.4426950408889634f;

// The rows of a chunk slot.
struct Chunk {
    int64_t r0;   // its first row, of all B * T
    int nr;       // rows
};
__device__ __forceinline__ bool find_chunk(const SsmArgs &p, int64_t slot, Chunk &c) {
    if (p.cu) {
        if (!p.ctrl->valid || slot >= p.ctrl->total_chunks) return false;
        const int n = upper_bound_minus_one(p.chunk_start, p.N + 1, (int)slot);
        const int s = p.cu[n] + p.L * ((int)slot - p.chunk_start[n]);
        c.r0 = s;
        c.nr = min(p.L, p.cu[n + 1] - s);
    } else {
        const int per = (p.T + p.L - 1) / p.L;
        const int seq = (int)(slot / per);
        const int k = (int)(slot % per);
        c.r0 = (int64_t)seq * p.T + (int64_t)k * p.L;
        c.nr = min(p.L, p.T - k * p.L);
    }
    return c.nr > 0;
}

__device__ __forceinline__ float step_size(float raw, float bias, int softplus) {
    const float v = raw + bias;
    return softplus ? softplus_f(v) : v;
}

// d_i and a_i (log2, cumulative) of a chunk's rows in shared memory; rows past nr have d = 0
// and the last row's a.  a is kept as a sum of two floats, a + lo: under strong decay a_i runs
// to thousands while the rows next to each other still differ by little, and the difference
// of two single floats would lose those digits.  All threads call; ends with a barrier.
template <typename T>
__device__ __forceinline__ void chunk_decays(const SsmArgs &p, const Chunk &c, int h, float *d,
                                             float *a, float *lo) {
    __shared__ double first_half;
    const int i = threadIdx.x;
    double s = 0.0;
    if (i < kL) {
        float v = 0.f;
        if (i < c.nr) {
            const float raw = to_f32(static_cast<const T *>(p.dt)[(c.r0 + i) * p.dt_stride + h]);
            v = step_size(raw, p.dt_bias ? p.dt_bias[h] : 0.f, p.softplus);
        }
        d[i] = v;
        s = v * (-expf(p.A_log[h]) * kLog2e);
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const double u = __shfl_up_sync(0xffffffffu, s, o);
            if ((i & 31) >= o) s += u;
        }
        if (i == 31) first_half = s;
    }
    __syncthreads();
    if (i < kL) {
        if (i >= 32) s += first_half;
        a[i] = (float)s;
        lo[i] = (float)(s - (double)a[i]);
    }
    __syncthreads();
}
// 2^{a_i - a_j}
__device__ __forceinline__ float decay_between(const float *a, const float *lo, int i, int j) {
    return ex2_ftz((a[i] - a[j]) + (lo[i] - lo[j]));
}

// A 64 x 64 tile of a row-major matrix into shared memory, zero outside rows x cols, each
// row times scale[row] (null: 1); as it is (dst[r][c]) or transposed (dst[c][r]).
template <bool TR, typename T>
__device__ __forceinline__ void load_tile(float *dst, const T *src, int64_t stride, int rows, int cols,
                                          const float *scale) {
    for (int e = threadIdx.x; e < kL * kL; e += blockDim.x) {
        const int r = e / kL, c = e % kL;
        float v = r < rows && c < cols ? to_f32(src[r * stride + c]) : 0.f;
        if (scale) v = r < rows ? v * scale[r] : 0.f;
        dst[TR ? c * kLD + r : r * kLD + c] = v;
    }
}

// acc[i][j] += sum_k A[k][4 ty + i] B[k][4 tx + j] over the 64 rows of two shared tiles
// (256 threads, ty = tid / 16, tx = tid % 16).
__device__ __forceinline__ void mm64(float (&acc)[4][4], const float *A, const float *B) {
    const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
#pragma unroll 8
    for (int k = 0; k < kL; ++k) {
        const float4 u = *reinterpret_cast<const float4 *>(A + k * kLD + 4 * ty);
        const float4 v = *reinterpret_cast<const float4 *>(B + k * kLD + 4 * tx);
        const float m[4] = {u.x, u.y, u.z, u.w}, n[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(m[i], n[j], acc[i][j]);
    }
}

// A chunk's own state term, [Ns, P] of one head, tile by tile (64 x 64):
//   forward  (BWD false): sum_j 2^{a_end - a_j} d_j B_j x_j^T  -> states, and 2^{a_end}
//   backward (BWD true):  sum_i 2^{a_i} C_i dy_i^T             -> dstates
template <typename T, bool BWD>
__global__ void __launch_bounds__(256) ssm_chunk_state_kernel(SsmArgs p) {
    extern __shared__ float sm[];
    float *As = sm, *Bs = sm + kTile, *d = Bs + kTile, *a = d + kL, *lo = a + kL, *wgt = lo + kL;
    const int nt = (p.Ns + kL - 1) / kL, pt = (p.P + kL - 1) / kL;
    int64_t id = blockIdx.x;
    const int p0 = (int)(id % pt) * kL;
    id /= pt;
    const int n0 = (int)(id % nt) * kL;
    id /= nt;
    const int h = (int)(id % p.H);
    const int64_t slot = id / p.H;
    Chunk c;
    if (!find_chunk(p, slot, c)) return;
    const int g = h / (p.H / p.G);
    chunk_decays<T>(p, c, h, d, a, lo);
    if (threadIdx.x < kL) {
        const int i = threadIdx.x;
        wgt[i] = BWD ? ex2_ftz(a[i]) : decay_between(a, lo, kL - 1, i) * d[i];
    }
    __syncthreads();
    const int ncols = min(kL, p.Ns - n0), pcols = min(kL, p.P - p0);
    if constexpr (BWD) {
        load_tile<false>(As, static_cast<const T *>(p.Cm) + c.r0 * p.c_stride + g * p.Ns + n0, p.c_stride,
                         c.nr, ncols, nullptr);
        load_tile<false>(Bs, static_cast<const T *>(p.dy) + (c.r0 * p.H + h) * p.P + p0,
                         (int64_t)p.H * p.P, c.nr, pcols, wgt);
    } else {
        load_tile<false>(As, static_cast<const T *>(p.Bm) + c.r0 * p.b_stride + g * p.Ns + n0, p.b_stride,
                         c.nr, ncols, nullptr);
        load_tile<false>(Bs, static_cast<const T *>(p.x) + c.r0 * p.x_stride + (int64_t)h * p.P + p0,
                         p.x_stride, c.nr, pcols, wgt);
    }
    __syncthreads();
    float acc[4][4] = {};
    mm64(acc, As, Bs);
    const int64_t unit = slot * p.H + h;
    float *out = (BWD ? p.dstates : p.states) + unit * p.Ns * p.P;
    const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int n = n0 + 4 * ty + i, q = p0 + 4 * tx + j;
            if (n < p.Ns && q < p.P) out[(int64_t)n * p.P + q] = acc[i][j];
        }
    if (!BWD && n0 == 0 && p0 == 0 && threadIdx.x == 0) p.decay[unit] = ex2_ftz(a[kL - 1]);
}

// The scan over a sequence's chunks, VEC state entries per thread.  Forward: states holds
// the chunks' own terms and gets the state at each chunk's start; the last state goes to
// ht.  Reverse: dstates holds the chunks' terms and gets the gradient at each chunk's end;
// what is left goes to dh0.  2 x states bytes moved; loads of the next chunks are issued
// ahead of the (serial) multiply-adds.
template <int VEC, bool REV>
__global__ void __launch_bounds__(128) ssm_state_pass_kernel(SsmArgs p) {
    const int64_t np = (int64_t)p.Ns * p.P;
    const int64_t blocks_per = (np + 128 * VEC - 1) / (128 * VEC);
    const int64_t sh = blockIdx.x / blocks_per;
    const int64_t e = ((blockIdx.x % blocks_per) * 128 + threadIdx.x) * VEC;
    if (e >= np) return;
    const int h = (int)(sh % p.H), n = (int)(sh / p.H);
    int64_t first;
    int nc;
    if (p.cu) {
        if (!p.ctrl->valid) return;
        first = p.chunk_start[n];
        nc = p.chunk_start[n + 1] - p.chunk_start[n];
    } else {
        nc = (p.T + p.L - 1) / p.L;
        first = (int64_t)n * nc;
    }
    const float *from = REV ? p.dht : p.h0;
    float *to = REV ? p.dh0 : p.ht;
    float *st = (REV ? p.dstates : p.states) + first * p.H * np + h * np + e;
    const float *dec = p.decay + first * p.H + h;
    float run[VEC];
#pragma unroll
    for (int j = 0; j < VEC; ++j) run[j] = 0.f;
    if (from) {
        if constexpr (VEC == 4) {
            const float4 f = *reinterpret_cast<const float4 *>(from + sh * np + e);
            run[0] = f.x; run[1] = f.y; run[2] = f.z; run[3] = f.w;
        } else {
            run[0] = from[sh * np + e];
        }
    }
    constexpr int U = 4;
    for (int k0 = 0; k0 < nc; k0 += U) {
        float own[U][VEC], dk[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (k0 + u < nc) {
                const int64_t k = REV ? nc - 1 - (k0 + u) : k0 + u;
                const float *src = st + k * p.H * np;
                dk[u] = dec[k * p.H];
                if constexpr (VEC == 4) {
                    const float4 f = *reinterpret_cast<const float4 *>(src);
                    own[u][0] = f.x; own[u][1] = f.y; own[u][2] = f.z; own[u][3] = f.w;
                } else {
                    own[u][0] = *src;
                }
            }
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (k0 + u < nc) {
                const int64_t k = REV ? nc - 1 - (k0 + u) : k0 + u;
                float *dst = st + k * p.H * np;
                if constexpr (VEC == 4)
                    *reinterpret_cast<float4 *>(dst) = make_float4(run[0], run[1], run[2], run[3]);
                else
                    *dst = run[0];
#pragma unroll
                for (int j = 0; j < VEC; ++j) run[j] = fmaf(dk[u], run[j], own[u][j]);
            }
    }
    if (to) {
        if constexpr (VEC == 4)
            *reinterpret_cast<float4 *>(to + sh * np + e) = make_float4(run[0], run[1], run[2], run[3]);
        else
            to[sh * np + e] = run[0];
    }
}

// One chunk of one head: y, 64 columns at a time.
template <typename T>
__global__ void __launch_bounds__(256) ssm_chunk_out_kernel(SsmArgs p) {
    extern __shared__ float sm[];
    float *Ct = sm, *Bt = Ct + kTile, *Sx = Bt + kTile, *d = Sx + kTile, *a = d + kL;
    float *lo = a + kL;
    const int pt = (p.P + kL - 1) / kL;
    int64_t id = blockIdx.x;
    const int p0 = (int)(id % pt) * kL;
    id /= pt;
    const int h = (int)(id % p.H);
    const int64_t slot = id / p.H;
    Chunk c;
    if (!find_chunk(p, slot, c)) return;
    const int g = h / (p.H / p.G), pcols = min(kL, p.P - p0);
    const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
    chunk_decays<T>(p, c, h, d, a, lo);
    const int64_t unit = slot * p.H + h;
    float gram[4][4] = {}, y[4][4] = {};
    for (int n0 = 0; n0 < p.Ns; n0 += kL) {
        const int ncols = min(kL, p.Ns - n0);
        load_tile<true>(Ct, static_cast<const T *>(p.Cm) + c.r0 * p.c_stride + g * p.Ns + n0, p.c_stride,
                        c.nr, ncols, nullptr);
        load_tile<true>(Bt, static_cast<const T *>(p.Bm) + c.r0 * p.b_stride + g * p.Ns + n0, p.b_stride,
                        c.nr, ncols, nullptr);
        load_tile<false>(Sx, p.states + unit * p.Ns * p.P + (int64_t)n0 * p.P + p0, p.P, ncols, pcols,
                         nullptr);
        __syncthreads();
        mm64(gram, Ct, Bt);
        mm64(y, Ct, Sx);
        __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = 4 * ty + i;
        const float er = ex2_ftz(a[r]);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int s = 4 * tx + j;
            Ct[s * kLD + r] = s <= r ? gram[i][j] * decay_between(a, lo, r, s) * d[s] : 0.f;
            y[i][j] *= er;
        }
    }
    load_tile<false>(Sx, static_cast<const T *>(p.x) + c.r0 * p.x_stride + (int64_t)h * p.P + p0, p.x_stride,
                     c.nr, pcols, nullptr);
    __syncthreads();
    float inter[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) inter[i][j] = y[i][j];
    mm64(y, Ct, Sx);
    // a non-finite x_s reaches rows r < s through 0 x_s: such rows are summed again up to r
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (!isfinite(y[i][j])) {
                y[i][j] = inter[i][j];
                for (int s = 0; s <= 4 * ty + i; ++s)
                    y[i][j] = fmaf(Ct[s * kLD + 4 * ty + i], Sx[s * kLD + 4 * tx + j], y[i][j]);
            }
    const float D = p.D ? p.D[h] : 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int r = 4 * ty + i, q = 4 * tx + j;
            if (r < c.nr && q < pcols)
                static_cast<T *>(p.y)[((c.r0 + r) * p.H + h) * p.P + p0 + q] =
                    from_f32<T>(p.D ? fmaf(D, Sx[r * kLD + q], y[i][j]) : y[i][j]);
        }
}

// One chunk of one head: dx, the head's shares of dB and dC, ddt, and the chunk's shares of
// dA_log, dD and ddt_bias.  With G_ij = C_i . B_j, Z_ij = dy_i . x_j, e_ij = 2^{a_i - a_j}
// (j <= i, else 0), S the state at the chunk's start and E the state gradient at its end:
//     dx_j = sum_i G_ij e_ij d_j dy_i + d_j 2^{a_end - a_j} E^T B_j + D dy_j
//     dC_i = sum_j Z_ij e_ij d_j B_j + 2^{a_i} S dy_i
//     dB_j = sum_i Z_ij e_ij d_j C_i + d_j 2^{a_end - a_j} E x_j
// and, through the exponents, with Q_ij = Z_ij G_ij e_ij d_j,
// u_i = 2^{a_i} C_i . S dy_i and v_j = d_j 2^{a_end - a_j} B_j . E x_j:
// the log decay of row t (which every pair i >= t > j passes) gets
//     l_t = sum_{i >= t > j} Q_ij + sum_{i >= t} u_i + sum_{j < t} v_j + 2^{a_end} <E, S>,
//     dd_t = A l_t + sum_i Q_it / d_t + v_t / d_t,   dA = sum_t d_t l_t.
// l_t is summed term by term: taken as a running difference of row and column sums, a pair
// far from t would leave its rounding in l_t, which a strong decay's A d_t then multiplies.
// (The quotients are formed without the division.)
template <typename T>
__global__ void __launch_bounds__(256) ssm_chunk_grads_kernel(SsmArgs p) {
    extern __shared__ float sm[];
    float *M = sm, *W = M + kTile, *X = W + kTile, *Y = X + kTile, *d = Y + kTile, *a = d + kL;
    float *lo = a + kL, *ea = lo + kL, *el = ea + kL, *l = el + kL, *dd = l + kL, *red = dd + kL;  // red: 16 x 64
    const int h = (int)(blockIdx.x % p.H);
    const int64_t slot = blockIdx.x / p.H;
    Chunk c;
    if (!find_chunk(p, slot, c)) return;
    const int g = h / (p.H / p.G), tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
    const int64_t unit = slot * p.H + h, np = (int64_t)p.Ns * p.P;
    const T *Cg = static_cast<const T *>(p.Cm) + c.r0 * p.c_stride + g * p.Ns;
    const T *Bg = static_cast<const T *>(p.Bm) + c.r0 * p.b_stride + g * p.Ns;
    const T *xg = static_cast<const T *>(p.x) + c.r0 * p.x_stride + (int64_t)h * p.P;
    const T *dyg = static_cast<const T *>(p.dy) + (c.r0 * p.H + h) * p.P;
    const int64_t ys = (int64_t)p.H * p.P;
    chunk_decays<T>(p, c, h, d, a, lo);
    if (tid < kL) {
        ea[tid] = ex2_ftz(a[tid]);
        el[tid] = decay_between(a, lo, kL - 1, tid);
    }
    float G[4][4] = {}, Z[4][4] = {};
    for (int n0 = 0; n0 < p.Ns; n0 += kL) {
        load_tile<true>(X, Cg + n0, p.c_stride, c.nr, min(kL, p.Ns - n0), nullptr);
        load_tile<true>(Y, Bg + n0, p.b_stride, c.nr, min(kL, p.Ns - n0), nullptr);
        __syncthreads();
        mm64(G, X, Y);
        __syncthreads();
    }
    float dD = 0.f;
    for (int p0 = 0; p0 < p.P; p0 += kL) {
        load_tile<true>(X, dyg + p0, ys, c.nr, min(kL, p.P - p0), nullptr);
        load_tile<true>(Y, xg + p0, p.x_stride, c.nr, min(kL, p.P - p0), nullptr);
        __syncthreads();
        mm64(Z, X, Y);
        __syncthreads();
    }
    // M_ij = G_ij e_ij d_j, W_ij = Z_ij e_ij d_j; Q below the diagonal, and its column sums
    float col[4] = {};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = 4 * ty + i;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int s = 4 * tx + j;
            const float e = s <= r ? decay_between(a, lo, r, s) : 0.f;
            if (s == r) dD += Z[i][j];
            M[r * kLD + s] = G[i][j] * e * d[s];
            W[r * kLD + s] = Z[i][j] * e * d[s];
            const float q = Z[i][j] * G[i][j] * e;
            X[r * kLD + s] = s < r ? q * d[s] : 0.f;
            col[j] += q;
        }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) red[ty * kL + 4 * tx + j] = col[j];
    __syncthreads();
    {   // each row's sums over the columns before t, four threads a row
        float *q = X + (tid >> 2) * kLD + 16 * (tid & 3), s[16], run = 0.f;
#pragma unroll
        for (int k = 0; k < 16; ++k) {
            s[k] = run;
            run += q[k];
        }
        float before = run;
#pragma unroll
        for (int o = 1; o < 4; o <<= 1) {
            const float x = __shfl_up_sync(0xffffffffu, before, o, 4);
            if ((tid & 3) >= o) before += x;
        }
        before = __shfl_up_sync(0xffffffffu, before, 1, 4);
        if ((tid & 3) == 0) before = 0.f;
#pragma unroll
        for (int k = 0; k < 16; ++k) q[k] = before + s[k];
    }
    if (tid < kL) {
        float s = 0.f;
        for (int k = 0; k < 16; ++k) s += red[k * kL + tid];
        dd[tid] = s;            // sum_i Q_it / d_t
    }
    __syncthreads();
    {   // sum_{i >= t} sum_{j < t} Q_ij, sixteen rows a thread
        const int c0 = tid & (kL - 1), r0 = 16 * (tid >> 6);
        float s = 0.f;
        for (int r = max(r0, c0); r < r0 + 16; ++r) s += X[r * kLD + c0];
        red[tid] = s;
    }
    __syncthreads();
    if (tid < kL) l[tid] = (red[tid] + red[kL + tid]) + (red[2 * kL + tid] + red[3 * kL + tid]);
    const float D = p.D ? p.D[h] : 0.f;
    // dx, 64 columns at a time
    for (int p0 = 0; p0 < p.P; p0 += kL) {
        const int pcols = min(kL, p.P - p0);
        float acc[4][4] = {};
        for (int n0 = 0; n0 < p.Ns; n0 += kL) {
            const int ncols = min(kL, p.Ns - n0);
            __syncthreads();
            load_tile<true>(X, Bg + n0, p.b_stride, c.nr, ncols, nullptr);
            load_tile<false>(Y, p.dstates + unit * np + (int64_t)n0 * p.P + p0, p.P, ncols, pcols, nullptr);
            __syncthreads();
            mm64(acc, X, Y);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[i][j] *= el[4 * ty + i] * d[4 * ty + i];
        __syncthreads();
        load_tile<false>(Y, dyg + p0, ys, c.nr, pcols, nullptr);
        __syncthreads();
        mm64(acc, M, Y);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int r = 4 * ty + i, q = 4 * tx + j;
                if (r < c.nr && q < pcols)
                    static_cast<T *>(p.dx)[((c.r0 + r) * p.H + h) * p.P + p0 + q] =
                        from_f32<T>(p.D ? fmaf(D, Y[r * kLD + q], acc[i][j]) : acc[i][j]);
            }
    }
    // dC and dB, 64 columns at a time; u_i and v_j on the way
    float u[4] = {}, v[4] = {}, es = 0.f;
    for (int n0 = 0; n0 < p.Ns; n0 += kL) {
        const int ncols = min(kL, p.Ns - n0);
        float ac[4][4] = {}, ab[4][4] = {};
        for (int p0 = 0; p0 < p.P; p0 += kL) {
            const int pcols = min(kL, p.P - p0);
            __syncthreads();
            load_tile<true>(X, dyg + p0, ys, c.nr, pcols, nullptr);
            load_tile<true>(Y, p.states + unit * np + (int64_t)n0 * p.P + p0, p.P, ncols, pcols, nullptr);
            __syncthreads();
            mm64(ac, X, Y);
            __syncthreads();
            load_tile<true>(X, xg + p0, p.x_stride, c.nr, pcols, nullptr);
            // E's tile over S's, entry by entry: <E, S> on the way
            for (int e = tid; e < kL * kL; e += 256) {
                const int r = e / kL, q = e % kL;
                const float f = r < ncols && q < pcols
                                    ? p.dstates[unit * np + (int64_t)(n0 + r) * p.P + p0 + q] : 0.f;
                es = fmaf(f, Y[q * kLD + r], es);
                Y[q * kLD + r] = f;
            }
            __syncthreads();
            mm64(ab, X, Y);
        }
        __syncthreads();
        load_tile<false>(X, Cg + n0, p.c_stride, c.nr, ncols, nullptr);
        load_tile<false>(Y, Bg + n0, p.b_stride, c.nr, ncols, nullptr);
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = 4 * ty + i;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int q = 4 * tx + j;
                ac[i][j] *= ea[r];
                ab[i][j] *= el[r];
                u[i] = fmaf(ac[i][j], X[r * kLD + q], u[i]);
                v[i] = fmaf(ab[i][j], Y[r * kLD + q], v[i]);
                ab[i][j] *= d[r];
            }
        }
        mm64(ab, W, X);          // sum_i W_ij C_i
        // sum_j W_ij B_j: W's rows are i here, so the left operand is its transpose
        {
#pragma unroll 4
            for (int k = 0; k < kL; ++k) {
                const float4 b = *reinterpret_cast<const float4 *>(Y + k * kLD + 4 * tx);
                const float n[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float m = W[(4 * ty + i) * kLD + k];
#pragma unroll
                    for (int j = 0; j < 4; ++j) ac[i][j] = fmaf(m, n[j], ac[i][j]);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int r = 4 * ty + i, q = 4 * tx + j;
                if (r < c.nr && q < ncols) {
                    const int64_t at = ((c.r0 + r) * p.H + h) * p.Ns + n0 + q;
                    p.dCh[at] = ac[i][j];
                    p.dBh[at] = ab[i][j];
                }
            }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) {
            u[i] += __shfl_xor_sync(0xffffffffu, u[i], o);
            v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
        }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (tx == 0) {
            const int r = 4 * ty + i;
            dd[r] += v[i];
            ea[r] = u[i];          // read above for the last time, but for the last row's
            red[r] = v[i] * d[r];
        }
    // block sums: <E, S> and dD
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        es += __shfl_xor_sync(0xffffffffu, es, o);
        dD += __shfl_xor_sync(0xffffffffu, dD, o);
    }
    if ((tid & 31) == 0) {
        red[kL + (tid >> 5)] = es;
        red[kL + 8 + (tid >> 5)] = dD;
    }
    __syncthreads();
    if (tid < 32) {  // rows tid and tid + 32
        float e = tid < 8 ? red[kL + tid] : 0.f, dds = tid < 8 ? red[kL + 8 + tid] : 0.f;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            e += __shfl_xor_sync(0xffffffffu, e, o);
            dds += __shfl_xor_sync(0xffffffffu, dds, o);
        }
        // u from the right (with the row itself), v from the left (without it)
        float u0 = ea[tid], u1 = ea[tid + 32], v0 = red[tid], v1 = red[tid + 32];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const float x0 = __shfl_down_sync(0xffffffffu, u0, o), x1 = __shfl_down_sync(0xffffffffu, u1, o);
            const float y0 = __shfl_up_sync(0xffffffffu, v0, o), y1 = __shfl_up_sync(0xffffffffu, v1, o);
            if (tid + o < 32) {
                u0 += x0;
                u1 += x1;
            }
            if (tid >= o) {
                v0 += y0;
                v1 += y1;
            }
        }
        u0 += __shfl_sync(0xffffffffu, u1, 0);
        const float half = __shfl_sync(0xffffffffu, v0, 31);
        v0 = __shfl_up_sync(0xffffffffu, v0, 1);
        v1 = __shfl_up_sync(0xffffffffu, v1, 1);
        if (tid == 0) v0 = v1 = 0.f;
        const float end = ex2_ftz(a[kL - 1]) * e;
        const float l0 = l[tid] + (u0 + (v0 + end)), l1 = l[tid + 32] + (u1 + (half + v1 + end));
        const float A = -expf(p.A_log[h]), bias = p.dt_bias ? p.dt_bias[h] : 0.f;
        float sA = 0.f, sb = 0.f;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int t = tid + 32 * k;
            const float l = k ? l1 : l0;
            if (t < c.nr) {
                const int64_t row = c.r0 + t;
                float gd = fmaf(A, l, dd[t]);
                if (p.softplus) {
                    const float raw = to_f32(static_cast<const T *>(p.dt)[row * p.dt_stride + h]) + bias;
                    gd *= 1.f / (1.f + expf(-raw));
                }
                static_cast<T *>(p.ddt)[row * p.H + h] = from_f32<T>(gd);
                sA = fmaf(d[t], l, sA);
                sb += gd;
            }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            sA += __shfl_xor_sync(0xffffffffu, sA, o);
            sb += __shfl_xor_sync(0xffffffffu, sb, o);
        }
        if (tid == 0) {
            p.sums[(slot * 3 + 0) * p.H + h] = sA * A;
            p.sums[(slot * 3 + 1) * p.H + h] = dds;
            p.sums[(slot * 3 + 2) * p.H + h] = sb;
        }
    }
}

// dB and dC: the sum of a group's heads' shares, in the heads' order.
template <typename T>
__global__ void __launch_bounds__(256) ssm_group_sum_kernel(SsmArgs p, int64_t rows) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= rows * p.G * p.Ns) return;
    const int n = (int)(i % p.Ns);
    const int64_t rg = i / p.Ns, row = rg / p.G;
    const int g = (int)(rg % p.G), per = p.H / p.G;
    float b = 0.f, c = 0.f;
    // rows past the last offset belong to no sequence: zero
    const bool in = !p.cu || (p.ctrl->valid && row < p.cu[p.N]);
    for (int k = 0; in && k < per; ++k) {
        const int64_t at = (row * p.H + g * per + k) * p.Ns + n;
        b += p.dBh[at];
        c += p.dCh[at];
    }
    static_cast<T *>(p.dB)[i] = from_f32<T>(b);
    static_cast<T *>(p.dC)[i] = from_f32<T>(c);
}

// dA_log, dD and ddt_bias from the chunks' shares: one warp per (sum, head), every lane
// adding every 32nd chunk.
__global__ void __launch_bounds__(128) ssm_param_sum_kernel(SsmArgs p) {
    follow();
    const int id = blockIdx.x * 4 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (id >= 3 * p.H) return;
    const int k = id / p.H, h = id % p.H;
    const int64_t slots = p.cu ? (p.ctrl->valid ? p.ctrl->total_chunks : 0) : p.slots;
    float s = 0.f;
    for (int64_t c = lane; c < slots; c += 32) s += p.sums[(c * 3 + k) * p.H + h];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    float *out = k == 0 ? p.dA_log : k == 1 ? p.dD : p.ddt_bias;
    if (lane == 0 && out) out[h] = s;
}

// One token of one sequence and head: the state is read once, advanced, stored, and read
// out on the way.  2 x 4 Ns P bytes against 5 Ns P flops: bandwidth-bound.  A thread owns
// VEC adjacent columns and every NG-th state row, so a warp's accesses are contiguous.
// Measured: 512 sequences x 32 heads x 128 x 64, 166 us (1.07 GB, 6.5 TB/s); with 63 columns,
// one per thread, 246 us.
template <typename T, int VEC>
__global__ void __launch_bounds__(256) ssm_step_kernel(SsmStepArgs p) {
    __shared__ float red[256 * VEC];
    const int64_t nh = blockIdx.x;
    const int h = (int)(nh % p.H), n = (int)(nh / p.H), g = h / (p.H / p.G);
    const int pq = p.P / VEC, ng = blockDim.x / pq;
    const int q = (threadIdx.x % pq) * VEC, rg = threadIdx.x / pq;
    const int slot = state_slot(p.idx, n, p.slots, p.status);
    T *y = static_cast<T *>(p.y) + nh * p.P;
    if (slot < 0) {
        for (int i = threadIdx.x; i < p.P; i += blockDim.x) y[i] = from_f32<T>(0.f);
        return;
    }
    float *st = p.state + ((int64_t)slot * p.H + h) * p.Ns * p.P;
    const T *Bm = static_cast<const T *>(p.Bm) + n * p.b_stride + g * p.Ns;
    const T *Cm = static_cast<const T *>(p.Cm) + n * p.c_stride + g * p.Ns;
    const T *x = static_cast<const T *>(p.x) + n * p.x_stride + (int64_t)h * p.P;
    const float raw = to_f32(static_cast<const T *>(p.dt)[n * p.dt_stride + h]);
    const float d = step_size(raw, p.dt_bias ? p.dt_bias[h] : 0.f, p.softplus);
    const float dec = expf(-expf(p.A_log[h]) * d);
    float xv[VEC], dx[VEC], acc[VEC] = {};
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
        xv[j] = to_f32(x[q + j]);
        dx[j] = d * xv[j];
    }
    constexpr int U = 8;
    for (int r0 = rg; r0 < p.Ns; r0 += U * ng) {
        float s[U][VEC];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int r = r0 + u * ng;
            if (r < p.Ns) {
                if constexpr (VEC == 4) {
                    const float4 f = *reinterpret_cast<const float4 *>(st + (int64_t)r * p.P + q);
                    s[u][0] = f.x; s[u][1] = f.y; s[u][2] = f.z; s[u][3] = f.w;
                } else {
                    s[u][0] = st[(int64_t)r * p.P + q];
                }
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int r = r0 + u * ng;
            if (r < p.Ns) {
                const float b = to_f32(Bm[r]), c = to_f32(Cm[r]);
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    s[u][j] = fmaf(dec, s[u][j], b * dx[j]);
                    acc[j] = fmaf(c, s[u][j], acc[j]);
                }
                if constexpr (VEC == 4)
                    *reinterpret_cast<float4 *>(st + (int64_t)r * p.P + q) =
                        make_float4(s[u][0], s[u][1], s[u][2], s[u][3]);
                else
                    st[(int64_t)r * p.P + q] = s[u][0];
            }
        }
    }
#pragma unroll
    for (int j = 0; j < VEC; ++j) red[rg * p.P + q + j] = acc[j];
    __syncthreads();
    const float D = p.D ? p.D[h] : 0.f;
    for (int i = threadIdx.x; i < p.P; i += blockDim.x) {
        float s = 0.f;
        for (int k = 0; k < ng; ++k) s += red[k * p.P + i];
        y[i] = from_f32<T>(p.D ? fmaf(D, to_f32(x[i]), s) : s);
    }
}

constexpr size_t kSmemState = (2 * kTile + 4 * kL) * 4;
constexpr size_t kSmemOut = (3 * kTile + 3 * kL) * 4;
constexpr size_t kSmemGrads = (4 * kTile + 7 * kL + 16 * kL) * 4;

template <typename K>
cudaError_t allow_smem(K kernel, size_t bytes) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
}

template <typename T>
cudaError_t ssm_setup() {
    static DeviceOnce once;
    int dev = 0;
    return once.run(&dev, [](int) {
        cudaError_t e = allow_smem(ssm_chunk_state_kernel<T, false>, kSmemState);
        if (e == cudaSuccess) e = allow_smem(ssm_chunk_state_kernel<T, true>, kSmemState);
        if (e == cudaSuccess) e = allow_smem(ssm_chunk_out_kernel<T>, kSmemOut);
        if (e == cudaSuccess) e = allow_smem(ssm_chunk_grads_kernel<T>, kSmemGrads);
        return e;
    });
}

template <typename T, bool BWD>
cudaError_t chunk_states(const SsmArgs &a, cudaStream_t st) {
    const int64_t tiles = (int64_t)((a.Ns + kL - 1) / kL) * ((a.P + kL - 1) / kL);
    const int64_t blocks = a.slots * a.H * tiles;
    if (blocks == 0) return cudaSuccess;
    if (blocks > INT32_MAX) return cudaErrorInvalidValue;
    prof_begin(BWD ? "ssm_chunk_dstate" : "ssm_chunk_state", st);
    ssm_chunk_state_kernel<T, BWD><<<(unsigned)blocks, 256, kSmemState, st>>>(a);
    prof_end(st);
    return cudaGetLastError();
}

template <bool REV>
cudaError_t state_pass(const SsmArgs &a, cudaStream_t st) {
    const int64_t np = (int64_t)a.Ns * a.P;
    const bool vec = np % 4 == 0 && aligned_to(REV ? a.dht : a.h0, 16) && aligned_to(REV ? a.dh0 : a.ht, 16);
    const int64_t per = (np + 128 * (vec ? 4 : 1) - 1) / (128 * (vec ? 4 : 1));
    const int64_t blocks = (int64_t)a.N * a.H * per;
    if (blocks == 0) return cudaSuccess;
    if (blocks > INT32_MAX) return cudaErrorInvalidValue;
    prof_begin(REV ? "ssm_dstate_pass" : "ssm_state_pass", st);
    if (vec)
        ssm_state_pass_kernel<4, REV><<<(unsigned)blocks, 128, 0, st>>>(a);
    else
        ssm_state_pass_kernel<1, REV><<<(unsigned)blocks, 128, 0, st>>>(a);
    prof_end(st);
    return cudaGetLastError();
}

template <typename T>
cudaError_t states(const SsmArgs &a, cudaStream_t st) {
    cudaError_t e = ssm_setup<T>();
    if (e != cudaSuccess) return e;
    if (a.cu && (e = launch_validate_offsets(a.cu, a.N, a.T, a.status, a.ctrl, a.chunk_start, st, a.L)) !=
                    cudaSuccess)
        return e;
    if ((e = chunk_states<T, false>(a, st)) != cudaSuccess) return e;
    return state_pass<false>(a, st);
}

template <typename T>
cudaError_t fwd(const SsmArgs &a, cudaStream_t st) {
    cudaError_t e = states<T>(a, st);
    if (e != cudaSuccess) return e;
    const int64_t blocks = a.slots * a.H * ((a.P + kL - 1) / kL);
    if (blocks == 0) return cudaSuccess;
    if (blocks > INT32_MAX) return cudaErrorInvalidValue;
    prof_begin("ssm_chunk_out", st);
    ssm_chunk_out_kernel<T><<<(unsigned)blocks, 256, kSmemOut, st>>>(a);
    prof_end(st);
    return cudaGetLastError();
}

cudaError_t param_sums(const SsmArgs &a, cudaStream_t st) {
    prof_begin("ssm_param_sum", st);
    const bool first = a.slots == 0 && a.N == 0;  // neither chunks nor states
    const cudaError_t e = launch_next(first, ssm_param_sum_kernel, (3 * a.H + 3) / 4, 128, 0, st, a);
    prof_end(st);
    return e;
}

template <typename T>
cudaError_t bwd(const SsmArgs &a, cudaStream_t st) {
    cudaError_t e = ssm_setup<T>();
    if (e != cudaSuccess) return e;
    if ((e = chunk_states<T, true>(a, st)) != cudaSuccess) return e;
    if ((e = state_pass<true>(a, st)) != cudaSuccess) return e;
    const int64_t rows = (int64_t)a.B * a.T;
    if (a.slots > 0) {  // (slots x H fits a grid: chunk_states has checked it)
        prof_begin("ssm_chunk_grads", st);
        ssm_chunk_grads_kernel<T><<<(unsigned)(a.slots * a.H), 256, kSmemGrads, st>>>(a);
        prof_end(st);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
    }
    const int64_t elems = rows * a.G * a.Ns;
    if (elems > 0) {
        prof_begin("ssm_group_sum", st);
        ssm_group_sum_kernel<T><<<(unsigned)((elems + 255) / 256), 256, 0, st>>>(a, rows);
        prof_end(st);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
    }
    return param_sums(a, st);
}

}  // namespace

int ssm_chunk_len(kda_dtype dt, int Ns, int P) { return ssm_tc_supported(dt, Ns, P) ? 128 : kL; }

namespace {
cudaError_t tc_states(const SsmArgs &a, cudaStream_t st) {
    if (a.cu) {
        const cudaError_t e =
            launch_validate_offsets(a.cu, a.N, a.T, a.status, a.ctrl, a.chunk_start, st, a.L);
        if (e != cudaSuccess) return e;
    }
    return launch_ssm_tc_states(a, st);
}
}  // namespace

cudaError_t launch_ssm_states(const SsmArgs &a, kda_dtype dt, cudaStream_t st) {
    if (ssm_tc_supported(dt, a.Ns, a.P)) return tc_states(a, st);
    return dt == KDA_DTYPE_BF16 ? states<__nv_bfloat16>(a, st) : states<float>(a, st);
}
cudaError_t launch_ssm_fwd(const SsmArgs &a, kda_dtype dt, cudaStream_t st) {
    if (ssm_tc_supported(dt, a.Ns, a.P)) {
        const cudaError_t e = tc_states(a, st);
        return e != cudaSuccess ? e : launch_ssm_tc_out(a, st);
    }
    return dt == KDA_DTYPE_BF16 ? fwd<__nv_bfloat16>(a, st) : fwd<float>(a, st);
}
cudaError_t launch_ssm_bwd(const SsmArgs &a, kda_dtype dt, cudaStream_t st) {
    if (ssm_tc_supported(dt, a.Ns, a.P)) {
        cudaError_t e = launch_ssm_tc_dstates(a, st);
        if (e == cudaSuccess) e = launch_ssm_tc_bwd(a, st);
        return e == cudaSuccess ? param_sums(a, st) : e;
    }
    return dt == KDA_DTYPE_BF16 ? bwd<__nv_bfloat16>(a, st) : bwd<float>(a, st);
}

cudaError_t launch_ssm_step(const SsmStepArgs &a, kda_dtype dt, cudaStream_t st) {
    const int64_t blocks = (int64_t)a.N * a.H;
    if (blocks == 0) return cudaSuccess;
    if (blocks > INT32_MAX) return cudaErrorInvalidValue;
    const bool vec = a.P % 4 == 0 && aligned_to(a.state, 16);
    const int pq = vec ? a.P / 4 : a.P;
    const unsigned threads = (unsigned)(pq * (256 / pq > 0 ? 256 / pq : 1));
    prof_begin("ssm_step", st);
    if (dt == KDA_DTYPE_BF16) {
        if (vec) ssm_step_kernel<__nv_bfloat16, 4><<<(unsigned)blocks, threads, 0, st>>>(a);
        else ssm_step_kernel<__nv_bfloat16, 1><<<(unsigned)blocks, threads, 0, st>>>(a);
    } else {
        if (vec) ssm_step_kernel<float, 4><<<(unsigned)blocks, threads, 0, st>>>(a);
        else ssm_step_kernel<float, 1><<<(unsigned)blocks, threads, 0, st>>>(a);
    }
    prof_end(st);
    return cudaGetLastError();
}

}  // namespace kda
