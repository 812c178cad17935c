// kda_conv.cu -- the short causal depthwise convolution that a recurrent block puts in
// front of its state update (KDA's q, k, v; the scan's x, B, C): forward, gradients and
// the single-token form.
//
//     pre_t[c] = bias[c] + sum_{k < W} w[c, k] x_{t - W + 1 + k}[c],   y = pre or silu(pre)
//
// where rows before a sequence's first are its carried state (the W - 1 rows that came
// before), or zero.  2 W flops against 2 elements moved: bandwidth-bound at every size.
// A thread owns a few adjacent channels and walks down a strip of rows with the last
// W - 1 rows in registers, so each row is read once (and W - 1 rows more per strip, from
// L2).  All arithmetic is fp32; outputs are rounded once.
#include "kda_block.cuh"

namespace kda {
namespace {

constexpr int kConvThreads = 128;

template <typename T>
__device__ __forceinline__ float sigmoid_of(float x) {
    if constexpr (sizeof(T) == 4)
        return 1.f / (1.f + expf(-x));
    else  // the fast exponential and division: about 2^-21, far inside the output's rounding
        return __fdividef(1.f, 1.f + __expf(-x));
}

// The sequence that row t (of all B * T rows) belongs to: its index, first row and end.
// False past the last offset.  Stays in bounds, and end > t, for any offsets.
__device__ __forceinline__ bool find_seq(const ConvArgs &p, int64_t t, int &n, int64_t &s,
                                         int64_t &e) {
    if (p.cu) {
        n = upper_bound_minus_one(p.cu, p.N + 1, (int)t);
        if (n >= p.N) return false;
        s = min((int64_t)max(p.cu[n], 0), t);
        e = min((int64_t)p.cu[n + 1], (int64_t)p.T);
        if (e <= t) return false;
    } else {
        n = (int)(t / p.T);
        s = (int64_t)n * p.T;
        e = s + p.T;
    }
    return true;
}

template <typename T, int VEC, int W, bool AL>
__global__ void __launch_bounds__(kConvThreads) conv_fwd_kernel(ConvArgs p) {
    const int cblocks = (p.C + VEC * kConvThreads - 1) / (VEC * kConvThreads);
    const int64_t strip = blockIdx.x / cblocks;
    const int c = ((int)(blockIdx.x % cblocks) * kConvThreads + threadIdx.x) * VEC;
    if (p.cu && blockIdx.x == 0) check_offsets(p.cu, p.N, p.T, p.status);
    if (c >= p.C) return;
    const int nc = min(VEC, p.C - c);
    const T *x = static_cast<const T *>(p.x) + c;
    const T *st = static_cast<const T *>(p.state_in);

    if (strip >= p.strips) {  // the final state of one sequence: its last W - 1 rows
        const int n = (int)(strip - p.strips);
        int64_t s, e;
        if (p.cu) {
            s = min(max(p.cu[n], 0), p.T);
            e = min((int64_t)max((int64_t)p.cu[n + 1], s), (int64_t)p.T);
        } else {
            s = (int64_t)n * p.T;
            e = s + p.T;
        }
        T *out = static_cast<T *>(p.state_out) + (int64_t)n * (W - 1) * p.C + c;
#pragma unroll
        for (int k = 0; k < W - 1; ++k) {
            const int64_t r = e - (W - 1) + k;
            float v[VEC] = {};
            if (r >= s)
                load_vec<T, VEC, AL>(x + r * p.x_stride, nc, v);
            else if (st)
                load_vec<T, VEC, AL>(st + ((int64_t)n * (W - 1) + (W - 1) + (r - s)) * p.C + c, nc, v);
            store_vec<T, VEC, AL>(out + (int64_t)k * p.C, nc, v);
        }
        return;
    }

    float w[W][VEC], bias[VEC];
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
        const bool in = j < nc;
        bias[j] = in && p.bias ? p.bias[c + j] : 0.f;
#pragma unroll
        for (int k = 0; k < W; ++k) w[k][j] = in ? p.w[(int64_t)(c + j) * W + k] : 0.f;
    }
    T *y = static_cast<T *>(p.y) + c;
    constexpr int U = 4;  // rows loaded ahead of their arithmetic
    const int64_t t1 = min((strip + 1) * (int64_t)p.strip, (int64_t)p.B * p.T);
    for (int64_t t = strip * p.strip; t < t1;) {
        int n;
        int64_t s, e;
        if (!find_seq(p, t, n, s, e)) return;
        e = min(e, t1);
        float win[W - 1 + U][VEC];
#pragma unroll
        for (int k = 0; k < W - 1; ++k) {
            const int64_t r = t - (W - 1) + k;
#pragma unroll
            for (int j = 0; j < VEC; ++j) win[k][j] = 0.f;
            if (r >= s)
                load_vec<T, VEC, AL>(x + r * p.x_stride, nc, win[k]);
            else if (st)
                load_vec<T, VEC, AL>(st + ((int64_t)n * (W - 1) + (W - 1) + (r - s)) * p.C + c, nc,
                                     win[k]);
        }
        for (; t < e; t += U) {
            const int rows = (int)min((int64_t)U, e - t);
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (u < rows) load_vec<T, VEC, AL>(x + (t + u) * p.x_stride, nc, win[W - 1 + u]);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (u >= rows) break;
                float o[VEC];
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    float a = bias[j];
#pragma unroll
                    for (int k = 0; k < W; ++k) a = fmaf(w[k][j], win[u + k][j], a);
                    o[j] = p.silu ? a * sigmoid_of<T>(a) : a;
                }
                store_vec<T, VEC, AL>(y + (t + u) * p.C, nc, o);
            }
            if (rows < U) {  // the sequence or the strip ends inside this group
                t += rows;
                break;
            }
#pragma unroll
            for (int k = 0; k < W - 1; ++k)
#pragma unroll
                for (int j = 0; j < VEC; ++j) win[k][j] = win[U + k][j];
        }
    }
}

// Gradients.  With dpre_u = dy_u act'(pre_u), dx_t = sum_m w[W-1-m] dpre_{t+m} over the
// rows t + m of t's sequence, plus the final state's gradient for the last W - 1 rows;
// rows before the sequence are the carried state's.  A thread walks "position" t from
// W - 1 rows before its strip to the strip's last row, holding x and dpre of rows
// t .. t + W - 1; the row that enters is u = t + W - 1.  dw and dbias take the rows of
// the strip alone; each strip leaves its sums in p.part and a second kernel adds the
// strips in order, so that no result depends on the order of atomics.
template <typename T, int VEC, int W, bool AL>
__global__ void __launch_bounds__(kConvThreads) conv_bwd_kernel(ConvArgs p) {
    const int cblocks = (p.C + VEC * kConvThreads - 1) / (VEC * kConvThreads);
    const int64_t strip = blockIdx.x / cblocks;
    const int c = ((int)(blockIdx.x % cblocks) * kConvThreads + threadIdx.x) * VEC;
    if (p.cu && blockIdx.x == 0) check_offsets(p.cu, p.N, p.T, p.status);
    if (c >= p.C) return;
    const int nc = min(VEC, p.C - c);
    const T *x = static_cast<const T *>(p.x) + c;
    const T *dy = static_cast<const T *>(p.dy) + c;
    const T *st = static_cast<const T *>(p.state_in);
    const T *dso = static_cast<const T *>(p.dstate_out);
    T *dx = static_cast<T *>(p.dx) + c;
    T *dsi = static_cast<T *>(p.dstate_in);

    float w[W][VEC], bias[VEC], dw[W][VEC], db[VEC];
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
        const bool in = j < nc;
        bias[j] = in && p.bias ? p.bias[c + j] : 0.f;
        db[j] = 0.f;
#pragma unroll
        for (int k = 0; k < W; ++k) {
            w[k][j] = in ? p.w[(int64_t)(c + j) * W + k] : 0.f;
            dw[k][j] = 0.f;
        }
    }
    const int64_t t0 = strip * p.strip, t1 = min(t0 + p.strip, (int64_t)p.B * p.T);
    for (int64_t t = t0; t < t1;) {
        int n;
        int64_t s, e;
        if (!find_seq(p, t, n, s, e)) break;
        const int64_t end = min(e, t1);
        float xw[W][VEC] = {}, dp[W][VEC] = {};
#pragma unroll
        for (int k = 0; k < W - 1; ++k) {  // rows t - (W - 1) .. t - 1
            const int64_t r = t - (W - 1) + k;
            if (r >= s)
                load_vec<T, VEC, AL>(x + r * p.x_stride, nc, xw[k + 1]);
            else if (st)
                load_vec<T, VEC, AL>(st + ((int64_t)n * (W - 1) + (W - 1) + (r - s)) * p.C + c, nc,
                                     xw[k + 1]);
        }
        // xw[k] holds row pos + k once the entering row is in; before it, shifted by one
        constexpr int U = 4;
        for (int64_t pos0 = t - (W - 1); pos0 < end; pos0 += U) {
            float xn[U][VEC], gn[U][VEC];
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const int64_t u = pos0 + i + W - 1;
#pragma unroll
                for (int j = 0; j < VEC; ++j) xn[i][j] = gn[i][j] = 0.f;
                if (u < e && pos0 + i < end) {
                    load_vec<T, VEC, AL>(x + u * p.x_stride, nc, xn[i]);
                    load_vec<T, VEC, AL>(dy + u * p.C, nc, gn[i]);
                }
            }
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const int64_t pos = pos0 + i, u = pos + W - 1;
                if (pos >= end) break;
#pragma unroll
                for (int k = 0; k < W - 1; ++k)
#pragma unroll
                    for (int j = 0; j < VEC; ++j) {
                        xw[k][j] = xw[k + 1][j];
                        dp[k][j] = dp[k + 1][j];
                    }
                const bool own = u >= t && u < end;
                float o[VEC];
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    xw[W - 1][j] = xn[i][j];
                    float g = gn[i][j];
                    if (p.silu) {
                        float a = bias[j];
#pragma unroll
                        for (int k = 0; k < W; ++k) a = fmaf(w[k][j], xw[k][j], a);
                        const float sg = sigmoid_of<T>(a);
                        // a select: a row past the sequence has g = 0 whatever sigmoid gives
                        g = u < e ? g * (sg * (1.f + a * (1.f - sg))) : 0.f;
                    }
                    dp[W - 1][j] = g;
                    if (own) {
                        db[j] += g;
#pragma unroll
                        for (int k = 0; k < W; ++k) dw[k][j] = fmaf(g, xw[k][j], dw[k][j]);
                    }
                    float d = 0.f;
#pragma unroll
                    for (int m = 0; m < W; ++m) d = fmaf(w[W - 1 - m][j], dp[m][j], d);
                    o[j] = d;
                }
                const bool state_row = pos < s;
                if (state_row ? (dsi != nullptr && t == s) : pos >= t) {
                    const int64_t k = pos - (e - (W - 1));  // its row of the final state
                    if (dso && k >= 0) {
                        float f[VEC];
                        load_vec<T, VEC, AL>(dso + ((int64_t)n * (W - 1) + k) * p.C + c, nc, f);
#pragma unroll
                        for (int j = 0; j < VEC; ++j) o[j] += f[j];
                    }
                    T *dst = state_row
                                 ? dsi + ((int64_t)n * (W - 1) + (W - 1) + (pos - s)) * p.C + c
                                 : dx + pos * p.C;
                    store_vec<T, VEC, AL>(dst, nc, o);
                }
            }
        }
        t = end;
    }
    float *part = p.part + strip * (int64_t)(W + 1) * p.C + c;
#pragma unroll
    for (int j = 0; j < VEC; ++j)
        if (j < nc) {
#pragma unroll
            for (int k = 0; k < W; ++k) part[(int64_t)k * p.C + j] = dw[k][j];
            part[(int64_t)W * p.C + j] = db[j];
        }
}

// Empty sequences: the carried state passes through, and so does its gradient.
template <typename T>
__global__ void __launch_bounds__(128) conv_bwd_empty_kernel(ConvArgs p) {
    const int n = blockIdx.x;
    const bool empty = p.cu ? p.cu[n + 1] <= p.cu[n] : p.T == 0;
    if (!empty) return;
    const int64_t row = (int64_t)(p.W - 1) * p.C;
    const T *src = static_cast<const T *>(p.dstate_out);
    T *dst = static_cast<T *>(p.dstate_in);
    for (int64_t i = threadIdx.x; i < row; i += blockDim.x)
        dst[n * row + i] = src ? src[n * row + i] : from_f32<T>(0.f);
}

// dw[c][k] and dbias[c] from the strips' partial sums, in the order of the strips: eight
// threads per entry each add every eighth strip, then their sums are added.
__global__ void __launch_bounds__(256) conv_bwd_sum_kernel(const float *part, int64_t strips, int C,
                                                           int W, float *dw, float *dbias) {
    __shared__ float red[8][33];
    const int lane = threadIdx.x & 31, grp = threadIdx.x >> 5;
    const int64_t i = (int64_t)blockIdx.x * 32 + lane, total = (int64_t)(W + 1) * C;
    float s = 0.f;
    if (i < total)
        for (int64_t r = grp; r < strips; r += 8) s += part[r * total + i];
    red[grp][lane] = s;
    __syncthreads();
    if (grp == 0 && i < total) {
        for (int g = 1; g < 8; ++g) s += red[g][lane];
        const int k = (int)(i / C), c = (int)(i % C);
        if (k < W)
            dw[(int64_t)c * W + k] = s;
        else if (dbias)
            dbias[c] = s;
    }
}

template <typename T, int VEC, int W, bool AL>
__global__ void __launch_bounds__(kConvThreads) conv_step_kernel(ConvStepArgs p) {
    const int cblocks = (p.C + VEC * kConvThreads - 1) / (VEC * kConvThreads);
    const int n = blockIdx.x / cblocks;
    const int c = ((int)(blockIdx.x % cblocks) * kConvThreads + threadIdx.x) * VEC;
    const int slot = state_slot(p.idx, n, p.slots, p.status);
    if (c >= p.C) return;
    const int nc = min(VEC, p.C - c);
    T *y = static_cast<T *>(p.y) + (int64_t)n * p.C + c;
    float o[VEC] = {};
    if (slot >= 0) {
        T *st = static_cast<T *>(p.state) + (int64_t)slot * (W - 1) * p.C + c;
        float win[W][VEC];
#pragma unroll
        for (int k = 0; k < W - 1; ++k) load_vec<T, VEC, AL>(st + (int64_t)k * p.C, nc, win[k]);
        load_vec<T, VEC, AL>(static_cast<const T *>(p.x) + (int64_t)n * p.x_stride + c, nc, win[W - 1]);
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
            const int cj = c + min(j, nc - 1);
            float a = p.bias ? p.bias[cj] : 0.f;
#pragma unroll
            for (int k = 0; k < W; ++k) a = fmaf(p.w[(int64_t)cj * W + k], win[k][j], a);
            o[j] = p.silu ? a * sigmoid_of<T>(a) : a;
        }
#pragma unroll
        for (int k = 0; k < W - 1; ++k) store_vec<T, VEC, AL>(st + (int64_t)k * p.C, nc, win[k + 1]);
    }
    store_vec<T, VEC, AL>(y, nc, o);
}

// Whether every row of the given tensors starts on a `bytes` boundary.
bool rows_aligned(const void *const *ptrs, int count, int64_t row_bytes, int64_t x_row_bytes,
                  size_t bytes) {
    for (int i = 0; i < count; ++i)
        if (!aligned_to(ptrs[i], bytes)) return false;
    return row_bytes % (int64_t)bytes == 0 && x_row_bytes % (int64_t)bytes == 0;
}

template <typename F>
cudaError_t by_width(int W, F &&f) {
    switch (W) {
        case 2: f(std::integral_constant<int, 2>()); break;
        case 3: f(std::integral_constant<int, 3>()); break;
        case 4: f(std::integral_constant<int, 4>()); break;
        default: return cudaErrorInvalidValue;
    }
    return cudaGetLastError();
}

int strip_for(int64_t rows, int64_t threads_per_row, int most) {
    int strip = most;
    while (strip > 8 && (rows + strip - 1) / strip * threads_per_row < 152 * 1024) strip /= 2;
    return strip;
}

}  // namespace

// 64 rows where that still gives 152 x 1024 threads (half of what the GPU holds): a strip
// re-reads W - 1 rows, 5% of its traffic at 64; fewer rows where the input is short.
int conv_strip(int B, int T, int C, int vec) {
    return strip_for((int64_t)B * T, (C + vec - 1) / vec, 64);
}
int conv_bwd_strip(int B, int T, int C) {
    return strip_for((int64_t)B * T, (C + 3) / 4, 128);
}

cudaError_t launch_conv_fwd(ConvArgs a, kda_dtype dt, cudaStream_t st) {
    const size_t e = dt == KDA_DTYPE_BF16 ? 2 : 4;
    const void *ptrs[] = {a.x, a.y, a.state_in, a.state_out};
    const bool al = rows_aligned(ptrs, 4, (int64_t)(a.C * e), (int64_t)(a.x_stride * e), 16);
    const int vec = dt == KDA_DTYPE_BF16 && al ? 8 : 4;
    a.strip = conv_strip(a.B, a.T, a.C, vec);
    const int64_t rows = (int64_t)a.B * a.T;
    a.strips = (rows + a.strip - 1) / a.strip;
    const int64_t cblocks = (a.C + vec * kConvThreads - 1) / (vec * kConvThreads);
    const int64_t blocks = cblocks * (a.strips + (a.state_out ? a.N : 0));
    if (blocks == 0) return cudaSuccess;
    if (blocks > INT32_MAX) return cudaErrorInvalidValue;
    prof_begin("conv_fwd", st);
    const cudaError_t err = by_width(a.W, [&](auto W) {
        const unsigned g = (unsigned)blocks;
        if (dt == KDA_DTYPE_BF16) {
            if (al)
                conv_fwd_kernel<__nv_bfloat16, 8, W(), true><<<g, kConvThreads, 0, st>>>(a);
            else
                conv_fwd_kernel<__nv_bfloat16, 4, W(), false><<<g, kConvThreads, 0, st>>>(a);
        } else if (al) {
            conv_fwd_kernel<float, 4, W(), true><<<g, kConvThreads, 0, st>>>(a);
        } else {
            conv_fwd_kernel<float, 4, W(), false><<<g, kConvThreads, 0, st>>>(a);
        }
    });
    prof_end(st);
    return err;
}

cudaError_t launch_conv_bwd(ConvArgs a, kda_dtype dt, cudaStream_t st) {
    const size_t e = dt == KDA_DTYPE_BF16 ? 2 : 4;
    const void *ptrs[] = {a.x, a.dy, a.dx, a.state_in, a.dstate_out, a.dstate_in};
    const bool al = rows_aligned(ptrs, 6, (int64_t)(a.C * e), (int64_t)(a.x_stride * e), 4 * e);
    a.strip = conv_bwd_strip(a.B, a.T, a.C);
    const int64_t rows = (int64_t)a.B * a.T;
    a.strips = (rows + a.strip - 1) / a.strip;
    const int64_t cblocks = (a.C + 4 * kConvThreads - 1) / (4 * kConvThreads);
    const int64_t blocks = cblocks * a.strips;
    if (blocks > INT32_MAX) return cudaErrorInvalidValue;
    cudaError_t err = cudaSuccess;
    if (blocks > 0) {
        prof_begin("conv_bwd", st);
        err = by_width(a.W, [&](auto W) {
            const unsigned g = (unsigned)blocks;
            if (dt == KDA_DTYPE_BF16) {
                if (al)
                    conv_bwd_kernel<__nv_bfloat16, 4, W(), true><<<g, kConvThreads, 0, st>>>(a);
                else
                    conv_bwd_kernel<__nv_bfloat16, 4, W(), false><<<g, kConvThreads, 0, st>>>(a);
            } else if (al) {
                conv_bwd_kernel<float, 4, W(), true><<<g, kConvThreads, 0, st>>>(a);
            } else {
                conv_bwd_kernel<float, 4, W(), false><<<g, kConvThreads, 0, st>>>(a);
            }
        });
        prof_end(st);
        if (err != cudaSuccess) return err;
    }
    if (a.dstate_in && a.N > 0 && (a.cu || a.T == 0)) {
        prof_begin("conv_bwd_empty", st);
        if (dt == KDA_DTYPE_BF16)
            conv_bwd_empty_kernel<__nv_bfloat16><<<(unsigned)a.N, 128, 0, st>>>(a);
        else
            conv_bwd_empty_kernel<float><<<(unsigned)a.N, 128, 0, st>>>(a);
        prof_end(st);
        if ((err = cudaGetLastError()) != cudaSuccess) return err;
    }
    const int64_t total = (int64_t)(a.W + 1) * a.C;
    prof_begin("conv_bwd_sum", st);
    conv_bwd_sum_kernel<<<(unsigned)((total + 31) / 32), 256, 0, st>>>(a.part, a.strips, a.C, a.W,
                                                                       a.dw, a.dbias);
    prof_end(st);
    return cudaGetLastError();
}

cudaError_t launch_conv_step(const ConvStepArgs &a, kda_dtype dt, cudaStream_t st) {
    const size_t e = dt == KDA_DTYPE_BF16 ? 2 : 4;
    const void *ptrs[] = {a.x, a.y, a.state};
    const bool al = rows_aligned(ptrs, 3, (int64_t)(a.C * e), (int64_t)(a.x_stride * e), 4 * e);
    const int64_t blocks = (int64_t)a.N * ((a.C + 4 * kConvThreads - 1) / (4 * kConvThreads));
    if (blocks == 0) return cudaSuccess;
    if (blocks > INT32_MAX) return cudaErrorInvalidValue;
    prof_begin("conv_step", st);
    const cudaError_t err = by_width(a.W, [&](auto W) {
        const unsigned g = (unsigned)blocks;
        if (dt == KDA_DTYPE_BF16) {
            if (al)
                conv_step_kernel<__nv_bfloat16, 4, W(), true><<<g, kConvThreads, 0, st>>>(a);
            else
                conv_step_kernel<__nv_bfloat16, 4, W(), false><<<g, kConvThreads, 0, st>>>(a);
        } else if (al) {
            conv_step_kernel<float, 4, W(), true><<<g, kConvThreads, 0, st>>>(a);
        } else {
            conv_step_kernel<float, 4, W(), false><<<g, kConvThreads, 0, st>>>(a);
        }
    });
    prof_end(st);
    return err;
}

}  // namespace kda
