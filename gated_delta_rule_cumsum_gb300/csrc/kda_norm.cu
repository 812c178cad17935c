// kda_norm.cu -- a block's entry: the residual's addition and the RMS norm in one pass,
// with the output in the input's type or in 8 bits with scales, and the gradients.
//
//     h = x + res,   y = h w / sqrt(mean(h^2) + eps)
//     8 bits: scale = max |y| / top over a row (or over 128 columns of it; 1 where every
//     y is 0, NaN where one is), q = round(y (1 / scale)), top = 448 (e4m3) or 127 (int8)
//
// A row stays in its threads' registers between the sums and the output, so every input
// is read once and every output written once: bandwidth-bound (2 flops a byte).  The sum
// h is kept in fp32 for the norm; the stored h is rounded once, beside it.
//
// Measured, GB300, bf16: forward 16384 x 2048 43.5 us (268 MB, 6.2 TB/s), 8192 x 4096 to e4m3
// 48 us (235 MB, 4.9 TB/s); backward 16384 x 2048 52 us (268 MB, 5.2 TB/s).
// Spills (bytes stored per thread, aligned rows): bf16 forward of 2049 to 4096 columns 8, 28 to 8
// bits; bf16 backward of 513 to 8192 columns 16; fp32 forward past 4096 columns 84, backward 264; and
// in blocks of 1024 threads, bf16 past 8192 columns 304 forward and 536 backward, fp32 backward
// 1064: at 16384 columns 3.7 TB/s forward, 1.7 backward (bf16), 5.7 and 1.5 (fp32).
#include <cuda_fp8.h>

#include <algorithm>

#include "kda_block.cuh"

namespace kda {
namespace {

// Threads that share a row: `tpr` (a multiple of 32); blockDim.x / tpr rows per block.
// red holds one float per warp and value; a caller takes two in turn, so that a warp which
// is one sum ahead writes the other one.
template <int N>
__device__ __forceinline__ void row_sum(float (&v)[N], int tpr, float *red) {
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
    if (tpr == 32) return;
    const int warps = tpr >> 5, warp = threadIdx.x >> 5, first = (threadIdx.x / tpr) * warps;
    if ((threadIdx.x & 31) == 0)
#pragma unroll
        for (int i = 0; i < N; ++i) red[i * 32 + warp] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
        float s = 0.f;
        for (int k = 0; k < warps; ++k) s += red[i * 32 + first + k];
        v[i] = s;
    }
}
// The larger, or NaN if either is NaN: a NaN in a row has to show in its scale, since int8
// has no code for it.
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float row_max(float v, int tpr, float *red) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = max_nan(v, __shfl_xor_sync(0xffffffffu, v, o));
    if (tpr == 32) return v;
    const int warps = tpr >> 5, warp = threadIdx.x >> 5, first = (threadIdx.x / tpr) * warps;
    if ((threadIdx.x & 31) == 0) red[warp] = v;
    __syncthreads();
    for (int k = 0; k < warps; ++k) v = max_nan(v, red[first + k]);
    return v;
}

// The j-th column of a row's vector v.  Vector loads want a thread's columns adjacent; where
// rows are not aligned for those, a warp's 32 VEC columns are dealt to its lanes in turn, so
// that each scalar access of the warp is still contiguous (8192 x 4095 bf16: 98 us forward
// against 175 with adjacent columns; the backward, whose time is in its sums, keeps them
// adjacent: 147 us against 138, but 166 against 197 at 16384 x 2049).  Either way a group of 128 columns lies in one warp.
template <int VEC, bool AL>
__device__ __forceinline__ int col_of(int v, int j) {
    return AL ? v * VEC + j : (v & ~31) * VEC + (v & 31) + 32 * j;
}
// The columns of vector v, converted, to a row of `cols` columns.
template <typename T, int VEC, bool AL>
__device__ __forceinline__ void store_cols(T *row, int v, int cols, const float (&f)[VEC]) {
    if constexpr (AL) {
        if (v * VEC < cols) store_vec<T, VEC, true>(row + v * VEC, VEC, f);
    } else {
#pragma unroll
        for (int j = 0; j < VEC; ++j)
            if (col_of<VEC, AL>(v, j) < cols) row[col_of<VEC, AL>(v, j)] = from_f32<T>(f[j]);
    }
}

// The same to 8 bits.
template <int VEC, bool AL>
__device__ __forceinline__ void store_q(uint8_t *row, int c, int cols, const float (&v)[VEC], int out) {
    union {
        uint8_t b[VEC];
        uint32_t w[VEC / 4];
    } u;
    if (out == KDA_NORM_E4M3) {
#pragma unroll
        for (int i = 0; i < VEC; i += 2) {
            const __nv_fp8x2_storage_t f =
                __nv_cvt_float2_to_fp8x2(make_float2(v[i], v[i + 1]), __NV_SATFINITE, __NV_E4M3);
            u.b[i] = (uint8_t)(f & 0xff);
            u.b[i + 1] = (uint8_t)(f >> 8);
        }
    } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i)
            u.b[i] = (uint8_t)(int8_t)__float2int_rn(fminf(fmaxf(v[i], -127.f), 127.f));
    }
    if constexpr (AL) {
        if (c * VEC >= cols) return;
        if constexpr (VEC == 8) *reinterpret_cast<uint2 *>(row + c * VEC) = make_uint2(u.w[0], u.w[1]);
        else *reinterpret_cast<uint32_t *>(row + c * VEC) = u.w[0];
    } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i)
            if (col_of<VEC, AL>(c, i) < cols) row[col_of<VEC, AL>(c, i)] = u.b[i];
    }
}

// VEC columns as they lie in memory: loaded for the next row while this one is worked on.
template <typename T, int VEC, bool AL>
struct alignas(VEC * sizeof(T)) Vec {
    T v[VEC];
    // VEC adjacent columns, the first n of them where the row is not aligned
    __device__ __forceinline__ void load(const T *p, int n) {
        static_assert(VEC * sizeof(T) == 16, "vectors of 16 bytes");
        if constexpr (AL) {
            *reinterpret_cast<uint4 *>(v) = *reinterpret_cast<const uint4 *>(p);
        } else {
#pragma unroll
            for (int j = 0; j < VEC; ++j) v[j] = j < n ? p[j] : from_f32<T>(0.f);
        }
    }
    // the columns of vector c of a row of `cols` columns; those past them stay
    __device__ __forceinline__ void load_cols(const T *row, int c, int cols) {
        if constexpr (AL) {
            if (c * VEC < cols) load(row + c * VEC, VEC);
        } else {
#pragma unroll
            for (int j = 0; j < VEC; ++j)
                if (col_of<VEC, AL>(c, j) < cols) v[j] = row[col_of<VEC, AL>(c, j)];
        }
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int j = 0; j < VEC; ++j) v[j] = from_f32<T>(0.f);
    }
    __device__ __forceinline__ void widen(float (&f)[VEC]) const { load_vec<T, VEC, true>(v, VEC, f); }
    // in pairs, for the packed operations
    __device__ __forceinline__ void widen(uint64_t (&f)[VEC / 2]) const {
        const uint32_t *u = reinterpret_cast<const uint32_t *>(v);
#pragma unroll
        for (int j = 0; j < VEC / 2; ++j)
            f[j] = sizeof(T) == 4 ? pack2(u[2 * j], u[2 * j + 1]) : pack2(u[j] << 16, u[j] & 0xffff0000u);
    }
};
// Blocks of MAXT threads that an SM holds in the forward: of 256 threads four with one or two
// vectors per thread (64 registers), two with four, which need more of them.
constexpr int blocks_per_sm(int maxt, int nv) { return maxt > 256 ? 1 : nv == 4 ? 2 : 4; }

// NV vectors of VEC columns per thread: thread i of a row holds vectors i, i + tpr, ...
// Eight (bf16) or four (fp32) adjacent columns per thread make a 128-column scale group
// 16 or 32 adjacent lanes of one warp.  A grid that fills the GPU once walks over the rows:
// the weights stay in registers, and a row's loads are issued while the row before it is
// summed and stored.
template <typename T, int VEC, int NV, bool AL, bool Q, int MAXT>
__global__ void __launch_bounds__(MAXT, blocks_per_sm(MAXT, NV)) norm_fwd_kernel(NormArgs p, int tpr) {
    __shared__ float red[2][2][32];  // [sum, largest], in turn
    const int rpb = blockDim.x / tpr, tid = threadIdx.x % tpr;
    const int64_t first = (int64_t)blockIdx.x * rpb + threadIdx.x / tpr, step = (int64_t)gridDim.x * rpb;
    // every thread makes the same number of rounds: the sums have block-wide barriers
    const int64_t rounds = (p.rows + step - 1) / step;
    float w[NV][VEC];
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
            const int c = col_of<VEC, AL>(tid + i * tpr, j);
            w[i][j] = c < p.cols ? p.w[c] : 0.f;
        }
    Vec<T, VEC, AL> xn[NV], rn[NV];
    auto fetch = [&](int64_t row) {
        const T *x = static_cast<const T *>(p.x) + row * p.cols, *r = static_cast<const T *>(p.res) + row * p.cols;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            xn[i].zero();  // rows and columns past the last add nothing
            rn[i].zero();
            if (row < p.rows) {
                xn[i].load_cols(x, tid + i * tpr, p.cols);
                if (p.res) rn[i].load_cols(r, tid + i * tpr, p.cols);
            }
        }
    };
    fetch(first);
    const int groups = p.group ? (p.cols + 127) / 128 : 1;
    for (int64_t k = 0; k < rounds; ++k) {
        const int64_t row = first + k * step;
        const bool live = row < p.rows;
        float v[NV][VEC], ss[1] = {0.f};
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            float r[VEC];
            xn[i].widen(v[i]);
            rn[i].widen(r);
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                v[i][j] += r[j];
                ss[0] = fmaf(v[i][j], v[i][j], ss[0]);
            }
        }
        if (k + 1 < rounds) fetch(row + step);
        if (p.h) {
            T *h = static_cast<T *>(p.h) + row * p.cols;
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (live) store_cols<T, VEC, AL>(h, tid + i * tpr, p.cols, v[i]);
        }
        row_sum<1>(ss, tpr, red[0][k & 1]);
        const float rstd = 1.f / sqrtf(ss[0] / (float)p.cols + p.eps);
        float amax = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                v[i][j] = v[i][j] * rstd * w[i][j];
                if (Q) amax = max_nan(amax, fabsf(v[i][j]));
            }
            if constexpr (!Q)
                if (live) store_cols<T, VEC, AL>(static_cast<T *>(p.y) + row * p.cols, tid + i * tpr, p.cols, v[i]);
        }
        if constexpr (Q) {
            const float top = p.out == KDA_NORM_E4M3 ? 448.f : 127.f;
            uint8_t *q = static_cast<uint8_t *>(p.y) + row * p.cols;
            if (p.group == 0) amax = row_max(amax, tpr, red[1][k & 1]);
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                // scales of the vector's columns: one, or (dealt to the lanes) one per four
                constexpr int S = AL ? 1 : VEC / 4;
                const int c = tid + i * tpr;
                float m[S], inv[S];
#pragma unroll
                for (int s = 0; s < S; ++s) {
                    m[s] = p.group ? 0.f : amax;
                    if (p.group) {
#pragma unroll
                        for (int j = 0; j < VEC / S; ++j) m[s] = max_nan(m[s], fabsf(v[i][VEC / S * s + j]));
#pragma unroll
                        for (int o = AL ? 64 / VEC : 16; o > 0; o >>= 1)
                            m[s] = max_nan(m[s], __shfl_xor_sync(0xffffffffu, m[s], o));
                    }
                    // at least the smallest normal number, so that 1 / scale is finite
                    const float scale = m[s] == 0.f ? 1.f : max_nan(m[s] / top, 1.17549435e-38f);
                    inv[s] = 1.f / scale;
                    const int first = col_of<VEC, AL>(c, VEC / S * s);
                    if (live && first < p.cols && (p.group ? first % 128 == 0 : first == 0))
                        p.scale[row * groups + (p.group ? first / 128 : 0)] = scale;
                }
#pragma unroll
                for (int j = 0; j < VEC; ++j) v[i][j] *= inv[j * S / VEC];
                if (live) store_q<VEC, AL>(q, c, p.cols, v[i], p.out);
            }
        }
    }
}

// Gradients at the stored h:  with g = dy w, xhat = h rstd,
//     dx = rstd (g - xhat mean(g xhat)) + dres,    dw = sum over rows of dy xhat.
// Both row sums (h^2 and g h) come from one exchange.  The grid walks over the rows as the
// forward's does; a thread keeps its columns' share of dw in registers and leaves it in p.part,
// and a second kernel adds the shares in a fixed order.
// Two vectors per thread (of eight columns in bf16, four in fp32) rather than as many threads:
// what a row costs beside its columns (sums over threads, addresses, a barrier) is shared.
template <typename T, int VEC, int NV, bool AL, int MAXT, int BLOCKS>
__global__ void __launch_bounds__(MAXT, BLOCKS) norm_bwd_kernel(NormArgs p, int tpr) {
    follow();
    __shared__ float red[2][64];
    constexpr int VP = VEC / 2;
    const int rpb = blockDim.x / tpr, tid = threadIdx.x % tpr;
    uint64_t dw[NV][VP] = {}, w[NV][VP];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (tid + i * tpr) * VEC, n = min(VEC, p.cols - c);
#pragma unroll
        for (int j = 0; j < VP; ++j)
            w[i][j] = pack2(2 * j < n ? p.w[c + 2 * j] : 0.f, 2 * j + 1 < n ? p.w[c + 2 * j + 1] : 0.f);
    }
    const int64_t first = (int64_t)blockIdx.x * rpb + threadIdx.x / tpr, step = (int64_t)gridDim.x * rpb;
    const int64_t rounds = (p.rows + step - 1) / step, apart = step * p.cols;
    Vec<T, VEC, AL> hn[NV], gn[NV], rn[NV];
    int64_t at = first * p.cols + tid * VEC;  // of the row in hand; the next one's are on their way
    auto fetch = [&](int64_t row, int64_t next) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int n = min(VEC, p.cols - (tid + i * tpr) * VEC);
            hn[i].zero();
            gn[i].zero();
            rn[i].zero();
            if (row < p.rows && n > 0) {
                hn[i].load(static_cast<const T *>(p.h) + next + i * tpr * VEC, n);
                gn[i].load(static_cast<const T *>(p.dy) + next + i * tpr * VEC, n);
                if (p.dres) rn[i].load(static_cast<const T *>(p.dres) + next + i * tpr * VEC, n);
            }
        }
    };
    fetch(first, at);
    for (int64_t k = 0; k < rounds; ++k, at += apart) {
        const int64_t row = first + k * step;
        uint64_t h[NV][VP], g[NV][VP], s2[2] = {0, 0};
        Vec<T, VEC, AL> r[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            hn[i].widen(h[i]);
            gn[i].widen(g[i]);
            r[i] = rn[i];
#pragma unroll
            for (int j = 0; j < VP; ++j) {
                s2[0] = fma2(h[i][j], h[i][j], s2[0]);
                s2[1] = fma2(mul2(g[i][j], w[i][j]), h[i][j], s2[1]);
            }
        }
        if (k + 1 < rounds) fetch(row + step, at + apart);
        float s[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            float x, y;
            unpack2(s2[i], x, y);
            s[i] = x + y;
        }
        row_sum<2>(s, tpr, red[k & 1]);
        // (0 for threads without a row: with eps = 0 their zeros would give dw NaN)
        const float rstd = row < p.rows ? 1.f / sqrtf(s[0] / (float)p.cols + p.eps) : 0.f;
        const float m = -s[1] / (float)p.cols * rstd;  // - mean(g xhat)
        const uint64_t rstd2 = pack2(rstd, rstd), m2 = pack2(m, m);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int n = min(VEC, p.cols - (tid + i * tpr) * VEC);
            uint64_t res[VP];
            r[i].widen(res);
            float o[VEC];
#pragma unroll
            for (int j = 0; j < VP; ++j) {
                const uint64_t xh = mul2(h[i][j], rstd2);
                dw[i][j] = fma2(g[i][j], xh, dw[i][j]);
                unpack2(fma2(rstd2, fma2(xh, m2, mul2(g[i][j], w[i][j])), res[j]), o[2 * j], o[2 * j + 1]);
            }
            if (row < p.rows && n > 0) store_vec<T, VEC, AL>(static_cast<T *>(p.dx) + at + i * tpr * VEC, n, o);
        }
    }
    float *part = p.part + first * p.cols;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (tid + i * tpr) * VEC;
#pragma unroll
        for (int j = 0; j < VP; ++j) {
            float x, y;
            unpack2(dw[i][j], x, y);
            if (c + 2 * j < p.cols) part[c + 2 * j] = x;
            if (c + 2 * j + 1 < p.cols) part[c + 2 * j + 1] = y;
        }
    }
}

// dw: 32 warps to 32 columns, each adding every 32nd share, then their sums in order.
__global__ void __launch_bounds__(1024) norm_bwd_sum_kernel(const float *part, int64_t parts, int cols,
                                                            float *dw) {
    follow();
    __shared__ float red[32][33];
    const int lane = threadIdx.x & 31, grp = threadIdx.x >> 5;
    const int64_t c = (int64_t)blockIdx.x * 32 + lane;
    float s = 0.f;
    if (c < cols) {
#pragma unroll 8
        for (int64_t r = grp; r < parts; r += 32) s += part[r * cols + c];
    }
    red[grp][lane] = s;
    __syncthreads();
    if (grp == 0 && c < cols) {
        for (int g = 1; g < 32; ++g) s += red[g][lane];
        dw[c] = s;
    }
}

// Threads per row, vectors per thread and rows per block of a row of `vecs` vectors; short
// rows share a block of 128 threads.
struct RowPlan {
    int tpr, nv, rpb;
};
RowPlan plan_of(int vecs, int nv) {
    RowPlan r{};
    r.nv = nv;
    r.tpr = ((vecs + nv - 1) / nv + 31) / 32 * 32;
    r.rpb = r.tpr < 128 ? 128 / r.tpr : 1;
    return r;
}
// Forward: the fewest vectors per thread (1, 2 or 4) that keep a row within 256 threads
// (16384 x 2048 bf16: 43.5 us, 47.9 with two), and four with up to 1024 threads for the
// longest rows (16384 columns).
RowPlan fwd_plan(int vecs) { return plan_of(vecs, vecs <= 256 ? 1 : vecs <= 512 ? 2 : 4); }
// Backward: two vectors per thread from 64 vectors on (8192 x 2048 bf16: 27 us against 32 with
// one; 16384 x 1024: 29.4 against 30.6), and four of fp32 where two would take more than 512
// threads.
RowPlan bwd_plan(int cols, bool bf) {
    const int vecs = bf ? (cols + 7) / 8 : (cols + 3) / 4;
    return plan_of(vecs, vecs <= 64 ? 1 : bf || vecs <= 1024 ? 2 : 4);
}

bool norm_aligned(const NormArgs &a, size_t e, const void *const *ptrs, int count) {
    const size_t bytes = 16;
    for (int i = 0; i < count; ++i)
        if (!aligned_to(ptrs[i], bytes)) return false;
    return ((size_t)a.cols * e) % bytes == 0 && aligned_to(a.w, 16);
}

// f(vectors per thread, most threads per block)
template <typename F>
void by_plan(const RowPlan &r, F &&f) {
    if (r.tpr > 256)
        f(std::integral_constant<int, 4>(), std::integral_constant<int, 1024>());
    else if (r.nv == 1)
        f(std::integral_constant<int, 1>(), std::integral_constant<int, 256>());
    else if (r.nv == 2)
        f(std::integral_constant<int, 2>(), std::integral_constant<int, 256>());
    else
        f(std::integral_constant<int, 4>(), std::integral_constant<int, 256>());
}

// Blocks of either direction: what the GPU's 152 SMs hold at once, at most one per row (the
// backward leaves one row of partial sums per row that a block works on at a time).
int64_t row_blocks(int64_t rows, const RowPlan &r, int threads_per_sm) {
    const int64_t want = kSms * (int64_t)std::max(threads_per_sm / (r.tpr * r.rpb), 1);
    return std::min(want, (rows + r.rpb - 1) / r.rpb);
}
int64_t fwd_blocks(int64_t rows, const RowPlan &r) {
    return row_blocks(rows, r, r.tpr > 256 ? 1024 : 256 * blocks_per_sm(256, r.nv));
}
int64_t bwd_blocks(int64_t rows, const RowPlan &r) { return row_blocks(rows, r, r.nv == 1 ? 768 : 512); }

}  // namespace

int64_t norm_bwd_parts(int64_t rows, int cols, kda_dtype dt) {
    const RowPlan r = bwd_plan(cols, dt == KDA_DTYPE_BF16);
    return bwd_blocks(rows, r) * r.rpb;
}

cudaError_t launch_norm_fwd(const NormArgs &a, kda_dtype dt, cudaStream_t st) {
    if (a.rows == 0) return cudaSuccess;
    const void *ptrs[] = {a.x, a.res, a.h, a.y};
    const bool bf = dt == KDA_DTYPE_BF16, q = a.out != KDA_NORM_SAME;
    const bool al = norm_aligned(a, bf ? 2 : 4, ptrs, 4);
    const int vec = bf ? 8 : 4;
    const RowPlan r = fwd_plan((a.cols + vec - 1) / vec);
    if (r.tpr > 1024) return cudaErrorInvalidValue;
    const int64_t blocks = fwd_blocks(a.rows, r);
    prof_begin("norm_fwd", st);
    by_plan(r, [&](auto NV, auto MAXT) {
        const unsigned g = (unsigned)blocks, t = (unsigned)(r.tpr * r.rpb);
#define KDA_NORM_FWD(T, VEC, AL, Q) norm_fwd_kernel<T, VEC, NV(), AL, Q, MAXT()><<<g, t, 0, st>>>(a, r.tpr)
        if (bf) {
            if (al) {
                if (q) KDA_NORM_FWD(__nv_bfloat16, 8, true, true);
                else KDA_NORM_FWD(__nv_bfloat16, 8, true, false);
            } else {
                if (q) KDA_NORM_FWD(__nv_bfloat16, 8, false, true);
                else KDA_NORM_FWD(__nv_bfloat16, 8, false, false);
            }
        } else if (al) {
            if (q) KDA_NORM_FWD(float, 4, true, true);
            else KDA_NORM_FWD(float, 4, true, false);
        } else {
            if (q) KDA_NORM_FWD(float, 4, false, true);
            else KDA_NORM_FWD(float, 4, false, false);
        }
#undef KDA_NORM_FWD
    });
    prof_end(st);
    return cudaGetLastError();
}

cudaError_t launch_norm_bwd(const NormArgs &a, kda_dtype dt, cudaStream_t st) {
    const bool bf = dt == KDA_DTYPE_BF16;
    const void *ptrs[] = {a.h, a.dy, a.dres, a.dx};
    const bool al = norm_aligned(a, bf ? 2 : 4, ptrs, 4);
    const RowPlan r = bwd_plan(a.cols, bf);
    if (r.tpr > 1024) return cudaErrorInvalidValue;
    const int64_t blocks = bwd_blocks(a.rows, r);
    if (blocks > 0) {
        using std::integral_constant;
        prof_begin("norm_bwd", st);
        auto go = [&](auto NV, auto MAXT, auto BLOCKS) {
            const unsigned g = (unsigned)blocks, t = (unsigned)(r.tpr * r.rpb);
            constexpr int nv = NV(), maxt = MAXT(), per_sm = BLOCKS();
            if constexpr (nv <= 2) {
                if (bf && al) norm_bwd_kernel<__nv_bfloat16, 8, nv, true, maxt, per_sm><<<g, t, 0, st>>>(a, r.tpr);
                if (bf && !al) norm_bwd_kernel<__nv_bfloat16, 8, nv, false, maxt, per_sm><<<g, t, 0, st>>>(a, r.tpr);
            }
            if constexpr (nv == 4 || maxt <= 512) {
                if (!bf && al) norm_bwd_kernel<float, 4, nv, true, maxt, per_sm><<<g, t, 0, st>>>(a, r.tpr);
                if (!bf && !al) norm_bwd_kernel<float, 4, nv, false, maxt, per_sm><<<g, t, 0, st>>>(a, r.tpr);
            }
        };
        using One = integral_constant<int, 1>;
        using Two = integral_constant<int, 2>;
        using Four = integral_constant<int, 4>;
        using Short = integral_constant<int, 256>;
        using Long = integral_constant<int, 512>;
        using Longest = integral_constant<int, 1024>;
        if (r.nv == 1) go(One(), Short(), integral_constant<int, 3>());
        else if (r.nv == 2 && r.tpr <= 256) go(Two(), Short(), Two());
        else if (r.nv == 2) r.tpr <= 512 ? go(Two(), Long(), One()) : go(Two(), Longest(), One());
        else r.tpr <= 512 ? go(Four(), Long(), One()) : go(Four(), Longest(), One());
        prof_end(st);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    prof_begin("norm_bwd_sum", st);
    const cudaError_t e = launch_next(blocks == 0, norm_bwd_sum_kernel, (a.cols + 31) / 32, 1024, 0, st, a.part,
                                      blocks * r.rpb, a.cols, a.dw);
    prof_end(st);
    return e;
}

}  // namespace kda
