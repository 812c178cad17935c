// kda_gated_norm.cu -- the norms around a gated block: the output norm with its gate, per group of
// columns, and the norm of a block's output, gated, onto the scaled residual stream with the next
// block's norm behind it.  With rms(x) = x / sqrt(mean x^2 + eps), a = the activated gate:
//   gated     y = rms(x) w a,  or  rms(x a) w  (gate first)
//   sandwich  h = s residual + a rms(x) w_post,  y = rms(h) w_pre
// Both directions are bound by HBM: every tensor is read once and written once (the sandwich's
// gradients form h again from x, the residual and the gate, unrounded, rather than read it).
// A team of threads has a group (or a row): NV vectors of VEC columns per thread, all of them in
// registers.  Teams are parts of a warp, a warp or a block, so that a thread has one to four
// 16-byte vectors of each tensor; without 16-byte alignment (32 for the weights of bf16 inputs)
// a thread's columns are dealt in turn.
// Measured, bf16, inputs not in L2: gated 8192 x 4096 in one group 35 us (5.7 TB/s), 8192 x 16 groups of 128 21 us
// (4.8), its gradients 39 us and 6 for their sums (4.3 TB/s: issue slots, 69% busy); sandwich 8192 x 4096 without a gate
// 47 us (5.7 TB/s), 8192 x 2048 with one 32 us (5.2), its gradients 72 us and 10 (3.7 TB/s: the registers, which
// leave 16 warps an SM).
#include <initializer_list>

#include "kda_block.cuh"

namespace kda {
namespace {

using bf16 = __nv_bfloat16;

// Sums of N values over a team's TS threads, in all of them.  A block's sums go through one of
// two buffers in turn: a buffer is written again one barrier after its last read.
struct TeamBuf {
    float v[2][3][32];
};
template <int TS, int N>
__device__ __forceinline__ void team_sum(float (&x)[N], TeamBuf &buf, int &turn) {
    constexpr int W = TS < 32 ? TS : 32;
#pragma unroll
    for (int o = W / 2; o > 0; o >>= 1)
#pragma unroll
        for (int n = 0; n < N; ++n) x[n] += __shfl_xor_sync(0xffffffffu, x[n], o);
    if constexpr (TS > 32) {
        const int warp = threadIdx.x >> 5;
        if ((threadIdx.x & 31) == 0)
#pragma unroll
            for (int n = 0; n < N; ++n) buf.v[turn][n][warp] = x[n];
        __syncthreads();
#pragma unroll
        for (int n = 0; n < N; ++n) {
            float s = 0.f;
#pragma unroll
            for (int w = 0; w < TS / 32; ++w) s += buf.v[turn][n][w];
            x[n] = s;
        }
        turn ^= 1;
    }
}

// What a thread has of a row: NV vectors of VEC elements, as pairs of fp32 (the packed operations take
// half the issue slots).
template <int VEC, int NV>
struct Pairs {
    static constexpr int N = VEC * NV / 2;
    uint64_t v[N];
};
// The row as it lies in memory, to be widened where it is used: loaded a row ahead.
template <typename T, int VEC, int NV>
struct Raw {
    uint4 v[VEC == 1 ? 1 : NV];
    T e[VEC == 1 ? NV : 1];
};
// Vector k of a thread begins at column (k TS + t) VEC; zeros where the thread has none.
template <int TS, typename T, int VEC, int NV>
__device__ __forceinline__ void get(const T *p, int t, int n, bool in, Raw<T, VEC, NV> &r) {
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int c = (k * TS + t) * VEC;
        if constexpr (VEC == 1)
            r.e[k] = in && c < n ? p[c] : from_f32<T>(0.f);
        else
            r.v[k] = in && c < n ? *reinterpret_cast<const uint4 *>(p + c) : make_uint4(0u, 0u, 0u, 0u);
    }
}
template <typename T, int VEC, int NV>
__device__ __forceinline__ void widen(const Raw<T, VEC, NV> &r, Pairs<VEC, NV> &x) {
    if constexpr (VEC == 1) {
#pragma unroll
        for (int k = 0; k < NV; k += 2) x.v[k / 2] = pack2(to_f32(r.e[k]), to_f32(r.e[k + 1]));
    } else {
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const uint32_t w[4] = {r.v[k].x, r.v[k].y, r.v[k].z, r.v[k].w};
            if constexpr (VEC == 8) {
#pragma unroll
                for (int j = 0; j < 4; ++j) x.v[k * 4 + j] = pack2(w[j] << 16, w[j] & 0xffff0000u);
            } else {
                x.v[k * 2] = pack2(w[0], w[1]);
                x.v[k * 2 + 1] = pack2(w[2], w[3]);
            }
        }
    }
}
template <int TS, typename T, int VEC, int NV>
__device__ __forceinline__ void put(T *p, int t, int n, bool in, const Pairs<VEC, NV> &x) {
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int c = (k * TS + t) * VEC;
        if (!in || c >= n) continue;
        if constexpr (VEC == 1) {
            p[c] = from_f32<T>(__uint_as_float((uint32_t)(x.v[k / 2] >> (k & 1 ? 32 : 0))));
        } else {
            float f[VEC];
#pragma unroll
            for (int j = 0; j < VEC / 2; ++j) unpack2(x.v[k * VEC / 2 + j], f[2 * j], f[2 * j + 1]);
            store_vec<T, VEC, true>(p + c, VEC, f);
        }
    }
}
// The weights of the thread's columns; all ones for a null pointer.
template <int TS, int VEC, int NV>
__device__ __forceinline__ void weights(const float *w, int t, int n, Pairs<VEC, NV> &x) {
    if (!w) {
#pragma unroll
        for (int e = 0; e < Pairs<VEC, NV>::N; ++e) x.v[e] = pack2(1.f, 1.f);
    } else if constexpr (VEC == 1) {
#pragma unroll
        for (int k = 0; k < NV; k += 2) {
            const int c = k * TS + t;
            x.v[k / 2] = pack2(c < n ? w[c] : 0.f, c + TS < n ? w[c + TS] : 0.f);
        }
    } else {
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int c = (k * TS + t) * VEC;
            uint64_t *to = x.v + k * VEC / 2;
#pragma unroll
            for (int j = 0; j < VEC / 2; ++j) to[j] = 0;
            if (c >= n) continue;
            if constexpr (VEC == 8) {
                // one load: two of 16 bytes would each touch every line of the warp's columns, which took 84% of
                // the L1's cycles (the sandwich norm of 8192 x 4096: 72 us so, 52 us now)
                asm("ld.global.v4.b64 {%0,%1,%2,%3}, [%4];"
                    : "=l"(to[0]), "=l"(to[1]), "=l"(to[2]), "=l"(to[3])
                    : "l"(w + c));
            } else {
                const ulonglong2 f = *reinterpret_cast<const ulonglong2 *>(w + c);
                to[0] = f.x;
                to[1] = f.y;
            }
        }
    }
}
__device__ __forceinline__ uint64_t both(float x) { return pack2(x, x); }
__device__ __forceinline__ float sum_of(uint64_t x) {
    float a, b;
    unpack2(x, a, b);
    return a + b;
}

// exp(x) for a gate: of fp32 tensors the exact one (two steps of 2^-23; the division behind it, two more, is the
// fast one, since the exact one took 4 to 8% of the kernels' time).  bf16 outputs are rounded to 2^-8 and
// take the fast one, off by its exponent's rounding, (2 + 1.2 |x|) 2^-24: 2^-19 at |x| = 20, 2^-17 at 80.
template <typename T>
__device__ __forceinline__ float gate_exp(float x) {
    if constexpr (sizeof(T) == 2)
        return __expf(x);
    else
        return expf(x);
}
// The activated gate.  (A sigmoid below 2^-126, z < -87.3, comes out as 0.)
template <typename T>
__device__ __forceinline__ uint64_t gate_of(uint64_t z, int act) {
    float a, b;
    unpack2(z, a, b);
    const uint64_t s = pack2(__fdividef(1.f, 1.f + gate_exp<T>(-a)), __fdividef(1.f, 1.f + gate_exp<T>(-b)));
    return act == KDA_GATE_SILU ? mul2(z, s) : s;
}
// m = sigmoid(-|z|), the smaller one of sigmoid(z) and 1 - sigmoid(z), from which the gradients form both: the
// derivative m (1 - m) keeps its digits where the sigmoid is next to 1, while s (1 - s) of a rounded s is off by
// 1% at z = 12 and 0 from z = 17 on.
template <typename T>
__device__ __forceinline__ uint64_t small_of(uint64_t z) {
    float a, b;
    unpack2(z, a, b);
    const float u = gate_exp<T>(-fabsf(a)), v = gate_exp<T>(-fabsf(b));
    return pack2(__fdividef(u, 1.f + u), __fdividef(v, 1.f + v));
}
__device__ __forceinline__ uint64_t sigmoid_from(uint64_t z, uint64_t m) {  // m or 1 - m
    float a, b, u, v;
    unpack2(z, a, b);
    unpack2(m, u, v);
    return pack2(fabsf((a < 0.f ? 0.f : 1.f) - u), fabsf((b < 0.f ? 0.f : 1.f) - v));
}
__device__ __forceinline__ uint64_t gate_from(uint64_t z, uint64_t m, int act) {
    const uint64_t s = sigmoid_from(z, m);
    return act == KDA_GATE_SILU ? mul2(z, s) : s;
}
__device__ __forceinline__ uint64_t dgate_from(uint64_t z, uint64_t m, int act) {
    const uint64_t d = fma2(mul2(m, both(-1.f)), m, m);  // m (1 - m)
    return act == KDA_GATE_SILU ? fma2(z, d, sigmoid_from(z, m)) : d;
}

constexpr int kTeamThreads = 256;  // of a block of teams of a warp or less
__host__ __device__ constexpr int block_threads(int ts) { return ts <= 32 ? kTeamThreads : ts; }
__host__ __device__ constexpr int block_teams(int ts) { return block_threads(ts) / ts; }
// Blocks of a forward kernel on an SM, by what a thread has of a tensor's row: `count` elements of `size`
// bytes.  They stay and walk the rows, the next row's loads ahead.  Measured with the 16 columns that a
// thread has of 8192 rows of 4096 in bf16: 768 threads an SM 52 us (sandwich) and 38 us (gated), 512
// (no spills) 60 and 42; 8 columns and 1024 threads 62 and 45; 32 columns and 512 threads 50 and 37, but with a
// gate 45 us where 16 columns take 35 (sandwich, 2048 columns).  Blocks of 512 threads (groups of 4097 to 8192
// columns in bf16) do not add up to 768: there is one of them on an SM.
__host__ __device__ constexpr int fwd_blocks(int ts, int count, int size) {
    const int threads = count <= 8 && count * size <= 16 ? 1024 : count * size <= 32 ? 768 : 512;
    return threads / block_threads(ts) > 0 ? threads / block_threads(ts) : 1;
}
template <typename T, typename U>
dim3 fwd_grid(int64_t units) {
    const int64_t blocks = (units + block_teams(U::ts) - 1) / block_teams(U::ts);
    const int64_t most = (int64_t)kSms * fwd_blocks(U::ts, U::vec * U::nv, sizeof(T));
    return dim3((unsigned)(blocks < most ? blocks : most));
}
// Of a backward kernel: 512 threads, which leaves 128 registers each.
__host__ __device__ constexpr int bwd_blocks(int ts) { return 512 / block_threads(ts) > 0 ? 512 / block_threads(ts) : 1; }

// ------------------------------------------------------------------ gated norm
template <typename T, int VEC, int NV, int TS>
__global__ void __launch_bounds__(block_threads(TS), fwd_blocks(TS, VEC * NV, sizeof(T)))
    gated_fwd_kernel(GatedNormArgs p) {
    using P = Pairs<VEC, NV>;
    __shared__ TeamBuf buf;
    int turn = 0;
    constexpr int TPB = block_teams(TS);
    const int t = threadIdx.x % TS, team = threadIdx.x / TS, n = p.group;
    const int64_t units = p.rows * p.parts;
    Raw<T, VEC, NV> xr, zr;
    int64_t at = 0;  // of the unit asked for last: its output
    int g0 = 0;
    auto fetch = [&](int64_t unit) {
        const bool live = unit < units;
        const uint32_t u = live ? (uint32_t)unit : 0u;  // units are counted in 31 bits
        const int64_t row = u / (uint32_t)p.parts;
        g0 = (int)(u % (uint32_t)p.parts) * n;
        at = row * ((int64_t)p.parts * n) + g0;
        get<TS>(static_cast<const T *>(p.x) + row * p.x_stride + g0, t, n, live, xr);
        get<TS>(static_cast<const T *>(p.z) + row * p.z_stride + g0, t, n, live, zr);
    };
    fetch((int64_t)blockIdx.x * TPB + team);
    for (int64_t u0 = (int64_t)blockIdx.x * TPB; u0 < units; u0 += (int64_t)gridDim.x * TPB) {
        const int64_t to = at;
        const float *wp = p.w + (p.shared ? 0 : g0);
        P x, a, w;
        widen(xr, x);
        widen(zr, a);
        fetch(u0 + team + (int64_t)gridDim.x * TPB);
        uint64_t ss = 0;
#pragma unroll
        for (int e = 0; e < P::N; ++e) {
            a.v[e] = gate_of<T>(a.v[e], p.act);
            if (p.first) x.v[e] = mul2(x.v[e], a.v[e]);
            ss = fma2(x.v[e], x.v[e], ss);  // (columns past the group are zeros, whatever the gate)
        }
        float s[1] = {sum_of(ss)};
        team_sum<TS>(s, buf, turn);
        const uint64_t r = both(1.f / sqrtf(s[0] / n + p.eps));
        weights<TS>(wp, t, n, w);
#pragma unroll
        for (int e = 0; e < P::N; ++e) {
            x.v[e] = mul2(mul2(x.v[e], r), w.v[e]);
            if (!p.first) x.v[e] = mul2(x.v[e], a.v[e]);
        }
        put<TS>(static_cast<T *>(p.y) + to, t, n, u0 + team < units, x);
    }
}

// Sums of a block's teams for its columns, in the teams' order, into part.
template <int TS, int VEC, int NV>
__device__ __forceinline__ void teams_store(const Pairs<VEC, NV> &acc, float *part, int n) {
    auto column = [](int e) {  // of value e of a thread, less VEC times its place in the team
        return VEC == 1 ? e * TS : e / VEC * TS * VEC + e % VEC;
    };
    if constexpr (block_teams(TS) == 1) {
#pragma unroll
        for (int e = 0; e < VEC * NV; ++e) {
            const int c = column(e) + (int)threadIdx.x * VEC;
            if (c < n) part[c] = __uint_as_float((uint32_t)(acc.v[e / 2] >> (e & 1 ? 32 : 0)));
        }
    } else {
        __shared__ float sums[block_teams(TS)][TS * NV * VEC];
#pragma unroll
        for (int e = 0; e < VEC * NV; ++e)
            sums[threadIdx.x / TS][column(e) + (int)threadIdx.x % TS * VEC] =
                __uint_as_float((uint32_t)(acc.v[e / 2] >> (e & 1 ? 32 : 0)));
        __syncthreads();
        for (int c = threadIdx.x; c < n; c += block_threads(TS)) {
            float s = 0.f;
#pragma unroll
            for (int m = 0; m < block_teams(TS); ++m) s += sums[m][c];
            part[c] = s;
        }
    }
}

// A block stays with one group of columns unless they share their weights, and walks the rows; its sums per
// column stay in registers.
template <typename T, int VEC, int NV, int TS>
__global__ void __launch_bounds__(block_threads(TS), bwd_blocks(TS))
    gated_bwd_kernel(GatedNormArgs p) {
    using P = Pairs<VEC, NV>;
    __shared__ TeamBuf buf;
    int turn = 0;
    constexpr int TPB = block_teams(TS);
    const int t = threadIdx.x % TS, team = threadIdx.x / TS, n = p.group;
    const int64_t out_stride = (int64_t)p.parts * n;
    // units of this block: (row, group) in order where the weights are shared, rows else
    const int64_t units = p.shared ? p.rows * p.parts : p.rows;
    const int64_t blocks = p.shared ? gridDim.x : gridDim.x / p.parts;
    const int64_t b = p.shared ? blockIdx.x : blockIdx.x / p.parts;
    const int own = p.shared ? 0 : (int)(blockIdx.x % p.parts) * n;
    P dw = {}, w;
    weights<TS>(p.w + own, t, n, w);
    Raw<T, VEC, NV> xr, zr, dr;
    auto fetch = [&](int64_t unit) {
        const bool live = unit < units;
        const int64_t row = !live ? 0 : p.shared ? (uint32_t)unit / (uint32_t)p.parts : unit;
        const int g0 = !live ? 0 : p.shared ? (int)((uint32_t)unit % (uint32_t)p.parts) * n : own;
        get<TS>(static_cast<const T *>(p.x) + row * p.x_stride + g0, t, n, live, xr);
        get<TS>(static_cast<const T *>(p.z) + row * p.z_stride + g0, t, n, live, zr);
        get<TS>(static_cast<const T *>(p.dy) + row * out_stride + g0, t, n, live, dr);
    };
    fetch(b * TPB + team);
    for (int64_t u0 = b * TPB; u0 < units; u0 += blocks * TPB) {
        const int64_t unit = u0 + team;
        const bool live = unit < units;
        const int64_t row = !live ? 0 : p.shared ? (uint32_t)unit / (uint32_t)p.parts : unit;
        const int g0 = !live ? 0 : p.shared ? (int)((uint32_t)unit % (uint32_t)p.parts) * n : own;
        // sigmoid(-|z|) for the second round: formed again in blocks of 1024 threads, whose 64 registers a thread
        // would spill it (4096 x 16384: bf16 495 us kept and 332 formed again, fp32 870 and 668), but for fp32 with
        // scalar accesses, where the exponential's registers spill in its place (2048 x 16382: 659 and 1073)
        constexpr bool keep = TS < 1024 || (VEC == 1 && sizeof(T) == 4);
        P x, z, sg, d;
        widen(xr, x);
        widen(zr, z);
        widen(dr, d);
        fetch(unit + blocks * TPB);
        uint64_t vv = 0, ev = 0;
#pragma unroll
        for (int e = 0; e < P::N; ++e) {
            if (keep) sg.v[e] = small_of<T>(z.v[e]);
            const uint64_t a = keep ? gate_from(z.v[e], sg.v[e], p.act) : gate_of<T>(z.v[e], p.act);
            const uint64_t v = p.first ? mul2(x.v[e], a) : x.v[e];  // what is normalised
            uint64_t g = mul2(d.v[e], w.v[e]);                      // dL/d(rms(v))
            if (!p.first) g = mul2(g, a);
            vv = fma2(v, v, vv);
            ev = fma2(g, v, ev);
        }
        float s[2] = {sum_of(vv), sum_of(ev)};
        team_sum<TS>(s, buf, turn);
        // (0 for a team without a row: with eps = 0 its zeros would give the sums NaN)
        const float rs = live ? 1.f / sqrtf(s[0] / n + p.eps) : 0.f;
        const uint64_t r = both(rs), m = both(-(s[1] / n * rs * rs * rs));
#pragma unroll
        for (int e = 0; e < P::N; ++e) {
            const uint64_t sm = keep ? sg.v[e] : small_of<T>(z.v[e]);
            const uint64_t a = gate_from(z.v[e], sm, p.act), da = dgate_from(z.v[e], sm, p.act);
            const uint64_t gw = mul2(d.v[e], w.v[e]), xv = x.v[e];
            if (p.first) {
                const uint64_t v = mul2(xv, a), dt = fma2(v, m, mul2(r, gw));
                dw.v[e] = fma2(d.v[e], mul2(v, r), dw.v[e]);
                x.v[e] = mul2(dt, a);
                z.v[e] = mul2(mul2(dt, xv), da);
            } else {
                const uint64_t xh = mul2(xv, r);
                dw.v[e] = fma2(mul2(d.v[e], xh), a, dw.v[e]);
                x.v[e] = fma2(xv, m, mul2(mul2(r, gw), a));
                z.v[e] = mul2(mul2(gw, xh), da);
            }
        }
        put<TS>(static_cast<T *>(p.dx) + row * out_stride + g0, t, n, live, x);
        put<TS>(static_cast<T *>(p.dz) + row * out_stride + g0, t, n, live, z);
    }
    teams_store<TS>(dw, p.part + (int64_t)blockIdx.x * n, n);
}

// ------------------------------------------------------------------ sandwich norm
template <typename T, int VEC, int NV, int TS, bool GATED>
__global__ void __launch_bounds__(block_threads(TS), fwd_blocks(TS, VEC * NV, sizeof(T)))
    sandwich_fwd_kernel(SandwichArgs p) {
    using P = Pairs<VEC, NV>;
    __shared__ TeamBuf buf;
    int turn = 0;
    constexpr int TPB = block_teams(TS);
    const int t = threadIdx.x % TS, team = threadIdx.x / TS, n = p.cols;
    Raw<T, VEC, NV> xr, hr, zr;
    auto fetch = [&](int64_t row) {
        const bool live = row < p.rows;
        const int64_t at = live ? row * n : 0;
        get<TS>(static_cast<const T *>(p.x) + at, t, n, live, xr);
        get<TS>(static_cast<const T *>(p.res) + at, t, n, live, hr);
        if (GATED) get<TS>(static_cast<const T *>(p.z) + at, t, n, live, zr);
    };
    fetch((int64_t)blockIdx.x * TPB + team);
    for (int64_t r0 = (int64_t)blockIdx.x * TPB; r0 < p.rows; r0 += (int64_t)gridDim.x * TPB) {
        const bool live = r0 + team < p.rows;
        const int64_t at = (live ? r0 + team : 0) * n;
        P x, h, z, w;
        widen(xr, x);
        widen(hr, h);
        if (GATED) widen(zr, z);
        fetch(r0 + team + (int64_t)gridDim.x * TPB);
        uint64_t ss = 0;
#pragma unroll
        for (int e = 0; e < P::N; ++e) ss = fma2(x.v[e], x.v[e], ss);
        float s[1] = {sum_of(ss)};
        team_sum<TS>(s, buf, turn);
        const uint64_t r = both(1.f / sqrtf(s[0] / n + p.eps));
        weights<TS>(p.w_post, t, n, w);
#pragma unroll
        for (int e = 0; e < P::N; ++e) {
            x.v[e] = mul2(mul2(x.v[e], r), w.v[e]);
            if (GATED) x.v[e] = mul2(x.v[e], gate_of<T>(z.v[e], p.act));
        }
        weights<TS>(p.rs, t, n, w);
        ss = 0;
#pragma unroll
        for (int e = 0; e < P::N; ++e) {
            h.v[e] = fma2(h.v[e], w.v[e], x.v[e]);
            ss = fma2(h.v[e], h.v[e], ss);
        }
        put<TS>(static_cast<T *>(p.h) + at, t, n, live, h);
        s[0] = sum_of(ss);
        team_sum<TS>(s, buf, turn);
        const uint64_t rh = both(1.f / sqrtf(s[0] / n + p.eps));
        weights<TS>(p.w_pre, t, n, w);
#pragma unroll
        for (int e = 0; e < P::N; ++e) h.v[e] = mul2(mul2(h.v[e], rh), w.v[e]);
        put<TS>(static_cast<T *>(p.y) + at, t, n, live, h);
    }
}

template <typename T, int VEC, int NV, int TS, bool GATED>
__global__ void __launch_bounds__(block_threads(TS), bwd_blocks(TS))
    sandwich_bwd_kernel(SandwichArgs p) {
    using P = Pairs<VEC, NV>;
    __shared__ TeamBuf buf;
    int turn = 0;
    constexpr int TPB = block_teams(TS);
    const int t = threadIdx.x % TS, team = threadIdx.x / TS, n = p.cols;
    P dpost = {}, dpre = {}, drs = {};
    Raw<T, VEC, NV> xr, rr, zr, yr, hr;
    auto fetch = [&](int64_t row) {
        const bool live = row < p.rows;
        const int64_t at = live ? row * n : 0;
        get<TS>(static_cast<const T *>(p.x) + at, t, n, live, xr);
        get<TS>(static_cast<const T *>(p.res) + at, t, n, live, rr);
        if (GATED) get<TS>(static_cast<const T *>(p.z) + at, t, n, live, zr);
        get<TS>(static_cast<const T *>(p.dy) + at, t, n, live, yr);
        get<TS>(static_cast<const T *>(p.dh) + at, t, n, live && p.dh, hr);
    };
    fetch((int64_t)blockIdx.x * TPB + team);
    for (int64_t r0 = (int64_t)blockIdx.x * TPB; r0 < p.rows; r0 += (int64_t)gridDim.x * TPB) {
        const bool live = r0 + team < p.rows;
        const int64_t at = (live ? r0 + team : 0) * n;
        P x, res, z, dy, dh, h, w, f;
        weights<TS>(p.w_post, t, n, w);
        weights<TS>(p.rs, t, n, f);
        widen(xr, x);
        widen(rr, res);
        if (GATED) widen(zr, z);
        widen(yr, dy);
        widen(hr, dh);
        uint64_t ss = 0, hh = 0, th = 0;
#pragma unroll
        for (int e = 0; e < P::N; ++e) ss = fma2(x.v[e], x.v[e], ss);
        float s[1] = {sum_of(ss)};
        team_sum<TS>(s, buf, turn);
        const float rx = live ? 1.f / sqrtf(s[0] / n + p.eps) : 0.f;  // (as in the gated norm)
        const uint64_t r = both(rx);
        // h again, and what its norm's gradient needs
#pragma unroll
        for (int e = 0; e < P::N; ++e) {
            uint64_t b = mul2(mul2(x.v[e], r), w.v[e]);
            if (GATED) b = mul2(b, gate_of<T>(z.v[e], p.act));
            h.v[e] = fma2(res.v[e], f.v[e], b);
            hh = fma2(h.v[e], h.v[e], hh);
        }
        P wp;
        weights<TS>(p.w_pre, t, n, wp);
#pragma unroll
        for (int e = 0; e < P::N; ++e) th = fma2(mul2(dy.v[e], wp.v[e]), h.v[e], th);
        float two[2] = {sum_of(hh), sum_of(th)};
        fetch(r0 + team + (int64_t)gridDim.x * TPB);  // (asked for ahead of the first sum: 8 us more of 72)
        team_sum<TS>(two, buf, turn);
        const float rhf = live ? 1.f / sqrtf(two[0] / n + p.eps) : 0.f;
        const uint64_t rh = both(rhf), m = both(-(two[1] / n * rhf * rhf * rhf));
        ss = 0;
#pragma unroll
        for (int e = 0; e < P::N; ++e) {
            dpre.v[e] = fma2(dy.v[e], mul2(h.v[e], rh), dpre.v[e]);
            const uint64_t xh = mul2(x.v[e], r);
            const uint64_t g = fma2(h.v[e], m, fma2(rh, mul2(dy.v[e], wp.v[e]), dh.v[e]));  // dL/dh
            drs.v[e] = fma2(g, res.v[e], drs.v[e]);
            res.v[e] = mul2(g, f.v[e]);
            uint64_t ga = g;
            if (GATED) {
                const uint64_t sm = small_of<T>(z.v[e]);
                ga = mul2(g, gate_from(z.v[e], sm, p.act));
                z.v[e] = mul2(mul2(mul2(g, w.v[e]), xh), dgate_from(z.v[e], sm, p.act));
            }
            dpost.v[e] = fma2(ga, xh, dpost.v[e]);
            dy.v[e] = mul2(ga, w.v[e]);  // dL/d(rms(x))
            ss = fma2(dy.v[e], x.v[e], ss);
        }
        put<TS>(static_cast<T *>(p.dres) + at, t, n, live, res);
        if (GATED) put<TS>(static_cast<T *>(p.dz) + at, t, n, live, z);
        s[0] = sum_of(ss);
        team_sum<TS>(s, buf, turn);
        const uint64_t mx = both(-(s[0] / n * rx * rx * rx));
#pragma unroll
        for (int e = 0; e < P::N; ++e) x.v[e] = fma2(x.v[e], mx, mul2(r, dy.v[e]));
        put<TS>(static_cast<T *>(p.dx) + at, t, n, live, x);
    }
    float *part = p.part + (int64_t)blockIdx.x * n;
    const int64_t plane = (int64_t)gridDim.x * n;
    teams_store<TS>(dpost, part, n);
    if constexpr (TPB > 1) __syncthreads();
    teams_store<TS>(dpre, part + plane, n);
    if constexpr (TPB > 1) __syncthreads();
    if (p.drs) teams_store<TS>(drs, part + 2 * plane, n);
}

// to[c] = the sum over the parts' rows, in a fixed order: 32 warps take every 32nd row each.
__global__ void __launch_bounds__(1024) part_sum_kernel(const float *part, int64_t parts, int n, float *to0, float *to1,
                                                        float *to2) {
    __shared__ float sums[32][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
    part += blockIdx.y * parts * n;
    float s[4] = {};
    if (c < n) {
        int64_t r = warp;
        for (; r + 96 < parts; r += 128)
#pragma unroll
            for (int k = 0; k < 4; ++k) s[k] += part[(r + 32 * k) * n + c];
        for (; r < parts; r += 32) s[0] += part[r * n + c];
    }
    sums[warp][lane] = (s[0] + s[1]) + (s[2] + s[3]);
    __syncthreads();
    if (warp == 0 && c < n) {
        float x = 0.f;
#pragma unroll
        for (int w = 0; w < 32; ++w) x += sums[w][lane];
        (blockIdx.y == 0 ? to0 : blockIdx.y == 1 ? to1 : to2)[c] = x;
    }
}

// Which variant takes a group of n columns: the first of the type's list that holds it.
template <int V, int N, int S>
struct Team {
    static constexpr int vec = V, nv = N, ts = S;
};
template <typename F>
cudaError_t first_of(int, F &&) {
    return cudaErrorInvalidValue;
}
template <typename F, typename Head, typename... Tail>
cudaError_t first_of(int n, F &&f, Head head, Tail... tail) {
    return Head::vec * Head::nv * Head::ts >= n ? f(head) : first_of(n, f, tail...);
}
// Forward: 16 columns per thread past 64 (see fwd_blocks; groups of 128 of 8192 x 2048, inputs in L2: 18.6 us so, 20.3
// with eight each).
template <typename T, typename F>
cudaError_t with_fwd_team(int n, bool vec, F &&f) {
    if (!vec)
        return first_of(n, f, Team<1, 4, 32>(), Team<1, 8, 32>(), Team<1, 8, 128>(), Team<1, 8, 512>(),
                        Team<1, 8, 1024>(), Team<1, 16, 1024>());
    if constexpr (sizeof(T) == 2)
        return first_of(n, f, Team<8, 1, 8>(), Team<8, 2, 8>(), Team<8, 2, 16>(), Team<8, 2, 32>(), Team<8, 2, 64>(),
                        Team<8, 2, 128>(), Team<8, 2, 256>(), Team<8, 2, 512>(), Team<8, 2, 1024>());
    else
        return first_of(n, f, Team<4, 1, 16>(), Team<4, 1, 32>(), Team<4, 2, 32>(), Team<4, 4, 32>(), Team<4, 4, 64>(),
                        Team<4, 4, 128>(), Team<4, 4, 256>(), Team<4, 4, 512>(), Team<4, 4, 1024>());
}
// Backward: more threads rather than more registers, eight columns each: the gradients keep up to nine
// values per column.
template <typename T, typename F>
cudaError_t with_team(int n, bool vec, F &&f) {
    if (!vec)
        return first_of(n, f, Team<1, 4, 32>(), Team<1, 8, 32>(), Team<1, 8, 128>(), Team<1, 8, 512>(),
                        Team<1, 8, 1024>(), Team<1, 16, 1024>());
    if constexpr (sizeof(T) == 2)
        return first_of(n, f, Team<8, 1, 8>(), Team<8, 1, 16>(), Team<8, 1, 32>(), Team<8, 1, 128>(),
                        Team<8, 1, 256>(), Team<8, 1, 512>(), Team<8, 1, 1024>(), Team<8, 2, 1024>());
    else
        return first_of(n, f, Team<4, 1, 16>(), Team<4, 1, 32>(), Team<4, 2, 32>(), Team<4, 2, 128>(),
                        Team<4, 2, 256>(), Team<4, 2, 512>(), Team<4, 2, 1024>(), Team<4, 4, 1024>());
}

bool all_at(size_t bytes, std::initializer_list<const void *> ps) {
    for (const void *q : ps)
        if (!aligned_to(q, bytes)) return false;
    return true;
}

// A backward kernel's blocks: what runs at once where a block has 256 threads or less (twice as many, for
// half the rows each: 88 us for 84 of the sandwich's gradients at 8192 x 2048, and twice the sums to add up).
constexpr int kBwdBlocks = 2 * kSms;

template <typename T>
cudaError_t gated(const GatedNormArgs &a, bool bwd, cudaStream_t st) {
    const int64_t units = a.rows * a.parts;
    constexpr int per = 16 / sizeof(T);
    const bool vec = a.group % per == 0 && a.x_stride % per == 0 && a.z_stride % per == 0 &&
                     all_at(16, {a.x, a.z, a.y, a.dy, a.dx, a.dz}) && all_at(4 * per, {a.w});
    if (!bwd) {
        if (units == 0) return cudaSuccess;
        return with_fwd_team<T>(a.group, vec, [&](auto t) {
            using U = decltype(t);
            return run("gated_fwd", gated_fwd_kernel<T, U::vec, U::nv, U::ts>, fwd_grid<T, U>(units),
                       block_threads(U::ts), 0, st, a);
        });
    }
    const int64_t rows = gated_bwd_rows(a.rows, a.parts, a.shared);
    const int n = a.shared ? a.group : a.group * a.parts;
    cudaError_t e = cudaSuccess;
    if (rows > 0)
        e = with_team<T>(a.group, vec, [&](auto t) {
            using U = decltype(t);
            return run("gated_bwd", gated_bwd_kernel<T, U::vec, U::nv, U::ts>,
                       dim3((unsigned)(a.shared ? rows : rows * a.parts)), block_threads(U::ts), 0, st, a);
        });
    if (e == cudaSuccess)
        e = run("part_sum", part_sum_kernel, dim3((unsigned)((n + 31) / 32)), 1024, 0, st, (const float *)a.part, rows, n,
                a.dw, a.dw, a.dw);
    return e;
}

template <typename T>
cudaError_t sandwich(const SandwichArgs &a, bool bwd, cudaStream_t st) {
    constexpr int per = 16 / sizeof(T);
    const bool vec = a.cols % per == 0 && all_at(16, {a.x, a.res, a.z, a.h, a.y, a.dy, a.dh, a.dx, a.dres, a.dz}) &&
                     all_at(4 * per, {a.w_post, a.w_pre, a.rs});
    cudaError_t e = cudaSuccess;
    if (a.rows > 0 && !bwd)
        e = with_fwd_team<T>(a.cols, vec, [&](auto t) {
            using U = decltype(t);
            return run("sandwich_fwd", a.z ? sandwich_fwd_kernel<T, U::vec, U::nv, U::ts, true>
                                           : sandwich_fwd_kernel<T, U::vec, U::nv, U::ts, false>,
                       fwd_grid<T, U>(a.rows), block_threads(U::ts), 0, st, a);
        });
    if (a.rows > 0 && bwd)
        e = with_team<T>(a.cols, vec, [&](auto t) {
            using U = decltype(t);
            return run("sandwich_bwd", a.z ? sandwich_bwd_kernel<T, U::vec, U::nv, U::ts, true>
                                           : sandwich_bwd_kernel<T, U::vec, U::nv, U::ts, false>,
                       dim3((unsigned)sandwich_bwd_rows(a.rows)), block_threads(U::ts), 0, st, a);
        });
    if (!bwd) return e;
    const int64_t blocks = sandwich_bwd_rows(a.rows);
    if (e == cudaSuccess)
        e = run("part_sum", part_sum_kernel, dim3((unsigned)((a.cols + 31) / 32), a.drs ? 3 : 2), 1024, 0, st,
                (const float *)a.part, blocks, a.cols, a.dw_post, a.dw_pre, a.drs);
    return e;
}

}  // namespace

// Rows of partial sums of the weights' gradients (a block has one, or with weights of their own for
// the groups a block per group): whatever the variant, since the workspace is sized without one.
int64_t gated_bwd_rows(int64_t rows, int parts, bool shared) {
    const int64_t most = shared ? kBwdBlocks : kBwdBlocks / parts > 1 ? kBwdBlocks / parts : 1;
    const int64_t units = shared ? rows * parts : rows;
    return units < most ? units : most;
}
int64_t sandwich_bwd_rows(int64_t rows) { return rows < kBwdBlocks ? rows : kBwdBlocks; }

cudaError_t launch_gated_norm(const GatedNormArgs &a, kda_dtype dt, bool bwd, cudaStream_t st) {
    return dt == KDA_DTYPE_BF16 ? gated<bf16>(a, bwd, st) : gated<float>(a, bwd, st);
}
cudaError_t launch_sandwich(const SandwichArgs &a, kda_dtype dt, bool bwd, cudaStream_t st) {
    return dt == KDA_DTYPE_BF16 ? sandwich<bf16>(a, bwd, st) : sandwich<float>(a, bwd, st);
}

}  // namespace kda
