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
// L2).  All arithmetic is fp32, in pairs (the packed operations take two values an issue slot);
// outputs are rounded once.
//
// Measured, GB300, 8192 rows x 6144 channels x 4 taps, bf16: forward 37 us (201 MB, 5.4 TB/s),
// backward 75 us (302 MB, 4.0 TB/s; issue slots 52% busy) and 5 us for the strips' sums.
// Where rows are not aligned for vectors (6145 channels) 59 and 120 us.
#include <type_traits>

#include "kda_block.cuh"

namespace kda {
namespace {

constexpr int kConvThreads = 128;

template <typename T>
__device__ __forceinline__ float sigmoid_of(float x) {
    if constexpr (sizeof(T) == 4) return 1.f / (1.f + expf(-x));
    // the approximate exponential and reciprocal, one special-function operation each: a
    // relative error near 2^-22, far inside a bf16 output's rounding
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + ex2_ftz(-1.4426950408889634f * x)));
    return r;
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

// A thread's four channels.  Vector loads want them adjacent; where rows are not aligned for
// those, they lie 32 apart, so that each scalar load of a warp is still one line.
constexpr int kCh = 4;
struct Four {
    uint64_t p[2];
    __device__ __forceinline__ void zero() { p[0] = p[1] = 0; }
};
__device__ __forceinline__ void fma4(Four &a, const Four &x, const Four &y) {
    a.p[0] = fma2(x.p[0], y.p[0], a.p[0]);
    a.p[1] = fma2(x.p[1], y.p[1], a.p[1]);
}
template <typename T, bool AL>
struct Channels {
    int c, C;
    __device__ __forceinline__ Channels(int block, int C_) : C(C_) {
        const int base = block * kCh * kConvThreads;
        c = AL ? base + (int)threadIdx.x * kCh
               : base + ((int)threadIdx.x >> 5) * 32 * kCh + ((int)threadIdx.x & 31);
    }
    __device__ __forceinline__ int at(int j) const { return AL ? c + j : c + 32 * j; }
    __device__ __forceinline__ bool in(int j) const { return at(j) < C; }
    // f(channel) of each, 0 past the last
    template <typename F>
    __device__ __forceinline__ Four of(F &&f) const {
        float v[kCh];
#pragma unroll
        for (int j = 0; j < kCh; ++j) v[j] = in(j) ? f(at(j)) : 0.f;
        return {{pack2(v[0], v[1]), pack2(v[2], v[3])}};
    }
    // raw: as it lies in memory, converted where it is used
    using Raw = typename std::conditional<sizeof(T) == 4, float4, uint2>::type;
    __device__ __forceinline__ Raw load(const T *row) const {
        Raw r{};
        if constexpr (AL) {
            r = *reinterpret_cast<const Raw *>(row + c);
        } else {
            T *e = reinterpret_cast<T *>(&r);
#pragma unroll
            for (int j = 0; j < kCh; ++j)
                if (in(j)) e[j] = row[at(j)];
        }
        return r;
    }
    // as fp32, in pairs for the packed operations
    static __device__ __forceinline__ void widen(const Raw &r, Four &v) {
        if constexpr (sizeof(T) == 4) {
            v.p[0] = pack2(r.x, r.y);
            v.p[1] = pack2(r.z, r.w);
        } else {
            v.p[0] = pack2(r.x << 16, r.x & 0xffff0000u);
            v.p[1] = pack2(r.y << 16, r.y & 0xffff0000u);
        }
    }
    __device__ __forceinline__ void load(const T *row, Four &v) const { widen(load(row), v); }
    __device__ __forceinline__ void store(T *row, const Four &f) const {
        float v[kCh];
        unpack2(f.p[0], v[0], v[1]);
        unpack2(f.p[1], v[2], v[3]);
        if constexpr (AL) {
            store_vec<T, kCh, true>(row + c, kCh, v);
        } else {
#pragma unroll
            for (int j = 0; j < kCh; ++j)
                if (in(j)) row[at(j)] = from_f32<T>(v[j]);
        }
    }
};

// The sigmoid of four channels.
template <typename T>
__device__ __forceinline__ Four sigmoid4(const Four &a) {
    Four r;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        float x, y;
        unpack2(a.p[h], x, y);
        r.p[h] = pack2(sigmoid_of<T>(x), sigmoid_of<T>(y));
    }
    return r;
}

// The row r of a sequence that starts at s: of x, or of the carried state before it, or zero.
template <typename T, bool AL>
__device__ __forceinline__ void row_or_state(const ConvArgs &p, const Channels<T, AL> &ch, int W, int n,
                                             int64_t s, int64_t r, Four &v) {
    const T *st = static_cast<const T *>(p.state_in);
    v.zero();
    if (r >= s)
        ch.load(static_cast<const T *>(p.x) + r * p.x_stride, v);
    else if (st)
        ch.load(st + ((int64_t)n * (W - 1) + (W - 1) + (r - s)) * p.C, v);
}

__device__ __forceinline__ uint32_t smem_u32(const void *p) { return (uint32_t)__cvta_generic_to_shared(p); }
template <int BYTES>
__device__ __forceinline__ void copy_async(uint32_t to, const void *from) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(to), "l"(from), "n"(BYTES) : "memory");
}

// A thread's rows on their way, U at a time and GROUPS - 1 such groups ahead, R tensors beside
// each other: a ring in shared memory that asynchronous copies fill.  Every thread copies and
// reads its own channels alone, so nothing but its own copies is waited for.  Rows that are
// not aligned for copies of four channels come through registers, one group ahead (fp32,
// 15000 x 1537: 42 us against 57 with copies of 4 bytes; there are none of 2).  Groups, 8192 x
// 6144 bf16: forward 38.4, 36.2 and 37.3 us with 3, 4 and 6; backward 81.7 and 74.2 with 2 and 3.
template <typename T, bool AL, int U, int GROUPS, int R>
struct Ahead {
    static constexpr bool kRing = AL;
    using Ch = Channels<T, AL>;
    using Raw = typename Ch::Raw;
    struct Smem {
        Raw at[kRing ? GROUPS : 1][R][U][kRing ? kConvThreads : 1];
    };
    const Ch &ch;
    Smem &s;
    const T *src[R];        // the next group to fetch
    int64_t stride[R];
    int left, in, out;      // groups to fetch; ring places
    Raw reg[kRing ? 1 : R][kRing ? 1 : U];
    __device__ __forceinline__ Ahead(const Ch &c, Smem &sm) : ch(c), s(sm) {}
    __device__ __forceinline__ void fetch() {
        if (left > 0) {
            --left;
#pragma unroll
            for (int r = 0; r < R; ++r) {
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const T *g = src[r] + u * stride[r];
                    if constexpr (!kRing) {
                        reg[r][u] = ch.load(g);
                    } else {
                        copy_async<sizeof(Raw)>(smem_u32(&s.at[in][r][u][threadIdx.x]), g + ch.c);
                    }
                }
                src[r] += U * stride[r];
            }
        }
        if constexpr (kRing) {
            asm volatile("cp.async.commit_group;" ::: "memory");
            in = in + 1 == GROUPS ? 0 : in + 1;
        }
    }
    // `groups` of U rows from src on; before the first take(), and again once all are taken
    __device__ __forceinline__ void start(int groups) {
        left = groups;
        in = out = 0;  // what was fetched before has been taken
#pragma unroll
        for (int k = 0; k < (kRing ? GROUPS - 1 : 1); ++k) fetch();
    }
    // The next group, as fp32 (tensor r's rows to to(r, u)), and one more fetched: into the
    // place that the group before it was read from.
    template <typename F>
    __device__ __forceinline__ void take(F &&to) {
        if constexpr (kRing) asm volatile("cp.async.wait_group %0;" ::"n"(GROUPS - 2) : "memory");
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if constexpr (kRing) Ch::widen(s.at[out][r][u][threadIdx.x], to(r, u));
                else Ch::widen(reg[r][u], to(r, u));
            }
        if constexpr (kRing) out = out + 1 == GROUPS ? 0 : out + 1;
        fetch();
    }
};

// (Blocks per SM: unaligned bf16, 8192 x 6145, 59 us with six, 86 with what the compiler takes.)
template <typename T, int W, bool AL>
__global__ void __launch_bounds__(kConvThreads, AL || sizeof(T) == 4 ? 0 : 6) conv_fwd_kernel(ConvArgs p) {
    constexpr int U = 4;
    using Ch = Channels<T, AL>;
    using Rows = Ahead<T, AL, U, 4, 1>;
    __shared__ typename Rows::Smem ring;
    const int cblocks = (p.C + kCh * kConvThreads - 1) / (kCh * kConvThreads);
    const int64_t strip = blockIdx.x / cblocks;
    const Ch ch((int)(blockIdx.x % cblocks), p.C);
    if (p.cu && blockIdx.x == 0) check_offsets(p.cu, p.N, p.T, p.status);
    if (!ch.in(0)) return;
    const T *x = static_cast<const T *>(p.x);

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
#pragma unroll
        for (int k = 0; k < W - 1; ++k) {
            Four v;
            row_or_state<T, AL>(p, ch, W, n, s, e - (W - 1) + k, v);
            ch.store(static_cast<T *>(p.state_out) + ((int64_t)n * (W - 1) + k) * p.C, v);
        }
        return;
    }

    Four w[W];
    const Four bias = ch.of([&](int c) { return p.bias ? p.bias[c] : 0.f; });
#pragma unroll
    for (int k = 0; k < W; ++k) w[k] = ch.of([&](int c) { return p.w[(int64_t)c * W + k]; });
    T *y = static_cast<T *>(p.y);
    const int64_t t1 = min((strip + 1) * (int64_t)p.strip, (int64_t)p.B * p.T);
    Rows rows(ch, ring);
    rows.stride[0] = p.x_stride;
    for (int64_t t = strip * p.strip; t < t1;) {
        int n;
        int64_t s, e;
        if (!find_seq(p, t, n, s, e)) return;
        e = min(e, t1);
        int left = (int)(e - t);
        const T *px = x + t * p.x_stride;
        T *py = y + t * p.C;
        rows.src[0] = px;
        rows.start(left / U);
        Four win[W - 1 + U];
#pragma unroll
        for (int k = 0; k < W - 1; ++k) row_or_state<T, AL>(p, ch, W, n, s, t - (W - 1) + k, win[k]);
        auto out = [&](int u, T *row) {  // from rows u .. u + W - 1 of the window
            Four a = bias;
#pragma unroll
            for (int k = 0; k < W; ++k) fma4(a, w[k], win[u + k]);
            if (p.silu) {
                const Four sg = sigmoid4<T>(a);
                a.p[0] = mul2(a.p[0], sg.p[0]);
                a.p[1] = mul2(a.p[1], sg.p[1]);
            }
            ch.store(row, a);
        };
        for (; left >= U; left -= U) {
            rows.take([&](int, int u) -> Four & { return win[W - 1 + u]; });
#pragma unroll
            for (int u = 0; u < U; ++u) out(u, py + (int64_t)u * p.C);
            px += U * p.x_stride;
            py += (int64_t)U * p.C;
#pragma unroll
            for (int k = 0; k < W - 1; ++k) win[k] = win[U + k];
        }
#pragma unroll 1
        for (; left > 0; --left) {
            ch.load(px, win[W - 1]);
            out(0, py);
            px += p.x_stride;
            py += p.C;
#pragma unroll
            for (int k = 0; k < W - 1; ++k) win[k] = win[k + 1];
        }
        t = e;
    }
}

// Gradients.  With dpre_u = dy_u act'(pre_u), dx_t = sum_m w[W-1-m] dpre_{t+m} over the
// rows t + m of t's sequence, plus the final state's gradient for the last W - 1 rows;
// rows before the sequence are the carried state's.  A thread walks "position" t from
// W - 1 rows before its strip to the strip's last row, holding x and dpre of rows
// t .. t + W - 1; the row that enters is u = t + W - 1.  dw and dbias take the rows of
// the strip alone; each strip leaves its sums in p.part and a second kernel adds the
// strips in order, so that no result depends on the order of atomics.  (Blocks per SM: four where
// that leaves registers for all of it; unaligned bf16 would spill: 125 us with three, 185 with four.)
template <typename T, int W, bool AL>
__global__ void __launch_bounds__(kConvThreads, AL && sizeof(T) == 2 ? 4 : 3) conv_bwd_kernel(ConvArgs p) {
    follow();
    constexpr int U = 4;
    using Ch = Channels<T, AL>;
    using Rows = Ahead<T, AL, U, 3, 2>;
    __shared__ typename Rows::Smem ring;
    const int cblocks = (p.C + kCh * kConvThreads - 1) / (kCh * kConvThreads);
    const int64_t strip = blockIdx.x / cblocks;
    const Ch ch((int)(blockIdx.x % cblocks), p.C);
    if (p.cu && blockIdx.x == 0) check_offsets(p.cu, p.N, p.T, p.status);
    if (!ch.in(0)) return;
    const T *x = static_cast<const T *>(p.x), *dy = static_cast<const T *>(p.dy);
    const T *dso = static_cast<const T *>(p.dstate_out);
    T *dx = static_cast<T *>(p.dx), *dsi = static_cast<T *>(p.dstate_in);

    Four w[W], dw[W], db;
    const Four bias = ch.of([&](int c) { return p.bias ? p.bias[c] : 0.f; });
    db.zero();
#pragma unroll
    for (int k = 0; k < W; ++k) {
        w[k] = ch.of([&](int c) { return p.w[(int64_t)c * W + k]; });
        dw[k].zero();
    }
    Rows rows(ch, ring);
    rows.stride[0] = p.x_stride;
    rows.stride[1] = p.C;
    const int64_t t0 = strip * p.strip, t1 = min(t0 + p.strip, (int64_t)p.B * p.T);
    for (int64_t t = t0; t < t1;) {
        int n;
        int64_t s, e;
        if (!find_seq(p, t, n, s, e)) break;
        const int64_t end = min(e, t1);
        // positions whose entering row is the strip's own: from t on
        int left = max((int)(end - (W - 1) - t), 0);
        rows.src[0] = x + (t + W - 1) * p.x_stride;
        rows.src[1] = dy + (t + W - 1) * p.C;
        rows.start(left / U);
        // windows of a group of positions pos .. pos + U - 1: rows pos .. pos + W - 2 + U
        Four xw[W - 1 + U], dp[W - 1 + U];
#pragma unroll
        for (int k = 0; k < W - 1; ++k) {
            row_or_state<T, AL>(p, ch, W, n, s, t - (W - 1) + k, xw[k]);
            dp[k].zero();
        }
        // dp of the entering row at window place q, from dy; and its share of dw, dbias
        auto enter = [&](int q, bool own) {
            if (p.silu) {
                constexpr uint64_t one = 0x3f8000003f800000ull;
                Four a = bias;
#pragma unroll
                for (int k = 0; k < W; ++k) fma4(a, w[k], xw[q - (W - 1) + k]);
                const Four sg = sigmoid4<T>(a);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint64_t f = mul2(sg.p[h], fma2(a.p[h], sub2(one, sg.p[h]), one));
                    dp[q].p[h] = mul2(dp[q].p[h], f);
                }
            }
            if (own) {
                db.p[0] = add2(db.p[0], dp[q].p[0]);
                db.p[1] = add2(db.p[1], dp[q].p[1]);
#pragma unroll
                for (int k = 0; k < W; ++k) fma4(dw[k], dp[q], xw[q - (W - 1) + k]);
            }
        };
        auto leave = [&](int q) {  // dx of window place q
            Four o;
            o.zero();
#pragma unroll
            for (int m = 0; m < W; ++m) fma4(o, w[W - 1 - m], dp[q + m]);
            return o;
        };
        auto move = [&](int by) {
#pragma unroll
            for (int k = 0; k < W - 1; ++k) {
                xw[k] = xw[by + k];
                dp[k] = dp[by + k];
            }
        };
        // one position with every check: the first and last ones, where rows of the state or of
        // the next strip take part
        auto step = [&](int64_t pos) {
            const int64_t u = pos + W - 1;
            xw[W - 1].zero();
            dp[W - 1].zero();
            if (u < e) {  // (a row past the sequence adds nothing whatever sigmoid would give)
                ch.load(x + u * p.x_stride, xw[W - 1]);
                ch.load(dy + u * p.C, dp[W - 1]);
                enter(W - 1, u < end);
            }
            const bool state_row = pos < s;
            if (state_row ? dsi != nullptr && t == s : pos >= t) {
                Four o = leave(0);
                const int64_t k = pos - (e - (W - 1));  // its row of the final state
                if (dso && k >= 0) {
                    Four f;
                    ch.load(dso + ((int64_t)n * (W - 1) + k) * p.C, f);
                    o.p[0] = add2(o.p[0], f.p[0]);
                    o.p[1] = add2(o.p[1], f.p[1]);
                }
                ch.store(state_row ? dsi + ((int64_t)n * (W - 1) + (W - 1) + (pos - s)) * p.C : dx + pos * p.C, o);
            }
            move(1);
        };
        int64_t pos = t - (W - 1);
#pragma unroll 1
        for (; pos < t; ++pos) step(pos);
        T *po = dx + pos * p.C;
        for (; left >= U; left -= U, pos += U) {
            rows.take([&](int r, int u) -> Four & { return r == 0 ? xw[W - 1 + u] : dp[W - 1 + u]; });
#pragma unroll
            for (int i = 0; i < U; ++i) {
                enter(W - 1 + i, true);
                ch.store(po + (int64_t)i * p.C, leave(i));
            }
            po += (int64_t)U * p.C;
            move(U);
        }
#pragma unroll 1
        for (; pos < end; ++pos) step(pos);
        t = end;
    }
    float *part = p.part + strip * (int64_t)(W + 1) * p.C;
    auto leave_sums = [&](float *row, const Four &f) {
        float v[kCh];
        unpack2(f.p[0], v[0], v[1]);
        unpack2(f.p[1], v[2], v[3]);
#pragma unroll
        for (int j = 0; j < kCh; ++j)
            if (ch.in(j)) row[ch.at(j)] = v[j];
    };
#pragma unroll
    for (int k = 0; k < W; ++k) leave_sums(part + (int64_t)k * p.C, dw[k]);
    leave_sums(part + (int64_t)W * p.C, db);
}

// Empty sequences: the carried state passes through, and so does its gradient.
template <typename T>
__global__ void __launch_bounds__(128) conv_bwd_empty_kernel(ConvArgs p) {
    follow();
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
    follow();
    __shared__ float red[8][33];
    const int lane = threadIdx.x & 31, grp = threadIdx.x >> 5;
    const int64_t i = (int64_t)blockIdx.x * 32 + lane, total = (int64_t)(W + 1) * C;
    float s = 0.f;
    if (i < total) {
#pragma unroll 8
        for (int64_t r = grp; r < strips; r += 8) s += part[r * total + i];
    }
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

// One token per row.  A thread takes `per` batch rows, four at a time, so that its channels'
// weights (twice the bytes of a row's state) are read once for all of them: 512 x 6144, 11.4 us
// (25 MB from memory), 27.6 us with one row a thread.
constexpr int kStepRows = 4;
template <typename T, int W, bool AL>
__global__ void __launch_bounds__(kConvThreads) conv_step_kernel(ConvStepArgs p, int per) {
    using Ch = Channels<T, AL>;
    const int cblocks = (p.C + kCh * kConvThreads - 1) / (kCh * kConvThreads);
    const int n0 = (int)(blockIdx.x / cblocks) * per, n1 = min(n0 + per, p.N);
    const Ch ch((int)(blockIdx.x % cblocks), p.C);
    if (blockIdx.x % cblocks == 0)
        for (int n = n0 + threadIdx.x; n < n1; n += kConvThreads)
            if (p.idx && p.idx[n] >= p.slots) report(p.status, KDA_DEVICE_BAD_INDEX);
    if (!ch.in(0)) return;
    Four w[W];
    const Four bias = ch.of([&](int c) { return p.bias ? p.bias[c] : 0.f; });
#pragma unroll
    for (int k = 0; k < W; ++k) w[k] = ch.of([&](int c) { return p.w[(int64_t)c * W + k]; });
    for (int n = n0; n < n1; n += kStepRows) {
        typename Ch::Raw raw[kStepRows][W];
        T *st[kStepRows];
#pragma unroll
        for (int r = 0; r < kStepRows; ++r) {
            st[r] = nullptr;
            if (n + r >= n1) continue;
            const int slot = p.idx ? p.idx[n + r] : n + r;
            if (slot < 0 || slot >= p.slots) continue;  // an unused row, or a reported one
            st[r] = static_cast<T *>(p.state) + (int64_t)slot * (W - 1) * p.C;
#pragma unroll
            for (int k = 0; k < W - 1; ++k) raw[r][k] = ch.load(st[r] + (int64_t)k * p.C);
            raw[r][W - 1] = ch.load(static_cast<const T *>(p.x) + (int64_t)(n + r) * p.x_stride);
        }
#pragma unroll
        for (int r = 0; r < kStepRows; ++r) {
            if (n + r >= n1) break;
            Four o;
            o.zero();
            if (st[r]) {
                Four win[W];
#pragma unroll
                for (int k = 0; k < W; ++k) Ch::widen(raw[r][k], win[k]);
                o = bias;
#pragma unroll
                for (int k = 0; k < W; ++k) fma4(o, w[k], win[k]);
                if (p.silu) {
                    const Four sg = sigmoid4<T>(o);
                    o.p[0] = mul2(o.p[0], sg.p[0]);
                    o.p[1] = mul2(o.p[1], sg.p[1]);
                }
#pragma unroll
                for (int k = 0; k < W - 1; ++k) ch.store(st[r] + (int64_t)k * p.C, win[k + 1]);
            }
            ch.store(static_cast<T *>(p.y) + (int64_t)(n + r) * p.C, o);
        }
    }
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

int strip_for(int64_t rows, int C, int most) {
    const int64_t per_row = (C + kCh - 1) / kCh;
    int strip = most;
    while (strip > 8 && (rows + strip - 1) / strip * per_row < kSms * 1024) strip /= 2;
    return strip;
}

// f(type, taps, aligned)
template <typename F>
cudaError_t by_kind(kda_dtype dt, int W, bool al, F &&f) {
    using std::integral_constant;
    return by_width(W, [&](auto taps) {
        if (dt == KDA_DTYPE_BF16) {
            if (al) f(__nv_bfloat16(), taps, integral_constant<bool, true>());
            else f(__nv_bfloat16(), taps, integral_constant<bool, false>());
        } else {
            if (al) f(float(), taps, integral_constant<bool, true>());
            else f(float(), taps, integral_constant<bool, false>());
        }
    });
}
int64_t channel_blocks(int C) { return (C + kCh * kConvThreads - 1) / (kCh * kConvThreads); }

}  // namespace

// Long strips re-read little (W - 1 rows each) and leave few partial sums; short inputs get
// shorter ones, down to 8 rows, until there are 152 x 1024 threads (2048 channels: at 512 rows
// 4.3 us forward and 10.4 us backward against 7.9 and 22.4 with the longest strips, at 64 rows
// 3.4 and 7.7 against 7.5 and 13.5; at 8192 x 6144 no difference).
int conv_bwd_strip(int B, int T, int C) { return strip_for((int64_t)B * T, C, 128); }

cudaError_t launch_conv_fwd(ConvArgs a, kda_dtype dt, cudaStream_t st) {
    const size_t e = dt == KDA_DTYPE_BF16 ? 2 : 4;
    const void *ptrs[] = {a.x, a.y, a.state_in, a.state_out};
    const bool al = rows_aligned(ptrs, 4, (int64_t)(a.C * e), (int64_t)(a.x_stride * e), kCh * e);
    const int64_t rows = (int64_t)a.B * a.T;
    a.strip = strip_for(rows, a.C, 64);
    a.strips = (rows + a.strip - 1) / a.strip;
    const int64_t blocks = channel_blocks(a.C) * (a.strips + (a.state_out ? a.N : 0));
    if (blocks == 0) return cudaSuccess;
    if (blocks > INT32_MAX) return cudaErrorInvalidValue;
    prof_begin("conv_fwd", st);
    const cudaError_t err = by_kind(dt, a.W, al, [&](auto t, auto W, auto AL) {
        conv_fwd_kernel<decltype(t), W(), AL()><<<(unsigned)blocks, kConvThreads, 0, st>>>(a);
    });
    prof_end(st);
    return err;
}

cudaError_t launch_conv_bwd(ConvArgs a, kda_dtype dt, cudaStream_t st) {
    const size_t e = dt == KDA_DTYPE_BF16 ? 2 : 4;
    const void *ptrs[] = {a.x, a.dy, a.dx, a.state_in, a.dstate_out, a.dstate_in};
    const bool al = rows_aligned(ptrs, 6, (int64_t)(a.C * e), (int64_t)(a.x_stride * e), kCh * e);
    a.strip = conv_bwd_strip(a.B, a.T, a.C);
    const int64_t rows = (int64_t)a.B * a.T;
    a.strips = (rows + a.strip - 1) / a.strip;
    const int64_t blocks = channel_blocks(a.C) * a.strips;
    if (blocks > INT32_MAX) return cudaErrorInvalidValue;
    cudaError_t err = cudaSuccess;
    bool first = blocks == 0;  // no kernel of this call so far
    if (blocks > 0) {
        prof_begin("conv_bwd", st);
        err = by_kind(dt, a.W, al, [&](auto t, auto W, auto AL) {
            conv_bwd_kernel<decltype(t), W(), AL()><<<(unsigned)blocks, kConvThreads, 0, st>>>(a);
        });
        prof_end(st);
        if (err != cudaSuccess) return err;
    }
    if (a.dstate_in && a.N > 0 && (a.cu || a.T == 0)) {
        prof_begin("conv_bwd_empty", st);
        err = dt == KDA_DTYPE_BF16 ? launch_next(first, conv_bwd_empty_kernel<__nv_bfloat16>, a.N, 128, 0, st, a)
                                   : launch_next(first, conv_bwd_empty_kernel<float>, a.N, 128, 0, st, a);
        prof_end(st);
        first = false;
        if (err != cudaSuccess) return err;
    }
    const int64_t total = (int64_t)(a.W + 1) * a.C;
    prof_begin("conv_bwd_sum", st);
    err = launch_next(first, conv_bwd_sum_kernel, (total + 31) / 32, 256, 0, st, a.part, a.strips, a.C, a.W, a.dw,
                      a.dbias);
    prof_end(st);
    return err;
}

cudaError_t launch_conv_step(const ConvStepArgs &a, kda_dtype dt, cudaStream_t st) {
    const size_t e = dt == KDA_DTYPE_BF16 ? 2 : 4;
    const void *ptrs[] = {a.x, a.y, a.state};
    const bool al = rows_aligned(ptrs, 3, (int64_t)(a.C * e), (int64_t)(a.x_stride * e), kCh * e);
    // as many rows per thread as leave 8 blocks for every SM
    const int64_t cb = channel_blocks(a.C), most = (int64_t)a.N * cb / (kSms * 8);
    const int per = most < 1 ? 1 : most > 32 ? 32 : (int)most;
    const int64_t blocks = (a.N + per - 1) / per * cb;
    if (blocks == 0) return cudaSuccess;
    if (blocks > INT32_MAX) return cudaErrorInvalidValue;
    prof_begin("conv_step", st);
    const cudaError_t err = by_kind(dt, a.W, al, [&](auto t, auto W, auto AL) {
        conv_step_kernel<decltype(t), W(), AL()><<<(unsigned)blocks, kConvThreads, 0, st>>>(a, per);
    });
    prof_end(st);
    return err;
}

}  // namespace kda
