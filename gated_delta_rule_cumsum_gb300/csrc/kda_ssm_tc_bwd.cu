// kda_ssm_tc_bwd.cu -- the scan's gradients on the tensor cores: what ssm_chunk_grads_kernel
// (kda_ssm.cu, with the formulas) does per chunk of 128 rows and head, in two kernels, one
// for each side of the chunk's pairs (i, j), because the operand that a product reads from
// tensor memory has to have its rows in the lanes:
//
//   i side (a lane is a row i):  Z = dy x^T;  W = Z e d (hi, lo);  Q = Z G e d
//       dC += W B + (2^{a_i} dy) S^T,   u_i = 2^{a_i} dy_i . (C S)_i,   and the sums of Q
//   j side (a lane is a row j):  Z^T, G^T;  W^T, M^T (hi, lo)
//       dB += W^T C + (w x) E^T,   dx = M^T dy + w (B E) + D dy,   v_j = w_j x_j . (B E)_j
//
// dB and dC are summed over a group's heads in tensor memory: a CTA takes a part of a group's
// units (head, 64 columns) of one chunk, one after another, and leaves one fp32 tile per
// part; a last kernel adds the parts in order.  What the kernels make themselves goes into
// the products in two bf16 parts (2^-17); sums, W's and Q's elements are fp32.  The states S
// and E come in three parts (2^-25) where they make u, v and B E, which the fp32 gradients of
// A_log and dt_bias sum with either sign over all rows: with two parts these were off by 2^-18 of
// the root of the sum of their terms' squares, 5e-5 of a single head's whose sum cancels.  dB
// and dC, bf16, take two of the three.
//
// Measured, GB300, 8192 rows, 32 heads of 64, one group, 128 state rows: i side 77 us, j side
// 103 us.  A unit takes about 8 and 12 thousand cycles, of which
// its products take a third (the tensor pipe is active 28 to 31% of the time): the rest is the chain from products to
// factors and back, in warps that can only read their own quarter of the rows, so that one
// quarter's warps have most of the triangle.  Issuing the next unit's first products ahead of a
// unit's last ones, and the rows' loads earlier, moved the waits and not the sum (within 2%).
#include "kda_ssm_tc.cuh"

namespace kda {
namespace {

using bf16 = __nv_bfloat16;
constexpr int kGThreads = 512, kGAll = kGThreads + 32, kGWarps = kGThreads / 32;

struct GradUnit {
    int h, tile;
    int64_t unit;  // (slot, head, tile)
};
struct GradWork {
    int64_t slot;
    int g, part, first, count, pt, per_group;  // count >= 1: there are no more parts than units
    TcChunk c;
    __device__ __forceinline__ bool start(const SsmArgs &p) {
        pt = tiles_of(p.P);
        per_group = p.H / p.G;
        int64_t id = blockIdx.x;
        part = (int)(id % p.parts);
        id /= p.parts;
        g = (int)(id % p.G);
        slot = id / p.G;
        if (!tc_find_chunk(p, slot, c)) return false;
        const int units = per_group * pt;
        first = (int)((int64_t)units * part / p.parts);
        count = (int)((int64_t)units * (part + 1) / p.parts) - first;
        return true;
    }
    __device__ __forceinline__ GradUnit at(const SsmArgs &p, int it) const {
        GradUnit r;
        const int u = first + it;
        r.h = g * per_group + u / pt;
        r.tile = u % pt;
        r.unit = (slot * p.H + r.h) * pt + r.tile;
        return r;
    }
    __device__ __forceinline__ float *share(const SsmArgs &p, float *base) const {
        return base + ((slot * p.G + g) * p.parts + part) * (int64_t)kTL * p.Ns;
    }
};

// 128 x 64 of bf16 rows by the 512 row threads: pieces of rows r0, r0 + 64 of column c8.
template <bool AL>
__device__ __forceinline__ void load_tile64(uint8_t *tile, const bf16 *src, int64_t stride, int nr, int cols) {
    const int tid = threadIdx.x, c8 = (tid >> 3) & 7, r0 = (tid >> 6) * 8 + (tid & 7);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const int r = r0 + 64 * k;
        uint8_t *dst = tile + (r >> 3) * (kPT * 16) + c8 * 128 + (r & 7) * 16;
        const bool in = r < nr && c8 * 8 < cols;
        const bf16 *s = src + r * stride + c8 * 8;
        if constexpr (AL) {
            cp_async16(tc::smem_addr(dst), in ? s : src, in);
        } else {
            alignas(16) bf16 v[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = in ? s[j] : __float2bfloat16_rn(0.f);
            *reinterpret_cast<uint4 *>(dst) = *reinterpret_cast<const uint4 *>(v);
        }
    }
}
// kTL x COLS (32, 64 or 128) of bf16 rows by the 512 row threads.
template <bool AL, int COLS>
__device__ __forceinline__ void load_wide(uint8_t *tile, const bf16 *src, int64_t stride, int nr, int nc) {
    constexpr int CPR = COLS / 8, IT = kTL * CPR / kGThreads, STEP = kGThreads / CPR;
    const int tid = threadIdx.x, c8 = (tid >> 3) % CPR, r0 = (tid >> 3) / CPR * 8 + (tid & 7);
#pragma unroll
    for (int k = 0; k < IT; ++k) {
        const int r = r0 + k * STEP;
        uint8_t *dst = tile + (r >> 3) * (COLS * 16) + c8 * 128 + (r & 7) * 16;
        const bool in = r < nr && c8 * 8 < nc;
        const bf16 *s = src + r * stride + c8 * 8;
        if constexpr (AL) {
            cp_async16(tc::smem_addr(dst), in ? s : src, in);
        } else {
            alignas(16) bf16 v[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = in && c8 * 8 + j < nc ? s[j] : __float2bfloat16_rn(0.f);
            *reinterpret_cast<uint4 *>(dst) = *reinterpret_cast<const uint4 *>(v);
        }
    }
}

// The sums over a warp's 32 lanes of each of 16 values: lane l ends with that of value l % 16.
__device__ __forceinline__ float lane_sums(float (&v)[16]) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int s = 8; s > 0; s >>= 1) {
        const bool up = lane & s;
#pragma unroll
        for (int k = 0; k < s; ++k) {
            const float give = up ? v[k] : v[k + s], keep = up ? v[k + s] : v[k];
            v[k] = keep + __shfl_xor_sync(0xffffffffu, give, s);
        }
    }
    return v[0] + __shfl_xor_sync(0xffffffffu, v[0], 16);
}

// A products' operand of 128 rows in tensor memory, 16 of K after 16: at + 16 k holds eight
// columns of hi and eight of lo.
__device__ __forceinline__ void mma_split(uint32_t d, uint32_t at, uint64_t b, uint32_t b_inc, uint32_t idesc,
                                          int steps, uint32_t acc) {
#pragma unroll 1
    for (int k = 0; k < steps; ++k) {
        mma_bf16_ts(d, at + 16 * k, b, idesc, acc);
        mma_bf16_ts(d, at + 16 * k + 8, b, idesc, 1);
        b += b_inc;
        acc = 1;
    }
}

// A part's fp32 tile of 128 rows from tensor memory: lane = row, a quarter of the columns per
// warp (at least 8).  In memory [Ns / 4][128][4], so that a warp's stores are contiguous.
__device__ __forceinline__ int64_t share_off(int row, int col) { return ((int64_t)(col >> 2) * kTL + row) * 4; }
template <int NK>
__device__ __forceinline__ void store_share(float *out, uint32_t tm, int warp, int lane, int Ns) {
    constexpr int W = NK / 4;
    const int quad = warp & 3, c0 = (warp >> 2) * W, r = quad * 32 + lane;
#pragma unroll
    for (int c = 0; c < W; c += 8) {
        float t[8];
        tc::tmem_ld8(tc::tmem_at(tm, quad * 32, c0 + c), t);
        if (c0 + c < Ns) {
            *reinterpret_cast<float4 *>(out + share_off(r, c0 + c)) = make_float4(t[0], t[1], t[2], t[3]);
            *reinterpret_cast<float4 *>(out + share_off(r, c0 + c + 4)) = make_float4(t[4], t[5], t[6], t[7]);
        }
    }
}

// ------------------------------------------------------------------------- i side
// Tensor memory: G (0), Z then W over it (128), dC (256), C S (384), 2^{a_i} dy (448).
template <int NK>
struct GradISmem {
    uint8_t C[kTL * NK * 2], B[kTL * NK * 2];
    struct Stage {
        uint8_t x[kTL * kPT * 2], dy[kTL * kPT * 2], S[2 * NK * kPT * 2];
        RowDecays dec;
    } st[2];
    uint8_t S_lo[NK * kPT * 2];
    float rs[4][kTL], rq[4][kTL], us[4][kTL];
    uint64_t lo_full, full[2], rows[2], z_done, dy_ready, e_done, w_ready, done, g_done, cb;
    uint32_t slot_addr;
    int dead;
};

template <bool AL, int NK>
__global__ void __launch_bounds__(kGAll, 1) ssm_tc_grad_i_kernel(SsmArgs p) {
    extern __shared__ __align__(1024) uint8_t raw_smem[];
    GradISmem<NK> &s = *reinterpret_cast<GradISmem<NK> *>(raw_smem);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    GradWork w;
    if (!w.start(p)) {  // (the chunk table is older than the kernel before)
        follow();
        return;
    }
    const int n = w.count;
    __builtin_assume(n > 0);
    for (int st = 0; st < 2; ++st)  // state rows past Ns are zeros
        for (int e = tid; e < 2 * NK * kPT * 2 / 16; e += kGAll)
            reinterpret_cast<uint4 *>(s.st[st].S)[e] = make_uint4(0u, 0u, 0u, 0u);
    for (int e = tid; e < NK * kPT * 2 / 16; e += kGAll)
        reinterpret_cast<uint4 *>(s.S_lo)[e] = make_uint4(0u, 0u, 0u, 0u);
    if (tid == 0) {
        for (int k = 0; k < 2; ++k) {
            tc::mbar_init(&s.full[k], 1);
            tc::mbar_init(&s.rows[k], kGWarps);
        }
        tc::mbar_init(&s.z_done, 1);
        tc::mbar_init(&s.e_done, 1);
        tc::mbar_init(&s.done, 1);
        tc::mbar_init(&s.dy_ready, kGWarps);
        tc::mbar_init(&s.lo_full, 1);
        tc::mbar_init(&s.w_ready, kGWarps);
        tc::mbar_init(&s.cb, kGWarps);
        tc::mbar_init(&s.g_done, 1);
        tc::mbar_fence_init();
        s.dead = 0;
    }
    tc::fence_async_smem();
    const uint32_t tm = tmem_open(&s.slot_addr, 512);
    follow();
    const uint32_t G = tm, W = tm + 128, dC = tm + 256, E = tm + 384, DY = tm + 448;
    volatile int *dead = &s.dead;
    if (warp == kGWarps) {
        if (lane == 0) {
            const int64_t tile = state_tile_bytes(p.Ns);
            int fetched = 0;
            auto fetch = [&](int it) {
                fetched = it + 1;
                const GradUnit u = w.at(p, it);
                auto &st = s.st[it & 1];
                uint64_t *bar = &s.full[it & 1];
                const uint8_t *src = reinterpret_cast<const uint8_t *>(p.states) + u.unit * 2 * tile;
                tc::mbar_arrive_expect_tx(bar, (uint32_t)(2 * tile + sizeof(RowDecays)));
                tc::bulk_g2s(st.S, src, (uint32_t)tile, bar);
                tc::bulk_g2s(st.S + NK * kPT * 2, src + tile, (uint32_t)tile, bar);
                tc::bulk_g2s(&st.dec, static_cast<const RowDecays *>(p.rows) + w.slot * p.H + u.h, sizeof(RowDecays),
                             bar);
            };
            int fetched_lo = 0;
            auto fetch_lo = [&](int it) {
                fetched_lo = it + 1;
                tc::mbar_arrive_expect_tx(&s.lo_full, (uint32_t)tile);
                tc::bulk_g2s(s.S_lo, static_cast<const uint8_t *>(p.states_lo) + w.at(p, it).unit * tile, (uint32_t)tile,
                             &s.lo_full);
            };
            const uint64_t ck = tc::sdesc(tc::smem_addr(s.C), 128, NK * 16);   // K-major
            const uint64_t bk = tc::sdesc(tc::smem_addr(s.B), 128, NK * 16);
            const uint64_t bmn = tc::sdesc(tc::smem_addr(s.B), NK * 16, 128);  // rows = K
            fetch(0);
            fetch_lo(0);
            if (n > 1) fetch(1);
            bool ok = wait_or_die(&s.cb, 0, dead, p.status);
            tc::tc_fence_after();
            if (ok) {
                mma_steps(G, ck, 16, bk, 16, tc::idesc_bf16(128, 128, false, false), NK / 16, 0);
                tc::mma_commit(&s.g_done);
            }
            for (int it = 0; it < n; ++it) {
                auto &st = s.st[it & 1];
                const uint32_t ph = it & 1, ph2 = (it >> 1) & 1;
                const uint32_t xa = tc::smem_addr(st.x), ya = tc::smem_addr(st.dy), sa = tc::smem_addr(st.S);
                ok = wait_or_die(&s.rows[it & 1], ph2, dead, p.status);
                tc::tc_fence_after();
                if (ok) {  // Z over the W of the unit before, which the products before have read
                    mma_steps(W, tc::sdesc(ya, 128, kPT * 16), 16, tc::sdesc(xa, 128, kPT * 16), 16,
                              tc::idesc_bf16(128, 128, false, false), kPT / 16, 0);
                    tc::mma_commit(&s.z_done);
                }
                ok = ok && wait_or_die(&s.full[it & 1], ph2, dead, p.status) &&
                     wait_or_die(&s.lo_full, ph, dead, p.status);
                if (ok) {
                    const uint64_t smn = tc::sdesc(sa, kPT * 16, 128);
                    const uint32_t id = tc::idesc_bf16(128, kPT, false, true);
                    mma_steps(E, ck, 16, tc::sdesc(tc::smem_addr(s.S_lo), kPT * 16, 128), 2 * kPT, id, NK / 16, 0);
                    mma_steps(E, ck, 16, smn + NK * kPT * 2 / 16, 2 * kPT, id, NK / 16, 1);
                    mma_steps(E, ck, 16, smn, 2 * kPT, id, NK / 16, 1);
                    tc::mma_commit(&s.e_done);
                }
                ok = ok && wait_or_die(&s.dy_ready, ph, dead, p.status);
                tc::tc_fence_after();
                if (ok) {
                    const uint64_t sk = tc::sdesc(sa, 128, kPT * 16);  // [n][p]: K-major
                    const uint32_t id = tc::idesc_bf16(128, NK, false, false);
                    mma_split(dC, DY, sk, 16, id, kPT / 16, it > 0);
#pragma unroll 1
                    for (int k = 0; k < kPT / 16; ++k)
                        mma_bf16_ts(dC, DY + 16 * k, sk + NK * kPT * 2 / 16 + 16 * k, id, 1);
                }
                // C S was the last reader of lo
                if (it + 1 < n && wait_or_die(&s.e_done, ph, dead, p.status)) fetch_lo(it + 1);
                ok = ok && wait_or_die(&s.w_ready, ph, dead, p.status);
                tc::tc_fence_after();
                if (ok) {
                    mma_split(dC, W, bmn, 2 * NK, tc::idesc_bf16(128, NK, false, true), kTL / 16, 1);
                    tc::mma_commit(&s.done);
                }
                // the stage is free once this unit is multiplied and its rows are read
                if (it + 2 < n && wait_or_die(&s.done, ph, dead, p.status)) fetch(it + 2);
            }
            if (*dead) {  // what is on its way lands before the block ends
                for (int it = max(fetched - 2, 0); it < fetched; ++it)
                    tc::mbar_wait(&s.full[it & 1], (it >> 1) & 1, 10000000ull);
                tc::mbar_wait(&s.lo_full, (fetched_lo - 1) & 1, 10000000ull);
            }
        }
        __syncwarp();
    } else {
        const int quad = warp & 3, part = warp >> 2, i = quad * 32 + lane;
        auto warp_arrive = [&](uint64_t *bar) {
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(bar);
        };
        auto load = [&](int it) {
            const GradUnit u = w.at(p, it);
            const int col = u.tile * kPT, cols = min(kPT, p.P - col);
            load_tile64<AL>(s.st[it & 1].x,
                            static_cast<const bf16 *>(p.x) + w.c.r0 * p.x_stride + (int64_t)u.h * p.P + col,
                            p.x_stride, w.c.nr, cols);
            load_tile64<AL>(s.st[it & 1].dy, static_cast<const bf16 *>(p.dy) + (w.c.r0 * p.H + u.h) * p.P + col,
                            (int64_t)p.H * p.P, w.c.nr, cols);
        };
        load_wide<AL, NK>(s.C, static_cast<const bf16 *>(p.Cm) + w.c.r0 * p.c_stride + w.g * p.Ns, p.c_stride, w.c.nr,
                          p.Ns);
        load_wide<AL, NK>(s.B, static_cast<const bf16 *>(p.Bm) + w.c.r0 * p.b_stride + w.g * p.Ns, p.b_stride, w.c.nr,
                          p.Ns);
        load(0);
        cp_async_wait_all();
        tc::fence_async_smem();
        warp_arrive(&s.cb);
        warp_arrive(&s.rows[0]);
        wait_or_die(&s.g_done, 0, dead, p.status);
        for (int it = 0; it < n; ++it) {
            const GradUnit u = w.at(p, it);
            auto &st = s.st[it & 1];
            const uint32_t ph = it & 1, ph2 = (it >> 1) & 1;
            wait_or_die(&s.full[it & 1], ph2, dead, p.status);
            const RowDecays &r = st.dec;
            const float ai = r.a[i], li = r.lo[i], ea = ex2_ftz(ai);
            // 2^{a_i} dy, sixteen columns a warp
            float dy[16];
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                float f[8];
                load_vec<bf16, 8, true>(reinterpret_cast<const bf16 *>(st.dy + (i >> 3) * (kPT * 16) +
                                                                      (part * 2 + q) * 128 + (i & 7) * 16),
                                        8, f);
#pragma unroll
                for (int k = 0; k < 8; ++k) dy[8 * q + k] = ea * f[k];
            }
            {
                uint32_t o[16];
#pragma unroll
                for (int q = 0; q < 8; ++q) split2(dy[2 * q], dy[2 * q + 1], o[q], o[8 + q]);
                tmem_st16_nowait(tc::tmem_at(DY, quad * 32, part * 16), o);
                tmem_wait_st();
                tc::tc_fence_before();
                warp_arrive(&s.dy_ready);
            }
            // W over Z, and the sums of Q below the diagonal
            wait_or_die(&s.z_done, ph, dead, p.status);
            tc::tc_fence_after();
            float before = 0.f;  // of row i, over this warp's columns so far
#pragma unroll 1
            for (int k = 0; k < 2; ++k) {
                const int J = 2 * part + k;
                const uint32_t at = tc::tmem_at(W, quad * 32, J * kSub);
                uint32_t o[16];
                if (J > 2 * quad + 1) {
#pragma unroll
                    for (int q = 0; q < 16; ++q) o[q] = 0u;
                } else {
                    uint32_t z[16], gm[16];
                    tmem_ld16_nowait(at, z);
                    tmem_ld16_nowait(tc::tmem_at(G, quad * 32, J * kSub), gm);
                    float c[16];  // Q, below the diagonal
                    if (J < 2 * quad) {
                        const int e = J * kSub + kSub - 1;
                        const float to_ref = ex2_ftz((ai - r.a[e]) + (li - r.lo[e]));
                        const uint64_t ref2 = pack2(to_ref, to_ref);
                        tmem_wait_ld();
#pragma unroll
                        for (int q = 0; q < 8; ++q) {
                            const uint64_t f = *reinterpret_cast<const uint64_t *>(&r.fd[J * kSub + 2 * q]);
                            const uint64_t v = mul2(pack2(z[2 * q], z[2 * q + 1]), mul2(ref2, f));
                            unpack2(mul2(v, pack2(gm[2 * q], gm[2 * q + 1])), c[2 * q], c[2 * q + 1]);
                            split2p(v, o[q], o[8 + q]);
                        }
                    } else {
                        tmem_wait_ld();
#pragma unroll
                        for (int q = 0; q < 8; ++q) {
                            float v[2];
#pragma unroll
                            for (int x = 0; x < 2; ++x) {
                                const int j = J * kSub + 2 * q + x;
                                const float f = ex2_ftz((ai - r.a[j]) + (li - r.lo[j])) * r.d[j];
                                // selects: above the diagonal the exponential may overflow
                                v[x] = j <= i ? __uint_as_float(z[2 * q + x]) * f : 0.f;
                                c[2 * q + x] = j < i ? v[x] * __uint_as_float(gm[2 * q + x]) : 0.f;
                            }
                            split2(v[0], v[1], o[q], o[8 + q]);
                        }
                    }
                    // sums over the columns before t, of the rows i >= t: a column's place takes
                    // the running sum of the row
#pragma unroll
                    for (int q = 0; q < 16; ++q) {
                        const float x = c[q];
                        c[q] = before;
                        before += x;
                    }
                    if (J >= 2 * quad) {
#pragma unroll
                        for (int q = 0; q < 16; ++q) c[q] = J * kSub + q <= i ? c[q] : 0.f;
                    }
                    const float sum = lane_sums(c);
                    if (lane < 16) s.rq[quad][J * kSub + lane] = sum;
                }
                tmem_st16_nowait(at, o);
            }
            s.rs[part][i] = before;
            tmem_wait_st();
            tc::tc_fence_before();
            warp_arrive(&s.w_ready);
            if (it + 1 < n) load(it + 1);  // into the stage of the unit before: its products are done
            // u_i
            wait_or_die(&s.e_done, ph, dead, p.status);
            tc::tc_fence_after();
            {
                uint32_t e[16];
                tmem_ld16_nowait(tc::tmem_at(E, quad * 32, part * 16), e);
                tmem_wait_ld();
                float sum = 0.f;
#pragma unroll
                for (int q = 0; q < 16; ++q) sum = fmaf(dy[q], __uint_as_float(e[q]), sum);
                s.us[part][i] = sum;
            }
            bar_sync(1, kGThreads);
            // the columns of the warps to the left: all rows of a quad lie past the columns of
            // a part before its own, and from row t on in its own
            if (part > 0 && part <= quad) {
                float left = 0.f;
                for (int k = 0; k < part; ++k) left += s.rs[k][i];
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const float x = __shfl_down_sync(0xffffffffu, left, o);
                    if (lane + o < 32) left += x;
                }
                if (part < quad) left = __shfl_sync(0xffffffffu, left, 0);
                s.rq[quad][part * 32 + lane] += left;
            }
            bar_sync(1, kGThreads);
            if (tid < kTL) {
                float *out = p.rowg + u.unit * 4 * kTL;
                float sum = 0.f;
                for (int q = tid >> 5; q < 4; ++q) sum += s.rq[q][tid];
                out[tid] = sum;
                out[kTL + tid] = (s.us[0][tid] + s.us[1][tid]) + (s.us[2][tid] + s.us[3][tid]);
            }
            wait_or_die(&s.done, ph, dead, p.status);
            tc::tc_fence_after();
            if (it + 1 < n) {
                cp_async_wait_all();
                tc::fence_async_smem();
                tc::tc_fence_before();  // what was read of this unit's sums
                warp_arrive(&s.rows[(it + 1) & 1]);
            }
            bar_sync(1, kGThreads);  // s.rq, s.rs, s.us are free
        }
        store_share<NK>(w.share(p, p.dCh), dC, warp, lane, p.Ns);
    }
    tmem_close(tm, 512);
}

// ------------------------------------------------------------------------- j side
// Tensor memory: G^T then M^T over it (0), Z^T then W^T over it (128), dB (256), M^T dy (384),
// B E (448).
template <int NK>
struct GradJSmem {
    uint8_t C[kTL * NK * 2], B[kTL * NK * 2];
    uint8_t x[2][kTL * kPT * 2], dy[2][kTL * kPT * 2];
    uint8_t E[3 * NK * kPT * 2];    // hi, mid, lo
    uint8_t wx[2][kTL * kPT * 2];   // w x, hi and lo
    RowDecays dec[2];
    float qs[4][kTL], vs[4][kTL], dds[kGWarps];
    uint64_t full[2], rows[2], z_done, wx_ready, xi_done, e_done, m_ready, done, cb;
    uint32_t slot_addr;
    int dead;
};

template <bool AL, int NK>
__global__ void __launch_bounds__(kGAll, 1) ssm_tc_grad_j_kernel(SsmArgs p, int dx_aligned) {
    extern __shared__ __align__(1024) uint8_t raw_smem[];
    GradJSmem<NK> &s = *reinterpret_cast<GradJSmem<NK> *>(raw_smem);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    GradWork w;
    if (!w.start(p)) {  // (the chunk table is older than the kernel before)
        follow();
        return;
    }
    const int n = w.count;
    __builtin_assume(n > 0);
    for (int e = tid; e < 3 * NK * kPT * 2 / 16; e += kGAll)
        reinterpret_cast<uint4 *>(s.E)[e] = make_uint4(0u, 0u, 0u, 0u);
    if (tid == 0) {
        for (int k = 0; k < 2; ++k) {
            tc::mbar_init(&s.full[k], 1);
            tc::mbar_init(&s.rows[k], kGWarps);
        }
        tc::mbar_init(&s.z_done, 1);
        tc::mbar_init(&s.xi_done, 1);
        tc::mbar_init(&s.e_done, 1);
        tc::mbar_init(&s.done, 1);
        tc::mbar_init(&s.wx_ready, kGWarps);
        tc::mbar_init(&s.m_ready, kGWarps);
        tc::mbar_init(&s.cb, kGWarps);
        tc::mbar_fence_init();
        s.dead = 0;
    }
    tc::fence_async_smem();
    const uint32_t tm = tmem_open(&s.slot_addr, 512);
    follow();
    const uint32_t M = tm, W = tm + 128, dB = tm + 256, DX = tm + 384, XI = tm + 448;
    volatile int *dead = &s.dead;
    if (warp == kGWarps) {
        if (lane == 0) {
            const int64_t tile = state_tile_bytes(p.Ns);
            int fetched = 0;
            auto fetch = [&](int it) {
                fetched = it + 1;
                const GradUnit u = w.at(p, it);
                uint64_t *bar = &s.full[it & 1];
                const uint8_t *src = reinterpret_cast<const uint8_t *>(p.dstates) + u.unit * 2 * tile;
                tc::mbar_arrive_expect_tx(bar, (uint32_t)(3 * tile + sizeof(RowDecays)));
                tc::bulk_g2s(s.E, src, (uint32_t)tile, bar);
                tc::bulk_g2s(s.E + NK * kPT * 2, src + tile, (uint32_t)tile, bar);
                tc::bulk_g2s(s.E + 2 * NK * kPT * 2, static_cast<const uint8_t *>(p.dstates_lo) + u.unit * tile,
                             (uint32_t)tile, bar);
                tc::bulk_g2s(&s.dec[it & 1], static_cast<const RowDecays *>(p.rows) + w.slot * p.H + u.h,
                             sizeof(RowDecays), bar);
            };
            const uint64_t ck = tc::sdesc(tc::smem_addr(s.C), 128, NK * 16);   // K-major
            const uint64_t bk = tc::sdesc(tc::smem_addr(s.B), 128, NK * 16);
            const uint64_t cmn = tc::sdesc(tc::smem_addr(s.C), NK * 16, 128);  // rows = K
            const uint32_t ea = tc::smem_addr(s.E);
            const uint64_t emn = tc::sdesc(ea, kPT * 16, 128), ek = tc::sdesc(ea, 128, kPT * 16);
            constexpr uint64_t emid = NK * kPT * 2 / 16;
            fetch(0);
            bool ok = wait_or_die(&s.cb, 0, dead, p.status);
            for (int it = 0; it < n; ++it) {
                const uint32_t ph = it & 1, ph2 = (it >> 1) & 1;
                const uint32_t xa = tc::smem_addr(s.x[it & 1]), ya = tc::smem_addr(s.dy[it & 1]);
                ok = wait_or_die(&s.rows[it & 1], ph2, dead, p.status);
                tc::tc_fence_after();
                if (ok) {  // over M^T and W^T of the unit before: it is multiplied
                    const uint32_t id = tc::idesc_bf16(128, 128, false, false);
                    mma_steps(M, bk, 16, ck, 16, id, NK / 16, 0);
                    mma_steps(W, tc::sdesc(xa, 128, kPT * 16), 16, tc::sdesc(ya, 128, kPT * 16), 16, id, kPT / 16, 0);
                    tc::mma_commit(&s.z_done);
                }
                ok = ok && wait_or_die(&s.full[it & 1], ph2, dead, p.status);
                if (ok) {
                    const uint32_t id = tc::idesc_bf16(128, kPT, false, true);
                    mma_steps(XI, bk, 16, emn + 2 * emid, 2 * kPT, id, NK / 16, 0);
                    mma_steps(XI, bk, 16, emn + emid, 2 * kPT, id, NK / 16, 1);
                    mma_steps(XI, bk, 16, emn, 2 * kPT, id, NK / 16, 1);
                    tc::mma_commit(&s.xi_done);
                }
                ok = ok && wait_or_die(&s.wx_ready, ph, dead, p.status);
                tc::tc_fence_after();
                if (ok) {  // (hi + lo) E_hi + hi E_mid
                    const uint32_t id = tc::idesc_bf16(128, NK, false, false);
                    const uint64_t hi = tc::sdesc(tc::smem_addr(s.wx[0]), 128, kPT * 16);
                    const uint64_t lo = tc::sdesc(tc::smem_addr(s.wx[1]), 128, kPT * 16);
                    mma_steps(dB, hi, 16, ek, 16, id, kPT / 16, it > 0);
                    mma_steps(dB, lo, 16, ek, 16, id, kPT / 16, 1);
                    mma_steps(dB, hi, 16, ek + emid, 16, id, kPT / 16, 1);
                    tc::mma_commit(&s.e_done);
                }
                ok = ok && wait_or_die(&s.m_ready, ph, dead, p.status);
                tc::tc_fence_after();
                if (ok) {
                    mma_split(DX, M, tc::sdesc(ya, kPT * 16, 128), 2 * kPT, tc::idesc_bf16(128, kPT, false, true),
                              kTL / 16, 0);
                    mma_split(dB, W, cmn, 2 * NK, tc::idesc_bf16(128, NK, false, true), kTL / 16, 1);
                    tc::mma_commit(&s.done);
                }
                // E is free: the products that read it come before those that wait for M
                if (it + 1 < n && wait_or_die(&s.e_done, ph, dead, p.status)) fetch(it + 1);
            }
            if (*dead) tc::mbar_wait(&s.full[(fetched - 1) & 1], ((fetched - 1) >> 1) & 1, 10000000ull);
        }
        __syncwarp();
    } else {
        const int quad = warp & 3, part = warp >> 2, j = quad * 32 + lane;
        auto warp_arrive = [&](uint64_t *bar) {
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(bar);
        };
        auto load = [&](int it) {
            const GradUnit u = w.at(p, it);
            const int col = u.tile * kPT, cols = min(kPT, p.P - col);
            load_tile64<AL>(s.x[it & 1],
                            static_cast<const bf16 *>(p.x) + w.c.r0 * p.x_stride + (int64_t)u.h * p.P + col,
                            p.x_stride, w.c.nr, cols);
            load_tile64<AL>(s.dy[it & 1], static_cast<const bf16 *>(p.dy) + (w.c.r0 * p.H + u.h) * p.P + col,
                            (int64_t)p.H * p.P, w.c.nr, cols);
        };
        load_wide<AL, NK>(s.C, static_cast<const bf16 *>(p.Cm) + w.c.r0 * p.c_stride + w.g * p.Ns, p.c_stride, w.c.nr,
                          p.Ns);
        load_wide<AL, NK>(s.B, static_cast<const bf16 *>(p.Bm) + w.c.r0 * p.b_stride + w.g * p.Ns, p.b_stride, w.c.nr,
                          p.Ns);
        load(0);
        cp_async_wait_all();
        tc::fence_async_smem();
        warp_arrive(&s.cb);
        warp_arrive(&s.rows[0]);
        for (int it = 0; it < n; ++it) {
            const GradUnit u = w.at(p, it);
            const uint32_t ph = it & 1, ph2 = (it >> 1) & 1;
            wait_or_die(&s.full[it & 1], ph2, dead, p.status);
            const RowDecays &r = s.dec[it & 1];
            const float D = p.D ? p.D[u.h] : 0.f;
            {   // w x in two parts: each thread's pieces, rows r0 and r0 + 64
                const int c8 = (tid >> 3) & 7, r0 = (tid >> 6) * 8 + (tid & 7);
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int rr = r0 + 64 * k;
                    const uint32_t off = (uint32_t)((rr >> 3) * (kPT * 16) + c8 * 128 + (rr & 7) * 16);
                    float f[8];
                    load_vec<bf16, 8, true>(reinterpret_cast<const bf16 *>(s.x[it & 1] + off), 8, f);
                    const float sc = r.w[rr];
                    uint4 hi, lo;
                    split2(f[0] * sc, f[1] * sc, hi.x, lo.x);
                    split2(f[2] * sc, f[3] * sc, hi.y, lo.y);
                    split2(f[4] * sc, f[5] * sc, hi.z, lo.z);
                    split2(f[6] * sc, f[7] * sc, hi.w, lo.w);
                    *reinterpret_cast<uint4 *>(s.wx[0] + off) = hi;
                    *reinterpret_cast<uint4 *>(s.wx[1] + off) = lo;
                }
                tc::fence_async_smem();
                warp_arrive(&s.wx_ready);
            }
            // M^T over G^T and W^T over Z^T; the sums of Q / d_j over i
            const float aj = r.a[j], lj = r.lo[j], dj = r.d[j];
            wait_or_die(&s.z_done, ph, dead, p.status);
            tc::tc_fence_after();
            float qsum = 0.f;
#pragma unroll 1
            for (int k = 0; k < 2; ++k) {
                const int I = 2 * part + k;
                const uint32_t mt = tc::tmem_at(M, quad * 32, I * kSub), wt = tc::tmem_at(W, quad * 32, I * kSub);
                uint32_t om[16], ow[16];
                uint64_t mo[8], zo[8];
                if (I < 2 * quad) {
#pragma unroll
                    for (int q = 0; q < 16; ++q) om[q] = ow[q] = 0u;
                } else {
                    tmem_ld16_nowait(mt, om);
                    tmem_ld16_nowait(wt, ow);
                    const float to_first = ex2_ftz((r.a[I * kSub] - aj) + (r.lo[I * kSub] - lj));
                    tmem_wait_ld();
                    if (I > 2 * quad + 1) {
                        const uint64_t first2 = pack2(to_first, to_first), d2 = pack2(dj, dj);
                        uint64_t sum2 = 0;
#pragma unroll
                        for (int q = 0; q < 8; ++q) {
                            const uint64_t f = mul2(first2, *reinterpret_cast<const uint64_t *>(&r.fi[I * kSub + 2 * q]));
                            const uint64_t g = pack2(om[2 * q], om[2 * q + 1]);
                            const uint64_t z = mul2(pack2(ow[2 * q], ow[2 * q + 1]), f);
                            sum2 = fma2(z, g, sum2);
                            mo[q] = mul2(g, mul2(f, d2));
                            zo[q] = mul2(z, d2);
                        }
                        float x, y;
                        unpack2(sum2, x, y);
                        qsum += x + y;
                    } else {
#pragma unroll
                        for (int q = 0; q < 8; ++q) {
                            float m[2], z[2];
#pragma unroll
                            for (int x = 0; x < 2; ++x) {
                                const int i = I * kSub + 2 * q + x;
                                const bool in = i >= j;  // selects: the exponential may overflow elsewhere
                                const float f = ex2_ftz((r.a[i] - aj) + (r.lo[i] - lj));
                                const float zf = in ? __uint_as_float(ow[2 * q + x]) * f : 0.f;
                                const float gf = in ? __uint_as_float(om[2 * q + x]) : 0.f;
                                qsum = fmaf(zf, gf, qsum);
                                m[x] = in ? gf * f * dj : 0.f;
                                z[x] = zf * dj;
                            }
                            mo[q] = pack2(m[0], m[1]);
                            zo[q] = pack2(z[0], z[1]);
                        }
                    }
#pragma unroll
                    for (int q = 0; q < 8; ++q) {
                        split2p(mo[q], om[q], om[8 + q]);
                        split2p(zo[q], ow[q], ow[8 + q]);
                    }
                }
                tmem_st16_nowait(mt, om);
                tmem_st16_nowait(wt, ow);
            }
            tmem_wait_st();
            tc::tc_fence_before();
            warp_arrive(&s.m_ready);
            if (it + 1 < n) load(it + 1);
            s.qs[part][j] = qsum;
            // B E: its product with x, and its share of dx
            const int c16 = part * 2;
            float xv[16], yv[16];
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                float f[8];
                const uint32_t off = (uint32_t)((j >> 3) * (kPT * 16) + (c16 + q) * 128 + (j & 7) * 16);
                load_vec<bf16, 8, true>(reinterpret_cast<const bf16 *>(s.x[it & 1] + off), 8, f);
#pragma unroll
                for (int k = 0; k < 8; ++k) xv[8 * q + k] = f[k];
                load_vec<bf16, 8, true>(reinterpret_cast<const bf16 *>(s.dy[it & 1] + off), 8, f);
#pragma unroll
                for (int k = 0; k < 8; ++k) yv[8 * q + k] = f[k];
            }
            float dd = 0.f, vsum = 0.f;
#pragma unroll
            for (int q = 0; q < 16; ++q) dd = fmaf(xv[q], yv[q], dd);
            const float wj = r.w[j];
            wait_or_die(&s.xi_done, ph, dead, p.status);
            tc::tc_fence_after();
            {
                uint32_t e[16];
                tmem_ld16_nowait(tc::tmem_at(XI, quad * 32, part * 16), e);
                tmem_wait_ld();
#pragma unroll
                for (int q = 0; q < 16; ++q) {
                    const float f = __uint_as_float(e[q]);
                    vsum = fmaf(xv[q], f, vsum);
                    yv[q] = p.D ? fmaf(D, yv[q], wj * f) : wj * f;
                }
            }
            s.vs[part][j] = vsum;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) dd += __shfl_xor_sync(0xffffffffu, dd, o);
            if (lane == 0) s.dds[warp] = dd;
            if (it + 1 < n) {
                cp_async_wait_all();
                tc::fence_async_smem();
            }
            wait_or_die(&s.done, ph, dead, p.status);
            tc::tc_fence_after();
            {   // dx over dy's tile, whose readers are through, for stores of whole rows
                uint32_t e[16];
                tmem_ld16_nowait(tc::tmem_at(DX, quad * 32, part * 16), e);
                tmem_wait_ld();
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const uint32_t off = (uint32_t)((j >> 3) * (kPT * 16) + (c16 + q) * 128 + (j & 7) * 16);
                    uint32_t o[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        o[k] = pack_bf16(yv[8 * q + 2 * k] + __uint_as_float(e[8 * q + 2 * k]),
                                         yv[8 * q + 2 * k + 1] + __uint_as_float(e[8 * q + 2 * k + 1]));
                    *reinterpret_cast<uint4 *>(s.dy[it & 1] + off) = make_uint4(o[0], o[1], o[2], o[3]);
                }
            }
            tc::tc_fence_before();  // DX, XI and the rows before the next unit's products
            if (it + 1 < n) warp_arrive(&s.rows[(it + 1) & 1]);
            bar_sync(1, kGThreads);
            {   // a thread's pieces are those that it loads: no other thread's copy overtakes it
                const int c8 = (tid >> 3) & 7, r0 = (tid >> 6) * 8 + (tid & 7), col = u.tile * kPT + c8 * 8;
                bf16 *dx = static_cast<bf16 *>(p.dx) + (w.c.r0 * p.H + u.h) * p.P + col;
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int rr = r0 + 64 * k;
                    const uint8_t *src = s.dy[it & 1] + (rr >> 3) * (kPT * 16) + c8 * 128 + (rr & 7) * 16;
                    bf16 *dst = dx + (int64_t)rr * p.H * p.P;
                    if (rr < w.c.nr && col < p.P) {
                        if (dx_aligned) {
                            *reinterpret_cast<uint4 *>(dst) = *reinterpret_cast<const uint4 *>(src);
                        } else {
#pragma unroll
                            for (int e = 0; e < 8; ++e) dst[e] = reinterpret_cast<const bf16 *>(src)[e];
                        }
                    }
                }
            }
            if (tid < kTL) {
                float *out = p.rowg + u.unit * 4 * kTL + 2 * kTL;
                const RowDecays &rr = s.dec[it & 1];
                const float el = ex2_ftz((rr.a[kTL - 1] - rr.a[tid]) + (rr.lo[kTL - 1] - rr.lo[tid]));
                const float v = el * ((s.vs[0][tid] + s.vs[1][tid]) + (s.vs[2][tid] + s.vs[3][tid]));
                out[tid] = ((s.qs[0][tid] + s.qs[1][tid]) + (s.qs[2][tid] + s.qs[3][tid])) + v;
                out[kTL + tid] = v * rr.d[tid];
            }
            if (tid == 0) {
                float sum = 0.f;
                for (int k = 0; k < kGWarps; ++k) sum += s.dds[k];
                p.dDp[u.unit] = sum;
            }
            bar_sync(1, kGThreads);
        }
        store_share<NK>(w.share(p, p.dBh), dB, warp, lane, p.Ns);
    }
    tmem_close(tm, 512);
}

// ------------------------------------------------- the steps' gradients, per (chunk, head)
__global__ void __launch_bounds__(kTL) ssm_tc_step_grads_kernel(SsmArgs p) {
    follow();
    __shared__ float su[4], sv[4], red[3][4];
    const int h = (int)(blockIdx.x % p.H), t = threadIdx.x, warp = t >> 5, lane = t & 31;
    const int64_t slot = blockIdx.x / p.H;
    TcChunk c;
    if (!tc_find_chunk(p, slot, c)) return;
    const int pt = tiles_of(p.P), es_n = (int)ssm_tc_es_per(p.Ns, p.P);
    const int64_t sh = slot * p.H + h;
    float R = 0.f, u = 0.f, q = 0.f, v = 0.f, e = 0.f, dD = 0.f;
    for (int k = 0; k < pt; ++k) {
        const float *g = p.rowg + (sh * pt + k) * 4 * kTL;
        R += g[t];
        u += g[kTL + t];
        q += g[2 * kTL + t];
        v += g[3 * kTL + t];
    }
    for (int k = lane; k < es_n; k += 32) e += p.es[sh * es_n + k];
    if (t == 0)
        for (int k = 0; k < pt; ++k) dD += p.dDp[sh * pt + k];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) e += __shfl_xor_sync(0xffffffffu, e, o);
    // u from the right (with the row itself), v from the left (without it)
    float ur = u, vl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const float x = __shfl_down_sync(0xffffffffu, ur, o), y = __shfl_up_sync(0xffffffffu, vl, o);
        if (lane + o < 32) ur += x;
        if (lane >= o) vl += y;
    }
    if (lane == 0) su[warp] = ur;
    if (lane == 31) sv[warp] = vl;
    vl = __shfl_up_sync(0xffffffffu, vl, 1);
    if (lane == 0) vl = 0.f;
    __syncthreads();
    for (int k = warp + 1; k < 4; ++k) ur += su[k];
    float vb = 0.f;
    for (int k = 0; k < warp; ++k) vb += sv[k];
    const float l = R + (ur + ((vb + vl) + p.decay[sh] * e));
    const float A = -expf(p.A_log[h]), bias = p.dt_bias ? p.dt_bias[h] : 0.f;
    const RowDecays *rd = static_cast<const RowDecays *>(p.rows) + sh;
    float sA = 0.f, sb = 0.f;
    if (t < c.nr) {
        const int64_t row = c.r0 + t;
        float gd = fmaf(A, l, q);
        if (p.softplus) {
            const float raw = to_f32(static_cast<const bf16 *>(p.dt)[row * p.dt_stride + h]) + bias;
            gd *= 1.f / (1.f + expf(-raw));
        }
        static_cast<bf16 *>(p.ddt)[row * p.H + h] = __float2bfloat16_rn(gd);
        sA = rd->d[t] * l;
        sb = gd;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        sA += __shfl_xor_sync(0xffffffffu, sA, o);
        sb += __shfl_xor_sync(0xffffffffu, sb, o);
    }
    if (lane == 0) {
        red[0][warp] = sA;
        red[1][warp] = sb;
    }
    __syncthreads();
    if (t == 0) {
        p.sums[(slot * 3 + 0) * p.H + h] = A * ((red[0][0] + red[0][1]) + (red[0][2] + red[0][3]));
        p.sums[(slot * 3 + 1) * p.H + h] = dD;
        p.sums[(slot * 3 + 2) * p.H + h] = (red[1][0] + red[1][1]) + (red[1][2] + red[1][3]);
    }
}

// dB and dC rows of a chunk and group, 16 to a block: the sum of the parts, in their order.
constexpr int kSumRows = 16;
__global__ void __launch_bounds__(256) ssm_tc_group_sum_kernel(SsmArgs p, int aligned) {
    follow();
    const int64_t sg = blockIdx.x / (kTL / kSumRows);
    const int row0 = (int)(blockIdx.x % (kTL / kSumRows)) * kSumRows;
    const int g = (int)(sg % p.G);
    TcChunk c;
    if (!tc_find_chunk(p, sg / p.G, c)) return;
    const int64_t tile = (int64_t)kTL * p.Ns;
    const float *b = p.dBh + sg * p.parts * tile, *cc = p.dCh + sg * p.parts * tile;
    // eight columns a thread; sixteen lanes take a column's rows
    for (int k = threadIdx.x; k < kSumRows * (p.Ns / 8); k += 256) {
        const int r = row0 + k % kSumRows, n = k / kSumRows * 8;
        if (r >= c.nr) continue;
        float sb[8] = {}, sc[8] = {};
        for (int q = 0; q < p.parts; ++q) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int64_t at = q * tile + share_off(r, n + 4 * h);
                const float4 x = *reinterpret_cast<const float4 *>(b + at);
                const float4 y = *reinterpret_cast<const float4 *>(cc + at);
                sb[4 * h] += x.x; sb[4 * h + 1] += x.y; sb[4 * h + 2] += x.z; sb[4 * h + 3] += x.w;
                sc[4 * h] += y.x; sc[4 * h + 1] += y.y; sc[4 * h + 2] += y.z; sc[4 * h + 3] += y.w;
            }
        }
        const int64_t at = ((c.r0 + r) * p.G + g) * p.Ns + n;
        bf16 *dB = static_cast<bf16 *>(p.dB) + at, *dC = static_cast<bf16 *>(p.dC) + at;
        if (aligned) {
            store_vec<bf16, 8, true>(dB, 8, sb);
            store_vec<bf16, 8, true>(dC, 8, sc);
        } else {
            store_vec<bf16, 8, false>(dB, 8, sb);
            store_vec<bf16, 8, false>(dC, 8, sc);
        }
    }
}

template <typename K>
cudaError_t allow(K kernel, size_t bytes) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
}
// at least this much, so that two CTAs never ask one SM for 1024 tensor-memory columns
constexpr size_t at_least(size_t n) { return n > 120 * 1024 ? n : 120 * 1024; }
template <bool AL, int NK>
cudaError_t allow_kernels() {
    cudaError_t e = allow(ssm_tc_grad_i_kernel<AL, NK>, at_least(sizeof(GradISmem<NK>)));
    if (e == cudaSuccess) e = allow(ssm_tc_grad_j_kernel<AL, NK>, at_least(sizeof(GradJSmem<NK>)));
    return e;
}
cudaError_t bwd_setup() {
    static DeviceOnce once;
    int dev = 0;
    return once.run(&dev, [](int) {
        cudaError_t e = allow_kernels<true, 32>();
        if (e == cudaSuccess) e = allow_kernels<false, 32>();
        if (e == cudaSuccess) e = allow_kernels<true, 64>();
        if (e == cudaSuccess) e = allow_kernels<false, 64>();
        if (e == cudaSuccess) e = allow_kernels<true, 128>();
        if (e == cudaSuccess) e = allow_kernels<false, 128>();
        return e;
    });
}

template <bool AL, int NK>
cudaError_t grads(const SsmArgs &a, unsigned blocks, cudaStream_t st) {
    prof_begin("ssm_tc_grad_i", st);
    cudaError_t e = launch_after(ssm_tc_grad_i_kernel<AL, NK>, blocks, kGAll, at_least(sizeof(GradISmem<NK>)), st, a);
    prof_end(st);
    if (e != cudaSuccess) return e;
    prof_begin("ssm_tc_grad_j", st);
    e = launch_after(ssm_tc_grad_j_kernel<AL, NK>, blocks, kGAll, at_least(sizeof(GradJSmem<NK>)), st, a,
                     aligned_to(a.dx, 16));
    prof_end(st);
    return e;
}

}  // namespace

// The split of a group's units, into no more parts than units, that takes the fewest rounds of units
// on 152 SMs.  64 chunks of
// one group with 32 units: 2 parts, 387 us for a training pass when this was measured; 1, 4, 5 and
// 7 parts 558, 409, 462 and 425 us.  Equal stretches over all SMs, across chunks, were slower too: each
// chunk begins with its B and C and ends with its tile of sums.
int ssm_tc_parts(int64_t slots, int G, int units) {
    const int64_t items = slots * G;
    if (items == 0 || units <= 1) return 1;
    int best = 1;
    int64_t cost = INT64_MAX;
    for (int k = 1; k <= units && k <= 32; ++k) {
        const int64_t rounds = (items * k + kSms - 1) / kSms;
        const int64_t c = rounds * ((units + k - 1) / k + 1);  // + 1: a CTA's start and end
        if (c < cost) {
            cost = c;
            best = k;
        }
    }
    return best;
}
int ssm_tc_tiles(int P) { return tiles_of(P); }
size_t ssm_tc_es_floats(int Ns, int P) { return (size_t)ssm_tc_es_per(Ns, P); }

cudaError_t launch_ssm_tc_bwd(const SsmArgs &a, cudaStream_t st) {
    cudaError_t e = bwd_setup();
    if (e != cudaSuccess) return e;
    const int64_t blocks = a.slots * a.G * a.parts, heads = a.slots * a.H;
    if (blocks > INT32_MAX || heads > INT32_MAX || a.slots * a.G * (kTL / kSumRows) > INT32_MAX)
        return cudaErrorInvalidValue;
    if (blocks == 0) return cudaSuccess;
    const bool al = aligned_to(a.x, 16) && aligned_to(a.Bm, 16) && aligned_to(a.Cm, 16) && aligned_to(a.dy, 16) &&
                    a.x_stride % 8 == 0 && a.b_stride % 8 == 0 && a.c_stride % 8 == 0;
    const unsigned g = (unsigned)blocks;
    if (a.Ns <= 32)
        e = al ? grads<true, 32>(a, g, st) : grads<false, 32>(a, g, st);
    else if (a.Ns <= 64)
        e = al ? grads<true, 64>(a, g, st) : grads<false, 64>(a, g, st);
    else
        e = al ? grads<true, 128>(a, g, st) : grads<false, 128>(a, g, st);
    if (e != cudaSuccess) return e;
    prof_begin("ssm_tc_step_grads", st);
    e = launch_after(ssm_tc_step_grads_kernel, heads, kTL, 0, st, a);
    prof_end(st);
    if (e != cudaSuccess) return e;
    prof_begin("ssm_tc_group_sum", st);
    e = launch_after(ssm_tc_group_sum_kernel, a.slots * a.G * (kTL / kSumRows), 256, 0, st, a,
                     aligned_to(a.dB, 16) && aligned_to(a.dC, 16));
    prof_end(st);
    return e;
}

}  // namespace kda
