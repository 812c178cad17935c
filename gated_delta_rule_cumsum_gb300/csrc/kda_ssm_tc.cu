// kda_ssm_tc.cu -- the scan's forward on the tensor cores (bf16 inputs, state rows and
// columns multiples of 8): the chunk form of kda_ssm.cu with chunks of 128 rows, every
// product a tcgen05.mma with fp32 accumulation.
//
// Precision.  x, B and C are bf16 and enter the products exactly.  What the kernel makes
// itself is split into bf16 parts that are multiplied one after another into the same
// accumulator: the decay-weighted x of a chunk's state in three (2^-25: the final state is
// an fp32 output; the smallest part first, since an addition to the full sum may cost it a
// unit in the last place, however small the addend), the masked gram and the state in front of
// y in two (2^-17: y is rounded to bf16 at the end).  One part alone would put up to 2^-8,
// y's own rounding, beside it.
#include "kda_ssm_tc.cuh"

namespace kda {
namespace {

using bf16 = __nv_bfloat16;

// Work is the list of units (slot, head, 64-column tile), in that order; each of a persistent
// grid's CTAs takes an equal stretch of it, so that consecutive units of a CTA mostly share a
// chunk and group and its B and C stay in shared memory.  A walk over units keeps its place
// by counting: the divisions of an index would cost more than a unit's elementwise work.
struct Walk {
    int64_t slot;
    int h, tile, g, pt, per_group;
    TcChunk c;
    __device__ __forceinline__ void start(const SsmArgs &p, int64_t unit) {
        pt = tiles_of(p.P);
        per_group = p.H / p.G;
        tile = (int)(unit % pt);
        const int64_t sh = unit / pt;
        h = (int)(sh % p.H);
        slot = sh / p.H;
        g = h / per_group;
        tc_find_chunk(p, slot, c);
    }
    __device__ __forceinline__ void next(const SsmArgs &p, bool find) {
        if (++tile < pt) return;
        tile = 0;
        if (++h % per_group == 0) ++g;
        if (h < p.H) return;
        h = g = 0;
        ++slot;
        if (find) tc_find_chunk(p, slot, c);
    }
};
__device__ __forceinline__ void work_range(int64_t total, int64_t &first, int64_t &last) {
    first = total * blockIdx.x / gridDim.x;
    last = total * (blockIdx.x + 1) / gridDim.x;
}
__device__ __forceinline__ int64_t slots_now(const SsmArgs &p) {
    return p.cu ? (p.ctrl->valid ? p.ctrl->total_chunks : 0) : p.slots;
}

// 128 x COLS of bf16 into a core-matrix tile by TH threads; rows past nr and columns past nc (a
// multiple of 8 when AL) are zeros.  Eight lanes take eight rows of one 16-byte column, so that
// neither side conflicts.
constexpr int kRowThreads = 512;
template <bool AL, int COLS, int TH>
__device__ __forceinline__ void load_rows(uint8_t *tile, const bf16 *src, int64_t stride, int nr, int nc) {
    constexpr int CPR = COLS / 8, IT = kTL * CPR / TH, STEP = TH / CPR;
    static_assert(STEP % 8 == 0 && IT * STEP == kTL, "whole groups of rows per round");
    const int tid = threadIdx.x, c8 = (tid >> 3) % CPR, r0 = (tid >> 3) / CPR * 8 + (tid & 7);
    const uint32_t off = (uint32_t)((r0 >> 3) * (COLS * 16) + c8 * 128 + (r0 & 7) * 16);
    const bf16 *s = src + r0 * stride + c8 * 8;
#pragma unroll
    for (int k = 0; k < IT; ++k) {
        const bool in = c8 * 8 < nc && r0 + k * STEP < nr;
        const uint32_t at = off + k * STEP / 8 * (COLS * 16);
        if constexpr (AL) {
            cp_async16(tc::smem_addr(tile) + at, in ? s + k * STEP * stride : src, in);
        } else {
            alignas(16) bf16 v[8];
#pragma unroll
            for (int j = 0; j < 8; ++j)
                v[j] = in && c8 * 8 + j < nc ? s[k * STEP * stride + j] : __float2bfloat16_rn(0.f);
            *reinterpret_cast<uint4 *>(tile + at) = *reinterpret_cast<const uint4 *>(v);
        }
    }
}

// -------------------------------------------------------------- the rows' decays
// One block per chunk and 16 heads: dt comes in whole sectors (16 heads of a row), then a warp
// per head scans its 128 rows, four per lane.  The running sums are of pairs of floats: see
// kda_ssm.cu for why, and the fp64 units are far too few to be asked.
// Measured: 8192 rows x 32 heads, 5 us; bound by latency.
constexpr int kRowHeads = 16;
__global__ void __launch_bounds__(32 * kRowHeads) ssm_tc_rows_kernel(SsmArgs p) {
    follow();
    __shared__ bf16 dts[kRowHeads][kTL + 4];
    const int hb = (p.H + kRowHeads - 1) / kRowHeads, h0 = (int)(blockIdx.x % hb) * kRowHeads;
    const int64_t slot = blockIdx.x / hb;
    TcChunk c;
    if (!tc_find_chunk(p, slot, c)) return;
    for (int e = threadIdx.x; e < kTL * kRowHeads; e += 32 * kRowHeads) {
        const int r = e / kRowHeads, k = e % kRowHeads;
        dts[k][r] = r < c.nr && h0 + k < p.H
                        ? static_cast<const bf16 *>(p.dt)[(c.r0 + r) * p.dt_stride + h0 + k]
                        : __float2bfloat16_rn(0.f);
    }
    __syncthreads();
    const int lane = threadIdx.x & 31, h = h0 + (threadIdx.x >> 5);
    if (h >= p.H) return;
    const float A = -expf(p.A_log[h]) * kLog2eTc, bias = p.dt_bias ? p.dt_bias[h] : 0.f;
    float d[4], a[4], lo[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int r = 4 * lane + k;
        const float raw = to_f32(dts[threadIdx.x >> 5][r]) + bias;
        d[k] = r < c.nr ? (p.softplus ? softplus_f(raw) : raw) : 0.f;
        a[k] = d[k] * A;
        lo[k] = fmaf(d[k], A, -a[k]);
        if (k > 0) pair_add(a[k], lo[k], a[k - 1], lo[k - 1]);
    }
    float sh = a[3], sl = lo[3];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const float uh = __shfl_up_sync(0xffffffffu, sh, o), ul = __shfl_up_sync(0xffffffffu, sl, o);
        if (lane >= o) pair_add(sh, sl, uh, ul);
    }
    const float eh = __shfl_sync(0xffffffffu, sh, 31), el = __shfl_sync(0xffffffffu, sl, 31);
    const float ph = __shfl_up_sync(0xffffffffu, sh, 1), pl = __shfl_up_sync(0xffffffffu, sl, 1);
#pragma unroll
    for (int k = 0; k < 4; ++k)
        if (lane > 0) pair_add(a[k], lo[k], ph, pl);
    // the last row of the block of 16: the fourth row of the last of its four lanes
    const float rh = __shfl_sync(0xffffffffu, a[3], lane | 3), rl = __shfl_sync(0xffffffffu, lo[3], lane | 3);
    const float ih = __shfl_sync(0xffffffffu, a[0], lane & ~3), il = __shfl_sync(0xffffffffu, lo[0], lane & ~3);
    float fd[4], w[4], fi[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        fi[k] = ex2_ftz((a[k] - ih) + (lo[k] - il));
        fd[k] = ex2_ftz((rh - a[k]) + (rl - lo[k])) * d[k];
        w[k] = ex2_ftz((eh - a[k]) + (el - lo[k])) * d[k];
    }
    RowDecays *rd = static_cast<RowDecays *>(p.rows) + slot * p.H + h;
    auto put = [&](float *to, const float (&v)[4]) {
        *reinterpret_cast<float4 *>(to + 4 * lane) = make_float4(v[0], v[1], v[2], v[3]);
    };
    put(rd->a, a);
    put(rd->lo, lo);
    put(rd->d, d);
    put(rd->fd, fd);
    put(rd->w, w);
    put(rd->fi, fi);
    if (lane == 0) p.decay[slot * p.H + h] = ex2_ftz(eh);
}

// ------------------------------------------------------------- a chunk's own state
// out[n][q] = sum_j w_j B_j[n] v_j[q] over the chunk's rows j:
//   forward:  v = x,  w_j = 2^{a_end - a_j} d_j   (states)
//   backward: B is C, v = dy, w_i = 2^{a_i}       (dstates)
// The operands are the tiles as they lie in memory, rows = K: both MN-major.  The result goes
// where the pass over chunks will leave hi and lo rows: columns 8 g .. 8 g + 3 in the hi row's
// 16 bytes, 8 g + 4 .. 8 g + 7 in the lo row's; a warp writes whole 128-byte lines.
// A product of 64 columns takes 57 cycles per 16 of K, one of 128 columns 64: two units of a
// group are taken together.  Sixteen warps split x and store results, one more issues the
// products; while a pair is multiplied, the one before it is stored and the next one's x is
// split into the other buffer.
// Measured: 8192 rows, 32 heads of 64, 128 state rows, 30 us either way (105 MB with what stays
// in L2); the tensor pipe is active 21% and issue slots 34% of the time: bound by each warp's
// chain of loads, splits and stores.
constexpr int kTcThreads = kRowThreads + 32, kRowWarps = kRowThreads / 32;
template <int MT>
struct StateSmem {
    uint8_t B[kTL * MT * 2];
    uint8_t X[2][3 * kTL * 2 * kPT * 2];  // hi, mid, lo tiles of [128][128]
    // of even and odd pairs: a warp may be a pair ahead of another, so one barrier for both
    // could count it twice
    uint64_t ready[2], done[2];
    uint32_t slot_addr;
    int dead;
};
template <bool AL, bool BWD, int MT>
__global__ void __launch_bounds__(kTcThreads, 1) ssm_tc_state_kernel(SsmArgs p) {
    extern __shared__ __align__(1024) uint8_t raw_smem[];
    StateSmem<MT> &s = *reinterpret_cast<StateSmem<MT> *>(raw_smem);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, pt = tiles_of(p.P);
    const int per_group = p.H / p.G, units = per_group * pt, pairs = (units + 1) / 2;  // of a group
    int64_t at, last;
    work_range(slots_now(p) * p.G * pairs, at, last);
    if (at >= last) {  // (the chunk table is older than the kernel before)
        follow();
        return;
    }
    const int n = (int)(last - at);
    if (tid == 0) {
        for (int k = 0; k < 2; ++k) {
            tc::mbar_init(&s.ready[k], kRowWarps);
            tc::mbar_init(&s.done[k], 1);
        }
        tc::mbar_fence_init();
        s.dead = 0;
    }
    const uint32_t tm = tmem_open(&s.slot_addr, 256);
    follow();
    volatile int *dead = &s.dead;
    if (warp == kRowWarps) {
        if (lane == 0) {
            const uint32_t idesc = tc::idesc_bf16(MT, 2 * kPT, true, true);
            const uint64_t a = tc::sdesc(tc::smem_addr(s.B), MT * 16, 128);
            constexpr uint64_t part = kTL * 2 * kPT * 2 / 16;
            for (int k = 0; k < n; ++k) {
                const bool ok = wait_or_die(&s.ready[k & 1], (k >> 1) & 1, dead, p.status);
                tc::tc_fence_after();
                if (!ok) continue;
                const uint64_t x = tc::sdesc(tc::smem_addr(s.X[k & 1]), 2 * kPT * 16, 128);
                const uint32_t d = tm + (k & 1) * 128;
#pragma unroll 1
                for (int q = 2; q >= 0; --q) mma_steps(d, a, 2 * MT, x + q * part, 4 * kPT, idesc, kTL / 16, q < 2);
                tc::mma_commit(&s.done[k & 1]);
            }
        }
        __syncwarp();
    } else {
        const int64_t vs = BWD ? (int64_t)p.H * p.P : p.x_stride;
        // a thread's pieces of x: rows r0 + 32 k of 16-byte column c8 of the pair's 16
        const int c8 = (tid >> 3) & 15, r0 = (tid >> 7) * 8 + (tid & 7), half = c8 >> 3;
        constexpr int IT = kTL / 32;
        uint4 xr[IT];
        float wr[IT];
        // the pair being fetched
        int pair = (int)(at % pairs), g = (int)(at / pairs % p.G);
        int64_t slot = at / pairs / p.G;
        TcChunk c;
        tc_find_chunk(p, slot, c);
        auto fetch = [&]() {
            const int u = 2 * pair + half;
            const int h = g * per_group + min(u, units - 1) / pt, q = u % pt * kPT + (c8 & 7) * 8;
            const bf16 *v = static_cast<const bf16 *>(BWD ? p.dy : p.x) + (c.r0 + r0) * vs + (int64_t)h * p.P + q;
            const RowDecays *rd = static_cast<const RowDecays *>(p.rows) + slot * p.H + h;
            const bool col = u < units && q < p.P;
#pragma unroll
            for (int k = 0; k < IT; ++k) {
                xr[k] = make_uint4(0u, 0u, 0u, 0u);
                if (col && r0 + 32 * k < c.nr) {
                    if constexpr (AL) {
                        xr[k] = *reinterpret_cast<const uint4 *>(v + 32 * k * vs);
                    } else {
                        alignas(16) bf16 e[8];
#pragma unroll
                        for (int j = 0; j < 8; ++j) e[j] = v[32 * k * vs + j];
                        xr[k] = *reinterpret_cast<const uint4 *>(e);
                    }
                }
                wr[k] = BWD ? rd->a[r0 + 32 * k] : rd->w[r0 + 32 * k];
            }
        };
        // where the pair before goes: its first unit (slot, head, tile), and how many
        int64_t out_unit = 0;
        int out_count = 0;
        auto store = [&](int k) {
            const bool ok = wait_or_die(&s.done[k & 1], (k >> 1) & 1, dead, p.status);
            tc::tc_fence_after();
            // M = 64 puts row r in lane (r / 16) * 32 + r % 16; 32 columns per warp
            const int quad = warp & 3, g0 = (warp >> 2) * 4, u = g0 >> 3;
            const int row = MT == 128 ? quad * 32 + lane : quad * 16 + lane;
            float t[32];
            tc::tmem_ld32(tc::tmem_at(tm + (k & 1) * 128, quad * 32, g0 * 8), t);
            if (ok && row < p.Ns && (MT == 128 || lane < 16) && u < out_count) {
                uint8_t *out = reinterpret_cast<uint8_t *>(BWD ? p.dstates : p.states) +
                               (out_unit + u) * 2 * state_tile_bytes(p.Ns) + state_off(row, g0 & 7);
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    *reinterpret_cast<float4 *>(out + q * 128) =
                        make_float4(t[8 * q], t[8 * q + 1], t[8 * q + 2], t[8 * q + 3]);
                    *reinterpret_cast<float4 *>(out + q * 128 + state_tile_bytes(p.Ns)) =
                        make_float4(t[8 * q + 4], t[8 * q + 5], t[8 * q + 6], t[8 * q + 7]);
                }
            }
        };
        fetch();
        int64_t b_slot = -1;
        int b_g = -1;
        for (int k = 0; k < n; ++k) {
            if (slot != b_slot || g != b_g) {  // the products that read the tile before are done
                if (k > 0) wait_or_die(&s.done[(k - 1) & 1], ((k - 1) >> 1) & 1, dead, p.status);
                const int64_t stride = BWD ? p.c_stride : p.b_stride;
                load_rows<AL, MT, kRowThreads>(s.B, static_cast<const bf16 *>(BWD ? p.Cm : p.Bm) + c.r0 * stride + g * p.Ns,
                                  stride, c.nr, p.Ns);
                b_slot = slot;
                b_g = g;
            }
            uint8_t *X = s.X[k & 1];  // pair k - 2 has left it: its store waited
#pragma unroll
            for (int q = 0; q < IT; ++q) {
                const int r = r0 + 32 * q;
                const uint32_t off = (uint32_t)((r >> 3) * (2 * kPT * 16) + c8 * 128 + (r & 7) * 16);
                const float w = BWD ? ex2_ftz(wr[q]) : wr[q];
                float f[8];
                load_vec<bf16, 8, true>(reinterpret_cast<const bf16 *>(&xr[q]), 8, f);
                uint4 hi, mid, lo;
                split3(f[0] * w, f[1] * w, hi.x, mid.x, lo.x);
                split3(f[2] * w, f[3] * w, hi.y, mid.y, lo.y);
                split3(f[4] * w, f[5] * w, hi.z, mid.z, lo.z);
                split3(f[6] * w, f[7] * w, hi.w, mid.w, lo.w);
                *reinterpret_cast<uint4 *>(X + off) = hi;
                *reinterpret_cast<uint4 *>(X + kTL * 2 * kPT * 2 + off) = mid;
                *reinterpret_cast<uint4 *>(X + 2 * kTL * 2 * kPT * 2 + off) = lo;
            }
            cp_async_wait_all();
            tc::fence_async_smem();
            tc::tc_fence_before();  // and the loads of pair k - 2's result
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&s.ready[k & 1]);
            const int64_t unit = (slot * p.H + g * per_group) * pt + 2 * pair;
            const int count = min(2, units - 2 * pair);
            if (k + 1 < n) {
                if (++pair == pairs) {
                    pair = 0;
                    if (++g == p.G) {
                        g = 0;
                        ++slot;
                        tc_find_chunk(p, slot, c);
                    }
                }
                fetch();
            }
            if (k > 0) store(k - 1);
            out_unit = unit;
            out_count = count;
        }
        store(n - 1);
    }
    tmem_close(tm, 256);
}

// The pass over a sequence's chunks (see ssm_state_pass_kernel), 8 columns of one state row
// per thread, in the order they lie in memory; the running state stays fp32 and is left at
// each chunk as hi and mid rows, and as lo rows where the backward will want them.
// Measured: the same size, forward 16 us (134 MB, part of it in L2), with lo rows 24 us (168 MB,
// 7.0 TB/s); reverse 42 us (268 MB, 6.4 TB/s).
template <bool REV>
__global__ void __launch_bounds__(128) ssm_tc_pass_kernel(SsmArgs p, int vec) {
    follow();
    const int pt = tiles_of(p.P), per_tile = p.Ns * 8;
    const int64_t np = (int64_t)p.Ns * p.P;
    const int64_t per = ((int64_t)pt * per_tile + 127) / 128, sh = blockIdx.x / per;
    const int64_t id = (blockIdx.x % per) * 128 + threadIdx.x;
    const int e = (int)(id % per_tile), tl = (int)(id / per_tile);
    const int n = (e >> 6) * 8 + (e & 7), g = tl * 8 + ((e >> 3) & 7);
    // columns past P of the last tile go along: they are zero in what the chunks left, and the
    // products read every column of every part
    const bool live = tl < pt, mine = live && g * 8 < p.P;
    if (!REV && !live) return;
    const int h = (int)(sh % p.H), seq = (int)(sh / p.H);
    int64_t first;
    int nc;
    if (p.cu) {
        if (!p.ctrl->valid) return;
        first = p.chunk_start[seq];
        nc = p.chunk_start[seq + 1] - p.chunk_start[seq];
    } else {
        nc = (p.T + kTL - 1) / kTL;
        first = (int64_t)seq * nc;
    }
    const float *from = REV ? p.dht : p.h0;
    float *to = REV ? p.dh0 : p.ht;
    const int64_t user = sh * np + (int64_t)n * p.P + g * 8;
    float run[8] = {};
    if (from && mine) {
        if (vec) {
            const float4 x = *reinterpret_cast<const float4 *>(from + user);
            const float4 y = *reinterpret_cast<const float4 *>(from + user + 4);
            run[0] = x.x; run[1] = x.y; run[2] = x.z; run[3] = x.w;
            run[4] = y.x; run[5] = y.y; run[6] = y.z; run[7] = y.w;
        } else {
            for (int j = 0; j < 8; ++j) run[j] = from[user + j];
        }
    }
    const int64_t tile = state_tile_bytes(p.Ns), lo_hop = (int64_t)p.H * pt * tile, hop = 2 * lo_hop;
    const int64_t lo_at = first * lo_hop + ((int64_t)h * pt + tl) * tile + (int64_t)e * 16;
    uint8_t *st_lo = static_cast<uint8_t *>(REV ? p.dstates_lo : p.states_lo);
    const bool keep_lo = st_lo != nullptr;
    st_lo += lo_at;
    const uint8_t *sf_lo = static_cast<const uint8_t *>(p.states_lo) + lo_at;
    uint8_t *st = reinterpret_cast<uint8_t *>(REV ? p.dstates : p.states) + first * hop +
                  ((int64_t)h * pt + tl) * 2 * tile + (int64_t)e * 16;
    const float *dec = p.decay + first * p.H + h;
    // reverse: the sum of E S over the warp's entries, one per chunk
    const uint8_t *sf = reinterpret_cast<const uint8_t *>(p.states) + first * hop +
                        ((int64_t)h * pt + tl) * 2 * tile + (int64_t)e * 16;
    float *es = p.es + (first * p.H + h) * per * 4 + (blockIdx.x % per) * 4 + (threadIdx.x >> 5);
    constexpr int U = 4;
    for (int k0 = 0; k0 < nc; k0 += U) {
        float4 own[U][2];
        uint4 sv[U][3];  // reverse: the states' hi, mid and lo rows
        float dk[U], es4[U] = {};
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (k0 + u < nc && live) {
                const int64_t k = REV ? nc - 1 - (k0 + u) : k0 + u;
                own[u][0] = *reinterpret_cast<const float4 *>(st + k * hop);
                own[u][1] = *reinterpret_cast<const float4 *>(st + k * hop + tile);
                if constexpr (REV) {
                    sv[u][0] = *reinterpret_cast<const uint4 *>(sf + k * hop);
                    sv[u][1] = *reinterpret_cast<const uint4 *>(sf + k * hop + tile);
                    sv[u][2] = *reinterpret_cast<const uint4 *>(sf_lo + k * lo_hop);
                }
                dk[u] = dec[k * p.H];
            }
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (k0 + u < nc && live) {
                const int64_t k = REV ? nc - 1 - (k0 + u) : k0 + u;
                if constexpr (REV) {
                    float h8[8], m8[8], l8[8];
                    load_vec<bf16, 8, true>(reinterpret_cast<const bf16 *>(&sv[u][0]), 8, h8);
                    load_vec<bf16, 8, true>(reinterpret_cast<const bf16 *>(&sv[u][1]), 8, m8);
                    load_vec<bf16, 8, true>(reinterpret_cast<const bf16 *>(&sv[u][2]), 8, l8);
#pragma unroll
                    for (int j = 0; j < 8; ++j) es4[u] = fmaf(run[j], h8[j] + (m8[j] + l8[j]), es4[u]);
                }
                uint4 hi, mid, lo;
                split3(run[0], run[1], hi.x, mid.x, lo.x);
                split3(run[2], run[3], hi.y, mid.y, lo.y);
                split3(run[4], run[5], hi.z, mid.z, lo.z);
                split3(run[6], run[7], hi.w, mid.w, lo.w);
                *reinterpret_cast<uint4 *>(st + k * hop) = hi;
                *reinterpret_cast<uint4 *>(st + k * hop + tile) = mid;
                if (keep_lo) *reinterpret_cast<uint4 *>(st_lo + k * lo_hop) = lo;
                const float f[8] = {own[u][0].x, own[u][0].y, own[u][0].z, own[u][0].w,
                                    own[u][1].x, own[u][1].y, own[u][1].z, own[u][1].w};
#pragma unroll
                for (int j = 0; j < 8; ++j) run[j] = fmaf(dk[u], run[j], f[j]);
            }
        if constexpr (REV) {  // four sums over the warp at once: lane l ends with that of chunk l % 4
            const int lane = threadIdx.x & 31;
            const bool up2 = lane & 2, up1 = lane & 1;
            const float a = (up2 ? es4[2] : es4[0]) + __shfl_xor_sync(0xffffffffu, up2 ? es4[0] : es4[2], 2);
            const float b = (up2 ? es4[3] : es4[1]) + __shfl_xor_sync(0xffffffffu, up2 ? es4[1] : es4[3], 2);
            float c = (up1 ? b : a) + __shfl_xor_sync(0xffffffffu, up1 ? a : b, 1);
#pragma unroll
            for (int o = 16; o > 2; o >>= 1) c += __shfl_xor_sync(0xffffffffu, c, o);
            if (lane < U && k0 + lane < nc) es[(int64_t)(nc - 1 - (k0 + lane)) * p.H * per * 4] = c;
        }
    }
    if (to && mine) {
        if (vec) {
            *reinterpret_cast<float4 *>(to + user) = make_float4(run[0], run[1], run[2], run[3]);
            *reinterpret_cast<float4 *>(to + user + 4) = make_float4(run[4], run[5], run[6], run[7]);
        } else {
            for (int j = 0; j < 8; ++j) to[user + j] = run[j];
        }
    }
}

// ------------------------------------------------------------------ a chunk's output
// y = M x + 2^{a_i} C S + D x with M_ij = (C_i . B_j) 2^{a_i - a_j} d_j below and on the
// diagonal.  Per chunk and group once, per unit the rest:
//   G = C B^T           both tiles K-major; stays in tensor memory (columns 0 .. 127)
//   M (columns 128 ..)  from G: each 16 columns become 8 of bf16 hi and 8 of lo pairs, which
//                       the next product reads from tensor memory as its left operand
//   E = C (S_hi, S_lo)  C from tensor memory (64 columns, once per chunk and group: read from
//                       shared memory it would be two thirds of the product's traffic there,
//                       and shared memory is what the products wait for); S MN-major
//   I = (M_hi, M_lo) x  x MN-major                         E and I: 64 columns each
// Sixteen warps bring x, two units ahead, and form M (warp w: rows 32 (w % 4) .., every fourth
// block of 16 columns); eight form y; one issues the products and the bulk copies of states
// and decays, two units ahead.  A unit's M and its product I follow one another; E of the next
// unit and y of the one before run beside them.
// Measured: 8192 rows, 64 heads of 64, 128 state rows, 79 us; 5.6 thousand cycles a unit, of
// which the products take about a third; bound by the chain G -> M -> I and by issue slots (42%
// busy, unevenly: the warps of the last rows have the most of M to form).
constexpr int kYWarps = 8, kOutThreads = kRowThreads + 32 * kYWarps + 32;
template <int NK>
struct OutSmem {
    uint8_t C[kTL * NK * 2], B[kTL * NK * 2];
    uint8_t x[4][kTL * kPT * 2];
    uint8_t S[2][2 * NK * kPT * 2];
    uint8_t y[kTL * kPT * 2];
    RowDecays dec[4];
    int bad[8][kPT], any_bad[8];   // of the last units' x: per column the first row not finite
    // A wait on a phase's parity has to happen before the next phase but one is over: a barrier
    // has as many copies as its waiters may be rounds apart.
    uint64_t full[4], x_free[4], i_done[2], e_free, m_ready, e_done, cb_ready, g_done;
    uint32_t slot_addr;
    int dead;
};

// A non-finite x_j would reach the rows before it through the zeros above M's diagonal.  Each
// thread looks at the pieces of x it loaded (rows row + 16 k of 16-byte column c8): such elements
// become zero, and the first row they occur in is noted per column; y is NaN from there on.
template <int PIECES>
__device__ __forceinline__ void drop_non_finite(uint8_t *x, int row, int c8, int *bad, int *any_bad) {
#pragma unroll
    for (int k = 0; k < PIECES; ++k) {
        const int r = row + 16 * k;
        uint32_t *w = reinterpret_cast<uint32_t *>(x + (r >> 3) * (kPT * 16) + c8 * 128 + (r & 7) * 16);
        const uint4 v = *reinterpret_cast<const uint4 *>(w);
        const uint32_t e = 0x7f807f80u;
        const uint32_t hit = __vcmpeq2(v.x & e, e) | __vcmpeq2(v.y & e, e) | __vcmpeq2(v.z & e, e) |
                             __vcmpeq2(v.w & e, e);
        if (hit) {
            for (int j = 0; j < 8; ++j)
                if (((w[j >> 1] >> (16 * (j & 1))) & 0x7f80u) == 0x7f80u) {
                    atomicMin(&bad[c8 * 8 + j], r);
                    w[j >> 1] &= j & 1 ? 0x0000ffffu : 0xffff0000u;
                }
            *any_bad = 1;
        }
    }
}

// 16 columns of M from the same of G: row i, columns 16 J ...  Pairs of columns go through the
// packed fp32 operations, two to an instruction.
__device__ __forceinline__ void m_block(const RowDecays &r, int i, int quad, int J, float ai, float li,
                                        const uint32_t (&gram)[16], uint32_t (&o)[16]) {
    if (J < 2 * quad) {
        const int e = J * kSub + kSub - 1;
        const float to_ref = ex2_ftz((ai - r.a[e]) + (li - r.lo[e]));
        const uint64_t ref2 = pack2(to_ref, to_ref);
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            const uint64_t f = *reinterpret_cast<const uint64_t *>(&r.fd[J * kSub + 2 * q]);
            split2p(mul2(pack2(gram[2 * q], gram[2 * q + 1]), mul2(ref2, f)), o[q], o[8 + q]);
        }
    } else {
        const uint64_t a2 = pack2(ai, ai), l2 = pack2(li, li);
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            const int j = J * kSub + 2 * q;
            const uint64_t a = *reinterpret_cast<const uint64_t *>(&r.a[j]);
            const uint64_t l = *reinterpret_cast<const uint64_t *>(&r.lo[j]);
            const uint64_t d = *reinterpret_cast<const uint64_t *>(&r.d[j]);
            float x, y;
            unpack2(add2(sub2(a2, a), sub2(l2, l)), x, y);
            unpack2(mul2(pack2(gram[2 * q], gram[2 * q + 1]), mul2(pack2(ex2_ftz(x), ex2_ftz(y)), d)), x, y);
            x = j <= i ? x : 0.f;  // a select: above the diagonal the exponential may overflow
            y = j + 1 <= i ? y : 0.f;
            split2(x, y, o[q], o[8 + q]);
        }
    }
}

template <bool AL, int NK>
__global__ void __launch_bounds__(kOutThreads, 1) ssm_tc_out_kernel(SsmArgs p, int y_aligned) {
    extern __shared__ __align__(1024) uint8_t raw_smem[];
    OutSmem<NK> &s = *reinterpret_cast<OutSmem<NK> *>(raw_smem);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, pt = tiles_of(p.P);
    int64_t first, last;
    work_range(slots_now(p) * p.H * pt, first, last);
    if (first >= last) {  // (the chunk table is older than the kernel before)
        follow();
        return;
    }
    const int n = (int)(last - first);
    // state rows Ns .. NK - 1 of the operand are zeros (the copies bring Ns rows)
    for (int e = tid; e < 2 * 2 * NK * kPT * 2 / 16; e += kOutThreads)
        reinterpret_cast<uint4 *>(s.S)[e] = make_uint4(0u, 0u, 0u, 0u);
    if (tid < kPT)
        for (int k = 0; k < 8; ++k) s.bad[k][tid] = kTL;
    if (tid < 8) s.any_bad[tid] = 0;
    if (tid == 0) {
        for (int k = 0; k < 4; ++k) tc::mbar_init(&s.full[k], 1);
        for (int k = 0; k < 4; ++k) tc::mbar_init(&s.x_free[k], kYWarps);
        for (int k = 0; k < 2; ++k) {
            tc::mbar_init(&s.i_done[k], 1);
        }
        tc::mbar_init(&s.e_free, kYWarps);
        tc::mbar_init(&s.m_ready, kRowWarps);
        tc::mbar_init(&s.e_done, 1);
        tc::mbar_init(&s.cb_ready, kRowWarps);
        tc::mbar_init(&s.g_done, 1);
        tc::mbar_fence_init();
        s.dead = 0;
    }
    tc::fence_async_smem();
    const uint32_t tm = tmem_open(&s.slot_addr, 512);
    follow();
    const uint32_t G = tm, M = tm + 128, E = tm + 256, I = tm + 320, CT = tm + 384;
    volatile int *dead = &s.dead;
    auto warp_arrive = [&](uint64_t *bar) {  // one arrival per warp
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(bar);
    };
    const int quad = warp & 3, i = quad * 32 + lane;

    if (warp == kRowWarps + kYWarps) {  // ------------------------------------ products and copies
        if (lane == 0) {
            const uint64_t c_desc = tc::sdesc(tc::smem_addr(s.C), 128, NK * 16);
            const uint64_t b_desc = tc::sdesc(tc::smem_addr(s.B), 128, NK * 16);
            const uint32_t id_g = tc::idesc_bf16(128, 128, false, false);
            const uint32_t id_e = tc::idesc_bf16(128, kPT, false, true);
            const int64_t tile = state_tile_bytes(p.Ns);
            int groups = 0, fetched = 0;
            auto fetch = [&](int it) {
                fetched = it + 1;
                const int64_t u = first + it;
                const uint8_t *src = reinterpret_cast<const uint8_t *>(p.states) + u * 2 * tile;
                uint64_t *bar = &s.full[it & 3];
                tc::mbar_arrive_expect_tx(bar, (uint32_t)(2 * tile + sizeof(RowDecays)));
                tc::bulk_g2s(s.S[it & 1], src, (uint32_t)tile, bar);
                tc::bulk_g2s(s.S[it & 1] + NK * kPT * 2, src + tile, (uint32_t)tile, bar);
                tc::bulk_g2s(&s.dec[it & 3], static_cast<const RowDecays *>(p.rows) + (pt == 1 ? u : u / pt),
                             sizeof(RowDecays), bar);
            };
            Walk w;
            w.start(p, first);
            int64_t at_slot = -1;
            int at_g = -1;
            auto start = [&](int it) {  // G of a new chunk or group, and E
                bool ok = true;
                if (it > 0) w.next(p, false);
                if (w.slot != at_slot || w.g != at_g) {
                    at_slot = w.slot;
                    at_g = w.g;
                    ok = wait_or_die(&s.cb_ready, groups & 1, dead, p.status);
                    ++groups;
                    tc::tc_fence_after();
                    if (ok) {
                        mma_steps(G, c_desc, 16, b_desc, 16, id_g, NK / 16, 0);
                        tc::mma_commit(&s.g_done);
                    }
                }
                ok = ok && wait_or_die(&s.full[it & 3], (it >> 2) & 1, dead, p.status);
                if (it > 0) ok = ok && wait_or_die(&s.e_free, (it - 1) & 1, dead, p.status);
                tc::tc_fence_after();
                if (ok) {
                    uint64_t sd = tc::sdesc(tc::smem_addr(s.S[it & 1]), kPT * 16, 128);
#pragma unroll 1
                    for (int k = 0; k < NK / 16; ++k) {
                        mma_bf16_ts(E, CT + 8 * k, sd, id_e, k > 0);
                        mma_bf16_ts(E, CT + 8 * k, sd + NK * kPT * 2 / 16, id_e, 1);
                        sd += 2 * kPT;
                    }
                    tc::mma_commit(&s.e_done);
                }
            };
            fetch(0);
            if (n > 1) fetch(1);
            start(0);
            for (int it = 0; it < n; ++it) {
                const bool ok = wait_or_die(&s.m_ready, it & 1, dead, p.status);
                tc::tc_fence_after();
                if (ok) {
                    uint64_t xd = tc::sdesc(tc::smem_addr(s.x[it & 3]), kPT * 16, 128);
#pragma unroll 1
                    for (int k = 0; k < kTL / 16; ++k) {
                        mma_bf16_ts(I, M + k * 16, xd, id_e, k > 0);
                        mma_bf16_ts(I, M + k * 16 + 8, xd, id_e, 1);
                        xd += 2 * kPT;
                    }
                    tc::mma_commit(&s.i_done[it & 1]);
                }
                // E has left this unit's states, and M is formed from its decays
                if (it + 2 < n && wait_or_die(&s.e_done, it & 1, dead, p.status)) fetch(it + 2);
                if (it + 1 < n) start(it + 1);
            }
            if (*dead)  // copies may still be on their way here
                for (int it = max(fetched - 2, 0); it < fetched; ++it)
                    tc::mbar_wait(&s.full[it & 3], (it >> 2) & 1, 10000000ull);
        }
        __syncwarp();
    } else if (warp < kRowWarps) {  // ---------------------------------------------- M
        const uint32_t mrow = tc::tmem_at(M, quad * 32, 0), grow = tc::tmem_at(G, quad * 32, 0);
        const int part = warp >> 2, last_J = 2 * quad + 1;
        for (int J = part; J < 8; J += 4)  // blocks above the diagonal: zero, once
            if (J > last_J) {
                const uint32_t z[16] = {};
                tmem_st16_nowait(mrow + J * kSub, z);
            }
        tmem_wait_st();
        Walk w, ahead;
        w.start(p, first);
        ahead = w;
        // pieces of x: rows x_row, x_row + 16 of the 16-byte column x_c8
        const int qt = part * 32 + lane, x_c8 = (qt >> 3) & 7, x_row = quad * 32 + (qt >> 6) * 8 + (qt & 7);
        auto load_x = [&](int it) {
            if (it > 0) ahead.next(p, true);
            const int col = ahead.tile * kPT + x_c8 * 8;
            const bf16 *src = static_cast<const bf16 *>(p.x) + (ahead.c.r0 + x_row) * p.x_stride +
                              (int64_t)ahead.h * p.P + col;
            uint8_t *dst = s.x[it & 3] + (x_row >> 3) * (kPT * 16) + x_c8 * 128 + (x_row & 7) * 16;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const bool in = col < p.P && x_row + 16 * k < ahead.c.nr;
                const bf16 *from = src + 16 * k * p.x_stride;
                if constexpr (AL) {
                    cp_async16(tc::smem_addr(dst) + 2 * k * kPT * 16, in ? from : static_cast<const bf16 *>(p.x), in);
                } else {
                    alignas(16) bf16 v[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[j] = in ? from[j] : __float2bfloat16_rn(0.f);
                    *reinterpret_cast<uint4 *>(dst + 2 * k * kPT * 16) = *reinterpret_cast<const uint4 *>(v);
                }
            }
        };
        load_x(0);
        asm volatile("cp.async.commit_group;" ::: "memory");
        if (n > 1) load_x(1);
        asm volatile("cp.async.commit_group;" ::: "memory");
        int64_t at_slot = -1;
        int at_g = -1, groups = 0;
        for (int it = 0; it < n; ++it) {
            if (it + 2 < n) {  // over unit it - 2, whose y is formed
                if (it >= 2) wait_or_die(&s.x_free[(it + 2) & 3], ((it - 2) >> 2) & 1, dead, p.status);
                load_x(it + 2);
            }
            // this unit's x is here
            asm volatile("cp.async.commit_group;\n\tcp.async.wait_group 2;" ::: "memory");
            drop_non_finite<2>(s.x[it & 3], x_row, x_c8, s.bad[it & 7], &s.any_bad[it & 7]);
            tc::fence_async_smem();
            if (it > 0) {
                w.next(p, true);
                wait_or_die(&s.i_done[(it - 1) & 1], ((it - 1) >> 1) & 1, dead, p.status);  // M is free
            }
            if (w.slot != at_slot || w.g != at_g) {  // and with it C and B
                load_rows<AL, NK, kRowThreads>(s.C, static_cast<const bf16 *>(p.Cm) + w.c.r0 * p.c_stride + w.g * p.Ns,
                                                p.c_stride, w.c.nr, p.Ns);
                load_rows<AL, NK, kRowThreads>(s.B, static_cast<const bf16 *>(p.Bm) + w.c.r0 * p.b_stride + w.g * p.Ns,
                                                p.b_stride, w.c.nr, p.Ns);
                cp_async_wait_all();
                tc::fence_async_smem();
                bar_sync(5, kRowThreads);
                if (part < NK / 32) {  // 32 columns of C's rows, in pairs
                    alignas(16) uint32_t o[16];
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        *reinterpret_cast<uint4 *>(&o[4 * q]) = *reinterpret_cast<const uint4 *>(
                            s.C + (i >> 3) * (NK * 16) + (part * 4 + q) * 128 + (i & 7) * 16);
                    tmem_st16_nowait(tc::tmem_at(CT, quad * 32, part * 16), o);
                    tmem_wait_st();
                    tc::tc_fence_before();
                }
                warp_arrive(&s.cb_ready);
                at_slot = w.slot;
                at_g = w.g;
                wait_or_die(&s.g_done, groups & 1, dead, p.status);
                ++groups;
            }
            wait_or_die(&s.full[it & 3], (it >> 2) & 1, dead, p.status);
            tc::tc_fence_after();
            const RowDecays &r = s.dec[it & 3];
            const float ai = r.a[i], li = r.lo[i];
#pragma unroll 1
            for (int J = part; J <= last_J; J += 4) {
                uint32_t v[16], o[16];
                tmem_ld16_nowait(grow + J * kSub, v);
                tmem_wait_ld();
                m_block(r, i, quad, J, ai, li, v, o);
                tmem_st16_nowait(mrow + J * kSub, o);
            }
            tmem_wait_st();
            tc::tc_fence_before();
            warp_arrive(&s.m_ready);
        }
    } else {  // --------------------------------------------------------------------- y
        Walk w;
        w.start(p, first);
        const int half = (warp >> 2) & 1, qt = half * 32 + lane, yt = tid - kRowThreads;
        for (int it = 0; it < n; ++it) {
            if (it > 0) w.next(p, true);
            wait_or_die(&s.full[it & 3], (it >> 2) & 1, dead, p.status);
            const float ea = ex2_ftz(s.dec[it & 3].a[i]), D = p.D ? p.D[w.h] : 0.f;
            const uint64_t ea2 = pack2(ea, ea), D2 = pack2(D, D);
            wait_or_die(&s.i_done[it & 1], (it >> 1) & 1, dead, p.status);
            tc::tc_fence_after();
            const uint8_t *x = s.x[it & 3] + (i >> 3) * (kPT * 16) + (i & 7) * 16;
            const bool any_bad = s.any_bad[it & 7] != 0;
            const uint32_t at = tc::tmem_at(E, quad * 32, half * 32);
#pragma unroll 1
            for (int k = 0; k < 2; ++k) {
                uint32_t e[16], u[16];
                tmem_ld16_nowait(at + k * 16, e);
                tmem_ld16_nowait(at + 64 + k * 16, u);
                tmem_wait_ld();
                if (k == 1) {
                    tc::tc_fence_before();
                    warp_arrive(&s.e_free);
                }
                const int c16 = half * 4 + k * 2;  // 16-byte columns c16, c16 + 1
                if (any_bad) {
#pragma unroll
                    for (int q = 0; q < 16; ++q)
                        if (i >= s.bad[it & 7][c16 * 8 + q]) u[q] = 0x7fffffffu;
                }
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const uint4 xv = *reinterpret_cast<const uint4 *>(x + (c16 + q) * 128);
                    const uint32_t xw[4] = {xv.x, xv.y, xv.z, xv.w};
                    uint32_t o[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int at = 8 * q + 2 * j;
                        uint64_t f = fma2(ea2, pack2(e[at], e[at + 1]), pack2(u[at], u[at + 1]));
                        if (p.D) f = fma2(D2, pack2(xw[j] << 16, xw[j] & 0xffff0000u), f);
                        float lo, hi;
                        unpack2(f, lo, hi);
                        o[j] = pack_bf16(lo, hi);
                    }
                    // 16-byte pieces of a 128-byte row, moved by the row against conflicts
                    *reinterpret_cast<uint4 *>(s.y + i * 128 + (((c16 + q) ^ (i & 7)) << 4)) =
                        make_uint4(o[0], o[1], o[2], o[3]);
                }
            }
            warp_arrive(&s.x_free[it & 3]);
            bar_sync(1 + quad, 64);
            const int c8 = qt & 7, pcols = min(kPT, p.P - w.tile * kPT);
            bf16 *y = static_cast<bf16 *>(p.y) + (w.c.r0 * p.H + w.h) * p.P + w.tile * kPT + c8 * 8;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int r = quad * 32 + (qt >> 3) + 8 * k;
                const uint4 v = *reinterpret_cast<const uint4 *>(s.y + r * 128 + ((c8 ^ (r & 7)) << 4));
                if (r < w.c.nr && c8 * 8 < pcols) {
                    bf16 *dst = y + (int64_t)r * p.H * p.P;
                    if (y_aligned) {
                        *reinterpret_cast<uint4 *>(dst) = v;
                    } else {
                        const bf16 *b8 = reinterpret_cast<const bf16 *>(&v);
#pragma unroll
                        for (int j = 0; j < 8; ++j) dst[j] = b8[j];
                    }
                }
            }
            bar_sync(1 + quad, 64);  // the quad's rows of s.y are free
            // marks for a unit five ahead, over those of a unit three back: no warp is that far off
            if (yt < kPT) s.bad[(it + 5) & 7][yt] = kTL;
            if (yt == 0) s.any_bad[(it + 5) & 7] = 0;
        }
    }
    tmem_close(tm, 512);
}

template <int MT>
constexpr size_t state_smem() { return sizeof(StateSmem<MT>); }
template <int NK>
constexpr size_t out_smem() {
    return sizeof(OutSmem<NK>) > 120 * 1024 ? sizeof(OutSmem<NK>) : 120 * 1024;  // one CTA per SM
}

template <typename K>
cudaError_t allow(K kernel, size_t bytes) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
}
template <bool AL, int NK>
cudaError_t allow_kernels() {
    cudaError_t e = allow(ssm_tc_out_kernel<AL, NK>, out_smem<NK>());
    if (NK >= 64) {
        constexpr int MT = NK >= 64 ? NK : 64;
        if (e == cudaSuccess) e = allow(ssm_tc_state_kernel<AL, false, MT>, state_smem<MT>());
        if (e == cudaSuccess) e = allow(ssm_tc_state_kernel<AL, true, MT>, state_smem<MT>());
    }
    return e;
}
int g_sms[64];
cudaError_t tc_setup(int *sms) {
    static DeviceOnce once;
    int dev = 0;
    const cudaError_t err = once.run(&dev, [](int d) {
        cudaError_t e = cudaDeviceGetAttribute(&g_sms[d], cudaDevAttrMultiProcessorCount, d);
        if (e == cudaSuccess) e = allow_kernels<true, 32>();
        if (e == cudaSuccess) e = allow_kernels<false, 32>();
        if (e == cudaSuccess) e = allow_kernels<true, 64>();
        if (e == cudaSuccess) e = allow_kernels<false, 64>();
        if (e == cudaSuccess) e = allow_kernels<true, 128>();
        if (e == cudaSuccess) e = allow_kernels<false, 128>();
        return e;
    });
    if (err == cudaSuccess) *sms = g_sms[dev];
    return err;
}

// Whether every row of the inputs starts on a 16-byte boundary.
bool tc_aligned(const SsmArgs &a) {
    return aligned_to(a.x, 16) && aligned_to(a.Bm, 16) && aligned_to(a.Cm, 16) && a.x_stride % 8 == 0 &&
           a.b_stride % 8 == 0 && a.c_stride % 8 == 0;
}

// f(aligned, padded state rows): 32, 64 or 128, so that indices are shifts.  8192 rows, 32 heads
// of 64, forward and gradients: 16 state rows 287 us (321 padded to 128), 64 state rows 315
// (342); rows of x, B and C that are not aligned for 16-byte copies, 440 us against 387.
template <typename F>
void by_tile(bool al, int Ns, F &&f) {
    using std::integral_constant;
    auto rows = [&](auto AL) {
        if (Ns <= 32)
            f(AL, integral_constant<int, 32>());
        else if (Ns <= 64)
            f(AL, integral_constant<int, 64>());
        else
            f(AL, integral_constant<int, 128>());
    };
    if (al)
        rows(integral_constant<bool, true>());
    else
        rows(integral_constant<bool, false>());
}

}  // namespace

bool ssm_tc_supported(kda_dtype dt, int Ns, int P) {
    return dt == KDA_DTYPE_BF16 && Ns % 8 == 0 && Ns <= 128 && P % 8 == 0;
}

template <bool BWD>
static cudaError_t tc_states(const SsmArgs &a, cudaStream_t st) {
    int sms = 0;
    cudaError_t e = tc_setup(&sms);
    if (e != cudaSuccess) return e;
    const int64_t pairs = a.slots * a.G * (((int64_t)a.H / a.G * tiles_of(a.P) + 1) / 2);
    const int64_t blocks = pairs < sms ? pairs : sms;
    const int64_t row_blocks = a.slots * ((a.H + kRowHeads - 1) / kRowHeads);
    if (row_blocks > INT32_MAX) return cudaErrorInvalidValue;
    if (pairs > 0 && !BWD) {
        prof_begin("ssm_tc_rows", st);
        ssm_tc_rows_kernel<<<(unsigned)row_blocks, 32 * kRowHeads, 0, st>>>(a);
        prof_end(st);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
    }
    if (pairs > 0) {
        const bool al = tc_aligned(a) && (!BWD || aligned_to(a.dy, 16));
        prof_begin(BWD ? "ssm_tc_dstate" : "ssm_tc_state", st);
        by_tile(al, a.Ns, [&](auto AL, auto NK) {
            constexpr int MT = NK() >= 64 ? NK() : 64;
            if constexpr (BWD) {  // the backward's first kernel
                ssm_tc_state_kernel<AL(), BWD, MT><<<(unsigned)blocks, kTcThreads, state_smem<MT>(), st>>>(a);
                e = cudaGetLastError();
            } else {
                e = launch_after(ssm_tc_state_kernel<AL(), BWD, MT>, blocks, kTcThreads, state_smem<MT>(), st, a);
            }
        });
        prof_end(st);
        if (e != cudaSuccess) return e;
    }
    const int64_t groups = (int64_t)tiles_of(a.P) * a.Ns * 8;
    const int64_t pass = (int64_t)a.N * a.H * ((groups + 127) / 128);
    if (pass > INT32_MAX) return cudaErrorInvalidValue;
    if (pass > 0) {
        const int vec = aligned_to(BWD ? a.dht : a.h0, 16) && aligned_to(BWD ? a.dh0 : a.ht, 16);
        prof_begin(BWD ? "ssm_tc_dpass" : "ssm_tc_pass", st);
        // (plainly: blocks this small, let in early, crowd on the SMs that are free first)
        ssm_tc_pass_kernel<BWD><<<(unsigned)pass, 128, 0, st>>>(a, vec);
        e = cudaGetLastError();
        prof_end(st);
    }
    return e;
}

cudaError_t launch_ssm_tc_states(const SsmArgs &a, cudaStream_t st) { return tc_states<false>(a, st); }
cudaError_t launch_ssm_tc_dstates(const SsmArgs &a, cudaStream_t st) { return tc_states<true>(a, st); }

cudaError_t launch_ssm_tc_out(const SsmArgs &a, cudaStream_t st) {
    int sms = 0;
    cudaError_t e = tc_setup(&sms);
    if (e != cudaSuccess) return e;
    const int64_t units = a.slots * a.H * tiles_of(a.P), blocks = units < sms ? units : sms;
    if (units == 0) return cudaSuccess;
    prof_begin("ssm_tc_out", st);
    by_tile(tc_aligned(a), a.Ns, [&](auto AL, auto NK) {
        e = launch_after(ssm_tc_out_kernel<AL(), NK()>, blocks, kOutThreads, out_smem<NK()>(), st, a,
                         aligned_to(a.y, 16));
    });
    prof_end(st);
    return e;
}

size_t ssm_state_bytes(kda_dtype dt, int Ns, int P) {
    return ssm_tc_supported(dt, Ns, P) ? (size_t)(tiles_of(P) * 2 * state_tile_bytes(Ns))
                                       : (size_t)Ns * P * 4;
}
size_t ssm_state_lo_bytes(kda_dtype dt, int Ns, int P) {
    return ssm_tc_supported(dt, Ns, P) ? (size_t)(tiles_of(P) * state_tile_bytes(Ns)) : 0;
}
size_t ssm_rows_bytes(kda_dtype dt, int Ns, int P) {
    return ssm_tc_supported(dt, Ns, P) ? sizeof(RowDecays) : 0;
}

}  // namespace kda
