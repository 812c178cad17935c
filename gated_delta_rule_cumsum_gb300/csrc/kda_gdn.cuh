// kda_gdn.cuh -- the gated delta rule with one decay per head: argument structs, launchers
// and what its kernels share.  Not part of the public ABI.
//
// Per sequence and value head, S an fp32 [K, V] state, g a base-2 log decay:
//     S_t = 2^{g_t} S_{t-1} + beta_t k_t (v_t - (2^{g_t} S_{t-1})^T k_t)^T,   o_t = S_t^T q_t
// (q with the readout scale).  In chunks of L rows, with a the inclusive cumulative sum of g from
// the chunk's start, c = 2^a, e = 2^{a_end - a}, G_ij = 2^{a_i - a_j} for i >= j:
//     A = (K K^T . G) below the diagonal, M = (I + diag(beta) A)^-1, P = (Q K^T . G) on and below it
//     U = M diag(beta) (V - diag(c) K S),  O = diag(c) Q S + P U,  S' = 2^{a_end} S + K^T diag(e) U
// and, for dO and E = dL/dS',
//     dU = P^T dO + diag(e) K E,  Z = M^T dU,  dV = diag(beta) Z
//     dS = 2^{a_end} E + Q^T diag(c) dO - K^T diag(c beta) Z
//     X = dO U^T . G, Y = -diag(beta) (Z U^T . G) below the diagonal
//     dQ = X K + diag(c) dO S^T,  dK = X^T Q + (Y + Y^T) K - diag(c beta) Z S^T + diag(e) U E^T
//     dbeta_i = Z_i . v_i - c_i Z_i . S^T k_i - sum_j A_ij (Z U^T)_ij
//     dg_t = sum_{i >= t > j} (X . Q K^T + Y . K K^T)_ij + sum_{i >= t} (c_i q_i . S dO_i - c_i beta_i
//            k_i . S Z_i) + sum_{j < t} e_j k_j . E U_j + 2^{a_end} <S, E>     (natural units)
// The last line sums over the pairs that a decay lies between: as a running difference of row and
// column sums it would keep the rounding of far pairs, which cancel.
#pragma once

#include "kda_ssm_tc.cuh"

namespace kda {

struct GdnArgs {
    const void *q, *k, *v;         // [B, T, H, K] twice, [B, T, HV, V]: rows *_stride apart
    const float *g;                // [B, T, HV]
    const void *beta;              // [B, T, HV]
    const float *h0;               // [N, HV, K, V] or null
    const int32_t *cu;
    void *o;
    float *ht;
    int32_t *status;
    int64_t q_stride, k_stride, v_stride;
    int B, T, H, HV, K, V, N, l2;
    int give_up;                   // KDA_GDN_FLAG_TEST_WAIT_TIMEOUT: waits for copies run out at once
    float scale, g_scale;
    int L;                         // chunk length
    int c0, c1;                    // a launch's chunks within every (dense) sequence; c1 == 0: all
    // workspace
    ChunkCtrl *ctrl;
    int32_t *chunk_start;          // [N + 1] (packed only)
    int64_t slots;
    float *norms;                  // [B T][H][2]: 1 / |q|, 1 / |k| (with the norm only)
    float *rows;                   // per (slot, value head): GdnRows
    // CUDA-core path, fp32, per unit: M, A, P ([L][L] each); W and diag(e rk) K ([L][K up to a multiple
    // of 4] each); per 32 value columns, the state at the chunk's start ([K][32]) and U ([L][32])
    float *mats, *wk, *states, *us;
    // tensor-core path, per unit (kda_gdn_tc.cuh; a tile is 32 KB, two parts two tiles): M (null: not
    // kept), W, the state at the chunk's start, U; U0 in fp32; and per (slot, head) K
    uint8_t *mt, *wt, *st, *ut, *kt;
    float *u0;
    float *carry;                  // [N][HV][K][V]: the state between two launches of a pass
    // backward
    const void *dout;              // [B, T, HV, V]
    const float *dht;
    void *dq, *dk, *dv, *dbeta;    // the inputs' layouts, contiguous, in their type
    float *dg, *dh0;
    float *dstates, *zs;           // CUDA-core path, as states and us: B0, then E; dU, then Z
    uint8_t *et, *dut;             // tensor-core path: E, dU
    float *du0, *b0;               // P^T dO and Q^T diag(c) dO, in fp32
    float *dcarry;                 // as carry, of the reverse pass
    float *dqh, *dkh;              // [B T][HV][K]: each value head's share of dq, dk
};
int gdn_chunk_len(kda_dtype dt, int K, int V);
bool gdn_tc_supported(kda_dtype dt, int K, int V);
constexpr size_t kGdnTile = 128 * 128 * 2;  // bytes of a tensor-core path's tile
// Floats per (slot, value head) of the arrays above.
size_t gdn_rows_floats(int L);
size_t gdn_mats_floats(int L);
size_t gdn_wk_floats(int L, int K);
size_t gdn_u_floats(int L, int V);
size_t gdn_state_floats(int K, int V);

cudaError_t launch_gdn_fwd(const GdnArgs &a, kda_dtype dt, cudaStream_t st);
cudaError_t launch_gdn_bwd(const GdnArgs &a, kda_dtype dt, bool states_kept, cudaStream_t st);

struct GdnStepArgs {
    const void *q, *k, *v;
    const float *g;
    const void *beta;
    float *state;                  // [slots, HV, K, V], updated in place
    const int32_t *idx;
    void *o;
    int32_t *status;
    int64_t q_stride, k_stride, v_stride;
    int N, slots, H, HV, K, V, l2;
    float scale, g_scale;
};
cudaError_t launch_gdn_step(const GdnStepArgs &a, kda_dtype dt, cudaStream_t st);

namespace {

// What the chunk kernels know of a chunk's rows, per (slot, value head): L floats each of a and
// lo (the cumulative log2 decay as a pair of floats: under strong decay it runs to thousands while
// the differences that count are small), c = 2^a, e = 2^{a_end - a}, beta, and the factors rq and
// rk that q's and k's rows are multiplied by (the norms' reciprocals, rq with the readout scale).
// Keeping the norm a factor of the row leaves the products' operands the exact inputs.  fd = rk 2^{ref -
// a}, ref the decay at the last row of the row's block of 16: for a row i past j's block, 2^{a_i -
// a_j} rk_j = 2^{a_i - ref} fd_j, one exponential per row and block in place of one per element, and
// both factors' exponents are <= 0.  Rows past the chunk's end: a stays, e = 1, beta = rq = rk = 0.
constexpr int kGdnRowArrays = 8;
struct GdnRows {
    const float *a, *lo, *c, *e, *b, *rq, *rk, *fd;
    float *at;
    __device__ __forceinline__ GdnRows(const GdnArgs &p, int64_t unit) : GdnRows(p.rows + unit * kGdnRowArrays * p.L, p.L) {}
    __device__ __forceinline__ GdnRows(float *from, int L) {
        at = from;
        a = at; lo = at + L; c = at + 2 * L; e = at + 3 * L;
        b = at + 4 * L; rq = at + 5 * L; rk = at + 6 * L; fd = at + 7 * L;
    }
};

struct GdnChunk {
    int64_t r0;  // first row
    int nr;      // rows
};
__device__ __forceinline__ bool gdn_find_chunk(const GdnArgs &p, int slot, GdnChunk &c) {
    if (p.cu) {
        if (!p.ctrl->valid || slot >= p.ctrl->total_chunks) return false;
        const int n = upper_bound_minus_one(p.chunk_start, p.N + 1, slot);
        const int s = p.cu[n] + p.L * (slot - p.chunk_start[n]);
        c.r0 = s;
        c.nr = min(p.L, p.cu[n + 1] - s);
    } else {
        const int per = (p.T + p.L - 1) / p.L;
        const int seq = slot / per, k = slot % per;
        c.r0 = (int64_t)seq * p.T + (int64_t)k * p.L;
        c.nr = min(p.L, p.T - k * p.L);
    }
    return c.nr > 0;
}
// A wait for copies (see wait_or_die): at its block's end a dead block waits for those it asked for, 10 ms
// at most, so that they do not land in the shared memory of the block that comes next.
__device__ __forceinline__ bool copies_or_die(const GdnArgs &p, uint64_t *bar, uint32_t parity, volatile int *dead) {
    if (!p.give_up) return wait_or_die(bar, parity, dead, p.status);
    *dead = 1;
    report(p.status, KDA_DEVICE_TIMEOUT);
    return false;
}
// The chunk slot and value head of a launch's unit; slots * HV fits 31 bits.
__device__ __forceinline__ void gdn_unit(const GdnArgs &p, int id, int &slot, int &hv) {
    hv = id % p.HV;
    slot = id / p.HV;
    if (p.c1 > 0) {
        const int per = p.c1 - p.c0;
        slot = slot / per * ((p.T + p.L - 1) / p.L) + p.c0 + slot % per;
    }
}
// A sequence's first chunk slot, its chunks and its first row; false: offsets that are not valid.
__device__ __forceinline__ bool gdn_sequence(const GdnArgs &p, int seq, int64_t &first, int &nc, int64_t &row,
                                             int &len) {
    if (p.cu) {
        if (!p.ctrl->valid) return false;
        first = p.chunk_start[seq];
        nc = p.chunk_start[seq + 1] - p.chunk_start[seq];
        row = p.cu[seq];
        len = p.cu[seq + 1] - p.cu[seq];
    } else {
        nc = (p.T + p.L - 1) / p.L;
        first = (int64_t)seq * nc;
        row = (int64_t)seq * p.T;
        len = p.T;
    }
    return true;
}

}  // namespace
}  // namespace kda
