// kda_block.cuh -- the recurrent block's operators beside KDA itself (short causal
// convolution, selective state-space scan, residual RMS norm): their argument structs
// and launchers, and small helpers they share.  Not part of the public ABI.
#pragma once

#include "kda_internal.cuh"

namespace kda {

// The SMs of a GB300.  A constant where a split of the work depends on it: sizes of workspaces follow
// from some of these splits, and they are asked for without a device.  (Other counts would cost
// time, not correctness.)
constexpr int kSms = 152;

// ------------------------------------------------------------ short convolution
struct ConvArgs {
    const void *x, *state_in;      // [B, T, C] rows x_stride apart; [N, W-1, C]
    const float *w, *bias;         // [C, W]; [C] or null
    const int32_t *cu;
    void *y, *state_out;           // forward outputs
    const void *dy, *dstate_out;   // backward
    void *dx, *dstate_in;
    float *dw, *dbias;
    float *part;                   // backward: [parts][W + 1][C] partial sums of dw and dbias
    int32_t *status;
    int64_t x_stride;
    int B, T, C, W, N, silu;
    int strip;                     // rows a thread walks
    int64_t strips;                // over all B * T rows
};
// Rows per strip of the backward (its workspace holds one row of sums per strip).
int conv_bwd_strip(int B, int T, int C);
cudaError_t launch_conv_fwd(ConvArgs a, kda_dtype dt, cudaStream_t st);
cudaError_t launch_conv_bwd(ConvArgs a, kda_dtype dt, cudaStream_t st);

struct ConvStepArgs {
    const void *x;
    const float *w, *bias;
    void *state;                   // [slots, W-1, C], updated in place
    const int32_t *idx;            // [N] or null
    void *y;
    int32_t *status;
    int64_t x_stride;
    int N, slots, C, W, silu;
};
cudaError_t launch_conv_step(const ConvStepArgs &a, kda_dtype dt, cudaStream_t st);

// ------------------------------------------------------------------------- norm
struct NormArgs {
    const void *x, *res;           // [rows, cols]; res may be null
    const float *w;
    void *h, *y;                   // h may be null (not stored)
    float *scale;                  // 8-bit outputs: [rows, groups]
    int64_t rows;
    int cols, group, out;          // group: columns per scale (0: the row); out: kda_norm_out
    float eps;
    // backward
    const void *dy, *dres;
    void *dx;
    float *dw, *part;
};
int64_t norm_bwd_parts(int64_t rows, int cols, kda_dtype dt);
cudaError_t launch_norm_fwd(const NormArgs &a, kda_dtype dt, cudaStream_t st);
cudaError_t launch_norm_bwd(const NormArgs &a, kda_dtype dt, cudaStream_t st);

// ------------------------------------------------------------------------- scan
struct SsmArgs {
    const void *x, *dt, *Bm, *Cm;  // rows x_stride, dt_stride, b_stride, c_stride apart
    const float *A_log, *D, *dt_bias, *h0;
    const int32_t *cu;
    void *y;
    float *ht;
    int32_t *status;
    int64_t x_stride, dt_stride, b_stride, c_stride;
    int B, T, H, G, Ns, P, N, softplus;  // Ns: state rows, N: sequences
    int L;                               // chunk length
    // workspace
    ChunkCtrl *ctrl;
    int32_t *chunk_start;          // [N + 1] (packed only)
    int64_t slots;
    float *states;                 // per (slot, head) ssm_state_bytes: the state at each chunk's
                                   // start ([Ns][P] fp32, or the tensor-core path's tiles)
    void *states_lo;               // tensor-core path: the third tile of each state, for the
                                   // backward (null: not wanted)
    void *rows;                    // per (slot, head) ssm_rows_bytes: the rows' decays
    float *decay;                  // [slots][H]: each chunk's decay from start to end
    // backward
    const void *dy;
    const float *dht;
    void *dx, *ddt, *dB, *dC;
    float *dA_log, *dD, *ddt_bias, *dh0;
    float *dstates;                // the state gradient at each chunk's end, as states
    void *dstates_lo;
    // fp32 path: the heads' shares of dB and dC ([rows][H][Ns]); tensor-core path: those of the
    // parts a group's heads are split in ([slots][G][parts][128][Ns])
    float *dBh, *dCh;
    int parts;
    float *sums;                   // [slots][3][H]: the chunks' shares of dA_log, dD, ddt_bias
    // tensor-core path, per (slot, head, 64-column tile): what the rows' decay gradients are
    // made of (4 x 128), and dD; per (slot, head) the shares of <E, S>
    float *rowg, *dDp, *es;
};
int ssm_chunk_len(kda_dtype dt, int Ns, int P);
cudaError_t launch_ssm_fwd(const SsmArgs &a, kda_dtype dt, cudaStream_t st);
// The chunk states alone (the first part of the forward).
cudaError_t launch_ssm_states(const SsmArgs &a, kda_dtype dt, cudaStream_t st);
cudaError_t launch_ssm_bwd(const SsmArgs &a, kda_dtype dt, cudaStream_t st);
// The tensor-core path (kda_ssm_tc.cu): bf16, Ns a multiple of 8 up to 128, P of 8.
bool ssm_tc_supported(kda_dtype dt, int Ns, int P);
size_t ssm_state_bytes(kda_dtype dt, int Ns, int P);
size_t ssm_state_lo_bytes(kda_dtype dt, int Ns, int P);
size_t ssm_rows_bytes(kda_dtype dt, int Ns, int P);
cudaError_t launch_ssm_tc_states(const SsmArgs &a, cudaStream_t st);
cudaError_t launch_ssm_tc_dstates(const SsmArgs &a, cudaStream_t st);
cudaError_t launch_ssm_tc_out(const SsmArgs &a, cudaStream_t st);
cudaError_t launch_ssm_tc_bwd(const SsmArgs &a, cudaStream_t st);
// The parts a group's units are split in for dB and dC; the bytes of the arrays above.
int ssm_tc_parts(int64_t slots, int G, int units);
int ssm_tc_tiles(int P);
size_t ssm_tc_es_floats(int Ns, int P);

struct SsmStepArgs {
    const void *x, *dt, *Bm, *Cm;
    const float *A_log, *D, *dt_bias;
    float *state;                  // [slots, H, Ns, P], updated in place
    const int32_t *idx;
    void *y;
    int32_t *status;
    int64_t x_stride, dt_stride, b_stride, c_stride;
    int N, slots, H, G, Ns, P, softplus;
};
cudaError_t launch_ssm_step(const SsmStepArgs &a, kda_dtype dt, cudaStream_t st);

// ---------------------------------------------------------------------- launches
// The kernels of one call follow each other through the workspace.  A later one may be launched
// with its start allowed while the one before still runs: its blocks take their places as the
// others leave theirs, and wait in follow() until all of those are through.  Every block of a
// kernel that takes part comes to follow(), before it touches what a kernel of the same call
// wrote (but the chunk table, which is older than the kernel before) and before it returns, so that a
// kernel's end is also that of all before it.  The first kernel of a call is launched plainly and
// waits for whatever the stream holds.  Scan, 8192 rows, 32 heads of 64, 128 state rows: a training
// pass of 11 launches went from 421 to 404 us with it (388 now, by later steps); with the passes over
// chunks let in early as well it was 455, since small blocks crowd on the SMs that are free first.  The CUDA-core
// kernels are launched plainly too (one row of 32 heads, fp32: forward 32 us, 49 let in early).
__device__ __forceinline__ void follow() {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
}
// launch_next: `first` where no kernel of the call has been launched before.
template <typename... P, typename... A>
cudaError_t launch_next(bool first, void (*kernel)(P...), int64_t blocks, unsigned threads, size_t smem, cudaStream_t st,
                        A... args) {
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = &attr;
    cfg.numAttrs = first ? 0 : 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
    if (e != cudaSuccess) cudaGetLastError();  // reported by the return value alone
    return e;
}
template <typename... P, typename... A>
cudaError_t launch_after(void (*kernel)(P...), int64_t blocks, unsigned threads, size_t smem, cudaStream_t st, A... args) {
    return launch_next(false, kernel, blocks, threads, smem, st, args...);
}

// ---------------------------------------------------------------------- helpers
// Two fp32 values in a register pair, and the packed operations on them.
__device__ __forceinline__ uint64_t pack2(uint32_t x, uint32_t y) { return (uint64_t)y << 32 | x; }
__device__ __forceinline__ uint64_t pack2(float x, float y) {
    return pack2(__float_as_uint(x), __float_as_uint(y));
}
__device__ __forceinline__ void unpack2(uint64_t v, float &x, float &y) {
    x = __uint_as_float((uint32_t)v);
    y = __uint_as_float((uint32_t)(v >> 32));
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t sub2(uint64_t a, uint64_t b) {
    return fma2(b, 0xbf800000bf800000ull, a);  // a - b: exact products by -1, one rounding
}

// VEC consecutive elements as fp32: one vector load when the address is aligned for it
// (ALIGNED), else scalar loads of the first `n`, zeros after.
template <typename T, int VEC, bool ALIGNED>
__device__ __forceinline__ void load_vec(const T *p, int n, float (&v)[VEC]) {
    if constexpr (ALIGNED) {
        if constexpr (sizeof(T) == 4) {
            static_assert(VEC == 4, "fp32 vectors of four");
            const float4 f = *reinterpret_cast<const float4 *>(p);
            v[0] = f.x; v[1] = f.y; v[2] = f.z; v[3] = f.w;
        } else if constexpr (VEC == 8) {
            const uint4 u = *reinterpret_cast<const uint4 *>(p);
            const __nv_bfloat162 *h = reinterpret_cast<const __nv_bfloat162 *>(&u);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 f = __bfloat1622float2(h[i]);
                v[2 * i] = f.x;
                v[2 * i + 1] = f.y;
            }
        } else {
            static_assert(VEC == 4, "bf16 vectors of four or eight");
            const uint2 u = *reinterpret_cast<const uint2 *>(p);
            const __nv_bfloat162 *h = reinterpret_cast<const __nv_bfloat162 *>(&u);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float2 f = __bfloat1622float2(h[i]);
                v[2 * i] = f.x;
                v[2 * i + 1] = f.y;
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i) v[i] = i < n ? to_f32(p[i]) : 0.f;
    }
}

template <typename T, int VEC, bool ALIGNED>
__device__ __forceinline__ void store_vec(T *p, int n, const float (&v)[VEC]) {
    if constexpr (ALIGNED) {
        if constexpr (sizeof(T) == 4) {
            *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
        } else {
            alignas(2 * VEC) __nv_bfloat162 h[VEC / 2];
#pragma unroll
            for (int i = 0; i < VEC / 2; ++i) h[i] = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
            if constexpr (VEC == 8)
                *reinterpret_cast<uint4 *>(p) = *reinterpret_cast<const uint4 *>(h);
            else
                *reinterpret_cast<uint2 *>(p) = *reinterpret_cast<const uint2 *>(h);
        }
    } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i)
            if (i < n) p[i] = from_f32<T>(v[i]);
    }
}

inline bool aligned_to(const void *p, size_t a) { return (uintptr_t)p % a == 0; }

// The packed-offset checks of every call, by the threads of one block: the work itself
// clamps what it reads from the offsets, so bad ones cannot lead out of bounds.
__device__ __forceinline__ void check_offsets(const int32_t *cu, int N, int T, int32_t *status) {
    bool ok = true;
    for (int n = threadIdx.x; n < N; n += blockDim.x)
        ok = ok && cu[n] >= 0 && cu[n] <= cu[n + 1] && cu[n + 1] <= T;
    if (threadIdx.x == 0) ok = ok && cu[0] == 0 && cu[N] >= 0 && cu[N] <= T;
    if (!ok) report(status, KDA_DEVICE_BAD_CU_SEQLENS);
}

// The state slot of a batch row: its index, or the row itself without an index table.
// Negative entries are unused rows; entries past the last slot are reported.  -1: skip.
__device__ __forceinline__ int state_slot(const int32_t *idx, int n, int slots, int32_t *status) {
    const int s = idx ? idx[n] : n;
    if (s >= slots) {
        if (threadIdx.x == 0) report(status, KDA_DEVICE_BAD_INDEX);
        return -1;
    }
    return s < 0 ? -1 : s;
}

}  // namespace kda
