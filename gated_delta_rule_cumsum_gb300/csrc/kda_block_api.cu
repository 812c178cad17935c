// kda_block_api.cu -- the extern "C" entry points of the recurrent block's operators
// (short convolution, state-space scan, residual RMS norm): host-side argument checks,
// workspace carving and launches.
#include <climits>
#include <cmath>
#include <cstdarg>
#include <cstdio>

#include "kda_block.cuh"

namespace kda {
void set_last_error(const char *msg);
}

namespace {

kda_status fail(kda_status st, const char *fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof(buf), fmt, ap);
    va_end(ap);
    kda::set_last_error(buf);
    return st;
}

kda_status done(cudaError_t e, const char *op) {
    if (e != cudaSuccess)
        return fail(KDA_ERR_CUDA, "%s: %s (%s)", op, cudaGetErrorName(e), cudaGetErrorString(e));
    kda::set_last_error("");
    return KDA_OK;
}

cudaStream_t to_stream(kda_stream_t s) { return reinterpret_cast<cudaStream_t>(s); }

kda_status check_dtype(const char *op, int dt) {
    if (dt != KDA_DTYPE_F32 && dt != KDA_DTYPE_BF16)
        return fail(KDA_ERR_INVALID_ARG, "%s: unknown dtype %d", op, dt);
    return KDA_OK;
}

// All rows of a call, and those rows rounded up to whole chunks, are counted in 32 bits.
bool rows_ok(int B, int T) { return (int64_t)B * T <= INT_MAX - 255; }

// The batch of a conv or scan shape: dense (num_seqs == B) or packed (B == 1).
kda_status check_batch(const char *op, int B, int T, int num_seqs, const int32_t *cu) {
    if (B <= 0 || T < 0) return fail(KDA_ERR_INVALID_ARG, "%s: B=%d T=%d", op, B, T);
    if (cu) {
        if (B != 1)
            return fail(KDA_ERR_INVALID_ARG, "%s: packed sequences (cu_seqlens) need B == 1, got %d",
                        op, B);
        if (num_seqs < 0) return fail(KDA_ERR_INVALID_ARG, "%s: num_seqs=%d < 0", op, num_seqs);
    } else if (num_seqs != B) {
        return fail(KDA_ERR_INVALID_ARG, "%s: num_seqs=%d must equal B=%d without cu_seqlens", op,
                    num_seqs, B);
    }
    if (!rows_ok(B, T)) return fail(KDA_ERR_UNSUPPORTED, "%s: too many rows", op);
    return KDA_OK;
}

kda_status check_workspace(const char *op, const void *ws, size_t have, size_t need, size_t align) {
    if (need > 0 && (!ws || have < need))
        return fail(KDA_ERR_INVALID_ARG, "%s: workspace of %zu bytes needed, %zu given", op, need, have);
    if ((uintptr_t)ws % align != 0)
        return fail(KDA_ERR_INVALID_ARG, "%s: workspace must be %zu-byte aligned", op, align);
    return KDA_OK;
}

kda_status check_stride(const char *op, const char *name, int64_t given, int64_t cols, int64_t *out) {
    *out = given == 0 ? cols : given;
    if (*out < cols)
        return fail(KDA_ERR_INVALID_ARG, "%s: %s=%lld is less than a row's %lld elements", op, name,
                    (long long)given, (long long)cols);
    return KDA_OK;
}

kda_status check_conv(const char *op, const kda_conv_shape *s, const int32_t *cu, kda::ConvArgs *a) {
    if (!s) return fail(KDA_ERR_INVALID_ARG, "%s: shape is NULL", op);
    kda_status st = check_batch(op, s->B, s->T, s->num_seqs, cu);
    if (st != KDA_OK) return st;
    if ((st = check_dtype(op, s->dtype)) != KDA_OK) return st;
    if (s->C <= 0) return fail(KDA_ERR_INVALID_ARG, "%s: C=%d must be positive", op, s->C);
    if (s->W < 2 || s->W > 4) return fail(KDA_ERR_UNSUPPORTED, "%s: W=%d (supported: 2, 3, 4)", op, s->W);
    if (s->flags & ~KDA_CONV_FLAG_SILU)
        return fail(KDA_ERR_UNSUPPORTED, "%s: unknown flag bits 0x%x", op, s->flags);
    *a = kda::ConvArgs();
    if ((st = check_stride(op, "x_stride", s->x_stride, s->C, &a->x_stride)) != KDA_OK) return st;
    a->cu = cu;
    a->B = s->B; a->T = s->T; a->C = s->C; a->W = s->W; a->N = s->num_seqs;
    a->silu = (s->flags & KDA_CONV_FLAG_SILU) ? 1 : 0;
    return KDA_OK;
}

struct SsmWs {
    size_t ctrl, chunk_start, decay, rows, states, states_lo, total;
};
int64_t ssm_slots(const kda_ssm_shape *s, bool packed, int L) {
    const int64_t per = ((int64_t)s->T + L - 1) / L;
    return packed ? per + s->num_seqs : (int64_t)s->B * per;
}
// Sized for packed input where the shape may be packed (B == 1): it covers a dense call
// of the same shape, and the layout does not depend on which of the two is made.
bool may_be_packed(const kda_ssm_shape *s) { return s->B == 1; }
SsmWs ssm_ws(const kda_ssm_shape *s) {
    SsmWs w;
    const int L = kda::ssm_chunk_len(s->dtype, s->N, s->P);
    const int64_t slots = ssm_slots(s, may_be_packed(s), L);
    w.ctrl = 0;
    w.chunk_start = 256;
    w.decay = w.chunk_start + kda::align_up(sizeof(int32_t) * ((size_t)s->num_seqs + 1), 256);
    w.rows = kda::align_up(w.decay + (size_t)slots * s->H * 4, 256);
    w.states = kda::align_up(w.rows + (size_t)slots * s->H * kda::ssm_rows_bytes(s->dtype, s->N, s->P), 256);
    const size_t heads = (size_t)slots * s->H;
    w.states_lo = kda::align_up(w.states + heads * kda::ssm_state_bytes(s->dtype, s->N, s->P), 256);
    w.total = kda::align_up(
        w.states_lo + (s->flags & KDA_SSM_FLAG_NO_SAVE ? 0 : heads * kda::ssm_state_lo_bytes(s->dtype, s->N, s->P)),
        256);
    return w;
}
struct SsmBwdWs {
    size_t dstates, dstates_lo, dBh, dCh, sums, rowg, dDp, es, fwd, total;
    int parts;
};
SsmBwdWs ssm_bwd_ws(const kda_ssm_shape *s, bool saved) {
    SsmBwdWs w;
    const int L = kda::ssm_chunk_len(s->dtype, s->N, s->P);
    const bool tc = kda::ssm_tc_supported(s->dtype, s->N, s->P);
    const size_t slots = (size_t)ssm_slots(s, may_be_packed(s), L), heads = slots * s->H;
    const size_t tiles = tc ? kda::ssm_tc_tiles(s->P) : 0;
    w.parts = tc ? kda::ssm_tc_parts((int64_t)slots, s->G, (int)(s->H / s->G * tiles)) : 1;
    const size_t share = tc ? slots * s->G * w.parts * L * s->N * 4 : (size_t)s->B * s->T * s->H * s->N * 4;
    w.dstates = 0;
    w.dstates_lo = kda::align_up(heads * kda::ssm_state_bytes(s->dtype, s->N, s->P), 256);
    w.dBh = kda::align_up(w.dstates_lo + heads * kda::ssm_state_lo_bytes(s->dtype, s->N, s->P), 256);
    w.dCh = kda::align_up(w.dBh + share, 256);
    w.sums = kda::align_up(w.dCh + share, 256);
    w.rowg = kda::align_up(w.sums + heads * 3 * 4, 256);
    w.dDp = kda::align_up(w.rowg + heads * tiles * 4 * L * 4, 256);
    w.es = kda::align_up(w.dDp + heads * tiles * 4, 256);
    w.fwd = kda::align_up(w.es + (tc ? heads * kda::ssm_tc_es_floats(s->N, s->P) * 4 : 0), 256);
    w.total = w.fwd + (saved ? 0 : ssm_ws(s).total);
    return w;
}

bool ssm_sizes_ok(const kda_ssm_shape *s) {
    return s && s->B > 0 && s->T >= 0 && rows_ok(s->B, s->T) && s->H > 0 && s->G > 0 && s->H % s->G == 0 && s->N > 0 &&
           s->N <= 256 && s->P > 0 && s->P <= 256 && s->num_seqs >= 0;
}

kda_status check_ssm(const char *op, const kda_ssm_shape *s, const int32_t *cu, kda::SsmArgs *a) {
    if (!s) return fail(KDA_ERR_INVALID_ARG, "%s: shape is NULL", op);
    kda_status st = check_batch(op, s->B, s->T, s->num_seqs, cu);
    if (st != KDA_OK) return st;
    if ((st = check_dtype(op, s->dtype)) != KDA_OK) return st;
    if (s->H <= 0 || s->G <= 0 || s->N <= 0 || s->P <= 0 || s->H % s->G != 0)
        return fail(KDA_ERR_INVALID_ARG, "%s: H=%d G=%d N=%d P=%d (positive, H %% G == 0)", op, s->H,
                    s->G, s->N, s->P);
    if (s->N > 256 || s->P > 256)
        return fail(KDA_ERR_UNSUPPORTED, "%s: N=%d, P=%d (supported: up to 256)", op, s->N, s->P);
    if (s->flags & ~(KDA_SSM_FLAG_DT_SOFTPLUS | KDA_SSM_FLAG_NO_SAVE))
        return fail(KDA_ERR_UNSUPPORTED, "%s: unknown flag bits 0x%x", op, s->flags);
    *a = kda::SsmArgs();
    if ((st = check_stride(op, "x_stride", s->x_stride, (int64_t)s->H * s->P, &a->x_stride)) != KDA_OK ||
        (st = check_stride(op, "dt_stride", s->dt_stride, s->H, &a->dt_stride)) != KDA_OK ||
        (st = check_stride(op, "b_stride", s->b_stride, (int64_t)s->G * s->N, &a->b_stride)) != KDA_OK ||
        (st = check_stride(op, "c_stride", s->c_stride, (int64_t)s->G * s->N, &a->c_stride)) != KDA_OK)
        return st;
    a->cu = cu;
    a->B = s->B; a->T = s->T; a->H = s->H; a->G = s->G; a->Ns = s->N; a->P = s->P;
    a->N = s->num_seqs;
    a->softplus = (s->flags & KDA_SSM_FLAG_DT_SOFTPLUS) ? 1 : 0;
    a->L = kda::ssm_chunk_len(s->dtype, s->N, s->P);
    a->slots = ssm_slots(s, cu != nullptr, a->L);
    if (a->slots > INT_MAX) return fail(KDA_ERR_UNSUPPORTED, "%s: too many chunks", op);
    return KDA_OK;
}

void carve_fwd(const kda_ssm_shape *s, char *ws, kda::SsmArgs *a) {
    const SsmWs w = ssm_ws(s);
    a->ctrl = reinterpret_cast<kda::ChunkCtrl *>(ws + w.ctrl);
    a->chunk_start = reinterpret_cast<int32_t *>(ws + w.chunk_start);
    a->decay = reinterpret_cast<float *>(ws + w.decay);
    a->rows = ws + w.rows;
    a->states = reinterpret_cast<float *>(ws + w.states);
    a->states_lo = s->flags & KDA_SSM_FLAG_NO_SAVE ? nullptr : ws + w.states_lo;
}

bool norm_ok(const kda_norm_shape *s) { return s && s->rows >= 0 && s->cols >= 1 && s->cols <= 16384; }

kda_status check_norm(const char *op, const kda_norm_shape *s) {
    if (!s) return fail(KDA_ERR_INVALID_ARG, "%s: shape is NULL", op);
    if (s->rows < 0 || s->cols < 1)
        return fail(KDA_ERR_INVALID_ARG, "%s: rows=%lld cols=%d", op, (long long)s->rows, s->cols);
    if (s->cols > 16384) return fail(KDA_ERR_UNSUPPORTED, "%s: cols=%d > 16384", op, s->cols);
    if (!(s->eps >= 0.f) || !std::isfinite(s->eps))
        return fail(KDA_ERR_INVALID_ARG, "%s: eps must be finite and >= 0", op);
    return check_dtype(op, s->dtype);
}

}  // namespace

extern "C" {

kda_status kda_short_conv_fwd(const void *x, const float *w, const float *bias, const void *state_in,
                              const int32_t *cu_seqlens, const kda_conv_shape *shape, void *y,
                              void *state_out, int32_t *dev_status, kda_stream_t stream) {
    const char *op = "kda_short_conv_fwd";
    kda::ConvArgs a;
    kda_status st = check_conv(op, shape, cu_seqlens, &a);
    if (st != KDA_OK) return st;
    if (!w || ((int64_t)a.B * a.T > 0 && (!x || !y)))
        return fail(KDA_ERR_INVALID_ARG, "%s: x, w and y must be non-NULL", op);
    if (state_out && state_out == state_in)
        return fail(KDA_ERR_INVALID_ARG, "%s: state_out must not alias state_in", op);
    if (y && y == x) return fail(KDA_ERR_INVALID_ARG, "%s: y must not alias x", op);
    a.x = x; a.w = w; a.bias = bias; a.state_in = state_in; a.y = y; a.state_out = state_out;
    a.status = dev_status;
    return done(kda::launch_conv_fwd(a, shape->dtype, to_stream(stream)), op);
}

size_t kda_short_conv_bwd_workspace_size(const kda_conv_shape *s) {
    if (!s || s->B <= 0 || s->T < 0 || s->C <= 0 || s->W < 2 || s->W > 4) return 0;
    const int64_t strip = kda::conv_bwd_strip(s->B, s->T, s->C), rows = (int64_t)s->B * s->T;
    return (size_t)((rows + strip - 1) / strip) * (s->W + 1) * s->C * 4;
}

kda_status kda_short_conv_bwd(const void *x, const float *w, const float *bias, const void *state_in,
                              const int32_t *cu_seqlens, const kda_conv_shape *shape, const void *dy,
                              const void *dstate_out, void *dx, float *dw, float *dbias,
                              void *dstate_in, void *workspace, size_t workspace_bytes,
                              int32_t *dev_status, kda_stream_t stream) {
    const char *op = "kda_short_conv_bwd";
    kda::ConvArgs a;
    kda_status st = check_conv(op, shape, cu_seqlens, &a);
    if (st != KDA_OK) return st;
    const int64_t rows = (int64_t)a.B * a.T;
    if (!w || !dw || (rows > 0 && (!x || !dy || !dx)))
        return fail(KDA_ERR_INVALID_ARG, "%s: x, w, dy, dx and dw must be non-NULL", op);
    if ((st = check_workspace(op, workspace, workspace_bytes, kda_short_conv_bwd_workspace_size(shape),
                              16)) != KDA_OK)
        return st;
    if (dx && (dx == x || dx == dy)) return fail(KDA_ERR_INVALID_ARG, "%s: dx must not alias x or dy", op);
    a.x = x; a.w = w; a.bias = bias; a.state_in = state_in; a.dy = dy; a.dstate_out = dstate_out;
    a.dx = dx; a.dw = dw; a.dbias = dbias; a.dstate_in = dstate_in;
    a.part = static_cast<float *>(workspace);
    a.status = dev_status;
    if (cu_seqlens && rows > 0) {
        const size_t e = shape->dtype == KDA_DTYPE_BF16 ? 2 : 4;
        const cudaError_t err = cudaMemsetAsync(dx, 0, (size_t)rows * a.C * e, to_stream(stream));
        if (err != cudaSuccess) return done(err, op);
    }
    return done(kda::launch_conv_bwd(a, shape->dtype, to_stream(stream)), op);
}

kda_status kda_short_conv_step(const void *x, const float *w, const float *bias, void *state,
                               const int32_t *state_indices, int32_t num_slots,
                               const kda_conv_shape *shape, void *y, int32_t *dev_status,
                               kda_stream_t stream) {
    const char *op = "kda_short_conv_step";
    kda::ConvArgs c;
    kda_status st = check_conv(op, shape, nullptr, &c);
    if (st != KDA_OK) return st;
    if (c.T != 1) return fail(KDA_ERR_INVALID_ARG, "%s: T=%d must be 1", op, c.T);
    if (!x || !w || !y || (num_slots > 0 && !state))
        return fail(KDA_ERR_INVALID_ARG, "%s: x, w, state and y must be non-NULL", op);
    if (num_slots < 0 || (!state_indices && num_slots < c.B))
        return fail(KDA_ERR_INVALID_ARG, "%s: num_slots=%d for %d rows without state_indices", op,
                    num_slots, c.B);
    kda::ConvStepArgs a;
    a.x = x; a.w = w; a.bias = bias; a.state = state; a.idx = state_indices; a.y = y;
    a.status = dev_status;
    a.x_stride = c.x_stride;
    a.N = c.B; a.slots = num_slots; a.C = c.C; a.W = c.W; a.silu = c.silu;
    return done(kda::launch_conv_step(a, shape->dtype, to_stream(stream)), op);
}

size_t kda_ssm_workspace_size(const kda_ssm_shape *shape) {
    return ssm_sizes_ok(shape) ? ssm_ws(shape).total : 0;
}
size_t kda_ssm_bwd_workspace_size(const kda_ssm_shape *shape, int saved) {
    return ssm_sizes_ok(shape) ? ssm_bwd_ws(shape, saved != 0).total : 0;
}

kda_status kda_ssm_scan_fwd(const void *x, const void *dt, const float *A_log, const void *Bm,
                            const void *Cm, const float *D, const float *dt_bias, const float *h0,
                            const int32_t *cu_seqlens, const kda_ssm_shape *shape, void *y, float *ht,
                            void *workspace, size_t workspace_bytes, int32_t *dev_status,
                            kda_stream_t stream) {
    const char *op = "kda_ssm_scan_fwd";
    kda::SsmArgs a;
    kda_status st = check_ssm(op, shape, cu_seqlens, &a);
    if (st != KDA_OK) return st;
    if (!A_log || ((int64_t)a.B * a.T > 0 && (!x || !dt || !Bm || !Cm || !y)))
        return fail(KDA_ERR_INVALID_ARG, "%s: x, dt, A_log, Bm, Cm and y must be non-NULL", op);
    if ((st = check_workspace(op, workspace, workspace_bytes, kda_ssm_workspace_size(shape), 256)) != KDA_OK)
        return st;
    a.x = x; a.dt = dt; a.Bm = Bm; a.Cm = Cm; a.A_log = A_log; a.D = D; a.dt_bias = dt_bias;
    a.h0 = h0; a.y = y; a.ht = ht; a.status = dev_status;
    carve_fwd(shape, static_cast<char *>(workspace), &a);
    return done(kda::launch_ssm_fwd(a, shape->dtype, to_stream(stream)), op);
}

kda_status kda_ssm_scan_bwd(const void *x, const void *dt, const float *A_log, const void *Bm,
                            const void *Cm, const float *D, const float *dt_bias, const float *h0,
                            const int32_t *cu_seqlens, const kda_ssm_shape *shape, const void *dy,
                            const float *dht, void *dx, void *ddt, void *dB, void *dC, float *dA_log,
                            float *dD, float *ddt_bias, float *dh0, const void *saved,
                            void *workspace, size_t workspace_bytes, int32_t *dev_status,
                            kda_stream_t stream) {
    const char *op = "kda_ssm_scan_bwd";
    kda::SsmArgs a;
    kda_status st = check_ssm(op, shape, cu_seqlens, &a);
    if (st != KDA_OK) return st;
    if (shape->flags & KDA_SSM_FLAG_NO_SAVE)
        return fail(KDA_ERR_INVALID_ARG, "%s: KDA_SSM_FLAG_NO_SAVE is the forward's alone", op);
    const int64_t rows = (int64_t)a.B * a.T;
    if (!A_log || !dA_log || (rows > 0 && (!x || !dt || !Bm || !Cm || !dy || !dx || !ddt || !dB || !dC)))
        return fail(KDA_ERR_INVALID_ARG, "%s: x, dt, A_log, Bm, Cm, dy and dx, ddt, dB, dC, dA_log must "
                    "be non-NULL", op);
    if ((st = check_workspace(op, workspace, workspace_bytes,
                              kda_ssm_bwd_workspace_size(shape, saved != nullptr), 256)) != KDA_OK)
        return st;
    if ((uintptr_t)saved % 256 != 0)
        return fail(KDA_ERR_INVALID_ARG, "%s: saved must be 256-byte aligned", op);
    a.x = x; a.dt = dt; a.Bm = Bm; a.Cm = Cm; a.A_log = A_log; a.D = D; a.dt_bias = dt_bias;
    a.h0 = h0; a.status = dev_status;
    a.dy = dy; a.dht = dht; a.dx = dx; a.ddt = ddt; a.dB = dB; a.dC = dC;
    a.dA_log = dA_log; a.dD = dD; a.ddt_bias = ddt_bias; a.dh0 = dh0;
    char *ws = static_cast<char *>(workspace);
    const SsmBwdWs w = ssm_bwd_ws(shape, saved != nullptr);
    a.dstates = reinterpret_cast<float *>(ws + w.dstates);
    a.dstates_lo = ws + w.dstates_lo;
    a.dBh = reinterpret_cast<float *>(ws + w.dBh);
    a.dCh = reinterpret_cast<float *>(ws + w.dCh);
    a.sums = reinterpret_cast<float *>(ws + w.sums);
    a.rowg = reinterpret_cast<float *>(ws + w.rowg);
    a.dDp = reinterpret_cast<float *>(ws + w.dDp);
    a.es = reinterpret_cast<float *>(ws + w.es);
    a.parts = w.parts;
    cudaStream_t s = to_stream(stream);
    cudaError_t e = cudaSuccess;
    if (cu_seqlens && rows > 0) {
        const size_t es = shape->dtype == KDA_DTYPE_BF16 ? 2 : 4;
        e = cudaMemsetAsync(dx, 0, (size_t)rows * a.H * a.P * es, s);
        if (e == cudaSuccess) e = cudaMemsetAsync(ddt, 0, (size_t)rows * a.H * es, s);
        if (e == cudaSuccess) e = cudaMemsetAsync(dB, 0, (size_t)rows * a.G * a.Ns * es, s);
        if (e == cudaSuccess) e = cudaMemsetAsync(dC, 0, (size_t)rows * a.G * a.Ns * es, s);
        if (e != cudaSuccess) return done(e, op);
    }
    if (saved) {  // read only: the forward's stores
        carve_fwd(shape, static_cast<char *>(const_cast<void *>(saved)), &a);
    } else {
        carve_fwd(shape, ws + w.fwd, &a);
        if ((e = kda::launch_ssm_states(a, shape->dtype, s)) != cudaSuccess) return done(e, op);
    }
    return done(kda::launch_ssm_bwd(a, shape->dtype, s), op);
}

kda_status kda_ssm_step(const void *x, const void *dt, const float *A_log, const void *Bm,
                        const void *Cm, const float *D, const float *dt_bias, float *state,
                        const int32_t *state_indices, int32_t num_slots, const kda_ssm_shape *shape,
                        void *y, int32_t *dev_status, kda_stream_t stream) {
    const char *op = "kda_ssm_step";
    kda::SsmArgs c;
    kda_status st = check_ssm(op, shape, nullptr, &c);
    if (st != KDA_OK) return st;
    if (c.T != 1) return fail(KDA_ERR_INVALID_ARG, "%s: T=%d must be 1", op, c.T);
    if (!x || !dt || !A_log || !Bm || !Cm || !y || (num_slots > 0 && !state))
        return fail(KDA_ERR_INVALID_ARG, "%s: x, dt, A_log, Bm, Cm, state and y must be non-NULL", op);
    if (num_slots < 0 || (!state_indices && num_slots < c.B))
        return fail(KDA_ERR_INVALID_ARG, "%s: num_slots=%d for %d rows without state_indices", op,
                    num_slots, c.B);
    kda::SsmStepArgs a;
    a.x = x; a.dt = dt; a.Bm = Bm; a.Cm = Cm; a.A_log = A_log; a.D = D; a.dt_bias = dt_bias;
    a.state = state; a.idx = state_indices; a.y = y; a.status = dev_status;
    a.x_stride = c.x_stride; a.dt_stride = c.dt_stride; a.b_stride = c.b_stride; a.c_stride = c.c_stride;
    a.N = c.B; a.slots = num_slots; a.H = c.H; a.G = c.G; a.Ns = c.Ns; a.P = c.P;
    a.softplus = c.softplus;
    return done(kda::launch_ssm_step(a, shape->dtype, to_stream(stream)), op);
}

kda_status kda_add_rmsnorm_fwd(const void *x, const void *residual, const float *w,
                               const kda_norm_shape *shape, void *h, void *y, float *scale,
                               kda_stream_t stream) {
    const char *op = "kda_add_rmsnorm_fwd";
    kda_status st = check_norm(op, shape);
    if (st != KDA_OK) return st;
    if (shape->out != KDA_NORM_SAME && shape->out != KDA_NORM_E4M3 && shape->out != KDA_NORM_INT8)
        return fail(KDA_ERR_INVALID_ARG, "%s: unknown output type %d", op, (int)shape->out);
    if (shape->group != 0 && shape->group != 128)
        return fail(KDA_ERR_UNSUPPORTED, "%s: group=%d (supported: 0, 128)", op, shape->group);
    if (shape->rows > 0 && (!x || !w || !y || (shape->out != KDA_NORM_SAME && !scale)))
        return fail(KDA_ERR_INVALID_ARG, "%s: x, w, y (and scale for 8-bit outputs) must be non-NULL", op);
    kda::NormArgs a{};
    a.x = x; a.res = residual; a.w = w; a.h = h; a.y = y; a.scale = scale;
    a.rows = shape->rows; a.cols = shape->cols; a.group = shape->group; a.out = shape->out;
    a.eps = shape->eps;
    return done(kda::launch_norm_fwd(a, shape->dtype, to_stream(stream)), op);
}

size_t kda_add_rmsnorm_bwd_workspace_size(const kda_norm_shape *s) {
    return norm_ok(s) ? (size_t)kda::norm_bwd_parts(s->rows, s->cols, s->dtype) * s->cols * 4 : 0;
}

kda_status kda_add_rmsnorm_bwd(const void *dy, const void *h, const float *w, const void *dh,
                               const kda_norm_shape *shape, void *dx, float *dw, void *workspace,
                               size_t workspace_bytes, kda_stream_t stream) {
    const char *op = "kda_add_rmsnorm_bwd";
    kda_status st = check_norm(op, shape);
    if (st != KDA_OK) return st;
    if (!w || !dw || (shape->rows > 0 && (!dy || !h || !dx)))
        return fail(KDA_ERR_INVALID_ARG, "%s: dy, h, w, dx and dw must be non-NULL", op);
    if ((st = check_workspace(op, workspace, workspace_bytes, kda_add_rmsnorm_bwd_workspace_size(shape),
                              16)) != KDA_OK)
        return st;
    kda::NormArgs a{};
    a.dy = dy; a.h = const_cast<void *>(h); a.w = w; a.dres = dh; a.dx = dx; a.dw = dw;
    a.part = static_cast<float *>(workspace);
    a.rows = shape->rows; a.cols = shape->cols; a.eps = shape->eps;
    return done(kda::launch_norm_bwd(a, shape->dtype, to_stream(stream)), op);
}

}  // extern "C"
