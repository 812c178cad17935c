// kda_gdn_api.cu -- the extern "C" entry points of the gated delta rule and of the norms around a
// gated block: host-side argument checks, workspace carving and launches.
#include <climits>
#include <cmath>

#include "kda_check.cuh"
#include "kda_gdn.cuh"

namespace {

using namespace kda_check;

struct GdnWs {
    size_t ctrl, chunk_start, norms, rows, mats, wk, states, us, mt, wt, kt, u0, carry, total;
};
int64_t gdn_slots(const kda_gdn_shape *s, bool packed, int L) {
    const int64_t per = ((int64_t)s->T + L - 1) / L;
    return packed ? per + s->num_seqs : (int64_t)s->B * per;
}
// Sized for packed input where the shape may be packed (B == 1): it covers a dense call of the
// same shape, and the layout does not depend on which of the two is made.
GdnWs gdn_ws(const kda_gdn_shape *s) {
    GdnWs w;
    const int L = kda::gdn_chunk_len(s->dtype, s->K, s->V);
    const size_t units = (size_t)gdn_slots(s, s->B == 1, L) * s->HV;
    const bool save = !(s->flags & KDA_GDN_FLAG_NO_SAVE);
    w.ctrl = 0;
    w.chunk_start = 256;
    w.norms = w.chunk_start + kda::align_up(sizeof(int32_t) * ((size_t)s->num_seqs + 1), 256);
    w.rows = w.norms + (s->flags & KDA_GDN_FLAG_QK_L2NORM ? kda::align_up((size_t)s->B * s->T * s->H * 8, 256) : 0);
    w.mats = kda::align_up(w.rows + units * kda::gdn_rows_floats(L) * 4, 256);
    if (kda::gdn_tc_supported(s->dtype, s->K, s->V)) {
        const size_t tile = kda::kGdnTile;
        w.states = w.wk = w.mats;
        w.us = w.states + units * 2 * tile;
        w.mt = w.us + units * 2 * tile;
        w.wt = w.mt + (save ? units * 2 * tile : 0);
        w.u0 = w.wt + units * 2 * tile;
        w.kt = w.u0 + units * 2 * tile;
        w.carry = w.kt + units / s->HV * s->H * tile;
        w.total = w.carry + kda::align_up((size_t)s->num_seqs * s->HV * s->K * s->V * 4, 256);
        return w;
    }
    w.wk = w.mats + units * kda::gdn_mats_floats(L) * 4;
    w.states = w.wk + units * kda::gdn_wk_floats(L, s->K) * 4;
    w.us = w.states + units * kda::gdn_state_floats(s->K, s->V) * 4;
    w.total = w.us + units * kda::gdn_u_floats(L, s->V) * 4;
    w.mt = w.wt = w.kt = w.u0 = w.carry = 0;
    return w;
}
struct GdnBwdWs {
    size_t dstates, zs, du0, b0, dcarry, dqh, dkh, fwd, total;
};
GdnBwdWs gdn_bwd_ws(const kda_gdn_shape *s, bool saved) {
    GdnBwdWs w;
    const int L = kda::gdn_chunk_len(s->dtype, s->K, s->V);
    const size_t units = (size_t)gdn_slots(s, s->B == 1, L) * s->HV;
    const size_t heads = kda::align_up((size_t)s->B * s->T * s->HV * s->K * 4, 256);
    const bool tensor = kda::gdn_tc_supported(s->dtype, s->K, s->V);
    const size_t tiles = units * 2 * kda::kGdnTile;
    w.dstates = 0;
    w.zs = tensor ? tiles : units * kda::gdn_state_floats(s->K, s->V) * 4;
    w.du0 = w.zs + (tensor ? tiles : units * kda::gdn_u_floats(L, s->V) * 4);
    w.b0 = w.du0 + (tensor ? tiles : 0);
    w.dcarry = w.b0 + (tensor ? tiles : 0);
    w.dqh = w.dcarry + (tensor ? kda::align_up((size_t)s->num_seqs * s->HV * s->K * s->V * 4, 256) : 0);
    // (value heads that share no q and k have dq and dk stored directly)
    w.dkh = w.dqh + (tensor && s->HV == s->H ? 0 : heads);
    w.fwd = w.dkh + (w.dkh - w.dqh);
    w.total = w.fwd + (saved ? 0 : gdn_ws(s).total);
    return w;
}

bool gdn_sizes_ok(const kda_gdn_shape *s) {
    return s && s->B > 0 && s->T >= 0 && rows_ok(s->B, s->T) && s->H > 0 && s->HV > 0 && s->HV % s->H == 0 && s->K > 0 &&
           s->K <= 256 && s->V > 0 && s->V <= 256 && s->num_seqs >= 0 &&
           (s->dtype == KDA_DTYPE_F32 || s->dtype == KDA_DTYPE_BF16);
}

kda_status check_gdn(const char *op, const kda_gdn_shape *s, const int32_t *cu, kda::GdnArgs *a) {
    if (!s) return fail(KDA_ERR_INVALID_ARG, "%s: shape is NULL", op);
    kda_status st = check_batch(op, s->B, s->T, s->num_seqs, cu);
    if (st != KDA_OK) return st;
    if ((st = check_dtype(op, s->dtype)) != KDA_OK) return st;
    if (s->H <= 0 || s->HV <= 0 || s->K <= 0 || s->V <= 0 || s->HV % s->H != 0)
        return fail(KDA_ERR_INVALID_ARG, "%s: H=%d HV=%d K=%d V=%d (positive, HV %% H == 0)", op, s->H, s->HV, s->K,
                    s->V);
    if (s->K > 256 || s->V > 256)
        return fail(KDA_ERR_UNSUPPORTED, "%s: K=%d, V=%d (supported: up to 256)", op, s->K, s->V);
    if (s->flags & ~(KDA_GDN_FLAG_QK_L2NORM | KDA_GDN_FLAG_NO_SAVE | KDA_GDN_FLAG_TEST_WAIT_TIMEOUT))
        return fail(KDA_ERR_UNSUPPORTED, "%s: unknown flag bits 0x%x", op, s->flags);
    if (!std::isfinite(s->scale) || !std::isfinite(s->g_scale))
        return fail(KDA_ERR_INVALID_ARG, "%s: scale and g_scale must be finite", op);
    *a = kda::GdnArgs();
    if ((st = check_stride(op, "q_stride", s->q_stride, (int64_t)s->H * s->K, &a->q_stride)) != KDA_OK ||
        (st = check_stride(op, "k_stride", s->k_stride, (int64_t)s->H * s->K, &a->k_stride)) != KDA_OK ||
        (st = check_stride(op, "v_stride", s->v_stride, (int64_t)s->HV * s->V, &a->v_stride)) != KDA_OK)
        return st;
    a->cu = cu;
    a->B = s->B; a->T = s->T; a->H = s->H; a->HV = s->HV; a->K = s->K; a->V = s->V;
    a->N = s->num_seqs;
    a->l2 = (s->flags & KDA_GDN_FLAG_QK_L2NORM) ? 1 : 0;
    a->give_up = (s->flags & KDA_GDN_FLAG_TEST_WAIT_TIMEOUT) ? 1 : 0;
    a->scale = s->scale > 0.f ? s->scale : 1.f / std::sqrt((float)s->K);
    a->g_scale = s->g_scale;
    a->L = kda::gdn_chunk_len(s->dtype, s->K, s->V);
    a->slots = gdn_slots(s, cu != nullptr, a->L);
    // blocks per unit and per (sequence, head, 32 columns) are counted in 31 bits (units in steps of a grid)
    if (a->slots * s->HV > INT_MAX - 1024 || (int64_t)s->num_seqs * s->HV * 8 > INT_MAX ||
        (int64_t)s->B * s->T * s->H > INT_MAX)
        return fail(KDA_ERR_UNSUPPORTED, "%s: too many chunks, rows or sequences times heads", op);
    return KDA_OK;
}

void carve_fwd(const kda_gdn_shape *s, char *ws, kda::GdnArgs *a) {
    const GdnWs w = gdn_ws(s);
    const bool save = !(s->flags & KDA_GDN_FLAG_NO_SAVE);
    a->ctrl = reinterpret_cast<kda::ChunkCtrl *>(ws + w.ctrl);
    a->chunk_start = reinterpret_cast<int32_t *>(ws + w.chunk_start);
    a->norms = reinterpret_cast<float *>(ws + w.norms);
    a->rows = reinterpret_cast<float *>(ws + w.rows);
    if (kda::gdn_tc_supported(s->dtype, s->K, s->V)) {
        uint8_t *b = reinterpret_cast<uint8_t *>(ws);
        a->st = b + w.states;
        a->ut = b + w.us;
        a->mt = save ? b + w.mt : nullptr;
        a->wt = b + w.wt;
        a->kt = b + w.kt;
        a->u0 = reinterpret_cast<float *>(ws + w.u0);
        a->carry = reinterpret_cast<float *>(ws + w.carry);
        return;
    }
    a->mats = reinterpret_cast<float *>(ws + w.mats);
    a->wk = reinterpret_cast<float *>(ws + w.wk);
    a->states = reinterpret_cast<float *>(ws + w.states);
    a->us = reinterpret_cast<float *>(ws + w.us);
}

kda_status check_gated(const char *op, const kda_gated_norm_shape *s, kda::GatedNormArgs *a) {
    if (!s) return fail(KDA_ERR_INVALID_ARG, "%s: shape is NULL", op);
    if (s->rows < 0 || s->cols < 1 || s->group < 1 || s->cols % s->group != 0)
        return fail(KDA_ERR_INVALID_ARG, "%s: rows=%lld cols=%d group=%d (cols a multiple of group)", op,
                    (long long)s->rows, s->cols, s->group);
    if (s->cols > 131072 || s->group > 16384)
        return fail(KDA_ERR_UNSUPPORTED, "%s: cols=%d > 131072 or group=%d > 16384", op, s->cols, s->group);
    if (s->act != KDA_GATE_SIGMOID && s->act != KDA_GATE_SILU)
        return fail(KDA_ERR_INVALID_ARG, "%s: unknown activation %d", op, (int)s->act);
    if (!(s->eps >= 0.f) || !std::isfinite(s->eps))
        return fail(KDA_ERR_INVALID_ARG, "%s: eps must be finite and >= 0", op);
    kda_status st = check_dtype(op, s->dtype);
    if (st != KDA_OK) return st;
    *a = kda::GatedNormArgs();
    if ((st = check_stride(op, "x_stride", s->x_stride, s->cols, &a->x_stride)) != KDA_OK ||
        (st = check_stride(op, "gate_stride", s->gate_stride, s->cols, &a->z_stride)) != KDA_OK)
        return st;
    a->rows = s->rows;
    a->group = s->group;
    a->parts = s->cols / s->group;
    a->shared = s->shared_weight != 0;
    a->act = s->act;
    a->first = s->gate_first != 0;
    a->eps = s->eps;
    if (s->rows > INT_MAX / a->parts) return fail(KDA_ERR_UNSUPPORTED, "%s: too many rows", op);
    return KDA_OK;
}
bool gated_ok(const kda_gated_norm_shape *s) {
    return s && s->rows >= 0 && s->cols >= 1 && s->cols <= 131072 && s->group >= 1 && s->group <= 16384 &&
           s->cols % s->group == 0;
}

kda_status check_sandwich(const char *op, const kda_sandwich_shape *s, kda::SandwichArgs *a) {
    if (!s) return fail(KDA_ERR_INVALID_ARG, "%s: shape is NULL", op);
    if (s->rows < 0 || s->cols < 1)
        return fail(KDA_ERR_INVALID_ARG, "%s: rows=%lld cols=%d", op, (long long)s->rows, s->cols);
    if (s->cols > 16384) return fail(KDA_ERR_UNSUPPORTED, "%s: cols=%d > 16384", op, s->cols);
    if (s->rows > INT_MAX) return fail(KDA_ERR_UNSUPPORTED, "%s: too many rows", op);
    if (s->act != KDA_GATE_SIGMOID && s->act != KDA_GATE_SILU)
        return fail(KDA_ERR_INVALID_ARG, "%s: unknown activation %d", op, (int)s->act);
    if (!(s->eps >= 0.f) || !std::isfinite(s->eps))
        return fail(KDA_ERR_INVALID_ARG, "%s: eps must be finite and >= 0", op);
    *a = kda::SandwichArgs();
    a->rows = s->rows;
    a->cols = s->cols;
    a->act = s->act;
    a->eps = s->eps;
    return check_dtype(op, s->dtype);
}

}  // namespace

extern "C" {

size_t kda_gdn_workspace_size(const kda_gdn_shape *shape) { return gdn_sizes_ok(shape) ? gdn_ws(shape).total : 0; }
size_t kda_gdn_bwd_workspace_size(const kda_gdn_shape *shape, int saved) {
    return gdn_sizes_ok(shape) ? gdn_bwd_ws(shape, saved != 0).total : 0;
}

kda_status kda_gdn_fwd(const void *q, const void *k, const void *v, const float *g, const void *beta,
                       const float *h0, const int32_t *cu_seqlens, const kda_gdn_shape *shape, void *o,
                       float *ht, void *workspace, size_t workspace_bytes, int32_t *dev_status,
                       kda_stream_t stream) {
    const char *op = "kda_gdn_fwd";
    kda::GdnArgs a;
    kda_status st = check_gdn(op, shape, cu_seqlens, &a);
    if (st != KDA_OK) return st;
    if ((int64_t)a.B * a.T > 0 && (!q || !k || !v || !g || !beta || !o))
        return fail(KDA_ERR_INVALID_ARG, "%s: q, k, v, g, beta and o must be non-NULL", op);
    if (o && (o == q || o == k || o == v))
        return fail(KDA_ERR_INVALID_ARG, "%s: o must not alias q, k or v", op);
    if ((st = check_workspace(op, workspace, workspace_bytes, kda_gdn_workspace_size(shape), 256)) != KDA_OK)
        return st;
    a.q = q; a.k = k; a.v = v; a.g = g; a.beta = beta; a.h0 = h0; a.o = o; a.ht = ht; a.status = dev_status;
    carve_fwd(shape, static_cast<char *>(workspace), &a);
    return done(kda::launch_gdn_fwd(a, shape->dtype, to_stream(stream)), op);
}

kda_status kda_gdn_bwd(const void *q, const void *k, const void *v, const float *g, const void *beta,
                       const float *h0, const int32_t *cu_seqlens, const kda_gdn_shape *shape,
                       const void *dout, const float *dht, void *dq, void *dk, void *dv, float *dg,
                       void *dbeta, float *dh0, const void *saved, void *workspace,
                       size_t workspace_bytes, int32_t *dev_status, kda_stream_t stream) {
    const char *op = "kda_gdn_bwd";
    kda::GdnArgs a;
    kda_status st = check_gdn(op, shape, cu_seqlens, &a);
    if (st != KDA_OK) return st;
    if (shape->flags & KDA_GDN_FLAG_NO_SAVE)
        return fail(KDA_ERR_UNSUPPORTED, "%s: KDA_GDN_FLAG_NO_SAVE is a forward's", op);
    if ((int64_t)a.B * a.T > 0 && (!q || !k || !v || !g || !beta || !dout || !dq || !dk || !dv || !dg || !dbeta))
        return fail(KDA_ERR_INVALID_ARG, "%s: q, k, v, g, beta, dout and their gradients must be non-NULL", op);
    if ((uintptr_t)saved % 256 != 0) return fail(KDA_ERR_INVALID_ARG, "%s: saved must be 256-byte aligned", op);
    if ((st = check_workspace(op, workspace, workspace_bytes, kda_gdn_bwd_workspace_size(shape, saved != nullptr),
                              256)) != KDA_OK)
        return st;
    for (const void *to : {dq, dk, dv, dbeta, (void *)dg})
        for (const void *from : {q, k, v, (const void *)g, beta, dout})
            if (to && to == from) return fail(KDA_ERR_INVALID_ARG, "%s: a gradient must not alias an input", op);
    const GdnBwdWs w = gdn_bwd_ws(shape, saved != nullptr);
    char *ws = static_cast<char *>(workspace);
    a.q = q; a.k = k; a.v = v; a.g = g; a.beta = beta; a.h0 = h0; a.status = dev_status;
    a.dout = dout; a.dht = dht; a.dq = dq; a.dk = dk; a.dv = dv; a.dg = dg; a.dbeta = dbeta; a.dh0 = dh0;
    // (a saved workspace is only read)
    carve_fwd(shape, saved ? const_cast<char *>(static_cast<const char *>(saved)) : ws + w.fwd, &a);
    a.dstates = reinterpret_cast<float *>(ws + w.dstates);
    a.zs = reinterpret_cast<float *>(ws + w.zs);
    a.et = reinterpret_cast<uint8_t *>(ws + w.dstates);
    a.dut = reinterpret_cast<uint8_t *>(ws + w.zs);
    a.du0 = reinterpret_cast<float *>(ws + w.du0);
    a.b0 = reinterpret_cast<float *>(ws + w.b0);
    a.dcarry = reinterpret_cast<float *>(ws + w.dcarry);
    a.dqh = reinterpret_cast<float *>(ws + w.dqh);
    a.dkh = reinterpret_cast<float *>(ws + w.dkh);
    return done(kda::launch_gdn_bwd(a, shape->dtype, saved != nullptr, to_stream(stream)), op);
}

kda_status kda_gdn_step(const void *q, const void *k, const void *v, const float *g, const void *beta,
                        float *state, const int32_t *state_indices, int32_t num_slots,
                        const kda_gdn_shape *shape, void *o, int32_t *dev_status, kda_stream_t stream) {
    const char *op = "kda_gdn_step";
    kda::GdnArgs c;
    kda_status st = check_gdn(op, shape, nullptr, &c);
    if (st != KDA_OK) return st;
    if (c.T != 1) return fail(KDA_ERR_INVALID_ARG, "%s: T=%d must be 1", op, c.T);
    if (!q || !k || !v || !g || !beta || !o || (num_slots > 0 && !state))
        return fail(KDA_ERR_INVALID_ARG, "%s: q, k, v, g, beta, state and o must be non-NULL", op);
    if (num_slots < 0 || (!state_indices && num_slots < c.B))
        return fail(KDA_ERR_INVALID_ARG, "%s: num_slots=%d for %d rows without state_indices", op, num_slots, c.B);
    if (o == q || o == k || o == v) return fail(KDA_ERR_INVALID_ARG, "%s: o must not alias q, k or v", op);
    kda::GdnStepArgs a;
    a.q = q; a.k = k; a.v = v; a.g = g; a.beta = beta; a.state = state; a.idx = state_indices; a.o = o;
    a.status = dev_status;
    a.q_stride = c.q_stride; a.k_stride = c.k_stride; a.v_stride = c.v_stride;
    a.N = c.B; a.slots = num_slots; a.H = c.H; a.HV = c.HV; a.K = c.K; a.V = c.V; a.l2 = c.l2;
    a.scale = c.scale; a.g_scale = c.g_scale;
    return done(kda::launch_gdn_step(a, shape->dtype, to_stream(stream)), op);
}

kda_status kda_gated_rmsnorm_fwd(const void *x, const void *gate, const float *w,
                                 const kda_gated_norm_shape *shape, void *y, kda_stream_t stream) {
    const char *op = "kda_gated_rmsnorm_fwd";
    kda::GatedNormArgs a;
    kda_status st = check_gated(op, shape, &a);
    if (st != KDA_OK) return st;
    if (shape->rows > 0 && (!x || !gate || !w || !y))
        return fail(KDA_ERR_INVALID_ARG, "%s: x, gate, w and y must be non-NULL", op);
    a.x = x; a.z = gate; a.w = w; a.y = y;
    return done(kda::launch_gated_norm(a, shape->dtype, false, to_stream(stream)), op);
}

size_t kda_gated_rmsnorm_bwd_workspace_size(const kda_gated_norm_shape *s) {
    if (!gated_ok(s)) return 0;
    const bool shared = s->shared_weight != 0;
    return (size_t)kda::gated_bwd_rows(s->rows, s->cols / s->group, shared) * (shared ? s->group : s->cols) * 4;
}

kda_status kda_gated_rmsnorm_bwd(const void *dy, const void *x, const void *gate, const float *w,
                                 const kda_gated_norm_shape *shape, void *dx, void *dgate, float *dw,
                                 void *workspace, size_t workspace_bytes, kda_stream_t stream) {
    const char *op = "kda_gated_rmsnorm_bwd";
    kda::GatedNormArgs a;
    kda_status st = check_gated(op, shape, &a);
    if (st != KDA_OK) return st;
    if (!w || !dw || (shape->rows > 0 && (!dy || !x || !gate || !dx || !dgate)))
        return fail(KDA_ERR_INVALID_ARG, "%s: dy, x, gate, w, dx, dgate and dw must be non-NULL", op);
    if ((st = check_workspace(op, workspace, workspace_bytes, kda_gated_rmsnorm_bwd_workspace_size(shape), 16)) !=
        KDA_OK)
        return st;
    a.dy = dy; a.x = x; a.z = gate; a.w = w; a.dx = dx; a.dz = dgate; a.dw = dw;
    a.part = static_cast<float *>(workspace);
    return done(kda::launch_gated_norm(a, shape->dtype, true, to_stream(stream)), op);
}

kda_status kda_sandwich_norm_fwd(const void *x, const void *residual, const void *gate,
                                 const float *w_post, const float *w_pre, const float *residual_scale,
                                 const kda_sandwich_shape *shape, void *h, void *y, kda_stream_t stream) {
    const char *op = "kda_sandwich_norm_fwd";
    kda::SandwichArgs a;
    kda_status st = check_sandwich(op, shape, &a);
    if (st != KDA_OK) return st;
    if (shape->rows > 0 && (!x || !residual || !w_post || !w_pre || !h || !y))
        return fail(KDA_ERR_INVALID_ARG, "%s: x, residual, w_post, w_pre, h and y must be non-NULL", op);
    a.x = x; a.res = residual; a.z = gate; a.w_post = w_post; a.w_pre = w_pre; a.rs = residual_scale;
    a.h = h; a.y = y;
    return done(kda::launch_sandwich(a, shape->dtype, false, to_stream(stream)), op);
}

size_t kda_sandwich_norm_bwd_workspace_size(const kda_sandwich_shape *s) {
    if (!s || s->rows < 0 || s->cols < 1 || s->cols > 16384) return 0;
    return (size_t)kda::sandwich_bwd_rows(s->rows) * 3 * s->cols * 4;
}

kda_status kda_sandwich_norm_bwd(const void *dy, const void *dh, const void *x, const void *residual,
                                 const void *gate, const float *w_post, const float *w_pre,
                                 const float *residual_scale, const kda_sandwich_shape *shape, void *dx,
                                 void *dresidual, void *dgate, float *dw_post, float *dw_pre,
                                 float *dresidual_scale, void *workspace, size_t workspace_bytes,
                                 kda_stream_t stream) {
    const char *op = "kda_sandwich_norm_bwd";
    kda::SandwichArgs a;
    kda_status st = check_sandwich(op, shape, &a);
    if (st != KDA_OK) return st;
    if (!w_post || !w_pre || !dw_post || !dw_pre || (shape->rows > 0 && (!dy || !x || !residual || !dx || !dresidual)))
        return fail(KDA_ERR_INVALID_ARG, "%s: dy, x, residual, the weights and their gradients must be non-NULL", op);
    if ((shape->rows > 0 && gate && !dgate) || (residual_scale && !dresidual_scale))
        return fail(KDA_ERR_INVALID_ARG, "%s: dgate goes with gate, dresidual_scale with residual_scale", op);
    if ((st = check_workspace(op, workspace, workspace_bytes, kda_sandwich_norm_bwd_workspace_size(shape), 16)) !=
        KDA_OK)
        return st;
    a.dy = dy; a.dh = dh; a.x = x; a.res = residual; a.z = gate; a.w_post = w_post; a.w_pre = w_pre;
    a.rs = residual_scale; a.dx = dx; a.dres = dresidual; a.dz = gate ? dgate : nullptr;
    a.dw_post = dw_post; a.dw_pre = dw_pre; a.drs = residual_scale ? dresidual_scale : nullptr;
    a.part = static_cast<float *>(workspace);
    return done(kda::launch_sandwich(a, shape->dtype, true, to_stream(stream)), op);
}

}  // extern "C"
