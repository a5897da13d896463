// Entry points of the bf16 training products and the 8-bit activation
// checkpoints (declared in include/fwmoe.h): argument checks, workspace layout
// and launch sequences.  Host code only; nothing is allocated, nothing waits.
#include <stdint.h>

#include <algorithm>

#include "dense.h"

namespace fw {

DenseWs dense_ws(const fw_moe_dense_desc &d, int R) {
    DenseWs L{};
    const size_t E = d.n_experts, K = d.in_features, N = d.out_features;
    size_t off = sizeof(WsHeader);
    auto take = [&](size_t bytes) {
        const size_t at = off;
        off = (off + bytes + 255) & ~(size_t)255;
        return at;
    };
    L.max_tiles = (R + kDenseMinTileRows - 1) / kDenseMinTileRows + (int)E;
    L.active = take((E + 1) * sizeof(int4));
    L.tiles = take((size_t)L.max_tiles * sizeof(int4));
    L.split_cnt = take((size_t)kSplitTiles * 4);
    L.xq = take(d.ckpt == FW_ACT_NONE ? 0 : (size_t)R * K * 2);
    L.dz = take(2 * (size_t)R * N * 2);
    L.bpart = take((size_t)L.max_tiles * N * 4);
    L.total = off;
    return L;
}

}  // namespace fw

using namespace fw;

namespace {

constexpr int kMaxRows = 1 << 20, kMaxFeatures = 1 << 16;

bool al16(const void *p) { return ((uintptr_t)p & 15) == 0; }
bool al256(const void *p) { return ((uintptr_t)p & 255) == 0; }
int hip_status(hipError_t e) { return e == hipSuccess ? FW_OK : FW_EHIP; }
bool dtype_ok(int t) { return t == FW_F32 || t == FW_BF16; }

// A launch of `groups` workgroups of 256 threads fits HIP's 2^32 threads.
bool grid_ok(int64_t groups) { return groups < (int64_t)1 << 23; }

int check_dense(const fw_moe_dense_desc *d) {
    if (!d) return FW_EINVAL;
    for (int f : {d->in_features, d->out_features})
        if (f < 8 || f > kMaxFeatures || f % 8) return FW_EINVAL;
    if (d->n_experts < 1 || d->n_experts > kMaxExperts) return FW_EINVAL;
    if (d->fn < FW_FN_NONE || d->fn > FW_FN_RELU) return FW_EINVAL;
    if (d->ckpt < FW_ACT_NONE || d->ckpt > FW_ACT_INT8) return FW_EINVAL;
    if (!dtype_ok(d->out_dtype) || !dtype_ok(d->grad_dtype)) return FW_EINVAL;
    if (d->accumulate != 0 && d->accumulate != 1) return FW_EINVAL;
    if (d->ckpt != FW_ACT_NONE && d->in_features % 32) return FW_EUNSUPPORTED;
    if (!grid_ok(grad_tiles(d->n_experts, d->out_features, d->in_features, 2, 128))) return FW_EINVAL;
    return FW_OK;
}

int check_rows(const fw_moe_dense_desc *d, int32_t R) {
    if (R < 0 || R > kMaxRows) return FW_EINVAL;
    const int widest = std::max(d->in_features, d->out_features);
    return grid_ok(rows_tiles(R, d->n_experts, widest)) ? FW_OK : FW_EINVAL;
}

// The checks every product shares; `ptrs` may hold nullptr (not wanted).
int check_call(const fw_moe_dense_desc *d, int32_t R, const int32_t *offsets,
               std::initializer_list<const void *> needed, std::initializer_list<const void *> ptrs,
               const void *workspace, size_t ws_bytes) {
    if (d->n_experts > 1 && !offsets) return FW_EINVAL;
    for (const void *p : needed)
        if (!p) return FW_EINVAL;
    if (!workspace) return FW_EINVAL;
    for (const void *p : needed)
        if (!al16(p)) return FW_EALIGN;
    for (const void *p : ptrs)
        if (!al16(p)) return FW_EALIGN;
    if (!al16(offsets) || !al256(workspace)) return FW_EALIGN;
    if (ws_bytes < dense_ws(*d, R).total) return FW_EWORKSPACE;
    return FW_OK;
}

// What the launches of one call share.
struct Call {
    const fw_moe_dense_desc &d;
    int R;
    const int32_t *offsets;
    char *ws;
    DenseWs L;
    hipStream_t s;

    Call(const fw_moe_dense_desc &desc, int rows, const int32_t *off, void *w, void *stream)
        : d(desc), R(rows), offsets(off), ws((char *)w), L(dense_ws(desc, rows)),
          s((hipStream_t)stream) {}

    int schedule() const {
        return offsets ? hip_status(launch_dense_schedule(offsets, d.n_experts, R,
                                                          tile_rows(tile(8)), L, ws, s))
                       : FW_OK;
    }
    // the tile shape of a product with cols output columns (both matrices')
    DenseTile tile(int cols) const {
        return dense_tile(R, d.n_experts, cols,
                          offsets ? std::max(d.in_features, d.out_features) : 0);
    }
    bool few() const { return few_rows(R, d.n_experts, d.in_features); }
    const int4 *tiles() const { return offsets ? (const int4 *)(ws + L.tiles) : nullptr; }
    // forward-shaped product: x [R][K] times weights [N][K]
    RowsArgs rows(const void *x, const void *w0, const void *w1) const {
        RowsArgs a{};
        a.q = (const uint16_t *)x;
        a.w0 = (const uint16_t *)w0;
        a.w1 = (const uint16_t *)w1;
        a.w_stride = (size_t)d.out_features * d.in_features;
        a.Kd = d.in_features;
        a.nseg = 1;
        a.Np = d.out_features;
        a.R = R;
        a.E = d.n_experts;
        a.fn = d.fn;
        a.tiles = tiles();
        a.hdr = (WsHeader *)ws;
        a.max_tiles = L.max_tiles;
        a.tile = tile(w1 ? 2 * a.Np : a.Np);
        return a;
    }
    // dx = dz0 w0 (+ dz1 w1), dz1 behind dz0; dw0 = dz0^T x (and dw1); db from
    // its row tiles' partials.  Each only where its output is set (part: db's).
    int gradients(const uint16_t *dz, const uint16_t *x, const void *w0, const void *w1, void *dx,
                  void *dw0, void *dw1, const float *part, int part_rows, float *db) const {
        RowsArgs a = rows(dz, w0, w1);
        a.q_seg = (size_t)R * d.out_features;
        a.Kd = d.out_features;
        a.nseg = w1 ? 2 : 1;
        a.Np = d.in_features;
        a.tile = tile(a.Np);
        a.out = dx;
        a.out_f32 = d.grad_dtype == FW_F32;
        const int mats = dw1 ? 2 : 1;
        const size_t bytes = (size_t)mats * d.n_experts * d.out_features * d.in_features *
                             (a.out_f32 ? 4 : 2);
        const GradArgs g{dz, x, R, d.n_experts, d.out_features, d.in_features, mats, offsets, dw0,
                         dw1, a.out_f32, d.accumulate, bytes > ((size_t)256 << 20)};
        const BiasArgs b{part, offsets, R, d.out_features, L.max_tiles, part_rows, db,
                         d.accumulate};
        if (dx && dw0 && !offsets && R > 0) return hip_status(launch_pair(a, g, b, s));
        int rc;
        if (dx && R > 0 && (rc = hip_status(launch_rows(kInput, a, s))) != FW_OK) return rc;
        if (db && (rc = hip_status(launch_bias_grad(b, d.n_experts, s))) != FW_OK) return rc;
        return dw0 ? hip_status(launch_grad(g, s)) : FW_OK;
    }
    // x as bf16: itself, or the checkpoint's values in the workspace
    int values(const void *x, const void *scales, const uint16_t **out) const {
        *out = (const uint16_t *)x;
        if (d.ckpt == FW_ACT_NONE || R == 0) return FW_OK;
        *out = (const uint16_t *)(ws + L.xq);
        return hip_status(launch_ckpt_unpack(d.ckpt, (int64_t)R * (d.in_features / 32), x, scales,
                                             ws + L.xq, 1, s));
    }
};

int check_ckpt(const fw_moe_ckpt_desc *d, int32_t R) {
    if (!d) return FW_EINVAL;
    if (d->features < 32 || d->features > kMaxFeatures || d->features % 32) return FW_EINVAL;
    if (d->format != FW_ACT_MXFP8 && d->format != FW_ACT_INT8) return FW_EINVAL;
    if (!dtype_ok(d->src_dtype) || !dtype_ok(d->dst_dtype)) return FW_EINVAL;
    if (R < 0 || R > kMaxRows) return FW_EINVAL;
    // four lanes a block, 256 a workgroup
    if (!grid_ok(((int64_t)R * (d->features / 32) + 63) / 64)) return FW_EINVAL;
    return FW_OK;
}

}  // namespace

extern "C" {

int fw_moe_dense_validate(const fw_moe_dense_desc *desc) { return check_dense(desc); }

size_t fw_moe_dense_workspace_size(const fw_moe_dense_desc *desc, int32_t max_R) {
    if (check_dense(desc) != FW_OK || check_rows(desc, max_R) != FW_OK) return 0;
    return dense_ws(*desc, max_R).total;
}

int fw_moe_glu_forward(const fw_moe_dense_desc *desc, int32_t R, const void *x,
                       const void *w_gate, const void *w_up, const int32_t *expert_offsets,
                       void *h, void *workspace, size_t ws_bytes, void *stream) {
    int rc = check_dense(desc);
    if (rc != FW_OK) return rc;
    if ((rc = check_rows(desc, R)) != FW_OK) return rc;
    if (R == 0) return FW_OK;
    rc = check_call(desc, R, expert_offsets, {x, w_gate, w_up, h}, {}, workspace, ws_bytes);
    if (rc != FW_OK) return rc;
    const Call c(*desc, R, expert_offsets, workspace, stream);
    RowsArgs a = c.rows(x, w_gate, w_up);
    a.out = h;
    a.out_f32 = desc->out_dtype == FW_F32;
    if (c.few()) return hip_status(launch_few(true, a, expert_offsets, c.s));
    if ((rc = c.schedule()) != FW_OK) return rc;
    return hip_status(launch_rows(kGlu, a, c.s));
}

int fw_moe_glu_backward(const fw_moe_dense_desc *desc, int32_t R, const void *x,
                        const void *x_scales, const void *w_gate, const void *w_up,
                        const int32_t *expert_offsets, const void *dh, void *dx, void *dw_gate,
                        void *dw_up, void *h, void *workspace, size_t ws_bytes, void *stream) {
    int rc = check_dense(desc);
    if (rc != FW_OK) return rc;
    if ((rc = check_rows(desc, R)) != FW_OK) return rc;
    if ((dw_gate == nullptr) != (dw_up == nullptr)) return FW_EINVAL;
    if (!dx && !dw_gate && !h) return FW_EINVAL;
    if (R > 0 && (!x || !dh || (desc->ckpt != FW_ACT_NONE && !x_scales))) return FW_EINVAL;
    rc = check_call(desc, R, expert_offsets, {w_gate, w_up},
                    {x, x_scales, dh, dx, dw_gate, dw_up, h}, workspace, ws_bytes);
    if (rc != FW_OK) return rc;
    const Call c(*desc, R, expert_offsets, workspace, stream);
    const uint16_t *xv;
    uint16_t *dz = (uint16_t *)(c.ws + c.L.dz);
    if ((rc = c.values(x, x_scales, &xv)) != FW_OK) return rc;
    if (R > 0) {
        if ((rc = c.schedule()) != FW_OK) return rc;
        RowsArgs a = c.rows(xv, w_gate, w_up);
        a.dy = (const uint16_t *)dh;
        a.dz = dz;
        a.out = h;
        if ((rc = hip_status(launch_rows(kGluGrad, a, c.s))) != FW_OK) return rc;
    }
    return c.gradients(dz, xv, w_gate, w_up, dx, dw_gate, dw_up, nullptr, 1, nullptr);
}

int fw_moe_linear_forward(const fw_moe_dense_desc *desc, int32_t R, const void *x, const void *w,
                          const float *bias, const void *residual,
                          const int32_t *expert_offsets, void *y, void *workspace,
                          size_t ws_bytes, void *stream) {
    int rc = check_dense(desc);
    if (rc != FW_OK) return rc;
    if ((rc = check_rows(desc, R)) != FW_OK) return rc;
    if (R == 0) return FW_OK;
    rc = check_call(desc, R, expert_offsets, {x, w, y}, {bias, residual}, workspace, ws_bytes);
    if (rc != FW_OK) return rc;
    const Call c(*desc, R, expert_offsets, workspace, stream);
    RowsArgs a = c.rows(x, w, nullptr);
    a.bias = bias;
    a.residual = residual;
    a.out = y;
    a.out_f32 = desc->out_dtype == FW_F32;
    if (c.few()) return hip_status(launch_few(false, a, expert_offsets, c.s));
    if ((rc = c.schedule()) != FW_OK) return rc;
    return hip_status(launch_rows(kLinear, a, c.s));
}

int fw_moe_linear_backward(const fw_moe_dense_desc *desc, int32_t R, const void *x,
                           const void *x_scales, const void *w, const float *bias,
                           const int32_t *expert_offsets, const void *dy, void *dx, void *dw,
                           float *dbias, void *workspace, size_t ws_bytes, void *stream) {
    int rc = check_dense(desc);
    if (rc != FW_OK) return rc;
    if ((rc = check_rows(desc, R)) != FW_OK) return rc;
    if (!dx && !dw && !dbias) return FW_EINVAL;
    const bool act = desc->fn != FW_FN_NONE;
    // x serves dw and the recomputed z, w serves dx and z
    const bool need_x = dw || act, need_w = dx || act;
    if ((need_w && !w) || (R > 0 && !dy)) return FW_EINVAL;
    if (R > 0 && need_x && (!x || (desc->ckpt != FW_ACT_NONE && !x_scales))) return FW_EINVAL;
    rc = check_call(desc, R, expert_offsets, {}, {x, x_scales, w, bias, dy, dx, dw, dbias},
                    workspace, ws_bytes);
    if (rc != FW_OK) return rc;
    const Call c(*desc, R, expert_offsets, workspace, stream);
    const uint16_t *xv = nullptr, *dz = (const uint16_t *)dy;
    float *bpart = (float *)(c.ws + c.L.bpart);
    const int part_rows = tile_rows(c.tile(desc->out_features));
    if (need_x && (rc = c.values(x, x_scales, &xv)) != FW_OK) return rc;
    if (R > 0) {
        if ((rc = c.schedule()) != FW_OK) return rc;
        if (act) {
            RowsArgs a = c.rows(xv, w, nullptr);
            a.bias = bias;
            a.dy = dz;
            a.dz = (uint16_t *)(c.ws + c.L.dz);
            a.bpart = dbias ? bpart : nullptr;
            dz = a.dz;
            if ((rc = hip_status(launch_rows(kLinGrad, a, c.s))) != FW_OK) return rc;
        } else if (dbias) {
            rc = hip_status(launch_colsum(dz, R, desc->out_features, c.tiles(),
                                          (WsHeader *)c.ws, c.L.max_tiles, part_rows, bpart, c.s));
            if (rc != FW_OK) return rc;
        }
    }
    return c.gradients(dz, xv, w, nullptr, dx, dw, nullptr, bpart, part_rows, dbias);
}

int fw_moe_ckpt_pack(const fw_moe_ckpt_desc *desc, int32_t R, const void *x, void *codes,
                     void *scales, void *workspace, void *stream) {
    const int rc = check_ckpt(desc, R);
    if (rc != FW_OK) return rc;
    if (R == 0) return FW_OK;
    if (!x || !codes || !scales || !workspace) return FW_EINVAL;
    if (!al16(x) || !al16(codes) || !al16(scales) || !al256(workspace)) return FW_EALIGN;
    return hip_status(launch_ckpt_pack(desc->format, (int64_t)R * (desc->features / 32), x,
                                       desc->src_dtype == FW_BF16, codes, scales,
                                       (WsHeader *)workspace, (hipStream_t)stream));
}

int fw_moe_ckpt_unpack(const fw_moe_ckpt_desc *desc, int32_t R, const void *codes,
                       const void *scales, void *x, void *stream) {
    const int rc = check_ckpt(desc, R);
    if (rc != FW_OK) return rc;
    if (R == 0) return FW_OK;
    if (!codes || !scales || !x) return FW_EINVAL;
    if (!al16(x) || !al16(codes) || !al16(scales)) return FW_EALIGN;
    return hip_status(launch_ckpt_unpack(desc->format, (int64_t)R * (desc->features / 32), codes,
                                         scales, x, desc->dst_dtype == FW_BF16,
                                         (hipStream_t)stream));
}

}  // extern "C"
