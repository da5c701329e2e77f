// C ABI of the norms around a block (include/sgemm_norm.h): argument checks and
// launches.  Nothing here allocates, copies or synchronises.
#include "api_checks.h"
#include "norm_internal.h"

#include <algorithm>

using namespace sgemm;

namespace {

// Whether some output overlaps another output, or an input that it may not replace:
// bit j of in_place[i] lets output i be input j (same elements at the same places).
template <int NO, int NI>
bool overlaps(const Operand (&out)[NO], const Operand (&in)[NI], const unsigned (&in_place)[NO])
{
    for (int i = 0; i < NO; ++i) {
        for (int j = i + 1; j < NO; ++j)
            if (overlap(out[i], out[j]))
                return true;
        for (int j = 0; j < NI; ++j)
            if (overlap(out[i], in[j]) && !((in_place[i] >> j & 1) && out[i].same(in[j])))
                return true;
    }
    return false;
}

// (a gate for all rows has 0 where there are none)
bool gate_rows_ok(int64_t gate_rows, int64_t rows) { return gate_rows >= (rows > 0 ? 1 : 0); }

Operand vector(const void *p, int64_t n, int size) { return Operand{p, 1, n, n > 1 ? n : 1, size}; }

}  // namespace

extern "C" {

int sgemm_block_norm(int type, int w_type, int64_t rows, int64_t cols, const void *X, int64_t ldx, const void *O,
                     int64_t ldo, const void *W, const void *W_post, const void *GATE, int64_t ldg, int64_t gate_rows,
                     float alpha, float eps, void *H, int64_t ldh, void *Y, int64_t ldy, int q_format, void *Q,
                     int64_t ldq, float *S, int64_t lds, void *H8, int64_t ldh8, float *SH, int64_t ldsh, void *O8,
                     int64_t ldo8, float *SO, int64_t ldso, float *rstd, float *rstd_post, void *stream)
{
    if (!known_type(type) || (w_type != type && w_type != SGEMM_TYPE_F32) || !dim_ok(rows) || cols < 0 ||
        cols > SGEMM_RMSNORM_MAX_COLS || !(eps >= 0.0f) || std::isinf(eps) || !std::isfinite(alpha) ||
        (Q && q_format != SGEMM_F8_E4M3 && q_format != SGEMM_Q_I8))
        return SGEMM_ERR_INVALID_VALUE;
    if (!O)
        W_post = GATE = O8 = nullptr;
    if (!W_post)
        rstd_post = nullptr;
    if (GATE && !gate_rows_ok(gate_rows, rows))
        return SGEMM_ERR_INVALID_VALUE;
    if (!GATE || gate_rows > rows || rows == 0)
        gate_rows = rows > 0 ? rows : 1;
    const int size = type_bytes(type), w_size = type_bytes(w_type);
    const bool q_i8 = q_format == SGEMM_Q_I8;
    const Operand ox{X, rows, cols, ldx, size}, oo{O, rows, cols, ldo, size};
    const Operand og{GATE, ceil_div(rows, gate_rows), cols, ldg, w_size};
    const Operand ow = vector(Y || Q ? W : nullptr, cols, w_size), owp = vector(W_post, cols, w_size);
    const Operand oh{H, rows, cols, ldh, size}, oy{Y, rows, cols, ldy, size}, oq{Q, rows, cols, ldq, 1};
    const Operand oh8{H8, rows, cols, ldh8, 1}, oo8{O8, rows, cols, ldo8, 1};
    const Operand os = q_i8 ? vector(Q ? S : nullptr, rows, 4) : scales(Q ? S : nullptr, SGEMM_F8_ROW, rows, cols, lds);
    const Operand osh = scales(H8 ? SH : nullptr, SGEMM_F8_ROW, rows, cols, ldsh);
    const Operand oso = scales(O8 ? SO : nullptr, SGEMM_F8_ROW, rows, cols, ldso);
    const Operand ors = vector(rstd, rows, 4), orp = vector(rstd_post, rows, 4);
    if (!ox.shape_ok() || (O && !oo.shape_ok()) || (GATE && !og.shape_ok()) || (H && !oh.shape_ok()) ||
        (Y && !oy.shape_ok()) || (Q && (!oq.shape_ok() || !os.shape_ok())) ||
        (H8 && (!oh8.shape_ok() || !osh.shape_ok())) || (O8 && (!oo8.shape_ok() || !oso.shape_ok())))
        return SGEMM_ERR_INVALID_VALUE;
    if (rows == 0 || cols == 0 || (!H && !Y && !Q && !H8 && !O8 && !rstd && !rstd_post))
        return SGEMM_OK;
    if (!ox.present() || (O && !oo.present()) || (GATE && !og.present()) || ((Y || Q) && !ow.present()) ||
        (W_post && !owp.present()) || (H && !oh.present()) || (Y && !oy.present()) || (Q && !os.present()) ||
        (H8 && !osh.present()) || (O8 && !oso.present()) || (rstd && !ors.present()) || (rstd_post && !orp.present()))
        return SGEMM_ERR_INVALID_VALUE;
    const Operand outs[10] = {oh, oy, oq, os, oh8, osh, oo8, oso, ors, orp}, ins[5] = {ox, oo, og, ow, owp};
    const unsigned in_place[10] = {0b00011u};  // H may be X or O
    if (overlaps(outs, ins, in_place))
        return SGEMM_ERR_ALIAS;
    if (rmsnorm_work_items(rows, cols) > kMaxWorkItems)
        return SGEMM_ERR_INVALID_VALUE;
    const int dev = sgemm_f32_device_status();
    if (dev != SGEMM_OK)
        return dev;
    BlockNormArgs a;
    a.X = X;
    a.O = O;
    a.W = W;
    a.WP = W_post;
    a.G = GATE;
    a.H = H;
    a.Y = Y;
    a.Q = static_cast<uint8_t *>(Q);
    a.H8 = static_cast<uint8_t *>(H8);
    a.O8 = static_cast<uint8_t *>(O8);
    a.S = S;
    a.SH = SH;
    a.SO = SO;
    a.rstd = rstd;
    a.rstd_post = rstd_post;
    a.ldx = ldx;
    a.ldo = ldo;
    a.ldg = ldg;
    a.ldh = ldh;
    a.ldy = ldy;
    a.ldq = ldq;
    a.lds = lds;
    a.ldh8 = ldh8;
    a.ldsh = ldsh;
    a.ldo8 = ldo8;
    a.ldso = ldso;
    a.rows = (int)rows;
    a.cols = (int)cols;
    a.gate_rows = (int)gate_rows;
    a.alpha = alpha;
    a.eps = eps;
    a.w_f32 = w_type == SGEMM_TYPE_F32;
    a.q_i8 = q_i8;
    (void)hipGetLastError();
    return finish(launch_block_norm(a, type, reinterpret_cast<hipStream_t>(stream)));
}

int sgemm_block_norm_bwd_plan(int64_t rows, int64_t cols, int64_t gate_rows, int64_t *workspace_bytes)
{
    if (!dim_ok(rows) || cols < 0 || cols > SGEMM_RMSNORM_MAX_COLS || gate_rows < 0)
        return SGEMM_ERR_INVALID_VALUE;
    // A call that reads its gate for no output sums as one without a gate, which can be more
    // arrays: 129 to 256 gates of 513 to 1024 columns have a workgroup each.
    if (workspace_bytes)
        *workspace_bytes = std::max(block_norm_sums(rows, cols, gate_rows).parts, block_norm_sums(rows, cols, 0).parts) * cols * 4;
    return SGEMM_OK;
}

int sgemm_block_norm_bwd(int type, int w_type, int64_t rows, int64_t cols, const void *DY, int64_t lddy,
                         const void *DH, int64_t lddh, int kept, const void *H, int64_t ldh, const float *SH,
                         int64_t ldsh, const void *O, int64_t ldo, const float *SO, int64_t ldso, const void *W,
                         const void *W_post, const float *rstd, const float *rstd_post, const void *GATE, int64_t ldg,
                         int64_t gate_rows, float alpha, void *DX, int64_t lddx, void *DO, int64_t lddo, float *DW,
                         float *DW_post, float *DGATE, int64_t lddg, void *workspace, int64_t workspace_bytes,
                         void *stream)
{
    if (!known_type(type) || (w_type != type && w_type != SGEMM_TYPE_F32) || !dim_ok(rows) || cols < 0 ||
        cols > SGEMM_RMSNORM_MAX_COLS || (kept != 0 && kept != 1) || workspace_bytes < 0 || !std::isfinite(alpha) ||
        (GATE && !gate_rows_ok(gate_rows, rows)))
        return SGEMM_ERR_INVALID_VALUE;
    // (operands without rows may be NULL)
    if (rows > 0 && cols > 0 &&
        ((!DY && !DH) || (DW_post && !W_post) || (DGATE && !GATE) || ((W_post || DGATE) && !O)))
        return SGEMM_ERR_INVALID_VALUE;
    if (rows == 0) {
        GATE = W_post = nullptr;
        DGATE = nullptr;
    }
    // what no output needs is not read
    if (!DO && !DW_post && !DGATE)
        GATE = W_post = nullptr;
    const bool read_o = W_post || DGATE, sums = DW || DW_post || DGATE;
    if (!GATE || gate_rows > rows)
        gate_rows = rows > 0 ? rows : 1;
    const int size = type_bytes(type), w_size = type_bytes(w_type), k_size = kept ? 1 : size;
    const int64_t gates = ceil_div(rows, gate_rows);
    const Operand ody{DY, rows, cols, lddy, size}, odh{DH, rows, cols, lddh, size};
    const Operand oh{DY ? H : nullptr, rows, cols, ldh, k_size}, oo{read_o ? O : nullptr, rows, cols, ldo, k_size};
    const Operand osh = scales(kept && DY ? SH : nullptr, SGEMM_F8_ROW, rows, cols, ldsh);
    const Operand oso = scales(kept && read_o ? SO : nullptr, SGEMM_F8_ROW, rows, cols, ldso);
    const Operand ow = vector(DY ? W : nullptr, cols, w_size), owp = vector(W_post, cols, w_size);
    const Operand ors = vector(DY ? rstd : nullptr, rows, 4), orp = vector(W_post ? rstd_post : nullptr, rows, 4);
    const Operand og{GATE, gates, cols, ldg, w_size}, odg{DGATE, gates, cols, lddg, 4};
    const Operand odx{DX, rows, cols, lddx, size}, odo{DO, rows, cols, lddo, size};
    const Operand odw = vector(DW, cols, 4), odwp = vector(DW_post, cols, 4);
    const Operand ows{sums ? workspace : nullptr, 1, workspace_bytes, workspace_bytes, 1};
    if ((DY && (!ody.shape_ok() || !oh.shape_ok() || (kept && !osh.shape_ok()))) || (DH && !odh.shape_ok()) ||
        (read_o && (!oo.shape_ok() || (kept && !oso.shape_ok()))) || (GATE && !og.shape_ok()) ||
        (DX && !odx.shape_ok()) || (DO && !odo.shape_ok()) || (DGATE && !odg.shape_ok()))
        return SGEMM_ERR_INVALID_VALUE;
    if (cols == 0 || (rows == 0 && !sums) || (!DX && !DO && !sums))
        return SGEMM_OK;
    if ((DW && !odw.present()) || (DW_post && !odwp.present()))
        return SGEMM_ERR_INVALID_VALUE;
    if (rows > 0 &&
        ((DY && (!ody.present() || !oh.present() || (kept && !osh.present()) || !ow.present() || !ors.present())) ||
         (DH && !odh.present()) || (read_o && (!oo.present() || (kept && !oso.present()))) ||
         (W_post && (!owp.present() || !orp.present())) || (GATE && !og.present()) || (DX && !odx.present()) ||
         (DO && !odo.present()) || (DGATE && !odg.present())))
        return SGEMM_ERR_INVALID_VALUE;
    const int64_t need = sums ? block_norm_sums(rows, cols, gate_rows).parts * cols * 4 : 0;
    if (need > 0 && (!on(workspace, 16) || workspace_bytes < need))
        return SGEMM_ERR_INVALID_VALUE;
    const Operand outs[6] = {odx, odo, odw, odwp, odg, ows};
    const Operand ins[11] = {ody, odh, oh, oo, osh, oso, ow, owp, ors, orp, og};
    // DX may be DY, DH or H, DO may be DY, DH or O
    const unsigned in_place[6] = {kept ? 0b0011u : 0b0111u, kept ? 0b0011u : 0b1011u};
    if (rows > 0 && overlaps(outs, ins, in_place))
        return SGEMM_ERR_ALIAS;
    const int dev = sgemm_f32_device_status();
    if (dev != SGEMM_OK)
        return dev;
    BlockNormBwdArgs a;
    a.DY = DY;
    a.DH = DH;
    a.H = H;
    a.O = read_o ? O : nullptr;
    a.W = W;
    a.WP = W_post;
    a.G = GATE;
    a.SH = SH;
    a.SO = SO;
    a.rstd = rstd;
    a.rstd_post = rstd_post;
    a.DX = DX;
    a.DO = DO;
    a.DW = DW;
    a.DWP = DW_post;
    a.DG = DGATE;
    a.ws = static_cast<float *>(workspace);
    a.lddy = lddy;
    a.lddh = lddh;
    a.ldh = ldh;
    a.ldsh = ldsh;
    a.ldo = ldo;
    a.ldso = ldso;
    a.ldg = ldg;
    a.lddx = lddx;
    a.lddo = lddo;
    a.lddg = lddg;
    a.rows = (int)rows;
    a.cols = (int)cols;
    a.gate_rows = (int)gate_rows;
    a.alpha = alpha;
    a.w_f32 = w_type == SGEMM_TYPE_F32;
    a.groups = a.team = a.chunk = 0;
    (void)hipGetLastError();
    return finish(launch_block_norm_bwd(a, type, kept == 1, reinterpret_cast<hipStream_t>(stream)));
}

}  // extern "C"
