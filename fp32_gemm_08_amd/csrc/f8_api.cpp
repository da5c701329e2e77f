// C ABI of the 8-bit block-scaled family (include/sgemm_f8.h): argument checks
// and launches.  Nothing here allocates, copies or synchronises.
#include "api_checks.h"
#include "sgemm_f8.h"

using namespace sgemm;

namespace {

int threads_of(int kid) { return kid == KID_F8_ANY ? 256 : 512; }

}  // namespace

extern "C" {

int sgemm_f8_gemm_plan(int b_block, int64_t M, int64_t N, int64_t K, int aligned, int *kernel_id,
                       int64_t *tiles_m, int64_t *tiles_n, int64_t *splits, int64_t *workspace_bytes)
{
    if (!known_block(b_block) || !dim_ok(M) || !dim_ok(N) || !dim_ok(K) || (aligned != 0 && aligned != 1))
        return SGEMM_ERR_INVALID_VALUE;
    F8GemmPlan p;
    if (M > 0 && N > 0 && K > 0) {
        p = f8_gemm_plan(b_block == SGEMM_F8_ROW, M, N, K, aligned == 1, kAnyRoom, false);
        if (p.tiles_m * p.tiles_n * p.splits * threads_of(p.kid) > kMaxWorkItems)
            return SGEMM_ERR_INVALID_VALUE;
    }
    if (kernel_id)
        *kernel_id = p.kid;
    if (tiles_m)
        *tiles_m = p.tiles_m;
    if (tiles_n)
        *tiles_n = p.tiles_n;
    if (splits)
        *splits = p.splits;
    if (workspace_bytes)
        *workspace_bytes = p.bytes;
    return SGEMM_OK;
}

int sgemm_f8_gemm_workspace(int b_block, int64_t M, int64_t N, int64_t K, int aligned, int64_t *workspace_bytes)
{
    if (!known_block(b_block) || !dim_ok(M) || !dim_ok(N) || !dim_ok(K) || (aligned != 0 && aligned != 1))
        return SGEMM_ERR_INVALID_VALUE;
    if (workspace_bytes)
        *workspace_bytes = M > 0 && N > 0 && K > 0
                               ? f8_gemm_plan(b_block == SGEMM_F8_ROW, M, N, K, aligned == 1, kAnyRoom, true).bytes
                               : 0;
    return SGEMM_OK;
}

int sgemm_f8_gemm(int format_a, int format_b, int b_block, int c_type, int64_t M, int64_t N, int64_t K,
                  float alpha, const void *A, int64_t lda, const float *SA, int64_t ldsa, const void *B,
                  int64_t ldb, const float *SB, int64_t ldsb, float beta, void *C, int64_t ldc,
                  void *workspace, int64_t workspace_bytes, void *stream)
{
    if (!known_format(format_a) || !known_format(format_b) || !known_block(b_block) || !known_type(c_type) ||
        !dim_ok(M) || !dim_ok(N) || !dim_ok(K) || workspace_bytes < 0)
        return SGEMM_ERR_INVALID_VALUE;
    const Operand oa{A, M, K, lda, 1}, ob{B, N, K, ldb, 1}, oc{C, M, N, ldc, type_bytes(c_type)};
    const Operand osa = scales(SA, SGEMM_F8_ROW, M, K, ldsa), osb = scales(SB, b_block, N, K, ldsb);
    const Operand ows{workspace, 1, workspace_bytes, workspace_bytes, 1};
    if (!oa.shape_ok() || !ob.shape_ok() || !oc.shape_ok() || !osa.shape_ok() || !osb.shape_ok())
        return SGEMM_ERR_INVALID_VALUE;
    if (M == 0 || N == 0)
        return SGEMM_OK;
    if (!oc.present())
        return SGEMM_ERR_INVALID_VALUE;
    const bool product = alpha != 0.0f && K > 0;
    if (!product && beta == 1.0f)
        return SGEMM_OK;
    if (!product) {
        const int dev = sgemm_f32_device_status();
        if (dev != SGEMM_OK)
            return dev;
        (void)hipGetLastError();
        return finish(launch_f8_scale(C, ldc, (int)M, (int)N, c_type, beta, reinterpret_cast<hipStream_t>(stream)));
    }
    if (!oa.present() || !ob.present() || !osa.present() || !osb.present() ||
        (workspace != nullptr && !on(workspace, 16)))
        return SGEMM_ERR_INVALID_VALUE;
    const Operand outs[2] = {oc, ows}, ins[4] = {oa, ob, osa, osb};
    if (aliased(outs, ins, -1, 0))
        return SGEMM_ERR_ALIAS;
    F8GemmArgs a;
    a.A = static_cast<const uint8_t *>(A);
    a.B = static_cast<const uint8_t *>(B);
    a.SA = SA;
    a.SB = SB;
    a.C = C;
    a.ws = static_cast<float *>(workspace);
    a.lda = lda;
    a.ldb = ldb;
    a.ldsa = ldsa;
    a.ldsb = ldsb;
    a.ldc = ldc;
    a.M = (int)M;
    a.N = (int)N;
    a.K = (int)K;
    a.kb_split = 0;
    a.alpha = alpha;
    a.beta = beta;
    a.c_type = c_type;
    const F8GemmPlan p = f8_call_plan(a, oa.rows_on(16) && ob.rows_on(16), b_block == SGEMM_F8_ROW,
                                      workspace ? workspace_bytes : 0);
    if (p.tiles_m * p.tiles_n * p.splits * threads_of(p.kid) > kMaxWorkItems)
        return SGEMM_ERR_INVALID_VALUE;
    const int dev = sgemm_f32_device_status();
    if (dev != SGEMM_OK)
        return dev;
    (void)hipGetLastError();
    return finish(launch_f8_gemm(a, p, format_a, format_b, b_block == SGEMM_F8_ROW,
                                 reinterpret_cast<hipStream_t>(stream)));
}

int sgemm_f8_quantize(int block, int format, int x_type, int64_t rows, int64_t cols, const void *X, int64_t ldx,
                      void *Q, int64_t ldq, float *S, int64_t lds, void *QT, int64_t ldqt, float *ST,
                      int64_t ldst, void *stream)
{
    if (!known_block(block) || !known_format(format) || !known_type(x_type) || !dim_ok(rows) || !dim_ok(cols))
        return SGEMM_ERR_INVALID_VALUE;
    const Operand ox{X, rows, cols, ldx, type_bytes(x_type)};
    const Operand oq{Q, rows, cols, ldq, 1}, oqt{QT, cols, rows, ldqt, 1};
    const Operand os = scales(Q ? S : nullptr, block, rows, cols, lds);
    const Operand ost = scales(QT ? ST : nullptr, block, cols, rows, ldst);
    if (!ox.shape_ok() || (Q && (!oq.shape_ok() || !os.shape_ok())) || (QT && (!oqt.shape_ok() || !ost.shape_ok())))
        return SGEMM_ERR_INVALID_VALUE;
    if (rows == 0 || cols == 0 || (!Q && !QT))
        return SGEMM_OK;
    if (!ox.present() || (Q && !os.present()) || (QT && !ost.present()))
        return SGEMM_ERR_INVALID_VALUE;
    const Operand outs[4] = {oq, os, oqt, ost}, ins[1] = {ox};
    if (aliased(outs, ins, -1, 0))
        return SGEMM_ERR_ALIAS;
    if (ceil_div(rows, F8_BLOCK) * ceil_div(cols, F8_BLOCK) * 256 > kMaxWorkItems)
        return SGEMM_ERR_INVALID_VALUE;
    const int dev = sgemm_f32_device_status();
    if (dev != SGEMM_OK)
        return dev;
    F8QuantArgs a;
    a.X = X;
    a.Q = static_cast<uint8_t *>(Q);
    a.QT = static_cast<uint8_t *>(QT);
    a.S = S;
    a.ST = ST;
    a.ldx = ldx;
    a.ldq = ldq;
    a.lds = lds;
    a.ldqt = ldqt;
    a.ldst = ldst;
    a.rows = (int)rows;
    a.cols = (int)cols;
    a.tiles_c = 0;
    (void)hipGetLastError();
    return finish(launch_f8_quantize(a, block == SGEMM_F8_TILE, format, x_type, reinterpret_cast<hipStream_t>(stream)));
}

int sgemm_f8_requantize(int format_x, int format, int64_t rows, int64_t cols, const void *X, int64_t ldx,
                        const float *SX, int64_t ldsx, void *QT, int64_t ldqt, float *ST, int64_t ldst, void *stream)
{
    if (!known_format(format_x) || !known_format(format) || !dim_ok(rows) || !dim_ok(cols))
        return SGEMM_ERR_INVALID_VALUE;
    const Operand ox{X, rows, cols, ldx, 1}, oqt{QT, cols, rows, ldqt, 1};
    const Operand osx = scales(SX, SGEMM_F8_ROW, rows, cols, ldsx), ost = scales(ST, SGEMM_F8_ROW, cols, rows, ldst);
    if (!ox.shape_ok() || !osx.shape_ok() || !oqt.shape_ok() || !ost.shape_ok())
        return SGEMM_ERR_INVALID_VALUE;
    if (rows == 0 || cols == 0)
        return SGEMM_OK;
    if (!ox.present() || !osx.present() || !oqt.present() || !ost.present())
        return SGEMM_ERR_INVALID_VALUE;
    const Operand outs[2] = {oqt, ost}, ins[2] = {ox, osx};
    if (aliased(outs, ins, -1, 0))
        return SGEMM_ERR_ALIAS;
    if (ceil_div(rows, F8_BLOCK) * ceil_div(cols, F8_BLOCK) * 256 > kMaxWorkItems)
        return SGEMM_ERR_INVALID_VALUE;
    const int dev = sgemm_f32_device_status();
    if (dev != SGEMM_OK)
        return dev;
    F8QuantArgs a;
    a.X = X;
    a.Q = nullptr;
    a.QT = static_cast<uint8_t *>(QT);
    a.S = nullptr;
    a.ST = ST;
    a.ldx = ldx;
    a.ldq = a.lds = 0;
    a.ldqt = ldqt;
    a.ldst = ldst;
    a.rows = (int)rows;
    a.cols = (int)cols;
    a.tiles_c = 0;
    a.SX = SX;
    a.ldsx = ldsx;
    (void)hipGetLastError();
    return finish(launch_f8_requantize(a, format_x, format, reinterpret_cast<hipStream_t>(stream)));
}

int sgemm_f8_rmsnorm(int type, int w_type, int64_t rows, int64_t cols, const void *X, int64_t ldx, const void *R,
                     int64_t ldr, const void *W, float eps, void *H, int64_t ldh, void *Y, int64_t ldy, void *Q,
                     int64_t ldq, float *S, int64_t lds, float *rstd, void *stream)
{
    if (!known_type(type) || (w_type != type && w_type != SGEMM_TYPE_F32) || !dim_ok(rows) || cols < 0 ||
        cols > SGEMM_RMSNORM_MAX_COLS || !(eps >= 0.0f) || std::isinf(eps))
        return SGEMM_ERR_INVALID_VALUE;
    const int size = type_bytes(type);
    const Operand ox{X, rows, cols, ldx, size}, orr{R, rows, cols, ldr, size};
    const Operand ow{W, 1, cols, cols > 1 ? cols : 1, type_bytes(w_type)};
    const Operand oh{H, rows, cols, ldh, size}, oy{Y, rows, cols, ldy, size}, oq{Q, rows, cols, ldq, 1};
    const Operand os = scales(Q ? S : nullptr, SGEMM_F8_ROW, rows, cols, lds);
    const Operand ors{rstd, 1, rows, rows > 1 ? rows : 1, 4};
    if (!ox.shape_ok() || (R && !orr.shape_ok()) || (H && !oh.shape_ok()) || (Y && !oy.shape_ok()) ||
        (Q && (!oq.shape_ok() || !os.shape_ok())))
        return SGEMM_ERR_INVALID_VALUE;
    if (rows == 0 || cols == 0 || (!H && !Y && !Q && !rstd))
        return SGEMM_OK;
    if (!ox.present() || !ow.present() || (R && !orr.present()) || (H && !oh.present()) || (Y && !oy.present()) ||
        (Q && !os.present()) || (rstd && !ors.present()))
        return SGEMM_ERR_INVALID_VALUE;
    const Operand outs[5] = {oh, oy, oq, os, ors}, ins[3] = {ox, orr, ow};
    if (aliased(outs, ins, 0, 0b011u))
        return SGEMM_ERR_ALIAS;
    if (rmsnorm_work_items(rows, cols) > kMaxWorkItems)
        return SGEMM_ERR_INVALID_VALUE;
    const int dev = sgemm_f32_device_status();
    if (dev != SGEMM_OK)
        return dev;
    NormArgs a;
    a.X = X;
    a.R = R;
    a.W = W;
    a.H = H;
    a.Y = Y;
    a.Q = static_cast<uint8_t *>(Q);
    a.S = S;
    a.rstd = rstd;
    a.ldx = ldx;
    a.ldr = ldr;
    a.ldh = ldh;
    a.ldy = ldy;
    a.ldq = ldq;
    a.lds = lds;
    a.rows = (int)rows;
    a.cols = (int)cols;
    a.eps = eps;
    a.w_f32 = w_type == SGEMM_TYPE_F32;
    (void)hipGetLastError();
    return finish(launch_rmsnorm(a, type, reinterpret_cast<hipStream_t>(stream)));
}

int sgemm_f8_rmsnorm_bwd_plan(int64_t rows, int64_t cols, int64_t *workspace_bytes)
{
    if (!dim_ok(rows) || cols < 0 || cols > SGEMM_RMSNORM_MAX_COLS)
        return SGEMM_ERR_INVALID_VALUE;
    if (workspace_bytes)
        *workspace_bytes = rmsnorm_bwd_groups(rows, cols) * cols * 4;
    return SGEMM_OK;
}

int sgemm_f8_rmsnorm_bwd(int type, int w_type, int64_t rows, int64_t cols, const void *DY, int64_t lddy,
                         const void *H, int64_t ldh, const void *W, const float *rstd, const void *DH, int64_t lddh,
                         void *DX, int64_t lddx, float *DW, void *workspace, int64_t workspace_bytes, void *stream)
{
    if (!known_type(type) || (w_type != type && w_type != SGEMM_TYPE_F32) || !dim_ok(rows) || cols < 0 ||
        cols > SGEMM_RMSNORM_MAX_COLS || workspace_bytes < 0)
        return SGEMM_ERR_INVALID_VALUE;
    const int size = type_bytes(type);
    const Operand ody{DY, rows, cols, lddy, size}, oh{H, rows, cols, ldh, size}, odh{DH, rows, cols, lddh, size};
    const Operand ow{W, 1, cols, cols > 1 ? cols : 1, type_bytes(w_type)};
    const Operand ors{rstd, 1, rows, rows > 1 ? rows : 1, 4};
    const Operand odx{DX, rows, cols, lddx, size}, odw{DW, 1, cols, cols > 1 ? cols : 1, 4};
    const Operand ows{DW ? workspace : nullptr, 1, workspace_bytes, workspace_bytes, 1};
    if (!ody.shape_ok() || !oh.shape_ok() || (DH && !odh.shape_ok()) || !odx.shape_ok())
        return SGEMM_ERR_INVALID_VALUE;
    if (cols == 0 || (rows == 0 && !DW))
        return SGEMM_OK;
    if (DW && !odw.present())
        return SGEMM_ERR_INVALID_VALUE;
    if (rows > 0 && (!ody.present() || !oh.present() || !ow.present() || !ors.present() || (DH && !odh.present()) ||
                     !odx.present()))
        return SGEMM_ERR_INVALID_VALUE;
    const int64_t groups = rmsnorm_bwd_groups(rows, cols);
    if (DW && groups > 0 && (!on(workspace, 16) || workspace_bytes < groups * cols * 4))
        return SGEMM_ERR_INVALID_VALUE;
    const Operand outs[3] = {odx, odw, ows}, ins[5] = {ody, oh, odh, ow, ors};
    if (aliased(outs, ins, 0, 0b00111u))
        return SGEMM_ERR_ALIAS;
    const int dev = sgemm_f32_device_status();
    if (dev != SGEMM_OK)
        return dev;
    NormBwdArgs a;
    a.DY = DY;
    a.H = H;
    a.W = W;
    a.DH = DH;
    a.rstd = rstd;
    a.DX = DX;
    a.DW = DW;
    a.ws = static_cast<float *>(workspace);
    a.lddy = lddy;
    a.ldh = ldh;
    a.lddh = lddh;
    a.lddx = lddx;
    a.rows = (int)rows;
    a.cols = (int)cols;
    a.groups = (int)groups;
    a.w_f32 = w_type == SGEMM_TYPE_F32;
    (void)hipGetLastError();
    return finish(launch_rmsnorm_bwd(a, type, reinterpret_cast<hipStream_t>(stream)));
}

}  // extern "C"
