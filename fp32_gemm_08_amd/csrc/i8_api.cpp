// C ABI of the products of 8-bit integers (include/sgemm_i8.h): argument checks and
// launches.  Nothing here allocates, copies or synchronises.
#include "api_checks.h"
#include "i8_internal.h"

using namespace sgemm;

namespace {

bool dims_ok(int64_t M, int64_t N, int64_t K) { return dim_ok(M) && dim_ok(N) && K >= 0 && K <= SGEMM_I8_MAX_K; }

// Whether the plan's grid is within one launch.
bool launchable(const I8GemmPlan &p) { return p.tiles_m * p.tiles_n * p.splits * p.threads <= kMaxWorkItems; }

}  // namespace

extern "C" {

int sgemm_i8_gemm_plan(int64_t M, int64_t N, int64_t K, int aligned, int *kernel_id, int64_t *tiles_m,
                       int64_t *tiles_n, int64_t *splits, int64_t *workspace_bytes)
{
    if (!dims_ok(M, N, K) || (aligned != 0 && aligned != 1))
        return SGEMM_ERR_INVALID_VALUE;
    I8GemmPlan p;
    if (M > 0 && N > 0 && K > 0) {
        p = i8_gemm_plan(M, N, K, aligned == 1, kAnyRoom, false);
        if (!launchable(p))
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

int sgemm_i8_gemm_workspace(int64_t M, int64_t N, int64_t K, int aligned, int64_t *workspace_bytes)
{
    if (!dims_ok(M, N, K) || (aligned != 0 && aligned != 1))
        return SGEMM_ERR_INVALID_VALUE;
    if (workspace_bytes)
        *workspace_bytes = M > 0 && N > 0 && K > 0 ? i8_gemm_plan(M, N, K, aligned == 1, kAnyRoom, true).bytes : 0;
    return SGEMM_OK;
}

int sgemm_i8_gemm(int c_type, int64_t M, int64_t N, int64_t K, float alpha, const int8_t *A, int64_t lda,
                  const float *SA, const int8_t *B, int64_t ldb, const float *SB, float beta, void *C, int64_t ldc,
                  void *workspace, int64_t workspace_bytes, void *stream)
{
    if (!known_type(c_type) || !dims_ok(M, N, K) || workspace_bytes < 0)
        return SGEMM_ERR_INVALID_VALUE;
    const Operand oa{A, M, K, lda, 1}, ob{B, N, K, ldb, 1}, oc{C, M, N, ldc, type_bytes(c_type)};
    const Operand osa{SA, 1, M, M > 1 ? M : 1, 4}, osb{SB, 1, N, N > 1 ? N : 1, 4};
    const Operand ows{workspace, 1, workspace_bytes, workspace_bytes, 1};
    if (!oa.shape_ok() || !ob.shape_ok() || !oc.shape_ok())
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
    I8GemmArgs a;
    a.A = reinterpret_cast<const uint8_t *>(A);
    a.B = reinterpret_cast<const uint8_t *>(B);
    a.SA = SA;
    a.SB = SB;
    a.C = C;
    a.ws = static_cast<int *>(workspace);
    a.lda = lda;
    a.ldb = ldb;
    a.ldc = ldc;
    a.M = (int)M;
    a.N = (int)N;
    a.K = (int)K;
    a.tiles_m = a.tiles_n = a.kb_split = 0;
    a.alpha = alpha;
    a.beta = beta;
    a.c_type = c_type;
    const bool aligned = oa.rows_on(16) && ob.rows_on(16) && (M <= 1 || lda <= F8_MAX_LD) && (N <= 1 || ldb <= F8_MAX_LD);
    const I8GemmPlan p = i8_gemm_plan(M, N, K, aligned, workspace ? workspace_bytes : 0, true);
    if (!launchable(p))
        return SGEMM_ERR_INVALID_VALUE;
    const int dev = sgemm_f32_device_status();
    if (dev != SGEMM_OK)
        return dev;
    (void)hipGetLastError();
    return finish(launch_i8_gemm(a, p, reinterpret_cast<hipStream_t>(stream)));
}

int sgemm_i8_quantize(int x_type, int64_t rows, int64_t cols, const void *X, int64_t ldx, int8_t *Q, int64_t ldq,
                      float *S, void *stream)
{
    if (!known_type(x_type) || !dim_ok(rows) || !dim_ok(cols))
        return SGEMM_ERR_INVALID_VALUE;
    const Operand ox{X, rows, cols, ldx, type_bytes(x_type)}, oq{Q, rows, cols, ldq, 1};
    const Operand os{S, 1, rows, rows > 1 ? rows : 1, 4};
    if (!ox.shape_ok() || !oq.shape_ok())
        return SGEMM_ERR_INVALID_VALUE;
    if (rows == 0 || cols == 0)
        return SGEMM_OK;
    if (!ox.present() || !oq.present() || !os.present())
        return SGEMM_ERR_INVALID_VALUE;
    const Operand outs[2] = {oq, os}, ins[1] = {ox};
    if (aliased(outs, ins, -1, 0))
        return SGEMM_ERR_ALIAS;
    if (i8_quantize_work_items(rows, cols) > kMaxWorkItems)
        return SGEMM_ERR_INVALID_VALUE;
    const int dev = sgemm_f32_device_status();
    if (dev != SGEMM_OK)
        return dev;
    I8QuantArgs a;
    a.X = X;
    a.Q = reinterpret_cast<uint8_t *>(Q);
    a.S = S;
    a.ldx = ldx;
    a.ldq = ldq;
    a.rows = (int)rows;
    a.cols = (int)cols;
    (void)hipGetLastError();
    return finish(launch_i8_quantize(a, x_type, reinterpret_cast<hipStream_t>(stream)));
}

}  // extern "C"
