// abi_matmul.hip -- the extern "C" entry points of the products whose both
// operands are e4m3, of their quantizer, and of the gradients of routed rows:
// argument validation, then launch.
//
// As in abi.hip, validation looks at pointer values, dimensions and sizes
// only, so a refused call is safe with any pointers.
#include "qg_check.h"
#include "qg_matmul.h"

namespace {

using namespace qg;

// Operands, sizes and epilogue of a product; a status.
int fill(MatmulArgs &p, const void *w, const float *scale_inv, const void *x, long long ldx,
         const float *x_scale, long long lds, int T, void *y, long long ldy, int R, int I, int O,
         int dtype, const qgemv_epilogue *epilogue, bool with_residual)
{
    LinearArgs &a = p.a;
    a.w = static_cast<const uint8_t *>(w);
    a.scales = scale_inv;
    a.x = x;
    a.ldx = ldx;
    a.y = y;
    a.ldy = ldy;
    a.T = T;
    a.R = R;
    a.I = I;
    a.O = O;
    a.gs = 128;
    a.ng = (I + 127) / 128;
    a.dtype = dtype;
    p.xs = x_scale;
    p.ldxs = lds;
    if (int e = take(a, 1, epilogue, with_residual)) return e;
    if (lds < a.ng) return QGEMV_E_DIMS;
    return misaligned(x_scale, 4) ? QGEMV_E_ALIGN : QGEMV_OK;
}

bool overlapping(const MatmulArgs &p, const void *workspace, size_t ws_bytes)
{
    const LinearArgs &a = p.a;
    return qg::overlapping(a, 1, (long long)a.O * a.I, 4LL * a.ng * ((a.O + 127) / 128), workspace,
                           ws_bytes, rows_of(p.xs, a.T, 4LL * a.ng, 4 * p.ldxs));
}

bool bad_routed(int T, int K, int R, int I)
{
    return T < 0 || T > MAX_DIM || R < 0 || R > MAX_DIM || K < 1 || K > 64 || I < 1 || I > MAX_DIM;
}

}  // namespace

extern "C" {

int qgemv_fp8_quantize(const void *x, long long ldx, int S, int I, int dtype, void *codes,
                       long long ldc, float *scales, long long lds, void *stream)
{
    if (bad_sizes(S, I, 1)) return QGEMV_E_DIMS;
    if (bad_dtype(dtype)) return QGEMV_E_ARG;
    if (S > 0 && (!x || !codes || !scales)) return QGEMV_E_NULL;
    const long long ng = (I + 127) / 128, el = element(dtype);
    if (ldx < I || ldc < I || lds < ng) return QGEMV_E_DIMS;
    if (misaligned(x, el) || misaligned(scales, 4)) return QGEMV_E_ALIGN;
    if (S == 0) return QGEMV_OK;
    const Rows all[] = {rows_of(x, S, I * el, ldx * el), rows_of(codes, S, I, ldc),
                        rows_of(scales, S, 4 * ng, 4 * lds)};
    if (overlaps_any(all[1], all, 1) || overlaps_any(all[2], all, 2)) return QGEMV_E_OVERLAP;
    return launched(launch_fp8_quantize(x, ldx, S, I, dtype, static_cast<uint8_t *>(codes), ldc,
                                        scales, lds, (hipStream_t)stream));
}

size_t qgemv_matmul_workspace(int S, int I, int O, int dtype, int gated)
{
    if (bad_sizes(S, I, O) || S == 0 || bad_dtype(dtype) || (gated && (O & 1))) return 0;
    return matmul_workspace(S, I, O, dtype, gated != 0);
}

int qgemv_fp8b128_matmul(const void *w, const float *scale_inv, const void *x, long long ldx,
                         const float *x_scale, long long lds, void *y, long long ldy, int S, int I,
                         int O, int dtype, const qgemv_epilogue *epilogue, void *workspace,
                         size_t ws_bytes, void *stream)
{
    if (bad_sizes(S, I, O)) return QGEMV_E_DIMS;
    if (S > 0 && (!w || !scale_inv || !x || !x_scale || !y)) return QGEMV_E_NULL;
    MatmulArgs p{};
    p.a.E = 1;
    if (int e = fill(p, w, scale_inv, x, ldx, x_scale, lds, S, y, ldy, S, I, O, dtype, epilogue,
                     true))
        return e;
    if (S == 0) return QGEMV_OK;
    if (too_large(S, O)) return QGEMV_E_DIMS;
    const size_t need = matmul_workspace(S, I, O, dtype, p.a.gated);
    if (need > 0 && (!workspace || misaligned(workspace, 256) || ws_bytes < need))
        return QGEMV_E_WORKSPACE;
    if (overlapping(p, workspace, need)) return QGEMV_E_OVERLAP;
    return launched(launch_matmul(p, workspace, (hipStream_t)stream));
}

size_t qgemv_matmul_grouped_workspace(int R, int E)
{
    if (R < 0 || R > MAX_DIM || E < 1 || E > MAX_EXPERTS) return 0;
    return matmul_grouped_workspace(R, E);
}

int qgemv_fp8b128_matmul_grouped(const void *w, const float *scale_inv, long long w_stride,
                                 long long s_stride, int E, const int32_t *offsets,
                                 const int32_t *rows, const void *x, long long ldx,
                                 const float *x_scale, long long lds, int T, void *y,
                                 long long ldy, int R, int I, int O, int dtype,
                                 const qgemv_epilogue *epilogue, void *workspace, size_t ws_bytes,
                                 void *stream)
{
    if (bad_sizes(R, I, O) || E < 1 || E > MAX_EXPERTS || T < 0 || T > MAX_DIM)
        return QGEMV_E_DIMS;
    if (R > 0 && (rows ? T < 1 : T < R)) return QGEMV_E_DIMS;
    if (R > 0 && (!w || !scale_inv || !offsets || !x || !x_scale || !y)) return QGEMV_E_NULL;
    if (misaligned(offsets, 4) || misaligned(rows, 4)) return QGEMV_E_ALIGN;
    const long long ng = (I + 127) / 128, blocks = (O + 127) / 128;
    if (w_stride < (long long)O * I || s_stride < blocks * ng) return QGEMV_E_IDS;
    MatmulArgs p{};
    p.a.E = E;
    p.a.w_stride = w_stride;
    p.a.s_stride = s_stride;
    p.a.offsets = offsets;
    p.a.rows = rows;
    if (int e = fill(p, w, scale_inv, x, ldx, x_scale, lds, T, y, ldy, R, I, O, dtype, epilogue,
                     false))
        return e;
    if (R == 0) return QGEMV_OK;
    if (too_large(R, O) || !matmul_launchable(p)) return QGEMV_E_DIMS;
    const size_t need = matmul_grouped_workspace(R, E);
    if (!workspace || misaligned(workspace, 256) || ws_bytes < need) return QGEMV_E_WORKSPACE;
    if (overlapping(p, workspace, need)) return QGEMV_E_OVERLAP;
    return launched(launch_matmul(p, workspace, (hipStream_t)stream));
}

int qgemv_moe_dispatch(const void *x, long long ldx, int T, const int32_t *tokens, int R, int I,
                       void *y, long long ldy, int dtype, void *stream)
{
    if (bad_routed(T, 1, R, I)) return QGEMV_E_DIMS;
    if (bad_dtype(dtype)) return QGEMV_E_ARG;
    if (R > 0 && (!tokens || !y || (T > 0 && !x))) return QGEMV_E_NULL;
    if (ldx < I || ldy < I) return QGEMV_E_DIMS;
    const long long el = element(dtype);
    if (misaligned(x, el) || misaligned(y, el) || misaligned(tokens, 4)) return QGEMV_E_ALIGN;
    if (R == 0) return QGEMV_OK;
    const Rows in[] = {rows_of(x, T, I * el, ldx * el), block(tokens, 4LL * R)};
    if (overlaps_any(rows_of(y, R, I * el, ldy * el), in, 2)) return QGEMV_E_OVERLAP;
    return launched(
        launch_moe_dispatch(x, ldx, T, tokens, R, I, y, ldy, dtype, (hipStream_t)stream));
}

int qgemv_moe_dispatch_grad(const void *dy, long long lddy, int R, const int32_t *pos, int T,
                            int K, int I, void *dx, long long lddx, int dtype, void *stream)
{
    if (bad_routed(T, K, R, I)) return QGEMV_E_DIMS;
    if (bad_dtype(dtype)) return QGEMV_E_ARG;
    if (T > 0 && (!pos || !dx || (R > 0 && !dy))) return QGEMV_E_NULL;
    if (lddy < I || lddx < I) return QGEMV_E_DIMS;
    const long long el = element(dtype);
    if (misaligned(dy, el) || misaligned(dx, el) || misaligned(pos, 4)) return QGEMV_E_ALIGN;
    if (T == 0) return QGEMV_OK;
    const Rows in[] = {rows_of(dy, R, I * el, lddy * el), block(pos, 4LL * T * K)};
    if (overlaps_any(rows_of(dx, T, I * el, lddx * el), in, 2)) return QGEMV_E_OVERLAP;
    return launched(
        launch_moe_dispatch_grad(dy, lddy, R, pos, T, K, I, dx, lddx, dtype, (hipStream_t)stream));
}

int qgemv_moe_combine_grad(const void *dy, long long lddy, const void *h, long long ldh, int R,
                           const int32_t *tokens, const int32_t *pos, const float *gates, int T,
                           int K, int O, void *dh, long long lddh, float *dgates, int dtype,
                           void *stream)
{
    if (bad_routed(T, K, R, O)) return QGEMV_E_DIMS;
    if (bad_dtype(dtype)) return QGEMV_E_ARG;
    if (T > 0 && (!dy || !pos || !gates || !dgates || (R > 0 && (!h || !tokens || !dh))))
        return QGEMV_E_NULL;
    if (lddy < O || ldh < O || lddh < O) return QGEMV_E_DIMS;
    const long long el = element(dtype);
    if (misaligned(dy, el) || misaligned(h, el) || misaligned(dh, el) || misaligned(tokens, 4) ||
        misaligned(pos, 4) || misaligned(gates, 4) || misaligned(dgates, 4))
        return QGEMV_E_ALIGN;
    if (T == 0) return QGEMV_OK;
    const long long n = 4LL * T * K;
    const Rows all[] = {rows_of(dy, T, O * el, lddy * el), rows_of(h, R, O * el, ldh * el),
                        block(tokens, 4LL * R), block(pos, n), block(gates, n),
                        rows_of(dh, R, O * el, lddh * el), block(dgates, n)};
    if (overlaps_any(all[5], all, 5) || overlaps_any(all[6], all, 6)) return QGEMV_E_OVERLAP;
    return launched(launch_moe_combine_grad(dy, lddy, h, ldh, R, tokens, pos, gates, T, K, O, dh,
                                            lddh, dgates, dtype, (hipStream_t)stream));
}

}  // extern "C"
