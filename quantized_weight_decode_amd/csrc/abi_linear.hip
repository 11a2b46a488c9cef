// abi_linear.hip -- the extern "C" entry points of the products with an
// epilogue and of the routed slots: argument validation, then launch.
//
// As in abi.hip, validation looks at pointer values, dimensions and sizes
// only, so a refused call is safe with any pointers.
#include "qg_check.h"

namespace {

using namespace qg;

int dense(qg::WeightFormat fmt, const void *w, const float *scales, const void *x, long long ldx,
          void *y, long long ldy, int S, int I, int O, int gs, int dtype,
          const qgemv_epilogue *epilogue, void *workspace, size_t ws_bytes, void *stream)
{
    if (bad_sizes(S, I, O)) return QGEMV_E_DIMS;
    if (gs < 2 || (gs & 1) || gs > MAX_DIM) return QGEMV_E_GS;
    if (S > 0 && (!w || !scales || !x || !y)) return QGEMV_E_NULL;
    qg::LinearArgs a{};
    a.w = static_cast<const uint8_t *>(w);
    a.scales = scales;
    a.x = x;
    a.y = y;
    a.ldx = ldx;
    a.ldy = ldy;
    a.T = a.R = S;
    a.E = 1;
    a.I = I;
    a.O = O;
    a.gs = gs;
    a.ng = (I + gs - 1) / gs;
    a.dtype = dtype;
    if (int e = take(a, element(dtype), epilogue, true)) return e;
    if (S == 0) return QGEMV_OK;
    if (too_large(S, O)) return QGEMV_E_DIMS;
    const size_t need = qg::linear_workspace(S, S, 0, I, dtype);
    if (need > 0 && (!workspace || misaligned(workspace, 256) || ws_bytes < need))
        return QGEMV_E_WORKSPACE;
    const bool i4 = fmt == qg::FMT_I4G;
    if (overlapping(a, element(dtype), (long long)O * (i4 ? (I + 1) / 2 : I),
                    4LL * a.ng * (i4 ? O : (O + 127) / 128), workspace, need))
        return QGEMV_E_OVERLAP;
    return launched(qg::launch_linear(fmt, a, workspace, (hipStream_t)stream));
}

}  // namespace

extern "C" {

size_t qgemv_linear_workspace(int S, int I, int O, int dtype)
{
    if (bad_sizes(S, I, O) || bad_dtype(dtype)) return 0;
    return qg::linear_workspace(S, S, 0, I, dtype);
}

int qgemv_i4g_linear(const void *w, const float *scales, const void *x, long long ldx, void *y,
                     long long ldy, int S, int I, int O, int gs, int dtype,
                     const qgemv_epilogue *epilogue, void *workspace, size_t ws_bytes,
                     void *stream)
{
    return dense(qg::FMT_I4G, w, scales, x, ldx, y, ldy, S, I, O, gs, dtype, epilogue, workspace,
                 ws_bytes, stream);
}

int qgemv_fp8b128_linear(const void *w, const float *scale_inv, const void *x, long long ldx,
                         void *y, long long ldy, int S, int I, int O, int dtype,
                         const qgemv_epilogue *epilogue, void *workspace, size_t ws_bytes,
                         void *stream)
{
    return dense(qg::FMT_FP8, w, scale_inv, x, ldx, y, ldy, S, I, O, 128, dtype, epilogue,
                 workspace, ws_bytes, stream);
}

size_t qgemv_grouped_workspace(int T, int R, int E, int I, int O, int dtype)
{
    if (bad_sizes(R, I, O) || T < 0 || T > MAX_DIM || E < 1 || E > MAX_EXPERTS ||
        bad_dtype(dtype))
        return 0;
    return qg::linear_workspace(T, R, E, I, dtype);
}

int qgemv_i4g_grouped(const void *w, const float *scales, long long w_stride, long long s_stride,
                      int E, const int32_t *offsets, const int32_t *rows, const void *x,
                      long long ldx, int T, void *y, long long ldy, int R, int I, int O, int gs,
                      int dtype, const qgemv_epilogue *epilogue, void *workspace,
                      size_t ws_bytes, void *stream)
{
    if (bad_sizes(R, I, O) || E < 1 || E > MAX_EXPERTS || T < 0 || T > MAX_DIM)
        return QGEMV_E_DIMS;
    if (R > 0 && (rows ? T < 1 : T < R)) return QGEMV_E_DIMS;
    if (gs < 2 || (gs & 1) || gs > MAX_DIM) return QGEMV_E_GS;
    if (R > 0 && (!w || !scales || !offsets || !x || !y)) return QGEMV_E_NULL;
    if (misaligned(offsets, 4) || misaligned(rows, 4)) return QGEMV_E_ALIGN;
    const long long rb = ((long long)I + 1) / 2, ng = ((long long)I + gs - 1) / gs;
    if (w_stride < (long long)O * rb || s_stride < (long long)O * ng) return QGEMV_E_IDS;
    qg::LinearArgs a{};
    a.w = static_cast<const uint8_t *>(w);
    a.scales = scales;
    a.w_stride = w_stride;
    a.s_stride = s_stride;
    a.x = x;
    a.y = y;
    a.ldx = ldx;
    a.ldy = ldy;
    a.rows = rows;
    a.offsets = offsets;
    a.T = T;
    a.R = R;
    a.E = E;
    a.I = I;
    a.O = O;
    a.gs = gs;
    a.ng = (int)ng;
    a.dtype = dtype;
    if (int e = take(a, element(dtype), epilogue, false)) return e;
    if (R == 0) return QGEMV_OK;
    if (too_large(R, O) || !qg::linear_launchable(qg::FMT_I4G, a)) return QGEMV_E_DIMS;
    const size_t need = qg::linear_workspace(T, R, E, I, dtype);
    if (!workspace || misaligned(workspace, 256) || ws_bytes < need) return QGEMV_E_WORKSPACE;
    if (overlapping(a, element(dtype), O * rb, 4 * O * ng, workspace, need)) return QGEMV_E_OVERLAP;
    return launched(qg::launch_linear(qg::FMT_I4G, a, workspace, (hipStream_t)stream));
}

size_t qgemv_moe_group_workspace(int T, int K, int E)
{
    if (T < 0 || K < 1 || E < 1 || E > MAX_EXPERTS || (long long)T * K > MAX_DIM) return 0;
    return qg::moe_group_workspace(T, K, E);
}

int qgemv_moe_group(const int32_t *ids, int T, int K, int E, int32_t *offsets, int32_t *tokens,
                    int32_t *pos, void *workspace, size_t ws_bytes, void *stream)
{
    if (T < 0 || K < 1 || E < 1 || E > MAX_EXPERTS || (long long)T * K > MAX_DIM)
        return QGEMV_E_DIMS;
    if (!offsets || (T > 0 && (!ids || !tokens || !pos))) return QGEMV_E_NULL;
    if (misaligned(ids, 4) || misaligned(offsets, 4) || misaligned(tokens, 4) ||
        misaligned(pos, 4))
        return QGEMV_E_ALIGN;
    const size_t need = qg::moe_group_workspace(T, K, E);
    if (need > 0 && (!workspace || misaligned(workspace, 4) || ws_bytes < need))
        return QGEMV_E_WORKSPACE;
    const long long n = 4LL * T * K;
    const Rows all[] = {block(ids, n), block(offsets, 4LL * (E + 1)), block(tokens, n),
                        block(pos, n), block(workspace, (long long)need)};
    for (int i = 1; i < 5; i++)
        if (overlaps_any(all[i], all, i)) return QGEMV_E_OVERLAP;
    return launched(qg::launch_moe_group(ids, T, K, E, offsets, tokens, pos, workspace,
                                         (hipStream_t)stream));
}

int qgemv_moe_combine(const void *h, long long ldh, int R, const int32_t *pos,
                      const float *gates, int T, int K, int O, const void *residual,
                      long long ldr, void *y, long long ldy, int dtype, void *stream)
{
    if (T < 0 || T > MAX_DIM || R < 0 || R > MAX_DIM || K < 1 || K > 64 || O < 1 || O > MAX_DIM)
        return QGEMV_E_DIMS;
    if (bad_dtype(dtype)) return QGEMV_E_ARG;
    if (T > 0 && (!pos || !gates || !y || (R > 0 && !h))) return QGEMV_E_NULL;
    if (ldh < O || ldy < O || (residual && ldr < O)) return QGEMV_E_DIMS;
    const uintptr_t el = element(dtype);
    if (misaligned(h, el) || misaligned(y, el) || misaligned(residual, el) ||
        misaligned(pos, 4) || misaligned(gates, 4))
        return QGEMV_E_ALIGN;
    if (T == 0) return QGEMV_OK;
    const long long n = 4LL * T * K;
    const Rows yr = rows_of(y, T, O * (long long)el, ldy * (long long)el);
    const Rows in[] = {rows_of(h, R, O * (long long)el, ldh * (long long)el), block(pos, n),
                       block(gates, n)};
    const bool in_place = residual == y && (T == 1 || ldr == ldy);
    if (overlaps_any(yr, in, 3) ||
        (!in_place && overlap(yr, rows_of(residual, T, O * (long long)el, ldr * (long long)el))))
        return QGEMV_E_OVERLAP;
    return launched(qg::launch_moe_combine(h, ldh, R, pos, gates, T, K, O, residual, ldr, y, ldy,
                                           dtype, (hipStream_t)stream));
}

}  // extern "C"
