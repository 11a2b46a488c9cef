// qg_check.h -- argument checks that the entry points of the many-token products
// and the routed slots share (host only).
#pragma once

#include "qg_linear.h"
#include "qg_rows.h"

namespace qg {

constexpr int MAX_DIM = 1 << 24;
constexpr int MAX_EXPERTS = 1024;

inline bool misaligned(const void *p, uintptr_t n) { return ((uintptr_t)p & (n - 1)) != 0; }

inline int launched(hipError_t e) { return e == hipSuccess ? QGEMV_OK : QGEMV_E_HIP; }

inline bool bad_dtype(int dtype) { return dtype != QGEMV_F32 && dtype != QGEMV_BF16; }

inline int element(int dtype) { return dtype == QGEMV_BF16 ? 2 : 4; }

inline bool bad_sizes(int rows, int I, int O)
{
    return rows < 0 || rows > MAX_DIM || I < 1 || O < 1 || I > MAX_DIM || O > MAX_DIM;
}

// y against what a product reads (the residual may be y itself), and the
// scratch against both.  x_el: bytes of an element of x.
inline bool overlapping(const LinearArgs &a, long long x_el, long long w_bytes, long long s_bytes,
                        const void *workspace, size_t ws_bytes, Rows more = {})
{
    const long long el = a.dtype == QGEMV_BF16 ? 2 : 4, oc = a.gated ? a.O / 2 : a.O;
    const Rows y = rows_of(a.y, a.R, oc * el, a.ldy * el);
    const Rows res = rows_of(a.residual, a.R, oc * el, a.ldr * el);
    const Rows in[] = {rows_of(a.x, a.T, a.I * x_el, a.ldx * x_el),
                       rows_of(a.w, a.E, w_bytes, a.offsets ? a.w_stride : w_bytes),
                       rows_of(a.scales, a.E, s_bytes, a.offsets ? a.s_stride * 4 : s_bytes),
                       block(a.bias, (long long)a.E * a.O * el),
                       block(a.rows, (long long)a.R * 4),
                       block(a.offsets, (long long)(a.E + 1) * 4), more};
    constexpr int N = sizeof(in) / sizeof(in[0]);
    const Rows ws = block(workspace, (long long)ws_bytes);
    const bool in_place = a.residual == a.y && (a.R == 1 || a.ldr == a.ldy);
    return overlaps_any(y, in, N) || (!in_place && overlap(y, res)) || overlap(y, ws) ||
           overlap(res, ws) || overlaps_any(ws, in, N);
}

// more products than any memory holds outputs for
inline bool too_large(long long rows, int O) { return rows * O > 1LL << 39; }

// Fills a's epilogue from the arguments and checks it with a's type and strides.
inline int take(LinearArgs &a, uintptr_t x_el, const qgemv_epilogue *e, bool with_residual)
{
    if (bad_dtype(a.dtype)) return QGEMV_E_ARG;
    a.act = e ? e->act : QGEMV_ACT_NONE;
    a.gated = e ? e->gated : 0;
    a.bias = e ? e->bias : nullptr;
    a.residual = e ? e->residual : nullptr;
    a.ldr = a.residual ? e->ld_residual : 0;
    if (a.act < QGEMV_ACT_NONE || a.act > QGEMV_ACT_GELU_TANH || (a.gated != 0 && a.gated != 1))
        return QGEMV_E_ARG;
    if (a.residual && !with_residual) return QGEMV_E_ARG;
    if (a.gated && (a.O & 1)) return QGEMV_E_DIMS;
    const int oc = a.gated ? a.O / 2 : a.O;
    if (a.ldx < a.I || a.ldy < oc || (a.residual && a.ldr < oc)) return QGEMV_E_DIMS;
    const uintptr_t el = element(a.dtype);
    if (misaligned(a.scales, 4) || misaligned(a.x, x_el) || misaligned(a.y, el) ||
        misaligned(a.bias, el) || misaligned(a.residual, el))
        return QGEMV_E_ALIGN;
    return QGEMV_OK;
}

}  // namespace qg
