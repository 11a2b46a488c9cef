// qg_linear.h -- launchers and device helpers of the many-token products with
// an epilogue (dense and grouped by expert) and of the routed slots.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "qgemv.h"

namespace qg {

enum WeightFormat { FMT_I4G = 0, FMT_FP8 = 1 };

// One product Y = epilogue(X . W^T), dense (tiles == nullptr) or grouped.
struct LinearArgs {
    const uint8_t *w;
    const float *scales;
    long long w_stride, s_stride;   // from one expert to the next (bytes, floats)
    const void *x;                  // [T][ldx], type dtype
    void *y;                        // [R][ldy], type dtype
    long long ldx, ldy, ldr;        // row strides in elements
    const void *bias;               // [O] per expert, or nullptr
    const void *residual;           // [R][ldr], or nullptr
    const int32_t *rows;            // grouped: row of x for each row of y, or nullptr
    const int32_t *offsets;         // grouped: [E + 1] device array, else nullptr
    int T, R, E;                    // rows of x, rows of y, experts (dense: T == R, E == 1)
    int I, O, gs, ng;               // ng: scales per row of W (i4g) or of blocks (fp8)
    int dtype, act, gated;
};

// Workspace bytes of a product (an upper bound over its kernels; a function
// of these sizes only).  E = 0: dense.
size_t linear_workspace(int T, int R, int E, int I, int dtype);
// Whether the kernel chosen for a product fits a launch (dense ones always: they
// are cut into slices of rows).
bool linear_launchable(WeightFormat fmt, const LinearArgs &a);
hipError_t launch_linear(WeightFormat fmt, const LinearArgs &a, void *ws, hipStream_t st);

// The f16 tile kernels (linear_tile.hip): shapes they take, workspace, launch
// with row tiles of bm: bf16 64, 96 or 128 (narrow 32 or 64), f32 32 or 64
// (narrow 32); tiles == nullptr: dense.
struct RowTile;
bool tile_fits(WeightFormat fmt, const LinearArgs &a);
size_t tile_workspace(int T, int I, int dtype);
int tile_rows(int I);                    // rows whose packed plane stays below 4 GB
bool planes_fit(int T, int I);           // those of T rows do
long long tile_items(const LinearArgs &a, bool narrow, int bm, int ntm);   // work items
hipError_t launch_tile(WeightFormat fmt, const LinearArgs &a, bool narrow, int bm,
                       const RowTile *tiles, int ntm, void *ws, hipStream_t st);

// The stream kernel (linear_stream.hip): the rows of its tiles for a product, 0
// where others are better or it does not fit.
int stream_rows(WeightFormat fmt, const LinearArgs &a);
long long stream_items(WeightFormat fmt, const LinearArgs &a, int rows, int ntm);
hipError_t launch_stream(WeightFormat fmt, const LinearArgs &a, int rows, const RowTile *tiles,
                         int ntm, hipStream_t st);

// A dimension of a launch holds fewer than 2^32 work items.
constexpr long long MAX_ITEMS = 0xFFFFFFFFLL;

inline size_t align256(size_t n) { return (n + 255) & ~(size_t)255; }

// routed slots: sort by expert, and the gate-weighted return
size_t moe_group_workspace(int T, int K, int E);
hipError_t launch_moe_group(const int32_t *ids, int T, int K, int E, int32_t *offsets,
                            int32_t *tokens, int32_t *pos, void *ws, hipStream_t st);
hipError_t launch_moe_combine(const void *h, long long ldh, int R, const int32_t *pos,
                              const float *gates, int T, int K, int O, const void *residual,
                              long long ldr, void *y, long long ldy, int dtype, hipStream_t st);

}  // namespace qg

namespace qg {

// -- element types -----------------------------------------------------------
struct F32 {
    typedef float raw;
    static __device__ __forceinline__ float get(raw v) { return v; }
    static __device__ __forceinline__ raw put(float v) { return v; }
};
struct BF16 {
    typedef uint16_t raw;
    static __device__ __forceinline__ float get(raw v)
    {
        return __builtin_bit_cast(float, (uint32_t)v << 16);
    }
    // round to nearest even (the type's one rounding of a result)
    static __device__ __forceinline__ raw put(float v)
    {
        return __builtin_bit_cast(uint16_t, (__bf16)v);
    }
};

// (w & mask) | bits in one instruction: it takes one scalar operand and no
// literal here, so the constants are shown to the compiler as values in a
// scalar and a vector register.  (The instruction itself stays the compiler's,
// which keeps its distance to a matrix instruction that reads the result.)
__device__ __forceinline__ uint32_t and_or(uint32_t w, uint32_t mask, uint32_t bits)
{
    asm("" : "+s"(mask));
    asm("" : "+v"(bits));
    return (w & mask) | bits;
}

// -- epilogue ----------------------------------------------------------------
// act(a) in f32.  silu a / (1 + e^-a); gelu a/2 (1 + erf(a / sqrt 2)), written
// with erfc for negative a, where 1 + erf cancels; gelu_tanh the tanh form,
// a * sigmoid(2u).  The quotient by a reciprocal is within two roundings.
template <int ACT>
__device__ __forceinline__ float activate(float a)
{
    if (ACT == QGEMV_ACT_RELU) return a < 0.0f ? 0.0f : a;       // NaN stays NaN
    if (ACT == QGEMV_ACT_SILU) return a * __builtin_amdgcn_rcpf(1.0f + expf(-a));
    if (ACT == QGEMV_ACT_GELU) {
        const float z = a * 0.70710678118654752f;
        return a * (z < 0.0f ? 0.5f * erfcf(-z) : 0.5f + 0.5f * erff(z));
    }
    if (ACT == QGEMV_ACT_GELU_TANH) {
        const float u = 0.79788456080286536f * (a + 0.044715f * a * a * a);
        return a * __builtin_amdgcn_rcpf(1.0f + expf(-2.0f * u));
    }
    return a;
}

// The ends of a workgroup's outputs: bias and activation (and gate), residual,
// store.  A thread takes the outputs first, first + stride, ... below count;
// get(i, row, col, v, up) gives output i's row and column of y (col >= the
// columns of y: none) and its sums.  The loads of U outputs are in flight
// together.
template <typename XT, int ACT, int U, typename Get>
__device__ __forceinline__ void finish_act(const LinearArgs &a, int expert, int first, int stride,
                                           int count, Get get)
{
    typedef typename XT::raw raw;
    const int oc = a.gated ? a.O / 2 : a.O;
    const raw *const bias =
        a.bias ? static_cast<const raw *>(a.bias) + (size_t)expert * a.O : nullptr;
#pragma unroll 1
    for (int i0 = first; i0 < count; i0 += U * stride) {
        float v[U], up[U], rs[U];
        int row[U], col[U];
#pragma unroll
        for (int u = 0; u < U; u++) {
            const int i = i0 + u * stride;
            get(i < count ? i : i0, row[u], col[u], v[u], up[u]);
            if (i >= count) col[u] = oc;
            rs[u] = 0.0f;
            if (col[u] >= oc) continue;
            if (a.residual)
                rs[u] = XT::get(
                    static_cast<const raw *>(a.residual)[(size_t)row[u] * a.ldr + col[u]]);
            if (bias) {
                v[u] += XT::get(bias[col[u]]);
                if (a.gated) up[u] += XT::get(bias[oc + col[u]]);
            }
        }
#pragma unroll
        for (int u = 0; u < U; u++) {
            float r = activate<ACT>(v[u]);
            if (a.gated) r *= up[u];
            if (col[u] < oc)
                static_cast<raw *>(a.y)[(size_t)row[u] * a.ldy + col[u]] = XT::put(r + rs[u]);
        }
    }
}

template <typename XT, int U, typename Get>
__device__ __forceinline__ void finish(const LinearArgs &a, int expert, int first, int stride,
                                       int count, Get get)
{
    switch (a.act) {
    case QGEMV_ACT_RELU:
        return finish_act<XT, QGEMV_ACT_RELU, U>(a, expert, first, stride, count, get);
    case QGEMV_ACT_SILU:
        return finish_act<XT, QGEMV_ACT_SILU, U>(a, expert, first, stride, count, get);
    case QGEMV_ACT_GELU:
        return finish_act<XT, QGEMV_ACT_GELU, U>(a, expert, first, stride, count, get);
    case QGEMV_ACT_GELU_TANH:
        return finish_act<XT, QGEMV_ACT_GELU_TANH, U>(a, expert, first, stride, count, get);
    default:
        return finish_act<XT, QGEMV_ACT_NONE, U>(a, expert, first, stride, count, get);
    }
}

// One tile of rows: rows [row0, row0 + n) of y, all of one expert.
struct RowTile {
    int expert, row0, n, pad;
};

}  // namespace qg
