// quantize.hip -- activations to e4m3 with a scale per row and 128 columns.
#include "qg_device.h"
#include "qg_matmul.h"

namespace qg {

namespace {

// Block b of a row: s = max|x| / 448 (448 is e4m3's largest value), at least
// 2^-126; code = e4m3(x / s), quotients and codes rounded to nearest even.  The
// floor keeps x / s at 448 or below where max|x| / 448 would lose bits; values
// below 2^-117 keep an absolute step instead.  A block that holds an infinity
// or NaN gets the scale NaN and codes of NaN: its row of a product is NaN.
//
// 16 lanes per block, eight columns each, the block in registers between its
// maximum and its codes: x is read once.  Bound by HBM for many rows, by the
// launch for few.
template <typename XT, bool VEC>
__global__ __launch_bounds__(256) void quantize(const typename XT::raw *__restrict__ x,
                                                long long ldx, unsigned groups, unsigned ng,
                                                int I, uint8_t *__restrict__ codes,
                                                long long ldc, float *__restrict__ scales,
                                                long long lds)
{
    typedef typename XT::raw raw;
    const unsigned g = blockIdx.x * 16u + threadIdx.x / 16u;
    if (g >= groups) return;                             // uniform over a block's lanes
    const unsigned row = g / ng, b = g - row * ng;
    const int c = (int)b * 128 + (int)(threadIdx.x & 15) * 8;
    const raw *const src = x + (long long)row * ldx + c;
    const bool whole = c + 8 <= I;
    float v[8];
    if (VEC && whole) {
        typedef raw rawx8 __attribute__((ext_vector_type(8)));
        const rawx8 t = *reinterpret_cast<const rawx8 *>(src);
#pragma unroll
        for (int j = 0; j < 8; j++) v[j] = XT::get(t[j]);
    } else {
#pragma unroll
        for (int j = 0; j < 8; j++) v[j] = c + j < I ? XT::get(src[j]) : 0.0f;
    }
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 8; j++)
        m = max(m, __builtin_bit_cast(uint32_t, v[j]) & 0x7FFFFFFFu);
#pragma unroll
    for (int d = 8; d > 0; d /= 2) m = max(m, (uint32_t)__shfl_xor((int)m, d));
    const bool finite = m < 0x7F800000u;
    const float s = finite ? fmaxf(__builtin_bit_cast(float, m) / 448.0f, 0x1p-126f)
                           : __builtin_nanf("");
    if ((threadIdx.x & 15) == 0) scales[(long long)row * lds + b] = s;
    u32x2 q;
#pragma unroll
    for (int h = 0; h < 2; h++) {
        int w = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * h] / s, v[4 * h + 1] / s, 0, false);
        w = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * h + 2] / s, v[4 * h + 3] / s, w, true);
        q[h] = finite ? (uint32_t)w : 0x7F7F7F7Fu;
    }
    uint8_t *const dst = codes + (long long)row * ldc + c;
    if (VEC && whole) {
        *reinterpret_cast<u32x2 *>(dst) = q;
    } else {
#pragma unroll
        for (int j = 0; j < 8; j++)
            if (c + j < I) dst[j] = (uint8_t)(q[j / 4] >> (8 * (j % 4)));
    }
}

template <typename XT>
hipError_t run_quantize(const void *x, long long ldx, int S, int I, uint8_t *codes,
                        long long ldc, float *scales, long long lds, hipStream_t st)
{
    typedef typename XT::raw raw;
    const bool vec = (((uintptr_t)x | (uintptr_t)(ldx * sizeof(raw))) & 15) == 0 &&
                     (((uintptr_t)codes | (uintptr_t)ldc) & 7) == 0;
    const int ng = (I + 127) / 128;
    // as many rows per launch as its work items allow
    const int most = (int)((MAX_ITEMS - 255) / 16 / ng);
    for (int r = 0; r < S; r += most) {
        const int n = S - r < most ? S - r : most;
        const unsigned groups = (unsigned)n * (unsigned)ng;
        const dim3 grid((groups + 15) / 16);
        const raw *const src = static_cast<const raw *>(x) + r * ldx;
        if (vec)
            hipLaunchKernelGGL((quantize<XT, true>), grid, dim3(256), 0, st, src, ldx, groups, ng,
                               I, codes + r * ldc, ldc, scales + r * lds, lds);
        else
            hipLaunchKernelGGL((quantize<XT, false>), grid, dim3(256), 0, st, src, ldx, groups,
                               ng, I, codes + r * ldc, ldc, scales + r * lds, lds);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        if (S - r <= most) break;                        // (r + most could pass an int)
    }
    return hipSuccess;
}

}  // namespace

hipError_t launch_fp8_quantize(const void *x, long long ldx, int S, int I, int dtype,
                               uint8_t *codes, long long ldc, float *scales, long long lds,
                               hipStream_t st)
{
    return dtype == QGEMV_BF16 ? run_quantize<BF16>(x, ldx, S, I, codes, ldc, scales, lds, st)
                               : run_quantize<F32>(x, ldx, S, I, codes, ldc, scales, lds, st);
}

}  // namespace qg
