// quantize.hip -- activations to e4m3 with a scale per row and 128 columns.
#include "qg_device.h"
#include "qg_matmul.h"

namespace qg {

namespace {

// Block b of a row: scale = max|x| / 448 (448 is e4m3's largest value), at least
// 2^-126; code = the e4m3 value nearest to x over the exact quotient max|x| / 448
// (over 2^-126 where that is larger), ties to even.  The floor keeps x / scale at 448
// or below where max|x| / 448 would lose bits; values below 2^-117 keep an absolute
// step instead.  A block that holds an infinity or NaN gets the scale NaN and codes
// of NaN: its row of a product is NaN.
//
// x / scale by a reciprocal is within 3 2^-24 of the quotient, so both of its codes a
// 2^-21 below and above are the code, but for the few (about one in 10^5) whose
// quotient lies that near to the middle of two: those compare 448 |x| / max|x| in 64
// bits with the middle.  (448 |x| is exact there and the division's rounding cannot
// reach the middle: a quotient of 24-bit numbers that is not the middle is 2^-32 away
// from it at least.)  An f32 quotient's two roundings would now and then decide
// otherwise.
//
// 16 lanes per block, eight columns each, the block in registers between its
// maximum and its codes: x is read once.  Bound by HBM for many rows (2049 x 11000
// f32: 17.7 us, 6.4 TB/s, as a plain read of as many bytes), by the launch for few.
__device__ __forceinline__ uint32_t exact_code(float v, float amax, uint32_t below, uint32_t above)
{
    // codes of one sign, next to each other
    const float mid = 0.5f * (__builtin_amdgcn_cvt_f32_fp8((int)below, 0) +
                              __builtin_amdgcn_cvt_f32_fp8((int)above, 0));
    const double floor_max = 448.0 * 0x1p-126;
    const double m = (double)amax > floor_max ? (double)amax : floor_max;
    const double q = fabs((double)v) * 448.0 / m, middle = fabs((double)mid);
    return q < middle ? below : q > middle ? above : (below & 1) ? above : below;
}

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
        typedef typename Eight<raw>::type rawx8;
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
    const float r = 1.0f / s;
    u32x2 q, up;                                         // codes a little towards zero, and away
#pragma unroll
    for (int h = 0; h < 2; h++) {
        int w[2];
#pragma unroll
        for (int k = 0; k < 2; k++) {
            const float f = r * (k ? 1.0f + 0x1p-21f : 1.0f - 0x1p-21f);
            w[k] = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * h] * f, v[4 * h + 1] * f, 0, false);
            w[k] = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * h + 2] * f, v[4 * h + 3] * f, w[k], true);
        }
        q[h] = (uint32_t)w[0];
        up[h] = (uint32_t)w[1];
    }
    if (!finite) {
        q = u32x2{0x7F7F7F7Fu, 0x7F7F7F7Fu};
    } else if (q.x != up.x || q.y != up.y) {
        const float amax = __builtin_bit_cast(float, m);
#pragma unroll
        for (int j = 0; j < 8; j++) {
            const int sh = 8 * (j % 4);
            const uint32_t lo = (q[j / 4] >> sh) & 255, hi = (up[j / 4] >> sh) & 255;
            if (lo != hi) q[j / 4] ^= (lo ^ exact_code(v[j], amax, lo, hi)) << sh;
        }
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
