// qg_tile.h -- what the matrix-core tile kernels share: fragment types, fp8
// codes to f16, memory-to-LDS loads, and the order of a tile's rows in LDS.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace qg {

typedef float f32x4v __attribute__((ext_vector_type(4)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

// Eight E4M3 codes (two dwords, byte order = column order) in f16, exactly.
__device__ __forceinline__ f16x8 fp8x8_f16(uint32_t a, uint32_t b)
{
    const f16x2 r0 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)a, 1.0f, false);
    const f16x2 r1 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)a, 1.0f, true);
    const f16x2 r2 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)b, 1.0f, false);
    const f16x2 r3 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)b, 1.0f, true);
    return f16x8{r0.x, r0.y, r1.x, r1.y, r2.x, r2.y, r3.x, r3.y};
}

// Memory to LDS without registers: lane i's 16 (4) bytes from base + off go to
// LDS bytes lds + 16 i (4 i); lds is uniform over the wave.  The compiler does
// not count these loads: the K loop waits for them itself (wait_loads), and
// holds no other vector-memory loads.  m0 is reserved, so that no value of the
// compiler's lives there; that it is named keeps its own uses of it, which set
// it first, on one side of these.  (The warning says that it is reserved.)
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void load_lds16(const void *base, uint32_t off, uint32_t lds)
{
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2"
                 :: "s"(lds), "v"(off), "s"(base) : "memory", "m0");
}
__device__ __forceinline__ void load_lds4(const void *base, uint32_t off, uint32_t lds)
{
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, %2"
                 :: "s"(lds), "v"(off), "s"(base) : "memory", "m0");
}
#pragma clang diagnostic pop

// All but the wave's last n loads have arrived, for every wave of the group.
template <int N>
__device__ __forceinline__ void wait_loads()
{
    asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" :: "i"(N) : "memory");
}

// Where a row's 16-byte chunk c of a K step sits in its 128 bytes: c ^
// swizzle(row).  A 16-byte LDS read of a wave is served in four passes, lanes
// 0-3, 12-15, 20-27, then 4-11, 16-19, 28-31, then the same of the upper half;
// with this key the 16 lanes of each pass touch all 64 banks once, for both
// column orders (counted in the fp8 tile kernel, whose weights are read the same
// way: no conflict; with row % 8 or row / 2 % 8 as key each read took twice as
// long.  int4's weights, read 4 or 8 bytes at a time, spend 15 % of the LDS
// cycles on conflicts).
__device__ __forceinline__ int swizzle(int row)
{
    const int j = row >> 1;
    return (j & 1) | ((j >> 1) & 2) | ((j ^ (j >> 1)) & 2) << 1;
}

}  // namespace qg
