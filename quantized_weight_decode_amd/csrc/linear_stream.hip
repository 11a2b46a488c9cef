// linear_stream.hip -- up to 16 rows of x times packed weights, bound by the
// weights' bytes, dense or grouped by expert, with the epilogue.
#include "qg_device.h"
#include "qg_launch.h"
#include "qg_linear.h"

namespace qg {

namespace {

typedef float f32x4v __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int SW = 8;           // waves of a workgroup
constexpr int SC = 128;         // columns of a chunk

// Dwords of a lane group's 32 columns to dwords of eight columns of each 32:
// in, lane group g holds dwords 0..3 of columns 32 g ..; out, dword t holds
// columns 32 t + 8 g .. (a 4 x 4 transpose over lane groups and dwords).
__device__ __forceinline__ void swap32(uint32_t &a, uint32_t &b)
{
    const auto r = __builtin_amdgcn_permlane32_swap(a, b, false, false);
    a = r[0];
    b = r[1];
}
__device__ __forceinline__ void swap16(uint32_t &a, uint32_t &b)
{
    const auto r = __builtin_amdgcn_permlane16_swap(a, b, false, false);
    a = r[0];
    b = r[1];
}
__device__ __forceinline__ void transpose4(uint32_t d[4])
{
    swap32(d[0], d[2]);
    swap32(d[1], d[3]);
    swap16(d[0], d[1]);
    swap16(d[2], d[3]);
}

__device__ __forceinline__ bf16x8 join(bf16x2 a, bf16x2 b, bf16x2 c, bf16x2 d)
{
    return bf16x8{a.x, a.y, b.x, b.y, c.x, c.y, d.x, d.y};
}

// Four E4M3 codes times 2^e in bf16, exactly.
template <int E>
__device__ __forceinline__ bf16x2 cvt_lo(uint32_t w)
{
    return __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)w, (float)(1 << E), false);
}
template <int E>
__device__ __forceinline__ bf16x2 cvt_hi(uint32_t w)
{
    return __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)w, (float)(1 << E), true);
}

// Eight nibbles in the column order 0 2 4 6 1 3 5 7, in bf16.  Read as E4M3
// codes, 0..15 are n 2^-9, so bytes of one nibble each convert two at a time.
// Plain: the nibbles q.
__device__ __forceinline__ bf16x8 nib8_bf16(uint32_t w)
{
    const uint32_t lo = w & 0x0F0F0F0Fu, hi = (w >> 4) & 0x0F0F0F0Fu;
    return join(cvt_lo<9>(lo), cvt_hi<9>(lo), cvt_lo<9>(hi), cvt_hi<9>(hi));
}
// Signed: q - 8.  t = the two's complement nibble; its code is t for t < 8,
// else 0x90 - t (sign bit and 16 - t) = (t ^ 0x8F) + 1.
__device__ __forceinline__ uint32_t signed_codes(uint32_t t)
{
    const uint32_t m = t & 0x08080808u, u = m >> 3;
    const uint32_t f = (m << 4) + ((m << 1) - u);        // 0x8F in negative bytes
    return (t ^ f) + u;
}
__device__ __forceinline__ bf16x8 nib8_bf16_signed(uint32_t w)
{
    const uint32_t x = w ^ 0x88888888u;
    const uint32_t lo = signed_codes(x & 0x0F0F0F0Fu);
    const uint32_t hi = signed_codes((x >> 4) & 0x0F0F0F0Fu);
    return join(cvt_lo<9>(lo), cvt_hi<9>(lo), cvt_lo<9>(hi), cvt_hi<9>(hi));
}

__device__ __forceinline__ uint32_t low_halves(uint32_t a, uint32_t b)
{
    return __builtin_amdgcn_perm(b, a, 0x05040100u);
}
__device__ __forceinline__ uint32_t high_halves(uint32_t a, uint32_t b)
{
    return __builtin_amdgcn_perm(b, a, 0x07060302u);
}

// Eight activations of a lane as bf16 parts, in the weights' column order.
template <typename XT, int FMT>
struct XFrag;
template <int FMT>
struct XFrag<BF16, FMT> {
    static constexpr int NP = 1;
    u32x4 v;
    __device__ __forceinline__ void load(const uint16_t *p, bool ok)
    {
        v = u32x4{0, 0, 0, 0};
        if (ok) v = *reinterpret_cast<const u32x4 *>(p);
    }
    __device__ __forceinline__ void parts(bf16x8 out[1]) const
    {
        u32x4 o = v;
        if (FMT == FMT_I4G) {
            o.x = low_halves(v.x, v.y);
            o.y = low_halves(v.z, v.w);
            o.z = high_halves(v.x, v.y);
            o.w = high_halves(v.z, v.w);
        }
        out[0] = __builtin_bit_cast(bf16x8, o);
    }
};
// f32 = three bf16 parts of eight bits each, exactly: each part is the high
// half of what is left.
template <int FMT>
struct XFrag<F32, FMT> {
    static constexpr int NP = 3;
    f32x4 a, b;
    __device__ __forceinline__ void load(const float *p, bool ok)
    {
        a = b = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        if (ok) {
            a = *reinterpret_cast<const f32x4 *>(p);
            b = *reinterpret_cast<const f32x4 *>(p + 4);
        }
    }
    __device__ __forceinline__ void parts(bf16x8 out[3]) const
    {
        uint32_t h[3][8];
#pragma unroll
        for (int j = 0; j < 8; j++) {
            float v = j < 4 ? a[j & 3] : b[j & 3];
#pragma unroll
            for (int q = 0; q < 3; q++) {
                h[q][j] = __builtin_bit_cast(uint32_t, v);
                v -= __builtin_bit_cast(float, h[q][j] & 0xFFFF0000u);
            }
        }
#pragma unroll
        for (int q = 0; q < 3; q++) {
            u32x4 o;
            if (FMT == FMT_I4G) {
                o.x = high_halves(h[q][0], h[q][2]);
                o.y = high_halves(h[q][4], h[q][6]);
                o.z = high_halves(h[q][1], h[q][3]);
                o.w = high_halves(h[q][5], h[q][7]);
            } else {
                o.x = high_halves(h[q][0], h[q][1]);
                o.y = high_halves(h[q][2], h[q][3]);
                o.z = high_halves(h[q][4], h[q][5]);
                o.w = high_halves(h[q][6], h[q][7]);
            }
            out[q] = __builtin_bit_cast(bf16x8, o);
        }
    }
};

struct StreamArgs {
    LinearArgs a;
    const RowTile *tiles;
    int ntn;
};

// Stream kernel.  A workgroup of 8 waves makes up to 16 rows of y x 16 NB
// rows of W; the waves take the chunks of 128 columns in turn, so that
// together they read 512 bytes of a row at a time, and their sums are joined
// through LDS in a fixed order.  v_mfma_f32_16x16x32_bf16, lane l: A row of x
// l % 16, B row of W l % 16, eight columns from the lane group l / 16.
// Weights and activations of D chunks are in flight per wave.
//
// bf16 activations multiply the nibbles q themselves, and the group's sum
// starts from -8 sum(x), one more matrix instruction per group: |error| <=
// 2^-24 (sum q|x| + 8 sum |x|) per rounding, far inside bf16's own.  f32
// activations multiply q - 8, whose unpacking costs 2.5 instead of 0.9
// instructions per weight: an outlier of x at a zero weight must not cost the
// small elements their bits.
template <int FMT, typename XT, int NB, bool GATED, int FG, int D>
__global__ __launch_bounds__(512, 2) void linear_stream(StreamArgs p)
{
    typedef typename XT::raw raw;
    typedef XFrag<XT, FMT> Frag;
    constexpr int NP = Frag::NP;
    constexpr bool OFFSET = FMT == FMT_I4G && NP == 1;
    constexpr int NG = SC / FG;                          // scale groups of a chunk
    constexpr int TPG = 4 / NG;                          // 32-column steps of a group
    constexpr int WL = FMT == FMT_FP8 ? 2 : 1;           // 16-byte loads per row and chunk
    constexpr int YC = GATED ? NB * 8 : NB * 16;         // columns of y
    constexpr int LDR = NB * 16 + 4;
    __shared__ float red[SW][16][LDR];
    const LinearArgs &a = p.a;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int li = lane & 15, lg = lane >> 4;
    const int oc = GATED ? a.O / 2 : a.O;
    const int nt = (int)(blockIdx.x % p.ntn), mt = (int)(blockIdx.x / p.ntn);
    RowTile t;
    if (p.tiles) t = p.tiles[mt];
    else t = RowTile{0, mt * 16, min(16, a.R - mt * 16), 0};
    if (t.n <= 0) return;                                // uniform over the workgroup

    const bool xok = li < t.n;
    int xrow = t.row0 + (xok ? li : 0);
    if (a.rows) {
        xrow = a.rows[xrow];
        if (xrow < 0 || xrow >= a.T) xrow = 0;           // marked in the epilogue
    }
    const raw *xp = static_cast<const raw *>(a.x) + (size_t)xrow * a.ldx;

    const size_t rb = FMT == FMT_I4G ? (size_t)a.I / 2 : (size_t)a.I;
    const uint8_t *wbase = a.w + (size_t)t.expert * a.w_stride;
    const float *sbase = a.scales + (size_t)t.expert * a.s_stride;
    uint32_t woff[NB], soff[NB];
#pragma unroll
    for (int n = 0; n < NB; n++) {
        const int half = GATED ? n / (NB / 2) : 0;
        const int c = nt * YC + (GATED ? n % (NB / 2) : n) * 16 + li;
        const int row = (c < oc ? c : oc - 1) + half * oc;
        woff[n] = (uint32_t)(row * rb);
        soff[n] = (uint32_t)(FMT == FMT_I4G ? row : row >> 7) * (uint32_t)a.ng;
    }

    u32x4 wr[D][NB][WL];
    float sr[D][NB][NG];
    Frag xr[D][4];
    const int chunks = (a.I + SC - 1) / SC;
    const int gs = FMT == FMT_FP8 ? 128 : a.gs;
    auto load = [&](int d, int c) {
        const int k0 = (c < chunks ? c : chunks - 1) * SC;
#pragma unroll
        for (int u = 0; u < WL; u++) {
            const uint32_t kb = min((uint32_t)(FMT == FMT_I4G ? k0 / 2 + 16 * lg
                                                              : k0 + 64 * u + 16 * lg),
                                    (uint32_t)rb - 16);
#pragma unroll
            for (int n = 0; n < NB; n++)
                wr[d][n][u] = ld_stream(reinterpret_cast<const u32x4 *>(wbase + woff[n] + kb));
        }
#pragma unroll
        for (int g = 0; g < NG; g++) {
            const int k = min(k0 + g * FG, a.I - 1);
            const uint32_t gi = (uint32_t)(k / gs);
#pragma unroll
            for (int n = 0; n < NB; n++) sr[d][n][g] = sbase[soff[n] + gi];
        }
#pragma unroll
        for (int s = 0; s < 4; s++) {
            const int k = FMT == FMT_I4G ? k0 + 32 * s + 8 * lg
                                         : k0 + 64 * (s >> 1) + 16 * lg + 8 * (s & 1);
            xr[d][s].load(xp + k, xok && k < a.I && c < chunks);
        }
    };

    f32x4v acc[NB];
#pragma unroll
    for (int n = 0; n < NB; n++) acc[n] = f32x4v{0.0f, 0.0f, 0.0f, 0.0f};

    auto multiply = [&](int d) {
        uint32_t wd[NB][4 * WL];
#pragma unroll
        for (int n = 0; n < NB; n++) {
#pragma unroll
            for (int u = 0; u < WL; u++)
#pragma unroll
                for (int j = 0; j < 4; j++) wd[n][4 * u + j] = wr[d][n][u][j];
            if (FMT == FMT_I4G) transpose4(wd[n]);
        }
#pragma unroll
        for (int g = 0; g < NG; g++) {
            bf16x8 xv[TPG][NP];
#pragma unroll
            for (int s = 0; s < TPG; s++) xr[d][g * TPG + s].parts(xv[s]);
            f32x4v z = {0.0f, 0.0f, 0.0f, 0.0f};
            if (OFFSET) {
                const u32x4 m8 = {0xC100C100u, 0xC100C100u, 0xC100C100u, 0xC100C100u};
#pragma unroll
                for (int s = 0; s < TPG; s++)
                    z = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                        xv[s][0], __builtin_bit_cast(bf16x8, m8), z, 0, 0, 0);
            }
#pragma unroll
            for (int n = 0; n < NB; n++) {
                f32x4v sum = z;
#pragma unroll
                for (int s = 0; s < TPG; s++) {
                    const int st = g * TPG + s;
                    bf16x8 wv;
                    if (FMT == FMT_I4G) {
                        wv = OFFSET ? nib8_bf16(wd[n][st]) : nib8_bf16_signed(wd[n][st]);
                    } else {
                        const uint32_t p0 = wd[n][(2 * st) % (4 * WL)];
                        const uint32_t p1 = wd[n][(2 * st + 1) % (4 * WL)];
                        wv = join(cvt_lo<0>(p0), cvt_hi<0>(p0), cvt_lo<0>(p1), cvt_hi<0>(p1));
                    }
#pragma unroll
                    for (int q = NP - 1; q >= 0; q--)    // small parts first
                        sum = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xv[s][q], wv, sum, 0, 0, 0);
                }
#pragma unroll
                for (int r = 0; r < 4; r++) acc[n][r] = fmaf(sr[d][n][g], sum[r], acc[n][r]);
            }
        }
    };

#pragma unroll
    for (int d = 0; d < D; d++) load(d, wave + d * SW);
    for (int c = wave; c < chunks; c += D * SW) {
#pragma unroll
        for (int d = 0; d < D; d++) {                    // slots past the end hold zeros of x
            multiply(d);
            __builtin_amdgcn_sched_barrier(0);
            load(d, c + (d + D) * SW);
            __builtin_amdgcn_sched_barrier(0);
        }
    }

#pragma unroll
    for (int n = 0; n < NB; n++)
#pragma unroll
        for (int r = 0; r < 4; r++) red[wave][4 * lg + r][n * 16 + li] = acc[n][r];
    __syncthreads();
#pragma unroll 1
    for (int i = tid; i < t.n * YC; i += SW * 64) {
        const int r = i / YC, c = i % YC;
        const int col = nt * YC + c;
        if (col >= oc) continue;
        float v = 0.0f, up = 0.0f;
#pragma unroll
        for (int w = 0; w < SW; w++) {
            v += red[w][r][c];
            if (GATED) up += red[w][r][c + YC];
        }
        if (a.rows) {
            const int xi = a.rows[t.row0 + r];
            if (xi < 0 || xi >= a.T) v = up = __builtin_nanf("");
        }
        finish<XT>(a, t.expert, t.row0 + r, col, v, up);
    }
}

template <int FMT, typename XT, int NB, bool GATED>
void run_nb(const StreamArgs &p, unsigned grid, hipStream_t st)
{
    constexpr int D = 2;
#define QG_RUN(FG)                                                                          \
    hipLaunchKernelGGL((linear_stream<FMT, XT, NB, GATED, FG, D>), dim3(grid), dim3(SW * 64), 0, \
                       st, p)
    if constexpr (FMT == FMT_FP8) {
        QG_RUN(128);
    } else {
        if (p.a.gs % 128 == 0) QG_RUN(128);
        else if (p.a.gs % 64 == 0) QG_RUN(64);
        else QG_RUN(32);
    }
#undef QG_RUN
}

template <int FMT, typename XT>
void run_stream(const StreamArgs &p, int nb, unsigned grid, hipStream_t st)
{
    if (p.a.gated) {
        if (nb == 4) run_nb<FMT, XT, 4, true>(p, grid, st);
        else run_nb<FMT, XT, 2, true>(p, grid, st);
    } else if (nb == 4) {
        run_nb<FMT, XT, 4, false>(p, grid, st);
    } else if (nb == 3) {
        run_nb<FMT, XT, 3, false>(p, grid, st);
    } else if (nb == 2) {
        run_nb<FMT, XT, 2, false>(p, grid, st);
    } else {
        run_nb<FMT, XT, 1, false>(p, grid, st);
    }
}

}  // namespace

bool stream_fits(WeightFormat fmt, const LinearArgs &a)
{
    const int el = a.dtype == QGEMV_BF16 ? 2 : 4;
    return tile_fits(fmt, a) && (((uintptr_t)a.x | (uintptr_t)(a.ldx * el)) & 15) == 0;
}

hipError_t launch_stream(WeightFormat fmt, const LinearArgs &a, const RowTile *tiles, int ntm,
                         hipStream_t st)
{
    // Row blocks per workgroup: the count that leaves the busiest CU the
    // fewest row blocks; among equals the largest, which shares each x
    // fragment among the most rows.
    const int oc = a.gated ? a.O / 2 : a.O;
    const long long ncu = cu_count();
    int best = 0, ntn = 0;
    long long cost = 0;
    for (int nb = 4; nb >= 1; nb--) {
        if (a.gated && (nb & 1)) continue;
        const int yc = a.gated ? nb * 8 : nb * 16;
        const int n = (oc + yc - 1) / yc;
        const long long c = (((long long)n * ntm + ncu - 1) / ncu) * nb;
        if (!best || c < cost) {
            best = nb;
            cost = c;
            ntn = n;
        }
    }
    StreamArgs p{a, tiles, ntn};
    const long long grid = (long long)ntm * ntn;
    if (grid > 0x7FFFFFFFLL) return hipErrorInvalidValue;
    if (fmt == FMT_I4G) {
        if (a.dtype == QGEMV_BF16) run_stream<FMT_I4G, BF16>(p, best, (unsigned)grid, st);
        else run_stream<FMT_I4G, F32>(p, best, (unsigned)grid, st);
    } else {
        if (a.dtype == QGEMV_BF16) run_stream<FMT_FP8, BF16>(p, best, (unsigned)grid, st);
        else run_stream<FMT_FP8, F32>(p, best, (unsigned)grid, st);
    }
    return hipGetLastError();
}

}  // namespace qg
