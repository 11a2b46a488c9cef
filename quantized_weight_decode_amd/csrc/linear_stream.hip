// linear_stream.hip -- few rows of x times packed weights, bound by the
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

// Codes enter the matrix instructions times 2^-k, and a row's scales times 2^k,
// so that a scale group's sum stays finite for every finite x: with group sums
// of up to 128 columns in units of max |x|, fp8 448 * 128 < 2^16, int4 q - 8 8 *
// 128 < 2^11, and int4 16 + q from -24 sum x on 31 * 128 < 2^12 (the partial
// sums stay within it).  Powers of two: the codes stay exact, and sums below
// 2^-126 are subnormal, which the matrix instructions keep (to 2^-149).
constexpr int FP8_DOWN = 16, SIGNED_DOWN = 11, OFFSET_DOWN = 12;

constexpr float pow2(int e) { return e < 0 ? 1.0f / (float)(1 << -e) : (float)(1 << e); }

// Two E4M3 codes times 2^e in bf16, exactly.
template <int E>
__device__ __forceinline__ bf16x2 cvt_lo(uint32_t w)
{
    return __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)w, pow2(E), false);
}
template <int E>
__device__ __forceinline__ bf16x2 cvt_hi(uint32_t w)
{
    return __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)w, pow2(E), true);
}

// Eight nibbles as (16 + q) 2^-OFFSET_DOWN in bf16 (0x4180 | 8 q is 16 + q), in
// the column order 0 4 1 5 2 6 3 7; and -24 times the same.
constexpr uint32_t bf16_pair(uint32_t bits) { return (bits - (OFFSET_DOWN << 7)) * 0x10001u; }
__device__ __forceinline__ bf16x8 nib8_bf16(uint32_t w)
{
    constexpr uint32_t M = 0x00780078u, B = bf16_pair(0x4180u);
    const u32x4 o = {and_or(w << 3, M, B), and_or(w >> 1, M, B), and_or(w >> 5, M, B),
                     and_or(w >> 9, M, B)};
    return __builtin_bit_cast(bf16x8, o);
}
// Eight nibbles as (q - 8) 2^-SIGNED_DOWN, in the column order 0 2 4 6 1 3 5 7.  Read as E4M3
// codes, 0..15 are n 2^-9, so bytes of one nibble each convert two at a time.
// t = the two's complement nibble; its code is t for t < 8,
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
    constexpr int E = 9 - SIGNED_DOWN;
    return join(cvt_lo<E>(lo), cvt_hi<E>(lo), cvt_lo<E>(hi), cvt_hi<E>(hi));
}

__device__ __forceinline__ uint32_t low_halves(uint32_t a, uint32_t b)
{
    return __builtin_amdgcn_perm(b, a, 0x05040100u);
}
__device__ __forceinline__ uint32_t high_halves(uint32_t a, uint32_t b)
{
    return __builtin_amdgcn_perm(b, a, 0x07060302u);
}

// Eight activations of a lane, read from LDS as they are in memory, as NP bf16
// parts in the weights' column order.
template <typename XT, int FMT>
struct XFrag;
template <int FMT>
struct XFrag<BF16, FMT> {
    static constexpr int NP = 1;
    static __device__ __forceinline__ void parts(const char *p, bf16x8 out[1])
    {
        const u32x4 v = *reinterpret_cast<const u32x4 *>(p);
        u32x4 o = v;
        if (FMT == FMT_I4G) {
            o.x = low_halves(v.x, v.z);
            o.y = high_halves(v.x, v.z);
            o.z = low_halves(v.y, v.w);
            o.w = high_halves(v.y, v.w);
        }
        out[0] = __builtin_bit_cast(bf16x8, o);
    }
};
// f32 = three bf16 parts of eight bits each, exactly: each part is the high
// half of what is left.
template <int FMT>
struct XFrag<F32, FMT> {
    static constexpr int NP = 3;
    static __device__ __forceinline__ void parts(const char *p, bf16x8 out[3])
    {
        const f32x4 a = *reinterpret_cast<const f32x4 *>(p);
        const f32x4 b = *reinterpret_cast<const f32x4 *>(p + 16);
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

// A lane's 16 bytes of x on the way to LDS as bf16 in the weights' column order
// (of each eight), f32 as three parts of eight bits each, exactly: each part is
// the high half of what is left.
template <typename XT, int FMT>
struct XParts;
template <int FMT>
struct XParts<BF16, FMT> {                               // eight columns
    static constexpr int NP = 1;
    static __device__ __forceinline__ void store(char *at, int, int, u32x4 v)
    {
        u32x4 o = v;
        if (FMT == FMT_I4G) {
            o.x = low_halves(v.x, v.z);
            o.y = high_halves(v.x, v.z);
            o.z = low_halves(v.y, v.w);
            o.w = high_halves(v.y, v.w);
        }
        *reinterpret_cast<u32x4 *>(at) = o;
    }
};
template <int FMT>
struct XParts<F32, FMT> {                                // four columns, odd: the last of eight
    static constexpr int NP = 3;
    static __device__ __forceinline__ void store(char *at, int odd, int part_stride, u32x4 v)
    {
        uint32_t *const to = reinterpret_cast<uint32_t *>(at);
#pragma unroll
        for (int q = 0; q < 3; q++) {
            uint32_t *const d = to + q * (part_stride / 4);
            if (FMT == FMT_I4G) {
                d[odd] = high_halves(v.x, v.z);
                d[odd + 2] = high_halves(v.y, v.w);
            } else {
                d[2 * odd] = high_halves(v.x, v.y);
                d[2 * odd + 1] = high_halves(v.z, v.w);
            }
#pragma unroll
            for (int j = 0; j < 4; j++) {
                const uint32_t all = v[j], high = all & 0xFFFF0000u;
                v[j] = __builtin_bit_cast(uint32_t, __builtin_bit_cast(float, all) -
                                                        __builtin_bit_cast(float, high));
            }
        }
    }
};

struct StreamArgs {
    LinearArgs a;
    const RowTile *tiles;
    int ntn;
};

// Stream kernel.  A workgroup of 8 waves makes up to ROWS rows of y x 16 NB
// rows of W; the waves take blocks of P chunks of 128 columns in turn, and
// their sums are joined through LDS in a fixed order.
// v_mfma_f32_16x16x32_bf16, lane l: A row of x l % 16, B row of W l % 16, eight
// columns from the lane group l / 16.
//
// Lanes next to each other load 16-byte pieces of one row (a load of 64 lanes
// in 64 different rows takes the vector cache 64 cycles, whatever its width),
// whole 128-byte lines at a time.  Each wave passes its block through its own
// part of LDS to get the fragments' order, and as soon as the weights are in
// LDS asks for its next block, so that one block per wave is always in flight.
//
// bf16 activations multiply 16 + q, and the group's sum starts from -24 sum(x),
// one more matrix instruction per group: a rounding is up to 2^-24 (sum (16 + q)
// |x| + 24 sum |x|) of the group.  With all of x of one size that is 48 / 4 times
// 2^-24 of the sum of |(q - 8) x|, far below bf16's 2^-9; one element 10^4 times
// the others at a zero weight adds 2^-24 * 48 * 10^4 = 0.03 of them, still below
// the rounding of an output of 2000 columns (2^-9 of 4 sqrt(2000)), one of 10^6
// no longer.  f32 activations multiply q - 8, whose unpacking costs 2.5 instead
// of 0.9 instructions per weight: their outputs would show it much sooner.
//
// ROWS = 16 or 32: x goes to LDS as it is in memory, and each fragment is turned into
// bf16 parts as it is read; three parts of f32 take three matrix instructions.
// ROWS = 4 (dense): the parts are made on the way to LDS, once per element
// instead of once per lane of a fragment, and the three parts of four rows are
// the rows of one fragment; their sums are added in the end.  One f32 row of
// 6144 x 12288 15.7 us (with ROWS = 16 20.8), of 7168 x 2048 7.9 (11.9); bf16
// 12.4 (13.3) and 6.6 (7.4).
// 42 MB of weights and scales at the 4.8 TB/s of a large copy take 8.8 us; two
// blocks in flight per wave (14.3 us) and blocks of 512 columns (13.8) are
// slower than one of 256.
template <int FMT, typename XT, int NB, bool GATED, int FG, int P, int ROWS>
__global__ __launch_bounds__(512, 2) void linear_stream(StreamArgs p)
{
    typedef typename XT::raw raw;
    typedef XFrag<XT, FMT> Frag;
    constexpr bool FEW = ROWS == 4;
    constexpr int MT = FEW ? 1 : ROWS / 16;              // row tiles
    constexpr int NP = FEW ? 1 : Frag::NP;               // matrix instructions per step
    constexpr int XQ = FEW ? Frag::NP : 1;               // parts of x beside each other
    constexpr bool OFFSET = FMT == FMT_I4G && Frag::NP == 1;
    constexpr float UP = pow2(FMT == FMT_FP8 ? FP8_DOWN : OFFSET ? OFFSET_DOWN : SIGNED_DOWN);
    constexpr int NG = SC / FG;                          // scale groups of a chunk
    constexpr int TPG = 4 / NG;                          // 32-column steps of a group
    constexpr int WC = FMT == FMT_FP8 ? 8 : 4;           // 16-byte pieces of a row and chunk
    constexpr int WP = P * WC;                           // and block
    constexpr int WL = NB * 16 * WP / 64;                // weight loads of a lane and block
    constexpr int WROW = WP * 16 + 16;                   // LDS row stride, bytes
    constexpr int NGB = P * NG;                          // scale groups of a block
    constexpr int SL = (NB * 16 * NGB + 63) / 64;        // scale loads
    constexpr int XP = SC * sizeof(raw) / 16;            // 16-byte pieces of a row and chunk of x
    constexpr int XR = 64 / XP;                          // rows of x per load
    constexpr int XL = ROWS / XR;                        // loads of x
    constexpr int XROW = (FEW ? P * SC * 2 : SC * (int)sizeof(raw)) + 16;   // LDS row stride, bytes
    constexpr int YC = GATED ? NB * 8 : NB * 16;         // columns of y
    constexpr int LDR = NB * 16 + 4;
    constexpr int WB = NB * 16 * WROW, SB = SL * 256;
    constexpr int WAVE_LDS = WB + SB + ROWS * XQ * XROW;
    constexpr int RED = SW * 16 * MT * LDR * 4;
    __shared__ __align__(16) char smem[SW * WAVE_LDS > RED ? SW * WAVE_LDS : RED];
    const LinearArgs &a = p.a;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int li = lane & 15, lg = lane >> 4;
    const int oc = GATED ? a.O / 2 : a.O;
    const int nt = (int)(blockIdx.x % p.ntn), mt = (int)(blockIdx.x / p.ntn);
    RowTile t;
    if (p.tiles) t = p.tiles[mt];
    else t = RowTile{0, mt * ROWS, min(ROWS, a.R - mt * ROWS), 0};
    t.n = __builtin_amdgcn_readfirstlane(t.n);
    t.expert = __builtin_amdgcn_readfirstlane(t.expert);
    if (t.n <= 0) return;                                // uniform over the workgroup

    // x: lane's piece lane % XP of row lane / XP + XR i of the tile
    const raw *xp[XL];
#pragma unroll
    for (int i = 0; i < XL; i++) {
        int r = lane / XP + XR * i;
        r = t.row0 + (r < t.n ? r : 0);
        if (a.rows) {
            r = a.rows[r];
            if (r < 0 || r >= a.T) r = 0;                // marked in the epilogue
        }
        xp[i] = static_cast<const raw *>(a.x) + (size_t)r * a.ldx +
                (lane % XP) * (16 / sizeof(raw));
    }

    const size_t rb = FMT == FMT_I4G ? (size_t)a.I / 2 : (size_t)a.I;
    const uint8_t *const wbase = a.w + (size_t)t.expert * a.w_stride;
    const float *const sbase = a.scales + (size_t)t.expert * a.s_stride;
    // row i of the workgroup's 16 NB
    auto weight_row = [&](int i) {
        const int n = i >> 4;
        const int half = GATED ? n / (NB / 2) : 0;
        const int c = nt * YC + (GATED ? n % (NB / 2) : n) * 16 + (i & 15);
        return (c < oc ? c : oc - 1) + half * oc;
    };
    uint32_t woff[WL], soff[SL];
#pragma unroll
    for (int i = 0; i < WL; i++)
        woff[i] = (uint32_t)(weight_row((lane + 64 * i) / WP) * rb);
#pragma unroll
    for (int i = 0; i < SL; i++) {
        const int row = weight_row(min((lane + 64 * i) / NGB, NB * 16 - 1));
        soff[i] = (uint32_t)(FMT == FMT_I4G ? row : row >> 7) * (uint32_t)a.ng;
    }
    const int lane_k = (lane % WP) * (FMT == FMT_FP8 ? 16 : 32);

    // the wave's LDS: weights, scales, rows of x
    char *const wl = smem + wave * WAVE_LDS;
    float *const sl = reinterpret_cast<float *>(wl + WB);
    char *const xl = wl + WB + SB;
    if (!FEW)                                            // rows past the tile's: zero
        for (int i = lane; i < ROWS * XROW / 16; i += 64)
            reinterpret_cast<u32x4 *>(xl)[i] = u32x4{0, 0, 0, 0};

    u32x4 wr[WL], xr[P][XL];
    float sr[SL];
    const int blocks = (a.I + P * SC - 1) / (P * SC);
    const int gs = FMT == FMT_FP8 ? 128 : a.gs;
    const int nx = (t.n + XR - 1) / XR;                  // loads of x that hold rows
    // A wave without a block, and a lane behind the row's end, load valid data
    // again (of x, the row's first piece); it meets zeros of x.
    auto load_w = [&](int c) {
        const int k0 = min(c, blocks - 1) * (P * SC);
        const uint32_t kb = min((uint32_t)(FMT == FMT_I4G ? (k0 + lane_k) / 2 : k0 + lane_k),
                                (uint32_t)rb - 16);
#pragma unroll
        for (int i = 0; i < WL; i++)
            wr[i] = ld_stream(reinterpret_cast<const u32x4 *>(wbase + (woff[i] + kb)));
        const uint32_t gi = (uint32_t)min(k0 + (lane % NGB) * FG, a.I - 1) / (uint32_t)gs;
#pragma unroll
        for (int i = 0; i < SL; i++) sr[i] = sbase[soff[i] + gi];
    };
    auto x_inside = [&](int c, int q) {                  // this lane's columns exist
        return (c * P + q) * SC + (lane % XP) * (int)(16 / sizeof(raw)) < a.I;
    };
    auto load_x = [&](int c) {
#pragma unroll
        for (int q = 0; q < P; q++) {
            const int kx =
                x_inside(c, q) ? (c * P + q) * SC : -(lane % XP) * (int)(16 / sizeof(raw));
#pragma unroll
            for (int i = 0; i < XL; i++)
                if (i < nx) xr[q][i] = *reinterpret_cast<const u32x4 *>(xp[i] + kx);
        }
    };
    // to LDS; only this wave uses this part, and its LDS operations complete in
    // order
    auto store_w = [&]() {
#pragma unroll
        for (int i = 0; i < WL; i++)
            *reinterpret_cast<u32x4 *>(wl + ((lane + 64 * i) / WP) * WROW + (lane % WP) * 16) =
                wr[i];
#pragma unroll
        for (int i = 0; i < SL; i++) sl[lane + 64 * i] = sr[i] * UP;
    };
    auto store_x = [&](int c, int q) {
#pragma unroll
        for (int i = 0; i < XL; i++) {
            const u32x4 v = x_inside(c, q) ? xr[q][i] : u32x4{0, 0, 0, 0};
            const int r = lane / XP + XR * i;
            if (FEW) {
                constexpr int PW = 16 / sizeof(raw);     // columns of a piece
                const int k = q * SC + (lane % XP) * PW;
                if (i < nx)
                    XParts<XT, FMT>::store(xl + r * XROW + k / 8 * 16, k / 4 & 1, ROWS * XROW, v);
            } else if (i < nx && r < t.n)
                *reinterpret_cast<u32x4 *>(xl + r * XROW + (lane % XP) * 16) =
                    v;
        }
    };

    f32x4v acc[MT][NB];
#pragma unroll
    for (int m = 0; m < MT; m++)
#pragma unroll
        for (int n = 0; n < NB; n++) acc[m][n] = f32x4v{0.0f, 0.0f, 0.0f, 0.0f};

    auto multiply = [&](int q) {                         // chunk q of the block
        uint32_t wd[NB][WC];
#pragma unroll
        for (int n = 0; n < NB; n++) {
            const char *row = wl + (n * 16 + li) * WROW + q * (WC * 16);
#pragma unroll
            for (int u = 0; u < WC / 4; u++) {
                const u32x4 v = *reinterpret_cast<const u32x4 *>(row + 64 * u + 16 * lg);
#pragma unroll
                for (int j = 0; j < 4; j++) wd[n][4 * u + j] = v[j];
            }
            if (FMT == FMT_I4G) transpose4(wd[n]);
        }
#pragma unroll
        for (int g = 0; g < NG; g++) {
            bf16x8 xv[MT][TPG][NP];
            f32x4v z[MT];
#pragma unroll
            for (int m = 0; m < MT; m++) {
#pragma unroll
                for (int s = 0; s < TPG; s++) {
                    const int st = g * TPG + s;
                    const int k = FMT == FMT_I4G ? 32 * st + 8 * lg
                                                 : 64 * (st >> 1) + 16 * lg + 8 * (st & 1);
                    if (FEW)                             // rows behind the last repeat others
                        xv[m][s][0] = *reinterpret_cast<const bf16x8 *>(
                            xl + (li % (ROWS * XQ)) * XROW + (q * SC + k) * 2);
                    else
                        Frag::parts(xl + (16 * m + li) * XROW + k * sizeof(raw), xv[m][s]);
                }
                z[m] = f32x4v{0.0f, 0.0f, 0.0f, 0.0f};
                if (OFFSET) {
                    constexpr uint32_t M = bf16_pair(0xC1C0u);
                    const u32x4 m24 = {M, M, M, M};
#pragma unroll
                    for (int s = 0; s < TPG; s++)
                        z[m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                            xv[m][s][0], __builtin_bit_cast(bf16x8, m24), z[m], 0, 0, 0);
                }
            }
#pragma unroll
            for (int n = 0; n < NB; n++) {
                const float sc = sl[(n * 16 + li) * NGB + q * NG + g];
                f32x4v sum[MT];
#pragma unroll
                for (int m = 0; m < MT; m++) sum[m] = z[m];
#pragma unroll
                for (int s = 0; s < TPG; s++) {
                    const int st = g * TPG + s;
                    bf16x8 wv;
                    if (FMT == FMT_I4G) {
                        wv = OFFSET ? nib8_bf16(wd[n][st]) : nib8_bf16_signed(wd[n][st]);
                    } else {
                        const uint32_t p0 = wd[n][(2 * st) % WC];
                        const uint32_t p1 = wd[n][(2 * st + 1) % WC];
                        constexpr int E = -FP8_DOWN;
                        wv = join(cvt_lo<E>(p0), cvt_hi<E>(p0), cvt_lo<E>(p1), cvt_hi<E>(p1));
                    }
#pragma unroll
                    for (int m = 0; m < MT; m++)
#pragma unroll
                        for (int q = NP - 1; q >= 0; q--)    // small parts first
                            sum[m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xv[m][s][q], wv,
                                                                             sum[m], 0, 0, 0);
                }
#pragma unroll
                for (int m = 0; m < MT; m++)
#pragma unroll
                    for (int r = 0; r < 4; r++)
                        acc[m][n][r] = fmaf(sc, sum[m][r], acc[m][n][r]);
            }
            if (NG == 4) __builtin_amdgcn_sched_barrier(0);    // keeps registers down
        }
    };

    load_x(wave);
    load_w(wave);
    for (int c = wave; c < blocks; c += SW) {
        const bool more = c + SW < blocks;               // uniform over the wave
        store_w();
#pragma unroll
        for (int q = 0; q < (FEW ? P : 1); q++) store_x(c, q);
        __builtin_amdgcn_sched_barrier(0);
        if (more) load_w(c + SW);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int q = 0; q < P; q++) {
            if (!FEW && q > 0) store_x(c, q);
            __builtin_amdgcn_wave_barrier();             // lanes read each other's pieces
            if (more && q == (FEW ? 0 : P - 1)) load_x(c + SW);
            multiply(q);
            __builtin_amdgcn_sched_barrier(0);
        }
    }

    __syncthreads();
    float (*const red)[16 * MT][LDR] = reinterpret_cast<float (*)[16 * MT][LDR]>(smem);
#pragma unroll
    for (int m = 0; m < MT; m++)
#pragma unroll
        for (int n = 0; n < NB; n++)
#pragma unroll
            for (int r = 0; r < 4; r++)
                red[wave][16 * m + 4 * lg + r][n * 16 + li] = acc[m][n][r];
    __syncthreads();
    finish<XT, 2>(a, t.expert, tid, SW * 64, t.n * YC,
                  [&](int i, int &row, int &col, float &v, float &up) {
                      const int r = i / YC, c = i % YC;
                      row = t.row0 + r;
                      col = nt * YC + c;
                      v = up = 0.0f;
#pragma unroll
                      for (int w = 0; w < SW; w++)
#pragma unroll
                          for (int q = XQ - 1; q >= 0; q--) {
                              v += red[w][q * 4 + r][c];
                              if (GATED) up += red[w][q * 4 + r][c + YC];
                          }
                      if (a.rows) {
                          const int xi = a.rows[row];
                          if (xi < 0 || xi >= a.T) v = up = __builtin_nanf("");
                      }
                  });
}

// Most row blocks that 32 rows of x leave registers for, 0: none worth it.  int4:
// three; four spill 360 bytes per lane (32 x 4096 x 14336 21.2 us, the narrow
// kernel 16.9), and three 128 with a scale per 32 columns (32 x 6144 x 12288 35.9
// us, the narrow kernel 22.3).  Two (and with them int4's gated products, whose
// blocks come in pairs) cover no more rows of W than two workgroups of 16 rows.
constexpr int wide_blocks(int fmt, int fg, bool gated)
{
    return fmt == FMT_FP8 ? 4 : gated || fg == 32 ? 0 : 3;
}
// Columns of a scale group that the kernel is built for.
int group_columns(WeightFormat fmt, int gs)
{
    return fmt == FMT_FP8 || gs % 128 == 0 ? 128 : gs % 64 == 0 ? 64 : 32;
}

template <int FMT, typename XT, int NB, bool GATED>
void run_nb(const StreamArgs &p, int rows, unsigned grid, hipStream_t st)
{
    constexpr int P = FMT == FMT_I4G ? 2 : 1;
#define QG_RUN_R(FG, ROWS)                                                                  \
    hipLaunchKernelGGL((linear_stream<FMT, XT, NB, GATED, FG, P, ROWS>), dim3(grid),        \
                       dim3(SW * 64), 0, st, p)
#define QG_RUN(FG)                                                                          \
    do {                                                                                    \
        if (rows == 4) QG_RUN_R(FG, 4);                                                     \
        else if (rows == 16) QG_RUN_R(FG, 16);                                              \
        else if constexpr (sizeof(typename XT::raw) == 2 && NB > 2 &&                       \
                           NB <= wide_blocks(FMT, FG, GATED))                               \
            QG_RUN_R(FG, 32);                                                               \
    } while (0)
    if constexpr (FMT == FMT_FP8) {
        QG_RUN(128);
    } else {
        const int fg = group_columns(FMT_I4G, p.a.gs);
        if (fg == 128) QG_RUN(128);
        else if (fg == 64) QG_RUN(64);
        else QG_RUN(32);
    }
#undef QG_RUN
#undef QG_RUN_R
}

template <int FMT, typename XT>
void run_stream(const StreamArgs &p, int rows, int nb, unsigned grid, hipStream_t st)
{
    if (p.a.gated) {
        if (nb == 4) run_nb<FMT, XT, 4, true>(p, rows, grid, st);
        else run_nb<FMT, XT, 2, true>(p, rows, grid, st);
    } else if (nb == 4) {
        run_nb<FMT, XT, 4, false>(p, rows, grid, st);
    } else if (nb == 3) {
        run_nb<FMT, XT, 3, false>(p, rows, grid, st);
    } else if (nb == 2) {
        run_nb<FMT, XT, 2, false>(p, rows, grid, st);
    } else {
        run_nb<FMT, XT, 1, false>(p, rows, grid, st);
    }
}

}  // namespace

// Up to 16 rows, and more while all workgroups fit the GPU at once, with 16 or
// (bf16) 32 rows each; a grouped bf16 product up to 9 rows for an expert on
// average, a grouped f32 one up to 8 in all.  us, this kernel and tiles:
// 16 rows: bf16, 64 x 4096 x 4096 10.8 and 15.4, 96 x 4096 x 4096 (384 workgroups)
// 20.4 and 15.8; 32 x 7168 x 2048 8.7 and 20.5; f32, 64 x 4096 x 4096 17.5 and 20.6,
// 64 x 14336 x 4096 48.2 and 47.7, 32 x 2048 x 6144 9.6 and 13.8.
// 32 rows: int4, 17 x 6144 x 12288 16.1 and 19.8, 32 x 6144 x 12288 18.7 and 20.8
// (two of 16 rows 26.4), 64 x 2048 x 6144 9.4 and 11.6; fp8, 32 x 7168 x 16384 25.8
// and 33.1, 64 x 16384 x 7168 44.8 and 52.0.
// Grouped bf16, 7168 x 2048, 256 experts: 128 tokens of 8 (4 rows) 396 and 465,
// 256 (8) 531 and 557, 320 (10) 591 and 574, 512 (16) 789 and 622; 2048 x 1024,
// 32 experts: 8 rows 24.1 and 27.7, 10 rows 32.2 and 28.8.
// Grouped f32, 2048 x 4096, 8 experts: 2 rows in all 11.6 and 14.9, 8 rows 20.4 and
// 21.0, 16 rows 27.1 and 24.8; 7168 x 2048, 64 rows 200 and 154.
int stream_rows(WeightFormat fmt, const LinearArgs &a)
{
    const int el = a.dtype == QGEMV_BF16 ? 2 : 4;
    if (!tile_fits(fmt, a) || (((uintptr_t)a.x | (uintptr_t)(a.ldx * el)) & 15) != 0) return 0;
    if (a.offsets) {
        const bool few = a.dtype == QGEMV_BF16 ? a.R <= 9 * (long long)a.E : a.R <= 8;
        return few ? 16 : 0;
    }
    if (a.R <= 4) return 4;
    const long long ncu = cu_count(), O = a.O;
    if (a.R <= 16 || (a.R + 15) / 16 * ((O + 63) / 64) <= ncu) return 16;
    const int cols = 16 * wide_blocks(fmt, group_columns(fmt, a.gs), a.gated);
    return a.dtype == QGEMV_BF16 && cols && (a.R + 31) / 32 * ((O + cols - 1) / cols) <= ncu ? 32
                                                                                          : 0;
}

// Row blocks per workgroup: the count that leaves the busiest CU the least to
// do, a workgroup of 16 rows of x counted as its row blocks and 1.5 for its x
// (48 x 4096 x 4096 f32: one workgroup of four blocks per CU 17.5 us, three of
// one 27.7); among equals the largest, which shares each x fragment among
// the most rows, but for up to four rows of bf16 by int4, where that is
// cheap, the smallest (1 x 6144 x 12288: 12.4 us, three
// blocks 13.0; f32 16.3 and 16.0; fp8 1 x 7168 x 16384: 22.7, four 21.4).
// Four blocks of 16 f32 rows with a scale per 32 columns spill 84 bytes per lane,
// three none, within 1 % of each other: 16 x 6144 x 12288 25.3 and 25.1, 5 x
// 16384 x 7168 36.6 and 36.6.
static void pick_blocks(WeightFormat fmt, const LinearArgs &a, int rows, int ntm, int &best,
                        int &ntn)
{
    const int oc = a.gated ? a.O / 2 : a.O;
    const long long ncu = cu_count();
    const bool small = rows == 4 && fmt == FMT_I4G && a.dtype == QGEMV_BF16;
    best = ntn = 0;
    double cost = 0.0;
    // (32 rows: three or four, in one round of the CUs)
    const int most = rows == 32 ? wide_blocks(fmt, group_columns(fmt, a.gs), a.gated) : 4;
    for (int nb = most; nb >= (rows == 32 ? 3 : 1); nb--) {
        if (a.gated && (nb & 1)) continue;
        const int yc = a.gated ? nb * 8 : nb * 16;
        const int n = (oc + yc - 1) / yc;
        const double c = (double)(((long long)n * ntm + ncu - 1) / ncu) *
                         (nb + (rows == 4 ? 0.0 : 1.5));
        if (!best || c < cost || (c == cost && small)) {
            best = nb;
            cost = c;
            ntn = n;
        }
    }
}

long long stream_items(WeightFormat fmt, const LinearArgs &a, int rows, int ntm)
{
    int best, ntn;
    pick_blocks(fmt, a, rows, ntm, best, ntn);
    return (long long)ntm * ntn * (SW * 64);
}

hipError_t launch_stream(WeightFormat fmt, const LinearArgs &a, int rows, const RowTile *tiles,
                         int ntm, hipStream_t st)
{
    int best, ntn;
    pick_blocks(fmt, a, rows, ntm, best, ntn);
    StreamArgs p{a, tiles, ntn};
    const long long grid = (long long)ntm * ntn;
    if (fmt == FMT_I4G) {
        if (a.dtype == QGEMV_BF16) run_stream<FMT_I4G, BF16>(p, rows, best, (unsigned)grid, st);
        else run_stream<FMT_I4G, F32>(p, rows, best, (unsigned)grid, st);
    } else {
        if (a.dtype == QGEMV_BF16) run_stream<FMT_FP8, BF16>(p, rows, best, (unsigned)grid, st);
        else run_stream<FMT_FP8, F32>(p, rows, best, (unsigned)grid, st);
    }
    return hipGetLastError();
}

}  // namespace qg
