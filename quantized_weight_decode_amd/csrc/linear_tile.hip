// linear_tile.hip -- many rows of x times packed weights on the f16 matrix
// cores, dense or grouped by expert, with the epilogue.
#include "qg_device.h"
#include "qg_linear.h"
#include "qg_tile.h"

namespace qg {

namespace {

// ---------------------------------------------------------------------------
// Packed activations.
//
// Each row of x is scaled by a power of two, x' = x 2^(15 - E) with max|x| in
// [2^(E-1), 2^E) over its finite values, so that 2^14 <= max|x'| < 2^15, and
// stored as f16: bf16 values exactly down to 2^-28 of the maximum (below it
// to 2^-39 of the maximum); f32 values as two planes, hi = f16(x') and lo =
// f16(x' - hi), together within 2^-22 of themselves down to 2^-17 of the
// maximum and within 2^-39 of it below, where lo is subnormal (an f32 sum's own
// roundings are of that size).
// The exponent E - 15 is undone on the f32 sum.  int4 weights unpack in the
// column order 0 4 1 5 2 6 3 7 of each eight; x is stored in that order.
// Rows are padded with zeros to whole K steps.
//
// One workgroup of TH threads per row, the row in registers between the
// maximum and the scaling (NCH pieces of eight per thread; NCH = 0: rows too
// long for that are read twice), VEC: rows on 16 bytes.  Bound by HBM for many
// rows (x read once, 2 or 4 bytes per element written), by latency for few.
// ---------------------------------------------------------------------------
template <typename XT>
__device__ __forceinline__ void load8(const typename XT::raw *src, bool vec, float v[8])
{
    typedef typename XT::raw raw;
    if (vec) {
        typedef typename Eight<raw>::type rawx8;
        const rawx8 t = *reinterpret_cast<const rawx8 *>(src);
#pragma unroll
        for (int j = 0; j < 8; j++) v[j] = XT::get(t[j]);
    } else {
#pragma unroll
        for (int j = 0; j < 8; j++) v[j] = XT::get(src[j]);
    }
}

// largest finite |v| by its bits
__device__ __forceinline__ uint32_t max_bits(uint32_t m, const float v[8])
{
#pragma unroll
    for (int j = 0; j < 8; j++) {
        const uint32_t b = __builtin_bit_cast(uint32_t, v[j]) & 0x7FFFFFFFu;
        m = b < 0x7F800000u && b > m ? b : m;
    }
    return m;
}

template <int FMT>
__device__ __forceinline__ void store8(const float v[8], int shift, _Float16 *hi, _Float16 *lo)
{
    f16x8 h, l;
#pragma unroll
    for (int j = 0; j < 8; j++) {
        const float t = ldexpf(v[FMT == FMT_I4G ? (j >> 1) + 4 * (j & 1) : j], shift);
        h[j] = (_Float16)t;
        l[j] = (_Float16)(t - (float)h[j]);
    }
    *reinterpret_cast<f16x8 *>(hi) = h;
    if (lo) *reinterpret_cast<f16x8 *>(lo) = l;
}

template <typename XT, int FMT, int TH, int NCH, bool VEC>
__global__ __launch_bounds__(TH) void pack_rows(const typename XT::raw *__restrict__ x,
                                                long long ldx, int I, int Ip, int ldp,
                                                _Float16 *__restrict__ hi,
                                                _Float16 *__restrict__ lo,
                                                int *__restrict__ rexp)
{
    __shared__ uint32_t wmax[TH / 64];
    const int tid = threadIdx.x;
    const long long t = blockIdx.x;
    const typename XT::raw *src = x + (size_t)t * ldx;
    hi += (size_t)t * ldp;
    if (lo) lo += (size_t)t * ldp;
    float v[NCH ? NCH : 1][8];
    uint32_t m = 0;
    if (NCH) {
#pragma unroll
        for (int i = 0; i < NCH; i++) {
            const int c = (tid + TH * i) * 8;            // I is a multiple of 32
#pragma unroll
            for (int j = 0; j < 8; j++) v[i][j] = 0.0f;
            if (c < I) load8<XT>(src + c, VEC, v[i]);
        }
#pragma unroll
        for (int i = 0; i < NCH; i++) m = max_bits(m, v[i]);
    } else {
        for (int c = tid * 8; c < I; c += TH * 8) {
            load8<XT>(src + c, VEC, v[0]);
            m = max_bits(m, v[0]);
        }
    }
#pragma unroll
    for (int d = 32; d > 0; d /= 2) {
        const uint32_t o = (uint32_t)__shfl_xor((int)m, d);
        m = o > m ? o : m;
    }
    if (TH > 64) {
        if ((tid & 63) == 0) wmax[tid >> 6] = m;
        __syncthreads();
        m = 0;
#pragma unroll
        for (int i = 0; i < TH / 64; i++) m = wmax[i] > m ? wmax[i] : m;
    }
    int E = 0;
    if (m) frexpf(__builtin_bit_cast(float, m), &E);
    if (tid == 0) rexp[t] = E - 15;
    if (NCH) {
#pragma unroll
        for (int i = 0; i < NCH; i++) {
            const int c = (tid + TH * i) * 8;
            if (c < Ip) store8<FMT>(v[i], 15 - E, hi + c, lo ? lo + c : nullptr);
        }
    } else {
        for (int c = tid * 8; c < Ip; c += TH * 8) {
#pragma unroll
            for (int j = 0; j < 8; j++) v[0][j] = 0.0f;
            if (c < I) load8<XT>(src + c, VEC, v[0]);
            store8<FMT>(v[0], 15 - E, hi + c, lo ? lo + c : nullptr);
        }
    }
}

template <typename XT, int FMT, bool VEC>
void run_pack(const LinearArgs &a, int Ip, int ldp, _Float16 *hi, _Float16 *lo, int *rexp, hipStream_t st)
{
#define QG_PACK(TH, NCH)                                                                    \
    hipLaunchKernelGGL((pack_rows<XT, FMT, TH, NCH, VEC>), dim3(a.T), dim3(TH), 0, st,      \
                       static_cast<const typename XT::raw *>(a.x), a.ldx, a.I, Ip, ldp, hi, lo, rexp)
    if (Ip <= 2048) QG_PACK(64, 4);
    else if (Ip <= 8192) QG_PACK(256, 4);
    else if (Ip <= 16384) QG_PACK(256, 8);
    else QG_PACK(256, 0);
#undef QG_PACK
}

template <typename XT>
hipError_t pack(WeightFormat fmt, const LinearArgs &a, int Ip, int ldp, _Float16 *hi,
                _Float16 *lo, int *rexp, hipStream_t st)
{
    const bool vec =
        (((uintptr_t)a.x | (uintptr_t)(a.ldx * sizeof(typename XT::raw))) & 15) == 0;
    if (fmt == FMT_I4G) {
        if (vec) run_pack<XT, FMT_I4G, true>(a, Ip, ldp, hi, lo, rexp, st);
        else run_pack<XT, FMT_I4G, false>(a, Ip, ldp, hi, lo, rexp, st);
    } else {
        if (vec) run_pack<XT, FMT_FP8, true>(a, Ip, ldp, hi, lo, rexp, st);
        else run_pack<XT, FMT_FP8, false>(a, Ip, ldp, hi, lo, rexp, st);
    }
    return hipGetLastError();
}

// Eight nibbles of a dword as q - 8 in f16, exactly, in the column order 0 4
// 1 5 2 6 3 7: 0x6400 | q is 1024 + q, and 0x6400 | 16 q is 1024 + 16 q =
// 16 (q - 8) + 1152.
__device__ __forceinline__ f16x8 nib8_f16(uint32_t w)
{
    const f16x2 one = {(_Float16)1.0f, (_Float16)1.0f};
    const f16x2 sixteenth = {(_Float16)0.0625f, (_Float16)0.0625f};
    const f16x2 c0 = {(_Float16)-1032.0f, (_Float16)-1032.0f};
    const f16x2 c1 = {(_Float16)-72.0f, (_Float16)-72.0f};
    const uint32_t w8 = w >> 8;
    const f16x2 a = __builtin_bit_cast(f16x2, and_or(w, 0x000F000Fu, 0x64006400u));
    const f16x2 b = __builtin_bit_cast(f16x2, and_or(w, 0x00F000F0u, 0x64006400u));
    const f16x2 c = __builtin_bit_cast(f16x2, and_or(w8, 0x000F000Fu, 0x64006400u));
    const f16x2 d = __builtin_bit_cast(f16x2, and_or(w8, 0x00F000F0u, 0x64006400u));
    const f16x2 r0 = a * one + c0, r1 = b * sixteenth + c1;
    const f16x2 r2 = c * one + c0, r3 = d * sixteenth + c1;
    return f16x8{r0.x, r0.y, r1.x, r1.y, r2.x, r2.y, r3.x, r3.y};
}

constexpr int BAD_ROW = -0x7FFFFFFF;     // exponent of a row of y without a row of x

constexpr int TK = 64;          // columns per K step
constexpr int TN = 256;         // rows of W per workgroup tile

struct TileArgs {
    LinearArgs a;
    const _Float16 *hi, *lo;
    const int *rexp;
    const RowTile *tiles;
    int Ip, ldp, ntm, ntn;                               // padded columns, row stride of hi, lo
    uint32_t g32, gmagic;                                // gs / 32 and 2^32 over it, rounded down
};

// Scale group of column 32 k32, by multiplication (the quotient is at most one
// too small).
__device__ __forceinline__ uint32_t scale_group(uint32_t k32, uint32_t g32, uint32_t magic)
{
    const uint32_t q = __umulhi(k32, magic);
    return q + ((q + 1) * g32 <= k32 ? 1u : 0u);
}

// A wave's weights and scales on their way through its part of LDS: ROWS rows
// of W by stages of 64 bytes per row (WS K steps: two of int4, one of fp8),
// two stages.  64 bytes at a time: loads of 32 bytes in one K step and the
// next 32 of the same line in the next one stall the vector cache while the
// line is on its way (routed prompt of 1024 tokens: half of all cycles).
// Lanes next to each other load 16-byte pieces of one row.  Piece c of a row
// sits at c ^ key(row), which spreads a fragment's rows over the banks.
template <int FMT, int FG, int ROWS>
struct Weights {
    static constexpr int WS = FMT == FMT_FP8 ? 1 : 2;
    static constexpr int SG = WS * TK / FG;              // scale groups of a stage
    static constexpr int NS = TK / FG;                   // and of a K step
    static constexpr int WL = ROWS * 4 / 64, SL = ROWS * SG / 64, LOADS = WL + SL;
    static constexpr uint32_t WBYTES = ROWS * 64, BYTES = WBYTES + ROWS * SG * 4;
    static constexpr int NB = ROWS / 16;
    uint32_t woff[WL], soff[SL], piece;

    static __device__ __forceinline__ int key(int row)
    {
        const int j = (row >> 2) & 3;
        return j ^ ((j & 1) << 1);
    }
    // row(i): row i of the wave's, as a row of W
    template <typename Row>
    __device__ __forceinline__ void init(const LinearArgs &a, uint32_t rb, int lane, Row row)
    {
#pragma unroll
        for (int i = 0; i < WL; i++) woff[i] = (uint32_t)row(lane / 4 + 16 * i) * rb;
        piece = ((lane & 3) ^ key(lane / 4)) * 16;
#pragma unroll
        for (int i = 0; i < SL; i++) {
            const int r = row((lane + 64 * i) / SG);
            soff[i] = (uint32_t)(FMT == FMT_I4G ? r : r >> 7) * (uint32_t)a.ng;
        }
    }
    // Stage st into LDS at `lds`.  Behind the row's end its last bytes are read
    // again, which meet zeros of x.
    __device__ __forceinline__ void load(const TileArgs &p, const uint8_t *wbase,
                                         const float *sbase, uint32_t rb, int st, uint32_t lds,
                                         int lane) const
    {
        const uint32_t kb = min((uint32_t)st * 64 + piece, rb - 16);
#pragma unroll
        for (int i = 0; i < WL; i++) load_lds16(wbase, woff[i] + kb, lds + 1024 * i);
        const uint32_t k32 = (uint32_t)st * (WS * TK / 32) + (lane % SG) * (FG / 32);
        const uint32_t g = min(scale_group(k32, p.g32, p.gmagic), (uint32_t)p.a.ng - 1);
#pragma unroll
        for (int i = 0; i < SL; i++)
            load_lds4(sbase, (soff[i] + g) * 4, lds + WBYTES + 256 * i);
    }
    // The lane's fragments and scales of K step `half` of the stage at `at`.
    static __device__ __forceinline__ void unpack(const char *at, int half, int lane,
                                                  f16x8 (&bv)[NB][2], float (&sc)[NB][NS])
    {
        const int li = lane & 15, lg = lane >> 4;
        const float *const sl = reinterpret_cast<const float *>(at + WBYTES) + half * NS;
        const char *row = at + li * 64;
        if (FMT == FMT_FP8) row += (lg ^ key(li)) * 16;
        else if (FG == 64) row += (((lg >> 1) ^ key(li) ^ (half * 2)) * 16) + (lg & 1) * 8;
        else row += ((key(li) ^ (half * 2)) * 16) + lg * 4;
#pragma unroll
        for (int n = 0; n < NB; n++) {
            const char *const r = row + n * 1024;
            if constexpr (FMT == FMT_FP8) {
                const u32x4 v = *reinterpret_cast<const u32x4 *>(r);
                bv[n][0] = fp8x8_f16(v.x, v.y);
                bv[n][1] = fp8x8_f16(v.z, v.w);
            } else if constexpr (FG == 64) {
                const u32x2 v = *reinterpret_cast<const u32x2 *>(r);
                bv[n][0] = nib8_f16(v.x);
                bv[n][1] = nib8_f16(v.y);
            } else {
                // the other 16 bytes of the K step: piece ^ 1
                const char *const o = at + ((r - at) ^ 16);
                bv[n][0] = nib8_f16(*reinterpret_cast<const uint32_t *>(r));
                bv[n][1] = nib8_f16(*reinterpret_cast<const uint32_t *>(o));
            }
#pragma unroll
            for (int j = 0; j < NS; j++) sc[n][j] = sl[(n * 16 + li) * SG + j];
        }
    }
};

// One K step of a wave: 16 MF rows of x (packed in LDS at sm, NP planes of 8
// MF rows x 128 bytes) times its unpacked weights, added to acc.
//
// Steps of two 16 x 16 blocks (n, n + 1) of one row block m and scale group j:
// a step's sums are added to the totals while the next step's matrix
// instructions run.  The scheduling barrier keeps the compiler from running
// ahead and holding many steps' values.  RAGGED: only mf row blocks.
template <int NP, int MF, int NB, int FG, bool RAGGED>
__device__ __forceinline__ void multiply_step(f32x4v (&acc)[MF][NB], const f16x8 (&bv)[NB][2],
                                              const float (&sc)[NB][TK / FG], const char *sm,
                                              int lane, int mf)
{
    constexpr int NS = TK / FG, NH = NB / 2, SPM = NH * NS;   // steps of a row block
    constexpr int CH = MF * 16 * 8;
    const int li = lane & 15, lg = lane >> 4;
    const f16x8 *const xs = reinterpret_cast<const f16x8 *>(sm);
    f16x8 am[2][NP][2];
    f32x4v g[2][2];
    auto read_a = [&](int m) {
#pragma unroll
        for (int q = 0; q < NP; q++)
#pragma unroll
            for (int h = 0; h < 2; h++) {
                const int ch = FG == 64 ? 2 * lg + h : 4 * h + lg;
                am[m & 1][q][h] = xs[q * CH + (m * 16 + li) * 8 + (ch ^ swizzle(li))];
            }
    };
    auto flush = [&](int s) {
        const int m = s / SPM, j = (s / NH) % NS, n = (s % NH) * 2;
#pragma unroll
        for (int i = 0; i < 2; i++)
#pragma unroll
            for (int r = 0; r < 4; r++)
                acc[m][n + i][r] = fmaf(sc[n + i][j], g[s & 1][i][r], acc[m][n + i][r]);
        // (not to be moved past the branches below)
        asm volatile("" : "+v"(acc[m][n]), "+v"(acc[m][n + 1]));
    };
    read_a(0);
#pragma unroll
    for (int m = 0; m < MF; m++) {
        if (!RAGGED || m < mf) {                         // uniform over the workgroup
            if (m + 1 < MF) read_a(m + 1);
#pragma unroll
            for (int s = m * SPM; s < (m + 1) * SPM; s++) {
                const int j = (s / NH) % NS, n = (s % NH) * 2;
                f32x4v t0 = {0.0f, 0.0f, 0.0f, 0.0f}, t1 = t0;
#pragma unroll
                for (int h = j * (2 / NS); h < (j + 1) * (2 / NS); h++)
#pragma unroll
                    for (int q = NP - 1; q >= 0; q--) {  // small parts first
                        t0 = __builtin_amdgcn_mfma_f32_16x16x32_f16(am[m & 1][q][h], bv[n][h], t0,
                                                                    0, 0, 0);
                        t1 = __builtin_amdgcn_mfma_f32_16x16x32_f16(am[m & 1][q][h],
                                                                    bv[n + 1][h], t1, 0, 0, 0);
                    }
                g[s & 1][0] = t0;
                g[s & 1][1] = t1;
                if (s > 0) flush(s - 1);
#pragma unroll
                for (int i = 0; i < 4 * NP / NS; i++) {
                    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
                    __builtin_amdgcn_sched_group_barrier(0x002, 2 * NS, 0);
                }
                __builtin_amdgcn_sched_barrier(0);
            }
        } else if (m == mf) {                            // the tile's last sums
            flush(m * SPM - 1);
        }
    }
    if (!RAGGED || mf == MF) flush(MF * SPM - 1);
}

// Tile kernel.  A workgroup of 4 waves makes 16 MF rows of y x 256 rows of W;
// each wave all 16 MF rows x 64 rows of W, so a weight is unpacked once per
// workgroup.  Everything comes by memory-to-LDS loads: the packed activations
// shared by the four waves, 16-byte chunks XOR-swizzled by row, each wave's
// weights and scales in a part of its own.  v_mfma_f32_16x16x32_f16, lane l: A
// row l % 16, B column l % 16, eight k from the lane group l / 16; D rows
// 4 (l / 16) + i, column l % 16.  The k order inside a K step is free as long
// as A and B agree: with one scale per 64 columns a lane group owns 16
// consecutive columns (8 bytes of int4), with one per 32 it owns eight of each
// 32.
// A scale group's products are summed from zero and added to the total as
// acc += s * sum in f32, one FMA per output and group, beside two matrix
// instructions.  RAGGED (grouped): row blocks of 16 behind the tile's rows are
// neither loaded nor multiplied; a dense product does without those branches
// (5 % faster at 2048 rows).
// Bound by the matrix cores and the unpacking beside them: int4 2048 x 6144 x
// 12288 bf16 gated, packing included, 309 us (1000 TFLOP/s), matrix cores busy
// 48 % of the CUs' busy cycles, five vector instructions per matrix instruction;
// the library's bf16 product of the same size takes 289 us (1069 TFLOP/s), of
// 8192^3 1364 TFLOP/s.  Routed prompts (4096 tokens of 8 of 256 experts, 7168 x
// 2048) fetch 7.8 GB in 1450 us, 3.6 times their bytes: 3.5 GB of weights, once
// per row tile, the rest x by the column blocks; matrix cores busy 36 %.
template <int FMT, typename XT, int NP, int MF, bool GATED, int FG, bool RAGGED>
__global__ __launch_bounds__(256, 2) void linear_tile(TileArgs p)
{
    constexpr int BM = 16 * MF;
    constexpr int CH = BM * 8;                           // 16-byte chunks of a plane
    constexpr int PT = CH / 256;                         // per thread
    static_assert(CH % 256 == 0, "whole chunks per thread");
    constexpr int LDO = TN + 4;                          // epilogue row stride, floats
    typedef Weights<FMT, FG, 64> W;
    constexpr int NS = TK / FG;                          // scales per row and step
    // LDS: AST stages of one K step of activations, two of each wave's weights.
    // Two workgroups share the 160 KB of a CU (one workgroup with more steps of
    // loads in flight: 28 % slower for fp8 at 2048 x 8192 x 8192); where the
    // activations are small, two steps of them are in flight.
    constexpr int AST = MF * NP >= 8 || FMT == FMT_FP8 ? 2 : 3;
    constexpr uint32_t XB = NP * CH * 16, WO = AST * XB, LDS = WO + 8 * W::BYTES;
    constexpr int EP = MF % 4 == 0 ? 4 : MF % 3 == 0 ? 3 : MF;   // row blocks of an epilogue pass
    constexpr uint32_t OS = EP * 16 * LDO * sizeof(float);
    __shared__ __align__(16) char smem[LDS > OS ? LDS : OS];
    __shared__ int rx[BM];
    const LinearArgs &a = p.a;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int li = lane & 15, lg = lane >> 4;
    const int oc = GATED ? a.O / 2 : a.O;

    // Workgroups are dealt to the 8 XCDs in turn.
    int mt, nt;
    RowTile t;
    if (RAGGED) {
        // A row tile's columns together on one XCD (they share its x), tiles
        // dealt out one by one: the empty ones at the list's end, of unknown
        // number, must not leave one XCD without work.
        const int xcd = blockIdx.x % 8, in = blockIdx.x / 8;
        mt = in / p.ntn * 8 + xcd;
        nt = in % p.ntn;
        if (mt >= p.ntm) return;
        t = p.tiles[mt];
        t.expert = __builtin_amdgcn_readfirstlane(t.expert);
        if (t.n <= 0) return;
    } else {
        // Consecutive tiles to one XCD, a column block's rows together (they
        // share its weights).
        const int nb = gridDim.x, q8 = nb / 8, r8 = nb % 8;
        const int xcd = blockIdx.x % 8, in = blockIdx.x / 8;
        const int b = xcd * q8 + min(xcd, r8) + in;
        nt = b / p.ntm;
        mt = b % p.ntm;
        t = RowTile{0, mt * BM, min(BM, a.R - mt * BM), 0};
    }

    // row exponents; a bad row index is marked and reads row 0
    if (tid < BM) {
        int e = 0;
        if (tid < t.n) {
            int r = t.row0 + tid;
            if (a.rows) r = a.rows[r];
            e = r < 0 || r >= a.T ? BAD_ROW : p.rexp[r];
        }
        rx[tid] = e;
    }

    // activation chunks of this thread: row c / 8, swizzled chunk c % 8
    uint32_t aoff[PT];
#pragma unroll
    for (int i = 0; i < PT; i++) {
        const int c = tid + 256 * i;
        const int row = c >> 3;
        int r = t.row0 + (row < t.n ? row : 0);
        if (a.rows) {
            r = a.rows[r];
            r = r < 0 || r >= a.T ? 0 : r;
        }
        aoff[i] = ((uint32_t)r * (uint32_t)p.ldp + ((c & 7) ^ swizzle(row)) * 8) * 2;
    }

    const uint32_t rb = FMT == FMT_I4G ? (uint32_t)a.I / 2 : (uint32_t)a.I;
    const uint8_t *const wbase = a.w + (size_t)t.expert * a.w_stride;
    const float *const sbase = a.scales + (size_t)t.expert * a.s_stride;
    constexpr int CW = GATED ? 32 : 64;                  // columns of y per wave
    W w;
    w.init(a, rb, lane, [&](int i) {                     // block i / 16 of the wave's rows
        const int n = i >> 4;
        const int c = nt * (4 * CW) + wave * CW + (GATED ? n & 1 : n) * 16 + (i & 15);
        return (c < oc ? c : oc - 1) + (GATED && n >= 2 ? oc : 0);
    });

    f32x4v acc[MF][4];
#pragma unroll
    for (int m = 0; m < MF; m++)
#pragma unroll
        for (int n = 0; n < 4; n++) acc[m][n] = f32x4v{0.0f, 0.0f, 0.0f, 0.0f};

    // row blocks to multiply and activation loads that hold rows: all of them
    // in a dense product, the tile's own in a grouped one
    const int mf = RAGGED ? __builtin_amdgcn_readfirstlane((t.n + 15) / 16) : MF;
    const int na = RAGGED ? __builtin_amdgcn_readfirstlane((t.n + 31) / 32) : PT;
    const uint32_t lds0 = __builtin_amdgcn_readfirstlane(
        (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char *)smem);
    const int steps = p.Ip / TK;

    // Loads of a step past the last repeat it.
    auto load_x = [&](int s, int stage) {
        const int k0 = min(s, steps - 1) * TK;
#pragma unroll
        for (int q = 0; q < NP; q++)
#pragma unroll
            for (int i = 0; i < PT; i++)
                if (!RAGGED || i < na)
                    load_lds16((q ? p.lo : p.hi) + k0, aoff[i],
                               lds0 + stage * XB + (q * CH + wave * 64 + 256 * i) * 16);
    };
    auto load_w = [&](int st) {
        w.load(p, wbase, sbase, rb, st, lds0 + WO + ((st & 1) * 4 + wave) * W::BYTES, lane);
    };

    __syncthreads();                                     // rx; earlier loads are done
    load_x(0, 0);
    load_w(0);
    if (AST == 3) load_x(1, 1);
    int stage = 0;
    for (int s = 0; s < steps; s++) {
        // This step's data is there, and the stages that the last one read are
        // free.  Later loads may be on their way: one step of x (AST == 3), and
        // in a weight stage's second step the next one.
        const int half = s % W::WS;
        const int later = (AST == 3 ? na : 0) + (half ? 8 : 0);
        switch (later) {
        case 0: wait_loads<0>(); break;
        case 1: wait_loads<NP>(); break;
        case 2: wait_loads<2 * NP>(); break;
        case 3: wait_loads<3 * NP>(); break;
        case 8: wait_loads<W::LOADS>(); break;
        case 9: wait_loads<NP + W::LOADS>(); break;
        case 10: wait_loads<2 * NP + W::LOADS>(); break;
        default: wait_loads<3 * NP + W::LOADS>(); break;
        }
        // (fp8's next weights are due a step before the x asked for here)
        if (W::WS == 1) load_w(s + 1);
        load_x(s + AST - 1, stage == 0 ? AST - 1 : stage - 1);
        if (W::WS == 2 && half == 0) load_w(s / 2 + 1);
        const char *const sm = smem + stage * XB;
        f16x8 bv[4][2];
        float sc[4][NS];
        W::unpack(smem + WO + (((s / W::WS) & 1) * 4 + wave) * W::BYTES, half, lane, bv, sc);
        multiply_step<NP, MF, 4, FG, RAGGED>(acc, bv, sc, sm, lane, mf);
        stage = stage == AST - 1 ? 0 : stage + 1;
    }
    // loads past the last step still write LDS
    wait_loads<0>();

    // Epilogue, EP row blocks at a time through LDS: whole rows are stored.
    float *os = reinterpret_cast<float *>(smem);
    constexpr int YC = 4 * CW;                           // columns of y
#pragma unroll
    for (int m0 = 0; m0 < MF; m0 += EP) {
        if (m0 * 16 >= t.n) break;                       // uniform over the workgroup
        if (m0 > 0) __syncthreads();
#pragma unroll
        for (int m = m0; m < m0 + EP; m++)
#pragma unroll
            for (int n = 0; n < 4; n++)
#pragma unroll
                for (int r = 0; r < 4; r++)
                    os[((m - m0) * 16 + 4 * lg + r) * LDO + wave * 64 + n * 16 + li] =
                        acc[m][n][r];
        __syncthreads();
        finish<XT, 4>(a, t.expert, tid, 256, min(t.n - m0 * 16, EP * 16) * YC,
                      [&](int i, int &row, int &col, float &v, float &up) {
                          const int r = i / YC, c = i % YC;
                          const int e = rx[m0 * 16 + r];
                          const float *o = os + r * LDO + (GATED ? (c / 32) * 64 + c % 32 : c);
                          row = t.row0 + m0 * 16 + r;
                          col = nt * YC + c;
                          v = ldexpf(o[0], e);
                          up = GATED ? ldexpf(o[32], e) : 0.0f;
                          if (e == BAD_ROW) v = up = __builtin_nanf("");
                      });
    }
}

// All but this wave's last n loads have arrived.
template <int N>
__device__ __forceinline__ void wait_own_loads()
{
    asm volatile("s_waitcnt vmcnt(%0)" :: "i"(N) : "memory");
}

// Narrow kernel: the tile kernel's arithmetic for products too small to fill
// the GPU with its tiles.  A workgroup makes up to 16 MB rows of y x 16 NB
// rows of W; its KW waves take the K steps in turn, each with stages of LDS of
// its own, so the K loop needs no barrier, and their sums are joined through
// LDS in a fixed order.  Bound by the loads in flight, which LDS limits: 64 x
// 6144 x 12288 bf16 31 us, 40 MB of weights; the tile kernel's 48 workgroups
// take 89 us.
template <int FMT, typename XT, int NP, int MB, bool GATED, int FG, bool RAGGED, int KW>
__global__ __launch_bounds__(KW * 64, (KW + 3) / 4) void linear_narrow(TileArgs p)
{
    typedef Weights<FMT, FG, 64> W;
    constexpr int NB = 4, NS = TK / FG;
    constexpr int AL = MB * 2;                           // loads of x per plane and step
    constexpr int CH = MB * 16 * 8;                      // 16-byte chunks of a plane
    constexpr uint32_t XB = NP * CH * 16, WO = 2 * XB, OWN = WO + 2 * W::BYTES;   // two stages
    constexpr int LDR = NB * 16 + 4;
    constexpr uint32_t RED = KW * MB * 16 * LDR * 4;
    __shared__ __align__(16) char smem[KW * OWN > RED ? KW * OWN : RED];
    const LinearArgs &a = p.a;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int li = lane & 15, lg = lane >> 4;
    const int oc = GATED ? a.O / 2 : a.O;
    constexpr int YC = GATED ? NB * 8 : NB * 16;         // columns of y
    const int nt = (int)(blockIdx.x % p.ntn), mt = (int)(blockIdx.x / p.ntn);
    RowTile t;
    if (p.tiles) t = p.tiles[mt];
    else t = RowTile{0, mt * (16 * MB), min(16 * MB, a.R - mt * (16 * MB)), 0};
    t.n = __builtin_amdgcn_readfirstlane(t.n);
    t.expert = __builtin_amdgcn_readfirstlane(t.expert);
    if (t.n <= 0) return;                                // uniform over the workgroup

    uint32_t aoff[AL];                                   // lane: row c / 8, chunk c % 8
#pragma unroll
    for (int i = 0; i < AL; i++) {
        const int c = lane + 64 * i;
        const int row = c >> 3;
        int r = t.row0 + (row < t.n ? row : 0);
        if (a.rows) {
            r = a.rows[r];
            r = r < 0 || r >= a.T ? 0 : r;
        }
        aoff[i] = ((uint32_t)r * (uint32_t)p.ldp + ((c & 7) ^ swizzle(row & 15)) * 8) * 2;
    }
    const uint32_t rb = FMT == FMT_I4G ? (uint32_t)a.I / 2 : (uint32_t)a.I;
    const uint8_t *const wbase = a.w + (size_t)t.expert * a.w_stride;
    const float *const sbase = a.scales + (size_t)t.expert * a.s_stride;
    W w;
    w.init(a, rb, lane, [&](int i) {
        const int n = i >> 4;
        const int half = GATED ? n / (NB / 2) : 0;
        const int c = nt * YC + (GATED ? n % (NB / 2) : n) * 16 + (i & 15);
        return (c < oc ? c : oc - 1) + half * oc;
    });
    const int mf = __builtin_amdgcn_readfirstlane((t.n + 15) / 16);
    const uint32_t lds0 = __builtin_amdgcn_readfirstlane(
        (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char *)smem) + wave * OWN;
    const char *const own = smem + wave * OWN;
    const int steps = p.Ip / TK;
    const int stages = (steps + W::WS - 1) / W::WS;      // of weights

    // The wave's i-th step is step i % WS of weight stage wave + KW (i / WS);
    // loads past the last repeat it.
    auto load_x = [&](int i, int stage) {
        const int s = (wave + KW * (i / W::WS)) * W::WS + i % W::WS;
        const int k0 = min(s, steps - 1) * TK;
#pragma unroll
        for (int q = 0; q < NP; q++)
#pragma unroll
            for (int j = 0; j < AL; j++)
                load_lds16((q ? p.lo : p.hi) + k0, aoff[j],
                           lds0 + stage * XB + q * (CH * 16) + 1024 * j);
    };
    auto load_w = [&](int i) {                           // the wave's i-th weight stage
        const int st = min(wave + KW * i, stages - 1);
        w.load(p, wbase, sbase, rb, st, lds0 + WO + (i & 1) * W::BYTES, lane);
    };

    f32x4v acc[MB][NB];
#pragma unroll
    for (int m = 0; m < MB; m++)
#pragma unroll
        for (int n = 0; n < NB; n++) acc[m][n] = f32x4v{0.0f, 0.0f, 0.0f, 0.0f};

    __builtin_amdgcn_s_waitcnt(QG_WAIT_VM0);             // earlier loads are done
    load_x(0, 0);
    load_w(0);
    // a stage behind the last step of a last half stage has zero steps
    const int mine = wave < stages ? (stages - 1 - wave) / KW + 1 : 0;
    const int last = (stages - 1) % KW == wave ? steps - (stages - 1) * W::WS : W::WS;
    const int count = mine ? (mine - 1) * W::WS + last : 0;
    int stage = 0;
    for (int i = 0; i < count; i++) {
        // as the tile kernel's
        const int half = i % W::WS;
        if (half) wait_own_loads<W::LOADS>();
        else wait_own_loads<0>();
        if (W::WS == 1) load_w(i + 1);
        load_x(i + 1, stage ^ 1);
        if (W::WS == 2 && half == 0) load_w(i / 2 + 1);
        f16x8 bv[NB][2];
        float sc[NB][NS];
        W::unpack(own + WO + ((i / W::WS) & 1) * W::BYTES, half, lane, bv, sc);
        multiply_step<NP, MB, NB, FG, RAGGED>(acc, bv, sc, own + stage * XB, lane, mf);
        stage ^= 1;
    }
    wait_own_loads<0>();                                 // loads past the last step
    __syncthreads();

    float (*const red)[MB * 16][LDR] = reinterpret_cast<float (*)[MB * 16][LDR]>(smem);
#pragma unroll
    for (int m = 0; m < MB; m++)
#pragma unroll
        for (int n = 0; n < NB; n++)
#pragma unroll
            for (int r = 0; r < 4; r++)
                red[wave][m * 16 + 4 * lg + r][n * 16 + li] = acc[m][n][r];
    __syncthreads();
    finish<XT, 4>(a, t.expert, tid, KW * 64, t.n * YC,
                  [&](int i, int &row, int &col, float &v, float &up) {
                      const int r = i / YC, c = i % YC;
                      row = t.row0 + r;
                      col = nt * YC + c;
                      const int xr = a.rows ? a.rows[row] : row;
                      const int e = xr < 0 || xr >= a.T ? BAD_ROW : p.rexp[xr];
                      v = up = 0.0f;
#pragma unroll
                      for (int w = 0; w < KW; w++) {
                          v += red[w][r][c];
                          if (GATED) up += red[w][r][c + YC];
                      }
                      v = ldexpf(v, e);
                      up = ldexpf(up, e);
                      if (e == BAD_ROW) v = up = __builtin_nanf("");
                  });
}

#define QG_RUN1(FG, G, R)                                                                   \
    hipLaunchKernelGGL((linear_tile<FMT, XT, NP, MF, G, FG, R>), dim3(grid), dim3(256), 0, st, p)
#define QG_RUN(FG)                                                                          \
    do {                                                                                    \
        if constexpr (FMT == FMT_I4G) {                  /* grouped: int4, largest tiles */ \
            if (p.tiles) {                                                                  \
                if constexpr (MF == (NP == 1 ? 8 : 4)) {                                    \
                    if (p.a.gated) QG_RUN1(FG, true, true);                                 \
                    else QG_RUN1(FG, false, true);                                          \
                }                                                                           \
                break;                                                                      \
            }                                                                               \
        }                                                                                   \
        if (p.a.gated) QG_RUN1(FG, true, false);                                            \
        else QG_RUN1(FG, false, false);                                                     \
    } while (0)

template <int FMT, typename XT, int MF>
hipError_t run_tile(const TileArgs &p, unsigned grid, hipStream_t st)
{
    constexpr int NP = sizeof(typename XT::raw) == 4 ? 2 : 1;
    if constexpr (FMT == FMT_FP8) {
        QG_RUN(64);
    } else {
        if (p.a.gs % 64 == 0) QG_RUN(64);
        else QG_RUN(32);
    }
    return hipGetLastError();
}

// Waves of a narrow workgroup with planes x row blocks of packed x: 8 where
// their stages fit the 160 KB of LDS, else 6.
constexpr int narrow_waves(int planes) { return planes <= 2 ? 8 : 6; }

template <int FMT, typename XT, int MB>
hipError_t run_narrow(const TileArgs &p, unsigned grid, hipStream_t st)
{
    constexpr int NP = sizeof(typename XT::raw) == 4 ? 2 : 1;
    constexpr int KW = narrow_waves(NP * MB);
#define QG_RUN2(FG, G, R)                                                                   \
    hipLaunchKernelGGL((linear_narrow<FMT, XT, NP, MB, G, FG, R, KW>), dim3(grid),     \
                       dim3(KW * 64), 0, st, p)
#define QG_RUN3(FG)                                                                         \
    do {                                                                                    \
        if constexpr (FMT == FMT_I4G) {                  /* grouped: int4 */                \
            if (p.tiles) {                                                                  \
                if (p.a.gated) QG_RUN2(FG, true, true);                                     \
                else QG_RUN2(FG, false, true);                                              \
                break;                                                                      \
            }                                                                               \
        }                                                                                   \
        if (p.a.gated) QG_RUN2(FG, true, false);                                            \
        else QG_RUN2(FG, false, false);                                                     \
    } while (0)
    if constexpr (FMT == FMT_FP8) {
        QG_RUN3(64);
    } else {
        if (p.a.gs % 64 == 0) QG_RUN3(64);
        else QG_RUN3(32);
    }
#undef QG_RUN2
#undef QG_RUN3
    return hipGetLastError();
}

int padded(int I) { return (I + TK - 1) / TK * TK; }
// Row stride of the packed planes: an odd count of 256 bytes, so that a K
// step's pieces of a tile's rows lie in all of the 16 L2 channels.
int plane_stride(int I) { return ((padded(I) + 127) / 128 | 1) * 128; }

}  // namespace

size_t tile_workspace(int T, int I, int dtype)
{
    return align256((size_t)T * sizeof(int)) +
           align256((size_t)T * plane_stride(I) * 2) * (dtype == QGEMV_BF16 ? 1 : 2);
}

int tile_rows(int I)
{
    const size_t n = ((1ull << 32) - 1) / ((size_t)plane_stride(I) * 2) / 128 * 128;
    return n > (1 << 24) ? 1 << 24 : n < 128 ? 128 : (int)n;
}

bool planes_fit(int T, int I) { return (size_t)T * plane_stride(I) * 2 < (1ull << 32); }

bool tile_fits(WeightFormat fmt, const LinearArgs &a)
{
    const size_t rb = fmt == FMT_I4G ? (size_t)a.I / 2 : (size_t)a.I;
    return a.I % 32 == 0 && (fmt == FMT_FP8 || a.gs % 32 == 0) && ((uintptr_t)a.w & 15) == 0 &&
           (!a.offsets || a.w_stride % 16 == 0) && rb * a.O < (1ull << 32) &&
           (size_t)a.ng * a.O * 4 < (1ull << 32) && planes_fit(a.T, a.I);
}

// Workgroups of a launch, and tiles across y.
static long long tile_grid(const LinearArgs &a, bool narrow, int ntm, int &ntn)
{
    const int tn = narrow ? 64 : TN;
    const int cols = a.gated ? tn / 2 : tn, oc = a.gated ? a.O / 2 : a.O;
    ntn = (oc + cols - 1) / cols;
    // the grouped tile kernel deals row tiles by eights
    return (long long)(a.offsets && !narrow ? (ntm + 7) / 8 * 8 : ntm) * ntn;
}

long long tile_items(const LinearArgs &a, bool narrow, int bm, int ntm)
{
    const int planes = (a.dtype == QGEMV_BF16 ? 1 : 2) * bm / 16;
    int ntn;
    return tile_grid(a, narrow, ntm, ntn) * (narrow ? narrow_waves(planes) * 64 : 256);
}

hipError_t launch_tile(WeightFormat fmt, const LinearArgs &a, bool narrow, int bm,
                       const RowTile *tiles, int ntm, void *ws, hipStream_t st)
{
    TileArgs p{};
    p.a = a;
    p.Ip = padded(a.I);
    p.ldp = plane_stride(a.I);
    p.g32 = (uint32_t)a.gs / 32;
    p.gmagic = 0xFFFFFFFFu / p.g32;
    char *at = static_cast<char *>(ws);
    int *rexp = reinterpret_cast<int *>(at);
    at += align256((size_t)a.T * sizeof(int));
    _Float16 *hi = reinterpret_cast<_Float16 *>(at);
    at += align256((size_t)a.T * p.ldp * 2);
    _Float16 *lo = a.dtype == QGEMV_BF16 ? nullptr : reinterpret_cast<_Float16 *>(at);
    p.hi = hi;
    p.lo = lo;
    p.rexp = rexp;
    p.tiles = tiles;
    p.ntm = ntm;
    const long long grid = tile_grid(a, narrow, ntm, p.ntn);
    const hipError_t e = a.dtype == QGEMV_BF16 ? pack<BF16>(fmt, a, p.Ip, p.ldp, hi, lo, rexp, st)
                                               : pack<F32>(fmt, a, p.Ip, p.ldp, hi, lo, rexp, st);
    if (e != hipSuccess) return e;
#define QG_TILE(XT, MF)                                                                     \
    (fmt == FMT_I4G ? run_tile<FMT_I4G, XT, MF>(p, (unsigned)grid, st)                      \
                    : run_tile<FMT_FP8, XT, MF>(p, (unsigned)grid, st))
#define QG_NARROW(XT, MB)                                                                   \
    (fmt == FMT_I4G ? run_narrow<FMT_I4G, XT, MB>(p, (unsigned)grid, st)                    \
                    : run_narrow<FMT_FP8, XT, MB>(p, (unsigned)grid, st))
    if (a.dtype == QGEMV_F32) {
        if (narrow) return QG_NARROW(F32, 2);
        return bm == 64 ? QG_TILE(F32, 4) : QG_TILE(F32, 2);
    }
    if (narrow) return bm == 64 ? QG_NARROW(BF16, 4) : QG_NARROW(BF16, 2);
    return bm == 128 ? QG_TILE(BF16, 8) : bm == 96 ? QG_TILE(BF16, 6) : QG_TILE(BF16, 4);
#undef QG_NARROW
#undef QG_TILE
}

}  // namespace qg
