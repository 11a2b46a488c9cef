// route.hip -- routed slots sorted by expert, and the experts' rows returned
// to their tokens.
#include "qg_device.h"
#include "qg_linear.h"

namespace qg {

namespace {

// ---------------------------------------------------------------------------
// Slots sorted by expert: a stable counting sort of N = T * K ids below E.
//
// Row of slot i = (slots of smaller experts) + (earlier slots of its expert).
// The slots are cut into blocks of `chunk`, a block into 8 waves of
// consecutive slots; each wave counts its experts in its own LDS histogram,
// the histograms are turned into each wave's first row per expert, and a
// second pass hands out the rows in slot order: lanes of equal id find each
// other by ballots over the id's bits.  Counts are integers, so the LDS
// atomics' order does not show in the result.  Several blocks need the
// earlier blocks' counts first: a histogram kernel writes them, and every
// block sums what it needs (at most 256 blocks).  Bound by latency: reading
// the ids twice from the caches, one launch for up to 2048 slots, else two.
// ---------------------------------------------------------------------------
constexpr int GT = 512;                  // threads of a block
constexpr int GW = GT / 64;
constexpr int GROUP_CHUNK = 2048;
constexpr int GROUP_BLOCKS = 256;

int group_chunk(long long n)
{
    long long c = (n + GROUP_BLOCKS - 1) / GROUP_BLOCKS;
    c = (c + GT - 1) / GT * GT;          // whole rounds of every wave
    return (int)(c < GROUP_CHUNK ? GROUP_CHUNK : c);
}

__global__ __launch_bounds__(GT) void group_count(const int32_t *__restrict__ ids, int n, int E,
                                                  int chunk, int *__restrict__ counts)
{
    extern __shared__ int hist[];
    for (int e = threadIdx.x; e < E; e += GT) hist[e] = 0;
    __syncthreads();
    const int first = blockIdx.x * chunk, last = min(n, first + chunk);
    for (int i = first + (int)threadIdx.x; i < last; i += GT) {
        const int id = ids[i];
        if (id >= 0 && id < E) atomicAdd(&hist[id], 1);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += GT) counts[(size_t)blockIdx.x * E + e] = hist[e];
}

__global__ __launch_bounds__(GT) void group_rows(const int32_t *__restrict__ ids, int n, int K,
                                                 int E, int chunk,
                                                 const int *__restrict__ counts, int nblk,
                                                 int32_t *__restrict__ offsets,
                                                 int32_t *__restrict__ tokens,
                                                 int32_t *__restrict__ pos)
{
    extern __shared__ int hist[];        // [GW][E], then all slots, earlier blocks' slots
    __shared__ int wsum[GW];
    __shared__ int total_s;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, blk = blockIdx.x;
    for (int i = tid; i < GW * E; i += GT) hist[i] = 0;
    __syncthreads();
    const int per = chunk / GW;          // a multiple of 64
    const int first = blk * chunk + wave * per;
    const int last = min(n, first + per);
    int *mine = hist + wave * E;
    for (int i = first + lane; i < last; i += 64) {
        const int id = ids[i];
        if (id >= 0 && id < E) atomicAdd(&mine[id], 1);
    }
    __syncthreads();

    // all slots of each expert and those of the earlier blocks: waves take
    // blocks in turn, lanes experts
    int *const all_s = hist + GW * E, *const before_s = all_s + E;
    for (int e = tid; e < E; e += GT) {
        int n0 = 0;
        if (nblk == 1)
            for (int w = 0; w < GW; w++) n0 += hist[w * E + e];
        all_s[e] = n0;
        before_s[e] = 0;
    }
    if (nblk > 1) {
        __syncthreads();
        for (int e = lane; e < E; e += 64) {
            int sum = 0, early = 0;
#pragma unroll 8
            for (int b = wave; b < nblk; b += GW) {
                const int c = counts[(size_t)b * E + e];
                sum += c;
                early += b < blk ? c : 0;
            }
            atomicAdd(&all_s[e], sum);
            atomicAdd(&before_s[e], early);
        }
    }
    __syncthreads();

    // thread: experts 2 tid and 2 tid + 1 (E <= 1024)
    int before[2] = {0, 0}, all[2] = {0, 0};
#pragma unroll
    for (int j = 0; j < 2; j++) {
        const int e = 2 * tid + j;
        if (e >= E) continue;
        all[j] = all_s[e];
        before[j] = before_s[e];
    }
    int incl = all[0] + all[1];
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const int v = __shfl_up(incl, d);
        if (lane >= d) incl += v;
    }
    if (lane == 63) wsum[wave] = incl;
    __syncthreads();
    int base = incl - all[0] - all[1];
    for (int w = 0; w < wave; w++) base += wsum[w];
    if (tid == GT - 1) total_s = base + all[0] + all[1];
#pragma unroll
    for (int j = 0; j < 2; j++) {
        const int e = 2 * tid + j;
        if (e >= E) continue;
        if (blk == 0) {
            offsets[e] = base;
            if (e == E - 1) offsets[E] = base + all[j];
        }
        int run = base + before[j];
        for (int w = 0; w < GW; w++) {
            const int c = hist[w * E + e];
            hist[w * E + e] = run;
            run += c;
        }
        base += all[j];
    }
    __syncthreads();

    int bits = 1;
    while ((1 << bits) < E) bits++;
    for (int i0 = first; i0 < last; i0 += 64) {
        const int i = i0 + lane;
        const int id = i < last ? ids[i] : -1;
        const bool ok = id >= 0 && id < E;
        unsigned long long same = __ballot(ok);
        for (int b = 0; b < bits; b++) {
            const unsigned long long set = __ballot((id >> b) & 1);
            same &= ((id >> b) & 1) ? set : ~set;
        }
        const unsigned long long below = same & ((1ull << lane) - 1);
        int row = -1;
        if (ok) row = mine[id] + __popcll(below);
        __builtin_amdgcn_wave_barrier();
        // only this wave touches its histogram, and a wave's LDS operations
        // complete in order
        if (ok && below == 0) mine[id] = row + __popcll(same);
        __builtin_amdgcn_wave_barrier();
        if (i < last) pos[i] = row;
        if (ok) tokens[row] = i / K;
    }
    // rows behind the last valid slot
    const int total = total_s;
    for (int i = first + lane; i < last; i += 64)
        if (i >= total) tokens[i] = -1;
}

// ---------------------------------------------------------------------------
// y[t] = sum_k gates[t][k] h[pos[t][k]] (+ residual[t]).
//
// One pass: each row of h is read once and summed in registers in f32, k
// ascending.  Bound by HBM: T K O elements in, T O out.  A thread owns VEC
// consecutive columns of one token (16 bytes where everything is aligned for
// it), a wave one token, so positions and gates are scalar; the loads of
// eight experts are in flight together.
// ---------------------------------------------------------------------------
template <typename XT, int VEC>
__global__ __launch_bounds__(256) void combine(const typename XT::raw *__restrict__ h,
                                               long long ldh, int R,
                                               const int32_t *__restrict__ pos,
                                               const float *__restrict__ gates, int T, int K,
                                               int O, const typename XT::raw *residual,
                                               long long ldr, typename XT::raw *y, long long ldy,
                                               int ncb)
{
    typedef typename XT::raw raw;
    typedef raw vec __attribute__((ext_vector_type(VEC)));
    const int tb = (int)(blockIdx.x / ncb), cb = (int)(blockIdx.x % ncb);
    const int t = __builtin_amdgcn_readfirstlane(tb * (int)blockDim.y + (int)threadIdx.y);
    const int c = (cb * (int)blockDim.x + (int)threadIdx.x) * VEC;
    if (t >= T || c >= O) return;
    const bool whole = c + VEC <= O;
    float acc[VEC];
#pragma unroll
    for (int j = 0; j < VEC; j++) acc[j] = 0.0f;
    const int32_t *pt = pos + (size_t)t * K;
    const float *gt = gates + (size_t)t * K;
    bool bad = false;
    for (int k0 = 0; k0 < K; k0 += 8) {
        vec v[8];
        float g[8];
#pragma unroll
        for (int i = 0; i < 8; i++) {
            v[i] = vec(0);
            g[i] = 0.0f;
            if (k0 + i >= K) continue;
            const int r = pt[k0 + i];
            if (r < 0 || r >= R) {
                bad = true;
                continue;
            }
            g[i] = gt[k0 + i];
            const raw *src = h + (size_t)r * ldh + c;
            if (whole) v[i] = *reinterpret_cast<const vec *>(src);
            else
#pragma unroll
                for (int j = 0; j < VEC; j++)
                    if (c + j < O) v[i][j] = src[j];
        }
#pragma unroll
        for (int i = 0; i < 8; i++)
            if (k0 + i < K)
#pragma unroll
                for (int j = 0; j < VEC; j++) acc[j] = fmaf(g[i], XT::get(v[i][j]), acc[j]);
    }
    const raw *rs = residual ? residual + (size_t)t * ldr + c : nullptr;
    raw *dst = y + (size_t)t * ldy + c;
    vec out, rv = vec(0);
    if (rs) {
        if (whole) rv = *reinterpret_cast<const vec *>(rs);
        else
#pragma unroll
            for (int j = 0; j < VEC; j++)
                if (c + j < O) rv[j] = rs[j];
    }
#pragma unroll
    for (int j = 0; j < VEC; j++)
        out[j] = XT::put(bad ? __builtin_nanf("") : acc[j] + XT::get(rv[j]));
    if (whole) *reinterpret_cast<vec *>(dst) = out;
    else
#pragma unroll
        for (int j = 0; j < VEC; j++)
            if (c + j < O) dst[j] = out[j];
}

template <typename XT, int VEC>
hipError_t run_combine(const void *h, long long ldh, int R, const int32_t *pos,
                       const float *gates, int T, int K, int O, const void *residual,
                       long long ldr, void *y, long long ldy, hipStream_t st)
{
    typedef typename XT::raw raw;
    const int nch = (O + VEC - 1) / VEC;
    const int bx = nch > 192 ? 256 : nch > 64 ? 128 : 64;
    const int by = 256 / bx;
    const int ncb = (nch + bx - 1) / bx;
    // as many tokens per launch as its work items allow
    const long long most = MAX_ITEMS / bx / ncb * by;
    for (long long t = 0; t < T; t += most) {
        const int n = (int)(T - t < most ? T - t : most);
        hipLaunchKernelGGL((combine<XT, VEC>), dim3((unsigned)((n + by - 1) / by * ncb)),
                           dim3(bx, by), 0, st, static_cast<const raw *>(h), ldh, R, pos + t * K,
                           gates + t * K, n, K, O,
                           residual ? static_cast<const raw *>(residual) + t * ldr : nullptr, ldr,
                           static_cast<raw *>(y) + t * ldy, ldy, ncb);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace

size_t moe_group_workspace(int T, int K, int E)
{
    const long long n = (long long)T * K;
    const int chunk = group_chunk(n);
    const long long nblk = (n + chunk - 1) / chunk;
    return nblk > 1 ? (size_t)nblk * E * sizeof(int) : 0;
}

hipError_t launch_moe_group(const int32_t *ids, int T, int K, int E, int32_t *offsets,
                            int32_t *tokens, int32_t *pos, void *ws, hipStream_t st)
{
    const int n = T * K;
    const int chunk = group_chunk(n);
    int nblk = (n + chunk - 1) / chunk;
    if (nblk < 1) nblk = 1;                              // T = 0: the offsets
    int *counts = static_cast<int *>(ws);
    if (nblk > 1) {
        hipLaunchKernelGGL(group_count, dim3(nblk), dim3(GT), E * sizeof(int), st, ids, n, E,
                           chunk, counts);
        hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL(group_rows, dim3(nblk), dim3(GT), (GW + 2) * E * sizeof(int), st, ids, n, K, E,
                       chunk, counts, nblk, offsets, tokens, pos);
    return hipGetLastError();
}

hipError_t launch_moe_combine(const void *h, long long ldh, int R, const int32_t *pos,
                              const float *gates, int T, int K, int O, const void *residual,
                              long long ldr, void *y, long long ldy, int dtype, hipStream_t st)
{
    // 16 bytes per thread where every row starts on 16 bytes, else one element
    const int el = dtype == QGEMV_BF16 ? 2 : 4;
    const uintptr_t any = (uintptr_t)h | (uintptr_t)y | (uintptr_t)residual |
                          (uintptr_t)(ldh * el) | (uintptr_t)(ldy * el) |
                          (uintptr_t)(residual ? ldr * el : 0);
    const bool wide = (any & 15) == 0;
    if (dtype == QGEMV_BF16)
        return wide ? run_combine<BF16, 8>(h, ldh, R, pos, gates, T, K, O, residual, ldr, y, ldy,
                                           st)
                    : run_combine<BF16, 1>(h, ldh, R, pos, gates, T, K, O, residual, ldr, y, ldy,
                                           st);
    return wide ? run_combine<F32, 4>(h, ldh, R, pos, gates, T, K, O, residual, ldr, y, ldy, st)
                : run_combine<F32, 1>(h, ldh, R, pos, gates, T, K, O, residual, ldr, y, ldy, st);
}

}  // namespace qg
