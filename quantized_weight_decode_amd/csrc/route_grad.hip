// route_grad.hip -- token rows put in expert order, the gradient of that, and
// the gradient of the experts' gate-weighted return.
#include "qg_device.h"
#include "qg_launch.h"
#include "qg_matmul.h"

namespace qg {

namespace {

// A thread's VEC consecutive columns of a row: one load or store where all of
// them exist, else element by element.
template <typename XT, int VEC>
struct Piece {
    typedef typename XT::raw raw;
    typedef raw vec __attribute__((ext_vector_type(VEC)));
    vec v;
    __device__ __forceinline__ void load(const raw *p, int left)
    {
        v = vec(0);
        if (left >= VEC) {
            v = *reinterpret_cast<const vec *>(p);
        } else {
#pragma unroll
            for (int j = 0; j < VEC; j++)
                if (j < left) v[j] = p[j];
        }
    }
    __device__ __forceinline__ void store(raw *p, int left) const
    {
        if (left >= VEC) {
            *reinterpret_cast<vec *>(p) = v;
        } else {
#pragma unroll
            for (int j = 0; j < VEC; j++)
                if (j < left) p[j] = v[j];
        }
    }
    // past the caches
    __device__ __forceinline__ void store_past(raw *p, int left) const
    {
        if (left >= VEC) {
            __builtin_nontemporal_store(v, reinterpret_cast<vec *>(p));
        } else {
#pragma unroll
            for (int j = 0; j < VEC; j++)
                if (j < left) p[j] = v[j];
        }
    }
};

// ---------------------------------------------------------------------------
// y[r] = x[tokens[r]].  A wave has one row, so its index is scalar; rows of index
// -1 are left as they were.  Bound by HBM: R rows written, T read (each token's
// row again for every expert of it, from the caches, which the stores therefore
// pass by: 4096 tokens of 8, 7168 bf16, 150 us with ordinary stores and a piece per
// thread).  A thread has four pieces of the row in flight.
// ---------------------------------------------------------------------------
template <typename XT, int VEC>
__global__ __launch_bounds__(256) void dispatch(const typename XT::raw *__restrict__ x,
                                                long long ldx, int T,
                                                const int32_t *__restrict__ tokens, int R, int I,
                                                typename XT::raw *__restrict__ y, long long ldy,
                                                int ncb)
{
    constexpr int U = 4;
    const int rb = (int)(blockIdx.x / ncb), cb = (int)(blockIdx.x % ncb);
    const int r = __builtin_amdgcn_readfirstlane(rb * (int)blockDim.y + (int)threadIdx.y);
    const int step = (int)blockDim.x * VEC, c = cb * U * step + (int)threadIdx.x * VEC;
    if (r >= R) return;
    const int t = tokens[r];
    if (t == -1) return;
    const bool bad = t < 0 || t >= T;
    Piece<XT, VEC> p[U];
#pragma unroll
    for (int i = 0; i < U; i++)
        p[i].load(x + (long long)(bad ? 0 : t) * ldx + c + i * step, bad ? 0 : I - c - i * step);
#pragma unroll
    for (int i = 0; i < U; i++) {
        if (bad)
#pragma unroll
            for (int j = 0; j < VEC; j++) p[i].v[j] = XT::put(__builtin_nanf(""));
        p[i].store_past(y + (long long)r * ldy + c + i * step, I - c - i * step);
    }
}

// ---------------------------------------------------------------------------
// dx[t] = sum over k of dy[pos[t][k]], f32, k ascending; a slot of index -1 had
// no row and adds nothing.  As the experts' return: one pass, eight rows in
// flight.
// ---------------------------------------------------------------------------
template <typename XT, int VEC>
__global__ __launch_bounds__(256) void dispatch_grad(const typename XT::raw *__restrict__ dy,
                                                     long long lddy, int R,
                                                     const int32_t *__restrict__ pos, int T,
                                                     int K, int I,
                                                     typename XT::raw *__restrict__ dx,
                                                     long long lddx, int ncb)
{
    const int tb = (int)(blockIdx.x / ncb), cb = (int)(blockIdx.x % ncb);
    const int t = __builtin_amdgcn_readfirstlane(tb * (int)blockDim.y + (int)threadIdx.y);
    const int c = (cb * (int)blockDim.x + (int)threadIdx.x) * VEC;
    if (t >= T || c >= I) return;
    const int32_t *const pt = pos + (long long)t * K;
    float acc[VEC];
#pragma unroll
    for (int j = 0; j < VEC; j++) acc[j] = 0.0f;
    bool bad = false;
    for (int k0 = 0; k0 < K; k0 += 8) {
        Piece<XT, VEC> p[8];
#pragma unroll
        for (int i = 0; i < 8; i++) {
            const int r = k0 + i < K ? pt[k0 + i] : -1;
            p[i].load(dy + (long long)(r < 0 || r >= R ? 0 : r) * lddy + c,
                      r < 0 || r >= R ? 0 : I - c);
            bad |= r < -1 || r >= R;
        }
#pragma unroll
        for (int i = 0; i < 8; i++)
#pragma unroll
            for (int j = 0; j < VEC; j++) acc[j] += XT::get(p[i].v[j]);
    }
    Piece<XT, VEC> out;
#pragma unroll
    for (int j = 0; j < VEC; j++) out.v[j] = XT::put(bad ? __builtin_nanf("") : acc[j]);
    out.store(dx + (long long)t * lddx + c, I - c);
}

// ---------------------------------------------------------------------------
// The gradients of y[t] = sum_k gates[t][k] h[pos[t][k]]:
//     dh[r] = (sum of gates[t][k] over k with pos[t][k] = r) dy[t],  t = tokens[r]
//     dgates[t][k] = sum over columns of h[pos[t][k]] dy[t]
// A workgroup has KB slots of token first + t, so dy's row is read once for them, h's
// rows once and dh's are written once: bound by HBM.  A row belongs to the one
// token that tokens names, so no two tokens write it; a slot that names a row
// out of range or of another token gets a NaN and writes none.  Products and
// sums are f32; a thread's columns, then lanes, then waves are summed in a
// fixed order.  4096 tokens of 8, 7168 bf16: 204 us, 4.9 TB/s (1 GB).
// ---------------------------------------------------------------------------
template <typename XT, int VEC, int KB>
__global__ __launch_bounds__(256) void combine_grad(
    const typename XT::raw *__restrict__ dy, long long lddy,
    const typename XT::raw *__restrict__ h, long long ldh, int R,
    const int32_t *__restrict__ tokens, const int32_t *__restrict__ pos,
    const float *__restrict__ gates, int first, int K, int O,
    typename XT::raw *__restrict__ dh, long long lddh, float *__restrict__ dgates, int nkb)
{
    __shared__ float part[4][KB];
    const int t = (int)(blockIdx.x / nkb), k0 = (int)(blockIdx.x % nkb) * KB;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    // lane k has slot k of the token (K <= 64): its row, whether that is the token's
    // own, its gate
    const int32_t *const pt = pos + (long long)t * K;
    const int pk = lane < K ? pt[lane] : -1;
    const bool range = pk >= 0 && pk < R;
    const float gk = lane < K ? gates[(long long)t * K + lane] : 0.0f;
    const bool mine = range && tokens[pk] == first + t;
    const unsigned long long valid = __ballot(range), owned = __ballot(mine);
    int r[KB];
    bool in[KB], own[KB];
    float g[KB], dot[KB];
#pragma unroll
    for (int i = 0; i < KB; i++) {
        const int k = k0 + i < K ? k0 + i : 0;
        in[i] = k0 + i < K && (valid >> k & 1);
        own[i] = in[i] && (owned >> k & 1);
        r[i] = in[i] ? __builtin_amdgcn_readlane(pk, k) : 0;
        dot[i] = 0.0f;
        // a row that several of the token's slots name has all their gates
        g[i] = 0.0f;
        unsigned long long same = __ballot(lane < K && pk == r[i]);
        while (same) {                                   // uniform over the wave
            const int at = __builtin_ctzll(same);
            g[i] += __builtin_bit_cast(
                float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, gk), at));
            same &= same - 1;
        }
    }
    const typename XT::raw *const dyt = dy + (long long)t * lddy;
    for (int c = tid * VEC; c < O; c += 256 * VEC) {
        Piece<XT, VEC> d, p[KB];
        d.load(dyt + c, O - c);
#pragma unroll
        for (int i = 0; i < KB; i++)
            p[i].load(h + (long long)r[i] * ldh + c, in[i] ? O - c : 0);
#pragma unroll
        for (int i = 0; i < KB; i++) {
            Piece<XT, VEC> out;
#pragma unroll
            for (int j = 0; j < VEC; j++) {
                const float v = XT::get(d.v[j]);
                dot[i] = fmaf(XT::get(p[i].v[j]), v, dot[i]);
                out.v[j] = XT::put(g[i] * v);
            }
            if (own[i]) out.store(dh + (long long)r[i] * lddh + c, O - c);
        }
    }
#pragma unroll
    for (int i = 0; i < KB; i++) {
#pragma unroll
        for (int d = 32; d > 0; d /= 2) dot[i] += __shfl_xor(dot[i], d);
        if (lane == 0) part[wave][i] = dot[i];
    }
    __syncthreads();
    if (tid < KB && k0 + tid < K) {
        const bool ok = owned >> (k0 + tid) & 1;
        const float sum = (part[0][tid] + part[1][tid]) + (part[2][tid] + part[3][tid]);
        dgates[(long long)t * K + k0 + tid] = ok ? sum : __builtin_nanf("");
    }
}

// Threads across a row of nch pieces, `each` of them per thread, rows per workgroup,
// workgroups per row.
struct Shape {
    int bx, by, ncb;
};
Shape shape_of(int nch, int each = 1)
{
    const int bx = nch > 192 * each ? 256 : nch > 64 * each ? 128 : 64;
    return {bx, 256 / bx, (nch + bx * each - 1) / (bx * each)};
}

// Slices of n rows whose launches of `items` work items per row hold fewer than
// 2^32 of them: f(first row, rows).
template <typename F>
hipError_t sliced(long long n, long long items, int by, F f)
{
    const long long most = MAX_ITEMS / items / by * by;
    for (long long r = 0; r < n; r += most) {
        f(r, (int)(n - r < most ? n - r : most));
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

bool aligned16(uintptr_t any) { return (any & 15) == 0; }

template <typename XT, int VEC>
hipError_t run_dispatch(const void *x, long long ldx, int T, const int32_t *tokens, int R, int I,
                        void *y, long long ldy, hipStream_t st)
{
    typedef typename XT::raw raw;
    const Shape s = shape_of((I + VEC - 1) / VEC, 4);
    return sliced(R, (long long)s.bx * s.ncb, s.by, [&](long long r, int n) {
        hipLaunchKernelGGL((dispatch<XT, VEC>), dim3((unsigned)((n + s.by - 1) / s.by * s.ncb)),
                           dim3(s.bx, s.by), 0, st, static_cast<const raw *>(x), ldx, T,
                           tokens + r, n, I, static_cast<raw *>(y) + r * ldy, ldy, s.ncb);
    });
}

template <typename XT, int VEC>
hipError_t run_dispatch_grad(const void *dy, long long lddy, int R, const int32_t *pos, int T,
                             int K, int I, void *dx, long long lddx, hipStream_t st)
{
    typedef typename XT::raw raw;
    const Shape s = shape_of((I + VEC - 1) / VEC);
    return sliced(T, (long long)s.bx * s.ncb, s.by, [&](long long t, int n) {
        hipLaunchKernelGGL((dispatch_grad<XT, VEC>),
                           dim3((unsigned)((n + s.by - 1) / s.by * s.ncb)), dim3(s.bx, s.by), 0,
                           st, static_cast<const raw *>(dy), lddy, R, pos + t * K, n, K, I,
                           static_cast<raw *>(dx) + t * lddx, lddx, s.ncb);
    });
}

}  // namespace

hipError_t launch_moe_dispatch(const void *x, long long ldx, int T, const int32_t *tokens, int R,
                               int I, void *y, long long ldy, int dtype, hipStream_t st)
{
    const int el = dtype == QGEMV_BF16 ? 2 : 4;
    const bool wide = aligned16((uintptr_t)x | (uintptr_t)y | (uintptr_t)(ldx * el) |
                                (uintptr_t)(ldy * el));
    if (dtype == QGEMV_BF16)
        return wide ? run_dispatch<BF16, 8>(x, ldx, T, tokens, R, I, y, ldy, st)
                    : run_dispatch<BF16, 1>(x, ldx, T, tokens, R, I, y, ldy, st);
    return wide ? run_dispatch<F32, 4>(x, ldx, T, tokens, R, I, y, ldy, st)
                : run_dispatch<F32, 1>(x, ldx, T, tokens, R, I, y, ldy, st);
}

hipError_t launch_moe_dispatch_grad(const void *dy, long long lddy, int R, const int32_t *pos,
                                    int T, int K, int I, void *dx, long long lddx, int dtype,
                                    hipStream_t st)
{
    const int el = dtype == QGEMV_BF16 ? 2 : 4;
    const bool wide = aligned16((uintptr_t)dy | (uintptr_t)dx | (uintptr_t)(lddy * el) |
                                (uintptr_t)(lddx * el));
    if (dtype == QGEMV_BF16)
        return wide ? run_dispatch_grad<BF16, 8>(dy, lddy, R, pos, T, K, I, dx, lddx, st)
                    : run_dispatch_grad<BF16, 1>(dy, lddy, R, pos, T, K, I, dx, lddx, st);
    return wide ? run_dispatch_grad<F32, 4>(dy, lddy, R, pos, T, K, I, dx, lddx, st)
                : run_dispatch_grad<F32, 1>(dy, lddy, R, pos, T, K, I, dx, lddx, st);
}

hipError_t launch_moe_combine_grad(const void *dy, long long lddy, const void *h, long long ldh,
                                   int R, const int32_t *tokens, const int32_t *pos,
                                   const float *gates, int T, int K, int O, void *dh,
                                   long long lddh, float *dgates, int dtype, hipStream_t st)
{
    const int el = dtype == QGEMV_BF16 ? 2 : 4;
    const bool wide = aligned16((uintptr_t)dy | (uintptr_t)h | (uintptr_t)dh |
                                (uintptr_t)(lddy * el) | (uintptr_t)(ldh * el) |
                                (uintptr_t)(lddh * el));
    // eight slots per workgroup, two where eight would leave CUs without work.  Twos and
    // eights, us: kernel of 33 tokens of 8, 2048 f32 4.8 and 12.7; calls of 7168 bf16, 200
    // tokens 14.2 and 14.6, 300 17.1 and 20.7, 512 26.5 and 25.6, 1024 47.1 and 44.9
    const bool few = (long long)T * ((K + 7) / 8) < cu_count();
    const int nkb = few ? (K + 1) / 2 : (K + 7) / 8;
#define QG_GRAD(XT, VEC)                                                                    \
    do {                                                                                    \
        if (few) QG_GRAD1(XT, VEC, 2);                                                      \
        else QG_GRAD1(XT, VEC, 8);                                                          \
    } while (0)
#define QG_GRAD1(XT, VEC, KB)                                                               \
    hipLaunchKernelGGL((combine_grad<XT, VEC, KB>), dim3((unsigned)(n * nkb)), dim3(256), 0, st, \
                       static_cast<const XT::raw *>(dy) + t * lddy, lddy,                   \
                       static_cast<const XT::raw *>(h), ldh, R, tokens, pos + t * K,        \
                       gates + t * K, (int)t, K, O, static_cast<XT::raw *>(dh), lddh,       \
                       dgates + t * K, nkb)
    return sliced(T, 256LL * nkb, 1, [&](long long t, int n) {
        if (dtype == QGEMV_BF16) {
            if (wide) QG_GRAD(BF16, 8);
            else QG_GRAD(BF16, 1);
        } else {
            if (wide) QG_GRAD(F32, 4);
            else QG_GRAD(F32, 1);
        }
    });
#undef QG_GRAD
#undef QG_GRAD1
}

}  // namespace qg
