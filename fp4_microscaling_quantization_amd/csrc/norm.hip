// Layer norm and root-mean-square norm, forward and backward (include/mxq.h
// holds the formulas).  All of it is bound by memory: each row is read once and
// held in registers.
#include <math.h>

#include "mxq_host.hpp"
#include "rows.hpp"

namespace mxq {

namespace {

// ---- forward -------------------------------------------------------------------------

struct FwdArgs {
    int64_t ld_x, rows;
    int cols, layer;
    const float *gamma, *beta;
    float eps;
    void *y;
    int32_t y_dtype;
    int64_t ld_y;
    float *mean, *rstd;
};

// gamma and beta of the E columns from c on; rows shorter than a vector start at a
// negative c
template <bool SHORT, int E>
__device__ __forceinline__ void affine(float (&g)[E], float (&b)[E], const FwdArgs &a, int c)
{
#pragma unroll
    for (int j = 0; j < E; j += 4) {
        gv4u vg = {0x3F800000u, 0x3F800000u, 0x3F800000u, 0x3F800000u}, vb = {0u, 0u, 0u, 0u};
        if constexpr (SHORT) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if (c + j + k >= 0) {
                    vg[k] = a.gamma ? as_u(a.gamma[c + j + k]) : vg[k];
                    vb[k] = a.beta ? as_u(a.beta[c + j + k]) : vb[k];
                }
            }
        } else {
            if (a.gamma)
                vg = load_vec(a.gamma + c + j);
            if (a.beta)
                vb = load_vec(a.beta + c + j);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            g[j + k] = as_f(vg[k]);
            b[j + k] = as_f(vb[k]);
        }
    }
}

template <int NT> __device__ __forceinline__ float row_sum(float v, float *lds)
{
    if constexpr (NT == 64)
        return wave_sum(v);
    else
        return block_sum<NT>(v, lds);
}

// R rows a workgroup, NT x NV vectors of each in registers; a longer row (LONG, R = 1) is
// read again for each of the three passes.  The variance is the mean square of the
// differences from the mean, a second pass over registers: mean(x^2) - mu^2 loses
// what the two have in common.  Two rows share the loads of gamma and beta, which for
// a bf16 row are four times its own bytes (from L2: the row streams through L1).  Bound by
// memory: 8192 x 4096 bf16 24 us, 5.7 TB/s (34 us with one row a wave).  Rows that a wave does
// not hold have nobody to share with: 8192 x 8192 bf16 71 us, 3.8 TB/s.  fp32 from bf16, where a
// store's lanes are 32 bytes apart: 8192 x 4096 66 us, 3.1 TB/s (fp32 from fp32 54 us, 5.0).
template <class X, int NT, int NV, int R, bool LONG, bool SHORT>
__global__ void __launch_bounds__(NT) k_norm_fwd(const X *x, FwdArgs a)
{
    using H = Held<X, NT, NV>;
    constexpr int E = kElems<X>;
    __shared__ float lds[NT / 64];
    const float inv = 1.0f / (float)a.cols;
    for (int64_t first = (int64_t)blockIdx.x * R; first < a.rows; first += (int64_t)gridDim.x * R) {
        // an odd last row is worked on R times, and written once
        const X *xr[R];
        H h[R];
#pragma unroll
        for (int q = 0; q < R; ++q) {
            xr[q] = x + (first + q < a.rows ? first + q : first) * a.ld_x;
            if (!LONG)
                h[q].template load<SHORT, true>(xr[q], a.cols);
        }
        // f(vector's number, the stretch's first column, its columns)
        const auto each = [&](auto f) {
            const int cols = fresh(a.cols);
            if (!LONG) {
#pragma unroll
                for (int q = 0; q < R; ++q)
                    h[q].again();
            }
            for (int at = 0;;) {
                const int n = min(cols - at, H::kMost);
                if (LONG)
                    h[0].template load<SHORT, false>(xr[0] + at, n);
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    if (!H::any(i, n))
                        break;
                    f(i, at, n);
                }
                if (!LONG || cols - at <= H::kMost)
                    break;
                at += H::kMost;
            }
        };
        float mu[R], rs[R];
#pragma unroll
        for (int q = 0; q < R; ++q)
            mu[q] = rs[q] = 0.0f;
        if (a.layer) {
            each([&](int i, int, int n) {
#pragma unroll
                for (int q = 0; q < R; ++q) {
                    float v[E];
                    h[q].get(i, n, 0.0f, v);
#pragma unroll
                    for (int j = 0; j < E; ++j)
                        mu[q] += v[j];
                }
            });
#pragma unroll
            for (int q = 0; q < R; ++q)
                mu[q] = row_sum<NT>(mu[q], lds) * inv;
        }
        each([&](int i, int, int n) {
#pragma unroll
            for (int q = 0; q < R; ++q) {
                float v[E];
                h[q].get(i, n, mu[q], v);
#pragma unroll
                for (int j = 0; j < E; ++j)
                    rs[q] = fmaf(v[j] - mu[q], v[j] - mu[q], rs[q]);
            }
        });
#pragma unroll
        for (int q = 0; q < R; ++q)
            rs[q] = 1.0f / sqrtf(row_sum<NT>(rs[q], lds) * inv + a.eps);
        each([&](int i, int at, int n) {
            float g[E], b[E];
            affine<SHORT>(g, b, a, at + H::start(i, n));
#pragma unroll
            for (int q = 0; q < R; ++q) {
                if (q > 0 && first + q >= a.rows)
                    break;
                float v[E];
                h[q].get(i, v);
#pragma unroll
                for (int j = 0; j < E; ++j)
                    v[j] = (v[j] - mu[q]) * rs[q] * g[j] + b[j];
                const int64_t to = (first + q) * a.ld_y + at;
                if (a.y_dtype == MXQ_OUT_F32)
                    H::put((float *)a.y + to, i, n, v);
                else
                    H::put((bf16_t *)a.y + to, i, n, v);
            }
        });
        if (threadIdx.x == 0) {
#pragma unroll
            for (int q = 0; q < R; ++q) {
                if (first + q >= a.rows)
                    break;
                if (a.mean && a.layer)
                    a.mean[first + q] = mu[q];
                if (a.rstd)
                    a.rstd[first + q] = rs[q];
            }
        }
    }
}

// ---- backward ------------------------------------------------------------------------

struct BwdArgs {
    int64_t ld_dy, ld_x, rows;
    int cols, layer;
    const float *gamma, *mean, *rstd;
    void *dx;
    int32_t dx_dtype;
    int64_t ld_dx;
    float *part;  // NULL: no sums over the rows
};

// U consecutive elements of a row: a vector, or half of a bf16 one (U = 4)
template <class T, int U> struct Unit {
    using V = typename std::conditional<U * sizeof(T) == 16, gv4u, gv2u>::type;
    V v;
    __device__ __forceinline__ void load(const T *p)
    {
        if constexpr (sizeof(V) == 16)
            v = load_vec<true>(p);
        else
            v = __builtin_nontemporal_load((const MXQ_GLOBAL typename Unaligned<T>::v2 *)p);
    }
    __device__ __forceinline__ void clear() { v = V(0u); }
    // as Held::again
    __device__ __forceinline__ void again() { asm volatile("" : "+v"(v)); }
    __device__ __forceinline__ void get(float (&f)[U]) const
    {
#pragma unroll
        for (int j = 0; j < U; ++j) {
            if constexpr (sizeof(T) == 4)
                f[j] = as_f(v[j]);
            else
                f[j] = as_f(j % 2 ? v[j / 2] & 0xFFFF0000u : v[j / 2] << 16);
        }
    }
};

// NT threads as NT / TR groups, each on a row of its own: thread t of a group has
// the units (u TR + t) of U columns, 16 in all, for every row that the workgroup takes.  So
// gamma, and the sums over the rows of dy n and dy, stay in its registers, and dy
// and x come from memory once for dx and the sums together.  The next row is
// loaded before the present one is worked on.  With 1024 threads there are 128 registers:
// gamma is in LDS then, and a row is loaded in its turn, unless all is bf16 and dbeta is
// not asked for (BIAS).  Bound by memory: 8192 x 4096 fp32 dY, bf16 x and dx (268 MB)
// 52 us, 5.1 TB/s; 1000 x 14336 bf16 25 us, where a workgroup has at most four rows.
// One barrier a row: the row's two sums go through alternating places in LDS.
constexpr int kOwn = 16;  // columns of a thread
template <class D, class X> constexpr int kUnit = sizeof(D) + sizeof(X) == 4 ? 8 : 4;

template <class D, class X, int NT, int TR, bool BIAS>
__global__ void __launch_bounds__(NT, NT / 256) k_norm_bwd(const D *dy, const X *x, BwdArgs a)
{
    constexpr int G = NT / TR, W = TR / 64, EL = kOwn, U = kUnit<D, X>, NU = EL / U;
    constexpr bool kLdsGamma = NT == 1024;
    constexpr bool kAhead = NT < 1024 || (!BIAS && sizeof(D) + sizeof(X) == 4);
    __shared__ float lds[2][2][NT / 64];
    __shared__ float sums[G > 1 ? EL * NT : 1];
    __shared__ gv4u gammas[kLdsGamma ? EL / 4 : 1][kLdsGamma ? TR : 1];
    const int t = threadIdx.x % TR, g = threadIdx.x / TR, wave = threadIdx.x / 64;
    const float inv = 1.0f / (float)a.cols;

    float gamma[kLdsGamma ? 1 : EL], dg[EL], db[BIAS ? EL : 1];
#pragma unroll
    for (int e = 0; e < EL; ++e) {
        const int c = vec_start<U>((e / U * TR + t) * U, a.cols) + e % U;
        const float v = a.gamma ? a.gamma[c] : 1.0f;
        if constexpr (kLdsGamma)
            gammas[e / 4][t][e % 4] = as_u(v);  // read by the same thread only
        else
            gamma[e] = v;
        dg[e] = 0.0f;
        if constexpr (BIAS)
            db[e] = 0.0f;
    }
    const auto gamma_of = [&](int u, float (&out)[U]) {
#pragma unroll
        for (int j = 0; j < U; ++j) {
            if constexpr (kLdsGamma)
                out[j] = as_f(gammas[(u * U + j) / 4][t][j % 4]);
            else
                out[j] = gamma[u * U + j];
        }
    };

    Unit<D, U> ud[NU], nd[kAhead ? NU : 1];
    Unit<X, U> ux[NU], nx[kAhead ? NU : 1];
    float mu = 0.0f, rs = 0.0f, nmu = 0.0f, nrs = 0.0f;
    // a row beyond the last: rstd and dy are 0, so that nothing is added
    const auto load_or_none = [&](int64_t r, Unit<D, U> *d, Unit<X, U> *xx, float &m, float &s) {
        if (r < a.rows) {
            const D *dr = dy + r * a.ld_dy;
            const X *xr = x + r * a.ld_x;
            const int cols = fresh(a.cols);
#pragma unroll
            for (int u = 0; u < NU; ++u) {
                const int c = vec_start<U>((u * TR + t) * U, cols);
                d[u].load(dr + c);
                xx[u].load(xr + c);
            }
            m = a.layer ? a.mean[r] : 0.0f;
            s = a.rstd[r];
        } else {
#pragma unroll
            for (int u = 0; u < NU; ++u) {
                d[u].clear();
                xx[u].clear();
            }
            m = s = 0.0f;
        }
    };

    const int64_t step = (int64_t)gridDim.x * G;
    int64_t r = (int64_t)blockIdx.x * G + g;
    const int64_t first = (int64_t)blockIdx.x * G;  // the workgroup's rounds are uniform
    if (kAhead)
        load_or_none(r, nd, nx, nmu, nrs);
    int turn = 0;
    for (int64_t base = first; base < a.rows; base += step, r += step, turn ^= 1) {
        const int cols = fresh(a.cols);
        if (kAhead) {
#pragma unroll
            for (int u = 0; u < NU; ++u) {
                ud[u] = nd[u];
                ux[u] = nx[u];
            }
            mu = nmu;
            rs = nrs;
            if (base + step < a.rows)
                load_or_none(r + step, nd, nx, nmu, nrs);
        } else {
            load_or_none(r, ud, ux, mu, rs);
        }
        float su = 0.0f, sun = 0.0f;
#pragma unroll
        for (int u = 0; u < NU; ++u) {
            float d[U], v[U], gu[U];
            ud[u].get(d);
            ux[u].get(v);
            gamma_of(u, gu);
            if ((u + 1) * TR * U > cols) {
                // what is another unit's, or beyond the row, adds nothing
                const int c = (u * TR + t) * U, skip = c - vec_start<U>(c, cols);
#pragma unroll
                for (int j = 0; j < U; ++j)
                    d[j] = j >= skip ? d[j] : 0.0f;
            }
#pragma unroll
            for (int j = 0; j < U; ++j) {
                const int e = u * U + j;
                const float n = (v[j] - mu) * rs, w = d[j] * gu[j];
                su += w;
                sun = fmaf(w, n, sun);
                dg[e] = fmaf(d[j], n, dg[e]);
                if constexpr (BIAS)
                    db[e] += d[j];
            }
        }
        if (!a.dx)
            continue;
        su = wave_sum(su);
        sun = wave_sum(sun);
        if constexpr (W > 1) {
            if (threadIdx.x % 64 == 0) {
                lds[turn][0][wave] = su;
                lds[turn][1][wave] = sun;
            }
            __syncthreads();
            su = sun = 0.0f;
#pragma unroll
            for (int k = 0; k < W; ++k) {
                su += lds[turn][0][g * W + k];
                sun += lds[turn][1][g * W + k];
            }
        }
        const float mun = sun * inv, muu = a.layer ? su * inv : 0.0f;
        if (r < a.rows) {
#pragma unroll
            for (int u = 0; u < NU; ++u) {
                const int c = (u * TR + t) * U;
                float d[U], v[U], gu[U];
                gamma_of(u, gu);
                ud[u].again();
                ux[u].again();
                ud[u].get(d);
                ux[u].get(v);
#pragma unroll
                for (int j = 0; j < U; ++j) {
                    const float n = (v[j] - mu) * rs, w = d[j] * gu[j];
                    d[j] = rs * (fmaf(-n, mun, w) - muu);
                }
                const int from = vec_start<U>(c, cols);
                if (c < cols) {
                    if (a.dx_dtype == MXQ_OUT_F32)
                        store_from((float *)a.dx + r * a.ld_dx + from, d, c - from);
                    else
                        store_from((bf16_t *)a.dx + r * a.ld_dx + from, d, c - from);
                }
            }
        }
    }
    if (!a.part)
        return;
    // part [2][workgroups][EL][TR]: the sums in the order of the threads
    const int64_t slots = EL * TR;
#pragma unroll
    for (int which = 0; which < (BIAS ? 2 : 1); ++which) {
        float *to = a.part + ((int64_t)which * gridDim.x + blockIdx.x) * slots;
        if constexpr (G == 1) {
#pragma unroll
            for (int e = 0; e < EL; ++e)
                to[e * TR + t] = which ? db[BIAS ? e : 0] : dg[e];
        } else {
            __syncthreads();
#pragma unroll
            for (int e = 0; e < EL; ++e)
                sums[e * NT + threadIdx.x] = which ? db[BIAS ? e : 0] : dg[e];
            __syncthreads();
            for (int s = threadIdx.x; s < EL * TR; s += NT) {
                float v = 0.0f;
#pragma unroll
                for (int k = 0; k < G; ++k)
                    v += sums[s / TR * NT + k * TR + s % TR];
                to[s] = v;
            }
        }
    }
}

// dgamma and dbeta (blockIdx.y) from the workgroups' sums: 64 slots a workgroup,
// its 16 waves on a sixteenth of the sums each.  Latency: 3 to 5 us for 2 to 17 MB, most of
// them in the caches.
__global__ void __launch_bounds__(1024)
k_norm_sum(const float *part, int64_t groups, int tr, int unit, int cols, float *dgamma,
           float *dbeta)
{
    __shared__ float lds[16][64];
    float *out = blockIdx.y ? dbeta : dgamma;
    if (!out)
        return;
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, slots = tr * kOwn;
    const int s = blockIdx.x * 64 + lane;
    const float *p = part + blockIdx.y * groups * slots + s;
    float v = 0.0f;
#pragma unroll 16
    for (int64_t k = w; k < groups; k += 16)
        v += p[k * slots];
    lds[w][lane] = v;
    __syncthreads();
    if (w == 0) {
        v = 0.0f;
#pragma unroll
        for (int k = 0; k < 16; ++k)
            v += lds[k][lane];
        const int e = s / tr, c = (e / unit * tr + s % tr) * unit, from = min(c, cols - unit);
        if (e % unit >= c - from)
            out[from + e % unit] = v;
    }
}

// ---- backward of other rows ------------------------------------------------------------
// Rows wider than 1024 threads hold, and rows shorter than a vector.  dx a row at a time, from
// two reads of dy and x, the sums a column at a time, from another; one element a thread.  They
// are right and no more: layer norm of 2048 x 16392 bf16 187 us (1.1 TB/s of what has to move)
// where 2048 x 16384 in the kernel above takes 54, fp32 286 and 86 us; 262144 x 7 bf16 520 us,
// 262144 x 8 162 us.

constexpr int kWideNT = 256;

template <class D, class X>
__global__ void __launch_bounds__(kWideNT) k_norm_wide_dx(const D *dy, const X *x, BwdArgs a)
{
    __shared__ float lds[kWideNT / 64];
    const float inv = 1.0f / (float)a.cols;
    for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
        const D *dr = dy + r * a.ld_dy;
        const X *xr = x + r * a.ld_x;
        const float mu = a.layer ? a.mean[r] : 0.0f, rs = a.rstd[r];
        const auto weighed = [&](int64_t c) { return load_one(dr + c) * (a.gamma ? a.gamma[c] : 1.0f); };
        float su = 0.0f, sun = 0.0f;
        for (int64_t c = threadIdx.x; c < a.cols; c += kWideNT) {
            const float w = weighed(c);
            su += w;
            sun = fmaf(w, (load_one(xr + c) - mu) * rs, sun);
        }
        const float mun = block_sum<kWideNT>(sun, lds) * inv;
        const float muu = a.layer ? block_sum<kWideNT>(su, lds) * inv : 0.0f;
        for (int64_t c = threadIdx.x; c < a.cols; c += kWideNT) {
            const float n = (load_one(xr + c) - mu) * rs;
            const float v = rs * (fmaf(-n, mun, weighed(c)) - muu);
            if (a.dx_dtype == MXQ_OUT_F32)
                ((float *)a.dx)[r * a.ld_dx + c] = v;
            else
                ((bf16_t *)a.dx)[r * a.ld_dx + c] = (bf16_t)v;
        }
    }
}

// part [2][strips][slots], the slots here the columns
template <class D, class X>
__global__ void __launch_bounds__(kWideNT)
k_norm_wide_sums(const D *dy, const X *x, BwdArgs a, int64_t slots)
{
    const int64_t c = (int64_t)blockIdx.x * kWideNT + threadIdx.x;
    if (c >= a.cols)
        return;
    const int64_t strips = gridDim.y;
    float dg = 0.0f, db = 0.0f;
    for (int64_t r = blockIdx.y; r < a.rows; r += strips) {
        const float d = load_one(dy + r * a.ld_dy + c), mu = a.layer ? a.mean[r] : 0.0f;
        dg = fmaf(d, (load_one(x + r * a.ld_x + c) - mu) * a.rstd[r], dg);
        db += d;
    }
    a.part[blockIdx.y * slots + c] = dg;
    a.part[(strips + blockIdx.y) * slots + c] = db;
}
__global__ void __launch_bounds__(kWideNT)
k_norm_wide_sum(const float *part, int64_t strips, int64_t slots, int cols, float *dgamma,
                float *dbeta)
{
    const int64_t c = (int64_t)blockIdx.x * kWideNT + threadIdx.x;
    float *out = blockIdx.y ? dbeta : dgamma;
    if (c >= cols || !out)
        return;
    float v = 0.0f;
    for (int64_t s = 0; s < strips; ++s)
        v += part[(blockIdx.y * strips + s) * slots + c];
    out[c] = v;
}

// ---- the host's side -------------------------------------------------------------------

unsigned row_grid(int64_t rows) { return (unsigned)(rows < kMaxGrid ? rows : kMaxGrid); }
bool dtype_ok(int32_t d) { return d == MXQ_OUT_F32 || d == MXQ_OUT_BF16; }
bool aligned(const void *p, int32_t d)
{
    return reinterpret_cast<uintptr_t>(p) % (d == MXQ_OUT_F32 ? 4 : 2) == 0;
}
bool aligned4(const void *p) { return reinterpret_cast<uintptr_t>(p) % 4 == 0; }

// f(null pointer of the element type) for a dtype code that was checked
template <class F> void with_type(int32_t d, F f)
{
    if (d == MXQ_OUT_F32)
        f((float *)nullptr);
    else
        f((bf16_t *)nullptr);
}

// Rows from which a wave takes two: 1024 x 4096 bf16 7.2 us with one and 9.5 with two, 2048
// rows 9.3 and 11.2, 8192 rows 34 and 24.
constexpr int64_t kTwoRows = 4096;

// How the backward pass lays a problem out.  tr threads of a row hold 16 columns each;
// the workgroups are those that fill the chip once.  512 threads: 2048 x 4096 bf16 20.6 us,
// with 256 threads, so twice the workgroups and sums to add up, 24.5; 300 rows 14.0 and 14.6;
// 515 x 200 fp32 7.8 and 8.7.  Where that makes no more than kFewGroups workgroups, 256
// threads: 64 x 1024 bf16 7.2 us against 9.1, 40 x 4096 fp32 7.2 against 8.2.  Rows that take more
// than 512 threads: 1024, against the kernels for other rows (RMS, bf16) 16 x 8200 8.4 us and 21,
// 2048 x 9216 34 and 128, 8192 x 16384 144 and 598.
struct BwdPlan {
    int nt, tr;      // nt 0: the kernels for other rows
    int64_t groups;  // workgroups (other rows: strips), each with a set of sums
    int64_t slots;   // sums of a set
};
constexpr int64_t kCus = 256, kFewGroups = 32;

BwdPlan plan_bwd(int64_t rows, int64_t cols)
{
    BwdPlan p = {};
    if (cols > 1024 * kOwn || cols < 8) {
        p.groups = rows < kCus ? rows : kCus;
        p.slots = cols;
        return p;
    }
    p.tr = 64;
    while ((int64_t)p.tr * kOwn < cols)
        p.tr *= 2;
    p.nt = p.tr > 512 ? 1024 : p.tr <= 256 && rows <= kFewGroups * (512 / p.tr) ? 256 : 512;
    const int64_t per = p.nt / p.tr, need = (rows + per - 1) / per;
    p.groups = need < kCus ? need : kCus;
    p.slots = (int64_t)p.tr * kOwn;
    return p;
}

template <class D, class X>
void launch_bwd(const BwdPlan &p, const D *dy, const X *x, const BwdArgs &a, bool bias,
                hipStream_t s)
{
    const auto k = p.nt == 1024  ? (bias ? k_norm_bwd<D, X, 1024, 1024, true>
                                         : k_norm_bwd<D, X, 1024, 1024, false>)
                   : p.nt == 512 ? (p.tr == 64    ? k_norm_bwd<D, X, 512, 64, true>
                                    : p.tr == 128 ? k_norm_bwd<D, X, 512, 128, true>
                                    : p.tr == 256 ? k_norm_bwd<D, X, 512, 256, true>
                                                  : k_norm_bwd<D, X, 512, 512, true>)
                                 : (p.tr == 64    ? k_norm_bwd<D, X, 256, 64, true>
                                    : p.tr == 128 ? k_norm_bwd<D, X, 256, 128, true>
                                                  : k_norm_bwd<D, X, 256, 256, true>);
    hipLaunchKernelGGL(k, dim3((unsigned)p.groups), dim3(p.nt), 0, s, dy, x, a);
}

}  // namespace

}  // namespace mxq

using namespace mxq;

extern "C" mxq_status mxq_norm_forward(int32_t kind, const void *x, int32_t x_dtype, int64_t ld_x,
                                       int64_t rows, int64_t cols, const float *gamma,
                                       const float *beta, float eps, void *y, int32_t y_dtype,
                                       int64_t ld_y, float *mean, float *rstd, void *stream)
{
    if ((kind != MXQ_NORM_LAYER && kind != MXQ_NORM_RMS) || !dtype_ok(x_dtype) ||
        !dtype_ok(y_dtype) || !(eps >= 0.0f) || !(eps < INFINITY))
        return MXQ_ERR_UNSUPPORTED;
    if (rows < 0 || cols < 1 || cols > INT32_MAX || ld_x < cols || ld_y < cols)
        return MXQ_ERR_SHAPE;
    if (rows == 0)
        return MXQ_OK;
    if (!x || !y)
        return MXQ_ERR_NULL;
    if (!aligned(x, x_dtype) || !aligned(y, y_dtype) || !aligned4(gamma) || !aligned4(beta) ||
        !aligned4(mean) || !aligned4(rstd))
        return MXQ_ERR_ALIGN;
    const FwdArgs a = {ld_x, rows,    (int)cols, kind == MXQ_NORM_LAYER, gamma, beta, eps,
                       y,    y_dtype, ld_y,      mean,                   rstd};
    with_type(x_dtype, [&](auto *xt) {
        using X = std::remove_pointer_t<decltype(xt)>;
        const X *xx = static_cast<const X *>(x);
        hipStream_t s = static_cast<hipStream_t>(stream);
        constexpr int64_t one = 64 * 8 * kElems<X>;  // what a wave holds
        // The fewest threads that hold the row, a wave (no barrier) if one does; two rows a wave
        // when there are enough.  64 and 256 threads, bf16: 3000 x 4096 11.4 and 16.6 us, 8192 x
        // 2048 13.4 and 24.4, but 16 x 4096 5.4 and 3.8, 1024 x 4096 7.9 and 6.1.  256 and 1024:
        // 1024 x 8192 8.6 and 17.2, 8192 x 8192 71 and 121, 8192 x 16384 142 and 158, but 16 x
        // 16384 6.8 and 5.5.
        const bool two = cols >= kElems<X> && cols <= one && rows >= kTwoRows;
        const auto k = cols < kElems<X>   ? k_norm_fwd<X, 64, 8, 1, false, true>
                       : two              ? k_norm_fwd<X, 64, 8, 2, false, false>
                       : cols <= one      ? k_norm_fwd<X, 64, 8, 1, false, false>
                       : cols <= 4 * one  ? k_norm_fwd<X, 256, 8, 1, false, false>
                       : cols <= 16 * one ? k_norm_fwd<X, 1024, 8, 1, false, false>
                                          : k_norm_fwd<X, 1024, 8, 1, true, false>;
        const int nt = cols <= one ? 64 : cols <= 4 * one ? 256 : 1024;
        hipLaunchKernelGGL(k, dim3(row_grid(two ? (rows + 1) / 2 : rows)), dim3(nt), 0, s, xx, a);
    });
    return hipGetLastError() == hipSuccess ? MXQ_OK : MXQ_ERR_DEVICE;
}

extern "C" size_t mxq_norm_backward_workspace_size(int64_t rows, int64_t cols)
{
    if (rows < 0 || cols < 1 || cols > INT32_MAX)
        return 0;
    const BwdPlan p = plan_bwd(rows, cols);
    return (size_t)p.groups * (size_t)p.slots * 2 * sizeof(float);
}

extern "C" mxq_status mxq_norm_backward(int32_t kind, const void *dy, int32_t dy_dtype,
                                        int64_t ld_dy, const void *x, int32_t x_dtype,
                                        int64_t ld_x, int64_t rows, int64_t cols,
                                        const float *gamma, const float *mean, const float *rstd,
                                        void *dx, int32_t dx_dtype, int64_t ld_dx, float *dgamma,
                                        float *dbeta, void *workspace, size_t ws_bytes,
                                        void *stream)
{
    if ((kind != MXQ_NORM_LAYER && kind != MXQ_NORM_RMS) || !dtype_ok(dy_dtype) ||
        !dtype_ok(x_dtype) || !dtype_ok(dx_dtype))
        return MXQ_ERR_UNSUPPORTED;
    if (rows < 0 || cols < 1 || cols > INT32_MAX || ld_dy < cols || ld_x < cols ||
        (dx && ld_dx < cols))
        return MXQ_ERR_SHAPE;
    if (rows > 0 && (!dy || !x || !rstd || (kind == MXQ_NORM_LAYER && !mean)))
        return MXQ_ERR_NULL;
    if (!aligned(dy, dy_dtype) || !aligned(x, x_dtype) || !aligned(dx, dx_dtype) ||
        !aligned4(gamma) || !aligned4(mean) || !aligned4(rstd) || !aligned4(dgamma) ||
        !aligned4(dbeta) || !aligned4(workspace))
        return MXQ_ERR_ALIGN;
    const bool sums = dgamma || dbeta;
    if (sums && rows > 0 && (!workspace || ws_bytes < mxq_norm_backward_workspace_size(rows, cols)))
        return MXQ_ERR_WORKSPACE;
    if (!sums && (rows == 0 || !dx))
        return MXQ_OK;
    hipStream_t s = static_cast<hipStream_t>(stream);
    const BwdPlan p = plan_bwd(rows, cols);
    float *part = sums ? static_cast<float *>(workspace) : nullptr;
    const BwdArgs a = {ld_dy, ld_x, rows, (int)cols, kind == MXQ_NORM_LAYER, gamma,
                       mean,  rstd, dx,   dx_dtype,  ld_dx,                  part};
    const unsigned wide = (unsigned)((cols + kWideNT - 1) / kWideNT);
    if (rows > 0)
        with_type(dy_dtype, [&](auto *dt) {
            with_type(x_dtype, [&](auto *xt) {
                using D = std::remove_pointer_t<decltype(dt)>;
                using X = std::remove_pointer_t<decltype(xt)>;
                const D *d = static_cast<const D *>(dy);
                const X *xx = static_cast<const X *>(x);
                if (p.nt) {
                    launch_bwd(p, d, xx, a, dbeta != nullptr, s);
                    return;
                }
                // the sums first: dx may lie over dy or x
                if (sums)
                    hipLaunchKernelGGL((k_norm_wide_sums<D, X>), dim3(wide, (unsigned)p.groups),
                                       dim3(kWideNT), 0, s, d, xx, a, p.slots);
                if (dx)
                    hipLaunchKernelGGL((k_norm_wide_dx<D, X>), dim3(row_grid(rows)), dim3(kWideNT),
                                       0, s, d, xx, a);
            });
        });
    if (sums && p.nt)
        hipLaunchKernelGGL(k_norm_sum, dim3((unsigned)(p.slots / 64), 2), dim3(1024), 0, s, part,
                           p.groups, p.tr, dy_dtype == MXQ_OUT_BF16 && x_dtype == MXQ_OUT_BF16 ? 8 : 4,
                           (int)cols, dgamma, dbeta);
    else if (sums)
        hipLaunchKernelGGL(k_norm_wide_sum, dim3(wide, 2), dim3(kWideNT), 0, s, part, p.groups,
                           p.slots, (int)cols, dgamma, dbeta);
    return hipGetLastError() == hipSuccess ? MXQ_OK : MXQ_ERR_DEVICE;
}
