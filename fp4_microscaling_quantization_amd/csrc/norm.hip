// Layer norm and root-mean-square norm, forward and backward (include/mxq.h
// holds the formulas).  All of it is bound by memory: each row is read once and
// held in registers.
#include <math.h>

#include "mxq_host.hpp"
#include "rows.hpp"

namespace mxq {

namespace {

constexpr int64_t kMaxGrid = 1 << 20;  // workgroups of a launch over rows; more rows loop

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

// n gamma + beta of the E columns from c on; rows shorter than a vector start at a
// negative c
template <bool SHORT, int E>
__device__ __forceinline__ void affine(float (&f)[E], const FwdArgs &a, int c)
{
    if (SHORT) {
#pragma unroll
        for (int j = 0; j < E; ++j)
            if (c + j >= 0)
                f[j] = f[j] * (a.gamma ? a.gamma[c + j] : 1.0f) + (a.beta ? a.beta[c + j] : 0.0f);
        return;
    }
#pragma unroll
    for (int j = 0; j < E; j += 4) {
        if (a.gamma) {
            const gv4u v = load_vec(a.gamma + c + j);
#pragma unroll
            for (int k = 0; k < 4; ++k)
                f[j + k] *= as_f(v[k]);
        }
        if (a.beta) {
            const gv4u v = load_vec(a.beta + c + j);
#pragma unroll
            for (int k = 0; k < 4; ++k)
                f[j + k] += as_f(v[k]);
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

// One workgroup per row, NT x NV vectors of it in registers; a longer row (LONG)
// is read again for each of the three passes.  The variance is the mean square of
// the differences from the mean, a second pass over registers: mean(x^2) - mu^2
// loses what the two have in common.
template <class X, int NT, int NV, bool LONG, bool SHORT>
__global__ void __launch_bounds__(NT) k_norm_fwd(const X *x, FwdArgs a)
{
    using H = Held<X, NT, NV>;
    constexpr int E = kElems<X>;
    __shared__ float lds[NT / 64];
    const float inv = 1.0f / (float)a.cols;
    for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
        const X *xr = x + r * a.ld_x;
        H h;
        if (!LONG)
            h.template load<SHORT, true>(xr, a.cols);
        // f(vector's number, the stretch's first column, its columns)
        const auto each = [&](auto f) {
            const int cols = fresh(a.cols);
            if (!LONG)
                h.again();
            for (int at = 0;;) {
                const int n = min(cols - at, H::kMost);
                if (LONG)
                    h.template load<SHORT, false>(xr + at, n);
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    if (!h.any(i, n))
                        break;
                    f(i, at, n);
                }
                if (!LONG || cols - at <= H::kMost)
                    break;
                at += H::kMost;
            }
        };
        float mu = 0.0f;
        if (a.layer) {
            float s = 0.0f;
            each([&](int i, int, int n) {
                float v[E];
                h.get(i, n, 0.0f, v);
#pragma unroll
                for (int j = 0; j < E; ++j)
                    s += v[j];
            });
            mu = row_sum<NT>(s, lds) * inv;
        }
        float s2 = 0.0f;
        each([&](int i, int, int n) {
            float v[E];
            h.get(i, n, mu, v);
#pragma unroll
            for (int j = 0; j < E; ++j)
                s2 = fmaf(v[j] - mu, v[j] - mu, s2);
        });
        const float rs = 1.0f / sqrtf(row_sum<NT>(s2, lds) * inv + a.eps);
        each([&](int i, int at, int n) {
            float v[E];
            h.get(i, v);
#pragma unroll
            for (int j = 0; j < E; ++j)
                v[j] = (v[j] - mu) * rs;
            affine<SHORT>(v, a, at + h.start(i, n));
            if (a.y_dtype == MXQ_OUT_F32)
                h.put((float *)a.y + r * a.ld_y + at, i, n, v);
            else
                h.put((bf16_t *)a.y + r * a.ld_y + at, i, n, v);
        });
        if (threadIdx.x == 0) {
            if (a.mean && a.layer)
                a.mean[r] = mu;
            if (a.rstd)
                a.rstd[r] = rs;
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

// 8 consecutive elements of a row, of either type
template <class T> struct Unit {
    static constexpr int V = 8 / kElems<T>;
    gv4u v[V];
    __device__ __forceinline__ void load(const T *p)
    {
#pragma unroll
        for (int k = 0; k < V; ++k)
            v[k] = load_vec<true>(p + k * kElems<T>);
    }
    // as Held::again
    __device__ __forceinline__ void again()
    {
#pragma unroll
        for (int k = 0; k < V; ++k)
            asm volatile("" : "+v"(v[k]));
    }
    __device__ __forceinline__ void get(float (&f)[8]) const
    {
        if constexpr (V == 1) {
            unpack(v[0], f, (T *)nullptr);
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k)
                f[k] = as_f(v[k / 4][k % 4]);
        }
    }
};

// NT threads as NT / TR groups, each on a row of its own: thread t of a group has
// the NU units (u TR + t) of 8 columns, for every row that the workgroup takes.  So
// gamma, and the sums over the rows of dy n and dy, stay in its registers, and dy
// and x come from memory once for dx and the sums together.  The next row is
// loaded before the present one is worked on, where the registers have room.
// One barrier a row: the row's two sums go through alternating places in LDS.
template <class D, class X, int NT, int TR, int NU>
__global__ void __launch_bounds__(NT, NT / 256) k_norm_bwd(const D *dy, const X *x, BwdArgs a)
{
    constexpr int G = NT / TR, W = TR / 64, EL = 8 * NU;
    constexpr bool kAhead = NU * 4 * (Unit<D>::V + Unit<X>::V) <= 64;
    __shared__ float lds[2][2][NT / 64];
    __shared__ float sums[G > 1 ? EL * NT : 1];
    const int t = threadIdx.x % TR, g = threadIdx.x / TR, wave = threadIdx.x / 64;
    const float inv = 1.0f / (float)a.cols;

    float gamma[EL], dg[EL], db[EL];
#pragma unroll
    for (int e = 0; e < EL; ++e) {
        const int c = vec_start<8>((e / 8 * TR + t) * 8, a.cols) + e % 8;
        gamma[e] = a.gamma ? a.gamma[c] : 1.0f;
        dg[e] = db[e] = 0.0f;
    }

    Unit<D> ud[NU], nd[kAhead ? NU : 1];
    Unit<X> ux[NU], nx[kAhead ? NU : 1];
    float mu = 0.0f, rs = 0.0f, nmu = 0.0f, nrs = 0.0f;
    const auto load = [&](int64_t r, Unit<D> *d, Unit<X> *xx, float &m, float &s) {
        const D *dr = dy + r * a.ld_dy;
        const X *xr = x + r * a.ld_x;
        const int cols = fresh(a.cols);
#pragma unroll
        for (int u = 0; u < NU; ++u) {
            const int c = vec_start<8>((u * TR + t) * 8, cols);
            d[u].load(dr + c);
            xx[u].load(xr + c);
        }
        m = a.layer ? a.mean[r] : 0.0f;
        s = a.rstd[r];
    };
    // a row beyond the last: rstd and dy are 0, so that nothing is added
    const auto load_or_none = [&](int64_t r, Unit<D> *d, Unit<X> *xx, float &m, float &s) {
        if (r < a.rows) {
            load(r, d, xx, m, s);
        } else {
#pragma unroll
            for (int u = 0; u < NU; ++u) {
#pragma unroll
                for (int k = 0; k < Unit<D>::V; ++k)
                    d[u].v[k] = (gv4u){0u, 0u, 0u, 0u};
#pragma unroll
                for (int k = 0; k < Unit<X>::V; ++k)
                    xx[u].v[k] = (gv4u){0u, 0u, 0u, 0u};
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
            float d[8], v[8];
            ud[u].get(d);
            ux[u].get(v);
            if ((u + 1) * TR * 8 > cols) {
                // what is another unit's, or beyond the row, adds nothing
                const int c = (u * TR + t) * 8, skip = c - vec_start<8>(c, cols);
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    d[j] = j >= skip ? d[j] : 0.0f;
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int e = u * 8 + j;
                const float n = (v[j] - mu) * rs, w = d[j] * gamma[e];
                su += w;
                sun = fmaf(w, n, sun);
                dg[e] = fmaf(d[j], n, dg[e]);
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
                const int c = (u * TR + t) * 8;
                float d[8], v[8];
                ud[u].again();
                ux[u].again();
                ud[u].get(d);
                ux[u].get(v);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float n = (v[j] - mu) * rs, w = d[j] * gamma[u * 8 + j];
                    d[j] = rs * (fmaf(-n, mun, w) - muu);
                }
                const int from = vec_start<8>(c, cols);
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
    for (int which = 0; which < 2; ++which) {
        float *to = a.part + ((int64_t)which * gridDim.x + blockIdx.x) * slots;
        if constexpr (G == 1) {
#pragma unroll
            for (int e = 0; e < EL; ++e)
                to[e * TR + t] = which ? db[e] : dg[e];
        } else {
            __syncthreads();
#pragma unroll
            for (int e = 0; e < EL; ++e)
                sums[e * NT + threadIdx.x] = which ? db[e] : dg[e];
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
// its 16 waves on a sixteenth of the sums each.
__global__ void __launch_bounds__(1024)
k_norm_sum(const float *part, int64_t groups, int tr, int slots, int cols, float *dgamma,
           float *dbeta)
{
    __shared__ float lds[16][64];
    float *out = blockIdx.y ? dbeta : dgamma;
    if (!out)
        return;
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    const int s = blockIdx.x * 64 + lane;
    const float *p = part + blockIdx.y * groups * slots + s;
    float v = 0.0f;
    for (int64_t k = w; k < groups; k += 16)
        v += p[k * slots];
    lds[w][lane] = v;
    __syncthreads();
    if (w == 0) {
        v = 0.0f;
#pragma unroll
        for (int k = 0; k < 16; ++k)
            v += lds[k][lane];
        const int e = s / tr, c = (e / 8 * tr + s % tr) * 8, from = vec_start<8>(c, cols);
        if (e % 8 >= c - from)
            out[from + e % 8] = v;
    }
}

// ---- backward of other rows ------------------------------------------------------------
// Wider rows, and rows shorter than a vector.  dx a row at a time, the sums a column at a time; dy and x are read once for each.

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

// How the backward pass lays a problem out.  tr threads of a row hold 16 columns
// each, 32 for rows over 8192; the workgroups are those that fill the chip once.
// Few rows: workgroups of 256 threads spread them over more CUs.
struct BwdPlan {
    int nt, tr, nu;      // nt 0: the wide kernels
    int64_t groups;      // workgroups (wide: strips), each with a set of sums
    int64_t slots;       // sums of a set
};
constexpr int64_t kCus = 256;

BwdPlan plan_bwd(int64_t rows, int64_t cols)
{
    BwdPlan p = {};
    if (cols > 16384 || cols < 8) {
        p.groups = rows < kCus ? rows : kCus;
        p.slots = cols;
        return p;
    }
    p.nu = cols > 8192 ? 4 : 2;
    p.tr = 64;
    while ((int64_t)p.tr * 8 * p.nu < cols)
        p.tr *= 2;
    p.nt = p.tr <= 256 && rows < kCus * (512 / p.tr) ? 256 : 512;
    const int64_t per = p.nt / p.tr, need = (rows + per - 1) / per;
    const int64_t most = p.nt == 256 ? 2 * kCus : kCus;
    p.groups = need < most ? need : most;
    p.slots = (int64_t)p.tr * 8 * p.nu;
    return p;
}

template <class D, class X>
void launch_bwd(const BwdPlan &p, const D *dy, const X *x, const BwdArgs &a, hipStream_t s)
{
    const auto go = [&](auto nt, auto tr, auto nu) {
        constexpr int NT = decltype(nt)::value, TR = decltype(tr)::value, NU = decltype(nu)::value;
        hipLaunchKernelGGL((k_norm_bwd<D, X, NT, TR, NU>), dim3((unsigned)p.groups), dim3(NT), 0,
                           s, dy, x, a);
    };
    using i2 = std::integral_constant<int, 2>;
    using i4 = std::integral_constant<int, 4>;
    using i64 = std::integral_constant<int, 64>;
    using i128 = std::integral_constant<int, 128>;
    using i256 = std::integral_constant<int, 256>;
    using i512 = std::integral_constant<int, 512>;
    if (p.nt == 256) {
        if (p.tr == 64)
            go(i256(), i64(), i2());
        else if (p.tr == 128)
            go(i256(), i128(), i2());
        else
            go(i256(), i256(), i2());
    } else if (p.nu == 4) {
        go(i512(), i512(), i4());
    } else {
        if (p.tr == 64)
            go(i512(), i64(), i2());
        else if (p.tr == 128)
            go(i512(), i128(), i2());
        else if (p.tr == 256)
            go(i512(), i256(), i2());
        else
            go(i512(), i512(), i2());
    }
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
        // a wave per row while it holds the row: no barrier
        const auto k = cols < kElems<X>   ? k_norm_fwd<X, 64, 8, false, true>
                       : cols <= one      ? k_norm_fwd<X, 64, 8, false, false>
                       : cols <= 4 * one  ? k_norm_fwd<X, 256, 8, false, false>
                       : cols <= 16 * one ? k_norm_fwd<X, 1024, 8, false, false>
                                          : k_norm_fwd<X, 1024, 8, true, false>;
        const int nt = cols <= one ? 64 : cols <= 4 * one ? 256 : 1024;
        hipLaunchKernelGGL(k, dim3(row_grid(rows)), dim3(nt), 0, s, xx, a);
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
                    launch_bwd(p, d, xx, a, s);
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
                           p.groups, p.tr, (int)p.slots, (int)cols, dgamma, dbeta);
    else if (sums)
        hipLaunchKernelGGL(k_norm_wide_sum, dim3(wide, 2), dim3(kWideNT), 0, s, part, p.groups,
                           p.slots, (int)cols, dgamma, dbeta);
    return hipGetLastError() == hipSuccess ? MXQ_OK : MXQ_ERR_DEVICE;
}
