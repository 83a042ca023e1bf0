// Layer norm and root-mean-square norm, forward and backward (mxq_norm_forward,
// mxq_norm_backward in include/mxq.h hold the formulas).
//
// Forward: one workgroup per row.  Backward: one workgroup per row for dx; the
// gradients of gamma and beta sum dy n and dy over the rows, first over strips
// of rows into the workspace, then over the strips, both in a fixed order.
#include <math.h>

#include "mxq_host.hpp"
#include "rows.hpp"

namespace mxq {

namespace {

constexpr int kNT = 256;
constexpr int64_t kMaxGrid = 1 << 20;  // workgroups of a launch over rows; more rows loop
constexpr int64_t kStrips = 256;       // row strips of the column sums

template <class X, class Y>
__global__ void __launch_bounds__(kNT)
k_norm_fwd(int kind, const X *x, int64_t ld_x, int64_t rows, int cols, const float *gamma,
           const float *beta, float eps, Y *y, int64_t ld_y, float *mean, float *rstd)
{
    __shared__ float lds[kNT / 64];
    for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
        const X *xr = x + r * ld_x;
        Y *yr = y + r * ld_y;
        float mu = 0.0f;
        if (kind == MXQ_NORM_LAYER) {
            float s = 0.0f;
            for (int i = threadIdx.x; i < cols; i += kNT)
                s += (float)xr[i];
            mu = block_sum<kNT>(s, lds) / (float)cols;
        }
        float s2 = 0.0f;
        for (int i = threadIdx.x; i < cols; i += kNT) {
            const float c = (float)xr[i] - mu;
            s2 = fmaf(c, c, s2);
        }
        const float rs = 1.0f / sqrtf(block_sum<kNT>(s2, lds) / (float)cols + eps);
        for (int i = threadIdx.x; i < cols; i += kNT) {
            const float n = ((float)xr[i] - mu) * rs;
            yr[i] = (Y)fmaf(n, gamma ? gamma[i] : 1.0f, beta ? beta[i] : 0.0f);
        }
        if (threadIdx.x == 0) {
            if (mean && kind == MXQ_NORM_LAYER)
                mean[r] = mu;
            if (rstd)
                rstd[r] = rs;
        }
    }
}

template <class D, class X, class O>
__global__ void __launch_bounds__(kNT)
k_norm_dx(int kind, const D *dy, int64_t ld_dy, const X *x, int64_t ld_x, int64_t rows, int cols,
          const float *gamma, const float *mean, const float *rstd, O *dx, int64_t ld_dx)
{
    __shared__ float lds[kNT / 64];
    for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
        const D *dr = dy + r * ld_dy;
        const X *xr = x + r * ld_x;
        O *o = dx + r * ld_dx;
        const float mu = kind == MXQ_NORM_LAYER ? mean[r] : 0.0f, rs = rstd[r];
        float su = 0.0f, sun = 0.0f;
        for (int i = threadIdx.x; i < cols; i += kNT) {
            const float u = (float)dr[i] * (gamma ? gamma[i] : 1.0f);
            su += u;
            sun = fmaf(u, ((float)xr[i] - mu) * rs, sun);
        }
        const float mun = block_sum<kNT>(sun, lds) / (float)cols;
        const float mu_u = kind == MXQ_NORM_LAYER ? block_sum<kNT>(su, lds) / (float)cols : 0.0f;
        for (int i = threadIdx.x; i < cols; i += kNT) {
            const float u = (float)dr[i] * (gamma ? gamma[i] : 1.0f);
            const float n = ((float)xr[i] - mu) * rs;
            o[i] = (O)(rs * (fmaf(-n, mun, u) - mu_u));
        }
    }
}

// part [2][strips][cols]: the sums of dy n and of dy over the rows of a strip
template <class D, class X>
__global__ void __launch_bounds__(kNT)
k_norm_dcols(int kind, const D *dy, int64_t ld_dy, const X *x, int64_t ld_x, int64_t rows,
             int cols, const float *mean, const float *rstd, float *part)
{
    const int c = blockIdx.x * kNT + threadIdx.x;
    if (c >= cols)
        return;
    const int64_t strips = gridDim.y;
    float sg = 0.0f, sb = 0.0f;
    for (int64_t r = blockIdx.y; r < rows; r += strips) {
        const float d = (float)dy[r * ld_dy + c];
        const float mu = kind == MXQ_NORM_LAYER ? mean[r] : 0.0f;
        sg = fmaf(d, ((float)x[r * ld_x + c] - mu) * rstd[r], sg);
        sb += d;
    }
    part[blockIdx.y * (int64_t)cols + c] = sg;
    part[(strips + blockIdx.y) * cols + c] = sb;
}

__global__ void __launch_bounds__(kNT)
k_norm_dsum(const float *part, int64_t strips, int cols, float *dgamma, float *dbeta)
{
    const int c = blockIdx.x * kNT + threadIdx.x;
    if (c >= cols)
        return;
    float sg = 0.0f, sb = 0.0f;
    for (int64_t s = 0; s < strips; ++s) {
        sg += part[s * cols + c];
        sb += part[(strips + s) * cols + c];
    }
    if (dgamma)
        dgamma[c] = sg;
    if (dbeta)
        dbeta[c] = sb;
}

int64_t strips_of(int64_t rows) { return rows < kStrips ? rows : kStrips; }
unsigned row_grid(int64_t rows) { return (unsigned)(rows < kMaxGrid ? rows : kMaxGrid); }

bool dtype_ok(int32_t d) { return d == MXQ_OUT_F32 || d == MXQ_OUT_BF16; }
bool aligned(const void *p, int32_t d) { return reinterpret_cast<uintptr_t>(p) % (d == MXQ_OUT_F32 ? 4 : 2) == 0; }

// f(null pointer of the element type) for a dtype code that was checked
template <class F> void with_type(int32_t d, F f)
{
    if (d == MXQ_OUT_F32)
        f((float *)nullptr);
    else
        f((bf16_t *)nullptr);
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
    if (!aligned(x, x_dtype) || !aligned(y, y_dtype) || !aligned(gamma, MXQ_OUT_F32) ||
        !aligned(beta, MXQ_OUT_F32) || !aligned(mean, MXQ_OUT_F32) || !aligned(rstd, MXQ_OUT_F32))
        return MXQ_ERR_ALIGN;
    hipStream_t s = static_cast<hipStream_t>(stream);
    with_type(x_dtype, [&](auto *xt) {
        with_type(y_dtype, [&](auto *yt) {
            using X = std::remove_pointer_t<decltype(xt)>;
            using Y = std::remove_pointer_t<decltype(yt)>;
            hipLaunchKernelGGL((k_norm_fwd<X, Y>), dim3(row_grid(rows)), dim3(kNT), 0, s, kind,
                               static_cast<const X *>(x), ld_x, rows, (int)cols, gamma, beta, eps,
                               static_cast<Y *>(y), ld_y, mean, rstd);
        });
    });
    return hipGetLastError() == hipSuccess ? MXQ_OK : MXQ_ERR_DEVICE;
}

extern "C" size_t mxq_norm_backward_workspace_size(int64_t rows, int64_t cols)
{
    if (rows < 0 || cols < 1 || cols > INT32_MAX)
        return 0;
    return (size_t)strips_of(rows) * (size_t)cols * 2 * sizeof(float);
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
        !aligned(gamma, MXQ_OUT_F32) || !aligned(mean, MXQ_OUT_F32) ||
        !aligned(rstd, MXQ_OUT_F32) || !aligned(dgamma, MXQ_OUT_F32) ||
        !aligned(dbeta, MXQ_OUT_F32) || !aligned(workspace, MXQ_OUT_F32))
        return MXQ_ERR_ALIGN;
    const bool sums = dgamma || dbeta;
    if (sums && rows > 0 && (!workspace || ws_bytes < mxq_norm_backward_workspace_size(rows, cols)))
        return MXQ_ERR_WORKSPACE;
    if (!sums && (rows == 0 || !dx))
        return MXQ_OK;
    hipStream_t s = static_cast<hipStream_t>(stream);
    const unsigned gx = (unsigned)((cols + kNT - 1) / kNT);
    const int64_t strips = strips_of(rows);
    float *part = static_cast<float *>(workspace);
    with_type(dy_dtype, [&](auto *dt) {
        with_type(x_dtype, [&](auto *xt) {
            using D = std::remove_pointer_t<decltype(dt)>;
            using X = std::remove_pointer_t<decltype(xt)>;
            const D *d = static_cast<const D *>(dy);
            const X *xx = static_cast<const X *>(x);
            // the column sums first: dx may overwrite dy or x
            if (sums && rows > 0)
                hipLaunchKernelGGL((k_norm_dcols<D, X>), dim3(gx, (unsigned)strips), dim3(kNT), 0,
                                   s, kind, d, ld_dy, xx, ld_x, rows, (int)cols, mean, rstd, part);
            if (dx && rows > 0)
                with_type(dx_dtype, [&](auto *ot) {
                    using O = std::remove_pointer_t<decltype(ot)>;
                    hipLaunchKernelGGL((k_norm_dx<D, X, O>), dim3(row_grid(rows)), dim3(kNT), 0, s,
                                       kind, d, ld_dy, xx, ld_x, rows, (int)cols, gamma, mean,
                                       rstd, static_cast<O *>(dx), ld_dx);
                });
        });
    });
    if (sums)
        hipLaunchKernelGGL(k_norm_dsum, dim3(gx), dim3(kNT), 0, s, part, strips, (int)cols, dgamma,
                           dbeta);
    return hipGetLastError() == hipSuccess ? MXQ_OK : MXQ_ERR_DEVICE;
}
