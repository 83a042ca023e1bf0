// The global norm of a list of gradients, and the gradients scaled down to a largest
// norm.
//
//   sum_sq = sum over all elements of g^2,  norm = sqrt(sum_sq),
//   c = min(1, max_norm / (norm + eps)),    out = c g.
//
// Both are bound by memory: one read for the norm, one read and one write for the
// clipping.  The squares are summed in fp64, where they are exact and neither overflow
// nor vanish; its two instructions an element hide behind the loads.
//
// 2.0 GB of bf16: norm 298 us, 6.7 TB/s.  5.6 GB of fp32 to bf16: norm 0.80 ms (6.9 TB/s),
// clipping 1.53 (5.5).  700 tensors, 91 MB in both: 32 us, bound by launches and by finding
// and starting on short tensors.
//
// The list goes to the kernels as an argument (no table in device memory that would have
// to be copied there, or be kept), a batch of it a launch.  A workgroup takes one chunk of
// one tensor, and finds it by counting the tensors that start at or before it.  The
// workgroups' sums are added up by one workgroup in a fixed order.
#include "mxq_host.hpp"
#include "rows.hpp"
#include "vocab.hpp"

namespace mxq {
namespace {

constexpr int kThreads = 256;
constexpr int kMostTensors = 1024;  // of a launch: 28 KB of arguments
constexpr int64_t kTypeBit = int64_t(1) << 62, kOutBit = int64_t(1) << 61;  // set: bf16
constexpr int64_t kCached = int64_t(192) << 20;  // bytes that stay in the last-level cache
// elements of a list (more than the memory holds), and workgroups of a launch: its threads are
// counted in 32 bits
constexpr int64_t kMostElements = int64_t(1) << 38;
constexpr int64_t kMostGroups = int64_t(1) << 23;

template <int N> struct Batch {
    const void *g[N];
    void *out[N];
    int64_t n[N];       // and the types' bits
    uint32_t first[N];  // the tensor's first workgroup
    int32_t count;
    int32_t chunk;  // elements of a workgroup
};

// the tensor of workgroup w: the last that starts at or before it
template <int N> __device__ __forceinline__ int tensor_of(const Batch<N> &b, uint32_t w)
{
    const int lane = threadIdx.x & 63;
    int n = 0;
#pragma unroll
    for (int i = 0; i < N; i += 64)
        if (i < b.count)
            n += __popcll(__ballot(i + lane < b.count && b.first[i + lane] <= w));
    return __builtin_amdgcn_readfirstlane(n) - 1;
}

// f(vector of E floats, index) for the workgroup's elements [0, n) at p, and f1(value, index)
// for those behind the last whole vector
constexpr int kAhead = 4;  // vectors of a thread in flight
template <class T, bool ONCE, int E, class F, class F1>
__device__ __forceinline__ void for_elements(const T *p, int n, F f, F1 f1)
{
    constexpr bool WHOLE = E == kElems<T>;
    static_assert(WHOLE || 2 * E == kElems<T>, "16 bytes or 8");
    using Raw = std::conditional_t<WHOLE, gv4u, gv2u>;
    using At = std::conditional_t<WHOLE, typename Unaligned<T>::v4, typename Unaligned<T>::v2>;
    const auto load = [&](int v) -> Raw {
        const auto *at = (const MXQ_GLOBAL At *)(p + (int64_t)v * E);
        return ONCE ? __builtin_nontemporal_load(at) : *at;
    };
    const int vectors = n / E;
    int v = threadIdx.x;
    for (; v + (kAhead - 1) * kThreads < vectors; v += kAhead * kThreads) {
        Raw raw[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
            raw[i] = load(v + i * kThreads);
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            float x[E];
            unpack(raw[i], x, (T *)nullptr);
            f(x, (v + i * kThreads) * E);
        }
    }
    for (; v < vectors; v += kThreads) {
        float x[E];
        unpack(load(v), x, (T *)nullptr);
        f(x, v * E);
    }
    const int rest = vectors * E + threadIdx.x;
    if (rest < n)
        f1(load_one(p + rest), rest);
}

template <bool ONCE, class T> __device__ __forceinline__ double squares(const T *p, int n)
{
    double s[2] = {0.0, 0.0};
    for_elements<T, ONCE, kElems<T>>(
        p, n,
        [&](const float(&x)[kElems<T>], int) {
#pragma unroll
            for (int j = 0; j < kElems<T>; ++j)
                s[j & 1] = fma((double)x[j], (double)x[j], s[j & 1]);
        },
        [&](float x, int) { s[0] = fma((double)x, (double)x, s[0]); });
    return s[0] + s[1];
}

__device__ __forceinline__ double wave_sum_double(double v)
{
#pragma unroll
    for (int d = 1; d < 64; d *= 2)
        v += __shfl_xor(v, d);
    return v;
}
template <int NT> __device__ __forceinline__ double block_sum_double(double v, double *lds)
{
    v = wave_sum_double(v);
    if ((threadIdx.x & 63) == 0)
        lds[threadIdx.x >> 6] = v;
    __syncthreads();
    double s = 0.0;
#pragma unroll
    for (int w = 0; w < NT / 64; ++w)
        s += lds[w];
    return s;
}

// ONCE: there is more than the caches hold until the clipping reads it again (2.0 GB of bf16
// 298 us with the hint, 336 without; 256 MB and their clipping 110 and 140; 100 MB that lie
// in the caches 54 and 23)
template <bool ONCE, int N>
__global__ __launch_bounds__(kThreads) void k_grad_squares(Batch<N> b, double *part)
{
    __shared__ double lds[kThreads / 64];
    const int t = tensor_of(b, blockIdx.x);
    const int64_t from = (int64_t)(blockIdx.x - b.first[t]) * b.chunk;
    const int64_t left = (b.n[t] & (kOutBit - 1)) - from;
    const int n = (int)(left < b.chunk ? left : b.chunk);
    const double s = b.n[t] & kTypeBit ? squares<ONCE>(static_cast<const bf16_t *>(b.g[t]) + from, n)
                                       : squares<ONCE>(static_cast<const float *>(b.g[t]) + from, n);
    const double all = block_sum_double<kThreads>(s, lds);
    if (threadIdx.x == 0)
        part[blockIdx.x] = all;
}

constexpr int kFinalThreads = 1024;
__global__ __launch_bounds__(kFinalThreads) void k_grad_norm(const double *part, int64_t n,
                                                             float *norm, double *sum_sq)
{
    __shared__ double lds[kFinalThreads / 64];
    double s[4] = {0.0, 0.0, 0.0, 0.0};
    int64_t i = threadIdx.x;
    for (; i + 3 * kFinalThreads < n; i += 4 * kFinalThreads)
#pragma unroll
        for (int k = 0; k < 4; ++k)
            s[k] += part[i + k * kFinalThreads];
    for (; i < n; i += kFinalThreads)
        s[0] += part[i];
    const double all = block_sum_double<kFinalThreads>((s[0] + s[1]) + (s[2] + s[3]), lds);
    if (threadIdx.x == 0) {
        if (sum_sq)
            *sum_sq = all;
        if (norm)
            *norm = (float)sqrt(all);
    }
}

// c as m 2^e, m an fp32 number in [1/2, 1]: c itself may be below fp32's normal numbers where c g
// is not
struct Scale {
    float m;
    int e;
};
// Four elements a lane where an output is fp32, so that a wave's store has no gaps (32 x 2^22
// bf16 to fp32 213 us with eight elements in two stores, 149 with four in one).
template <class T, class O>
__device__ __forceinline__ void scale_chunk(const T *p, O *out, int n, Scale c)
{
    constexpr int E = kElems<T> < kElems<O> ? kElems<T> : kElems<O>;
    for_elements<T, true, E>(
        p, n,
        [&](const float(&x)[E], int at) {
            float y[E];
#pragma unroll
            for (int j = 0; j < E; ++j)
                y[j] = __builtin_ldexpf(x[j] * c.m, c.e);
            store_vec(out + at, y);
        },
        [&](float x, int at) { out[at] = (O)__builtin_ldexpf(x * c.m, c.e); });
}

template <int N>
__global__ __launch_bounds__(kThreads) void k_grad_clip(Batch<N> b, const double *sum_sq,
                                                        float max_norm, float eps)
{
    const int t = tensor_of(b, blockIdx.x);
    const int64_t from = (int64_t)(blockIdx.x - b.first[t]) * b.chunk;
    const int64_t left = (b.n[t] & (kOutBit - 1)) - from;
    const int n = (int)(left < b.chunk ? left : b.chunk);
    const double q = (double)max_norm / (sqrt(*sum_sq) + (double)eps);
    Scale c = {1.0f, 0};
    if (!(q >= 1.0)) {  // NaN stays NaN
        int e = 0;
        c.m = (float)frexp(q, &e);
        c.e = e;
    } else if (b.out[t] == b.g[t]) {
        return;
    }
    const bool wide = !(b.n[t] & kTypeBit), out_wide = !(b.n[t] & kOutBit);
    const auto go = [&](auto *tt, auto *ot) {
        using T = std::remove_pointer_t<decltype(tt)>;
        using O = std::remove_pointer_t<decltype(ot)>;
        scale_chunk(static_cast<const T *>(b.g[t]) + from, static_cast<O *>(b.out[t]) + from, n, c);
    };
    if (wide)
        out_wide ? go((float *)nullptr, (float *)nullptr) : go((float *)nullptr, (bf16_t *)nullptr);
    else
        out_wide ? go((bf16_t *)nullptr, (float *)nullptr) : go((bf16_t *)nullptr, (bf16_t *)nullptr);
}

// ---- the host's side -------------------------------------------------------------

// Elements of a workgroup, from all there are: enough workgroups for the chip first, then
// fewer, longer ones.
int chunk_of(int64_t elements)
{
    int chunk = 4096;
    while (chunk < 32768 && elements / chunk > 4096)
        chunk *= 2;
    return chunk;
}

mxq_status check_grads(const mxq_grad *grads, int64_t count, bool out, int64_t &elements)
{
    elements = 0;
    if (count < 0 || count > INT32_MAX)
        return MXQ_ERR_SHAPE;
    if (count > 0 && !grads)
        return MXQ_ERR_NULL;
    for (int64_t i = 0; i < count; ++i) {
        const mxq_grad &g = grads[i];
        if (!dtype_ok(g.dtype) || (out && !dtype_ok(g.out_dtype)))
            return MXQ_ERR_UNSUPPORTED;
        if (g.n < 0 || g.n > kMostElements || (elements += g.n) > kMostElements)
            return MXQ_ERR_SHAPE;
        if (g.n > 0 && (!g.g || (out && !g.out)))
            return MXQ_ERR_NULL;
        if (!aligned(g.g, g.dtype) || (out && !aligned(g.out, g.out_dtype)))
            return MXQ_ERR_ALIGN;
        if (out && g.out == g.g && g.out_dtype != g.dtype && g.n > 0)
            return MXQ_ERR_UNSUPPORTED;
    }
    return MXQ_OK;
}

// The workgroups of all launches for the list.
int64_t groups_of(const mxq_grad *grads, int64_t count, int chunk)
{
    int64_t all = 0;
    for (int64_t i = 0; i < count; ++i)
        all += (grads[i].n + chunk - 1) / chunk;
    return all;
}

// launch(batch, workgroups) for the list, N tensors at a time
template <int N, class F>
void for_batches_of(const mxq_grad *grads, int64_t count, int chunk, F launch)
{
    Batch<N> b;
    b.count = 0;
    b.chunk = chunk;
    uint32_t groups = 0;
    const auto flush = [&] {
        if (b.count > 0)
            launch(b, groups);
        b.count = 0;
        groups = 0;
    };
    for (int64_t i = 0; i < count; ++i) {
        const mxq_grad &g = grads[i];
        if (g.n == 0)
            continue;
        const int64_t need = (g.n + chunk - 1) / chunk;
        if (b.count == N || (b.count > 0 && groups + need > kMostGroups))
            flush();
        b.g[b.count] = g.g;
        b.out[b.count] = g.out;
        b.n[b.count] = g.n | (g.dtype == MXQ_OUT_BF16 ? kTypeBit : 0) |
                       (g.out_dtype == MXQ_OUT_BF16 ? kOutBit : 0);
        b.first[b.count++] = groups;
        groups += (uint32_t)need;
    }
    flush();
}
// with the shortest argument that holds the list: 10 tensors 8 us with room for 32, 21 with
// room for 1000; 700 tensors 34 us in one launch each, 60 in launches of 128
template <class F> void for_batches(const mxq_grad *grads, int64_t count, int chunk, F launch)
{
    if (count <= 32)
        for_batches_of<32>(grads, count, chunk, launch);
    else if (count <= 256)
        for_batches_of<256>(grads, count, chunk, launch);
    else
        for_batches_of<kMostTensors>(grads, count, chunk, launch);
}

}  // namespace
}  // namespace mxq

using namespace mxq;

extern "C" size_t mxq_grad_norm_workspace_size(const mxq_grad *grads, int64_t count)
{
    int64_t elements;
    if (check_grads(grads, count, false, elements))
        return 0;
    return 8 * (size_t)groups_of(grads, count, chunk_of(elements));
}

extern "C" mxq_status mxq_grad_norm(const mxq_grad *grads, int64_t count, float *norm,
                                    double *sum_sq, void *workspace, size_t ws_bytes, void *stream)
{
    int64_t elements;
    const mxq_status st = check_grads(grads, count, false, elements);
    if (st)
        return st;
    if (!norm && !sum_sq)
        return MXQ_ERR_NULL;
    if (!aligned4(norm) || reinterpret_cast<uintptr_t>(sum_sq) % 8 ||
        reinterpret_cast<uintptr_t>(workspace) % 8)
        return MXQ_ERR_ALIGN;
    const int chunk = chunk_of(elements);
    const int64_t parts = groups_of(grads, count, chunk);
    if (parts > 0 && (!workspace || ws_bytes < 8 * (size_t)parts))
        return MXQ_ERR_WORKSPACE;
    hipStream_t s = static_cast<hipStream_t>(stream);
    double *part = static_cast<double *>(workspace);
    int64_t bytes = 0;
    for (int64_t i = 0; i < count; ++i)
        bytes += grads[i].n * (grads[i].dtype == MXQ_OUT_BF16 ? 2 : 4);
    for_batches(grads, count, chunk, [&](const auto &b, uint32_t groups) {
        constexpr int N = sizeof(b.n) / sizeof(b.n[0]);
        const auto k = bytes > kCached ? k_grad_squares<true, N> : k_grad_squares<false, N>;
        hipLaunchKernelGGL(k, dim3(groups), dim3(kThreads), 0, s, b, part);
        part += groups;
    });
    hipLaunchKernelGGL(k_grad_norm, dim3(1), dim3(kFinalThreads), 0, s,
                       static_cast<const double *>(workspace), parts, norm, sum_sq);
    return launched();
}

extern "C" mxq_status mxq_grad_clip(const mxq_grad *grads, int64_t count, const double *sum_sq,
                                    float max_norm, float eps, void *stream)
{
    int64_t elements;
    const mxq_status st = check_grads(grads, count, true, elements);
    if (st)
        return st;
    if (!(max_norm >= 0.0f) || !(max_norm < INFINITY) || !(eps >= 0.0f) || !(eps < INFINITY))
        return MXQ_ERR_UNSUPPORTED;
    if (!sum_sq)
        return MXQ_ERR_NULL;
    if (reinterpret_cast<uintptr_t>(sum_sq) % 8)
        return MXQ_ERR_ALIGN;
    if (elements == 0)
        return MXQ_OK;
    hipStream_t s = static_cast<hipStream_t>(stream);
    for_batches(grads, count, chunk_of(elements), [&](const auto &b, uint32_t groups) {
        hipLaunchKernelGGL(k_grad_clip, dim3(groups), dim3(kThreads), 0, s, b, sum_sq, max_norm, eps);
    });
    return launched();
}
