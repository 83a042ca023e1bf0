// Row operators over a vocabulary (include/mxq.h holds the formulas): token log
// probabilities with entropy and top alternatives, distillation from a
// teacher's alternatives, and their gradients.  One workgroup per row.
#include <math.h>

#include "mxq_host.hpp"
#include "rows.hpp"

namespace mxq {

namespace {

constexpr int kNT = 256;
constexpr int64_t kMaxGrid = 1 << 20;  // workgroups of a launch over rows; more rows loop

// The logits' values as an order: larger keys come first, equal values by
// index (the low half, complemented).  -0 counts as 0.
__device__ __forceinline__ uint64_t order_key(float z, int i)
{
    const uint32_t u = as_u(z + 0.0f);
    const uint32_t o = (u >> 31) ? ~u : (u | 0x80000000u);
    return ((uint64_t)o << 32) | (uint32_t)~i;
}
__device__ __forceinline__ float key_value(uint64_t k)
{
    const uint32_t o = (uint32_t)(k >> 32);
    return as_f((o >> 31) ? (o & 0x7FFFFFFFu) : ~o);
}
constexpr uint64_t kMaskedKey = 0x00800000ull << 32;  // above it: more than -inf

// (z - m) / T of a row whose maximum is m; m of a row with every logit masked
// counts as 0.
__device__ __forceinline__ float base_of(float m) { return m == -INFINITY ? 0.0f : m; }

struct RowStats {
    float m, s, a;  // maximum, sum of exp(d), sum of exp(d) d, d = (z - m) / T
};

template <class T>
__device__ RowStats row_stats(const T *z, int vocab, float temperature, float *lds)
{
    float m = -INFINITY;
    for (int i = threadIdx.x; i < vocab; i += kNT)
        m = fmaxf(m, (float)z[i]);
    RowStats st;
    st.m = block_max<kNT>(m, lds);
    const float b = base_of(st.m);
    float s = 0.0f, a = 0.0f;
    for (int i = threadIdx.x; i < vocab; i += kNT) {
        const float d = ((float)z[i] - b) / temperature;
        const float e = expf(d);
        s += e;
        a += e == 0.0f ? 0.0f : e * d;
    }
    st.s = block_sum<kNT>(s, lds);
    st.a = block_sum<kNT>(a, lds);
    return st;
}

__device__ __forceinline__ float log_q(float z, const RowStats &st, float temperature)
{
    return st.s == 0.0f ? -INFINITY : (z - base_of(st.m)) / temperature - logf(st.s);
}

template <class T>
__global__ void __launch_bounds__(kNT)
k_logprobs(const T *logits, int64_t ld, int64_t rows, int vocab, float temperature,
           const int32_t *tokens, float *logprob, float *entropy, float *stats, int top_k,
           int32_t *top_ids, float *top_logprobs)
{
    __shared__ float lds[kNT / 64];
    __shared__ uint64_t best;
    for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
        const T *z = logits + r * ld;
        const RowStats st = row_stats(z, vocab, temperature, lds);
        const bool none = st.s != st.s;
        if (threadIdx.x == 0) {
            if (logprob) {
                const int t = tokens[r];
                logprob[r] = t < 0 ? 0.0f
                             : (t >= vocab || none) ? NAN
                                                    : log_q((float)z[t], st, temperature);
            }
            if (entropy)
                entropy[r] = st.s == 0.0f ? 0.0f : logf(st.s) - st.a / st.s;
            stats[2 * r] = st.m;
            stats[2 * r + 1] = st.s;
        }
        uint64_t below = ~0ull;
        for (int k = 0; k < top_k; ++k) {
            if (threadIdx.x == 0)
                best = 0;
            __syncthreads();
            uint64_t mine = 0;
            for (int i = threadIdx.x; i < vocab; i += kNT) {
                const uint64_t key = order_key((float)z[i], i);
                if (key < below && key > mine)
                    mine = key;
            }
            atomicMax((unsigned long long *)&best, (unsigned long long)mine);
            __syncthreads();
            below = best;
            __syncthreads();
            if (threadIdx.x == 0) {
                const bool have = below >= kMaskedKey && !none;
                top_ids[r * top_k + k] = have ? (int32_t)~(uint32_t)below : -1;
                top_logprobs[r * top_k + k] = none   ? NAN
                                              : have ? log_q(key_value(below), st, temperature)
                                                     : -INFINITY;
            }
        }
        __syncthreads();
    }
}

// A row's teacher, one alternative per lane of every wave: its id (-1: absent)
// and probability, their sum P, and sum p log p.
struct Teacher {
    int id;
    float p, logp, sum;
    bool bad, used;  // an id beyond the vocabulary; a present p other than 0
};
__device__ __forceinline__ Teacher teacher_row(const int32_t *ids, const float *lps, int64_t r,
                                               int top_k, int renormalize, int vocab)
{
    const int lane = threadIdx.x & 63;
    Teacher t;
    t.id = lane < top_k ? ids[r * top_k + lane] : -1;
    t.bad = __any(t.id >= vocab);
    t.logp = t.id >= 0 ? lps[r * top_k + lane] : -INFINITY;
    if (renormalize) {
        const float m = base_of(wave_max(t.logp));
        const float s = wave_sum(expf(t.logp - m));
        if (s != 0.0f)
            t.logp = t.logp - m - logf(s);
    }
    t.p = expf(t.logp);
    t.sum = wave_sum(t.p);
    t.used = __any(!(t.p == 0.0f));
    return t;
}

// dz of one row: w T (P q - p scattered), q = exp((z - m) / T) / S.
template <class T, class O>
__device__ void distill_gradient(const T *z, O *o, int vocab, float temperature, const Teacher &t,
                                 float w, float m, float s)
{
    const bool zero = w == 0.0f || (!t.used && !t.bad);
    // the logits at the alternatives, before anything is written (o may be z)
    const bool have = t.id >= 0 && t.id < vocab;
    const float zt = have ? (float)z[t.id] : 0.0f;
    __syncthreads();
    const float b = base_of(m), wt = w * temperature;
    auto prob = [&](float zi) { return s == 0.0f ? 0.0f : expf((zi - b) / temperature) / s; };
    for (int i = threadIdx.x; i < vocab; i += kNT)
        o[i] = (O)(zero ? 0.0f : t.bad ? NAN : wt * (t.sum * prob((float)z[i])));
    __syncthreads();
    if (zero || t.bad)
        return;
    // an id that comes twice: each of its lanes takes the sum and writes the same value
    float p = 0.0f;
    for (int j = 0; j < 64; ++j) {
        const int id = __shfl(t.id, j);
        const float pj = __shfl(t.p, j);
        p += id == t.id ? pj : 0.0f;
    }
    if (have && threadIdx.x < 64)
        o[t.id] = (O)(wt * (t.sum * prob(zt) - p));
}

// FORWARD: loss (and stats where stats is there); GRADIENT: dlogits, from
// stats where FORWARD is not asked for.
template <class T, class O, bool FORWARD, bool GRADIENT>
__global__ void __launch_bounds__(kNT)
k_distill(const T *logits, int64_t ld, int64_t rows, int vocab, float temperature,
          const int32_t *ids, const float *lps, int top_k, int renormalize, const float *weight,
          float *loss, float *stats, O *dlogits, int64_t ld_o)
{
    __shared__ float lds[kNT / 64];
    for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
        const T *z = logits + r * ld;
        const Teacher t = teacher_row(ids, lps, r, top_k, renormalize, vocab);
        const float w = weight ? weight[r] : 1.0f;
        RowStats st = {0.0f, 1.0f, 0.0f};
        if (FORWARD) {
            if (w != 0.0f)
                st = row_stats(z, vocab, temperature, lds);
            float term = 0.0f;
            if (t.id >= 0 && t.id < vocab && t.p != 0.0f)
                term = t.p * (t.logp - log_q((float)z[t.id], st, temperature));
            const float sum = wave_sum(term);
            if (threadIdx.x == 0) {
                const bool zero = w == 0.0f || (!t.used && !t.bad);
                loss[r] = zero ? 0.0f : t.bad ? NAN : w * (temperature * temperature * sum);
                if (stats) {
                    stats[2 * r] = st.m;
                    stats[2 * r + 1] = st.s;
                }
            }
        } else {
            st.m = stats[2 * r];
            st.s = stats[2 * r + 1];
        }
        if (GRADIENT)
            distill_gradient(z, dlogits + r * ld_o, vocab, temperature, t, w, st.m, st.s);
        __syncthreads();
    }
}

template <class T, class O>
__global__ void __launch_bounds__(kNT)
k_logprobs_bwd(const T *logits, int64_t ld, int64_t rows, int vocab, float temperature,
               const int32_t *tokens, const float *stats, const float *entropy,
               const float *d_logprob, const float *d_entropy, O *dlogits, int64_t ld_o)
{
    for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
        const T *z = logits + r * ld;
        O *o = dlogits + r * ld_o;
        const int token = d_logprob ? tokens[r] : -1;
        const float gl = token < 0 ? 0.0f : token >= vocab ? NAN : d_logprob[r];
        const float gh = d_entropy ? d_entropy[r] : 0.0f, h = d_entropy ? entropy[r] : 0.0f;
        const RowStats st = {stats[2 * r], stats[2 * r + 1], 0.0f};
        const float b = base_of(st.m), ls = logf(st.s);
        for (int i = threadIdx.x; i < vocab; i += kNT) {
            const float d = ((float)z[i] - b) / temperature;
            const float q = st.s == 0.0f ? 0.0f : expf(d) / st.s;
            const float lq = q == 0.0f ? 0.0f : d - ls + h;
            const float g = (i == token ? gl : 0.0f) - q * fmaf(gh, lq, gl);
            o[i] = (O)(g / temperature);
        }
    }
}

bool dtype_ok(int32_t d) { return d == MXQ_OUT_F32 || d == MXQ_OUT_BF16; }
bool aligned(const void *p, int32_t d)
{
    return reinterpret_cast<uintptr_t>(p) % (d == MXQ_OUT_F32 ? 4 : 2) == 0;
}
bool aligned4(const void *p) { return reinterpret_cast<uintptr_t>(p) % 4 == 0; }
unsigned row_grid(int64_t rows) { return (unsigned)(rows < kMaxGrid ? rows : kMaxGrid); }

template <class F> void with_type(int32_t d, F f)
{
    if (d == MXQ_OUT_F32)
        f((float *)nullptr);
    else
        f((bf16_t *)nullptr);
}

// The checks that every call shares: the logits and the temperature.
mxq_status check_logits(const void *logits, int32_t dtype, int64_t ld, int64_t rows, int64_t vocab,
                        float temperature)
{
    if (!dtype_ok(dtype) || !(temperature > 0.0f) || !(temperature < INFINITY))
        return MXQ_ERR_UNSUPPORTED;
    if (rows < 0 || vocab < 1 || vocab > INT32_MAX || ld < vocab)
        return MXQ_ERR_SHAPE;
    if (rows > 0 && !logits)
        return MXQ_ERR_NULL;
    return aligned(logits, dtype) ? MXQ_OK : MXQ_ERR_ALIGN;
}
mxq_status check_gradient(const void *dlogits, int32_t dtype, int64_t ld, int64_t rows,
                          int64_t vocab)
{
    if (!dtype_ok(dtype))
        return MXQ_ERR_UNSUPPORTED;
    if (ld < vocab)
        return MXQ_ERR_SHAPE;
    if (rows > 0 && !dlogits)
        return MXQ_ERR_NULL;
    return aligned(dlogits, dtype) ? MXQ_OK : MXQ_ERR_ALIGN;
}
mxq_status check_teacher(int64_t rows, const int32_t *ids, const float *lps, int32_t top_k,
                         int32_t renormalize, const float *weight)
{
    if (top_k < 1 || top_k > MXQ_TOP_MAX || (renormalize != 0 && renormalize != 1))
        return MXQ_ERR_UNSUPPORTED;
    if (rows > 0 && (!ids || !lps))
        return MXQ_ERR_NULL;
    return aligned4(ids) && aligned4(lps) && aligned4(weight) ? MXQ_OK : MXQ_ERR_ALIGN;
}

mxq_status launched() { return hipGetLastError() == hipSuccess ? MXQ_OK : MXQ_ERR_DEVICE; }

template <bool FORWARD, bool GRADIENT>
mxq_status launch_distill(const void *logits, int32_t dtype, int64_t ld, int64_t rows,
                          int64_t vocab, float temperature, const int32_t *ids, const float *lps,
                          int32_t top_k, int32_t renormalize, const float *weight, float *loss,
                          float *stats, void *dlogits, int32_t o_dtype, int64_t ld_o, void *stream)
{
    hipStream_t s = static_cast<hipStream_t>(stream);
    with_type(dtype, [&](auto *tt) {
        with_type(o_dtype, [&](auto *ot) {
            using T = std::remove_pointer_t<decltype(tt)>;
            using O = std::remove_pointer_t<decltype(ot)>;
            hipLaunchKernelGGL((k_distill<T, O, FORWARD, GRADIENT>), dim3(row_grid(rows)),
                               dim3(kNT), 0, s, static_cast<const T *>(logits), ld, rows,
                               (int)vocab, temperature, ids, lps, top_k, renormalize, weight, loss,
                               stats, static_cast<O *>(dlogits), ld_o);
        });
    });
    return launched();
}

}  // namespace

}  // namespace mxq

using namespace mxq;

extern "C" size_t mxq_vocab_workspace_size(int64_t rows, int64_t vocab, int32_t top_k)
{
    (void)rows;
    (void)vocab;
    (void)top_k;
    return 0;
}

extern "C" mxq_status mxq_token_logprobs(const void *logits, int32_t dtype, int64_t ld,
                                         int64_t rows, int64_t vocab, float temperature,
                                         const int32_t *tokens, float *logprob, float *entropy,
                                         float *stats, int32_t top_k, int32_t *top_ids,
                                         float *top_logprobs, void *workspace, size_t ws_bytes,
                                         void *stream)
{
    const mxq_status st = check_logits(logits, dtype, ld, rows, vocab, temperature);
    if (st)
        return st;
    if (top_k < 0 || top_k > MXQ_TOP_MAX)
        return MXQ_ERR_UNSUPPORTED;
    if (rows == 0)
        return MXQ_OK;
    if (!stats || (logprob && !tokens) || (top_k > 0 && (!top_ids || !top_logprobs)))
        return MXQ_ERR_NULL;
    if (!aligned4(tokens) || !aligned4(logprob) || !aligned4(entropy) || !aligned4(stats) ||
        !aligned4(top_ids) || !aligned4(top_logprobs) ||
        reinterpret_cast<uintptr_t>(workspace) % 8)
        return MXQ_ERR_ALIGN;
    const size_t need = mxq_vocab_workspace_size(rows, vocab, top_k);
    if (need > 0 && (!workspace || ws_bytes < need))
        return MXQ_ERR_WORKSPACE;
    hipStream_t s = static_cast<hipStream_t>(stream);
    with_type(dtype, [&](auto *tt) {
        using T = std::remove_pointer_t<decltype(tt)>;
        hipLaunchKernelGGL((k_logprobs<T>), dim3(row_grid(rows)), dim3(kNT), 0, s,
                           static_cast<const T *>(logits), ld, rows, (int)vocab, temperature,
                           tokens, logprob, entropy, stats, top_k, top_ids, top_logprobs);
    });
    return launched();
}

extern "C" mxq_status mxq_token_logprobs_backward(
    const void *logits, int32_t dtype, int64_t ld, int64_t rows, int64_t vocab, float temperature,
    const int32_t *tokens, const float *stats, const float *entropy, const float *d_logprob,
    const float *d_entropy, void *dlogits, int32_t dlogits_dtype, int64_t ld_dlogits, void *stream)
{
    mxq_status st = check_logits(logits, dtype, ld, rows, vocab, temperature);
    if (!st)
        st = check_gradient(dlogits, dlogits_dtype, ld_dlogits, rows, vocab);
    if (st || rows == 0)
        return st;
    if (!stats || (d_logprob && !tokens) || (d_entropy && !entropy))
        return MXQ_ERR_NULL;
    if (!aligned4(tokens) || !aligned4(stats) || !aligned4(entropy) || !aligned4(d_logprob) ||
        !aligned4(d_entropy))
        return MXQ_ERR_ALIGN;
    hipStream_t s = static_cast<hipStream_t>(stream);
    with_type(dtype, [&](auto *tt) {
        with_type(dlogits_dtype, [&](auto *ot) {
            using T = std::remove_pointer_t<decltype(tt)>;
            using O = std::remove_pointer_t<decltype(ot)>;
            hipLaunchKernelGGL((k_logprobs_bwd<T, O>), dim3(row_grid(rows)), dim3(kNT), 0, s,
                               static_cast<const T *>(logits), ld, rows, (int)vocab, temperature,
                               tokens, stats, entropy, d_logprob, d_entropy,
                               static_cast<O *>(dlogits), ld_dlogits);
        });
    });
    return launched();
}

extern "C" mxq_status mxq_distill_forward(const void *logits, int32_t dtype, int64_t ld,
                                          int64_t rows, int64_t vocab, float temperature,
                                          const int32_t *teacher_ids,
                                          const float *teacher_logprobs, int32_t top_k,
                                          int32_t renormalize, const float *weight, float *loss,
                                          float *stats, void *workspace, size_t ws_bytes,
                                          void *stream)
{
    mxq_status st = check_logits(logits, dtype, ld, rows, vocab, temperature);
    if (!st)
        st = check_teacher(rows, teacher_ids, teacher_logprobs, top_k, renormalize, weight);
    if (st || rows == 0)
        return st;
    if (!loss || !stats)
        return MXQ_ERR_NULL;
    if (!aligned4(loss) || !aligned4(stats) || reinterpret_cast<uintptr_t>(workspace) % 8)
        return MXQ_ERR_ALIGN;
    const size_t need = mxq_vocab_workspace_size(rows, vocab, 0);
    if (need > 0 && (!workspace || ws_bytes < need))
        return MXQ_ERR_WORKSPACE;
    return launch_distill<true, false>(logits, dtype, ld, rows, vocab, temperature, teacher_ids,
                                       teacher_logprobs, top_k, renormalize, weight, loss, stats,
                                       nullptr, MXQ_OUT_F32, 0, stream);
}

extern "C" mxq_status mxq_distill_backward(const void *logits, int32_t dtype, int64_t ld,
                                           int64_t rows, int64_t vocab, float temperature,
                                           const int32_t *teacher_ids,
                                           const float *teacher_logprobs, int32_t top_k,
                                           int32_t renormalize, const float *weight,
                                           const float *stats, void *dlogits,
                                           int32_t dlogits_dtype, int64_t ld_dlogits, void *stream)
{
    mxq_status st = check_logits(logits, dtype, ld, rows, vocab, temperature);
    if (!st)
        st = check_gradient(dlogits, dlogits_dtype, ld_dlogits, rows, vocab);
    if (!st)
        st = check_teacher(rows, teacher_ids, teacher_logprobs, top_k, renormalize, weight);
    if (st || rows == 0)
        return st;
    if (!stats)
        return MXQ_ERR_NULL;
    if (!aligned4(stats))
        return MXQ_ERR_ALIGN;
    return launch_distill<false, true>(logits, dtype, ld, rows, vocab, temperature, teacher_ids,
                                       teacher_logprobs, top_k, renormalize, weight, nullptr,
                                       const_cast<float *>(stats), dlogits, dlogits_dtype,
                                       ld_dlogits, stream);
}

extern "C" mxq_status mxq_distill(const void *logits, int32_t dtype, int64_t ld, int64_t rows,
                                  int64_t vocab, float temperature, const int32_t *teacher_ids,
                                  const float *teacher_logprobs, int32_t top_k,
                                  int32_t renormalize, const float *weight, float *loss,
                                  void *dlogits, int32_t dlogits_dtype, int64_t ld_dlogits,
                                  void *workspace, size_t ws_bytes, void *stream)
{
    mxq_status st = check_logits(logits, dtype, ld, rows, vocab, temperature);
    if (!st)
        st = check_gradient(dlogits, dlogits_dtype, ld_dlogits, rows, vocab);
    if (!st)
        st = check_teacher(rows, teacher_ids, teacher_logprobs, top_k, renormalize, weight);
    if (st || rows == 0)
        return st;
    if (!loss)
        return MXQ_ERR_NULL;
    if (!aligned4(loss) || reinterpret_cast<uintptr_t>(workspace) % 8)
        return MXQ_ERR_ALIGN;
    const size_t need = mxq_vocab_workspace_size(rows, vocab, 0);
    if (need > 0 && (!workspace || ws_bytes < need))
        return MXQ_ERR_WORKSPACE;
    return launch_distill<true, true>(logits, dtype, ld, rows, vocab, temperature, teacher_ids,
                                      teacher_logprobs, top_k, renormalize, weight, loss, nullptr,
                                      dlogits, dlogits_dtype, ld_dlogits, stream);
}
