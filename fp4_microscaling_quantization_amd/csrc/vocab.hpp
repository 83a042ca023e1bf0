// What the operators over a vocabulary share (token log probabilities,
// distillation): the softmax statistics of a row, and the host's checks.
#pragma once

#include <float.h>

#include "mxq_host.hpp"
#include "rows.hpp"

namespace mxq {

// Vectors of 16 bytes that a thread holds of a row.  With the widest workgroup
// (1024 threads) that is 256 KB, half of a CU's registers: 131072 bf16 or 65536
// fp32 logits.  Longer rows take several stretches.
constexpr int kHeld = 16;
// They are taken in groups of 16 elements.
template <class T> constexpr int kGroup = 16 / kElems<T>;
template <class T> constexpr int kGroups = kHeld / kGroup<T>;

// What the kernels take of the temperature: 1 / T and log2(e) / T.
struct Heat {
    float t, inv, log2;
};

// (z - m) / T for a row's maximum m; m of a row with every logit masked counts
// as 0, so that the differences are -inf and not NaN.
__device__ __forceinline__ float base_of(float m) { return m == -INFINITY ? 0.0f : m; }

// Softmax statistics: the maximum m, s = sum exp(d), a = sum exp(d) d with
// d = (z - m) / T in units of log2 (2^d = exp).  One pass: a thread's m starts
// at the lowest finite value, and s and a move to a new maximum as it comes.
// The difference is taken before the product with log2(e) / T: the product of
// the lowest finite value would be -inf, a row of such values has to be uniform.
struct RowStats {
    float m, s, a;
};
constexpr float kFloorLog2 = -256.0f;  // 2^d is 0 far above it: d stays finite in a

// s and a of a state, seen from a maximum `to` >= its own.  Far below it (2^-256
// is 0 in fp32) they are 0; NaN stays NaN.
__device__ __forceinline__ void move_to(RowStats &st, float to, float log2)
{
    const float d = fmaxf((st.m - to) * log2, kFloorLog2);
    const float e = __builtin_amdgcn_exp2f(d);
    st.a = e * fmaf(st.s, d, st.a);
    st.s *= e;
    st.m = to;
}

// takes the values in; half: the maxima of their two halves
template <bool ENTROPY, int N>
__device__ __forceinline__ void absorb(RowStats &st, const float (&f)[N], float log2,
                                       float (&half)[2])
{
    half[0] = f[0];
    half[1] = f[N / 2];
#pragma unroll
    for (int j = 1; j < N / 2; ++j) {
        half[0] = fmaxf(half[0], f[j]);
        half[1] = fmaxf(half[1], f[N / 2 + j]);
    }
    const float m = fmaxf(st.m, fmaxf(half[0], half[1]));
    const float d = fmaxf((st.m - m) * log2, kFloorLog2);
    const float sc = __builtin_amdgcn_exp2f(d);
    if (ENTROPY)
        st.a = sc * fmaf(st.s, d, st.a);
    float s = 0.0f, a = 0.0f;
#pragma unroll
    for (int j = 0; j < N; ++j) {
        const float dj = (f[j] - m) * log2;
        const float e = __builtin_amdgcn_exp2f(dj);
        s += e;
        if (ENTROPY)
            a = fmaf(e, fmaxf(dj, kFloorLog2), a);
    }
    st.s = fmaf(st.s, sc, s);
    if (ENTROPY)
        st.a += a;
    st.m = m;
}

// The statistics of a held stretch of n elements into the threads' own states, 16
// elements at a time: what a step costs beside its exponentials is shared by them.
// most: the maxima of the thread's groups, half: those of the groups' first and second
// halves.  lead: what of the stretch lies before the row.
template <bool ENTROPY, class T, int NT>
__device__ __forceinline__ void absorb_held(RowStats &st, const Held<T, NT, kHeld> &h, int n,
                                            int lead, float log2, float (&most)[kGroups<T>],
                                            float (&half)[2])
{
    constexpr int E = kElems<T>, G = kGroup<T>;
    n = fresh(n);
    half[0] = half[1] = -INFINITY;
#pragma unroll
    for (int i = 0; i < kHeld; i += G) {
        most[i / G] = -INFINITY;
        if (h.any(i, n)) {
            float f[16];
#pragma unroll
            for (int g = 0; g < G; ++g) {
                float part[E];
                h.get(i + g, n, -INFINITY, part, lead);
#pragma unroll
                for (int j = 0; j < E; ++j)
                    f[g * E + j] = part[j];
            }
            float h2[2];
            absorb<ENTROPY>(st, f, log2, h2);
            most[i / G] = fmaxf(h2[0], h2[1]);
            half[0] = fmaxf(half[0], h2[0]);
            half[1] = fmaxf(half[1], h2[1]);
        }
    }
}

// The workgroup's statistics from its threads', in every thread, joined in a
// fixed order; m is -inf where s is 0.  lds: 3 NT / 64 floats.
template <int NT>
__device__ __forceinline__ RowStats block_stats(RowStats st, float log2, float *lds)
{
    constexpr int W = NT / 64;
    move_to(st, wave_max(st.m), log2);
    st.s = wave_sum(st.s);
    st.a = wave_sum(st.a);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) {
        const int w = threadIdx.x >> 6;
        lds[w] = st.m;
        lds[W + w] = st.s;
        lds[2 * W + w] = st.a;
    }
    __syncthreads();
    float m = lds[0];
#pragma unroll
    for (int w = 1; w < W; ++w)
        m = fmaxf(m, lds[w]);
    RowStats all = {m, 0.0f, 0.0f};
#pragma unroll
    for (int w = 0; w < W; ++w) {
        RowStats one = {lds[w], lds[W + w], lds[2 * W + w]};
        move_to(one, m, log2);
        all.s += one.s;
        all.a += one.a;
    }
    if (all.s == 0.0f)
        all.m = -INFINITY;
    return all;
}

// The same over a wave's lanes.
__device__ __forceinline__ RowStats wave_stats(RowStats st, float log2)
{
    move_to(st, wave_max(st.m), log2);
    st.s = wave_sum(st.s);
    st.a = wave_sum(st.a);
    if (st.s == 0.0f)
        st.m = -INFINITY;
    return st;
}

// log q of a logit; -inf throughout a row with every logit masked
__device__ __forceinline__ float log_q(float z, const RowStats &st, const Heat &h)
{
    return st.s == 0.0f ? -INFINITY : (z - base_of(st.m)) * h.inv - logf(st.s);
}

// ---- few rows ----------------------------------------------------------------------
// A workgroup per row leaves the chip empty when there are few; then several take a
// part of the row each, and a second launch joins them.  The workspace holds the
// parts' alternatives, then their m, s and a, each [rows][parts].
constexpr int kMaxParts = 64;  // a wave joins them
struct Parts {
    int count, length;  // parts of a row, logits of a part
    uint64_t *keys;     // [rows][count][top_k]
    float *stats;       // [3][rows][count]
};

// the row's statistics from its parts', in every lane
__device__ __forceinline__ RowStats part_stats(const Parts &p, int64_t rows, int64_t r, float log2)
{
    const int lane = threadIdx.x & 63;
    const float *f = p.stats + r * p.count + lane;
    const int64_t all = rows * p.count;
    RowStats st = {-FLT_MAX, 0.0f, 0.0f};
    // a part with every logit masked has m = -inf, and must stay at s = 0
    if (lane < p.count)
        st = {fmaxf(f[0], -FLT_MAX), f[all], f[2 * all]};
    return wave_stats(st, log2);
}

// ---- the host's side -------------------------------------------------------------

constexpr int64_t kMaxVocab = INT32_MAX - 63;  // an index and a shift to a boundary fit 32 bits

inline unsigned row_grid(int64_t rows) { return (unsigned)(rows < kMaxGrid ? rows : kMaxGrid); }
// Parts so that about 1024 workgroups of 256 threads run, four on a CU; a part has 4096
// logits at least, below that a workgroup's time is not its loads'.  A second launch and
// a second search have to pay: 16 x 128256 bf16, 20 alternatives, 17.4 us against 31 in
// one launch, 16 x 32000 17.7 against 13.3, 900 x 128256 60 against 58.
inline Parts parts_of(int64_t rows, int64_t vocab, int32_t top_k, void *workspace)
{
    int64_t want = rows > 512 || vocab < 49152 ? 1 : (1024 + rows - 1) / rows;
    want = want < vocab / 4096 ? want : vocab / 4096;
    want = want < kMaxParts ? want : kMaxParts;
    Parts p = {1, (int)vocab, nullptr, nullptr};
    if (want > 1) {
        p.length = (int)(((vocab + want - 1) / want + 15) / 16 * 16);
        p.count = (int)((vocab + p.length - 1) / p.length);
        p.keys = static_cast<uint64_t *>(workspace);
        p.stats = reinterpret_cast<float *>(p.keys + rows * p.count * top_k);
    }
    return p;
}
// The statistics (and the first top_k alternatives) of all parts of all rows; dtype and
// sizes were checked.
void launch_parts(const void *logits, int32_t dtype, int64_t ld, int64_t rows, int64_t vocab,
                  const Heat &heat, int32_t top_k, const Parts &parts, hipStream_t s);

inline Heat heat_of(float t)
{
    return {t, (float)(1.0 / (double)t), (float)(1.4426950408889634 / (double)t)};
}
inline bool dtype_ok(int32_t d) { return d == MXQ_OUT_F32 || d == MXQ_OUT_BF16; }
inline bool aligned(const void *p, int32_t d)
{
    return reinterpret_cast<uintptr_t>(p) % (d == MXQ_OUT_F32 ? 4 : 2) == 0;
}
inline bool aligned4(const void *p) { return reinterpret_cast<uintptr_t>(p) % 4 == 0; }
inline mxq_status launched() { return hipGetLastError() == hipSuccess ? MXQ_OK : MXQ_ERR_DEVICE; }

// f(null pointer of the element type) for a dtype code that was checked
template <class F> void with_type(int32_t d, F f)
{
    if (d == MXQ_OUT_F32)
        f((float *)nullptr);
    else
        f((bf16_t *)nullptr);
}

// f(integral constants: threads of a workgroup, whether the row is shorter than a
// vector) for rows of n elements of T: the fewest threads that hold a row from a
// boundary on, so that rows share a CU, up to `MOST`.  A wave a row only where there are
// enough rows to fill the chip with waves: log probabilities of 8192 x 1000 bf16 17 us
// against 48 with 256 threads, but of 1024 x 8000 14.3 against 12.7.  With 256, 512 and 1024
// threads where 256 hold the row: distillation of 4096 x 32000 bf16 102, 105 and 142 us, 4096 x
// 16000 59, 76 and 121, 600 x 32000 21.0, 22.0 and 27.6, but 64 x 32000 10.7, 8.8 and 9.3; with 512
// and 1024, 4096 x 64000 186 and 213.  What is only read takes 256 at any length (MOST): log
// probabilities with 32 alternatives of 2048 x 128256 bf16 114, 122 and 136 us, 2048 x 32000 37, 44
// and 71, without 25.5, 26.5 and 43, but 2048 x 64000 without 48.5, 44 and 61, 64 x 32000 with 32
// 12.6, 10.4 and 9.6.
constexpr int64_t kWaveRows = 2048;
template <class T, int MOST, class F> void with_threads(int64_t rows, int64_t n, F f)
{
    constexpr int64_t one = 64 * kHeld * kElems<T>;  // what a wave holds
    constexpr std::false_type whole;
    const int64_t most = n + kElems<T> - 1;
    if (n < kElems<T>)
        f(std::integral_constant<int, 64>(), std::true_type());
    else if (most <= one && rows >= kWaveRows)
        f(std::integral_constant<int, 64>(), whole);
    else if (MOST == 256 || most <= 4 * one)
        f(std::integral_constant<int, 256>(), whole);
    else if (most <= 8 * one)
        f(std::integral_constant<int, MOST < 512 ? 256 : 512>(), whole);
    else
        f(std::integral_constant<int, MOST>(), whole);
}

// The checks that every call over a vocabulary shares: the logits and the
// temperature (1 / temperature has to be finite).
inline mxq_status check_logits(const void *logits, int32_t dtype, int64_t ld, int64_t rows,
                               int64_t vocab, float temperature)
{
    if (!dtype_ok(dtype) || !(temperature >= FLT_MIN) || !(temperature < INFINITY))
        return MXQ_ERR_UNSUPPORTED;
    if (rows < 0 || vocab < 1 || vocab > kMaxVocab || ld < vocab)
        return MXQ_ERR_SHAPE;
    if (rows > 0 && !logits)
        return MXQ_ERR_NULL;
    return aligned(logits, dtype) ? MXQ_OK : MXQ_ERR_ALIGN;
}
inline mxq_status check_gradient(const void *dlogits, int32_t dtype, int64_t ld, int64_t rows,
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

}  // namespace mxq
