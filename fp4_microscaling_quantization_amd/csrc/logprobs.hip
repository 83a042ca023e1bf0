// Token log probabilities with entropy and top alternatives
// (mxq_token_logprobs; include/mxq.h holds the formulas; the gradient is in
// distill.hip).
//
// One workgroup per row, which holds the row in registers a stretch at a time:
// the logits come from memory once, and the search for the alternatives goes
// over registers.
#include "vocab.hpp"

namespace mxq {

namespace {

// ---- the order of the alternatives ---------------------------------------------------
// Larger keys come first: the logit's value (-0 as 0), then the index, the lower
// one first.  Keys of a row are unique.  0 is below every key.
__device__ __forceinline__ uint32_t order_of(float z)
{
    const uint32_t u = as_u(z + 0.0f);
    return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ uint64_t key_of(float z, int i)
{
    return ((uint64_t)order_of(z) << 32) | (uint32_t)~i;
}
__device__ __forceinline__ float key_value(uint64_t k)
{
    const uint32_t o = (uint32_t)(k >> 32);
    return as_f((o >> 31) ? (o & 0x7FFFFFFFu) : ~o);
}
__device__ __forceinline__ int key_index(uint64_t k) { return (int)~(uint32_t)k; }
// the keys of the logits above -inf (whose order is 0x007FFFFF)
constexpr uint64_t kLeastKey = 0x00800000ull << 32;

template <int X> __device__ __forceinline__ uint64_t key_xor(uint64_t k)
{
    uint32_t lo = (uint32_t)k, hi = (uint32_t)(k >> 32);
    if constexpr (X < 16) {
        lo = lane_xor<X>(lo);
        hi = lane_xor<X>(hi);
    } else {
        lo = (uint32_t)__shfl_xor((int)lo, X);
        hi = (uint32_t)__shfl_xor((int)hi, X);
    }
    return ((uint64_t)hi << 32) | lo;
}
// one step of a bitonic network: lanes X apart, the larger key to the lower lane
// where `falling`
template <int X> __device__ __forceinline__ uint64_t order_step(uint64_t k, bool falling)
{
    const uint64_t other = key_xor<X>(k);
    const bool lower = (threadIdx.x & X) == 0;
    return (k > other) == (lower == falling) ? k : other;
}
template <int X> __device__ __forceinline__ uint64_t order_steps(uint64_t k, bool falling)
{
    k = order_step<X>(k, falling);
    if constexpr (X > 1)
        k = order_steps<X / 2>(k, falling);
    return k;
}
// a wave's 64 keys in falling order
__device__ __forceinline__ uint64_t wave_sort(uint64_t k)
{
    const int lane = threadIdx.x & 63;
    k = order_steps<1>(k, (lane & 2) == 0);
    k = order_steps<2>(k, (lane & 4) == 0);
    k = order_steps<4>(k, (lane & 8) == 0);
    k = order_steps<8>(k, (lane & 16) == 0);
    k = order_steps<16>(k, (lane & 32) == 0);
    return order_steps<32>(k, true);
}
// the first 64 of two falling lists, in falling order; the second one is given
// turned round (lane l has its 63 - l th), so the larger of each pair are the
// first 64 and rise and fall once
__device__ __forceinline__ uint64_t wave_merge(uint64_t a, uint64_t b_turned)
{
    return order_steps<32>(a > b_turned ? a : b_turned, true);
}

// The first 64 of the workgroup's NT keys, in falling order, in the lanes of every
// wave.  lds: NT keys.
template <int NT> __device__ __forceinline__ uint64_t block_top(uint64_t k, uint64_t *lds)
{
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    k = wave_sort(k);
    __syncthreads();
#pragma unroll
    for (int half = NT / 128; half >= 1; half /= 2) {
        if (w >= half && w < 2 * half)
            lds[threadIdx.x] = k;
        __syncthreads();
        if (w < half)
            k = wave_merge(k, lds[(w + half) * 64 + 63 - lane]);
    }
    if (w == 0)
        lds[lane] = k;
    __syncthreads();
    return lds[lane];
}

// The first top_k alternatives of the held stretch (n logits, the first of them
// entry `at` of the row) and of the list `best` from before it, as a list again.
//
// A bound that top_k alternatives reach is known at once: the top_k th of the
// threads' maxima over the row so far (`most`; a thread without an alternative has
// the lowest finite value, which bounds nothing).  What reaches it goes to a buffer of NT keys; random rows have
// hardly more than top_k such entries.  Where the buffer is too small (many equal
// logits, or the large ones all in a few threads), the top_k th of what it holds is a
// higher bound, and the search goes again, until it is not.  Every entry of the
// buffer is an alternative of the row, so each bound leaves top_k above it.
template <class T, int NT>
__device__ __forceinline__ uint64_t top_held(uint64_t best, Held<T, NT, kHeld> &held, int at, int n,
                                             float most, int top_k, uint64_t *lds,
                                             uint64_t *buffer, int *count)
{
    constexpr int E = kElems<T>;
    const int lane = threadIdx.x & 63;
    auto kth = [&](uint64_t list) {
        const uint64_t k = (uint64_t)__shfl((unsigned long long)list, top_k - 1);
        return k > kLeastKey ? k : kLeastKey;
    };
    uint64_t bound = kth(block_top<NT>((uint64_t)order_of(most) << 32, lds));
    const uint64_t before = kth(best);
    bound = bound > before ? bound : before;
    for (;;) {
        // the list so far is in the buffer from the start
        if (threadIdx.x < 64)
            buffer[threadIdx.x] = best;
        if (threadIdx.x == 0)
            *count = 64;
        held.again();
        int mine = at + held.at(0);  // opaque, or the indices of all entries are kept in registers
        asm volatile("" : "+v"(mine));
        __syncthreads();
        const float least = key_value(bound);
        const int n2 = fresh(n);
        if (__any(most >= least)) {
#pragma unroll
            for (int i = 0; i < kHeld; ++i) {
                if (!held.any(i, n2))
                    continue;
                float f[E];
                held.get(i, f);
                float m = f[0];
#pragma unroll
                for (int j = 1; j < E; ++j)
                    m = fmaxf(m, f[j]);
                if (!__any(m >= least))
                    continue;
#pragma unroll
                for (int j = 0; j < E; ++j) {
                    const uint64_t key = key_of(f[j], mine + i * NT * E + j);
                    const bool in = f[j] >= least && key >= bound;
                    const uint64_t mask = __ballot(in);
                    if (mask == 0)
                        continue;
                    // one atomic for the wave's lanes
                    const int leader = __ffsll((unsigned long long)mask) - 1;
                    int to = 0;
                    if (lane == leader)
                        to = atomicAdd(count, __popcll(mask));
                    to = __shfl(to, leader) + __popcll(mask & ((1ull << lane) - 1));
                    if (in && to < NT)
                        buffer[to] = key;
                }
            }
        }
        __syncthreads();
        const int have = *count;
        const uint64_t list = block_top<NT>((int)threadIdx.x < have ? buffer[threadIdx.x] : 0, lds);
        if (have <= NT)
            return list;
        bound = kth(list);
        __syncthreads();
    }
}

// ---- the kernels -----------------------------------------------------------------------

struct LogprobOut {
    const int32_t *tokens;
    float *logprob, *entropy, *stats;
    int32_t top_k;
    int32_t *top_ids;
    float *top_logprobs;
};

// what a row's outputs are, from its statistics and list; called by one wave
template <class T>
__device__ __forceinline__ void write_row(const LogprobOut &out, const T *z, int64_t r, int vocab,
                                          const RowStats &st, uint64_t list, const Heat &heat)
{
    const int lane = threadIdx.x & 63;
    const bool none = st.s != st.s;
    if (lane == 0) {
        out.stats[2 * r] = st.m;
        out.stats[2 * r + 1] = st.s;
        if (out.logprob) {
            const int t = out.tokens[r];
            out.logprob[r] = t < 0                  ? 0.0f
                             : (t >= vocab || none) ? NAN
                                                    : log_q(load_one(z + t), st, heat);
        }
        if (out.entropy)
            out.entropy[r] = st.s == 0.0f ? 0.0f : logf(st.s) - 0.69314718055994531f * (st.a / st.s);
    }
    if (lane < out.top_k) {
        const bool have = list >= kLeastKey && !none;
        out.top_ids[r * out.top_k + lane] = have ? key_index(list) : -1;
        out.top_logprobs[r * out.top_k + lane] = none   ? NAN
                                                 : have ? log_q(key_value(list), st, heat)
                                                        : -INFINITY;
    }
}

template <class T, int NT, bool TOP>
__global__ void __launch_bounds__(NT, 4)
k_logprobs(const T *logits, int64_t ld, int64_t rows, int vocab, Heat heat, LogprobOut out)
{
    using H = Held<T, NT, kHeld>;
    __shared__ float lds[3 * NT / 64];
    __shared__ uint64_t keys[TOP ? NT : 1], buffer[TOP ? NT : 1];
    __shared__ int count;
    for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
        const T *z = logits + r * ld;
        H held;
        RowStats st = {-FLT_MAX, 0.0f, 0.0f};
        uint64_t list = 0;
        for (int at = 0;;) {
            const int n = min(vocab - at, H::kMost);
            held.load(z + at, fresh(n), kMaskedBits<T>);
            absorb_held<true>(st, held, n, heat.log2);
            if (TOP)
                list = top_held(list, held, at, n, st.m, out.top_k, keys, buffer, &count);
            if (vocab - at <= H::kMost)
                break;
            at += H::kMost;
        }
        st = block_stats<NT>(st, heat.log2, lds);
        if (threadIdx.x < 64)
            write_row(out, z, r, vocab, st, list, heat);
        __syncthreads();
    }
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
    const LogprobOut out = {tokens, logprob, entropy, stats, top_k, top_ids, top_logprobs};
    hipStream_t s = static_cast<hipStream_t>(stream);
    with_type(dtype, [&](auto *tt) {
        using T = std::remove_pointer_t<decltype(tt)>;
        with_threads<T>(vocab, [&](auto nt) {
            constexpr int NT = decltype(nt)::value;
            const auto *z = static_cast<const T *>(logits);
            if (top_k > 0)
                hipLaunchKernelGGL((k_logprobs<T, NT, true>), dim3(row_grid(rows)), dim3(NT), 0, s,
                                   z, ld, rows, (int)vocab, heat_of(temperature), out);
            else
                hipLaunchKernelGGL((k_logprobs<T, NT, false>), dim3(row_grid(rows)), dim3(NT), 0,
                                   s, z, ld, rows, (int)vocab, heat_of(temperature), out);
        });
    });
    return launched();
}
