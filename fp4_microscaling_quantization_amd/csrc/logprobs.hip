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
// one step of a bitonic network: lanes X apart, the larger one to the lower lane where
// `falling`; for keys and for values
template <int X> __device__ __forceinline__ uint64_t order_step(uint64_t k, bool falling)
{
    const uint64_t other = key_xor<X>(k);
    const bool lower = (threadIdx.x & X) == 0;
    return (k > other) == (lower == falling) ? k : other;
}
template <int X> __device__ __forceinline__ uint32_t order_step(uint32_t v, bool falling)
{
    uint32_t other;
    if constexpr (X < 16)
        other = lane_xor<X>(v);
    else
        other = (uint32_t)__shfl_xor((int)v, X);
    const bool lower = (threadIdx.x & X) == 0;
    return lower == falling ? max(v, other) : min(v, other);
}
template <int X, class K> __device__ __forceinline__ K order_steps(K k, bool falling)
{
    k = order_step<X>(k, falling);
    if constexpr (X > 1)
        k = order_steps<X / 2>(k, falling);
    return k;
}
// a wave's 64 keys or values in falling order
template <class K> __device__ __forceinline__ K wave_sort(K k)
{
    const int lane = threadIdx.x & 63;
    k = order_steps<1>(k, (lane & 2) == 0);
    k = order_steps<2>(k, (lane & 4) == 0);
    k = order_steps<4>(k, (lane & 8) == 0);
    k = order_steps<8>(k, (lane & 16) == 0);
    k = order_steps<16>(k, (lane & 32) == 0);
    return order_steps<32>(k, true);
}
__device__ __forceinline__ uint64_t turned(uint64_t k)
{
    return (uint64_t)__shfl((unsigned long long)k, 63 - (threadIdx.x & 63));
}
__device__ __forceinline__ uint32_t turned(uint32_t v)
{
    return (uint32_t)__shfl((int)v, 63 - (threadIdx.x & 63));
}
// the first 64 of two falling lists, in falling order: with one turned round, the
// larger of each pair are the first 64, and rise and fall once
template <class K> __device__ __forceinline__ K wave_merge(K a, K b)
{
    b = turned(b);
    return order_steps<32>(a > b ? a : b, true);
}

// What the search for the alternatives keeps in LDS.
constexpr int kBuffer = 512, kPlaces = 128;
struct Search {
    uint64_t buffer[kBuffer];
    uint64_t bound;
    uint32_t most[kPlaces];
    int count;
};

// the first 64 of the falling list `list` and of n keys in LDS, by one wave
__device__ __forceinline__ uint64_t list_of(uint64_t list, const uint64_t *keys, int n)
{
    const int lane = threadIdx.x & 63;
    for (int at = 0; at < n; at += 64) {
        const uint64_t k = wave_sort(at + lane < n ? keys[at + lane] : (uint64_t)0);
        list = __all(list == 0) ? k : wave_merge(list, k);
    }
    return list;
}

// The first top_k alternatives of the held stretch (n logits, the first of them entry
// `at` of the row, or `lead` before it) and of wave 0's list from before it, as wave 0's list.  most: the
// thread's maxima of its groups of 16, top: its maximum over the row so far (the lowest
// finite value where it has none).
//
// A bound that top_k alternatives reach is known at once: the threads' maxima go into
// 128 (64) places, the largest of each stays, and the top_k th of those is the bound
// (one wave: the places are its lanes' maxima, for over 32 alternatives of two halves
// of what they hold); twice as many places as alternatives keep it close (a random row has about
// 1.4 top_k logits that reach it).  Each wave goes over its registers, the groups whose
// maximum reaches the bound, and puts what it finds into a buffer, which wave 0
// sorts.  Where the buffer is too small (many equal logits, or the large ones all in a
// few threads), the top_k th of what it holds is a higher bound, and the search goes
// again, until it is not: every key of the buffer is an alternative of the row.
// Measured beside it (1501 x 50257 fp32, 64 alternatives, 73 us): listing the groups
// and reading them again with all lanes, 80 us, as the reads queue behind the other
// workgroups' streams; ordering by counting larger keys with all waves, 106 us.  Keys of
// several stretches sorted at once, 2% faster here and 3% on 2048 x 128256 bf16, but 2 to
// 4% slower on rows of eight stretches (1024 x 128256 fp32), where the list's own last key
// is the closer bound.
template <class T, int NT>
__device__ __forceinline__ uint64_t top_held(uint64_t list, Held<T, NT, kHeld> &held, int at, int n, int lead,
                                             const float (&most)[kGroups<T>],
                                             const float (&half)[2], float top, int top_k,
                                             Search &lds)
{
    constexpr int E = kElems<T>, G = kGroup<T>;
    const int lane = threadIdx.x & 63, places = top_k > 32 ? kPlaces : kPlaces / 2;
    const auto kth = [&](uint64_t l) {
        const uint64_t k = (uint64_t)__shfl((unsigned long long)l, top_k - 1);
        return k > kLeastKey ? k : kLeastKey;
    };
    const auto start = [&](uint32_t sorted) {
        const uint64_t k = kth((uint64_t)sorted << 32), before = kth(list);
        if (lane == 0) {
            lds.bound = k > before ? k : before;
            lds.count = 0;
        }
    };
    if constexpr (NT == 64) {
        // a wave has its row in one stretch
        if (top_k > 32)
            start(wave_merge(wave_sort(order_of(half[0])), wave_sort(order_of(half[1]))));
        else
            start(wave_sort(order_of(top)));
    } else {
        if (threadIdx.x < kPlaces)
            lds.most[threadIdx.x] = 0;
        __syncthreads();
        atomicMax(&lds.most[threadIdx.x & (places - 1)], order_of(top));
        __syncthreads();
        if (threadIdx.x < 64) {
            const uint32_t v = wave_sort(lds.most[lane]);
            start(places == kPlaces ? wave_merge(v, wave_sort(lds.most[64 + lane])) : v);
        }
    }
    __syncthreads();
    for (;;) {
        const uint64_t bound = lds.bound;
        const float least = key_value(bound);
        held.again();
        const int n2 = fresh(n);
        int mine = at + held.at(0);  // opaque, or the indices of all entries are kept in registers
        asm volatile("" : "+v"(mine));
#pragma unroll
        for (int i = 0; i < kHeld; i += G) {
            if (!__any(most[i / G] >= least))
                continue;
#pragma unroll
            for (int k = i; k < i + G; ++k) {
                float f[E];
                held.get(k, n2, -INFINITY, f, lead);
                const int back = held.whole(k, n2) ? 0 : held.skip(k, n2);
#pragma unroll
                for (int j = 0; j < E; ++j) {
                    if (f[j] >= least) {
                        const uint64_t key = key_of(f[j], mine - back + k * NT * E + j);
                        if (key >= bound) {
                            const int to = atomicAdd(&lds.count, 1);
                            if (to < kBuffer)
                                lds.buffer[to] = key;
                        }
                    }
                }
            }
        }
        __syncthreads();
        const int have = lds.count;
        if (have <= kBuffer)
            return threadIdx.x < 64 ? list_of(list, lds.buffer, have) : 0;
        __syncthreads();
        if (threadIdx.x < 64) {
            const uint64_t k = kth(list_of(list, lds.buffer, kBuffer));
            if (lane == 0) {
                lds.bound = k;
                lds.count = 0;
            }
        }
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

// The statistics of n logits at z, entry `first` of their row the first, and wave 0's list
// of their alternatives.
template <class T, int NT, bool TOP, bool SHORT, class S>
__device__ __forceinline__ RowStats whole_part(const T *z, int first, int n, int top_k,
                                               const Heat &heat, float *lds, S &search,
                                               uint64_t &list)
{
    using H = Held<T, NT, kHeld>;
    RowStats st = {-FLT_MAX, 0.0f, 0.0f};
    list = 0;
    int lead = lead_of<T, SHORT>(z);
    z -= lead;
    n += lead;
    first -= lead;
    for (int at = 0;;) {
        const int here = min(n - at, H::kMost);
        H held;
        held.template load<SHORT, true>(z + at, here);
        float most[kGroups<T>], half[2];
        absorb_held<true>(st, held, here, lead, heat.log2, most, half);
        if constexpr (TOP)
            list = top_held(list, held, first + at, here, lead, most, half, st.m, top_k, search);
        if (n - at <= H::kMost)
            break;
        at += H::kMost;
        lead = 0;
    }
    return block_stats<NT>(st, heat.log2, lds);
}

// One workgroup per row, four of 256 threads on a CU.  2048 x 128256 bf16 (525 MB): 86 to
// 95 us without alternatives (5.5 to 6.1 TB/s, memory), 114 us with 32 and 128 us with 64,
// where the search's latency and the vector arithmetic (12 instructions an element,
// VALUBusy 73%) come on top.  1501 x 50257 fp32: 49 us without (6.2 TB/s), 72 us with 64.
template <class T, int NT, bool TOP, bool SHORT>
__global__ void __launch_bounds__(NT, 4)
k_logprobs(const T *logits, int64_t ld, int64_t rows, int vocab, Heat heat, LogprobOut out)
{
    __shared__ float lds[3 * NT / 64];
    __shared__ typename std::conditional<TOP, Search, char>::type search;
    for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
        const T *z = logits + r * ld;
        uint64_t list;
        const RowStats st =
            whole_part<T, NT, TOP, SHORT>(z, 0, vocab, out.top_k, heat, lds, search, list);
        if (threadIdx.x < 64)
            write_row(out, z, r, vocab, st, list, heat);
        __syncthreads();
    }
}

// One workgroup per part of a row: 4 x 128256 bf16 with 20 alternatives 7.9 us, and 5.2 us
// for the join.
constexpr int kPartNT = 256;
template <class T, bool TOP>
__global__ void __launch_bounds__(kPartNT, 4)
k_parts(const T *logits, int64_t ld, int64_t rows, int vocab, Heat heat, int top_k, Parts parts)
{
    __shared__ float lds[3 * kPartNT / 64];
    __shared__ typename std::conditional<TOP, Search, char>::type search;
    const int64_t b = blockIdx.x, r = b / parts.count;
    const int at = (int)(b - r * parts.count) * parts.length;
    uint64_t list;
    const RowStats st = whole_part<T, kPartNT, TOP, false>(logits + r * ld + at, at,
                                                  min(vocab - at, parts.length), top_k, heat, lds,
                                                  search, list);
    if (threadIdx.x == 0) {
        const int64_t all = rows * parts.count;
        parts.stats[b] = st.m;
        parts.stats[all + b] = st.s;
        parts.stats[2 * all + b] = st.a;
    }
    if (TOP && (int)threadIdx.x < top_k)
        parts.keys[b * top_k + threadIdx.x] = list;
}

// A row's outputs from its parts: each wave merges a share of the lists, then the waves
// theirs in a tree.
constexpr int kJoinNT = 512;
template <class T>
__global__ void __launch_bounds__(kJoinNT)
k_logprobs_join(const T *logits, int64_t ld, int64_t rows, int vocab, Heat heat, LogprobOut out,
                Parts parts)
{
    constexpr int W = kJoinNT / 64;
    __shared__ uint64_t lists[W][64];
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    const int64_t r = blockIdx.x;
    uint64_t list = 0;
    if (out.top_k > 0) {
        for (int p = w; p < parts.count; p += W) {
            const uint64_t k =
                lane < out.top_k ? parts.keys[(r * parts.count + p) * out.top_k + lane] : 0;
            list = p == w ? k : wave_merge(list, k);
        }
        for (int half = W / 2; half >= 1; half /= 2) {
            lists[w][lane] = list;
            __syncthreads();
            if (w < half)
                list = wave_merge(list, lists[w + half][lane]);
            __syncthreads();
        }
    }
    if (w == 0)
        write_row(out, logits + r * ld, r, vocab, part_stats(parts, rows, r, heat.log2), list,
                  heat);
}

}  // namespace

}  // namespace mxq

void mxq::launch_parts(const void *logits, int32_t dtype, int64_t ld, int64_t rows, int64_t vocab,
                       const Heat &heat, int32_t top_k, const Parts &parts, hipStream_t s)
{
    with_type(dtype, [&](auto *tt) {
        using T = std::remove_pointer_t<decltype(tt)>;
        hipLaunchKernelGGL((top_k > 0 ? k_parts<T, true> : k_parts<T, false>),
                           dim3((unsigned)(rows * parts.count)), dim3(kPartNT), 0, s,
                           static_cast<const T *>(logits), ld, rows, (int)vocab, heat, top_k,
                           parts);
    });
}

using namespace mxq;

extern "C" size_t mxq_vocab_workspace_size(int64_t rows, int64_t vocab, int32_t top_k)
{
    if (rows < 1 || vocab < 1 || vocab > kMaxVocab || top_k < 0 || top_k > MXQ_TOP_MAX)
        return 0;
    const Parts p = parts_of(rows, vocab, top_k, nullptr);
    // and a row's m and s, joined
    return p.count == 1 ? 0 : (size_t)rows * (p.count * (8 * (size_t)top_k + 12) + 8);
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
    const Parts parts = parts_of(rows, vocab, top_k, workspace);
    if (parts.count > 1)
        launch_parts(logits, dtype, ld, rows, vocab, heat_of(temperature), top_k, parts, s);
    with_type(dtype, [&](auto *tt) {
        using T = std::remove_pointer_t<decltype(tt)>;
        if (parts.count > 1) {
            hipLaunchKernelGGL((k_logprobs_join<T>), dim3((unsigned)rows), dim3(kJoinNT), 0, s,
                               static_cast<const T *>(logits), ld, rows, (int)vocab,
                               heat_of(temperature), out, parts);
            return;
        }
        with_threads<T, 256>(rows, vocab, [&](auto nt, auto is_short) {
            constexpr int NT = decltype(nt)::value;
            constexpr bool SHORT = decltype(is_short)::value;
            const auto k = top_k > 0 ? k_logprobs<T, NT, true, SHORT> : k_logprobs<T, NT, false, SHORT>;
            hipLaunchKernelGGL(k, dim3(row_grid(rows)), dim3(NT), 0, s,
                               static_cast<const T *>(logits), ld, rows, (int)vocab,
                               heat_of(temperature), out);
        });
    });
    return launched();
}
