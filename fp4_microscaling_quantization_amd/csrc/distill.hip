// Distillation from a teacher's top alternatives (mxq_distill and its two
// halves), and the gradient of token log probabilities (both have the form
// dz = q (k0 + k1 d) apart from a few entries; include/mxq.h holds the formulas).
//
// mxq_distill with many rows is one pass: a workgroup holds its row in
// registers, of a longer row the last stretch, with a part of the first in LDS,
// so the logits come from memory once and the gradient goes there once.  Few long
// rows go as the statistics of their parts, then a gradient of chunks, as do the
// two halves on their own.
#include "vocab.hpp"

namespace mxq {

namespace {

// ---- the teacher -------------------------------------------------------------------

struct TeacherArgs {
    const int32_t *ids;
    const float *lps;
    int32_t top_k, renormalize;
    const float *weight;
};

// A row's teacher, one alternative per lane: its id (-1: absent), log p and p (0 where
// absent); their sum; whether an id is beyond the vocabulary; whether some p is not 0.
struct Teacher {
    int id;
    float p, logp, sum;
    bool bad, used;
};
__device__ __forceinline__ Teacher teacher_row(const TeacherArgs &a, int64_t r, int vocab)
{
    unsigned lane = threadIdx.x & 63;
    asm volatile("" : "+v"(lane));  // or both addresses are kept for the loop over rows, and spilled
    Teacher t;
    t.id = lane < (unsigned)a.top_k ? (a.ids + r * a.top_k)[lane] : -1;
    t.bad = __any(t.id >= vocab);
    t.logp = t.id >= 0 ? (a.lps + r * a.top_k)[lane] : -INFINITY;
    if (a.renormalize) {
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
// The same for a workgroup: wave 0 has it, the others what the whole row needs, after a
// barrier, through share_teacher.
struct Shared {
    float sum;
    int bad, used;
    // what wave 0 writes after the row's gradient, and where (-1: nothing): here and not in
    // registers, which k_distill_rows has none to spare of
    int id[64];
    float dz[64];
};
__device__ __forceinline__ Teacher wave0_teacher(const TeacherArgs &a, int64_t r, int vocab,
                                                 Shared &lds)
{
    Teacher t = {-1, 0.0f, 0.0f, 0.0f, false, false};
    if (threadIdx.x < 64) {
        t = teacher_row(a, r, vocab);
        if (threadIdx.x == 0) {
            lds.sum = t.sum;
            lds.bad = t.bad;
            lds.used = t.used;
        }
    }
    return t;
}
__device__ __forceinline__ void share_teacher(Teacher &t, const Shared &lds)
{
    t.sum = lds.sum;
    t.bad = lds.bad;
    t.used = lds.used;
}
__device__ __forceinline__ bool counts(const Teacher &t, float w)
{
    return w != 0.0f && (t.used || t.bad);
}
// the loss of a row that counts; zt: the student's logit at the lane's id
__device__ __forceinline__ float row_loss(const Teacher &t, float zt, bool have, float w,
                                          const RowStats &st, const Heat &h)
{
    const float term = have && t.p != 0.0f ? t.p * (t.logp - log_q(zt, st, h)) : 0.0f;
    const float sum = wave_sum(term);
    // temperature^2 need not be an fp32 number: the sum is of the order of 1 / T or 1 / T^2
    return t.bad ? NAN : w * (h.t * (h.t * sum));
}

// ---- gradients -----------------------------------------------------------------------

// dz = 2^d (k0 + k1 d), d = (z - b) log2 (in units of log2): what every entry of
// a row has; the 1 / S, the weight and the temperature are in k0 and k1.
struct Gradient {
    float b, k0, k1;
};
template <bool SLOPE>
__device__ __forceinline__ float gradient_at(float z, const Gradient &g, float log2)
{
    const float d = (z - g.b) * log2;
    const float e = __builtin_amdgcn_exp2f(d);
    return e * (SLOPE ? fmaf(g.k1, fmaxf(d, kFloorLog2), g.k0) : g.k0);
}
__device__ __forceinline__ Gradient distill_gradient(const Teacher &t, float w, const RowStats &st,
                                                     const Heat &h)
{
    if (t.bad)
        return {0.0f, NAN, 0.0f};
    // a row with every logit masked: q = 0
    return {base_of(st.m), st.s == 0.0f ? 0.0f : w * h.t * t.sum / st.s, 0.0f};
}

// a held stretch's gradient to o
template <bool SLOPE, class T, class O, int NT, int NV>
__device__ __forceinline__ void write_gradient(const Held<T, NT, NV> &held, O *o, int n, int lead,
                                               const Gradient &g, float log2)
{
    constexpr int E = kElems<T>;
    n = fresh(n);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        if (held.any(i, n)) {
            float f[E];
            held.get(i, f);
#pragma unroll
            for (int j = 0; j < E; ++j)
                f[j] = gradient_at<SLOPE>(f[j], g, log2);
            held.put(o, i, n, f, lead);
        }
    }
}

// n entries at o, all `value`
template <class O, int NT> __device__ __forceinline__ void write_all(O *o, int n, float value)
{
    constexpr int E = kElems<O>;
    asm volatile("" : "+v"(value));  // or its vector is kept for the loop over rows, and spilled
    float f[E];
#pragma unroll
    for (int j = 0; j < E; ++j)
        f[j] = value;
    for (int64_t at = (int)threadIdx.x * E; at < n; at += NT * E) {
        if (at + E <= n) {
            store_vec(o + at, f);
        } else {
            for (int64_t k = at; k < n; ++k)
                o[k] = (O)value;
        }
    }
}

// The gradient at the lane's id, if that is in [from, to), with its p: zt is the logit
// there, loaded before the row was written (the gradient may lie over the logits).  An
// id that comes twice: each of its lanes has the sum of both p, and so the same value.
__device__ __forceinline__ float id_gradient(const Teacher &t, float zt, int from, int to,
                                             const Gradient &g, float wt, float log2)
{
    const bool mine = t.id >= from && t.id < to;
    float p = 0.0f;
    for (uint64_t left = __ballot(mine); left; left &= left - 1) {
        const int j = __ffsll((unsigned long long)left) - 1;
        const int id = __builtin_amdgcn_readlane(t.id, j);
        const float pj = as_f((uint32_t)__builtin_amdgcn_readlane((int)as_u(t.p), j));
        p += id == t.id ? pj : 0.0f;
    }
    return fmaf(-wt, p, gradient_at<false>(zt, g, log2));
}
// The entries of these ids once more; called by one wave, after a barrier.
template <class O>
__device__ __forceinline__ void write_ids(O *o, const Teacher &t, float zt, int from, int to,
                                          const Gradient &g, float wt, float log2)
{
    const float dz = id_gradient(t, zt, from, to, g, wt, log2);
    if (t.id >= from && t.id < to)
        o[t.id] = (O)dz;
}

// ---- whole rows ----------------------------------------------------------------------

// The loss (and stats) of a row that counts, by one wave.
__device__ __forceinline__ void write_loss(float *loss, float *stats, int64_t r, const Teacher &t,
                                           float zt, float w, int vocab, const RowStats &st,
                                           const Heat &heat)
{
    const float l = row_loss(t, zt, t.id >= 0 && t.id < vocab, w, st, heat);
    if ((threadIdx.x & 63) == 0) {
        loss[r] = counts(t, w) ? l : 0.0f;
        if (stats) {
            stats[2 * r] = st.m;
            stats[2 * r + 1] = st.s;
        }
    }
}
// those of a row with w = 0
__device__ __forceinline__ void write_no_loss(float *loss, float *stats, int64_t r)
{
    if (threadIdx.x == 0) {
        loss[r] = 0.0f;
        if (stats) {
            stats[2 * r] = 0.0f;
            stats[2 * r + 1] = 1.0f;
        }
    }
}
// the logit at the lane's id, where that is in [from, to); it is there before the next
// barrier, behind which the gradient may be written over it
template <class T>
__device__ __forceinline__ float logit_at(const T *z, const Teacher &t, int from, int to)
{
    float zt = t.id >= from && t.id < to ? load_one(z + t.id) : 0.0f;
    asm volatile("" : "+v"(zt));
    return zt;
}

// One workgroup per row: loss and stats.  Bound by memory, reads only: 4096 x 128256 fp32
// 308 us, 6.8 TB/s.
template <class T, int NT, bool SHORT>
__global__ void __launch_bounds__(NT, 4)
k_distill_loss(const T *logits, int64_t ld, int64_t rows, int vocab, Heat heat, TeacherArgs ta,
               float *loss, float *stats)
{
    using H = Held<T, NT, kHeld>;
    __shared__ float lds[3 * NT / 64];
    for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
        const T *z = logits + r * ld;
        const float w = ta.weight ? ta.weight[r] : 1.0f;
        if (w == 0.0f) {
            write_no_loss(loss, stats, r);
            continue;
        }
        RowStats st = {-FLT_MAX, 0.0f, 0.0f};
        int lead = lead_of<T, SHORT>(z);
        const T *start = z - lead;
        const int all = vocab + lead;
        for (int at = 0;;) {
            const int n = min(all - at, H::kMost);
            H held;
            held.template load<SHORT, true>(start + at, n);
            float most[kGroups<T>], half[2];
            absorb_held<false>(st, held, n, lead, heat.log2, most, half);
            if (all - at <= H::kMost)
                break;
            at += H::kMost;
            lead = 0;
        }
        st = block_stats<NT>(st, heat.log2, lds);
        if (threadIdx.x < 64) {
            const Teacher t = teacher_row(ta, r, vocab);
            write_loss(loss, stats, r, t, logit_at(z, t, 0, vocab), w, vocab, st, heat);
        }
        __syncthreads();
    }
}

// The same from the parts of few rows, one wave a row.  stats is null if neither the
// caller nor the gradient asks for them.
template <class T>
__global__ void __launch_bounds__(64)
k_distill_join(const T *logits, int64_t ld, int64_t rows, int vocab, Heat heat, TeacherArgs ta,
               Parts parts, float *loss, float *stats)
{
    const int64_t r = blockIdx.x;
    const float w = ta.weight ? ta.weight[r] : 1.0f;
    if (w == 0.0f) {
        write_no_loss(loss, stats, r);
        return;
    }
    const T *z = logits + r * ld;
    const Teacher t = teacher_row(ta, r, vocab);
    write_loss(loss, stats, r, t, logit_at(z, t, 0, vocab), w, vocab,
               part_stats(parts, rows, r, heat.log2), heat);
}

// One workgroup per row: loss and dlogits.  The row is held; of a row longer than the
// registers hold (LONG), half of the first stretch stays in LDS, and what is left before
// the last stretch is read again for the gradient, from the last-level cache.  Bound by
// memory: 4096 x 128256 fp32 to bf16 with a tenth of the rows ignored, 2.94 GB, 531 us
// (5.5 TB/s; the LDS saved 53 us of the second reading), and 4096 x 32000 fp32 to bf16,
// which is held whole, 134 us (5.9 TB/s).  bf16 to fp32 2048 x 128256 497 us (3.2 TB/s; to bf16
// 196 us, 5.4): a store's lanes, 16 bytes each, are 32 bytes apart.  Registers are short: 8 spilled
// ones, 32 bytes a thread that nothing read again, cost 17 us of the first case.  The fp32 forms
// spill none now; those of bf16 rows longer than the registers hold, which have `lead` on top,
// still spill 13 (to bf16) and 4 (to fp32).
constexpr int kStaged = 8;  // vectors a thread has in LDS: 128 KB of the CU's 160
template <class T, class O, int NT, bool LONG, bool SHORT>
__global__ void __launch_bounds__(NT, 4)
k_distill_rows(const T *logits, int64_t ld, int64_t rows, int vocab, Heat heat, TeacherArgs ta,
               float *loss, O *dlogits, int64_t ld_o)
{
    using H = Held<T, NT, kHeld>;
    __shared__ float lds[3 * NT / 64];
    __shared__ gv4u staged[LONG ? kStaged : 1][LONG ? NT : 1];
    __shared__ Shared teacher;
    for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
        const T *z = logits + r * ld;
        O *o = dlogits + r * ld_o;
        const float w = ta.weight ? ta.weight[r] : 1.0f;
        if (w == 0.0f) {
            write_no_loss(loss, nullptr, r);
            write_all<O, NT>(o, vocab, 0.0f);
            continue;
        }
        H held;
        RowStats st = {-FLT_MAX, 0.0f, 0.0f};
        int at = 0, n = 0;
        float most[kGroups<T>], half[2];
        const int lead = lead_of<T, SHORT>(z);
        const T *start = z - lead;
        if constexpr (LONG) {
            for (; vocab + lead - at > H::kMost; at += H::kMost) {
                held.template load<false, false>(start + at, H::kMost);
                absorb_held<false>(st, held, H::kMost, at == 0 ? lead : 0, heat.log2, most, half);
                if (at == 0) {
#pragma unroll
                    for (int i = 0; i < kStaged; ++i)
                        staged[i][threadIdx.x] = held.v[i];  // read by the same thread only
                }
            }
        }
        n = vocab + lead - at;
        held.template load<SHORT, true>(start + at, n);
        absorb_held<false>(st, held, n, at == 0 ? lead : 0, heat.log2, most, half);
        Teacher t = wave0_teacher(ta, r, vocab, teacher);
        const float zt = logit_at(z, t, 0, vocab);
        st = block_stats<NT>(st, heat.log2, lds);
        share_teacher(t, teacher);
        held.again();
        if (threadIdx.x < 64)
            write_loss(loss, nullptr, r, t, zt, w, vocab, st, heat);
        if (!counts(t, w)) {
            write_all<O, NT>(o, vocab, 0.0f);
        } else {
            const Gradient g = distill_gradient(t, w, st, heat);
            if (threadIdx.x < 64) {
                teacher.id[threadIdx.x] = t.bad ? -1 : t.id;
                teacher.dz[threadIdx.x] = id_gradient(t, zt, 0, vocab, g, w * heat.t, heat.log2);
            }
            for (;;) {
                write_gradient<false>(held, o - lead + at, n, at == 0 ? lead : 0, g, heat.log2);
                if (!LONG || at == 0)
                    break;
                at -= H::kMost;
                n = H::kMost;
                if (at > 0) {
                    held.template load<false, true>(start + at, n);
                } else {
#pragma unroll
                    for (int i = 0; i < kHeld; ++i)
                        held.v[i] = i < kStaged ? staged[i][threadIdx.x]
                                                : load_vec<true>(lane_at<H::E>(start + i * NT * H::E));
                }
            }
            __syncthreads();
            if (threadIdx.x < 64 && teacher.id[threadIdx.x] >= 0)
                o[teacher.id[threadIdx.x]] = (O)teacher.dz[threadIdx.x];
        }
        __syncthreads();
    }
}

// ---- gradients of chunks --------------------------------------------------------------

// A chunk of a row per workgroup: short enough that a few rows fill the chip, and
// that several workgroups share a CU, so that one's loads run under another's
// stores.  4096 x 128256 fp32 to bf16 505 us, 6.2 TB/s; 2048 x 50257 bf16 85 us, 4.9 TB/s
// (chunks of twice the vectors 538 and 93 us, of half 590 and 101 us).  bf16 to fp32 2048 x
// 128256 349 us, 4.5 TB/s, for the stores' sake (k_distill_rows).
// Short rows, when there are many, are one chunk of a wave each.
template <class T, int NT> using Chunk = Held<T, NT, NT == 64 ? 8 : 4>;

// Chunk number `chunk` of the row at z: entries from `at` on, n of them with the `lead`
// that lie before them; false: the row has none.  The chunks of a row that starts off a
// 16-byte boundary are shifted, so the last may be a chunk more.
template <class H, bool SHORT, class T>
__device__ __forceinline__ bool chunk_of(const T *z, int vocab, int chunk, int &at, int &n,
                                         int &lead)
{
    const int shift = lead_of<T, SHORT>(z);
    const int64_t from = (int64_t)chunk * H::kMost;  // from the boundary
    if (from >= (int64_t)vocab + shift)
        return false;
    lead = chunk == 0 ? shift : 0;
    at = (int)(from + lead - shift);
    n = (int)min((int64_t)vocab + shift - from, (int64_t)H::kMost);
    return true;
}

// PARTS: the rows' statistics come from their parts, and the first chunk's workgroup
// writes the loss; the gradient must not lie over the logits then.
template <class T, class O, int NT, bool PARTS, bool SHORT>
__global__ void __launch_bounds__(NT)
k_distill_chunks(const T *logits, int64_t ld, int64_t rows, int vocab, int chunks, Heat heat,
                 TeacherArgs ta, const float *stats, Parts parts, float *loss, O *dlogits,
                 int64_t ld_o)
{
    using H = Chunk<T, NT>;
    __shared__ Shared teacher;
    for (int64_t b = blockIdx.x; b < rows * chunks; b += gridDim.x) {
        const int64_t r = b / chunks;
        const T *z = logits + r * ld;
        O *o = dlogits + r * ld_o;
        // the row's entries from `at` on, or `lead` before them
        int at, n, lead;
        if (!chunk_of<H, SHORT>(z, vocab, (int)(b - r * chunks), at, n, lead))
            continue;
        const float w = ta.weight ? ta.weight[r] : 1.0f;
        if (w == 0.0f) {
            if (PARTS && at == 0)
                write_no_loss(loss, nullptr, r);
            write_all<O, NT>(o + at, n - lead, 0.0f);
            continue;
        }
        H held;
        held.template load<SHORT, true>(z + at - lead, n);
        Teacher t = wave0_teacher(ta, r, vocab, teacher);
        const int end = at + n - lead;
        const float zt = logit_at(z, t, at, end);
        RowStats st;
        if constexpr (PARTS) {
            st = part_stats(parts, rows, r, heat.log2);
            if (at == 0 && threadIdx.x < 64)
                write_loss(loss, nullptr, r, t, logit_at(z, t, 0, vocab), w, vocab, st, heat);
        } else {
            st = {stats[2 * r], stats[2 * r + 1], 0.0f};
        }
        // everything is read before anything is written over it
        held.again();
        __syncthreads();
        share_teacher(t, teacher);
        if (!counts(t, w)) {
            write_all<O, NT>(o + at, n - lead, 0.0f);
            __syncthreads();
            continue;
        }
        const Gradient g = distill_gradient(t, w, st, heat);
        write_gradient<false>(held, o + at - lead, n, lead, g, heat.log2);
        __syncthreads();
        if (threadIdx.x < 64 && !t.bad)
            write_ids(o, t, zt, at, end, g, w * heat.t, heat.log2);
    }
}

// The gradient of log probabilities and entropy: 1024 x 32000 fp32 to bf16 38 us, 5.2 TB/s
// (chunks of twice the vectors 36, but 26 against 23 from bf16, and 3.9 against 3.3 for 4
// rows of 128256).  bf16 to fp32 2048 x 128256 456 us, 3.5 TB/s; to bf16 187 us, 5.6.
template <class T, class O, int NT, bool SHORT>
__global__ void __launch_bounds__(NT)
k_logprobs_bwd(const T *logits, int64_t ld, int64_t rows, int vocab, int chunks, Heat heat,
               const int32_t *tokens, const float *stats, const float *entropy,
               const float *d_logprob, const float *d_entropy, O *dlogits, int64_t ld_o)
{
    using H = Chunk<T, NT>;
    constexpr float kLn2 = 0.69314718055994531f;
    for (int64_t b = blockIdx.x; b < rows * chunks; b += gridDim.x) {
        const int64_t r = b / chunks;
        const T *z = logits + r * ld;
        O *o = dlogits + r * ld_o;
        int at, n, lead;
        if (!chunk_of<H, SHORT>(z, vocab, (int)(b - r * chunks), at, n, lead))
            continue;
        H held;
        held.template load<SHORT, true>(z + at - lead, n);
        const int token = d_logprob ? tokens[r] : -1;
        const float gl = token < 0 ? 0.0f : token >= vocab ? NAN : d_logprob[r] * heat.inv;
        const float gh = d_entropy ? d_entropy[r] * heat.inv : 0.0f;
        const float m = stats[2 * r], s = stats[2 * r + 1];
        // -(gl + gh (log q + H)) / S with log q = d - log S: a constant and a slope in d
        Gradient g = {base_of(m), 0.0f, 0.0f};
        if (s != 0.0f) {
            const float c = d_entropy ? fmaf(gh, entropy[r] - logf(s), gl) : gl;
            g.k0 = -c / s;
            g.k1 = -gh * kLn2 / s;
        } else if (token >= vocab) {
            g.k0 = NAN;
        }
        const bool here = token >= at && token < at + n - lead;
        float zt = here ? load_one(z + token) : 0.0f;
        asm volatile("" : "+v"(zt));
        held.again();
        __syncthreads();
        write_gradient<true>(held, o + at - lead, n, lead, g, heat.log2);
        __syncthreads();
        if (here && threadIdx.x == 0)
            o[token] = (O)(gl + gradient_at<true>(zt, g, heat.log2));
    }
}

mxq_status check_teacher(int64_t rows, const TeacherArgs &t)
{
    if (t.top_k < 1 || t.top_k > MXQ_TOP_MAX || (t.renormalize != 0 && t.renormalize != 1))
        return MXQ_ERR_UNSUPPORTED;
    if (rows > 0 && (!t.ids || !t.lps))
        return MXQ_ERR_NULL;
    return aligned4(t.ids) && aligned4(t.lps) && aligned4(t.weight) ? MXQ_OK : MXQ_ERR_ALIGN;
}

// f(threads of a chunk's workgroup, chunks of a row, grid of a launch over them)
template <class T, class F> void with_chunks(int64_t rows, int64_t vocab, F f)
{
    // a row may start up to kElems - 1 elements after its first chunk's boundary
    const int64_t most = vocab + kElems<T> - 1;
    const auto go = [&](auto nt) {
        constexpr int64_t size = Chunk<T, decltype(nt)::value>::kMost;
        const int chunks = (int)((most + size - 1) / size);
        f(nt, chunks, (unsigned)(rows < kMaxGrid / chunks ? rows * chunks : kMaxGrid));
    };
    if (vocab < kElems<T> || (most <= Chunk<T, 64>::kMost && rows >= kWaveRows))
        go(std::integral_constant<int, 64>());
    else
        go(std::integral_constant<int, 256>());
}

// Whether mxq_distill takes whole rows where there are parts too.  Parts read the logits
// twice and are two launches, which pays for a few long rows: 4 x 128256 fp32 7.6 us
// against 17.0 whole, 48 rows 17.3 against 19.3, 64 rows 21.6 against 19.4; of bf16 64
// rows 15.4 against 17.4, 96 rows 20.5 against 17.8 (the one limit in bytes is a little
// late for bf16); rows of up to 128 KB gain little, 16 x 50257 bf16 9.8 against 10.3.
bool whole_rows(int64_t rows, int64_t vocab, int32_t dtype)
{
    const int64_t row = vocab * (dtype == MXQ_OUT_F32 ? 4 : 2);
    return row <= 128 << 10 || rows > (24 << 20) / row;
}

struct Logits {
    const void *z;
    int32_t dtype;
    int64_t ld, rows, vocab;
    Heat heat;
};

void launch_loss(const Logits &a, const TeacherArgs &ta, float *loss, float *stats, hipStream_t s)
{
    with_type(a.dtype, [&](auto *tt) {
        using T = std::remove_pointer_t<decltype(tt)>;
        with_threads<T, 256>(a.rows, a.vocab, [&](auto nt, auto is_short) {
            constexpr int NT = decltype(nt)::value;
            hipLaunchKernelGGL((k_distill_loss<T, NT, decltype(is_short)::value>),
                               dim3(row_grid(a.rows)), dim3(NT), 0, s,
                               static_cast<const T *>(a.z), a.ld, a.rows, (int)a.vocab, a.heat, ta,
                               loss, stats);
        });
    });
}
void launch_join(const Logits &a, const TeacherArgs &ta, const Parts &parts, float *loss,
                 float *stats, hipStream_t s)
{
    with_type(a.dtype, [&](auto *tt) {
        using T = std::remove_pointer_t<decltype(tt)>;
        hipLaunchKernelGGL((k_distill_join<T>), dim3((unsigned)a.rows), dim3(64), 0, s,
                           static_cast<const T *>(a.z), a.ld, a.rows, (int)a.vocab, a.heat, ta,
                           parts, loss, stats);
    });
}
void launch_rows(const Logits &a, const TeacherArgs &ta, float *loss, void *dlogits,
                 int32_t o_dtype, int64_t ld_o, hipStream_t s)
{
    with_type(a.dtype, [&](auto *tt) {
        with_type(o_dtype, [&](auto *ot) {
            using T = std::remove_pointer_t<decltype(tt)>;
            using O = std::remove_pointer_t<decltype(ot)>;
            with_threads<T, 1024>(a.rows, a.vocab, [&](auto nt, auto is_short) {
                constexpr int NT = decltype(nt)::value;
                constexpr bool SHORT = decltype(is_short)::value;
                auto k = k_distill_rows<T, O, NT, false, SHORT>;
                // a row that starts off a boundary may need one more stretch
                if constexpr (NT == 1024) {
                    if (a.vocab + kElems<T> - 1 > Held<T, NT, kHeld>::kMost)
                        k = k_distill_rows<T, O, NT, true, false>;
                }
                hipLaunchKernelGGL(k, dim3(row_grid(a.rows)), dim3(NT), 0, s,
                                   static_cast<const T *>(a.z), a.ld, a.rows, (int)a.vocab, a.heat,
                                   ta, loss, static_cast<O *>(dlogits), ld_o);
            });
        });
    });
}
// parts with count > 1: the statistics and the loss from there; else from stats
void launch_chunks(const Logits &a, const TeacherArgs &ta, const float *stats, const Parts &parts,
                   float *loss, void *dlogits, int32_t o_dtype, int64_t ld_o, hipStream_t s)
{
    with_type(a.dtype, [&](auto *tt) {
        with_type(o_dtype, [&](auto *ot) {
            using T = std::remove_pointer_t<decltype(tt)>;
            using O = std::remove_pointer_t<decltype(ot)>;
            with_chunks<T>(a.rows, a.vocab, [&](auto nt, int chunks, unsigned grid) {
                constexpr int NT = decltype(nt)::value;
                auto k = k_distill_chunks<T, O, NT, false, false>;
                if constexpr (NT == 64) {
                    if (a.vocab < kElems<T>)
                        k = k_distill_chunks<T, O, 64, false, true>;
                } else if (parts.count > 1) {  // rows with parts are longer than a wave's chunk
                    k = k_distill_chunks<T, O, NT, true, false>;
                }
                hipLaunchKernelGGL(k, dim3(grid), dim3(NT), 0, s, static_cast<const T *>(a.z),
                                   a.ld, a.rows, (int)a.vocab, chunks, a.heat, ta, stats, parts,
                                   loss, static_cast<O *>(dlogits), ld_o);
            });
        });
    });
}

}  // namespace

}  // namespace mxq

using namespace mxq;

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
            with_chunks<T>(rows, vocab, [&](auto nt, int chunks, unsigned grid) {
                constexpr int NT = decltype(nt)::value;
                auto k = k_logprobs_bwd<T, O, NT, false>;
                if constexpr (NT == 64) {
                    if (vocab < kElems<T>)
                        k = k_logprobs_bwd<T, O, 64, true>;
                }
                hipLaunchKernelGGL(k, dim3(grid), dim3(NT), 0, s, static_cast<const T *>(logits),
                                   ld, rows, (int)vocab, chunks, heat_of(temperature), tokens,
                                   stats, entropy, d_logprob, d_entropy,
                                   static_cast<O *>(dlogits), ld_dlogits);
            });
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
    const TeacherArgs ta = {teacher_ids, teacher_logprobs, top_k, renormalize, weight};
    mxq_status st = check_logits(logits, dtype, ld, rows, vocab, temperature);
    if (!st)
        st = check_teacher(rows, ta);
    if (st || rows == 0)
        return st;
    if (!loss || !stats)
        return MXQ_ERR_NULL;
    if (!aligned4(loss) || !aligned4(stats) || reinterpret_cast<uintptr_t>(workspace) % 8)
        return MXQ_ERR_ALIGN;
    const size_t need = mxq_vocab_workspace_size(rows, vocab, 0);
    if (need > 0 && (!workspace || ws_bytes < need))
        return MXQ_ERR_WORKSPACE;
    hipStream_t s = static_cast<hipStream_t>(stream);
    const Logits a = {logits, dtype, ld, rows, vocab, heat_of(temperature)};
    const Parts parts = parts_of(rows, vocab, 0, workspace);
    if (parts.count > 1) {
        launch_parts(logits, dtype, ld, rows, vocab, a.heat, 0, parts, s);
        launch_join(a, ta, parts, loss, stats, s);
    } else {
        launch_loss(a, ta, loss, stats, s);
    }
    return launched();
}

extern "C" mxq_status mxq_distill_backward(const void *logits, int32_t dtype, int64_t ld,
                                           int64_t rows, int64_t vocab, float temperature,
                                           const int32_t *teacher_ids,
                                           const float *teacher_logprobs, int32_t top_k,
                                           int32_t renormalize, const float *weight,
                                           const float *stats, void *dlogits,
                                           int32_t dlogits_dtype, int64_t ld_dlogits, void *stream)
{
    const TeacherArgs ta = {teacher_ids, teacher_logprobs, top_k, renormalize, weight};
    mxq_status st = check_logits(logits, dtype, ld, rows, vocab, temperature);
    if (!st)
        st = check_gradient(dlogits, dlogits_dtype, ld_dlogits, rows, vocab);
    if (!st)
        st = check_teacher(rows, ta);
    if (st || rows == 0)
        return st;
    if (!stats)
        return MXQ_ERR_NULL;
    if (!aligned4(stats))
        return MXQ_ERR_ALIGN;
    launch_chunks({logits, dtype, ld, rows, vocab, heat_of(temperature)}, ta, stats,
                  {1, (int)vocab, nullptr, nullptr}, nullptr, dlogits, dlogits_dtype, ld_dlogits,
                  static_cast<hipStream_t>(stream));
    return launched();
}

extern "C" mxq_status mxq_distill(const void *logits, int32_t dtype, int64_t ld, int64_t rows,
                                  int64_t vocab, float temperature, const int32_t *teacher_ids,
                                  const float *teacher_logprobs, int32_t top_k,
                                  int32_t renormalize, const float *weight, float *loss,
                                  void *dlogits, int32_t dlogits_dtype, int64_t ld_dlogits,
                                  void *workspace, size_t ws_bytes, void *stream)
{
    const TeacherArgs ta = {teacher_ids, teacher_logprobs, top_k, renormalize, weight};
    mxq_status st = check_logits(logits, dtype, ld, rows, vocab, temperature);
    if (!st)
        st = check_gradient(dlogits, dlogits_dtype, ld_dlogits, rows, vocab);
    if (!st)
        st = check_teacher(rows, ta);
    if (st || rows == 0)
        return st;
    if (!loss)
        return MXQ_ERR_NULL;
    if (!aligned4(loss) || reinterpret_cast<uintptr_t>(workspace) % 8)
        return MXQ_ERR_ALIGN;
    const size_t need = mxq_vocab_workspace_size(rows, vocab, 0);
    if (need > 0 && (!workspace || ws_bytes < need))
        return MXQ_ERR_WORKSPACE;
    hipStream_t s = static_cast<hipStream_t>(stream);
    const Logits a = {logits, dtype, ld, rows, vocab, heat_of(temperature)};
    const Parts parts = parts_of(rows, vocab, 0, workspace);
    if (parts.count == 1 || whole_rows(rows, vocab, dtype)) {
        launch_rows(a, ta, loss, dlogits, dlogits_dtype, ld_dlogits, s);
        return launched();
    }
    launch_parts(logits, dtype, ld, rows, vocab, a.heat, 0, parts, s);
    if (dlogits != logits) {
        launch_chunks(a, ta, nullptr, parts, loss, dlogits, dlogits_dtype, ld_dlogits, s);
        return launched();
    }
    // the loss reads logits of the whole row: before anything is written over them
    float *stats = parts.stats + 3 * rows * parts.count;
    launch_join(a, ta, parts, loss, stats, s);
    launch_chunks(a, ta, stats, {1, (int)vocab, nullptr, nullptr}, nullptr, dlogits, dlogits_dtype,
                  ld_dlogits, s);
    return launched();
}
