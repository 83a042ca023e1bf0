// Softmax cross entropy from the hidden states and the output layer's weight, without
// the logits z = x w^T ever being in memory.
//
//   forward   a tile of logits stays in the registers of the product; each row leaves
//             its maximum m and sum s = sum exp((z - m) / T) over the tile's vocabulary,
//             and a second kernel joins them over the tiles.
//   backward  a piece of the vocabulary at a time: the product again, turned into
//             dz = weight / T (exp((z - m) / T) / s - 1[v = target]) in bf16, which the two
//             products dx += dz w and dw = dz^T x then read.
//
// Rows that do not count are left out of all of it: the rows that do are packed first.
#include "product.hpp"
#include "rows.hpp"
#include "vocab.hpp"

namespace mxq {
namespace {

typedef uint16_t u16;

struct CeRows {
    const int32_t *targets;  // < 0: the row does not count
    const float *weight;     // NULL: 1; 0: the row does not count
    int64_t rows;
};
struct CeWeight {
    const u16 *w;
    int64_t ld;
    int vocab, hidden;
};
struct CePacked {
    int *count;        // rows that count
    int *place;        // [rows]: a row's place among them, -1: none
    int *row;          // [count]
    float *at_target;  // [count]: the logit at the target
    u16 *x;            // [count, up to a whole step][ld], zero behind both
    int ld;            // hidden, up to a whole step
};

// the statistics of two stretches of a row, as one
__device__ __forceinline__ void join_stats(RowStats &st, float2 o, float log2)
{
    const float m = fmaxf(st.m, o.x), base = base_of(m);
    st.s = fmaf(st.s, __builtin_amdgcn_exp2f((st.m - base) * log2),
                o.y * __builtin_amdgcn_exp2f((o.x - base) * log2));
    st.m = m;
}

// ---- packing ---------------------------------------------------------------------

__device__ __forceinline__ bool row_counts(const CeRows &a, int64_t r)
{
    return a.targets[r] >= 0 && !(a.weight && a.weight[r] == 0.0f);
}

constexpr int kPackThreads = 256;

// The rows that count, in order: where each went (or -1), which it was, and how many,
// and their values.  A workgroup finds its place by counting all rows in front of its
// own.  Behind the last row and the last value are zeros, up to whole steps of the
// products over either.
__global__ __launch_bounds__(kPackThreads) void k_ce_pack(CeRows a, int64_t per, const bf16_t *x,
                                                          int64_t ld, int hidden, CePacked to)
{
    __shared__ int partial[kPackThreads / 64];
    const int64_t first = (int64_t)blockIdx.x * per;
    const int64_t end = first + per < a.rows ? first + per : a.rows;
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    int before = 0;
    for (int64_t r = threadIdx.x; r < first; r += kPackThreads)
        before += row_counts(a, r);
    for (int d = 1; d < 64; d *= 2)
        before += __shfl_xor(before, d);
    if (lane == 0)
        partial[wave] = before;
    __syncthreads();
    int place = 0;
    for (int w = 0; w < kPackThreads / 64; ++w)
        place += partial[w];
    for (int64_t base = first; base < end; base += 64) {
        // every wave works out the same
        const int64_t mine = base + lane;
        const bool in = mine < end && row_counts(a, mine);
        const uint64_t all = __ballot(in);
        const int at = place + __popcll(all & ((1ull << lane) - 1));
        if (wave == 0 && mine < end) {
            to.place[mine] = in ? at : -1;
            if (in)
                to.row[at] = (int)mine;
        }
        int n = place;
        for (uint64_t left = all; left; left &= left - 1, ++n) {
            const int64_t r = base + __builtin_ctzll(left);
            for (int c = threadIdx.x * 8; c < to.ld; c += kPackThreads * 8)
                *reinterpret_cast<gv4u *>(to.x + (int64_t)n * to.ld + c) =
                    c < hidden ? load_vec(x + r * ld + c) : (gv4u){0u, 0u, 0u, 0u};
        }
        place += __popcll(all);
    }
    if (blockIdx.x == gridDim.x - 1) {
        if (threadIdx.x == 0)
            *to.count = place;
        const int stop = (place + kStepK - 1) / kStepK * kStepK;
        for (int64_t c = (int64_t)place * to.ld + threadIdx.x * 8; c < (int64_t)stop * to.ld;
             c += kPackThreads * 8)
            *reinterpret_cast<gv4u *>(to.x + c) = (gv4u){0u, 0u, 0u, 0u};
    }
}

// ---- logits ----------------------------------------------------------------------

using Logit = Product<2, 4, 8, 4, true, true>;

// the tile's product: w rows from p0, packed x rows from q0
template <class Tile>
__device__ __forceinline__ void logits(Tile &t, uint8_t *lds, const CeWeight &w,
                                       const CePacked &x, int p0, int count, int q0)
{
    t.start(lds, w.ld, w.vocab - p0, x.ld, count - q0, w.hidden);
    const uint8_t *p = reinterpret_cast<const uint8_t *>(w.w + (int64_t)p0 * w.ld);
    const uint8_t *q = reinterpret_cast<const uint8_t *>(x.x + (int64_t)q0 * x.ld);
    const int steps = (w.hidden + kStepK - 1) / kStepK;
    t.run(steps, p, kStepK * 2, q, kStepK * 2, (int)(blockIdx.x & 7) * steps / 8);
}

// Maximum and sum of every packed row over the tile's vocabulary, and the logit at its
// target.
__global__ __launch_bounds__(Logit::kThreads, 1) void k_ce_stats(CeWeight w, CeRows a,
                                                                 CePacked x, Heat heat,
                                                                 float2 *part, int64_t stride)
{
    __shared__ __align__(16) uint8_t lds[Logit::kLds];
    const int count = *x.count;
    const int np = (w.vocab + Logit::kP - 1) / Logit::kP, nq = (count + Logit::kQ - 1) / Logit::kQ;
    if ((int)blockIdx.x >= np * nq)
        return;
    int tp, tq;
    product_tile(blockIdx.x, np, nq, tp, tq);
    const int p0 = tp * Logit::kP, q0 = tq * Logit::kQ;
    Logit t;
    logits(t, lds, w, x, p0, count, q0);

    __syncthreads();
    float2 *joint = reinterpret_cast<float2 *>(lds);  // [WP][kQ]
#pragma unroll
    for (int j = 0; j < Logit::NQ; ++j) {
        const int q = t.q_of(j);
        const int target = q0 + q < count ? a.targets[x.row[q0 + q]] : -1;
        float m = -INFINITY;
#pragma unroll
        for (int i = 0; i < Logit::NP; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int p = p0 + t.p_of(i) + r;
                if (p >= w.vocab)
                    t.acc[i][j][r] = -INFINITY;
                if (p == target)
                    x.at_target[q0 + q] = t.acc[i][j][r];
                m = fmaxf(m, t.acc[i][j][r]);
            }
        m = fmaxf(m, __shfl_xor(m, 16));
        m = fmaxf(m, __shfl_xor(m, 32));
        const float base = base_of(m);
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < Logit::NP; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                s += __builtin_amdgcn_exp2f((t.acc[i][j][r] - base) * heat.log2);
        s += __shfl_xor(s, 16);
        s += __shfl_xor(s, 32);
        if (t.lane < 16)
            joint[t.wp * Logit::kQ + q] = make_float2(m, s);
    }
    __syncthreads();
    for (int q = threadIdx.x; q < Logit::kQ && q0 + q < count; q += Logit::kThreads) {
        RowStats st = {joint[q].x, joint[q].y, 0.0f};
        for (int k = 1; k < Logit::WP; ++k)
            join_stats(st, joint[k * Logit::kQ + q], heat.log2);
        part[(int64_t)tp * stride + q0 + q] = make_float2(st.m, st.s);
    }
}

// The rows' losses and stats from the tiles': 16 rows a workgroup, 16 threads a row.
__global__ __launch_bounds__(256) void k_ce_loss(CeRows a, CePacked x, int vocab, int tiles,
                                                 const float2 *part, int64_t stride, Heat heat,
                                                 float *loss, float2 *stats)
{
    __shared__ float2 joint[16][16];
    const int r = threadIdx.x & 15, k = threadIdx.x >> 4;
    const int64_t row = (int64_t)blockIdx.x * 16 + r;
    const int at = row < a.rows ? x.place[row] : -1;
    RowStats st = {-INFINITY, 0.0f, 0.0f};
    if (at >= 0)
        for (int i = k; i < tiles; i += 16)
            join_stats(st, part[(int64_t)i * stride + at], heat.log2);
    joint[k][r] = make_float2(st.m, st.s);
    __syncthreads();
    if (k > 0 || row >= a.rows)
        return;
    if (at < 0) {
        loss[row] = 0.0f;
        stats[row] = make_float2(0.0f, 1.0f);
        return;
    }
    for (int i = 1; i < 16; ++i)
        join_stats(st, joint[i][r], heat.log2);
    const int target = a.targets[row];
    const float l = target < vocab ? -log_q(x.at_target[at], st, heat) : NAN;
    loss[row] = (a.weight ? a.weight[row] : 1.0f) * l;
    stats[row] = make_float2(st.m, st.s);
}

// ---- gradients -------------------------------------------------------------------

// dz of a piece of the vocabulary, [rows][width] in bf16; zero behind the last row (up
// to the tile's end) and the last of the vocabulary.
__global__ __launch_bounds__(Logit::kThreads, 1) void k_ce_dlogits(CeWeight w, CeRows a,
                                                                   CePacked x, Heat heat,
                                                                   const float2 *stats, int piece0,
                                                                   int width, u16 *dz, int ld)
{
    __shared__ __align__(16) uint8_t lds[Logit::kLds];
    const int count = *x.count;
    const int np = (min(width, w.vocab - piece0) + Logit::kP - 1) / Logit::kP, nq = (count + Logit::kQ - 1) / Logit::kQ;
    if ((int)blockIdx.x >= np * nq)
        return;
    int tp, tq;
    product_tile(blockIdx.x, np, nq, tp, tq);
    const int p0 = piece0 + tp * Logit::kP, q0 = tq * Logit::kQ;
    Logit t;
    logits(t, lds, w, x, p0, count, q0);
#pragma unroll
    for (int j = 0; j < Logit::NQ; ++j) {
        const int q = q0 + t.q_of(j);
        const bool in = q < count;
        const int row = in ? x.row[q] : 0;
        const int target = in ? a.targets[row] : -1;
        const float2 st = in ? stats[row] : make_float2(0.0f, 1.0f);
        float scale = in ? (a.weight ? a.weight[row] : 1.0f) * heat.inv : 0.0f;
        if (target >= w.vocab)
            scale = NAN;
        const float base = base_of(st.x);
        const float inv = st.y == 0.0f ? 0.0f : scale / st.y;
        u16 *to = dz + (int64_t)q * ld + tp * Logit::kP;
#pragma unroll
        for (int i = 0; i < Logit::NP; ++i) {
            float d[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int p = p0 + t.p_of(i) + r;
                d[r] = __builtin_amdgcn_exp2f((t.acc[i][j][r] - base) * heat.log2) * inv;
                d[r] -= p == target ? scale : 0.0f;
                d[r] = in && p < w.vocab ? d[r] : 0.0f;
            }
            *reinterpret_cast<gv2u *>(to + t.p_of(i)) = (gv2u){pack_bf16(d[0], d[1]), pack_bf16(d[2], d[3])};
        }
    }
}

using Dx = Product<2, 4, 8, 4, false, true>;

// A part of dx = dz w: the products of a stretch of the piece's vocabulary, added to
// (or, for the first piece, written as) slab blockIdx.y of fp32 sums.
__global__ __launch_bounds__(Dx::kThreads, 1) void k_ce_dx(CeWeight w, CePacked x, int piece0,
                                                           int width, int steps, const u16 *dz, int ld,
                                                           float *sums, int64_t slab, int add)
{
    __shared__ __align__(16) uint8_t lds[Dx::kLds];
    const int count = *x.count;
    const int np = (w.hidden + Dx::kP - 1) / Dx::kP, nq = (count + Dx::kQ - 1) / Dx::kQ;
    if ((int)blockIdx.x >= np * nq)
        return;
    int tp, tq;
    product_tile(blockIdx.x, np, nq, tp, tq);
    const int p0 = tp * Dx::kP, q0 = tq * Dx::kQ;
    const int v0 = (int)blockIdx.y * steps * kStepK;
    const int have = min(width, w.vocab - piece0) - v0;  // of the stretch's vocabulary
    const int n = max(0, min(steps, (have + kStepK - 1) / kStepK));
    Dx t;
    const uint8_t *p = reinterpret_cast<const uint8_t *>(w.w + (int64_t)(piece0 + v0) * w.ld + p0);
    const uint8_t *q = reinterpret_cast<const uint8_t *>(dz + (int64_t)q0 * ld + v0);
    t.start(lds, w.ld, w.hidden - p0, ld, Dx::kQ, max(0, have));
    t.run(n, p, kStepK * 2 * (uint32_t)w.ld, q, kStepK * 2);
    float *to = sums + blockIdx.y * slab;
#pragma unroll
    for (int j = 0; j < Dx::NQ; ++j)
#pragma unroll
        for (int i = 0; i < Dx::NP; ++i) {
            const int q1 = q0 + t.q_of(j), p1 = p0 + t.p_of(i);
            if (q1 < count && p1 < w.hidden) {
                v4f *at = reinterpret_cast<v4f *>(to + (int64_t)q1 * w.hidden + p1);
                *at = add ? *at + t.acc[i][j] : t.acc[i][j];
            }
        }
}

// dx from the slabs of sums, every row of it
__global__ __launch_bounds__(256) void k_ce_dx_rows(int64_t rows, int hidden, const int *place,
                                                    const float *sums, int64_t slab, int slabs,
                                                    bf16_t *dx, int64_t ld)
{
    const int64_t r = blockIdx.x;
    const int at = place[r];
    for (int c = threadIdx.x * 4; c < hidden; c += 256 * 4) {
        v4f v = {0.f, 0.f, 0.f, 0.f};
        if (at >= 0)
            for (int s = 0; s < slabs; ++s)
                v += *reinterpret_cast<const v4f *>(sums + s * slab + (int64_t)at * hidden + c);
        const float f[4] = {v[0], v[1], v[2], v[3]};
        store_vec(dx + r * ld + c, f);
    }
}

using Dw = Product<2, 4, 8, 4, false, false>;

// dw = dz^T x of a piece of the vocabulary
__global__ __launch_bounds__(Dw::kThreads, 1) void k_ce_dw(CeWeight w, CePacked x, int piece0,
                                                           int width, const u16 *dz, int ld,
                                                           u16 *dw, int64_t ld_dw)
{
    __shared__ __align__(16) uint8_t lds[Dw::kLds];
    const int np = (w.hidden + Dw::kP - 1) / Dw::kP;
    const int have = min(width, w.vocab - piece0);
    const int nq = (have + Dw::kQ - 1) / Dw::kQ;
    int tp, tq;
    product_tile(blockIdx.x, np, nq, tp, tq);
    const int p0 = tp * Dw::kP, q0 = tq * Dw::kQ;
    Dw t;
    t.start(lds, x.ld, x.ld - p0, ld, width - q0, kStepK);
    const uint8_t *p = reinterpret_cast<const uint8_t *>(x.x + p0);
    const uint8_t *q = reinterpret_cast<const uint8_t *>(dz + q0);
    t.run((*x.count + kStepK - 1) / kStepK, p, kStepK * 2 * x.ld, q, kStepK * 2 * ld);
#pragma unroll
    for (int j = 0; j < Dw::NQ; ++j)
#pragma unroll
        for (int i = 0; i < Dw::NP; ++i) {
            const int q1 = q0 + t.q_of(j), p1 = p0 + t.p_of(i);
            if (q1 < have && p1 < w.hidden)
                *reinterpret_cast<gv2u *>(dw + (int64_t)(piece0 + q1) * ld_dw + p1) =
                    (gv2u){pack_bf16(t.acc[i][j][0], t.acc[i][j][1]), pack_bf16(t.acc[i][j][2], t.acc[i][j][3])};
        }
}

// ---- the host's side -------------------------------------------------------------

constexpr int64_t kMostRows = INT32_MAX - 255;
constexpr int64_t kMostLd = int64_t(1) << 22;  // 256 rows of it: an offset of 32 bits

int64_t up(int64_t n, int64_t to) { return (n + to - 1) / to * to; }

// Pieces of a workspace, each from a 256-byte boundary
struct Carve {
    uint8_t *at;
    size_t used = 0;
    template <class T> T *take(int64_t n)
    {
        T *p = reinterpret_cast<T *>(at + used);
        used += (size_t)up(n * (int64_t)sizeof(T), 256);
        return p;
    }
};

// A leading dimension of workspace rows of n values: not a multiple of 2 KiB, whose lines of
// one k would share the L2's channels.  x.ld counts them in the zeros behind a row's values.
int64_t pitch(int64_t n) { return n % 1024 ? n : n + kStepK; }

CePacked take_packed(Carve &c, int64_t rows, int64_t hidden)
{
    CePacked x;
    x.count = c.take<int>(1);
    x.place = c.take<int>(rows);
    x.row = c.take<int>(rows);
    x.at_target = c.take<float>(rows);
    x.ld = (int)pitch(up(hidden, kStepK));
    x.x = c.take<u16>(up(rows, kStepK) * x.ld);
    return x;
}

struct ForwardPlan {
    CePacked x;
    float2 *part;
    int64_t tiles, stride;
    size_t bytes;
};
ForwardPlan forward_plan(int64_t rows, int64_t hidden, int64_t vocab, void *ws)
{
    ForwardPlan f;
    Carve c = {static_cast<uint8_t *>(ws)};
    f.x = take_packed(c, rows, hidden);
    f.tiles = (vocab + Logit::kP - 1) / Logit::kP;
    f.stride = up(rows, 16);
    f.part = c.take<float2>(f.tiles * f.stride);
    f.bytes = c.used;
    return f;
}

struct BackwardPlan {
    CePacked x;
    u16 *dz;
    float *sums;
    int64_t width, ld, pieces, slab, slabs, steps;
    size_t bytes;
};
BackwardPlan backward_plan(int64_t rows, int64_t hidden, int64_t vocab, void *ws)
{
    BackwardPlan b;
    Carve c = {static_cast<uint8_t *>(ws)};
    b.x = take_packed(c, rows, hidden);
    // a piece's dz stays in the last-level cache for the two products that read it
    const int64_t padded = up(rows > 0 ? rows : 1, Logit::kQ), most = up(vocab, Logit::kP);
    int64_t width = (int64_t(1) << 26) / padded / Logit::kP * Logit::kP;
    width = width < Logit::kP ? Logit::kP : width < most ? width : most;
    b.pieces = (vocab + width - 1) / width;
    b.width = up((vocab + b.pieces - 1) / b.pieces, Logit::kP);
    b.pieces = (vocab + b.width - 1) / b.width;
    b.ld = pitch(b.width);
    b.dz = c.take<u16>(padded * b.ld);
    // the vocabulary in stretches until the products for dx fill the chip
    const int64_t tiles = (hidden + Dx::kP - 1) / Dx::kP * (padded / Dx::kQ);
    const int64_t room = b.width / 512 > 0 ? b.width / 512 : 1;
    b.slabs = tiles >= 256 ? 1 : 256 / tiles < room ? 256 / tiles : room;
    b.steps = (b.width / kStepK + b.slabs - 1) / b.slabs;
    b.slab = rows * hidden;
    b.sums = c.take<float>(b.slab * b.slabs);
    b.bytes = c.used;
    return b;
}

bool sizes_ok(int64_t rows, int64_t hidden, int64_t vocab)
{
    return rows >= 0 && rows <= kMostRows && vocab >= 1 && vocab <= kMaxVocab - 256 &&
           hidden >= 32 && hidden % 32 == 0 && hidden <= kMostLd;
}

mxq_status check(const void *x, int64_t ld_x, const void *w, int64_t ld_w, int64_t rows,
                 int64_t hidden, int64_t vocab, float temperature, const int32_t *targets,
                 const float *weight)
{
    if (!(temperature >= FLT_MIN) || !(temperature < INFINITY))
        return MXQ_ERR_UNSUPPORTED;
    if (!sizes_ok(rows, hidden, vocab) || ld_x < hidden || ld_w < hidden || ld_w > kMostLd)
        return MXQ_ERR_SHAPE;
    if (!w || (rows > 0 && (!x || !targets)))
        return MXQ_ERR_NULL;
    if (reinterpret_cast<uintptr_t>(x) % 2 || reinterpret_cast<uintptr_t>(w) % 16 || ld_w % 8 ||
        !aligned4(targets) || !aligned4(weight))
        return MXQ_ERR_ALIGN;
    return MXQ_OK;
}

void launch_pack(const CeRows &a, const void *x, int64_t ld, int64_t hidden, const CePacked &to,
                 hipStream_t s)
{
    // 16 rows a workgroup, more where counting the rows in front would cost more than that
    const int64_t per = up(a.rows / 1024 < 16 ? 16 : a.rows / 1024, 16);
    const int64_t groups = a.rows > 0 ? (a.rows + per - 1) / per : 1;
    hipLaunchKernelGGL(k_ce_pack, dim3((unsigned)groups), dim3(kPackThreads), 0, s, a, per,
                       static_cast<const bf16_t *>(x), ld, (int)hidden, to);
}

}  // namespace
}  // namespace mxq

using namespace mxq;

extern "C" size_t mxq_linear_ce_forward_workspace_size(int64_t rows, int64_t hidden, int64_t vocab)
{
    return rows > 0 && sizes_ok(rows, hidden, vocab) ? forward_plan(rows, hidden, vocab, nullptr).bytes : 0;
}

extern "C" size_t mxq_linear_ce_backward_workspace_size(int64_t rows, int64_t hidden, int64_t vocab)
{
    return sizes_ok(rows, hidden, vocab) ? backward_plan(rows, hidden, vocab, nullptr).bytes : 0;
}

extern "C" mxq_status mxq_linear_ce_forward(const void *x, int64_t ld_x, const void *w,
                                            int64_t ld_w, int64_t rows, int64_t hidden,
                                            int64_t vocab, float temperature,
                                            const int32_t *targets, const float *weight,
                                            float *loss, float *stats, void *workspace,
                                            size_t ws_bytes, void *stream)
{
    const mxq_status st = check(x, ld_x, w, ld_w, rows, hidden, vocab, temperature, targets, weight);
    if (st)
        return st;
    if (rows == 0)
        return MXQ_OK;
    if (!loss || !stats)
        return MXQ_ERR_NULL;
    if (!aligned4(loss) || reinterpret_cast<uintptr_t>(stats) % 8 ||
        reinterpret_cast<uintptr_t>(workspace) % 16)
        return MXQ_ERR_ALIGN;
    const ForwardPlan f = forward_plan(rows, hidden, vocab, workspace);
    if (!workspace || ws_bytes < f.bytes)
        return MXQ_ERR_WORKSPACE;
    const int64_t groups = f.tiles * ((rows + Logit::kQ - 1) / Logit::kQ);
    if (groups > INT32_MAX)
        return MXQ_ERR_SHAPE;
    hipStream_t s = static_cast<hipStream_t>(stream);
    const CeRows a = {targets, weight, rows};
    const CeWeight cw = {static_cast<const u16 *>(w), ld_w, (int)vocab, (int)hidden};
    const Heat heat = heat_of(temperature);
    launch_pack(a, x, ld_x, hidden, f.x, s);
    hipLaunchKernelGGL(k_ce_stats, dim3((unsigned)groups), dim3(Logit::kThreads), 0, s, cw, a, f.x,
                       heat, f.part, f.stride);
    hipLaunchKernelGGL(k_ce_loss, dim3((unsigned)((rows + 15) / 16)), dim3(256), 0, s, a, f.x,
                       (int)vocab, (int)f.tiles, f.part, f.stride, heat, loss,
                       reinterpret_cast<float2 *>(stats));
    return launched();
}

extern "C" mxq_status mxq_linear_ce_backward(const void *x, int64_t ld_x, const void *w,
                                             int64_t ld_w, int64_t rows, int64_t hidden,
                                             int64_t vocab, float temperature,
                                             const int32_t *targets, const float *weight,
                                             const float *stats, void *dx, int64_t ld_dx, void *dw,
                                             int64_t ld_dw, void *workspace, size_t ws_bytes,
                                             void *stream)
{
    const mxq_status st = check(x, ld_x, w, ld_w, rows, hidden, vocab, temperature, targets, weight);
    if (st)
        return st;
    if ((dx && ld_dx < hidden) || (dw && (ld_dw < hidden || ld_dw > kMostLd)))
        return MXQ_ERR_SHAPE;
    if ((rows > 0 && !stats) || (!dx && !dw && rows > 0))
        return MXQ_ERR_NULL;
    if (reinterpret_cast<uintptr_t>(stats) % 8 || reinterpret_cast<uintptr_t>(dx) % 2 ||
        reinterpret_cast<uintptr_t>(dw) % 16 || (dw && ld_dw % 8) ||
        reinterpret_cast<uintptr_t>(workspace) % 16)
        return MXQ_ERR_ALIGN;
    if (!dw && rows == 0)
        return MXQ_OK;
    const BackwardPlan b = backward_plan(rows, hidden, vocab, workspace);
    if (!workspace || ws_bytes < b.bytes)
        return MXQ_ERR_WORKSPACE;
    const int64_t nq = (rows + Logit::kQ - 1) / Logit::kQ;
    const int64_t z_groups = b.width / Logit::kP * nq;
    const int64_t x_tiles = (hidden + Dx::kP - 1) / Dx::kP * nq;
    if (z_groups > INT32_MAX || x_tiles > INT32_MAX)
        return MXQ_ERR_SHAPE;
    hipStream_t s = static_cast<hipStream_t>(stream);
    const CeRows a = {targets, weight, rows};
    const CeWeight cw = {static_cast<const u16 *>(w), ld_w, (int)vocab, (int)hidden};
    const Heat heat = heat_of(temperature);
    launch_pack(a, x, ld_x, hidden, b.x, s);
    for (int64_t i = 0; i < b.pieces; ++i) {
        const int piece0 = (int)(i * b.width);
        const int64_t have = vocab - piece0 < b.width ? vocab - piece0 : b.width;
        const int64_t w_tiles = (hidden + Dw::kP - 1) / Dw::kP * ((have + Dw::kQ - 1) / Dw::kQ);
        if (rows > 0) {
            const int64_t np = (have + Logit::kP - 1) / Logit::kP;
            hipLaunchKernelGGL(k_ce_dlogits, dim3((unsigned)(np * nq)), dim3(Logit::kThreads), 0, s,
                               cw, a, b.x, heat, reinterpret_cast<const float2 *>(stats), piece0,
                               (int)b.width, b.dz, (int)b.ld);
            if (dx)
                hipLaunchKernelGGL(k_ce_dx, dim3((unsigned)x_tiles, (unsigned)b.slabs),
                                   dim3(Dx::kThreads), 0, s, cw, b.x, piece0, (int)b.width,
                                   (int)b.steps, b.dz, (int)b.ld, b.sums, b.slab, i > 0);
        }
        if (dw)
            hipLaunchKernelGGL(k_ce_dw, dim3((unsigned)w_tiles), dim3(Dw::kThreads), 0, s, cw, b.x,
                               piece0, (int)b.width, b.dz, (int)b.ld, static_cast<u16 *>(dw), ld_dw);
    }
    if (dx && rows > 0)
        hipLaunchKernelGGL(k_ce_dx_rows, dim3((unsigned)rows), dim3(256), 0, s, rows, (int)hidden,
                           b.x.place, b.sums, b.slab, (int)b.slabs, static_cast<bf16_t *>(dx),
                           ld_dx);
    return launched();
}
