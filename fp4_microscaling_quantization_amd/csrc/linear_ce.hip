// Softmax cross entropy from the hidden states and the output layer's weight, without
// the logits z = x w^T ever being in memory.
//
//   forward   a tile of logits stays in the registers of the product; each row leaves
//             its maximum m and sum s = sum exp((z - m) / T) over the tile's vocabulary,
//             and a second kernel joins them over the tiles.
//   backward  a piece of the vocabulary at a time: the product again, turned into
//             dz = weight / T (exp((z - m) / T) / s - 1[v = target]) in bf16, which the two
//             products dx += dz w and dw = dz^T x then read; what the rounding of dz left at
//             the targets is added to both.
//
// Rows that do not count are left out of all of it: the rows that do are packed first.
//
// Few rows are bound by the weight's bytes, many by the matrix cores.  24 rows under
// 128256 x 4096: forward 183 us, 5.7 TB/s.  16 under 32003 x 4096: backward 167 us, of it
// dz 40 (6.6 TB/s), dx 43, dw 60 (written at 4.4).  8192 rows, of which 7373 count, under
// 128256 x 4096: forward 5.5 ms (1.40 PF); backward 17.7 ms, of it dz 5.8 (1.34 PF), dx 6.2
// (1.25), dw 5.5 (1.41), packing, sums and the join of dx 0.1.
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
    int all;           // >= 0: no rows are packed, these are all of them, in their places
    int *count;        // rows that count
    int *place;        // [rows]: a row's place among them, -1: none
    int *row;          // [count]
    float *at_target;  // [count]: the logit at the target
    u16 *x;            // [count, up to a whole step][ld], zero behind both
    int ld;            // hidden, up to a whole step
};

__device__ __forceinline__ bool row_counts(const CeRows &a, int64_t r)
{
    const int target = a.targets[r];
    const float weight = a.weight ? a.weight[r] : 1.0f;  // both are on their way
    return (target >= 0) & (weight != 0.0f);
}

// dz is rounded to bf16 for the products behind it.  The largest entry of most rows is the one
// at the target, near -weight / T: its rounding would be most of what is off in dx and dw, and
// with all weights alike and most q small it would be off by the same up to 0.4% in every row.  So
// what that one entry's rounding left is kept in fp32, and its part of dx and dw is added to their
// sums.  (1351 rows under 50257 x 1600 at a temperature of 0.7: dx and dw are off by 0.31% in the mean
// without it, by 0.17% with it, as fp32 products are: it is their own rounding.  It takes 8 us of 685, and
// of 17.7 ms for 7373 rows under 128256 x 4096 less than can be told.)
__device__ __forceinline__ float rounding_left(float d)
{
    const float stored = (float)(bf16_t)d;
    return fabsf(stored) < INFINITY ? d - stored : 0.0f;
}
// rest times a value of the other operand.  The rounded entry's product has the infinities and NaN.
__device__ __forceinline__ float rest_of(float rest, float other)
{
    return fabsf(other) < INFINITY ? rest * other : 0.0f;
}

// the statistics of two stretches of a row, as one
__device__ __forceinline__ void join_stats(RowStats &st, float2 o, float log2)
{
    const float m = fmaxf(st.m, o.x), base = base_of(m);
    st.s = fmaf(st.s, __builtin_amdgcn_exp2f((st.m - base) * log2),
                o.y * __builtin_amdgcn_exp2f((o.x - base) * log2));
    st.m = m;
}

// ---- packing ---------------------------------------------------------------------

constexpr int kPackThreads = 256;

// The sum over the workgroup of a count
__device__ __forceinline__ int block_count(int n)
{
    __shared__ int partial[kPackThreads / 64];
    for (int d = 1; d < 64; d *= 2)
        n += __shfl_xor(n, d);
    if ((threadIdx.x & 63) == 0)
        partial[threadIdx.x >> 6] = n;
    __syncthreads();
    n = 0;
    for (int w = 0; w < kPackThreads / 64; ++w)
        n += partial[w];
    return n;
}

// Rows by their targets, for what Rests adds to dw: those with their target in a tile of dw are
// neighbours in a list, in order.  A workgroup makes one tile's part: it counts all rows, those in
// the tile and those in front of it, a quarter of the rows a wave, then goes through them once more.
// A row whose target is beyond the vocabulary is in no list, and one with every logit masked is not
// either: it may hold infinities, which times the zeros of other entries would be none.  (x of the others is
// finite: an infinity there makes every logit infinite, and the row has no distribution.)
struct CeTargets {
    int tiles, shift, vocab;  // of dw, 1 << shift entries wide
    const float2 *stats;
    int *rows, *starts;
};
__device__ __forceinline__ void list_targets(const CeRows &a, const CeTargets &to, int tile)
{
    constexpr int WAVES = kPackThreads / 64;
    __shared__ int sums[3][WAVES];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t part = (a.rows + WAVES * 64 - 1) / (WAVES * 64) * 64;
    const int64_t first = wave * part, end = first + part < a.rows ? first + part : a.rows;
    const uint64_t below = (1ull << lane) - 1;
    int counts = 0, here = 0, before = 0;
    // f(which of 64 rows count, are in the tile, are in front of it), `ahead` times 64 rows in flight
    const auto go_by = [&](auto ahead, auto f) {
        constexpr int AHEAD = decltype(ahead)::value;
        for (int64_t base = first; base < end; base += AHEAD * 64) {
            int target[AHEAD];
            float weight[AHEAD], s[AHEAD];
#pragma unroll
            for (int u = 0; u < AHEAD; ++u) {
                const int64_t at = base + u * 64 + lane, r = at < end ? at : end - 1;
                target[u] = at < end ? a.targets[r] : -1;
                weight[u] = a.weight ? a.weight[r] : 1.0f;
                s[u] = to.stats[r].y;
            }
#pragma unroll
            for (int u = 0; u < AHEAD; ++u) {
                const bool in = (target[u] >= 0) & (weight[u] != 0.0f);
                const bool ok = in & (target[u] < to.vocab) & (s[u] != 0.0f);
                f(__ballot(in), __ballot(ok && target[u] >> to.shift == tile),
                  __ballot(ok && target[u] >> to.shift < tile));
            }
        }
    };
    const auto go = [&](auto f) {
        if (part == 64)
            go_by(std::integral_constant<int, 1>{}, f);
        else
            go_by(std::integral_constant<int, 4>{}, f);
    };
    go([&](uint64_t in, uint64_t mine, uint64_t front) {
        counts += __popcll(in);
        here += __popcll(mine);
        before += __popcll(front);
    });
    if (lane == 0) {
        sums[0][wave] = counts;
        sums[1][wave] = here;
        sums[2][wave] = before;
    }
    __syncthreads();
    int start = 0, all = 0;
    counts = here = 0;
    for (int w = 0; w < WAVES; ++w) {
        start += sums[2][w];
        all += sums[1][w];
        counts += w < wave ? sums[0][w] : 0;
        here += w < wave ? sums[1][w] : 0;
    }
    if (threadIdx.x == 0) {
        to.starts[tile] = start;
        if (tile == to.tiles - 1)
            to.starts[tile + 1] = start + all;
    }
    if (all == 0)
        return;
    go([&](uint64_t in, uint64_t mine, uint64_t) {
        if (mine >> lane & 1)
            to.rows[start + here + __popcll(mine & below)] = counts + __popcll(in & below);
        counts += __popcll(in);
        here += __popcll(mine);
    });
}

// The rows that count, in order: where each went (or -1), which it was, how many, and
// their values, with zeros behind the last value up to a whole step.  A workgroup takes
// `per` rows, and finds their place by counting all rows in front of them.  The kStepK - 1
// behind `groups` write zeros behind the last row up to a whole step, which the product
// over the rows reads, a row each.  The ones behind those list rows by their targets (list_targets).
__global__ __launch_bounds__(kPackThreads) void k_ce_pack(CeRows a, int64_t per, int groups,
                                                          const bf16_t *x, int64_t ld, int hidden,
                                                          CePacked to, CeTargets lists)
{
    const int lane = threadIdx.x & 63;
    if ((int)blockIdx.x >= groups + kStepK - 1) {
        list_targets(a, lists, (int)blockIdx.x - (groups + kStepK - 1));
        return;
    }
    const bool behind = (int)blockIdx.x >= groups;
    const int64_t first = behind ? a.rows : (int64_t)blockIdx.x * per;
    const int64_t end = first + per < a.rows ? first + per : a.rows;
    int place = 0;
#pragma unroll 8
    for (int64_t r = threadIdx.x; r < first; r += kPackThreads)
        place += row_counts(a, r);
    place = block_count(place);
    if (behind) {
        const int row = place + (int)blockIdx.x - groups;
        if (row < (place + kStepK - 1) / kStepK * kStepK)
            for (int c = threadIdx.x * 8; c < to.ld; c += kPackThreads * 8)
                *reinterpret_cast<gv4u *>(to.x + (int64_t)row * to.ld + c) = (gv4u){0u, 0u, 0u, 0u};
        return;
    }
    for (int64_t base = first; base < end; base += 64) {
        // every wave works out the same
        const int64_t mine = base + lane;
        const bool in = mine < end && row_counts(a, mine);
        const uint64_t all = __ballot(in);
        const int at = place + __popcll(all & ((1ull << lane) - 1));
        if (threadIdx.x < 64 && mine < end) {
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
    if ((int)blockIdx.x == groups - 1 && threadIdx.x == 0)
        *to.count = place;
}

// ---- logits ----------------------------------------------------------------------

// Tiles, p x q.  Many: for products that fill the chip with them.  CUT, ONCE: P_CUT, P_ONCE.
template <bool P_ALONG, bool Q_ALONG, bool CUT>
using Many = Product<2, 4, 8, 4, 2, P_ALONG, Q_ALONG, CUT>;  // 256 x 256
// For those that do not: half as large, and a step more in flight.
template <bool P_ALONG, bool Q_ALONG, bool CUT>
using Half = Product<2, 4, 4, 4, 3, P_ALONG, Q_ALONG, CUT>;  // 128 x 256
// A quarter: one to a CU with four steps in LDS, two with two.
template <bool P_ALONG, bool Q_ALONG, bool CUT, bool ONCE = false>
using Deep = Product<4, 2, 2, 4, 4, P_ALONG, Q_ALONG, CUT, ONCE>;  // 128 x 128
template <bool P_ALONG, bool Q_ALONG, bool CUT, bool ONCE = false>
using Twin = Product<4, 1, 2, 8, 2, P_ALONG, Q_ALONG, CUT, ONCE>;  // 128 x 128
// Few rows, where the weight is what there is to read.  (16 rows under 32003 x 4096 56 us with
// three or four steps in LDS, 69 with two.)
template <bool P_ALONG, bool Q_ALONG, bool CUT, bool ONCE = false>
using Few = Product<4, 1, 2, 2, 3, P_ALONG, Q_ALONG, CUT, ONCE>;  // 128 x 32
// Products of so few tiles that each has a CU, or half of one, to itself: what they take is the
// time of their steps one after another, and a smaller tile's are shorter.
template <bool P_ALONG, bool Q_ALONG, bool CUT, bool ONCE = false>
using Small = Product<2, 2, 2, 2, 4, P_ALONG, Q_ALONG, CUT, ONCE>;  // 64 x 64
template <bool P_ALONG, bool Q_ALONG, bool CUT, bool ONCE = false>
using Slim = Product<4, 1, 1, 2, 6, P_ALONG, Q_ALONG, CUT, ONCE>;  // 64 x 32
// dw of rows that are one step of the product over them
using Outer = Product<2, 2, 4, 4, 1, false, false, false>;  // 128 x 128

// the tile's product: w rows from p0, packed x rows from q0; meanwhile: see Product::run
template <class Tile, class F>
__device__ __forceinline__ void logits(Tile &t, uint8_t *lds, const CeWeight &w,
                                       const CePacked &x, int p0, int count, int q0, F meanwhile)
{
    const int rows = x.all >= 0 ? count : (count + kStepK - 1) / kStepK * kStepK;
    t.start(lds, w.ld, w.vocab - p0, x.ld, rows - q0, w.hidden);
    const uint8_t *p = reinterpret_cast<const uint8_t *>(w.w + (int64_t)p0 * w.ld);
    const uint8_t *q = reinterpret_cast<const uint8_t *>(x.x + (int64_t)q0 * x.ld);
    const int steps = (w.hidden + kStepK - 1) / kStepK;
    t.run(steps, p, kStepK * 2, q, kStepK * 2, (int)(blockIdx.x & 7) * steps / 8, meanwhile);
}

// Maximum and sum of every packed row over the tile's vocabulary, and the logit at its
// target.
template <class Tile>
__global__ __launch_bounds__(Tile::kThreads, 1) void k_ce_stats(CeWeight w, CeRows a, CePacked x,
                                                                Heat heat, float2 *part,
                                                                int64_t stride)
{
    __shared__ __align__(16) uint8_t lds[Tile::kLds];
    const int count = x.all >= 0 ? x.all : *x.count;
    const int np = (w.vocab + Tile::kP - 1) / Tile::kP, nq = (count + Tile::kQ - 1) / Tile::kQ;
    if ((int)blockIdx.x >= np * nq)
        return;
    int tp, tq;
    product_tile(blockIdx.x, np, nq, tp, tq);
    const int p0 = tp * Tile::kP, q0 = tq * Tile::kQ;
    __shared__ int targets[Tile::kQ];  // of the tile's rows, within the tile
    Tile t;
    logits(t, lds, w, x, p0, count, q0, [&] {
        for (int q = threadIdx.x; q < Tile::kQ; q += Tile::kThreads)
            targets[q] = q0 + q < count ? a.targets[x.all >= 0 ? q0 + q : x.row[q0 + q]] - p0 : -1;
    });

    float2 *joint = reinterpret_cast<float2 *>(lds);  // [WP][kQ]
    const bool whole = p0 + Tile::kP <= w.vocab;
#pragma unroll
    for (int j = 0; j < Tile::NQ; ++j) {
        const int q = t.q_of(j);
        const int target = targets[q];
        if (!whole) {
#pragma unroll
            for (int i = 0; i < Tile::NP; ++i)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    if (p0 + t.p_of(i) + r >= w.vocab)
                        t.acc[i][j][r] = -INFINITY;
        }
        // few tiles hold a target of theirs
        if (__any((unsigned)target < (unsigned)Tile::kP)) {
#pragma unroll
            for (int i = 0; i < Tile::NP; ++i)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    if (t.p_of(i) + r == target && p0 + target < w.vocab)
                        x.at_target[q0 + q] = t.acc[i][j][r];
        }
        float m = -INFINITY;
#pragma unroll
        for (int i = 0; i < Tile::NP; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                m = fmaxf(m, t.acc[i][j][r]);
        m = fmaxf(m, __shfl_xor(m, 16));
        m = fmaxf(m, __shfl_xor(m, 32));
        const float base = base_of(m);
        float s[2] = {0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < Tile::NP; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                s[r & 1] += __builtin_amdgcn_exp2f((t.acc[i][j][r] - base) * heat.log2);
        s[0] += s[1];
        s[0] += __shfl_xor(s[0], 16);
        s[0] += __shfl_xor(s[0], 32);
        if (t.lane < 16)
            joint[t.wp * Tile::kQ + q] = make_float2(m, s[0]);
    }
    __syncthreads();
    for (int q = threadIdx.x; q < Tile::kQ && q0 + q < count; q += Tile::kThreads) {
        RowStats st = {joint[q].x, joint[q].y, 0.0f};
        for (int k = 1; k < Tile::WP; ++k)
            join_stats(st, joint[k * Tile::kQ + q], heat.log2);
        part[(int64_t)tp * stride + q0 + q] = make_float2(st.m, st.s);
    }
}

// The rows' losses and stats from the tiles': ROWS rows a workgroup.
template <int ROWS>
__global__ __launch_bounds__(256) void k_ce_loss(CeRows a, CePacked x, int vocab, int tiles,
                                                 const float2 *part, int64_t stride, Heat heat,
                                                 float *loss, float2 *stats)
{
    constexpr int K = 256 / ROWS, WAVES = 4;  // threads of a row
    __shared__ float2 joint[WAVES][ROWS];
    const int r = threadIdx.x % ROWS, k = threadIdx.x / ROWS;
    const int64_t row = (int64_t)blockIdx.x * ROWS + r;
    int at = -1;
    if (row < a.rows)
        at = x.all < 0 ? x.place[row] : row_counts(a, row) ? (int)row : -1;
    RowStats st = {-INFINITY, 0.0f, 0.0f};
    if (at >= 0) {
        constexpr int AHEAD = 4;
        int i = k;
        for (; i + (AHEAD - 1) * K < tiles; i += AHEAD * K) {
            float2 p[AHEAD];
#pragma unroll
            for (int u = 0; u < AHEAD; ++u)
                p[u] = part[(int64_t)(i + u * K) * stride + at];
#pragma unroll
            for (int u = 0; u < AHEAD; ++u)
                join_stats(st, p[u], heat.log2);
        }
        for (; i < tiles; i += K)
            join_stats(st, part[(int64_t)i * stride + at], heat.log2);
    }
#pragma unroll
    for (int d = ROWS; d < 64; d *= 2)
        join_stats(st, make_float2(__shfl_xor(st.m, d), __shfl_xor(st.s, d)), heat.log2);
    if ((threadIdx.x & 63) < ROWS)
        joint[threadIdx.x >> 6][r] = make_float2(st.m, st.s);
    __syncthreads();
    if (k > 0 || row >= a.rows)
        return;
#pragma unroll
    for (int w = 1; w < WAVES; ++w)
        join_stats(st, joint[w][r], heat.log2);
    if (at < 0) {
        loss[row] = 0.0f;
        stats[row] = make_float2(0.0f, 1.0f);
        return;
    }
    const int target = a.targets[row];
    const float l = target < vocab ? -log_q(x.at_target[at], st, heat) : NAN;
    loss[row] = (a.weight ? a.weight[row] : 1.0f) * l;
    stats[row] = make_float2(st.m, st.s);
}

// ---- gradients -------------------------------------------------------------------

// The backward pass over pieces of `width` of the vocabulary
struct Backward {
    CeWeight w;
    CeRows a;
    CePacked x;
    Heat heat;
    const float2 *stats;
    int width, ld;   // of dz
    u16 *dz;         // of a piece, [rows][ld]
    int *by_target;  // [count]: packed rows by their targets' tiles of dw, in order within each
    int *starts;     // [tiles and one]: where in it a tile's begin
    int4 *left;      // [count]: a row's target, and what the rounding of dz left there (fp32)
    float *sums;     // slabs of [count][hidden]
    int fill, room;  // workgroups that fill the chip, and most slabs
    u16 *dw;
    int64_t ld_dw;

    __device__ __forceinline__ int first(int piece) const { return piece * width; }
    __device__ __forceinline__ int have(int piece) const
    {
        return min(width, w.vocab - first(piece));
    }
};

// The products for dx are split over stretches of a piece's vocabulary until they fill the
// chip; each stretch has its own slab of sums.  How many rows count is only known here.
__host__ __device__ __forceinline__ int slabs_of(int tiles, int fill, int room)
{
    return tiles >= fill ? 1 : max(1, min(fill / max(1, tiles), room));
}

// Tile `at` of the piece's dz, [rows][ld] in bf16; zero behind the last row (up to the
// tile's end, and a whole step) and the last of the vocabulary.
template <class Tile>
__device__ __forceinline__ void dlogits(uint8_t *lds, const Backward &b, int piece, int at)
{
    const int count = *b.x.count;
    const int np = (b.have(piece) + Tile::kP - 1) / Tile::kP;
    const int nq = (count + Tile::kQ - 1) / Tile::kQ;
    if (at >= np * nq)
        return;
    int tp, tq;
    product_tile(at, np, nq, tp, tq);
    const int p0 = b.first(piece) + tp * Tile::kP, q0 = tq * Tile::kQ;
    // what the tile's rows take: the maximum, weight / (T s), weight / T and the target within the
    // tile
    __shared__ float4 rows_of[Tile::kQ];
    Tile t;
    logits(t, lds, b.w, b.x, p0, count, q0, [&] {
        for (int q = threadIdx.x; q < Tile::kQ; q += Tile::kThreads) {
            float4 v = make_float4(0.0f, 0.0f, 0.0f, __int_as_float(-1));
            if (q0 + q < count) {
                const int row = b.x.row[q0 + q];
                const int target = b.a.targets[row];
                const float2 st = b.stats[row];
                float scale = (b.a.weight ? b.a.weight[row] : 1.0f) * b.heat.inv;
                const bool foreign = target >= b.w.vocab;
                if (foreign)
                    scale = NAN;
                // (q is 0 in a row with every logit masked, NaN in one with a foreign target)
                v = make_float4(base_of(st.x), st.y == 0.0f && !foreign ? 0.0f : scale / st.y,
                                scale, __int_as_float(target - p0));
            }
            rows_of[q] = v;
        }
    });
    const bool whole = p0 + Tile::kP <= b.w.vocab;
#pragma unroll
    for (int j = 0; j < Tile::NQ; ++j) {
        const bool in = q0 + t.q_of(j) < count;
        const float4 row = rows_of[t.q_of(j)];
        const float base = row.x, inv = row.y, scale = row.z;
        const int target = __float_as_int(row.w);
        const bool near = __any((unsigned)target < (unsigned)Tile::kP);
        bool found = false;
        float rest = 0.0f;
#pragma unroll
        for (int i = 0; i < Tile::NP; ++i) {
            float d[4];
#pragma unroll
            for (int r = 0; r < 4; ++r)
                d[r] = __builtin_amdgcn_exp2f((t.acc[i][j][r] - base) * b.heat.log2) * inv;
            if (near) {
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    if (t.p_of(i) + r == target) {
                        d[r] -= scale;
                        rest = rounding_left(d[r]);
                        found = true;
                    }
            }
            if (!whole || q0 + Tile::kQ > count) {
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    d[r] = in && p0 + t.p_of(i) + r < b.w.vocab ? d[r] : 0.0f;
            }
            t.put(lds, i, j, (gv2u){pack_bf16(d[0], d[1]), pack_bf16(d[2], d[3])});
        }
        if (found)
            b.left[q0 + t.q_of(j)] = make_int4(p0 + target, __float_as_int(rest), 0, 0);
    }
    u16 *to = b.dz + (int64_t)q0 * b.ld + tp * Tile::kP;
    t.template flush<false>(lds, to, b.ld, Tile::kQ, Tile::kP);
    // what is left of a step behind the last tile
    if constexpr (Tile::kQ < kStepK) {
        constexpr int WIDE = Tile::kP / 8;
        const int rows = (count + kStepK - 1) / kStepK * kStepK;
        if (tq == nq - 1)
            for (int q = Tile::kQ + threadIdx.x / WIDE; q < rows - q0; q += Tile::kThreads / WIDE)
                *reinterpret_cast<gv4u *>(to + (int64_t)q * b.ld + threadIdx.x % WIDE * 8) =
                    (gv4u){0u, 0u, 0u, 0u};
    }
}

// Tile `at` of all slabs' for dx = dz w, added to (for the first piece, written as) the sums.
template <class Tile>
__device__ __forceinline__ void dx_part(uint8_t *lds, const Backward &b, int piece, int at)
{
    const int count = *b.x.count;
    const int np = (b.w.hidden + Tile::kP - 1) / Tile::kP, nq = (count + Tile::kQ - 1) / Tile::kQ;
    const int slabs = slabs_of(np * nq, b.fill, b.room);
    const int slab = at / max(1, np * nq);
    if (slab >= slabs || nq == 0)
        return;
    at -= slab * np * nq;
    int tp, tq;
    product_tile(at, np, nq, tp, tq);
    const int p0 = tp * Tile::kP, q0 = tq * Tile::kQ;
    const int steps = (b.width / kStepK + slabs - 1) / slabs;
    const int v0 = slab * steps * kStepK;
    const int have = b.have(piece) - v0;  // of the stretch's vocabulary, to the piece's end
    const int n = max(0, min(steps, (have + kStepK - 1) / kStepK));
    Tile t;
    const uint8_t *p =
        reinterpret_cast<const uint8_t *>(b.w.w + (int64_t)(b.first(piece) + v0) * b.w.ld + p0);
    const uint8_t *q = reinterpret_cast<const uint8_t *>(b.dz + (int64_t)q0 * b.ld + v0);
    // dz is zero behind the vocabulary's last
    t.start(lds, b.w.ld, b.w.hidden - p0, b.ld, Tile::kQ, max(0, have));
    t.run(n, p, kStepK * 2 * (uint32_t)b.w.ld, q, kStepK * 2, 0, [] {});
    float *to = b.sums + (int64_t)slab * count * b.w.hidden;
#pragma unroll
    for (int j = 0; j < Tile::NQ; ++j)
#pragma unroll
        for (int i = 0; i < Tile::NP; ++i) {
            const int q1 = q0 + t.q_of(j), p1 = p0 + t.p_of(i);
            if (q1 < count && p1 < b.w.hidden) {
                v4f *sum = reinterpret_cast<v4f *>(to + (int64_t)q1 * b.w.hidden + p1);
                *sum = piece > 0 ? *sum + t.acc[i][j] : t.acc[i][j];
            }
        }
}

// What the rounding of dz left at the targets, times x, into the sums of a tile of dw: the rows with
// their target in the tile are a product of their own, up to 64 of them a step, behind the tile's.
// Their x is fetched from where it lies; the other operand is zero but for one value a row (in bf16: off
// by 2^-9 of what is 2^-9 of dz), which is put into the LDS and taken out again.
//
// Most tiles have at most 32 such rows.  Those are fetched to a place of their own with the tile's
// own first steps (dw of 1024 rows under 16000 x 512 26.8 us, 30.8 with all of them fetched behind the
// tile's product, 24.5 without any), except where there is one step only and the workgroups share a CU.
// Many rows to an entry cost the most: dw of 8192 rows under 1000 x 4096 92 us, 76 without.
template <class Tile> struct Rests {
    using SideP = typename Tile::SideP;
    using SideQ = typename Tile::SideQ;
    static constexpr bool kEarly = Tile::kSlots > 1;
    static constexpr int kOther = Tile::kSlots * SideP::kBytes;  // the other operand's place
    struct Shared {
        uint8_t early[kEarly ? SideP::kBytes / 2 : 16];  // x of 32 rows
        int4 left[2][64];
    };
    const Backward &b;
    Shared &shared;
    int from, end;    // the tile's rows in the list, from the next step's
    int fetched = 0;  // early

    __device__ __forceinline__ Rests(const Backward &b_, Shared &shared_, int tile)
        : b(b_), shared(shared_), from(__builtin_amdgcn_readfirstlane(b.starts[tile])),
          end(__builtin_amdgcn_readfirstlane(b.starts[tile + 1]))
    {
    }
    // Fetches the next rows, up to `most`: COPIES copies of x a wave to `to`, its first one's place, and
    // what is left of them (all waves the same) to a slot; returns how many.
    template <int COPIES>
    __device__ __forceinline__ int fetch(const Tile &t, int most, int slot, uint32_t to, int p0)
    {
        const int all = min(end - from, most);
        if (all <= 0)
            return 0;
        const int row = b.by_target[from + min(t.lane, all - 1)];
        from += all;
        const uint8_t *zeros = reinterpret_cast<const uint8_t *>(kZeros);
        copy16(t.lane < all ? reinterpret_cast<const uint8_t *>(b.left + row) : zeros,
               __builtin_amdgcn_readfirstlane(lds_address(shared.left[slot])));
#pragma unroll
        for (int n = 0; n < COPIES; ++n) {
            const int cc = t.wave + n * Tile::kWaves;
            const int k = cc * (512 / Tile::kP) + t.lane / (Tile::kP / 8);
            const uint8_t *at = reinterpret_cast<const uint8_t *>(
                b.x.x + (int64_t)__shfl(row, k) * b.x.ld + p0);
            copy16(k < all ? at + SideP::offset(cc, t.lane, 0, b.x.ld - p0) : zeros,
                   to + n * (Tile::kWaves * 1024));
        }
        return all;
    }
    // while the tile's first steps are fetched; p0: its first hidden value
    __device__ __forceinline__ void early(const Tile &t, int p0)
    {
        if constexpr (kEarly)
            fetched = fetch<Tile::kPerP / 2>(
                t, 32, 0,
                __builtin_amdgcn_readfirstlane(lds_address(shared.early) + t.wave * 1024), p0);
    }
    // behind the tile's product; v0: its first entry of the vocabulary
    __device__ __forceinline__ void add(Tile &t, uint8_t *lds, int v0, int p0)
    {
        int now = kEarly ? fetched : fetch<Tile::kPerP>(t, 64, 0, t.at_p, p0);
        if (now <= 0)
            return;
        for (int i = threadIdx.x * 16; i < SideQ::kBytes; i += Tile::kThreads * 16)
            *reinterpret_cast<gv4u *>(lds + kOther + i) = (gv4u){0u, 0u, 0u, 0u};
        uint16_t *value = nullptr;
        int slot = 0;
        uint32_t at = kEarly ? lds_address(shared.early) : lds_address(lds);
        while (now > 0) {
            // the step's rows have landed, and everyone is done with those before
            Tile::template wait<0>();
            barrier_no_fence();
            const int4 left = shared.left[slot][t.lane];
            // (within the tile, whatever became of the targets in the meantime)
            const int column = t.lane < now && (unsigned)(left.x - v0) < (unsigned)Tile::kQ ? left.x - v0 : -1;
            if (t.wave == 0) {
                if (value)
                    *value = 0;
                value = column < 0 ? nullptr
                                   : reinterpret_cast<uint16_t *>(lds + kOther + SideQ::place(t.lane, column));
                if (value)
                    *value = __builtin_bit_cast(uint16_t, (__bf16)__int_as_float(left.y));
            }
            int then = 0;
            if (kEarly)
                then = fetch<Tile::kPerP>(t, 64, slot ^ 1, t.at_p + (slot ^ 1) * SideP::kBytes, p0);
            Tile::template wait<63>();
            barrier_no_fence();
            t.read_p.start(at, t.wp, t.lane);
            t.read_q.start(lds_address(lds) + kOther, t.wq, t.lane);
            uint64_t on[Tile::NQ];
#pragma unroll
            for (int j = 0; j < Tile::NQ; ++j)
                on[j] = __ballot(column >> 4 == t.wq + Tile::WQ * j);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if (now <= 32 * h)
                    break;
                v8bf x[Tile::NP];
#pragma unroll
                for (int i = 0; i < Tile::NP; ++i)
                    x[i] = t.read_p.read(i, h);
#pragma unroll
                for (int j = 0; j < Tile::NQ; ++j)
                    if ((uint32_t)(on[j] >> (32 * h))) {
                        const v8bf rests = t.read_q.read(j, h);
#pragma unroll
                        for (int i = 0; i < Tile::NP; ++i)
                            t.acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x[i], rests, t.acc[i][j], 0, 0, 0);
                    }
            }
            if constexpr (kEarly) {
                now = then;
                slot ^= 1;
                at = lds_address(lds) + slot * SideP::kBytes;
            } else {
                barrier_no_fence();
                now = fetch<Tile::kPerP>(t, 64, 0, t.at_p, p0);
            }
        }
        barrier_no_fence();
    }
};

// Tile `at` of dw = dz^T x of the piece's vocabulary.
template <class Tile>
__device__ __forceinline__ void dw_part(uint8_t *lds, const Backward &b, int piece, int at)
{
    const int np = (b.w.hidden + Tile::kP - 1) / Tile::kP;
    const int have = b.have(piece);
    const int nq = (have + Tile::kQ - 1) / Tile::kQ;
    if (at >= np * nq)
        return;
    int tp, tq;
    product_tile(at, np, nq, tp, tq);
    const int p0 = tp * Tile::kP, q0 = tq * Tile::kQ;
    __shared__ __align__(16) typename Rests<Tile>::Shared shared;
    const int v0 = b.first(piece) + q0;
    const int count = *b.x.count;
    Rests<Tile> rests(b, shared, v0 / Tile::kQ);  // on its way with the count
    Tile t;
    t.start(lds, b.x.ld, b.x.ld - p0, b.ld, b.width - q0, kStepK);
    const uint8_t *p = reinterpret_cast<const uint8_t *>(b.x.x + p0);
    const uint8_t *q = reinterpret_cast<const uint8_t *>(b.dz + q0);
    t.run((count + kStepK - 1) / kStepK, p, kStepK * 2 * b.x.ld, q, kStepK * 2 * b.ld, 0,
          [&] { rests.early(t, p0); });
    t.place();  // nothing more is kept over the product, whose tiles fill the registers
    rests.add(t, lds, v0, p0);
    t.place();
#pragma unroll
    for (int j = 0; j < Tile::NQ; ++j)
#pragma unroll
        for (int i = 0; i < Tile::NP; ++i) {
            const v4f v = t.acc[i][j];
            t.put(lds, i, j, (gv2u){pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])});
        }
    t.template flush<true>(lds, b.dw + (int64_t)(b.first(piece) + q0) * b.ld_dw + p0, b.ld_dw,
                           have - q0, b.w.hidden - p0);
}

template <class Tile>
__global__ __launch_bounds__(Tile::kThreads, 1) void k_ce_dlogits(Backward b, int piece)
{
    __shared__ __align__(16) uint8_t lds[Tile::kLds];
    dlogits<Tile>(lds, b, piece, blockIdx.x);
}
template <class Tile>
__global__ __launch_bounds__(Tile::kThreads, 1) void k_ce_dx(Backward b, int piece)
{
    __shared__ __align__(16) uint8_t lds[Tile::kLds];
    dx_part<Tile>(lds, b, piece, blockIdx.x);
}
template <class Tile>
__global__ __launch_bounds__(Tile::kThreads, Tile::kLds <= 32768 ? 4 : 1) void k_ce_dw(Backward b,
                                                                                     int piece)
{
    __shared__ __align__(16) uint8_t lds[Tile::kLds];
    dw_part<Tile>(lds, b, piece, blockIdx.x);
}

// dx from the slabs of sums, every row of it, 1024 columns at a time; p, q: the tile of the
// products for dx
__global__ __launch_bounds__(256) void k_ce_dx_rows(Backward b, int p, int q, bf16_t *dx, int64_t ld)
{
    const int hidden = b.w.hidden, wide = (hidden + 1023) / 1024;
    const int count = *b.x.count;
    const int slabs = slabs_of((hidden + p - 1) / p * ((count + q - 1) / q), b.fill, b.room);
    const int64_t slab = (int64_t)count * hidden;
    for (int64_t i = blockIdx.x; i < b.a.rows * wide; i += gridDim.x) {
        const int64_t r = i / wide;
        const int c = (int)(i % wide) * 1024 + threadIdx.x * 4;
        if (c >= hidden)
            continue;
        const int at = b.x.place[r], target = b.a.targets[r];
        v4f v = {0.f, 0.f, 0.f, 0.f};
        if (at >= 0) {
            const bool here = target < b.w.vocab;
            const gv2u raw = *(const MXQ_GLOBAL gv2u *)(b.w.w + (int64_t)(here ? target : 0) * b.w.ld + c);
            const float rest = here ? __int_as_float(b.left[at].y) : 0.0f;
            const float *from = b.sums + (int64_t)at * hidden + c;
#pragma unroll 8
            for (int s = 0; s < slabs; ++s)
                v += *reinterpret_cast<const v4f *>(from + s * slab);
            float w[4];
            unpack(raw, w, (bf16_t *)nullptr);
#pragma unroll
            for (int k = 0; k < 4; ++k)
                v[k] += rest_of(rest, w[k]);
        }
        const float f[4] = {v[0], v[1], v[2], v[3]};
        store_vec(dx + r * ld + c, f);
    }
}

// ---- the host's side -------------------------------------------------------------

// What is taken: offsets within a tile fit 32 bits, and launches their number of threads.
constexpr int64_t kMostRows = int64_t(1) << 22, kMostVocab = int64_t(1) << 24;
constexpr int64_t kMostHidden = int64_t(1) << 16, kMostLogits = int64_t(1) << 37;
constexpr int64_t kMostLd = int64_t(1) << 22;

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
    x.all = -1;
    x.count = c.take<int>(1);
    x.place = c.take<int>(rows);
    x.row = c.take<int>(rows);
    x.at_target = c.take<float>(rows);
    x.ld = (int)pitch(up(hidden, kStepK));
    x.x = c.take<u16>(up(rows, kStepK) * x.ld);
    return x;
}

int64_t tiles_of(int64_t n, int64_t tile) { return (n + tile - 1) / tile; }

template <class T> struct Tag {
    using Tile = T;
};
constexpr int kCus = 256;
// Logits of a piece of the vocabulary: 256 MiB of dz.  (8192 x 4096 x 128256 with 2^25 to 2^28
// of them 19.4, 18.8, 18.5 and 18.3 ms: fewer pieces add to the sums of dx less often.  Pieces
// whose weight stays in the last-level cache leave CUs idle with few rows: 100 x 4096 x 128256
// in pieces of 16384 1123 us, in one 737.)
// (The tests have a build whose pieces are a tile wide.)
#ifndef MXQ_PIECE_LOGITS
#define MXQ_PIECE_LOGITS (1 << 27)
#endif
constexpr int64_t kPieceLogits = MXQ_PIECE_LOGITS;

// f(Tag<Tile>) for the logits of a stretch of the vocabulary.  ONCE: its weight is read by
// nobody else soon; where all rows are one tile, it then leaves the caches to what is (24 x
// 4096 x 128256 in the forward pass 205 us without the hint, 182 with it).
template <bool ONCE, bool CUT, class F> void with_logits_of(int64_t rows, int64_t vocab, F f)
{
    // Forward passes, with weights that no cache holds yet: 4 rows under 8000 x 4096 (125 tiles) Slim
    // 21 us, Few 34; 16 under 32003 x 4096 (501) 56 and 50.  100 rows under 8000 x 4096 (250) Small
    // 36 us, Deep 42; under 16000 (500) 64 and 49.  200 under 8000 x 4096 (500) Small 58, Half 68;
    // 300 (625) 77 and 64.  100 under 32000 x 4096 (250) Deep 64 us, Twin 78; under 128256 222 and 203.
    // 200 under 32000 x 4096 (125) Half 79 us, Many 126; 400 (250) 153 and 135.
    // Deep and Twin above 128 rows: 200 under 8000 x 4096 54 and 70 (Small 57), under 16000 x 4096 62
    // and 76 (Half 71), under 32000 x 4096 114 and 114, under 32000 x 1024 38 and 36 (Half 30); 400
    // under 8000 x 1024 24 and 29 (Half 27), under 16000 x 4096 115 and 115 (Half 76), under 32000 x
    // 1024 68 and 63 (Many 43).  Deep's few better sizes, by 13% at most, lie on both sides of these rules.
    const int64_t small = tiles_of(vocab, 64) * tiles_of(rows, 64);
    if (rows <= 32 && small <= kCus)
        f(Tag<Slim<true, true, CUT, ONCE>>{});
    else if (rows <= 32)
        f(Tag<Few<true, true, CUT, ONCE>>{});
    else if (small <= (rows <= 128 ? kCus : 2 * kCus))
        f(Tag<Small<true, true, CUT, ONCE>>{});
    else if (rows <= 128 && tiles_of(vocab, 128) <= kCus)
        f(Tag<Deep<true, true, CUT, ONCE>>{});
    else if (rows <= 128)
        f(Tag<Twin<true, true, CUT, ONCE>>{});
    else if (tiles_of(vocab, 256) * tiles_of(rows, 256) <= kCus / 2)
        f(Tag<Half<true, true, CUT>>{});
    else
        f(Tag<Many<true, true, CUT>>{});
}
template <bool ONCE, class F>
void with_logits(int64_t rows, int64_t hidden, int64_t vocab, F f)
{
    // looking for a last step that is not whole, along k, costs 2 to 4%
    if (hidden % kStepK)
        with_logits_of<ONCE, true>(rows, vocab, f);
    else
        with_logits_of<ONCE, false>(rows, vocab, f);
}
// for dx, whose tiles are made enough by stretches of the vocabulary, where it is long enough
constexpr int kStretch = 512;
int64_t most_stretches(int64_t width) { return width / kStretch > 0 ? width / kStretch : 1; }
template <bool CUT, class F> void with_dx_of(int64_t rows, int64_t hidden, int64_t width, F f)
{
    // backward passes of 200 rows under 1000 x 4096 (16 tiles of all stretches) Deep 70 us, Many 80;
    // 1024 under 16000 x 512 (248) 88 and 95; 200 under 16000 x 4096 (496) 174 and 172; 800 under
    // 16000 x 4096 (1984) 376 and 337
    if (rows <= 32)
        f(Tag<Few<false, true, CUT>>{});
    else if (rows <= 128)
        f(Tag<Twin<false, true, CUT>>{});
    else if (tiles_of(hidden, 256) * tiles_of(rows, 256) * most_stretches(width) <= kCus)
        f(Tag<Deep<false, true, CUT>>{});
    else
        f(Tag<Many<false, true, CUT>>{});
}
template <class F> void with_dx(int64_t rows, int64_t hidden, int64_t width, int64_t vocab, F f)
{
    if (vocab % kStepK)
        with_dx_of<true>(rows, hidden, width, f);
    else
        with_dx_of<false>(rows, hidden, width, f);
}
// for dw
template <class F> void with_dw(int64_t rows, int64_t hidden, int64_t vocab, F f)
{
    // 1024 rows under 8000 x 512 (64 tiles) forward and backward Deep 70 us, Many 83.  Passes for dw
    // alone, Deep, Twin and Many: 1024 under 1000 x 4096 (64 tiles) 47, 52 and 61 us, under 4000 x
    // 4096 (256) 110, 104 and 97; 512 under 8000 x 1024 (128) 44, 41 and 44; 200 under 16000 x 512
    // (126) 33, 30 and 33, under 32000 x 4096 235, 191 and 180; 100 under 8000 x 4096 67, 57 and 57,
    // under 32000 x 4096 164, 135 and 131, under 128256 x 4096 652, 563 and 521: up to 128 rows Twin
    // and Many are even, but under the largest vocabularies.
    if (rows <= kStepK)
        f(Tag<Outer>{});
    else if (tiles_of(vocab, 256) * tiles_of(hidden, 256) <= kCus / 2)
        f(Tag<Deep<false, false, false>>{});
    else if (rows <= 2 * kStepK)
        f(Tag<Twin<false, false, false>>{});
    else
        f(Tag<Many<false, false, false>>{});
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
    with_logits<true>(rows, hidden, vocab, [&](auto t) {
        f.tiles = tiles_of(vocab, decltype(t)::Tile::kP);
    });
    f.stride = up(rows, 16);
    f.part = c.take<float2>(f.tiles * f.stride);
    f.bytes = c.used;
    return f;
}

struct BackwardPlan {
    Backward b;  // without the caller's pointers
    int64_t pieces;
    int64_t dx_groups, dx_p, dx_q;  // workgroups of the products for dx, and their tile
    int dw_q;                       // entries of the vocabulary of a tile of dw
    size_t bytes;
};
// a piece's width is a multiple of it, and so is how many rows dz has: of every tile's
constexpr int kWidthStep = 256, kRowStep = 256;
BackwardPlan backward_plan(int64_t rows, int64_t hidden, int64_t vocab, void *ws,
                           int64_t piece_logits = kPieceLogits)
{
    BackwardPlan f;
    Carve c = {static_cast<uint8_t *>(ws)};
    Backward &b = f.b;
    b.x = take_packed(c, rows, hidden);
    const int64_t padded = up(rows > 0 ? rows : 1, kRowStep);
    const int64_t most = up(vocab, kWidthStep);
    int64_t width = piece_logits / padded / kWidthStep * kWidthStep;
    width = width < kWidthStep ? kWidthStep : width < most ? width : most;
    width = up(tiles_of(vocab, tiles_of(vocab, width)), kWidthStep);
    f.pieces = tiles_of(vocab, width);
    b.width = (int)width;
    b.ld = (int)pitch(width);
    b.dz = c.take<u16>(padded * b.ld);
    with_dw(rows, hidden, width, [&](auto t) { f.dw_q = decltype(t)::Tile::kQ; });
    b.by_target = c.take<int>(rows);
    b.starts = c.take<int>(tiles_of(vocab, f.dw_q) + 1);
    b.left = c.take<int4>(rows);
    with_dx(rows, hidden, width, vocab, [&](auto t) {
        using Tile = typename decltype(t)::Tile;
        const int64_t np = tiles_of(hidden, Tile::kP), tiles = np * tiles_of(rows, Tile::kQ);
        b.fill = kCus * (Tile::kLds <= 65536 ? 2 : 1) * (rows <= 32 ? 2 : 1);
        b.room = (int)most_stretches(width);
        // slabs x tiles are at most `fill` where there is more than one slab
        const int64_t slab_rows = Tile::kQ * (b.fill / np);
        const int64_t all = slab_rows < b.room * rows ? slab_rows : b.room * rows;
        b.sums = c.take<float>((rows > all ? rows : all) * hidden);
        f.dx_groups = tiles > b.fill ? tiles : b.fill;
        f.dx_p = Tile::kP;
        f.dx_q = Tile::kQ;
    });
    f.bytes = c.used;
    return f;
}

bool sizes_ok(int64_t rows, int64_t hidden, int64_t vocab)
{
    return rows >= 0 && rows <= kMostRows && vocab >= 1 && vocab <= kMostVocab &&
           rows * vocab <= kMostLogits && hidden >= 32 && hidden % 32 == 0 && hidden <= kMostHidden;
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
                 bool zeros, const CeTargets &lists, hipStream_t s)
{
    // about 1024 workgroups: more would read the rows in front of their own more often
    const int64_t per = a.rows > 1024 ? tiles_of(a.rows, 1024) : 1;
    const int groups = (int)(a.rows > 0 ? tiles_of(a.rows, per) : 1);
    hipLaunchKernelGGL(k_ce_pack, dim3((unsigned)(groups + (zeros ? kStepK - 1 + lists.tiles : 0))),
                       dim3(kPackThreads), 0, s, a, per, groups, static_cast<const bf16_t *>(x), ld,
                       (int)hidden, to, lists);
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
    ForwardPlan f = forward_plan(rows, hidden, vocab, workspace);
    if (!workspace || ws_bytes < f.bytes)
        return MXQ_ERR_WORKSPACE;
    hipStream_t s = static_cast<hipStream_t>(stream);
    const CeRows a = {targets, weight, rows};
    const CeWeight cw = {static_cast<const u16 *>(w), ld_w, (int)vocab, (int)hidden};
    const Heat heat = heat_of(temperature);
    with_logits<true>(rows, hidden, vocab, [&](auto t) {
        using Tile = typename decltype(t)::Tile;
        const int64_t groups = f.tiles * tiles_of(rows, Tile::kQ);
        // Few rows are read where they are, if they can be: the ones that do not count cost little
        // there, and packing a launch (one row under 32000 x 1024 19 us with it, 15 without).
        if (rows <= 128 && reinterpret_cast<uintptr_t>(x) % 16 == 0 &&
            ld_x % 8 == 0 && hidden % kStepK == 0 && ld_x <= kMostLd) {
            f.x.all = (int)rows;
            f.x.x = const_cast<u16 *>(static_cast<const u16 *>(x));
            f.x.ld = (int)ld_x;
        } else {
            launch_pack(a, x, ld_x, hidden, f.x, false, {}, s);
        }
        hipLaunchKernelGGL(k_ce_stats<Tile>, dim3((unsigned)groups), dim3(Tile::kThreads), 0, s, cw,
                           a, f.x, heat, f.part, f.stride);
        // 16 rows a workgroup read whole lines; few rows would leave the chip empty
        const auto loss_of = [&](auto per) {
            constexpr int ROWS = decltype(per)::value;
            hipLaunchKernelGGL(k_ce_loss<ROWS>, dim3((unsigned)tiles_of(rows, ROWS)), dim3(256), 0,
                               s, a, f.x, (int)vocab, (int)f.tiles, f.part, f.stride, heat, loss,
                               reinterpret_cast<float2 *>(stats));
        };
        if (rows <= 512)
            loss_of(std::integral_constant<int, 1>{});
        else
            loss_of(std::integral_constant<int, 16>{});
    });
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
    const BackwardPlan f = backward_plan(rows, hidden, vocab, workspace);
    if (!workspace || ws_bytes < f.bytes)
        return MXQ_ERR_WORKSPACE;
    Backward b = f.b;
    hipStream_t s = static_cast<hipStream_t>(stream);
    b.w = {static_cast<const u16 *>(w), ld_w, (int)vocab, (int)hidden};
    b.a = {targets, weight, rows};
    b.heat = heat_of(temperature);
    b.stats = reinterpret_cast<const float2 *>(stats);
    b.dw = static_cast<u16 *>(dw);
    b.ld_dw = ld_dw;
    const CeTargets lists = {dw ? (int)tiles_of(vocab, f.dw_q) : 0, __builtin_ctz(f.dw_q), (int)vocab, b.stats,
                             b.by_target, b.starts};
    launch_pack(b.a, x, ld_x, hidden, b.x, true, lists, s);
    const auto have = [&](int64_t piece) {
        return vocab - piece * b.width < b.width ? vocab - piece * b.width : (int64_t)b.width;
    };
    const int n_dx = dx && rows > 0 ? (int)f.dx_groups : 0;
    with_logits<false>(rows, hidden, b.width, [&](auto tz) {
        with_dx(rows, hidden, b.width, vocab, [&](auto tx) {
            with_dw(rows, hidden, b.width, [&](auto tw) {
                using Logit = typename decltype(tz)::Tile;
                using Dx = typename decltype(tx)::Tile;
                using Dw = typename decltype(tw)::Tile;
                const auto n_z = [&](int64_t piece) {
                    return tiles_of(have(piece), Logit::kP) * tiles_of(rows, Logit::kQ);
                };
                const auto n_dw = [&](int64_t piece) {
                    return dw ? tiles_of(hidden, Dw::kP) * tiles_of(have(piece), Dw::kQ) : 0;
                };
                const auto launch = [&](auto kernel, int threads, int64_t groups, auto... args) {
                    if (groups > 0)
                        hipLaunchKernelGGL(kernel, dim3((unsigned)groups), dim3(threads), 0, s, b,
                                           args...);
                };
                for (int i = 0; i < (int)f.pieces; ++i) {
                    launch(k_ce_dlogits<Logit>, Logit::kThreads, n_z(i), i);
                    launch(k_ce_dx<Dx>, Dx::kThreads, n_dx, i);
                    launch(k_ce_dw<Dw>, Dw::kThreads, n_dw(i), i);
                }
            });
        });
    });
    if (n_dx > 0)
        hipLaunchKernelGGL(k_ce_dx_rows, dim3(row_grid(rows * tiles_of(hidden, 1024))), dim3(256),
                           0, s, b, (int)f.dx_p, (int)f.dx_q, static_cast<bf16_t *>(dx), ld_dx);
    return launched();
}

#ifdef MXQ_TESTS
// For the tests, in their build of the library alone: the kernels that calls of these sizes take, with
// pieces of up to piece_logits logits.  tiles: [forward logits, backward logits, dx, dw][their p, q, steps
// in LDS, whether a last step may be cut]; plan: pieces, their width, most slabs of dx.
extern "C" void mxq_linear_ce_kernels(int64_t rows, int64_t hidden, int64_t vocab,
                                      int64_t piece_logits, int32_t *tiles, int32_t *plan)
{
    const BackwardPlan f = backward_plan(rows, hidden, vocab, nullptr, piece_logits);
    const auto put = [&](int i) {
        return [&tiles, i](auto t) {
            using Tile = typename decltype(t)::Tile;
            const int32_t v[4] = {Tile::kP, Tile::kQ, Tile::kSlots, Tile::kCut};
            for (int k = 0; k < 4; ++k)
                tiles[4 * i + k] = v[k];
        };
    };
    with_logits<true>(rows, hidden, vocab, put(0));
    with_logits<false>(rows, hidden, f.b.width, put(1));
    with_dx(rows, hidden, f.b.width, vocab, put(2));
    with_dw(rows, hidden, f.b.width, put(3));
    const int64_t of_dx = tiles_of(hidden, f.dx_p) * tiles_of(rows, f.dx_q);
    plan[0] = (int32_t)f.pieces;
    plan[1] = f.b.width;
    plan[2] = slabs_of((int)of_dx, f.b.fill, f.b.room);
}
#endif
