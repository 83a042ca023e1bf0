// A tile of a bf16 matrix product on the matrix cores, for the operators that put
// their own arithmetic behind it.
//
//   out[q][p] = sum over k of P[p][k] Q[q][k], fp32, p the contiguous side of out
//
// v_mfma_f32_16x16x32_bf16: lane (g, li) = (lane / 16, lane % 16) supplies row li of
// each operand and its values k = 8 g .. 8 g + 7; it holds rows 4 g .. 4 g + 3 of column
// li of the product, that is four neighbours of out's contiguous side.
//
// An operand lies in memory in one of two ways:
//   along k (ALONG):   a row of the operand is contiguous in k.  A step's tile is
//                      [rows][64 k], 128 bytes a row; a fragment is one 16-byte read.
//   across k (!ALONG): a value of k is a contiguous run over the operand's rows.  A
//                      step's tile is [64 k][rows]; the LDS turns it while it is read
//                      (ds_read_b64_tr_b16: the 16 lanes of a group read four k of 16
//                      rows, and lane li gets the four k of row li), two reads a
//                      fragment.
// Both are copied as they lie, 16 bytes a lane, into LDS.  A lane's place in LDS is
// fixed (16 bytes times its number), so the order within a tile is made by what each
// lane fetches: 16-byte chunks are exchanged within a row (chunk c of row r lies at
// c ^ x(r)) so that the 16 lanes that read at a time touch every bank once.  (The 32 lanes
// of two groups that read across k meet in half of the banks, and half of those reads' LDS
// cycles wait.  An exchange that takes the group's bit too leaves none of them, and the
// backward pass below takes 17.72 ms with it, 17.67 without.)
//
// What bounds it: the matrix cores, and the power that they take.  256 x 256 tiles take
// 1.4 us a step of 64 k and 7.5 us a tile besides (its start, its epilogue): 1.38 to
// 1.43 PF over 4096 k, 1.65 and more when the operands are zeros.  In 8192 x 4096 x 16384
// the matrix cores are busy for 72 to 76% of the cycles, at 2.0 GHz of 2.4.  A read or a
// copy between every few products takes their waits out: all copies first are 2% slower, all
// last 5%.
#pragma once

#include <type_traits>

#include "lds_copy.hpp"
#include "mxq_device.hpp"

namespace mxq {

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef short v4s __attribute__((ext_vector_type(4)));
typedef float v4f __attribute__((ext_vector_type(4)));

__device__ const __attribute__((aligned(16))) uint32_t kZeros[4] = {0u, 0u, 0u, 0u};

constexpr int kStepK = 64;  // k of a step: two halves of one fragment's 32 each

// One operand's tile of ROWS rows.
template <int ROWS, bool ALONG> struct Side {
    static constexpr int kBytes = ROWS * kStepK * 2;
    static constexpr int kChunks = kBytes / 1024;  // 1 KiB copies of a wave
    static_assert(ALONG || ROWS >= 128, "fragments across k are read from 256 bytes and more");

    // What lane `lane` fetches for copy cc of a step, in bytes from the tile's first
    // element; ld in elements; rows past the last of `have` >= 1 fetch it again (their
    // products are not used).  kNone: k past the last of `have_k`.
    static constexpr uint32_t kNone = ~0u;
    static __device__ __forceinline__ uint32_t offset(int cc, int lane, int64_t ld, int have,
                                                      int have_k = kStepK)
    {
        if constexpr (ALONG) {
            const int row = 8 * cc + (lane >> 3);
            const int chunk = (lane & 7) ^ ((row >> 1) & 7);
            if (chunk * 8 >= have_k)
                return kNone;
            return (uint32_t)(min(row, have - 1) * ld * 2 + chunk * 16);
        } else {
            constexpr int PER = ROWS / 8;  // chunks of one k
            const int k = cc * (64 / PER) + lane / PER;
            const int chunk = (lane % PER) ^ (2 * (k & 7));
            if (k >= have_k)
                return kNone;
            return (uint32_t)(k * ld * 2 + min(chunk * 8, have - 8) * 2);
        }
    }

    // where value k of row `row` of an operand across k lies in a step's tile, in bytes
    static __device__ __forceinline__ int place(int k, int row)
    {
        static_assert(!ALONG, "across k");
        return k * (ROWS * 2) + ((row >> 3) ^ (2 * (k & 7))) * 16 + (row & 7) * 2;
    }

    // Where a wave's fragments lie: wave w of W takes fragments (of 16 rows) w, w + W, ...
    // A lane keeps kBases addresses; fragment i and the half are constants from there.
    template <int W> struct Reader {
        static constexpr int kBases = ALONG ? 2 : W >= 4 ? 1 : 4 / W;
        static_assert(ALONG || W <= 4, "the third bit of a fragment's number is a constant's");
        uint32_t base[kBases];

        __device__ __forceinline__ void start(uint32_t l, int w, int lane)
        {
            const int g = lane >> 4, li = lane & 15;
            if constexpr (ALONG) {
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    base[h] = l + w * 2048 + li * 128 + (((4 * h + g) ^ (li >> 1)) * 16);
            } else {
                // fragment t = w + W i lies at pair t ^ (k & 7) of its k, k & 7 = 4 u + li / 4
                // for the read u of the two: the pair's two low bits are the lane's and the
                // base's, the third is a constant's
                const int k = 8 * g + (li >> 2);
#pragma unroll
                for (int b = 0; b < kBases; ++b)
                    base[b] = l + k * (ROWS * 2) + (((w + W * b) & 3) ^ (li >> 2)) * 32 +
                              ((li >> 1) & 1) * 16 + (li & 1) * 8;
            }
        }
        __device__ __forceinline__ void move(int by)
        {
#pragma unroll
            for (int b = 0; b < kBases; ++b)
                base[b] += by;
        }
        // fragment i of half h
        __device__ __forceinline__ v8bf read(int i, int h) const
        {
            if constexpr (ALONG) {
                typedef __attribute__((address_space(3))) const v8bf lds_v8bf;
                return *(lds_v8bf *)(uintptr_t)(base[h] + i * (W * 2048));
            } else {
                typedef __attribute__((address_space(3))) v4s lds_v4s;
                const int t = W * i;  // and w, whose two low bits are in the base
                v4s r[2];
#pragma unroll
                for (int u = 0; u < 2; ++u)
                    r[u] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                        (lds_v4s *)(uintptr_t)(base[i % kBases] + h * (32 * ROWS * 2) +
                                               u * (4 * ROWS * 2) + (t >> 3) * 256 +
                                               (((t >> 2) & 1) ^ u) * 128));
                typedef short v8s __attribute__((ext_vector_type(8)));
                return __builtin_bit_cast(
                    v8bf, (v8s)__builtin_shufflevector(r[0], r[1], 0, 1, 2, 3, 4, 5, 6, 7));
            }
        }
    };
};

// the pointer in scalar registers
__device__ __forceinline__ const uint8_t *uniform(const uint8_t *p)
{
    const uint64_t a = reinterpret_cast<uint64_t>(p);
    const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)a);
    const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)(a >> 32));
    return reinterpret_cast<const uint8_t *>((uint64_t)hi << 32 | lo);
}

// A workgroup of WP x WQ waves, each with NP x NQ tiles of 16 x 16, and SLOTS steps in LDS
// (1: there is one step only).  P_CUT: the last step of P may have fewer k, where Q is zero.
// P_ONCE: P is not read again.
template <int WP_, int WQ_, int NP_, int NQ_, int SLOTS, bool P_ALONG, bool Q_ALONG, bool P_CUT,
          bool P_ONCE = false>
struct Product {
    static constexpr int WP = WP_, WQ = WQ_, NP = NP_, NQ = NQ_;
    static constexpr int kP = 16 * WP * NP, kQ = 16 * WQ * NQ, kWaves = WP * WQ;
    static constexpr int kThreads = 64 * kWaves, kSlots = SLOTS;
    static constexpr bool kCut = P_CUT;
    using SideP = Side<kP, P_ALONG>;
    using SideQ = Side<kQ, Q_ALONG>;
    static constexpr int kLds = SLOTS * (SideP::kBytes + SideQ::kBytes);
    static constexpr int kPerP = SideP::kChunks / kWaves, kPerQ = SideQ::kChunks / kWaves;
    static constexpr int kPer = kPerP + kPerQ;
    static_assert(kPerP * kWaves == SideP::kChunks && kPerQ * kWaves == SideQ::kChunks,
                  "copies split evenly");
    static_assert((SLOTS - 1) * kPer < 64, "a wait counts up to 63 copies");
    // waits for the wave's LDS reads, and until at most N of its copies are still in flight
    template <int N> static __device__ __forceinline__ void wait()
    {
        __builtin_amdgcn_s_waitcnt(0x0070 | (N & 15) | (N >> 4) << 14);
    }

    // the first of `left` <= N steps that are fetched has landed
    template <int N> static __device__ __forceinline__ void wait_behind(int left)
    {
        if constexpr (N <= 1)
            wait<0>();
        else if (left >= N)
            wait<(N - 1) * kPer>();
        else
            wait_behind<N - 1>(left);
    }

    v4f acc[NP][NQ];
    // Where registers allow, the halves of two steps are summed apart and joined at the end: a
    // sum's rounding is relative to what it holds.  (Maxima near 10.7 of rows under 32000 x 4096 are
    // off by 3.9e-6 in the root mean square with one sum, by 1.05e-6 with four, under 32000 x 1024 by
    // 1.9 and 0.7; the calls take 1 to 3% longer.)
    static constexpr int kSets = NP * NQ <= 4 && SLOTS > 1 ? 4 : 1;
    v4f more[kSets][NP][NQ];  // without the first, which is acc
    int lane, wave, wp, wq;
    typename SideP::template Reader<WP> read_p;
    typename SideQ::template Reader<WQ> read_q;
    uint32_t off_p[kPerP], off_q[kPerQ];
    uint32_t at_p, at_q;  // the wave's first copies in LDS
    // P_CUT: a last step with fewer k, and what is fetched of P there (Q is zero behind it)
    int cut_step;
    uint32_t cut_p[kPerP];

    __device__ __forceinline__ void place()
    {
        int thread = threadIdx.x;
        asm volatile("" : "+v"(thread));
        lane = thread & 63;
        wave = __builtin_amdgcn_readfirstlane(thread >> 6);
        wp = wave % WP;
        wq = wave / WP;
    }
    // lds: the workgroup's; p, q: leading dimensions and how many rows there are from the
    // tile's first; k: how many there are of it
    __device__ __forceinline__ void start(uint8_t *lds, int64_t ldp, int have_p, int64_t ldq,
                                          int have_q, int k)
    {
        place();
        const uint32_t l = (uint32_t)(uintptr_t)((__attribute__((address_space(3))) uint8_t *)lds);
        read_p.start(l, wp, lane);
        read_q.start(l + SLOTS * SideP::kBytes, wq, lane);
        at_p = __builtin_amdgcn_readfirstlane(l + wave * 1024);
        at_q = __builtin_amdgcn_readfirstlane(l + SLOTS * SideP::kBytes + wave * 1024);
        cut_step = k % kStepK ? k / kStepK : -1;
        const int left = k % kStepK ? k % kStepK : kStepK;
#pragma unroll
        for (int i = 0; i < kPerP; ++i) {
            off_p[i] = SideP::offset(wave + i * kWaves, lane, ldp, have_p);
            if constexpr (P_CUT)
                cut_p[i] = SideP::offset(wave + i * kWaves, lane, ldp, have_p, left);
        }
#pragma unroll
        for (int i = 0; i < kPerQ; ++i)
            off_q[i] = SideQ::offset(wave + i * kWaves, lane, ldq, have_q);
#pragma unroll
        for (int i = 0; i < NP; ++i)
#pragma unroll
            for (int j = 0; j < NQ; ++j)
                for (int set = 0; set < kSets; ++set)
                    (set ? more[set][i][j] : acc[i][j]) = (v4f){0.f, 0.f, 0.f, 0.f};
    }
    // copy n of step s, to the slot `slot`
    __device__ __forceinline__ void copy(int n, int s, int slot, const uint8_t *p, const uint8_t *q)
    {
        const uint32_t to = at_p + slot * SideP::kBytes + n * (kWaves * 1024);
        if (n < kPerP && P_CUT && s == cut_step)
            // zeros behind the last k: Q's zeros times an infinity would be no zeros
            copy16(cut_p[n] == SideP::kNone ? reinterpret_cast<const uint8_t *>(kZeros)
                                            : p + cut_p[n],
                   to);
        else if (n < kPerP)
            copy16<P_ONCE>(p, off_p[n], to);
        else
            copy16<false>(q, off_q[n - kPerP],
                          at_q + slot * SideQ::kBytes + (n - kPerP) * (kWaves * 1024));
    }
    // fragment n of a half: P's first, all of Q's, the rest of P's
    __device__ __forceinline__ void fragment(int n, int h, v8bf (&fp)[NP], v8bf (&fq)[NQ]) const
    {
        if (n == 0 || n > NQ)
            fp[n ? n - NQ : 0] = read_p.read(n ? n - NQ : 0, h);
        else
            fq[n - 1] = read_q.read(n - 1, h);
    }
    // The products of a half's fragments, and between them what item(n) issues for n of
    // 0 .. ITEMS - 1: reads and copies in front of the products would hold the wave until
    // the LDS and the address unit have taken them.
    template <int ITEMS, int SET, class Item>
    __device__ __forceinline__ void products(const v8bf (&fp)[NP], const v8bf (&fq)[NQ], Item item)
    {
        constexpr int ALL = NP * NQ;
#pragma unroll
        for (int n = 0; n < (ITEMS ? ITEMS : 1); ++n) {
            if (ITEMS) {
                item(n);
                __builtin_amdgcn_sched_barrier(0);
            }
#pragma unroll
            for (int m = n * ALL / (ITEMS ? ITEMS : 1); m < (n + 1) * ALL / (ITEMS ? ITEMS : 1); ++m)
            {
                v4f &sum = SET ? more[SET][m / NQ][m % NQ] : acc[m / NQ][m % NQ];
                sum = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fp[m / NQ], fq[m % NQ], sum, 0, 0, 0);
            }
            if (ITEMS)
                __builtin_amdgcn_sched_barrier(0);
        }
    }
    // `steps` steps from the (uniform) addresses p and q of the first one's tiles, each
    // dp and dq bytes further.  All of the LDS is free again when it returns.
    //
    // Each half's fragments are read during the half before it, so a step's slot has been
    // read when its first half is done: there, once a step, is the barrier, and the step
    // SLOTS further is fetched behind it into the same slot.  With two slots it lands during
    // the second half and the next step's first one.
    // The steps are taken in a circle from step `first`.  meanwhile() runs while the first
    // steps are fetched; the workgroup meets a barrier behind it.
    template <class F>
    __device__ __forceinline__ void run(int steps, const uint8_t *p, uint32_t dp, const uint8_t *q,
                                        uint32_t dq, int first, F meanwhile)
    {
        if (steps <= 0)
            return;
        steps = SLOTS == 1 ? 1 : __builtin_amdgcn_readfirstlane(steps);
        p = uniform(p);
        q = uniform(q);
        int at = __builtin_amdgcn_readfirstlane(first);  // the step that is fetched next
        const auto next = [&] { at = at + 1 < steps ? at + 1 : 0; };
#pragma unroll
        for (int i = 0; i < SLOTS; ++i)
            if (i < steps) {
#pragma unroll
                for (int n = 0; n < kPer; ++n)
                    copy(n, at, i, p + (uint64_t)(uint32_t)at * dp, q + (uint64_t)(uint32_t)at * dq);
                next();
            }
        // of `left` steps that are fetched, the first has landed
        const auto landed = [&](int left) { wait_behind<SLOTS>(left); };
        meanwhile();
        landed(min(steps, SLOTS));
        barrier_no_fence();
        v8bf fp[2][NP], fq[2][NQ];
        constexpr int FRAGMENTS = NP + NQ;
#pragma unroll
        for (int n = 0; n < FRAGMENTS; ++n)
            fragment(n, 0, fp[0], fq[0]);
        int slot = 0;
        // left: steps from this one on; set: of sums, for its first half
        const auto step = [&](int left, auto copies, auto last, auto set) {
            constexpr bool COPY = decltype(copies)::value, LAST = decltype(last)::value;
            constexpr int SET = decltype(set)::value % kSets, THEN = (SET + 1) % kSets;
            __builtin_amdgcn_sched_barrier(0);
            products<FRAGMENTS, SET>(fp[0], fq[0], [&](int n) { fragment(n, 1, fp[1], fq[1]); });
            if constexpr (LAST) {
                products<0, THEN>(fp[1], fq[1], [](int) {});
            } else {
                // this wave's copies of the next step have landed, its reads of this one are
                // done ...
                if constexpr (COPY)
                    wait<(SLOTS > 2 ? SLOTS - 2 : 0) * kPer>();
                else
                    landed(left - 1);
                // ... and everyone's
                barrier_no_fence();
                __builtin_amdgcn_sched_barrier(0);
                const int behind = slot + 1 < SLOTS ? 1 : 1 - SLOTS;
                read_p.move(behind * SideP::kBytes);
                read_q.move(behind * SideQ::kBytes);
                const uint8_t *ps = p + (uint64_t)(uint32_t)at * dp;
                const uint8_t *qs = q + (uint64_t)(uint32_t)at * dq;
                constexpr int COPIES = COPY ? kPer : 0;
                products<FRAGMENTS + COPIES, THEN>(fp[1], fq[1], [&](int n) {
                    // a copy and a fragment in turn, copies first: they take longest
                    constexpr int TURNS = COPIES < FRAGMENTS ? COPIES : FRAGMENTS;
                    if (n < 2 * TURNS ? n % 2 == 0 : COPIES > FRAGMENTS)
                        copy(n < 2 * TURNS ? n / 2 : n - TURNS, at, slot, ps, qs);
                    else
                        fragment(n < 2 * TURNS ? n / 2 : n - TURNS, 0, fp[0], fq[0]);
                });
                slot += behind;
                if constexpr (COPY)
                    next();
            }
        };
        constexpr std::true_type yes{};
        constexpr std::false_type no{};
        constexpr std::integral_constant<int, 0> even{};
        constexpr std::integral_constant<int, 2> odd{};
        int s = 0;
        if constexpr (SLOTS > 1) {
            if constexpr (kSets > 1)
                for (; s + SLOTS + 1 < steps; s += 2) {
                    step(0, yes, no, even);
                    step(0, yes, no, odd);
                }
            for (; s + SLOTS < steps; ++s)
                step(0, yes, no, even);
            if constexpr (kSets > 1)
                for (; s + 2 < steps; s += 2) {
                    step(steps - s, no, no, odd);
                    step(steps - s - 1, no, no, even);
                }
            for (; s + 1 < steps; ++s)
                step(steps - s, no, no, odd);
        }
        step(1, no, yes, even);
#pragma unroll
        for (int set = 1; set < kSets; ++set)
#pragma unroll
            for (int i = 0; i < NP; ++i)
#pragma unroll
                for (int j = 0; j < NQ; ++j)
                    acc[i][j] += more[set][i][j];
        __builtin_amdgcn_sched_barrier(0);
        wait<0>();
        barrier_no_fence();
    }
    // The tile in bf16 through the LDS, so that it leaves as whole lines: put() every
    // acc[i][j], packed, then flush().  16-byte chunk c of row q lies at c ^ q, of up to 16 chunks.
    static_assert(kP * kQ * 2 <= kLds, "the tile in bf16 fits where its operands were");
    static constexpr int kSwap = (kP < 128 ? kP / 8 : 16) - 1;
    __device__ __forceinline__ void put(uint8_t *lds, int i, int j, gv2u packed) const
    {
        const int p = p_of(i), q = q_of(j);
        typedef __attribute__((address_space(3))) gv2u lds_gv2u;
        *(lds_gv2u *)(__attribute__((address_space(3))) uint8_t *)(
            lds + q * (kP * 2) + ((p >> 3) ^ (q & kSwap)) * 16 + (p & 4) * 2) = packed;
    }
    // its first `rows` rows of q and `cols` (a multiple of 8) of p; ONCE: not read again
    template <bool ONCE>
    __device__ __forceinline__ void flush(const uint8_t *lds, uint16_t *to, int64_t ld, int rows,
                                          int cols) const
    {
        __syncthreads();
        constexpr int WIDE = kP / 8;  // chunks of a row
        const int c = threadIdx.x % WIDE;
        if (c * 8 >= cols)
            return;
#pragma unroll 4
        for (int q = threadIdx.x / WIDE; q < kQ; q += kThreads / WIDE) {
            typedef __attribute__((address_space(3))) const gv4u lds_gv4u;
            const gv4u v = *(lds_gv4u *)(__attribute__((address_space(3))) const uint8_t *)(
                lds + q * (kP * 2) + (c ^ (q & kSwap)) * 16);
            if (q < rows) {
                MXQ_GLOBAL gv4u *at = (MXQ_GLOBAL gv4u *)(to + (int64_t)q * ld + c * 8);
                if constexpr (ONCE)
                    __builtin_nontemporal_store(v, at);
                else
                    *at = v;
            }
        }
    }
    // p of acc[i][.][0] and q of acc[.][j] within the tile
    __device__ __forceinline__ int p_of(int i) const { return 16 * (wp + WP * i) + 4 * (lane >> 4); }
    __device__ __forceinline__ int q_of(int j) const { return 16 * (wq + WQ * j) + (lane & 15); }
};

// Tile (tp, tq) of workgroup w of np x nq.  Workgroups go round-robin over the 8 XCDs, so
// in a band of eight tiles of p each XCD gets nq tiles, neighbours in q: the 32 CUs of an
// XCD share eight panels of P and nq / 8 of Q in its L2, and all XCDs read the same eight
// panels of P at a time.  (A contiguous run of all tiles for each XCD reads P once for each
// from HBM unless nq is a multiple of 32: 8192 x 4096 x 128256 with 29 tiles of q 6.2 ms
// against 5.7.)
__device__ __forceinline__ void product_tile(int w, int np, int nq, int &tp, int &tq)
{
    const int band = w / (8 * nq) * 8;
    const int wide = min(8, np - band);
    const int loc = w - band * nq, all = wide * nq;
    const int place = loc < all / 8 * 8 ? (loc % 8) * (all / 8) + loc / 8 : loc;
    tq = place / wide;
    tp = band + place % wide;
}

}  // namespace mxq
