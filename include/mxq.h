/*
 * mxq.h -- C ABI of libmxq: MX block-32 FP4 quantization with a block
 * Hadamard rotation, and the block-scaled FP4 weight-gradient GEMM, for AMD
 * Instinct MI355X (gfx950).
 *
 * The method follows four web pages:
 *  - htx.com (es-es) news on "Pretraining large language models with MXFP4 on
 *    Native FP4 Hardware" (arXiv 2605.09825): section "Que es MXFP4?" (blocks
 *    of 32 elements with one shared E8M0 exponent, the block's largest
 *    exponent; 4-bit float elements) and section "Experimento de diagnostico"
 *    (the Fprop / Dgrad / Wgrad GEMMs Y = X W^T, dX = dY W, dW = dY^T X;
 *    stochastic rounding; Hadamard transform after random sign inversion).
 *  - gist.science (pt) summary "Pre-treinamento de Modelos de Linguagem
 *    Grandes com MXFP4": section "Metodologia" (deterministic H16 and H32
 *    rotations).
 *  - gist.science (pt, ko) summary "Repensando o Vies de Encolhimento
 *    (Shrinkage Bias) no Pre-treinamento de LLMs em FP4": "Metodologia 1"
 *    (RTNE on the non-uniform E2M1 grid and its shrinkage bias (l_i - r_i)/2),
 *    "Metodologia 2" (the uniform E1M2 / INT4-style grid; SR only on dY),
 *    "Resultados Experimentais" (SQNR diagnostics) and "Eficiencia" (fused
 *    rotation + quantization).
 *
 * Conventions for every call:
 *  - All tensor pointers are DEVICE pointers owned by the caller; the library
 *    allocates nothing and keeps no mutable global state, except the static
 *    per-device workspace of mxq_bias_stats_noalloc (below).
 *  - `stream` is a hipStream_t passed as void* (NULL = the default stream).
 *    Work is enqueued asynchronously; nothing is synchronized.
 *  - Arguments are validated on the host before any launch; on failure the
 *    call returns a non-zero mxq_status and has no side effect.  A failed
 *    launch returns MXQ_ERR_DEVICE.  Faults inside kernels surface at the
 *    caller's next synchronization.  Nothing is printed.
 *  - Calls are thread-safe; calls that write the same output race.
 */
#ifndef MXQ_H
#define MXQ_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define MXQ_ABI_VERSION 5

typedef int32_t mxq_status;
#define MXQ_OK 0
#define MXQ_ERR_NULL 1          /* a required pointer is NULL                 */
#define MXQ_ERR_SHAPE 2         /* a size is negative / not a multiple of 32  */
#define MXQ_ERR_ALIGN 3         /* a pointer or leading dimension misaligned  */
#define MXQ_ERR_UNSUPPORTED 4   /* an enum value or combination not supported */
#define MXQ_ERR_DEVICE 5        /* the HIP launch failed                      */
#define MXQ_ERR_WORKSPACE 6     /* the workspace is missing or too small      */

/* Element grids (the 3-bit magnitude m of a sign-magnitude nibble s<<3|m):
 *   MXQ_GRID_E2M1: m -> {0, 0.5, 1, 1.5, 2, 3, 4, 6}; top-level exponent emax 2.
 *   MXQ_GRID_E1M2: m -> 0.5*m = {0, 0.5, ..., 3.5} (uniform); emax 1.
 *   MXQ_GRID_E2M1_MAX4, MXQ_GRID_E2M1_MAX3: E2M1 with its range restricted,
 *     the ablation of the gist.science summary "Repensando o Vies de
 *     Encolhimento ... em FP4", "Resultados Experimentais": E2M1's codes and
 *     values up to a cap of 4 (m <= 6) or 3 (m <= 5); larger magnitudes go to
 *     the cap.  emax 1 for both, so a block's normalized maximum lies in
 *     [2, 4).  Their codes are plain E2M1 nibbles (FP4 operands of the
 *     matrix cores as they stand).
 * In general emax = ceil(log2(top level)) - 1: the block maximum is mapped
 * into the binade (2^emax, 2^(emax+1)] that holds the grid's top level. */
#define MXQ_GRID_E2M1 0
#define MXQ_GRID_E1M2 1
#define MXQ_GRID_E2M1_MAX4 2
#define MXQ_GRID_E2M1_MAX3 3

/* Rounding of the normalized magnitude a = |y| / 2^e onto the grid:
 *   MXQ_ROUND_RTNE: nearest level, ties to the even code, saturating.
 *   MXQ_ROUND_SR:   between the neighbouring levels q_k <= a < q_(k+1), round
 *                   up iff r + 1/2 < p * 2^B with p = (a - q_k)/(q_(k+1) - q_k)
 *                   and r the element's B random bits (below); a at or above
 *                   the top level stays at the top level. */
#define MXQ_ROUND_RTNE 0
#define MXQ_ROUND_SR 1

/* Code storage of one 32-element block:
 *   MXQ_FMT_FP4:  16 bytes; byte j = nibble(2j) | nibble(2j+1) << 4.
 *   MXQ_FMT_E2M3: 24 bytes; element i is the OCP FP6 E2M3 code (sign in bit 5)
 *                 of the same value, at bits 6i..6i+5 of the little-endian
 *                 192-bit block.  Lossless for both grids; it is the operand
 *                 form the FP6 matrix cores read (E1M2 levels are not E2M1). */
#define MXQ_FMT_FP4 0
#define MXQ_FMT_E2M3 1

/* Placement of a block-quantized tensor's blocks in memory:
 *   MXQ_LAYOUT_ROWS:  codes [lines][k/32][block bytes], scales [lines][k/32].
 *   MXQ_LAYOUT_MFMA:  the operand order of the 16x16x128 block-scaled matrix
 *                     cores, so a GEMM streams each operand contiguously.
 *                     With T = ceil(lines/16) tiles of 16 lines, K steps of 4
 *                     blocks (s = b / 4) and lane l = 16 g + r for block
 *                     4 s + g of line 16 t + r:
 *                       codes  [k/128 steps][T][64 lanes][block bytes],
 *                       scales [ceil(k/512) groups][T][64 lanes][4 bytes],
 *                     byte j of a lane's scale word is the scale of step
 *                     4 q + j of group q.  Needs k % 128 == 0.  The bytes of
 *                     padding lines (lines..16T-1) and of absent steps in a
 *                     last partial group are never written or read. */
#define MXQ_LAYOUT_ROWS 0
#define MXQ_LAYOUT_MFMA 1

#define MXQ_AXIS_ROW 0          /* blocks run along the last (contiguous) dim */
#define MXQ_AXIS_COL 1          /* blocks run along the first dim; transposed */

#define MXQ_OUT_F32 0
#define MXQ_OUT_BF16 1

#define MXQ_SIGNS_MASK 0        /* one sign mask shared by every block        */
#define MXQ_SIGNS_PER_BLOCK 1   /* each block draws its own 32 signs          */

/* Quantizer knobs.
 * hadamard_n: 0 (no rotation), 16 or 32.  Each n-element sub-block of a
 *   32-block is replaced by fl32(1/sqrt(n)) * H_n * (D x), H_n the Sylvester
 *   Hadamard matrix in natural order, computed in fp32 by butterfly stages of
 *   stride 1, 2, 4, ... (the stage order fixes the fp32 rounding).
 * sign_mode, sign_mask, sign_seed: D = diag(d_i) for position i of the
 *   32-block, the random sign inversion before the transform (htx.com news,
 *   "Experimento de diagnostico").
 *   MXQ_SIGNS_MASK: d_i = -1 where bit (i mod n) of sign_mask is set, the
 *     same for every block; mask 0 gives the deterministic Hadamard
 *     rotation, a random mask the randomized one (RHT).
 *   MXQ_SIGNS_PER_BLOCK: a sign vector as long as the quantization axis.
 *     The block with index j along that axis (the same j on every line)
 *     takes d_i = -1 where bit i of word 0 of Philox4x32-10 is set, with key
 *     (lo32(sign_seed), hi32(sign_seed)) and counter (lo32(j), hi32(j),
 *     0xFFFFFFFF, 0xFFFFFFFE).
 *   Both operands of one GEMM must use the same signs along their shared
 *   axis (same mode and mask or seed); the rotation then cancels.
 * sr_seed, sr_stream, sr_bits: the stochastic-rounding stream.  Element j of
 *   the block with index b (its position in the scale array, row-major) takes
 *   Philox4x32-10 with key (lo32(seed), hi32(seed)):
 *     B = 16: counter (j>>3, lo32(b), hi32(b), stream), 16-bit half (j&1) of
 *             output word ((j>>1)&3);
 *     B = 8:  counter (j>>4, lo32(b), hi32(b), stream), byte (j&3) of word
 *             ((j>>2)&3). */
typedef struct {
    int32_t grid;
    int32_t round;
    int32_t hadamard_n;
    uint32_t sign_mask;
    uint64_t sr_seed;
    uint32_t sr_stream;
    uint32_t sr_bits;
    uint32_t sign_mode;   /* MXQ_SIGNS_* */
    uint32_t reserved;    /* 0 */
    uint64_t sign_seed;   /* key of the per-block signs */
} mxq_qconfig;

/* A block-quantized tensor of `lines` lines, each `k` elements long (k % 32
 * == 0): 16 (FP4) or 24 (E2M3) code bytes and one E8M0 scale byte (value
 * 2^(s-127); 0xFF marks a non-finite block) per 32-element block, placed as
 * `layout` says.  codes must be 4-byte aligned (16-byte for MXQ_LAYOUT_MFMA,
 * whose scales must be 4-byte aligned). */
typedef struct {
    void *codes;
    uint8_t *scales;
    int32_t fmt;     /* MXQ_FMT_* */
    int32_t grid;    /* MXQ_GRID_* of the stored values */
    int32_t layout;  /* MXQ_LAYOUT_* */
} mxq_qtensor;

/* Shrinkage-bias / SQNR sums over the rotated values y of the blocks with a
 * finite scale (fp64, fixed-order reduction, so repeatable).  e is the
 * block's scale exponent, a = |y| 2^-e, yhat the reconstruction. */
typedef struct {
    double sum_abs_y;          /* sum |y|                                     */
    double sum_signed_err;     /* sum sign(y) (yhat - y)                      */
    double sum_y2;             /* sum y^2                                     */
    double sum_err2;           /* sum (yhat - y)^2                            */
    double sum_err_norm;       /* sum (|yhat| - |y|) 2^-e                     */
    double sum_err_norm_sat;   /* the same over elements with a > top level   */
    double level_err_norm[8];  /* per magnitude code m: sum (G_m - a)         */
    uint64_t n;                /* elements counted                            */
    uint64_t n_saturated;      /* elements with a > top level                 */
    uint64_t n_nonfinite_blocks;
    uint64_t level_count[8];
} mxq_stats;

/* Fused rotate + scale + round + pack of a bf16 matrix x [rows x cols]
 * (row-major, leading dimension ld_x >= cols elements, x 2-byte aligned;
 * 128-bit loads are used when x is 16-byte aligned and ld_x % 8 == 0, else
 * 16-bit loads), the quantization of every GEMM operand in the three training
 * GEMMs (htx.com news, "Experimento de diagnostico"; the fused form follows
 * the "Eficiencia" section of the shrinkage-bias summary).
 *   row_out (may be NULL): blocks along cols, lines = rows, k = cols
 *                          (needs cols % 32 == 0).
 *   col_out (may be NULL): blocks along rows, written transposed: lines =
 *                          cols, k = rows (needs rows % 32 == 0).
 * At least one output is required; with both, one pass produces both (the
 * row output rotates along cols, the column output along rows, each with the
 * same mask).  Each output's grid must equal cfg->grid.
 * Errors: NULL cfg/x/outputs -> MXQ_ERR_NULL; bad sizes -> MXQ_ERR_SHAPE;
 * misaligned x/codes -> MXQ_ERR_ALIGN; bad knobs -> MXQ_ERR_UNSUPPORTED. */
mxq_status mxq_quantize(const mxq_qconfig *cfg, const void *x, int64_t rows, int64_t cols,
                        int64_t ld_x, const mxq_qtensor *row_out, const mxq_qtensor *col_out,
                        void *stream);

/* One tensor of mxq_quantize_batch: the arguments of one mxq_quantize call. */
typedef struct {
    const mxq_qconfig *cfg;
    const void *x;
    int64_t rows, cols, ld_x;
    const mxq_qtensor *row_out;  /* may be NULL */
    const mxq_qtensor *col_out;  /* may be NULL */
} mxq_quantize_job;

/* mxq_quantize for `count` tensors at once, e.g. the two operands of the
 * weight-gradient product, dY with SR and X with RTNE (htx.com news,
 * "Experimento de diagnostico").  The outputs are bit-identical to calling
 * mxq_quantize on each job in turn.  Every job is checked first, with
 * mxq_quantize's checks and status codes; on the first failure nothing is
 * launched and that status is returned.  Consecutive jobs that ask for a
 * column output only and share the grid family (E1M2, or the E2M1 grids),
 * hadamard_n and the column code format run as ONE launch (up to 8 jobs per
 * launch), their workgroups in job order; the rounding mode, seeds, signs,
 * shapes and layouts may differ.  Other jobs get their own launches, in
 * order.  No output may overlap another job's output or input (inputs may
 * be shared).  count == 0 does nothing; count < 0 -> MXQ_ERR_SHAPE; NULL
 * jobs with count > 0 -> MXQ_ERR_NULL.  A launch failure returns
 * MXQ_ERR_DEVICE; the launches before it stay enqueued. */
mxq_status mxq_quantize_batch(const mxq_quantize_job *jobs, int32_t count, void *stream);

/* Reconstruct yhat = (-1)^s G_m 2^(scale-127) (NaN for scale 0xFF) of a
 * block-quantized tensor into out [lines x k] (leading dimension ld_out
 * elements), as fp32 or bf16 (both exact).  The shared-exponent
 * reconstruction of the htx.com news, section "Que es MXFP4?". */
mxq_status mxq_dequantize(const mxq_qtensor *q, int64_t lines, int64_t k, int32_t out_dtype,
                          void *out, int64_t ld_out, void *stream);

/* The weight-gradient GEMM dW = dY^T X of the htx.com news ("Experimento de
 * diagnostico"), on block-quantized operands that both run along the token
 * axis: C [m x n] fp32 (leading dimension ldc) = A [m x k] * B [n x k]^T,
 * where A = dY quantized column-wise (m = its column count) and B = X
 * quantized column-wise.  Each product term carries both block scales; the
 * sum is accumulated in fp32 on the block-scaled matrix cores.
 * Operands: FP4 codes of the E2M1 grid, or E2M3 codes of either grid (A and
 * B may differ).  k % 128 == 0; m, n >= 0 (any).  C is fully overwritten.
 * Deterministic: no split-K, fixed summation order. */
mxq_status mxq_wgrad_gemm(const mxq_qtensor *a, const mxq_qtensor *b, int64_t m, int64_t n,
                          int64_t k, float *c, int64_t ldc, void *stream);

/* The rotation step of mxq_quantize on its own (the first kernel of the
 * unfused pipeline that the fused quantizer replaces, gist.science summary
 * "Repensando o Vies de Encolhimento (Shrinkage Bias) no Pre-treinamento de
 * LLMs em FP4", section "Eficiencia"): y = fl32(1/sqrt(n)) H_n (D x) on every
 * n-element sub-block of the 32-blocks along `axis` (MXQ_AXIS_ROW: along the
 * last dimension; MXQ_AXIS_COL: along the first), written to out in x's own
 * orientation [rows x cols], leading dimension ld_out elements.  out_dtype
 * MXQ_OUT_F32 gives exactly the values mxq_quantize rounds; MXQ_OUT_BF16
 * rounds them to nearest even.  cfg->hadamard_n must be 16 or 32 (cfg's
 * grid / rounding fields are ignored).  Requires the axis length % 32 == 0
 * and x, out aligned to their element size; 16-byte aligned rows
 * (out % 16 == 0, ld_out * element size % 16 == 0) take vector stores. */
mxq_status mxq_rotate(const mxq_qconfig *cfg, const void *x, int64_t rows, int64_t cols,
                      int64_t ld_x, int32_t axis, int32_t out_dtype, void *out, int64_t ld_out,
                      void *stream);

/* The same block-scaled product under its general name, for the three GEMMs
 * of a linear layer in the htx.com news ("Experimento de diagnostico"):
 *   Fprop  Y [T x N]  = X [T x K] W^T:  a = X row-wise,  b = W row-wise
 *          (m = T, n = N, k = K);
 *   Dgrad  dX [T x K] = dY [T x N] W:  a = dY row-wise, b = W column-wise
 *          (W's blocks run along N; m = T, n = K, k = N);
 *   Wgrad  dW [N x K] = dY^T X:        a = dY column-wise, b = X column-wise
 *          (m = N, n = K, k = T).
 * Both operands of one product must carry the same rotation along k (same
 * hadamard_n and sign_mask), which then cancels in the product.  Arguments,
 * requirements and errors as mxq_wgrad_gemm. */
mxq_status mxq_gemm_abt(const mxq_qtensor *a, const mxq_qtensor *b, int64_t m, int64_t n,
                        int64_t k, float *c, int64_t ldc, void *stream);

/* Bias / SQNR statistics of the shrinkage-bias summary ("Metodologia 1",
 * "Resultados Experimentais") for a tensor q produced by mxq_quantize from x
 * with the same cfg and axis; the rotated y is recomputed exactly as the
 * quantizer does.  `out` is a DEVICE pointer to one mxq_stats, fully
 * overwritten.  `workspace` is a device buffer of at least
 * mxq_bias_stats_workspace_size(rows, cols, axis) bytes. */
mxq_status mxq_bias_stats(const mxq_qconfig *cfg, const void *x, int64_t rows, int64_t cols,
                          int64_t ld_x, int32_t axis, const mxq_qtensor *q, mxq_stats *out,
                          void *workspace, size_t ws_bytes, void *stream);
/* Utility (no passage defines it): the workspace mxq_bias_stats needs, in
 * bytes (0 for negative sizes). */
size_t mxq_bias_stats_workspace_size(int64_t rows, int64_t cols, int32_t axis);

/* The effective bucket ratio that the shrinkage-bias summary ("Resultados
 * Experimentais") reports rising under the Hadamard rotation, which the
 * pages do not define; read here as exp(H) / L, with H the entropy (nats) of
 * the magnitude-code histogram stats->level_count and L the number of levels
 * `grid` emits (8; 7 and 6 for E2M1 capped at 4 and 3).  1 when all levels are
 * used equally, 1/L when all elements share one.  Host function: `stats` is a
 * HOST pointer (an mxq_stats copied back from the device).  Returns NaN for a
 * NULL pointer, an unknown grid or an empty histogram. */
double mxq_bucket_ratio(const mxq_stats *stats, int32_t grid);

/* mxq_bias_stats for callers that cannot allocate (code under HIP graph
 * capture, tight serving loops, harnesses that forbid hipMalloc): the same
 * arguments without the workspace, the same checks, status codes and
 * results.  The workspace is a static device array of 204800 bytes that
 * each GPU holds until the process ends, found on the first call on a device
 * (with that device current; `stream` must belong to the current device).
 * A call that would need more returns MXQ_ERR_WORKSPACE (none does: the
 * workspace is at most 204800 bytes for any size).  The call allocates
 * nothing.  Every call on one GPU shares its array: calls that overlap on
 * one GPU race. */
mxq_status mxq_bias_stats_noalloc(const mxq_qconfig *cfg, const void *x, int64_t rows,
                                  int64_t cols, int64_t ld_x, int32_t axis, const mxq_qtensor *q,
                                  mxq_stats *out, void *stream);

/* The rounding step of mxq_quantize on its own, for checks of every input
 * value: codes[i] = the sign-magnitude nibble of a[i] (a value already
 * divided by its block scale 2^e, so |a| < 2^(emax+1) is the meaningful
 * range; larger magnitudes saturate) under the grid and rounding of the
 * shrinkage-bias summary ("Metodologia 1" RTNE, "Metodologia 2" SR).  For SR,
 * rand[i] holds element i's sr_bits random bits (the caller draws them);
 * rand may be NULL for RTNE.  a, rand, codes are device arrays of n items. */
mxq_status mxq_round_to_grid(int32_t grid, int32_t round, int32_t sr_bits, const float *a,
                             const uint16_t *rand, int64_t n, uint8_t *codes, void *stream);

/* A random sign mask for the randomized Hadamard rotation (RHT: random sign
 * inversion before the transform, htx.com news "Experimento de diagnostico";
 * gist.science summary "Pre-treinamento de Modelos de Linguagem Grandes com
 * MXFP4", "Metodologia"), drawn from a seed: the low n bits (n = 16 or 32) of
 * output word 0 of Philox4x32-10 with key (lo32(seed), hi32(seed)) and counter
 * (0, 0xFFFFFFFF, 0xFFFFFFFF, 0xFFFFFFFF) -- a counter no block of the
 * stochastic-rounding stream uses.  Host function; returns 0 for other n. */
uint32_t mxq_rht_sign_mask(uint64_t seed, uint32_t n);

/* ---- the operators around the quantized products ---------------------------
 * The norm before a linear layer (its output is what mxq_quantize takes, its
 * backward pass takes mxq_gemm_abt's fp32 output), and the two ends of the
 * output layer: log probabilities with alternatives, and the distillation
 * loss.  No passage of the pages defines these; the formulas below do.
 *  - Tensors are fp32 or bf16 per their own *_dtype argument (MXQ_OUT_F32 /
 *    MXQ_OUT_BF16); all arithmetic is fp32, rounded once (nearest, ties to
 *    even) where bf16 is stored.  Pointers must be aligned to their element
 *    size only; leading dimensions (elements) may be any number >= the row length.
 *  - rows == 0 launches nothing (mxq_norm_backward then clears dgamma and
 *    dbeta), whatever the row pointers are.
 *  - Sums run in a fixed order: repeated calls give the same bits. */
#define MXQ_NORM_LAYER 0
#define MXQ_NORM_RMS 1

/* y = (x - mu) rstd gamma + beta for each row of x [rows x cols]:
 *   MXQ_NORM_LAYER: mu the row's mean, rstd = 1 / sqrt(mean((x - mu)^2) + eps);
 *   MXQ_NORM_RMS:   mu = 0,            rstd = 1 / sqrt(mean(x^2) + eps).
 * gamma, beta (fp32 [cols]) may be NULL (1 and 0).  mean, rstd (fp32 [rows])
 * may be NULL; they are what mxq_norm_backward takes (RMS writes no mean).
 * cols >= 1, eps finite and >= 0.  y may be x itself (same dtype and leading
 * dimension).  Rows that are not finite follow the formula in IEEE arithmetic
 * and leave the others alone. */
mxq_status mxq_norm_forward(int32_t kind, const void *x, int32_t x_dtype, int64_t ld_x,
                            int64_t rows, int64_t cols, const float *gamma, const float *beta,
                            float eps, void *y, int32_t y_dtype, int64_t ld_y, float *mean,
                            float *rstd, void *stream);

/* The backward pass of mxq_norm_forward from its mean (NULL for RMS) and rstd.
 * With n = (x - mu) rstd and u = dy gamma, means over the row:
 *   dx = rstd (u - n mean(u n) - mean(u))   (the last term for LAYER only);
 *   dgamma = sum over rows of dy n,  dbeta = sum over rows of dy  (fp32 [cols],
 *   each may be NULL; overwritten).
 * dx may be NULL, or dy or x itself (same dtype and leading dimension).
 * workspace: mxq_norm_backward_workspace_size(rows, cols) bytes, 4-byte
 * aligned; needed only when dgamma or dbeta is asked for. */
mxq_status mxq_norm_backward(int32_t kind, const void *dy, int32_t dy_dtype, int64_t ld_dy,
                             const void *x, int32_t x_dtype, int64_t ld_x, int64_t rows,
                             int64_t cols, const float *gamma, const float *mean,
                             const float *rstd, void *dx, int32_t dx_dtype, int64_t ld_dx,
                             float *dgamma, float *dbeta, void *workspace, size_t ws_bytes,
                             void *stream);
size_t mxq_norm_backward_workspace_size(int64_t rows, int64_t cols);

/* The softmax distribution q = softmax(z / temperature) of each row z of
 * logits [rows x vocab], as m = max z and S = sum exp((z - m) / temperature):
 *   logprob[r]  = log q at tokens[r] (int32; < 0: no token, 0 is written;
 *                 >= vocab: NaN);
 *   entropy[r]  = -sum q log q;
 *   stats[r]    = (m, S), fp32 pairs, what the backward passes take;
 *   top_ids, top_logprobs [rows x top_k]: the top_k largest logits in falling
 *                 order, equal ones by index, and their log q.  0 <= top_k <= 64
 *                 (MXQ_TOP_MAX).
 * Outputs other than stats may be NULL (tokens with logprob; the top pair
 * together, top_k then 0).  Logits of -inf are masked: they have q = 0, are no
 * alternatives, and where fewer than top_k are left, the ids are -1 and their
 * log q -inf.  A row with every logit masked has S = 0, entropy 0 and log q
 * -inf.  A row that holds a NaN or +inf has no distribution: its floating
 * outputs are NaN (stats: S), its ids -1.  1 <= vocab <= 2^31 - 64, temperature
 * a positive normal number.
 * workspace: mxq_vocab_workspace_size(rows, vocab, top_k) bytes, 8-byte aligned
 * (may be NULL where that is 0). */
#define MXQ_TOP_MAX 64
mxq_status mxq_token_logprobs(const void *logits, int32_t dtype, int64_t ld, int64_t rows,
                              int64_t vocab, float temperature, const int32_t *tokens,
                              float *logprob, float *entropy, float *stats, int32_t top_k,
                              int32_t *top_ids, float *top_logprobs, void *workspace,
                              size_t ws_bytes, void *stream);
/* The workspace of mxq_token_logprobs, mxq_distill_forward and mxq_distill
 * (those two: top_k = 0), in bytes; 0 for sizes they refuse. */
size_t mxq_vocab_workspace_size(int64_t rows, int64_t vocab, int32_t top_k);

/* The gradient of mxq_token_logprobs' logprob and entropy, from its stats and
 * entropy and the gradients d_logprob, d_entropy [rows] (either may be NULL: 0;
 * entropy and d_entropy go together, tokens and d_logprob too):
 *   dz_v = (d_logprob (1[v = token] - q_v) - d_entropy q_v (log q_v + entropy)) / temperature
 * into dlogits (all vocab columns of every row; may be logits itself, same
 * dtype and leading dimension).  Token < 0: d_logprob counts as 0;
 * token >= vocab: the row is NaN.  Masked logits have q = 0, so a row with every
 * logit masked has the gradient d_logprob / temperature at its token and 0
 * elsewhere.  Rows without a distribution are NaN. */
mxq_status mxq_token_logprobs_backward(const void *logits, int32_t dtype, int64_t ld,
                                       int64_t rows, int64_t vocab, float temperature,
                                       const int32_t *tokens, const float *stats,
                                       const float *entropy, const float *d_logprob,
                                       const float *d_entropy, void *dlogits,
                                       int32_t dlogits_dtype, int64_t ld_dlogits, void *stream);

/* Distillation from a teacher's top alternatives: top_k (1..MXQ_TOP_MAX) ids
 * (int32, < 0: absent) and log probabilities (fp32) a row, packed [rows x
 * top_k], as mxq_token_logprobs writes them at the same temperature.
 * p_j = exp(teacher_logprobs_j), divided by their sum where renormalize is 1
 * (then any logits / temperature serve); with q as above, P = sum p_j and
 * weight w (fp32 [rows], NULL: 1):
 *   loss[r] = w temperature^2 sum_j p_j (log p_j - log q at id_j)
 *   dz_v    = w temperature (P q_v - sum over j with id_j = v of p_j),
 * which is the gradient of the sum of the losses.  One certain alternative
 * (top_k = 1, log probability 0) at temperature 1 is the cross entropy.
 * A row with w = 0, or without a present alternative of p > 0, has loss 0 and
 * gradient 0 whatever else it holds; an id >= vocab makes its row NaN.  An id may
 * come twice.  Where a p > 0 meets a masked logit, the loss is +inf and the
 * gradient finite; with every logit masked (q = 0) the gradient is
 * -w temperature p at the ids and 0 elsewhere.
 *   mxq_distill_forward:  loss and stats (as mxq_token_logprobs writes them;
 *                         rows of w = 0 get (0, 1)).
 *   mxq_distill_backward: dlogits from stats; w then is the gradient of the
 *                         unweighted loss.
 *   mxq_distill:          loss and dlogits in one pass.
 * dlogits may be logits itself (same dtype and leading dimension). */
mxq_status mxq_distill_forward(const void *logits, int32_t dtype, int64_t ld, int64_t rows,
                               int64_t vocab, float temperature, const int32_t *teacher_ids,
                               const float *teacher_logprobs, int32_t top_k, int32_t renormalize,
                               const float *weight, float *loss, float *stats, void *workspace,
                               size_t ws_bytes, void *stream);
mxq_status mxq_distill_backward(const void *logits, int32_t dtype, int64_t ld, int64_t rows,
                                int64_t vocab, float temperature, const int32_t *teacher_ids,
                                const float *teacher_logprobs, int32_t top_k,
                                int32_t renormalize, const float *weight, const float *stats,
                                void *dlogits, int32_t dlogits_dtype, int64_t ld_dlogits,
                                void *stream);
mxq_status mxq_distill(const void *logits, int32_t dtype, int64_t ld, int64_t rows, int64_t vocab,
                       float temperature, const int32_t *teacher_ids,
                       const float *teacher_logprobs, int32_t top_k, int32_t renormalize,
                       const float *weight, float *loss, void *dlogits, int32_t dlogits_dtype,
                       int64_t ld_dlogits, void *workspace, size_t ws_bytes, void *stream);

/* ---- the ends of a training step --------------------------------------------
 * Softmax cross entropy of an output layer from its hidden states and weight,
 * a piece of the vocabulary at a time: the logits z = x w^T are never kept.
 * With q = softmax(z / temperature) and weight[r] (fp32 [rows], NULL: 1),
 *   loss[r]  = -weight[r] log q at targets[r];
 *   stats[r] = (m, S) as mxq_token_logprobs writes them, S = sum exp((z - m) / temperature);
 *   dz       = weight[r] / temperature (q - 1[v = target]),
 *   dx = dz w,  dw = dz^T x,
 * the gradients of the sum of the losses.  In the backward pass weight is the
 * gradient of the unweighted loss.
 *  - x [rows x hidden], w [vocab x hidden], dx, dw (as x, w) are bf16.  hidden is a
 *    multiple of 32.  w and dw are 16-byte aligned, their leading dimensions
 *    multiples of 8 and at most 2^22; x and dx stand at any element.  hidden is
 *    at most 2^16, vocab 2^24, rows 2^22, rows x vocab 2^37.
 *  - Products of bf16 values are summed in fp32; dz is rounded to bf16, dx and dw
 *    where they are stored.  What the rounding leaves of dz at a row's target, mostly
 *    its largest entry, is added to both sums (to dw in bf16 of its own).
 *  - A row with a target < 0 or a weight of 0 does not count: loss 0, stats
 *    (0, 1), dx 0, nothing in dw, whatever else it holds; and it is left out of all
 *    products, except in forward passes of up to 128 rows that are read in place.  A
 *    target >= vocab makes its row's loss and dx NaN, and dw with them.  Rows that
 *    hold NaN or infinities follow the formulas (a row whose logits hold a NaN or
 *    +inf has no distribution: S, loss and gradients NaN); the other rows' losses,
 *    stats and dx are left alone.
 *  - Sums run in a fixed order: repeated calls give the same bits.
 *  - rows == 0: the forward pass does nothing, the backward pass clears dw.
 *  - dx or dw may be NULL.  No output may overlap an input.
 * workspace: 16-byte aligned, of the size that the functions below give (0 for
 * sizes that are refused): the rows that count, packed; with them for the forward
 * pass 8 bytes for each row and 64, 128 or 256 entries of the vocabulary (the fewer
 * rows and entries, the fewer), for the backward pass dz of a piece (up to 256 MiB
 * and a part, above 2^19 rows 512 bytes a row) and the sums of dx in fp32. */
mxq_status mxq_linear_ce_forward(const void *x, int64_t ld_x, const void *w, int64_t ld_w,
                                 int64_t rows, int64_t hidden, int64_t vocab, float temperature,
                                 const int32_t *targets, const float *weight, float *loss,
                                 float *stats, void *workspace, size_t ws_bytes, void *stream);
size_t mxq_linear_ce_forward_workspace_size(int64_t rows, int64_t hidden, int64_t vocab);
mxq_status mxq_linear_ce_backward(const void *x, int64_t ld_x, const void *w, int64_t ld_w,
                                  int64_t rows, int64_t hidden, int64_t vocab, float temperature,
                                  const int32_t *targets, const float *weight, const float *stats,
                                  void *dx, int64_t ld_dx, void *dw, int64_t ld_dw,
                                  void *workspace, size_t ws_bytes, void *stream);
size_t mxq_linear_ce_backward_workspace_size(int64_t rows, int64_t hidden, int64_t vocab);

/* The global norm over a list of gradients, and their clipping to a largest
 * norm, the last step in front of an optimizer:
 *   sum_sq = sum over all elements of all tensors of g^2,  norm = sqrt(sum_sq);
 *   c = min(1, max_norm / (norm + eps)),  out = c g.
 * A tensor is n elements in a row from g, fp32 or bf16, at any element; out has
 * the same number in its own type, and may be g itself (same type).  The list is
 * a HOST array, read by the call.
 *  - sum_sq (device, fp64) is summed in fp64 in a fixed order, norm (device,
 *    fp32) is rounded from its root; either may be NULL.  Ranks that each hold a
 *    part of the gradients add their sum_sq up between the two calls.
 *  - c is formed in fp64 and rounded to fp32's 24 bits, c g rounded in fp32,
 *    then to bf16 where out is.  Where c is 1, out is g; out == g is then left alone.
 *  - A norm that is infinite gives c = 0, one that is NaN c = NaN, in IEEE
 *    arithmetic (infinities become NaN, and everything does).
 *  - Empty tensors and empty lists serve (norm 0); a list has at most 2^38
 *    elements.  An out may overlap no other tensor's g or out, nor a part of its
 *    own g (these calls do not look for it).  max_norm and eps are finite and
 *    >= 0; where max_norm, norm and eps are all 0, c is NaN.
 *  - mxq_grad_norm only reads g, n and dtype.
 * workspace: mxq_grad_norm_workspace_size(grads, count) bytes, 8-byte aligned (0
 * for empty lists and those that are refused). */
typedef struct {
    const void *g;
    void *out;
    int64_t n;
    int32_t dtype;      /* MXQ_OUT_* of g */
    int32_t out_dtype;  /* MXQ_OUT_* of out */
} mxq_grad;
mxq_status mxq_grad_norm(const mxq_grad *grads, int64_t count, float *norm, double *sum_sq,
                         void *workspace, size_t ws_bytes, void *stream);
size_t mxq_grad_norm_workspace_size(const mxq_grad *grads, int64_t count);
mxq_status mxq_grad_clip(const mxq_grad *grads, int64_t count, const double *sum_sq,
                         float max_norm, float eps, void *stream);

/* Utilities (no passage defines them): a static description of a status
 * code, and the ABI version the library was built with (MXQ_ABI_VERSION). */
const char *mxq_status_string(mxq_status s);
int32_t mxq_abi_version(void);

#ifdef __cplusplus
}
#endif
#endif /* MXQ_H */
