/*
 * mixed_gemm.h -- C ABI of the smoothed, outlier-split, dual-branch W4A4
 * linear layer for AMD Instinct MI355X (gfx950).
 *
 * The layer is the one of "W4A4 Quantization for Inference on
 * Wan2.2-I2V-A14B" (arXiv 2606.29337):
 *   Eq. (1)  Y = (X / s)(s * W), s applied along input channels;
 *   Eq. (2)  s_j = act_max_j^alpha / w_max_j^(1 - alpha);
 *   Eq. (4)  O = top-k input channels by max_t |x_tj|;
 *   Eq. (5)  Y = X_J W^(q)_J + X_O W^(hp)_O: MXFP4 W4A4 bulk + BF16 outliers.
 * The life cycle is calibrate -> plan(alpha, k) -> forward.
 *
 * Conventions shared by every call
 * --------------------------------
 *  - X is [M][K] row-major (tokens x input channels); W is [N][K] row-major
 *    (nn.Linear layout, K contiguous); Y is [M][N] row-major bf16.
 *  - bf16 values travel as uint16_t bit patterns.
 *  - Every pointer argument is a DEVICE pointer owned by the caller; the
 *    library allocates no device memory and keeps no device state between
 *    calls.  Base pointers must be 16-byte aligned.
 *  - Every call validates its arguments on the host, then enqueues its
 *    kernels on `stream` and returns without synchronizing.  A device fault
 *    surfaces at the caller's next synchronization on that stream.
 *  - Return value: MG_OK (0) or a negative mg_status; mg_last_error() gives a
 *    message for the last failing call on the calling thread.
 *  - Inputs must be finite; NaN/Inf inputs give unspecified results.
 *  - MXFP4 = E2M1 elements + one E8M0 scale per 32 consecutive K (OCP MX):
 *    scale code c = floor(log2 amax) - 2 + 127 (clamped at 0), elements
 *    rounded to nearest, ties to the even code, saturating at +-6, sign copied
 *    (so -0 encodes as 0x8).  Two elements per byte, even K in the low nibble.
 */
#ifndef MIXED_GEMM_H
#define MIXED_GEMM_H

#include <stddef.h>
#include <stdint.h>
#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    MG_OK = 0,
    MG_ERR_ARG = -1,         /* null pointer, bad alpha, bad enum value          */
    MG_ERR_SHAPE = -2,       /* K or N not a multiple of 32, k > K, negative size */
    MG_ERR_DTYPE = -3,       /* dtype not MG_F32 / MG_BF16                        */
    MG_ERR_ALIGN = -4,       /* a base pointer not 16-byte aligned                */
    MG_ERR_UNSUPPORTED = -5, /* a size beyond the documented limits               */
    MG_ERR_HIP = -6          /* a HIP runtime call failed (launch error)          */
} mg_status;

typedef enum { MG_F32 = 0, MG_BF16 = 1 } mg_dtype;

/* Weight block-scale layout (the block-packing paragraph after Eq. (5) and
 * its Fig. 8):
 * MG_W_1X32   one E8M0 per (output row n, 32 consecutive K);
 * MG_W_32X32  one E8M0 per aligned tile of 32 output rows x 32 K (requires N % 32 == 0);
 * MG_W_128X1  one E8M0 per K-major stripe of 128 consecutive K of one output
 *             row (the last stripe of a row covers the remaining K when
 *             K % 128 != 0). */
typedef enum { MG_W_1X32 = 0, MG_W_32X32 = 1, MG_W_128X1 = 2 } mg_wlayout;

/* Score the outlier set of Eq. (4) ranks:
 * MG_SCORE_MAX       the calibration maximum a_j = max_t |x_tj| (Eq. (4) as written);
 * MG_SCORE_SMOOTHED  the smoothed maximum max_t |x_tj / s_j| = RN(a_j / s_j). */
typedef enum { MG_SCORE_MAX = 0, MG_SCORE_SMOOTHED = 1 } mg_score;

/* Plan descriptor.  K, N: input / output widths (multiples of 32, K <= 65536);
 * k: number of outlier columns, 0 <= k <= K; layout: mg_wlayout;
 * smooth: 1 to apply Eq. (2) with alpha in (0, 1), 0 for s = 1;
 * score: mg_score. */
typedef struct {
    int32_t K, N, k;
    int32_t layout;
    int32_t smooth;
    int32_t score;
    double alpha;
} mg_plan_desc;

/* Plan buffers (caller-allocated, sizes from mg_plan_bytes, in this order):
 *  s   [K]        f32  smoothing scales, Eq. (2), evaluated in f64, rounded once;
 *  rcp [K]        f32  RN(1/s_j), used inside the exact division of the forward;
 *  O   [k]        i32  outlier channels, ascending (null allowed when k == 0);
 *  pos [K]        i32  index of channel j in O, or -1;
 *  Wq  [N][K/2]   u8   MXFP4 payload of the folded bulk weights RN(s_j W[n][j]),
 *                      outlier columns set to +0 before encoding, in fragment
 *                      order (below);
 *  Ws             u8   E8M0 scale of each (row, 32-block), in scale windows
 *                      (below) -- for MG_W_32X32 the tile's code repeated on
 *                      each of its 32 rows, for MG_W_128X1 the stripe's code
 *                      on each of its 32-blocks;
 *  Wst                 compact codes: [N/32][K/32] u8 tile codes (MG_W_32X32),
 *                      [N][ceil(K/128)] u8 stripe codes (MG_W_128X1); null
 *                      allowed for MG_W_1X32;
 *  WO  [N][k]     bf16 folded outlier columns (2k bytes per row) in fragment
 *                      order; null allowed when k == 0.
 *
 * Fragment order (Wq, Aq: rows of K/2 bytes; WO, XO: rows of 2k bytes).  The
 * [rows][row_bytes] byte matrix is cut into blocks of 32 rows x 32 bytes --
 * one operand of a 32x32x64 FP4 or 32x32x16 bf16 matrix-core instruction --
 * each stored as 1024 contiguous bytes: block (g = r / 32, c = byte / 32) at
 * (g * ns + c) * 1024 with ns = 2 * ceil(row_bytes / 64) (an even number of
 * 32-byte slices per row), and inside it byte b of row r's slice at
 *     16 * (r % 32 + 32 * (b / 16)) + b % 16,
 * for ceil(rows / 32) * ns * 1024 bytes in all.  Pads -- rows up to the next
 * multiple of 32 and bytes up to ns * 32 per row -- hold 0 (zero codes, +0).
 * The dual GEMM copies whole 1 KB blocks, and a block's 16-byte pieces are
 * already in the order the instruction's 64 lanes take them.
 *
 * Scale windows (Ws, As).  The E8M0 codes of a [rows][K/32] scale matrix are
 * stored in windows of 256 rows x 16 blocks (512 channels), 16 bytes per row,
 * 4096 contiguous bytes per window, windows of a 256-row group consecutive.
 * Inside a window row the codes of the even blocks come first, then those of
 * the odd blocks: the code of (row r, block b) is at byte
 *     ((r / 256) * nwin + b / 16) * 4096 + (r % 256) * 16 + 8 * (b % 2) + (b % 16) / 2,
 * nwin = ceil(K / 512), for ceil(rows / 256) * nwin * 4096 bytes in all.  The
 * layout depends on K only (a buffer sized for more rows serves fewer).  The
 * writers fill the whole last 256-row group: blocks past K/32 and rows past
 * the matrix hold code 0, the code of an all-zero block.  The dual GEMM copies
 * one window of its 256x256 output tile's rows as 4 KB of contiguous memory. */
typedef struct {
    mg_plan_desc d;
    float* s;
    float* rcp;
    int32_t* O;
    int32_t* pos;
    uint8_t* Wq;
    uint8_t* Ws;
    uint8_t* Wst;
    uint16_t* WO;
} mg_plan;

/* Per-forward activation workspace (sizes from mg_act_bytes):
 *  Aq [M][K/2] u8 MXFP4 payload of the bulk quotients in fragment order, As
 *  the E8M0 code of each (row, 32-block) in scale windows, XO [M][k] bf16
 *  outlier quotients in fragment order (null allowed when k == 0); see mg_plan. */
typedef struct {
    uint8_t* Aq;
    uint8_t* As;
    uint16_t* XO;
} mg_act;

/* Library version (major*10000 + minor*100 + patch). */
int mg_version(void);

/* Message for the last failing call on this thread ("" if none). */
const char* mg_last_error(void);

/* Host-only size queries.  out[8] = bytes of s, rcp, O, pos, Wq, Ws, Wst, WO;
 * out[3] = bytes of Aq, As, XO for M rows.  A zero size means "may be null". */
int mg_plan_bytes(const mg_plan_desc* d, size_t out[8]);
int mg_act_bytes(const mg_plan_desc* d, int64_t M, size_t out[3]);

/* ---- calibration: per-input-channel activation maxima and weight column
 * ranges (the calibration paragraph before Eq. (4); Eq. (4)'s score). ---- */

/* act_max[0..K) := +0.  Start of a calibration run. */
int mg_calib_reset(float* act_max, int32_t K, hipStream_t stream);

/* act_max[j] = max(act_max[j], max_t |X[t][j]|) over the M rows of X
 * (dtype MG_F32 or MG_BF16).  Exact, order-independent: batches may be fed
 * in any order and split anywhere.  M == 0 is a no-op. */
int mg_calib_act(const void* X, int32_t dtype, int64_t M, int32_t K, float* act_max,
                 hipStream_t stream);

/* w_max[j] = max_n |W[n][j]| (overwrites w_max). */
int mg_weight_range(const void* W, int32_t dtype, int32_t N, int32_t K, float* w_max,
                    hipStream_t stream);

/* ---- percentile calibration statistic: an alternative score for Eq. (4)'s
 * top-k (the tail-aware percentile calibration page builds its channel mask
 * from a percentile of the activation tail, to damp rare calibration
 * outliers; it gives no formula or level -- the reading here is the nearest
 * rank). ----
 *
 * score[j] = the value of rank r = ceil(q T) (1-based, clamped to [1, T]) in
 * ascending order of |x_tj| over all T calibration rows of all batches, for
 * 0 < q <= 1 (q = 1 gives act_max; r is computed in double precision).  The
 * result is exact (one of the inputs' magnitudes), by a two-pass radix
 * selection on the bf16 bit patterns of |x|:
 *   mg_pct_reset; mg_pct_count(pass 0) on every batch; mg_pct_select(pass 0);
 *                 mg_pct_count(pass 1) on every batch; mg_pct_select(pass 1).
 * Pass 0 counts, per channel, the high byte of each |x|; its select finds the
 * byte holding rank r and the rank inside it, and clears the counts; pass 1
 * counts the low bits of the values with that high byte; its select writes
 * score.  Both passes must see the same rows (in any order and split);
 * otherwise the result is unspecified (NaN where a rank is not found).  With
 * no rows counted, score is 0.  bf16 X only.  The score may be passed to
 * mg_outlier_set in place of act_max (s still comes from act_max).
 *
 * State, caller-owned device memory: hist [K][256] u32 (1 KiB per channel),
 * sel [K][2] i32 (selected high byte, rank inside it).  One state serves one
 * statistic at a time; calls on one state must be stream-ordered. */
typedef struct {
    uint32_t* hist;      /* [K][256] */
    int32_t* sel;        /* [K][2]   */
    int32_t K;           /* multiple of 32 */
    int32_t reserved;    /* 0 */
} mg_pct;

/* Clears hist: the start of a percentile calibration run. */
int mg_pct_reset(const mg_pct* st, hipStream_t stream);

/* Adds the M rows of X [M][K] (bf16) to pass `pass` (0 or 1).  M == 0 is a
 * no-op; M above 65535^2 (4.29e9) rows in one call is MG_ERR_UNSUPPORTED
 * (split the batch).  Pass 1 reads sel (written by mg_pct_select pass 0). */
int mg_pct_count(const mg_pct* st, int32_t pass, const uint16_t* X, int64_t M, hipStream_t stream);

/* Pass 0: from the counts and q, sel := (high byte, rank inside it) per
 * channel, and hist is cleared (score unused, may be NULL).  Pass 1:
 * score[0..K) := the statistic (q unused).  q must lie in (0, 1]. */
int mg_pct_select(const mg_pct* st, int32_t pass, double q, float* score, hipStream_t stream);

/* ---- planning (offline, once per layer) ---- */

/* Eq. (2): s, rcp from act_max and w_max (floor 1e-5 on both before the
 * powers); s = rcp = 1 when d.smooth == 0. */
int mg_smooth_scales(const mg_plan* p, const float* act_max, const float* w_max,
                     hipStream_t stream);

/* Eq. (4): O = the k channels first in the order (score desc, index asc),
 * stored ascending, and pos.  The score is act_max (MG_SCORE_MAX) or
 * RN(act_max / s) (MG_SCORE_SMOOTHED, which reads p->s: call
 * mg_smooth_scales first). */
int mg_outlier_set(const mg_plan* p, const float* act_max, hipStream_t stream);

/* Eq. (1) fold + extraction + block packing of W [N][K] (dtype MG_F32 or
 * MG_BF16) into Wq, Ws, (Wst), WO, reading p->s and p->pos. */
int mg_fold_pack(const mg_plan* p, const void* W, int32_t dtype, hipStream_t stream);

/* All three planning steps in order. */
int mg_plan_build(const mg_plan* p, const float* act_max, const float* w_max, const void* W,
                  int32_t dtype, hipStream_t stream);

/* ---- forward (per batch) ---- */

/* Runtime activation path (the integration paragraph after Eq. (5): at
 * inference a calibrated layer's input is divided in place by s, quantized to
 * 4 bits, and its outlier columns go to the narrow high-precision branch;
 * Eq. (1)'s X / s and Eq. (5)'s split into J and O):
 * q = RN_f32(X[m][j] / s_j) (exact IEEE division), XO[m][pos_j] = bf16(q),
 * bulk q with outlier columns set to +0 MXFP4-encoded into Aq/As.  M == 0 is
 * a no-op. */
int mg_quantize_act(const mg_plan* p, const void* X, int32_t dtype, int64_t M,
                    const mg_act* a, hipStream_t stream);

/* Eq. (5): Y[m][n] = sum_j Aq*Wq with their E8M0 scales + sum_i XO[m][i] WO[n][i],
 * accumulated in fp32.  y_dtype MG_BF16: Y is the layer output [M][N] bf16,
 * the fp32 sum rounded once to nearest-even.  y_dtype MG_F32: Y [M][N] f32
 * holds the fp32 sums unrounded (for callers that keep fp32 activations and
 * for checking the accumulation itself).  M == 0 is a no-op.  Each operand
 * (Aq, As, Wq, Ws, XO, WO) must stay below 3 GiB (32-bit buffer offsets),
 * else MG_ERR_UNSUPPORTED; Y has no limit (it is addressed per output tile).
 * Any K (a multiple of 32) and any k run on the same fast path. */
int mg_dual_gemm(const mg_plan* p, const mg_act* a, int64_t M, void* Y, int32_t y_dtype,
                 hipStream_t stream);

/* mg_quantize_act and mg_calib_act on the same X in one pass: the quantized
 * operands as mg_quantize_act writes them, and act_max[j] = max(act_max[j],
 * max_t |X[t][j]|) over every channel (outlier channels included) as
 * mg_calib_act computes it.  For routing that detects the outlier channels of
 * one step while it runs on the set chosen from the previous step (outlier
 * channels persist across steps; MixQ's quantization ahead of detection,
 * whose port to diffusion steps the pages name as future work).  Same
 * arguments and errors as mg_quantize_act, plus act_max [K] f32 (running;
 * reset it with mg_calib_reset). */
int mg_quantize_act_stats(const mg_plan* p, const void* X, int32_t dtype, int64_t M, const mg_act* a,
                          float* act_max, hipStream_t stream);

/* mg_quantize_act followed by mg_dual_gemm. */
int mg_forward(const mg_plan* p, const void* X, int32_t dtype, int64_t M, const mg_act* a,
               void* Y, int32_t y_dtype, hipStream_t stream);

/* mg_forward for callers that cannot allocate device memory: code under HIP
 * graph capture, tight serving loops, harnesses that forbid hipMalloc.  The
 * activation workspace (Aq, As, XO) is not passed in: it lives in a fixed
 * 64 MiB array inside the library, one copy per GPU, created when the library
 * is first used on that GPU and held until the process ends.  The call makes
 * no hipMalloc / hipFree and no allocating library call.
 * Limit: the workspace of M rows -- Aq, As, XO as mg_act_bytes gives them,
 * each rounded up to 256 bytes -- must fit in 64 MiB (K = 5120, k = 64: up to
 * about 23,500 rows), else MG_ERR_UNSUPPORTED before anything is launched.
 * Every call on one GPU shares that GPU's array, which keeps the last call's
 * contents (nothing in it has to start at zero: the quantize step writes every
 * byte the GEMM reads).  Calls ordered on one stream are safe; calls that
 * overlap on one GPU (other streams, or threads without ordering) race and
 * give wrong results.  Otherwise the arguments, errors and results are those
 * of mg_forward. */
int mg_forward_noalloc(const mg_plan* p, const void* X, int32_t dtype, int64_t M, void* Y, int32_t y_dtype,
                       hipStream_t stream);

/* Between the two projections of the FFN block (the integration paragraph:
 * the calibrated FFN linear layers take their inputs after the SiLU/GELU
 * gates): out[i] = gelu_tanh(in[i]) for n bf16 values (in == out allowed),
 * gelu_tanh(y) = 0.5 y (1 + tanh(sqrt(2/pi) (y + 0.044715 y^3))).  Evaluated in f32 as the equal y / (1 + exp(-2u))
 * (u the tanh argument) with the hardware exp2 and reciprocal, then rounded
 * to bf16: a faithful bf16 rounding (one of the two bf16 neighbours) of the
 * exact value for every finite input where that is at least 2^-24 in
 * magnitude; smaller results are at most 2^-24 (very negative y give -0). */
int mg_gelu_tanh_bf16(const uint16_t* in, uint16_t* out, int64_t n, hipStream_t stream);

/* The FFN block's second projection fed straight from the first one's bf16
 * output Y [M][K] (K = p->d.K = the first projection's N): quantizes the
 * hidden activation h = bf16_RNE(gelu_tanh(Y)) -- bit for bit what
 * mg_gelu_tanh_bf16 followed by mg_quantize_act computes -- in one pass,
 * without writing h (GELU-gated FFN inputs: the integration paragraph).
 * Same arguments and errors as mg_quantize_act with dtype MG_BF16. */
int mg_gelu_quantize_act(const mg_plan* p, const uint16_t* Y, int64_t M, const mg_act* a, hipStream_t stream);

/* The FFN block's two projections joined in the first one's GEMM epilogue
 * ("W4A4 Quantization for Inference on Wan2.2-I2V-A14B": the integration
 * paragraph -- FFN inputs after the GELU gate are quantized like every
 * linear input -- and Eq. (5) for the first projection): mg_dual_gemm of
 * plan p0 on the workspace a0 (M rows), whose bf16 output is never written;
 * instead each output tile goes through GELU-tanh and the second
 * projection's quantizer (plan p2, p2->d.K == p0->d.N) into a2.  a2 holds bit
 * for bit what mg_dual_gemm(p0, a0, M, Y, MG_BF16) followed by
 * mg_gelu_quantize_act(p2, Y, M, a2) writes, including every pad byte.
 * Device pointers as in those calls; errors: theirs, and MG_ERR_SHAPE when
 * p2->d.K != p0->d.N.  a2 must not overlap a0 or the plans. */
int mg_dual_gemm_gelu_quant(const mg_plan* p0, const mg_act* a0, int64_t M, const mg_plan* p2, const mg_act* a2,
                            hipStream_t stream);

/* ---- around the block: the norm ahead of it with its modulation, the bias
 * and activation of its projections, the gated residual after it (and the
 * norm after it).  The FFN block of the diffusion transformer the layer is
 * for runs as
 *     h = norm(x) (1 + scale) + shift;  x = x + gate * ffn(h)
 * with shift, scale and gate made from the time step, one row per sample (or
 * per token).  Sums, statistics and all arithmetic are in f32; every result
 * is rounded once, to nearest even, to the type it is stored in.  In these
 * calls X, Y, O, H are rows `ld` elements apart (ld >= their width) that only
 * need their element's alignment; finite inputs are not required: NaN and
 * infinities spread as the formulas say, within their row, except that padding
 * rows take nothing from their inputs (below).  Two limits: a norm's bias is
 * multiplied by 1 + scale before it is added, so where that product is
 * infinite the sum of two infinities can be NaN; and a norm that is not finite
 * has unspecified codes in mg_norm_quantize_act, as everywhere in the quantize
 * step. ---- */

typedef enum { MG_NORM_LAYER = 0, MG_NORM_RMS = 1 } mg_norm_kind;

/* n_j = (x_j - mean) / sqrt(var + eps) w_j + b_j with the row's mean and
 * (biased) variance (MG_NORM_LAYER), or x_j / sqrt(mean x^2 + eps) w_j + b_j
 * (MG_NORM_RMS).  weight, bias [K] of type dtype (MG_F32 or MG_BF16), either
 * may be NULL (1, 0); eps >= 0. */
typedef struct {
    const void* weight;
    const void* bias;
    int32_t dtype;
    int32_t kind;
    double eps;
} mg_norm;

/* Modulation rows: scale, shift, gate are [rows][width] matrices of type
 * dtype whose rows are ld elements apart (three column ranges of one matrix,
 * for instance); each may be NULL (0, 0, 1).  Token row r uses modulation row
 * i(r) = index[r], or r / group when index is NULL (then the M token rows
 * must not run past `rows` groups).  An index outside [0, rows) marks a
 * padding token: its norm output is 0 whatever its input holds, and a
 * residual passes it through unchanged. */
typedef struct {
    const void* scale;
    const void* shift;
    const void* gate;
    const int32_t* index;
    int64_t group;
    int64_t ld;
    int32_t rows;
    int32_t dtype;
} mg_mod;

/* H[r] = n (1 + scale_i(r)) + shift_i(r), n the norm of X[r], r < M; K <= 65536
 * channels.  mod may be NULL (H = n).  H may be X where type and ld agree;
 * M == 0 is a no-op. */
int mg_norm_mod(const mg_norm* norm, const mg_mod* mod, const void* X, int32_t dtype, int64_t ldx, int64_t M,
                int32_t K, void* H, int32_t h_dtype, int64_t ldh, hipStream_t stream);

/* The residual after a block, and the norm ahead of the next one in the same
 * pass: O[r] = X[r] + gate_i(r) p(Y[r]), p the norm `post` of the block's
 * output or nothing (post NULL); and, where norm is given, H[r] = the
 * norm-and-modulation of that sum (before it is rounded to O's type) with
 * norm and mod as in mg_norm_mod.  O has X's type; gate (its `gate` rows and
 * i(r)) and mod may be NULL.  O may be X, and H may be Y, where type and ld
 * agree. */
typedef struct {
    const void* X;
    const void* Y;
    void* O;
    void* H;              /* NULL where norm is NULL */
    int64_t ldx, ldy, ldo, ldh;
    int32_t dtype;        /* of X and O */
    int32_t y_dtype, h_dtype;
    int32_t reserved;     /* 0 */
    const mg_mod* gate;
    const mg_norm* post;
    const mg_norm* norm;
    const mg_mod* mod;
} mg_residual;
int mg_residual_norm(const mg_residual* a, int64_t M, int32_t K, hipStream_t stream);

/* mg_norm_mod into bf16 and mg_quantize_act of the result in one pass: the
 * operands of the projection behind the norm, bit for bit what those two
 * calls write (pads included) in every row whose norm is finite, without
 * writing the normalized rows.
 * K = p->d.K. */
int mg_norm_quantize_act(const mg_plan* p, const mg_norm* norm, const mg_mod* mod, const void* X, int32_t dtype,
                         int64_t ldx, int64_t M, const mg_act* a, hipStream_t stream);

typedef enum { MG_ACT_NONE = 0, MG_ACT_GELU_TANH = 1, MG_ACT_SILU = 2 } mg_act_fn;

/* Epilogue of the dual GEMM on its fp32 sums v[m][n]:
 *     v += bias[n];  v = act(v);  Y = residual[m][n] + gate_i(m)[n] v
 * with bias [N] of bias_dtype or NULL, mod's gate rows and i(m) as above (mod
 * NULL: gate 1; only its gate is used), residual rows ldr elements apart of
 * residual_dtype, or NULL (0).  A padding row gets Y = residual (0 without
 * one).  GELU-tanh and SiLU are evaluated in f32 with the hardware exp2 and
 * reciprocal.  Bases must be 16-byte aligned, ld of the residual and of the
 * gate rows a multiple of 8 elements, else MG_ERR_ALIGN.  Y may be the
 * residual (same type, ldr == N). */
typedef struct {
    const void* bias;
    const void* residual;
    const mg_mod* mod;
    int64_t ldr;
    int32_t bias_dtype;
    int32_t residual_dtype;
    int32_t act;          /* mg_act_fn */
    int32_t reserved;     /* 0 */
} mg_epilogue;

/* mg_dual_gemm with the epilogue above; e may be NULL.  The order of the fp32
 * sums may differ from mg_dual_gemm's (few rows take a kernel of their own
 * that splits K), but is fixed: the same call gives the same bits. */
int mg_dual_gemm_ep(const mg_plan* p, const mg_act* a, int64_t M, const mg_epilogue* e, void* Y, int32_t y_dtype,
                    hipStream_t stream);

/* mg_quantize_act followed by mg_dual_gemm_ep. */
int mg_forward_ep(const mg_plan* p, const void* X, int32_t dtype, int64_t M, const mg_act* a, const mg_epilogue* e,
                  void* Y, int32_t y_dtype, hipStream_t stream);

/* ---- 8-bit block-scaled layers: for projections that 4 bits cost too much,
 * and for training.  The backward passes are those of the plain products and of
 * the gated block: an epilogue (bias, activation, gate, residual) has none, nor
 * have the 4-bit layers.
 *
 * An 8-bit matrix holds [rows][cols] values as OCP FP8 codes (E4M3, largest
 * magnitude 448, or E5M2, 57344) and one E8M0 scale 2^(c - 127) for each row's
 * 128 consecutive columns.  A value v is stored as the code nearest to
 * v / 2^(c - 127), ties to even, with the smallest c >= 1 under which the
 * block's largest magnitude does not exceed the format's: nothing saturates,
 * and the scale costs no precision.  A weight has one c for each tile of
 * 128 x 128 (repeated on the tile's rows), so its transpose holds the same
 * codes.  A block (a weight: a tile) that holds a NaN or an infinity is NaN throughout,
 * and so is everything computed from it.  Magnitudes from 2^128 (1 - 2^-5) on (E5M2: 1 -
 * 2^-4) are finite in f32 but round to 2^128, which is not: they come back as
 * infinities, and count as such in a transpose.
 *
 * cols is a multiple of 32, rows any number; q and s are device buffers of
 * mg_f8_bytes bytes, s [..] u32:
 *  q  fragment order: blocks of 32 rows x 32 columns, 1024 contiguous bytes
 *     each, block (g = r / 32, c = col / 32) at (g * ns + c) * 1024 with ns =
 *     4 * ceil(cols / 128); inside it the code of (r, col) is at byte
 *         16 * (r % 32 + 32 * ((col / 4) % 2)) + 4 * ((col % 32) / 8) + col % 4.
 *     Two blocks are one operand of the 32x32x64 matrix-core instruction, and
 *     a block's 16-byte pieces are the output columns that one lane of that
 *     instruction holds: a product's epilogue writes the next one's operand.
 *     Columns up to the next multiple of 128 hold 0; rows up to the next
 *     multiple of 32 are unspecified.
 *  s  the code c of (r, col) is byte (col / 128) % 4 of word
 *         ((r / 256) * ceil(cols / 512) + col / 512) * 256 + r % 256;
 *     bytes of columns and rows past the matrix are unspecified.
 * Both depend on cols and not on rows (a buffer sized for more rows serves
 * fewer).
 * What a call writes, workspaces too, overlaps neither its other outputs nor its
 * inputs (an epilogue's residual may be Y itself). ---- */

typedef enum { MG_E4M3 = 0, MG_E5M2 = 1 } mg_f8_format;

typedef struct {
    uint8_t* q;
    uint32_t* s;
    int64_t rows;
    int32_t cols;
    int32_t format;       /* mg_f8_format */
} mg_f8;

/* Host-only size query: out[2] = bytes of q and s. */
int mg_f8_bytes(int64_t rows, int32_t cols, size_t out[2]);

/* x := X [x.rows][x.cols] (MG_F32 or MG_BF16, rows ldx elements apart, aligned to
 * their elements).  rows == 0 is a no-op here and below.  This is also an
 * activation's checkpoint: 1 1/128 bytes an element instead of 2 or 4. */
int mg_f8_quantize(const void* X, int32_t dtype, int64_t ldx, const mg_f8* x, hipStream_t stream);

/* X := the values that x holds (exact in f32; in bf16 exact as well, but for
 * values below its normal range). */
int mg_f8_dequantize(const mg_f8* x, void* X, int32_t dtype, int64_t ldx, hipStream_t stream);

/* xt [x.cols][x.rows rounded up to 32] := x transposed, with scales along x's rows: each
 * column's 128 consecutive rows share one, chosen by the rule above, and the
 * values are rounded again where they fall below the format's normal range
 * under it (2^-14 of the block's largest in E4M3, 2^-30 in E5M2).  The operands
 * of a product over tokens.  Columns of xt past x's rows hold 0.  Same format. */
int mg_f8_transpose(const mg_f8* x, const mg_f8* xt, hipStream_t stream);

/* What a backward pass starts with, in one launch: dy := dY [M][N] as
 * mg_f8_quantize makes it, and the transposes as mg_f8_transpose makes them: dyt of dy,
 * at of a and bt of b, two E4M3 matrices of M rows that the forward pass kept (each
 * pair may be NULL, and dyt). */
int mg_f8_prepare_back(const void* dY, int32_t dtype, int64_t ldy, const mg_f8* dy, const mg_f8* dyt, const mg_f8* a,
                       const mg_f8* at, const mg_f8* b, const mg_f8* bt, hipStream_t stream);

/* w [N][K] := W [N][K] with a scale for each 128 x 128 tile, and wt [K][N] its
 * transpose where not NULL.  E4M3; K and N multiples of 32. */
int mg_f8_pack_w(const void* W, int32_t dtype, int64_t ldw, const mg_f8* w, const mg_f8* wt, hipStream_t stream);

/* Y[m][n] = ep(sum_j a[m][j] w[n][j]), accumulated in fp32, a [M][K], w [N][K],
 * K and N multiples of 32, w E4M3; Y [M][N] MG_BF16 or MG_F32, e the epilogue
 * of mg_dual_gemm_ep or NULL (an activation with an E4M3 a only).  MG_BF16
 * results come from the 8-bit matrix instructions, which add eight products at
 * a time, each cut off at 2^-13 of the largest, to an fp32 sum: they are 1.5e-5
 * (normal values) to 5e-5 (a few channels 25 times the others) of their norm
 * away from the exact products, a hundredth of bf16's own rounding.  MG_F32
 * results keep fp32's precision: the codes are widened and multiplied by the
 * bf16 instructions, at half the rate.  Each operand must stay below 3 GiB, and
 * N and the residual's row distance at most 2^20 - 256.  The order of the sums
 * depends on the sizes alone. */
int mg_f8_gemm(const mg_f8* a, const mg_f8* w, const mg_epilogue* e, void* Y, int32_t y_dtype, hipStream_t stream);

/* mg_f8_quantize of X into act (E4M3), then mg_f8_gemm of it.  save 1 leaves
 * X's codes in act, for the backward pass; with save 0 act is workspace, and a
 * few rows (at most 16 and 28 K values, fewer where N is large) are quantized
 * inside the product, in one launch: the same codes, sums in another order. */
int mg_f8_forward(const void* X, int32_t dtype, int64_t ldx, const mg_f8* act, int32_t save, const mg_f8* w,
                  const mg_epilogue* e, void* Y, int32_t y_dtype, hipStream_t stream);

/* ---- the gated feed-forward block
 *     h = act(x Wg^T) * (x Wu^T),  y = h Wd^T,
 * x [M][K], Wg, Wu [F][K], Wd [N][F].  Gate and up projection are one product
 * with the weight w13 [2 Fp][K], Fp = F rounded up to a multiple of 128: runs
 * of 128 gate rows and 128 up rows in turn, rows past F zero.  Its output
 * columns come in the same order: gu [M][2 Fp] holds the sums g = x Wg^T and
 * u = x Wu^T, dgu their gradients.  y = mg_f8_gemm(h, wd). ---- */

/* w13 := Wg and Wu [F][K] (K = w13.cols; w13.rows = 2 Fp), w13t [K][2 Fp] its
 * transpose where not NULL. */
int mg_gated_pack_w(const void* Wg, const void* Wu, int32_t dtype, int64_t ldw, int32_t F, const mg_f8* w13,
                    const mg_f8* w13t, hipStream_t stream);

/* Bytes of scratch (16-byte aligned device memory, free after the call's
 * kernels) of mg_gated_gemm (with or without gu) or mg_gated_forward, and of
 * mg_gated_gemm_back, with M rows, hidden width F and a product over C columns;
 * 0 where the call needs none. */
int mg_gated_scratch_bytes(int64_t M, int32_t F, int32_t C, size_t out[2]);

/* h [M][F] (E4M3) := the 8-bit codes of act(g) u, formed from the fp32 sums; gu
 * [M][2 Fp] (E4M3) := the codes of g and u, for the backward pass, where not
 * NULL.  With gu the sums keep fp32's precision, whatever M; without it they come
 * from the 8-bit matrix instructions where M is large, and five codes of h in a
 * thousand lie a step beside the nearest, where the value is all but halfway
 * between the two: h is as far from its value as otherwise (2.65e-2 of the norm). */
int mg_gated_gemm(const mg_f8* x, const mg_f8* w13, int32_t act, const mg_f8* h, const mg_f8* gu, void* scratch,
                  hipStream_t stream);

/* The whole block: X [M][K] quantized into x, mg_gated_gemm, and y = ep(h Wd^T)
 * as mg_f8_gemm makes it.  With gu, x, gu and h hold what the backward pass needs;
 * without it they are workspace, and a few rows take two launches. */
int mg_gated_forward(const void* X, int32_t dtype, int64_t ldx, const mg_f8* x, const mg_f8* w13, int32_t act,
                     const mg_f8* h, const mg_f8* gu, void* scratch, const mg_f8* wd, const mg_epilogue* e, void* Y,
                     int32_t y_dtype, hipStream_t stream);

/* dgu [M][2 Fp] (dy's format) := the codes of dh u act'(g) and dh act(g), with dh = dy Wd in
 * fp32 (dy [M][N], wdt [F][N] the transpose of wd) and g, u the values of gu;
 * dgut [2 Fp][M rounded up to 32] := the transpose of dgu, as mg_f8_transpose makes it,
 * where not NULL. */
int mg_gated_gemm_back(const mg_f8* dy, const mg_f8* wdt, const mg_f8* gu, int32_t act, const mg_f8* dgu,
                       const mg_f8* dgut, void* scratch, hipStream_t stream);

/* dWg, dWu [F][K] (y_dtype) := the gradients of the two weights, from dgut [2
 * Fp][M] and xt [K][M] (the transposes of dgu and x). */
int mg_gated_gemm_dw(const mg_f8* dgut, const mg_f8* xt, int32_t F, void* dWg, void* dWu, int32_t y_dtype,
                     hipStream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* MIXED_GEMM_H */
