/*
 * ttq.h -- C ABI of the TTQ linear projection on AMD Instinct MI355X (gfx950).
 *
 * TTQ (activation-aware test-time quantization, arXiv:2603.19296) quantizes
 * the weights of a linear layer on the fly from the activations of the
 * current call, with no calibration data and no state kept between calls.
 * For activations X (d input channels x T tokens) and weights W (d' x d)
 * one call computes
 *
 *   n_i      = ||X_{i,:}||_p                        L_p norm of channel i
 *   D_ii     = (n_i + lambda)^alpha                 damped diagonal
 *   W_hat    = Q[W D^{1/2}] D^{-1/2}                group quantize-dequantize
 *   Y        = W_hat X + B (A X)                    plus the static low rank
 *
 * as defined in "TTQ: Activation-Aware Test-Time Quantization to Accelerate
 * LLM Inference On The Fly" (gist.science zh summary, Sec. 2.1 for D and
 * W_hat, Sec. 2.2 for the low-rank term; the nl and it summaries, Sec. 2,
 * restate both).  Q is the asymmetric b-bit affine quantizer of the blog
 * "Test-time quantization: quantising on the fly with no calibration
 * dataset", section "The maths that matter", applied to groups of `group`
 * consecutive input channels of each output row, with a min-anchored real
 * zero point: s = (max - min)/(2^b - 1), q = clamp(rint((u - min)/s)),
 * u_hat = min + s q.  Codes are decided in IEEE float32:
 *   dh = float32(D^{1/2}); u = w*dh; s = (max-min)/N; inv = 1/s (0 if s=0);
 *   t = (u - min)*inv; q = clamp(rint_half_even(t), 0, N)
 * with every operation correctly rounded and no fused multiply-add.  The
 * statistics (norms and powers) are evaluated in float64.
 *
 * Memory layout (all row-major, bfloat16 = raw 16-bit patterns):
 *   W  [d_out][d]      bf16    (nn.Linear weight layout)
 *   X  [T][d]          bf16    (token-major; batched: [R][T][d])
 *   B  [d_out][rank]   bf16    A [rank][d] bf16   (both NULL if rank == 0)
 *   Y  [T][d_out]      float32 (batched: [R][T][d_out])
 *
 * Ownership and ordering: every pointer is caller-owned device memory (or
 * NULL where optional).  The library never allocates, frees or synchronizes
 * on the calling path: it validates arguments on the host, enqueues kernels
 * on `stream` (a hipStream_t; NULL is the null stream) and returns.  Device
 * faults surface at the caller's next synchronization.  Results are
 * deterministic: identical inputs give bit-identical outputs.
 *
 * Accuracy of Y: the contraction accumulates in float32.  Its activation
 * operand x' = x D^{-1/2} is float32 for one token, fp16 scaled by a power
 * of two per (group, token) for 2..16 tokens (any float32 magnitude), and
 * bf16 above; above 128 tokens the dequantized weights are rounded once to
 * bf16 and contracted with the bf16 X.
 *
 * Errors: validation happens before anything is enqueued, so a negative
 * status means nothing was launched -- except TTQ_EHIP, which reports a
 * failed launch (some earlier kernels of the same call may have been
 * enqueued); the raw hipError_t is then available from ttq_last_hip_error().
 */
#ifndef TTQ_H_
#define TTQ_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Status codes. */
enum {
  TTQ_OK = 0,
  TTQ_EINVAL = -1,       /* a size or scalar argument is out of range          */
  TTQ_ENULL = -2,        /* a required pointer is NULL                          */
  TTQ_EALIGN = -3,       /* a pointer is not aligned as required                */
  TTQ_EWORKSPACE = -4,   /* workspace smaller than ttq_workspace_bytes()        */
  TTQ_EUNSUPPORTED = -5, /* valid by the method, not supported by this library  */
  TTQ_EHIP = -100        /* a HIP runtime call failed; see ttq_last_hip_error() */
};

/* flags */
#define TTQ_FLAG_FORCE_FUSED 1u    /* use the single-pass fused path (T <= 128) */
#define TTQ_FLAG_FORCE_TWO_PHASE 2u /* quantize pass + GEMM, at any T            */

/* Quantizer formats (ttq_params.qformat).  The method derives the scale from
 * the activations and leaves the code format open (lo0 blog "Test-time
 * quantization: quantising on the fly with no calibration dataset", section
 * "What TTQ is NOT": orthogonal to INT4 or FP8; section "The maths that
 * matter" for the symmetric scale and the affine form with a zero point).
 * For one group of u = w D^{1/2} (float32, no fused operations, inv = 1/s or
 * 0 when s = 0, rint = round half to even):
 *   TTQ_QF_ASYM   s = (max - min)/N, q = clamp(rint((u - min) inv), 0, N),
 *                 u_hat = min + s q                 (N = 2^b - 1; default)
 *   TTQ_QF_SYM    s = max|u| / Z (Z = 2^{b-1} - 1, b >= 2),
 *                 k = clamp(rint(u inv), -Z, Z), u_hat = s k, code q = k + Z
 *   TTQ_QF_INTZP  lo = min(min u, 0), hi = max(max u, 0), s = (hi - lo)/N,
 *                 z = rint(lo inv), q = clamp(rint(u inv) - z, 0, N),
 *                 u_hat = s (q + z)   (integer zero point; zero is exact)
 *   TTQ_QF_FP8    b = 8: s = max|u| / 448, code = the OCP FP8 E4M3 pattern
 *                 of the nearest E4M3 value v (ties to even) of
 *                 clamp(u inv, -448, 448), u_hat = s v (the sign bit is
 *                 that of u inv, also when v is zero)
 * The per-group term stored beside the scales (mins_out, and the `mins` of
 * ttq_quantize / ttq_qmatmul) is the offset m with u_hat = m + s q for the
 * integer formats: the minimum (ASYM), -(Z s) (SYM), z s (INTZP), each
 * rounded once to float32; it is 0 for FP8, whose codes decode to E4M3
 * values.  Codes are decided exactly as stated; Y uses these stored terms. */
#define TTQ_QF_ASYM 0u
#define TTQ_QF_SYM 1u
#define TTQ_QF_INTZP 2u
#define TTQ_QF_FP8 3u

/* One projection's shape and the method's constants.
 *   d      input channels; >= 1 and a multiple of `group`
 *   d_out  output channels; >= 0
 *   T      tokens per request; >= 0 (T = 0: Y is empty, codes/scales are
 *          still produced from zero statistics)
 *   rank   low-rank r; 0 = no low-rank term; otherwise a multiple of 8, <= 1024
 *   bits   code width b in 1..8 (2..8 for TTQ_QF_SYM, 8 for TTQ_QF_FP8)
 *   group  group size along d: 32, 64, 128 or 256
 *   p      norm order, finite and > 0 (1 and 2 are exact; others use pow)
 *   lambda damping, finite and >= 0
 *   alpha  exponent, finite and >= 0 (0 gives D = I, i.e. plain RTN)
 *   flags  0, or one TTQ_FLAG_* path override
 *   qformat one of TTQ_QF_* (0 = the asymmetric quantizer)                   */
typedef struct ttq_params {
  int64_t d;
  int64_t d_out;
  int64_t T;
  int64_t rank;
  int32_t bits;
  int32_t group;
  double p;
  double lambda;
  double alpha;
  uint32_t flags;
  uint32_t qformat;
} ttq_params;

/* Device workspace, in bytes, that ttq_linear (n_requests = 1) or
 * ttq_linear_batched needs for these parameters.  Writes *bytes; returns a
 * status (the same validation as the compute calls, minus pointers). */
int ttq_workspace_bytes(const ttq_params* prm, int64_t n_requests,
                        size_t* bytes);

/* One TTQ linear call (one request).
 *   W, X             required (X may be NULL when T == 0); 16-byte aligned
 *   B, A             required iff rank > 0; 16-byte aligned
 *   Y                [T][d_out] float32; required iff T*d_out > 0; 4-byte aligned
 *   codes_out        optional [d_out][d] uint8 codes q
 *   scales_out       optional [d_out][d/group] float32 scales s
 *   mins_out         optional [d_out][d/group] float32 group offsets m (the
 *                    minima for TTQ_QF_ASYM; see TTQ_QF_*)
 *   dhalf_out        optional [d] float32 D^{1/2} as fed to the code decision
 *   workspace        device scratch of at least ttq_workspace_bytes(prm, 1);
 *                    256-byte aligned; contents need not be initialized and
 *                    are clobbered; must not be shared by concurrent calls
 *   stream           hipStream_t to enqueue on
 * Returns TTQ_OK or a negative status. */
int ttq_linear(const ttq_params* prm, const void* W, const void* X,
               const void* B, const void* A, float* Y, uint8_t* codes_out,
               float* scales_out, float* mins_out, float* dhalf_out,
               void* workspace, size_t workspace_bytes, void* stream);

/* R independent requests on one shared W (and B, A): each request has its
 * own statistics D computed from its own X (multitenant traffic).  X is
 * [R][T][d], Y [R][T][d_out]; the optional outputs gain a leading [R]
 * dimension.  n_requests = 0 is a valid no-op. */
int ttq_linear_batched(const ttq_params* prm, int64_t n_requests,
                       const void* W, const void* X, const void* B,
                       const void* A, float* Y, uint8_t* codes_out,
                       float* scales_out, float* mins_out, float* dhalf_out,
                       void* workspace, size_t workspace_bytes, void* stream);

/* ---- allocation-free variant ----------------------------------------------
 * For callers that cannot allocate device memory: code under HIP graph
 * capture, tight serving loops, harnesses that forbid hipMalloc.  Same
 * arguments and results as ttq_linear_batched (n_requests = 1 is ttq_linear),
 * minus the workspace: the library takes it from a static device array of
 * TTQ_NOALLOC_SCRATCH_BYTES that every GPU it runs on holds until the process
 * ends (its address is looked up on the first call on each device, with that
 * device current).  The call allocates nothing, frees nothing and calls no
 * allocating routine.  All calls on one GPU share that GPU's array, which
 * keeps the last call's contents (no kernel needs it cleared): calls that
 * overlap on one GPU -- concurrent streams or threads -- race and must be
 * serialised by the caller.
 * Errors: as ttq_linear_batched, plus TTQ_EWORKSPACE when the call needs more
 * scratch than TTQ_NOALLOC_SCRATCH_BYTES (ttq_workspace_bytes gives the need;
 * checked on the host, nothing is enqueued), and TTQ_EHIP when the array's
 * address cannot be obtained. */
#define TTQ_NOALLOC_SCRATCH_BYTES ((size_t)64 << 20)
int ttq_linear_noalloc(const ttq_params* prm, int64_t n_requests,
                       const void* W, const void* X, const void* B,
                       const void* A, float* Y, uint8_t* codes_out,
                       float* scales_out, float* mins_out, float* dhalf_out,
                       void* stream);

/* ---- continuous batching: requests of different lengths in one X --------
 * n_segments requests packed one after another: request i owns the token
 * rows seg_offsets[i] .. seg_offsets[i+1]-1 of X [T][d] and Y [T][d_out],
 * where prm->T is the total token count.  The pages leave open how scales
 * are derived when one batch mixes requests ("Test-time quantization:
 * quantising on the fly with no calibration dataset", lo0 blog, section "What
 * we have not covered"); here every request keeps its own statistics D, as
 * in ttq_linear_batched, and its codes, scales and Y rows equal those of
 * ttq_linear on that request alone, bit for bit (with a low-rank term, up to
 * 64 MiB of low-rank partial sums per batch).
 *   seg_offsets  host array of n_segments + 1 non-decreasing token offsets,
 *                seg_offsets[0] = 0, seg_offsets[n_segments] = prm->T;
 *                empty requests (equal offsets) are allowed
 *   optional outputs gain a leading [n_segments] dimension, as in
 *   ttq_linear_batched; all other arguments as for ttq_linear.
 * The requests of one length class (1; 2..16; 17..32; 33..64; 65..128
 * tokens; up to 64 at a time) are computed as one batch, shorter ones padded
 * with zero tokens (which leave the norms unchanged) through workspace copies
 * unless the batch is a run of consecutive requests of one length; when codes,
 * scales or D^{1/2} are asked for, a batch takes only consecutive requests.
 * Longer requests, or any request when a path flag is set, run alone.
 * n_segments = 0 is a no-op.
 * Errors: TTQ_ENULL for a NULL seg_offsets (n_segments > 0); TTQ_EINVAL for
 * offsets that do not start at 0, end at prm->T or decrease, and for the
 * conditions of ttq_linear_batched. */
int ttq_segmented_workspace_bytes(const ttq_params* prm, int64_t n_segments,
                                  const int64_t* seg_offsets, size_t* bytes);
int ttq_linear_segmented(const ttq_params* prm, int64_t n_segments,
                         const int64_t* seg_offsets, const void* W,
                         const void* X, const void* B, const void* A, float* Y,
                         uint8_t* codes_out, float* scales_out, float* mins_out,
                         float* dhalf_out, void* workspace,
                         size_t workspace_bytes, void* stream);

/* Which path a call with these parameters takes: 0 = fused single pass over
 * W (statistics kernel + one fused quantize/MFMA kernel), 1 = two phase
 * (statistics, quantize pass writing W_hat, MFMA GEMM), 2 = single launch
 * for one token (T = 1, d <= 12288, no path flag), 3 = two phase with the
 * weight tiles quantized inside the MFMA GEMM (129 <= T <= 256, d a
 * multiple of 128, group <= 128, no path flag; a call that asks for codes or
 * scales adds a pass over W that writes only them).  Paths 1 and 3 give
 * bit-identical Y.
 * Negative = status. */
int ttq_path(const ttq_params* prm, int64_t n_requests);

/* ---- quantize once per prompt, decode from the stored codes -------------
 * The statistics can be taken once per input prompt ("TTQ: Activation-Aware
 * Test-Time Quantization ...", nl summary, Sec. 2; zh summary, Sec. 3-4:
 * the speed-up comes from contracting stored low-bit weights, because
 * moving weights is the bottleneck).  ttq_quantize computes D from the
 * prompt's X and stores the codes, the per-group (s, min) and D^{-1/2};
 * ttq_qmatmul then computes, for the activations X of a later step,
 *   Y = X ((min + s q) D^{-1/2})^T + (X A^T) B^T
 * with those stored values (nothing is recomputed from the step's X).
 *
 * Code storage: each b-bit code takes the smallest container c of 1, 2, 4
 * or 8 bits that holds it; channel j of a row sits at bit (j*c) % 8 of byte
 * (j*c) / 8 of that row (least significant bits first).  A row takes
 * ttq_packed_row_bytes = d*c/8 bytes; d*c must be a multiple of 128 bits
 * (always true for the supported group sizes when c >= 4; checked). */

/* Bytes of one row of packed codes for these parameters (writes *bytes). */
int ttq_packed_row_bytes(const ttq_params* prm, int64_t* bytes);

/* Device workspace for ttq_quantize / ttq_qmatmul (writes *bytes). */
int ttq_quantize_workspace_bytes(const ttq_params* prm, size_t* bytes);
int ttq_qmatmul_workspace_bytes(const ttq_params* prm, size_t* bytes);

/* Quantize W for the prompt X ([T][d] bf16, T = prm->T >= 0; T = 0 gives
 * D from zero statistics, as in ttq_linear).
 *   codes       [d_out][row_bytes] packed codes, 16-byte aligned, required
 *   scales      [d_out][d/group] float32 s, required
 *   mins        [d_out][d/group] float32 group offsets m (minima for
 *               TTQ_QF_ASYM; see TTQ_QF_*), required
 *   dhalf_inv   [d] float32 D^{-1/2} = float32(1 / D^{1/2}), required
 *   dhalf_out   optional [d] float32 D^{1/2} as fed to the code decision
 * rank and the path flags are not read (the low-rank factors are used as
 * given by ttq_qmatmul); unknown flag bits are still TTQ_EINVAL.  Same
 * validation, alignment and error rules as ttq_linear otherwise. */
int ttq_quantize(const ttq_params* prm, const void* W, const void* X,
                 uint8_t* codes, float* scales, float* mins, float* dhalf_inv,
                 float* dhalf_out, void* workspace, size_t workspace_bytes,
                 void* stream);

/* Y [T][d_out] float32 for the step activations X ([T][d] bf16, T =
 * prm->T) from the stored codes, scales, mins and dhalf_inv of ttq_quantize
 * (same d, d_out, bits, group and qformat: TTQ_QF_FP8 codes decode as E4M3
 * values, every other format as integers with the stored offsets, u_hat =
 * mins + scales * code).  B, A as in ttq_linear (rank = prm->rank).
 * codes 16-byte aligned, dhalf_inv 16-byte aligned, the rest as in
 * ttq_linear.  p, lambda, alpha and TTQ_FLAG_FORCE_FUSED are not used;
 * Routes: T = 1, a single kernel over the codes (unless x D^{-1/2} of the
 * token does not fit 128 KiB of LDS: d above about 30000); T <= 128, the
 * codes on the matrix cores; otherwise a GEMM that expands the codes to
 * bf16 weights tile by tile in LDS (d a multiple of 128), else a pass that
 * writes the expanded weights followed by a GEMM.  TTQ_FLAG_FORCE_TWO_PHASE
 * takes that last route at any T; both expansions give the same Y bits. */
int ttq_qmatmul(const ttq_params* prm, const uint8_t* codes,
                const float* scales, const float* mins, const float* dhalf_inv,
                const void* X, const void* B, const void* A, float* Y,
                void* workspace, size_t workspace_bytes, void* stream);

/* ---- low-rank adapters of many requests ----------------------------------
 * Beside a shared projection, whose low-rank term B (A X) is one for all rows,
 * each row of a batch may add a pair of its own, held in a set of n_adapters:
 *   Y[t] = base[t] + scale[e] B_e (A_e x_t),   e = index[t].
 * Of prm only d, d_out, T and rank are read: rank is that of every pair
 * (smaller ones padded with zeros), a multiple of 8 up to 128; d is a multiple
 * of 8 (TTQ_EUNSUPPORTED otherwise).
 *   X      [T][d] bf16           A   [n_adapters][rank][d] bf16
 *   B      [n_adapters][d_out][rank] bf16
 *   scale  optional [n_adapters] float32 (1 without)
 *   index  [T] int32 on the device; a row whose index lies outside
 *          [0, n_adapters) has no pair: Y[t] = base[t]
 *   base   optional [T][d_out] float32, e.g. what ttq_linear or ttq_qmatmul
 *          gave (0 without); may be Y itself, but not otherwise overlap it
 *   Y      [T][d_out] float32
 *   workspace of at least ttq_adapters_workspace_bytes (0 for small steps)
 * Up to 128 rows (decode steps) may name as many pairs as they are; more are
 * taken as prompts, with runs of rows of one pair.  Any order is right, but more
 * than 128 rows of mixed pairs are several times faster in calls of 128 rows
 * each (256 rows with 100 pairs: 72 us in two calls, 473 us in one).
 * Both products accumulate in float32 and A_e x_t enters the second one with
 * all its 24 bits, as a sum of three parts.  An infinity in A_e x_t keeps its
 * sign in the outputs; one in B_e makes its own output infinite or NaN (a part
 * that is 0 times it).  n_adapters = 0 copies base.  X, A and B are 16-byte
 * aligned, the rest as for ttq_linear; the same error rules. */
int ttq_adapters_workspace_bytes(const ttq_params* prm, int64_t n_adapters,
                                 size_t* bytes);
int ttq_adapters(const ttq_params* prm, int64_t n_adapters, const void* X,
                 const void* A, const void* B, const float* scale,
                 const int32_t* index, const float* base, float* Y,
                 void* workspace, size_t workspace_bytes, void* stream);

/* ---- a mixture-of-experts layer from stored codes ------------------------
 * The decode step of a layer whose MLP is `experts` gated MLPs, each kept as
 * ttq_quantize leaves its weights, for a few tokens (T <= 128):
 *   l_e = router[e] . x_t               scores, summed in float64
 *   chosen: the top_k largest scores, equal ones by the lower index, NaN last
 *   w_j = exp(l_j - max) / sum of it over the chosen experts
 *         (TTQ_MOE_RENORMALIZE) or over all of them (without)
 *   h   = silu(gate) * up,  gate and up rows of (m + s q) D^{-1/2} times x_t
 *   Y[t] = sum_j w_j (down rows of expert j times h)
 *   T, d, ff       tokens, channels of the layer, width of an expert; d and ff
 *                  multiples of group (and rows of whole 16 bytes of codes)
 *   experts, top_k up to 256 and 16; top_k <= experts
 *   bits, group, qformat   of all stored codes, as for ttq_quantize
 *   X        [T][d] bf16; router [experts][d] bf16
 *   gu_*     gate rows, then up rows: codes [experts][2 ff][row_bytes(d)],
 *            scales, mins [experts][2 ff][d/group], dhalf_inv [experts][d]
 *   dn_*     codes [experts][d][row_bytes(ff)], scales, mins
 *            [experts][d][ff/group], dhalf_inv [experts][ff]
 *   Y        [T][d] float32
 *   ids_out, weights_out   optional [T][top_k] int32 / float32, best first
 *   workspace of at least ttq_moe_workspace_bytes
 * The contractions accumulate in float32, with x D^{-1/2} and h D^{-1/2} in
 * all their 24 bits.  A token whose x D^{-1/2}, or whose h D^{-1/2} for one of
 * its experts, holds an infinity or a NaN (h overflows float32 at 3.4e38) has a
 * row of NaN; the other rows are as they would be without it.
 * Larger T, experts or top_k are TTQ_EUNSUPPORTED.  X,
 * router, codes, dhalf_inv and Y are 16-byte aligned, the rest their type's;
 * the error rules of ttq_linear. */
#define TTQ_MOE_RENORMALIZE 1u
typedef struct ttq_moe_params {
  int64_t T;
  int64_t d;
  int64_t ff;
  int32_t experts;
  int32_t top_k;
  int32_t bits;
  int32_t group;
  uint32_t flags;
  uint32_t qformat;
} ttq_moe_params;
int ttq_moe_workspace_bytes(const ttq_moe_params* prm, size_t* bytes);
int ttq_moe(const ttq_moe_params* prm, const void* X, const void* router,
            const uint8_t* gu_codes, const float* gu_scales,
            const float* gu_mins, const float* gu_dhalf_inv,
            const uint8_t* dn_codes, const float* dn_scales,
            const float* dn_mins, const float* dn_dhalf_inv, float* Y,
            int32_t* ids_out, float* weights_out, void* workspace,
            size_t workspace_bytes, void* stream);

/* ---- a cache quantized as it is written ----------------------------------
 * The quantizer of ttq_quantize applied to rows as they are produced, such as
 * the K and V rows of a decoder ("Test-time quantization: quantising on the
 * fly with no calibration dataset", lo0 blog: KV-cache scales derived on the
 * fly by the same logic).  A cache has n_slots rows of d channels (all heads
 * of a token, K and V side by side or in two caches), each laid out as a weight
 * row of ttq_quantize is: `bits` wide codes packed in ttq_packed_row_bytes,
 * and float32 scales and mins per group:
 *   codes [n_slots][row_bytes], scales, mins [n_slots][d/group].
 * Formats and the float32 code decision are those of TTQ_QF_*, except that a
 * scale is the group's range times the float32 nearest to 1/N (1/Z for
 * TTQ_QF_SYM, 1/448 for TTQ_QF_FP8) instead of the range divided by it.  So a
 * row's bits are not those that ttq_quantize gives it: scales are up to three
 * half units in the last place apart, and a value half way between two levels
 * may get the other one (0.01 to 0.14 % of the levels of normal bfloat16 rows,
 * which are often half way, next to none with dhalf); either is within half a
 * step of it.
 * With dhalf, the D^{1/2} of each channel (e.g. dhalf_out of ttq_quantize for
 * the prompt's queries), the codes are those of x D^{1/2}; reading with
 * dhalf_inv = 1 / dhalf undoes it.
 * Of prm only d, T, bits, group and qformat are read.
 *
 * ttq_cache_write quantizes T rows: row t of X goes to cache row slots[t].
 *   x_type   TTQ_BF16 or TTQ_F32
 *   X        [T] rows of d values, ldx >= d elements apart (a column range of
 *            a wider matrix is fine); 16-byte aligned, as is every row
 *   dhalf    optional [d] float32
 *   slots    [T] int64 on the device; a row whose slot lies outside
 *            [0, n_slots) is not written (padding: -1).  The other slots of a
 *            call must be distinct: of a slot named twice the stored row may
 *            be a mixture of both.
 * A group that holds an infinity or a NaN, or whose range is no finite
 * float32, reads back as NaN; a scale below 2^-126 counts as 0.
 *
 * ttq_cache_read gives rows 0 .. lens[i] - 1 of n_seq sequences as out[i][t],
 * out being [n_seq][T][d] of out_type (TTQ_BF16: rounded once).  Cache rows
 * are grouped in pages of page_tokens (a power of two up to 4096); row t of
 * sequence i is cache row pages[i][t / page_tokens] * page_tokens
 * + t % page_tokens.  pages [n_seq][max_pages] and lens [n_seq] are int32 on
 * the device.  A length past T or past the pages is cut to them, a negative
 * one is 0.  Rows behind a sequence's length, and rows whose page lies outside
 * the cache, are left as they were.
 *   dhalf_inv  optional [d] float32; out 16-byte aligned
 * Neither call needs a workspace.  Alignment: X, dhalf, dhalf_inv, codes and
 * out 16 bytes, the rest their type's.  Error rules as for ttq_linear
 * (TTQ_EALIGN also for an ldx that breaks the row alignment). */
#define TTQ_BF16 0
#define TTQ_F32 1
int ttq_cache_write(const ttq_params* prm, int64_t n_slots, int32_t x_type,
                    const void* X, int64_t ldx, const float* dhalf,
                    const int64_t* slots, uint8_t* codes, float* scales,
                    float* mins, void* stream);
int ttq_cache_read(const ttq_params* prm, int64_t n_slots, int64_t n_seq,
                   int64_t max_pages, int32_t page_tokens, const int32_t* pages,
                   const int32_t* lens, const uint8_t* codes,
                   const float* scales, const float* mins,
                   const float* dhalf_inv, int32_t out_type, void* out,
                   void* stream);

/* ---- attention over such a cache -----------------------------------------
 * The rest of what a decoder does with its cache in a step: where the step's
 * rows go (ttq_cache_extend), its heads' norms and rotation with K and V
 * quantized into their rows in the same pass (ttq_cache_rope), and attention
 * over the stored codes (ttq_cache_attention).  ttq_heads says where the heads
 * lie:
 *   d, bits, group, qformat   the cache's, as for ttq_cache_write
 *   n_slots    its rows
 *   heads, kv_heads, head_dim  query heads (a multiple of the K/V heads: query
 *              head h reads K/V head h / (heads / kv_heads)) and their channels:
 *              64, 128 or 256
 *   k_first, v_first   channels of a row at which the K and the V heads begin,
 *              multiples of group.  K and V may lie side by side in one cache
 *              (the same pointers, two ranges that do not overlap) or in two
 *              caches of this format (two sets of pointers).
 * kv_heads * head_dim is a multiple of group. */
typedef struct ttq_heads {
  int64_t d;
  int64_t n_slots;
  int64_t k_first;
  int64_t v_first;
  int32_t heads;
  int32_t kv_heads;
  int32_t head_dim;
  int32_t bits;
  int32_t group;
  uint32_t qformat;
} ttq_heads;

/* Page tables and slot maps of a step, from its request lengths, on the device.
 * A cache of n_pages pages of page_tokens rows (a power of two up to 4096); a
 * table pages [n_seq][max_pages] of the pages that each sequence holds, and a
 * stack of free ones: free_pages [n_pages], the first *free_count are free.
 *   lens   [n_seq] rows that each sequence holds (its first
 *          ceil(lens / page_tokens) table entries are in use)
 *   added  [n_seq] rows that this step adds to it; negative: it has ended.
 * The step's rows are packed in the order of the sequences into T rows.
 *   lens_out   [n_seq] lens + added; 0 for an ended sequence
 *   offsets    [n_seq + 1] the first row of each sequence (at most T)
 *   positions  [T] the position of each row in its sequence (0 behind the last)
 *   slots      [T] its cache row, as ttq_cache_write takes it (-1 behind the last)
 * Pages of ended sequences go onto the stack first, in order (what would pass
 * n_pages is dropped).  New pages are taken from its top, in the order of the
 * sequences; pages, free_pages (above *free_count) are updated, and
 * free_count_out is what is left.
 * A sequence that would pass max_pages, whose rows would pass row T, or for which
 * no pages are left (nor for any behind it that needs some) is refused: it gets
 * no page, its slots are -1, and its length becomes -1 - lens, which
 * ttq_cache_read and ttq_cache_attention take as empty, and a later
 * ttq_cache_extend as lens, so that it may try again.
 * lens_out may be lens and free_count_out free_count; no other two may overlap.
 * Alignment: the types'.  n_seq up to 65535; error rules as for ttq_linear. */
int ttq_cache_extend(int64_t n_seq, int64_t T, int64_t max_pages,
                     int64_t n_pages, int32_t page_tokens, const int32_t* lens,
                     const int32_t* added, int32_t* pages, int32_t* free_pages,
                     const int32_t* free_count, int32_t* lens_out,
                     int32_t* free_count_out, int32_t* offsets,
                     int32_t* positions, int64_t* slots, void* stream);

/* Norms and rotation of T rows' query and key heads, with K and V quantized into
 * the cache rows slots [T] in the same pass:
 *   y = (x r) w,  r = 1 / sqrt(mean(x^2) + eps)    per head, with q_weight or
 *                 k_weight [head_dim] float32; y = x without (NULL)
 *   (a, b) -> (a c - b s, b c + a s),  c, s = cos, sin(positions[t] inv_freq[i])
 * for the pairs i < rot_dim / 2 of a head: channels (i, i + rot_dim / 2), or
 * (2i, 2i + 1) with TTQ_ROPE_INTERLEAVED; channels from rot_dim on stay.
 *   Q [T] rows of heads * head_dim, K and V [T] rows of kv_heads * head_dim
 *             values of x_type, ldq, ldk, ldv elements apart (column ranges of
 *             one projection's result are fine); 16-byte aligned, as is every row
 *   inv_freq  [rot_dim / 2] float32; rot_dim a multiple of 16 up to head_dim, or
 *             0: no rotation (inv_freq and positions may be NULL)
 *   Q_out     [T][heads][head_dim] bf16
 *   slots, k_*, v_*   as for ttq_cache_write, K and V of a row at k_first and
 *             v_first; k_dhalf, v_dhalf optional [d] (the one of the row)
 * The angle is the product in float64, its cosine and sine and r are rounded to
 * float32 from float64; the products and sums above are float32, each rounded, none
 * fused.  So the stored codes, scales and offsets are those that ttq_cache_write
 * gives for the float32 rows.  Q = NULL (heads = 0): only K and V.
 * Alignment: pointers 16 bytes (slots 8, positions, scales and mins 4). */
#define TTQ_ROPE_INTERLEAVED 1u
int ttq_cache_rope(const ttq_heads* hd, int64_t T, int32_t x_type,
                   const void* Q, int64_t ldq, const void* K, int64_t ldk,
                   const void* V, int64_t ldv, const float* q_weight,
                   const float* k_weight, double eps, const float* inv_freq,
                   int32_t rot_dim, uint32_t flags, const int32_t* positions,
                   void* Q_out, const int64_t* slots, const float* k_dhalf,
                   const float* v_dhalf, uint8_t* k_codes, float* k_scales,
                   float* k_mins, uint8_t* v_codes, float* v_scales,
                   float* v_mins, void* stream);

/* Causal attention of T rows over the cached K and V of their sequences:
 *   out[t][h] = sum_j p_j v_j,  p = softmax_j(scale q . k_j)
 * over the keys j of row t's sequence with j <= pos and, with window > 0,
 * j > pos - window.  Row r of a sequence's n rows has pos = lens - n + r: its own
 * K and V are in the cache already.  k_j and v_j are the stored values
 * (m + s q) D^{-1/2}.
 *   Q        [T] rows of heads * head_dim bf16, ldq elements apart, 16-byte
 *            aligned, as is every row
 *   offsets  [n_seq + 1] int32: sequence i has rows offsets[i] .. offsets[i+1]-1
 *            (as ttq_cache_extend gives them); NULL: one row each, T = n_seq.
 *            Rows of no sequence are left as they were.
 *   pages, lens, max_pages, page_tokens   as for ttq_cache_read
 *   max_len  an upper bound of lens that the caller knows (work is divided by
 *            it; keys behind it are not seen), 0: what the pages hold
 *   k_dhalf_inv, v_dhalf_inv   optional [d] float32
 *   out      [T][heads][head_dim] bf16
 *   workspace of at least ttq_cache_attention_workspace_bytes
 * A row that sees no key (an empty or negative length, or every page outside the
 * cache: such keys are not seen) is 0.  Nothing of a key that a row does not see
 * enters it, an infinity or NaN neither; of one that it sees, K's makes the head's
 * row NaN, V's the channels of its group (at least).  A query that is not finite makes
 * its head's row NaN.  (E4M3 codes are finite, as ttq_cache_write stores them.)
 * Products are those of q D^{-1/2} and p in 11 bits (fp16, scaled by powers of two)
 * with exact codes, whose scales enter K's in float32 and V's in 11 bits (what these
 * leave out goes, for the middle of the codes, into the offsets); where a sequence
 * has 64 and more rows of a K/V head on average, with k and v as fp16 values.
 * Scores, sums and the softmax are float32; weights of less than 2^-32 of a row's
 * largest may count as 0.  The sizes of keys may be any that float32 holds, side by
 * side up to 2^100 apart (a row that sees one further above may be infinite): those with
 * a group about 2^8 larger or smaller than the others' cost time (each is added by
 * itself), no bits.  Nor do they pass into rows that do not see them, but that roundings
 * may follow their size where a window is shorter than the 16 (256) rows of a K/V head
 * that are done together.
 * bits 3 to 8 (others: TTQ_EUNSUPPORTED, as are n_slots from 2^31 on); of a sequence
 * at most 2^31 - 4097 keys are seen.
 * heads * T up to 2^31 - 1. */
int ttq_cache_attention_workspace_bytes(const ttq_heads* hd, int64_t T,
                                        int64_t n_seq, int64_t max_pages,
                                        int32_t page_tokens, int64_t max_len,
                                        size_t* bytes);
int ttq_cache_attention(const ttq_heads* hd, int64_t T, int64_t n_seq,
                        int64_t max_pages, int32_t page_tokens, int64_t max_len,
                        int64_t window, double scale, const void* Q,
                        int64_t ldq, const int32_t* offsets,
                        const int32_t* pages, const int32_t* lens,
                        const uint8_t* k_codes, const float* k_scales,
                        const float* k_mins, const uint8_t* v_codes,
                        const float* v_scales, const float* v_mins,
                        const float* k_dhalf_inv, const float* v_dhalf_inv,
                        void* out, void* workspace, size_t workspace_bytes,
                        void* stream);

/* Human-readable text of a status code (static storage). */
const char* ttq_status_string(int status);

/* The hipError_t of the last failed HIP call on this thread (0 if none). */
int ttq_last_hip_error(void);

/* Library version string (static storage). */
const char* ttq_version(void);

/* ---- measurement ------------------------------------------------------
 * When enabled, every kernel the library launches is bracketed by a pair of
 * hipEvents recorded on the launch stream, and ttq_timing_query() sums
 * their elapsed times per kernel kind.  For measurement only: the timing
 * state is process-global and not thread-safe; query synchronizes on the
 * recorded events. */
int ttq_timing_enable(int on);
int ttq_timing_reset(void);
int ttq_kernel_count(void);
const char* ttq_kernel_name(int kernel);
int ttq_timing_query(int kernel, double* total_ms, int64_t* launches);

/* Plain streaming read, the measured ceiling of a one-pass kernel over W (not
 * part of the method): reads `bytes` bytes of device memory at `src` once,
 * in the launch shape of the one-token projection (one workgroup of 16
 * waves per 128 KiB, 64 bytes per lane in flight), and writes the 32-bit XOR
 * of each workgroup's words to sink[ceil(bytes / 131072)] (device memory)
 * so that no load is elided.  Timed as the kernel kind "stream_read".
 * `bytes` is a multiple of 16 (TTQ_EINVAL otherwise); `src` 16-byte and
 * `sink` 4-byte aligned (TTQ_EALIGN); both non-NULL when bytes > 0
 * (TTQ_ENULL).  Enqueued on `stream`. */
int ttq_stream_read(const void* src, int64_t bytes, uint32_t* sink, void* stream);

/* ---- low-rank factors by PCA
 * The static low-rank factors of the projection are initialised by PCA, and
 * may be adapted online ("TTQ: Activation-Aware Test-Time Quantization ...",
 * nl summary, Sec. 2; it summary, Sec. 2; zh summary, Sec. 2.2); the pages
 * give no algorithm.  This call computes
 *   B  [d_out][rank] bf16: an orthonormal basis of the top-rank left
 *      principal subspace of M = W (T = 0), or of M = W D^{1/2} with D from
 *      the activations X (T > 0; p, lambda, alpha as in ttq_linear);
 *   A  [rank][d] bf16 = B^T W;
 *   Wres optional [d_out][d] bf16 = bf16(W - B A), computed from the bf16
 *      B and A, so that ttq_linear(Wres, X, B, A) projects with
 *      W ~ Q_D[Wres] + B A;
 * by randomized subspace iteration (Halko, Martinsson and Tropp, 2011):
 * Q = orth(M Omega), then `iters` times Z = orth(M^T Q), Q = orth(M Z), with
 * orth = CholeskyQR (float32 panels, float64 Cholesky; two passes for the
 * final basis, one for the intermediate panels), B = Q.  When M has rank
 * below `rank` (e.g. W = 0) the columns past the rank are not determined by
 * M: a column whose Gram pivot is at the float32 noise level (1e-5 of the
 * largest) is dropped, and in the first pass of the final basis replaced by
 * a pseudo-random column before the second pass,
 * so B is orthonormal in every case (A and Wres do not depend on the choice).
 *   prm     d, d_out >= 1; rank in {8, 16, 32, 64, 128}, <= min(d, d_out);
 *           T >= 0 (T > 0 needs d % 8 == 0); bits, group, flags and qformat
 *           are not read
 *   iters   power iterations, 0..16
 *   W       [d_out][d] bf16; X [T][d] bf16 (T > 0; NULL otherwise)
 *   Omega   [d][rank] float32, the caller's Gaussian test matrix
 *   workspace at least ttq_lowrank_pca_workspace_bytes, 256-byte aligned
 * All pointers 16-byte aligned device memory.  Same error rules as
 * ttq_linear; the result is deterministic for given inputs. */
int ttq_lowrank_pca_workspace_bytes(const ttq_params* prm, int32_t iters,
                                    size_t* bytes);
int ttq_lowrank_pca(const ttq_params* prm, int32_t iters, const void* W,
                    const void* X, const float* Omega, void* B_out,
                    void* A_out, void* Wres_out, void* workspace,
                    size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* TTQ_H_ */
