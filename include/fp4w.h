/*
 * fp4w.h - block-scaled weight-only FP4 / FP8 matmul for AMD MI355X (gfx950).
 *
 * C ABI.  Plain pointers and sizes only; the library never allocates, frees or
 * synchronises (fp4w_matmul_w4a4_noalloc uses a device array that is part of
 * the library's code object).  Every call validates its arguments, enqueues its kernel(s) on
 * `stream` (a hipStream_t, NULL = the default stream) and returns.  Faults in a
 * kernel surface at the caller's next synchronisation.
 *
 * Sources, cited by page title and section:
 *   [FP4 doc] "MatMulBlockQuantizedFp4Weight - CUDA Operator Documentation"
 *             (ONNX Runtime 1.29.0 contrib-op docs)
 *   [FP8 doc] "MatMulBlockQuantizedFp8Weight - CUDA Operator Documentation"
 *   [Blog]    "ONNX Runtime #32128 - Why Dequantizing 4-Bit Weights Became the
 *             Most Expensive Kernel in H200 Prefill"
 *
 * Common conventions
 *   - All tensor pointers are DEVICE pointers owned by the caller, row-major
 *     and contiguous.  Scalars passed by pointer (weight_scale_2) are device
 *     pointers too: the kernel reads the value, so no host sync is needed.
 *   - T (dtype) is FP16 or BF16 and is the type of A, bias and Y ([FP8 doc] §1
 *     type constraints; [FP4 doc] §1: Y has A's type).  M is the product of
 *     A's leading dimensions; Y is [M, N].
 *   - Scale column of element k: min(k / block_size, scale_cols - 1).  A
 *     partial final K block therefore uses the last scale column ([FP8 doc]
 *     §2); scale_cols may be ceil(K / block_size) or, when K % block_size != 0,
 *     floor(K / block_size) >= 1.  The same rule applies to FP4.
 *   - M == 0 or N == 0: returns FP4W_OK and launches nothing ([FP4 doc] §3,
 *     empty output).  K == 0: Y = bias, or 0 without bias (an empty sum).
 *   - Y must not overlap any input (FP4W_ERR_ALIAS).
 *   - Unaligned pointers or shapes outside a fast kernel's predicate run the
 *     generic kernel; correctness never depends on the fast path.
 *   - Accumulation is FP32.  The result is rounded once to T (round to
 *     nearest even) after the tensor scale and bias are applied.
 *   - Re-entrant and stateless; calls on different streams may overlap
 *     (except fp4w_matmul_w4a4_noalloc calls on one device, which share that
 *     device's scratch).
 */
#ifndef FP4W_H
#define FP4W_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* FP4W_F32 is only a type of router logits (fp4w_moe_route). */
typedef enum { FP4W_F16 = 0, FP4W_BF16 = 1, FP4W_F32 = 2 } fp4w_dtype;

typedef enum {
  FP4W_OK = 0,
  FP4W_ERR_NULL = -1,   /* a required pointer is NULL */
  FP4W_ERR_SHAPE = -2,  /* negative size, odd K for FP4, bad scale_cols, size overflow */
  FP4W_ERR_DTYPE = -3,  /* dtype is not FP4W_F16 / FP4W_BF16 (or an unknown activation or score) */
  FP4W_ERR_BLOCK = -4,  /* block_size < 1 */
  FP4W_ERR_PATH = -5,   /* a forced path (the *_ex calls) does not apply to these arguments */
  FP4W_ERR_LAUNCH = -6, /* HIP reported an error when the kernel was enqueued */
  FP4W_ERR_ALIAS = -7   /* the output overlaps an input */
} fp4w_status;

/* Kernel paths.  FP4W_PATH_AUTO picks the fastest applicable one. */
typedef enum {
  FP4W_PATH_AUTO = 0,
  FP4W_PATH_NONE = 1,            /* empty output: nothing launched */
  FP4W_PATH_FP4_GEMV = 2,        /* MFMA decode GEMV: 1 <= M <= 8, block_size 16, K % 32 == 0 */
  FP4W_PATH_FP4_GEMM = 3,        /* fused MFMA prefill GEMM: block_size 16, K % 64 == 0 */
  FP4W_PATH_FP4_GENERIC = 4,     /* any legal FP4 arguments */
  FP4W_PATH_FP8_GEMV = 5,        /* MFMA decode GEMV: 1 <= M <= 8, block_size % 64 == 0, K % 16 == 0 */
  FP4W_PATH_FP8_GEMM = 6,        /* MFMA prefill GEMM: block_size % 64 == 0, K % 64 == 0 */
  FP4W_PATH_FP8_GENERIC = 7,     /* any legal FP8 arguments */
  FP4W_PATH_DEQUANT_VEC = 8,     /* vectorised dequant: K % 8 == 0, block_size % 8 == 0 */
  FP4W_PATH_DEQUANT_GENERIC = 9, /* any legal dequant arguments */
  FP4W_PATH_QDQ_VEC = 10,        /* vectorised activation QDQ: M*K % 8 == 0 */
  FP4W_PATH_QDQ_GENERIC = 11,    /* any legal QDQ arguments */
  FP4W_PATH_FP4_SKINNY = 12,     /* MFMA skinny matmul: 1 <= M <= 64, block_size 16, K % 128 == 0 */
  FP4W_PATH_FP8_SKINNY = 13,     /* MFMA skinny matmul: 1 <= M <= 64, block_size % 128 == 0, K % 128 == 0 */
  FP4W_PATH_FP8_DEQUANT_VEC = 14,    /* vectorised FP8 dequant: K % 16 == 0, block_size % 16 == 0 */
  FP4W_PATH_FP8_DEQUANT_GENERIC = 15, /* any legal FP8 dequant arguments */
  FP4W_PATH_NVFP4_VEC = 16,     /* NVFP4 activation quantize / QDQ, 16-byte loads (aligned pointers) */
  FP4W_PATH_NVFP4_GENERIC = 17, /* any legal NVFP4 activation arguments */
  FP4W_PATH_MOE_FP4_STREAM = 18,  /* K % 64 == 0, I % 64 == 0, block_size 16 */
  FP4W_PATH_MOE_FP4_GENERIC = 19, /* any legal fp4w_moe arguments */
  FP4W_PATH_MOE_FP8_STREAM = 20,  /* K % 64 == 0, I % 64 == 0, block_size % 128 == 0 */
  FP4W_PATH_MOE_FP8_GENERIC = 21, /* any legal fp8w_moe arguments */
  FP4W_PATH_ATTN_DECODE = 22,  /* max_new * Hq / Hk <= 64, D 64 or 128, page_size % 16 == 0 */
  FP4W_PATH_ATTN_PROMPT = 23,  /* D 64 or 128, page_size % 16 == 0 */
  FP4W_PATH_ATTN_GENERIC = 24  /* any legal fp8w_attention arguments */
} fp4w_path;

/* Operation selector for fp4w_select_path. */
typedef enum {
  FP4W_OP_FP4_MATMUL = 0,
  FP4W_OP_FP8_MATMUL = 1,
  FP4W_OP_FP4_DEQUANT = 2,
  FP4W_OP_FP8_QDQ = 3, /* fp8w_qdq_activation: only M and K are used */
  FP4W_OP_FP8_DEQUANT = 4, /* fp8w_dequant: M is ignored */
  FP4W_OP_NVFP4_ACT = 5 /* fp4w_quantize_activation / fp4w_qdq_activation: only M and K are used */
} fp4w_op;

/*
 * fp4w_matmul - weight-only FP4 matmul, Y = A * dequant(B)^T (+ bias).
 * [FP4 doc] header and §2 Weight Format:
 *   B_dq[n, k] = e2m1(B[n, k]) * e4m3(weight_scale[n, k / block_size]) * weight_scale_2
 *
 *   A              T[M, K]
 *   B              uint8[N, K/2]: two E2M1 codes per byte, low nibble = even k,
 *                  high nibble = odd k.  K must be even.
 *   weight_scale   uint8[N, scale_cols]: raw E4M3 ("fn") bytes, unswizzled.
 *   weight_scale_2 device float*: FP32 tensor scale.
 *   bias           T[N] or NULL.
 *   Y              T[M, N] (written).
 * Errors: FP4W_ERR_NULL (A, B, weight_scale, weight_scale_2 or Y NULL while
 * M, N > 0), FP4W_ERR_SHAPE, FP4W_ERR_BLOCK, FP4W_ERR_DTYPE, FP4W_ERR_ALIAS,
 * FP4W_ERR_LAUNCH.  Nothing is launched when an error is returned.
 */
int fp4w_matmul(const void* A, int64_t M, int64_t K, const uint8_t* B, int64_t N,
                const uint8_t* weight_scale, int64_t scale_cols, int64_t block_size,
                const float* weight_scale_2, const void* bias, void* Y, int dtype, void* stream);

/* Same as fp4w_matmul, with the kernel path forced (FP4W_PATH_AUTO, _FP4_GEMV,
 * _FP4_SKINNY, _FP4_GEMM or _FP4_GENERIC).  FP4W_ERR_PATH if the path does not
 * apply. */
int fp4w_matmul_ex(const void* A, int64_t M, int64_t K, const uint8_t* B, int64_t N,
                   const uint8_t* weight_scale, int64_t scale_cols, int64_t block_size,
                   const float* weight_scale_2, const void* bias, void* Y, int dtype, void* stream,
                   int path);

/*
 * fp8w_matmul - weight-only FP8 matmul ([FP8 doc] §2 Tensor and Scale Format):
 *   Y[m, n] = sum_k A[m, k] * (e4m3(B[n, k]) * b_scale[n, k / block_size]) + bias[n]
 *
 *   A        T[M, K]
 *   B        uint8[N, K]: E4M3 ("fn") bytes.
 *   b_scale  float[N, scale_cols]: FP32 block scales.
 *   bias     T[N] or NULL.   Y  T[M, N].
 * Errors as fp4w_matmul (no evenness rule on K).
 */
int fp8w_matmul(const void* A, int64_t M, int64_t K, const uint8_t* B, int64_t N,
                const float* b_scale, int64_t scale_cols, int64_t block_size, const void* bias,
                void* Y, int dtype, void* stream);

/* Path-forcing variant (FP4W_PATH_AUTO, _FP8_GEMV, _FP8_SKINNY, _FP8_GEMM,
 * _FP8_GENERIC). */
int fp8w_matmul_ex(const void* A, int64_t M, int64_t K, const uint8_t* B, int64_t N,
                   const float* b_scale, int64_t scale_cols, int64_t block_size, const void* bias,
                   void* Y, int dtype, void* stream, int path);

/*
 * fp4w_quantize_activation - step 1 of the FP4 operator's native FP4 x FP4
 * (W4A4) path ([FP4 doc] §6 Native SM120 FP4 x FP4 Path): the activation as
 * packed E2M1 codes with one E4M3 scale per 16-element block (NVFP4).  The
 * pages name the format but no rounding rule; this library uses, per block
 * of 16 consecutive k of one row:
 *   scale = e4m3( min( RNE_f32(amax / 6), 448 ) )   (NaN in the block -> NaN, 0x7F)
 *   code  = e2m1( RNE_f32(a / scale) )               (scale == 0 -> code 0)
 * amax = max |a|; both divisions are IEEE FP32 divisions; e4m3 and e2m1 give
 * the nearest value with ties to the even code; e2m1 saturates at 6 and keeps
 * the sign (a negative quotient rounding to zero gives code 0x8); a NaN
 * quotient gives code 0.  Bit-exact.
 *
 *   A       T[M, K], K % 16 == 0.
 *   codes   uint8[M, K/2] (written): two codes per byte, low nibble = even k
 *           (the weight layout of [FP4 doc] §2).
 *   scales  uint8[M, K/16] (written): E4M3 "fn" bytes.
 * M == 0 or K == 0: FP4W_OK, nothing launched.  Errors: FP4W_ERR_NULL,
 * FP4W_ERR_SHAPE (negative sizes, K % 16 != 0, overflow), FP4W_ERR_DTYPE,
 * FP4W_ERR_ALIAS (codes or scales overlap A or each other),
 * FP4W_ERR_LAUNCH.
 */
int fp4w_quantize_activation(const void* A, int64_t M, int64_t K, uint8_t* codes, uint8_t* scales,
                             int dtype, void* stream);

/* Path-forcing variant (FP4W_PATH_AUTO, _NVFP4_VEC, _NVFP4_GENERIC). */
int fp4w_quantize_activation_ex(const void* A, int64_t M, int64_t K, uint8_t* codes, uint8_t* scales,
                                int dtype, void* stream, int path);

/*
 * fp4w_qdq_activation - the same quantization, decoded back to T:
 *   out[m, k] = e2m1(code) * e4m3(scale)
 * which is exact in FP16 and BF16 (at most 6 significand bits; nonzero
 * magnitudes within [2^-10, 2688]); NaN where the block's scale is NaN.
 *
 *   A    T[M, K], K % 16 == 0.
 *   out  T[M, K] (written).  out == A is allowed (in place); any other
 *        overlap with A is FP4W_ERR_ALIAS.
 * Errors as fp4w_quantize_activation.
 */
int fp4w_qdq_activation(const void* A, int64_t M, int64_t K, void* out, int dtype, void* stream);

/* Path-forcing variant (FP4W_PATH_AUTO, _NVFP4_VEC, _NVFP4_GENERIC). */
int fp4w_qdq_activation_ex(const void* A, int64_t M, int64_t K, void* out, int dtype, void* stream,
                           int path);

/*
 * fp4w_matmul_w4a4 - the FP4 operator's native FP4 x FP4 path ([FP4 doc] §6):
 * the activation quantized as above, times the FP4 weights, plus bias,
 * accumulated in FP32 and rounded once to T:
 *   Y[m, n] = sum_k qdq(A)[m, k] * B_dq[n, k] + bias[n]
 * gfx950's scaled MFMA takes power-of-two (E8M0) scales per 32 elements and
 * cannot apply E4M3 scales per 16 exactly, so this runs as A_work =
 * fp4w_qdq_activation(A) (exact in T), then fp4w_matmul(A_work, ...), whose
 * kernels fold the weight scales into exact BF16/FP16 MFMA operands.  Both
 * steps are enqueued on `stream`.  For a decode GEMV (M <= 8) with
 * M x K <= 24576, A and A_work distinct and A 16-byte aligned, the two are
 * one launch: the GEMV quantize-dequantizes its own LDS copy of A (the same
 * values, bit for bit) and writes it to A_work as well.  The pages' guards (block_size 16,
 * K % 32, N % 32, M > 8) choose this path inside their operator; called
 * directly it takes any arguments fp4w_matmul takes with K % 16 == 0.
 *
 *   A_work   T[M, K] caller-owned workspace that receives qdq(A) (the
 *            library allocates nothing).  A_work == A is allowed and
 *            overwrites A; any other overlap with A is FP4W_ERR_ALIAS, as is
 *            an overlap of A_work with B, weight_scale, weight_scale_2, bias
 *            or Y, or of Y with A.
 *   Other arguments and errors as fp4w_matmul; K % 16 != 0 is
 *   FP4W_ERR_SHAPE.  Every argument is validated before anything is
 *   launched.
 */
int fp4w_matmul_w4a4(const void* A, int64_t M, int64_t K, const uint8_t* B, int64_t N,
                     const uint8_t* weight_scale, int64_t scale_cols, int64_t block_size,
                     const float* weight_scale_2, const void* bias, void* A_work, void* Y, int dtype,
                     void* stream);

/* Size of the library-owned device scratch of fp4w_matmul_w4a4_noalloc. */
#define FP4W_STATIC_SCRATCH_BYTES (32 * 1024 * 1024)

/*
 * fp4w_matmul_w4a4_noalloc - fp4w_matmul_w4a4 for callers that cannot
 * allocate: code under HIP graph capture, serving loops that make no
 * allocations, harnesses that forbid hipMalloc.  The quantized activation
 * goes to a library-owned device array of FP4W_STATIC_SCRATCH_BYTES instead
 * of a caller workspace; the call allocates nothing.
 *
 *   Arguments, results and errors as fp4w_matmul_w4a4 without A_work.
 *   M * K * 2 > FP4W_STATIC_SCRATCH_BYTES is FP4W_ERR_SHAPE.
 *   Each device the library runs on holds its own copy of the array until
 *   the process ends.  Its address is taken on the first call on a device,
 *   with that device current (FP4W_ERR_LAUNCH if HIP cannot provide it).
 *   Every call writes the part it reads before reading it, but all calls on
 *   one device share that device's copy: calls that overlap on one device
 *   (on two streams, or from two threads) race on it, and the caller must
 *   order them.
 */
int fp4w_matmul_w4a4_noalloc(const void* A, int64_t M, int64_t K, const uint8_t* B, int64_t N,
                             const uint8_t* weight_scale, int64_t scale_cols, int64_t block_size,
                             const float* weight_scale_2, const void* bias, void* Y, int dtype,
                             void* stream);

/*
 * fp4w_dequant - expand packed FP4 weights to T[N, K] ([FP4 doc] §5 step 1;
 * [Blog] vectorised dequant).  out[n, k] = RNE_T(RNE_f32(e2m1 * e4m3 * ws2)):
 * the E2M1 x E4M3 product is exact, the FP32 multiply by weight_scale_2 rounds
 * once, then the FP32 value is rounded to T.  Bit-exact; no FTZ.
 *
 *   B, weight_scale, weight_scale_2: as fp4w_matmul.   out: T[N, K] (written).
 * N == 0 or K == 0: FP4W_OK, nothing launched.
 */
int fp4w_dequant(const uint8_t* B, int64_t N, int64_t K, const uint8_t* weight_scale,
                 int64_t scale_cols, int64_t block_size, const float* weight_scale_2, void* out,
                 int dtype, void* stream);

/* Path-forcing variant (FP4W_PATH_AUTO, _DEQUANT_VEC, _DEQUANT_GENERIC). */
int fp4w_dequant_ex(const uint8_t* B, int64_t N, int64_t K, const uint8_t* weight_scale,
                    int64_t scale_cols, int64_t block_size, const float* weight_scale_2, void* out,
                    int dtype, void* stream, int path);

/*
 * fp8w_dequant - expand FP8 weights to T[N, K], the first step of the FP8
 * operator's default path ([FP8 doc] §5 Default Path, step 1).
 *   out[n, k] = RNE_T(RNE_f32(e4m3(B[n, k]) * b_scale[n, min(k / block_size, scale_cols - 1)]))
 * The E4M3 value is exact in FP32; the product with the FP32 block scale
 * rounds once, then the FP32 value is rounded to T.  Bit-exact; no FTZ.
 *
 *   B, b_scale, scale_cols, block_size: as fp8w_matmul.   out: T[N, K] (written).
 * N == 0 or K == 0: FP4W_OK, nothing launched.  Errors: FP4W_ERR_NULL,
 * FP4W_ERR_SHAPE, FP4W_ERR_BLOCK, FP4W_ERR_DTYPE, FP4W_ERR_ALIAS, FP4W_ERR_LAUNCH.
 */
int fp8w_dequant(const uint8_t* B, int64_t N, int64_t K, const float* b_scale, int64_t scale_cols,
                 int64_t block_size, void* out, int dtype, void* stream);

/* Path-forcing variant (FP4W_PATH_AUTO, _FP8_DEQUANT_VEC, _FP8_DEQUANT_GENERIC). */
int fp8w_dequant_ex(const uint8_t* B, int64_t N, int64_t K, const float* b_scale, int64_t scale_cols,
                    int64_t block_size, void* out, int dtype, void* stream, int path);

/*
 * fp8w_qdq_activation - the activation step of the FP8 operator's optional
 * W8A8 mode ([FP8 doc] §6, Optional W8A8 Activation Path):
 *   out[m, k] = RNE_T( RNE_f32( e4m3( sat( RNE_f32(A[m, k] / a_scale) ) ) * a_scale ) )
 * The quotient is an IEEE FP32 division; e4m3() rounds to nearest even; sat()
 * clamps magnitudes above 448 (the largest finite E4M3 "fn" value) to 448 and
 * keeps NaN; the decoded value times a_scale is rounded once in FP32, then to
 * T.  Bit-exact.
 *
 *   A        T[M, K]
 *   a_scale  device float*: the per-tensor activation scale (expected > 0;
 *            other values just follow the IEEE steps above).
 *   out      T[M, K] (written).  out == A is allowed (in place); any other
 *            overlap with A is FP4W_ERR_ALIAS.
 * M == 0 or K == 0: FP4W_OK, nothing launched.  Errors: FP4W_ERR_NULL,
 * FP4W_ERR_SHAPE, FP4W_ERR_DTYPE, FP4W_ERR_ALIAS, FP4W_ERR_LAUNCH.
 */
int fp8w_qdq_activation(const void* A, int64_t M, int64_t K, const float* a_scale, void* out,
                        int dtype, void* stream);

/* Path-forcing variant (FP4W_PATH_AUTO, _QDQ_VEC, _QDQ_GENERIC). */
int fp8w_qdq_activation_ex(const void* A, int64_t M, int64_t K, const float* a_scale, void* out,
                           int dtype, void* stream, int path);

/*
 * fp8w_matmul_w8a8 - the FP8 operator with its optional a_scale input
 * ([FP8 doc] §3 dispatch chain, whose first step quantizes/dequantizes A when
 * a_scale is present, and §6): A_work = fp8w_qdq_activation(A), then
 * Y = fp8w_matmul(A_work, ...).  Both steps are enqueued on `stream`.
 *
 *   A_work   T[M, K] caller-owned workspace that receives the quantized
 *            activation (the library allocates nothing).  A_work == A is
 *            allowed and overwrites A; any other overlap with A is
 *            FP4W_ERR_ALIAS, as is an overlap of Y with A_work.
 *   a_scale  device float*, as fp8w_qdq_activation.
 *   Other arguments and errors as fp8w_matmul.  Every argument is validated
 *   before anything is launched.
 */
int fp8w_matmul_w8a8(const void* A, int64_t M, int64_t K, const uint8_t* B, int64_t N,
                     const float* b_scale, int64_t scale_cols, int64_t block_size,
                     const float* a_scale, const void* bias, void* A_work, void* Y, int dtype,
                     void* stream);

/* ------------------------------------------------------------------------
 * Around a mixture-of-experts block: the norm between blocks, the routing of
 * tokens to experts, and the expert layer on FP4 or FP8 weights.
 * ------------------------------------------------------------------------ */

/*
 * fp4w_block_norm - the norms after one block and before the next, with the
 * block's gate and the residual scale, in one pass over x:
 *   b = x                                                       (post_weight NULL)
 *     = x * rsqrt(mean(x^2) + eps) * (weight_offset + post_weight)
 *   r = residual + scale * gate * b                             (residual_out)
 *   y = r * rsqrt(mean(r^2) + eps) * (weight_offset + pre_weight)
 * Means are over a row's K values.  Everything is FP32; residual_out and y
 * are each rounded once, y from the unrounded r.  (So a row whose sum of
 * squares passes FP32's range, with values of some 1e19, is normed to 0.)
 *
 *   x             T[M, K]: a block's output (or, alone, an embedding).
 *   post_weight   T[K] or NULL: no norm of x.
 *   gate          T[gate_rows, K] or NULL (a gate of one); gate_rows is 1
 *                 (one row for every token) or M.
 *   residual      T[M, K] or NULL (zero).
 *   pre_weight    T[K]; NULL exactly when y is NULL.
 *   residual_out  T[M, K] (written) or NULL; not NULL together with y.
 *   y             T[M, K] (written) or NULL.
 * residual_out == x, residual_out == residual, y == x and y == residual are
 * allowed (in place); any other overlap is FP4W_ERR_ALIAS.  M == 0 or K == 0:
 * FP4W_OK, nothing launched.  Errors: FP4W_ERR_NULL, FP4W_ERR_SHAPE,
 * FP4W_ERR_DTYPE, FP4W_ERR_ALIAS, FP4W_ERR_LAUNCH.
 */
int fp4w_block_norm(const void* x, int64_t M, int64_t K, const void* post_weight, const void* gate,
                    int64_t gate_rows, float scale, const void* residual, const void* pre_weight,
                    float weight_offset, float eps, void* residual_out, void* y, int dtype,
                    void* stream);

#define FP4W_MOE_MAX_EXPERTS 1024
#define FP4W_MOE_MAX_TOPK 64

typedef enum { FP4W_SCORE_SOFTMAX = 0, FP4W_SCORE_SIGMOID = 1 } fp4w_score;
typedef enum { FP4W_ACT_SILU = 0, FP4W_ACT_GELU_TANH = 1 } fp4w_activation;

/*
 * fp4w_moe_route - the experts of each token and their weights:
 *   score   = softmax(logits) over the E experts, or sigmoid(logits)
 *   key     = logits (select_bias NULL), or score + select_bias in FP64
 *   ids     = the topk largest keys in falling order, ties to the lowest index
 *   weights = scale * score[ids], divided by the sum of the topk scores when
 *             `renormalize` is nonzero (0 where that sum is 0)
 * Renormalised weights are right however small the scores are, to where FP64
 * ends: a score below e^-700 (softmax: e^-700 times the row's largest) counts
 * as 0, so choices masked by the type's lowest value weigh nothing beside
 * others.  The bias only takes part in the choice.  An expert whose logit or
 * key is -inf or NaN is masked: it is never chosen.  Masked by its logit, it
 * adds nothing to a softmax; masked by select_bias alone, its share of the
 * softmax stays (it shows where `renormalize` is 0).  Places that no expert is
 * left for get id -1 and weight 0, which fp4w_moe skips; a row with every
 * expert masked is all such places.  Logits of +inf share the softmax among
 * themselves.
 *
 *   logits       logits_dtype[M, E]: FP4W_F16, FP4W_BF16 or FP4W_F32.
 *   select_bias  float[E] or NULL.
 *   ids          int32[M, topk] (written).   weights  float[M, topk] (written).
 * E <= FP4W_MOE_MAX_EXPERTS and topk <= FP4W_MOE_MAX_TOPK (topk > E is
 * legal).  M is not limited.  M == 0 or topk == 0: FP4W_OK, nothing launched.
 * Errors: FP4W_ERR_NULL, FP4W_ERR_SHAPE, FP4W_ERR_DTYPE (an unknown type or
 * score), FP4W_ERR_ALIAS, FP4W_ERR_LAUNCH.
 */
int fp4w_moe_route(const void* logits, int64_t M, int64_t E, int64_t topk, int score,
                   const float* select_bias, int renormalize, float scale, int32_t* ids,
                   float* weights, int logits_dtype, void* stream);

/*
 * Bytes of caller-owned workspace that fp4w_moe and fp8w_moe need for these
 * sizes, or a negative fp4w_status for illegal ones.  It does not fall when a
 * size grows, so what a largest batch needs serves every smaller call.
 * Host-only.
 */
int64_t fp4w_moe_workspace(int64_t M, int64_t topk, int64_t K, int64_t I);

/*
 * fp4w_moe - a whole mixture-of-experts layer on FP4 weights, made for a few
 * tokens (decode, small batches) and taking any number.  With e = ids[m, j] and W1[e], W3[e] the
 * first and last I rows of w13[e]:
 *   h    = act(A[m] . W1[e]^T) * (A[m] . W3[e]^T)
 *   Y[m] = sum_j weights[m, j] * (h . W2[e]^T)
 *   act  = silu(g) = g / (1 + exp(-g)), or gelu in its tanh form
 * Weights are those of fp4w_matmul: e2m1 * e4m3(block of block_size k) *
 * scale_2 of the expert.  An id outside [0, E) contributes nothing (a masked
 * or absent choice, an expert on another device); a token without any gets
 * zeros.  A token may name an expert twice: both count.  Accumulation is
 * FP32, h is kept to 16 significand bits at least, and Y is rounded once; the
 * result for a token does not depend on the order in which the GPU works.
 *
 *   A            T[M, K]
 *   ids          int32[M, topk]    weights  float[M, topk]
 *   w13          uint8[E, 2 I, K/2]; gate rows, then up rows.
 *   w13_scale    uint8[E, 2 I, ceil(K / block_size)]: E4M3 bytes.
 *   w13_scale_2  float[E] (device)
 *   w2           uint8[E, K, I/2]
 *   w2_scale     uint8[E, K, ceil(I / block_size)]
 *   w2_scale_2   float[E] (device)
 *   workspace    at least fp4w_moe_workspace(M, topk, K, I) bytes, 4-byte
 *                aligned; what it holds before does not matter.  Calls that
 *                may run at once (two streams, two replayed graphs) need
 *                one each.
 *   Y            T[M, K] (written).
 * K and I must be even, E <= FP4W_MOE_MAX_EXPERTS, topk <= FP4W_MOE_MAX_TOPK
 * and M, M * topk < 2^31.  A call works through its tokens in parts of at most
 * 4096 choices, one after the other in the same workspace, and every part
 * reads the weights of the experts that its tokens name.  M == 0 or K == 0: FP4W_OK,
 * nothing launched.  topk == 0, E == 0 or I == 0: Y = 0 (an empty sum).
 * Errors: FP4W_ERR_NULL, FP4W_ERR_SHAPE (also a workspace that is too small
 * or unaligned), FP4W_ERR_BLOCK, FP4W_ERR_DTYPE (also an unknown activation),
 * FP4W_ERR_ALIAS (Y or the workspace overlaps an input or the other),
 * FP4W_ERR_LAUNCH.
 */
int fp4w_moe(const void* A, int64_t M, int64_t K, const int32_t* ids, const float* weights,
             int64_t topk, const uint8_t* w13, const uint8_t* w13_scale, const float* w13_scale_2,
             const uint8_t* w2, const uint8_t* w2_scale, const float* w2_scale_2, int64_t E,
             int64_t I, int64_t block_size, int activation, void* workspace,
             int64_t workspace_bytes, void* Y, int dtype, void* stream);

/* Path-forcing variant (FP4W_PATH_AUTO, _MOE_FP4_STREAM, _MOE_FP4_GENERIC). */
int fp4w_moe_ex(const void* A, int64_t M, int64_t K, const int32_t* ids, const float* weights,
                int64_t topk, const uint8_t* w13, const uint8_t* w13_scale,
                const float* w13_scale_2, const uint8_t* w2, const uint8_t* w2_scale,
                const float* w2_scale_2, int64_t E, int64_t I, int64_t block_size, int activation,
                void* workspace, int64_t workspace_bytes, void* Y, int dtype, void* stream,
                int path);

/*
 * fp8w_moe - the same layer on FP8 weights as fp8w_matmul takes them: E4M3
 * bytes with FP32 scales per block_size k of a row.
 *   w13  uint8[E, 2 I, K]    w13_scale  float[E, 2 I, ceil(K / block_size)]
 *   w2   uint8[E, K, I]      w2_scale   float[E, K, ceil(I / block_size)]
 * Other arguments, results and errors as fp4w_moe (K and I may be odd).
 */
int fp8w_moe(const void* A, int64_t M, int64_t K, const int32_t* ids, const float* weights,
             int64_t topk, const uint8_t* w13, const float* w13_scale, const uint8_t* w2,
             const float* w2_scale, int64_t E, int64_t I, int64_t block_size, int activation,
             void* workspace, int64_t workspace_bytes, void* Y, int dtype, void* stream);

/* Path-forcing variant (FP4W_PATH_AUTO, _MOE_FP8_STREAM, _MOE_FP8_GENERIC). */
int fp8w_moe_ex(const void* A, int64_t M, int64_t K, const int32_t* ids, const float* weights,
                int64_t topk, const uint8_t* w13, const float* w13_scale, const uint8_t* w2,
                const float* w2_scale, int64_t E, int64_t I, int64_t block_size, int activation,
                void* workspace, int64_t workspace_bytes, void* Y, int dtype, void* stream,
                int path);

/* ------------------------------------------------------------------------
 * Between the projections of an attention block: norms and rotation of the
 * query and key heads, a paged cache of keys and values in 8 bits, and
 * attention over it.
 *
 * Rows.  q, k and v are [M, heads, D] with the D values of a head and the
 * heads of a token side by side; the stride from one token to the next is an
 * argument, in values, at least heads * D (so they may be parts of one
 * projection's output).
 *
 * Rotation.  cos and sin are float[rope_rows, rope_dims / 2] with rope_rows at
 * least 1, the tables of a token's position; the first rope_dims (even, at most D) values of a head are
 * rotated in pairs, (i, i + rope_dims / 2), or (2 i, 2 i + 1) if `interleaved`
 * is nonzero:   (a, b) -> (a cos - b sin, b cos + a sin).
 * Both NULL: no rotation.  A position outside [0, rope_rows) makes a token's
 * rotated values NaN.
 *
 * Cache.  Pages of page_size tokens:
 *   k_cache  uint8[num_pages, Hk, page_size, D]   E4M3 "fn" codes
 *   v_cache  uint8[num_pages, Hk, D, page_size]   (the tokens of one value side by side)
 *   k_scale, v_scale  uint8[num_pages, Hk]        powers of two: 2^(byte - 127),
 *                                                 NaN for 255 (OCP MX's E8M0)
 * A stored value is its code times its page's scale for that head.  Powers of
 * two cost a floating-point code nothing but the end of its range, and make
 * scaling exact.
 *
 * Sequences.  Sequence b holds seq_lens[b] tokens, the new ones of the call
 * among them; token t of it is in page page_table[b, t / page_size], slot
 * t % page_size.  Its new tokens are the rows starts[b] .. starts[b + 1] - 1 of
 * the call, in order, and are the last ones of the sequence.  starts (int32
 * [B + 1], not falling, from 0 to at most M) may be NULL if M == B: one new
 * token for each.  Rows from starts[B] on belong to no sequence: what would be
 * written for them is left as it was.  Tokens at or behind max_pages *
 * page_size, and those of a page id outside [0, num_pages), are absent: they
 * are not written, and nobody attends them.
 * ------------------------------------------------------------------------ */

#define FP8W_MAX_HEAD_SIZE 1024

/*
 * fp4w_qk_norm_rope - norms of queries and keys for each head, with the
 * rotation in the same pass:
 *   n = x                                                       (weight NULL)
 *     = x * rsqrt(mean(x^2) + eps) * (weight_offset + weight)
 *   out = n with its first rope_dims values rotated
 * in FP32, rounded once to T.  The mean is over a head's D values.
 *
 *   q  T[M, Hq, D]    k  T[M, Hk, D]   (Hq or Hk may be 0)
 *   q_weight, k_weight  T[D] or NULL, each for itself.
 *   positions  int32[M], or NULL: row m is position m.
 *   q_out, k_out  T, as q and k with strides of their own (written).  An
 *       output may be its input (with the same stride); any other overlap of
 *       an output with an input or the other output is FP4W_ERR_ALIAS.
 * M == 0 or D == 0 or no heads: FP4W_OK, nothing launched.  Errors:
 * FP4W_ERR_NULL, FP4W_ERR_SHAPE (also D > FP8W_MAX_HEAD_SIZE, an odd or too
 * large rope_dims, cos without sin), FP4W_ERR_DTYPE, FP4W_ERR_ALIAS,
 * FP4W_ERR_LAUNCH.
 */
int fp4w_qk_norm_rope(const void* q, int64_t q_stride, int64_t Hq, const void* k, int64_t k_stride,
                      int64_t Hk, int64_t M, int64_t D, const void* q_weight, const void* k_weight,
                      float weight_offset, float eps, const float* cos, const float* sin,
                      int64_t rope_rows, int64_t rope_dims, int interleaved,
                      const int32_t* positions, void* q_out, int64_t q_out_stride, void* k_out,
                      int64_t k_out_stride, int dtype, void* stream);

/*
 * fp8w_kv_append - new keys and values into the cache, with the norms and the
 * rotation on the way (all optional):
 *   k is normed by k_weight and rotated as above, in FP32 and not rounded
 *   before it becomes codes; v is taken as it is; q, where given, goes to
 *   q_out as in fp4w_qk_norm_rope.
 * Per page and head, for keys and values apart:
 *   e = the smallest integer >= -126 with |x| <= 448 * 2^e for every finite new
 *       value x in the page; where the page also holds earlier tokens of the
 *       sequence, not less than the page's exponent so far
 *   code = e4m3(x * 2^-e), to nearest, ties to the even code; NaN for an
 *       infinity or NaN
 * Where e grew, the earlier tokens' codes become e4m3(code * 2^(old - e)),
 * which is exact but for values below 2^(e - 6).  Other slots of the page keep
 * what they hold.
 *
 *   k, v   T[M, Hk, D] with strides.   q  T[M, Hq, D] or NULL (then Hq = 0).
 *   positions  int32[M] for the rotation, or NULL: the token's place in its
 *          sequence.
 *   q_out  T (written); may be q with the same stride.
 * A page may be appended to through one place of the page table only: two
 * sequences that name one page, or one that names it twice, race on it.
 * Sequences that share full pages only read them.
 * M == 0, B == 0 or D == 0: FP4W_OK, nothing launched.  Errors as above, and
 * FP4W_ERR_SHAPE for a page_size < 1 or max_pages * page_size >= 2^31;
 * FP4W_ERR_ALIAS if a part of the cache overlaps an input, q_out or another.
 */
int fp8w_kv_append(const void* k, int64_t k_stride, const void* v, int64_t v_stride, int64_t M,
                   int64_t Hk, int64_t D, const void* q, int64_t q_stride, int64_t Hq,
                   const void* q_weight, const void* k_weight, float weight_offset, float eps,
                   const float* cos, const float* sin, int64_t rope_rows, int64_t rope_dims,
                   int interleaved, const int32_t* positions, void* q_out, int64_t q_out_stride,
                   const int32_t* starts, int64_t B, const int32_t* seq_lens,
                   const int32_t* page_table, int64_t max_pages, uint8_t* k_cache,
                   uint8_t* k_scale, uint8_t* v_cache, uint8_t* v_scale, int64_t num_pages,
                   int64_t page_size, int dtype, void* stream);

/*
 * Bytes of caller-owned workspace that fp8w_attention needs for these sizes,
 * or a negative fp4w_status for illegal ones.  It does not depend on how long
 * the sequences are, and does not fall when M, B or max_new grows.  Host-only.
 */
int64_t fp8w_attention_workspace(int64_t M, int64_t Hq, int64_t Hk, int64_t D, int64_t B,
                                 int64_t max_new);

/*
 * fp8w_attention - attention of the new tokens over the cache.  For row m, at
 * position p = seq_lens[b] - (starts[b + 1] - starts[b]) + (m - starts[b]) of
 * its sequence, and query head h, which reads the key and value head
 * h / (Hq / Hk):
 *   s_t = scale * sum_d q[m, h, d] * K_t[d]
 *   Y[m, h] = sum_t exp(s_t) V_t / sum_t exp(s_t)
 *   lse[m, h] = log sum_t exp(s_t)
 * over the tokens t of the sequence that are held (t < seq_lens[b], their page
 * present), with t <= p if `causal` is nonzero and t > p - window if window >
 * 0.  Without any, Y is 0 and lse -inf; where every score is -inf (an infinite
 * query) both are NaN, as 0 / 0 is.  What slots of other tokens hold, NaN
 * among it, does not show.  Scores, softmax and sums are FP32; Y is rounded
 * once.  The result for a row does not depend on the order in which the GPU
 * works, but its last bits may on the rest of the batch (where its sum is cut).
 * The decode and prompt kernels (heads of 64 and 128 in pages of a multiple of
 * 16 tokens, everything 16-byte aligned) take both sides of the second product
 * in T: the softmax's numerators, rounded, and the values, in steps of 2^-23
 * (FP16) or 2^-109 (BF16) at the least.  There, for FP16, a stored value of 2^17
 * or more counts as NaN, as does any but 0 in a page with a value scale of 2^24
 * or more (appended FP16 stays below both).  The generic kernel has no such
 * rounding and no such limit.
 *
 *   q        T[M, Hq, D] with a stride.   Hq is a multiple of Hk.
 *   max_new  no sequence has more new tokens (rows behind it are left as they
 *            were); it chooses the kernel.  1 if starts is NULL.
 *   max_pages  how far the table reaches has a part in the choice too: up to 16
 *            rows (new tokens x Hq / Hk) over tables with room for at most 1024
 *            tokens take one launch, wider ones two, whatever the lengths are.
 *   workspace  at least fp8w_attention_workspace(...) bytes, 16-byte aligned;
 *            what it holds before does not matter.  Calls that may run at once
 *            (two streams, two replayed graphs) need one each.
 *   Y        T[M, Hq, D] (written), contiguous.   lse  float[M, Hq] (written) or NULL.
 * M == 0, B == 0, Hq == 0 or D == 0: FP4W_OK, nothing launched.  Errors:
 * FP4W_ERR_NULL, FP4W_ERR_SHAPE (also a workspace that is too small or
 * unaligned), FP4W_ERR_DTYPE, FP4W_ERR_ALIAS, FP4W_ERR_LAUNCH.
 */
int fp8w_attention(const void* q, int64_t q_stride, int64_t M, int64_t Hq, int64_t Hk, int64_t D,
                   const int32_t* starts, int64_t B, const int32_t* seq_lens,
                   const int32_t* page_table, int64_t max_pages, int64_t max_new,
                   const uint8_t* k_cache, const uint8_t* k_scale, const uint8_t* v_cache,
                   const uint8_t* v_scale, int64_t num_pages, int64_t page_size, float scale,
                   int causal, int64_t window, void* workspace, int64_t workspace_bytes, void* Y,
                   float* lse, int dtype, void* stream);

/* Path-forcing variant (FP4W_PATH_AUTO, _ATTN_DECODE, _ATTN_PROMPT, _ATTN_GENERIC). */
int fp8w_attention_ex(const void* q, int64_t q_stride, int64_t M, int64_t Hq, int64_t Hk, int64_t D,
                      const int32_t* starts, int64_t B, const int32_t* seq_lens,
                      const int32_t* page_table, int64_t max_pages, int64_t max_new,
                      const uint8_t* k_cache, const uint8_t* k_scale, const uint8_t* v_cache,
                      const uint8_t* v_scale, int64_t num_pages, int64_t page_size, float scale,
                      int causal, int64_t window, void* workspace, int64_t workspace_bytes, void* Y,
                      float* lse, int dtype, void* stream, int path);

/*
 * fp4w_select_path - the path FP4W_PATH_AUTO takes for these sizes, assuming
 * 16-byte-aligned pointers ([FP4 doc] §3 and [FP8 doc] §3 dispatch chains,
 * re-derived for this library).  `op` is an fp4w_op.  For dequant, M is
 * ignored.  Returns an fp4w_path, or a negative fp4w_status for illegal
 * arguments.  Host-only; never touches the GPU.
 */
int fp4w_select_path(int op, int64_t M, int64_t N, int64_t K, int64_t block_size,
                     int64_t scale_cols);

/* Static strings; never NULL. */
const char* fp4w_status_string(int status);
const char* fp4w_path_name(int path);

#ifdef __cplusplus
}
#endif

#endif /* FP4W_H */
