/*
 * ckl_ops.h -- C ABI of libckl.so, the operators around the loss of ckl.h: the
 * norm that makes the student's hidden states H (forward and backward), the
 * 8-bit form in which a forward pass keeps an activation for its backward
 * pass, and sampling token ids from logits.
 *
 * The conventions are those of ckl.h: row-major arrays in device memory owned
 * by the caller, nothing allocated or kept between calls, host-detectable
 * errors returned before anything is enqueued, work enqueued on `stream` (a
 * cudaStream_t of the current device) without waiting.  Every call may be
 * captured into a CUDA graph.  bf16 arrays are uint16_t bit patterns; where an
 * array may have one of two types, a CKL_DTYPE_* argument says which.
 */
#ifndef CKL_OPS_H_
#define CKL_OPS_H_

#include "ckl.h"

#ifdef __cplusplus
extern "C" {
#endif

enum {
  CKL_DTYPE_BF16 = 0,
  CKL_DTYPE_F32 = 1
};

/* Elements of a row that share a scale in the 8-bit form. */
#define CKL_ACT8_GROUP 32
/* Largest vocabulary of ckl_sample. */
#define CKL_SAMPLE_MAX_V 2097152
/* Bit of ckl_sample's device_status: a NaN or +inf logit, or a row's parameter
 * or number out of range. */
#define CKL_SAMPLE_BAD_INPUT 16

/*
 * Activations in 8 bits.  A row of d elements has round_up(d, 32) / 32 groups;
 * a group keeps an exponent byte b and per element an integer q of -127..127,
 * and the element's value is q 2^(b - 133).  b is the smallest that holds the
 * group's largest magnitude after rounding to the nearest integer (ties to
 * even; at most 254, so the largest floats clamp to 127), so that an element is
 * off by at most the group's largest magnitude / 127, or 2^-134 where that is
 * more (fp32 groups below 2^-127: the scale goes no lower than 2^-133, bf16's
 * smallest value).  An element that is not finite is stored as q = -128, reads
 * back as NaN, and does not count towards its group's scale.  Values of q read back exactly in bf16 and fp32.
 *
 * ckl_act8_pack:   x [T, d] -> q [T, d], exponents [T, groups]
 * ckl_act8_unpack: q, exponents -> x [T, d]
 * T >= 0, 1 <= d < 2^31, T d < 2^62.  x aligned to its element.  Rows are taken 16
 * bytes at a time when they are a multiple of that long and x is 16-byte and q
 * 8-byte aligned, and an element at a time otherwise; results are the same.
 */
CKL_API int ckl_act8_pack(const void* x, int32_t dtype, int64_t T, int64_t d, int8_t* q,
                          uint8_t* exponents, void* stream);
CKL_API int ckl_act8_unpack(const int8_t* q, const uint8_t* exponents, int64_t T, int64_t d,
                            int32_t dtype, void* x, void* stream);

/*
 * Layer norm (mean != NULL) or RMS norm (mean == NULL) of the rows of x:
 *   mu = mean(x) or 0,  r = (mean((x - mu)^2) + eps)^-1/2
 *   y = (x - mu) r gamma + beta
 *   x, y       [T, d] of type dtype
 *   gamma      [d] of type param_dtype; NULL = 1
 *   beta       [d] of type param_dtype; NULL = 0
 *   mean, rstd [T] fp32  out: mu and r, for the backward; mean may be NULL
 *   q, exponents         out: x in 8 bits, for a backward that does not keep
 *                        x (ckl_act8_pack's result); both NULL = none
 * A row whose (x - mu)^2 add up to more than the largest float gets r = 0.
 * T >= 0, 1 <= d < 2^31 - 2^17, T d < 2^60, eps >= 0 and finite.  Arrays aligned
 * to their elements; rows are taken 16 bytes at a time when they are a multiple
 * of that long and x, y, gamma and beta are 16-byte and q 8-byte aligned.  y may
 * be x.
 */
CKL_API int ckl_norm_forward(const void* x, int32_t dtype, const void* gamma, const void* beta,
                             int32_t param_dtype, int64_t T, int64_t d, float eps, void* y,
                             float* mean, float* rstd, int8_t* q, uint8_t* exponents,
                             void* stream);

/* Workspace bytes of ckl_norm_backward; 0 for sizes outside its range.  8 d bytes
 * for each row, 160 at most; for d > 16384 for each 64 rows, 64 at most. */
CKL_API size_t ckl_norm_workspace_bytes(int64_t T, int64_t d);

/*
 * The norm's backward, with xh = (x - mu) r and a = dy gamma:
 *   dx = r (a - mean(a) - xh mean(a xh))   (without mean(a) when mean == NULL)
 *   dgamma = sum_t dy xh,  dbeta = sum_t dy
 *   dy, dx     [T, d] of type dtype; dx may be dy
 *   x          [T, d] of type dtype, or NULL: q and exponents instead
 *   mean, rstd [T] fp32 from the forward; mean NULL without centring
 *   gamma      as in the forward
 *   dgamma     [d] fp32  out, or NULL
 *   dbeta      [d] fp32  out, or NULL
 *   accumulate non-zero: dgamma and dbeta are added to
 *   workspace  >= ckl_norm_workspace_bytes(T, d) bytes, 16-byte aligned (may be
 *              NULL when dgamma and dbeta are); calls that share it must not
 *              overlap on the GPU
 * The sums over t are taken in a fixed order: the same call gives the same bits.
 */
CKL_API int ckl_norm_backward(const void* dy, int32_t dtype, const void* x, const int8_t* q,
                              const uint8_t* exponents, const float* mean, const float* rstd,
                              const void* gamma, int32_t param_dtype, int64_t T, int64_t d,
                              void* dx, float* dgamma, float* dbeta, int32_t accumulate,
                              void* workspace, size_t workspace_bytes, void* stream);

/*
 * Token ids drawn from rows of logits.  The tokens of a row are ordered by
 * descending logit, equal logits by lowest id; with w = exp((z - max) /
 * temperature), the kept tokens are the shortest of three prefixes:
 *   top_k  the first top_k (<= 0 or >= V: all)
 *   top_p  the smallest prefix with at least top_p of the mass of the top_k
 *          (>= 1: all; at least one token)
 *   min_p  the tokens with w >= min_p (0: all)
 * With S their mass, u draws the first token whose running mass passes u S;
 * its log-prob is log(w / S), under the distribution drawn from.
 * temperature 0 takes the first token, with log-prob 0.  Weights and sums are
 * fp64; equal calls give equal results.
 *   logits [T, V] bf16, ld elements (>= V) from a row to the next.  -inf is
 *          never drawn.
 *   u      [T, N] fp32 in [0, 1)
 *   temperature (>= 0), top_k, top_p (> 0), min_p (0..1): for every row, or
 *          per row ([T] device arrays that are used where they are not NULL)
 *   ids    [T, N] int32 out; logp [T, N] fp32 out, may be NULL
 *   device_status: may be NULL; CKL_SAMPLE_BAD_INPUT is OR'ed into it (the
 *          caller clears it) when a row has a NaN or +inf logit or a parameter
 *          out of range, or a number of u is
 * Such rows (for u: such draws), and rows without a finite logit, get id -1
 * and log-prob NaN.  N draws with replacement of a teacher's row, with equal
 * log-probs, are a teacher cache whose gradient is unbiased: ckl_forward takes
 * repeated ids as they are.
 * Rows of more than 4096 logits (2048 with one draw) are fast while their logits
 * are 0 or 2^-40 <= |z| < 256, or so low that they weigh under 2^-64 of the
 * largest (-inf; a mask's lowest finite value at temperatures up to about 5).
 * Other rows give the same results, thirty to sixty times slower with one draw
 * (128256 logits 1.2 ms) and some 0.13 ms a draw more with several.
 * T >= 0, 1 <= V <= CKL_SAMPLE_MAX_V (CKL_ERR_UNSUPPORTED above), N >= 1,
 * T N < 2^31.
 */
CKL_API int ckl_sample(const uint16_t* logits, int64_t ld, int64_t T, int64_t V, const float* u,
                       int32_t N, double temperature, int32_t top_k, double top_p, double min_p,
                       const float* temperature_rows, const int32_t* top_k_rows,
                       const float* top_p_rows, const float* min_p_rows, int32_t* ids,
                       float* logp, int32_t* device_status, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* CKL_OPS_H_ */
