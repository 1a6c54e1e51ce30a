/*
 * mqconv_block.h -- C ABI of the operators that stand around the convolutions
 * of mqconv.h in a trained network: group normalization with an activation
 * (forward and backward), dropout from a counter-based generator, and the
 * replay cache (samples quantized as they are stored, and read back).
 *
 * The conventions of mqconv.h hold: device pointers owned by the caller, work
 * enqueued on `stream`, every argument checked before any HIP call, an
 * mq_status returned, equal inputs giving bit-identical outputs. Descriptors
 * (mq_norm, mq_drop, mq_cache) are HOST structs, read during the call only.
 * fp32 tensors are [H][W][N][C], 4-byte aligned; every tensor holds at most
 * 2^30 elements, channel padding included.
 */
#ifndef MQCONV_BLOCK_H
#define MQCONV_BLOCK_H

#include "mqconv.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Activations. MQ_ACT_SILU: u / (1 + exp(-u)); MQ_ACT_GELU: u times the
 * normal distribution's integral (the erf form). Both keep their digits in the
 * negative tail, but for about |u| and 1.5 u^2 roundings (2^-24 of the result),
 * and may be 0 where the exponential leaves fp32's normal range (SiLU from -87,
 * GELU from -13 on). A plain 32-bit integer, as mq_elem; an unknown value is
 * rejected with MQ_ERR_FORMAT. */
enum { MQ_ACT_NONE = 0, MQ_ACT_RELU = 1, MQ_ACT_SILU = 2, MQ_ACT_GELU = 3 };
typedef int32_t mq_act;

/* ---------------------------------------------------------------------------
 * Dropout
 * ---------------------------------------------------------------------------
 * Whether an element is kept depends on its place and the seed alone, so the
 * mask is never stored: a backward pass makes it again. The element on memory
 * row `row` (its index divided by C) and channel c takes the 16-bit number
 * r = half word c mod 8 (word (c mod 8) / 2, its low half first) of
 * Philox4x32-10 (Salmon et al., SC'11) at counter (row, c / 8, 1, 0) with key
 * (s & 0xffffffff, s >> 32), s = seed + *step (seed where step is NULL). It
 * is dropped, set to +0 whatever it holds, when r < q, q = p * 65536 rounded
 * to the nearest integer, and multiplied by 65536 / (65536 - q) (fp32)
 * otherwise: the factor belongs to the probability that is realized, q /
 * 65536, so the expectation is unchanged exactly. p = 1 drops everything.
 * The third counter word keeps these numbers apart from those of
 * mqconv_quantize_sr (0 there) under an equal seed. */
typedef struct {
  float p;              /* in [0, 1], else MQ_ERR_UNSUPPORTED */
  uint64_t seed;
  const uint64_t* step; /* device, 8-byte aligned, or NULL: read when the kernel runs, so a
                           captured graph draws a new mask at every replay */
} mq_drop;

/* y = drop(x) + residual (residual NULL: drop(x)), fp32 [H][W][N][C]. The
 * gradient of x is the same call on the gradient of y (without residual). y
 * may be x or residual. */
int mqconv_dropout(const float* x, const float* residual, int32_t h, int32_t w, int32_t n, int32_t c,
                   const mq_drop* drop, float* y, void* stream);

/* mqconv_dropout without residual whose output is MX-quantized: dst (ACT or
 * GRAD, (H, W, N, C)) receives what mqconv_quantize of the fp32 result would
 * write; the fp32 result never reaches memory. */
int mqconv_dropout_mx(const float* x, const mq_drop* drop, mq_mx dst, void* stream);

/* ---------------------------------------------------------------------------
 * Group normalization with an activation, channels last
 * ---------------------------------------------------------------------------
 * The C channels form `groups` groups of D = C / groups neighbours; a sample's
 * group holds M = H * W * D values:
 *   mean[n,g] = sum x / M;  rstd[n,g] = 1 / sqrt(sum (x - mean)^2 / M + eps)
 *   u = gamma[c] * (x - mean) * rstd + beta[c];   y = drop(act(u))
 * gamma, beta: fp32 [C], NULL for 1 and 0. mean, rstd: fp32 [N][groups],
 * written by the forward pass (NULL: not kept) and read by the backward.
 * drop: NULL for none. Values are summed in fp64, squared deviations in fp32
 * around the mean of at most 64 values and joined in fp64 around a mean, so
 * rstd has fp32's accuracy whatever the mean is. Deviations of 1.8e19 and more
 * overflow (rstd is 0 then), from 2.3e18 on they may, and the squares of those
 * below 1e-19 lose digits. x - mean itself has to stay in fp32's range.
 *   Backward, from dy (gradient of y) and the forward's x, mean, rstd:
 *   g = drop(dy) * act'(u);  xh = (x - mean) * rstd
 *   dbeta[c] = sum g;  dgamma[c] = sum g * xh          (over H, W, N)
 *   dx = rstd * (gamma g - mean_M(gamma g) - xh * mean_M(gamma g xh))
 * act'(0) is 0 for MQ_ACT_RELU. dgamma, dbeta may be NULL. Sums over pixels
 * and samples are fp64, their partial results kept in fp32. */
typedef struct {
  int32_t h, w, n, c; /* all >= 1 */
  int32_t groups;     /* divides c, else MQ_ERR_SHAPE */
  mq_act act;
  float eps;          /* finite, >= 0, else MQ_ERR_UNSUPPORTED */
} mq_norm;

/* Workspace (device bytes, 16-byte aligned) of the calls below; op 0:
 * forward, 1: backward (the same for fp32 and MX outputs). 0 for invalid
 * arguments. */
size_t mqconv_group_norm_workspace_bytes(const mq_norm* gn, int op);

/* y: fp32 [H][W][N][C], fully overwritten; may be x. */
int mqconv_group_norm(const mq_norm* gn, const float* x, const float* gamma, const float* beta, const mq_drop* drop,
                      float* y, float* mean, float* rstd, void* ws, size_t ws_bytes, void* stream);

/* mqconv_group_norm whose output is MX-quantized, the next convolution's
 * activation quantized once: yq (ACT, (H, W, N, C), any format, bp 1 or 32)
 * receives what mqconv_quantize of the fp32 y would write. */
int mqconv_group_norm_mx(const mq_norm* gn, const float* x, const float* gamma, const float* beta,
                         const mq_drop* drop, mq_mx yq, float* mean, float* rstd, void* ws, size_t ws_bytes,
                         void* stream);

/* dx: fp32 [H][W][N][C], fully overwritten; may be dy or x. gamma, beta and
 * drop as in the forward call. */
int mqconv_group_norm_backward(const mq_norm* gn, const float* dy, const float* x, const float* gamma,
                               const float* beta, const float* mean, const float* rstd, const mq_drop* drop,
                               float* dx, float* dgamma, float* dbeta, void* ws, size_t ws_bytes, void* stream);

/* mqconv_group_norm_backward whose dx is MX-quantized, the gradient that the
 * previous convolution takes: dxq (GRAD, (H, W, N, C), any format, bp 1 or
 * 32) receives what mqconv_quantize of the fp32 dx would write. */
int mqconv_group_norm_backward_mx(const mq_norm* gn, const float* dy, const float* x, const float* gamma,
                                  const float* beta, const float* mean, const float* rstd, const mq_drop* drop,
                                  mq_mx dxq, float* dgamma, float* dbeta, void* ws, size_t ws_bytes, void* stream);

/* ---------------------------------------------------------------------------
 * Replay cache
 * ---------------------------------------------------------------------------
 * A memory of `slots` samples, each an activation (H, W, 1, C) quantized as
 * mqconv_quantize would with line blocks (bp 1), so that a sample's bytes do
 * not depend on the batch it came with:
 *   codes  [slots][H][W][row_bytes]     scales [slots][H][W][ncb]
 * A slot holds at most 2^30 elements; a cache is as large as memory allows
 * (its addresses are 64-bit). `slot` arguments are DEVICE arrays of slot
 * numbers. */
typedef struct {
  void* codes;     /* device, 16-byte aligned */
  uint8_t* scales; /* device, 16-byte aligned */
  mq_elem fmt;
  int32_t slots, h, w, c;
} mq_cache;

/* Bytes of a cache's buffers; 0 for invalid arguments. */
size_t mqconv_cache_codes_bytes(mq_elem fmt, int32_t slots, int32_t h, int32_t w, int32_t c);
size_t mqconv_cache_scales_bytes(int32_t slots, int32_t h, int32_t w, int32_t c);

/* Stores samples n0 .. n0 + count - 1 of x (fp32 [H][W][N][C]) in slots
 * slot[0] .. slot[count - 1]. A slot number outside [0, slots) leaves its
 * sample out; of several samples with one slot the last one is stored.
 * count: 1 .. MQ_CACHE_COUNT_MAX, n0 + count <= n, else MQ_ERR_SHAPE. */
#define MQ_CACHE_COUNT_MAX 4096
int mqconv_cache_write(mq_cache cache, const float* x, int32_t n, int32_t n0, int32_t count, const int32_t* slot,
                       void* stream);

/* Writes the values of slots slot[0] .. slot[count - 1] to samples n0 .. n0 +
 * count - 1 of x (fp32 [H][W][N][C]; the other samples stay as they are, so
 * a batch can be filled from the cache and elsewhere). A slot number outside
 * [0, slots) reads as zeros; a block with scale byte 0xFF as NaN. */
int mqconv_cache_read(mq_cache cache, const int32_t* slot, int32_t count, float* x, int32_t n, int32_t n0,
                      void* stream);

/* mqconv_cache_read of slots slot[0] .. slot[N - 1] into a packed activation
 * xq (ACT, (H, W, N, C), any format, bp 1 or 32): exactly what
 * mqconv_quantize of the fp32 values would write, so a stored sample's codes
 * and scales come back unchanged with bp 1 and the cache's format, and are
 * quantized again for other formats or squares. */
int mqconv_cache_read_mx(mq_cache cache, const int32_t* slot, mq_mx xq, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MQCONV_BLOCK_H */
