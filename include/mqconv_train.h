/*
 * mqconv_train.h -- C ABI of what a layer needs, beside the calls of mqconv.h
 * and mqconv_block.h, to be trained in the two-level 4-bit format: layer
 * normalization over the channels (forward and backward).
 *
 * The conventions of mqconv.h hold: device pointers owned by the caller, work
 * enqueued on `stream`, every argument checked before any HIP call, an
 * mq_status returned, equal inputs giving bit-identical outputs. Descriptors
 * are HOST structs, read during the call only. fp32 tensors are 4-byte aligned;
 * activations and gradients are [H][W][N][C], weights [Cout][Kh][Kw][Cin].
 */
#ifndef MQCONV_TRAIN_H
#define MQCONV_TRAIN_H

#include "mqconv.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---------------------------------------------------------------------------
 * Layer normalization, channels last
 * ---------------------------------------------------------------------------
 * A row is the C channels of one pixel and sample:
 *   s = x + residual (x where residual is NULL)
 *   mean = sum s / C;  rstd = 1 / sqrt(sum (s - mean)^2 / C + eps)
 *   y[c] = gamma[c] * (s[c] - mean) * rstd + beta[c]
 * gamma, beta: fp32 [C], NULL for 1 and 0. sum: fp32 [H][W][N][C], s as the
 * skip path behind the norm takes it; given exactly where residual is (else
 * MQ_ERR_NULL, or MQ_ERR_UNSUPPORTED for a sum of nothing). mean, rstd: fp32
 * [H][W][N], written by the forward pass (NULL: not kept) and read by the
 * backward.
 *   Backward, from dy (gradient of y), the forward's s as x, mean and rstd:
 *   g = gamma dy;  xh = (x - mean) * rstd
 *   dx = rstd * (g - mean_C(g) - xh * mean_C(g xh)) + dskip
 *   dbeta[c] = sum dy;  dgamma[c] = sum dy * xh        (over H, W, N)
 * dskip: the gradient that reaches s on the skip path, or NULL. dx is the
 * gradient of x and of residual. dgamma, dbeta may be NULL. All sums are fp64;
 * a workgroup's share of dgamma and dbeta is kept in fp32. A row that holds a
 * NaN or an infinity is NaN; other rows are not touched by it. */
typedef struct {
  int32_t h, w, n, c; /* all >= 1 */
  float eps;          /* finite, >= 0, else MQ_ERR_UNSUPPORTED */
} mq_layer_norm;

/* Workspace (device bytes, 16-byte aligned) of the calls that take one; op 0:
 * mqconv_layer_norm_mx, 1: backward (fp32 and MX). 0 for invalid arguments. */
size_t mqconv_layer_norm_workspace_bytes(const mq_layer_norm* ln, int op);

/* y: fp32 [H][W][N][C], fully overwritten; y and sum may each be x or
 * residual, but not the same tensor. */
int mqconv_layer_norm(const mq_layer_norm* ln, const float* x, const float* residual, const float* gamma,
                      const float* beta, float* sum, float* y, float* mean, float* rstd, void* stream);

/* mqconv_layer_norm whose output is MX-quantized: yq (ACT, (H, W, N, C), any
 * format, bp 1 or 32) receives what mqconv_quantize of the fp32 y would
 * write. */
int mqconv_layer_norm_mx(const mq_layer_norm* ln, const float* x, const float* residual, const float* gamma,
                         const float* beta, float* sum, mq_mx yq, float* mean, float* rstd, void* ws,
                         size_t ws_bytes, void* stream);

/* dx: fp32 [H][W][N][C], fully overwritten; may be dy, x or dskip. */
int mqconv_layer_norm_backward(const mq_layer_norm* ln, const float* dy, const float* x, const float* gamma,
                               const float* mean, const float* rstd, const float* dskip, float* dx, float* dgamma,
                               float* dbeta, void* ws, size_t ws_bytes, void* stream);

/* mqconv_layer_norm_backward whose dx is MX-quantized: dxq (GRAD, (H, W, N,
 * C), any format, bp 1 or 32) receives what mqconv_quantize of the fp32 dx
 * would write. */
int mqconv_layer_norm_backward_mx(const mq_layer_norm* ln, const float* dy, const float* x, const float* gamma,
                                  const float* mean, const float* rstd, const float* dskip, mq_mx dxq, float* dgamma,
                                  float* dbeta, void* ws, size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MQCONV_TRAIN_H */
