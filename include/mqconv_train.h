/*
 * mqconv_train.h -- C ABI of what a layer needs, beside the calls of mqconv.h
 * and mqconv_block.h, to be trained in the two-level 4-bit format: layer
 * normalization over the channels (forward and backward), the three products
 * of a convolution on two-level codes, and the orthogonalised update of the
 * weights.
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
 * a workgroup's share of dgamma and dbeta is kept in fp32. y is made of mean
 * and rstd as they are kept, rounded to fp32; they and x - mean have to stay in
 * fp32's normal range. A row that holds a NaN or an infinity is NaN; other rows
 * are not touched by it. */
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

/* ---------------------------------------------------------------------------
 * Products of two-level codes
 * ---------------------------------------------------------------------------
 * The three products of a convolution (mqconv.h; a linear layer is a 1 x 1
 * convolution of a 1 x 1 image whose samples are its rows) on operands that
 * mqconv_nvfp_quantize wrote, each quantized once: its blocks of 8 x 8 serve the
 * sums along either of their sides. An element's value is value(q) * B * T;
 * value(q) * B is exact in 16 bits, products are exact, sums fp32 (products
 * below 2^-26 of a sum may be lost in it), and T T' is applied to them. A block
 * with the scale byte 0x7F (NaN) makes every output that it is part of NaN;
 * outputs that pair its values with zero padding alone are left open. */
typedef struct {
  const void* codes;           /* device, 16-byte aligned: the packed layout of the role */
  const uint8_t* block_scales; /* device: E4M3 bytes (mqconv_nvfp_scales_bytes); between dwords some calls copy them */
  const float* tensor_scale;   /* device, 4-byte aligned: one value */
  mq_elem fmt;
  mq_role role;
  int32_t d0, d1, d2, d3;      /* ACT/GRAD: (H, W, N, C); WEIGHT: (Cout, Kh, Kw, Cin) */
} mq_nvfp;

/* Workspace (device bytes, 16-byte aligned); op 0 forward, 1 backward data, 2
 * backward weight, fa/fb the operands' formats in the order of the call. 0 for
 * invalid arguments, and where an operand's rounded-up size (channels to 64;
 * backward weight: samples to 8 instead) is 2^30 - 128 elements or more, which
 * the calls refuse with MQ_ERR_SHAPE. */
size_t mqconv_nvfp_gemm_workspace_bytes(const mq_conv* cv, int op, mq_elem fa, mq_elem fb);

/* Y: fp32 [Ho][Wo][N][Cout], fully overwritten. xq ACT, wq WEIGHT, any formats. */
int mqconv_nvfp_forward(const mq_conv* cv, mq_nvfp xq, mq_nvfp wq, float* y, void* ws, size_t ws_bytes, void* stream);

/* dX: fp32 [H][W][N][Cin], fully overwritten. dyq GRAD, wq WEIGHT. */
int mqconv_nvfp_backward_data(const mq_conv* cv, mq_nvfp dyq, mq_nvfp wq, float* dx, void* ws, size_t ws_bytes,
                              void* stream);

/* dW: fp32 [Cout][Kh][Kw][Cin], fully overwritten. dyq GRAD, xq ACT. */
int mqconv_nvfp_backward_weight(const mq_conv* cv, mq_nvfp dyq, mq_nvfp xq, float* dw, void* ws, size_t ws_bytes,
                                void* stream);

/* ---------------------------------------------------------------------------
 * Orthogonalised weight update (Newton-Schulz steps, as the Muon optimizer's)
 * ---------------------------------------------------------------------------
 * A weight [Cout][Kh][Kw][Cin] is the matrix of `rows` = Cout and `cols` = Kh
 * Kw Cin. With U its gradient or momentum:
 *   X = U / (|U|_F + eps);   steps times:  X <- a X + (b S + c S^2) X,  S = X X^T
 * so a singular value x becomes p(x) = a x + b x^3 + c x^5, step after step,
 * and the singular vectors stay: a few steps bring every singular value near
 * 1 that is not far below the largest. |U|_F and the products' sums are held
 * in 32 bits or more; every factor of a product in two f16 parts, off by 2^-22
 * of itself or by 2^-40 (2^-39 for the factor of a step, a I + b S + c S^2),
 * whichever is more, so results have the accuracy of fp32 products.
 * Parts of U whose share of |U|_F is below 2^-40 may be lost; a NaN or an
 * infinity in U makes its whole result NaN; U = 0 gives 0 (NaN with eps = 0,
 * as the formula does). */
typedef struct {
  int32_t steps; /* 1 .. MQ_NEWTON_STEPS_MAX, else MQ_ERR_UNSUPPORTED */
  float a, b, c; /* finite, and such that |x| < 1.41 and |a + b x^2 + c x^4| < 3.99 wherever the steps lead from
                    x in [0, 1], else MQ_ERR_UNSUPPORTED; (3.4445, -4.7750, 2.0315) is the usual choice */
  float eps;     /* finite, >= 0, else MQ_ERR_UNSUPPORTED */
} mq_newton;
#define MQ_NEWTON_STEPS_MAX 32

/* The optimizer step around it, for gradient g, momentum m and weight w:
 *   m <- momentum * m + g
 *   U  = nesterov ? g + momentum * m : m
 *   w <- (1 - r * decay) * w - r * s * X(U),   r = lr * *rate (lr where rate is NULL)
 * s: 1 (MQ_SCALE_NONE), sqrt(max(1, rows / cols)) (MQ_SCALE_ASPECT) or
 * 0.2 sqrt(max(rows, cols)) (MQ_SCALE_RMS). */
enum { MQ_SCALE_NONE = 0, MQ_SCALE_ASPECT = 1, MQ_SCALE_RMS = 2 };
typedef struct {
  mq_newton newton;
  float lr, momentum, decay; /* finite, else MQ_ERR_UNSUPPORTED */
  int32_t nesterov;          /* 0 or 1 */
  int32_t scale;             /* MQ_SCALE_*, else MQ_ERR_FORMAT */
  const float* rate;         /* device, 4-byte aligned, or NULL: read when the kernel runs, so a captured graph
                                follows a schedule */
} mq_muon;

/* The weights of one call: 1 .. MQ_UPDATE_GROUP_MAX matrices, which share
 * launches. Arrays are HOST arrays, read during the call only. */
#define MQ_UPDATE_GROUP_MAX 32

/* Workspace (device bytes, 16-byte aligned) of the calls below for these
 * matrices; 0 for invalid arguments. A matrix is refused with MQ_ERR_SHAPE
 * where its extents, rounded up to 32, have a product or a smaller one's
 * square of 2^29 - 64 or more. */
size_t mqconv_orthogonalize_workspace_bytes(int32_t count, const int32_t* rows, const int32_t* cols);

/* x[i] (fp32 [rows][cols], fully overwritten) = X(u[i]); x[i] may be u[i],
 * otherwise outputs must not overlap anything. */
int mqconv_orthogonalize(const mq_newton* newton, int32_t count, const int32_t* rows, const int32_t* cols,
                         const float* const* u, float* const* x, void* ws, size_t ws_bytes, void* stream);

/* One optimizer step: m[i] and w[i] are updated from g[i]. Nothing may
 * overlap. */
int mqconv_muon_update(const mq_muon* opt, int32_t count, const int32_t* rows, const int32_t* cols,
                       const float* const* g, float* const* m, float* const* w, void* ws, size_t ws_bytes,
                       void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MQCONV_TRAIN_H */
