"""A residual block trained in the two-level 4-bit format.

The block adds a 3x3 convolution of its layer-normed input to that input. One
training step:
  1. layer norm over the channels (mqconv_layer_norm), then the convolution's
     two operands as two-level E2M1 codes (NvfpTensor.quantize);
  2. the product of the codes (mqconv_nvfp_forward), added to the input;
  3. backwards, the gradient is quantized once for both products
     (mqconv_nvfp_backward_weight, mqconv_nvfp_backward_data), and the norm's
     backward pass (mqconv_layer_norm_backward) adds the skip path's gradient;
  4. the weight moves along its orthogonalised momentum (mqconv_muon_update),
     gamma and beta by plain descent.
The inputs are random and the target is what a block of other weights makes of
them. The fp32 weight is kept beside its codes and quantized again every step.

  python examples/two_level_block.py [--steps 40] [--batch 32] [--size 20] [--channels 64]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import microscaling_quantized_convolution_mxq_amd as mq  # noqa: E402
from microscaling_quantized_convolution_mxq_amd.workloads import ConvShape  # noqa: E402


class Block:
    """Parameters, descriptors and buffers of a block for batches of one size."""

    def __init__(self, n: int, size: int, c: int, rate: float = 0.05, seed: int = 1):
        self.shape = s = ConvShape(n, c, size, size, c)
        act, weight = (size, size, n, c), (c, 3, 3, c)
        g = torch.Generator(device="cuda").manual_seed(seed)
        normal = lambda *d: torch.randn(*d, generator=g, device="cuda")  # noqa: E731
        f32 = lambda *d: torch.empty(*d, device="cuda")  # noqa: E731
        self.w = normal(*weight) * (2 / (9 * c)) ** 0.5
        self.gamma, self.beta = 1 + 0.1 * normal(c), 0.1 * normal(c)
        self.momentum = torch.zeros_like(self.w)
        self.norm = mq.mq_layer_norm(*act)
        self.muon = mq.mq_muon(rate, momentum=0.9, scale=mq.MUON_SCALE_ASPECT)
        self.hq = mq.NvfpTensor.empty(mq.ROLE_ACT, mq.E2M1, act)
        self.wq = mq.NvfpTensor.empty(mq.ROLE_WEIGHT, mq.E2M1, weight)
        self.gq = mq.NvfpTensor.empty(mq.ROLE_GRAD, mq.E2M1, act)
        self.mean, self.rstd = f32(*act[:3]), f32(*act[:3])
        self.h, self.y, self.dh, self.dx = f32(*act), f32(*act), f32(*act), f32(*act)
        self.dw, self.dgamma, self.dbeta = f32(*weight), f32(c), f32(c)
        need = [mq.mqconv_nvfp_gemm_workspace_bytes(s, op, mq.E2M1, mq.E2M1) for op in (mq.OP_FWD, mq.OP_DGRAD, mq.OP_WGRAD)]
        need += [mq.mqconv_nvfp_workspace_bytes(), mq.mqconv_layer_norm_workspace_bytes(self.norm, mq.NORM_BWD),
                 mq.mqconv_orthogonalize_workspace_bytes([weight])]
        self.ws = torch.empty(max(need), dtype=torch.uint8, device="cuda")  # the calls follow one another

    def forward(self, x):
        mq.mqconv_layer_norm(self.norm, x, self.gamma, self.beta, self.h, self.mean, self.rstd)
        self.hq.quantize(self.h, self.ws)
        self.wq.quantize(self.w, self.ws)
        mq.mqconv_nvfp_forward(self.shape, self.hq, self.wq, self.y, self.ws)
        return self.y.add_(x)

    def backward(self, x, dy):
        self.gq.quantize(dy, self.ws)
        mq.mqconv_nvfp_backward_weight(self.shape, self.gq, self.hq, self.dw, self.ws)
        mq.mqconv_nvfp_backward_data(self.shape, self.gq, self.wq, self.dh, self.ws)
        mq.mqconv_layer_norm_backward(self.norm, self.dh, x, self.gamma, self.mean, self.rstd, self.dx, self.dgamma, self.dbeta,
                                      self.ws, dskip=dy)
        return self.dx

    def step(self, rate: float = 0.05):
        mq.mqconv_muon_update(self.muon, [self.dw], [self.momentum], [self.w], self.ws)
        self.gamma.sub_(self.dgamma, alpha=rate)
        self.beta.sub_(self.dbeta, alpha=rate)


def train(steps: int, n: int, size: int, c: int, seed: int = 1):
    """Losses of `steps` steps."""
    g = torch.Generator(device="cuda").manual_seed(seed + 100)
    block, teacher = Block(n, size, c, seed=seed), Block(n, size, c, seed=seed + 1)
    losses = []
    for _ in range(steps):
        x = torch.randn(size, size, n, c, generator=g, device="cuda")
        diff = block.forward(x) - teacher.forward(x)
        losses.append(diff.square().mean())
        block.backward(x, diff * (2 / diff.numel()))
        block.step()
    return [float(v) for v in losses]


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--steps", type=int, default=40)
    ap.add_argument("--batch", type=int, default=32)
    ap.add_argument("--size", type=int, default=20)
    ap.add_argument("--channels", type=int, default=64)
    a = ap.parse_args()
    for k, v in enumerate(train(a.steps, a.batch, a.size, a.channels)):
        if k % 5 == 0 or k == a.steps - 1:
            print(f"step {k:3d}  loss {v:.4f}", flush=True)


if __name__ == "__main__":
    main()
