"""A latent-replay training step on quantized tensors.

A head (group norm with SiLU and dropout, then a 3x3 convolution) is trained
on batches that mix new latents with replayed ones:
  1. the new latents are stored in a replay cache as 4-bit codes
     (mqconv_cache_write), and older samples read back behind them in the
     batch (mqconv_cache_read);
  2. group norm, SiLU and dropout write the batch straight as the
     convolution's quantized activation (mqconv_group_norm_mx);
  3. the convolution runs on the codes (mqconv_forward);
  4. backwards, the loss gradient is quantized once for both products
     (mqconv_backward_weight, mqconv_backward_data), and the norm's backward
     pass (mqconv_group_norm_backward) makes its dropout mask again and gives
     the gradients of gamma and beta, and of the latents as MX codes for
     whatever convolution made them (mqconv_group_norm_backward_mx).
The latents are random and the target is what a head of other weights makes of
them without dropout, so the loss has somewhere to fall.

  python examples/latent_replay.py [--steps 40] [--batch 64] [--size 20] [--channels 256]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import microscaling_quantized_convolution_mxq_amd as mq  # noqa: E402
from microscaling_quantized_convolution_mxq_amd.workloads import WORKLOADS, ConvShape  # noqa: E402


class Head:
    """Parameters, plans and buffers of the trained head for batches of one size."""

    def __init__(self, n: int, size: int, c: int, cout: int, groups: int = 32, p: float = 0.1, seed: int = 1):
        wl = WORKLOADS["c4"]  # 4-bit latents, E4M3 weights, E5M2 gradients
        self.fx, self.fw, self.fdy = wl.fx, wl.fw, wl.fdy
        self.shape = s = ConvShape(n, c, size, size, cout)
        g = torch.Generator(device="cuda").manual_seed(seed)
        normal = lambda *d: torch.randn(*d, generator=g, device="cuda")  # noqa: E731
        self.w = normal(cout, 3, 3, c) * (2 / (9 * c)) ** 0.5
        self.gamma, self.beta = 1 + 0.1 * normal(c), 0.1 * normal(c)
        self.norm = mq.mq_norm(size, size, n, c, groups, mq.ACT_SILU)
        self.step = torch.zeros(1, dtype=torch.int64, device="cuda")  # moves the dropout's seed
        self.drop = mq.mq_drop(p, seed, self.step)

        f32 = lambda *d: torch.empty(*d, device="cuda")  # noqa: E731
        act = (size, size, n, c)
        self.hq = mq.MxTensor.empty(mq.ROLE_ACT, self.fx, 32, act)
        self.wq = mq.MxTensor.empty(mq.ROLE_WEIGHT, self.fw, 32, (cout, 3, 3, c))
        self.gq = mq.MxTensor.empty(mq.ROLE_GRAD, self.fdy, 32, (size, size, n, cout))
        self.dxq = mq.MxTensor.empty(mq.ROLE_GRAD, self.fdy, 32, act)
        self.mean, self.rstd = f32(n, groups), f32(n, groups)
        self.y, self.dh, self.dw = f32(size, size, n, cout), f32(*act), f32(cout, 3, 3, c)
        self.dgamma, self.dbeta = f32(c), f32(c)
        self.params = [self.w, self.gamma, self.beta]
        for param, grad in zip(self.params, (self.dw, self.dgamma, self.dbeta)):
            param.grad = grad  # the calls write the gradients where the optimizer reads them
        need = [mq.mqconv_group_norm_workspace_bytes(self.norm, k) for k in (mq.NORM_FWD, mq.NORM_BWD)]
        need += [mq.mqconv_workspace_bytes(s, mq.OP_DGRAD, self.fdy, self.fw),
                 mq.mqconv_workspace_bytes(s, mq.OP_WGRAD, self.fdy, self.fx)]
        self.ws = torch.empty(max(need), dtype=torch.uint8, device="cuda")  # the calls follow one another

    def forward(self, x, dropout: bool = True):
        mq.mqconv_group_norm_mx(self.norm, x, self.gamma, self.beta, self.hq, self.mean, self.rstd, self.ws,
                                drop=self.drop if dropout else None)
        mq.mqconv_quantize(self.w, self.wq)
        mq.mqconv_forward(self.shape, self.hq, self.wq, self.y, self.ws)
        return self.y

    def backward(self, x, dy):
        mq.mqconv_quantize(dy, self.gq)
        mq.mqconv_backward_weight(self.shape, self.gq, self.hq, self.dw, self.ws)
        mq.mqconv_backward_data(self.shape, self.gq, self.wq, self.dh, self.ws)
        mq.mqconv_group_norm_backward_mx(self.norm, self.dh, x, self.gamma, self.beta, self.mean, self.rstd, self.dxq,
                                         self.dgamma, self.dbeta, self.ws, drop=self.drop)


def train(steps: int, n: int, size: int, c: int, cout: int, slots: int = 512, rate: float = 0.64, seed: int = 1):
    """Losses of `steps` steps on batches of n / 8 new and the rest replayed latents."""
    g = torch.Generator(device="cuda").manual_seed(seed + 100)
    cache = mq.MxCache.empty(mq.E2M1, slots, size, size, c)
    head, teacher = Head(n, size, c, cout, seed=seed), Head(n, size, c, cout, seed=seed + 1)
    # not plain descent: the activations share a mean, which alone would hold its rate below 1 / (9 c);
    # steps shrink with the number of channels that a weight's step is summed over
    adam = torch.optim.Adam(head.params, lr=rate / c, betas=(0.9, 0.99))
    x = torch.empty(size, size, n, c, device="cuda")
    new = max(1, n // 8)
    latents = lambda k: torch.randn(size, size, k, c, generator=g, device="cuda").relu_()  # noqa: E731
    filled = 0
    while filled < min(slots, n):  # a first memory to replay from
        k = min(n, slots - filled)
        mq.mqconv_cache_write(cache, latents(k), torch.arange(filled, filled + k, dtype=torch.int32, device="cuda"))
        filled += k
    losses = []
    for step in range(steps):
        fresh = latents(new)
        to = (filled + torch.arange(new, dtype=torch.int32, device="cuda")) % slots  # the oldest give way
        mq.mqconv_cache_write(cache, fresh, to)
        old = torch.randint(0, min(filled, slots), (n - new,), generator=g, device="cuda", dtype=torch.int32)
        filled += new
        x[:, :, :new] = fresh
        mq.mqconv_cache_read(cache, old, x, n0=new)
        diff = head.forward(x) - teacher.forward(x, dropout=False)
        losses.append(diff.square().mean())
        head.backward(x, diff * (2 / (size * size * n)))
        adam.step()
        head.step += 1
    return [float(v) for v in losses]


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--steps", type=int, default=40)
    ap.add_argument("--batch", type=int, default=64)
    ap.add_argument("--size", type=int, default=20)
    ap.add_argument("--channels", type=int, default=256)
    a = ap.parse_args()
    for k, v in enumerate(train(a.steps, a.batch, a.size, a.channels, a.channels)):
        if k % 5 == 0 or k == a.steps - 1:
            print(f"step {k:3d}  loss {v:.4f}", flush=True)


if __name__ == "__main__":
    main()
