"""A transformer's MLP block, trained and served with the library's operators.

    y = x + act(layernorm(x) W1^T + b1) W2^T + b2

Forward takes three launches: layer norm, the first product with its bias and activation, the
second with its bias and the residual. For training the first product also keeps its
pre-activation in 8 bits; the activation itself is not kept but computed again from those in the
backward pass, so a row costs 2 h bytes (codes and a BF16 buffer that every block can share)
rather than 4 h.

    python examples/mlp_block.py [--rows 4096] [--width 4096] [--hidden 16384] [--steps 20]

trains one block on synthetic data (its output towards a fixed target), prints the loss and the
time of a step, and then the time of the forward pass for single tokens.
"""

from __future__ import annotations

import argparse
import os
import sys

import torch

if __name__ == "__main__":
    sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import blas3_tensor_core_gb300 as bm


class MlpBlock:
    """Parameters (BF16 weights, FP32 vectors), their gradients, and the buffers of up to `rows` rows.

    width and hidden are multiples of 32. Calls run on the current stream, and one block's
    calls must not overlap.
    """

    def __init__(self, rows, width, hidden, act="gelu", device="cuda"):
        if width % 32 or hidden % 32:
            raise ValueError("width and hidden must be multiples of 32")
        bf16 = dict(dtype=torch.bfloat16, device=device)
        f32 = dict(dtype=torch.float32, device=device)
        self.rows, self.width, self.hidden, self.act = rows, width, hidden, act
        self.w1 = (torch.randn(hidden, width, **f32) / width ** 0.5).bfloat16()
        self.w2 = (torch.randn(width, hidden, **f32) / hidden ** 0.5).bfloat16()
        self.b1, self.b2 = torch.zeros(hidden, **f32), torch.zeros(width, **f32)
        self.gamma, self.beta = torch.ones(width, **f32), torch.zeros(width, **f32)
        self.dw1, self.dw2 = torch.empty_like(self.w1), torch.empty_like(self.w2)
        self.db1, self.db2 = torch.empty_like(self.b1), torch.empty_like(self.b2)
        self.dgamma, self.dbeta = torch.empty_like(self.gamma), torch.empty_like(self.beta)
        self._normed = torch.empty(rows, width, **bf16)      # kept for the backward pass
        self._mean, self._rstd = torch.empty(rows, **f32), torch.empty(rows, **f32)
        self._wide = torch.empty(rows, hidden, **bf16)       # scratch: the activation
        self._grad = torch.empty(rows, hidden, **bf16)       # scratch: the pre-activation's gradient
        self._narrow = torch.empty(rows, width, **bf16)      # scratch: the normed rows' gradient, or served normed rows
        self._ones = torch.ones(1, (rows + 7) // 8 * 8, **bf16)
        needed = max(bm.bm_gemm_bf16_dact_workspace_size(rows, hidden, width, 1),
                     bm.bm_layernorm_backward_workspace_size(rows, width),
                     bm.bm_gemm_bf16_bias_act_workspace_size(rows, hidden, width),
                     bm.bm_gemm_bf16_bias_act_workspace_size(rows, width, hidden),
                     bm.workspace_size(hidden, width, rows), bm.workspace_size(width, hidden, rows),
                     bm.workspace_size(rows, width, hidden), bm.workspace_size(1, width, rows), 256)
        self._workspace = torch.empty(needed, dtype=torch.uint8, device=device)
        self._x = self._checkpoint = None

    def forward(self, x, train=True):
        """y for x [m, width], m <= rows; with `train` what `backward` needs is kept (x itself by reference);
        without, what an earlier training forward kept stays."""
        m, ws = x.shape[0], self._workspace
        normed, wide, y = (self._normed if train else self._narrow)[:m], self._wide[:m], torch.empty_like(x)
        stats = dict(mean=self._mean[:m], rstd=self._rstd[:m]) if train else {}
        bm.layernorm(x, self.gamma, self.beta, normed, **stats)
        if train:
            if self._checkpoint is None or self._checkpoint[0].shape[0] != m:
                self._checkpoint = bm.mxfp8_empty(m, self.hidden, device=x.device)
            self._x = x
        bm.gemm_bias_act(normed, self.w1, wide, bias=self.b1, act=self.act, transB=True, workspace=ws,
                         checkpoint=self._checkpoint if train else None)
        bm.gemm_bias_act(wide, self.w2, y, bias=self.b2, residual=x, transB=True, workspace=ws)
        return y

    def backward(self, dy):
        """dx for the last training forward's dy; the parameters' gradients go to dw1, db1, ..."""
        m, ws, x = dy.shape[0], self._workspace, self._x
        wide, grad, narrow, dx = self._wide[:m], self._grad[:m], self._narrow[:m], torch.empty_like(x)
        bm.gemm(self._ones[:, :m], dy, self.db2.view(1, -1), workspace=ws)
        bm.gemm_dact(dy, self.w2, grad, self._checkpoint, act=self.act, dbias=self.db1, workspace=ws)
        bm.act_mxfp8(self._checkpoint, wide, act=self.act)
        bm.gemm(dy, wide, self.dw2, transA=True, workspace=ws)
        bm.gemm(grad, self._normed[:m], self.dw1, transA=True, workspace=ws)
        bm.gemm(grad, self.w1, narrow, workspace=ws)
        bm.layernorm_backward(narrow, x, self.gamma, self._mean[:m], self._rstd[:m], dx, self.dgamma, self.dbeta,
                              dres=dy, workspace=ws)
        return dx

    def update(self, rate):
        """One step of plain gradient descent."""
        for p, g in ((self.w1, self.dw1), (self.w2, self.dw2), (self.b1, self.db1), (self.b2, self.db2),
                     (self.gamma, self.dgamma), (self.beta, self.dbeta)):
            p.add_(g, alpha=-rate)


def train(block, x, target, steps, rate):
    """Losses (mean square error) of `steps` steps, and the time of one in ms."""
    losses, times = [], []
    for _ in range(steps):
        start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        start.record()
        dy = (block.forward(x) - target).mul_(2.0 / x.numel() ** 0.5)
        block.backward(dy)
        block.update(rate)
        end.record()
        losses.append((dy.float().square().sum() / 4).item())
        times.append(start.elapsed_time(end))
    return losses, sorted(times)[len(times) // 2]


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--rows", type=int, default=4096)
    ap.add_argument("--width", type=int, default=4096)
    ap.add_argument("--hidden", type=int, default=16384)
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--rate", type=float, default=0.01)
    args = ap.parse_args(argv)
    torch.manual_seed(0)
    block = MlpBlock(args.rows, args.width, args.hidden)
    x = torch.randn(args.rows, args.width, device="cuda").bfloat16()
    target = x + 0.5 * torch.randn(1, args.width, device="cuda").bfloat16()
    losses, ms = train(block, x, target, args.steps, args.rate)
    print(f"{args.rows} x {args.width}, hidden {args.hidden}: loss {losses[0]:.4f} -> {losses[-1]:.4f}, "
          f"{ms:.3f} ms a step")

    token = x[:1]
    for _ in range(3):
        block.forward(token, train=False)
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    for _ in range(100):
        block.forward(token, train=False)
    end.record()
    end.synchronize()
    print(f"one token: {10 * start.elapsed_time(end):.1f} us a forward pass")
    return losses


if __name__ == "__main__":
    main()
