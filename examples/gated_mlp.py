"""A transformer's gated MLP block, trained and served with the library's operators.

    y = x + (act(n Wg^T) * (n Wu^T)) Wd^T,  n = layernorm(x)

Forward takes three launches: layer norm, both projections with the activation and their
product in one, the down projection with the residual. For training the gate's and the up
projection's results are kept in BF16, side by side in one buffer; the product of the two is
computed again in the backward pass, by the same call that turns the buffer into the gradients
of its two halves. Both weights lie in one matrix, so what is left of the backward pass are
plain products over whole buffers.

The weights are updated as the Muon optimiser does it: by the averaged gradient, made
orthogonal by Newton-Schulz products.

    python examples/gated_mlp.py [--rows 4096] [--width 4096] [--hidden 16384] [--steps 20]

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


class GatedMlp:
    """Parameters (BF16 weights, FP32 vectors), their gradients and averages, and the buffers of up to `rows` rows.

    width and hidden are multiples of 32. Calls run on the current stream, and one block's
    calls must not overlap.
    """

    def __init__(self, rows, width, hidden, act="silu", device="cuda"):
        if width % 32 or hidden % 32:
            raise ValueError("width and hidden must be multiples of 32")
        bf16 = dict(dtype=torch.bfloat16, device=device)
        f32 = dict(dtype=torch.float32, device=device)
        self.rows, self.width, self.hidden, self.act = rows, width, hidden, act
        self.w_in = (torch.randn(2 * hidden, width, **f32) / width ** 0.5).bfloat16()  # the gate's rows, then the up projection's
        self.w_out = (torch.randn(width, hidden, **f32) / hidden ** 0.5).bfloat16()
        self.gamma, self.beta = torch.ones(width, **f32), torch.zeros(width, **f32)
        self.dw_in, self.dw_out = torch.empty_like(self.w_in), torch.empty_like(self.w_out)
        self.dgamma, self.dbeta = torch.empty_like(self.gamma), torch.empty_like(self.beta)
        self.averages = [torch.zeros_like(w, dtype=torch.float32) for w in (self.w_in, self.w_out)]
        self._normed = torch.empty(rows, width, **bf16)      # kept for the backward pass
        self._mean, self._rstd = torch.empty(rows, **f32), torch.empty(rows, **f32)
        self._both = torch.empty(rows, 2 * hidden, **bf16)   # kept: gate and up, then their gradients
        self._wide = torch.empty(rows, hidden, **bf16)       # scratch: act(gate) * up
        self._narrow = torch.empty(rows, width, **bf16)      # scratch: the normed rows' gradient, or served normed rows
        needed = max(bm.bm_layernorm_backward_workspace_size(rows, width),
                     bm.bm_gemm_bf16_bias_act_workspace_size(rows, width, hidden),
                     bm.workspace_size(2 * hidden, width, rows), bm.workspace_size(width, hidden, rows),
                     bm.workspace_size(rows, width, 2 * hidden),
                     bm.orthogonalize_workspace_size(hidden, width), bm.orthogonalize_workspace_size(width, hidden))
        self._workspace = torch.empty(needed, dtype=torch.uint8, device=device)
        self._x = None

    def forward(self, x, train=True):
        """y for x [m, width], m <= rows; with `train` what `backward` needs is kept (x itself by reference);
        without, what an earlier training forward kept stays."""
        m, n = x.shape[0], self.hidden
        normed, wide, y = (self._normed if train else self._narrow)[:m], self._wide[:m], torch.empty_like(x)
        stats = dict(mean=self._mean[:m], rstd=self._rstd[:m]) if train else {}
        bm.layernorm(x, self.gamma, self.beta, normed, **stats)
        kept = dict(gate=self._both[:m, :n], up=self._both[:m, n:]) if train else {}
        bm.gemm_glu(normed, self.w_in[:n], self.w_in[n:], wide, act=self.act, transB=True, **kept)
        bm.gemm_bias_act(wide, self.w_out, y, residual=x, transB=True, workspace=self._workspace)
        if train:
            self._x = x
        return y

    def backward(self, dy):
        """dx for the last training forward's dy (once: the kept buffer becomes its gradient); the parameters'
        gradients go to dw_in, dw_out, dgamma, dbeta."""
        if self._x is None:
            raise RuntimeError("backward needs a training forward before it")
        m, n, ws, x = dy.shape[0], self.hidden, self._workspace, self._x
        both, wide, narrow, dx = self._both[:m], self._wide[:m], self._narrow[:m], torch.empty_like(x)
        gate, up = both[:, :n], both[:, n:]
        bm.gemm_dglu(dy, self.w_out, gate, up, gate, up, act=self.act, hidden=wide)
        bm.gemm(dy, wide, self.dw_out, transA=True, workspace=ws)
        bm.gemm(both, self._normed[:m], self.dw_in, transA=True, workspace=ws)
        bm.gemm(both, self.w_in, narrow, workspace=ws)
        bm.layernorm_backward(narrow, x, self.gamma, self._mean[:m], self._rstd[:m], dx, self.dgamma, self.dbeta,
                              dres=dy, workspace=ws)
        self._x = None
        return dx

    def update(self, rate, momentum=0.95, decay=0.0):
        """One step: the weights by their averaged gradients made orthogonal, the vectors by plain descent. Each of
        the three projections is a matrix of its own to the update."""
        n = self.hidden
        for average, gradient in zip(self.averages, (self.dw_in, self.dw_out)):
            average.mul_(momentum).add_(gradient)
        for w, average in ((self.w_in[:n], self.averages[0][:n]), (self.w_in[n:], self.averages[0][n:]),
                           (self.w_out, self.averages[1])):
            size = 0.2 * max(w.shape) ** 0.5
            bm.orthogonalize(average, w, alpha=-rate * size, beta=1.0 - rate * decay, workspace=self._workspace)
        self.gamma.add_(self.dgamma, alpha=-rate)
        self.beta.add_(self.dbeta, alpha=-rate)


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
    block = GatedMlp(args.rows, args.width, args.hidden)
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
