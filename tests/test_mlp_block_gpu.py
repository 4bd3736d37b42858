"""The example block against the same block in 64 bits, and its training loop."""

from __future__ import annotations

import importlib.util
import os

import numpy as np
import pytest

import mlp_ref as ref

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("mlp_block", os.path.join(ROOT, "examples", "mlp_block.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def np64(t):
    return t.detach().double().cpu().numpy()


def off(got, want):
    return np.linalg.norm(np64(got) - want) / np.linalg.norm(want)


# Every tensor that leaves an operator in BF16 is off by at most 2^-8 of each element, so by 2^-8 of its
# norm; products with random matrices and the slopes (|act'| <= 1.13) carry such an error on with a factor
# near 1, and 2 allows for it. `roundings` is how many lie on the way to the result.
def close(got, want, roundings):
    assert off(got, want) <= 2 * roundings * 2.0 ** -8


@pytest.mark.parametrize("m, rows, width, hidden, act", [(200, 256, 160, 416, "gelu"), (512, 512, 512, 1024, "silu"),
                                                         (24, 64, 320, 640, "gelu_tanh"), (1, 8, 256, 512, "relu")])
def test_block_against_64_bits(example, m, rows, width, hidden, act):
    import torch

    import blas3_tensor_core_gb300 as bm
    torch.manual_seed(m)
    block = example.MlpBlock(rows, width, hidden, act)
    for v in (block.b1, block.b2, block.beta):
        v.normal_(0.0, 0.3)
    block.gamma.normal_(1.0, 0.2)
    x = torch.randn(m, width, device="cuda").bfloat16()
    dy = torch.randn(m, width, device="cuda").bfloat16()
    y = block.forward(x)
    z_kept = bm.act_mxfp8(block._checkpoint, torch.empty(m, hidden, device="cuda"))
    dx = block.backward(dy)
    served = block.forward(x, train=False)

    X, D, W1, W2, g = (np64(t) for t in (x, dy, block.w1, block.w2, block.gamma))
    mean, r = X.mean(axis=1, keepdims=True), 1.0 / np.sqrt(X.var(axis=1, keepdims=True) + 1e-5)
    xh = (X - mean) * r
    u = xh * g + np64(block.beta)
    z = u @ W1.T + np64(block.b1)
    mlp = ref.act(z, act) @ W2.T + np64(block.b2)
    close(y - x, mlp, 4 + np.linalg.norm(X) / np.linalg.norm(mlp))     # (y and y - x: two of y's own size)
    assert torch.equal(served, y) or off(served, np64(y)) <= 2 * 2.0 ** -8
    # the checkpoint: codes within 2^-4 of z, or of a group's largest value over 2^15 or so; z's own error beside it
    assert off(z_kept, z) <= 2.0 ** -4 + 2 * 2.0 ** -8
    # backward, from the 8-bit values that were kept
    zk = np64(z_kept)
    h, dz = ref.act(zk, act), (D @ W2) * ref.slope(zk, act)
    du = dz @ W1
    v = du * g
    want = r * (v - v.mean(axis=1, keepdims=True) - xh * (v * xh).mean(axis=1, keepdims=True)) + D
    close(block.db2, D.sum(axis=0), 1)
    close(block.db1, dz.sum(axis=0), 1)
    close(block.dw2, D.T @ h, 2)
    close(block.dw1, dz.T @ u, 3)
    close(block.dgamma, (du * xh).sum(axis=0), 2)
    close(block.dbeta, du.sum(axis=0), 2)
    close(dx, want, 4)


def test_training_lowers_the_loss(example, capsys):
    losses = example.main(["--rows", "256", "--width", "256", "--hidden", "512", "--steps", "12", "--rate", "0.05"])
    assert losses[-1] < 0.5 * losses[0]
    assert "one token" in capsys.readouterr().out
