"""The gated example block against the same block in 64 bits: its output, its gradients, its update, and that it
runs."""

from __future__ import annotations

import importlib.util
import os

import numpy as np
import pytest

import gated_ref
import mlp_ref as ref

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("gated_mlp", os.path.join(ROOT, "examples", "gated_mlp.py"))
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


@pytest.mark.parametrize("m, rows, width, hidden, act", [(200, 256, 160, 416, "silu"), (512, 512, 512, 1024, "gelu"),
                                                         (24, 64, 320, 640, "gelu_tanh"), (1, 8, 256, 512, "relu")])
def test_block_against_64_bits(example, m, rows, width, hidden, act):
    import torch
    torch.manual_seed(m)
    block = example.GatedMlp(rows, width, hidden, act)
    block.beta.normal_(0.0, 0.3)
    block.gamma.normal_(1.0, 0.2)
    x = torch.randn(m, width, device="cuda").bfloat16()
    dy = torch.randn(m, width, device="cuda").bfloat16()
    y = block.forward(x)
    G, U = np64(block._both[:m, :hidden]), np64(block._both[:m, hidden:])
    served = block.forward(x[:1], train=False)      # (between a training forward and its backward)
    dx = block.backward(dy)

    X, D, g = np64(x), np64(dy), np64(block.gamma)
    Wg, Wu, Wd = np64(block.w_in[:hidden]), np64(block.w_in[hidden:]), np64(block.w_out)
    mean, r = X.mean(axis=1, keepdims=True), 1.0 / np.sqrt(X.var(axis=1, keepdims=True) + 1e-5)
    xh = (X - mean) * r
    n = xh * g + np64(block.beta)
    gate, up = n @ Wg.T, n @ Wu.T
    mlp = (ref.act(gate, act) * up) @ Wd.T
    close(y - x, mlp, 5 + np.linalg.norm(X) / np.linalg.norm(mlp))     # (y and y - x: two of y's own size)
    assert off(served, np64(y[:1])) <= 2 * 2.0 ** -8
    assert np.linalg.norm(G - gate) <= 4 * 2.0 ** -8 * np.linalg.norm(gate)
    assert np.linalg.norm(U - up) <= 4 * 2.0 ** -8 * np.linalg.norm(up)
    # backward, from the values that were kept
    dh = D @ Wd
    dg, du, h = dh * U * ref.slope(G, act), dh * ref.act(G, act), ref.act(G, act) * U
    dn = dg @ Wg + du @ Wu
    v = dn * g
    want = r * (v - v.mean(axis=1, keepdims=True) - xh * (v * xh).mean(axis=1, keepdims=True)) + D
    close(block.dw_out, D.T @ h, 2)
    close(block.dw_in, np.concatenate([dg.T @ n, du.T @ n]), 3)
    close(block.dgamma, (dn * xh).sum(axis=0), 2)
    close(block.dbeta, dn.sum(axis=0), 2)
    close(dx, want, 4)
    with pytest.raises(RuntimeError):
        block.backward(dy)

    # the update: each projection by its own averaged gradient made orthogonal
    before = [np64(w) for w in (block.w_in[:hidden], block.w_in[hidden:], block.w_out)]
    gradients = [np64(w) for w in (block.dw_in[:hidden], block.dw_in[hidden:], block.dw_out)]
    block.update(0.02, decay=0.1)
    for w, old, grad in zip((block.w_in[:hidden], block.w_in[hidden:], block.w_out), before, gradients):
        steps = [gated_ref.STEP] * 5
        step = 0.02 * 0.2 * max(w.shape) ** 0.5
        exact, model = gated_ref.newton_schulz(grad, steps), gated_ref.rounded_steps(grad, steps)
        want = (1 - 0.02 * 0.1) * old - step * exact
        limit = 2.0 ** -8 * np.linalg.norm(want) + step * (2 * np.linalg.norm(model - exact) + 1e-4 * np.linalg.norm(exact))
        assert np.linalg.norm(np64(w) - want) <= limit


def test_it_trains_and_serves(example, capsys):
    losses = example.main(["--rows", "256", "--width", "256", "--hidden", "512", "--steps", "4"])
    assert len(losses) == 4 and np.isfinite(losses).all()
    assert "one token" in capsys.readouterr().out


@pytest.mark.parametrize("act", ["gelu", "gelu_tanh", "silu"])
def test_gradients_against_differences(act):
    """The block's formulas above, by central differences of sum(y dy) in 64 bits at h = 1e-5: third derivatives
    below 10 of the sums' size, and rounding 1e-16 / h of it."""
    rng = np.random.default_rng(5)
    n, Wg, Wu, Wd, D = (rng.normal(size=s) for s in ((6, 8), (10, 8), (10, 8), (8, 10), (6, 8)))

    def loss(n, Wg, Wu, Wd):
        return (((ref.act(n @ Wg.T, act) * (n @ Wu.T)) @ Wd.T) * D).sum()

    G, U, dh = n @ Wg.T, n @ Wu.T, D @ Wd
    dg, du, h = dh * U * ref.slope(G, act), dh * ref.act(G, act), ref.act(G, act) * U
    args, grads = [n, Wg, Wu, Wd], [dg @ Wg + du @ Wu, dg.T @ n, du.T @ n, D.T @ h]
    for k, want in enumerate(grads):
        d = rng.normal(size=want.shape)
        d /= np.linalg.norm(d)
        up, down = [list(args) for _ in range(2)]
        up[k], down[k] = args[k] + 1e-5 * d, args[k] - 1e-5 * d
        assert abs((loss(*up) - loss(*down)) / 2e-5 - (want * d).sum()) <= 1e-6 * (1 + np.linalg.norm(want))
