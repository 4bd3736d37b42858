"""Element offsets past 32 bits in a gated MLP's products and in the orthogonalised update."""

import numpy as np
import pytest

import gated_ref
from gpu_helpers import check_no_device_error, torch
from test_gated_ops_gpu import bf16_tol, gpu_bf16
from test_mlp_ops_gpu import _built, assert_close, bm, np64  # noqa: F401

pytestmark = pytest.mark.gpu


def room(nbytes):
    free, _ = torch().cuda.mem_get_info()
    if free < nbytes + (2 << 30):
        pytest.skip(f"needs {nbytes >> 30} GB of device memory")


def test_products_past_32_bits(bm):
    """m n = 2.3e9 elements: rows at both ends and in the middle against 64 bits."""
    t = torch()
    m, n, k = 143000, 16088, 64
    room(8 * m * n)
    gen = t.Generator(device="cuda").manual_seed(1)

    def normal(rows, cols, std):
        return (t.randn(rows, cols, generator=gen, device="cuda") * std).bfloat16()

    x, wg, wu, wd = normal(m, k, 1.0), normal(n, k, k ** -0.5), normal(n, k, k ** -0.5), normal(k, n, k ** -0.5)
    h = t.empty(m, n, **gpu_bf16())
    both = t.empty(m, 2 * n, **gpu_bf16())
    rows = t.tensor([0, 1, 127, 66750, m // 2, m - 129, m - 2, m - 1], device="cuda")
    bm.gemm_glu(x, wg, wu, h, gate=both[:, :n], up=both[:, n:], transB=True)
    check_no_device_error()
    a, bg, bu = np64(x[rows]), np64(wg).T, np64(wu).T
    want, err = gated_ref.glu(a, bg, bu, k, 1.0, "silu")
    kept = np64(both[rows])
    for got, w, e in zip((np64(h[rows]), kept[:, :n], kept[:, n:]), want, err):
        assert_close(got, w, bf16_tol(w, e), "forward")
    bm.gemm_dglu(x, wd, both[:, :n], both[:, n:], both[:, :n], both[:, n:], hidden=h)
    check_no_device_error()
    want, err = gated_ref.dglu(a, np64(wd), k, 1.0, kept[:, :n], kept[:, n:], "silu")
    after = np64(both[rows])
    for got, w, e in zip((after[:, :n], after[:, n:], np64(h[rows])), want, err):
        assert_close(got, w, bf16_tol(w, e), "backward")


@pytest.mark.parametrize("tall", [True, False])
def test_update_past_32_bits(bm, tall):
    """2.2e9 elements, all zero but a block at the far end: the block comes out as it does alone (to a rounding: its
    sums are added in other groups), and zeros stay zeros."""
    t = torch()
    shape, block = ((110000, 20000), (300, 256)) if tall else ((20000, 110000), (256, 300))
    size = bm.orthogonalize_workspace_size(*shape)
    room(size + 4 * shape[0] * shape[1])
    x = t.zeros(*shape, **gpu_bf16())
    gen = t.Generator(device="cuda").manual_seed(2)
    x[-block[0]:, -block[1]:] = t.randn(*block, generator=gen, device="cuda").bfloat16()
    c = t.full(shape, float("nan"), **gpu_bf16())
    ws = t.empty(size, dtype=t.uint8, device="cuda")
    bm.orthogonalize(x, c, steps=2, workspace=ws)
    check_no_device_error()
    got = np64(c[-block[0]:, -block[1]:])
    given = np64(x[-block[0]:, -block[1]:])
    steps = [gated_ref.STEP] * 2
    want, model = gated_ref.newton_schulz(given, steps), gated_ref.rounded_steps(given, steps)
    norm = np.linalg.norm(want)
    assert np.linalg.norm(got - want) <= (2.0 ** -8 + 1e-4) * norm + 2 * np.linalg.norm(model - want)
    c[-block[0]:, -block[1]:] = 0
    assert not c.any()
