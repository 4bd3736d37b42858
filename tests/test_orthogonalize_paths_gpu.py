"""Forms of the orthogonalised update that its sizes alone do not reach on a whole GB300, and what its documentation
says of its numbers, against the 64-bit form (gated_ref.py)."""

import contextlib

import numpy as np
import pytest

import gated_ref
import mlp_ref as ref
from test_mlp_ops_gpu import _built, assert_close, bm  # noqa: F401
from test_orthogonalize_gpu import momentum, run

pytestmark = pytest.mark.gpu


@contextlib.contextmanager
def largest_cluster(bm, ctas):
    bm.bm_debug_limit_clusters(ctas)
    try:
        yield
    finally:
        bm.bm_debug_limit_clusters(0)


def assert_one_step(bm, size, seed, coeffs=(gated_ref.STEP,), alpha=-0.7, beta=0.9, **kw):
    """One step element by element, as test_orthogonalize_gpu.py holds it."""
    coeffs = list(coeffs)
    rng = np.random.default_rng(seed)
    got, x, before = run(bm, 3e-5 * momentum(rng, *size, "gauss"), "f32", 1, coeffs, alpha, beta, **kw)
    want = alpha * gated_ref.newton_schulz(x, coeffs)
    err = np.abs(alpha) * gated_ref.one_step_bound(x, coeffs)
    if beta != 0.0:
        want = want + beta * before
        err = err + 2 * ref.U32 * (np.abs(want) + np.abs(beta * before))
    assert_close(got, want, 1.01 * (err + ref.rounding(want, True)), f"{size}")


@pytest.mark.parametrize("limit", [1, 2, 4, 8])
@pytest.mark.parametrize("size", [(128, 200), (256, 100), (64, 300), (500, 128), (128, 513), (77, 700), (850, 61),
                                  (128, 1024), (128, 1025), (2000, 96)], ids=lambda s: f"{s[0]}x{s[1]}")
def test_where_clusters_have_no_room(bm, size, limit):
    """A CTA per 128 lines of the longer side, 2 to 16 of them: they meet through the workspace where a cluster of them
    does not fit."""
    with largest_cluster(bm, limit):
        assert_one_step(bm, size, sum(size))
        rng = np.random.default_rng(size[1])
        got, given, _ = run(bm, momentum(rng, *size, "falling"), "bf16")
    steps = [gated_ref.STEP] * 5
    want, model = gated_ref.newton_schulz(given, steps), gated_ref.rounded_steps(given, steps)
    norm = np.linalg.norm(want)
    assert np.linalg.norm(got - want) <= (2.0 ** -8 + 1e-4) * norm + 2 * np.linalg.norm(model - want)


@pytest.mark.parametrize("size", [(128, 2200), (2500, 100), (17, 5000), (128, 500)], ids=lambda s: f"{s[0]}x{s[1]}")
def test_where_the_grid_has_no_room(bm, size):
    """A cooperative launch that CUDA refuses: the products of any size take the call."""
    bm.bm_debug_limit_grid(2)
    try:
        with largest_cluster(bm, 2):
            assert_one_step(bm, size, sum(size))
            assert_one_step(bm, size, 2 + sum(size), beta=0.0)
    finally:
        bm.bm_debug_limit_grid(0)
    assert_one_step(bm, size, sum(size))
