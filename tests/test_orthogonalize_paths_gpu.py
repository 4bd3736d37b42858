"""Forms of the orthogonalised update that its sizes alone do not reach on a whole GB300, and what its documentation
says of its numbers, against the 64-bit form (gated_ref.py)."""

import contextlib

import numpy as np
import pytest

import gated_ref
import mlp_ref as ref
from gpu_helpers import check_no_device_error, tile_variant, torch
from test_mlp_ops_gpu import Out, _built, assert_close, bm, np64, padded  # noqa: F401
from test_orthogonalize_gpu import momentum, run, workspace

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


SCALES = (0, -40, 40, -60, 60, -120, 118, -146)


@pytest.mark.parametrize("size", [(40, 100), (500, 40), (40, 1500), (128, 3000), (300, 150), (700, 1200)],
                         ids=lambda s: f"{s[0]}x{s[1]}")
def test_x0_to_its_last_bits_at_any_scale(bm, size):
    """One step of (1, 0, 0) gives X0 = X / |X|, whose size does not matter up to FP32's ends. Integers below 128 have
    squares whose FP32 sums are exact (512 of them at most before FP64 goes on), and no scale changes their bits. Added
    to minus its BF16 value X0 shows what a BF16 result does not hold: two FP16 halves of 256 X0 leave 2^-22 of a value
    and half of FP16's smallest step, 2^-25 / 256; the factor and its product are two roundings of FP32."""
    t = torch()
    rng = np.random.default_rng(size[0])
    k = rng.integers(-127, 128, size).astype(np.float64)
    want = k / np.sqrt((k * k).sum())
    ws = workspace(bm, *size)
    rounded = t.from_numpy(want).bfloat16()
    rest = want - rounded.double().numpy()
    tol = 2.0 ** -22 * np.abs(want) + 2.0 ** -33 + 3 * 2.0 ** -24 * np.abs(want) + 1.01 * ref.rounding(rest, True)
    step = dict(steps=1, coeffs=(1.0, 0.0, 0.0), eps=0.0, workspace=ws)
    for e in SCALES:
        X = padded(k * 2.0 ** e, t.float32)
        C = Out(*size, t.bfloat16)
        bm.orthogonalize(X, C.view, **step)
        # (where X0 lies within those errors of the middle of two BF16 values either may come: 2^-13 of them)
        got, there = C.view.clone(), rounded.cuda()
        apart = (got.view(t.int16).int() - there.view(t.int16).int())[got != there].abs()
        assert apart.numel() <= k.size // 100 and (apart <= 1).all(), f"2^{e}"
        C.view.copy_(-rounded)
        bm.orthogonalize(X, C.view, beta=1.0, **step)
        assert_close(np64(C.view), rest, tol, f"2^{e}")
        C.check_guard()
    check_no_device_error()


@pytest.mark.parametrize("rows,variant", [(64, 0), (200, 0), (64, 2), (200, 3)])
@pytest.mark.parametrize("wide", [True, False])
def test_a_long_side_of_dense_rows(bm, rows, variant, wide):
    """A over 2^18 columns: a truncating accumulator loses at most a unit of its sum in 16 products, 7.5e-9 of it per
    column. A row of A X against its own X gives that row's sum of squares once more (and its other products, which are
    2^-9 of it): BF16's rounding and FP16's are as often up as down and leave 2^-8 / sqrt(2^18) of it."""
    n = 2 ** 18
    rng = np.random.default_rng(18)
    got, x, _ = run(bm, rng.normal(size=(rows, n) if wide else (n, rows)), "f32", 1, [(0.0, 1.0, 0.0)], variant=variant)
    want = gated_ref.newton_schulz(x, [(0.0, 1.0, 0.0)])
    axis = 1 if wide else 0
    ratio = (got * x).sum(axis=axis) / (want * x).sum(axis=axis) - 1.0
    assert np.abs(ratio).max() <= 7.5e-9 * n + 4 * 2.0 ** -8 / np.sqrt(n), np.abs(ratio).max()


@pytest.mark.parametrize("size,k,variant", [
    ((3000, 3100), 8, 0), ((3100, 2900), 8, 0), ((4200, 4100), 8, 0), ((3000, 2900), 8, 2), ((600, 8000), 7, 0),
    ((1030, 515), 6, 0), ((120, 16000), 5, 0), ((1900, 128), 5, 0), ((100, 100), 5, 0)],
    ids=lambda v: f"{v[0]}x{v[1]}" if isinstance(v, tuple) else str(v))
def test_integers_bit_for_bit(bm, size, k, variant):
    """4^k entries of 1 or -1 have the norm 2^k, so that X0 is these times 2^-k, A integers G times 4^-k, and with
    (1, 4^k, 16^k) X' = (1 + G + G^2) X0: integers that FP16 and FP32 hold, whatever the order of their sums. Rounded
    once they are the result. A second step of (1, 0, 0) takes X' through its two halves. Sizes: a shorter side above
    2816 gives more than 76 pair tiles of A's triangle (variant 2: more than 152 of 128 x 128), so that a CTA goes from
    one to the next (17 x 18 / 2 tiles: to a third) with accumulators in turn, inputs fetched ahead and staging blocks
    given back; then split tiles, and one kernel."""
    t = torch()
    rng = np.random.default_rng(size[0])
    x = np.zeros(size[0] * size[1])
    x[rng.choice(x.size, 4 ** k, replace=False)] = rng.choice((-1.0, 1.0), 4 ** k)
    x = x.reshape(size)
    y = x if size[0] <= size[1] else x.T
    gram = y @ y.T
    square = gram @ gram
    off = ~np.eye(len(gram), dtype=bool)
    want = y + gram @ y + square @ y
    assert np.abs(gram[off]).max() <= 2048 and np.abs((gram + square)[off]).max() <= 2048  # integers of FP16
    # what FP16 can hold: X times 256, and the next A off its diagonal
    assert np.abs(want).max() * 2.0 ** (8 - k) <= 65280 and np.abs((want @ want.T)[off]).max() / 4.0 ** k <= 65504
    want = t.from_numpy(np.ascontiguousarray(want if size[0] <= size[1] else want.T)) / 2 ** k
    steps = [(1.0, 4.0 ** k, 16.0 ** k), (1.0, 0.0, 0.0)]
    X, ws = padded(x, t.bfloat16), workspace(bm, *size)
    for count in (1, 2):
        C = Out(*size, t.bfloat16)
        with tile_variant(variant):
            bm.orthogonalize(X, C.view, steps=count, coeffs=steps[:count], eps=0.0, workspace=ws)
        check_no_device_error()
        C.check_guard()
        assert t.equal(C.view.cpu(), want.bfloat16()), count
