"""The orthogonalised update on a GB300 against its 64-bit form (gated_ref.py).

One step is held element by element to the bound of its roundings; five steps, whose map amplifies and
contracts, to the error that the same rounding points make in 64-bit arithmetic (twice it, for the FP32 sums
and for where each rounding falls) beside the rounding to BF16.
"""

import numpy as np
import pytest

import gated_ref
import mlp_ref as ref
from gpu_helpers import check_no_device_error, tile_variant, torch
from test_mlp_ops_gpu import Out, _built, assert_close, bm, dtype_of, np64, padded  # noqa: F401

pytestmark = pytest.mark.gpu

SIZES = [(1, 1), (1, 200), (200, 1), (3, 5), (16, 16), (64, 1000), (1000, 64), (127, 129), (130, 131), (128, 128),
         (257, 300), (300, 257), (520, 520), (100, 2100), (1030, 515),
         (600, 8000), (8000, 600),   # several tiles a CTA, a last wave in halves
         # shorter side at most 128: one CTA, clusters of two to sixteen, grids
         (128, 127), (61, 250), (257, 128), (128, 1024), (1024, 100), (128, 1025), (1025, 3), (128, 2048), (2050, 77),
         (17, 5000)]


def momentum(rng, m, n, kind):
    """Matrices whose singular values are of a size, fall off, or are a few over noise."""
    if kind == "gauss":
        return rng.normal(size=(m, n))
    r = min(m, n)
    u, _ = np.linalg.qr(rng.normal(size=(m, r)))
    v, _ = np.linalg.qr(rng.normal(size=(n, r)))
    i = np.arange(1, r + 1.0)
    x = (u * (i ** -1.5 if kind == "falling" else np.where(i <= 4, 1.0, 0.0))) @ v.T
    return x + (0.02 / np.sqrt(max(m, n))) * rng.normal(size=(m, n)) if kind == "few" else x


def workspace(bm, m, n):
    t = torch()
    return t.randint(0, 256, (bm.orthogonalize_workspace_size(m, n),), dtype=t.uint8, device="cuda")


def run(bm, x, x_type="f32", steps=5, coeffs=None, alpha=1.0, beta=0.0, variant=0, in_place=False):
    """(result, X and the C before as they were given, the buffer)."""
    t = torch()
    m, n = x.shape
    X = padded(x, dtype_of(x_type))
    C = Out(m, n, t.bfloat16)
    before = None
    if beta != 0.0:
        C.view.copy_(t.randn(m, n, device="cuda"))
        before = np64(C.view)
    if in_place:
        C.view.copy_(X)
        X = C.view
    given = np64(X)
    with tile_variant(variant):
        bm.orthogonalize(X, C.view, alpha=alpha, beta=beta, steps=steps, coeffs=coeffs, workspace=workspace(bm, m, n))
    t.cuda.synchronize()
    check_no_device_error()
    C.check_guard()
    return np64(C.view), given, before


@pytest.mark.parametrize("variant", [0, 1, 2, 3], ids=["auto", "single128x256", "single128x128", "pair256x256"])
@pytest.mark.parametrize("size", SIZES, ids=lambda s: f"{s[0]}x{s[1]}")
def test_one_step_element_by_element(bm, size, variant):
    rng = np.random.default_rng(size[0] + 3 * size[1])
    for coeffs, x_type, alpha, beta in (([gated_ref.STEP], "f32", 1.0, 0.0), ([(0.5, -1.5, 2.0)], "bf16", -0.7, 0.9),
                                        ([(0.0, 1.0, 0.0)], "f32", 1.0, 0.0), ([(1.0, 0.0, 0.0)], "f32", 2.0, 0.0)):
        got, x, before = run(bm, 3e-5 * momentum(rng, *size, "gauss"), x_type, 1, coeffs, alpha, beta, variant)
        want = alpha * gated_ref.newton_schulz(x, coeffs)
        err = np.abs(alpha) * gated_ref.one_step_bound(x, coeffs)
        if beta != 0.0:
            want = want + beta * before
            err = err + 2 * ref.U32 * (np.abs(want) + np.abs(beta * before))
        assert_close(got, want, 1.01 * (err + ref.rounding(want, True)), f"{coeffs}")


@pytest.mark.parametrize("kind", ["gauss", "falling", "few"])
@pytest.mark.parametrize("size", SIZES, ids=lambda s: f"{s[0]}x{s[1]}")
def test_five_steps(bm, size, kind):
    rng = np.random.default_rng(size[0] + size[1])
    for x_type, variant in (("f32", 0), ("bf16", 3)):
        got, x, _ = run(bm, 1e-4 * momentum(rng, *size, kind), x_type, variant=variant)
        steps = [gated_ref.STEP] * 5
        want, model = gated_ref.newton_schulz(x, steps), gated_ref.rounded_steps(x, steps)
        norm = np.linalg.norm(want)
        # (64-bit arithmetic with the same roundings; each step's FP32 sums, 1e-6 of |X|, grow with a like them)
        limit = 2.0 ** -8 + 2 * np.linalg.norm(model - want) / norm + 1e-4
        assert np.linalg.norm(got - want) <= limit * norm


def test_singular_values_land_where_the_polynomial_takes_them(bm):
    """An X of known singular values: those of the result are five polynomials of them."""
    t = torch()
    rng = np.random.default_rng(6)
    u, _ = np.linalg.qr(rng.normal(size=(96, 96)))
    v, _ = np.linalg.qr(rng.normal(size=(160, 96)))
    s = np.linspace(0.02, 1.0, 96)
    got, x, _ = run(bm, (u * s) @ v.T)
    p = np.sort(s / np.linalg.norm(s))
    for _ in range(5):
        p = gated_ref.STEP[0] * p + gated_ref.STEP[1] * p ** 3 + gated_ref.STEP[2] * p ** 5
    # each is off by at most the spectral norm of the error: below the rounding's Frobenius norm, 2^-8 |C|, and 1e-3 |C|
    assert np.abs(np.sort(np.linalg.svd(got, compute_uv=False)) - np.sort(p)).max() <= (2.0 ** -8 + 1e-3) * np.linalg.norm(p)
    assert 0.6 < p[5:].min() and p.max() < 1.3


def test_each_step_has_its_coefficients(bm):
    rng = np.random.default_rng(2)
    coeffs = [(4.0, -8.0, 5.0), (3.0, -3.2, 1.3), (2.0, -1.5, 0.5)]
    got, x, _ = run(bm, momentum(rng, 90, 200, "gauss"), steps=3, coeffs=coeffs)
    want, model = gated_ref.newton_schulz(x, coeffs), gated_ref.rounded_steps(x, coeffs)
    norm = np.linalg.norm(want)
    assert np.linalg.norm(got - want) <= 2.0 ** -8 * norm + 2 * np.linalg.norm(model - want) + 1e-4 * norm
    with pytest.raises(ValueError, match="coeffs"):
        run(bm, x, steps=2, coeffs=coeffs)


@pytest.mark.parametrize("size", [(90, 120), (100, 600), (1500, 64), (300, 280)])
def test_many_steps_converge_to_the_orthogonal_factor(bm, size):
    """(15, -10, 3) / 8 takes every singular value to 1: after 64 steps X is U V^T. What is left is the rounding of
    the last steps: there each operand is off by 2^-11 of its values at most, the three of them by 2^-9 of |X|."""
    rng = np.random.default_rng(size[0])
    x = rng.normal(size=size)
    got, x, _ = run(bm, x, steps=64, coeffs=(1.875, -1.25, 0.375))
    u, _, vt = np.linalg.svd(x, full_matrices=False)
    want = u @ vt
    assert np.linalg.norm(got - want) <= (2.0 ** -8 + 2.0 ** -9) * np.linalg.norm(want)


@pytest.mark.parametrize("size", [(40, 100), (100, 600), (4000, 128), (300, 257)])
def test_in_place_and_the_same_bits_again(bm, size):
    rng = np.random.default_rng(4)
    x = momentum(rng, *size, "falling")
    first, _, _ = run(bm, x, "bf16")
    again, _, _ = run(bm, x, "bf16", in_place=True)
    assert np.array_equal(first, again)


@pytest.mark.parametrize("size", [(40, 100), (500, 40), (40, 1500), (300, 150)])
def test_any_scale(bm, size):
    """X0 does not depend on X's size: powers of two up to FP32's ends change no bit of it, though its squares
    under- or overflow FP32 (eps = 0)."""
    t = torch()
    rng = np.random.default_rng(9)
    x = rng.integers(-8, 9, size).astype(np.float64)   # (significands that survive in subnormal values)
    ws = workspace(bm, *size)
    results = []
    for e in (0, -60, 60, -120, 124, -146):
        X, C = padded(x * 2.0 ** e, t.float32), t.empty(size[0], -(-size[1] // 8) * 8, dtype=t.bfloat16, device="cuda")
        bm.orthogonalize(X, C[:, :size[1]], eps=0.0, workspace=ws)
        results.append(np64(C[:, :size[1]]))
    norm = np.linalg.norm(results[0])
    for r in results[1:]:
        # (the scale factor is a product of FP64 or FP32 arithmetic: 2^-24 apart, which may turn a rounding)
        assert np.linalg.norm(r - results[0]) <= (2.0 ** -8 + 2e-3) * norm
    check_no_device_error()


def test_zero_nan_and_infinity(bm):
    t = torch()
    for m, n in ((30, 50), (50, 600), (1400, 40), (300, 280)):
        ws = workspace(bm, m, n)
        X = t.zeros(m, n + 6 if n % 4 else n, device="cuda")[:, :n]
        C = Out(m, n, t.bfloat16)
        bm.orthogonalize(X, C.view, workspace=ws)
        assert (np64(C.view) == 0).all()
        bm.orthogonalize(X, C.view, eps=0.0, workspace=ws)
        assert np.isnan(np64(C.view)).all()
        for bad in (float("nan"), float("inf"), -float("inf")):
            X.normal_()
            X[m // 2, n // 3] = bad
            bm.orthogonalize(X, C.view, workspace=ws)
            assert np.isnan(np64(C.view)).all()
        # C is not read with beta == 0, nor X with alpha == 0
        C.view.fill_(float("nan"))
        bm.orthogonalize(t.randn(m, n + 6 if n % 4 else n, device="cuda")[:, :n], C.view, workspace=ws)
        assert np.isfinite(np64(C.view)).all()
        C.view.fill_(3.0)
        bm.orthogonalize(X, C.view, alpha=0.0, beta=0.5, workspace=ws)
        assert (np64(C.view) == 1.5).all()
        C.check_guard()
    check_no_device_error()


def test_captured_and_replayed(bm):
    t = torch()
    rng = np.random.default_rng(31)
    for m, n in ((64, 96), (400, 96), (64, 1800), (64, 2800), (300, 200)):
        X = padded(momentum(rng, m, n, "gauss"), t.bfloat16)
        W = t.randn(m, n, device="cuda").bfloat16()
        ws = workspace(bm, m, n)
        twice = W.clone()
        for _ in range(2):
            bm.orthogonalize(X, twice, alpha=-0.1, beta=0.9, workspace=ws)
        side, graph = t.cuda.Stream(), t.cuda.CUDAGraph()
        side.wait_stream(t.cuda.current_stream())
        C = W.clone()
        with t.cuda.graph(graph, stream=side):
            bm.orthogonalize(X, C, alpha=-0.1, beta=0.9, workspace=ws)
        t.cuda.synchronize()
        assert t.equal(C, W)
        graph.replay()
        graph.replay()
        t.cuda.synchronize()
        assert t.equal(C, twice)
    check_no_device_error()


def test_the_longest_that_one_kernel_takes(bm):
    """A CTA for each 128 lines of the longer side up to the SMs' number; one line more takes the products of any
    size. Both agree with 64 bits."""
    t = torch()
    rng = np.random.default_rng(14)
    sms = t.cuda.get_device_properties(0).multi_processor_count
    for m, n in ((128 * sms, 20), (128 * sms + 1, 20), (20, 128 * sms)):
        got, x, _ = run(bm, rng.normal(size=(m, n)))
        steps = [gated_ref.STEP] * 5
        want, model = gated_ref.newton_schulz(x, steps), gated_ref.rounded_steps(x, steps)
        norm = np.linalg.norm(want)
        assert np.linalg.norm(got - want) <= (2.0 ** -8 + 1e-4) * norm + 2 * np.linalg.norm(model - want)


def test_two_streams_at_once(bm):
    """Calls of which each waits for all its CTAs, on two streams with a workspace each."""
    t = torch()
    rng = np.random.default_rng(77)
    xs = [padded(momentum(rng, 100, 12000, "gauss"), t.bfloat16) for _ in range(2)]
    ws = [workspace(bm, 100, 12000) for _ in range(2)]
    want = []
    for x, w in zip(xs, ws):
        want.append(bm.orthogonalize(x, t.empty(100, 12000, dtype=t.bfloat16, device="cuda"), workspace=w))
    t.cuda.synchronize()
    streams, got = [t.cuda.Stream() for _ in range(2)], [t.empty_like(w) for w in want]
    for _ in range(10):
        for x, w, c, stream in zip(xs, ws, got, streams):
            bm.orthogonalize(x, c, workspace=w, stream=stream)
    t.cuda.synchronize()
    check_no_device_error()
    assert all(t.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("size", [(100, 700), (90, 4000), (260, 300)])
def test_two_graphs_share_a_workspace(bm, size):
    """Captured apart, replayed in turn on one stream: each finds the workspace as the other left it."""
    t = torch()
    rng = np.random.default_rng(size[1])
    m, n = size
    ws = workspace(bm, m, n)
    xs = [padded(momentum(rng, m, n, "gauss"), t.bfloat16) for _ in range(2)]
    cs = [t.zeros(m, n + (-n) % 8, dtype=t.bfloat16, device="cuda")[:, :n] for _ in range(2)]
    want = []
    for x, c in zip(xs, cs):
        want.append(bm.orthogonalize(x, c, workspace=workspace(bm, m, n)).clone())
        c.zero_()
    t.cuda.synchronize()
    side, graphs = t.cuda.Stream(), [t.cuda.CUDAGraph() for _ in range(2)]
    side.wait_stream(t.cuda.current_stream())
    for g, x, c in zip(graphs, xs, cs):
        with t.cuda.graph(g, stream=side):
            bm.orthogonalize(x, c, workspace=ws)
    for _ in range(3):
        for g in graphs:
            g.replay()
    t.cuda.synchronize()
    check_no_device_error()
    assert all(t.equal(c, w) for c, w in zip(cs, want))


def test_coefficients_of_any_sequence(bm):
    t = torch()
    X, ws = t.randn(40, 48, device="cuda"), workspace(bm, 40, 48)
    a, b, c, d = (t.empty(40, 48, dtype=t.bfloat16, device="cuda") for _ in range(4))
    bm.orthogonalize(X, a, steps=2, workspace=ws)
    bm.orthogonalize(X, b, steps=2, coeffs=np.array(gated_ref.STEP, np.float32), workspace=ws)
    bm.orthogonalize(X, c, steps=2, coeffs=[gated_ref.STEP, list(gated_ref.STEP)], workspace=ws)
    bm.orthogonalize(X, d, steps=3, coeffs=[gated_ref.STEP] * 3, workspace=ws)
    assert t.equal(a, b) and t.equal(a, c) and not t.equal(a, d)
    for bad in ([], [1.0, 2.0], [gated_ref.STEP], [gated_ref.STEP, (1.0, 2.0)]):
        with pytest.raises(ValueError, match="coeffs"):
            bm.orthogonalize(X, a, steps=2, coeffs=bad, workspace=ws)
    with pytest.raises(bm.BMError):
        bm.orthogonalize(X, a)                        # no workspace
    with pytest.raises(ValueError):
        bm.orthogonalize(X, a[:39], workspace=ws)
    with pytest.raises(TypeError):
        bm.orthogonalize(X, t.empty(40, 48, device="cuda"), workspace=ws)


def test_stalled_copy_is_reported(bm):
    t = torch()
    stream = t.cuda.current_stream().cuda_stream
    bm.bm_set_wait_timeout_ms(20)
    try:
        for (m, n), variant in (((300, 304), 2), ((300, 304), 3), ((100, 104), 0), ((100, 504), 0), ((2000, 104), 0),
                                ((3000, 104), 0)):
            X, C = t.randn(m, n, device="cuda").bfloat16(), t.zeros(m, n, device="cuda").bfloat16()
            ws = workspace(bm, m, n)
            bm.bm_debug_inject_stall(1)
            with tile_variant(variant):
                bm.orthogonalize(X, C, workspace=ws)
            bm.bm_debug_inject_stall(0)
            assert bm.bm_get_last_device_error(stream) == bm.BM_ERR_TIMEOUT
            with tile_variant(variant):
                bm.orthogonalize(X, C, workspace=ws)
            assert bm.bm_get_last_device_error(stream) == bm.BM_OK
            assert t.isfinite(C).all()
    finally:
        bm.bm_debug_inject_stall(0)
        bm.bm_set_wait_timeout_ms(2000)
