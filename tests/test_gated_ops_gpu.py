"""A gated MLP's products on a GB300 against their 64-bit forms (gated_ref.py).

Tolerances are the error bounds of the FP32 arithmetic and the rounding to BF16 (2^-8 of a value), element by
element; small integers pin the products bit for bit. Outputs sit in buffers of canaries (padding columns and
rows must keep them) and padding of the inputs holds NaN.
"""

import numpy as np
import pytest

import gated_ref
import mlp_ref as ref
from gpu_helpers import check_no_device_error, tile_variant, torch
from test_mlp_ops_gpu import Out, _built, assert_close, bm, np64, padded, random_operands  # noqa: F401

pytestmark = pytest.mark.gpu


def bf16_tol(want, err):
    return 1.01 * (ref.rounding(want, True) + err)


GLU = [
    # m, n, k, act, transA, transB, kept
    (1, 1, 1, "silu", 0, 1, True),
    (1, 8, 8, "gelu", 0, 0, False),
    (1, 4096, 512, "silu", 0, 1, False),
    (3, 1000, 2056, "gelu_tanh", 0, 1, True),
    (16, 64, 4096, "silu", 0, 1, False),
    (17, 264, 520, "none", 0, 1, True),
    (31, 65, 700, "silu", 0, 0, True),
    (33, 130, 1100, "relu", 1, 0, False),
    (40, 513, 96, "gelu", 1, 1, True),
    (64, 512, 4096, "relu", 0, 0, True),
    (100, 63, 4100, "silu", 0, 1, True),
    (128, 2000, 256, "gelu", 0, 1, False),
    (128, 4863, 130, "gelu", 0, 1, True),       # as many tiles as half the SMs: few rows' kernel
    (128, 4865, 130, "silu", 1, 0, True),       # and one more: the tile kernel
    (20, 200, 60, "silu", 0, 1, True),          # one k-block, one CTA a cluster
    (32, 72, 8200, "gelu_tanh", 0, 0, True),
    (32, 9730, 96, "silu", 0, 1, True),         # an SM for each tile, and one tile more than that
    (8, 9800, 96, "silu", 1, 0, True),          # more tiles than SMs
    (9, 9800, 96, "relu", 0, 1, True),
    (129, 257, 72, "silu", 0, 1, True),
    (200, 520, 1000, "gelu_tanh", 1, 0, True),
    (300, 1100, 64, "gelu", 0, 1, False),
    (1000, 2162, 520, "silu", 0, 0, True),
    (2560, 2304, 576, "silu", 0, 1, True),      # several tiles a CTA, a last wave in halves
    (2500, 2301, 840, "gelu", 0, 0, True),
    (1111, 2048, 520, "silu", 0, 1, True),      # 128 x 256 tiles in one wave
]


def run_glu(bm, case, alpha=0.75, variant=0, seed=0):
    m, n, k, act, ta, tb, kept = case
    t = torch()
    rng = np.random.default_rng(seed + m + 7 * n + 13 * k)
    A, Wg, a, bg = random_operands(rng, m, n, k, ta, tb)
    bu = rng.normal(size=(k, n)) / np.sqrt(k)
    Wu = padded(bu.T if tb else bu, t.bfloat16)
    bu = np64(Wu).T if tb else np64(Wu)
    H, G, U = (Out(m, n, t.bfloat16) for _ in range(3))
    with tile_variant(variant):
        bm.gemm_glu(A, Wg, Wu, H.view, act=act, gate=G.view if kept else None, up=U.view if kept else None, alpha=alpha,
                    transA=bool(ta), transB=bool(tb))
    t.cuda.synchronize()
    check_no_device_error()
    want, err = gated_ref.glu(a, bg, bu, k, alpha, act)
    for out, w, e, name in list(zip((H, G, U), want, err, "HGU"))[:3 if kept else 1]:
        assert_close(np64(out.view), w, bf16_tol(w, e), name)
    for out in (H, G, U):
        out.check_guard()
    if not kept:
        assert (G.raw == 0x5A).all() and (U.raw == 0x5A).all()


def ids(c):
    return "x".join(map(str, c[:3])) + f"_{c[3]}"


@pytest.mark.parametrize("case", GLU, ids=ids)
def test_glu(bm, case):
    run_glu(bm, case)


TILED = [(129, 257, 72, "silu", 0, 1, True), (200, 520, 1000, "gelu_tanh", 1, 0, True), (700, 600, 192, "gelu", 0, 1, True),
         (520, 1031, 1100, "relu", 0, 0, True), (260, 72, 64, "silu", 1, 1, False)]


@pytest.mark.parametrize("variant", [1, 2, 3], ids=["single128x256", "single128x128", "pair256x256"])
@pytest.mark.parametrize("case", TILED, ids=ids)
def test_glu_on_every_tile(bm, case, variant):
    run_glu(bm, case, variant=variant, seed=variant)


INTEGER = [(1, 24, 40, 0, 1), (5, 100, 24, 0, 0), (48, 160, 64, 1, 1), (70, 33, 24, 1, 0), (300, 520, 24, 0, 1),
           (513, 1030, 24, 0, 0)]


@pytest.mark.parametrize("variant", [0, 1, 2, 3])
@pytest.mark.parametrize("case", INTEGER, ids=lambda c: "x".join(map(str, c[:3])))
def test_integers_bit_for_bit(bm, case, variant):
    """Small integers: every FP32 sum is exact and every result has at most 8 significant bits or is rounded once
    to nearest even, so the outputs are exactly those of integer arithmetic."""
    m, n, k, ta, tb = case
    t = torch()
    rng = np.random.default_rng(m + n)
    a, bg, bu = (rng.integers(-1, 2, s) for s in ((m, k), (k, n), (k, n)))
    A = padded(a.T if ta else a, t.bfloat16)
    Wg, Wu = (padded(b.T if tb else b, t.bfloat16) for b in (bg, bu))
    H, G, U, dG, dU, again = (Out(m, n, t.bfloat16) for _ in range(6))

    def rounded(x):
        return t.from_numpy(np.asarray(x, np.float32)).bfloat16().double().numpy()

    with tile_variant(variant):
        bm.gemm_glu(A, Wg, Wu, H.view, act="relu", gate=G.view, up=U.view, alpha=2.0, transA=bool(ta), transB=bool(tb))
        bm.gemm_dglu(A, Wg, G.view, U.view, dG.view, dU.view, act="relu", hidden=again.view, transA=bool(ta),
                     transB=bool(tb))
    g, u = 2.0 * (a @ bg), 2.0 * (a @ bu)
    assert np.array_equal(np64(G.view), rounded(g)) and np.array_equal(np64(U.view), rounded(u))
    assert np.array_equal(np64(H.view), rounded(np.maximum(g, 0) * u))
    g, u, dh = rounded(g), rounded(u), a @ bg
    assert np.array_equal(np64(dG.view), rounded(dh * u * (g > 0)))
    assert np.array_equal(np64(dU.view), rounded(dh * np.maximum(g, 0)))
    assert np.array_equal(np64(again.view), rounded(np.maximum(g, 0) * u))
    for out in (H, G, U, dG, dU, again):
        out.check_guard()
    check_no_device_error()


DGLU = [
    # m, n, k, act, transA, transB, hidden
    (1, 1, 1, "silu", 0, 0, True),
    (1, 8, 8, "gelu", 0, 1, False),
    (1, 4096, 512, "silu", 0, 0, True),
    (7, 1000, 2056, "gelu_tanh", 0, 0, True),
    (17, 264, 520, "none", 0, 1, True),
    (33, 130, 1100, "relu", 1, 0, False),
    (64, 512, 4096, "relu", 0, 0, True),
    (65, 9727, 128, "silu", 0, 1, True),
    (100, 9729, 130, "gelu", 0, 0, True),
    (128, 133, 4100, "gelu_tanh", 1, 1, True),
    (31, 20000, 72, "silu", 0, 0, True),
    (129, 257, 72, "silu", 0, 1, True),
    (200, 520, 1000, "gelu", 1, 1, True),
    (300, 1100, 64, "gelu", 0, 1, False),
    (1000, 2162, 520, "silu", 0, 0, True),
    (2560, 4608, 576, "silu", 0, 0, True),
    (2500, 4601, 840, "gelu", 0, 0, False),
]


def run_dglu(bm, case, alpha=0.75, variant=0, seed=0, in_place=False):
    m, n, k, act, ta, tb, hidden = case
    t = torch()
    rng = np.random.default_rng(seed + m + 7 * n + 13 * k)
    A, B, a, b = random_operands(rng, m, n, k, ta, tb)
    dG, dU, H = (Out(m, n, t.bfloat16) for _ in range(3))
    values = [1.2 * rng.normal(size=(m, n)) for _ in range(2)]
    values[0][rng.random((m, n)) < 0.02] *= 40.0     # (saturated gates)
    values[0][rng.random((m, n)) < 0.02] = 0.0
    G, U = (padded(v, t.bfloat16) for v in values)
    if in_place:
        dG.view.copy_(G)
        dU.view.copy_(U)
        G, U = dG.view, dU.view
    g, u = np64(G), np64(U)
    with tile_variant(variant):
        bm.gemm_dglu(A, B, G, U, dG.view, dU.view, act=act, hidden=H.view if hidden else None, alpha=alpha,
                     transA=bool(ta), transB=bool(tb))
    t.cuda.synchronize()
    check_no_device_error()
    want, err = gated_ref.dglu(a, b, k, alpha, g, u, act)
    for out, w, e, name in list(zip((dG, dU, H), want, err, ("dG", "dU", "H")))[:3 if hidden else 2]:
        assert_close(np64(out.view), w, bf16_tol(w, e), name)
    for out in (dG, dU, H):
        out.check_guard()
    if not hidden:
        assert (H.raw == 0x5A).all()


@pytest.mark.parametrize("case", DGLU, ids=ids)
def test_dglu(bm, case):
    run_dglu(bm, case)


@pytest.mark.parametrize("case", [DGLU[3], DGLU[9], DGLU[11], DGLU[14], DGLU[15]], ids=ids)
def test_dglu_in_place(bm, case):
    run_dglu(bm, case, in_place=True)


@pytest.mark.parametrize("variant", [1, 2, 3], ids=["single128x256", "single128x128", "pair256x256"])
@pytest.mark.parametrize("case", TILED, ids=ids)
def test_dglu_on_every_tile(bm, case, variant):
    run_dglu(bm, case, variant=variant, seed=variant, in_place=variant == 2)


# ------------------------------------------------------------------ gradients against differences
@pytest.mark.parametrize("act", ["none", "gelu", "gelu_tanh", "silu"])
def test_gradient_against_differences(act):
    """The formula that the kernel is held to, against central differences of sum(act(g) u dh) in 64 bits: h^2 times a
    third derivative below 4, and the rounding 1e-16 / h, at h = 1e-5."""
    rng = np.random.default_rng(3)
    g, u, dh = (rng.normal(size=(20, 30)) for _ in range(3))
    h = 1e-5
    (dg, du, _), _ = gated_ref.dglu(dh, np.eye(30), 30, 1.0, g, u, act)
    by_g = (ref.act(g + h, act) - ref.act(g - h, act)) / (2 * h) * u * dh
    by_u = ref.act(g, act) * ((u + h) - (u - h)) / (2 * h) * dh
    scale = 1 + np.abs(u * dh)
    assert (np.abs(dg - by_g) <= 1e-9 * scale).all() and (np.abs(du - by_u) <= 1e-9 * (1 + np.abs(g * dh))).all()


@pytest.mark.parametrize("m", [3, 200])
def test_without_products(bm, m):
    """k == 0 or alpha == 0: zeros (and H computed again); A and the weights are not read."""
    t = torch()
    rng = np.random.default_rng(m)
    n = 133
    for k, alpha in ((0, 1.0), (64, 0.0)):
        A = t.full((m, max(k, 8)), float("nan"), device="cuda").bfloat16()[:, :k]
        W = t.full((n, max(k, 8)), float("nan"), device="cuda").bfloat16()[:, :k]
        H, G, U = (Out(m, n, t.bfloat16) for _ in range(3))
        bm.gemm_glu(A, W, W, H.view, act="gelu", gate=G.view, up=U.view, alpha=alpha, transB=True)
        for out in (H, G, U):
            assert (np64(out.view) == 0).all()
            out.check_guard()
        g, u = (padded(rng.normal(size=(m, n)), t.bfloat16) for _ in range(2))
        dG, dU, H = (Out(m, n, t.bfloat16) for _ in range(3))
        bm.gemm_dglu(A, W, g, u, dG.view, dU.view, act="gelu", hidden=H.view, alpha=alpha, transB=True)
        (_, _, h), (_, _, e) = gated_ref.dglu(np.zeros((m, 1)), np.zeros((1, n)), 1, 1.0, np64(g), np64(u), "gelu")
        assert (np64(dG.view) == 0).all() and (np64(dU.view) == 0).all()
        assert_close(np64(H.view), h, bf16_tol(h, e), "H")
        for out in (dG, dU, H):
            out.check_guard()
    check_no_device_error()


def test_nan_and_infinity_stay_in_their_rows_and_columns(bm):
    t = torch()
    rng = np.random.default_rng(8)
    for m, n, k in ((40, 96, 128), (300, 520, 136)):
        a, bg, bu = rng.normal(size=(m, k)), rng.normal(size=(k, n)), rng.normal(size=(k, n))
        a[5, 3] = np.nan
        bu[7, 11] = np.inf
        A, Wg, Wu = padded(a, t.bfloat16), padded(bg, t.bfloat16), padded(bu, t.bfloat16)
        H, G, U = (Out(m, n, t.bfloat16) for _ in range(3))
        bm.gemm_glu(A, Wg, Wu, H.view, act="silu", gate=G.view, up=U.view)
        g, u, h = np64(G.view), np64(U.view), np64(H.view)
        assert np.isnan(g[5]).all() and np.isfinite(np.delete(g, 5, 0)).all()
        assert np.isnan(u[5]).all() and np.isinf(np.delete(u[:, 11], 5)).all()
        keep = np.delete(np.delete(u, 5, 0), 11, 1)
        assert np.isfinite(keep).all() and np.isfinite(np.delete(np.delete(h, 5, 0), 11, 1)).all()
        assert np.isnan(h[5]).all() and not np.isfinite(np.delete(h[:, 11], 5)).any()


def test_halves_of_one_buffer(bm):
    """Both weights in one [2 n, k] and G, U (then dG, dU) in one [m, 2 n]: the rest of the backward pass is two
    plain products over them."""
    t = torch()
    rng = np.random.default_rng(12)
    m, n, k = 200, 264, 320
    x = padded(rng.normal(size=(m, k)), t.bfloat16)
    w = padded(rng.normal(size=(2 * n, k)) / np.sqrt(k), t.bfloat16)
    wd = padded(rng.normal(size=(k, n)) / np.sqrt(n), t.bfloat16)
    dy = padded(rng.normal(size=(m, k)), t.bfloat16)
    gu = t.empty(m, 2 * n, dtype=t.bfloat16, device="cuda")
    h, dx, dw = t.empty(m, n, **gpu_bf16()), t.empty(m, k, device="cuda"), t.empty(2 * n, k, device="cuda")
    bm.gemm_glu(x, w[:n], w[n:], h, gate=gu[:, :n], up=gu[:, n:], transB=True)
    kept = np64(gu)
    bm.gemm_dglu(dy, wd, gu[:, :n], gu[:, n:], gu[:, :n], gu[:, n:], hidden=h)
    bm.gemm(gu, w, dx)
    bm.gemm(gu, x, dw, transA=True)
    check_no_device_error()
    (dg, du, _), (eg, eu, _) = gated_ref.dglu(np64(dy), np64(wd), k, 1.0, kept[:, :n], kept[:, n:], "silu")
    both, err = np.concatenate([dg, du], 1), np.concatenate([eg, eu], 1)
    assert_close(np64(gu), both, bf16_tol(both, err), "dG dU")
    got = np64(gu)                                    # (the plain products are held to what they read)
    for out, a, b, kk in ((dx, got, np64(w), 2 * n), (dw, got.T, np64(x), m)):
        want, e = ref.product(a, b, kk)
        assert_close(np64(out), want, e + ref.rounding(want, False), "plain product")


def gpu_bf16():
    return dict(dtype=torch().bfloat16, device="cuda")


def test_captured_and_replayed_on_another_stream(bm):
    t = torch()
    rng = np.random.default_rng(21)
    for m, n, k in ((4, 320, 256), (300, 520, 192)):
        A, Wg, _, _ = random_operands(rng, m, n, k, 0, 1)
        Wu = padded(rng.normal(size=(n, k)) / np.sqrt(k), t.bfloat16)
        D, Wd, _, _ = random_operands(rng, m, n, k, 0, 0)
        outs = [t.empty(m, n + n % 8, **gpu_bf16())[:, :n] for _ in range(6)]
        H, G, U, dG, dU, again = outs

        def calls():
            bm.gemm_glu(A, Wg, Wu, H, gate=G, up=U, transB=True)
            bm.gemm_dglu(D, Wd, G, U, dG, dU, hidden=again)

        calls()
        t.cuda.synchronize()
        first = [o.clone() for o in outs]
        side = t.cuda.Stream()
        graph = t.cuda.CUDAGraph()
        side.wait_stream(t.cuda.current_stream())
        with t.cuda.stream(side):
            calls()
            with t.cuda.graph(graph, stream=side):
                calls()
            for o in outs:
                o.fill_(float("nan"))
            graph.replay()
            graph.replay()
        t.cuda.synchronize()
        assert all(t.equal(o, f) for o, f in zip(outs, first))
        A.copy_(2 * A)          # a replay reads what the buffers hold then
        graph.replay()
        t.cuda.synchronize()
        assert t.equal(G, 2 * first[1]) and t.equal(U, 2 * first[2])
    check_no_device_error()


def test_a_stream_as_an_argument(bm):
    """Work queued on the given stream, in its order, whatever the current one is."""
    t = torch()
    side = t.cuda.Stream()
    x, w = t.randn(200, 256, device="cuda").bfloat16(), (t.randn(264, 256, device="cuda") / 16).bfloat16()
    h, g, u, dg, du = (t.empty(200, 264, **gpu_bf16()) for _ in range(5))
    bm.gemm_glu(x, w, w, h, gate=g, up=u, transB=True)
    bm.gemm_dglu(x, w, g, u, dg, du, transB=True)
    t.cuda.synchronize()
    first = [o.clone() for o in (h, g, u, dg, du)]
    t.cuda.synchronize()
    with t.cuda.stream(side):
        t.cuda._sleep(20_000_000)        # about 10 ms: what follows on this stream waits for it
        for o in (h, g, u, dg, du):
            o.fill_(float("nan"))
    bm.gemm_glu(x, w, w, h, gate=g, up=u, transB=True, stream=side)
    bm.gemm_dglu(x, w, g, u, dg, du, transB=True, stream=side)
    side.synchronize()
    assert all(t.equal(a, b) for a, b in zip((h, g, u, dg, du), first))
    check_no_device_error()


def test_stalled_copy_is_reported(bm):
    """A copy that never comes: the waits run out, the status word says so, and the next call works."""
    t = torch()
    w = t.ones(300, 128, **gpu_bf16())
    everything = [t.zeros(300, 304, **gpu_bf16())[:, :300] for _ in range(3)]
    stream = t.cuda.current_stream().cuda_stream
    bm.bm_set_wait_timeout_ms(50)
    try:
        for variant in (0, 1, 2, 3):
            rows = 300 if variant else 40           # (few rows have a kernel of their own)
            x, (h, g, u) = t.ones(rows, 128, **gpu_bf16()), (o[:rows] for o in everything)
            for call in (lambda: bm.gemm_glu(x, w, w, h, transB=True),
                         lambda: bm.gemm_dglu(x, w, h, h, g, u, transB=True)):
                bm.bm_debug_inject_stall(1)
                with tile_variant(variant):
                    call()
                bm.bm_debug_inject_stall(0)
                assert bm.bm_get_last_device_error(stream) == bm.BM_ERR_TIMEOUT
                with tile_variant(variant):
                    call()
                assert bm.bm_get_last_device_error(stream) == bm.BM_OK
    finally:
        bm.bm_debug_inject_stall(0)
        bm.bm_set_wait_timeout_ms(2000)
