"""The operators around an MLP's products, on a GB300, against their 64-bit forms (mlp_ref.py).

Tolerances are the error bounds of the FP32 arithmetic, element by element, derived in mlp_ref.py and
beside each test; integer data pin the products, the checkpoints and the residual sums bit for bit.
Outputs sit in buffers of canaries (padding columns and rows must keep them) and padding of the inputs
holds NaN.
"""

import numpy as np
import pytest

import mlp_ref as ref
from gpu_helpers import check_no_device_error, tile_variant, torch

pytestmark = pytest.mark.gpu

CHUNK = 1024  # K of one accumulator piece, at most, when an output is FP32 or a checkpoint is kept


@pytest.fixture(scope="module", autouse=True)
def _built():
    from blas3_tensor_core_gb300 import build
    build.build()
    assert torch().cuda.is_available()


@pytest.fixture(scope="module")
def bm():
    import blas3_tensor_core_gb300
    return blas3_tensor_core_gb300


def np64(t):
    return t.detach().double().cpu().numpy()


def padded(values, dtype, pad=8, fill=float("nan")):
    """[rows, cols] view of `values` in a buffer whose rows are a multiple of 16 bytes (+ pad) of `fill`."""
    t = torch()
    rows, cols = values.shape
    ld = -(-cols // 8) * 8 + pad
    buf = t.full((rows, ld), fill, dtype=dtype, device="cuda")
    buf[:, :cols] = t.as_tensor(np.asarray(values, np.float64)).to(dtype).cuda()
    return buf[:, :cols]


class Out:
    """A [rows, cols] output inside a buffer of canaries."""

    def __init__(self, rows, cols, dtype, pad=8):
        t = torch()
        self.rows, self.cols = rows, cols
        size = t.empty(0, dtype=dtype).element_size()
        ld = -(-cols // 16) * 16 + pad * (16 if size == 1 else 1)
        self.raw = t.full((rows + 3, ld * size), 0x5A, dtype=t.uint8, device="cuda")
        self.view = self.raw.view(dtype)[:rows, :cols]
        self.size = size

    def check_guard(self):
        raw = self.raw.cpu().numpy()
        assert (raw[self.rows:] == 0x5A).all(), "rows past the output were written"
        assert (raw[:, self.cols * self.size:] == 0x5A).all(), "columns past the output were written"


def dtype_of(name):
    t = torch()
    return {"f32": t.float32, "bf16": t.bfloat16}[name]


def assert_close(got, want, tol, what):
    bad = ~(np.abs(got - want) <= tol)
    if bad.any():
        i = tuple(np.argwhere(bad)[0])
        raise AssertionError(f"{what}: {bad.sum()} of {bad.size} off, first at {i}: got {got[i]!r} want {want[i]!r} "
                             f"tol {tol[i]!r}; worst |err|/tol {np.nanmax(np.abs(got - want) / tol):.3g}")


class Ckpt:
    """Checkpoint buffers with canaries: codes [m, n] and the tiled scales."""

    def __init__(self, m, n):
        t = torch()
        self.m, self.n = m, n
        self.codes = Out(m, n, t.uint8, pad=1)
        size = -(-m // 128) * -(-n // 128) * 512
        self.raw_scales = t.full((size + 64,), 0x5A, dtype=t.uint8, device="cuda")
        self.pair = (self.codes.view, self.raw_scales[:size])

    def fill(self, z, scale_fill=0):
        t = torch()
        q, s = ref.quantize(z)
        self.codes.view.copy_(t.from_numpy(q).cuda())
        self.pair[1].copy_(t.from_numpy(ref.tile_scales(s, self.m, self.n, scale_fill)).cuda())
        return self

    def arrays(self):
        return self.pair[0].cpu().numpy(), self.pair[1].cpu().numpy()

    def check_guard(self):
        self.codes.check_guard()
        assert (self.raw_scales[self.pair[1].numel():] == 0x5A).all()


def random_operands(rng, m, n, k, ta, tb, std_b=None):
    a = rng.normal(size=(m, k))
    b = rng.normal(size=(k, n)) * (1.0 / np.sqrt(max(k, 1)) if std_b is None else std_b)
    t = torch()
    A = padded(a.T if ta else a, t.bfloat16)
    B = padded(b.T if tb else b, t.bfloat16)
    a64, b64 = np64(A), np64(B)
    return A, B, a64.T if ta else a64, b64.T if tb else b64


def workspace(nbytes=32 << 20):
    t = torch()
    return t.randint(0, 256, (nbytes,), dtype=t.uint8, device="cuda")  # contents need no initialisation


# ------------------------------------------------------------------ forward product
LINEAR = [
    # m, n, k, act, c, bias, residual, ta, tb, checkpoint
    (1, 16, 64, "gelu", "bf16", "bf16", False, 0, 1, False),
    (1, 8, 8, "silu", "f32", "f32", True, 0, 0, False),
    (1, 1, 1, "relu", "f32", "bf16", True, 0, 1, True),
    (3, 1000, 2056, "gelu_tanh", "bf16", "f32", True, 0, 1, False),
    (17, 264, 520, "none", "f32", "none", True, 0, 1, False),
    (33, 130, 1100, "silu", "bf16", "f32", False, 1, 0, False),
    (40, 513, 96, "gelu", "f32", "bf16", True, 1, 1, False),
    (64, 512, 4096, "relu", "bf16", "f32", True, 0, 0, False),
    (65, 96, 4100, "gelu", "f32", "f32", False, 0, 1, True),
    (129, 257, 72, "silu", "bf16", "f32", True, 0, 1, True),
    (200, 520, 1000, "gelu_tanh", "f32", "bf16", True, 1, 0, True),
    (300, 1100, 64, "gelu", "bf16", "bf16", False, 0, 1, True),
    (512, 512, 2048, "gelu", "bf16", "f32", True, 0, 1, True),
    (1000, 2162, 520, "silu", "f32", "f32", True, 0, 0, False),
    (2048, 5120, 200, "gelu", "bf16", "f32", True, 0, 1, True),
    (512, 512, 4096, "gelu", "f32", "f32", True, 0, 1, True),       # every tile split along K
    (300, 500, 8192, "silu", "bf16", "none", False, 0, 0, False),
    (2560, 4608, 1040, "gelu", "f32", "f32", True, 0, 1, True),     # several tiles a CTA, several chunks
    (2560, 4600, 1040, "gelu_tanh", "bf16", "bf16", True, 0, 0, False),
    (2500, 4601, 840, "silu", "f32", "f32", False, 0, 1, True),
]


def linear_reference(a, b, k, alpha, bias, name, r, c):
    prod, err = ref.product(a, b, k, CHUNK if c == "f32" else None)
    z = alpha * prod + bias
    z_err = np.abs(alpha) * err + ref.U32 * (np.abs(alpha * prod) + np.abs(z))
    h = ref.act(z, name)
    out = h + r
    # |act'| <= 1.13 carries z's error over; one FP32 rounding per sum, then the store's
    tol = 1.2 * z_err + ref.act_error(z, name) + ref.U32 * (np.abs(h) + np.abs(out)) + ref.rounding(out, c == "bf16") * 1.01
    return z, z_err, out, tol


def run_linear(bm, case, alpha=0.75, variant=0, ws=True, seed=0):
    m, n, k, name, c, bias_t, residual, ta, tb, ckpt = case
    rng = np.random.default_rng(seed + m + 7 * n + 13 * k)
    t = torch()
    A, B, a, b = random_operands(rng, m, n, k, ta, tb)
    bias = None if bias_t == "none" else t.from_numpy(rng.normal(size=n)).to(dtype_of(bias_t)).cuda()
    R = padded(rng.normal(size=(m, n)), dtype_of(c)) if residual else None
    C = Out(m, n, dtype_of(c))
    q = Ckpt(m, n) if ckpt else None
    with tile_variant(variant):
        bm.gemm_bias_act(A, B, C.view, bias=bias, act=name, residual=R, alpha=alpha, transA=bool(ta), transB=bool(tb),
                         checkpoint=q.pair if ckpt else None, workspace=workspace() if ws else None)
    t.cuda.synchronize()
    check_no_device_error()
    z, z_err, want, tol = linear_reference(a, b, k, alpha, 0.0 if bias is None else np64(bias), name,
                                           np64(R) if residual else 0.0, c)
    assert_close(np64(C.view), want, tol, "C")
    C.check_guard()
    if ckpt:
        q.check_guard()
        back = ref.decode(*q.arrays(), m, n)
        # E4M3 rounds at 2^-4 of a value (2^-10 of the group's power of two when small) and
        # saturates within 1/8 of the largest
        groups = np.repeat(np.maximum.reduceat(np.abs(z), np.arange(0, n, 32), axis=1), 32, axis=1)[:, :n]
        assert_close(back, z, 0.126 * np.abs(z) + groups * 2.0 ** -16 + 2 * z_err, "checkpoint")


@pytest.mark.parametrize("case", LINEAR, ids=lambda c: "x".join(map(str, c[:3])) + f"_{c[3]}_{c[4]}")
def test_linear(bm, case):
    run_linear(bm, case)


@pytest.mark.parametrize("variant", [1, 2, 3], ids=["single128x256", "single128x128", "pair256x256"])
@pytest.mark.parametrize("case", [LINEAR[9], LINEAR[10], (700, 600, 192, "silu", "bf16", "f32", True, 0, 1, True),
                                  (520, 1032, 1100, "relu", "f32", "f32", True, 0, 1, True)],
                         ids=lambda c: "x".join(map(str, c[:3])))
def test_linear_on_every_tile(bm, case, variant):
    run_linear(bm, case, variant=variant, seed=variant)


def test_linear_without_workspace(bm):
    run_linear(bm, LINEAR[8], ws=False)
    run_linear(bm, LINEAR[12], ws=False)


# tiles of a partly filled last wave run as two halves of their columns (256 x 256 pair tiles)
@pytest.mark.parametrize("c,residual", [("bf16", True), ("f32", False)])
def test_linear_half_units(bm, c, residual):
    st, plan = bm.bm_gemm_bf16_plan(2560, 2304, 576)
    assert st == bm.BM_OK and plan.n_splits == 2, plan.as_dict()
    run_linear(bm, (2560, 2304, 576, "gelu", c, "f32", residual, 0, 1, True))


INTEGER = [(1, 24, 40, 0, 1), (5, 100, 24, 0, 0), (48, 160, 64, 1, 1), (70, 33, 24, 1, 0), (300, 520, 24, 0, 1),
           (513, 1030, 24, 0, 0), (256, 256, 24, 0, 1), (65, 384, 2048, 0, 1)]


@pytest.mark.parametrize("c", ["f32", "bf16"])
@pytest.mark.parametrize("case", INTEGER, ids=lambda c: "x".join(map(str, c[:3])))
def test_linear_integers_bit_for_bit(bm, case, c):
    """Small integers: every FP32 sum is exact, so C, the codes and the scales (padding included) are
    those of exact arithmetic. z = 2 AB + bias has at most 8 significant bits when it is checked
    against the oracle's BF16 quantization rule (ref.quantize equals it)."""
    m, n, k, ta, tb = case
    rng = np.random.default_rng(m + n)
    t = torch()
    sparse = 1.0 if k <= 64 else 0.02   # (keeps |z| below 256 for long K)
    a = rng.integers(-1, 2, (m, k)) * (rng.random((m, k)) < sparse)
    b = rng.integers(-1, 2, (k, n))
    A, B = padded(a.T if ta else a, t.bfloat16), padded(b.T if tb else b, t.bfloat16)
    bias = rng.integers(-3, 4, n)
    r = rng.integers(-4, 5, (m, n))
    R, C, q = padded(r, dtype_of(c)), Out(m, n, dtype_of(c)), Ckpt(m, n)
    z = 2.0 * (a @ b) + bias
    assert np.abs(z).max() < 250
    for ckpt in (True, False):
        bm.gemm_bias_act(A, B, C.view, bias=t.from_numpy(bias).float().cuda(), act="relu", residual=R, alpha=2.0,
                         transA=bool(ta), transB=bool(tb), checkpoint=q.pair if ckpt else None, workspace=workspace())
        assert np.array_equal(np64(C.view), np.maximum(z, 0) + r)
        C.check_guard()
    check_no_device_error()
    codes, scales = q.arrays()
    wq, ws = ref.quantize(z)
    assert np.array_equal(scales, ref.tile_scales(ws, m, n, 0))
    assert np.array_equal(np.where(codes == 128, 0, codes), np.where(wq == 128, 0, wq))  # (the sign of a zero)
    q.check_guard()


def test_linear_residual_may_be_the_output(bm):
    t = torch()
    rng = np.random.default_rng(5)
    for m, n, k, c in [(300, 520, 136, "bf16"), (20, 520, 136, "f32"), (257, 1030, 136, "f32"), (128, 256, 4096, "bf16")]:
        A, B, a, b = random_operands(rng, m, n, k, 0, 1)
        r = padded(rng.normal(size=(m, n)), dtype_of(c), fill=0.0)
        before = np64(r)
        bm.gemm_bias_act(A, B, r, residual=r, transB=True, workspace=workspace())
        _, _, want, tol = linear_reference(a, b, k, 1.0, 0.0, "none", before, c)
        assert_close(np64(r), want, tol, "C")
    check_no_device_error()


@pytest.mark.parametrize("m", [4, 200])
def test_linear_without_products(bm, m):
    """k == 0 or alpha == 0: z is the bias, and A and B are not read (NaN there changes nothing)."""
    t = torch()
    n = 200
    rng = np.random.default_rng(9)
    bias = t.from_numpy(rng.normal(size=n)).float().cuda()
    A, B = padded(np.full((m, 64), np.nan), t.bfloat16), padded(np.full((n, 64), np.nan), t.bfloat16)
    for k, alpha in ((64, 0.0), (0, 1.0)):
        C, q = Out(m, n, t.float32), Ckpt(m, n)
        bm.gemm_bias_act(A[:, :k], B[:, :k], C.view, bias=bias, act="gelu", alpha=alpha, transB=True, checkpoint=q.pair)
        z = np.broadcast_to(np64(bias), (m, n))
        assert_close(np64(C.view), ref.act(z, "gelu"), ref.act_error(z, "gelu"), "C")
        wq, ws = ref.quantize(z)
        codes, scales = q.arrays()
        assert np.array_equal(codes, wq) and np.array_equal(scales, ref.tile_scales(ws, m, n, 0))
        C.check_guard()


@pytest.mark.parametrize("m", [3, 150])
def test_linear_special_values(bm, m):
    """An infinity or a NaN reaches its own row's outputs only, and marks its group of the checkpoint."""
    t = torch()
    n, k = 100, 72
    rng = np.random.default_rng(2)
    a = rng.normal(size=(m, k))
    a[1, 5] = np.inf
    a[2, 7] = np.nan
    A, B = padded(a, t.bfloat16), padded(np.abs(rng.normal(size=(n, k))) + 0.1, t.bfloat16)
    C, q = Out(m, n, t.float32), Ckpt(m, n)
    bm.gemm_bias_act(A, B, C.view, act="relu", transB=True, checkpoint=q.pair, workspace=workspace())
    bm.gemm_bias_act(A, B, C.view, act="relu", transB=True, workspace=workspace())
    got = np64(C.view)
    assert np.isposinf(got[1]).all() and np.isnan(got[2]).all()
    keep = np.arange(m) > 2
    keep[0] = True
    assert np.isfinite(got[keep]).all()
    codes, scales = q.arrays()
    s = scales[ref.scale_offsets(m, n)]
    assert (s[1:3] == 255).all() and (codes[1:3] == 0x7F).all() and (s[keep] != 255).all()
    C.check_guard()


# ------------------------------------------------------------------ backward product
DACT = [
    # m, n, k, act, c, ta, tb
    (1, 40, 64, "gelu", "bf16", 0, 0),
    (1, 1, 8, "silu", "f32", 0, 1),
    (31, 300, 2056, "gelu_tanh", "f32", 0, 0),
    (64, 512, 4096, "silu", "bf16", 0, 0),
    (129, 257, 72, "relu", "bf16", 0, 1),
    (300, 1032, 1000, "gelu", "f32", 1, 0),
    (777, 1320, 520, "silu", "bf16", 0, 0),
    (1000, 2162, 96, "gelu", "f32", 0, 1),
    (2560, 2304, 576, "gelu", "bf16", 0, 0),
    (400, 512, 4096, "gelu", "bf16", 0, 0),        # every tile split along K
    (2560, 4608, 1040, "gelu", "bf16", 0, 0),      # several tiles a CTA, several chunks
    (100, 16400, 72, "silu", "f32", 0, 1),         # few rows, more columns than SMs
]


@pytest.mark.parametrize("variant", [0, 1, 2, 3], ids=["auto", "single128x256", "single128x128", "pair256x256"])
@pytest.mark.parametrize("case", DACT, ids=lambda c: "x".join(map(str, c[:3])) + f"_{c[3]}_{c[4]}")
def test_dact(bm, case, variant):
    m, n, k, name, c, ta, tb = case
    if variant and m * n * k > 600_000_000:
        pytest.skip("the automatic choice covers the largest")
    rng = np.random.default_rng(m + n + k)
    t = torch()
    A, B, a, b = random_operands(rng, m, n, k, ta, tb)
    z = rng.normal(size=(m, n)) * 2.0
    z[0, : min(n, 32)] = 0.0                     # a group of zeros
    q = Ckpt(m, n).fill(z, scale_fill=255)       # (padding entries are never read)
    C = Out(m, n, dtype_of(c))
    dbias = t.full((n + 8,), 7.0, device="cuda")
    ws = workspace(bm.bm_gemm_bf16_dact_workspace_size(m, n, k, 1))
    alpha = -0.5
    with tile_variant(variant):
        bm.gemm_dact(A, B, C.view, q.pair, act=name, dbias=dbias[:n], alpha=alpha, transA=bool(ta), transB=bool(tb),
                     workspace=ws)
    check_no_device_error()
    zq = ref.decode(*q.arrays(), m, n)
    prod, err = ref.product(a, b, k, CHUNK)      # (dbias asks for the chunks)
    g, d = alpha * prod, ref.slope(zq, name)
    want = g * d
    dz_err = np.abs(alpha) * err * np.abs(d) + np.abs(g) * ref.act_error(zq, name) + 2 * ref.U32 * np.abs(want)
    assert_close(np64(C.view), want, dz_err + 1.01 * ref.rounding(want, c == "bf16"), "C")
    # the sums: 5 + ceil(m / 128) additions of FP32 partials and a tree over 32 of them, at most
    sum_err = dz_err.sum(axis=0) + (12 + -(-m // 128)) * ref.U32 * np.abs(want).sum(axis=0)
    assert_close(np64(dbias[:n]), want.sum(axis=0), sum_err, "dbias")
    assert (dbias[n:] == 7.0).all()
    C.check_guard()
    first = (C.raw.clone(), dbias.clone())
    with tile_variant(variant):
        bm.gemm_dact(A, B, C.view, q.pair, act=name, dbias=dbias[:n], alpha=alpha, transA=bool(ta), transB=bool(tb),
                     workspace=ws)
    assert t.equal(first[0], C.raw) and t.equal(first[1], dbias)   # the same bits again
    with tile_variant(variant):
        bm.gemm_dact(A, B, C.view, q.pair, act=name, dbias=dbias[:n], accumulate=True, alpha=alpha, transA=bool(ta),
                     transB=bool(tb), workspace=ws)
    assert t.equal(dbias[:n], 2 * first[1][:n])                    # x + x is exact


def test_dact_least_workspace_and_none(bm):
    t = torch()
    m, n, k = 300, 520, 2048
    rng = np.random.default_rng(4)
    A, B, a, b = random_operands(rng, m, n, k, 0, 0)
    q = Ckpt(m, n).fill(rng.normal(size=(m, n)))
    least = -(-4 * -(-m // 32) * n // 256) * 256
    prod, err = ref.product(a, b, k, CHUNK)
    want = prod * ref.slope(ref.decode(*q.arrays(), m, n), "silu")
    for dbias, ws in ((t.empty(n, device="cuda"), workspace(least)), (None, None)):
        C = Out(m, n, t.float32)
        bm.gemm_dact(A, B, C.view, q.pair, act="silu", dbias=dbias, workspace=ws)
        assert_close(np64(C.view), want, 1.2 * err + np.abs(prod) * 1e-5 + 1e-6, "C")
        if dbias is not None:
            assert_close(np64(dbias), want.sum(axis=0), (1.2 * err + np.abs(prod) * 1e-5 + 1e-6).sum(axis=0), "dbias")
    check_no_device_error()


def test_dact_without_products_and_rows(bm):
    t = torch()
    m, n = 200, 100
    q = Ckpt(m, n).fill(np.ones((m, n)))
    A, B = padded(np.full((m, 64), np.nan), t.bfloat16), padded(np.full((64, n), np.nan), t.bfloat16)
    C, dbias = Out(m, n, t.bfloat16), t.full((n,), 3.0, device="cuda")
    bm.gemm_dact(A, B, C.view, q.pair, act="gelu", dbias=dbias, alpha=0.0, workspace=workspace())
    assert (np64(C.view) == 0).all() and (dbias == 0).all()
    dbias.fill_(3.0)
    none = (q.pair[0][:0], q.pair[1])
    bm.gemm_dact(A[:0], B, C.view[:0], none, act="gelu", dbias=dbias, accumulate=True, workspace=workspace())
    assert (dbias == 3.0).all()
    bm.gemm_dact(A[:0], B, C.view[:0], none, act="gelu", dbias=dbias, workspace=workspace())
    assert (dbias == 0.0).all()
    C.check_guard()


def test_dact_rows_past_the_end_do_not_reach_the_sums(bm):
    """B holds an infinity: rows of the last tile past m (zeros times infinity) stay out of dbias."""
    t = torch()
    m, n, k = 130, 64, 64
    a, b = np.zeros((m, k)), np.ones((k, n))
    a[:, 0] = 1.0
    b[3, 5] = np.inf
    a[:, 3] = 1.0
    A, B = padded(a, t.bfloat16), padded(b, t.bfloat16)
    q = Ckpt(m, n).fill(np.ones((m, n)))
    C, dbias = Out(m, n, t.float32), t.empty(n, device="cuda")
    bm.gemm_dact(A, B, C.view, q.pair, act="relu", dbias=dbias, workspace=workspace())
    got = dbias.cpu().numpy()
    assert np.isposinf(got[5]) and (np.delete(got, 5) == 2.0 * m).all()


@pytest.mark.parametrize("name", ref.ACTS)
def test_gradient_is_a_difference_of_the_forward(bm, name):
    """The library's act' against differences of the library's own act at neighbouring values: decoded
    checkpoints z and z + h on a grid the checkpoint holds exactly (multiples of 1/8 in [1, 2) of each
    group's power of two), so the difference quotient is act' at the midpoint within h^2 |act'''| / 24
    plus the two values' errors over h."""
    t = torch()
    n = 32 * 24
    z = (np.arange(n) % 32 / 16.0 - 1.0)[None, :] * 2.0   # steps of 1/8 in [-2, 2)
    mid, h = z[:, :-1] + 0.0625, 0.125
    H = t.empty((1, n), device="cuda")
    q = Ckpt(1, n).fill(z)
    assert np.array_equal(ref.decode(*q.arrays(), 1, n), z)
    bm.act_mxfp8(q.pair, H, act=name)
    diff = np.diff(np64(H), axis=1) / h
    want = ref.slope(mid, name)
    inside = (np.diff(z, axis=1) > 0)
    tol = h * h * 3.0 / 24 + 2 * ref.act_error(mid, name) / h + 1e-6
    assert (np.abs(diff - want)[inside] <= tol[inside]).all()
    # and the library's act' at the grid itself, through a product with the identity
    one = padded(np.ones((1, 8)) * np.eye(1, 8), t.bfloat16)
    B = padded(np.eye(8, n) * 0 + (np.arange(8) == 0)[:, None], t.bfloat16)
    G = t.empty((1, n), device="cuda")
    bm.gemm_dact(one, B, G, q.pair, act=name)
    assert_close(np64(G), ref.slope(z, name), ref.act_error(z, name) + ref.U32, "act'")


# ------------------------------------------------------------------ activation from the checkpoint
@pytest.mark.parametrize("name", ref.ACTS)
@pytest.mark.parametrize("h", ["f32", "bf16"])
def test_act_every_code_and_scale(bm, name, h):
    """All 256 codes under every scale code of 100 .. 135 and the ends of the range."""
    t = torch()
    scales = np.concatenate([np.arange(100, 136), [0, 1, 2, 50, 200, 245, 246, 255]]).astype(np.uint8)
    rows, n = len(scales), 256
    q = Ckpt(rows, n)
    q.pair[0].copy_(t.arange(256, device="cuda").to(t.uint8).expand(rows, n))
    q.pair[1].copy_(t.from_numpy(ref.tile_scales(np.repeat(scales[:, None], 8, 1), rows, n)).cuda())
    H = Out(rows, n, dtype_of(h))
    bm.act_mxfp8(q.pair, H.view, act=name)
    z = ref.decode(*q.arrays(), rows, n)
    with np.errstate(over="ignore", invalid="ignore"):
        want = np.where(np.isnan(z), np.nan, ref.act(np.clip(z, -1e8, 1e8), name) if name not in ("none", "relu") else
                        ref.act(z, name))
        big = np.abs(z) > 1e8
        want = np.where(big & (name not in ("none", "relu")), np.maximum(z, 0), want)
    got = np64(H.view)
    nan = np.isnan(want)
    assert np.array_equal(nan, np.isnan(got))
    tol = ref.act_error(np.minimum(np.abs(z), 1e30), name)
    tol = np.where(np.abs(z) > 20, np.abs(want) * 1e-6 + 1e-6, tol)
    tol = tol + (ref.rounding(want, True) if h == "bf16" else 0.0) + 2.0 ** -134
    if name in ("none", "relu") and h == "f32":
        assert np.array_equal(got[~nan], want[~nan])
    assert_close(got[~nan], want[~nan], tol[~nan], "H")
    H.check_guard()


@pytest.mark.parametrize("rows,n", [(1, 1), (1, 15), (2, 33), (129, 130), (100, 1320), (5, 5000), (1030, 64)])
@pytest.mark.parametrize("h", ["f32", "bf16"])
def test_act_shapes(bm, rows, n, h):
    rng = np.random.default_rng(rows + n)
    q = Ckpt(rows, n).fill(rng.normal(size=(rows, n)) * 2, scale_fill=255)
    H = Out(rows, n, dtype_of(h))
    bm.act_mxfp8(q.pair, H.view, act="gelu")
    z = ref.decode(*q.arrays(), rows, n)
    want = ref.act(z, "gelu")
    assert_close(np64(H.view), want, ref.act_error(z, "gelu") + ref.rounding(want, h == "bf16"), "H")
    H.check_guard()


# ------------------------------------------------------------------ layer norm
NORM_SHAPES = [(1, 1), (1, 8), (3, 7), (9, 255), (4, 256), (40, 511), (17, 1024), (5, 1025), (33, 2162), (700, 5120),
               (2, 8192), (3, 8200), (2, 16385), (1, 32768), (2, 33001)]


def norm_inputs(rng, rows, n, offset=3.0):
    x = rng.normal(size=(rows, n)) * np.exp(rng.normal(size=n)) + offset * rng.normal(size=(rows, 1))
    return x


@pytest.mark.parametrize("types", [("bf16", "bf16", "f32"), ("f32", "bf16", "bf16"), ("bf16", "f32", "bf16"),
                                   ("f32", "f32", "f32")], ids="_".join)
@pytest.mark.parametrize("shape", NORM_SHAPES, ids=lambda s: f"{s[0]}x{s[1]}")
def test_layernorm(bm, shape, types):
    rows, n = shape
    xt, yt, pt = types
    rng = np.random.default_rng(rows * 7 + n)
    t = torch()
    X = padded(norm_inputs(rng, rows, n), dtype_of(xt))
    gamma = t.from_numpy(rng.normal(size=n) + 1.0).to(dtype_of(pt)).cuda()
    beta = t.from_numpy(rng.normal(size=n)).to(dtype_of(pt)).cuda()
    Y = Out(rows, n, dtype_of(yt))
    mean, rstd = t.full((rows + 1,), 9.0, device="cuda"), t.full((rows + 1,), 9.0, device="cuda")
    eps = 1e-5
    bm.layernorm(X, gamma, beta, Y.view, mean=mean[:rows], rstd=rstd[:rows], eps=eps)
    x, g, b = np64(X), np64(gamma), np64(beta)
    want, m, r = ref.layernorm(x, g, b, eps)
    check_norm(np64(Y.view), np64(mean[:rows]), np64(rstd[:rows]), x, g, b, want, m, r, yt == "bf16")
    assert mean[rows] == 9.0 and rstd[rows] == 9.0
    Y.check_guard()


def check_norm(y, mean, rstd, x, g, b, want, m, r, bf16):
    """Sums of a row: at most 40 roundings deep (8 elements, 4 vectors, 5 + 5 shuffle steps, and up to 5
    more vectors of the long form), each half an ulp of sum |.|."""
    depth = 40 * ref.U32 / 2
    mean_tol = depth * np.abs(x).mean(axis=1) + ref.U32 * np.abs(m)
    assert_close(mean, m, mean_tol + 1e-45, "mean")
    # variance: relative 2 (depth + U32); a wrong mean adds its square (negligible) to it
    var = 1.0 / r ** 2
    rstd_tol = r * (depth + 4 * ref.U32) + r * (mean_tol ** 2) / var
    assert_close(rstd, r, rstd_tol, "rstd")
    d = np.abs(x - m[:, None])
    xh_err = (mean_tol[:, None] + ref.U32 * d) * r[:, None] + d * rstd_tol[:, None] + ref.U32 * d * r[:, None]
    tol = xh_err * np.abs(g) + ref.U32 * (d * r[:, None] * np.abs(g) + np.abs(want)) + 1.01 * ref.rounding(want, bf16)
    assert_close(y, want, tol, "Y")


def test_layernorm_parameters_may_be_missing_and_output_in_place(bm):
    rng = np.random.default_rng(1)
    t = torch()
    x0 = rng.normal(size=(20, 600)) + 50.0
    for gamma, beta in ((None, None), (t.full((600,), 2.0, device="cuda"), None), (None, t.ones(600, device="cuda"))):
        X = padded(x0, t.float32, fill=0.0)
        x = np64(X)
        bm.layernorm(X, gamma, beta, X)
        g = 1.0 if gamma is None else 2.0
        b = 0.0 if beta is None else 1.0
        want, m, r = ref.layernorm(x, g * np.ones(600), b, 1e-5)
        d = np.abs(x - m[:, None])
        tol = (40 * ref.U32 * 51.0 * r[:, None] + 60 * ref.U32 * d * r[:, None]) * g + ref.U32 * np.abs(want)
        assert_close(np64(X), want, tol, "Y")


def test_layernorm_constant_rows_and_special_values(bm):
    """A constant row has variance 0: Y is beta and rstd 1 / sqrt(eps). A NaN or an infinity stays in its row."""
    t = torch()
    x = np.random.default_rng(2).normal(size=(6, 300))
    x[1] = 4.0
    x[2, 10] = np.inf
    x[3, 299] = np.nan
    X, Y = padded(x, t.float32), Out(6, 300, t.float32)
    beta, rstd = t.full((300,), 0.5, device="cuda"), t.empty(6, device="cuda")
    bm.layernorm(X, None, beta, Y.view, rstd=rstd, eps=1e-4)
    y = np64(Y.view)
    assert (y[1] == 0.5).all() and abs(rstd[1].item() - 100.0) < 1e-4
    assert np.isnan(y[2]).all() and np.isnan(y[3]).all()
    assert np.isfinite(y[[0, 1, 4, 5]]).all()


NORM_BWD_SHAPES = [(1, 1), (1, 8), (3, 7), (700, 255), (4, 256), (40, 1025), (301, 2162), (1500, 5120), (2, 8192),
                   (3, 16000), (5, 16400), (2, 33001)]


@pytest.mark.parametrize("types", [("bf16", "bf16", "f32", True), ("f32", "bf16", "bf16", False),
                                   ("bf16", "f32", "bf16", True), ("f32", "f32", "f32", True)],
                         ids=lambda t: "_".join(map(str, t)))
@pytest.mark.parametrize("shape", NORM_BWD_SHAPES, ids=lambda s: f"{s[0]}x{s[1]}")
def test_layernorm_backward(bm, shape, types):
    rows, n = shape
    xt, yt, pt, has_res = types
    rng = np.random.default_rng(rows * 5 + n)
    t = torch()
    X = padded(norm_inputs(rng, rows, n), dtype_of(xt))
    dY = padded(rng.normal(size=(rows, n)), dtype_of(yt))
    dres = padded(rng.normal(size=(rows, n)), dtype_of(xt)) if has_res else None
    gamma = t.from_numpy(rng.normal(size=n) + 1.0).to(dtype_of(pt)).cuda()
    x, dy, g = np64(X), np64(dY), np64(gamma)
    _, m, r = ref.layernorm(x, g, 0.0, 1e-5)
    mean, rstd = t.from_numpy(m).float().cuda(), t.from_numpy(r).float().cuda()
    m, r = np64(mean), np64(rstd)
    dX = Out(rows, n, dtype_of(xt))
    dgamma, dbeta = t.full((n + 8,), 7.0, device="cuda"), t.full((n + 8,), 7.0, device="cuda")
    ws = workspace(bm.bm_layernorm_backward_workspace_size(rows, n))
    args = dict(dres=dres, workspace=ws)
    bm.layernorm_backward(dY, X, gamma, mean, rstd, dX.view, dgamma[:n], dbeta[:n], **args)
    want, wg, wb = ref.layernorm_backward(dy, x, g, m, r)
    res = np64(dres) if has_res else 0.0
    xh = (x - m[:, None]) * r[:, None]
    u = dy * g
    depth = 40 * ref.U32 / 2
    s2 = np.abs((u * xh).mean(axis=1, keepdims=True))
    tol = r[:, None] * (2 * ref.U32 * np.abs(u) + depth * np.abs(u).mean(axis=1, keepdims=True)
                        + np.abs(xh) * (depth + 3 * ref.U32) * np.abs(u * xh).mean(axis=1, keepdims=True)
                        + 3 * ref.U32 * np.abs(xh) * s2 + 2 * ref.U32 * np.abs(want) / r[:, None])
    want = want + res
    tol = tol + ref.U32 * (np.abs(want) + np.abs(res)) + 1.01 * ref.rounding(want, xt == "bf16")
    assert_close(np64(dX.view), want, tol, "dX")
    # column sums: a block's own rows in turn, then the blocks' (at most 32 in turn and a tree)
    depth = (rows / 100 + 45) * ref.U32 / 2
    assert_close(np64(dgamma[:n]), wg, depth * np.abs(dy * xh).sum(axis=0) + 3 * ref.U32 * np.abs(dy * xh).sum(axis=0), "dgamma")
    assert_close(np64(dbeta[:n]), wb, depth * np.abs(dy).sum(axis=0), "dbeta")
    assert (dgamma[n:] == 7.0).all() and (dbeta[n:] == 7.0).all()
    dX.check_guard()
    first = dX.raw.clone(), dgamma.clone(), dbeta.clone()
    bm.layernorm_backward(dY, X, gamma, mean, rstd, dX.view, dgamma[:n], dbeta[:n], **args)
    assert all(t.equal(a, b) for a, b in zip(first, (dX.raw, dgamma, dbeta)))
    bm.layernorm_backward(dY, X, gamma, mean, rstd, dX.view, dgamma[:n], dbeta[:n], accumulate=True, **args)
    assert t.equal(dgamma[:n], 2 * first[1][:n]) and t.equal(dbeta[:n], 2 * first[2][:n])
    bm.layernorm_backward(dY, X, gamma, mean, rstd, dX.view, dres=dres)      # without the parameters' gradients
    assert t.equal(first[0], dX.raw)


@pytest.mark.parametrize("n", [600, 16400])
def test_layernorm_backward_in_place(bm, n):
    """dX over dY, and over dres."""
    t = torch()
    rng = np.random.default_rng(n)
    rows = 50
    X, dY, dres = (padded(rng.normal(size=(rows, n)), t.float32, fill=0.0) for _ in range(3))
    x = np64(X)
    _, m, r = ref.layernorm(x, 1.0, 0.0, 1e-5)
    mean, rstd = t.from_numpy(m).float().cuda(), t.from_numpy(r).float().cuda()
    plain, sums = t.empty_like(X), [t.empty(n, device="cuda") for _ in range(4)]
    ws = workspace(bm.bm_layernorm_backward_workspace_size(rows, n))
    bm.layernorm_backward(dY, X, None, mean, rstd, plain, sums[0], sums[1], dres=dres, workspace=ws)
    for target in ("dY", "dres"):
        y2, r2 = dY.clone(), dres.clone()
        out = y2 if target == "dY" else r2
        bm.layernorm_backward(y2, X, None, mean, rstd, out, sums[2], sums[3], dres=r2, workspace=ws)
        assert t.equal(out, plain) and t.equal(sums[0], sums[2]) and t.equal(sums[1], sums[3])


def test_layernorm_backward_no_rows(bm):
    t = torch()
    n = 64
    X = t.empty((0, n), device="cuda")
    s = t.empty(0, device="cuda")
    dg, db = t.full((n,), 2.0, device="cuda"), t.full((n,), 2.0, device="cuda")
    bm.layernorm_backward(X, X, None, s, s, X, dg, db, accumulate=True)
    assert (dg == 2.0).all()
    bm.layernorm_backward(X, X, None, s, s, X, dg, db)
    assert (dg == 0.0).all() and (db == 0.0).all()


# ------------------------------------------------------------------ streams, graphs, waits
def test_calls_follow_their_stream_and_replay_from_a_graph(bm):
    """The whole set on a side stream, then captured and replayed on new inputs."""
    t = torch()
    m, d, f = 130, 256, 520
    rng = np.random.default_rng(8)
    x = t.from_numpy(rng.normal(size=(m, d))).bfloat16().cuda()
    w = t.from_numpy(rng.normal(size=(f, d)) / 16).bfloat16().cuda()
    y, h, g = t.empty_like(x), t.empty((m, f), dtype=t.bfloat16, device="cuda"), t.empty((m, f), device="cuda")
    mean, rstd, dbias = t.empty(m, device="cuda"), t.empty(m, device="cuda"), t.empty(f, device="cuda")
    dx, dg, db = t.empty_like(x), t.empty(d, device="cuda"), t.empty(d, device="cuda")
    ck, ws = bm.mxfp8_empty(m, f), workspace()

    def step():
        bm.layernorm(x, None, None, y, mean=mean, rstd=rstd)
        bm.gemm_bias_act(y, w, h, act="silu", transB=True, checkpoint=ck, workspace=ws)
        bm.gemm_dact(y, w, g, ck, act="silu", dbias=dbias, transB=True, workspace=ws)
        bm.layernorm_backward(y, x, None, mean, rstd, dx, dg, db, workspace=ws)
        bm.act_mxfp8(ck, h, act="silu")
        return [v.clone() for v in (y, h, g, dbias, dx, dg, db)]

    want = step()
    t.cuda.synchronize()
    side = t.cuda.Stream()
    with t.cuda.stream(side):
        got = step()
    side.synchronize()
    assert all(t.equal(a, b) for a, b in zip(want, got))
    graph = t.cuda.CUDAGraph()
    with t.cuda.graph(graph):
        got = step()
    x2 = t.from_numpy(rng.normal(size=(m, d))).bfloat16().cuda()
    for src in (x2, x.clone()):
        x.copy_(src)
        graph.replay()
        t.cuda.synchronize()
        again = [v.clone() for v in got]
        fresh = step()
        assert all(t.equal(a, b) for a, b in zip(again, fresh))
    assert all(t.equal(a, b) for a, b in zip(want, fresh))
    check_no_device_error()


@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("m", [8, 512])
def test_a_stalled_copy_is_reported_and_the_context_survives(bm, m, backward):
    """A stage whose copy is never issued: the wait runs out, the status says so, the next call is right."""
    t = torch()
    n, k = 512, 256
    rng = np.random.default_rng(6)
    A, B, a, b = random_operands(rng, m, n, k, 0, 1)
    q = Ckpt(m, n).fill(np.ones((m, n)))
    C = Out(m, n, t.float32)

    def call():
        if backward:
            bm.gemm_dact(A, B, C.view, q.pair, act="relu", transB=True)
        else:
            bm.gemm_bias_act(A, B, C.view, transB=True)

    stream = t.cuda.current_stream().cuda_stream
    assert bm.bm_get_last_device_error(stream) == bm.BM_OK
    bm.bm_set_wait_timeout_ms(50)
    bm.bm_debug_inject_stall(1)
    try:
        call()
        assert bm.bm_get_last_device_error(stream) == bm.BM_ERR_TIMEOUT
    finally:
        bm.bm_debug_inject_stall(0)
        bm.bm_set_wait_timeout_ms(2000)
    call()
    assert bm.bm_get_last_device_error(stream) == bm.BM_OK
    prod, err = ref.product(a, b, k, CHUNK)
    assert_close(np64(C.view), prod, err + ref.U32 * np.abs(prod), "C")
