"""Paths of the operators around an MLP's products that the shape lists of test_mlp_ops_gpu.py do not
reach, and properties of them that one call cannot show."""

import numpy as np
import pytest

import mlp_ref as ref
import test_mlp_ops_gpu as ops
from gpu_helpers import check_no_device_error, tile_variant, torch
from test_mlp_ops_gpu import (_built, assert_close, bm, Ckpt, dtype_of, np64,  # noqa: F401 (fixtures)
                              Out, padded, random_operands, workspace)

pytestmark = pytest.mark.gpu


def integers(gen, lo, hi, rows, cols, dtype):
    """Random integers in rows of a multiple of 16 bytes, with NaN behind them."""
    t = torch()
    buf = t.full((rows, -(-cols // 8) * 8 + 8), float("nan"), dtype=dtype, device="cuda")
    buf[:, :cols] = t.randint(lo, hi, (rows, cols), generator=gen, device="cuda").to(dtype)
    return buf[:, :cols]


# ------------------------------------------------------------------ fused products
@pytest.mark.parametrize("variant", [0, 1, 2, 3], ids=["auto", "single128x256", "single128x128", "pair256x256"])
@pytest.mark.parametrize("m,n,c", [(1111, 2162, "f32"), (3000, 4601, "f32"), (2500, 4601, "bf16"), (140, 35, "bf16")])
def test_residual_into_rows_off_16_bytes(bm, m, n, c, variant):
    """Rows of C that end off a 16-byte boundary are stored from the block that the residual's next
    piece is copied into, piece after piece and tile after tile (3000 x 4601: several a CTA). Integers,
    so that every element is exact; again and again, into a C that holds NaN and over the residual."""
    t = torch()
    k = 24
    gen = t.Generator(device="cuda").manual_seed(m + variant)
    A, B = integers(gen, -1, 2, m, k, t.bfloat16), integers(gen, -1, 2, n, k, t.bfloat16)
    most = 100 if c == "bf16" else 1 << 20
    R = integers(gen, -most, most, m, n, dtype_of(c))
    want = (A.double() @ B.double().T + R.double()).to(dtype_of(c))
    with tile_variant(variant):
        for turn in range(8):
            C = Out(m, n, dtype_of(c))
            C.view.copy_(R) if turn % 2 else C.view.fill_(float("nan"))
            bm.gemm_bias_act(A, B, C.view, residual=C.view if turn % 2 else R, transB=True)
            assert t.equal(C.view, want)
            C.check_guard()
    check_no_device_error()


@pytest.mark.parametrize("m", [20, 300])
@pytest.mark.parametrize("bias_t", ["f32", "bf16"])
def test_a_bias_that_the_call_before_wrote(bm, m, bias_t):
    """The call starts while the one before it, which writes the bias into the same buffer each time,
    still runs; no host work lies between the two. Integers: exact."""
    t = torch()
    n, k = 1056, 64
    gen = t.Generator(device="cuda").manual_seed(m)
    A, B = integers(gen, -1, 2, m, k, t.bfloat16), integers(gen, -1, 2, n, k, t.bfloat16)
    rows = [integers(gen, -8, 9, 64, n, t.bfloat16) for _ in range(6)]
    ones = t.ones((1, 64), dtype=t.bfloat16, device="cuda")
    row = t.zeros((1, n), dtype=dtype_of(bias_t), device="cuda")
    outs = [t.empty((m, n), device="cuda") for _ in range(24)]
    t.cuda.synchronize()
    for i, C in enumerate(outs):
        bm.gemm(ones, rows[i % 6], row, alpha=0.125 if bias_t == "bf16" else 1.0)
        bm.gemm_bias_act(A, B, C, bias=row[0], transB=True)
    product = A.double() @ B.double().T
    for i, C in enumerate(outs):
        bias = rows[i % 6].double().sum(dim=0)
        bias = (bias * 0.125).to(t.bfloat16).double() if bias_t == "bf16" else bias
        assert t.equal(C.double(), product + bias)


def test_quantization_of_what_the_call_before_wrote(bm):
    t = torch()
    m, n, k = 256, 512, 64
    gen = t.Generator(device="cuda").manual_seed(3)
    A = integers(gen, -1, 2, m, k, t.bfloat16)
    weights = [integers(gen, -1, 2, n, k, t.bfloat16) for _ in range(6)]
    X = t.empty((m, n), dtype=t.bfloat16, device="cuda")
    pairs = [bm.mxfp8_empty(m, n) for _ in range(24)]
    stream = t.cuda.current_stream().cuda_stream
    t.cuda.synchronize()
    for i, (q, s) in enumerate(pairs):
        bm.gemm(A, weights[i % 6], X, transB=True)
        assert bm.bm_quantize_mxfp8(m, n, X.data_ptr(), n, q.data_ptr(), n, s.data_ptr(), stream) == bm.BM_OK
    for i, (q, s) in enumerate(pairs):
        codes, scales = ref.quantize(np64(A) @ np64(weights[i % 6]).T)
        assert np.array_equal(np.where(q.cpu().numpy() == 128, 0, q.cpu().numpy()), np.where(codes == 128, 0, codes))
        assert np.array_equal(s.cpu().numpy(), ref.tile_scales(scales, m, n))


# ------------------------------------------------------------------ precision of the products
def chunk_error(parts):
    """The stated bound of the relative error (of norms) that the tensor core's truncation leaves in a
    product whose K runs through accumulators in parts of so many k-blocks of 64."""
    parts = np.asarray(parts, np.float64)
    return 7e-8 * np.sqrt((parts ** 3).sum() / parts.sum())


def tile_parts(k, codes):
    """The tile kernel's parts of K for an FP32 output or a checkpoint, as its chunk rule states them."""
    kb = -(-k // 64)
    if kb >= 24:
        first, rest = (16 if kb >= 48 and not codes else 12), 8
    elif codes and kb > 2:
        first = rest = min(6, (kb + 1) // 2)
    elif kb > 12:
        first, rest = (kb + 1) // 2, 8
    else:
        first = rest = kb
    first, rest = -(-first // 2) * 2, -(-rest // 2) * 2      # (two k-blocks a stage)
    parts = [min(first, kb)] + ([min(first, kb - first)] if kb > first else [])
    while sum(parts) < kb:
        parts.append(min(rest, kb - sum(parts)))
    return parts


def off(got, want):
    return np.linalg.norm(np64(got) - want) / np.linalg.norm(want)


def check_precision(bm, m, n, k, codes, bound, variant=0, trans_a=False):
    """FP32 C (beside a checkpoint: its codes too) and dbias against 64 bits, as relative errors of norms."""
    t = torch()
    gen = t.Generator(device="cuda").manual_seed(m + n + k)
    A = t.randn((k, -(-m // 8) * 8) if trans_a else (m, k), generator=gen, device="cuda").bfloat16()
    A = A[:, :m] if trans_a else A
    B = (t.randn((n, k), generator=gen, device="cuda") / k ** 0.5).bfloat16()
    z = (np64(A).T if trans_a else np64(A)) @ np64(B).T
    C, q = t.full((m, n), float("nan"), device="cuda"), Ckpt(m, n)
    with tile_variant(variant):
        bm.gemm_bias_act(A, B, C, transA=trans_a, transB=True, checkpoint=q.pair if codes else None)
    assert off(C, z) <= bound
    if codes:
        # C is z here: scales and codes are exactly those of its FP32 values
        codes_got, scales = q.arrays()
        scales = scales[ref.scale_offsets(m, n)]
        wq, ws = ref.quantize(np64(C))
        assert np.array_equal(codes_got, wq) and np.array_equal(scales, ws)
        # Against those of the 64-bit z: a group's scale may be its neighbour where the largest value
        # lies within z's error of a power of two (ten times the error's norm, for one element); in the
        # others a code may be the nearest value's neighbour, on the other side of a tie within z's
        # error. The normal z of these inputs lie 40 to 60 ties per unit of their standard deviation
        # apart, so 100 errors bound the share.
        wq, ws = ref.quantize(z)
        peak = np.maximum.reduceat(np.abs(z), np.arange(0, n, 32), axis=1)[scales != ws]
        power = 2.0 ** np.round(np.log2(peak))
        assert (np.abs(peak - power) <= 10 * bound * z.std()).all()
        differ = (codes_got != wq) & np.repeat(scales == ws, 32, axis=1)[:, :n]
        assert differ.mean() <= 100 * bound
        step = np.abs(codes_got[differ].astype(int) - wq[differ].astype(int))
        tiny = np.abs(ref.decode(*q.arrays(), m, n)[differ]) < 1e-3       # (or the sign of a 0)
        assert ((step == 1) | tiny).all()
        return
    dbias, G = t.full((n,), float("nan"), device="cuda"), t.full((m, n), float("nan"), device="cuda")
    ones = Ckpt(m, n).fill(np.ones((m, n)))
    ws = workspace(-(-(4 * -(-m // 32) * -(-n // 4) * 4) // 256) * 256)      # (the least: no split along K)
    with tile_variant(variant):
        bm.gemm_dact(A, B, G, ones.pair, dbias=dbias, transA=trans_a, transB=True, workspace=ws)
    assert off(G, z) <= bound
    assert off(dbias, z.sum(axis=0)) <= bound + 4 * ref.U32   # (FP32 sums of m values, in a tree)
    check_no_device_error()


@pytest.mark.parametrize("variant", [1, 2, 3], ids=["single128x256", "single128x128", "pair256x256"])
@pytest.mark.parametrize("k", [512, 1000, 1536, 2048, 4096, 8192])
@pytest.mark.parametrize("codes", [False, True], ids=["f32", "checkpoint"])
def test_precision_of_chunked_products(bm, k, codes, variant):
    """The stated error of the parts of K; K in one piece (1.1e-9 K) does not meet it."""
    parts = tile_parts(k, codes)
    bound = chunk_error(parts)
    assert len(parts) == 1 or bound < 0.9 * 1.1e-9 * k
    check_precision(bm, 768, 1024, k, codes, bound, variant)
    if codes and k >= 4096:
        assert bound <= 1.15 * 1.5e-10 * k      # an FP32 product's own error at these lengths


@pytest.mark.parametrize("codes", [False, True], ids=["f32", "checkpoint"])
@pytest.mark.parametrize("m,n,k,trans_a,chunk", [
    # the longest chunk in k-blocks (8, or 4 beside a checkpoint, where they fit the tensor memory)
    (8, 2048, 8192, False, (8, 4)), (24, 4096, 4096, False, (8, 4)), (64, 4096, 8192, False, (8, 4)),
    (100, 4096, 8192, False, (8, 8)), (128, 2048, 4096, False, (8, 4)),
    (40, 4096, 8192, True, (8, 4)), (20, 16400, 8192, True, (16, 16)),   # one CTA a tile: 128 k-blocks in 8 parts
    (20, 16400, 16384, True, (32, 32)),
])
def test_precision_of_few_rows(bm, m, n, k, trans_a, chunk, codes):
    bound = chunk_error([chunk[codes]])
    assert bound < 0.25 * 1.1e-9 * k
    check_precision(bm, m, n, k, codes, bound, trans_a=trans_a)


# ------------------------------------------------------------------ layer norm
def test_layernorm_of_rows_past_65535_strips(bm):
    """Two rows of 2^27 + 8 columns, both directions, against 64 bits on the device. A thread adds up to
    2^17 + 8 elements in turn before the tree (10 steps), each sum with half an ulp of sum |.|."""
    t = torch()
    rows, n = 2, (1 << 27) + 8
    gen = t.Generator(device="cuda").manual_seed(1)
    X, dY = (t.randn((rows, n), generator=gen, device="cuda").bfloat16() for _ in range(2))
    gamma = (1.0 + 0.2 * t.randn(n, generator=gen, device="cuda")).bfloat16()
    Y, dX = (t.full_like(X, float("nan")) for _ in range(2))
    mean, rstd = t.empty(rows, device="cuda"), t.empty(rows, device="cuda")
    bm.layernorm(X, gamma, None, Y, mean=mean, rstd=rstd)
    dgamma, dbeta = t.full((n,), float("nan"), device="cuda"), t.full((n,), float("nan"), device="cuda")
    ws = t.empty(bm.bm_layernorm_backward_workspace_size(rows, n), dtype=t.uint8, device="cuda")
    bm.layernorm_backward(dY, X, gamma, mean, rstd, dX, dgamma, dbeta, workspace=ws)
    check_no_device_error()
    depth = ((1 << 17) + 18) * ref.U32 / 2
    sums = t.zeros(n, dtype=t.float64, device="cuda"), t.zeros(n, dtype=t.float64, device="cuda")
    size = t.zeros(n, dtype=t.float64, device="cuda")
    for r in range(rows):
        x, dy, g = X[r].double(), dY[r].double(), gamma.double()
        m = x.mean()
        s = 1.0 / ((x - m).square().mean() + 1e-5).sqrt()
        assert abs(mean[r] - m) <= depth * x.abs().mean() + 1e-7
        assert abs(rstd[r] / s - 1) <= depth + 1e-6
        m, s = mean[r].double(), rstd[r].double()
        xh, u = (x - m) * s, dy * g
        y = xh * g
        assert ((Y[r].double() - y).abs() <= y.abs() * 2.0 ** -8 * 1.01 + 1e-6).all()
        want = s * (u - u.mean() - xh * (u * xh).mean())
        slack = 1.1 * depth * (u.abs().mean() + xh.abs() * (u * xh).abs().mean())
        assert ((dX[r].double() - want).abs() <= want.abs() * 2.0 ** -8 * 1.01 + slack + 1e-6).all()
        sums[0].add_(dy * xh)
        sums[1].add_(dy)
        size.add_((dy * xh).abs())
    assert ((dgamma.double() - sums[0]).abs() <= 8 * ref.U32 * size + 1e-6).all()
    assert ((dbeta.double() - sums[1]).abs() <= 1e-6 + 2 * ref.U32 * (dY[0].double().abs() + dY[1].double().abs())).all()


TYPES = [("bf16", "bf16", "f32"), ("f32", "bf16", "bf16"), ("bf16", "f32", "bf16"), ("f32", "f32", "f32")]


@pytest.mark.parametrize("types", TYPES, ids="_".join)
@pytest.mark.parametrize("shape", [
    # a warp per row: one, two and four vectors a lane, whole and partly filled, odd row counts
    (608, 1), (613, 255), (2500, 256), (13001, 96), (1300, 511), (1300, 512), (700, 1023), (2501, 1000),
    # the ring with a partly filled last vector, and more rows a block than it has stages
    (4001, 1025), (3101, 2162), (2001, 5117), (1001, 10239)], ids=lambda s: f"{s[0]}x{s[1]}")
def test_layernorm_of_many_rows(bm, shape, types):
    ops.test_layernorm(bm, shape, types)


@pytest.mark.parametrize("rows,n", [(701, 260), (2003, 700), (3103, 2166)])
def test_layernorm_of_many_rows_in_place_and_special_values(bm, rows, n):
    """Y over X; a NaN or an infinity stays in its row, and a constant row gives beta."""
    t = torch()
    x = np.random.default_rng(n).normal(size=(rows, n)) + 20.0
    x[1] = 4.0
    x[rows // 2, n - 1] = np.inf
    x[rows - 2, 3] = np.nan
    X = padded(x, t.float32)
    x = np64(X)
    beta, rstd = t.full((n,), 0.5, device="cuda"), t.empty(rows, device="cuda")
    Y = Out(rows, n, t.float32)
    bm.layernorm(X, None, beta, Y.view, eps=1e-4)
    bm.layernorm(X, None, beta, X, rstd=rstd, eps=1e-4)
    y = np64(X)
    bad = np.zeros(rows, bool)
    bad[[rows // 2, rows - 2]] = True
    assert np.isnan(y[bad]).all() and (y[1] == 0.5).all() and abs(rstd[1].item() - 100.0) < 1e-4
    want, m, r = ref.layernorm(x[~bad], 1.0, 0.5, 1e-4)
    d = np.abs(x[~bad] - m[:, None]) * r[:, None]
    assert_close(y[~bad], want, 40 * ref.U32 * 25.0 * r[:, None] + 60 * ref.U32 * d + ref.U32 * np.abs(want), "Y")
    assert np.array_equal(np64(Y.view)[~bad], y[~bad]) and np.isnan(np64(Y.view)[bad]).all()
    Y.check_guard()


@pytest.mark.parametrize("types", [(*p, i != 1) for i, p in enumerate(TYPES)], ids=lambda t: "_".join(map(str, t)))
@pytest.mark.parametrize("shape", [(12001, 255), (12001, 512), (6001, 1030), (5501, 2162), (701, 16000), (601, 11999)],
                         ids=lambda s: f"{s[0]}x{s[1]}")
def test_layernorm_backward_of_many_rows(bm, shape, types):
    """More rows a block than its ring has stages, with and without a partly filled last vector."""
    ops.test_layernorm_backward(bm, shape, types)


# ------------------------------------------------------------------ few rows, more column tiles than half the SMs
@pytest.mark.parametrize("c", ["f32", "bf16"])
@pytest.mark.parametrize("m,ta,tb", [(1, 0, 1), (20, 0, 0), (32, 0, 1), (30, 1, 0)])
def test_few_rows_of_many_columns(bm, m, ta, tb, c):
    """129 column tiles: one CTA each, whose ring wraps (33 k-blocks), forward and backward."""
    ops.run_linear(bm, (m, 16400, 2056, "gelu", c, "f32", True, ta, tb, True))
    ops.test_dact(bm, (m, 16400, 2056, "silu", c, ta, tb), 0)


# ------------------------------------------------------------------ every call writes its outputs
@pytest.mark.parametrize("m,n,k", [(31, 300, 2056), (300, 1032, 1000), (400, 512, 4096), (2560, 4608, 1040)])
def test_products_write_the_same_bits_again(bm, m, n, k):
    t = torch()
    rng = np.random.default_rng(m)
    A, B, _, _ = random_operands(rng, m, n, k, 0, 1)
    bias = t.from_numpy(rng.normal(size=n)).float().cuda()
    R = padded(rng.normal(size=(m, n)), t.float32)
    ws = workspace(max(bm.bm_gemm_bf16_dact_workspace_size(m, n, k, 1), 32 << 20))
    runs = []
    for _ in range(3):
        C, G, q = Out(m, n, t.float32), Out(m, n, t.bfloat16), Ckpt(m, n)
        plain, dbias = Out(m, n, t.float32), t.full((n,), float("nan"), device="cuda")
        for o in (C, G, plain):
            o.view.fill_(float("nan"))
        bm.gemm_bias_act(A, B, C.view, bias=bias, act="gelu", residual=R, transB=True, checkpoint=q.pair, workspace=ws)
        bm.gemm_bias_act(A, B, plain.view, bias=bias, act="gelu", residual=R, transB=True, workspace=ws)
        bm.gemm_dact(A, B, G.view, q.pair, act="gelu", dbias=dbias, transB=True, workspace=ws)
        assert not any(v.isnan().any() for v in (C.view, plain.view, G.view, dbias))
        twice = dbias.clone()
        bm.gemm_dact(A, B, G.view, q.pair, act="gelu", dbias=twice, accumulate=True, transB=True, workspace=ws)
        assert t.equal(twice, 2 * dbias)
        runs.append([v.clone() for v in (C.raw, plain.raw, G.raw, dbias, q.codes.raw, q.raw_scales)])
    assert all(t.equal(a, b) for other in runs[1:] for a, b in zip(runs[0], other))
    check_no_device_error()


@pytest.mark.parametrize("c", ["f32", "bf16"])
@pytest.mark.parametrize("case", ops.INTEGER, ids=lambda c: "x".join(map(str, c[:3])))
def test_integers_without_a_checkpoint(bm, case, c):
    m, n, k, ta, tb = case
    rng = np.random.default_rng(m + n)
    t = torch()
    a = rng.integers(-1, 2, (m, k)) * (rng.random((m, k)) < (1.0 if k <= 64 else 0.02))
    b = rng.integers(-1, 2, (k, n))
    A, B = padded(a.T if ta else a, t.bfloat16), padded(b.T if tb else b, t.bfloat16)
    bias, r = rng.integers(-3, 4, n), rng.integers(-4, 5, (m, n))
    z = 2.0 * (a @ b) + bias
    assert np.abs(z).max() < 250
    C = Out(m, n, dtype_of(c))
    C.view.fill_(float("nan"))
    bm.gemm_bias_act(A, B, C.view, bias=t.from_numpy(bias).float().cuda(), act="relu", residual=padded(r, dtype_of(c)),
                     alpha=2.0, transA=bool(ta), transB=bool(tb), workspace=workspace())
    assert np.array_equal(np64(C.view), np.maximum(z, 0) + r)
    C.check_guard()


@pytest.mark.parametrize("rows,n", [(700, 255), (301, 2162), (5, 16400), (3000, 5120)])
def test_layernorm_backward_writes_the_same_bits_again(bm, rows, n):
    t = torch()
    rng = np.random.default_rng(rows)
    X, dY = (padded(rng.normal(size=(rows, n)), t.bfloat16) for _ in range(2))
    _, m, r = ref.layernorm(np64(X), 1.0, 0.0, 1e-5)
    mean, rstd = t.from_numpy(m).float().cuda(), t.from_numpy(r).float().cuda()
    ws = workspace(bm.bm_layernorm_backward_workspace_size(rows, n))
    runs = []
    for sums in (True, True, False):
        dX = Out(rows, n, t.bfloat16)
        dX.view.fill_(float("nan"))
        dgamma, dbeta = (t.full((n,), float("nan"), device="cuda") if sums else None for _ in range(2))
        bm.layernorm_backward(dY, X, None, mean, rstd, dX.view, dgamma, dbeta, workspace=ws if sums else None)
        assert not dX.view.isnan().any() and not (sums and (dgamma.isnan().any() or dbeta.isnan().any()))
        runs.append((dX.raw, dgamma, dbeta))
    assert all(t.equal(a, b) for a, b in zip(runs[0], runs[1])) and t.equal(runs[0][0], runs[2][0])


def test_calls_on_a_side_stream_write_their_outputs(bm):
    """The outputs hold NaN, set on that stream, when the calls begin; nothing runs on the default one."""
    t = torch()
    m, d, f = 130, 256, 520
    rng = np.random.default_rng(8)
    x, w = padded(rng.normal(size=(m, d)), t.bfloat16), padded(rng.normal(size=(f, d)) / 16, t.bfloat16)
    runs = []
    for stream in (t.cuda.current_stream(), t.cuda.Stream()):
        stream.wait_stream(t.cuda.current_stream())
        with t.cuda.stream(stream):
            y, h = t.empty((m, d), dtype=t.bfloat16, device="cuda"), t.empty((m, f), dtype=t.bfloat16, device="cuda")
            g, dx = t.empty((m, f), device="cuda"), t.empty((m, d), dtype=t.bfloat16, device="cuda")
            vectors = [t.empty(s, device="cuda") for s in (m, m, f, d, d)]
            outs = [y, h, g, dx, *vectors]
            for v in outs:
                v.fill_(float("nan"))
            mean, rstd, dbias, dg, db = vectors
            ck, ws = bm.mxfp8_empty(m, f), workspace()
            bm.layernorm(x, None, None, y, mean=mean, rstd=rstd)
            bm.gemm_bias_act(y, w, h, act="silu", transB=True, checkpoint=ck, workspace=ws)
            bm.gemm_dact(y, w, g, ck, act="silu", dbias=dbias, transB=True, workspace=ws)
            bm.layernorm_backward(y, x, None, mean, rstd, dx, dg, db, workspace=ws)
            again = t.full_like(h, float("nan"))
            bm.act_mxfp8(ck, again, act="silu")
        stream.synchronize()
        runs.append([*outs, again])
    assert not any(v.isnan().any() for v in runs[1])
    assert all(t.equal(a, b) for a, b in zip(*runs))
    check_no_device_error()
