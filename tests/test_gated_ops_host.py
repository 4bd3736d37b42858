"""Refusals and sizes of a gated MLP's operators and of the orthogonalised update (CPU only).

Every call fails its argument checks before any CUDA call, or is a no-op; the pointers are made up."""

import pytest

import blas3_tensor_core_gb300 as bm
from blas3_tensor_core_gb300 import build as bm_build

INVALID, MISALIGNED, WORKSPACE, OK = (bm.BM_ERR_INVALID_VALUE, bm.BM_ERR_MISALIGNED, bm.BM_ERR_WORKSPACE, bm.BM_OK)


@pytest.fixture(scope="module", autouse=True)
def _built():
    bm_build.build()


def glu(m=64, n=64, k=64, ta=0, tb=1, alpha=1.0, A=0x1000, lda=64, BG=0x2000, ldbg=64, BU=0x3000, ldbu=64, act=4,
        H=0x4000, ldh=64, G=None, ldg=0, U=None, ldu=0):
    return bm.bm_gemm_bf16_glu(m, n, k, ta, tb, alpha, A, lda, BG, ldbg, BU, ldbu, act, H, ldh, G, ldg, U, ldu, None)


KEPT = dict(G=0x5000, ldg=64, U=0x6000, ldu=64)


@pytest.mark.parametrize("change,status", [
    (dict(m=-1), INVALID), (dict(n=-2), INVALID), (dict(k=2 ** 31), INVALID), (dict(n=2 ** 30, ldh=2 ** 30), INVALID),
    (dict(ta=2), INVALID), (dict(tb=-1), INVALID), (dict(act=5), INVALID), (dict(act=-1), INVALID),
    (dict(lda=63), INVALID), (dict(ldbg=8), INVALID), (dict(ldbu=56), INVALID), (dict(ldh=32), INVALID),
    (dict(tb=0, k=8, n=72, ldbg=72, ldh=72, ldbu=64), INVALID),
    (dict(H=None), INVALID), (dict(A=None), INVALID), (dict(BG=None), INVALID), (dict(BU=None), INVALID),
    (dict(KEPT, G=None), INVALID), (dict(KEPT, U=None), INVALID), (dict(KEPT, ldg=56), INVALID),
    (dict(KEPT, ldu=56), INVALID), (dict(A=0x1008), MISALIGNED), (dict(BG=0x2002), MISALIGNED),
    (dict(BU=0x3008), MISALIGNED), (dict(H=0x4004), MISALIGNED), (dict(lda=68), MISALIGNED), (dict(ldbu=66), MISALIGNED),
    (dict(ldh=68), MISALIGNED), (dict(KEPT, G=0x5008), MISALIGNED), (dict(KEPT, ldu=68), MISALIGNED),
    (dict(m=0), OK), (dict(n=0), OK), (dict(m=0, H=None), OK),
])
def test_glu_refusals(change, status):
    assert glu(**change) == status


def dglu(m=64, n=64, k=64, ta=0, tb=0, alpha=1.0, A=0x1000, lda=64, B=0x2000, ldb=64, G=0x3000, ldg=64, U=0x4000, ldu=64,
         act=4, dG=0x5000, lddg=64, dU=0x6000, lddu=64, H=None, ldh=0):
    return bm.bm_gemm_bf16_dglu(m, n, k, ta, tb, alpha, A, lda, B, ldb, G, ldg, U, ldu, act, dG, lddg, dU, lddu, H, ldh,
                                None)


@pytest.mark.parametrize("change,status", [
    (dict(m=-1), INVALID), (dict(k=-1), INVALID), (dict(n=2 ** 31), INVALID), (dict(ta=3), INVALID), (dict(act=7), INVALID),
    (dict(lda=32), INVALID), (dict(ldb=32), INVALID), (dict(ldg=60), INVALID), (dict(ldu=60), INVALID),
    (dict(lddg=60), INVALID), (dict(lddu=60), INVALID), (dict(H=0x7000, ldh=60), INVALID), (dict(G=None), INVALID),
    (dict(U=None), INVALID), (dict(dG=None), INVALID), (dict(dU=None), INVALID), (dict(A=None), INVALID),
    (dict(B=None), INVALID), (dict(G=0x3002), MISALIGNED), (dict(U=0x4008), MISALIGNED), (dict(dG=0x5008), MISALIGNED),
    (dict(dU=0x6004), MISALIGNED), (dict(H=0x7008, ldh=64), MISALIGNED), (dict(H=0x7000, ldh=68), MISALIGNED),
    (dict(ldg=66), MISALIGNED), (dict(lddu=68), MISALIGNED), (dict(ldb=66), MISALIGNED), (dict(A=0x1001), MISALIGNED),
    (dict(m=0), OK), (dict(n=0), OK), (dict(n=0, G=None, dU=None), OK),
])
def test_dglu_refusals(change, status):
    assert dglu(**change) == status


def orth(m=64, n=64, alpha=1.0, X=0x1000, ldx=64, xt=1, steps=5, coeffs=None, eps=1e-7, beta=0.0, C=0x2000, ldc=64,
         ws=0x3000, wsb=1 << 30):
    return bm.bm_orthogonalize_bf16(m, n, alpha, X, ldx, xt, steps, coeffs, eps, beta, C, ldc, ws, wsb, None)


@pytest.mark.parametrize("change,status", [
    (dict(m=-1), INVALID), (dict(n=2 ** 31), INVALID), (dict(xt=2), INVALID), (dict(steps=0), INVALID),
    (dict(steps=65), INVALID), (dict(steps=-1), INVALID), (dict(eps=-1e-9), INVALID), (dict(eps=float("nan")), INVALID),
    (dict(eps=float("inf")), INVALID), (dict(ldx=56), INVALID), (dict(ldc=56), INVALID), (dict(X=None), INVALID),
    (dict(C=None), INVALID), (dict(X=0x1008), MISALIGNED), (dict(C=0x2008), MISALIGNED), (dict(ldx=68), MISALIGNED),
    (dict(ldx=66, xt=0), MISALIGNED), (dict(ldc=68), MISALIGNED), (dict(ws=None, wsb=0), WORKSPACE),
    (dict(ws=None), WORKSPACE), (dict(ws=0x3010), WORKSPACE), (dict(wsb=4096), WORKSPACE),
    (dict(m=0), OK), (dict(n=0), OK), (dict(m=0, C=None, ws=None, wsb=0), OK),
])
def test_orthogonalize_refusals(change, status):
    assert orth(**change) == status


def test_orthogonalize_workspace():
    size = bm.orthogonalize_workspace_size
    assert size(0, 64) == size(64, 0) == size(-1, 64) == 0
    for m, n in ((1, 1), (7, 1000), (1000, 7), (1024, 1024), (16384, 4096), (100000, 65536)):
        s = min(m, n)
        floor = 8 * m * n + 4 * s * s + 8 * s
        assert size(m, n) % 256 == 0 and floor <= size(m, n) <= 1.01 * floor + 128 * (m + s) + (33 << 20)
        assert orth(m=m, n=n, ldx=-(-n // 8) * 8, ldc=-(-n // 8) * 8, wsb=size(m, n) - 1) == WORKSPACE


def test_helpers_refuse_before_the_library():
    torch = pytest.importorskip("torch")
    b = torch.zeros(8, 64, dtype=torch.bfloat16)
    h = torch.zeros(8, 8, dtype=torch.bfloat16)
    f = torch.zeros(8, 64)
    with pytest.raises(TypeError, match="bfloat16"):
        bm.gemm_glu(f, b, b, h, transB=True)
    with pytest.raises(ValueError, match="inconsistent"):
        bm.gemm_glu(b, b, b, b, transB=True)
    with pytest.raises(ValueError, match="one type and shape"):
        bm.gemm_glu(b, b, b[:4], h, transB=True)
    with pytest.raises(ValueError, match="kept together"):
        bm.gemm_glu(b, b, b, h, gate=h, transB=True)
    with pytest.raises(ValueError, match="CUDA"):
        bm.gemm_glu(b, b, b, h, transB=True)
    with pytest.raises(ValueError, match="CUDA"):
        bm.gemm_dglu(b, b, h, h, h, h, transB=True)
    with pytest.raises(ValueError, match="CUDA"):
        bm.orthogonalize(b, b)
    with pytest.raises(TypeError, match="H must be bfloat16"):
        bm._bf16_rows(f, "H", 8, 64)
    with pytest.raises(ValueError, match="must be"):
        bm._bf16_rows(b, "H", 8, 63)
    assert bm._bf16_rows(None, "gate", 8, 64) == (None, 0)
