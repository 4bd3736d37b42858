"""Refusals and sizes of the operators around an MLP's products (CPU only).

Every call fails its argument checks before any CUDA call, or is a no-op; the pointers are made up."""

import pytest

import blas3_tensor_core_gb300 as bm
from blas3_tensor_core_gb300 import build as bm_build

INVALID, MISALIGNED, WORKSPACE, OK = (bm.BM_ERR_INVALID_VALUE, bm.BM_ERR_MISALIGNED, bm.BM_ERR_WORKSPACE, bm.BM_OK)


@pytest.fixture(scope="module", autouse=True)
def _built():
    bm_build.build()


def linear(m=64, n=64, k=64, ta=0, tb=1, alpha=1.0, A=0x1000, lda=64, B=0x2000, ldb=64, bias=0x3000, bt=0, act=2,
           R=None, ldr=0, C=0x4000, ldc=64, ct=1, Q=None, ldq=0, S=None, ws=None, wsb=0):
    return bm.bm_gemm_bf16_bias_act(m, n, k, ta, tb, alpha, A, lda, B, ldb, bias, bt, act, R, ldr, C, ldc, ct, Q, ldq, S,
                                    ws, wsb, None)


@pytest.mark.parametrize("change,status", [
    (dict(m=-1), INVALID), (dict(n=-2), INVALID), (dict(k=2 ** 31), INVALID), (dict(ta=2), INVALID),
    (dict(act=5), INVALID), (dict(act=-1), INVALID), (dict(ct=2), INVALID), (dict(bt=2), INVALID),
    (dict(lda=63), INVALID), (dict(ldb=8), INVALID), (dict(ldc=32), INVALID), (dict(C=None), INVALID),
    (dict(A=None), INVALID), (dict(B=None), INVALID), (dict(Q=0x5000, ldq=64), INVALID),
    (dict(S=0x5000), INVALID), (dict(Q=0x5000, ldq=48, S=0x6000), INVALID), (dict(R=0x7000, ldr=56), INVALID),
    (dict(A=0x1008), MISALIGNED), (dict(C=0x4004), MISALIGNED), (dict(bias=0x3004), MISALIGNED),
    (dict(R=0x7008, ldr=64), MISALIGNED), (dict(R=0x7000, ldr=68), MISALIGNED), (dict(ldc=68), MISALIGNED),
    (dict(Q=0x5000, ldq=72, S=0x6000), MISALIGNED), (dict(Q=0x5008, ldq=64, S=0x6000), MISALIGNED),
    (dict(Q=0x5000, ldq=64, S=0x6008), MISALIGNED), (dict(ws=0x8010, wsb=512), WORKSPACE), (dict(wsb=512), WORKSPACE),
    (dict(m=0), OK), (dict(n=0), OK), (dict(m=0, C=None), OK),
])
def test_linear_refusals(change, status):
    assert linear(**change) == status


def dact(m=64, n=64, k=64, ta=0, tb=0, alpha=1.0, A=0x1000, lda=64, B=0x2000, ldb=64, Q=0x5000, ldq=64, S=0x6000, act=2,
         C=0x4000, ldc=64, ct=1, dbias=None, acc=0, ws=None, wsb=0):
    return bm.bm_gemm_bf16_dact(m, n, k, ta, tb, alpha, A, lda, B, ldb, Q, ldq, S, act, C, ldc, ct, dbias, acc, ws, wsb,
                                None)


@pytest.mark.parametrize("change,status", [
    (dict(m=-1), INVALID), (dict(act=9), INVALID), (dict(Q=None), INVALID), (dict(S=None), INVALID),
    (dict(Q=None, S=None), INVALID), (dict(ldq=32), INVALID), (dict(ldb=32), INVALID), (dict(C=None), INVALID),
    (dict(dbias=0x9008, ws=0x8000, wsb=1 << 20), MISALIGNED), (dict(ldq=72), MISALIGNED),
    (dict(dbias=0x9000), WORKSPACE), (dict(dbias=0x9000, ws=0x8000, wsb=256), WORKSPACE),
    (dict(dbias=0x9000, ws=0x8010, wsb=1 << 20), WORKSPACE),
    (dict(n=0), OK), (dict(m=0), OK), (dict(m=0, dbias=0x9000, acc=1), OK),
])
def test_dact_refusals(change, status):
    assert dact(**change) == status


def act(rows=8, n=64, Q=0x1000, ldq=64, S=0x2000, a=1, H=0x3000, ldh=64, ht=1):
    return bm.bm_act_mxfp8(rows, n, Q, ldq, S, a, H, ldh, ht, None)


@pytest.mark.parametrize("change,status", [
    (dict(rows=-1), INVALID), (dict(n=2 ** 31), INVALID), (dict(a=6), INVALID), (dict(ht=3), INVALID),
    (dict(Q=None), INVALID), (dict(S=None), INVALID), (dict(H=None), INVALID), (dict(ldq=63), INVALID),
    (dict(ldh=63), INVALID), (dict(ldq=72), MISALIGNED), (dict(ldh=66), MISALIGNED), (dict(H=0x3002), MISALIGNED),
    (dict(rows=0), OK), (dict(n=0), OK),
])
def test_act_refusals(change, status):
    assert act(**change) == status


def norm(rows=8, n=64, X=0x1000, ldx=64, xt=1, g=0x2000, b=0x3000, pt=0, eps=1e-5, Y=0x4000, ldy=64, yt=1, mean=None,
         rstd=None):
    return bm.bm_layernorm(rows, n, X, ldx, xt, g, b, pt, eps, Y, ldy, yt, mean, rstd, None)


@pytest.mark.parametrize("change,status", [
    (dict(rows=-1), INVALID), (dict(n=-1), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID),
    (dict(xt=2), INVALID), (dict(yt=2), INVALID), (dict(pt=2), INVALID), (dict(ldx=60), INVALID),
    (dict(ldy=60), INVALID), (dict(X=None), INVALID), (dict(Y=None), INVALID), (dict(X=0x1008), MISALIGNED),
    (dict(ldx=68), MISALIGNED), (dict(ldy=66, yt=0), MISALIGNED), (dict(g=0x2004), MISALIGNED),
    (dict(b=0x2004), MISALIGNED), (dict(mean=0x5002), MISALIGNED), (dict(rstd=0x5001), MISALIGNED),
    (dict(rows=0), OK), (dict(n=0), OK),
])
def test_layernorm_refusals(change, status):
    assert norm(**change) == status


def norm_bwd(rows=8, n=64, dY=0x1000, lddy=64, yt=1, X=0x2000, ldx=64, xt=1, g=0x3000, pt=0, mean=0x4000, rstd=0x5000,
             dres=None, lddres=0, dX=0x6000, lddx=64, dg=None, db=None, acc=0, ws=None, wsb=0):
    return bm.bm_layernorm_backward(rows, n, dY, lddy, yt, X, ldx, xt, g, pt, mean, rstd, dres, lddres, dX, lddx, dg, db,
                                    acc, ws, wsb, None)


@pytest.mark.parametrize("change,status", [
    (dict(rows=-1), INVALID), (dict(n=2 ** 31), INVALID), (dict(xt=2), INVALID), (dict(yt=-1), INVALID),
    (dict(lddy=60), INVALID), (dict(lddx=60), INVALID), (dict(dres=0x7000, lddres=60), INVALID),
    (dict(dg=0x8000), INVALID), (dict(db=0x8000), INVALID), (dict(dY=None), INVALID), (dict(X=None), INVALID),
    (dict(dX=None), INVALID), (dict(mean=None), INVALID), (dict(rstd=None), INVALID), (dict(dY=0x1008), MISALIGNED),
    (dict(lddx=68), MISALIGNED), (dict(dres=0x7008, lddres=64), MISALIGNED), (dict(g=0x3002), MISALIGNED),
    (dict(mean=0x4002), MISALIGNED), (dict(dg=0x8004, db=0x9000, ws=0xA000, wsb=1 << 24), MISALIGNED),
    (dict(dg=0x8000, db=0x9000), WORKSPACE), (dict(dg=0x8000, db=0x9000, ws=0xA000, wsb=256), WORKSPACE),
    (dict(dg=0x8000, db=0x9000, ws=0xA010, wsb=1 << 24), WORKSPACE),
    (dict(n=0), OK), (dict(rows=0), OK), (dict(rows=0, dg=0x8000, db=0x9000, acc=1), OK),
])
def test_layernorm_backward_refusals(change, status):
    assert norm_bwd(**change) == status


def test_workspace_sizes():
    assert bm.bm_gemm_bf16_bias_act_workspace_size(0, 64, 64) == 0
    assert bm.bm_gemm_bf16_bias_act_workspace_size(4096, 4096, 4096) == 0       # whole tiles, or halves
    assert bm.bm_gemm_bf16_bias_act_workspace_size(512, 512, 4096) > 0          # every tile split along K
    least = 4 * (4096 // 32) * 16384
    assert bm.bm_gemm_bf16_dact_workspace_size(4096, 16384, 4096, 1) == least
    assert bm.bm_gemm_bf16_dact_workspace_size(4096, 16384, 4096, 0) == 0
    assert bm.bm_gemm_bf16_dact_workspace_size(0, 64, 64, 1) == 0
    assert bm.bm_layernorm_backward_workspace_size(0, 64) == 0
    for rows, n in ((1, 1), (100, 5120), (16384, 5120), (16384, 33001)):
        size = bm.bm_layernorm_backward_workspace_size(rows, n)
        assert size % (2 * 8 * 4) == 0 and 8 * n <= size <= 8 * (n + 7) * min(rows, 8 * 152)


def test_helpers_refuse_before_the_library():
    torch = pytest.importorskip("torch")
    x = torch.zeros(8, 64)
    with pytest.raises(ValueError, match="CUDA"):
        bm.layernorm(x, None, None, x)
    b = torch.zeros(8, 64, dtype=torch.bfloat16)
    with pytest.raises(TypeError, match="bfloat16"):
        bm.gemm_bias_act(x, b, x, transB=True)
    with pytest.raises(ValueError, match="inconsistent"):
        bm.gemm_bias_act(b, b, torch.zeros(8, 9), transB=True)
    with pytest.raises(ValueError, match="CUDA"):
        bm.gemm_bias_act(b, b, torch.zeros(8, 8), transB=True)
    with pytest.raises(ValueError, match="act must be"):
        bm._act("tanh")
    q, s = torch.zeros(8, 64, dtype=torch.uint8), torch.zeros(512, dtype=torch.uint8)
    assert bm._checkpoint((q, s), 8, 64)[1] == 64
    for bad in ((q[:4], s), (q, s[:100]), (q.t(), s)):
        with pytest.raises(ValueError):
            bm._checkpoint(bad, 8, 64)
    with pytest.raises(TypeError):
        bm._checkpoint((q.float(), s), 8, 64)
