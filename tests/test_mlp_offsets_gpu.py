"""Element and byte offsets past 2^31 (and past 2^32 bytes): the last rows of large tensors are, bit for bit, what the
same call gives for those rows alone. Enough of them are compared that both calls take the same kernel."""

from __future__ import annotations

import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def bm():
    import blas3_tensor_core_gb300 as module
    return module


def tail(t, rows):
    return t[t.shape[0] - rows:]


def test_layernorm_offsets(bm):
    import torch
    rows, n, last = 420000, 5128, 1300       # 2.15e9 elements, 4.3 GB a tensor
    torch.manual_seed(1)
    X = torch.randn(1000, n, device="cuda").bfloat16().repeat(rows // 1000, 1)
    tail(X, last).copy_(torch.randn(last, n, device="cuda"))
    gamma, beta = torch.randn(n, device="cuda"), torch.randn(n, device="cuda")
    Y, mean, rstd = torch.empty_like(X), torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    bm.layernorm(X, gamma, beta, Y, mean=mean, rstd=rstd)
    x = tail(X, last).clone()
    y, m1, r1 = torch.empty_like(x), torch.empty(last, device="cuda"), torch.empty(last, device="cuda")
    bm.layernorm(x, gamma, beta, y, mean=m1, rstd=r1)
    assert torch.equal(tail(Y, last), y) and torch.equal(mean[-last:], m1) and torch.equal(rstd[-last:], r1)
    assert torch.isfinite(Y[0]).all() and not torch.equal(Y[0], Y[-1])

    dX = torch.empty_like(X)
    bm.layernorm_backward(Y, X, gamma, mean, rstd, dX, dres=Y)
    dx = torch.empty_like(x)
    bm.layernorm_backward(y, x, gamma, m1, r1, dx, dres=y)
    assert torch.equal(tail(dX, last), dx)


def test_product_and_checkpoint_offsets(bm):
    import torch
    m, n, k, last = 270080, 8192, 64, 2560   # 2.2e9 elements: codes past 2^31 bytes, C past 2^32
    torch.manual_seed(2)
    A = torch.randint(-3, 4, (m, k), device="cuda").bfloat16()       # (integers: every order of summing is exact)
    W = torch.randint(-3, 4, (n, k), device="cuda").bfloat16()
    C, ck = torch.empty(m, n, dtype=torch.bfloat16, device="cuda"), bm.mxfp8_empty(m, n)
    bm.gemm_bias_act(A, W, C, act="relu", transB=True, checkpoint=ck)
    a = tail(A, last).contiguous()
    c, ck1 = torch.empty(last, n, dtype=torch.bfloat16, device="cuda"), bm.mxfp8_empty(last, n)
    bm.gemm_bias_act(a, W, c, act="relu", transB=True, checkpoint=ck1)
    assert torch.equal(tail(C, last), c) and torch.equal(tail(ck[0], last), ck1[0])
    assert m % 128 == 0 and torch.equal(ck[1].view(-1)[-ck1[1].numel():], ck1[1].view(-1))

    H, h = C, c                              # the activation again, and the product that reads the checkpoint
    bm.act_mxfp8(ck, H, act="gelu")
    bm.act_mxfp8(ck1, h, act="gelu")
    assert torch.equal(tail(H, last), h)
    B = W.t().contiguous()
    bm.gemm_dact(A, B, C, ck, act="silu")
    bm.gemm_dact(a, B, c, ck1, act="silu")
    assert torch.equal(tail(C, last), c)
