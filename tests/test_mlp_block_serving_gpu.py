"""Serving with the example block between a training forward pass and its backward pass."""

import pytest

from test_mlp_block_gpu import example  # noqa: F401 (fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("served", [1, 48, 200])
def test_serving_leaves_the_training_pass_alone(example, served):
    import torch
    torch.manual_seed(served)
    block = example.MlpBlock(256, 160, 416)
    x, dy = (torch.randn(200, 160, device="cuda").bfloat16() for _ in range(2))
    token = torch.randn(served, 160, device="cuda").bfloat16()
    grads = (block.dw1, block.db1, block.dw2, block.db2, block.dgamma, block.dbeta)
    block.forward(x)
    want = [block.backward(dy)] + [g.clone() for g in grads]
    alone = block.forward(token, train=False)
    for g in grads:
        g.fill_(float("nan"))
    block.forward(x)
    assert torch.equal(block.forward(token, train=False), alone)
    got = [block.backward(dy), *grads]
    assert all(torch.equal(a, b) for a, b in zip(want, got))
