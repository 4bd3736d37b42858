"""The 64-bit forms that the GPU tests compare with: slopes and layer norm's gradients against
central differences, the MXFP8 rule against the CPU oracle's. No GPU."""

import numpy as np
import pytest

import bm_inputs as gen
import mlp_ref as ref
import oracle


@pytest.mark.parametrize("name", ref.ACTS)
def test_slopes_are_differences_of_the_activations(name):
    z = np.linspace(-6.0, 6.0, 241) + 0.013      # (no point on relu's corner)
    h = 1e-5
    diff = (ref.act(z + h, name) - ref.act(z - h, name)) / (2 * h)
    # third derivatives below 3: truncation h^2 / 2, rounding 1e-15 / h
    assert np.max(np.abs(diff - ref.slope(z, name))) < 2e-9


def test_layernorm_gradients_are_differences():
    rng = np.random.default_rng(3)
    rows, n, eps, h = 3, 7, 1e-5, 1e-6
    x, gamma, beta = rng.normal(size=(rows, n)) + 2.0, rng.normal(size=n), rng.normal(size=n)
    dy = rng.normal(size=(rows, n))

    def loss(x, gamma, beta):
        return (ref.layernorm(x, gamma, beta, eps)[0] * dy).sum()

    _, mean, rstd = ref.layernorm(x, gamma, beta, eps)
    dx, dg, db = ref.layernorm_backward(dy, x, gamma, mean, rstd)
    for i in range(rows):
        for j in range(n):
            e = np.zeros((rows, n))
            e[i, j] = h
            assert abs((loss(x + e, gamma, beta) - loss(x - e, gamma, beta)) / (2 * h) - dx[i, j]) < 1e-7
    for j in range(n):
        e = np.zeros(n)
        e[j] = h
        assert abs((loss(x, gamma + e, beta) - loss(x, gamma - e, beta)) / (2 * h) - dg[j]) < 1e-7
        assert abs((loss(x, gamma, beta + e) - loss(x, gamma, beta - e)) / (2 * h) - db[j]) < 1e-7


@pytest.mark.parametrize("rows,cols", [(3, 32), (5, 70), (130, 33)])
def test_mx_rule_equals_the_oracle(rows, cols):
    bits = gen.matrix_bf16(rows, cols, "normal", seed=rows)
    bits[0, :5] = gen.f32_to_bf16_bits(np.array([0.0, -0.0, 448.0, 1e-38, -3e38], np.float32))
    bits[1, 1] = gen.f32_to_bf16_bits(np.array([np.inf], np.float32))[0]
    q, s = ref.quantize(gen.bf16_bits_to_f32(bits).astype(np.float64))
    oq, os_ = oracle.default().quantize_mxfp8(bits)
    assert np.array_equal(s, os_)
    assert np.array_equal(q, oq)


def test_decode_inverts_the_layout():
    rng = np.random.default_rng(1)
    z = rng.normal(size=(133, 161)) * 2.0 ** rng.integers(-3, 4, size=(133, 161))
    q, s = ref.quantize(z)
    back = ref.decode(q, ref.tile_scales(s, 133, 161), 133, 161)
    # a group's values are rounded at 2^-4 of themselves, or saturate at 448/512 of its power of two
    assert np.max(np.abs(back - z) / np.maximum(np.abs(z), np.abs(z).max(axis=1, keepdims=True) * 2.0 ** -9)) <= 0.125
