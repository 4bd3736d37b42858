"""Sizes of the orthogonalised update at the ends of its arguments' ranges (CPU only: the checks come before any CUDA
call, the pointers are made up)."""

import pytest

import blas3_tensor_core_gb300 as bm
from test_gated_ops_host import INVALID, WORKSPACE, _built, orth  # noqa: F401


@pytest.mark.parametrize("m,n", [(2 ** 31 - 1, 2 ** 31 - 1), (2 ** 30, 2 ** 31 - 1), (2 ** 31 - 1, 2 ** 27 + 1),
                                 (2 ** 40, 2 ** 40), (2 ** 31, 64), (64, 2 ** 31)])
def test_sizes_that_cannot_be_counted_are_refused(m, n):
    """8 m n bytes and more of workspace leave 64 bits: no size is given, and no workspace is enough."""
    assert bm.orthogonalize_workspace_size(m, n) == 0
    assert orth(m=m, n=n, ldx=n, ldc=n, wsb=2 ** 63) == INVALID


@pytest.mark.parametrize("m,n", [(2 ** 31 - 1, 2 ** 27 - 16), (64, 2 ** 31 - 1), (2 ** 31 - 1, 16), (2 ** 29, 2 ** 29)])
def test_the_largest_sizes_have_a_workspace(m, n):
    s, ld = min(m, n), n + -n % 8
    assert 8 * m * n + 4 * s * s <= bm.orthogonalize_workspace_size(m, n) < 2 ** 63
    assert orth(m=m, n=n, ldx=ld, ldc=ld, wsb=8 * m * n) == WORKSPACE


def test_coefficients_of_any_sequence_or_array():
    numpy, torch = pytest.importorskip("numpy"), pytest.importorskip("torch")
    one, several = (2.0, -1.5, 0.5), [(2.0, -1.5, 0.5), (4.0, -8.0, 5.0), (3.0, -3.25, 1.25)]
    for steps in (1, 3, 5):
        for coeffs in (one, list(one), numpy.array(one, numpy.float32), torch.tensor(one), [torch.tensor(c) for c in one]):
            assert bm._step_coeffs(coeffs, steps) == [*one] * steps
    want = [v for c in several for v in c]
    for coeffs in (several, numpy.array(several), torch.tensor(several), [torch.tensor(c) for c in several]):
        assert bm._step_coeffs(coeffs, 3) == want
    for bad in ([], (1.0, 2.0), torch.tensor(one)[:2], torch.tensor(several), [one], torch.tensor(1.0).reshape(1)):
        with pytest.raises(ValueError, match="coeffs"):
            bm._step_coeffs(bad, 2)
