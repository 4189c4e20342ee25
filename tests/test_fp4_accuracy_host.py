"""The accuracy tests' tolerance tells: it takes a model of the kernels'
roundings, and refuses the same model without the folds or without a weight's
second part."""
import numpy as np
import pytest

from tests import fp4_ref, fp4_tight


def _case(n, spread):
    rng = np.random.default_rng(n)
    q = fp4_ref.from_bf16_bits(fp4_ref.to_bf16_bits(rng.standard_normal((4, 128)) * spread)).astype(np.float64)
    k = fp4_ref.rows(rng, n, 1).astype(np.float64)
    v = np.abs(fp4_ref.rows(rng, n, 1)).astype(np.float64)
    return q, k, v, n - 1, 0, 0, fp4_ref.SM


@pytest.mark.parametrize("n", [2, 9, 100, 20000])
def test_tolerance_takes_the_kernels_roundings(n):
    case = _case(n, 0.05)
    assert (np.abs(fp4_tight.chained(*case) - fp4_ref.attend(*case)) <= fp4_tight.tolerance(*case)).all()


def test_tolerance_refuses_one_chain():
    case = _case(20000, 0.05)
    off = np.abs(fp4_tight.chained(*case, fold=0) - fp4_ref.attend(*case))
    assert (off > fp4_tight.tolerance(*case)).mean() > 0.5


@pytest.mark.parametrize("n", [2, 9])
def test_tolerance_refuses_one_part(n):
    case = _case(n, 0.05)
    off = np.abs(fp4_tight.chained(*case, parts=1) - fp4_ref.attend(*case))
    assert (off > fp4_tight.tolerance(*case)).mean() > 0.25
