"""Norms of the experts' errors where the activated products (by way of the positions' weights) are very small or
large, for every kernel: as exact as where they are about 1 (norm_bounds)."""
import numpy as np
import pytest

from test_gpu_norms import FFN, FfnInputs, lib  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("power", [-112, -104, 92])
@pytest.mark.parametrize("case", FFN, ids=str)
def test_products_near_the_ends_of_fp32(lib, case, power):  # noqa: F811
    c = FfnInputs(*case)
    want, bound = c.want()
    c.weights *= np.float32(2.0 ** power)
    y = c.call().astype(np.float64) * 2.0 ** -power
    off = np.linalg.norm(y - want, axis=1)
    assert (off <= bound).all(), (off / bound).max()
