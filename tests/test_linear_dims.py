"""Which head sizes linear attention takes, without a GPU: every other one is refused before anything is launched."""
import ctypes

import pytest

import quantized_weight_gguf_gb300 as q
from quantized_weight_gguf_gb300 import build_lib


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build_lib.build()
    q.load()


def test_head_sizes():
    def refused(dk, dv):
        a = q.qmm_linear_args(n_seqs=0, n_new=1, n_heads=2, n_qk_heads=2, dk=dk, dv=dv, scale=1.0)
        return q.load().qmm_linear_attend(ctypes.byref(a)) == 2
    sizes = [*range(-33, 300), 512, 1 << 31, (1 << 32) + 64, -(1 << 32) + 64, 1 << 62]
    assert [n for n in sizes if not refused(n, 64)] == [32, 64, 96, 128]
    assert [n for n in sizes if not refused(64, n)] == list(range(32, 257, 32))
