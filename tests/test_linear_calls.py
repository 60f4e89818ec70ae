"""Host-side checks of the linear attention call, without a GPU: every refusal with its status before anything is
launched."""
import ctypes

import pytest

import quantized_weight_gguf_gb300 as q
from quantized_weight_gguf_gb300 import build_lib


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build_lib.build()
    q.load()


def _args(**kw):
    base = dict(q=16, k=32, v=48, q_stride=256, k_stride=256, v_stride=512, decay=64, decay_stride=4, state=80,
                state_out=96, out=112, out_stride=512, lens=128, n_seqs=2, n_new=5, n_heads=4, n_qk_heads=2, dk=128,
                dv=128, scale=0.1, workspace=None, workspace_bytes=0, stream=None, flags=0)
    base.update(kw)
    return q.qmm_linear_args(**base)


SHAPE, NULL, ALIGN = 2, 5, 6


@pytest.mark.parametrize("kw,status", [
    (dict(n_new=0), SHAPE), (dict(dk=16), SHAPE), (dict(dk=48), SHAPE), (dict(dk=160), SHAPE), (dict(dv=16), SHAPE),
    (dict(dv=100), SHAPE), (dict(dv=288), SHAPE), (dict(n_heads=0), SHAPE), (dict(n_qk_heads=0), SHAPE),
    (dict(n_heads=5), SHAPE), (dict(n_heads=65540), SHAPE), (dict(n_seqs=-1), SHAPE), (dict(n_seqs=1 << 23), SHAPE),
    (dict(n_new=1 << 31), SHAPE), (dict(decay_stride=3), SHAPE), (dict(decay_stride=-4), SHAPE),
    (dict(decay_stride=1 << 33), SHAPE), (dict(scale=float("nan")), SHAPE), (dict(flags=2), SHAPE),
    (dict(q_stride=255), SHAPE), (dict(k_stride=0), SHAPE), (dict(v_stride=511), SHAPE), (dict(out_stride=1 << 33), SHAPE),
    (dict(q=None), NULL), (dict(k=None), NULL), (dict(v=None), NULL), (dict(out=None), NULL), (dict(decay=None), NULL),
    (dict(state=None), NULL), (dict(state_out=None), NULL), (dict(q=18), ALIGN), (dict(v=49), ALIGN),
    (dict(decay=66), ALIGN), (dict(lens=129), ALIGN), (dict(state=84), ALIGN), (dict(state_out=100), ALIGN),
])
def test_refusals(kw, status):
    a = _args(**kw)
    assert q.load().qmm_linear_attend(ctypes.byref(a)) == status
    assert q.qmm_last_error()
    if status == SHAPE and "stride" not in next(iter(kw)):
        assert q.qmm_linear_attend_workspace_bytes(a) == 0


def test_no_sequences_need_nothing():
    a = _args(n_seqs=0, q=None, k=None, v=None, out=None, state=None, state_out=None, decay=None, lens=None)
    assert q.load().qmm_linear_attend(ctypes.byref(a)) == 0
    assert q.load().qmm_linear_attend(None) == NULL
