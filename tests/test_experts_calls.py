"""Host-side checks of the mixture-of-experts calls, without a GPU: every refusal with its status before anything is
launched, scratch sizes, and what the Python calls refuse."""
import ctypes

import pytest

import quantized_weight_gguf_gb300 as q
from quantized_weight_gguf_gb300 import build_lib

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build_lib.build()
    q.load()


def _route(**kw):
    base = dict(logits=16, logits_stride=64, n_pos=3, n_experts=64, top_k=8, score=0, normalize=1, scale=1.0, ids=64,
                weights=128, stream=None, flags=0)
    base.update(kw)
    return q.qmm_route_args(**base)


def _ffn(**kw):
    base = dict(act=1, fmt=q.FORMATS["q4_k"], fmt_down=q.FORMATS["q6_k"], w_gate=16, w_up=32, w_down=48, w_len=0,
                w_down_len=0, x=64, ids=128, weights=192, y=256, k=512, n_ff=256, n_experts=8, n_pos=4, top_k=2,
                accumulate=0, workspace=None, workspace_bytes=0, stream=None, flags=0)
    base.update(kw)
    return q.qmm_experts_ffn_args(**base)


def _status(call, args):
    return getattr(q.load(), call)(ctypes.byref(args))


FORMAT, SHAPE, SIZE, NULL, ALIGN = 1, 2, 3, 5, 6


@pytest.mark.parametrize("kw,status", [
    (dict(n_experts=0), SHAPE), (dict(n_experts=4097), SHAPE), (dict(top_k=0), SHAPE), (dict(top_k=65), SHAPE),
    (dict(n_experts=4, top_k=5), SHAPE), (dict(n_pos=-1), SHAPE), (dict(n_pos=(1 << 30) + 1), SHAPE),
    (dict(logits_stride=63), SHAPE), (dict(logits_stride=1 << 33), SHAPE), (dict(score=2), FORMAT),
    (dict(scale=float("nan")), SHAPE), (dict(scale=float("inf")), SHAPE), (dict(flags=1), SHAPE),
    (dict(logits=None), NULL), (dict(ids=None), NULL), (dict(weights=None), NULL), (dict(logits=18), ALIGN),
    (dict(ids=65), ALIGN), (dict(weights=130), ALIGN),
])
def test_route_refusals(kw, status):
    assert _status("qmm_route_experts", _route(**kw)) == status
    assert q.qmm_last_error()


def test_route_of_no_positions_needs_nothing():
    assert _status("qmm_route_experts", _route(n_pos=0, logits=None, ids=None, weights=None)) == 0


@pytest.mark.parametrize("kw,status", [
    (dict(act=0), FORMAT), (dict(act=3), FORMAT), (dict(fmt=7), FORMAT), (dict(fmt_down=8), FORMAT), (dict(fmt=-1), FORMAT),
    (dict(k=0), SHAPE), (dict(k=100), SHAPE), (dict(k=288), SHAPE), (dict(n_ff=0), SHAPE), (dict(n_ff=288), SHAPE),
    (dict(k=1 << 21), SHAPE), (dict(fmt=1, k=33), SHAPE), (dict(n_experts=0), SHAPE), (dict(n_experts=4097), SHAPE),
    (dict(top_k=0), SHAPE), (dict(top_k=65), SHAPE), (dict(n_pos=-1), SHAPE), (dict(n_pos=32768), SHAPE),
    (dict(n_pos=1 << 62), SHAPE), (dict(flags=4), SHAPE), (dict(w_len=1000), SIZE),
    (dict(w_len=8 * 256 * 288 - 1), SIZE), (dict(w_down_len=8 * 512 * 210 + 1), SIZE),
    (dict(w_gate=None), NULL), (dict(w_up=None), NULL), (dict(w_down=None), NULL), (dict(x=None), NULL),
    (dict(ids=None), NULL), (dict(weights=None), NULL), (dict(y=None), NULL),
    (dict(w_gate=8), ALIGN), (dict(w_up=24), ALIGN), (dict(w_down=50), ALIGN), (dict(x=66), ALIGN), (dict(ids=129), ALIGN),
    (dict(weights=194), ALIGN), (dict(y=257), ALIGN),
])
def test_ffn_refusals(kw, status):
    a = _ffn(**kw)
    assert _status("qmm_experts_ffn", a) == status
    assert q.qmm_last_error()
    if status in (FORMAT, SHAPE, SIZE):
        assert q.qmm_experts_ffn_workspace_bytes(a) == 0


def test_ffn_of_no_positions_needs_nothing():
    a = _ffn(n_pos=0, w_gate=None, w_up=None, w_down=None, x=None, ids=None, weights=None, y=None)
    assert _status("qmm_experts_ffn", a) == 0
    assert q.qmm_experts_ffn_workspace_bytes(a) == 0


def test_null_arguments():
    assert q.load().qmm_route_experts(None) == NULL
    assert q.load().qmm_experts_ffn(None) == NULL


def test_python_calls_take_device_tensors_only():
    x = torch.zeros((2, 64))
    with pytest.raises(ValueError):
        q.route_experts(x, 2)
    w = torch.zeros(4 * 32 * 68, dtype=torch.uint8)
    with pytest.raises(ValueError):
        q.experts_ffn("swiglu", "q8_0", w, w, "q8_0", w, x, torch.zeros((2, 2), dtype=torch.int32), torch.zeros((2, 2)), 64,
                      32, 4)
