"""The hybrid layer example (product, linear attention, product, router, choice of experts, experts' network): every
call of the library on the way against its formula in 64 bits on the inputs that it got, and the captured decoding
step against the eager one."""
import importlib.util
import os

import numpy as np
import pytest

import experts_reference
import linear_reference
import oracle

torch = pytest.importorskip("torch")
import quantized_weight_gguf_gb300 as q  # noqa: E402

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SIZES = dict(width=256, n_heads=4, n_qk=2, head_dim=32, n_experts=12, top_k=3, n_ff=512, n_seqs=2)


@pytest.fixture(scope="module")
def example():
    from quantized_weight_gguf_gb300 import build_lib
    build_lib.build()
    q.load()
    oracle.build()
    spec = importlib.util.spec_from_file_location("hybrid_layer", os.path.join(ROOT, "examples", "hybrid_layer.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    yield mod
    q.qmm_device_status()


def _np(t):
    return t.detach().cpu().numpy().copy()


@pytest.mark.parametrize("n_new", [1, 5, 40, 150])
def test_every_call_follows_its_formula(example, monkeypatch, n_new):
    layer = example.HybridLayer(seed=n_new, **SIZES)
    seen = []

    def spy(name):
        call = getattr(q, name)

        def record(*args, **kw):
            before = [_np(a) if torch.is_tensor(a) else a for a in args]
            y0 = _np(kw["y"]) if "y" in kw else None
            out = call(*args, **kw)
            torch.cuda.synchronize()
            after = [_np(a) if torch.is_tensor(a) else a for a in args]
            seen.append((name, before, y0, out if isinstance(out, tuple) else (out,), after))
            seen[-1] = seen[-1][:3] + (tuple(_np(o) for o in seen[-1][3]), after)
            return out
        monkeypatch.setattr(q, name, record)

    for name in ("matmul", "linear_attend", "route_experts", "experts_ffn"):
        spy(name)
    torch.manual_seed(n_new)
    x = torch.randn(2, 30, 256, device="cuda:0")
    layer(x)                                     # a prompt, so that the calls that are looked at find a state
    del seen[:]
    layer(torch.randn(2, n_new, 256, device="cuda:0"))
    assert q.qmm_device_status() == 0
    assert [s[0] for s in seen] == ["matmul", "linear_attend", "matmul", "matmul", "route_experts", "experts_ffn"]
    for name, args, y0, out, after in seen:
        if name == "matmul":
            fmt, w, xs, k, n = args
            want, size = oracle.matmul(fmt, w, xs.reshape(-1, k), k, n)
            if y0 is not None:
                want, size = want + y0.reshape(want.shape), size + np.abs(y0.reshape(want.shape))
            ok, _, _, msg = oracle.check(out[0].reshape(want.shape), want, size)
            assert ok, msg
        elif name == "linear_attend":
            want, state, tol, s_tol = linear_reference.attend(*args[:5], None, args[0].shape[-1] ** -0.5)
            assert (np.abs(out[0] - want) <= tol).all()
            assert (np.abs(after[4] - state) <= s_tol).all()
        elif name == "route_experts":
            ids, weights = experts_reference.route(args[0], args[1], "softmax", True, 1.0)
            assert np.array_equal(out[0], ids)
            # differences of logits are rounded once (2^-24 of the largest), exp and the division a few times
            assert (np.abs(out[1] - weights) <= (2.0 ** -22 + 2.0 ** -23 * np.abs(args[0]).max()) * weights).all()
        else:
            act, fmt, wg, wu, fmt_down, wd, xs, ids, weights, k, n_ff, n_exp = args
            want, tol = experts_reference.ffn(act, fmt, wg, wu, fmt_down, wd, xs, ids, weights, k, n_ff, n_exp,
                                              y0)
            assert (np.abs(out[0].reshape(want.shape) - want) <= tol).all()


def test_replayed_steps_are_the_eager_ones(example):
    eager, captured = (example.HybridLayer(seed=9, **SIZES) for _ in range(2))
    torch.manual_seed(2)
    prompt = torch.randn(2, 70, 256, device="cuda:0")
    x, y = (layer(prompt.clone())[:, -1:].contiguous() for layer in (eager, captured))
    assert torch.equal(x, y) and torch.equal(eager.state, captured.state)
    held = captured.state.clone(), y.clone()
    captured(y)                                  # sets up what the library owns; taken back
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        captured(y)
    captured.state.copy_(held[0])
    y.copy_(held[1])
    for _ in range(5):
        eager(x)
        graph.replay()
        assert torch.equal(x, y) and torch.equal(eager.state, captured.state)
    assert q.qmm_device_status() == 0


def test_refuses_tensors_that_are_not_on_the_current_device(example, monkeypatch):
    """The kernels go to the current device: with another one current, the calls launch nothing."""
    layer = example.HybridLayer(seed=1, **SIZES)
    x = torch.randn(2, 1, 256, device="cuda:0")
    logits = torch.randn(2, 12, device="cuda:0")
    ids, weights = q.route_experts(logits, 3)
    heads = [torch.randn(2, 1, h, 32, device="cuda:0") for h in (2, 2, 4)]
    decay = torch.zeros(4, device="cuda:0")
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 1)
    with pytest.raises(ValueError, match="current device"):
        q.route_experts(logits, 3, ids=ids, weights=weights)
    with pytest.raises(ValueError, match="current device"):
        q.experts_ffn("swiglu", "q4_k", layer.w_gate, layer.w_up, "q6_k", layer.w_down, x.view(2, 256), ids, weights,
                      256, 512, 12, y=torch.empty_like(x.view(2, 256)))
    with pytest.raises(ValueError, match="current device"):
        q.linear_attend(*heads, decay, layer.state, out=torch.empty_like(heads[2]))
