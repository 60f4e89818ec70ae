"""The choice of experts on the GPU against the rule in 64 bits (experts_reference): ids equal, weights within a few
roundings."""
import numpy as np
import pytest

import experts_reference as ref

torch = pytest.importorskip("torch")
import quantized_weight_gguf_gb300 as q  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from quantized_weight_gguf_gb300 import build_lib
    build_lib.build()
    q.load()
    yield
    q.qmm_device_status()


def _check(logits, top_k, score, normalize, scale, **kw):
    ids, w = q.route_experts(torch.from_numpy(logits).to(DEV), top_k, score=score, normalize=normalize, scale=scale, **kw)
    torch.cuda.synchronize()
    ids, w = ids.cpu().numpy(), w.cpu().numpy()
    want, ww = ref.route(logits, top_k, score, normalize, scale)
    np.testing.assert_array_equal(ids, want)
    # A weight is a quotient of exponentials of a difference of logits (fp32: U of the logits' sizes before the
    # exponential, which turns it into a relative error; expf 2 steps, log1pf 1) over a sum of up to 4096 of them
    # (5 additions across lanes after at most 128 in a lane).
    big = np.abs(np.where(np.isfinite(logits) & (np.abs(logits) < 1e30), logits, 0)).max(-1, keepdims=True, initial=0)
    tol = np.abs(ww) * ref.U * (4 * big + 160) + 1e-37
    ok = (np.abs(w - ww) <= tol) | (np.isnan(w) & np.isnan(ww))
    assert ok.all(), (w[~ok][:4], ww[~ok][:4])
    return ids, w


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("normalize", [True, False])
@pytest.mark.parametrize("n_pos,n_experts,top_k", [(1, 8, 2), (1, 1, 1), (3, 33, 33), (5, 64, 8), (130, 128, 8),
                                                   (9, 200, 5), (2, 512, 64), (3, 513, 7), (2, 4096, 64)])
def test_matches_the_rule(n_pos, n_experts, top_k, score, normalize):
    rng = np.random.default_rng(n_experts * 8 + top_k)
    logits = (rng.standard_normal((n_pos, n_experts)) * 3).astype(np.float32)
    _check(logits, top_k, score, normalize, 1.0 if normalize else 2.5)


@pytest.mark.parametrize("n_experts", [8, 100, 600])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_ties_go_to_the_lowest_index(n_experts, score):
    rng = np.random.default_rng(7)
    logits = rng.integers(-1, 2, (40, n_experts)).astype(np.float32)
    logits[0] = 0.0
    logits[1, ::2] = -0.0   # equal to +0
    logits[1, 1::2] = 0.0
    _check(logits, min(8, n_experts), score, True, 1.0)


@pytest.mark.parametrize("n_experts", [16, 300, 1000])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("normalize", [True, False])
def test_switched_off_and_extreme(n_experts, score, normalize):
    rng = np.random.default_rng(11)
    low = np.finfo(np.float32).min
    logits = rng.standard_normal((9, n_experts)).astype(np.float32)
    logits[0] = -np.inf                       # nothing left
    logits[1, 3:] = -np.inf                   # three left
    logits[2] = low                           # the lowest value is a value
    logits[3, 1:] = low
    logits[4] = np.where(rng.random(n_experts) < 0.5, -np.inf, low)
    logits[5] = -200.0 + logits[5]            # every score tiny
    logits[6] = 3e38                          # equal and large
    logits[7, 5] = np.nan                     # not taken, and shows
    logits[8] = np.nan
    ids, w = _check(logits, 6, score, normalize, 1.5)
    assert (ids[0] == -1).all() and (w[0] == 0).all()
    assert (ids[1, 3:] == -1).all() and 5 not in ids[7]


def test_plus_infinity():
    logits = np.zeros((1, 16), np.float32)
    logits[0, 4] = np.inf
    for score in ("softmax", "sigmoid"):
        ids, w = q.route_experts(torch.from_numpy(logits).to(DEV), 2, score=score)
        assert ids[0].tolist() == [4, 0]
        w = w.cpu().numpy()
        assert np.isnan(w).all() if score == "softmax" else np.allclose(w, [[2 / 3, 1 / 3]])


def test_strided_rows_given_outputs_and_empty():
    rng = np.random.default_rng(3)
    wide = torch.from_numpy(rng.standard_normal((20, 90)).astype(np.float32)).to(DEV)
    part = wide[:, 11:75]
    ids = torch.full((20, 4), 77, dtype=torch.int32, device=DEV)
    w = torch.empty((20, 4), device=DEV)
    got = q.route_experts(part, 4, ids=ids, weights=w)
    assert got[0] is ids and got[1] is w
    a = q.route_experts(part.contiguous(), 4)
    assert torch.equal(a[0], ids) and torch.equal(a[1], w)
    e = q.route_experts(torch.empty((0, 8), device=DEV), 2)
    assert e[0].shape == (0, 2)


def test_captured_and_on_another_stream():
    g = torch.Generator(device=DEV).manual_seed(5)
    logits = torch.randn((50, 64), device=DEV, generator=g)
    want = q.route_experts(logits, 8)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    ids, w = (torch.empty_like(t) for t in want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        q.route_experts(logits, 8, ids=ids, weights=w)
    logits.copy_(torch.randn((50, 64), device=DEV, generator=g))
    graph.replay()
    torch.cuda.synchronize()
    again = q.route_experts(logits, 8)
    assert torch.equal(again[0], ids) and torch.equal(again[1], w)
    assert not torch.equal(want[0], ids)
