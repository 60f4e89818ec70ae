"""The experts' network on a stream that is not torch's current one, while that one is busy: nothing that a call needs
may wait there."""
import numpy as np
import pytest

import qmm_synth

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


def _case(n_pos, top_k=2, n_exp=4, k=512, n_ff=256):
    rng = np.random.default_rng(n_pos)
    w = [torch.from_numpy(qmm_synth.gen_weights("q8_0", a, b * n_exp, rng)).to(DEV) for a, b in ((k, n_ff), (k, n_ff), (n_ff, k))]
    x = torch.from_numpy(rng.standard_normal((n_pos, k)).astype(np.float32)).to(DEV)
    ids = torch.from_numpy(rng.integers(0, n_exp, (n_pos, top_k)).astype(np.int32)).to(DEV)
    weights = torch.from_numpy(rng.random((n_pos, top_k)).astype(np.float32)).to(DEV)

    def call(ids=ids, weights=weights, **kw):
        return q.experts_ffn("swiglu", "q8_0", w[0], w[1], "q8_0", w[2], x, ids, weights, k, n_ff, n_exp, **kw)
    return call, ids, weights


@pytest.mark.parametrize("n_pos", [1, 6, 100])
def test_adding_to_no_y_is_the_sum_alone(n_pos):
    call, _, _ = _case(n_pos)
    want = call()
    assert torch.equal(call(accumulate=True), want)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    torch.cuda._sleep(100_000_000)               # some 50 ms of work on the current stream
    y = call(accumulate=True, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(y, want)


def test_weights_that_would_have_to_be_copied_are_refused():
    call, ids, weights = _case(1, top_k=8)
    want = call()
    assert torch.equal(call(ids=ids[0], weights=weights[0]), want)
    assert torch.equal(call(ids=ids[0], weights=weights), want)
    with pytest.raises(ValueError):
        call(ids=ids[0], weights=weights.view(4, 2).t())
    with pytest.raises(ValueError):
        call(ids=ids[0], weights=weights.repeat(2, 1).t()[:, 0].as_strided((8,), (2,)))


@pytest.mark.parametrize("n_pos", [1, 6])
def test_scratch_of_a_call_on_the_default_stream_stays_its_own(n_pos):
    """Its memory is not handed out on the current stream while the default one, which is busy, has yet to use it."""
    call, _, _ = _case(n_pos)
    want = call()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        y = torch.empty_like(want)
        with torch.cuda.stream(torch.cuda.default_stream()):
            torch.cuda._sleep(100_000_000)
        call(y=y, stream=0)
        others = [torch.full((size,), 255, dtype=torch.uint8, device=DEV) for size in (1 << 12, 1 << 14, 1 << 16, 1 << 18)]
    torch.cuda.synchronize()
    assert torch.equal(y, want) and all((o == 255).all() for o in others)
