"""What the calls keep for the next one: scratch of ordinary sizes, nothing of large ones."""
import numpy as np
import pytest

import qmm_synth

torch = pytest.importorskip("torch")
import quantized_weight_gguf_gb300 as q  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def test_scratch_of_a_large_call_goes_back():
    from quantized_weight_gguf_gb300 import build_lib
    build_lib.build()
    q.load()
    rng = np.random.default_rng(0)
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    k, n_ff, n_exp, n_pos, top_k = 2048, 256, 2, 8191, 8
    wg, wu, wd = (torch.from_numpy(qmm_synth.gen_weights("q8_0", a, b * n_exp, rng)).to(DEV)
                  for a, b in ((k, n_ff), (k, n_ff), (n_ff, k)))
    x = torch.randn(n_pos, k, device=DEV)
    ids = torch.randint(0, n_exp, (n_pos, top_k), dtype=torch.int32, device=DEV)
    weights = torch.rand(n_pos, top_k, device=DEV)

    def call(n, **kw):
        return q.experts_ffn("swiglu", "q8_0", wg, wu, "q8_0", wd, x[:n], ids[:n], weights[:n], k, n_ff, n_exp, **kw)
    small = call(40)                             # its scratch is kept
    y = call(n_pos)                              # more than 800 MB of scratch
    torch.cuda.synchronize()
    held = torch.cuda.memory_allocated()
    again = [call(n_pos) for _ in range(3)]
    torch.cuda.synchronize()
    assert all(torch.equal(y, a) for a in again)
    del again
    assert torch.cuda.memory_allocated() == held
    own = sum(t.numel() * t.element_size() for t in (wg, wu, wd, x, ids, weights, y, small))
    assert held - before < own + (1 << 28) + (1 << 21)
    assert torch.equal(call(40), small)
    q.qmm_device_status()
