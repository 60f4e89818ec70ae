"""The attention block example (product, append, attention, product) against
the same steps in 64 bits: a prompt chunk, then single tokens, the cache read
back between them."""
import importlib.util
import os

import numpy as np
import pytest

import kv_reference as ref
import oracle

torch = pytest.importorskip("torch")
import quantized_weight_gguf_gb300 as q  # noqa: E402

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    from quantized_weight_gguf_gb300 import build_lib
    build_lib.build()
    q.load()
    oracle.build()
    path = os.path.join(ROOT, "examples", "attention_block.py")
    spec = importlib.util.spec_from_file_location("attention_block", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    yield mod
    q.qmm_device_status()


@pytest.mark.parametrize("cache", ["q8_0", "f16"])
def test_block_follows_its_steps_in_64_bits(example, cache):
    """Each call's output against the 64-bit product of the weights with the attention of the rows
    that the cache holds. Bar: the products' own 1e-4 of sum |x w|, for the second product on the
    attention's output, plus the first one's, carried through the softmax: a score of
    unit-sized q and k moves by at most 1e-3, and the output by as much of its size."""
    width, h, n, d, n_seqs = 512, 8, 2, 64, 2
    block = example.AttentionBlock(width, h, n, d, n_seqs, 64, cache, page=16, seed=3)
    w_qkv = q.dequant("q4_k", block.w_qkv, width, block.n_qkv).double().cpu().numpy()
    w_out = q.dequant("q4_k", block.w_out, h * d, width).double().cpu().numpy()
    rope = block.rope.cpu().numpy()
    rng = np.random.default_rng(4)
    table = block.page_table.cpu().numpy()
    held = 0
    for n_new in (19, 1, 1, 3):
        x0 = rng.standard_normal((n_seqs, n_new, width)).astype(np.float32)
        x = torch.from_numpy(x0.copy()).to("cuda:0")
        block(x)
        torch.cuda.synchronize()
        held += n_new
        assert block.lens.tolist() == [held] * n_seqs
        k, v = (t.double().cpu().numpy() for t in q.kv_read(block.cache, block.page_table, block.lens, held, first=0))
        x64 = x0.astype(np.float64)
        x64 /= np.sqrt((x64 ** 2).mean(-1, keepdims=True) + 1e-6)
        qkv = (x64 @ w_qkv.T).reshape(n_seqs, n_new, -1, d)
        for s in range(n_seqs):
            for i in range(n_new):
                pos = held - n_new + i
                rows = ref.rotate(qkv[s, i, :h], pos, rope, d, "half", np.float64)
                o, _ = ref.attention(rows, k[s], v[s], 0, pos, d ** -0.5)
                want = x0[s, i] + w_out @ o.reshape(-1)
                bar = 1e-4 * np.abs(w_out) @ np.abs(o.reshape(-1)) + 2e-3 * np.abs(w_out) @ np.full(h * d, np.abs(v[s]).max())
                assert (np.abs(x[s, i].double().cpu().numpy() - want) <= bar + 1e-6).all()
                # what the cache holds of the new key is the product's, rotated
                want_k = ref.rotate(qkv[s, i, h:h + n], pos, rope, d, "half", np.float64)
                step = 0.01 if cache == "q8_0" else 1e-3
                assert np.abs(k[s, pos] - want_k).max() <= step * np.abs(want_k).max() + 1e-3
    assert q.qmm_device_status() == 0
    assert (table == block.page_table.cpu().numpy()).all()
