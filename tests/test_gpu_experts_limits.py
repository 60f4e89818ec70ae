"""The experts' network at the ends of what it accepts: thousands of experts (several for each thread that sorts), 65535
pairs, against the formula in 64 bits (experts_reference, where the tolerance is derived)."""
import numpy as np
import pytest

import experts_reference as ref
import oracle
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
    oracle.build()
    yield
    q.qmm_device_status()


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def _check(fmt, n_pos, n_exp, top_k, ids=None, k=32, n_ff=32):
    rng = np.random.default_rng(n_pos + n_exp)
    wg, wu, wd = (qmm_synth.gen_weights(fmt, a, b * n_exp, rng, **({"std": 0.2} if fmt == "bf16" else {}))
                  for a, b in ((k, n_ff), (k, n_ff), (n_ff, k)))
    x = rng.standard_normal((n_pos, k)).astype(np.float32)
    ids = rng.integers(0, n_exp, (n_pos, top_k)) if ids is None else ids
    ids = ids.astype(np.int32)
    weights = rng.random(ids.shape).astype(np.float32)
    y = q.experts_ffn("swiglu", fmt, _dev(wg), _dev(wu), fmt, _dev(wd), _dev(x), _dev(ids), _dev(weights), k, n_ff, n_exp)
    torch.cuda.synchronize()
    q.qmm_device_status()
    want, tol = ref.ffn("swiglu", fmt, wg, wu, fmt, wd, x, ids, weights, k, n_ff, n_exp)
    bad = ~(np.abs(y.cpu().numpy() - want) <= tol)
    assert not bad.any(), (bad.sum(), np.argwhere(bad)[:4])


@pytest.mark.parametrize("n_exp", [255, 256, 257, 300, 513, 1000, 4096])
@pytest.mark.parametrize("per_expert", [0.5, 3, 12, 30])
def test_many_experts(n_exp, per_expert):
    top_k = 7
    _check("q8_0", max(2, int(per_expert * n_exp / top_k)) if n_exp < 4096 or per_expert < 30 else 9362, n_exp, top_k)


@pytest.mark.parametrize("fmt", ["q4_0", "bf16"])
@pytest.mark.parametrize("n_exp", [3, 700, 4096])
def test_65535_pairs(fmt, n_exp):
    _check(fmt, 13107, n_exp, 5)


def test_all_pairs_are_the_last_of_many_experts_or_none():
    ids = np.full((200, 8), 4095)
    ids[::3, 2:] = -1
    ids[5] = -1
    _check("q8_0", 200, 4096, 8, ids=ids)


def test_64_slots_and_one_position():
    _check("q8_0", 1, 4096, 64)
    _check("q8_0", 70, 1000, 64)
