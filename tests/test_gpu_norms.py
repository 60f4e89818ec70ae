"""Norms of the errors of the experts' network (per position) and of linear attention (per head) on the GPU, for every
kernel that they take, within the bounds of norm_bounds."""
import numpy as np
import pytest

import norm_bounds
import oracle
import qmm_synth

torch = pytest.importorskip("torch")
import quantized_weight_gguf_gb300 as q  # noqa: E402

DEV = "cuda:0"


class FfnInputs:
    def __init__(self, act, fmt, fmt_down, n_pos, k, n_ff, n_exp, top_k):
        rng = np.random.default_rng(100 * n_pos + k + n_ff)
        self.act, self.fmt, self.fmt_down, self.k, self.n_ff, self.n_exp = act, fmt, fmt_down, k, n_ff, n_exp

        def weights(f, a, n):
            return qmm_synth.gen_weights(f, a, n, rng, **({"std": a ** -0.5} if f in ("bf16", "f16") else {}))
        self.wg, self.wu = (weights(fmt, k, n_ff * n_exp) for _ in range(2))
        self.wd = weights(fmt_down, n_ff, k * n_exp)
        self.x = rng.standard_normal((n_pos, k)).astype(np.float32)
        self.ids = rng.integers(0, n_exp, (n_pos, top_k)).astype(np.int32)
        self.weights = (0.5 + rng.random((n_pos, top_k))).astype(np.float32)

    def want(self, x=None):
        return norm_bounds.ffn(self.act, self.fmt, self.wg, self.wu, self.fmt_down, self.wd, self.x if x is None else x,
                               self.ids, self.weights, self.k, self.n_ff, self.n_exp)

    def call(self):
        wg, wu, wd, x, ids, w = (torch.from_numpy(np.ascontiguousarray(a)).to(DEV)
                                 for a in (self.wg, self.wu, self.wd, self.x, self.ids, self.weights))
        return q.experts_ffn(self.act, self.fmt, wg, wu, self.fmt_down, wd, x, ids, w, self.k, self.n_ff,
                             self.n_exp).cpu().numpy()


class LinearInputs:
    def __init__(self, n_new, n_heads, n_qk, dk, dv, rate):
        rng = np.random.default_rng(n_new + dk + dv)
        self.q, self.k = (rng.standard_normal((1, n_new, n_qk, dk)).astype(np.float32) for _ in range(2))
        self.v = rng.standard_normal((1, n_new, n_heads, dv)).astype(np.float32)
        self.decay = (-rate * np.abs(rng.standard_normal((1, n_new, n_heads)))).astype(np.float32)
        self.state = rng.standard_normal((1, n_heads, dk, dv)).astype(np.float32)
        self.scale = dk ** -0.5

    def want(self, **other):
        a = {n: other.get(n, getattr(self, n)) for n in ("q", "k", "v")}
        return norm_bounds.linear(a["q"], a["k"], a["v"], self.decay, self.state, self.scale)

    def call(self):
        *args, state = (torch.from_numpy(a).to(DEV) for a in (self.q, self.k, self.v, self.decay, self.state))
        out = q.linear_attend(*args, state, scale=self.scale)
        return out.cpu().numpy(), state.cpu().numpy()


# one position; few rows; tiles of 8, 16 and 48 columns
FFN = [("swiglu", f, d, n_pos, 512 if f in ("q4_k", "q6_k") else 1376, 256 if d in ("q4_k", "q6_k") else 352, n_exp, 2)
       for f, d in (("q4_0", "q5_0"), ("q4_k", "q6_k"), ("q8_0", "q8_0"), ("q5_0", "q4_k"), ("q6_k", "q4_0"), ("bf16", "f16"),
                    ("f16", "bf16"))
       for n_pos, n_exp in ((1, 4), (4, 12), (6, 4), (24, 4), (45, 4))] \
    + [("geglu", "q5_0", "q4_k", 150, 2080, 512, 2, 1), ("geglu", "q4_k", "q8_0", 3, 4096, 1024, 8, 2)]
LINEAR = [(1, 2, 2, 64, 64, 0.1), (8, 2, 1, 128, 128, 0.1), (9, 2, 2, 64, 64, 0.1), (33, 2, 1, 128, 128, 0.01),
          (300, 3, 3, 96, 160, 0.3), (700, 2, 2, 32, 256, 2.0), (2000, 2, 1, 128, 128, 1e-4)]


@pytest.fixture()
def lib():
    from quantized_weight_gguf_gb300 import build_lib
    build_lib.build()
    q.load()
    oracle.build()
    yield
    q.qmm_device_status()


@pytest.mark.gpu
@pytest.mark.parametrize("case", FFN, ids=str)
def test_norms_of_the_experts_errors(lib, case):
    c = FfnInputs(*case)
    want, bound = c.want()
    off = np.linalg.norm(c.call() - want, axis=1)
    assert (off <= bound).all(), (off / bound).max()


@pytest.mark.gpu
@pytest.mark.parametrize("case", LINEAR, ids=str)
def test_norms_of_linear_attentions_errors(lib, case):
    c = LinearInputs(*case)
    w_out, w_state, o_bound, s_bound = c.want()
    out, state = c.call()
    for got, want, bound, axes in ((out, w_out, o_bound, (1, 3)), (state, w_state, s_bound, (2, 3))):
        off = np.linalg.norm(got - want, axis=axes)
        assert (off <= bound).all(), (off / bound).max()
