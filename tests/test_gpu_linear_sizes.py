"""Linear attention over values of very different sizes, against its recurrence in 64 bits (linear_causal, where the
tolerance is derived): a row is as exact as the rows up to its own, decayed, let it be."""
import numpy as np
import pytest

import linear_causal as ref

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


class Case:
    def __init__(self, n_new, n_heads=2, n_qk=2, dk=64, dv=64, rate=0.05):
        rng = np.random.default_rng(n_new)
        self.q, self.k = (rng.standard_normal((1, n_new, n_qk, dk)).astype(np.float32) for _ in range(2))
        self.v = rng.standard_normal((1, n_new, n_heads, dv)).astype(np.float32)
        self.decay = (-rate * np.abs(rng.standard_normal((1, n_new, n_heads)))).astype(np.float32)
        self.state = rng.standard_normal((1, n_heads, dk, dv)).astype(np.float32)
        self.scale = 0.125

    def call(self):
        *args, state = (torch.from_numpy(a).to(DEV) for a in (self.q, self.k, self.v, self.decay, self.state))
        out = q.linear_attend(*args, state, scale=self.scale)
        torch.cuda.synchronize()
        return out.cpu().numpy(), state.cpu().numpy()

    def check(self):
        out, state = self.call()
        w_out, w_state, tol, s_tol = ref.attend(self.q, self.k, self.v, self.decay, self.state, self.scale)
        for name, a, b, t in (("out", out, w_out, tol), ("state", state, w_state, s_tol)):
            bad = ~(np.abs(a - b) <= t)
            assert not bad.any(), (name, bad.sum(), np.argwhere(bad)[:3], a[bad][:3], b[bad][:3], t[bad][:3])


@pytest.mark.parametrize("n_new,at", [(6, 4), (20, 18), (32, 31), (40, 16), (100, 50), (400, 397), (400, 140)])
@pytest.mark.parametrize("what", ["k", "v", "k and v", "a dim of v"])
@pytest.mark.parametrize("power", [24, 60])
def test_a_large_row_leaves_the_rows_before_it_as_they_are(n_new, at, what, power):
    c = Case(n_new)
    if "k" in what:
        c.k[:, at] *= np.float32(2.0 ** power)
    if what in ("v", "k and v"):
        c.v[:, at] *= np.float32(2.0 ** power)
    if what == "a dim of v":
        c.v[:, at, :, 5] *= np.float32(2.0 ** power)
    c.check()


@pytest.mark.parametrize("n_new,at", [(7, 1), (20, 2), (40, 16), (40, 30), (100, 50), (400, 140)])
@pytest.mark.parametrize("what", ["k", "v", "state"])
@pytest.mark.parametrize("power", [24, 60])
def test_a_large_row_that_is_cleared_leaves_the_rows_after_it_as_they_are(n_new, at, what, power):
    c = Case(n_new)
    a = {"k": c.k[:, at], "v": c.v[:, at], "state": c.state}[what]
    a *= np.float32(2.0 ** power)
    c.decay[:, at + 3] = -np.inf
    c.check()
    c.decay[:, at + 3] = -40.0
    c.check()


@pytest.mark.parametrize("n_new", [7, 30, 100, 400])
@pytest.mark.parametrize("what", ["k", "v"])
def test_rows_that_fade_as_fast_as_they_shrink(n_new, what):
    """Every row is half as large as the one before and forgets it as fast; at the end 2^-126 of the first one."""
    c = Case(n_new)
    at = np.arange(n_new) % 100
    getattr(c, what)[:] *= (2.0 ** (60.0 - at * 1.26))[None, :, None, None].astype(np.float32)
    c.decay[:] = -2.0
    c.check()


# powers of two that q, k, v and the state are multiplied by: what they give, and the products on the way there, are
# numbers that fp32 holds
RANGES = [(0, 0, -106, -106), (0, -106, 0, -106), (-83, -17, -17, -34), (-110, 0, 0, 0), (100, -60, -40, -100),
          (60, -100, 40, -60), (-100, 60, 40, 100), (-90, 100, 15, 115), (110, -52, -53, -105), (-20, 118, -118, 0),
          (0, -100, 118, 18), (118, -110, -5, -115), (4, 56, 56, 112), (-8, 2, 112, 114)]


@pytest.mark.parametrize("n_new", [5, 9, 40, 70, 400])
@pytest.mark.parametrize("powers", RANGES)
def test_sizes_whose_products_fp32_holds(n_new, powers):
    c = Case(n_new)
    for name, n in zip("qkv", powers):
        a = getattr(c, name)
        a *= np.float32(2.0 ** n)
    c.state *= np.float32(2.0 ** powers[3])
    c.check()


@pytest.mark.parametrize("n_new", [5, 9, 70, 400])
def test_large_values_that_meet_zeros_give_zeros(n_new):
    """q at one dim, k and the state's rows at others: every output is exactly zero, and the state what k v give."""
    c = Case(n_new)
    c.q[:], c.k[:] = 0, 0
    c.q[..., 3], c.k[..., 5] = 2.0 ** 100, 2.0 ** 60
    c.state *= np.float32(2.0 ** 60)
    c.state[:, :, 3] = 0
    out, _ = c.call()
    assert (out == 0).all()
    c.check()


@pytest.mark.parametrize("n_new", [5, 40, 400])
def test_rows_of_zeros_among_small_and_large_ones(n_new):
    for power in (-100, 0, 100):
        c = Case(n_new)
        c.q *= np.float32(2.0 ** -power)
        c.v *= np.float32(2.0 ** power)
        c.state *= np.float32(2.0 ** power)
        for a in (c.q, c.k, c.v):
            a[:, ::3] = 0
        c.check()
        c.v[:] = 0
        c.check()
