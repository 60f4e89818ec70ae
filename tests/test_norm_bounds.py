"""The norms' bounds reject what they are there for, without a GPU: results from operands rounded to one fp16 (or bf16)
term, for the shapes of test_gpu_norms; and they pass what plain fp32 sums give."""
import numpy as np
import pytest

import experts_reference as experts
import norm_bounds
import oracle
from test_gpu_norms import FFN, LINEAR, FfnInputs, LinearInputs


def half(a):
    return a.astype(np.float16).astype(np.float32)


@pytest.mark.parametrize("case", FFN, ids=str)
def test_one_term_of_x_or_h_is_noticed(case):
    oracle.build()
    c = FfnInputs(*case)
    want, bound = c.want()
    got, _ = c.want(x=half(c.x))
    assert (np.linalg.norm(got - want, axis=1) > 3 * bound).all()
    # the activated products: h rounded, one expert after the other
    y = np.zeros(want.shape)
    for p in range(c.x.shape[0]):
        for s in range(c.ids.shape[1]):
            g, u, d = (oracle.dequant(f, w.reshape(c.n_exp, -1)[c.ids[p, s]], *kn).astype(np.float64) for f, w, kn in
                       ((c.fmt, c.wg, (c.k, c.n_ff)), (c.fmt, c.wu, (c.k, c.n_ff)), (c.fmt_down, c.wd, (c.n_ff, c.k))))
            h = experts.act(c.act, g @ c.x[p]) * (u @ c.x[p]) * c.weights[p, s]
            y[p] += d @ (half(h / np.abs(h).max()) * np.abs(h).max())
        if p == 3:
            break
    n = p + 1
    assert (np.linalg.norm(y[:n] - want[:n], axis=1) > 3 * bound[:n]).all()


@pytest.mark.parametrize("case", FFN[:4], ids=str)
def test_plain_fp32_sums_pass(case):
    oracle.build()
    c = FfnInputs(*case)
    want, bound = c.want()
    for p in range(min(3, c.x.shape[0])):
        y = np.zeros(c.k, np.float32)
        for s in range(c.ids.shape[1]):
            g, u, d = (oracle.dequant(f, w.reshape(c.n_exp, -1)[c.ids[p, s]], *kn) for f, w, kn in
                       ((c.fmt, c.wg, (c.k, c.n_ff)), (c.fmt, c.wu, (c.k, c.n_ff)), (c.fmt_down, c.wd, (c.n_ff, c.k))))
            h = (experts.act(c.act, g @ c.x[p]) * (u @ c.x[p]) * c.weights[p, s]).astype(np.float32)
            y += d @ h
        assert np.linalg.norm(y - want[p]) <= bound[p]


@pytest.mark.parametrize("case", [c for c in LINEAR if c[0] > 8], ids=str)
@pytest.mark.parametrize("what", ["q", "k", "v"])
def test_one_term_of_q_k_or_v_is_noticed(case, what):
    c = LinearInputs(*case)
    out, state, o_bound, s_bound = c.want()
    got, got_state, _, _ = c.want(**{what: half(getattr(c, what))})
    assert (np.linalg.norm(got - out, axis=(1, 3)) > 3 * o_bound).all()
    if what != "q":
        assert (np.linalg.norm(got_state - state, axis=(2, 3)) > 3 * s_bound).all()
