"""The experts' feed-forward network on the GPU against the formula in 64 bits over the oracle's weights
(experts_reference, where the tolerance is derived)."""
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


def _weights(fmt, k, n, rng):
    if fmt in ("bf16", "f16"):
        return qmm_synth.gen_weights(fmt, k, n, rng, std=k ** -0.5)
    return qmm_synth.gen_weights(fmt, k, n, rng)


class Case:
    def __init__(self, act, fmt, fmt_down, n_pos, k, n_ff, n_exp, top_k, seed=0):
        rng = np.random.default_rng(1000 * n_pos + k + n_ff + seed)
        self.act, self.fmt, self.fmt_down = act, fmt, fmt_down
        self.k, self.n_ff, self.n_exp = k, n_ff, n_exp
        self.wg, self.wu = (_weights(fmt, k, n_ff * n_exp, rng) for _ in range(2))
        self.wd = _weights(fmt_down, n_ff, k * n_exp, rng)
        self.x = rng.standard_normal((n_pos, k)).astype(np.float32)
        self.ids = rng.integers(0, n_exp, (n_pos, top_k)).astype(np.int32)
        self.weights = rng.random((n_pos, top_k)).astype(np.float32)

    def device(self):
        if not hasattr(self, "_d"):
            self._d = [_dev(a) for a in (self.wg, self.wu, self.wd)]
        return self._d

    def call(self, x=None, ids=None, weights=None, **kw):
        wg, wu, wd = self.device()
        return q.experts_ffn(self.act, self.fmt, wg, wu, self.fmt_down, wd,
                             _dev(self.x) if x is None else x, _dev(self.ids) if ids is None else ids,
                             _dev(self.weights) if weights is None else weights, self.k, self.n_ff, self.n_exp, **kw)

    def check(self, y=None, y0=None, status=0):
        if y is None:
            y = self.call() if y0 is None else self.call(y=_dev(y0), accumulate=True)
        torch.cuda.synchronize()
        if status == 0:
            q.qmm_device_status()
        else:
            with pytest.raises(q.QmmError) as e:
                q.qmm_device_status()
            assert e.value.status == status
        want, tol = ref.ffn(self.act, self.fmt, self.wg, self.wu, self.fmt_down, self.wd, self.x, self.ids,
                            self.weights, self.k, self.n_ff, self.n_exp, y0)
        got = y.cpu().numpy()
        bad = ~(np.abs(got - want) <= tol)
        assert not bad.any(), (bad.sum(), got[bad][:4], want[bad][:4], tol[bad][:4])
        return got


FORMATS = ["q4_0", "q4_k", "q6_k", "q8_0", "q5_0", "f16", "bf16"]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("n_pos,n_exp,top_k", [(1, 5, 3), (2, 4, 1), (9, 3, 2), (40, 5, 2), (70, 3, 2)])
def test_every_format(fmt, n_pos, n_exp, top_k):
    Case("swiglu", fmt, fmt, n_pos, 512, 256, n_exp, top_k).check()


@pytest.mark.parametrize("fmt,fmt_down", [("q4_k", "q6_k"), ("q5_0", "q8_0"), ("q4_k", "bf16"), ("bf16", "q4_0"),
                                          ("q6_k", "q5_0"), ("f16", "q4_k")])
@pytest.mark.parametrize("n_pos", [1, 6, 33])
def test_mixed_formats(fmt, fmt_down, n_pos):
    Case("geglu", fmt, fmt_down, n_pos, 768, 512, 4, 2).check()


@pytest.mark.parametrize("fmt,k,n_ff", [("q4_0", 32, 32), ("q4_0", 96, 160), ("q5_0", 288, 96), ("q8_0", 1376, 352),
                                        ("q8_0", 32, 1056), ("q6_k", 256, 1280), ("q4_k", 1280, 256),
                                        ("f16", 2, 2), ("f16", 34, 70), ("bf16", 130, 258), ("bf16", 1290, 30),
                                        ("f16", 644, 332)])
@pytest.mark.parametrize("n_pos", [1, 3, 20])
def test_odd_sizes(fmt, k, n_ff, n_pos):
    Case("swiglu", fmt, fmt, n_pos, k, n_ff, 3, 2).check()


@pytest.mark.parametrize("fmt,fmt_down", [(f, f) for f in FORMATS] + [("q4_k", "q8_0"), ("q8_0", "q6_k"), ("f16", "q5_0")])
def test_few_rows_to_many_experts(fmt, fmt_down):
    Case("swiglu", fmt, fmt_down, 5, 768, 512, 24, 4).check()


@pytest.mark.parametrize("fmt,k", [("q4_k", 5120), ("q4_k", 5376), ("q8_0", 5152), ("bf16", 5130), ("q6_k", 5376)])
@pytest.mark.parametrize("n_pos", [1, 2])
def test_wide_rows(fmt, k, n_pos):
    Case("geglu", fmt, "q8_0", n_pos, k, 64, 4, 2).check()


@pytest.mark.parametrize("n_pos", [1, 12])
def test_accumulates(n_pos):
    c = Case("geglu", "q4_k", "q6_k", n_pos, 512, 256, 6, 3)
    c.check(y0=np.random.default_rng(1).standard_normal((n_pos, c.k)).astype(np.float32))


@pytest.mark.parametrize("n_pos", [1, 7])
def test_in_place(n_pos):
    c = Case("swiglu", "q8_0", "q8_0", n_pos, 512, 256, 6, 3)
    x = _dev(c.x)
    y = c.call(x=x, y=x, accumulate=True)
    assert y.data_ptr() == x.data_ptr()
    want, tol = ref.ffn(c.act, c.fmt, c.wg, c.wu, c.fmt_down, c.wd, c.x, c.ids, c.weights, c.k, c.n_ff, c.n_exp, c.x)
    assert (np.abs(y.cpu().numpy() - want) <= tol).all()


@pytest.mark.parametrize("fmt", ["q4_k", "bf16"])
@pytest.mark.parametrize("n_pos", [1, 5, 40])
def test_empty_slots_and_repeated_experts(fmt, n_pos):
    c = Case("swiglu", fmt, fmt, n_pos, 256, 256, 4, 4)
    c.ids[0] = [2, 2, -1, 2]                    # the same index three times, one slot empty
    c.weights[0, 2] = np.nan                    # of an empty slot: not read
    if n_pos > 1:
        c.ids[1] = -1                           # a position without experts
        c.weights[1] = np.inf
    got = c.check()
    if n_pos > 1:
        assert (got[1] == 0).all()


@pytest.mark.parametrize("n_pos", [1, 30])
def test_every_position_takes_one_expert(n_pos):
    c = Case("swiglu", "q4_0", "q4_0", n_pos, 256, 96, 200, 2)
    c.ids[:] = 199
    c.check()


@pytest.mark.parametrize("n_pos", [1, 4])
def test_no_expert_at_all(n_pos):
    c = Case("swiglu", "q4_k", "q4_k", n_pos, 512, 256, 4, 2)
    c.ids[:] = -1
    assert (c.check() == 0).all()
    y0 = np.random.default_rng(1).standard_normal((n_pos, c.k)).astype(np.float32)
    assert (c.check(y0=y0) == y0).all()


@pytest.mark.parametrize("n_pos", [1, 8])
def test_bad_ids_add_nothing_and_are_reported(n_pos):
    c = Case("swiglu", "q8_0", "q8_0", n_pos, 512, 256, 4, 3)
    c.ids[0, 1] = 4
    c.check(status=11)
    c.ids[0, 1] = -2
    c.check(status=11)
    c.ids[0, 1] = 2 ** 31 - 1
    c.check(status=11)
    c.ids[0, 1] = 3
    c.check()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("n_pos", [1, 10])
def test_slices_that_no_id_names_are_not_read(fmt, n_pos):
    """Their bytes are NaN in every format that has NaN; the results are those without them."""
    c = Case("swiglu", fmt, fmt, n_pos, 256, 256, 5, 2)
    c.ids %= 2
    c.ids[c.ids == 1] = 3
    for w in (c.wg, c.wu, c.wd):
        per = w.reshape(5, -1)
        per[[0, 2, 4]] = np.where(np.isin([0, 2, 4], np.unique(c.ids))[:, None], per[[0, 2, 4]], 0xFF)
    c.check()


@pytest.mark.parametrize("fmt", ["q4_k", "q8_0", "bf16"])
@pytest.mark.parametrize("n_pos", [1, 12])
def test_values_of_any_size(fmt, n_pos):
    """Rows of x from 1e-30 to 1e30, and values within a row that differ by 2^20."""
    c = Case("swiglu", fmt, fmt, n_pos, 512, 256, 4, 2)
    c.x *= (2.0 ** np.random.default_rng(2).integers(-10, 11, c.x.shape)).astype(np.float32)
    c.weights[:] = 1.0
    c.check()
    c.x[0] = c.x[0] * np.float32(1e-30)
    c.check()


@pytest.mark.parametrize("n_pos", [1, 9])
def test_a_nan_or_inf_stays_in_its_position(n_pos):
    c = Case("swiglu", "q4_k", "q6_k", max(n_pos, 2), 512, 256, 4, 2)
    for bad in (np.nan, np.inf, -np.inf):
        x = c.x.copy()
        x[0, 77] = bad
        if n_pos == 1:
            y = c.call(x=_dev(x[:1]), ids=_dev(c.ids[:1]), weights=_dev(c.weights[:1])).cpu().numpy()
        else:
            y = c.call(x=_dev(x)).cpu().numpy()
            assert np.isfinite(y[1:]).all()
            np.testing.assert_array_equal(y[1:], c.call().cpu().numpy()[1:])
        assert not np.isfinite(y[0]).any()


def test_the_same_call_gives_the_same_result():
    c = Case("geglu", "q4_k", "q6_k", 50, 512, 512, 5, 3)
    first = c.call()
    for _ in range(5):
        assert torch.equal(first, c.call())


@pytest.mark.parametrize("n_pos", [1, 7])
def test_a_positions_result_does_not_depend_on_the_others(n_pos):
    """Appending positions changes no bit of the first ones while the tile's width stays the same."""
    c = Case("swiglu", "q5_0", "q8_0", n_pos + 6, 288, 96, 64, 2)
    all_y = c.call()
    some = c.call(x=_dev(c.x[3:]), ids=_dev(c.ids[3:]), weights=_dev(c.weights[3:]))
    assert torch.equal(all_y[3:], some)


@pytest.mark.parametrize("n_pos", [1, 6])
def test_captured_twice_and_on_streams(n_pos):
    """Two graphs with workspaces of their own, replayed with new inputs, and calls on two streams at once."""
    c = Case("swiglu", "q4_k", "q4_k", n_pos, 512, 512, 6, 3)
    x, ids, w = _dev(c.x), _dev(c.ids), _dev(c.weights)
    want = c.call(x=x, ids=ids, weights=w).clone()
    graphs, outs = [], []
    for _ in range(2):
        y, g = torch.empty_like(x), torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.call(x=x, ids=ids, weights=w, y=y)
        graphs.append(g)
        outs.append(y)
    for g in graphs:
        g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)
    ids.copy_((ids + 1) % c.n_exp)
    x.mul_(0.5)
    want2 = c.call(x=x, ids=ids, weights=w)
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    for s in (a, b):
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(20):
        with torch.cuda.stream(a):
            graphs[0].replay()
        with torch.cuda.stream(b):
            graphs[1].replay()
        other = c.call(x=x, ids=ids, weights=w, stream=a)
    torch.cuda.synchronize()
    assert all(torch.equal(o, want2) for o in (*outs, other))


def test_given_workspace_and_no_positions():
    c = Case("swiglu", "q8_0", "q8_0", 5, 512, 256, 4, 2)
    want = c.call()
    ws = torch.empty(1 << 22, dtype=torch.uint8, device=DEV)
    assert torch.equal(c.call(workspace=ws), want)
    with pytest.raises(q.QmmError) as e:
        c.call(workspace=ws[:1024])
    assert e.value.status == 9
    none = c.call(x=torch.empty((0, 512), device=DEV), ids=torch.empty((0, 2), dtype=torch.int32, device=DEV),
                  weights=torch.empty((0, 2), device=DEV))
    assert none.shape == (0, 512)


def test_refuses_other_tensors():
    c = Case("swiglu", "q8_0", "q8_0", 2, 64, 32, 4, 2)
    x, ids, w = _dev(c.x), _dev(c.ids), _dev(c.weights)
    for kw in (dict(x=x.cpu()), dict(ids=ids.long()), dict(weights=w.cpu()), dict(weights=w[:1]), dict(x=x.double()),
               dict(y=torch.empty((2, 32), device=DEV)), dict(x=x.t().contiguous().t())):
        with pytest.raises(ValueError):
            c.call(**kw)


# Experts with more than 20 rows each: tiles of up to 48 pairs, whole, partly filled and empty.
@pytest.mark.parametrize("fmt,fmt_down,k,n_ff", [
    ("q4_0", "q4_0", 32, 32), ("q4_0", "q5_0", 96, 160), ("q5_0", "q8_0", 288, 96), ("q8_0", "q8_0", 1376, 352),
    ("q8_0", "q4_0", 32, 1056), ("q6_k", "q6_k", 256, 1280), ("q4_k", "q4_k", 1280, 256), ("q4_k", "q6_k", 512, 768),
    ("q6_k", "q5_0", 768, 416), ("q5_0", "q4_k", 2080, 512)])
@pytest.mark.parametrize("n_pos,n_exp,top_k", [(21, 1, 1), (48, 1, 1), (49, 1, 1), (97, 4, 2), (150, 2, 1)])
def test_many_rows(fmt, fmt_down, k, n_ff, n_pos, n_exp, top_k):
    Case("geglu" if n_pos == 97 else "swiglu", fmt, fmt_down, n_pos, k, n_ff, n_exp, top_k).check()


def test_many_rows_accumulate_in_place_and_leave_slots_empty():
    c = Case("swiglu", "q4_k", "q8_0", 60, 512, 256, 3, 2)
    c.check(y0=np.random.default_rng(1).standard_normal((60, c.k)).astype(np.float32))
    x = _dev(c.x)
    c.check(y=c.call(x=x, y=x))
    rng = np.random.default_rng(2)
    c.ids[rng.random(c.ids.shape) < 0.2] = -1
    c.ids[7] = -1
    c.ids[8] = 2
    c.check()
    c.ids[:] = 1
    c.check()


def test_many_rows_of_any_size():
    c = Case("swiglu", "q4_k", "q5_0", 64, 768, 512, 2, 1)
    c.x *= np.exp2(np.random.default_rng(3).integers(-30, 30, (64, 1))).astype(np.float32)
    c.x[5] = 0
    c.check()


def test_a_nan_or_inf_among_many_rows_stays_in_its_position():
    c = Case("swiglu", "q8_0", "q4_k", 70, 512, 512, 2, 1)
    clean = c.call().cpu().numpy()
    c.x[3, 100], c.x[11, 7] = np.nan, np.inf
    got = c.call().cpu().numpy()
    bad = [3, 11]
    assert not np.isfinite(got[bad]).any()
    keep = np.setdiff1d(np.arange(70), bad)
    assert np.array_equal(got[keep], clean[keep])


def test_many_rows_captured_and_on_another_stream():
    c = Case("swiglu", "q4_k", "q4_k", 130, 512, 256, 4, 2)
    want = c.call().cpu().numpy()
    x, y = _dev(c.x), torch.empty(130, c.k, device=DEV)
    ids, weights = _dev(c.ids), _dev(c.weights)
    c.call(x=x, ids=ids, weights=weights, y=y)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.call(x=x, ids=ids, weights=weights, y=y)
    s = torch.cuda.Stream()
    for _ in range(3):
        y.zero_()
        g.replay()
        assert np.array_equal(y.cpu().numpy(), want)
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            z = c.call(x=x, ids=ids, weights=weights)
        s.synchronize()
        assert np.array_equal(z.cpu().numpy(), want)


def test_many_rows_on_two_streams_at_once():
    """Both calls' CTAs share SMs and their tensor memory, also with the tensor-core product of qmm_matmul."""
    cases = [Case("swiglu", f, f, 200, 1024, 512, 4, 2, seed=i) for i, f in enumerate(("q4_k", "q8_0"))]
    want = [c.call().cpu().numpy() for c in cases]
    args = [(_dev(c.x), _dev(c.ids), _dev(c.weights)) for c in cases]
    streams = [torch.cuda.Stream() for _ in range(3)]
    outs = [[torch.empty(200, 1024, device=DEV) for _ in range(6)] for _ in cases]
    rng = np.random.default_rng(4)
    w, x = _dev(qmm_synth.gen_weights("q4_k", 1024, 4096, rng)), _dev(rng.standard_normal((256, 1024)).astype(np.float32))
    dense = q.matmul("q4_k", w, x, 1024, 4096)
    torch.cuda.synchronize()
    for i in range(6):
        for c, a, s, o in zip(cases, args, streams, outs):
            with torch.cuda.stream(s):
                c.call(x=a[0], ids=a[1], weights=a[2], y=o[i])
        with torch.cuda.stream(streams[2]):
            again = q.matmul("q4_k", w, x, 1024, 4096)
    torch.cuda.synchronize()
    q.qmm_device_status()
    assert torch.equal(again, dense)
    for o, y in zip(outs, want):
        assert all(np.array_equal(t.cpu().numpy(), y) for t in o)


@pytest.mark.parametrize("n_pos", [30, 64])
def test_many_rows_without_any_expert(n_pos):
    c = Case("swiglu", "q4_k", "q4_k", n_pos, 256, 256, 1, 1)
    c.ids[:] = -1
    c.check()
    c.ids[5] = 7                                 # of none
    c.check(status=11)

