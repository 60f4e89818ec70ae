"""Linear attention on the GPU against its recurrence in 64 bits (linear_reference, where the tolerance is derived)."""
import numpy as np
import pytest

import linear_reference as ref

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


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


class Case:
    def __init__(self, n_seqs, n_new, n_heads, n_qk, dk, dv, lens=None, constant=False, seed=0, rate=(0.002, 1.0)):
        rng = np.random.default_rng(seed + n_new * 1000 + dk + dv)
        self.q = rng.standard_normal((n_seqs, n_new, n_qk, dk)).astype(np.float32)
        self.k = rng.standard_normal((n_seqs, n_new, n_qk, dk)).astype(np.float32)
        self.v = rng.standard_normal((n_seqs, n_new, n_heads, dv)).astype(np.float32)
        per_head = np.exp(np.linspace(np.log(rate[0]), np.log(rate[1]), n_heads))
        self.constant = constant
        d = -per_head if constant else -per_head * np.abs(rng.standard_normal((n_seqs, n_new, n_heads)))
        self.decay = d.astype(np.float32)
        self.state = rng.standard_normal((n_seqs, n_heads, dk, dv)).astype(np.float32)
        self.lens = None if lens is None else np.array(lens, np.int32)
        self.scale = np.float32(dk ** -0.5)

    def call(self, **kw):
        state = _dev(self.state)
        args = [_dev(a) for a in (self.q, self.k, self.v, self.decay)]
        lens = None if self.lens is None else _dev(self.lens)
        out = q.linear_attend(*args, state, lens, **kw)
        after = kw.get("state_out", state)
        torch.cuda.synchronize()
        q.qmm_device_status()
        return out.cpu().numpy(), after.cpu().numpy()

    def want(self):
        decay = np.broadcast_to(self.decay, self.v.shape[:3])
        return ref.attend(self.q, self.k, self.v, decay, self.state, self.lens, float(self.scale))

    def check(self, got=None, **kw):
        out, state = got or self.call(**kw)
        w_out, w_state, tol, s_tol = self.want()
        for name, a, b, t in (("out", out, w_out, tol), ("state", state, w_state, s_tol)):
            bad = ~((np.abs(a - b) <= t) | (~np.isfinite(a) & ~np.isfinite(b)))
            assert not bad.any(), (name, bad.sum(), np.argwhere(bad)[:3], a[bad][:3], b[bad][:3], t[bad][:3])
        return out, state


DIMS = [(32, 32), (64, 64), (96, 96), (128, 128), (64, 96), (128, 256), (32, 160), (96, 224), (128, 32)]


@pytest.mark.parametrize("dk,dv", DIMS)
@pytest.mark.parametrize("n_new", [1, 2, 8])
def test_row_by_row(n_new, dk, dv):
    Case(3, n_new, 4, 2, dk, dv).check()


@pytest.mark.parametrize("dk,dv", DIMS)
@pytest.mark.parametrize("n_new", [9, 33, 300])
def test_chunks(n_new, dk, dv):
    Case(2, n_new, 4, 2, dk, dv).check()


@pytest.mark.parametrize("n_new", [10, 31, 32, 63, 64, 65, 127, 128, 129, 255, 256, 257, 1000])
@pytest.mark.parametrize("constant", [False, True])
def test_lengths(n_new, constant):
    Case(1, n_new, 2, 1, 64, 64, constant=constant).check()


@pytest.mark.parametrize("n_new", [1, 4, 20, 100, 700])
@pytest.mark.parametrize("in_place", [True, False])
def test_padding_idle_and_beginning_sequences(n_new, in_place):
    """Sequences that continue, begin with the first row, begin inside, hold one position, hold none (also a negative
    count); what padding rows hold is NaN, and a state that is not used too."""
    lens = [n_new + 7, n_new, max(1, n_new // 2), 1, 0, -3, 2 ** 31 - 1, max(1, n_new - 33)]
    c = Case(len(lens), n_new, 4, 2, 32, 64, lens=lens)
    for s, n in enumerate(lens):
        pad = slice(0, n_new - min(max(n, 0), n_new))
        for a in (c.q, c.k, c.v, c.decay):
            a[s, pad] = np.nan
        if 0 < n <= n_new:
            c.state[s] = np.nan
    kw = {} if in_place else {"state_out": torch.full(c.state.shape, 5.0, device=DEV)}
    out, state = c.check(**kw)
    assert (out[4] == 0).all() and (state[4] == c.state[4]).all() and (state[5] == c.state[5]).all()
    assert (out[3, :n_new - 1] == 0).all()


@pytest.mark.parametrize("n_new", [3, 50, 600])
def test_extreme_decays(n_new):
    """Heads that never forget, forget at once, and clear their state at some rows; positive decays count as 0."""
    c = Case(2, n_new, 6, 3, 64, 64)
    rng = np.random.default_rng(0)
    c.decay[..., 0] = 0.0
    c.decay[..., 1] = -30.0
    c.decay[..., 2] = np.where(rng.random(c.decay.shape[:2]) < 0.2, -np.inf, c.decay[..., 2])
    c.decay[..., 3] = -np.inf
    c.decay[..., 4] = np.where(rng.random(c.decay.shape[:2]) < 0.5, 3.0, c.decay[..., 4])
    c.decay[..., 5] = -3.0e38
    c.check()


@pytest.mark.parametrize("n_new", [2000])
def test_long_memory(n_new):
    """A decay close to 1 over a long prompt: the state's errors do not pile up beyond the bound."""
    Case(1, n_new, 1, 1, 128, 128, rate=(1e-5, 1e-5)).check()


@pytest.mark.parametrize("n_new", [4, 70, 400])
def test_values_of_any_size(n_new):
    c = Case(1, n_new, 2, 2, 64, 64)
    rng = np.random.default_rng(1)
    for a in (c.q, c.k, c.v):
        a *= (2.0 ** rng.integers(-20, 21, a.shape[:2] + (1, 1))).astype(np.float32)
    c.check()
    c.q *= np.float32(1e-25)
    c.k *= np.float32(1e15)
    c.state *= np.float32(1e15)
    c.check()
    c.q[:] = 0
    c.check()
    c.k[:] = 0
    c.state[:] = 0
    c.check()


@pytest.mark.parametrize("n_new,at", [(5, 2), (40, 20), (40, 35), (300, 140)])
@pytest.mark.parametrize("what", ["q", "k", "v", "decay"])
@pytest.mark.parametrize("bad", [np.nan, np.inf])
def test_what_is_not_finite_shows_from_its_row_on_and_nowhere_else(n_new, at, what, bad):
    if what == "decay" and bad == np.inf:
        bad = np.nan
    c = Case(2, n_new, 4, 2, 64, 64)
    clean_out, clean_state, tol, s_tol = c.want()
    a = getattr(c, what)
    a[(0, at, 1) if what == "decay" else (0, at, 1, 5)] = bad
    out, state = c.call()
    heads = {"q": [2, 3], "k": [2, 3], "v": [1], "decay": [1]}[what]
    dims = [5] if what == "v" else list(range(64))
    rows = [at] if what == "q" else list(range(at, n_new))
    hit = np.zeros(out.shape, bool)
    hit[np.ix_([0], rows, heads, dims)] = True
    assert not np.isfinite(out[hit]).any()
    assert (np.abs(out - clean_out) <= tol)[~hit].all()
    s_hit = np.zeros(state.shape, bool)
    if what == "v" and n_new > ref.STEP_ROWS:
        s_hit[0, 1, :, 5] = True
    elif what == "v":
        s_hit[0, 1, :, 5] = True
    elif what != "q":
        s_hit[np.ix_([0], heads)] = True
    if what == "k" and n_new <= ref.STEP_ROWS:
        # row by row the state's row of that dim of k alone is hit
        assert not np.isfinite(state[0, 2:, 5]).any()
    else:
        assert not np.isfinite(state[s_hit]).any()
    assert (np.abs(state - clean_state) <= s_tol)[~s_hit].all()


@pytest.mark.parametrize("bad", [np.nan, np.inf])
@pytest.mark.parametrize("n_new", [3, 40])
def test_a_state_that_is_not_finite_stays_in_its_dim(n_new, bad):
    c = Case(1, n_new, 2, 1, 64, 64)
    clean_out, clean_state, tol, s_tol = c.want()
    c.state[0, 1, 7, 9] = bad
    out, state = c.call()
    assert not np.isfinite(out[0, 0, 1, 9]).any() and not np.isfinite(state[0, 1, 7, 9]).any()
    keep = np.ones(64, bool)
    keep[9] = False
    assert (np.abs(out - clean_out) <= tol)[0, :, 0].all() and (np.abs(out - clean_out) <= tol)[0, :, 1, keep].all()
    assert (np.abs(state - clean_state) <= s_tol)[0, 1][:, keep].all()


@pytest.mark.parametrize("n_new", [3, 77])
@pytest.mark.parametrize("shift", [0, 1, 4])
def test_strided_rows(n_new, shift):
    """q, k, v and the decays as parts of one product's rows, 16-byte aligned or not, out as part of a wider row."""
    c = Case(2, n_new, 4, 2, 32, 64)
    width = 2 * 2 * 32 + 4 * 64 + 4 + shift
    wide = torch.full((2, n_new, width + 3), float("nan"), device=DEV)
    parts, at = [], shift
    for a in (c.q, c.k, c.v, c.decay):
        w = int(np.prod(a.shape[2:]))
        wide[..., at:at + w] = _dev(a.reshape(2, n_new, w))
        parts.append(wide[..., at:at + w].unflatten(-1, a.shape[2:]) if a.ndim == 4 else wide[..., at:at + w])
        at += w
    out = torch.full((2, n_new, 4 * 64 + 9), 3.0, device=DEV)
    state = _dev(c.state)
    q.linear_attend(*parts, state, out=out[..., 5:5 + 256].unflatten(-1, (4, 64)))
    torch.cuda.synchronize()
    got = out[..., 5:261].reshape(2, n_new, 4, 64).cpu().numpy()
    c.check(got=(got, state.cpu().numpy()))
    assert (out[..., :5] == 3).all() and (out[..., 261:] == 3).all()


def test_a_prompt_in_pieces_and_steps():
    """A prompt at once, in chunks, and its last rows one by one give the same within the bounds."""
    n = 200
    c = Case(2, n, 4, 4, 64, 64, lens=[n, n - 20])
    want, w_state, tol, s_tol = c.want()
    state = torch.full(c.state.shape, float("nan"), device=DEV)
    got = []
    args = [_dev(a) for a in (c.q, c.k, c.v, c.decay)]
    at = 0
    for size in (37, 64, 9, 83, 1, 1, 5):
        lens = torch.tensor([at + size, max(at + size - 20, 0)], dtype=torch.int32, device=DEV)
        got.append(q.linear_attend(*(a[:, at:at + size].contiguous() for a in args), state, lens))
        at += size
    assert at == n
    got = torch.cat(got, 1).cpu().numpy()
    assert (np.abs(got - want) <= 2 * tol).all()
    assert (np.abs(state.cpu().numpy() - w_state) <= 2 * s_tol).all()


@pytest.mark.parametrize("n_new", [1, 40, 900])
def test_the_same_call_gives_the_same_result(n_new):
    c = Case(1, n_new, 3, 1, 128, 128)
    first = c.call()
    for _ in range(4):
        again = c.call()
        assert (first[0] == again[0]).all() and (first[1] == again[1]).all()


@pytest.mark.parametrize("n_new", [1, 700])
def test_captured_twice_and_on_streams(n_new):
    c = Case(1, n_new, 3, 3, 64, 64)
    args = [_dev(a) for a in (c.q, c.k, c.v, c.decay)]
    state = _dev(c.state)
    pairs = [(torch.empty_like(args[2]), torch.empty_like(state)) for _ in range(3)]
    q.linear_attend(*args, state, out=pairs[0][0], state_out=pairs[0][1])
    graphs = []
    for o, s in pairs[1:]:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            q.linear_attend(*args, state, out=o, state_out=s)
        graphs.append(g)
    args[2].mul_(0.5)
    q.linear_attend(*args, state, out=pairs[0][0], state_out=pairs[0][1])
    streams = [torch.cuda.Stream() for _ in graphs]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(10):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for o, s in pairs[1:]:
        assert torch.equal(o, pairs[0][0]) and torch.equal(s, pairs[0][1])


def test_many_sequences_and_given_workspace():
    c = Case(70, 1, 8, 4, 64, 64)
    c.check()
    c = Case(40, 12, 8, 4, 32, 32)
    c.check()
    c = Case(1, 1000, 2, 1, 64, 64)
    ws = torch.empty(1 << 24, dtype=torch.uint8, device=DEV)
    c.check(workspace=ws)
    with pytest.raises(q.QmmError) as e:
        c.call(workspace=ws[:256])
    assert e.value.status == 9


def test_refuses_other_tensors():
    c = Case(2, 3, 4, 2, 32, 64)
    x, k, v, d, s = (_dev(a) for a in (c.q, c.k, c.v, c.decay, c.state))
    lens = torch.ones(2, dtype=torch.int32, device=DEV)
    for args, kw in (((x.cpu(), k, v, d, s), {}), ((x, k, v, d, s[:1]), {}), ((x, k[:, :2], v, d, s), {}),
                     ((x, k, v, d[:, :2], s), {}), ((x, k, v, d.double(), s), {}), ((x, k, v, d, s.cpu()), {}),
                     ((x, k, v, d, s, lens.long()), {}), ((x, k, v, d, s, lens[:1]), {}),
                     ((x.transpose(2, 3), k, v, d, s), {}), ((x, k, v, d, s), dict(out=v[:, :2])),
                     ((x, k, v, d, s), dict(state_out=s[..., :32])), ((x, k, v, d, s.transpose(2, 3)), {})):
        with pytest.raises(ValueError):
            q.linear_attend(*args, **kw)
    with pytest.raises(q.QmmError):
        q.linear_attend(x[..., :16].contiguous(), k[..., :16].contiguous(), v, d, s[:, :, :16].contiguous())
