"""Attention over the paged key-value cache, on the GPU, against the formula in
64 bits on what the cache's bytes stand for (kv_reference, where the tolerance
is derived)."""
import numpy as np
import pytest

import kv_reference as ref

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


def _fill(host, table, lens, rng, k_gain=1.0, k_shift=0.0, v_gain=1.0):
    for s, n in enumerate(lens):
        for p in range(n):
            for h in range(host.n_kv):
                page, o = table[s, p // host.page], p % host.page
                host.put(0, page, h, o, rng.standard_normal(host.dim) * k_gain + k_shift)
                host.put(1, page, h, o, rng.standard_normal(host.dim) * v_gain)


def _check(host, cache, table, lens, xq, window=0, scale=None, **kw):
    n_seqs, n_new, n_heads, dim = xq.shape
    dt, dl = _dev(table), _dev(np.array(lens, np.int32))
    out = q.attend(cache, _dev(xq), dt, dl, window=window, scale=scale, **kw)
    torch.cuda.synchronize()
    assert q.qmm_device_status() == 0
    out = out.cpu().numpy()
    sc = np.float32(dim ** -0.5 if scale is None else scale).astype(np.float64)
    for s, n in enumerate(lens):
        k, v = host.values(0, table[s], n), host.values(1, table[s], n)
        for i in range(n_new):
            last = n - n_new + i
            first = max(0, last + 1 - window) if window else 0
            want, tol = ref.attention(xq[s, i], k, v, first, last, sc)
            bad = ~(np.abs(out[s, i] - want) <= tol)
            assert not bad.any(), (s, i, np.abs(out[s, i] - want)[bad][:4], tol[bad][:4])
    return out


def _garbage(rng):
    """Bytes that are NaN or huge in every format."""
    def fill(shape):
        g = rng.integers(0, 256, shape, dtype=np.uint8)
        g[:, ::3] = 0xFF
        return g
    return fill


def _setup(rng, fk, fv, lens, page, n_kv, dim, **kw):
    table, n_pages = ref.make_table(rng, lens, page)
    host = ref.Pages(fk, fv, n_pages, page, n_kv, dim, _garbage(rng))
    _fill(host, table, lens, rng, **kw)
    return table, host, q.KvCache(fk, fv, _dev(host.raw), page, n_kv, dim)


# one position, around the strip's and the page's ends, several pages, an empty sequence
LENS = [1, 15, 16, 17, 0, 33, 100]


@pytest.mark.parametrize("fmt", range(len(ref.FORMATS)))
@pytest.mark.parametrize("dim", [64, 96, 128, 192, 256])
def test_formats_and_head_dims(fmt, dim):
    fk, fv = ref.FORMATS[fmt]
    rng = np.random.default_rng(100 * fmt + dim)
    table, host, cache = _setup(rng, fk, fv, LENS, 32, 2, dim)
    xq = (2 * rng.standard_normal((len(LENS), 1, 8, dim))).astype(np.float32)
    _check(host, cache, table, LENS, xq)


@pytest.mark.parametrize("fmt", range(len(ref.FORMATS)))
@pytest.mark.parametrize("dim", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("n_new,window", [(1, 0), (3, 0), (1, 650)])
def test_items_split_over_blocks(fmt, dim, n_new, window):
    """Tables much wider than the lengths, as a server holds them: long and short items, an empty one."""
    fk, fv = ref.FORMATS[fmt]
    rng = np.random.default_rng(1000 * fmt + dim + n_new)
    lens, page = [700, 0, 17, 260], 32
    table, n_pages = ref.make_table(rng, lens, page, width=4096)
    host = ref.Pages(fk, fv, n_pages, page, 2, dim, _garbage(rng))
    _fill(host, table, lens, rng)
    cache = q.KvCache(fk, fv, _dev(host.raw), page, 2, dim)
    xq = rng.standard_normal((len(lens), n_new, 8, dim)).astype(np.float32)
    _check(host, cache, table, lens, xq, window=window)


@pytest.mark.parametrize("n_heads,n_kv", [(1, 1), (3, 3), (6, 2), (5, 1), (8, 1), (9, 1), (16, 1), (34, 2)])
@pytest.mark.parametrize("fmt", [0, 2])
def test_head_layouts(n_heads, n_kv, fmt):
    fk, fv = ref.FORMATS[fmt]
    rng = np.random.default_rng(n_heads)
    lens = [40, 7, 129]
    table, host, cache = _setup(rng, fk, fv, lens, 16, n_kv, 64)
    xq = rng.standard_normal((3, 1, n_heads, 64)).astype(np.float32)
    _check(host, cache, table, lens, xq)


@pytest.mark.parametrize("page", [16, 48, 64, 256])
@pytest.mark.parametrize("fmt", [1, 4])
def test_page_sizes_and_a_long_sequence(page, fmt):
    fk, fv = ref.FORMATS[fmt]
    rng = np.random.default_rng(page)
    lens = [1500, 3, 255]
    table, host, cache = _setup(rng, fk, fv, lens, page, 1, 128)
    xq = rng.standard_normal((3, 1, 4, 128)).astype(np.float32)
    _check(host, cache, table, lens, xq)


@pytest.mark.parametrize("n_new,window", [(1, 1), (1, 16), (1, 21), (4, 0), (7, 5), (20, 0), (3, 1000)])
@pytest.mark.parametrize("fmt", [0, 3])
def test_several_new_rows_and_windows(n_new, window, fmt):
    """Each row sees its own positions; rows before a sequence's start give zeros."""
    fk, fv = ref.FORMATS[fmt]
    rng = np.random.default_rng(10 * n_new + window)
    lens = [n_new, 2, 50, 0, 97]
    table, host, cache = _setup(rng, fk, fv, lens, 16, 2, 64)
    xq = rng.standard_normal((5, n_new, 6, 64)).astype(np.float32)
    out = _check(host, cache, table, lens, xq, window=window)
    assert not out[3].any()
    if n_new > 2:
        assert not out[1, :n_new - 2].any()


@pytest.mark.parametrize("fmt", range(len(ref.FORMATS)))
def test_nan_outside_a_rows_range_does_not_reach_it(fmt):
    """Later drafted positions and positions behind the window hold NaN; rows that do not see them
    are as if they held anything else. The row that sees one is NaN."""
    fk, fv = ref.FORMATS[fmt]
    rng = np.random.default_rng(fmt)
    lens, window, n_new = [45], 20, 3
    table, host, cache = _setup(rng, fk, fv, lens, 16, 1, 64)
    for p in (44, 10, 22, 23):    # rows 42, 43, 44 see from 23, 24, 25 on
        for which in (0, 1):
            x = np.full((1, 1, 1, 64), np.nan, np.float32)
            one = q.KvCache(fk, fv, cache.pages, 16, 1, 64)
            t, n = _dev(table), _dev(np.array([p + 1], np.int32))
            q.kv_append(one, _dev(x), _dev(x), t, n)
    xq = rng.standard_normal((1, n_new, 4, 64)).astype(np.float32)
    out = q.attend(cache, _dev(xq), _dev(table), _dev(np.array(lens, np.int32)), window=window)
    out = out.cpu().numpy()
    assert np.isnan(out[0, 0]).all() and np.isnan(out[0, 2]).all()
    k, v = host.values(0, table[0], 45), host.values(1, table[0], 45)
    want, tol = ref.attention(xq[0, 1], k, v, 24, 43, np.float64(np.float32(0.125)))
    assert (np.abs(out[0, 1] - want) <= tol).all()


@pytest.mark.parametrize("fmt", range(len(ref.FORMATS)))
@pytest.mark.parametrize("n_heads,n_kv,n_new,window", [(1, 1, 8, 0), (2, 2, 11, 19), (12, 1, 2, 0), (5, 1, 7, 3),
                                                       (6, 3, 33, 16)])
def test_new_rows_that_share_an_item(fmt, n_heads, n_kv, n_new, window):
    """Rows of several new positions are worked on together: each keeps its own range, and a NaN in
    a position that only the later ones see stays with those."""
    fk, fv = ref.FORMATS[fmt]
    rng = np.random.default_rng(n_new + n_heads)
    lens = [n_new + 40, n_new - 1, n_new + 3, 0]
    table, host, cache = _setup(rng, fk, fv, lens, 16, n_kv, 96)
    xq = rng.standard_normal((4, n_new, n_heads, 96)).astype(np.float32)
    _check(host, cache, table, lens, xq, window=window)
    bad = lens[0] - n_new // 2
    x = torch.full((1, 1, n_kv, 96), np.nan, device=DEV)
    q.kv_append(cache, x, x, _dev(table[:1]), _dev(np.array([bad + 1], np.int32)))
    out = q.attend(cache, _dev(xq), _dev(table), _dev(np.array(lens, np.int32)), window=window).cpu().numpy()
    k, v = host.values(0, table[0], lens[0]), host.values(1, table[0], lens[0])
    for i in range(n_new):
        last = lens[0] - n_new + i
        first = max(0, last + 1 - window) if window else 0
        if first <= bad <= last:
            assert np.isnan(out[0, i]).all()
        else:
            want, tol = ref.attention(xq[0, i], k, v, first, last, np.float64(np.float32(96 ** -0.5)))
            assert (np.abs(out[0, i] - want) <= tol).all()


@pytest.mark.parametrize("fmt", range(len(ref.FORMATS)))
@pytest.mark.parametrize("n", [1, 17, 33, 65, 129, 600])
def test_a_nan_that_is_seen_shows(fmt, n):
    """A NaN at the last position alone, wherever that falls among the strips; a query row with a
    NaN beside one without."""
    fk, fv = ref.FORMATS[fmt]
    rng = np.random.default_rng(n)
    table, host, cache = _setup(rng, fk, fv, [n], 16, 1, 64)
    xq = rng.standard_normal((1, 1, 3, 64)).astype(np.float32)
    xq[0, 0, 1, 5] = np.nan
    dt, dl = _dev(table), _dev(np.array([n], np.int32))
    out = q.attend(cache, _dev(xq), dt, dl).cpu().numpy()[0, 0]
    assert np.isnan(out[1]).all()
    want, tol = ref.attention(xq[0, 0, ::2], host.values(0, table[0], n), host.values(1, table[0], n), 0,
                              n - 1, np.float64(np.float32(0.125)))
    assert (np.abs(out[::2] - want) <= tol).all()
    x = torch.full((1, 1, 1, 64), np.nan, device=DEV)
    q.kv_append(cache, x, torch.zeros_like(x), dt, dl)
    assert np.isnan(q.attend(cache, _dev(xq), dt, dl).cpu().numpy()).all()


@pytest.mark.parametrize("fmt", range(len(ref.FORMATS)))
@pytest.mark.parametrize("kind", ["peaked", "shifted", "large_q", "tiny_v", "large_v", "negative_scale"])
def test_ranges_of_scores_and_values(fmt, kind):
    """Softmaxes with one heavy weight, a common offset of all scores (the maximum far from 0),
    large and tiny queries, values far from 1, a negative scale."""
    fk, fv = ref.FORMATS[fmt]
    rng = np.random.default_rng(7 + fmt)
    kw = {"peaked": dict(k_gain=4.0), "shifted": dict(k_shift=3.0), "tiny_v": dict(v_gain=2e-3),
          "large_v": dict(v_gain=900.0)}.get(kind, {})
    lens = [200, 31]
    table, host, cache = _setup(rng, fk, fv, lens, 32, 1, 128, **kw)
    xq = rng.standard_normal((2, 1, 8, 128)).astype(np.float32)
    xq[:, :, ::2] *= 1e-4
    if kind == "shifted":
        xq = np.abs(xq)
    if kind == "large_q":
        xq *= 2e4
    _check(host, cache, table, lens, xq, scale=-0.3 if kind == "negative_scale" else None)


def test_strided_rows_and_given_output():
    """q and out as parts of wider rows, off the 16-byte boundary too."""
    rng = np.random.default_rng(2)
    lens = [30, 77, 5]
    table, host, cache = _setup(rng, "q8_0", "q8_0", lens, 16, 2, 96)
    xq = rng.standard_normal((3, 2, 4, 96)).astype(np.float32)
    for shift, wide in ((0, 6 * 96), (96, 6 * 96), (1, 4 * 96 + 3)):
        buf = torch.full((3, 2, wide), 7.0, device=DEV)
        res = torch.full((3, 2, wide), 7.0, device=DEV)
        at = slice(shift, shift + 4 * 96)
        dq, do = buf[..., at].unflatten(-1, (4, 96)), res[..., at].unflatten(-1, (4, 96))
        dq.copy_(_dev(xq))
        got = q.attend(cache, dq, _dev(table), _dev(np.array(lens, np.int32)), out=do)
        plain = q.attend(cache, _dev(xq), _dev(table), _dev(np.array(lens, np.int32)))
        assert got.data_ptr() == do.data_ptr() and torch.equal(got, plain)
        assert (res[..., :shift] == 7).all() and (res[..., shift + 4 * 96:] == 7).all()
    _check(host, cache, table, lens, xq)


def test_the_same_call_gives_the_same_bits_and_owned_or_given_scratch():
    rng = np.random.default_rng(4)
    lens = [900, 2, 333, 0]
    table, host, cache = _setup(rng, "q8_0", "q4_0", lens, 64, 2, 128)
    xq = _dev(rng.standard_normal((4, 2, 8, 128)).astype(np.float32))
    dt, dl = _dev(table), _dev(np.array(lens, np.int32))
    first = q.attend(cache, xq, dt, dl)
    ws = torch.empty(64 << 20, dtype=torch.uint8, device=DEV)
    for _ in range(10):
        assert torch.equal(q.attend(cache, xq, dt, dl), first)
        assert torch.equal(q.attend(cache, xq, dt, dl, workspace=ws), first)
    c = cache.view(dt, dl)
    out = torch.empty_like(xq)
    a = q.qmm_attend_args(c, 2, 8, xq.data_ptr(), out.data_ptr(), 8 * 128, 8 * 128, 128 ** -0.5, 0, None, 0,
                          torch.cuda.current_stream().cuda_stream, 0)
    q.qmm_attend(a)                       # the library's own scratch
    assert torch.equal(out, first)


def test_out_of_range_pages_count_as_absent_and_are_reported():
    rng = np.random.default_rng(6)
    lens = [64]
    table, host, cache = _setup(rng, "f16", "f16", lens, 16, 1, 64)
    xq = rng.standard_normal((1, 1, 2, 64)).astype(np.float32)
    broken = table.copy()
    broken[0, 1] = 1 << 20
    out = q.attend(cache, _dev(xq), _dev(broken), _dev(np.array(lens, np.int32)))
    with pytest.raises(q.QmmError) as e:
        q.qmm_device_status()
    assert e.value.status == 12 and q.qmm_device_status() == 0
    k, v = host.values(0, table[0], 64), host.values(1, table[0], 64)
    keep = [p for p in range(64) if not 16 <= p < 32]
    want, tol = ref.attention(xq[0, 0], k[keep], v[keep], 0, 47, np.float64(np.float32(0.125)))
    assert (np.abs(out.cpu().numpy()[0, 0] - want) <= tol).all()
    # a length past the table: cut to the table's capacity
    out = q.attend(cache, _dev(xq), _dev(table), _dev(np.array([100], np.int32)))
    with pytest.raises(q.QmmError):
        q.qmm_device_status()
    want, tol = ref.attention(xq[0, 0], k, v, 0, 63, np.float64(np.float32(0.125)))
    assert (np.abs(out.cpu().numpy()[0, 0] - want) <= tol).all()


def test_an_appended_token_is_attended_to_in_stream_order_and_in_a_graph():
    """append -> attend, captured once and replayed on new inputs."""
    rng = np.random.default_rng(8)
    page, n_kv, dim, n_heads = 16, 2, 128, 8
    lens_h = [5, 40]
    table, n_pages = ref.make_table(rng, [48, 48], page)
    cache = q.KvCache("q8_0", "q8_0", torch.zeros((n_pages, q.qmm_kv_page_bytes("q8_0", "q8_0", page, n_kv, dim)),
                                                  dtype=torch.uint8, device=DEV), page, n_kv, dim)
    dt = _dev(table)
    lens = _dev(np.array(lens_h, np.int32))
    old = _dev(rng.standard_normal((2, 48, n_kv, dim)).astype(np.float32))
    q.kv_append(cache, old, old, dt, _dev(np.array([48, 48], np.int32)))
    xq, xk, xv = (torch.zeros((2, 1, h, dim), device=DEV) for h in (n_heads, n_kv, n_kv))
    qo, out = torch.empty_like(xq), torch.empty_like(xq)
    rope = q.rope_table(64, dim, device=DEV)
    ws = torch.empty(64 << 20, dtype=torch.uint8, device=DEV)

    def step():
        q.kv_append(cache, xk, xv, dt, lens, q=xq, q_out=qo, rope=rope)
        q.attend(cache, qo, dt, lens, out=out, workspace=ws)

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for _ in range(3):
        for t in (xq, xk, xv):
            t.copy_(_dev(rng.standard_normal(tuple(t.shape)).astype(np.float32)))
        lens.add_(1)
        g.replay()
        torch.cuda.synchronize()
        host = ref.Pages("q8_0", "q8_0", n_pages, page, n_kv, dim)
        host.raw[:] = cache.pages.cpu().numpy()
        for s, n in enumerate(lens.tolist()):
            want, tol = ref.attention(qo[s, 0].cpu().numpy(), host.values(0, table[s], n),
                                      host.values(1, table[s], n), 0, n - 1, np.float64(np.float32(dim ** -0.5)))
            assert (np.abs(out[s, 0].cpu().numpy() - want) <= tol).all()
    assert q.qmm_device_status() == 0


def test_scratch_of_streams_and_of_a_capture():
    """Without a given workspace: calls of different needs on several streams at once, and captured."""
    rng = np.random.default_rng(9)
    cases = []
    for lens, n_heads, dim in (([3], 4, 64), ([5000, 70, 900], 16, 256), ([333] * 5, 8, 128)):
        table, host, cache = _setup(rng, "q4_0", "q4_0", lens, 32, 2, dim)
        xq = _dev(rng.standard_normal((len(lens), 1, n_heads, dim)).astype(np.float32))
        dt, dl = _dev(table), _dev(np.array(lens, np.int32))
        ws = torch.empty(64 << 20, dtype=torch.uint8, device=DEV)
        cases.append((cache, xq, dt, dl, q.attend(cache, xq, dt, dl, workspace=ws)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for _ in range(5):
        for s in streams:
            with torch.cuda.stream(s):
                got += [(q.attend(*c[:4]), c[4]) for c in cases]
            got += [(q.attend(*c[:4], stream=s), c[4]) for c in cases]
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        got += [(q.attend(*c[:4]), c[4]) for c in cases]
    for _ in range(3):
        g.replay()
        got += [(q.attend(*c[:4]), c[4]) for c in cases]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in got)


@pytest.mark.parametrize("fmt", range(len(ref.FORMATS)))
@pytest.mark.parametrize("n_new", [1, 3])
def test_a_bad_page_among_strips_taken_together(fmt, n_new):
    """A page id out of range inside a run of strips: its positions are absent, the others stay."""
    fk, fv = ref.FORMATS[fmt]
    rng = np.random.default_rng(20 + fmt)
    n, page = 400, 16
    table, host, cache = _setup(rng, fk, fv, [n], page, 1, 64)
    xq = rng.standard_normal((1, n_new, 3, 64)).astype(np.float32)
    broken = table.copy()
    bad = [1, 6, 7, 12, 24]
    broken[0, bad] = [host.raw.shape[0], -5, 1 << 30, -1, host.raw.shape[0] + 7]
    out = q.attend(cache, _dev(xq), _dev(broken), _dev(np.array([n], np.int32))).cpu().numpy()
    with pytest.raises(q.QmmError) as e:
        q.qmm_device_status()
    assert e.value.status == 12 and q.qmm_device_status() == 0
    k, v = host.values(0, table[0], n), host.values(1, table[0], n)
    for i in range(n_new):
        keep = [p for p in range(n - n_new + 1 + i) if p // page not in bad]
        want, tol = ref.attention(xq[0, i], k[keep], v[keep], 0, len(keep) - 1, np.float64(np.float32(0.125)))
        assert (np.abs(out[0, i] - want) <= tol).all()


@pytest.mark.parametrize("fmt", [0, 2])
def test_pages_past_32_bits(fmt):
    """The pages in use lie beyond 4 GiB of the pool."""
    fk, fv = ref.FORMATS[fmt]
    rng = np.random.default_rng(30)
    n, page, n_kv, dim = 90, 16, 2, 128
    per = q.qmm_kv_page_bytes(fk, fv, page, n_kv, dim)
    table, n_pages = ref.make_table(rng, [n], page)
    host = ref.Pages(fk, fv, n_pages, page, n_kv, dim)
    _fill(host, table, [n], rng)
    first = (1 << 32) // per + 1
    pages = torch.empty((first + n_pages, per), dtype=torch.uint8, device=DEV)
    pages[first:] = _dev(host.raw)
    cache = q.KvCache(fk, fv, pages, page, n_kv, dim)
    xq = rng.standard_normal((1, 1, 6, dim)).astype(np.float32)
    out = q.attend(cache, _dev(xq), _dev(table + first), _dev(np.array([n], np.int32))).cpu().numpy()
    want, tol = ref.attention(xq[0, 0], host.values(0, table[0], n), host.values(1, table[0], n), 0, n - 1,
                              np.float64(np.float32(dim ** -0.5)))
    assert (np.abs(out[0, 0] - want) <= tol).all() and q.qmm_device_status() == 0
