"""Appending to the paged key-value cache and reading it back, on the GPU,
against the plain statements in kv_reference: the packed bytes are those of the
header's fp32 formulas bit for bit, what is read back is what the bytes stand
for exactly, and the held values are as near to the 64-bit rotated rows as the
formats allow."""
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


def _garbage(rng):
    return lambda shape: rng.integers(0, 256, shape, dtype=np.uint8)


def _rows(rng, shape):
    """Rows of unit scale with zeros, one-sided and tiny blocks among them."""
    x = rng.standard_normal(shape).astype(np.float32)
    flat = x.reshape(-1, 32)
    flat[::7] = 0
    flat[1::11] = np.abs(flat[1::11])
    flat[2::13] *= 1e-6
    flat[3::17] *= 300
    return x


CASES = [
    # fmt, n_seqs, n_new, n_heads, n_kv, dim, page, lens, n_rot, style
    (0, 1, 1, 4, 1, 64, 16, [1], 0, "half"),
    (2, 3, 1, 8, 2, 128, 32, [17, 33, 0], 128, "half"),
    (2, 2, 5, 6, 3, 96, 16, [3, 40], 96, "pairs"),
    (3, 2, 7, 2, 2, 64, 48, [48, 100], 32, "half"),
    (1, 2, 3, 5, 1, 256, 64, [64, 65], 256, "half"),
    (4, 3, 33, 4, 2, 192, 32, [33, 90, 12], 64, "pairs"),
    (0, 2, 18, 2, 1, 512, 16, [18, 47], 512, "half"),
    (3, 1, 20, 1, 1, 32, 16, [29], 8, "pairs"),
    (4, 2, 2, 3, 1, 224, 16, [2, 31], 48, "half"),
]


@pytest.mark.parametrize("fmt,n_seqs,n_new,n_heads,n_kv,dim,page,lens,n_rot,style", CASES)
@pytest.mark.parametrize("fused", [True, False])
def test_append_packs_bit_for_bit_and_reads_back(fmt, n_seqs, n_new, n_heads, n_kv, dim, page, lens,
                                                 n_rot, style, fused):
    fk, fv = ref.FORMATS[fmt]
    rng = np.random.default_rng(dim + page + n_new)
    table, n_pages = ref.make_table(rng, lens, page)
    host = ref.Pages(fk, fv, n_pages, page, n_kv, dim, _garbage(rng))
    cache = q.KvCache(fk, fv, _dev(host.raw), page, n_kv, dim)
    x = _rows(rng, (n_seqs, n_new, n_heads + 2 * n_kv, dim))
    xq, xk, xv = x[:, :, :n_heads], x[:, :, n_heads:n_heads + n_kv], x[:, :, n_heads + n_kv:]
    rope = q.rope_table(max(max(lens), 1), n_rot, device="cpu").numpy() if n_rot else None
    if fused:   # views of one product's output rows
        d = _dev(x)
        dq, dk, dv = d[:, :, :n_heads], d[:, :, n_heads:n_heads + n_kv], d[:, :, n_heads + n_kv:]
    else:       # rows of their own that start off a 16-byte boundary
        def off(a):
            flat = torch.empty(a.size + 1, device=DEV)
            flat[1:] = _dev(a).reshape(-1)
            return flat[1:].view(a.shape)
        dq, dk, dv = off(xq), off(xk), off(xv)
    got_q = q.kv_append(cache, dk, dv, _dev(table), _dev(np.array(lens, np.int32)), q=dq,
                        rope=None if rope is None else _dev(rope), rope_style=style)
    torch.cuda.synchronize()
    assert q.qmm_device_status() == 0
    want_q = np.zeros((n_seqs, n_new, n_heads, dim), np.float32)
    for s in range(n_seqs):
        for i in range(n_new):
            pos = lens[s] - n_new + i
            if pos < 0:
                continue
            rk, rq = xk[s, i], xq[s, i]
            if n_rot:
                rk = ref.rotate(rk, pos, rope, n_rot, style, np.float32)
                rq = ref.rotate(rq, pos, rope, n_rot, style, np.float32)
            want_q[s, i] = rq
            for h in range(n_kv):
                host.put(0, table[s, pos // page], h, pos % page, rk[h])
                host.put(1, table[s, pos // page], h, pos % page, xv[s, i, h])
    assert np.array_equal(got_q.cpu().numpy(), want_q)
    # every byte: the new rows as the formulas say, everything else untouched
    assert np.array_equal(cache.pages.cpu().numpy(), host.raw)
    # read back the same rows: exactly what the bytes stand for, zeros for padding
    k, v = q.kv_read(cache, _dev(table), _dev(np.array(lens, np.int32)), n_new)
    for which, got in ((0, k), (1, v)):
        want = np.zeros((n_seqs, n_new, n_kv, dim))
        for s in range(n_seqs):
            n = min(lens[s], n_new)
            if n:
                want[s, n_new - n:] = host.values(which, table[s], lens[s])[lens[s] - n:]
        assert np.array_equal(got.cpu().numpy().astype(np.float64), want)


@pytest.mark.parametrize("fmt", range(len(ref.FORMATS)))
def test_held_values_are_near_the_64_bit_rows(fmt):
    """Half a step of the format from the row rotated in 64 bits. The step: the f16 scale d (for
    Q4_0 one more on the side that the codes do not reach), with d itself rounded to f16 (2^-11 of
    the block's magnitude); fp32 rotation errs by 2^-23 of it."""
    fk, fv = ref.FORMATS[fmt]
    rng = np.random.default_rng(5)
    n, n_kv, dim, page = 40, 2, 128, 16
    table, n_pages = ref.make_table(rng, [n], page)
    cache = q.KvCache.empty(fk, fv, n_pages, page, n_kv, dim, device=DEV)
    x = rng.standard_normal((2, 1, n, n_kv, dim)).astype(np.float32)
    rope = q.rope_table(n, dim, device="cpu")
    lens = _dev(np.array([n], np.int32))
    q.kv_append(cache, _dev(x[0]), _dev(x[1]), _dev(table), lens, rope=rope.to(DEV))
    got = q.kv_read(cache, _dev(table), lens, n, first=0)
    for which, f in ((0, fk), (1, fv)):
        want = x[which][0].astype(np.float64)
        if which == 0:
            want = np.stack([ref.rotate(want[p], p, rope.numpy(), dim, "half", np.float64)
                             for p in range(n)])
        err = np.abs(got[which][0].cpu().numpy() - want)
        top = np.abs(want).reshape(n, n_kv, -1, 32).max(-1).repeat(32, -1).reshape(want.shape)
        step = {"f16": np.abs(want) * 2.0 ** -11, "bf16": np.abs(want) * 2.0 ** -8,
                "q8_0": top * (0.5 / 127 + 2.0 ** -11), "q4_0": top * (1.0 / 8 + 2.0 ** -11)}[f]
        assert (err <= step + 2.0 ** -22 * top).all(), f


@pytest.mark.parametrize("fmt", range(len(ref.FORMATS)))
def test_read_of_random_bytes(fmt):
    """Any codes and scales (NaN and Inf among them) read back as the header says; positions
    outside the sequence are zeros; `first` and the last-rows form agree."""
    fk, fv = ref.FORMATS[fmt]
    rng = np.random.default_rng(9 + fmt)
    lens, page, n_kv, dim = [37, 0, 16], 16, 3, 96
    table, n_pages = ref.make_table(rng, lens, page)
    host = ref.Pages(fk, fv, n_pages, page, n_kv, dim, _garbage(rng))
    cache = q.KvCache(fk, fv, _dev(host.raw), page, n_kv, dim)
    dl = _dev(np.array(lens, np.int32))
    for first, count in ((0, 40), (7, 30), (None, 21), (36, 2), (50, 3)):
        got = q.kv_read(cache, _dev(table), dl, count, first=first)
        for which in (0, 1):
            want = np.zeros((3, count, n_kv, dim))
            for s, n in enumerate(lens):
                vals = host.values(which, table[s], n)
                for i in range(count):
                    p = (n - count if first is None else first) + i
                    if 0 <= p < n:
                        want[s, i] = vals[p]
            with np.errstate(over="ignore", invalid="ignore"):
                assert np.array_equal(got[which].cpu().numpy().astype(np.float64), want, equal_nan=True)
    assert q.qmm_device_status() == 0


@pytest.mark.parametrize("fmt", [("q8_0", "q8_0"), ("q4_0", "q4_0")])
def test_blocks_with_inf_or_nan_read_back_as_nan_and_large_ones_saturate(fmt):
    page, dim = 16, 64
    cache = q.KvCache.empty(*fmt, 1, page, 1, dim, device=DEV)
    x = np.ones((1, 4, 1, dim), np.float32)
    x[0, 0, 0, 3] = np.nan
    x[0, 1, 0, 40] = -np.inf
    x[0, 2, 0, :32] = 3e38
    table, lens = _dev(np.zeros((1, 1), np.int32)), _dev(np.array([4], np.int32))
    q.kv_append(cache, _dev(x), _dev(x), table, lens)
    for got in q.kv_read(cache, table, lens, 4):
        g = got.cpu().numpy()[0, :, 0]
        assert np.isnan(g[0, :32]).all() and np.abs(g[0, 32:] - 1).max() < 1e-3
        assert np.isnan(g[1, 32:]).all() and np.abs(g[1, :32] - 1).max() < 1e-3
        top = 65504.0 * (127 if fmt[0] == "q8_0" else 8)
        assert (g[2, :32] == top).all() or (np.abs(g[2, :32]) == top).all()
        assert np.abs(g[3] - 1).max() < 1e-3


def test_q_in_place_and_strided_tables():
    rng = np.random.default_rng(3)
    lens, page, n_kv, dim, n_heads, n_new = [20, 50], 16, 2, 128, 4, 3
    table, n_pages = ref.make_table(rng, lens, page)
    wide = torch.full((2, table.shape[1] + 5), -7, dtype=torch.int32, device=DEV)
    wide[:, 2:2 + table.shape[1]] = _dev(table)
    cache = q.KvCache.empty("f16", "f16", n_pages, page, n_kv, dim, device=DEV)
    x = [_dev(rng.standard_normal((2, n_new, h, dim)).astype(np.float32)) for h in (n_heads, n_kv, n_kv)]
    rope = q.rope_table(64, dim, device=DEV)
    dl = _dev(np.array(lens, np.int32))
    out = q.kv_append(cache, x[1], x[2], _dev(table), dl, q=x[0], rope=rope)
    keep = cache.pages.clone()
    view = wide[:, 2:2 + table.shape[1]]
    same = q.kv_append(cache, x[1], x[2], view, dl, q=x[0], q_out=x[0], rope=rope)
    torch.cuda.synchronize()
    assert same.data_ptr() == x[0].data_ptr() and torch.equal(same, out)
    assert torch.equal(keep, cache.pages)
    a, b = q.kv_read(cache, view, dl, 50, first=0), q.kv_read(cache, _dev(table), dl, 50, first=0)
    # bytes compared, since uninitialised positions may hold NaN
    assert all(torch.equal(i.view(torch.int32), j.view(torch.int32)) for i, j in zip(a, b))


def test_out_of_range_tables_lengths_and_positions_are_reported():
    page, dim = 16, 64
    x = torch.ones((1, 1, 1, dim), device=DEV)
    for table, n, rope_len in ([[5]], 1, 8), ([[-1]], 1, 8), ([[0]], 17, 32), ([[0]], 9, 8):
        cache = q.KvCache("f16", "f16", torch.zeros((2, 2 * 16 * 2 * dim), dtype=torch.uint8, device=DEV),
                          page, 1, dim)
        t, lens = _dev(np.array(table, np.int32)), _dev(np.array([n], np.int32))
        q.kv_append(cache, x, x, t, lens, rope=q.rope_table(rope_len, dim, device=DEV))
        with pytest.raises(q.QmmError) as e:
            q.qmm_device_status()
        assert e.value.status == 12
        assert q.qmm_device_status() == 0
        assert not cache.pages.any()          # nothing was written
    k, _ = q.kv_read(cache, _dev(np.array([[9]], np.int32)), _dev(np.array([3], np.int32)), 3)
    assert not k.any()
    with pytest.raises(q.QmmError):
        q.qmm_device_status()


def test_offsets_past_32_bits():
    """A pool of more than 4 GiB: the last page's rows land at its end and nowhere else."""
    page, n_kv, dim = 256, 8, 128
    per = q.qmm_kv_page_bytes("f16", "f16", page, n_kv, dim)
    n_pages = (1 << 32) // per + 3
    pages = torch.zeros((n_pages, per), dtype=torch.uint8, device=DEV)
    cache = q.KvCache("f16", "f16", pages, page, n_kv, dim)
    x = torch.ones((1, 1, n_kv, dim), device=DEV)
    table, lens = _dev(np.array([[n_pages - 1]], np.int32)), _dev(np.array([page], np.int32))
    q.kv_append(cache, x, x, table, lens)
    k, v = q.kv_read(cache, table, lens, 1)
    assert (k == 1).all() and (v == 1).all()
    assert int(pages[:-1].max()) == 0 and q.qmm_device_status() == 0


def test_append_then_read_in_a_stream_of_their_own():
    """Chained calls on a side stream see one another's writes."""
    rng = np.random.default_rng(1)
    page, n_kv, dim, n = 32, 2, 128, 64
    cache = q.KvCache.empty("q8_0", "q8_0", 3, page, n_kv, dim, device=DEV)
    table, lens = _dev(np.array([[2, 0]], np.int32)), _dev(np.array([n], np.int32))
    x = _dev(rng.standard_normal((1, n, n_kv, dim)).astype(np.float32))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for i in range(5):
        with torch.cuda.stream(side):
            q.kv_append(cache, x * (i + 1), x, table, lens)
            k, _ = q.kv_read(cache, table, lens, n)
    side.synchronize()
    top = (x * 5).abs().view(1, n, n_kv, -1, 32).amax(-1, keepdim=True)
    err = (k - x * 5).abs().view(1, n, n_kv, -1, 32)
    assert (err <= top * (0.5 / 127 + 2.0 ** -11)).all()
