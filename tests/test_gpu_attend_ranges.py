"""Attention over the paged key-value cache, on the GPU, at the ends of what its
numbers can hold: small and very unequal V scales, infinities, values near
fp32's limits, lengths beyond the table. Against the formula in 64 bits with
kv_reference's tolerance."""
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


def _appended(rng, fk, fv, k, v, page=32):
    """A cache that holds rows k, v [n, n_kv, dim] of one sequence, its table on the host, and the
    values that its bytes stand for."""
    n, n_kv, dim = k.shape
    table, n_pages = ref.make_table(rng, [n], page)
    cache = q.KvCache.empty(fk, fv, n_pages, page, n_kv, dim, device=DEV)
    q.kv_append(cache, _dev(k[None].astype(np.float32)), _dev(v[None].astype(np.float32)), _dev(table),
                _dev(np.array([n], np.int32)))
    host = ref.Pages(fk, fv, n_pages, page, n_kv, dim)
    host.raw[:] = cache.pages.cpu().numpy()
    return cache, table, host.values(0, table[0], n), host.values(1, table[0], n)


def _attend(cache, table, n, xq, **kw):
    out = q.attend(cache, _dev(xq[None]), _dev(table), _dev(np.array([n], np.int32)), **kw)
    return out.cpu().numpy()[0]


def _check(cache, table, k, v, xq, window=0):
    """xq [n_new, n_heads, dim] at the last positions of k and v."""
    n, dim, n_new = len(k), k.shape[2], len(xq)
    out = _attend(cache, table, n, xq, window=window)
    assert q.qmm_device_status() == 0
    for i in range(n_new):
        last = n - n_new + i
        first = max(0, last + 1 - window) if window else 0
        want, tol = ref.attention(xq[i], k, v, first, last, np.float64(np.float32(dim ** -0.5)))
        bad = ~(np.abs(out[i] - want) <= tol)
        assert not bad.any(), (i, np.abs(out[i] - want)[bad][:4], tol[bad][:4], (np.abs(out[i] - want) / tol).max())
    return out


@pytest.mark.parametrize("fmt", range(len(ref.FORMATS)))
@pytest.mark.parametrize("width", [4, 64])
@pytest.mark.parametrize("over,n_new,window,n_heads", [(2, 4, 2, 1), (5, 8, 3, 1), (1, 3, 0, 4), (30, 40, 20, 2),
                                                       (9, 3, 2, 1), (750, 200, 650, 1)])
def test_rows_beyond_the_table_leave_the_others_theirs(fmt, width, over, n_new, window, n_heads):
    """A length past the table's capacity with several new rows (short tables: whole items, wide
    ones: split): a row sees what of its range lies within the table, zeros where nothing does."""
    fk, fv = ref.FORMATS[fmt]
    rng = np.random.default_rng(over)
    page, dim = 16, 64
    cap = width * page
    k, v = rng.standard_normal((2, cap, 1, dim))
    cache, table, k, v = _appended(rng, fk, fv, k, v, page)
    assert table.shape[1] == width
    xq = rng.standard_normal((n_new, n_heads, dim)).astype(np.float32)
    n = cap + over
    out = _attend(cache, table, n, xq, window=window)
    with pytest.raises(q.QmmError) as e:
        q.qmm_device_status()
    assert e.value.status == 12 and q.qmm_device_status() == 0
    for i in range(n_new):
        last = n - n_new + i
        first = max(0, last + 1 - window) if window else 0
        want, tol = ref.attention(xq[i], k, v, first, min(last, cap - 1), np.float64(np.float32(0.125)))
        assert (np.abs(out[i] - want) <= tol).all(), (i, first, last)


QUANTISED_V = [("q8_0", "q8_0"), ("q4_0", "q4_0"), ("q8_0", "q4_0")]


@pytest.mark.parametrize("fk,fv", QUANTISED_V)
@pytest.mark.parametrize("n_new", [1, 3])
@pytest.mark.parametrize("size", [1.0, 1e-3, 1e-4, 3e-5, 1e-5])
def test_small_values_under_a_peaked_softmax(fk, fv, n_new, size):
    """V from 1 down to where its f16 scales are subnormal, 4000 positions, a few of which weigh
    nearly everything."""
    rng = np.random.default_rng(int(-100 * np.log10(size)) + n_new)
    k, v = rng.standard_normal((2, 4000, 1, 64))
    cache, table, k, v = _appended(rng, fk, fv, 4 * k, size * v)
    _check(cache, table, k, v, rng.standard_normal((n_new, 4, 64)).astype(np.float32))


@pytest.mark.parametrize("fk,fv", QUANTISED_V)
@pytest.mark.parametrize("dim", [64, 96, 128, 192, 256])
def test_blocks_of_very_different_size(fk, fv, dim):
    """The 32-dim blocks of a head differ by up to 2^18, each of them held to its own size; the
    positions' sizes grow and shrink by 2^4 along the sequence."""
    rng = np.random.default_rng(dim)
    n = 700
    k, v = rng.standard_normal((2, n, 2, dim))
    size = 2.0 ** np.linspace(2, -16, dim // 32).repeat(32) * 2.0 ** (2 * np.sin(np.arange(n) / 40.0))[:, None, None]
    cache, table, k, v = _appended(rng, fk, fv, k, size * v)
    xq = rng.standard_normal((2, 6, dim)).astype(np.float32)
    _check(cache, table, k, v, xq)
    _check(cache, table, k, v, xq[:1])
    _check(cache, table, k, v, xq, window=301)


@pytest.mark.parametrize("fk,fv", QUANTISED_V)
@pytest.mark.parametrize("n_new", [1, 5])
def test_scales_up_to_the_largest(fk, fv, n_new):
    """V grows along the sequence from 1e-4 to values whose f16 scales are the largest there are,
    and falls again; rows of several new positions see different ends of it."""
    rng = np.random.default_rng(n_new)
    n = 600
    k, v = rng.standard_normal((2, n, 1, 64))
    up = np.concatenate((np.linspace(-4, 5, n - 40), np.linspace(5, 3, 40)))
    cache, table, k, v = _appended(rng, fk, fv, 0.1 * k, 10.0 ** up[:, None, None] * v)
    xq = rng.standard_normal((n_new, 3, 64)).astype(np.float32)
    _check(cache, table, k, v, xq)
    _check(cache, table, k, v, xq, window=30)


@pytest.mark.parametrize("fk,fv", QUANTISED_V)
def test_a_large_position_that_only_later_rows_see(fk, fv):
    """Rows that do not see the one huge value keep their precision for small ones."""
    rng = np.random.default_rng(3)
    n, n_new = 90, 6
    k, v = rng.standard_normal((2, n, 1, 64))
    v[:n - 3] *= 1e-4
    v[n - 3:] *= 1e5
    cache, table, k, v = _appended(rng, fk, fv, k, v)
    _check(cache, table, k, v, rng.standard_normal((n_new, 1, 64)).astype(np.float32))


@pytest.mark.parametrize("fk,fv", QUANTISED_V)
@pytest.mark.parametrize("n_new", [1, 3])
def test_zero_blocks_and_zero_values(fk, fv, n_new):
    """Blocks of zeros (a scale of 0) beside others, positions of zeros, and V of zeros alone."""
    rng = np.random.default_rng(11)
    n = 300
    k, v = rng.standard_normal((2, n, 1, 96))
    v[:, :, 32:64] = 0
    v[::3] = 0
    v[150:] *= 1e-4
    xq = rng.standard_normal((n_new, 3, 96)).astype(np.float32)
    cache, table, kk, vv = _appended(rng, fk, fv, k, v)
    out = _check(cache, table, kk, vv, xq)
    assert not out[:, :, 32:64].any()
    cache, table, kk, vv = _appended(rng, fk, fv, k, np.zeros_like(v))
    assert not _attend(cache, table, n, xq).any()


@pytest.mark.parametrize("fmt", ["f16", "bf16"])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("n_new", [1, 3])
def test_infinite_k_that_is_seen_makes_the_row_nan(fmt, sign, n_new):
    """Whatever the query's sign and last bits are: exact in 16 bits, rounded up, rounded down. Rows
    that do not see the position are as without it."""
    rng = np.random.default_rng(4)
    n, at = 70, 68
    k, v = rng.standard_normal((2, n, 1, 64))
    k[at, 0, 7] = sign * np.inf
    cache, table, k, v = _appended(rng, fmt, fmt, k, v)
    assert np.isinf(k[at, 0, 7])
    xq = rng.standard_normal((n_new, 8, 64)).astype(np.float32)
    xq[:, :, 7] = np.array([1.0, -1.0, 1.0 + 2.0 ** -13, 1.0 - 2.0 ** -13, -1.0 - 2.0 ** -13, -1.0 + 2.0 ** -13,
                            0.0, 1.0 + 2.0 ** -23], np.float32)
    out = _attend(cache, table, n, xq)
    assert q.qmm_device_status() == 0
    for i in range(n_new):
        last = n - n_new + i
        if last >= at:
            assert np.isnan(out[i]).all(), i
        else:
            want, tol = ref.attention(xq[i], k, v, 0, last, np.float64(np.float32(0.125)))
            assert (np.abs(out[i] - want) <= tol).all()


@pytest.mark.parametrize("fk,fv", [f for f in ref.FORMATS if f[0] != "f16" and f[0] != "bf16"])
@pytest.mark.parametrize("which", [0, 1])
def test_infinite_scales(fk, fv, which):
    """A scale of Inf, which kv_append does not write: in K it makes rows that see the position NaN,
    in V the 32 dims of its block Inf or NaN and no others."""
    rng = np.random.default_rng(5)
    n, at = 50, 20
    k, v = rng.standard_normal((2, n, 1, 64)).astype(np.float32)
    table, n_pages = ref.make_table(rng, [n], 16)
    host = ref.Pages(fk, fv, n_pages, 16, 1, 64)
    for p in range(n):
        host.put(0, table[0, p // 16], 0, p % 16, k[p, 0])
        host.put(1, table[0, p // 16], 0, p % 16, v[p, 0])
    clean = host.values(1, table[0], n)
    kk = host.values(0, table[0], n)
    start = 0 if which == 0 else sum(ref.half_bytes(fk, 64))
    codes = ref.half_bytes((fk, fv)[which], 64)[0]
    strip = host.strips[table[0, at // 16], 0, 0]
    strip[start + codes:start + codes + 64].view(np.uint16).reshape(2, 16)[1, at % 16] = 0x7C00
    cache = q.KvCache(fk, fv, _dev(host.raw), 16, 1, 64)
    xq = rng.standard_normal((1, 8, 64)).astype(np.float32)
    out = _attend(cache, table, n, xq)
    if which == 0:
        assert np.isnan(out).all()
    else:
        assert not np.isfinite(out[0, :, 32:]).any()
        want, tol = ref.attention(xq[0], kk, clean, 0, n - 1, np.float64(np.float32(0.125)))
        assert (np.abs(out[0] - want) <= tol)[:, :32].all()


@pytest.mark.parametrize("fmt", ["f16", "bf16"])
@pytest.mark.parametrize("sign", [1, -1])
def test_infinite_v_stays_in_its_dim(fmt, sign):
    rng = np.random.default_rng(6)
    n = 70
    k, v = rng.standard_normal((2, n, 1, 64))
    clean = v.copy()
    v[33, 0, 9] = sign * np.inf
    cache, table, k, got = _appended(rng, fmt, fmt, k, v)
    clean = np.where(np.isinf(got), 0.0, got)
    xq = rng.standard_normal((1, 8, 64)).astype(np.float32)
    out = _attend(cache, table, n, xq)
    assert not np.isfinite(out[0, :, 9]).any()
    want, tol = ref.attention(xq[0], k, clean, 0, n - 1, np.float64(np.float32(0.125)))
    others = np.arange(64) != 9
    assert (np.abs(out[0] - want) <= tol)[:, others].all()


@pytest.mark.parametrize("n", [1, 40, 3000])
@pytest.mark.parametrize("size", [1e-30, 1e34, 1e37])
def test_bf16_values_near_the_ends_of_fp32(n, size):
    """Averages of values up to 1e37 (under 5.4 of a deviation) and down to 1e-30."""
    rng = np.random.default_rng(n)
    k, v = rng.standard_normal((2, n, 1, 64))
    cache, table, k, v = _appended(rng, "bf16", "bf16", k, size * v)
    assert np.isfinite(v).all()
    _check(cache, table, k, v, rng.standard_normal((1, 4, 64)).astype(np.float32))
