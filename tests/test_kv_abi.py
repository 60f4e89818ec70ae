"""Host-side checks of the paged key-value cache calls, without a GPU: page
sizes, every refusal with its status before anything is launched, and the
tests' own statement of the layout."""
import ctypes

import numpy as np
import pytest

import kv_reference as ref
import quantized_weight_gguf_gb300 as q
from quantized_weight_gguf_gb300 import build_lib

FMT = {name: q.FORMATS[name] for name in ("f16", "bf16", "q8_0", "q4_0", "q4_k")}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build_lib.build()
    q.load()


@pytest.mark.parametrize("fk,fv,page,heads,dim,expect", [
    ("f16", "f16", 16, 1, 64, 16 * 64 * 4),
    ("bf16", "bf16", 32, 8, 128, 32 * 8 * 128 * 4),
    ("q8_0", "q8_0", 64, 2, 128, 64 * 2 * 2 * (128 + 8)),
    ("q4_0", "q4_0", 48, 3, 96, 48 * 3 * 2 * (48 + 6)),
    ("q8_0", "q4_0", 16, 1, 256, 16 * (256 + 16 + 128 + 16)),
    ("f16", "q8_0", 16, 1, 64, 0),
    ("q4_0", "q8_0", 16, 1, 64, 0),
    ("q4_k", "q4_k", 16, 1, 64, 0),
    ("f16", "f16", 24, 1, 64, 0),
    ("f16", "f16", 0, 1, 64, 0),
    ("f16", "f16", 16, 0, 64, 0),
    ("f16", "f16", 16, 1, 48, 0),
    ("f16", "f16", 16, 1, 544, 0),
])
def test_page_bytes(fk, fv, page, heads, dim, expect):
    assert q.qmm_kv_page_bytes(fk, fv, page, heads, dim) == expect
    if expect:
        assert heads * (page // 16) * ref.strip_bytes(fk, fv, dim) == expect


def _cache(**kw):
    base = dict(fmt_k=FMT["q8_0"], fmt_v=FMT["q8_0"], pages=16 * 100, pages_len=0, n_pages=4, page_size=32,
                n_kv_heads=2, head_dim=128, page_table=16 * 200, table_stride=3, max_pages=3, lens=16 * 300,
                n_seqs=2)
    base.update(kw)
    return q.qmm_kv_cache(**base)


def _append(cache=None, **kw):
    base = dict(n_new=1, k=16 * 400, v=16 * 500, k_stride=256, v_stride=256, q=16 * 600, q_out=16 * 700,
                q_stride=1024, q_out_stride=1024, n_heads=8, rope=16 * 800, rope_len=96, n_rot=128,
                rope_style=0, stream=None, flags=0)
    base.update(kw)
    return q.qmm_kv_append_args(cache=cache or _cache(), **base)


def _attend(cache=None, **kw):
    base = dict(n_new=1, n_heads=8, q=16 * 600, out=16 * 700, q_stride=1024, out_stride=1024, scale=0.1, window=0,
                workspace=None, workspace_bytes=0, stream=None, flags=0)
    base.update(kw)
    return q.qmm_attend_args(cache=cache or _cache(), **base)


def _read(cache=None, **kw):
    base = dict(first=0, count=5, k=16 * 400, v=16 * 500, stream=None, flags=0)
    base.update(kw)
    return q.qmm_kv_read_args(cache=cache or _cache(), **base)


CACHE_REFUSALS = [
    (dict(fmt_k=9), 1), (dict(fmt_v=FMT["f16"]), 1), (dict(fmt_k=FMT["q4_k"], fmt_v=FMT["q4_k"]), 1),
    (dict(page_size=40), 2), (dict(page_size=65552), 2), (dict(n_kv_heads=0), 2), (dict(head_dim=100), 2),
    (dict(head_dim=1024), 2), (dict(n_pages=-1), 2), (dict(n_pages=1 << 31), 2), (dict(n_seqs=-1), 2),
    (dict(n_seqs=1 << 31), 2), (dict(max_pages=-1), 2), (dict(table_stride=2), 2), (dict(pages_len=17), 3),
    (dict(pages=None), 5), (dict(page_table=None), 5), (dict(lens=None), 5), (dict(pages=16 * 100 + 8), 6),
    (dict(lens=16 * 300 + 2), 6), (dict(page_table=16 * 200 + 1), 6),
]


@pytest.mark.parametrize("kw,status", CACHE_REFUSALS)
def test_every_call_refuses_a_bad_cache(kw, status):
    lib, c = q.load(), _cache(**kw)
    for call, args in ((lib.qmm_kv_append, _append(c)), (lib.qmm_kv_read, _read(c)), (lib.qmm_attend, _attend(c))):
        assert call(ctypes.byref(args)) == status, q.qmm_last_error()
        assert q.qmm_last_error() != ""


@pytest.mark.parametrize("kw,status", [
    (dict(n_new=0), 2), (dict(n_new=1 << 30), 2), (dict(k=None), 5), (dict(v=None), 5), (dict(q_out=None), 5),
    (dict(k=16 * 400 + 2), 6), (dict(q_out=16 * 700 + 3), 6), (dict(k_stride=255), 2), (dict(q_stride=1023), 2),
    (dict(n_heads=0), 2), (dict(n_rot=4), 2), (dict(n_rot=136), 2), (dict(n_rot=12), 2), (dict(rope_len=-1), 2),
    (dict(rope_style=2), 1), (dict(rope=16 * 800 + 4), 6), (dict(flags=1), 2),
    (dict(q_out=16 * 600, q_out_stride=1028), 2),
])
def test_append_refusals(kw, status):
    with pytest.raises(q.QmmError) as e:
        q.qmm_kv_append(_append(**kw))
    assert e.value.status == status, q.qmm_last_error()


@pytest.mark.parametrize("kw,status", [
    (dict(first=-2), 4), (dict(first=1 << 31), 4), (dict(count=-1), 2), (dict(count=1 << 30), 2),
    (dict(k=16 * 400 + 1), 6), (dict(flags=4), 2),
])
def test_read_refusals(kw, status):
    with pytest.raises(q.QmmError) as e:
        q.qmm_kv_read(_read(**kw))
    assert e.value.status == status, q.qmm_last_error()


@pytest.mark.parametrize("kw,status", [
    (dict(n_new=0), 2), (dict(n_heads=7), 2), (dict(n_heads=0), 2), (dict(q=None), 5), (dict(out=None), 5),
    (dict(q=16 * 600 + 2), 6), (dict(q_stride=1000), 2), (dict(out_stride=8), 2), (dict(scale=float("nan")), 2),
    (dict(scale=float("inf")), 2), (dict(window=-1), 2), (dict(flags=2), 2),
])
def test_attend_refusals(kw, status):
    a = _attend(**kw)
    with pytest.raises(q.QmmError) as e:
        q.qmm_attend(a)
    assert e.value.status == status, q.qmm_last_error()


@pytest.mark.parametrize("dim", [32, 160, 224, 320, 512])
def test_attend_refuses_other_head_dims(dim):
    a = _attend(_cache(head_dim=dim), q_stride=8 * dim, out_stride=8 * dim)
    with pytest.raises(q.QmmError) as e:
        q.qmm_attend(a)
    assert e.value.status == 10
    assert q.qmm_attend_workspace_bytes(a) == 0


def test_null_arguments_and_empty_work_touch_no_device():
    lib = q.load()
    assert lib.qmm_kv_append(None) == lib.qmm_kv_read(None) == lib.qmm_attend(None) == 5
    none = _cache(n_seqs=0, lens=None, page_table=None)
    assert q.qmm_kv_append(_append(none)) == 0
    assert q.qmm_kv_read(_read(none)) == 0
    assert q.qmm_attend(_attend(none)) == 0
    assert q.qmm_kv_read(_read(count=0)) == 0
    assert q.qmm_kv_read(_read(k=None, v=None)) == 0


def test_tensor_helpers_refuse_wrong_shapes():
    import torch
    size = q.qmm_kv_page_bytes("f16", "f16", 16, 2, 64)
    cache = q.KvCache("f16", "f16", torch.zeros((3, size), dtype=torch.uint8), 16, 2, 64)
    table, lens = torch.zeros((2, 4), dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    x = torch.zeros((2, 1, 2, 64))
    with pytest.raises(ValueError):
        q.KvCache("f16", "f16", torch.zeros((3, size + 1), dtype=torch.uint8), 16, 2, 64)
    with pytest.raises(q.QmmError):
        q.KvCache("f16", "q8_0", torch.zeros((3, size), dtype=torch.uint8), 16, 2, 64)
    for bad in (lambda: q.kv_append(cache, x[:, :, :1], x, table, lens),
                lambda: q.kv_append(cache, x, x.double(), table, lens),
                lambda: q.kv_append(cache, x, x, table.long(), lens),
                lambda: q.kv_append(cache, x, x, table[:1], lens),
                lambda: q.kv_append(cache, x, x, table, lens, rope=torch.zeros(4, 64)),
                lambda: q.kv_append(cache, x.transpose(2, 3), x, table, lens),
                lambda: q.kv_read(cache, table, lens, 2, k=torch.zeros(2, 3, 2, 64)),
                lambda: q.attend(cache, x[..., :32], table, lens),
                lambda: q.attend(cache, x, table, lens, out=torch.zeros(2, 2, 2, 64)),
                lambda: q.attend(cache, x, table.t(), lens)):
        with pytest.raises(ValueError):
            bad()


def test_rope_table_is_the_angles_cosine_and_sine():
    t = q.rope_table(50, 16, base=500.0, scale=0.5, device="cpu").double().numpy()
    a = np.arange(8)
    for p in (0, 1, 49):
        ang = p * 0.5 * 500.0 ** (-2 * a / 16)
        assert np.allclose(t[p, :, 0], np.cos(ang), atol=2.0 ** -24)
        assert np.allclose(t[p, :, 1], np.sin(ang), atol=2.0 ** -24)


# ------------------------------------------------- the reference's own pins ----

def test_reference_packing_by_hand():
    x = np.zeros(32, np.float32)
    x[:4] = [127.0, -127.0, 63.4, -1.6]
    codes, d = ref.pack(x, "q8_0")
    assert d[0] == 1.0 and list(codes.view(np.int8)[0, :4]) == [127, -127, 63, -2]
    x[:4] = [8.0, -7.0, 3.4, -8.0]        # +8 and -8 tie: the maximum is taken, so d = -1
    codes, d = ref.pack(x, "q4_0")
    assert d[0] == -1.0
    assert [codes[0, 0] & 15, codes[0, 0] >> 4, codes[0, 1] & 15, codes[0, 1] >> 4] == [0, 15, 5, 15]
    assert list(ref.unpack(codes, d, "q4_0")[:4]) == [8.0, -7.0, 3.0, -7.0]
    for fmt, bits in (("f16", 0x3C00), ("bf16", 0x3F80)):
        codes, _ = ref.pack(np.ones(32, np.float32), fmt)
        assert codes.view(np.uint16)[0] == bits


@pytest.mark.parametrize("fmt", range(len(ref.FORMATS)))
def test_reference_pages_hold_what_is_put(fmt):
    fk, fv = ref.FORMATS[fmt]
    rng = np.random.default_rng(1)
    host = ref.Pages(fk, fv, 3, 32, 2, 64)
    x = rng.standard_normal((2, 2, 64)).astype(np.float32)
    for which in (0, 1):
        for h in (0, 1):
            host.put(which, 2, h, 19, x[which, h])
            codes, d = ref.pack(x[which, h], (fk, fv)[which])
            got = host.values(which, [1, 2], 52)[51, h]
            assert np.array_equal(got, ref.unpack(codes, d, (fk, fv)[which]))
            assert np.abs(got - x[which, h]).max() < 0.5
    # only that position's bytes were touched
    assert (host.raw != 0).sum() <= 2 * 2 * ref.strip_bytes(fk, fv, 64) // 32


def test_reference_attention_of_one_position_is_its_value():
    rng = np.random.default_rng(2)
    k, v = rng.standard_normal((2, 5, 1, 64))
    out, tol = ref.attention(rng.standard_normal((2, 64)), k, v, 3, 3, 0.125)
    assert np.array_equal(out, np.stack((v[3, 0], v[3, 0]))) and (tol > 0).all()
    out, _ = ref.attention(rng.standard_normal((2, 64)), k, v, 1, 0, 0.125)
    assert not out.any()
