"""Workloads of the paged key-value cache operators: appending (rotary embedding and quantising write),
reading back, and attention of new tokens over the cache.

``run`` computes a workload in its plain form (elementary torch operations in fp32) or, where ``own`` is
true, through the library's calls. ``exact`` states the operators' definitions in fp64.

A cache is a uint8 tensor of pages. A page holds page_size positions of every kv head; inside it, a strip
holds 16 positions of one head, and K and V of a strip lie one after the other:

    [page][kv head][strip]{K codes [plane][16][row bytes], K scales [dim / 32][16] f16, V codes, V scales}

f16 and bf16 have planes of 16 dims (rows of 32 bytes) and no scales; q8_0 has planes of 32 dims (32 bytes)
and q4_0 planes of 32 dims (16 bytes, byte i holding dims 2i in its low and 2i + 1 in its high nibble, plus 8).
"""
import math

import numpy as np
import torch

own = False

DEVICE = "cuda:0"
STRIP = 16                                    # positions per strip
ROW_BYTES = {"f16": 32, "bf16": 32, "q8_0": 32, "q4_0": 16}
PLANE_DIMS = {"f16": 16, "bf16": 16, "q8_0": 32, "q4_0": 32}
QUANTISED = ("q8_0", "q4_0")


# ------------------------------------------------------------------ cases ----

def _attend(name, fmt_k, fmt_v, n_seqs, n_new, n_heads, n_kv, dim, page, max_len, ragged, empty=0, window=0):
    return {"name": name, "kind": "attend", "fmt_k": fmt_k, "fmt_v": fmt_v, "n_seqs": n_seqs, "n_new": n_new,
            "n_heads": n_heads, "n_kv": n_kv, "dim": dim, "page": page, "max_len": max_len, "ragged": ragged,
            "empty": empty, "window": window}


def _append(name, fmt_k, fmt_v, n_seqs, n_new, n_heads, n_kv, dim, page, max_len, ragged, n_rot, style):
    return {"name": name, "kind": "append", "fmt_k": fmt_k, "fmt_v": fmt_v, "n_seqs": n_seqs, "n_new": n_new,
            "n_heads": n_heads, "n_kv": n_kv, "dim": dim, "page": page, "max_len": max_len, "ragged": ragged,
            "empty": 0, "n_rot": n_rot, "style": style}


def _read(name, fmt_k, fmt_v, n_seqs, n_kv, dim, page, max_len, ragged):
    return {"name": name, "kind": "read", "fmt_k": fmt_k, "fmt_v": fmt_v, "n_seqs": n_seqs, "n_kv": n_kv,
            "dim": dim, "page": page, "max_len": max_len, "ragged": ragged, "empty": 0}


def listed():
    return [
        # one user, the first words of an answer: a call's latency
        _attend("one_short", "q8_0", "q8_0", 1, 1, 8, 1, 256, 16, 45, 0.0),
        # one user, a long document in the cache: a few heads' work over the whole GPU
        _attend("one_long", "q8_0", "q8_0", 1, 1, 32, 8, 128, 64, 131071, 0.0),
        # a serving batch in 16 bits, every length different
        _attend("batch_f16", "f16", "f16", 64, 1, 32, 8, 128, 32, 8190, 0.9),
        # the same kind of batch in 8 bits, a few slots idle (no position at all)
        _attend("batch_q8", "q8_0", "q8_0", 48, 1, 32, 8, 128, 64, 6001, 0.9, empty=3),
        # one kv head per query head, 4-bit cache, small pages
        _attend("mha_q4", "q4_0", "q4_0", 16, 1, 16, 16, 64, 16, 9000, 0.5),
        # sliding-window layers with wide heads
        _attend("window_bf16", "bf16", "bf16", 96, 1, 8, 1, 256, 128, 16000, 0.8, window=1024),
        # checking a few drafted tokens at once: K in 8 bits, V in 4
        _attend("drafts_q8q4", "q8_0", "q4_0", 8, 5, 24, 4, 96, 32, 5003, 0.7),
        # one decoding step of a batch: the new token's q and k rotated, k and v written
        _append("append_step", "q8_0", "q8_0", 64, 1, 32, 8, 128, 64, 4097, 0.9, 128, "half"),
        # a prompt's chunk
        _append("append_chunk", "f16", "f16", 2, 4000, 32, 8, 128, 32, 6000, 0.2, 64, "pairs"),
        # the same in 4 bits, with wide heads
        _append("append_chunk_q4", "q4_0", "q4_0", 3, 1777, 8, 2, 256, 16, 2048, 0.1, 256, "half"),
        # a short shared prefix read back
        _read("read_short", "q8_0", "q8_0", 1, 8, 128, 64, 200, 0.0),
        # a batch's caches read back, as when they are moved to another format
        _read("read_batch", "q8_0", "q4_0", 16, 8, 128, 32, 8111, 0.8),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(("attend", "attend", "attend", "append", "read"))
    fmt_k, fmt_v = rng.choice((("f16", "f16"), ("bf16", "bf16"), ("q8_0", "q8_0"), ("q4_0", "q4_0"), ("q8_0", "q4_0")))
    dim = rng.choice((64, 96, 128, 192, 256))
    page = rng.choice((16, 32, 48, 64, 128, 256))
    n_kv = rng.choice((1, 2, 4, 5, 8, 16))
    n_seqs = _log(rng, 1, 96)
    n_new = 1 if rng.random() < 0.7 else _log(rng, 2, 8)
    most = 64 * 8190 * 8 * 128 // 2             # elements of K in the largest listed cases, about
    per = n_seqs * n_kv * dim * (n_new if kind == "attend" else 1)
    ragged = round(rng.uniform(0.0, 0.98), 3)
    if kind == "attend":
        group = rng.choice((1, 2, 3, 4, 6, 8, 12, 16))
        max_len = _log(rng, 1, max(2, min(131071, most // (per * max(1, group // 8)))))
        window = _log(rng, 1, 2 * max_len) if rng.random() < 0.3 else 0
        got = _attend("", fmt_k, fmt_v, n_seqs, n_new, n_kv * group, n_kv, dim, page, max_len, ragged,
                      empty=rng.choice((0, 0, 1)) if n_seqs > 1 else 0, window=window)
    elif kind == "append":
        group = rng.choice((1, 2, 4, 7, 8))
        n_new = _log(rng, 1, max(1, min(8192, (8000 * 48 * 128) // (n_seqs * n_kv * (group + 2) * dim))))
        max_len = n_new + _log(rng, 1, 4000)
        ragged = math.floor(1000 * rng.uniform(0.0, 1.0 - n_new / max_len)) / 1000
        got = _append("", fmt_k, fmt_v, n_seqs, n_new, n_kv * group, n_kv, dim, page, max_len, ragged,
                      rng.choice((32, dim // 2, dim)), rng.choice(("half", "pairs")))
    else:
        max_len = _log(rng, 1, max(2, min(65536, 16 * 8111 * 8 * 128 // (n_seqs * n_kv * dim))))
        got = _read("", fmt_k, fmt_v, n_seqs, n_kv, dim, page, max_len, ragged)
    del got["name"]
    return got


def _lens(c):
    """The sequences' lengths: the first is max_len, the others up to `ragged` of it shorter, the last `empty` none."""
    out = [c["max_len"] - int(c["ragged"] * c["max_len"] * ((0.6180339887 * i) % 1.0)) for i in range(c["n_seqs"])]
    return [0 if i >= c["n_seqs"] - c["empty"] else max(n, 1) for i, n in enumerate(out)]


# ----------------------------------------------------------------- layout ----

def _half_bytes(fmt, dim):
    """Bytes of K's (or V's) codes and scales in a strip."""
    codes = dim // PLANE_DIMS[fmt] * STRIP * ROW_BYTES[fmt]
    return codes, dim // 32 * STRIP * 2 if fmt in QUANTISED else 0


def _strip_bytes(c):
    return sum(_half_bytes(c["fmt_k"], c["dim"])) + sum(_half_bytes(c["fmt_v"], c["dim"]))


def _token_bytes(c):
    return _strip_bytes(c) // STRIP


def _parts(pages, c, which):
    """Codes [page, head, strip, plane, 16, row] and scales [page, head, strip, dim / 32, 16] (or None) of K or V."""
    fmt, dim = c["fmt_k"] if which == 0 else c["fmt_v"], c["dim"]
    strips = pages.view(*pages.shape[:-1], c["n_kv"], c["page"] // STRIP, _strip_bytes(c))
    at = 0 if which == 0 else sum(_half_bytes(c["fmt_k"], dim))
    codes, scales = _half_bytes(fmt, dim)
    d = strips[..., at:at + codes].unflatten(-1, (dim // PLANE_DIMS[fmt], STRIP, ROW_BYTES[fmt]))
    if not scales:
        return d, None
    return d, strips[..., at + codes:at + codes + scales].view(torch.float16).unflatten(-1, (dim // 32, STRIP))


def _unpack(codes, scales, fmt, out):
    """Values [.., dims of a plane] in the type `out` from codes and scales."""
    if fmt == "f16":
        return codes.contiguous().view(torch.float16).to(out)
    if fmt == "bf16":
        return codes.contiguous().view(torch.bfloat16).to(out)
    if fmt == "q8_0":
        q = codes.contiguous().view(torch.int8).to(out)
    else:
        q = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).to(out) - 8
    return q * scales.to(out).unsqueeze(-1)


def _pack(x, fmt):
    """Codes [.., planes, row bytes] uint8 and scales [.., dim / 32] f16 (or None) of fp32 rows [.., dim]."""
    if fmt in ("f16", "bf16"):
        h = x.to(torch.float16 if fmt == "f16" else torch.bfloat16).contiguous()
        return h.view(torch.uint8).unflatten(-1, (-1, 32)), None
    b = x.unflatten(-1, (-1, 32))
    if fmt == "q8_0":
        top = b.abs().amax(-1)
        d = (top / torch.full_like(top, 127.0)).half()
    else:
        high, low = b.amax(-1), b.amin(-1)
        d = (torch.where(high >= -low, high, low) * -0.125).half()
    f = d.float()
    inv = torch.where(f != 0, torch.ones_like(f) / f, torch.zeros_like(f)).unsqueeze(-1)
    if fmt == "q8_0":
        return torch.round(b * inv).clamp(-127, 127).to(torch.int8).view(torch.uint8), d
    q = (torch.round(b * inv) + 8).clamp(0, 15).to(torch.uint8)
    return q[..., 0::2] | (q[..., 1::2] << 4), d


def _positions(lens, rows):
    """Position of each sequence's row i of `rows` new ones; negative where the sequence is shorter."""
    return lens.long().unsqueeze(1) - rows + torch.arange(rows, device=lens.device)


def _write(pages, c, table, pos, k, v):
    """Writes fp32 rows k, v [sequence, row, head, dim] at the positions, in place."""
    keep = pos >= 0
    at = pos.clamp(min=0)
    page = table.long().gather(1, at // c["page"])[keep]
    strip, t = (at % c["page"] // STRIP)[keep], (at % STRIP)[keep]
    for which, x in enumerate((k, v)):
        codes, scales = _parts(pages, c, which)
        new, d = _pack(x[keep], c["fmt_k"] if which == 0 else c["fmt_v"])
        codes[page, :, strip, :, t] = new
        if scales is not None:
            scales[page, :, strip, :, t] = d


def _values(pages, c, table):
    """K and V of every position of the sequences, [sequence, position, head, dim]."""
    mine = pages[table.long().clamp(min=0)]
    got = []
    for which in (0, 1):
        codes, scales = _parts(mine, c, which)
        x = _unpack(codes, scales, c["fmt_k"] if which == 0 else c["fmt_v"], torch.float32)
        got.append(x.permute(0, 1, 3, 5, 2, 4, 6).flatten(1, 3).flatten(-2))
    return got


# ---------------------------------------------------------------- prepare ----

def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEVICE)
    g.manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=g, device=DEVICE)

    lens = _lens(c)
    need = [-(-n // c["page"]) for n in lens]
    n_pages, width = sum(need) + 3, max(max(need), 1)
    order = torch.randperm(n_pages, generator=g, device=DEVICE).cpu().tolist()
    table, used = np.full((c["n_seqs"], width), -1, np.int32), 0
    for s, n in enumerate(need):
        table[s, :n] = order[used:used + n]
        used += n
    st = {"case": c, "table": torch.from_numpy(table).to(DEVICE),
          "lens": torch.tensor(lens, dtype=torch.int32, device=DEVICE),
          "pages": torch.zeros((n_pages, c["page"] // STRIP * c["n_kv"] * _strip_bytes(c)), dtype=torch.uint8,
                               device=DEVICE)}
    # what earlier tokens left in the cache: keys and values of unit scale with a few strong channels
    gain = 1.0 + 3.0 * (torch.rand((c["n_kv"], c["dim"]), generator=g, device=DEVICE) > 0.97)
    for which, fmt in enumerate((c["fmt_k"], c["fmt_v"])):
        codes, scales = _parts(st["pages"], c, which)
        x = normal(n_pages, c["n_kv"], c["page"] // STRIP, STRIP, c["dim"])
        new, d = _pack(x * gain[:, None, None] if which == 0 else x, fmt)
        codes.copy_(new.movedim(3, 4))
        if scales is not None:
            scales.copy_(d.movedim(3, 4))
        del x, new, d
    if c["kind"] == "attend":
        st["q"] = normal(c["n_seqs"], c["n_new"], c["n_heads"], c["dim"]) * 1.5
        st["out"] = torch.empty_like(st["q"])
    if c["kind"] == "append":
        # one product's output row holds q, k and v of a token side by side
        width = (c["n_heads"] + 2 * c["n_kv"]) * c["dim"]
        st["qkv"] = normal(c["n_seqs"], c["n_new"], width)
        turns = 10000.0 ** (-2.0 * torch.arange(c["n_rot"] // 2, dtype=torch.float64) / c["n_rot"])
        angle = torch.arange(c["max_len"], dtype=torch.float64).unsqueeze(1) * turns
        st["rope"] = torch.stack((angle.cos(), angle.sin()), -1).float().to(DEVICE)
        st["q_out"] = torch.empty((c["n_seqs"], c["n_new"], c["n_heads"], c["dim"]), device=DEVICE)
    return st


def _qkv(st):
    """q, k and v of a product's output rows, as views."""
    c = st["case"]
    heads = st["qkv"].unflatten(-1, (-1, c["dim"]))
    h, n = c["n_heads"], c["n_kv"]
    return heads[..., :h, :], heads[..., h:h + n, :], heads[..., h + n:, :]


# -------------------------------------------------------------------- run ----

def _turned(x, rope, c, pos):
    """x [sequence, row, head, dim] with its first n_rot dims rotated by the table's rows at the positions."""
    r = rope[pos.clamp(min=0)].unsqueeze(2)
    cos, sin = r[..., 0], r[..., 1]
    half = c["n_rot"] // 2
    turn = x[..., :c["n_rot"]]
    a, b = (turn[..., :half], turn[..., half:]) if c["style"] == "half" else (turn[..., 0::2], turn[..., 1::2])
    y = (a * cos - b * sin, a * sin + b * cos)
    y = torch.cat(y, -1) if c["style"] == "half" else torch.stack(y, -1).flatten(-2)
    return torch.cat((y, x[..., c["n_rot"]:]), -1)


def _seen(lens, n_new, length, window):
    """Which positions [sequence, row, position] a sequence's new rows attend to."""
    pos = _positions(lens, n_new).unsqueeze(-1)
    t = torch.arange(length, device=lens.device)
    seen = t <= pos
    return seen & (t > pos - window) if window else seen


def _plain_attend(st):
    c = st["case"]
    k, v = _values(st["pages"], c, st["table"])
    seen = _seen(st["lens"], c["n_new"], k.shape[1], c["window"])
    k = k.permute(0, 2, 3, 1)                                            # [sequence, kv head, dim, position]
    v = torch.where(seen.any(1)[:, :, None, None], v, 0.0).transpose(1, 2)
    q = st["q"].unflatten(2, (c["n_kv"], -1)).permute(0, 2, 1, 3, 4)     # [sequence, kv head, row, group, dim]
    s = torch.matmul(q.flatten(2, 3), k).unflatten(2, q.shape[2:4]) * (1.0 / math.sqrt(c["dim"]))
    mask = seen[:, None, :, None, :]
    s = torch.where(mask, s, -math.inf)
    top = s.amax(-1, keepdim=True)
    p = torch.where(mask, torch.exp(s - torch.where(torch.isfinite(top), top, 0.0)), 0.0)
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.flatten(2, 3), v).unflatten(2, q.shape[2:4])
    o = torch.where(total > 0, o / torch.where(total > 0, total, 1.0), 0.0)
    return o.permute(0, 2, 1, 3, 4).flatten(2, 3)


def _plain_read(st, starts, count):
    c = st["case"]
    pos = starts.long().unsqueeze(1) + torch.arange(count, device=starts.device)
    ok = (pos >= 0) & (pos < st["lens"].long().unsqueeze(1))
    at = torch.where(ok, pos, 0)
    page = st["table"].long().clamp(min=0).gather(1, at // c["page"])
    strip, t, got = at % c["page"] // STRIP, at % STRIP, []
    for which, fmt in enumerate((c["fmt_k"], c["fmt_v"])):
        codes, scales = _parts(st["pages"], c, which)
        codes = codes[page, :, strip, :, t]                              # [sequence, row, head, plane, row bytes]
        x = _unpack(codes, None if scales is None else scales[page, :, strip, :, t], fmt, torch.float32)
        got.append(torch.where(ok[:, :, None, None], x.flatten(-2), 0.0))
    return tuple(got)


def _plain_append(st):
    c = st["case"]
    q, k, v = _qkv(st)
    pos = _positions(st["lens"], c["n_new"])
    _write(st["pages"], c, st["table"], pos, _turned(k, st["rope"], c, pos), v)
    return _plain_read(st, pos[:, 0], c["n_new"]) + (_turned(q, st["rope"], c, pos),)


def _library(st):
    """The library and its handle of the state's pages."""
    import quantized_weight_gguf_gb300 as lib
    if "cache" not in st:
        c = st["case"]
        st["cache"] = lib.KvCache(c["fmt_k"], c["fmt_v"], st["pages"], c["page"], c["n_kv"], c["dim"])
    return lib, st["cache"]


def run(state):
    st, c = state, state["case"]
    if c["kind"] == "attend":
        if not own:
            return _plain_attend(st)
        lib, cache = _library(st)
        return lib.attend(cache, st["q"], st["table"], st["lens"], window=c["window"], out=st["out"])
    if c["kind"] == "append":
        if not own:
            return _plain_append(st)
        lib, cache = _library(st)
        q, k, v = _qkv(st)
        lib.kv_append(cache, k, v, st["table"], st["lens"], q=q, q_out=st["q_out"], rope=st["rope"], rope_style=c["style"])
        return lib.kv_read(cache, st["table"], st["lens"], c["n_new"]) + (st["q_out"],)
    if not own:
        return _plain_read(st, torch.zeros_like(st["lens"]), c["max_len"])
    lib, cache = _library(st)
    return lib.kv_read(cache, st["table"], st["lens"], c["max_len"], first=0)


# ------------------------------------------------------------------- work ----

def work(case):
    c, lens = case, _lens(case)
    row = c["n_kv"] * _token_bytes(c)
    if c["kind"] == "read":
        # cached rows read; fp32 k and v written for every row asked for
        return {"bytes": sum(lens) * row + 8 * c["n_seqs"] * c["max_len"] * c["n_kv"] * c["dim"], "flops": 0}
    if c["kind"] == "append":
        # q, k, v read and q written in fp32, the table's rows read; k and v written to the cache, read again
        # and returned in fp32
        n = sum(min(x, c["n_new"]) for x in lens)
        values = n * c["dim"] * (2 * c["n_heads"] + 4 * c["n_kv"])
        return {"bytes": 4 * values + 2 * n * row + 4 * c["n_new"] * c["n_rot"],
                "flops": 3 * n * c["n_rot"] * (c["n_heads"] + c["n_kv"])}
    cached = pairs = 0
    for n in lens:
        seen = [min(n - c["n_new"] + 1 + i, c["window"] or n) for i in range(c["n_new"])]
        seen = [max(x, 0) for x in seen]
        pairs += sum(seen)
        cached += min(n, (c["window"] or n) + c["n_new"] - 1)
    values = c["n_seqs"] * c["n_new"] * c["n_heads"] * c["dim"]
    return {"bytes": cached * row + 8 * values, "flops": 4 * pairs * c["n_heads"] * c["dim"]}


# ------------------------------------------------------------------ exact ----

def _exact_rows(state, which, s, n):
    """K or V of positions 0 .. n - 1 of sequence s in fp64, [position, head, dim], from the pages' bytes."""
    c = state["case"]
    fmt = (c["fmt_k"], c["fmt_v"])[which]
    h, dim, strips = c["n_kv"], c["dim"], c["page"] // STRIP
    ids = state["table"][s, :-(-n // c["page"])].long()
    raw = state["pages"][ids].reshape(len(ids), h, strips, _strip_bytes(c))
    kc, ks = _half_bytes(c["fmt_k"], dim)
    vc = _half_bytes(c["fmt_v"], dim)[0]
    begin, size = (0, kc) if which == 0 else (kc + ks, vc)
    body = raw[..., begin:begin + size].contiguous()
    if fmt == "f16":
        x = body.view(torch.float16).double()
    elif fmt == "bf16":
        x = body.view(torch.bfloat16).double()
    elif fmt == "q8_0":
        x = body.view(torch.int8).double()
    else:
        x = torch.empty((*body.shape, 2), dtype=torch.float64, device=body.device)
        x[..., 0] = (body % 16).double() - 8.0
        x[..., 1] = (body // 16).double() - 8.0
    per = PLANE_DIMS[fmt]
    x = x.reshape(len(ids), h, strips, dim // per, STRIP, per)
    if fmt in QUANTISED:
        d = raw[..., begin + size:begin + size + dim // 32 * STRIP * 2].contiguous().view(torch.float16).double()
        x = x * d.reshape(len(ids), h, strips, dim // 32, STRIP, 1)
    x = x.permute(0, 2, 4, 1, 3, 5)
    return x.reshape(len(ids) * c["page"], h, dim)[:n]


def _exact_attend(state):
    c = state["case"]
    out = torch.zeros(state["q"].shape, dtype=torch.float64, device=state["q"].device)
    group = c["n_heads"] // c["n_kv"]
    for s, n in enumerate(_lens(c)):
        if n == 0:
            continue
        k, v = _exact_rows(state, 0, s, n), _exact_rows(state, 1, s, n)
        for i in range(c["n_new"]):
            last = n - c["n_new"] + i
            if last < 0:
                continue
            first = max(0, last + 1 - c["window"]) if c["window"] else 0
            q = state["q"][s, i].double().reshape(c["n_kv"], group, c["dim"])
            e = torch.einsum("hgd,thd->hgt", q, k[first:last + 1]) / math.sqrt(c["dim"])
            w = torch.softmax(e, -1)
            out[s, i] = torch.einsum("hgt,thd->hgd", w, v[first:last + 1]).reshape(c["n_heads"], c["dim"])
    return out


def _exact_kept(x, fmt):
    """What the cache holds of fp64 rows [.., dim] (numpy), as fp64 values."""
    if fmt == "f16":
        return x.astype(np.float16).astype(np.float64)
    if fmt == "bf16":
        m, e = np.frexp(x)                         # eight significant bits, ties to even
        return np.ldexp(np.rint(m * 256.0) / 256.0, e)
    b = x.reshape(*x.shape[:-1], -1, 32)
    if fmt == "q8_0":
        d = (np.abs(b).max(-1) / 127.0).astype(np.float16).astype(np.float64)[..., None]
        q = np.clip(np.rint(np.divide(b, d, out=np.zeros_like(b), where=d != 0)), -127, 127)
    else:
        big = np.where(b.max(-1) >= -b.min(-1), b.max(-1), b.min(-1))
        d = (big / -8.0).astype(np.float16).astype(np.float64)[..., None]
        q = np.clip(np.rint(np.divide(b, d, out=np.zeros_like(b), where=d != 0)), -8, 7)
    return (q * d).reshape(x.shape)


def _exact_append(state):
    c = state["case"]
    x = state["qkv"].double().cpu().numpy().reshape(c["n_seqs"], c["n_new"], -1, c["dim"])
    rope = state["rope"].double().cpu().numpy()
    pos = np.array(_lens(c))[:, None] - c["n_new"] + np.arange(c["n_new"])
    gone = (pos < 0)[:, :, None, None]
    cos, sin = (rope[np.maximum(pos, 0)][..., i][:, :, None, :] for i in (0, 1))
    h, n, r = c["n_heads"], c["n_kv"], c["n_rot"]
    t = x[:, :, :h + n].copy()
    i0, i1 = (slice(0, r // 2), slice(r // 2, r)) if c["style"] == "half" else (slice(0, r, 2), slice(1, r, 2))
    a, b = t[..., i0].copy(), t[..., i1].copy()
    t[..., i0] = a * cos - b * sin
    t[..., i1] = a * sin + b * cos
    k = np.where(gone, 0.0, _exact_kept(t[:, :, h:], c["fmt_k"]))
    v = np.where(gone, 0.0, _exact_kept(x[:, :, h + n:], c["fmt_v"]))
    return k, v, t[:, :, :h]


def exact(case, seed):
    c = case
    state = prepare(c, seed)
    if c["kind"] == "attend":
        return _exact_attend(state)
    if c["kind"] == "append":
        return _exact_append(state)
    lens, outs = _lens(c), []
    for which in (0, 1):
        x = torch.zeros((c["n_seqs"], c["max_len"], c["n_kv"], c["dim"]), dtype=torch.float64, device=DEVICE)
        for s, n in enumerate(lens):
            x[s, :n] = _exact_rows(state, which, s, n)
        outs.append(x)
    return tuple(outs)
