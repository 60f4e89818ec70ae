"""Plain statements of the paged key-value cache operators for the tests, in
numpy: the page layout that include/qmm.h documents, packing as the fp32
formulas say, and rotation and attention in 64 bits. Written from the header,
apart from the kernels."""
import numpy as np

FORMATS = [("f16", "f16"), ("bf16", "bf16"), ("q8_0", "q8_0"), ("q4_0", "q4_0"), ("q8_0", "q4_0")]
QUANTISED = ("q8_0", "q4_0")


def half_bytes(fmt, dim):
    if fmt in ("f16", "bf16"):
        return 32 * dim, 0
    return (16 * dim if fmt == "q8_0" else 8 * dim), dim


def strip_bytes(fk, fv, dim):
    return sum(half_bytes(fk, dim)) + sum(half_bytes(fv, dim))


def bf16_bits(x):
    u = x.astype(np.float32).view(np.uint32).astype(np.uint64)
    return ((u + 0x7FFF + ((u >> 16) & 1)) >> 16).astype(np.uint16)


def pack(x, fmt):
    """Codes [.., dim / 32, bytes] and scales [.., dim / 32] f16 (or None) of finite fp32 rows, by
    the header's fp32 formulas."""
    x = x.astype(np.float32)
    if fmt == "f16":
        h = x.astype(np.float16).view(np.uint16)
        return np.ascontiguousarray(h).view(np.uint8), None
    if fmt == "bf16":
        return np.ascontiguousarray(bf16_bits(x)).view(np.uint8), None
    b = x.reshape(*x.shape[:-1], -1, 32)
    with np.errstate(over="ignore"):
        if fmt == "q8_0":
            d = np.abs(b).max(-1) / np.float32(127)
        else:
            hi, lo = b.max(-1), b.min(-1)
            d = np.where(hi >= -lo, hi, lo) * np.float32(-0.125)
        d = np.clip(d, -65504, 65504).astype(np.float16)
    f = d.astype(np.float32)
    with np.errstate(divide="ignore"):
        inv = np.where(f != 0, np.float32(1) / f, np.float32(0))[..., None]
    q = np.rint(b * inv)
    if fmt == "q8_0":
        return np.clip(q, -127, 127).astype(np.int8).view(np.uint8), d
    q = np.clip(q + 8, 0, 15).astype(np.uint8)
    return q[..., 0::2] | (q[..., 1::2] << 4), d


def unpack(codes, d, fmt):
    """Values [.., dim] in 64 bits (any bytes, NaN and Inf among them)."""
    with np.errstate(invalid="ignore"):
        return _unpack(codes, d, fmt)


def _unpack(codes, d, fmt):
    if fmt == "f16":
        return codes.view(np.float16).astype(np.float64)
    if fmt == "bf16":
        return (codes.view(np.uint16).astype(np.uint32) << 16).view(np.float32).astype(np.float64)
    q = codes.view(np.int8).astype(np.float64) if fmt == "q8_0" else \
        np.stack((codes & 15, codes >> 4), -1).reshape(*codes.shape[:-1], -1).astype(np.float64) - 8
    v = q * d.astype(np.float64)[..., None]
    return v.reshape(*v.shape[:-2], -1)


class Pages:
    """A pool of pages in host memory, [n_pages][kv head][strip][strip bytes]."""

    def __init__(self, fk, fv, n_pages, page, n_kv, dim, fill=None):
        self.fk, self.fv, self.page, self.n_kv, self.dim = fk, fv, page, n_kv, dim
        size = n_kv * (page // 16) * strip_bytes(fk, fv, dim)
        self.raw = np.zeros((n_pages, size), np.uint8) if fill is None else fill((n_pages, size))
        self.strips = self.raw.reshape(n_pages, n_kv, page // 16, -1)

    def parts(self, which):
        fmt = (self.fk, self.fv)[which]
        at = 0 if which == 0 else sum(half_bytes(self.fk, self.dim))
        c, s = half_bytes(fmt, self.dim)
        per = 16 if fmt in ("f16", "bf16") else 32
        codes = self.strips[..., at:at + c].reshape(*self.strips.shape[:3], self.dim // per, 16, -1)
        scales = None
        if s:
            scales = np.ascontiguousarray(self.strips[..., at + c:at + c + s]).view(np.float16)
            scales = scales.reshape(*self.strips.shape[:3], self.dim // 32, 16)
        return codes, scales

    def put(self, which, page, h, offset, x):
        """fp32 row x [dim] at an offset of a page."""
        fmt = (self.fk, self.fv)[which]
        strip, t = divmod(offset, 16)
        at = 0 if which == 0 else sum(half_bytes(self.fk, self.dim))
        c, s = half_bytes(fmt, self.dim)
        mine = self.strips[page, h, strip]
        codes, d = pack(x, fmt)
        per = 16 if fmt in ("f16", "bf16") else 32
        codes = codes.reshape(self.dim // per, -1)
        mine[at:at + c].reshape(self.dim // per, 16, -1)[:, t] = codes
        if s:
            mine[at + c:at + c + s].reshape(self.dim // 32, 16, 2)[:, t] = \
                np.ascontiguousarray(d).view(np.uint8).reshape(-1, 2)

    def values(self, which, table, n):
        """K or V of positions 0 .. n - 1 under a table row, [n, n_kv, dim] in 64 bits."""
        fmt = (self.fk, self.fv)[which]
        codes, scales = self.parts(which)
        out = np.zeros((n, self.n_kv, self.dim))
        for p in range(n):
            pg, o = int(table[p // self.page]), p % self.page
            c = np.ascontiguousarray(codes[pg, :, o // 16, :, o % 16])
            if scales is None:
                out[p] = unpack(c.reshape(self.n_kv, -1), None, fmt)
            else:
                out[p] = unpack(c, scales[pg, :, o // 16, :, o % 16], fmt)
        return out


def rotate(x, pos, rope, n_rot, style, dtype):
    """x [.., dim] rotated by the table's row `pos`, in dtype (float32: products and sums rounded
    one by one; float64: exact but for its rounding)."""
    x = x.astype(dtype).copy()
    c, s = rope[pos, :, 0].astype(dtype), rope[pos, :, 1].astype(dtype)
    i0, i1 = (slice(0, n_rot // 2), slice(n_rot // 2, n_rot)) if style == "half" else \
        (slice(0, n_rot, 2), slice(1, n_rot, 2))
    a, b = x[..., i0].copy(), x[..., i1].copy()
    x[..., i0] = a * c - b * s
    x[..., i1] = a * s + b * c
    return x


def make_table(rng, lens, page, extra=2, width=None):
    """A page table over a shuffled pool (entries past each length -1) and the pool's size."""
    need = [-(-max(int(n), 0) // page) for n in lens]
    n_pages = sum(need) + extra
    order = rng.permutation(n_pages)
    table = np.full((len(lens), max(width or 0, max(need + [1]))), -1, np.int32)
    used = 0
    for s, n in enumerate(need):
        table[s, :n] = order[used:used + n]
        used += n
    return table, n_pages


def attention(q, k, v, first, last, scale):
    """One row: q [n_heads, dim], k and v [n, n_kv, dim] in 64 bits, positions first .. last.
    Returns the output and its tolerance.

    The tolerance: a weight p_t = e^(s_t - max) / sum is off by the errors of its score and of the
    sums around it. A score's error is at most (dim / 16 + 8) 2^-23 M, M = max_t |scale| sum |q k|:
    q enters as terms of at least 22 bits, the products are exact, and each of the dim / 16 steps
    of an fp32 sum rounds or cuts once. The weights' relative error is twice that (the total has
    it too), plus a few roundings of the exponential; the sum over positions rounds once per 16 of
    them. All are relative to sum_t p_t |v_t|."""
    n_heads, dim = q.shape
    out = np.zeros((n_heads, dim))
    tol = np.zeros((n_heads, dim))
    if last < first:
        return out, tol
    g = n_heads // k.shape[1]
    for h in range(n_heads):
        kk, vv = k[first:last + 1, h // g], v[first:last + 1, h // g]
        s = scale * (kk @ q[h].astype(np.float64))
        p = np.exp(s - s.max())
        p /= p.sum()
        out[h] = p @ vv
        m = (abs(scale) * (np.abs(kk) @ np.abs(q[h].astype(np.float64)))).max()
        steps = 2 * (dim / 16 + 8) * m + (last + 1 - first) / 16 + 16
        tol[h] = steps * 2.0 ** -23 * (p @ np.abs(vv))
    return out, tol
