"""Plain statements of the mixture-of-experts calls for the tests, in 64 bits: the choice of experts, and the
experts' feed-forward network over the oracle's weights with a bound on what the library may be off by. Written from
the header, apart from the kernels."""
import numpy as np

import oracle

U = 2.0 ** -24           # half a step of fp32, relative


def magnitudes(fmt, w, k, n):
    """fp64 weights [n, k] and the sizes of the terms they are made of: |w|, and for Q4_K |d sc q| + dmin m, which
    are multiplied by x separately."""
    v = oracle.dequant(fmt, w, k, n).astype(np.float64)
    if fmt != "q4_k":
        return v, np.abs(v)
    b = np.array(w, dtype=np.uint8).reshape(n, k // 256, 144)
    b[..., 16:] = 0      # codes of 0 leave the min term
    mins = np.abs(oracle.dequant(fmt, b.reshape(-1), k, n).astype(np.float64))
    return v, np.abs(v + mins) + mins


def dot_error(x, mag, digits=False):
    """Bound on the error of x . w for rows x [p, k] and weights of sizes mag [n, k]: an x value is kept to 2^-22
    of itself or 2^-38 of the largest of its block of 32, or of its row; a block's products are summed by at most 6 tensor-core
    steps that cut (2^-23 each, of the sizes summed) and its scales multiplied in fp32 (a few U); at most two
    additions per 16 values follow. With `digits` an x value is kept as three signed digits of 8 bits on one step
    for its block, which is at most 2^-22 of the block's largest: half of it, 2^-23, is lost at most."""
    k = x.shape[1]
    c = 2.0 ** -22 + (k / 8 + 80) * U
    pad = np.zeros((x.shape[0], -k % 32))
    top = np.abs(np.concatenate((x, pad), 1)).reshape(x.shape[0], -1, 32).max(-1).repeat(32, 1)[:, :k]
    if not digits:
        top = np.abs(x).max(1, keepdims=True).repeat(k, 1)
    return c * (np.abs(x) @ mag.T) + 2.0 ** (-23 if digits else -38) * (top @ mag.T)


def act(name, g):
    with np.errstate(over="ignore"):
        if name == "swiglu":
            return g / (1.0 + np.exp(-g))
        return g / (1.0 + np.exp(-2.0 * np.sqrt(2.0 / np.pi) * (g + 0.044715 * g ** 3)))


def ffn(name, fmt, wg, wu, fmt_down, wd, x, ids, weights, k, n_ff, n_exp, y0=None):
    """y [n_pos, k] in 64 bits and the bound on the library's error."""
    n_pos, top_k = ids.shape
    y, err = np.zeros((n_pos, k)), np.zeros((n_pos, k))
    wg, wu, wd = (w.reshape(n_exp, -1) for w in (wg, wu, wd))
    size = np.zeros((n_pos, k))
    for e in np.unique(ids):
        if not 0 <= e < n_exp:
            continue
        pos, slot = np.nonzero(ids == e)
        xe = x[pos].astype(np.float64)
        (g, gm), (u, um) = magnitudes(fmt, wg[e], k, n_ff), magnitudes(fmt, wu[e], k, n_ff)
        d, dm = magnitudes(fmt_down, wd[e], n_ff, k)
        gate, up = xe @ g.T, xe @ u.T
        # where experts get a row each at most, quantised weights meet x as digits
        one = ids.size <= n_exp or n_pos == 1
        eg, eu = (dot_error(xe, m, one and fmt not in ("bf16", "f16")) for m in (gm, um))
        w = weights[pos, slot].astype(np.float64)[:, None]
        a = act(name, gate)
        h = a * up * w
        # both activations' derivatives stay below 1.2; the activation and two products round a few times
        eh = np.abs(w) * (1.2 * eg * np.abs(up) + np.abs(a) * eu + 1.2 * eg * eu) + 32 * U * np.abs(h)
        np.add.at(y, pos, h @ d.T)
        np.add.at(err, pos, eh @ dm.T + dot_error(np.abs(h) + eh, dm, one and fmt_down not in ("bf16", "f16")))
        np.add.at(size, pos, np.abs(h) @ dm.T)
    if y0 is not None:
        y, size = y + y0, size + np.abs(y0)
    # the sum over the slots (and y's old value)
    return y, err + (top_k + 2) * U * size + 1e-37


def route(logits, top_k, score, normalize, scale):
    """ids [n_pos, top_k] and weights in 64 bits."""
    n_pos, n = logits.shape
    l = logits.astype(np.float64)
    ids = np.full((n_pos, top_k), -1, np.int32)
    weights = np.zeros((n_pos, top_k))
    for p in range(n_pos):
        order = sorted((i for i in range(n) if l[p, i] > -np.inf), key=lambda i: (-l[p, i], i))[:top_k]
        ids[p, :len(order)] = order
        if not order:
            continue
        best = l[p, order]
        with np.errstate(invalid="ignore", over="ignore"):
            if score == "softmax":
                s = best - best[0]
                over = best if normalize else l[p]
                w = np.exp(s) / np.nansum(np.exp(np.where(np.isnan(over), -np.inf, over) - best[0]))
            else:
                s = np.minimum(best, 0) - np.log1p(np.exp(-np.abs(best)))
                w = np.exp(s - s[0]) / np.exp(s - s[0]).sum() if normalize else np.exp(s)
        if np.isnan(l[p]).any():
            w = np.full(len(order), np.nan)
        weights[p, :len(order)] = w * scale
    return ids, weights
