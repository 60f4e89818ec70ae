"""How far results of the experts' network and of linear attention may be off as a whole: the norm of a position's
(a head's) errors. Beside the element-wise bounds of experts_reference and linear_reference, which hold for the
worst signs and are wide, these take roundings as what they are over random values, independent of one another, so that
squares add: narrow enough to notice values that were rounded to one 16-bit term.

U = 2^-24 is fp32's half step. A dot of K products of x and w, whose squares sum to D^2, is off by no more than (root
mean square)
    D (sqrt(K / 16) + 16) U :
at most an addition per 16 products, each off by U of a partial sum (itself D at most); and 16 U for what follows all of a
dot alike: the tensor cores' cut sums within a block (6 of them), the scales' roundings (4) and an operand's terms: 22 bits
of a value are 1.2 U root mean square, digits on a step of 2^-22 of the largest of 32 values (2 to 2.5 times their root mean
square, 1 / sqrt(12) of a step) 3 U."""
import numpy as np

import experts_reference as experts

U = 2.0 ** -24


def ffn(name, fmt, wg, wu, fmt_down, wd, x, ids, weights, k, n_ff, n_exp, y0=None):
    """y [n_pos, k] in 64 bits and the bound [n_pos] on the norms of its errors."""
    n_pos, top_k = ids.shape
    y, var = np.zeros((n_pos, k)), np.zeros((n_pos, k))
    wg, wu, wd = (w.reshape(n_exp, -1) for w in (wg, wu, wd))
    c_in, c_down = ((np.sqrt(n / 16) + 16) * U for n in (k, n_ff))
    for e in np.unique(ids):
        if not 0 <= e < n_exp:
            continue
        pos, slot = np.nonzero(ids == e)
        xe = x[pos].astype(np.float64)
        (g, gm), (u, um) = experts.magnitudes(fmt, wg[e], k, n_ff), experts.magnitudes(fmt, wu[e], k, n_ff)
        d, dm = experts.magnitudes(fmt_down, wd[e], n_ff, k)
        gate, up = xe @ g.T, xe @ u.T
        w = weights[pos, slot].astype(np.float64)[:, None]
        a = experts.act(name, gate)
        h = a * up * w
        # the activations' derivatives stay below 1.2; the activation and two products round a few times
        vh = w ** 2 * ((1.2 * up * c_in) ** 2 * (xe ** 2 @ (gm ** 2).T) + (a * c_in) ** 2 * (xe ** 2 @ (um ** 2).T)) \
            + (16 * U * h) ** 2
        np.add.at(y, pos, h @ d.T)
        np.add.at(var, pos, vh @ (dm ** 2).T + c_down ** 2 * (h ** 2 @ (dm ** 2).T))
    if y0 is not None:
        y = y + y0
    # the sum over the slots (and y's old value)
    return y, np.sqrt(var.sum(1)) + top_k * U * np.linalg.norm(y, axis=1)


def linear(q, k, v, decay, state, scale):
    """out, the state after the last row, and the bounds on the norms of their errors, [n_seqs, n_heads] each. decay
    [n_seqs, n_new, n_heads]. As for a dot, with the state as a sum over T chunks of 32 rows (or rows), each with two
    roundings of the sum and a decay's two steps (2 U each) after it: (4 sqrt(T) + 16) U of the root of the squares'
    sums; an output adds a dot of dk products over it."""
    n_seqs, n_new, n_heads, dv = v.shape
    dk = q.shape[3]
    q, k = (np.repeat(x.astype(np.float64), n_heads // q.shape[2], 2) for x in (q, k))
    v, S = v.astype(np.float64), state.astype(np.float64).copy()
    V = S ** 2
    out, var = np.zeros(v.shape), np.zeros((n_seqs, n_heads))
    c = (4 * np.sqrt(n_new / 32 if n_new > 8 else n_new) + 16) * U
    for i in range(n_new):
        a = np.exp(np.minimum(decay[:, i].astype(np.float64), 0))[..., None, None]
        S = S * a + k[:, i][..., None] * v[:, i][..., None, :]
        V = V * a ** 2 + (k[:, i] ** 2)[..., None] * (v[:, i] ** 2)[..., None, :]
        out[:, i] = np.einsum("shd,shdv->shv", q[:, i], S) * scale
        var += np.einsum("shd,shdv->sh", q[:, i] ** 2, V) * scale ** 2
    per_out = np.hypot(c, (np.sqrt(dk / 16) + 16) * U)
    return out, S, np.sqrt(var) * per_out, np.sqrt(V.sum((2, 3))) * c
