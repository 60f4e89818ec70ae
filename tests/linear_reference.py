"""Plain statement of linear attention for the tests: the recurrence in 64 bits, row by row, with a bound on what the
library may be off by. Written from the header, apart from the kernels."""
import numpy as np

STEP_ROWS = 8    # rows up to which the library takes them one by one


def attend(q, k, v, decay, state, lens, scale):
    """out, state after the last row, and the bounds on their errors. decay [n_seqs, n_new, n_heads]."""
    n_seqs, n_new, n_heads, dv = v.shape
    group = n_heads // q.shape[2]
    q, k = (np.repeat(x.astype(np.float64), group, 2) for x in (q, k))
    v, s_all = v.astype(np.float64), state.astype(np.float64).copy()
    out, tol, s_tol = np.zeros(v.shape), np.zeros(v.shape), np.zeros(s_all.shape)
    # Terms keep 2^-22 of a value or 2^-38 of the largest beside it: sizes enlarged by 2^-16 of that largest stand for
    # both. A handful of such errors, cutting sums and fp32 roundings a row (2^-20 in all), and per chunk of 32 a decay
    # (exp2f, 2 steps of 2^-23) and the state's sums (a few 2^-24). One by one: two roundings and expf's 2 steps a row.
    per = 2.0 ** -20 + (n_new / 32 * 2.0 ** -20 if n_new > STEP_ROWS else n_new * 2.0 ** -21)
    small = 2.0 ** -16
    with np.errstate(invalid="ignore", over="ignore"):
        for s in range(n_seqs):
            n = n_new + 1 if lens is None else int(lens[s])
            if n <= 0:
                continue
            if n <= n_new:
                s_all[s] = 0
            first = max(0, n_new - n)
            S, A = s_all[s], np.abs(s_all[s])
            rows = slice(first, n_new)
            v_top = np.abs(v[s, rows]).max(0)                      # [head, dv]
            k_top = np.abs(k[s, rows]).max((0, 2))                 # [head]
            for i in range(first, n_new):
                g = np.minimum(decay[s, i].astype(np.float64), 0)
                g = np.where(np.isnan(decay[s, i]), np.nan, g)
                a = np.exp(g)[:, None, None]
                S = S * a + k[s, i][:, :, None] * v[s, i][:, None, :]
                ka = np.abs(k[s, i]) + small * np.abs(k[s, i]).max(-1, keepdims=True)
                A = A * a + ka[:, :, None] * (np.abs(v[s, i]) + small * v_top)[:, None, :]
                qa = np.abs(q[s, i])
                out[s, i] = np.einsum("hd,hdv->hv", q[s, i], S) * scale
                wide = A + small * A.max(1, keepdims=True)
                q_top = qa.max(-1, keepdims=True)
                t = np.einsum("hd,hdv->hv", qa + small * q_top, wide) * per
                tol[s, i] = (t + 32 * 2.0 ** -31 * q_top * k_top[:, None] * v_top) * abs(scale) + 1e-37
            s_all[s], s_tol[s] = S, A * per + 1e-37
    return out, s_all, tol, s_tol
