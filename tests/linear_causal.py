"""Linear attention for the tests: the recurrence in 64 bits with a bound on the library's error that knows of a row only
what the header lets it depend on, the rows up to its own and what the decays have left of them. Written from the
header, apart from the kernels."""
import numpy as np

STEP_ROWS = 8    # rows up to which the library takes them one by one


def attend(q, k, v, decay, state, scale, floor=2.0 ** -138):
    """out, state after the last row, and the bounds on their errors. decay [n_seqs, n_new, n_heads].

    A row's q and k keep 2^-22 of a value or 2^-38 of the row's largest: sizes enlarged by 2^-16 of that largest stand
    for both. So does what a state's dim holds beside its largest. What rows add to the state (v times the row's largest
    k) keeps 2^-38 of the dim's largest of up to 32 rows, as they are decayed: 2^-33 in all, 2^-11 beside the factor
    below. That factor: a handful of such errors, cutting sums and fp32 roundings a row (2^-20 in all), and per chunk
    of 32 a decay and the state's sums (2^-20); one by one two roundings and a decay's two steps a row."""
    n_seqs, n_new, n_heads, dv = v.shape
    group = n_heads // q.shape[2]
    q, k = (np.repeat(x.astype(np.float64), group, 2) for x in (q, k))
    v, s_all = v.astype(np.float64), state.astype(np.float64).copy()
    per = 2.0 ** -20 + (n_new / 32 * 2.0 ** -20 if n_new > STEP_ROWS else n_new * 2.0 ** -21)
    out, tol, s_tol = np.zeros(v.shape), np.zeros(v.shape), np.zeros(s_all.shape)
    for s in range(n_seqs):
        S, A = s_all[s], np.abs(s_all[s])
        B = np.zeros((n_heads, dv))
        for i in range(n_new):
            a = np.exp(np.minimum(decay[s, i].astype(np.float64), 0))[:, None, None]
            S = S * a + k[s, i][:, :, None] * v[s, i][:, None, :]
            k_size, k_top = np.abs(k[s, i]), np.abs(k[s, i]).max(-1, keepdims=True)
            A = A * a + (k_size + 2.0 ** -16 * k_top)[:, :, None] * np.abs(v[s, i])[:, None, :]
            B = B * a[:, 0] + k_top * np.abs(v[s, i])
            wide = A + 2.0 ** -16 * A.max(1, keepdims=True) + 2.0 ** -11 * B[:, None, :]
            q_size = np.abs(q[s, i])
            q_size = q_size + 2.0 ** -16 * q_size.max(-1, keepdims=True)
            out[s, i] = np.einsum("hd,hdv->hv", q[s, i], S) * scale
            tol[s, i] = np.einsum("hd,hdv->hv", q_size, wide) * (per * abs(scale)) + floor
        s_all[s], s_tol[s] = S, wide * per + floor
    return out, s_all, tol, s_tol
