"""Plain 64-bit forms of the serving operators for the tests: numpy, one
sequence, head and row at a time, written from the formulas in include/qmm.h
and sharing no code with the library."""
import numpy as np


def rope_table(rows, dim, base=10000.0):
    """fp32 [rows][dim / 2][2] of (cos, sin)."""
    f = base ** (-np.arange(0, dim, 2) / dim)
    a = np.arange(rows)[:, None] * f
    return np.stack([np.cos(a), np.sin(a)], -1).astype(np.float32)


def rotate(x, pos, table, adjacent):
    """x [..., dim] at one position."""
    if table is None:
        return x
    y = np.array(x, dtype=np.float64)
    n = table.shape[1]
    c, s = table[pos, :, 0].astype(np.float64), table[pos, :, 1].astype(np.float64)
    a = slice(0, 2 * n, 2) if adjacent else slice(0, n)
    b = slice(1, 2 * n, 2) if adjacent else slice(n, 2 * n)
    y[..., a], y[..., b] = x[..., a] * c - x[..., b] * s, x[..., a] * s + x[..., b] * c
    return y


def attend(q, k, v, pos, scale, causal=True, window=0):
    """One row of one head: q [dim] (rotated), k and v [tokens][dim]. Returns
    out [dim], lse, and what error bounds need: sum p |v| and the largest
    scale * sum |q| |k| of a token it sees."""
    j = np.arange(len(k))
    sees = (j <= pos) if causal else np.ones(len(k), bool)
    if window:
        sees &= j > pos - window
    if not sees.any():
        return np.zeros(v.shape[1]), -np.inf, np.zeros(v.shape[1]), 0.0
    x = scale * (k[sees] @ q)
    m = x.max()
    p = np.exp(x - m)
    l = p.sum()
    size = scale * (np.abs(k[sees]) @ np.abs(q)).max()
    return (p / l) @ v[sees], m + np.log(l), (p / l) @ np.abs(v[sees]), size


def logprobs(x, given, top):
    """One row of logits: lse, entropy, log probabilities of `given`, ids and
    log probabilities of the `top` most likely (ties by rising id)."""
    x = np.asarray(x, dtype=np.float64)
    m = x.max()
    if m == -np.inf:
        lse, ent, lp = -np.inf, 0.0, np.full(len(x), -np.inf)
    else:
        log_l = np.log(np.exp(x - m).sum())
        lse, lp = m + log_l, (x - m) - log_l
        p = np.exp(lp)
        ent = -(p[p > 0] * lp[p > 0]).sum()
    ids = np.argsort(-x, kind="stable")[:top]
    return lse, ent, lp[given], ids, lp[ids]
