"""Plain fp64 statements of the serving operators (rotary positions, paged append, paged decode),
from their definitions, for the tests. NumPy on the host; shares nothing with the library."""
import numpy as np


def rotate(x, positions, freqs, interleaved=False, scale=1.0, backward=False):
    """x [N, H, D] -> the first 2 len(freqs) elements of every head rotated."""
    x = np.asarray(x, dtype=np.float64)
    f = np.asarray(freqs, dtype=np.float64)
    angle = np.asarray(positions, dtype=np.float64)[:, None, None] * f
    c, n = scale * np.cos(angle), scale * np.sin(angle) * (-1.0 if backward else 1.0)
    m = len(f)
    y = x.copy()
    a, b = (x[..., 0:2 * m:2], x[..., 1:2 * m:2]) if interleaved else (x[..., :m], x[..., m:2 * m])
    ya, yb = c * a - n * b, n * a + c * b
    if interleaved:
        y[..., 0:2 * m:2], y[..., 1:2 * m:2] = ya, yb
    else:
        y[..., :m], y[..., m:2 * m] = ya, yb
    return y


def new_rows(lengths, counts):
    """(row, sequence, position) of every new token, counts[b] of them ending sequence b."""
    out, row = [], 0
    for b, (L, n) in enumerate(zip(lengths, counts)):
        for t in range(n):
            out.append((row, b, L - n + t))
            row += 1
    return out


def decode(q, q_idx, k_pages, v_pages, k_idx_pages, table, lengths, k, bk, scale=None):
    """q [B, S, Hq, d] ... -> (o [B, S, Hq, d], ids [B, S, G, k], weight [B, S, Hq, d]): the last is
    the sum of softmax weight * |v|, which error bounds are made of."""
    q, q_idx = np.asarray(q, dtype=np.float64), np.asarray(q_idx, dtype=np.float64)
    B, S, Hq, d = q.shape
    ps, G = k_pages.shape[1:3]
    R = Hq // G
    scale = 1.0 / np.sqrt(d) if scale is None else scale
    o, weight = np.zeros_like(q), np.zeros_like(q)
    ids = np.full((B, S, G, k), -1, dtype=np.int32)
    for b in range(B):
        n = int(lengths[b])
        if n == 0:
            continue
        pages = np.asarray(table[b][:-(-n // ps)], dtype=np.int64)
        kk, vv, ki = (np.asarray(t[pages], dtype=np.float64).reshape(-1, G, t.shape[3])[:n]
                      for t in (k_pages, v_pages, k_idx_pages))
        for s in range(S):
            p = n - S + s
            if p < 0:
                continue
            local = p // bk
            for g in range(G):
                if local + 1 <= k:
                    chosen = np.arange(local + 1)
                else:
                    score = (ki[:local * bk, g] @ q_idx[b, s, g]).reshape(local, bk).max(axis=1)
                    order = np.argsort(-score, kind="stable")   # equal scores: the lower block first
                    chosen = np.sort(np.append(order[:k - 1], local))
                ids[b, s, g, :len(chosen)] = chosen
                tok = (chosen[:, None] * bk + np.arange(bk)).reshape(-1)
                tok = tok[tok <= p]
                for h in range(g * R, (g + 1) * R):
                    z = scale * (kk[tok, g] @ q[b, s, h])
                    w = np.exp(z - z.max())
                    w /= w.sum()
                    o[b, s, h] = w @ vv[tok, g]
                    weight[b, s, h] = w @ np.abs(vv[tok, g])
    return o, ids, weight
