"""Token-by-token generation in fp64 on the CPU: the recurrent KDA step on cached states and absorbed
latent attention over a paged cache.  Written from the definitions, row by row; every function also
returns the sums of absolute values that its rounding-error bounds are stated in."""
from __future__ import annotations

import numpy as np

LAT, ROPE, HEAD = 512, 64, 128


def runs(n_rows, n_seqs, row_start=None):
    """[(sequence, first row, rows)]."""
    if row_start is None:
        assert n_rows == n_seqs
        return [(b, b, 1) for b in range(n_seqs)]
    return [(b, int(row_start[b]), int(row_start[b + 1] - row_start[b])) for b in range(n_seqs)]


def kda_step(state, src, dst, q, k, v, g, beta, row_start=None):
    """(o, new state, abs(o), abs(state)): abs are the same recurrences with every term's magnitude."""
    H, d = q.shape[1:]
    new, mag = state.copy(), np.abs(state)
    o, oa = np.full(q.shape, np.nan), np.full(q.shape, np.nan)
    for b, first, m in runs(len(q), len(src), row_start):
        if src[b] < 0:
            continue
        for h in range(H):
            S = state[src[b], h].copy()
            A = np.abs(S)
            for t in range(first, first + m):
                a, kk = np.exp(g[t, h]), k[t, h]
                S, A = a[:, None] * S, a[:, None] * A
                S = S + beta[t, h] * np.outer(kk, v[t, h] - S.T @ kk)
                A = A + beta[t, h] * np.outer(np.abs(kk), np.abs(v[t, h]) + A.T @ np.abs(kk))
                o[t, h], oa[t, h] = S.T @ q[t, h], A.T @ np.abs(q[t, h])
            new[dst[b], h], mag[dst[b], h] = S, A
    return o, new, oa, mag


def rotate(x, pos):
    """Half-split rotation (base 10000) of the 64 rotary values at integer position pos."""
    ang = float(pos) * 10000.0 ** (-2.0 * np.arange(ROPE // 2) / ROPE)
    a, b = x[..., :ROPE // 2], x[..., ROPE // 2:]
    return np.concatenate([a * np.cos(ang) - b * np.sin(ang), a * np.sin(ang) + b * np.cos(ang)], -1)


def append(cache, table, kv_len, c, kr, row_start=None):
    new = cache.copy()
    page = cache.shape[1]
    for b, first, m in runs(len(c), len(kv_len), row_start):
        for i in range(m):
            p = int(kv_len[b]) - m + i
            if p >= 0:
                new[table[b, p // page], p % page] = np.concatenate([c[first + i], rotate(kr[first + i], p)])
    return new


def absorb(q, w_b, kv_len, row_start=None):
    """(qa, abs(qa)); rows of no sequence are NaN."""
    n, H, _ = q.shape
    w = w_b[:H * HEAD].reshape(H, HEAD, LAT)
    out, mag = np.full((n, H, LAT + ROPE), np.nan), np.full((n, H, LAT + ROPE), np.nan)
    for b, first, m in runs(n, len(kv_len), row_start):
        for i in range(m):
            x = q[first + i]
            rot = rotate(x[:, HEAD:], int(kv_len[b]) - m + i)
            out[first + i] = np.concatenate([np.einsum("hi,hil->hl", x[:, :HEAD], w), rot], -1)
            half = np.abs(x[:, HEAD:HEAD + 32]) + np.abs(x[:, HEAD + 32:])
            mag[first + i] = np.concatenate([np.einsum("hi,hil->hl", np.abs(x[:, :HEAD]), np.abs(w)), half, half], -1)
    return out, mag


def expand(o, w_b):
    H = o.shape[1]
    w = w_b[H * HEAD:].reshape(H, HEAD, LAT)
    return np.einsum("thl,hil->thi", o, w), np.einsum("thl,hil->thi", np.abs(o), np.abs(w))


def attention(qa, cache, table, kv_len, scale, row_start=None):
    """(o, lse, sum p |c|, largest sum |q||k| scale of a row); rows of no sequence are NaN."""
    n, H, _ = qa.shape
    o, oa = np.full((n, H, LAT), np.nan), np.full((n, H, LAT), np.nan)
    lse, sa = np.full((n, H), np.nan), np.zeros((n, H))
    for b, first, m in runs(n, len(kv_len), row_start):
        L = int(kv_len[b])
        mem = np.zeros((0, LAT + ROPE))
        if L > 0 and m > 0:
            mem = cache[table[b, :-(-L // cache.shape[1])]].reshape(-1, LAT + ROPE)[:L]
        for i in range(m):
            seen = mem[:max(L - m + 1 + i, 0)]
            if len(seen) == 0:
                o[first + i], oa[first + i], lse[first + i] = 0, 0, -np.inf
                continue
            z = scale * (qa[first + i] @ seen.T)
            mx = z.max(-1, keepdims=True)
            p = np.exp(z - mx)
            s = p.sum(-1, keepdims=True)
            p /= s
            o[first + i], oa[first + i] = p @ seen[:, :LAT], p @ np.abs(seen[:, :LAT])
            lse[first + i] = (mx + np.log(s))[:, 0]
            sa[first + i] = scale * (np.abs(qa[first + i]) @ np.abs(seen.T)).max(-1)
    return o, lse, oa, sa


def expanded_attention(q, c, kr, w_b, scale):
    """Causal latent attention of one sequence in its expanded form: q [T, H, 192], c [T, 512], kr [T, 64],
    all positions 0 .. T - 1 (unrotated): [k_nope | v] = c W_b^T.  Returns [T, H, 128]."""
    T, H, _ = q.shape
    kn = np.einsum("tl,hil->thi", c, w_b[:H * HEAD].reshape(H, HEAD, LAT))
    v = np.einsum("tl,hil->thi", c, w_b[H * HEAD:].reshape(H, HEAD, LAT))
    k = np.concatenate([kn, np.stack([np.tile(rotate(kr[t], t), (H, 1)) for t in range(T)])], -1)
    qr = np.stack([np.concatenate([q[t, :, :HEAD], rotate(q[t, :, HEAD:], t)], -1) for t in range(T)])
    out = np.zeros((T, H, HEAD))
    for t in range(T):
        z = scale * np.einsum("he,jhe->hj", qr[t], k[:t + 1])
        p = np.exp(z - z.max(-1, keepdims=True))
        out[t] = np.einsum("hj,jhi->hi", p / p.sum(-1, keepdims=True), v[:t + 1])
    return out
