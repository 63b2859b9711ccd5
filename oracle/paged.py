"""Paged cache, position rotation, ragged causal and differential attention (oracle; test
infrastructure only): plain numpy from the definitions, fp64 unless the canonical fp32
sequence is asked for."""

import numpy as np


def rope(x, cos, sin, pos, interleaved=False):
    """Rows x [n, heads, d] turned by their positions pos [n], in the dtype of x, each product
    and sum rounded once (pair (a, b) -> (a c - b s, a s + b c)); elements past rot_dim pass."""
    x = np.array(x, copy=True)
    half = cos.shape[1]
    first = np.arange(0, 2 * half, 2) if interleaved else np.arange(half)
    second = first + (1 if interleaved else half)
    c, s = (t[np.asarray(pos)].astype(x.dtype)[:, None] for t in (cos, sin))
    a, b = x[..., first].copy(), x[..., second].copy()
    x[..., first] = a * c - b * s
    x[..., second] = a * s + b * c
    return x


def places(seq_lens, cu_q):
    """(row, sequence, position) of every row of the batch that has a place; and the rows that
    belong to a sequence but lie before its start."""
    at, none = [], []
    for b, n in enumerate(seq_lens):
        t = int(cu_q[b + 1] - cu_q[b])
        for i in range(t):
            pos = int(n) - t + i
            (at if pos >= 0 else none).append((int(cu_q[b]) + i, b, pos))
    return at, none


def sequence_rows(pages, table, b, n):
    """Packed rows [n, Hkv, 68] of sequence b (pages uint8 [n_pages, Hkv, P, 68])."""
    P = pages.shape[2]
    t = np.arange(n)
    return pages[table[b, t // P], :, t % P]


def dequantize(codec, rows, unrotate=True):
    return codec.dequantize(rows.reshape(-1, 68), unrotate=unrotate).reshape(*rows.shape[:2], codec.d)


def attention(kc, vc, kp, vp, table, seq_lens, cu_q, q, n_rows, scale=0.0, turn=None):
    """fp64 [n_rows, Hq, 128]; rows of no sequence NaN, rows without a key 0.  turn(q, pos): the
    queries' rotation."""
    Hq, d = q.shape[1], q.shape[2]
    g = Hq // kp.shape[1]
    scale = scale or 1.0 / np.sqrt(d)
    out = np.full((n_rows, Hq, d), np.nan)
    for b, n in enumerate(seq_lens):
        a, e = int(cu_q[b]), int(cu_q[b + 1])
        out[a:e] = 0.0
        if n <= 0:
            continue
        K = dequantize(kc, sequence_rows(kp, table, b, n))
        V = dequantize(vc, sequence_rows(vp, table, b, n))
        for i in range(a, e):
            pos = n - (e - i)
            if pos < 0:
                continue
            x = q[i:i + 1].astype(np.float64)
            x = (turn(x, np.array([pos])) if turn else x)[0]
            s = np.einsum("hd,thd->ht", x, np.repeat(K[:pos + 1], g, axis=1)) * scale
            w = np.exp(s - s.max(axis=1, keepdims=True))
            w /= w.sum(axis=1, keepdims=True)
            out[i] = np.einsum("ht,thd->hd", w, np.repeat(V[:pos + 1], g, axis=1))
    return out


def differential(att, lam, gain=None, eps=1e-5, out_scale=1.0):
    """Head pairs of att [n, Hq, d]: d = a_2p - lam a_2p+1, RMS norm with gain, scale."""
    d = att[:, 0::2] - np.asarray(lam, np.float64)[..., None] * att[:, 1::2]
    if gain is not None:
        d = d / np.sqrt((d * d).mean(-1, keepdims=True) + eps) * np.asarray(gain, np.float64)
    return d * out_scale
