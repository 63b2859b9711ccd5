"""Drafted trees over the paged cache: positions, attention, verification, kept paths (oracle; test
infrastructure only): plain numpy from the definitions."""

from fractions import Fraction

import numpy as np

from oracle import paged


def lines(parents):
    """The ancestors of every node of one tree, the node itself last."""
    out = []
    for i, p in enumerate(parents):
        out.append((out[p] if 0 <= p < i else []) + [i])
    return out


def positions(seq_lens, cu_q, parents):
    """Position of every row: context length plus depth."""
    pos = np.zeros(len(parents), int)
    for b, n in enumerate(seq_lens):
        a, e = int(cu_q[b]), int(cu_q[b + 1])
        for i, line in enumerate(lines(parents[a:e])):
            pos[a + i] = int(n) - (e - a) + len(line) - 1
    return pos


def attention(kc, vc, kp, vp, table, seq_lens, cu_q, parents, q, n_rows, scale=0.0, turn=None):
    """fp64 [n_rows, Hq, 128]; rows of no sequence NaN, rows without a slot 0."""
    Hq, d = q.shape[1], q.shape[2]
    g = Hq // kp.shape[1]
    scale = scale or 1.0 / np.sqrt(d)
    out = np.full((n_rows, Hq, d), np.nan)
    pos = positions(seq_lens, cu_q, parents)
    for b, n in enumerate(seq_lens):
        a, e = int(cu_q[b]), int(cu_q[b + 1])
        out[a:e] = 0.0
        if n <= 0 or e == a:
            continue
        K = paged.dequantize(kc, paged.sequence_rows(kp, table, b, n))
        V = paged.dequantize(vc, paged.sequence_rows(vp, table, b, n))
        c = n - (e - a)
        for i, line in enumerate(lines(parents[a:e])):
            if c + i < 0:
                continue
            at = list(range(max(c, 0))) + [c + j for j in line if c + j >= 0]
            x = q[a + i:a + i + 1].astype(np.float64)
            x = (turn(x, np.maximum(pos[a + i:a + i + 1], 0)) if turn else x)[0]
            s = np.einsum("hd,thd->ht", x, np.repeat(K[at], g, axis=1)) * scale
            w = np.exp(s - s.max(axis=1, keepdims=True))
            w /= w.sum(axis=1, keepdims=True)
            out[a + i] = np.einsum("ht,thd->hd", w, np.repeat(V[at], g, axis=1))
    return out


def verify(parents, tokens, target, u_accept, u_next, draft=None):
    """One sequence's walk in exact rational arithmetic: (path, next token); target, draft [T, vocab]."""
    F = np.frompyfunc(lambda x: Fraction(float(x)), 1, 1)
    at, path, T = 0, [0], len(parents)
    while True:
        r, Z, taken = F(target[at]), Fraction(1), None
        q = None if draft is None else F(draft[at])
        for c in [i for i in range(at + 1, T) if parents[i] == at]:
            x = int(tokens[c])
            if not 0 <= x < len(r):
                continue
            u = Fraction(float(u_accept[c]))
            if u * Z * (1 if q is None else q[x]) < r[x]:
                taken = c
                break
            if q is None:
                Z -= r[x]
                r[x] = Fraction(0)
            else:
                rest = np.maximum(r - Z * q, Fraction(0))
                if rest.sum() > 0:
                    r, Z = rest, rest.sum()
        if taken is None:
            break
        at = taken
        path.append(at)
    total, t = Fraction(0), Fraction(float(u_next)) * r.sum()
    for w, x in enumerate(r):
        total += x
        if total > t:
            return path, w
    return path, -1


ONE = 1 << 62


def fixed(p):
    """Probabilities in whole multiples of 2^-62, rounded down: Python ints; what is no number in [0, 1] as 0 or 1."""
    x = np.nan_to_num(np.asarray(p, np.float64), nan=0.0, posinf=1.0, neginf=0.0)
    return np.floor(np.clip(x, 0.0, 1.0) * 2.0 ** 62).astype(np.uint64).astype(object)


def verify_fixed(parents, tokens, target, u_accept, u_next, draft=None):
    """The walk as the kernel's numbers make it: weights and Z in multiples of 2^-62 (Z q rounded down to one),
    random numbers in multiples of 2^-64."""
    def random(u):
        u = min(max(float(u), 0.0), 1.0 - 2.0 ** -24) if u == u else 0.0
        return int(u * 2.0 ** 64)

    at, path, T = 0, [0], len(parents)
    while True:
        r, Z, taken = fixed(target[at]), ONE, None
        q = None if draft is None else fixed(draft[at])
        for c in [i for i in range(at + 1, T) if parents[i] == at]:
            x = int(tokens[c])
            if not 0 <= x < len(r):
                continue
            if (random(u_accept[c]) * (Z if q is None else Z * q[x] >> 62)) >> 64 < r[x]:
                taken = c
                break
            if q is None:
                Z, r[x] = max(Z - r[x], 0), 0
            else:
                rest = np.maximum(r - (Z * q >> 62), 0)
                if rest.sum() > 0:
                    r, Z = rest, min(rest.sum(), 2 * ONE - 1)
        if taken is None:
            break
        at = taken
        path.append(at)
    t = (r.sum() * random(u_next)) >> 64
    over = np.flatnonzero(np.cumsum(r) > t)
    return path, int(over[0]) if len(over) else -1


def keep(pages, table, seq_lens, cu_q, paths):
    """The pages (a copy) with every sequence's path moved to the front of its nodes' slots, and the new
    lengths."""
    P, out, lens = pages.shape[2], pages.copy(), []
    for b, n in enumerate(seq_lens):
        T = int(cu_q[b + 1] - cu_q[b])
        c = int(n) - T
        for j, at in enumerate(paths[b] if T else []):
            if c + j >= 0:
                s, d = c + at, c + j
                out[table[b, d // P], :, d % P] = pages[table[b, s // P], :, s % P]
        lens.append(max(c + len(paths[b]), 0) if T else int(n))
    return out, lens
