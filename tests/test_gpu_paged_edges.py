"""Paged calls at the ends of their contract: keys and values of extreme norms, scores without a
maximum, pairs of small differences, a batch without max_q."""

import numpy as np
import pytest

from gpu_util import RTOL, lib
from oracle import paged
from oracle.formats import unpack_turbo4
from test_gpu_paged import Setup, check_attention, device_rows, dt, run_attention, set_norms

pytestmark = pytest.mark.gpu

# lens, new, Hq, Hkv, P, output type; the position whose value has (almost) no norm: behind the first key
# block of its warp, and behind its CTA's first tile of keys
DOMINANT = [
    ([32] * 6, [1] * 6, 6, 1, 16, "f32", 8),
    ([500] * 170, [1] * 170, 4, 1, 32, "bf16", 300),
    ([500] * 170, [1] * 170, 3, 1, 64, "f16", 247),
    ([32] * 6, [2] * 6, 6, 1, 16, "bf16", 8),
    ([500] * 40, [2] * 40, 16, 1, 32, "bf16", 300),
    ([500] * 40, [20] * 40, 8, 1, 32, "bf16", 300),
    ([500] * 40, [2] * 40, 4, 1, 32, "f16", 300),
]


@pytest.mark.parametrize("norm", [0.0, 2.0 ** -80])
@pytest.mark.parametrize("case", DOMINANT, ids=lambda c: f"{c[5]}-t{max(c[1])}-g{c[2] // c[3]}-n{max(c[0])}")
def test_a_value_of_no_norm_that_takes_all_the_weight(case, norm):
    """One key of norm 4000 moves its score by some 350 z nats (z normal); its value is (almost) zero.  A row
    where it leads by 60 nats is at most n exp(-60) of the largest value, one where it trails by 60 does
    not feel it, and a score's own error is 7e-5 (one part: 1e-3) of |q| |k| / sqrt(128) ~ 4000, below 8 nats."""
    lens, new, Hq, Hkv, P, out_dtype, at = case
    tq = lib()
    s = Setup(tq, lens, new, Hkv, P, 83, ("dense", "wht"), ragged=max(new) > 1)
    some = range(0, len(lens), max(1, len(lens) // 12))
    for b in some:
        set_norms(s, 0, {(b, 0, at): 4000.0})
        set_norms(s, 1, {(b, 0, at): norm})
    got, ref = run_attention(s, Hq, "f32", out_dtype)
    got32 = got.float().cpu().numpy().astype(np.float64)
    assert np.all(np.isfinite(got32[:s.n]))
    led, trailed = [], []
    for b in some:
        K = paged.dequantize(s.codec[0], paged.sequence_rows(s.host[0], s.table, b, lens[b]))[:, 0]
        for i in range(s.cu[b], s.cu[b + 1]):
            n = lens[b] - (s.cu[b + 1] - i) + 1
            x = s.q32[i].astype(np.float64) @ K[:n].T / np.sqrt(128)
            lead = x[:, at] - np.delete(x, at, axis=1).max(axis=1)
            led += [(i, h) for h in np.nonzero(lead >= 60)[0]]
            trailed += [(i, h) for h in np.nonzero(lead <= -60)[0]]
    assert len(led) >= 10 and len(trailed) >= 10
    V = [paged.dequantize(s.codec[1], paged.sequence_rows(s.host[1], s.table, b, lens[b])) for b in some]
    big = max(np.abs(v).max() for v in V)
    for i, h in led:
        assert np.abs(got32[i, h]).max() <= max(lens) * np.exp(-52) * big
    keep = np.zeros(got32.shape[:2], bool)
    for i, h in trailed:
        keep[i, h] = True
    for b in range(len(lens)):
        if b not in some:
            keep[s.cu[b]:s.cu[b + 1]] = True
    import torch
    ref[~keep] = 0
    check_attention(torch.from_numpy(np.where(keep[..., None], got32, 0)), ref, out_dtype)


NO_MAXIMUM = [  # lens, new, Hq, Hkv, P, output type
    ([130, 40], [2, 2], 8, 2, 16, "bf16"),
    ([130, 40], [2, 2], 8, 2, 16, "f16"),
    ([130, 70], [2, 70], 8, 1, 16, "bf16"),
    ([130, 40], [1, 1], 8, 2, 16, "bf16"),
    ([260, 40], [1, 1], 12, 2, 64, "f32"),
]


@pytest.mark.parametrize("case", NO_MAXIMUM, ids=lambda c: f"{c[5]}-t{max(c[1])}-g{c[2] // c[3]}")
def test_scores_that_are_all_nan_reach_the_row(case):
    """A last tile of keys whose norms are all NaN, and a row of q that is NaN: the rows that see them are not
    finite, the others are as if they were not there."""
    import torch
    lens, new, Hq, Hkv, P, out_dtype = case
    tq = lib()
    s = Setup(tq, lens, new, Hkv, P, 89, ("wht", "dense"), ragged=max(new) > 1)
    first = lens[0] - 2 if max(new) > 1 else lens[0] - 1  # NaN from here on, for the last KV head
    set_norms(s, 0, {(0, Hkv - 1, t): np.nan for t in range(first, lens[0])})
    q, q32 = device_rows(s.rng.standard_normal((s.n_rows, Hq, 128)), "f32")
    last = s.n - 1
    q[last, 1, 5] = float("nan")
    out = torch.full((s.n_rows, Hq, 128), 7.0, dtype=dt(out_dtype), device="cuda")
    tq.tq_paged_attention(*s.ctx, s.kv, s.batch, q, out, s.workspace(Hq))
    assert s.status() == 0
    ref = s.oracle(q32)
    bad = np.zeros((s.n_rows, Hq), bool)
    for i in range(s.cu[0], s.cu[1]):
        if lens[0] - (s.cu[1] - i) >= first:
            bad[i, Hq - Hq // Hkv:] = True
    bad[last, 1] = True
    got = out.float().cpu().numpy()
    assert bad.sum() > 1 and not np.isfinite(got[bad]).any()
    ref[bad] = 0
    check_attention(torch.from_numpy(np.where(bad[..., None], 0, got)), ref, out_dtype)


BIG = [  # lens, new, Hq, Hkv, P, output type
    ([600, 40], [1, 1], 4, 2, 16, "f32"),
    ([600, 40], [1, 1], 12, 2, 64, "f32"),
    ([600, 40], [3, 40], 4, 2, 16, "f32"),
    ([600, 40], [3, 3], 32, 2, 32, "bf16"),
    ([600, 300], [20, 200], 16, 2, 32, "bf16"),
]


@pytest.mark.parametrize("case", BIG, ids=lambda c: f"{c[5]}-t{max(c[1])}-g{c[2] // c[3]}")
def test_value_norms_up_to_the_limit(case):
    """Values of norms 2^126 and 2^127 everywhere (bf16 chunks: 2^118 and 2^119): the usual relative bound.  A norm
    that is not finite (there: 2^120) makes the rows that see it not finite, and no others."""
    import torch
    lens, new, Hq, Hkv, P, out_dtype = case
    tq = lib()
    s = Setup(tq, lens, new, Hkv, P, 97, ("dense", "wht"), ragged=max(new) > 1)
    top = 119 if out_dtype == "bf16" else 127
    set_norms(s, 1, {(b, h, t): 2.0 ** (top - t % 2) for b, n in enumerate(lens) for h in range(Hkv) for t in range(n)})
    got, ref = run_attention(s, Hq, "bf16", out_dtype)
    small = 2.0 ** (1 - top)
    got = got.float().cpu().numpy().astype(np.float64) * small
    check_attention(torch.from_numpy(got), ref * small, out_dtype)
    spots = [(0, 1, 577), (1, 0, 38)]
    set_norms(s, 1, {x: 2.0 ** 120 if out_dtype == "bf16" else np.inf for x in spots})
    got, ref = run_attention(s, Hq, "bf16", out_dtype)
    got = got.float().cpu().numpy().astype(np.float64)
    bad = np.zeros((s.n_rows, Hq), bool)
    g = Hq // Hkv
    for b, h, pos in spots:
        for i in range(s.cu[b], s.cu[b + 1]):
            if lens[b] - (s.cu[b + 1] - i) >= pos:
                bad[i, h * g:(h + 1) * g] = True
    assert bad.any() and not np.isfinite(got[bad]).any()
    ref[bad] = 0
    check_attention(torch.from_numpy(np.where(bad[..., None], 0, got * small)), ref * small, out_dtype)


@pytest.mark.parametrize("case", [([700], [1], 4, 1, 16, "f32"), ([700], [1], 8, 1, 16, "f32"),
                                  ([700, 90], [3, 3], 4, 1, 16, "f32"), ([700, 90], [3, 3], 16, 1, 16, "bf16"),
                                  ([700, 90], [40, 60], 8, 1, 16, "bf16")],
                         ids=lambda c: f"{c[5]}-t{max(c[1])}-g{c[2] // c[3]}")
def test_weights_beside_values_of_the_largest_norm(case):
    """A few values of norm 2^64 (the largest that the encode writes), the others zero: every key still counts in
    the weights.  The large ones lie in three blocks of 32 keys, so that some warps, halves and tiles hold
    zeros alone.  Outputs are a share of the large values; the usual relative bound."""
    import torch
    lens, new, Hq, Hkv, P, out_dtype = case
    tq = lib()
    s = Setup(tq, lens, new, Hkv, P, 101, ("wht", "wht"), ragged=max(new) > 1)
    set_norms(s, 1, {(b, 0, t): 1.8e19 if t // 32 % 7 == 3 and t % 3 == 0 else 0.0
                     for b, n in enumerate(lens) for t in range(n)})
    got, ref = run_attention(s, Hq, "bf16", out_dtype)
    scale = 2.0 ** -64
    back = torch.from_numpy(got.float().cpu().numpy().astype(np.float64) * scale)
    check_attention(back, ref * scale, out_dtype)


@pytest.mark.parametrize("case", [([40, 9], [1, 1], 4), ([40, 9], [2, 9], 4), ([2000], [1], 4), ([2000], [3], 4)],
                         ids=lambda c: f"t{max(c[1])}-n{max(c[0])}")
def test_differential_norm_of_small_pairs(case):
    """eps = 0 and lambda = 0: the row over its rms, 1.5 in rms whatever the values' norms while their squares are
    fp32's (2^-45), and finite, no larger, where they are not (2^-70, 2^-72, where the mean's square root
    would be that of zero).  The relative bound of a row counts twice: for the row and for its norm."""
    import torch
    lens, new, Hq = case
    tq = lib()
    s = Setup(tq, lens, new, 1, 16, 103, ("wht", "dense"), ragged=max(new) > 1)
    mix = tq.DiffMix(torch.zeros(Hq // 2, device="cuda"), torch.ones(128, device="cuda"), eps=0.0, out_scale=1.5)
    q, q32 = device_rows(s.rng.standard_normal((s.n_rows, Hq, 128)), "f32")
    for e in (-45, -70, -72):
        set_norms(s, 1, {(b, 0, t): 2.0 ** e for b, n in enumerate(lens) for t in range(n)})
        out = torch.full((s.n_rows, Hq // 2, 128), 7.0, device="cuda")
        tq.tq_paged_diff_attention(*s.ctx, s.kv, s.batch, q, mix, out, s.workspace(Hq))
        assert s.status() == 0
        got = out.cpu().numpy().astype(np.float64)
        assert np.all(np.isfinite(got))
        ref = paged.differential(s.oracle(q32), np.zeros(Hq // 2), np.ones(128), 0.0, 1.5)
        err, size = np.linalg.norm(got - ref, axis=-1), np.linalg.norm(ref, axis=-1)
        if e == -45:
            assert np.all(err <= 2 * RTOL * size)
        assert np.all(np.linalg.norm(got, axis=-1) <= (1 + 2 * RTOL) * size)


def test_offsets_without_the_most_rows():
    """max_q left out: every row of a ragged batch is computed."""
    tq = lib()
    s = Setup(tq, [70, 9, 30], [5, 9, 1], 2, 16, 107)
    s.batch = tq.PagedBatch(s.d_lens, s.batch.cu_q, n_tokens=s.n_rows)
    got, ref = run_attention(s, 8, "bf16", "f32")
    check_attention(got, ref, "f32")


def one_part(s, b, q32, Hq):
    """Sequence b's rows in fp64: by the formula, and with q, the keys, the probabilities, the values, the
    quotient and R each rounded once to fp16, in the kernel's units (the centroids times the alpha that
    makes their fp16 table's error smallest, q times log2(e) / (sqrt(128) alpha))."""
    f16 = lambda x: x.astype(np.float16).astype(np.float64)  # noqa: E731
    n, lo, hi = s.lens[b], int(s.cu[b]), int(s.cu[b + 1])
    g, pos = Hq // s.Hkv, n - (hi - lo) + np.arange(hi - lo)
    table, alpha, norms = [], [], []
    for c, h in zip(s.codec, s.host):
        mag = np.abs(c.c32[:8]).astype(np.float64)
        a = 1 + np.arange(65536) / 65536
        v = a[:, None] * mag
        alpha.append(a[(np.abs(v.astype(np.float32).astype(np.float16) - v) / v).max(1).argmin()])
        norm, idx = unpack_turbo4(paged.sequence_rows(h, s.table, b, n).reshape(-1, 68))
        table.append(c.c32.astype(np.float64)[idx].reshape(n, s.Hkv, 128))
        norms.append(norm.astype(np.float64).reshape(n, s.Hkv, 1))
    ref, em = np.empty((2, hi - lo, Hq, 128))
    seen = np.arange(n) <= pos[:, None]
    for h in range(Hq):
        q = q32[lo:hi, h].astype(np.float64) @ s.codec[0].rot.R.T
        K, V = (norms[i][:, h // g] * table[i][:, h // g] for i in range(2))
        x = np.where(seen, q @ K.T / np.sqrt(128), -np.inf)
        w = np.exp(x - x.max(1, keepdims=True))
        ref[:, h] = w @ V / w.sum(1, keepdims=True) @ s.codec[1].rot.R
        K1, V1 = (f16(norms[i][:, h // g] * 2.0 ** 8 * f16(alpha[i] * table[i][:, h // g])) * 2.0 ** -8 for i in range(2))
        x = np.where(seen, f16(q * (1 / np.log(2) / np.sqrt(128) / alpha[0])) @ K1.T, -np.inf)
        p = 2.0 ** (x - x.max(1, keepdims=True) + 7)
        o = f16(p) @ V1 / p.sum(1, keepdims=True) / alpha[1]
        up = 2.0 ** (13 - np.floor(np.log2(np.abs(o).max(1, keepdims=True))))
        em[:, h] = f16(o * up) / up @ f16(s.codec[1].rot.R)
    return ref, em


@pytest.mark.parametrize("rot", ["wht", "dense"])
@pytest.mark.parametrize("n", [300, 6000])
def test_bf16_chunks_add_what_their_operands_round(rot, n):
    """What a bf16 chunk is off beyond the rounding of its output, in rms over all elements: the rounding of the
    formula's own values is independent of the rest, so the squares subtract.  The rest is that of the six
    operands' roundings (two of them, of other draws than the emulation's, and 1.5% of noise in the
    difference: 10%), and below 1e-3 of the rows' norm."""
    tq = lib()
    s = Setup(tq, [n, 150], [128, 100], 2, 64, 109, (rot, rot))
    import torch
    q, q32 = device_rows(s.rng.standard_normal((s.n_rows, 8, 128)), "bf16")
    out = torch.zeros((s.n_rows, 8, 128), dtype=torch.bfloat16, device="cuda")
    tq.tq_paged_attention(*s.ctx, s.kv, s.batch, q, out, s.workspace(8))
    assert s.status() == 0
    ref, em = (np.concatenate(x) for x in zip(*(one_part(s, b, q32, 8) for b in range(2))))
    nearest = torch.from_numpy(ref).to(torch.bfloat16).double().numpy()
    got = out.float().cpu().numpy().astype(np.float64)
    square = lambda x: float((x * x).sum())  # noqa: E731
    for rows in (slice(0, 128), slice(128, 228)):
        size = square(ref[rows])
        rest = np.sqrt(max(square((got - ref)[rows]) - square((nearest - ref)[rows]), 0) / size)
        emulated = np.sqrt(square((em - ref)[rows]) / size)
        print(f"{rot} {n}: {rest:.3e}, emulated {emulated:.3e}")
        assert rest <= 1.1 * emulated and rest <= 1e-3
