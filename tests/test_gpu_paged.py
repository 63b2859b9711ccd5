"""Paged cache on the GPU (append, gather, attention, differential attention) against the fp64
oracle, its refusals and device flags, and runs of the calls together."""

import ctypes

import numpy as np
import pytest

import synth
from gpu_util import ATOL, BAND, RTOL, band_ok, lib
from oracle import paged
from oracle.formats import Codec, unpack_turbo4

pytestmark = pytest.mark.gpu

HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}  # half a step, relative


def dt(name):
    import torch
    return {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}[name]


def device_rows(x32, dtype):
    """fp32 numpy -> CUDA tensor of dtype, and the exact fp32 values it holds."""
    import torch
    t = torch.from_numpy(np.ascontiguousarray(x32, np.float32)).to(dt(dtype))
    return t.cuda(), t.float().numpy()


class Setup:
    """Random pages for a ragged batch.  Records of tokens no sequence holds are all ones (NaN
    norms), so that a read past a sequence's end shows."""

    def __init__(self, tq, lens, new, Hkv, P, seed, rot=("wht", "wht"), pad=0, ragged=True, codebook=None, fill=True,
                 width=None):
        import torch
        rng = np.random.default_rng(seed)
        self.tq, self.rng, self.lens, self.Hkv, self.P = tq, rng, list(lens), Hkv, P
        self.cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        self.n, self.n_rows = int(self.cu[-1]), int(self.cu[-1]) + pad
        pages = [(n + P - 1) // P for n in lens]
        self.n_pages = sum(pages) + 3
        order = rng.permutation(self.n_pages)
        self.table = np.full((len(lens), width or max(max(pages), 1)), -7, np.int32)
        at = 0
        for b, k in enumerate(pages):
            self.table[b, :k] = order[at:at + k]
            at += k
        self.codec = [Codec("turbo4", rotation=r, rot_seed=31 + i, codebook=codebook) for i, r in enumerate(rot)]
        self.ctx = [tq.Ctx("turbo4", r, 31 + i, codebook=codebook) for i, r in enumerate(rot)]
        self.host = []
        for c in self.codec:
            buf = np.full((self.n_pages, Hkv, P, 68), 255, np.uint8)
            for b, n in enumerate(lens if fill else []):
                rows, _ = c.encode((rng.standard_normal((n * Hkv, 128)) * rng.lognormal(0, 0.3, (n * Hkv, 1))).astype(np.float32)) \
                    if n else (np.zeros((0, 68), np.uint8), None)
                t = np.arange(n)
                if n:
                    buf[self.table[b, t // P], :, t % P] = rows.reshape(n, Hkv, 68)
            self.host.append(buf)
        self.pages = [torch.from_numpy(h.copy()).cuda() for h in self.host]
        self.kv = tq.PagedKV(self.pages[0], self.pages[1], torch.from_numpy(self.table).cuda(), P, Hkv)
        self.d_lens = torch.tensor(self.lens, dtype=torch.int32, device="cuda")
        if ragged:
            self.batch = tq.PagedBatch(self.d_lens, torch.from_numpy(self.cu).cuda(), max(max(new), 1), self.n_rows)
        else:
            self.batch = tq.PagedBatch(self.d_lens)

    def status(self):
        import torch
        torch.cuda.synchronize()
        return self.tq.tq_ctx_device_status(self.ctx[0])

    def rope(self, rot_dim, interleaved, n_pos=None):
        import torch
        if not rot_dim:
            return None, None
        c, s = self.tq.tq_make_rope_table(rot_dim, n_pos or max(max(self.lens), 1))
        r = self.tq.Rope(torch.from_numpy(c).cuda(), torch.from_numpy(s).cuda(), interleaved)
        return r, lambda x, pos: paged.rope(x, c, s, pos, interleaved)

    def workspace(self, Hq):
        import torch
        n = self.tq.tq_paged_workspace_size(*self.ctx, self.kv, self.batch, Hq)
        return torch.full((max(n, 256),), 255, dtype=torch.uint8, device="cuda")  # no initialisation needed

    def oracle(self, q32, turn=None, scale=0.0):
        return paged.attention(*self.codec, *self.host, self.table, self.lens, self.cu, q32, self.n_rows, scale, turn)


def check_attention(got, ref, dtype, what=""):
    """Rows of no sequence untouched (the caller filled them with 7); the others within the documented
    2e-3 / 1e-3 before the rounding to dtype, which adds half a step."""
    got = got.float().cpu().numpy().astype(np.float64)
    out = np.isnan(ref).all(axis=(1, 2))
    assert np.all(got[out] == 7.0), f"{what}: padded rows written"
    got, ref = got[~out], ref[~out]
    assert np.all(np.isfinite(got)), f"{what}: not finite"
    assert np.max(np.abs(got - ref) - HALF[dtype] * np.abs(ref), initial=0) <= ATOL, what
    num = np.linalg.norm(got - ref, axis=-1) - HALF[dtype] * np.linalg.norm(ref, axis=-1)
    assert np.max(num - RTOL * np.linalg.norm(ref, axis=-1), initial=0) <= 1e-30, what


def centroid_error(codec):
    """Largest relative error of the fp16 centroid table: the centroids times the alpha in [1, 2) (65536
    steps) that makes it smallest."""
    mag = np.abs(codec.c32[:8]).astype(np.float64)
    v = (1 + np.arange(65536) / 65536)[:, None] * mag
    return (np.abs(v.astype(np.float32).astype(np.float16) - v) / v).max(1).min()


def check_sharp(s, got, ref, q32, scale, what):
    """Large scores: with every product q_i k_i off by the centroid table's error e (q in two fp16 parts,
    2^-22, and the sums are far below it) a score is off by at most d = (e + 2^-20) |scale| |q| max|k|;
    the weights then move by factors in [exp(-2d), exp(2d)], so the output, a mean of the values, by at
    most (exp(2d) - 1) (max|v| + |out|) an element, on top of the documented 2e-3."""
    got = got.float().cpu().numpy().astype(np.float64)
    assert np.all(np.isfinite(got)), what
    for b, n in enumerate(s.lens):
        rows = slice(int(s.cu[b]), int(s.cu[b + 1]))
        K, V = (paged.dequantize(c, paged.sequence_rows(h, s.table, b, n)) for c, h in zip(s.codec, s.host))
        d = (centroid_error(s.codec[0]) + 2.0 ** -20) * abs(scale) * np.linalg.norm(K, axis=-1).max() \
            * np.linalg.norm(q32[rows], axis=-1, keepdims=True)
        tol = ATOL + np.expm1(2 * d) * (np.abs(V).max() + np.abs(ref[rows]))
        assert np.max(np.abs(got[rows] - ref[rows]) - tol) <= 0, what


def run_attention(s, Hq, dtype, out_dtype, rot_dim=0, interleaved=False, strided=False, scale=0.0):
    import torch
    x = s.rng.standard_normal((s.n_rows, 3 * Hq if strided else Hq, 128))
    t, x32 = device_rows(x, dtype)
    q, q32 = (t[:, Hq:2 * Hq], x32[:, Hq:2 * Hq]) if strided else (t, x32)
    rope, turn = s.rope(rot_dim, interleaved)
    out = torch.full((s.n_rows, Hq, 128), 7.0, dtype=dt(out_dtype), device="cuda")
    s.tq.tq_paged_attention(*s.ctx, s.kv, s.batch, q, out, s.workspace(Hq), rope=rope, scale=scale)
    assert s.status() == 0
    s.q32 = q32
    return out, s.oracle(q32, turn, scale)


# ------------------------------------------------------------------------------ append

APPEND = [
    # lens, new, Hkv, P, dtype, rot_dim, interleaved, pad, strided
    ([5], [5], 1, 16, "f32", 0, False, 0, False),
    ([1, 700, 64], [1, 1, 1], 8, 64, "bf16", 128, False, 0, True),
    ([33, 17, 0, 250], [33, 2, 0, 130], 3, 16, "f16", 64, True, 5, False),
    ([40, 3, 129], [7, 5, 129], 2, 32, "bf16", 64, False, 1, True),  # a sequence shorter than its rows
    ([300], [300], 4, 256, "f32", 32, False, 0, False),
    ([90, 1], [90, 1], 5, 128, "f16", 128, True, 0, True),
    ([257, 31], [200, 31], 1, 16, "bf16", 32, True, 64, False),
]


@pytest.mark.parametrize("case", APPEND, ids=lambda c: f"{c[4]}-p{c[3]}-r{c[5]}{'i' if c[6] else ''}-h{c[2]}")
@pytest.mark.parametrize("rot", [("wht", "wht"), ("dense", "dense"), ("wht", "dense")], ids="/".join)
def test_append_writes_the_oracles_records(case, rot):
    tq = lib()
    lens, new, Hkv, P, dtype, rot_dim, inter, pad, strided = case
    s = Setup(tq, lens, new, Hkv, P, 1, rot, pad, fill=False)
    wide = 3 * Hkv if strided else Hkv
    t, x32 = device_rows(s.rng.standard_normal((s.n_rows, wide, 128)) * 3, dtype)
    u, y32 = device_rows(s.rng.standard_normal((s.n_rows, wide, 128)), dtype)
    u[s.n // 2], y32[s.n // 2] = 0, 0  # a zero row
    k, k32 = (t[:, Hkv:2 * Hkv], x32[:, Hkv:2 * Hkv]) if strided else (t, x32)
    v, v32 = (u[:, :Hkv], y32[:, :Hkv]) if strided else (u, y32)
    rope, turn = s.rope(rot_dim, inter)
    tq.tq_paged_append(*s.ctx, s.kv, s.batch, k, v, rope=rope)
    assert s.status() == 0
    at, _ = paged.places(lens, s.cu)
    rows, seq, pos = (np.array(c, int) for c in zip(*at))
    k32 = turn(k32[rows], pos) if turn else k32[rows]
    for i, x in enumerate((k32, v32[rows])):
        rec, info = s.codec[i].encode(np.ascontiguousarray(x.reshape(-1, 128), np.float32))
        want = s.host[i].copy()
        want[s.table[seq, pos // P], :, pos % P] = rec.reshape(len(rows), Hkv, 68)
        got = s.pages[i].cpu().numpy()
        if rot[i] == "wht":
            assert np.array_equal(got, want)
            continue
        mine = got[s.table[seq, pos // P], :, pos % P].reshape(-1, 68)
        touched = np.zeros(want.shape[:3], bool)
        touched[s.table[seq, pos // P], :, pos % P] = True
        assert np.array_equal(got[~touched], want[~touched])
        n1, idx1 = unpack_turbo4(mine)
        n0, idx0 = unpack_turbo4(rec)
        assert np.array_equal(n1, n0)
        ok, n_diff = band_ok(idx1, idx0, info["y"], s.codec[i].b32, BAND)
        assert ok, n_diff


APPEND_MANY = [  # dense rotations in 16-row tiles: above 16 rows per SM
    ([900, 0, 333], [900, 0, 20], 4, 64, "bf16", 128, False, 3, True),
    ([611, 77, 64], [600, 50, 64], 5, 16, "f16", 64, True, 0, False),
    ([2600], [2590], 1, 32, "f32", 32, False, 11, False),
    ([130, 170, 90, 1, 300], [130, 170, 90, 1, 300], 8, 128, "f32", 0, False, 0, True),
]


@pytest.mark.parametrize("case", APPEND_MANY, ids=lambda c: f"{c[4]}-p{c[3]}-r{c[5]}{'i' if c[6] else ''}-h{c[2]}")
@pytest.mark.parametrize("rot", [("dense", "dense"), ("dense", "wht")], ids="/".join)
def test_append_of_many_dense_rows(case, rot):
    test_append_writes_the_oracles_records(case, rot)


def test_append_of_many_dense_rows_at_the_ends_of_the_range():
    """Norms down to fp32's smallest, rows of zeros, and non-finite rows, in the tiles of other rows."""
    tq = lib()
    s = Setup(tq, [400], [400], 8, 16, 5, ("dense", "dense"), fill=False)
    x = s.rng.standard_normal((400, 8, 128))
    x[5:90] *= 2.0 ** -s.rng.integers(90, 130, (85, 8, 1))
    x[100] = 0
    x[110, 3, 1:] = 0
    x[110, 3, 0] = 2.0 ** -149
    k, k32 = device_rows(x, "f32")
    bad = np.zeros((400, 8), bool)
    for i, h, value in ((200, 0, np.nan), (201, 7, np.inf), (202, 3, -np.inf)):
        k[i, h, 9], bad[i, h] = float(value), True
    tq.tq_paged_append(*s.ctx, s.kv, s.batch, k, k)
    assert s.status() == 0
    for i in range(2):
        rec, info = s.codec[i].encode(np.ascontiguousarray(k32.reshape(-1, 128), np.float32))
        got = s.pages[i].cpu().numpy()[s.table[0, :25]].transpose(0, 2, 1, 3).reshape(-1, 68)
        n1, idx1 = unpack_turbo4(got)
        n0, idx0 = unpack_turbo4(rec)
        ok = ~bad.reshape(-1)
        assert np.array_equal(n1[ok], n0[ok])
        fine, n_diff = band_ok(idx1[ok], idx0[ok], info["y"].reshape(-1, 128)[ok], s.codec[i].b32, BAND)
        assert fine, n_diff


def test_append_equals_set_rows_through_slots():
    """Without a rotation the call is tq_quantize_set_rows at the pages' row slots."""
    import torch
    tq = lib()
    s = Setup(tq, [100, 37, 260], [100, 1, 60], 4, 32, 5, fill=False)
    k = torch.randn((s.n_rows, 4, 128), device="cuda").bfloat16()
    v = torch.randn((s.n_rows, 4, 128), device="cuda").bfloat16()
    tq.tq_paged_append(*s.ctx, s.kv, s.batch, k, v)
    assert s.status() == 0
    at, _ = paged.places(s.lens, s.cu)
    rows, seq, pos = (np.array(c, int) for c in zip(*at))
    slot = (s.table[seq, pos // 32][:, None] * 4 + np.arange(4)) * 32 + (pos % 32)[:, None]
    ids = torch.from_numpy(slot.reshape(-1).astype(np.int64)).cuda()
    for i, x in enumerate((k, v)):
        other = torch.from_numpy(s.host[i].copy()).cuda()
        tq.tq_quantize_set_rows(s.ctx[i], x[rows].reshape(-1, 128), other, row_ids=ids)
        torch.cuda.synchronize()
        assert torch.equal(other, s.pages[i])


def test_append_non_finite_rows_keep_to_themselves():
    """NaN and infinite rows give records the contract leaves open, and touch no other record."""
    tq = lib()
    s = Setup(tq, [9], [9], 2, 16, 5, fill=False)
    k, k32 = device_rows(s.rng.standard_normal((9, 2, 128)), "f32")
    k[3, 1, 5], k[6, 0, 99] = float("nan"), float("inf")
    tq.tq_paged_append(*s.ctx, s.kv, s.batch, k, k)
    rec = s.codec[0].encode(k32.reshape(-1, 128))[0].reshape(9, 2, 68)
    got = s.pages[0].cpu().numpy()[s.table[0, 0], :, :9].transpose(1, 0, 2)
    same = (got == rec).all(-1)
    bad = np.zeros((9, 2), bool)
    bad[3, 1] = bad[6, 0] = True
    assert np.array_equal(same | bad, np.ones_like(same)) and not same[3, 1]


# ------------------------------------------------------------------------------ gather

@pytest.mark.parametrize("rot", ["wht", "dense"])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("shape", [([40], 1, 16), ([3, 0, 300, 129], 3, 64), ([513, 17], 8, 128)],
                         ids=["one", "ragged", "heads8"])
def test_gather_reconstructs(rot, dtype, shape):
    """fp32: a sum of 128 products in any order is off by at most 130 * 2^-24 n sum|R c| <= 130 * 2^-24 n |c|
    (Cauchy-Schwarz, unit rows of R); twice that allows the norm and parts of operands.  16-bit
    outputs: each operand may be held in fp16 (half a step 2^-11 each), plus half a step."""
    import torch
    tq = lib()
    lens, Hkv, P = shape
    s = Setup(tq, lens, lens, Hkv, P, 7, (rot, rot), pad=3)
    for unrotate in (True, False):
        outs = [torch.full((s.n_rows, Hkv, 128), 7.0, dtype=dt(dtype), device="cuda") for _ in range(2)]
        tq.tq_paged_gather(*s.ctx, s.kv, s.batch, *outs, unrotate=unrotate)
        assert s.status() == 0
        for i in range(2):
            got = outs[i].float().cpu().numpy().astype(np.float64)
            assert np.all(got[s.n:] == 7.0)
            for b, n in enumerate(lens):
                rows = paged.sequence_rows(s.host[i], s.table, b, n)
                ref = paged.dequantize(s.codec[i], rows, unrotate)
                norm = np.linalg.norm(ref, axis=-1, keepdims=True)
                tol = norm * (260 * 2.0 ** -24 if dtype == "f32" else 2.0 ** -10) + HALF[dtype] * np.abs(ref)
                assert np.max(np.abs(got[s.cu[b]:s.cu[b + 1]] - ref) - tol, initial=0) <= 0


def test_gather_one_side_and_rows_without_a_place():
    import torch
    tq = lib()
    s = Setup(tq, [2, 20], [3, 4], 2, 16, 8)
    both = [torch.full((7, 2, 128), 7.0, device="cuda") for _ in range(2)]
    tq.tq_paged_gather(*s.ctx, s.kv, s.batch, *both)
    for i in range(2):
        one = torch.full((7, 2, 128), 7.0, device="cuda")
        tq.tq_paged_gather(*s.ctx, s.kv, s.batch, *((one, None) if i == 0 else (None, one)))
        assert s.status() == 0
        assert torch.equal(one, both[i]) and torch.all(one[0] == 0) and torch.all(one[1] != 0)


# ------------------------------------------------------------------------------ attention, single rows

SINGLE = [
    # lens, Hq, Hkv, P, dtype, out, rot_dim, interleaved, strided, rot
    ([1], 4, 1, 16, "bf16", "bf16", 128, False, False, ("wht", "wht")),
    ([15, 16, 17, 0, 33], 8, 2, 16, "f16", "f16", 64, True, True, ("dense", "dense")),
    ([240, 241, 479, 481], 4, 4, 32, "f32", "f32", 0, False, False, ("wht", "dense")),
    ([1000, 3, 0, 640], 12, 2, 64, "bf16", "f32", 32, False, True, ("dense", "wht")),
    ([129, 700], 24, 2, 128, "f16", "f16", 128, True, False, ("wht", "wht")),
    ([300, 511], 16, 1, 256, "bf16", "bf16", 128, False, False, ("dense", "dense")),
    ([257], 3, 1, 16, "f32", "bf16", 0, False, False, ("wht", "wht")),
    ([2500, 1, 77], 32, 8, 64, "bf16", "bf16", 128, False, True, ("dense", "dense")),
    ([700], 10, 2, 16, "bf16", "f16", 64, False, False, ("wht", "wht")),
    ([90] * 40, 2, 1, 32, "bf16", "bf16", 0, False, False, ("wht", "wht")),
    ([450, 20], 64, 1, 32, "f16", "f32", 0, False, False, ("dense", "wht")),
]


@pytest.mark.parametrize("ragged", [False, True], ids=["rows", "cu"])
@pytest.mark.parametrize("case", SINGLE, ids=lambda c: f"g{c[1] // c[2]}-p{c[3]}-{c[4]}-{len(c[0])}x{max(c[0])}")
def test_single_rows(case, ragged):
    tq = lib()
    lens, Hq, Hkv, P, dtype, out_dtype, rot_dim, inter, strided, rot = case
    s = Setup(tq, lens, [1] * len(lens), Hkv, P, 11, rot, ragged=ragged)
    got, ref = run_attention(s, Hq, dtype, out_dtype, rot_dim, inter, strided)
    check_attention(got, ref, out_dtype)


@pytest.mark.parametrize("codebook", ["lloyd", "sphere"])
def test_other_codebooks_and_scale(codebook):
    tq = lib()
    s = Setup(tq, [333, 20], [1, 1], 2, 16, 12, ("dense", "wht"), codebook=codebook, ragged=False)
    got, ref = run_attention(s, 8, "f32", "f32", scale=0.31)
    check_attention(got, ref, "f32")


def test_sharp_softmax_and_zero_rows():
    """Scores up to several hundred (one key takes everything), a negative scale, zero norms."""
    import torch
    tq = lib()
    s = Setup(tq, [500, 250], [1, 1], 1, 16, 13, ragged=False)
    for h, d in zip(s.host, s.pages):
        h[s.table[0, :3], :, 2:9, :4] = 0  # zero norms
        d.copy_(torch.from_numpy(h))
    for scale in (8.0, -8.0):
        got, ref = run_attention(s, 4, "f32", "f32", scale=scale)
        check_sharp(s, got, ref, s.q32, scale, f"scale {scale}")


# ------------------------------------------------------------------------------ attention, chunks

CHUNK = [
    # lens, new, Hq, Hkv, P, dtype, out, rot_dim, interleaved, pad, rot
    ([2], [2], 4, 1, 16, "bf16", "bf16", 128, False, 0, ("wht", "wht")),
    ([130, 40, 0, 7], [130, 3, 0, 7], 8, 2, 16, "f16", "f16", 64, True, 9, ("dense", "dense")),
    ([300, 129], [5, 128], 6, 1, 32, "bf16", "bf16", 128, False, 1, ("dense", "wht")),
    ([257], [200], 4, 4, 64, "f32", "f32", 0, False, 0, ("wht", "dense")),
    ([400, 1, 127], [33, 1, 127], 16, 2, 128, "bf16", "bf16", 32, True, 0, ("wht", "wht")),
    ([385, 256], [64, 2], 12, 1, 256, "f16", "bf16", 128, False, 0, ("dense", "dense")),
    ([3, 140], [5, 12], 2, 2, 16, "bf16", "f32", 0, False, 4, ("wht", "wht")),  # more rows than tokens
    ([200], [70], 64, 1, 16, "bf16", "bf16", 0, False, 0, ("wht", "wht")),
    ([1500], [40], 8, 1, 64, "f16", "f16", 128, False, 0, ("dense", "dense")),
    ([140], [140], 10, 2, 16, "f16", "f32", 64, False, 0, ("wht", "wht")),
]


@pytest.mark.parametrize("case", CHUNK, ids=lambda c: f"g{c[2] // c[3]}-p{c[4]}-{c[5]}-t{max(c[1])}of{max(c[0])}")
def test_chunks(case):
    tq = lib()
    lens, new, Hq, Hkv, P, dtype, out_dtype, rot_dim, inter, pad, rot = case
    s = Setup(tq, lens, new, Hkv, P, 17, rot, pad)
    got, ref = run_attention(s, Hq, dtype, out_dtype, rot_dim, inter, strided=True)
    check_attention(got, ref, out_dtype)


@pytest.mark.parametrize("out_dtype", ["bf16", "f16"])
def test_chunks_of_many_short_sequences(out_dtype):
    """More sequences than the plan's threads take at once, most of them below a tile's rows, some empty."""
    tq = lib()
    rng = np.random.default_rng(61)
    new = rng.integers(0, 7, 700)
    new[5], new[300] = 90, 41
    lens = new + rng.integers(0, 30, 700) * rng.integers(0, 2, 700)
    s = Setup(tq, lens.tolist(), new.tolist(), 1, 16, 61, ("dense", "wht"), pad=3)
    got, ref = run_attention(s, 3, "bf16", out_dtype, 64)
    check_attention(got, ref, out_dtype)


@pytest.mark.parametrize("most", [5, 1])
def test_a_batch_of_mostly_idle_slots(most):
    """45,000 slots, 60 of them in use (the plan's prefix sums then lie in the workspace)."""
    tq = lib()
    rng = np.random.default_rng(67)
    new, lens = np.zeros(45000, int), np.zeros(45000, int)
    used = np.concatenate([rng.choice(44999, 59, replace=False), [44999]])
    new[used] = rng.integers(1, most + 1, 60)
    lens[used] = new[used] + rng.integers(0, 40, 60)
    s = Setup(tq, lens.tolist(), new.tolist(), 1, 16, 67, ("dense", "wht"), pad=2)
    got, ref = run_attention(s, 2, "bf16", "bf16", 32)
    check_attention(got, ref, "bf16")


@pytest.mark.parametrize("out_dtype", ["bf16", "f32"])
def test_chunks_of_many_query_tiles(out_dtype):
    """A sequence of more query tiles than a warp has lanes, between short ones."""
    tq = lib()
    s = Setup(tq, [40, 1230, 9], [3, 1200, 9], 1, 32, 62, ("wht", "dense"))
    got, ref = run_attention(s, 16, "bf16", out_dtype, 128)
    check_attention(got, ref, out_dtype)


def test_single_rows_of_many_sequences():
    tq = lib()
    rng = np.random.default_rng(63)
    lens = rng.integers(0, 60, 500)
    lens[77], lens[401] = 3000, 700
    for Hq in (3, 7):  # one group of heads, two
        s = Setup(tq, lens.tolist(), [1] * 500, 1, 16, 63, ("wht", "dense"), ragged=False)
        got, ref = run_attention(s, Hq, "bf16", "f32", 32)
        check_attention(got, ref, "f32")


def test_chunks_sharp_softmax():
    tq = lib()
    s = Setup(tq, [500, 250], [100, 250], 1, 16, 13)
    for scale in (8.0, -8.0):
        got, ref = run_attention(s, 4, "f32", "f32", scale=scale)
        check_sharp(s, got, ref, s.q32, scale, f"scale {scale}")


def set_norms(s, side, norms):
    """norms: {(sequence, head, position): norm}, into the records of one side."""
    import torch
    for (b, h, pos), n in norms.items():
        s.host[side][s.table[b, pos // s.P], h, pos % s.P, :4] = np.frombuffer(np.float32(n).tobytes(), np.uint8)
    s.pages[side].copy_(torch.from_numpy(s.host[side]))


NORMS = [  # lens, new, Hq, Hkv, P, output type
    ([70, 40], [70, 3], 8, 2, 16, "bf16"),
    ([300, 40], [2, 40], 8, 2, 32, "bf16"),
    ([70, 40], [70, 3], 8, 2, 16, "f16"),
    ([70, 40], [1, 1], 8, 2, 64, "bf16"),
    ([520, 40], [1, 1], 12, 2, 64, "f16"),
]


@pytest.mark.parametrize("case", NORMS, ids=lambda c: f"{c[5]}-t{max(c[1])}-n{max(c[0])}-g{c[2] // c[3]}")
def test_norms_without_a_value_reach_the_rows_that_see_them(case):
    """NaN and infinite norms of keys and values: the rows that see one are not finite, the others are as if
    it were not there."""
    tq = lib()
    lens, new, Hq, Hkv, P, out_dtype = case
    s = Setup(tq, lens, new, Hkv, P, 43, ("wht", "dense"), ragged=max(new) > 1)
    spots = [(0, 0, 1, 33, np.nan), (1, 0, 0, 50, np.inf), (1, 1, 1, 38, np.nan), (1, 0, 1, 52, np.nan)]
    for side, b, h, pos, n in spots:
        set_norms(s, side, {(b, h, pos): n})
    got, ref = run_attention(s, Hq, "bf16", out_dtype)
    bad = np.zeros((s.n_rows, Hq), bool)
    for b in range(2):
        for i in range(s.cu[b], s.cu[b + 1]):
            at = lens[b] - (s.cu[b + 1] - i)
            for _, b2, h, pos, _ in spots:
                if b2 == b and at >= pos:
                    bad[i, h * (Hq // Hkv):(h + 1) * (Hq // Hkv)] = True
    got32 = got.float().cpu().numpy()
    assert not np.isfinite(got32[bad]).any() and bad.any()
    import torch
    ref[bad] = 0
    check_attention(torch.from_numpy(np.where(bad[..., None], 0, got32)).cuda(), ref, out_dtype)


@pytest.mark.parametrize("keys", [8.0, 1.0])
@pytest.mark.parametrize("case", [([90, 64], [90, 40], 8, 2, 16, "bf16"), ([90, 64], [90, 40], 2, 2, 16, "f16"),
                                  ([200], [1], 8, 2, 32, "f32"), ([200], [1], 6, 1, 32, "f32")],
                         ids=lambda c: f"{c[5]}-t{max(c[1])}-g{c[2] // c[3]}")
def test_norms_of_a_wide_range(case, keys):
    """Value norms 2^-16 .. 2^15 within 32 keys, rising with the position, so that early rows see the small
    ones alone; key norms `keys` times 2^-3 .. 2^2.  The usual relative bound holds for each row.  On top:
    bf16 outputs of several rows carry values as fp16 with the largest of 32 norms at 2^12 .. 2^13, so
    an element is off by up to 2^-25 2^(15 - 12) where that is more than its relative half step (a mean of
    values: times sqrt(128) for a row); fp16 outputs have steps of 2^-24 below 2^-14.  keys = 8: scores up
    to 32 |q| / sqrt(128): off by d <= (2^-11 + 2^-11) |q| max|k| / sqrt(128) with one part (the centroids'
    error e else), which moves the mean by (exp(2d) - 1) (max|v| + |out|) over the values the row sees."""
    tq = lib()
    lens, new, Hq, Hkv, P, out_dtype = case
    s = Setup(tq, lens, new, Hkv, P, 47, ("dense", "wht"), ragged=max(new) > 1)
    for b, n in enumerate(lens):
        for h in range(Hkv):
            set_norms(s, 1, {(b, h, t): 2.0 ** (t % 32 - 16) for t in range(n)})
            set_norms(s, 0, {(b, h, t): keys * 2.0 ** ((5 * t) % 6 - 3) for t in range(n)})
    got, ref = run_attention(s, Hq, "bf16", out_dtype)
    got = got.float().cpu().numpy().astype(np.float64)
    num = np.linalg.norm(got[:s.n] - ref[:s.n], axis=-1)
    den = np.linalg.norm(ref[:s.n], axis=-1)
    tol = (RTOL + HALF[out_dtype]) * den
    if out_dtype == "bf16":
        tol += 2.0 ** -25 * 2.0 ** (15 - 12) * np.sqrt(128)
    if out_dtype == "f16":
        tol += 2.0 ** -24 * np.sqrt(128)
    if keys > 1:
        e = 2.0 ** -10 if out_dtype == "bf16" else centroid_error(s.codec[0]) + 2.0 ** -20
        d = e * np.linalg.norm(s.q32[:s.n], axis=-1) * keys * 4 / np.sqrt(128)
        for b, n in enumerate(lens):
            for i in range(s.cu[b], s.cu[b + 1]):
                last = n - (s.cu[b + 1] - i)
                tol[i] += np.expm1(2 * d[i]) * (2.0 ** (min(last, 31) - 16) + den[i])
    assert np.all(num <= tol)


# ------------------------------------------------------------------------------ differential

DIFF = [
    # lens, new, Hq, Hkv, P, dtype, per row, norm, pad
    ([50, 0, 333], [1, 1, 1], 8, 2, 16, "bf16", True, True, 0),
    ([700], [1], 4, 2, 64, "f16", False, True, 0),
    ([260, 17], [1, 1], 12, 1, 32, "f32", True, False, 0),
    ([260, 0, 19], [90, 0, 19], 8, 2, 16, "bf16", True, True, 6),
    ([130], [130], 16, 1, 128, "f16", False, True, 0),
    ([77, 300], [77, 9], 6, 1, 64, "f32", True, False, 2),
]


@pytest.mark.parametrize("case", DIFF, ids=lambda c: f"g{c[2] // c[3]}-{c[5]}-t{max(c[1])}-{'norm' if c[7] else 'plain'}")
def test_differential(case):
    """a_h within RTOL of its norm gives |delta d| <= E = RTOL (|a_2p| + lambda |a_2p+1|).  Without a norm
    that is the row's error.  With it, f(d) = d / rms(d) has |delta f| <= 2 sqrt(128) |delta d| / |d|
    to first order (the quotient and its norm), doubled here for the second order; out_scale and the
    gain multiply it; half a step of the output type comes on top."""
    import torch
    tq = lib()
    lens, new, Hq, Hkv, P, dtype, per_row, norm, pad = case
    s = Setup(tq, lens, new, Hkv, P, 19, ("dense", "wht"), pad, ragged=max(new) > 1)
    q, q32 = device_rows(s.rng.standard_normal((s.n_rows, Hq, 128)), dtype)
    lam = s.rng.uniform(0.1, 0.9, (s.n_rows, Hq // 2) if per_row else (Hq // 2,)).astype(np.float32)
    gain = s.rng.uniform(0.5, 1.5, 128).astype(np.float32) if norm else None
    mix = tq.DiffMix(torch.from_numpy(lam).cuda(), torch.from_numpy(gain).cuda() if norm else None, 1e-6, 0.7)
    rope, turn = s.rope(128, False)
    out = torch.full((s.n_rows, Hq // 2, 128), 7.0, dtype=dt(dtype), device="cuda")
    tq.tq_paged_diff_attention(*s.ctx, s.kv, s.batch, q, mix, out, s.workspace(Hq), rope=rope)
    assert s.status() == 0
    att = s.oracle(q32, turn)
    ref = paged.differential(att, lam, gain, 1e-6, 0.7)
    got = out.float().cpu().numpy().astype(np.float64)
    outside = np.isnan(ref).all(axis=(1, 2))
    assert np.all(got[outside] == 7.0)
    d = paged.differential(att, lam)
    E = RTOL * (np.linalg.norm(att[:, 0::2], axis=-1) + np.abs(lam) * np.linalg.norm(att[:, 1::2], axis=-1))
    tol = 0.7 * E
    if norm:
        dn = np.maximum(np.linalg.norm(d, axis=-1), 1e-30)
        tol = 0.7 * gain.max() * 4 * np.sqrt(128) * E / dn
    tol = tol + HALF[dtype] * np.linalg.norm(ref, axis=-1) + 1e-30
    err = np.linalg.norm(got - ref, axis=-1)
    assert np.all(err[~outside] <= tol[~outside])
    empty = np.array([np.all(att[i] == 0) for i in range(s.n_rows)])
    assert np.all(got[empty] == 0)


# ------------------------------------------------------------------------------ together

def test_steps_together_and_captured():
    """A prompt appended and attended in chunks, then decode steps through one captured graph whose
    lengths, rows and outputs live in fixed buffers; the cache equals the one an eager run leaves
    and every step's output the oracle's over it."""
    import torch
    tq = lib()
    B, Hq, Hkv, P, steps = 3, 8, 2, 16, 5
    prompt, final = [40, 17, 1], [45, 22, 6]
    s = Setup(tq, final, [1] * B, Hkv, P, 23, ("wht", "dense"), fill=False, ragged=False)
    rope, turn = s.rope(128, False)
    gen = torch.Generator(device="cuda").manual_seed(3)
    rows = lambda n, h: torch.randn((n, h, 128), generator=gen, device="cuda").bfloat16()  # noqa: E731
    cu = torch.tensor(np.concatenate([[0], np.cumsum(prompt)]), dtype=torch.int32, device="cuda")
    lens = torch.tensor(prompt, dtype=torch.int32, device="cuda")
    first = tq.PagedBatch(lens, cu, max(prompt), sum(prompt))
    k, v, q = rows(sum(prompt), Hkv), rows(sum(prompt), Hkv), rows(sum(prompt), Hq)
    out = torch.empty_like(q)
    ws = tq.alloc_workspace(max(tq.tq_paged_workspace_size(*s.ctx, s.kv, b, Hq) for b in (first, s.batch)))
    tq.tq_paged_append(*s.ctx, s.kv, first, k, v, rope=rope)
    tq.tq_paged_attention(*s.ctx, s.kv, first, q, out, ws, rope=rope)
    assert s.status() == 0
    host = [p.cpu().numpy() for p in s.pages]
    ref = paged.attention(*s.codec, *host, s.table, prompt, cu.cpu().numpy(), q.float().cpu().numpy(), sum(prompt), 0.0, turn)
    check_attention(out, ref, "bf16", "prompt")

    step_k, step_v, step_q = rows(B, Hkv), rows(B, Hkv), rows(B, Hq)
    out1 = torch.empty_like(step_q)
    s.d_lens.copy_(lens + 1)

    def step():
        tq.tq_paged_append(*s.ctx, s.kv, s.batch, step_k, step_v, rope=rope)
        tq.tq_paged_attention(*s.ctx, s.kv, s.batch, step_q, out1, ws, rope=rope)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()  # warm-up outside the capture, on the capture's stream
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    for i in range(steps):
        s.d_lens.copy_(lens + 1 + i)
        for t in (step_k, step_v, step_q):
            t.copy_(torch.randn(t.shape, generator=gen, device="cuda"))
        out1.fill_(9)
        graph.replay()
        assert s.status() == 0
        replayed, cache = out1.clone(), [p.clone() for p in s.pages]
        step()
        torch.cuda.synchronize()
        assert torch.equal(out1, replayed) and all(torch.equal(a, b) for a, b in zip(cache, s.pages))
        host = [p.cpu().numpy() for p in s.pages]
        now = [n + 1 + i for n in prompt]
        ref = paged.attention(*s.codec, *host, s.table, now, np.arange(B + 1), step_q.float().cpu().numpy(), B, 0.0, turn)
        check_attention(out1, ref, "bf16", f"step {i}")


def test_shared_pages_same_result():
    """Two sequences that share their first pages read the same keys."""
    import torch
    tq = lib()
    s = Setup(tq, [64, 64], [1, 1], 2, 16, 29, ragged=False)
    s.table[1, :3] = s.table[0, :3]
    s.kv.block_table.copy_(torch.from_numpy(s.table))
    got, ref = run_attention(s, 4, "f32", "f32")
    check_attention(got, ref, "f32")


def test_two_streams_and_repeated_calls_agree():
    """The same call twice gives the same bits; two calls at once on two streams, each with its own
    workspace and output, give theirs."""
    import torch
    tq = lib()
    s = Setup(tq, [1900, 3, 777], [1, 1, 1], 2, 32, 31, ragged=False)
    c = Setup(tq, [600, 250], [200, 100], 2, 32, 37)
    jobs = []
    for x in (s, c):
        q = torch.randn((x.n_rows, 8, 128), device="cuda").bfloat16()
        first = torch.empty_like(q)
        tq.tq_paged_attention(*x.ctx, x.kv, x.batch, q, first, x.workspace(8))
        jobs.append((x, q, first, x.workspace(8)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in jobs]
    for _ in range(5):
        outs = []
        for st, (x, q, first, ws) in zip(streams, jobs):
            o = torch.zeros_like(first)
            torch.cuda.synchronize()
            outs.append(o)
        for st, o, (x, q, first, ws) in zip(streams, outs, jobs):
            tq.tq_paged_attention(*x.ctx, x.kv, x.batch, q, o, ws, stream=st)
        torch.cuda.synchronize()
        for o, (x, q, first, ws) in zip(outs, jobs):
            assert torch.equal(o, first)


@pytest.mark.parametrize("rot", [("wht", "wht"), ("dense", "dense")], ids="/".join)
def test_captured_chunks_follow_the_batch(rot):
    """Append, read back, chunk attention and the differential one captured together; replayed after the
    rows, the offsets and the lengths changed in place they give an eager run's bits."""
    import torch
    tq = lib()
    s = Setup(tq, [700, 520, 90], [400, 300, 60], 4, 32, 71, rot, pad=40)
    cu = torch.from_numpy(s.cu).cuda()
    batch = tq.PagedBatch(s.d_lens, cu, 420, s.n_rows)
    rope, _ = s.rope(128, False)
    k, v = (torch.randn((s.n_rows, 4, 128), device="cuda").bfloat16() for _ in range(2))
    q = torch.randn((s.n_rows, 16, 128), device="cuda").bfloat16()
    mix = tq.DiffMix(torch.rand(8, device="cuda"), torch.ones(128, device="cuda"))
    ws = torch.empty(max(tq.tq_paged_workspace_size(*s.ctx, s.kv, batch, 16), 256), dtype=torch.uint8, device="cuda")

    def outputs():
        return [torch.full((s.n_rows, h, 128), 7.0, dtype=d, device="cuda")
                for h, d in ((16, torch.bfloat16), (16, torch.float16), (8, torch.bfloat16), (4, torch.float16))]

    def run(o):
        tq.tq_paged_append(*s.ctx, s.kv, batch, k, v, rope=rope)
        tq.tq_paged_attention(*s.ctx, s.kv, batch, q, o[0], ws, rope=rope)
        tq.tq_paged_attention(*s.ctx, s.kv, batch, q, o[1], ws, rope=rope)
        tq.tq_paged_diff_attention(*s.ctx, s.kv, batch, q, mix, o[2], ws, rope=rope)
        tq.tq_paged_gather(*s.ctx, s.kv, batch, o[3], None)

    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    held = outputs()
    with torch.cuda.stream(stream):
        run(held)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=stream):
        run(held)
    for lens, new in (([700, 520, 90], [400, 300, 60]), ([610, 333, 70], [20, 333, 1]), ([5, 0, 96], [0, 0, 96])):
        s.d_lens.copy_(torch.tensor(lens, dtype=torch.int32))
        cu.copy_(torch.from_numpy(np.concatenate([[0], np.cumsum(new)]).astype(np.int32)))
        for t in (k, v, q):
            t.normal_()
        for o in held:
            o.fill_(7.0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        pages = [p.clone() for p in s.pages]
        eager = outputs()
        run(eager)
        assert s.status() == 0
        for a, b in zip(held + pages, eager + list(s.pages)):
            assert torch.equal(a, b)


def test_offsets_past_32_bits():
    """Pages of more than 2^32 bytes; the sequence's pages lie at the end."""
    import torch
    tq = lib()
    s = Setup(tq, [500, 300], [1, 140], 8, 64, 41)
    n_big = (1 << 32) // (8 * 64 * 68) + 40
    shift = n_big - s.n_pages
    big = []
    for p in s.pages:
        t = torch.empty((n_big, 8, 64, 68), dtype=torch.uint8, device="cuda")
        t[shift:] = p
        big.append(t)
    table = torch.from_numpy(np.where(s.table < 0, s.table, s.table + shift)).cuda()
    s.kv = tq.PagedKV(big[0], big[1], table, 64, 8)
    got, ref = run_attention(s, 16, "bf16", "bf16", 128)
    check_attention(got, ref, "bf16")
    k = torch.randn((s.n_rows, 8, 128), device="cuda")
    tq.tq_paged_append(*s.ctx, s.kv, s.batch, k, k)
    o = [torch.empty_like(k) for _ in range(2)]
    tq.tq_paged_gather(*s.ctx, s.kv, s.batch, *o)
    assert s.status() == 0
    cos = torch.nn.functional.cosine_similarity(o[0], k, dim=-1)
    assert float(cos.min()) > 0.95  # 4-bit rows: about 0.99


def test_no_rows_is_a_no_op():
    import torch
    tq = lib()
    s = Setup(tq, [10], [1], 1, 16, 43)
    none = tq.PagedBatch(torch.zeros(0, dtype=torch.int32, device="cuda"))
    q = torch.zeros((0, 2, 128), device="cuda")
    before = [p.clone() for p in s.pages]
    ws = tq.alloc_workspace(tq.tq_paged_workspace_size(*s.ctx, s.kv, none, 2))
    tq.tq_paged_append(*s.ctx, s.kv, none, q[:, :1], q[:, :1])
    tq.tq_paged_attention(*s.ctx, s.kv, none, q, q.clone(), ws)
    cu = tq.PagedBatch(s.d_lens, torch.zeros(2, dtype=torch.int32, device="cuda"), 4, 5)  # rows, all of them padding
    out = torch.full((5, 2, 128), 7.0, device="cuda")
    ws = tq.alloc_workspace(tq.tq_paged_workspace_size(*s.ctx, s.kv, cu, 2))
    tq.tq_paged_attention(*s.ctx, s.kv, cu, torch.zeros_like(out), out, ws)
    tq.tq_paged_append(*s.ctx, s.kv, cu, out[:, :1], out[:, :1])
    assert s.status() == 0
    assert torch.all(out == 7.0) and all(torch.equal(a, b) for a, b in zip(before, s.pages))


# ------------------------------------------------------------------------------ flags and refusals

def test_bad_pages_lengths_and_positions_are_flagged():
    import torch
    tq = lib()
    s = Setup(tq, [40, 30], [1, 1], 2, 16, 47, ragged=False)
    good, _ = run_attention(s, 4, "f32", "f32")
    q = torch.randn((2, 4, 128), device="cuda")
    out, ws = torch.empty_like(q), s.workspace(4)
    want = torch.empty_like(q)
    tq.tq_paged_attention(*s.ctx, s.kv, s.batch, q, want, ws)
    for bad in (-1, s.n_pages, 2 ** 31 - 1):
        t = s.kv.block_table.clone()
        t[1, 1] = bad
        kv = tq.PagedKV(*s.pages, t, 16, 2)
        tq.tq_paged_attention(*s.ctx, kv, s.batch, q, out, ws)
        assert s.status() == 5 and torch.equal(out[0], want[0])  # the other sequence is whole
        k = torch.randn((2, 2, 128), device="cuda")
        before = [p.clone() for p in s.pages]
        tq.tq_paged_append(*s.ctx, kv, s.batch, k, k)
        assert s.status() == 5
        for a, p in zip(before, s.pages):
            diff = (a != p).any(-1).nonzero()
            assert diff.shape[0] and {int(x) for x in diff[:, 0]} == {int(s.table[0, 2])}
            p.copy_(a)
        tq.tq_paged_gather(*s.ctx, kv, s.batch, k.clone(), k)
        assert s.status() == 5
    for n in (-3, 49):  # the block table holds 48 tokens
        s.d_lens[1] = n
        tq.tq_paged_attention(*s.ctx, s.kv, s.batch, q, out, ws)
        st = s.status()
        assert st in (2, 5) if n > 0 else st == 2
        assert torch.equal(out[0], want[0])
        assert n > 0 or torch.all(out[1] == 0)
    s.d_lens[1] = 30
    short, _ = s.rope(64, False, n_pos=20)
    tq.tq_paged_attention(*s.ctx, s.kv, s.batch, q, out, ws, rope=short)
    assert s.status() == 6
    tq.tq_paged_attention(*s.ctx, s.kv, s.batch, q, out, ws)
    assert s.status() == 0 and torch.equal(out, want)


def test_refusals():
    import torch
    tq = lib()
    L = tq.lib
    s = Setup(tq, [40, 30], [1, 1], 2, 16, 53, ragged=False)
    q = torch.randn((2, 4, 128), device="cuda")
    out, ws = torch.full_like(q, 7.0), s.workspace(4)
    n_ws = tq.tq_paged_workspace_size(*s.ctx, s.kv, s.batch, 4)

    def call(kv=(), batch=(), rows=(), rope=None, ctx=None, Hq=4, out_p=None, dtype=0, ws_p=None, ws_n=None, diff=None,
             scale=0.0):
        a, b, r = (type(x).from_buffer_copy(x) for x in (s.kv.c, s.batch.c, tq.tq_rows(q.data_ptr(), 0, 512, 128)))
        for c, kw in ((a, kv), (b, batch), (r, rows)):
            for name, val in kw:
                setattr(c, name, val)
        k, v = ctx or s.ctx
        args = [k.handle, v.handle, ctypes.byref(a), ctypes.byref(b), ctypes.byref(r), Hq, ctypes.byref(rope) if rope else None]
        tail = [scale, out.data_ptr() if out_p is None else out_p, dtype, ws.data_ptr() if ws_p is None else ws_p,
                n_ws if ws_n is None else ws_n, None]
        if diff is not None:
            return L.tq_paged_diff_attention(*args, ctypes.byref(diff), *tail)
        return L.tq_paged_attention(*args, *tail)

    INV, UNS, ALI, WS = tq.TQ_ERR_INVALID_ARG, tq.TQ_ERR_UNSUPPORTED, tq.TQ_ERR_ALIGNMENT, tq.TQ_ERR_WORKSPACE
    assert call() == tq.TQ_OK
    torch.cuda.synchronize()
    out.fill_(7.0)
    for size in (0, 8, 24, 48, 512):
        assert call(kv=[("page_size", size)]) == INV
    for f in ("n_pages", "Hkv", "table_len"):
        assert call(kv=[(f, 0)]) == INV
    assert call(kv=[("table_stride", 1)]) == INV
    assert call(kv=[("k_pages", None)]) == INV and call(kv=[("block_table", None)]) == INV
    assert call(kv=[("v_pages", s.pages[1].data_ptr() + 8)]) == ALI
    assert call(kv=[("block_table", s.kv.block_table.data_ptr() + 2)]) == ALI
    assert call(batch=[("max_q", 0)]) == INV and call(batch=[("max_q", 2)]) == INV
    assert call(batch=[("n_tokens", 3)]) == INV and call(batch=[("B", -1)]) == INV
    assert call(batch=[("max_len", 49)]) == INV and call(batch=[("max_len", -1)]) == INV
    assert call(batch=[("seq_lens", None)]) == INV
    assert call(rows=[("data", None)]) == INV and call(rows=[("dtype", 3)]) == INV
    assert call(rows=[("data", q.data_ptr() + 4)]) == ALI and call(rows=[("token_stride", 513)]) == ALI
    assert call(rows=[("head_stride", 64)]) == INV and call(rows=[("token_stride", -512)]) == INV
    assert call(Hq=3) == INV and call(Hq=0) == INV and call(Hq=2 * 66) == UNS
    assert call(dtype=5) == INV and call(out_p=0) == INV and call(out_p=out.data_ptr() + 4) == ALI
    assert call(ws_n=n_ws - 1) == WS and call(ws_p=0) == WS and call(ws_p=ws.data_ptr() + 16) == ALI
    assert call(scale=float("nan")) == INV and call(scale=float("inf")) == INV
    cs = torch.ones((48, 64), device="cuda")
    rope = lambda **kw: tq.tq_rope(**{"cos_table": cs.data_ptr(), "sin_table": cs.data_ptr(), "n_pos": 48, "rot_dim": 128,  # noqa: E731
                                      "interleaved": 0, **kw})
    assert call(rope=rope(rot_dim=96)) == UNS and call(rope=rope(n_pos=0)) == INV and call(rope=rope(interleaved=2)) == INV
    assert call(rope=rope(cos_table=None)) == INV and call(rope=rope(sin_table=cs.data_ptr() + 4)) == ALI
    three, big = tq.Ctx("turbo3"), tq.Ctx("turbo4", d=256)
    assert call(ctx=(s.ctx[0], three)) == UNS and call(ctx=(big, s.ctx[1])) == UNS
    lam = torch.ones((2, 2), device="cuda")
    diff = lambda **kw: tq.tq_diff(**{"lambda_w": lam.data_ptr(), "lambda_stride": 2, "gain": None, "eps": 0.0, "out_scale": 1.0, **kw})  # noqa: E731
    assert call(diff=diff(lambda_w=None)) == INV and call(diff=diff(lambda_stride=1)) == INV
    assert call(diff=diff(eps=-1.0)) == INV and call(diff=diff(out_scale=float("inf"))) == INV
    assert call(diff=diff(gain=cs.data_ptr() + 4)) == ALI and call(diff=diff(lambda_w=lam.data_ptr() + 2)) == ALI
    assert call(diff=diff(), Hq=2) == INV  # one q-head per KV head: no pair
    L.tq_test_ctx_set_device(s.ctx[0].handle, 1)
    L.tq_test_ctx_set_device(s.ctx[1].handle, 1)
    assert call() == INV
    L.tq_test_ctx_set_device(s.ctx[0].handle, 0)
    assert call() == INV  # the two contexts on different devices
    L.tq_test_ctx_set_device(s.ctx[1].handle, 0)
    a, b = ctypes.byref(s.kv.c), ctypes.byref(s.batch.c)
    r = tq.tq_rows(q.data_ptr(), 0, 512, 128)
    r16 = tq.tq_rows(q.data_ptr(), 1, 512, 128)
    H = [x.handle for x in s.ctx]
    assert L.tq_paged_append(*H, a, b, ctypes.byref(r), None, None, None) == INV
    assert L.tq_paged_append(*H, a, b, ctypes.byref(r), ctypes.byref(r16), None, None) == INV
    assert L.tq_paged_gather(*H, a, b, 1, None, None, 0, None) == INV
    assert L.tq_paged_gather(*H, a, b, 1, out.data_ptr() + 4, None, 0, None) == ALI
    assert L.tq_paged_gather(*H, a, b, 1, out.data_ptr(), None, 9, None) == INV
    torch.cuda.synchronize()
    assert torch.all(out == 7.0) and s.status() == 0


def test_python_refusals():
    """What the binding can see and the library cannot: tensors off the GPU, a block table of fewer rows than
    sequences, workspaces and outputs that are too small."""
    import torch
    tq = lib()
    s = Setup(tq, [40, 30], [1, 1], 2, 16, 54, ragged=False)
    q = torch.randn((2, 4, 128), device="cuda")
    kv = torch.randn((2, 2, 128), device="cuda")
    out, ws = torch.full_like(q, 7.0), s.workspace(4)
    one = tq.PagedKV(s.pages[0], s.pages[1], s.kv.block_table[:1], 16, 2)
    bad = [lambda: tq.tq_paged_attention(*s.ctx, one, s.batch, q, out, ws),
           lambda: tq.tq_paged_append(*s.ctx, one, s.batch, kv, kv),
           lambda: tq.tq_paged_gather(*s.ctx, one, s.batch, kv, None),
           lambda: tq.tq_paged_attention(*s.ctx, s.kv, s.batch, q.cpu(), out, ws),
           lambda: tq.tq_paged_attention(*s.ctx, s.kv, s.batch, q, out.cpu(), ws),
           lambda: tq.tq_paged_attention(*s.ctx, s.kv, s.batch, q, out[:1], ws),
           lambda: tq.tq_paged_append(*s.ctx, s.kv, s.batch, kv, kv.cpu()),
           lambda: tq.tq_paged_attention(*s.ctx, tq.PagedKV(s.pages[0].cpu(), s.pages[1], s.kv.block_table, 16, 2), s.batch, q, out, ws),
           lambda: tq.tq_paged_attention(*s.ctx, tq.PagedKV(s.pages[0], s.pages[1], s.kv.block_table.cpu(), 16, 2), s.batch, q, out, ws),
           lambda: tq.tq_paged_attention(*s.ctx, s.kv, tq.PagedBatch(s.d_lens.cpu()), q, out, ws),
           lambda: tq.tq_paged_attention(*s.ctx, s.kv, s.batch, q, out, ws, rope=tq.Rope(torch.ones(4, 64), torch.ones(4, 64))),
           lambda: tq.tq_paged_diff_attention(*s.ctx, s.kv, s.batch, q, tq.DiffMix(torch.ones(2)), out[:, :2].contiguous(), ws)]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    torch.cuda.synchronize()
    assert s.status() == 0 and torch.all(out == 7.0)
