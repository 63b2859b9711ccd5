"""The paged oracle against the contiguous one and against properties of its definitions, and the
host-only parts of the paged interface (the rotation table, the binding's argument checks)."""

import numpy as np
import pytest

import oracle
from oracle import paged
from oracle.formats import Codec


def make(lens, Hkv, P, seed, codec):
    rng = np.random.default_rng(seed)
    width = max(max((n + P - 1) // P for n in lens), 1)
    need = sum((n + P - 1) // P for n in lens)
    order = rng.permutation(need + 2)
    table = np.zeros((len(lens), width), np.int32)
    at = 0
    pages = np.full((need + 2, Hkv, P, 68), 255, np.uint8)
    dense = []
    for b, n in enumerate(lens):
        k = (n + P - 1) // P
        table[b, :k] = order[at:at + k]
        at += k
        rows, _ = codec.encode(rng.standard_normal((n * Hkv, 128)).astype(np.float32)) if n else (
            np.zeros((0, 68), np.uint8), None)
        rows = rows.reshape(n, Hkv, 68)
        for t in range(n):
            pages[table[b, t // P], :, t % P] = rows[t]
        dense.append(rows)
    return pages, table, dense


def test_single_rows_equal_the_contiguous_reference():
    codec = Codec("turbo4", rotation="wht", rot_seed=3)
    lens, Hkv, Hq, P = [37, 16, 1], 2, 6, 16
    pages, table, dense = make(lens, Hkv, P, 0, codec)
    q = np.random.default_rng(1).standard_normal((3, Hq, 128))
    out = paged.attention(codec, codec, pages, pages, table, lens, np.arange(4), q, 3)
    for b in range(3):
        X = codec.dequantize(dense[b].reshape(-1, 68)).reshape(lens[b], Hkv, 128).transpose(1, 0, 2)[None]
        ref, _ = oracle.attention_reference(q[b:b + 1], X, X)
        assert np.max(np.abs(out[b] - ref[0])) < 1e-12


def test_chunks_equal_single_rows_and_empty_rows_are_zero():
    codec = Codec("turbo4", rotation="dense", rot_seed=3)
    lens, Hkv, P = [21, 0, 2], 1, 16
    pages, table, _ = make(lens, Hkv, P, 2, codec)
    cu = np.array([0, 4, 5, 8])  # the last sequence has three rows and two tokens
    q = np.random.default_rng(1).standard_normal((9, 2, 128))
    out = paged.attention(codec, codec, pages, pages, table, lens, cu, q, 9)
    for i in range(4):
        one = paged.attention(codec, codec, pages, pages, table, [18 + i], np.array([0, 1]), q[i:i + 1], 1)
        assert np.max(np.abs(one[0] - out[i])) < 1e-13
    assert np.all(out[4] == 0) and np.all(out[5] == 0) and np.all(np.isnan(out[8]))
    assert np.all(out[6] != 0)


@pytest.mark.parametrize("rot_dim", [32, 64, 128])
@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_keeps_norms_and_relative_positions(rot_dim, interleaved):
    half = rot_dim // 2
    ang = np.arange(50)[:, None] * 10000.0 ** (-np.arange(half) / half)
    cos, sin = np.cos(ang), np.sin(ang)
    x, y = np.random.default_rng(0).standard_normal((2, 1, 1, 128))
    turn = lambda v, p: paged.rope(v, cos, sin, np.array([p]), interleaved)  # noqa: E731
    assert abs(np.linalg.norm(turn(x, 33)) - np.linalg.norm(x)) < 1e-12
    assert abs(np.sum(turn(x, 40) * turn(y, 33)) - np.sum(turn(x, 7) * turn(y, 0))) < 1e-11
    assert np.array_equal(turn(x, 5)[..., rot_dim:], x[..., rot_dim:])


def test_differential_of_equal_maps():
    a = np.random.default_rng(0).standard_normal((3, 2, 128))
    same = np.repeat(a[:, :1], 2, axis=1)
    out = paged.differential(same, np.full((3, 1), 0.25))
    assert np.allclose(out[:, 0], 0.75 * same[:, 0])
    n = paged.differential(a, np.zeros((3, 1)), np.ones(128), 0.0, 2.0)
    assert np.allclose(np.sqrt((n * n).mean(-1)), 2.0)


@pytest.fixture(scope="module")
def tq():
    import __graft_entry__
    __graft_entry__.build()
    import compressed_attention_gb300 as m
    return m


@pytest.mark.parametrize("rot_dim,base", [(128, 10000.0), (64, 500000.0), (32, 10000.0)])
def test_rope_table(tq, rot_dim, base):
    """fp64 angles rounded once: off by at most half an fp32 step, plus the fp64 angle's own error
    (position 2^17 times an angle rounded to 2^-53, well below 2^-30)."""
    c, s = tq.tq_make_rope_table(rot_dim, 131072, base)
    p = np.array([0, 1, 2, 1000, 65537, 131071])
    ang = p[:, None] * base ** (-2.0 * np.arange(rot_dim // 2) / rot_dim)
    assert np.max(np.abs(c[p] - np.cos(ang))) <= 2.0 ** -24 * 0.51 + 2.0 ** -30
    assert np.max(np.abs(s[p] - np.sin(ang))) <= 2.0 ** -24 * 0.51 + 2.0 ** -30


def test_host_refusals(tq):
    import ctypes
    lib = tq.lib
    z = np.zeros(64, np.float32)
    assert lib.tq_make_rope_table(48, 1e4, 1, z.ctypes.data, z.ctypes.data) == tq.TQ_ERR_UNSUPPORTED
    assert lib.tq_make_rope_table(64, 0.0, 1, z.ctypes.data, z.ctypes.data) == tq.TQ_ERR_INVALID_ARG
    assert lib.tq_make_rope_table(64, float("nan"), 1, z.ctypes.data, z.ctypes.data) == tq.TQ_ERR_INVALID_ARG
    assert lib.tq_make_rope_table(64, 1e4, -1, z.ctypes.data, z.ctypes.data) == tq.TQ_ERR_INVALID_ARG
    assert lib.tq_make_rope_table(64, 1e4, 1, None, z.ctypes.data) == tq.TQ_ERR_INVALID_ARG
    n = ctypes.c_size_t(9)
    assert lib.tq_paged_append(None, None, None, None, None, None, None, None) == tq.TQ_ERR_INVALID_ARG
    assert lib.tq_paged_gather(None, None, None, None, 1, None, None, 0, None) == tq.TQ_ERR_INVALID_ARG
    assert lib.tq_paged_workspace_size(None, None, None, None, 1, ctypes.byref(n)) == tq.TQ_ERR_INVALID_ARG
    assert lib.tq_paged_workspace_size(None, None, None, None, 1, None) == tq.TQ_ERR_INVALID_ARG
    assert n.value == 9
    assert lib.tq_paged_attention(None, None, None, None, None, 1, None, 0.0, None, 0, None, 0,
                                  None) == tq.TQ_ERR_INVALID_ARG
    assert lib.tq_paged_diff_attention(None, None, None, None, None, 1, None, None, 0.0, None, 0, None, 0,
                                       None) == tq.TQ_ERR_INVALID_ARG
    assert b"differential" in lib.tq_last_error()


def test_binding_refusals(tq):
    import torch
    u8 = torch.zeros((4, 2, 16, 68), dtype=torch.uint8)
    tab = torch.zeros((2, 2), dtype=torch.int32)
    tq.PagedKV(u8, u8, tab, 16, 2)
    for bad in (lambda: tq.PagedKV(u8.float(), u8, tab, 16, 2), lambda: tq.PagedKV(u8, u8[:3], tab, 16, 2),
                lambda: tq.PagedKV(u8, u8, tab.long(), 16, 2), lambda: tq.PagedKV(u8, u8, tab.t(), 16, 2),
                lambda: tq.PagedKV(u8, u8, tab, 48, 2), lambda: tq.PagedKV(u8[:, :1], u8[:, :1], tab, 16, 1)):
        with pytest.raises(ValueError):
            bad()
    lens = torch.ones(2, dtype=torch.int32)
    cu = torch.arange(3, dtype=torch.int32)
    assert tq.PagedBatch(lens).n_tokens == 2
    for bad in (lambda: tq.PagedBatch(lens.long()), lambda: tq.PagedBatch(lens, cu), lambda: tq.PagedBatch(lens, cu[:2], 1, 2)):
        with pytest.raises(ValueError):
            bad()
    cs = torch.ones((8, 64))
    tq.Rope(cs, cs)
    for bad in (lambda: tq.Rope(cs, cs[:4]), lambda: tq.Rope(cs.double(), cs), lambda: tq.Rope(cs[:, ::2], cs[:, ::2])):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(ValueError):
        tq.DiffMix(cs[0], norm_weight=torch.ones(64))

    class Ctx:
        handle = None
    kv, b = tq.PagedKV(u8, u8, tab, 16, 2), tq.PagedBatch(lens)
    row = torch.zeros((2, 2, 128))
    for bad in (lambda: tq.tq_paged_append(Ctx, Ctx, kv, b, row[:1], row), lambda: tq.tq_paged_append(Ctx, Ctx, kv, b, row, row[:, :1]),
                lambda: tq.tq_paged_append(Ctx, Ctx, kv, b, row[..., :64], row), lambda: tq.tq_paged_gather(Ctx, Ctx, kv, b, None, None),
                lambda: tq.tq_paged_gather(Ctx, Ctx, kv, b, row, row.half()),
                lambda: tq.tq_paged_attention(Ctx, Ctx, kv, b, row, row[:, :1], None),
                lambda: tq.tq_paged_attention(Ctx, Ctx, kv, b, row, torch.zeros((2, 2, 256))[..., ::2], None),
                lambda: tq.tq_paged_diff_attention(Ctx, Ctx, kv, b, row, tq.DiffMix(torch.ones(2)), row[:, :1], None)):
        with pytest.raises(ValueError):
            bad()
