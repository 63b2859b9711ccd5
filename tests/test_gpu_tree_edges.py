"""Edges of the drafted trees' calls on the GPU: batches without rows, offsets past their bounds, steps of several
layers, vocabularies and batches at which the verification is laid out differently, norms of a wide range."""

import ctypes

import numpy as np
import pytest

from gpu_util import lib
from oracle import paged, tree
from test_gpu_paged import HALF, centroid_error, check_attention, set_norms
from test_gpu_tree import ATTENTION, FullTrees, Trees, Walks, run_tree

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("draft", [True, False], ids=["draft", "no-draft"])
def test_verify_of_idle_slots_alone(draft):
    """A batch of sequences without rows: empty arrays (whose addresses are null), empty paths."""
    import torch
    tq = lib()
    ctx = tq.Ctx("turbo4")
    i32 = dict(dtype=torch.int32, device="cuda")
    batch = tq.PagedBatch(torch.zeros(3, **i32), torch.zeros(4, **i32), 5, 0)
    none, rows = torch.zeros(0, **i32), torch.zeros((0, 70), dtype=torch.bfloat16, device="cuda")
    path, n, nxt = torch.full((3, 6), 9, **i32), torch.full((3,), 9, **i32), torch.full((3,), 9, **i32)
    tq.tq_tree_verify(ctx, batch, none, none, rows, none.float(), torch.rand(3, device="cuda"), path, n, nxt,
                      draft=rows if draft else None)
    assert tq.tq_ctx_device_status(ctx) == 0
    assert n.tolist() == [0] * 3 and nxt.tolist() == [-1] * 3 and path.tolist() == [[-1] * 5 + [9]] * 3


def test_keep_of_paths_longer_than_max_q():
    """Offsets that name more nodes than max_q, and a path of as many: what lies behind a row of max_q entries is not
    the path's (the last row's end may be the buffer's), so it is not taken."""
    import torch
    tq = lib()
    s = Trees(tq, [50, 40], [6, 6], 2, 16, 89)
    s.batch.c.max_q = 4
    buffer = torch.tensor([0, 1, 2, 3, 9, 9, 9, 9, 0, 2, 3, 4, 5, 6, 7, 8], dtype=torch.int32, device="cuda")
    path = buffer.view(2, 8)[:, :4]
    for n, took in ((4, True), (5, False), (6, False)):
        for p, h in zip(s.pages, s.host):
            p.copy_(torch.from_numpy(h))
        lens = torch.zeros_like(s.d_lens)
        tq.tq_paged_tree_keep(*s.ctx, s.kv, s.batch, path, torch.tensor([4, n], dtype=torch.int32, device="cuda"), lens)
        assert s.status() == (0 if took else 7) and lens.tolist() == [48, 38 if took else 34]
        for p, h in zip(s.pages, s.host):
            want, _ = tree.keep(h, s.table, s.lens, s.cu, [[0, 1, 2, 3], [0, 2, 3, 4] if took else []])
            assert np.array_equal(p.cpu().numpy(), want)


@pytest.mark.parametrize("captured", [False, True], ids=["eager", "captured"])
def test_steps_of_several_layers(captured):
    """Three layers' caches over two steps: append and attention in each, one verification's path kept in each, the
    lengths written over in the last layer's call alone.  Every layer holds what the oracle's append and keep leave."""
    import torch
    tq = lib()
    B, T, Hkv, P, layers = 3, 6, 2, 16, 3
    lens0 = [40, 21, 6]  # of the context; the last sequence's tree lies across its first page's end
    rng = np.random.default_rng(97)
    setups = [Trees(tq, [n + T for n in lens0], [T] * B, Hkv, P, 101 + i, wide=2, width=8) for i in range(layers)]
    first = setups[0]
    for s in setups:
        s.table[:] = rng.permutation(24).reshape(3, 8)
        n_pages = 24
        host = [np.zeros((n_pages, Hkv, P, 68), np.uint8) for _ in range(2)]
        for x in host:
            x[..., 4:] = rng.integers(0, 256, x[..., 4:].shape)
            x[..., :4] = np.ones(x.shape[:-1], np.float32)[..., None].view(np.uint8)
        s.host = host
        s.pages = [torch.from_numpy(h.copy()).cuda() for h in host]
        s.kv = tq.PagedKV(*s.pages, torch.from_numpy(s.table).cuda(), P, Hkv)
    lens, batch, parents = first.d_lens, first.batch, first.d_parents
    lens_of = [torch.zeros_like(lens) for _ in range(layers - 1)] + [lens]
    k = [torch.zeros((B * T, Hkv, 128), device="cuda") for _ in range(layers)]
    v, q = [x.clone() for x in k], [torch.zeros((B * T, 4, 128), device="cuda") for _ in range(layers)]
    out, ws = [torch.zeros_like(x) for x in q], first.tree_workspace(4)
    path = torch.zeros((B, T), dtype=torch.int32, device="cuda")
    n_path = torch.zeros(B, dtype=torch.int32, device="cuda")

    def step():
        for s, ki, vi, qi, oi in zip(setups, k, v, q, out):
            tq.tq_paged_tree_append(*s.ctx, s.kv, batch, parents, ki, vi)
            tq.tq_paged_tree_attention(*s.ctx, s.kv, batch, parents, qi, oi, ws)
        for s, x in zip(setups, lens_of):
            tq.tq_paged_tree_keep(*s.ctx, s.kv, batch, path, n_path, x)
        lens.add_(T)

    if captured:
        start = [[p.clone() for p in s.pages] for s in setups] + [lens.clone()]
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            step()
        for s, held in zip(setups, start):
            for p, x in zip(s.pages, held):
                p.copy_(x)
        lens.copy_(start[-1])
    at = [n + T for n in lens0]
    for _ in range(2):
        paths = []
        for b in range(B):
            line, i = [], int(rng.integers(T))
            while i >= 0:
                line.append(i)
                i = int(first.parents[b * T + i])
            paths.append(line[::-1])
        path.copy_(torch.tensor([x + [-1] * (T - len(x)) for x in paths], dtype=torch.int32))
        n_path.copy_(torch.tensor([len(x) for x in paths], dtype=torch.int32))
        for x in (*k, *v, *q):
            x.copy_(torch.from_numpy(rng.standard_normal(tuple(x.shape)).astype(np.float32)))
        if captured:
            graph.replay()
        else:
            step()
        for i, s in enumerate(setups):
            for side, rows in enumerate((k[i], v[i])):
                rec, _ = s.codec[side].encode(rows.cpu().numpy().reshape(-1, 128))
                rec = rec.reshape(B, T, Hkv, 68)
                for b in range(B):
                    slot = np.arange(at[b] - T, at[b])
                    s.host[side][s.table[b, slot // P], :, slot % P] = rec[b]
            s.lens = at
            ref = tree.attention(*s.codec, *s.host, s.table, at, s.cu, first.parents, q[i].cpu().numpy(), B * T)
            check_attention(out[i], ref, "f32")
            for side in range(2):
                s.host[side], want = tree.keep(s.host[side], s.table, at, s.cu, paths)
                assert np.array_equal(s.pages[side].cpu().numpy(), s.host[side]), (i, side)
            assert s.status() == 0
        for x in lens_of[:-1]:
            assert x.tolist() == want
        at = [n + T for n in want]
        assert lens.tolist() == at


# ------------------------------------------------------------------------------ verification

class FixedWalks(Walks):
    """Walks compared with the walk in the kernel's own numbers, which large vocabularies are quick in."""

    def check(self, ctx):
        path, n, nxt = self.run(ctx)
        assert lib().tq_ctx_device_status(ctx) == 0
        for b, m in enumerate(self.new):
            rows = slice(int(self.cu[b]), int(self.cu[b]) + m)
            want = ([], -1) if m == 0 else tree.verify_fixed(
                list(self.parents[rows]), self.tokens[rows], self.host[0][rows], self.u[rows], self.u_next[b],
                None if self.host[1] is None else self.host[1][rows])
            assert (list(path[b, :n[b]]), nxt[b]) == want, b
            assert np.all(path[b, n[b]:self.max_q] == -1) and np.all(path[b, self.max_q:] == -5)


@pytest.mark.parametrize("draft", [True, False], ids=["draft", "no-draft"])
@pytest.mark.parametrize("B, dtype", [(30, "bf16"), (20, "f32"), (38, "f16"), (45, "f32"), (90, "bf16"), (170, "f16"), (400, "f32")])
def test_verify_every_cluster_size(B, dtype, draft):
    """Sequences that take clusters of 8 (20 to 38 of them), 4, 2 and 1 CTAs on 152 SMs, with a draft's rows and without."""
    ctx = lib().Ctx("turbo4")
    w = FixedWalks([4, 0, 1, 7] * (B // 4) + [3] * (B % 4), 1203, dtype, B, draft, 3, pad=2)
    assert len(w.new) == B
    w.check(ctx)


@pytest.mark.parametrize("draft, dtype", [(True, "f32"), (True, "bf16"), (False, "f16"), (False, "f32")])
def test_verify_vocabularies_past_131072(draft, dtype):
    ctx = lib().Ctx("turbo4")
    for V, new in ((151936, [5, 2]), (262145, [4]), (1000003, [2])):
        FixedWalks(new, V, dtype, V, draft, 3).check(ctx)


@pytest.mark.parametrize("draft", [True, False], ids=["draft", "no-draft"])
def test_verify_weights_next_to_its_whole_multiples(draft):
    """Weights of 2^-75 to 2^-30 beside one of nearly all, and random numbers as small: tests and draws that turn
    on the last of the 62 bits."""
    import torch
    ctx = lib().Ctx("turbo4")
    other = 0
    for seed in range(6):
        rng = np.random.default_rng(seed)
        w = FixedWalks([7, 4, 9], 97, "f32", seed, draft, 3)
        rows = [np.exp2(rng.uniform(-75, -30, (w.n, 97))).astype(np.float32) for _ in range(2)]
        for x in rows:
            x[:, 5] = 1 - 2.0 ** -20
        w.host = (rows[0], rows[1] if draft else None)
        w.tokens[:] = rng.integers(0, 97, w.n)
        w.u[:] = np.exp2(rng.uniform(-70, -20, w.n))
        w.u_next[:] = np.exp2(rng.uniform(-64, -40, w.B))
        w.target.copy_(torch.from_numpy(rows[0]))
        if draft:
            w.draft.copy_(torch.from_numpy(rows[1]))
        for at, x in ((1, w.tokens), (3, w.u), (4, w.u_next)):
            w.d[at].copy_(torch.from_numpy(x))
        w.check(ctx)
        for b, m in enumerate(w.new):
            r = slice(int(w.cu[b]), int(w.cu[b]) + m)
            args = (list(w.parents[r]), w.tokens[r], rows[0][r], w.u[r], w.u_next[b], rows[1][r] if draft else None)
            other += tree.verify(*args) != tree.verify_fixed(*args)
    assert other  # the inputs reach what the rounding decides


def test_verify_refuses_vocabularies_past_its_rows_strides():
    """2^31 - 1 tokens would pass the groups' 32-bit counts: a row's stride, at least the vocabulary, is at most 2^29."""
    import torch
    tq = lib()
    w = Walks([3], 40, "f32", 3, True, 1)
    ctx = tq.Ctx("turbo4")
    for V, stride in ((2 ** 31 - 1, 2 ** 31 - 1), (2 ** 29 + 1, 2 ** 29 + 1), (40, 2 ** 29 + 1)):
        p = tq.tq_probs(w.target.data_ptr(), 0, V, stride)
        st = tq.lib.tq_tree_verify(ctx.handle, w.batch.ref, w.d[0].data_ptr(), w.d[1].data_ptr(), ctypes.byref(p), None, w.d[3].data_ptr(),
                                   w.d[4].data_ptr(), w.out[0].data_ptr(), 5, w.out[1].data_ptr(), w.out[2].data_ptr(), None)
        assert st == tq.TQ_ERR_INVALID_ARG
    torch.cuda.synchronize()
    assert all(torch.all(x == -5) for x in w.out) and tq.tq_ctx_device_status(ctx) == 0


# ------------------------------------------------------------------------------ attention

def columns(s, Hq):
    n = ctypes.c_int32(-1)
    assert s.tq.lib.tq_test_tree_columns(*(c.handle for c in s.ctx), s.kv.ref, s.batch.ref, Hq, ctypes.byref(n)) == s.tq.TQ_OK
    return n.value


def test_which_units_a_batch_takes():
    """The batches that stand for units of 64 columns take them, and the smaller ones units of 32; single nodes the decode."""
    tq = lib()
    for lens, new, Hq, Hkv, P, pad, wide in ATTENTION:
        cols = max(new) * Hq // Hkv
        if cols > 32:
            assert columns(FullTrees(tq, lens, new, Hkv, P, 11, wide, pad=pad, fill=False), Hq) == 64
        small = columns(Trees(tq, lens, new, Hkv, P, 11, wide, pad=pad, fill=False), Hq)
        assert small == (0 if max(new) == 1 else 64 if Hq // Hkv > 32 else 32) or cols > 32
    for lens, new, Hq in (([700, 260], [10, 12], 8), ([1500, 300], [6, 9], 24), ([231], [20], 6)):
        assert columns(FullTrees(tq, lens, new, 2, 32, 1, fill=False), Hq) == 64


@pytest.mark.parametrize("out_dtype", ["bf16", "f16", "f32"])
def test_long_contexts_in_units_of_64_columns(out_dtype):
    for P, Hq, lens, new in ((16, 8, [9000, 14000], [20, 11]), (128, 16, [20000], [9])):
        s = FullTrees(lib(), lens, new, 2, P, 13)
        assert columns(s, Hq) == 64
        got, ref = run_tree(s, Hq, "bf16", out_dtype, 128)
        check_attention(got, ref, out_dtype, f"p{P}")


def bound(s, q32, Hq, out_dtype):
    """fp64 [n, Hq]: how far a row may be off, from A = sum_t w_t |v_t| and the roundings on the way.  A score is off by at
    most d = scale |q| max|k| (c + e + r): c the fp16 centroids' relative error, e that of q's parts (one fp16: 2^-11 of an
    element and 2^-25 at least beside a largest of 2^-8, sqrt(128) of them: 2^-13; two: 2^-25 beside 2^-4, 2^-17), r = 2^-15
    for R in two bf16 parts with one product left out; weights move by factors in [exp(-2d), exp(2d)].  A weight times its value's norm is one fp16
    (2^-11) or two (2^-20) whose largest of the row lies at 2^7 and more, the smallest step 2^-24: 2^-31 a key of the
    largest term.  Centroids c and R r once more; 2^-18 for exponentials and fp32 sums over up to 1,000 keys."""
    two = out_dtype != "bf16"
    g, n = Hq // s.Hkv, s.n
    c = max(centroid_error(x) for x in s.codec)
    out = np.zeros((n, Hq))
    for b, length in enumerate(s.lens):
        a, e = int(s.cu[b]), int(s.cu[b + 1])
        K, V = (paged.dequantize(x, paged.sequence_rows(h, s.table, b, length)) for x, h in zip(s.codec, s.host))
        kn, vn = (np.repeat(np.linalg.norm(x, axis=-1), g, axis=1) for x in (K, V))   # [length, Hq]
        ctx = length - (e - a)
        for i, line in enumerate(tree.lines(s.parents[a:e])):
            at = list(range(ctx)) + [ctx + j for j in line]
            x = q32[a + i].astype(np.float64)
            sc = np.einsum("hd,thd->ht", x, np.repeat(K[at], g, axis=1)) / np.sqrt(128)
            w = np.exp(sc - sc.max(1, keepdims=True))
            w /= w.sum(1, keepdims=True)
            terms = w * vn[at].T
            d = np.linalg.norm(x, axis=-1) * kn[at].max(0) / np.sqrt(128) * (c + (2.0 ** -17 if two else 2.0 ** -11 + 2.0 ** -13) + 2.0 ** -15)
            rel = np.expm1(2 * d) + (2.0 ** -20 if two else 2.0 ** -11) + c + 2.0 ** -15 + 2.0 ** -18
            out[a + i] = rel * terms.sum(1) + 2.0 ** -31 * len(at) * terms.max(1)
    return out


@pytest.mark.parametrize("keys", [1.0, 8.0])
@pytest.mark.parametrize("out_dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("kind", [Trees, FullTrees], ids=["32", "64"])
def test_value_norms_of_a_wide_range_row_by_row(kind, out_dtype, keys):
    """Small values alone; small ones first and large ones tiles later; the other way round; none at first; norms that
    rise and fall within 32 keys.  Every row is held to its own size, so that a row of small values counts as much as
    one of large ones."""
    tq = lib()
    Hq, Hkv = 8, 2
    s = kind(tq, [700, 300, 450], [10, 12, 9] if kind is FullTrees else [8, 7, 3], Hkv, 32, 103, rot=("wht", "dense"))
    assert columns(s, Hq) == (64 if kind is FullTrees else 32)
    low = -12 if out_dtype == "f16" else -40
    for b, h, norm in ((0, 0, lambda t: 2.0 ** (low + t % 5)), (0, 1, lambda t: 2.0 ** (low if t < 390 else 8)),
                       (1, 0, lambda t: 2.0 ** (8 if t < 140 else low)), (1, 1, lambda t: 0.0 if t < 200 else 2.0 ** low),
                       (2, 0, lambda t: 2.0 ** (t % 32 - 16)), (2, 1, lambda t: 2.0 ** (8 if t >= 447 else low))):
        set_norms(s, 1, {(b, h, t): norm(t) for t in range(s.lens[b])})
        set_norms(s, 0, {(b, h, t): keys * 2.0 ** ((5 * t) % 6 - 3) for t in range(s.lens[b])})
    got, ref = run_tree(s, Hq, "f32", out_dtype)
    got, ref = got.float().cpu().numpy().astype(np.float64)[:s.n], ref[:s.n]
    step = 2.0 ** -25 * np.sqrt(128) if out_dtype == "f16" else 0.0
    err = np.linalg.norm(got - ref, axis=-1)
    tol = bound(s, s.q32, Hq, out_dtype) + HALF[out_dtype] * np.linalg.norm(ref, axis=-1) * 1.01 + step
    assert np.all(err <= tol), np.max(err / tol)
