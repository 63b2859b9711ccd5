"""Drafted trees over the paged cache on the GPU (append, attention, verification, kept paths) against
the fp64 oracle, their refusals and device flags, and steps of the calls together."""

import ctypes

import numpy as np
import pytest

from gpu_util import BAND, band_ok, lib
from oracle import paged, tree
from oracle.formats import unpack_turbo4
from test_gpu_paged import Setup, check_attention, check_sharp, device_rows, dt

pytestmark = pytest.mark.gpu


def random_tree(rng, n, wide):
    return [-1] + [int(rng.integers(max(0, i - wide), i)) for i in range(1, n)]


class Trees(Setup):
    """Setup whose rows are nodes: `wide` nodes back at most is a node's parent (0: only roots)."""

    def __init__(self, tq, lens, new, Hkv, P, seed, wide=4, **kw):
        import torch
        super().__init__(tq, lens, new, Hkv, P, seed, **kw)
        self.parents = np.full(self.n_rows, -9, np.int32)  # (padding holds no parent)
        for b, t in enumerate(new):
            self.parents[self.cu[b]:self.cu[b + 1]] = random_tree(self.rng, t, wide) if wide and t else -1
        self.batch = tq.PagedBatch(self.d_lens, torch.from_numpy(self.cu).cuda(), max(max(new), 1), self.n_rows)
        self.d_parents = torch.from_numpy(self.parents).cuda()

    def tree_workspace(self, Hq):
        import torch
        n = self.tq.tq_paged_tree_workspace_size(*self.ctx, self.kv, self.batch, Hq)
        return torch.full((max(n, 256),), 255, dtype=torch.uint8, device="cuda")  # no initialisation needed

    def tree_oracle(self, q32, turn=None, scale=0.0):
        return tree.attention(*self.codec, *self.host, self.table, self.lens, self.cu, self.parents[:self.n], q32,
                              self.n_rows, scale, turn)


def run_tree(s, Hq, dtype, out_dtype, rot_dim=0, interleaved=False, strided=False, scale=0.0, mul=1.0):
    import torch
    x = s.rng.standard_normal((s.n_rows, 3 * Hq if strided else Hq, 128)) * mul
    t, x32 = device_rows(x, dtype)
    q, q32 = (t[:, Hq:2 * Hq], x32[:, Hq:2 * Hq]) if strided else (t, x32)
    rope, turn = s.rope(rot_dim, interleaved)
    out = torch.full((s.n_rows, Hq, 128), 7.0, dtype=dt(out_dtype), device="cuda")
    s.tq.tq_paged_tree_attention(*s.ctx, s.kv, s.batch, s.d_parents, q, out, s.tree_workspace(Hq), rope=rope, scale=scale)
    assert s.status() == 0
    s.q32 = q32
    return out, s.tree_oracle(q32, turn, scale)


# ------------------------------------------------------------------------------ append

@pytest.mark.parametrize("rot", [("wht", "wht"), ("dense", "dense"), ("wht", "dense")], ids="/".join)
@pytest.mark.parametrize("case", [
    # lens, nodes, Hkv, P, dtype, rot_dim, interleaved, pad, strided, wide
    ([5], [5], 1, 16, "f32", 128, False, 0, False, 2),
    ([1, 700, 64], [1, 9, 64], 8, 64, "bf16", 128, False, 0, True, 5),
    ([33, 17, 0, 250], [33, 2, 0, 128], 3, 16, "f16", 64, True, 5, False, 1),  # chains, the longest of 128
    ([40, 3, 129], [7, 5, 129], 2, 32, "bf16", 64, False, 1, True, 3),  # a sequence shorter than its nodes
    ([900, 333, 90], [128, 100, 90], 8, 32, "bf16", 32, True, 3, False, 16),  # dense rotations in 16-row tiles
    ([70], [30], 2, 16, "f16", 0, False, 0, False, 4),
], ids=lambda c: f"{c[4]}-p{c[3]}-r{c[5]}{'i' if c[6] else ''}-h{c[2]}")
def test_append_turns_keys_by_their_nodes_positions(case, rot):
    tq = lib()
    lens, new, Hkv, P, dtype, rot_dim, inter, pad, strided, wide = case
    s = Trees(tq, lens, new, Hkv, P, 1, wide, rot=rot, pad=pad, fill=False)
    if max(new) > 128:  # (the append takes any number; the batch says 128 at most)
        s.batch.c.max_q = 128
    width = 3 * Hkv if strided else Hkv
    t, x32 = device_rows(s.rng.standard_normal((s.n_rows, width, 128)) * 3, dtype)
    u, y32 = device_rows(s.rng.standard_normal((s.n_rows, width, 128)), dtype)
    k, k32 = (t[:, Hkv:2 * Hkv], x32[:, Hkv:2 * Hkv]) if strided else (t, x32)
    v, v32 = (u[:, :Hkv], y32[:, :Hkv]) if strided else (u, y32)
    rope, turn = s.rope(rot_dim, inter)
    tq.tq_paged_tree_append(*s.ctx, s.kv, s.batch, s.d_parents, k, v, rope=rope)
    assert s.status() == 0
    at, _ = paged.places(lens, s.cu)
    rows, seq, slot = (np.array(c, int) for c in zip(*at))
    pos = np.maximum(tree.positions(lens, s.cu, s.parents[:s.n])[rows], 0)
    k32 = turn(k32[rows], pos) if turn else k32[rows]
    for i, x in enumerate((k32, v32[rows])):
        rec, info = s.codec[i].encode(np.ascontiguousarray(x.reshape(-1, 128), np.float32))
        want = s.host[i].copy()
        want[s.table[seq, slot // P], :, slot % P] = rec.reshape(len(rows), Hkv, 68)
        got = s.pages[i].cpu().numpy()
        if rot[i] == "wht":
            assert np.array_equal(got, want)
            continue
        n1, idx1 = unpack_turbo4(got[s.table[seq, slot // P], :, slot % P].reshape(-1, 68))
        n0, idx0 = unpack_turbo4(rec)
        assert np.array_equal(n1, n0)
        ok, n_diff = band_ok(idx1, idx0, info["y"], s.codec[i].b32, BAND)
        assert ok, n_diff


# ------------------------------------------------------------------------------ attention

ATTENTION = [
    # lens, nodes, Hq, Hkv, P, pad, wide
    ([1], [1], 1, 1, 16, 0, 4),
    ([5], [5], 2, 1, 16, 0, 0),                       # roots alone, no context
    ([600], [8], 8, 2, 64, 0, 4),
    ([127, 128, 129, 257], [3, 4, 1, 2], 8, 2, 16, 0, 2),   # ends about a tile of keys
    ([300, 0, 77, 1, 512], [7, 1, 0, 1, 20], 12, 2, 32, 5, 3),  # idle slots, a sequence without rows, padding
    ([200, 3], [128, 3], 4, 4, 16, 1, 16),            # the widest tree, trees that hold the whole sequence
    ([2500, 40], [33, 40], 16, 2, 128, 0, 1),         # chains; several units of a sequence
    ([900], [64], 24, 2, 256, 0, 8),                  # twelve heads per KV head
    ([130, 70], [2, 1], 64, 1, 32, 0, 1),             # 64 heads per KV head
    ([20, 350], [24, 90], 6, 3, 16, 2, 5),            # a sequence shorter than its nodes
    ([3000, 1, 2999, 17], [6, 1, 5, 6], 32, 8, 64, 0, 4),
    ([180] * 40, [5] * 40, 10, 2, 16, 0, 2),          # five heads per KV head, many short sequences
]


@pytest.mark.parametrize("out_dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("case", ATTENTION, ids=lambda c: f"t{max(c[1])}-n{max(c[0])}-h{c[2]}x{c[3]}-p{c[4]}")
def test_attention(case, out_dtype):
    lens, new, Hq, Hkv, P, pad, wide = case
    rot = ("dense", "wht") if Hq % 3 else ("wht", "dense")
    s = Trees(lib(), lens, new, Hkv, P, 11, wide, rot=rot, pad=pad)
    got, ref = run_tree(s, Hq, {"bf16": "bf16", "f16": "f32", "f32": "f16"}[out_dtype], out_dtype,
                        rot_dim=[128, 64, 32, 0][len(lens) % 4], interleaved=bool(Hq % 4), strided=bool(pad))
    check_attention(got, ref, out_dtype)


def test_attention_over_long_contexts():
    """Contexts that several CTAs share, of several page sizes."""
    tq = lib()
    for P, Hq, t, lens in ((16, 8, 4, [9000, 14000]), (64, 4, 20, [20000]), (256, 8, 16, [5000, 16, 7001])):
        s = Trees(tq, lens, [min(t, n) for n in lens], 2, P, 13)
        for dtype in ("bf16", "f16"):
            got, ref = run_tree(s, Hq, dtype, dtype, 128)
            check_attention(got, ref, dtype, f"p{P} {dtype}")


def test_attention_of_few_sequences_among_idle_slots():
    """Sequences hundreds of slots apart, more than a warp looks at together, and two that share their context's pages."""
    import torch
    rng = np.random.default_rng(5)
    new, lens = [0] * 300, [0] * 300
    for b in (3, 31, 32, 33, 131, 299):
        new[b] = int(rng.integers(1, 9))
        lens[b] = new[b] + int(rng.integers(0, 700))
    lens[40] = 33  # without rows
    for od in ("bf16", "f32"):
        lens[31] = lens[32] = 256 + max(new)
        s = Trees(lib(), lens, new, 2, 64, 19)
        s.table[32, :4] = s.table[31, :4]
        s.kv = s.tq.PagedKV(*s.pages, torch.from_numpy(s.table).cuda(), 64, 2)
        got, ref = run_tree(s, 8, "bf16", od, 64)
        check_attention(got, ref, od)


@pytest.mark.parametrize("Hq", [2, 8, 24])
def test_scores_in_the_hundreds(Hq):
    """Sharp softmax: the running maximum rises from tile to tile and between CTAs."""
    s = Trees(lib(), [1500, 300], [6, 9], 2, 32, 17)
    got, ref = run_tree(s, Hq, "f32", "f32", 64, scale=3.0)
    check_sharp(s, got, ref, s.q32, 3.0, "sharp")
    got, ref = run_tree(s, Hq, "f32", "f32", 64, scale=-1e-3)
    check_attention(got, ref, "f32", "flat")


@pytest.mark.parametrize("out_dtype", ["bf16", "f16"])
def test_norms_out_of_the_ordinary(out_dtype):
    """Keys and values of very large and very small norms, zero norms; a row of q of zeros; every row's
    weights are compared where they decide."""
    import torch
    s = Trees(lib(), [700, 260], [10, 12], 2, 16, 19)
    rng = np.random.default_rng(5)
    for i, powers in ((0, [-20, -3, 0, 1]), (1, [-30, -10, 0, 8])):
        nat = s.host[i][..., :4].copy().view("<f4")
        scale = rng.choice(np.exp2(np.array(powers, np.float32)), nat.shape).astype(np.float32)
        scale[rng.random(nat.shape) < 0.05] = 0
        held = np.isfinite(nat)
        nat[held] *= scale[held]
        s.host[i][..., :4] = nat.view(np.uint8)
        s.pages[i].copy_(torch.from_numpy(s.host[i]))
    got, ref = run_tree(s, 8, "f32", out_dtype)
    got, ref = got.float().cpu().numpy()[:s.n], ref[:s.n]
    half = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}[out_dtype]
    big = max(np.abs(ref).max(), 1.0)  # outputs are sums of values of up to 2^8 the ordinary norm: the stated 2e-3 grows with it
    assert np.all(np.isfinite(got)) and np.max(np.abs(got - ref) - half * np.abs(ref)) <= 2e-3 * big


class FullTrees(Trees):
    """A batch whose sizes allow full trees over a million tokens: past 32 columns, units of 64."""

    def __init__(self, tq, lens, new, Hkv, P, seed, wide=4, pad=0, **kw):
        full = len(lens) * max(max(new), 1) - sum(new)
        super().__init__(tq, lens, new, Hkv, P, seed, wide, pad=max(pad, full), width=(1 << 20) // P, **kw)


@pytest.mark.parametrize("out_dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("case", [c for c in ATTENTION if max(c[1]) * c[2] // c[3] > 32],
                         ids=lambda c: f"t{max(c[1])}-n{max(c[0])}-h{c[2]}x{c[3]}-p{c[4]}")
def test_attention_in_units_of_64_columns(case, out_dtype, monkeypatch):
    monkeypatch.setitem(globals(), "Trees", FullTrees)
    test_attention(case, out_dtype)


@pytest.mark.parametrize("again", [test_attention_over_long_contexts, lambda: test_scores_in_the_hundreds(8),
                                   lambda: test_scores_in_the_hundreds(24),
                                   lambda: test_norms_out_of_the_ordinary("bf16"),
                                   lambda: test_norms_out_of_the_ordinary("f16")],
                         ids=["long", "sharp-8", "sharp-24", "norms-bf16", "norms-f16"])
def test_hard_inputs_in_units_of_64_columns(again, monkeypatch):
    monkeypatch.setitem(globals(), "Trees", FullTrees)
    again()


@pytest.mark.parametrize("out_dtype", ["bf16", "f16"])
def test_nan_norms_in_units_of_64_columns(out_dtype):
    """60 columns in one unit; a node's value (or key) is NaN: its own columns and its descendants', no other."""
    import torch
    s = FullTrees(lib(), [231], [20], 2, 32, 29, wide=6)
    clean, _ = run_tree(s, 6, "bf16", out_dtype)
    seen = [set() for _ in range(20)]
    for i, p in enumerate(s.parents[:20].tolist()):
        seen[i] = {i} | (seen[p] if p >= 0 else set())
    rows = torch.from_numpy(s.q32).bfloat16().cuda()
    for side in (0, 1):
        for node in (0, 3, 11, 19):
            pages = [p.clone() for p in s.pages]
            t = 211 + node
            pages[side][int(s.table[0, t // 32]), 1, t % 32, :4] = torch.tensor([0, 0, 192, 127], dtype=torch.uint8)
            out = torch.empty_like(clean)
            s.tq.tq_paged_tree_attention(*s.ctx, s.tq.PagedKV(*pages, s.kv.block_table, 32, 2), s.batch, s.d_parents, rows,
                                         out, s.tree_workspace(6))
            hit = [i for i in range(20) if node in seen[i]]
            keep = [i for i in range(20) if node not in seen[i]]
            assert not torch.isfinite(out[hit][:, 3:]).any(-1).any() and torch.equal(out[:20, :3], clean[:20, :3])
            assert torch.equal(out[keep], clean[keep])
    assert s.status() == 0


def test_nan_norms_reach_the_nodes_that_see_them():
    import torch
    s = Trees(lib(), [200, 150], [6, 3], 2, 16, 23, fill=True)
    s.parents[:6] = [-1, 0, 0, 1, 2, 3]
    s.d_parents.copy_(torch.from_numpy(s.parents))
    clean, _ = run_tree(s, 4, "bf16", "bf16")
    for side in (0, 1):
        for node, hit in ((2, {2, 4}), (1, {1, 3, 5}), (4, {4})):
            pages = [p.clone() for p in s.pages]
            t = 194 + node
            pages[side][int(s.table[0, t // 16]), 1, t % 16, :4] = torch.tensor([0, 0, 192, 127], dtype=torch.uint8)
            kv = s.tq.PagedKV(*pages, s.kv.block_table, 16, 2)
            rows = torch.from_numpy(s.q32).bfloat16().cuda()
            out = torch.empty((9, 4, 128), dtype=torch.bfloat16, device="cuda")
            s.tq.tq_paged_tree_attention(*s.ctx, kv, s.batch, s.d_parents, rows, out, s.tree_workspace(4))
            bad = {int(i) for i in (~torch.isfinite(out)).any(-1)[:, 2:].any(-1).nonzero()[:, 0]}
            assert bad == hit
            assert torch.equal(out[:, :2], clean[:, :2])
            keep = [i for i in range(9) if i not in hit]
            assert torch.equal(out[keep], clean[keep])
    assert s.status() == 0


def test_a_single_node_is_a_decode_row():
    """T = 1: the same bits as tq_paged_attention of single rows."""
    import torch
    s = Trees(lib(), [900, 30, 0], [1, 1, 1], 2, 16, 29)
    got, ref = run_tree(s, 8, "bf16", "bf16", 128)
    check_attention(got, ref, "bf16")
    rope, _ = s.rope(128, False)
    q = torch.from_numpy(s.q32).bfloat16().cuda()
    out = torch.empty_like(got)
    s.tq.tq_paged_attention(*s.ctx, s.kv, s.batch, q, out, s.workspace(8), rope=rope)
    assert torch.equal(out, got)


def test_parents_out_of_order_are_flagged():
    """Such a node follows the context; the others are as they were."""
    import torch
    s = Trees(lib(), [100, 60], [5, 4], 2, 16, 31, wide=1)
    good, _ = run_tree(s, 4, "bf16", "bf16", 64)
    q, rope = torch.from_numpy(s.q32).bfloat16().cuda(), s.rope(64, False)[0]
    for node, bad in ((3, 3), (3, 4), (3, -2), (3, 2 ** 31 - 1), (3, -2 ** 31), (0, 0)):
        s.d_parents.copy_(torch.from_numpy(s.parents))
        s.d_parents[node] = bad
        out = torch.full_like(good, 7.0)
        s.tq.tq_paged_tree_attention(*s.ctx, s.kv, s.batch, s.d_parents, q, out, s.tree_workspace(4), rope=rope)
        assert s.status() == 7
        s.d_parents[node] = -1
        want = torch.full_like(good, 7.0)
        s.tq.tq_paged_tree_attention(*s.ctx, s.kv, s.batch, s.d_parents, q, want, s.tree_workspace(4), rope=rope)
        assert s.status() == 0 and torch.equal(out, want)
        k = torch.randn((9, 2, 128), device="cuda")
        s.d_parents[node] = bad
        s.tq.tq_paged_tree_append(*s.ctx, s.kv, s.batch, s.d_parents, k, k, rope=rope)
        assert s.status() == 7
        for p, h in zip(s.pages, s.host):
            p.copy_(torch.from_numpy(h))


def test_bad_pages_and_lengths_are_flagged():
    import torch
    s = Trees(lib(), [40, 30], [4, 3], 2, 16, 37)
    want, _ = run_tree(s, 4, "f32", "f32")
    q, ws = torch.from_numpy(s.q32).cuda(), s.tree_workspace(4)
    for bad in (-1, s.n_pages, 2 ** 31 - 1):
        t = s.kv.block_table.clone()
        t[1, 1] = bad
        out = torch.full_like(want, 7.0)
        s.tq.tq_paged_tree_attention(*s.ctx, s.tq.PagedKV(*s.pages, t, 16, 2), s.batch, s.d_parents, q, out, ws)
        assert s.status() == 5 and torch.equal(out[:4], want[:4])
    for n in (-3, 49):
        s.d_lens[1] = n
        out = torch.full_like(want, 7.0)
        s.tq.tq_paged_tree_attention(*s.ctx, s.kv, s.batch, s.d_parents, q, out, ws)
        assert s.status() in ((2, 5) if n > 0 else (2,)) and torch.equal(out[:4], want[:4])
        assert n > 0 or torch.all(out[4:] == 0)
    s.d_lens[1] = 30
    s.batch.c.max_q = 3  # the first sequence's last node is left out
    out = torch.full_like(want, 7.0)
    s.tq.tq_paged_tree_attention(*s.ctx, s.kv, s.batch, s.d_parents, q, out, ws)
    assert s.status() == 2 and torch.equal(out[:3], want[:3]) and torch.equal(out[4:], want[4:])


# ------------------------------------------------------------------------------ verification

class Walks:
    def __init__(self, new, V, dtype, seed, draft=True, wide=2, pad=0, stride=None, sharp=2.0):
        import torch
        rng = np.random.default_rng(seed)
        self.B, self.V, self.new = len(new), V, new
        self.cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        self.n = int(self.cu[-1]) + pad
        self.parents = np.full(self.n, -1, np.int32)
        self.tokens = rng.integers(0, V, self.n).astype(np.int32)
        logits = sharp * rng.standard_normal((self.n, V))
        near = logits + 0.8 * rng.standard_normal((self.n, V))
        soft = lambda x: np.exp(x - x.max(-1, keepdims=True)) / np.exp(x - x.max(-1, keepdims=True)).sum(-1, keepdims=True)  # noqa: E731
        wide_rows = np.zeros((2, self.n, stride or V))
        wide_rows[..., :V] = soft(logits), soft(near)
        wide_rows[..., V:] = np.nan
        t = [torch.from_numpy(x.astype(np.float32)).to(dt(dtype)).cuda()[:, :V] for x in wide_rows]
        self.target, self.draft = t[0], t[1] if draft else None
        p, q = (x.float().cpu().numpy() for x in t)
        self.host = (p, q if draft else None)
        for b, m in enumerate(new):
            lo = self.cu[b]
            if m:
                self.parents[lo:lo + m] = random_tree(rng, m, wide)
            for i in range(1, m):
                row = soft(near)[lo + self.parents[lo + i]]
                self.tokens[lo + i] = rng.choice(V, p=row) if draft else np.argsort(-row)[min(i, V) - 1]
        self.u, self.u_next = rng.random(self.n).astype(np.float32), rng.random(self.B).astype(np.float32)
        ints = lambda x: torch.from_numpy(np.asarray(x, np.int32)).cuda()  # noqa: E731
        self.max_q = max(max(new), 1)
        self.batch = lib().PagedBatch(ints(np.zeros(self.B)), ints(self.cu), self.max_q, self.n)
        self.d = [ints(self.parents), ints(self.tokens), self.target, torch.from_numpy(self.u).cuda(),
                  torch.from_numpy(self.u_next).cuda()]
        self.out = [torch.full((self.B, self.max_q + 2), -5, dtype=torch.int32, device="cuda"),
                    torch.full((self.B,), -5, dtype=torch.int32, device="cuda"),
                    torch.full((self.B,), -5, dtype=torch.int32, device="cuda")]

    def run(self, ctx):
        import torch
        lib().tq_tree_verify(ctx, self.batch, *self.d, *self.out, draft=self.draft)
        torch.cuda.synchronize()
        return [x.cpu().numpy() for x in self.out]

    def check(self, ctx, status=0):
        path, n, nxt = self.run(ctx)
        assert lib().tq_ctx_device_status(ctx) == status
        depth = 0
        for b, m in enumerate(self.new):
            rows = slice(int(self.cu[b]), int(self.cu[b]) + m)
            if m == 0:
                want, w = [], -1
            else:
                want, w = tree.verify(list(self.parents[rows]), self.tokens[rows], self.host[0][rows], self.u[rows],
                                      self.u_next[b], None if self.host[1] is None else self.host[1][rows])
            assert n[b] == len(want) and list(path[b, :len(want)]) == want, b
            assert np.all(path[b, len(want):self.max_q] == -1) and np.all(path[b, self.max_q:] == -5)
            assert nxt[b] == w, b
            depth = max(depth, len(want))
        return depth


@pytest.mark.parametrize("draft", [True, False], ids=["draft", "no-draft"])
@pytest.mark.parametrize("case", [
    # nodes, vocab, dtype, wide, pad, stride
    ([1], 1, "f32", 1, 0, None),
    ([2, 1], 2, "f32", 1, 0, None),
    ([5, 0, 3, 8], 33, "f32", 2, 3, 40),
    ([6] * 9, 257, "bf16", 3, 0, None),
    ([12, 1, 7], 1000, "f16", 4, 1, 1003),
    ([9, 4], 5003, "f32", 8, 0, 5004),
    ([128, 40], 300, "f32", 40, 2, None),
    ([16, 16, 16], 4099, "bf16", 1, 0, None),
], ids=lambda c: f"t{max(c[0])}-v{c[1]}-{c[2]}")
def test_verify(case, draft):
    new, V, dtype, wide, pad, stride = case
    ctx = lib().Ctx("turbo4")
    for seed in range(4):
        Walks(new, V, dtype, seed, draft, wide, pad, stride).check(ctx)


def test_verify_many_sequences_and_rows_that_lie_differently():
    """A CTA per sequence and every smaller cluster on the way; the draft's rows start elsewhere than the target's
    do within 16 bytes, the vocabulary's last group is short."""
    import torch
    ctx = lib().Ctx("turbo4")
    for B, dtype in ((700, "bf16"), (170, "f32"), (90, "f16"), (45, "bf16")):
        w = Walks([4, 0, 1, 2] * (B // 4) + [3] * (B % 4), 203, dtype, B, True, 2)
        held = w.draft.clone()
        for at in (1, 5):
            wide = torch.full((w.n, 209), float("nan"), dtype=held.dtype, device="cuda")
            w.draft = wide[:, at:at + 203]
            w.draft.copy_(held)
            w.check(ctx)


def test_verify_large_vocabularies():
    """Slices of several rounds per warp; residuals of several failed tests."""
    ctx = lib().Ctx("turbo4")
    w = Walks([4, 3], 60001, "f32", 3, True, 3)
    w.u[:] = 0.98  # most tests fail
    w.d[3].fill_(0.98)
    w.u[:] = w.d[3].cpu().numpy()
    w.check(ctx)
    Walks([3], 131072, "bf16", 5, True, 1).check(ctx)
    Walks([5], 100003, "f16", 6, False, 4).check(ctx)


def test_verify_follows_one_hot_targets_and_rows_without_weight():
    import torch
    ctx = lib().Ctx("turbo4")
    w = Walks([5], 50, "f32", 7, False, 1)
    choice = np.array([3, 11, 4, 20, 9])
    w.target.zero_()
    w.target[torch.arange(5), torch.from_numpy(choice)] = 1
    w.d[1].copy_(torch.tensor([0, 3, 11, 4, 21], dtype=torch.int32))
    path, n, nxt = w.run(ctx)
    assert list(path[0, :5]) == [0, 1, 2, 3, -1] and n[0] == 4 and nxt[0] == 20
    for rows in (0.0, float("nan"), -1.0):
        w.target.fill_(rows)
        path, n, nxt = w.run(ctx)
        assert n[0] == 1 and nxt[0] == -1
    w.target.fill_(5.0)  # counts as ones: sums past 2, no stated outcome but a token or -1
    path, n, nxt = w.run(ctx)
    assert -1 <= nxt[0] < 50 and 1 <= n[0] <= 5
    same = Walks([4], 40, "f32", 9, True, 3)  # the draft is the target: everything is taken
    same.draft.copy_(same.target)
    same.d[0].copy_(torch.tensor([-1, 0, 1, 2], dtype=torch.int32))
    path, n, nxt = same.run(ctx)
    assert n[0] == 4 and 0 <= nxt[0] < 40
    # random numbers of zero, and what lies outside [0, 1)
    w = Walks([6, 6, 6, 6], 97, "f32", 11, True, 2)
    for bad, good in ((float("nan"), 0.0), (-2.0, 0.0), (3.0, float(np.float32(1 - 2.0 ** -24)))):
        w.d[3].fill_(bad), w.d[4].fill_(bad)
        got = w.run(ctx)
        w.u[:] = good
        w.u_next[:] = good
        w.d[3].fill_(good), w.d[4].fill_(good)
        want = w.run(ctx)
        assert all(np.array_equal(a, b) for a, b in zip(got, want))
        w.check(ctx)
    assert lib().tq_ctx_device_status(ctx) == 0


@pytest.mark.parametrize("V", [3, 700])
def test_verify_keeps_a_residual_that_a_test_would_empty(V):
    """Rows that do not sum to 1: the first refused child leaves r = 1/4 on two tokens, the second one would leave
    nothing, so r stays and the next token is drawn from it."""
    import torch
    ctx = lib().Ctx("turbo4")
    w = Walks([3, 4], V, "f32", 16, True, 1)
    w.target.zero_(), w.draft.zero_()
    for t, rows in ((w.target, (0.75, 0.75, 0.125)), (w.draft, (0.5, 0.5, 0.5))):
        t[:, [0, V - 2, V - 1]] = torch.tensor(rows, device="cuda")
    w.host = (w.target.cpu().numpy(), w.draft.cpu().numpy())
    w.parents[:] = [-1, 0, 0, -1, 0, 0, 0]
    w.tokens[:] = V - 1
    w.u[:] = 0.9
    w.d[0].copy_(torch.from_numpy(w.parents)), w.d[1].copy_(torch.from_numpy(w.tokens)), w.d[3].fill_(0.9)
    for u in (0.25, 0.75):
        w.u_next[:] = u
        w.d[4].fill_(u)
        w.check(ctx)
        assert w.run(ctx)[2].tolist() == [0 if u < 0.5 else V - 2] * 2


def test_verify_flags_tokens_parents_and_too_many_nodes():
    import torch
    ctx = lib().Ctx("turbo4")
    w = Walks([6, 5], 64, "f32", 13, False, 2)
    for i, bad in ((1, 64), (2, -1), (3, 2 ** 31 - 1)):
        w.tokens[i] = bad
        w.d[1][i] = bad
    w.check(ctx, status=7)
    w = Walks([6, 5], 64, "f32", 14, True, 1)
    w.d[0][3] = 3  # its own parent: follows the context, reached from nowhere
    w.parents[3] = -1
    w.check(ctx, status=7)
    w = Walks([6, 5], 64, "f32", 15, True, 1)
    w.batch.c.max_q = 5
    path, n, nxt = w.run(ctx)
    assert lib().tq_ctx_device_status(ctx) == 2 and n[0] <= 5 and np.all(path[:, 5:] == -5)


def test_verify_without_offsets_draws_from_every_row():
    import torch
    tq = lib()
    ctx = tq.Ctx("turbo4")
    w = Walks([1] * 7, 1001, "f32", 17)
    want = w.run(ctx)
    w.batch = tq.PagedBatch(torch.zeros(7, dtype=torch.int32, device="cuda"))
    got = w.run(ctx)
    assert np.array_equal(got[2], want[2]) and np.all(got[1] == 1) and np.all(got[0][:, 0] == 0)


# ------------------------------------------------------------------------------ kept paths

def some_path(rng, parents):
    return tree.lines(parents)[int(rng.integers(len(parents)))]


@pytest.mark.parametrize("case", [
    # lens, nodes, Hkv, P, wide, pad
    ([9], [1], 1, 16, 1, 0),
    ([70, 300], [20, 64], 8, 16, 2, 3),
    ([40, 3, 0, 129, 0], [7, 5, 0, 128, 1], 2, 32, 1, 0),  # shorter than its nodes, without rows, idle
    ([400], [100], 3, 64, 1, 0),
    ([60, 61], [30, 30], 130, 16, 1, 0),  # more heads than a chunk holds
    ([200] * 50, [12] * 50, 2, 128, 3, 0),
], ids=lambda c: f"t{max(c[1])}-h{c[2]}-p{c[3]}")
@pytest.mark.parametrize("in_place", [False, True], ids=["lens", "in-place"])
def test_keep(case, in_place):
    import torch
    tq = lib()
    lens, new, Hkv, P, wide, pad = case
    s = Trees(tq, lens, new, Hkv, P, 41, wide, pad=pad, fill=False)
    for i, p in enumerate(s.pages):
        s.host[i] = s.rng.integers(0, 256, p.shape, dtype=np.uint8)
        p.copy_(torch.from_numpy(s.host[i]))
    width = s.batch.c.max_q + 3
    for turn in range(3):
        paths = []
        for b, t in enumerate(new):
            tr = list(s.parents[s.cu[b]:s.cu[b + 1]])
            paths.append([] if not t else (list(range(t)) if turn == 2 else some_path(s.rng, tr)))
            if turn == 1 and t:  # any ascending nodes
                paths[-1] = sorted(s.rng.choice(t, int(s.rng.integers(0, t + 1)), replace=False).tolist())
        d_path = torch.full((len(lens), width), -1, dtype=torch.int32)
        for b, x in enumerate(paths):
            d_path[b, :len(x)] = torch.tensor(x, dtype=torch.int32)
        n_path = torch.tensor([len(x) for x in paths], dtype=torch.int32).cuda()
        s.d_lens.copy_(torch.tensor(lens, dtype=torch.int32))
        new_lens = s.d_lens if in_place else torch.full_like(s.d_lens, -9)
        for p, h in zip(s.pages, s.host):
            p.copy_(torch.from_numpy(h))
        tq.tq_paged_tree_keep(*s.ctx, s.kv, s.batch, d_path.cuda(), n_path, new_lens)
        assert s.status() == 0
        for p, h in zip(s.pages, s.host):
            want, want_lens = tree.keep(h, s.table, lens, s.cu, paths)
            assert np.array_equal(p.cpu().numpy(), want)
        assert new_lens.tolist() == want_lens


def test_keep_of_sequences_cut_by_n_tokens():
    """Offsets past n_tokens: the slots are those that the append gives the rows."""
    import torch
    tq = lib()
    s = Trees(tq, [50, 40], [6, 5], 2, 16, 73)
    rows = torch.randn((11, 2, 128), device="cuda")
    s.batch.c.n_tokens = s.batch.n_tokens = 9
    tq.tq_paged_tree_append(*s.ctx, s.kv, s.batch, s.d_parents, rows, rows)
    held = [p.cpu().numpy() for p in s.pages]
    path = torch.tensor([[0, 5, 0, 0, 0, 0], [1, 2, 0, 0, 0, 0]], dtype=torch.int32, device="cuda")
    lens = torch.zeros_like(s.d_lens)
    tq.tq_paged_tree_keep(*s.ctx, s.kv, s.batch, path, torch.tensor([2, 2], dtype=torch.int32).cuda(), lens)
    assert s.status() == 0 and lens.tolist() == [46, 37]
    for p, h in zip(s.pages, held):
        want, _ = tree.keep(h, s.table, [50, 40], s.cu, [[0, 5], [1, 2]])
        assert np.array_equal(p.cpu().numpy(), want)


def test_keep_refuses_paths_out_of_order():
    import torch
    tq = lib()
    s = Trees(tq, [50, 40], [6, 5], 2, 16, 43)
    before = [p.clone() for p in s.pages]
    for bad, n in (([1, 1], 2), ([2, 1], 2), ([-1, 2], 2), ([0, 6], 2), ([0, 1], 7), ([0, 1], -1), ([0, 2 ** 31 - 1], 2)):
        path = torch.full((2, 8), 0, dtype=torch.int32)
        path[0, :2] = torch.tensor(bad, dtype=torch.int32)
        path[1, :3] = torch.tensor([0, 2, 3])
        n_path = torch.tensor([n, 3], dtype=torch.int32).cuda()
        lens = torch.zeros_like(s.d_lens)
        tq.tq_paged_tree_keep(*s.ctx, s.kv, s.batch, path.cuda(), n_path, lens)
        assert s.status() == 7 and lens.tolist() == [44, 38]
        for a, p, h in zip(before, s.pages, s.host):
            want, _ = tree.keep(h, s.table, [50, 40], s.cu, [[], [0, 2, 3]])
            assert np.array_equal(p.cpu().numpy(), want)
            p.copy_(a)
    t = s.kv.block_table.clone()
    t[0, 2] = -1  # slots 32 .. 47 of the first sequence: its nodes 0 .. 3
    path = torch.tensor([[0, 4, 5, 0, 0, 0], [1, 2, 0, 0, 0, 0]], dtype=torch.int32, device="cuda")
    lens = torch.zeros_like(s.d_lens)
    tq.tq_paged_tree_keep(*s.ctx, tq.PagedKV(*s.pages, t, 16, 2), s.batch, path,
                          torch.tensor([3, 2], dtype=torch.int32).cuda(), lens)
    assert s.status() == 5 and lens.tolist() == [47, 37]
    for p, h in zip(s.pages, s.host):
        want, _ = tree.keep(h, s.table, [50, 40], s.cu, [[], [1, 2]])
        assert np.array_equal(p.cpu().numpy(), want)


# ------------------------------------------------------------------------------ together

def test_speculative_steps_together_and_captured():
    """Steps of a captured graph (append, attention, verification, keep, lengths in place) leave the cache,
    the lengths and the outputs of eager ones, and the cache that plain appends of the accepted tokens leave."""
    import torch
    tq = lib()
    B, T, Hq, Hkv, P, V = 3, 7, 8, 2, 16, 61
    s = Trees(tq, [60, 33, 20], [T] * B, Hkv, P, 47, wide=3, fill=False, width=10)
    s.table[:] = s.rng.permutation(30).reshape(3, 10)
    pages = [torch.zeros((30, Hkv, P, 68), dtype=torch.uint8, device="cuda") for _ in range(2)]
    kv = tq.PagedKV(*pages, torch.from_numpy(s.table).cuda(), P, Hkv)
    rope, _ = s.rope(128, False, n_pos=160)
    gen = torch.Generator(device="cuda").manual_seed(3)
    rand = lambda *shape: torch.randn(shape, generator=gen, device="cuda")  # noqa: E731
    kv0 = [rand(sum(s.lens) - B * T, Hkv, 128).bfloat16() for _ in range(2)]
    ctx_lens = torch.tensor([n - T for n in s.lens], dtype=torch.int32, device="cuda")
    cu0 = torch.tensor(np.concatenate([[0], np.cumsum([n - T for n in s.lens])]), dtype=torch.int32, device="cuda")
    prompt = tq.PagedBatch(ctx_lens.clone(), cu0, 64, int(cu0[-1]))
    tq.tq_paged_append(*s.ctx, kv, prompt, *kv0, rope=rope)
    start = [p.clone() for p in pages]
    lens = s.d_lens
    batch = s.batch
    q, k, v = rand(B * T, Hq, 128).bfloat16(), rand(B * T, Hkv, 128).bfloat16(), rand(B * T, Hkv, 128).bfloat16()
    target, draft = (torch.softmax(2 * rand(B * T, V), -1) for _ in range(2))
    tokens = torch.zeros(B * T, dtype=torch.int32, device="cuda")
    u, u_next = torch.zeros(B * T, device="cuda"), torch.zeros(B, device="cuda")
    out = torch.zeros((B * T, Hq, 128), dtype=torch.bfloat16, device="cuda")
    path = torch.zeros((B, T), dtype=torch.int32, device="cuda")
    n_path, nxt = (torch.zeros(B, dtype=torch.int32, device="cuda") for _ in range(2))
    ws = s.tree_workspace(Hq)

    def step():
        tq.tq_paged_tree_append(*s.ctx, kv, batch, s.d_parents, k, v, rope=rope)
        tq.tq_paged_tree_attention(*s.ctx, kv, batch, s.d_parents, q, out, ws, rope=rope)
        tq.tq_tree_verify(s.ctx[0], batch, s.d_parents, tokens, target, u, u_next, path, n_path, nxt, draft=draft)
        tq.tq_paged_tree_keep(*s.ctx, kv, batch, path, n_path, lens)
        lens.add_(T)  # the next step's nodes

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    for p, x in zip(pages, start):
        p.copy_(x)
    lens.copy_(ctx_lens + T)
    rows, total = [[] for _ in range(B)], 0
    for i in range(6):
        for t in (q, k, v):
            t.copy_(rand(*t.shape))
        for t in (target, draft):
            t.copy_(torch.softmax(2 * rand(*t.shape), -1))
        draft.copy_((0.4 * draft + 0.6 * target))
        tokens.copy_(torch.multinomial(draft[(torch.arange(B * T, device="cuda") // T * T) + s.d_parents.clamp(min=0)], 1, generator=gen)[:, 0])
        u.copy_(torch.rand(B * T, generator=gen, device="cuda")), u_next.copy_(torch.rand(B, generator=gen, device="cuda"))
        held = [x.clone() for x in (*pages, lens)]
        graph.replay()
        torch.cuda.synchronize()
        replayed = [x.clone() for x in (*pages, lens, out, path, n_path, nxt)]
        for x, h in zip((*pages, lens), held):
            x.copy_(h)
        for x in (out, path, n_path, nxt):
            x.fill_(0)
        step()
        assert s.status() == 0
        assert all(torch.equal(a, b) for a, b in zip(replayed, (*pages, lens, out, path, n_path, nxt)))
        for b in range(B):
            at = path[b, :int(n_path[b])].long() + b * T
            rows[b].append((k[at].clone(), v[at].clone()))
            total += len(at)
            assert 0 <= int(nxt[b]) < V
    assert total > 6 * B  # drafted tokens were taken
    # the accepted rows appended plainly, a sequence's positions being its slots
    for p, x in zip(pages, start):
        p.copy_(x)
    kept = [p.clone() for p in replayed[:2]]
    n = [sum(len(x[0]) for x in r) for r in rows]
    cu = torch.tensor(np.concatenate([[0], np.cumsum(n)]), dtype=torch.int32, device="cuda")
    ends = ctx_lens + torch.tensor(n, dtype=torch.int32, device="cuda")
    plain = tq.PagedBatch(ends, cu, max(n), sum(n))
    tq.tq_paged_append(*s.ctx, kv, plain, *(torch.cat([x[i] for r in rows for x in r]) for i in (0, 1)), rope=rope)
    assert s.status() == 0
    for b, e in enumerate(ends.tolist()):
        for a, c in zip(kept, pages):
            at = torch.arange(e, device="cuda")
            page = kv.block_table[b].long()[at // P]
            assert torch.equal(a[page, :, at % P], c[page, :, at % P])
    assert torch.equal(ends + T, replayed[2])


def test_two_streams_and_repeated_calls_agree():
    import torch
    tq = lib()
    jobs = []
    for lens, new in (([1900, 30, 777], [8, 8, 8]), ([600, 250], [60, 33])):
        s = Trees(tq, lens, new, 2, 32, 53)
        q = torch.randn((s.n_rows, 8, 128), device="cuda").bfloat16()
        first = torch.empty_like(q)
        tq.tq_paged_tree_attention(*s.ctx, s.kv, s.batch, s.d_parents, q, first, s.tree_workspace(8))
        jobs.append((s, q, first, s.tree_workspace(8)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in jobs]
    for _ in range(5):
        outs = [torch.zeros_like(j[2]) for j in jobs]
        torch.cuda.synchronize()
        for st, o, (s, q, first, ws) in zip(streams, outs, jobs):
            tq.tq_paged_tree_attention(*s.ctx, s.kv, s.batch, s.d_parents, q, o, ws, stream=st)
        torch.cuda.synchronize()
        for o, (s, q, first, ws) in zip(outs, jobs):
            assert torch.equal(o, first)


def test_lengths_written_just_before_each_call():
    """Calls back to back, the lengths changed by the kernel ahead of each."""
    import torch
    tq = lib()
    for lens, new in (([900, 300, 77, 1500], [8, 8, 8, 8]), ([700] * 40, [4] * 40)):
        s = Trees(tq, lens, new, 2, 32, 79)
        q = torch.randn((s.n_rows, 8, 128), device="cuda").bfloat16()
        ws, want = s.tree_workspace(8), []
        turns = [s.d_lens.clone(), s.d_lens - 37]
        for t in turns:
            s.d_lens.copy_(t)
            torch.cuda.synchronize()
            want.append(torch.empty_like(q))
            tq.tq_paged_tree_attention(*s.ctx, s.kv, s.batch, s.d_parents, q, want[-1], ws)
            torch.cuda.synchronize()
        assert not torch.equal(*want)
        outs = [torch.empty_like(q) for _ in range(100)]
        for i, o in enumerate(outs):
            s.d_lens.copy_(turns[i % 2])
            tq.tq_paged_tree_attention(*s.ctx, s.kv, s.batch, s.d_parents, q, o, ws)
        torch.cuda.synchronize()
        assert s.status() == 0 and all(torch.equal(o, want[i % 2]) for i, o in enumerate(outs))


def test_offsets_past_32_bits():
    """Pages of more than 2^32 bytes; the sequence's pages lie at the end."""
    import torch
    tq = lib()
    s = Trees(tq, [500, 300], [9, 40], 8, 64, 59)
    n_big = (1 << 32) // (8 * 64 * 68) + 40
    shift = n_big - s.n_pages
    big = []
    for p in s.pages:
        t = torch.empty((n_big, 8, 64, 68), dtype=torch.uint8, device="cuda")
        t[shift:] = p
        big.append(t)
    table = torch.from_numpy(np.where(s.table < 0, s.table, s.table + shift)).cuda()
    s.kv = tq.PagedKV(big[0], big[1], table, 64, 8)
    got, ref = run_tree(s, 16, "bf16", "bf16", 128)
    check_attention(got, ref, "bf16")
    paths = [[0, 3, 8], [1, 2, 30]]
    path = torch.full((2, 40), -1, dtype=torch.int32)
    for b, x in enumerate(paths):
        path[b, :3] = torch.tensor(x)
    lens = torch.zeros_like(s.d_lens)
    tq.tq_paged_tree_keep(*s.ctx, s.kv, s.batch, path.cuda(), torch.tensor([3, 3], dtype=torch.int32).cuda(), lens)
    assert s.status() == 0
    for p, h in zip(big, s.host):
        want, _ = tree.keep(h, s.table, s.lens, s.cu, paths)
        assert np.array_equal(p[shift:].cpu().numpy(), want)


def test_no_rows_is_a_no_op():
    import torch
    tq = lib()
    s = Trees(tq, [10], [1], 1, 16, 61)
    none = tq.PagedBatch(torch.zeros(0, dtype=torch.int32, device="cuda"))
    z = torch.zeros(0, dtype=torch.int32, device="cuda")
    q = torch.zeros((0, 2, 128), device="cuda")
    before = [p.clone() for p in s.pages]
    ws = tq.alloc_workspace(tq.tq_paged_tree_workspace_size(*s.ctx, s.kv, none, 2))
    tq.tq_paged_tree_append(*s.ctx, s.kv, none, z, q[:, :1], q[:, :1])
    tq.tq_paged_tree_attention(*s.ctx, s.kv, none, z, q, q.clone(), ws)
    tq.tq_paged_tree_keep(*s.ctx, s.kv, none, z.view(0, 1).expand(0, 1), z, z)
    cu = tq.PagedBatch(s.d_lens, torch.zeros(2, dtype=torch.int32, device="cuda"), 4, 5)  # rows, all of them padding
    out = torch.full((5, 2, 128), 7.0, device="cuda")
    p5 = torch.zeros(5, dtype=torch.int32, device="cuda")
    ws = tq.alloc_workspace(tq.tq_paged_tree_workspace_size(*s.ctx, s.kv, cu, 2))
    tq.tq_paged_tree_attention(*s.ctx, s.kv, cu, p5, torch.zeros_like(out), out, ws)
    tq.tq_paged_tree_append(*s.ctx, s.kv, cu, p5, out[:, :1], out[:, :1])
    lens = torch.zeros_like(s.d_lens)
    tq.tq_paged_tree_keep(*s.ctx, s.kv, cu, torch.zeros((1, 4), dtype=torch.int32, device="cuda"), p5[:1], lens)
    assert s.status() == 0 and lens.tolist() == [10]
    assert torch.all(out == 7.0) and all(torch.equal(a, b) for a, b in zip(before, s.pages))


# ------------------------------------------------------------------------------ refusals

def test_refusals():
    import torch
    tq = lib()
    L = tq.lib
    INV, UNS, ALI, WS = tq.TQ_ERR_INVALID_ARG, tq.TQ_ERR_UNSUPPORTED, tq.TQ_ERR_ALIGNMENT, tq.TQ_ERR_WORKSPACE
    s = Trees(tq, [40, 30], [3, 2], 2, 16, 67)
    H = [c.handle for c in s.ctx]
    q = torch.randn((5, 4, 128), device="cuda")
    out, ws = torch.full_like(q, 7.0), s.tree_workspace(4)
    n_ws = tq.tq_paged_tree_workspace_size(*s.ctx, s.kv, s.batch, 4)
    held = [p.clone() for p in s.pages]
    par = s.d_parents.data_ptr()

    def batch(**kw):
        c = type(s.batch.c).from_buffer_copy(s.batch.c)
        for name, val in kw.items():
            setattr(c, name, val)
        return ctypes.byref(c)

    def attend(b=None, parents=par, Hq=4, ws_n=n_ws, dtype=0, ctx=H):
        r = tq.tq_rows(q.data_ptr(), 0, 512, 128)
        return L.tq_paged_tree_attention(*ctx, s.kv.ref, b or batch(), parents, ctypes.byref(r), Hq, None, 0.0,
                                         out.data_ptr(), dtype, ws.data_ptr(), ws_n, None)

    assert attend() == tq.TQ_OK
    torch.cuda.synchronize()
    out.fill_(7.0)
    assert attend(batch(max_q=129)) == UNS and attend(parents=None) == INV and attend(parents=par + 2) == ALI
    assert attend(Hq=3) == INV and attend(Hq=2 * 66) == UNS and attend(ws_n=n_ws - 1) == WS and attend(dtype=4) == INV
    assert attend(batch(max_q=0)) == INV and attend(ctx=[None, H[1]]) == INV
    n = ctypes.c_size_t()
    assert L.tq_paged_tree_workspace_size(*H, s.kv.ref, batch(max_q=129), 4, ctypes.byref(n)) == UNS
    assert L.tq_paged_tree_workspace_size(*H, s.kv.ref, batch(), 4, None) == INV
    kr = tq.tq_rows(q.data_ptr(), 0, 512, 128)

    def append(b=None, parents=par, rows=kr):
        return L.tq_paged_tree_append(*H, s.kv.ref, b or batch(), parents, ctypes.byref(rows), ctypes.byref(kr), None, None)

    assert append(batch(max_q=129)) == UNS and append(parents=None) == INV and append(parents=par + 1) == ALI
    assert append(rows=tq.tq_rows(None, 0, 512, 128)) == INV
    path = torch.zeros((2, 3), dtype=torch.int32, device="cuda")
    cnt, new = torch.zeros(2, dtype=torch.int32, device="cuda"), torch.full((2,), 7, dtype=torch.int32, device="cuda")

    def keep(b=None, p=path.data_ptr(), stride=3, c=cnt.data_ptr(), o=new.data_ptr()):
        return L.tq_paged_tree_keep(*H, s.kv.ref, b or batch(), p, stride, c, o, None)

    assert keep(batch(max_q=129)) == UNS and keep(stride=0) == INV and keep(p=None) == INV and keep(c=None) == INV
    assert keep(o=None) == INV and keep(o=new.data_ptr() + 2) == ALI and keep(batch(n_tokens=0)) == INV
    rows = torch.rand((5, 11), device="cuda")
    tok, u = torch.zeros(5, dtype=torch.int32, device="cuda"), torch.zeros(5, device="cuda")

    def verify(b=None, t=(), d=None, parents=par, tokens=tok.data_ptr(), ua=u.data_ptr(), stride=3, nxt=new.data_ptr(), ctx=H[0]):
        tp = tq.tq_probs(rows.data_ptr(), 0, 11, 11)
        for name, val in t:
            setattr(tp, name, val)
        return L.tq_tree_verify(ctx, b or batch(), parents, tokens, ctypes.byref(tp), ctypes.byref(d) if d else None, ua,
                                u.data_ptr(), path.data_ptr(), stride, cnt.data_ptr(), nxt, None)

    assert verify(batch(max_q=129)) == UNS and verify(batch(max_q=0)) == INV and verify(batch(cu_q=None)) == INV
    assert verify(ctx=None) == INV and verify(parents=None) == INV and verify(tokens=None) == INV and verify(ua=None) == INV
    assert verify(stride=2) == INV and verify(nxt=None) == INV and verify(nxt=new.data_ptr() + 1) == ALI
    assert verify(t=[("data", None)]) == INV and verify(t=[("dtype", 3)]) == INV and verify(t=[("vocab", 0)]) == INV
    assert verify(t=[("row_stride", 10)]) == INV and verify(t=[("data", rows.data_ptr() + 2)]) == ALI
    assert verify(d=tq.tq_probs(rows.data_ptr(), 1, 11, 11)) == INV and verify(d=tq.tq_probs(rows.data_ptr(), 0, 10, 11)) == INV
    L.tq_test_ctx_set_device(H[0], 1)
    assert verify() == INV and keep() == INV and append() == INV and attend() == INV
    L.tq_test_ctx_set_device(H[0], 0)
    torch.cuda.synchronize()
    assert torch.all(out == 7.0) and torch.all(new == 7) and s.status() == 0
    assert all(torch.equal(a, b) for a, b in zip(held, s.pages))


def test_python_refusals():
    import torch
    tq = lib()
    s = Trees(tq, [40, 30], [3, 2], 2, 16, 71)
    q = torch.randn((5, 4, 128), device="cuda")
    kv = torch.randn((5, 2, 128), device="cuda")
    out, ws = torch.full_like(q, 7.0), s.tree_workspace(4)
    par = s.d_parents
    path, cnt = torch.zeros((2, 3), dtype=torch.int32, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda")
    rows, u = torch.rand((5, 11), device="cuda"), torch.zeros(5, device="cuda")

    def verify(parents=par, tokens=par, target=rows, ua=u, un=u, p=path, n=cnt, draft=None):
        tq.tq_tree_verify(s.ctx[0], s.batch, parents, tokens, target, ua, un, p, n, cnt, draft=draft)

    bad = [lambda: tq.tq_paged_tree_attention(*s.ctx, s.kv, s.batch, par[:4], q, out, ws),
           lambda: tq.tq_paged_tree_attention(*s.ctx, s.kv, s.batch, par.cpu(), q, out, ws),
           lambda: tq.tq_paged_tree_attention(*s.ctx, s.kv, s.batch, par.long(), q, out, ws),
           lambda: tq.tq_paged_tree_append(*s.ctx, s.kv, s.batch, par.repeat(2)[::2], kv, kv),
           lambda: tq.tq_paged_tree_append(*s.ctx, s.kv, s.batch, par, kv.cpu(), kv),
           lambda: tq.tq_paged_tree_keep(*s.ctx, s.kv, s.batch, path[:, :2], cnt, cnt),
           lambda: tq.tq_paged_tree_keep(*s.ctx, s.kv, s.batch, path, cnt[:1], cnt),
           lambda: tq.tq_paged_tree_keep(*s.ctx, s.kv, s.batch, path.long(), cnt, cnt),
           lambda: verify(target=rows[:4]), lambda: verify(target=rows.cpu()), lambda: verify(target=rows.t()),
           lambda: verify(draft=rows[0]), lambda: verify(ua=u.double()), lambda: verify(un=u[:1]),
           lambda: verify(tokens=par.long()), lambda: verify(p=path.t()), lambda: verify(n=cnt.cpu())]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    with pytest.raises(tq.TQError):
        verify(draft=rows.bfloat16())
    torch.cuda.synchronize()
    assert s.status() == 0 and torch.all(out == 7.0)
