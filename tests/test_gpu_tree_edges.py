"""Edges of the drafted trees' calls on the GPU: batches without rows, offsets past their bounds, steps of several
layers, vocabularies and batches at which the verification is laid out differently, norms of a wide range."""

import numpy as np
import pytest

from gpu_util import lib
from oracle import tree
from test_gpu_paged import check_attention
from test_gpu_tree import Trees

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
