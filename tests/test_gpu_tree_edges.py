"""Edges of the drafted trees' calls on the GPU: batches without rows, offsets past their bounds, steps of several
layers, vocabularies and batches at which the verification is laid out differently, norms of a wide range."""

import numpy as np
import pytest

from gpu_util import lib
from oracle import tree
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
