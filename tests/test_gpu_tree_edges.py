"""Edges of the drafted trees' calls on the GPU: batches without rows, offsets past their bounds, steps of several
layers, vocabularies and batches at which the verification is laid out differently, norms of a wide range."""

import numpy as np
import pytest

from gpu_util import lib

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
