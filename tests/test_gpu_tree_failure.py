"""Failure detection of the trees' attention without a fault: a testing hook keeps the work back until the kernel's
bounded waits for it have run out (2 s) and hands it over then, so that warps that have given up meet warps that
have not.  The kernel records status 3 and returns, and the context keeps working."""

import ctypes

import pytest

from gpu_util import lib
from test_gpu_paged import check_attention
from test_gpu_tree import FullTrees, Trees, run_tree

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind, Hq, out_dtype", [(Trees, 4, "bf16"), (Trees, 4, "f32"), (FullTrees, 16, "bf16"),
                                                 (FullTrees, 16, "f16")], ids=["32-bf16", "32-f32", "64-bf16", "64-f16"])
def test_a_wait_that_runs_out_ends_the_kernel(kind, Hq, out_dtype):
    import torch
    tq = lib()
    s = kind(tq, [3000, 700, 90], [20, 9, 1], 2, 32, 83)
    got, ref = run_tree(s, Hq, "bf16", out_dtype)
    check_attention(got, ref, out_dtype)
    q = torch.from_numpy(s.q32).bfloat16().cuda()
    out, ws = torch.empty_like(got), s.tree_workspace(Hq)
    rows = tq.tq_rows(q.data_ptr(), 1, Hq * 128, 128)
    assert tq.lib.tq_test_tree_wait_timeout(*(c.handle for c in s.ctx), s.kv.ref, s.batch.ref, s.d_parents.data_ptr(),
                                            ctypes.byref(rows), Hq, out.data_ptr(), {"f32": 0, "bf16": 1, "f16": 2}[out_dtype],
                                            ws.data_ptr(), ws.numel(), None) == tq.TQ_OK
    assert s.status() == 3 and s.status() == 0
    out.fill_(7.0)
    s.tq.tq_paged_tree_attention(*s.ctx, s.kv, s.batch, s.d_parents, q, out, ws)
    assert s.status() == 0 and torch.equal(out[:s.n], got[:s.n])
