"""Contexts: what making one costs, and that its tables are whole when it returns."""

import time

import numpy as np
import pytest

from gpu_util import BAND, band_ok, lib
from oracle.formats import Codec, unpack_turbo4

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rot,step,most_ms", [("wht", 1, 1.2), ("dense", 1, 3.0), ("dense", 0, 1.2)])
def test_a_context_is_made_in_about_a_millisecond(rot, step, most_ms):
    """The fastest of 20: 0.05 ms under the WHT and with the dense matrix of a seed that was used before, 0.9 with a
    new one's factorisation; several times that is a step of their construction that went back to single
    elements on the host (2.4 and 6.5 ms)."""
    tq = lib()
    best = 1e9
    for i in range(20):
        t = time.perf_counter()
        ctx = tq.Ctx("turbo4", rot, 100 + i * step)
        best = min(best, time.perf_counter() - t)
        del ctx
    assert best * 1e3 <= most_ms


@pytest.mark.parametrize("rot", ["wht", "dense"])
def test_a_new_context_serves_another_stream_at_once(rot):
    """Used on a stream of its own right after it was made: the tables written on the device are there."""
    import torch
    tq = lib()
    x = torch.randn((4096, 128), device="cuda").bfloat16()
    want = None
    for i in range(8):
        ctx, st = tq.Ctx("turbo4", rot, 5), torch.cuda.Stream()
        st.wait_stream(torch.cuda.current_stream())
        rec = torch.zeros((4096 * 68,), dtype=torch.uint8, device="cuda")
        out = torch.zeros((64, 64, 128), device="cuda")
        kv = tq.PagedKV(rec.view(64, 1, 64, 68), rec.view(64, 1, 64, 68),
                        torch.arange(64, dtype=torch.int32, device="cuda").view(1, 64), 64, 1)
        batch = tq.PagedBatch(torch.tensor([4096], dtype=torch.int32, device="cuda"),
                              torch.tensor([0, 4096], dtype=torch.int32, device="cuda"), 4096, 4096)
        torch.cuda.synchronize()
        tq.tq_quantize_set_rows(ctx, x, rec, stream=st)
        tq.tq_paged_gather(ctx, ctx, kv, batch, out.view(4096, 1, 128), None, stream=st)
        torch.cuda.synchronize()
        got = (rec.cpu().numpy(), out.cpu().numpy())
        want = want or got
        assert all(np.array_equal(a, b) for a, b in zip(got, want))
    codec, x32 = Codec("turbo4", rotation=rot, rot_seed=5), x.float().cpu().numpy()
    rows = want[0].reshape(-1, 68)
    rec, info = codec.encode(x32)
    (n1, idx1), (n0, idx0) = unpack_turbo4(rows), unpack_turbo4(rec)
    assert np.array_equal(n1, n0) and band_ok(idx1, idx0, info["y"], codec.b32, BAND if rot == "dense" else 0.0)[0]
    # a sum of 128 products of unit rows, in any order, with parts of operands: 260 * 2^-24 of the norm
    ref = codec.dequantize(rows)
    assert np.all(np.abs(want[1].reshape(-1, 128) - ref) <= 260 * 2.0 ** -24 * np.linalg.norm(ref, axis=1, keepdims=True))
