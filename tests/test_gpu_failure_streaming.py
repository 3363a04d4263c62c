"""Kernel waits that give up in the sinks and paged attention, on the GPU, without faulting or hanging it:
the failure-detection hooks make the softmax (elementwise) warps wait on a barrier that nothing signals, with a
short limit. The waits run out, device status 3 is recorded, every role winds down (copies and MMAs in flight
drained, tensor memory freed), no row is written, and the next call on the same workspace is right."""
import pytest
import torch

import test_gpu_paged as paged
import test_gpu_sinks as sinks

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def pha():
    from paired_heads_b200 import build

    build.build()
    from paired_heads_b200 import pha as mod

    return mod


SINKS = [
    # lens, H, Hkv, hd, window, sinks, paired
    ((1,), 2, 2, 64, 16, 2, False),                        # one tile; most CTAs have nothing
    ((300, 5, 190), 6, 6, 128, 128, 8, True),
    ((100,) * 90, 8, 2, 64, 64, 4, False),                 # many items of one key tile
    ((4100, 1500), 4, 1, 128, 60, 4, False),               # far pieces
    ((9000,), 8, 2, 64, 0, 0, False),                      # items cut between CTAs, full rings
]


@pytest.mark.parametrize("case", SINKS, ids=str)
def test_sinks_waits_that_run_out(pha, case):
    lens, H, Hkv, hd, window, n_sinks, pair = case
    c = sinks.Case(lens, H, Hkv, hd, BF16, window, n_sinks, pair, seed=2)
    o, lse = c.forward(pha)
    want = c.backward(pha, o, lse)
    for _ in range(2):
        nan, nan_lse = torch.full_like(o, float("nan")), torch.full_like(lse, float("nan"))
        pha.pha_test_attn_sinks_fwd_stalled(c.q, c.k, c.v, c.cu, c.max_len, nan, nan_lse, c.ws, 2000, **c.kw)
        assert pha.pha_attn_status(c.ws)[0] == 3
        assert torch.isnan(nan).all() and torch.isnan(nan_lse).all()
        got, got_lse = c.forward(pha, ws=c.ws)
        assert pha.pha_attn_status(c.ws)[0] == 0
        assert torch.equal(got, o) and torch.equal(got_lse, lse)

        grads = [torch.full_like(x, float("nan")) for x in want]
        args = (c.q, c.k, c.v, o, lse, c.dout, c.cu, c.max_len, *grads, c.ws_bwd)
        pha.pha_test_attn_sinks_bwd_stalled(*args, 2000, **c.kw)
        assert pha.pha_attn_status(c.ws_bwd)[0] == 3
        assert all(torch.isnan(g).all() for g in grads)
        pha.pha_attn_sinks_bwd(*args, **c.kw)
        assert pha.pha_attn_status(c.ws_bwd)[0] == 0
        assert all(torch.equal(a, b) for a, b in zip(grads, want))


@pytest.mark.parametrize("case", [
    ((40,), (333,), 4, 2, 64, 16, 0, 0, False),
    ((130, 1, 257), (300, 77, 257), 6, 6, 128, 16, 0, 0, True),
    ((100, 300, 1, 2), (1111, 300, 900, 5), 12, 12, 64, 32, 128, 16, False),
    ((500,), (4000,), 6, 2, 64, 4, 300, 40, False),        # gathered row by row
    ((1000,), (9000,), 8, 2, 128, 64, 0, 0, False),
], ids=str)
def test_paged_waits_that_run_out(pha, case):
    q, kv, H, Hkv, hd, page, window, n_sinks, pair = case
    c = paged.Case(q, kv, H, Hkv, hd, BF16, page, window, n_sinks, pair, seed=3)
    o, lse = c.run(pha)
    for _ in range(2):
        nan, nan_lse = torch.full_like(o, float("nan")), torch.full_like(lse, float("nan"))
        pha.pha_test_attn_paged_fwd_stalled(c.q, c.k, c.v, c.table, c.cu, c.lens, c.max_q, c.max_kv, nan, nan_lse,
                                            c.ws, 2000, status=c.status, **c.kw)
        assert c.status.item() == 3
        assert torch.isnan(nan).all() and torch.isnan(nan_lse).all()
        c.status.zero_()
        c.call(pha, nan, nan_lse, c.ws)
        assert c.status.item() == 0
        assert torch.equal(nan, o) and torch.equal(nan_lse, lse)
