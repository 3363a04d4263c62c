"""Argument checks of the sinks and paged-cache entry points: refused on the host, before any CUDA
call (so they run on CPU), and the binding's checks of types, shapes and layouts."""
import ctypes

import pytest

from paired_heads_b200 import build as pha_build

A, MIS = 0x10000, 0x10004


@pytest.fixture(scope="module")
def pha():
    pha_build.build()
    from paired_heads_b200 import pha as mod

    return mod


def test_new_entry_points_are_exported(pha):
    names = pha.exported_symbols()
    for n in ("pha_attn_sinks_fwd", "pha_attn_sinks_bwd", "pha_attn_paged_fwd", "pha_cache_append",
              "pha_cache_fork", "pha_cache_reserve", "pha_cache_free", "pha_cache_trim",
              "pha_cache_compact", "pha_attn_fwd"):
        assert n in names
        assert hasattr(pha.library(), n)


def _sinks(pha, bwd=False, **kw):
    a = dict(q=A, k=A, v=A, cu=A, batch=1, max_len=128, total=128, H=4, Hkv=4, hd=64, dtype=0,
             window=64, sinks=4, paired=0, scale=0.0, o=A, lse=A, dout=A, dq=A, dk=A, dv=A, ws=A,
             bytes=10)
    a.update(kw)
    f = ctypes.c_float(a["scale"])
    shape = (a["cu"], a["batch"], a["max_len"], a["total"], a["H"], a["Hkv"], a["hd"], a["dtype"],
             a["window"], a["sinks"], a["paired"], f)
    if bwd:
        return pha.library().pha_attn_sinks_bwd(a["q"], a["k"], a["v"], a["o"], a["lse"], a["dout"],
                                                *shape, a["dq"], a["dk"], a["dv"], a["ws"],
                                                a["bytes"], None)
    return pha.library().pha_attn_sinks_fwd(a["q"], a["k"], a["v"], *shape, a["o"], a["lse"],
                                            a["ws"], a["bytes"], None)


@pytest.mark.parametrize("bwd", [False, True])
@pytest.mark.parametrize("kw,code", [
    ({}, -3),                                  # a valid problem: only the workspace is too small
    (dict(sinks=128), -3),
    (dict(window=0), -3),                      # no window: the sinks change nothing
    (dict(ws=None, bytes=1 << 30), -3),
    (dict(ws=MIS, bytes=1 << 30), -3),
    (dict(sinks=-1), -1),
    (dict(sinks=129), -2),
    (dict(H=6, Hkv=4), -1),
    (dict(H=5, Hkv=5, paired=1), -1),
    (dict(H=6, Hkv=3, paired=1), -1),
    (dict(hd=96), -2),
    (dict(dtype=1, hd=160), -2),
    (dict(dtype=1, hd=96), -3),
    (dict(dtype=7), -1),
    (dict(batch=0), -1),
    (dict(total=-1), -1),
    (dict(paired=2), -1),
    (dict(scale=float("nan")), -1),
    (dict(q=MIS), -1),
    (dict(v=None), -1),
    (dict(lse=A + 2), -1),
    (dict(cu=None), -1),
    (dict(total=1 << 24, H=128, Hkv=128), -1),  # more rows than 31 bits count
    (dict(total=(1 << 24) - 1, H=128, Hkv=128), -3),
])
def test_sinks_argument_errors(pha, bwd, kw, code):
    assert _sinks(pha, bwd, **kw) == code


def test_sinks_backward_needs_the_forwards_outputs(pha):
    for kw in (dict(lse=None), dict(o=None), dict(dout=None), dict(dq=None), dict(dk=MIS)):
        assert _sinks(pha, True, **kw) == -1
    assert _sinks(pha, True, total=0, q=None, k=None, v=None, o=None, lse=None, dout=None, dq=None,
                  dk=None, dv=None, ws=None) == 0      # nothing to do


def _paged(pha, **kw):
    a = dict(q=A, k=A, v=A, table=A, max_pages=8, n_pages=64, page=16, cu=A, lens=A, batch=2, max_q=4,
             max_kv=100, total=8, H=4, Hkv=4, hd=64, dtype=0, window=0, sinks=0, paired=0, scale=0.0,
             o=A, lse=A, ws=A, bytes=10, status=A)
    a.update(kw)
    return pha.library().pha_attn_paged_fwd(
        a["q"], a["k"], a["v"], a["table"], a["max_pages"], a["n_pages"], a["page"], a["cu"],
        a["lens"], a["batch"], a["max_q"], a["max_kv"], a["total"], a["H"], a["Hkv"], a["hd"],
        a["dtype"], a["window"], a["sinks"], a["paired"], ctypes.c_float(a["scale"]), a["o"],
        a["lse"], a["ws"], a["bytes"], a["status"], None)


@pytest.mark.parametrize("kw,code", [
    ({}, -3),
    (dict(page=1), -3),
    (dict(page=24), -1),                       # no power of two
    (dict(page=0), -1),
    (dict(n_pages=0), -1),
    (dict(max_pages=0), -1),
    (dict(n_pages=1 << 27, page=16), -1),      # more rows than 31 bits count
    (dict(total=1 << 24, H=128, Hkv=4), -1),
    (dict(total=(1 << 24) - 1, H=128, Hkv=4), -3),
    (dict(sinks=-1), -1),
    (dict(sinks=1000, window=5), -3),
    (dict(hd=96), -2),
    (dict(dtype=1, hd=129), -2),
    (dict(dtype=3), -1),
    (dict(H=6, Hkv=4), -1),
    (dict(H=3, Hkv=3, paired=1), -1),
    (dict(max_q=-1), -1),
    (dict(batch=0), -1),
    (dict(scale=float("nan")), -1),
    (dict(q=None), -1),
    (dict(k=MIS), -1),
    (dict(table=None), -1),
    (dict(table=A + 2), -1),
    (dict(cu=None), -1),
    (dict(lens=None), -1),
    (dict(status=A + 1), -1),
    (dict(ws=None, bytes=1 << 30), -3),
    (dict(total=0, q=None, o=None, lse=None, ws=None), 0),
])
def test_paged_argument_errors(pha, kw, code):
    assert _paged(pha, **kw) == code


def test_paged_workspace_bytes(pha):
    import torch

    size = lambda **kw: pha.pha_attn_paged_workspace_bytes(**{**dict(
        batch=4, max_q=1, max_kv=500, total_q=4, n_heads=8, n_kv_heads=2, head_dim=64,
        dtype=torch.bfloat16), **kw})
    assert size() >= 256
    assert size(batch=0) == 0 and size(n_heads=7) == 0 and size(max_kv=-1) == 0
    assert size(max_kv=1 << 20) >= size()
    # a window bounds what splits can be worth
    assert size(max_kv=1 << 20, window=64) <= size(max_kv=1 << 20)


def _append(pha, **kw):
    a = dict(k=A, v=A, kp=A, vp=A, table=A, max_pages=8, n_pages=64, page=16, cu=A, lens=A, batch=2,
             total=8, Hkv=4, hd=64, esize=2, status=A)
    a.update(kw)
    return pha.library().pha_cache_append(
        a["k"], a["v"], a["kp"], a["vp"], a["table"], a["max_pages"], a["n_pages"], a["page"],
        a["cu"], a["lens"], a["batch"], a["total"], a["Hkv"], a["hd"], a["esize"], a["status"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(total=0), 0),
    (dict(total=-1), -1),
    (dict(page=12), -1),
    (dict(esize=8), -1),
    (dict(Hkv=1, hd=4), -1),                   # rows of 8 bytes
    (dict(k=MIS), -1),
    (dict(vp=None), -1),
    (dict(table=None), -1),
    (dict(lens=A + 2), -1),
    (dict(status=A + 2), -1),
])
def test_append_argument_errors(pha, kw, code):
    assert _append(pha, **kw) == code


def test_cache_call_argument_errors(pha):
    lib = pha.library()
    big = pha.pha_cache_workspace_bytes(64, 4)
    assert pha.pha_cache_workspace_bytes(0, 4) == 0 and pha.pha_cache_workspace_bytes(4, 0) == 0

    def fork(table=A, lens=A, refs=A, src=A, dst=A, n=2, ws=A, size=big, pages=64, status=None):
        return lib.pha_cache_fork(table, 8, lens, 4, refs, pages, src, dst, n, ws, size, status, None)

    assert fork(size=big - 1) == -3 and fork(ws=None) == -3 and fork(ws=MIS) == -3
    for kw in (dict(table=None), dict(lens=None), dict(refs=A + 1), dict(src=None), dict(dst=A + 2),
               dict(n=-1), dict(n=5), dict(pages=0), dict(status=A + 3)):
        assert fork(**kw) == -1, kw

    def reserve(page=16, seqs=A, new=A, k=A, v=A, layers=1, nbytes=4096, ws=None):
        return lib.pha_cache_reserve(A, 8, A, 4, A, 64, page, seqs, new, 2, k, v, layers, nbytes, ws,
                                     big, None, None)

    assert reserve() == -3
    for kw in (dict(page=10), dict(seqs=None), dict(new=A + 2), dict(k=None), dict(v=MIS),
               dict(layers=0), dict(nbytes=24), dict(nbytes=0)):
        assert reserve(**kw) == -1, kw

    def free(seqs=A, ws=None):
        return lib.pha_cache_free(A, 8, A, 4, A, 64, seqs, 2, ws, big, None, None)

    assert free() == -3 and free(seqs=None) == -1

    def trim(window=5, sinks=0, page=16, paired=0):
        return lib.pha_cache_trim(A, 8, None, 4, A, 64, page, window, sinks, paired, None, None)

    assert trim() == -1                        # lengths are needed
    for kw in (dict(window=0), dict(sinks=-1), dict(page=3), dict(paired=2)):
        assert trim(**kw) == -1

    def compact(k=A, layers=1, nbytes=4096, ws=None):
        return lib.pha_cache_compact(A, 8, 4, A, 64, k, A, layers, nbytes, ws, big, None, None)

    assert compact() == -3
    assert compact(k=None) == -1 and compact(layers=0) == -1 and compact(nbytes=8) == -1


def test_binding_checks_tensors(pha):
    """The binding refuses what the library cannot see, before the library is called."""
    import torch

    q = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    ws = torch.zeros(1 << 12, dtype=torch.uint8)
    cu = torch.tensor([0, 4], dtype=torch.int32)
    kw = dict(window=2, sinks=1)
    with pytest.raises(ValueError, match="CUDA"):
        pha.pha_attn_sinks_fwd(q, q, q, cu, 4, q, None, ws, **kw)
    with pytest.raises(ValueError, match="contiguous"):
        pha.pha_attn_sinks_fwd(torch.zeros(2, 4, 64, dtype=torch.bfloat16).transpose(0, 1), q, q, cu, 4,
                               q, None, ws, **kw)
    with pytest.raises(TypeError):
        pha.pha_attn_sinks_fwd(q.to(torch.float16), q, q, cu, 4, q, None, ws, **kw)
    with pytest.raises(TypeError, match="o:"):
        pha.pha_attn_sinks_fwd(q, q, q, cu, 4, q.float(), None, ws, **kw)
    i32 = dict(dtype=torch.int32)
    with pytest.raises(TypeError, match="page_table"):
        pha.pha_cache_trim(torch.zeros(2, 3, dtype=torch.int64), torch.zeros(2, **i32),
                           torch.zeros(9, **i32), 16, window=4)


def test_sinks_backward_workspace_follows_the_tokens(pha):
    """A loose max_len costs nothing: no document is longer than all tokens."""
    def size(batch, max_len, total, window=300, sinks=4, paired=False, H=8, Hkv=2, hd=128):
        return pha.pha_attn_sinks_bwd_workspace_bytes(batch, max_len, total, H, Hkv, hd, window=window,
                                                      sinks=sinks, paired=paired)

    for paired in (False, True):
        for total in (1, 127, 4096, 70000):
            for batch in (1, 3, 200):
                for window in (0, 1, 300, total, 2 ** 31 - 1):
                    kw = dict(batch=batch, total=total, window=window, paired=paired)
                    assert 0 < size(max_len=2 ** 31 - 1, **kw) == size(max_len=total, **kw) >= size(max_len=1, **kw)
    # rows of total tokens and one ragged tile (and piece) a document, however many documents there are
    per_item = 16 * 8
    assert size(5000, 4096, 4096) <= size(1, 4096, 4096) + 5000 * (2 * per_item + per_item + 16 + 2 * 2 * 4 * 2 * 128 * 4) + 8192


def test_sinks_workspace_bytes_never_wrap(pha):
    """Bounds of batch and max_len whose workspace would not fit 64 bits are invalid arguments; below, the size
    covers 24 bytes for each row tile that a batch of longest documents has."""
    for H, Hkv, paired in ((256, 2, True), (2, 2, False), (34, 2, False)):
        pack = H // Hkv
        for batch in (1, 1000, 1 << 19, 1 << 20, 1 << 29, 2 ** 31 - 1):
            for max_len in (1, 5000, 1 << 28, 1 << 29, 2 ** 31 - 1):
                size = pha.pha_attn_sinks_workspace_bytes(batch, max_len, H, Hkv, 64, window=0, sinks=4,
                                                          paired=paired)
                length = min(max_len, 1 << 29)         # total_tokens is at most that
                if batch * length > 1 << 48:
                    assert size == 0, (batch, max_len)
                    assert _sinks(pha, batch=batch, max_len=max_len, H=H, Hkv=Hkv, paired=int(paired), bytes=2 ** 63) == -1
                else:
                    tiles = batch * -(-length * (2 if paired else 1) // (256 // pack))
                    assert size >= 24 * tiles, (batch, max_len)


def test_windows_past_32_bits_do_not_wrap(pha, monkeypatch):
    """The library is called with the nearest count that fits: a window of 2^32 + 5 hides nothing (no more than
    one of 2^31 - 1) and is not one of 5, and sinks of 2^32 + 4 are not 4."""
    import torch

    seen = []
    q = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    ws = torch.zeros(1 << 12, dtype=torch.uint8)
    i32 = lambda *shape: torch.zeros(*shape, dtype=torch.int32)
    pool = torch.zeros(3, 4, 2, 64, dtype=torch.bfloat16)
    lse = torch.zeros(4, 2)
    calls = {
        "pha_attn_sinks_fwd": (11, lambda **kw: pha.pha_attn_sinks_fwd(q, q, q, i32(2), 4, q, None, ws, **kw)),
        "pha_attn_sinks_bwd": (14, lambda **kw: pha.pha_attn_sinks_bwd(q, q, q, q, lse, q, i32(2), 4, q, q, q, ws, **kw)),
        "pha_attn_paged_fwd": (17, lambda **kw: pha.pha_attn_paged_fwd(
            q, pool, pool, i32(1, 3), i32(2), i32(1), 4, 9, q, None, ws, **kw)),
        "pha_cache_trim": (7, lambda **kw: pha.pha_cache_trim(i32(2, 3), i32(2), i32(9), 16, **kw)),
    }
    monkeypatch.setattr(pha, "_run", lambda fn, wanted, args, stream: seen.append((fn, args)))
    top, low = 2 ** 31 - 1, -2 ** 31
    for given, wanted in ((2 ** 31, top), (2 ** 32 + 5, top), (2 ** 63, top), (low - 1, low), (-2 ** 40, low),
                          (top, top), (77, 77), (-1, -1)):
        for fn, (at, call) in calls.items():
            call(window=given, sinks=3)
            call(window=9, sinks=given)
            (name, a), (_, b) = seen[-2:]
            assert name == fn and a[at:at + 2] == (wanted, 3) and b[at:at + 2] == (9, wanted), (fn, given)
    pha.pha_cache_trim(i32(2, 3), i32(2), i32(9), 2 ** 32 + 16, window=5)
    assert seen[-1][1][6] == top                       # (no power of two: refused)
    size = lambda w, s: (pha.pha_attn_sinks_workspace_bytes(1, 900, 2, 2, 64, window=w, sinks=s),
                         pha.pha_attn_sinks_bwd_workspace_bytes(1, 900, 900, 2, 2, 64, window=w, sinks=s),
                         pha.pha_attn_paged_workspace_bytes(1, 1, 90000, 1, 2, 2, 64, torch.bfloat16, window=w, sinks=s))
    assert size(2 ** 32 + 5, 1) == size(0, 1) != size(5, 1)
    assert size(5, 2 ** 32 + 4)[:2] == (0, 0) and size(5, 2 ** 32 + 4)[2] == size(0, 0)[2]


def test_stall_hooks_argument_errors(pha):
    """Failure-detection hooks: the limits of the stall, then the checks of the call itself."""
    lib, f = pha.library(), ctypes.c_float(0.0)
    for n in ("pha_test_attn_sinks_fwd_stalled", "pha_test_attn_sinks_bwd_stalled", "pha_test_attn_paged_fwd_stalled"):
        assert n in pha.exported_symbols()

    def fwd(us, dtype=0, sinks=4, ws=A):
        return lib.pha_test_attn_sinks_fwd_stalled(A, A, A, A, 1, 128, 128, 4, 4, 64, dtype, 64, sinks, 0, f, A, A, ws,
                                                   10, us, None)

    def bwd(us, dtype=0, sinks=4, ws=A):
        return lib.pha_test_attn_sinks_bwd_stalled(A, A, A, A, A, A, A, 1, 128, 128, 4, 4, 64, dtype, 64, sinks, 0, f,
                                                   A, A, A, ws, 10, us, None)

    def paged(us, dtype=0, max_q=100, sinks=4, ws=A, size=10):
        return lib.pha_test_attn_paged_fwd_stalled(A, A, A, A, 8, 64, 16, A, A, 2, max_q, 128, 128, 4, 4, 64, dtype, 64,
                                                   sinks, 0, f, A, A, ws, size, None, us, None)

    for call in (fwd, bwd, paged):
        assert call(0) == call(-1) == call(100001) == -1
        assert call(1) == call(100000) == -3               # everything fits but the workspace
        assert call(5, sinks=-1) == -1 and call(5, ws=None) == -3
    assert fwd(5, dtype=1) == bwd(5, dtype=1) == -2        # float32 has no waits
    assert paged(5, dtype=1, size=1 << 40) == -2 and paged(5, max_q=4, size=1 << 40) == -2
