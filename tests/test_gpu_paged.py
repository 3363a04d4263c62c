"""pha_attn_paged_fwd on the GPU against float64 (tests/streaming.py states the bounds): single tokens,
chunks and mixtures, pages of every size, windows, sinks, the paired view. Needs a B200."""
import numpy as np
import pytest
import torch

from streaming import Reference, f64

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def pha():
    from paired_heads_b200 import build

    build.build()
    from paired_heads_b200 import pha as mod

    return mod


class Case:
    """New tokens q_lens over caches of kv_lens tokens whose pages lie scattered in a pool. Every row
    of the pool that holds no token is NaN, every table entry without tokens is garbage."""

    def __init__(self, q_lens, kv_lens, H, Hkv, hd, dtype, page, window=0, sinks=0, paired=False, seed=0,
                 tail=0, spare_pages=3, max_q=None, max_kv=None, scale=0.0):
        rng = np.random.default_rng(seed)
        g = torch.Generator().manual_seed(seed)
        need = [-(-n // page) for n in kv_lens]
        self.n_pages = sum(need) + spare_pages
        order = rng.permutation(self.n_pages)
        self.max_pages = max(max(need), 1) + 2
        table = np.full((len(kv_lens), self.max_pages), -1, np.int32)
        table[:, -1] = 1 << 30
        pool = [torch.full((self.n_pages, page, Hkv, hd), float("nan")) for _ in range(2)]
        self.keys = []
        at = 0
        for b, n in enumerate(kv_lens):
            table[b, :need[b]] = order[at:at + need[b]]
            at += need[b]
            kv = [torch.randn(n, Hkv, hd, generator=g).to(dtype) for _ in range(2)]
            self.keys.append([f64(x) for x in kv])
            for p, x in zip(pool, kv):
                for e in range(need[b]):
                    rows = x[e * page:(e + 1) * page]
                    p[table[b, e], :len(rows)] = rows.float()
        self.k, self.v = (p.to(dtype).cuda() for p in pool)
        self.table = torch.from_numpy(table).cuda()
        total = sum(q_lens) + tail
        self.q = torch.randn(total, H, hd, generator=g).to(dtype).cuda()
        self.cu = torch.tensor(np.concatenate([[0], np.cumsum(q_lens)]), dtype=torch.int32).cuda()
        self.lens = torch.tensor(kv_lens, dtype=torch.int32).cuda()
        self.max_q = max(q_lens) if max_q is None else max_q
        self.max_kv = max(kv_lens) if max_kv is None else max_kv
        self.kw = dict(window=window, sinks=sinks, paired=paired)
        self.scale, self.dtype, self.H, self.Hkv, self.hd = scale, dtype, H, Hkv, hd
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def workspace(self, pha):
        ws = torch.empty(pha.pha_attn_paged_workspace_bytes(
            len(self.lens), self.max_q, self.max_kv, self.q.shape[0], self.H, self.Hkv, self.hd,
            self.dtype, **self.kw), dtype=torch.uint8, device="cuda")
        return ws.fill_(255)

    def call(self, pha, o, lse, ws, stream=None):
        pha.pha_attn_paged_fwd(self.q, self.k, self.v, self.table, self.cu, self.lens, self.max_q,
                               self.max_kv, o, lse, ws, scale=self.scale, status=self.status,
                               stream=stream, **self.kw)

    def run(self, pha):
        o = torch.full_like(self.q, float("nan"))
        lse = torch.full(self.q.shape[:2], float("nan"), device="cuda")
        self.ws = self.workspace(pha)
        self.call(pha, o, lse, self.ws)
        return o, lse

    def reference(self):
        return Reference(f64(self.q), self.cu.cpu().numpy(), lambda b: self.keys[b][0],
                         lambda b: self.keys[b][1], scale=self.scale, dtype=self.dtype, **self.kw)

    def drop_unseen_pages(self):
        """Table entries of pages that no query sees become -1, as pha_cache_trim leaves them."""
        mult = 2 if self.kw["paired"] else 1
        page = self.k.shape[1] * mult
        cu, t = self.cu.cpu().numpy(), self.table.cpu().numpy()
        for b, n in enumerate(self.lens.tolist()):
            first = (n - (cu[b + 1] - cu[b])) * mult
            for e in range(-(-n * mult // page)):
                if e * page >= self.kw["sinks"] and (e + 1) * page <= first - self.kw["window"] + 1:
                    t[b, e] = -1
        self.table.copy_(torch.from_numpy(t))


CASES = [
    # q_lens, kv_lens, H, Hkv, hd, dtype, page, window, sinks, paired
    ((1,), (1,), 2, 2, 64, BF16, 16, 0, 0, False),
    ((1,), (333,), 12, 12, 64, BF16, 16, 0, 0, False),
    ((1, 1, 1, 1), (1, 16, 17, 700), 32, 8, 128, BF16, 16, 0, 0, False),
    ((1,) * 9, (5, 2000, 64, 65, 127, 128, 129, 1, 900), 8, 2, 64, BF16, 64, 0, 0, False),
    ((1, 1, 1), (5000, 17, 3000), 6, 6, 128, BF16, 32, 200, 8, True),       # streams, paired
    ((1, 1), (4000, 90), 8, 8, 64, BF16, 128, 100, 3, False),
    ((1, 1), (900, 40), 4, 4, 64, BF16, 1, 64, 5, False),                   # pages of one token
    ((1, 1), (900, 40), 4, 4, 128, BF16, 1024, 0, 0, False),                # one page holds all
    ((1,), (9000,), 16, 1, 64, BF16, 64, 0, 0, False),                      # 16 heads on one
    ((1,), (3000,), 32, 1, 64, BF16, 64, 0, 0, False),                      # 32
    ((1, 1), (700, 10), 130, 1, 64, BF16, 64, 0, 0, False),                 # 130
    ((1, 1), (2500, 600), 258, 1, 64, BF16, 64, 77, 6, False),              # 258: more than a tile's rows
    ((4, 4, 3), (100, 1000, 3), 8, 2, 64, BF16, 16, 0, 0, False),           # a few tokens each
    ((4, 2), (600, 611), 4, 4, 128, BF16, 16, 33, 2, False),
    ((0, 1, 0, 5, 0), (7, 9, 0, 50, 3), 4, 2, 64, BF16, 8, 0, 0, False),    # nobody new in some
    ((200,), (200,), 4, 4, 64, BF16, 16, 0, 0, False),                      # a prompt from nothing
    ((333,), (1500,), 8, 2, 128, BF16, 64, 0, 0, False),
    ((130, 1, 257), (300, 77, 257), 6, 6, 128, BF16, 16, 0, 0, True),
    ((100, 300, 1, 2), (1111, 300, 900, 5), 12, 12, 64, BF16, 32, 128, 16, False),
    ((500,), (4000,), 6, 2, 64, BF16, 128, 300, 40, False),                 # groups of 3
    ((70, 20), (3000, 2000), 2, 1, 128, BF16, 256, 0, 0, False),            # few rows, long caches
    ((40,), (6000,), 2, 2, 64, BF16, 16, 1000, 1, True),
    ((300,), (900,), 4, 4, 64, BF16, 16, 50, 200, False),                   # more sinks than a tile
    ((64,), (2000,), 4, 4, 64, BF16, 32, 1, 0, False),                      # only itself
    ((1, 1), (100, 3000), 4, 2, 16, F32, 16, 0, 0, False),
    ((5, 40), (300, 41), 4, 4, 96, F32, 8, 17, 5, True),
    ((3,), (50,), 2, 1, 5, F32, 4, 0, 0, False),
    ((1,), (2500,), 4, 4, 128, F32, 64, 600, 100, False),
]


@pytest.mark.parametrize("case", CASES, ids=str)
def test_paged_attention(pha, case):
    c = Case(*case, seed=len(case[0]) + case[1][0])
    ref = c.reference()
    o, lse = c.run(pha)
    ref.check(o, lse)
    assert c.status.item() == 0
    if c.kw["window"]:
        c.drop_unseen_pages()          # pages nobody sees may be gone
        o2, lse2 = c.run(pha)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
        assert c.status.item() == 0
    # the same bits again, without the log-sum-exp
    o3 = torch.empty_like(o)
    c.call(pha, o3, None, c.ws)
    w = ref.written.reshape(o.shape[0], -1).any(1)
    assert torch.equal(o[torch.from_numpy(w)], o3[torch.from_numpy(w)])


@pytest.mark.parametrize("dtype,hd,q", [(BF16, 64, 1), (BF16, 128, 3), (BF16, 64, 40), (F32, 32, 2)])
def test_rows_behind_the_last_sequence(pha, dtype, hd, q):
    c = Case((q, q), (300, 200), 4, 2, hd, dtype, 16, tail=9, max_q=q + 30, max_kv=100000)
    c.q[-9:] = float("nan")
    o, lse = c.run(pha)
    c.reference().check(o, lse)


@pytest.mark.parametrize("q", [1, 100])
def test_bad_lengths_are_reported(pha, q):
    good = Case((q, q), (300, 200), 4, 2, 64, BF16, 16)
    for lens in ([q - 1, 200], [301, 200], [1 << 29, 200], [-5, 200]):
        c = Case((q, q), (300, 200), 4, 2, 64, BF16, 16)
        ref = c.reference()
        c.lens.copy_(torch.tensor(lens, dtype=torch.int32))
        o, lse = c.run(pha)
        assert c.status.item() == 1, lens
        assert torch.isnan(o[:q]).all() and torch.isnan(lse[:q]).all()
        if q == 1:
            assert not torch.isnan(o[q:]).any()
    assert good.status.item() == 0


@pytest.mark.parametrize("q", [1, 60])
@pytest.mark.parametrize("entry", [-1, 1 << 30])
def test_bad_pages_are_reported(pha, q, entry):
    c = Case((q, q), (300, 200), 4, 2, 64, BF16, 16)
    c.table[0, 3] = entry
    ref = c.reference()
    o, lse = c.run(pha)
    assert c.status.item() == 4
    # the other sequence is right
    a, z = c.cu[1].item(), c.cu[2].item()
    got, want = f64(o)[a:z], ref.o.reshape(o.shape)[a:z]
    assert (np.abs(got - want) <= ref.bo.reshape(o.shape)[a:z]).all()


@pytest.mark.parametrize("q,kv,heads,dtype", [
    ((1, 1), (300, 5000), (8, 2), BF16),     # decoding: one range, and several
    ((3, 1), (40, 2000), (4, 4), BF16),
    ((90, 40), (300, 9000), (8, 2), BF16),   # chunks, some of them cut between shares
    ((2, 3), (90, 3000), (4, 2), F32),
])
def test_a_nan_query_stays_in_its_row(pha, q, kv, heads, dtype):
    c = Case(q, kv, *heads, 64, dtype, 16)
    rows = [0, c.q.shape[0] - 1]
    c.q[rows[0], 1] = float("nan")
    c.q[rows[1], 2, 3] = float("nan")
    o, lse = c.run(pha)
    assert torch.isnan(o[rows[0], 1]).all() and torch.isnan(lse[rows[0], 1])
    assert torch.isnan(o[rows[1], 2]).all() and torch.isnan(lse[rows[1], 2])
    assert torch.isnan(o).sum().item() == 2 * 64 and torch.isnan(lse).sum().item() == 2
    for x, h in ((rows[0], 1), (rows[1], 2)):
        c.q[x, h] = 0
    ref = c.reference()
    good, good_lse = c.run(pha)
    ref.check(good, good_lse)
    for x, h in ((rows[0], 1), (rows[1], 2)):
        o[x, h], lse[x, h] = good[x, h], good_lse[x, h]
    ref.check(o, lse)


def test_one_workspace_for_every_kind_of_step(pha):
    """Decoding, chunks and their captured forms take turns on one workspace of the largest size."""
    cases = [Case((1,) * 5, (900, 20, 4000, 1, 77), 8, 2, 64, BF16, 16, seed=1),
             Case((90, 3, 200), (2000, 700, 200), 8, 2, 128, BF16, 32, seed=2),
             Case((2, 2), (3000, 100), 6, 6, 128, BF16, 16, window=100, sinks=4, paired=True, seed=3),
             Case((50, 1, 0, 64), (400, 900, 3, 64), 4, 4, 64, BF16, 64, window=64, sinks=9, seed=4),
             Case((5, 1), (900, 2500), 4, 2, 32, F32, 16, seed=5)]
    refs = [c.reference() for c in cases]
    ws = max((c.workspace(pha) for c in cases), key=lambda w: w.numel())
    outs = [(torch.empty_like(c.q), torch.empty(c.q.shape[:2], device="cuda")) for c in cases]
    graphs = []
    for c, (o, lse) in zip(cases, outs):
        c.call(pha, o, lse, ws)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.call(pha, o, lse, ws)
        graphs.append(g)
    for turn in range(3):
        for i in (0, 1, 2, 3, 4, 3, 1, 0, 4, 2):
            o, lse = outs[i]
            o.fill_(float("nan"))
            lse.fill_(float("nan"))
            if (turn + i) % 2:
                graphs[i].replay()
            else:
                cases[i].call(pha, o, lse, ws)
            refs[i].check(o, lse)
    assert all(c.status.item() == 0 for c in cases)


def test_a_long_float32_cache_with_many_ranges(pha):
    """Ranges of keys past 65,535 get longer instead of more."""
    n = 65535 * 1024 + 5000
    k = torch.zeros(n // 256 + 1, 256, 1, 1, device="cuda")
    v = torch.ones_like(k)
    table = torch.arange(k.shape[0], dtype=torch.int32, device="cuda")[None]
    q = torch.ones(1, 1, 1, device="cuda")
    k.view(-1)[n - 3] = 30.0                   # e^30 against n terms of e^0
    v.view(-1)[n - 3] = 3.0
    o, lse = torch.empty_like(q), torch.empty(1, 1, device="cuda")
    one = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
    ws = torch.empty(pha.pha_attn_paged_workspace_bytes(1, 1, n, 1, 1, 1, 1, F32), dtype=torch.uint8, device="cuda")
    pha.pha_attn_paged_fwd(q, k, v, table, one(0, 1), one(n), 1, n, o, lse, ws, scale=1.0)
    e = np.exp(30.0)
    assert abs(o.item() - (3 * e + n - 1) / (e + n - 1)) < 1e-5
    assert abs(lse.item() - np.log(e + n - 1)) < 1e-4


def test_decode_graph_follows_growing_lengths(pha):
    """One captured step serves lengths that grow on the device, up to max_kv."""
    c = Case((1, 1, 1), (400, 37, 260), 8, 2, 64, BF16, 16, max_kv=500)
    o = torch.full_like(c.q, float("nan"))
    lse = torch.full(c.q.shape[:2], float("nan"), device="cuda")
    ws = c.workspace(pha)
    c.call(pha, o, lse, ws)
    full = c.lens.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.call(pha, o, lse, ws)
    keys = c.keys
    for cut in (250, 36, 3, 0):
        lens = torch.clamp(full - cut, min=1)
        c.lens.copy_(lens)
        c.keys = [[x[:n] for x in kv] for kv, n in zip(keys, lens.tolist())]
        o.fill_(float("nan"))
        lse.fill_(float("nan"))
        g.replay()
        c.reference().check(o, lse)
    assert c.status.item() == 0


def test_two_streams_at_once(pha):
    """Calls on two streams with workspaces of their own."""
    cases = [Case((1,) * 8, (900,) * 8, 8, 2, 64, BF16, 16, seed=1), Case((90, 40), (2000, 700), 8, 2, 128, BF16, 32, seed=2)]
    refs = [c.reference() for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    outs = [(torch.full_like(c.q, float("nan")), torch.full(c.q.shape[:2], float("nan"), device="cuda"),
             c.workspace(pha)) for c in cases]
    torch.cuda.synchronize()
    for _ in range(5):
        for c, s, (o, lse, ws) in zip(cases, streams, outs):
            c.call(pha, o, lse, ws, stream=s)
    torch.cuda.synchronize()
    for ref, (o, lse, _) in zip(refs, outs):
        ref.check(o, lse)


def test_long_cache_offsets_pass_32_bits(pha):
    """A pool whose last bytes lie past 2^32: 1.1 million rows of 8 x 128 values (bf16, 2.2 GB each for
    K and V); the sequence's pages are the last ones."""
    hkv, hd, page = 8, 128, 256
    n_pages = (1 << 31) // (page * hkv * hd) + 40       # element offsets beyond 2^31, bytes beyond 2^32
    k = torch.zeros(n_pages, page, hkv, hd, dtype=BF16, device="cuda")
    v = torch.zeros_like(k)
    g = torch.Generator(device="cuda").manual_seed(0)
    k[-4:].normal_(generator=g)
    v[-4:].normal_(generator=g)
    c = Case((1, 30), (600, 700), hkv * 4, hkv, hd, BF16, page)
    table = np.array([[n_pages - 1, n_pages - 3, n_pages - 2], [n_pages - 2, n_pages - 4, n_pages - 1]])
    c.k, c.v, c.table = k, v, torch.tensor(table, dtype=torch.int32).cuda()
    c.keys = [[f64(x[t.tolist()].reshape(-1, hkv, hd)[:n]) for x in (k, v)] for t, n in
              zip(torch.tensor(table), (600, 700))]
    ref = c.reference()
    o, lse = c.run(pha)
    ref.check(o, lse)
    # and the single token alone (the decoding path)
    c.q, c.cu, c.lens = c.q[:1].contiguous(), c.cu[:2].contiguous(), c.lens[:1].contiguous()
    c.table, c.max_q, c.max_kv = c.table[:1].contiguous(), 1, 600
    ref = c.reference()
    o, lse = c.run(pha)
    ref.check(o, lse)


WINDOWED = [c for c in CASES if c[7] and c[5] is BF16] + [
    # chunks whose first column lies inside a box or a page, sinks below it and across it
    ((300, 33), (1000, 815), 4, 2, 128, BF16, 64, 77, 0, False),
    ((150,), (700,), 2, 2, 64, BF16, 32, 400, 148, False),                  # the sinks end in that box
    ((150,), (700,), 2, 2, 64, BF16, 8, 531, 30, False),                    # the box begins with sinks
    ((90, 90, 90, 90), (500, 501, 515, 531), 12, 4, 64, BF16, 16, 200, 3, False),
    ((200,), (600,), 4, 4, 128, BF16, 256, 250, 5, True),
]


@pytest.mark.parametrize("case", WINDOWED, ids=str)
def test_keys_that_no_query_sees_may_hold_anything(pha, case):
    """NaN and infinities in keys and values between the sinks and the first query's window: they lie in
    the boxes, pages and tiles of visible ones, and change no bit."""
    c = Case(*case, seed=len(case[0]) + case[1][0])
    ref = c.reference()
    clean = c.run(pha)
    mult, hkv = (2, c.Hkv // 2) if c.kw["paired"] else (1, c.Hkv)
    page = c.k.shape[1] * mult
    cu, table = c.cu.cpu().numpy(), c.table.cpu().numpy()
    n = 0
    for pool, bad in ((c.k, float("nan")), (c.v, float("inf"))):
        rows = pool.view(-1, hkv, c.hd)
        for b, kv in enumerate(c.lens.tolist()):
            first = (kv - (cu[b + 1] - cu[b])) * mult
            for j in range(c.kw["sinks"], max(first - c.kw["window"] + 1, 0)):
                rows[table[b, j // page] * page + j % page] = bad if j % 3 else -bad
                n += 1
    assert n or max(case[1]) * mult <= c.kw["window"] + max(case[0]) * mult + c.kw["sinks"]
    o, lse = c.run(pha)
    ref.check(o, lse)
    w = torch.from_numpy(ref.written.reshape(o.shape[0], -1).any(1))
    assert torch.equal(o[w], clean[0][w]) and torch.equal(lse[w], clean[1][w])
    assert c.status.item() == 0


BAD_LENGTHS = [
    # what is wrong with the first of three sequences of q new tokens over (300, 200, 64)
    ("kv_lens", lambda c, q: c.lens.__setitem__(0, q - 1)),           # fewer than the new tokens
    ("kv_lens", lambda c, q: c.lens.__setitem__(0, -5)),
    ("kv_lens", lambda c, q: c.lens.__setitem__(0, 301)),             # beyond max_kv
    ("kv_lens", lambda c, q: c.lens.__setitem__(0, 1 << 29)),
    ("cu_seqlens", lambda c, q: c.cu.__setitem__(0, -1)),             # a row before q
    ("max_q", lambda c, q: c.cu.copy_(torch.tensor([0, q + 1, 2 * q + 1, 3 * q + 1]))),
]


@pytest.mark.parametrize("q", [1, 3, 60])
@pytest.mark.parametrize("dtype,hd", [(BF16, 64), (F32, 16)])
@pytest.mark.parametrize("bad", range(len(BAD_LENGTHS)))
def test_a_bad_sequence_leaves_the_others_right(pha, dtype, hd, q, bad):
    c = Case((q, q, q), (300, 200, 64), 4, 2, hd, dtype, 16, tail=1)
    BAD_LENGTHS[bad][1](c, q)
    lens = c.lens.clone()
    c.lens.copy_(torch.tensor([300, 200, 64], dtype=torch.int32))
    cu = c.cu.clone()
    c.cu.clamp_(min=0)
    ref = c.reference()                        # (of the others: the first one's rows are not looked at)
    c.lens.copy_(lens)
    c.cu.copy_(cu)
    o, lse = c.run(pha)
    assert c.status.item() == 1
    cu = c.cu.tolist()
    assert torch.isnan(o[:cu[1]]).all() and torch.isnan(lse[:cu[1]]).all()
    ref.written[:cu[1]] = False
    ref.check(o, lse)


@pytest.mark.parametrize("q", [1, 2, 60])
@pytest.mark.parametrize("dtype,hd", [(BF16, 64), (F32, 16)])
def test_sequences_wholly_outside_q_are_reported(pha, dtype, hd, q):
    """Rows behind q and before it: status 1 whoever else is fine."""
    for cu in ([0, q, 2 * q, 3 * q + 1], [0, q, 2 * q, 2 * q + 1], [-q, 0, q, 2 * q]):
        c = Case((q, q, q), (300, 200, 64), 4, 2, hd, dtype, 16, max_q=q + 1)
        c.q = c.q[:2 * q].contiguous()
        good = [b for b in range(3) if cu[b] >= 0 and cu[b + 1] <= 2 * q]
        c.cu.copy_(torch.tensor(cu))
        o, lse = c.run(pha)
        assert c.status.item() == 1, cu
        whole = Case((q, q, q), (300, 200, 64), 4, 2, hd, dtype, 16, max_q=q + 1)
        ref = Reference(f64(c.q), [cu[b] for b in good] + [cu[good[-1] + 1]], lambda i: whole.keys[good[i]][0],
                        lambda i: whole.keys[good[i]][1], scale=c.scale, dtype=dtype, **c.kw)
        ref.check(o, lse, cu)


@pytest.mark.parametrize("dtype,hd,q", [(BF16, 64, 1), (F32, 8, 1)])
def test_more_sequences_than_a_grid_has_columns(pha, dtype, hd, q):
    """70,000 sequences; then a call that allows no new tokens where a sequence has some."""
    n = 70000
    c = Case((q,) * 3 + (0,) * (n - 6) + (q,) * 3, (40, 3, 17) + (0,) * (n - 6) + (1, 9, 33), 2, 1, hd, dtype, 16)
    ref = c.reference()
    o, lse = c.run(pha)
    ref.check(o, lse)
    assert c.status.item() == 0
    c.max_q = 0
    o, lse = c.run(pha)
    assert c.status.item() == 1
    assert torch.isnan(o).all() and torch.isnan(lse).all()


@pytest.mark.parametrize("dtype,hd,q", [(BF16, 64, 1000), (BF16, 64, 4), (F32, 8, 40)])
def test_sequences_that_overlap_are_reported(pha, dtype, hd, q):
    """cu_seqlens that goes back and forth: more rows than q has, however they are counted. Status 1, and
    nothing outside q's rows is written."""
    c = Case((q,) + (0,) * 9, (q + 5,) * 10, 2, 1, hd, dtype, 16, max_q=q)
    c.cu.copy_(torch.tensor([0, q] * 5 + [0]))
    o = torch.full((q + 8, 2, hd), float("nan"), device="cuda").to(dtype)
    lse = torch.full((q + 8, 2), float("nan"), device="cuda")
    c.call(pha, o[4:-4], lse[4:-4], c.workspace(pha))
    assert c.status.item() == 1
    assert torch.isnan(o[:4]).all() and torch.isnan(o[-4:]).all()
    assert torch.isnan(lse[:4]).all() and torch.isnan(lse[-4:]).all()
