"""The cache's pages on the GPU: append, fork, reserve, free, trim, compact against a plain
implementation (tests/streaming.py), everything bit for bit, and a run of them together with the
attention over the pages. Needs a B200."""
import numpy as np
import pytest
import torch

from streaming import Pages, Reference, f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def pha():
    from paired_heads_b200 import build

    build.build()
    from paired_heads_b200 import pha as mod

    return mod


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32).cuda()


class Cache:
    """A cache on the GPU and its plain twin."""

    def __init__(self, pha, n_pages, page, n_seqs, max_pages, layers=2, hkv=2, hd=64, dtype=torch.bfloat16):
        g = torch.Generator().manual_seed(n_pages)
        self.pha = pha
        self.table = torch.full((n_seqs, max_pages), -1, dtype=torch.int32).cuda()
        self.lens = torch.zeros(n_seqs, dtype=torch.int32).cuda()
        self.refs = torch.zeros(n_pages, dtype=torch.int32).cuda()
        # any bits will do: the pools are compared as integers
        self.k, self.v = (torch.randn(layers, n_pages, page, hkv, hd, generator=g).to(dtype).cuda() for _ in range(2))
        self.ws = torch.full((pha.pha_cache_workspace_bytes(n_pages, n_seqs),), 255, dtype=torch.uint8).cuda()
        self.status = torch.zeros(1, dtype=torch.int32).cuda()
        self.plain = Pages(*(x.cpu().numpy().copy() for x in (self.table, self.lens, self.refs)),
                           *(f64(x) for x in (self.k, self.v)))

    def fork(self, src, dst):
        self.pha.pha_cache_fork(self.table, self.lens, self.refs, i32(src), i32(dst), self.ws, status=self.status)

    def reserve(self, seqs, new):
        self.pha.pha_cache_reserve(self.table, self.lens, self.refs, i32(seqs), i32(new), self.k, self.v, self.ws,
                                   status=self.status)

    def free(self, seqs):
        self.pha.pha_cache_free(self.table, self.lens, self.refs, i32(seqs), self.ws, status=self.status)

    def trim(self, page, window, sinks, paired=False):
        self.pha.pha_cache_trim(self.table, self.lens, self.refs, page, window=window, sinks=sinks,
                                paired=paired, status=self.status)

    def compact(self):
        self.pha.pha_cache_compact(self.table, self.refs, self.k, self.v, self.ws, status=self.status)

    def same(self, status=0):
        p = self.plain
        assert np.array_equal(self.table.cpu().numpy(), p.table)
        assert np.array_equal(self.lens.cpu().numpy(), p.lens)
        assert np.array_equal(self.refs.cpu().numpy(), p.refs)
        assert np.array_equal(f64(self.k), p.k) and np.array_equal(f64(self.v), p.v)
        assert self.status.item() == status

    def count(self):
        return self.pha.pha_attn_status(self.ws)


@pytest.mark.parametrize("page,hkv,hd,dtype", [(16, 2, 64, torch.bfloat16), (1, 1, 8, torch.bfloat16),
                                               (64, 8, 128, torch.bfloat16), (8, 3, 20, torch.float32),
                                               (32, 2, 128, torch.uint8)])
def test_append(pha, page, hkv, hd, dtype):
    rng = np.random.default_rng(page)
    q = np.array([1, 0, 37, 200, 1, 5])
    kv = q + np.array([0, 4, 100, 13, 31, 0])
    need = -(-kv // page)
    n_pages = int(need.sum()) + 2
    table = np.full((6, need.max() + 1), -1, np.int32)
    order, at = rng.permutation(n_pages), 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    draw = lambda *s: torch.from_numpy(rng.integers(0, 100, s)).to(dtype).cuda()
    total = int(q.sum()) + 3                                # 3 rows behind the last sequence
    k, v = draw(total, hkv, hd), draw(total, hkv, hd)
    kp, vp = draw(n_pages, page, hkv, hd), draw(n_pages, page, hkv, hd)
    want = [kp.clone(), vp.clone()]
    cu = np.concatenate([[0], np.cumsum(q)])
    for b in range(6):
        for i in range(q[b]):
            pos = kv[b] - q[b] + i
            for w, x in zip(want, (k, v)):
                w[table[b, pos // page], pos % page] = x[cu[b] + i]
    status = torch.zeros(1, dtype=torch.int32).cuda()
    pha.pha_cache_append(k, v, kp, vp, i32(table), i32(cu), i32(kv), status=status)
    assert torch.equal(kp, want[0]) and torch.equal(vp, want[1])
    assert status.item() == 0
    # tokens without a place are left out and reported; the others are written
    before = [kp.clone(), vp.clone()]
    for bad, code in ((-1, 4), (n_pages, 4)):
        t = table.copy()
        t[3, 0] = bad
        status.zero_()
        pha.pha_cache_append(k, v, kp, vp, i32(t), i32(cu), i32(kv), status=status)
        assert status.item() == (code if kv[3] - q[3] < page else 0)
    for lens in (kv - 300, kv + 10 ** 6):
        status.zero_()
        pha.pha_cache_append(k, v, kp, vp, i32(table), i32(cu), i32(lens), status=status)
        assert status.item() == 1
    assert torch.equal(kp, before[0]) and torch.equal(vp, before[1])


def test_append_far_into_a_large_pool(pha):
    """Byte offsets past 2^32."""
    hkv, hd, page = 8, 128, 256
    n_pages = (1 << 31) // (page * hkv * hd) + 2
    kp = torch.zeros(n_pages, page, hkv, hd, dtype=torch.bfloat16, device="cuda")
    k = torch.randn(3, hkv, hd, device="cuda").to(torch.bfloat16)
    pha.pha_cache_append(k, k, kp, kp, i32([[0, n_pages - 1]]), i32([0, 3]), i32([260]))
    assert torch.equal(kp[n_pages - 1, 1:4], k)
    assert kp[:, :1].abs().max() == 0 and kp[:-1].abs().max() == 0


@pytest.mark.parametrize("page,n_pages", [(16, 64), (1, 300), (64, 20), (4, 20000)])
def test_fork_reserve_free(pha, page, n_pages):
    c = Cache(pha, n_pages, page, n_seqs=9, max_pages=40, layers=1 if n_pages > 1000 else 2)
    p = c.plain
    steps = [([0], [5]), ([1, 2], [page, 2 * page + 1]), ([3], [0]), ([0, 1, 2], [1, 1, page])]
    for seqs, new in steps:
        c.reserve(seqs, new)
        assert p.reserve(seqs, new) is not None
        c.same()
    c.fork([0, 0, 2, 0], [4, 5, 6, 7])
    p.fork([0, 0, 2, 0], [4, 5, 6, 7])
    c.same()
    # everyone grows, the sharers copy their common last page; then only one of two sharers does
    for seqs, new in (([4, 5], [1, page + 3]), ([7, 0, 6], [1, 1, 2]), ([2], [1])):
        c.reserve(seqs, new)
        taken = p.reserve(seqs, new)
        c.same()
        assert c.count() == (0, taken)
    c.free([5, 0])
    p.free([5, 0])
    c.same()
    c.reserve([8, 5], [2 * page, 3])                        # freed pages are taken again
    p.reserve([8, 5], [2 * page, 3])
    c.same()
    c.free([1, 2, 3, 4, 5, 6, 7, 8])
    p.free([1, 2, 3, 4, 5, 6, 7, 8])
    c.same()
    assert p.refs.max() == 0


def test_sharers_that_all_grow_leave_the_common_page_free(pha):
    c = Cache(pha, 12, 8, 4, 6)
    p = c.plain
    c.reserve([0], [11]); p.reserve([0], [11])
    c.fork([0], [1]); p.fork([0], [1])
    c.reserve([0, 1], [2, 2]); p.reserve([0, 1], [2, 2])
    c.same()
    assert (p.refs == 0).sum() == 12 - 3                    # one full page shared, two copies


def test_refused_changes_change_nothing(pha):
    c = Cache(pha, 10, 8, 5, 4)
    c.reserve([0, 1], [20, 9])
    c.plain.reserve([0, 1], [20, 9])
    c.same()
    cases = [
        (lambda: c.reserve([2, 3], [32, 32]), 5),           # 8 pages, 5 are free
        (lambda: c.reserve([2], [33]), 1),                  # longer than the table
        (lambda: c.reserve([2, 2], [1, 1]), 1),             # twice in the list
        (lambda: c.reserve([5], [1]), 1),                   # no sequence
        (lambda: c.reserve([-1], [1]), 1),
        (lambda: c.reserve([0], [-1]), 1),
        (lambda: c.reserve([2], [2 ** 31 - 1]), 1),
        (lambda: c.fork([0], [1]), 1),                      # the destination is not empty
        (lambda: c.fork([0, 0], [2, 2]), 1),
        (lambda: c.fork([2, 0], [3, 2]), 1),                # a source that is a destination
        (lambda: c.fork([2], [2]), 1),
        (lambda: c.fork([7], [2]), 1),
        (lambda: c.fork([0], [9]), 1),
        (lambda: c.free([0, 0]), 1),
        (lambda: c.free([0, -1]), 1),
        (lambda: c.free([5]), 1),
    ]
    for n, (call, code) in enumerate(cases):
        c.status.zero_()
        call()
        c.same(status=code)
        assert c.count() == (code, 0), n
    # a last page that is none
    c.status.zero_()
    c.table[1, 1] = -1
    c.plain.table[1, 1] = -1
    c.reserve([1], [1])
    c.same(status=4)
    # the word keeps the largest code; empty lists are fine
    c.free([])
    c.fork([], [])
    c.reserve([], [])
    c.same(status=4)
    assert c.count() == (0, 0)


@pytest.mark.parametrize("window,sinks,paired", [(1, 0, False), (20, 0, False), (20, 3, False), (64, 17, True),
                                                 (1000, 4, False), (7, 100, True)])
def test_trim(pha, window, sinks, paired):
    c = Cache(pha, 200, 8, 6, 30)
    seqs, new = [0, 1, 2, 3, 4], [1, 8, 65, 200, 223]
    c.reserve(seqs, new); c.plain.reserve(seqs, new)
    c.fork([3], [5]); c.plain.fork([3], [5])
    c.trim(8, window, sinks, paired)
    c.plain.trim(window, sinks, 2 if paired else 1)
    c.same()
    c.trim(8, window, sinks, paired)                        # nothing more to drop
    c.same()
    c.reserve([4, 5], [1, 9]); c.plain.reserve([4, 5], [1, 9])
    c.same()


@pytest.mark.parametrize("n_pages,page,seed", [(40, 8, 0), (300, 16, 1), (9000, 4, 2), (20000, 1, 3)])
def test_compact(pha, n_pages, page, seed):
    rng = np.random.default_rng(seed)
    n_seqs = 12
    c = Cache(pha, n_pages, page, n_seqs, max(2, n_pages // 8), layers=1 if n_pages > 1000 else 3, hkv=1)
    p = c.plain
    seqs = list(range(8))
    new = rng.integers(1, max(2, page * n_pages // 12), 8).tolist()
    c.reserve(seqs, new); p.reserve(seqs, new)
    c.fork([1, 2], [8, 9]); p.fork([1, 2], [8, 9])
    c.free([0, 3, 5]); p.free([0, 3, 5])
    c.reserve([10], [3 * page]); p.reserve([10], [3 * page])
    c.compact()
    moved = p.compact()
    c.same()
    assert c.count() == (0, moved)
    assert (p.refs[: (p.refs > 0).sum()] > 0).all()
    c.compact()                                             # nothing left to move
    c.same()
    assert c.count() == (0, 0)
    c.free([1, 2, 4, 6, 7, 8, 9, 10]); p.free([1, 2, 4, 6, 7, 8, 9, 10])
    c.compact()                                             # an empty pool
    c.same()


def test_a_serving_run(pha):
    """Prompts taken in by chunks, forked, decoded with a window and sinks, trimmed and compacted on
    the way: the attention of every step equals float64 over the tokens each sequence has."""
    rng = np.random.default_rng(7)
    page, hkv, hd, H, window, sinks = 16, 2, 64, 8, 48, 5
    n_seqs, max_pages = 6, 24
    c = Cache(pha, 64, page, n_seqs, max_pages, layers=2, hkv=hkv, hd=hd)
    tokens = [[[np.zeros((0, hkv, hd))] * 2 for _ in range(2)] for _ in range(n_seqs)]   # [seq][layer][K, V]
    scratch = {}

    def step(new):
        """new: {sequence: tokens}; reserve, append and attend in both layers."""
        seqs = [s for s in new if new[s]]
        c.reserve(seqs, [new[s] for s in seqs])
        q_lens = np.array([new.get(s, 0) for s in range(n_seqs)])
        cu = np.concatenate([[0], np.cumsum(q_lens)])
        t = int(cu[-1])
        for layer in range(2):
            q, k, v = (torch.from_numpy(rng.standard_normal((t, h, hd))).to(torch.bfloat16).cuda() for h in (H, hkv, hkv))
            for s in range(n_seqs):
                for n, x in enumerate((k, v)):
                    both = list(tokens[s][layer])
                    both[n] = np.concatenate([both[n], f64(x)[cu[s]:cu[s + 1]]])
                    tokens[s][layer] = both
            pha.pha_cache_append(k, v, c.k[layer], c.v[layer], c.table, i32(cu), c.lens, status=c.status)
            o = torch.full_like(q, float("nan"))
            lse = torch.full((t, H), float("nan"), device="cuda")
            kw = dict(window=window, sinks=sinks)
            size = pha.pha_attn_paged_workspace_bytes(n_seqs, int(q_lens.max()), max_pages * page, t, H, hkv, hd,
                                                      torch.bfloat16, **kw)
            if scratch.get("n", 0) < size:
                scratch.update(n=size, ws=torch.empty(size, dtype=torch.uint8, device="cuda"))
            pha.pha_attn_paged_fwd(q, c.k[layer], c.v[layer], c.table, i32(cu), c.lens, int(q_lens.max()),
                                   max_pages * page, o, lse, scratch["ws"], status=c.status, **kw)
            Reference(f64(q), cu, lambda b: tokens[b][layer][0], lambda b: tokens[b][layer][1], window, sinks, False,
                      0.0, torch.bfloat16).check(o, lse, (new, layer))
        assert c.status.item() == 0

    step({0: 100, 1: 30})
    step({0: 77, 1: 1})
    c.fork([0, 0], [2, 3])
    for s in (2, 3):
        tokens[s] = [list(x) for x in tokens[0]]
    for _ in range(3):
        step({0: 1, 1: 1, 2: 1, 3: 1})
    c.trim(page, window, sinks)
    step({0: 1, 1: 40, 2: 1, 3: 20})
    c.free([0])
    tokens[0] = [[np.zeros((0, hkv, hd))] * 2 for _ in range(2)]
    c.compact()
    step({1: 1, 2: 3, 3: 1})
    c.trim(page, window, sinks)
    c.compact()
    step({0: 60, 1: 1, 2: 1, 3: 1, 5: 2})


def test_page_calls_in_a_graph(pha):
    """Fork, reserve, free captured and replayed: each replay does the whole cycle again."""
    c = Cache(pha, 40, 8, 6, 8)
    c.reserve([0, 1], [13, 30]); c.plain.reserve([0, 1], [13, 30])
    src, dst, new = i32([0, 0, 1]), i32([2, 3, 4]), i32([1, 9, 2])

    def cycle():
        pha.pha_cache_fork(c.table, c.lens, c.refs, src, dst, c.ws, status=c.status)
        pha.pha_cache_reserve(c.table, c.lens, c.refs, dst, new, c.k, c.v, c.ws, status=c.status)
        pha.pha_cache_free(c.table, c.lens, c.refs, dst, c.ws, status=c.status)

    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cycle()
    for _ in range(3):
        g.replay()
        c.plain.fork([0, 0, 1], [2, 3, 4])
        c.plain.reserve([2, 3, 4], [1, 9, 2])
        c.plain.free([2, 3, 4])
        c.same()


def test_reserving_more_than_31_bits_of_pages(pha):
    """The pages asked for add up past 2^31: refused as too many, nothing changed."""
    n_seqs, max_pages = 4, 1 << 29
    table = torch.empty(n_seqs, max_pages, dtype=torch.int32, device="cuda")
    lens, refs = i32([0] * n_seqs), i32([0] * 8)
    pool = [torch.zeros(1, 8, 1, 1, 8, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    ws = torch.empty(pha.pha_cache_workspace_bytes(8, n_seqs), dtype=torch.uint8, device="cuda")
    status = i32([0])
    pha.pha_cache_reserve(table, lens, refs, i32(range(4)), i32([max_pages] * 4), *pool, ws, status=status)
    assert status.item() == 5 and not lens.any() and not refs.any()
    assert pha.pha_attn_status(ws) == (5, 0)


def test_reserving_past_31_bits_of_tokens(pha):
    page, max_pages = 1 << 20, 1 << 12
    table = torch.full((1, max_pages), -1, dtype=torch.int32, device="cuda")
    have = (1 << 31) - 10
    table[0, (have - 1) // page] = 1
    lens, refs = i32([have]), i32([0, 1, 0])
    pool = [torch.zeros(1, 3, page, 1, 8, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    ws = torch.empty(pha.pha_cache_workspace_bytes(3, 1), dtype=torch.uint8, device="cuda")
    for new, code in ((9, 0), (1, 1)):
        status = i32([0])
        pha.pha_cache_reserve(table, lens, refs, i32([0]), i32([new]), *pool, ws, status=status)
        assert status.item() == code and lens.item() == (1 << 31) - 1
        assert refs.tolist() == [0, 1, 0]


@pytest.mark.parametrize("fill", ["zeros", "in range", "no page"])
def test_tables_of_empty_sequences_may_hold_anything(pha, fill):
    """A fresh table is not -1: the entries of a sequence without tokens name no pages. Reserve leaves -1
    behind what it hands out, fork of and free of empty sequences touch no page."""
    n_pages, page, n_seqs, max_pages = 30, 8, 7, 40
    c = Cache(pha, n_pages, page, n_seqs, max_pages)
    p = c.plain
    rng = np.random.default_rng(1)
    junk = {"zeros": np.zeros, "in range": lambda s: rng.integers(0, n_pages, s),
            "no page": lambda s: rng.choice([-7, n_pages, 1 << 30], s)}[fill]((n_seqs, max_pages))
    c.table.copy_(i32(junk))
    touched = set()

    def same():
        rows = sorted(touched)
        assert np.array_equal(c.table.cpu().numpy()[rows], p.table[rows])
        assert np.array_equal(c.lens.cpu().numpy(), p.lens)
        assert np.array_equal(c.refs.cpu().numpy(), p.refs)
        assert np.array_equal(f64(c.k), p.k) and np.array_equal(f64(c.v), p.v)
        assert c.status.item() == 0

    def step(call, *lists, rows):
        getattr(c, call)(*lists)
        getattr(p, call)(*lists)
        touched.update(rows)
        same()

    step("reserve", [0, 1], [20, 3], rows=[0, 1])
    step("reserve", [2], [0], rows=[])                      # no tokens, no pages: still empty
    assert c.count() == (0, 0)
    step("free", [3], rows=[3])                             # never held anything
    assert c.count() == (0, 0)
    step("fork", [0, 4, 4], [5, 3, 6], rows=[5, 3, 6])      # of an empty one too
    assert c.count() == (0, 3)
    step("reserve", [3, 5], [9, 1], rows=[])
    step("compact", rows=[])
    step("free", [0, 5, 4], rows=[4])
    step("reserve", [4, 0], [17, 1], rows=[])
    step("compact", rows=[])
    step("free", [0, 1, 3, 4, 6], rows=[])
    assert not p.refs.any()
