"""pha_attn_sinks_fwd / pha_attn_sinks_bwd on the GPU against float64 (tests/streaming.py states the
bounds). Needs a B200."""
import numpy as np
import pytest
import torch

from streaming import E, Reference, f64

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def pha():
    from paired_heads_b200 import build

    build.build()
    from paired_heads_b200 import pha as mod

    return mod


class Case:
    """Packed documents of the given lengths between `head` and `tail` rows that are in none."""

    def __init__(self, lens, H, Hkv, hd, dtype, window, sinks, paired, seed=0, head=0, tail=0,
                 scale=0.0, max_len=None):
        g = torch.Generator().manual_seed(seed)
        total = head + sum(lens) + tail
        draw = lambda n: torch.randn(total, n, hd, generator=g).to(dtype).cuda()
        self.q, self.k, self.v, self.dout = draw(H), draw(Hkv), draw(Hkv), draw(H)
        self.cu = torch.tensor(head + np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32).cuda()
        self.max_len = max(lens) if max_len is None else max_len
        self.kw = dict(window=window, sinks=sinks, paired=paired)
        self.scale, self.dtype = scale, dtype
        self.shape = (len(lens), self.max_len, H, Hkv, hd)

    def workspace(self, pha):
        return torch.empty(pha.pha_attn_sinks_workspace_bytes(*self.shape, **self.kw),
                           dtype=torch.uint8, device="cuda")

    def forward(self, pha, ws=None, stream=None):
        self.ws = self.workspace(pha) if ws is None else ws
        o = torch.full_like(self.q, float("nan"))
        lse = torch.full(self.q.shape[:2], float("nan"), device="cuda")
        pha.pha_attn_sinks_fwd(self.q, self.k, self.v, self.cu, self.max_len, o, lse, self.ws,
                               scale=self.scale, stream=stream, **self.kw)
        return o, lse

    def backward(self, pha, o, lse, stream=None):
        b, ml, h, hkv, hd = self.shape
        ws = torch.empty(pha.pha_attn_sinks_bwd_workspace_bytes(b, ml, self.q.shape[0], h, hkv, hd,
                                                                **self.kw),
                         dtype=torch.uint8, device="cuda")
        ws.fill_(255)
        grads = [torch.full_like(x, float("nan")) for x in (self.q, self.k, self.v)]
        pha.pha_attn_sinks_bwd(self.q, self.k, self.v, o, lse, self.dout, self.cu, self.max_len,
                               *grads, ws, scale=self.scale, stream=stream, **self.kw)
        self.ws_bwd = ws
        return grads

    def reference(self, grads=False):
        cu = self.cu.cpu().numpy()
        k, v = f64(self.k), f64(self.v)
        return Reference(f64(self.q), cu, lambda b: k[cu[b]:cu[b + 1]], lambda b: v[cu[b]:cu[b + 1]],
                         scale=self.scale, dtype=self.dtype, dout=f64(self.dout) if grads else None,
                         **self.kw)


def check_grads(case, ref, grads):
    """bf16: 1.25 times the derived bound plus half a step of the result (the float32 sums add terms
    near 1e-6 of the same, as in test_gpu_bwd); f32: rtol 1e-4 + 1e-5 of the largest, as there."""
    cu = case.cu.cpu().numpy()
    for name, got, want, bound, heads in (
            ("dq", grads[0], ref.dq, ref.bq, case.q.shape[1]),
            ("dk", grads[1], ref.dk, ref.bk, case.k.shape[1]),
            ("dv", grads[2], ref.dv, ref.bv, case.v.shape[1])):
        got = f64(got)
        inside = np.zeros(len(got), bool)
        inside[cu[0]:cu[-1]] = True
        if name == "dq":
            want, bound = want.reshape(got.shape)[inside], bound.reshape(got.shape)[inside]
        else:
            want, bound = (np.concatenate([x.reshape(-1, *got.shape[1:]) for x in y]) for y in (want, bound))
        assert (got[~inside] == 0).all(), f"{name}: rows outside every document are zero"
        got = got[inside]
        assert np.isfinite(got).all(), name
        top = float(np.abs(want).max())
        lim = (1.25 * (bound + 2.0 ** -8 * np.abs(want)) + 1e-6 * top if case.dtype == BF16
               else 1e-4 * np.abs(want) + 1e-5 * top)
        over = np.abs(got - want) - lim
        assert (over <= 0).all(), (name, float(over.max()), np.argwhere(over > 0)[:4].tolist())


CASES = [
    # lens, H, Hkv, hd, dtype, window, sinks, paired
    ((1,), 2, 2, 64, BF16, 1, 1, False),
    ((300, 5, 190), 6, 6, 128, BF16, 128, 8, True),      # the record's window with sinks
    ((700, 129, 1), 8, 2, 128, BF16, 100, 4, False),     # groups of 4
    ((64, 0, 1, 130), 2, 2, 64, BF16, 1, 3, True),       # window 1, an empty document
    ((1100,), 4, 4, 64, BF16, 257, 128, False),          # a whole tile of sinks
    ((2000, 40), 4, 2, 128, BF16, 300, 1, False),
    ((900,), 6, 2, 64, BF16, 64, 33, False),             # groups of 3: rows of a tile straddle tokens
    ((530, 1030), 12, 4, 64, BF16, 130, 16, True),       # paired groups of 3
    ((600,), 4, 4, 128, BF16, 0, 5, False),              # no window: the sinks change nothing
    ((400, 400), 4, 4, 128, BF16, 150, 0, False),        # no sinks
    ((500,), 2, 1, 64, BF16, 5000, 7, False),            # a window past the document
    ((384,), 34, 2, 64, BF16, 90, 10, False),            # groups of 17
    ((260,), 256, 1, 64, BF16, 70, 2, False),            # one kv head for 256
    ((4100, 1500), 2, 2, 64, BF16, 60, 4, False),        # sinks that many far queries see
    ((3000,), 4, 1, 128, BF16, 200, 100, False),
    ((2600,), 2, 2, 128, BF16, 1100, 9, True),
    ((64, 1, 37, 130), 4, 2, 16, F32, 9, 3, False),
    ((150, 20), 4, 4, 96, F32, 17, 33, True),
    ((90,), 2, 1, 5, F32, 8, 2, False),                  # an odd head_dim
    ((333,), 3, 3, 128, F32, 0, 4, False),
]


@pytest.mark.parametrize("case", CASES, ids=str)
def test_forward_and_backward(pha, case):
    lens, H, Hkv, hd, dtype, window, sinks, paired = case
    c = Case(lens, H, Hkv, hd, dtype, window, sinks, paired, seed=len(lens) + window)
    o, lse = c.forward(pha)
    ref = c.reference(grads=True)
    ref.check(o, lse)
    assert pha.pha_attn_status(c.ws)[0] == 0
    grads = c.backward(pha, o, lse)
    check_grads(c, ref, grads)
    # the same inputs give the same bits, whatever the workspace held
    o2, lse2 = c.forward(pha)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    for a, b in zip(grads, c.backward(pha, o, lse)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("H,Hkv,hd,window,paired", [(6, 6, 128, 128, True), (16, 4, 128, 300, False),
                                                    (6, 3, 64, 128, False)])
def test_a_busy_device_gives_the_bits_of_a_document_alone(pha, H, Hkv, hd, window, paired):
    """Loads of a full device come late and in any order; a document's gradients do not depend on what
    else is computed beside it (its tiles, pieces and sums are its own)."""
    lens = [1479, 700, 2047, 130, 1, 1024] * 6
    c = Case(lens, H, Hkv, hd, BF16, window, 8, paired, seed=3)
    o, lse = c.forward(pha)
    grads = c.backward(pha, o, lse)
    for _ in range(3):
        for a, b in zip(grads, c.backward(pha, o, lse)):
            assert torch.equal(a, b)
    cu = c.cu.tolist()
    for i in (0, 2, 3, 20, 35):
        lo, hi = cu[i], cu[i + 1]
        one = Case([hi - lo], H, Hkv, hd, BF16, window, 8, paired, max_len=c.max_len)
        one.q, one.k, one.v, one.dout = (x[lo:hi].clone() for x in (c.q, c.k, c.v, c.dout))
        for a, b in zip(grads, one.backward(pha, o[lo:hi].clone(), lse[lo:hi].clone())):
            assert torch.equal(a[lo:hi], b)


@pytest.mark.parametrize("dtype,hd", [(BF16, 64), (BF16, 128), (F32, 32)])
def test_rows_outside_the_documents(pha, dtype, hd):
    c = Case((150, 290), 4, 2, hd, dtype, 40, 6, False, head=3, tail=70, max_len=1000, scale=0.3)
    # neighbours of the documents hold anything
    for x in (c.q, c.k, c.v, c.dout):
        x[:3] = float("nan")
        x[-70:] = float("inf")
    o, lse = c.forward(pha)
    ref = c.reference(grads=True)
    ref.check(o, lse)
    o[:3] = lse[:3] = o[-70:] = lse[-70:] = 0
    check_grads(c, ref, c.backward(pha, o, lse))


@pytest.mark.parametrize("dtype,hd", [(BF16, 64), (F32, 16)])
def test_sinks_that_cover_nothing_equal_the_plain_window(pha, dtype, hd):
    """sinks 0 is pha_attn_fwd with the same window (each within its own rounding)."""
    c = Case((300, 77), 4, 4, hd, dtype, 50, 0, False)
    o, lse = c.forward(pha)
    ws = torch.empty(pha.pha_attn_workspace_bytes(2, 300, 4, hd, False), dtype=torch.uint8, device="cuda")
    o2, lse2 = torch.empty_like(o), torch.empty_like(lse)
    pha.pha_attn_fwd(c.q, c.k, c.v, c.cu, 300, o2, lse2, ws, window=50)
    ref = c.reference()
    ref.check(o, lse)
    assert np.abs(f64(lse - lse2)).max() <= 2 * ref.bl.max()
    bound = 2 * ref.bo.reshape(o.shape)
    assert (np.abs(f64(o) - f64(o2)) <= bound).all()


def test_large_logits(pha):
    """Logits of a few thousand: the running maximum carries them (bf16 inputs are exact)."""
    c = Case((260, 300), 2, 2, 64, BF16, 64, 4, False, scale=40.0)
    o, lse = c.forward(pha)
    c.reference().check(o, lse)


def test_gradient_against_differences(pha):
    """<gradient, direction> against central differences of sum(o * dout) in float64."""
    c = Case((37, 20), 4, 2, 16, F32, 7, 3, False, seed=5)
    o, lse = c.forward(pha)
    grads = c.backward(pha, o, lse)
    rng = np.random.default_rng(0)
    cu = c.cu.cpu().numpy()
    base = [f64(x) for x in (c.q, c.k, c.v)]
    go = f64(c.dout)

    def loss(q, k, v):
        r = Reference(q, cu, lambda b: k[cu[b]:cu[b + 1]], lambda b: v[cu[b]:cu[b + 1]], 7, 3, False,
                      0.0, F32)
        return float((r.o.reshape(go.shape) * go).sum())

    h = 1e-4
    for n in range(3):
        d = rng.standard_normal(base[n].shape)
        up, down = list(base), list(base)
        up[n], down[n] = base[n] + h * d, base[n] - h * d
        num = (loss(*up) - loss(*down)) / (2 * h)
        got = float((f64(grads[n]) * d).sum())
        # differences: h^2 of third derivatives, ~1e-7 relative to the sum of magnitudes; gradients:
        # the float32 bound of check_grads
        mag = float((np.abs(f64(grads[n])) * np.abs(d)).sum())
        assert abs(num - got) <= 2e-5 * mag, (n, num, got, mag)


def test_malformed_documents_are_reported(pha):
    c = Case((100, 60), 2, 2, 64, BF16, 16, 2, False)
    for bad in ([0, 120, 100], [-1, 100, 160], [0, 100, 161], [0, 10, 160]):   # the last: too long
        c.cu = torch.tensor(bad, dtype=torch.int32).cuda()
        o, lse = c.forward(pha)
        assert pha.pha_attn_status(c.ws)[0] == 1, bad
        assert torch.isnan(o).all() and torch.isnan(lse).all(), bad


def test_no_tokens_and_no_lse(pha):
    c = Case((0,), 2, 2, 64, BF16, 16, 2, False, max_len=0)
    o, lse = c.forward(pha)
    assert o.numel() == 0
    c = Case((200,), 2, 2, 64, BF16, 16, 2, False)
    o, lse = c.forward(pha)
    o2 = torch.empty_like(o)
    pha.pha_attn_sinks_fwd(c.q, c.k, c.v, c.cu, 200, o2, None, c.ws, **c.kw)
    assert torch.equal(o, o2)


def test_another_stream_and_a_graph(pha):
    c = Case((300, 170), 4, 2, 64, BF16, 70, 5, False)
    ref = c.reference()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        o, lse = c.forward(pha)
    torch.cuda.current_stream().wait_stream(side)
    ref.check(o, lse)
    # captured once, replayed on new inputs (two graphs that share one workspace)
    bufs = [(torch.empty_like(o), torch.empty_like(lse)) for _ in range(2)]
    graphs = []
    for ob, lb in bufs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            pha.pha_attn_sinks_fwd(c.q, c.k, c.v, c.cu, c.max_len, ob, lb, c.ws, **c.kw)
        graphs.append(g)
    c.q.copy_(torch.randn_like(c.q.float()).to(BF16))
    c.cu.copy_(torch.tensor([0, 170, 470], dtype=torch.int32))
    ref = c.reference()
    for g, (ob, lb) in zip(graphs, bufs):
        ob.fill_(float("nan"))
        lb.fill_(float("nan"))
        g.replay()
        ref.check(ob, lb)


def test_training_step_in_a_graph(pha):
    """Forward and backward captured together and replayed equal the eager calls."""
    c = Case((300, 170), 4, 2, 128, BF16, 70, 5, False)
    o, lse = c.forward(pha)
    eager = c.backward(pha, o, lse)
    out = [torch.zeros_like(x) for x in (o, lse, *eager)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pha.pha_attn_sinks_fwd(c.q, c.k, c.v, c.cu, c.max_len, out[0], out[1], c.ws, **c.kw)
        pha.pha_attn_sinks_bwd(c.q, c.k, c.v, out[0], out[1], c.dout, c.cu, c.max_len, *out[2:],
                               c.ws_bwd, **c.kw)
    g.replay()
    for a, b in zip((o, lse, *eager), out):
        assert torch.equal(a, b)


def test_one_workspace_for_every_shape(pha):
    """Different problems take turns on one forward and one backward workspace, eagerly and captured."""
    cases = [Case((700, 129, 1), 8, 2, 128, BF16, 100, 4, False, seed=1),
             Case((300, 5, 190), 6, 6, 128, BF16, 128, 8, True, seed=2),
             Case((1500,), 2, 2, 64, BF16, 60, 4, False, seed=3),
             Case((700, 129, 1), 8, 2, 128, BF16, 100, 0, False, seed=1),
             Case((64, 1, 37), 4, 2, 16, F32, 9, 3, False, seed=4)]
    wants = []
    for c in cases:
        o, lse = c.forward(pha)
        wants.append((o, lse, c.backward(pha, o, lse)))
    fwd = max((c.workspace(pha) for c in cases), key=lambda w: w.numel())
    sizes = [pha.pha_attn_sinks_bwd_workspace_bytes(c.shape[0], c.shape[1], c.q.shape[0], *c.shape[2:], **c.kw)
             for c in cases]
    bwd = torch.zeros(max(sizes), dtype=torch.uint8, device="cuda")
    outs = [[torch.empty_like(x) for x in (o, lse, *g)] for o, lse, g in wants]

    def step(i):
        c, (o, lse, *g) = cases[i], outs[i]
        pha.pha_attn_sinks_fwd(c.q, c.k, c.v, c.cu, c.max_len, o, lse, fwd, **c.kw)
        pha.pha_attn_sinks_bwd(c.q, c.k, c.v, o, lse, c.dout, c.cu, c.max_len, *g, bwd, **c.kw)

    graphs = []
    for i in range(len(cases)):
        step(i)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step(i)
        graphs.append(g)
    for turn in range(3):
        for i in (0, 1, 2, 3, 4, 0, 3, 2, 1, 4, 2, 2, 0):
            for x in outs[i]:
                x.fill_(float("nan"))
            graphs[i].replay() if (turn + i) % 2 else step(i)
            for got, want in zip(outs[i], (wants[i][0], wants[i][1], *wants[i][2])):
                assert torch.equal(got, want)


@pytest.mark.parametrize("lens,window,sinks", [((1, 1, 1), 5, 2), ((1,), 0, 0), ((300, 1, 130), 1, 0), ((1, 1), 1, 3)])
@pytest.mark.parametrize("dtype,H,Hkv,hd", [(BF16, 4, 2, 128), (BF16, 2, 2, 64), (F32, 4, 1, 48)])
def test_queries_that_see_one_key_alone(pha, dtype, H, Hkv, hd, lens, window, sinks):
    """Their softmax is 1 whatever q and k: dq and dk are zero, exactly, and dv the sum of dout."""
    c = Case(lens, H, Hkv, hd, dtype, window, sinks, False, seed=7)
    o, lse = c.forward(pha)
    assert torch.equal(o.view(-1, Hkv, H // Hkv, hd), c.v[:, :, None].expand(-1, -1, H // Hkv, -1))
    dq, dk, dv = c.backward(pha, o, lse)
    assert not dq.any() and not dk.any()
    want = c.dout.double().view(-1, Hkv, H // Hkv, hd).sum(2)
    # P is 1 up to the rounding of the log-sum-exp (2^-22 of scores up to 2^6) and, in bf16, 1 itself
    assert ((dv.double() - want).abs() <= torch.finfo(dtype).eps / 2 * want.abs() + 2.0 ** -16 * want.abs().max()).all()


@pytest.mark.parametrize("lens,window,sinks,paired", [((6, 2, 3, 16, 17), 268, 33, False), ((2, 5), 3, 1, True),
                                                      ((40, 700), 6, 2, False), ((700,), 7, 2, False),
                                                      ((1000, 3), 90, 8, True)])
@pytest.mark.parametrize("hd", [64, 128])
def test_rows_with_few_keys_keep_the_precision(pha, hd, lens, window, sinks, paired):
    """Norms of the errors of dq, dk: the results' rounding and that of dS, each uniform within half a
    step (2^-8 of the value at most; a root mean square of 2^-8 / sqrt(3) is the most that gives), and as
    much again for D and for the few rows of a short case: 2^-8 sqrt(3 / 3). Documents of a few tokens were
    off by twice that with D from the rounded o."""
    c = Case(lens, 4, 2, hd, BF16, window, sinks, paired, seed=11)
    o, lse = c.forward(pha)
    grads = c.backward(pha, o, lse)
    ref = c.reference(grads=True)
    check_grads(c, ref, grads)
    want = [ref.dq.reshape(grads[0].shape), *(np.concatenate([x.reshape(-1, 2, hd) for x in y]) for y in (ref.dk, ref.dv))]
    for got, w in zip(grads, want):
        assert np.linalg.norm(f64(got) - w) <= 2.0 ** -8 * np.linalg.norm(w)


@pytest.mark.parametrize("dtype,hd", [(BF16, 64), (BF16, 128), (F32, 24)])
@pytest.mark.parametrize("window,paired", [(2 ** 31 - 1, False), (2 ** 31 - 200, True), (2 ** 30 + 77, True),
                                           (1400, True)])
def test_loose_bounds_and_windows_past_everything(pha, dtype, hd, window, paired):
    """max_len far above every document with a window below it: the window hides nothing, and no sum of a
    position and the window wraps."""
    c = Case((700,), 4, 2, hd, dtype, window, 3, paired, max_len=2 ** 31 - 1, tail=5)
    o, lse = c.forward(pha)
    assert pha.pha_attn_status(c.ws)[0] == 0
    ref = c.reference(grads=True)
    ref.check(o, lse)
    check_grads(c, ref, c.backward(pha, o, lse))
    assert pha.pha_attn_status(c.ws_bwd)[0] == 0
    # the bits of a call without a window over a tight bound
    tight = Case((700,), 4, 2, hd, dtype, 0, 0, paired, tail=5)
    for a, b in zip(c.backward(pha, o, lse), tight.backward(pha, o, lse)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype,hd", [(BF16, 64), (F32, 16)])
def test_many_documents_of_every_length(pha, dtype, hd):
    """Lists and pieces at their bound: ragged tiles in every document, empty ones between."""
    lens = [1, 0, 129, 257, 0, 1, 1, 385, 128, 127, 0, 1300, 1, 2, 3, 0, 1153] if dtype is BF16 else [1, 0, 33, 2, 0, 65, 1]
    c = Case(lens, 2, 1, hd, dtype, 3, 2, False, max_len=10 ** 6)
    o, lse = c.forward(pha)
    ref = c.reference(grads=True)
    ref.check(o, lse)
    check_grads(c, ref, c.backward(pha, o, lse))
    assert pha.pha_attn_status(c.ws_bwd)[0] == 0


MALFORMED = [[0, 120, 100], [-1, 100, 160], [0, 100, 161], [0, 10, 160],          # (the last: too long)
             [170, 170, 170], [0, -3, 160], [-5, -4, -3], [2 ** 31 - 1, 0, 160], [0, 2 ** 31 - 1, -2 ** 31],
             [40, 100, 130]]                                                        # well formed, rows around it


@pytest.mark.parametrize("dtype,H,Hkv,hd,window,sinks,paired", [
    (BF16, 2, 2, 64, 16, 2, False), (BF16, 4, 2, 128, 16, 2, True), (BF16, 4, 2, 64, 5, 2, False),   # (5 + 2: D from keys)
    (BF16, 2, 2, 128, 7, 0, True), (BF16, 2, 1, 64, 0, 3, False), (F32, 4, 2, 24, 9, 3, False), (F32, 2, 2, 16, 0, 0, True)])
def test_malformed_documents_in_both_directions(pha, dtype, H, Hkv, hd, window, sinks, paired):
    """Status 1, nothing written forward, and no gradient row other than zeros outside [cu[0], cu[-1]); the same
    workspaces then serve well-formed documents."""
    c = Case((100, 60), H, Hkv, hd, dtype, window, sinks, paired, max_len=130)
    good = c.cu.clone()
    o, lse = c.forward(pha)
    want = c.backward(pha, o, lse)
    ws, n = c.ws_bwd, c.q.shape[0]
    for bad in MALFORMED:
        ok = bad == MALFORMED[-1]
        c.cu.copy_(torch.tensor(bad, dtype=torch.int32))
        got, got_lse = c.forward(pha, ws=c.ws)
        assert pha.pha_attn_status(c.ws)[0] == (0 if ok else 1), bad
        if not ok:
            assert torch.isnan(got).all() and torch.isnan(got_lse).all(), bad
        grads = [torch.full_like(x, float("nan")) for x in want]
        pha.pha_attn_sinks_bwd(c.q, c.k, c.v, o, lse, c.dout, c.cu, c.max_len, *grads, ws, **c.kw)
        assert pha.pha_attn_status(ws)[0] == (0 if ok else 1), bad
        lo, hi = max(min(bad[0], n), 0), max(min(bad[2], n), 0)
        for g in grads:
            inside = g[lo:max(hi, lo)]
            assert ok or torch.isnan(inside).all(), bad
            assert (torch.isnan(g) | (g == 0)).all() or ok, bad
            if ok:
                assert torch.isfinite(g).all() and not g[:lo].any() and not g[hi:].any()
        c.cu.copy_(good)
        grads = [torch.full_like(x, float("nan")) for x in want]
        pha.pha_attn_sinks_bwd(c.q, c.k, c.v, o, lse, c.dout, c.cu, c.max_len, *grads, ws, **c.kw)
        for a, b in zip(grads, want):
            assert torch.equal(a, b), bad


def test_malformed_documents_with_far_pieces(pha):
    """Sinks that many query tiles see: the pieces' sums are not taken either."""
    c = Case((4100, 1500), 2, 2, 64, BF16, 60, 4, False, max_len=4200)
    o, lse = c.forward(pha)
    want = c.backward(pha, o, lse)
    good = c.cu.clone()
    for bad in ([0, 4300, 5600], [0, 4100, 5601], [-1, 4099, 5600], [0, 4100, 4000]):
        c.cu.copy_(torch.tensor(bad, dtype=torch.int32))
        grads = [torch.full_like(x, float("nan")) for x in want]
        pha.pha_attn_sinks_bwd(c.q, c.k, c.v, o, lse, c.dout, c.cu, c.max_len, *grads, c.ws_bwd, **c.kw)
        assert pha.pha_attn_status(c.ws_bwd)[0] == 1, bad
        for g in grads:
            assert torch.isnan(g[:min(bad[2], 5600)]).all() and not g[min(bad[2], 5600):].any(), bad
    c.cu.copy_(good)
    grads = [torch.full_like(x, float("nan")) for x in want]
    pha.pha_attn_sinks_bwd(c.q, c.k, c.v, o, lse, c.dout, c.cu, c.max_len, *grads, c.ws_bwd, **c.kw)
    for a, b in zip(grads, want):
        assert torch.equal(a, b)
