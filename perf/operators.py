"""The serving and streaming operators that perf measurements run: attention with a sliding window
and visible first tokens (sinks), forward and backward; attention of new tokens over a paged cache;
and the pages of that cache (append, fork, reserve, free, trim, compact).

``own`` False runs the plain forms (elementary torch operations in float32); ``own`` True runs the
library's entry points (paired_heads_b200.pha) on the same state.

Layouts are the library's: q [tokens][H][hd], k / v [tokens][Hkv][hd], documents packed one after
another; a cache layer is [pages][page_size][Hkv][hd] and a sequence's tokens follow its row of the
page table. Paired cases read the same bytes as [2 tokens][H/2][hd]; windows and sinks count slots
of that view.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
BLOCK = 128  # query rows the plain forms take at a time


# ------------------------------------------------------------------------------------- the cases

def listed():
    return [
        # a unit-test sized model step in float32: launch latency
        dict(name="sinks_f32_small", kind="sinks", docs="list", lens="64,1,37,130", heads=4, kv_heads=2, hd=16,
             dtype="f32", window=9, sinks=3, paired=False, train=True),
        # the paired-head record's packed training row (65,536 tokens, window 128) with 8 sink slots
        dict(name="sinks_train_paired", kind="sinks", docs="geometric", total=65536, mean=512, cap=2048, heads=6,
             kv_heads=6, hd=128, dtype="bf16", window=128, sinks=8, paired=True, train=True),
        # long-context training with grouped heads
        dict(name="sinks_train_gqa", kind="sinks", docs="list", lens="8192,8192", heads=32, kv_heads=8, hd=128,
             dtype="bf16", window=1024, sinks=4, paired=False, train=True),
        # evaluation of a GPT-2 sized model on long documents: forward only
        dict(name="sinks_fwd_gpt2", kind="sinks", docs="list", lens="8192,8192,8192,8191", heads=12, kv_heads=12,
             hd=64, dtype="bf16", window=1024, sinks=16, paired=False, train=False),
        # one user, one token, a short history: latency
        dict(name="decode_one", kind="paged", batch=1, q_min=1, q_max=1, kv_min=333, kv_max=333, heads=12,
             kv_heads=12, hd=64, dtype="bf16", page=16, window=0, sinks=0, paired=False),
        # a full serving batch of single tokens over ragged histories
        dict(name="decode_batch", kind="paged", batch=64, q_min=1, q_max=1, kv_min=1, kv_max=8192, heads=32,
             kv_heads=8, hd=128, dtype="bf16", page=64, window=0, sinks=0, paired=False),
        # endless streams: single tokens that see 4096 slots back and 8 sink slots
        dict(name="decode_stream_paired", kind="paged", batch=32, q_min=1, q_max=1, kv_min=2000, kv_max=65536,
             heads=6, kv_heads=6, hd=128, dtype="bf16", page=32, window=4096, sinks=8, paired=True),
        # two long prompts taken in by chunks: the last chunk over a 16K cache
        dict(name="chunk_long", kind="paged", batch=2, q_min=1000, q_max=1024, kv_min=16000, kv_max=16384, heads=32,
             kv_heads=8, hd=128, dtype="bf16", page=128, window=0, sinks=0, paired=False),
        # a mixed step: single tokens and prompt chunks of many users together
        dict(name="chunk_mixed", kind="paged", batch=24, q_min=1, q_max=300, kv_min=300, kv_max=4096, heads=12,
             kv_heads=12, hd=64, dtype="bf16", page=16, window=1024, sinks=16, paired=False),
        # the keys and values of a prefill step written to one layer's pages
        dict(name="append_prefill", kind="append", batch=40, q_min=1, q_max=3200, kv_extra=2000, kv_heads=8, hd=128,
             dtype="bf16", page=64),
        # parallel sampling: every prompt forked, room for the next tokens (a shared last page is
        # copied), the samples freed again
        dict(name="pages_fork", kind="fork", prompts=8, samples=8, kv_min=100, kv_max=2000, new=5, kv_heads=8, hd=128,
             dtype="bf16", page=64, layers=4),
        # a fragmented pool after a burst: what no window sees is released, the rest moved together
        dict(name="pages_compact", kind="compact", seqs=48, kv_min=1, kv_max=6000, spare=0.5, window=2048, sinks=16,
             kv_heads=8, hd=128, dtype="bf16", page=64, layers=2),
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["sinks", "sinks", "paged", "paged", "paged", "append", "fork", "compact"])
    page = rng.choice([8, 16, 32, 64, 128, 256])
    kv_heads = rng.choice([1, 2, 4, 6, 8])
    hd = rng.choice([64, 128])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    heads = kv_heads * rng.choice([1, 1, 2, 3, 4, 8])
    paired = kv_heads % 2 == 0 and rng.random() < 0.4
    if kind == "sinks":
        f32 = dtype == "f32"
        total = _log(rng, 1, 900 if f32 else 16000)
        return dict(kind="sinks", docs="geometric", total=total, mean=_log(rng, max(1, total // 40), max(2, total)), cap=total,
                    heads=heads, kv_heads=kv_heads, hd=rng.choice([16, 32, 64, 96, 128]) if f32 else hd, dtype=dtype,
                    window=_log(rng, 1, 2048), sinks=rng.choice([0, 1, 3, 4, 8, 16, 33, 64, 128]), paired=paired,
                    train=rng.random() < 0.7)
    if kind == "paged":
        f32 = dtype == "f32"
        q_max = rng.choice([1, 1, _log(rng, 2, 700)])
        batch = _log(rng, 1, 64 if q_max == 1 else 8)
        kv_max = max(q_max, _log(rng, 1, 2000 if f32 else (16000 if batch <= 16 else 4000)))
        return dict(kind="paged", batch=batch, q_min=rng.choice([1, q_max]), q_max=q_max,
                    kv_min=rng.choice([q_max, kv_max]), kv_max=kv_max, heads=heads, kv_heads=kv_heads,
                    hd=rng.choice([16, 32, 64, 96, 128]) if f32 else hd, dtype=dtype, page=page,
                    window=rng.choice([0, _log(rng, 1, 4096)]), sinks=rng.choice([0, 1, 4, 8, 16, 100]), paired=paired)
    if kind == "append":
        return dict(kind="append", batch=_log(rng, 1, 64), q_min=1, q_max=_log(rng, 1, 1500), kv_extra=_log(rng, 1, 3000),
                    kv_heads=kv_heads, hd=hd, dtype=dtype, page=page)
    if kind == "fork":
        kv_max = _log(rng, 1, 2000)
        return dict(kind="fork", prompts=_log(rng, 1, 16), samples=_log(rng, 1, 8), kv_min=rng.choice([1, kv_max]),
                    kv_max=kv_max, new=_log(rng, 1, 200), kv_heads=kv_heads, hd=hd, dtype=dtype, page=page,
                    layers=rng.choice([1, 2, 3]))
    kv_max = _log(rng, 1, 4000)
    return dict(kind="compact", seqs=_log(rng, 1, 48), kv_min=rng.choice([1, kv_max]), kv_max=kv_max,
                spare=rng.choice([0.1, 0.5, 2.0]), window=_log(rng, 1, 4096), sinks=rng.choice([0, 1, 4, 16, 100]),
                kv_heads=kv_heads, hd=hd, dtype=dtype, page=page, layers=rng.choice([1, 2, 3]))


def _doc_lens(case):
    """The documents of a training row: given, or geometric lengths cut to fill the row."""
    if case["docs"] == "list":
        return [int(x) for x in case["lens"].split(",")]
    total = case["total"]
    n = np.minimum(np.random.default_rng(total).geometric(1.0 / max(1, case["mean"]), size=total), case["cap"])
    ends = np.minimum(np.cumsum(n), total)
    ends = ends[: int(np.searchsorted(ends, total)) + 1]
    return np.diff(np.concatenate([[0], ends])).tolist()


def _ragged(case):
    """Chunk and cache lengths of a paged batch (the case's own, whatever the seed): the first
    sequence has the longest of both."""
    rng = np.random.default_rng([case["batch"], case["q_max"], 77])
    n = case["batch"]
    q = rng.integers(case["q_min"], case["q_max"] + 1, n)
    q[0] = case["q_max"]
    if case["kind"] == "append":
        kv = q + rng.integers(0, case["kv_extra"] + 1, n)
    else:
        kv = np.maximum(rng.integers(case["kv_min"], case["kv_max"] + 1, n), q)
        kv[0] = case["kv_max"]
    return q, kv


# ------------------------------------------------------------------------------------ the inputs

def _randn(seed, *shape, dtype):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda", dtype=dtype)


def _ints(a):
    return torch.as_tensor(np.asarray(a), dtype=torch.int32).cuda()


def _held(case):
    """Tokens that the sequences of a managed cache hold (the case's own, whatever the seed)."""
    rng = np.random.default_rng([case["kv_max"], 5])
    return rng.integers(case["kv_min"], case["kv_max"] + 1, case["prompts" if case["kind"] == "fork" else "seqs"])


def _tables(lens, page, n_pages, rng):
    """Page tables of sequences whose pages lie scattered over the pool: (table, pages used)."""
    need = -(-np.asarray(lens) // page)
    table = np.full((len(need), max(1, int(need.max()))), -1, np.int32)
    at = np.arange(table.shape[1])[None, :] < need[:, None]
    table[at] = rng.permutation(n_pages)[: int(need.sum())]
    return table, at


def prepare(case, seed):
    dt = DTYPES[case["dtype"]]
    kind, hd, hkv = case["kind"], case["hd"], case["kv_heads"]
    rng = np.random.default_rng([seed, 5])
    s = dict(case=case)
    if kind == "sinks":
        lens = _doc_lens(case)
        total = sum(lens)
        h = case["heads"]
        s.update(q=_randn(seed * 8 + 1, total, h, hd, dtype=dt), k=_randn(seed * 8 + 2, total, hkv, hd, dtype=dt),
                 v=_randn(seed * 8 + 3, total, hkv, hd, dtype=dt), cu=_ints(np.concatenate([[0], np.cumsum(lens)])),
                 max_len=max(lens))
        s["o"], s["lse"] = torch.empty_like(s["q"]), torch.empty(total, h, device="cuda")
        if case["train"]:
            s["dout"] = _randn(seed * 8 + 4, total, h, hd, dtype=dt)
            s["dq"], s["dk"], s["dv"] = (torch.empty_like(s[n]) for n in ("q", "k", "v"))
        return s
    page = case["page"]
    if kind in ("paged", "append"):
        q, kv = _ragged(case)
        used = int((-(-kv // page)).sum())
        n_pages = used + max(1, used // 8)
        table, _ = _tables(kv, page, n_pages, rng)
        s.update(table=_ints(table), cu=_ints(np.concatenate([[0], np.cumsum(q)])), lens=_ints(kv), max_q=int(q.max()),
                 max_kv=int(kv.max()), k_pages=_randn(seed * 8 + 2, n_pages, page, hkv, hd, dtype=dt),
                 v_pages=_randn(seed * 8 + 3, n_pages, page, hkv, hd, dtype=dt),
                 status=torch.zeros(1, dtype=torch.int32, device="cuda"))
        if kind == "append":
            s.update(k=_randn(seed * 8 + 5, int(q.sum()), hkv, hd, dtype=dt),
                     v=_randn(seed * 8 + 6, int(q.sum()), hkv, hd, dtype=dt))
        else:
            s["q"] = _randn(seed * 8 + 1, int(q.sum()), case["heads"], hd, dtype=dt)
            s["o"], s["lse"] = torch.empty_like(s["q"]), torch.empty(int(q.sum()), case["heads"], device="cuda")
        return s
    layers = case["layers"]
    if kind == "fork":
        p, n = case["prompts"], case["samples"]
        kv = _held(case)
        room = -(-(kv.max() + case["new"]) // page)
        used = int((-(-kv // page)).sum())
        n_pages = used + p * n * (-(-case["new"] // page) + 1)
        table, at = _tables(kv, page, n_pages, rng)
        full = np.full((p * (n + 1), room), -1, np.int32)
        full[:p, : table.shape[1]] = table
        lens = np.concatenate([kv, np.zeros(p * n, np.int64)])
        s.update(src=_ints(np.repeat(np.arange(p), n)), dst=_ints(p + np.arange(p * n)),
                 new=_ints(np.full(p * n, case["new"])))
    else:
        lens = _held(case)
        used = int((-(-lens // page)).sum())
        n_pages = used + int(math.ceil(used * case["spare"]))
        full, at = _tables(lens, page, n_pages, rng)
        table = full
    refs = np.zeros(n_pages, np.int32)
    refs[table[at]] = 1
    s.update(table=_ints(full), lens=_ints(lens), refs=_ints(refs),
             k_cache=_randn(seed * 8 + 2, layers, n_pages, page, hkv, hd, dtype=dt),
             v_cache=_randn(seed * 8 + 3, layers, n_pages, page, hkv, hd, dtype=dt),
             status=torch.zeros(1, dtype=torch.int32, device="cuda"))
    s["table0"], s["refs0"] = s["table"].clone(), s["refs"].clone()
    return s


# ------------------------------------------------------------------------------- the plain forms

def _attend(q, k, v, vis, scale):
    """q [n][B][g][x][d], k / v [n][K][g][d], vis [n][B][K]: weights, output and log-sum-exp."""
    sc = torch.einsum("nbgxd,nkgd->ngxbk", q, k) * scale
    m5 = vis[:, None, None]
    sc = sc.masked_fill(~m5, -math.inf)
    m = sc.amax(-1, keepdim=True).clamp_min(-3e38)
    p = torch.exp(sc - m)
    l = p.sum(-1, keepdim=True)
    p = p / l.clamp_min(1e-30)
    return p, torch.einsum("ngxbk,nkgd->nbgxd", p, v), (m + torch.log(l))[..., 0]


def _plain_sinks(s):
    c = s["case"]
    mult = 2 if c["paired"] else 1
    h, g, hd, w, n_sink = c["heads"] // mult, c["kv_heads"] // mult, c["hd"], c["window"], c["sinks"]
    q, k, v = (s[n].float().view(-1, x, hd) for n, x in (("q", h), ("k", g), ("v", g)))
    cu = s["cu"].long() * mult
    lens = cu[1:] - cu[:-1]
    nb = (lens + BLOCK - 1) // BLOCK
    doc = torch.repeat_interleave(torch.arange(len(lens), device="cuda"), nb)
    first = torch.cumsum(nb, 0) - nb
    lo, hi = cu[doc], cu[doc + 1]
    start = lo + (torch.arange(len(doc), device="cuda") - first[doc]) * BLOCK
    rows = start[:, None] + torch.arange(BLOCK, device="cuda")
    reach = min(w, s["max_len"] * mult)  # no key lies further back than the longest document
    band = start[:, None] - (reach - 1) + torch.arange(BLOCK + reach - 1, device="cuda")
    sink = lo[:, None] + torch.arange(min(n_sink, s["max_len"] * mult), device="cuda")
    keys = torch.cat([band, sink], 1)
    back = rows[:, :, None] - keys[:, None, :]
    vis = (back >= 0) & (keys >= lo[:, None])[:, None, :] & (rows < hi[:, None])[:, :, None]
    is_sink = (torch.arange(keys.shape[1], device="cuda") >= band.shape[1])
    vis &= torch.where(is_sink, back >= w, back < w)
    ok = rows < hi[:, None]
    at = rows.clamp(max=q.shape[0] - 1)
    ka = keys.clamp(0, q.shape[0] - 1)
    scale = hd ** -0.5
    qb = q[at].view(*at.shape, g, h // g, hd)
    kb, vb = k[ka], v[ka]
    p, o, lse = _attend(qb, kb, vb, vis, scale)
    out = torch.zeros_like(q)
    out[rows[ok]] = o.reshape(*at.shape, h, hd)[ok]
    lse_out = torch.zeros(q.shape[0], h, device="cuda")
    lse_out[rows[ok]] = lse.permute(0, 3, 1, 2).reshape(*at.shape, h)[ok]
    dt = s["q"].dtype
    got = dict(o=out.view(s["q"].shape).to(dt), lse=lse_out.view(-1, c["heads"]))
    if not c["train"]:
        return got
    dob = s["dout"].float().view(-1, h, hd)[at].view(*at.shape, g, h // g, hd)
    dob = dob * ok[:, :, None, None, None]
    dp = torch.einsum("nbgxd,nkgd->ngxbk", dob, vb)
    ds = p * (dp - (p * dp).sum(-1, keepdim=True))
    dq = torch.zeros_like(q)
    dq[rows[ok]] = (torch.einsum("ngxbk,nkgd->nbgxd", ds, kb) * scale).reshape(*at.shape, h, hd)[ok]
    dk, dv = torch.zeros_like(k), torch.zeros_like(v)
    dk.index_add_(0, ka.reshape(-1), (torch.einsum("ngxbk,nbgxd->nkgd", ds, qb) * scale).reshape(-1, g, hd))
    dv.index_add_(0, ka.reshape(-1), torch.einsum("ngxbk,nbgxd->nkgd", p, dob).reshape(-1, g, hd))
    got.update(dq=dq.view(s["q"].shape).to(dt), dk=dk.view(s["k"].shape).to(dt), dv=dv.view(s["v"].shape).to(dt))
    return got


def _flat_rows(table, pos, page):
    """Rows of the pool (pages times page size) that hold positions pos [n][K] of the sequences."""
    pages = torch.gather(table.long(), 1, (pos // page).clamp(0, table.shape[1] - 1))
    return pages.clamp(min=0) * page + pos % page


def _plain_paged(s):
    c = s["case"]
    mult = 2 if c["paired"] else 1
    h, g, hd, w, n_sink = c["heads"] // mult, c["kv_heads"] // mult, c["hd"], c["window"], c["sinks"]
    page = c["page"] * mult
    q = s["q"].float().view(-1, h, hd)
    cu, kv = s["cu"].long() * mult, s["lens"].long() * mult
    ql = cu[1:] - cu[:-1]
    max_q, max_kv = s["max_q"] * mult, s["max_kv"] * mult
    i = torch.arange(max_q, device="cuda")
    rows = cu[:-1, None] + i
    ok = i < ql[:, None]
    pos = (kv - ql)[:, None] + i
    width = max_kv if w == 0 else min(max_kv, w + max_q - 1)
    lo = (pos[:, :1] - w + 1).clamp(min=0) if w else torch.zeros_like(pos[:, :1])
    sink = torch.arange(min(n_sink, max_kv) if w else 0, device="cuda").expand(len(kv), -1)
    keys = torch.cat([lo + torch.arange(width, device="cuda"), sink], 1)
    back = pos[:, :, None] - keys[:, None, :]
    vis = (back >= 0) & ok[:, :, None]
    if w:
        is_sink = torch.arange(keys.shape[1], device="cuda") >= width
        vis &= torch.where(is_sink, back >= w, back < w)
    at = rows.clamp(max=q.shape[0] - 1)
    flat = _flat_rows(s["table"], keys, page)
    kb, vb = (s[n].view(-1, g, hd)[flat].float() for n in ("k_pages", "v_pages"))
    _, o, lse = _attend(q[at].view(*at.shape, g, h // g, hd), kb, vb, vis, hd ** -0.5)
    out = torch.zeros_like(q)
    out[rows[ok]] = o.reshape(*at.shape, h, hd)[ok]
    lse_out = torch.zeros(q.shape[0], h, device="cuda")
    lse_out[rows[ok]] = lse.permute(0, 3, 1, 2).reshape(*at.shape, h)[ok]
    return dict(o=out.view(s["q"].shape).to(s["q"].dtype), lse=lse_out.view(-1, c["heads"]))


def _plain_append(s):
    page = s["case"]["page"]
    cu, kv = s["cu"].long(), s["lens"].long()
    ql = cu[1:] - cu[:-1]
    t = torch.arange(s["k"].shape[0], device="cuda")
    b = torch.searchsorted(cu, t, right=True) - 1
    pos = kv[b] - ql[b] + t - cu[b]
    flat = s["table"].long()[b, pos // page] * page + pos % page
    hkv, hd = s["k"].shape[1:]
    s["k_pages"].view(-1, hkv, hd)[flat] = s["k"]
    s["v_pages"].view(-1, hkv, hd)[flat] = s["v"]
    return dict(k_pages=s["k_pages"], v_pages=s["v_pages"])


def _plain_fork(s):
    page = s["case"]["page"]
    table, lens, refs, src, dst = s["table"], s["lens"], s["refs"], s["src"].long(), s["dst"].long()
    # fork: the samples share their prompt's pages
    table[dst] = table[src]
    lens[dst] = lens[src]
    held = table[dst]
    refs.index_add_(0, held[held >= 0].long(), torch.ones_like(held[held >= 0]))
    # reserve: pages for the new tokens, lowest free page first; a shared last page is copied
    n = lens[dst].long()
    new = s["new"].long()
    have = (n + page - 1) // page
    last = torch.gather(table[dst].long(), 1, (have - 1).clamp(min=0)[:, None])[:, 0]
    copied = (new > 0) & (n % page != 0) & (refs[last.clamp(min=0)] > 1)
    need = (n + new + page - 1) // page - have + copied
    first = torch.cumsum(need, 0) - need
    free = torch.nonzero(refs == 0)[:, 0]
    j = torch.arange(int(need.max()), device="cuda")
    at = j < need[:, None]
    got = free[(first[:, None] + j)[at]]
    table[dst[:, None].expand(at.shape)[at], ((have - copied.long())[:, None] + j)[at]] = got.int()
    refs[got] = 1
    old, to = last[copied], free[first[copied]]
    refs.index_add_(0, old, torch.full_like(old, -1, dtype=torch.int32))
    lens[dst] += new.int()
    s["k_cache"][:, to] = s["k_cache"][:, old]
    s["v_cache"][:, to] = s["v_cache"][:, old]
    out = dict(table=table.clone(), lens=lens.clone(), refs=refs.clone())
    # free: the samples let go of their pages
    held = table[dst]
    refs.index_add_(0, held[held >= 0].long(), torch.full_like(held[held >= 0], -1))
    table[dst] = -1
    lens[dst] = 0
    out.update(freed=refs, k_cache=s["k_cache"], v_cache=s["v_cache"])
    return out


def _plain_compact(s):
    c = s["case"]
    page = c["page"]
    table, refs = s["table"], s["refs"]
    table.copy_(s["table0"])
    refs.copy_(s["refs0"])
    # trim: pages that the next token's window and the sinks leave out
    begin = torch.arange(table.shape[1], device="cuda") * page
    out = (table >= 0) & (begin >= c["sinks"]) & (begin + page <= (s["lens"][:, None] - c["window"] + 1))
    gone = table[out].long()
    refs.index_add_(0, gone, torch.full_like(gone, -1, dtype=torch.int32))
    table[out] = -1
    # compact: the live pages behind the first n_live move into the free ones before it, in order
    live = refs > 0
    n_live = live.sum()
    at = torch.arange(len(refs), device="cuda")
    src, hole = torch.nonzero(live & (at >= n_live))[:, 0], torch.nonzero(~live & (at < n_live))[:, 0]
    s["k_cache"][:, hole] = s["k_cache"][:, src]
    s["v_cache"][:, hole] = s["v_cache"][:, src]
    to = at.clone()
    to[src] = hole
    table.copy_(torch.where(table >= 0, to[table.long().clamp(min=0)].int(), table))
    refs[hole] = refs[src]
    refs[src] = 0
    return dict(table=table, refs=refs, k_cache=s["k_cache"], v_cache=s["v_cache"])


# --------------------------------------------------------------------------- the library's calls

def _scratch(s, name, nbytes):
    """A workspace that the program keeps with its state."""
    if name not in s:
        s[name] = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    return s[name]


def _own_sinks(s):
    from paired_heads_b200 import pha

    c = s["case"]
    kw = dict(window=c["window"], sinks=c["sinks"], paired=c["paired"])
    batch = s["cu"].shape[0] - 1
    if "ws" not in s:
        _scratch(s, "ws", pha.pha_attn_sinks_workspace_bytes(batch, s["max_len"], c["heads"], c["kv_heads"], c["hd"],
                                                             **kw))
    pha.pha_attn_sinks_fwd(s["q"], s["k"], s["v"], s["cu"], s["max_len"], s["o"], s["lse"], s["ws"], **kw)
    if not c["train"]:
        return dict(o=s["o"], lse=s["lse"])
    if "wsb" not in s:
        _scratch(s, "wsb", pha.pha_attn_sinks_bwd_workspace_bytes(batch, s["max_len"], s["q"].shape[0], c["heads"],
                                                                  c["kv_heads"], c["hd"], **kw))
    pha.pha_attn_sinks_bwd(s["q"], s["k"], s["v"], s["o"], s["lse"], s["dout"], s["cu"], s["max_len"], s["dq"],
                           s["dk"], s["dv"], s["wsb"], **kw)
    return dict(o=s["o"], lse=s["lse"], dq=s["dq"], dk=s["dk"], dv=s["dv"])


def _own_paged(s):
    from paired_heads_b200 import pha

    c = s["case"]
    kw = dict(window=c["window"], sinks=c["sinks"], paired=c["paired"])
    if "ws" not in s:
        _scratch(s, "ws", pha.pha_attn_paged_workspace_bytes(c["batch"], s["max_q"], s["max_kv"], s["q"].shape[0],
                                                             c["heads"], c["kv_heads"], c["hd"], s["q"].dtype, **kw))
    pha.pha_attn_paged_fwd(s["q"], s["k_pages"], s["v_pages"], s["table"], s["cu"], s["lens"], s["max_q"],
                           s["max_kv"], s["o"], s["lse"], s["ws"], status=s["status"], **kw)
    return dict(o=s["o"], lse=s["lse"])


def _own_append(s):
    from paired_heads_b200 import pha

    pha.pha_cache_append(s["k"], s["v"], s["k_pages"], s["v_pages"], s["table"], s["cu"], s["lens"],
                         status=s["status"])
    return dict(k_pages=s["k_pages"], v_pages=s["v_pages"])


def _own_fork(s):
    from paired_heads_b200 import pha

    if "ws" not in s:
        _scratch(s, "ws", pha.pha_cache_workspace_bytes(s["refs"].shape[0], s["table"].shape[0]))
    table, lens, refs = s["table"], s["lens"], s["refs"]
    pha.pha_cache_fork(table, lens, refs, s["src"], s["dst"], s["ws"], status=s["status"])
    pha.pha_cache_reserve(table, lens, refs, s["dst"], s["new"], s["k_cache"], s["v_cache"], s["ws"],
                          status=s["status"])
    out = dict(table=table.clone(), lens=lens.clone(), refs=refs.clone())
    pha.pha_cache_free(table, lens, refs, s["dst"], s["ws"], status=s["status"])
    out.update(freed=refs, k_cache=s["k_cache"], v_cache=s["v_cache"])
    return out


def _own_compact(s):
    from paired_heads_b200 import pha

    c = s["case"]
    if "ws" not in s:
        _scratch(s, "ws", pha.pha_cache_workspace_bytes(s["refs"].shape[0], s["table"].shape[0]))
    s["table"].copy_(s["table0"])
    s["refs"].copy_(s["refs0"])
    pha.pha_cache_trim(s["table"], s["lens"], s["refs"], c["page"], window=c["window"], sinks=c["sinks"],
                       status=s["status"])
    pha.pha_cache_compact(s["table"], s["refs"], s["k_cache"], s["v_cache"], s["ws"], status=s["status"])
    return dict(table=s["table"], refs=s["refs"], k_cache=s["k_cache"], v_cache=s["v_cache"])


def run(state):
    kind = state["case"]["kind"]
    if own:
        calls = dict(sinks=_own_sinks, paged=_own_paged, append=_own_append, fork=_own_fork, compact=_own_compact)
    else:
        calls = dict(sinks=_plain_sinks, paged=_plain_paged, append=_plain_append, fork=_plain_fork,
                     compact=_plain_compact)
    return calls[kind](state)


# ------------------------------------------------------------------------------ work and exactness

def _pairs(first, n, window, sinks):
    """Visible (query, key) pairs of queries at positions first .. first + n - 1."""
    i = np.arange(first + 1, first + n + 1, dtype=np.int64)
    if not window:
        return int(i.sum())
    return int((np.minimum(i, window) + np.minimum(sinks, np.maximum(i - window, 0))).sum())


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    kind, hd, hkv = case["kind"], case["hd"], case["kv_heads"]
    mult = 2 if case.get("paired") else 1
    if kind == "sinks":
        lens = _doc_lens(case)
        total, h = sum(lens), case["heads"]
        pairs = sum(_pairs(0, n * mult, case["window"], case["sinks"]) for n in lens) * (h // mult)
        fwd = total * (2 * h + 2 * hkv) * hd * e + total * h * 4
        if not case["train"]:
            return {"bytes": fwd, "flops": 4 * hd * pairs}
        return {"bytes": fwd + total * (2 * h + 2 * hkv) * hd * e, "flops": 14 * hd * pairs}
    if kind in ("paged", "append"):
        q, kv = _ragged(case)
        if kind == "append":
            return {"bytes": 4 * int(q.sum()) * hkv * hd * e, "flops": 0}
        w, n_sink, h = case["window"], case["sinks"], case["heads"]
        pairs = sum(_pairs(int(b - a) * mult, int(a) * mult, w, n_sink) for a, b in zip(q, kv)) * (h // mult)
        lo = np.maximum((kv - q) * mult - w + 1, 0) if w else np.zeros_like(kv)
        seen = int((kv * mult - lo + np.minimum(n_sink, lo)).sum()) * (hkv // mult)
        return {"bytes": 2 * seen * hd * e + int(q.sum()) * h * (2 * hd * e + 4), "flops": 4 * hd * pairs}
    page = case["page"]
    row = case["layers"] * 2 * page * hkv * hd * e
    if kind == "fork":
        kv = _held(case)
        copies = int((kv % page != 0).sum()) * case["samples"]
        held = int((-(-kv // page)).sum()) * (case["samples"] + 1)
        return {"bytes": 2 * copies * row + 16 * held, "flops": 0}
    lens = _held(case)
    need = -(-lens // page)
    begin = np.arange(int(need.max()))[None, :] * page
    held = begin < (need * page)[:, None]
    gone = held & (begin >= case["sinks"]) & (begin + page <= (lens - case["window"] + 1)[:, None])
    used = int(need.sum())
    n_pages, live = used + int(math.ceil(used * case["spare"])), int(held.sum() - gone.sum())
    moved = live * (1.0 - live / n_pages)  # expected: live pages lie anywhere in the pool
    return {"bytes": 2 * moved * row + 8 * n_pages + 8 * held.size, "flops": 0}


def _exact_rows(q, k, v, vis, scale):
    """One head in float64: q [n][d] over k, v [m][d] where vis [n][m]."""
    sc = torch.where(vis, (q @ k.T) * scale, torch.full((), -math.inf, dtype=torch.float64, device="cuda"))
    lse = torch.logsumexp(sc, 1)
    p = torch.exp(sc - lse[:, None])
    return p, p @ v, lse


def _exact_vis(first, n, m, w, n_sink):
    i = torch.arange(first, first + n, device="cuda")[:, None]
    j = torch.arange(m, device="cuda")[None, :]
    vis = j <= i
    return vis & ((i - j < w) | (j < n_sink)) if w else vis


def exact(case, seed):
    if case["kind"] not in ("sinks", "paged"):
        return None  # copies and whole numbers
    s = prepare(case, seed)
    mult = 2 if case["paired"] else 1
    h, g, hd = case["heads"] // mult, case["kv_heads"] // mult, case["hd"]
    scale, w, n_sink = 1.0 / math.sqrt(hd), case["window"], case["sinks"]
    q = s["q"].double().view(-1, h, hd)
    o, lse = torch.zeros_like(q), torch.zeros(q.shape[0], h, dtype=torch.float64, device="cuda")
    cu = [x * mult for x in s["cu"].tolist()]
    if case["kind"] == "paged":
        kv = [x * mult for x in s["lens"].tolist()]
        for b in range(len(kv)):
            a, z = cu[b], cu[b + 1]
            pages = s["table"][b, : -(-kv[b] // (case["page"] * mult))].long()
            k, v = (s[n][pages].reshape(-1, g, hd)[: kv[b]].double() for n in ("k_pages", "v_pages"))
            vis = _exact_vis(kv[b] - (z - a), z - a, kv[b], w, n_sink)
            for x in range(h):
                _, o[a:z, x], lse[a:z, x] = _exact_rows(q[a:z, x], k[:, x * g // h], v[:, x * g // h], vis, scale)
        return dict(o=o.view(s["q"].shape), lse=lse.view(-1, case["heads"]))
    k, v = (s[n].double().view(-1, g, hd) for n in ("k", "v"))
    train = case["train"]
    if train:
        do = s["dout"].double().view(-1, h, hd)
        dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    for a, z in zip(cu[:-1], cu[1:]):
        vis = _exact_vis(0, z - a, z - a, w, n_sink)
        for x in range(h):
            y = x * g // h
            p, o[a:z, x], lse[a:z, x] = _exact_rows(q[a:z, x], k[a:z, y], v[a:z, y], vis, scale)
            if train:
                dp = do[a:z, x] @ v[a:z, y].T
                ds = p * (dp - (do[a:z, x] * o[a:z, x]).sum(1, keepdim=True))
                dq[a:z, x] = scale * (ds @ k[a:z, y])
                dk[a:z, y] += scale * (ds.T @ q[a:z, x])
                dv[a:z, y] += p.T @ do[a:z, x]
    got = dict(o=o.view(s["q"].shape), lse=lse.view(-1, case["heads"]))
    if train:
        got.update(dq=dq.view(s["q"].shape), dk=dk.view(s["k"].shape), dv=dv.view(s["v"].shape))
    return got
