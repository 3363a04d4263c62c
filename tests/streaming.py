"""Plain float64 references (numpy) of the streaming mask, the paged cache and its page management,
and the error bounds that the GPU tests hold the kernels to.

Bounds. u is half a step of the type (bf16 2^-8, f32 2^-24), e = 2^-24. For a row with weights P over
its n visible keys and A = sum_j P_j |v_j|:
* logits: a float32 dot product of hd terms, scaled: |ds| <= g = (hd + 4) e scale max_j sum_d |q_d k_jd|
  (products exact or rounded once, any order of summation);
* weights and the log-sum-exp: a relative error of at most e^g - 1 ~ g from the logits and 2^-21 from
  the exponential (base 2, two units of float32), so lse is off by at most 1.01 g + 2^-20 + n e;
* o: numerator and denominator each carry that error and their sums n e more; bf16 rounds each weight
  once (u A) and both types round the result once (u |o|):
      |do| <= (2.02 g + 2^-19 + 2 n e + [bf16] u) A + u |o|.
Splitting the keys and joining the parts adds a few e of the same terms, covered by the 2^-19.
"""
import numpy as np
import torch

U = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
E = 2.0 ** -24


def f64(t):
    return t.detach().to("cpu", torch.float64).numpy()


def visible(first, n, m, window, sinks):
    """[n][m]: queries at positions first .. first + n - 1 against key positions 0 .. m - 1."""
    i, j = np.arange(first, first + n)[:, None], np.arange(m)[None, :]
    vis = j <= i
    if window > 0:
        vis = vis & ((i - j < window) | (j < sinks))
    return vis


def attend(q, k, v, vis, scale):
    """One head: (P, o, lse, bound of o without the stored rounding, bound of lse)."""
    s = np.where(vis, q @ k.T * scale, -np.inf)
    m = s.max(1, keepdims=True)
    p = np.exp(s - m)
    l = p.sum(1, keepdims=True)
    p = p / l
    g = (q.shape[1] + 4) * E * scale * np.where(vis, np.abs(q) @ np.abs(k).T, 0).max(1)
    n = vis.sum(1)
    a = p @ np.abs(v)
    return p, p @ v, (m + np.log(l))[:, 0], (2.02 * g + 2.0 ** -19 + 2 * n * E)[:, None] * a, a, \
        1.01 * g + 2.0 ** -20 + n * E


class Reference:
    """Forward (and gradients) of packed sequences: q [T][H][hd] with rows cu; keys per sequence
    k_of(b), v_of(b) [kv][Hkv][hd] in tokens, the queries being the last ones."""

    def __init__(self, q, cu, k_of, v_of, window, sinks, paired, scale, dtype, dout=None):
        mult = 2 if paired else 1
        hd = q.shape[2]
        h = q.shape[1] // mult
        scale = scale if scale > 0 else hd ** -0.5
        u, low = U[dtype], dtype == torch.bfloat16
        Q = q.reshape(-1, h, hd)
        self.o, self.bo = np.zeros_like(Q), np.zeros_like(Q)
        self.lse, self.bl = np.zeros(Q.shape[:2]), np.zeros(Q.shape[:2])
        self.written = np.zeros(len(Q), bool)
        if dout is not None:
            g_out = dout.reshape(-1, h, hd)
            self.dq, self.bq = np.zeros_like(Q), np.zeros_like(Q)
            self.dk, self.dv, self.bk, self.bv = [], [], [], []
        for b in range(len(cu) - 1):
            a, z = int(cu[b]) * mult, int(cu[b + 1]) * mult
            if z == a:
                continue
            K = k_of(b)
            g = K.shape[1] // mult
            K, V = K.reshape(-1, g, hd), v_of(b).reshape(-1, g, hd)
            vis = visible(len(K) - (z - a), z - a, len(K), window, sinks)
            self.written[a:z] = True
            if dout is not None:
                grads = [np.zeros_like(K) for _ in range(4)]
            for x in range(h):
                y = x // (h // g)
                p, o, lse, bo, ab, bl = attend(Q[a:z, x], K[:, y], V[:, y], vis, scale)
                self.o[a:z, x], self.lse[a:z, x], self.bl[a:z, x] = o, lse, bl
                self.bo[a:z, x] = bo + (u * ab if low else 0) + u * np.abs(o)
                if dout is None:
                    continue
                go = g_out[a:z, x]
                dp = go @ V[:, y].T
                ds = p * (dp - (p * dp).sum(1, keepdims=True))
                self.dq[a:z, x] = scale * ds @ K[:, y]
                grads[0][:, y] += scale * ds.T @ Q[a:z, x]
                grads[1][:, y] += p.T @ go
                # the tensor-core backward: P, dS and O in bf16 (see test_gpu_bwd's derivation)
                d_err = 2 * u * (p * (np.abs(go) @ np.abs(V[:, y]).T)).sum(1)
                self.bq[a:z, x] = scale * (u * np.abs(ds) @ np.abs(K[:, y])
                                           + d_err[:, None] * (p @ np.abs(K[:, y])))
                grads[2][:, y] += scale * (u * np.abs(ds).T @ np.abs(Q[a:z, x])
                                           + (p * d_err[:, None]).T @ np.abs(Q[a:z, x]))
                grads[3][:, y] += u * p.T @ np.abs(go)
            if dout is not None:
                for to, x in zip((self.dk, self.dv, self.bk, self.bv), grads):
                    to.append(x)

    def check(self, o, lse, what=""):
        """o (and lse) of the kernel, NaN-filled before the call: bounds inside, untouched outside."""
        got = f64(o).reshape(self.o.shape)
        w = self.written
        assert np.isfinite(got[w]).all(), what
        over = np.abs(got - self.o)[w] - self.bo[w]
        assert (over <= 0).all(), (what, float(over.max()), np.argwhere(over > 0)[:3])
        assert np.isnan(got[~w]).all(), f"{what}: rows outside every sequence were written"
        if lse is not None:
            l = f64(lse).reshape(self.lse.shape)
            over = np.abs(l - self.lse)[w] - self.bl[w]
            assert (over <= 0).all(), (what, "lse", float(over.max()))
            assert np.isnan(l[~w]).all(), what


# ------------------------------------------------------------------------- page management (int)

class Pages:
    """A cache's bookkeeping and contents, done plainly: table [seqs][max], lens, refs, pools
    [layers][pages][page_size][width] (numpy)."""

    def __init__(self, table, lens, refs, k, v):
        self.table, self.lens, self.refs, self.k, self.v = table, lens, refs, k, v
        self.page = k.shape[2]

    def fork(self, src, dst):
        for s, d in zip(src, dst):
            self.table[d], self.lens[d] = self.table[s], self.lens[s]
            for page in self.table[s]:
                if page >= 0:
                    self.refs[page] += 1

    def reserve(self, seqs, new):
        """Number of pages taken, or None (too few: nothing changed)."""
        free = [p for p in range(len(self.refs)) if self.refs[p] == 0]
        before, plan, taken = self.refs.copy(), [], 0
        for s, n in zip(seqs, new):
            have, want = -(-self.lens[s] // self.page), -(-(self.lens[s] + n) // self.page)
            last = self.table[s, have - 1] if n > 0 and self.lens[s] % self.page else -1
            copy = last >= 0 and before[last] > 1
            need = want - have + copy
            plan.append((s, n, have - copy, free[taken:taken + need], last if copy else -1))
            taken += need
        if taken > len(free):
            return None
        old = (self.k.copy(), self.v.copy())
        for s, n, at, pages, last in plan:
            for j, p in enumerate(pages):
                self.table[s, at + j] = p
                self.refs[p] = 1
            if last >= 0:
                self.refs[last] -= 1
                self.k[:, pages[0]], self.v[:, pages[0]] = old[0][:, last], old[1][:, last]
            self.lens[s] += n
        return taken

    def free(self, seqs):
        for s in seqs:
            for page in self.table[s]:
                if page >= 0:
                    self.refs[page] -= 1
            self.table[s], self.lens[s] = -1, 0

    def trim(self, window, sinks, mult=1):
        for s in range(len(self.lens)):
            for e in range(self.table.shape[1]):
                begin, end = e * self.page * mult, (e + 1) * self.page * mult
                if self.table[s, e] >= 0 and begin >= sinks and end <= self.lens[s] * mult - window + 1:
                    self.refs[self.table[s, e]] -= 1
                    self.table[s, e] = -1

    def compact(self):
        live = int((self.refs > 0).sum())
        src = [p for p in range(live, len(self.refs)) if self.refs[p] > 0]
        dst = [p for p in range(live) if self.refs[p] <= 0]
        to = {s: d for s, d in zip(src, dst)}
        for s, d in to.items():
            self.k[:, d], self.v[:, d] = self.k[:, s], self.v[:, s]
            self.refs[d], self.refs[s] = self.refs[s], 0
        for s in range(len(self.lens)):
            for e in range(self.table.shape[1]):
                self.table[s, e] = to.get(int(self.table[s, e]), self.table[s, e])
        return len(src)
