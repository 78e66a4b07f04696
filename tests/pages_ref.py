"""Plain 64-bit implementations of the operators of long contexts (numpy), a batch to run them on, and
the error bounds of their GPU forms, for the tests.

Bounds.  Page bounds and selections are exact.  A page score is an fp32 sum of 2 D exact products and
one product with the scale: off by at most (2 D + 1) 2^-23 scale sum |q| max(|hi|, |lo|); the largest of
several heads by the largest of theirs.  Attention: step_ref.attention_row; in f16 the weights stand at
2^7 for the reference maximum, so each is off by up to 2^-32 of the row's largest besides (a
subnormal's half step): n 2^-32 max |v| over the weights' sum.
"""
import numpy as np

import step_ref as ref

SUBNORMAL = 2.0 ** -32


def visible(lens, nq):
    """(row, sequence, tokens seen) of every query."""
    row = 0
    for s, (n, m) in enumerate(zip(lens, nq)):
        for i in range(m):
            yield row, s, max(0, int(n) - int(m) + 1 + i)
            row += 1


def scores(q, hi, lo, scale):
    """q [G, D], hi and lo [n, D] in float64: (scores [n], bound [n])."""
    with np.errstate(invalid="ignore"):
        x = np.maximum(q[:, None] * hi, q[:, None] * lo).sum(-1) * scale  # [G, n]
        size = (np.abs(q[:, None]) * np.maximum(np.abs(hi), np.abs(lo))).sum(-1) * abs(scale)
    return x.max(0), (2 * q.shape[1] + 1) * 2.0 ** -23 * size.max(0)


def select(x, n, sinks, recent, k):
    """The list of one row: x [n] scores."""
    if n <= k:
        return list(range(n)) + [-1] * (k - n)
    mid = range(sinks, n - recent)
    key = [(-np.inf if np.isnan(x[j]) else -x[j] if not np.isposinf(x[j]) else -np.finfo(np.float64).max, j)
           for j in mid]
    best = sorted(key)[:k - sinks - recent]
    return sorted(list(range(sinks)) + [j for _, j in best] + list(range(n - recent, n)))


def attention(q, k, v, scale, dtype):
    """One (row, head): q [D], k and v [n, D] of the tokens it reads: (o, bound)."""
    o, tol = ref.attention_row(q, k, v, scale, dtype)
    if dtype == "f16" and len(k):
        x = k @ q * scale
        tol = tol + len(k) * SUBNORMAL * np.abs(v).max(0) / np.exp(x - x.max()).sum()
    return o, tol


class Batch:
    """Sequences over shuffled pages, everything that no token fills NaN.  groups: (sequences,
    prefix) pairs of hp_attention_prefix; the pages that lie whole inside a prefix are shared, and the
    slots of a prefix's last part page in the other sequences' pages hold NaN too."""

    def __init__(self, hp, lens, H, G, D, P, dtype="bf16", nq=None, it=0, seed=0, groups=None, behind=0, flags=0,
                 host=False, k_scale=1.0):
        import torch
        rng = np.random.default_rng(seed)
        self.rng, self.hp = rng, hp
        self.lens, self.H, self.G, self.D, self.P, self.dtype = np.array(lens, np.int64), H, G, D, P, dtype
        S = len(lens)
        self.nq = np.ones(S, np.int64) if nq is None else np.array(nq, np.int64)
        self.T, self.behind = int(self.nq.sum()) + behind, behind
        self.it, dt = it, ref.torch_dtype(dtype)
        self.dt = dt
        need = -(-self.lens // P)
        self.groups = groups
        first = np.concatenate([[0], np.cumsum([g for g, _ in groups])]).astype(np.int64) if groups else None
        self.first = first
        total, shared = int(need.sum()), []
        self.pages = total + 3
        perm = rng.permutation(self.pages)
        self.ptr = np.concatenate([[0], np.cumsum(need)]).astype(np.int64)
        self.table = perm[:total].astype(np.int64)
        self.prefix = np.zeros(S, np.int64)
        self.lead = np.arange(S)
        if groups:
            for g, (n, pre) in enumerate(groups):
                for s in range(first[g], first[g + 1]):
                    self.prefix[s], self.lead[s] = pre, first[g]
                    w = pre // P
                    self.table[self.ptr[s]:self.ptr[s] + w] = self.table[self.ptr[first[g]]:self.ptr[first[g]] + w]
        gen = torch.Generator().manual_seed(seed)
        k = (torch.randn((self.pages, P, H, D), generator=gen) * k_scale).to(dt)
        v = torch.randn((self.pages, P, H, D), generator=gen).to(dt)
        live = torch.zeros((self.pages, P), dtype=torch.bool)
        for s in range(S):
            a = self.prefix[s] if self.lead[s] != s else 0
            t = np.arange(a, self.lens[s])
            pg = self.table[self.ptr[s] + t // P]
            live[torch.from_numpy(pg), torch.from_numpy(t % P)] = True
        k[~live], v[~live] = float("nan"), float("nan")
        self.hk, self.hv = k, v
        where = (lambda x: x.pin_memory()) if host else (lambda x: x.cuda())
        self.k, self.v = where(k), where(v)
        tt = torch.int64 if it else torch.int32
        self.tt = tt
        dev = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda().to(tt)  # noqa: E731
        self.dev = dev
        self.d_table, self.d_ptr, self.d_lens = dev(self.table), dev(self.ptr), dev(self.lens)
        self.d_q_ptr = dev(np.concatenate([[0], np.cumsum(self.nq)]))
        if groups:
            self.d_group = dev(first)
            self.d_prefix = dev([p for _, p in groups])
        self.flags = flags | (hp.HOST_MEMORY if host else 0)
        self.desc = self.describe()
        self.hq = torch.randn((self.T, H * G, D), generator=gen).to(dt)
        self.q = self.hq.cuda()
        self.out = torch.full((self.T, H * G, D), 7.0, dtype=dt, device="cuda")
        self.status = torch.full((1,), 99, dtype=torch.int32, device="cuda")
        self.scale = 1.0 / D ** 0.5

    def describe(self, pool=None, **kw):
        f = dict(num_pages=self.pages, page_size=self.P, num_heads=self.H, head_dim=self.D, dtype=self.dtype,
                 index_type=self.it, flags=self.flags)
        f.update(kw)
        return self.hp.PagedDesc(self.k if pool is None else pool, self.d_table, self.d_ptr, self.d_lens, **f)

    def offsets(self):
        """q_ptr, or None where a query a sequence needs none."""
        return None if self.behind == 0 and (self.nq == 1).all() else self.d_q_ptr

    def code(self):
        c = int(self.status.item())
        return self.hp.status_name(c)

    def token_rows(self, s, t):
        """K and V (float64, [len(t), H, D]) of tokens t of sequence s, a shared prefix through the
        slice of its group's first sequence."""
        own = np.where(t < self.prefix[s], self.lead[s], s)
        pg = self.table[self.ptr[own] + t // self.P]
        return (self.hk[pg, t % self.P].double().numpy(), self.hv[pg, t % self.P].double().numpy())

    def check(self, tokens, rows=None, out=None):
        """out against 64 bits; tokens(row, seq, seen, head) gives the tokens that (row, head) reads."""
        got = (self.out if out is None else out).double().cpu().numpy()
        q = self.hq.double().numpy()
        worst = 0.0
        for row, s, seen in visible(self.lens, self.nq):
            if rows is not None and row not in rows:
                continue
            cache = {}
            for h in range(self.H):
                t = np.asarray(tokens(row, s, seen, h), np.int64)
                key = t.tobytes()
                if key not in cache:
                    cache[key] = self.token_rows(s, t)
                k, v = cache[key]
                for g in range(self.G):
                    o, tol = attention(q[row, h * self.G + g], k[:, h], v[:, h], self.scale, self.dtype)
                    err = np.abs(got[row, h * self.G + g] - o)
                    assert (err <= tol).all(), (row, s, seen, h, g, float(np.nanmax(err / tol)), got[row, h * self.G + g][:4], o[:4])
                    worst = max(worst, float((err / np.maximum(tol, 1e-30)).max()))
        if self.behind:
            assert (got[self.T - self.behind:] == 7.0).all()
        return worst
