"""The operators of long contexts over a paged K/V cache, as they are measured: cases, inputs,
the plain form of each operator in elementary torch operations, the library's calls, and a
64-bit evaluation of each definition.

Five operators.  The first four make a decode step over long sequences read only the pages that
matter to its queries; the fifth reads a prefix that sequences share once for all of them:

  bounds   hp_page_bounds: per page and K/V head the largest and the smallest key in each
           dimension, kept up to date as tokens are appended.
  scores   hp_page_scores: for each query and K/V head an upper bound of the scores that its
           tokens can reach, page by page, from those bounds.
  select   hp_select_pages: the pages with the highest bounds (whole numbers; ties to the lowest
           page), the first and the last pages always among them, in ascending order.
  pages    hp_attention_pages: attention over the selected pages.
  prefix   hp_attention_prefix: attention of groups of sequences that share their first tokens.
"""
import math

import numpy as np
import torch

own = False

TORCH = {"bf16": torch.bfloat16, "f16": torch.float16}


# ------------------------------------------------------------------------------- cases
def listed():
    return [
        # a decode step of 64 sequences, a token each: the page that the token fell into
        dict(name="bounds_decode_64", op="bounds", seqs=64, lo=500, hi=2048, new_lo=1, new_hi=1,
             page=16, hkv=8, dim=128, dtype="bf16", shape=1),
        # eleven prompts, each behind a cached beginning, odd lengths
        dict(name="bounds_prompts_11", op="bounds", seqs=11, lo=0, hi=900, new_lo=1, new_hi=7001,
             page=64, hkv=4, dim=128, dtype="f16", shape=2),
        # one sequence of 8,000 tokens; latency counts
        dict(name="scores_decode_1", op="scores", seqs=1, lo=8001, hi=8001, nq=1, page=16, hkv=8,
             group=4, dim=128, dtype="bf16", shape=3),
        # a batch of long contexts, 131,072 tokens at most, some short
        dict(name="scores_decode_64_long", op="scores", seqs=64, lo=100, hi=131072, nq=1, page=16,
             hkv=8, group=4, dim=128, dtype="bf16", shape=4),
        # two queries a sequence (one drafted), 64 dims, pages of 32
        dict(name="scores_drafted_20", op="scores", seqs=20, lo=0, hi=30011, nq=2, page=32, hkv=4,
             group=8, dim=64, dtype="f16", shape=5),
        # the selection behind scores_decode_1
        dict(name="select_decode_1", op="select", rows=1, lo=501, hi=501, hkv=8, keep=64, sinks=1,
             recent=2, page=16, shape=6),
        # the selection of a large batch of long contexts, coarse scores (many ties)
        dict(name="select_decode_256", op="select", rows=256, lo=0, hi=8192, hkv=8, keep=256,
             sinks=2, recent=4, page=16, shape=7),
        # one sequence, 64 of its 500 pages: latency counts
        dict(name="pages_decode_1", op="pages", seqs=1, lo=8001, hi=8001, nq=1, keep=64, page=16,
             hkv=8, group=4, dim=128, dtype="bf16", shape=8),
        # an ordinary batch, 2,048 tokens of each sequence, some sequences shorter than that
        dict(name="pages_decode_64", op="pages", seqs=64, lo=0, hi=16000, nq=1, keep=128, page=16,
             hkv=8, group=4, dim=128, dtype="bf16", shape=9),
        # eight requests with one system prompt of 1,000 tokens, a few tokens of their own
        dict(name="prefix_decode_8", op="prefix", seqs=8, groups=1, pre_lo=1000, pre_hi=1000,
             lo=0, hi=90, nq=1, page=16, hkv=8, group=4, dim=128, dtype="bf16", shape=10),
        # 128 sequences behind a system prompt of 2,048 tokens, 64 to 1,024 tokens of their own
        dict(name="prefix_decode_128", op="prefix", seqs=128, groups=1, pre_lo=2048, pre_hi=2048,
             lo=64, hi=1024, nq=1, page=16, hkv=8, group=4, dim=128, dtype="bf16", shape=11),
        # three long documents and 250 questions about them, odd lengths
        dict(name="prefix_documents_250", op="prefix", seqs=250, groups=3, pre_lo=20000,
             pre_hi=40000, lo=0, hi=333, nq=1, page=16, hkv=8, group=8, dim=128, dtype="f16",
             shape=12),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.4)))))


def draw(rng):
    op = rng.choice(["bounds", "scores", "select", "pages", "pages", "prefix", "prefix"])
    shape = rng.randrange(1 << 30)
    dtype = rng.choice(["bf16", "f16"])
    page = rng.choice([8, 16, 32, 64])
    hkv = rng.choice([1, 2, 4, 8])
    if op == "bounds":
        prompts = rng.random() < 0.5
        return dict(op=op, seqs=_log_int(rng, 1, 12 if prompts else 256), lo=0,
                    hi=_log_int(rng, 1, 2048), new_lo=1 if prompts else rng.choice([0, 1]),
                    new_hi=_log_int(rng, 2, 7000) if prompts else 1, page=page, hkv=hkv,
                    dim=rng.choice([64, 128, 256]), dtype=dtype, shape=shape)
    if op == "scores":
        seqs = _log_int(rng, 1, 64)
        return dict(op=op, seqs=seqs, lo=0, hi=_log_int(rng, 64, min(131072, 131072 * 16 // seqs)),
                    nq=rng.choice([1, 1, 1, 2, 3]), page=page, hkv=hkv,
                    group=rng.choice([1, 2, 3, 4, 8]), dim=rng.choice([64, 128]), dtype=dtype,
                    shape=shape)
    if op == "select":
        keep = _log_int(rng, 8, 512)
        return dict(op=op, rows=_log_int(rng, 1, 256), lo=0, hi=_log_int(rng, 2 * keep, 8192),
                    hkv=hkv, keep=keep, sinks=rng.randrange(0, 4), recent=rng.randrange(0, 5),
                    page=page, shape=shape)
    if op == "pages":
        seqs = _log_int(rng, 1, 64)
        return dict(op=op, seqs=seqs, lo=0, hi=_log_int(rng, 16, 16000),
                    nq=rng.choice([1, 1, 1, 2, 3]), keep=_log_int(rng, 1, 2048 // page),
                    page=page, hkv=hkv, group=rng.choice([1, 2, 4, 5, 8]),
                    dim=rng.choice([64, 128, 256]), dtype=dtype, shape=shape)
    seqs = _log_int(rng, 1, 256)
    pre = _log_int(rng, 16, 30000)
    return dict(op=op, seqs=seqs, groups=min(seqs, rng.choice([1, 1, 2, 3, 7])),
                pre_lo=rng.choice([pre, pre // 3]), pre_hi=pre, lo=0, hi=_log_int(rng, 4, 1024),
                nq=rng.choice([1, 1, 1, 2]) if seqs <= 128 else 1, page=page, hkv=hkv,
                group=rng.choice([1, 2, 4, 8]), dim=rng.choice([64, 128, 128]), dtype=dtype,
                shape=shape)


def _np(case):
    return np.random.default_rng(case["shape"])


def _few(case, lens):
    """Where lengths start at zero, an empty and a one-token sequence are among them; the first
    one is the longest."""
    lens[0] = case["hi"]
    if case["lo"] == 0 and len(lens) > 4:
        lens[1], lens[2] = 0, 1
    return lens


def _shape(case):
    """Lengths and query counts (bounds: new tokens) of the sequences."""
    r, n = _np(case), case["seqs"]
    if case["op"] == "bounds":
        new = r.integers(case["new_lo"], case["new_hi"] + 1, n)
        return r.integers(case["lo"], case["hi"] + 1, n) + new, new
    lens = _few(case, r.integers(case["lo"], case["hi"] + 1, n))
    return lens, np.full(n, case["nq"])


def _select_shape(case):
    r = _np(case)
    return _few(case, r.integers(case["lo"], case["hi"] + 1, case["rows"]))


def _prefix_shape(case):
    """(first sequence of each group and the end, prefix of each group, length of each sequence)"""
    r, S, g = _np(case), case["seqs"], case["groups"]
    first = np.concatenate([[0], np.sort(r.choice(np.arange(1, S), g - 1, replace=False)), [S]])
    pre = r.integers(case["pre_lo"], case["pre_hi"] + 1, g)
    tail = r.integers(case["lo"], case["hi"] + 1, S)
    if S > 4 and case["lo"] == 0:
        tail[1], tail[2] = 0, 1  # one that adds nothing yet, one with a token of its own
    tail = np.maximum(tail, case["nq"] - 1)  # every query sees the whole prefix
    return first.astype(np.int64), pre, np.repeat(pre, np.diff(first)) + tail


def _visible(lens, nq):
    """Tokens each query sees: the n queries of a sequence are its last n tokens."""
    return np.concatenate([np.maximum(0, l - n + 1 + np.arange(n)) for l, n in zip(lens, nq)])


def work(case):
    """Bytes and operations one pass cannot do without."""
    op = case["op"]
    if op == "select":
        n, H = _select_shape(case), case["hkv"]
        return {"bytes": 4 * H * (int(n.sum()) + len(n) * case["keep"]) + 4 * len(n),
                "flops": H * int(n.sum())}
    H, D, P = case["hkv"], case["dim"], case["page"]
    if op == "bounds":
        lens, new = _shape(case)
        first = (lens - new) // P * P
        rows = int((lens - first)[new > 0].sum())
        pages = int((-(-lens // P) - first // P)[new > 0].sum())
        return {"bytes": 2 * H * D * (rows + 2 * pages) + 4 * pages + 12 * len(lens),
                "flops": 2 * rows * H * D}
    G = case["group"]
    if op == "scores":
        lens, nq = _shape(case)
        T, pages = int(nq.sum()), int((-(-lens // P)).sum())
        rows = int((-(-_visible(lens, nq) // P)).sum())
        return {"bytes": pages * (H * 2 * D * 2 + 4) + T * H * G * D * 2 + 4 * rows * H,
                "flops": 4 * rows * H * G * D}
    if op == "pages":
        lens, nq = _shape(case)
        # (drafted queries keep seven eighths of the pages of the query before them)
        took = np.minimum(lens, case["keep"] * P)
        share = 1 + (case["nq"] - 1) / 8
        T, tokens = int(nq.sum()), int((took * share).sum())
        return {"bytes": H * tokens * D * 2 * 2 + T * H * case["keep"] * 4 + 2 * T * H * G * D * 2,
                "flops": 4 * int((took * nq).sum()) * H * G * D}
    first, pre, lens = _prefix_shape(case)
    tail = int((lens - np.repeat(pre, np.diff(first))).sum())
    T = case["seqs"] * case["nq"]
    seen = int(_visible(lens, np.full(len(lens), case["nq"])).sum())
    return {"bytes": (int(pre.sum()) + tail) * H * D * 4 + 2 * T * H * G * D * 2,
            "flops": 4 * seen * H * G * D}


# ------------------------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _randn(g, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def _dev(a, dtype=torch.int32):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda().to(dtype)


def _ptr(n):
    return np.concatenate([[0], np.cumsum(n)])


def _tables(g, need):
    """Shuffled pages of sequences that take need[s] each: (table, seq_ptr, pages in the pool)."""
    total = int(need.sum())
    table = torch.randperm(total + 3, generator=g, device="cuda")[:total].to(torch.int32)
    return table, _ptr(need), total + 3


def _pool(g, pages, page, hkv, dim, dtype, live):
    """Rows in the slots that `live` names; what lies in the others is not a number."""
    pool = _randn(g, (pages, page, hkv, dim), dtype)
    pool.view(pages * page, -1)[~live] = float("nan")
    return pool


def _live(table, ptr, lens, pages, page):
    """Which slots of the pool hold a token."""
    live = torch.zeros(pages * page, dtype=torch.bool, device="cuda")
    at = _dev(np.repeat(ptr[:-1], lens), torch.int64)
    t = _dev(np.concatenate([np.arange(n) for n in lens] + [np.zeros(0, np.int64)]), torch.int64)
    live[table.long()[at + t // page] * page + t % page] = True
    return live


def _inputs(case, seed):
    g, op = _gen(seed), case["op"]
    s = dict(case)
    H, P = case["hkv"], case["page"]
    if op == "select":
        n = _select_shape(case)
        s["host_n"], s["max_pages"] = n, max(1, int(n.max()))
        s["host_lens"] = np.maximum(n * P - n % P, 0) if P > 1 else n  # pages that end inside
        s["host_q"] = np.ones(len(n), np.int64)
        # as the scores of one layer spread; 16 bits of them, so that equal ones are common
        s["scores"] = _randn(g, (len(n), H, s["max_pages"]), torch.bfloat16, 8.0).float()
        s["lens"], s["seq_ptr"] = _dev(s["host_lens"]), _dev(_ptr(n))
        return s
    D, dt = case["dim"], TORCH[case["dtype"]]
    s["dt"] = dt
    if op == "prefix":
        return _prefix_inputs(s, case, g)
    lens, nq = _shape(case)
    s["host_lens"], s["host_q"] = lens, nq
    table, ptr, pages = _tables(g, -(-lens // P))
    s.update(table=table, host_ptr=ptr, pages=pages, lens=_dev(lens), seq_ptr=_dev(ptr),
             q_ptr=_dev(_ptr(nq)))
    if op == "scores":
        # bounds of 16 to 64 keys of unit spread: about two from the middle each way
        mid = _randn(g, (pages, H, D), torch.float32, 0.4)
        s["bounds"] = torch.stack([mid + 1.7, mid - 1.7], 2).to(dt)
        s["max_pages"] = max(1, int((-(-lens // P)).max()))
    else:
        live = _live(table, ptr, lens, pages, P)
        s["k_pool"] = _pool(g, pages, P, H, D, dt, live)
    if op == "bounds":
        s["bounds"] = _randn(g, (pages, H, 2, D), dt)
        return s
    T, Hq = int(nq.sum()), H * case["group"]
    s["scale"] = 1.0 / math.sqrt(D)
    s["q"] = _randn(g, (T, Hq, D), dt)
    if op == "pages":
        s["v_pool"] = _pool(g, pages, P, H, D, dt, live)
        s["selected"] = _lists(g, lens, case)
    return s


def _lists(g, lens, case):
    """Ascending page lists of each query and K/V head: the first and the last page, the others
    at random; a drafted query changes an eighth of the list of the query before it."""
    H, k, P, nq = case["hkv"], case["keep"], case["page"], case["nq"]
    n = _dev(-(-lens // P), torch.int64)
    most = max(1, int((-(-lens // P)).max()))
    out = torch.full((len(lens), nq, H, k), -1, dtype=torch.int32, device="cuda")
    j = torch.arange(most, device="cuda")
    key = torch.rand((len(lens), H, most), generator=g, device="cuda")
    for i in range(nq):
        if i:
            other = torch.rand(key.shape, generator=g, device="cuda")
            key = torch.where(torch.rand(key.shape, generator=g, device="cuda") < 0.125, other, key)
        x = torch.where((j == 0) | (j == n[:, None, None] - 1), 2.0, key)
        x = torch.where(j < n[:, None, None], x, -1.0)
        top = x.topk(min(k, most), dim=-1)
        page = torch.where(top.values >= 0, top.indices, most).sort(-1).values
        out[:, i, :, :page.shape[-1]] = torch.where(page < most, page, -1).to(torch.int32)
    return out.view(-1, H, k)


def _prefix_inputs(s, case, g):
    H, D, P, dt = case["hkv"], case["dim"], case["page"], s["dt"]
    first, pre, lens = _prefix_shape(case)
    S, nq = case["seqs"], case["nq"]
    grp = np.repeat(np.arange(case["groups"]), np.diff(first))
    whole = pre[grp] // P                      # pages that a group's sequences share
    need = -(-lens // P)
    own_pages = need - whole                   # from the page in which the prefix ends
    shared = pre // P
    perm = np.random.default_rng([case["shape"], 1]).permutation(int(own_pages.sum() + shared.sum()) + 3)
    pages, at = len(perm), 0
    shares, parts = [], []
    for n in shared:
        shares.append(perm[at:at + n])
        at += n
    for q in range(S):
        parts.append(np.concatenate([shares[grp[q]], perm[at:at + own_pages[q]]]))
        at += own_pages[q]
    ptr = _ptr(need)
    table = _dev(np.concatenate(parts))
    live = _live(table, ptr, lens, pages, P)
    s.update(host_first=first, host_pre=pre, host_lens=lens, host_ptr=ptr, host_q=np.full(S, nq),
             pages=pages, table=table, seq_ptr=_dev(ptr), lens=_dev(lens), group_ptr=_dev(first),
             prefix_lens=_dev(pre), q_ptr=_dev(_ptr(np.full(S, nq))), scale=1.0 / math.sqrt(D))
    for name in ("k_pool", "v_pool"):
        s[name] = _pool(g, pages, P, H, D, dt, live)
    # where a prefix ends inside a page every sequence holds a copy of that page's beginning
    host = np.concatenate(parts)
    src, dst = [], []
    for q in range(S):
        a, rest = ptr[first[grp[q]]] + whole[q], pre[grp[q]] % P
        b = ptr[q] + whole[q]
        if rest and a != b:
            src.append(host[a] * P + np.arange(rest))
            dst.append(host[b] * P + np.arange(rest))
    if src:
        src, dst = _dev(np.concatenate(src), torch.int64), _dev(np.concatenate(dst), torch.int64)
        for name in ("k_pool", "v_pool"):
            flat = s[name].view(pages * P, -1)
            flat[dst] = flat[src]
    s["q"] = _randn(g, (S * nq, H * case["group"], D), dt)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    op = s["op"]
    if op == "scores":
        s["scores"] = torch.zeros((s["q"].shape[0], s["hkv"], s["max_pages"]), device="cuda")
    elif op == "select":
        s["selected"] = torch.zeros((s["rows"], s["hkv"], s["keep"]), dtype=torch.int32,
                                    device="cuda")
    elif op in ("pages", "prefix"):
        s["out"] = torch.zeros_like(s["q"])
    if own:
        _prepare_own(s)
    return s


def _prepare_own(s):
    """The descriptors and workspaces a user's program keeps between steps."""
    from paged_kv_cache_hp_gb300 import hp
    op = s["op"]
    s["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    one = "nq" not in s or s["nq"] == 1  # a query (a new token) a sequence needs no offsets
    s["q_off"] = None if one else s["q_ptr"]
    if op == "select":  # reads the lengths alone
        s["desc"] = hp.PagedDesc(None, None, s["seq_ptr"], s["lens"], num_pages=0,
                                 page_size=s["page"], num_heads=s["hkv"], head_dim=128,
                                 dtype="bf16", index_type=hp.IDX_U32, table_len=0)
        return
    pool = s["bounds"] if op == "scores" else s["k_pool"]
    s["desc"] = hp.PagedDesc(pool, s["table"], s["seq_ptr"], s["lens"], num_pages=s["pages"],
                             page_size=s["page"], num_heads=s["hkv"], head_dim=s["dim"],
                             dtype=s["dtype"], index_type=hp.IDX_U32)
    if op == "bounds":
        s["new_off"] = None if (s["host_q"] == 1).all() else s["q_ptr"]
        s["total_new"] = int(s["host_q"].sum())
    elif op == "prefix":
        T, Hq = s["q"].shape[:2]
        rc, n = hp.hp_attention_prefix_workspace_bytes(s["desc"], s["groups"], T, Hq)
        assert rc == 0, hp.status_name(rc)
        s["ws"] = torch.empty(n, dtype=torch.uint8, device="cuda")


# --------------------------------------------------------------------------- one pass
def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    from paged_kv_cache_hp_gb300 import hp
    op = s["op"]
    if op == "bounds":
        hp.hp_page_bounds(s["desc"], s["new_off"], s["total_new"], s["bounds"], s["status"])
        return s["bounds"]
    if op == "select":
        hp.hp_select_pages(s["desc"], s["q_off"], s["rows"], s["scores"], s["max_pages"],
                           s["sinks"], s["recent"], s["keep"], s["selected"], s["status"])
        return s["selected"]
    T, Hq = s["q"].shape[:2]
    if op == "scores":
        hp.hp_page_scores(s["desc"], s["bounds"], s["q"], s["q_off"], T, Hq, s["scale"],
                          s["scores"], s["max_pages"], s["status"])
        return s["scores"]
    if op == "pages":
        hp.hp_attention_pages(s["desc"], s["v_pool"], s["q"], s["q_off"], T, Hq, s["scale"],
                              s["selected"], s["keep"], s["out"], s["status"])
        return s["out"]
    hp.hp_attention_prefix(s["desc"], s["v_pool"], s["group_ptr"], s["prefix_lens"], s["groups"],
                           s["q"], s["q_off"], T, Hq, s["scale"], s["out"], s["ws"], s["status"])
    return s["out"]


def _run_plain(s):
    return {"bounds": _plain_bounds, "scores": _plain_scores, "select": _plain_select,
            "pages": _plain_pages, "prefix": _plain_prefix}[s["op"]](s)


def _plain_bounds(s):
    P, H, D = s["page"], s["hkv"], s["dim"]
    slot = torch.arange(P, device="cuda")
    for q, (n, new) in enumerate(zip(s["host_lens"].tolist(), s["host_q"].tolist())):
        if not new:
            continue
        a, b = (n - new) // P, -(-n // P)
        page = s["table"][int(s["host_ptr"][q]) + a:int(s["host_ptr"][q]) + b].long()
        rows = s["k_pool"][page].float()                       # [pages, P, H, D]
        seen = (torch.arange(a, b, device="cuda")[:, None] * P + slot < n)[..., None, None]
        hi = rows.masked_fill(~seen, float("-inf")).amax(1)
        lo = rows.masked_fill(~seen, float("inf")).amin(1)
        s["bounds"][page] = torch.stack([hi, lo], 2).to(s["dt"])
    return s["bounds"]


def _queries(s):
    """(row of q, sequence, tokens it sees) of every query."""
    row = 0
    for q, (n, m) in enumerate(zip(s["host_lens"].tolist(), s["host_q"].tolist())):
        for i in range(m):
            yield row, q, max(0, n - m + 1 + i)
            row += 1


def _plain_scores(s):
    H, G, D, P = s["hkv"], s["group"], s["dim"], s["page"]
    for row, q, seen in _queries(s):
        n = -(-seen // P)
        if not n:
            continue
        first = int(s["host_ptr"][q])
        b = s["bounds"][s["table"][first:first + n].long()].float()  # [n, H, 2, D]
        x = s["q"][row].float().view(H, G, D)
        up = torch.einsum("hgd,nhd->hgn", x.clamp(min=0), b[:, :, 0]) + \
            torch.einsum("hgd,nhd->hgn", x.clamp(max=0), b[:, :, 1])
        s["scores"][row, :, :n] = up.amax(1) * s["scale"]
    return s["scores"]


def _plain_select(s):
    k, most = s["keep"], s["max_pages"]
    n = _dev(s["host_n"], torch.int64)[:, None, None]
    j = torch.arange(most, device="cuda")
    forced = (j < n) & ((j < s["sinks"]) | (j >= n - s["recent"]))
    middle = (j < n) & ~forced
    order = torch.sort(s["scores"], dim=-1, descending=True, stable=True).indices
    ranked = torch.gather(middle.expand(order.shape), 2, order)
    take = ranked & (ranked.cumsum(-1) <= k - forced.sum(-1, keepdim=True))
    chosen = torch.zeros_like(take).scatter(2, order, take) | forced
    at = torch.where(chosen, chosen.cumsum(-1) - 1, k)
    out = torch.full(chosen.shape[:2] + (k + 1,), -1, dtype=torch.int64, device="cuda")
    out.scatter_(2, at, j.expand(at.shape).contiguous())
    s["selected"].copy_(out[:, :, :k])
    return s["selected"]


def _softmax(x):
    e = torch.exp(x - x.amax(-1, keepdim=True))
    return e / e.sum(-1, keepdim=True)


def _plain_pages(s):
    H, G, D, P = s["hkv"], s["group"], s["dim"], s["page"]
    heads = torch.arange(H, device="cuda")[:, None, None]
    slot = torch.arange(P, device="cuda")
    for row, q, seen in _queries(s):
        if not seen:
            s["out"][row] = 0
            continue
        sel = s["selected"][row].long()                              # [H, k]
        t = sel[:, :, None] * P + slot                               # [H, k, P]
        hide = ((sel < 0)[:, :, None] | (t >= seen)).reshape(H, 1, -1)
        page = s["table"][int(s["host_ptr"][q]) + sel.clamp(min=0)].long()[:, :, None]
        k = s["k_pool"][page, slot, heads].float().reshape(H, -1, D)
        v = s["v_pool"][page, slot, heads].float().reshape(H, -1, D)
        v = v.masked_fill(hide.reshape(H, -1, 1), 0)
        x = s["q"][row].float().view(H, G, D) @ k.transpose(1, 2) * s["scale"]
        x = x.masked_fill(hide, float("-inf"))
        s["out"][row] = (_softmax(x) @ v).reshape(H * G, D).to(s["dt"])
    return s["out"]


def _token_rows(s, pool, q, a, b):
    """Tokens a .. b - 1 of sequence q, 32 bits, [tokens, H, D]."""
    P = s["page"]
    first = int(s["host_ptr"][q])
    page = s["table"][first + a // P:first + -(-b // P)].long()
    return s[pool][page].flatten(0, 1)[a % P:a % P + b - a].float()


def _plain_prefix(s):
    H, G, D, nq = s["hkv"], s["group"], s["dim"], s["nq"]
    for g, pre in enumerate(s["host_pre"].tolist()):
        a, b = int(s["host_first"][g]), int(s["host_first"][g + 1])
        k, v = (_token_rows(s, p, a, 0, pre).transpose(0, 1) for p in ("k_pool", "v_pool"))
        x = s["q"][a * nq:b * nq].float().view(-1, H, G, D) * s["scale"]
        head = torch.einsum("rhgd,htd->rhgt", x, k)
        top = head.amax(-1, keepdim=True)
        e = torch.exp(head - top)
        total, acc = e.sum(-1, keepdim=True), torch.einsum("rhgt,htd->rhgd", e, v)
        for q in range(a, b):
            r = slice((q - a) * nq, (q - a + 1) * nq)
            n = int(s["host_lens"][q])
            t, l, o = top[r], total[r], acc[r]
            if n > pre:  # the sequence's own tokens
                kt, vt = (_token_rows(s, p, q, pre, n) for p in ("k_pool", "v_pool"))
                y = torch.einsum("rhgd,thd->rhgt", x[r], kt)
                last = n - nq + torch.arange(nq, device="cuda")
                y = y.masked_fill((torch.arange(pre, n, device="cuda") > last[:, None])[:, None, None],
                                  float("-inf"))
                m = torch.maximum(t, y.amax(-1, keepdim=True))
                f, w = torch.exp(t - m), torch.exp(y - m)
                l = l * f + w.sum(-1, keepdim=True)
                o = o * f + torch.einsum("rhgt,thd->rhgd", w, vt)
            s["out"][q * nq:(q + 1) * nq] = (o / l).reshape(nq, H * G, D).to(s["dt"])
    return s["out"]


# --------------------------------------------------------------------- 64-bit definition
def exact(case, seed):
    if case["op"] == "select":
        return None  # whole numbers, which the plain form gives as they are
    s = _inputs(case, seed)
    return {"bounds": _exact_bounds, "scores": _exact_scores, "pages": _exact_attention,
            "prefix": _exact_attention}[s["op"]](s)


def _exact_bounds(s):
    """Token by token: every new page's bounds are met by each of its tokens in turn."""
    P = s["page"]
    out = s["bounds"].double()
    page, offs, fresh = [], [], []
    for q, (n, new) in enumerate(zip(s["host_lens"].tolist(), s["host_q"].tolist())):
        if new:
            t = np.arange((n - new) // P * P, n)
            page.append(s["host_ptr"][q] + t // P)
            offs.append(t % P)
    if not page:
        return out
    page, offs = s["table"].long()[_dev(np.concatenate(page), torch.int64)], np.concatenate(offs)
    for i in range(P):
        here = _dev(np.flatnonzero(offs == i), torch.int64)
        p = page[here]
        row = s["k_pool"][p, i].double()
        if i == 0:
            out[p, :, 0], out[p, :, 1] = row, row
        else:
            out[p, :, 0] = torch.maximum(out[p, :, 0], row)
            out[p, :, 1] = torch.minimum(out[p, :, 1], row)
    return out


def _exact_scores(s):
    """The largest product with either bound, dimension by dimension."""
    H, G, D, P = s["hkv"], s["group"], s["dim"], s["page"]
    out = torch.zeros((s["q"].shape[0], H, s["max_pages"]), dtype=torch.float64, device="cuda")
    for row, q, seen in _queries(s):
        n = -(-seen // P)
        ids = s["table"].long()[int(s["host_ptr"][q]):int(s["host_ptr"][q]) + n]
        x = s["q"][row].double().view(H, G, D)
        for a in range(0, n, 2048):  # (in pieces that fit the memory)
            b = s["bounds"][ids[a:a + 2048]].double()
            best = None
            for g in range(G):
                up = torch.maximum(x[:, g] * b[:, :, 0], x[:, g] * b[:, :, 1]).sum(-1) * s["scale"]
                best = up if best is None else torch.maximum(best, up)
            out[row, :, a:a + len(best)] = best.t()
    return out


def _exact_attention(s):
    """softmax(scale q . k) v over the tokens each query reads, head by head."""
    H, G, D, P = s["hkv"], s["group"], s["dim"], s["page"]
    T = s["q"].shape[0]
    out = torch.zeros((T, H * G, D), dtype=torch.float64, device="cuda")
    table, ptr = s["table"].cpu().numpy().astype(np.int64), s["host_ptr"]
    kf, vf = (s[n].view(-1, H, D) for n in ("k_pool", "v_pool"))
    lists = s["selected"].cpu().numpy() if s["op"] == "pages" else None

    def rows(q, t, h):
        at = _dev(table[ptr[q] + t // P] * P + t % P, torch.int64)
        return kf[at, h].double(), vf[at, h].double()

    def weigh(x, k, v):
        y = x @ k.t() * s["scale"]
        m = y.amax(-1, keepdim=True)
        e = torch.exp(y - m)
        return m, e.sum(-1, keepdim=True), e @ v

    if lists is not None:
        for row, q, seen in _queries(s):
            for h in range(H):
                j = lists[row, h]
                t = (j[j >= 0][:, None] * P + np.arange(P)).ravel()
                t = t[t < seen]
                if len(t):
                    k, v = rows(q, t, h)
                    _, l, o = weigh(s["q"][row, h * G:(h + 1) * G].double(), k, v)
                    out[row, h * G:(h + 1) * G] = o / l
        return out
    info = list(_queries(s))
    for g, pre in enumerate(s["host_pre"].tolist()):
        a, b = int(s["host_first"][g]), int(s["host_first"][g + 1])
        mine = [x for x in info if a <= x[1] < b]
        r0, r1 = mine[0][0], mine[-1][0] + 1
        for h in range(H):
            k, v = rows(a, np.arange(pre), h)
            x = s["q"][r0:r1, h * G:(h + 1) * G].double()
            step = max(1, 50_000_000 // (pre * G))
            parts = [weigh(x[i:i + step], k, v) for i in range(0, r1 - r0, step)]
            m, l, o = (torch.cat(p) for p in zip(*parts))
            for row, q, seen in mine:
                i = row - r0
                if seen > pre:
                    k2, v2 = rows(q, np.arange(pre, seen), h)
                    m2, l2, o2 = weigh(x[i], k2, v2)
                    top = torch.maximum(m[i], m2)
                    f, f2 = torch.exp(m[i] - top), torch.exp(m2 - top)
                    y = (o[i] * f + o2 * f2) / (l[i] * f + l2 * f2)
                else:
                    y = o[i] / l[i]
                out[row, h * G:(h + 1) * G] = y
    return out
