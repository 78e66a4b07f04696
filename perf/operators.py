"""The serving-step operators over a paged cache, as they are measured: cases, inputs, the
plain form of each operator in elementary torch operations, the library's calls, and a
64-bit evaluation of each definition.

Five operators, in the order a serving step calls them:

  tables         hp_step_tables: the requests' lengths and the tokens each adds -> grown block
                 tables, slot map and positions (whole numbers only).
  qk             hp_qk_norm_rope_append: RMS norm of each query and key head, the position
                 rotation (one or several axes), the K and V rows into their pages.
  latent_append  hp_latent_append: RMS norm of a token's shared latent vector, rotation of its
                 shared key and of the queries' rotary parts, the latent row into its page.
  decode         hp_latent_decode: attention over the paged latent rows, absorbed form (one or
                 a few query tokens per sequence).
  prefill        hp_latent_prefill: attention of prompt tokens over the same rows, expanded
                 form (keys and values projected up from the latent for every head).
"""
import math

import numpy as np
import torch

own = False

LATENT, ROPE, NOPE, VDIM = 512, 64, 128, 128  # widths of the latent rows and of a head
TORCH = {"bf16": torch.bfloat16, "f16": torch.float16}
EPS = 1e-6
THETA = 10000.0


# ------------------------------------------------------------------------------- cases
def listed():
    return [
        # one decode step of a small server: 32 running requests, a token each
        dict(name="tables_decode_32", op="tables", seqs=32, page=16, lo=64, hi=2048, prompts=0,
             new_hi=1, wide=False, shape=1),
        # a large mixed step: 4096 requests, one in eight a prompt of up to 2000 tokens,
        # 64-bit indices
        dict(name="tables_mixed_4096", op="tables", seqs=4096, page=16, lo=0, hi=8000, prompts=8,
             new_hi=2000, wide=True, shape=2),
        # a decode step of 64 sequences, 32 query heads on 8 K/V heads of 128 dims
        dict(name="qk_decode_64", op="qk", tokens=64, hq=32, hkv=8, dim=128, rot=128, axes=1,
             inter=False, dtype="bf16", page=16, shape=3),
        # a prompt chunk with image tokens: three position axes, odd token count
        dict(name="qk_prompt_8193_axes3", op="qk", tokens=8193, hq=32, hkv=8, dim=128, rot=128,
             axes=3, inter=False, dtype="f16", page=16, shape=4),
        # a decode step of 128 sequences of a 128-head latent-attention layer
        dict(name="latent_append_decode_128", op="latent_append", tokens=128, heads=128,
             inter=True, dtype="bf16", page=64, shape=5),
        # a long prompt chunk of a 16-head shard of such a layer
        dict(name="latent_append_prompt_16001", op="latent_append", tokens=16001, heads=16,
             inter=True, dtype="bf16", page=64, shape=6),
        # the smallest call: one sequence, 16 heads; latency counts
        dict(name="decode_1_h16", op="decode", seqs=1, heads=16, lo=1777, hi=1777, nq=1, page=16,
             dtype="bf16", shape=7),
        # an ordinary decode batch at 128 heads: ragged, some sequences empty or a token long
        dict(name="decode_64_h128", op="decode", seqs=64, heads=128, lo=0, hi=8191, nq=1, page=64,
             dtype="bf16", shape=8),
        # long contexts on a 32-head shard, two query tokens each (one drafted)
        dict(name="decode_16_h32_long", op="decode", seqs=16, heads=32, lo=20000, hi=131072, nq=2,
             page=16, dtype="f16", shape=9),
        # a few short prompts, odd lengths, on a 16-head shard
        dict(name="prefill_3_short", op="prefill", seqs=3, heads=16, lo=1, hi=97, prefix=0,
             page=16, dtype="bf16", shape=10),
        # eight prompts of about 2000 tokens, each behind a cached prefix
        dict(name="prefill_8_prefix", op="prefill", seqs=8, heads=16, lo=900, hi=2500,
             prefix=1500, page=16, dtype="f16", shape=11),
        # two long prompts, 32 heads
        dict(name="prefill_2_long", op="prefill", seqs=2, heads=32, lo=9000, hi=12289, prefix=0,
             page=64, dtype="bf16", shape=12),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.4)))))


def draw(rng):
    op = rng.choice(["tables", "qk", "latent_append", "decode", "decode", "prefill", "prefill"])
    shape = rng.randrange(1 << 30)
    dtype = rng.choice(["bf16", "f16"])
    page = rng.choice([8, 16, 32, 64, 128])
    if op == "tables":
        return dict(op=op, seqs=_log_int(rng, 1, 4096), page=rng.choice([1, 5, 16, 64]),
                    lo=0, hi=_log_int(rng, 16, 8000), prompts=rng.choice([0, 8, 16]),
                    new_hi=_log_int(rng, 1, 1500), wide=rng.random() < 0.5, shape=shape)
    if op == "qk":
        hkv = rng.choice([1, 2, 4, 8])
        dim = rng.choice([64, 80, 128, 256])
        hq = hkv * rng.choice([1, 3, 4, 8])
        axes = rng.choice([1, 1, 2, 3, 4])
        return dict(op=op, tokens=_log_int(rng, 1, 8193 * 48 * 128 // ((hq + 2 * hkv) * dim)
                                           if (hq + 2 * hkv) * dim > 48 * 128 else 8193),
                    hq=hq, hkv=hkv, dim=dim, rot=rng.choice([dim, dim // 2 // 16 * 16]),
                    axes=axes, inter=rng.random() < 0.5, dtype=dtype, page=page, shape=shape)
    if op == "latent_append":
        heads = rng.choice([8, 16, 32, 64, 128])
        return dict(op=op, tokens=_log_int(rng, 1, 16000 * 16 // max(heads, 16)), heads=heads,
                    inter=rng.random() < 0.5, dtype=dtype, page=page, shape=shape)
    if op == "decode":
        heads = rng.choice([8, 16, 24, 32, 64, 128])
        seqs = _log_int(rng, 1, 128)
        nq = rng.choice([1, 1, 1, 2, 3])
        hi = _log_int(rng, 16, max(17, min(65536, 120_000_000 // (seqs * heads * nq))))
        return dict(op=op, seqs=seqs, heads=heads, lo=0, hi=hi, nq=nq, page=page, dtype=dtype,
                    shape=shape)
    heads = rng.choice([4, 8, 16, 32])
    seqs = _log_int(rng, 1, 12)
    hi = _log_int(rng, 8, int(min(8000, 8000 * math.sqrt(16 / (seqs * heads)))))
    return dict(op=op, seqs=seqs, heads=heads, lo=1, hi=hi,
                prefix=rng.choice([0, 0, hi // 3, hi]), page=page, dtype=dtype, shape=shape)


def _np(case):
    return np.random.default_rng(case["shape"])


def _decode_shape(case):
    r = _np(case)
    lens = r.integers(case["lo"], case["hi"] + 1, case["seqs"])
    if case["lo"] == 0 and case["seqs"] > 4:  # an empty and a one-token sequence among them
        lens[1], lens[2] = 0, 1
    return lens, np.full(case["seqs"], case["nq"])


def _prefill_shape(case):
    r = _np(case)
    new = r.integers(case["lo"], case["hi"] + 1, case["seqs"])
    pre = r.integers(0, case["prefix"] + 1, case["seqs"])
    return new + pre, new


def _tables_shape(case):
    r = _np(case)
    S, P = case["seqs"], case["page"]
    lens = r.integers(case["lo"], case["hi"] + 1, S)
    new = np.ones(S, np.int64)
    if case["prompts"]:
        pick = r.random(S) * case["prompts"] < 1
        new[pick] = r.integers(1, case["new_hi"] + 1, int(pick.sum()))
        lens[pick] = 0
    new[r.random(S) < 0.05] = 0  # finished or waiting requests add nothing
    have = -(-lens // P) + (r.random(S) < 0.1)  # some hold a page in reserve
    need = np.maximum(have, -(-(lens + new) // P))
    return lens, new, have, need


def work(case):
    """Bytes and operations one pass cannot do without."""
    op = case["op"]
    if op == "tables":
        lens, new, have, need = _tables_shape(case)
        w, S = (8 if case["wide"] else 4), case["seqs"]
        grown = int((need - have).sum())
        T = int(new.sum())
        read = w * (3 * S + 1 + int(have.sum()) + grown)
        write = w * (3 * S + 2 + int(need.sum()) + T) + 8 * T
        return {"bytes": read + write, "flops": 0}
    if op == "qk":
        T, D = case["tokens"], case["dim"]
        heads = case["hq"] + 2 * case["hkv"]
        rows = 2 * T * heads * D * 2
        return {"bytes": rows + T * (8 + 8 * case["axes"] + 4 * case["rot"]),
                "flops": T * (case["hq"] + case["hkv"]) * (4 * D + 3 * case["rot"])}
    if op == "latent_append":
        T, H = case["tokens"], case["heads"]
        return {"bytes": T * (2 * 2 * (LATENT + ROPE) + 2 * 2 * H * ROPE + 16 + 4 * ROPE),
                "flops": T * (4 * LATENT + 3 * ROPE * (H + 1))}
    if op == "decode":
        lens, nq = _decode_shape(case)
        H, W = case["heads"], LATENT + ROPE
        vis = sum(max(0, int(l) - int(n) + 1 + i) for l, n in zip(lens, nq) for i in range(n))
        return {"bytes": int(lens.sum()) * W * 2 + int(nq.sum()) * H * (W + LATENT) * 2,
                "flops": 2 * vis * H * (W + LATENT)}
    lens, new = _prefill_shape(case)
    H = case["heads"]
    pairs = sum(int(n) * int(l - n) + int(n) * (int(n) + 1) // 2 for l, n in zip(lens, new))
    L, T = int(lens.sum()), int(new.sum())
    return {"bytes": 2 * (L * (LATENT + ROPE) + H * (NOPE + VDIM) * LATENT
                          + T * H * (NOPE + ROPE + VDIM)),
            "flops": 2 * pairs * H * (NOPE + ROPE + VDIM) + 2 * L * LATENT * H * (NOPE + VDIM)}


# ------------------------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _randn(g, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def _cos_sin(max_pos, rot):
    """[max_pos, rot]: rot / 2 cosines, then rot / 2 sines of pos * THETA^(-2 i / rot)."""
    i = torch.arange(rot // 2, device="cuda", dtype=torch.float64)
    ang = torch.arange(max_pos, device="cuda", dtype=torch.float64)[:, None] * THETA ** (-2 * i / rot)
    return torch.cat([ang.cos(), ang.sin()], 1).float()


def _sections(rot, axes):
    half = rot // 2
    cut = [half // 4] + [(half - half // 4) // (axes - 1)] * (axes - 1) if axes > 1 else [half]
    cut[-1] += half - sum(cut)
    return cut


def _slots(g, tokens, page):
    """A slot for each token in a pool a quarter larger than they need, a few tokens without
    one (the padding rows of a padded batch)."""
    pages = -(-tokens * 5 // (4 * page)) + 2
    slot = torch.randperm(pages * page, generator=g, device="cuda")[:tokens].to(torch.int64)
    if tokens > 16:
        slot[-(tokens // 50 + 1):] = -1
    return slot, pages


def _paged_batch(g, lens, page, dtype):
    """Latent rows of a batch in a pool of shuffled pages: (pool, table, seq_ptr, lens)."""
    need = -(-lens // page)
    pages = int(need.sum()) + 3
    table = torch.randperm(pages, generator=g, device="cuda")[:int(need.sum())].to(torch.int32)
    seq_ptr = np.concatenate([[0], np.cumsum(need)])
    pool = _randn(g, (pages, page, LATENT + ROPE), dtype)
    # what lies in the slots that no sequence has filled is not a number
    live = torch.zeros(pages * page, dtype=torch.bool, device="cuda")
    at = torch.from_numpy(np.repeat(seq_ptr[:-1], lens)).cuda()
    t = torch.from_numpy(np.concatenate([np.arange(n) for n in lens] + [np.zeros(0, np.int64)])).cuda()
    live[table.long()[at + t // page] * page + t % page] = True
    pool.view(-1, LATENT + ROPE)[~live] = float("nan")
    return pool, table, torch.from_numpy(seq_ptr.astype(np.int32)).cuda(), \
        torch.from_numpy(lens.astype(np.int32)).cuda()


def _inputs(case, seed):
    g, op = _gen(seed), case["op"]
    s = dict(case)
    if op == "tables":
        lens, new, have, need = _tables_shape(case)
        it = torch.int64 if case["wide"] else torch.int32
        pages = int(need.sum()) + 17
        perm = torch.randperm(pages, generator=g, device="cuda").to(it)
        dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda().to(it)  # noqa: E731
        n = int(have.sum())
        s.update(table=perm[:n].clone(), seq_ptr=dev(np.concatenate([[0], np.cumsum(have)])),
                 lens=dev(lens), new=dev(new), free=perm[n:].clone(), entries=int(need.sum()),
                 cap=int(new.sum()) + 5, it=it)
        return s
    dt = TORCH[case["dtype"]]
    s["dt"] = dt
    if op in ("qk", "latent_append"):
        T = case["tokens"]
        s["slot"], s["pages"] = _slots(g, T, case["page"])
        s["rot"] = case["rot"] if op == "qk" else ROPE
        axes = case.get("axes", 1)
        s["max_pos"] = 16384
        s["pos"] = torch.randint(0, s["max_pos"], (axes, T), generator=g, device="cuda",
                                 dtype=torch.int32)
        s["sections"] = _sections(s["rot"], axes)
        s["table"] = _cos_sin(s["max_pos"], s["rot"])
    if op == "qk":
        hq, hkv, D = case["hq"], case["hkv"], case["dim"]
        s["qkv"] = _randn(g, (T, (hq + 2 * hkv) * D), dt, 2.0)  # one projection's output
        s["qw"] = (1 + _randn(g, (D,), torch.float32, 0.1)).to(dt)
        s["kw"] = (1 + _randn(g, (D,), torch.float32, 0.1)).to(dt)
        s["k_pool"] = _randn(g, (s["pages"], case["page"], hkv, D), dt)
        s["v_pool"] = _randn(g, (s["pages"], case["page"], hkv, D), dt)
        s["q_out"] = torch.zeros((T, hq, D), dtype=dt, device="cuda")
    elif op == "latent_append":
        H = case["heads"]
        s["kv"] = _randn(g, (T, LATENT + ROPE), dt, 3.0)  # latent and shared key, one projection
        s["w"] = (1 + _randn(g, (LATENT,), torch.float32, 0.1)).to(dt)
        s["q"] = _randn(g, (T, H, NOPE + ROPE), dt)  # nope part first, then the rotary part
        s["q_out"] = torch.zeros((T, H, ROPE), dtype=dt, device="cuda")
        s["pool"] = _randn(g, (s["pages"], case["page"], LATENT + ROPE), dt)
    elif op == "decode":
        lens, nq = _decode_shape(case)
        s["host_lens"], s["host_q"] = lens, nq
        s["pool"], s["table"], s["seq_ptr"], s["lens"] = _paged_batch(g, lens, case["page"], dt)
        T = int(nq.sum())
        s["q"] = _randn(g, (T, case["heads"], LATENT + ROPE), dt)
        s["q_ptr"] = torch.from_numpy(np.concatenate([[0], np.cumsum(nq)]).astype(np.int32)).cuda()
        s["scale"] = 1.0 / math.sqrt(NOPE + ROPE)
    else:
        lens, new = _prefill_shape(case)
        s["host_lens"], s["host_q"] = lens, new
        s["pool"], s["table"], s["seq_ptr"], s["lens"] = _paged_batch(g, lens, case["page"], dt)
        T, H = int(new.sum()), case["heads"]
        s["q"] = _randn(g, (T, H, NOPE + ROPE), dt)
        s["q_ptr"] = torch.from_numpy(np.concatenate([[0], np.cumsum(new)]).astype(np.int32)).cuda()
        s["w_kv"] = _randn(g, (H, NOPE + VDIM, LATENT), dt, LATENT ** -0.5)
        s["scale"] = 1.0 / math.sqrt(NOPE + ROPE)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:
        _prepare_own(s)
    return s


def _prepare_own(s):
    """The buffers, descriptors and workspaces a user's program keeps between steps."""
    from paged_kv_cache_hp_gb300 import hp
    op, dev = s["op"], "cuda"
    s["status"] = torch.zeros(1, dtype=torch.int32, device=dev)
    it = hp.IDX_U64 if s.get("wide") else hp.IDX_U32
    if op == "tables":
        S, cap, ity = s["seqs"], s["cap"], s["it"]
        e = lambda n, t=ity: torch.empty(n, dtype=t, device=dev)  # noqa: E731
        s["o_table"], s["o_ptr"], s["o_lens"], s["o_new"] = e(s["entries"]), e(S + 1), e(S), e(S + 1)
        s["o_slot"], s["o_pos"], s["o_tot"] = e(cap, torch.int64), e(cap), e(3, torch.int64)
        s["step"] = hp.step_desc(
            block_table=s["table"], seq_ptr=s["seq_ptr"], seq_lens=s["lens"], new_lens=s["new"],
            free_pages=s["free"], page_size=s["page"], index_type=it, table_out=s["o_table"],
            seq_ptr_out=s["o_ptr"], lens_out=s["o_lens"], new_ptr_out=s["o_new"],
            slot_map=s["o_slot"], positions=s["o_pos"], totals=s["o_tot"])
        rc, n = hp.hp_step_tables_workspace_bytes(S)
        assert rc == 0
        s["ws"] = torch.empty(n, dtype=torch.uint8, device=dev)
    elif op == "qk":
        hq, hkv, D = s["hq"], s["hkv"], s["dim"]
        s["rope"] = hp.rope_desc(cos_sin=s["table"], positions=s["pos"], sections=s["sections"],
                                 interleaved=s["inter"], index_type=it)
        q, k, v = s["qkv"].split([hq * D, hkv * D, hkv * D], 1)
        s["desc"] = hp.qk_desc(q=q, k=k, v=v, q_out=s["q_out"], q_weight=s["qw"],
                               k_weight=s["kw"], eps=EPS, num_q_heads=hq, num_kv_heads=hkv,
                               head_dim=D, dtype=s["dtype"], slot_map=s["slot"],
                               k_pool=s["k_pool"], v_pool=s["v_pool"], num_pages=s["pages"],
                               page_size=s["page"])
    elif op == "latent_append":
        s["rope"] = hp.rope_desc(cos_sin=s["table"], positions=s["pos"], sections=s["sections"],
                                 interleaved=s["inter"], index_type=it)
        s["desc"] = hp.latent_desc(latent=s["kv"][:, :LATENT], k_rope=s["kv"][:, LATENT:],
                                   q_rope=s["q"][:, :, NOPE:], q_out=s["q_out"],
                                   latent_weight=s["w"], eps=EPS, dtype=s["dtype"],
                                   slot_map=s["slot"], pool=s["pool"], num_pages=s["pages"],
                                   page_size=s["page"])
    else:
        s["desc"] = hp.PagedDesc(s["pool"], s["table"], s["seq_ptr"], s["lens"],
                                 num_pages=s["pool"].shape[0], page_size=s["page"], num_heads=1,
                                 head_dim=LATENT + ROPE, dtype=s["dtype"], index_type=it)
        T, H = s["q"].shape[:2]
        if op == "decode":
            s["out"] = torch.empty((T, H, LATENT), dtype=s["dt"], device=dev)
            rc, n = hp.hp_latent_decode_workspace_bytes(s["desc"], LATENT, T, H)
        else:
            s["out"] = torch.empty((T, H, VDIM), dtype=s["dt"], device=dev)
            s["kv_tokens"] = int(s["host_lens"].sum())
            rc, n = hp.hp_latent_prefill_workspace_bytes(s["desc"], LATENT, NOPE, VDIM, T, H,
                                                         s["kv_tokens"])
        assert rc == 0, hp.status_name(rc)
        s["ws"] = torch.empty(n, dtype=torch.uint8, device=dev)


# --------------------------------------------------------------------------- one pass
def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    from paged_kv_cache_hp_gb300 import hp
    op = s["op"]
    if op == "tables":
        hp.hp_step_tables(s["step"], s["ws"], s["status"])
        return s["o_table"], s["o_ptr"], s["o_lens"], s["o_new"], s["o_slot"], s["o_pos"], s["o_tot"]
    if op == "qk":
        hp.hp_qk_norm_rope_append(s["desc"], s["rope"], s["status"])
        return s["q_out"], s["k_pool"], s["v_pool"]
    if op == "latent_append":
        hp.hp_latent_append(s["desc"], s["rope"], s["status"])
        return s["q_out"], s["pool"]
    T, H = s["q"].shape[:2]
    if op == "decode":
        hp.hp_latent_decode(s["desc"], LATENT, s["q"], s["q_ptr"], T, H, s["scale"], s["out"],
                            s["ws"], s["status"])
    else:
        hp.hp_latent_prefill(s["desc"], LATENT, s["w_kv"], NOPE, VDIM, s["q"], s["q_ptr"], T, H,
                             s["scale"], s["out"], s["kv_tokens"], s["ws"], s["status"])
    return s["out"]


def _run_plain(s):
    return {"tables": _plain_tables, "qk": _plain_qk, "latent_append": _plain_latent_append,
            "decode": _plain_decode, "prefill": _plain_prefill}[s["op"]](s)


def _plain_tables(s):
    P, S, cap, it, dev = s["page"], s["seqs"], s["cap"], s["it"], "cuda"
    lens, new, sp = s["lens"].long(), s["new"].long(), s["seq_ptr"].long()
    have = sp[1:] - sp[:-1]
    need = torch.maximum(have, (lens + new + P - 1) // P)
    zero = torch.zeros(1, dtype=torch.int64, device=dev)
    ptr = torch.cat([zero, need.cumsum(0)])
    taken = torch.cat([zero, (need - have).cumsum(0)])
    nptr = torch.cat([zero, new.cumsum(0)])
    e = torch.arange(s["entries"], device=dev)
    q = torch.searchsorted(ptr, e, right=True) - 1
    j = e - ptr[q]
    old = j < have[q]
    src = torch.where(old, sp[q] + j, s["table"].numel() + taken[q] + j - have[q])
    table = torch.cat([s["table"], s["free"]])[src]
    t = torch.arange(cap, device=dev)
    real = t < nptr[-1]
    r = (torch.searchsorted(nptr, t, right=True) - 1).clamp(max=S - 1)
    pos = lens[r] + t - nptr[r]
    page = table.long()[(ptr[r] + pos // P).clamp(max=max(s["entries"] - 1, 0))]
    slot = torch.where(real, page * P + pos % P, torch.full_like(pos, -1))
    pos = torch.where(real, pos, torch.zeros_like(pos))
    return (table, ptr.to(it), (lens + new).to(it), nptr.to(it), slot, pos.to(it),
            torch.stack([ptr[-1], nptr[-1], taken[-1]]))


def _angles(s):
    """cos and sin of each token's rotation, [T, rot / 2], each pair on its axis' position."""
    axis = torch.repeat_interleave(torch.arange(len(s["sections"]), device="cuda"),
                                   torch.tensor(s["sections"], device="cuda"),
                                   output_size=s["rot"] // 2)
    pos = s["pos"].long()[axis].t()                       # [T, rot / 2]
    pair = torch.arange(s["rot"] // 2, device="cuda")
    return s["table"][pos, pair], s["table"][pos, pair + s["rot"] // 2]


def _rotate(x, cos, sin, rot, inter):
    """x [T, H, D] with its first rot dims rotated."""
    y = x.clone()
    a, b = (slice(0, rot, 2), slice(1, rot, 2)) if inter else (slice(0, rot // 2), slice(rot // 2, rot))
    c, n = cos[:, None], sin[:, None]
    y[..., a] = x[..., a] * c - x[..., b] * n
    y[..., b] = x[..., b] * c + x[..., a] * n
    return y


def _plain_norm(x, w):
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w.float()


def _plain_qk(s):
    T, hq, hkv, D = s["tokens"], s["hq"], s["hkv"], s["dim"]
    x = s["qkv"].float().view(T, hq + 2 * hkv, D)
    cos, sin = _angles(s)
    q = _rotate(_plain_norm(x[:, :hq], s["qw"]), cos, sin, s["rot"], s["inter"])
    k = _rotate(_plain_norm(x[:, hq:hq + hkv], s["kw"]), cos, sin, s["rot"], s["inter"])
    live = s["slot"] >= 0
    at = s["slot"][live]
    s["q_out"][live] = q[live].to(s["dt"])
    s["k_pool"].view(-1, hkv, D)[at] = k[live].to(s["dt"])
    s["v_pool"].view(-1, hkv, D)[at] = x[live, hq + hkv:].to(s["dt"])
    return s["q_out"], s["k_pool"], s["v_pool"]


def _plain_latent_append(s):
    kv = s["kv"].float()
    cos, sin = _angles(s)
    c = _plain_norm(kv[:, :LATENT], s["w"])
    k = _rotate(kv[:, None, LATENT:], cos, sin, ROPE, s["inter"])[:, 0]
    q = _rotate(s["q"][:, :, NOPE:].float(), cos, sin, ROPE, s["inter"])
    live = s["slot"] >= 0
    s["q_out"][live] = q[live].to(s["dt"])
    s["pool"].view(-1, LATENT + ROPE)[s["slot"][live]] = torch.cat([c, k], 1)[live].to(s["dt"])
    return s["q_out"], s["pool"]


def _rows(s, first, n):
    """The n latent rows of the sequence whose slice starts at entry `first`, 32 bits."""
    pages = s["table"][first:first + -(-n // s["page"])].long()
    return s["pool"][pages].reshape(-1, LATENT + ROPE)[:n].float()


def _softmax(x):
    e = torch.exp(x - x.max(-1, keepdim=True).values)
    return e / e.sum(-1, keepdim=True)


def _hidden(n, L):
    """[n, L]: which of a sequence's L tokens its n queries, the last n tokens, do not see."""
    i = torch.arange(n, device="cuda")
    return torch.arange(L, device="cuda")[None, :] > (L - n + i)[:, None]


def _plain_decode(s):
    out = torch.zeros(s["q"].shape[:2] + (LATENT,), dtype=s["dt"], device="cuda")
    first = q0 = 0
    for L, n in zip(s["host_lens"].tolist(), s["host_q"].tolist()):
        skip = max(0, n - L)  # queries before the sequence's first token see nothing
        if L and n > skip:
            c = _rows(s, first, L)
            q = s["q"][q0 + skip:q0 + n].float()
            x = torch.einsum("nhd,td->nht", q, c) * s["scale"]
            x.masked_fill_(_hidden(n - skip, L)[:, None], float("-inf"))
            out[q0 + skip:q0 + n] = torch.einsum("nht,td->nhd", _softmax(x), c[:, :LATENT]).to(s["dt"])
        first += -(-L // s["page"])
        q0 += n
    return out


def _plain_prefill(s):
    H = s["heads"]
    out = torch.empty((s["q"].shape[0], H, VDIM), dtype=s["dt"], device="cuda")
    first = q0 = 0
    for L, n in zip(s["host_lens"].tolist(), s["host_q"].tolist()):
        c = _rows(s, first, L)
        hide = _hidden(n, L)
        for h in range(H):
            kv = c[:, :LATENT] @ s["w_kv"][h].float().t()
            k = torch.cat([kv[:, :NOPE], c[:, LATENT:]], 1)
            x = s["q"][q0:q0 + n, h].float() @ k.t() * s["scale"]
            x.masked_fill_(hide, float("-inf"))
            out[q0:q0 + n, h] = (_softmax(x) @ kv[:, NOPE:]).to(s["dt"])
        first += -(-L // s["page"])
        q0 += n
    return out


# --------------------------------------------------------------------- 64-bit definition
def exact(case, seed):
    op = case["op"]
    if op == "tables" or work(case)["flops"] > 9e12:
        return None  # whole numbers, which the plain form gives as they are; or too long
    s = _inputs(case, seed)
    if op == "qk":
        return _exact_qk(s)
    if op == "latent_append":
        return _exact_latent_append(s)
    if op == "decode":
        return _exact_attention(s, absorbed=True)
    return _exact_attention(s, absorbed=False)


def _turn(v, s, t):
    """Rotates the vectors v [heads, dims] of token t as complex numbers."""
    half = s["rot"] // 2
    pos = np.repeat(s["h_pos"][:, t], s["sections"])
    z = s["h_tab"][pos, np.arange(half)] + 1j * s["h_tab"][pos, half + np.arange(half)]
    y = v.copy()
    if s["inter"]:
        w = (v[:, 0:2 * half:2] + 1j * v[:, 1:2 * half:2]) * z
        y[:, 0:2 * half:2], y[:, 1:2 * half:2] = w.real, w.imag
    else:
        w = (v[:, :half] + 1j * v[:, half:2 * half]) * z
        y[:, :half], y[:, half:2 * half] = w.real, w.imag
    return y


def _host64(t):
    return t.double().cpu().numpy()


def _exact_qk(s):
    hq, hkv, D = s["hq"], s["hkv"], s["dim"]
    x, slot = _host64(s["qkv"]).reshape(-1, hq + 2 * hkv, D), s["slot"].cpu().numpy()
    s["h_pos"], s["h_tab"] = s["pos"].cpu().numpy(), _host64(s["table"])
    w = np.concatenate([np.tile(_host64(s["qw"]), (hq, 1)), np.tile(_host64(s["kw"]), (hkv, 1))])
    q_out, kp, vp = _host64(s["q_out"]), _host64(s["k_pool"]), _host64(s["v_pool"])
    for t, at in enumerate(slot):
        if at < 0:
            continue
        v = x[t, :hq + hkv]
        y = _turn(v / np.sqrt((v ** 2).sum(1, keepdims=True) / D + EPS) * w, s, t)
        q_out[t] = y[:hq]
        kp[at // s["page"], at % s["page"]] = y[hq:]
        vp[at // s["page"], at % s["page"]] = x[t, hq + hkv:]
    return torch.from_numpy(q_out), torch.from_numpy(kp), torch.from_numpy(vp)


def _exact_latent_append(s):
    kv, q, slot = _host64(s["kv"]), _host64(s["q"]), s["slot"].cpu().numpy()
    s["h_pos"], s["h_tab"], w = s["pos"].cpu().numpy(), _host64(s["table"]), _host64(s["w"])
    q_out, pool = _host64(s["q_out"]), _host64(s["pool"])
    for t, at in enumerate(slot):
        if at < 0:
            continue
        q_out[t] = _turn(q[t, :, NOPE:], s, t)
        c = kv[t, :LATENT]
        row = pool[at // s["page"], at % s["page"]]
        row[:LATENT] = c / math.sqrt((c ** 2).sum() / LATENT + EPS) * w
        row[LATENT:] = _turn(kv[t:t + 1, LATENT:], s, t)[0]
    return torch.from_numpy(q_out), torch.from_numpy(pool)


def _exact_attention(s, absorbed):
    """softmax(scale q . k) v over each query's tokens, head by head and in blocks of queries
    (64-bit products on the GPU); expanded keys and values where not absorbed."""
    T, H = s["q"].shape[:2]
    out = torch.zeros((T, H, LATENT if absorbed else VDIM), dtype=torch.float64, device="cuda")
    flat = s["pool"].view(-1, LATENT + ROPE)
    ptr = s["seq_ptr"].cpu().numpy()
    table = s["table"].cpu().numpy().astype(np.int64)
    q0 = 0
    for i, (L, n) in enumerate(zip(s["host_lens"].tolist(), s["host_q"].tolist())):
        t = np.arange(L)
        at = table[ptr[i] + t // s["page"]] * s["page"] + t % s["page"] if L else t
        row = flat[torch.from_numpy(at).cuda()].double()
        for h in (0,) if absorbed else range(H):
            for a in range(0, n, 2048):
                b = min(n, a + 2048)
                seen = L - n + b  # tokens the block's last query sees
                if seen <= 0:
                    continue
                if absorbed:
                    q = s["q"][q0 + a:q0 + b].double()           # [m, H, W]
                    k, v = row[:seen], row[:seen, :LATENT]
                else:
                    q = s["q"][q0 + a:q0 + b, h:h + 1].double()  # [m, 1, 192]
                    up = s["w_kv"][h].double()
                    k = torch.cat([row[:seen, :LATENT] @ up[:NOPE].t(), row[:seen, LATENT:]], 1)
                    v = row[:seen, :LATENT] @ up[NOPE:].t()
                x = (q @ k.t()) * s["scale"]
                last = L - n + torch.arange(a, b, device="cuda")
                x = torch.where(torch.arange(seen, device="cuda") <= last[:, None, None], x,
                                torch.full_like(x, float("-inf")))
                top = x.amax(-1, keepdim=True)
                e = torch.exp(x - torch.where(torch.isinf(top), torch.zeros_like(top), top))
                total = e.sum(-1, keepdim=True)
                y = e @ v / torch.where(total == 0, torch.ones_like(total), total)
                if absorbed:
                    out[q0 + a:q0 + b] = y
                else:
                    out[q0 + a:q0 + b, h] = y[:, 0]
        q0 += n
    return out

