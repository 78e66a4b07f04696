"""GPU parity of the serving-step operators where a sum, a mask or an index is at its edge, against
the plain 64-bit implementations of step_ref.py; what its bounds do not cover is derived here."""
import numpy as np
import pytest

import step_ref as ref
from helpers import index_tensor
from test_gpu_step import (A, Latent, cores, dev, host, make_step, run_decode, run_prefill,
                           selecting_weights, status_tensor)

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ small weights in f16
# A weight far below its row's largest is subnormal in f16: its rounding is off by half of the
# smallest subnormal, 2^-25, however small it is.  The kernels hold a row's weights scaled so that
# its reference maximum stands at 2^7, and that reference is at most the true maximum: in units of the
# largest weight each is off by at most 2^-32 besides the relative u.  n weights then move the
# value sum by at most n 2^-32 max |v|, divided by the sum of the weights (in the same units).
SUBNORMAL = 2.0 ** -32
TAIL = np.arange(23.0, 7.0, -1.0) + 0.625  # nats below the largest score, a head each


def tail_rows(n, peak, W, dt, seed):
    """Rows whose dim 0 is 1 at the peak and 0 elsewhere, dims 1 .. 8 the other way round; the
    others are random."""
    import torch
    rows = torch.randn((n, W), generator=torch.Generator().manual_seed(seed))
    rows[:, 0] = 0.0
    rows[:, 1:9] = 1.0
    rows[peak, 0] = 1.0
    rows[peak, 1:9] = 0.0
    return rows.to(dt)


def fill(b, s, rows):
    """Puts `rows` into sequence s of the batch's pool."""
    import torch
    table, sp = (t.cpu().numpy().astype(np.int64) for t in b.desc._keep[1:3])
    t = np.arange(len(rows))
    P = b.pool.shape[0] // b.desc.c.num_pages
    b.pool[torch.from_numpy(table[sp[s] + t // P] * P + t % P).cuda()] = rows.cuda()
    b.rows[s] = rows.double().numpy()


def check_tail(b, s, q, k, v, scale, got, tag):
    o, tol = ref.attention_row(q, k, v, scale, "f16")
    x = k @ q * scale
    tol = tol + len(k) * SUBNORMAL * np.abs(v).max(0) / np.exp(x - x.max()).sum()
    err = np.abs(got - o)
    assert np.isfinite(got).all() and (err <= tol).all(), (*tag, float((err / tol).max()))


@pytest.mark.parametrize("kernel", ["cuda_cores", "default"])
@pytest.mark.parametrize("peak", [0, 3000, 7999])
def test_f16_flat_tail_under_one_peak(hp, kernel, peak):
    """One token far above 7,999 equal ones, 8 to 24 nats by head: the tail's share of dims where
    the peak has nothing is right, its weights being tiny and many.  200 sequences share the tokens'
    pages, so that a worker's range holds whole ones."""
    n, S, scale, H, P = 8000, 200, 1 / 16, len(TAIL), 64
    b = Latent(hp, A([n]), A([1]), H, 512, 576, P, "f16", seed=31)
    fill(b, 0, tail_rows(n, peak, 576, b.dt, 1))
    table = b.desc._keep[1].cpu().numpy().view(np.uint32)
    sp = (np.arange(S + 1) * len(table)).astype(np.uint32)
    b.desc = hp.PagedDesc(b.pool, index_tensor(np.tile(table, S), "cuda"), index_tensor(sp, "cuda"),
                          index_tensor(np.full(S, n, np.uint32), "cuda"), num_pages=b.desc.c.num_pages, page_size=P,
                          num_heads=1, head_dim=576, dtype="f16", index_type=0, flags=cores(hp, kernel))
    b.T, b.q_ptr = S, None
    real = b.queries

    def queries(width):
        import torch
        real(width)
        b.q.zero_()
        b.q[:, :, 0] = torch.from_numpy(16 * TAIL)
        return b.q.cuda()
    b.queries = queries
    got = run_decode(b, scale)
    for s in (0, 1, 77, 198, 199):
        for h in range(H):
            check_tail(b, 0, b.q[s, h].double().numpy(), b.rows[0], b.rows[0][:, :512], scale, got[s, h],
                       ("decode", s, h))


@pytest.mark.parametrize("kernel", ["cuda_cores", "default"])
@pytest.mark.parametrize("peak", [0, 3000, 7999])
def test_f16_flat_tail_under_one_peak_expanded(hp, kernel, peak):
    """The same through the expanded form: three queries at the end of 8,000 tokens."""
    import torch
    n, scale, H = 8000, 1 / 16, len(TAIL)
    b = Latent(hp, A([n]), A([3]), H, 512, 576, 64, "f16", seed=32, flags=cores(hp, kernel))
    fill(b, 0, tail_rows(n, peak, 576, b.dt, 2))
    w = torch.zeros((H, 256, 512), dtype=b.dt)  # every row picks one latent dim: K and V are exact
    w[:, :128, 0] = 1.0
    w[:, 128 + torch.arange(128), 1 + torch.arange(128)] = 1.0
    real = b.queries

    def queries(width):
        real(width)
        b.q.zero_()
        b.q[:, :, 0] = torch.from_numpy(16 * TAIL)
        return b.q.cuda()
    b.queries = queries
    got = run_prefill(b, 128, 128, w, scale)
    for i in range(3):
        c = b.rows[0][:n - 2 + i]
        k = np.concatenate([np.repeat(c[:, :1], 128, 1), c[:, 512:]], 1)
        for h in range(H):
            check_tail(b, 0, b.q[i, h].double().numpy(), k, c[:, 1:129], scale, got[i, h], ("prefill", i, h))


# ------------------------------------------------- values a query does not see
def spoil(b, s, t, row):
    """Token t of sequence s holds `row` (the formula's rows are left as they were)."""
    import torch
    table, sp = (x.cpu().numpy().astype(np.int64) for x in b.desc._keep[1:3])
    P = b.pool.shape[0] // b.desc.c.num_pages
    b.pool[int(table[sp[s] + t // P]) * P + t % P] = torch.as_tensor(row, dtype=b.dt, device="cuda")


@pytest.mark.parametrize("kernel", ["cuda_cores", "default"])
@pytest.mark.parametrize("dtype,lens,nq,H,P,bad", [
    ("bf16", A([300, 70, 64]), A([3, 40, 64]), 16, 16, (298, 51, 33)), ("f16", A([130, 20]), A([2, 3]), 100, 8, (129, 18)),
    ("bf16", A([65, 128, 7]), A([5, 8, 9]), 1, 64, (64, 123, 0)), ("f16", A([4000, 640]), A([7, 200]), 40, 16, (3994, 640 - 130)),
    ("bf16", A([30001]), A([4]), 128, 64, (29999,)), ("bf16", A([64, 128]), A([2, 66]), 64, 16, (63, 126)),
])
@pytest.mark.parametrize("value", ["nan", "inf", "-inf"])
def test_decode_of_tokens_a_query_does_not_see(hp, kernel, dtype, lens, nq, H, P, bad, value):
    """A token whose row is not finite spoils the queries that see it and no other: drafted tokens in
    one step, in several, in one tile of heads and in more."""
    b = Latent(hp, lens, nq, H, 512, 576, P, dtype, seed=41, flags=cores(hp, kernel))
    for s, t in enumerate(bad):
        spoil(b, s, t, [float(value)] * 576)
    got = run_decode(b, 0.07)
    q = b.q.double().numpy()
    for s, i, n in b.seen():
        if n > bad[s]:
            assert np.isnan(got[i]).all(), (s, i)
            continue
        c = b.rows[s][:n]
        for h in range(0, H, max(1, H // 5)):
            o, tol = ref.attention_row(q[i, h], c, c[:, :512], 0.07, dtype)
            assert (np.abs(got[i, h] - o) <= tol).all(), (s, i, h)
        assert np.isfinite(got[i]).all(), (s, i)


@pytest.mark.parametrize("kernel", ["cuda_cores", "default"])
@pytest.mark.parametrize("behind", [0, 1, 60, 127, 128, 129, 200, 254, 300])
@pytest.mark.parametrize("value", ["nan", "inf"])
def test_prefill_of_tokens_a_query_does_not_see(hp, kernel, behind, value):
    """The same through the expanded form, the token at the end of its sequence and further before it:
    in one tile's last block of keys, in both tiles', in blocks of a later unit of queries."""
    lens, nq = A([700, 300, 129, 513]), A([257, 300, 129, 256])
    b = Latent(hp, lens, nq, 2, 512, 576, 16, "bf16" if behind % 2 else "f16", seed=behind, flags=cores(hp, kernel))
    w = selecting_weights(2, 128, 128, 512, b.dt, 7)
    bad = [max(0, int(n) - 1 - behind) for n in lens]
    for s, t in enumerate(bad):
        spoil(b, s, t, [float(value)] * 576)
    got = run_prefill(b, 128, 128, w, 0.07)
    q, wd = b.q.double().numpy(), w.double().numpy()
    for s, i, n in b.seen():
        if n > bad[s]:
            assert np.isnan(got[i]).all(), (s, i)
            continue
        assert np.isfinite(got[i]).all(), (s, i)
        if i % 7 and n < bad[s] - 3:
            continue
        c = b.rows[s][:n]
        for h in range(2):
            kv = c[:, :512] @ wd[h].T
            o, tol = ref.attention_row(q[i, h], np.concatenate([kv[:, :128], c[:, 512:]], 1), kv[:, 128:], 0.07, b.dtype)
            assert (np.abs(got[i, h] - o) <= tol).all(), (s, i, h)


@pytest.mark.parametrize("kernel", ["cuda_cores", "default"])
@pytest.mark.parametrize("behind", [0, 5, 128, 200, 400])
def test_prefill_values_past_the_range_of_f16(hp, kernel, behind):
    """One expanded value of one token is past f16's range, with keys that are not: the infinity in
    its dim for the queries that see the token, every other number as it would be."""
    import torch
    lens, nq = A([700, 300]), A([300, 300])
    b = Latent(hp, lens, nq, 2, 512, 576, 16, "f16", seed=50 + behind, flags=cores(hp, kernel))
    w = selecting_weights(2, 128, 128, 512, b.dt, 7)
    w[:, :, 7] = 0.0
    w[:, 128 + 69] = 0.0
    w[:, 128 + 69, 7] = 2.0  # value dim 69 is twice latent dim 7
    sign = {0: 1.0, 1: -1.0}
    bad = [max(0, int(n) - 1 - behind) for n in lens]
    for s, t in enumerate(bad):
        row = torch.from_numpy(b.rows[s][t]).clone()
        row[7] = sign[s] * 40000.0
        spoil(b, s, t, row)
        b.rows[s][t, 7] = 0.0
    real = b.queries

    def queries(width):
        real(width)
        b.q *= 0.25  # scores near zero: every weight is a normal number
        return b.q.cuda()
    b.queries = queries
    got = run_prefill(b, 128, 128, w, 0.07)
    q, wd = b.q.double().numpy(), w.double().numpy()
    for s, i, n in b.seen():
        if n > bad[s]:
            assert (got[i, :, 69] == sign[s] * np.inf).all(), (s, i)
        if i % 5 and abs(n - bad[s]) > 3:
            continue
        c = b.rows[s][:n]
        for h in range(2):
            kv = c[:, :512] @ wd[h].T
            o, tol = ref.attention_row(q[i, h], np.concatenate([kv[:, :128], c[:, 512:]], 1), kv[:, 128:], 0.07, "f16")
            ok = np.abs(got[i, h] - o) <= tol
            assert ok[:69].all() and ok[70:].all() and (ok[69] or n > bad[s]), (s, i, h)


# ------------------------------------------------------------- pages past every pool
@pytest.mark.parametrize("S", [3, 1500])
@pytest.mark.parametrize("it,page,P", [
    (1, 2 ** 64 - 1, 16), (1, 2 ** 60, 16), (1, 2 ** 60 + 1, 16), (1, 2 ** 59, 16), (1, 2 ** 63, 1), (1, 2 ** 58, 48),
    (0, 2 ** 32 - 1, 16), (0, 2 ** 32 - 1, 2 ** 33), (0, 2 ** 31, 2 ** 33 + 8),
])
def test_slots_of_a_page_past_every_pool(hp, S, it, page, P):
    """A table entry whose slots do not fit 63 bits names no slot of a pool (a product of 64 bits
    wraps to another page's, or below zero to a padding row): the append refuses its tokens."""
    import torch
    lens, new = np.full(S, min(P, 40) - 1), np.full(S, 1)
    s = make_step(hp, lens, new, np.full(S, 1), P, it)
    table = s["d"].keep[0]
    rows = s["d"].table_len
    bad = (0, S - 1)
    for b in bad:
        table[b] = page - 2 ** (64 if it else 32) if page >= 2 ** (63 if it else 31) else page
    assert hp.hp_step_tables(s["d"], s["ws"], s["status"]) == 0
    torch.cuda.synchronize()
    assert s["status"].item() == 0 and rows == S
    slots = s["o"]["slot_map"].cpu().numpy()
    want = min(page * P + int(lens[0]), 2 ** 63 - 1)
    at = s["table"].astype(object) * P + lens
    for i in range(S):
        assert int(slots[i]) == (want if i in bad else at[i]), i
    if P > 64:
        return
    T, pages = len(slots), S + 3
    kv = torch.randn((T, 576)).to(torch.bfloat16).cuda()
    pool = torch.zeros((pages, P, 576), dtype=torch.bfloat16, device="cuda")
    rope = hp.rope_desc(cos_sin=dev(ref.cos_sin(60, 64)), sections=(32,), positions=s["o"]["positions"], index_type=it)
    d = hp.latent_desc(latent=kv[:, :512], k_rope=kv[:, 512:], dtype="bf16", slot_map=s["o"]["slot_map"], pool=pool,
                       num_pages=pages, page_size=P)
    st = status_tensor()
    assert hp.hp_latent_append(d, rope, st) == 0
    torch.cuda.synchronize()
    assert hp.status_name(st.item()) == "HP_ERR_PAGE_ID"
    assert int((pool != 0).any(2).sum()) == S - 2


# ------------------------------------------------------------- a step, number by number
def test_steps_over_a_latent_cache_row_by_row(hp):
    """Tables, append (queries rotated in place), prompts and decode of three steps on one stream, no wait
    between them: the rotated queries, the rows in the pages and both forms' outputs, each against the
    formula with its own bound."""
    import torch
    H, R, Dr, Dn, Dv, P, pages, S = 4, 512, 64, 128, 128, 16, 64, 3
    dt, W, scale = torch.bfloat16, 576, 0.09
    g = torch.Generator().manual_seed(12)
    cs = ref.cos_sin(512, Dr)
    csd, w = dev(cs), selecting_weights(H, Dn, Dv, R, dt, 2)
    wd, w64 = w.cuda(), w.double().numpy()
    gain = (1 + 0.2 * torch.randn(R, generator=g)).to(dt)
    gd = gain.cuda()
    pool = torch.full((pages, P, W), float("nan"), dtype=dt, device="cuda")
    lens, have, table = A([0, 0, 0]), A([0, 0, 0]), np.zeros(0, np.uint32)
    free = np.random.default_rng(1).permutation(pages).astype(np.uint32)
    stream = torch.cuda.Stream()
    for new in (A([33, 1, 140]), A([1, 3, 1]), A([0, 20, 2])):
        need, T, total = np.maximum(have, -(-(lens + new) // P)), int(new.sum()), int((lens + new).sum())
        i32 = dict(dtype=torch.int32, device="cuda")
        o = dict(table_out=torch.empty(int(need.sum()), **i32), seq_ptr_out=torch.empty(S + 1, **i32),
                 lens_out=torch.empty(S, **i32), new_ptr_out=torch.empty(S + 1, **i32),
                 slot_map=torch.empty(T, dtype=torch.int64, device="cuda"), positions=torch.empty(T, **i32))
        d = hp.step_desc(block_table=index_tensor(table, "cuda") if len(table) else None,
                         seq_ptr=index_tensor(np.concatenate([[0], np.cumsum(have)]).astype(np.uint32), "cuda"),
                         seq_lens=index_tensor(lens.astype(np.uint32), "cuda"),
                         new_lens=index_tensor(new.astype(np.uint32), "cuda"),
                         free_pages=index_tensor(free, "cuda"), page_size=P, index_type=0, **o)
        kv = torch.randn((T, W), generator=g).to(dt)
        q = torch.randn((T, H, Dn + Dr), generator=g).to(dt)
        kvd, qd, ws1 = kv.cuda(), q.cuda(), torch.empty(hp.hp_step_tables_workspace_bytes(S)[1], dtype=torch.uint8, device="cuda")
        rope = hp.rope_desc(cos_sin=csd, positions=o["positions"], sections=(Dr // 2,), interleaved=True)
        ld = hp.latent_desc(latent=kvd[:, :R], k_rope=kvd[:, R:], q_rope=qd[:, :, Dn:], q_out=qd[:, :, Dn:],
                            latent_weight=gd, dtype="bf16", slot_map=o["slot_map"], pool=pool, num_pages=pages, page_size=P)
        pd = hp.PagedDesc(pool, o["table_out"], o["seq_ptr_out"], o["lens_out"], num_pages=pages, page_size=P,
                          num_heads=1, head_dim=W, dtype="bf16", index_type=0)
        n = max(hp.hp_latent_prefill_workspace_bytes(pd, R, Dn, Dv, T, H, total)[1],
                hp.hp_latent_decode_workspace_bytes(pd, R, T, H)[1])
        ws2 = torch.empty(n, dtype=torch.uint8, device="cuda")
        out, lat = torch.empty((T, H, Dv), dtype=dt, device="cuda"), torch.empty((T, H, R), dtype=dt, device="cuda")
        st = [status_tensor() for _ in range(4)]
        torch.cuda.synchronize()
        with torch.cuda.stream(stream):
            assert hp.hp_step_tables(d, ws1, st[0]) == 0
            assert hp.hp_latent_append(ld, rope, st[1]) == 0
            assert hp.hp_latent_prefill(pd, R, wd, Dn, Dv, qd, o["new_ptr_out"], T, H, scale, out, total, ws2, st[2]) == 0
            qa = torch.cat([torch.einsum("thd,hdr->thr", qd[:, :, :Dn].float(), wd[:, :Dn].float()),
                            qd[:, :, Dn:].float()], 2).to(dt)
            assert hp.hp_latent_decode(pd, R, qa, o["new_ptr_out"], T, H, scale, lat, ws2, st[3]) == 0
        stream.synchronize()
        assert [x.item() for x in st] == [0] * 4
        want = ref.step_tables(lens, new, np.concatenate([[0], np.cumsum(have)]), table, free, P)
        assert o["table_out"].cpu().numpy().view(np.uint32).tolist() == want[0]
        assert o["slot_map"].cpu().tolist() == want[4]
        # the rows stored and the queries
        pos, slots = np.array(want[5])[None], np.array(want[4])
        cos, sin = ref.angles(cs, pos, (Dr // 2,))
        x, rows = kv.double().numpy(), host(pool).reshape(-1, W)
        c = ref.norm(x[:, :R], gain.double().numpy(), 1e-6)
        k = ref.rotate(x[:, None, R:], cos, sin, True)[:, 0]
        assert (np.abs(rows[slots, :R] - c) <= ref.rope_bound(c, c, "bf16")).all()
        assert (np.abs(rows[slots, R:] - k) <= ref.rope_bound(k, x[:, R:], "bf16")).all()
        x, turned = q.double().numpy(), host(qd)
        y = ref.rotate(x[:, :, Dn:], cos, sin, True)
        assert np.array_equal(turned[:, :, :Dn], x[:, :, :Dn])
        assert (np.abs(turned[:, :, Dn:] - y) <= ref.rope_bound(y, x[:, :, Dn:], "bf16")).all()
        # both forms, from the rows and queries as they are stored
        qh, got, gat, i = host(qa), host(out), host(lat), 0
        for s in range(S):
            at = np.arange(lens[s] + new[s])
            mine = np.array(want[0][want[1][s]:want[1][s + 1]])
            cache = rows[mine[at // P] * P + at % P]
            for j in range(new[s]):
                seen = cache[:lens[s] + j + 1]
                for h in range(H):
                    e = seen[:, :R] @ w64[h].T
                    r, tol = ref.attention_row(turned[i, h], np.concatenate([e[:, :Dn], seen[:, R:]], 1), e[:, Dn:], scale, "bf16")
                    assert (np.abs(got[i, h] - r) <= tol).all(), (s, j, h)
                    r, tol = ref.attention_row(qh[i, h], seen, seen[:, :R], scale, "bf16")
                    assert (np.abs(gat[i, h] - r) <= tol).all(), (s, j, h)
                i += 1
        lens, have, table = lens + new, need, np.array(want[0], np.uint32)
        free = np.array([p for p in free if p not in set(want[0])], np.uint32)


# ------------------------------------------------------------------- plans, shared and reused
@pytest.mark.parametrize("kernel", ["cuda_cores", "default"])
@pytest.mark.parametrize("S", [1, 5, 128, 129])
def test_planned_layers_behind_a_whole_call(hp, kernel, S):
    """hp_latent_decode leaves its plan in the workspace, made by a launch of its own or by the first
    kernel: planned calls over other layers' pools follow it, then again behind other queries."""
    import torch
    lens = np.random.default_rng(S).integers(0, 400, S)
    nq = np.random.default_rng(S + 1).integers(0, 3, S)
    nq[0] = 1
    b = Latent(hp, lens, nq, 16, 512, 576, 16, "bf16", seed=S, flags=cores(hp, kernel))
    q = b.queries(576)
    rc, n = hp.hp_latent_decode_workspace_bytes(b.desc, 512, b.T, 16)
    ws, alone = (torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda") for _ in range(2))
    pools = [b.pool, b.pool * 0.5, b.pool.flip(1).contiguous()]
    layers = [b.desc] + [hp.PagedDesc(p, *b.desc._keep[1:4], num_pages=b.desc.c.num_pages, page_size=16, num_heads=1,
                                      head_dim=576, dtype="bf16", index_type=0, flags=cores(hp, kernel)) for p in pools[1:]]
    outs = [torch.full((b.T, 16, 512), 9.0, dtype=b.dt, device="cuda") for _ in layers]
    want = [torch.full((b.T, 16, 512), 9.0, dtype=b.dt, device="cuda") for _ in layers]
    for _ in range(2):
        for i, d in enumerate(layers):
            call = hp.hp_latent_decode_planned if i else hp.hp_latent_decode
            assert call(d, 512, q, b.q_ptr, b.T, 16, 0.07, outs[i], ws, b.status) == 0
        for d, o in zip(layers, want):
            assert hp.hp_latent_decode(d, 512, q, b.q_ptr, b.T, 16, 0.07, o, alone, b.status) == 0
        torch.cuda.synchronize()
        assert b.status.item() == 0
        for x, y in zip(outs, want):
            assert torch.equal(x.view(torch.int16), y.view(torch.int16))
        check = host(outs[0])
        for s, t, k in b.seen():
            if t % 17 == 0:
                c = b.rows[s][:k]
                o, tol = ref.attention_row(b.q[t, 3].double().numpy(), c, c[:, :512], 0.07, "bf16")
                assert (np.abs(check[t, 3] - o) <= tol).all()
        b.q = torch.randn(b.q.shape).to(b.dt)
        q.copy_(b.q)


# ---------------------------------------------------------------- order, bounds, threads
def small_step(hp, S, H, seed, form_q):
    """Buffers and calls of one step over a latent cache: tables, append, decode and prompts' form."""
    import torch
    P, W, R, dt = 16, 576, 512, torch.bfloat16
    rng = np.random.default_rng(seed)
    lens = rng.integers(0, 150, S)
    new = np.full(S, form_q)
    s = make_step(hp, lens, new, -(-lens // P), P, 0, pad=0)
    n = int(np.maximum(-(-lens // P), -(-(lens + new) // P)).sum())
    s["o"]["table_out"] = s["o"]["table_out"][:n].clone()
    s["d"] = hp.step_desc(block_table=s["d"].keep[0], seq_ptr=s["d"].keep[1], seq_lens=s["d"].keep[2],
                          new_lens=s["d"].keep[3], free_pages=s["d"].keep[4], page_size=P, index_type=0, **s["o"])
    T, pages = int(new.sum()), len(s["table"]) + len(s["free"])
    x = dict(pool=torch.zeros((pages, P, W), dtype=dt, device="cuda"), kv=torch.zeros((T, W), dtype=dt, device="cuda"),
             q=torch.zeros((T, H, W), dtype=dt, device="cuda"), qp=torch.zeros((T, H, 192), dtype=dt, device="cuda"),
             out=torch.zeros((T, H, R), dtype=dt, device="cuda"), outp=torch.zeros((T, H, 128), dtype=dt, device="cuda"))
    cs = dev(ref.cos_sin(200, 64))
    rope = hp.rope_desc(cos_sin=cs, sections=(32,), positions=s["o"]["positions"])
    ld = hp.latent_desc(latent=x["kv"][:, :R], k_rope=x["kv"][:, R:], q_rope=x["q"][:, :, R:], q_out=x["q"][:, :, R:],
                        latent_weight=torch.ones(R, dtype=dt, device="cuda"), dtype="bf16", slot_map=s["o"]["slot_map"],
                        pool=x["pool"], num_pages=pages, page_size=P)
    pd = hp.PagedDesc(x["pool"], s["o"]["table_out"], s["o"]["seq_ptr_out"], s["o"]["lens_out"], num_pages=pages,
                      page_size=P, num_heads=1, head_dim=W, dtype="bf16", index_type=0)
    total = int((lens + new).sum())
    w = selecting_weights(H, 128, 128, R, dt, seed).cuda()
    sizes = (hp.hp_latent_decode_workspace_bytes(pd, R, T, H)[1],
             hp.hp_latent_prefill_workspace_bytes(pd, R, 128, 128, T, H, total)[1])
    wss = [torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda") for n in sizes]
    st = [status_tensor() for _ in range(4)]
    qptr = s["o"]["new_ptr_out"]
    calls = [
        lambda stream=None: hp.hp_step_tables(s["d"], s["ws"], st[0], stream),
        lambda stream=None: hp.hp_latent_append(ld, rope, st[1], stream),
        lambda stream=None: hp.hp_latent_decode(pd, R, x["q"], qptr, T, H, 0.07, x["out"], wss[0], st[2], stream),
        lambda stream=None: hp.hp_latent_prefill(pd, R, w, 128, 128, x["qp"], qptr, T, H, 0.07, x["outp"], total, wss[1],
                                                 st[3], stream),
    ]
    return x, calls, st, (s, wss, w, pd, ld, rope, cs)


@pytest.mark.parametrize("S,H,n", [(3, 4, 1), (40, 16, 2), (130, 4, 1), (20, 80, 3)])
def test_a_stream_without_waits_gives_what_waits_give(hp, S, H, n):
    """Twenty steps in a row on one stream, each input written by a kernel just before the call that
    reads it and overwritten just after: no call starts on what is not written yet, none loses what
    it still reads."""
    import torch
    x, calls, st, keep = small_step(hp, S, H, 3, n)
    rounds = 20
    inputs = [{k: torch.randn(x[k].shape, device="cuda").to(x[k].dtype) for k in ("kv", "q", "qp")} for _ in range(rounds)]
    torch.cuda.synchronize()
    results = []
    for wait in (True, False):
        got = []
        x["pool"].zero_()
        for i in range(rounds):
            for k, v in inputs[i].items():
                torch.mul(v, 1.0, out=x[k])
            for call in calls:
                assert call() == 0
                if wait:
                    torch.cuda.synchronize()
            got.append([x[k].clone() for k in ("out", "outp", "pool", "q")])
            for k in ("kv", "q", "qp", "out", "outp"):
                x[k].fill_(float("nan"))
        torch.cuda.synchronize()
        assert [t.item() for t in st] == [0] * 4
        results.append(got)
    for a, b in zip(*results):
        for y, z in zip(a, b):
            assert torch.equal(y, z) and torch.isfinite(y.float()).all()


def test_two_threads_call_at_once(hp):
    """Two host threads, a stream and buffers each: the same results as one after the other."""
    import threading

    import torch
    runs = [small_step(hp, 30, 16, 5, 1), small_step(hp, 7, 4, 6, 2)]
    for x, calls, st, keep in runs:
        for k in ("kv", "q", "qp"):
            x[k].normal_()
    torch.cuda.synchronize()
    start = [{k: v.clone() for k, v in x.items()} for x, *_ in runs]
    want = []
    for x, calls, st, keep in runs:
        for call in calls:
            assert call() == 0
        torch.cuda.synchronize()
        want.append({k: v.clone() for k, v in x.items()})
    errors = []

    def work(i):
        x, calls, st, keep = runs[i]
        stream = torch.cuda.Stream()
        try:
            for _ in range(30):
                with torch.cuda.stream(stream):
                    for k, v in start[i].items():
                        x[k].copy_(v)
                    assert [call(stream) for call in calls] == [0] * 4
                stream.synchronize()
                assert [t.item() for t in st] == [0] * 4
                for k, v in want[i].items():
                    assert torch.equal(x[k], v), k
        except BaseException as e:  # noqa: BLE001
            errors.append((i, e))
    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors


@pytest.mark.parametrize("kernel", ["cuda_cores", "default"])
def test_nothing_is_written_past_a_buffer(hp, kernel):
    """Workspaces of exactly the size asked for and outputs of exactly the rows, between guards."""
    import torch
    from conftest import guarded, guards_intact
    for lens, nq, H in ((A([300, 0, 70]), A([3, 2, 1]), 100), (A([9000]), A([1]), 16), (np.full(200, 60), np.full(200, 2), 4),
                        (A([257, 1]), A([257, 1]), 3)):
        b = Latent(hp, lens, nq, H, 512, 576, 16, "bf16", seed=9, flags=cores(hp, kernel))
        w = selecting_weights(H, 128, 128, 512, b.dt, 3).cuda()
        kv = int(lens.sum())
        for form, width, dv in (("decode", 576, 512), ("prefill", 192, 128)):
            q = b.queries(width)
            n = (hp.hp_latent_decode_workspace_bytes(b.desc, 512, b.T, H) if form == "decode" else
                 hp.hp_latent_prefill_workspace_bytes(b.desc, 512, 128, 128, b.T, H, kv))[1]
            wbuf, ws = guarded(n)
            obuf, out = guarded(b.T * H * dv * 2)
            o = out.view(b.dt).view(b.T, H, dv)
            if form == "decode":
                rc = hp.hp_latent_decode(b.desc, 512, q, b.q_ptr, b.T, H, 0.07, o, ws, b.status)
            else:
                rc = hp.hp_latent_prefill(b.desc, 512, w, 128, 128, q, b.q_ptr, b.T, H, 0.07, o, kv, ws, b.status)
            torch.cuda.synchronize()
            assert rc == 0 and b.status.item() == 0
            assert guards_intact(wbuf, n) and guards_intact(obuf, b.T * H * dv * 2)
            assert torch.isfinite(o.float()).all()


def test_large_steps_in_a_graph(hp):
    """Tables of 1,500 sequences and appends that report in both ways, captured together and replayed on
    other lengths and rows."""
    import torch
    P, dt = 16, torch.bfloat16
    rng = np.random.default_rng(2)
    S = 1500
    lens, new = rng.integers(0, 100, S), rng.integers(0, 5, S)
    s = make_step(hp, lens, new, np.full(S, 8), P, 0, pad=1000)  # slices that need not grow
    T, pages = s["o"]["slot_map"].numel(), len(s["table"]) + len(s["free"])
    cs = dev(ref.cos_sin(300, 128))
    st = [status_tensor() for _ in range(2)]
    kv = torch.zeros((T, 576), dtype=dt, device="cuda")
    x = torch.zeros((T, 48 * 128), dtype=dt, device="cuda")
    pool = torch.zeros((pages, P, 576), dtype=dt, device="cuda")
    kp, vp = (torch.zeros((pages, P, 8, 128), dtype=dt, device="cuda") for _ in range(2))
    cs64 = dev(ref.cos_sin(300, 64))
    ld = hp.latent_desc(latent=kv[:, :512], k_rope=kv[:, 512:], dtype="bf16", slot_map=s["o"]["slot_map"], pool=pool,
                        num_pages=pages, page_size=P)
    qd = hp.qk_desc(q=x[:, :4096], k=x[:, 4096:5120], v=x[:, 5120:], q_out=x[:, :4096], num_q_heads=32, num_kv_heads=8,
                    head_dim=128, dtype="bf16", slot_map=s["o"]["slot_map"], k_pool=kp, v_pool=vp, num_pages=pages,
                    page_size=P)
    r64 = hp.rope_desc(cos_sin=cs64, sections=(32,), positions=s["o"]["positions"])
    r128 = hp.rope_desc(cos_sin=cs, sections=(64,), positions=s["o"]["positions"])

    def calls():
        assert hp.hp_step_tables(s["d"], s["ws"], s["status"]) == 0
        assert hp.hp_latent_append(ld, r64, st[0]) == 0
        assert hp.hp_qk_norm_rope_append(qd, r128, st[1]) == 0
    calls()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls()
    for seed in (1, 2):
        r = np.random.default_rng(seed)
        lens, new = r.integers(0, 100, S), r.integers(0, 5, S)
        s["d"].keep[2].copy_(torch.from_numpy(lens.astype(np.int32)))
        s["d"].keep[3].copy_(torch.from_numpy(new.astype(np.int32)))
        kv.normal_()
        rows = torch.randn(x.shape).to(dt).cuda()
        results = []
        for run in (graph.replay, calls):
            x.copy_(rows)
            for t in (pool, kp, vp):
                t.fill_(3.0)
            run()
            torch.cuda.synchronize()
            assert [t.item() for t in (s["status"], *st)] == [0] * 3
            results.append([t.clone() for t in (pool, kp, vp, x, *s["o"].values())])
        for a, c in zip(*results):
            assert torch.equal(a, c)
        n = int(new.sum())
        want = ref.step_tables(lens, new, s["sp"], s["table"], s["free"], P)
        assert s["o"]["slot_map"].cpu().tolist() == want[4] + [-1] * (T - n)
        at = torch.tensor(want[4], device="cuda")
        assert torch.equal(pool.view(-1, 576)[at][:, :512], kv[:n, :512])
        assert torch.equal(vp.view(-1, 1024)[at], rows[:n, 5120:]) and torch.equal(x[n:], rows[n:])


@pytest.mark.parametrize("S", [2, 130])
def test_planned_calls_behind_a_batch_that_fails(hp, S):
    """A whole call whose batch breaks a rule leaves a plan that says so: a planned call behind it writes
    nothing and keeps the code."""
    import torch
    b = Latent(hp, np.full(S, 40), np.full(S, 1), 16, 512, 576, 16, "bf16", seed=S)
    q = b.queries(576)
    ws = torch.full((hp.hp_latent_decode_workspace_bytes(b.desc, 512, b.T, 16)[1],), 0xFF, dtype=torch.uint8, device="cuda")
    out = torch.full((b.T, 16, 512), 9.0, dtype=b.dt, device="cuda")
    good = b.desc._keep[1].clone()
    b.desc._keep[1][3 * S - 1] = 10 ** 6
    assert hp.hp_latent_decode(b.desc, 512, q, b.q_ptr, b.T, 16, 0.07, out, ws, b.status) == 0
    b.desc._keep[1].copy_(good)
    assert hp.hp_latent_decode_planned(b.desc, 512, q, b.q_ptr, b.T, 16, 0.07, out, ws, b.status) == 0
    torch.cuda.synchronize()
    assert hp.status_name(b.status.item()) == "HP_ERR_PAGE_ID" and (out == 9).all()
