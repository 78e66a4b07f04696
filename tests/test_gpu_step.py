"""GPU parity of the serving-step operators against plain 64-bit implementations (step_ref.py,
where the bounds are derived)."""
import numpy as np
import pytest

import step_ref as ref
from helpers import index_tensor

pytestmark = pytest.mark.gpu

IDX = {0: np.uint32, 1: np.uint64}


def dev(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def host(t):
    return t.double().cpu().numpy()


def status_tensor():
    import torch
    return torch.full((1,), 77, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------------- step tables
def make_step(hp, lens, new, have, P, it, spare=3, pad=4, free=None):
    import torch
    rng = np.random.default_rng(len(lens) + P)
    need = np.maximum(have, -(-(lens + new) // P))
    pages = rng.permutation(int(need.sum()) + spare).astype(IDX[it])
    n = int(have.sum())
    s = dict(lens=lens, new=new, sp=np.concatenate([[0], np.cumsum(have)]).astype(IDX[it]),
             table=pages[:n], free=pages[n:] if free is None else pages[n:][:free], P=P)
    tt = torch.int32 if it == 0 else torch.int64
    total, T, S = int(need.sum()), int(new.sum()), len(lens)

    def full(k, t=tt):
        return torch.full((k,), -9, dtype=t, device="cuda")
    s["o"] = dict(table_out=full(total + 2), seq_ptr_out=full(S + 1), lens_out=full(S),
                  new_ptr_out=full(S + 1), slot_map=full(T + pad, torch.int64),
                  positions=full(T + pad), totals=full(3, torch.int64))
    s["d"] = hp.step_desc(block_table=index_tensor(s["table"], "cuda"),
                          seq_ptr=index_tensor(s["sp"], "cuda"),
                          seq_lens=index_tensor(lens.astype(IDX[it]), "cuda"),
                          new_lens=index_tensor(new.astype(IDX[it]), "cuda"),
                          free_pages=index_tensor(s["free"], "cuda"), page_size=P, index_type=it,
                          **s["o"])
    rc, n = hp.hp_step_tables_workspace_bytes(S)
    s["ws"] = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")
    s["status"] = status_tensor()
    return s


def check_step(hp, s):
    import torch
    torch.cuda.synchronize()
    assert s["status"].item() == 0
    want = ref.step_tables(s["lens"], s["new"], s["sp"], s["table"], s["free"], s["P"])
    got = {k: v.cpu().numpy() for k, v in s["o"].items()}
    n, T = len(want[0]), len(want[4])
    assert got["table_out"][:n].tolist() == want[0] and (got["table_out"][n:] == -9).all()
    assert got["seq_ptr_out"].tolist() == want[1] and got["lens_out"].tolist() == want[2]
    assert got["new_ptr_out"].tolist() == want[3]
    assert got["slot_map"][:T].tolist() == want[4] and (got["slot_map"][T:] == -1).all()
    assert got["positions"][:T].tolist() == want[5] and (got["positions"][T:] == 0).all()
    assert got["totals"].tolist() == [n, T, want[6]]


@pytest.mark.parametrize("it", [0, 1])
@pytest.mark.parametrize("S,P,hi,prompts", [
    (1, 16, 0, True), (1, 1, 5, False), (2, 5, 40, True), (33, 16, 300, True), (700, 3, 60, True),
    (1024, 16, 100, False), (1025, 16, 100, True), (5000, 64, 500, False), (3, 16, 40000, True),
    (2048, 16, 300, True), (4097, 1, 9, True), (300000, 16, 3, False),
])
def test_step_tables(hp, S, P, hi, prompts, it):
    rng = np.random.default_rng(S * 7 + P)
    lens = rng.integers(0, hi + 1, S)
    new = rng.integers(0, 3, S)
    if prompts:
        new[rng.random(S) < 0.3] = hi + 7
    have = -(-lens // P) + (rng.random(S) < 0.2) * 2
    s = make_step(hp, lens, new, have, P, it)
    for _ in range(2):  # a second call on the same workspace gives the same tables
        assert hp.hp_step_tables(s["d"], s["ws"], s["status"]) == 0
        check_step(hp, s)


def test_step_tables_without_sequences_or_tokens(hp):
    z = np.zeros(0, np.int64)
    s = make_step(hp, z, z, z, 16, 0)
    assert hp.hp_step_tables(s["d"], s["ws"], s["status"]) == 0
    check_step(hp, s)
    s = make_step(hp, np.array([5, 0, 31]), np.zeros(3, np.int64), np.array([1, 0, 3]), 16, 1, pad=0)
    assert hp.hp_step_tables(s["d"], s["ws"], s["status"]) == 0
    check_step(hp, s)


@pytest.mark.parametrize("what,name", [
    ("start", "SEQ_PTR_START"), ("order", "SEQ_PTR_ORDER"), ("end", "SEQ_PTR_END"), ("len", "LEN"),
    ("grow", "LEN"), ("free", "CAPACITY"), ("cap", "OUT_SIZE"), ("tokens", "OUT_SIZE"),
])
def test_step_tables_verdicts(hp, what, name):
    """A rule that fails names itself, and nothing else is written."""
    import torch
    lens, new = np.array([20, 3, 40]), np.array([1, 30, 2])
    s = make_step(hp, lens, new, np.array([2, 1, 3]), 16, 0, free=1 if what == "free" else None)  # two pages are taken
    d = s["d"]
    sp, ln, nw = d.keep[1], d.keep[2], d.keep[3]
    if what == "start":
        sp[0] = 1
    elif what == "order":
        sp[1] = 5
    elif what == "end":
        d.table_len -= 1
    elif what == "len":
        ln[1] = 17
    elif what == "grow":
        nw[2] = -20  # 2^32 - 20 more tokens
    elif what == "cap":
        d.table_cap = 7
    elif what == "tokens":
        d.token_cap = 32
    assert hp.hp_step_tables(d, s["ws"], s["status"]) == 0
    torch.cuda.synchronize()
    assert hp.status_name(s["status"].item()) == "HP_ERR_" + name
    for t in s["o"].values():
        assert (t == -9).all()


# ------------------------------------------------- norm + rotation + append, K/V heads
def rope_inputs(hp, rng, T, rot, sections, inter, it=0, max_pos=50000):
    table = ref.cos_sin(max_pos, rot)
    pos = rng.integers(0, max_pos, (len(sections), T))
    r = hp.rope_desc(cos_sin=dev(table), positions=index_tensor(pos.astype(IDX[it]), "cuda"),
                     sections=sections, interleaved=inter, index_type=it)
    return r, ref.angles(table, pos, sections)


def slots_for(rng, T, slots):
    slot = rng.permutation(slots)[:T].astype(np.int64)
    slot[rng.random(T) < 0.1] = -1
    return slot


@pytest.mark.parametrize("dtype,D,rot,sections,inter,norm,T,hq,hkv", [
    ("bf16", 128, 128, (64,), False, "qk", 37, 32, 8), ("f16", 128, 128, (64,), True, "qk", 5, 8, 8),
    ("bf16", 128, 64, (32,), False, "qk", 9, 4, 1), ("f16", 128, 64, (8, 12, 12), True, "k", 9, 6, 2),
    ("bf16", 128, 128, (16, 24, 24), False, "qk", 70, 7, 7), ("f32", 128, 128, (64,), False, "qk", 11, 3, 2),
    ("f32", 80, 80, (10, 10, 10, 10), True, "", 6, 5, 5), ("bf16", 80, 80, (40,), False, "q", 33, 5, 1),
    ("f16", 80, 32, (0, 16), False, "qk", 3, 2, 2), ("bf16", 64, 64, (32,), False, "qk", 300, 16, 2),
    ("bf16", 256, 256, (128,), False, "qk", 21, 4, 2), ("f16", 256, 64, (3, 29), True, "qk", 2, 1, 1),
    ("bf16", 8, 0, (), False, "qk", 5, 3, 1), ("f32", 24, 16, (8,), False, "qk", 4, 0, 3),
    ("bf16", 128, 128, (64,), False, "qk", 1, 32, 8), ("bf16", 128, 128, (64,), False, "qk", 3001, 12, 4),
])
def test_qk_norm_rope_append(hp, dtype, D, rot, sections, inter, norm, T, hq, hkv):
    import torch
    rng = np.random.default_rng(D + rot + T + hq)
    dt, P = ref.torch_dtype(dtype), 16
    pages = (T + 40) // P + 2
    g = torch.Generator().manual_seed(T + D)
    # one fused projection, each row followed by 16 elements of something else
    width = (hq + 2 * hkv) * D + 16
    qkv = (torch.randn((T, width), generator=g) * 3).to(dt)
    x = qkv.double().numpy()
    w = {k: (1 + 0.2 * torch.randn(D, generator=g)).to(dt) if k in norm else None for k in "qk"}
    pools = [torch.randn((pages, P, hkv, D), generator=g).to(dt) for _ in "kv"]
    slot = slots_for(rng, T, pages * P)
    rope, (cos, sin) = rope_inputs(hp, rng, T, rot, sections, inter, it=T % 2) if rot else (None, (None, None))
    qd, kp, vp = qkv.cuda(), pools[0].cuda(), pools[1].cuda()
    q_out = torch.full((T, hq * D + 8), 5.0, dtype=dt, device="cuda")
    q, k, v, _ = qd.split([hq * D, hkv * D, hkv * D, 16], 1)
    d = hp.qk_desc(q=q if hq else None, k=k, v=v, q_out=q_out if hq else None, num_q_heads=hq,
                   num_kv_heads=hkv, head_dim=D, dtype=dtype, slot_map=dev(slot), k_pool=kp,
                   v_pool=vp, num_pages=pages, page_size=P,
                   q_weight=None if w["q"] is None else w["q"].cuda(),
                   k_weight=None if w["k"] is None else w["k"].cuda())
    st = status_tensor()
    assert hp.hp_qk_norm_rope_append(d, rope, st) == 0
    torch.cuda.synchronize()
    assert st.item() == 0
    live = slot >= 0
    heads = {}
    for name, a, n in (("q", 0, hq), ("k", hq * D, hkv)):
        h = x[:, a:a + n * D].reshape(T, n, D)
        h = ref.norm(h, None if w[name] is None else w[name].double().numpy(), 1e-6)
        y = ref.rotate(h, cos, sin, inter) if rot else h
        heads[name] = y, ref.rope_bound(y, h, dtype)
    got = host(q_out)[:, :hq * D].reshape(T, hq, D)
    y, tol = heads["q"]
    assert (np.abs(got - y) <= tol)[live].all()
    assert (got[~live] == 5).all() and (host(q_out)[:, hq * D:] == 5).all()
    want_k, want_v = pools[0].double().numpy(), pools[1].double().numpy()
    gk, gv = host(kp).reshape(-1, hkv, D), host(vp).reshape(-1, hkv, D)
    y, tol = heads["k"]
    assert (np.abs(gk[slot[live]] - y[live]) <= tol[live]).all()
    assert np.array_equal(gv[slot[live]], x[live][:, (hq + hkv) * D:(hq + 2 * hkv) * D].reshape(-1, hkv, D))
    rest = np.ones(pages * P, bool)
    rest[slot[live]] = False
    assert np.array_equal(gk[rest], want_k.reshape(-1, hkv, D)[rest])
    assert np.array_equal(gv[rest], want_v.reshape(-1, hkv, D)[rest])
    assert np.array_equal(host(qd), x)  # the inputs are left as they were
    if hq and norm == "qk":  # in place: q_out is q
        d.q_out, d.q_out_stride = d.q, d.q_stride
        assert hp.hp_qk_norm_rope_append(d, rope, st) == 0
        torch.cuda.synchronize()
        again = host(qd)[:, :hq * D].reshape(T, hq, D)
        assert np.array_equal(again[live], got[live])


def test_append_skips_what_it_cannot_place(hp):
    """A slot past the pool and a position past the table: the token is skipped, the first
    one's code reported, the others stored; infinities outside the rotated part stay."""
    import torch
    T, D = 40, 128
    rng = np.random.default_rng(1)
    x = torch.randn((T, 3 * D)).to(torch.bfloat16)
    x[3, D + 100] = float("inf")
    slot = np.arange(T, dtype=np.int64)
    rope, _ = rope_inputs(hp, rng, T, 64, (32,), False)
    for bad_slot, bad_pos, code in (((7, 9), (), "PAGE_ID"), ((9,), (8,), "LEN"), ((), (39,), "LEN")):
        kp = torch.zeros((3, 16, 1, D), dtype=torch.bfloat16, device="cuda")
        vp, sl = kp.clone(), slot.copy()
        for b in bad_slot:
            sl[b] = 48
        pos = rope.keep[1].clone()
        for b in bad_pos:
            pos[0, b] = 50000
        r = hp.rope_desc(cos_sin=rope.keep[0], positions=pos, sections=(32,))
        xd, q_out = x.cuda(), torch.full((T, D), 7.0, dtype=torch.bfloat16, device="cuda")
        d = hp.qk_desc(q=xd[:, :D], k=xd[:, D:2 * D], v=xd[:, 2 * D:], q_out=q_out, num_q_heads=1,
                       num_kv_heads=1, head_dim=D, dtype="bf16", slot_map=dev(sl), k_pool=kp,
                       v_pool=vp, num_pages=3, page_size=16)
        st = status_tensor()
        assert hp.hp_qk_norm_rope_append(d, r, st) == 0
        torch.cuda.synchronize()
        assert hp.status_name(st.item()) == "HP_ERR_" + code
        skipped = set(bad_slot) | set(bad_pos)
        for t in range(T):
            assert bool((q_out[t] == 7).all()) == (t in skipped)
            assert bool((vp.view(-1, D)[t] == 0).all()) == (t in skipped)
        assert torch.isinf(kp.view(-1, D)[3, 100]) and not torch.isnan(kp).any()


@pytest.mark.parametrize("dtype,R,rot,inter,norm,T,H", [
    ("bf16", 512, 64, True, True, 1, 128), ("bf16", 512, 64, False, True, 41, 16),
    ("f16", 512, 64, True, True, 700, 5), ("f32", 256, 32, False, True, 9, 3),
    ("bf16", 1024, 128, True, True, 3, 2), ("f16", 8, 16, False, True, 33, 1),
    ("bf16", 320, 64, True, False, 12, 7), ("f16", 136, 256, False, True, 4, 3),
    ("bf16", 512, 64, True, True, 6, 0), ("bf16", 512, 64, True, True, 4001, 8),
])
def test_latent_append(hp, dtype, R, rot, inter, norm, T, H):
    import torch
    rng = np.random.default_rng(R + rot + T)
    dt, P = ref.torch_dtype(dtype), 8
    pages = (T + 20) // P + 2
    g = torch.Generator().manual_seed(R + T)
    kv = (torch.randn((T, R + rot), generator=g) * 4).to(dt)
    q = torch.randn((T, H, 128 + rot), generator=g).to(dt)
    w = (1 + 0.2 * torch.randn(R, generator=g)).to(dt) if norm else None
    pool0 = torch.randn((pages, P, R + rot), generator=g).to(dt)
    slot = slots_for(rng, T, pages * P)
    half = rot // 2
    rope, (cos, sin) = rope_inputs(hp, rng, T, rot, (half - 3, 3) if T % 2 else (half,), inter)
    kd, qd, pool = kv.cuda(), q.cuda(), pool0.cuda()
    full = torch.full((T, H, R + rot), 5.0, dtype=dt, device="cuda")  # absorbed queries
    d = hp.latent_desc(latent=kd[:, :R], k_rope=kd[:, R:], q_rope=qd[:, :, 128:] if H else None,
                       q_out=full[:, :, R:] if H else None, latent_weight=None if w is None else w.cuda(),
                       dtype=dtype, slot_map=dev(slot), pool=pool, num_pages=pages, page_size=P)
    st = status_tensor()
    assert hp.hp_latent_append(d, rope, st) == 0
    torch.cuda.synchronize()
    assert st.item() == 0
    live = slot >= 0
    x = kv.double().numpy()
    c = ref.norm(x[:, :R], None if w is None else w.double().numpy(), 1e-6)
    k = ref.rotate(x[:, None, R:], cos, sin, inter)[:, 0]
    got = host(pool).reshape(-1, R + rot)
    tol_c = ref.rope_bound(c, c, dtype)
    tol_k = ref.rope_bound(k, x[:, R:], dtype)
    assert (np.abs(got[slot[live], :R] - c[live]) <= tol_c[live]).all()
    assert (np.abs(got[slot[live], R:] - k[live]) <= tol_k[live]).all()
    rest = np.ones(pages * P, bool)
    rest[slot[live]] = False
    assert np.array_equal(got[rest], pool0.double().numpy().reshape(-1, R + rot)[rest])
    if H:
        xq = q.double().numpy()[:, :, 128:]
        y = ref.rotate(xq, cos, sin, inter)
        gq = host(full)
        assert (np.abs(gq[:, :, R:] - y) <= ref.rope_bound(y, xq, dtype))[live].all()
        assert (gq[~live] == 5).all() and (gq[:, :, :R] == 5).all()


# -------------------------------------------------------------------- latent attention
class Latent:
    """A batch over a paged latent cache; the slots no sequence has filled hold NaN."""

    def __init__(self, hp, lens, nq, H, R, W, P, dtype, it=0, seed=0, flags=0, rows_behind=0,
                 qscale=1.0, with_ptr=True):
        import torch
        g = torch.Generator().manual_seed(seed)
        rng = np.random.default_rng(seed)
        self.hp, self.lens, self.nq, self.H, self.R, self.W, self.dtype = hp, lens, nq, H, R, W, dtype
        self.dt = ref.torch_dtype(dtype)
        need = -(-lens // P)
        pages = int(need.sum()) + 2
        table = rng.permutation(pages)[:int(need.sum())].astype(IDX[it])
        sp = np.concatenate([[0], np.cumsum(need)]).astype(IDX[it])
        pool = torch.full((pages * P, W), float("nan")).to(self.dt)
        self.rows = []
        for s, n in enumerate(lens):
            t = np.arange(n)
            at = table[int(sp[s]) + t // P].astype(np.int64) * P + t % P
            r = torch.randn((int(n), W), generator=g).to(self.dt)
            pool[torch.from_numpy(at)] = r
            self.rows.append(r.double().numpy())
        self.pool = pool.cuda()
        self.T = int(nq.sum()) + rows_behind
        self.q_ptr_host = np.concatenate([[0], np.cumsum(nq)])
        self.q_ptr = index_tensor(self.q_ptr_host.astype(IDX[it]), "cuda") if with_ptr else None
        self.g, self.qscale = g, qscale
        self.desc = hp.PagedDesc(self.pool, index_tensor(table, "cuda") if len(table) else None,
                                 index_tensor(sp, "cuda"),
                                 index_tensor(lens.astype(IDX[it]), "cuda"), num_pages=pages,
                                 page_size=P, num_heads=1, head_dim=W, dtype=dtype, index_type=it,
                                 flags=flags)
        self.status = status_tensor()

    def queries(self, width):
        import torch
        self.q = (torch.randn((self.T, self.H, width), generator=self.g) * self.qscale).to(self.dt)
        return self.q.cuda()

    def seen(self):
        """(sequence, query row, tokens it sees) of every query."""
        for s, n in enumerate(self.nq):
            for i in range(n):
                yield s, int(self.q_ptr_host[s]) + i, max(0, int(self.lens[s]) - int(n) + 1 + i)


def run_decode(b, scale):
    import torch
    hp = b.hp
    q = b.queries(b.W)
    rc, n = hp.hp_latent_decode_workspace_bytes(b.desc, b.R, b.T, b.H)
    assert rc == 0
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")
    outs = []
    for _ in range(2):
        out = torch.full((b.T, b.H, b.R), 9.0, dtype=b.dt, device="cuda")
        rc = hp.hp_latent_decode(b.desc, b.R, q, b.q_ptr, b.T, b.H, scale, out, ws, b.status)
        torch.cuda.synchronize()
        assert hp.status_name(rc) == "HP_OK" and hp.status_name(b.status.item()) == "HP_OK"
        outs.append(out)
    assert torch.equal(outs[0].view(torch.int16), outs[1].view(torch.int16))  # bit for bit
    return host(outs[0])


def check_decode(b, got, scale, rows=None):
    q = b.q.double().numpy()
    for s, t, n in b.seen():
        if rows is not None and t not in rows:
            continue
        c = b.rows[s][:n]
        for h in range(b.H):
            o, tol = ref.attention_row(q[t, h], c, c[:, :b.R], scale, b.dtype)
            assert np.isfinite(got[t, h]).all(), (s, t, h)
            err = np.abs(got[t, h] - o)
            assert (err <= tol).all(), (s, t, h, float((err / np.maximum(tol, 1e-30)).max()))
    assert (got[int(b.q_ptr_host[-1]):] == 9).all()  # rows behind the last sequence


def cores(hp, name):
    return hp.ATTN_CUDA_CORES if name == "cuda_cores" else 0


A = np.array


@pytest.mark.parametrize("kernel", ["cuda_cores", "default"])
@pytest.mark.parametrize("dtype,lens,nq,H,P", [
    ("bf16", A([1]), A([1]), 1, 16), ("bf16", A([64, 65, 63]), A([1, 1, 1]), 16, 16),
    ("f16", A([0, 1, 2, 130, 0]), A([1, 1, 1, 1, 1]), 8, 64),
    ("bf16", A([300, 17, 129]), A([2, 3, 1]), 24, 8), ("f16", A([777]), A([4]), 64, 32),
    ("bf16", A([200, 128, 5]), A([1, 1, 1]), 128, 64), ("bf16", A([3, 0, 700]), A([5, 2, 7]), 40, 128),
    ("f16", A([130, 259]), A([1, 2]), 100, 16), ("bf16", A([9000]), A([1]), 16, 64),
    ("f16", A([2500, 3, 1100]), A([1, 1, 1]), 65, 16), ("bf16", A([190, 100]), A([0, 3]), 128, 192),
    ("bf16", A([64] * 200), A([1] * 200), 3, 64), ("f16", A([5000, 4097]), A([2, 1]), 128, 16),
])
def test_latent_decode(hp, kernel, dtype, lens, nq, H, P):
    b = Latent(hp, lens, nq, H, 512, 576, P, dtype, it=H % 2, seed=H + P, flags=cores(hp, kernel),
               rows_behind=2 if H % 3 else 0)
    scale = 1 / np.sqrt(192)
    check_decode(b, run_decode(b, scale), scale)


@pytest.mark.parametrize("dtype,R,W,P,H,lens", [
    ("bf16", 512, 576, 1, 4, A([70, 3])), ("f16", 512, 576, 5, 7, A([200, 64])),
    ("bf16", 64, 72, 16, 3, A([100, 0, 33])), ("f16", 256, 320, 16, 16, A([150])),
    ("bf16", 320, 352, 24, 5, A([80, 81])), ("f16", 512, 520, 7, 2, A([129])),
])
def test_latent_decode_other_shapes(hp, dtype, R, W, P, H, lens):
    nq = np.arange(1, len(lens) + 1)
    b = Latent(hp, lens, nq, H, R, W, P, dtype, it=P % 2, seed=R + W)
    check_decode(b, run_decode(b, 0.1), 0.1)


@pytest.mark.parametrize("kernel", ["cuda_cores", "default"])
def test_latent_decode_one_query_each_without_offsets(hp, kernel):
    lens = A([40, 0, 333])
    b = Latent(hp, lens, np.ones(3, np.int64), 16, 512, 576, 16, "bf16", flags=cores(hp, kernel),
               with_ptr=False)
    check_decode(b, run_decode(b, 0.07), 0.07)


@pytest.mark.parametrize("kernel", ["cuda_cores", "default"])
def test_latent_decode_peaked_and_rising_scores(hp, kernel):
    """Scores of a few hundred: one token carries the weight, and the running maximum moves
    late and often."""
    b = Latent(hp, A([1500, 90]), A([1, 2]), 32, 512, 576, 16, "f16", seed=3, qscale=6.0,
               flags=cores(hp, kernel))
    check_decode(b, run_decode(b, 1.0), 1.0)


@pytest.mark.parametrize("kernel", ["cuda_cores", "default"])
def test_latent_decode_long_cache(hp, kernel):
    """One long sequence over the whole GPU, sampled rows; a batch of many next to it."""
    b = Latent(hp, A([70001]), A([2]), 32, 512, 576, 64, "bf16", seed=5, flags=cores(hp, kernel))
    check_decode(b, run_decode(b, 0.07), 0.07)
    lens = np.random.default_rng(2).integers(0, 900, 300)
    b = Latent(hp, lens, np.ones(300, np.int64), 128, 512, 576, 64, "bf16", seed=6,
               flags=cores(hp, kernel))
    got = run_decode(b, 0.07)
    check_decode(b, got, 0.07, rows={0, 7, 150, 299})


def test_latent_decode_many_empty_sequences(hp):
    """3000 sequences, most of them empty: every query of an empty one gets zeros, whichever CTAs
    have work of their own."""
    lens = np.where(np.random.default_rng(5).random(3000) < 0.01, 70, 0)
    for nq in (np.ones(3000, np.int64), np.random.default_rng(6).integers(0, 3, 3000)):
        b = Latent(hp, lens, nq, 4, 512, 576, 16, "bf16", seed=7)
        check_decode(b, run_decode(b, 0.07), 0.07)


def test_latent_decode_verdicts(hp):
    import torch
    for what, name in (("page", "PAGE_ID"), ("len", "LEN"), ("qstart", "NEW_PTR_START"),
                       ("qorder", "NEW_PTR_ORDER"), ("qend", "NEW_PTR_END")):
        b = Latent(hp, A([40, 20]), A([1, 1]), 16, 512, 576, 16, "bf16")
        q = b.queries(576)
        T = b.T
        if what == "page":
            b.desc._keep[1][1] = 1000
        elif what == "len":
            b.desc._keep[3][1] = 33
        elif what == "qstart":
            b.q_ptr[0] = 1
        elif what == "qorder":
            b.q_ptr[1] = 3
        else:
            T = 1
        rc, n = hp.hp_latent_decode_workspace_bytes(b.desc, 512, T, 16)
        ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
        out = torch.full((b.T, 16, 512), 9.0, dtype=b.dt, device="cuda")
        assert hp.hp_latent_decode(b.desc, 512, q, b.q_ptr, T, 16, 1.0, out, ws, b.status) == 0
        torch.cuda.synchronize()
        assert hp.status_name(b.status.item()) == "HP_ERR_" + name and (out == 9).all()


def run_prefill(b, Dn, Dv, w, scale, kv_tokens=None):
    import torch
    hp = b.hp
    q = b.queries(Dn + b.W - b.R)
    kv = int(b.lens.sum()) if kv_tokens is None else kv_tokens
    rc, n = hp.hp_latent_prefill_workspace_bytes(b.desc, b.R, Dn, Dv, b.T, b.H, kv)
    assert rc == 0
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")  # NaN in every type
    out = torch.full((b.T, b.H, Dv), 9.0, dtype=b.dt, device="cuda")
    rc = hp.hp_latent_prefill(b.desc, b.R, w.cuda(), Dn, Dv, q, b.q_ptr, b.T, b.H, scale, out, kv,
                              ws, b.status)
    torch.cuda.synchronize()
    assert hp.status_name(rc) == "HP_OK" and hp.status_name(b.status.item()) == "HP_OK"
    return host(out)


def check_prefill(b, got, Dn, Dv, w, scale, exact_kv, sample=None):
    """exact_kv: the expanded keys and values are exact in the type (their error terms are 0)."""
    q, wd = b.q.double().numpy(), w.double().numpy()
    u = 0.0 if exact_kv else ref.U[b.dtype]
    cache = {}
    for s, t, n in b.seen():
        if sample is not None and t not in sample:
            continue
        for h in range(b.H):
            if (s, h) not in cache:
                c = b.rows[s]
                kv = c[:, :b.R] @ wd[h].T
                big = 0.0 if exact_kv else b.R * 2.0 ** -23 * float((np.abs(c[:, :b.R]) @ np.abs(wd[h]).T).max(initial=0))
                cache[s, h] = np.concatenate([kv[:, :Dn], c[:, b.R:]], 1), kv[:, Dn:], big
            k, v, big = cache[s, h]
            o, tol = ref.attention_row(q[t, h], k[:n], v[:n], scale, b.dtype, ds_extra=u)
            if n and not exact_kv:
                p = np.exp(k[:n] @ q[t, h] * scale - (k[:n] @ q[t, h] * scale).max())
                tol = tol + u * (p / p.sum()) @ np.abs(v[:n]) + big * (1 + 4 * abs(scale) * np.abs(q[t, h]).sum())
            err = np.abs(got[t, h] - o)
            assert np.isfinite(got[t, h]).all(), (s, t, h)
            assert (err <= tol).all(), (s, t, h, float((err / np.maximum(tol, 1e-30)).max()))
    assert (got[int(b.q_ptr_host[-1]):] == 9).all()


def selecting_weights(H, Dn, Dv, R, dt, seed):
    """w_kv whose every row picks one latent dimension (times +-1): K and V are exact."""
    import torch
    g = torch.Generator().manual_seed(seed)
    w = torch.zeros((H, Dn + Dv, R))
    pick = torch.randint(0, R, (H, Dn + Dv, 1), generator=g)
    sign = torch.randint(0, 2, (H, Dn + Dv, 1), generator=g) * 2.0 - 1
    return w.scatter_(2, pick, sign).to(dt)


PREFILL = [
    ("bf16", A([1]), A([1]), 1, 16), ("f16", A([5, 128, 129]), A([5, 128, 129]), 2, 16),
    ("bf16", A([300, 0, 17]), A([100, 3, 17]), 3, 8), ("bf16", A([260, 700]), A([257, 1]), 2, 64),
    ("f16", A([513, 64, 3]), A([300, 64, 9]), 4, 32), ("bf16", A([1100]), A([900]), 1, 5),
    ("f16", A([40] * 20), A([1] * 20), 16, 16), ("bf16", A([384, 383, 385]), A([256, 255, 257]), 2, 128),
]


@pytest.mark.parametrize("kernel", ["cuda_cores", "default"])
@pytest.mark.parametrize("dtype,lens,nq,H,P", PREFILL)
def test_latent_prefill(hp, kernel, dtype, lens, nq, H, P):
    import torch
    b = Latent(hp, lens, nq, H, 512, 576, P, dtype, it=H % 2, seed=H + P, flags=cores(hp, kernel),
               rows_behind=H % 3)
    w = selecting_weights(H, 128, 128, 512, b.dt, P)
    got = run_prefill(b, 128, 128, w, 0.07)
    check_prefill(b, got, 128, 128, w, 0.07, exact_kv=True)
    g = torch.Generator().manual_seed(P)
    w = (torch.randn((H, 256, 512), generator=g) / 512 ** 0.5).to(b.dt)
    got = run_prefill(b, 128, 128, w, 0.07, kv_tokens=int(lens.sum()) + 200)
    check_prefill(b, got, 128, 128, w, 0.07, exact_kv=False)


@pytest.mark.parametrize("dtype,R,W,Dn,Dv,H,P", [
    ("bf16", 512, 576, 64, 128, 3, 16), ("f16", 256, 288, 128, 256, 2, 16), ("bf16", 64, 72, 16, 16, 5, 3),
    ("f16", 512, 560, 192, 48, 1, 1), ("bf16", 320, 384, 256, 240, 2, 64),
])
def test_latent_prefill_other_shapes(hp, dtype, R, W, Dn, Dv, H, P):
    b = Latent(hp, A([90, 33]), A([50, 33]), H, R, W, P, dtype, seed=R + Dn)
    w = selecting_weights(H, Dn, Dv, R, b.dt, R)
    check_prefill(b, run_prefill(b, Dn, Dv, w, 0.08), Dn, Dv, w, 0.08, exact_kv=True)


@pytest.mark.parametrize("kernel", ["cuda_cores", "default"])
def test_latent_prefill_long_and_peaked(hp, kernel):
    b = Latent(hp, A([3001]), A([2900]), 2, 512, 576, 64, "bf16", seed=9, flags=cores(hp, kernel),
               qscale=5.0)
    w = selecting_weights(2, 128, 128, 512, b.dt, 4)
    got = run_prefill(b, 128, 128, w, 0.3)
    check_prefill(b, got, 128, 128, w, 0.3, exact_kv=True,
                  sample={0, 1, 127, 128, 255, 256, 1000, 2047, 2898, 2899})


def test_latent_prefill_many_heads(hp):
    """11 blocks of 128 rows x 64 heads, several tiles of the expansion per CTA: selecting weights
    (exact keys and values) and random ones, sampled queries."""
    import torch
    for exact in (True, False):
        b = Latent(hp, A([600, 641]), A([600, 300]), 64, 512, 576, 16, "bf16", seed=13)
        w = selecting_weights(64, 128, 128, 512, b.dt, 5)
        if not exact:
            w = (torch.randn((64, 256, 512), generator=torch.Generator().manual_seed(3)) / 512 ** 0.5).to(b.dt)
        got = run_prefill(b, 128, 128, w, 0.07)
        check_prefill(b, got, 128, 128, w, 0.07, exact_kv=exact, sample={0, 127, 130, 599, 600, 777, 899})


def test_latent_prefill_kv_tokens_too_small(hp):
    import torch
    b = Latent(hp, A([40, 30]), A([4, 4]), 2, 512, 576, 16, "bf16")
    q = b.queries(192)
    rc, n = hp.hp_latent_prefill_workspace_bytes(b.desc, 512, 128, 128, 8, 2, 69)
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    out = torch.full((8, 2, 128), 9.0, dtype=b.dt, device="cuda")
    w = selecting_weights(2, 128, 128, 512, b.dt, 1).cuda()
    assert hp.hp_latent_prefill(b.desc, 512, w, 128, 128, q, b.q_ptr, 8, 2, 1.0, out, 69, ws, b.status) == 0
    torch.cuda.synchronize()
    assert hp.status_name(b.status.item()) == "HP_ERR_OUT_SIZE" and (out == 9).all()


# ------------------------------------------------------------------- used together
def test_a_prompt_and_decode_steps_over_a_latent_cache(hp):
    """Three steps of a small server on a side stream, the tables built on the GPU each time:
    prompts through the expanded form, then decode through the absorbed one, and the two forms
    agree on the same queries (the absorbed queries made from W^K, the values mapped by W^V)."""
    import torch
    H, R, Dr, Dn, Dv, P, pages = 4, 512, 64, 128, 128, 16, 64
    dt = torch.bfloat16
    g = torch.Generator().manual_seed(11)
    stream = torch.cuda.Stream()
    pool = torch.full((pages, P, R + Dr), float("nan"), dtype=dt, device="cuda")
    table_cs = dev(ref.cos_sin(512, Dr))
    w = selecting_weights(H, Dn, Dv, R, dt, 2)
    lw = torch.ones(R, dtype=dt, device="cuda")
    lens, have = A([0, 0, 0]), A([0, 0, 0])
    table = np.zeros(0, np.uint32)
    free = np.random.default_rng(0).permutation(pages).astype(np.uint32)
    scale, S = 1 / np.sqrt(Dn + Dr), 3
    for new in (A([33, 1, 70]), A([1, 1, 1]), A([0, 20, 1])):
        need = np.maximum(have, -(-(lens + new) // P))
        T = int(new.sum())
        o = dict(table_out=torch.empty(int(need.sum()), dtype=torch.int32, device="cuda"),
                 seq_ptr_out=torch.empty(S + 1, dtype=torch.int32, device="cuda"),
                 lens_out=torch.empty(S, dtype=torch.int32, device="cuda"),
                 new_ptr_out=torch.empty(S + 1, dtype=torch.int32, device="cuda"),
                 slot_map=torch.empty(T, dtype=torch.int64, device="cuda"),
                 positions=torch.empty(T, dtype=torch.int32, device="cuda"))
        d = hp.step_desc(block_table=index_tensor(table, "cuda") if len(table) else None,
                         seq_ptr=index_tensor(np.concatenate([[0], np.cumsum(have)]).astype(np.uint32), "cuda"),
                         seq_lens=index_tensor(lens.astype(np.uint32), "cuda"),
                         new_lens=index_tensor(new.astype(np.uint32), "cuda"),
                         free_pages=index_tensor(free, "cuda"), page_size=P, index_type=0, **o)
        rc, n = hp.hp_step_tables_workspace_bytes(S)
        ws = torch.empty(n, dtype=torch.uint8, device="cuda")
        st = status_tensor()
        kv = torch.randn((T, R + Dr), generator=g).to(dt).cuda()
        q = torch.randn((T, H, Dn + Dr), generator=g).to(dt).cuda()
        rope = hp.rope_desc(cos_sin=table_cs, positions=o["positions"], sections=(Dr // 2,),
                            interleaved=True)
        ld = hp.latent_desc(latent=kv[:, :R], k_rope=kv[:, R:], q_rope=q[:, :, Dn:],
                            q_out=q[:, :, Dn:], latent_weight=lw, dtype="bf16",
                            slot_map=o["slot_map"], pool=pool, num_pages=pages, page_size=P)
        pd = hp.PagedDesc(pool, o["table_out"], o["seq_ptr_out"], o["lens_out"], num_pages=pages,
                          page_size=P, num_heads=1, head_dim=R + Dr, dtype="bf16", index_type=0)
        total = int((lens + new).sum())
        rc, n1 = hp.hp_latent_prefill_workspace_bytes(pd, R, Dn, Dv, T, H, total)
        rc, n2 = hp.hp_latent_decode_workspace_bytes(pd, R, T, H)
        ws2 = torch.empty(max(n1, n2), dtype=torch.uint8, device="cuda")
        out = torch.empty((T, H, Dv), dtype=dt, device="cuda")
        lat = torch.empty((T, H, R), dtype=dt, device="cuda")
        wd = w.cuda()
        torch.cuda.synchronize()
        with torch.cuda.stream(stream):
            assert hp.hp_step_tables(d, ws, st) == 0
            assert hp.hp_latent_append(ld, rope, st) == 0
            assert hp.hp_latent_prefill(pd, R, wd, Dn, Dv, q, o["new_ptr_out"], T, H, scale, out,
                                        total, ws2, st) == 0
            # W^K picks: the absorbed query is exact in fp32 and rounded once here
            qa = torch.cat([torch.einsum("thd,hdr->thr", q[:, :, :Dn].float(), wd[:, :Dn].float()),
                            q[:, :, Dn:].float()], 2).to(dt)
            assert hp.hp_latent_decode(pd, R, qa, o["new_ptr_out"], T, H, scale, lat, ws2, st) == 0
            via = torch.einsum("thr,hdr->thd", lat.float(), wd[:, Dn:].float())
        stream.synchronize()
        assert st.item() == 0
        # both forms are within u |o| + (u + small) A of the same sums, A <= max |v|; the
        # absorbed query's sums of several picks are rounded once more (u of its score terms)
        vmax = float(pool[torch.isfinite(pool)].abs().max())
        ds = float((q.float().abs().sum(-1).max()) * vmax * scale) * 2 * ref.U["bf16"]
        assert float((out.float() - via).abs().max()) <= (6 * ref.U["bf16"] + 2 * min(ds, 0.02)) * vmax
        lens, have = lens + new, need
        table = o["table_out"].cpu().numpy().view(np.uint32)
        free = np.array([p for p in free if p not in set(table.tolist())], np.uint32)


def test_tables_norm_append_and_decode_attention(hp):
    """hp_step_tables -> hp_qk_norm_rope_append -> hp_attention_decode, one call captured into
    a graph and replayed on new inputs: same rows as the calls made one by one."""
    import torch
    Hq, Hkv, D, P, S, pages = 8, 2, 128, 16, 4, 40
    rng = np.random.default_rng(3)
    lens, new = A([30, 16, 0, 47]), A([1, 1, 1, 1])
    s = make_step(hp, lens, new, -(-lens // P), P, 0, spare=20, pad=0)
    T = 4
    x = torch.randn((T, (Hq + 2 * Hkv) * D)).to(torch.bfloat16).cuda()
    kp = torch.randn((pages, P, Hkv, D)).to(torch.bfloat16).cuda()
    vp = torch.randn((pages, P, Hkv, D)).to(torch.bfloat16).cuda()
    qo = torch.zeros((T, Hq, D), dtype=torch.bfloat16, device="cuda")
    w = torch.ones(D, dtype=torch.bfloat16, device="cuda")
    q, k, v = x.split([Hq * D, Hkv * D, Hkv * D], 1)
    rope = hp.rope_desc(cos_sin=dev(ref.cos_sin(100, D)), positions=s["o"]["positions"],
                        sections=(D // 2,))
    qd = hp.qk_desc(q=q, k=k, v=v, q_out=qo, q_weight=w, k_weight=w, num_q_heads=Hq,
                    num_kv_heads=Hkv, head_dim=D, dtype="bf16", slot_map=s["o"]["slot_map"],
                    k_pool=kp, v_pool=vp, num_pages=pages, page_size=P)
    n = int(np.maximum(-(-lens // P), -(-(lens + new) // P)).sum())
    s["o"]["table_out"] = s["o"]["table_out"][:n].clone()  # 64-byte aligned, exactly the entries
    s["d"] = hp.step_desc(block_table=s["d"].keep[0], seq_ptr=s["d"].keep[1], seq_lens=s["d"].keep[2],
                          new_lens=s["d"].keep[3], free_pages=s["d"].keep[4], page_size=P,
                          index_type=0, **s["o"])
    pd = hp.PagedDesc(kp, s["o"]["table_out"], s["o"]["seq_ptr_out"], s["o"]["lens_out"],
                      num_pages=pages, page_size=P, num_heads=Hkv, head_dim=D, dtype="bf16",
                      index_type=0)
    rc, nws = hp.hp_attention_decode_workspace_bytes(pd, Hq)
    aws = torch.zeros(nws, dtype=torch.uint8, device="cuda")
    out = torch.zeros((S, Hq, D), dtype=torch.float32, device="cuda")
    st = status_tensor()

    def calls():
        assert hp.hp_step_tables(s["d"], s["ws"], s["status"]) == 0
        assert hp.hp_qk_norm_rope_append(qd, rope, st) == 0
        assert hp.hp_attention_decode(pd, vp, qo, Hq, 0.09, out, aws, st) == 0
    calls()
    torch.cuda.synchronize()
    check_step(hp, s)
    assert st.item() == 0
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls()
    for _ in range(2):
        x.copy_(torch.randn(x.shape).to(torch.bfloat16))
        graph.replay()
        torch.cuda.synchronize()
        first = out.clone(), kp.clone(), vp.clone(), qo.clone()
        calls()
        torch.cuda.synchronize()
        assert st.item() == 0
        for a, c in zip(first, (out, kp, vp, qo)):
            assert torch.equal(a, c) and torch.isfinite(a.float()).all()
    # the appended row is the one attention reads: sequence 2 holds one token, its value
    slot = int(s["o"]["slot_map"][2])
    row = vp.view(-1, Hkv, D)[slot].float()
    assert torch.allclose(out[2], row.repeat_interleave(Hq // Hkv, 0), rtol=0, atol=1e-5)


def test_two_captured_graphs_and_planned_layers(hp):
    """Two graphs of latent decode with a workspace each, replayed in turn; and two layers'
    pools behind one plan."""
    import torch
    runs = []
    for seed in (1, 2):
        b = Latent(hp, A([300, 70, 0]), A([1, 2, 1]), 16, 512, 576, 16, "bf16", seed=seed)
        q = b.queries(576)
        rc, n = hp.hp_latent_decode_workspace_bytes(b.desc, 512, b.T, 16)
        ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
        out = torch.zeros((b.T, 16, 512), dtype=b.dt, device="cuda")
        call = lambda b=b, q=q, ws=ws, out=out: hp.hp_latent_decode(  # noqa: E731
            b.desc, 512, q, b.q_ptr, b.T, 16, 0.07, out, ws, b.status)
        assert call() == 0
        torch.cuda.synchronize()
        want = out.clone()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            assert call() == 0
        runs.append((b, q, out, want, graph, ws))
    for _ in range(3):
        for b, q, out, want, graph, ws in runs:
            out.zero_()
            graph.replay()
    torch.cuda.synchronize()
    for b, q, out, want, graph, ws in runs:
        assert torch.equal(out, want) and b.status.item() == 0
    b, q, out, want, _, ws = runs[0]
    pool2 = b.pool * 0.5
    d2 = hp.PagedDesc(pool2, *b.desc._keep[1:4], num_pages=b.desc.c.num_pages, page_size=16,
                      num_heads=1, head_dim=576, dtype="bf16", index_type=0)
    single = torch.zeros_like(out)
    ws2 = torch.zeros_like(ws)
    assert hp.hp_latent_decode(d2, 512, q, b.q_ptr, b.T, 16, 0.07, single, ws2, b.status) == 0
    assert hp.hp_latent_plan(b.desc, 512, b.q_ptr, b.T, 16, ws, b.status) == 0
    o1, o2 = torch.zeros_like(out), torch.zeros_like(out)
    for d, o in ((b.desc, o1), (d2, o2)):
        assert hp.hp_latent_decode_planned(d, 512, q, b.q_ptr, b.T, 16, 0.07, o, ws, b.status) == 0
    torch.cuda.synchronize()
    assert b.status.item() == 0 and torch.equal(o1, want) and torch.equal(o2, single)


# ------------------------------------------------------------ what the calls also allow
@pytest.mark.parametrize("form", ["decode", "prefill"])
def test_a_wait_that_runs_out_is_reported(hp, form):
    """HP_TEST_STALL: the first load of each CTA is armed and never issued, so every role's waits
    run out in turn; the call reports HP_ERR_TIMEOUT and the next one on the same context is
    right."""
    import torch
    b = Latent(hp, A([300, 70]), A([2, 70]), 8, 512, 576, 16, "bf16", seed=4)
    w = selecting_weights(8, 128, 128, 512, b.dt, 3)
    q = b.queries(576 if form == "decode" else 192)
    out = torch.zeros((b.T, 8, 512 if form == "decode" else 128), dtype=b.dt, device="cuda")
    if form == "decode":
        rc, n = hp.hp_latent_decode_workspace_bytes(b.desc, 512, b.T, 8)
    else:
        rc, n = hp.hp_latent_prefill_workspace_bytes(b.desc, 512, 128, 128, b.T, 8, 370)
    ws, wd = torch.zeros(n, dtype=torch.uint8, device="cuda"), w.cuda()
    for flags, name in ((hp.TEST_STALL, "HP_ERR_TIMEOUT"), (0, "HP_OK")):
        b.desc.c.flags = flags
        out.fill_(9)
        if form == "decode":
            rc = hp.hp_latent_decode(b.desc, 512, q, b.q_ptr, b.T, 8, 0.07, out, ws, b.status)
        else:
            rc = hp.hp_latent_prefill(b.desc, 512, wd, 128, 128, q, b.q_ptr, b.T, 8, 0.07, out, 370, ws, b.status)
        torch.cuda.synchronize()
        assert rc == 0 and hp.status_name(b.status.item()) == name
    if form == "decode":
        check_decode(b, host(out), 0.07)
    else:
        check_prefill(b, host(out), 128, 128, w, 0.07, exact_kv=True)


def test_scales_of_any_sign(hp):
    """A negative scale turns the order of the scores, a zero one weighs every seen token alike."""
    for scale in (-0.09, 0.0):
        for kernel in (0, hp.ATTN_CUDA_CORES):
            b = Latent(hp, A([200, 3]), A([2, 3]), 16, 512, 576, 16, "bf16", seed=8, flags=kernel)
            check_decode(b, run_decode(b, scale), scale)
            w = selecting_weights(16, 128, 128, 512, b.dt, 6)
            check_prefill(b, run_prefill(b, 128, 128, w, scale), 128, 128, w, scale, exact_kv=True)


def test_masked_tokens_of_any_value_in_a_one_query_batch(hp):
    """Slots past a length hold NaN in every test above; here infinities and the type's lowest
    values, in the last page and in pages no sequence names."""
    import torch
    for fill in (float("inf"), float("-inf"), -65504.0):
        b = Latent(hp, A([65, 1, 127]), A([1, 1, 1]), 16, 512, 576, 32, "f16", seed=12)
        b.pool[torch.isnan(b.pool)] = fill
        check_decode(b, run_decode(b, 0.07), 0.07)
        b.nq = A([65, 1, 100])
        b.q_ptr_host = np.concatenate([[0], np.cumsum(b.nq)])
        b.q_ptr = index_tensor(b.q_ptr_host.astype(np.uint32), "cuda")
        b.T = 166
        w = selecting_weights(16, 128, 128, 512, b.dt, 6)
        check_prefill(b, run_prefill(b, 128, 128, w, 0.07), 128, 128, w, 0.07, exact_kv=True)


def test_pool_rows_past_32_bits(hp):
    """A pool of more than 2^32 bytes: the last pages' rows, written by the append, read by both
    forms."""
    import torch
    P, W = 64, 576
    pages = (1 << 32) // (P * W * 2) + 40
    pool = torch.zeros((pages, P, W), dtype=torch.bfloat16, device="cuda")
    T, H = 100, 4
    slot = (np.arange(T) + (pages - 2) * P).astype(np.int64)
    g = torch.Generator().manual_seed(1)
    kv = torch.randn((T, W), generator=g).to(torch.bfloat16)
    rope = hp.rope_desc(cos_sin=dev(ref.cos_sin(10, 64)), sections=(32,),
                        positions=torch.zeros((1, T), dtype=torch.int32, device="cuda"))
    kd = kv.cuda()
    d = hp.latent_desc(latent=kd[:, :512], k_rope=kd[:, 512:], dtype="bf16", slot_map=dev(slot),
                       pool=pool, num_pages=pages, page_size=P)
    st = status_tensor()
    assert hp.hp_latent_append(d, rope, st) == 0
    torch.cuda.synchronize()
    assert st.item() == 0 and torch.equal(pool.view(-1, W)[-128:-28].cpu(), kv)
    b = Latent(hp, A([T]), A([3]), H, 512, W, P, "bf16", seed=2)
    b.rows = [kv.double().numpy()]
    b.pool = pool
    b.desc = hp.PagedDesc(pool, index_tensor(np.array([pages - 2, pages - 1], np.uint32), "cuda"),
                          b.desc._keep[2], b.desc._keep[3], num_pages=pages, page_size=P, num_heads=1,
                          head_dim=W, dtype="bf16", index_type=0)
    for kernel in (0, hp.ATTN_CUDA_CORES):
        b.desc.c.flags = kernel
        check_decode(b, run_decode(b, 0.07), 0.07)
    b.desc.c.flags = 0
    w = selecting_weights(H, 128, 128, 512, b.dt, 6)
    check_prefill(b, run_prefill(b, 128, 128, w, 0.07), 128, 128, w, 0.07, exact_kv=True)


def test_two_batches_at_once_on_two_streams(hp):
    """Calls on two streams, a workspace each, while a large one runs on the other."""
    import torch
    big = Latent(hp, np.full(64, 1500), np.ones(64, np.int64), 128, 512, 576, 64, "bf16", seed=1)
    small = Latent(hp, A([90, 300]), A([1, 2]), 16, 512, 576, 16, "f16", seed=2)
    runs = []
    for b in (big, small):
        q = b.queries(576)
        rc, n = hp.hp_latent_decode_workspace_bytes(b.desc, 512, b.T, b.H)
        runs.append((b, q, torch.zeros(n, dtype=torch.uint8, device="cuda"),
                     torch.zeros((b.T, b.H, 512), dtype=b.dt, device="cuda"), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(4):
        for b, q, ws, out, s in runs:
            assert hp.hp_latent_decode(b.desc, 512, q, b.q_ptr, b.T, b.H, 0.07, out, ws, b.status, s) == 0
    torch.cuda.synchronize()
    for b, q, ws, out, s in runs:
        assert b.status.item() == 0
        check_decode(b, host(out), 0.07, rows={0, 1, 2, 40})


@pytest.mark.parametrize("kernel", ["cuda_cores", "default"])
def test_a_nan_query_keeps_its_nan_to_itself(hp, kernel):
    """NaN in one (query, head) row: that row of out is NaN, whether one worker saw all its tokens
    or many share the sequence, and every other row is as it would be; so in both forms, with NaN
    queries behind the last sequence too."""
    import torch
    for lens, nq in ((A([300, 40]), A([3, 2])), (A([30000, 5]), A([1, 2]))):
        for form in ("decode", "prefill"):
            b = Latent(hp, lens, nq, 8, 512, 576, 16, "bf16", seed=21, rows_behind=2, flags=cores(hp, kernel))
            w, real = selecting_weights(8, 128, 128, 512, b.dt, 6), b.queries

            def queries(width):
                real(width)
                b.clean = b.q.clone()
                b.q[0, 3, 5] = float("nan")
                b.q[-2:] = float("nan")
                return b.q.cuda()
            b.queries = queries
            if form == "decode":
                got = run_decode(b, 0.07)
            else:
                got = run_prefill(b, 128, 128, w, 0.07)
            assert np.isnan(got[0, 3]).all(), form
            # the row's clean result in its place, the whole is checked against the formula
            b.q, b.queries = b.clean, lambda width: b.clean.cuda()
            if form == "decode":
                got[0, 3] = run_decode(b, 0.07)[0, 3]
                check_decode(b, got, 0.07)
            else:
                got[0, 3] = run_prefill(b, 128, 128, w, 0.07)[0, 3]
                check_prefill(b, got, 128, 128, w, 0.07, exact_kv=True)


@pytest.mark.parametrize("R,W,P", [(512, 576, 16), (128, 192, 6)])
def test_latent_attention_over_a_pool_in_host_memory(hp, R, W, P):
    """HP_HOST_MEMORY: the pool's page-locked copy gives the device pool's results."""
    import torch
    for form in ("decode", "prefill"):
        outs = []
        for flags in (hp.ATTN_CUDA_CORES if form == "decode" else 0, hp.HOST_MEMORY):
            b = Latent(hp, A([100, 0, 333]), A([2, 1, 40]), 4, R, W, P, "f16", seed=3, flags=flags)
            if flags == hp.HOST_MEMORY:
                pinned = torch.empty(b.pool.shape, dtype=b.pool.dtype, pin_memory=True)
                pinned.copy_(b.pool)
                b.desc = hp.PagedDesc(pinned, *b.desc._keep[1:4], num_pages=b.desc.c.num_pages, page_size=P,
                                      num_heads=1, head_dim=W, dtype="f16", index_type=0, flags=flags)
            w = selecting_weights(4, 128, 128, R, b.dt, 6)
            outs.append(run_decode(b, 0.07) if form == "decode" else run_prefill(b, 128, 128, w, 0.07))
        assert np.array_equal(*outs)


def test_many_heads_and_large_pages(hp):
    """1,000 heads (eight groups of 128 rows a query and a ragged one), and pages of 4,096 slots."""
    b = Latent(hp, A([130]), A([1]), 1000, 512, 576, 16, "bf16", seed=1)
    check_decode(b, run_decode(b, 0.07), 0.07)
    for kernel in (0, hp.ATTN_CUDA_CORES):
        b = Latent(hp, A([4097, 9000]), A([1, 3]), 4, 512, 576, 4096, "f16", seed=2, flags=kernel)
        check_decode(b, run_decode(b, 0.07), 0.07)
    w = selecting_weights(4, 128, 128, 512, b.dt, 6)
    b = Latent(hp, A([4097, 200]), A([1, 3]), 4, 512, 576, 4096, "f16", seed=2)
    check_prefill(b, run_prefill(b, 128, 128, w, 0.07), 128, 128, w, 0.07, exact_kv=True)


def test_prefill_of_one_query_each_without_offsets(hp):
    b = Latent(hp, A([40, 0, 333]), np.ones(3, np.int64), 4, 512, 576, 16, "bf16", with_ptr=False)
    w = selecting_weights(4, 128, 128, 512, b.dt, 6)
    check_prefill(b, run_prefill(b, 128, 128, w, 0.07), 128, 128, w, 0.07, exact_kv=True)


@pytest.mark.parametrize("form", ["decode", "prefill"])
def test_no_query_at_all(hp, form):
    """total_q = 0 over sequences that have tokens, and no sequence: the descriptor is checked,
    nothing is written."""
    import torch
    for lens in (A([40, 9]), np.zeros(0, np.int64)):
        b = Latent(hp, lens, np.zeros(len(lens), np.int64), 4, 512, 576, 16, "bf16")
        w = selecting_weights(4, 128, 128, 512, b.dt, 6).cuda()
        ws = torch.zeros(1 << 27, dtype=torch.uint8, device="cuda")
        if form == "decode":
            rc = hp.hp_latent_decode(b.desc, 512, None, b.q_ptr, 0, 4, 1.0, None, ws, b.status)
        else:
            rc = hp.hp_latent_prefill(b.desc, 512, w, 128, 128, None, b.q_ptr, 0, 4, 1.0, None, 49, ws, b.status)
        torch.cuda.synchronize()
        assert hp.status_name(rc) == "HP_OK" and b.status.item() == 0
        if len(lens):
            b.desc._keep[3][1] = 33
            if form == "decode":
                hp.hp_latent_decode(b.desc, 512, None, b.q_ptr, 0, 4, 1.0, None, ws, b.status)
            else:
                hp.hp_latent_prefill(b.desc, 512, w, 128, 128, None, b.q_ptr, 0, 4, 1.0, None, 49, ws, b.status)
            torch.cuda.synchronize()
            assert hp.status_name(b.status.item()) == "HP_ERR_LEN"


@pytest.mark.parametrize("what,name", [
    ("start", "SEQ_PTR_START"), ("order", "SEQ_PTR_ORDER"), ("end", "SEQ_PTR_END"), ("len", "LEN"),
    ("grow", "LEN"), ("free", "CAPACITY"), ("cap", "OUT_SIZE"), ("tokens", "OUT_SIZE"),
])
def test_step_tables_verdicts_of_a_large_step(hp, what, name):
    """The same rules where several CTAs scan: 3,001 sequences, the fault in the last block."""
    import torch
    lens, new = np.full(3001, 20), np.full(3001, 20)
    s = make_step(hp, lens, new, np.full(3001, 2), 16, 0, free=1 if what == "free" else None)
    d = s["d"]
    bt, sp, ln, nw = d.keep[0], d.keep[1], d.keep[2], d.keep[3]
    if what == "start":
        sp[0] = 1
    elif what == "order":
        sp[2900] = 2
    elif what == "end":
        sp[3001] = 6003
    elif what == "len":
        ln[2999] = 33
    elif what == "grow":
        nw[2999] = -20
    elif what == "cap":
        d.table_cap = 3001 * 3 - 1
    elif what == "tokens":
        d.token_cap = 3001 * 20 - 1
    assert hp.hp_step_tables(d, s["ws"], s["status"]) == 0
    torch.cuda.synchronize()
    assert hp.status_name(s["status"].item()) == "HP_ERR_" + name
    for t in s["o"].values():
        assert (t == -9).all()


@pytest.mark.parametrize("T", [2, 5000])
def test_appends_of_tokens_without_a_place(hp, T):
    """Batches on either side of the two ways of reporting: every token's slot out of the pool,
    one position out of the table besides; padding alone; the same calls without a status."""
    import torch
    P, W, pages = 16, 576, 400
    kv = torch.randn((T, W)).to(torch.bfloat16).cuda()
    cs = dev(ref.cos_sin(10, 64))
    pool = torch.zeros((pages, P, W), dtype=torch.bfloat16, device="cuda")
    for slot, far, name in ((pages * P, False, "HP_ERR_PAGE_ID"), (pages * P, True, "HP_ERR_LEN"),
                            (2 ** 62, False, "HP_ERR_PAGE_ID"), (-1, False, "HP_OK"), (-1, True, "HP_OK"),
                            (-2 ** 63, False, "HP_OK")):
        pos = torch.zeros((1, T), dtype=torch.int32, device="cuda")
        pos[0, T - 1] = -1 if far else 9  # 2^32 - 1
        rope = hp.rope_desc(cos_sin=cs, sections=(32,), positions=pos)
        d = hp.latent_desc(latent=kv[:, :512], k_rope=kv[:, 512:], dtype="bf16",
                           slot_map=dev(np.full(T, slot, np.int64)), pool=pool, num_pages=pages, page_size=P)
        for st in (status_tensor(), None):
            assert hp.hp_latent_append(d, rope, st) == 0
            torch.cuda.synchronize()
            assert st is None or hp.status_name(st.item()) == name
            assert not pool.any()


def test_a_whole_latent_step_in_one_graph(hp):
    """Tables, append, prompts and decode of one step captured together; replayed on new lengths,
    rows and queries the graph gives what the calls give one by one."""
    import torch
    S, H, R, P, W, pages, T = 5, 4, 512, 16, 576, 64, 90
    dt = torch.bfloat16
    lens, new = torch.zeros(S, dtype=torch.int32).cuda(), torch.zeros(S, dtype=torch.int32).cuda()
    # each sequence has 10 pages, so that its slice does not grow
    table = torch.randperm(pages)[:10 * S].int().cuda()
    sp = (torch.arange(S + 1) * 10).int().cuda()
    o = dict(table_out=torch.empty(10 * S, dtype=torch.int32, device="cuda"),
             seq_ptr_out=torch.empty(S + 1, dtype=torch.int32, device="cuda"),
             lens_out=torch.empty(S, dtype=torch.int32, device="cuda"),
             new_ptr_out=torch.empty(S + 1, dtype=torch.int32, device="cuda"),
             slot_map=torch.empty(T, dtype=torch.int64, device="cuda"),
             positions=torch.empty(T, dtype=torch.int32, device="cuda"))
    sd = hp.step_desc(block_table=table, seq_ptr=sp, seq_lens=lens, new_lens=new, free_pages=None, page_size=P,
                      index_type=0, **o)
    rc, n = hp.hp_step_tables_workspace_bytes(S)
    sws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    pool = torch.zeros((pages, P, W), dtype=dt, device="cuda")
    kv = torch.zeros((T, W), dtype=dt, device="cuda")
    q = torch.zeros((T, H, 192), dtype=dt, device="cuda")
    qa = torch.zeros((T, H, W), dtype=dt, device="cuda")
    rope = hp.rope_desc(cos_sin=dev(ref.cos_sin(200, 64)), positions=o["positions"], sections=(32,))
    ld = hp.latent_desc(latent=kv[:, :R], k_rope=kv[:, R:], dtype="bf16", slot_map=o["slot_map"], pool=pool,
                        num_pages=pages, page_size=P)
    pd = hp.PagedDesc(pool, o["table_out"], o["seq_ptr_out"], o["lens_out"], num_pages=pages, page_size=P,
                      num_heads=1, head_dim=W, dtype="bf16", index_type=0)
    kv_cap = 10 * S * P
    rc, n1 = hp.hp_latent_prefill_workspace_bytes(pd, R, 128, 128, T, H, kv_cap)
    rc, n2 = hp.hp_latent_decode_workspace_bytes(pd, R, T, H)
    ws = torch.zeros(max(n1, n2), dtype=torch.uint8, device="cuda")
    w = selecting_weights(H, 128, 128, R, dt, 2).cuda()
    out, lat = torch.zeros((T, H, 128), dtype=dt).cuda(), torch.zeros((T, H, R), dtype=dt).cuda()
    st = [status_tensor() for _ in range(4)]

    def calls():
        assert hp.hp_step_tables(sd, sws, st[0]) == 0
        assert hp.hp_latent_append(ld, rope, st[1]) == 0
        assert hp.hp_latent_prefill(pd, R, w, 128, 128, q, o["new_ptr_out"], T, H, 0.07, out, kv_cap, ws, st[2]) == 0
        assert hp.hp_latent_decode(pd, R, qa, o["new_ptr_out"], T, H, 0.07, lat, ws, st[3]) == 0
    calls()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls()
    for ln, nw in (([0, 0, 0, 0, 0], [90, 0, 0, 0, 0]), ([90, 0, 5, 140, 1], [1, 30, 0, 20, 1]),
                   ([100, 1, 1, 1, 1], [0, 0, 0, 0, 0]), ([99, 98, 97, 96, 95], [1, 1, 1, 1, 1])):
        lens.copy_(torch.tensor(ln))
        new.copy_(torch.tensor(nw))
        for t in (kv, q, qa):
            t.copy_(torch.randn(t.shape).to(dt))
        results = []
        for run in (graph.replay, calls):
            pool.copy_(torch.ones(1, dtype=dt))
            out.fill_(9)
            lat.fill_(9)
            run()
            torch.cuda.synchronize()
            assert [x.item() for x in st] == [0] * 4
            results.append([t.clone() for t in (out, lat, pool, *o.values())])
        for a, c in zip(*results):
            assert torch.equal(a, c) and torch.isfinite(a.float()).all()
        assert (out[sum(nw):] == 9).all() and (lat[sum(nw):] == 9).all() and not (lat[:sum(nw)] == 9).all(-1).any()


def test_tables_and_appends_on_two_streams(hp):
    """Steps of different sizes on two streams at once, a workspace each."""
    import torch
    rng = np.random.default_rng(8)
    runs = []
    for S in (4000, 30):
        lens, new = rng.integers(0, 300, S), rng.integers(0, 4, S)
        s = make_step(hp, lens, new, -(-lens // 16), 16, 0, pad=0)
        T = int(new.sum())
        kv = torch.randn((T, 576)).to(torch.bfloat16).cuda()
        rope = hp.rope_desc(cos_sin=dev(ref.cos_sin(310, 64)), sections=(32,), positions=s["o"]["positions"])
        pages = len(s["table"]) + len(s["free"])
        pool = torch.zeros((pages, 16, 576), dtype=torch.bfloat16, device="cuda")
        d = hp.latent_desc(latent=kv[:, :512], k_rope=kv[:, 512:], dtype="bf16", slot_map=s["o"]["slot_map"],
                           pool=pool, num_pages=pages, page_size=16)
        runs.append((s, d, rope, pool, kv, status_tensor(), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(5):
        for s, d, rope, pool, kv, st, stream in runs:
            assert hp.hp_step_tables(s["d"], s["ws"], s["status"], stream) == 0
            assert hp.hp_latent_append(d, rope, st, stream) == 0
    for s, d, rope, pool, kv, st, stream in runs:
        check_step(hp, s)
        assert st.item() == 0 and torch.equal(pool.view(-1, 576)[s["o"]["slot_map"]][:, :512], kv[:, :512])


@pytest.mark.parametrize("form", ["decode", "prefill"])
@pytest.mark.parametrize("S", [1, 3, 128, 129])
def test_plans_of_small_and_large_batches(hp, form, S):
    """Up to 128 sequences (and 4,096 table entries) the first kernel makes the plan itself, beyond
    a launch before it does: the same results and the same verdicts on both sides, the first rule
    that fails naming itself, nothing else written."""
    import torch
    rng = np.random.default_rng(S)
    lens, nq = rng.integers(1, 200, S), rng.integers(0, 3, S)
    nq[0], lens[-1] = 1, 20
    nq = np.minimum(nq, lens)
    w = selecting_weights(4, 128, 128, 512, ref.torch_dtype("bf16"), 6)

    def make():
        return Latent(hp, lens, nq, 4, 512, 576, 16, "bf16", it=S % 2, seed=S, rows_behind=1)
    b = make()
    if form == "decode":
        check_decode(b, run_decode(b, 0.07), 0.07)
    else:
        check_prefill(b, run_prefill(b, 128, 128, w, 0.07), 128, 128, w, 0.07, exact_kv=True)
    T = b.T
    faults = ["page", "len", "end", "start", "order", "qstart", "qorder", "qend", "page+len", "start+len"]
    for what in faults + (["room"] if form == "prefill" else []):
        if S == 1 and what in ("order", "qorder"):
            continue
        b = make()
        table, sp, ln = b.desc._keep[1], b.desc._keep[2], b.desc._keep[3]
        kv, name = int(lens.sum()), {"page": "PAGE_ID", "len": "LEN", "end": "SEQ_PTR_END", "start": "SEQ_PTR_START",
                                     "order": "SEQ_PTR_ORDER", "qstart": "NEW_PTR_START", "qorder": "NEW_PTR_ORDER",
                                     "qend": "NEW_PTR_END", "room": "OUT_SIZE"}[what.split("+")[0]]
        if "page" in what:
            table[len(table) - 1] = 10 ** 6
        if "len" in what:
            ln[S - 1] = 33
        if what == "end":
            sp[S] += 1
        if "start" in what and what[0] != "q":
            sp[0] = 1
        if what == "order":
            sp[S // 2] = int(sp[S // 2 + 1]) + 1
        if what == "qstart":
            b.q_ptr[0] = 1
        if what == "qorder":
            b.q_ptr[S // 2] = T + 5
        if what == "room":
            kv -= 1
        total = T - 2 if what == "qend" else T
        if form == "decode":
            q = b.queries(576)
            out = torch.full((T, 4, 512), 9.0, dtype=b.dt, device="cuda")
            rc, n = hp.hp_latent_decode_workspace_bytes(b.desc, 512, T, 4)
        else:
            q = b.queries(192)
            out = torch.full((T, 4, 128), 9.0, dtype=b.dt, device="cuda")
            rc, n = hp.hp_latent_prefill_workspace_bytes(b.desc, 512, 128, 128, T, 4, kv)
        if total <= 0:
            continue
        ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")
        if form == "decode":
            rc = hp.hp_latent_decode(b.desc, 512, q, b.q_ptr, total, 4, 0.1, out, ws, b.status)
        else:
            rc = hp.hp_latent_prefill(b.desc, 512, w.cuda(), 128, 128, q, b.q_ptr, total, 4, 0.1, out, kv, ws, b.status)
        torch.cuda.synchronize()
        assert hp.status_name(rc) == "HP_OK" and hp.status_name(b.status.item()) == "HP_ERR_" + name, what
        assert (out == 9).all(), what


@pytest.mark.parametrize("pages", [4096, 4097])
def test_plans_of_short_and_long_tables(hp, pages):
    """One sequence whose table is as long as its plan's own check takes, and one entry longer; a bad
    last entry is seen on both sides."""
    import torch
    for kind in ("decode", "prefill"):
        b = Latent(hp, A([pages * 8 - 3]), A([2]), 2, 512, 576, 8, "f16", seed=pages)
        w = selecting_weights(2, 128, 128, 512, b.dt, 6)
        if kind == "decode":
            check_decode(b, run_decode(b, 0.07), 0.07)
        else:
            check_prefill(b, run_prefill(b, 128, 128, w, 0.07), 128, 128, w, 0.07, exact_kv=True)
        b.desc._keep[1][pages - 1] = 2 ** 30
        rc, n = hp.hp_latent_decode_workspace_bytes(b.desc, 512, 2, 2)
        ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
        out = torch.full((2, 2, 512), 9.0, dtype=b.dt, device="cuda")
        q = torch.zeros((2, 2, 576), dtype=b.dt, device="cuda")
        assert hp.hp_latent_decode(b.desc, 512, q, b.q_ptr, 2, 2, 0.1, out, ws, b.status) == 0
        torch.cuda.synchronize()
        assert hp.status_name(b.status.item()) == "HP_ERR_PAGE_ID" and (out == 9).all()


def test_appends_report_whatever_the_rows(hp):
    """3,000 tokens of 2 KiB and of 18 KiB, whose codes are gathered in two ways: the smallest code
    of the batch, the tokens without a fault stored."""
    import torch
    T, D, P = 3000, 128, 16
    cs = dev(ref.cos_sin(50, D))
    for hq, hkv in ((1, 1), (32, 2)):
        x = torch.randn((T, (hq + 2 * hkv) * D)).to(torch.bfloat16).cuda()
        q, k, v = x.split([hq * D, hkv * D, hkv * D], 1)
        for slots, far, name in (((), (), "HP_OK"), ((2999,), (), "HP_ERR_PAGE_ID"), ((5, 2050), (2998,), "HP_ERR_LEN"),
                                 ((), (2049,), "HP_ERR_LEN")):
            slot, pos = np.arange(T, dtype=np.int64), np.zeros((2, T), np.uint32)
            for t in slots:
                slot[t] = 190 * P
            for t in far:
                pos[1, t] = 50
            kp = torch.zeros((190, P, hkv, D), dtype=torch.bfloat16, device="cuda")
            vp, qo, st = torch.zeros_like(kp), torch.zeros((T, hq * D), dtype=torch.bfloat16, device="cuda"), status_tensor()
            r = hp.rope_desc(cos_sin=cs, positions=index_tensor(pos, "cuda"), sections=(32, 32))
            d = hp.qk_desc(q=q, k=k, v=v, q_out=qo, num_q_heads=hq, num_kv_heads=hkv, head_dim=D, dtype="bf16",
                           slot_map=dev(slot), k_pool=kp, v_pool=vp, num_pages=190, page_size=P)
            assert hp.hp_qk_norm_rope_append(d, r, st) == 0
            torch.cuda.synchronize()
            assert hp.status_name(st.item()) == name
            live = np.ones(T, bool)
            live[list(slots) + list(far)] = False
            got = vp.view(-1, hkv * D)[:T].cpu()
            assert torch.equal(got[live], v.cpu()[live]) and not got[~live].any() and not qo.cpu()[~live].any()


@pytest.mark.parametrize("form", ["decode", "prefill"])
def test_a_large_batch_in_a_graph(hp, form):
    """200 sequences, whose plan is a launch of its own, captured and replayed on other queries."""
    import torch
    lens = np.random.default_rng(4).integers(1, 150, 200)
    b = Latent(hp, lens, np.ones(200, np.int64), 4, 512, 576, 16, "bf16", seed=4)
    w = selecting_weights(4, 128, 128, 512, b.dt, 6)
    wd, q = w.cuda(), b.queries(576 if form == "decode" else 192)
    kv = int(lens.sum())
    if form == "decode":
        rc, n = hp.hp_latent_decode_workspace_bytes(b.desc, 512, b.T, 4)
    else:
        rc, n = hp.hp_latent_prefill_workspace_bytes(b.desc, 512, 128, 128, b.T, 4, kv)
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")
    out = torch.zeros((b.T, 4, 512 if form == "decode" else 128), dtype=b.dt, device="cuda")

    def call():
        if form == "decode":
            return hp.hp_latent_decode(b.desc, 512, q, b.q_ptr, b.T, 4, 0.07, out, ws, b.status)
        return hp.hp_latent_prefill(b.desc, 512, wd, 128, 128, q, b.q_ptr, b.T, 4, 0.07, out, kv, ws, b.status)
    assert call() == 0
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        assert call() == 0
    for _ in range(2):
        b.q = torch.randn(q.shape).to(b.dt)
        q.copy_(b.q)
        out.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        assert b.status.item() == 0
        if form == "decode":
            check_decode(b, host(out), 0.07)
        else:
            check_prefill(b, host(out), 128, 128, w, 0.07, exact_kv=True)
