"""The operators of long contexts where an index, a mask or a call order is at its edge, and together as a
serving step uses them."""
import numpy as np
import pytest

import pages_ref as ref
import step_ref
from pages_ref import Batch, visible
from test_gpu_pages import check_bounds, check_scores, lists, list_tokens, make_bounds, run_bounds, run_pages, run_scores
from test_gpu_prefix import everything, make, run, workspace

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------- what is skipped, and said
@pytest.mark.parametrize("many", [False, True])
@pytest.mark.parametrize("what,code", [("page", "HP_ERR_PAGE_ID"), ("slice", "HP_ERR_LEN"), ("reversed", "HP_ERR_LEN"),
                                       ("end", "HP_ERR_LEN"), ("index", "HP_ERR_LEN")])
def test_a_query_whose_pages_do_not_hold_is_skipped(hp, what, code, many):
    """One CTA looks at small calls; in large ones whoever meets the error reports it."""
    import torch
    S = 300 if many else 4
    lens = np.full(S, 100)
    b = Batch(hp, lens, 2, 2, 64, 16, seed=4)
    k = 7
    sel = np.tile(np.arange(k, dtype=np.int32), (S, 2, 1))
    bad = {1}  # row 1 (its head 0 only where its list is wrong)
    if what == "page":
        b.d_table[7 + 3] = b.pages
    elif what == "slice":
        b.d_lens[1] = 7 * 16 + 1
        sel[1, :, 0] = 7
    elif what == "reversed":
        b.d_ptr[1] = 7 * S
        bad = {0, 1}  # (both slices have that end)
    elif what == "end":
        b.d_ptr[2] = 7 * S + 1
        bad = {1, 2}
    elif what == "index":
        sel[1, 0, 2] = 7
    sel = torch.from_numpy(sel)
    run_pages(b, sel)
    if what == "reversed":  # a longer slice of row 0 is no error by itself
        bad = {1}
    assert b.code() == code
    good = [r for r in range(S) if r not in bad and not (what == "slice" and r == 1)]
    b.check(list_tokens(b, sel), rows=set(good[:3] + good[-3:]))
    got = b.out.float().cpu().numpy()
    for r in bad:
        assert (got[r, :2] == 7.0).all()
        if what == "index":
            assert (got[r, 2:] != 7.0).any()
    # what follows starts again
    b2 = Batch(hp, lens[:3], 2, 2, 64, 16, seed=4)
    b2.status = b.status
    sel2 = lists(b2, 3)
    run_pages(b2, sel2)
    assert b2.code() == "HP_OK"


@pytest.mark.parametrize("many", [False, True])
def test_bounds_and_scores_of_pages_that_do_not_hold(hp, many):
    import torch
    S = 1500 if many else 5
    b = Batch(hp, np.full(S, 33), 2, 1, 64, 16, seed=6)
    b.d_table[3 + 2] = b.pages + 5          # sequence 1, page 2
    b.d_lens[3] = 49                        # sequence 3: more than its slice
    got, before = run_bounds(b, np.ones(S, np.int64), it_null=True)
    assert b.code() == "HP_ERR_LEN"
    want = np.ones(S, np.int64)
    want[[1, 3]] = 0
    check_bounds(b, want, got, before)
    bounds = make_bounds(b)
    out = run_scores(b, bounds.cuda(), 4)
    assert b.code() == "HP_ERR_LEN"
    assert (out[3] == -77.0).all() and (out[1, :, 2] == -77.0).all() and (out[1, :, :2] != -77.0).all()
    b.d_lens[3] = 33
    out = run_scores(b, bounds.cuda(), 2)   # no room for the third page
    assert b.code() == "HP_ERR_OUT_SIZE" and (out == -77.0).all()


@pytest.mark.parametrize("q_ptr,code", [([0, 2, 1, 4], "HP_ERR_NEW_PTR_ORDER"), ([1, 2, 3, 4], "HP_ERR_NEW_PTR_START"),
                                        ([0, 1, 2, 5], "HP_ERR_NEW_PTR_END")])
def test_offsets_that_do_not_hold(hp, q_ptr, code):
    import torch
    b = Batch(hp, [50, 60, 70], 2, 1, 64, 16, nq=[1, 1, 2], seed=3)
    b.d_q_ptr = b.dev(q_ptr)
    run_pages(b, lists(b, 3))
    assert b.code() == code
    assert run_scores(b, make_bounds(b).cuda(), 5).shape == (4, 2, 5) and b.code() == code
    x = torch.zeros((4, 2, 5), device="cuda")
    out = torch.zeros((4, 2, 2), dtype=torch.int32, device="cuda")
    assert hp.hp_select_pages(b.desc, b.d_q_ptr, 4, x, 5, 0, 0, 2, out, b.status) == 0 and b.code() == code
    bounds = make_bounds(b).cuda()
    assert hp.hp_page_bounds(b.desc, b.d_q_ptr, 4, bounds, b.status) == 0 and b.code() == code
    g = make(hp, [(2, 20), (1, 0)], [30, 40, 70], 2, 1, 64, 16, nq=[1, 1, 2])
    g.d_q_ptr = g.dev(q_ptr)
    run(g)
    assert g.code() == code and (g.out == 7.0).all()


def test_sequences_of_2_31_tokens_are_refused_on_the_device(hp):
    b = Batch(hp, [50, 60], 1, 1, 64, 16, it=1, seed=3)
    b.d_lens[1] = 1 << 31
    run_pages(b, lists(b, 2))
    assert b.code() == "HP_ERR_LEN" and (b.out[1] == 7.0).all() and (b.out[0] != 7.0).any()
    run_scores(b, make_bounds(b).cuda(), 9)
    assert b.code() == "HP_ERR_LEN"
    run_bounds(b, [1, 1], it_null=True)
    assert b.code() == "HP_ERR_LEN"


@pytest.mark.parametrize("kernel", ["tensor_cores", "cuda_cores"])
@pytest.mark.parametrize("what,code", [
    ("ptr_start", "SEQ_PTR_START"), ("ptr_order", "SEQ_PTR_ORDER"), ("ptr_end", "SEQ_PTR_END"), ("page", "PAGE_ID"),
    ("len", "LEN"), ("group_start", "GROUP"), ("group_order", "GROUP"), ("group_end", "GROUP"), ("prefix", "PREFIX"),
    ("prefix_query", "PREFIX"), ("prefix_empty", "PREFIX"),
])
def test_prefix_verdicts(hp, kernel, what, code):
    """A rule that fails leaves nothing but the status; the planned call behind it keeps it."""
    b = make(hp, [(2, 40), (2, 20), (1, 0)], [9, 3, 5, 6, 40], 2, 4, 64, 16, kernel=kernel, nq=[1, 2, 1, 1, 1])
    if what == "ptr_start":
        b.d_ptr[0] = 1
    elif what == "ptr_order":
        b.d_ptr[2] = 1
    elif what == "ptr_end":
        b.d_ptr[5] -= 1
        b.d_lens[4] = 3
    elif what == "page":
        b.d_table[-1] = b.pages
    elif what == "len":
        b.d_lens[2] = 33
    elif what == "group_start":
        b.d_group[0] = 1
    elif what == "group_order":
        b.d_group[1] = 5
    elif what == "group_end":
        b.d_group[3] = 4
    elif what == "prefix":
        b.d_prefix[1] = 26
    elif what == "prefix_query":
        b.d_prefix[0] = 43
    elif what == "prefix_empty":
        b.d_prefix[2] = 1 << 20
    ws = run(b)
    assert b.code() == "HP_ERR_" + code
    assert (b.out == 7.0).all()
    rc = hp.hp_attention_prefix_planned(b.desc, b.v, b.d_group, b.d_prefix, 3, b.q, b.d_q_ptr, b.T, 8, b.scale, b.out, ws,
                                        b.status)
    assert rc == 0 and b.code() == "HP_ERR_" + code and (b.out == 7.0).all()
    b.status.fill_(99)
    assert hp.hp_attention_prefix_plan(b.desc, b.d_group, b.d_prefix, 3, b.d_q_ptr, b.T, 8, ws, b.status) == 0
    assert b.code() == "HP_ERR_" + code


def test_prefix_verdict_of_a_long_table(hp):
    """The plan's CTAs each look at a part of the table; the first bad entry's rule is found wherever it is."""
    import torch
    b = make(hp, [(3, 100000)], [5, 6, 7], 1, 1, 64, 8)
    for at in (0, 12500, 25007, 37502):
        keep = b.d_table[at].clone()
        b.d_table[at] = b.pages + 1
        run(b)
        assert b.code() == "HP_ERR_PAGE_ID" and (b.out == 7.0).all(), at
        b.d_table[at] = keep
    run(b)
    assert b.code() == "HP_OK"
    b.check(everything, rows={1})


@pytest.mark.parametrize("kernel", ["tensor_cores", "cuda_cores"])
def test_prefix_without_queries(hp, kernel):
    import torch
    b = make(hp, [(2, 20)], [3, 4], 1, 2, 128, 16, kernel=kernel, nq=[0, 0], behind=2)
    run(b)
    assert b.code() == "HP_OK" and (b.out == 7.0).all()
    rc = hp.hp_attention_prefix(b.desc, b.v, b.d_group, b.d_prefix, 1, b.q, b.d_q_ptr, 0, 2, b.scale, b.out, workspace(b),
                                b.status)
    assert rc == 0 and b.code() == "HP_OK"


# ------------------------------------------------------------------- values at their edges
@pytest.mark.parametrize("op", ["pages", "prefix", "prefix_cuda_cores"])
def test_values_that_are_not_finite_spoil_their_own_queries(hp, op):
    """A NaN key of one sequence's own token, an infinite value of another's, a NaN query."""
    import torch
    kernel = "cuda_cores" if op.endswith("cores") else "tensor_cores"
    b = make(hp, [(4, 200)], [40, 50, 60, 20], 2, 4, 128, 16, kernel=kernel, nq=[1, 3, 1, 1], seed=8)
    at = lambda s, t: (int(b.table[b.ptr[s] + t // 16]), t % 16)  # noqa: E731
    p, i = at(1, 249)                  # sequence 1's last token: its last query alone sees it
    b.hk[p, i, 0, 5] = float("nan")
    p, i = at(2, 230)
    b.hv[p, i, 1, 9] = float("inf")
    b.hq[5, 3, 2] = float("nan")
    b.k.copy_(b.hk), b.v.copy_(b.hv), b.q.copy_(b.hq)
    if op == "pages":
        n = -(-int(b.lens.max()) // 16)
        sel = torch.full((b.T, 2, n), -1, dtype=torch.int32)
        for row, s, seen in visible(b.lens, b.nq):
            for h in range(2):
                m = -(-int(b.lens[s]) // 16)
                sel[row, h, :m] = torch.arange(m)
        b.prefix[:] = 0
        for s in range(1, 4):          # every sequence through its own slice: the shared part's last page too
            w, (src, _) = 200 // 16, at(0, 192)
            dst = int(b.table[b.ptr[s] + w])
            b.hk[dst, :8], b.hv[dst, :8] = b.hk[src, :8], b.hv[src, :8]
        b.k.copy_(b.hk), b.v.copy_(b.hv)
        run_pages(b, sel)
    else:
        run(b)
    assert b.code() == "HP_OK"
    got = b.out.float().cpu().numpy()
    bad = np.zeros(got.shape, bool)
    bad[3, :4] = True                  # row 3: the last of sequence 1's three
    bad[4, 4:, 9] = True
    bad[5, 3] = True
    assert np.isfinite(got[~bad]).all()
    assert np.isnan(got[3, :4]).all() and not np.isfinite(got[4, 4:, 9]).any() and np.isnan(got[5, 3]).all()
    b.check(everything, rows={0, 1, 2})


@pytest.mark.parametrize("op", ["pages", "prefix", "prefix_cuda_cores"])
@pytest.mark.parametrize("scale", [0.0, -0.3, 4.0])
def test_scales_of_any_sign_and_peaked_scores(hp, op, scale):
    kernel = "cuda_cores" if op.endswith("cores") else "tensor_cores"
    b = make(hp, [(3, 300)], [20, 0, 7], 1, 8, 64, 16, "f16", kernel, seed=9, k_scale=3.0)
    b.scale = scale
    if op == "pages":
        b = Batch(hp, [320, 300, 307], 1, 8, 64, 16, "f16", seed=9, k_scale=3.0)
        b.scale = scale
        sel = lists(b, 20, holes=False)
        run_pages(b, sel)
        b.check(list_tokens(b, sel))
    else:
        run(b)
        b.check(everything)
    assert b.code() == "HP_OK"


def test_a_rising_score_moves_the_reference_in_every_block(hp):
    """Keys that grow along the prefix: every block of 128 keys, and every block of a warp, rescales."""
    import torch
    for kernel in ("tensor_cores", "cuda_cores"):
        b = make(hp, [(3, 1500)], [40, 0, 9], 1, 2, 128, 16, kernel=kernel, seed=10)
        for s in range(3):
            for t in range(int(b.lens[s])):
                own = b.lead[s] if t < 1500 else s
                b.hk[int(b.table[b.ptr[own] + t // 16]), t % 16, 0] = t / 400.0
        b.hq[:] = 1.0
        b.k.copy_(b.hk), b.q.copy_(b.hq)
        run(b)
        assert b.code() == "HP_OK"
        b.check(everything)


# ------------------------------------------------------- pools, pages and rows at their edges
def test_pool_rows_past_32_bits(hp):
    """Rows whose element offsets pass 2^32 (page 2,100,000 of 16 x 2 x 64 elements: 4.3e9)."""
    import torch
    P, H, D, pages = 16, 2, 64, 2_200_000
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 20 GB of free device memory")
    b = make(hp, [(3, 100)], [30, 7, 0], H, 4, D, P, seed=11)
    place = torch.from_numpy(np.random.default_rng(2).permutation(100_000)[:b.pages] + 2_100_000)
    for name in ("k", "v"):
        big = torch.empty((pages, P, H, D), dtype=torch.bfloat16, device="cuda")
        big[place.cuda()] = getattr(b, name)
        setattr(b, name, big)
    b.d_table = b.dev(place.numpy()[b.table])
    b.pages = pages
    b.desc = b.describe()
    run(b)
    assert b.code() == "HP_OK"
    b.check(everything)
    b.desc = b.describe(flags=hp.ATTN_CUDA_CORES)
    b.out.fill_(7.0)
    run(b)
    b.check(everything)
    bounds = torch.zeros((pages, H, 2, D), dtype=torch.bfloat16, device="cuda")
    assert hp.hp_page_bounds(b.desc, None, 3, bounds, b.status) == 0 and b.code() == "HP_OK"
    for s, n in enumerate(b.lens):
        j = (int(n) - 1) // P
        rows = b.hk[int(b.table[b.ptr[s] + j]), :int(n) - j * P]
        lo = 0 if s == 0 or j * P >= 100 else 100 - j * P  # (this batch holds a prefix's end in the first sequence alone)
        if lo == 0:
            got = bounds[int(b.d_table[b.ptr[s] + j])].cpu()
            assert (got[:, 0] == rows.amax(0)).all() and (got[:, 1] == rows.amin(0)).all()


def test_pools_in_host_memory(hp):
    """K and V in page-locked host memory, read in place."""
    b = Batch(hp, [200, 33, 90], 2, 4, 128, 16, seed=12, host=True)
    sel = lists(b, 5)
    run_pages(b, sel)
    assert b.code() == "HP_OK"
    b.check(list_tokens(b, sel))
    got, before = run_bounds(b, [50, 1, 0])
    check_bounds(b, [50, 1, 0], got, before)
    g = make(hp, [(2, 50), (1, 9)], [7, 30, 2], 2, 4, 64, 16, host=True)
    run(g)
    assert g.code() == "HP_OK"
    g.check(everything)


def test_outputs_stay_within_their_buffers(hp):
    """Guards around every output."""
    import torch
    from conftest import guarded, guards_intact
    b = make(hp, [(3, 50)], [7, 0, 9], 2, 3, 64, 16, "f16", nq=[1, 1, 2])
    sel = lists(b, 3)

    def window(t, fill=0xEE):
        n = t.numel() * t.element_size()
        buf, w = guarded(n)
        return buf, n, w.view(t.dtype).view(t.shape)

    for op in ("pages", "prefix", "bounds", "scores", "select"):
        if op in ("pages", "prefix"):
            buf, n, b.out = window(b.out)
            run_pages(b, sel) if op == "pages" else run(b)
        elif op == "bounds":
            buf, n, o = window(make_bounds(b))
            hp.hp_page_bounds(b.desc, b.d_q_ptr, b.T, o, b.status)
        elif op == "scores":
            buf, n, o = window(torch.zeros((b.T, 2, 4), device="cuda"))
            d = make_bounds(b).cuda()
            assert hp.hp_page_scores(b.describe(pool=d), d, b.q, b.d_q_ptr, b.T, 6, b.scale, o, 4, b.status) == 0
        else:
            buf, n, o = window(torch.zeros((b.T, 2, 3), dtype=torch.int32, device="cuda"))
            x = torch.rand((b.T, 2, 4), device="cuda")
            assert hp.hp_select_pages(b.desc, b.d_q_ptr, b.T, x, 4, 1, 1, 3, o, b.status) == 0
        assert b.code() == "HP_OK", op
        assert guards_intact(buf, n), op


# --------------------------------------------------------------- streams, graphs, layers
def test_layers_behind_one_plan_and_two_graphs(hp):
    """One plan, two layers' pools, captured; a second graph with a workspace of its own; both replayed in
    turn and side by side, twice each, with inputs changed in between."""
    import torch
    batches = [make(hp, [(20, 500), (9, 100)], [i % 37 for i in range(29)], 2, 4, 128, 16, seed=20 + i) for i in range(2)]
    for b in batches:  # a second layer: K and V exchanged
        b.out2, b.ws = torch.zeros_like(b.out), workspace(b)
        b.desc2 = b.describe(pool=b.v)

    def step(b):
        assert hp.hp_attention_prefix_plan(b.desc, b.d_group, b.d_prefix, 2, None, b.T, 8, b.ws, b.status) == 0
        for d, v, o in ((b.desc, b.v, b.out), (b.desc2, b.k, b.out2)):
            assert hp.hp_attention_prefix_planned(d, v, b.d_group, b.d_prefix, 2, b.q, None, b.T, 8, b.scale, o, b.ws,
                                                  b.status) == 0

    def check(b):
        assert b.code() == "HP_OK"
        b.check(everything, rows={0, 13, 28})
        b.hk, b.hv = b.hv, b.hk
        b.check(everything, rows={1, 20}, out=b.out2)
        b.hk, b.hv = b.hv, b.hk

    graphs, streams = [], [torch.cuda.Stream(), torch.cuda.Stream()]
    for b, st in zip(batches, streams):
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            step(b)
        st.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            step(b)
        graphs.append(g)
    for turn in range(2):
        for b in batches:
            b.hq = torch.randn(b.hq.shape, generator=torch.Generator().manual_seed(turn)).to(b.dt)
            b.q.copy_(b.hq)
            b.out.fill_(7.0), b.out2.fill_(7.0)
        torch.cuda.synchronize()
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
                g.replay()
        torch.cuda.synchronize()
        for b in batches:
            check(b)


def test_the_same_call_gives_the_same_bits(hp):
    import torch
    b = make(hp, [(50, 900)], [(7 * i) % 90 for i in range(50)], 2, 8, 128, 16, seed=30)
    sel = lists(b, 40)
    outs = []
    for _ in range(3):
        run(b)
        outs.append([b.out.clone()])
        run_pages(b, sel)
        outs[-1].append(b.out.clone())
    for o in outs[1:]:
        # (bits: the lists name slots that hold NaN, the copies of the prefix's end)
        assert all(torch.equal(x.view(torch.int16), y.view(torch.int16)) for x, y in zip(o, outs[0]))


def test_a_wait_that_runs_out_is_reported(hp):
    """The loads of the first block are never issued: every role gives up, the call reports it, the next one
    is right."""
    b = make(hp, [(20, 500)], [3] * 20, 1, 8, 128, 16, seed=31)
    b.desc = b.describe(flags=hp.TEST_STALL | hp.ATTN_TENSOR_CORES)
    run(b)
    assert b.code() == "HP_ERR_TIMEOUT"
    b.desc = b.describe()
    run(b)
    assert b.code() == "HP_OK"
    b.check(everything, rows={0, 19})


# ------------------------------------------------------------------------ all together
@pytest.mark.parametrize("graph", [False, True])
def test_decode_steps_over_selected_pages(hp, graph):
    """Prompts, then decode steps: tables, norm + rotation + append, bounds, scores, selection, attention over
    the selected pages, on one stream; against 64 bits from the stored keys on.  With as many pages as there
    are, attention over all of them by hp_attention_decode agrees."""
    import torch
    from test_gpu_step import make_step
    P, H, G, D, k = 16, 2, 4, 128, 6
    lens = np.array([150, 40, 97, 0, 201])
    S = len(lens)
    gen = torch.Generator().manual_seed(40)
    rnd = lambda *s: torch.randn(s, generator=gen).to(torch.bfloat16).cuda()  # noqa: E731
    pages, need = 120, -(-lens // P)
    perm = np.random.default_rng(3).permutation(pages).astype(np.int64)
    kp, vp = rnd(pages, P, H, D), rnd(pages, P, H, D)
    bounds = torch.full((pages, H, 2, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    table = perm[:need.sum()]
    free = list(perm[need.sum():])
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda().to(torch.int32)  # noqa: E731
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ptr = np.concatenate([[0], np.cumsum(need)])
    d0 = hp.PagedDesc(kp, dev(table), dev(ptr), dev(lens), num_pages=pages, page_size=P, num_heads=H, head_dim=D,
                      dtype="bf16", index_type=0)
    new = dev(np.concatenate([[0], np.cumsum(lens)]))
    assert hp.hp_page_bounds(d0, new, int(lens.sum()), bounds, status) == 0 and int(status.item()) == 0
    cos = torch.from_numpy(step_ref.cos_sin(400, D)).cuda()
    for step in range(3):
        fp = dev(free)
        e = lambda n, t=torch.int32: torch.full((n,), -5, dtype=t, device="cuda")  # noqa: E731
        t_out, p_out, l_out, n_out = e(80), e(S + 1), e(S), e(S + 1)
        slots, pos, tot = e(S, torch.int64), e(S), e(3, torch.int64)
        sd = hp.step_desc(block_table=dev(table), seq_ptr=dev(ptr), seq_lens=dev(lens), new_lens=dev(np.ones(S)),
                          free_pages=fp, page_size=P, index_type=0, table_out=t_out, seq_ptr_out=p_out, lens_out=l_out,
                          new_ptr_out=n_out, slot_map=slots, positions=pos, totals=tot)
        rc, n = hp.hp_step_tables_workspace_bytes(S)
        ws = torch.empty(n, dtype=torch.uint8, device="cuda")
        qkv = rnd(S, (H * G + 2 * H) * D)
        q, kk, vv = qkv.split([H * G * D, H * D, H * D], 1)
        q_out = torch.empty((S, H * G, D), dtype=torch.bfloat16, device="cuda")
        qd = hp.qk_desc(q=q, k=kk, v=vv, q_out=q_out.view(S, -1), num_q_heads=H * G, num_kv_heads=H, head_dim=D,
                        dtype="bf16", slot_map=slots, k_pool=kp, v_pool=vp, num_pages=pages, page_size=P)
        rope = hp.rope_desc(cos_sin=cos, positions=pos, sections=[D // 2])
        max_pages, scale = 20, D ** -0.5
        grown = int(np.maximum(need, -(-(lens + 1) // P)).sum())
        desc = hp.PagedDesc(kp, t_out, p_out, l_out, num_pages=pages, page_size=P, num_heads=H, head_dim=D, dtype="bf16",
                            index_type=0, table_len=grown)
        sc = torch.zeros((S, H, max_pages), device="cuda")
        sel = torch.zeros((S, H, k), dtype=torch.int32, device="cuda")
        all_sel = torch.zeros((S, H, max_pages), dtype=torch.int32, device="cuda")
        out, out_all = torch.zeros_like(q_out), torch.zeros_like(q_out)

        def calls():
            for rc in (hp.hp_step_tables(sd, ws, status), hp.hp_qk_norm_rope_append(qd, rope, status),
                       hp.hp_page_bounds(desc, None, S, bounds, status),
                       hp.hp_page_scores(desc, bounds, q_out, None, S, H * G, scale, sc, max_pages, status),
                       hp.hp_select_pages(desc, None, S, sc, max_pages, 1, 2, k, sel, status),
                       hp.hp_attention_pages(desc, vp, q_out, None, S, H * G, scale, sel, k, out, status),
                       hp.hp_select_pages(desc, None, S, sc, max_pages, 1, 2, max_pages, all_sel, status),
                       hp.hp_attention_pages(desc, vp, q_out, None, S, H * G, scale, all_sel, max_pages, out_all, status)):
                assert rc == 0

        if graph:
            st = torch.cuda.Stream()
            st.wait_stream(torch.cuda.current_stream())
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=st):
                calls()
            g.replay()
        else:
            calls()
        torch.cuda.synchronize()
        assert int(status.item()) == 0
        took = int(tot[2].item())
        free = free[took:]
        table, ptr, lens = (x.cpu().numpy().astype(np.int64) for x in (t_out[:grown], p_out, l_out))
        need = np.diff(ptr)
        hk, hv, hq = kp.double().cpu().numpy(), vp.double().cpu().numpy(), q_out.double().cpu().numpy()
        hb, x = bounds.cpu(), sc.double().cpu().numpy()
        for s in range(S):
            pg = table[ptr[s]:ptr[s + 1]]
            m = -(-int(lens[s]) // P)
            for j in range(m):
                rows = kp[int(pg[j]), :min(P, int(lens[s]) - j * P)].cpu()
                assert (hb[int(pg[j]), :, 0] == rows.amax(0)).all() and (hb[int(pg[j]), :, 1] == rows.amin(0)).all()
            for h in range(H):
                b64 = hb[pg[:m], h].double().numpy()
                want, tol = ref.scores(hq[s, h * G:(h + 1) * G], b64[:, 0], b64[:, 1], scale)
                assert (np.abs(x[s, h, :m] - want) <= tol).all()
                picked = sel[s, h].tolist()
                assert picked == ref.select(x[s, h], m, 1, 2, k)
                t = np.concatenate([np.arange(j * P, min((j + 1) * P, lens[s])) for j in picked if j >= 0]).astype(np.int64)
                for o, toks in ((out, t), (out_all, np.arange(lens[s]))):
                    at = pg[toks // P], toks % P
                    for g in range(G):
                        w, tol = ref.attention(hq[s, h * G + g], hk[at][:, h], hv[at][:, h], scale, "bf16")
                        assert (np.abs(o[s, h * G + g].double().cpu().numpy() - w) <= tol).all()
        # hp_attention_decode over everything: fp32 results, within both operators' rounding of out_all
        rc, n = hp.hp_attention_decode_workspace_bytes(desc, H * G)
        full = torch.zeros((S, H * G, D), device="cuda")
        assert hp.hp_attention_decode(desc, vp, q_out, H * G, scale, full, torch.empty(n, dtype=torch.uint8, device="cuda"),
                                      status) == 0
        assert int(status.item()) == 0
        assert float((full - out_all.float()).abs().max()) <= 2 * 2.0 ** -8 * float(vp.float().abs().max())
