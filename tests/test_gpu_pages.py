"""GPU parity of the operators that read some of a long sequence's pages: bounds, scores, selection,
attention over lists (pages_ref.py holds the plain 64-bit forms and the error bounds)."""
import numpy as np
import pytest

import pages_ref as ref
from pages_ref import Batch, visible

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------------- bounds
def run_bounds(b, new, it_null=False):
    import torch
    new = np.array(new, np.int64)
    gen = torch.Generator().manual_seed(5)
    bounds = torch.randn((b.pages, b.H, 2, b.D), generator=gen).to(b.dt).cuda()
    before = bounds.cpu()
    ptr = None if it_null else b.dev(np.concatenate([[0], np.cumsum(new)]))
    total = len(new) if it_null else int(new.sum())
    assert b.hp.hp_page_bounds(b.desc, ptr, total, bounds, b.status) == 0
    return bounds.cpu(), before


def check_bounds(b, new, got, before):
    want = before.clone()
    for s, n in enumerate(b.lens):
        if new[s] == 0:
            continue
        for j in range(int(n - new[s]) // b.P, -(-int(n) // b.P)):
            page = int(b.table[b.ptr[s] + j])
            rows = b.hk[page, :min(b.P, int(n) - j * b.P)]
            want[page, :, 0], want[page, :, 1] = rows.amax(0), rows.amin(0)
    assert (got == want).all()


@pytest.mark.parametrize("it", [0, 1])
@pytest.mark.parametrize("dtype,lens,new,H,D,P", [
    ("bf16", [1], [1], 1, 64, 8), ("f16", [17, 0, 1, 16], [1, 0, 1, 16], 8, 128, 16),
    ("bf16", [100, 64, 65, 200, 33], [30, 64, 1, 0, 33], 3, 64, 16), ("f16", [1000, 7], [999, 7], 5, 256, 64),
    ("bf16", [300, 299], [300, 2], 16, 128, 1), ("f16", [77, 600], [50, 600], 2, 64, 513), ("bf16", [41], [39], 1, 64, 5),
])
def test_page_bounds(hp, dtype, lens, new, H, D, P, it):
    b = Batch(hp, lens, H, 1, D, P, dtype, it=it, seed=len(lens))
    got, before = run_bounds(b, new)
    assert b.code() == "HP_OK"
    check_bounds(b, new, got, before)


def test_page_bounds_of_last_tokens(hp):
    """Without offsets every sequence's last token is new, and an empty one has none."""
    lens = [1, 0, 16, 17, 500] * 30
    b = Batch(hp, lens, 4, 1, 128, 16)
    got, before = run_bounds(b, np.minimum(lens, 1), it_null=True)
    assert b.code() == "HP_OK"
    check_bounds(b, np.minimum(lens, 1), got, before)


def test_page_bounds_of_a_large_prompt(hp):
    """More entries than one CTA looks at (the status is cleared before the kernel)."""
    lens = [9000, 3, 5000]
    b = Batch(hp, lens, 2, 1, 128, 16, "f16")
    got, before = run_bounds(b, lens)
    assert b.code() == "HP_OK"
    check_bounds(b, lens, got, before)


def test_page_bounds_of_keys_that_are_not_finite(hp):
    import torch
    b = Batch(hp, [20], 1, 1, 64, 16)
    page = int(b.table[0])
    for slot, d, x in ((3, 0, float("nan")), (4, 1, float("inf")), (5, 1, -float("inf")), (6, 2, float("-inf"))):
        b.hk[page, slot, 0, d] = x
    b.k.copy_(b.hk)
    got, _ = run_bounds(b, [20])
    assert torch.isnan(got[page, 0, :, 0]).all()
    assert got[page, 0, 0, 1] == float("inf") and got[page, 0, 1, 1] == -float("inf")
    assert got[page, 0, 1, 2] == -float("inf") and torch.isfinite(got[page, 0, 0, 2])
    assert torch.isfinite(got[page, 0, :, 3:]).all()


# ------------------------------------------------------------------------- scores
def make_bounds(b, seed=3):
    import torch
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn((2, b.pages, b.H, b.D), generator=gen).to(b.dt)
    return torch.stack([torch.maximum(x[0], x[1]), torch.minimum(x[0], x[1])], 2).contiguous()


def run_scores(b, bounds, max_pages):
    import torch
    out = torch.full((b.T, b.H, max_pages), -77.0, device="cuda")
    desc = b.describe(pool=bounds)
    rc = b.hp.hp_page_scores(desc, bounds, b.q, b.offsets(), b.T, b.H * b.G, b.scale, out, max_pages, b.status)
    assert rc == 0
    return out.cpu().numpy()


def check_scores(b, bounds, got, skip=()):
    q, bd = b.hq.double().numpy(), bounds.double().cpu().numpy()
    left = np.ones(got.shape, bool)
    for row, s, seen in visible(b.lens, b.nq):
        n = -(-seen // b.P)
        if row in skip:
            continue
        pages = b.table[b.ptr[s]:b.ptr[s] + n]
        for h in range(b.H):
            x, tol = ref.scores(q[row, h * b.G:(h + 1) * b.G], bd[pages, h, 0], bd[pages, h, 1], b.scale)
            g = got[row, h, :n]
            fine = np.isfinite(x)
            assert (np.abs(g[fine] - x[fine]) <= tol[fine]).all(), (row, h)
            assert (np.isnan(g) == np.isnan(x)).all() and (g[np.isinf(x)] == x[np.isinf(x)]).all(), (row, h)
        left[row, :, :n] = False
    assert (got[left] == -77.0).all()


@pytest.mark.parametrize("it", [0, 1])
@pytest.mark.parametrize("dtype,lens,nq,H,G,D,P,behind", [
    ("bf16", [5], None, 1, 1, 64, 16, 0), ("f16", [1000, 0, 1, 17], None, 8, 4, 128, 16, 0),
    ("bf16", [300, 77, 0, 256], [1, 2, 1, 3], 3, 5, 64, 8, 2), ("f16", [4097, 100], [3, 0], 2, 16, 256, 32, 0),
    ("bf16", [40, 2, 700], [2, 3, 1], 9, 9, 128, 5, 1), ("f16", [2000], None, 4, 8, 64, 1, 0),
])
def test_page_scores(hp, dtype, lens, nq, H, G, D, P, behind, it):
    b = Batch(hp, lens, H, G, D, P, dtype, nq=nq, it=it, behind=behind, seed=7)
    bounds = make_bounds(b)
    most = max(1, int((-(-b.lens // P)).max())) + 3
    got = run_scores(b, bounds.cuda(), most)
    assert b.code() == "HP_OK"
    check_scores(b, bounds, got)


def test_page_scores_of_many_pages(hp):
    """Enough pages for several blocks a warp, and more than one CTA looks at."""
    lens = np.random.default_rng(1).integers(0, 9000, 40)
    b = Batch(hp, lens, 8, 2, 64, 4, seed=9)
    bounds = make_bounds(b)
    got = run_scores(b, bounds.cuda(), 2250)
    assert b.code() == "HP_OK"
    check_scores(b, bounds, got)


def test_page_scores_of_bounds_that_are_not_finite(hp):
    """An infinite bound counts on the side of the query that meets it; a NaN gives NaN."""
    b = Batch(hp, [16 * 12], 2, 4, 64, 16, seed=2)
    bounds = make_bounds(b)
    inf, page = float("inf"), [int(x) for x in b.table]
    bounds[page[1], 0, 1, 5] = -inf
    bounds[page[2], 0, 0, 6] = inf
    bounds[page[3], 0, 0, 7] = float("nan")
    bounds[page[3], 0, 1, 7] = float("nan")
    bounds[page[4], 1, 0, 8], bounds[page[4], 1, 1, 8] = inf, -inf
    bounds[page[5], 1, 0, 9], bounds[page[5], 1, 1, 9] = -inf, -inf
    got = run_scores(b, bounds.cuda(), 12)
    check_scores(b, bounds, got)
    assert np.isnan(got[0, 0, 3]) and np.isposinf(got[0, 1, 4])
    b.hq[0, 5, 3] = float("nan")  # a query of the second group
    b.q.copy_(b.hq)
    got = run_scores(b, make_bounds(b).cuda(), 12)
    assert np.isnan(got[0, 1]).all() and np.isfinite(got[0, 0]).all()


def test_no_token_scores_above_its_page(hp):
    """What the bounds are for: bounds and scores together, against every token's score."""
    lens = [333, 64, 1]
    b = Batch(hp, lens, 2, 3, 128, 16, "f16", seed=12)
    got, _ = run_bounds(b, lens)
    x = run_scores(b, got.cuda(), 21)
    q = b.hq.double().numpy()
    for row, s, seen in visible(b.lens, b.nq):
        k, _ = b.token_rows(s, np.arange(seen))
        for h in range(b.H):
            top = (np.einsum("gd,td->gt", q[row, 3 * h:3 * h + 3], k[:, h]) * b.scale).max(0)
            over = top - x[row, h][np.arange(seen) // b.P]
            assert over.max() <= 257 * 2.0 ** -23 * 128 * 16 * b.scale


# ---------------------------------------------------------------------- selection
def run_select(hp, n, H, x, sinks, recent, k, P=16, nq=None, it=0, behind=0, max_pages=None):
    import torch
    n = np.array(n, np.int64)
    tt = torch.int64 if it else torch.int32
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda().to(tt)  # noqa: E731
    nq = np.ones(len(n), np.int64) if nq is None else np.array(nq, np.int64)
    lens = n * P - (np.arange(len(n)) % P) * (n > 0)
    T = int(nq.sum()) + behind
    desc = hp.PagedDesc(None, None, dev(np.zeros(len(n) + 1)), dev(lens), num_pages=0, page_size=P, num_heads=H,
                        head_dim=128, dtype="bf16", index_type=it, table_len=0)
    out = torch.full((T, H, k), -9, dtype=torch.int32, device="cuda")
    status = torch.full((1,), 99, dtype=torch.int32, device="cuda")
    ptr = None if behind == 0 and (nq == 1).all() else dev(np.concatenate([[0], np.cumsum(nq)]))
    rc = hp.hp_select_pages(desc, ptr, T, x.cuda(), x.shape[2], sinks, recent, k, out, status)
    assert rc == 0
    return out.cpu().numpy(), hp.status_name(int(status.item())), lens, nq


def check_select(x, got, lens, nq, H, P, sinks, recent, k):
    xs = x.double().numpy()
    row = 0
    for row, s, seen in visible(lens, nq):
        n = -(-seen // P)
        for h in range(H):
            assert got[row, h].tolist() == ref.select(xs[row, h], n, sinks, recent, k), (row, h, n)
    assert (got[int(nq.sum()):] == -9).all()


@pytest.mark.parametrize("it", [0, 1])
@pytest.mark.parametrize("n,H,sinks,recent,k,coarse", [
    ([1], 1, 0, 0, 1, 0), ([0, 5, 4, 6], 2, 1, 1, 5, 0), ([100, 64, 65, 3], 3, 1, 2, 64, 0.5),
    ([512, 300], 2, 0, 0, 299, 0.25), ([513, 2048, 2047], 1, 2, 4, 100, 4.0), ([8192, 8193, 100], 2, 0, 1, 512, 0),
    ([20000, 9000], 1, 3, 3, 1000, 0.5), ([700], 2, 4, 4, 8, 0), ([3000], 1, 0, 0, 2999, 1.0), ([50], 1, 0, 0, 1, 0),
])
def test_select_pages(hp, n, H, sinks, recent, k, coarse, it):
    import torch
    gen = torch.Generator().manual_seed(k)
    x = torch.randn((len(n), H, max(n) + 2), generator=gen) * 5
    if coarse:
        x = (x / coarse).round() * coarse  # (with zeros of both signs)
    got, code, lens, nq = run_select(hp, n, H, x, sinks, recent, k, it=it)
    assert code == "HP_OK"
    check_select(x, got, lens, nq, H, 16, sinks, recent, k)


@pytest.mark.parametrize("n", [90, 1000, 5000, 10000])
def test_select_pages_of_special_scores(hp, n):
    """Infinities, NaN, zeros of both signs, equal scores, the smallest numbers."""
    import torch
    rng = np.random.default_rng(n)
    pool = np.array([0.0, -0.0, np.inf, -np.inf, np.nan, 1.0, 1.0, -1.0, 1e-45, -1e-45, 3e38, -3e38], np.float32)
    x = torch.from_numpy(pool[rng.integers(0, len(pool), (3, 2, n))])
    x[1] = 0.0
    x[2, 1] = float("-inf")
    for k in (5, n // 3, n - 1):
        got, code, lens, nq = run_select(hp, [n, n, n], 2, x, 1, 1, k)
        assert code == "HP_OK"
        check_select(x, got, lens, nq, 2, 16, 1, 1, k)


def test_select_pages_of_drafted_queries(hp):
    import torch
    nq, P = [3, 0, 2, 1], 2
    n = [40, 9, 2, 600]
    x = torch.randn((8, 2, 600))
    got, code, lens, nq = run_select(hp, n, 2, x, 1, 1, 7, P=P, nq=nq, behind=2)
    assert code == "HP_OK"
    check_select(x, got, lens, nq, 2, P, 1, 1, 7)


# ---------------------------------------------------------------- attention of lists
def lists(b, k, seed=0, holes=True):
    """Page lists in any order, pages named twice, places without a page."""
    import torch
    rng = np.random.default_rng(seed)
    out = np.full((b.T, b.H, k), -1, np.int32)
    for row, s, seen in visible(b.lens, b.nq):
        n = -(-int(b.lens[s]) // b.P)
        for h in range(b.H):
            if n:
                out[row, h] = rng.integers(0, n, k)
                if holes:
                    out[row, h, rng.random(k) < 0.2] = -1 - rng.integers(0, 5)
    return torch.from_numpy(out)


def run_pages(b, sel, stream=None):
    rc = b.hp.hp_attention_pages(b.desc, b.v, b.q, b.offsets(), b.T, b.H * b.G, b.scale, sel.cuda(), sel.shape[2],
                                 b.out, b.status, stream)
    assert rc == 0, b.hp.status_name(rc)


def list_tokens(b, sel):
    sel = sel.numpy()

    def tokens(row, s, seen, h):
        j = sel[row, h][sel[row, h] >= 0].astype(np.int64)
        t = (j[:, None] * b.P + np.arange(b.P)).ravel()
        return t[t < seen]
    return tokens


@pytest.mark.parametrize("it", [0, 1])
@pytest.mark.parametrize("dtype,lens,nq,H,G,D,P,k,behind", [
    ("bf16", [1], None, 1, 1, 128, 16, 1, 0), ("f16", [100, 0, 1, 33], None, 2, 4, 128, 16, 3, 0),
    ("bf16", [500, 90, 257], [2, 1, 3], 8, 4, 128, 16, 12, 2), ("f16", [900, 31], [1, 4], 3, 8, 64, 8, 40, 0),
    ("bf16", [400, 5, 77], None, 4, 5, 256, 32, 6, 0), ("f16", [200], None, 1, 16, 64, 5, 17, 0),
    ("bf16", [333, 10], [2, 1], 2, 9, 128, 1, 50, 1), ("f16", [300, 20], None, 2, 11, 256, 7, 9, 0),
    ("bf16", [5000], None, 1, 2, 64, 4096, 2, 0), ("bf16", [3000, 2999], None, 1, 8, 128, 3, 700, 0),
])
def test_attention_pages(hp, dtype, lens, nq, H, G, D, P, k, behind, it):
    b = Batch(hp, lens, H, G, D, P, dtype, nq=nq, it=it, behind=behind, seed=k)
    sel = lists(b, k, seed=1)
    run_pages(b, sel)
    assert b.code() == "HP_OK"
    b.check(list_tokens(b, sel))


@pytest.mark.parametrize("S,H,k", [(1, 1, 8), (1, 1, 16), (1, 2, 64), (20, 8, 32), (40, 8, 8), (80, 8, 4)])
def test_attention_pages_cut_among_ctas(hp, S, H, k):
    """From one CTA to eight a (query, head)."""
    rng = np.random.default_rng(S)
    b = Batch(hp, rng.integers(1, 2000, S), H, 4, 128, 16, seed=3)
    sel = lists(b, k, seed=2)
    run_pages(b, sel)
    assert b.code() == "HP_OK"
    b.check(list_tokens(b, sel), rows=set(range(0, S, max(1, S // 5))))
