"""What the operators of long contexts leave out where a page does not hold: the page (bounds, scores) or the
query's K/V head (lists), with everything else as it should be."""
import numpy as np
import pytest

import pages_ref as ref
from pages_ref import Batch
from test_gpu_pages import check_bounds, list_tokens, make_bounds, run_bounds, run_pages, run_scores

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("many", [False, True])
def test_bounds_leave_out_the_page_alone(hp, many):
    """Prompts of seven pages: one entry outside the pool, one slice that ends a page early."""
    S = 200 if many else 3
    b = Batch(hp, [100] * S, 2, 1, 64, 16, seed=6)
    b.d_table[7 + 2] = b.pages
    b.d_ptr[S] -= 1                      # the last sequence's seventh page
    b.desc = b.describe(table_len=7 * S - 1)
    got, before = run_bounds(b, [100] * S)
    assert b.code() == "HP_ERR_LEN"
    left = [int(b.table[7 + 2]), int(b.table[7 * S - 1])]
    assert (got[left] == before[left]).all()
    for j, page in enumerate(left):      # (as if they had been there)
        rows = b.hk[page, :16 if j == 0 else 4]
        got[page, :, 0], got[page, :, 1] = rows.amax(0), rows.amin(0)
    check_bounds(b, [100] * S, got, before)


@pytest.mark.parametrize("many", [False, True])
def test_scores_leave_out_the_page_alone(hp, many):
    S = 300 if many else 4
    b = Batch(hp, [100] * S, 2, 3, 64, 16, seed=7)
    b.d_table[7 + 3] = b.pages
    bounds = make_bounds(b)
    got = run_scores(b, bounds.cuda(), 9)
    assert b.code() == "HP_ERR_PAGE_ID"
    q, bd = b.hq.double().numpy(), bounds.double().numpy()
    for r in (0, 1, S - 1):
        for h in range(2):
            pages = b.table[7 * r:7 * r + 7]
            x, tol = ref.scores(q[r, 3 * h:3 * h + 3], bd[pages, h, 0], bd[pages, h, 1], b.scale)
            fine = np.arange(7) != (3 if r == 1 else -1)
            assert (np.abs(got[r, h, :7] - x) <= tol)[fine].all()
            assert (got[r, h, :7][~fine] == -77.0).all() and (got[r, h, 7:] == -77.0).all()


@pytest.mark.parametrize("many", [False, True])
def test_lists_leave_out_the_head_that_names_a_page_that_does_not_hold(hp, many):
    import torch
    S = 300 if many else 4
    b = Batch(hp, [100] * S, 2, 2, 64, 16, seed=8)
    b.d_table[7 + 3] = b.pages
    sel = np.tile(np.array([0, 2, 5], np.int32), (S, 2, 1))
    sel[1, 1] = [3, 1, -1]               # head 1 of row 1 alone meets the bad entry
    sel = torch.from_numpy(sel)
    run_pages(b, sel)
    assert b.code() == "HP_ERR_PAGE_ID"
    assert (b.out[1, 2:] == 7.0).all()
    tokens = list_tokens(b, sel)
    b.check(tokens, rows={0, 2, S - 1})
    k, v = b.token_rows(1, tokens(1, 1, 100, 0))
    for h in range(2):
        o, tol = ref.attention(b.hq[1, h].double().numpy(), k[:, 0], v[:, 0], b.scale, "bf16")
        assert (np.abs(b.out[1, h].double().cpu().numpy() - o) <= tol).all()
