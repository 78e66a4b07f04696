"""Offsets that do not hold, where they are all that a call of the operators of long contexts looks at."""
import pytest

from pages_ref import Batch

pytestmark = pytest.mark.gpu

NAMES = ["bounds", "scores", "select", "pages"]


def call(hp, b, name, ptr, total):
    import torch
    x = torch.zeros((4, b.H, 8), device="cuda")
    sel = torch.zeros((4, b.H, 4), dtype=torch.int32, device="cuda")
    bounds = torch.zeros((b.pages, b.H, 2, b.D), dtype=b.dt, device="cuda")
    b.status.fill_(99)
    rc = {"bounds": lambda: hp.hp_page_bounds(b.desc, ptr, total, bounds, b.status),
          "scores": lambda: hp.hp_page_scores(b.desc, bounds, b.q, ptr, total, b.H * b.G, 1.0, x, 8, b.status),
          "select": lambda: hp.hp_select_pages(b.desc, ptr, total, x, 8, 0, 0, 4, sel, b.status),
          "pages": lambda: hp.hp_attention_pages(b.desc, b.v, b.q, ptr, total, b.H * b.G, 1.0, sel, 4, b.out, b.status)}[name]()
    assert rc == 0
    assert not x.any() and not sel.any() and not bounds.any() and (b.out == 7.0).all()
    return b.code()


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("ptr,code", [([0, 0, 0, 0], "OK"), ([0, 0, 0, 4], "ERR_NEW_PTR_END"),
                                      ([1, 1, 1, 1], "ERR_NEW_PTR_END"), ([0, 2, 1, 0], "ERR_NEW_PTR_ORDER")])
def test_offsets_of_no_rows(hp, name, ptr, code):
    """total_q (total_new) 0: no outputs, the offsets' verdict (the lowest code) all the same."""
    b = Batch(hp, [50, 60, 70], 2, 1, 64, 16, seed=3)
    assert call(hp, b, name, b.dev(ptr), 0) == "HP_" + code


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("first,total,code", [(0, 0, "OK"), (0, 4, "OK"), (1, 4, "ERR_NEW_PTR_START"),
                                              (5, 4, "ERR_NEW_PTR_END")])
def test_offsets_of_no_sequences(hp, name, first, total, code):
    """One entry, which is the first and the last; the rows (a padded batch) are nobody's."""
    b = Batch(hp, [50, 60, 70, 1], 2, 1, 64, 16, seed=3)
    b.desc = b.describe(num_seqs=0)
    assert call(hp, b, name, b.dev([first]), total) == "HP_" + code
