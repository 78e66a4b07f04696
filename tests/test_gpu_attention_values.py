"""Attention over page lists and behind shared prefixes at values where a softmax's form matters: scores
of minus infinity, and weights that differ by less than a step of the pool's type."""
import numpy as np
import pytest

import step_ref
from pages_ref import Batch
from test_gpu_pages import run_pages
from test_gpu_prefix import make, run

pytestmark = pytest.mark.gpu

OPS = ["pages", "prefix_cuda_cores", "prefix_tensor_cores"]


def batch(hp, op, S, pre, tails, H, G, D, dtype, **kw):
    """One group behind a prefix of `pre` tokens; for `pages` the same lengths, nothing shared."""
    if op == "pages":
        return Batch(hp, pre + np.array(tails), H, G, D, 16, dtype, **kw)
    return make(hp, [(S, pre)], tails, H, G, D, 16, dtype, op[len("prefix_"):], **kw)


def attend(b, op):
    """The operator over everything that each query sees."""
    import torch
    b.k.copy_(b.hk), b.v.copy_(b.hv), b.q.copy_(b.hq)
    if op == "pages":
        n = -(-b.lens // 16)
        sel = torch.full((b.T, b.H, int(n.max())), -1, dtype=torch.int32)
        row = 0
        for s, m in enumerate(b.nq):
            for _ in range(m):
                sel[row, :, :n[s]] = torch.arange(int(n[s]))
                row += 1
        run_pages(b, sel)
    else:
        run(b)
    assert b.code() == "HP_OK"
    return b.out.double().cpu().numpy()


def place(b, s, t):
    own = b.lead[s] if t < b.prefix[s] else s
    return int(b.table[b.ptr[own] + t // 16]), t % 16


def definition(b, row, s, seen, head):
    """softmax(x) V in 64 bits, infinities and all."""
    k, v = b.token_rows(s, np.arange(seen))
    q = b.hq[row, head].double().numpy()
    with np.errstate(invalid="ignore"):
        x = k[:, head // b.G] @ q * b.scale
        p = np.exp(x - x.max())
        return (p[:, None] * v[:, head // b.G]).sum(0) / p.sum()


# ------------------------------------------------------------------- minus infinity
@pytest.mark.parametrize("op", OPS)
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("S,pre,tails,G,D", [(1, 1, [0], 1, 128), (3, 40, [1, 0, 60], 4, 128), (2, 2000, [5, 9], 8, 64),
                                             (70, 300, list(range(70)), 4, 128)])
def test_rows_whose_scores_are_all_minus_infinity(hp, op, dtype, S, pre, tails, G, D):
    """Every key of K/V head 0 is infinite against its queries (0 / 0), those of head 1 are not.  Parts of one
    row, halves of a tile, tiles of more than 128 rows."""
    b = batch(hp, op, S, pre, tails, 2, G, D, dtype, seed=S)
    b.hk[:, :, 0, 3] = float("-inf")
    b.hq[:, :G, 3] = 1.0
    got = attend(b, op)
    assert np.isnan(got[:, :G]).all()
    assert np.isfinite(got[:, G:]).all()
    for s in range(min(S, 8)):
        want, tol = step_ref.attention_row(b.hq[s, G].double().numpy(),
                                           *(x[:, 1] for x in b.token_rows(s, np.arange(int(b.lens[s])))), b.scale, dtype)
        assert (np.abs(got[s, G] - want) <= tol).all()


@pytest.mark.parametrize("op", OPS)
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("first,last", [(0, 16), (0, 700), (128, 384), (500, 900), (899, 900), (0, 899)])
def test_tokens_whose_scores_are_minus_infinity(hp, op, dtype, first, last):
    """A run of tokens weighs nothing; the value of one of them, infinite in one dimension, counts as zero
    times infinity, wherever the run is cut.  One sequence (8 parts, 2 halves), 700 of its tokens a prefix."""
    b = batch(hp, op, 1, 700, [200], 1, 4, 128, dtype, seed=first + last)
    for t in range(first, last):
        p, i = place(b, 0, t)
        b.hk[p, i, 0, 3] = float("-inf")
    b.hq[:, :, 3] = 1.0
    p, i = place(b, 0, last - 1)
    b.hv[p, i, 0, 9] = float("inf")
    got = attend(b, op)
    for h in range(4):
        want = definition(b, 0, 0, 900, h)
        assert np.isnan(want[9]) and np.isnan(got[0, h, 9])
        fine = np.arange(128) != 9
        k, v = b.token_rows(0, np.array([t for t in range(900) if not first <= t < last]))
        o, tol = step_ref.attention_row(b.hq[0, h].double().numpy(), k[:, 0], v[:, 0], b.scale, dtype)
        assert np.abs(want[fine] - o[fine]).max() <= 1e-12
        assert (np.abs(got[0, h] - o) <= tol)[fine].all()


@pytest.mark.parametrize("op", OPS)
def test_queries_without_tokens_beside_minus_infinity(hp, op):
    """A query that sees nothing has zeros; one whose only token scores minus infinity has NaN; plus infinity
    is NaN too."""
    b = batch(hp, op, 3, 0, [0, 1, 40], 1, 2, 64, "bf16", seed=5)
    b.hk[:, :, 0, 3] = float("-inf")
    b.hq[:, :, 3] = 1.0
    b.hq[2, 1, 3] = -1.0
    got = attend(b, op)
    assert (got[0] == 0.0).all() and np.isnan(got[1:]).all()


@pytest.mark.parametrize("op", OPS)
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("t", [0, 77, 230])
def test_an_infinite_value_with_a_weight_is_infinite(hp, op, dtype, t):
    """Its token's key is zero, so that its weight is e^-4 of the largest or so: both parts of it times the infinity
    have the infinity's sign."""
    b = batch(hp, op, 2, 200, [31, 31], 1, 4, 128, dtype, seed=t)
    for s in range(2):
        p, i = place(b, s, t)
        b.hk[p, i], b.hv[p, i, 0, 9], b.hv[p, i, 0, 10] = 0.0, float("inf"), float("-inf")
    got = attend(b, op)
    assert (got[:, :, 9] == np.inf).all() and (got[:, :, 10] == -np.inf).all()
    assert np.isfinite(np.delete(got, (9, 10), 2)).all()


# --------------------------------------------------------------------------- weights
@pytest.mark.parametrize("op", OPS[:2])
@pytest.mark.parametrize("dtype,step", [("bf16", 2.0 ** -10), ("f16", 2.0 ** -13)])
@pytest.mark.parametrize("S,pre,tails,G,D", [(1, 2, [0], 1, 128), (3, 40, [2, 0, 60], 4, 128), (2, 2000, [6, 10], 8, 64),
                                             (1, 96, [32], 16, 64), (2, 640, [64, 2], 3, 256),
                                             (70, 300, [2 * i for i in range(70)], 4, 128)])
def test_weights_keep_more_bits_than_the_pool(hp, op, dtype, step, S, pre, tails, G, D):
    """Half of the tokens score 0 and have value 1, half -step and -1: out = (1 - e^-step) / (1 + e^-step), about
    step / 2.  Rounded to the pool's type the two weights are equal (step is an eighth of bf16's 2^-7 above 1 and
    of f16's 2^-10, a quarter of those below), and out is zero.

    The scores are exact.  A weight as two parts of the pool's type: the first leaves less than u of it (u = 2^-7,
    2^-10, a unit of the last place), the second is rounded to half a unit of its own, u^2 / 2, with 2^-20
    of the weight besides.  The scaled score and the exponential are off by less than 2^-21.  The value sum of n tokens
    adds ones of both signs in turn, 16 at a time, so that its partial sums stay below 16 and its n / 8
    additions (both parts') are off by 2^-20 each at most: 2^-23 of the n that it is divided by, and as much for
    what joins the parts.  The sum of the weights is off by a factor.  The result is rounded once: half a unit."""
    b = batch(hp, op, S, pre, tails, 1, G, D, dtype, seed=S)
    for s in range(S):
        for t in range(int(b.lens[s])):
            p, i = place(b, s, t)
            b.hk[p, i], b.hv[p, i] = 0.0, 1.0 - 2 * (t % 2)
            b.hk[p, i, 0, 0] = -float(t % 2)
    b.hq[:] = 0.0
    b.hq[:, :, 0] = 1.0
    b.scale = step
    got = attend(b, op)
    want = np.tanh(step / 2)
    u = {"bf16": 2.0 ** -7, "f16": 2.0 ** -10}[dtype]
    tol = want * u / 2 + u * u / 2 + 2.0 ** -20 + 2.0 ** -21 + 2.0 ** -22
    assert tol < want / 4
    assert np.abs(got - want).max() <= tol, np.abs(got - want).max() / want
