"""GPU parity of attention behind shared prefixes (pages_ref.py holds the plain 64-bit form and the
error bounds)."""
import numpy as np
import pytest

from pages_ref import Batch

pytestmark = pytest.mark.gpu


def make(hp, groups, tails, H, G, D, P, dtype="bf16", kernel="tensor_cores", **kw):
    """groups: (sequences, prefix); tails: each sequence's tokens behind it."""
    pre = np.repeat([p for _, p in groups], [n for n, _ in groups])
    flags = {"cuda_cores": hp.ATTN_CUDA_CORES, "tensor_cores": hp.ATTN_TENSOR_CORES, "default": 0}[kernel]
    return Batch(hp, pre + np.array(tails), H, G, D, P, dtype, groups=groups, flags=flags, **kw)


def workspace(b):
    import torch
    rc, n = b.hp.hp_attention_prefix_workspace_bytes(b.desc, len(b.groups), b.T, b.H * b.G)
    assert rc == 0
    return torch.full((n,), 0xEE, dtype=torch.uint8, device="cuda")


def run(b, ws=None, stream=None):
    ws = workspace(b) if ws is None else ws
    rc = b.hp.hp_attention_prefix(b.desc, b.v, b.d_group, b.d_prefix, len(b.groups), b.q, b.offsets(), b.T,
                                  b.H * b.G, b.scale, b.out, ws, b.status, stream)
    assert rc == 0, b.hp.status_name(rc)
    return ws


def everything(row, s, seen, h):
    return np.arange(seen)


@pytest.mark.parametrize("kernel", ["tensor_cores", "cuda_cores"])
@pytest.mark.parametrize("dtype,groups,tails,nq,H,G,D,P,it,behind", [
    ("bf16", [(1, 1)], [0], None, 1, 1, 128, 16, 0, 0),
    ("f16", [(2, 16)], [0, 5], None, 2, 4, 128, 16, 1, 0),
    ("bf16", [(3, 40)], [1, 0, 60], None, 8, 4, 128, 16, 0, 0),
    ("f16", [(1, 0), (2, 130), (4, 7)], [9, 3, 200, 1, 2, 0, 4], None, 2, 8, 64, 8, 0, 0),
    ("bf16", [(4, 300), (3, 0), (0, 50), (2, 129)], [1, 2, 3, 40, 0, 1, 77, 5, 6], None, 3, 3, 128, 32, 1, 0),
    ("f16", [(3, 257), (2, 128)], [4, 2, 9, 3, 17], [2, 1, 3, 2, 4], 4, 2, 128, 16, 0, 3),
    ("bf16", [(2, 500)], [33, 7], [1, 2], 1, 16, 64, 64, 0, 0),
    ("f16", [(2, 90), (1, 20)], [5, 8, 1], None, 2, 2, 256, 16, 0, 0),
    ("bf16", [(2, 93)], [5, 8], None, 2, 7, 128, 5, 0, 0),
    ("f16", [(40, 200), (30, 100)], list(range(70)), None, 2, 8, 128, 16, 0, 0),
    ("bf16", [(5, 1000)], [1, 1, 9, 0, 2], [0, 1, 2, 0, 1], 2, 4, 64, 24, 0, 2),
])
def test_attention_prefix(hp, kernel, dtype, groups, tails, nq, H, G, D, P, it, behind):
    b = make(hp, groups, tails, H, G, D, P, dtype, kernel, nq=nq, it=it, behind=behind, seed=len(tails))
    run(b)
    assert b.code() == "HP_OK"
    b.check(everything)


@pytest.mark.parametrize("kernel", ["tensor_cores", "cuda_cores"])
@pytest.mark.parametrize("S,H,G,D,pre,tail", [(130, 2, 4, 128, 700, 90), (33, 8, 8, 64, 2000, 40), (3, 1, 4, 128, 9000, 3),
                                              (300, 1, 1, 128, 260, 20)])
def test_attention_prefix_of_many_rows(hp, kernel, S, H, G, D, pre, tail):
    """Several tiles of rows, prefixes cut among workers."""
    rng = np.random.default_rng(S)
    b = make(hp, [(S, pre)], rng.integers(0, tail, S), H, G, D, 16, "bf16", kernel, seed=S)
    run(b)
    assert b.code() == "HP_OK"
    b.check(everything, rows={0, 1, S // 2, S - 1})


@pytest.mark.parametrize("S,pre", [(3, 3000), (60, 3600), (1, 33000)])
def test_the_librarys_choice(hp, S, pre):
    """Below and above the sizes from which the prefix is read on the tensor cores (60 x 3,600 tokens of 8
    heads of 128: 885 MB, most of it the same pages; one sequence of 33,000 tokens)."""
    b = make(hp, [(S, pre)], [(3 * i) % 50 for i in range(S)], 8, 4, 128, 16, kernel="default", seed=S)
    run(b)
    assert b.code() == "HP_OK"
    b.check(everything, rows={0, S // 2, S - 1})
    out = b.out.clone()
    other = hp.ATTN_TENSOR_CORES if S * pre * 4096 >= 384 << 20 or pre >= 32768 else hp.ATTN_CUDA_CORES
    b.desc = b.describe(flags=other)
    b.out.fill_(7.0)
    run(b)
    assert (b.out.view(-1) == out.view(-1)).all()  # the same kernels
