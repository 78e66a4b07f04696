"""The entry points of long contexts without a GPU: workspace sizes, and every refusal the host makes, on
made-up addresses (each call below fails a check before any launch)."""
import ctypes
import os
import re

import numpy as np
import pytest

A = 0x100000  # addresses, 256-byte aligned and never touched
CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "paged_kv_cache_hp_gb300", "csrc")


@pytest.fixture(scope="module")
def hpc():
    from paged_kv_cache_hp_gb300 import build, hp
    build.build()
    hp.lib()
    return hp


def desc(hpc, **kw):
    f = dict(rank=3, paged_axis=0, has_shard=0, flags=0, dtype=2, index_type=0, num_pages=8, page_size=16, num_heads=2,
             head_dim=128, num_seqs=3, table_len=6, scales_len=0, page_pool=A, block_table=A, seq_ptr=A, seq_lens=A,
             scales=None)
    f.update(kw)
    d = hpc.HpPagedDesc()
    for k, v in f.items():
        setattr(d, k, v)
    return d


DESC = [
    (dict(rank=2), "RANK"), (dict(paged_axis=1), "PAGED_AXIS"), (dict(has_shard=1), "SHARD"),
    (dict(index_type=2), "INDEX_TYPE"), (dict(dtype=9), "DTYPE"), (dict(dtype=0), "DTYPE"), (dict(dtype=3), "DTYPE"),
    (dict(page_size=0), "ZERO_DIM"), (dict(num_heads=0), "ZERO_DIM"), (dict(head_dim=96), "ARG"),
    (dict(page_size=4097), "ARG"), (dict(num_heads=65537), "ARG"), (dict(seq_ptr=None), "NULL"),
    (dict(seq_lens=None), "NULL"), (dict(block_table=None), "NULL"), (dict(seq_ptr=A + 8), "ALIGN"),
]
CALLS = {
    "hp_page_bounds": lambda d, **k: [d, k.get("ptr"), k.get("total", 3), k.get("bounds", A), None, None],
    "hp_page_scores": lambda d, **k: [d, k.get("bounds", A), k.get("q", A), k.get("ptr"), k.get("total", 3), k.get("hq", 4),
                                      k.get("scale", 0.1), k.get("scores", A), k.get("pages", 9), None, None],
    "hp_select_pages": lambda d, **k: [d, k.get("ptr"), k.get("total", 3), k.get("scores", A), k.get("pages", 9),
                                       k.get("sinks", 1), k.get("recent", 1), k.get("k", 4), k.get("selected", A), None, None],
    "hp_attention_pages": lambda d, **k: [d, k.get("v", A), k.get("q", A), k.get("ptr"), k.get("total", 3), k.get("hq", 4),
                                          k.get("scale", 0.1), k.get("selected", A), k.get("k", 4), k.get("out", A), None, None],
    "hp_attention_prefix": lambda d, **k: [d, k.get("v", A), k.get("group", A), k.get("pre", A), k.get("groups", 2),
                                           k.get("q", A), k.get("ptr"), k.get("total", 3), k.get("hq", 4), k.get("scale", 0.1),
                                           k.get("out", A), k.get("ws", A), k.get("wsn", 1 << 40), None, None],
    "hp_attention_prefix_plan": lambda d, **k: [d, k.get("group", A), k.get("pre", A), k.get("groups", 2), k.get("ptr"),
                                                k.get("total", 3), k.get("hq", 4), k.get("ws", A), k.get("wsn", 1 << 40), None,
                                                None],
}
CALLS["hp_attention_prefix_planned"] = CALLS["hp_attention_prefix"]


def call(hpc, name, d, **kw):
    ref = None if d is None else ctypes.byref(d)
    return hpc.status_name(getattr(hpc.lib(), name)(*CALLS[name](ref, **kw)))


@pytest.mark.parametrize("name", sorted(CALLS))
def test_descriptor_refusals(hpc, name):
    assert call(hpc, name, None) == "HP_ERR_NULL"
    for kw, code in DESC:
        assert call(hpc, name, desc(hpc, **kw)) == "HP_ERR_" + code, kw
    if name != "hp_page_scores":  # (its pool is the bounds')
        assert call(hpc, name, desc(hpc, page_pool=None)) == "HP_ERR_NULL"
        assert call(hpc, name, desc(hpc, page_pool=A + 16)) == "HP_ERR_ALIGN"


OFFSETS = [(dict(total=4), "ARG"), (dict(total=1 << 40), "OVERFLOW"), (dict(ptr=A + 2), "ALIGN")]
HEADS = [(dict(hq=0), "ARG"), (dict(hq=3), "ARG"), (dict(hq=34), "ARG"), (dict(scale=float("nan")), "ARG"),
         (dict(q=None), "NULL"), (dict(q=A + 8), "ALIGN")]
ROWS = OFFSETS + HEADS + [(dict(v=None), "NULL"), (dict(out=None), "NULL"), (dict(v=A + 32), "ALIGN"),
                          (dict(out=A + 8), "ALIGN"), (dict(ptr=A, total=1 << 39), "OVERFLOW")]
PREFIX = [(dict(groups=4), "ARG"), (dict(groups=0), "ARG"), (dict(group=None), "NULL"), (dict(pre=None), "NULL"),
          (dict(group=A + 2), "ALIGN"), (dict(pre=A + 1), "ALIGN"), (dict(ws=None), "WORKSPACE"), (dict(ws=A + 64), "WORKSPACE"),
          (dict(wsn=100), "WORKSPACE")]
ARGS = {
    "hp_page_bounds": OFFSETS + [(dict(bounds=None), "NULL"), (dict(bounds=A + 32), "ALIGN"),
                                 (dict(ptr=A, total=1 << 39), "OVERFLOW")],
    "hp_page_scores": OFFSETS + HEADS + [(dict(scale=-0.1), "ARG"), (dict(bounds=None), "NULL"), (dict(bounds=A + 16), "ALIGN"),
                                         (dict(scores=None), "NULL"), (dict(scores=A + 2), "ALIGN"),
                                         (dict(pages=1 << 31), "OVERFLOW"), (dict(ptr=A, total=1 << 39), "OVERFLOW")],
    "hp_select_pages": OFFSETS + [(dict(k=0), "ARG"), (dict(k=1 << 31), "ARG"), (dict(sinks=3, recent=2), "ARG"),
                                  (dict(sinks=0xFFFFFFFF, recent=5), "ARG"), (dict(scores=None), "NULL"),
                                  (dict(selected=None), "NULL"), (dict(scores=A + 1), "ALIGN"), (dict(selected=A + 2), "ALIGN"),
                                  (dict(pages=1 << 31), "OVERFLOW"), (dict(ptr=A, total=1 << 39), "OVERFLOW")],
    "hp_attention_pages": ROWS + [(dict(selected=None), "NULL"), (dict(selected=A + 2), "ALIGN"), (dict(k=0), "ARG"),
                                  (dict(k=1 << 27), "ARG")],
    "hp_attention_prefix": ROWS + PREFIX,
    "hp_attention_prefix_planned": ROWS + PREFIX,
    "hp_attention_prefix_plan": OFFSETS[:1] + OFFSETS[2:] + HEADS[:3] + PREFIX,
}


@pytest.mark.parametrize("name,kw,code", [(n, kw, code) for n in sorted(ARGS) for kw, code in ARGS[n]])
def test_argument_refusals(hpc, name, kw, code):
    assert call(hpc, name, desc(hpc), **kw) == "HP_ERR_" + code


def test_select_pages_takes_no_table_and_no_pool(hpc):
    """The first thing wrong here is k, so the descriptor passed."""
    d = desc(hpc, num_pages=0, page_pool=None, table_len=0, block_table=None)
    assert call(hpc, "hp_select_pages", d, k=0) == "HP_ERR_ARG"


def test_prefix_workspace(hpc):
    n = ctypes.c_uint64(0)
    f = hpc.lib().hp_attention_prefix_workspace_bytes
    d = desc(hpc)
    assert f(ctypes.byref(d), 2, 3, 4, ctypes.byref(n)) == 0
    need = n.value
    assert call(hpc, "hp_attention_prefix", d, wsn=need - 1) == "HP_ERR_WORKSPACE"
    assert hpc.status_name(f(None, 2, 3, 4, ctypes.byref(n))) == "HP_ERR_NULL"
    assert hpc.status_name(f(ctypes.byref(d), 2, 3, 4, None)) == "HP_ERR_NULL"
    for big in ((1 << 32, 3, 4), (2, 1 << 32, 4), (2, 1 << 31, 1 << 20)):
        assert hpc.status_name(f(ctypes.byref(d), *big, ctypes.byref(n))) == "HP_ERR_OVERFLOW"


def test_prefix_workspace_holds_records_where_the_tensor_cores_can_leave_any(hpc):
    """A row's 24 bytes of plan each, and for head_dim 64 and 128 with pages of a multiple of 8 two records a
    (query, head) of a float2 and head_dim floats, with 160 x 256 more; the flags change nothing."""
    f = hpc.lib().hp_attention_prefix_workspace_bytes

    def size(total, hq, **kw):
        n = ctypes.c_uint64(0)
        assert f(ctypes.byref(desc(hpc, **kw)), 2, total, hq, ctypes.byref(n)) == 0
        return n.value

    for dim, page, records in ((64, 16, 1), (128, 8, 1), (128, 24, 1), (128, 4096, 1), (256, 16, 0), (128, 12, 0), (64, 1, 0)):
        small = size(0, 32, head_dim=dim, page_size=page)
        grown = size(4096, 32, head_dim=dim, page_size=page) - small
        assert grown >= 4096 * 24 + records * 2 * 4096 * 32 * (dim * 4 + 8)
        assert grown <= 4096 * 40 + records * 2 * 4096 * 32 * (dim * 4 + 8) + 1024
        assert (small > 160 * 256 * dim * 4) == bool(records)
        for flags in (hpc.ATTN_CUDA_CORES, hpc.ATTN_TENSOR_CORES, hpc.HOST_MEMORY):
            assert size(0, 32, head_dim=dim, page_size=page, flags=flags) == small
    d = desc(hpc, head_dim=256)
    need = size(3, 4, head_dim=256)
    assert call(hpc, "hp_attention_prefix", d, wsn=need - 1) == "HP_ERR_WORKSPACE"


def test_status_names(hpc):
    assert hpc.status_name(-36) == "HP_ERR_GROUP" and hpc.status_name(-37) == "HP_ERR_PREFIX"


def test_binding_refuses_strides_it_has_no_field_for(hpc):
    import torch
    x = torch.zeros((4, 8, 128), dtype=torch.bfloat16)[:, ::2]
    with pytest.raises(ValueError, match="q has to be contiguous"):
        hpc.hp_attention_pages(None, None, x, None, 4, 4, 1.0, None, 1, None)
    with pytest.raises(ValueError, match="scores has to be contiguous"):
        hpc.hp_select_pages(None, None, 4, torch.zeros((4, 2, 9))[..., :8], 8, 0, 0, 1, None)


# ------------------------------------------------------------------------- sources
FILES = ["hp_pages.cu", "hp_attn_rows.cu", "hp_prefix.cu", "hp_prefix_tc.cu", "hp_pages.cuh", "hp_rows.cuh", "hp_prefix.cuh",
         "hp_mma.cuh"]


def code(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def test_no_read_only_loads_behind_a_kernel_that_may_still_write():
    for name in FILES:
        assert not re.search(r"__ldg|\.nc\.|__restrict__", code(name)), name


def test_dependent_kernels_wait_before_they_look_at_memory():
    """Every kernel waits for the one before it on every path, before its first return or access."""
    seen = 0
    for name in FILES:
        for m in re.finditer(r"__global__ void.*?\n\{\n(.*?)\n\}\n", code(name), re.S):
            body = m.group(1)
            at = body.find("pdl_wait();")
            assert at >= 0, name
            before = body[:at]
            assert "return" not in before and not re.search(r"a\.\w+\s*(\[|->)|index_at|find_query", before), (name, before)
            seen += 1
    assert seen == 8
