"""The serving-step entry points without a GPU: workspace sizes, and every refusal the host
makes, on made-up addresses (each call below fails a check before any launch)."""
import ctypes
import os
import subprocess
import sys

import pytest

A = 0x100000  # addresses, 64-byte aligned and never touched


@pytest.fixture(scope="module")
def hpc():
    from paged_kv_cache_hp_gb300 import build, hp
    build.build()
    hp.lib()
    return hp


def fill(struct, **kw):
    for k, v in kw.items():
        setattr(struct, k, v)
    return struct


def step(hpc, **kw):
    f = dict(index_type=0, page_size=16, num_seqs=2, table_len=3, num_free=4, table_cap=8,
             token_cap=8, block_table=A, seq_ptr=A, seq_lens=A, new_lens=A, free_pages=A,
             table_out=A, seq_ptr_out=A, lens_out=A, new_ptr_out=A, slot_map=A, positions=A,
             totals=A)
    f.update(kw)
    return fill(hpc.HpStepDesc(), **f)


@pytest.mark.parametrize("kw,name", [
    (dict(index_type=2), "INDEX_TYPE"), (dict(page_size=0), "ZERO_PAGE_SIZE"),
    (dict(reserved=1), "ARG"), (dict(num_seqs=1 << 58), "OVERFLOW"),
    (dict(token_cap=1 << 60), "OVERFLOW"), (dict(seq_ptr=0), "NULL"), (dict(seq_lens=0), "NULL"),
    (dict(new_lens=0), "NULL"), (dict(block_table=0), "NULL"), (dict(free_pages=0), "NULL"),
    (dict(table_out=0), "NULL"), (dict(lens_out=0), "NULL"), (dict(new_ptr_out=0), "NULL"),
    (dict(seq_ptr_out=0), "NULL"), (dict(slot_map=0), "NULL"), (dict(positions=0), "NULL"),
    (dict(new_lens=A + 2), "ALIGN"), (dict(index_type=1, positions=A + 4), "ALIGN"),
    (dict(slot_map=A + 4), "ALIGN"), (dict(totals=A + 4), "ALIGN"),
])
def test_step_tables_refusals(hpc, kw, name):
    d = step(hpc, **kw)
    assert hpc.status_name(hpc.lib().hp_step_tables(ctypes.byref(d), A, 1 << 20, None, None)) \
        == "HP_ERR_" + name


@pytest.mark.parametrize("kw", [
    dict(num_seqs=1 << 38, table_cap=1 << 40, token_cap=1 << 40), dict(num_seqs=(1 << 37) + 1),
    dict(num_seqs=1 << 38), dict(table_cap=1 << 41, token_cap=1),
])
def test_step_tables_beyond_one_grid(hpc, kw):
    """Sizes whose fill would not fit one launch are refused before any launch, also together (a
    CTA takes 2,048 entries or tokens, or 256 sequences; a grid has up to 2^31 - 1)."""
    d = step(hpc, **kw)
    assert hpc.status_name(hpc.lib().hp_step_tables(ctypes.byref(d), A, 1 << 60, None, None)) == "HP_ERR_OVERFLOW"
    most = -(-(1 << 41) // 2048) + 2 + (1 << 37) // 256 + 1
    assert most < 1 << 31


def test_step_tables_workspace(hpc):
    rc, n = hpc.hp_step_tables_workspace_bytes(100)
    assert rc == 0 and n == 256 + 2 * 1024 + 3 * 8 * 256
    d = step(hpc, num_seqs=100)
    for ws, size in ((None, 1 << 20), (A + 16, 1 << 20), (A, n - 1)):
        assert hpc.status_name(hpc.lib().hp_step_tables(ctypes.byref(d), ws, size, None, None)) \
            == "HP_ERR_WORKSPACE"
    assert hpc.status_name(hpc.lib().hp_step_tables(None, A, 1 << 20, None, None)) == "HP_ERR_NULL"
    assert hpc.status_name(hpc.lib().hp_step_tables_workspace_bytes(1, None)) == "HP_ERR_NULL"


def rope(hpc, section=(64,), **kw):
    f = dict(cos_sin=A, positions=A, max_pos=100, rot_dim=128, axes=len(section), interleaved=0,
             index_type=0)
    f.update(kw)
    r = fill(hpc.HpRopeDesc(), **f)
    for i, n in enumerate(section):
        r.section[i] = n
    return r


def qk(hpc, **kw):
    f = dict(dtype=2, num_q_heads=4, num_kv_heads=2, head_dim=128, eps=1e-6, num_tokens=3, q=A,
             k=A, v=A, q_stride=512, k_stride=256, v_stride=256, q_out=A, q_out_stride=512,
             q_weight=A, k_weight=A, slot_map=A, k_pool=A, v_pool=A, num_pages=4, page_size=16)
    f.update(kw)
    return fill(hpc.HpQkDesc(), **f)


ROPE_REFUSALS = [
    (dict(index_type=3), "INDEX_TYPE"), (dict(rot_dim=24, section=(12,)), "ARG"),
    (dict(rot_dim=0, section=(0,)), "ARG"), (dict(rot_dim=512, section=(256,)), "ARG"),
    (dict(axes=0), "ARG"), (dict(axes=5), "ARG"), (dict(section=(32, 31)), "ARG"),
    (dict(interleaved=2), "ARG"), (dict(max_pos=1 << 60), "OVERFLOW"), (dict(positions=0), "NULL"),
    (dict(cos_sin=0), "NULL"), (dict(cos_sin=A + 4), "ALIGN"), (dict(positions=A + 2), "ALIGN"),
]


@pytest.mark.parametrize("kw,name", [
    (dict(dtype=3), "DTYPE"), (dict(dtype=5), "DTYPE"), (dict(num_kv_heads=0), "ZERO_DIM"),
    (dict(head_dim=0), "ZERO_DIM"), (dict(head_dim=100), "ARG"), (dict(head_dim=264), "ARG"),
    (dict(reserved=1), "ARG"), (dict(head_dim=64), "ARG"),  # rot_dim 128 > 64
    (dict(page_size=0), "ZERO_DIM"), (dict(num_pages=1 << 62), "OVERFLOW"), (dict(k=0), "NULL"),
    (dict(v=0), "NULL"), (dict(q=0), "NULL"), (dict(q_out=0), "NULL"), (dict(slot_map=0), "NULL"),
    (dict(k_pool=0), "NULL"), (dict(v_pool=0), "NULL"), (dict(q=A + 8), "ALIGN"),
    (dict(k_stride=252), "ALIGN"), (dict(q_out_stride=516), "ALIGN"), (dict(v_pool=A + 8), "ALIGN"),
    (dict(k_weight=A + 4), "ALIGN"), (dict(slot_map=A + 4), "ALIGN"),
    (dict(v_stride=1 << 62), "OVERFLOW"),
])
def test_qk_refusals(hpc, kw, name):
    d, r = qk(hpc, **kw), rope(hpc)
    assert hpc.status_name(hpc.lib().hp_qk_norm_rope_append(
        ctypes.byref(d), ctypes.byref(r), None, None)) == "HP_ERR_" + name
    assert hpc.status_name(hpc.lib().hp_qk_norm_rope_append(None, None, None, None)) == "HP_ERR_NULL"


@pytest.mark.parametrize("kw,name", ROPE_REFUSALS)
def test_rope_refusals(hpc, kw, name):
    r = rope(hpc, **kw)
    assert hpc.status_name(hpc.lib().hp_qk_norm_rope_append(
        ctypes.byref(qk(hpc)), ctypes.byref(r), None, None)) == "HP_ERR_" + name
    assert hpc.status_name(hpc.lib().hp_latent_append(
        ctypes.byref(latent(hpc)), ctypes.byref(r), None, None)) == "HP_ERR_" + name


def latent(hpc, **kw):
    f = dict(dtype=2, latent_dim=512, num_q_heads=16, eps=1e-6, num_tokens=3, latent=A,
             latent_stride=576, latent_weight=A, k_rope=A, k_rope_stride=576, q_rope=A,
             q_stride=16 * 192, q_head_stride=192, q_out=A, q_out_stride=1024,
             q_out_head_stride=64, slot_map=A, pool=A, num_pages=4, page_size=16)
    f.update(kw)
    return fill(hpc.HpLatentDesc(), **f)


@pytest.mark.parametrize("kw,name", [
    (dict(dtype=4), "DTYPE"), (dict(latent_dim=0), "ZERO_DIM"), (dict(latent_dim=500), "ARG"),
    (dict(latent_dim=1032), "ARG"), (dict(page_size=0), "ZERO_DIM"), (dict(latent=0), "NULL"),
    (dict(k_rope=0), "NULL"), (dict(q_rope=0), "NULL"), (dict(q_out=0), "NULL"),
    (dict(slot_map=0), "NULL"), (dict(pool=0), "NULL"), (dict(latent_stride=580), "ALIGN"),
    (dict(q_head_stride=68), "ALIGN"), (dict(q_out_head_stride=4), "ALIGN"),
    (dict(k_rope=A + 8), "ALIGN"), (dict(pool=A + 8), "ALIGN"), (dict(num_pages=1 << 60), "OVERFLOW"),
])
def test_latent_append_refusals(hpc, kw, name):
    d = latent(hpc, **kw)
    r = rope(hpc, section=(32,), rot_dim=64)
    assert hpc.status_name(hpc.lib().hp_latent_append(
        ctypes.byref(d), ctypes.byref(r), None, None)) == "HP_ERR_" + name
    assert hpc.status_name(hpc.lib().hp_latent_append(
        ctypes.byref(d), None, None, None)) == "HP_ERR_NULL"


def paged(hpc, **kw):
    f = dict(rank=3, paged_axis=0, has_shard=0, flags=0, dtype=2, index_type=0, num_pages=4,
             page_size=16, num_heads=1, head_dim=576, num_seqs=2, table_len=3, scales_len=0,
             page_pool=A, block_table=A, seq_ptr=A, seq_lens=A, scales=0)
    f.update(kw)
    return fill(hpc.HpPagedDesc(), **f)


LATENT_REFUSALS = [
    (dict(rank=2), {}, "RANK"), (dict(dtype=0), {}, "DTYPE"), (dict(dtype=3), {}, "DTYPE"),
    (dict(num_heads=2), {}, "ARG"), (dict(), dict(R=0), "ARG"), (dict(), dict(R=500), "ARG"),
    (dict(head_dim=1088), dict(R=1024), "ARG"), (dict(head_dim=512), {}, "ARG"),
    (dict(head_dim=584), {}, "ARG"), (dict(head_dim=580), {}, "ARG"),
    (dict(page_size=1 << 27), {}, "ARG"), (dict(), dict(H=0), "ARG"), (dict(), dict(H=4097), "ARG"),
    (dict(), dict(T=1 << 50), "OVERFLOW"), (dict(page_pool=A + 32), {}, "ALIGN"),
    (dict(), dict(q_ptr=None, T=3), "ARG"), (dict(), dict(q_ptr=A + 2), "ALIGN"),
    (dict(index_type=1), dict(q_ptr=A + 4), "ALIGN"), (dict(), dict(q=None), "NULL"),
    (dict(), dict(out=None), "NULL"), (dict(), dict(q=A + 8), "ALIGN"), (dict(), dict(out=A + 8), "ALIGN"),
    (dict(), dict(ws=None), "WORKSPACE"), (dict(), dict(ws=A + 64), "WORKSPACE"),
    (dict(), dict(size=1 << 12), "WORKSPACE"),
]


@pytest.mark.parametrize("dk,ck,name", LATENT_REFUSALS)
def test_latent_attention_refusals(hpc, dk, ck, name):
    c = dict(R=512, H=16, T=2, q=A, q_ptr=A, out=A, ws=A, size=1 << 40)
    c.update(ck)
    d = paged(hpc, **dk)
    L = hpc.lib()
    got = {
        "decode": L.hp_latent_decode(ctypes.byref(d), c["R"], c["q"], c["q_ptr"], c["T"], c["H"],
                                     1.0, c["out"], c["ws"], c["size"], None, None),
        "planned": L.hp_latent_decode_planned(ctypes.byref(d), c["R"], c["q"], c["q_ptr"], c["T"],
                                              c["H"], 1.0, c["out"], c["ws"], c["size"], None, None),
        "prefill": L.hp_latent_prefill(ctypes.byref(d), c["R"], A, 128, 128, c["q"], c["q_ptr"],
                                       c["T"], c["H"], 1.0, c["out"], 40, c["ws"], c["size"],
                                       None, None),
    }
    if not {"q", "out"} & set(ck):
        got["plan"] = L.hp_latent_plan(ctypes.byref(d), c["R"], c["q_ptr"], c["T"], c["H"],
                                       c["ws"], c["size"], None, None)
    assert {k: hpc.status_name(v) for k, v in got.items()} == {k: "HP_ERR_" + name for k in got}


@pytest.mark.parametrize("kw,name", [
    (dict(nope=0), "ARG"), (dict(nope=24), "ARG"), (dict(nope=272), "ARG"), (dict(v=8), "ARG"),
    (dict(v=512), "ARG"), (dict(w=None), "NULL"), (dict(w=A + 8), "ALIGN"),
    (dict(kv=1 << 60), "OVERFLOW"),
])
def test_latent_prefill_refusals(hpc, kw, name):
    c = dict(nope=128, v=128, w=A, kv=40)
    c.update(kw)
    d = paged(hpc)
    assert hpc.status_name(hpc.lib().hp_latent_prefill(
        ctypes.byref(d), 512, c["w"], c["nope"], c["v"], A, A, 2, 16, 1.0, A, c["kv"], A, 1 << 40,
        None, None)) == "HP_ERR_" + name


def test_latent_workspace_sizes(hpc):
    class D:
        c = paged(hpc, num_seqs=100)
        ref = ctypes.byref(c)
    rc, n = hpc.hp_latent_decode_workspace_bytes(D, 512, 100, 128)
    # the plan, 160 SMs x 128 record rows of (max, sum, 512 accumulators) fp32, and an entry of
    # 32 bytes for each of up to 320 workers
    assert rc == 0 and n == 256 + 2 * 1024 + 160 * 128 * 514 * 4 + 320 * 32
    rc, n = hpc.hp_latent_prefill_workspace_bytes(D, 512, 128, 128, 1000, 16, 5000)
    rows = -(-(5000 + 127 * 100) // 128) * 128
    units = -(-(1000 // 256 + 100) * 32 // 256) * 256  # blocks of 256 queries, 32 bytes each
    assert rc == 0 and n == 256 + 2 * 1024 + rows * 576 * 2 + rows * 16 * 256 * 2 + units


def test_the_library_needs_no_torch(hpc):
    """Loading, names of codes, workspace queries and refusals work where torch cannot be imported;
    it is asked for the current stream by the first call that names none."""
    code = """if True:
        import sys
        sys.modules["torch"] = None  # import torch raises ImportError
        from paged_kv_cache_hp_gb300 import hp
        assert hp.lib() is hp.lib()
        assert hp.status_name(0) == "HP_OK"
        assert hp.hp_step_tables_workspace_bytes(100)[0] == 0
        d = hp.HpStepDesc()
        d.index_type = 2
        assert hp.status_name(hp.hp_step_tables(d, None, None, 0)) == "HP_ERR_INDEX_TYPE"
        try:
            hp.hp_step_tables(d, None)
        except ImportError:
            print("asked")
    """
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "asked", r.stderr


def test_descriptors_refuse_strides_they_cannot_say(hpc):
    """A descriptor built over tensors has fields for some strides only; a tensor with others would
    be read as if it had none."""
    import torch
    bf, i64 = torch.bfloat16, torch.int64
    x, slot, pool = torch.zeros((4, 3 * 128), dtype=bf), torch.zeros(4, dtype=i64), torch.zeros((2, 16, 1, 128), dtype=bf)
    q = dict(q=x[:, :128], k=x[:, 128:256], v=x[:, 256:], q_out=torch.zeros((4, 1, 128), dtype=bf), num_q_heads=1,
             num_kv_heads=1, head_dim=128, dtype="bf16", slot_map=slot, k_pool=pool, v_pool=pool, num_pages=2, page_size=16)
    assert hpc.qk_desc(**q).k_stride == 3 * 128
    wide = torch.zeros((4, 256), dtype=bf)
    for name, t in (("q", wide[:, ::2]), ("k", torch.zeros((128, 4), dtype=bf).t()), ("q_out", torch.zeros((4, 128, 2), dtype=bf)[..., 0]),
                    ("v", torch.zeros((4, 4, 2, 32), dtype=bf).transpose(1, 2)), ("slot_map", torch.zeros(8, dtype=i64)[::2]),
                    ("k_pool", torch.zeros((2, 1, 16, 128), dtype=bf).expand(2, 3, 16, 128).transpose(1, 2))):
        with pytest.raises(ValueError, match=name):
            hpc.qk_desc(**{**q, name: t})
    lat = torch.zeros((4, 576), dtype=bf)
    qr = torch.zeros((4, 2, 192), dtype=bf)
    d = dict(latent=lat[:, :512], k_rope=lat[:, 512:], q_rope=qr[:, :, 128:], q_out=qr.transpose(0, 1).contiguous().transpose(0, 1)[:, :, 128:],
             dtype="bf16", slot_map=slot, pool=torch.zeros((2, 16, 576), dtype=bf), num_pages=2, page_size=16)
    got = hpc.latent_desc(**d)
    assert (got.q_stride, got.q_head_stride, got.q_out_stride, got.q_out_head_stride) == (384, 192, 192, 768)
    for name, t in (("latent", torch.zeros((512, 4), dtype=bf).t()), ("k_rope", lat[:, 448::2]), ("q_rope", qr.transpose(1, 2)),
                    ("pool", torch.zeros((16, 2, 576), dtype=bf).transpose(0, 1))):
        with pytest.raises(ValueError, match=name):
            hpc.latent_desc(**{**d, name: t})
    cs, pos = torch.zeros((50, 64)), torch.zeros((3, 4), dtype=torch.int32)
    assert hpc.rope_desc(cos_sin=cs, positions=pos, sections=(8, 12, 12)).max_pos == 50
    for kw in (dict(cos_sin=torch.zeros((50, 128))[:, :64]), dict(positions=torch.zeros((4, 3), dtype=torch.int32).t())):
        with pytest.raises(ValueError, match=next(iter(kw))):
            hpc.rope_desc(**{**dict(cos_sin=cs, positions=pos, sections=(8, 12, 12)), **kw})
    one = torch.zeros(4, dtype=torch.int32)
    s = dict(seq_ptr=one, seq_lens=one[:3], new_lens=one[:3], page_size=16, index_type=0, seq_ptr_out=one, lens_out=one[:3],
             new_ptr_out=one)
    assert hpc.step_desc(**s).num_seqs == 3
    with pytest.raises(ValueError, match="new_lens"):
        hpc.step_desc(**{**s, "new_lens": torch.zeros(6, dtype=torch.int32)[::2]})
