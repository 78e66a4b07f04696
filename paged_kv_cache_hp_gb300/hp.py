"""Thin ctypes binding of libhp.so (include/hp.h): argument marshalling only.

Every function here has the name of the C entry point it calls and returns that
call's integer status (``HP_OK`` = 0); ``status_name`` turns it into the name
``hp_status_string`` gives.  Tensors are torch tensors on the current CUDA
device; their ``data_ptr()`` is passed through unchanged, and ``stream``
defaults to torch's current stream.  Nothing in this module computes any part
of the path: all of it runs in the library's CUDA kernels.  If libhp.so has not
been built, the first call raises.
"""
from __future__ import annotations

import ctypes
import os
import threading

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libhp.so")

HP_OK = 0
DTYPES = {"f32": 0, "f16": 1, "bf16": 2, "i8": 3, "u8": 4, "f64": 5}
IDX_U32, IDX_U64 = 0, 1
PERMISSIVE, HAS_QUANT, HOST_MEMORY, TEST_STALL = 0x1, 0x2, 0x4, 0x100
ATTN_TENSOR_CORES, ATTN_CUDA_CORES = 0x8, 0x10

_lock = threading.Lock()
_lib = None


class HpPagedDesc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_uint32) for n in
                ("rank", "paged_axis", "has_shard", "flags", "dtype", "index_type")] + \
               [(n, ctypes.c_uint64) for n in
                ("num_pages", "page_size", "num_heads", "head_dim", "num_seqs", "table_len",
                 "scales_len")] + \
               [(n, ctypes.c_void_p) for n in
                ("page_pool", "block_table", "seq_ptr", "seq_lens", "scales")]


class HpQuantDesc(ctypes.Structure):
    _fields_ = [("scheme_tag", ctypes.c_uint32), ("axis", ctypes.c_uint32),
                ("block_size", ctypes.c_uint64), ("count", ctypes.c_uint64),
                ("scales", ctypes.c_void_p), ("zero_points", ctypes.c_void_p)]


PER_TENSOR, PER_CHANNEL, PER_BLOCK_AFFINE = 0x01, 0x02, 0x03


def quant_desc(scheme_tag, scales, zero_points=None, axis=0, block_size=0, count=None):
    """An hp_quant_desc over device tensors (kept alive on the result's `keep`)."""
    q = HpQuantDesc()
    q.scheme_tag, q.axis, q.block_size = scheme_tag, axis, block_size
    q.count = (0 if scales is None else scales.numel()) if count is None else count
    q.scales, q.zero_points = _p(scales), _p(zero_points)
    q.keep = (scales, zero_points)
    return q


class HpStepDesc(ctypes.Structure):
    _fields_ = [("index_type", ctypes.c_uint32), ("reserved", ctypes.c_uint32)] + \
               [(n, ctypes.c_uint64) for n in
                ("num_seqs", "page_size", "table_len", "num_free", "table_cap", "token_cap")] + \
               [(n, ctypes.c_void_p) for n in
                ("block_table", "seq_ptr", "seq_lens", "new_lens", "free_pages", "table_out",
                 "seq_ptr_out", "lens_out", "new_ptr_out", "slot_map", "positions", "totals")]


class HpRopeDesc(ctypes.Structure):
    _fields_ = [("cos_sin", ctypes.c_void_p), ("positions", ctypes.c_void_p),
                ("max_pos", ctypes.c_uint64), ("rot_dim", ctypes.c_uint32),
                ("axes", ctypes.c_uint32), ("section", ctypes.c_uint32 * 4),
                ("interleaved", ctypes.c_uint32), ("index_type", ctypes.c_uint32)]


class HpQkDesc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_uint32) for n in
                ("dtype", "num_q_heads", "num_kv_heads", "head_dim")] + \
               [("eps", ctypes.c_float), ("reserved", ctypes.c_uint32),
                ("num_tokens", ctypes.c_uint64)] + \
               [(n, ctypes.c_void_p) for n in ("q", "k", "v")] + \
               [(n, ctypes.c_uint64) for n in ("q_stride", "k_stride", "v_stride")] + \
               [("q_out", ctypes.c_void_p), ("q_out_stride", ctypes.c_uint64)] + \
               [(n, ctypes.c_void_p) for n in
                ("q_weight", "k_weight", "slot_map", "k_pool", "v_pool")] + \
               [("num_pages", ctypes.c_uint64), ("page_size", ctypes.c_uint64)]


class HpLatentDesc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_uint32) for n in ("dtype", "latent_dim", "num_q_heads")] + \
               [("eps", ctypes.c_float), ("num_tokens", ctypes.c_uint64),
                ("latent", ctypes.c_void_p), ("latent_stride", ctypes.c_uint64),
                ("latent_weight", ctypes.c_void_p), ("k_rope", ctypes.c_void_p),
                ("k_rope_stride", ctypes.c_uint64), ("q_rope", ctypes.c_void_p),
                ("q_stride", ctypes.c_uint64), ("q_head_stride", ctypes.c_uint64),
                ("q_out", ctypes.c_void_p), ("q_out_stride", ctypes.c_uint64),
                ("q_out_head_stride", ctypes.c_uint64), ("slot_map", ctypes.c_void_p),
                ("pool", ctypes.c_void_p), ("num_pages", ctypes.c_uint64),
                ("page_size", ctypes.c_uint64)]


def _numel(t):
    return 0 if t is None else t.numel()


def _dtype(d):
    return DTYPES[d] if isinstance(d, str) else d


def _contiguous(what, **tensors):
    """Refuses tensors whose strides the descriptor has no field for."""
    for name, t in tensors.items():
        if t is not None and not t.is_contiguous():
            raise ValueError("%s: %s has to be contiguous, its strides are %s" % (what, name, tuple(t.stride())))


def _inner(what, dims, **tensors):
    """Refuses tensors whose dimensions from `dims` on are not one contiguous piece."""
    for name, t in tensors.items():
        if t is None or t.numel() == 0:
            continue
        row = t
        for _ in range(dims):
            row = row[0]
        if not row.is_contiguous():
            raise ValueError("%s: %s has to be contiguous from dimension %d on, its strides are %s"
                             % (what, name, dims, tuple(t.stride())))


def step_desc(*, seq_ptr, seq_lens, new_lens, page_size, index_type, seq_ptr_out, lens_out,
              new_ptr_out, block_table=None, free_pages=None, table_out=None, slot_map=None,
              positions=None, totals=None, **fields):
    """An hp_step_desc over device tensors (kept alive on the result's `keep`); the counts
    come from the tensors unless given by name."""
    d = HpStepDesc()
    bufs = dict(block_table=block_table, seq_ptr=seq_ptr, seq_lens=seq_lens, new_lens=new_lens,
                free_pages=free_pages, table_out=table_out, seq_ptr_out=seq_ptr_out,
                lens_out=lens_out, new_ptr_out=new_ptr_out, slot_map=slot_map,
                positions=positions, totals=totals)
    _contiguous("step_desc", **bufs)
    d.index_type, d.page_size = index_type, page_size
    d.num_seqs, d.table_len, d.num_free = _numel(seq_lens), _numel(block_table), _numel(free_pages)
    d.table_cap, d.token_cap = _numel(table_out), _numel(slot_map)
    for name, t in bufs.items():
        setattr(d, name, _p(t))
    for name, v in fields.items():
        setattr(d, name, v)
    d.keep = tuple(bufs.values())
    return d


def rope_desc(*, cos_sin, positions, sections, interleaved=False, index_type=IDX_U32, **fields):
    """An hp_rope_desc: cos_sin fp32 [max_pos, rot_dim], positions [axes, num_tokens], both
    contiguous."""
    d = HpRopeDesc()
    _contiguous("rope_desc", cos_sin=cos_sin, positions=positions)
    d.cos_sin, d.positions = _p(cos_sin), _p(positions)
    d.max_pos, d.rot_dim = cos_sin.shape
    d.axes = len(sections)
    for i, n in enumerate(sections[:4]):
        d.section[i] = n
    d.interleaved, d.index_type = int(interleaved), index_type
    for name, v in fields.items():
        setattr(d, name, v)
    d.keep = (cos_sin, positions)
    return d


def qk_desc(*, q, k, v, q_out, num_q_heads, num_kv_heads, head_dim, dtype, slot_map, k_pool,
            v_pool, num_pages, page_size, q_weight=None, k_weight=None, eps=1e-6, **fields):
    """An hp_qk_desc over device tensors: q, k, v and q_out with the token as their first
    dimension (its stride is taken from the tensor), heads and dims contiguous in it; the others
    contiguous."""
    d = HpQkDesc()
    _inner("qk_desc", 1, q=q, k=k, v=v, q_out=q_out)
    _contiguous("qk_desc", q_weight=q_weight, k_weight=k_weight, slot_map=slot_map, k_pool=k_pool, v_pool=v_pool)
    d.dtype, d.num_q_heads, d.num_kv_heads = _dtype(dtype), num_q_heads, num_kv_heads
    d.head_dim, d.eps, d.num_tokens = head_dim, eps, slot_map.numel()
    bufs = dict(q=q, k=k, v=v, q_out=q_out, q_weight=q_weight, k_weight=k_weight,
                slot_map=slot_map, k_pool=k_pool, v_pool=v_pool)
    for name, t in bufs.items():
        setattr(d, name, _p(t))
    for name, t in (("q", q), ("k", k), ("v", v), ("q_out", q_out)):
        setattr(d, name + "_stride", 0 if t is None else t.stride(0))
    d.num_pages, d.page_size = num_pages, page_size
    for name, val in fields.items():
        setattr(d, name, val)
    d.keep = tuple(bufs.values())
    return d


def latent_desc(*, latent, k_rope, dtype, slot_map, pool, num_pages, page_size, q_rope=None,
                q_out=None, latent_weight=None, eps=1e-6, **fields):
    """An hp_latent_desc over device tensors: latent [tokens, latent_dim], k_rope [tokens,
    rope_dim], q_rope and q_out [tokens, heads, rope_dim], each with its own strides of tokens and
    heads; the others contiguous."""
    d = HpLatentDesc()
    _inner("latent_desc", 1, latent=latent, k_rope=k_rope)
    _inner("latent_desc", 2, q_rope=q_rope, q_out=q_out)
    _contiguous("latent_desc", latent_weight=latent_weight, slot_map=slot_map, pool=pool)
    d.dtype, d.latent_dim, d.eps = _dtype(dtype), latent.shape[1], eps
    d.num_q_heads = 0 if q_rope is None else q_rope.shape[1]
    d.num_tokens = slot_map.numel()
    bufs = dict(latent=latent, latent_weight=latent_weight, k_rope=k_rope, q_rope=q_rope,
                q_out=q_out, slot_map=slot_map, pool=pool)
    for name, t in bufs.items():
        setattr(d, name, _p(t))
    d.latent_stride, d.k_rope_stride = latent.stride(0), k_rope.stride(0)
    if q_rope is not None:
        d.q_stride, d.q_head_stride = q_rope.stride(0), q_rope.stride(1)
    if q_out is not None:
        d.q_out_stride, d.q_out_head_stride = q_out.stride(0), q_out.stride(1)
    d.num_pages, d.page_size = num_pages, page_size
    for name, val in fields.items():
        setattr(d, name, val)
    d.keep = tuple(bufs.values())
    return d


def lib():
    """The loaded library; raises RuntimeError when libhp.so is missing."""
    global _lib
    if _lib is not None:  # set once, complete: no lock on the calls of a step
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(
                    "libhp.so is not built (%s); run paged_kv_cache_hp_gb300.build.build()"
                    % LIB_PATH)
            L = ctypes.CDLL(LIB_PATH)
            i, u64, vp = ctypes.c_int, ctypes.c_uint64, ctypes.c_void_p
            u32 = ctypes.c_uint32
            D = ctypes.POINTER(HpPagedDesc)
            pu64 = ctypes.POINTER(ctypes.c_uint64)
            sig = {
                "hp_status_string": (ctypes.c_char_p, [i]),
                "hp_workspace_bytes": (i, [D, pu64]),
                "hp_validate": (i, [D, vp, u64, pu64, vp]),
                "hp_plan": (i, [D, u64, vp, u64, vp, vp]),
                "hp_gather": (i, [D, vp, u64, vp, u64, vp, vp]),
                "hp_gather_planned": (i, [D, vp, vp, vp, vp]),
                "hp_gather_dequant": (i, [D, vp, u64, vp, u64, vp, vp]),
                "hp_gather_dequant_planned": (i, [D, vp, vp, vp, vp]),
                "hp_scatter_append": (i, [D, vp, vp, u64, vp, u64, vp, vp]),
                "hp_append_plan": (i, [D, vp, u64, vp, u64, vp, vp]),
                "hp_scatter_append_planned": (i, [D, vp, vp, u64, vp, vp, vp]),
                "hp_validate_append": (i, [D, vp, u64, vp, u64, pu64, vp]),
                "hp_lane_validate": (i, [u64, u64, vp, u64, pu64]),
                "hp_lane_gather": (i, [vp, vp, u64, u64, u64, u64, u64, ctypes.c_uint32, u64,
                                       vp, ctypes.c_uint32, vp, vp]),
                "hp_lane_append": (i, [vp, vp, u64, u64, u64, u64, u64, ctypes.c_uint32, u64,
                                       u64, vp, ctypes.c_uint32, vp, vp]),
                "hp_gather_noalloc": (i, [D, vp, u64, vp, vp]),
                "hp_copy_pages": (i, [vp, u64, u64, ctypes.c_uint32, vp, vp, u64, ctypes.c_uint32,
                                      vp, vp]),
                "hp_attention_decode_workspace_bytes": (i, [D, ctypes.c_uint32, pu64]),
                "hp_attention_decode": (i, [D, vp, vp, ctypes.c_uint32, ctypes.c_float, vp, vp,
                                            u64, vp, vp]),
                "hp_attention_plan": (i, [D, ctypes.c_uint32, vp, u64, vp, vp]),
                "hp_attention_decode_planned": (i, [D, vp, vp, ctypes.c_uint32, ctypes.c_float,
                                                    vp, vp, u64, vp, vp]),
                "hp_from_kernel_layout": (i, [vp, vp, u64, u64, u64, u64, u64, ctypes.c_uint32,
                                              vp]),
                "hp_to_kernel_layout": (i, [vp, vp, u64, u64, u64, u64, u64, ctypes.c_uint32,
                                            vp]),
                "hp_table_workspace_bytes": (i, [u64, pu64]),
                "hp_padded_to_csr": (i, [vp, vp, u64, u64, u64, ctypes.c_uint32, vp, u64, vp, vp,
                                         u64, vp, vp]),
                "hp_csr_to_padded": (i, [vp, u64, vp, u64, u64, u64, ctypes.c_uint32, vp, vp, u64,
                                         vp, vp]),
                "hp_zero_tails_scratch_bytes": (i, [D, pu64]),
                "hp_zero_tails": (i, [D, vp, u64, vp, u64, vp, vp]),
                "hp_gather_dequant_q": (i, [D, ctypes.POINTER(HpQuantDesc), vp, u64, vp, u64, vp,
                                            vp]),
                "hp_gather_dequant_q_planned": (i, [D, ctypes.POINTER(HpQuantDesc), vp, vp, vp,
                                                    vp]),
                "hp_step_tables_workspace_bytes": (i, [u64, pu64]),
                "hp_step_tables": (i, [ctypes.POINTER(HpStepDesc), vp, u64, vp, vp]),
                "hp_qk_norm_rope_append": (i, [ctypes.POINTER(HpQkDesc),
                                               ctypes.POINTER(HpRopeDesc), vp, vp]),
                "hp_latent_append": (i, [ctypes.POINTER(HpLatentDesc),
                                         ctypes.POINTER(HpRopeDesc), vp, vp]),
                "hp_latent_decode_workspace_bytes": (i, [D, u32, u64, u32, pu64]),
                "hp_latent_plan": (i, [D, u32, vp, u64, u32, vp, u64, vp, vp]),
                "hp_latent_decode": (i, [D, u32, vp, vp, u64, u32, ctypes.c_float, vp, vp, u64,
                                         vp, vp]),
                "hp_latent_decode_planned": (i, [D, u32, vp, vp, u64, u32, ctypes.c_float, vp,
                                                 vp, u64, vp, vp]),
                "hp_latent_prefill_workspace_bytes": (i, [D, u32, u32, u32, u64, u32, u64, pu64]),
                "hp_latent_prefill": (i, [D, u32, vp, u32, u32, vp, vp, u64, u32, ctypes.c_float,
                                          vp, u64, vp, u64, vp, vp]),
                "hp_page_bounds": (i, [D, vp, u64, vp, vp, vp]),
                "hp_page_scores": (i, [D, vp, vp, vp, u64, u32, ctypes.c_float, vp, u64, vp, vp]),
                "hp_select_pages": (i, [D, vp, u64, vp, u64, u32, u32, u32, vp, vp, vp]),
                "hp_attention_pages": (i, [D, vp, vp, vp, u64, u32, ctypes.c_float, vp, u32, vp,
                                           vp, vp]),
                "hp_attention_prefix_workspace_bytes": (i, [D, u64, u64, u32, pu64]),
                "hp_attention_prefix": (i, [D, vp, vp, vp, u64, vp, vp, u64, u32, ctypes.c_float,
                                            vp, vp, u64, vp, vp]),
                "hp_attention_prefix_plan": (i, [D, vp, vp, u64, vp, u64, u32, vp, u64, vp, vp]),
                "hp_attention_prefix_planned": (i, [D, vp, vp, vp, u64, vp, vp, u64, u32,
                                                    ctypes.c_float, vp, vp, u64, vp, vp]),
            }
            for name, (res, args) in sig.items():
                f = getattr(L, name)
                f.restype, f.argtypes = res, args
            _lib = L
    return _lib


def status_name(code: int) -> str:
    return lib().hp_status_string(code).decode()


def _p(t):
    return None if t is None else t.data_ptr()


def _current_stream():
    """torch's current stream on the current device, as an integer.  The first call without a
    stream finds the way to ask (the library itself needs no torch): the raw-handle query costs a
    tenth of building a Stream object (3 us on the Grace host, half of a small call's time)."""
    global _current_stream
    import torch
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    if raw is not None:
        _current_stream = lambda: raw(torch.cuda.current_device())  # noqa: E731
    else:
        _current_stream = lambda: torch.cuda.current_stream().cuda_stream  # noqa: E731
    return _current_stream()


def _stream(stream):
    if stream is None:
        return _current_stream()
    return getattr(stream, "cuda_stream", stream)


class PagedDesc:
    """An hp_paged_desc over device tensors, which it keeps alive.

    ``pool`` is any device tensor whose bytes are the page pool; ``table``,
    ``seq_ptr`` and ``lens`` are int32/int64 (or uint32/uint64) device tensors of
    the index type; ``scales`` an fp32 device tensor.  Field overrides (rank,
    has_shard, num_seqs, table_len, ...) exist so that malformed descriptors can
    be expressed.
    """

    def __init__(self, pool, table, seq_ptr, lens, *, num_pages, page_size, num_heads, head_dim,
                 dtype, index_type, scales=None, flags=0, rank=3, paged_axis=0, has_shard=0,
                 num_seqs=None, table_len=None, scales_len=None):
        self._keep = (pool, table, seq_ptr, lens, scales)
        d = HpPagedDesc()
        d.rank, d.paged_axis, d.has_shard, d.flags = rank, paged_axis, has_shard, flags
        d.dtype = DTYPES[dtype] if isinstance(dtype, str) else dtype
        d.index_type = index_type
        d.num_pages, d.page_size, d.num_heads, d.head_dim = num_pages, page_size, num_heads, head_dim
        d.num_seqs = (0 if lens is None else lens.numel()) if num_seqs is None else num_seqs
        d.table_len = (0 if table is None else table.numel()) if table_len is None else table_len
        d.scales_len = (0 if scales is None else scales.numel()) if scales_len is None else scales_len
        d.page_pool, d.block_table, d.seq_ptr = _p(pool), _p(table), _p(seq_ptr)
        d.seq_lens, d.scales = _p(lens), _p(scales)
        self.c = d

    @property
    def ref(self):
        return ctypes.byref(self.c)


def hp_workspace_bytes(desc: PagedDesc):
    n = ctypes.c_uint64(0)
    rc = lib().hp_workspace_bytes(desc.ref, ctypes.byref(n))
    return rc, n.value


def hp_validate(desc, workspace, stream=None):
    """Returns (status, first_bad)."""
    first = ctypes.c_uint64(0)
    rc = lib().hp_validate(desc.ref, _p(workspace), _wsn(workspace), ctypes.byref(first),
                           _stream(stream))
    return rc, first.value


def hp_validate_append(desc, new_ptr, total_new, workspace, stream=None):
    first = ctypes.c_uint64(0)
    rc = lib().hp_validate_append(desc.ref, _p(new_ptr), total_new, _p(workspace),
                                  _wsn(workspace), ctypes.byref(first), _stream(stream))
    return rc, first.value


def _wsn(workspace):
    return 0 if workspace is None else workspace.numel() * workspace.element_size()


def hp_plan(desc, out_tokens, workspace, d_status=None, stream=None):
    return lib().hp_plan(desc.ref, out_tokens, _p(workspace), _wsn(workspace), _p(d_status),
                         _stream(stream))


def hp_gather(desc, out, out_tokens, workspace, d_status=None, stream=None):
    return lib().hp_gather(desc.ref, _p(out), out_tokens, _p(workspace), _wsn(workspace),
                           _p(d_status), _stream(stream))


def hp_gather_planned(desc, out, workspace, d_status=None, stream=None):
    return lib().hp_gather_planned(desc.ref, _p(out), _p(workspace), _p(d_status), _stream(stream))


def hp_gather_dequant(desc, out, out_tokens, workspace, d_status=None, stream=None):
    return lib().hp_gather_dequant(desc.ref, _p(out), out_tokens, _p(workspace), _wsn(workspace),
                                   _p(d_status), _stream(stream))


def hp_gather_dequant_planned(desc, out, workspace, d_status=None, stream=None):
    return lib().hp_gather_dequant_planned(desc.ref, _p(out), _p(workspace), _p(d_status),
                                           _stream(stream))


def hp_scatter_append(desc, new_rows, new_ptr, total_new, workspace, d_status=None, stream=None):
    return lib().hp_scatter_append(desc.ref, _p(new_rows), _p(new_ptr), total_new, _p(workspace),
                                   _wsn(workspace), _p(d_status), _stream(stream))


def hp_append_plan(desc, new_ptr, total_new, workspace, d_status=None, stream=None):
    return lib().hp_append_plan(desc.ref, _p(new_ptr), total_new, _p(workspace), _wsn(workspace),
                                _p(d_status), _stream(stream))


def hp_scatter_append_planned(desc, new_rows, new_ptr, total_new, workspace, d_status=None,
                              stream=None):
    return lib().hp_scatter_append_planned(desc.ref, _p(new_rows), _p(new_ptr), total_new,
                                           _p(workspace), _p(d_status), _stream(stream))


def hp_lane_validate(capacity, page_tokens, table_host):
    """table_host: a contiguous uint64 numpy array (or None).  Returns (status, detail pair)."""
    det = (ctypes.c_uint64 * 2)()
    n = 0 if table_host is None else len(table_host)
    ptr = None if table_host is None or n == 0 else table_host.ctypes.data
    rc = lib().hp_lane_validate(capacity, page_tokens, ptr, n, det)
    return rc, (det[0], det[1])


def hp_lane_gather(pool, table, capacity, page_tokens, batch, kv_heads, width, dtype, n, out,
                   d_status=None, stream=None, flags=0):
    dt = DTYPES[dtype] if isinstance(dtype, str) else dtype
    return lib().hp_lane_gather(_p(pool), _p(table), capacity, page_tokens, batch, kv_heads,
                                width, dt, n, _p(out), flags, _p(d_status), _stream(stream))


def hp_lane_append(pool, table, capacity, page_tokens, batch, kv_heads, width, dtype, n, m,
                   new_rows, d_status=None, stream=None, flags=0):
    dt = DTYPES[dtype] if isinstance(dtype, str) else dtype
    return lib().hp_lane_append(_p(pool), _p(table), capacity, page_tokens, batch, kv_heads,
                                width, dt, n, m, _p(new_rows), flags, _p(d_status),
                                _stream(stream))


def hp_gather_dequant_q(desc, quant, out, out_tokens, workspace, d_status=None, stream=None):
    return lib().hp_gather_dequant_q(desc.ref, None if quant is None else ctypes.byref(quant),
                                     _p(out), out_tokens, _p(workspace), _wsn(workspace),
                                     _p(d_status), _stream(stream))


def hp_gather_dequant_q_planned(desc, quant, out, workspace, d_status=None, stream=None):
    return lib().hp_gather_dequant_q_planned(desc.ref,
                                             None if quant is None else ctypes.byref(quant),
                                             _p(out), _p(workspace), _p(d_status),
                                             _stream(stream))


def hp_copy_pages(pool, num_pages, page_bytes, index_type, src_pages, dst_pages, num_pairs,
                  d_status=None, stream=None, flags=0):
    return lib().hp_copy_pages(_p(pool), num_pages, page_bytes, index_type, _p(src_pages),
                               _p(dst_pages), num_pairs, flags, _p(d_status), _stream(stream))


def hp_zero_tails_scratch_bytes(desc):
    n = ctypes.c_uint64(0)
    rc = lib().hp_zero_tails_scratch_bytes(desc.ref, ctypes.byref(n))
    return rc, n.value


def hp_zero_tails(desc, workspace, scratch, d_status=None, stream=None):
    return lib().hp_zero_tails(desc.ref, _p(workspace), _wsn(workspace), _p(scratch),
                               _wsn(scratch), _p(d_status), _stream(stream))


def hp_attention_decode_workspace_bytes(desc, num_q_heads):
    n = ctypes.c_uint64(0)
    rc = lib().hp_attention_decode_workspace_bytes(desc.ref, num_q_heads, ctypes.byref(n))
    return rc, n.value


def hp_attention_decode(desc, v_pool, q, num_q_heads, scale, out, workspace, d_status=None,
                        stream=None):
    return lib().hp_attention_decode(desc.ref, _p(v_pool), _p(q), num_q_heads, float(scale),
                                     _p(out), _p(workspace), _wsn(workspace), _p(d_status),
                                     _stream(stream))


def hp_attention_plan(desc, num_q_heads, workspace, d_status=None, stream=None):
    return lib().hp_attention_plan(desc.ref, num_q_heads, _p(workspace), _wsn(workspace),
                                   _p(d_status), _stream(stream))


def hp_attention_decode_planned(desc, v_pool, q, num_q_heads, scale, out, workspace,
                                d_status=None, stream=None):
    return lib().hp_attention_decode_planned(desc.ref, _p(v_pool), _p(q), num_q_heads,
                                             float(scale), _p(out), _p(workspace),
                                             _wsn(workspace), _p(d_status), _stream(stream))


def _ref(struct):
    return None if struct is None else ctypes.byref(struct)


def hp_step_tables_workspace_bytes(num_seqs):
    n = ctypes.c_uint64(0)
    rc = lib().hp_step_tables_workspace_bytes(num_seqs, ctypes.byref(n))
    return rc, n.value


def hp_step_tables(step, workspace, d_status=None, stream=None):
    return lib().hp_step_tables(_ref(step), _p(workspace), _wsn(workspace), _p(d_status),
                                _stream(stream))


def hp_qk_norm_rope_append(qk, rope, d_status=None, stream=None):
    return lib().hp_qk_norm_rope_append(_ref(qk), _ref(rope), _p(d_status), _stream(stream))


def hp_latent_append(latent, rope, d_status=None, stream=None):
    return lib().hp_latent_append(_ref(latent), _ref(rope), _p(d_status), _stream(stream))


def hp_latent_decode_workspace_bytes(desc, latent_dim, total_q, num_q_heads):
    n = ctypes.c_uint64(0)
    rc = lib().hp_latent_decode_workspace_bytes(desc.ref, latent_dim, total_q, num_q_heads,
                                                ctypes.byref(n))
    return rc, n.value


def hp_latent_decode(desc, latent_dim, q, q_ptr, total_q, num_q_heads, scale, out, workspace,
                     d_status=None, stream=None):
    return lib().hp_latent_decode(desc.ref, latent_dim, _p(q), _p(q_ptr), total_q, num_q_heads,
                                  float(scale), _p(out), _p(workspace), _wsn(workspace),
                                  _p(d_status), _stream(stream))


def hp_latent_plan(desc, latent_dim, q_ptr, total_q, num_q_heads, workspace, d_status=None,
                   stream=None):
    return lib().hp_latent_plan(desc.ref, latent_dim, _p(q_ptr), total_q, num_q_heads,
                                _p(workspace), _wsn(workspace), _p(d_status), _stream(stream))


def hp_latent_decode_planned(desc, latent_dim, q, q_ptr, total_q, num_q_heads, scale, out,
                             workspace, d_status=None, stream=None):
    return lib().hp_latent_decode_planned(desc.ref, latent_dim, _p(q), _p(q_ptr), total_q,
                                          num_q_heads, float(scale), _p(out), _p(workspace),
                                          _wsn(workspace), _p(d_status), _stream(stream))


def hp_latent_prefill_workspace_bytes(desc, latent_dim, nope_dim, v_dim, total_q, num_q_heads,
                                      kv_tokens):
    n = ctypes.c_uint64(0)
    rc = lib().hp_latent_prefill_workspace_bytes(desc.ref, latent_dim, nope_dim, v_dim, total_q,
                                                 num_q_heads, kv_tokens, ctypes.byref(n))
    return rc, n.value


def hp_latent_prefill(desc, latent_dim, w_kv, nope_dim, v_dim, q, q_ptr, total_q, num_q_heads,
                      scale, out, kv_tokens, workspace, d_status=None, stream=None):
    return lib().hp_latent_prefill(desc.ref, latent_dim, _p(w_kv), nope_dim, v_dim, _p(q),
                                   _p(q_ptr), total_q, num_q_heads, float(scale), _p(out),
                                   kv_tokens, _p(workspace), _wsn(workspace), _p(d_status),
                                   _stream(stream))


def hp_page_bounds(desc, new_ptr, total_new, bounds, d_status=None, stream=None):
    _contiguous("hp_page_bounds", new_ptr=new_ptr, bounds=bounds)
    return lib().hp_page_bounds(desc.ref, _p(new_ptr), total_new, _p(bounds), _p(d_status),
                                _stream(stream))


def hp_page_scores(desc, bounds, q, q_ptr, total_q, num_q_heads, scale, scores, max_pages,
                   d_status=None, stream=None):
    _contiguous("hp_page_scores", bounds=bounds, q=q, q_ptr=q_ptr, scores=scores)
    return lib().hp_page_scores(desc.ref, _p(bounds), _p(q), _p(q_ptr), total_q, num_q_heads,
                                float(scale), _p(scores), max_pages, _p(d_status),
                                _stream(stream))


def hp_select_pages(desc, q_ptr, total_q, scores, max_pages, sinks, recent, k, selected,
                    d_status=None, stream=None):
    _contiguous("hp_select_pages", q_ptr=q_ptr, scores=scores, selected=selected)
    return lib().hp_select_pages(desc.ref, _p(q_ptr), total_q, _p(scores), max_pages, sinks,
                                 recent, k, _p(selected), _p(d_status), _stream(stream))


def hp_attention_pages(desc, v_pool, q, q_ptr, total_q, num_q_heads, scale, selected, k, out,
                       d_status=None, stream=None):
    _contiguous("hp_attention_pages", v_pool=v_pool, q=q, q_ptr=q_ptr, selected=selected, out=out)
    return lib().hp_attention_pages(desc.ref, _p(v_pool), _p(q), _p(q_ptr), total_q, num_q_heads,
                                    float(scale), _p(selected), k, _p(out), _p(d_status),
                                    _stream(stream))


def hp_attention_prefix_workspace_bytes(desc, num_groups, total_q, num_q_heads):
    n = ctypes.c_uint64(0)
    rc = lib().hp_attention_prefix_workspace_bytes(desc.ref, num_groups, total_q, num_q_heads,
                                                   ctypes.byref(n))
    return rc, n.value


def hp_attention_prefix(desc, v_pool, group_ptr, prefix_lens, num_groups, q, q_ptr, total_q,
                        num_q_heads, scale, out, workspace, d_status=None, stream=None):
    _contiguous("hp_attention_prefix", v_pool=v_pool, group_ptr=group_ptr,
                prefix_lens=prefix_lens, q=q, q_ptr=q_ptr, out=out)
    return lib().hp_attention_prefix(desc.ref, _p(v_pool), _p(group_ptr), _p(prefix_lens),
                                     num_groups, _p(q), _p(q_ptr), total_q, num_q_heads,
                                     float(scale), _p(out), _p(workspace), _wsn(workspace),
                                     _p(d_status), _stream(stream))


def hp_attention_prefix_plan(desc, group_ptr, prefix_lens, num_groups, q_ptr, total_q,
                             num_q_heads, workspace, d_status=None, stream=None):
    _contiguous("hp_attention_prefix_plan", group_ptr=group_ptr, prefix_lens=prefix_lens,
                q_ptr=q_ptr)
    return lib().hp_attention_prefix_plan(desc.ref, _p(group_ptr), _p(prefix_lens), num_groups,
                                          _p(q_ptr), total_q, num_q_heads, _p(workspace),
                                          _wsn(workspace), _p(d_status), _stream(stream))


def hp_attention_prefix_planned(desc, v_pool, group_ptr, prefix_lens, num_groups, q, q_ptr,
                                total_q, num_q_heads, scale, out, workspace, d_status=None,
                                stream=None):
    _contiguous("hp_attention_prefix_planned", v_pool=v_pool, group_ptr=group_ptr,
                prefix_lens=prefix_lens, q=q, q_ptr=q_ptr, out=out)
    return lib().hp_attention_prefix_planned(desc.ref, _p(v_pool), _p(group_ptr),
                                             _p(prefix_lens), num_groups, _p(q), _p(q_ptr),
                                             total_q, num_q_heads, float(scale), _p(out),
                                             _p(workspace), _wsn(workspace), _p(d_status),
                                             _stream(stream))


def hp_from_kernel_layout(src, dst, num_blocks, block_size, num_heads, head_dim, x, dtype,
                          stream=None):
    dt = DTYPES[dtype] if isinstance(dtype, str) else dtype
    return lib().hp_from_kernel_layout(_p(src), _p(dst), num_blocks, block_size, num_heads,
                                       head_dim, x, dt, _stream(stream))


def hp_to_kernel_layout(src, dst, num_blocks, block_size, num_heads, head_dim, x, dtype,
                        stream=None):
    dt = DTYPES[dtype] if isinstance(dtype, str) else dtype
    return lib().hp_to_kernel_layout(_p(src), _p(dst), num_blocks, block_size, num_heads,
                                     head_dim, x, dt, _stream(stream))


def hp_table_workspace_bytes(batch):
    n = ctypes.c_uint64(0)
    rc = lib().hp_table_workspace_bytes(batch, ctypes.byref(n))
    return rc, n.value


def hp_padded_to_csr(padded, lens, batch, max_blocks, page_size, index_type, table_out,
                     table_cap, seq_ptr_out, workspace, d_status=None, stream=None):
    return lib().hp_padded_to_csr(_p(padded), _p(lens), batch, max_blocks, page_size, index_type,
                                  _p(table_out), table_cap, _p(seq_ptr_out), _p(workspace),
                                  _wsn(workspace), _p(d_status), _stream(stream))


def hp_csr_to_padded(table, table_len, seq_ptr, batch, max_blocks, pad, index_type, padded_out,
                     workspace, d_status=None, stream=None):
    return lib().hp_csr_to_padded(_p(table), table_len, _p(seq_ptr), batch, max_blocks, pad,
                                  index_type, _p(padded_out), _p(workspace), _wsn(workspace),
                                  _p(d_status), _stream(stream))


def hp_gather_noalloc(desc, out, out_tokens, d_status=None, stream=None):
    """hp_gather with the library's built-in scratch instead of a caller workspace, for
    callers that cannot allocate device memory (at most 16384 sequences; calls must not
    overlap on the GPU)."""
    return lib().hp_gather_noalloc(desc.ref, _p(out), out_tokens, _p(d_status), _stream(stream))


def workspace_for(desc: PagedDesc, device="cuda"):
    """A zeroed, 256-byte-aligned uint8 device workspace of hp_workspace_bytes bytes."""
    import torch
    rc, n = hp_workspace_bytes(desc)
    if rc:
        raise RuntimeError(status_name(rc))
    return torch.zeros(max(n, 256), dtype=torch.uint8, device=device)
