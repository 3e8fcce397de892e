"""libpagedkv -- paged KV-cache write and paged decode attention for GB300.

Python binding of the C ABI in ``include/pagedkv.h``: every function here has
the C entry point's name and only marshals arguments (torch tensors -> device
pointers, shapes -> sizes, the current torch stream -> cudaStream_t).  All of
the work runs in the CUDA kernels of ``libpagedkv.so``; there is no other
implementation behind these names.  Build the library with
``paged_kv_cache_131_gb300._build.build()`` (or ``__graft_entry__.build()``).
"""

from __future__ import annotations

import ctypes
import os

__all__ = [
    "PkvError", "pkv_view", "pkv_write_desc", "pkv_decode_options", "library_path", "load",
    "pkv_cache_write", "pkv_decode_attention", "pkv_decode_workspace_bytes",
    "pkv_decode_workspace_init", "pkv_get_device_error", "pkv_status_string",
    "pkv_last_error_string", "pkv_version", "EXPORTED_SYMBOLS", "pkv_chunk_attention",
    "pkv_chunk_workspace_bytes", "pkv_norm_rope", "pkv_cache_desc", "pkv_norm_rope_write",
    "pkv_norm_rope_write_fp8", "pkv_cache_read_fp8", "pkv_tree_attention",
    "pkv_tree_attention_fp8", "pkv_tree_workspace_bytes", "pkv_tree_accept",
    "PKV_MAX_TREE_NODES", "PKV_MAX_ACCEPT_DEPTH",
    "PKV_COMPUTE_AUTO", "PKV_COMPUTE_SIMT", "PKV_COMPUTE_MMA", "PKV_SCHEDULE_AUTO",
    "PKV_SCHEDULE_GRID", "PKV_SCHEDULE_BALANCED", "DEVICE_ERRORS",
]

_HERE = os.path.dirname(os.path.abspath(__file__))
library_path = os.path.join(_HERE, "libpagedkv.so")

PKV_COMPUTE_AUTO, PKV_COMPUTE_SIMT, PKV_COMPUTE_MMA = 0, 1, 2
PKV_SCHEDULE_AUTO, PKV_SCHEDULE_GRID, PKV_SCHEDULE_BALANCED = 0, 1, 2
PKV_MAX_TREE_NODES, PKV_MAX_ACCEPT_DEPTH = 256, 256
DEVICE_ERRORS = {0: "none", 1: "slot", 2: "block_id", 3: "seq_len", 4: "timeout", 5: "position",
                 6: "path"}

EXPORTED_SYMBOLS = [
    "pkv_cache_write", "pkv_decode_attention", "pkv_decode_attention_ex",
    "pkv_decode_workspace_bytes", "pkv_decode_workspace_bytes_ex", "pkv_decode_workspace_init",
    "pkv_get_device_error", "pkv_status_string", "pkv_last_error_string", "pkv_version",
    "pkv_decode_attention_noalloc", "pkv_cache_write_multi", "pkv_copy_blocks",
    "pkv_cache_write_fp8", "pkv_decode_attention_fp8", "pkv_chunk_attention",
    "pkv_chunk_workspace_bytes", "pkv_norm_rope_write", "pkv_norm_rope_write_fp8",
    "pkv_cache_read_fp8", "pkv_tree_attention", "pkv_tree_attention_fp8",
    "pkv_tree_workspace_bytes", "pkv_tree_accept",
]


class PkvError(RuntimeError):
    def __init__(self, status: int, where: str):
        msg = pkv_status_string(status)
        if status == -6:
            msg += f" [{pkv_last_error_string()}]"
        super().__init__(f"{where}: {msg}")
        self.status = status


class pkv_view(ctypes.Structure):
    _fields_ = [("offset", ctypes.c_int64), ("layer_stride", ctypes.c_int64),
                ("block_stride", ctypes.c_int64), ("row_width", ctypes.c_int64),
                ("layer", ctypes.c_int32)]


class pkv_write_desc(ctypes.Structure):
    _fields_ = [("src", ctypes.c_void_p), ("cache", ctypes.c_void_p), ("view", pkv_view)]


class pkv_decode_options(ctypes.Structure):
    _fields_ = [("partition_size", ctypes.c_int32), ("compute", ctypes.c_int32),
                ("schedule", ctypes.c_int32)]


class pkv_norm_rope(ctypes.Structure):
    _fields_ = [("q_weight", ctypes.c_void_p), ("k_weight", ctypes.c_void_p),
                ("eps", ctypes.c_float), ("cos_sin", ctypes.c_void_p),
                ("max_position", ctypes.c_int64), ("rot_dim", ctypes.c_int32),
                ("interleaved", ctypes.c_int32)]


class pkv_cache_desc(ctypes.Structure):
    _fields_ = [("cache", ctypes.c_void_p), ("view", pkv_view)]


_lib = None
_i32, _i64, _p, _sz = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p, ctypes.c_size_t


def load(path: str | None = None):
    """Load libpagedkv.so (raises if it has not been built)."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    path = path or library_path
    if not os.path.exists(path):
        raise ImportError(f"libpagedkv.so is not built ({path}); run "
                          "paged_kv_cache_131_gb300._build.build()")
    lib = ctypes.CDLL(path)
    lib.pkv_cache_write.restype = ctypes.c_int
    lib.pkv_cache_write.argtypes = [_p, _p, _p, _i64, _p, _p, pkv_view, _i32, _i64, _p]
    lib.pkv_cache_write_multi.restype = ctypes.c_int
    lib.pkv_cache_write_multi.argtypes = [ctypes.POINTER(pkv_write_desc), _i32, _p, _i64, _i32,
                                          _i64, _p]
    lib.pkv_cache_write_fp8.restype = ctypes.c_int
    lib.pkv_cache_write_fp8.argtypes = [_p, _p, _p, _i64, _p, _p, _p, _p, _i32, _i32, _i32, _i64,
                                        _p]
    lib.pkv_copy_blocks.restype = ctypes.c_int
    lib.pkv_copy_blocks.argtypes = [_p, pkv_view, _i32, _i32, _p, _i64, _i64, _p]
    dec = [_p, _p, _p, _p, _p, _p, ctypes.c_float, _i32, _i32, _i32, _i32, _i32, _i32, _i32,
           _i64, _p, _sz]
    lib.pkv_decode_attention.restype = ctypes.c_int
    lib.pkv_decode_attention.argtypes = dec + [_p]
    lib.pkv_decode_attention_ex.restype = ctypes.c_int
    lib.pkv_decode_attention_ex.argtypes = dec + [ctypes.POINTER(pkv_decode_options), _p]
    lib.pkv_decode_attention_fp8.restype = ctypes.c_int
    lib.pkv_decode_attention_fp8.argtypes = dec[:4] + [_p, _p] + dec[4:] + [_p]
    lib.pkv_decode_attention_noalloc.restype = ctypes.c_int
    lib.pkv_decode_attention_noalloc.argtypes = dec[:15] + [_p]
    lib.pkv_chunk_attention.restype = ctypes.c_int
    lib.pkv_chunk_attention.argtypes = [_p, _p, _p, _p, _p, _p, _p, ctypes.c_float, _i32, _i32,
                                        _i32, _i32, _i32, _i32, _i32, _i32, _i32, _i64, _p, _sz,
                                        _p]
    lib.pkv_chunk_workspace_bytes.restype = _sz
    lib.pkv_chunk_workspace_bytes.argtypes = [_i32] * 7
    nrw = [_p, _p, _p, _p, _i64, _i64, _i64, ctypes.POINTER(pkv_norm_rope), _p, _p, _i64, _p, _p]
    lib.pkv_norm_rope_write.restype = ctypes.c_int
    lib.pkv_norm_rope_write.argtypes = nrw + [_i32, _i32, _i32, _i32, _i64, _p]
    lib.pkv_norm_rope_write_fp8.restype = ctypes.c_int
    lib.pkv_norm_rope_write_fp8.argtypes = nrw + [_p, _p, _i32, _i32, _i32, _i32, _i64, _p]
    lib.pkv_cache_read_fp8.restype = ctypes.c_int
    lib.pkv_cache_read_fp8.argtypes = [_p, _p, _p, _i64, _p, _p, _p, _p, _i32, _i32, _i32, _i64,
                                       _p]
    tree = [_p, _p, _p, _i32, ctypes.c_float] + [_i32] * 9 + [_i64, _p, _sz, _p]
    lib.pkv_tree_attention.restype = ctypes.c_int
    lib.pkv_tree_attention.argtypes = [_p] * 5 + tree
    lib.pkv_tree_attention_fp8.restype = ctypes.c_int
    lib.pkv_tree_attention_fp8.argtypes = [_p] * 7 + tree
    lib.pkv_tree_workspace_bytes.restype = _sz
    lib.pkv_tree_workspace_bytes.argtypes = [_i32] * 7
    lib.pkv_tree_accept.restype = ctypes.c_int
    lib.pkv_tree_accept.argtypes = [ctypes.POINTER(pkv_cache_desc), _i32, _i32, _p, _i32, _p, _p,
                                    _i32, _i32, _i32, _i64, _p]
    lib.pkv_decode_workspace_bytes.restype = _sz
    lib.pkv_decode_workspace_bytes.argtypes = [_i32, _i32, _i32, _i32, _i32]
    lib.pkv_decode_workspace_bytes_ex.restype = _sz
    lib.pkv_decode_workspace_bytes_ex.argtypes = [_i32, _i32, _i32, _i32, _i32, _i32]
    lib.pkv_decode_workspace_init.restype = ctypes.c_int
    lib.pkv_decode_workspace_init.argtypes = [_p, _sz, _p]
    lib.pkv_get_device_error.restype = ctypes.c_int
    lib.pkv_get_device_error.argtypes = [ctypes.POINTER(_i32), ctypes.POINTER(_i64), _p]
    lib.pkv_status_string.restype = ctypes.c_char_p
    lib.pkv_status_string.argtypes = [ctypes.c_int]
    lib.pkv_last_error_string.restype = ctypes.c_char_p
    lib.pkv_last_error_string.argtypes = []
    lib.pkv_version.restype = ctypes.c_int
    lib.pkv_version.argtypes = []
    if path == library_path:
        _lib = lib
    return lib


# ------------------------------------------------------------------ marshalling


def _dev(t, name, dtype=None):
    """Device pointer of a CUDA tensor (None -> NULL)."""
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    return t.data_ptr()


def _stream(stream):
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    return getattr(stream, "cuda_stream", stream)


def _check(status: int, where: str) -> int:
    if status != 0:
        raise PkvError(status, where)
    return status


def pkv_cache_write(k, v, slot_mapping, k_cache, v_cache, view, block_size: int,
                    num_blocks: int, stream=None, check: bool = True) -> int:
    """Scatter ``k`` (and ``v``) rows to their slots: see pkv_cache_write in pagedkv.h.

    k, v: CUDA tensors of num_tokens rows of ``view.row_width`` bytes; slot_mapping:
    CUDA int64 [num_tokens]; caches: CUDA tensors (any dtype, used as bytes);
    view: pkv_view or an object with offset/layer_stride/block_stride/row_width
    (and optionally layer).
    """
    import torch
    if not isinstance(view, pkv_view):
        view = pkv_view(view.offset, view.layer_stride, view.block_stride, view.row_width,
                        getattr(view, "layer", 0))
    n = slot_mapping.numel()
    if k.numel() * k.element_size() != n * view.row_width:
        raise ValueError("k must hold num_tokens rows of view.row_width bytes")
    if v is not None and v.numel() * v.element_size() != n * view.row_width:
        raise ValueError("v must hold num_tokens rows of view.row_width bytes")
    st = load().pkv_cache_write(
        _dev(k, "k"), _dev(v, "v"), _dev(slot_mapping, "slot_mapping", torch.int64), n,
        _dev(k_cache, "k_cache"), _dev(v_cache, "v_cache"), view, block_size, num_blocks,
        _stream(stream))
    return _check(st, "pkv_cache_write") if check else st


def _as_view(view) -> pkv_view:
    if isinstance(view, pkv_view):
        return view
    return pkv_view(view.offset, view.layer_stride, view.block_stride, view.row_width,
                    getattr(view, "layer", 0))


def pkv_cache_write_multi(writes, slot_mapping, block_size: int, num_blocks: int, stream=None,
                          check: bool = True) -> int:
    """One launch for several writes sharing ``slot_mapping``: see pkv_cache_write_multi.

    writes: sequence of (src, cache, view) with CUDA tensors and pkv_view-like views.
    """
    import torch
    n = slot_mapping.numel()
    arr = (pkv_write_desc * max(1, len(writes)))()
    for i, (src, cache, view) in enumerate(writes):
        view = _as_view(view)
        if src.numel() * src.element_size() != n * view.row_width:
            raise ValueError(f"write {i}: src must hold num_tokens rows of row_width bytes")
        arr[i] = pkv_write_desc(_dev(src, f"writes[{i}].src"), _dev(cache, f"writes[{i}].cache"),
                                view)
    st = load().pkv_cache_write_multi(arr, len(writes),
                                      _dev(slot_mapping, "slot_mapping", torch.int64), n,
                                      block_size, num_blocks, _stream(stream))
    return _check(st, "pkv_cache_write_multi") if check else st


def pkv_copy_blocks(cache, view, num_layers: int, block_size: int, block_mapping,
                    num_blocks: int, stream=None, check: bool = True) -> int:
    """Copy whole blocks of a view for each (src, dst) row of ``block_mapping``
    (CUDA int64 [N, 2]): see pkv_copy_blocks in pagedkv.h."""
    import torch
    st = load().pkv_copy_blocks(_dev(cache, "cache"), _as_view(view), num_layers, block_size,
                                _dev(block_mapping, "block_mapping", torch.int64),
                                block_mapping.numel() // 2, num_blocks, _stream(stream))
    return _check(st, "pkv_copy_blocks") if check else st


def pkv_decode_attention(out, q, k_cache, v_cache, block_tables, seq_lens, scale: float,
                         num_heads: int, num_kv_heads: int, head_dim: int, block_size: int,
                         max_seq_len: int, num_blocks: int, workspace=None, stream=None,
                         partition_size: int = 0, compute: int = PKV_COMPUTE_AUTO,
                         schedule: int = PKV_SCHEDULE_AUTO, check: bool = True) -> int:
    """Paged decode attention: see pkv_decode_attention(_ex) in pagedkv.h.

    out, q: CUDA fp16 [S, H, D]; caches: CUDA fp16 [NB, bs, Hk, D];
    block_tables: CUDA int32 [S, MB]; seq_lens: CUDA int32 [S];
    workspace: CUDA uint8 tensor (zero-filled before first use) or None.
    """
    import torch
    S = q.shape[0]
    if tuple(out.shape) != tuple(q.shape):
        raise ValueError("out must have q's shape")
    ws_ptr, ws_bytes = None, 0
    if workspace is not None:
        ws_ptr, ws_bytes = _dev(workspace, "workspace"), workspace.numel() * workspace.element_size()
    args = (_dev(out, "out", torch.float16), _dev(q, "q", torch.float16),
            _dev(k_cache, "k_cache", torch.float16), _dev(v_cache, "v_cache", torch.float16),
            _dev(block_tables, "block_tables", torch.int32), _dev(seq_lens, "seq_lens", torch.int32),
            float(scale), num_heads, num_kv_heads, head_dim, block_size, S,
            block_tables.shape[1] if block_tables.dim() == 2 else 0, int(max_seq_len),
            int(num_blocks), ws_ptr, ws_bytes)
    lib = load()
    if partition_size == 0 and compute == PKV_COMPUTE_AUTO and schedule == PKV_SCHEDULE_AUTO:
        st = lib.pkv_decode_attention(*args, _stream(stream))
    else:
        opts = pkv_decode_options(partition_size, compute, schedule)
        st = lib.pkv_decode_attention_ex(*args, ctypes.byref(opts), _stream(stream))
    return _check(st, "pkv_decode_attention") if check else st


def pkv_chunk_attention(out, q, k_cache, v_cache, block_tables, seq_lens, query_start,
                        scale: float, num_heads: int, num_kv_heads: int, head_dim: int,
                        block_size: int, max_query_len: int, max_seq_len: int, num_blocks: int,
                        workspace=None, stream=None, check: bool = True) -> int:
    """Causal attention of each sequence's new tokens: see pkv_chunk_attention in
    pagedkv.h.

    out, q: CUDA fp16 [Tq, H, D]; caches: CUDA fp16 [NB, bs, Hk, D];
    block_tables: CUDA int32 [S, MB]; seq_lens: CUDA int32 [S];
    query_start: CUDA int32 [S + 1]; workspace: CUDA uint8 tensor (zero-filled
    before first use).
    """
    import torch
    if tuple(out.shape) != tuple(q.shape):
        raise ValueError("out must have q's shape")
    ws_ptr, ws_bytes = None, 0
    if workspace is not None:
        ws_ptr, ws_bytes = _dev(workspace, "workspace"), workspace.numel() * workspace.element_size()
    S = seq_lens.numel()
    st = load().pkv_chunk_attention(
        _dev(out, "out", torch.float16), _dev(q, "q", torch.float16),
        _dev(k_cache, "k_cache", torch.float16), _dev(v_cache, "v_cache", torch.float16),
        _dev(block_tables, "block_tables", torch.int32), _dev(seq_lens, "seq_lens", torch.int32),
        _dev(query_start, "query_start", torch.int32), float(scale), num_heads, num_kv_heads,
        head_dim, block_size, S, block_tables.shape[1] if block_tables.dim() == 2 else 0,
        q.shape[0], int(max_query_len), int(max_seq_len), int(num_blocks), ws_ptr, ws_bytes,
        _stream(stream))
    return _check(st, "pkv_chunk_attention") if check else st


def pkv_chunk_workspace_bytes(num_seqs: int, num_heads: int, num_kv_heads: int, head_dim: int,
                              num_query_tokens: int, max_query_len: int, max_seq_len: int) -> int:
    return load().pkv_chunk_workspace_bytes(num_seqs, num_heads, num_kv_heads, head_dim,
                                            num_query_tokens, max_query_len, max_seq_len)


def pkv_cache_write_fp8(k, v, slot_mapping, k_cache, v_cache, k_scale, v_scale, block_size: int,
                        num_blocks: int, stream=None, check: bool = True) -> int:
    """Quantize-on-write of fp16 rows k, v [T, Hk, D] into E4M3 caches
    (uint8 [NB, bs, Hk, D]) and fp32 scales [NB, bs, Hk]: see pagedkv.h."""
    import torch
    NB, bs, Hk, D = k_cache.shape
    st = load().pkv_cache_write_fp8(
        _dev(k, "k", torch.float16), _dev(v, "v", torch.float16),
        _dev(slot_mapping, "slot_mapping", torch.int64), slot_mapping.numel(),
        _dev(k_cache, "k_cache", torch.uint8), _dev(v_cache, "v_cache", torch.uint8),
        _dev(k_scale, "k_scale", torch.float32), _dev(v_scale, "v_scale", torch.float32),
        Hk, D, block_size, num_blocks, _stream(stream))
    return _check(st, "pkv_cache_write_fp8") if check else st


def pkv_decode_attention_fp8(out, q, k_cache, v_cache, k_scale, v_scale, block_tables, seq_lens,
                             scale: float, num_heads: int, num_kv_heads: int, head_dim: int,
                             block_size: int, max_seq_len: int, num_blocks: int, workspace,
                             stream=None, check: bool = True) -> int:
    """Paged decode attention over E4M3 caches: see pkv_decode_attention_fp8."""
    import torch
    st = load().pkv_decode_attention_fp8(
        _dev(out, "out", torch.float16), _dev(q, "q", torch.float16),
        _dev(k_cache, "k_cache", torch.uint8), _dev(v_cache, "v_cache", torch.uint8),
        _dev(k_scale, "k_scale", torch.float32), _dev(v_scale, "v_scale", torch.float32),
        _dev(block_tables, "block_tables", torch.int32), _dev(seq_lens, "seq_lens", torch.int32),
        float(scale), num_heads, num_kv_heads, head_dim, block_size, q.shape[0],
        block_tables.shape[1], int(max_seq_len), int(num_blocks), _dev(workspace, "workspace"),
        workspace.numel() * workspace.element_size(), _stream(stream))
    return _check(st, "pkv_decode_attention_fp8") if check else st


# The speculative step's calls are short kernels in a latency-bound loop: their
# tensors are checked with one pass of cheap attribute reads each, and the
# stream is taken as a raw handle (a torch.cuda.Stream object costs 3 us).


def _current(t, name):
    """The current device's index, which ``t`` must be on."""
    import torch
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    if dev != torch.cuda.current_device():
        raise ValueError(f"{name} is on {t.device}, not on the current device")
    return dev


def _arg(t, name, dtype, shape, dev):
    """Device pointer of a contiguous tensor of this dtype and shape on device ``dev``."""
    if t is None:
        raise ValueError(f"{name} is missing")
    if t.dtype is not dtype or t.shape != shape or t.get_device() != dev or not t.is_contiguous():
        if t.get_device() != dev:
            raise ValueError(f"{name} must be a CUDA tensor of device {dev}, is on {t.device}")
        if t.dtype is not dtype:
            raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
        if t.shape != shape:
            raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _raw_stream(stream, dev):
    if stream is None:
        import torch
        return torch._C._cuda_getCurrentRawStream(dev)
    return getattr(stream, "cuda_stream", stream)


def _token_rows(t, name, dtype, shape, dev):
    """(device pointer, token stride in elements) of rows [T, heads, D] whose heads
    are packed; tokens may be strided (a slice of a packed QKV row)."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != dev:
        _arg(t, name, dtype, shape, dev)
    T, h, D = shape
    st, sh, sd = t.stride()
    if (D > 1 and sd != 1) or (h > 1 and sh != D):
        raise ValueError(f"{name}: a token's heads must be packed")
    return t.data_ptr(), st if T > 1 else h * D


def _workspace(workspace, dev):
    """(device pointer, bytes) of a workspace tensor, or of none."""
    if workspace is None:
        return None, 0
    if workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous CUDA tensor of the call's device")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


def _norm_rope_write(name, q_out, q, k, v, positions, slot_mapping, k_cache, v_cache, scales,
                     cos_sin, q_weight, k_weight, eps, interleaved, block_size, num_blocks,
                     stream, check):
    import torch
    f16, i64, f32 = torch.float16, torch.int64, torch.float32
    dev = _current(q, "q")
    if q.dim() != 3 or k.dim() != 3:
        raise ValueError("q must be [T, H, D], k [T, Hk, D]")
    T, H, D = q.shape
    Hk = k.shape[1]
    qp, qs = _token_rows(q, "q", f16, (T, H, D), dev)
    kp, ks = _token_rows(k, "k", f16, (T, Hk, D), dev)
    vp, vs = _token_rows(v, "v", f16, (T, Hk, D), dev)
    rot = max_pos = 0
    table = pos = None
    if cos_sin is not None:
        if cos_sin.dim() != 2:
            raise ValueError("cos_sin must be [max_position, rot_dim]")
        max_pos, rot = cos_sin.shape
        table = _arg(cos_sin, "cos_sin", f32, (max_pos, rot), dev)
        if rot:
            pos = _arg(positions, "positions", i64, (T,), dev)
    nr = pkv_norm_rope(
        None if q_weight is None else _arg(q_weight, "q_weight", f16, (D,), dev),
        None if k_weight is None else _arg(k_weight, "k_weight", f16, (D,), dev),
        eps, table, max_pos, rot, bool(interleaved))
    kind = f16 if scales is None else torch.uint8
    if num_blocks is None:
        num_blocks = k_cache.shape[0]
    rows = (num_blocks, block_size, Hk, D)
    args = [_arg(q_out, "q_out", f16, (T, H, D), dev), qp, kp, vp, qs, ks, vs, ctypes.byref(nr),
            pos, _arg(slot_mapping, "slot_mapping", i64, (T,), dev), T,
            _arg(k_cache, "k_cache", kind, rows, dev), _arg(v_cache, "v_cache", kind, rows, dev)]
    if scales is not None:
        args += [_arg(scales[0], "k_scale", f32, rows[:3], dev),
                 _arg(scales[1], "v_scale", f32, rows[:3], dev)]
    st = getattr(load(), name)(*args, H, Hk, D, block_size, num_blocks, _raw_stream(stream, dev))
    return _check(st, name) if check else st


def pkv_norm_rope_write(q_out, q, k, v, positions, slot_mapping, k_cache, v_cache, cos_sin=None,
                        q_weight=None, k_weight=None, eps: float = 1e-6,
                        interleaved: bool = False, block_size: int = 16,
                        num_blocks: int | None = None, stream=None, check: bool = True) -> int:
    """Per-head norm, rotation and cache write in one pass: see pkv_norm_rope_write
    in pagedkv.h.

    q [T, H, D], k, v [T, Hk, D]: CUDA fp16, tokens may be strided; q_out: CUDA
    fp16 [T, H, D]; positions, slot_mapping: CUDA int64 [T]; caches: CUDA fp16
    [NB, bs, Hk, D]; cos_sin: CUDA fp32 [max_position, rot_dim] or None;
    q_weight, k_weight: CUDA fp16 [D] or None; num_blocks: the caches' NB when not
    given.
    """
    return _norm_rope_write("pkv_norm_rope_write", q_out, q, k, v, positions, slot_mapping,
                            k_cache, v_cache, None, cos_sin, q_weight, k_weight, eps, interleaved,
                            block_size, num_blocks, stream, check)


def pkv_norm_rope_write_fp8(q_out, q, k, v, positions, slot_mapping, k_cache, v_cache, k_scale,
                            v_scale, cos_sin=None, q_weight=None, k_weight=None,
                            eps: float = 1e-6, interleaved: bool = False, block_size: int = 16,
                            num_blocks: int | None = None, stream=None, check: bool = True) -> int:
    """pkv_norm_rope_write into E4M3 caches (uint8 [NB, bs, Hk, D]) and fp32 scales
    [NB, bs, Hk]: see pagedkv.h."""
    return _norm_rope_write("pkv_norm_rope_write_fp8", q_out, q, k, v, positions, slot_mapping,
                            k_cache, v_cache, (k_scale, v_scale), cos_sin, q_weight, k_weight, eps,
                            interleaved, block_size, num_blocks, stream, check)


def pkv_cache_read_fp8(k, v, slot_mapping, k_cache, v_cache, k_scale, v_scale, block_size: int,
                       num_blocks: int, stream=None, check: bool = True) -> int:
    """Rows of E4M3 caches read back into fp16 k, v [T, Hk, D]: see pkv_cache_read_fp8
    in pagedkv.h (v, v_cache, v_scale may all be None)."""
    import torch
    f16, f32, u8 = torch.float16, torch.float32, torch.uint8
    dev = _current(k, "k")
    T, Hk, D = k.shape
    rows = (num_blocks, block_size, Hk, D)
    ptrs = [_arg(k, "k", f16, (T, Hk, D), dev), _arg(k_cache, "k_cache", u8, rows, dev),
            _arg(k_scale, "k_scale", f32, rows[:3], dev)]
    if v is None and v_cache is None and v_scale is None:
        ptrs += [None, None, None]
    else:
        ptrs += [_arg(v, "v", f16, (T, Hk, D), dev), _arg(v_cache, "v_cache", u8, rows, dev),
                 _arg(v_scale, "v_scale", f32, rows[:3], dev)]
    st = load().pkv_cache_read_fp8(
        ptrs[0], ptrs[3], _arg(slot_mapping, "slot_mapping", torch.int64, (T,), dev), T, ptrs[1],
        ptrs[4], ptrs[2], ptrs[5], Hk, D, block_size, num_blocks, _raw_stream(stream, dev))
    return _check(st, "pkv_cache_read_fp8") if check else st


def _tree_attention(name, out, q, k_cache, v_cache, scales, block_tables, seq_lens, query_start,
                    tree_mask, scale, num_heads, num_kv_heads, head_dim, block_size,
                    max_query_len, max_seq_len, num_blocks, workspace, stream, check):
    import torch
    f16, f32, i32 = torch.float16, torch.float32, torch.int32
    dev = _current(q, "q")
    if block_tables.dim() != 2 or tree_mask.dim() != 2:
        raise ValueError("block_tables must be [S, MB], tree_mask [Tq, words]")
    Tq, S = q.shape[0], seq_lens.numel()
    MB, words = block_tables.shape[1], tree_mask.shape[1]
    qshape = (Tq, num_heads, head_dim)
    rows = (num_blocks, block_size, num_kv_heads, head_dim)
    kind = f16 if scales is None else torch.uint8
    args = [_arg(out, "out", f16, qshape, dev), _arg(q, "q", f16, qshape, dev),
            _arg(k_cache, "k_cache", kind, rows, dev), _arg(v_cache, "v_cache", kind, rows, dev)]
    if scales is not None:
        args += [_arg(scales[0], "k_scale", f32, rows[:3], dev),
                 _arg(scales[1], "v_scale", f32, rows[:3], dev)]
    st = getattr(load(), name)(
        *args, _arg(block_tables, "block_tables", i32, (S, MB), dev),
        _arg(seq_lens, "seq_lens", i32, (S,), dev),
        _arg(query_start, "query_start", i32, (S + 1,), dev),
        _arg(tree_mask, "tree_mask", torch.int64, (Tq, words), dev), words, scale, num_heads,
        num_kv_heads, head_dim, block_size, S, MB, Tq, max_query_len, max_seq_len, num_blocks,
        *_workspace(workspace, dev), _raw_stream(stream, dev))
    return _check(st, name) if check else st


def pkv_tree_attention(out, q, k_cache, v_cache, block_tables, seq_lens, query_start, tree_mask,
                       scale: float, num_heads: int, num_kv_heads: int, head_dim: int,
                       block_size: int, max_query_len: int, max_seq_len: int, num_blocks: int,
                       workspace=None, stream=None, check: bool = True) -> int:
    """Attention of a tree of drafted tokens per sequence: see pkv_tree_attention in
    pagedkv.h.

    out, q: CUDA fp16 [Tq, H, D]; caches: CUDA fp16 [NB, bs, Hk, D];
    block_tables: CUDA int32 [S, MB]; seq_lens: CUDA int32 [S]; query_start:
    CUDA int32 [S + 1]; tree_mask: CUDA int64 [Tq, words] (bit j % 64 of word
    j // 64: sees drafted token j); workspace: CUDA uint8 tensor of
    pkv_tree_workspace_bytes(...) bytes.
    """
    return _tree_attention("pkv_tree_attention", out, q, k_cache, v_cache, None, block_tables,
                           seq_lens, query_start, tree_mask, scale, num_heads, num_kv_heads,
                           head_dim, block_size, max_query_len, max_seq_len, num_blocks, workspace,
                           stream, check)


def pkv_tree_attention_fp8(out, q, k_cache, v_cache, k_scale, v_scale, block_tables, seq_lens,
                           query_start, tree_mask, scale: float, num_heads: int,
                           num_kv_heads: int, head_dim: int, block_size: int, max_query_len: int,
                           max_seq_len: int, num_blocks: int, workspace=None, stream=None,
                           check: bool = True) -> int:
    """pkv_tree_attention over E4M3 caches (uint8) and fp32 scales: see pagedkv.h."""
    return _tree_attention("pkv_tree_attention_fp8", out, q, k_cache, v_cache, (k_scale, v_scale),
                           block_tables, seq_lens, query_start, tree_mask, scale, num_heads,
                           num_kv_heads, head_dim, block_size, max_query_len, max_seq_len,
                           num_blocks, workspace, stream, check)


def pkv_tree_workspace_bytes(num_seqs: int, num_heads: int, num_kv_heads: int, head_dim: int,
                             num_query_tokens: int, max_query_len: int, max_seq_len: int) -> int:
    return int(load().pkv_tree_workspace_bytes(num_seqs, num_heads, num_kv_heads, head_dim,
                                               num_query_tokens, max_query_len, max_seq_len))


def _view_inside(cache, view, num_layers, block_size, num_blocks, name):
    """Refuses a view whose last row (of num_layers layers from view.layer on) lies
    past the end of the tensor ``cache``."""
    end = (view.offset + (view.layer + num_layers - 1) * view.layer_stride +
           (num_blocks - 1) * view.block_stride + block_size * view.row_width)
    if end > cache.nbytes:
        raise ValueError(f"{name}: the view's rows end at byte {end}, past the end of its tensor "
                         f"({cache.nbytes} bytes)")


def pkv_tree_accept(caches, num_layers: int, path, ctx_lens, block_tables, block_size: int,
                    num_blocks: int, stream=None, check: bool = True) -> int:
    """Move the cache rows of each sequence's accepted path to their positions: see
    pkv_tree_accept in pagedkv.h.

    caches: sequence of (cache, view) with a CUDA tensor, used as bytes, and a
    pkv_view-like view, whose rows -- num_layers layers from view.layer on, num_blocks
    blocks each -- lie inside the tensor (ValueError otherwise); path: CUDA int32
    [S, max_depth], negative past a path's end; ctx_lens: CUDA int32 [S];
    block_tables: CUDA int32 [S, MB].
    """
    import torch
    i32 = torch.int32
    dev = _current(path, "path")
    if path.dim() != 2 or block_tables.dim() != 2:
        raise ValueError("path must be [S, max_depth], block_tables [S, MB]")
    S, depth = path.shape
    MB = block_tables.shape[1]
    arr = (pkv_cache_desc * max(1, len(caches)))()
    for i, (cache, view) in enumerate(caches):
        arr[i].cache = _arg(cache, f"caches[{i}]", cache.dtype, cache.shape, dev)
        view = arr[i].view = _as_view(view)
        if S and depth and num_layers:
            _view_inside(cache, view, num_layers, block_size, num_blocks, f"caches[{i}]")
    st = load().pkv_tree_accept(
        arr, len(caches), num_layers, _arg(path, "path", i32, (S, depth), dev), depth,
        _arg(ctx_lens, "ctx_lens", i32, (S,), dev),
        _arg(block_tables, "block_tables", i32, (S, MB), dev), S, MB, block_size, num_blocks,
        _raw_stream(stream, dev))
    return _check(st, "pkv_tree_accept") if check else st


def pkv_decode_workspace_bytes(num_seqs: int, num_heads: int, num_kv_heads: int, head_dim: int,
                               max_seq_len: int, partition_size: int = 0) -> int:
    return int(load().pkv_decode_workspace_bytes_ex(num_seqs, num_heads, num_kv_heads, head_dim,
                                                    max_seq_len, partition_size))


def pkv_decode_workspace_init(workspace, stream=None) -> int:
    if workspace is None:
        return 0
    return _check(load().pkv_decode_workspace_init(
        _dev(workspace, "workspace"), workspace.numel() * workspace.element_size(),
        _stream(stream)), "pkv_decode_workspace_init")


def pkv_get_device_error(stream=None) -> tuple[int, int]:
    """Synchronise ``stream``; return and clear (kind, index) of the device error record."""
    kind, index = _i32(0), _i64(-1)
    _check(load().pkv_get_device_error(ctypes.byref(kind), ctypes.byref(index), _stream(stream)),
           "pkv_get_device_error")
    return kind.value, index.value


def pkv_status_string(status: int) -> str:
    return load().pkv_status_string(status).decode()


def pkv_last_error_string() -> str:
    return load().pkv_last_error_string().decode()


def pkv_version() -> int:
    return load().pkv_version()
