"""Thin Python binding of liblci.so (include/lci.h).

Argument marshalling only: every function checks the torch tensors it is given
(device, dtype, contiguity, shapes), takes their device pointers and the
current CUDA stream, and calls the C entry point of the same name. Outputs and
workspaces are torch allocations; the computation runs entirely in the
library's CUDA kernels. There is no fallback: if liblci.so is missing or fails
to load, every call raises.
"""
from __future__ import annotations

import ctypes
import os
import threading
import weakref
from typing import Dict, Optional, Tuple

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "liblci.so")

LCI_OK = 0
STATUS_NAMES = {0: "LCI_OK", 1: "LCI_ERR_INVALID_ARG", 2: "LCI_ERR_UNSUPPORTED",
                3: "LCI_ERR_WORKSPACE", 4: "LCI_ERR_CUDA", 5: "LCI_ERR_DEVICE_BOUNDS",
                6: "LCI_ERR_TIMEOUT"}
LCI_F32, LCI_BF16, LCI_E4M3 = 0, 1, 2
PHASES = {"auto": 0, "prefill": 1, "decode": 2}

# Every entry point of include/lci.h: name -> (restype, argtypes)
_vp, _i32, _sz, _f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t, ctypes.c_float
_st = ctypes.c_int
SIGNATURES = {
    "lci_version": (ctypes.c_char_p, []),
    "lci_status_string": (ctypes.c_char_p, [_st]),
    "lci_last_error": (ctypes.c_char_p, []),
    "lci_create_block_table": (_st, [_vp, _i32, _i32, _i32, _i32, _i32, _i32, _st,
                                     ctypes.POINTER(_vp)]),
    "lci_destroy_block_table": (_st, [_vp]),
    "lci_validate_block_table": (_st, [_vp, _vp]),
    "lci_block_compress": (_st, [_vp, _st, _i32, _i32, _i32, _i32, _i32, _vp, _vp]),
    "lci_index_select_workspace_size": (_st, [_i32, _i32, _i32, _i32, _i32, _i32, _st,
                                              ctypes.POINTER(_sz)]),
    "lci_index_select": (_st, [_vp, _vp, _st, _i32, _i32, _i32, _i32, _i32, _i32, _vp, _vp, _i32,
                               _st, _vp, _vp, _sz, _vp]),
    "lci_sparse_attn_workspace_size": (_st, [_i32, _i32, _i32, _i32, _vp, _st,
                                             ctypes.POINTER(_sz)]),
    "lci_sparse_attn": (_st, [_vp, _i32, _i32, _i32, _vp, _vp, _vp, _vp, _i32, _vp, _vp, _f32,
                              _st, _vp, _vp, _sz, _vp]),
    "lci_get_device_status": (_st, [_vp]),
    "lci_sparse_decode_workspace_size": (_st, [_i32, _i32, _i32, _i32, _i32, _i32, _vp,
                                               ctypes.POINTER(_sz)]),
    "lci_sparse_decode": (_st, [_vp, _vp, _st, _i32, _i32, _i32, _i32, _i32, _vp, _vp, _i32, _vp,
                                _i32, _vp, _vp, _vp, _f32, _vp, _vp, _vp, _sz, _vp]),
    "lci_index_select_noalloc": (_st, [_vp, _vp, _st, _i32, _i32, _i32, _i32, _i32, _i32, _vp, _vp,
                                       _i32, _st, _vp, _vp]),
    "lci_sparse_attn_pipelined": (_st, [_vp, _i32, _i32, _i32, _vp, _vp, _vp, _vp, _i32, _vp, _vp,
                                        _f32, _vp, _vp, _vp]),
    "lci_set_wait_limit_ns": (_st, [ctypes.c_uint64]),
    "lci_sparse_decode_persistent": (_st, [_vp, _vp, _st, _i32, _i32, _i32, _i32, _i32, _vp, _vp,
                                           _i32, _vp, _i32, _vp, _vp, _vp, _f32, _vp, _vp, _vp,
                                           _sz, _vp]),
    "lci_gated_state_scan": (_st, [_vp, _vp, _vp, _st, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _i32,
                                   _i32, _vp, _vp]),
    "lci_block_scores_at": (_st, [_vp, _vp, _st, _i32, _i32, _i32, _i32, _i32, _vp, _i32, _vp,
                                  _vp]),
    "lci_ids_shift": (_st, [_vp, ctypes.c_int64, _i32, _i32, _i32, _vp, _vp]),
    "lci_topk_merge": (_st, [_vp, _vp, _i32, ctypes.c_int64, _i32, _vp, _vp]),
    "lci_sparse_attn_partial": (_st, [_vp, _i32, _i32, _i32, _vp, _vp, _vp, _vp, _i32, _vp, _vp,
                                      _f32, _st, _vp, _vp, _vp]),
    "lci_attn_merge": (_st, [_vp, _vp, _st, _i32, ctypes.c_int64, _i32, _vp, _vp]),
    "lci_kc_update": (_st, [_vp, _st, _i32, _i32, _i32, _i32, _vp, _vp, _vp, _vp, _vp]),
    "lci_index_select_paged_workspace_size": (_st, [_i32, _i32, _i32, _i32, _i32, _vp, _st, _st,
                                                    ctypes.POINTER(_sz)]),
    "lci_index_select_paged": (_st, [_vp, _vp, _st, _i32, _i32, _i32, _i32, _vp, _vp, _vp, _i32,
                                     _st, _vp, _vp, _sz, _vp]),
    "lci_kv_append_q8": (_st, [_vp, _vp, _st, _i32, _i32, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp]),
    "lci_sparse_attn_q8": (_st, [_vp, _st, _i32, _i32, _i32, _vp, _vp, _vp, _vp, _vp, _vp, _i32,
                                 _vp, _vp, _f32, _vp, _st, _vp, _vp, _vp, _vp]),
    "lci_block_weight_update": (_st, [_vp, _vp, _i32, _i32, _i32, _i32, _i32, _f32, _vp, _vp]),
    "lci_cache_evict": (_st, [_vp, _i32, _vp, _vp, _i32, _i32, _i32, _vp, _vp, _vp, _vp, _vp, _vp]),
    "lci_call_prepared": (_st, [_st, _vp, _vp]),
    "lci_get_wait_limit_ns": (_st, [ctypes.POINTER(ctypes.c_uint64)]),
}

_lib = None
_lock = threading.Lock()


class LciError(RuntimeError):
    def __init__(self, status: int, where: str, message: str):
        self.status = status
        super().__init__(f"{where}: {STATUS_NAMES.get(status, status)}: {message}")


def load_library() -> ctypes.CDLL:
    """Load liblci.so (built by long_context_indexer_b200.build); raise if absent."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(f"liblci.so not found at {LIB_PATH}; build it with "
                                   "`python -m long_context_indexer_b200.build`")
            lib = ctypes.CDLL(LIB_PATH)
            for name, (res, args) in SIGNATURES.items():
                fn = getattr(lib, name)
                fn.restype = res
                fn.argtypes = args
            _lib = lib
    return _lib


def _check(status: int, where: str) -> None:
    if status != LCI_OK:
        msg = load_library().lci_last_error().decode(errors="replace")
        raise LciError(status, where, msg)


def version() -> str:
    return load_library().lci_version().decode()


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return LCI_F32
    if t.dtype == torch.bfloat16:
        return LCI_BF16
    raise TypeError(f"lci: unsupported dtype {t.dtype} (float32 or bfloat16)")


def _dev(t: torch.Tensor, name: str, dtype: Optional[torch.dtype] = None, ndim: Optional[int] = None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"lci: {name} must be a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError(f"lci: {name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"lci: {name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"lci: {name} must be {dtype}, got {t.dtype}")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"lci: {name} must have {ndim} dims, got {t.dim()}")
    return ctypes.c_void_p(t.data_ptr())


# ---------------------------------------------------------------- workspaces

_ws: Dict[Tuple[int, str], torch.Tensor] = {}


def workspace(device: torch.device, nbytes: int, tag: str) -> torch.Tensor:
    """A zero-initialised, 256-byte aligned device buffer of at least nbytes.

    Workspaces hold arrival counters that the library leaves at zero after
    every call, but only in the layout of the shape they were used with. So a
    cached buffer is keyed by ``tag``, which callers make unique per layout
    (entry point and the sizes the layout depends on), and is zero-filled once
    when first allocated.
    """
    key = (torch.device(device).index or 0, tag)
    buf = _ws.get(key)
    if buf is None or buf.numel() < nbytes:
        buf = torch.zeros(max(nbytes, 256), dtype=torch.uint8, device=device)
        _ws[key] = buf
    return buf


# ---------------------------------------------------------------- block table

def _closed_table(*args):
    raise ValueError("lci: the block table of this prepared call was closed")


class BlockTable:
    """Owns an lci_block_table handle; keeps the table tensor alive."""

    def __init__(self, table: torch.Tensor, num_pages: int, block_size: int, num_kv_heads: int,
                 head_dim: int, dtype: torch.dtype):
        ptr = _dev(table, "block_table", torch.int32, 2)
        self.table = table
        self.batch, self.max_blocks = table.shape
        self.num_pages, self.block_size = int(num_pages), int(block_size)
        self.num_kv_heads, self.head_dim = int(num_kv_heads), int(head_dim)
        self.dtype = dtype
        handle = ctypes.c_void_p()
        lib = load_library()
        code = LCI_E4M3 if dtype == torch.float8_e4m3fn else _dtype_code(torch.empty(0, dtype=dtype))
        _check(lib.lci_create_block_table(ptr, self.batch, self.max_blocks, self.num_pages,
                                          self.block_size, self.num_kv_heads, self.head_dim, code,
                                          ctypes.byref(handle)), "lci_create_block_table")
        self._handle = handle
        self._lib = lib

    @property
    def handle(self) -> ctypes.c_void_p:
        return self._handle

    def validate(self, stream=None) -> None:
        _check(self._lib.lci_validate_block_table(self._handle, _stream(stream)),
               "lci_validate_block_table")

    _prepared = None  # the calls that hold the handle

    def register(self, call) -> None:
        """``call`` holds the handle in its prepared arguments: close() makes it refuse."""
        if self._prepared is None:
            self._prepared = weakref.WeakSet()
        self._prepared.add(call)

    def close(self) -> None:
        for call in self._prepared or ():
            call._fn = _closed_table
        if getattr(self, "_handle", None):
            self._lib.lci_destroy_block_table(self._handle)
            self._handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def create_block_table(table: torch.Tensor, k_pool: torch.Tensor) -> BlockTable:
    """Block table over pools shaped [num_pages, H_kv, block_size, head_dim]."""
    P, H_kv, bs, hd = k_pool.shape
    return BlockTable(table, P, bs, H_kv, hd, k_pool.dtype)


# ---------------------------------------------------------------- entry points

def block_compress(k_idx: torch.Tensor, block_size: int, out: Optional[torch.Tensor] = None,
                   stream=None) -> torch.Tensor:
    """A0: [B, T, H, D] per-token indexer keys -> [B, ceil(T/bs), H, D] block means."""
    B, T, H, D = k_idx.shape
    NB = (T + block_size - 1) // block_size
    if out is None:
        out = torch.empty((B, NB, H, D), dtype=k_idx.dtype, device=k_idx.device)
    _check(load_library().lci_block_compress(_dev(k_idx, "k_idx", None, 4), _dtype_code(k_idx), B, T,
                                             H, D, block_size, _dev(out, "out", k_idx.dtype, 4),
                                             _stream(stream)), "lci_block_compress")
    return out


def index_select_workspace_size(B, S, H_i, d_c, nb_max, topk, phase="auto") -> int:
    n = ctypes.c_size_t()
    _check(load_library().lci_index_select_workspace_size(B, S, H_i, d_c, nb_max, topk,
                                                          PHASES[phase], ctypes.byref(n)),
           "lci_index_select_workspace_size")
    return n.value


def index_select(q_c: torch.Tensor, k_c: torch.Tensor, block_size: int, ctx_len: torch.Tensor,
                 q_start: torch.Tensor, topk: int, phase: str = "auto",
                 ids: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None,
                 stream=None) -> torch.Tensor:
    """A1+A2: ids [B, S, topk] int32, ranked (score desc, id asc), -1 padded."""
    B, S, H_i, d_c = q_c.shape
    nb_max = k_c.shape[1]
    if k_c.shape[0] != B or k_c.shape[2:] != q_c.shape[2:] or k_c.dtype != q_c.dtype:
        raise ValueError("lci: k_c must be [B, nb_max, H_i, d_c] with q_c's dtype")
    if ids is None:
        ids = torch.empty((B, S, topk), dtype=torch.int32, device=q_c.device)
    need = index_select_workspace_size(B, S, H_i, d_c, nb_max, topk, phase)
    if ws is None:
        ws = workspace(q_c.device, need, f"index_select:{B}x{S}x{nb_max}:{H_i * d_c}")
    _check(load_library().lci_index_select(
        _dev(q_c, "q_c", None, 4), _dev(k_c, "k_c", q_c.dtype, 4), _dtype_code(q_c), B, S, H_i, d_c,
        block_size, nb_max, _dev(ctx_len, "ctx_len", torch.int32, 1),
        _dev(q_start, "q_start", torch.int32, 1), topk, PHASES[phase],
        _dev(ids, "ids", torch.int32, 3), _dev(ws, "workspace"), ws.numel() * ws.element_size(),
        _stream(stream)), "lci_index_select")
    return ids


def index_select_noalloc(q_c: torch.Tensor, k_c: torch.Tensor, block_size: int,
                         ctx_len: torch.Tensor, q_start: torch.Tensor, topk: int,
                         phase: str = "auto", ids: Optional[torch.Tensor] = None,
                         stream=None) -> torch.Tensor:
    """index_select through lci_index_select_noalloc: no workspace, no device
    allocation inside the library (its scratch is a fixed array in liblci.so)."""
    B, S, H_i, d_c = q_c.shape
    nb_max = k_c.shape[1]
    if k_c.shape[0] != B or k_c.shape[2:] != q_c.shape[2:] or k_c.dtype != q_c.dtype:
        raise ValueError("lci: k_c must be [B, nb_max, H_i, d_c] with q_c's dtype")
    if ids is None:
        ids = torch.empty((B, S, topk), dtype=torch.int32, device=q_c.device)
    _check(load_library().lci_index_select_noalloc(
        _dev(q_c, "q_c", None, 4), _dev(k_c, "k_c", q_c.dtype, 4), _dtype_code(q_c), B, S, H_i, d_c,
        block_size, nb_max, _dev(ctx_len, "ctx_len", torch.int32, 1),
        _dev(q_start, "q_start", torch.int32, 1), topk, PHASES[phase],
        _dev(ids, "ids", torch.int32, 3), _stream(stream)), "lci_index_select_noalloc")
    return ids


def sparse_attn_workspace_size(B, S, H_q, topk, table: BlockTable, phase="auto") -> int:
    n = ctypes.c_size_t()
    _check(load_library().lci_sparse_attn_workspace_size(B, S, H_q, topk, table.handle,
                                                         PHASES[phase], ctypes.byref(n)),
           "lci_sparse_attn_workspace_size")
    return n.value


def sparse_attn(q: torch.Tensor, k_pool: torch.Tensor, v_pool: torch.Tensor, table: BlockTable,
                ids: torch.Tensor, ctx_len: torch.Tensor, q_start: torch.Tensor,
                scale: float = 0.0, phase: str = "auto", out: Optional[torch.Tensor] = None,
                ws: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """A3+A4: exact softmax attention over the selected blocks. out [B, S, H_q, hd]."""
    B, S, H_q, hd = q.shape
    topk = ids.shape[-1]
    if tuple(ids.shape) != (B, S, topk):
        raise ValueError("lci: ids must be [B, S, topk]")
    if tuple(k_pool.shape) != (table.num_pages, table.num_kv_heads, table.block_size,
                               table.head_dim) or v_pool.shape != k_pool.shape:
        raise ValueError("lci: pools do not match the block table")
    if q.dtype != table.dtype or k_pool.dtype != q.dtype or v_pool.dtype != q.dtype:
        raise TypeError("lci: q and the pools must share the block table's dtype")
    if hd != table.head_dim:
        raise ValueError("lci: q's head_dim differs from the block table's")
    if out is None:
        out = torch.empty_like(q)
    need = sparse_attn_workspace_size(B, S, H_q, topk, table, phase)
    if ws is None:
        ws = workspace(q.device, need, f"sparse_attn:{B}x{S}x{H_q}x{topk}:{table.max_blocks}:"
                                       f"{table.num_kv_heads}x{table.block_size}")
    _check(load_library().lci_sparse_attn(
        _dev(q, "q", None, 4), B, S, H_q, _dev(k_pool, "k_pool"), _dev(v_pool, "v_pool"),
        table.handle, _dev(ids, "ids", torch.int32, 3), topk, _dev(ctx_len, "ctx_len", torch.int32, 1),
        _dev(q_start, "q_start", torch.int32, 1), float(scale), PHASES[phase],
        _dev(out, "out", q.dtype, 4), _dev(ws, "workspace"), ws.numel() * ws.element_size(),
        _stream(stream)), "lci_sparse_attn")
    return out


_decode_ws_sizes: Dict[Tuple[int, ...], int] = {}


def sparse_decode_workspace_size(B, S, H_i, d_c, topk, H_q, table: BlockTable) -> int:
    key = (B, S, H_i, d_c, topk, H_q, table.max_blocks, table.num_kv_heads, table.block_size,
           table.head_dim, str(table.dtype))
    n = _decode_ws_sizes.get(key)
    if n is None:
        c = ctypes.c_size_t()
        _check(load_library().lci_sparse_decode_workspace_size(B, S, H_i, d_c, topk, H_q,
                                                               table.handle, ctypes.byref(c)),
               "lci_sparse_decode_workspace_size")
        n = _decode_ws_sizes[key] = c.value
    return n


def sparse_decode(q_c: torch.Tensor, k_c: torch.Tensor, ctx_len: torch.Tensor,
                  q_start: torch.Tensor, topk: int, q: torch.Tensor, k_pool: torch.Tensor,
                  v_pool: torch.Tensor, table: BlockTable, scale: float = 0.0,
                  ids: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                  ws: Optional[torch.Tensor] = None, stream=None, persistent: bool = False):
    """index_select + sparse_attn in one call (rows attended as they are selected).

    Returns (ids [B, S, topk] int32, out [B, S, H_q, hd])."""
    B, S, H_i, d_c = q_c.shape
    nb_max = k_c.shape[1]
    H_q = q.shape[2]
    if tuple(q.shape[:2]) != (B, S):
        raise ValueError("lci: q must be [B, S, H_q, hd] with q_c's B and S")
    if tuple(k_pool.shape) != (table.num_pages, table.num_kv_heads, table.block_size,
                               table.head_dim) or v_pool.shape != k_pool.shape:
        raise ValueError("lci: pools do not match the block table")
    if ids is None:
        ids = torch.empty((B, S, topk), dtype=torch.int32, device=q_c.device)
    if out is None:
        out = torch.empty_like(q)
    need = sparse_decode_workspace_size(B, S, H_i, d_c, topk, H_q, table)
    if ws is None:
        ws = workspace(q_c.device, need, f"sparse_decode:{B}x{S}x{nb_max}:{H_i * d_c}:{topk}:"
                                         f"{H_q}x{table.num_kv_heads}x{table.block_size}")
    name = "lci_sparse_decode_persistent" if persistent else "lci_sparse_decode"
    _check(getattr(load_library(), name)(
        _dev(q_c, "q_c", None, 4), _dev(k_c, "k_c", q_c.dtype, 4), _dtype_code(q_c), B, S, H_i,
        d_c, nb_max, _dev(ctx_len, "ctx_len", torch.int32, 1),
        _dev(q_start, "q_start", torch.int32, 1), topk, _dev(q, "q", q_c.dtype, 4), H_q,
        _dev(k_pool, "k_pool", q_c.dtype), _dev(v_pool, "v_pool", q_c.dtype), table.handle,
        float(scale), _dev(ids, "ids", torch.int32, 3), _dev(out, "out", q_c.dtype, 4),
        _dev(ws, "workspace"), ws.numel() * ws.element_size(), _stream(stream)), name)
    return ids, out


class PagedKeys:
    """Block keys stored per page of a paged KV cache (one key per page), with
    the fp32 running sums the online producer extends."""

    def __init__(self, num_pages: int, H_i: int, d_c: int, dtype: torch.dtype, device):
        self.kc = torch.zeros((num_pages, H_i, d_c), dtype=dtype, device=device)
        self.kc_sum = torch.zeros((num_pages, H_i * d_c), dtype=torch.float32, device=device)

    def update(self, k_idx: torch.Tensor, start: torch.Tensor, table: BlockTable,
               stream=None) -> None:
        """Append k_idx [B, T, H_i, d_c] at positions start[b] .. start[b]+T-1."""
        B, T, H_i, d_c = k_idx.shape
        if k_idx.dtype != self.kc.dtype or tuple(self.kc.shape[1:]) != (H_i, d_c):
            raise ValueError("lci: k_idx must match the paged keys' dtype and [H_i, d_c]")
        if self.kc.shape[0] != table.num_pages:
            raise ValueError("lci: paged keys and block table differ in page count")
        _check(load_library().lci_kc_update(
            _dev(k_idx, "k_idx", None, 4), _dtype_code(k_idx), B, T, H_i, d_c,
            _dev(start, "start", torch.int32, 1), table.handle, _dev(self.kc_sum, "kc_sum"),
            _dev(self.kc, "kc"), _stream(stream)), "lci_kc_update")


def index_select_paged(q_c: torch.Tensor, keys: "PagedKeys", table: BlockTable,
                       ctx_len: torch.Tensor, q_start: torch.Tensor, topk: int,
                       phase: str = "auto", ids: Optional[torch.Tensor] = None,
                       ws: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """index_select with block keys read from the paged pool through the table."""
    B, S, H_i, d_c = q_c.shape
    kc = keys.kc if isinstance(keys, PagedKeys) else keys
    if kc.dtype != q_c.dtype or tuple(kc.shape[1:]) != (H_i, d_c):
        raise ValueError("lci: paged keys must be [num_pages, H_i, d_c] with q_c's dtype")
    if ids is None:
        ids = torch.empty((B, S, topk), dtype=torch.int32, device=q_c.device)
    lib = load_library()
    n = ctypes.c_size_t()
    _check(lib.lci_index_select_paged_workspace_size(B, S, H_i, d_c, topk, table.handle,
                                                     _dtype_code(q_c), PHASES[phase],
                                                     ctypes.byref(n)),
           "lci_index_select_paged_workspace_size")
    if ws is None:
        ws = workspace(q_c.device, n.value,
                       f"index_select_paged:{B}x{S}x{table.max_blocks}:{H_i * d_c}:{phase}")
    _check(lib.lci_index_select_paged(
        _dev(q_c, "q_c", None, 4), _dev(kc, "kc", q_c.dtype, 3), _dtype_code(q_c), B, S, H_i, d_c,
        table.handle, _dev(ctx_len, "ctx_len", torch.int32, 1),
        _dev(q_start, "q_start", torch.int32, 1), topk, PHASES[phase],
        _dev(ids, "ids", torch.int32, 3), _dev(ws, "workspace"), ws.numel() * ws.element_size(),
        _stream(stream)), "lci_index_select_paged")
    return ids


def block_scores_at(q_c: torch.Tensor, k_c: torch.Tensor, ids: torch.Tensor,
                    out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """scores [B, S, topk] fp32 of the given block ids (-inf for -1)."""
    B, S, H_i, d_c = q_c.shape
    topk = ids.shape[-1]
    if tuple(ids.shape) != (B, S, topk):
        raise ValueError("lci: ids must be [B, S, topk]")
    if out is None:
        out = torch.empty((B, S, topk), dtype=torch.float32, device=q_c.device)
    _check(load_library().lci_block_scores_at(
        _dev(q_c, "q_c", None, 4), _dev(k_c, "k_c", q_c.dtype, 4), _dtype_code(q_c), B, S, H_i, d_c,
        k_c.shape[1], _dev(ids, "ids", torch.int32, 3), topk, _dev(out, "scores", torch.float32, 3),
        _stream(stream)), "lci_block_scores_at")
    return out


def ids_shift(ids: torch.Tensor, lo: int, hi: int, offset: int,
              out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """(lo <= id < hi) ? id + offset : -1, elementwise."""
    if out is None:
        out = torch.empty_like(ids)
    _check(load_library().lci_ids_shift(_dev(ids, "ids", torch.int32), ids.numel(), int(lo),
                                        int(hi), int(offset), _dev(out, "out", torch.int32),
                                        _stream(stream)), "lci_ids_shift")
    return out


def topk_merge(scores: torch.Tensor, ids: torch.Tensor, out: Optional[torch.Tensor] = None,
               stream=None) -> torch.Tensor:
    """Merge [L, ..., topk] ranked lists into the top-k [..., topk] of their union."""
    L, topk = ids.shape[0], ids.shape[-1]
    if scores.shape != ids.shape:
        raise ValueError("lci: scores and ids must have the same shape")
    rows = ids[0].numel() // topk
    if out is None:
        out = torch.empty(ids.shape[1:], dtype=torch.int32, device=ids.device)
    _check(load_library().lci_topk_merge(_dev(scores, "scores", torch.float32),
                                         _dev(ids, "ids", torch.int32), L, rows, topk,
                                         _dev(out, "out", torch.int32), _stream(stream)),
           "lci_topk_merge")
    return out


def sparse_attn_partial(q: torch.Tensor, k_pool: torch.Tensor, v_pool: torch.Tensor,
                        table: BlockTable, ids: torch.Tensor, ctx_len: torch.Tensor,
                        q_start: torch.Tensor, scale: float = 0.0, phase: str = "auto",
                        out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                        stream=None):
    """sparse_attn plus the base-2 log-sum-exp [B, S, H_q] of each row's logits."""
    B, S, H_q, hd = q.shape
    topk = ids.shape[-1]
    if tuple(ids.shape) != (B, S, topk):
        raise ValueError("lci: ids must be [B, S, topk]")
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((B, S, H_q), dtype=torch.float32, device=q.device)
    _check(load_library().lci_sparse_attn_partial(
        _dev(q, "q", table.dtype, 4), B, S, H_q, _dev(k_pool, "k_pool", table.dtype),
        _dev(v_pool, "v_pool", table.dtype), table.handle, _dev(ids, "ids", torch.int32, 3), topk,
        _dev(ctx_len, "ctx_len", torch.int32, 1), _dev(q_start, "q_start", torch.int32, 1),
        float(scale), PHASES[phase], _dev(out, "out", q.dtype, 4),
        _dev(lse, "lse", torch.float32, 3), _stream(stream)), "lci_sparse_attn_partial")
    return out, lse


def attn_merge(o: torch.Tensor, lse: torch.Tensor, out: Optional[torch.Tensor] = None,
               stream=None) -> torch.Tensor:
    """Combine partials o [L, ..., hd] with lse [L, ...] into out [..., hd]."""
    L, hd = o.shape[0], o.shape[-1]
    if tuple(lse.shape) != tuple(o.shape[:-1]):
        raise ValueError("lci: lse must be o's shape without the last dim")
    if out is None:
        out = torch.empty(o.shape[1:], dtype=o.dtype, device=o.device)
    _check(load_library().lci_attn_merge(_dev(o, "o", None), _dev(lse, "lse", torch.float32),
                                         _dtype_code(o), L, lse[0].numel(), hd,
                                         _dev(out, "out", o.dtype), _stream(stream)),
           "lci_attn_merge")
    return out


def gated_state_scan(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, gate: torch.Tensor,
                     state: torch.Tensor, chunk: int = 128, out: Optional[torch.Tensor] = None,
                     state_out: Optional[torch.Tensor] = None, stream=None):
    """N4: chunked gated state scan. q, k [B, T, H, dk], v [B, T, H, dv] (bf16),
    gate [B, H, ceil(T/chunk)] and state [B, H, dk, dv] (fp32). Returns
    (out [B, T, H, dv] fp32, final state); state_out=state updates in place."""
    B, T, H, dk = q.shape
    dv = v.shape[3]
    if tuple(k.shape) != (B, T, H, dk) or tuple(v.shape[:3]) != (B, T, H):
        raise ValueError("lci: q, k, v shapes disagree")
    if tuple(gate.shape) != (B, H, -(-T // chunk)) or tuple(state.shape) != (B, H, dk, dv):
        raise ValueError("lci: gate must be [B, H, nchunks] and state [B, H, dk, dv]")
    if out is None:
        out = torch.empty((B, T, H, dv), dtype=torch.float32, device=q.device)
    if state_out is None:
        state_out = torch.empty_like(state)
    _check(load_library().lci_gated_state_scan(
        _dev(q, "q", None, 4), _dev(k, "k", q.dtype, 4), _dev(v, "v", q.dtype, 4), _dtype_code(q),
        _dev(gate, "gate", torch.float32, 3), _dev(state, "state", torch.float32, 4),
        _dev(state_out, "state_out", torch.float32, 4), B, T, H, dk, dv, chunk,
        _dev(out, "out", torch.float32, 4), _stream(stream)), "lci_gated_state_scan")
    return out, state_out


# ---------------------------------------------------------------- 8-bit paged cache

class _ScoreOptions(ctypes.Structure):
    _fields_ = [("cap", _f32), ("d_slopes", _vp), ("d_first", _vp), ("d_last", _vp)]


# The handle of a device's current stream, and the current device, without
# building an object.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                      lambda device: torch.cuda.current_stream(device).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)

# Entry points that lci_call_prepared makes, by its lci_call.
_PREPARED = {"lci_kv_append_q8": 0, "lci_sparse_attn_q8": 1, "lci_block_weight_update": 2,
             "lci_cache_evict": 3}


class _Arg(ctypes.Union):
    _fields_ = [("ptr", _vp), ("i32", _i32), ("f32", _f32)]


def _pack_args(name: str, args: tuple):
    """The arguments of an entry point, without its stream, as lci_call_prepared takes them."""
    types = SIGNATURES[name][1][:-1]
    if len(types) != len(args):
        raise TypeError(f"lci: {name} takes {len(types)} arguments and a stream")
    packed = (_Arg * len(args))()
    for slot, kind, value in zip(packed, types, args):
        if kind is _vp:
            slot.ptr = value.value if isinstance(value, _vp) else value
        elif kind is _f32:
            slot.f32 = value
        else:
            if not -2 ** 31 <= value < 2 ** 31:
                raise ValueError(f"lci: {name}: {value} does not fit 32 bits")
            slot.i32 = value
    return packed


class PreparedCall:
    """A checked call of one entry point, for a loop that makes it every step:
    the tensors were checked and their pointers taken when it was prepared, and
    each call launches it on the current stream of the tensors' device, or on
    ``stream``. It works on the same tensors every time; ``result`` holds the
    outputs. Returns ``result``."""

    def __init__(self, name: str, args: tuple, result, device: torch.device, keep: tuple):
        self.result = result
        self._name, self._keep = name, keep
        self._packed = _pack_args(name, args)
        self._call = _PREPARED[name]
        self._args = ctypes.addressof(self._packed)
        self._fn = load_library().lci_call_prepared
        self._device = device.index
        for t in keep:
            if isinstance(t, BlockTable):
                t.register(self)

    def __call__(self, stream=None):
        raw = _raw_stream(self._device) if stream is None else stream.cuda_stream
        if _current_device() == self._device:
            rc = self._fn(self._call, self._args, raw)
        else:
            with torch.cuda.device(self._device):
                rc = self._fn(self._call, self._args, raw)
        if rc != LCI_OK:
            _check(rc, self._name)
        return self.result


def _opt(t: Optional[torch.Tensor], name: str, dtype: torch.dtype, shape: tuple):
    """Pointer of an optional tensor of a given type and shape (NULL if absent)."""
    return None if t is None else _shaped(t, name, dtype, shape)


def _shaped(t: torch.Tensor, name: str, dtype: torch.dtype, shape: tuple):
    p = _dev(t, name, dtype)
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"lci: {name} must be {list(shape)}, got {list(t.shape)}")
    return p


def _one_device(*tensors) -> torch.device:
    devices = {t.device for t in tensors if t is not None}
    if len(devices) != 1:
        raise ValueError(f"lci: tensors are on different devices: {sorted(map(str, devices))}")
    return devices.pop()


class Q8Cache:
    """A paged KV cache held in 8 bits: e4m3 pools ``k``, ``v`` [num_pages, H_kv,
    block_size, head_dim] and a scale per page and KV head, ``k_scale``,
    ``v_scale`` [num_pages, H_kv] fp32. An element stands for scale * value."""

    def __init__(self, num_pages: int, num_kv_heads: int, block_size: int, head_dim: int, device):
        shape = (num_pages, num_kv_heads, block_size, head_dim)
        self.k = torch.zeros(shape, dtype=torch.float8_e4m3fn, device=device)
        self.v = torch.zeros(shape, dtype=torch.float8_e4m3fn, device=device)
        self.k_scale = torch.ones(shape[:2], dtype=torch.float32, device=device)
        self.v_scale = torch.ones(shape[:2], dtype=torch.float32, device=device)

    @classmethod
    def wrap(cls, k: torch.Tensor, v: torch.Tensor, k_scale: torch.Tensor,
             v_scale: torch.Tensor) -> "Q8Cache":
        """A cache over existing tensors."""
        c = cls.__new__(cls)
        c.k, c.v, c.k_scale, c.v_scale = k, v, k_scale, v_scale
        return c

    def _pointers(self, table: "BlockTable"):
        shape = (table.num_pages, table.num_kv_heads, table.block_size, table.head_dim)
        if table.dtype != torch.float8_e4m3fn:
            raise TypeError("lci: the block table is not over e4m3 pools")
        return (_shaped(self.k, "k pool", torch.float8_e4m3fn, shape),
                _shaped(self.v, "v pool", torch.float8_e4m3fn, shape),
                _shaped(self.k_scale, "k_scale", torch.float32, shape[:2]),
                _shaped(self.v_scale, "v_scale", torch.float32, shape[:2]))

    def append(self, k_new: torch.Tensor, v_new: torch.Tensor, start: torch.Tensor,
               table: "BlockTable", count: Optional[torch.Tensor] = None, stream=None) -> None:
        """Append k_new, v_new [B, T, H_kv, hd] at positions start[b] ..; see kv_append_q8."""
        kv_append_q8(self, table, k_new, v_new, start, count=count, stream=stream)


def prepare_kv_append_q8(cache: Q8Cache, table: BlockTable, k_new: torch.Tensor,
                         v_new: torch.Tensor, start: torch.Tensor,
                         count: Optional[torch.Tensor] = None) -> PreparedCall:
    """kv_append_q8 as a PreparedCall."""
    B, T = k_new.shape[:2]
    shape = (B, T, table.num_kv_heads, table.head_dim)
    kp, vp, ks, vs = cache._pointers(table)
    dev = _one_device(table.table, cache.k, cache.v, cache.k_scale, cache.v_scale, k_new, v_new,
                      start, count)
    args = (_shaped(k_new, "k_new", k_new.dtype, shape), _shaped(v_new, "v_new", k_new.dtype, shape),
            _dtype_code(k_new), B, T, _shaped(start, "start", torch.int32, (B,)),
            _opt(count, "count", torch.int32, (B,)), table.handle, kp, vp, ks, vs)
    return PreparedCall("lci_kv_append_q8", args, (cache.k, cache.v, cache.k_scale, cache.v_scale),
                        dev, (cache, table, k_new, v_new, start, count))


def kv_append_q8(cache: Q8Cache, table: BlockTable, k_new: torch.Tensor, v_new: torch.Tensor,
                 start: torch.Tensor, count: Optional[torch.Tensor] = None, stream=None):
    """New tokens' K and V [B, T, H_kv, hd] (bf16 or fp32) enter the cache at
    positions start[b] .. (count[b] of them, T where count is None). A page's
    scale grows when a new token needs it; stored codes are then rounded to it.
    Returns (k, v, k_scale, v_scale), the cache's own tensors."""
    return prepare_kv_append_q8(cache, table, k_new, v_new, start, count)(stream)


def prepare_sparse_attn_q8(q: torch.Tensor, cache: Q8Cache, table: BlockTable, ids: torch.Tensor,
                           ctx_len: torch.Tensor, q_start: torch.Tensor, scale: float = 0.0,
                           cap: float = 0.0, slopes: Optional[torch.Tensor] = None,
                           first: Optional[torch.Tensor] = None,
                           last: Optional[torch.Tensor] = None, phase: str = "auto",
                           out: Optional[torch.Tensor] = None, lse=False,
                           mass=False) -> PreparedCall:
    """sparse_attn_q8 as a PreparedCall."""
    if q.dim() != 4 or ids.dim() != 3:
        raise ValueError("lci: q must be [B, S, H_q, hd] and ids [B, S, topk]")
    B, S, H_q, hd = q.shape
    topk = ids.shape[-1]
    if hd != table.head_dim:
        raise ValueError("lci: q's head_dim differs from the block table's")
    kp, vp, ks, vs = cache._pointers(table)
    if out is None:
        out = torch.empty_like(q)
    if lse is True:
        lse = torch.empty((B, S, H_q), dtype=torch.float32, device=q.device)
    if mass is True:
        mass = torch.empty((B, S, table.num_kv_heads, topk), dtype=torch.float32, device=q.device)
    lse = None if lse is False else lse
    mass = None if mass is False else mass
    dev = _one_device(q, table.table, cache.k, cache.v, cache.k_scale, cache.v_scale, ids, ctx_len,
                      q_start, slopes, first, last, out, lse, mass)
    options = _ScoreOptions(float(cap), _opt(slopes, "slopes", torch.float32, (H_q,)),
                            _opt(first, "first", torch.int32, (B, S)),
                            _opt(last, "last", torch.int32, (B, S)))
    args = (_dev(q, "q", None, 4), _dtype_code(q), B, S, H_q, kp, vp, ks, vs, table.handle,
            _shaped(ids, "ids", torch.int32, (B, S, topk)), topk,
            _shaped(ctx_len, "ctx_len", torch.int32, (B,)),
            _shaped(q_start, "q_start", torch.int32, (B,)), float(scale), ctypes.addressof(options),
            PHASES[phase], _shaped(out, "out", q.dtype, tuple(q.shape)),
            _opt(lse, "lse", torch.float32, (B, S, H_q)),
            _opt(mass, "mass", torch.float32, (B, S, table.num_kv_heads, topk)))
    result = out if lse is None and mass is None else tuple(
        t for t in (out, lse, mass) if t is not None)
    return PreparedCall("lci_sparse_attn_q8", args, result, dev,
                        (q, cache, table, ids, ctx_len, q_start, slopes, first, last, options, out,
                         lse, mass))


def sparse_attn_q8(q: torch.Tensor, cache: Q8Cache, table: BlockTable, ids: torch.Tensor,
                   ctx_len: torch.Tensor, q_start: torch.Tensor, scale: float = 0.0,
                   cap: float = 0.0, slopes: Optional[torch.Tensor] = None,
                   first: Optional[torch.Tensor] = None, last: Optional[torch.Tensor] = None,
                   phase: str = "auto", out: Optional[torch.Tensor] = None, lse=False, mass=False,
                   stream=None):
    """A3+A4 over the 8-bit cache: attention of q [B, S, H_q, hd] (bf16 or fp32)
    over the selected blocks ids [B, S, topk].

    cap > 0 (2^-100 .. 2^100) caps the scaled scores z at cap * tanh(z / cap); slopes [H_q] fp32
    subtracts slopes[h] * |p - t|; first / last [B, S] int32 bound the tokens a
    query attends (document mask: first = its document's start; prefix mask:
    last = max(p, prefix - 1)). lse and mass are True or output tensors: the
    base-2 log-sum-exp [B, S, H_q], and the softmax weight each selected block
    received [B, S, H_kv, topk], summed over the KV head's query heads. phase
    "prefill" or "decode" picks the schedule where the sizes alone do not tell: a
    prompt much shorter than the table, a late chunk whose queries share few blocks.
    Returns out, or (out[, lse][, mass]) with those asked for."""
    return prepare_sparse_attn_q8(q, cache, table, ids, ctx_len, q_start, scale, cap, slopes, first,
                                  last, phase, out, lse, mass)(stream)


def prepare_block_weight_update(weight: torch.Tensor, ids: torch.Tensor, mass: torch.Tensor,
                                decay: float = 1.0) -> PreparedCall:
    """block_weight_update as a PreparedCall."""
    if weight.dim() != 2 or ids.dim() != 3 or mass.dim() != 4:
        raise ValueError("lci: weight must be [B, NB], ids [B, S, topk], mass [B, S, H_kv, topk]")
    B, NB = weight.shape
    S, H_kv, topk = mass.shape[1:]
    dev = _one_device(weight, ids, mass)
    args = (_shaped(ids, "ids", torch.int32, (B, S, topk)),
            _shaped(mass, "mass", torch.float32, (B, S, H_kv, topk)), B, S, H_kv, topk, NB,
            float(decay), _dev(weight, "weight", torch.float32, 2))
    return PreparedCall("lci_block_weight_update", args, (weight,), dev, (weight, ids, mass))


def block_weight_update(weight: torch.Tensor, ids: torch.Tensor, mass: torch.Tensor,
                        decay: float = 1.0, stream=None) -> torch.Tensor:
    """weight[b, j] = decay * weight[b, j] + the mass that block j received
    (ids [B, S, topk], mass [B, S, H_kv, topk] of sparse_attn_q8), in place.
    Returns weight [B, NB] fp32."""
    return prepare_block_weight_update(weight, ids, mass, decay)(stream)[0]


def prepare_cache_evict(table: BlockTable, ctx_len: torch.Tensor, weight: torch.Tensor, budget: int,
                        sink: int = 0, recent: int = 1, in_place: bool = False) -> PreparedCall:
    """cache_evict as a PreparedCall; its outputs are tensors of their own unless
    ``in_place`` is set, so that calling it again gives the same."""
    if weight.dim() != 2:
        raise ValueError("lci: weight must be [B, max_blocks]")
    B, NB = weight.shape
    if NB != table.max_blocks:
        raise ValueError("lci: weight must be [B, max_blocks]")
    if B > table.batch:
        raise ValueError("lci: weight has more sequences than the block table")
    dev = _one_device(table.table, ctx_len, weight)
    pt = _dev(table.table, "block_table", torch.int32, 2)
    pc = _shaped(ctx_len, "ctx_len", torch.int32, (B,))
    pw = _dev(weight, "weight", torch.float32, 2)
    if in_place:
        new = (table.table, ctx_len, weight)
    else:
        new = (torch.empty((B, NB), dtype=torch.int32, device=dev), torch.empty_like(ctx_len),
               torch.empty_like(weight))
    kept = torch.empty((B, max(int(budget), 0)), dtype=torch.int32, device=dev)
    freed = torch.empty((B,), dtype=torch.int32, device=dev)
    args = (table.handle, B, pc, pw, int(budget), int(sink), int(recent),
            *(ctypes.c_void_p(t.data_ptr()) for t in new + (kept, freed)))
    return PreparedCall("lci_cache_evict", args, new + (kept, freed), dev,
                        (table, ctx_len, weight) + new + (kept, freed))


def cache_evict(table: BlockTable, ctx_len: torch.Tensor, weight: torch.Tensor, budget: int,
                sink: int = 0, recent: int = 1, in_place: bool = True, stream=None):
    """Trim every sequence to ``budget`` blocks: the first ``sink``, the last
    ``recent`` and the heaviest of the rest stay, in order; freed pages follow
    the kept ones in the table row. Returns (table [B, NB], ctx_len [B], weight
    [B, NB], kept [B, budget] old block ids, freed [B]); in place these are the
    block table's own tensor, ctx_len and weight."""
    return prepare_cache_evict(table, ctx_len, weight, budget, sink, recent, in_place)(stream)


def sparse_attn_pipelined(q: torch.Tensor, k_pool: torch.Tensor, v_pool: torch.Tensor,
                          table: BlockTable, ids: torch.Tensor, ctx_len: torch.Tensor,
                          q_start: torch.Tensor, ready: torch.Tensor, scale: float = 0.0,
                          out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """sparse_attn whose query rows each start once ready[row] (uint32 as int32,
    [B, S]) is published nonzero by the caller's producer."""
    B, S, H_q, hd = q.shape
    topk = ids.shape[-1]
    if tuple(ids.shape) != (B, S, topk) or tuple(ready.shape) != (B, S):
        raise ValueError("lci: ids must be [B, S, topk] and ready [B, S]")
    if tuple(k_pool.shape) != (table.num_pages, table.num_kv_heads, table.block_size,
                               table.head_dim) or v_pool.shape != k_pool.shape:
        raise ValueError("lci: pools do not match the block table")
    if out is None:
        out = torch.empty_like(q)
    _check(load_library().lci_sparse_attn_pipelined(
        _dev(q, "q", table.dtype, 4), B, S, H_q, _dev(k_pool, "k_pool", table.dtype),
        _dev(v_pool, "v_pool", table.dtype), table.handle, _dev(ids, "ids", torch.int32, 3), topk,
        _dev(ctx_len, "ctx_len", torch.int32, 1), _dev(q_start, "q_start", torch.int32, 1),
        float(scale), _dev(ready, "ready", torch.int32, 2), _dev(out, "out", q.dtype, 4),
        _stream(stream)), "lci_sparse_attn_pipelined")
    return out


def set_wait_limit_ns(ns: int) -> None:
    """Limit of every bounded device wait on the current device (nanoseconds)."""
    _check(load_library().lci_set_wait_limit_ns(int(ns)), "lci_set_wait_limit_ns")


def get_wait_limit_ns() -> int:
    v = ctypes.c_uint64()
    _check(load_library().lci_get_wait_limit_ns(ctypes.byref(v)), "lci_get_wait_limit_ns")
    return v.value


class SparseDecodeStep:
    """A decode step prepared once, for a loop that calls it every step: the
    tensors are checked and their device pointers taken here, the workspace is
    allocated, and each call makes only the lci_sparse_decode C call on the
    given stream (the caller updates the buffers' contents between calls, e.g.
    by copying the new tokens' queries into q_c and q)."""

    def __init__(self, q_c: torch.Tensor, k_c: torch.Tensor, ctx_len: torch.Tensor,
                 q_start: torch.Tensor, topk: int, q: torch.Tensor, k_pool: torch.Tensor,
                 v_pool: torch.Tensor, table: BlockTable, scale: float = 0.0,
                 ids: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                 ws: Optional[torch.Tensor] = None, stream=None, persistent: bool = False):
        B, S, H_i, d_c = q_c.shape
        nb_max = k_c.shape[1]
        H_q = q.shape[2]
        if tuple(q.shape[:2]) != (B, S):
            raise ValueError("lci: q must be [B, S, H_q, hd] with q_c's B and S")
        if tuple(k_pool.shape) != (table.num_pages, table.num_kv_heads, table.block_size,
                                   table.head_dim) or v_pool.shape != k_pool.shape:
            raise ValueError("lci: pools do not match the block table")
        self.ids = torch.empty((B, S, topk), dtype=torch.int32, device=q_c.device) \
            if ids is None else ids
        self.out = torch.empty_like(q) if out is None else out
        need = sparse_decode_workspace_size(B, S, H_i, d_c, topk, H_q, table)
        self.ws = torch.zeros(max(need, 256), dtype=torch.uint8, device=q_c.device) \
            if ws is None else ws
        if self.ws.numel() * self.ws.element_size() < need:
            raise ValueError("lci: workspace too small")
        self._keep = (q_c, k_c, ctx_len, q_start, q, k_pool, v_pool, table)
        self._name = "lci_sparse_decode_persistent" if persistent else "lci_sparse_decode"
        self._fn = getattr(load_library(), self._name)
        table.register(self)
        self._stream = _stream(stream)
        self._args = (
            _dev(q_c, "q_c", None, 4), _dev(k_c, "k_c", q_c.dtype, 4), _dtype_code(q_c), B, S, H_i,
            d_c, nb_max, _dev(ctx_len, "ctx_len", torch.int32, 1),
            _dev(q_start, "q_start", torch.int32, 1), topk, _dev(q, "q", q_c.dtype, 4), H_q,
            _dev(k_pool, "k_pool", q_c.dtype), _dev(v_pool, "v_pool", q_c.dtype), table.handle,
            ctypes.c_float(scale), _dev(self.ids, "ids", torch.int32, 3),
            _dev(self.out, "out", q_c.dtype, 4), _dev(self.ws, "workspace"),
            ctypes.c_size_t(self.ws.numel() * self.ws.element_size()), self._stream)

    def __call__(self, stream=None) -> None:
        """Launch the step on its stream, or on `stream` if given (e.g. the
        stream a CUDA graph is being captured on)."""
        args = self._args if stream is None else self._args[:-1] + (_stream(stream),)
        rc = self._fn(*args)
        if rc != LCI_OK:
            _check(rc, self._name)

    def capture(self, h2d=(), d2h=()) -> "torch.cuda.CUDAGraph":
        """The step with its transfers as one CUDA graph, for a serving loop
        that replays it every step: the copies ``dst.copy_(src)`` of ``h2d``
        (device tensors filled from pinned host tensors), this step, then the
        copies of ``d2h`` (pinned host tensors filled from device tensors). The
        graph reads and writes the same buffers on every replay; the caller
        refills the host inputs and reads the host outputs between replays
        (after synchronising). Call the step once before capturing it."""
        for dst, src in list(h2d) + list(d2h):
            host = dst if dst.device.type == "cpu" else src
            if not host.is_pinned():
                raise ValueError("lci: graph transfers need pinned host tensors")
        g = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g):
            for dst, src in h2d:
                dst.copy_(src, non_blocking=True)
            self(torch.cuda.current_stream())  # the capturing stream
            for dst, src in d2h:
                dst.copy_(src, non_blocking=True)
        torch.cuda.synchronize()
        return g


def get_device_status(stream=None) -> None:
    """Synchronise the stream; raise LciError (LCI_ERR_TIMEOUT or
    LCI_ERR_DEVICE_BOUNDS) if a device wait ran out or a bounds check fired."""
    _check(load_library().lci_get_device_status(_stream(stream)), "lci_get_device_status")
