"""Python binding of libdsv4kv (C ABI in include/dsv4kv.h).

Argument marshalling only: every step of the path runs in the library's
sm_100a kernels.  PyTorch provides device memory and the current stream.
The binding raises if the shared library is missing or a call fails; there is
no CPU fallback.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
import struct
from dataclasses import dataclass
from typing import Optional

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libdsv4kv.so")

BF16, FP8_E4M3_ROW, FP4_E2M1_G16, FP8_E4M3_ROW_ROPE_BF16 = 0, 1, 2, 3
DEV_BAD_INDEX, DEV_TIMEOUT, DEV_INCONSISTENT, DEV_BAD_POOL = 0x1, 0x2, 0x4, 0x8
DEV_BAD_PAGE, DEV_BAD_LENGTH, DEV_NO_PAGES, DEV_BAD_TREE = 0x10, 0x20, 0x40, 0x80
STATUS_NAMES = {0: "OK", 1: "ERR_INVALID_ARG", 2: "ERR_UNSUPPORTED", 3: "ERR_WORKSPACE", 4: "ERR_CUDA"}


class Dsv4kvError(RuntimeError):
    def __init__(self, status: int, where: str, text: str):
        super().__init__(f"{where}: {STATUS_NAMES.get(status, status)}: {text}")
        self.status = status


class CacheDesc(ctypes.Structure):
    _fields_ = [("fmt", ctypes.c_int32), ("dim", ctypes.c_int32), ("rows", ctypes.c_int64),
                ("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p)]


class PagedDesc(ctypes.Structure):
    _fields_ = [("fmt", ctypes.c_int32), ("dim", ctypes.c_int32), ("page_rows", ctypes.c_int32),
                ("table_stride", ctypes.c_int32), ("pool_pages", ctypes.c_int64), ("table", ctypes.c_void_p),
                ("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p)]


class PageTableDesc(ctypes.Structure):
    _fields_ = [("table", ctypes.c_void_p), ("page_rows", ctypes.c_int32), ("table_stride", ctypes.c_int32),
                ("pool_pages", ctypes.c_int64)]


_lib: Optional[ctypes.CDLL] = None

_c = ctypes
_SIGS = {
    "dsv4kv_last_error": (_c.c_char_p, []),
    "dsv4kv_version": (_c.c_char_p, []),
    "dsv4kv_compress_entries": (_c.c_int64, [_c.c_int64, _c.c_int32, _c.c_int32]),
    "dsv4kv_compress": (_c.c_int, [_c.c_void_p, _c.c_void_p, _c.c_int32, _c.c_int64, _c.c_int32, _c.c_int32,
                                   _c.c_int32, _c.c_int32, _c.c_int64, _c.c_int32, _c.c_double, _c.c_int32,
                                   _c.c_void_p, _c.c_void_p]),
    "dsv4kv_quantize": (_c.c_int, [_c.c_void_p, _c.c_int32, _c.c_int64, _c.c_int32, _c.c_int32, _c.c_void_p,
                                   _c.c_void_p, _c.c_void_p]),
    "dsv4kv_index_topk_workspace_bytes": (_c.c_size_t, [_c.c_int32, _c.c_int64, _c.c_int32]),
    "dsv4kv_index_topk": (_c.c_int, [_c.c_void_p, _c.POINTER(CacheDesc), _c.c_int32, _c.c_int64, _c.c_int32,
                                     _c.c_void_p, _c.c_void_p, _c.c_void_p, _c.c_size_t, _c.c_void_p]),
    "dsv4kv_index_score": (_c.c_int, [_c.c_void_p, _c.POINTER(CacheDesc), _c.c_int32, _c.c_int64, _c.c_int32,
                                      _c.c_void_p, _c.c_size_t, _c.c_void_p]),
    "dsv4kv_append": (_c.c_int, [_c.c_void_p, _c.c_void_p, _c.c_int32, _c.c_int64, _c.c_int32, _c.c_int32,
                                 _c.c_int32, _c.c_int32, _c.c_int32, _c.c_double, _c.c_void_p, _c.c_void_p,
                                 _c.c_void_p, _c.c_int64, _c.c_void_p]),
    "dsv4kv_index_topk_pool_workspace_bytes": (_c.c_size_t, [_c.c_int32, _c.c_int32, _c.c_int32]),
    "dsv4kv_index_topk_pool": (_c.c_int, [_c.c_void_p, _c.POINTER(CacheDesc), _c.c_int32, _c.c_int64, _c.c_void_p,
                                          _c.c_int32, _c.c_int32, _c.c_void_p, _c.c_void_p, _c.c_void_p,
                                          _c.c_size_t, _c.c_void_p]),
    "dsv4kv_index_select": (_c.c_int, [_c.c_int32, _c.c_int64, _c.c_int32, _c.c_void_p, _c.c_void_p, _c.c_void_p,
                                       _c.c_size_t, _c.c_void_p]),
    "dsv4kv_index_topk_noalloc_max_scratch_bytes": (_c.c_size_t, []),
    "dsv4kv_index_topk_noalloc": (_c.c_int, [_c.c_void_p, _c.POINTER(CacheDesc), _c.c_int32, _c.c_int64, _c.c_int32,
                                             _c.c_void_p, _c.c_void_p, _c.c_void_p]),
    "dsv4kv_index_topk_noalloc_status": (_c.c_int, [_c.c_void_p, _c.c_int32, _c.c_void_p]),
    "dsv4kv_selftest_wait_timeout": (_c.c_int, [_c.c_void_p, _c.c_void_p]),
    "dsv4kv_sparse_decode_workspace_bytes": (_c.c_size_t, [_c.c_int32, _c.c_int32, _c.c_int32, _c.c_int32,
                                                           _c.c_int32]),
    "dsv4kv_sparse_decode": (_c.c_int, [_c.c_void_p, _c.POINTER(CacheDesc), _c.POINTER(CacheDesc), _c.c_void_p,
                                        _c.c_int32, _c.c_int32, _c.c_int64, _c.c_int32, _c.c_int32, _c.c_int64,
                                        _c.c_float, _c.c_int32, _c.c_double, _c.c_int32, _c.c_void_p,
                                        _c.c_void_p, _c.c_size_t, _c.c_void_p]),
    "dsv4kv_index_topk_paged_workspace_bytes": (_c.c_size_t, [_c.c_int32, _c.c_int64, _c.c_int32, _c.c_int32,
                                                              _c.c_int32]),
    "dsv4kv_index_topk_paged": (_c.c_int, [_c.c_void_p, _c.POINTER(PagedDesc), _c.c_int32, _c.c_void_p, _c.c_int64,
                                           _c.c_int32, _c.c_int32, _c.c_int32, _c.c_void_p, _c.c_void_p,
                                           _c.c_void_p, _c.c_size_t, _c.c_void_p]),
    "dsv4kv_sparse_decode_paged_workspace_bytes": (_c.c_size_t, [_c.c_int32, _c.c_int32, _c.c_int32, _c.c_int32,
                                                                 _c.c_int32]),
    "dsv4kv_sparse_decode_paged": (_c.c_int, [_c.c_void_p, _c.POINTER(PagedDesc), _c.POINTER(PagedDesc),
                                              _c.c_void_p, _c.c_int32, _c.c_int32, _c.c_void_p, _c.c_int64,
                                              _c.c_int32, _c.c_int32, _c.c_int32, _c.c_float, _c.c_int32,
                                              _c.c_double, _c.c_int32, _c.c_void_p, _c.c_void_p, _c.c_size_t,
                                              _c.c_void_p]),
    "dsv4kv_dense_decode_paged_workspace_bytes": (_c.c_size_t, [_c.c_int32, _c.c_int32, _c.c_int32, _c.c_int64,
                                                                _c.c_int32, _c.c_int32]),
    "dsv4kv_dense_decode_paged": (_c.c_int, [_c.c_void_p, _c.POINTER(PagedDesc), _c.POINTER(PagedDesc), _c.c_int32,
                                             _c.c_int32, _c.c_void_p, _c.c_int64, _c.c_int32, _c.c_int32,
                                             _c.c_float, _c.c_int32, _c.c_double, _c.c_int32, _c.c_void_p,
                                             _c.c_void_p, _c.c_size_t, _c.c_void_p]),
    "dsv4kv_paged_step_workspace_bytes": (_c.c_size_t, [_c.c_int32]),
    "dsv4kv_block_table_update": (_c.c_int, [_c.c_void_p, _c.c_void_p, _c.c_int32, _c.c_int64, _c.c_int32, _c.c_int32,
                                             _c.c_int32, _c.c_int32, _c.c_void_p, _c.c_int32, _c.c_int64, _c.c_void_p,
                                             _c.c_int64, _c.c_void_p, _c.c_void_p, _c.c_void_p, _c.c_size_t,
                                             _c.c_void_p]),
    "dsv4kv_slot_map": (_c.c_int, [_c.c_void_p, _c.c_void_p, _c.c_int32, _c.c_int64, _c.c_int32, _c.c_int32,
                                   _c.c_int32, _c.c_void_p, _c.c_void_p, _c.c_int64,
                                   _c.c_void_p, _c.c_void_p, _c.c_void_p, _c.c_void_p, _c.c_void_p, _c.c_void_p,
                                   _c.c_size_t, _c.c_void_p]),
    "dsv4kv_append_paged": (_c.c_int, [_c.c_void_p, _c.c_void_p, _c.c_int32, _c.c_int64, _c.c_void_p, _c.c_void_p,
                                       _c.c_void_p, _c.c_void_p, _c.c_void_p, _c.c_int32, _c.c_int32, _c.c_int32,
                                       _c.c_int32, _c.c_int64, _c.c_int32, _c.c_double, _c.c_void_p,
                                       _c.c_void_p, _c.c_void_p, _c.c_void_p, _c.c_size_t,
                                       _c.c_void_p]),
    "dsv4kv_tree_decode_paged_workspace_bytes": (_c.c_size_t, [_c.c_int32, _c.c_int32, _c.c_int32, _c.c_int32,
                                                               _c.c_int64, _c.c_int64, _c.c_int32, _c.c_int32,
                                                               _c.c_int32]),
    "dsv4kv_tree_decode_paged": (_c.c_int, [_c.c_void_p, _c.c_void_p, _c.c_void_p,
                                            _c.c_void_p, _c.c_void_p, _c.c_void_p, _c.c_void_p, _c.c_int32,
                                            _c.c_int32, _c.c_int64, _c.c_int32, _c.c_void_p, _c.c_int64, _c.c_int32,
                                            _c.c_int32, _c.c_int32, _c.c_float, _c.c_int32, _c.c_double, _c.c_int32,
                                            _c.c_void_p, _c.c_void_p, _c.c_size_t, _c.c_void_p]),
    "dsv4kv_dense_decode_workspace_bytes": (_c.c_size_t, [_c.c_int32, _c.c_int32, _c.c_int32, _c.c_int64,
                                                          _c.c_int32]),
    "dsv4kv_dense_decode": (_c.c_int, [_c.c_void_p, _c.POINTER(CacheDesc), _c.POINTER(CacheDesc), _c.c_int32,
                                       _c.c_int32, _c.c_int64, _c.c_int32, _c.c_int64, _c.c_float, _c.c_int32,
                                       _c.c_double, _c.c_int32, _c.c_void_p, _c.c_void_p, _c.c_size_t,
                                       _c.c_void_p]),
}


def lib() -> ctypes.CDLL:
    """Load libdsv4kv.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: build it with `python -m compressed_sparse_kv_b200.build`")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _lib = L
    return _lib


def _check(status: int, where: str) -> None:
    if status != 0:
        raise Dsv4kvError(status, where, lib().dsv4kv_last_error().decode())


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream(stream) -> Optional[int]:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream


@dataclass
class Cache:
    """A cache tensor [B][rows][dim] in one of the three formats."""
    fmt: int
    codes: torch.Tensor                      # bf16/u16 [B][rows][dim], u8 [B][rows][dim] or [B][rows][dim/2]
    scales: Optional[torch.Tensor] = None    # None, f32 [B][rows], u8 [B][rows][dim/16]
    dim: int = 512

    @property
    def rows(self) -> int:
        return int(self.codes.shape[1]) if self.codes.dim() >= 2 else 0

    def desc(self) -> CacheDesc:
        return CacheDesc(self.fmt, self.dim, self.rows, _ptr(self.codes), _ptr(self.scales))


@dataclass
class PagedCache:
    """A paged cache: rows of every sequence in pages of `page_rows` rows of one shared pool.
    Row i of sequence b is pool row table[b][i // page_rows] * page_rows + i % page_rows."""
    fmt: int
    codes: torch.Tensor                      # pool rows: [pool_pages * page_rows][row bytes or channels]
    table: torch.Tensor                      # int32 [B][table_stride] page numbers
    page_rows: int
    scales: Optional[torch.Tensor] = None    # pool scales per row (fp8: f32 [rows], fp4: u8 [rows][dim/16])
    dim: int = 512

    @property
    def pool_pages(self) -> int:
        return int(self.codes.shape[0]) // self.page_rows

    def desc(self) -> PagedDesc:
        return PagedDesc(self.fmt, self.dim, self.page_rows, int(self.table.shape[1]), self.pool_pages,
                         _ptr(self.table), _ptr(self.codes), _ptr(self.scales))


@dataclass
class PageTable:
    """The page numbers of a cache without its rows (a PagedCache will do wherever one is taken)."""
    table: torch.Tensor                      # int32 [B][table_stride]
    page_rows: int
    pool_pages: int


@dataclass
class SlotMap:
    """Where the new tokens of a step go (slot_map): token i of the packed batch belongs to sequence seq[i] at position
    pos[i]; win_slot / comp_slot are the pool rows that it writes (-1: none); cu[b] is sequence b's first token."""
    cu: torch.Tensor                         # int32 [B + 1]
    seq: torch.Tensor                        # int32 [capacity], -1 behind the last token
    pos: torch.Tensor                        # int64 [capacity]
    win_slot: torch.Tensor                   # int32 [capacity]
    comp_slot: torch.Tensor                  # int32 [capacity]


# The serving-step calls run once per layer and step, so their checks are written to cost well under a microsecond each:
# every tensor is dense, of its type, on the call's device (its index) and of its shape.
_I32, _I64, _F32, _BF, _U8 = torch.int32, torch.int64, torch.float32, torch.bfloat16, torch.uint8
_BF_WORDS = (torch.bfloat16, torch.uint16, torch.int16)      # bf16 rows may come as 16-bit words
_PAGED = struct.Struct("@iiiiqPPP")   # dsv4kv_paged_cache
_CACHE = struct.Struct("@iiqPP")      # dsv4kv_cache
_TABLE = struct.Struct("@Piiq")       # dsv4kv_page_table


def _is(t, dtype, dev: int) -> bool:
    return t.dtype is dtype and t.get_device() == dev and t.is_contiguous()


def _refuse(t, dtype, shape: str, dev: int, where: str, name: str):
    raise ValueError(f"{where}: {name} must be a contiguous {dtype} tensor {shape} on device {dev}, "
                     f"got {t.dtype} {list(t.shape)} on {t.device}")


def _on(dev: int, stream, where: str):
    """(context, stream handle) of a call: on its tensors' device and `stream`, or that device's current stream; what
    the call allocates inside the context belongs to that stream."""
    if dev < 0:
        raise ValueError(f"{where}: the tensors must be on a CUDA device")
    if stream is not None:
        if stream.device.index != dev:
            raise ValueError(f"{where}: the stream is on {stream.device}, the tensors on device {dev}")
        return torch.cuda.stream(stream), stream.cuda_stream
    here = dev == torch.cuda.current_device()
    return _HERE if here else torch.cuda.device(dev), torch.cuda.current_stream(dev).cuda_stream


_HERE = contextlib.nullcontext()
_ROW_BYTES = {BF16: 1024, FP8_E4M3_ROW: 512, FP4_E2M1_G16: 256, FP8_E4M3_ROW_ROPE_BF16: 576}
_SCALE_BYTES = {FP8_E4M3_ROW: 4, FP4_E2M1_G16: 32, FP8_E4M3_ROW_ROPE_BF16: 4}


def _rows(c, rows: int, dev: int, where: str, name: str) -> tuple[int, int]:
    """(codes, scales) of a 512-channel cache that holds at least `rows` rows, densely, of its format's types, on the
    device."""
    t, fmt = c.codes, c.fmt
    per = _ROW_BYTES.get(fmt, 0) if c.dim == 512 else 0        # (else: the library's own refusal)
    if t.get_device() != dev or not t.is_contiguous() or t.numel() * t.element_size() < rows * per:
        raise ValueError(f"{where}: {name}.codes must be contiguous, on device {dev}, and hold {rows} rows")
    if t.dtype not in _BF_WORDS if fmt == BF16 else fmt in _SCALE_BYTES and t.element_size() != 1:
        raise ValueError(f"{where}: {name}.codes must be {'bf16' if fmt == BF16 else 'bytes'}, got {t.dtype}")
    if fmt == BF16:
        return t.data_ptr(), 0
    s = c.scales
    if s is None or s.get_device() != dev or not s.is_contiguous() or (
            per and s.numel() * s.element_size() < rows * _SCALE_BYTES[fmt]):
        raise ValueError(f"{where}: {name}.scales must be contiguous, on device {dev}, and hold {rows} rows")
    if s.element_size() != 1 if fmt == FP4_E2M1_G16 else fmt in _SCALE_BYTES and s.dtype is not _F32:
        raise ValueError(f"{where}: {name}.scales must be {'bytes' if fmt == FP4_E2M1_G16 else 'float32'}, got {s.dtype}")
    return t.data_ptr(), s.data_ptr()


def _paged(c, b: int, dev: int, where: str, name: str) -> bytes:
    """The descriptor of a paged cache of b sequences."""
    t = c.table
    if not (_is(t, _I32, dev) and t.dim() == 2 and t.shape[0] == b):
        _refuse(t, _I32, f"[{b}, ...]", dev, where, name + ".table")
    page, pages = c.page_rows, c.pool_pages
    codes, scales = _rows(c, page * pages, dev, where, name)
    return _PAGED.pack(c.fmt, c.dim, page, t.shape[1], pages, t.data_ptr(), codes, scales)


def _table(c, b: int, dev: int, where: str, name: str):
    if c is None:
        return None
    t = c.table
    if not (_is(t, _I32, dev) and t.dim() == 2 and t.shape[0] == b):
        _refuse(t, _I32, f"[{b}, ...]", dev, where, name)
    return _TABLE.pack(t.data_ptr(), c.page_rows, t.shape[1], c.pool_pages)


def _lengths(t_old, t_new, where: str) -> tuple[int, int]:
    dev, b = t_old.get_device(), t_old.numel()
    for t, name in ((t_old, "t_old"), (t_new, "t_new")):
        if not (_is(t, _I64, dev) and t.shape == (b,)):
            _refuse(t, _I64, f"[{b}]", dev, where, name)
    return dev, b


def _workspace(ws, nbytes: int, dev: int, where: str):
    if ws is None:
        return new_workspace(nbytes, dev)
    if not (_is(ws, _U8, dev) and ws.dim() == 1):
        _refuse(ws, _U8, "[bytes]", dev, where, "ws")
    return ws


def new_workspace(nbytes: int, device=None) -> torch.Tensor:
    """Zero-filled workspace.  A call leaves it ready for the next one of its kind; decode calls leave partial sums in
    it, so zero it again before an index call takes it over."""
    return torch.zeros(max(int(nbytes), 16), dtype=torch.uint8, device=device or "cuda")


def workspace_status(ws: torch.Tensor) -> int:
    """The sticky device status word of a workspace (DEV_* flags)."""
    return int(ws[:4].view(torch.int32).item())


def compress_entries(t: int, window: int, stride: int) -> int:
    return int(lib().dsv4kv_compress_entries(t, window, stride))


def compress(s_raw: torch.Tensor, w: torch.Tensor, stride: int, window: int, pos0: int = 0, rope_dim: int = 64,
             rope_base: float = 10000.0, out_fp32: bool = False, out: Optional[torch.Tensor] = None,
             stream=None) -> torch.Tensor:
    """s_raw bf16 [B][t][D], w f32 [K][D] -> entries [B][N][D] (bf16 or f32)."""
    b, t, d = s_raw.shape
    n = compress_entries(t, window, stride)
    if out is None:
        out = torch.empty((b, n, d), dtype=torch.float32 if out_fp32 else torch.bfloat16, device=s_raw.device)
    _check(lib().dsv4kv_compress(_ptr(s_raw), _ptr(w), b, t, d, int(w.shape[0]), stride, window, pos0, rope_dim,
                                 rope_base, int(out_fp32), _ptr(out), _stream(stream)), "dsv4kv_compress")
    return out


def append(s_new: torch.Tensor, w: torch.Tensor, t: int, stride: int, window: int, raw_ring: torch.Tensor,
           win_ring: Optional[torch.Tensor], comp: torch.Tensor, rope_dim: int = 64, rope_base: float = 10000.0,
           stream=None) -> None:
    """Append the states s_new bf16 [B][D] of position t: raw ring [B][W+K][D], window ring [B][W][D] and,
    when an entry's block leaves the window, that entry into comp [B][rows][D] (all bf16)."""
    b, d = int(s_new.shape[0]), int(s_new.shape[1])
    _check(lib().dsv4kv_append(_ptr(s_new), _ptr(w), b, t, d, int(w.shape[0]), stride, window, rope_dim, rope_base,
                               _ptr(raw_ring), _ptr(win_ring) if win_ring is not None else None, _ptr(comp),
                               int(comp.shape[1]), _stream(stream)), "dsv4kv_append")


def quantize(x: torch.Tensor, fmt: int, codes: Optional[torch.Tensor] = None,
             scales: Optional[torch.Tensor] = None, stream=None) -> tuple[torch.Tensor, torch.Tensor]:
    """Rows x [..., D] (bf16 or f32) -> (codes, scales) in a quantised cache format: fp8 rows
    (codes [..., D], scales f32 [...]), fp4 (codes [..., D/2], E4M3 scales [..., D/16]) or fp8
    with the last 64 channels in bf16 (row bytes [..., D + 64], scales f32 [...])."""
    d = int(x.shape[-1])
    rows = x.numel() // d
    lead = tuple(x.shape[:-1])
    row_bytes = {FP8_E4M3_ROW: d, FP4_E2M1_G16: d // 2, FP8_E4M3_ROW_ROPE_BF16: d + 64}.get(fmt, d)
    if codes is None:
        codes = torch.empty(lead + (row_bytes,), dtype=torch.uint8, device=x.device)
    if scales is None:
        scales = (torch.empty(lead + (d // 16,), dtype=torch.uint8, device=x.device) if fmt == FP4_E2M1_G16
                  else torch.empty(lead, dtype=torch.float32, device=x.device))
    _check(lib().dsv4kv_quantize(_ptr(x), int(x.dtype == torch.float32), rows, d, fmt, _ptr(codes), _ptr(scales),
                                 _stream(stream)), "dsv4kv_quantize")
    return codes, scales


def index_topk_workspace_bytes(batch: int, n: int, k: int) -> int:
    return int(lib().dsv4kv_index_topk_workspace_bytes(batch, n, k))


def index_topk(qidx: torch.Tensor, keys: Cache, n: int, k: int, idx_out: Optional[torch.Tensor] = None,
               count_out: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None,
               stream=None) -> tuple[torch.Tensor, torch.Tensor]:
    """qidx bf16 [B][128], keys [B][>=n][128] -> (idx int32 [B][k] ascending, -1 padded; count int32 [B])."""
    b = int(qidx.shape[0])
    dev = qidx.device
    if idx_out is None:
        idx_out = torch.empty((b, k), dtype=torch.int32, device=dev)
    if count_out is None:
        count_out = torch.empty((b,), dtype=torch.int32, device=dev)
    if ws is None:
        ws = new_workspace(index_topk_workspace_bytes(b, n, k), dev)
    d = keys.desc()
    _check(lib().dsv4kv_index_topk(_ptr(qidx), ctypes.byref(d), b, n, k, _ptr(idx_out), _ptr(count_out), _ptr(ws),
                                   ws.numel(), _stream(stream)), "dsv4kv_index_topk")
    return idx_out, count_out


def index_score(qidx: torch.Tensor, keys: Cache, n: int, k: int, ws: torch.Tensor, stream=None) -> None:
    """The scoring half of index_topk: scores and histogram into ws (index_topk_workspace_bytes sized)."""
    d = keys.desc()
    _check(lib().dsv4kv_index_score(_ptr(qidx), ctypes.byref(d), int(qidx.shape[0]), n, k, _ptr(ws), ws.numel(),
                                    _stream(stream)), "dsv4kv_index_score")


def index_select(batch: int, n: int, k: int, idx_out: torch.Tensor, count_out: Optional[torch.Tensor],
                 ws: torch.Tensor, stream=None) -> tuple[torch.Tensor, Optional[torch.Tensor]]:
    """The selection half of index_topk, from the workspace index_score filled."""
    _check(lib().dsv4kv_index_select(batch, n, k, _ptr(idx_out), _ptr(count_out) if count_out is not None else None,
                                     _ptr(ws), ws.numel(), _stream(stream)), "dsv4kv_index_select")
    return idx_out, count_out


def index_topk_pool(qidx: torch.Tensor, keys: Cache, n: int, pool: torch.Tensor, k: int,
                    idx_out: Optional[torch.Tensor] = None, count_out: Optional[torch.Tensor] = None,
                    ws: Optional[torch.Tensor] = None, stream=None) -> tuple[torch.Tensor, torch.Tensor]:
    """Top-k re-index inside a candidate pool: pool int32 [B][P] (ascending entries, negative = none)
    -> (idx int32 [B][k] ascending, -1 padded; count int32 [B])."""
    b = int(qidx.shape[0])
    p = int(pool.shape[1]) if pool.dim() == 2 else 0
    if idx_out is None:
        idx_out = torch.empty((b, k), dtype=torch.int32, device=qidx.device)
    if count_out is None:
        count_out = torch.empty((b,), dtype=torch.int32, device=qidx.device)
    if ws is None:
        ws = new_workspace(int(lib().dsv4kv_index_topk_pool_workspace_bytes(b, p, k)), qidx.device)
    d = keys.desc()
    _check(lib().dsv4kv_index_topk_pool(_ptr(qidx), ctypes.byref(d), b, n, _ptr(pool), p, k, _ptr(idx_out),
                                        _ptr(count_out), _ptr(ws), ws.numel(), _stream(stream)),
           "dsv4kv_index_topk_pool")
    return idx_out, count_out


def index_topk_noalloc(qidx: torch.Tensor, keys: Cache, n: int, k: int, idx_out: Optional[torch.Tensor] = None,
                       count_out: Optional[torch.Tensor] = None, stream=None) -> tuple[torch.Tensor, torch.Tensor]:
    """index_topk with the library's static device scratch instead of a workspace (for callers that
    cannot allocate device memory; concurrent calls on the GPU race)."""
    b = int(qidx.shape[0])
    if idx_out is None:
        idx_out = torch.empty((b, k), dtype=torch.int32, device=qidx.device)
    if count_out is None:
        count_out = torch.empty((b,), dtype=torch.int32, device=qidx.device)
    d = keys.desc()
    _check(lib().dsv4kv_index_topk_noalloc(_ptr(qidx), ctypes.byref(d), b, n, k, _ptr(idx_out), _ptr(count_out),
                                           _stream(stream)), "dsv4kv_index_topk_noalloc")
    return idx_out, count_out


def index_topk_noalloc_status(clear: bool = False, stream=None) -> int:
    """The device status word (DEV_* flags) that the calls of index_topk_noalloc have accumulated in the
    static scratch since it was last cleared; `clear` zeroes it after reading."""
    word = torch.zeros(1, dtype=torch.int32).pin_memory()
    s = torch.cuda.current_stream() if stream is None else stream
    _check(lib().dsv4kv_index_topk_noalloc_status(_ptr(word), int(clear), _stream(s)),
           "dsv4kv_index_topk_noalloc_status")
    s.synchronize()
    return int(word.item()) & 0xffffffff


def selftest_wait_timeout(status: torch.Tensor, stream=None) -> None:
    """Launch the library's bounded-wait self-test: after about one second on the GPU it ORs DEV_TIMEOUT
    into `status` (one int32 on the device)."""
    _check(lib().dsv4kv_selftest_wait_timeout(_ptr(status), _stream(stream)), "dsv4kv_selftest_wait_timeout")


def sparse_decode_workspace_bytes(batch: int, heads: int, k: int, window: int, dim: int = 512) -> int:
    return int(lib().dsv4kv_sparse_decode_workspace_bytes(batch, heads, dim, k, window))


def dense_decode_workspace_bytes(batch: int, heads: int, n: int, window: int, dim: int = 512) -> int:
    return int(lib().dsv4kv_dense_decode_workspace_bytes(batch, heads, dim, n, window))


def sparse_decode(q: torch.Tensor, comp: Cache, win: Cache, idx: torch.Tensor, n: int, window: int, t: int,
                  sm_scale: Optional[float] = None, rope_dim: int = 64, rope_base: float = 10000.0,
                  out_fp32: bool = False, out: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None,
                  stream=None) -> torch.Tensor:
    """q bf16 [B][H][512] -> out [B][H][512]; idx int32 [B][k] from index_topk."""
    b, h, d = q.shape
    k = int(idx.shape[1])
    if sm_scale is None:
        sm_scale = d ** -0.5
    if out is None:
        out = torch.empty((b, h, d), dtype=torch.float32 if out_fp32 else torch.bfloat16, device=q.device)
    if ws is None:
        ws = new_workspace(sparse_decode_workspace_bytes(b, h, k, window, d), q.device)
    cd, wd = comp.desc(), win.desc()
    _check(lib().dsv4kv_sparse_decode(_ptr(q), ctypes.byref(cd), ctypes.byref(wd), _ptr(idx), b, h, n, window, k, t,
                                      sm_scale, rope_dim, rope_base, int(out_fp32), _ptr(out), _ptr(ws), ws.numel(),
                                      _stream(stream)), "dsv4kv_sparse_decode")
    return out


def dense_decode(q: torch.Tensor, comp: Cache, win: Cache, n: int, window: int, t: int,
                 sm_scale: Optional[float] = None, rope_dim: int = 64, rope_base: float = 10000.0,
                 out_fp32: bool = False, out: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None,
                 stream=None) -> torch.Tensor:
    """q bf16 [B][H][512] -> out [B][H][512] over all n compressed rows plus the window."""
    b, h, d = q.shape
    if sm_scale is None:
        sm_scale = d ** -0.5
    if out is None:
        out = torch.empty((b, h, d), dtype=torch.float32 if out_fp32 else torch.bfloat16, device=q.device)
    if ws is None:
        ws = new_workspace(dense_decode_workspace_bytes(b, h, n, window, d), q.device)
    cd, wd = comp.desc(), win.desc()
    _check(lib().dsv4kv_dense_decode(_ptr(q), ctypes.byref(cd), ctypes.byref(wd), b, h, n, window, t, sm_scale,
                                     rope_dim, rope_base, int(out_fp32), _ptr(out), _ptr(ws), ws.numel(),
                                     _stream(stream)), "dsv4kv_dense_decode")
    return out


def index_topk_paged(qidx: torch.Tensor, keys: PagedCache, t_seq: torch.Tensor, t_max: int, k: int,
                     window: int = 128, stride: int = 4, idx_out: Optional[torch.Tensor] = None,
                     count_out: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None,
                     stream=None) -> tuple[torch.Tensor, torch.Tensor]:
    """Ragged, paged top-k: t_seq int64 [B] (device) query positions, sequence b has
    max(0, (t_b - window) // stride) keys -> (idx int32 [B][k] ascending, -1 padded; count int32 [B])."""
    b = int(qidx.shape[0])
    dev = qidx.device
    if idx_out is None:
        idx_out = torch.empty((b, k), dtype=torch.int32, device=dev)
    if count_out is None:
        count_out = torch.empty((b,), dtype=torch.int32, device=dev)
    if ws is None:
        ws = new_workspace(int(lib().dsv4kv_index_topk_paged_workspace_bytes(b, t_max, window, stride, k)), dev)
    d = keys.desc()
    _check(lib().dsv4kv_index_topk_paged(_ptr(qidx), ctypes.byref(d), b, _ptr(t_seq), t_max, window, stride, k,
                                         _ptr(idx_out), _ptr(count_out), _ptr(ws), ws.numel(), _stream(stream)),
           "dsv4kv_index_topk_paged")
    return idx_out, count_out


def sparse_decode_paged(q: torch.Tensor, comp: PagedCache, win: PagedCache, idx: torch.Tensor, t_seq: torch.Tensor,
                        t_max: int, window: int = 128, stride: int = 4, sm_scale: Optional[float] = None,
                        rope_dim: int = 64, rope_base: float = 10000.0, out_fp32: bool = False,
                        out: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None,
                        stream=None) -> torch.Tensor:
    """Ragged, paged c4a decode: q bf16 [B][H][512], idx int32 [B][k] from index_topk_paged."""
    b, h, d = q.shape
    k = int(idx.shape[1])
    if sm_scale is None:
        sm_scale = d ** -0.5
    if out is None:
        out = torch.empty((b, h, d), dtype=torch.float32 if out_fp32 else torch.bfloat16, device=q.device)
    if ws is None:
        ws = new_workspace(int(lib().dsv4kv_sparse_decode_paged_workspace_bytes(b, h, d, k, window)), q.device)
    cd, wd = comp.desc(), win.desc()
    _check(lib().dsv4kv_sparse_decode_paged(_ptr(q), ctypes.byref(cd), ctypes.byref(wd), _ptr(idx), b, h, _ptr(t_seq),
                                            t_max, window, stride, k, sm_scale, rope_dim, rope_base, int(out_fp32),
                                            _ptr(out), _ptr(ws), ws.numel(), _stream(stream)),
           "dsv4kv_sparse_decode_paged")
    return out


def dense_decode_paged(q: torch.Tensor, comp: PagedCache, win: PagedCache, t_seq: torch.Tensor, t_max: int,
                       window: int = 128, stride: int = 128, sm_scale: Optional[float] = None, rope_dim: int = 64,
                       rope_base: float = 10000.0, out_fp32: bool = False, out: Optional[torch.Tensor] = None,
                       ws: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Ragged, paged c128a decode over every sequence's n_b entries plus its window rows."""
    b, h, d = q.shape
    if sm_scale is None:
        sm_scale = d ** -0.5
    if out is None:
        out = torch.empty((b, h, d), dtype=torch.float32 if out_fp32 else torch.bfloat16, device=q.device)
    if ws is None:
        ws = new_workspace(int(lib().dsv4kv_dense_decode_paged_workspace_bytes(b, h, d, t_max, window, stride)),
                           q.device)
    cd, wd = comp.desc(), win.desc()
    _check(lib().dsv4kv_dense_decode_paged(_ptr(q), ctypes.byref(cd), ctypes.byref(wd), b, h, _ptr(t_seq), t_max,
                                           window, stride, sm_scale, rope_dim, rope_base, int(out_fp32), _ptr(out),
                                           _ptr(ws), ws.numel(), _stream(stream)), "dsv4kv_dense_decode_paged")
    return out


def paged_step_workspace_bytes(batch: int) -> int:
    return int(lib().dsv4kv_paged_step_workspace_bytes(batch))


def block_table_update(t_old: torch.Tensor, t_new: torch.Tensor, pages, free_pages: torch.Tensor,
                       free_count: torch.Tensor, t_max: int, window: int = 128, stride: int = 4, lookahead: int = 0,
                       free_count_out: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None,
                       stream=None) -> torch.Tensor:
    """Take pages for the sequences that grow from t_old to t_new (int64 [B]) and give back those of the ones that
    shrink: pages (PageTable or PagedCache) gets its table rows filled in place, free_pages int32 [cap] is a stack of
    free_count (int64 [1]) page numbers.  stride 0: the table of a window cache.  Returns the new count
    (free_count_out; pass free_count itself to update it in place)."""
    where = "block_table_update"
    dev, b = _lengths(t_old, t_new, where)
    table = pages.table
    if not (_is(table, _I32, dev) and table.dim() == 2 and table.shape[0] == b):
        _refuse(table, _I32, f"[{b}, ...]", dev, where, "table")
    if not (_is(free_pages, _I32, dev) and free_pages.dim() == 1):
        _refuse(free_pages, _I32, "[cap]", dev, where, "free_pages")
    if not (_is(free_count, _I64, dev) and free_count.numel() == 1):
        _refuse(free_count, _I64, "[1]", dev, where, "free_count")
    ctx, s = _on(dev, stream, where)
    with ctx:
        if free_count_out is None:
            free_count_out = torch.empty_like(free_count)
        elif not (_is(free_count_out, _I64, dev) and free_count_out.numel() == 1):
            _refuse(free_count_out, _I64, "[1]", dev, where, "free_count_out")
        ws = _workspace(ws, 16, dev, where)
        _check(lib().dsv4kv_block_table_update(
            t_old.data_ptr(), t_new.data_ptr(), b, t_max, window, stride, lookahead, pages.page_rows, table.data_ptr(),
            table.shape[1], pages.pool_pages, free_pages.data_ptr(), free_pages.shape[0],
            free_count.data_ptr(), free_count_out.data_ptr(), ws.data_ptr(), ws.numel(), s), "dsv4kv_block_table_update")
    return free_count_out


def new_slot_map(batch: int, capacity: int, device=None) -> SlotMap:
    e = lambda n, dt: torch.empty(n, dtype=dt, device="cuda" if device is None else device)  # noqa: E731
    return SlotMap(e(batch + 1, torch.int32), e(capacity, torch.int32), e(capacity, torch.int64),
                   e(capacity, torch.int32), e(capacity, torch.int32))


def _need_slots(m: SlotMap, b: int, cap: int, dev: int, where: str) -> None:
    if not (_is(m.cu, _I32, dev) and m.cu.shape == (b + 1,)):
        _refuse(m.cu, _I32, f"[{b + 1}]", dev, where, "cu")
    for t, dt, name in ((m.seq, _I32, "seq"), (m.pos, _I64, "pos"), (m.win_slot, _I32, "win_slot"),
                        (m.comp_slot, _I32, "comp_slot")):
        if not (_is(t, dt, dev) and t.shape == (cap,)):
            _refuse(t, dt, f"[{cap}]", dev, where, name)


def slot_map(t_old: torch.Tensor, t_new: torch.Tensor, comp, win, capacity: int, t_max: int, window: int = 128,
             stride: int = 4, lookahead: int = 0, out: Optional[SlotMap] = None, ws: Optional[torch.Tensor] = None,
             stream=None) -> SlotMap:
    """Sequence, position and cache slots of the new tokens t_old[b] .. t_new[b] - 1 of every sequence, packed in
    order of b; comp and win are PageTables or PagedCaches (comp may be None, win too when window is 0)."""
    where = "slot_map"
    dev, b = _lengths(t_old, t_new, where)
    cd, wd = _table(comp, b, dev, where, "comp.table"), _table(win, b, dev, where, "win.table")
    ctx, s = _on(dev, stream, where)
    with ctx:
        if out is None:
            out = new_slot_map(b, capacity, dev)
        else:
            _need_slots(out, b, capacity, dev, where)
        ws = _workspace(ws, 16, dev, where)
        _check(lib().dsv4kv_slot_map(
            t_old.data_ptr(), t_new.data_ptr(), b, t_max, window, stride, lookahead, cd, wd, capacity,
            out.cu.data_ptr(), out.seq.data_ptr(), out.pos.data_ptr(), out.win_slot.data_ptr(),
            out.comp_slot.data_ptr(), ws.data_ptr(), ws.numel(), s), "dsv4kv_slot_map")
    return out


def append_paged(s_new: torch.Tensor, w: torch.Tensor, slots: SlotMap, raw_ring: torch.Tensor,
                 win: Optional[PagedCache], comp: PagedCache, stride: int, window: int = 128, lookahead: int = 0,
                 max_new: Optional[int] = None, rope_dim: int = 64, rope_base: float = 10000.0,
                 ws: Optional[torch.Tensor] = None, stream=None) -> None:
    """Append the states s_new bf16 [capacity][512] of a slot map's tokens: raw_ring bf16 [B][window + K][512], the
    window rows and the entries that are due (w f32 [K][512]) into the paged caches, in their format.  max_new: no
    sequence has more new tokens (a tight one saves a launch)."""
    where = "append_paged"
    dev, b, taps, cap = s_new.get_device(), raw_ring.shape[0], w.shape[0], slots.seq.shape[0]
    _need_slots(slots, b, cap, dev, where)
    if not (_is(s_new, _BF, dev) and s_new.shape == (cap, 512)):
        _refuse(s_new, _BF, f"[{cap}, 512]", dev, where, "s_new")
    if not (_is(w, _F32, dev) and w.shape == (taps, 512)):
        _refuse(w, _F32, "[K, 512]", dev, where, "w")
    if not (_is(raw_ring, _BF, dev) and raw_ring.shape == (b, window + taps, 512)):
        _refuse(raw_ring, _BF, f"[B, {window + taps}, 512]", dev, where, "raw_ring")
    cd = _paged(comp, b, dev, where, "comp")
    wd = None if win is None else _paged(win, b, dev, where, "win")
    ctx, s = _on(dev, stream, where)
    with ctx:
        ws = _workspace(ws, 16, dev, where)
        _check(lib().dsv4kv_append_paged(
            s_new.data_ptr(), w.data_ptr(), b, cap, slots.cu.data_ptr(), slots.seq.data_ptr(), slots.pos.data_ptr(),
            slots.win_slot.data_ptr(), slots.comp_slot.data_ptr(), taps, stride, window, lookahead,
            cap if max_new is None else max_new, rope_dim, rope_base, raw_ring.data_ptr(), wd, cd, ws.data_ptr(),
            ws.numel(), s), "dsv4kv_append_paged")


def tree_decode_paged_workspace_bytes(batch: int, heads: int, max_nodes: int, nodes: int, t_max: int, window: int = 128,
                                      stride: int = 128, k: Optional[int] = None) -> int:
    """k: places per node of the sparse form's idx, None for the dense form."""
    return int(lib().dsv4kv_tree_decode_paged_workspace_bytes(batch, heads, 512, max_nodes, nodes, t_max, window,
                                                              stride, k or 0))


def tree_decode_paged(q: torch.Tensor, comp: PagedCache, win: PagedCache, draft: Cache, cu: torch.Tensor,
                      parent: torch.Tensor, t_seq: torch.Tensor, t_max: int, max_nodes: int, window: int = 128,
                      stride: int = 128, idx: Optional[torch.Tensor] = None, sm_scale: Optional[float] = None,
                      rope_dim: int = 64, rope_base: float = 10000.0, out_fp32: bool = False,
                      out: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None,
                      stream=None) -> torch.Tensor:
    """Attention of drafted tokens over paged caches: q bf16 [nodes][H][512] and the rows of draft (codes
    [1][nodes][...]) packed by sequence (cu int32 [B + 1]); parent int32 [nodes] numbers within the sequence, -1 for a
    child of the last cached token.  idx int32 [nodes][k]: each node's selected entries (c4a); None: all (c128a)."""
    where = "tree_decode_paged"
    n, h, d = q.shape
    dev, b = q.get_device(), t_seq.numel()
    if not (_is(q, _BF, dev) and d == 512):
        _refuse(q, _BF, "[nodes, H, 512]", dev, where, "q")
    if not (_is(cu, _I32, dev) and cu.shape == (b + 1,)):
        _refuse(cu, _I32, f"[{b + 1}]", dev, where, "cu")
    if not (_is(parent, _I32, dev) and parent.shape == (n,)):
        _refuse(parent, _I32, f"[{n}]", dev, where, "parent")
    if not (_is(t_seq, _I64, dev) and t_seq.dim() == 1):
        _refuse(t_seq, _I64, "[B]", dev, where, "t_seq")
    cd, wd = _paged(comp, b, dev, where, "comp"), _paged(win, b, dev, where, "win")
    dd = _CACHE.pack(draft.fmt, draft.dim, n, *_rows(draft, n, dev, where, "draft"))
    k, ip = 0, None
    if idx is not None:
        if not (_is(idx, _I32, dev) and idx.dim() == 2 and idx.shape[0] == n):
            _refuse(idx, _I32, f"[{n}, k]", dev, where, "idx")
        k, ip = idx.shape[1], idx.data_ptr()
    if sm_scale is None:
        sm_scale = d ** -0.5
    ctx, s = _on(dev, stream, where)
    with ctx:
        dt = _F32 if out_fp32 else _BF
        if out is None:
            out = torch.empty((n, h, d), dtype=dt, device=q.device)
        elif not (_is(out, dt, dev) and out.shape == q.shape):
            _refuse(out, dt, f"[{n}, {h}, 512]", dev, where, "out")
        if ws is None:
            ws = new_workspace(tree_decode_paged_workspace_bytes(b, h, max_nodes, n, t_max, window, stride, k), q.device)
        else:
            ws = _workspace(ws, 0, dev, where)
        _check(lib().dsv4kv_tree_decode_paged(
            q.data_ptr(), cd, wd, dd, cu.data_ptr(), parent.data_ptr(), ip, b, h, n, max_nodes, t_seq.data_ptr(), t_max,
            window, stride, k, sm_scale, rope_dim, rope_base, out_fp32, out.data_ptr(), ws.data_ptr(), ws.numel(), s),
            "dsv4kv_tree_decode_paged")
    return out
