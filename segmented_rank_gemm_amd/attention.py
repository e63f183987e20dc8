"""The operators around the projections (``include/lora_attention.h``): the norm
in front of a projection, the rotation and cache write behind it, and attention
over the 4-bit paged cache.

As in the rest of the binding, the functions carry the C entry points' names and
only marshal arguments: shapes and strides come from the tensors, the stream is
the current one unless given, and every step runs in the library's HIP kernels.
"""

from __future__ import annotations

import ctypes
from typing import Optional, Tuple

import torch

__all__ = [
    "lora_rms_norm", "lora_kv_append", "lora_kv_read", "lora_kv_attention",
    "lora_kv_attention_workspace_bytes", "kv_attention_workspace", "kv_cache_shape", "rope_table",
    "SUPPORTED_HEAD_DIMS", "SUPPORTED_PAGE_SIZES",
]

SUPPORTED_HEAD_DIMS = (64, 128)
SUPPORTED_PAGE_SIZES = (16, 32, 64, 128, 256)

_VP = ctypes.c_void_p
_I32 = ctypes.c_int32
_I64 = ctypes.c_int64


def _declare(L: ctypes.CDLL) -> None:
    """Argument types of the entry points, on the loaded library."""
    L.lora_rms_norm.argtypes = [_VP, _I64, _VP, _I64, _VP, ctypes.c_double, _I32, _I32, _VP, _I64,
                                _VP, _I64, _VP, _I64, _VP, _I32, _VP]
    L.lora_rms_norm.restype = ctypes.c_int
    L.lora_kv_append.argtypes = [_VP, _I64, _VP, _VP, _VP, _I32, _I32, _I32, _I32, _I32, _I32, _I32,
                                 _VP, _I64, _VP, _I32, _I32, _VP]
    L.lora_kv_append.restype = ctypes.c_int
    L.lora_kv_read.argtypes = [_VP, _I32, _I32, _I32, _VP, _I32, _I32, _VP, _I64, _VP, _I64, _VP]
    L.lora_kv_read.restype = ctypes.c_int
    L.lora_kv_attention_workspace_bytes.argtypes = [_I32] * 6
    L.lora_kv_attention_workspace_bytes.restype = _I64
    L.lora_kv_attention.argtypes = [_VP, _I64, _VP, _VP, _VP, _I64, _VP, _I32, _I32, _I32, _I32,
                                    _I32, _I32, _I32, _I32, _I32, ctypes.c_float, _I32, _VP, _I64,
                                    _VP, _I64, _VP]
    L.lora_kv_attention.restype = ctypes.c_int


from . import LoraError, _dev_ptr, _flat_dev_bytes, _stream_handle, lib  # noqa: E402

_declare(lib())
# the entry points themselves: looking them up costs as much as a check
_rms_norm, _kv_append = lib().lora_rms_norm, lib().lora_kv_append
_kv_read, _kv_attention = lib().lora_kv_read, lib().lora_kv_attention


# The checks below run on every call, and a decode step's calls are as short as
# they are: each looks at a tensor's type, shape and strides once, and what is
# wrong is found out only when something is.
_BF16, _F32, _E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
_I32T, _I64T, _U8 = torch.int32, torch.int64, torch.uint8


def _refuse(t, dtype: torch.dtype, shape, name: str, layout: str) -> None:
    _dev_ptr(t, dtype, name)  # raises what the rest of the binding raises
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, is {list(t.shape)}")
    raise ValueError(f"{name} must {layout}, has strides {t.stride()}")


def _matrix(t: torch.Tensor, dtype: torch.dtype, rows: int, width: int, name: str):
    """Address and row stride of a [rows, width] matrix with unit column stride."""
    try:
        if t.dtype is dtype and t.is_cuda and t.shape == (rows, width):
            stride, unit = t.stride()
            if unit == 1 or width == 1:
                # a single row's stride is never used for an address: any that passes will do
                return t.data_ptr(), stride if rows > 1 else width
    except AttributeError:
        pass
    _refuse(t, dtype, (rows, width), name, "have unit column stride")


def _heads(t: torch.Tensor, rows: int, heads: int, head_dim: int, name: str):
    """Address and row stride of a bf16 [rows, heads, head_dim] tensor whose heads
    lie one behind another."""
    try:
        if t.dtype is _BF16 and t.is_cuda and t.shape == (rows, heads, head_dim):
            stride, between, unit = t.stride()
            if (unit == 1 or head_dim == 1) and (between == head_dim or heads == 1):
                return t.data_ptr(), stride if rows > 1 else heads * head_dim
    except AttributeError:
        pass
    _refuse(t, _BF16, (rows, heads, head_dim), name, "have each row's heads contiguous")


def _vector(t: torch.Tensor, dtype: torch.dtype, n: int, name: str) -> int:
    try:
        if t.dtype is dtype and t.is_cuda and t.shape == (n,) and (n <= 1 or t.stride(0) == 1):
            return t.data_ptr()
    except AttributeError:
        pass
    _refuse(t, dtype, (n,), name, "be contiguous")


_MOST = 0x7FFFFFFF  # the library's sizes are 32-bit: ctypes would cut others down to that


def _fit(**sizes: int) -> None:
    for name, n in sizes.items():
        if not -_MOST <= n <= _MOST:
            raise ValueError(f"{name} {n} does not fit 32 bits")


def _dims(t: torch.Tensor, n: int, name: str):
    shape = getattr(t, "shape", ())
    if len(shape) != n:
        raise ValueError(f"{name} must be a {n}-D tensor")
    return shape


def kv_cache_shape(num_pages: int, kv_heads: int, head_dim: int, page_size: int):
    """Shape of the uint8 cache tensor: [num_pages, 2, kv_heads, page_bytes]."""
    if head_dim not in SUPPORTED_HEAD_DIMS or page_size not in SUPPORTED_PAGE_SIZES:
        raise ValueError(f"head_dim is one of {SUPPORTED_HEAD_DIMS} and page_size one of "
                         f"{SUPPORTED_PAGE_SIZES}")
    return (int(num_pages), 2, int(kv_heads), page_size * (head_dim // 2 + head_dim // 32))


def _cache(cache: torch.Tensor, head_dim: int, page_size: Optional[int]) -> Tuple[int, int, int, int]:
    """Address, pages, kv_heads and page size of a cache for this head_dim.  The bytes
    of a page are a product of the two: heads of 128 in pages of 64 tokens and heads
    of 64 in pages of 128 have one shape, and only a caller's page_size tells them apart."""
    ptr = _dev_ptr(cache, _U8, "cache")
    shape = cache.shape
    if len(shape) != 4 or shape[1] != 2 or not cache.is_contiguous():
        raise ValueError("cache must be contiguous [num_pages, 2, kv_heads, page_bytes]")
    pages, _, heads, size = shape
    row = head_dim // 2 + head_dim // 32  # bytes of one token's head
    if row < 1 or size % row:
        raise ValueError(f"cache pages of {size} bytes hold no heads of {head_dim}")
    if page_size is not None and size != page_size * row:
        raise ValueError(f"cache pages of {size} bytes hold {size // row} heads of {head_dim}, "
                         f"not page_size {page_size}")
    return ptr, pages, heads, size // row


def rope_table(rows: int, rot_dim: int, base: float = 10000.0, device="cuda") -> torch.Tensor:
    """fp32 [rows, rot_dim]: cosines, then sines, of position * base^(-2i / rot_dim).
    The angles are taken in 64 bits: those of far positions pass what 32 resolve."""
    i = torch.arange(0, rot_dim, 2, device=device, dtype=torch.float64)
    angles = torch.arange(rows, device=device, dtype=torch.float64)[:, None] * base ** (-i / rot_dim)
    return torch.cat([angles.cos(), angles.sin()], dim=1).float()


def lora_rms_norm(x: torch.Tensor, weight: torch.Tensor, eps: float,
                  residual: Optional[torch.Tensor] = None,
                  residual_out: Optional[torch.Tensor] = None, y: Optional[torch.Tensor] = None,
                  y8: Optional[torch.Tensor] = None, scales: Optional[torch.Tensor] = None,
                  stream: Optional[torch.cuda.Stream] = None) -> None:
    """x, residual, residual_out, y: bf16 [tokens, hidden] (any row strides that
    are multiples of 8); weight: bf16 [hidden]; y8: float8_e4m3fn [tokens,
    hidden]; scales: fp32 [tokens, groups], groups scales a row (1: one a row,
    else hidden / 32, / 64, / 128 or / 256).  residual_out = x + residual, y its
    norm, y8 the norm in 8 bits; any of the three may be left out."""
    T, hidden = _dims(x, 2, "x")
    px, ldx = _matrix(x, _BF16, T, hidden, "x")
    pr = ldr = po = ldo = py = ldy = p8 = ld8 = ps = 0
    group = hidden
    if residual is not None:
        pr, ldr = _matrix(residual, _BF16, T, hidden, "residual")
    if residual_out is not None:
        po, ldo = _matrix(residual_out, _BF16, T, hidden, "residual_out")
    if y is not None:
        py, ldy = _matrix(y, _BF16, T, hidden, "y")
    if y8 is not None:
        p8, ld8 = _matrix(y8, _E4M3, T, hidden, "y8")
    if scales is not None:
        groups = _dims(scales, 2, "scales")[1]
        ps, ld = _matrix(scales, _F32, T, groups, "scales")
        if groups < 1 or hidden % groups or ld != groups:
            raise ValueError(f"scales must be contiguous, a whole number of them a row of {hidden}")
        group = hidden // groups
    status = _rms_norm(
        px, ldx, pr, ldr, _vector(weight, _BF16, hidden, "weight"), eps, T, hidden, po, ldo, py, ldy,
        p8, ld8, ps, group, _stream_handle(stream))
    if status:
        raise LoraError("lora_rms_norm", status)


def lora_kv_append(qkv: torch.Tensor, positions: Optional[torch.Tensor], slots: torch.Tensor,
                   rope: Optional[torch.Tensor], cache: torch.Tensor, q_out: torch.Tensor,
                   interleaved: bool = False, stream: Optional[torch.cuda.Stream] = None,
                   page_size: Optional[int] = None) -> None:
    """qkv: bf16 [tokens, (q_heads + 2 kv_heads) * head_dim]; positions: int32
    [tokens]; slots: int64 [tokens]; rope: fp32 [rows, rot_dim] (rope_table), or
    None for no rotation; cache: uint8 (kv_cache_shape); q_out: bf16 [tokens,
    q_heads, head_dim]; page_size: the cache's, to be checked (here and below): without
    it, it is what head_dim makes of the cache's shape, also where that is another's."""
    T, q_heads, head_dim = _dims(q_out, 3, "q_out")
    pq, ldq = _heads(q_out, T, q_heads, head_dim, "q_out")
    pc, pages, kv_heads, page_size = _cache(cache, head_dim, page_size)
    px, ldx = _matrix(qkv, _BF16, T, (q_heads + 2 * kv_heads) * head_dim, "qkv")
    rows = rot = pr = pp = 0
    if rope is not None:
        rows, rot = _dims(rope, 2, "rope")
        pr, ld = _matrix(rope, _F32, rows, rot, "rope")
        if ld != rot:
            raise ValueError("rope must be contiguous")
        pp = _vector(positions, _I32T, T, "positions")
    status = _kv_append(
        px, ldx, pp, _vector(slots, _I64T, T, "slots"), pr, rows, rot, 1 if interleaved else 0, T,
        q_heads, kv_heads, head_dim, pq, ldq, pc, pages, page_size, _stream_handle(stream))
    if status:
        raise LoraError("lora_kv_append", status)


def lora_kv_read(slots: torch.Tensor, cache: torch.Tensor, k_out: Optional[torch.Tensor],
                 v_out: Optional[torch.Tensor], stream: Optional[torch.cuda.Stream] = None,
                 page_size: Optional[int] = None) -> None:
    """What the cache holds at slots (int64 [tokens]); k_out, v_out: bf16 [tokens,
    kv_heads, head_dim], one of them may be None."""
    like = k_out if k_out is not None else v_out
    if like is None:
        raise ValueError("lora_kv_read needs k_out or v_out")
    T, heads, head_dim = _dims(like, 3, "k_out and v_out")
    pc, pages, kv_heads, page_size = _cache(cache, head_dim, page_size)
    pk = ldk = pv = ldv = 0
    if k_out is not None:
        pk, ldk = _heads(k_out, T, kv_heads, head_dim, "k_out")
    if v_out is not None:
        pv, ldv = _heads(v_out, T, kv_heads, head_dim, "v_out")
    status = _kv_read(
        _vector(slots, _I64T, T, "slots"), T, kv_heads, head_dim, pc, pages, page_size, pk, ldk, pv,
        ldv, _stream_handle(stream))
    if status:
        raise LoraError("lora_kv_read", status)


def lora_kv_attention_workspace_bytes(num_seqs: int, max_query_len: int, max_seq_len: int,
                                      q_heads: int, kv_heads: int, head_dim: int) -> int:
    _fit(num_seqs=num_seqs, max_query_len=max_query_len, max_seq_len=max_seq_len, q_heads=q_heads,
         kv_heads=kv_heads, head_dim=head_dim)
    return int(lib().lora_kv_attention_workspace_bytes(num_seqs, max_query_len, max_seq_len, q_heads,
                                                       kv_heads, head_dim))


def kv_attention_workspace(num_seqs: int, max_query_len: int, max_seq_len: int, q_heads: int,
                           kv_heads: int, head_dim: int, device="cuda") -> Optional[torch.Tensor]:
    """A workspace for lora_kv_attention, reused call after call (one stream at a
    time); None where the sizes need none."""
    n = lora_kv_attention_workspace_bytes(num_seqs, max_query_len, max_seq_len, q_heads, kv_heads,
                                          head_dim)
    return torch.empty(n, dtype=torch.uint8, device=device) if n else None


def lora_kv_attention(q: torch.Tensor, query_start: torch.Tensor, seq_lens: torch.Tensor,
                      page_table: torch.Tensor, cache: torch.Tensor, out: torch.Tensor,
                      scale: float, workspace: Optional[torch.Tensor], max_query_len: int,
                      window: int = 0, max_seq_len: Optional[int] = None,
                      stream: Optional[torch.cuda.Stream] = None,
                      page_size: Optional[int] = None) -> None:
    """q, out: bf16 [tokens, q_heads, head_dim]; query_start: int32 [num_seqs + 1];
    seq_lens: int32 [num_seqs]; page_table: int32 [num_seqs, pages a sequence];
    max_seq_len: None: all that the page table can hold; workspace: of
    kv_attention_workspace for these sizes (that max_seq_len among them)."""
    T, q_heads, head_dim = _dims(q, 3, "q")
    pq, ldq = _heads(q, T, q_heads, head_dim, "q")
    po, ldo = _heads(out, T, q_heads, head_dim, "out")
    pc, pages, kv_heads, page_size = _cache(cache, head_dim, page_size)
    B, per_seq = _dims(page_table, 2, "page_table")
    pt, ldt = _matrix(page_table, _I32T, B, per_seq, "page_table")
    if max_seq_len is None:
        max_seq_len = per_seq * page_size
    elif not 1 <= max_seq_len <= per_seq * page_size:
        raise ValueError(f"max_seq_len {max_seq_len} is not within the page table's "
                         f"{per_seq * page_size} tokens")
    if not (-_MOST <= window <= _MOST and -_MOST <= max_query_len <= _MOST and max_seq_len <= _MOST):
        _fit(window=window, max_query_len=max_query_len, max_seq_len=max_seq_len)
    wptr, wbytes = (0, 0) if workspace is None else _flat_dev_bytes(workspace, "workspace")
    status = _kv_attention(
        pq, ldq, _vector(query_start, _I32T, B + 1, "query_start"),
        _vector(seq_lens, _I32T, B, "seq_lens"), pt, ldt, pc, pages, page_size, T, B, max_query_len,
        max_seq_len, q_heads, kv_heads, head_dim, scale, window, po, ldo, wptr, wbytes,
        _stream_handle(stream))
    if status:
        raise LoraError("lora_kv_attention", status)
