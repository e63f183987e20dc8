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


from . import (_check, _dev_ptr, _flat_dev_bytes, _stream_handle, lib)  # noqa: E402

_declare(lib())


def _rows(t: torch.Tensor, name: str, dtype=torch.bfloat16, width: Optional[int] = None,
          tokens: Optional[int] = None) -> Tuple[int, int]:
    """Address and row stride of a [tokens, width] matrix with unit column stride."""
    ptr = _dev_ptr(t, dtype, name)
    if t.dim() != 2 or (t.shape[1] > 1 and t.stride(1) != 1):
        raise ValueError(f"{name} must be 2-D with unit column stride")
    if width is not None and t.shape[1] != width:
        raise ValueError(f"{name} must be {width} wide, is {t.shape[1]}")
    if tokens is not None and t.shape[0] != tokens:
        raise ValueError(f"{name} must have {tokens} rows, has {t.shape[0]}")
    return ptr, _stride(t)


def _stride(t: torch.Tensor) -> int:
    # a single row's stride is never used for an address: any value that passes will do
    return int(t.stride(0)) if t.shape[0] > 1 else _width(t)


def _width(t: torch.Tensor) -> int:
    n = 1
    for s in t.shape[1:]:
        n *= int(s)
    return n


def _heads(t: torch.Tensor, name: str, tokens: Optional[int] = None,
           heads: Optional[int] = None, head_dim: Optional[int] = None) -> Tuple[int, int]:
    """Address and row stride of a bf16 [tokens, heads, head_dim] tensor whose
    heads lie one behind another."""
    ptr = _dev_ptr(t, torch.bfloat16, name)
    if t.dim() != 3 or t.stride(2) != 1 or (t.shape[1] > 1 and t.stride(1) != t.shape[2]):
        raise ValueError(f"{name} must be [tokens, heads, head_dim], each token's heads contiguous")
    if ((tokens is not None and t.shape[0] != tokens) or (heads is not None and t.shape[1] != heads)
            or (head_dim is not None and t.shape[2] != head_dim)):
        raise ValueError(f"{name} must be [{tokens}, {heads}, {head_dim}], is {list(t.shape)}")
    return ptr, _stride(t)


def _vector(t: torch.Tensor, dtype: torch.dtype, name: str, n: int) -> int:
    ptr = _dev_ptr(t, dtype, name)
    if t.dim() != 1 or t.shape[0] != n or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous [{n}]")
    return ptr


def kv_cache_shape(num_pages: int, kv_heads: int, head_dim: int, page_size: int):
    """Shape of the uint8 cache tensor: [num_pages, 2, kv_heads, page_bytes]."""
    if head_dim not in SUPPORTED_HEAD_DIMS or page_size not in SUPPORTED_PAGE_SIZES:
        raise ValueError(f"head_dim is one of {SUPPORTED_HEAD_DIMS} and page_size one of "
                         f"{SUPPORTED_PAGE_SIZES}")
    return (int(num_pages), 2, int(kv_heads), page_size * (head_dim // 2 + head_dim // 32))


def _cache(cache: torch.Tensor, head_dim: int) -> Tuple[int, int, int, int]:
    """Address, pages, kv_heads and page size of a cache for this head_dim."""
    ptr = _dev_ptr(cache, torch.uint8, "cache")
    if cache.dim() != 4 or cache.shape[1] != 2 or not cache.is_contiguous():
        raise ValueError("cache must be contiguous [num_pages, 2, kv_heads, page_bytes]")
    row = head_dim // 2 + head_dim // 32  # bytes of one token's head
    if row < 1 or cache.shape[3] % row:
        raise ValueError(f"cache pages of {cache.shape[3]} bytes hold no heads of {head_dim}")
    return ptr, int(cache.shape[0]), int(cache.shape[2]), int(cache.shape[3]) // row


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
    px, ldx = _rows(x, "x")
    T, hidden = x.shape
    args = {}
    for name, t in (("residual", residual), ("residual_out", residual_out), ("y", y)):
        args[name] = (0, 0) if t is None else _rows(t, name, width=hidden, tokens=T)
    p8, ld8, ps, group = 0, 0, 0, hidden
    if y8 is not None:
        p8, ld8 = _rows(y8, "y8", torch.float8_e4m3fn, hidden, T)
    if scales is not None:
        ps = _dev_ptr(scales, torch.float32, "scales")
        if scales.dim() != 2 or scales.shape[0] != T or not scales.is_contiguous():
            raise ValueError("scales must be contiguous [tokens, groups]")
        if scales.shape[1] < 1 or hidden % scales.shape[1]:
            raise ValueError(f"{scales.shape[1]} scales do not divide a row of {hidden}")
        group = hidden // scales.shape[1]
    _check("lora_rms_norm", lib().lora_rms_norm(
        px, ldx, *args["residual"], _vector(weight, torch.bfloat16, "weight", hidden), float(eps),
        int(T), int(hidden), *args["residual_out"], *args["y"], p8, ld8, ps, group,
        _stream_handle(stream)))


def lora_kv_append(qkv: torch.Tensor, positions: Optional[torch.Tensor], slots: torch.Tensor,
                   rope: Optional[torch.Tensor], cache: torch.Tensor, q_out: torch.Tensor,
                   interleaved: bool = False, stream: Optional[torch.cuda.Stream] = None) -> None:
    """qkv: bf16 [tokens, (q_heads + 2 kv_heads) * head_dim]; positions: int32
    [tokens]; slots: int64 [tokens]; rope: fp32 [rows, rot_dim] (rope_table), or
    None for no rotation; cache: uint8 (kv_cache_shape); q_out: bf16 [tokens,
    q_heads, head_dim]."""
    pq, ldq = _heads(q_out, "q_out")
    T, q_heads, head_dim = q_out.shape
    pc, pages, kv_heads, page_size = _cache(cache, head_dim)
    px, ldx = _rows(qkv, "qkv", width=(q_heads + 2 * kv_heads) * head_dim, tokens=T)
    rows = rot = pr = pp = 0
    if rope is not None:
        pr = _dev_ptr(rope, torch.float32, "rope")
        if rope.dim() != 2 or not rope.is_contiguous():
            raise ValueError("rope must be contiguous [rows, rot_dim]")
        rows, rot = rope.shape
        pp = _vector(positions, torch.int32, "positions", T)
    _check("lora_kv_append", lib().lora_kv_append(
        px, ldx, pp, _vector(slots, torch.int64, "slots", T), pr, rows, rot, int(bool(interleaved)),
        T, q_heads, kv_heads, head_dim, pq, ldq, pc, pages, page_size, _stream_handle(stream)))


def lora_kv_read(slots: torch.Tensor, cache: torch.Tensor, k_out: Optional[torch.Tensor],
                 v_out: Optional[torch.Tensor], stream: Optional[torch.cuda.Stream] = None) -> None:
    """What the cache holds at slots (int64 [tokens]); k_out, v_out: bf16 [tokens,
    kv_heads, head_dim], one of them may be None."""
    like = k_out if k_out is not None else v_out
    if like is None:
        raise ValueError("lora_kv_read needs k_out or v_out")
    if like.dim() != 3:
        raise ValueError("k_out and v_out must be [tokens, kv_heads, head_dim]")
    T, kv_heads, head_dim = like.shape
    pc, pages, heads, page_size = _cache(cache, head_dim)
    outs = []
    for name, t in (("k_out", k_out), ("v_out", v_out)):
        outs += (0, 0) if t is None else _heads(t, name, T, heads, head_dim)
    _check("lora_kv_read", lib().lora_kv_read(
        _vector(slots, torch.int64, "slots", T), T, heads, head_dim, pc, pages, page_size, *outs,
        _stream_handle(stream)))


def lora_kv_attention_workspace_bytes(num_seqs: int, max_query_len: int, max_seq_len: int,
                                      q_heads: int, kv_heads: int, head_dim: int) -> int:
    return int(lib().lora_kv_attention_workspace_bytes(num_seqs, max_query_len, max_seq_len, q_heads,
                                                       kv_heads, head_dim))


def kv_attention_workspace(num_seqs: int, max_query_len: int, max_seq_len: int, q_heads: int,
                           kv_heads: int, head_dim: int, device="cuda") -> Optional[torch.Tensor]:
    """A zero-filled workspace for lora_kv_attention, reused call after call (one
    stream at a time); None where the sizes need none."""
    n = lora_kv_attention_workspace_bytes(num_seqs, max_query_len, max_seq_len, q_heads, kv_heads,
                                          head_dim)
    return torch.zeros(n, dtype=torch.uint8, device=device) if n else None


def lora_kv_attention(q: torch.Tensor, query_start: torch.Tensor, seq_lens: torch.Tensor,
                      page_table: torch.Tensor, cache: torch.Tensor, out: torch.Tensor,
                      scale: float, workspace: Optional[torch.Tensor], max_query_len: int,
                      window: int = 0, max_seq_len: Optional[int] = None,
                      stream: Optional[torch.cuda.Stream] = None) -> None:
    """q, out: bf16 [tokens, q_heads, head_dim]; query_start: int32 [num_seqs + 1];
    seq_lens: int32 [num_seqs]; page_table: int32 [num_seqs, pages a sequence];
    max_seq_len: None: all that the page table can hold; workspace: of
    kv_attention_workspace for these sizes (that max_seq_len among them)."""
    pq, ldq = _heads(q, "q")
    T, q_heads, head_dim = q.shape
    pc, pages, kv_heads, page_size = _cache(cache, head_dim)
    po, ldo = _heads(out, "out", T, q_heads, head_dim)
    pt = _dev_ptr(page_table, torch.int32, "page_table")
    if page_table.dim() != 2 or (page_table.shape[1] > 1 and page_table.stride(1) != 1):
        raise ValueError("page_table must be [num_seqs, pages] with unit column stride")
    B, per_seq = page_table.shape
    if max_seq_len is None:
        max_seq_len = per_seq * page_size
    elif not 1 <= max_seq_len <= per_seq * page_size:
        raise ValueError(f"max_seq_len {max_seq_len} is not within the page table's "
                         f"{per_seq * page_size} tokens")
    wptr, wbytes = (0, 0) if workspace is None else _flat_dev_bytes(workspace, "workspace")
    _check("lora_kv_attention", lib().lora_kv_attention(
        pq, ldq, _vector(query_start, torch.int32, "query_start", B + 1),
        _vector(seq_lens, torch.int32, "seq_lens", B), pt, _stride(page_table), pc, pages, page_size,
        T, B, int(max_query_len), int(max_seq_len), q_heads, kv_heads, head_dim, float(scale),
        int(window), po, ldo, wptr, wbytes, _stream_handle(stream)))
