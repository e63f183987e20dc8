"""Drafted tokens and caches of bounded length (``include/lora_cache.h``): trees of
drafted tokens and attention for them over the 4-bit paged cache, the weight that each
cached token draws, the choice of the tokens that a cache keeps, and their move.

As in the rest of the binding, the functions carry the C entry points' names and
only marshal arguments: shapes and strides come from the tensors, the stream is
the current one unless given, and every step runs in the library's HIP kernels.
"""

from __future__ import annotations

import ctypes
from typing import Optional

import torch

from . import LoraError, _dev_ptr, _flat_dev_bytes, _stream_handle, lib
from .attention import (_F32, _I32, _I32T, _I64, _I64T, _MOST, _VP, SUPPORTED_PAGE_SIZES, _cache, _dims, _fit,
                        _heads, _matrix, _vector)

__all__ = [
    "lora_draft_masks", "lora_kv_tree_attention", "lora_kv_tree_attention_workspace_bytes",
    "kv_tree_attention_workspace", "lora_kv_attention_mass", "lora_kv_select",
    "lora_kv_select_workspace_bytes", "kv_select_workspace", "lora_kv_compact",
    "kv_mass_shape", "LORA_MAX_MASK_WORDS",
]

LORA_MAX_MASK_WORDS = 8


def _declare(L: ctypes.CDLL) -> None:
    """Argument types of the entry points, on the loaded library."""
    step = [_VP, _VP, _VP, _I64, _VP, _I32, _I32, _I32, _I32, _I32, _I32, _I32, _I32, _I32,
            ctypes.c_float, _I32, _VP, _I32]  # from query_start to mask_words
    L.lora_draft_masks.argtypes = [_VP, _VP, _I32, _I32, _VP, _I32, _VP, _VP, _VP]
    L.lora_kv_tree_attention_workspace_bytes.argtypes = [_I32] * 6
    L.lora_kv_tree_attention_workspace_bytes.restype = _I64
    L.lora_kv_tree_attention.argtypes = [_VP, _I64, *step, _VP, _I64, _VP, _I64, _VP, _I64, _VP]
    L.lora_kv_attention_mass.argtypes = [_VP, _I64, _VP, _I64, *step, _VP, _VP]
    L.lora_kv_select.argtypes = [_VP, _I32, _I32, _VP, _VP, _I64, _I32, _I32, _I32, _I32, _I32, _VP, _I32,
                                 _VP, _VP, _I64, _VP]
    L.lora_kv_select_workspace_bytes.argtypes = [_I32] * 3
    L.lora_kv_select_workspace_bytes.restype = _I64
    L.lora_kv_compact.argtypes = [_VP, _I32, _I32, _VP, _VP, _VP, _I64, _I32, _VP, _I64, _I32, _VP, _I32,
                                  _I32, _I32, _I32, _I32, _VP, _VP]
    for f in (L.lora_draft_masks, L.lora_kv_tree_attention, L.lora_kv_attention_mass, L.lora_kv_select,
              L.lora_kv_compact):
        f.restype = ctypes.c_int


_declare(lib())
_draft_masks, _tree_attention = lib().lora_draft_masks, lib().lora_kv_tree_attention
_attention_mass, _select, _compact = lib().lora_kv_attention_mass, lib().lora_kv_select, lib().lora_kv_compact
_select_bytes = lib().lora_kv_select_workspace_bytes


def _current_device() -> int:
    return torch._C._cuda_getDevice()


# Of a process that has a single device, one tensor says what there is to say (each of
# the others costs 0.1 us of a call that takes 8).
_SEVERAL_DEVICES = torch.cuda.device_count() > 1


def _stream_for(stream: Optional[torch.cuda.Stream], t: torch.Tensor, *others: Optional[torch.Tensor]) -> int:
    """The stream's handle; refuses a call that has a tensor on another device than it."""
    device = _current_device() if stream is None else stream.device_index
    if t.get_device() != device or _SEVERAL_DEVICES and any(o is not None and o.get_device() != device for o in others):
        on = sorted({o.get_device() for o in (t, *others) if o is not None})
        raise ValueError(f"the tensors are on devices {on}, the stream is device {device}'s")
    return _stream_handle(stream)


def kv_mass_shape(num_pages: int, kv_heads: int, page_size: int):
    """Shape of the fp32 mass beside a cache: [num_pages, kv_heads, page_size]."""
    if page_size not in SUPPORTED_PAGE_SIZES:
        raise ValueError(f"page_size is one of {SUPPORTED_PAGE_SIZES}")
    return (int(num_pages), int(kv_heads), int(page_size))


def _whole(t: torch.Tensor, dtype: torch.dtype, shape, name: str) -> int:
    """Address of a contiguous tensor of this shape."""
    ptr = _dev_ptr(t, dtype, name)
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, is {list(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous, has strides {t.stride()}")
    return ptr


def _words(masks: torch.Tensor, tokens: int):
    words = _dims(masks, 2, "masks")[1]
    if not words:  # no address either: the library would take them for none at all
        raise ValueError("masks have no words")
    return _whole(masks, _I64T, (tokens, words), "masks"), words


def lora_draft_masks(parents: torch.Tensor, query_start: torch.Tensor, masks: Optional[torch.Tensor] = None,
                     positions: Optional[torch.Tensor] = None, first_positions: Optional[torch.Tensor] = None,
                     stream: Optional[torch.cuda.Stream] = None) -> None:
    """parents: int32 [tokens], the parent's number in its sequence, -1 for a root;
    query_start: int32 [num_seqs + 1]; masks: int64 [tokens, words], which drafted tokens
    each one descends from (itself among them); positions: int32 [tokens], the depth in
    the tree from first_positions (int32 [num_seqs], or None: 0) on.  One of masks and
    positions may be left out."""
    T = _dims(parents, 1, "parents")[0]
    B = _dims(query_start, 1, "query_start")[0] - 1
    pm, words = _words(masks, T) if masks is not None else (0, LORA_MAX_MASK_WORDS)
    pp = _vector(positions, _I32T, T, "positions") if positions is not None else 0
    pf = _vector(first_positions, _I32T, B, "first_positions") if first_positions is not None else 0
    status = _draft_masks(_vector(parents, _I32T, T, "parents"), _vector(query_start, _I32T, B + 1, "query_start"),
                          T, B, pm, words, pf, pp,
                          _stream_for(stream, parents, query_start, masks, positions, first_positions))
    if status:
        raise LoraError("lora_draft_masks", status)


def lora_kv_tree_attention_workspace_bytes(num_seqs: int, max_query_len: int, max_seq_len: int, q_heads: int,
                                           kv_heads: int, head_dim: int) -> int:
    _fit(num_seqs=num_seqs, max_query_len=max_query_len, max_seq_len=max_seq_len, q_heads=q_heads,
         kv_heads=kv_heads, head_dim=head_dim)
    return int(lib().lora_kv_tree_attention_workspace_bytes(num_seqs, max_query_len, max_seq_len, q_heads,
                                                            kv_heads, head_dim))


def kv_tree_attention_workspace(num_seqs: int, max_query_len: int, max_seq_len: int, q_heads: int,
                                kv_heads: int, head_dim: int, device="cuda") -> Optional[torch.Tensor]:
    """A workspace for lora_kv_tree_attention, reused call after call (one stream at a
    time); None where the sizes need none."""
    n = lora_kv_tree_attention_workspace_bytes(num_seqs, max_query_len, max_seq_len, q_heads, kv_heads, head_dim)
    return torch.empty(n, dtype=torch.uint8, device=device) if n else None


def _step(query_start, seq_lens, page_table, page_size, max_seq_len, max_query_len, window):
    """(num_seqs, max_seq_len, and the addresses of the three)."""
    B, per_seq = _dims(page_table, 2, "page_table")
    pt, ldt = _matrix(page_table, _I32T, B, per_seq, "page_table")
    if max_seq_len is None:
        max_seq_len = per_seq * page_size
    elif not 1 <= max_seq_len <= per_seq * page_size:
        raise ValueError(f"max_seq_len {max_seq_len} is not within the page table's "
                         f"{per_seq * page_size} tokens")
    if not (-_MOST <= window <= _MOST and -_MOST <= max_query_len <= _MOST and max_seq_len <= _MOST):
        _fit(window=window, max_query_len=max_query_len, max_seq_len=max_seq_len)
    ps = _vector(query_start, _I32T, B + 1, "query_start") if query_start is not None else 0
    return B, max_seq_len, ps, _vector(seq_lens, _I32T, B, "seq_lens"), pt, ldt


def lora_kv_tree_attention(q: torch.Tensor, query_start: torch.Tensor, seq_lens: torch.Tensor,
                           page_table: torch.Tensor, cache: torch.Tensor, out: torch.Tensor, scale: float,
                           masks: Optional[torch.Tensor], workspace: Optional[torch.Tensor],
                           max_query_len: int, window: int = 0, max_seq_len: Optional[int] = None,
                           lse: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None,
                           page_size: Optional[int] = None) -> None:
    """Arguments as for lora_kv_attention, and masks: int64 [tokens, words] of
    lora_draft_masks, or None: each query sees the tokens up to its own; lse: fp32
    [tokens, q_heads], the logarithms of the rows' sums, or None; workspace: of
    kv_tree_attention_workspace for these sizes."""
    T, q_heads, head_dim = _dims(q, 3, "q")
    pq, ldq = _heads(q, T, q_heads, head_dim, "q")
    po, ldo = _heads(out, T, q_heads, head_dim, "out")
    pc, pages, kv_heads, page_size = _cache(cache, head_dim, page_size)
    B, max_seq_len, ps, pn, pt, ldt = _step(query_start, seq_lens, page_table, page_size, max_seq_len,
                                            max_query_len, window)
    pm, words = _words(masks, T) if masks is not None else (0, 0)
    pl, ldl = _matrix(lse, _F32, T, q_heads, "lse") if lse is not None else (0, 0)
    wptr, wbytes = (0, 0) if workspace is None else _flat_dev_bytes(workspace, "workspace")
    status = _tree_attention(
        pq, ldq, ps, pn, pt, ldt, pc, pages, page_size, T, B, max_query_len, max_seq_len, q_heads, kv_heads,
        head_dim, scale, window, pm, words, po, ldo, pl, ldl, wptr, wbytes,
        _stream_for(stream, q, query_start, seq_lens, page_table, cache, out, masks, lse, workspace))
    if status:
        raise LoraError("lora_kv_tree_attention", status)


def lora_kv_attention_mass(q: torch.Tensor, lse: torch.Tensor, query_start: torch.Tensor,
                           seq_lens: torch.Tensor, page_table: torch.Tensor, cache: torch.Tensor,
                           mass: torch.Tensor, scale: float, masks: Optional[torch.Tensor], max_query_len: int,
                           window: int = 0, max_seq_len: Optional[int] = None,
                           stream: Optional[torch.cuda.Stream] = None, page_size: Optional[int] = None) -> None:
    """The arguments of the lora_kv_tree_attention that wrote lse, and mass: fp32
    (kv_mass_shape), to which the attention that the tokens drew is added; that of
    the step's own tokens is put there.  Rows whose lse is -infinity count for nothing:
    those of rejected drafts are set so, before lora_kv_compact moves the others."""
    T, q_heads, head_dim = _dims(q, 3, "q")
    pq, ldq = _heads(q, T, q_heads, head_dim, "q")
    pl, ldl = _matrix(lse, _F32, T, q_heads, "lse")
    pc, pages, kv_heads, page_size = _cache(cache, head_dim, page_size)
    B, max_seq_len, ps, pn, pt, ldt = _step(query_start, seq_lens, page_table, page_size, max_seq_len,
                                            max_query_len, window)
    pm, words = _words(masks, T) if masks is not None else (0, 0)
    status = _attention_mass(
        pq, ldq, pl, ldl, ps, pn, pt, ldt, pc, pages, page_size, T, B, max_query_len, max_seq_len, q_heads,
        kv_heads, head_dim, scale, window, pm, words, _whole(mass, _F32, (pages, kv_heads, page_size), "mass"),
        _stream_for(stream, q, lse, query_start, seq_lens, page_table, cache, mass, masks))
    if status:
        raise LoraError("lora_kv_attention_mass", status)


def lora_kv_select_workspace_bytes(num_seqs: int, kv_heads: int, max_seq_len: int) -> int:
    _fit(num_seqs=num_seqs, kv_heads=kv_heads, max_seq_len=max_seq_len)
    return int(lib().lora_kv_select_workspace_bytes(num_seqs, kv_heads, max_seq_len))


def kv_select_workspace(num_seqs: int, kv_heads: int, max_seq_len: int, device="cuda") -> Optional[torch.Tensor]:
    """A workspace for lora_kv_select, reused call after call (one stream at a time);
    None where the sizes need none."""
    n = lora_kv_select_workspace_bytes(num_seqs, kv_heads, max_seq_len)
    return torch.empty(n, dtype=torch.uint8, device=device) if n else None


def lora_kv_select(mass: torch.Tensor, seq_lens: torch.Tensor, page_table: torch.Tensor, sinks: int, recent: int,
                   kept: torch.Tensor, new_lens: torch.Tensor, max_seq_len: Optional[int] = None,
                   stream: Optional[torch.cuda.Stream] = None, workspace: Optional[torch.Tensor] = None) -> None:
    """mass: fp32 (kv_mass_shape); kept: int32 [num_seqs, kv_heads, budget], each key
    head's tokens, ascending, -1 past the last; new_lens: int32 [num_seqs].  Kept are the
    first sinks tokens, the last recent and the heaviest of the others; workspace: of
    kv_select_workspace for these sizes, or None: one from torch's allocator."""
    pages, kv_heads, page_size = _dims(mass, 3, "mass")
    budget = _dims(kept, 3, "kept")[2]
    B, max_seq_len, _, pn, pt, ldt = _step(None, seq_lens, page_table, page_size, max_seq_len, 1, 0)
    _fit(sinks=sinks, recent=recent, budget=budget, pages=pages)
    handle = _stream_for(stream, mass, seq_lens, page_table, kept, new_lens, workspace)
    if workspace is None and max_seq_len > 0:
        need = _select_bytes(B, kv_heads, max_seq_len)
        if need:
            with torch.cuda.stream(stream):  # whose later work alone may be given it again
                workspace = torch.empty(need, dtype=torch.uint8, device=mass.device)
    wptr, wbytes = (0, 0) if workspace is None else _flat_dev_bytes(workspace, "workspace")
    status = _select(
        _whole(mass, _F32, (pages, kv_heads, page_size), "mass"), pages, page_size, pn, pt, ldt, B, kv_heads,
        max_seq_len, sinks, recent, _whole(kept, _I32T, (B, kv_heads, budget), "kept"), budget,
        _vector(new_lens, _I32T, B, "new_lens"), wptr, wbytes, handle)
    if status:
        raise LoraError("lora_kv_select", status)


def lora_kv_compact(kept: torch.Tensor, counts: torch.Tensor, page_table: torch.Tensor, cache: torch.Tensor,
                    head_dim: int, mass: Optional[torch.Tensor] = None, first: Optional[torch.Tensor] = None,
                    dst_table: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None,
                    page_size: Optional[int] = None) -> None:
    """kept: int32 [num_seqs, kv_heads or 1, n]: of each sequence, and key head (or all
    of them), the tokens that move to the places first + 0, first + 1, ..., counted from
    first (int32 [num_seqs], or None: 0), in place each above the one before; counts: int32 [num_seqs], how many of the n;
    page_table, dst_table: int32 [num_seqs, pages a sequence], where they are and where
    they go (None: in place; other pages than those); mass: fp32 (kv_mass_shape), moved
    along."""
    B, lists, n = _dims(kept, 3, "kept")
    pc, pages, kv_heads, page_size = _cache(cache, head_dim, page_size)
    per_seq = _dims(page_table, 2, "page_table")[1]
    pt, ldt = _matrix(page_table, _I32T, B, per_seq, "page_table")
    pd = ldd = per_dst = 0
    if dst_table is not None:
        per_dst = _dims(dst_table, 2, "dst_table")[1]
        pd, ldd = _matrix(dst_table, _I32T, B, per_dst, "dst_table")
        if B and not per_dst:
            raise ValueError("dst_table holds no pages")
    pm = _whole(mass, _F32, (pages, kv_heads, page_size), "mass") if mass is not None else 0
    pf = _vector(first, _I32T, B, "first") if first is not None else 0
    status = _compact(
        _whole(kept, _I32T, (B, lists, n), "kept"), lists, n, _vector(counts, _I32T, B, "counts"), pf, pt, ldt,
        per_seq, pd, ldd, per_dst, pc, pages, page_size, B, kv_heads, head_dim, pm,
        _stream_for(stream, cache, kept, counts, page_table, mass, first, dst_table))
    if status:
        raise LoraError("lora_kv_compact", status)
