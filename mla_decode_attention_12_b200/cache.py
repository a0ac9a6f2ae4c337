"""Calls that write the paged latent cache and summarise it.

``mla_append_kvcache`` turns a step's new tokens into cache rows (norm, position rotation, 16-bit or
"FP8 with scale" rows) and rotates the queries in the same pass; ``mla_summarize_pages`` keeps the
8-bit page keys that page selection scores.  Formulas and errors: ``include/mla_decode.h``.
"""
from __future__ import annotations

import torch

from . import _lib
from .api import _DTYPES, FP8_ROW_BYTES, MLA_BF16_FP8KV, _ptr, _stream


def _cache_dtype(kvcache: torch.Tensor, is_fp8_kvcache: bool) -> tuple[int, int]:
    """(dtype code, d_qk) of a contiguous cache on a CUDA device."""
    if not kvcache.is_cuda or not kvcache.is_contiguous() or kvcache.dim() != 4:
        raise ValueError("kvcache must be a contiguous CUDA tensor [num_blocks, 64, h_kv, row]")
    if is_fp8_kvcache:
        if kvcache.dtype != torch.uint8 or kvcache.shape[-1] != FP8_ROW_BYTES:
            raise ValueError("an FP8 cache is a uint8 kvcache of 656-byte rows")
        return MLA_BF16_FP8KV, 576
    if kvcache.dtype not in _DTYPES:
        raise ValueError("kvcache must be bfloat16 or float16 (or uint8 with is_fp8_kvcache)")
    return _DTYPES[kvcache.dtype], kvcache.shape[-1]


def _check_ints(dev: torch.device, **tensors) -> None:
    for name, (t, dim) in tensors.items():
        if t.dtype != torch.int32 or t.dim() != dim or not t.is_contiguous() or t.device != dev:
            raise ValueError(f"{name} must be a contiguous int32 tensor of {dim} dimension(s) on {dev}")


def _check_status(status: torch.Tensor | None, dev: torch.device) -> None:
    if status is not None and (status.dtype != torch.int32 or status.numel() != 1 or status.device != dev):
        raise ValueError(f"status must be an int32 tensor of one value on {dev}")


def _stride(t: torch.Tensor, dim: int) -> int:
    """Stride of a dimension, 0 where it has one entry (and its stride says nothing)."""
    return t.stride(dim) if t.shape[dim] > 1 else 0


def mla_append_kvcache(latent: torch.Tensor, k_pe: torch.Tensor | None, positions: torch.Tensor | None,
                       cos_sin: torch.Tensor | None, slots: torch.Tensor, kvcache: torch.Tensor, *,
                       norm_weight: torch.Tensor | None = None, norm_eps: float = 1e-6,
                       q_pe: torch.Tensor | None = None, q: torch.Tensor | None = None, interleaved: bool = True,
                       is_fp8_kvcache: bool = False, status: torch.Tensor | None = None) -> None:
    """Write new tokens' rows into the paged cache, and rotate the queries' position columns.

    ``latent`` [tokens, 512] and ``k_pe`` [tokens, 64] (rows may be strided: slices of one projection's
    output); ``positions`` int32 [tokens]; ``cos_sin`` float32 [max_position, 64] (32 cosines, then 32
    sines); ``slots`` int32 [tokens] flat cache rows (page * 64 + offset, negative: padding, not
    written; distinct).  ``norm_weight`` [512]: the latent is RMS-normalised with ``norm_eps`` first.
    ``kvcache`` [num_blocks, 64, 1, 576] of the inputs' type, or uint8 [num_blocks, 64, 1, 656] with
    ``is_fp8_kvcache`` (bfloat16 inputs; quantized per 128 latent columns from the float32 norm), or
    [num_blocks, 64, 1, 512] with neither position columns nor queries.

    ``q_pe`` [tokens, h_q, 64] with ``q`` [tokens, h_q, 576]: ``q[..., 512:]`` receives the rotated
    ``q_pe`` (which may be that slice itself).  ``interleaved``: a pair is columns (2 i, 2 i + 1), else
    (i, i + 32).  ``status`` int32 [1]: receives a device-side error (a slot outside the cache or a
    position outside the table; such a token is skipped).
    """
    dtype, d_qk = _cache_dtype(kvcache, is_fp8_kvcache)
    dev = kvcache.device
    dt = torch.bfloat16 if is_fp8_kvcache else kvcache.dtype
    num_blocks, page, h_kv, _ = kvcache.shape
    if slots.dim() != 1:
        raise ValueError("slots must be int32 [tokens]")
    tokens = slots.shape[0]
    rope = d_qk == 576
    _check_ints(dev, slots=(slots, 1))
    _check_status(status, dev)

    def rows(name, t, shape):
        if t.dtype != dt or t.device != dev or tuple(t.shape) != shape:
            raise ValueError(f"{name} must be {dt} {list(shape)} on {dev}")
        if shape[-1] > 1 and t.stride(-1) != 1:
            raise ValueError(f"{name}: the last dimension must be contiguous")

    rows("latent", latent, (tokens, 512))
    if norm_weight is not None:
        rows("norm_weight", norm_weight, (512,))
    if rope:
        if k_pe is None or positions is None or cos_sin is None:
            raise ValueError("rows of 576 need k_pe, positions and cos_sin")
        rows("k_pe", k_pe, (tokens, 64))
        _check_ints(dev, positions=(positions, 1))
        if positions.shape[0] != tokens:
            raise ValueError("positions must be int32 [tokens]")
        if cos_sin.dtype != torch.float32 or cos_sin.dim() != 2 or cos_sin.shape[1] != 64 or not cos_sin.is_contiguous() \
                or cos_sin.device != dev:
            raise ValueError(f"cos_sin must be contiguous float32 [max_position, 64] on {dev}")
    elif k_pe is not None or q_pe is not None or q is not None:
        raise ValueError("rows of 512 have no position columns")
    if (q_pe is None) != (q is None):
        raise ValueError("q_pe and q come together")
    h_q, qs = 0, (0, 0, 0, 0)
    if q is not None:
        if q.dim() != 3:
            raise ValueError("q must be [tokens, h_q, 576]")
        h_q = q.shape[1]
        rows("q", q, (tokens, h_q, 576))
        rows("q_pe", q_pe, (tokens, h_q, 64))
        if h_q == 0:
            raise ValueError("q must have at least one head")
        qs = (_stride(q_pe, 0), _stride(q_pe, 1), _stride(q, 0), _stride(q, 1))
    if tokens == 0:
        return
    with torch.cuda.device(dev):
        _lib.check(_lib.load().mla_append_kvcache(
            _ptr(latent), _stride(latent, 0), _ptr(k_pe), _stride(k_pe, 0) if rope else 0, _ptr(norm_weight), float(norm_eps),
            _ptr(positions) if rope else None, _ptr(cos_sin) if rope else None, cos_sin.shape[0] if rope else 0, _ptr(slots),
            tokens, _ptr(kvcache), num_blocks, page, h_kv, d_qk, dtype, int(bool(interleaved)), _ptr(q_pe), qs[0], qs[1],
            _ptr(q), qs[2], qs[3], h_q, _ptr(status), _stream(dev)), "mla_append_kvcache")


def mla_summarize_pages(kvcache: torch.Tensor, block_table: torch.Tensor, prev_seqlens: torch.Tensor,
                        cache_seqlens: torch.Tensor, page_keys: torch.Tensor, page_scales: torch.Tensor, *,
                        is_fp8_kvcache: bool = False, status: torch.Tensor | None = None) -> None:
    """Keep the page keys of the pages that a step completed (each request's cache grew from
    ``prev_seqlens`` to ``cache_seqlens`` tokens, int32 [batch]).

    ``page_keys`` int8 [num_blocks, d_qk] and ``page_scales`` float32 [num_blocks] are indexed by
    physical page; keys of other pages are left as they were.  A page's key is the mean of its 64
    rows in units of ``max |mean| / 127``.  ``status`` int32 [1]: receives a device-side error (a
    block-table entry outside the cache, a length beyond the table).
    """
    dtype, d_qk = _cache_dtype(kvcache, is_fp8_kvcache)
    dev = kvcache.device
    num_blocks, page, h_kv, _ = kvcache.shape
    _check_ints(dev, block_table=(block_table, 2), prev_seqlens=(prev_seqlens, 1), cache_seqlens=(cache_seqlens, 1))
    _check_status(status, dev)
    batch = cache_seqlens.shape[0]
    if block_table.shape[0] != batch or prev_seqlens.shape[0] != batch:
        raise ValueError("inconsistent shapes")
    check_page_keys(page_keys, page_scales, num_blocks, d_qk, dev)
    if batch == 0 or block_table.shape[1] == 0:
        return
    with torch.cuda.device(dev):
        _lib.check(_lib.load().mla_summarize_pages(
            _ptr(kvcache), num_blocks, page, h_kv, d_qk, dtype, _ptr(block_table), block_table.shape[1], _ptr(prev_seqlens),
            _ptr(cache_seqlens), batch, _ptr(page_keys), _ptr(page_scales), _ptr(status), _stream(dev)),
            "mla_summarize_pages")


def check_page_keys(page_keys, page_scales, num_blocks: int, d_qk: int, dev: torch.device) -> None:
    if page_keys.dtype != torch.int8 or tuple(page_keys.shape) != (num_blocks, d_qk) or not page_keys.is_contiguous() \
            or page_keys.device != dev:
        raise ValueError(f"page_keys must be contiguous int8 [{num_blocks}, {d_qk}] on {dev}")
    if page_scales.dtype != torch.float32 or tuple(page_scales.shape) != (num_blocks,) or not page_scales.is_contiguous() \
            or page_scales.device != dev:
        raise ValueError(f"page_scales must be contiguous float32 [{num_blocks}] on {dev}")
