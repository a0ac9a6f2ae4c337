"""Calls that write the paged latent cache and summarise it.

``mla_append_kvcache`` turns a step's new tokens into cache rows (norm, position rotation, 16-bit or
"FP8 with scale" rows) and rotates the queries in the same pass; ``mla_summarize_pages`` keeps the
8-bit page keys that page selection scores.  Formulas and errors: ``include/mla_decode.h``.
"""
from __future__ import annotations

import torch

from . import _lib


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
    st = _lib.binding().append(latent, k_pe, positions, cos_sin, slots, kvcache, norm_weight, norm_eps, q_pe, q,
                               bool(interleaved), bool(is_fp8_kvcache), status)
    if st:
        _lib.check(st, "mla_append_kvcache")


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
    st = _lib.binding().summarize(kvcache, block_table, prev_seqlens, cache_seqlens, page_keys, page_scales, bool(is_fp8_kvcache),
                                  status)
    if st:
        _lib.check(st, "mla_summarize_pages")
