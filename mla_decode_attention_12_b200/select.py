"""Block-sparse decoding: pages chosen for each query token by a cheap score of their 8-bit keys.

``mla_select_pages`` scores the keys that ``mla_summarize_pages`` keeps and returns each token's pages as
a block table; ``flash_mla_page_sparse`` decodes over them.  Formulas: ``include/mla_decode.h``.
"""
from __future__ import annotations

import torch

from . import _lib
from .api import DecodeCall, get_mla_metadata


def mla_select_pages(q: torch.Tensor, page_keys: torch.Tensor, page_scales: torch.Tensor, block_table: torch.Tensor,
                     cache_seqlens: torch.Tensor, topn: int, *, n_first: int = 1, n_last: int = 1, causal: bool = True,
                     status: torch.Tensor | None = None):
    """The ``topn`` best pages of each query token; ``(page_table int32 [b * s_q, topn], page_seqlens int32 [b * s_q])``.

    ``q`` [b, s_q, h_q, d_qk] bf16 or fp16 (at most 128 heads); ``page_keys`` int8 [num_blocks, d_qk] and
    ``page_scales`` float32 [num_blocks]; ``block_table`` int32 [b, max_blocks]; ``cache_seqlens`` int32 [b].
    Token s of a request sees ``L - s_q + 1 + s`` cached rows (``causal``), or all L.  A page's score is
    the largest over heads of the 8-bit query times the key; the first ``n_first`` and the last ``n_last``
    (at least one: it may be partly filled) pages are always in, equal scores go to the lower page.
    Rows of ``page_table`` list physical pages in ascending order of their place in the sequence, then -1:
    a block table for ``flash_mla_with_kvcache`` with one request per token and ``page_seqlens`` as its
    lengths.  ``status`` int32 [1]: receives a device-side error.
    """
    st, table, lens = _lib.binding().select(q, page_keys, page_scales, block_table, cache_seqlens, topn, n_first, n_last,
                                            bool(causal), status)
    if st:
        _lib.check(st, "mla_select_pages")
    return table, lens


def flash_mla_page_sparse(q: torch.Tensor, kvcache: torch.Tensor, block_table: torch.Tensor, cache_seqlens: torch.Tensor,
                          dv: int, page_keys: torch.Tensor, page_scales: torch.Tensor, topn: int, *, n_first: int = 1,
                          n_last: int = 1, causal: bool = True, is_fp8_kvcache: bool = False,
                          softmax_scale: float | None = None, workspace: torch.Tensor | None = None,
                          status: torch.Tensor | None = None):
    """MLA decode over the ``topn`` pages that score best for each query token; ``(o [b, s_q, h_q, dv], lse [b, s_q, h_q])``.

    The selection of ``mla_select_pages`` (with the same arguments), then the paged decode over it; a
    token that sees at most ``topn`` pages attends all of them.  ``kvcache`` and ``is_fp8_kvcache`` as for
    ``flash_mla_with_kvcache``; the lse is that of the attended rows.  ``status`` int32 [1]: receives a
    device-side error of the selection or the decode (without it, the decode's goes to the workspace).
    """
    table, lens = mla_select_pages(q, page_keys, page_scales, block_table, cache_seqlens, topn, n_first=n_first, n_last=n_last,
                                   causal=causal, status=status)
    b, s_q, h_q, d_qk = q.shape
    md, num_splits = get_mla_metadata(lens, h_q, 1, is_fp8_kvcache=is_fp8_kvcache)
    o, lse = DecodeCall(q.view(b * s_q, 1, h_q, d_qk), kvcache, table, lens, dv, md, num_splits, is_fp8_kvcache=is_fp8_kvcache,
                        softmax_scale=softmax_scale, workspace=workspace, status=status).run()
    return o.view(b, s_q, h_q, dv), lse.view(b, s_q, h_q)
