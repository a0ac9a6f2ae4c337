"""Attention of ragged runs of new tokens (chunks of prompts beside decode steps) over the paged cache.

``get_mla_metadata_varlen`` once per step, then ``flash_mla_varlen_with_kvcache`` once per layer.
Formulas and errors: ``include/mla_decode.h``.
"""
from __future__ import annotations

from typing import NamedTuple

import torch

from . import _lib
from .api import get_workspace, workspace_zero_bytes


class VarlenPlan(NamedTuple):
    """A step's schedule (device memory) and the sizes that it was made for."""
    data: torch.Tensor   # int32, opaque
    batch: int
    total_q: int
    h_q: int
    num_parts: int
    causal: bool


def get_mla_metadata_varlen(cu_seqlens_q: torch.Tensor, cache_seqlens: torch.Tensor, total_q: int, h_q: int,
                            h_kv: int = 1, *, causal: bool = True, is_fp8_kvcache: bool = False,
                            num_parts: int | None = None, out: VarlenPlan | None = None) -> VarlenPlan:
    """Schedule of one step's ragged runs, for every layer of the step.

    ``cu_seqlens_q`` int32 [batch + 1]: run b is the query tokens ``[cu_seqlens_q[b], cu_seqlens_q[b + 1])``
    of ``total_q``; ``cache_seqlens`` int32 [batch]: cached tokens of each request, the run's own included.
    ``out``: a plan of the same sizes, written again (for captured graphs).
    """
    causal = bool(causal)
    if out is not None:
        if (out.batch, out.total_q, out.h_q, out.causal) != (cache_seqlens.numel(), total_q, h_q, causal) or \
                num_parts not in (None, out.num_parts):
            raise ValueError("out is a plan of other sizes")
        num_parts = out.num_parts
    st, parts, data = _lib.binding().varlen_plan(cu_seqlens_q, cache_seqlens, total_q, h_q, h_kv, causal, bool(is_fp8_kvcache),
                                                 num_parts, None if out is None else out.data)
    if st:
        _lib.check(st, "mla_get_metadata_varlen")
    return VarlenPlan(data, cache_seqlens.shape[0], total_q, h_q, parts, causal)


def get_mla_metadata_varlen_host(cu_seqlens_q, cache_seqlens, h_q: int, h_kv: int = 1, *, causal: bool = True,
                                 is_fp8_kvcache: bool = False, num_parts: int = 74):
    """The same schedule on the host (numpy): (md [num_parts, 8], groups [number of groups, 8])."""
    import numpy as np

    cu = np.ascontiguousarray(cu_seqlens_q, dtype=np.int32)
    sl = np.ascontiguousarray(cache_seqlens, dtype=np.int32)
    if cu.size != sl.size + 1:
        raise ValueError("cu_seqlens_q must have one entry more than cache_seqlens")
    total_q = int(cu[-1])
    lib = _lib.load()
    plan = np.zeros(max(1, lib.mla_varlen_plan_ints(sl.size, total_q, h_q, h_kv, num_parts)), np.int32)
    _lib.check(lib.mla_get_metadata_varlen_host(cu.ctypes.data, sl.ctypes.data, sl.size, total_q, h_q, h_kv, int(bool(causal)),
                                                num_parts, int(bool(is_fp8_kvcache)), plan.ctypes.data),
               "mla_get_metadata_varlen_host")
    groups = int(sum(-(-int(n) * h_q // 128) for n in np.diff(cu)))
    return plan[:num_parts * 8].reshape(num_parts, 8), plan[num_parts * 8:num_parts * 8 + groups * 8].reshape(groups, 8)


def varlen_workspace_bytes(num_parts: int) -> int:
    """Workspace of ``flash_mla_varlen_with_kvcache``; its control block must start zeroed (``workspace_zero_bytes``)."""
    n = _lib.load().mla_decode_varlen_workspace_bytes(num_parts)
    if n == 0:
        raise ValueError("invalid number of partitions")
    return n


_varlen_bytes: dict = {}  # workspace size by partition count


def _call_workspace(num_parts: int, dev: torch.device) -> torch.Tensor:
    """The stream's cached workspace; inside a graph capture one of the graph's own."""
    if dev.type != "cuda":
        raise ValueError("q must be on a CUDA device")
    sizes = _varlen_bytes.get(num_parts)
    if sizes is None:
        sizes = _varlen_bytes[num_parts] = (varlen_workspace_bytes(num_parts), workspace_zero_bytes(1, 1, 1, 1))
    return get_workspace(sizes[0], dev, sizes[1])


def flash_mla_varlen_with_kvcache(q: torch.Tensor, kvcache: torch.Tensor, block_table: torch.Tensor,
                                  cu_seqlens_q: torch.Tensor, cache_seqlens: torch.Tensor, dv: int, plan: VarlenPlan,
                                  causal: bool = True, is_fp8_kvcache: bool = False, *, softmax_scale: float | None = None,
                                  workspace: torch.Tensor | None = None, out: torch.Tensor | None = None,
                                  lse: torch.Tensor | None = None, status: torch.Tensor | None = None,
                                  max_scratch_bytes: int | None = None):
    """MLA attention of ragged runs over a paged cache; ``(o [total_q, h_q, dv], lse [total_q, h_q] float32)``.

    ``q`` [total_q, h_q, d_qk]; ``kvcache``, ``block_table`` [batch, max_blocks] and the FP8 cache as for
    ``flash_mla_with_kvcache``.  Token i of a run of n tokens over L cached ones sees the first
    ``L - n + 1 + i`` of them (``causal``), or all L.  ``plan`` comes from ``get_mla_metadata_varlen``
    with the same ``cu_seqlens_q``, ``cache_seqlens`` and ``causal``.  Rows past ``cu_seqlens_q[batch]`` are
    not written (of ``out`` and ``lse`` passed in, they stay as they were).  ``status`` int32 [1]: receives a
    device-side error of the call (a block-table entry outside the cache, a length beyond the table, runs
    that do not split the tokens); without it, the error goes to the workspace.

    Over an FP8 cache, runs of about three groups of 128 query rows and more have their pages dequantized
    once, into 73.7 KB for every entry of the block table (whatever the lengths), allocated for the call: up to
    ``max_scratch_bytes`` (8 GiB, if None).  A call that would need more, or does not get it, reads the FP8 rows
    at every use: slower, with no memory of its own.  Where the memory is known to be missing,
    ``max_scratch_bytes=0`` spares each call the attempt.
    """
    data, batch, total_q, h_q, num_parts, planned_causal = plan
    if q.dim() != 3 or (batch, total_q, h_q, planned_causal) != (cache_seqlens.numel(), q.shape[0], q.shape[1], bool(causal)):
        raise ValueError("the plan was made for another call, or q is not [total_q, h_q, d_qk]")
    if workspace is None:
        workspace = _call_workspace(num_parts, q.device)
    scale = 0.0 if softmax_scale is None else softmax_scale  # 0: 1 / sqrt(d_qk)
    st, out, lse = _lib.binding().varlen(q, kvcache, block_table, cu_seqlens_q, cache_seqlens, dv, data, num_parts, scale,
                                         bool(is_fp8_kvcache), workspace, out, lse, status, max_scratch_bytes)
    if st:
        _lib.check(st, "mla_decode_varlen")
    return out, lse
