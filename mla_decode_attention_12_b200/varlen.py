"""Attention of ragged runs of new tokens (chunks of prompts beside decode steps) over the paged cache.

``get_mla_metadata_varlen`` once per step, then ``flash_mla_varlen_with_kvcache`` once per layer.
Formulas and errors: ``include/mla_decode.h``.
"""
from __future__ import annotations

import math
from dataclasses import dataclass

import torch

from . import _lib
from .api import _DTYPES, _ptr, _stream, get_workspace, num_sm_parts, workspace_zero_bytes
from .cache import _cache_dtype, _check_ints


@dataclass(frozen=True)
class VarlenPlan:
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
    dev = cu_seqlens_q.device
    if not cu_seqlens_q.is_cuda:
        raise ValueError("cu_seqlens_q must be on a CUDA device")
    _check_ints(dev, cu_seqlens_q=(cu_seqlens_q, 1), cache_seqlens=(cache_seqlens, 1))
    batch = cache_seqlens.shape[0]
    if cu_seqlens_q.shape[0] != batch + 1:
        raise ValueError("cu_seqlens_q must have one entry more than cache_seqlens")
    if num_parts is None:
        num_parts = out.num_parts if out is not None else num_sm_parts(dev)
    lib = _lib.load()
    ints = lib.mla_varlen_plan_ints(batch, total_q, h_q, h_kv, num_parts)
    if ints == 0:
        raise ValueError("invalid or unsupported sizes for the schedule")
    plan = VarlenPlan(out.data if out is not None else torch.empty(ints, dtype=torch.int32, device=dev), batch, int(total_q),
                      int(h_q), num_parts, bool(causal))
    if out is not None and (out != plan or out.data.device != dev or out.data.numel() != ints):
        raise ValueError("out is a plan of other sizes")
    with torch.cuda.device(dev):
        _lib.check(lib.mla_get_metadata_varlen(_ptr(cu_seqlens_q), _ptr(cache_seqlens), batch, total_q, h_q, h_kv,
                                               int(plan.causal), num_parts, int(bool(is_fp8_kvcache)), _ptr(plan.data),
                                               _stream(dev)), "mla_get_metadata_varlen")
    return plan


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


def _call_workspace(nbytes: int, dev: torch.device) -> torch.Tensor:
    """The stream's cached workspace; inside a graph capture one of the graph's own, whose control block each replay
    zeroes (two graphs captured on one stream may be replayed on two)."""
    zero = workspace_zero_bytes(1, 1, 1, 1)
    with torch.cuda.device(dev):
        if not torch.cuda.is_current_stream_capturing():
            return get_workspace(nbytes, dev, zero)
        ws = torch.empty(nbytes, dtype=torch.uint8, device=dev)
        ws[:zero].zero_()
        return ws


def flash_mla_varlen_with_kvcache(q: torch.Tensor, kvcache: torch.Tensor, block_table: torch.Tensor,
                                  cu_seqlens_q: torch.Tensor, cache_seqlens: torch.Tensor, dv: int, plan: VarlenPlan,
                                  causal: bool = True, is_fp8_kvcache: bool = False, *, softmax_scale: float | None = None,
                                  workspace: torch.Tensor | None = None, out: torch.Tensor | None = None,
                                  lse: torch.Tensor | None = None):
    """MLA attention of ragged runs over a paged cache; ``(o [total_q, h_q, dv], lse [total_q, h_q] float32)``.

    ``q`` [total_q, h_q, d_qk]; ``kvcache``, ``block_table`` [batch, max_blocks] and the FP8 cache as for
    ``flash_mla_with_kvcache``.  Token i of a run of n tokens over L cached ones sees the first
    ``L - n + 1 + i`` of them (``causal``), or all L.  ``plan`` comes from ``get_mla_metadata_varlen``
    with the same ``cu_seqlens_q``, ``cache_seqlens`` and ``causal``.  Rows past ``cu_seqlens_q[batch]`` are
    not written (of ``out`` and ``lse`` passed in, they stay as they were).
    """
    dtype, d_qk = _cache_dtype(kvcache, is_fp8_kvcache)
    dev = kvcache.device
    dt = torch.bfloat16 if is_fp8_kvcache else kvcache.dtype
    if q.dim() != 3 or q.dtype != dt or q.shape[2] != d_qk or not q.is_contiguous() or q.device != dev:
        raise ValueError(f"q must be contiguous {dt} [total_q, h_q, {d_qk}] on {dev}")
    total_q, h_q, _ = q.shape
    _check_ints(dev, block_table=(block_table, 2), cu_seqlens_q=(cu_seqlens_q, 1), cache_seqlens=(cache_seqlens, 1))
    batch = cache_seqlens.shape[0]
    if block_table.shape[0] != batch or cu_seqlens_q.shape[0] != batch + 1:
        raise ValueError("inconsistent shapes")
    if (plan.batch, plan.total_q, plan.h_q, plan.causal) != (batch, total_q, h_q, bool(causal)) or plan.data.device != dev:
        raise ValueError("the plan was made for another call")
    if out is None:
        out = torch.empty(total_q, h_q, dv, dtype=dt, device=dev)
    elif out.dtype != dt or tuple(out.shape) != (total_q, h_q, dv) or not out.is_contiguous() or out.device != dev:
        raise ValueError(f"out must be contiguous {dt} [{total_q}, {h_q}, {dv}] on {dev}")
    if lse is None:
        lse = torch.empty(total_q, h_q, dtype=torch.float32, device=dev)
    elif lse.dtype != torch.float32 or tuple(lse.shape) != (total_q, h_q) or not lse.is_contiguous() or lse.device != dev:
        raise ValueError(f"lse must be contiguous float32 [{total_q}, {h_q}] on {dev}")
    if workspace is None:
        workspace = _call_workspace(varlen_workspace_bytes(plan.num_parts), dev)
    elif workspace.device != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace must be contiguous and on {dev}")
    if batch == 0 or total_q == 0:
        return out, lse
    num_blocks, page, h_kv, _ = kvcache.shape
    scale = float(softmax_scale) if softmax_scale is not None else 1.0 / math.sqrt(d_qk)
    with torch.cuda.device(dev):
        _lib.check(_lib.load().mla_decode_varlen(
            _ptr(q), total_q, h_q, d_qk, _ptr(kvcache), num_blocks, page, h_kv, _ptr(block_table), batch,
            block_table.shape[1], dv, dtype, _ptr(plan.data), plan.num_parts, scale, _ptr(out), _ptr(lse), _ptr(workspace),
            workspace.numel() * workspace.element_size(), _stream(dev)), "mla_decode_varlen")
    return out, lse
