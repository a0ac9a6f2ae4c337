"""Ragged runs over an FP8 cache whose pages are dequantized first: what is read, and what memory it takes."""
import ctypes

import pytest
import torch

import mla_decode_attention_12_b200 as mla
from cache_helpers import DV
from test_gpu_varlen import check, make, run

pytestmark = pytest.mark.gpu


def on_gpu(s):
    return {k: v.cuda() for k, v in s.items() if isinstance(v, torch.Tensor)}


@pytest.mark.parametrize("length", [300, 2 ** 31 - 1])
def test_runs_without_tokens_are_not_dequantized(length):
    # an inactive entry of a padded batch: a stale length, no pages
    s = make("fp8", [6, 0], [200, 300], 128, seed=41)
    s["table"][1] = -1
    s["seqlens"][1] = length
    ws = torch.zeros(mla.varlen_workspace_bytes(74), dtype=torch.uint8, device="cuda")
    o, lse = run(s, workspace=ws, num_parts=74)
    assert mla.read_device_status(ws) == 0
    check(s, o, lse)
    # the same through the direct path
    from mla_decode_attention_12_b200 import _lib
    d = on_gpu(s)
    plan = mla.get_mla_metadata_varlen(d["cu"], d["seqlens"], 6, 128, is_fp8_kvcache=True, num_parts=74)
    assert _lib.load().mla_decode_varlen_scratch_bytes(2, 6, 128, d["table"].shape[1], 2) > 0
    assert _lib.load().mla_decode_varlen(
        d["q"].data_ptr(), 6, 128, 576, d["cache"].data_ptr(), d["cache"].shape[0], 64, 1, d["table"].data_ptr(), 2,
        d["table"].shape[1], d["seqlens"].data_ptr(), DV, 2, plan.data.data_ptr(), 74, ctypes.c_float(s["scale"]), o.data_ptr(),
        lse.data_ptr(), ws.data_ptr(), ws.numel(), None, 0, torch.cuda.current_stream().cuda_stream) == 0
    torch.cuda.synchronize()
    assert mla.read_device_status(ws) == 0
    check(s, o, lse)


def wide(width):
    """Two runs that are dequantized first, with a block table far wider than their pages."""
    s = make("fp8", [5, 9], [140, 2600], 128, seed=42)
    s["table"] = torch.nn.functional.pad(s["table"], (0, width - s["table"].shape[1]), value=-1).contiguous()
    d = on_gpu(s)
    return s, d, mla.get_mla_metadata_varlen(d["cu"], d["seqlens"], 14, 128, is_fp8_kvcache=True)


def call(s, d, plan, **kw):
    return mla.flash_mla_varlen_with_kvcache(d["q"], d["cache"], d["table"], d["cu"], d["seqlens"], DV, plan, True, True,
                                             softmax_scale=s["scale"], **kw)


def test_a_call_that_does_not_get_its_scratch():
    s, d, plan = wide(16384)  # 2.4 GB of scratch
    call(s, d, plan, max_scratch_bytes=0)  # the stream's workspace exists from here on
    torch.cuda.empty_cache()
    limit = torch.cuda.memory_reserved() + (1 << 29)
    torch.cuda.set_per_process_memory_fraction(limit / torch.cuda.get_device_properties(0).total_memory)
    try:
        with pytest.raises(torch.cuda.OutOfMemoryError):
            torch.empty(2 << 30, dtype=torch.uint8, device="cuda")
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        o, lse = call(s, d, plan, status=status)
        assert int(status) == 0
        check(s, o, lse)
    finally:
        torch.cuda.set_per_process_memory_fraction(1.0)


def test_the_caller_bounds_the_scratch():
    from mla_decode_attention_12_b200 import _lib
    s, d, plan = wide(2048)
    need = _lib.load().mla_decode_varlen_scratch_bytes(2, 14, 128, 2048, 2)
    assert need > 2 * 2048 * 64 * 1152
    call(s, d, plan)
    for most, taken in ((0, False), (need - 1, False), (need, True), (None, True)):
        torch.cuda.synchronize()
        torch.cuda.reset_peak_memory_stats()
        before = torch.cuda.memory_allocated()
        o, lse = call(s, d, plan, max_scratch_bytes=most)
        assert (torch.cuda.max_memory_allocated() - before > need) == taken
        check(s, o, lse)
    for bad in (-1, 1.5, "much"):
        with pytest.raises(ValueError):
            call(s, d, plan, max_scratch_bytes=bad)
