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
