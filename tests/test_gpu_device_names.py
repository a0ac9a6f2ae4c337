"""Calls that take a device take it without an index too (the current one)."""
import pytest
import torch

import mla_decode_attention_12_b200 as mla

pytestmark = pytest.mark.gpu


def test_workspace_of_the_current_device():
    zero = mla.workspace_zero_bytes(1, 1, 16, 1)
    ws = mla.api.get_workspace(1 << 20, torch.device("cuda"), zero)
    assert ws.is_cuda and ws.numel() >= 1 << 20 and not ws[:zero].any()
    assert mla.num_sm_parts("cuda") == mla.num_sm_parts() == mla.num_sm_parts(torch.device("cuda", torch.cuda.current_device()))
