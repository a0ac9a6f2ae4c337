"""Host devices are refused before anything is launched (no GPU)."""
import pytest
import torch

import mla_decode_attention_12_b200 as mla


def test_workspace_and_decode_on_the_host():
    with pytest.raises(ValueError):
        mla.api.get_workspace(1 << 20, torch.device("cpu"), 1 << 10)
    q = torch.zeros(1, 1, 16, 576, dtype=torch.bfloat16)
    kv = torch.zeros(2, 64, 1, 576, dtype=torch.bfloat16)
    i = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError):
        mla.DecodeCall(q, kv, i.view(1, 1), i, 512, torch.zeros(74, 8, dtype=torch.int32), torch.zeros(2, dtype=torch.int32))
