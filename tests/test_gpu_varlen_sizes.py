"""Schedules of ragged runs and of the decode at sizes where the kernel's shared memory changes form."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import mla_decode_attention_12_b200 as mla

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

RAGGED = """
import numpy as np, torch
import mla_decode_attention_12_b200 as mla
new, lens, h_q = np.array({new}), np.array({lens}, dtype=np.int32), {h_q}
cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
md, groups = mla.get_mla_metadata_varlen_host(cu, lens, h_q)
plan = mla.get_mla_metadata_varlen(torch.from_numpy(cu).cuda(), torch.from_numpy(lens).cuda(), int(cu[-1]), h_q, num_parts=74)
got = plan.data.cpu().numpy()
assert np.array_equal(got[:74 * 8].reshape(74, 8), md)
assert np.array_equal(got[74 * 8:74 * 8 + groups.size].reshape(-1, 8), groups)
"""

DENSE = """
import numpy as np, torch
import mla_decode_attention_12_b200 as mla
lens = (np.arange({batch}) * 37 % 900).astype(np.int32)
md, ns = mla.get_mla_metadata(torch.from_numpy(lens).cuda(), 128, 1, num_parts=74)
want_md, want_ns = mla.get_mla_metadata_host(lens, 128)
assert np.array_equal(md.cpu().numpy(), want_md) and np.array_equal(ns.cpu().numpy(), want_ns)
"""


def in_a_fresh_process(code):
    done = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert done.returncode == 0, done.stderr[-2000:]


# Dynamic and static shared memory together pass 48 KB where the dynamic part alone does not.  A kernel's larger limit
# stays set for the process once a larger schedule asked for it, so each size is the first of its process.
@pytest.mark.parametrize("new,lens,h_q", [("[6040]", "[7000]", 128), ("[12100]", "[12100]", 64), ("[90] * 63 + [210]", "[400] * 64", 128)])
def test_ragged_schedule_next_to_48_kb(new, lens, h_q):
    in_a_fresh_process(RAGGED.format(new=new, lens=lens, h_q=h_q))


@pytest.mark.parametrize("batch", [3020, 3034])
def test_dense_schedule_next_to_48_kb(batch):
    in_a_fresh_process(DENSE.format(batch=batch))
