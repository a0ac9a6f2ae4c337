"""Ragged runs by the thousand: more than the schedule keeps in shared memory."""
import numpy as np
import pytest
import torch

import mla_decode_attention_12_b200 as mla
from cache_helpers import random_cache
from test_gpu_varlen import check, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("batch", [4096, 4097, 16384])
def test_more_runs_than_are_cached(batch):
    """Up to 4,096 runs the schedule keeps starts and lengths in shared memory, beyond that it reads them again."""
    rng = np.random.default_rng(batch)
    new, lens = rng.integers(0, 4, batch), rng.integers(0, 129, batch).astype(np.int32)
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    d_cu, d_lens = torch.from_numpy(cu).cuda(), torch.from_numpy(lens).cuda()
    for causal in (True, False):
        md, groups = mla.get_mla_metadata_varlen_host(cu, lens, 16, causal=causal)
        plan = mla.get_mla_metadata_varlen(d_cu, d_lens, int(cu[-1]), 16, num_parts=74, causal=causal)
        got = plan.data.cpu().numpy()
        assert np.array_equal(got[:74 * 8].reshape(74, 8), md)
        assert np.array_equal(got[74 * 8:74 * 8 + groups.size].reshape(-1, 8), groups)
    # and the attention by it, over a few pages that the requests share
    g = torch.Generator().manual_seed(batch)
    s = dict(kind="bf16", new=new.tolist(), lens=lens.tolist(), q=torch.randn(int(cu[-1]), 16, 576, generator=g).bfloat16(),
             cu=torch.from_numpy(cu), seqlens=torch.from_numpy(lens),
             table=torch.randint(0, 50, (batch, 2), generator=g, dtype=torch.int32), cache=random_cache("bf16", 50, 576, 1),
             scale=576 ** -0.5)
    check(s, *run(s), only=set(range(0, batch, 37)) | {batch - 1})


def test_runs_that_do_not_split_the_tokens_among_many():
    batch = 5000
    cu = np.arange(batch + 1).astype(np.int32)
    cu[4500] = 4499 - 7
    lens = torch.full((batch,), 5, dtype=torch.int32, device="cuda")
    plan = mla.get_mla_metadata_varlen(torch.from_numpy(cu).cuda(), lens, batch, 16, num_parts=74)
    md = plan.data[:74 * 8].view(74, 8).cpu()
    assert (md[:, 5] == 6).all() and (md[:, :4] == 0).all()
