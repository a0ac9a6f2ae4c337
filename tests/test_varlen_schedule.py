"""The schedule of ragged runs on the host: every page of every group exactly once, balanced; refusals (no GPU)."""
import numpy as np
import pytest

import mla_decode_attention_12_b200 as mla
from mla_decode_attention_12_b200 import _lib, build

FAKE = 1 << 20


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return _lib.load()


def groups_by_hand(new, lens, h_q, causal):
    got, t0 = [], 0
    for b, (n, length) in enumerate(zip(new, lens)):
        rows = n * h_q
        for at in range(0, rows, 128):
            size = min(128, rows - at)
            last = (at + size - 1) // h_q  # the group's last token in the run
            limit = min(max(length - n + 1 + last, 0), length) if causal else length
            got.append((b, t0 * h_q + at, size, limit, length))
        t0 += n
    return got


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("new,lens,h_q", [
    ([1], [1], 1), ([1, 17, 5], [200, 256, 5], 16), ([300, 0, 1, 40], [300, 64, 8192, 20], 20), ([0, 0], [5, 7], 128),
    ([200] * 9, [4096] * 9, 128), ([1] * 100, list(range(0, 7000, 70)), 64), ([7, 3], [0, 0], 128), ([50, 2], [10, 500], 8),
])
@pytest.mark.parametrize("parts", [1, 3, 74])
def test_every_page_once(new, lens, h_q, causal, parts):
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    md, groups = mla.get_mla_metadata_varlen_host(cu, lens, h_q, causal=causal, num_parts=parts)
    want = groups_by_hand(new, lens, h_q, causal)
    want = [g for c in range(parts) for g in want[c::parts]]  # groups 0, P, 2 P, ..., then 1, P + 1, ...
    assert [tuple(int(v) for v in (g[0], g[1], g[2], g[3], g[5])) for g in groups] == want
    pages = [-(-g[3] // 64) for g in want]
    cover = [np.zeros(n, int) for n in pages]
    empty = np.zeros(len(want), int)
    splits = np.zeros(len(want), int)
    cost = []
    for m in md:
        vb, blk, end_vb, end_blk, idx = (int(x) for x in m[:5])
        c, first = 0, True
        while vb < end_vb or (vb == end_vb and blk < end_blk):
            hi = end_blk if vb == end_vb else pages[vb]
            cover[vb][blk:hi] += 1
            empty[vb] += pages[vb] == 0
            assert splits[vb] == (idx if first else 0)  # consecutive partitions hold consecutive splits
            splits[vb] += 1
            c += hi - blk + 12
            vb, blk, first = vb + 1, 0, False
        cost.append(c)
    for n, c, e in zip(pages, cover, empty):
        assert (c == 1).all() and e == (n == 0)
    assert [int(g[6]) for g in groups] == list(splits)
    total = sum(n + 12 for n in pages)
    assert max(cost, default=0) <= 12 + max(-(-(total - 12) // parts), 12) + 12


def test_visible_rows_of_a_group_row():
    _, groups = mla.get_mla_metadata_varlen_host([0, 5], [9], 20, num_parts=4)
    seen, length = int(groups[0][4]), int(groups[0][5])
    assert [min(max(seen + t, 0), length) for t in range(5)] == [5, 6, 7, 8, 9]


@pytest.mark.parametrize("over,code", [
    (dict(total_q=-1), 1), (dict(h_q=0), 1), (dict(q=None), 1), (dict(plan=None), 1), (dict(o=None), 1), (dict(lse=None), 1),
    (dict(table=None), 1), (dict(ws=None), 1), (dict(q=FAKE + 2), 1), (dict(o=FAKE + 8), 1), (dict(plan=FAKE + 4), 1),
    (dict(ws=FAKE + 16), 1), (dict(num_blocks=0), 1), (dict(max_blocks=0), 1), (dict(dtype=9), 1), (dict(parts=0), 1),
    (dict(page=32), 2), (dict(h_kv=2), 2), (dict(d_qk=192), 2), (dict(dv=256), 2), (dict(dtype=2, d_qk=512), 2),
    (dict(batch=16385), 2), (dict(total_q=1 << 24), 2), (dict(ws_bytes=100), 3), (dict(lens=None), 1),
    (dict(dtype=2, total_q=99, scratch=FAKE, scratch_bytes=1000), 3), (dict(dtype=2, total_q=99, scratch=FAKE + 64, scratch_bytes=1 << 40), 1),
])
def test_decode_refuses(lib, over, code):
    a = dict(q=FAKE, total_q=9, h_q=64, d_qk=576, kvcache=FAKE, num_blocks=8, page=64, h_kv=1, table=FAKE, batch=2,
             max_blocks=4, lens=FAKE, dv=512, dtype=0, plan=FAKE, parts=74, scale=0.0, o=FAKE, lse=FAKE, ws=FAKE,
             ws_bytes=1 << 40, scratch=None, scratch_bytes=0, stream=None)
    a.update(over)
    assert lib.mla_decode_varlen(*a.values()) == code


def test_no_runs_or_tokens_is_a_no_op(lib):
    for batch, total in ((0, 0), (3, 0)):
        assert lib.mla_decode_varlen(None, total, 64, 576, None, 8, 64, 1, None, batch, 4, None, 512, 0, None, 74, 0.0, None,
                                     None, None, 0, None, 0, None) == 0


def test_scratch_is_for_fp8_pages_that_several_groups_read(lib):
    size = lib.mla_decode_varlen_scratch_bytes
    assert size(2, 100, 64, 10, 0) == 0 and size(2, 100, 64, 10, 1) == 0
    assert size(2, 100, 64, 10, 2) >= 2 * 10 * 64 * 1152
    assert size(2, 11, 64, 10, 2) == 0   # 5.5 groups for two runs
    assert size(2, 12, 64, 10, 2) > 0    # 6
    assert size(64, 10 ** 5, 64, 2048, 2) == 0  # 9.7 GB


def test_metadata_refuses(lib):
    assert lib.mla_get_metadata_varlen(None, FAKE, 2, 9, 64, 1, 1, 74, 0, FAKE, None) == 1
    assert lib.mla_get_metadata_varlen(FAKE, FAKE, 2, 9, 64, 1, 2, 74, 0, FAKE, None) == 1
    assert lib.mla_get_metadata_varlen(FAKE, FAKE, 2, 9, 64, 2, 1, 74, 0, FAKE, None) == 2
    assert lib.mla_get_metadata_varlen(FAKE, FAKE, 2, 9, 64, 1, 1, 74, 0, FAKE + 4, None) == 1
    assert lib.mla_varlen_plan_ints(2, 9, 64, 1, 74) >= 74 * 8 + (9 * 64 // 128 + 2) * 8
    assert lib.mla_varlen_plan_ints(2, 9, 64, 2, 74) == 0
    for cu in ([1, 0], [0, 3, 2], [-1, 2]):
        with pytest.raises(mla.MLAError):
            mla.get_mla_metadata_varlen_host(cu, [5] * (len(cu) - 1), 16)
