"""A call that records a device error, and the calls after it on the same stream and workspace.

An error that is tolerated (a length beyond the block table, a page outside the cache, runs that do not split the tokens)
costs the healthy requests nothing, in its own call or a later one, and nothing has to be cleared.  A call whose wait gave
up leaves the workspace's counters as it found them.
"""
import ctypes
import os

import numpy as np
import pytest
import torch

import mla_decode_attention_12_b200 as mla
from cache_helpers import DV, HALF_STEP, PAGE, attend64, cache_rows64, random_cache
from test_gpu_varlen import check, make, run

pytestmark = pytest.mark.gpu

SENTINEL = 7.0
CONTROL = 256  # the status word's part of the control block; the counters follow


def on_gpu(s):
    return {k: v.cuda() for k, v in s.items() if isinstance(v, torch.Tensor)}


def sentinels(s):
    rows, heads = s["q"].shape[:2]
    return (torch.full((rows, heads, DV), SENTINEL, dtype=s["q"].dtype, device="cuda"),
            torch.full((rows, heads), SENTINEL, device="cuda"))


def dense(s, status=None, workspace=None):
    """The requests of s (runs of one token) through the dense decode, into prefilled outputs."""
    d = on_gpu(s)
    b, heads = len(s["new"]), s["q"].shape[1]
    md, ns = mla.get_mla_metadata(d["seqlens"], heads, 1, is_fp8_kvcache=s["kind"] == "fp8")
    o, lse = sentinels(s)
    mla.flash_mla_with_kvcache(d["q"].view(b, 1, heads, -1), d["cache"], d["table"], d["seqlens"], DV, md, ns, False,
                               s["kind"] == "fp8", softmax_scale=s["scale"], out=o.view(b, 1, heads, DV),
                               lse=lse.view(b, 1, heads), workspace=workspace)
    return o, lse


def ragged(s, **kw):
    o, lse = sentinels(s)
    run(s, out=o, lse=lse, **kw)
    return o, lse


def healthy(kind="bf16", seed=51):
    """Requests that are split over many partitions."""
    return make(kind, [1, 1], [9000, 14000], 64, seed=seed)


def with_error(error, kind="bf16"):
    s = make(kind, [1, 1], [9000, 14000], 64, seed=52)
    only = [0]
    if error == "length":
        s["seqlens"][1] = 14000 + 64 * 200  # beyond the table, which is 219 pages wide
    elif error == "page":
        s["table"][1, 100] = s["cache"].shape[0] + 3
    else:
        s["cu"] = torch.tensor([0, 2, 1], dtype=torch.int32)
        only = []
    return s, only


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("error", ["length", "page", "runs"])
def test_calls_after_a_tolerated_error(error, kind):
    bad, only = with_error(error, kind)
    good = healthy(kind)
    with torch.cuda.stream(torch.cuda.Stream()):  # its own default workspace
        for _ in range(3):
            o, lse = ragged(bad)
            check(bad, o, lse, only=only)
            check(good, *ragged(good))
            check(good, *dense(good))
    torch.cuda.synchronize()


def test_dense_calls_after_a_tolerated_error():
    bad, _ = with_error("page")
    good = healthy()
    with torch.cuda.stream(torch.cuda.Stream()):
        for _ in range(3):
            check(bad, *dense(bad), only=[0])
            check(good, *ragged(good))
            check(good, *dense(good))
    torch.cuda.synchronize()


def test_calls_after_a_page_sparse_decode_of_a_bad_page():
    heads = 64
    lens = [64 * 150, 64 * 90 + 7]
    s = make("bf16", [1, 1], lens, heads, seed=53)
    g = torch.Generator().manual_seed(54)
    pages = s["cache"].shape[0]
    keys = torch.randint(-127, 128, (pages, 576), generator=g).to(torch.int8).cuda()
    scales = (torch.rand(pages, generator=g) * 0.01 + 1e-3).cuda()
    d = on_gpu(s)
    bad = d["table"].clone()
    bad[1, 0] = pages + 1  # the first page is always chosen
    with torch.cuda.stream(torch.cuda.Stream()):
        for table in (bad, d["table"], bad, d["table"]):
            t, n = mla.mla_select_pages(d["q"].view(2, 1, heads, 576), keys, scales, table, d["seqlens"], 80)
            o, lse = mla.flash_mla_page_sparse(d["q"].view(2, 1, heads, 576), d["cache"], table, d["seqlens"], DV, keys, scales, 80)
            torch.cuda.synchronize()
            u, rows = HALF_STEP[torch.bfloat16], cache_rows64(s["cache"], False)
            for b in range(2 if table is not bad else 1):
                i = torch.arange(int(n[b]))
                kv = rows[t[b].cpu().long()[i // PAGE] * PAGE + i % PAGE]
                q = s["q"][b]
                want, want_l = attend64(q, kv, torch.full((heads,), int(n[b])), 576 ** -0.5)
                size = torch.softmax(q.double() @ kv.T * 576 ** -0.5, -1) @ kv[:, :DV].abs()
                assert ((o[b, 0].cpu().double() - want).abs() <= (u + 2.0 ** -12) * size + u * want.abs() * (1 + 2.0 ** -7)).all()
                assert ((lse[b, 0].cpu().double() - want_l).abs() <= 2.0 ** -14 * (1 + want_l.abs())).all()
            check(s, *dense(s))


@pytest.fixture(scope="module")
def withholding_lib():
    # the build of test_gpu_failure.py: page 3 of partition 0's first chunk never loads, waits are bounded at 0.2 s
    from mla_decode_attention_12_b200 import _lib, build
    out = os.path.join(os.path.dirname(build.LIB), "_mla_decode_test_withhold.so")
    return _lib.bind(build.build(extra=["-DMLA_TEST_WITHHOLD_K_PAGE=3", "-DMLA_WAIT_TIMEOUT_NS=200000000ull"], out=out))


def untouched(o, lse):
    return (o == SENTINEL).all(-1) & (lse == SENTINEL)


@pytest.mark.parametrize("parts", [4, 9])
def test_a_wait_that_gave_up_leaves_the_counters_zero(withholding_lib, parts):
    """Ragged runs: nothing of the aborted cluster's groups is written, the others are right, and the workspace serves the
    next call without being cleared."""
    s = make("bf16", [1, 2, 1, 1], [3000, 5000, 700, 64], 128, seed=55)
    d = on_gpu(s)
    plan = mla.get_mla_metadata_varlen(d["cu"], d["seqlens"], 5, 128, num_parts=parts)
    md, groups = mla.get_mla_metadata_varlen_host(s["cu"].numpy(), s["seqlens"].numpy(), 128, num_parts=parts)
    assert tuple(md[0][:2]) == (0, 0) and (md[0][2] > 0 or md[0][3] > 3)
    ws = torch.zeros(mla.varlen_workspace_bytes(parts), dtype=torch.uint8, device="cuda")
    o, lse = sentinels(s)
    stream = torch.cuda.current_stream().cuda_stream
    for _ in range(2):
        st = withholding_lib.mla_decode_varlen(
            d["q"].data_ptr(), 5, 128, 576, d["cache"].data_ptr(), d["cache"].shape[0], 64, 1, d["table"].data_ptr(), 4,
            d["table"].shape[1], d["seqlens"].data_ptr(), DV, 0, plan.data.data_ptr(), parts, ctypes.c_float(s["scale"]),
            o.data_ptr(), lse.data_ptr(), ws.data_ptr(), ws.numel(), None, 0, stream)
        assert st == 0
        torch.cuda.synchronize()
        assert not ws[CONTROL:mla.workspace_zero_bytes(1, 1, 1, 1)].any()
        assert int(ws[:4].view(torch.int32)) == 5
        # the groups that partition 0 works on, and no others, are unwritten
        lost = set(range(0, int(md[0][2]) + (1 if md[0][3] > 0 else 0)))
        blank = untouched(o, lse).cpu().view(-1)
        for v, gr in enumerate(groups):
            rows = blank[int(gr[1]):int(gr[1]) + int(gr[2])]
            assert bool(rows.all()) == (v in lost) and bool(rows.any()) == (v in lost), v
        rest = [b for b in range(4) if not any(int(groups[v][0]) == b for v in lost)]
        assert rest
        check({**s, "q": s["q"]}, torch.where((o == SENTINEL), 0.0, o), torch.where(lse == SENTINEL, 0.0, lse), only=rest)
    check(s, *ragged(s, workspace=ws, num_parts=parts))  # the status word still holds the error
    assert mla.read_device_status(ws) == 5
    check(s, *ragged(s, workspace=ws, num_parts=parts))
    assert mla.read_device_status(ws) == 0


def test_a_dense_wait_that_gave_up_leaves_the_counters_zero(withholding_lib):
    from mla_decode_attention_12_b200 import _lib
    s = make("bf16", [1, 1, 1, 1], [3000, 5000, 700, 64], 128, seed=56)
    d = on_gpu(s)
    md, ns = mla.get_mla_metadata(d["seqlens"], 128, 1, num_parts=4)
    ws = torch.zeros(mla.workspace_bytes(4, 1, 128, 1, 74), dtype=torch.uint8, device="cuda")
    o, lse = sentinels(s)
    call = mla.DecodeCall(d["q"].view(4, 1, 128, 576), d["cache"], d["table"], d["seqlens"], DV, md, ns, softmax_scale=s["scale"],
                          workspace=ws, out=o.view(4, 1, 128, DV), lse=lse.view(4, 1, 128))
    _lib.check(withholding_lib.mla_decode_with_kvcache(*call.args, torch.cuda.current_stream().cuda_stream), "decode")
    torch.cuda.synchronize()
    assert not ws[CONTROL:mla.workspace_zero_bytes(1, 1, 1, 1)].any()
    assert untouched(o[:1], lse[:1]).all() and not untouched(o, lse).all()
    check(s, *dense(s, workspace=ws))
    assert mla.read_device_status(ws) == 5


@pytest.mark.parametrize("error", ["length", "page", "runs"])
def test_status_of_a_ragged_call(error):
    bad, only = with_error(error)
    good = healthy()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = torch.zeros(mla.varlen_workspace_bytes(mla.num_sm_parts()), dtype=torch.uint8, device="cuda")

    def call(s):
        d = on_gpu(s)
        plan = mla.get_mla_metadata_varlen(d["cu"], d["seqlens"], 2, 64)
        o, lse = sentinels(s)
        return mla.flash_mla_varlen_with_kvcache(d["q"], d["cache"], d["table"], d["cu"], d["seqlens"], DV, plan,
                                                 softmax_scale=s["scale"], workspace=ws, out=o, lse=lse, status=status)

    check(bad, *call(bad), only=only)
    assert int(status) == 6 and not ws[:mla.workspace_zero_bytes(1, 1, 1, 1)].any()
    check(good, *call(good))
    assert int(status) == 6  # the first error stays
    status.zero_()
    check(good, *call(good))
    assert int(status) == 0


def test_status_of_a_dequantized_page():
    s = make("fp8", [5, 9], [140, 260], 128, seed=57)
    d = on_gpu(s)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    plan = mla.get_mla_metadata_varlen(d["cu"], d["seqlens"], 14, 128, is_fp8_kvcache=True)
    for table, want in ((d["table"].masked_fill(torch.arange(d["table"].shape[1]).cuda() == 1, -1), 6), (d["table"], 0)):
        status.zero_()
        o, lse = mla.flash_mla_varlen_with_kvcache(d["q"], d["cache"], table, d["cu"], d["seqlens"], DV, plan, True, True,
                                                   softmax_scale=s["scale"], status=status)
        assert int(status) == want
    check(s, o, lse)


def test_status_of_a_page_sparse_decode():
    heads, lens = 16, [64 * 40, 64 * 30]
    s = make("bf16", [1, 1], lens, heads, seed=58)
    pages = s["cache"].shape[0]
    keys, scales = torch.zeros(pages, 576, dtype=torch.int8).cuda(), torch.zeros(pages).cuda()
    d = on_gpu(s)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def call(table, topn):
        status.zero_()
        return mla.flash_mla_page_sparse(d["q"].view(2, 1, heads, 576), d["cache"], table, d["seqlens"], DV, keys, scales, topn,
                                         status=status)

    bad = d["table"].clone()
    bad[0, 0] = pages
    for topn in (8, 64):
        call(bad, topn)
        assert int(status) == 6
        o, lse = call(d["table"], topn)
        assert int(status) == 0
    check(s, o.view(2, heads, DV), lse.view(2, heads))
    for refused in (torch.zeros(2, dtype=torch.int32, device="cuda"), torch.zeros(1, device="cuda"), torch.zeros(1, dtype=torch.int32)):
        with pytest.raises(ValueError):
            mla.flash_mla_page_sparse(d["q"].view(2, 1, heads, 576), d["cache"], d["table"], d["seqlens"], DV, keys, scales, 8,
                                      status=refused)
        with pytest.raises(ValueError):
            mla.flash_mla_varlen_with_kvcache(d["q"], d["cache"], d["table"], d["cu"], d["seqlens"], DV,
                                              mla.get_mla_metadata_varlen(d["cu"], d["seqlens"], 2, heads), status=refused)
