"""flash_mla_varlen_with_kvcache on the GPU against attention in 64 bits."""
import numpy as np
import pytest
import torch

import mla_decode_attention_12_b200 as mla
from cache_helpers import (DTYPES, DV, HALF_STEP, PAGE, attend64, cache_rows64, random_cache, request_rows, table_of)

pytestmark = pytest.mark.gpu


def make(kind, new, lens, heads, d=576, seed=0, extra_q=0):
    g = torch.Generator().manual_seed(seed)
    table, pages = table_of(lens, seed)
    cu = torch.tensor([0] + list(np.cumsum(new)), dtype=torch.int32)
    q = torch.randn(int(cu[-1]) + extra_q, heads, d, generator=g).to(DTYPES[kind])
    return dict(kind=kind, new=new, lens=lens, q=q, cu=cu, seqlens=torch.tensor(lens, dtype=torch.int32), table=table,
                cache=random_cache(kind, pages, d, seed + 1), scale=d ** -0.5)


def run(s, *, causal=True, num_parts=None, workspace=None, out=None, lse=None, plan=None, dev=None):
    dev = dev or {k: v.cuda() for k, v in s.items() if isinstance(v, torch.Tensor)}
    fp8 = s["kind"] == "fp8"
    q = dev["q"]
    plan = plan or mla.get_mla_metadata_varlen(dev["cu"], dev["seqlens"], q.shape[0], q.shape[1], causal=causal,
                                               is_fp8_kvcache=fp8, num_parts=num_parts)
    return mla.flash_mla_varlen_with_kvcache(q, dev["cache"], dev["table"], dev["cu"], dev["seqlens"], DV, plan, causal, fp8,
                                             softmax_scale=s["scale"], workspace=workspace, out=out, lse=lse)


def check(s, o, lse, causal=True, only=None):
    """Every element within what the roundings allow.  With u the half step of the type: the weights are
    rounded to it once (u of sum p |v|), the result once (u |o|); float32 logits (576 products of size
    |q| |k| / 24) and sums add well below 2^-12 of sum p |v|.  fp16 weights below 2^-14 lose 2^-25 each."""
    dt = DTYPES[s["kind"]]
    u = HALF_STEP[dt]
    rows = cache_rows64(s["cache"], s["kind"] == "fp8")
    o, lse = o.cpu().double(), lse.cpu().double()
    heads, at = s["q"].shape[1], 0
    for b, (n, length) in enumerate(zip(s["new"], s["lens"])):
        if n and (only is None or b in only):
            kv = request_rows(rows, s["table"], b, length)
            sees = torch.full((n,), length) if not causal else (length - n + 1 + torch.arange(n)).clamp(0, length)
            n_vis = sees.repeat_interleave(heads)
            q = s["q"][at:at + n].reshape(-1, s["q"].shape[2])
            want, want_l = attend64(q, kv, n_vis, s["scale"])
            # sum p |v|: the same weights over |v|
            x = (q.double() @ kv.T * s["scale"]).masked_fill(torch.arange(length)[None] >= n_vis[:, None], -torch.inf)
            p = torch.nan_to_num(torch.softmax(x, -1)) if length else x
            size = p @ kv[:, :DV].abs()
            tol = (u + 2.0 ** -12) * size + u * want.abs() * (1 + 2.0 ** -7)
            if dt == torch.float16:
                tol = tol + 2.0 ** -25 * (1 + kv[:, :DV].abs().sum(0))
            got, got_l = o[at:at + n].reshape(-1, DV), lse[at:at + n].reshape(-1)
            assert torch.isfinite(got).all()
            worst = ((got - want).abs() - tol).max()
            assert worst <= 0, (b, float(worst))
            fin = torch.isfinite(want_l)
            assert torch.equal(torch.isfinite(got_l), fin) and (got_l[~fin] == -torch.inf).all()
            assert ((got_l - want_l)[fin].abs() <= 2.0 ** -14 * (1 + want_l[fin].abs())).all()
        at += n


CASES = [
    ([1], [1], 1), ([1], [64], 128), ([3], [3], 128), ([1, 17, 5], [200, 256, 193], 16), ([65, 1, 0, 9], [65, 700, 64, 300], 20),
    ([130], [130], 3), ([0, 2], [0, 130], 128), ([4, 2], [2, 0], 16), ([40, 1, 33], [555, 64, 1000], 64), ([6], [5000], 96),
]


@pytest.mark.parametrize("kind,d", [("bf16", 576), ("bf16", 512), ("fp16", 576), ("fp16", 512), ("fp8", 576)])
@pytest.mark.parametrize("new,lens,heads", CASES)
def test_parity(kind, d, new, lens, heads):
    s = make(kind, new, lens, heads, d, seed=len(new) + heads)
    check(s, *run(s))


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("parts", [1, 2, 7, 110])
def test_partitions_and_splits(kind, parts):
    s = make(kind, [1, 30, 2], [3000, 2000, 4500], 32, seed=parts)
    check(s, *run(s, num_parts=parts))


def test_one_request_split_over_all_partitions():
    s = make("bf16", [1], [20000], 128, seed=3)
    check(s, *run(s))
    s = make("fp16", [2], [30000], 8, seed=4)
    check(s, *run(s))


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
def test_without_causal_mask(kind):
    s = make(kind, [5, 1, 20], [100, 1, 333], 48, seed=6)
    check(s, *run(s, causal=False), causal=False)


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("new", [[3, 1], [6, 4]])  # an FP8 cache: read directly, and dequantized first
def test_rows_that_no_group_sees_may_hold_nan(kind, new):
    # 128 heads: one token per group; the rows of later tokens, the tails and unowned pages are poisoned
    lens = [70, 100]
    s = make(kind, new, lens, 128, seed=7)
    clean = run(s)
    cache = s["cache"].clone()
    flat = cache.view(-1, cache.shape[-1])
    poison = torch.ones(flat.shape[0], dtype=torch.bool)
    for b, length in enumerate(lens):
        i = torch.arange(length)
        poison[s["table"][b].long()[i // PAGE] * PAGE + i % PAGE] = False
    if kind == "fp8":
        flat[poison] = 0xFF
    else:
        flat[poison] = float("nan")
    s["cache"] = cache
    o, lse = run(s)
    assert torch.equal(o, clean[0]) and torch.equal(lse, clean[1])
    # the last token's row poisoned: the run's earlier tokens do not see it
    last = 69
    row = int(s["table"][0, last // PAGE]) * PAGE + last % PAGE
    flat[row] = 0xFF if kind == "fp8" else float("nan")
    o, lse = run(s)
    n = new[0] - 1
    assert torch.equal(o[:n], clean[0][:n]) and torch.equal(lse[:n], clean[1][:n])


def test_rows_behind_the_last_run_stay():
    s = make("bf16", [3, 9], [40, 300], 20, seed=8, extra_q=7)
    s["q"][12:] = float("nan")  # a batch padded to a fixed size
    out = torch.full((19, 20, DV), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((19, 20), 5.0, device="cuda")
    run(s, out=out, lse=lse)
    check(s, out, lse)
    assert (out[12:] == 7.0).all() and (lse[12:] == 5.0).all()


def test_rows_before_the_first_run_stay():
    s = make("bf16", [3, 9], [40, 300], 20, seed=30, extra_q=2)
    s["q"] = torch.cat([s["q"][12:], s["q"][:12]])
    s["cu"] += 2
    out = torch.full((14, 20, DV), 7.0, dtype=torch.bfloat16, device="cuda")
    o, lse = run(s, out=out)
    assert (o[:2] == 7.0).all()
    s["q"] = s["q"][2:]
    check(s, o[2:], lse[2:])


@pytest.mark.parametrize("new,lens", [([], []), ([0, 0], [5, 70]), ([0], [0])])
def test_no_runs_or_no_tokens(new, lens):
    s = make("bf16", new, lens, 16, seed=31)
    s["table"] = s["table"].reshape(len(lens), -1) if lens else torch.zeros(0, 3, dtype=torch.int32)
    o, lse = run(s)
    assert o.shape == (0, 16, DV) and lse.shape == (0, 16)
    if lens:  # and with rows of a padded batch behind them
        s["q"] = torch.zeros(5, 16, 576, dtype=torch.bfloat16)
        out = torch.full((5, 16, DV), 7.0, dtype=torch.bfloat16, device="cuda")
        run(s, out=out)
        assert (out == 7.0).all()


@pytest.mark.parametrize("kind,new", [("bf16", [2, 3]), ("fp8", [1, 1]), ("fp8", [5, 7])])
def test_pages_past_32_bit_offsets(kind, new):
    # a cache of 4.3 GB and more: the byte offsets of its last pages pass 2^32
    lens = [200, 65]
    s = make(kind, new, lens, 128, seed=32)
    pages = 60000 if kind == "bf16" else 110000
    d = {k: v.cuda() for k, v in s.items() if isinstance(v, torch.Tensor)}
    small = s["cache"]
    d["cache"] = torch.empty(pages, *small.shape[1:], dtype=small.dtype, device="cuda")
    d["cache"][pages - small.shape[0]:] = small.cuda()
    d["table"] = torch.where(d["table"] >= 0, d["table"] + (pages - small.shape[0]), -1).to(torch.int32)
    check(s, *run(s, dev=d))


def test_a_plan_written_again():
    s = make("bf16", [3, 30], [40, 300], 20, seed=33)
    d = {k: v.cuda() for k, v in s.items() if isinstance(v, torch.Tensor)}
    plan = mla.get_mla_metadata_varlen(d["cu"], d["seqlens"], 33, 20)
    s["new"], s["lens"] = [13, 20], [64, 257]  # within the pages of the table
    d["cu"].copy_(torch.tensor([0, 13, 33]))
    d["seqlens"].copy_(torch.tensor(s["lens"]))
    again = mla.get_mla_metadata_varlen(d["cu"], d["seqlens"], 33, 20, out=plan)
    assert again.data is plan.data or again.data.data_ptr() == plan.data.data_ptr()
    for _ in range(2):  # two layers with one plan
        check(s, *run(s, dev=d, plan=again))
    with pytest.raises(ValueError):
        mla.get_mla_metadata_varlen(d["cu"], d["seqlens"], 33, 10, out=plan)
    with pytest.raises(ValueError):
        mla.get_mla_metadata_varlen(d["cu"], d["seqlens"], 33, 20, causal=False, out=plan)


def test_same_as_the_dense_decode():
    # runs of equal length are what the dense decode computes
    s = make("bf16", [2] * 5, [500, 64, 129, 2, 1000], 64, seed=9)
    o, lse = run(s)
    q = s["q"].view(5, 2, 64, 576).cuda()
    md, ns = mla.get_mla_metadata(s["seqlens"].cuda(), 128, 1)
    o2, lse2 = mla.flash_mla_with_kvcache(q, s["cache"].cuda(), s["table"].cuda(), s["seqlens"].cuda(), DV, md, ns, causal=True,
                                          softmax_scale=s["scale"])
    check(s, o2.view(10, 64, DV), lse2.view(10, 64))
    check(s, o, lse)


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
def test_device_schedule_equals_the_host_one(kind):
    rng = np.random.default_rng(1)
    for batch, h_q in ((1, 128), (37, 16), (700, 20), (5, 128)):
        new = rng.integers(0, 60 if batch > 100 else 900, batch)
        lens = rng.integers(0, 5000, batch)
        cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        md, groups = mla.get_mla_metadata_varlen_host(cu, lens, h_q, is_fp8_kvcache=kind == "fp8")
        plan = mla.get_mla_metadata_varlen(torch.from_numpy(cu).cuda(), torch.from_numpy(lens.astype(np.int32)).cuda(),
                                           int(cu[-1]), h_q, is_fp8_kvcache=kind == "fp8", num_parts=74)
        got = plan.data.cpu().numpy()
        assert np.array_equal(got[:74 * 8].reshape(74, 8), md)
        assert np.array_equal(got[74 * 8:74 * 8 + groups.size].reshape(-1, 8), groups)


def test_schedule_too_large_for_shared_memory():
    # 40,000 groups: the cost prefixes live behind the table
    cu = np.array([0, 30000, 40000], np.int32)
    lens = np.array([30000, 12000], np.int32)
    md, groups = mla.get_mla_metadata_varlen_host(cu, lens, 128)
    plan = mla.get_mla_metadata_varlen(torch.from_numpy(cu).cuda(), torch.from_numpy(lens).cuda(), 40000, 128, num_parts=74)
    got = plan.data.cpu().numpy()
    assert np.array_equal(got[:74 * 8].reshape(74, 8), md)
    assert np.array_equal(got[74 * 8:74 * 8 + groups.size].reshape(-1, 8), groups)


@pytest.mark.parametrize("cu", [[0, 5, 3], [0, 4, 99], [-1, 4, 5]])
def test_runs_that_do_not_split_the_tokens_are_recorded(cu):
    s = make("bf16", [4, 5], [40, 60], 16, seed=10)
    s["cu"] = torch.tensor(cu, dtype=torch.int32)
    ws = torch.zeros(mla.varlen_workspace_bytes(74), dtype=torch.uint8, device="cuda")
    out = torch.full((9, 16, DV), 7.0, dtype=torch.bfloat16, device="cuda")
    run(s, workspace=ws, out=out, num_parts=74)
    assert mla.read_device_status(ws) == 6 and (out == 7.0).all()
    s["cu"] = torch.tensor([0, 4, 9], dtype=torch.int32)
    check(s, *run(s, workspace=ws, num_parts=74))
    assert mla.read_device_status(ws) == 0


def test_bad_pages_and_long_lengths_are_recorded():
    s = make("bf16", [4, 5], [140, 260], 16, seed=11)
    ws = torch.zeros(mla.varlen_workspace_bytes(74), dtype=torch.uint8, device="cuda")
    good = s["table"].clone()
    s["table"][1, 2] = s["cache"].shape[0] + 5
    o, lse = run(s, workspace=ws, num_parts=74)
    assert mla.read_device_status(ws) == 6
    check(s, o, lse, only=[0])
    s["table"] = good
    for length in (10 ** 5, 2 ** 31 - 1):  # more pages than the table has: not followed past it
        s["seqlens"][1] = length
        run(s, workspace=ws, num_parts=74)
        assert mla.read_device_status(ws) == 6
    s["seqlens"][1] = -3       # a length below zero is an empty cache
    s["lens"][1] = 0
    check(s, *run(s, workspace=ws, num_parts=74))
    assert mla.read_device_status(ws) == 0


def test_bad_pages_of_a_dequantized_cache():
    s = make("fp8", [5, 9], [140, 260], 128, seed=21)
    ws = torch.zeros(mla.varlen_workspace_bytes(74), dtype=torch.uint8, device="cuda")
    good = s["table"].clone()
    s["table"][0, 1] = -1
    run(s, workspace=ws, num_parts=74)  # (its outputs are unspecified)
    assert mla.read_device_status(ws) == 6
    s["table"] = good
    check(s, *run(s, workspace=ws, num_parts=74))
    assert mla.read_device_status(ws) == 0


def test_dequantized_pages_are_the_pages_read_directly():
    # the same runs through the C entry point, with and without scratch
    import ctypes

    from mla_decode_attention_12_b200 import _lib
    s = make("fp8", [5, 9, 20], [140, 2600, 999], 128, seed=22)
    d = {k: v.cuda() for k, v in s.items() if isinstance(v, torch.Tensor)}
    plan = mla.get_mla_metadata_varlen(d["cu"], d["seqlens"], 34, 128, is_fp8_kvcache=True)
    ws = torch.zeros(mla.varlen_workspace_bytes(plan.num_parts), dtype=torch.uint8, device="cuda")
    lib = _lib.load()
    size = lib.mla_decode_varlen_scratch_bytes(3, 34, 128, d["table"].shape[1], 2)
    assert size > 0
    scratch = torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda")
    for sc in (scratch, None):
        o = torch.empty(34, 128, DV, dtype=torch.bfloat16, device="cuda")
        lse = torch.empty(34, 128, device="cuda")
        st = lib.mla_decode_varlen(
            d["q"].data_ptr(), 34, 128, 576, d["cache"].data_ptr(), d["cache"].shape[0], 64, 1, d["table"].data_ptr(), 3,
            d["table"].shape[1], d["seqlens"].data_ptr(), DV, 2, plan.data.data_ptr(), plan.num_parts, ctypes.c_float(0.0),
            o.data_ptr(), lse.data_ptr(), ws.data_ptr(), ws.numel(), None if sc is None else sc.data_ptr(), size,
            torch.cuda.current_stream().cuda_stream)
        assert st == 0
        torch.cuda.synchronize()
        check(s, o, lse)
    assert mla.read_device_status(ws) == 0


def test_two_graphs_replayed_on_two_streams():
    a, b = make("bf16", [1, 20], [4000, 900], 64, seed=12), make("bf16", [2], [6000], 128, seed=13)
    graphs = []
    for s in (a, b):
        dev = {k: v.cuda() for k, v in s.items() if isinstance(v, torch.Tensor)}
        run(s, dev=dev)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            res = run(s, dev=dev)
        graphs.append((graph, res, dev))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(10):
        for (graph, _, _), st in zip(graphs, streams):
            with torch.cuda.stream(st):
                graph.replay()
    torch.cuda.synchronize()
    for s, (_, res, _) in zip((a, b), graphs):
        check(s, *res)


def test_replay_follows_new_lengths_of_a_padded_batch():
    # one captured step, replayed with other lengths: the plan is part of the graph
    s = make("bf16", [1, 7, 0, 0], [300, 500, 0, 0], 32, seed=14, extra_q=6)
    s["table"] = torch.arange(40, dtype=torch.int32).view(4, 10)
    s["cache"] = random_cache("bf16", 40, 576, 15)
    dev = {k: v.cuda() for k, v in s.items() if isinstance(v, torch.Tensor)}
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        res = run(s, dev=dev)
    for new, lens in (([1, 7, 0, 0], [300, 500, 0, 0]), ([3, 1, 9, 1], [640, 33, 9, 64])):
        dev["cu"].copy_(torch.tensor([0] + list(np.cumsum(new)), dtype=torch.int32))
        dev["seqlens"].copy_(torch.tensor(lens, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        s.update(new=new, lens=lens)
        check(s, *res)


def test_refusals():
    s = make("bf16", [4, 5], [140, 260], 16, seed=16)
    d = {k: v.cuda() for k, v in s.items() if isinstance(v, torch.Tensor)}
    plan = mla.get_mla_metadata_varlen(d["cu"], d["seqlens"], 9, 16)

    def go(**over):
        a = {**d, "plan": plan, "causal": True, **over}
        return mla.flash_mla_varlen_with_kvcache(a["q"], a["cache"], a["table"], a["cu"], a["seqlens"], a.get("dv", DV), a["plan"],
                                                 a["causal"], a.get("fp8", False), out=a.get("out"), lse=a.get("lse"))

    go()
    for bad in (dict(q=d["q"].half()), dict(q=d["q"][..., :512]), dict(q=d["q"][:8]), dict(q=d["q"].transpose(0, 1)),
                dict(causal=False), dict(table=d["table"][:1]), dict(cu=d["cu"][:2]), dict(cu=d["cu"].long()), dict(fp8=True),
                dict(out=torch.empty(9, 16, 511, device="cuda")), dict(lse=torch.empty(8, 16, device="cuda")),
                dict(cache=d["cache"].cpu()), dict(seqlens=d["seqlens"].cpu())):
        with pytest.raises(ValueError):
            go(**bad)
    with pytest.raises(mla.MLAError):
        go(dv=256)
    with pytest.raises(ValueError):
        mla.get_mla_metadata_varlen(d["cu"], d["seqlens"], 9, 16, 2)
    other = mla.get_mla_metadata_varlen(d["cu"], d["seqlens"], 9, 32)
    with pytest.raises(ValueError):
        go(plan=other)
