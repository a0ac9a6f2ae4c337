"""The default workspace of captured calls: each graph has its own."""
import pytest
import torch

import mla_decode_attention_12_b200 as mla
from cache_helpers import DV, PAGE
from test_gpu_varlen import check, make, run

pytestmark = pytest.mark.gpu


def dense_step(s):
    """A decode step of s (runs of one token) through the dense decode, as a call that can be captured."""
    d = {k: v.cuda() for k, v in s.items() if isinstance(v, torch.Tensor)}
    b, heads = len(s["new"]), s["q"].shape[1]
    q = d["q"].view(b, 1, heads, -1)
    fp8 = s["kind"] == "fp8"

    def step():
        md, ns = mla.get_mla_metadata(d["seqlens"], heads, 1, is_fp8_kvcache=fp8)
        o, lse = mla.flash_mla_with_kvcache(q, d["cache"], d["table"], d["seqlens"], DV, md, ns, False, fp8, softmax_scale=s["scale"])
        return o.view(b, heads, DV), lse.view(b, heads)

    return step


def indexed_step(s):
    """The same by the token-level sparse decode: every cached row listed."""
    d = {k: v.cuda() for k, v in s.items() if isinstance(v, torch.Tensor)}
    b, heads, topk = len(s["new"]), s["q"].shape[1], max(s["lens"])
    ind = torch.full((b, 1, topk), -1, dtype=torch.int32)
    for r, n in enumerate(s["lens"]):
        i = torch.arange(n)
        ind[r, 0, :n] = (s["table"][r].long()[i // PAGE] * PAGE + i % PAGE).to(torch.int32)
    ind = ind.cuda()
    q = d["q"].view(b, 1, heads, -1)

    def step():
        md, ns = mla.get_mla_metadata(d["seqlens"], heads, 1, h_q=heads, topk=topk)
        o, lse = mla.flash_mla_with_kvcache(q, d["cache"], None, None, DV, md, ns, False, s["kind"] == "fp8", ind,
                                            softmax_scale=s["scale"])
        return o.view(b, heads, DV), lse.view(b, heads)

    return step


def captured(step):
    """(graph, its results, the step: it holds the inputs that the graph reads)"""
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        res = step()
    return graph, res, step


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("make_step", [dense_step, indexed_step])
def test_two_graphs_replayed_on_two_streams(make_step, kind):
    cases = [make(kind, [1, 1], [9000, 4000], 64, seed=61), make(kind, [1], [12000], 128, seed=62)]
    work = [captured(make_step(s)) for s in cases]  # captured without a call before
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(10):
        for (graph, _, _), st in zip(reversed(work), streams):
            with torch.cuda.stream(st):
                graph.replay()
    torch.cuda.synchronize()
    for s, (_, res, _) in zip(cases, work):
        check(s, *res)


def test_two_prefill_graphs_replayed_on_two_streams():
    cases = [make("bf16", [1] * 6, [3000] * 6, 64, seed=63), make("bf16", [1] * 3, [5000] * 3, 128, seed=64)]
    work = []
    for s in cases:
        kv = s["cache"].view(-1, 1, 576).cuda()
        n = len(s["new"])
        rows = torch.stack([s["table"][r].long()[torch.arange(s["lens"][r]) // PAGE] * PAGE + torch.arange(s["lens"][r]) % PAGE
                            for r in range(n)])
        q, ind = s["q"].cuda(), rows.to(torch.int32).view(n, 1, -1).contiguous().cuda()
        work.append(captured(lambda q=q, kv=kv, ind=ind, s=s: mla.flash_mla_sparse_fwd(q, kv, ind, s["scale"])))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(10):
        for (graph, _, _), st in zip(work, streams):
            with torch.cuda.stream(st):
                graph.replay()
    torch.cuda.synchronize()
    for s, (_, (out, _, lse2), _) in zip(cases, work):
        check(s, out, lse2 * 0.6931471805599453)


def test_eager_calls_after_a_capture():
    s = make("bf16", [1, 1], [9000, 4000], 64, seed=65)
    step = dense_step(s)
    graph, res, _ = captured(step)
    check(s, *step())
    graph.replay()
    torch.cuda.synchronize()
    check(s, *res)
    del graph, res
    check(s, *step())
    check(s, *run(s))
