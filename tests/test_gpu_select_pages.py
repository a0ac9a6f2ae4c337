"""mla_select_pages and flash_mla_page_sparse on the GPU: the choice against whole-number scores, the steps together."""
import math

import numpy as np
import pytest
import torch

import mla_decode_attention_12_b200 as mla
from cache_helpers import DTYPES, DV, HALF_STEP, PAGE, attend64, cache_rows64, random_cache, rotation_table, table_of

pytestmark = pytest.mark.gpu


def make(lens, s_q, heads, *, kind="bf16", d=576, seed=0, width=None, pages=None):
    g = torch.Generator().manual_seed(seed)
    table, n = table_of(lens, seed, width=width)
    return dict(q=torch.randn(len(lens), s_q, heads, d, generator=g).to(DTYPES[kind]), table=table,
                seqlens=torch.tensor(lens, dtype=torch.int32),
                keys=torch.randint(-127, 128, (n, d), generator=g).to(torch.int8), scales=torch.rand(n, generator=g) * 0.01 + 1e-3)


def scores_of(s, b, tok, pages):
    """Scores of one token's pages: whole numbers in int64, then float32 products as the header says."""
    q = s["q"][b, tok].float()
    scale = (q.abs().amax(-1, keepdim=True) * torch.tensor(1 / 127, dtype=torch.float32)).clamp(min=2.0 ** -126)
    whole = torch.round(q / scale).long()
    keys = s["keys"][pages].long()
    inner = (whole[:, None, :] * keys[None]).sum(-1) if whole.shape[0] * keys.shape[0] < 4096 else \
        torch.stack([(keys * w).sum(-1) for w in whole])
    best = (inner.float() * scale).amax(0)
    return (best * s["scales"][pages]).numpy()


def expected(s, topn, first, last, causal=True):
    batch, s_q = s["q"].shape[:2]
    table = np.full((batch * s_q, topn), -1, np.int32)
    lens = np.zeros(batch * s_q, np.int32)
    for b in range(batch):
        for tok in range(s_q):
            n = int(s["seqlens"][b])
            n = max(n - s_q + 1 + tok, 0) if causal else max(n, 0)
            pages = -(-n // PAGE)
            if pages == 0:
                continue
            phys = s["table"][b, :pages].long()
            chosen = set(range(pages))
            if pages > topn:
                sc = scores_of(s, b, tok, phys)
                forced = set(range(first)) | set(range(pages - last, pages))
                others = sorted((j for j in range(pages) if j not in forced), key=lambda j: (-sc[j], j))
                chosen = forced | set(others[:topn - len(forced)])
            chosen = sorted(chosen)
            table[b * s_q + tok, :len(chosen)] = phys[chosen].numpy()
            lens[b * s_q + tok] = (len(chosen) - 1) * PAGE + n - (pages - 1) * PAGE
    return table, lens


def run(s, topn, first=1, last=1, causal=True, status=None):
    d = {k: v.cuda() for k, v in s.items()}
    t, n = mla.mla_select_pages(d["q"], d["keys"], d["scales"], d["table"], d["seqlens"], topn, n_first=first, n_last=last,
                                causal=causal, status=status)
    return t.cpu().numpy(), n.cpu().numpy()


def check(s, topn, first=1, last=1, causal=True):
    got, want = run(s, topn, first, last, causal), expected(s, topn, first, last, causal)
    assert np.array_equal(got[1], want[1])
    assert np.array_equal(got[0], want[0])


@pytest.mark.parametrize("kind,d", [("bf16", 576), ("fp16", 576), ("bf16", 512), ("fp16", 512)])
@pytest.mark.parametrize("lens,s_q,heads,topn,first,last", [
    ([1], 1, 1, 1, 0, 1), ([64 * 20], 1, 128, 5, 1, 1), ([64 * 200 + 3, 70, 0, 5000], 2, 16, 8, 1, 2),
    ([64 * 128, 64 * 129, 64 * 257 - 1], 1, 100, 16, 0, 3), ([3, 64 * 40], 4, 20, 4, 2, 2), ([9000] * 5, 1, 33, 64, 0, 1),
    ([64 * 300 + 1, 64 * 7], 1, 96, 10, 1, 1),
])
def test_choice(kind, d, lens, s_q, heads, topn, first, last):
    check(make(lens, s_q, heads, kind=kind, d=d, seed=len(lens) + heads), topn, first, last)


def test_without_causal_mask():
    check(make([64 * 30 + 1, 64 * 30], 3, 16, seed=2), 6, 1, 1, causal=False)


def test_many_tokens_of_different_lengths():
    rng = np.random.default_rng(3)
    check(make([int(x) for x in rng.integers(0, 4000, 160)], 4, 8, seed=4), 7, 1, 1)


def test_long_contexts():
    check(make([64 * 5000 + 5, 64 * 2049], 1, 16, seed=5), 100, 1, 4)      # a CTA of 1024 threads
    check(make([64 * 17000 + 5], 1, 4, seed=6), 300, 1, 4)                # more pages than registers hold


def test_equal_scores_go_to_the_lower_page():
    s = make([64 * 300], 1, 16, seed=7)
    s["keys"][:] = s["keys"][0]
    s["scales"][:] = 0.5
    check(s, 20, 1, 1)
    s["keys"][::3] = 0       # zero scores, where the others are positive or negative
    check(s, 20, 0, 2)
    s["keys"][:] = 0
    s["scales"][::2] = -0.5  # zeros of both signs are equal
    check(s, 33, 1, 1)


def test_scores_far_apart_and_close_together():
    for outlier in (1e30, 3e38, 1e-30):  # all others share a few bins, or overflow both ways, or vanish
        s = make([64 * 700, 64 * 3000], 1, 16, seed=13)
        s["scales"][::97] = outlier
        check(s, 50, 1, 2)
    s = make([64 * 1500], 1, 4, seed=14)
    s["keys"][:] = s["keys"][0]
    s["scales"] = 1.0 + torch.arange(s["scales"].shape[0]) * 2.0 ** -23  # neighbours in float32
    check(s, 40, 0, 1)
    s["scales"][:] = 1e-45
    check(s, 40, 3, 3)
    check(s, 6, 3, 3)  # nothing competes


def test_zero_queries_and_scores_that_are_not_finite():
    s = make([64 * 50], 1, 16, seed=8)
    s["q"][:] = 0
    check(s, 9)
    s = make([64 * 50], 1, 16, seed=9)
    bad = s["table"][0, [3, 20, 30]].long()
    s["scales"][bad[0]], s["scales"][bad[1]], s["scales"][bad[2]] = math.nan, math.inf, -math.inf
    t, n = run(s, 10, 1, 2)
    assert n[0] == 640 and (t[0] >= 0).all() and len(set(t[0])) == 10
    assert t[0][-1] == s["table"][0, 49] and t[0][-2] == s["table"][0, 48] and t[0][0] == s["table"][0, 0]
    assert int(bad[0]) not in t[0]


def test_bad_entries_and_long_lengths_are_recorded():
    s = make([64 * 30, 64 * 30], 1, 16, seed=10)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    s["table"][0, 7] = 10 ** 6
    want = expected({**s, "table": s["table"].clamp(max=s["keys"].shape[0] - 1)}, 8, 1, 1)
    t, n = run(s, 8, status=status)
    assert int(status) == 6 and np.array_equal(t[1], want[0][1]) and np.array_equal(n, want[1])
    s = make([64 * 30, 64 * 30], 1, 16, seed=10)
    s["seqlens"][1] = 10 ** 9
    status.zero_()
    t, n = run(s, 8, status=status)
    s["seqlens"][1] = 64 * 30
    want = expected(s, 8, 1, 1)
    assert int(status) == 6 and np.array_equal(t, want[0]) and np.array_equal(n, want[1])
    s["seqlens"][0] = -2 ** 31
    t, n = run(s, 8)
    assert n[0] == 0 and (t[0] == -1).all()


def test_graph_replay_follows_new_lengths():
    s = make([64 * 90, 64 * 10], 2, 32, seed=11)
    s["table"][1] = s["table"][0]
    d = {k: v.cuda() for k, v in s.items()}

    def step():
        return mla.mla_select_pages(d["q"], d["keys"], d["scales"], d["table"], d["seqlens"], 6, n_first=1, n_last=2)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        res = step()
    for lens in ([64 * 90, 64 * 10], [64 * 3, 64 * 77 + 9], [0, 1]):
        d["seqlens"].copy_(torch.tensor(lens, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        s["seqlens"] = torch.tensor(lens, dtype=torch.int32)
        want = expected(s, 6, 1, 2)
        assert np.array_equal(res[0].cpu().numpy(), want[0]) and np.array_equal(res[1].cpu().numpy(), want[1])


def test_side_streams_at_once():
    cases = [make([64 * 1000 + k], 1, 64, seed=20 + k) for k in range(3)]
    devs = [{k: v.cuda() for k, v in s.items()} for s in cases]
    torch.cuda.synchronize()
    streams, res = [torch.cuda.Stream() for _ in cases], [None] * 3
    for _ in range(5):
        for i, (d, st) in enumerate(zip(devs, streams)):
            with torch.cuda.stream(st):
                res[i] = mla.mla_select_pages(d["q"], d["keys"], d["scales"], d["table"], d["seqlens"], 12)
    torch.cuda.synchronize()
    for s, (t, n) in zip(cases, res):
        want = expected(s, 12, 1, 1)
        assert np.array_equal(t.cpu().numpy(), want[0]) and np.array_equal(n.cpu().numpy(), want[1])


def test_captured_sparse_decodes_replayed_at_once():
    """Two graphs of flash_mla_page_sparse, captured on one stream and replayed on two."""
    work = []
    for seed, lens, heads in ((31, [64 * 60, 64 * 33 + 5], 128), (32, [64 * 500], 64)):
        s = make(lens, 1, heads, seed=seed)
        cache = random_cache("bf16", s["keys"].shape[0], 576, seed)
        d = {k: v.cuda() for k, v in s.items()}
        dc = cache.cuda()

        def step(d=d, dc=dc):
            return mla.flash_mla_page_sparse(d["q"], dc, d["table"], d["seqlens"], DV, d["keys"], d["scales"], 32)

        step()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            res = step()
        work.append((s, cache, graph, res, step))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(10):
        for (_, _, graph, _, _), st in zip(work, streams):
            with torch.cuda.stream(st):
                graph.replay()
    torch.cuda.synchronize()
    u = HALF_STEP[torch.bfloat16]
    for s, cache, _, (o, lse), _ in work:
        t, n = expected(s, 32, 1, 1)
        rows = cache_rows64(cache, False)
        for b in range(len(n)):
            i = torch.arange(int(n[b]))
            kv = rows[torch.from_numpy(t[b]).long()[i // PAGE] * PAGE + i % PAGE]
            q = s["q"][b, 0]
            vis = torch.full((q.shape[0],), int(n[b]))
            want, want_l = attend64(q, kv, vis, 576 ** -0.5)
            size = torch.softmax(q.double() @ kv.T * 576 ** -0.5, -1) @ kv[:, :DV].abs()
            assert ((o[b, 0].cpu().double() - want).abs() <= (u + 2.0 ** -12) * size + u * want.abs() * (1 + 2.0 ** -7)).all()
            assert ((lse[b, 0].cpu().double() - want_l).abs() <= 2.0 ** -14 * (1 + want_l.abs())).all()


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
def test_a_serving_step(kind):
    """Append a prompt in two runs, attend it, keep the page keys, then decode over the chosen pages."""
    heads, batch, fp8 = 16, 2, kind == "fp8"
    g = torch.Generator().manual_seed(1)
    total = [64 * 12 + 20, 64 * 9]
    table, pages = table_of([n + 64 for n in total], 2)
    table_d = table.cuda()
    cache = torch.zeros(pages, PAGE, 1, 656, dtype=torch.uint8, device="cuda") if fp8 else \
        torch.zeros(pages, PAGE, 1, 576, dtype=torch.bfloat16, device="cuda")
    keys, scales = torch.zeros(pages, 576, dtype=torch.int8, device="cuda"), torch.zeros(pages, device="cuda")
    cos_sin = rotation_table(2000).cuda()
    weight = (1 + 0.1 * torch.randn(DV, generator=g)).bfloat16().cuda()
    length = [0, 0]

    def step(new):
        """One layer's work on `new` tokens per request; returns the queries and the ragged attention's result."""
        before, q_at = list(length), [0] + list(np.cumsum(new))
        pos = torch.cat([torch.arange(length[b], length[b] + new[b]) for b in range(batch)])
        slots = torch.cat([table[b].long()[(i := torch.arange(length[b], length[b] + new[b])) // PAGE] * PAGE + i % PAGE
                           for b in range(batch)]).to(torch.int32)
        for b in range(batch):
            length[b] += new[b]
        down = torch.randn(len(pos), 576, generator=g).bfloat16().cuda()
        q = torch.randn(len(pos), heads, 576, generator=g).bfloat16().cuda()
        mla.mla_append_kvcache(down[:, :DV], down[:, DV:], pos.to(torch.int32).cuda(), cos_sin, slots.cuda(), cache,
                               norm_weight=weight, q_pe=q[..., DV:], q=q, is_fp8_kvcache=fp8)
        cu = torch.tensor(q_at, dtype=torch.int32, device="cuda")
        lens = torch.tensor(length, dtype=torch.int32, device="cuda")
        plan = mla.get_mla_metadata_varlen(cu, lens, len(pos), heads, is_fp8_kvcache=fp8)
        o, lse = mla.flash_mla_varlen_with_kvcache(q, cache, table_d, cu, lens, DV, plan, is_fp8_kvcache=fp8)
        mla.mla_summarize_pages(cache, table_d, torch.tensor(before, dtype=torch.int32, device="cuda"), lens, keys, scales,
                                is_fp8_kvcache=fp8)
        return q, o, lse

    u = HALF_STEP[torch.bfloat16]

    def close(o, lse, q, kv, n_vis):
        want, want_l = attend64(q, kv, n_vis, 576 ** -0.5)
        x = (q.double() @ kv.T * 576 ** -0.5).masked_fill(torch.arange(kv.shape[0])[None] >= n_vis[:, None], -torch.inf)
        tol = (u + 2.0 ** -12) * (torch.softmax(x, -1) @ kv[:, :DV].abs()) + u * want.abs() * (1 + 2.0 ** -7)
        assert ((o.cpu().double() - want).abs() <= tol).all()
        assert ((lse.cpu().double() - want_l).abs() <= 2.0 ** -14 * (1 + want_l.abs())).all()

    for new in ([500, 64 * 9 - 3], [64 * 12 + 20 - 500, 3]):
        q, o, lse = step(new)
        rows = cache_rows64(cache, fp8)
        at = 0
        for b in range(batch):
            i = torch.arange(length[b])
            kv = rows[table[b].long()[i // PAGE] * PAGE + i % PAGE]
            picks = torch.tensor(sorted({0, new[b] // 2, new[b] - 1}))
            n_vis = (length[b] - new[b] + 1 + picks).repeat_interleave(heads)
            close(o[at + picks].reshape(-1, DV), lse[at + picks].reshape(-1), q[at + picks].cpu().reshape(-1, 576), kv, n_vis)
            at += new[b]
    # decode one token over 5 of the 13 and 10 pages
    q, o_all, lse_all = step([1, 1])
    lens = torch.tensor(length, dtype=torch.int32, device="cuda")
    o, lse = mla.flash_mla_page_sparse(q.view(2, 1, heads, 576), cache, table_d, lens, DV, keys, scales, 5, n_first=1, n_last=2,
                                       is_fp8_kvcache=fp8)
    got_t, got_n = mla.mla_select_pages(q.view(2, 1, heads, 576), keys, scales, table_d, lens, 5, n_first=1, n_last=2)
    s = dict(q=q.view(2, 1, heads, 576).cpu(), table=table, seqlens=lens.cpu(), keys=keys.cpu(), scales=scales.cpu())
    want_t, want_n = expected(s, 5, 1, 2)
    assert np.array_equal(got_t.cpu().numpy(), want_t) and np.array_equal(got_n.cpu().numpy(), want_n)
    rows = cache_rows64(cache, fp8)
    for b in range(batch):
        n = int(want_n[b])
        i = torch.arange(n)
        kv = rows[torch.from_numpy(want_t[b]).long()[i // PAGE] * PAGE + i % PAGE]
        close(o[b].reshape(-1, DV), lse[b].reshape(-1), q[b].cpu(), kv, torch.full((heads,), n))
    # with room for every page it is the dense result
    o, lse = mla.flash_mla_page_sparse(q.view(2, 1, heads, 576), cache, table_d, lens, DV, keys, scales, 64, is_fp8_kvcache=fp8)
    for b in range(batch):
        i = torch.arange(length[b])
        kv = rows[table[b].long()[i // PAGE] * PAGE + i % PAGE]
        close(o[b].reshape(-1, DV), lse[b].reshape(-1), q[b].cpu(), kv, torch.full((heads,), length[b]))


def test_refusals():
    s = make([640, 640], 1, 16, seed=12)
    d = {k: v.cuda() for k, v in s.items()}

    def go(topn=4, first=1, last=1, **over):
        a = {**d, **over}
        return mla.mla_select_pages(a["q"], a["keys"], a["scales"], a["table"], a["seqlens"], topn, n_first=first, n_last=last)

    go()
    for bad in (dict(q=d["q"].float()), dict(q=d["q"][0]), dict(keys=d["keys"][:, :512]), dict(keys=d["keys"].short()),
                dict(scales=d["scales"][:3]), dict(table=d["table"][:1]), dict(seqlens=d["seqlens"].long()), dict(q=d["q"].cpu())):
        with pytest.raises(ValueError):
            go(**bad)
    for bad in (dict(topn=0), dict(topn=1), dict(last=0), dict(first=-1), dict(topn=5, first=3, last=3)):
        with pytest.raises(mla.MLAError):
            go(**bad)
    with pytest.raises(mla.MLAError):
        mla.mla_select_pages(torch.zeros(1, 1, 129, 576, dtype=torch.bfloat16, device="cuda"), d["keys"], d["scales"], d["table"][:1],
                             d["seqlens"][:1], 4)
