"""Cases of the cache-side operators beside the MLA decode: what they compute in plain torch, and the library's calls.

Four operators of a serving step over the paged latent cache (pages of 64 tokens, rows of 512 latent and 64
position columns, 16-bit or "FP8 with scale"):

* ``append``: new tokens' latents are normalised, their position parts rotated, and both written (quantized for
  an FP8 cache) into the cache rows that ``slots`` names; the queries' position parts are rotated in the same pass.
* ``chunk``: attention of ragged runs of new tokens over the paged cache, causal from the bottom right.
* ``summarize``: one 8-bit key for every page that a step completed (the mean of its rows).
* ``select``: for each query token the pages whose keys score best, as a block table of its own.

``own`` false: plain torch.  ``own`` true: the calls of ``mla_decode_attention_12_b200``.
"""
import math
import random

import torch

own = False

PAGE = 64
DV = 512
ROPE = 64
FP8_ROW = 656  # 512 e4m3 values, 4 float32 scales, 64 bfloat16 position values
EPS = 1e-6
TINY = 2.0 ** -126  # the least scale of a block of an FP8 row
KINDS = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp8": torch.bfloat16}


# ---------------------------------------------------------------- cases
def listed():
    return [
        # one request's decode step on a rank with 16 heads: nothing but latency
        {"name": "append_one", "op": "append", "kind": "bf16", "tokens": 1, "heads": 16, "pages": 8, "positions": 4096,
         "pad": 0, "interleaved": True},
        # a decode step of 64 requests over an FP8 cache, 128 heads
        {"name": "append_step_fp8", "op": "append", "kind": "fp8", "tokens": 64, "heads": 128, "pages": 64,
         "positions": 131072, "pad": 5, "interleaved": True},
        # a long prompt's layer: 8192 tokens, 128 heads, 16-bit cache
        {"name": "append_prompt", "op": "append", "kind": "bf16", "tokens": 8192, "heads": 128, "pages": 160,
         "positions": 32768, "pad": 0, "interleaved": False},
        # three short ragged runs on a rank with 16 heads: the smallest attention call
        {"name": "chunk_short", "op": "chunk", "kind": "bf16", "batch": 3, "ones": 1, "heads": 16, "dqk": 576,
         "new_lo": 5, "new_hi": 17, "len_lo": 193, "len_hi": 256, "lens": 1},
        # 60 decoding requests and 2 prompts' pieces in one call
        {"name": "chunk_mixed", "op": "chunk", "kind": "bf16", "batch": 62, "ones": 60, "heads": 128, "dqk": 576,
         "new_lo": 200, "new_hi": 256, "len_lo": 1024, "len_hi": 8192, "lens": 2},
        # chunked prefill of four prompts
        {"name": "chunk_prompt", "op": "chunk", "kind": "bf16", "batch": 4, "ones": 0, "heads": 128, "dqk": 576,
         "new_lo": 900, "new_hi": 1024, "len_lo": 4096, "len_hi": 8192, "lens": 3},
        # pieces of eight prompts over an FP8 cache, 64 heads
        {"name": "chunk_fp8", "op": "chunk", "kind": "fp8", "batch": 8, "ones": 0, "heads": 64, "dqk": 576,
         "new_lo": 100, "new_hi": 260, "len_lo": 1024, "len_hi": 8192, "lens": 4},
        # fp16 rows without position columns, 64 heads, short pieces of 32 sequences
        {"name": "chunk_fp16_norope", "op": "chunk", "kind": "fp16", "batch": 32, "ones": 4, "heads": 64, "dqk": 512,
         "new_lo": 3, "new_hi": 60, "len_lo": 512, "len_hi": 16384, "lens": 5},
        # the decode step at which 64 requests' pages fill up, FP8 cache
        {"name": "summarize_step_fp8", "op": "summarize", "kind": "fp8", "batch": 64, "new_lo": 64, "new_hi": 64,
         "len_lo": 1024, "len_hi": 8192, "lens": 6},
        # four long prompts just read in
        {"name": "summarize_prompt", "op": "summarize", "kind": "bf16", "batch": 4, "new_lo": 8192, "new_hi": 65536,
         "len_lo": 65536, "len_hi": 65536, "lens": 7},
        # a few requests, 16 heads, two query tokens each
        {"name": "select_short", "op": "select", "kind": "bf16", "batch": 4, "s_q": 2, "heads": 16, "topn": 16,
         "first": 1, "last": 2, "len_lo": 2000, "len_hi": 8192, "lens": 8},
        # 64 long contexts, 128 heads
        {"name": "select_long", "op": "select", "kind": "bf16", "batch": 64, "s_q": 1, "heads": 128, "topn": 64,
         "first": 1, "last": 4, "len_lo": 16384, "len_hi": 131072, "lens": 9},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "chunk", "chunk", "summarize", "select"])
    kind = rng.choice(["bf16", "fp16", "fp8"])
    heads = rng.choice([8, 16, 20, 32, 64, 96, 128])
    lens = rng.randrange(1 << 30)
    if op == "append":
        tokens = _log(rng, 1, 8192)
        return {"op": op, "kind": kind, "tokens": tokens, "heads": heads, "pages": tokens // 64 + 1 + _log(rng, 1, 64),
                "positions": _log(rng, 1024, 131072), "pad": rng.randrange(0, 1 + tokens // 8),
                "interleaved": rng.random() < 0.5}
    if op == "chunk":
        batch = _log(rng, 1, 48)
        hi = _log(rng, 64, 16384)
        new = _log(rng, 1, min(hi, max(1, 1024 // batch)))
        return {"op": op, "kind": kind, "batch": batch, "ones": rng.randrange(0, batch + 1), "heads": heads,
                "dqk": 576 if kind == "fp8" else rng.choice([576, 512]), "new_lo": max(1, new // 2), "new_hi": new,
                "len_lo": max(new, hi // 4), "len_hi": hi, "lens": lens}
    if op == "summarize":
        hi = _log(rng, 64, 65536)
        new = _log(rng, 1, hi)
        return {"op": op, "kind": kind, "batch": max(1, min(64, 160000 // hi)), "new_lo": max(1, new // 2), "new_hi": new,
                "len_lo": new, "len_hi": hi, "lens": lens}
    hi = _log(rng, 256, 131072)
    first, last = rng.randrange(0, 3), rng.randrange(1, 5)
    return {"op": op, "kind": "bf16" if kind == "fp8" else kind, "batch": _log(rng, 1, 32), "s_q": rng.choice([1, 1, 2, 4]),
            "heads": heads, "topn": max(first + last, _log(rng, 4, 128)), "first": first, "last": last,
            "len_lo": max(1, hi // 8), "len_hi": hi, "lens": lens}


def _lengths(case):
    """(new tokens, cached tokens) of each request: of the case alone, so that work() knows them."""
    rng = random.Random(case["lens"])
    got = []
    for b in range(case["batch"]):
        new = 1 if b < case.get("ones", 0) else rng.randint(case.get("new_lo", 1), case.get("new_hi", 1))
        new = case.get("s_q", new)
        got.append((new, max(new, rng.randint(case["len_lo"], case["len_hi"]))))
    return got


def work(case):
    op, e = case["op"], 2
    row = FP8_ROW if case["kind"] == "fp8" else e * case.get("dqk", DV + ROPE)
    if op == "append":
        t, live = case["tokens"], case["tokens"] - case["pad"]
        moved = t * 2 * case["heads"] * ROPE * e            # the queries' position parts, in and out
        moved += live * ((DV + ROPE) * e + row)             # the new tokens, in and out
        moved += t * (2 * ROPE * 2 + 8) + DV * e            # angles, positions and slots, the norm's weights
        return {"bytes": moved, "flops": 6 * t * case["heads"] * ROPE // 2 + live * 5 * DV}
    lens = _lengths(case)
    if op == "chunk":
        rows = sum(n for n, _ in lens) * case["heads"]
        moved = sum(n for _, n in lens) * row + rows * ((case["dqk"] + DV) * e + 4)
        seen = sum(new * length - new * (new - 1) // 2 for new, length in lens) * case["heads"]
        return {"bytes": moved, "flops": 2 * (case["dqk"] + DV) * seen}
    if op == "summarize":
        pages = sum(length // PAGE - (length - new) // PAGE for new, length in lens)
        return {"bytes": pages * (PAGE * row + DV + ROPE + 4) + 8 * len(lens), "flops": pages * PAGE * (DV + ROPE)}
    pages = sum(-(-length // PAGE) for _, length in lens)
    tokens = case["batch"] * case["s_q"]
    d = DV + ROPE
    return {"bytes": pages * (d + 8) + tokens * (case["heads"] * d * e + 4 * case["topn"] + 4),
            "flops": 2 * pages * case["s_q"] * case["heads"] * d}


# ---------------------------------------------------------------- inputs
def _fp8_rows(n, g):
    """n "FP8 with scale" rows of latents of about unit size."""
    rows = torch.empty(n, FP8_ROW, dtype=torch.uint8, device="cuda")
    x = torch.randn(n, 4, 128, generator=g, device="cuda")
    scale = x.abs().amax(-1, keepdim=True) / 448
    rows[:, :DV].view(torch.float8_e4m3fn).copy_((x / scale).to(torch.float8_e4m3fn).view(n, DV))
    rows[:, DV:DV + 16].view(torch.float32).copy_(scale.view(n, 4))
    rows[:, DV + 16:].view(torch.bfloat16).copy_(torch.randn(n, ROPE, generator=g, device="cuda").bfloat16())
    return rows


def _cache(kind, pages, dqk, g):
    if kind == "fp8":
        return _fp8_rows(pages * PAGE, g).view(pages, PAGE, 1, FP8_ROW)
    return torch.randn(pages, PAGE, 1, dqk, generator=g, device="cuda", dtype=torch.float32).to(KINDS[kind])


def _tables(lens, g):
    """Block table of shuffled pages (-1 past a request's pages) and how many pages there are."""
    need = torch.tensor([-(-n // PAGE) for _, n in lens])
    total, most = int(need.sum()) + 1, max(1, int(need.max()))
    perm = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    at = (torch.cumsum(need, 0) - need)[:, None] + torch.arange(most)[None]
    table = perm[at.clamp(max=total - 1).cuda()]
    return table.masked_fill((torch.arange(most)[None] >= need[:, None]).cuda(), -1).contiguous(), total


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt, op = KINDS[case["kind"]], case["op"]
    fp8 = case["kind"] == "fp8"

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)

    if op == "append":
        t, h = case["tokens"], case["heads"]
        half = torch.arange(ROPE // 2, device="cuda", dtype=torch.float64)
        angle = torch.arange(case["positions"], device="cuda", dtype=torch.float64)[:, None] * 10000.0 ** (-half / (ROPE // 2))
        order = torch.randperm(case["pages"], generator=g, device="cuda")
        line = torch.arange(t, device="cuda")
        if t <= 256:  # a decode step: each token goes to a page of its own, or near it
            line = torch.randperm(case["pages"] * PAGE, generator=g, device="cuda")[:t]
        slots = (order[line // PAGE] * PAGE + line % PAGE).to(torch.int32)
        if case["pad"]:
            slots[t - case["pad"]:] = -1  # a batch padded to a captured graph's size
        down = normal(t, DV + ROPE).to(dt)       # what the down projection gives: latent, then position part
        up = normal(t, h, 128 + ROPE).to(dt)     # what the query projection gives for each head
        return {"op": op, "fp8": fp8, "interleaved": case["interleaved"], "latent": down[:, :DV], "k_pe": down[:, DV:],
                "q_pe": up[..., 128:], "weight": (1 + 0.1 * normal(DV)).to(dt), "slots": slots,
                "positions": torch.randint(0, case["positions"], (t,), generator=g, device="cuda", dtype=torch.int32),
                "cos_sin": torch.cat([angle.cos(), angle.sin()], 1).float().contiguous(),
                "q": normal(t, h, DV + ROPE).to(dt), "cache": _cache(case["kind"], case["pages"], DV + ROPE, g)}
    lens = _lengths(case)
    table, pages = _tables(lens, g)
    length = torch.tensor([n for _, n in lens], dtype=torch.int32, device="cuda")
    if op == "chunk":
        ends = torch.cumsum(torch.tensor([0] + [n for n, _ in lens]), 0)
        return {"op": op, "fp8": fp8, "lens": lens, "table": table, "length": length,
                "starts": ends.to(torch.int32).cuda(), "q": normal(int(ends[-1]), case["heads"], case["dqk"]).to(dt),
                "cache": _cache(case["kind"], pages, case["dqk"], g), "scale": 1 / math.sqrt(case["dqk"])}
    keys = torch.randint(-127, 128, (pages, DV + ROPE), generator=g, device="cuda", dtype=torch.int32).to(torch.int8)
    scales = torch.rand(pages, generator=g, device="cuda") * 0.01 + 0.001
    if op == "summarize":
        before = length - torch.tensor([n for n, _ in lens], dtype=torch.int32, device="cuda")
        return {"op": op, "fp8": fp8, "table": table, "before": before, "length": length, "keys": keys, "scales": scales,
                "cache": _cache(case["kind"], pages, DV + ROPE, g)}
    return {"op": op, "q": normal(case["batch"], case["s_q"], case["heads"], DV + ROPE).to(dt), "table": table,
            "length": length, "keys": keys, "scales": scales, "topn": case["topn"], "first": case["first"],
            "last": case["last"]}


# ---------------------------------------------------------------- one pass
def run(s):
    return {"append": _append, "chunk": _chunk, "summarize": _summarize, "select": _select}[s["op"]](s)


def _cache_parts(cache, fp8):
    """A cache as the values that it holds: 16-bit rows, or e4m3 latents, their scales and the position columns."""
    if not fp8:
        return [cache]
    return [cache[..., :DV].view(torch.float8_e4m3fn), cache[..., DV:DV + 16].view(torch.float32),
            cache[..., DV + 16:].view(torch.bfloat16)]


def _rotate(x, cos, sin, interleaved):
    a, b = (x[..., 0::2], x[..., 1::2]) if interleaved else (x[..., :ROPE // 2], x[..., ROPE // 2:])
    u, v = a * cos - b * sin, b * cos + a * sin
    return torch.stack([u, v], -1).flatten(-2) if interleaved else torch.cat([u, v], -1)


def _append(s):
    if own:
        import mla_decode_attention_12_b200 as mla

        mla.mla_append_kvcache(s["latent"], s["k_pe"], s["positions"], s["cos_sin"], s["slots"], s["cache"],
                               norm_weight=s["weight"], norm_eps=EPS, q_pe=s["q_pe"], q=s["q"],
                               interleaved=s["interleaved"], is_fp8_kvcache=s["fp8"])
        return {"cache": _cache_parts(s["cache"], s["fp8"]), "q": s["q"]}
    angles = s["cos_sin"][s["positions"]]
    cos, sin = angles[:, :ROPE // 2], angles[:, ROPE // 2:]
    s["q"][..., DV:] = _rotate(s["q_pe"].float(), cos[:, None], sin[:, None], s["interleaved"]).to(s["q"].dtype)
    x = s["latent"].float()
    y = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * s["weight"].float()
    k = _rotate(s["k_pe"].float(), cos, sin, s["interleaved"]).to(s["q"].dtype)
    live = s["slots"] >= 0
    at = s["slots"][live].long()
    if not s["fp8"]:
        s["cache"].view(-1, DV + ROPE)[at] = torch.cat([y.to(k.dtype), k], 1)[live]
        return {"cache": _cache_parts(s["cache"], False), "q": s["q"]}
    blocks = y.view(-1, 4, 128)
    scale = (blocks.abs().amax(-1, keepdim=True) * (1 / 448)).clamp(min=TINY)
    codes = (blocks / scale).to(torch.float8_e4m3fn).view(torch.uint8).view(-1, DV)
    rows = torch.cat([codes, scale.view(-1, 4).view(torch.uint8), k.view(torch.uint8)], 1)
    s["cache"].view(-1, FP8_ROW)[at] = rows[live]
    return {"cache": _cache_parts(s["cache"], True), "q": s["q"]}


def _rows(cache, pages, fp8):
    """The rows of the pages, in 32 bits: an FP8 row's latents are bfloat16(code * scale), as the format says."""
    got = cache[pages.long()].flatten(0, -2)
    if not fp8:
        return got.float()
    codes, scale, rope = _cache_parts(got, True)
    return torch.cat([(codes.float().view(-1, 4, 128) * scale[..., None]).bfloat16().view(-1, DV).float(), rope.float()], 1)


def _chunk(s):
    if own:
        import mla_decode_attention_12_b200 as mla

        plan = mla.get_mla_metadata_varlen(s["starts"], s["length"], s["q"].shape[0], s["q"].shape[1], causal=True,
                                           is_fp8_kvcache=s["fp8"])
        return mla.flash_mla_varlen_with_kvcache(s["q"], s["cache"], s["table"], s["starts"], s["length"], DV, plan,
                                                 causal=True, softmax_scale=s["scale"], is_fp8_kvcache=s["fp8"])
    heads = s["q"].shape[1]
    o = torch.empty(s["q"].shape[0], heads, DV, dtype=s["q"].dtype, device="cuda")
    lse = torch.empty(s["q"].shape[0], heads, device="cuda")
    at = 0
    for b, (new, length) in enumerate(s["lens"]):  # request by request: padding them to one size would cost more
        k = _rows(s["cache"], s["table"][b, :-(-length // PAGE)], s["fp8"])[:length]
        x = s["q"][at:at + new].float().flatten(0, 1) @ k.T * s["scale"]
        sees = length - new + torch.arange(new, device="cuda").repeat_interleave(heads)
        x.masked_fill_(torch.arange(length, device="cuda")[None] > sees[:, None], -math.inf)
        m = x.amax(1, keepdim=True)
        p = torch.exp(x - m)
        total = p.sum(1, keepdim=True)
        o[at:at + new] = ((p @ k[:, :DV]) / total).view(new, heads, DV).to(o.dtype)
        lse[at:at + new] = (m + torch.log(total)).view(new, heads)
        at += new
    return o, lse


def _summarize(s):
    if own:
        import mla_decode_attention_12_b200 as mla

        mla.mla_summarize_pages(s["cache"], s["table"], s["before"], s["length"], s["keys"], s["scales"],
                                is_fp8_kvcache=s["fp8"])
    else:
        j = torch.arange(s["table"].shape[1], device="cuda")[None]
        pages = s["table"][(j >= (s["before"] // PAGE)[:, None]) & (j < (s["length"] // PAGE)[:, None])]
        # in 64 bits: a mean next to the border between two 8-bit values has to fall on the right side of it
        mean = (_rows(s["cache"], pages, s["fp8"]).view(-1, PAGE, DV + ROPE).double().sum(1) / PAGE).float()
        scale = (mean.abs().amax(1, keepdim=True) * (1 / 127)).clamp(min=TINY)
        s["keys"][pages.long()] = torch.round(mean / scale).to(torch.int8)
        s["scales"][pages.long()] = scale[:, 0]
    return s["keys"], s["scales"]


def _select(s):
    if own:
        import mla_decode_attention_12_b200 as mla

        return mla.mla_select_pages(s["q"], s["keys"], s["scales"], s["table"], s["length"], s["topn"],
                                    n_first=s["first"], n_last=s["last"])
    batch, s_q, heads, d = s["q"].shape
    most, topn = s["table"].shape[1], s["topn"]
    q = s["q"].float()
    scale = (q.abs().amax(-1, keepdim=True) * (1 / 127)).clamp(min=TINY)
    whole = torch.round(q / scale)                                   # 8-bit queries, one scale for each head
    pages = s["table"].clamp(min=0).long()
    products = whole.view(batch, s_q * heads, d) @ s["keys"][pages].float().transpose(1, 2)  # whole numbers below 2^24
    score = (products.view(batch, s_q, heads, most) * scale).amax(2) * s["scales"][pages][:, None]
    sees = s["length"][:, None] - s_q + 1 + torch.arange(s_q, device="cuda")[None]
    sees = sees.clamp(min=0)
    n = ((sees + PAGE - 1) // PAGE)[..., None]
    j = torch.arange(most, device="cuda")
    score = score.masked_fill((j < s["first"]) | (j >= n - s["last"]), math.inf).masked_fill(j >= n, -math.inf)
    best = torch.sort(score, dim=-1, descending=True, stable=True).indices[..., :topn]
    got = best.shape[-1]
    best = torch.where(best < n, best, most).sort(-1).values
    table = torch.full((batch * s_q, topn), -1, dtype=torch.int32, device="cuda")
    mine = s["table"][:, None].expand(-1, s_q, -1)
    table[:, :got] = torch.where(best < most, mine.gather(2, best.clamp(max=most - 1)), -1).view(-1, got)
    lens = torch.where(n[..., 0] > 0, (n[..., 0].clamp(max=topn) - 1) * PAGE + sees - (n[..., 0] - 1) * PAGE, 0)
    return table, lens.view(-1).to(torch.int32)


# ---------------------------------------------------------------- the definitions in 64 bits
def _e4m3(x):
    """The e4m3 value next to each of x (|x| <= 448), ties to the even one."""
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(x / step) * step


def _exact_rows(cache, fp8):
    if not fp8:
        return cache.double().view(-1, cache.shape[-1])
    flat = cache.view(-1, FP8_ROW)
    codes = flat[:, :DV].view(torch.float8_e4m3fn).float()
    scale = flat[:, DV:DV + 16].view(torch.float32).repeat_interleave(128, 1)
    return torch.cat([(codes * scale).bfloat16().double(), flat[:, DV + 16:].view(torch.bfloat16).double()], 1)


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "append":
        pos = s["positions"].long()
        turn = torch.complex(s["cos_sin"][pos, :ROPE // 2].double(), s["cos_sin"][pos, ROPE // 2:].double())

        def rotated(x, t):
            x = x.double()
            pairs = x.unflatten(-1, (ROPE // 2, 2)) if s["interleaved"] else x.unflatten(-1, (2, ROPE // 2)).transpose(-1, -2)
            z = torch.view_as_real(torch.complex(pairs[..., 0].contiguous(), pairs[..., 1].contiguous()) * t)
            return (z if s["interleaved"] else z.transpose(-1, -2)).flatten(-2)

        q = s["q"].double()
        q[..., DV:] = rotated(s["q_pe"], turn[:, None])
        x = s["latent"].double()
        y = x / torch.sqrt((x * x).sum(-1, keepdim=True) / DV + EPS) * s["weight"].double()
        k = rotated(s["k_pe"], turn)
        live = s["slots"] >= 0
        at = s["slots"][live].long()
        if not s["fp8"]:
            cache = s["cache"].double()
            cache.view(-1, DV + ROPE)[at] = torch.cat([y, k], 1)[live]
            return {"cache": [cache], "q": q}
        parts = [p.double() for p in _cache_parts(s["cache"], True)]
        scale = (y.view(-1, 4, 128).abs().amax(-1) / 448).clamp(min=TINY)
        parts[0].view(-1, DV)[at] = _e4m3(y / scale.repeat_interleave(128, 1))[live]
        parts[1].view(-1, 4)[at] = scale[live]
        parts[2].view(-1, ROPE)[at] = k[live]
        return {"cache": parts, "q": q}
    if s["op"] == "chunk":
        rows = _exact_rows(s["cache"], s["fp8"])
        heads = s["q"].shape[1]
        o = torch.zeros(*s["q"].shape[:2], DV, dtype=torch.float64, device="cuda")
        lse = torch.zeros(*s["q"].shape[:2], dtype=torch.float64, device="cuda")
        at = 0
        for b, (new, length) in enumerate(s["lens"]):
            i = torch.arange(length, device="cuda")
            kv = rows[s["table"][b].long()[i // PAGE] * PAGE + i % PAGE]
            for t0 in range(0, new, 64):
                t1 = min(new, t0 + 64)
                x = torch.einsum("thd,jd->thj", s["q"][at + t0:at + t1].double(), kv) * s["scale"]
                hidden = i[None] >= (length - new + 1 + torch.arange(t0, t1, device="cuda"))[:, None]
                x = x.masked_fill(hidden[:, None], -math.inf)
                lse[at + t0:at + t1] = torch.logsumexp(x, -1)
                o[at + t0:at + t1] = torch.einsum("thj,jd->thd", torch.softmax(x, -1), kv[:, :DV])
            at += new
        return o, lse
    if s["op"] == "summarize":
        rows = _exact_rows(s["cache"], s["fp8"]).view(-1, PAGE, DV + ROPE)
        scales = s["scales"].double()
        before, length = s["before"].tolist(), s["length"].tolist()
        touched = [s["table"][b, before[b] // PAGE:length[b] // PAGE] for b in range(len(length))]
        touched = torch.cat(touched).long()
        mean = rows[touched].sum(1) / PAGE
        scales[touched] = (mean.abs().amax(1) / 127).clamp(min=TINY)
        return None, scales  # the keys are whole numbers
    return None  # whole numbers alone: the pages chosen
