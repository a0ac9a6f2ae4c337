"""mla_append_kvcache on the GPU against its formula in 64 bits."""
import pytest
import torch

import mla_decode_attention_12_b200 as mla
from cache_helpers import DTYPES, DV, FP8_ROW, HALF_STEP, PAGE, fp8_parts, norm64, random_cache, rotate64, rotation_table

pytestmark = pytest.mark.gpu


def make(kind, tokens, heads, *, pages=None, norm=True, pad=0, seed=0, positions=500, amp=1.0, d=576):
    g = torch.Generator().manual_seed(seed)
    dt = DTYPES[kind]
    pages = pages or tokens // PAGE + 2
    slots = torch.randperm(pages * PAGE, generator=g)[:tokens].to(torch.int32)
    if pad:
        slots[torch.randperm(tokens, generator=g)[:pad]] = -1
    down = (amp * torch.randn(tokens, 576, generator=g)).to(dt)
    up = torch.randn(tokens, heads, 192, generator=g).to(dt)
    return dict(kind=kind, latent=down[:, :DV], k_pe=down[:, DV:] if d == 576 else None, q_pe=up[..., 128:],
                q=torch.randn(tokens, heads, 576, generator=g).to(dt), slots=slots,
                weight=(1 + 0.2 * torch.randn(DV, generator=g)).to(dt) if norm else None,
                positions=torch.randint(0, positions, (tokens,), generator=g, dtype=torch.int32),
                cos_sin=rotation_table(positions), cache=random_cache(kind, pages, d, seed + 1))


def call(s, *, interleaved=True, queries=True, eps=1e-6, status=None):
    """Runs the operator on copies of the inputs that keep their strides; returns (cache, q) on the CPU."""
    def gpu(t):
        if t is None:
            return None
        base = t if t._base is None else t._base
        moved = base.cuda()
        return moved if t is base else moved.as_strided(t.shape, t.stride(), t.storage_offset())

    cache, q = gpu(s["cache"]), gpu(s["q"]) if queries else None
    mla.mla_append_kvcache(gpu(s["latent"]), gpu(s["k_pe"]), gpu(s["positions"]), gpu(s["cos_sin"]), gpu(s["slots"]), cache,
                           norm_weight=gpu(s["weight"]), norm_eps=eps, q_pe=gpu(s["q_pe"]) if queries else None, q=q,
                           interleaved=interleaved, is_fp8_kvcache=s["kind"] == "fp8", status=status)
    torch.cuda.synchronize()
    return cache.cpu(), None if q is None else q.cpu()


def check_rows(s, cache, interleaved, eps, written):
    """Written rows against the formula; every other row bit for bit as it was."""
    dt = DTYPES[s["kind"]]
    half = HALF_STEP[dt]
    y = norm64(s["latent"], s["weight"], eps)
    # float32 arithmetic of y: 21 additions deep, a reciprocal square root and two products: < 2^-18 of y
    tol_y = (half + 2.0 ** -18) * y.abs() + 2.0 ** -25
    rows = s["slots"][written].long()
    flat, old = cache.reshape(-1, cache.shape[-1]), s["cache"].reshape(-1, s["cache"].shape[-1])
    others = torch.ones(flat.shape[0], dtype=torch.bool)
    others[rows] = False
    assert torch.equal(flat[others].view(torch.uint8), old[others].view(torch.uint8))
    if s["k_pe"] is not None:
        k, size = rotate64(s["k_pe"], s["cos_sin"][s["positions"].long()], interleaved)
        tol_k = half * k.abs() + 2.0 ** -22 * size + 2.0 ** -25  # two products and a sum in float32
    if s["kind"] == "fp8":
        codes, scale, rope = (p[rows] for p in fp8_parts(cache))
        want = (y.view(-1, 4, 128).abs().amax(-1) * (1 / 448)).clamp(min=2.0 ** -126)[written]
        assert (scale - want).abs().le(2.0 ** -17 * want).all()
        yw = y[written].view(-1, 4, 128)
        got = codes.view(-1, 4, 128) * scale[..., None]
        # half a step of e4m3: 2^-4 of the value, 2^-10 scales below the smallest normal code
        tol = torch.maximum(2.0 ** -4 * yw.abs(), 2.0 ** -10 * want[..., None]) * (1 + 2.0 ** -8)
        assert (got - yw).abs().le(tol).all()
        assert codes.abs().max() <= 448
    else:
        assert (flat[rows, :DV].double() - y[written]).abs().le(tol_y[written]).all()
        rope = flat[rows, DV:].double()
    if s["k_pe"] is not None:
        assert (rope - k[written]).abs().le(tol_k[written]).all()


def check_queries(s, q, interleaved, rotated=None):
    half = HALF_STEP[DTYPES[s["kind"]]]
    assert torch.equal(q[..., :DV], s["q"][..., :DV])
    want, size = rotate64(s["q_pe"], s["cos_sin"][s["positions"].long()][:, None], interleaved)
    err = (q[..., DV:].double() - want).abs()
    ok = err <= half * want.abs() + 2.0 ** -22 * size + 2.0 ** -25
    if rotated is not None:
        assert torch.equal(q[~rotated], s["q"][~rotated])
        ok = ok[rotated]
    assert ok.all()


@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("kind", ["bf16", "fp16", "fp8"])
@pytest.mark.parametrize("tokens,heads,pad", [(1, 1, 0), (3, 16, 1), (129, 5, 20), (64, 128, 0), (1000, 20, 3)])
def test_rows_and_queries(kind, tokens, heads, pad, interleaved):
    s = make(kind, tokens, heads, pad=pad, seed=tokens)
    cache, q = call(s, interleaved=interleaved)
    check_rows(s, cache, interleaved, 1e-6, s["slots"] >= 0)
    check_queries(s, q, interleaved)


@pytest.mark.parametrize("kind", ["bf16", "fp16", "fp8"])
def test_no_norm_no_queries(kind):
    s = make(kind, 77, 4, norm=False, seed=5)
    cache, _ = call(s, queries=False)
    check_rows(s, cache, True, 0.0, s["slots"] >= 0)


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
def test_rows_without_position_columns(kind):
    s = make(kind, 70, 4, seed=6, d=512)
    cache, _ = call(s, queries=False)
    check_rows(s, cache, True, 1e-6, s["slots"] >= 0)


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("amp", [0.0, 2.0 ** -40, 2.0 ** 40])
def test_tiny_and_large_latents(kind, amp):
    # zeros (scale 2^-126, codes 0), values whose squares underflow next to eps, large ones
    s = make(kind, 9, 2, seed=7, amp=amp, norm=amp > 0)
    cache, _ = call(s, queries=False)
    check_rows(s, cache, True, 1e-6, s["slots"] >= 0)


def test_all_padding_writes_nothing():
    s = make("bf16", 40, 3, seed=8)
    s["slots"][:] = -7
    cache, q = call(s)
    assert torch.equal(cache, s["cache"])
    check_queries(s, q, True)


def test_no_tokens():
    s = make("fp8", 0, 3, pages=2, seed=8)
    cache, _ = call(s)
    assert torch.equal(cache, s["cache"])


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
def test_bad_slots_and_positions_are_skipped_and_recorded(kind):
    s = make(kind, 50, 6, seed=9)
    good_slots, good_pos = s["slots"].clone(), s["positions"].clone()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    call(s, status=status)
    assert int(status) == 0
    s["slots"][3] = s["cache"].shape[0] * PAGE  # one row past the cache
    s["slots"][4] = 2 ** 31 - 1
    s["positions"][10] = 500                    # one past the table
    s["positions"][11] = -1
    written = torch.ones(50, dtype=torch.bool)
    written[[3, 4, 10, 11]] = False
    cache, q = call(s, status=status)
    assert int(status) == 6
    rotated = torch.ones(50, dtype=torch.bool)
    rotated[[10, 11]] = False
    s["slots"], s["positions"] = good_slots, good_pos
    check_rows(s, cache, True, 1e-6, written)
    check_queries(s, q, True, rotated)
    s["slots"][3] = 10 ** 6
    call(s)  # without a status word the row is skipped all the same


@pytest.mark.parametrize("interleaved", [True, False])
def test_rotation_in_place_and_transposed_queries(interleaved):
    s = make("bf16", 33, 12, seed=10)
    s["q"][..., DV:] = s["q_pe"]
    dev = {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in s.items()}
    q = dev["q"].clone()
    mla.mla_append_kvcache(dev["latent"], dev["k_pe"], dev["positions"], dev["cos_sin"], dev["slots"], dev["cache"],
                           norm_weight=dev["weight"], q_pe=q[..., DV:], q=q, interleaved=interleaved)
    check_queries(s, q.cpu(), interleaved)
    qt = dev["q"].transpose(0, 1).contiguous().transpose(0, 1)  # heads outside tokens
    mla.mla_append_kvcache(dev["latent"], dev["k_pe"], dev["positions"], dev["cos_sin"], dev["slots"], dev["cache"],
                           norm_weight=dev["weight"], q_pe=dev["q_pe"], q=qt, interleaved=interleaved)
    check_queries(s, qt.cpu(), interleaved)


def test_rows_past_32_bit_offsets():
    # a cache of 4.8 GB: byte offsets of its last rows pass 2^32
    pages = 65536
    s = make("bf16", 5, 2, seed=11)
    cache = torch.empty(pages, PAGE, 1, 576, dtype=torch.bfloat16, device="cuda")
    rows = torch.tensor([pages * PAGE - 1, pages * PAGE - 64, 3_800_000, 1_900_000, 0], dtype=torch.int32)
    dev = {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in s.items()}
    mla.mla_append_kvcache(dev["latent"], dev["k_pe"], dev["positions"], dev["cos_sin"], rows.cuda(), cache,
                           norm_weight=dev["weight"])
    got = cache.view(-1, 576)[rows.cuda().long()].cpu()
    small = torch.zeros(1, PAGE, 1, 576, dtype=torch.bfloat16)
    small.view(-1, 576)[:5] = got
    s["cache"], s["slots"] = torch.zeros_like(small), torch.arange(5, dtype=torch.int32)
    check_rows(s, small, True, 1e-6, s["slots"] >= 0)


def test_side_stream_and_graph_replay():
    s = make("fp8", 100, 16, seed=12)
    dev = {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in s.items()}

    def step(cache, q):
        mla.mla_append_kvcache(dev["latent"], dev["k_pe"], dev["positions"], dev["cos_sin"], dev["slots"], cache,
                               norm_weight=dev["weight"], q_pe=dev["q_pe"], q=q, is_fp8_kvcache=True)

    cache, q = dev["cache"].clone(), dev["q"].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(cache, q)
    side.synchronize()
    check_rows(s, cache.cpu(), True, 1e-6, s["slots"] >= 0)
    check_queries(s, q.cpu(), True)
    cache2, q2 = dev["cache"].clone(), dev["q"].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(cache2, q2)
    cache2.copy_(dev["cache"])
    q2.copy_(dev["q"])
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(cache2, cache) and torch.equal(q2, q)


def test_refusals():
    s = make("bf16", 8, 4, seed=13)
    d = {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in s.items()}

    def run(**over):
        a = {**d, **over}
        mla.mla_append_kvcache(a["latent"], a["k_pe"], a["positions"], a["cos_sin"], a["slots"], a["cache"],
                               norm_weight=a["weight"], q_pe=a["q_pe"], q=a["q"], is_fp8_kvcache=a.get("fp8", False),
                               status=a.get("status"))

    run()
    wide = torch.zeros(8, 600, dtype=torch.bfloat16, device="cuda")
    for bad in (dict(latent=d["latent"].float()), dict(latent=d["latent"][:, :511]), dict(slots=d["slots"].long()),
                dict(slots=d["slots"][:7]), dict(positions=d["positions"][:7]), dict(cos_sin=d["cos_sin"].half()),
                dict(q=None), dict(q=d["q"][:, :3]), dict(weight=d["weight"].float()), dict(fp8=True),
                dict(k_pe=None), dict(cache=d["cache"].cpu()), dict(slots=d["slots"].cpu()),
                dict(latent=wide.t()[:512].t().t().contiguous().t()),
                dict(status=torch.zeros(2, dtype=torch.int32, device="cuda"))):
        with pytest.raises(ValueError):
            run(**bad)
    for bad in (dict(latent=wide[:, 1:513]),                       # rows not on 16-byte boundaries
                dict(q=d["q"][:, :1].expand(8, 4, 576)),           # heads of q that overlap
                dict(cache=torch.zeros(2, 32, 1, 576, dtype=torch.bfloat16, device="cuda"))):
        with pytest.raises(mla.MLAError):
            run(**bad)
