"""mla_summarize_pages on the GPU against its formula in 64 bits."""
import pytest
import torch

import mla_decode_attention_12_b200 as mla
from cache_helpers import PAGE, cache_rows64, random_cache, table_of

pytestmark = pytest.mark.gpu


def expected(cache, table, before, after, keys, scales, fp8):
    """The formula: exact means (sums of 64 16-bit values fit 64 bits), then float32 step by step."""
    rows = cache_rows64(cache, fp8).view(cache.shape[0], PAGE, -1)
    keys, scales = keys.clone(), scales.clone()
    for b in range(len(after)):
        for j in range(before[b] // PAGE, after[b] // PAGE):
            page = int(table[b, j])
            m = (rows[page].sum(0) / PAGE).float()
            s = (m.abs().amax() * torch.tensor(1 / 127, dtype=torch.float32)).clamp(min=2.0 ** -126)
            keys[page] = torch.round(m / s).to(torch.int8)
            scales[page] = s
    return keys, scales


def run(kind, before, after, d=576, seed=0, cache=None, width=None):
    table, pages = table_of(after, seed, width=width)
    cache = random_cache(kind, pages, d, seed) if cache is None else cache
    g = torch.Generator().manual_seed(seed + 9)
    keys = torch.randint(-127, 128, (pages, d), generator=g).to(torch.int8)
    scales = torch.rand(pages, generator=g)
    got_k, got_s = keys.cuda(), scales.cuda()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    mla.mla_summarize_pages(cache.cuda(), table.cuda(), torch.tensor(before, dtype=torch.int32).cuda(),
                            torch.tensor(after, dtype=torch.int32).cuda(), got_k, got_s, is_fp8_kvcache=kind == "fp8",
                            status=status)
    assert int(status) == 0
    want_k, want_s = expected(cache, table, before, after, keys, scales, kind == "fp8")
    # equal to the last bit: the sum keeps more bits than the rounding to float32 needs
    assert torch.equal(got_s.cpu(), want_s)
    assert torch.equal(got_k.cpu(), want_k)


@pytest.mark.parametrize("kind,d", [("bf16", 576), ("bf16", 512), ("fp16", 576), ("fp16", 512), ("fp8", 576)])
@pytest.mark.parametrize("before,after", [
    ([0], [64]), ([63], [64]), ([64], [127]), ([0], [63]), ([1, 0, 200, 128], [500, 0, 201, 192]),
    ([0] * 40, list(range(0, 40 * 37, 37))), ([64 * 9], [64 * 40 + 5]),
])
def test_keys(kind, d, before, after):
    run(kind, before, after, d, seed=len(after))


def test_more_requests_than_one_prefix_sum():
    after = [(i * 53) % 300 for i in range(700)]
    before = [max(0, n - (i * 29) % 200) for i, n in enumerate(after)]
    run("bf16", before, after, seed=3)


def test_more_pages_than_blocks():
    run("fp8", [0, 64 * 100], [64 * 400, 64 * 350 + 17], seed=4)


def test_zero_and_cancelling_pages():
    table, pages = table_of([64, 64, 64], 0)
    cache = torch.zeros(pages, PAGE, 1, 576, dtype=torch.bfloat16)
    p1, p2 = int(table[1, 0]), int(table[2, 0])
    cache[p1, 0::2], cache[p1, 1::2] = 3.0e38, -3.0e38   # a mean of zero from sums that come near the largest float
    cache[p2, 0], cache[p2, 1], cache[p2, 2] = 2.0 ** 20, 2.0 ** -20, -(2.0 ** 20)
    run("bf16", [0, 0, 0], [64, 64, 64], cache=cache)


def test_bad_entries_are_skipped_and_recorded():
    table, pages = table_of([256, 256], 5)
    cache = random_cache("bf16", pages, 576, 5)
    keys = torch.zeros(pages, 576, dtype=torch.int8)
    scales = torch.zeros(pages)
    want_k, want_s = expected(cache, table, [0, 0], [256, 128], keys, scales, False)
    bad = table.clone()
    bad[1, 2], bad[1, 3] = pages, -1
    k, s = keys.cuda(), scales.cuda()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    lens = torch.tensor([256, 256], dtype=torch.int32)
    mla.mla_summarize_pages(cache.cuda(), bad.cuda(), torch.zeros(2, dtype=torch.int32).cuda(), lens.cuda(), k, s, status=status)
    assert int(status) == 6 and torch.equal(k.cpu(), want_k) and torch.equal(s.cpu(), want_s)
    status.zero_()
    k, s = keys.cuda(), scales.cuda()
    lens[0] = 10 ** 6  # beyond the table: its pages past the table are skipped
    lens[1] = 128
    mla.mla_summarize_pages(cache.cuda(), table.cuda(), torch.zeros(2, dtype=torch.int32).cuda(), lens.cuda(), k, s, status=status)
    assert int(status) == 6 and torch.equal(k.cpu(), want_k) and torch.equal(s.cpu(), want_s)


def test_negative_lengths_are_empty():
    table, pages = table_of([128], 5)
    cache = random_cache("bf16", pages, 576, 5)
    k, s = torch.zeros(pages, 576, dtype=torch.int8).cuda(), torch.zeros(pages).cuda()
    mla.mla_summarize_pages(cache.cuda(), table.cuda(), torch.tensor([-100], dtype=torch.int32).cuda(),
                            torch.tensor([-5], dtype=torch.int32).cuda(), k, s)
    assert not k.any() and not s.any()


def test_refusals():
    table, pages = table_of([128], 5)
    a = dict(cache=random_cache("bf16", pages, 576, 5).cuda(), table=table.cuda(),
             before=torch.zeros(1, dtype=torch.int32).cuda(), after=torch.full((1,), 128, dtype=torch.int32).cuda(),
             keys=torch.zeros(pages, 576, dtype=torch.int8).cuda(), scales=torch.zeros(pages).cuda(), fp8=False)

    def go(**over):
        b = {**a, **over}
        mla.mla_summarize_pages(b["cache"], b["table"], b["before"], b["after"], b["keys"], b["scales"], is_fp8_kvcache=b["fp8"])

    go()
    for bad in (dict(fp8=True), dict(table=a["table"].long()), dict(before=a["before"].repeat(2)), dict(keys=a["keys"][:, :512]),
                dict(keys=a["keys"].float()), dict(scales=a["scales"][:-1]), dict(cache=a["cache"].float()),
                dict(after=a["after"].cpu())):
        with pytest.raises(ValueError):
            go(**bad)
