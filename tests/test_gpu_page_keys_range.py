"""Page keys at the ends of the value range and of the address range."""
import pytest
import torch

import mla_decode_attention_12_b200 as mla
from cache_helpers import FP8_ROW, PAGE, cache_rows64, random_cache, table_of
from test_gpu_page_keys import expected, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [576, 512])
def test_column_sums_past_the_largest_float(d):
    # 64 finite rows of one sign: the sum passes the largest float, the mean does not
    table, pages = table_of([64, 64, 64], 0)
    g = torch.Generator().manual_seed(1)
    cache = torch.zeros(pages, PAGE, 1, d)
    for page, size in zip((int(table[b, 0]) for b in range(3)), (1e37, 3.3e38, 2.0 ** -130)):
        cache[page] = size * (0.5 + 0.5 * torch.rand(PAGE, 1, d, generator=g))
    cache = cache.bfloat16()
    assert torch.isfinite(cache.float()).all() and cache.float().sum(1).isinf().any()
    run("bf16", [0, 0, 0], [64, 64, 64], d=d, cache=cache)


def test_fp8_column_sums_past_the_largest_float():
    table, pages = table_of([64, 64], 0)
    cache = random_cache("fp8", pages, 576, 3)
    rows = cache.view(-1, FP8_ROW)
    rows[:, :512] &= 0x7F  # one sign
    page = int(table[0, 0])
    scale = torch.full((PAGE, 4), 5e35)
    rows[page * PAGE:(page + 1) * PAGE, 512:528] = scale.view(torch.uint8)
    run("fp8", [0, 0], [64, 64], cache=cache)


def test_values_spread_over_more_bits_than_the_sum_keeps():
    """The sum's error is at most 2^-40 of the column's sum of |r| (see the header).  With D = 2^-40 sum |r| / 64 over
    the worst column and M the exact largest |mean|: the scale is within (D + 2^-23 M) / 127, and scale * key within
    half a scale, D and the scale's own error of each mean."""
    table, pages = table_of([64], 0)
    g = torch.Generator().manual_seed(2)
    page = int(table[0, 0])
    for low in (-20, -40, -60):
        rows = torch.randn(32, 576, generator=g) * torch.exp2(torch.randint(low, 1, (32, 576), generator=g).float())
        rows = rows.bfloat16()
        order = torch.randperm(PAGE, generator=g)
        both = torch.cat([rows, -rows])[order]  # every value meets its negative somewhere
        both[0] += (torch.randn(576, generator=g) * 2.0 ** -30).bfloat16()
        cache = torch.zeros(pages, PAGE, 1, 576, dtype=torch.bfloat16)
        cache[page] = both[:, None]
        keys, scales = torch.zeros(pages, 576, dtype=torch.int8).cuda(), torch.zeros(pages).cuda()
        mla.mla_summarize_pages(cache.cuda(), table.cuda(), torch.zeros(1, dtype=torch.int32).cuda(),
                                torch.full((1,), 64, dtype=torch.int32).cuda(), keys, scales)
        x = both.double()
        mean, slack = x.sum(0) / PAGE, 2.0 ** -40 * x.abs().sum(0).max() / PAGE
        most = mean.abs().max()
        scale = scales[page].cpu().double()
        off = (slack + 2.0 ** -23 * most) / 127
        assert (scale - most / 127).abs() <= off + 2.0 ** -126
        got = keys[page].cpu().double() * scale
        assert ((got - mean).abs() <= scale * (0.5 + 2.0 ** -16) + slack + 127 * off).all()


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
def test_pages_past_32_bit_offsets(kind):
    # a cache of 4.3 GB and more: the byte offsets of its last pages pass 2^32
    pages = 60000 if kind == "bf16" else 110000
    small = random_cache(kind, 6, 576, 7)
    cache = torch.empty(pages, *small.shape[1:], dtype=small.dtype, device="cuda")
    cache[pages - 6:] = small.cuda()
    table = torch.tensor([[5, 0, 3]], dtype=torch.int32)
    keys, scales = torch.zeros(pages, 576, dtype=torch.int8).cuda(), torch.zeros(pages).cuda()
    mla.mla_summarize_pages(cache, (table + pages - 6).cuda(), torch.zeros(1, dtype=torch.int32).cuda(),
                            torch.full((1,), 200, dtype=torch.int32).cuda(), keys, scales, is_fp8_kvcache=kind == "fp8")
    want_k, want_s = expected(small, table, [0], [200], torch.zeros(6, 576, dtype=torch.int8), torch.zeros(6), kind == "fp8")
    assert torch.equal(keys[pages - 6:].cpu(), want_k) and torch.equal(scales[pages - 6:].cpu(), want_s)
    assert not keys[:pages - 6].any() and not scales[:pages - 6].any()
