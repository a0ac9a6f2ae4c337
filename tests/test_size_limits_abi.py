"""Sizes whose loop counters would pass 32 bits are refused on the host (no GPU)."""
import pytest

from mla_decode_attention_12_b200 import _lib, build

FAKE = 1 << 20


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.load()


@pytest.mark.parametrize("topn", [1 << 25, 2 ** 31 - 1])
def test_selection_of_more_pages_than_a_block_table_holds(lib, topn):
    # the selection fills places n .. topn - 1 in steps of 256 or 1,024: near 2^31 the counter would turn negative
    assert lib.mla_select_pages(FAKE, 1, 1, 16, 576, 0, FAKE, FAKE, 8, FAKE, 4, FAKE, 1, topn, 1, 1, FAKE, FAKE, FAKE, 1 << 40,
                                None, None) == 2


@pytest.mark.parametrize("batch", [(1 << 30) + 1, 2 ** 31 - 1])
def test_page_keys_of_more_requests_than_their_chunks_count(lib, batch):
    # requests are taken 512 at a time: past 2^31 - 512 the counter would turn negative
    assert lib.mla_summarize_pages(FAKE, 8, 64, 1, 576, 0, FAKE, 1, FAKE, FAKE, batch, FAKE, FAKE, None, None) == 2
