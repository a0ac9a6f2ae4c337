"""The decode calls with a status word of the caller's: host-side refusals (no GPU)."""
import pytest

from mla_decode_attention_12_b200 import _lib, build

FAKE = 1 << 20


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.load()


def dense(lib, **over):
    a = dict(q=FAKE, batch=2, s_q=1, h_q=16, d_qk=576, kvcache=FAKE, num_blocks=8, page=64, h_kv=1, table=FAKE, max_blocks=4,
             lens=FAKE, dv=512, dtype=0, md=FAKE, parts=74, splits=FAKE, causal=0, scale=0.0, active=0, o=FAKE, lse=FAKE, ws=FAKE,
             ws_bytes=1 << 40, status=FAKE, stream=None)
    a.update(over)
    return lib.mla_decode_with_kvcache_status(*a.values())


def ragged(lib, **over):
    a = dict(q=FAKE, total_q=9, h_q=64, d_qk=576, kvcache=FAKE, num_blocks=8, page=64, h_kv=1, table=FAKE, batch=2, max_blocks=4,
             lens=FAKE, dv=512, dtype=0, plan=FAKE, parts=74, scale=0.0, o=FAKE, lse=FAKE, ws=FAKE, ws_bytes=1 << 40,
             scratch=None, scratch_bytes=0, status=FAKE, stream=None)
    a.update(over)
    return lib.mla_decode_varlen_status(*a.values())


@pytest.mark.parametrize("call", [dense, ragged])
def test_refusals(lib, call):
    assert call(lib, status=FAKE + 2) == 1
    assert call(lib, q=None) == 1 and call(lib, ws=None) == 1
    assert call(lib, page=32) == 2
    assert call(lib, ws_bytes=100) == 3
    assert call(lib, batch=0) == 0
