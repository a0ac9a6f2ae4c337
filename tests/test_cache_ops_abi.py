"""Host-side refusals of the cache operators' C entry points (no GPU)."""
import pytest

from mla_decode_attention_12_b200 import _lib, build

FAKE = 1 << 20


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.load()


def append(lib, **over):
    a = dict(latent=FAKE, latent_stride=576, k_pe=FAKE, k_pe_stride=576, weight=FAKE, eps=1e-6, positions=FAKE, cos_sin=FAKE,
             max_position=16, slots=FAKE, tokens=4, kvcache=FAKE, num_blocks=8, page=64, h_kv=1, d_qk=576, dtype=0,
             interleaved=1, q_pe=FAKE, qps_t=192 * 4, qps_h=192, q=FAKE, qs_t=576 * 4, qs_h=576, h_q=4, status=None, stream=None)
    a.update(over)
    return lib.mla_append_kvcache(*a.values())


@pytest.mark.parametrize("over,code", [
    (dict(latent=None), 1), (dict(k_pe=None), 1), (dict(positions=None), 1), (dict(cos_sin=None), 1), (dict(slots=None), 1),
    (dict(kvcache=None), 1), (dict(tokens=-1), 1), (dict(num_blocks=0), 1), (dict(dtype=3), 1), (dict(interleaved=2), 1),
    (dict(max_position=0), 1), (dict(q=None), 1), (dict(q_pe=None), 1), (dict(h_q=0), 1), (dict(eps=float("nan")), 1),
    (dict(eps=-1.0), 1), (dict(latent=FAKE + 2), 1), (dict(latent_stride=577), 1), (dict(latent_stride=-576), 1),
    (dict(qs_h=512), 1), (dict(qs_t=576), 1), (dict(d_qk=512), 1),
    (dict(page=32), 2), (dict(h_kv=2), 2), (dict(d_qk=192), 2),
    (dict(dtype=2, d_qk=512, k_pe=None, q_pe=None, q=None), 2), (dict(num_blocks=1 << 26), 2),
    (dict(tokens=1 << 24, h_q=128, qs_t=576 * 128, qps_t=192 * 128), 2),
])
def test_append_refuses(lib, over, code):
    assert append(lib, **over) == code


def test_append_of_no_tokens_is_a_no_op(lib):
    assert append(lib, tokens=0, latent=None, slots=None) == 0


def summarize(lib, **over):
    a = dict(kvcache=FAKE, num_blocks=8, page=64, h_kv=1, d_qk=576, dtype=0, table=FAKE, max_blocks=4, prev=FAKE, lens=FAKE,
             batch=2, keys=FAKE, scales=FAKE, status=None, stream=None)
    a.update(over)
    return lib.mla_summarize_pages(*a.values())


@pytest.mark.parametrize("over,code", [
    (dict(kvcache=None), 1), (dict(table=None), 1), (dict(prev=None), 1), (dict(lens=None), 1), (dict(keys=None), 1),
    (dict(scales=None), 1), (dict(batch=-1), 1), (dict(max_blocks=0), 1), (dict(num_blocks=0), 1), (dict(dtype=5), 1),
    (dict(keys=FAKE + 1), 1), (dict(scales=FAKE + 2), 1), (dict(kvcache=FAKE + 8), 1),
    (dict(page=16), 2), (dict(h_kv=2), 2), (dict(d_qk=128), 2), (dict(dtype=2, d_qk=512), 2), (dict(num_blocks=1 << 26), 2),
])
def test_summarize_refuses(lib, over, code):
    assert summarize(lib, **over) == code


def test_summarize_refuses_a_table_whose_pages_pass_32_bits(lib):
    assert summarize(lib, batch=512, max_blocks=1 << 22) == 2
    assert summarize(lib, batch=2, max_blocks=1 << 30) == 2


def test_summarize_of_no_requests_is_a_no_op(lib):
    assert summarize(lib, batch=0, kvcache=None) == 0


def select(lib, **over):
    a = dict(q=FAKE, batch=2, s_q=1, h_q=16, d_qk=576, dtype=0, keys=FAKE, scales=FAKE, num_blocks=8, table=FAKE, max_blocks=4,
             lens=FAKE, causal=1, topn=3, first=1, last=1, out=FAKE, out_lens=FAKE, ws=FAKE, ws_bytes=1 << 40, status=None,
             stream=None)
    a.update(over)
    return lib.mla_select_pages(*a.values())


@pytest.mark.parametrize("over,code", [
    (dict(q=None), 1), (dict(keys=None), 1), (dict(scales=None), 1), (dict(table=None), 1), (dict(lens=None), 1),
    (dict(out=None), 1), (dict(out_lens=None), 1), (dict(ws=None), 1), (dict(batch=-1), 1), (dict(s_q=0), 1), (dict(h_q=0), 1),
    (dict(max_blocks=0), 1), (dict(num_blocks=0), 1), (dict(causal=2), 1), (dict(dtype=7), 1), (dict(topn=0), 1),
    (dict(topn=1), 1), (dict(last=0), 1), (dict(first=-1), 1), (dict(first=2 ** 31 - 1, topn=2 ** 31 - 1), 1),
    (dict(q=FAKE + 2), 1), (dict(keys=FAKE + 4), 1), (dict(ws=FAKE + 8), 1),
    (dict(dtype=2), 2), (dict(d_qk=192), 2), (dict(h_q=129), 2), (dict(num_blocks=1 << 26), 2), (dict(max_blocks=1 << 26), 2),
    (dict(batch=1 << 28), 2), (dict(ws_bytes=16), 3),
])
def test_select_refuses(lib, over, code):
    assert select(lib, **over) == code


def test_select_of_no_requests_is_a_no_op(lib):
    assert select(lib, batch=0, q=None) == 0
    assert lib.mla_select_workspace_bytes(2, 3, 16, 576, 10) >= 2 * 3 * (16 * 580 + 10 * 4)
    assert lib.mla_select_workspace_bytes(2, 0, 16, 576, 10) == 0


def test_python_calls_refuse_host_tensors_and_other_things():
    import torch

    import mla_decode_attention_12_b200 as mla
    i = torch.zeros(2, dtype=torch.int32)
    table = torch.zeros(2, 3, dtype=torch.int32)
    bf = torch.zeros(2, 64, 1, 576, dtype=torch.bfloat16)
    keys, scales = torch.zeros(2, 576, dtype=torch.int8), torch.zeros(2)
    calls = [
        lambda: mla.mla_append_kvcache(bf[:, 0, 0, :512], bf[:, 0, 0, 512:], i, torch.zeros(4, 64), i, bf),
        lambda: mla.mla_append_kvcache(None, None, None, None, None, None),
        lambda: mla.mla_append_kvcache(bf[:, 0, 0, :512], None, None, None, "slots", bf),
        lambda: mla.mla_summarize_pages(bf, table, i, i, keys, scales),
        lambda: mla.mla_select_pages(bf[:, :1], keys, scales, table, i, 2),
        lambda: mla.mla_select_pages(None, keys, scales, table, i, 2),
        lambda: mla.get_mla_metadata_varlen(torch.zeros(3, dtype=torch.int32), i, 2, 16),
        lambda: mla.flash_mla_varlen_with_kvcache(bf[:, 0], bf, table, torch.zeros(3, dtype=torch.int32), i, 512,
                                                  mla.VarlenPlan(i, 2, 2, 1, 74, True)),
    ]
    for call in calls:
        with pytest.raises(ValueError):
            call()
