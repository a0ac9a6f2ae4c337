"""Blackwell-native (sm_100a) MLA decoding over a paged latent KV cache.

Public calls (the names of the pages' API; "FlashMLA" usage page, deepep.org):

* :func:`get_mla_metadata` -- tile-scheduler metadata, once per decoding step;
* :func:`flash_mla_with_kvcache` -- one decode call per layer, returns ``(o, lse)``
  (``indices=``: the token-level sparse decode);
* :func:`flash_mla_sparse_fwd` -- the sparse MLA prefill, returns ``(out, max_logits, lse)``.

* :func:`flash_mla_varlen_with_kvcache` -- ragged runs of new tokens (chunks of prompts beside decode
  steps) over the paged cache, with :func:`get_mla_metadata_varlen`.

Around the decode:

* :func:`mla_append_kvcache` -- new tokens' rows into the cache (norm, rotation, quantization);
* :func:`mla_summarize_pages` -- 8-bit page keys of completed pages;
* :func:`mla_select_pages` -- each query token's best pages by those keys, as a block table, and
  :func:`flash_mla_page_sparse` -- the decode over them.

All are thin wrappers over the C ABI in ``include/mla_decode.h``; the kernels
live in ``csrc/``.  ``workloads`` generates seeded synthetic inputs.
"""
from .api import (DecodeCall, flash_mla_sparse_fwd, flash_mla_with_kvcache, get_mla_metadata, get_mla_metadata_host,
                  get_mla_metadata_sparse_host, metadata_sizes, num_sm_parts, read_device_status, workspace_bytes,
                  workspace_zero_bytes)
from .cache import mla_append_kvcache, mla_summarize_pages
from .select import flash_mla_page_sparse, mla_select_pages
from .varlen import (VarlenPlan, flash_mla_varlen_with_kvcache, get_mla_metadata_varlen, get_mla_metadata_varlen_host,
                     varlen_workspace_bytes)
from ._lib import MLAError

__all__ = ["DecodeCall", "VarlenPlan", "flash_mla_page_sparse", "flash_mla_sparse_fwd", "flash_mla_varlen_with_kvcache",
           "flash_mla_with_kvcache", "get_mla_metadata", "get_mla_metadata_host", "get_mla_metadata_sparse_host",
           "get_mla_metadata_varlen", "get_mla_metadata_varlen_host", "metadata_sizes", "mla_append_kvcache",
           "mla_select_pages", "mla_summarize_pages", "num_sm_parts", "read_device_status", "varlen_workspace_bytes",
           "workspace_bytes", "workspace_zero_bytes", "MLAError"]
