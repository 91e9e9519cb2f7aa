"""GB300-native DSA indexer: paged index-key store and streaming score + top-k;
and the attention it serves: rotary positions, the paged K/V cache, attention of
drafted tokens over it and over the selection, of spans (capped and biased
scores, documents, prefixes, windows) and behind shared prefixes, and the page
tables and slot maps of a step.

The compute path is libdsaidx.so (CUDA, sm_103a), reached through the C ABI
in include/dsaidx.h; `dsaidx` is the Python binding over it.
"""
from .dsaidx import (FMT_BF16, FMT_FP4, FMT_FP8, HEADS, HEAD_DIM, PAGE_SIZE, Context, DsaError, Rope,
                     kv_page_bytes, lib, page_bytes, status_str)

__all__ = ["FMT_BF16", "FMT_FP8", "FMT_FP4", "HEADS", "HEAD_DIM", "PAGE_SIZE", "Context", "DsaError",
           "Rope", "kv_page_bytes", "lib", "page_bytes", "status_str"]
