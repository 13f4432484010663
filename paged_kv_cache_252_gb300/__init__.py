"""GB300-native paged decode attention over a blocked KV cache.

Hand-written CUDA for sm_103a behind a C ABI (``libpagedkv.so``), first of all:

* :func:`kv_cache_write` scatters new key/value tokens into their physical
  cache slots (fp16/bf16 copy, or fp16 -> FP8 E5M2 cast).
* :func:`paged_attention_decode` computes softmax(q K^T * scale) V for every
  sequence over its blocks, one CTA stream per KV head serving the whole GQA
  group, causal among a sequence's query tokens (speculative verify).

Around them, what a serving step runs:

* :func:`rotary_write` (and :func:`rotary_embed`) turns q and k by their positions and
  writes the cache in the same pass; :func:`rotary_inv_freq` gives the frequencies.
* :func:`paged_attention_prefill` is the attention of prompts and prompt chunks.
* :func:`kv_cache_write_int4` quantises tokens to four bits as they are written,
  :func:`paged_attention_decode_int4` (and the varlen, tree and chunked calls) attends over such a
  cache, and :func:`kv_cache_read` reads rows of a cache of any type back.
* :func:`kv_cache_accept` keeps the accepted drafts of a speculative verify, and
  :meth:`BlockAllocator.truncate` gives the dropped ones' blocks back.

:class:`BlockAllocator` (host, C++) hands out the blocks: sequences, fork with
copy-on-write (:func:`copy_blocks` performs the copies), and a prefix cache.

The Python layer only marshals torch tensors into pointers and sizes; every
step of the computation runs in the CUDA library. Importing this package does
not load the library; the first call does, and fails loudly if it is missing.
"""
from . import workloads  # noqa: F401
from .api import (  # noqa: F401
    KV_FP16, KV_BF16, KV_E5M2, KV_INT8, KV_INT4,
    kv_cache_write, paged_attention_decode, paged_attention_decode_varlen,
    paged_attention_decode_tree, paged_attention_decode_chunked, selftest_bounded_wait,
    paged_attention_decode_noalloc, decode_workspace_bytes,
    library_path, load_library, alloc_kv_cache, PagedKVError,
    BlockAllocator, copy_blocks,
    alloc_kv_scales, kv_cache_write_int8, paged_attention_decode_int8, int8_codes,
    rotary_inv_freq, rotary_embed, rotary_write, paged_attention_prefill, prefill_workspace_bytes, kv_cache_accept,
    kv_cache_write_int4, kv_cache_read, paged_attention_decode_int4,
)
