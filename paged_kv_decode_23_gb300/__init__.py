"""pkd: batch decode attention over a paged KV cache for GB300 (sm_103a).

``BatchDecodePagedKV`` mirrors FlashInfer's BatchDecodeWithPagedKVCacheWrapper plan()/run();
the work happens in ``_build/libpkd.so`` (hand-written CUDA kernels behind a C ABI declared
in ``include/pkd.h``).  ``append_paged_kv``, ``gather_paged_kv``, ``evict_paged_kv``, ``copy_pages``
and ``PageAllocator`` fill, read back, cut back and move the cache it reads.  Build it with ``paged_kv_decode_23_gb300.build.build()``.
"""
from ._lib import PkdError, LIB_PATH  # noqa: F401
from .cache import (PageAllocator, append_paged_kv, copy_pages, evict_paged_kv,  # noqa: F401
                    gather_paged_kv, make_cos_sin_cache)
from .decode import (BatchDecodePagedKV, BatchMLAPagedAttention,  # noqa: F401
                     CUDAGraphBatchDecodePagedKV, check_page_table, graph_workspace_bytes,
                     mla_graph_workspace_bytes, mla_plan_host, noalloc_check_status, plan_host,
                     workspace_bytes)

__all__ = ["BatchDecodePagedKV", "BatchMLAPagedAttention", "CUDAGraphBatchDecodePagedKV",
           "PageAllocator", "PkdError", "append_paged_kv", "check_page_table", "copy_pages",
           "evict_paged_kv", "gather_paged_kv", "graph_workspace_bytes", "make_cos_sin_cache", "mla_graph_workspace_bytes",
           "mla_plan_host", "noalloc_check_status", "plan_host", "workspace_bytes"]
