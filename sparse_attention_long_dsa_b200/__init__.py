"""DSA sparse attention for NVIDIA B200 (sm_100a): indexer -> top-k -> sparse MLA attention.

The compute lives in libdsa.so (hand-written CUDA behind the C ABI in include/dsa.h);
`binding` is a ctypes layer with the same function names, `pipeline.DeviceBatch` keeps a
batch resident in device memory and enqueues the three calls, `paged_cache.PagedCache` keeps a
growing paged cache with its block tables on the device, and `workloads` draws the seeded
synthetic inputs.
"""
from . import binding  # noqa: F401
from .binding import (DSAError, dsa_batch_extend, dsa_batch_release, dsa_batch_t, dsa_indexer_scores,  # noqa: F401
                      dsa_paged_attn_decode, dsa_qk_norm_rope, dsa_read_device_status, dsa_sparse_attn_decode,
                      dsa_sparse_attn_prefill, dsa_topk, dsa_workspace_size, make_batch, rope_part)

__version__ = "0.1.0"
