"""GB300 (sm_103a) absorbed-MLA attention for the speculative-decoding verify step.

The computation runs in hand-written CUDA kernels behind the C ABI declared in
``include/mla_verify_attn.h``; this package builds that library in-tree and
binds it with ctypes.  Next to the verify call on a latent cache there are the
same for separate keys and values with grouped query heads (``gqa_verify_attn``)
and the cache operators around a verify step: ``blocks_extend``, ``cache_append``,
``cache_keep`` and ``blocks_trim``.  ``inputs`` makes seeded synthetic workloads.
"""
from ._lib import (TWO_TERM_MAX_KEYS_DEFAULT, MLAError, forced, last_device_error, load_library,
                   paged_workspace_size, plan, set_timing_events, set_two_term_max_keys, strerror,
                   verify_attn, verify_attn_paged, verify_attn_raw, workspace_size)
from ._serving import (blocks_extend, blocks_trim, cache_append, cache_keep, gqa_cache_append,
                       gqa_cache_keep, gqa_verify_attn, gqa_verify_attn_paged, gqa_workspace_size)
from ._build import build

__all__ = ["TWO_TERM_MAX_KEYS_DEFAULT", "MLAError", "blocks_extend", "blocks_trim", "build", "cache_append",
           "cache_keep", "forced", "gqa_cache_append", "gqa_cache_keep", "gqa_verify_attn",
           "gqa_verify_attn_paged", "gqa_workspace_size", "last_device_error", "load_library",
           "paged_workspace_size", "plan", "set_timing_events", "set_two_term_max_keys", "strerror",
           "verify_attn", "verify_attn_paged", "verify_attn_raw", "workspace_size"]
