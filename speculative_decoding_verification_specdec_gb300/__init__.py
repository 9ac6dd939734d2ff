"""Batched speculative-decoding verification on GB300 (sm_103a).

The work happens in libspecdec.so (include/specdec.h); this package is its ctypes
binding, device marshalling, the seeded synthetic workloads and the acceptance metrics.
"""
from ._native import (  # noqa: F401
    SPECDEC_BF16,
    SPECDEC_F32,
    SPECDEC_KMAX,
    SpecdecError,
    kv_read,
    kv_write,
    launch_config,
    load,
    paged_attention,
    paged_attention_workspace_size,
    rope,
    rope_frequencies,
    specdec_verify,
    specdec_wait,
    status_string,
)
from .kvcache import PagedCache  # noqa: F401
from .metrics import acceptance_rates, mean_acceptance_length  # noqa: F401
