"""MI355X (gfx950) KDA: chunked prefill and recurrent decode in HIP.

``chunk_fwd`` and ``recurrent_step`` call the C ABI of ``libkda.so``
(include/kda.h) through ctypes; so do the operators that stand around the
recurrence in a layer and its sibling with a scalar decay a head
(``short_conv_*``, ``selective_scan_*``, ``group_norm_*``), and the cache of the
layers between that attend to every position (``kv_cache_*``, ``paged_attn``).  The library is loaded on first use and is
required: there is no CPU or PyTorch fallback.
"""
from .kda import (  # noqa: F401
    KDAError,
    Plan,
    chunk_bwd,
    chunk_bwd_workspace_size,
    chunk_fwd,
    chunk_fwd_noalloc,
    chunk_fwd_varlen,
    chunk_fwd_varlen_workspace_size,
    snapshot_count,
    chunk_plan,
    chunk_workspace_size,
    load_library,
    profile_start,
    profile_stop,
    recurrent_step,
    recurrent_steps,
    status_string,
    version,
)
from .mixer import (  # noqa: F401
    group_norm_bwd,
    group_norm_fwd,
    selective_scan_bwd,
    selective_scan_fwd,
    selective_scan_step,
    short_conv_bwd,
    short_conv_fwd,
    short_conv_step,
)
from .paged import (  # noqa: F401
    kv_cache_read,
    kv_cache_write,
    paged_attn,
)
from .build import LIB_PATH, build_library  # noqa: F401

__all__ = ["chunk_fwd", "chunk_fwd_noalloc", "chunk_bwd", "chunk_bwd_workspace_size", "chunk_fwd_varlen", "chunk_fwd_varlen_workspace_size", "snapshot_count", "recurrent_step", "recurrent_steps", "chunk_plan", "chunk_workspace_size", "profile_start", "profile_stop",
           "short_conv_fwd", "short_conv_bwd", "short_conv_step", "selective_scan_fwd", "selective_scan_bwd",
           "selective_scan_step",
           "group_norm_fwd", "group_norm_bwd", "kv_cache_write", "kv_cache_read", "paged_attn", "load_library", "build_library", "version", "status_string", "KDAError", "Plan"]
