"""GB300-native (sm_103a) Mamba-2 SSD varlen forward prefill scan.

The compute path is the CUDA library libssd_scan.so (C ABI in
include/ssd_scan.h, include/ssd_attn.h and include/ssd_layers.h); ``binding`` (the
scan), ``attention`` (the paged key/value cache and the attention over it, for the
attention layers of a hybrid model) and ``layers`` (what stands around the two) are
its thin Python front ends and ``workloads`` the seeded synthetic inputs.
"""
from .attention import (  # noqa: F401
    alloc_attn_workspace,
    ssd_attn_varlen_fwd,
    ssd_attn_varlen_workspace_size,
    ssd_kv_cache_read,
    ssd_kv_cache_write,
)
from .binding import (  # noqa: F401
    EXPORTED_SYMBOLS,
    SSDError,
    alloc_host_workspace,
    alloc_workspace,
    library,
    ssd_scan_varlen_fwd,
    ssd_scan_varlen_fwd_profiled,
    ssd_scan_varlen_fwd_states,
    ssd_scan_varlen_fwd_strided,
    ssd_scan_varlen_fwd_bf16_pool,
    ssd_scan_varlen_fwd_noalloc,
    ssd_scan_varlen_fwd_host,
    ssd_scan_varlen_host_plan,
    ssd_scan_varlen_host_read_errors,
    ssd_scan_varlen_host_workspace_size,
    ssd_scan_varlen_num_launches,
    ssd_scan_varlen_fused_walk,
    ssd_scan_varlen_read_errors,
    ssd_scan_varlen_short_threshold,
    ssd_scan_varlen_test_stall,
    ssd_scan_varlen_workspace_size,
    status_string,
)
from .layers import (  # noqa: F401
    alloc_rope_table,
    alloc_selective_scan_workspace,
    rope_frequencies,
    ssd_causal_conv_varlen_fwd,
    ssd_rms_norm_fwd,
    ssd_rope_kv_cache_write,
    ssd_rope_varlen_fwd,
    ssd_selective_scan_varlen_fwd,
    ssd_selective_scan_varlen_workspace_size,
)
