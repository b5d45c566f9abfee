"""GB300-native (sm_103a) exact attention, FlashAttention-2 style.

The compute path is libfa.so (hand-written tcgen05 / TMA / TMEM CUDA
kernels behind the C ABI of include/fa.h).  This package is its Python
binding: the ``fa_*`` functions have the C names and marshal torch tensors
and the current torch stream into the C calls; ``forward`` and ``backward``
also allocate the outputs.  PyTorch provides device memory and streams only.
"""

from ._binding import (  # noqa: F401
    FA_ERR_BAD_INDEX,
    FA_ERR_CUDA,
    FA_ERR_INVALID_ARG,
    FA_BWD_NOALLOC_SCRATCH_BYTES,
    FA_CAUSAL_BOTTOM_RIGHT,
    FA_CAUSAL_NONE,
    FA_CAUSAL_TOP_LEFT,
    FA_ERR_NO_MEMORY,
    FA_ERR_SCRATCH_TOO_SMALL,
    FA_ERR_TIMEOUT,
    FA_ERR_UNSUPPORTED,
    FA_OK,
    FaError,
    backward,
    declared_symbols,
    fa_abi_version,
    fa_bwd,
    fa_bwd_general,
    fa_bwd_gqa,
    fa_bwd_noalloc,
    fa_bwd_plan,
    fa_fwd,
    fa_fwd_ex,
    fa_fwd_general,
    fa_fwd_gqa,
    fa_fwd_plan,
    fa_kv4_cache_bytes,
    fa_kv4_fwd,
    fa_kv4_fwd_plan,
    fa_kv4_read,
    fa_kv4_write,
    fa_packed_bwd,
    fa_packed_fwd,
    fa_poll_status,
    fa_prefix_fwd,
    fa_rope,
    fa_rope_phases,
    fa_selftest_kv4_timeout,
    fa_selftest_wait_timeout,
    fa_set_wait_timeout_ns,
    fa_strerror,
    fa_launch_count,
    fa_timing_enable,
    fa_timing_read,
    fa_trim_workspace,
    forward,
    kv4_cache,
    kv4_forward,
    load,
    packed_backward,
    packed_forward,
    prefix_forward,
    rope,
    rope_frequencies,
    rope_phases,
)

FA_KERNEL_FWD = 0
FA_KERNEL_COMBINE = 1
FA_KERNEL_BWD_PRE = 2
FA_KERNEL_BWD = 3
FA_KERNEL_BWD_DQ = 4
FA_KERNEL_KV4_WRITE = 8
FA_KERNEL_KV4_READ = 9
FA_KERNEL_KV4_FWD = 10
FA_KERNEL_KV4_MERGE = 11
FA_KERNEL_ROPE = 16
FA_KERNEL_PACKED_PLAN = 17
FA_KERNEL_PACKED_FWD = 18
FA_KERNEL_PACKED_MERGE = 19
