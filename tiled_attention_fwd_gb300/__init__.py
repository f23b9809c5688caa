"""FlashAttention-2 forward (and backward) pass for GB300 (sm_103a), cross attention of ragged batches with its
gradient, and the serving form over a paged key/value cache whose tables are built on the GPU.

The compute path is the C-ABI library ``libfa_gb300.so`` (hand-written CUDA:
TMA + tcgen05 tensor-core kernels for bf16 and e4m3, SIMT kernel for fp32); this package
only loads it and marshals arguments.  Build it with
``python -m tiled_attention_fwd_gb300.build``.
"""
from ._lib import (CCrossBatch, CPagePool, CPagedBatch, CPagedCache, FAError, PagePool, PagedCache, backward, check_status,
                   cross_backward, cross_backward_workspace, cross_forward, cross_workspace, declared_functions, fa_abi_version, fa_bwd, fa_bwd_strided,
                   fa_bwd_workspace_bytes, fa_cross_bwd, fa_cross_bwd_workspace_bytes, fa_cross_fwd, fa_cross_fwd_workspace_bytes, fa_fwd, fa_fwd_f32, fa_fwd_fp8, fa_fwd_host, fa_fwd_host_workspace_bytes, fa_fwd_noalloc, fa_fwd_strided,
                   fa_paged_extend, fa_paged_fwd, fa_paged_fwd_workspace_bytes, fa_paged_read, fa_paged_release, fa_paged_write,
                   fa_selftest_wait, fa_set_wait_limit_ms, fa_status, fa_strerror, forward, forward_fp8, load,
                   paged_extend, paged_forward, paged_read, paged_release, paged_workspace, paged_write)

__all__ = [
    "CPagedBatch", "CPagedCache", "FAError", "PagedCache", "backward", "check_status", "declared_functions", "fa_abi_version", "fa_bwd", "fa_bwd_strided",
    "fa_bwd_workspace_bytes",
    "fa_fwd", "fa_fwd_f32", "fa_fwd_fp8", "fa_fwd_host", "fa_fwd_strided",
    "fa_fwd_host_workspace_bytes", "fa_fwd_noalloc", "fa_selftest_wait", "fa_set_wait_limit_ms", "fa_status", "fa_strerror", "forward", "forward_fp8", "load",
    "fa_paged_fwd", "fa_paged_fwd_workspace_bytes", "fa_paged_read", "fa_paged_write",
    "paged_forward", "paged_read", "paged_workspace", "paged_write",
    "CPagePool", "PagePool", "fa_paged_extend", "fa_paged_release", "paged_extend", "paged_release",
    "CCrossBatch", "cross_backward", "cross_backward_workspace", "cross_forward", "cross_workspace",
    "fa_cross_bwd", "fa_cross_bwd_workspace_bytes", "fa_cross_fwd", "fa_cross_fwd_workspace_bytes",
]
