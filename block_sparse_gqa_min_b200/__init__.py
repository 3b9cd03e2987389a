"""Group-shared block-sparse GQA decode attention for NVIDIA B200 (sm_100a).

The compute path is libsba.so (CUDA kernels behind the C ABI in include/sba.h);
`sba` is its thin ctypes binding and `workloads` the seeded synthetic inputs.
The library is built in-tree on first use (nvcc, sm_100a) and every call goes
through it; there is no CPU fallback.
"""
from . import sba, workloads  # noqa: F401
from .sba import (  # noqa: F401
    Cache,
    Cache4,
    SbaError,
    alloc_step,
    decode_step,
    evict_params,
    sba_accumulate_weights,
    sba_accumulate_weights_kv4,
    sba_append_kv,
    sba_append_kv4,
    sba_budget_from_sparsity,
    sba_combine,
    sba_decode_kv4,
    sba_decode_kv4_workspace_size,
    sba_default_num_splits,
    sba_evict,
    sba_evict_kv4,
    sba_num_selected,
    sba_read_kv4,
    sba_score_select,
    sba_score_select_kv4,
    sba_score_select_kv4_workspace_size,
    sba_sparse_decode,
    sba_status_string,
    sba_update_descriptors,
    sba_workspace_size,
    select_params,
)
