"""GB300-native fused softmax-attention backward.

The compute lives in the CUDA library ``_build/libattn_bwd.so`` (C ABI,
``include/attn_bwd.h``); this package only marshals torch tensors into that
ABI.  There is no CPU path: every call fails loudly when the library or a
CUDA device is missing.
"""
from ._binding import (  # noqa: F401
    AttnBwdError,
    LIB_PATH,
    attn_bwd,
    attn_bwd_gqa,
    attn_bwd_sparse,
    attn_fwd_gqa,
    backward,
    backward_host,
    check_error,
    dq_land,
    forward,
    gqa_main,
    gqa_workspace_size,
    host_scratch_size,
    library,
    preprocess,
    query_block_range,
    query_block_range_qk,
    selftest_timeout,
    sink_grad,
    sparse_backward,
    sparse_land,
    sparse_main,
    tail_plan,
    tile_schedule,
    tile_schedule_split,
    workspace_size,
)
from ._kv_cache import (  # noqa: F401
    KvPlan,
    forward_kv_cache,
    kv_block_tables,
    kv_cache_workspace_size,
    kv_cache_write,
    new_kv_cache,
)
from ._latent import (  # noqa: F401
    RopeTable,
    forward_latent,
    forward_latent_cache,
    latent_cache_workspace_size,
    latent_cache_write,
    latent_workspace_size,
    new_latent_cache,
    rope,
    rope_frequencies,
    rope_table,
    sparse_forward,
    sparse_forward_workspace_size,
)
