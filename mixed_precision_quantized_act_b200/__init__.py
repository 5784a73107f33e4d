"""MixLLM W4.4A8 linear layer for NVIDIA B200 (sm_100a).

The compute path is the CUDA library ``libmixllm_b200.so`` (C ABI in
``include/mixllm.h``); this package is its thin Python binding plus the seeded
synthetic workloads used by the tests and the benchmark.
"""
from ._lib import (  # noqa: F401
    GROUP,
    MixLLMError,
    SMALL_M_MAX,
    PackedLinear,
    empty_packed,
    gemm_debug_partials,
    gemm_w4w8a8,
    channel_salience,
    channel_salience_into,
    gemm_w4w8a8_into,
    gemm_w4w8a8_plain_i2f_into,
    gemm_w4w8a8_small_m,
    gemm_w4w8a8_small_m_noalloc_into,
    gemm_w4w8a8_small_m_into,
    linear,
    linear_into,
    linear_small_m_into,
    linear_small_m_workspace,
    linear_workspace,
    load,
    pack_weights,
    pack_weights_host,
    packed_sizes,
    quantize_act,
    quantize_act_into,
    select_top_t,
    select_top_t_into,
    select_top_t_workspace,
    selftest_bounds,
    selftest_wait_timeout,
    checked_build,
    small_m_kernel,
    small_m_debug_partials,
    small_m_workspace,
    small_m_workspace_bytes,
    sync_status,
    version,
)
from .kv4 import (  # noqa: F401
    KV4Cache,
    kv4_append_into,
    kv4_assign_into,
    kv4_attention,
    kv4_attention_into,
    kv4_attention_workspace,
    kv4_attention_workspace_bytes,
    kv4_cache,
    kv4_read_into,
    rope_table,
)
from .kv8 import (  # noqa: F401
    KV8Cache,
    kv8_append_into,
    kv8_attention,
    kv8_attention_into,
    kv8_attention_workspace,
    kv8_attention_workspace_bytes,
    kv8_cache,
    kv8_read_into,
)
from .norm import (  # noqa: F401
    dequantize_act,
    dequantize_act_into,
    head_norm_rope_into,
    residual_norm_into,
    residual_norm_quantize_into,
)
from .packfile import load_packed, save_packed  # noqa: F401
from .w8a8 import (  # noqa: F401
    W8Weights,
    w8a8_gemm_into,
    w8a8_linear,
    w8a8_linear_into,
    w8a8_linear_workspace,
    w8a8_linear_workspace_bytes,
    w8a8_pack,
    w8a8_quantize,
    w8a8_quantize_into,
)
