"""B200-native kernelized linear attention.

The compute lives in liblinattn.so (hand-written CUDA for sm_100a behind the
C ABI in include/la_api.h); ``api`` is its thin Python binding and
``inputs`` draws the seeded synthetic tensors used by tests and benchmarks.
"""
from .api import (  # noqa: F401
    GatedLinearAttention,
    HeadGroupNorm,
    LinearAttention,
    LinearAttentionError,
    la_backward,
    la_backward_gated,
    la_decode_step,
    la_decode_step_gated,
    la_forward,
    la_forward_gated,
    la_get_device_error,
    la_group_norm,
    la_group_norm_backward,
    la_launch_count,
    la_profile_collect,
    la_profile_enable,
    la_status_string,
    la_version,
    la_workspace_size,
    load_library,
)
