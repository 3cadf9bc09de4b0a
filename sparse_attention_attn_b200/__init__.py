"""B200-native shifted sparse attention (S2-Attn, LongLoRA's "shift short
attention"), forward and backward, as hand-written sm_100a CUDA behind a C ABI
(include/s2attn.h, libs2attn.so).  PyTorch provides device memory and streams.
"""
from .api import (CachePlan, ChunkAttention, QKNormRope, S2Attention, S2RopeAttention,  # noqa: F401
                  bwd_workspace_bytes, cache_append, cache_attention, cache_plan, dense_causal_attn, device_status,
                  hga_backward, hga_forward, lse_merge, nf4_dequantize, nf4_levels, nf4_qkv, qknorm_rope_backward,
                  qknorm_rope_forward, rope_apply, rope_table, s2_attn, s2_qknorm_attn, s2attn_backward,
                  s2attn_backward_rope, s2attn_forward, s2attn_forward_rope, seg_backward, seg_forward)
from ._lib import S2AttnError  # noqa: F401
