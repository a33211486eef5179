"""MI355X-native selective state-space causal scan (prefill + decode) for one GPU's channel slice.

``prefill`` and ``decode_step`` call the C ABI of include/ssm.h (libssm.so, hand-written
HIP kernels for gfx950) through a thin ctypes binding; ``q8_quantize`` and
``q8_dequant_sum`` call the block int8 codec of include/ssm_codec.h; ``Projector``,
``conv_silu`` and ``conv_xproj`` call the channel-sliced projections, the conv front and the two
fused, of include/ssm_proj.h; ``decode_fused`` runs a decoded token's conv front, x_proj, dt_proj and
decode step in two kernels (include/ssm_layer.h); ``rope``, ``KVCache`` with ``kv_write`` and ``kv_read``,
``attn_prefill`` and ``attn_decode_step`` are the attention operators of include/ssm_attn.h (``attn_layer`` is an
attention block of them); ``rms_norm`` and ``Q4Weight`` with ``q4_quantize``, ``q4_dequantize`` and ``q4_linear`` are the
residual norm and the 4-bit projections of include/ssm_block.h; ``inputs`` makes seeded synthetic workloads.  Importing the package does not load the
library; the first call does, and raises if it is not built.
"""
from ._lib import (PROJ_DT, PROJ_IN, PROJ_OUT, PROJ_X, Projector, SsmError, conv_silu, conv_xproj,  # noqa: F401
                   decode_fused, decode_fused_workspace_bytes, decode_step, decode_step_pool, load, prefill,
                   prefill_pool, q8_dequant_sum, q8_num_blocks, q8_quantize, workspace_bytes)
from .attn import (KVCache, attn_decode_step, attn_decode_workspace_bytes, attn_prefill, kv_read, kv_write,  # noqa: F401
                   rope, rope_frequencies)
from .block import Q4Weight, q4_dequantize, q4_linear, q4_quantize, rms_norm  # noqa: F401
