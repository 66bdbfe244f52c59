"""GB300 (sm_103a) fused 8-bit blockwise AdamW with stochastic rounding.

The compute lives in libq8adamw.so (C ABI: include/q8adamw.h for the steps,
include/q8train.h for the training-step operators around them); this package
is its Python binding (same names as the C entry points) plus a torch.optim
front end (bit_blockwise_adamw_gb300.optim) and autograd functions and modules
(bit_blockwise_adamw_gb300.nn).
"""
from ._binding import (  # noqa: F401
    BLOCK, DISTILL_MAX_K, EXPORTS, GELU, GELU_TANH, MAX_STEP, NORM_LAYER, NORM_MAX_DIM, NORM_NONE, NORM_RMS,
    SIGNED, SILU, SMALL_NUMEL, UNSIGNED, HParams, LionHParams, MomentumHParams, Q8Error, Tensor16, Tensor8,
    adamw8bit_sr_step, adamw_bf16_sr_step, hparams, library_path, lion8bit_sr_step, lion_hparams, load_library,
    momentum8bit_sr_step, momentum_hparams, pack_tensor16, pack_tensor8, q8_abi_version, q8_block_norm_backward,
    q8_block_norm_forward, q8_block_norm_workspace, q8_blockwise_dequantize, q8_blockwise_quantize, q8_codebook_init,
    q8_distill_topk_backward, q8_distill_topk_forward, q8_gated_ff_backward, q8_gated_ff_forward,
    q8_gated_ff_workspace, q8_last_error, q8_philox_fill, q8_prepare_device, q8_selftest_sqrt_div)
