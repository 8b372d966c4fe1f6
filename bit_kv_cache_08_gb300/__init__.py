"""KVarN 2-bit KV cache for GB300 (sm_103a): quantise-on-append and decode
attention as hand-written CUDA behind a C ABI (include/kvarn.h).

This package is the thin Python face of that library: ``build`` compiles it
in-tree, and the functions re-exported from ``_abi`` marshal torch tensors to
the C entry points of the same names.
"""
from ._abi import (BF16, DEVERR_BLOCK_ID, DEVERR_NONFINITE, DEVERR_POSITION, DEVERR_WAIT_TIMEOUT,  # noqa: F401
                   FLAG_NO_CHANNEL_PASS, FLAG_NO_ROTATION, FLAG_NO_TOKEN_PASS, FLAG_TEST_WAIT_TIMEOUT, FP32, KIND_K,
                   KIND_V, ROPE_HALF, ROPE_INTERLEAVED, Config, KVarNError, Rope, alloc_pool, alloc_prefill_workspace,
                   alloc_prefix_workspace, alloc_staging, alloc_workspace, append, append_rope, append_rope_bf16,
                   block_bytes, clear_error, decode_attn, decode_attn_bf16, decode_attn_noalloc, dequantize,
                   error_decomposition, head_block_bytes, header_symbols, lib, make_config, make_rope, prefill_attn,
                   prefill_workspace_bytes, prefix_attn, prefix_attn_bf16, prefix_workspace_bytes, quantize_block,
                   read_error, rope_frequencies, staging_bytes, status_string, version, workspace_bytes)
from .build import build  # noqa: F401
