"""GB300-native EAGLE-3 draft-and-verify step: CUDA kernels behind the libeagle3 C ABI.

The compute path is libeagle3.so (hand-written CUDA for sm_103a); this
package only builds it and marshals torch tensors into its C argument
structs.  See include/eagle3.h, include/eagle3_linear.h, include/eagle3_moe.h,
include/eagle3_fp8.h, include/eagle3_kv.h and include/eagle3_f32.h for the contract of every entry point.  `tiny` composes the fp32 blocks into the
small lossless configuration (vanilla and speculative greedy decoding).
"""
from ._lib import (EPI_BF16, EPI_BF16_RESIDUAL, EPI_BF16_ROPE, EPI_F32, EPI_SWIGLU, F32_EPI_NONE, F32_EPI_RESIDUAL, F32_EPI_SWIGLU,
                   GREEDY, MOE_SIGMOID, MOE_SOFTMAX, ROPE_BANDS, ROPE_BASE, ROPE_HALF, ROPE_INTERLEAVED, ROPE_LINEAR, ROPE_NONE,
                   ROPE_RAMP, SAMPLED, TOPK, Eagle3Error, eagle3_accept, eagle3_accept_lazy, eagle3_chain_verify, eagle3_spec_decode_metadata, eagle3_ttt_attn, eagle3_compact_kv, eagle3_draft_tree,
                   eagle3_f32_argmax, eagle3_f32_attn, eagle3_f32_gather, eagle3_f32_linear, eagle3_f32_rmsnorm,
                   eagle3_f32_rope, eagle3_grouped_linear, eagle3_linear, eagle3_linear_fp8, eagle3_moe_combine,
                   eagle3_moe_route, eagle3_quantize_fp8, eagle3_rmsnorm, eagle3_verify_attn, eagle3_verify_attn_noalloc,
                   eagle3_append_kv, eagle3_rope, eagle3_rope_table, eagle3_verify_attn_fp8, lib)

__all__ = ["GREEDY", "TOPK", "SAMPLED", "Eagle3Error", "eagle3_accept", "eagle3_accept_lazy", "eagle3_chain_verify",
           "eagle3_spec_decode_metadata", "eagle3_ttt_attn", "eagle3_compact_kv", "eagle3_verify_attn",
           "eagle3_verify_attn_noalloc", "eagle3_linear", "eagle3_draft_tree", "eagle3_rmsnorm", "EPI_BF16", "EPI_F32",
           "EPI_BF16_RESIDUAL", "EPI_BF16_ROPE", "EPI_SWIGLU", "F32_EPI_NONE", "F32_EPI_RESIDUAL", "F32_EPI_SWIGLU",
           "eagle3_f32_linear", "eagle3_f32_rmsnorm", "eagle3_f32_rope", "eagle3_f32_gather", "eagle3_f32_argmax",
           "eagle3_f32_attn", "MOE_SOFTMAX", "MOE_SIGMOID", "eagle3_moe_route", "eagle3_grouped_linear", "eagle3_moe_combine",
           "eagle3_quantize_fp8", "eagle3_linear_fp8", "ROPE_NONE", "ROPE_LINEAR", "ROPE_BASE", "ROPE_BANDS", "ROPE_RAMP",
           "ROPE_HALF", "ROPE_INTERLEAVED", "eagle3_rope_table", "eagle3_rope", "eagle3_append_kv", "eagle3_verify_attn_fp8",
           "lib"]
