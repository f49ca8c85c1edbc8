"""MaxSim scoring on MI355X (gfx950): fused late-interaction scoring kernels.

The product is the HIP library ``libmaxsim_amd.so`` behind the C ABI in
``include/maxsim.h`` (scoring), ``include/maxsim_embed.h`` (the embedding
head), ``include/maxsim_mx4.h`` (4-bit embeddings) and ``include/maxsim_loss.h``
(log probabilities of scores); ``binding`` exposes the same entry points to Python (torch tensors in
GPU memory, argument marshalling only). ``synth`` draws the
seeded synthetic workloads and ``workload`` holds the byte/flop model.
"""

from .binding import (MaxSimError, embed_tokens_i8, embed_tokens_mx4, maxsim_abi_version, maxsim_bwd,
                      maxsim_bwd_varlen, maxsim_chamfer_bwd, maxsim_chamfer_fwd, maxsim_dequantize_mx4,
                      maxsim_dropout_bwd, maxsim_dropout_fwd, maxsim_embed_i8, maxsim_fwd,
                      maxsim_fwd_i8, maxsim_fwd_i8_tok, maxsim_fwd_mx4, maxsim_fwd_pairs, maxsim_fwd_pairs_varlen,
                      maxsim_fwd_varlen, maxsim_linear_i8, maxsim_linear_mx4, maxsim_logprob_bwd,
                      maxsim_logprob_fwd, maxsim_logprob_workspace, maxsim_normalize_bwd,
                      maxsim_normalize_fwd, maxsim_quantize_mx4, maxsim_quantize_tok, maxsim_status_string, maxsim_topk,
                      two_stage_topk, two_stage_topk_mx4)

__all__ = ["MaxSimError", "maxsim_fwd", "maxsim_fwd_varlen", "maxsim_fwd_i8", "maxsim_fwd_i8_tok",
           "maxsim_fwd_pairs", "maxsim_fwd_pairs_varlen", "maxsim_topk", "two_stage_topk",
           "maxsim_bwd", "maxsim_bwd_varlen", "maxsim_chamfer_fwd", "maxsim_chamfer_bwd",
           "maxsim_quantize_tok", "maxsim_linear_i8", "maxsim_embed_i8", "embed_tokens_i8",
           "maxsim_normalize_fwd", "maxsim_normalize_bwd", "maxsim_dropout_fwd",
           "maxsim_dropout_bwd",
           "maxsim_quantize_mx4", "maxsim_dequantize_mx4", "maxsim_linear_mx4", "maxsim_fwd_mx4",
           "embed_tokens_mx4", "two_stage_topk_mx4",
           "maxsim_logprob_fwd", "maxsim_logprob_bwd", "maxsim_logprob_workspace",
           "maxsim_status_string", "maxsim_abi_version"]
