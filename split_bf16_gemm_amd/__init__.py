"""Low-M split-K bf16 GEMM for AMD Instinct MI355X (gfx950).

C = A @ W.T with A [M, K] and W [N, K] bf16, fp32 accumulation, a bf16 (or
fp32) result, K cut into split_k slices whose partials the last-arriving
slice adds in slice order.  The work runs in the HIP kernels of
``_lib/liblowm.so`` (C ABI in ``include/lowm.h``); this package only loads and
calls them.

Beside the GEMM stand the operators of a decode step around it (C ABI in
``include/lowm_ops.h``): residual_norm, quantize_rows,
gemm_i8, moe and token_logprobs.
"""
from .binding import (MAX_BATCH, BwProbe, GemmDesc, Library, LowmError, Tactic,
                      batched_workspace_bytes, counter_bytes, gemm, gemm_batched, load,
                      make_workspace, pick_split_k, tactic, workspace_bytes)
from .ops import (gemm_i8, make_gemm_i8_workspace, make_moe_workspace,
                  make_token_logprobs_workspace, moe, quantize_rows, residual_norm,
                  token_logprobs)

__all__ = ["MAX_BATCH", "BwProbe", "GemmDesc", "Library", "LowmError", "Tactic",
           "batched_workspace_bytes", "counter_bytes", "gemm", "gemm_batched", "gemm_i8", "load",
           "make_gemm_i8_workspace", "make_moe_workspace", "make_token_logprobs_workspace",
           "make_workspace", "moe", "pick_split_k", "quantize_rows", "residual_norm", "tactic",
           "token_logprobs", "workspace_bytes"]
