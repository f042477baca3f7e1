"""Low-M split-K bf16 GEMM for AMD Instinct MI355X (gfx950).

C = A @ W.T with A [M, K] and W [N, K] bf16, fp32 accumulation, a bf16 (or
fp32) result, K cut into split_k slices whose partials the last-arriving
slice adds in slice order.  The work runs in the HIP kernels of
``_lib/liblowm.so`` (C ABI in ``include/lowm.h``); this package only loads and
calls them.

Beside the GEMM stand the operators of a decode step around it (C ABI in
``include/lowm_ops.h``): residual_norm, quantize_rows,
gemm_i8, moe and token_logprobs; and its attention, over a paged 8-bit cache
(``include/lowm_cache.h``): rotary, cache_append, cache_read, cache_attention,
fork_pages and compact_pages.
"""
from .binding import (MAX_BATCH, BwProbe, GemmDesc, Library, LowmError, Tactic,
                      batched_workspace_bytes, counter_bytes, gemm, gemm_batched, load,
                      make_workspace, pick_split_k, tactic, workspace_bytes)
from .cache import (KVCache, cache_append, cache_attention, cache_read, compact_pages, fork_pages,
                    make_cache_attention_workspace, make_kv_cache, make_pages_workspace, rotary,
                    rotary_frequencies)
from .ops import (gemm_i8, make_gemm_i8_workspace, make_moe_workspace,
                  make_token_logprobs_workspace, moe, quantize_rows, residual_norm,
                  token_logprobs)

__all__ = ["MAX_BATCH", "BwProbe", "GemmDesc", "KVCache", "Library", "LowmError", "Tactic",
           "batched_workspace_bytes", "cache_append", "cache_attention", "cache_read",
           "compact_pages", "counter_bytes", "fork_pages", "gemm", "gemm_batched", "gemm_i8",
           "load", "make_cache_attention_workspace", "make_gemm_i8_workspace", "make_kv_cache",
           "make_moe_workspace", "make_pages_workspace", "make_token_logprobs_workspace",
           "make_workspace", "moe", "pick_split_k", "quantize_rows", "residual_norm", "rotary",
           "rotary_frequencies", "tactic", "token_logprobs", "workspace_bytes"]
