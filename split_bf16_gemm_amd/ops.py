"""The operators that stand next to the low-M GEMM in a decode step, over the
C ABI of include/lowm_ops.h.

Argument checks and marshalling only (in csrc/ops_binding.cpp): every step runs
in the HIP kernels of liblowm.so, on the caller's current stream (or ``stream``),
asynchronously and without allocating beyond the outputs a caller does not pass
(those belong to the stream the call runs on).  There is no fallback: when a
library is not built, or a call fails, this raises.
"""
from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util
from typing import Optional

import torch

from . import binding

BF16, F32, I8 = 0, 1, 2
NORM_POST, NORM_NO_PRE, NORM_CENTER = 1, 2, 4
MOE_SIGMOID, MOE_NO_RENORM = 1, 2

_vp, _i, _l, _f = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float


_size = ctypes.c_size_t


def _fields(*groups):
    return [(name, kind) for names, kind in groups for name in names.split()]


# The argument structs of lowm_ops.h.
class ResidualNormArgs(ctypes.Structure):
    _fields_ = _fields(("y r r_out x x_scale w_post w_pre gate", _vp),
                       ("ld_y ld_r ld_r_out ld_x gate_row gate_col", _l),
                       ("M D y_type r_type w_type gate_type x_type flags", _i),
                       ("residual_scale branch_scale eps", _f))


class GemmI8Args(ctypes.Structure):
    _fields_ = _fields(("A W a_scale w_scale C workspace", _vp), ("workspace_bytes", _size),
                       ("M N K a_type c_type", _i))


class MoeArgs(ctypes.Structure):
    _fields_ = _fields(("x router bias w13 w2 out ids gates workspace", _vp),
                       ("workspace_bytes", _size), ("T D I E top_k flags", _i),
                       ("routed_scale", _f))


class TokenLogprobsArgs(ctypes.Structure):
    _fields_ = _fields(("logits tokens logprob entropy rank top_logprob top_id workspace", _vp),
                       ("workspace_bytes", _size), ("ld", _l),
                       ("M V top_n logits_type tokens_bytes", _i))


_lib = None


def library() -> binding.Library:
    """liblowm.so with the operators' entry points declared."""
    global _lib
    if _lib is None:
        lib = binding.load()
        c = lib.lib
        c.lowm_residual_norm.argtypes = [_vp, _vp]
        c.lowm_quantize_rows.argtypes = [_vp, _i, _l, _i, _i, _vp, _vp, _vp]
        c.lowm_gemm_i8.argtypes = [_vp, _vp]
        c.lowm_gemm_i8_workspace_bytes.argtypes = [_i, _i, _i]
        c.lowm_gemm_i8_workspace_bytes.restype = ctypes.c_size_t
        c.lowm_moe.argtypes = [_vp, _vp]
        c.lowm_moe_workspace_bytes.argtypes = [_i, _i, _i, _i, _i]
        c.lowm_moe_workspace_bytes.restype = ctypes.c_size_t
        c.lowm_token_logprobs.argtypes = [_vp, _vp]
        c.lowm_token_logprobs_workspace_bytes.argtypes = [_i, _i, _i]
        c.lowm_token_logprobs_workspace_bytes.restype = ctypes.c_size_t
        _lib = lib
    return _lib


_calls = None


def _native():
    """The compiled calls (csrc/ops_binding.cpp), linked against liblowm.so."""
    global _calls
    if _calls is None:
        library()
        path = binding.LIBDIR / "ops_binding.so"
        if not path.exists():
            raise RuntimeError(f"{path.name} is not built; run "
                               "`python -m split_bf16_gemm_amd.build` (there is no fallback)")
        loader = importlib.machinery.ExtensionFileLoader("ops_binding", str(path))
        module = importlib.util.module_from_spec(
            importlib.util.spec_from_loader("ops_binding", loader))
        loader.exec_module(module)
        _calls = module
    return _calls


def _stream(stream, device) -> int:
    if stream is None:
        # a tensor that is not on a GPU is refused by the call itself
        return torch._C._cuda_getCurrentRawStream(device.index) if device.index is not None else 0
    if device.index is not None and stream.device != device:
        raise ValueError(f"the stream is of {stream.device}, the tensors are on {device}")
    return stream.cuda_stream


def _empty(shape, dtype, device, stream) -> torch.Tensor:
    """An uninitialised tensor that belongs to the stream its kernel runs on, so
    that its memory is not handed on while that kernel may still use it."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def residual_norm(y: torch.Tensor, residual: torch.Tensor, *, post_norm: bool = True,
                  post_weight: Optional[torch.Tensor] = None,
                  pre_norm: bool = True, pre_weight: Optional[torch.Tensor] = None,
                  gate: Optional[torch.Tensor] = None, branch_scale: float = 1.0,
                  residual_scale: float = 1.0, eps: float = 1e-6, center: bool = False,
                  quantize: bool = False, residual_out: Optional[torch.Tensor] = None,
                  out: Optional[torch.Tensor] = None, scale_out: Optional[torch.Tensor] = None,
                  stream=None):
    """(r', x, scale) at the border between two blocks:

        p  = norm(y) * post_weight                 (y itself without post_norm)
        r' = residual_scale * residual + branch_scale * gate * p
        x  = norm(r') * pre_weight                 (None without pre_norm)

    y and residual [M, D], bf16 or fp32 each; r' has the residual's type (pass
    ``residual_out=residual`` to update it in place); x is bf16, or with
    ``quantize`` int8 rows with fp32 ``scale`` [M] (else None), as gemm_i8 takes
    them.  gate: [D], [M, 1] or [M, D].  norm: root mean square, or with
    ``center`` also the mean taken off."""
    dev = residual.device
    flags = (NORM_POST if post_norm else 0) | (NORM_CENTER if center else 0)
    if residual_out is None:
        residual_out = _empty(residual.shape, residual.dtype, dev, stream)
    if pre_norm:
        if out is None:
            out = _empty(residual.shape, torch.int8 if quantize else torch.bfloat16, dev, stream)
        if not quantize:
            scale_out = None
        elif scale_out is None:
            scale_out = _empty(residual.shape[:1], torch.float32, dev, stream)
    elif quantize:
        raise ValueError("quantize needs pre_norm")
    else:
        flags |= NORM_NO_PRE
        out = scale_out = pre_weight = None
    rc = (_calls or _native()).residual_norm(
        y, residual, residual_out, out, scale_out, post_weight if post_norm else None, pre_weight,
        gate, flags, residual_scale, branch_scale, eps, _stream(stream, dev))
    if rc:
        library().check(rc)
    return residual_out, out, scale_out


def quantize_rows(x: torch.Tensor, *, out: Optional[torch.Tensor] = None,
                  scale_out: Optional[torch.Tensor] = None, stream=None):
    """(q, scale): int8 rows q = rint(x / scale), scale = max|x| / 127 per row
    (fp32), of x [M, K] bf16 or fp32.  A row with an infinity or a NaN gets the
    scale NaN."""
    dev = x.device
    if out is None:
        out = _empty(x.shape, torch.int8, dev, stream)
    if scale_out is None:
        scale_out = _empty(x.shape[:1], torch.float32, dev, stream)
    rc = (_calls or _native()).quantize_rows(x, out, scale_out, _stream(stream, dev))
    if rc:
        library().check(rc)
    return out, scale_out


def make_gemm_i8_workspace(M: int, N: int, K: int, device="cuda") -> Optional[torch.Tensor]:
    """A zeroed workspace of gemm_i8 for these sizes (None for sizes it rejects); it also serves
    any other sizes that need no more bytes, one call at a time, but no other operator."""
    n = library().lib.lowm_gemm_i8_workspace_bytes(M, N, K)
    return torch.zeros(n, dtype=torch.uint8, device=device) if n else None


def gemm_i8(A: torch.Tensor, W: torch.Tensor, w_scale: torch.Tensor, *,
            a_scale: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
            out_dtype: torch.dtype = torch.bfloat16,
            workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """(A @ W.T) * a_scale[:, None] * w_scale on the GPU, W [N, K] int8 with w_scale [N].

    A [M, K], M <= 64: int8 with a_scale [M] (as quantize_rows or residual_norm give them), or
    bf16, quantised per row within the call.  workspace: make_gemm_i8_workspace; an int8 A does
    without one, but its K is then not split over workgroups."""
    dev = A.device
    if out is None:
        out = _empty((A.shape[0], W.shape[0]), out_dtype, dev, stream)
    rc = (_calls or _native()).gemm_i8(A, W, w_scale, a_scale, out, workspace,
                                       _stream(stream, dev))
    if rc:
        library().check(rc)
    return out


def make_moe_workspace(T: int, D: int, I: int, E: int, top_k: int,
                       device="cuda") -> Optional[torch.Tensor]:
    """A zeroed workspace of moe for these sizes (None for T 0 and for sizes it rejects); it also
    serves any other sizes that need no more bytes, one call at a time, but no other operator."""
    n = library().lib.lowm_moe_workspace_bytes(T, D, I, E, top_k)
    return torch.zeros(n, dtype=torch.uint8, device=device) if n else None


def moe(x: torch.Tensor, router: torch.Tensor, w13: torch.Tensor, w2: torch.Tensor, top_k: int, *,
        score: str = "softmax", bias: Optional[torch.Tensor] = None, renormalize: bool = True,
        routed_scale: float = 1.0, workspace: Optional[torch.Tensor],
        out: Optional[torch.Tensor] = None, ids_out: Optional[torch.Tensor] = None,
        gates_out: Optional[torch.Tensor] = None, stream=None):
    """(out [T, D], ids [T, top_k], gates [T, top_k]) of a mixture-of-experts layer for T <= 64
    tokens x [T, D]: router [E, D], w13 [E, 2I, D] (gate rows, then up rows), w2 [E, D, I], all
    contiguous bf16.

    Each token takes the top_k experts with the largest router logits, or with a ``bias`` [E]
    (fp32) the largest score + bias; its gates are their scores ("softmax" over the experts or
    "sigmoid"), divided by their sum with ``renormalize``, times ``routed_scale``; out is the
    gated sum of w2 (silu(w13_gate x) * (w13_up x)).  workspace: make_moe_workspace (None will do
    where there are no tokens)."""
    if score not in ("softmax", "sigmoid"):
        raise ValueError(f"score must be 'softmax' or 'sigmoid', not {score!r}")
    dev = x.device
    if out is None:
        out = _empty(x.shape, torch.bfloat16, dev, stream)
    if ids_out is None:
        ids_out = _empty((x.shape[0], top_k), torch.int32, dev, stream)
    if gates_out is None:
        gates_out = _empty((x.shape[0], top_k), torch.float32, dev, stream)
    rc = (_calls or _native()).moe(
        x, router, bias, w13, w2, out, ids_out, gates_out, workspace, top_k,
        (MOE_SIGMOID if score == "sigmoid" else 0) | (0 if renormalize else MOE_NO_RENORM),
        routed_scale, _stream(stream, dev))
    if rc:
        library().check(rc)
    return out, ids_out, gates_out


def make_token_logprobs_workspace(M: int, V: int, top_n: int = 0,
                                  device="cuda") -> Optional[torch.Tensor]:
    """A zeroed workspace of token_logprobs for these sizes (None where it needs none); it serves
    any other sizes too, one call at a time."""
    n = library().lib.lowm_token_logprobs_workspace_bytes(M, V, top_n)
    return torch.zeros(n, dtype=torch.uint8, device=device) if n else None


def token_logprobs(logits: torch.Tensor, tokens: torch.Tensor, top_n: int = 0, *,
                   workspace: Optional[torch.Tensor] = None, outs=None, stream=None):
    """(logprob [M], entropy [M], rank [M], top_logprob [M, top_n], top_id [M, top_n]) of
    logits [M, V] (bf16 or fp32; -inf masks a token) and the given tokens [M] (int64 or int32).

    logprob and entropy are those of softmax(logits); rank counts the logits greater than the
    token's; the alternatives are the top_n most likely tokens, equal ones by id, -1 past the last
    unmasked one.  fp32 and int32 outputs (``outs``: five tensors to write into).  workspace:
    make_token_logprobs_workspace (many rows need none)."""
    dev = logits.device
    if outs is None:
        M = logits.shape[:1]
        top = (*M, top_n)
        outs = (_empty(M, torch.float32, dev, stream), _empty(M, torch.float32, dev, stream),
                _empty(M, torch.int32, dev, stream), _empty(top, torch.float32, dev, stream),
                _empty(top, torch.int32, dev, stream))
    logprob, entropy, rank, top_logprob, top_id = outs
    rc = (_calls or _native()).token_logprobs(logits, tokens, top_n, logprob, entropy, rank,
                                              top_logprob, top_id, workspace, _stream(stream, dev))
    if rc:
        library().check(rc)
    return logprob, entropy, rank, top_logprob, top_id
