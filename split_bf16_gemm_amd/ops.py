"""The operators that stand next to the low-M GEMM in a decode step, over the
C ABI of include/lowm_ops.h.

Argument checks and marshalling only: every step runs in the HIP kernels of
liblowm.so, on the caller's current stream (or ``stream``), asynchronously and
without allocating beyond the outputs a caller does not pass (those belong to
the stream the call runs on).  There is no
fallback: when the library is not built, or a call fails, this raises.
"""
from __future__ import annotations

import ctypes
import struct
from typing import Optional

import torch

from . import binding

BF16, F32, I8 = 0, 1, 2
_TYPES = {torch.bfloat16: BF16, torch.float32: F32, torch.int8: I8}
NORM_POST, NORM_NO_PRE, NORM_CENTER = 1, 2, 4
MOE_SIGMOID, MOE_NO_RENORM = 1, 2

_vp, _i, _l, _f = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float


def _layout(fields):
    """(ctypes.Structure's fields, struct format) of an argument struct of lowm_ops.h; a call
    packs its values in one go, which costs a fraction of setting a Structure's fields."""
    codes = {_vp: "P", _i: "i", _l: "q", _f: "f", ctypes.c_size_t: "N"}
    names = [(n, t) for types, t in fields for n in types.split()]
    # "0P": the size is rounded up to the struct's alignment, as in C
    form = struct.Struct("@" + "".join(codes[t] for _, t in names) + "0P")
    return names, form


_size = ctypes.c_size_t
_NORM_FIELDS, _NORM = _layout((
    ("y r r_out x x_scale w_post w_pre gate", _vp),
    ("ld_y ld_r ld_r_out ld_x gate_row gate_col", _l),
    ("M D y_type r_type w_type gate_type x_type flags", _i),
    ("residual_scale branch_scale eps", _f)))
_I8_FIELDS, _I8 = _layout((
    ("A W a_scale w_scale C workspace", _vp), ("workspace_bytes", _size),
    ("M N K a_type c_type", _i)))
_MOE_FIELDS, _MOE = _layout((
    ("x router bias w13 w2 out ids gates workspace", _vp), ("workspace_bytes", _size),
    ("T D I E top_k flags", _i), ("routed_scale", _f)))
_LOGPROBS_FIELDS, _LOGPROBS = _layout((
    ("logits tokens logprob entropy rank top_logprob top_id workspace", _vp),
    ("workspace_bytes", _size), ("ld", _l), ("M V top_n logits_type tokens_bytes", _i)))


class ResidualNormArgs(ctypes.Structure):
    _fields_ = _NORM_FIELDS


class GemmI8Args(ctypes.Structure):
    _fields_ = _I8_FIELDS


class MoeArgs(ctypes.Structure):
    _fields_ = _MOE_FIELDS


class TokenLogprobsArgs(ctypes.Structure):
    _fields_ = _LOGPROBS_FIELDS


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


def _stream(stream, device) -> int:
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(device.index)
    return stream.cuda_stream


def _empty(shape, dtype, device, stream) -> torch.Tensor:
    """An uninitialised tensor that belongs to the stream its kernel runs on, so
    that its memory is not handed on while that kernel may still use it."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _check(rc: int):
    if rc:
        library().check(rc)


def _need(ok: bool, what: str, error=ValueError):
    if not ok:
        raise error(what)


_REAL = {torch.bfloat16: BF16, torch.float32: F32}
_ONLY = {t: {t: c} for t, c in _TYPES.items()}


def _rows(name: str, t: torch.Tensor, shape, types):
    """(row pitch, type code) of a GPU tensor [M, D] with contiguous rows."""
    code = types.get(t.dtype)
    if code is None:
        raise TypeError(f"{name} must be one of {[str(x) for x in types]}, not {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on the GPU")
    if t.shape != shape or len(shape) != 2:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, not {tuple(shape)}")
    sm, sd = t.stride()
    m, d = shape
    if sd != 1 and d > 1:
        raise ValueError(f"{name} must have contiguous rows (stride {sd})")
    if sm < d:
        if m > 1:
            raise ValueError(f"{name}'s rows overlap (row stride {sm} of {d} elements)")
        sm = d
    return sm, code


def _dense(name: str, t: torch.Tensor, shape, dtype) -> int:
    """The address of a contiguous GPU tensor of this shape and type."""
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, not {t.dtype}")
    if t.shape != shape or not t.is_contiguous() or not t.is_cuda:
        raise ValueError(f"{name} must be a contiguous GPU tensor of shape {tuple(shape)}")
    return t.data_ptr()


def _gate(gate: torch.Tensor, M: int, D: int):
    """(address, type code, row stride, column stride) of a gate [D], [M, 1] or [M, D]."""
    code = _REAL.get(gate.dtype)
    _need(code is not None, "gate must be bf16 or fp32", TypeError)
    _need(gate.is_cuda, "gate must be on the GPU")
    shape = gate.shape
    if len(shape) == 1 and shape[0] == D:
        row, col = 0, gate.stride(0)
    elif len(shape) == 2 and shape[0] in (1, M) and shape[1] in (1, D):
        row, col = gate.stride()
        if shape[0] == 1:
            row = 0
        if shape[1] == 1:
            col = 0
    else:
        raise ValueError(f"gate has shape {tuple(shape)}: not [{D}], [{M}, 1] or [{M}, {D}]")
    if D == 1:
        col = 0
    _need(col in (0, 1) and row >= 0, "gate must have contiguous rows")
    return gate.data_ptr(), code, row, col


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
    lib = (_lib or library()).lib
    shape, dev = residual.shape, residual.device
    ld_r, r_type = _rows("residual", residual, shape, _REAL)
    ld_y, y_type = _rows("y", y, shape, _REAL)
    M, D = shape
    if residual_out is None:
        residual_out = _empty(shape, residual.dtype, dev, stream)
    ld_r_out, _ = _rows("residual_out", residual_out, shape, _ONLY[residual.dtype])
    flags = (NORM_POST if post_norm else 0) | (NORM_CENTER if center else 0)
    w_post = w_pre = w_type = 0
    first = None
    if post_norm and post_weight is not None:
        first = post_weight.dtype
        _need(first in _REAL, "post_weight must be bf16 or fp32", TypeError)
        w_post, w_type = _dense("post_weight", post_weight, (D,), first), _REAL[first]
    if pre_norm and pre_weight is not None:
        kind = pre_weight.dtype
        _need(kind in _REAL and first in (None, kind),
              "post_weight and pre_weight must both be bf16 or both fp32", TypeError)
        w_pre, w_type = _dense("pre_weight", pre_weight, (D,), kind), _REAL[kind]
    g = g_type = g_row = g_col = 0
    if gate is not None:
        g, g_type, g_row, g_col = _gate(gate, M, D)
    x = x_scale = ld_x = x_type = 0
    if pre_norm:
        want = torch.int8 if quantize else torch.bfloat16
        if out is None:
            out = _empty(shape, want, dev, stream)
        ld_x, x_type = _rows("out", out, shape, _ONLY[want])
        x = out.data_ptr()
        if quantize:
            if scale_out is None:
                scale_out = _empty((M,), torch.float32, dev, stream)
            x_scale = _dense("scale_out", scale_out, (M,), torch.float32)
    else:
        _need(not quantize, "quantize needs pre_norm")
        flags |= NORM_NO_PRE
        out = None
    rc = lib.lowm_residual_norm(
        _NORM.pack(y.data_ptr(), residual.data_ptr(), residual_out.data_ptr(), x, x_scale, w_post,
                   w_pre, g, ld_y, ld_r, ld_r_out, ld_x, g_row, g_col, M, D, y_type, r_type,
                   w_type, g_type, x_type, flags, residual_scale, branch_scale, eps),
        _stream(stream, dev))
    if rc:
        _check(rc)
    return residual_out, out, scale_out if quantize else None


def quantize_rows(x: torch.Tensor, *, out: Optional[torch.Tensor] = None,
                  scale_out: Optional[torch.Tensor] = None, stream=None):
    """(q, scale): int8 rows q = rint(x / scale), scale = max|x| / 127 per row
    (fp32), of x [M, K] bf16 or fp32.  A row with an infinity or a NaN gets the
    scale NaN."""
    ld, kind = _rows("x", x, x.shape, _REAL)
    M, K = x.shape
    if out is None:
        out = _empty((M, K), torch.int8, x.device, stream)
    if scale_out is None:
        scale_out = _empty((M,), torch.float32, x.device, stream)
    q = _dense("out", out, (M, K), torch.int8)
    scale = _dense("scale_out", scale_out, (M,), torch.float32)
    rc = (_lib or library()).lib.lowm_quantize_rows(x.data_ptr(), kind, ld, M, K, q, scale,
                                                    _stream(stream, x.device))
    if rc:
        _check(rc)
    return out, scale_out


def make_gemm_i8_workspace(M: int, N: int, K: int, device="cuda") -> Optional[torch.Tensor]:
    """A zeroed workspace of gemm_i8 for these sizes (None for sizes it rejects); it also serves
    any other sizes that need no more bytes, one call at a time."""
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
    lib = (_lib or library()).lib
    a_shape, w_shape = A.shape, W.shape
    if len(a_shape) != 2 or len(w_shape) != 2 or a_shape[1] != w_shape[1]:
        raise ValueError(f"shapes {tuple(a_shape)} and {tuple(w_shape)} do not chain")
    M, K = a_shape
    N = w_shape[0]
    dev, kind = A.device, A.dtype
    given = kind == torch.int8
    if not given and kind != torch.bfloat16:
        raise TypeError(f"A must be int8 or bfloat16, not {kind}")
    if out is None:
        out = _empty((M, N), out_dtype, dev, stream)
    c_type = _REAL.get(out.dtype)
    if c_type is None:
        raise TypeError(f"the output must be bf16 or fp32, not {out.dtype}")
    sa = ws = ws_bytes = 0
    if given:
        _need(a_scale is not None, "an int8 A needs a_scale")
        sa = _dense("a_scale", a_scale, (M,), torch.float32)
    else:
        _need(a_scale is None, "a bf16 A takes no a_scale")
    if workspace is not None:
        _need(workspace.is_cuda and workspace.is_contiguous(),
              "the workspace must be a contiguous GPU tensor (make_gemm_i8_workspace)")
        ws, ws_bytes = workspace.data_ptr(), workspace.nbytes
    elif not given:
        raise ValueError("a bf16 A needs a zeroed workspace (make_gemm_i8_workspace)")
    rc = lib.lowm_gemm_i8(
        _I8.pack(_dense("A", A, a_shape, kind), _dense("W", W, w_shape, torch.int8), sa,
                 _dense("w_scale", w_scale, (N,), torch.float32),
                 _dense("out", out, (M, N), out.dtype), ws, ws_bytes, M, N, K,
                 I8 if given else BF16, c_type), _stream(stream, dev))
    if rc:
        _check(rc)
    return out


def make_moe_workspace(T: int, D: int, I: int, E: int, top_k: int,
                       device="cuda") -> Optional[torch.Tensor]:
    """A zeroed workspace of moe for these sizes (None for sizes it rejects); it also serves
    any other sizes that need no more bytes, one call at a time."""
    n = library().lib.lowm_moe_workspace_bytes(T, D, I, E, top_k)
    return torch.zeros(n, dtype=torch.uint8, device=device) if n else None


def moe(x: torch.Tensor, router: torch.Tensor, w13: torch.Tensor, w2: torch.Tensor, top_k: int, *,
        score: str = "softmax", bias: Optional[torch.Tensor] = None, renormalize: bool = True,
        routed_scale: float = 1.0, workspace: torch.Tensor, out: Optional[torch.Tensor] = None,
        ids_out: Optional[torch.Tensor] = None, gates_out: Optional[torch.Tensor] = None,
        stream=None):
    """(out [T, D], ids [T, top_k], gates [T, top_k]) of a mixture-of-experts layer for T <= 64
    tokens x [T, D]: router [E, D], w13 [E, 2I, D] (gate rows, then up rows), w2 [E, D, I], all
    contiguous bf16.

    Each token takes the top_k experts with the largest router logits, or with a ``bias`` [E]
    (fp32) the largest score + bias; its gates are their scores ("softmax" over the experts or
    "sigmoid"), divided by their sum with ``renormalize``, times ``routed_scale``; out is the
    gated sum of w2 (silu(w13_gate x) * (w13_up x)).  workspace: make_moe_workspace."""
    lib = (_lib or library()).lib
    if x.dim() != 2 or w2.dim() != 3:
        raise ValueError("x must have two dimensions, w2 three")
    T, D = x.shape
    E, _, I = w2.shape
    if score not in ("softmax", "sigmoid"):
        raise ValueError(f"score must be 'softmax' or 'sigmoid', not {score!r}")
    dev = x.device
    if out is None:
        out = _empty((T, D), torch.bfloat16, dev, stream)
    if ids_out is None:
        ids_out = _empty((T, top_k), torch.int32, dev, stream)
    if gates_out is None:
        gates_out = _empty((T, top_k), torch.float32, dev, stream)
    if workspace is None or not workspace.is_cuda or not workspace.is_contiguous():
        raise ValueError("moe needs a zeroed workspace on the GPU (make_moe_workspace)")
    half = torch.bfloat16
    rc = lib.lowm_moe(
        _MOE.pack(_dense("x", x, (T, D), half), _dense("router", router, (E, D), half),
                  0 if bias is None else _dense("bias", bias, (E,), torch.float32),
                  _dense("w13", w13, (E, 2 * I, D), half), _dense("w2", w2, (E, D, I), half),
                  _dense("out", out, (T, D), half),
                  _dense("ids_out", ids_out, (T, top_k), torch.int32),
                  _dense("gates_out", gates_out, (T, top_k), torch.float32),
                  workspace.data_ptr(), workspace.nbytes, T, D, I, E, top_k,
                  (MOE_SIGMOID if score == "sigmoid" else 0)
                  | (0 if renormalize else MOE_NO_RENORM), routed_scale),
        _stream(stream, dev))
    if rc:
        _check(rc)
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
    lib = (_lib or library()).lib
    ld, kind = _rows("logits", logits, logits.shape, _REAL)
    M, V = logits.shape
    dev, t_type = logits.device, tokens.dtype
    if t_type not in (torch.int64, torch.int32):
        raise TypeError(f"tokens must be int64 or int32, not {t_type}")
    f32, i32 = torch.float32, torch.int32
    if outs is None:
        outs = (_empty((M,), f32, dev, stream), _empty((M,), f32, dev, stream),
                _empty((M,), i32, dev, stream), _empty((M, top_n), f32, dev, stream),
                _empty((M, top_n), i32, dev, stream))
    logprob, entropy, rank, top_logprob, top_id = outs
    need = lib.lowm_token_logprobs_workspace_bytes(M, V, top_n)
    ws = ws_bytes = 0
    if need:
        if workspace is None or not workspace.is_cuda or not workspace.is_contiguous():
            raise ValueError(f"{M} rows of {V} need a zeroed workspace on the GPU "
                             "(make_token_logprobs_workspace)")
        ws, ws_bytes = workspace.data_ptr(), workspace.nbytes
    rc = lib.lowm_token_logprobs(
        _LOGPROBS.pack(logits.data_ptr(), _dense("tokens", tokens, (M,), t_type),
                       _dense("logprob", logprob, (M,), f32),
                       _dense("entropy", entropy, (M,), f32), _dense("rank", rank, (M,), i32),
                       _dense("top_logprob", top_logprob, (M, top_n), f32),
                       _dense("top_id", top_id, (M, top_n), i32), ws, ws_bytes, ld, M, V, top_n,
                       kind, 8 if t_type == torch.int64 else 4),
        _stream(stream, dev))
    if rc:
        _check(rc)
    return logprob, entropy, rank, top_logprob, top_id
