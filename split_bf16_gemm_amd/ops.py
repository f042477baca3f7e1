"""The operators that stand next to the low-M GEMM in a decode step, over the
C ABI of include/lowm_ops.h.

Argument checks and marshalling only: every step runs in the HIP kernels of
liblowm.so, on the caller's current stream (or ``stream``), asynchronously and
without allocating beyond the outputs and workspaces a caller does not pass
(those belong to the stream the call runs on).  There is no
fallback: when the library is not built, or a call fails, this raises.
"""
from __future__ import annotations

import ctypes
from typing import Optional

import torch

from . import binding

BF16, F32, I8 = 0, 1, 2
_TYPES = {torch.bfloat16: BF16, torch.float32: F32, torch.int8: I8}
NORM_POST, NORM_NO_PRE, NORM_CENTER = 1, 2, 4
MOE_SIGMOID, MOE_NO_RENORM = 1, 2

_vp, _i, _l, _f = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float


class ResidualNormArgs(ctypes.Structure):
    _fields_ = [("y", _vp), ("r", _vp), ("r_out", _vp), ("x", _vp), ("x_scale", _vp),
                ("w_post", _vp), ("w_pre", _vp), ("gate", _vp),
                ("ld_y", _l), ("ld_r", _l), ("ld_r_out", _l), ("ld_x", _l),
                ("gate_row", _l), ("gate_col", _l), ("M", _i), ("D", _i),
                ("y_type", _i), ("r_type", _i), ("w_type", _i), ("gate_type", _i),
                ("x_type", _i), ("flags", _i),
                ("residual_scale", _f), ("branch_scale", _f), ("eps", _f)]


class GemmI8Args(ctypes.Structure):
    _fields_ = [("A", _vp), ("W", _vp), ("a_scale", _vp), ("w_scale", _vp), ("C", _vp),
                ("workspace", _vp), ("workspace_bytes", ctypes.c_size_t), ("M", _i), ("N", _i),
                ("K", _i), ("a_type", _i), ("c_type", _i)]


class MoeArgs(ctypes.Structure):
    _fields_ = [("x", _vp), ("router", _vp), ("bias", _vp), ("w13", _vp), ("w2", _vp),
                ("out", _vp), ("ids", _vp), ("gates", _vp), ("workspace", _vp),
                ("workspace_bytes", ctypes.c_size_t), ("T", _i), ("D", _i), ("I", _i),
                ("E", _i), ("top_k", _i), ("flags", _i), ("routed_scale", _f)]


class TokenLogprobsArgs(ctypes.Structure):
    _fields_ = [("logits", _vp), ("tokens", _vp), ("logprob", _vp), ("entropy", _vp),
                ("rank", _vp), ("top_logprob", _vp), ("top_id", _vp), ("workspace", _vp),
                ("workspace_bytes", ctypes.c_size_t), ("ld", _l), ("M", _i), ("V", _i),
                ("top_n", _i), ("logits_type", _i), ("tokens_bytes", _i)]


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
        stream = torch.cuda.current_stream(device)
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


def _rows(name: str, t: torch.Tensor, shape, types) -> int:
    """The row pitch of a GPU tensor [M, D] with contiguous rows."""
    if t.dtype not in types:
        raise TypeError(f"{name} must be one of {[str(x) for x in types]}, not {t.dtype}")
    if t.dim() != 2 or (shape is not None and t.shape != shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, not {shape and tuple(shape)}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on the GPU")
    m, d = t.shape
    sm, sd = t.stride()
    if sd != 1 and d > 1:
        raise ValueError(f"{name} must have contiguous rows (stride {sd})")
    return sm if m > 1 and sm >= d else _pitch(name, m, d, sm)


def _pitch(name, m, d, sm) -> int:
    if m > 1 and sm < d:
        raise ValueError(f"{name}'s rows overlap (row stride {sm} of {d} elements)")
    return d


def _dense(name: str, t: torch.Tensor, shape, dtype, device=None):
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, not {t.dtype}")
    if tuple(t.shape) != tuple(shape) or not t.is_contiguous() or not t.is_cuda:
        raise ValueError(f"{name} must be a contiguous GPU tensor of shape {tuple(shape)}")


_REAL = (torch.bfloat16, torch.float32)


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
    ld_r = _rows("residual", residual, None, _REAL)
    shape = residual.shape
    ld_y = _rows("y", y, shape, _REAL)
    M, D = shape
    dev = residual.device
    if residual_out is None:
        residual_out = _empty(shape, residual.dtype, dev, stream)
    flags = (NORM_POST if post_norm else 0) | (NORM_CENTER if center else 0)
    a = ResidualNormArgs(y=y.data_ptr(), r=residual.data_ptr(), r_out=residual_out.data_ptr(),
                         ld_y=ld_y, ld_r=ld_r,
                         ld_r_out=_rows("residual_out", residual_out, shape, (residual.dtype,)),
                         M=M, D=D, y_type=_TYPES[y.dtype], r_type=_TYPES[residual.dtype],
                         residual_scale=residual_scale, branch_scale=branch_scale, eps=eps)
    wtype = None
    if post_norm and post_weight is not None:
        wtype = post_weight.dtype
        _need(wtype in _REAL, "post_weight must be bf16 or fp32", TypeError)
        _dense("post_weight", post_weight, (D,), wtype)
        a.w_post = post_weight.data_ptr()
    if pre_norm and pre_weight is not None:
        _need(wtype in (None, pre_weight.dtype) and pre_weight.dtype in _REAL,
              "post_weight and pre_weight must both be bf16 or both fp32", TypeError)
        wtype = pre_weight.dtype
        _dense("pre_weight", pre_weight, (D,), wtype)
        a.w_pre = pre_weight.data_ptr()
    if wtype is not None:
        a.w_type = _TYPES[wtype]
    if gate is not None:
        _need(gate.dtype in _REAL, "gate must be bf16 or fp32", TypeError)
        _need(gate.is_cuda, "gate must be on the GPU")
        if gate.dim() == 1 and gate.shape[0] == D:
            row, col = 0, gate.stride(0)
        elif gate.dim() == 2 and gate.shape[0] in (1, M) and gate.shape[1] in (1, D):
            row = gate.stride(0) if gate.shape[0] == M and M > 1 else 0
            col = gate.stride(1) if gate.shape[1] == D and D > 1 else 0
        else:
            raise ValueError(f"gate has shape {tuple(gate.shape)}: not [{D}], [{M}, 1] or "
                             f"[{M}, {D}]")
        if D == 1:
            col = 0
        _need(col in (0, 1) and row >= 0, "gate must have contiguous rows")
        a.gate, a.gate_type, a.gate_row, a.gate_col = (gate.data_ptr(), _TYPES[gate.dtype], row,
                                                       col)
    if pre_norm:
        want = torch.int8 if quantize else torch.bfloat16
        if out is None:
            out = _empty(shape, want, dev, stream)
        a.ld_x = _rows("out", out, shape, (want,))
        a.x, a.x_type = out.data_ptr(), I8 if quantize else BF16
        if quantize:
            if scale_out is None:
                scale_out = _empty((M,), torch.float32, dev, stream)
            _dense("scale_out", scale_out, (M,), torch.float32)
            a.x_scale = scale_out.data_ptr()
    else:
        _need(not quantize, "quantize needs pre_norm")
        flags |= NORM_NO_PRE
        out = None
    a.flags = flags
    _check((_lib or library()).lib.lowm_residual_norm(ctypes.byref(a), _stream(stream, dev)))
    return residual_out, out, scale_out if quantize else None


def quantize_rows(x: torch.Tensor, *, out: Optional[torch.Tensor] = None,
                  scale_out: Optional[torch.Tensor] = None, stream=None):
    """(q, scale): int8 rows q = rint(x / scale), scale = max|x| / 127 per row
    (fp32), of x [M, K] bf16 or fp32.  A row with an infinity or a NaN gets the
    scale NaN."""
    ld = _rows("x", x, None, _REAL)
    M, K = x.shape
    if out is None:
        out = _empty((M, K), torch.int8, x.device, stream)
    if scale_out is None:
        scale_out = _empty((M,), torch.float32, x.device, stream)
    _dense("out", out, (M, K), torch.int8)
    _dense("scale_out", scale_out, (M,), torch.float32)
    _check((_lib or library()).lib.lowm_quantize_rows(
        x.data_ptr(), _TYPES[x.dtype], ld, M, K, out.data_ptr(), scale_out.data_ptr(),
        _stream(stream, x.device)))
    return out, scale_out


def make_gemm_i8_workspace(M: int, N: int, K: int, device="cuda") -> Optional[torch.Tensor]:
    """The workspace of gemm_i8 with a bf16 A of these sizes (None for sizes it rejects)."""
    n = library().lib.lowm_gemm_i8_workspace_bytes(M, N, K)
    return torch.empty(n, dtype=torch.uint8, device=device) if n else None


def gemm_i8(A: torch.Tensor, W: torch.Tensor, w_scale: torch.Tensor, *,
            a_scale: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
            out_dtype: torch.dtype = torch.bfloat16,
            workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """(A @ W.T) * a_scale[:, None] * w_scale on the GPU, W [N, K] int8 with w_scale [N].

    A [M, K], M <= 64: int8 with a_scale [M] (as quantize_rows or residual_norm give them), or
    bf16, quantised per row within the call (``workspace``: make_gemm_i8_workspace)."""
    if A.dim() != 2 or W.dim() != 2 or A.shape[1] != W.shape[1]:
        raise ValueError(f"shapes {tuple(A.shape)} and {tuple(W.shape)} do not chain")
    M, K = A.shape
    N = W.shape[0]
    dev = A.device
    given = A.dtype == torch.int8
    if not given and A.dtype != torch.bfloat16:
        raise TypeError(f"A must be int8 or bfloat16, not {A.dtype}")
    _dense("A", A, (M, K), A.dtype)
    _dense("W", W, (N, K), torch.int8)
    _dense("w_scale", w_scale, (N,), torch.float32)
    if out is None:
        out = _empty((M, N), out_dtype, dev, stream)
    if out.dtype not in _REAL:
        raise TypeError(f"the output must be bf16 or fp32, not {out.dtype}")
    _dense("out", out, (M, N), out.dtype)
    lib = (_lib or library()).lib
    a = GemmI8Args(A.data_ptr(), W.data_ptr(), None, w_scale.data_ptr(), out.data_ptr(), None, 0,
                   M, N, K, I8 if given else BF16, _TYPES[out.dtype])
    if given:
        _need(a_scale is not None, "an int8 A needs a_scale")
        _dense("a_scale", a_scale, (M,), torch.float32)
        a.a_scale = a_scale.data_ptr()
    else:
        _need(a_scale is None, "a bf16 A takes no a_scale")
        if workspace is None:
            need = lib.lowm_gemm_i8_workspace_bytes(M, N, K)
            workspace = _empty((need,), torch.uint8, dev, stream) if need else None
        if workspace is not None:
            a.workspace = workspace.data_ptr()
            a.workspace_bytes = workspace.numel() * workspace.element_size()
    _check(lib.lowm_gemm_i8(ctypes.byref(a), _stream(stream, dev)))
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
    if x.dim() != 2 or router.dim() != 2 or w13.dim() != 3 or w2.dim() != 3:
        raise ValueError("x and router must have two dimensions, w13 and w2 three")
    T, D = x.shape
    E, _, I = w2.shape
    for name, t, shape in (("x", x, (T, D)), ("router", router, (E, D)),
                           ("w13", w13, (E, 2 * I, D)), ("w2", w2, (E, D, I))):
        _dense(name, t, shape, torch.bfloat16)
    if score not in ("softmax", "sigmoid"):
        raise ValueError(f"score must be 'softmax' or 'sigmoid', not {score!r}")
    dev = x.device
    if out is None:
        out = _empty((T, D), torch.bfloat16, dev, stream)
    if ids_out is None:
        ids_out = _empty((T, top_k), torch.int32, dev, stream)
    if gates_out is None:
        gates_out = _empty((T, top_k), torch.float32, dev, stream)
    _dense("out", out, (T, D), torch.bfloat16)
    _dense("ids_out", ids_out, (T, top_k), torch.int32)
    _dense("gates_out", gates_out, (T, top_k), torch.float32)
    if bias is not None:
        _dense("bias", bias, (E,), torch.float32)
    if workspace is None or not workspace.is_cuda or not workspace.is_contiguous():
        raise ValueError("moe needs a zeroed workspace on the GPU (make_moe_workspace)")
    a = MoeArgs(x.data_ptr(), router.data_ptr(), None if bias is None else bias.data_ptr(),
                w13.data_ptr(), w2.data_ptr(), out.data_ptr(), ids_out.data_ptr(),
                gates_out.data_ptr(), workspace.data_ptr(),
                workspace.numel() * workspace.element_size(), T, D, I, E, top_k,
                (MOE_SIGMOID if score == "sigmoid" else 0)
                | (0 if renormalize else MOE_NO_RENORM), routed_scale)
    _check((_lib or library()).lib.lowm_moe(ctypes.byref(a), _stream(stream, dev)))
    return out, ids_out, gates_out


def make_token_logprobs_workspace(M: int, V: int, top_n: int = 0,
                                  device="cuda") -> Optional[torch.Tensor]:
    """The workspace of token_logprobs for these sizes (None where it needs none)."""
    n = library().lib.lowm_token_logprobs_workspace_bytes(M, V, top_n)
    return torch.empty(n, dtype=torch.uint8, device=device) if n else None


def token_logprobs(logits: torch.Tensor, tokens: torch.Tensor, top_n: int = 0, *,
                   workspace: Optional[torch.Tensor] = None, outs=None, stream=None):
    """(logprob [M], entropy [M], rank [M], top_logprob [M, top_n], top_id [M, top_n]) of
    logits [M, V] (bf16 or fp32; -inf masks a token) and the given tokens [M] (int64 or int32).

    logprob and entropy are those of softmax(logits); rank counts the logits greater than the
    token's; the alternatives are the top_n most likely tokens, equal ones by id, -1 past the last
    unmasked one.  fp32 and int32 outputs (``outs``: five tensors to write into)."""
    ld = _rows("logits", logits, None, _REAL)
    M, V = logits.shape
    dev = logits.device
    if tokens.dtype not in (torch.int64, torch.int32):
        raise TypeError(f"tokens must be int64 or int32, not {tokens.dtype}")
    _dense("tokens", tokens, (M,), tokens.dtype)
    if outs is None:
        outs = tuple(_empty(s, t, dev, stream)
                     for s, t in (((M,), torch.float32), ((M,), torch.float32),
                                  ((M,), torch.int32), ((M, top_n), torch.float32),
                                  ((M, top_n), torch.int32)))
    else:
        for name, t, shape, dtype in zip(
                ("logprob", "entropy", "rank", "top_logprob", "top_id"), outs,
                ((M,), (M,), (M,), (M, top_n), (M, top_n)),
                (torch.float32, torch.float32, torch.int32, torch.float32, torch.int32)):
            _dense(name, t, shape, dtype)
    lib = (_lib or library()).lib
    if workspace is None:
        need = lib.lowm_token_logprobs_workspace_bytes(M, V, top_n)
        workspace = _empty((need,), torch.uint8, dev, stream) if need else None
    a = TokenLogprobsArgs(
        logits.data_ptr(), tokens.data_ptr(), outs[0].data_ptr(), outs[1].data_ptr(),
        outs[2].data_ptr(), outs[3].data_ptr(), outs[4].data_ptr(),
        0 if workspace is None else workspace.data_ptr(),
        0 if workspace is None else workspace.numel() * workspace.element_size(),
        ld, M, V, top_n, _TYPES[logits.dtype], tokens.element_size())
    _check(lib.lowm_token_logprobs(ctypes.byref(a), _stream(stream, dev)))
    return tuple(outs)
