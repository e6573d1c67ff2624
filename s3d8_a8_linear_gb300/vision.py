"""A vision decoder's calls: normed rotary heads as tensors, attention of text tokens to
the encoder's states of their images, and the next token of each sequence.

As the rest of the binding, this module checks tensors and passes pointers and the
current stream; the work is in the CUDA library (``include/s3d8.h`` holds the formulas,
layouts and errors).

NormRope and CrossAttention may be captured into a CUDA graph with their backward pass, while
no eager autograd graph of the same leaves is alive: autograd joins that graph's stream to the
captured one, which CUDA refuses.
"""
from __future__ import annotations

import ctypes

import torch

from . import _check, _dev, _stream
from . import load as _load
from .decoder import _BF, _F, _F32, _I32T, _I64, _P, _SZ, _opt, _rows, _space, _Two


def declare(L):
    """Argument types of this module's entry points (called by load())."""
    I = ctypes.c_int
    heads = [_P, _Two, _I64, _P, _Two, _I64, _P, _P, _P, _P, _I64, _I64, I, _P, _I64, _I64, _F]
    kv = [_P, _Two, _P, _Two, _P, _Two]
    sizes = [_I64] * 5
    L.s3d8_norm_rope.argtypes = heads + [_P, _P, _P]
    L.s3d8_norm_rope_backward.argtypes = [_P, _Two, _P, _Two] + heads + [_P, _P, _P, _P, _P, _SZ, _P]
    L.s3d8_norm_rope_backward_workspace_size.argtypes = [_I64] * 4
    L.s3d8_cross_attention.argtypes = kv + [_P] + sizes + [_F, _P, _P, _P, _SZ, _P]
    L.s3d8_cross_attention_backward.argtypes = [_P, _Two] + kv + [_P, _P, _P] + sizes + [_F, _P, _P, _P, _P, _SZ, _P]
    L.s3d8_cross_attention_workspace_size.argtypes = sizes
    L.s3d8_cross_attention_backward_workspace_size.argtypes = sizes
    L.s3d8_sample.argtypes = [_P, _I64, _I64, _I64, _P, _P, _P, _P, _P, _P, _P, _P]
    for fn in ("norm_rope_backward", "cross_attention", "cross_attention_backward"):
        getattr(L, "s3d8_" + fn + "_workspace_size").restype = _SZ
    for fn in ("norm_rope", "norm_rope_backward", "cross_attention", "cross_attention_backward", "sample"):
        getattr(L, "s3d8_" + fn).restype = I


_NONE = (None, _Two(0, 0))


def _heads(t, name, shape=None):
    """Pointer and strides (token, head) of a bf16 tensor [tokens, heads, dim]."""
    if t.dim() != 3:
        raise ValueError(f"{name} must be 3-D [tokens, heads, dim], got {tuple(t.shape)}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must be {tuple(shape)}, got {tuple(t.shape)}")
    ptr, st = _rows(t, name, _BF)
    return ptr, _Two(*st)


def _same_device(first, **others):
    """The GPU of the call; every tensor has to be on it."""
    for name, t in others.items():
        if t is not None and t.device != first.device:
            raise ValueError(f"{name} must be on {first.device}, got {t.device}")
    return first.device


# ---- normed rotary heads ----------------------------------------------------


def _norm_rope_args(q, k, q_norm, k_norm, cos, sin, positions, eps, interleaved):
    T, Hq, D = q.shape if q.dim() == 3 else (0, 0, 0)
    args = [*_heads(q, "q"), Hq]
    args += [*_NONE, 0] if k is None else [*_heads(k, "k", (T, k.shape[1] if k.dim() == 3 else 0, D)), k.shape[1]]
    if k is None and k_norm is not None:
        raise ValueError("k_norm belongs to k")
    if (cos is None) != (sin is None):
        raise ValueError("cos and sin come together")
    if cos is not None and cos.dim() != 2:
        raise ValueError(f"cos must be 2-D [max_pos, rotary / 2], got {tuple(cos.shape)}")
    max_pos, half = (0, 0) if cos is None else cos.shape
    _same_device(q, k=k, q_norm=q_norm, k_norm=k_norm, cos=cos, sin=sin, positions=positions)
    return args + [_opt(q_norm, "q_norm", _BF, (D,)), _opt(k_norm, "k_norm", _BF, (D,)), _opt(cos, "cos", _F32),
                   _opt(sin, "sin", _F32, (max_pos, half)), max_pos, 2 * half, interleaved,
                   _opt(positions, "positions", _I32T, (T,)), T, D, eps]


def norm_rope(q: torch.Tensor, k: torch.Tensor | None = None, q_norm: torch.Tensor | None = None,
              k_norm: torch.Tensor | None = None, cos: torch.Tensor | None = None,
              sin: torch.Tensor | None = None, positions: torch.Tensor | None = None, eps: float = 1e-5,
              interleaved: bool = False, q_out: torch.Tensor | None = None, k_out: torch.Tensor | None = None):
    """RMS norm of each head of q [T, Hq, dim] and k [T, Hk, dim] (bf16, views allowed) by
    q_norm, k_norm [dim], and the rotation by cos/sin [max_pos, rotary/2] (fp32) at
    positions [T] (None: 0, 1, ...), in one pass -> (q', k').  What is None is left out."""
    args = _norm_rope_args(q, k, q_norm, k_norm, cos, sin, positions, eps, interleaved)
    if q_out is None:
        q_out = torch.empty(q.shape, dtype=_BF, device=q.device)
    if k is not None and k_out is None:
        k_out = torch.empty(k.shape, dtype=_BF, device=q.device)
    if k is None and k_out is not None:
        raise ValueError("k_out belongs to k")
    st = _load().s3d8_norm_rope(*args, _dev(q_out, "q_out", _BF, q.shape),
                                None if k is None else _dev(k_out, "k_out", _BF, k.shape), _stream(q.device))
    if st:
        _check("s3d8_norm_rope", st)
    return q_out, k_out


def norm_rope_backward_workspace(T: int, Hq: int, Hk: int, dim: int, device="cuda") -> torch.Tensor:
    """A workspace for norm_rope_backward calls of this size, to keep."""
    need = int(_load().s3d8_norm_rope_backward_workspace_size(T, Hq, Hk, dim))
    return torch.empty((max(need, 1),), dtype=torch.uint8, device=device)


def norm_rope_backward(dq: torch.Tensor, dk: torch.Tensor | None, q: torch.Tensor, k: torch.Tensor | None = None,
                       q_norm: torch.Tensor | None = None, k_norm: torch.Tensor | None = None,
                       cos: torch.Tensor | None = None, sin: torch.Tensor | None = None,
                       positions: torch.Tensor | None = None, eps: float = 1e-5, interleaved: bool = False,
                       workspace: torch.Tensor | None = None) -> dict:
    """Gradients of norm_rope: dq, dk are those of (q', k').  Returns a dict with "dq" and,
    where their argument is given, "dk" (bf16), "dq_norm" and "dk_norm" (fp32)."""
    args = _norm_rope_args(q, k, q_norm, k_norm, cos, sin, positions, eps, interleaved)
    if (dk is None) != (k is None):
        raise ValueError("dk belongs to k")
    dev, D = _same_device(q, dq=dq, dk=dk, workspace=workspace), q.shape[2]
    got = {"dq": torch.empty(q.shape, dtype=_BF, device=dev)}
    if k is not None:
        got["dk"] = torch.empty(k.shape, dtype=_BF, device=dev)
    for name, w in (("dq_norm", q_norm), ("dk_norm", k_norm)):
        if w is not None:
            got[name] = torch.empty((D,), dtype=_F32, device=dev)
    L = _load()
    ws = (None, 0)
    if q.shape[0] > 0:
        ws = _space(workspace, lambda: L.s3d8_norm_rope_backward_workspace_size(
            q.shape[0], q.shape[1], 0 if k is None else k.shape[1], D), dev)
    ptr = {name: t.data_ptr() for name, t in got.items()}
    st = L.s3d8_norm_rope_backward(*_heads(dq, "dq", q.shape), *(_NONE if k is None else _heads(dk, "dk", k.shape)),
                                   *args, ptr["dq"], ptr.get("dk"), ptr.get("dq_norm"), ptr.get("dk_norm"), *ws,
                                   _stream(dev))
    if st:
        _check("s3d8_norm_rope_backward", st)
    return got


class NormRope(torch.autograd.Function):
    """norm_rope with its gradients: apply(q, k, q_norm, k_norm, cos, sin, positions, eps,
    interleaved) -> (q', k').  Weight gradients come in the weights' bf16; a second
    derivative through it raises."""

    @staticmethod
    def forward(ctx, q, k=None, q_norm=None, k_norm=None, cos=None, sin=None, positions=None, eps=1e-5,
                interleaved=False):
        ctx.save_for_backward(q, k, q_norm, k_norm, cos, sin, positions)
        ctx.rest = (eps, interleaved)
        return norm_rope(q, k, q_norm, k_norm, cos, sin, positions, eps, interleaved)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dq, dk=None):
        q, k, *rest = ctx.saved_tensors
        g = norm_rope_backward(_rowed(dq), None if k is None else _rowed(dk), q, k, *rest, *ctx.rest)
        w = [None if g.get(n) is None else g[n].to(_BF) for n in ("dq_norm", "dk_norm")]
        return g["dq"], g.get("dk"), *w, None, None, None, None, None


def _rowed(t):
    """A gradient as the library takes it: whole 16-byte rows (autograd may hand over an
    expanded or transposed one)."""
    ok = t.stride(-1) == 1 and all(s % 8 == 0 for s in t.stride()[:-1]) and t.data_ptr() % 16 == 0
    return t if ok else t.clone(memory_format=torch.contiguous_format)


# ---- cross attention --------------------------------------------------------


def cross_attention_workspace(T: int, S: int, Hq: int, heads: int, dim: int, device="cuda") -> torch.Tensor:
    """A workspace for cross_attention calls of this size, to keep."""
    need = int(_load().s3d8_cross_attention_workspace_size(T, S, Hq, heads, dim))
    return torch.empty((max(need, 1),), dtype=torch.uint8, device=device)


def cross_attention_backward_workspace(T: int, S: int, Hq: int, heads: int, dim: int, device="cuda") -> torch.Tensor:
    """A workspace for cross_attention_backward calls of this size, to keep."""
    need = int(_load().s3d8_cross_attention_backward_workspace_size(T, S, Hq, heads, dim))
    return torch.empty((max(need, 1),), dtype=torch.uint8, device=device)


def _cross_args(q, k, v, spans, scale):
    args = [*_heads(q, "q"), *_heads(k, "k"), *_heads(v, "v", k.shape)]
    (T, Hq, D), (S, heads, dim) = q.shape, k.shape
    if D != dim:
        raise ValueError(f"q and k must have the same dim, got {D} and {dim}")
    _same_device(q, k=k, v=v, spans=spans)
    sizes = (T, S, Hq, heads, D)
    return args, _opt(spans, "spans", _I32T, (T, 2)), sizes, D ** -0.5 if scale is None else scale


def cross_attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, spans: torch.Tensor | None = None,
                    scale: float | None = None, out: torch.Tensor | None = None, lse: torch.Tensor | None = None,
                    workspace: torch.Tensor | None = None) -> torch.Tensor:
    """Attention of text tokens q [T, Hq, dim] to an encoder's states k, v [S, heads, dim]
    (bf16, views allowed): token t sees states spans[t, 0] .. spans[t, 1] - 1 (int32 [T, 2];
    None: all of them).  scale defaults to dim ** -0.5.  Returns bf16 [T, Hq, dim]; a token
    that sees nothing gets zeros.  lse [T, Hq] fp32, if given, receives the log-sum-exp of
    the scaled scores."""
    args, sp, sizes, scale = _cross_args(q, k, v, spans, scale)
    dev = _same_device(q, out=out, lse=lse, workspace=workspace)
    if out is None:
        out = torch.empty(q.shape, dtype=_BF, device=dev)
    L = _load()
    ws = _space(workspace, lambda: L.s3d8_cross_attention_workspace_size(*sizes), dev)
    st = L.s3d8_cross_attention(*args, sp, *sizes, scale, _dev(out, "out", _BF, q.shape),
                                None if lse is None else _dev(lse, "lse", _F32, q.shape[:2]), *ws, _stream(dev))
    if st:
        _check("s3d8_cross_attention", st)
    return out


def cross_attention_backward(dout: torch.Tensor, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                             out: torch.Tensor, lse: torch.Tensor, spans: torch.Tensor | None = None,
                             scale: float | None = None, workspace: torch.Tensor | None = None) -> dict:
    """Gradients of cross_attention from that of its output; out and lse as it gave them.
    Returns a dict with "dq", "dk" and "dv" (bf16)."""
    args, sp, sizes, scale = _cross_args(q, k, v, spans, scale)
    dev = _same_device(q, dout=dout, out=out, lse=lse, workspace=workspace)
    got = {"dq": torch.empty(q.shape, dtype=_BF, device=dev)}
    for name in ("dk", "dv"):
        got[name] = torch.empty(k.shape, dtype=_BF, device=dev)
    L = _load()
    ws = _space(workspace, lambda: L.s3d8_cross_attention_backward_workspace_size(*sizes), dev)
    st = L.s3d8_cross_attention_backward(*_heads(dout, "dout", q.shape), *args, _dev(out, "out", _BF, q.shape),
                                         _dev(lse, "lse", _F32, q.shape[:2]), sp, *sizes, scale,
                                         *(got[n].data_ptr() for n in ("dq", "dk", "dv")), *ws, _stream(dev))
    if st:
        _check("s3d8_cross_attention_backward", st)
    return got


class CrossAttention(torch.autograd.Function):
    """cross_attention with its gradients: apply(q, k, v, spans, scale) -> out; a second
    derivative through it raises."""

    @staticmethod
    def forward(ctx, q, k, v, spans=None, scale=None):
        lse = torch.empty(q.shape[:2], dtype=_F32, device=q.device)
        out = cross_attention(q, k, v, spans, scale, lse=lse)
        ctx.save_for_backward(q, k, v, spans, out, lse)
        ctx.scale = scale
        return out

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dout):
        q, k, v, spans, out, lse = ctx.saved_tensors
        g = cross_attention_backward(_rowed(dout), q, k, v, out, lse, spans, ctx.scale)
        return g["dq"], g["dk"], g["dv"], None, None


# ---- the next token ---------------------------------------------------------


def sample(logits: torch.Tensor, u: torch.Tensor, temperature: torch.Tensor | None = None,
           top_k: torch.Tensor | None = None, top_p: torch.Tensor | None = None, min_p: torch.Tensor | None = None,
           tokens: torch.Tensor | None = None, logprob: torch.Tensor | None = None) -> torch.Tensor:
    """The next token of each row of logits [B, V] (bf16) by its uniform number u [B] in
    [0, 1): weights exp((l - max) / temperature), of the first top_k tokens, of the fewest
    that have the share top_p, of those at least min_p times as likely as the first (all
    [B]; None: no limit; a temperature of 0 takes the largest logit).  Returns int32 [B], -1
    where every logit is -inf; logprob [B] fp32, if given, receives the log of the token's
    share of what was kept."""
    if logits.dim() != 2:
        raise ValueError(f"logits must be 2-D [B, V], got {tuple(logits.shape)}")
    B, V = logits.shape
    ptr, (stride,) = _rows(logits, "logits", _BF)
    dev = _same_device(logits, u=u, temperature=temperature, top_k=top_k, top_p=top_p, min_p=min_p, tokens=tokens,
                       logprob=logprob)
    if tokens is None:
        tokens = torch.empty((B,), dtype=_I32T, device=dev)
    st = _load().s3d8_sample(ptr, stride, B, V, _dev(u, "u", _F32, (B,)), _opt(temperature, "temperature", _F32, (B,)),
                             _opt(top_k, "top_k", _I32T, (B,)), _opt(top_p, "top_p", _F32, (B,)),
                             _opt(min_p, "min_p", _F32, (B,)), _dev(tokens, "tokens", _I32T, (B,)),
                             _opt(logprob, "logprob", _F32, (B,)), _stream(dev))
    if st:
        _check("s3d8_sample", st)
    return tokens
