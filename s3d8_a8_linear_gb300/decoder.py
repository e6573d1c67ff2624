"""Between two S3D8 linears of a text decoder: residual norms, rotary append into
a paged key/value cache, attention of one new token over it, and its pages.

As the rest of the binding, this module checks tensors and passes pointers and
the current stream; the work is in the CUDA library (``include/s3d8.h`` holds the
formulas, layouts and errors).
"""
from __future__ import annotations

import ctypes

import torch

from . import _check, _dev, _stream
from . import load as _load

KV_BF16, KV_INT8 = 0, 1
MAX_NORM_D = 16384

_P, _I64, _I32, _SZ, _F = (ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_size_t,
                           ctypes.c_float)


class KVCacheStruct(ctypes.Structure):
    """Mirror of s3d8_kv_cache (include/s3d8.h)."""
    _fields_ = [("k", _P), ("v", _P), ("k_scale", _P), ("v_scale", _P), ("k_stride", _I64 * 3),
                ("v_stride", _I64 * 3), ("scale_stride", _I64 * 3), ("pages", _I64),
                ("page_size", _I32), ("heads", _I32), ("dim", _I32), ("dtype", _I32)]


def declare(L):
    """Argument types of this module's entry points (called by load())."""
    cache, two = ctypes.POINTER(KVCacheStruct), _I64 * 2
    L.s3d8_residual_norm.argtypes = [_P, _P, _P, _P, _I64, ctypes.c_int, _P, _F, _F, _I64, _I64, _P,
                                     _P, _P, _P, _P]
    L.s3d8_residual_norm_backward.argtypes = [_P, _P, _P, _P, _P, _P, _I64, ctypes.c_int, _P, _F, _F,
                                              _I64, _I64, _P, _P, _P, _P, _P, _P, _SZ, _P]
    L.s3d8_residual_norm_backward_workspace_size.argtypes = [_I64, _I64]
    L.s3d8_rope_append.argtypes = [_P, two, _P, two, _P, two, _P, _P, _I64, _I64, ctypes.c_int, _P,
                                   _P, _I64, _I64, _P, _I64, _I64, cache, _P, _P]
    L.s3d8_norm_rope_append.argtypes = [_P, two, _P, two, _P, two, _P, _P, _I64, _I64, ctypes.c_int, _P,
                                        _P, _I64, _I64, _P, _I64, _I64, _P, _P, _F, cache, _P, _P]
    L.s3d8_paged_attention_workspace_size.argtypes = [cache, _I64, _I64]
    L.s3d8_paged_attention.argtypes = [_P, cache, _P, _I64, _P, _I64, _I64, _F, _I64, _P, _P, _P, _SZ, _P]
    L.s3d8_pages_workspace_size.argtypes = [_I64, _I64]
    L.s3d8_copy_pages.argtypes = [cache, _I64, _P, _P, _I64, _P]
    L.s3d8_extend_pages.argtypes = [_P, _I64, _I64, _P, _P, _I64, _I64, _P, _P, _I64, _P, _P, _SZ, _P]
    L.s3d8_fork_pages.argtypes = [cache, _I64, _P, _I64, _I64, _P, _P, _P, _P, _I64, _P, _P, _SZ, _P]
    L.s3d8_free_pages.argtypes = [_P, _I64, _I64, _P, _P, _I64, _P, _I64, _P]
    L.s3d8_compact_pages.argtypes = [cache, _I64, _P, _I64, _I64, _P, _P, _P, _SZ, _P]
    for fn in ("residual_norm_backward_workspace_size", "paged_attention_workspace_size",
               "pages_workspace_size"):
        getattr(L, "s3d8_" + fn).restype = _SZ
    for fn in ("residual_norm", "residual_norm_backward", "rope_append", "norm_rope_append",
               "paged_attention", "copy_pages", "extend_pages", "fork_pages", "free_pages", "compact_pages"):
        getattr(L, "s3d8_" + fn).restype = ctypes.c_int


def _opt(t, name, dtype, shape=None):
    return None if t is None else _dev(t, name, dtype, shape)


def _rows(t, name, dtype):
    """Pointer and leading strides of a CUDA tensor whose last axis is contiguous."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    *lead, last = t.stride()
    if last != 1 and t.shape[-1] != 1:
        raise ValueError(f"{name} must have contiguous columns")
    return t.data_ptr(), _strides(t.shape, lead) if 1 in t.shape else lead


def _strides(shape, strides):
    """The strides that matter: an axis of one element may have any (here 0)."""
    return [st if n > 1 else 0 for n, st in zip(shape, strides)]


def _space(workspace, need, device):
    """The caller's workspace, or a new one of need() bytes; its pointer and size."""
    if workspace is None:
        workspace = torch.empty((max(need(), 1),), dtype=torch.uint8, device=device)
    return _dev(workspace, "workspace", torch.uint8), workspace.numel()


# ---- residual norms ---------------------------------------------------------


_BF, _I8, _I32T, _F32 = torch.bfloat16, torch.int8, torch.int32, torch.float32


def _norm_args(h, y, w_post, gate, w_pre, tanh_gate, shape):
    """The arguments that both directions begin with (behind the pointer of h)."""
    if len(shape) != 2:
        raise ValueError("h must be 2-D [M, D]")
    cols = shape[1:]
    n = 0
    if gate is not None:
        n = gate.numel()
        if gate.dim() != 1:
            raise ValueError(f"gate must be 1-D, got {tuple(gate.shape)}")
    return (None if y is None else _dev(y, "y", _BF, shape),
            None if w_post is None else _dev(w_post, "w_post", _BF, cols),
            None if gate is None else _dev(gate, "gate", _BF), n, tanh_gate,
            None if w_pre is None else _dev(w_pre, "w_pre", _BF, cols))


def residual_norm(h: torch.Tensor, y: torch.Tensor | None = None, w_post: torch.Tensor | None = None,
                  gate: torch.Tensor | None = None, w_pre: torch.Tensor | None = None,
                  alpha: float = 1.0, eps: float = 1e-5, tanh_gate: bool = False,
                  h_out: torch.Tensor | None = None, x: torch.Tensor | None = None):
    """h' = h + alpha g norm(y) w_post and x = norm(h') w_pre on bf16 [M, D] ->
    (h', x).  Without w_post y enters as it is; without y the stream stays (h' is
    h); without w_pre there is no x (None).  gate: bf16 [1] or [D], through tanh
    with tanh_gate.  h_out may be h."""
    shape = h.shape
    args = _norm_args(h, y, w_post, gate, w_pre, tanh_gate, shape)
    if w_pre is not None and x is None:
        x = torch.empty_like(h)
    h_out = _stream_out(h, y, h_out)
    st = _load().s3d8_residual_norm(_dev(h, "h", _BF), *args, alpha, eps, shape[0], shape[1],
                                    None if y is None else _dev(h_out, "h_out", _BF, shape),
                                    None if x is None else _dev(x, "x", _BF, shape), None, None,
                                    _stream(h.device))
    if st:
        _check("s3d8_residual_norm", st)
    return h_out, x


def _stream_out(h, y, h_out):
    if y is None:
        if h_out is not None:
            raise ValueError("h_out needs y: without a block's output the stream does not change")
        return h
    return torch.empty_like(h) if h_out is None else h_out


def residual_norm_quant(h: torch.Tensor, y: torch.Tensor | None = None,
                        w_post: torch.Tensor | None = None, gate: torch.Tensor | None = None,
                        w_pre: torch.Tensor | None = None, alpha: float = 1.0, eps: float = 1e-5,
                        tanh_gate: bool = False, h_out: torch.Tensor | None = None,
                        xq: torch.Tensor | None = None, xscale: torch.Tensor | None = None):
    """As residual_norm with x as the codes and scales that quantize_act gives for
    it -> (h', xq int8 [M, D], xscale fp32 [M]), ready for linear()."""
    if w_pre is None:
        raise ValueError("residual_norm_quant needs w_pre")
    shape, dev = h.shape, h.device
    args = _norm_args(h, y, w_post, gate, w_pre, tanh_gate, shape)
    if xq is None:
        xq = torch.empty(shape, dtype=_I8, device=dev)
    if xscale is None:
        xscale = torch.empty(shape[:1], dtype=_F32, device=dev)
    h_out = _stream_out(h, y, h_out)
    st = _load().s3d8_residual_norm(_dev(h, "h", _BF), *args, alpha, eps, shape[0], shape[1],
                                    None if y is None else _dev(h_out, "h_out", _BF, shape), None,
                                    _dev(xq, "xq", _I8, shape), _dev(xscale, "xscale", _F32, shape[:1]),
                                    _stream(dev))
    if st:
        _check("s3d8_residual_norm", st)
    return h_out, xq, xscale


def residual_norm_backward_workspace(M: int, D: int, device="cuda") -> torch.Tensor:
    """A workspace for residual_norm_backward calls of this size, to keep."""
    need = int(_load().s3d8_residual_norm_backward_workspace_size(M, D))
    return torch.empty((max(need, 1),), dtype=torch.uint8, device=device)


def residual_norm_backward(dh: torch.Tensor | None, dx: torch.Tensor | None, h: torch.Tensor,
                           y: torch.Tensor | None = None, w_post: torch.Tensor | None = None,
                           gate: torch.Tensor | None = None, w_pre: torch.Tensor | None = None,
                           alpha: float = 1.0, eps: float = 1e-5, tanh_gate: bool = False,
                           workspace: torch.Tensor | None = None) -> dict:
    """Gradients of residual_norm: dh, dx are those of (h', x) (None: zero), h is h'
    as the forward call returned it.  Returns a dict with "dh" (of the forward
    call's h) and, where their argument is given, "dy" (bf16), "dw_post", "dw_pre"
    and "dgate" (fp32)."""
    shape, bf, dev = h.shape, torch.bfloat16, h.device
    args = _norm_args(h, y, w_post, gate, w_pre, tanh_gate, shape)
    M, D = shape
    got = {"dh": torch.empty_like(h)}
    if y is not None:
        got["dy"] = torch.empty_like(h)
    for name, w in (("dw_post", w_post), ("dgate", gate), ("dw_pre", w_pre)):
        if w is not None:
            got[name] = torch.empty(w.shape, dtype=torch.float32, device=dev)
    L = _load()
    ptr = {k: t.data_ptr() for k, t in got.items()}
    ws = (None, 0)
    if M > 0:
        ws = _space(workspace, lambda: L.s3d8_residual_norm_backward_workspace_size(M, D), dev)
    st = L.s3d8_residual_norm_backward(_opt(dh, "dh", bf, shape), _opt(dx, "dx", bf, shape),
                                       _dev(h, "h", bf), *args, alpha, eps, M, D, ptr["dh"], ptr.get("dy"), ptr.get("dw_pre"),
                                       ptr.get("dw_post"), ptr.get("dgate"), *ws, _stream(dev))
    _check("s3d8_residual_norm_backward", st)
    return got


class ResidualNorm(torch.autograd.Function):
    """residual_norm with its gradients: apply(h, y, w_post, gate, w_pre, alpha,
    eps, tanh_gate) -> (h', x).  Weight gradients come in the weights' bf16; a
    second derivative through it raises."""

    @staticmethod
    def forward(ctx, h, y, w_post, gate, w_pre, alpha=1.0, eps=1e-5, tanh_gate=False):
        h_out, x = residual_norm(h, y, w_post, gate, w_pre, alpha, eps, tanh_gate)
        ctx.save_for_backward(h_out, y, w_post, gate, w_pre)
        ctx.rest = (alpha, eps, tanh_gate)
        ctx.set_materialize_grads(False)
        return (h_out.view_as(h_out) if y is None else h_out), x

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dh, dx):
        h, y, w_post, gate, w_pre = ctx.saved_tensors
        if dh is None and dx is None:
            return (None,) * 8
        g = residual_norm_backward(None if dh is None else dh.contiguous(),
                                   None if dx is None else dx.contiguous(), h, y, w_post, gate, w_pre,
                                   *ctx.rest)
        w = [None if g.get(n) is None else g[n].to(torch.bfloat16) for n in ("dw_post", "dgate", "dw_pre")]
        return g["dh"], g.get("dy"), *w, None, None, None


# ---- the paged cache --------------------------------------------------------


class KVCache:
    """One layer's paged cache: k, v [pages, page_size, heads, dim] in bf16, or int8
    with fp32 scales [pages, page_size, heads].  The tensors may be views in any
    memory order (a [pages, heads, page_size, dim] cache is passed transposed) whose
    columns are contiguous.  Holds the tensors; checked once, here."""

    def __init__(self, k: torch.Tensor, v: torch.Tensor, k_scale: torch.Tensor | None = None,
                 v_scale: torch.Tensor | None = None):
        if k.dim() != 4 or k.shape != v.shape:
            raise ValueError(f"k and v must both be [pages, page_size, heads, dim], got "
                             f"{tuple(k.shape)} and {tuple(v.shape)}")
        if k.dtype not in (torch.bfloat16, torch.int8):
            raise TypeError(f"k must be torch.bfloat16 or torch.int8, got {k.dtype}")
        int8 = k.dtype == torch.int8
        if (k_scale is not None) != int8 or (v_scale is not None) != int8:
            raise ValueError("k_scale and v_scale belong to an int8 cache, and to no other")
        s = KVCacheStruct()
        s.k, ks = _rows(k, "k", k.dtype)
        s.v, vs = _rows(v, "v", k.dtype)
        s.k_stride[:], s.v_stride[:] = ks, vs
        if int8:
            scales = _strides(k_scale.shape, k_scale.stride())
            for t, name in ((k_scale, "k_scale"), (v_scale, "v_scale")):
                if t.shape != k.shape[:3] or _strides(t.shape, t.stride()) != scales:
                    raise ValueError(f"{name} must be [pages, page_size, heads], and both laid out alike")
                if not t.is_cuda or t.dtype != torch.float32:
                    raise TypeError(f"{name} must be a CUDA tensor of torch.float32")
            s.k_scale, s.v_scale = k_scale.data_ptr(), v_scale.data_ptr()
            s.scale_stride[:] = scales
        s.pages, s.page_size, s.heads, s.dim = k.shape
        s.dtype = KV_INT8 if int8 else KV_BF16
        if s.dim % 16 or not 16 <= s.dim <= 256:
            raise ValueError(f"dim must be a multiple of 16 up to 256, got {s.dim}")
        self.k, self.v, self.k_scale, self.v_scale, self.struct = k, v, k_scale, v_scale, s
        self.device, self.ref = k.device, ctypes.byref(s)
        self.pages, self.page_size, self.heads, self.dim = k.shape

    @classmethod
    def empty(cls, pages: int, page_size: int, heads: int, dim: int, dtype=torch.bfloat16,
              device="cuda") -> "KVCache":
        """A new cache with each head's tokens of a page together in memory."""
        k, v = (torch.empty((pages, heads, page_size, dim), dtype=dtype, device=device).transpose(1, 2)
                for _ in "kv")
        if dtype != torch.int8:
            return cls(k, v)
        return cls(k, v, *(torch.empty((pages, heads, page_size), dtype=torch.float32,
                                       device=device).transpose(1, 2) for _ in "kv"))


class KVPool:
    """The caches of several layers that share one block table."""

    def __init__(self, caches):
        self.caches = list(caches)
        if not self.caches:
            raise ValueError("a pool needs at least one cache")
        self.array = (KVCacheStruct * len(self.caches))(*[c.struct for c in self.caches])
        self.count, first = len(self.caches), self.caches[0]
        self.device, self.pages, self.page_size = first.device, first.pages, first.page_size


_Two = _I64 * 2


def rope_append(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cos: torch.Tensor, sin: torch.Tensor,
                positions: torch.Tensor, cache: KVCache, table: torch.Tensor,
                rows: torch.Tensor | None = None, q_out: torch.Tensor | None = None,
                interleaved: bool = False, q_norm: torch.Tensor | None = None,
                k_norm: torch.Tensor | None = None, eps: float = 1e-5) -> torch.Tensor:
    """Rotate q [T, Hq, dim] and k [T, heads, dim] by cos/sin [max_pos, rotary/2]
    (fp32) at positions [T], and store k, v as tokens `positions` of the block
    table's rows (rows None: token t of row t).  Returns the rotated q; a negative
    position marks a padding token.  q_norm, k_norm (bf16 [dim]): each head is
    normed in front of its rotation, in the same pass."""
    (qp, qs), (kp, ks), (vp, vs) = _rows(q, "q", _BF), _rows(k, "k", _BF), _rows(v, "v", _BF)
    shape = q.shape
    T, Hq, D = shape
    want = (T, cache.heads, cache.dim)
    if k.shape != want or v.shape != want or D != cache.dim:
        raise ValueError(f"k and v must be {want} and q [{T}, Hq, {cache.dim}], got {tuple(k.shape)}, "
                         f"{tuple(v.shape)} and {tuple(shape)}")
    if q_out is None:
        q_out = torch.empty(shape, dtype=_BF, device=q.device)
    turns = cos.shape
    max_pos, half = turns
    n, width = table.shape
    args = (qp, _Two(*qs), kp, _Two(*ks), vp, _Two(*vs), _dev(cos, "cos", _F32), _dev(sin, "sin", _F32, turns),
            max_pos, 2 * half, interleaved, _dev(positions, "positions", _I32T, shape[:1]),
            None if rows is None else _dev(rows, "rows", _I32T, shape[:1]), T, Hq, _dev(table, "table", _I32T),
            n, width)
    end = (cache.ref, _dev(q_out, "q_out", _BF, shape), _stream(q.device))
    if q_norm is None and k_norm is None:
        st = _load().s3d8_rope_append(*args, *end)
    else:
        for name, w in (("q_norm", q_norm), ("k_norm", k_norm)):
            if w is not None and w.device != q.device:
                raise ValueError(f"{name} must be on {q.device}, got {w.device}")
        st = _load().s3d8_norm_rope_append(*args, _opt(q_norm, "q_norm", _BF, (D,)), _opt(k_norm, "k_norm", _BF, (D,)),
                                           eps, *end)
    if st:
        _check("s3d8_rope_append", st)
    return q_out


def paged_attention_workspace(cache: KVCache, B: int, Hq: int) -> torch.Tensor:
    """A workspace for paged_attention calls of this size, to keep."""
    need = int(_load().s3d8_paged_attention_workspace_size(cache.ref, B, Hq))
    return torch.empty((max(need, 1),), dtype=torch.uint8, device=cache.device)


def paged_attention(q: torch.Tensor, cache: KVCache, table: torch.Tensor, lens: torch.Tensor,
                    scale: float | None = None, window: int = 0, out: torch.Tensor | None = None,
                    lse: torch.Tensor | None = None, workspace: torch.Tensor | None = None) -> torch.Tensor:
    """One new token's attention per sequence: q [B, Hq, dim] over the first lens[b]
    tokens (the last `window` of them, if set) of row b of the block table.  scale
    defaults to dim ** -0.5.  Returns bf16 [B, Hq, dim]; lse [B, Hq] fp32, if
    given, receives the log-sum-exp of the scaled scores."""
    shape, dev = q.shape, q.device
    if len(shape) != 3 or shape[2] != cache.dim:
        raise ValueError(f"q must be [B, Hq, {cache.dim}], got {tuple(shape)}")
    B, Hq, D = shape
    if out is None:
        out = torch.empty_like(q)
    rows, width = table.shape
    if rows != B:
        raise ValueError(f"table must be [{B}, width], got {tuple(table.shape)}")
    L = _load()
    ws = _space(workspace, lambda: L.s3d8_paged_attention_workspace_size(cache.ref, B, Hq), dev)
    st = L.s3d8_paged_attention(_dev(q, "q", _BF), cache.ref, _dev(table, "table", _I32T), width,
                                _dev(lens, "lens", _I32T, shape[:1]), B, Hq,
                                D ** -0.5 if scale is None else scale, window, _dev(out, "out", _BF, shape),
                                None if lse is None else _dev(lse, "lse", _F32, shape[:2]), *ws, _stream(dev))
    if st:
        _check("s3d8_paged_attention", st)
    return out


# ---- pages ------------------------------------------------------------------


def pages_workspace(pool: KVPool, rows: int) -> torch.Tensor:
    """A workspace for the calls below on this pool and a table of `rows` rows."""
    need = int(_load().s3d8_pages_workspace_size(pool.pages, rows))
    return torch.empty((max(need, 1),), dtype=torch.uint8, device=pool.device)


def _table(table, lens, refs):
    i32 = torch.int32
    rows, width = table.shape
    return rows, width, _dev(table, "table", i32), _opt(lens, "lens", i32, (rows,)), _dev(refs, "refs", i32)


def _meta_space(workspace, pages, rows, device):
    return _space(workspace, lambda: _load().s3d8_pages_workspace_size(pages, rows), device)


def copy_pages(pool: KVPool, src: torch.Tensor, dst: torch.Tensor) -> None:
    """Copy page src[i] to page dst[i] (int32) in every layer of the pool; pairs
    with a negative id are skipped."""
    n = src.numel()
    st = _load().s3d8_copy_pages(pool.array, pool.count, _dev(src, "src", torch.int32),
                                 _dev(dst, "dst", torch.int32, tuple(src.shape)), n, _stream(src.device))
    _check("s3d8_copy_pages", st)


def extend_pages(table: torch.Tensor, lens: torch.Tensor, refs: torch.Tensor, seqs: torch.Tensor,
                 add: torch.Tensor, page_size: int, workspace: torch.Tensor | None = None) -> torch.Tensor:
    """Grow rows seqs[i] by add[i] tokens, taking free pages lowest id first.
    Returns got [n] int32: 0 where pages or the table's width did not suffice."""
    rows, width, tp, lp, rp = _table(table, lens, refs)
    n, dev = seqs.numel(), table.device
    got = torch.empty((n,), dtype=torch.int32, device=dev)
    ws = _meta_space(workspace, refs.numel(), rows, dev)
    st = _load().s3d8_extend_pages(tp, rows, width, lp, rp, refs.numel(), page_size,
                                   _dev(seqs, "seqs", torch.int32), _dev(add, "add", torch.int32, (n,)), n,
                                   got.data_ptr(), *ws, _stream(dev))
    _check("s3d8_extend_pages", st)
    return got


def fork_pages(pool: KVPool, table: torch.Tensor, lens: torch.Tensor, refs: torch.Tensor,
               parents: torch.Tensor, children: torch.Tensor,
               workspace: torch.Tensor | None = None) -> torch.Tensor:
    """Make rows children[i] continuations of rows parents[i]: full pages shared, a
    partial last page copied in every layer.  Returns got [n] int32: 0 (and an
    empty child) where no page was left."""
    rows, width, tp, lp, rp = _table(table, lens, refs)
    if refs.numel() != pool.pages:
        raise ValueError(f"refs must have one count per page ({pool.pages}), got {refs.numel()}")
    n, dev = parents.numel(), table.device
    got = torch.empty((n,), dtype=torch.int32, device=dev)
    ws = _meta_space(workspace, pool.pages, rows, dev)
    st = _load().s3d8_fork_pages(pool.array, pool.count, tp, rows, width, lp, rp,
                                 _dev(parents, "parents", torch.int32),
                                 _dev(children, "children", torch.int32, (n,)), n, got.data_ptr(), *ws,
                                 _stream(dev))
    _check("s3d8_fork_pages", st)
    return got


def free_pages(table: torch.Tensor, lens: torch.Tensor, refs: torch.Tensor, seqs: torch.Tensor) -> None:
    """Release rows seqs[i]: one count less for each page held; empty rows."""
    rows, width, tp, lp, rp = _table(table, lens, refs)
    st = _load().s3d8_free_pages(tp, rows, width, lp, rp, refs.numel(), _dev(seqs, "seqs", torch.int32),
                                 seqs.numel(), _stream(table.device))
    _check("s3d8_free_pages", st)


def compact_pages(pool: KVPool, table: torch.Tensor, refs: torch.Tensor,
                  workspace: torch.Tensor | None = None) -> torch.Tensor:
    """Move the live pages to ids 0 .. live-1 in every layer, with refs and table.
    Returns live [1] int32 (on the device)."""
    rows, width, tp, _, rp = _table(table, None, refs)
    if refs.numel() != pool.pages:
        raise ValueError(f"refs must have one count per page ({pool.pages}), got {refs.numel()}")
    live = torch.empty((1,), dtype=torch.int32, device=table.device)
    ws = _meta_space(workspace, pool.pages, rows, table.device)
    st = _load().s3d8_compact_pages(pool.array, pool.count, tp, rows, width, rp, live.data_ptr(), *ws,
                                    _stream(table.device))
    _check("s3d8_compact_pages", st)
    return live
