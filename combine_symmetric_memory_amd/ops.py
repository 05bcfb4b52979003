"""Python binding of the operators around the MoE path (include/cco_ops.h):
the router, the products grouped by expert and the norms around a block.

    idx, w = route(logits, topk, ...)                    # cco_route
    dlogits = route_grad(logits, idx, dw, ...)           # cco_route_grad
    y  = group_product(first, count, x, w)               # cco_group_product
    dx = group_product_dx(first, count, dy, w)           # cco_group_product_dx
    dw = group_product_dw(first, count, dy, x)           # cco_group_product_dw
    out, u = block_norm(x, y, post=, gate=, pre=)        # cco_block_norm
    dx, dy, dpost, dgate, dpre = block_norm_grad(...)    # cco_block_norm_grad
    out, u, y = combine_norm(moe, x, w, post=, ...)      # cco_moe_combine_norm

Arguments are checked and marshalled here, the work is in the library's HIP
kernels.  Calls run on the tensors' device, on torch's current stream of it
unless `stream` is given; outputs that are not passed are made by torch.
Nothing is recorded for automatic differentiation, whatever the inputs
require: results carry no gradient, the calls named _grad, _dx and _dw
compute it.
"""
from __future__ import annotations

import contextlib
import ctypes

import torch

from . import _capi
from ._capi import check, lib
from .moe import MoE

_DTYPES = {torch.bfloat16: _capi.CCO_BF16, torch.float16: _capi.CCO_F16,
           torch.float32: _capi.CCO_F32}
_SCORES = {"softmax": _capi.CCO_SCORE_SOFTMAX, "sigmoid": _capi.CCO_SCORE_SIGMOID}


class _Elsewhere:
    """The tensors' device made current, and the stream of a call too, so
    that memory torch makes for the call belongs to that stream.  A call on
    torch's current stream of the current device does without."""

    def __init__(self, dev: torch.device, stream):
        self._stack = contextlib.ExitStack()
        self._dev, self._stream = dev, stream

    def __enter__(self):
        s = self._stream
        if isinstance(s, torch.cuda.Stream) and s.device != self._dev:
            raise ValueError("the stream is on %s, the tensors on %s" % (s.device, self._dev))
        self._stack.enter_context(torch.cuda.device(self._dev))
        if s is not None:
            if not isinstance(s, torch.cuda.Stream):
                s = int(s)
                s = torch.cuda.ExternalStream(s) if s else torch.cuda.default_stream()
            self._stack.enter_context(torch.cuda.stream(s))

    def __exit__(self, *exc):
        return self._stack.__exit__(*exc)


# torch's own query without the stream object around it (microseconds, which
# a call for a few tokens would notice), where this torch has it
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _away(dev: torch.device, stream) -> bool:
    return stream is not None or dev.index != torch.cuda.current_device()


def _dtype(t: torch.Tensor, name: str, allowed=None) -> int:
    code = _DTYPES.get(t.dtype)
    if code is None or (allowed is not None and t.dtype not in allowed):
        raise ValueError("%s has the unsupported type %s" % (name, t.dtype))
    return code


def _device(t: torch.Tensor, name: str) -> torch.device:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError("%s must be a device tensor" % name)
    return t.device


def _same(t: torch.Tensor | None, dev: torch.device, name: str, shape=None, dtype=None) -> None:
    """A dense tensor on `dev` of the given shape and type."""
    if t is None:
        return
    if not isinstance(t, torch.Tensor) or t.device != dev:
        raise ValueError("%s must be a tensor on %s" % (name, dev))
    if shape is not None and t.shape != shape:
        raise ValueError("%s must be %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    if dtype is not None and t.dtype != dtype:
        raise ValueError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)


def _rows(t: torch.Tensor, dev, name: str, cols: int | None = None, rows: int | None = None,
          dtype=None) -> int:
    """A [rows][cols] tensor with contiguous rows; returns its row distance."""
    if not isinstance(t, torch.Tensor) or t.device != dev:
        raise ValueError("%s must be a tensor on %s" % (name, dev))
    shape = t.shape
    if len(shape) != 2 or (cols is not None and shape[1] != cols) or \
       (rows is not None and shape[0] != rows):
        raise ValueError("%s must be [%s, %s], got %s" % (
            name, "rows" if rows is None else rows, "columns" if cols is None else cols,
            tuple(shape)))
    r, c = shape
    if r > _MAX_COUNT or c > _MAX_COUNT:
        _counts(name, r, c)
    if dtype is not None and t.dtype != dtype:
        raise ValueError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if t.is_contiguous():
        return c or 1
    ld, step = t.stride()
    if c > 1 and step != 1:
        raise ValueError("the rows of %s must be contiguous" % name)
    if r <= 1:
        return c or 1
    if ld < c:
        raise ValueError("the rows of %s overlap" % name)
    return ld or 1


# The C entries take counts as int32, and ctypes would cut larger ones off.
_MAX_COUNT = 2 ** 31 - 1


def _counts(what: str, *sizes: int) -> None:
    if max(sizes) > _MAX_COUNT or min(sizes) < -_MAX_COUNT:
        raise ValueError("%s: %s does not fit an int32" % (what, max(sizes, key=abs)))


def _p(t: torch.Tensor | None):
    return None if t is None else t.data_ptr()


# ------------------------------------------------------------- the router --
def _route_desc(experts, topk, score, renorm, scale, groups=1, kept=1):
    if score not in _SCORES:
        raise ValueError("score must be 'softmax' or 'sigmoid'")
    _counts("topk, groups and kept", int(topk), int(groups), int(kept))
    return _capi.cco_route_desc(int(experts), int(topk), _SCORES[score], int(bool(renorm)),
                                float(scale), int(groups), int(kept))


def route(logits: torch.Tensor, topk: int, *, score: str = "softmax", renorm: bool = False,
          scale: float = 1.0, bias: torch.Tensor | None = None, groups: int = 1, kept: int = 1,
          idx: torch.Tensor | None = None, w: torch.Tensor | None = None, stream=None):
    """cco_route -> (idx int32 [T, K], w fp32 [T, K]), the inputs of
    MoE.plan and MoE.dispatch.  logits [T, E] bf16, fp16 or fp32 with
    contiguous rows; bias fp32 [E]."""
    dev = _device(logits, "logits")
    if _away(dev, stream):
        with _Elsewhere(dev, stream):
            return route(logits, topk, score=score, renorm=renorm, scale=scale, bias=bias,
                         groups=groups, kept=kept, idx=idx, w=w)
    ld = _rows(logits, dev, "logits")
    code = _dtype(logits, "logits")
    T, E = logits.shape
    _same(bias, dev, "bias", (E,), torch.float32)
    d = _route_desc(E, topk, score, renorm, scale, groups, kept)
    if idx is None:
        idx = torch.empty((T, max(0, int(topk))), dtype=torch.int32, device=dev)
    else:
        _same(idx, dev, "idx", (T, topk), torch.int32)
    if w is None:
        w = torch.empty((T, max(0, int(topk))), dtype=torch.float32, device=dev)
    else:
        _same(w, dev, "w", (T, topk), torch.float32)
    check(lib.cco_route(ctypes.byref(d), logits.data_ptr(), code, ld, _p(bias), T,
                        idx.data_ptr(), w.data_ptr(), _raw_stream(dev.index)), "cco_route")
    return idx, w


def route_grad(logits: torch.Tensor, idx: torch.Tensor, dw: torch.Tensor, *,
               score: str = "softmax", renorm: bool = False, scale: float = 1.0,
               out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """cco_route_grad -> dlogits [T, E] of the logits' type, given dw fp32
    [T, K], the gradient to the weights of the experts idx int32 [T, K]."""
    dev = _device(logits, "logits")
    if _away(dev, stream):
        with _Elsewhere(dev, stream):
            return route_grad(logits, idx, dw, score=score, renorm=renorm, scale=scale, out=out)
    ld = _rows(logits, dev, "logits")
    code = _dtype(logits, "logits")
    T, E = logits.shape
    if not isinstance(idx, torch.Tensor) or idx.dim() != 2:
        raise ValueError("idx must be [T, K]")
    K = idx.shape[1]
    _same(idx, dev, "idx", (T, K), torch.int32)
    _same(dw, dev, "dw", (T, K), torch.float32)
    d = _route_desc(E, K, score, renorm, scale)
    if out is None:
        out, ldo = torch.empty((T, E), dtype=logits.dtype, device=dev), E
    else:
        ldo = _rows(out, dev, "out", E, T, logits.dtype)
    check(lib.cco_route_grad(ctypes.byref(d), logits.data_ptr(), code, ld, idx.data_ptr(),
                             dw.data_ptr(), T, out.data_ptr(), ldo, _raw_stream(dev.index)),
          "cco_route_grad")
    return out


# ------------------------------------------------------ products by group --
_HALF = (torch.bfloat16, torch.float16)


def _groups(first, count, rows, dev):
    if not isinstance(first, torch.Tensor) or first.dim() != 1:
        raise ValueError("first must be int32 [groups]")
    n = first.shape[0]
    _counts("first", n)
    _same(first, dev, "first", (n,), torch.int32)
    _same(count, dev, "count", (n,), torch.int32)
    return _capi.cco_groups(n, rows, first.data_ptr(), count.data_ptr())


def _workspace(op: int, g, n: int, k: int, dev):
    """(tensor or None, bytes) with which a product splits its reduction."""
    nbytes = lib.cco_group_product_workspace(op, ctypes.byref(g), n, k)
    return (torch.empty(nbytes, dtype=torch.uint8, device=dev) if nbytes else None), nbytes


def group_product(first: torch.Tensor, count: torch.Tensor, x: torch.Tensor, w: torch.Tensor, *,
                  out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """cco_group_product: y [rows, n], y[r] = x[r] w[g]^T for the rows r of
    every group g.  x [rows, k] and w [groups, n, k] bf16 or fp16; rows of no
    group keep what `out` holds (undefined without `out`)."""
    dev = _device(x, "x")
    if _away(dev, stream):
        with _Elsewhere(dev, stream):
            return group_product(first, count, x, w, out=out)
    code = _dtype(x, "x", _HALF)
    ldx = _rows(x, dev, "x")
    rows, k = x.shape
    g = _groups(first, count, rows, dev)
    if not isinstance(w, torch.Tensor) or w.dim() != 3:
        raise ValueError("w must be [groups, n, k]")
    n = w.shape[1]
    _counts("w", n)
    _same(w, dev, "w", (g.groups, n, k), x.dtype)
    if out is None:
        out = torch.empty((rows, n), dtype=x.dtype, device=dev)
    ldy = _rows(out, dev, "out", n, rows, x.dtype)
    ws, nbytes = _workspace(_capi.CCO_GROUP_PRODUCT, g, n, k, dev)
    check(lib.cco_group_product(ctypes.byref(g), code, x.data_ptr(), ldx, w.data_ptr(), n, k,
                                out.data_ptr(), ldy, _p(ws), nbytes, _raw_stream(dev.index)),
          "cco_group_product")
    return out


def group_product_dx(first: torch.Tensor, count: torch.Tensor, dy: torch.Tensor, w: torch.Tensor,
                     *, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """cco_group_product_dx: dx [rows, k], dx[r] = dy[r] w[g] for the rows r
    of every group g."""
    dev = _device(dy, "dy")
    if _away(dev, stream):
        with _Elsewhere(dev, stream):
            return group_product_dx(first, count, dy, w, out=out)
    code = _dtype(dy, "dy", _HALF)
    lddy = _rows(dy, dev, "dy")
    rows, n = dy.shape
    g = _groups(first, count, rows, dev)
    if not isinstance(w, torch.Tensor) or w.dim() != 3:
        raise ValueError("w must be [groups, n, k]")
    k = w.shape[2]
    _counts("w", k)
    _same(w, dev, "w", (g.groups, n, k), dy.dtype)
    if out is None:
        out = torch.empty((rows, k), dtype=dy.dtype, device=dev)
    lddx = _rows(out, dev, "out", k, rows, dy.dtype)
    ws, nbytes = _workspace(_capi.CCO_GROUP_DX, g, n, k, dev)
    check(lib.cco_group_product_dx(ctypes.byref(g), code, dy.data_ptr(), lddy, w.data_ptr(),
                                   n, k, out.data_ptr(), lddx, _p(ws), nbytes,
                                   _raw_stream(dev.index)),
          "cco_group_product_dx")
    return out


def group_product_dw(first: torch.Tensor, count: torch.Tensor, dy: torch.Tensor, x: torch.Tensor,
                     *, out: torch.Tensor | None = None, accumulate: bool = False,
                     stream=None) -> torch.Tensor:
    """cco_group_product_dw: dw [groups, n, k], dw[g] = sum over the rows r of
    group g of dy[r]^T x[r], in the operands' type or, with an fp32 `out`, in
    fp32; with `accumulate` added to what `out` holds."""
    dev = _device(dy, "dy")
    if _away(dev, stream):
        with _Elsewhere(dev, stream):
            return group_product_dw(first, count, dy, x, out=out, accumulate=accumulate)
    code = _dtype(dy, "dy", _HALF)
    lddy = _rows(dy, dev, "dy")
    rows, n = dy.shape
    ldx = _rows(x, dev, "x", None, rows, dy.dtype)
    k = x.shape[1]
    g = _groups(first, count, rows, dev)
    if out is None and accumulate:
        raise ValueError("accumulate needs out")
    if out is None:
        out = torch.empty((g.groups, n, k), dtype=dy.dtype, device=dev)
    _same(out, dev, "out", (g.groups, n, k))
    ws, nbytes = _workspace(_capi.CCO_GROUP_DW, g, n, k, dev)
    check(lib.cco_group_product_dw(ctypes.byref(g), code, dy.data_ptr(), lddy, x.data_ptr(),
                                   ldx, n, k, out.data_ptr(), _dtype(out, "out"),
                                   int(bool(accumulate)), _p(ws), nbytes,
                                   _raw_stream(dev.index)), "cco_group_product_dw")
    return out


# ---------------------------------------------------- norms around a block --
def _norm_desc(x: torch.Tensor, post, gate, token_gate, pre, scale, eps):
    dev, dtype = x.device, x.dtype
    if x.dim() != 2:
        raise ValueError("x must be [T, hidden]")
    T, H = x.shape
    if T > _MAX_COUNT or H > _MAX_COUNT:
        _counts("x", T, H)
    code = _dtype(x, "x")
    wdtype = None
    for name, v in (("post", post), ("pre", pre), ("gate", gate)):
        if v is not None:
            _same(v, dev, name, (H,))
            if wdtype is None:
                wdtype = v.dtype
                if wdtype != torch.float32 and wdtype != dtype:
                    raise ValueError("post, pre and gate must be fp32 or of x's type")
            elif v.dtype != wdtype:
                raise ValueError("post, pre and gate must share one type")
    kind = _capi.CCO_GATE_NONE
    if gate is not None:
        if token_gate is not None:
            raise ValueError("gate and token_gate exclude each other")
        kind = _capi.CCO_GATE_CHANNEL
    elif token_gate is not None:
        _same(token_gate, dev, "token_gate", (T,), torch.float32)
        kind, gate = _capi.CCO_GATE_TOKEN, token_gate
    return _capi.cco_block_norm_desc(H, code, code if wdtype is None else _DTYPES[wdtype], kind,
                                     scale, eps, _p(post), _p(gate), _p(pre))


def block_norm(x: torch.Tensor, y: torch.Tensor | None = None, *,
               post: torch.Tensor | None = None, gate: torch.Tensor | None = None,
               token_gate: torch.Tensor | None = None, pre: torch.Tensor | None = None,
               scale: float = 1.0, eps: float = 1e-6, out: torch.Tensor | None = None,
               u: torch.Tensor | None = None, stream=None):
    """cco_block_norm -> (out, u): out = x + scale gate (post ? rms_norm(y)
    post : y) and, with `pre`, u = rms_norm(out) pre.  Without y: (None, u),
    the norm of x.  x, y [T, hidden] bf16, fp16 or fp32, contiguous; post,
    pre and gate [hidden], fp32 or x's type; token_gate fp32 [T]."""
    dev = _device(x, "x")
    if _away(dev, stream):
        with _Elsewhere(dev, stream):
            return block_norm(x, y, post=post, gate=gate, token_gate=token_gate, pre=pre,
                              scale=scale, eps=eps, out=out, u=u)
    _same(x, dev, "x")
    d = _norm_desc(x, post, gate, token_gate, pre, scale, eps)
    _same(y, dev, "y", x.shape, x.dtype)
    if out is not None:
        _same(out, dev, "out", x.shape, x.dtype)
    elif y is not None:
        out = torch.empty_like(x)
    if u is not None:
        _same(u, dev, "u", x.shape, x.dtype)
    elif pre is not None:
        u = torch.empty_like(x)
    check(lib.cco_block_norm(ctypes.byref(d), x.data_ptr(), _p(y), x.shape[0], _p(out), _p(u),
                             _raw_stream(dev.index)), "cco_block_norm")
    return out, u


def block_norm_grad(x: torch.Tensor, y: torch.Tensor | None, dout: torch.Tensor | None,
                    du: torch.Tensor | None = None, *, post: torch.Tensor | None = None,
                    gate: torch.Tensor | None = None, token_gate: torch.Tensor | None = None,
                    pre: torch.Tensor | None = None, scale: float = 1.0, eps: float = 1e-6,
                    dx: torch.Tensor | None = None, dy: torch.Tensor | None = None, stream=None):
    """cco_block_norm_grad -> (dx, dy, dpost, dgate, dpre), None where there
    is nothing; dgate is the gradient of the gate that is given, and the
    gradients of post, gates and pre are fp32."""
    dev = _device(x, "x")
    if _away(dev, stream):
        with _Elsewhere(dev, stream):
            return block_norm_grad(x, y, dout, du, post=post, gate=gate, token_gate=token_gate,
                                   pre=pre, scale=scale, eps=eps, dx=dx, dy=dy)
    _same(x, dev, "x")
    d = _norm_desc(x, post, gate, token_gate, pre, scale, eps)
    T, H = x.shape
    for name, t in (("y", y), ("dout", dout), ("du", du), ("dx", dx), ("dy", dy)):
        _same(t, dev, name, x.shape, x.dtype)
    f32 = torch.float32
    if dx is None:
        dx = torch.empty_like(x)
    if y is not None and dy is None:
        dy = torch.empty_like(x)
    dpost = torch.empty(H, dtype=f32, device=dev) if post is not None else None
    dpre = torch.empty(H, dtype=f32, device=dev) if pre is not None else None
    dgate = None
    if gate is not None:
        dgate = torch.empty(H, dtype=f32, device=dev)
    elif token_gate is not None:
        dgate = torch.empty(T, dtype=f32, device=dev)
    nbytes = lib.cco_block_norm_grad_workspace(ctypes.byref(d), T)
    ws = torch.empty(nbytes, dtype=torch.uint8, device=dev) if nbytes else None
    check(lib.cco_block_norm_grad(ctypes.byref(d), x.data_ptr(), _p(y), _p(dout), _p(du), T,
                                  dx.data_ptr(), _p(dy), _p(dpost), _p(dgate), _p(dpre),
                                  _p(ws), nbytes, _raw_stream(dev.index)), "cco_block_norm_grad")
    return dx, dy, dpost, dgate, dpre


def combine_norm(moe: MoE, x: torch.Tensor, w: torch.Tensor, *, post: torch.Tensor | None = None,
                 gate: torch.Tensor | None = None, token_gate: torch.Tensor | None = None,
                 pre: torch.Tensor | None = None, scale: float = 1.0, eps: float = 1e-6,
                 out: torch.Tensor | None = None, u: torch.Tensor | None = None,
                 keep_y: bool = False, stream=None):
    """cco_moe_combine_norm -> (out, u, y): MoE.combine of the staging views
    and block_norm of its result in one launch; y, the combined rows, only
    with keep_y (None otherwise).  x bf16 [T, hidden], w fp32 [T, K].  For
    decoding batches; from some hundreds of tokens on the two calls are
    faster."""
    dev = _device(x, "x")
    if _away(dev, stream):
        with _Elsewhere(dev, stream):
            return combine_norm(moe, x, w, post=post, gate=gate, token_gate=token_gate, pre=pre,
                                scale=scale, eps=eps, out=out, u=u, keep_y=keep_y)
    if dev.index != moe.heap.device:
        raise ValueError("x must be on the layer's device")
    _same(x, dev, "x", None, torch.bfloat16)
    d = _norm_desc(x, post, gate, token_gate, pre, scale, eps)
    _same(w, dev, "w", (x.shape[0], moe.K), torch.float32)
    if out is None:
        out = torch.empty_like(x)
    if pre is not None and u is None:
        u = torch.empty_like(x)
    _same(out, dev, "out", x.shape, x.dtype)
    _same(u, dev, "u", x.shape, x.dtype)
    y = torch.empty_like(x) if keep_y else None
    check(lib.cco_moe_combine_norm(moe.handle, w.data_ptr(), ctypes.byref(d), x.data_ptr(),
                                   x.shape[0], _p(y), _p(out), _p(u), _raw_stream(dev.index)),
          "cco_moe_combine_norm")
    return out, u, y
