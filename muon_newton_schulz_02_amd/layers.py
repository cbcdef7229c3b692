"""Python binding of include/ma_layers.h: the operators that a layer's forward
and backward passes are made of, beside those of `grads`.

    ma_rms_norm_forward, ma_rms_norm_backward     norm of a residual stream with the
                          addition that feeds it, the output also held in 8 bits
    ma_rotary             feature pairs turned by positions of several axes, and back
    ma_token_logprob_forward, ma_token_logprob_backward     log probabilities of given
                          tokens, entropies and top alternatives, and the logits' gradient
    ma_attention_forward, ma_attention_backward     attention over packed sequences with
                          grouped heads

Manners are those of `grads`: names and meanings are the C ABI's, outputs and
workspaces are allocated as torch tensors where the caller passes none,
everything is asynchronous on `stream` (a torch.cuda.Stream, a raw hipStream_t
int, or None for torch's current stream of the tensors' device), and no result
carries autograd history: a forward pass returns what its backward pass takes.
"""

from __future__ import annotations

import ctypes as C
from typing import Optional

import torch

from . import _abi
from ._abi import MA_ROTARY_BLOCKS, MA_ROTARY_CYCLED, MA_ROTARY_HALF, MA_ROTARY_PAIRS
from .grads import (ActCheckpoint, _At, _check_cuda, _check_workspace, _dtype, _dtype_code, _elsewhere, _fail, _held,
                    _out_as, _out_like, _raw_stream, _rows, _same_device, _token_bytes, _whole, _workspace)

_LAYOUTS = {"half": MA_ROTARY_HALF, "pairs": MA_ROTARY_PAIRS}
_ORDERS = {"blocks": MA_ROTARY_BLOCKS, "cycled": MA_ROTARY_CYCLED}


def _same_type(x, what: str, like, name: str):
    if x.shape != like.shape or x.dtype != like.dtype:
        raise ValueError("%s %s %s does not belong to %s %s %s" % (
            what, tuple(x.shape), x.dtype, name, tuple(like.shape), like.dtype))


def _vector(x, what: str, n: int):
    _check_cuda(x, what)
    if x.dim() != 1 or x.shape[0] != n or (n > 1 and x.stride(0) != 1):
        raise ValueError("%s must be a contiguous vector of %d (got %s)" % (what, n, tuple(x.shape)))


def _per_row(x, what: str, shape):
    """A contiguous float32 value for each row."""
    _check_cuda(x, what)
    if x.dtype != torch.float32:
        raise TypeError("%s must be float32 (got %s)" % (what, x.dtype))
    if tuple(x.shape) != tuple(shape) or not x.is_contiguous():
        raise ValueError("%s must be contiguous, of shape %s (got %s)" % (what, tuple(shape), tuple(x.shape)))


def _ptr(x):
    return None if x is None else x.data_ptr()


# --------------------------------------------------------------------- norm --

def ma_rms_norm_forward(x, weight, residual=None, eps: float = 1e-6, weight_offset: float = 0.0, out=None,
                        sum_out=None, y_ckpt=None, stream=None):
    """(y, s, inv_rms, y held in 8 bits or None) with s = x + residual, inv_rms = 1 / sqrt(mean(s^2) + eps)
    over the last dimension and y = s * inv_rms * (weight + weight_offset).  Without a
    residual s is x itself.  y_ckpt (True, or an ActCheckpoint to fill) also holds y in 8 bits: the x of
    the following linear layers' ma_linear_grad.  With out=False y is only held (and None is returned for
    it).  s and inv_rms are what ma_rms_norm_backward takes."""
    _check_cuda(x, "x")
    dt = _dtype(x, "x")
    rows, cols, ld = _rows(x, "x")
    _vector(weight, "weight", cols)
    wdt = _dtype(weight, "weight")
    dev = x.device
    rld = sld = 0
    if residual is not None:
        _check_cuda(residual, "residual")
        _same_type(residual, "residual", x, "x")
        rld = _rows(residual, "residual")[2]
    elif sum_out is not None:
        raise ValueError("sum_out needs a residual (without one s is x)")
    hold = y_ckpt is not None and y_ckpt is not False
    if hold and y_ckpt is not True:
        _held(y_ckpt, "y_ckpt", dev, rows, cols)
    if out is False and not hold:
        raise ValueError("out=False needs y_ckpt")
    given = None if out is False else out
    _same_device(dev, ("weight", weight), ("residual", residual), ("out", given), ("sum_out", sum_out))
    if _elsewhere(dev, stream):
        used = [x, weight, residual, given, sum_out]
        if hold and y_ckpt is not True:
            used += y_ckpt._tensors()
        with _At(dev, stream, used):
            return ma_rms_norm_forward(x, weight, residual, eps, weight_offset, out, sum_out, y_ckpt)
    yld = 0
    y = None
    if out is not False:
        y = _out_as(out, "out", x)
        yld = _rows(y, "out")[2]
    s = x
    if residual is not None:
        s = _out_as(sum_out, "sum_out", x)
        sld = _rows(s, "sum_out")[2]
    inv = torch.empty(x.shape[:-1], dtype=torch.float32, device=dev)
    if hold and y_ckpt is True:
        y_ckpt = ActCheckpoint._empty(x.shape, rows, cols, dev)
    rc = _abi.load().ma_rms_norm_forward(
        x.data_ptr(), ld, _ptr(residual), rld, dt, rows, cols, weight.data_ptr(), wdt, weight_offset, eps,
        s.data_ptr() if residual is not None else None, sld, _ptr(y), yld, y_ckpt._pc if hold else None,
        y_ckpt._pe if hold else None, inv.data_ptr(), _raw_stream(dev.index))
    if rc:
        _fail(rc, "ma_rms_norm_forward")
    return y, s, inv, (y_ckpt if hold else None)


def ma_rms_norm_backward_workspace_size(rows: int, cols: int) -> int:
    n = C.c_size_t()
    rc = _abi.load().ma_rms_norm_backward_workspace_size(_whole(rows, "rows"), _whole(cols, "cols"), C.byref(n))
    if rc:
        _fail(rc, "ma_rms_norm_backward_workspace_size")
    return n.value


def ma_rms_norm_backward(dy, s, inv_rms, weight, dsum=None, weight_offset: float = 0.0, ds=None, dweight=None,
                         accumulate: bool = False, grad_dtype=torch.float32, workspace=None, stream=None):
    """(ds, dweight) from the gradient dy of y and the forward pass' s and inv_rms.  dsum is the gradient
    that reaches s past the norm, and is added to ds, which is the gradient of x and of the
    residual alike.  dweight is allocated in `grad_dtype` where none is passed; with accumulate the sum is
    added to it; dweight=False leaves it out (and returns None for it)."""
    _check_cuda(dy, "dy")
    _check_cuda(s, "s")
    _same_type(s, "s", dy, "dy")
    dt = _dtype(dy, "dy")
    rows, cols, ld = _rows(dy, "dy")
    sld = _rows(s, "s")[2]
    _vector(weight, "weight", cols)
    wdt = _dtype(weight, "weight")
    _per_row(inv_rms, "inv_rms", dy.shape[:-1])
    rld = 0
    if dsum is not None:
        _check_cuda(dsum, "dsum")
        _same_type(dsum, "dsum", dy, "dy")
        rld = _rows(dsum, "dsum")[2]
    dev = dy.device
    if accumulate and (dweight is None or dweight is False):
        raise ValueError("accumulate needs the gradient to add to (dweight)")
    given = None if dweight is False else dweight
    _same_device(dev, ("s", s), ("inv_rms", inv_rms), ("weight", weight), ("dsum", dsum), ("ds", ds),
                 ("dweight", given))
    _check_workspace(workspace, dev)
    if _elsewhere(dev, stream):
        with _At(dev, stream, (dy, s, inv_rms, weight, dsum, ds, given, workspace)):
            return ma_rms_norm_backward(dy, s, inv_rms, weight, dsum, weight_offset, ds, dweight, accumulate,
                                        grad_dtype, workspace)
    ds = _out_as(ds, "ds", dy)
    ws_ptr, ws_bytes, gdt = None, 0, 0
    dw = None
    if dweight is not False:
        dw = _out_like(dweight, "dweight", (cols,), grad_dtype, dev)
        if not dw.is_contiguous():
            raise ValueError("dweight must be contiguous")
        gdt = _dtype(dw, "dweight")
        ws, ws_ptr, ws_bytes = _workspace(workspace, ma_rms_norm_backward_workspace_size(rows, cols), dev)
    rc = _abi.load().ma_rms_norm_backward(
        dy.data_ptr(), ld, s.data_ptr(), sld, _ptr(dsum), rld, dt, rows, cols, inv_rms.data_ptr(),
        weight.data_ptr(), wdt, weight_offset, ds.data_ptr(), _rows(ds, "ds")[2], _ptr(dw), gdt,
        1 if accumulate else 0, ws_ptr, ws_bytes, _raw_stream(dev.index))
    if rc:
        _fail(rc, "ma_rms_norm_backward")
    return ds, dw


# ------------------------------------------------------------------- rotary --

def _heads(x, what: str):
    """(tokens, heads, features, token stride, head stride) of (..., heads, features)."""
    if x.dim() < 2:
        raise ValueError("%s must be (..., heads, features)" % what)
    heads, dim = x.shape[-2:]
    if dim > 1 and x.stride(-1) != 1 and x.numel():
        raise ValueError("the last dimension of %s must be contiguous" % what)
    tokens, stride, run = 1, heads * dim, None
    for d, st in zip(reversed(x.shape[:-2]), reversed(x.stride()[:-2])):
        tokens *= d
        if d == 1:
            continue
        if run is None:
            stride = st
        elif st != run:
            raise ValueError("the tokens of %s are not evenly spaced" % what)
        run = d * st
    return tokens, heads, dim, stride, (x.stride(-2) if heads > 1 else dim)


class Rotary:
    """How heads turn with positions: `sections` feature pairs for each axis (one number: a single axis),
    of which pair i of all turns at theta^(-i / pairs) radians per position, or with `restart` the j-th
    pair of an axis with n at theta^(-j / n).  `order` is 'blocks' (the axes' pairs one axis after the
    other) or 'cycled' (the axes in turn, without those that are used up), `layout` 'half' (pair i is
    features i and pairs + i) or 'pairs' (features 2 i and 2 i + 1)."""

    __slots__ = ("sections", "pairs", "axes", "theta", "layout", "order", "restart", "_freq", "_axis", "_layout")

    def __init__(self, sections, theta: float = 10000.0, layout: str = "half", order: str = "blocks",
                 restart: bool = False):
        sections = tuple(_whole(n, "a section", 32) for n in ((sections,) if isinstance(sections, int) else sections))
        if layout not in _LAYOUTS:
            raise ValueError("layout must be one of %s" % ", ".join(sorted(_LAYOUTS)))
        if order not in _ORDERS:
            raise ValueError("order must be one of %s" % ", ".join(sorted(_ORDERS)))
        self.sections, self.axes, self.pairs = sections, len(sections), sum(sections)
        self.theta, self.layout, self.order, self.restart = float(theta), layout, order, bool(restart)
        n = min(max(1, self.pairs), _abi.MA_ROTARY_MAX_PAIRS)          # (more are refused)
        self._freq, self._axis, self._layout = (C.c_double * n)(), (C.c_uint8 * n)(), _LAYOUTS[layout]
        rc = _abi.load().ma_rotary_frequencies((C.c_int32 * max(1, self.axes))(*sections), self.axes, self.theta,
                                               _ORDERS[order], int(self.restart), self._freq, self._axis)
        if rc:
            _fail(rc, "Rotary")

    def __reduce__(self):
        return Rotary, (self.sections, self.theta, self.layout, self.order, self.restart)

    @property
    def frequencies(self):
        """Radians per position of each pair."""
        return tuple(self._freq)

    @property
    def pair_axis(self):
        """The axis of each pair."""
        return tuple(self._axis)


def ma_rotary(x, positions, rotary: Rotary, inverse: bool = False, out=None, stream=None):
    """x (..., heads, features) with every head's pairs turned by their token's positions: int32 or int64,
    of shape (axes, ...) or, for a single axis, (...).  Features past the pairs are copied.  With inverse
    they turn back: the gradient of x from the gradient of the result.  `out` may be x itself."""
    _check_cuda(x, "x")
    _check_cuda(positions, "positions")
    if not isinstance(rotary, Rotary):
        raise TypeError("rotary must be a Rotary")
    dt = _dtype(x, "x")
    tokens, heads, dim, tok, head = _heads(x, "x")
    if positions.dtype not in (torch.int64, torch.int32):
        raise TypeError("positions must be int32 or int64 (got %s)" % positions.dtype)
    lead = tuple(x.shape[:-2])
    shape = tuple(positions.shape)
    if shape != (rotary.axes, *lead) and not (rotary.axes == 1 and shape == lead):
        raise ValueError("positions %s do not belong to x %s and %d axes" % (shape, tuple(x.shape), rotary.axes))
    axis = 0
    if shape == (rotary.axes, *lead):
        axis = positions.stride(0) if rotary.axes > 1 else 0
        if not positions[0].is_contiguous():
            raise ValueError("the positions of an axis must be contiguous")
    elif not positions.is_contiguous():
        raise ValueError("positions must be contiguous")
    dev = x.device
    _same_device(dev, ("positions", positions), ("out", out))
    if _elsewhere(dev, stream):
        with _At(dev, stream, (x, positions, out)):
            return ma_rotary(x, positions, rotary, inverse, out)
    out = _out_as(out, "out", x)
    _, _, _, otok, ohead = _heads(out, "out")
    rc = _abi.load().ma_rotary(x.data_ptr(), dt, tokens, heads, dim, tok, head, positions.data_ptr(),
                               positions.element_size(), rotary.axes, axis, rotary._freq, rotary._axis,
                               rotary.pairs, rotary._layout, 1 if inverse else 0, out.data_ptr(), otok, ohead,
                               _raw_stream(dev.index))
    if rc:
        _fail(rc, "ma_rotary")
    return out


# -------------------------------------------------- log probabilities of tokens --

def _tokens_of(tokens, what: str, shape):
    _check_cuda(tokens, what)
    if tuple(tokens.shape) != tuple(shape):
        raise ValueError("%s %s do not belong to rows %s" % (what, tuple(tokens.shape), tuple(shape)))
    if not tokens.is_contiguous():
        raise ValueError("%s must be contiguous" % what)
    return _token_bytes(tokens)


def ma_token_logprob_workspace_size(n_tokens: int, vocab: int, top: int = 0) -> int:
    n = C.c_size_t()
    rc = _abi.load().ma_token_logprob_workspace_size(_whole(n_tokens, "n_tokens"), _whole(vocab, "vocab"),
                                                     _whole(top, "top", 32), C.byref(n))
    if rc:
        _fail(rc, "ma_token_logprob_workspace_size")
    return n.value


def ma_token_logprob_forward(logits, tokens, scale: float = 1.0, top: int = 0, workspace=None, stream=None):
    """(logprob, entropy, lse, top_ids, top_logprobs) of softmax(scale * logits) over the last dimension, in
    float32: the log probability of each row's token (0 for one outside [0, vocab)), the entropy, the log of the
    sum that the backward pass takes, and the ids (in the tokens' type) and log probabilities of the `top`
    highest, ties to the lowest id (None for top = 0)."""
    _check_cuda(logits, "logits")
    dt = _dtype(logits, "logits")
    rows, vocab, ld = _rows(logits, "logits")
    shape = logits.shape[:-1]
    tb = _tokens_of(tokens, "tokens", shape)
    dev = logits.device
    _same_device(dev, ("tokens", tokens))
    _check_workspace(workspace, dev)
    if _elsewhere(dev, stream):
        with _At(dev, stream, (logits, tokens, workspace)):
            return ma_token_logprob_forward(logits, tokens, scale, top, workspace)
    top = int(top)
    need = ma_token_logprob_workspace_size(rows, vocab, top)
    logprob = torch.empty(shape, dtype=torch.float32, device=dev)
    entropy, lse = torch.empty_like(logprob), torch.empty_like(logprob)
    ids = best = None
    if top > 0:
        ids = torch.empty((*shape, top), dtype=tokens.dtype, device=dev)
        best = torch.empty((*shape, top), dtype=torch.float32, device=dev)
    ws, ws_ptr, ws_bytes = _workspace(workspace, need, dev)
    rc = _abi.load().ma_token_logprob_forward(
        logits.data_ptr(), dt, rows, vocab, ld, tokens.data_ptr(), tb, scale, logprob.data_ptr(),
        entropy.data_ptr(), lse.data_ptr(), top, _ptr(ids), _ptr(best), ws_ptr, ws_bytes, _raw_stream(dev.index))
    if rc:
        _fail(rc, "ma_token_logprob_forward")
    return logprob, entropy, lse, ids, best


def ma_token_logprob_backward(logits, tokens, lse, dlogprob, entropy=None, dentropy=None, scale: float = 1.0,
                              out=None, grad_dtype=None, stream=None):
    """The gradient of the logits from those of the log probabilities and (with the forward pass' entropy)
    of the entropies.  It is allocated in `grad_dtype` (default: the logits') where no `out` is passed;
    `out` may be the logits themselves."""
    _check_cuda(logits, "logits")
    dt = _dtype(logits, "logits")
    rows, vocab, ld = _rows(logits, "logits")
    shape = logits.shape[:-1]
    tb = _tokens_of(tokens, "tokens", shape)
    _per_row(lse, "lse", shape)
    _per_row(dlogprob, "dlogprob", shape)
    if (entropy is None) != (dentropy is None):
        raise ValueError("entropy and dentropy go together")
    if dentropy is not None:
        _per_row(entropy, "entropy", shape)
        _per_row(dentropy, "dentropy", shape)
    dev = logits.device
    _same_device(dev, ("tokens", tokens), ("lse", lse), ("dlogprob", dlogprob), ("entropy", entropy),
                 ("dentropy", dentropy), ("out", out))
    if _elsewhere(dev, stream):
        with _At(dev, stream, (logits, tokens, lse, dlogprob, entropy, dentropy, out)):
            return ma_token_logprob_backward(logits, tokens, lse, dlogprob, entropy, dentropy, scale, out, grad_dtype)
    out = _out_like(out, "out", logits.shape, grad_dtype or logits.dtype, dev)
    rc = _abi.load().ma_token_logprob_backward(
        logits.data_ptr(), dt, rows, vocab, ld, tokens.data_ptr(), tb, scale, lse.data_ptr(), _ptr(entropy),
        dlogprob.data_ptr(), _ptr(dentropy), out.data_ptr(), _dtype(out, "out"), _rows(out, "out")[2],
        _raw_stream(dev.index))
    if rc:
        _fail(rc, "ma_token_logprob_backward")
    return out


# ---------------------------------------------------------------- attention --

def _offsets(cu, what: str):
    _check_cuda(cu, what)
    if cu.dtype != torch.int32 or cu.dim() != 1 or not 1 <= cu.shape[0] <= 1 << 31 or not cu.is_contiguous():
        raise ValueError("%s must be a contiguous int32 vector of at most 2^31 offsets" % what)
    return cu.shape[0] - 1


def _attention_args(q, k, v, cu_q, cu_k, causal, scale):
    """(args, device) of the inputs that both passes share."""
    for what, x in (("q", q), ("k", k), ("v", v)):
        _check_cuda(x, what)
        if x.dim() != 3:
            raise ValueError("%s must be tokens x heads x features (got %s)" % (what, tuple(x.shape)))
    if k.shape != v.shape or k.dtype != q.dtype or v.dtype != q.dtype or k.shape[2] != q.shape[2]:
        raise ValueError("q %s %s, k %s %s and v %s %s do not belong together" % (
            tuple(q.shape), q.dtype, tuple(k.shape), k.dtype, tuple(v.shape), v.dtype))
    if (cu_q is None) != (cu_k is None):
        raise ValueError("cu_q and cu_k go together")
    if max(*q.shape[1:], k.shape[1]) >= 1 << 31 or q.shape[2] == 0:
        raise ValueError("q %s and k %s: heads without features, or more than 2^31" % (tuple(q.shape), tuple(k.shape)))
    a = _abi.ma_attention()
    a.dtype = _dtype(q, "q")
    a.n_queries, a.heads, a.head_dim = q.shape
    a.n_keys, a.kv_heads = k.shape[:2]
    a.causal = 1 if causal else 0
    a.scale = a.head_dim ** -0.5 if scale is None else scale
    a.n_seqs = 1
    if cu_q is not None:
        a.n_seqs = _offsets(cu_q, "cu_q")
        if _offsets(cu_k, "cu_k") != a.n_seqs:
            raise ValueError("cu_q and cu_k hold %d and %d offsets" % (cu_q.shape[0], cu_k.shape[0]))
        a.cu_q, a.cu_k = cu_q.data_ptr(), cu_k.data_ptr()
    _same_device(q.device, ("k", k), ("v", v), ("cu_q", cu_q), ("cu_k", cu_k))
    for name, x in (("q", q), ("k", k), ("v", v)):
        _set_heads(getattr(a, name), x, name)
    return a, q.device


def _set_heads(field, x, what: str):
    _, _, _, field.token_stride, field.head_stride = _heads(x, what)
    field.p = x.data_ptr()


def ma_attention_forward(q, k, v, cu_q=None, cu_k=None, causal: bool = True, scale: Optional[float] = None, out=None,
                         workspace=None, stream=None):
    """(o, lse) of softmax(scale q k^T) v: q (queries, heads, features), k and v (keys, key heads, features), where
    query head h reads key head h // (heads // key heads).  cu_q and cu_k (int32, one more than there are
    sequences) hold where packed sequences begin; without them everything is one sequence.  With `causal` the last
    query of a sequence sees its last key.  scale defaults to features^-1/2.  A query that sees no key
    has o = 0 and lse = -infinity; queries outside every sequence are left as they are in `out` (and undefined where
    none is passed).  o and lse (heads x queries, float32) are what ma_attention_backward takes."""
    a, dev = _attention_args(q, k, v, cu_q, cu_k, causal, scale)
    _same_device(dev, ("out", out))
    _check_workspace(workspace, dev)
    if _elsewhere(dev, stream):
        with _At(dev, stream, (q, k, v, cu_q, cu_k, out, workspace)):
            return ma_attention_forward(q, k, v, cu_q, cu_k, causal, scale, out, workspace)
    out = _out_as(out, "out", q)
    lse = torch.empty((a.heads, a.n_queries), dtype=torch.float32, device=dev)
    _set_heads(a.o, out, "out")
    a.lse = lse.data_ptr()
    lib = _abi.load()
    ws, ws_ptr, ws_bytes = _workspace(workspace, _space(lib.ma_attention_forward_workspace_size, a), dev)
    rc = lib.ma_attention_forward(C.byref(a), ws_ptr, ws_bytes, _raw_stream(dev.index))
    if rc:
        _fail(rc, "ma_attention_forward")
    return out, lse


def _space(size_of, a) -> int:
    n = C.c_size_t()
    rc = size_of(C.byref(a), C.byref(n))
    if rc:
        _fail(rc, size_of.__name__)
    return n.value


def _sizes_args(n_queries, n_keys, heads, kv_heads, head_dim, n_seqs, causal, dtype):
    """Arguments of contiguous, aligned arrays of these sizes."""
    a = _abi.ma_attention()
    a.causal = 1 if causal else 0
    heads, kv_heads, head_dim = _whole(heads, "heads", 32), _whole(kv_heads, "kv_heads", 32), _whole(head_dim, "head_dim", 32)
    a.dtype, a.heads, a.kv_heads, a.head_dim = _dtype_code(dtype, "q"), heads, kv_heads, head_dim
    a.n_queries, a.n_keys = _whole(n_queries, "n_queries"), _whole(n_keys, "n_keys")
    a.n_seqs, a.scale = _whole(n_seqs, "n_seqs", 32), 1.0
    a.cu_q = a.cu_k = 256          # (only looked at for being there)
    for field, n in ((a.q, heads), (a.k, kv_heads), (a.v, kv_heads), (a.o, heads), (a.dout, heads), (a.dq, heads),
                     (a.dk, kv_heads), (a.dv, kv_heads)):
        field.token_stride, field.head_stride = n * head_dim, head_dim
    return a


def ma_attention_forward_workspace_size(n_queries: int, n_keys: int, heads: int, kv_heads: int, head_dim: int,
                                        n_seqs: int = 1, causal: bool = True, dtype=torch.bfloat16) -> int:
    """Bytes that serve contiguous, 16-byte aligned arrays of these sizes (a call without a workspace
    allocates what its own arrays need)."""
    a = _sizes_args(n_queries, n_keys, heads, kv_heads, head_dim, n_seqs, causal, dtype)
    return _space(_abi.load().ma_attention_forward_workspace_size, a)


def ma_attention_backward_workspace_size(n_queries: int, n_keys: int, heads: int, kv_heads: int, head_dim: int,
                                         n_seqs: int = 1, causal: bool = True, dtype=torch.bfloat16) -> int:
    """Bytes that serve contiguous, 16-byte aligned arrays of these sizes (a call without a workspace
    allocates what its own arrays need)."""
    a = _sizes_args(n_queries, n_keys, heads, kv_heads, head_dim, n_seqs, causal, dtype)
    return _space(_abi.load().ma_attention_backward_workspace_size, a)


def ma_attention_backward(dout, q, k, v, out, lse, cu_q=None, cu_k=None, causal: bool = True,
                          scale: Optional[float] = None, dq=None, dk=None, dv=None, workspace=None, stream=None):
    """(dq, dk, dv) from the gradient dout of ma_attention_forward's output `out`, with its lse and the same
    other arguments.  Rows outside every sequence are left as they are (and undefined in gradients allocated
    here)."""
    a, dev = _attention_args(q, k, v, cu_q, cu_k, causal, scale)
    _check_cuda(dout, "dout")
    _check_cuda(out, "out")
    _same_type(dout, "dout", q, "q")
    _same_type(out, "out", q, "q")
    _per_row(lse, "lse", (a.heads, a.n_queries))
    _same_device(dev, ("dout", dout), ("out", out), ("lse", lse), ("dq", dq), ("dk", dk), ("dv", dv))
    _check_workspace(workspace, dev)
    if _elsewhere(dev, stream):
        with _At(dev, stream, (dout, q, k, v, out, lse, cu_q, cu_k, dq, dk, dv, workspace)):
            return ma_attention_backward(dout, q, k, v, out, lse, cu_q, cu_k, causal, scale, dq, dk, dv, workspace)
    dq, dk, dv = _out_as(dq, "dq", q), _out_as(dk, "dk", k), _out_as(dv, "dv", v)
    for name, x in (("o", out), ("dout", dout), ("dq", dq), ("dk", dk), ("dv", dv)):
        _set_heads(getattr(a, name), x, name)
    a.lse = lse.data_ptr()
    lib = _abi.load()
    ws, ws_ptr, ws_bytes = _workspace(workspace, _space(lib.ma_attention_backward_workspace_size, a), dev)
    rc = lib.ma_attention_backward(C.byref(a), ws_ptr, ws_bytes, _raw_stream(dev.index))
    if rc:
        _fail(rc, "ma_attention_backward")
    return dq, dk, dv
