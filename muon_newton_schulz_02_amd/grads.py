"""Python binding of include/ma_grads.h: the operators that produce the
gradients an optimizer step reads, and the 8-bit form in which activations
are kept between forward and backward.

    ma_embedding_lookup   out[t] = scale * table[tokens[t]]
    ma_embedding_grad     dtable[v] (+)= scale * sum of dout[t] over tokens[t] = v
    ma_act_pack, ma_act_unpack     an activation held in 8 bits, and read back
    ma_linear_grad        dW (+)= dY^T X from an X held in 8 bits
    ma_glu_forward, ma_glu_backward     h = act(gate) * up with gate and up
                          held in 8 bits, and its backward pass from them

Names and meanings are the C ABI's; this module marshals arguments, and
allocates outputs and workspaces as torch tensors where the caller passes
none.  Everything is asynchronous on `stream` (a torch.cuda.Stream, a raw
hipStream_t int, or None for torch's current stream of the tensors' device).
Tensors passed in belong to the caller and are not tracked by autograd.

Activations and gradients may have any number of leading dimensions; they
are matrices of (product of the leading dimensions) x (last dimension), whose
last dimension is contiguous and whose rows are evenly spaced.

`EmbeddingGrad` and `LinearGrad` describe a gradient that has not been formed
yet; MuonAdamW.step takes them in place of gradient tensors.
"""

from __future__ import annotations

import contextlib
import ctypes as C
from typing import NamedTuple, Optional

import torch

from . import _abi
from ._abi import MA_ACT_GELU_TANH, MA_ACT_GROUP, MA_ACT_SILU, MA_PARAM_BF16, MA_PARAM_FP32

_DTYPES = {torch.float32: MA_PARAM_FP32, torch.bfloat16: MA_PARAM_BF16}
_ACTS = {"silu": MA_ACT_SILU, "gelu_tanh": MA_ACT_GELU_TANH}


def _fail(rc: int, what: str):
    from . import MuonAdamWError
    raise MuonAdamWError(rc, "%s: %s" % (
        what, _abi.load().muon_adamw_last_error().decode("utf-8", "replace")))


# ------------------------------------------------------------- arguments --

def _dtype(x, what: str) -> int:
    try:
        return _DTYPES[x.dtype]
    except KeyError:
        raise TypeError("%s must be float32 or bfloat16 (got %s)" % (what, x.dtype)) from None


def _rows(x, what: str):
    """(rows, columns, row stride) of a tensor read as a matrix."""
    dim = x.dim()
    if dim == 2:
        rows, cols = x.shape
        stride, inner = x.stride()
    elif dim == 0:
        raise ValueError("%s must have at least one dimension" % what)
    else:
        rows, cols = 1, x.shape[-1]
        for d in x.shape[:-1]:
            rows *= d
        inner = x.stride(-1)
        stride = cols
        if rows > 1:
            # the leading dimensions have to fold into one evenly spaced axis
            run = None
            for d, s in zip(reversed(x.shape[:-1]), reversed(x.stride()[:-1])):
                if d == 1:
                    continue
                if run is None:
                    stride = s
                elif s != run:
                    raise ValueError("the rows of %s are not evenly spaced" % what)
                run = d * s
    if inner != 1 and cols > 1 and rows > 0:
        raise ValueError("the last dimension of %s must be contiguous" % what)
    return rows, cols, (stride if rows > 1 else cols)


def _check_cuda(x, what: str):
    if not isinstance(x, torch.Tensor):
        raise TypeError("%s must be a torch tensor" % what)
    if not x.is_cuda:
        raise ValueError("%s must live on the GPU" % what)


def _same_device(dev, *named):
    for what, x in named:
        if x is not None and x.device != dev:
            raise ValueError("%s is on %s, the call runs on %s" % (what, x.device, dev))


def _token_bytes(tokens) -> int:
    if tokens.dtype == torch.int64:
        return 8
    if tokens.dtype == torch.int32:
        return 4
    raise TypeError("tokens must be int32 or int64 (got %s)" % tokens.dtype)


# (the same numbers as torch.cuda.current_device() and current_stream(), without
# building the objects around them: a quarter of a small call's host time)
_device_now = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


class _Here:
    """The current stream of the current device, already right."""

    __slots__ = ("raw",)

    def __init__(self, raw):
        self.raw = raw

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        return False


class _Elsewhere(contextlib.ExitStack):
    """Another device or stream, made current for a call's allocations and
    launches."""

    def __init__(self, dev, stream, tensors):
        super().__init__()
        self.enter_context(torch.cuda.device(dev))
        if stream is None:
            self.raw = _raw_stream(dev.index)
            return
        if isinstance(stream, int):
            stream = torch.cuda.ExternalStream(stream, device=dev)
        self.raw = stream.cuda_stream
        if self.raw != _raw_stream(dev.index):
            # memory of another stream's tensors is not handed out again before this
            # stream is done with them
            for t in tensors:
                if t is not None:
                    t.record_stream(stream)
            self.enter_context(torch.cuda.stream(stream))


def _on(dev, stream, tensors):
    """The context a call allocates and launches in; `.raw` is its stream."""
    if stream is None and dev.index == _device_now():
        return _Here(_raw_stream(dev.index))
    return _Elsewhere(dev, stream, tensors)


def _out_like(out, what: str, shape, dtype, dev):
    if out is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    _check_cuda(out, what)
    if tuple(out.shape) != tuple(shape):
        raise ValueError("%s has shape %s, the call gives %s" % (what, tuple(out.shape),
                                                                 tuple(shape)))
    return out


def _out_as(out, what: str, x):
    """An output of x's shape and type."""
    if out is None:
        return torch.empty_like(x, memory_format=torch.contiguous_format)
    if out.dtype != x.dtype:
        raise TypeError("%s must be %s" % (what, x.dtype))
    return _out_like(out, what, x.shape, x.dtype, x.device)


def _workspace(workspace, need: int, dev):
    """(tensor, address, bytes) of a call's workspace."""
    if workspace is None:
        if need == 0:
            return None, None, 0
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
        return workspace, workspace.data_ptr(), need
    _check_cuda(workspace, "workspace")
    _same_device(dev, ("workspace", workspace))
    if not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


# ------------------------------------------------- activations in 8 bits --

class ActCheckpoint:
    """An activation held in 8 bits: `codes` (int8, rows x code pitch), `exps`
    (uint8, rows x exponent pitch) and its number of features `cols`; `shape` is
    the activation's (default: rows x cols).  It stands for codes * 2^(exps -
    127), one exponent for every 32 features of a token."""

    __slots__ = ("codes", "exps", "cols", "shape")

    def __init__(self, codes, exps, cols: int, shape=None):
        cols = int(cols)
        pitch = -(-cols // MA_ACT_GROUP) * MA_ACT_GROUP
        if cols < 1 or codes.dtype != torch.int8 or exps.dtype != torch.uint8:
            raise TypeError("codes must be int8, exps uint8 and cols at least 1")
        if codes.dim() != 2 or exps.dim() != 2 or codes.shape[1] != pitch or \
                exps.shape[1] != -(-pitch // (4 * MA_ACT_GROUP)) * 4 or \
                exps.shape[0] != codes.shape[0]:
            raise ValueError("codes %s and exps %s do not hold %d features" % (
                tuple(codes.shape), tuple(exps.shape), cols))
        if not codes.is_contiguous() or not exps.is_contiguous():
            raise ValueError("codes and exps must be contiguous")
        self.codes, self.exps, self.cols = codes, exps, cols
        if shape is None:
            shape = (codes.shape[0], cols)
        self.shape = tuple(shape)
        if self.shape[-1] != cols or self.numel() != codes.shape[0] * cols:
            raise ValueError("shape %s is not %d rows of %d features" % (self.shape,
                                                                         codes.shape[0], cols))

    def numel(self) -> int:
        n = 1
        for d in self.shape:
            n *= int(d)
        return n

    @property
    def rows(self) -> int:
        return self.codes.shape[0]

    @staticmethod
    def empty(shape, device) -> "ActCheckpoint":
        """An uninitialised holder for an activation of this shape."""
        shape = tuple(int(d) for d in shape)
        cols, rows = shape[-1], 1
        for d in shape[:-1]:
            rows *= d
        return ActCheckpoint._empty(shape, rows, cols, device)

    @staticmethod
    def _empty(shape, rows, cols, device):
        if cols < 1:
            raise ValueError("an activation needs at least one feature")
        pitch = -(-cols // MA_ACT_GROUP) * MA_ACT_GROUP
        c = object.__new__(ActCheckpoint)
        c.codes = torch.empty((rows, pitch), dtype=torch.int8, device=device)
        c.exps = torch.empty((rows, -(-pitch // (4 * MA_ACT_GROUP)) * 4), dtype=torch.uint8,
                             device=device)
        c.cols, c.shape = cols, tuple(shape)
        return c

    def _like(self):
        c = object.__new__(ActCheckpoint)
        c.codes, c.exps = torch.empty_like(self.codes), torch.empty_like(self.exps)
        c.cols, c.shape = self.cols, self.shape
        return c


def _held(c, what: str, rows=None, cols=None):
    if not isinstance(c, ActCheckpoint):
        raise TypeError("%s must be an ActCheckpoint" % what)
    if rows is not None and (c.rows != rows or c.cols != cols):
        raise ValueError("%s holds %d x %d, the call needs %d x %d" % (what, c.rows, c.cols, rows,
                                                                      cols))
    if not c.codes.is_cuda or not c.exps.is_cuda:
        raise ValueError("%s must live on the GPU" % what)
    return c


def ma_act_pack(x, out: Optional[ActCheckpoint] = None, stream=None) -> ActCheckpoint:
    """x (..., features) held in 8 bits."""
    _check_cuda(x, "x")
    dt = _dtype(x, "x")
    rows, cols, ld = _rows(x, "x")
    dev = x.device
    if out is not None:
        _held(out, "out", rows, cols)
        _same_device(dev, ("out", out.codes), ("out", out.exps))
    with _on(dev, stream, (x,) if out is None else (x, out.codes, out.exps)) as on:
        if out is None:
            out = ActCheckpoint._empty(x.shape, rows, cols, dev)
        rc = _abi.load().ma_act_pack(x.data_ptr(), dt, rows, cols, ld, out.codes.data_ptr(),
                                     out.exps.data_ptr(), on.raw)
    if rc:
        _fail(rc, "ma_act_pack")
    return out


def ma_act_unpack(ckpt: ActCheckpoint, dtype=torch.float32, out=None, stream=None):
    """The activation an ActCheckpoint stands for, in `dtype` (or out's)."""
    _held(ckpt, "ckpt")
    dev = ckpt.codes.device
    _same_device(dev, ("exps", ckpt.exps), ("out", out))
    with _on(dev, stream, (ckpt.codes, ckpt.exps, out)) as on:
        out = _out_like(out, "out", ckpt.shape, dtype, dev)
        rows, cols, ld = _rows(out, "out")
        rc = _abi.load().ma_act_unpack(ckpt.codes.data_ptr(), ckpt.exps.data_ptr(), rows, cols,
                                       out.data_ptr(), _dtype(out, "out"), ld, on.raw)
    if rc:
        _fail(rc, "ma_act_unpack")
    return out


# -------------------------------------------------------- embedding table --

def ma_embedding_lookup(table, tokens, scale: float = 1.0, out=None, out_dtype=None, stream=None):
    """scale * table[tokens], of shape tokens.shape + (hidden,), in `out_dtype`
    (default: the table's).  A token outside [0, vocab) gives a row of zeros."""
    _check_cuda(table, "table")
    _check_cuda(tokens, "tokens")
    if table.dim() != 2:
        raise ValueError("table must be vocab x hidden")
    vocab, hidden, ld = _rows(table, "table")
    tb = _token_bytes(tokens)
    if not tokens.is_contiguous():
        raise ValueError("tokens must be contiguous")
    dt = _dtype(table, "table")
    dev = table.device
    _same_device(dev, ("tokens", tokens), ("out", out))
    with _on(dev, stream, (table, tokens, out)) as on:
        out = _out_like(out, "out", tuple(tokens.shape) + (hidden,), out_dtype or table.dtype, dev)
        rows, _, old = _rows(out, "out")
        rc = _abi.load().ma_embedding_lookup(table.data_ptr(), dt, vocab, hidden, ld,
                                             tokens.data_ptr(), tb, rows, scale, out.data_ptr(),
                                             _dtype(out, "out"), old, on.raw)
    if rc:
        _fail(rc, "ma_embedding_lookup")
    return out


def ma_embedding_grad_workspace_size(n_tokens: int, vocab: int, hidden: int) -> int:
    lib = _abi.load()
    n = C.c_size_t()
    rc = lib.ma_embedding_grad_workspace_size(n_tokens, vocab, hidden, C.byref(n))
    if rc:
        _fail(rc, "ma_embedding_grad_workspace_size")
    return n.value


def ma_embedding_grad(dout, tokens, vocab: int, scale: float = 1.0, padding_token: int = -1,
                      out=None, accumulate: bool = False, grad_dtype=torch.float32,
                      workspace=None, stream=None):
    """The vocab x hidden gradient of ma_embedding_lookup's table from the
    gradient `dout` of its output: row v is scale * the sum of dout over the
    tokens equal to v (zero for none).  Tokens outside [0, vocab) or equal to
    padding_token add to no row.  With accumulate the sums are added to `out`.
    Where no `out` is passed the gradient is allocated in `grad_dtype`."""
    _check_cuda(dout, "dout")
    _check_cuda(tokens, "tokens")
    dt = _dtype(dout, "dout")
    rows, hidden, ld = _rows(dout, "dout")
    tb = _token_bytes(tokens)
    if not tokens.is_contiguous():
        raise ValueError("tokens must be contiguous")
    if tokens.shape != dout.shape[:-1]:
        raise ValueError("dout %s does not belong to tokens %s" % (tuple(dout.shape),
                                                                   tuple(tokens.shape)))
    if accumulate and out is None:
        raise ValueError("accumulate needs the gradient to add to (out)")
    dev = dout.device
    _same_device(dev, ("tokens", tokens), ("out", out))
    vocab = int(vocab)
    need = ma_embedding_grad_workspace_size(rows, vocab, hidden)
    with _on(dev, stream, (dout, tokens, out, workspace)) as on:
        out = _out_like(out, "out", (vocab, hidden), grad_dtype, dev)
        if not out.is_contiguous():
            raise ValueError("out must be contiguous")
        ws, ws_ptr, ws_bytes = _workspace(workspace, need, dev)
        rc = _abi.load().ma_embedding_grad(dout.data_ptr(), dt, ld, tokens.data_ptr(), tb, rows,
                                           vocab, hidden, scale, int(padding_token),
                                           out.data_ptr(), _dtype(out, "out"),
                                           1 if accumulate else 0, ws_ptr, ws_bytes, on.raw)
    if rc:
        _fail(rc, "ma_embedding_grad")
    return out


# ------------------------------------------------------------ linear layer --

def ma_linear_grad_workspace_size(n_tokens: int, n_out: int, n_in: int,
                                  dy_dtype=torch.bfloat16) -> int:
    n = C.c_size_t()
    rc = _abi.load().ma_linear_grad_workspace_size(n_tokens, n_out, n_in, _DTYPES[dy_dtype],
                                                   C.byref(n))
    if rc:
        _fail(rc, "ma_linear_grad_workspace_size")
    return n.value


def ma_linear_grad(dy, x: ActCheckpoint, out=None, accumulate: bool = False,
                   grad_dtype=torch.float32, workspace=None, stream=None):
    """The gradient dY^T X (n_out x n_in) of the weight of y = x W^T, from dy
    (..., n_out) and x held in 8 bits.  With accumulate it is added to `out`.
    Where no `out` is passed the gradient is allocated in `grad_dtype`."""
    _check_cuda(dy, "dy")
    dt = _dtype(dy, "dy")
    rows, n_out, ld = _rows(dy, "dy")
    _held(x, "x")
    if x.rows != rows or (len(dy.shape) == len(x.shape) and dy.shape[:-1] != x.shape[:-1]):
        raise ValueError("dy %s does not belong to x %s" % (tuple(dy.shape), x.shape))
    if accumulate and out is None:
        raise ValueError("accumulate needs the gradient to add to (out)")
    dev = dy.device
    _same_device(dev, ("x", x.codes), ("x", x.exps), ("out", out))
    lib = _abi.load()
    size = C.c_size_t()
    rc = lib.ma_linear_grad_workspace_size(rows, n_out, x.cols, dt, C.byref(size))
    if rc:
        _fail(rc, "ma_linear_grad")
    with _on(dev, stream, (dy, x.codes, x.exps, out, workspace)) as on:
        out = _out_like(out, "out", (n_out, x.cols), grad_dtype, dev)
        if not out.is_contiguous():
            raise ValueError("out must be contiguous")
        ws, ws_ptr, ws_bytes = _workspace(workspace, size.value, dev)
        rc = lib.ma_linear_grad(dy.data_ptr(), dt, rows, n_out, ld, x.codes.data_ptr(),
                                x.exps.data_ptr(), x.cols, out.data_ptr(), _dtype(out, "out"),
                                1 if accumulate else 0, ws_ptr, ws_bytes, on.raw)
    if rc:
        _fail(rc, "ma_linear_grad")
    return out


# -------------------------------------------------------- gated activation --

def _act(act) -> int:
    if isinstance(act, str):
        if act not in _ACTS:
            raise ValueError("act must be one of %s" % ", ".join(sorted(_ACTS)))
        return _ACTS[act]
    return int(act)


def ma_glu_forward(gate, up, act="silu", out=None, gate_ckpt: Optional[ActCheckpoint] = None,
                   up_ckpt: Optional[ActCheckpoint] = None, stream=None):
    """(h, gate held in 8 bits, up held in 8 bits) with h = act(gate) * up;
    act is 'silu' or 'gelu_tanh'."""
    _check_cuda(gate, "gate")
    _check_cuda(up, "up")
    if gate.shape != up.shape or gate.dtype != up.dtype:
        raise ValueError("gate and up differ: %s %s, %s %s" % (tuple(gate.shape), gate.dtype,
                                                               tuple(up.shape), up.dtype))
    dt = _dtype(gate, "gate")
    rows, cols, gld = _rows(gate, "gate")
    _, _, uld = _rows(up, "up")
    dev = gate.device
    _same_device(dev, ("up", up), ("out", out))
    for what, c in (("gate_ckpt", gate_ckpt), ("up_ckpt", up_ckpt)):
        if c is not None:
            _held(c, what, rows, cols)
            _same_device(dev, (what, c.codes), (what, c.exps))
    used = [gate, up, out] + [t for c in (gate_ckpt, up_ckpt) if c is not None
                              for t in (c.codes, c.exps)]
    with _on(dev, stream, used) as on:
        out = _out_as(out, "out", gate)
        gate_ckpt = gate_ckpt or ActCheckpoint._empty(gate.shape, rows, cols, dev)
        up_ckpt = up_ckpt or gate_ckpt._like()
        rc = _abi.load().ma_glu_forward(
            gate.data_ptr(), up.data_ptr(), dt, rows, cols, gld, uld, _act(act), out.data_ptr(),
            _rows(out, "out")[2], gate_ckpt.codes.data_ptr(), gate_ckpt.exps.data_ptr(),
            up_ckpt.codes.data_ptr(), up_ckpt.exps.data_ptr(), on.raw)
    if rc:
        _fail(rc, "ma_glu_forward")
    return out, gate_ckpt, up_ckpt


def ma_glu_backward(dh, gate: ActCheckpoint, up: ActCheckpoint, act="silu", dgate=None, dup=None,
                    h_ckpt=None, stream=None):
    """(dgate, dup) from the gradient dh of h and the held gate and up.  With
    h_ckpt (True, or an ActCheckpoint to fill) a third result is h at the held
    gate and up, itself held in 8 bits: the x of the down projection's
    ma_linear_grad."""
    _check_cuda(dh, "dh")
    dt = _dtype(dh, "dh")
    rows, cols, ld = _rows(dh, "dh")
    dev = dh.device
    _held(gate, "gate", rows, cols)
    _held(up, "up", rows, cols)
    _same_device(dev, ("gate", gate.codes), ("gate", gate.exps), ("up", up.codes),
                 ("up", up.exps), ("dgate", dgate), ("dup", dup))
    hold = h_ckpt is not None and h_ckpt is not False
    used = [dh, gate.codes, gate.exps, up.codes, up.exps, dgate, dup]
    if hold and h_ckpt is not True:
        _held(h_ckpt, "h_ckpt", rows, cols)
        _same_device(dev, ("h_ckpt", h_ckpt.codes), ("h_ckpt", h_ckpt.exps))
        used += [h_ckpt.codes, h_ckpt.exps]
    with _on(dev, stream, used) as on:
        dgate = _out_as(dgate, "dgate", dh)
        dup = _out_as(dup, "dup", dh)
        if hold and h_ckpt is True:
            h_ckpt = ActCheckpoint._empty(dh.shape, rows, cols, dev)
        rc = _abi.load().ma_glu_backward(
            dh.data_ptr(), dt, rows, cols, ld, gate.codes.data_ptr(), gate.exps.data_ptr(),
            up.codes.data_ptr(), up.exps.data_ptr(), _act(act), dgate.data_ptr(),
            _rows(dgate, "dgate")[2], dup.data_ptr(), _rows(dup, "dup")[2],
            h_ckpt.codes.data_ptr() if hold else None, h_ckpt.exps.data_ptr() if hold else None,
            on.raw)
    if rc:
        _fail(rc, "ma_glu_backward")
    return (dgate, dup, h_ckpt) if hold else (dgate, dup)


# -------------------------------------------------------- gradient sources --

class EmbeddingGrad(NamedTuple):
    """The gradient of an embedding table, to be formed by ma_embedding_grad."""
    dout: object
    tokens: object
    scale: float = 1.0
    padding_token: int = -1


class LinearGrad(NamedTuple):
    """The gradient of a linear layer's weight, to be formed by ma_linear_grad."""
    dy: object
    x: ActCheckpoint


def form_gradient(source, shape, out, accumulate: bool, stream=None):
    """Form one gradient source into (or add it to) `out`, a contiguous
    float32 or bfloat16 tensor of the parameter's shape."""
    if isinstance(source, EmbeddingGrad):
        return ma_embedding_grad(source.dout, source.tokens, shape[0], source.scale,
                                 source.padding_token, out=out, accumulate=accumulate,
                                 stream=stream)
    if isinstance(source, LinearGrad):
        return ma_linear_grad(source.dy, source.x, out=out, accumulate=accumulate, stream=stream)
    raise TypeError("expected an EmbeddingGrad or a LinearGrad, got %s" % type(source).__name__)
