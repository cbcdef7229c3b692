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


def _elsewhere(dev, stream) -> bool:
    """Whether a call is for another device or stream than the current ones."""
    return stream is not None or dev.index != _device_now()


class _At(contextlib.ExitStack):
    """Another device and stream made current, for a call's allocations and
    launches.  Tensors: those the call uses."""

    def __init__(self, dev, stream, tensors):
        super().__init__()
        if stream is not None and not isinstance(stream, int) and stream.device != dev:
            raise ValueError("the stream is on %s, the call runs on %s" % (stream.device, dev))
        try:
            self.enter_context(torch.cuda.device(dev))
            if stream is not None:
                self._take(dev, stream, tensors)
        except BaseException:
            self.close()
            raise

    def _take(self, dev, stream, tensors):
        if isinstance(stream, int):
            # (torch takes a 0 for no handle, and would make a stream of its own)
            stream = torch.cuda.ExternalStream(stream, device=dev) if stream else torch.cuda.default_stream(dev)
        if stream.cuda_stream != _raw_stream(dev.index):
            # memory of another stream's tensors is not handed out again before this
            # stream is done with them
            for t in tensors:
                if t is not None:
                    t.record_stream(stream)
            self.enter_context(torch.cuda.stream(stream))


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


def _check_workspace(workspace, dev):
    if workspace is None:
        return
    _check_cuda(workspace, "workspace")
    _same_device(dev, ("workspace", workspace))
    if not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")


def _workspace(workspace, need: int, dev):
    """(tensor, address, bytes) of a call's workspace."""
    if workspace is None:
        if need == 0:
            return None, None, 0
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
        return workspace, workspace.data_ptr(), need
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


# ------------------------------------------------- activations in 8 bits --

class ActCheckpoint:
    """An activation held in 8 bits: `codes` (int8, rows x code pitch), `exps`
    (uint8, rows x exponent pitch) and its number of features `cols`; `shape` is
    the activation's (default: rows x cols).  It stands for codes * 2^(exps -
    127), one exponent for every 32 features of a token.  The two arrays of one made
    here share an allocation: torch.save takes their clones, or the checkpoint."""

    # (one allocation holds both arrays of a checkpoint made here; its views are
    # made when asked for)
    __slots__ = ("cols", "rows", "shape", "device", "_buf", "_codes", "_exps", "_pc", "_pe", "_n")

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
        if codes.device != exps.device:
            raise ValueError("codes are on %s, exps on %s" % (codes.device, exps.device))
        self._codes, self._exps, self._buf = codes, exps, None
        self._pc, self._pe, self._n = codes.data_ptr(), exps.data_ptr(), codes.numel()
        self.cols, self.rows, self.device = cols, codes.shape[0], codes.device
        self.shape = (self.rows, cols) if shape is None else tuple(shape)
        n = 1
        for d in self.shape:
            n *= int(d)
        if self.shape[-1] != cols or n != self.rows * cols:
            raise ValueError("shape %s is not %d rows of %d features" % (self.shape, self.rows, cols))

    def __reduce__(self):
        # (a copy has arrays, and their addresses, of its own)
        return ActCheckpoint, (self.codes.clone(), self.exps.clone(), self.cols, self.shape)

    @staticmethod
    def empty(shape, device) -> "ActCheckpoint":
        """An uninitialised holder for an activation of this shape."""
        shape = tuple(int(d) for d in shape)
        rows = 1
        for d in shape[:-1]:
            rows *= d
        return ActCheckpoint._empty(shape, rows, shape[-1], device)

    @staticmethod
    def _empty(shape, rows, cols, device):
        if cols < 1:
            raise ValueError("an activation needs at least one feature")
        pitch = -(-cols // MA_ACT_GROUP) * MA_ACT_GROUP
        after = -(-rows * pitch // 256) * 256
        c = object.__new__(ActCheckpoint)
        c._buf = buf = torch.empty(after + rows * (-(-pitch // (4 * MA_ACT_GROUP)) * 4),
                                   dtype=torch.uint8, device=device)
        c._codes = c._exps = None
        c._pc = buf.data_ptr()
        c._pe = c._pc + after
        c.cols, c.rows, c.shape, c.device = cols, rows, tuple(shape), buf.device
        return c

    @property
    def codes(self):
        if self._codes is None:
            pitch = -(-self.cols // MA_ACT_GROUP) * MA_ACT_GROUP
            self._codes = self._buf[:self.rows * pitch].view(torch.int8).view(self.rows, pitch)
        return self._codes

    @property
    def exps(self):
        if self._exps is None:
            pitch = -(-self.cols // MA_ACT_GROUP) * MA_ACT_GROUP
            after = -(-self.rows * pitch // 256) * 256
            self._exps = self._buf[after:].view(self.rows, -(-pitch // (4 * MA_ACT_GROUP)) * 4)
        return self._exps

    def _place(self):
        """Look at the arrays again where their owner has given them other memory since (a
        .data, or a storage that was resized)."""
        c, e, pc = self._codes, self._exps, self._pc
        if self._buf is None:
            if c.data_ptr() == pc and e.data_ptr() == self._pe and \
                    c.numel() == self._n and e.shape[0] == self.rows:
                return
        elif self._buf.data_ptr() == pc and (c is None or c.data_ptr() == pc) and \
                (e is None or e.data_ptr() == self._pe):
            return
        for t in self._tensors():
            if t.numel() and t.untyped_storage().nbytes() < t.storage_offset() + t.numel():
                raise ValueError("the memory of this ActCheckpoint was freed")
        self.__init__(self.codes, self.exps, self.cols, self.shape)

    def _tensors(self):
        return (self._buf,) if self._buf is not None else (self._codes, self._exps)


def _held(c, what: str, dev, rows=None, cols=None):
    if not isinstance(c, ActCheckpoint):
        raise TypeError("%s must be an ActCheckpoint" % what)
    c._place()
    if rows is not None and (c.rows != rows or c.cols != cols):
        raise ValueError("%s holds %d x %d, the call needs %d x %d" % (what, c.rows, c.cols, rows,
                                                                      cols))
    if c.device.type != "cuda":
        raise ValueError("%s must live on the GPU" % what)
    if c.device != dev:
        raise ValueError("%s is on %s, the call runs on %s" % (what, c.device, dev))


def ma_act_pack(x, out: Optional[ActCheckpoint] = None, stream=None) -> ActCheckpoint:
    """x (..., features) held in 8 bits."""
    _check_cuda(x, "x")
    dt = _dtype(x, "x")
    rows, cols, ld = _rows(x, "x")
    dev = x.device
    if out is not None:
        _held(out, "out", dev, rows, cols)
    if _elsewhere(dev, stream):
        with _At(dev, stream, (x,) if out is None else (x, *out._tensors())):
            return ma_act_pack(x, out)
    if out is None:
        out = ActCheckpoint._empty(x.shape, rows, cols, dev)
    rc = _abi.load().ma_act_pack(x.data_ptr(), dt, rows, cols, ld, out._pc, out._pe,
                                 _raw_stream(dev.index))
    if rc:
        _fail(rc, "ma_act_pack")
    return out


def ma_act_unpack(ckpt: ActCheckpoint, dtype=torch.float32, out=None, stream=None):
    """The activation an ActCheckpoint stands for, in `dtype` (or out's)."""
    _held(ckpt, "ckpt", getattr(ckpt, "device", None))
    dev = ckpt.device
    _same_device(dev, ("out", out))
    if _elsewhere(dev, stream):
        with _At(dev, stream, (*ckpt._tensors(), out)):
            return ma_act_unpack(ckpt, dtype, out)
    if out is None:
        out = torch.empty(ckpt.shape, dtype=dtype, device=dev)
        ld = ckpt.cols
    else:
        out = _out_like(out, "out", ckpt.shape, dtype, dev)
        ld = _rows(out, "out")[2]
    rc = _abi.load().ma_act_unpack(ckpt._pc, ckpt._pe, ckpt.rows, ckpt.cols, out.data_ptr(),
                                   _dtype(out, "out"), ld, _raw_stream(dev.index))
    if rc:
        _fail(rc, "ma_act_unpack")
    return out


# -------------------------------------------------------- embedding table --

def ma_embedding_lookup(table, tokens, scale: float = 1.0, out=None, out_dtype=None, stream=None):
    """scale * table[tokens], of shape tokens.shape + (hidden,), in `out_dtype`
    (default: the table's; an `out` passed keeps its own).  A token outside [0,
    vocab) gives a row of zeros."""
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
    if _elsewhere(dev, stream):
        with _At(dev, stream, (table, tokens, out)):
            return ma_embedding_lookup(table, tokens, scale, out, out_dtype)
    if out is None:
        out = torch.empty((*tokens.shape, hidden), dtype=out_dtype or table.dtype, device=dev)
        old = hidden
    else:
        out = _out_like(out, "out", (*tokens.shape, hidden), None, dev)
        old = _rows(out, "out")[2]
    rc = _abi.load().ma_embedding_lookup(table.data_ptr(), dt, vocab, hidden, ld,
                                         tokens.data_ptr(), tb, tokens.numel(), scale,
                                         out.data_ptr(), _dtype(out, "out"), old,
                                         _raw_stream(dev.index))
    if rc:
        _fail(rc, "ma_embedding_lookup")
    return out


def ma_embedding_grad_workspace_size(n_tokens: int, vocab: int, hidden: int) -> int:
    n = C.c_size_t()
    rc = _abi.load().ma_embedding_grad_workspace_size(n_tokens, vocab, hidden, C.byref(n))
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
    _check_workspace(workspace, dev)
    if _elsewhere(dev, stream):
        with _At(dev, stream, (dout, tokens, out, workspace)):
            return ma_embedding_grad(dout, tokens, vocab, scale, padding_token, out, accumulate,
                                     grad_dtype, workspace)
    vocab = int(vocab)
    need = ma_embedding_grad_workspace_size(rows, vocab, hidden)
    out = _out_like(out, "out", (vocab, hidden), grad_dtype, dev)
    if not out.is_contiguous():
        raise ValueError("out must be contiguous")
    ws, ws_ptr, ws_bytes = _workspace(workspace, need, dev)
    rc = _abi.load().ma_embedding_grad(dout.data_ptr(), dt, ld, tokens.data_ptr(), tb, rows,
                                       vocab, hidden, scale, int(padding_token),
                                       out.data_ptr(), _dtype(out, "out"),
                                       1 if accumulate else 0, ws_ptr, ws_bytes,
                                       _raw_stream(dev.index))
    if rc:
        _fail(rc, "ma_embedding_grad")
    return out


# ------------------------------------------------------------ linear layer --

def ma_linear_grad_workspace_size(n_tokens: int, n_out: int, n_in: int,
                                  dy_dtype=torch.bfloat16) -> int:
    """Bytes that serve any dy of this shape, whatever its address and stride (a call without
    a workspace allocates what its own dy needs, which may be much less)."""
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
    dev = dy.device
    _held(x, "x", dev)
    if x.rows != rows or (dy.dim() == len(x.shape) and dy.shape[:-1] != x.shape[:-1]):
        raise ValueError("dy %s does not belong to x %s" % (tuple(dy.shape), x.shape))
    if accumulate and out is None:
        raise ValueError("accumulate needs the gradient to add to (out)")
    _same_device(dev, ("out", out))
    _check_workspace(workspace, dev)
    if _elsewhere(dev, stream):
        with _At(dev, stream, (dy, *x._tensors(), out, workspace)):
            return ma_linear_grad(dy, x, out, accumulate, grad_dtype, workspace)
    lib = _abi.load()
    size = C.c_size_t()
    rc = lib.ma_linear_grad_workspace_size_at(dy.data_ptr(), dt, rows, n_out, ld, x.cols,
                                              C.byref(size))
    if rc:
        _fail(rc, "ma_linear_grad")
    out = _out_like(out, "out", (n_out, x.cols), grad_dtype, dev)
    if not out.is_contiguous():
        raise ValueError("out must be contiguous")
    ws, ws_ptr, ws_bytes = _workspace(workspace, size.value, dev)
    rc = lib.ma_linear_grad(dy.data_ptr(), dt, rows, n_out, ld, x._pc, x._pe, x.cols,
                            out.data_ptr(), _dtype(out, "out"), 1 if accumulate else 0, ws_ptr,
                            ws_bytes, _raw_stream(dev.index))
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
    uld = _rows(up, "up")[2]
    dev = gate.device
    _same_device(dev, ("up", up), ("out", out))
    for what, c in (("gate_ckpt", gate_ckpt), ("up_ckpt", up_ckpt)):
        if c is not None:
            _held(c, what, dev, rows, cols)
    if _elsewhere(dev, stream):
        used = [t for c in (gate_ckpt, up_ckpt) if c is not None for t in c._tensors()]
        with _At(dev, stream, [gate, up, out] + used):
            return ma_glu_forward(gate, up, act, out, gate_ckpt, up_ckpt)
    out = _out_as(out, "out", gate)
    if gate_ckpt is None:
        gate_ckpt = ActCheckpoint._empty(gate.shape, rows, cols, dev)
    if up_ckpt is None:
        up_ckpt = ActCheckpoint._empty(gate.shape, rows, cols, dev)
    rc = _abi.load().ma_glu_forward(
        gate.data_ptr(), up.data_ptr(), dt, rows, cols, gld, uld, _act(act), out.data_ptr(),
        _rows(out, "out")[2], gate_ckpt._pc, gate_ckpt._pe, up_ckpt._pc, up_ckpt._pe,
        _raw_stream(dev.index))
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
    _held(gate, "gate", dev, rows, cols)
    _held(up, "up", dev, rows, cols)
    _same_device(dev, ("dgate", dgate), ("dup", dup))
    hold = h_ckpt is not None and h_ckpt is not False
    if hold and h_ckpt is not True:
        _held(h_ckpt, "h_ckpt", dev, rows, cols)
    if _elsewhere(dev, stream):
        used = [dh, *gate._tensors(), *up._tensors(), dgate, dup]
        if hold and h_ckpt is not True:
            used += h_ckpt._tensors()
        with _At(dev, stream, used):
            return ma_glu_backward(dh, gate, up, act, dgate, dup, h_ckpt)
    dgate = _out_as(dgate, "dgate", dh)
    dup = _out_as(dup, "dup", dh)
    if hold and h_ckpt is True:
        h_ckpt = ActCheckpoint._empty(dh.shape, rows, cols, dev)
    rc = _abi.load().ma_glu_backward(
        dh.data_ptr(), dt, rows, cols, ld, gate._pc, gate._pe, up._pc, up._pe, _act(act),
        dgate.data_ptr(), _rows(dgate, "dgate")[2], dup.data_ptr(), _rows(dup, "dup")[2],
        h_ckpt._pc if hold else None, h_ckpt._pe if hold else None, _raw_stream(dev.index))
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
