"""Python binding of the operators that end a training step (include/trimul.h): argument marshalling
only.

  AdamW    one step over many tensors, with states in 32 bits or in 8, which clips by the norm of a
           GradSet in the same pass
  Linear8  a linear layer whose operands are 8-bit floating point with a power of two for each block
           of 128, and its gradients

The functions keep the C names; the classes wrap them as those of ``pair_ops`` do: calls take ``stream`` (default:
the current one), do not wait on the host and may be captured; without the library or an sm_103 device
they raise.  Making an object waits, so that it may be used on any stream; in a capture it is made on the captured stream, and does
not wait.
"""

from __future__ import annotations

import functools

import numpy as np
import torch

from . import _lib
from .pair_ops import _TYPES, GradSet, _cuda, _empty, _fits, _one_of, _ptr, _raw, _refuse, _shared, _type
from .trimul import FLAG_CHECK, FLAG_INJECT_STALL, _check  # noqa: F401

_STATES = {"float32": 0, "8bit": 1}
_ROUNDING = {"nearest": 0, "stochastic": 1}
BLOCK = 128  # neighbours that share a scale in the 8-bit states
_BYTES = np.array([2, 4, 2], dtype=np.int64)  # of _TYPES


def _values(v, names):
    """A list or a dict as a list: a dict with the parameters' names (None: they have none) in the parameters' order, else as it is."""
    if not isinstance(v, dict):
        return v
    return [v[k] for k in names] if names is not None and v.keys() == set(names) else list(v.values())


def _listed(v, n, name, names=None):
    """A value for each of n tensors, from one for all, a list or a dict."""
    v = _values(v, names)
    if not isinstance(v, (list, tuple)):
        return [v] * n
    if len(v) != n:
        raise ValueError(f"{len(v)} {name} for {n} params")
    return list(v)


def _ready(dev):
    """Waits for what the current stream has been given, so that an object made there may be used on any stream (in a capture the
    graph's order holds)."""
    with torch.cuda.device(dev):
        if not torch.cuda.is_current_stream_capturing():
            torch.cuda.current_stream().synchronize()


class _Own:
    """An object's own memory, and the streams that it is used on: it is given out again behind the last kernel of each.  An external
    stream may be gone by then: there the caller keeps the object until its kernels have ended."""

    def __init__(self, tensors, dev):
        self.tensors, self.streams = tensors, {_raw(None, dev)}

    def use(self, stream, dev):
        raw = _raw(stream, dev)
        if raw not in self.streams:
            self.streams.add(raw)
            at = torch.cuda.current_stream(dev) if stream is None else stream
            if raw == 0 or at.stream_id != raw:  # (an external stream's number is its handle)
                for t in self.tensors:
                    t.record_stream(at)


class AdamW:
    """AdamW (decoupled weight decay) over a list (or dict) of parameters: step(grads).

    params: float32 or bf16, updated in place; copies: for each parameter a bf16 or float16 tensor of its shape that
    gets the new value rounded to nearest, or None (default: none); weight_decay: one number, or one for each
    parameter.  Dicts of these and of gradients that have the parameters' names go by them, others by their order.
    states: "float32", or "8bit" for e4m3 codes with a scale for each 128 neighbours.  rounding: how bf16 parameters and
    8-bit states are rounded, "stochastic" (at random, by a hash of `seed`, the step and the element) or "nearest".

    `state` has the states of all parameters behind one another, each from a multiple of 128 on (`starts`): "m", "v" and
    "count", the steps taken (int32, on the device), and with "8bit" "m_scale" and "v_scale" by blocks, "v" then being
    the codes of v's root.  A checkpoint keeps these tensors, and goes on by copying into them.  The object stands for
    the memory that its tensors have when it is made, and keeps it.  Steps of one object are one after the other: on several
    streams, or as graphs that are replayed, the caller sees to it.  No parameter or copy may lie over another one, nor a
    gradient over any of them."""

    def __init__(self, params, lr=1e-3, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.01, states="float32", copies=None,
                 rounding="stochastic", seed=0):
        self._names = list(params) if isinstance(params, dict) else None
        params = list(params.values() if isinstance(params, dict) else params)
        n = len(params)
        copies = _listed(copies, n, "copies", self._names)
        decay = _listed(weight_decay, n, "weight_decay", self._names)
        self.params, self.copies, self.lr = params, copies, lr
        self.device = _cuda(params[0], "params[0]") if params else torch.cuda.current_device()
        for k, (p, c) in enumerate(zip(params, copies)):
            _type(p.dtype, f"params[{k}]")
            if not _fits(p, p.dtype, p.shape, self.device):
                _refuse(p, p.dtype, p.shape, self.device, f"params[{k}]")
            if c is None:
                continue
            if c.dtype not in (torch.bfloat16, torch.float16):
                raise TypeError(f"copies[{k}] must be bf16 or float16, got {c.dtype}")
            if not _fits(c, c.dtype, p.shape, self.device):
                _refuse(c, c.dtype, p.shape, self.device, f"copies[{k}]")
        self._memory = [t.untyped_storage() for t in params + copies if t is not None]
        self.eight = _one_of(_STATES, states, "states") == 1
        numel = np.array([p.numel() for p in params], dtype=np.int64)
        padded = -(-numel // BLOCK) * BLOCK
        starts = np.concatenate([[0], np.cumsum(padded)])
        total, dev = int(starts[-1]), torch.device("cuda", self.device)
        self.starts = [int(v) for v in starts[:-1]]
        self._count = torch.zeros(2, dtype=torch.int32, device=dev)
        kind = torch.float8_e4m3fn if self.eight else torch.float32
        self.state = {k: torch.zeros(total, dtype=kind, device=dev) for k in "mv"}
        if self.eight:
            self.state.update({k + "_scale": torch.zeros(total // BLOCK, dtype=torch.float32, device=dev) for k in "mv"})
        self._own = _Own([*self.state.values(), self._count], self.device)
        self.state["count"], self._count_at = self._count[0], self._count.data_ptr()
        # one row of numbers for each tensor, as _lib.AdamwTensor lays them out
        rows = np.zeros(n, dtype=np.dtype([("param", "<i8"), ("copy", "<i8"), ("m", "<i8"), ("v", "<i8"),
                                           ("m_scale", "<i8"), ("v_scale", "<i8"), ("numel", "<i8"), ("weight_decay", "<f4"),
                                           ("param_type", "<i4"), ("copy_type", "<i4")], align=True))
        rows["param"] = [p.data_ptr() for p in params]
        rows["copy"] = [0 if c is None else c.data_ptr() for c in copies]
        rows["numel"], rows["weight_decay"] = numel, decay
        rows["param_type"] = [_TYPES[p.dtype] for p in params]
        rows["copy_type"] = [0 if c is None else _TYPES[c.dtype] for c in copies]
        for k in "mv":
            rows[k] = self.state[k].data_ptr() + starts[:-1] * (1 if self.eight else 4)
            if self.eight:
                rows[k + "_scale"] = self.state[k + "_scale"].data_ptr() + starts[:-1] // BLOCK * 4
        at = np.concatenate([rows["param"], rows["copy"]])
        both = _shared(at, at, np.concatenate([numel * _BYTES[rows["param_type"]], np.where(rows["copy"] != 0, 2 * numel, 0)]))
        if both:
            names = [f"{'params' if k < n else 'copies'}[{k % n}]" for k in both]
            raise ValueError(f"{names[1]} overlaps {names[0]}")
        self.table = (_lib.AdamwTensor * n).from_buffer(rows) if n else (_lib.AdamwTensor * 0)()
        self._p = _lib.AdamwParams(beta1=betas[0], beta2=betas[1], eps=eps, lr=0.0, states=int(self.eight),
                                   rounding=_one_of(_ROUNDING, rounding, "rounding"), seed=seed & 0xFFFFFFFF)
        _ready(self.device)

    def step(self, grads, lr=None, norm=None, max_norm=None, stream=None, flags: int = 0):
        """One step with `grads` (a GradSet, a list or a dict, in the parameters' order; bf16, float16 or float32).  Of a
        GradSet its tensors are read, not its `outs`: after a clip() into those, give the outs themselves.

        lr: for this step and the later ones, a number or a float32 tensor on the device, which a captured step reads
        each time; norm (GradSet.norm's, on the device) and max_norm: clip by it in the same pass; a norm that is not
        finite makes the step nothing."""
        if not isinstance(grads, GradSet):
            grads = GradSet(_values(grads, self._names))
        p = self._p
        if len(grads.table) != len(self.table):
            raise ValueError(f"{len(grads.table)} grads for {len(self.table)} params")
        if grads.device != self.device and len(self.table):
            raise ValueError(f"grads must be on cuda:{self.device}, got cuda:{grads.device}")
        lr = self.lr if lr is None else lr
        if (norm is None) != (max_norm is None):
            raise ValueError("give both norm and max_norm, or neither")
        p.norm, p.max_norm = self._one(norm, "norm"), 0.0 if max_norm is None else max_norm
        if isinstance(lr, torch.Tensor):
            p.lr, p.lr_device = 0.0, self._one(lr, "lr")
        else:
            p.lr, p.lr_device = lr, None
        self._own.use(stream, self.device)
        _check(_lib.load().trimul_adamw_step(p, self.table, grads.table, len(self.table), self._count_at, self.device,
                                             _raw(stream, self.device), flags))
        self.lr = lr  # (a step that is refused leaves it)

    def _one(self, t, name):
        if t is None:
            return None
        if t.dtype != torch.float32 or t.numel() != 1 or t.get_device() != self.device:
            raise ValueError(f"{name} must be one float32 on cuda:{self.device}")
        return t.data_ptr()


# ------------------------------------------------------------------ linear layer in 8 bits
# The smallest calls' workspace is the word in which a kernel says that it gave up.  Calls on one stream come one after the other, so
# each stream keeps one (an allocation is a tenth of such a call's time); what is captured has its own.
_WORD = 256
_words = {}


def _workspace(need, dev, device, stream, raw):
    if need > _WORD or stream is not None or torch.cuda.is_current_stream_capturing():
        return _empty(need, torch.uint8, device, stream)
    word = _words.get((dev, raw))
    if word is None:
        word = _words[dev, raw] = _empty(_WORD, torch.uint8, device, stream)
    return word


@functools.lru_cache(maxsize=1024)
def _forward_bytes(rows, N, K):
    return _lib.load().trimul_linear8_forward_workspace_bytes(rows, N, K)


def _rows(x, width, dev, name):
    """The rows of a bf16 tensor [..., width]."""
    if x.dim() < 1 or x.shape[-1] != width:
        raise ValueError(f"{name} must be [..., {width}], got {tuple(x.shape)}")
    if not _fits(x, torch.bfloat16, x.shape, dev):
        _refuse(x, torch.bfloat16, x.shape, dev, name)
    return x.numel() // width


@functools.lru_cache(maxsize=1024)
def _backward_bytes(rows, N, K):
    return _lib.load().trimul_linear8_backward_workspace_bytes(rows, N, K)


def trimul_linear8_pack(weight, packed=None, stream=None, flags: int = 0):
    """The weight [N, K] (bf16 or float32) as the calls below read it, a uint8 tensor; written to `packed` if that is given."""
    dev = _cuda(weight, "weight")
    kind = _type(weight.dtype, "weight")
    if weight.dim() != 2:
        raise ValueError(f"weight must be [N, K], got {tuple(weight.shape)}")
    if not weight.is_contiguous():
        raise ValueError("weight must be contiguous")
    N, K = weight.shape
    lib = _lib.load()
    need = lib.trimul_linear8_packed_bytes(N, K)
    if packed is None:
        packed = _empty(need, torch.uint8, weight.device, stream)
    elif not _fits(packed, torch.uint8, (need,), dev):
        _refuse(packed, torch.uint8, (need,), dev, "packed")
    _check(lib.trimul_linear8_pack(weight.data_ptr(), kind, N, K, packed.data_ptr(), need, dev, _raw(stream, dev), flags))
    return packed


def trimul_linear8_forward(packed, N, K, x, bias=None, out=None, stream=None, flags: int = 0):
    """x W^T + bias: bf16 [..., N] for bf16 x [..., K]; bias: float32 [N]."""
    dev = _packed(packed, N, K)
    if bias is not None and not _fits(bias, torch.float32, (N,), dev):
        _refuse(bias, torch.float32, (N,), dev, "bias")
    return _forward(packed, N, K, dev, x, bias, out, stream, flags)


def _forward(packed, N, K, dev, x, bias, out, stream, flags):  # packed and bias have been looked at
    shape = x.shape
    if len(shape) == 0 or shape[-1] != K or not _fits(x, torch.bfloat16, shape, dev):
        _rows(x, K, dev, "x")
    rows, shape = x.numel() // K, (*shape[:-1], N)
    if out is None:
        out = _empty(shape, torch.bfloat16, x.device, stream)
    elif not _fits(out, torch.bfloat16, shape, dev):
        _refuse(out, torch.bfloat16, shape, dev, "out")
    need, raw = _forward_bytes(rows, N, K), _raw(stream, dev)
    ws = _workspace(need, dev, x.device, stream, raw)
    _check(_lib.load().trimul_linear8_forward(packed.data_ptr(), _ptr(bias), x.data_ptr(), rows, N, K, out.data_ptr(), ws.data_ptr(), need,
                                              dev, raw, flags))
    return out


def trimul_linear8_backward(packed, N, K, x, dy, dx=None, dw=None, dbias=None, want=("dx", "dw", "dbias"), stream=None,
                            flags: int = 0):
    """{"dx", "dw", "dbias"} for dy (bf16 [..., N]) with respect to the output: bf16 like x, float32 [N, K] and [N]; those that
    `want` does not name are None."""
    return _backward(packed, N, K, _packed(packed, N, K), x, dy, dx, dw, dbias, want, stream, flags)


def _backward(packed, N, K, dev, x, dy, dx, dw, dbias, want, stream, flags):  # packed has been looked at
    rows = _rows(x, K, dev, "x")
    if _rows(dy, N, dev, "dy") != rows or dy.shape[:-1] != x.shape[:-1]:
        raise ValueError(f"dy must be {(*x.shape[:-1], N)}, got {tuple(dy.shape)}")
    for k in want:
        if k not in ("dx", "dw", "dbias"):
            raise ValueError(f"unknown gradient {k!r}: dx, dw and dbias are given")
    got = {}
    for name, t, dtype, shape in (("dx", dx, torch.bfloat16, x.shape), ("dw", dw, torch.float32, (N, K)), ("dbias", dbias, torch.float32, (N,))):
        if name not in want:
            if t is not None:
                raise ValueError(f"{name} is given but not among what is wanted, {tuple(want)}")
            got[name] = None
        elif t is None:
            got[name] = _empty(shape, dtype, x.device, stream)
        else:
            if not _fits(t, dtype, shape, dev):
                _refuse(t, dtype, shape, dev, name)
            got[name] = t
    need = _backward_bytes(rows, N, K)
    ws = _empty(need, torch.uint8, x.device, stream)
    _check(_lib.load().trimul_linear8_backward(packed.data_ptr(), x.data_ptr(), dy.data_ptr(), rows, N, K, _ptr(got["dx"]),
                                               _ptr(got["dw"]), _ptr(got["dbias"]), ws.data_ptr(), need, dev, _raw(stream, dev), flags))
    return got


def _packed(packed, N, K) -> int:
    """The device of a packed weight of these sizes."""
    dev = _cuda(packed, "packed")
    need = _lib.load().trimul_linear8_packed_bytes(N, K)
    if need == 0:
        raise ValueError(f"N ({N}) and K ({K}) must be multiples of 8 in [8, 65536]")
    if not _fits(packed, torch.uint8, (need,), dev):
        _refuse(packed, torch.uint8, (need,), dev, "packed")
    return dev


class Linear8:
    """A linear layer in 8 bits: forward(x) and backward(x, dy).

    The weight [N, K] (bf16 or float32) is rounded to 8 bits when the object is made, and again by pack(weight) after
    each change of it, such as an optimiser's step; the object keeps the 8-bit form, not the weight.  bias: float32 [N],
    read at each call."""

    def __init__(self, weight, bias=None):
        self.packed = trimul_linear8_pack(weight)
        self.N, self.K = weight.shape
        self.device = weight.get_device()
        if bias is not None and not _fits(bias, torch.float32, (self.N,), self.device):
            _refuse(bias, torch.float32, (self.N,), self.device, "bias")
        self.bias = bias
        self._own = _Own([self.packed], self.device)
        _ready(self.device)

    def pack(self, weight, stream=None, flags: int = 0):
        if tuple(weight.shape) != (self.N, self.K):
            raise ValueError(f"weight must be {(self.N, self.K)}, got {tuple(weight.shape)}")
        self._own.use(stream, self.device)
        trimul_linear8_pack(weight, self.packed, stream, flags)

    def forward(self, x, out=None, stream=None, flags: int = 0):
        self._own.use(stream, self.device)
        return _forward(self.packed, self.N, self.K, self.device, x, self.bias, out, stream, flags)

    __call__ = forward

    def backward(self, x, dy, dx=None, dw=None, dbias=None, want=None, stream=None, flags: int = 0):
        """{"dx", "dw", "dbias"}; dbias is None for a layer without bias (unless `want` names it), and so is what `want` does
        not name."""
        if want is None:
            want = ("dx", "dw", "dbias") if self.bias is not None else ("dx", "dw")
        self._own.use(stream, self.device)
        return _backward(self.packed, self.N, self.K, self.device, x, dy, dx, dw, dbias, want, stream, flags)
