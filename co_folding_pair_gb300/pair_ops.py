"""Python binding of the operators around the layer (include/trimul.h): argument
marshalling only.

Three operators join TriMul layers into a pair stack and its training step:

  RelPos    the relative position bias by buckets that a pair representation
            (or an attention) starts from, and its table's gradient
  Residual  the step from a layer's output back into the residual stream:
            norm after, gate, scale, norm before the next layer; and its gradients
  GradSet   the norm over many gradients, and clipping by it

The functions keep the C names; the classes wrap them as ``TriMul`` wraps the
layer's, and ``PairBlock`` is a layer with its residual step.  Every call takes
``stream`` (default: the current one) and allocates its outputs and workspace
there.  There is no fallback: without the library or an sm_103 device the calls
raise.
"""

from __future__ import annotations

import contextlib
import ctypes
import math

import numpy as np
import torch

from . import _lib
from . import trimul as _T
from .trimul import FLAG_CHECK, TrimulError, _check

FLAG_ACCUMULATE = 16  # trimul_relpos_backward only: add to dtable

_TYPES = {torch.bfloat16: 0, torch.float32: 1, torch.float16: 2}
_KINDS = {"linear": 0, "log": 1}
_LAYOUTS = {"pair": 0, "heads": 1}
_NORMS = {None: 0, "none": 0, "layer": 1, "rms": 2}


# The smallest calls take a few microseconds on the device, so what happens here
# counts: a tensor that is as it should be is passed by four quick looks (_fits),
# and only another one is looked at again for the message (_refuse).
def _fits(t, dtype, shape, dev) -> bool:
    return t.dtype is dtype and t.shape == shape and t.get_device() == dev and t.is_contiguous()


def _refuse(t, dtype, shape, dev, name):
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must be {tuple(shape)}, got {tuple(t.shape)}")
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on cuda:{dev}, got {t.device}")
    raise ValueError(f"{name} must be contiguous")


def _one_of(table, value, name):
    try:
        return table[value]
    except (KeyError, TypeError):
        raise ValueError(f"{name} must be one of {[k for k in table if k is not None]}, got {value!r}") from None


def _type(dtype, name, most=1) -> int:
    """The number of an element type: bf16 or float32, or (most 2) float16."""
    kind = _TYPES.get(dtype, 3)
    if kind > most:
        raise TypeError(f"{name} must be one of {[k for k, v in _TYPES.items() if v <= most]}, got {dtype}")
    return kind


def _cuda(t, name) -> int:
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"{name} must be on a CUDA device, got {t.device}")
    return dev


def _device(device) -> int:
    """The number of a device: the current one where none, or "cuda" without a number, is given."""
    at = torch.device("cuda" if device is None else device)
    if at.type != "cuda":
        raise ValueError(f"device must be a CUDA device, got {device}")
    return torch.cuda.current_device() if at.index is None else at.index


def _empty(shape, dtype, device, stream):
    """Uninitialised memory of `stream`, so that the allocator gives it out again in that stream's order."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _raw(stream, dev) -> int:
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream


def _ptr(t):
    return None if t is None else t.data_ptr()


# ------------------------------------------------------------------ relative position bias
class RelPosPlan:
    """An opaque trimul_relpos with its table's rows and its device."""

    def __init__(self, ptr, rows, device):
        self.ptr, self.rows, self.device = ptr, rows, device


def trimul_relpos_create(kind="linear", max_distance=32, num_buckets=None, bidirectional=True, groups=False,
                         device=None) -> RelPosPlan:
    """A plan: kind "linear" (distances clipped to max_distance) or "log" (num_buckets in all, half of each
    side's exact and the others log-spaced up to max_distance); `groups`: one table row more, the last, for
    pairs of different groups."""
    lib = _lib.load()
    p = _lib.RelposParams(_one_of(_KINDS, kind, "kind"), int(max_distance), int(num_buckets or 0),
                          int(bool(bidirectional)), int(bool(groups)))
    dev = _device(device)
    out = ctypes.c_void_p()
    _check(lib.trimul_relpos_create(ctypes.byref(out), ctypes.byref(p), dev))
    return RelPosPlan(out, trimul_relpos_rows(out), dev)


def trimul_relpos_rows(r) -> int:
    n = int(_lib.load().trimul_relpos_rows(r.ptr if isinstance(r, RelPosPlan) else r))
    if n < 0:
        raise TrimulError(1, _T.trimul_last_error())
    return n


def _positions(r, q_pos, k_pos, q_group, k_group):
    """B, I, J and the keys' positions and groups."""
    if q_pos.dim() != 2:
        raise ValueError(f"q_pos must be [B, length], got {tuple(q_pos.shape)}")
    shape, dev = q_pos.shape, r.device
    if not _fits(q_pos, torch.int32, shape, dev):
        _refuse(q_pos, torch.int32, shape, dev, "q_pos")
    B, I = shape
    if k_pos is None or k_pos is q_pos:
        k_pos, J = q_pos, I
        if k_group is None:
            k_group = q_group
    else:
        if k_pos.dim() != 2:
            raise ValueError(f"k_pos must be [B, length], got {tuple(k_pos.shape)}")
        J = k_pos.shape[1]
        if not _fits(k_pos, torch.int32, (B, J), dev):
            _refuse(k_pos, torch.int32, (B, J), dev, "k_pos")
    if (q_group is None) != (k_group is None):
        raise ValueError("give both q_group and k_group, or neither")
    if q_group is not None:
        if not _fits(q_group, torch.int32, shape, dev):
            _refuse(q_group, torch.int32, shape, dev, "q_group")
        if k_group is not q_group and not _fits(k_group, torch.int32, (B, J), dev):
            _refuse(k_group, torch.int32, (B, J), dev, "k_group")
    return B, I, J, k_pos, k_group


def trimul_relpos_forward(r: RelPosPlan, table, q_pos, k_pos=None, q_group=None, k_group=None, base=None,
                          layout="pair", dtype=torch.bfloat16, out=None, stream=None, flags: int = 0):
    """base + table[bucket] as [B, I, J, D] (layout "pair") or [B, D, I, J] ("heads").

    table: [rows, D] bf16 or float32; q_pos, q_group: int32 [B, I]; k_pos, k_group: int32 [B, J] (default: the
    queries'); base, if given, sets the type of the result (else `dtype`); `out` may be `base`."""
    lay = _one_of(_LAYOUTS, layout, "layout")
    B, I, J, k_pos, k_group = _positions(r, q_pos, k_pos, q_group, k_group)
    kind = table.dtype
    tt = _type(kind, "table")
    if table.dim() != 2 or table.shape[0] != r.rows:
        raise ValueError(f"table must be [{r.rows}, D], got {tuple(table.shape)}")
    D = table.shape[1]
    if not _fits(table, kind, (r.rows, D), r.device):
        _refuse(table, kind, (r.rows, D), r.device, "table")
    shape = (B, I, J, D) if lay == 0 else (B, D, I, J)
    dtype = dtype if base is None else base.dtype
    ot = _type(dtype, "dtype" if base is None else "base")
    if base is not None and not _fits(base, dtype, shape, r.device):
        _refuse(base, dtype, shape, r.device, "base")
    if out is None:
        out = _empty(shape, dtype, q_pos.device, stream)
    elif not _fits(out, dtype, shape, r.device):
        _refuse(out, dtype, shape, r.device, "out")
    _check(_lib.load().trimul_relpos_forward(r.ptr, table.data_ptr(), tt, q_pos.data_ptr(), k_pos.data_ptr(),
                                             _ptr(q_group), _ptr(k_group), _ptr(base), B, I, J, D, lay, out.data_ptr(),
                                             ot, _raw(stream, r.device), flags))
    return out


def trimul_relpos_backward(r: RelPosPlan, dout, q_pos, k_pos=None, q_group=None, k_group=None, layout="pair",
                           dtable=None, stream=None, flags: int = 0):
    """The table's gradient, float32 [rows, D], from dout [B, I, J, D] or [B, D, I, J] (bf16 or float32); with
    FLAG_ACCUMULATE it is added to `dtable`."""
    lay = _one_of(_LAYOUTS, layout, "layout")
    B, I, J, k_pos, k_group = _positions(r, q_pos, k_pos, q_group, k_group)
    ot = _type(dout.dtype, "dout")
    D = dout.shape[-1 if lay == 0 else 1] if dout.dim() == 4 else 0
    shape = (B, I, J, D) if lay == 0 else (B, D, I, J)
    if not _fits(dout, dout.dtype, shape, r.device):
        _refuse(dout, dout.dtype, shape, r.device, "dout")
    lib = _lib.load()
    need = lib.trimul_relpos_backward_workspace_bytes(r.ptr, B, I, J, D, lay, ot)
    if dtable is None:
        if flags & FLAG_ACCUMULATE:
            raise ValueError("FLAG_ACCUMULATE needs dtable")
        dtable = _empty((r.rows, D), torch.float32, dout.device, stream)
    elif not _fits(dtable, torch.float32, (r.rows, D), r.device):
        _refuse(dtable, torch.float32, (r.rows, D), r.device, "dtable")
    ws = _empty(need, torch.uint8, dout.device, stream)
    _check(lib.trimul_relpos_backward(r.ptr, dout.data_ptr(), ot, q_pos.data_ptr(), k_pos.data_ptr(), _ptr(q_group),
                                      _ptr(k_group), B, I, J, D, lay, dtable.data_ptr(), ws.data_ptr(), need,
                                      _raw(stream, r.device), flags))
    return dtable


def trimul_relpos_destroy(r: RelPosPlan):
    if r is not None and r.ptr:
        _check(_lib.load().trimul_relpos_destroy(r.ptr))
        r.ptr = ctypes.c_void_p()


class RelPos:
    """A bucketed relative position bias: construct -> forward / backward -> free.

    "log" buckets have device memory: making them waits for their copy, and free (or the object's end) for the device,
    so neither belongs into the capture of a graph."""

    def __init__(self, kind="linear", max_distance=32, num_buckets=None, bidirectional=True, groups=False, device=None):
        self.plan = trimul_relpos_create(kind, max_distance, num_buckets, bidirectional, groups, device)
        self.rows = self.plan.rows

    def forward(self, table, q_pos, k_pos=None, q_group=None, k_group=None, base=None, layout="pair",
                dtype=torch.bfloat16, out=None, stream=None, flags: int = 0):
        return trimul_relpos_forward(self.plan, table, q_pos, k_pos, q_group, k_group, base, layout, dtype, out, stream, flags)

    def backward(self, dout, q_pos, k_pos=None, q_group=None, k_group=None, layout="pair", dtable=None, stream=None,
                 flags: int = 0):
        return trimul_relpos_backward(self.plan, dout, q_pos, k_pos, q_group, k_group, layout, dtable, stream, flags)

    def free(self):
        trimul_relpos_destroy(self.plan)

    def __del__(self):
        try:
            if getattr(self, "plan", None) is not None and self.plan.ptr:
                trimul_relpos_destroy(self.plan)
        except Exception:
            pass


# ------------------------------------------------------------------ residual step
RESIDUAL_PARAMS = _lib.RESIDUAL_GRAD_FIELDS  # post_gamma, post_beta, pre_gamma, pre_beta, channel


def _residual(x, u, params, post_norm, pre_norm, gate, gate_sigmoid, mask, scale, eps):
    """The C parameter block of a call, its checks, the device and the gate's kind."""
    dev = _cuda(x, "x")
    if x.dim() != 4:
        raise ValueError(f"x must be [B, I, J, D], got {tuple(x.shape)}")
    shape, bf = x.shape, torch.bfloat16
    B, I, J, D = shape
    if not x.is_contiguous():
        raise ValueError("x must be contiguous")
    if not _fits(u, bf, shape, dev):
        _refuse(u, bf, shape, dev, "u")
    kind = 0  # trimul_gate
    if gate is not None:
        if gate.shape == shape:  # where I or J is 1, too
            kind = 1
        elif gate.shape == (B, 1, J, D):
            kind = 2
        elif gate.shape == (B, I, 1, D):
            kind = 3
        else:
            raise ValueError(f"gate must be one of {[(B, I, J, D), (B, 1, J, D), (B, I, 1, D)]}, got {tuple(gate.shape)}")
        if not _fits(gate, bf, gate.shape, dev):
            _refuse(gate, bf, gate.shape, dev, "gate")
    if mask is not None and not _fits(mask, bf, (B, I, J), dev):
        _refuse(mask, bf, (B, I, J), dev, "mask")
    at = []
    for k in RESIDUAL_PARAMS:
        v = params.get(k)
        if v is None:
            at.append(None)
        else:
            if not _fits(v, torch.float32, (D,), dev):
                _refuse(v, torch.float32, (D,), dev, k)
            at.append(v.data_ptr())
    for k in params:
        if k not in RESIDUAL_PARAMS:
            raise ValueError(f"unknown parameter {k!r}: {list(RESIDUAL_PARAMS)} are taken")
    xt = _type(x.dtype, "x")
    post, pre = _NORMS.get(post_norm), _NORMS.get(pre_norm)
    if post is None or pre is None:
        _one_of(_NORMS, post_norm, "post_norm")
        _one_of(_NORMS, pre_norm, "pre_norm")
    p = _lib.ResidualParams(D, xt, post, pre, *at, kind, 1 if gate_sigmoid else 0, scale, eps)
    return p, dev, kind


def trimul_residual_forward(x, u, params=None, post_norm=None, pre_norm=None, gate=None, gate_sigmoid=False,
                            mask=None, scale=1.0, eps=1e-5, out=None, normed=None, stream=None, flags: int = 0):
    """(out, normed): out = x + scale mask channel G(gate) Norm_post(u) and normed = Norm_pre(out), None without pre_norm.

    x: bf16 or float32 [B, I, J, D]; u: bf16 alike; params: float32 [D] tensors by name (post_gamma, post_beta,
    pre_gamma, pre_beta, channel), any of them absent; norms: "layer", "rms" or None; gate: bf16 [B, I, J, D],
    [B, 1, J, D] or [B, I, 1, D]; mask: bf16 [B, I, J].  out may be x."""
    p, dev, _ = _residual(x, u, params or {}, post_norm, pre_norm, gate, gate_sigmoid, mask, scale, eps)
    shape = x.shape
    if out is None:
        out = _empty(shape, x.dtype, x.device, stream)
    elif not _fits(out, x.dtype, shape, dev):
        _refuse(out, x.dtype, shape, dev, "out")
    if normed is not None:
        if not _fits(normed, torch.bfloat16, shape, dev):
            _refuse(normed, torch.bfloat16, shape, dev, "normed")
    elif p.pre_norm:
        normed = _empty(shape, torch.bfloat16, x.device, stream)
    _check(_lib.load().trimul_residual_forward(p, x.data_ptr(), u.data_ptr(), _ptr(gate), _ptr(mask), *shape[:3],
                                               out.data_ptr(), _ptr(normed), dev, _raw(stream, dev), flags))
    return out, normed


def trimul_residual_backward(x, u, dout, params=None, post_norm=None, pre_norm=None, gate=None, gate_sigmoid=False,
                             mask=None, scale=1.0, eps=1e-5, dnormed=None, dout2=None, dx=None, du=None, dgate=None,
                             grads=None, stream=None, flags: int = 0):
    """{"dx", "du", "dgate", "grads"} for the gradients dout (+ dout2) of out and dnormed of normed.

    The other arguments are the forward's (x as it was before).  dx may be dout.  dgate is None unless the gate is
    [B, I, J, D]; grads holds a float32 [D] tensor for each of `params` (give a dict to have them written there:
    only the names in it are computed)."""
    params = params or {}
    p, dev, kind = _residual(x, u, params, post_norm, pre_norm, gate, gate_sigmoid, mask, scale, eps)
    shape, xt, bf = x.shape, x.dtype, torch.bfloat16
    for t, name, dt in ((dout, "dout", xt), (dout2, "dout2", xt), (dnormed, "dnormed", bf), (dx, "dx", xt), (du, "du", bf),
                        (dgate, "dgate", bf)):
        if t is not None and not _fits(t, dt, shape, dev):
            _refuse(t, dt, shape, dev, name)
    D, device = shape[3], x.device
    lib = _lib.load()
    need = lib.trimul_residual_backward_workspace_bytes(p, *shape[:3])
    dx = _empty(shape, xt, device, stream) if dx is None else dx
    du = _empty(shape, bf, device, stream) if du is None else du
    if dgate is None and kind == 1:
        dgate = _empty(shape, bf, device, stream)
    if grads is None:
        grads = {k: _empty(D, torch.float32, device, stream) for k in params}
    else:
        for k, v in grads.items():
            if k not in RESIDUAL_PARAMS:
                raise ValueError(f"unknown parameter {k!r}: {list(RESIDUAL_PARAMS)} are taken")
            if not _fits(v, torch.float32, (D,), dev):
                _refuse(v, torch.float32, (D,), dev, k)
    ws = _empty(need, torch.uint8, device, stream)
    g = _lib.ResidualGrads(*[_ptr(grads.get(k)) for k in RESIDUAL_PARAMS])
    _check(lib.trimul_residual_backward(p, x.data_ptr(), u.data_ptr(), _ptr(gate), _ptr(mask), dout.data_ptr(),
                                        _ptr(dout2), _ptr(dnormed), *shape[:3], dx.data_ptr(), du.data_ptr(), _ptr(dgate),
                                        g, ws.data_ptr(), need, dev, _raw(stream, dev), flags))
    return {"dx": dx, "du": du, "dgate": dgate, "grads": grads}


class Residual:
    """A residual step with its parameters: forward(x, u) and backward(x, u, dout)."""

    def __init__(self, params=None, post_norm=None, pre_norm=None, gate_sigmoid=False, scale=1.0, eps=1e-5):
        self.params = dict(params or {})
        self.post_norm, self.pre_norm = post_norm, pre_norm
        self.gate_sigmoid, self.scale, self.eps = gate_sigmoid, scale, eps

    def forward(self, x, u, gate=None, mask=None, out=None, normed=None, stream=None, flags: int = 0):
        return trimul_residual_forward(x, u, self.params, self.post_norm, self.pre_norm, gate, self.gate_sigmoid, mask,
                                       self.scale, self.eps, out, normed, stream, flags)

    def backward(self, x, u, dout, dnormed=None, gate=None, mask=None, dout2=None, dx=None, du=None, dgate=None,
                 grads=None, stream=None, flags: int = 0):
        return trimul_residual_backward(x, u, dout, self.params, self.post_norm, self.pre_norm, gate, self.gate_sigmoid,
                                        mask, self.scale, self.eps, dnormed, dout2, dx, du, dgate, grads, stream, flags)


# ------------------------------------------------------------------ gradient norm and clipping
def _shared(data, out, size):
    """(k, i): the output i (out[i], size[i] bytes) lies over the tensor k or its output; None if none does but over its own."""
    some = np.flatnonzero(size)
    by = some[np.argsort(out[some], kind="stable")]
    begin, end = out[by], out[by] + size[by]
    bad = np.flatnonzero(end[:-1] > begin[1:])
    if bad.size:
        return int(by[bad[0]]), int(by[bad[0] + 1])
    # the outputs are apart, so the last one that begins before a tensor's end is the one that reaches furthest
    at = np.searchsorted(begin, data[some] + size[some]) - 1
    own = (by[at] == some) & (out[some] == data[some])
    bad = np.flatnonzero((at >= 0) & (end[at] > data[some]) & ~own)
    return (int(some[bad[0]]), int(by[at[bad[0]]])) if bad.size else None


class GradSet:
    """A list (or dict) of gradients whose norm is taken together: norm() and clip().

    `outs`: buffers of the same shapes and types for clipped copies (default: in place).  A set stands for the memory
    that its tensors have when it is made, keeps it, and reads it at each call: gradients that are new tensors each step
    (trimul_backward without `grads`, zero_grad with set_to_none) need a new set each step, as one that is kept goes on
    with the old memory.  bf16, float16 and float32 may be mixed; all on one device, contiguous.  clip() refuses a set with an output over another's memory, such as one tensor given
    twice."""

    def __init__(self, tensors, outs=None):
        tensors = list(tensors.values() if isinstance(tensors, dict) else tensors)
        outs = tensors if outs is None else list(outs.values() if isinstance(outs, dict) else outs)
        if len(outs) != len(tensors):
            raise ValueError(f"{len(outs)} outs for {len(tensors)} tensors")
        self.tensors, self.outs = tensors, outs
        self._memory = [t.untyped_storage() for t in tensors] + ([] if outs is tensors else [o.untyped_storage() for o in outs])
        self.device = _cuda(tensors[0], "tensors[0]") if tensors else torch.cuda.current_device()
        self.torch_device = torch.device("cuda", self.device)
        data, numel = [t.data_ptr() for t in tensors], [t.numel() for t in tensors]
        kinds = [_TYPES.get(t.dtype, 3) for t in tensors]
        fine = max(kinds, default=0) < 3 and all(t.get_device() == self.device and t.is_contiguous() for t in tensors)
        if outs is tensors:
            to = data
        else:
            to = [o.data_ptr() for o in outs]
            fine = fine and all(o.dtype is t.dtype and o.shape == t.shape and o.get_device() == self.device
                                and o.is_contiguous() for t, o in zip(tensors, outs))
        if not fine:
            for k, (t, o) in enumerate(zip(tensors, outs)):
                _type(t.dtype, f"tensors[{k}]", 2)
                for v, name in ((t, "tensors"), (o, "outs")):
                    if not _fits(v, t.dtype, t.shape, self.device):
                        _refuse(v, t.dtype, t.shape, self.device, f"{name}[{k}]")
        # one row of numbers for each tensor, as _lib.GradTensor lays them out
        rows = np.zeros((len(tensors), 4), dtype=np.int64)
        if tensors:
            rows[:, 0], rows[:, 1], rows[:, 2], rows[:, 3] = data, to, numel, kinds
        self.table = (_lib.GradTensor * len(tensors)).from_buffer(rows) if tensors else (_lib.GradTensor * 0)()
        self._rows, self._apart = rows, False
        self.workspace_bytes = _lib.load().trimul_grad_workspace_bytes(len(tensors))

    def _call(self, name, norm_type, norm, stream, flags, *first):
        if norm_type not in (2, math.inf):
            raise ValueError(f"norm_type must be 2 or infinity, got {norm_type}")
        if norm is None:
            norm = _empty((), torch.float32, self.torch_device, stream)
        elif norm.numel() != 1 or not _fits(norm, torch.float32, norm.shape, self.device):
            raise ValueError(f"norm must be one float32 on cuda:{self.device}")
        ws = _empty(self.workspace_bytes, torch.uint8, self.torch_device, stream)
        _check(getattr(_lib.load(), name)(self.table, len(self.table), *first, 0 if norm_type == 2 else 1, norm.data_ptr(),
                                          ws.data_ptr(), self.workspace_bytes, self.device, _raw(stream, self.device), flags))
        return norm

    def norm(self, norm_type=2.0, norm=None, stream=None, flags: int = 0):
        """The norm, a float32 tensor on the device (the host does not wait for it)."""
        return self._call("trimul_grad_norm", norm_type, norm, stream, flags)

    def clip(self, max_norm, norm_type=2.0, norm=None, stream=None, flags: int = 0):
        """Scale the gradients by min(1, max_norm / (norm + 1e-6)); returns the norm before it.  A norm that is not
        finite leaves them as they are."""
        if not self._apart:  # looked at once: the set's memory stays what it is
            data, out, numel, kinds = self._rows.T
            both = _shared(data, out, numel * np.where(kinds == _TYPES[torch.float32], 4, 2))
            if both:
                raise ValueError(f"outs[{both[1]}] overlaps tensors[{both[0]}] or its output")
            self._apart = True
        return self._call("trimul_grad_clip", norm_type, norm, stream, flags, float(max_norm))


def trimul_grad_norm(tensors, norm_type=2.0, norm=None, stream=None, flags: int = 0):
    """The norm over all the elements of `tensors` (a list or dict), a float32 tensor on their device."""
    return GradSet(tensors).norm(norm_type, norm, stream, flags)


def trimul_grad_clip(tensors, max_norm, norm_type=2.0, outs=None, norm=None, stream=None, flags: int = 0):
    """Clip `tensors` (a list or dict) by their common norm, in place or into `outs`; returns the norm."""
    return GradSet(tensors, outs).clip(max_norm, norm_type, norm, stream, flags)


# ------------------------------------------------------------------ a layer with its residual step
class PairBlock:
    """One TriMul layer and the step back into the stream: z' = z + scale channel gate Norm_post(TriMul(z)).

    forward(z) -> (z', normed or None); backward(z, dout) -> (dz, layer gradients, residual gradients, dgate), the layer
    computed again.  `residual` is a Residual; `layer` a TriMul."""

    def __init__(self, layer: _T.TriMul, residual: Residual):
        self.layer, self.residual = layer, residual

    def _layer(self, z, mask, stream):
        return self.layer(z, mask, out=_empty(z.shape, z.dtype, z.device, stream), stream=stream)

    def forward(self, z, mask=None, gate=None, stream=None):
        return self.residual.forward(z, self._layer(z, mask, stream), gate=gate, mask=mask, stream=stream)

    def backward(self, z, dout, mask=None, gate=None, dnormed=None, dout2=None, stream=None):
        """{"dx", "dz", "dgate", "layer_grads", "residual_grads"}: the gradient of z is dx + dz, its parts along the
        stream and through the layer.  Give both to the block below as dout and dout2: it adds them in 32 bits, in the
        pass that reads them."""
        u = self._layer(z, mask, stream)
        r = self.residual.backward(z, u, dout, dnormed=dnormed, dout2=dout2, gate=gate, mask=mask, stream=stream)
        with contextlib.nullcontext() if stream is None else torch.cuda.stream(stream):
            dz, grads = _T.trimul_backward(self.layer.handle, z, mask, r["du"], self.layer.direction, stream=stream)
        return {"dx": r["dx"], "dz": dz, "dgate": r["dgate"], "layer_grads": grads, "residual_grads": r["grads"]}
