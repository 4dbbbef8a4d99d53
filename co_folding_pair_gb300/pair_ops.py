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

import torch

from . import _lib
from . import trimul as _T
from .trimul import FLAG_CHECK, TrimulError, _check, _need, _stream, _vp

FLAG_ACCUMULATE = 16  # trimul_relpos_backward only: add to dtable

_TYPES = {torch.bfloat16: 0, torch.float32: 1, torch.float16: 2}
_KINDS = {"linear": 0, "log": 1}
_LAYOUTS = {"pair": 0, "heads": 1}
_NORMS = {None: 0, "none": 0, "layer": 1, "rms": 2}
_GATES = {"none": 0, "pair": 1, "row": 2, "col": 3}


def _one_of(table, value, name):
    try:
        return table[value]
    except (KeyError, TypeError):
        raise ValueError(f"{name} must be one of {[k for k in table if k is not None]}, got {value!r}") from None


def _type(dtype, name, kinds=(torch.bfloat16, torch.float32)):
    if dtype not in kinds:
        raise TypeError(f"{name} must be one of {list(kinds)}, got {dtype}")
    return _TYPES[dtype]


def _shape(t, shape, name):
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must be {tuple(shape)}, got {tuple(t.shape)}")


def _cuda(t, name):
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be on a CUDA device, got {t.device}")
    return t.device.index


def _within(stream):
    """Allocations inside belong to `stream`, so that the allocator gives them out again in its order."""
    return contextlib.nullcontext() if stream is None else torch.cuda.stream(stream)


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
    dev = torch.cuda.current_device() if device is None else torch.device(device).index or 0
    out = ctypes.c_void_p()
    _check(lib.trimul_relpos_create(ctypes.byref(out), ctypes.byref(p), dev))
    return RelPosPlan(out, trimul_relpos_rows(out), dev)


def trimul_relpos_rows(r) -> int:
    n = int(_lib.load().trimul_relpos_rows(r.ptr if isinstance(r, RelPosPlan) else r))
    if n < 0:
        raise TrimulError(1, _T.trimul_last_error())
    return n


def _positions(r, q_pos, k_pos, q_group, k_group):
    k_pos = q_pos if k_pos is None else k_pos
    if q_group is not None and k_group is None and k_pos is q_pos:
        k_group = q_group
    if (q_group is None) != (k_group is None):
        raise ValueError("give both q_group and k_group, or neither")
    for t, name, like in ((q_pos, "q_pos", None), (k_pos, "k_pos", None), (q_group, "q_group", q_pos),
                          (k_group, "k_group", k_pos)):
        if t is None:
            continue
        _need(t, torch.int32, name, r.device)
        if t.dim() != 2:
            raise ValueError(f"{name} must be [B, length], got {tuple(t.shape)}")
        if like is not None:
            _shape(t, like.shape, name)
    if k_pos.shape[0] != q_pos.shape[0]:
        raise ValueError(f"q_pos and k_pos must have the same B, got {q_pos.shape[0]} and {k_pos.shape[0]}")
    return k_pos, k_group


def trimul_relpos_forward(r: RelPosPlan, table, q_pos, k_pos=None, q_group=None, k_group=None, base=None,
                          layout="pair", dtype=torch.bfloat16, out=None, stream=None, flags: int = 0):
    """base + table[bucket] as [B, I, J, D] (layout "pair") or [B, D, I, J] ("heads").

    table: [rows, D] bf16 or float32; q_pos, q_group: int32 [B, I]; k_pos, k_group: int32 [B, J] (default: the
    queries'); base, if given, sets the type of the result (else `dtype`); `out` may be `base`."""
    lay = _one_of(_LAYOUTS, layout, "layout")
    k_pos, k_group = _positions(r, q_pos, k_pos, q_group, k_group)
    _need(table, table.dtype, "table", r.device)
    tt = _type(table.dtype, "table")
    if table.dim() != 2 or table.shape[0] != r.rows:
        raise ValueError(f"table must be [{r.rows}, D], got {tuple(table.shape)}")
    (B, I), J, D = q_pos.shape, k_pos.shape[1], table.shape[1]
    shape = (B, I, J, D) if lay == 0 else (B, D, I, J)
    dtype = dtype if base is None else base.dtype
    ot = _type(dtype, "dtype" if base is None else "base")
    if base is not None:
        _need(base, dtype, "base", r.device)
        _shape(base, shape, "base")
    if out is None:
        with _within(stream):
            out = torch.empty(shape, dtype=dtype, device=q_pos.device)
    else:
        _need(out, dtype, "out", r.device)
        _shape(out, shape, "out")
    _check(_lib.load().trimul_relpos_forward(r.ptr, _vp(table), tt, _vp(q_pos), _vp(k_pos), _vp(q_group), _vp(k_group),
                                             _vp(base), B, I, J, D, lay, _vp(out), ot, _stream(stream, r.device), flags))
    return out


def trimul_relpos_backward(r: RelPosPlan, dout, q_pos, k_pos=None, q_group=None, k_group=None, layout="pair",
                           dtable=None, stream=None, flags: int = 0):
    """The table's gradient, float32 [rows, D], from dout [B, I, J, D] or [B, D, I, J] (bf16 or float32); with
    FLAG_ACCUMULATE it is added to `dtable`."""
    lay = _one_of(_LAYOUTS, layout, "layout")
    k_pos, k_group = _positions(r, q_pos, k_pos, q_group, k_group)
    _need(dout, dout.dtype, "dout", r.device)
    ot = _type(dout.dtype, "dout")
    (B, I), J = q_pos.shape, k_pos.shape[1]
    D = dout.shape[-1 if lay == 0 else 1] if dout.dim() == 4 else 0
    _shape(dout, (B, I, J, D) if lay == 0 else (B, D, I, J), "dout")
    if dtable is None and flags & FLAG_ACCUMULATE:
        raise ValueError("FLAG_ACCUMULATE needs dtable")
    lib = _lib.load()
    need = lib.trimul_relpos_backward_workspace_bytes(r.ptr, B, I, J, D, lay, ot)
    with _within(stream):
        if dtable is None:
            dtable = torch.empty((r.rows, D), dtype=torch.float32, device=dout.device)
        ws = torch.empty(need, dtype=torch.uint8, device=dout.device)
    _need(dtable, torch.float32, "dtable", r.device)
    _shape(dtable, (r.rows, D), "dtable")
    _check(lib.trimul_relpos_backward(r.ptr, _vp(dout), ot, _vp(q_pos), _vp(k_pos), _vp(q_group), _vp(k_group), B, I, J,
                                      D, lay, _vp(dtable), _vp(ws), need, _stream(stream, r.device), flags))
    return dtable


def trimul_relpos_destroy(r: RelPosPlan):
    if r is not None and r.ptr:
        _check(_lib.load().trimul_relpos_destroy(r.ptr))
        r.ptr = ctypes.c_void_p()


class RelPos:
    """A bucketed relative position bias: construct -> forward / backward -> free."""

    def __init__(self, kind="linear", max_distance=32, num_buckets=None, bidirectional=True, groups=False, device=None):
        self.plan = trimul_relpos_create(kind, max_distance, num_buckets, bidirectional, groups, device)
        self.rows = self.plan.rows

    def forward(self, table, q_pos, k_pos=None, **kw):
        return trimul_relpos_forward(self.plan, table, q_pos, k_pos, **kw)

    def backward(self, dout, q_pos, k_pos=None, **kw):
        return trimul_relpos_backward(self.plan, dout, q_pos, k_pos, **kw)

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
    """The C parameter block of a call, its checks, and the gate's kind."""
    dev = _cuda(x, "x")
    _need(x, x.dtype, "x", dev)
    if x.dim() != 4:
        raise ValueError(f"x must be [B, I, J, D], got {tuple(x.shape)}")
    B, I, J, D = x.shape
    _need(u, torch.bfloat16, "u", dev)
    _shape(u, x.shape, "u")
    kind = "none"
    if gate is not None:
        _need(gate, torch.bfloat16, "gate", dev)
        kinds = {(B, I, J, D): "pair", (B, 1, J, D): "row", (B, I, 1, D): "col"}
        kinds[(B, I, J, D)] = "pair"  # where I or J is 1
        if tuple(gate.shape) not in kinds:
            raise ValueError(f"gate must be one of {list(kinds)}, got {tuple(gate.shape)}")
        kind = kinds[tuple(gate.shape)]
    if mask is not None:
        _need(mask, torch.bfloat16, "mask", dev)
        _shape(mask, (B, I, J), "mask")
    p = _lib.ResidualParams()
    p.D, p.stream_type = D, _type(x.dtype, "x")
    p.post_norm, p.pre_norm = _one_of(_NORMS, post_norm, "post_norm"), _one_of(_NORMS, pre_norm, "pre_norm")
    for k, v in params.items():
        if k not in RESIDUAL_PARAMS:
            raise ValueError(f"unknown parameter {k!r}: {list(RESIDUAL_PARAMS)} are taken")
        _need(v, torch.float32, k, dev)
        _shape(v, (D,), k)
        setattr(p, k, v.data_ptr())
    p.gate, p.gate_sigmoid = _GATES[kind], int(bool(gate_sigmoid))
    p.scale, p.eps = float(scale), float(eps)
    return p, dev, kind


def trimul_residual_forward(x, u, params=None, post_norm=None, pre_norm=None, gate=None, gate_sigmoid=False,
                            mask=None, scale=1.0, eps=1e-5, out=None, normed=None, stream=None, flags: int = 0):
    """(out, normed): out = x + scale mask channel G(gate) Norm_post(u) and normed = Norm_pre(out), None without pre_norm.

    x: bf16 or float32 [B, I, J, D]; u: bf16 alike; params: float32 [D] tensors by name (post_gamma, post_beta,
    pre_gamma, pre_beta, channel), any of them absent; norms: "layer", "rms" or None; gate: bf16 [B, I, J, D],
    [B, 1, J, D] or [B, I, 1, D]; mask: bf16 [B, I, J].  out may be x."""
    p, dev, _ = _residual(x, u, params or {}, post_norm, pre_norm, gate, gate_sigmoid, mask, scale, eps)
    B, I, J, D = x.shape
    with _within(stream):
        out = torch.empty_like(x) if out is None else out
        if normed is None and p.pre_norm:
            normed = torch.empty(x.shape, dtype=torch.bfloat16, device=x.device)
    _need(out, x.dtype, "out", dev)
    _shape(out, x.shape, "out")
    if normed is not None:
        _need(normed, torch.bfloat16, "normed", dev)
        _shape(normed, x.shape, "normed")
    _check(_lib.load().trimul_residual_forward(ctypes.byref(p), _vp(x), _vp(u), _vp(gate), _vp(mask), B, I, J, _vp(out),
                                               _vp(normed), dev, _stream(stream, dev), flags))
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
    B, I, J, D = x.shape
    bf = torch.bfloat16
    for t, name, dt in ((dout, "dout", x.dtype), (dout2, "dout2", x.dtype), (dnormed, "dnormed", bf)):
        if t is not None:
            _need(t, dt, name, dev)
            _shape(t, x.shape, name)
    lib = _lib.load()
    need = lib.trimul_residual_backward_workspace_bytes(ctypes.byref(p), B, I, J)
    with _within(stream):
        dx = torch.empty_like(x) if dx is None else dx
        du = torch.empty_like(u) if du is None else du
        if dgate is None and kind == "pair":
            dgate = torch.empty_like(gate)
        if grads is None:
            grads = {k: torch.empty(D, dtype=torch.float32, device=x.device) for k in params}
        ws = torch.empty(need, dtype=torch.uint8, device=x.device)
    g = _lib.ResidualGrads()
    for k, v in grads.items():
        if k not in RESIDUAL_PARAMS:
            raise ValueError(f"unknown parameter {k!r}: {list(RESIDUAL_PARAMS)} are taken")
        _need(v, torch.float32, k, dev)
        _shape(v, (D,), k)
        setattr(g, k, v.data_ptr())
    for t, name, dt in ((dx, "dx", x.dtype), (du, "du", bf), (dgate, "dgate", bf)):
        if t is not None:
            _need(t, dt, name, dev)
            _shape(t, x.shape, name)
    _check(lib.trimul_residual_backward(ctypes.byref(p), _vp(x), _vp(u), _vp(gate), _vp(mask), _vp(dout), _vp(dout2),
                                        _vp(dnormed), B, I, J, _vp(dx), _vp(du), _vp(dgate), ctypes.byref(g), _vp(ws),
                                        need, dev, _stream(stream, dev), flags))
    return {"dx": dx, "du": du, "dgate": dgate, "grads": grads}


class Residual:
    """A residual step with its parameters: forward(x, u) and backward(x, u, dout)."""

    def __init__(self, params=None, post_norm=None, pre_norm=None, gate_sigmoid=False, scale=1.0, eps=1e-5):
        self.params = dict(params or {})
        self.kw = {"post_norm": post_norm, "pre_norm": pre_norm, "gate_sigmoid": gate_sigmoid, "scale": scale, "eps": eps}

    def forward(self, x, u, **kw):
        return trimul_residual_forward(x, u, self.params, **self.kw, **kw)

    def backward(self, x, u, dout, **kw):
        return trimul_residual_backward(x, u, dout, self.params, **self.kw, **kw)


# ------------------------------------------------------------------ gradient norm and clipping
class GradSet:
    """A list (or dict) of gradients whose norm is taken together: norm() and clip().

    The tensors (and `outs`, buffers of the same shapes and types for clipped copies; default: in place) are kept,
    and read at each call.  bf16, float16 and float32 may be mixed; all on one device, contiguous, not overlapping."""

    def __init__(self, tensors, outs=None):
        tensors = list(tensors.values() if isinstance(tensors, dict) else tensors)
        outs = tensors if outs is None else list(outs.values() if isinstance(outs, dict) else outs)
        if len(outs) != len(tensors):
            raise ValueError(f"{len(outs)} outs for {len(tensors)} tensors")
        self.tensors, self.outs = tensors, outs
        self.device = _cuda(tensors[0], "tensors[0]") if tensors else torch.cuda.current_device()
        self.table = (_lib.GradTensor * len(tensors))()
        for k, (t, o) in enumerate(zip(tensors, outs)):
            kind = _type(t.dtype, f"tensors[{k}]", tuple(_TYPES))
            _need(t, t.dtype, f"tensors[{k}]", self.device)
            if o is not t:
                _need(o, t.dtype, f"outs[{k}]", self.device)
                _shape(o, t.shape, f"outs[{k}]")
            self.table[k] = _lib.GradTensor(t.data_ptr(), o.data_ptr(), t.numel(), kind)
        self.workspace_bytes = _lib.load().trimul_grad_workspace_bytes(len(tensors))

    def _call(self, name, norm_type, norm, stream, flags, *first):
        if norm_type not in (2, math.inf):
            raise ValueError(f"norm_type must be 2 or infinity, got {norm_type}")
        with _within(stream):
            dev = torch.device("cuda", self.device)
            norm = torch.empty((), dtype=torch.float32, device=dev) if norm is None else norm
            ws = torch.empty(self.workspace_bytes, dtype=torch.uint8, device=dev)
        _need(norm, torch.float32, "norm", self.device)
        if norm.numel() != 1:
            raise ValueError("norm must have one element")
        _check(getattr(_lib.load(), name)(self.table, len(self.table), *first, int(norm_type == math.inf), _vp(norm),
                                          _vp(ws), self.workspace_bytes, self.device, _stream(stream, self.device), flags))
        return norm

    def norm(self, norm_type=2.0, norm=None, stream=None, flags: int = 0):
        """The norm, a float32 tensor on the device (the host does not wait for it)."""
        return self._call("trimul_grad_norm", norm_type, norm, stream, flags)

    def clip(self, max_norm, norm_type=2.0, norm=None, stream=None, flags: int = 0):
        """Scale the gradients by min(1, max_norm / (norm + 1e-6)); returns the norm before it.  A norm that is not
        finite leaves them as they are."""
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

    def forward(self, z, mask=None, gate=None, stream=None):
        with _within(stream):
            u = self.layer(z, mask, stream=stream)
        return self.residual.forward(z, u, gate=gate, mask=mask, stream=stream)

    def backward(self, z, dout, mask=None, gate=None, dnormed=None, dout2=None, stream=None):
        """(dx, dz, ...): the gradient of z is dx + dz, its parts along the stream and through the layer.  Give both to
        the block below as dout and dout2: it adds them in 32 bits, in the pass that reads them."""
        with _within(stream):
            u = self.layer(z, mask, stream=stream)
            r = self.residual.backward(z, u, dout, dnormed=dnormed, dout2=dout2, gate=gate, mask=mask, stream=stream)
            dz, grads = _T.trimul_backward(self.layer.handle, z, mask, r["du"], self.layer.direction, stream=stream)
        return {"dx": r["dx"], "dz": dz, "dgate": r["dgate"], "layer_grads": grads, "residual_grads": r["grads"]}
