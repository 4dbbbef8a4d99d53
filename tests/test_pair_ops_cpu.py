"""CPU-only checks of the operators around the layer: bad arguments are refused,
with a message, before any device is touched."""

import ctypes

import pytest
import torch

from co_folding_pair_gb300 import _lib
from co_folding_pair_gb300 import pair_ops as P

INVALID, SHAPE = 1, 2
A = 1 << 20  # addresses that are only looked at; 1 MB apart


def refused(lib, status, want, text):
    assert status == want, lib.trimul_last_error()
    assert text in lib.trimul_last_error().decode()


@pytest.mark.parametrize("fields,want,text", [
    ((0, 0, 0, 1, 0), SHAPE, "max_distance (0)"),
    ((0, 40000, 0, 1, 0), SHAPE, "max_distance (40000)"),
    ((0, 32, 64, 1, 0), SHAPE, "must be 0 or 65"),
    ((0, 512, 0, 1, 0), SHAPE, "1025 buckets"),
    ((0, 1023, 0, 0, 1), SHAPE, "1024 buckets"),
    ((1, 128, 31, 1, 0), SHAPE, "must be even"),
    ((1, 128, 2, 1, 0), SHAPE, "at least 2"),
    ((1, 8, 32, 1, 0), SHAPE, "max_distance > 8"),
    ((1, 128, 0, 0, 0), SHAPE, "0 buckets"),
    ((2, 128, 32, 1, 0), INVALID, "unknown bucket kind 2"),
])
def test_relpos_plans_refused(lib, fields, want, text):
    r = ctypes.c_void_p(7)
    p = _lib.RelposParams(*fields)
    refused(lib, lib.trimul_relpos_create(ctypes.byref(r), ctypes.byref(p), 0), want, text)
    assert not r.value


def test_null_plans(lib):
    r = ctypes.c_void_p()
    assert lib.trimul_relpos_create(None, None, 0) == INVALID
    assert lib.trimul_relpos_create(ctypes.byref(r), None, 0) == INVALID
    assert lib.trimul_relpos_rows(None) == -1
    assert lib.trimul_relpos_forward(None, A, 0, A, A, None, None, None, 1, 8, 8, 8, 0, A, 0, None, 0) == INVALID
    assert lib.trimul_relpos_backward(None, A, 0, A, A, None, None, 1, 8, 8, 8, 0, A, A, 1 << 30, None, 0) == INVALID
    assert lib.trimul_relpos_backward_workspace_bytes(None, 1, 8, 8, 8, 0, 0) == 0
    assert lib.trimul_relpos_destroy(None) == 0


def _params(**kw):
    p = _lib.ResidualParams(D=32, stream_type=0, post_norm=1, pre_norm=1, scale=1.0, eps=1e-5)
    for k, v in kw.items():
        setattr(p, k, v)
    return p


FWD = {"x": A, "u": 2 * A, "gate": None, "mask": None, "B": 1, "I": 8, "J": 8, "out": 3 * A, "normed": 4 * A, "flags": 0}


def forward(lib, p, **kw):
    a = {**FWD, **kw}
    return lib.trimul_residual_forward(None if p is None else ctypes.byref(p), a["x"], a["u"], a["gate"], a["mask"],
                                       a["B"], a["I"], a["J"], a["out"], a["normed"], 0, None, a["flags"])


@pytest.mark.parametrize("fields,call,want,text", [
    ({"D": 12}, {}, SHAPE, "D (12)"),
    ({"D": 264}, {}, SHAPE, "D (264)"),
    ({}, {"B": 0}, SHAPE, "must be >= 1"),
    ({}, {"I": 50000, "J": 50000}, SHAPE, "2^31 pairs"),
    ({"stream_type": 2}, {}, INVALID, "stream_type"),
    ({"eps": 0.0}, {}, INVALID, "eps"),
    ({"eps": 1e-40}, {}, INVALID, "eps"),
    ({"eps": -1e-5}, {}, INVALID, "eps"),
    ({"scale": float("inf")}, {}, INVALID, "scale"),
    ({"post_norm": 3}, {}, INVALID, "unknown post_norm"),
    ({"post_norm": 0, "post_gamma": 5 * A}, {}, INVALID, "post_norm is NONE"),
    ({"pre_norm": 2, "pre_beta": 5 * A}, {}, INVALID, "pre_norm is not LAYER"),
    ({"pre_gamma": 5 * A + 4}, {}, INVALID, "16-byte aligned"),
    ({"gate": 4}, {"gate": 5 * A}, INVALID, "unknown gate"),
    ({"gate": 1}, {}, INVALID, "do not agree"),
    ({}, {"gate": 5 * A}, INVALID, "do not agree"),
    ({}, {"normed": None}, INVALID, "normed and pre_norm"),
    ({"pre_norm": 0}, {}, INVALID, "normed and pre_norm"),
    ({}, {"x": None}, INVALID, "is null"),
    ({}, {"u": 2 * A + 8}, INVALID, "16-byte aligned"),
    ({}, {"out": A + 64}, INVALID, "out overlaps x"),
    ({}, {"out": 2 * A}, INVALID, "out overlaps u"),
    ({}, {"normed": A}, INVALID, "normed overlaps x"),
    ({}, {"normed": 3 * A}, INVALID, "normed overlaps out"),
    ({"channel": 3 * A + 128}, {}, INVALID, "out overlaps channel"),
    ({}, {"flags": 8}, INVALID, "flags 0x8"),
])
def test_residual_forward_refused(lib, fields, call, want, text):
    refused(lib, forward(lib, _params(**fields), **call), want, text)


def test_residual_null_params(lib):
    assert forward(lib, None) == INVALID
    assert lib.trimul_residual_backward_workspace_bytes(None, 1, 8, 8) == 0
    assert lib.trimul_residual_backward_workspace_bytes(ctypes.byref(_params(D=4)), 1, 8, 8) == 0


BWD = {**FWD, "dout": 5 * A, "dout2": None, "dnormed": 6 * A, "dx": 7 * A, "du": 8 * A, "dgate": None, "ws": 9 * A,
       "bytes": A}


@pytest.mark.parametrize("fields,call,grads,text", [
    ({}, {"dout": None}, {}, "is null"),
    ({}, {"dnormed": None}, {}, "dnormed and pre_norm"),
    ({}, {"dgate": 10 * A}, {}, "only a gate of every pair"),
    ({"gate": 2}, {"gate": 11 * A, "dgate": 10 * A}, {}, "only a gate of every pair"),
    ({}, {"dx": A}, {}, "dx overlaps x"),
    ({}, {"dx": 5 * A + 16}, {}, "dx overlaps dout"),
    ({}, {"du": 5 * A}, {}, "du overlaps dout"),
    ({}, {"dout2": 5 * A + 8}, {}, "16-byte aligned"),
    ({}, {"bytes": 16}, {}, "are needed"),
    ({}, {"ws": None}, {}, "are needed"),
    ({}, {"ws": 9 * A + 4}, {}, "16-byte aligned"),
    ({"post_norm": 0}, {}, {"post_gamma": 12 * A}, "no post_gamma"),
    ({"pre_norm": 2}, {}, {"pre_beta": 12 * A}, "no pre_beta"),
    ({}, {}, {"pre_beta": 12 * A + 2}, "4-byte aligned"),
    ({}, {}, {"pre_beta": 12 * A, "pre_gamma": 12 * A + 64}, "overlaps the gradient of pre_gamma"),
    ({}, {"flags": 16}, {}, "flags 0x10"),
])
def test_residual_backward_refused(lib, fields, call, grads, text):
    a, p, g = {**BWD, **call}, _params(**fields), _lib.ResidualGrads(**grads)
    st = lib.trimul_residual_backward(ctypes.byref(p), a["x"], a["u"], a["gate"], a["mask"], a["dout"], a["dout2"],
                                      a["dnormed"], a["B"], a["I"], a["J"], a["dx"], a["du"], a["dgate"],
                                      ctypes.byref(g), a["ws"], a["bytes"], 0, None, a["flags"])
    refused(lib, st, INVALID, text)


@pytest.mark.parametrize("entry,call,want,text", [
    ((A, A, -1, 1), {}, SHAPE, "numel (-1)"),
    ((A, A, 1 << 43, 1), {}, SHAPE, "too large"),
    ((A, A, 8, 3), {}, INVALID, "unknown type"),
    ((None, A, 8, 1), {}, INVALID, "data is null"),
    ((A + 2, A, 8, 1), {}, INVALID, "not aligned to its type"),
    ((A, None, 8, 1), {}, INVALID, "out is null"),
    ((A, A + 1, 8, 0), {}, INVALID, "out is null or not aligned"),
    ((A, A + 16, 8, 1), {}, INVALID, "out overlaps data"),
    ((A, A, 8, 1), {"max": -1.0}, INVALID, "max_norm"),
    ((A, A, 8, 1), {"max": float("nan")}, INVALID, "max_norm"),
    ((A, A, 8, 1), {"kind": 2}, INVALID, "unknown norm"),
    ((A, A, 8, 1), {"norm": None}, INVALID, "norm is null"),
    ((A, A, 8, 1), {"bytes": 8}, INVALID, "are needed"),
    ((A, A, A, 1), {"norm": A + 64}, INVALID, "overlaps norm"),
    ((A, 4 * A, 8, 1), {"norm": 4 * A + 16}, INVALID, "overlaps norm"),
    ((A, 5 * A, 8, 1), {}, INVALID, "overlaps norm or the workspace"),
    ((A, A, 8, 1), {"norm": 5 * A + 32}, INVALID, "norm overlaps"),
    ((A, A, 8, 1), {"n": -1}, INVALID, "n (-1)"),
    ((A, A, 8, 1), {"flags": 2}, INVALID, "flags 0x2"),
])
def test_grad_clip_refused(lib, entry, call, want, text):
    a = {"n": 1, "max": 1.0, "kind": 0, "norm": 4 * A, "ws": 5 * A, "bytes": A, "flags": 0, **call}
    t = (_lib.GradTensor * 1)(_lib.GradTensor(*entry))
    refused(lib, lib.trimul_grad_clip(t, a["n"], a["max"], a["kind"], a["norm"], a["ws"], a["bytes"], 0, None, a["flags"]),
            want, text)
    assert lib.trimul_grad_norm(None, 1, 0, 4 * A, 5 * A, A, 0, None, 0) == INVALID
    assert lib.trimul_grad_workspace_bytes(-1) == 0


def test_binding_refusals():
    x = torch.zeros(1, 2, 2, 8, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA device"):
        P.trimul_residual_forward(x, x)
    with pytest.raises(ValueError, match="CUDA device"):
        P.trimul_grad_norm([x])
    with pytest.raises(TypeError, match="tensors"):
        P._type(torch.float64, "tensors[0]")
    with pytest.raises(ValueError, match="kind must be one of"):
        P.trimul_relpos_create("cubic")
    with pytest.raises(ValueError, match="post_norm must be one of"):
        P._one_of(P._NORMS, "batch", "post_norm")


@pytest.mark.parametrize("device", ["cpu", "meta"])
def test_plans_are_on_cuda_devices(device):
    with pytest.raises(ValueError, match="CUDA device"):
        P._device(device)
    assert P._device("cuda:3") == 3


@pytest.mark.parametrize("data,out,size,want", [
    ([100, 200, 300], [100, 200, 300], [100, 100, 50], None),         # in place, end to end
    ([300, 100, 200], [300, 100, 200], [50, 100, 100], None),         # in any order
    ([100, 100], [100, 100], [64, 64], (0, 1)),                       # one tensor twice
    ([100, 150], [100, 150], [64, 8], (0, 1)),                        # a part of it
    ([100, 100], [100, 100], [64, 0], None),                          # nothing of it
    ([100, 200], [500, 564], [64, 64], None),                         # out of place
    ([100, 100], [500, 564], [64, 64], None),                         # read twice, written apart
    ([100, 200], [200, 500], [64, 64], (1, 0)),                       # an output over another tensor
    ([100, 200], [500, 140], [64, 64], (0, 1)),
    ([100, 200], [100, 150], [64, 64], (0, 1)),
    ([100, 200], [100, 220], [64, 64], (1, 1)),                       # partly over its own
    ([], [], [], None),
    ([100], [100], [0], None),
])
def test_clipped_tensors_are_apart(data, out, size, want):
    import numpy as np
    assert P._shared(*[np.array(v, dtype=np.int64) for v in (data, out, size)]) == want
