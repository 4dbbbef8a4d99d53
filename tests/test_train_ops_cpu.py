"""CPU-only checks of AdamW's entry point: bad arguments are refused, with a message, before any device is touched."""

import ctypes

import pytest
import torch

from co_folding_pair_gb300 import _lib
from co_folding_pair_gb300 import train_ops as P

INVALID, SHAPE = 1, 2
A = 1 << 20  # addresses that are only looked at; 1 MB apart


def refused(lib, status, want, text):
    assert status == want, lib.trimul_last_error()
    assert text in lib.trimul_last_error().decode()


TENSOR = {"param": A, "m": 3 * A, "v": 4 * A, "m_scale": 5 * A, "v_scale": 6 * A, "numel": 256, "param_type": 1}
GRAD = {"data": 2 * A, "numel": 256, "type": 1}
PARAMS = {"beta1": 0.9, "beta2": 0.999, "eps": 1e-8, "lr": 1e-3, "states": 1}


@pytest.mark.parametrize("tensor,params,call,want,text", [
    ({"numel": -1}, {}, {"grad": {"numel": -1}}, SHAPE, "numel (-1)"),
    ({"numel": 1 << 40}, {}, {"grad": {"numel": 1 << 40}}, SHAPE, "too large"),
    ({"param_type": 2}, {}, {}, INVALID, "param_type must be"),
    ({}, {}, {"grad": {"type": 3}}, INVALID, "unknown type 3 of its gradient"),
    ({}, {}, {"grad": {"numel": 255}}, SHAPE, "its gradient has 255 elements, not 256"),
    ({"copy": 7 * A, "copy_type": 1}, {}, {}, INVALID, "copy_type must be"),
    ({"weight_decay": -0.1}, {}, {}, INVALID, "weight_decay"),
    ({"weight_decay": float("nan")}, {}, {}, INVALID, "weight_decay"),
    ({"param": None}, {}, {}, INVALID, "param is null"),
    ({"param": A + 2}, {}, {}, INVALID, "param is null or not aligned"),
    ({}, {}, {"grad": {"data": None}}, INVALID, "grad is null"),
    ({}, {}, {"grad": {"data": 2 * A + 1, "type": 0}}, INVALID, "grad is null or not aligned"),
    ({"copy": 7 * A + 1}, {}, {}, INVALID, "copy is not aligned"),
    ({"m": 3 * A + 8}, {}, {}, INVALID, "m or v is null"),
    ({"v": None}, {}, {}, INVALID, "m or v is null"),
    ({"m_scale": None}, {}, {}, INVALID, "m_scale or v_scale is null"),
    ({"v_scale": 6 * A + 2}, {}, {}, INVALID, "m_scale or v_scale is null"),
    ({}, {}, {"grad": {"data": A + 512}}, INVALID, "param overlaps grad"),
    ({"v": 3 * A + 128}, {}, {}, INVALID, "m overlaps v"),
    ({"v_scale": 5 * A + 4}, {}, {}, INVALID, "m_scale overlaps v_scale"),
    ({"copy": A + 1000}, {}, {}, INVALID, "param overlaps copy"),
    ({"m": 8 * A}, {}, {}, INVALID, "m overlaps count"),
    ({}, {"norm": A + 4}, {}, INVALID, "param overlaps norm"),
    ({}, {"lr_device": 4 * A}, {}, INVALID, "v overlaps lr_device"),
    ({}, {"norm": 8 * A + 4}, {}, INVALID, "count overlaps"),
    ({}, {}, {"grad": {"data": 8 * A}}, INVALID, "count overlaps grad"),
    ({}, {"beta1": 1.0}, {}, INVALID, "beta1"),
    ({}, {"beta2": -0.1}, {}, INVALID, "beta1"),
    ({}, {"beta2": float("nan")}, {}, INVALID, "beta1"),
    ({}, {"eps": 0.0}, {}, INVALID, "eps"),
    ({}, {"eps": 1e-40}, {}, INVALID, "eps"),
    ({}, {"lr": float("inf")}, {}, INVALID, "lr must be"),
    ({}, {"norm": 9 * A, "max_norm": float("nan")}, {}, INVALID, "max_norm"),
    ({}, {"states": 2}, {}, INVALID, "unknown states 2"),
    ({}, {"rounding": 2}, {}, INVALID, "unknown rounding 2"),
    ({}, {}, {"n": -1}, INVALID, "n (-1)"),
    ({}, {}, {"count": None}, INVALID, "count is null"),
    ({}, {}, {"count": 8 * A + 2}, INVALID, "count is null"),
    ({}, {}, {"flags": 16}, INVALID, "flags 0x10"),
])
def test_adamw_refused(lib, tensor, params, call, want, text):
    t = (_lib.AdamwTensor * 1)(_lib.AdamwTensor(**{**TENSOR, **tensor}))
    p = _lib.AdamwParams(**{**PARAMS, **params})
    c = {"n": 1, "count": 8 * A, "flags": 0, "grad": {}, **call}
    g = (_lib.GradTensor * 1)(_lib.GradTensor(**{**GRAD, **c["grad"]}))
    refused(lib, lib.trimul_adamw_step(ctypes.byref(p), t, g, c["n"], c["count"], 0, None, c["flags"]), want, text)


def test_adamw_null_arguments(lib):
    p = _lib.AdamwParams(**PARAMS)
    refused(lib, lib.trimul_adamw_step(None, None, None, 0, A, 0, None, 0), INVALID, "params is null")
    refused(lib, lib.trimul_adamw_step(ctypes.byref(p), None, None, 1, A, 0, None, 0), INVALID, "tensors or grads is null")


def test_binding_refusals():
    with pytest.raises(ValueError, match="CUDA device"):
        P.AdamW([torch.zeros(8)])
    with pytest.raises(ValueError, match="2 copies for 1 params"):
        P.AdamW([torch.zeros(8)], copies=[None, None])


FWD = {"packed": A, "bias": None, "x": 2 * A, "rows": 64, "N": 128, "K": 128, "y": 3 * A, "ws": 4 * A, "bytes": A, "flags": 0}


@pytest.mark.parametrize("call,want,text", [
    ({"N": 12}, SHAPE, "N (12)"),
    ({"K": 0}, SHAPE, "K (0)"),
    ({"K": 65544}, SHAPE, "K (65544)"),
    ({"rows": -1}, SHAPE, "rows (-1)"),
    ({"rows": 1 << 31}, SHAPE, "rows (2147483648)"),
    ({"packed": None}, INVALID, "packed is null"),
    ({"packed": A + 16}, INVALID, "256-byte aligned"),
    ({"bias": 5 * A + 4}, INVALID, "bias must be"),
    ({"x": None}, INVALID, "x or y is null"),
    ({"x": 2 * A + 2}, INVALID, "not 16-byte aligned"),
    ({"y": 3 * A + 8}, INVALID, "not 16-byte aligned"),
    ({"y": 2 * A}, INVALID, "y overlaps x"),
    ({"y": A + 256}, INVALID, "y overlaps packed"),
    ({"ws": 3 * A + 1024}, INVALID, "workspace overlaps y"),
    ({"bias": 4 * A}, INVALID, "workspace overlaps bias"),
    ({"bias": 3 * A + 64}, INVALID, "y overlaps bias"),
    ({"bytes": 100}, INVALID, "are needed"),
    ({"ws": None}, INVALID, "are needed"),
    ({"ws": 4 * A + 16}, INVALID, "256-byte aligned"),
    ({"N": 2048, "bytes": 4096}, INVALID, "are needed"),
    ({"flags": 16}, INVALID, "flags 0x10"),
])
def test_linear8_forward_refused(lib, call, want, text):
    a = {**FWD, **call}
    refused(lib, lib.trimul_linear8_forward(a["packed"], a["bias"], a["x"], a["rows"], a["N"], a["K"], a["y"], a["ws"], a["bytes"], 0,
                                            None, a["flags"]), want, text)


BWD = {**FWD, "dy": 5 * A, "dx": 6 * A, "dw": 7 * A, "db": 8 * A, "bytes": 1 << 30, "ws": 16 * A}


@pytest.mark.parametrize("call,want,text", [
    ({"N": 4}, SHAPE, "N (4)"),
    ({"dy": None}, INVALID, "x or dy is null"),
    ({"dx": 6 * A + 8}, INVALID, "not 16-byte aligned"),
    ({"dw": 7 * A + 4}, INVALID, "dW and dbias must be"),
    ({"db": 8 * A + 4}, INVALID, "dW and dbias must be"),
    ({"dx": 5 * A}, INVALID, "dx overlaps dy"),
    ({"dw": 2 * A}, INVALID, "dW overlaps x"),
    ({"db": 7 * A + 64}, INVALID, "dbias overlaps dW"),
    ({"ws": 8 * A}, INVALID, "workspace overlaps dbias"),
    ({"bytes": 100}, INVALID, "are needed"),
    ({"flags": 4}, INVALID, "flags 0x4"),
])
def test_linear8_backward_refused(lib, call, want, text):
    a = {**BWD, **call}
    refused(lib, lib.trimul_linear8_backward(a["packed"], a["x"], a["dy"], a["rows"], a["N"], a["K"], a["dx"], a["dw"], a["db"], a["ws"],
                                             a["bytes"], 0, None, a["flags"]), want, text)


@pytest.mark.parametrize("call,want,text", [
    ({"type": 2}, INVALID, "type must be"),
    ({"W": None}, INVALID, "W is null"),
    ({"W": A + 2}, INVALID, "W is null or not aligned"),
    ({"packed": 2 * A + 16}, INVALID, "256-byte aligned"),
    ({"bytes": 100}, INVALID, "are needed"),
    ({"packed": A + 256}, INVALID, "packed overlaps W"),
    ({"N": 20}, SHAPE, "N (20)"),
])
def test_linear8_pack_refused(lib, call, want, text):
    a = {"W": A, "type": 1, "N": 128, "K": 128, "packed": 2 * A, "bytes": A, **call}
    refused(lib, lib.trimul_linear8_pack(a["W"], a["type"], a["N"], a["K"], a["packed"], a["bytes"], 0, None, 0), want, text)


def test_linear8_sizes(lib):
    assert lib.trimul_linear8_packed_bytes(12, 8) == 0
    assert lib.trimul_linear8_forward_workspace_bytes(-1, 8, 8) == 0
    assert lib.trimul_linear8_backward_workspace_bytes(8, 8, 7) == 0
    # a wide layer has tiles enough for every pair of processors: dW is summed where it is wanted, not in slices
    assert lib.trimul_linear8_backward_workspace_bytes(128, 16384, 16384) < 64 << 20
    # codes [N][K] in rows of whole 16 bytes, and the tiles of scales for both of its uses
    assert lib.trimul_linear8_packed_bytes(128, 24) == 128 * 32 + 512 + 512


@pytest.mark.parametrize("N,K", [(8, 8), (264, 136), (256, 1024), (65536, 65536)])
def test_linear8_workspaces_of_no_rows(lib, N, K):
    """Asked for before each call, one of no rows among them, which needs no more than the smallest one with rows."""
    assert 0 < lib.trimul_linear8_forward_workspace_bytes(0, N, K) <= lib.trimul_linear8_forward_workspace_bytes(1, N, K)
    assert 0 < lib.trimul_linear8_backward_workspace_bytes(0, N, K) <= lib.trimul_linear8_backward_workspace_bytes(1, N, K)


def test_no_copy_is_sent_to_several_processors():
    """The library also runs on machines with several GPUs, where a load that a cluster shares may be closed: each block of threads
    loads what it reads."""
    import os
    import re
    for f in sorted(os.listdir(_lib.CSRC)):
        text = re.sub(r'"\s*\n\s*"', "", open(os.path.join(_lib.CSRC, f)).read())
        assert not re.search(r"cp\.async[\w.:]*multi" + "cast", text), f


def test_dicts_go_by_the_parameters_names():
    assert P._listed({"b": 2, "a": 1}, 2, "copies", ["a", "b"]) == [1, 2]
    assert P._listed({"b": 2, "a": 1}, 2, "copies") == P._listed({"b": 2, "a": 1}, 2, "copies", ["x", "y"]) == [2, 1]
    assert P._listed(0.1, 2, "weight_decay", ["a", "b"]) == [0.1, 0.1]
    with pytest.raises(ValueError, match="1 copies for 2 params"):
        P._listed({"a": 1}, 2, "copies", ["a", "b"])
