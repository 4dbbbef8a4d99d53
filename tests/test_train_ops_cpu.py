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


TENSOR = {"param": A, "grad": 2 * A, "m": 3 * A, "v": 4 * A, "m_scale": 5 * A, "v_scale": 6 * A, "numel": 256, "param_type": 1,
          "grad_type": 1}
PARAMS = {"beta1": 0.9, "beta2": 0.999, "eps": 1e-8, "lr": 1e-3, "states": 1}


@pytest.mark.parametrize("tensor,params,call,want,text", [
    ({"numel": -1}, {}, {}, SHAPE, "numel (-1)"),
    ({"numel": 1 << 40}, {}, {}, SHAPE, "too large"),
    ({"param_type": 2}, {}, {}, INVALID, "param_type must be"),
    ({"grad_type": 3}, {}, {}, INVALID, "unknown grad_type 3"),
    ({"copy": 7 * A, "copy_type": 1}, {}, {}, INVALID, "copy_type must be"),
    ({"weight_decay": -0.1}, {}, {}, INVALID, "weight_decay"),
    ({"weight_decay": float("nan")}, {}, {}, INVALID, "weight_decay"),
    ({"param": None}, {}, {}, INVALID, "param is null"),
    ({"param": A + 2}, {}, {}, INVALID, "param is null or not aligned"),
    ({"grad": None}, {}, {}, INVALID, "grad is null"),
    ({"grad": 2 * A + 1, "grad_type": 0}, {}, {}, INVALID, "grad is null or not aligned"),
    ({"copy": 7 * A + 1}, {}, {}, INVALID, "copy is not aligned"),
    ({"m": 3 * A + 8}, {}, {}, INVALID, "m or v is null"),
    ({"v": None}, {}, {}, INVALID, "m or v is null"),
    ({"m_scale": None}, {}, {}, INVALID, "m_scale or v_scale is null"),
    ({"v_scale": 6 * A + 2}, {}, {}, INVALID, "m_scale or v_scale is null"),
    ({"grad": A + 512}, {}, {}, INVALID, "param overlaps grad"),
    ({"v": 3 * A + 128}, {}, {}, INVALID, "m overlaps v"),
    ({"v_scale": 5 * A + 4}, {}, {}, INVALID, "m_scale overlaps v_scale"),
    ({"copy": A + 1000}, {}, {}, INVALID, "param overlaps copy"),
    ({"m": 8 * A}, {}, {}, INVALID, "m overlaps count"),
    ({}, {"norm": A + 4}, {}, INVALID, "param overlaps norm"),
    ({}, {"lr_device": 4 * A}, {}, INVALID, "v overlaps lr_device"),
    ({}, {"norm": 8 * A + 4}, {}, INVALID, "count overlaps"),
    ({"grad": 8 * A}, {}, {}, INVALID, "count overlaps grad"),
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
    c = {"n": 1, "count": 8 * A, "flags": 0, **call}
    refused(lib, lib.trimul_adamw_step(ctypes.byref(p), t, c["n"], c["count"], 0, None, c["flags"]), want, text)


def test_adamw_null_arguments(lib):
    p = _lib.AdamwParams(**PARAMS)
    refused(lib, lib.trimul_adamw_step(None, None, 0, A, 0, None, 0), INVALID, "params is null")
    refused(lib, lib.trimul_adamw_step(ctypes.byref(p), None, 1, A, 0, None, 0), INVALID, "tensors is null")


def test_binding_refusals():
    with pytest.raises(ValueError, match="CUDA device"):
        P.AdamW([torch.zeros(8)])
    with pytest.raises(ValueError, match="2 copies for 1 params"):
        P.AdamW([torch.zeros(8)], copies=[None, None])
