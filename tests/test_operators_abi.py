"""Host-side refusals of the packed and paged entry points (no GPU needed).

As in test_abi.py: fake, aligned device addresses; nothing is dereferenced and
nothing launched before validation passes.
"""
import ctypes

import pytest
import torch

from head_dim_attention_gb300 import _lib
from test_abi import ADDR, ALIGN, INVALID, UNSUPPORTED, t4

r = lambda x: None if x is None else ctypes.byref(x)  # noqa: E731


def packed(T=300, Hq=4, Hkv=2, D=512):
    return {"q": t4([1, Hq, T, D]), "k": t4([1, Hkv, T, D]), "v": t4([1, Hkv, T, D]), "out": t4([1, Hq, T, D]),
            "lse": t4([1, Hq, T, 1], dtype=_lib.FFPA_F32), "dout": t4([1, Hq, T, D]), "dq": t4([1, Hq, T, D]),
            "dk": t4([1, Hkv, T, D]), "dv": t4([1, Hkv, T, D]), "cu": ADDR, "n": 3, "causal": 1, "scale": 0.05}


def varlen_fwd(lib, a):
    return lib.ffpa_fwd_varlen(r(a["q"]), r(a["k"]), r(a["v"]), a["cu"], a["n"], a["causal"], a["scale"], r(a["out"]),
                               r(a["lse"]), None)


def varlen_bwd(lib, a):
    return lib.ffpa_bwd_varlen(r(a["q"]), r(a["k"]), r(a["v"]), a["cu"], a["n"], a["causal"], a["scale"], r(a["out"]),
                               r(a["lse"]), r(a["dout"]), r(a["dq"]), r(a["dk"]), r(a["dv"]), None)


VARLEN = [
    ("cu", None, INVALID), ("cu", ADDR + 2, ALIGN), ("n", 0, INVALID), ("n", -1, INVALID), ("n", (1 << 20) + 1, UNSUPPORTED),
    ("causal", 2, INVALID), ("scale", 0.0, INVALID), ("scale", float("inf"), INVALID), ("q", None, INVALID),
    ("k", t4([1, 2, 301, 512]), INVALID), ("v", t4([1, 2, 299, 512]), INVALID), ("q", t4([2, 4, 300, 512]), INVALID),
    ("out", t4([1, 4, 301, 512]), INVALID), ("out", None, INVALID), ("lse", t4([1, 4, 300, 1]), UNSUPPORTED),
    ("lse", t4([1, 4, 299, 1], dtype=_lib.FFPA_F32), INVALID), ("q", t4([1, 4, 300, 512], addr=ADDR + 2), ALIGN),
    ("k", t4([1, 3, 300, 512]), INVALID),
]


@pytest.mark.parametrize("name,value,expect", VARLEN)
def test_varlen_rejects(lib, name, value, expect):
    a = packed()
    a[name] = value
    if name in ("q",) and value is not None and value.shape[0] == 2:
        a["k"], a["v"], a["out"] = t4([2, 2, 300, 512]), t4([2, 2, 300, 512]), t4([2, 4, 300, 512])
    if name == "k" and value.shape[1] == 3:
        a["v"] = value
    if name in ("k",) and value.shape[2] != 300:
        a["v"] = value  # as many values as keys, but not as queries
    assert varlen_fwd(lib, a) == expect
    assert varlen_bwd(lib, a) == expect


def test_varlen_keys_must_match_queries(lib):
    a = packed()
    a["k"], a["v"] = t4([1, 2, 200, 512]), t4([1, 2, 200, 512])
    a["dk"], a["dv"] = a["k"], a["v"]
    assert varlen_fwd(lib, a) == INVALID
    assert varlen_bwd(lib, a) == INVALID


@pytest.mark.parametrize("D", [96, 1088, 0])
def test_varlen_head_dims(lib, D):
    assert varlen_fwd(lib, packed(D=max(D, 1))) == UNSUPPORTED


@pytest.mark.parametrize("name", ["lse", "dout", "dq", "dk", "dv"])
def test_varlen_bwd_needs_everything(lib, name):
    a = packed()
    a[name] = None
    assert varlen_bwd(lib, a) == INVALID


def test_binding_checks_integer_tensors():
    ok = torch.zeros(4, dtype=torch.int32)
    _lib._ints(ok, "cu_seqlens", 1)
    for bad in (torch.zeros(4, dtype=torch.int64), torch.zeros(2, 2, dtype=torch.int32), torch.zeros(8, dtype=torch.int32)[::2]):
        with pytest.raises(ValueError, match="cu_seqlens"):
            _lib._ints(bad, "cu_seqlens", 1)
