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
    assert _lib._row(torch.zeros(4, dtype=torch.int32), "cu_seqlens")[1] == 4
    _lib._ints(torch.zeros(2, 3, dtype=torch.int32), "block_table", (2, 3))
    for bad in (torch.zeros(4, dtype=torch.int64), torch.zeros(2, 2, dtype=torch.int32), torch.zeros(8, dtype=torch.int32)[::2],
                torch.zeros((), dtype=torch.int32)):
        with pytest.raises(ValueError, match="cu_seqlens"):
            _lib._row(bad, "cu_seqlens")
    with pytest.raises(ValueError, match="seq_lens"):
        _lib._ints(torch.zeros(4, dtype=torch.int32), "seq_lens", (5,))
    with pytest.raises(ValueError, match="block_table"):
        _lib._ints(torch.zeros(3, dtype=torch.int32), "block_table", (3, 3))


def test_packed_descriptors_are_the_described_ones():
    for t in (torch.zeros(2, 3, 5, 64, dtype=torch.bfloat16), torch.zeros(3, 5, 64, dtype=torch.float16).transpose(0, 1)[None]):
        got = _lib.FfpaTensor.from_buffer_copy(_lib._pack(t))
        assert (got.data, got.dtype, got.reserved) == (t.data_ptr(), _lib._dtype_code(t), 0)
        assert tuple(got.shape) == tuple(t.shape) and tuple(got.stride) == t.stride()
    lse = _lib.FfpaTensor.from_buffer_copy(_lib._pack_lse(torch.zeros(2, 3, 5)))
    assert tuple(lse.shape) == (2, 3, 5, 1) and tuple(lse.stride) == (15, 5, 1, 1)
    assert _lib._pack_lse(None) is None
    with pytest.raises(ValueError, match="4-D"):
        _lib._pack(torch.zeros(2, 3, 64))


# ------------------------------------------------------------------ paged cache

def tree(B=2, Hq=4, Hkv=2, T=3, D=512, page=16, pages=9):
    return {"q": t4([B, Hq, T, D]), "kc": t4([pages, Hkv, page, D]), "vc": t4([pages, Hkv, page, D]), "table": ADDR,
            "max_pages": 4, "lens": ADDR, "drafts": ADDR, "mask": ADDR, "mask_batch": B, "scale": 0.05,
            "out": t4([B, Hq, T, D]), "lse": t4([B, Hq, T, 1], dtype=_lib.FFPA_F32)}


def fwd_tree(lib, a):
    return lib.ffpa_fwd_tree(r(a["q"]), r(a["kc"]), r(a["vc"]), a["table"], a["max_pages"], a["lens"], a["drafts"],
                             a["mask"], a["mask_batch"], a["scale"], r(a["out"]), r(a["lse"]), None)


@pytest.mark.parametrize("name,value,expect", [
    ("table", None, INVALID), ("lens", None, INVALID), ("lens", ADDR + 2, ALIGN), ("drafts", ADDR + 1, ALIGN),
    ("max_pages", 0, INVALID), ("max_pages", 1 << 27, UNSUPPORTED), ("mask_batch", 3, INVALID), ("mask_batch", 0, INVALID),
    ("scale", -1.0, INVALID), ("q", t4([2, 4, 129, 512]), UNSUPPORTED), ("q", t4([2, 5, 3, 512]), INVALID),
    ("q", t4([2, 4, 3, 512], dtype=_lib.FFPA_F32), UNSUPPORTED), ("kc", t4([9, 2, 24, 512]), UNSUPPORTED),
    ("kc", t4([9, 2, 8, 512]), UNSUPPORTED), ("kc", t4([9, 2, 16, 448]), INVALID), ("kc", None, INVALID),
    ("vc", t4([8, 2, 16, 512]), INVALID), ("vc", t4([9, 2, 16, 512], dtype=_lib.FFPA_F16), INVALID),
    ("out", t4([2, 4, 4, 512]), INVALID), ("lse", t4([2, 4, 4, 1], dtype=_lib.FFPA_F32), INVALID),
    ("kc", t4([9, 2, 16, 512], addr=ADDR + 8), ALIGN),
])
def test_tree_rejects(lib, name, value, expect):
    a = tree()
    a[name] = value
    assert fwd_tree(lib, a) == expect


def plan(lib, **over):
    a = dict(lens=ADDR, new=ADDR, n=3, page=16, table=ADDR, per=4, free=ADDR, n_free=5, head=ADDR, cu=ADDR, slots=ADDR,
             max_new=7, lens_out=ADDR, head_out=ADDR)
    a.update(over)
    return lib.ffpa_cache_plan(a["lens"], a["new"], a["n"], a["page"], a["table"], a["per"], a["free"], a["n_free"],
                               a["head"], a["cu"], a["slots"], a["max_new"], a["lens_out"], a["head_out"], None)


@pytest.mark.parametrize("over,expect", [
    (dict(lens=None), INVALID), (dict(new=None), INVALID), (dict(table=None), INVALID), (dict(free=None), INVALID),
    (dict(head=None), INVALID), (dict(cu=None), INVALID), (dict(slots=None), INVALID), (dict(lens_out=None), INVALID),
    (dict(head_out=None), INVALID), (dict(n=0), INVALID), (dict(page=0), INVALID), (dict(per=0), INVALID),
    (dict(n_free=-1), INVALID), (dict(max_new=-1), INVALID), (dict(max_new=(1 << 30) + 1), UNSUPPORTED),
    (dict(slots=ADDR + 4), ALIGN), (dict(lens=ADDR + 2), ALIGN),
])
def test_plan_rejects(lib, over, expect):
    assert plan(lib, **over) == expect


@pytest.mark.parametrize("name,value,expect", [
    ("k", None, INVALID), ("slots", None, INVALID), ("slots", ADDR + 4, ALIGN), ("v", t4([1, 2, 6, 512]), INVALID),
    ("k", t4([2, 2, 5, 512]), INVALID), ("kc", t4([9, 3, 16, 512]), INVALID), ("vc", t4([9, 2, 24, 512]), INVALID),
    ("k", t4([1, 2, 5, 96]), UNSUPPORTED), ("k", t4([1, 2, 5, 512], dtype=_lib.FFPA_F32), UNSUPPORTED),
    ("kc", t4([9, 2, 16, 512], dtype=_lib.FFPA_F16), INVALID), ("v", t4([1, 2, 5, 512], addr=ADDR + 2), ALIGN),
])
def test_append_rejects(lib, name, value, expect):
    a = {"k": t4([1, 2, 5, 512]), "v": t4([1, 2, 5, 512]), "kc": t4([9, 2, 16, 512]), "vc": t4([9, 2, 16, 512]),
         "slots": ADDR}
    a[name] = value
    if name == "k" and value is not None and value.shape[3] == 96:
        a["v"] = value
    assert lib.ffpa_cache_append(r(a["k"]), r(a["v"]), r(a["kc"]), r(a["vc"]), a["slots"], None) == expect
