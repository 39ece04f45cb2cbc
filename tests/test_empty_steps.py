"""A step that brings nothing: no packed rows, no drafts, no new tokens.

The calls are checked as any other and do nothing.  No GPU is needed for the C
entry points: nothing is launched, and tensors without rows have null pointers,
as torch gives them.
"""
import pytest
import torch

from head_dim_attention_gb300 import _lib
from test_abi import ADDR, INVALID, UNSUPPORTED, t4
from test_operators_abi import fwd_tree, packed, plan, r, tree, varlen_bwd, varlen_fwd

ROWS = ("q", "k", "v", "out", "lse", "dout", "dq", "dk", "dv")


def without_rows():
    a = packed(T=0)
    for name in ROWS:
        a[name].data = None
    return a


def append(lib, T=0, slots=None, **over):
    k = t4([1, 2, T, 512])
    a = {"k": k, "v": k, "kc": t4([9, 2, 16, 512]), "vc": t4([9, 2, 16, 512])}
    if T == 0:
        k.data = None
    a.update(over)
    return lib.ffpa_cache_append(r(a["k"]), r(a["v"]), r(a["kc"]), r(a["vc"]), slots, None)


def test_packed_calls_without_rows(lib):
    assert varlen_fwd(lib, without_rows()) == 0
    assert varlen_bwd(lib, without_rows()) == 0
    a = without_rows()
    a["lse"] = None
    assert varlen_fwd(lib, a) == 0
    # what torch makes of an empty lse: strides of 1
    a["lse"] = t4([1, 4, 0, 1], dtype=_lib.FFPA_F32, stride=[4, 1, 1, 1])
    assert varlen_fwd(lib, a) == 0


@pytest.mark.parametrize("name,value,expect", [
    ("cu", None, INVALID), ("n", 0, INVALID), ("causal", 2, INVALID), ("scale", 0.0, INVALID),
    ("k", t4([1, 2, 1, 512]), INVALID), ("out", t4([1, 4, 1, 512]), INVALID), ("q", t4([1, 4, -1, 512]), INVALID),
    ("q", t4([1, 4, 0, 96]), UNSUPPORTED), ("out", None, INVALID),
])
def test_packed_calls_without_rows_are_checked(lib, name, value, expect):
    a = without_rows()
    a[name] = value
    assert varlen_fwd(lib, a) == expect
    assert varlen_bwd(lib, a) == expect


def test_unpacked_calls_still_need_rows(lib):
    a = without_rows()
    assert lib.ffpa_fwd(r(a["q"]), r(a["k"]), r(a["v"]), None, 1, 0.05, r(a["out"]), r(a["lse"]), None) == INVALID


def test_no_drafts(lib):
    a = tree(T=0)
    for name in ("q", "out", "lse"):
        a[name].data = None
    assert fwd_tree(lib, a) == 0
    a["lens"] = None
    assert fwd_tree(lib, a) == INVALID
    a = tree(T=3)
    a["q"].data = None
    assert fwd_tree(lib, a) == INVALID


def test_no_new_tokens(lib):
    assert append(lib) == 0
    assert append(lib, kc=t4([9, 2, 24, 512])) == UNSUPPORTED
    assert append(lib, T=5, slots=None) == INVALID
    k = t4([1, 2, 5, 512])
    k.data = None
    assert append(lib, T=5, slots=ADDR, k=k) == INVALID
    assert plan(lib, max_new=-1) == INVALID


@pytest.mark.gpu
def test_a_serving_step_without_new_tokens():
    from head_dim_attention_gb300 import attention_tree_fwd, attention_varlen_bwd, attention_varlen_fwd, cache_append, \
        cache_plan, ffpa_check_status
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    kw = dict(dtype=torch.bfloat16, device="cuda")
    table, lens = torch.arange(6, dtype=torch.int32, device="cuda").view(2, 3), i32([20, 33])
    before = table.clone()
    cu, slots, after, head = cache_plan(lens, i32([0, 0]), table, i32([7]), i32([0]), 16, 0)
    k, v = torch.empty(0, 2, 512, **kw).transpose(0, 1)[None], torch.empty(1, 2, 0, 512, **kw)
    kc, vc = (torch.randn(8, 2, 16, 512, **kw) for _ in range(2))
    kept = kc.clone(), vc.clone()
    cache_append(k, v, kc, vc, slots)
    q = torch.empty(1, 4, 0, 512, **kw)
    out, lse = attention_varlen_fwd(q, k, v, cu, causal=True)
    grads = attention_varlen_bwd(q, k, v, cu, out, lse, torch.empty_like(q), causal=True)
    none, _ = attention_tree_fwd(torch.empty(2, 4, 0, 512, **kw), kc, vc, table, lens)
    left = torch.full((2, 4, 3, 512), 7.0, **kw)
    attention_tree_fwd(torch.randn(2, 4, 3, 512, **kw), kc, vc, table, lens, draft_lens=i32([0, 0]), out=left)
    torch.cuda.synchronize()
    assert ffpa_check_status() == 0
    assert cu.tolist() == [0, 0, 0] and slots.numel() == 0 and after.tolist() == [20, 33] and head.tolist() == [0]
    assert torch.equal(table, before) and torch.equal(kc, kept[0]) and torch.equal(vc, kept[1])
    assert out.shape == (1, 4, 0, 512) and none.shape == (2, 4, 0, 512) and bool((left == 7.0).all())
    assert [x.shape[2] for x in grads] == [0, 0, 0]
