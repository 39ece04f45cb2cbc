"""The measurement hook with the packed and paged calls: an event before the first launch and one after each."""
import pytest
import torch

import head_dim_attention_gb300 as f
from head_dim_attention_gb300 import _lib

pytestmark = pytest.mark.gpu


def new(*shape):
    return torch.randn(*shape, device="cuda").half()


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def packed(D):
    q, k, v, dout = new(1, 2, 200, D), new(1, 1, 200, D), new(1, 1, 200, D), new(1, 2, 200, D)
    cu = i32([0, 70, 200])
    out, lse = f.attention_varlen_fwd(q, k, v, cu, causal=True)
    return q, k, v, cu, out, lse, dout


def plan(tokens):
    n = i32([0])
    return lambda: f.cache_plan(n, i32([tokens]), torch.zeros(1, 400, dtype=torch.int32, device="cuda"),
                                torch.arange(400, device="cuda").int(), i32([0]), 64, tokens)


def tree(n):
    kc, vc = new(n // 64, 1, 64, 128), new(n // 64, 1, 64, 128)
    table, q = torch.arange(n // 64, device="cuda").int()[None].contiguous(), new(1, 1, 1, 128)
    return lambda: f.attention_tree_fwd(q, kc, vc, table, i32([n]))


@pytest.mark.parametrize("which,launches", [
    ("fwd 128", 2), ("fwd 512", 2), ("fwd 832", 2), ("bwd 128", 5), ("bwd 512", 4), ("bwd 832", 4), ("tree 128", 1),
    ("tree 4096", 2), ("plan 8", 1), ("plan 9000", 2), ("append 0", 1),
])
def test_one_event_per_launch(which, launches):
    name, n = which.split()[0], int(which.split()[1])
    if name in ("fwd", "bwd"):
        q, k, v, cu, out, lse, dout = packed(n)
        call = (lambda: f.attention_varlen_fwd(q, k, v, cu, causal=True)) if name == "fwd" else \
            (lambda: f.attention_varlen_bwd(q, k, v, cu, out, lse, dout, causal=True))
    elif name == "append":
        k, cache, slots = new(1, 2, 5, 64), new(4, 2, 16, 64), torch.arange(5, device="cuda")
        call = lambda: f.cache_append(k, k, cache, cache.clone(), slots)  # noqa: E731
    else:
        call = plan(n) if name == "plan" else tree(n)
    call()
    events = [torch.cuda.Event(enable_timing=True) for _ in range(8)]
    for e in events:
        e.record()
    torch.cuda.synchronize()
    start = torch.cuda.Event(enable_timing=True)
    start.record()
    _lib.ffpa_set_timing_events(events)
    try:
        call()
    finally:
        _lib.ffpa_set_timing_events(None)
    torch.cuda.synchronize()
    assert f.ffpa_check_status() == 0
    since = [start.elapsed_time(e) for e in events]
    assert [t >= 0 for t in since] == [True] * (launches + 1) + [False] * (7 - launches)
    assert since[:launches + 1] == sorted(since[:launches + 1])
