"""Host threads that call the library through its C entry points, which run without the
interpreter's lock: a thread's first use of CUDA, and two threads at once with head
dimensions that share a kernel.

A kernel's shared memory differs from head dimension to head dimension; one
thread's call may not change what another's launch is allowed.
"""
import threading

import pytest
import torch

from head_dim_attention_gb300 import _lib, ffpa_check_status

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
CALLS = 1500


def tree_call(lib, D):
    """One token per request over pages; 16 rows at every D."""
    gen = torch.Generator(device="cuda").manual_seed(D)
    q = torch.randn(2, 4, 1, D, generator=gen, device="cuda").to(BF)
    kc, vc = (torch.randn(6, 2, 16, D, generator=gen, device="cuda").to(BF) for _ in range(2))
    table = torch.arange(6, dtype=torch.int32, device="cuda").view(2, 3)
    lens = torch.tensor([40, 17], dtype=torch.int32, device="cuda")
    out, lse = torch.zeros_like(q), torch.zeros(2, 4, 1, device="cuda")
    keep = (q, kc, vc, table, lens, out, lse)
    args = (_lib._pack(q), _lib._pack(kc), _lib._pack(vc), table.data_ptr(), 3, lens.data_ptr(), None, None, 0, D ** -0.5,
            _lib._pack(out), _lib._pack_lse(lse))
    return keep, [out, lse], lambda stream: lib.ffpa_fwd_tree(*args, stream)


def dense(D, rows, keys, k_rows=None):
    gen = torch.Generator(device="cuda").manual_seed(D + rows)
    q = torch.randn(1, 2, rows, D, generator=gen, device="cuda").to(BF)
    k, v = (torch.randn(1, 2, k_rows or keys, D, generator=gen, device="cuda").to(BF)[:, :, :keys] for _ in range(2))
    return q, k, v, torch.zeros_like(q), torch.zeros(1, 2, rows, device="cuda")


def forward_call(lib, D, rows=64, keys=64, spread=False):
    q, k, v, out, lse = dense(D, rows, keys)
    if spread:  # rows of K and V apart: the other decode kernel
        k, v = (torch.cat([x, x], 3)[..., :D] for x in (k, v))
    ds = [_lib.describe(x) for x in (q, k, v, out)] + [_lib.describe(lse, as_lse=True)]
    r = [_lib._ref(d) for d in ds]
    return (q, k, v, out, lse, ds), [out, lse], lambda stream: lib.ffpa_fwd(r[0], r[1], r[2], None, 0, D ** -0.5, r[3], r[4],
                                                                            stream)


def backward_call(lib, D):
    q, k, v, out, lse = dense(D, 64, 64)
    _lib.ffpa_fwd(q, k, v, None, 0, D ** -0.5, out, lse)
    dout = torch.ones_like(q)
    grads = [torch.zeros_like(x) for x in (q, k, v)]
    ds = [_lib.describe(x) for x in (q, k, v, out)] + [_lib.describe(lse, as_lse=True)] + \
        [_lib.describe(x) for x in (dout, *grads)]
    r = [_lib._ref(d) for d in ds]
    return (q, k, v, out, lse, dout, ds), grads, lambda stream: lib.ffpa_bwd(r[0], r[1], r[2], None, 0, D ** -0.5, *r[3:],
                                                                              stream)


@pytest.mark.parametrize("make", [tree_call, forward_call, backward_call], ids=["tree", "forward", "backward"])
def test_first_use_of_cuda_in_a_thread(lib, make):
    _, outs, call = make(lib, 128)
    assert call(None) == 0
    torch.cuda.synchronize()
    want = [x.clone() for x in outs]
    for x in outs:
        x.zero_()
    torch.cuda.synchronize()
    codes = []
    t = threading.Thread(target=lambda: codes.append(call(None)))
    t.start()
    t.join()
    torch.cuda.synchronize()
    assert codes == [0] and ffpa_check_status() == 0
    assert all(torch.equal(a, b) for a, b in zip(outs, want))


@pytest.mark.parametrize("make,small,large", [
    (tree_call, dict(D=64), dict(D=512)),
    (forward_call, dict(D=64), dict(D=256)),
    (forward_call, dict(D=64, rows=1, keys=300), dict(D=512, rows=1, keys=300)),
    (forward_call, dict(D=64, rows=1, keys=300, spread=True), dict(D=512, rows=1, keys=300, spread=True)),
    (forward_call, dict(D=64, rows=5, keys=300), dict(D=1024, rows=16, keys=300)),
    (backward_call, dict(D=64), dict(D=256)),
], ids=["tree", "forward", "decode", "decode, spread rows", "decode, many rows", "backward"])
def test_two_threads_with_different_head_dimensions(lib, make, small, large):
    calls = [make(lib, **small), make(lib, **large)]
    want = []
    for _, outs, call in calls:
        assert call(None) == 0
        torch.cuda.synchronize()
        want.append([x.clone() for x in outs])
    streams = [torch.cuda.Stream() for _ in calls]
    codes, gate = [[], []], threading.Barrier(2)

    def work(i):
        _, _, call = calls[i]
        gate.wait()
        for _ in range(CALLS):
            codes[i].append(call(streams[i].cuda_stream))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert [sum(c != 0 for c in x) for x in codes] == [0, 0]
    assert ffpa_check_status() == 0
    for (_, outs, _), expect in zip(calls, want):
        assert all(torch.equal(a, b) for a, b in zip(outs, expect))
