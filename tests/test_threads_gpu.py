"""Host threads that call the library through its C entry points."""
import threading

import pytest
import torch

from head_dim_attention_gb300 import _lib, ffpa_check_status

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


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
