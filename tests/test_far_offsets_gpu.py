"""Offsets past 32 bits and layouts other than the contiguous one, for the packed
and paged calls: a cache and packed tensors of more than 2^31 elements of which
only the far end is used, strided queries and outputs, tensors of another stream.
"""
import pytest
import torch

from head_dim_attention_gb300 import attention_tree_fwd, attention_varlen_bwd, attention_varlen_fwd, cache_append, \
    ffpa_check_status
from packed import check_tree, check_varlen_bwd, check_varlen_fwd

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16
i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731


def done():
    torch.cuda.synchronize()
    assert ffpa_check_status() == 0


@pytest.mark.parametrize("token_major", [False, True])
def test_cache_past_32_bits(token_major):
    # 2^31 / (4 * 16 * 512) = 65536 pages hold 2^31 elements: the request's pages lie past them
    pages, Hkv, page, D, n = 66000, 4, 16, 512, 100
    gen = torch.Generator(device="cuda").manual_seed(0)
    shape = (pages, page, Hkv, D) if token_major else (pages, Hkv, page, D)
    kc, vc = (torch.empty(shape, dtype=BF, device="cuda") for _ in range(2))
    if token_major:
        kc, vc = kc.transpose(1, 2), vc.transpose(1, 2)
    assert kc.numel() > 2 ** 31
    table = i32([[pages - 1 - 3 * k for k in range(7)]])
    k, v = (torch.randn(1, Hkv, n, D, generator=gen, device="cuda").to(BF) for _ in range(2))
    t = torch.arange(n, device="cuda")
    cache_append(k, v, kc, vc, table[0].long()[t // page] * page + t % page)
    q = torch.randn(1, 8, 1, D, generator=gen, device="cuda").to(BF)
    out, lse = attention_tree_fwd(q, kc, vc, table, i32([n]))
    done()
    check_tree(q, [k[0].transpose(0, 1)], [v[0].transpose(0, 1)], [n], [1], None, out, lse, D ** -0.5)


@pytest.mark.parametrize("D,H", [(512, 8), (256, 16)])
def test_packed_rows_past_32_bits(D, H):
    T, lens = 2 ** 31 // (H * D) + 600, [130, 65]
    first = T - sum(lens)
    q, dout, k, v = (torch.empty(T, h, D, dtype=BF, device="cuda").transpose(0, 1)[None] for h in (H, H, 1, 1))
    assert q.numel() > 2 ** 31
    gen = torch.Generator(device="cuda").manual_seed(1)
    for x in (q, dout, k, v):
        x[:, :, first:] = torch.randn(1, x.shape[1], sum(lens), D, generator=gen, device="cuda").to(BF)
    cu = i32([first, first + lens[0], T])
    out, lse = torch.empty_like(q), torch.empty(1, H, T, device="cuda")
    attention_varlen_fwd(q, k, v, cu, causal=True, out=out, lse=lse)
    grads = attention_varlen_bwd(q, k, v, cu, out, lse, dout, causal=True)
    done()
    check_varlen_fwd(q, k, v, lens, out, lse, True, D ** -0.5, first=first)
    check_varlen_bwd(q, k, v, lens, out, lse, dout, grads, True, D ** -0.5, first=first)


def test_strided_queries_and_outputs():
    # q as a slice of a wider projection, out in token order, k and v rows padded
    gen = torch.Generator(device="cuda").manual_seed(2)
    T, D, lens = 300, 320, [100, 200]
    wide = torch.randn(T, 4 + 2 + 2, D + 8, generator=gen, device="cuda").to(FP)
    q, k, v = (wide[:, a:b, :D].transpose(0, 1)[None] for a, b in ((0, 4), (4, 6), (6, 8)))
    out = torch.empty(T, 4, D + 16, dtype=FP, device="cuda")[..., :D].transpose(0, 1)[None]
    lse = torch.empty(1, 4, T, device="cuda")
    attention_varlen_fwd(q, k, v, i32([0, 100, 300]), causal=False, out=out, lse=lse)
    done()
    check_varlen_fwd(q, k, v, lens, out, lse, False, D ** -0.5)
    # drafts: queries and outputs token by token, [B, T, H, D]
    from packed import paged
    host = torch.Generator().manual_seed(2)
    kc, vc, table, dk, dv = paged(gen, host, [70, 33], 2, 16, D, FP, token_major=True)
    qt = torch.randn(2, 5, 4, D, generator=gen, device="cuda").to(FP).transpose(1, 2)
    ot = torch.empty(2, 5, 4, D, dtype=FP, device="cuda").transpose(1, 2)
    lt = torch.empty(2, 4, 5, device="cuda")
    attention_tree_fwd(qt, kc, vc, table, i32([70, 33]), out=ot, lse=lt)
    done()
    check_tree(qt, dk, dv, [70, 33], [5, 5], None, ot, lt, D ** -0.5)


def test_calls_on_another_stream():
    gen = torch.Generator(device="cuda").manual_seed(3)
    q, k, v = (torch.randn(1, h, 200, 512, generator=gen, device="cuda").to(BF) for h in (2, 1, 1))
    cu, side = i32([0, 200]), torch.cuda.Stream()
    out, lse = torch.empty_like(q), torch.empty(1, 2, 200, device="cuda")
    torch.cuda.synchronize()
    attention_varlen_fwd(q, k, v, cu, causal=True, out=out, lse=lse, stream=side.cuda_stream)
    side.synchronize()
    check_varlen_fwd(q, k, v, [200], out, lse, True, 512 ** -0.5)
    assert ffpa_check_status(side.cuda_stream) == 0
