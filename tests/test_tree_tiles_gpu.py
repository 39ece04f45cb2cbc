"""Drafted tokens over pages where a block takes many key tiles of one request after another.

Each tile's row maxima, weights and ring slots follow the tile before it without
a pause there, so these cases keep the softmax warps apart from one another: the
largest score of a row moves from warp to warp (32 keys each) and grows along the
context, another stream keeps the GPU busy, and every run has to give the same
bits.
"""
import pytest
import torch

from head_dim_attention_gb300 import attention_tree_fwd, ffpa_check_status
from packed import check_tree, paged

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16


def rising_keys(dense, kc, table, page, D):
    """Scales the requests' keys by 1 + (tile) / 2 and, of each 128 of them, one run of 32 by 3 more, another run in
    each tile; writes them into their pages."""
    for b, k in enumerate(dense):
        n = k.shape[0]
        pos = torch.arange(n, device="cuda")
        tile, warp = pos // 128, pos % 128 // 32
        factor = (1 + tile / 2) * torch.where(warp == (tile * 3 + b) % 4, 4.0, 1.0)
        # a row's scores reach about 16: its maximum grows past the 2^8 at which O is rescaled
        k.copy_((k.float() * (factor / factor.max()).clamp(min=0.05)[:, None, None]).to(k.dtype))
        for c in range((n + page - 1) // page):
            part = k[c * page:(c + 1) * page]
            kc[int(table[b, c]), :, :part.shape[0]] = part.transpose(0, 1)


def many_tiles(lens, T, Hq, D, page, dtype, runs, busy):
    gen, host = torch.Generator(device="cuda").manual_seed(D + T), torch.Generator().manual_seed(D + T)
    kc, vc, table, dk, dv = paged(gen, host, lens, 1, page, D, dtype)
    rising_keys(dk, kc, table, page, D)
    q = (4 * torch.randn(len(lens), Hq, T, D, generator=gen, device="cuda")).to(dtype)
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    x = torch.randn(4096, 4096, device="cuda", dtype=BF)
    torch.cuda.synchronize()
    results, side = [], torch.cuda.Stream()
    for _ in range(runs):
        if busy:
            with torch.cuda.stream(side):
                x @ x
        results.append(attention_tree_fwd(q, kc, vc, table, n))
    torch.cuda.synchronize()
    assert ffpa_check_status() == 0
    for out, lse in results[1:]:
        assert torch.equal(out, results[0][0]) and torch.equal(lse, results[0][1])
    check_tree(q, dk, dv, lens, [T] * len(lens), None, *results[0], D ** -0.5)


@pytest.mark.parametrize("T,Hq,D,dtype", [
    (1, 2, 64, BF),    # 16 rows
    (10, 2, 64, FP),   # 32
    (20, 2, 64, BF),   # 48
    (30, 2, 64, FP),   # 64
    (45, 2, 64, BF),   # 96: one buffer of scores
    (1, 8, 512, BF),
    (12, 8, 512, FP),
])
def test_row_maxima_from_tile_to_tile(T, Hq, D, dtype):
    lens = [1500 - 7 * i for i in range(80)]  # 12 key tiles each, about 6 to a block
    many_tiles(lens, T, Hq, D, 64, dtype, runs=12, busy=True)


@pytest.mark.parametrize("T,Hq,D,dtype", [
    (1, 4, 64, FP),     # five slots
    (1, 4, 128, FP),    # three, two blocks to an SM
    (24, 2, 256, BF),   # five
    (12, 8, 384, BF),   # three
    (8, 8, 512, BF),
    (12, 8, 512, BF),
    (8, 8, 704, FP),
    (1, 8, 832, FP),    # five
    (6, 8, 1024, BF),   # three
])
def test_rings_of_an_odd_number_of_slots(T, Hq, D, dtype):
    lens = [2300 - 31 * i for i in range(40)]  # 18 key tiles and fewer, whole rings many times over
    many_tiles(lens, T, Hq, D, 32, dtype, runs=3, busy=False)
