"""A chunk of new tokens behind cached ones, longer than one call's 128: written once, attended in pieces."""
import pytest
import torch

from head_dim_attention_gb300 import attention_tree_fwd, cache_append, cache_plan, ffpa_check_status
from packed import check_tree, make, paged

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D,page,dtype", [(512, 16, torch.bfloat16), (192, 128, torch.float16), (832, 64, torch.bfloat16)])
def test_chunk_in_pieces(D, page, dtype):
    gen, host = torch.Generator(device="cuda").manual_seed(D), torch.Generator().manual_seed(D)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    Hq, Hkv, lens, new = 4, 2, [77, 256], [300, 129]
    kc, vc, table, dk, dv = paged(gen, host, lens, Hkv, page, D, dtype, spare=40, fill=float("nan"))
    used = set(table.flatten().tolist())
    free = i32([x for x in range(kc.shape[0]) if x not in used])
    wide = torch.full((2, 40), -1, dtype=torch.int32, device="cuda")
    wide[:, :table.shape[1]] = table
    q, k, v = (make(gen, h, sum(new), D, dtype, True) for h in (Hq, Hkv, Hkv))
    cu, slots, after, _ = cache_plan(i32(lens), i32(new), wide, free, i32([0]), page, sum(new))
    cache_append(k, v, kc, vc, slots)
    first, dense = [0, 300], []
    for x, old in ((k, dk), (v, dv)):
        dense.append([torch.cat([old[b], x[0, :, first[b]:first[b] + new[b]].transpose(0, 1)]) for b in range(2)])
    for at in range(0, 300, 128):
        m = [max(0, min(128, n - at)) for n in new]
        n = [lens[b] + at + m[b] if m[b] else 0 for b in range(2)]
        piece = torch.zeros(2, Hq, 128, D, dtype=dtype, device="cuda")
        for b in range(2):
            piece[b, :, :m[b]] = q[0, :, first[b] + at:first[b] + at + m[b]]
        out, lse = torch.full_like(piece, 7.0), torch.full(piece.shape[:3], 7.0, device="cuda")
        attention_tree_fwd(piece, kc, vc, wide, i32(n), draft_lens=i32(m), out=out, lse=lse)
        torch.cuda.synchronize()
        assert ffpa_check_status() == 0
        check_tree(piece, [x[:j] for x, j in zip(dense[0], n)], [x[:j] for x, j in zip(dense[1], n)], n, m, None, out, lse,
                   D ** -0.5, untouched=7.0)
    assert after.tolist() == [377, 385]
