"""A paged cache: plans, writes, attention of drafted tokens, and a serving step
that runs them together.  Plans and writes are compared exactly, attention
within the bounds of packed.py.
"""
import pytest
import torch

from head_dim_attention_gb300 import attention_tree_fwd, attention_varlen_fwd, cache_append, cache_plan, \
    ffpa_check_status
from packed import check_tree, check_varlen_fwd, make, paged

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16
i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731


def done(want=0):
    torch.cuda.synchronize()
    assert ffpa_check_status() == want


# ------------------------------------------------------------------ plan

def plan_reference(lens, new, table, free, head, page, max_new):
    table, slots, cu = [list(r) for r in table], [], [0]
    for b, (n, m) in enumerate(zip(lens, new)):
        for k in range((n + page - 1) // page, (n + m + page - 1) // page):
            table[b][k] = free[head]
            head += 1
        slots += [table[b][t // page] * page + t % page for t in range(n, n + m)]
        cu.append(cu[-1] + m)
    return table, cu, slots + [-1] * (max_new - len(slots)), [a + b for a, b in zip(lens, new)], head


def plan_case(B, page, seed, longest=400, most=300):
    host = torch.Generator().manual_seed(seed)
    rand = lambda hi: int(torch.randint(0, hi + 1, (1,), generator=host))  # noqa: E731
    lens = [rand(longest) if rand(3) else 0 for _ in range(B)]
    new = [rand(most) if rand(2) else rand(1) for _ in range(B)]
    per = (longest + most + page - 1) // page + 1
    had = [(n + page - 1) // page for n in lens]
    order = torch.randperm(B * per + 20, generator=host).tolist()
    table = [[order.pop() for _ in range(h)] + [-7] * (per - h) for h in had]
    return lens, new, table, order, rand(5)


@pytest.mark.parametrize("B,page,pad", [(1, 16, 0), (3, 1, 5), (33, 16, 3), (200, 64, 0), (1025, 128, 9), (40, 7, 1)])
def test_plan(B, page, pad):
    lens, new, table, free, head = plan_case(B, page, B + page)
    max_new = sum(new) + pad
    t = i32(table)
    got = cache_plan(i32(lens), i32(new), t, i32(free), i32([head]), page, max_new)
    done()
    want = plan_reference(lens, new, table, free, head, page, max_new)
    assert t.tolist() == want[0]
    for g, w in zip(got, want[1:4]):
        assert g.tolist() == w
    assert got[3].tolist() == [want[4]]


def test_plan_large_step_and_in_place():
    lens, new, table, free, head = plan_case(64, 16, 5, longest=3000, most=2000)
    assert sum(new) > 20000
    t, n, at = i32(table), i32(lens), i32([head])
    cu, slots, n2, at2 = cache_plan(n, i32(new), t, i32(free), at, 16, sum(new), lens_out=n, free_head_out=at)
    done()
    assert n2 is n and at2 is at
    want = plan_reference(lens, new, table, free, head, 16, sum(new))
    assert t.tolist() == want[0] and cu.tolist() == want[1] and slots.tolist() == want[2]
    assert n.tolist() == want[3] and at.tolist() == [want[4]]


def test_plan_without_pages_or_columns_is_reported():
    # request 0 takes the last free page, request 1 finds none, request 2's table is full
    t = i32([[-1, -1], [-1, -1], [5, 6]])
    cu, slots, lens, head = cache_plan(i32([0, 0, 32]), i32([3, 2, 1]), t, i32([9]), i32([0]), 16, 8)
    done(1)
    assert t.tolist() == [[9, -1], [-1, -1], [5, 6]]
    assert cu.tolist() == [0, 3, 5, 6] and lens.tolist() == [3, 2, 33] and head.tolist() == [1]
    assert slots.tolist() == [144, 145, 146, -1, -1, -1, -1, -1]
    # negative lengths add nothing; more tokens than slots are reported
    t = i32([[1], [2]])
    cu, slots, lens, head = cache_plan(i32([-4, 3]), i32([2, 5]), t, i32([7]), i32([0]), 16, 3)
    done(1)
    assert cu.tolist() == [0, 0, 5] and slots.tolist() == [35, 36, 37] and head.tolist() == [0]


# ------------------------------------------------------------------ append

@pytest.mark.parametrize("T,Hkv,D,page,dtype,token_major,cache_token_major", [
    (1, 1, 64, 16, BF, True, False), (33, 4, 512, 16, FP, True, True), (257, 2, 320, 64, BF, False, False),
    (700, 8, 1024, 128, BF, True, False), (50, 3, 192, 256, FP, False, True),
])
def test_append(T, Hkv, D, page, dtype, token_major, cache_token_major):
    gen = torch.Generator(device="cuda").manual_seed(T)
    host = torch.Generator().manual_seed(T)
    pages = (T + page - 1) // page + 2
    k, v = make(gen, Hkv, T, D, dtype, token_major), make(gen, Hkv, T, D, dtype, token_major)
    shape = (pages, page, Hkv, D) if cache_token_major else (pages, Hkv, page, D)
    kc, vc = (torch.randn(shape, generator=gen, device="cuda").to(dtype) for _ in range(2))
    if cache_token_major:
        kc, vc = kc.transpose(1, 2), vc.transpose(1, 2)
    slots = torch.randperm(pages * page, generator=host)[:T]
    slots[::5] = -1
    want = []
    for c, x in ((kc, k), (vc, v)):
        w = c.clone()
        for t in range(T):
            if slots[t] >= 0:
                w[slots[t] // page, :, slots[t] % page] = x[0, :, t]
        want.append(w)
    cache_append(k, v, kc, vc, slots.cuda())
    done()
    assert torch.equal(kc, want[0]) and torch.equal(vc, want[1])


def test_append_past_the_last_page_is_skipped_and_reported():
    k = torch.ones(1, 2, 3, 64, dtype=BF, device="cuda")
    kc, vc = torch.zeros(2, 2, 16, 64, dtype=BF, device="cuda"), torch.zeros(2, 2, 16, 64, dtype=BF, device="cuda")
    cache_append(k, k, kc, vc, torch.tensor([31, 32, 1 << 40], device="cuda"))
    done(1)
    assert float(kc.float().sum()) == 128.0 and bool((kc[1, :, 15] == 1).all())


# ------------------------------------------------------------------ drafted tokens

def tree_of(host, B, T):
    sees = torch.zeros(B, T, T, dtype=torch.bool)
    for b in range(B):
        for i in range(T):
            parent = int(torch.randint(-1, i, (1,), generator=host)) if i else -1
            if parent >= 0:
                sees[b, i] |= sees[b, parent]
            sees[b, i, i] = True
    return sees.cuda()


def run_tree(lens, drafts, T, Hq, Hkv, D, page, dtype, mask=None, seed=0, fill=None, token_major=False, give=True):
    gen, host = torch.Generator(device="cuda").manual_seed(seed), torch.Generator().manual_seed(seed)
    kc, vc, table, dk, dv = paged(gen, host, lens, Hkv, page, D, dtype, token_major=token_major, fill=fill)
    B = len(lens)
    q = torch.randn(B, Hq, T, D, generator=gen, device="cuda").to(dtype)
    if mask == "tree":
        mask = tree_of(host, B, T)
    out, lse = torch.full_like(q, 7.0), torch.full(q.shape[:3], 7.0, device="cuda")
    attention_tree_fwd(q, kc, vc, table, i32(lens), draft_lens=i32(drafts) if give else None, tree_mask=mask,
                       out=out, lse=lse)
    done()
    check_tree(q, dk, dv, lens, drafts, mask, out, lse, D ** -0.5, untouched=7.0)
    return q, kc, vc, table, out, lse


@pytest.mark.parametrize("lens,T,Hq,Hkv,D,page,dtype", [
    ([1], 1, 1, 1, 64, 16, BF),
    ([1, 2, 16, 17], 1, 1, 1, 512, 16, BF),
    ([127, 128, 129, 300], 1, 8, 4, 512, 16, FP),
    ([1000, 3, 640], 1, 8, 1, 512, 64, BF),
    ([500, 77], 1, 16, 1, 128, 32, FP),
    ([2049], 1, 2, 2, 1024, 128, BF),
    ([300, 511], 1, 4, 2, 320, 256, BF),
    ([129, 255, 256], 1, 4, 4, 960, 256, FP),
    ([90] * 40, 1, 4, 2, 192, 16, BF),
])
def test_one_token(lens, T, Hq, Hkv, D, page, dtype):
    run_tree(lens, [1] * len(lens), T, Hq, Hkv, D, page, dtype, give=False)


@pytest.mark.parametrize("lens,drafts,T,Hq,Hkv,D,page,dtype,mask", [
    ([5], [5], 5, 2, 1, 64, 16, BF, None),                          # no context before the drafts
    ([200, 64, 7], [8, 3, 7], 8, 4, 2, 512, 16, FP, "tree"),
    ([130, 129, 0, 1], [5, 2, 0, 1], 5, 2, 2, 512, 32, BF, "tree"),  # drafts across a key tile; an empty entry
    ([700, 300, 140], [24, 0, 24], 24, 8, 2, 512, 64, BF, "tree"),   # 96 rows: two row tiles
    ([400, 128], [64, 64], 64, 4, 1, 640, 128, FP, "tree"),          # 256 rows
    ([260, 199], [33, 20], 33, 2, 1, 1024, 16, BF, "tree"),          # 66 rows of 32
    ([900], [128], 128, 4, 4, 256, 256, FP, "tree"),
    ([150, 40], [16, 9], 16, 4, 2, 768, 32, BF, None),
    ([333, 90], [12, 12], 12, 4, 1, 448, 16, BF, "tree"),            # 48 rows
    ([300, 64, 130], [20, 5, 11], 20, 4, 2, 896, 32, BF, "tree"),    # 40 rows of 48
    ([200, 140], [33, 25], 33, 4, 2, 1024, 64, FP, None),            # 66 rows of 48
])
def test_drafts(lens, drafts, T, Hq, Hkv, D, page, dtype, mask):
    run_tree(lens, drafts, T, Hq, Hkv, D, page, dtype, mask=mask, seed=1)


def test_long_context_is_shared_out_and_joined():
    run_tree([9000, 1, 4100], [4, 1, 2], 4, 4, 2, 512, 64, BF, mask="tree", seed=2)
    run_tree([20000], [1], 1, 1, 1, 64, 16, FP, seed=3)
    run_tree([9999], [3], 3, 8, 1, 512, 64, BF, mask="tree", seed=4)   # many pieces of one unit
    run_tree([5000, 7], [11, 7], 11, 2, 1, 1024, 16, FP, seed=5)


def test_many_requests():
    # more requests than threads of a block, empty ones among them
    lens = [(37 * i) % 90 for i in range(700)]
    run_tree(lens, [min(n, 1) for n in lens], 1, 2, 1, 64, 16, BF, seed=4)


def test_requests_may_share_pages():
    # three requests on one request's pages: all of them, a prefix that ends inside a page, one token
    gen, host = torch.Generator(device="cuda").manual_seed(9), torch.Generator().manual_seed(9)
    kc, vc, table, dk, dv = paged(gen, host, [200], 2, 32, 256, BF)
    lens, drafts = [200, 150, 1], [2, 1, 1]
    q = torch.randn(3, 4, 2, 256, generator=gen, device="cuda").to(BF)
    out, lse = torch.full_like(q, 7.0), torch.full(q.shape[:3], 7.0, device="cuda")
    attention_tree_fwd(q, kc, vc, table.repeat(3, 1), i32(lens), draft_lens=i32(drafts), out=out, lse=lse)
    done()
    check_tree(q, [dk[0][:n] for n in lens], [dv[0][:n] for n in lens], lens, drafts, None, out, lse, 256 ** -0.5,
               untouched=7.0)


def test_mask_that_leaves_nothing():
    mask = torch.zeros(1, 3, 3, dtype=torch.bool, device="cuda")
    mask[0, 1, 0] = True  # row 1 sees draft 0, rows 0 and 2 see no draft
    run_tree([3, 200], [3, 3], 3, 2, 1, 512, 16, BF, mask=mask, seed=5)


@pytest.mark.parametrize("page", [16, 64, 256])
@pytest.mark.parametrize("fill", [float("nan"), float("inf")])
def test_unused_rows_may_hold_anything(page, fill):
    run_tree([page + 3, 5, 129], [2, 1, 2], 2, 4, 2, 512, page, BF, seed=6, fill=fill)
    run_tree([page + 3, 5, 129], [2, 1, 2], 2, 4, 2, 320, page, FP, seed=6, fill=fill, token_major=True)


def test_large_scores_move_the_reference():
    # keys whose scores grow along the context by far more than 2^8 a tile
    gen, host = torch.Generator(device="cuda").manual_seed(7), torch.Generator().manual_seed(7)
    lens, D = [700, 650], 128
    kc, vc, table, dk, dv = paged(gen, host, lens, 1, 16, D, FP)
    q = torch.ones(2, 2, 1, D, dtype=FP, device="cuda")
    for b, n in enumerate(lens):
        up = torch.linspace(0, 6, n, device="cuda").to(FP)
        for t in range(n):
            dk[b][t] = up[t]
        for k in range((n + 15) // 16):
            part = dk[b][16 * k:16 * k + 16]
            kc[int(table[b, k]), :, :part.shape[0]] = part.transpose(0, 1)
    out, lse = attention_tree_fwd(q, kc, vc, table, i32(lens))
    done()
    check_tree(q, dk, dv, lens, [1, 1], None, out, lse, D ** -0.5)


def test_bad_lengths_and_pages_are_reported():
    gen, host = torch.Generator(device="cuda").manual_seed(8), torch.Generator().manual_seed(8)
    lens = [100, 60]
    kc, vc, table, dk, dv = paged(gen, host, lens, 1, 16, 512, BF)
    q = torch.randn(2, 2, 2, 512, generator=gen, device="cuda").to(BF)
    ok, _ = attention_tree_fwd(q, kc, vc, table, i32(lens))
    done()
    for bad_lens, bad_drafts in (([100, 1 << 20], None), ([100, -5], None), ([100, 60], [2, 3]), ([100, 60], [2, -1])):
        out, _ = attention_tree_fwd(q, kc, vc, table, i32(bad_lens), draft_lens=None if bad_drafts is None else i32(bad_drafts))
        done(1)
        assert torch.equal(out[0], ok[0])  # the other request is not touched by it
    broken = table.clone()
    broken[1, 0], broken[1, 1] = -1, 1 << 30
    out, _ = attention_tree_fwd(q, kc, vc, broken, i32(lens))
    done(1)
    assert torch.equal(out[0], ok[0])


def test_captured_tree_follows_lengths_and_two_graphs_live_together():
    gen, host = torch.Generator(device="cuda").manual_seed(9), torch.Generator().manual_seed(9)
    lens = [400, 300, 350]
    kc, vc, table, dk, dv = paged(gen, host, lens, 2, 32, 512, BF)
    q = torch.randn(3, 4, 3, 512, generator=gen, device="cuda").to(BF)
    n = i32(lens)
    attention_tree_fwd(q, kc, vc, table, n)
    torch.cuda.synchronize()
    runs = []
    for _ in range(2):
        out, lse = torch.empty_like(q), torch.empty(q.shape[:3], device="cuda")
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            attention_tree_fwd(q, kc, vc, table, n, out=out, lse=lse)
        runs.append((g, out, lse))
    for now in ([400, 300, 350], [17, 300, 129], [5, 0, 256]):
        n.copy_(i32(now))
        for _, out, lse in runs:
            out.fill_(7.0)
            lse.fill_(7.0)
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream(), torch.cuda.Stream()]
        for (g, _, _), s in zip(runs, streams):
            with torch.cuda.stream(s):
                g.replay()
        done()
        for _, out, lse in runs:
            check_tree(q, [x[:m] for x, m in zip(dk, now)], [x[:m] for x, m in zip(dv, now)], now,
                       [min(3, m) for m in now], None, out, lse, 512 ** -0.5, untouched=7.0)


# ------------------------------------------------------------------ a serving step

def test_prompts_then_drafts():
    """Prompts are planned, appended and attended packed; then a tree of drafts over the pages they filled."""
    gen = torch.Generator(device="cuda").manual_seed(10)
    host = torch.Generator().manual_seed(10)
    B, Hq, Hkv, D, page, T = 3, 4, 2, 512, 16, 5
    prompts = [37, 200, 128]
    table = torch.full((B, 20), -1, dtype=torch.int32, device="cuda")
    free = torch.randperm(60, generator=host).to(torch.int32).cuda()
    lens, head = i32([0] * B), i32([0])
    kc, vc = (torch.full((60, Hkv, page, D), float("nan"), dtype=BF, device="cuda") for _ in range(2))
    total = sum(prompts)
    q, k, v = (make(gen, h, total + 4, D, BF, True) for h in (Hq, Hkv, Hkv))
    cu, slots, lens, head = cache_plan(lens, i32(prompts), table, free, head, page, total + 4)
    cache_append(k, v, kc, vc, slots)
    out, lse = attention_varlen_fwd(q, k, v, cu, causal=True)
    done()
    check_varlen_fwd(q, k, v, prompts, out, lse, True, D ** -0.5)
    drafts = [5, 1, 3]
    q2, k2, v2 = (make(gen, h, sum(drafts), D, BF, True) for h in (Hq, Hkv, Hkv))
    cu2, slots2, lens2, head = cache_plan(lens, i32(drafts), table, free, head, page, sum(drafts))
    cache_append(k2, v2, kc, vc, slots2)
    qt = torch.zeros(B, Hq, T, D, dtype=BF, device="cuda")
    starts = [0, 5, 6]
    for b in range(B):
        qt[b, :, :drafts[b]] = q2[0, :, starts[b]:starts[b] + drafts[b]]
    mask = tree_of(host, B, T)
    out, lse = torch.full_like(qt, 7.0), torch.full(qt.shape[:3], 7.0, device="cuda")
    attention_tree_fwd(qt, kc, vc, table, lens2, draft_lens=i32(drafts), tree_mask=mask, out=out, lse=lse)
    done()
    first = [0, 37, 237]
    dense = []
    for x, x2 in ((k, k2), (v, v2)):
        dense.append([torch.cat([x[0, :, first[b]:first[b] + prompts[b]], x2[0, :, starts[b]:starts[b] + drafts[b]]], 1)
                      .transpose(0, 1) for b in range(B)])
    check_tree(qt, dense[0], dense[1], [a + b for a, b in zip(prompts, drafts)], drafts, mask, out, lse, D ** -0.5,
               untouched=7.0)
