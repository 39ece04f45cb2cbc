"""Packed-sequence attention, forward and backward, against 64-bit references
sequence by sequence (bounds derived in packed.py).

Lengths sit at and around the 128-row tile and the 64-row halves of the CTA
pairs; sequences may be empty; head dimensions cover every kernel the unpacked
call has (one CTA to 256, a pair to 512, O split at 576 and 640, the exchange
kernels above).
"""
import pytest
import torch

from head_dim_attention_gb300 import attention_bwd, attention_fwd, attention_varlen_bwd, attention_varlen_fwd, \
    ffpa_check_status
from packed import HALF_STEP, check_varlen_bwd, check_varlen_fwd, dense_fwd, make, starts, varlen_sees

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16


def cu_of(lens, first=0):
    return torch.tensor([first + x for x in starts(lens)], dtype=torch.int32, device="cuda")


def inputs(lens, Hq, Hkv, D, dtype, token_major=True, seed=0, tail=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    T = sum(lens) + tail
    return [make(gen, H, T, D, dtype, token_major) for H in (Hq, Hkv, Hkv, Hq)]


def done():
    torch.cuda.synchronize()
    assert ffpa_check_status() == 0


CASES = [
    ([1], 1, 1, 512, BF, True, True),
    ([2, 0, 1, 3], 4, 2, 512, FP, True, True),
    ([127, 128, 129, 1, 64, 65], 4, 2, 512, BF, True, True),
    ([300, 5, 257], 2, 1, 512, BF, False, False),
    ([200, 0, 77, 130], 2, 2, 64, FP, True, True),
    ([129, 31, 256], 4, 1, 128, BF, False, True),
    ([333, 100], 2, 1, 256, BF, True, False),
    ([190, 60, 129], 4, 2, 320, FP, True, True),
    ([140, 129], 2, 1, 448, BF, False, True),
    ([260, 40], 2, 2, 576, FP, True, True),
    ([131, 200], 2, 1, 640, BF, True, True),
    ([128, 1, 222], 2, 1, 704, FP, True, True),
    ([100, 300], 2, 2, 832, BF, False, False),
    ([257, 63, 0, 1], 2, 1, 1024, BF, True, True),
    ([40, 150], 2, 1, 960, FP, False, True),
]


@pytest.mark.parametrize("lens,Hq,Hkv,D,dtype,causal,token_major", CASES)
def test_forward(lens, Hq, Hkv, D, dtype, causal, token_major):
    q, k, v, _ = inputs(lens, Hq, Hkv, D, dtype, token_major)
    out, lse = attention_varlen_fwd(q, k, v, cu_of(lens), causal=causal)
    done()
    check_varlen_fwd(q, k, v, lens, out, lse, causal, D ** -0.5)


@pytest.mark.parametrize("lens,Hq,Hkv,D,dtype,causal,token_major", CASES)
def test_backward(lens, Hq, Hkv, D, dtype, causal, token_major):
    q, k, v, dout = inputs(lens, Hq, Hkv, D, dtype, token_major, seed=1)
    cu = cu_of(lens)
    out, lse = attention_varlen_fwd(q, k, v, cu, causal=causal)
    grads = attention_varlen_bwd(q, k, v, cu, out, lse, dout, causal=causal)
    done()
    check_varlen_bwd(q, k, v, lens, out, lse, dout, grads, causal, D ** -0.5)


def test_many_tiny_sequences():
    lens = [1, 2, 0, 3, 5] * 60
    q, k, v, dout = inputs(lens, 2, 1, 512, BF, seed=2)
    cu = cu_of(lens)
    out, lse = attention_varlen_fwd(q, k, v, cu, causal=True)
    grads = attention_varlen_bwd(q, k, v, cu, out, lse, dout, causal=True)
    done()
    check_varlen_fwd(q, k, v, lens, out, lse, True, 512 ** -0.5)
    check_varlen_bwd(q, k, v, lens, out, lse, dout, grads, True, 512 ** -0.5)


@pytest.mark.parametrize("D", [256, 512])
def test_one_sequence_is_the_unpacked_call(D):
    q, k, v, dout = inputs([300], 4, 2, D, BF, token_major=False, seed=3)
    cu = cu_of([300])
    out, lse = attention_varlen_fwd(q, k, v, cu, causal=True)
    grads = attention_varlen_bwd(q, k, v, cu, out, lse, dout, causal=True)
    o2, l2 = attention_fwd(q, k, v, causal=True)
    g2 = attention_bwd(q, k, v, out, lse, dout, causal=True)
    done()
    for a, b in zip((out, lse, *grads), (o2, l2, *g2)):
        assert torch.equal(a, b)  # the same kernels over the same tiles in the same order


def fill(t, value):
    return torch.full_like(t, value)


@pytest.mark.parametrize("D", [128, 512, 1024])
def test_rows_outside_are_left_and_values_stay_inside(D):
    # rows before, between the batch's end and T, and a sequence of NaN and infinities
    lens, first, tail = [90, 130, 70], 3, 9
    q, k, v, dout = inputs([first] + lens, 2, 1, D, BF, seed=4, tail=tail)
    cu = cu_of(lens, first)
    T = q.shape[2]

    def both():
        out, lse = fill(q, 7.0), torch.full(q.shape[:3], 7.0, device="cuda")
        attention_varlen_fwd(q, k, v, cu, causal=True, out=out, lse=lse)
        dq, dk, dv = fill(q, 7.0), fill(k, 7.0), fill(v, 7.0)
        attention_varlen_bwd(q, k, v, cu, out, lse, dout, causal=True, dq=dq, dk=dk, dv=dv)
        torch.cuda.synchronize()
        assert ffpa_check_status() == 0
        return out, lse, dq, dk, dv

    clean = both()
    mid = slice(first + lens[0], first + lens[0] + lens[1])
    outside = [slice(0, first), slice(T - tail, T)]
    for t in clean:
        for s in outside:
            assert bool((t[:, :, s] == 7.0).all())
    for t, bad in ((q, float("nan")), (k, float("inf")), (v, float("nan")), (dout, -float("inf"))):
        t[:, :, mid] = bad
        for s in outside:
            t[:, :, s] = float("nan")
    dirty = both()
    keep = torch.ones(T, dtype=torch.bool, device="cuda")
    keep[mid] = False
    for a, b in zip(clean, dirty):
        assert torch.equal(a[:, :, keep], b[:, :, keep])


def test_bad_starts_are_reported_and_touch_nothing():
    lens = [64, 50, 80]
    q, k, v, _ = inputs(lens, 2, 1, 512, BF, seed=5)
    # sequence 0 good, then a descent, a start past T, and a negative start
    cu = torch.tensor([0, 64, 40, 500, -3], dtype=torch.int32, device="cuda")
    out, lse = fill(q, 7.0), torch.full(q.shape[:3], 7.0, device="cuda")
    attention_varlen_fwd(q, k, v, cu, causal=True, out=out, lse=lse)
    torch.cuda.synchronize()
    assert ffpa_check_status() == 1  # FFPA_ERR_INVALID_ARG
    assert ffpa_check_status() == 0
    assert bool((out[:, :, 64:] == 7.0).all()) and bool((lse[:, :, 64:] == 7.0).all())
    check_varlen_fwd(q, k, v, [64], out, lse, True, 512 ** -0.5)


def test_captured_call_follows_new_lengths():
    T = 400
    q, k, v, dout = inputs([T], 4, 2, 512, BF, seed=6)
    cu = cu_of([100, 200, 100])
    out, lse = torch.empty_like(q), torch.empty(q.shape[:3], device="cuda")
    grads = [torch.empty_like(x) for x in (q, k, v)]

    def step():
        attention_varlen_fwd(q, k, v, cu, causal=True, out=out, lse=lse)
        attention_varlen_bwd(q, k, v, cu, out, lse, dout, causal=True, dq=grads[0], dk=grads[1], dv=grads[2])

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for lens in ([100, 200, 100], [1, 128, 271], [0, 0, 400]):
        cu.copy_(cu_of(lens))
        for t in (out, lse, *grads):
            t.fill_(float("nan"))
        graph.replay()
        done()
        check_varlen_fwd(q, k, v, lens, out, lse, True, 512 ** -0.5)
        check_varlen_bwd(q, k, v, lens, out, lse, dout, grads, True, 512 ** -0.5)


def test_two_streams_at_once():
    a, b = [150, 90, 260], [64, 300]
    ia, ib = inputs(a, 4, 2, 512, BF, seed=7), inputs(b, 4, 2, 512, BF, seed=8)
    torch.cuda.synchronize()
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    ca, cb = cu_of(a), cu_of(b)
    torch.cuda.synchronize()
    res = []
    for _ in range(5):
        with torch.cuda.stream(sa):
            ra = attention_varlen_fwd(*ia[:3], ca, causal=True)
        with torch.cuda.stream(sb):
            rb = attention_varlen_fwd(*ib[:3], cb, causal=True)
        res.append((ra, rb))
    done()
    for ra, rb in res:
        assert torch.equal(ra[0], res[0][0][0]) and torch.equal(rb[0], res[0][1][0])
    check_varlen_fwd(*ia[:3], a, *res[0][0], True, 512 ** -0.5)
    check_varlen_fwd(*ib[:3], b, *res[0][1], True, 512 ** -0.5)


def test_gradient_against_differences():
    # d/dt of sum(O dO) along a direction, by central differences of the 64-bit
    # forward, against the kernel's gradients: the difference of step t is off by
    # O(t^2), the gradients by at most 4 u of the sums of |gradient| |direction|
    lens, D = [33, 90], 512
    q, k, v, dout = inputs(lens, 2, 1, D, FP, seed=9)
    cu = cu_of(lens)
    out, lse = attention_varlen_fwd(q, k, v, cu, causal=True)
    grads = attention_varlen_bwd(q, k, v, cu, out, lse, dout, causal=True)
    done()
    gen = torch.Generator(device="cuda").manual_seed(10)

    def loss(q, k, v):
        total = torch.zeros((), dtype=torch.float64, device="cuda")
        for s, (a, n) in enumerate(zip(starts(lens), lens)):
            for h in range(2):
                o, _, _ = dense_fwd(q[0, h, a:a + n], k[0, 0, a:a + n], v[0, 0, a:a + n], varlen_sees(n, True),
                                    D ** -0.5)
                total += (o * dout[0, h, a:a + n].double()).sum()
        return total

    base = [x.double() for x in (q, k, v)]
    for i in range(3):
        d = torch.randn(base[i].shape, generator=gen, device="cuda", dtype=torch.float64)
        t = 1e-4
        up, down = list(base), list(base)
        up[i], down[i] = base[i] + t * d, base[i] - t * d
        slope = float(loss(*up) - loss(*down)) / (2 * t)
        along = float((grads[i].double() * d).sum())
        room = 4 * HALF_STEP[FP] * float((grads[i].double().abs() * d.abs()).sum())
        assert abs(slope - along) <= room


@pytest.mark.parametrize("D", range(64, 1025, 64))
def test_small_tensors(D):
    """Head dimensions and head counts of every kernel, over tensors and sequences that span a few KB to a few MB."""
    pick = [0, 1, 2, 17, 63, 64, 65, 100, 127, 128, 129, 200, 255, 256, 257, 390]
    host = torch.Generator().manual_seed(D)
    draw = lambda n: int(torch.randint(n, (1,), generator=host))  # noqa: E731
    for case in range(6):
        Hkv = 1 + draw(3)
        Hq, dtype, causal, token_major = Hkv * (1, 2, 4, 5)[draw(4)], (BF, FP)[case % 2], draw(3) > 0, draw(2) == 1
        lens = [pick[draw(16)] for _ in range(1 + draw(9))] + [1 + draw(40)]
        q, k, v, dout = inputs(lens, Hq, Hkv, D, dtype, token_major, seed=case)
        cu = cu_of(lens)
        out, lse = attention_varlen_fwd(q, k, v, cu, causal=causal)
        done()
        check_varlen_fwd(q, k, v, lens, out, lse, causal, D ** -0.5)
        grads = attention_varlen_bwd(q, k, v, cu, out, lse, dout, causal=causal)
        done()
        check_varlen_bwd(q, k, v, lens, out, lse, dout, grads, causal, D ** -0.5)
