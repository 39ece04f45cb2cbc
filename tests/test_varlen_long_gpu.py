"""Packed sequences of thousands of rows, forward and backward: rings and barrier phases
that wrap many times, many tiles of each work class, several calls in flight.

References and bounds as in packed.py, whose fp32 share holds for up to 4096 keys.
"""
import pytest
import torch

from head_dim_attention_gb300 import attention_bwd, attention_fwd, attention_varlen_bwd, attention_varlen_fwd, \
    ffpa_check_status
from packed import check_varlen_bwd, check_varlen_fwd, make, starts

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16


def inputs(lens, Hq, Hkv, D, dtype, token_major, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    cu = torch.tensor(starts(lens), dtype=torch.int32, device="cuda")
    return [make(gen, h, sum(lens), D, dtype, token_major) for h in (Hq, Hkv, Hkv, Hq)] + [cu]


def both(q, k, v, dout, cu, causal):
    out, lse = attention_varlen_fwd(q, k, v, cu, causal=causal)
    return out, lse, attention_varlen_bwd(q, k, v, cu, out, lse, dout, causal=causal)


def done():
    torch.cuda.synchronize()
    assert ffpa_check_status() == 0


@pytest.mark.parametrize("lens,Hq,Hkv,D,dtype,causal,token_major", [
    ([4095, 1, 130], 2, 1, 64, BF, True, True),
    ([1900, 2200], 2, 1, 128, FP, False, False),
    ([3001, 0, 900], 2, 2, 192, FP, True, True),
    ([2047, 1300], 2, 1, 256, BF, True, False),
    ([1100, 2500], 2, 1, 256, FP, False, True),
    ([2500, 640], 2, 1, 320, BF, False, True),
    ([4096, 513], 2, 1, 512, BF, True, True),
    ([2900, 1, 1030], 1, 1, 512, FP, False, False),
    ([2048, 900], 2, 1, 576, BF, True, True),
    ([1801, 1500], 2, 1, 704, FP, True, True),
    ([3000, 200], 1, 1, 832, BF, False, False),
    ([2300, 1025], 2, 1, 1024, BF, True, True),
])
def test_long_sequences(lens, Hq, Hkv, D, dtype, causal, token_major):
    q, k, v, dout, cu = inputs(lens, Hq, Hkv, D, dtype, token_major, seed=D)
    out, lse, grads = both(q, k, v, dout, cu, causal)
    done()
    check_varlen_fwd(q, k, v, lens, out, lse, causal, D ** -0.5)
    check_varlen_bwd(q, k, v, lens, out, lse, dout, grads, causal, D ** -0.5)


@pytest.mark.parametrize("D", [128, 192, 256, 512, 704])
def test_one_long_sequence_is_the_unpacked_call(D):
    q, k, v, dout, cu = inputs([5003], 2, 1, D, BF, False, seed=D + 1)
    out, lse, grads = both(q, k, v, dout, cu, True)
    o2, l2 = attention_fwd(q, k, v, causal=True)
    g2 = attention_bwd(q, k, v, out, lse, dout, causal=True)
    done()
    for a, b in zip((out, lse, *grads), (o2, l2, *g2)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("D", [256, 512, 832])
def test_backward_calls_on_two_streams_at_once(D):
    # each call's launches overlap one another, and the other stream's
    a, b = [900, 33, 1200], [128, 2000]
    ia, ib = inputs(a, 4, 2, D, BF, True, seed=5), inputs(b, 4, 2, D, BF, False, seed=6)
    oa, ob = (attention_varlen_fwd(*x[:3], x[4], causal=True) for x in (ia, ib))
    torch.cuda.synchronize()
    streams, results = [torch.cuda.Stream(), torch.cuda.Stream()], []
    for _ in range(6):
        pair = []
        for s, x, o in zip(streams, (ia, ib), (oa, ob)):
            with torch.cuda.stream(s):
                pair.append(attention_varlen_bwd(*x[:3], x[4], *o, x[3], causal=True))
        results.append(pair)
    done()
    for pair in results[1:]:
        for got, first in zip(pair, results[0]):
            assert all(torch.equal(g, f) for g, f in zip(got, first))
    for x, lens, o, grads in ((ia, a, oa, results[0][0]), (ib, b, ob, results[0][1])):
        check_varlen_bwd(*x[:3], lens, *o, x[3], grads, True, D ** -0.5)
