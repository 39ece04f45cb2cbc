"""The packed backward against differences of the forward, along directions in which the loss moves most.

d/dt of loss(x + t d) with loss = sum(O dO), by central differences of the 64-bit
forward, against sum(gradient d) with d the sign of the gradient: every element
counts with its full size, so a gradient off by a few percent anywhere shows.

Room, in packed.py's terms, but for the sum along d and not for each element: dQ = dS K
is off by dS's own errors e, so sum(dQ d) by sum_ij e_ij (d_i . k_j), and likewise dK
through q_i . d_j and dV through dO_i . d_j; O's rounding moves Delta of a row, and with
it every dS of the row by P scale; each gradient is rounded once (u of it, for a shared
head u of each query head's part at least). On top 2^-13 of sum |gradient| for the
differences: a step t changes no score by more than t D scale max|k| < 0.02 (t = 1e-4,
D <= 832, |k| < 5), and what a central difference leaves is below a sixth of that squared.
"""
import pytest
import torch

from head_dim_attention_gb300 import attention_varlen_bwd, attention_varlen_fwd, ffpa_check_status
from packed import FP32, HALF_STEP, dense_fwd, make, starts, varlen_sees

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16
STEP = 1e-4


def loss(q, k, v, dout, lens, causal, scale):
    group, total = q.shape[1] // k.shape[1], 0.0
    for a, n in zip(starts(lens), lens):
        sees = varlen_sees(n, causal, q.device)
        for h in range(q.shape[1]):
            o, _, _ = dense_fwd(q[0, h, a:a + n], k[0, h // group, a:a + n], v[0, h // group, a:a + n], sees, scale)
            total += float((o * dout[0, h, a:a + n].double()).sum())
    return total


def rooms(q, k, v, out, lse, dout, dirs, lens, causal, scale):
    """How far sum(gradient d) may be off for each of the three gradients."""
    u, group = HALF_STEP[q.dtype], q.shape[1] // k.shape[1]
    room = [0.0, 0.0, 0.0]
    for a, n in zip(starts(lens), lens):
        rows, sees = slice(a, a + n), varlen_sees(n, causal, q.device)
        for h in range(q.shape[1]):
            g = h // group
            qh, kh, vh, oh, doh = (x.double() for x in (q[0, h, rows], k[0, g, rows], v[0, g, rows], out[0, h, rows],
                                                        dout[0, h, rows]))
            dq, dk, dv = dirs[0][0, h, rows], dirs[1][0, g, rows], dirs[2][0, g, rows]
            o, _, pv = dense_fwd(qh, kh, vh, sees, scale)
            p = torch.where(sees, torch.exp(qh @ kh.T * scale - lse[0, h, rows].double()[:, None]), 0.0)
            ds = p * (doh @ vh.T - (doh * oh).sum(1, keepdim=True)) * scale
            raw = p * (doh.abs() @ vh.abs().T + (doh * oh).abs().sum(1, keepdim=True)) * scale
            slack = (2 * u + FP32) * ds.abs() + 2.0 ** -14 * raw
            delta = (doh.abs() * (u * o.abs() + (u + FP32) * pv)).sum(1)
            for i, c in ((0, dq @ kh.T), (1, qh @ dk.T)):
                room[i] += float((slack * c.abs()).sum() + (delta * (p * scale * c).sum(1).abs()).sum())
            room[2] += float(((u + FP32) * p * (doh @ dv.T).abs()).sum())
            room[0] += u * float(((ds @ kh) * dq).abs().sum())
            room[1] += u * float(((ds.T @ qh) * dk).abs().sum())
            room[2] += u * float(((p.T @ doh) * dv).abs().sum())
    return room


@pytest.mark.parametrize("lens,Hq,Hkv,D,dtype,causal", [
    ([33, 90], 2, 1, 512, FP, True),
    ([70, 1, 60], 2, 2, 256, FP, False),
    ([150], 4, 2, 64, FP, True),
    ([129, 40], 2, 1, 832, FP, True),
    ([60, 64], 2, 1, 512, BF, False),
])
def test_slopes_along_the_gradient(lens, Hq, Hkv, D, dtype, causal):
    gen = torch.Generator(device="cuda").manual_seed(D)
    q, k, v, dout = (make(gen, h, sum(lens), D, dtype, True) for h in (Hq, Hkv, Hkv, Hq))
    cu = torch.tensor(starts(lens), dtype=torch.int32, device="cuda")
    out, lse = attention_varlen_fwd(q, k, v, cu, causal=causal)
    grads = attention_varlen_bwd(q, k, v, cu, out, lse, dout, causal=causal)
    torch.cuda.synchronize()
    assert ffpa_check_status() == 0
    base, dirs = [x.double() for x in (q, k, v)], [torch.sign(g.double()) for g in grads]
    for i, room in enumerate(rooms(q, k, v, out, lse, dout, dirs, lens, causal, D ** -0.5)):
        up, down = list(base), list(base)
        up[i], down[i] = base[i] + STEP * dirs[i], base[i] - STEP * dirs[i]
        slope = (loss(*up, dout, lens, causal, D ** -0.5) - loss(*down, dout, lens, causal, D ** -0.5)) / (2 * STEP)
        along = float((grads[i].double() * dirs[i]).sum())
        room += 2.0 ** -13 * along
        assert room <= 0.06 * along, "the bound is too wide to tell"
        assert abs(slope - along) <= room, f"{'qkv'[i]}: slope {slope}, gradient {along}, room {room}"
