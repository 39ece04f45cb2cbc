"""64-bit references and derived error bounds for packed-sequence attention and paged caches.

Let u be half a step of the 16-bit type relative to a value (bf16 2^-8, fp16
2^-11).  The kernels keep scores, softmax statistics and sums in fp32 and
round three things to 16 bits: the output (u |O|), the weights fed to the
matrix instructions (each p_j to within u p_j, so O moves by at most
u sum_j p_j |v_j|; where the kernel adds the rounding residual it moves less)
and, in the backward, P and dS (dS = P (dP - Delta) uses the rounded P and is
rounded itself: 2 u |dS|).  FP32 effects are bounded by 2^-12 of the same sums:
a score's error is at most D 2^-24 sum_d |q_d k_d| scale, about 4e-5 at D = 1024
with unit-variance inputs' worst sums near 2 sqrt(D), ex2 is good to 2^-22, and
a sum of n terms in fp32 to n 2^-24 <= 2^-12 for n <= 4096.  In the backward the
difference dP - Delta cancels, so its fp32 error counts against the sums it is
formed from: 2^-14 of |dO| |V|^T + |dO| |O|.
"""
import torch

HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
FP32 = 2.0 ** -12
LSE_ATOL = 1e-3


def starts(lens):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return cu


def dense_fwd(q, k, v, sees, scale):
    """(O, lse, sum_j p_j |v_j|) in 64 bits of q [n, D], k/v [m, D]; sees [n, m] bool.  A row that sees nothing is 0
    with lse -inf."""
    q, k, v = q.double(), k.double(), v.double()
    s = (q @ k.T) * scale
    s = torch.where(sees, s, torch.full_like(s, -float("inf")))
    top = s.amax(1, keepdim=True)
    e = torch.exp(s - torch.where(torch.isinf(top), torch.zeros_like(top), top))
    total = e.sum(1, keepdim=True)
    p = torch.where(total > 0, e / total.clamp(min=1e-300), torch.zeros_like(e))
    lse = (top + torch.log(total))[:, 0]
    return p @ v, lse, p @ v.abs()


def dense_bwd(q, k, v, out, lse, dout, sees, scale, u):
    """(dQ, dK, dV) in 64 bits and their error bounds, from the forward's out and lse."""
    q, k, v, out, lse, dout = (x.double() for x in (q, k, v, out, lse, dout))
    p = torch.where(sees, torch.exp((q @ k.T) * scale - lse[:, None]), torch.zeros(1, dtype=torch.float64, device=q.device))
    dp = dout @ v.T
    delta = (dout * out).sum(1, keepdim=True)
    ds = p * (dp - delta) * scale
    raw = p * (dout.abs() @ v.abs().T + (dout * out).abs().sum(1, keepdim=True)) * scale
    slack = (2 * u + FP32) * ds.abs() + 2.0 ** -14 * raw
    dq, dk, dv = ds @ k, ds.T @ q, p.T @ dout
    return (dq, dk, dv), (u * dq.abs() + slack @ k.abs(), slack.T @ q.abs(), (u + FP32) * (p.T @ dout.abs()))


def inside(got, want, bound, what):
    """Every element within its bound (plus the smallest normal step of fp16)."""
    err = (got.double() - want).abs()
    bad = ~(err <= bound + 2.0 ** -24)
    if bool(bad.any()):
        i = int(torch.argmax(torch.where(bad, err - bound, torch.full_like(err, -1.0)).flatten()))
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outside the bound; worst at {i}: got "
                             f"{float(got.double().flatten()[i])!r} want {float(want.flatten()[i])!r} bound "
                             f"{float(bound.flatten()[i])!r}")


def make(gen, H, T, D, dtype, token_major):
    if token_major:
        return torch.randn(T, H, D, generator=gen, device="cuda").to(dtype).transpose(0, 1)[None]
    return torch.randn(1, H, T, D, generator=gen, device="cuda").to(dtype)


def varlen_sees(n, causal, device="cuda"):
    full = torch.ones(n, n, dtype=torch.bool, device=device)
    return full.tril() if causal else full


def check_varlen_fwd(q, k, v, lens, out, lse, causal, scale, first=0, what="O"):
    u = HALF_STEP[q.dtype]
    group = q.shape[1] // k.shape[1]
    row = first
    for s, n in enumerate(lens):
        rows = slice(row, row + n)
        row += n
        if n == 0:
            continue
        for h in range(q.shape[1]):
            o, l, pv = dense_fwd(q[0, h, rows], k[0, h // group, rows], v[0, h // group, rows],
                                 varlen_sees(n, causal), scale)
            inside(out[0, h, rows], o, u * o.abs() + (u + FP32) * pv, f"{what}[seq {s}, head {h}]")
            assert float((lse[0, h, rows].double() - l).abs().max()) <= LSE_ATOL, f"lse[seq {s}, head {h}]"


def check_varlen_bwd(q, k, v, lens, out, lse, dout, grads, causal, scale, first=0):
    u = HALF_STEP[q.dtype]
    group = q.shape[1] // k.shape[1]
    dq, dk, dv = grads
    row = first
    for s, n in enumerate(lens):
        rows = slice(row, row + n)
        row += n
        if n == 0:
            continue
        sees = varlen_sees(n, causal)
        for g in range(k.shape[1]):
            sums = [torch.zeros(n, q.shape[3], dtype=torch.float64, device=q.device) for _ in range(4)]
            for h in range(g * group, (g + 1) * group):
                (wq, wk, wv), (bq, bk, bv) = dense_bwd(q[0, h, rows], k[0, g, rows], v[0, g, rows], out[0, h, rows],
                                                       lse[0, h, rows], dout[0, h, rows], sees, scale, u)
                inside(dq[0, h, rows], wq, bq, f"dQ[seq {s}, head {h}]")
                for acc, x in zip(sums, (wk, wv, bk, bv)):
                    acc += x
            inside(dk[0, g, rows], sums[0], u * sums[0].abs() + sums[2], f"dK[seq {s}, head {g}]")
            inside(dv[0, g, rows], sums[1], u * sums[1].abs() + sums[3], f"dV[seq {s}, head {g}]")


def paged(gen, host, lens, Hkv, page, D, dtype, spare=3, token_major=False, fill=None):
    """Caches with the requests' tokens in shuffled pages, everything else `fill` (None: noise); the table and the
    requests' dense K and V."""
    counts = [(n + page - 1) // page for n in lens]
    pages = sum(counts) + spare
    shape = (pages, page, Hkv, D) if token_major else (pages, Hkv, page, D)
    caches, dense = [], []
    order = torch.randperm(pages, generator=host).tolist()
    table = torch.full((len(lens), max(max(counts), 1)), -1, dtype=torch.int32)
    used = 0
    for b, c in enumerate(counts):
        table[b, :c] = torch.tensor(order[used:used + c], dtype=torch.int32)
        used += c
    for _ in range(2):
        c = torch.randn(shape, generator=gen, device="cuda").to(dtype) if fill is None else \
            torch.full(shape, fill, dtype=dtype, device="cuda")
        c = c.transpose(1, 2) if token_major else c
        rows = []
        for b, n in enumerate(lens):
            x = torch.randn(n, Hkv, D, generator=gen, device="cuda").to(dtype)
            for k in range(counts[b]):
                part = x[k * page:(k + 1) * page]
                c[int(table[b, k]), :, :part.shape[0]] = part.transpose(0, 1)
            rows.append(x)
        caches.append(c)
        dense.append(rows)
    return caches[0], caches[1], table.cuda(), dense[0], dense[1]


def check_tree(q, dense_k, dense_v, lens, drafts, mask, out, lse, scale, untouched=None):
    u = HALF_STEP[q.dtype]
    B, Hq, T, D = q.shape
    for b in range(B):
        n, m = lens[b], drafts[b]
        if untouched is not None:
            assert bool((out[b, :, m:] == untouched).all()) and bool((lse[b, :, m:] == untouched).all()), f"rows past {m} of request {b}"
        if m == 0:
            continue
        sees = torch.ones(m, n, dtype=torch.bool, device="cuda")
        own = torch.ones(m, m, dtype=torch.bool, device="cuda").tril() if mask is None else \
            mask[b if mask.shape[0] > 1 else 0, :m, :m]
        sees[:, n - m:] = own
        group = Hq // dense_k[b].shape[1]
        for h in range(Hq):
            o, l, pv = dense_fwd(q[b, h, :m], dense_k[b][:, h // group], dense_v[b][:, h // group], sees, scale)
            inside(out[b, h, :m], o, u * o.abs() + (u + FP32) * pv, f"O[request {b}, head {h}]")
            got = lse[b, h, :m].double()
            gone = torch.isinf(l)
            assert torch.equal(torch.isinf(got) & (got < 0), gone), f"lse[request {b}, head {h}]"
            if not bool(gone.all()):
                assert float((got - l)[~gone].abs().max()) <= LSE_ATOL, f"lse[request {b}, head {h}]"
