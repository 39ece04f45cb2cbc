"""Packed-sequence attention and attention over a paged cache: what is measured.

Five kinds of case, named by ``case["op"]``:

  varlen_fwd  attention over prompts packed one after the other, O and lse
  varlen_bwd  its gradients dQ, dK, dV
  tree        attention of drafted tokens (a tree, or one token) over a paged cache
  plan        block tables and slot maps of a serving step from request lengths
  append      the step's keys and values written into the pages

``run`` computes each in elementary torch operations in 32 bits, or, where
``own`` is set, through the package's entry points.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def _ints(text):
    return [int(x) for x in text.split(",")]


def _text(values):
    return ",".join(str(int(v)) for v in values)


# ------------------------------------------------------------------ cases

def listed():
    return [
        # a handful of chat turns arriving together: one token, one empty slot of the batch, a few hundred tokens
        dict(name="varlen fwd short prompts", op="varlen_fwd", dtype="bf16", D=512, Hq=8, Hkv=4, causal=True,
             token_major=True, lens="1,17,0,64,130,300,45"),
        # prefill of long documents of very different lengths in one launch
        dict(name="varlen fwd long prompts", op="varlen_fwd", dtype="bf16", D=512, Hq=8, Hkv=8, causal=True,
             token_major=True, lens="8192,4999,2047,1146"),
        # an encoder's ragged batch: every token of a sequence sees the whole of it
        dict(name="varlen fwd ragged both ways", op="varlen_fwd", dtype="fp16", D=320, Hq=8, Hkv=2, causal=False,
             token_major=False, lens="511,1023,77,640,1500,333,129,900,128,2,711,257"),
        # a training step over documents packed to a fixed token budget
        dict(name="varlen bwd packed documents", op="varlen_bwd", dtype="bf16", D=512, Hq=8, Hkv=8, causal=True,
             token_major=True, lens="3001,128,2500,1,700,1200,662"),
        # a fine-tuning step on short samples at a small head dimension, shared heads
        dict(name="varlen bwd short samples", op="varlen_bwd", dtype="fp16", D=256, Hq=8, Hkv=4, causal=True,
             token_major=True, lens="90,200,33,128,310,1,64,255"),
        # decode: one token for each of a few requests with short contexts (latency)
        dict(name="tree one token few requests", op="tree", dtype="bf16", D=512, Hq=8, Hkv=4, page=16, T=1,
             lens="300,17,512,129", drafts="1,1,1,1", tree=False),
        # decode of a large batch, ragged contexts, all heads on one kv head
        dict(name="tree one token large batch", op="tree", dtype="bf16", D=512, Hq=8, Hkv=1, page=64, T=1,
             lens=_text([8192 - 113 * i for i in range(64)]), drafts=_text([1] * 64), tree=False),
        # speculative decoding: trees of up to 24 drafts over long contexts, some requests without drafts
        dict(name="tree drafts long contexts", op="tree", dtype="fp16", D=512, Hq=8, Hkv=2, page=32, T=24,
             lens="32768,9001,16384,1200,20011,777,30000,64,12345,4096,24,2500",
             drafts="24,24,17,24,8,24,24,1,24,24,24,12", tree=True),
        # a decode step of 96 requests: most stay in their page, some take a new one
        dict(name="plan decode step", op="plan", page=16, max_pages=512, lens=_text([(677 * i) % 6000 for i in range(96)]),
             new=_text([1] * 96), pad=0),
        # admission of prompts into a running batch
        dict(name="plan prompts", op="plan", page=64, max_pages=512,
             lens=_text([(991 * i) % 9000 if i % 3 else 0 for i in range(240)]),
             new=_text([1 if i % 3 else 64 + (1543 * i) % 4000 for i in range(240)]), pad=129),
        # one new token for each of 64 requests
        dict(name="append decode step", op="append", dtype="bf16", D=512, Hkv=4, page=16, pages=4096, tokens=64, pad=0,
             token_major=True),
        # prompts' keys and values
        dict(name="append prompts", op="append", dtype="bf16", D=512, Hkv=8, page=64, pages=512, tokens=16384, pad=37,
             token_major=True),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _heads(rng):
    hkv = rng.choice([1, 2, 4, 8])
    return rng.choice([h for h in (1, 2, 4, 8, 16) if h % hkv == 0]), hkv


def _split(rng, total, n, longest):
    """n lengths that add up to about total, ones and zeros among them."""
    w = [rng.expovariate(1.0) for _ in range(n)]
    lens = [min(longest, int(total * x / sum(w))) for x in w]
    for i in range(n):
        if n > 1 and rng.random() < 0.15:
            lens[i] = rng.choice([0, 1, 128, 129])
    if not any(lens):
        lens[0] = 1
    return lens


def draw(rng):
    op = rng.choice(["varlen_fwd", "varlen_bwd", "tree", "tree", "plan", "append"])
    dtype = rng.choice(["bf16", "fp16"])
    if op in ("varlen_fwd", "varlen_bwd"):
        D = rng.choice([64, 128, 256, 320, 448, 512, 512, 576, 640, 704, 832, 1024])
        hq, hkv = _heads(rng)
        # the work (sum of squares x heads x D) stays below the largest listed case's
        most = (96e6 if op == "varlen_fwd" else 17e6) * 8 * 512
        total = _log(rng, 16, 16384 if op == "varlen_fwd" else 8192)
        n = min(_log(rng, 1, 64), total)
        while True:
            lens = _split(rng, total, n, 8192)
            if sum(x * x for x in lens) * hq * D <= most and sum(lens) * hq * D <= 16384 * 8 * 512:
                break
            total = max(16, total // 2)
        return dict(op=op, dtype=dtype, D=D, Hq=hq, Hkv=hkv, causal=rng.random() < 0.75,
                    token_major=rng.random() < 0.5, lens=_text(lens))
    if op == "tree":
        D = rng.choice([64, 128, 192, 256, 320, 512, 512, 640, 768, 1024])
        hq, hkv = _heads(rng)
        T = rng.choice([1, 1, 1, 2, 5, 8, 16, 24, 33, 64])
        B = _log(rng, 1, 128)
        longest = _log(rng, 32, 32768)
        lens = [rng.randint(1, longest) for _ in range(B)]
        lens[0] = longest
        while sum(lens) * hkv * D > 129000 * 2 * 512 or sum(lens) * hq * T * D > 129000 * 8 * 24 * 512:
            lens = [max(1, x // 2) for x in lens]
        drafts = [min(x, T if rng.random() < 0.7 else rng.randint(0, T)) for x in lens]
        return dict(op=op, dtype=dtype, D=D, Hq=hq, Hkv=hkv, page=rng.choice([16, 32, 64, 128, 256]), T=T,
                    lens=_text(lens), drafts=_text(drafts), tree=T > 1 and rng.random() < 0.7)
    if op == "plan":
        B = _log(rng, 1, 512)
        page = rng.choice([16, 32, 64, 128, 256])
        lens, new = [], []
        for _ in range(B):
            fresh = rng.random() < 0.2
            lens.append(0 if fresh else rng.randint(0, 6000))
            new.append(rng.randint(1, 1500) if fresh else rng.choice([0, 1, 1, 1, 5, 24]))
        return dict(op=op, page=page, max_pages=(7600 + page - 1) // page, lens=_text(lens), new=_text(new),
                    pad=rng.choice([0, 1, 100]))
    D = rng.choice([64, 128, 256, 320, 512, 640, 1024])
    hkv = rng.choice([1, 2, 4, 8])
    page = rng.choice([16, 32, 64, 128, 256])
    tokens = _log(rng, 1, 16384 * 512 // D // 2)
    return dict(op=op, dtype=dtype, D=D, Hkv=hkv, page=page, pages=(tokens * 3 // 2 + 64) // page + 2, tokens=tokens,
                pad=rng.choice([0, 1, 50]), token_major=rng.random() < 0.7)


# ------------------------------------------------------------------ inputs

def _normal(gen, shape, dtype):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(dtype)


def _heads_tensor(gen, H, T, D, dtype, token_major):
    """[1, H, T, D], stored token by token (a projection's output) or head by head."""
    if token_major:
        return _normal(gen, (T, H, D), dtype).transpose(0, 1)[None]
    return _normal(gen, (1, H, T, D), dtype)


def _starts(lens):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return cu


def _random_tree(host, T):
    """A drafted tree: token i follows an earlier one (or the context) and sees itself and its ancestors."""
    sees = torch.zeros(T, T, dtype=torch.bool)
    for i in range(T):
        parent = int(torch.randint(-1, i, (1,), generator=host)) if i else -1
        if parent >= 0:
            sees[i] |= sees[parent]
        sees[i, i] = True
    return sees


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(1000003 + seed)
    host = torch.Generator().manual_seed(7919 + seed)
    op = case["op"]
    st = {"case": case, "op": op}
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    if op in ("varlen_fwd", "varlen_bwd"):
        dt, D, tm = DTYPES[case["dtype"]], case["D"], case["token_major"]
        lens = _ints(case["lens"])
        T = sum(lens)
        st.update(lens=lens, cu=ints(_starts(lens)), scale=D ** -0.5, causal=case["causal"],
                  q=_heads_tensor(gen, case["Hq"], T, D, dt, tm), k=_heads_tensor(gen, case["Hkv"], T, D, dt, tm),
                  v=_heads_tensor(gen, case["Hkv"], T, D, dt, tm))
        if op == "varlen_bwd":
            # what the forward of this step left behind, and the gradient that reaches O
            out, lse = _varlen_fwd(st)
            st.update(out=out, lse=lse, dout=_heads_tensor(gen, case["Hq"], T, D, dt, tm))
    elif op == "tree":
        dt, D, page = DTYPES[case["dtype"]], case["D"], case["page"]
        lens, drafts = _ints(case["lens"]), _ints(case["drafts"])
        B, T = len(lens), case["T"]
        counts = [(n + page - 1) // page for n in lens]
        pages, per = sum(counts) + 3, max(counts)
        order = torch.randperm(pages, generator=host)
        table = torch.full((B, per), -1, dtype=torch.int32)
        used = 0
        for b, c in enumerate(counts):
            table[b, :c] = order[used:used + c].to(torch.int32)
            used += c
        mask = torch.stack([_random_tree(host, T) for _ in range(B)]).cuda() if case["tree"] else None
        st.update(lens=lens, drafts=drafts, scale=D ** -0.5, mask=mask, table=table.cuda(), seq_lens=ints(lens),
                  draft_lens=ints(drafts), q=_normal(gen, (B, case["Hq"], T, D), dt),
                  k=_normal(gen, (pages, case["Hkv"], page, D), dt), v=_normal(gen, (pages, case["Hkv"], page, D), dt))
        # rows without a draft are left as they were
        st.update(out=torch.zeros(B, case["Hq"], T, D, dtype=dt, device="cuda"),
                  lse=torch.zeros(B, case["Hq"], T, device="cuda"))
    elif op == "plan":
        page, per = case["page"], case["max_pages"]
        lens, new = _ints(case["lens"]), _ints(case["new"])
        had = [(n + page - 1) // page for n in lens]
        need = [(a + b + page - 1) // page - h for a, b, h in zip(lens, new, had)]
        head = int(torch.randint(0, 50, (1,), generator=host))
        free = head + sum(need) + 7
        order = torch.randperm(free + sum(had), generator=host).to(torch.int32)
        table = torch.full((len(lens), per), -1, dtype=torch.int32)
        used = free
        for b, c in enumerate(had):
            table[b, :c] = order[used:used + c]
            used += c
        st.update(page=page, max_new=sum(new) + case["pad"], n_lens=ints(lens), n_new=ints(new), table=table.cuda(),
                  free=order[:free].cuda(), head=ints([head]))
    else:
        dt, D, page, n = DTYPES[case["dtype"]], case["D"], case["page"], case["tokens"]
        slots = torch.full((n + case["pad"],), -1, dtype=torch.int64)
        slots[:n] = torch.randperm(case["pages"] * page, generator=host)[:n]
        shape = (case["pages"], case["Hkv"], page, D)
        st.update(n=n, slots=slots.cuda(), k=_heads_tensor(gen, case["Hkv"], n + case["pad"], D, dt, case["token_major"]),
                  v=_heads_tensor(gen, case["Hkv"], n + case["pad"], D, dt, case["token_major"]),
                  k_cache=_normal(gen, shape, dt), v_cache=_normal(gen, shape, dt))
    return st


# ------------------------------------------------------------------ plain forms

def _hidden(n, device):
    i = torch.arange(n, device=device)
    return i[None, :] > i[:, None]


def _varlen_fwd(st):
    q, k, v = st["q"], st["k"], st["v"]
    group = q.shape[1] // k.shape[1]
    out = torch.zeros(q.shape, dtype=torch.float32, device=q.device)
    lse = torch.zeros(q.shape[:3], dtype=torch.float32, device=q.device)
    start = 0
    for n in st["lens"]:
        rows = slice(start, start + n)
        start += n
        if n == 0:
            continue
        hide = _hidden(n, q.device) if st["causal"] else None
        for h in range(q.shape[1]):
            s = (q[0, h, rows].float() @ k[0, h // group, rows].float().T) * st["scale"]
            if hide is not None:
                s = s.masked_fill(hide, -math.inf)
            top = s.amax(1, keepdim=True)
            e = torch.exp(s - top)
            total = e.sum(1, keepdim=True)
            out[0, h, rows] = (e @ v[0, h // group, rows].float()) / total
            lse[0, h, rows] = (top + torch.log(total))[:, 0]
    return out.to(q.dtype), lse


def _varlen_bwd(st):
    q, k, v, out, lse, dout = (st[x] for x in ("q", "k", "v", "out", "lse", "dout"))
    group = q.shape[1] // k.shape[1]
    f32 = dict(dtype=torch.float32, device=q.device)
    dq, dk, dv = (torch.zeros(x.shape, **f32) for x in (q, k, v))
    start = 0
    for n in st["lens"]:
        rows = slice(start, start + n)
        start += n
        if n == 0:
            continue
        hide = _hidden(n, q.device) if st["causal"] else None
        for h in range(q.shape[1]):
            g = h // group
            qf, kf, vf, df = (x.float() for x in (q[0, h, rows], k[0, g, rows], v[0, g, rows], dout[0, h, rows]))
            s = (qf @ kf.T) * st["scale"]
            if hide is not None:
                s = s.masked_fill(hide, -math.inf)
            p = torch.exp(s - lse[0, h, rows, None])
            delta = (df * out[0, h, rows].float()).sum(1, keepdim=True)
            ds = p * (df @ vf.T - delta) * st["scale"]
            dv[0, g, rows] += p.T @ df
            dk[0, g, rows] += ds.T @ qf
            dq[0, h, rows] = ds @ kf
    return dq.to(q.dtype), dk.to(q.dtype), dv.to(q.dtype)


def _tree(st):
    q, kc, vc, out, lse = st["q"], st["k"], st["v"], st["out"], st["lse"]
    B, Hq, T, D = q.shape
    Hkv, page = kc.shape[1], kc.shape[2]
    group = Hq // Hkv
    for b, (n, m) in enumerate(zip(st["lens"], st["drafts"])):
        if m == 0:
            continue
        ids = st["table"][b, :(n + page - 1) // page].long()
        k = kc[ids].transpose(0, 1).reshape(Hkv, -1, D)[:, :n].float()
        v = vc[ids].transpose(0, 1).reshape(Hkv, -1, D)[:, :n].float()
        x = q[b, :, :m].float().reshape(Hkv, group, m, D)
        s = torch.matmul(x.reshape(Hkv, group * m, D), k.transpose(1, 2)).reshape(Hkv, group, m, n) * st["scale"]
        if st["mask"] is None:
            hide = _hidden(m, q.device)
        else:
            hide = ~st["mask"][b, :m, :m]
        s[..., n - m:] = s[..., n - m:].masked_fill(hide, -math.inf)
        top = s.amax(-1, keepdim=True)
        e = torch.exp(s - top)
        total = e.sum(-1, keepdim=True)
        o = torch.matmul(e.reshape(Hkv, group * m, n), v).reshape(Hkv, group, m, D) / total
        out[b, :, :m] = o.reshape(Hq, m, D).to(q.dtype)
        lse[b, :, :m] = (top + torch.log(total)).reshape(Hq, m)
    return out, lse


def _plan(st):
    page, table, lens, new = st["page"], st["table"], st["n_lens"].long(), st["n_new"].long()
    zero = torch.zeros(1, dtype=torch.int64, device=table.device)
    cu = torch.cat([zero, torch.cumsum(new, 0)])
    had = (lens + page - 1) // page
    need = (lens + new + page - 1) // page - had
    taken = torch.cat([zero, torch.cumsum(need, 0)])
    col = torch.arange(table.shape[1], device=table.device)[None]
    pick = (st["head"].long() + taken[:-1])[:, None] + col - had[:, None]
    fresh = (col >= had[:, None]) & (col < (had + need)[:, None])
    table.copy_(torch.where(fresh, st["free"][pick.clamp(0, len(st["free"]) - 1)], table))
    t = torch.arange(st["max_new"], device=table.device)
    r = torch.searchsorted(cu[1:], t, right=True).clamp(max=len(lens) - 1)
    pos = lens[r] + t - cu[r]
    block = table[r, (pos // page).clamp(0, table.shape[1] - 1)].long()
    slots = torch.where(t < cu[-1], block * page + pos % page, torch.full_like(t, -1))
    return table, cu.int(), slots, (lens + new).int(), st["head"] + taken[-1].int()


def _append(st):
    n = st["n"]
    page = st["k_cache"].shape[2]
    block, at = st["slots"][:n] // page, st["slots"][:n] % page
    for cache, x in ((st["k_cache"], st["k"]), (st["v_cache"], st["v"])):
        cache[block, :, at] = x[0, :, :n].transpose(0, 1)
    return st["k_cache"], st["v_cache"]


def run(state):
    st, op = state, state["op"]
    if not own:
        return {"varlen_fwd": _varlen_fwd, "varlen_bwd": _varlen_bwd, "tree": _tree, "plan": _plan,
                "append": _append}[op](st)
    import head_dim_attention_gb300 as ffpa
    if op == "varlen_fwd":
        return ffpa.attention_varlen_fwd(st["q"], st["k"], st["v"], st["cu"], causal=st["causal"], scale=st["scale"])
    if op == "varlen_bwd":
        return ffpa.attention_varlen_bwd(st["q"], st["k"], st["v"], st["cu"], st["out"], st["lse"], st["dout"],
                                         causal=st["causal"], scale=st["scale"])
    if op == "tree":
        return ffpa.attention_tree_fwd(st["q"], st["k"], st["v"], st["table"], st["seq_lens"],
                                       draft_lens=st["draft_lens"], tree_mask=st["mask"], scale=st["scale"],
                                       out=st["out"], lse=st["lse"])
    if op == "plan":
        cu, slots, lens, head = ffpa.cache_plan(st["n_lens"], st["n_new"], st["table"], st["free"], st["head"],
                                                st["page"], st["max_new"])
        return st["table"], cu, slots, lens, head
    ffpa.cache_append(st["k"], st["v"], st["k_cache"], st["v_cache"], st["slots"])
    return st["k_cache"], st["v_cache"]


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    op = case["op"]
    if op in ("varlen_fwd", "varlen_bwd"):
        lens, D, hq, hkv = _ints(case["lens"]), case["D"], case["Hq"], case["Hkv"]
        pairs = sum(n * (n + 1) // 2 if case["causal"] else n * n for n in lens) * hq
        T = sum(lens)
        if op == "varlen_fwd":
            return {"bytes": 2 * T * D * (2 * hq + 2 * hkv) + 4 * T * hq + 4 * len(lens), "flops": 4 * pairs * D}
        return {"bytes": 2 * T * D * (4 * hq + 4 * hkv) + 4 * T * hq + 4 * len(lens), "flops": 10 * pairs * D}
    if op == "tree":
        lens, drafts, D, hq, hkv = _ints(case["lens"]), _ints(case["drafts"]), case["D"], case["Hq"], case["Hkv"]
        keys = sum(n for n, m in zip(lens, drafts) if m)
        rows = sum(drafts) * hq
        table = sum((n + case["page"] - 1) // case["page"] for n, m in zip(lens, drafts) if m)
        mask = sum(m * m for m in drafts) if case["tree"] else 0
        return {"bytes": 4 * keys * hkv * D + 4 * rows * D + 4 * rows + 4 * table + 8 * len(lens) + mask,
                "flops": 4 * D * hq * sum(n * m for n, m in zip(lens, drafts))}
    if op == "plan":
        lens, new, page = _ints(case["lens"]), _ints(case["new"]), case["page"]
        need = sum((a + b + page - 1) // page - (a + page - 1) // page for a, b in zip(lens, new))
        # lengths in and out, starts out, slots out, pages from the free list into the table, the pages written into
        return {"bytes": 16 * len(lens) + 8 * (sum(new) + case["pad"]) + 8 * need + 4 * sum(1 for x in new if x) + 12,
                "flops": 0}
    row = case["Hkv"] * case["D"] * 2
    return {"bytes": 4 * row * case["tokens"] + 8 * (case["tokens"] + case["pad"]), "flops": 0}


# ------------------------------------------------------------------ from the definitions, in 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "plan":
        return _exact_plan(case, st)
    if op == "append":
        caches = []
        for x, cache in (("k", "k_cache"), ("v", "v_cache")):
            flat = st[cache].double().transpose(1, 2).reshape(-1, case["Hkv"], case["D"])
            flat.index_copy_(0, st["slots"][:st["n"]], st[x][0].double().transpose(0, 1)[:st["n"]])
            caches.append(flat.reshape(case["pages"], case["page"], case["Hkv"], case["D"]).transpose(1, 2))
        return tuple(caches)
    if op == "tree":
        return _exact_tree(case, st)
    q, k, v = st["q"].double(), st["k"].double(), st["v"].double()
    share = case["Hq"] // case["Hkv"]
    if op == "varlen_fwd":
        out = torch.zeros_like(q)
        lse = torch.zeros(q.shape[:3], dtype=torch.float64, device=q.device)
    else:
        out, lse, dout = st["out"].double(), st["lse"].double(), st["dout"].double()
        grads = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    for a, z in zip(_starts(st["lens"]), _starts(st["lens"])[1:]):
        for lo in range(a, z, 2048):  # query rows lo .. hi - 1 against the keys they see
            hi = min(z, lo + 2048)
            end = hi if case["causal"] else z
            for h in range(case["Hq"]):
                kk, vv, qq = k[0, h // share, a:end], v[0, h // share, a:end], q[0, h, lo:hi]
                w = torch.einsum("id,jd->ij", qq, kk) * st["scale"]
                if case["causal"]:
                    w = w + torch.full_like(w, -math.inf).triu(lo - a + 1)
                if op == "varlen_fwd":
                    lse[0, h, lo:hi] = torch.logsumexp(w, 1)
                    out[0, h, lo:hi] = torch.einsum("ij,jd->id", torch.softmax(w, 1), vv)
                    continue
                w = (w - lse[0, h, lo:hi, None]).exp()
                d = dout[0, h, lo:hi]
                back = torch.einsum("id,jd->ij", d, vv) - torch.einsum("id,id->i", d, out[0, h, lo:hi])[:, None]
                back = back * w * st["scale"]
                grads[0][0, h, lo:hi] = torch.einsum("ij,jd->id", back, kk)
                grads[1][0, h // share, a:end] += torch.einsum("ij,id->jd", back, qq)
                grads[2][0, h // share, a:end] += torch.einsum("ij,id->jd", w, d)
    return (out, lse) if op == "varlen_fwd" else grads


def _exact_tree(case, st):
    q = st["q"].double()
    out, lse = st["out"].double(), st["lse"].double()
    share = case["Hq"] // case["Hkv"]
    for b, (n, m) in enumerate(zip(st["lens"], st["drafts"])):
        if not m:
            continue
        t = torch.arange(n, device=q.device)
        page, at = st["table"][b].long()[t // case["page"]], t % case["page"]
        sees = torch.ones(m, n, dtype=torch.bool, device=q.device)
        if st["mask"] is None:
            sees[:, n - m:] = torch.ones(m, m, dtype=torch.bool, device=q.device).tril()
        else:
            sees[:, n - m:] = st["mask"][b, :m, :m]
        for g in range(case["Hkv"]):
            k, v = st["k"][page, g, at].double(), st["v"][page, g, at].double()
            for h in range(g * share, (g + 1) * share):
                w = torch.einsum("id,jd->ij", q[b, h, :m], k) * st["scale"]
                w = torch.where(sees, w, torch.full_like(w, -math.inf))
                lse[b, h, :m] = torch.logsumexp(w, 1)
                out[b, h, :m] = torch.einsum("ij,jd->id", torch.softmax(w, 1), v)
    return out, lse


def _exact_plan(case, st):
    page = case["page"]
    lens, new = _ints(case["lens"]), _ints(case["new"])
    table, free, head = st["table"].tolist(), st["free"].tolist(), int(st["head"])
    slots = []
    for b, (n, m) in enumerate(zip(lens, new)):
        for t in range(n, n + m):
            if t % page == 0:
                table[b][t // page] = free[head]
                head += 1
            slots.append(table[b][t // page] * page + t % page)
    slots += [-1] * case["pad"]
    whole = lambda x: torch.tensor(x, dtype=torch.int32)  # noqa: E731
    return (whole(table), whole(_starts(new)), torch.tensor(slots, dtype=torch.int64),
            whole([a + b for a, b in zip(lens, new)]), whole([head]))
