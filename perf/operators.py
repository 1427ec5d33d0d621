"""The attention half of a served decoder layer, as measured cases: page tables and slots from
request lengths (kv_plan), head norms with the rotation and the cache write (qk_norm_rope), the
attention of new tokens over a paged cache (paged_attention) and the matrix product with bias,
activation and residual (linear).

Each operator is written twice: in elementary torch operations (`own` false) and as the calls of
this repository's package (`own` true).

Cache layout, for X = 16 bytes / element size: keys [pages][kv heads][D / X][page size][X],
values [pages][kv heads][page size][D], 8-bit scales [pages][kv heads][page size].
"""
import math
import random

import torch

own = False

FP8 = torch.float8_e4m3fn
FP8_MAX = 448.0


# ------------------------------------------------------------------ cases
def listed():
    return [
        # the page tables of a verify step (4 drafted tokens plus one) of 64 requests
        dict(name="plan verify 64 requests", op="plan", S=64, new=5, ctx=32768, page=16, pad=0, lengths=1),
        # a chunked prefill batch of many ragged requests, new and running, in a padded batch
        dict(name="plan 1024 ragged requests", op="plan", S=1024, new=40, ctx=16384, page=16, pad=700, lengths=2),
        # one verify step: the smallest call of a decode loop, 48 times per step
        dict(name="rope verify 5 tokens", op="rope", T=5, pad=0, hq=16, hkv=2, D=256, R=64, inter=False, fp8=False,
             norm=True, page=16, start=30000, factor=1.0, mscale=1.0),
        # a prefill chunk
        dict(name="rope prefill 8192 tokens", op="rope", T=8192, pad=0, hq=16, hkv=2, D=256, R=64, inter=False,
             fp8=False, norm=True, page=16, start=8192, factor=1.0, mscale=1.0),
        # a padded batch into an 8-bit cache, whole heads in the interleaved layout, far positions
        dict(name="rope ragged fp8 interleaved", op="rope", T=777, pad=23, hq=32, hkv=8, D=128, R=128, inter=True,
             fp8=True, norm=True, page=32, start=250000, factor=8.0, mscale=1.2),
        # a verify step of one request at a middling context
        dict(name="attn verify 5 x 4096", op="attn", S=1, new=5, ctx=4096, ragged=False, hq=16, hkv=2, D=256,
             fp8=False, page=16, window=0, cap=0.0, pad=0, lengths=3),
        # batched decoding: one token for each of 64 requests of very different lengths, 8-bit cache
        dict(name="attn decode 64 ragged fp8", op="attn", S=64, new=1, ctx=8192, ragged=True, hq=32, hkv=8, D=128,
             fp8=True, page=32, window=0, cap=0.0, pad=0, lengths=4),
        # the longest context, one token of one request
        dict(name="attn decode 1 x 262144", op="attn", S=1, new=1, ctx=262144, ragged=False, hq=16, hkv=2, D=256,
             fp8=False, page=16, window=0, cap=0.0, pad=0, lengths=5),
        # a mixed batch: chunks of prompts beside single tokens, a sliding window and capped scores
        dict(name="attn mixed windowed", op="attn", S=9, new=200, ctx=4000, ragged=True, hq=8, hkv=4, D=64,
             fp8=False, page=16, window=1000, cap=30.0, pad=13, lengths=6),
        # the fused query, key and value projection of a verify step
        dict(name="linear verify 5 x 5120 x 2048", op="linear", T=5, N=5120, K=2048, act="none", bias=False,
             residual=False, f32=False),
        # the output projection of a prefill chunk with the residual
        dict(name="linear 8192 x 2048 x 4096 res", op="linear", T=8192, N=2048, K=4096, act="none", bias=False,
             residual=True, f32=False),
        # an odd middling product with everything in its epilogue
        dict(name="linear 333 x 1000 x 1088 gelu", op="linear", T=333, N=1000, K=1088, act="gelu_tanh", bias=True,
             residual=True, f32=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["plan", "rope", "attn", "attn", "linear", "linear"])
    if op == "plan":
        S = _log(rng, 1, 1024)
        return dict(op=op, S=S, new=_log(rng, 1, 40), ctx=_log(rng, 64, 32768), page=rng.choice([16, 32, 64]),
                    pad=rng.choice([0, _log(rng, 1, 700)]), lengths=rng.randrange(1 << 20))
    if op == "rope":
        D = rng.choice([64, 128, 256])
        hkv = rng.choice([1, 2, 4, 8])
        return dict(op=op, T=_log(rng, 1, 6000), pad=rng.choice([0, _log(rng, 1, 100)]), hq=hkv * rng.choice([1, 2, 4]),
                    hkv=hkv, D=D, R=16 * rng.randint(0, D // 16), inter=rng.random() < 0.5, fp8=rng.random() < 0.5,
                    norm=rng.random() < 0.8, page=rng.choice([16, 32, 64]), start=_log(rng, 1, 250000),
                    factor=rng.choice([1.0, 2.0, 8.0]), mscale=rng.choice([1.0, 1.1]))
    if op == "attn":
        D = rng.choice([64, 128, 256])
        hkv = rng.choice([1, 2, 4, 8])
        S = _log(rng, 1, 64)
        new = rng.choice([1, 1, rng.randint(2, 8), _log(rng, 8, 200)])
        most = (1 << 26) // (S * hkv * D)         # the padded cache of the plain form
        ctx = _log(rng, 33, max(64, min(262144, most, (1 << 25) // (S * new * hkv * 4))))
        return dict(op=op, S=S, new=new, ctx=max(ctx, new), ragged=rng.random() < 0.7, hq=hkv * rng.choice([1, 2, 4]),
                    hkv=hkv, D=D, fp8=rng.random() < 0.5, page=rng.choice([16, 32, 64]),
                    window=rng.choice([0, 0, _log(rng, 16, 4096)]), cap=rng.choice([0.0, 0.0, 50.0]),
                    pad=rng.choice([0, rng.randint(1, 16)]), lengths=rng.randrange(1 << 20))
    T = rng.choice([rng.randint(1, 16), _log(rng, 1, 8192)])
    N = 8 * _log(rng, 4, 1000)
    K = 64 * max(1, min(_log(rng, 1, 128), (1 << 36) // (T * N * 64)))
    return dict(op=op, T=T, N=N, K=K, act=rng.choice(["none", "none", "silu", "gelu", "gelu_tanh", "relu"]),
                bias=rng.random() < 0.5, residual=rng.random() < 0.5, f32=rng.random() < 0.3)


def _lengths(case):
    """(cached, new) tokens of each request: whole contexts, or spread over their logarithm."""
    r = random.Random(case["lengths"])
    cached, new = [], []
    for s in range(case["S"]):
        if case["op"] == "plan":
            n = case["new"] if case["new"] <= 8 else r.choice([0, 1, 1, 5, r.randint(1, case["new"])])
            total = max(n, _log(r, 1, case["ctx"]))
            cached.append(total - n)
        else:
            n = case["new"] if case["new"] <= 8 or not case["ragged"] else r.choice([1, r.randint(1, case["new"])])
            total = max(n, _log(r, 16, case["ctx"])) if case["ragged"] else case["ctx"]
            cached.append(total - n)
        new.append(n)
    if case["op"] == "attn":                       # one request at the whole context
        cached[case["S"] // 2] = case["ctx"] - new[case["S"] // 2]
    return cached, new


def _pages(n, page):
    return -(-n // page)


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    return _PREPARE[case["op"]](case, torch.Generator(device="cuda").manual_seed(seed))


def _ints(v):
    return torch.tensor(v, dtype=torch.int32).cuda()


def _prepare_plan(case, g):
    cached, new = _lengths(case)
    S, P = case["S"], case["page"]
    W = _pages(case["ctx"], P)
    have = torch.tensor([_pages(c, P) for c in cached], device="cuda")
    total = S * W
    ids = torch.randperm(total, device="cuda", generator=g).to(torch.int32)
    table = torch.where(torch.arange(W, device="cuda")[None] < have[:, None], ids.view(S, W), -1).to(torch.int32)
    take = sum(_pages(c + n, P) - _pages(c, P) for c, n in zip(cached, new))
    free = torch.randperm(total, device="cuda", generator=g)[: take + 7].to(torch.int32).contiguous()
    T = sum(new) + case["pad"]
    st = dict(op="plan", S=S, W=W, P=P, T=T, cached=_ints(cached), new=_ints(new), table=table, free=free)
    if own:
        from routed_expert_ffn_amd import moe
        st["out"] = moe.KVPlan.allocate(S, T)      # a serving loop keeps these buffers
    return st


def _randn(g, *shape):
    return torch.randn(shape, device="cuda", generator=g)


def _prepare_rope(case, g):
    T, pad, hq, hkv, D, R, P = (case[k] for k in ("T", "pad", "hq", "hkv", "D", "R", "page"))
    rows = T + pad
    qkv = _randn(g, rows, hq + 2 * hkv, D)
    qkv *= torch.exp(0.3 * _randn(g, 1, hq + 2 * hkv, 1))          # heads of different sizes
    qkv = qkv.view(rows, -1).to(torch.bfloat16)
    pages = _pages(T, P) + 1
    order = torch.randperm(pages, device="cuda", generator=g)
    t = torch.arange(rows, device="cuda")
    slots = torch.where(t < T, order[torch.clamp(t // P, max=pages - 1)] * P + t % P, -1).to(torch.int32)
    start = int(torch.randint(0, case["start"] + 1, (1,), generator=g, device="cuda"))
    positions = (start + t).to(torch.int32)
    base = 10000000.0
    freq = (base ** (-torch.arange(0, R, 2, dtype=torch.float64) / max(R, 1)) / case["factor"]).float().cuda()
    st = dict(op="rope", hq=hq, hkv=hkv, D=D, R=R, P=P, pages=pages, inter=case["inter"], mscale=case["mscale"],
              eps=1e-6, qkv=qkv, slots=slots, positions=positions, freq=freq if R else None,
              qw=(1 + 0.1 * _randn(g, D)) if case["norm"] else None,
              kw=(1 + 0.1 * _randn(g, D)) if case["norm"] else None,
              q_out=torch.zeros(rows, hq, D, dtype=torch.bfloat16, device="cuda"))
    dt = FP8 if case["fp8"] else torch.bfloat16
    X = 16 if case["fp8"] else 8
    st["k"] = torch.zeros(pages, hkv, D // X, P, X, device="cuda", dtype=torch.uint8 if case["fp8"] else dt).view(dt)
    st["v"] = torch.zeros(pages, hkv, P, D, device="cuda", dtype=torch.uint8 if case["fp8"] else dt).view(dt)
    st["ks"] = torch.zeros(pages, hkv, P, device="cuda") if case["fp8"] else None
    st["vs"] = torch.zeros(pages, hkv, P, device="cuda") if case["fp8"] else None
    if own:
        from routed_expert_ffn_amd import moe
        st["cache"] = moe.KVCache(st["k"], st["v"], st["ks"], st["vs"])
    return st


def _prepare_attn(case, g):
    cached, new = _lengths(case)
    S, hq, hkv, D, P = (case[k] for k in ("S", "hq", "hkv", "D", "page"))
    total = [c + n for c, n in zip(cached, new)]
    W = _pages(case["ctx"], P)
    used = torch.tensor([_pages(n, P) for n in total], device="cuda")
    pages = int(used.sum()) + 1
    order = torch.randperm(pages, device="cuda", generator=g)
    first = torch.cumsum(used, 0) - used
    w = torch.arange(W, device="cuda")
    table = torch.where(w[None] < used[:, None], order[torch.clamp(first[:, None] + w[None], max=pages - 1)], 0)
    rows = sum(new) + case["pad"]
    q = _randn(g, rows, hq, D).to(torch.bfloat16)
    # keys after a head norm, with a few strong directions; values of the heads' own sizes
    k = _randn(g, pages, hkv, P, D)
    k += 0.5 * _randn(g, 1, hkv, 1, D)
    v = _randn(g, pages, hkv, P, D) * torch.exp(0.3 * _randn(g, 1, hkv, 1, 1))
    ks = vs = None
    X = 16 if case["fp8"] else 8
    if case["fp8"]:
        ks, vs = k.abs().amax(-1) / FP8_MAX, v.abs().amax(-1) / FP8_MAX
        k, v = (k / ks[..., None]).to(FP8).view(torch.uint8), (v / vs[..., None]).to(FP8).view(torch.uint8)
    else:
        k, v = k.to(torch.bfloat16), v.to(torch.bfloat16)
    k = k.view(pages, hkv, P, D // X, X).transpose(2, 3).contiguous()
    if case["fp8"]:
        k, v = k.view(FP8), v.view(FP8)
    offs = [0]
    for n in new:
        offs.append(offs[-1] + n)
    st = dict(op="attn", S=S, W=W, P=P, hq=hq, hkv=hkv, D=D, most=max(new), window=case["window"], cap=case["cap"],
              scale=D ** -0.5, q=q, k=k, v=v, ks=ks, vs=vs, table=table.to(torch.int32).contiguous(),
              offs=_ints(offs), lens=_ints(total), out=torch.zeros_like(q))
    if own:
        from routed_expert_ffn_amd import moe
        st["cache"] = moe.KVCache(k, v, ks, vs)
        # a serving loop keeps its workspace
        st["ws"] = torch.empty(moe.paged_attention_workspace_size(rows, hq, hkv, D, S), dtype=torch.uint8,
                               device="cuda")
    return st


def _prepare_linear(case, g):
    T, N, K = case["T"], case["N"], case["K"]
    x = _randn(g, T, K).to(torch.bfloat16)
    w = (_randn(g, N, K) * K ** -0.5).to(torch.bfloat16)
    out_dtype = torch.float32 if case["f32"] else torch.bfloat16
    st = dict(op="linear", x=x, w=w, act=case["act"], out_dtype=out_dtype,
              bias=0.1 * _randn(g, N) if case["bias"] else None,
              residual=_randn(g, T, N).to(out_dtype) if case["residual"] else None)
    if own:
        from routed_expert_ffn_amd import moe
        st["out"] = torch.empty(T, N, dtype=out_dtype, device="cuda")
        st["ws"] = torch.empty(max(1, moe.linear_workspace_size(T, N, K)), dtype=torch.uint8, device="cuda")
    return st


_PREPARE = dict(plan=_prepare_plan, rope=_prepare_rope, attn=_prepare_attn, linear=_prepare_linear)


# ------------------------------------------------------------------ one pass
def run(st):
    if own:
        return _run_own(st)
    return _RUN[st["op"]](st)


def _run_own(st):
    from routed_expert_ffn_amd import moe
    op = st["op"]
    if op == "plan":
        p = moe.kv_plan(st["cached"], st["new"], st["free"], st["table"], st["P"], st["T"], out=st["out"])
        return [st["table"], p.q_offsets, p.kv_len, p.positions, p.slots, p.counts]
    if op == "rope":
        moe.qk_norm_rope(st["qkv"], st["cache"], st["positions"], st["slots"], q_weight=st["qw"], k_weight=st["kw"],
                         eps=st["eps"], inv_freq=st["freq"], interleaved=st["inter"], rope_scale=st["mscale"],
                         out=st["q_out"])
        return [st["q_out"], st["k"], st["v"], st["ks"], st["vs"]]
    if op == "attn":
        return moe.paged_attention(st["q"], st["cache"], st["table"], st["offs"], st["lens"], scale=st["scale"],
                                   softcap=st["cap"], window=st["window"], out=st["out"], workspace=st["ws"])
    return moe.linear(st["x"], st["w"], bias=st["bias"], act=st["act"], residual=st["residual"], out=st["out"],
                      workspace=st["ws"])


def _run_plan(st):
    S, W, P, T = st["S"], st["W"], st["P"], st["T"]
    cached = torch.clamp(st["cached"].long(), 0, W * P)
    new = torch.minimum(torch.clamp(st["new"].long(), min=0), W * P - cached)
    offs = torch.clamp(torch.cat([new.new_zeros(1), torch.cumsum(new, 0)]), max=T)
    lens = cached + offs[1:] - offs[:-1]
    have, need = (cached + P - 1) // P, (lens + P - 1) // P
    take = need - have
    first = torch.cumsum(take, 0) - take
    w = torch.arange(W, device="cuda")[None]
    at = first[:, None] + w - have[:, None]
    fresh = (w >= have[:, None]) & (w < need[:, None])
    n = st["free"].numel()
    page = torch.where(at < n, st["free"].long()[torch.clamp(at, 0, n - 1)], -1)
    st["table"].copy_(torch.where(fresh, page, st["table"].long()))
    t = torch.arange(T, device="cuda")
    s = torch.clamp(torch.searchsorted(offs, t, right=True) - 1, max=S - 1)
    real = t < offs[-1]
    pos = torch.where(real, cached[s] + t - offs[s], 0)
    page = st["table"].long()[s, torch.clamp(pos // P, max=W - 1)]
    slots = torch.where(real & (page >= 0), page * P + pos % P, -1)
    counts = torch.stack([offs[-1], take.sum()])
    i32 = torch.int32
    return [st["table"], offs.to(i32), lens.to(i32), pos.to(i32), slots.to(i32), counts.to(i32)]


def _rotate(x, cos, sin, inter):
    """x [T][heads][R] fp32 by angles given as cos, sin [T][R / 2]."""
    half = x.shape[-1] // 2
    a, b = (x[..., 0::2], x[..., 1::2]) if inter else (x[..., :half], x[..., half:])
    c, s = cos[:, None], sin[:, None]
    u, v = a * c - b * s, b * c + a * s
    return torch.stack([u, v], -1).flatten(-2) if inter else torch.cat([u, v], -1)


def _run_rope(st):
    hq, hkv, D, R, P = (st[k] for k in ("hq", "hkv", "D", "R", "P"))
    x = st["qkv"].float().view(-1, hq + 2 * hkv, D)
    q, k, v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
    if st["qw"] is not None:
        q = q * torch.rsqrt((q * q).mean(-1, keepdim=True) + st["eps"]) * st["qw"]
        k = k * torch.rsqrt((k * k).mean(-1, keepdim=True) + st["eps"]) * st["kw"]
    if R:
        angle = st["positions"].double()[:, None] * st["freq"].double()[None]
        cos, sin = (torch.cos(angle) * st["mscale"]).float(), (torch.sin(angle) * st["mscale"]).float()
        q = torch.cat([_rotate(q[..., :R], cos, sin, st["inter"]), q[..., R:]], -1)
        k = torch.cat([_rotate(k[..., :R], cos, sin, st["inter"]), k[..., R:]], -1)
    real = st["slots"] >= 0
    st["q_out"].copy_(torch.where(real[:, None, None], q.to(torch.bfloat16), st["q_out"]))
    at = st["slots"][real].long()
    page, off = at // P, at % P
    k, v = k[real], v[real]
    if st["ks"] is not None:
        ks, vs = k.abs().amax(-1) / FP8_MAX, v.abs().amax(-1) / FP8_MAX
        st["ks"][page, :, off], st["vs"][page, :, off] = ks, vs
        k = (k / torch.where(ks > 0, ks, 1)[..., None]).to(FP8).view(torch.uint8)
        v = (v / torch.where(vs > 0, vs, 1)[..., None]).to(FP8).view(torch.uint8)
        st["k"].view(torch.uint8)[page, :, :, off] = k.view(-1, hkv, D // 16, 16)
        st["v"].view(torch.uint8)[page, :, off] = v
    else:
        st["k"][page, :, :, off] = k.to(torch.bfloat16).view(-1, hkv, D // 8, 8)
        st["v"][page, :, off] = v.to(torch.bfloat16)
    return [st["q_out"], st["k"], st["v"], st["ks"], st["vs"]]


def _gathered(st):
    """The requests' keys and values as [S][kv heads][W * P][D] fp32."""
    S, W, P, hkv, D = (st[k] for k in ("S", "W", "P", "hkv", "D"))
    at = st["table"].long().view(-1)
    raw = (lambda t: t.view(torch.uint8)) if st["ks"] is not None else (lambda t: t)
    k = raw(st["k"])[at].transpose(2, 3).reshape(S * W, hkv, P, D)
    v = raw(st["v"])[at]
    if st["ks"] is not None:
        k = k.view(FP8).float() * st["ks"][at][..., None]
        v = v.view(FP8).float() * st["vs"][at][..., None]
    shape = lambda t: t.float().view(S, W, hkv, P, D).transpose(1, 2).reshape(S, hkv, W * P, D)  # noqa: E731
    return shape(k), shape(v)


def _run_attn(st):
    S, hq, hkv, D, M = (st[k] for k in ("S", "hq", "hkv", "D", "most"))
    offs, lens = st["offs"].long(), st["lens"].long()
    n = offs[1:] - offs[:-1]
    i = torch.arange(M, device="cuda")
    row = torch.clamp(offs[:-1, None] + i, max=st["q"].shape[0] - 1)               # [S][M]
    q = st["q"][row].float().view(S, M, hkv, hq // hkv, D).permute(0, 2, 3, 1, 4).reshape(S, hkv, -1, D)
    k, v = _gathered(st)
    s = torch.matmul(q, k.transpose(2, 3).contiguous()) * st["scale"]              # [S][hkv][group * M][W * P]
    if st["cap"] > 0:
        s = st["cap"] * torch.tanh(s / st["cap"])
    j = torch.arange(k.shape[2], device="cuda")
    p = (lens - n)[:, None] + i                                                    # positions [S][M]
    seen = j[None, None] <= p[..., None]
    if st["window"] > 0:
        seen &= j[None, None] > p[..., None] - st["window"]
    seen = seen[:, None, None].expand(-1, hkv, hq // hkv, -1, -1).reshape(s.shape)
    s = s.masked_fill(~seen, -math.inf)
    top = s.amax(-1, keepdim=True)
    e = torch.exp(s - torch.where(torch.isinf(top), 0, top))
    total = e.sum(-1, keepdim=True)
    o = torch.matmul(e, v) / torch.where(total > 0, total, 1)
    o = o.view(S, hkv, hq // hkv, M, D).permute(0, 3, 1, 2, 4).reshape(S, M, hq, D).to(torch.bfloat16)
    real = i[None] < n[:, None]
    st["out"][row[real]] = o[real]
    return st["out"]


def _activation(z, act):
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    if act == "relu":
        return torch.clamp(z, min=0)
    return z


def _run_linear(st):
    z = torch.matmul(st["x"].float(), st["w"].float().t())
    if st["bias"] is not None:
        z = z + st["bias"]
    z = _activation(z, st["act"])
    if st["residual"] is not None:
        z = z + st["residual"].float()
    return z.to(st["out_dtype"])


_RUN = dict(plan=_run_plan, rope=_run_rope, attn=_run_attn, linear=_run_linear)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    op = case["op"]
    if op == "plan":
        cached, new = _lengths(case)
        take = sum(_pages(c + n, case["page"]) - _pages(c, case["page"]) for c, n in zip(cached, new))
        T = sum(new) + case["pad"]
        # lengths in; offsets, lengths, positions, slots out; each new page read and written once; the page
        # that a request's first new token may fall into
        return dict(bytes=4 * (2 * case["S"] + 2 * case["S"] + 1 + 2 * T + 2 * take + case["S"] + 2), flops=0)
    if op == "rope":
        T, hq, hkv, D = case["T"], case["hq"], case["hkv"], case["D"]
        cache = 2 * T * hkv * (D + 4 if case["fp8"] else 2 * D)
        return dict(bytes=2 * T * (hq + 2 * hkv) * D + 2 * T * hq * D + cache + 8 * (T + case["pad"]),
                    flops=T * (hq + hkv) * (4 * D + 3 * case["R"]))
    if op == "attn":
        cached, new = _lengths(case)
        kv = pairs = 0
        for c, n in zip(cached, new):
            lo = max(0, c + 1 - case["window"]) if case["window"] else 0
            kv += c + n - lo
            pairs += sum(min(c + i + 1, case["window"] or c + i + 1) for i in range(n))
        element = (case["D"] + 4) if case["fp8"] else 2 * case["D"]
        return dict(bytes=2 * kv * case["hkv"] * element + 4 * sum(new) * case["hq"] * case["D"]
                    + 4 * kv // case["page"], flops=4 * pairs * case["hq"] * case["D"])
    T, N, K = case["T"], case["N"], case["K"]
    e = 4 if case["f32"] else 2
    return dict(bytes=2 * (T * K + N * K) + e * T * N * (2 if case["residual"] else 1) + (4 * N if case["bias"] else 0),
                flops=2 * T * N * K)


# ------------------------------------------------------------------ the definitions in 64 bits
def exact(case, seed):
    return _EXACT[case["op"]](case, prepare(case, seed))


def _exact_plan(case, st):
    return None                                    # whole numbers only


def _to_fp8(y):
    """float64 -> the nearest e4m3 value (ties to even), as float64: 3 fraction bits, least exponent -6."""
    e = torch.clamp(torch.floor(torch.log2(torch.clamp(y.abs(), min=2.0 ** -30))), min=-6)
    step = torch.exp2(e - 3)
    return torch.clamp(torch.round(y / step) * step, -FP8_MAX, FP8_MAX)


def _exact_rope(case, st):
    hq, hkv, D, R, P = st["hq"], st["hkv"], st["D"], st["R"], st["P"]
    x = st["qkv"].double().reshape(-1, hq + 2 * hkv, D)
    T = case["T"]
    heads = []
    for h in range(hq + 2 * hkv):
        y = x[:T, h]
        w = None if st["qw"] is None or h >= hq + hkv else st["qw" if h < hq else "kw"].double()
        if w is not None:
            y = y / torch.sqrt((y ** 2).sum(-1, keepdim=True) / D + st["eps"]) * w
        if R and h < hq + hkv:
            first = torch.arange(0, R, 2, device="cuda") if st["inter"] else torch.arange(R // 2, device="cuda")
            second = first + (1 if st["inter"] else R // 2)
            turn = torch.polar(torch.full((T, R // 2), float(st["mscale"]), dtype=torch.float64, device="cuda"),
                               st["positions"][:T, None].double() * st["freq"].double())
            z = torch.complex(y[:, first], y[:, second]) * turn
            y = y.clone()
            y[:, first], y[:, second] = z.real, z.imag
        heads.append(y)
    y = torch.stack(heads, 1)
    q = st["q_out"].double()
    q[:T] = y[:, :hq]
    slots = st["slots"][:T].long()
    X = st["k"].shape[-1]
    k = torch.zeros(st["pages"] * P, hkv, D, dtype=torch.float64, device="cuda")
    v, ks, vs = torch.zeros_like(k), None, None
    kt, vt = y[:, hq:hq + hkv], y[:, hq + hkv:]
    if case["fp8"]:
        ks, vs = (torch.zeros(st["pages"] * P, hkv, dtype=torch.float64, device="cuda") for _ in range(2))
        ks[slots], vs[slots] = kt.abs().amax(-1) / FP8_MAX, vt.abs().amax(-1) / FP8_MAX
        kt, vt = _to_fp8(kt / ks[slots][..., None]), _to_fp8(vt / vs[slots][..., None])
        ks, vs = (t.view(-1, P, hkv).transpose(1, 2) for t in (ks, vs))
    k[slots], v[slots] = kt, vt
    return [q, k.view(-1, P, hkv, D // X, X).permute(0, 2, 3, 1, 4), v.view(-1, P, hkv, D).permute(0, 2, 1, 3), ks, vs]


def _exact_attn(case, st):
    hq, hkv, D, P = st["hq"], st["hkv"], st["D"], st["P"]
    out = st["out"].double()
    offs, lens = st["offs"].tolist(), st["lens"].tolist()
    for s in range(case["S"]):
        a, b, L = offs[s], offs[s + 1], lens[s]
        at = st["table"][s, :_pages(L, P)].long()
        j = torch.arange(L, device="cuda")
        p = torch.arange(L - (b - a), L, device="cuda")
        seen = (j[None] <= p[:, None]) & ((j[None] > p[:, None] - case["window"]) if case["window"] else True)
        for h in range(hkv):
            k = st["k"][at, h].double() if st["ks"] is None else st["k"].view(torch.uint8)[at, h].view(FP8).double()
            k = k.permute(0, 2, 1, 3).reshape(-1, D)[:L]
            v = st["v"][at, h].double() if st["vs"] is None else st["v"].view(torch.uint8)[at, h].view(FP8).double()
            v = v.reshape(-1, D)[:L]
            if st["ks"] is not None:
                k = k * st["ks"][at, h].double().reshape(-1)[:L, None]
                v = v * st["vs"][at, h].double().reshape(-1)[:L, None]
            for g in range(h * (hq // hkv), (h + 1) * (hq // hkv)):
                x = st["q"][a:b, g].double() @ k.t() * st["scale"]
                if case["cap"]:
                    x = case["cap"] * torch.tanh(x / case["cap"])
                out[a:b, g] = torch.softmax(torch.where(seen, x, -math.inf), -1) @ v
    return out


def _exact_linear(case, st):
    z = torch.nn.functional.linear(st["x"].double(), st["w"].double(), None if st["bias"] is None
                                   else st["bias"].double())
    f = torch.nn.functional
    z = dict(none=lambda t: t, silu=f.silu, gelu=f.gelu, relu=f.relu,
             gelu_tanh=lambda t: f.gelu(t, approximate="tanh"))[case["act"]](z)
    return z if st["residual"] is None else z + st["residual"].double()


_EXACT = dict(plan=_exact_plan, rope=_exact_rope, attn=_exact_attn, linear=_exact_linear)
