"""GPU: the attention half (page tables and slots, head norms + rotation + cache
write, paged attention, dense products) against plain 64-bit forms, at the
sizes and masks where each can go wrong."""
import math

import numpy as np
import pytest
import torch

from routed_expert_ffn_amd import moe

from . import attn_ref as ref

pytestmark = pytest.mark.gpu
BF, FP8 = torch.bfloat16, torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    moe.load()
    yield
    torch.cuda.synchronize()


def rng(seed):
    return torch.Generator().manual_seed(seed)


def ints(v):
    return torch.tensor(np.asarray(v, np.int32).reshape(-1)).cuda()


# ---------------------------------------------------------------- page tables and slots
PLANS = [
    # (cached, new, free pages, table width, page size, rows)
    ([0], [1], 3, 4, 16, 1),
    ([0], [0], 0, 1, 16, 0),
    ([15, 16, 17, 0, 31], [1, 1, 1, 5, 2], 9, 4, 16, 10),
    ([5, 0, 100], [3, 0, 60], 9, 16, 16, 80),                      # a padded batch
    ([5, 0, 100], [3, 40, 60], 9, 16, 16, 50),                     # rows run out inside the last request
    ([5, 0, 100], [3, 40, 60], 2, 16, 16, 120),                    # pages run out
    ([60, 64, 70, -3], [10, 9, 8, -1], 9, 4, 16, 40),              # the table is full, lengths past it, negative ones
    ([7] * 300, [1, 2, 3] * 100, 700, 3, 16, 640),                 # more requests than threads of a block
    (list(range(0, 2100)), [2] * 2100, 300, 70, 32, 4300),
    ([1023] * 4096, [2, 0] * 2048, 3000, 3, 1024, 4100),           # the most requests, the largest page
]


@pytest.mark.parametrize("case", range(len(PLANS)))
def test_kv_plan(case):
    cached, new, n_free, W, page, T = PLANS[case]
    g = np.random.default_rng(case)
    S = len(cached)
    table = g.permutation(S * W).reshape(S, W).astype(np.int32)
    if case == 3:
        table[2, 6] = -1                                           # a page that is not there
    free = g.permutation(5000)[:n_free].astype(np.int32)
    want = ref.plan(cached, new, free, table, page, T)
    dt = torch.from_numpy(table).cuda()
    for _ in range(2):                                             # a repeated call gives the same
        p = moe.kv_plan(ints(cached), ints(new), ints(free), dt, page, T)
        torch.cuda.synchronize()
        for name, t, w in zip(("q_offsets", "kv_len", "positions", "slots", "counts", "table"),
                              (p.q_offsets, p.kv_len, p.positions, p.slots, p.counts, dt), want):
            assert np.array_equal(t.cpu().numpy(), w), name


# ---------------------------------------------------------------- norms, rotation, cache write
ROPES = [
    # T, Hq, Hkv, D, rope_dim, interleaved, fp8, norm, page, first position, rope_scale
    (1, 1, 1, 64, 64, False, False, True, 16, 0, 1.0),
    (5, 16, 2, 256, 64, False, False, True, 16, 30000, 1.0),
    (5, 16, 2, 256, 64, True, True, True, 16, 30000, 1.0),
    (3, 8, 8, 128, 128, True, False, True, 64, 262000, 1.25),
    (3, 6, 2, 128, 128, False, True, False, 32, 7, 1.0),
    (4, 5, 1, 64, 16, False, True, True, 16, 1 << 30, 1.0),
    (7, 3, 3, 64, 0, False, False, True, 16, 3, 1.0),               # no rotation
    (2, 2, 1, 256, 256, False, False, False, 1024, 100, 1.0),       # no norm
    (300, 4, 2, 128, 96, False, True, True, 16, 5000, 1.1),         # many rows: 16 per block
    (259, 7, 1, 64, 32, True, False, True, 16, 11, 1.0),
    (273, 3, 2, 256, 256, False, False, True, 32, 9, 1.0),
]


def rope_inputs(case):
    T, Hq, Hkv, D, R, inter, fp8, norm, page, start, mscale = case
    g = rng(T * 1000 + D)
    n = Hq + 2 * Hkv
    qkv = (torch.randn(T, n * D, generator=g) * torch.exp(torch.randn(T, 1, generator=g))).to(BF)
    if T > 2:
        qkv.view(T, n, D)[1, -1] = 0                                # a head of zeros
    pages = -(-T // page) + 2
    order = torch.randperm(pages * page, generator=g)[:T].to(torch.int32)
    if T > 3:
        order[T // 2] = -1                                          # padding rows
        order[T - 1] = pages * page
    pos = torch.arange(start, start + T, dtype=torch.int64).to(torch.int32)
    freq = (10000.0 ** (-torch.arange(0, R, 2).double() / max(R, 1))).float() if R else None
    qw = (1 + 0.2 * torch.randn(D, generator=g)) if norm else None
    kw = (1 + 0.2 * torch.randn(D, generator=g)) if norm else None
    return qkv, pages, order, pos, freq, qw, kw


@pytest.mark.parametrize("case", ROPES, ids=lambda c: "-".join(map(str, c)))
def test_qk_norm_rope(case):
    T, Hq, Hkv, D, R, inter, fp8, norm, page, start, mscale = case
    qkv, pages, slots, pos, freq, qw, kw = rope_inputs(case)
    want, size = ref.qk_norm_rope(qkv, Hq, Hkv, D, pos, qw, kw, 1e-5, freq, inter, mscale)
    slack = ref.norm_rope_slack(size, D)
    dev = lambda t: None if t is None else t.cuda()  # noqa: E731
    cache = moe.KVCache.allocate(pages, page, Hkv, D, FP8 if fp8 else BF)
    for t in (cache.k, cache.v):
        t.view(torch.uint8).fill_(0x41)
    if fp8:
        cache.k_scale.fill_(7.0)
        cache.v_scale.fill_(7.0)
    q = torch.full((T, Hq, D), 9.0, dtype=BF, device="cuda")
    wide = torch.full((T, qkv.shape[1] + 40), math.nan, dtype=BF, device="cuda")      # rows that lie apart
    wide[:, :qkv.shape[1]] = qkv.cuda()
    moe.qk_norm_rope(wide[:, :qkv.shape[1]], cache, dev(pos), dev(slots), dev(qw), dev(kw), 1e-5, dev(freq), inter,
                     mscale, out=q)
    torch.cuda.synchronize()
    real = (slots >= 0) & (slots < pages * page)
    got = q.cpu().double()
    assert bool((got[~real] == 9.0).all()), "a padding row's output was written"
    bound = ref.BF16_HALF * want[:, :Hq].abs() + 1.01 * slack[:, :Hq]
    assert bool(((got - want[:, :Hq]).abs() <= bound)[real].all())
    at = slots[real].long()
    untouched = torch.ones(pages * page, dtype=torch.bool)
    untouched[at] = False
    for name, t, sc, h0 in (("k", cache.k, cache.k_scale, Hq), ("v", cache.v, cache.v_scale, Hq + Hkv)):
        raw = t.cpu()
        rows = ref.k_rows(raw.view(torch.uint8) if fp8 else raw) if name == "k" else (raw.view(torch.uint8) if fp8 else raw)
        rows = rows.transpose(1, 2).reshape(pages * page, Hkv, D)
        flat = rows if fp8 else rows.contiguous().view(torch.uint8)
        assert bool((flat[untouched] == 0x41).all()), f"{name}: another slot was written"
        y, e = want[real][:, h0:h0 + Hkv], slack[real][:, h0:h0 + Hkv]
        if name == "v":
            e = e * 0
        if not fp8:
            assert bool(((rows[at].double() - y).abs() <= ref.BF16_HALF * y.abs() + 1.01 * e).all()), name
        else:
            s = sc.cpu().transpose(1, 2).reshape(pages * page, Hkv)
            assert bool((s[untouched] == 7.0).all())
            s = s[at].double()
            amax = y.abs().amax(-1)
            assert bool(((s - amax / 448).abs() <= 1.01 * e.amax(-1) / 448 + 2 * ref.F32_HALF * s).all())
            val = rows[at].contiguous().view(FP8).float().double() * s[..., None]
            # half a step of e4m3: relative 2^-4, at least half of 2^-9 (its subnormal step) of the scale; the scale's
            # own error moves the element by the same share
            tol = torch.maximum(ref.FP8_HALF * y.abs(), 2.0 ** -10 * s[..., None]) + 1.2 * e + 4 * ref.F32_HALF * y.abs() \
                + 1.2 * (e.amax(-1) / torch.clamp(amax, min=1e-30))[..., None] * y.abs()
            assert bool(((val - y).abs() <= tol).all()), name


@pytest.mark.parametrize("fp8", [False, True])
def test_qk_norm_rope_keeps_infinities_in_their_head(fp8):
    T, Hq, Hkv, D = 3, 2, 2, 64
    qkv = torch.randn(T, Hq + 2 * Hkv, D, generator=rng(50)).to(BF)
    clean = qkv.clone()
    qkv[0, 0, 3], qkv[1, 2, 5], qkv[2, 5, 7] = math.nan, math.inf, math.inf           # a q, a k and a v head
    outs = []
    for x in (clean, qkv):
        cache = moe.KVCache.allocate(1, 16, Hkv, D, FP8 if fp8 else BF)
        for t in (cache.k, cache.v):
            t.view(torch.uint8).fill_(0)
        q = moe.qk_norm_rope(x.view(T, -1).cuda(), cache, ints([0, 1, 2]), ints([0, 1, 2]),
                             torch.ones(D, device="cuda"), torch.ones(D, device="cuda"))
        torch.cuda.synchronize()
        rows = ref.k_rows(cache.k.view(torch.uint8).cpu()).contiguous().view(FP8) if fp8 else ref.k_rows(cache.k.cpu())
        k = ref.as_values(rows, cache.k_scale.cpu() if fp8 else None)[0, :, :3]
        v = ref.as_values(cache.v.cpu(), cache.v_scale.cpu() if fp8 else None)[0, :, :3]
        outs.append((q.cpu().double(), k, v))
    for name, a, b, bad in zip("qkv", *outs, ((0, 0), (0, 1), (1, 2))):
        same = torch.ones(a.shape[:2], dtype=torch.bool)
        same[bad] = False
        assert torch.equal(a[same], b[same]), name
        assert not bool(torch.isfinite(b[bad]).all()), name


# ---------------------------------------------------------------- paged attention
def attn_state(lens, new, Hq, Hkv, D, page, fp8, seed=0, pad=0, W=None, spare=3, poison=True):
    """q, a cache whose unused places hold NaN, a page table whose unused entries are garbage."""
    g = rng(seed)
    S = len(lens)
    W = W or max(1, max(-(-n // page) for n in lens)) + 1
    used = [min(-(-n // page), W) for n in lens]
    pages = sum(used) + spare
    order = torch.randperm(pages, generator=g)
    table = torch.full((S, W), 0x7FFFFFF0, dtype=torch.int32)
    k = torch.full((pages, Hkv, page, D), math.nan if poison else 0.0)
    v = torch.full((pages, Hkv, page, D), math.nan if poison else 0.0)
    at = 0
    for s in range(S):
        for j in range(used[s]):
            p = int(order[at])
            at += 1
            table[s, j] = p
            m = min(page, lens[s] - j * page)
            k[p, :, :m] = torch.randn(Hkv, m, D, generator=g) + 0.5
            v[p, :, :m] = torch.randn(Hkv, m, D, generator=g) * 2
    T = sum(new) + pad
    q = torch.randn(T, Hq, D, generator=g).to(BF)
    offs = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    ks = vs = None
    if fp8:
        ks, vs = k.abs().amax(-1) / 448, v.abs().amax(-1) / 448
        k, v = (k / ks[..., None]).to(FP8), (v / vs[..., None]).to(FP8)
        kl = ref.k_layout(k.view(torch.uint8), 16).view(FP8)
    else:
        k, v = k.to(BF), v.to(BF)
        kl = ref.k_layout(k, 8)
    dev = lambda t: None if t is None else t.cuda()  # noqa: E731
    cache = moe.KVCache(dev(kl), dev(v.contiguous()), dev(ks), dev(vs))
    return dict(q=q, k=ref.as_values(k, ks), v=ref.as_values(v, vs), table=table, offs=offs, lens=np.array(lens, np.int32),
                cache=cache, page=page, D=D, T=T, rows=int(sum(new)))


def run_attn(st, scale=None, softcap=0.0, window=0, q=None, table=None):
    out = torch.full(st["q"].shape, 5.0, dtype=BF, device="cuda")
    moe.paged_attention(st["q"].cuda() if q is None else q, st["cache"],
                        (st["table"] if table is None else table).cuda(), ints(st["offs"]), ints(st["lens"]),
                        scale=scale, softcap=softcap, window=window, out=out)
    torch.cuda.synchronize()
    return out.cpu()


def check_attn(st, got, scale=None, softcap=0.0, window=0, table=None, v=None):
    scale = st["D"] ** -0.5 if scale is None else scale
    want, mass, reach = ref.attention(st["q"], st["k"], st["v"] if v is None else v,
                                      st["table"] if table is None else table, st["offs"], st["lens"], st["page"],
                                      scale, softcap, window)
    n = st["rows"]
    assert bool((got[n:] == 5.0).all()), "a row behind the last request was written"
    bound = ref.attention_bound(want, mass, reach, st["D"], int(max(st["lens"], default=1)))[:n]
    err = (got[:n].double() - want[:n]).abs()
    bad = ~(err <= bound)
    assert not bool(bad.any()), f"{int(bad.sum())} values off, worst {float((err - bound).max())} at {bad.nonzero()[0].tolist()}"


ATTNS = [
    # lens, new, Hq, Hkv, D, page, fp8, window, softcap
    ([1], [1], 1, 1, 64, 16, False, 0, 0.0),
    ([1], [1], 8, 1, 128, 16, True, 0, 0.0),
    ([33], [1], 16, 2, 256, 16, False, 0, 0.0),
    ([130], [5], 16, 2, 256, 16, True, 0, 0.0),
    ([16, 17, 31, 32, 33, 127, 128, 129], [1] * 8, 4, 2, 128, 16, False, 0, 0.0),
    ([257, 3, 64, 700], [1, 3, 5, 8], 8, 2, 128, 64, False, 0, 0.0),
    ([257, 3, 64, 700], [2, 3, 0, 8], 8, 2, 64, 32, True, 0, 30.0),
    ([300, 200], [40, 33], 8, 2, 128, 16, False, 0, 0.0),            # three and more row tiles
    ([300, 200], [40, 33], 6, 1, 64, 16, False, 70, 0.0),            # a group of 6
    ([90], [50], 3, 3, 64, 16, True, 20, 20.0),
    ([1500, 40], [4, 4], 4, 1, 128, 128, False, 100, 0.0),           # a window that leaves most pages out
    ([1500, 700], [1, 1], 2, 2, 256, 1024, False, 0, 0.0),
    ([5000], [1], 4, 1, 64, 16, False, 0, 0.0),                      # many splits
    ([3000, 10], [7, 7], 2, 1, 128, 32, True, 0, 0.0),
    ([5], [1], 64, 1, 64, 16, False, 0, 0.0),                        # the largest group
    ([130, 100], [16, 16], 32, 2, 256, 32, False, 0, 0.0),           # all row tiles at head_dim 256
    ([600, 33], [2, 3], 16, 1, 256, 16, True, 0, 25.0),
    ([300, 64], [3, 1], 12, 1, 128, 16, True, 40, 0.0),
    ([30, 17], [30, 17], 4, 2, 64, 16, False, 0, 0.0),               # whole prompts, three row tiles at head_dim 64
    ([48, 50, 3], [48, 50, 3], 2, 2, 128, 16, True, 0, 0.0),
    ([(i * 37) % 150 + 1 for i in range(70)], [1] * 70, 2, 1, 64, 16, False, 0, 0.0),     # more than 64 requests
    ([(i * 53) % 90 + 4 for i in range(300)], [i % 4 for i in range(300)], 2, 2, 64, 16, True, 30, 0.0),
]


@pytest.mark.parametrize("case", ATTNS, ids=lambda c: "-".join(map(str, c)).replace(" ", ""))
def test_paged_attention(case):
    lens, new, Hq, Hkv, D, page, fp8, window, cap = case
    st = attn_state(lens, new, Hq, Hkv, D, page, fp8, seed=sum(lens), pad=2)
    check_attn(st, run_attn(st, softcap=cap, window=window), softcap=cap, window=window)


@pytest.mark.parametrize("new", [1, 5, 10, 16, 23])                  # 4 rows each: one to four row tiles, and two units
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_paged_attention_every_shape(D, fp8, new):
    st = attn_state([new + 150, new, new + 7], [new] * 3, 8, 2, D, 32, fp8, seed=new, pad=1)
    check_attn(st, run_attn(st))
    check_attn(st, run_attn(st, softcap=5.0, window=37), softcap=5.0, window=37)


MANY_ROWS = [
    # whole prompts and chunks: more than 128 rows (query token x head) per key-value head and request
    ([300, 200], [300, 150], 8, 2, 128, 16, False, 0, 0.0),
    ([700, 5, 410], [400, 1, 300], 4, 1, 256, 16, False, 0, 0.0),
    ([700, 5, 410], [400, 0, 300], 4, 1, 256, 32, True, 0, 30.0),
    ([1200, 300], [333, 77], 4, 2, 64, 16, False, 100, 0.0),
    ([1200, 300, 64], [333, 77, 64], 4, 2, 64, 64, True, 100, 20.0),
    ([900], [129], 3, 3, 128, 16, True, 0, 0.0),                     # a row per token
    ([200, 100], [40, 30], 64, 1, 64, 32, False, 0, 0.0),            # the largest group
    ([3000], [70], 12, 2, 128, 1024, False, 0, 0.0),                 # a group of 6 across tiles, units in many shares
    ([5000], [200], 2, 1, 256, 16, False, 1, 0.0),                   # a window of one
    ([257] * 5, [257] * 5, 2, 2, 64, 16, False, 0, 0.0),
    ([256, 250], [256, 250], 4, 4, 256, 256, True, 40, 0.0),         # 512 positions at most: units stay whole
    ([(i * 37) % 150 + 60 for i in range(520)], [60] * 520, 2, 1, 64, 16, False, 0, 0.0),     # more requests than threads
]


def many_rows_state(lens, new, Hq, Hkv, D, page, fp8, seed, pad):
    """attn_state, with tables so wide (their far entries garbage) that the many-row kernel runs."""
    W = max(max(-(-n // page) for n in lens) + 1, (1 << 25) // (sum(new) * Hq * page) + 1)
    return attn_state(lens, new, Hq, Hkv, D, page, fp8, seed=seed, pad=pad, W=W)


@pytest.mark.parametrize("case", MANY_ROWS, ids=lambda c: "-".join(map(str, c[2:])).replace(" ", ""))
def test_paged_attention_many_rows(case):
    lens, new, Hq, Hkv, D, page, fp8, window, cap = case
    state = many_rows_state if window == 0 else attn_state
    st = state(lens, new, Hq, Hkv, D, page, fp8, seed=sum(lens), pad=3)
    check_attn(st, run_attn(st, softcap=cap, window=window), softcap=cap, window=window)


@pytest.mark.parametrize("D,fp8,window", [(64, False, 900), (128, True, 33), (256, False, 200)])
def test_paged_attention_many_rows_windowed(D, fp8, window):
    # enough rows that the many-row kernel runs: 1500 x 16 x (window + 1500 / 2) scores and more
    st = attn_state([1700, 1800], [1500, 1600], 16, 2, D, 16, fp8, seed=window, pad=1)
    check_attn(st, run_attn(st, softcap=20.0, window=window), softcap=20.0, window=window)


@pytest.mark.parametrize("new", [80, 150])
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_paged_attention_many_rows_every_shape(D, fp8, new):
    st = many_rows_state([new + 550, new, new + 7], [new] * 3, 8, 2, D, 32, fp8, seed=new, pad=1)
    a = run_attn(st)
    check_attn(st, a)
    assert torch.equal(a.view(torch.int16), run_attn(st).view(torch.int16))
    check_attn(st, run_attn(st, softcap=5.0, window=37), softcap=5.0, window=37)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("D", [64, 256])
def test_paged_attention_many_rows_that_see_nothing(D, fp8):
    st = many_rows_state([0, 2, 400, 600], [90, 80, 200, 300], 4, 2, D, 16, fp8, seed=3, pad=0)
    table = st["table"].clone()
    table[2] = -1                                    # request 2 has no page
    table[3, 9] = st["cache"].num_pages              # request 3 lacks positions 144..159 and 368..399
    table[3, 23:25] = -7
    got = run_attn(st, table=table)
    check_attn(st, got, table=table)
    assert bool((got[:168] == 0).all()) and bool((got[170:370] == 0).all())


@pytest.mark.parametrize("lens", [[2000], [640], [300]])             # past the table, up to it, more rows than positions
def test_paged_attention_many_rows_lengths_past_the_table(lens):
    st = attn_state(lens, [1000], 64, 1, 64, 16, False, seed=4, W=40)
    check_attn(st, run_attn(st))


@pytest.mark.parametrize("D,fp8", [(64, False), (128, True), (256, False)])
def test_paged_attention_many_rows_unseen_infinities_do_not_reach_a_row(D, fp8):
    st = many_rows_state([700], [300], 4, 2, D, 16, fp8, seed=5, pad=0)
    at = 650                                          # rows 0 .. 249 do not see it
    page, off = int(st["table"][0, at // 16]), at % 16
    if fp8:
        st["cache"].v.view(torch.uint8)[page, :, off, 3] = 0x7F
    else:
        st["cache"].v[page, :, off, 3] = math.inf
    st["v"][page, :, off, 3] = math.nan if fp8 else math.inf
    got = run_attn(st)
    want, mass, reach = ref.attention(st["q"], st["k"], st["v"], st["table"], st["offs"], st["lens"], 16, D ** -0.5,
                                      0.0, 0)
    bound = ref.attention_bound(want, mass, reach, D, 700)
    n = at - 400
    assert bool(((got[:n].double() - want[:n]).abs() <= bound[:n]).all())
    tail = got[n:].double()
    assert bool(torch.isnan(tail[:, :, 3]).all()) if fp8 else bool((tail[:, :, 3] == math.inf).all())
    rest = [d for d in range(D) if d != 3]
    assert bool(((tail - want[n:]).abs() <= bound[n:])[:, :, rest].all())


@pytest.mark.parametrize("fp8", [False, True])
def test_paged_attention_rows_that_see_nothing(fp8):
    # no cached position at all; more rows than positions; pages outside the cache
    st = attn_state([0, 2, 40, 50], [1, 5, 1, 2], 4, 2, 64, 16, fp8, seed=3)
    table = st["table"].clone()
    table[2] = -1                                    # request 2 has no page
    table[3, 1] = st["cache"].num_pages              # request 3 lacks positions 16..31
    got = run_attn(st, table=table)
    check_attn(st, got, table=table)
    assert bool((got[0] == 0).all()) and bool((got[1:4] == 0).all()) and bool((got[6] == 0).all())


def test_paged_attention_windows_of_one_and_of_everything():
    st = attn_state([200, 5], [7, 5], 4, 2, 64, 16, False, seed=9)
    check_attn(st, run_attn(st, window=1), window=1)
    a = run_attn(st)
    for w in (200, 1 << 30, (1 << 31) - 1):
        assert torch.equal(run_attn(st, window=w).view(torch.int16), a.view(torch.int16))


def test_paged_attention_scale_of_zero_and_below():
    st = attn_state([90, 700], [3, 1], 4, 2, 64, 16, True, seed=10)
    for scale in (0.0, -0.3):
        got = run_attn(st, scale=scale)
        want, mass, reach = ref.attention(st["q"], st["k"], st["v"], st["table"], st["offs"], st["lens"], 16, scale, 0.0, 0)
        bound = ref.attention_bound(want, mass, reach.abs(), 64, 700)
        assert bool(((got.double() - want).abs() <= bound).all())


def test_paged_attention_lengths_past_the_table():
    st = attn_state([100], [2], 2, 1, 64, 16, False, seed=4, W=4)    # 64 positions fit
    check_attn(st, run_attn(st))


@pytest.mark.parametrize("D,fp8", [(64, False), (128, False), (128, True), (256, False)])
def test_paged_attention_unseen_infinities_do_not_reach_a_row(D, fp8):
    # the newest tokens' values and keys are infinite or NaN: the rows before them do not see them
    st = attn_state([70], [6], 4, 2, D, 16, fp8, seed=5)
    page, off = int(st["table"][0, 67 // 16]), 67 % 16
    bad = math.nan if fp8 else math.inf
    if fp8:
        st["cache"].v.view(torch.uint8)[page, :, off, 3] = 0x7F
    else:
        st["cache"].v[page, :, off, 3] = math.inf
        st["cache"].v[page, 0, off, 5] = -math.inf
        st["v"][page, 0, off, 5] = -math.inf
    st["v"][page, :, off, 3] = bad
    got = run_attn(st)
    n = 3                                             # rows of positions 64, 65, 66
    want, mass, reach = ref.attention(st["q"], st["k"], st["v"], st["table"], st["offs"], st["lens"], 16, D ** -0.5,
                                      0.0, 0)
    bound = ref.attention_bound(want, mass, reach, D, 70)
    assert bool(((got[:n].double() - want[:n]).abs() <= bound[:n]).all())
    tail = got[n:].double()
    assert bool(torch.isnan(tail[:, :, 3]).all()) if fp8 else bool((tail[:, :, 3] == math.inf).all())
    if not fp8:
        assert bool((tail[:, :2, 5] == -math.inf).all())
    rest = [d for d in range(D) if d not in (3, 5)]
    assert bool(((tail - want[n:]).abs() <= bound[n:])[:, :, rest].all())


def test_paged_attention_nan_and_infinite_scores():
    # a NaN in one head's query, an infinite key: only the rows that meet them are NaN, as in the formula
    st = attn_state([40], [3], 4, 2, 64, 16, False, seed=6)
    st["q"][1, 2, 7] = math.nan
    got = run_attn(st)
    assert bool(torch.isnan(got[1, 2]).all())
    rest = torch.ones(3, 4, dtype=torch.bool)
    rest[1, 2] = False
    assert bool(torch.isfinite(got[rest]).all())


def test_paged_attention_strided_queries_and_scale():
    st = attn_state([77, 130], [2, 1], 4, 2, 128, 16, False, seed=7)
    wide = torch.full((3, 4 * 128 + 64), math.nan, dtype=BF, device="cuda")
    wide[:, :512] = st["q"].view(3, 512).cuda()
    check_attn(st, run_attn(st, scale=0.2, q=wide[:, :512].view(3, 4, 128)), scale=0.2)


def test_paged_attention_shared_pages_and_repeats_are_identical():
    # two requests that share every page; the same call twice gives the same bits, also with many splits
    st = attn_state([4000, 4000], [1, 1], 8, 1, 128, 16, False, seed=8)
    st["table"][1] = st["table"][0]
    st["q"][1] = st["q"][0]
    a, b = run_attn(st), run_attn(st)
    assert torch.equal(a.view(torch.int16), b.view(torch.int16))
    assert torch.equal(a[0].view(torch.int16), a[1].view(torch.int16))
    st["k"], st["v"] = st["k"].nan_to_num(), st["v"].nan_to_num()
    check_attn(st, a)


# ---------------------------------------------------------------- dense products
LINEARS = [
    # T, N, K, act, bias, residual, out dtype
    (1, 8, 64, None, False, False, BF),
    (1, 1000, 128, "silu", True, True, BF),
    (5, 2560, 2048, None, False, False, BF),
    (8, 520, 1088, "gelu", True, False, torch.float32),
    (16, 264, 512, "relu", True, True, BF),
    (17, 72, 192, "gelu_tanh", False, True, torch.float32),
    (33, 200, 256, "silu", False, False, BF),
    (64, 2048, 320, None, True, True, BF),
    (130, 136, 640, "gelu_tanh", True, True, torch.float32),
    (257, 512, 64, None, False, True, BF),
    (300, 1032, 128, "gelu", True, False, BF),
    (513, 768, 1024, None, False, True, torch.float32),
    (1100, 520, 192, "silu", True, True, BF),
    (3, 40, 4160, None, True, True, BF),             # K past one round of the waves
    (16, 264, 8256, "silu", False, True, torch.float32),
    (2, 20000, 64, None, False, False, BF),          # more weight rows than blocks hold at once
    (32, 4100 * 8, 64, "relu", True, False, BF),
    (1700, 1800, 320, "gelu", True, True, BF),       # 128-square tiles
    (3900, 3400, 192, None, False, True, BF),        # 256-square tiles
    (3841, 3336, 64, "gelu_tanh", True, False, torch.float32),
    (40, 264, 2112, "silu", True, True, torch.float32),     # k in two halves a block, the last step half full
    (33, 72, 2048, None, False, False, BF),
    (130, 200, 4160, "gelu", True, True, BF),
    (29, 2056, 2176, None, True, False, torch.float32),     # tiles below 33 rows
    (20, 2560, 128, "relu", False, True, BF),
]


@pytest.mark.parametrize("case", LINEARS, ids=lambda c: "-".join(map(str, c)).replace("torch.", ""))
def test_linear(case):
    T, N, K, act, bias, residual, dt = case
    g = rng(T * N + K)
    x = torch.randn(T, K, generator=g).to(BF)
    w = (torch.randn(N, K, generator=g) * K ** -0.5).to(BF)
    b = torch.randn(N, generator=g) if bias else None
    r = torch.randn(T, N, generator=g).to(dt) if residual else None
    want, size, y = ref.linear(x, w, b, act, r)
    wide = torch.full((T, K + 24), math.nan, dtype=BF, device="cuda")
    wide[:, :K] = x.cuda()
    dev = lambda t: None if t is None else t.cuda()  # noqa: E731
    bound = ref.linear_bound(want, size, y, K, dt)
    for xx in (wide[:, :K], x.cuda()):
        got = moe.linear(xx, dev(w), bias=dev(b), act=act, residual=dev(r), out_dtype=dt)
        assert got.dtype == dt and bool(((got.cpu().double() - want).abs() <= bound).all())
    if residual:                                     # in place on the residual stream
        rr = dev(r)
        assert moe.linear(x.cuda(), dev(w), bias=dev(b), act=act, residual=rr, out=rr) is rr
        assert bool(((rr.cpu().double() - want).abs() <= bound).all())


def test_linear_writes_its_output_only():
    T, N, K = 37, 72, 128
    buf = torch.full((T + 2, N), 3.0, dtype=BF, device="cuda")
    moe.linear(torch.randn(T, K, device="cuda").to(BF), torch.randn(N, K, device="cuda").to(BF), out=buf[1:-1])
    torch.cuda.synchronize()
    assert bool((buf[0] == 3.0).all()) and bool((buf[-1] == 3.0).all())


def test_linear_infinities_stay_in_their_row_and_column():
    T, N, K = 20, 40, 128
    x, w = torch.randn(T, K), torch.randn(N, K)
    x[3, 5], w[7, 9] = math.nan, math.inf
    got = moe.linear(x.to(BF).cuda(), w.to(BF).cuda()).cpu()
    fine = torch.isfinite(got)
    want = torch.ones(T, N, dtype=torch.bool)
    want[3], want[:, 7] = False, False
    assert torch.equal(fine, want)


# ---------------------------------------------------------------- far addresses, streams, graphs, all of it together
@pytest.mark.parametrize("fp8", [False, True])
def test_offsets_past_32_bits(fp8):
    # a cache of over 2^31 elements (2^32 bytes): its last pages are written and read
    D, Hkv, page, pages = 256, 2, 1024, 8300 if fp8 else 4200
    cache = moe.KVCache.allocate(pages, page, Hkv, D, FP8 if fp8 else BF)
    assert cache.k.numel() > 1 << 31
    T, Hq, first = 70, 4, pages - 2
    g = rng(11)
    qkv = torch.randn(T, (Hq + 2 * Hkv) * D, generator=g).to(BF)
    table = ints([first, 0]).view(1, 2)                            # positions 0 .. 1023; the next page is the last one
    plan = moe.kv_plan(ints([990]), ints([T]), ints([pages - 1]), table, page, T)
    moe.qk_norm_rope(qkv.cuda(), cache, plan.positions, plan.slots)                 # earlier positions stay unwritten
    q = qkv[:, :Hq * D].view(T, Hq, D)
    got = moe.paged_attention(q.cuda(), cache, table, plan.q_offsets, plan.kv_len, window=1)    # each row sees itself
    torch.cuda.synchronize()
    v = qkv.view(T, Hq + 2 * Hkv, D)[:, Hq + Hkv:].double().repeat_interleave(Hq // Hkv, 1)
    half = ref.FP8_HALF if fp8 else 0.0
    bound = (half + 2 * ref.BF16_HALF) * v.abs() + (2.0 ** -10 / 448 * v.abs().amax(-1, keepdim=True) if fp8 else 0)
    assert bool(((got.cpu().double() - v).abs() <= bound).all())


def test_two_streams_at_once():
    states = [attn_state([3000, 5], [1, 3], 8, 2, 128, 16, False, seed=s) for s in (20, 21)]
    x = torch.randn(64, 1024).to(BF).cuda()
    w = [torch.randn(512, 1024).to(BF).cuda() for _ in range(2)]
    alone = [run_attn(st) for st in states]
    lin = [moe.linear(x, v) for v in w]
    args = [(st["q"].cuda(), st["cache"], st["table"].cuda(), ints(st["offs"]), ints(st["lens"])) for st in states]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        got = [(moe.paged_attention(*a, stream=s), moe.linear(x, v, stream=s)) for a, v, s in zip(args, w, streams)]
        torch.cuda.synchronize()
        for (o, y), a, b, st in zip(got, alone, lin, states):
            n = st["rows"]
            assert torch.equal(o.cpu()[:n].view(torch.int16), a[:n].view(torch.int16))
            assert torch.equal(y.view(torch.int16), b.view(torch.int16))


class Model:
    """Two requests through the attention half and the MoE half of one small layer."""

    def __init__(self, fp8, T):
        g = rng(31)
        self.H, self.Hq, self.Hkv, self.D, self.page, self.S, self.T = 256, 4, 2, 64, 16, 2, T
        r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
        n = (self.Hq + 2 * self.Hkv) * self.D
        self.w_qkv = (r(n, self.H) / 16).to(BF).cuda()
        self.w_out = (r(self.H, self.Hq * self.D) / 16).to(BF).cuda()
        self.qw, self.kw = (1 + 0.1 * r(self.D)).cuda(), (1 + 0.1 * r(self.D)).cuda()
        self.freq = (10000.0 ** (-torch.arange(0, 32, 2) / 32)).float().cuda()
        self.wr = (r(16, self.H) / 16).cuda()
        self.wg, self.wu, self.wd = ((r(16, *s) / 16).to(BF).cuda() for s in ((128, self.H), (128, self.H), (self.H, 128)))
        self.cache = moe.KVCache.allocate(40, self.page, self.Hkv, self.D, FP8 if fp8 else BF)
        for t in (self.cache.k, self.cache.v):
            t.view(torch.uint8).fill_(0x7F)                        # NaN wherever nothing was written
        self.table = torch.full((2, 12), -1, dtype=torch.int32, device="cuda")
        self.free = torch.randperm(40, generator=g).to(torch.int32).cuda()
        self.cached, self.new = ints([0, 0]), ints([0, 0])
        self.x = torch.zeros(T, self.H, dtype=BF, device="cuda")
        self.plan = moe.KVPlan.allocate(2, T)
        self.ws = moe.AttentionWorkspace(T, self.H, self.Hq, self.cache, 2)
        self.lw = moe.LayerWorkspace(T, self.H, 16, 4, 128)
        self.y = torch.empty_like(self.x)

    def step(self):
        moe.kv_plan(self.cached, self.new, self.free, self.table, self.page, self.T, out=self.plan)
        h = moe.attention_layer(self.x, self.w_qkv, self.w_out, self.cache, self.plan, self.table, self.qw, self.kw,
                                inv_freq=self.freq, residual=self.x, ws=self.ws)
        moe.layer(h, self.wr, self.wg, self.wu, self.wd, 4, residual=h, lw=self.lw, out=self.y)

    def advance(self):
        """After a step: the new tokens are cached, and the pages that they took leave the list."""
        taken = int(self.plan.counts[1])
        self.cached += self.new
        self.free.copy_(torch.roll(self.free, -taken))


@pytest.mark.parametrize("fp8", [False, True])
def test_attention_layer_steps_match_the_formulas(fp8):
    # a ragged prompt chunk, a verify step, single tokens: each operator's output from its own inputs
    m = Model(fp8, 48)
    g = rng(32)
    for new in ([30, 17], [5, 0], [1, 5], [1, 1]):
        rows = sum(new)
        m.new.copy_(ints(new))
        m.x.copy_(torch.randn(m.T, m.H, generator=g).to(BF))
        m.step()
        torch.cuda.synchronize()
        cached = m.cached.cpu().numpy()
        want, size, y = ref.linear(m.x.cpu(), m.w_qkv.cpu(), None, None, None)
        qkv = m.ws.qkv.cpu()
        assert bool(((qkv.double() - want).abs() <= ref.linear_bound(want, size, y, m.H, BF)).all())
        pos = m.plan.positions.cpu()
        assert pos[:rows].tolist() == [c + i for c, n in zip(cached, new) for i in range(n)]
        want, size = ref.qk_norm_rope(qkv, m.Hq, m.Hkv, m.D, pos, m.qw.cpu(), m.kw.cpu(), 1e-6, m.freq.cpu(), False, 1.0)
        q = m.ws.q.cpu()[:rows].double()
        bound = ref.BF16_HALF * want.abs() + 1.01 * ref.norm_rope_slack(size, m.D)
        assert bool(((q - want[:rows, :m.Hq]).abs() <= bound[:rows, :m.Hq]).all())
        c = m.cache
        k, v = ref.k_rows(c.k.view(torch.uint8).cpu()).contiguous().view(FP8) if fp8 else ref.k_rows(c.k.cpu()), c.v.cpu()
        k, v = ref.as_values(k, c.k_scale.cpu() if fp8 else None), ref.as_values(v, c.v_scale.cpu() if fp8 else None)
        st = dict(q=m.ws.q.cpu(), k=k, v=v, table=m.table.cpu(), offs=m.plan.q_offsets.cpu().numpy(),
                  lens=m.plan.kv_len.cpu().numpy(), page=m.page, D=m.D, rows=rows)
        assert st["lens"].tolist() == [int(a) + b for a, b in zip(cached, new)]
        o = m.ws.o.cpu()
        want, mass, reach = ref.attention(st["q"], k, v, st["table"], st["offs"], st["lens"], m.page, m.D ** -0.5, 0.0, 0)
        bound = ref.attention_bound(want, mass, reach, m.D, int(max(st["lens"])))
        assert bool(((o.double() - want).abs() <= bound)[:rows].all())
        want, size, y = ref.linear(o.view(m.T, -1), m.w_out.cpu(), None, None, m.x.cpu())
        bound = ref.linear_bound(want, size, y, m.Hq * m.D, BF)
        assert bool(((m.ws.out.cpu().double() - want).abs() <= bound)[:rows].all())
        assert bool(torch.isfinite(m.y[:rows].float()).all())
        m.advance()


@pytest.mark.parametrize("fp8", [False, True])
def test_captured_decode_steps_replay(fp8):
    # one graph of a whole step, replayed while the lengths grow, against the same steps called one by one
    steps = [[3, 1], [2, 3], [1, 1], [4, 0], [1, 1], [1, 1], [0, 5], [1, 1]] * 3
    a, b = Model(fp8, 8), Model(fp8, 8)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        a.step()                                      # before any token: warms up, changes nothing
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            a.step()
    torch.cuda.synchronize()
    g = rng(33)
    for new in steps:
        x = torch.randn(8, 256, generator=g).to(BF).cuda()
        for m in (a, b):
            m.x.copy_(x)
            m.new.copy_(ints(new))
        graph.replay()
        b.step()
        torch.cuda.synchronize()
        rows = sum(new)
        assert torch.equal(a.plan.slots, b.plan.slots) and torch.equal(a.table, b.table)
        assert torch.equal(a.y[:rows].view(torch.int16), b.y[:rows].view(torch.int16))
        for m in (a, b):
            m.advance()
    assert int(a.cached.sum()) == sum(map(sum, steps))


def test_two_captured_graphs_share_a_workspace_in_turn():
    one = attn_state([2500], [2], 8, 1, 128, 16, False, seed=40)
    two = attn_state([900, 40], [1, 1], 8, 1, 128, 16, False, seed=41)
    alone = [run_attn(one), run_attn(two)]
    ws = torch.empty(max(moe.paged_attention_workspace_size(st["T"], 8, 1, 128, len(st["lens"])) for st in (one, two)),
                     dtype=torch.uint8, device="cuda")
    graphs, outs, keep = [], [], []
    for st in (one, two):
        args = (st["q"].cuda(), st["cache"], st["table"].cuda(), ints(st["offs"]), ints(st["lens"]))
        out = torch.empty_like(args[0])
        moe.paged_attention(*args, out=out, workspace=ws)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            moe.paged_attention(*args, out=out, workspace=ws)
        graphs.append(graph)
        outs.append(out)
        keep.append(args)
    for order in ((0, 1), (1, 0), (0, 0, 1, 1, 0)):
        for i in order:
            outs[i].zero_()
            graphs[i].replay()
        torch.cuda.synchronize()
        for i in set(order):
            assert torch.equal(outs[i].cpu().view(torch.int16), alone[i].view(torch.int16))
