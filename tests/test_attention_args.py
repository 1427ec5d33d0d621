"""The attention half's calls on the CPU: every refusal comes back with its
documented status before anything reaches the GPU."""
import ctypes
import os

import pytest
import torch

from routed_expert_ffn_amd import build, moe

FAKE = ctypes.c_void_p(0x10000)    # aligned, never dereferenced: every call below returns before a launch
ODD = ctypes.c_void_p(0x10008)
INVALID, UNSUPPORTED, WORKSPACE = moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_UNSUPPORTED, moe.MOE_ERR_WORKSPACE


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(build.LIB):
        build.build()
    return moe.load()


def cache(dtype=moe.BF16, pages=10, page=16, heads=2, D=128, k=0x10000, v=0x10000, ks=None, vs=None):
    return moe.KVCacheStruct(dtype, pages, page, heads, D, k, v, ks, vs)


CACHES = [
    (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(pages=0), INVALID), (dict(heads=0), INVALID),
    (dict(dtype=9), INVALID), (dict(ks=0x10000), INVALID),                     # scales without 8-bit elements
    (dict(dtype=moe.FP8_E4M3), INVALID),                                       # and the other way round
    (dict(dtype=moe.FP8_E4M3, ks=0x10000), INVALID), (dict(dtype=moe.F32), UNSUPPORTED),
    (dict(page=24), UNSUPPORTED), (dict(page=8), UNSUPPORTED), (dict(page=2048), UNSUPPORTED),
    (dict(D=96), UNSUPPORTED), (dict(pages=1 << 28), UNSUPPORTED), (dict(k=0x10008), UNSUPPORTED),
]


def test_kv_plan_refuses(L):
    base = dict(c=FAKE, n=FAKE, S=4, f=FAKE, nf=3, P=16, T=8, t=FAKE, W=4, o=FAKE, k=FAKE, p=FAKE, s=FAKE, cnt=FAKE)

    def call(**kw):
        a = dict(base, **kw)
        return L.moe_kv_plan(a["c"], a["n"], a["S"], a["f"], a["nf"], a["P"], a["T"], a["t"], a["W"], a["o"], a["k"],
                             a["p"], a["s"], a["cnt"], None)
    for name in ("c", "n", "f", "t", "o", "k", "p", "s", "cnt"):
        assert call(**{name: None}) == INVALID, name
    assert call(S=0) == INVALID and call(T=-1) == INVALID and call(W=0) == INVALID and call(nf=-1) == INVALID
    assert call(P=0) == INVALID and call(P=24) == UNSUPPORTED and call(P=8) == UNSUPPORTED
    assert call(S=4097) == UNSUPPORTED and call(W=1 << 27) == UNSUPPORTED
    assert call(t=ctypes.c_void_p(0x10002)) == UNSUPPORTED


def test_kv_plan_refuses_lengths_advanced_in_place(L):
    p = [ctypes.c_void_p(0x10000 + 0x1000 * i) for i in range(9)]
    for kv, offs in ((p[0], p[4]), (p[1], p[4]), (p[5], p[0]), (p[5], p[1])):
        assert L.moe_kv_plan(p[0], p[1], 4, p[2], 3, 16, 8, p[3], 4, offs, kv, p[6], p[7], p[8], None) == INVALID


def test_qk_norm_rope_refuses(L):
    base = dict(x=FAKE, xd=moe.BF16, st=20 * 128, T=3, h=16, c=cache(), qw=FAKE, kw=FAKE, f=FAKE, R=64, lay=0, p=FAKE,
                s=FAKE, o=FAKE, eps=1e-6, rs=1.0)

    def call(**kw):
        a = dict(base, **kw)
        return L.moe_qk_norm_rope(a["x"], a["xd"], a["st"], a["T"], a["h"], ctypes.byref(a["c"]) if a["c"] else None,
                                  a["qw"], a["kw"], a["eps"], a["f"], a["R"], a["lay"], a["rs"], a["p"], a["s"], a["o"],
                                  None)
    for kw, status in CACHES:
        assert call(c=cache(**kw)) == status, kw
    for name in ("x", "c", "f", "p", "s", "o"):
        assert call(**{name: None}) == INVALID, name
    assert call(T=-1) == INVALID and call(h=0) == INVALID and call(lay=2) == INVALID and call(xd=7) == INVALID
    for bad in (float("nan"), float("inf")):
        assert call(eps=bad) == INVALID and call(rs=bad) == INVALID
    assert call(eps=-1e-6) == INVALID
    assert call(R=-16) == INVALID and call(R=144) == INVALID and call(st=20 * 128 - 8) == INVALID
    assert call(xd=moe.F32) == UNSUPPORTED and call(R=24) == UNSUPPORTED and call(st=20 * 128 + 4) == UNSUPPORTED
    assert call(h=1021, st=1025 * 128) == UNSUPPORTED
    assert call(x=ODD) == UNSUPPORTED and call(o=ODD) == UNSUPPORTED and call(qw=ODD) == UNSUPPORTED


def test_paged_attn_refuses(L):
    nb = moe.paged_attention_workspace_size(3, 16, 2, 128, 2)
    base = dict(q=FAKE, qd=moe.BF16, st=16 * 128, T=3, h=16, c=cache(), t=FAKE, W=4, o=FAKE, k=FAKE, S=2, cap=0.0,
                win=0, out=FAKE, ws=FAKE, nb=nb, sc=0.1)

    def call(**kw):
        a = dict(base, **kw)
        return L.moe_paged_attn(a["q"], a["qd"], a["st"], a["T"], a["h"], ctypes.byref(a["c"]) if a["c"] else None,
                                a["t"], a["W"], a["o"], a["k"], a["S"], a["sc"], a["cap"], a["win"], a["out"], a["ws"],
                                a["nb"], None)
    for kw, status in CACHES:
        assert call(c=cache(**kw)) == status, kw
    for name in ("q", "c", "t", "o", "k", "out"):
        assert call(**{name: None}) == INVALID, name
    assert call(T=-1) == INVALID and call(S=0) == INVALID and call(W=0) == INVALID and call(win=-1) == INVALID
    assert call(cap=-1.0) == INVALID and call(cap=float("nan")) == INVALID and call(qd=9) == INVALID
    for bad in (float("nan"), float("inf")):
        assert call(cap=bad) == INVALID and call(sc=bad) == INVALID
    assert call(cap=1e-42) == INVALID and call(cap=3e38) == INVALID and call(sc=3e38) == INVALID   # scale / cap, x log2 e
    assert call(st=8) == INVALID and call(T=1 << 27, h=16, c=cache()) == INVALID
    assert call(qd=moe.F32) == UNSUPPORTED and call(S=4097) == UNSUPPORTED and call(h=15) == UNSUPPORTED
    assert call(h=130, st=130 * 128) == UNSUPPORTED                        # 65 query heads per key-value head
    assert call(st=16 * 128 + 4) == UNSUPPORTED and call(W=1 << 27) == UNSUPPORTED and call(q=ODD) == UNSUPPORTED
    assert call(nb=nb - 1) == WORKSPACE and call(ws=None) == WORKSPACE and call(ws=ODD) == WORKSPACE


def test_linear_refuses(L):
    base = dict(x=FAKE, xd=moe.BF16, st=128, w=FAKE, wd=moe.BF16, b=FAKE, act=0, r=FAKE, T=3, N=64, K=128, o=FAKE,
                od=moe.BF16, ws=FAKE, nb=1 << 30)

    def call(**kw):
        a = dict(base, **kw)
        return L.moe_linear(a["x"], a["xd"], a["st"], a["w"], a["wd"], a["b"], a["act"], a["r"], a["T"], a["N"],
                            a["K"], a["o"], a["od"], a["ws"], a["nb"], None)
    for name in ("x", "w", "o"):
        assert call(**{name: None}) == INVALID, name
    assert call(T=-1) == INVALID and call(N=0) == INVALID and call(K=0) == INVALID and call(st=120) == INVALID
    assert call(act=5) == INVALID and call(act=-1) == INVALID and call(od=moe.INT4_B32) == INVALID
    assert call(xd=moe.F32) == UNSUPPORTED and call(wd=moe.F32) == UNSUPPORTED and call(wd=moe.INT4_B32) == UNSUPPORTED
    assert call(K=96) == UNSUPPORTED and call(N=60) == UNSUPPORTED and call(st=132) == UNSUPPORTED
    for name in ("x", "w", "b", "r", "o"):
        assert call(**{name: ODD}) == UNSUPPORTED, name


def test_binding_refuses_before_the_library():
    bf = torch.bfloat16
    with pytest.raises(ValueError):                  # host tensors
        moe.KVCache(torch.zeros(1, 1, 8, 16, 8, dtype=bf), torch.zeros(1, 1, 16, 64, dtype=bf))
    with pytest.raises(TypeError):
        moe.KVCache(torch.zeros(1, 1, 8, 16, 8), torch.zeros(1, 1, 16, 64))
    with pytest.raises(TypeError):
        moe.KVCache.allocate(4, 16, 1, 64, dtype=torch.float16)


def test_workspace_sizes(L):
    assert moe.paged_attention_workspace_size(5, 16, 3, 128, 1) == 0       # no such head layout
    small = moe.paged_attention_workspace_size(1, 8, 1, 64, 1)
    assert 0 < small <= moe.paged_attention_workspace_size(4, 8, 1, 64, 1)
