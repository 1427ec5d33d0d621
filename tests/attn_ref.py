"""Plain 64-bit forms of the attention half's operators, and the layouts of the
paged cache, for the tests.  Nothing here calls the library."""
import math

import numpy as np
import torch

FP8 = torch.float8_e4m3fn
BF16_HALF = 2.0 ** -8      # half a step relative to the value: torch.finfo(torch.bfloat16).eps / 2
FP8_HALF = 2.0 ** -4
F32_HALF = 2.0 ** -24


def plan(cached, new, free, table, page, T):
    """kv_plan, one request and one token at a time: (q_offsets, kv_len, positions, slots, counts, table)."""
    S, W = table.shape
    table = table.copy()
    offs, lens, pos, slots = [0], [], np.zeros(T, np.int32), np.full(T, -1, np.int32)
    taken = 0
    for s in range(S):
        c = min(max(int(cached[s]), 0), W * page)
        have = -(-c // page)
        n = min(max(int(new[s]), 0), W * page - c, T - offs[-1])
        for i in range(n):
            p = c + i
            if p // page >= have:                       # the first token on a page that is not there yet
                table[s, have] = free[taken] if taken < len(free) else -1
                taken += 1
                have += 1
            e = int(table[s, p // page])
            pos[offs[-1] + i] = p
            slots[offs[-1] + i] = e * page + p % page if e >= 0 else -1
        offs.append(offs[-1] + n)
        lens.append(c + n)
    return (np.array(offs, np.int32), np.array(lens, np.int32), pos, slots, np.array([offs[-1], taken], np.int32),
            table)


def k_rows(k):
    """[pages][heads][D / X][page][X] -> [pages][heads][page][D]"""
    p, h, c, n, x = k.shape
    return k.permute(0, 1, 3, 2, 4).reshape(p, h, n, c * x)


def k_layout(rows, x):
    p, h, n, d = rows.shape
    return rows.view(p, h, n, d // x, x).permute(0, 1, 3, 2, 4).contiguous()


def as_values(t, scale=None):
    """Cache elements as float64 (e4m3 times its scale)."""
    v = t.to(torch.float32).double()
    return v if scale is None else v * scale.double()[..., None]


def attention(q, k, v, table, offs, lens, page, scale, softcap, window):
    """float64 [T][Hq][D] and, per element, sum p |v| / sum p and the largest sum |q||k| * scale of its row.
    k, v [pages][heads][page][D] float64; rows that belong to no request are NaN."""
    T, Hq, D = q.shape
    pages, Hkv = k.shape[:2]
    W = table.shape[1]
    out = torch.full((T, Hq, D), math.nan, dtype=torch.float64)
    mass, reach = torch.zeros_like(out), torch.zeros(T, Hq, dtype=torch.float64)
    for s in range(table.shape[0]):
        a, b, L = int(offs[s]), int(offs[s + 1]), int(lens[s])
        n = b - a
        for i in range(n):
            p = L - n + i
            seen = [j for j in range(max(0, p - window + 1) if window else 0, min(p + 1, W * page))
                    if 0 <= int(table[s, j // page]) < pages]
            if not seen:
                out[a + i] = 0
                continue
            j = torch.tensor(seen)
            pg, of = torch.as_tensor(table[s])[j // page].long(), j % page
            for h in range(Hq):
                kv = h // (Hq // Hkv)
                kk, vv, qq = k[pg, kv, of], v[pg, kv, of], q[a + i, h].double()
                x = kk @ qq * scale
                if softcap:
                    x = softcap * torch.tanh(x / softcap)
                w = torch.softmax(x, 0)
                out[a + i, h] = w @ vv
                mass[a + i, h] = w @ vv.abs()
                reach[a + i, h] = (kk.abs() @ qq.abs()).max() * abs(scale)
    return out, mass, reach


def attention_bound(out, mass, reach, D, positions):
    """How far a bf16 result may be.  Scores: fp32 sums of D products (each of the D - 1 additions and the scaling off
    by 2^-24 relative to sum |q||k|), so a probability is off by that much relatively, once in itself and once in
    the sum, plus 2^-20 for exp2 and the log2 e scaling of exponents up to 2^4; the weights w_j = p_j (1 + e_j) of both
    the product and the normalising sum are rounded to bf16, |e_j| <= half a step: sum w v / sum w - out =
    sum p_j e_j (v_j - out) / sum w, at most half a step of (sum p |v| / sum p + |out|); the second product sums
    `positions` terms in fp32; the result is rounded to bf16 (half a step)."""
    score = 2 * (D + 2) * F32_HALF * reach[..., None] + 2.0 ** -20
    return (BF16_HALF + score + 2 * positions * F32_HALF) * (mass + out.abs()) + BF16_HALF * out.abs()


def qk_norm_rope(qkv, Hq, Hkv, D, positions, qw, kw, eps, inv_freq, interleaved, rope_scale):
    """float64 [T][Hq + 2 Hkv][D], and the magnitude that its fp32 rounding errors are relative to."""
    T = qkv.shape[0]
    y = qkv.double().view(T, Hq + 2 * Hkv, D).clone()
    for h in range(Hq + Hkv):
        w = qw if h < Hq else kw
        if w is not None:
            y[:, h] = y[:, h] / torch.sqrt((y[:, h] ** 2).mean(-1, keepdim=True) + eps) * w.double()
    size = y.abs().clone()
    R = 0 if inv_freq is None else 2 * inv_freq.numel()
    for i in range(R // 2):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + R // 2)
        angle = positions.double() * float(inv_freq[i])
        c, s = torch.cos(angle)[:, None] * rope_scale, torch.sin(angle)[:, None] * rope_scale
        u, v = y[:, :Hq + Hkv, a].clone(), y[:, :Hq + Hkv, b].clone()
        y[:, :Hq + Hkv, a], y[:, :Hq + Hkv, b] = u * c - v * s, v * c + u * s
        size[:, :Hq + Hkv, a] = size[:, :Hq + Hkv, b] = (u.abs() + v.abs()) * abs(rope_scale)
    return y, size


def norm_rope_slack(size, D, rope_scale=1.0):
    """fp32 errors of norm and rotation, relative to `size`: the sum of D squares (D + 1 roundings, halved by the
    root), root, reciprocal, two products: (D / 2 + 6) 2^-24; the angle's remainder rounded to fp32 (|r| <= pi: 2^-22.3),
    sine and cosine to 2 units, the factor and two products and a sum: 16 2^-24."""
    return (D / 2 + 6 + 16) * F32_HALF * size


def activation(z, act):
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z / math.sqrt(2)))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    if act == "relu":
        return torch.clamp(z, min=0)
    return z


def linear(x, w, bias, act, residual):
    """float64 result, and sum |x||w| + |bias| per output."""
    z = x.double() @ w.double().t()
    size = x.double().abs() @ w.double().abs().t()
    if bias is not None:
        z, size = z + bias.double(), size + bias.double().abs()
    y = activation(z, act)
    return (y if residual is None else y + residual.double()), size, y


def linear_bound(out, size, y, K, dtype):
    """fp32 sums of K products (K additions relative to sum |x||w|), through an activation of slope at most 1.13
    whose own fp32 error is 8 units of |y| plus 2^-22 of |z| where 1 + tanh cancels; one addition of the
    residual; one rounding."""
    half = BF16_HALF if dtype == torch.bfloat16 else F32_HALF
    return 1.13 * (K + 1) * F32_HALF * size + 8 * F32_HALF * y.abs() + 2.0 ** -22 * size + (half + F32_HALF) * out.abs()
