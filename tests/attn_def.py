"""64-bit definition of the attention over the paged cache, position by position, with bounds of what each step of the
kernels may lose. Positions follow the header alone: token i of n stands at min(kv_len, 2^30 + 2^24) - n + i whatever its
table row holds, and a position outside the row holds no token."""
import math

import torch

from attn_util import DT, TOP, half_step

MOST = (1 << 30) + (1 << 24)


def definition(b, q, Hq, scale, window=0, sinks=0, T=None):
    """(out, lse, tolerance of out, tolerance of lse) in float64 for the rows that cu names below T (default: all of
    b's); NaN elsewhere.

    Bounds per output element, hc and ho half steps of the weights' type (fp16 over 8-bit caches) and of the output's,
    A = sum_j w_j |v_j|, X = scale * max_j sum |q k|:
      hc A               weights rounded once;
      k 2^-32 max|v| / l fp16 weights under 2^-14, off by 2^-25 each where the largest one is at least 2^7 and their sum l
                         times that (bf16 has fp32's exponents: nothing);
      2 ds A             scores: ds = (d + 16) 2^-24 X + 2^-22 (1.45 X + 110);
      k 2^-24 A          sums over the keys in fp32;
      ho |out|           output rounded once (below the smallest normal value: by half of that value's step)."""
    T = b.T if T is None else T
    d, G = b.d, Hq // b.Hkv
    out = torch.full((T, Hq, d), math.nan, dtype=torch.float64)
    lse = torch.full((T, Hq), math.nan, dtype=torch.float64)
    tol, tl = torch.zeros_like(out), torch.zeros_like(lse)
    f16 = b.kvt in TOP or b.qt == "f16"
    hc, ho = half_step("f16" if b.kvt in TOP else b.qt), half_step(b.qt)
    tiny = torch.finfo(DT[b.qt]).tiny * ho * 2
    cu = b.cu.tolist()
    for s in range(b.S):
        n, last = cu[s + 1] - cu[s], min(cu[s + 1], T)
        if last <= cu[s]:
            continue
        k = min(int(b.kv_len[s]), MOST)
        held = max(0, min(k, b.cols * b.page))
        K, have = b.rows(0, s, held)
        V, _ = b.rows(1, s, held)
        m = last - cu[s]
        x = q[cu[s]:last].double().view(m, b.Hkv, G, d).permute(1, 0, 2, 3).reshape(b.Hkv, m * G, d)
        p = (k - n + torch.arange(m)).repeat_interleave(G).view(-1, 1)
        j = torch.arange(held).view(1, -1)
        see = (j <= p) & have.view(1, -1)
        if window > 0:
            see = see & ((j > p - window) | (j < sinks))
        see = see[None].expand(b.Hkv, -1, -1)
        z = torch.where(see, x @ K.transpose(1, 2) * scale, -math.inf)
        some = see.any(-1, keepdim=True)
        big = torch.where(some, z.amax(-1, keepdim=True) if held else torch.zeros_like(x[..., :1]), 0.0)
        e = torch.where(see, torch.exp(z - big), 0.0)
        l = e.sum(-1, keepdim=True)
        w = torch.where(some, e / l, 0.0)
        plain = torch.where(torch.isfinite(V), V, 0.0)
        o = w @ plain
        for jj in (~torch.isfinite(V)).any(-1).any(0).nonzero().flatten().tolist():
            v = V[:, jj].unsqueeze(1)                         # what it holds shows wherever the key is seen
            o = torch.where(see[..., jj:jj + 1] & ~torch.isfinite(v), o + v, o)
        A = torch.nan_to_num(w) @ plain.abs()
        X = (x.abs() @ torch.nan_to_num(K.abs(), posinf=0.0).transpose(1, 2)).amax(-1, keepdim=True) * abs(scale) if held else torch.zeros_like(l)
        ds = (d + 16) * 2.0 ** -24 * X + 2.0 ** -22 * (1.45 * X + 110)
        vm = plain.abs().amax() if held else torch.zeros(())
        to = hc * A * 1.01 + ho * o.abs() * 1.01 + 2 * ds * A + held * 2.0 ** -24 * A + tiny
        if f16:
            to = to + held * 2.0 ** -32 * vm * 1.01 / torch.where(some, l, 1.0)
        L = torch.where(some, big + torch.log(torch.where(some, l, 1.0)), -math.inf)
        tz = ds + (held + 16) * 2.0 ** -24 + 2.0 ** -22 * torch.nan_to_num(L.abs(), posinf=0.0)

        def back(y):
            return y.view(b.Hkv, m, G, -1).permute(1, 0, 2, 3).reshape(m, Hq, -1)
        out[cu[s]:last], tol[cu[s]:last] = back(o), back(to)
        lse[cu[s]:last], tl[cu[s]:last] = back(L)[..., 0], back(tz)[..., 0]
    return out, lse, tol, tl
