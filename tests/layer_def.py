"""64-bit definitions of the block quantisation, the block-scaled product, the head norms with rotation, the attention mass
and the eviction, each with bounds of what the kernels' steps may lose."""
import math

import torch

from attn_util import DT, MIN_SCALE, TOP, half_step, quant_rows


def blocks(n):
    return -(-n // 128)


def quant_blocks(x, rows):
    """(codes as float64 [T, D], scales fp32 [ceil(T / rows), ceil(D / 128)]) of x (any type, on the CPU)."""
    T, D = x.shape
    R, C = -(-T // rows), blocks(D)
    p = torch.zeros((R * rows, C * 128), dtype=torch.float64)
    p[:T, :D] = x.double()
    p = p.view(R, rows, C, 128).transpose(1, 2).reshape(R, C, rows * 128)
    c, s = quant_rows(p, "e4m3", MIN_SCALE)
    return c.view(R, C, rows, 128).transpose(1, 2).reshape(R * rows, C * 128)[:T, :D], s


def spread(s, rows, T, K):
    """Scales of blocks of rows x 128, one for each element of [T, K]."""
    return s.double().repeat_interleave(rows, 0)[:T].repeat_interleave(128, 1)[:, :K]


def product(a, sa, b, sb, out):
    """(a b^T, bound) for codes as float64 [T, K], [N, K] and their scales.

    Bounds, A = sum of |products| with their scales: a block's 128 products are exact in fp32 and added by the matrix cores, each
    addition off by at most a step, 2^-23 (their rounding is not specified): 128 * 2^-23 A; scaling (two factors and an fma) and
    adding up to K / 128 blocks, split over waves, in fp32: (K / 128 + 16) 2^-24 A; rounded once to `out`. 16-bit results of more
    than 64 tokens: of each 8 products seven lose less than 2^-13 of the largest, which is at most the product of the largest
    factors among the 8."""
    T, K = a.shape
    x, w = a * spread(sa, 1, T, K), b * spread(sb, 128, b.shape[0], K)
    want = x @ w.t()
    nx, nw = torch.nan_to_num(x.abs(), posinf=0.0), torch.nan_to_num(w.abs(), posinf=0.0)
    A = nx @ nw.t()
    ho = 2.0 ** -24 if out == "f32" else half_step(out)
    tiny = torch.finfo(DT[out]).tiny * ho * 2
    tol = A * (128 * 2.0 ** -23 + (blocks(K) + 16) * 2.0 ** -24) + ho * want.abs() * 1.01 + tiny
    if T > 64 and out != "f32":
        tol = tol + 7 * 2.0 ** -13 * (nx.view(T, -1, 8).amax(-1) @ nw.view(b.shape[0], -1, 8).amax(-1).t())
    return want, tol


def head_rows(x, w, eps, pos, freq, inter, ty):
    """(rows normed and turned, bound) for x [N, H, d] (CPU, 16 bits) at integer positions pos [N].

    Bounds: fp32 sum of d squares and a reciprocal root (d / 2 + 12) 2^-24 relative, with the two factors; sine and cosine: the
    fraction of a turn rounded to fp32 (2^-26 turns, 2^-23.3 in angle) and functions good to four half steps: 1.5 * 2^-22 absolute;
    the angle's four roundings in 64 bits (one of them here): 2^-51 of it; two products and a sum: 3 * 2^-24; rounded once."""
    h = x.double()
    d = h.shape[-1]
    rel = 0.0
    if eps is not None:
        h = h / torch.sqrt(h.square().mean(-1, keepdim=True) + eps)
        h = h if w is None else h * w.double()
        rel = (d / 2 + 12) * 2.0 ** -24
    tol = h.abs() * rel
    if freq is not None:
        m = freq.numel()
        ia = torch.arange(m) * (2 if inter else 1)
        ib = ia + (1 if inter else m)
        ang = pos.double()[:, None] * freq.double()
        c, s = torch.cos(ang)[:, None], torch.sin(ang)[:, None]
        a, b = h[..., ia].clone(), h[..., ib].clone()
        both = a.abs() + b.abs()
        h = h.clone()
        h[..., ia], h[..., ib] = a * c - b * s, b * c + a * s
        turned = both * (rel + 1.5 * 2.0 ** -22 + ang.abs()[:, None] * 2.0 ** -51 + 3 * 2.0 ** -24)
        tol[..., ia] = turned
        tol[..., ib] = turned
    ho = half_step(ty)
    return h, tol + (h.abs() + tol) * ho * 1.01 + torch.finfo(DT[ty]).tiny * ho * 2


def mass(b, q, lse, Hq, scale, old, window=0, sinks=0, max_q=1 << 30):
    """(mass_out, bound) [S, Hkv, W] in float64; NaN where it stays as it was. lse [T, Hq] is an input.

    Bounds: x = score - lse in log2 units is off by ds = (d + 16) 2^-24 X + 2^-22 (1.45 (X + |lse|) + 4), X = |scale| sum |q k|, and
    over an 8-bit cache 2^-38 of the largest query element times sum |k|; the weight by twice that; sums in fp32: rows * 2^-24;
    added to what was there: 2^-24; weights below fp32's normal range may be lost."""
    S, W, G, d = b.S, old.shape[2], Hq // b.Hkv, b.d
    out = torch.full(old.shape, math.nan, dtype=torch.float64)
    tol = torch.zeros_like(out)
    cu = b.cu.tolist()
    for s in range(S):
        n = min(cu[s + 1], b.T) - cu[s]
        if n <= 0:
            continue
        L = int(b.kv_len[s])
        held = max(0, min(L, b.cols * b.page, W))
        if not held:
            continue
        K, have = b.rows(0, s, held)
        m = min(n, max_q)
        x = q[cu[s]:cu[s] + m].double().view(m, b.Hkv, G, d).permute(1, 0, 2, 3).reshape(b.Hkv, m * G, d)
        l = lse[cu[s]:cu[s] + m].double().view(m, b.Hkv, G).permute(1, 0, 2).reshape(b.Hkv, m * G, 1)
        p = (L - (cu[s + 1] - cu[s]) + torch.arange(m)).repeat_interleave(G).view(-1, 1)
        j = torch.arange(held).view(1, -1)
        see = (j <= p) & have.view(1, -1)
        if window > 0:
            see = see & ((j > p - window) | (j < sinks))
        see = see[None] & (l != -math.inf)
        z = x @ K.transpose(1, 2) * scale
        e = torch.where(see, torch.exp(z - l), 0.0)
        X = torch.nan_to_num(x.abs(), posinf=0.0) @ torch.nan_to_num(K.abs(), posinf=0.0).transpose(1, 2) * abs(scale)
        ds = (d + 16) * 2.0 ** -24 * X + 2.0 ** -22 * (1.45 * (X + torch.nan_to_num(l.abs(), posinf=0.0)) + 4)
        if b.kvt in TOP:
            big = torch.nan_to_num(x.abs(), posinf=0.0).amax() if m else 0.0
            ds = ds + 2.0 ** -38 * big * torch.nan_to_num(K.abs()).sum(-1).unsqueeze(1) * abs(scale)
        new = torch.arange(held) >= L - (cu[s + 1] - cu[s])
        was = torch.where(new, 0.0, old[s, :, :held].double())
        add = e.sum(1)
        out[s, :, :held] = was + add
        fin = torch.where(see & torch.isfinite(e), e, 0.0)
        tol[s, :, :held] = (2 * ds * fin).sum(1) + (m * G + 2) * 2.0 ** -24 * (fin.sum(1)) + 2.0 ** -24 * was.abs() + m * G * 2.0 ** -125
    return out, tol


def evicted(n, P, held, mass_, pos, keep, sinks, recent):
    """For one sequence and head with n slots: the slot that each of the first `keep` came from."""
    src = list(range(keep))
    if n <= keep:
        return src

    def order(j):
        m = float(mass_[j])
        if not held[j]:
            return (0, 0.0)
        if pos[j] < sinks or (recent and pos[j] >= P - recent):
            return (2, 0.0)
        return (1, m if m > 0 else 0.0)
    first = sorted(range(n), key=lambda j: order(j) + (-j,), reverse=True)[:keep]
    stay = set(first)
    holes = [j for j in range(keep) if j not in stay]
    movers = sorted(j for j in stay if j >= keep)
    assert len(holes) == len(movers)
    for h, m in zip(holes, movers):
        src[h] = m
    return src
