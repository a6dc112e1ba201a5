"""64-bit CPU definitions of the paged cache, the attention over it and the residual norm, and their error bounds."""
import math

import torch

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16, "i8": torch.int8,
      "e4m3": torch.float8_e4m3fn}
TOP = {"i8": 127.0, "e4m3": 448.0}
MIN_SCALE = 2.0 ** -60


def half_step(t):
    return torch.finfo(DT.get(t, t)).eps / 2


def quant_rows(x, kind, floor=MIN_SCALE):
    """(codes as float64, scales fp32) of the last axis of x (float64): the formula."""
    big = x.abs().amax(-1)
    ok = torch.isfinite(x).all(-1)
    s = torch.where(ok, big / TOP[kind], torch.zeros_like(big)).float()
    s = torch.where(s < floor, torch.zeros_like(s), s)
    v = torch.where((s > 0)[..., None] & ok[..., None], x / s.double().clamp(min=1e-300)[..., None], torch.zeros_like(x))
    if kind == "i8":
        c = v.round().clamp(-127, 127)
    else:
        m, e = torch.frexp(v)
        ulp = torch.pow(torch.tensor(2.0, dtype=torch.float64), (e - 4).clamp(min=-9).double())
        c = (torch.round(v / ulp) * ulp).clamp(-448, 448)
    return c, torch.where(ok, s, torch.full_like(s, math.nan))


class Paged:
    """A batch of sequences over a paged cache, on the CPU; .gpu() gives the tensors of a call."""

    def __init__(self, ns, ks, Hkv, d, page, qt, kvt, seed=0, pad=0, extra_pages=3, cols=None, v_scale=1.0):
        g = torch.Generator().manual_seed(seed)
        self.ns, self.ks, self.Hkv, self.d, self.page, self.qt, self.kvt = ns, ks, Hkv, d, page, qt, kvt
        self.S, self.N, self.T, self.g = len(ns), sum(ns), sum(ns) + pad, g
        need = [-(-max(k, 0) // page) for k in ks]
        self.n_pages = sum(need) + extra_pages
        self.cols = cols or max(1, max(need))
        ids = torch.randperm(self.n_pages, generator=g).to(torch.int32)
        self.table = torch.full((self.S, self.cols), -1, dtype=torch.int32)   # unused entries: no page
        at = 0
        for s, m in enumerate(need):
            self.table[s, :m] = ids[at:at + m][:self.cols]
            at += m
        self.cu = torch.tensor([0] + [sum(ns[:i + 1]) for i in range(self.S)], dtype=torch.int32)
        self.kv_len = torch.tensor(ks, dtype=torch.int32)
        shape = (self.n_pages, Hkv, page, d)
        x = torch.randn((2,) + shape, generator=g)
        x[1] *= v_scale
        self.set_values(x.to(DT[qt]))

    def set_values(self, x):
        """Cache contents from 16-bit values [2, pages, heads, page, d] (quantised for 8-bit caches)."""
        if self.kvt in TOP:
            c, s = quant_rows(x.double(), self.kvt)
            self.codes = c.float().to(DT[self.kvt])
            self.scales = s.contiguous()
            self.val = c * torch.nan_to_num(s.double(), nan=math.nan)[..., None]
        else:
            self.codes, self.scales, self.val = x.contiguous(), None, x.double()

    def gpu(self, dev):
        def up(t):
            return t.to(dev)
        if self.kvt == "e4m3":
            c = self.codes.view(torch.uint8).to(dev).view(torch.float8_e4m3fn)
        else:
            c = up(self.codes)
        kv = (c[0], c[1]) if self.scales is None else (c[0], c[1], up(self.scales[0]), up(self.scales[1]))
        return kv, up(self.cu), up(self.kv_len), up(self.table)

    def rows(self, which, s, upto):
        """[heads, upto, d] values of sequence s's first `upto` positions, and which of them exist."""
        pos = torch.arange(max(upto, 0))
        pg = pos // self.page
        pid = torch.where(pg < self.cols, self.table[s].long()[pg.clamp(max=self.cols - 1)], torch.full_like(pg, -1))
        have = (pid >= 0) & (pid < self.n_pages)
        v = self.val[which][pid.clamp(0, self.n_pages - 1), :, pos % self.page]
        return v.transpose(0, 1), have


def attention(b, q, Hq, scale, window=0, sinks=0):
    """(out, lse, tolerance of out, tolerance of lse) in float64, [T, Hq, ...]; NaN in rows of no sequence.

    Bounds, per output element, with half steps hc (weights; fp16 for 8-bit caches) and ho (output):
      weights rounded once: hc * A, A = sum_j w_j |v_j|; output rounded once: ho * |out|;
      scores are fp32 sums of d exact products: off by (d + 16) 2^-24 X, X = scale * max_j sum |q k|, and the log2
      arithmetic on numbers up to 1.45 X + 110 by 2^-22 of that; a weight's relative error is twice that sum;
      weights below the smallest normal value of fp16 lose 2^-25 each: keys * 2^-24 * max|v|;
      sums over the keys in fp32: keys * 2^-24 * A."""
    T, d, G = b.T, b.d, Hq // b.Hkv
    out = torch.full((T, Hq, d), math.nan, dtype=torch.float64)
    lse = torch.full((T, Hq), math.nan, dtype=torch.float64)
    tol, tl = torch.zeros_like(out), torch.zeros_like(lse)
    hc = half_step("f16" if b.kvt in TOP else b.qt)
    ho, tiny = half_step(b.qt), torch.finfo(DT[b.qt]).tiny * half_step(b.qt) * 2
    t = 0
    cap = b.cols * b.page
    for s in range(b.S):
        n = b.ns[s]
        k = min(max(int(b.kv_len[s]), 0), cap)
        if n:
            K, have = b.rows(0, s, k)
            V, _ = b.rows(1, s, k)
            x = q[t:t + n].double().view(n, b.Hkv, G, d).permute(1, 0, 2, 3)                 # [Hkv, n, G, d]
            p = (k - n) + torch.arange(n).view(1, n, 1, 1)
            j = torch.arange(k).view(1, 1, 1, k)
            see = have.view(1, 1, 1, k) & (j <= p)
            if window > 0:
                see = see & ((j > p - window) | (j < sinks))
            z = torch.einsum("hngd,hkd->hngk", x, K) * scale
            z = torch.where(see, z, torch.full_like(z, -math.inf))
            m = z.amax(-1, keepdim=True) if k else torch.full(z.shape[:3] + (1,), -math.inf, dtype=torch.float64)
            any_ = see.any(-1, keepdim=True).expand(m.shape)
            e = torch.where(see, torch.exp(z - torch.where(m == -math.inf, torch.zeros_like(m), m)), torch.zeros_like(z))
            l = e.sum(-1, keepdim=True)
            w = torch.where(any_, e / torch.where(any_, l, torch.ones_like(l)), torch.zeros_like(e))

            def mix(v):   # a key that is not seen adds nothing, whatever it holds
                vs = torch.where(torch.isfinite(v), v, torch.zeros_like(v))
                o = torch.einsum("hngk,hkd->hngd", w, vs)
                bad = (~torch.isfinite(v)).any(-1).any(0).nonzero().flatten().tolist()
                for jj in bad:
                    vj = v[:, jj].view(b.Hkv, 1, 1, d)
                    o = torch.where(see[..., jj:jj + 1] & ~torch.isfinite(vj), o + vj, o)
                return o
            o = mix(V)
            nat = torch.nan_to_num(V.abs(), nan=0.0, posinf=0.0)
            A = torch.einsum("hngk,hkd->hngd", torch.nan_to_num(w), nat)
            kk = torch.nan_to_num(K.abs(), nan=0.0, posinf=0.0)
            X = (torch.einsum("hngd,hkd->hngk", x.abs(), kk).amax(-1, keepdim=True) if k else torch.zeros_like(l)) * abs(scale)
            ds = (d + 16) * 2.0 ** -24 * X + 2.0 ** -22 * (1.45 * X + 110)
            vm = nat.amax() if k else torch.tensor(0.0)
            to = hc * A * 1.01 + ho * o.abs() + 2 * ds * A + k * 2.0 ** -24 * (A + vm) + tiny
            L = torch.where(any_, m + torch.log(torch.where(any_, l, torch.ones_like(l))), torch.full_like(m, -math.inf))
            tz = ds + (k + 16) * 2.0 ** -24 + 2.0 ** -22 * torch.nan_to_num(L.abs(), posinf=0.0, nan=0.0)

            def back(y):
                return y.permute(1, 0, 2, 3).reshape(n, Hq, -1)
            out[t:t + n], tol[t:t + n] = back(o), back(to)
            lse[t:t + n], tl[t:t + n] = back(L)[..., 0], back(tz)[..., 0]
        t += n
    return out, lse, tol, tl


def assert_near(got, want, tol, what=""):
    got = got.detach().cpu().double()
    fin = torch.isfinite(want)
    same = torch.where(torch.isnan(want), torch.isnan(got), got == want) | fin
    assert bool(same.all()), f"{what}: {int((~same).sum())} non-finite values differ"
    d = torch.where(fin, (got - want).abs(), torch.zeros_like(want))
    d = torch.where(torch.isnan(d), torch.full_like(d, math.inf), d)
    tol = torch.where(fin, tol, torch.zeros_like(tol))            # bounds are those of finite results
    r = (d / tol.clamp(min=1e-300)).max().item() if d.numel() else 0.0
    assert bool((d <= tol).all()), f"{what}: error up to {d.max().item():.3g}, {r:.3g} of its bound"
    return r
