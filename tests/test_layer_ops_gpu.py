"""Block quantisation, 8-bit product, head norms with rotation, attention mass and eviction on the GPU against their 64-bit
definitions (tests/layer_def.py)."""
import math

import pytest
import torch

from activation_sparse_ffn_predictor_amd import _lib
from attn_util import DT, Paged, assert_near, attention
from layer_def import blocks, evicted, head_rows, mass, product, quant_blocks

pytestmark = pytest.mark.gpu
E4M3 = torch.float8_e4m3fn


def say(*a):
    print(*a, flush=True)


def f64(t):
    if t.dtype == E4M3:
        t = t.view(torch.uint8).cpu().view(E4M3)
    return t.cpu().float().double()


def codes(c):
    """Codes (float64) as e4m3 on the CPU."""
    return c.float().to(E4M3)


def up(t, dev):
    return t.view(torch.uint8).to(dev).view(E4M3) if t.dtype == E4M3 else t.to(dev)


# ------------------------------------------------------------------------------------------------ block quantisation
QUANT = [(1, 8, "f32", 1), (1, 8192, "f16", 1), (3, 128, "bf16", 1), (5, 136, "f16", 1), (33, 1000, "bf16", 1),
         (17, 2056, "f32", 1), (300, 264, "f32", 1), (1, 8, "f16", 128), (127, 120, "bf16", 128), (129, 136, "f32", 128),
         (256, 256, "f16", 128), (300, 1032, "bf16", 128), (2, 65536, "f16", 1)]


def quant(dev, x, rows, pad=0):
    T, D = x.shape
    big = torch.full((T, D + pad), 3.0).to(x.dtype).to(dev)
    big[:, :D] = x.to(dev)
    y = torch.full((T + 1, D + pad), 7.0).to(E4M3).to(dev)
    sc = torch.full((-(-T // rows) + 1, blocks(D)), -1.0, device=dev)
    _lib.quant128(big[:, :D], y[:T, :D], sc[:-1], rows=rows)
    torch.cuda.synchronize()
    assert bool((f64(y[T]) == 7).all()) and bool((sc[-1] == -1).all())                 # nothing behind is written
    assert pad == 0 or bool((f64(y[:T, D:]) == 7).all())
    return f64(y[:T, :D]), sc[:-1].cpu()


@pytest.mark.parametrize("T,D,xt,rows", QUANT)
def test_quant(gpu_ready, T, D, xt, rows):
    g = torch.Generator().manual_seed(T * 7 + D)
    x = (torch.randn((T, D), generator=g) * torch.exp(2 * torch.randn(D, generator=g))).to(DT[xt])
    if T > 2:
        x[1] = 0                                                                       # (a block of zeros where rows == 1)
        x[2, : D // 2] *= 2.0 ** -12
    for pad in (0, 24):
        say(f"[quant {T} {D} {xt} {rows} pad {pad}]")
        y, s = quant(gpu_ready, x, rows, pad)
        wy, ws = quant_blocks(x, rows)
        assert torch.equal(s, ws)
        assert torch.equal(y, wy)


@pytest.mark.parametrize("xt", ["f32", "f16", "bf16"])
def test_quant_borders(gpu_ready, xt):
    """Every border between two codes, and its neighbours on both sides, times a scale that is no power of two."""
    top = torch.tensor([448.0])
    vals = [m / 8 * 2.0 ** e for e in range(-7, 9) for m in range(0, 33)]
    v = torch.tensor(sorted(set(x for x in vals if x <= 448)), dtype=torch.float64)
    for k in (1.0, 1.0 / 3, 0.7134):
        x = (v * k).to(DT[xt])
        bits = x.view(torch.int32 if xt == "f32" else torch.int16)
        near = torch.cat([x, (bits + 1).view(DT[xt]), (bits - 1).clamp(min=0).view(DT[xt])])
        near = torch.cat([near, -near])
        near = near[near.float().abs() <= float((top * k).to(DT[xt]))]
        n = -(-near.numel() // 127)
        m = torch.zeros(n * 127, dtype=DT[xt])
        m[:near.numel()] = near
        x = torch.cat([m.view(n, 127), (top * k).to(DT[xt]).expand(n, 1)], 1).contiguous()
        say(f"[borders {xt} {k}]")
        for rows in (1, 128):
            y, s = quant(gpu_ready, x, rows)
            wy, ws = quant_blocks(x, rows)
            assert torch.equal(s, ws) and torch.equal(y, wy)


@pytest.mark.parametrize("xt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows", [1, 128])
def test_quant_nonfinite_and_small(gpu_ready, xt, rows):
    x = torch.ones((4 * rows, 384)).to(DT[xt])
    x[0, 5], x[rows, 130], x[2 * rows, 383] = math.inf, math.nan, -math.inf
    x[3 * rows:, :128] = 0
    if xt != "f16":
        x[3 * rows:, 128:256] = 448 * 2.0 ** -61                                       # scale 2^-61: zeros
        x[3 * rows:, 256:] = 448 * 2.0 ** -60
    y, s = quant(gpu_ready, x, rows)
    wy, ws = quant_blocks(x, rows)
    assert torch.equal(torch.isnan(s), torch.isnan(ws)) and torch.equal(torch.nan_to_num(s), torch.nan_to_num(ws))
    assert torch.equal(y, wy)
    assert int(torch.isnan(s).sum()) == 3


# ------------------------------------------------------------------------------------------------ the product
MM = [(1, 8, 16, "f32"), (1, 4096, 4096, "f16"), (1, 1032, 8192, "bf16"), (3, 136, 144, "f32"), (16, 128, 1024, "f16"),
      (17, 264, 272, "bf16"), (32, 72, 128, "f32"), (37, 15360, 5120, "bf16"), (64, 512, 2048, "f16"), (65, 128, 128, "f32"),
      (100, 1000, 1040, "f16"), (128, 136, 384, "f32"), (129, 648, 528, "bf16"), (257, 264, 16, "f32"), (300, 2048, 4096, "f32"),
      (1000, 776, 656, "f16"), (2, 16, 65536, "f32"), (513, 1288, 1536, "f32"), (80, 8, 1024, "f32"), (2048, 2304, 2048, "bf16"),
      # every kernel that larger calls choose, k in one share and in several, with ends inside tiles, blocks and shares
      (4, 20008, 1168, "f16"), (9, 5128, 4112, "bf16"), (24, 1032, 4096, "f16"), (31, 24584, 640, "f32"), (48, 2056, 8208, "bf16"),
      (60, 16392, 912, "f16"), (100, 2056, 4112, "f32"), (90, 12808, 528, "f32"), (128, 10248, 4112, "f16"), (300, 4104, 4112, "bf16"),
      (512, 10248, 8208, "f16"), (200, 2056, 4096, "f32"), (2100, 8200, 656, "bf16"), (640, 10240, 1040, "f16"), (1500, 1032, 2064, "f32")]


def mm_case(T, N, K, seed=0):
    g = torch.Generator().manual_seed(seed + T * 3 + N * 5 + K)
    a, sa = quant_blocks(torch.randn((T, K), generator=g) * torch.exp(torch.randn(K, generator=g)), 1)
    b, sb = quant_blocks(torch.randn((N, K), generator=g) * torch.exp(torch.randn(N, 1, generator=g)), 128)
    return a, sa, b, sb


def mm(dev, a, sa, b, sb, ot, pad=0):
    T, K = a.shape
    N = b.shape[0]
    ga = torch.full((T + 1, K + 2 * pad), math.nan).to(E4M3)                            # what lies between the rows is not read
    gb = torch.full((N + 1, K + 2 * pad), math.nan).to(E4M3)
    ga[:T, :K], gb[:N, :K] = codes(a), codes(b)
    ga, gb = up(ga, dev), up(gb, dev)
    out = torch.full((T + 1, N + pad), 7.0).to(DT[ot]).to(dev)
    need = _lib.mm_workspace_size(T, N, K)
    ws = torch.full((need,), 255, dtype=torch.uint8, device=dev) if need else None     # (NaN, if it were read)
    _lib.mm_e4m3(ga[:T, :K], sa.to(dev), gb[:N, :K], sb.to(dev), out[:T, :N], ws)
    torch.cuda.synchronize()
    assert bool((out[T] == 7).all()) and (pad == 0 or bool((out[:T, N:] == 7).all()))
    return out[:T, :N]


@pytest.mark.parametrize("T,N,K,ot", MM)
def test_mm(gpu_ready, T, N, K, ot):
    a, sa, b, sb = mm_case(T, N, K)
    if T * N * K > 1 << 32:
        want, tol = (t.cpu() for t in product(a.to(gpu_ready), sa.to(gpu_ready), b.to(gpu_ready), sb.to(gpu_ready), ot))
    else:
        want, tol = product(a, sa, b, sb, ot)
    first = None
    for pad in (0, 8):
        say(f"[mm {T} {N} {K} {ot} pad {pad}]")
        out = mm(gpu_ready, a, sa, b, sb, ot, pad)
        say("  ", assert_near(out, want, tol, "out"))
        first = out.clone() if first is None else first
        assert torch.equal(out, first)                                                 # the same bits whatever the strides


@pytest.mark.parametrize("T", [5, 40, 200])
def test_mm_values(gpu_ready, T):
    """Every code once against every code: the products' own values; and a NaN code, scale or zero scale where it belongs."""
    dev = gpu_ready
    every = torch.arange(256, dtype=torch.uint8).view(E4M3)
    every = every[~torch.isnan(every.float())].float().double()                        # 254
    K = 256
    a = torch.zeros((T, K), dtype=torch.float64)
    b = torch.zeros((264, K), dtype=torch.float64)
    for t in range(T):
        a[t, (7 * t) % K] = every[(53 * t) % 254]
    b[:254] = every[:, None]
    sa, sb = torch.full((T, 2), 0.5), torch.full((3, 2), 2.0)
    say(f"[mm values {T}]")
    out = mm(dev, a, sa, b, sb, "f32")
    assert torch.equal(out.cpu().double(), a @ b.t())                                  # one product each: exact
    a[1, 3] = math.nan
    sa[2, 1], sb[1, 0] = math.nan, math.inf
    sa[3] = 0
    want, tol = product(torch.nan_to_num(a), torch.nan_to_num(sa, nan=1.0), b, torch.nan_to_num(sb, posinf=1.0), "f32")
    out = mm(dev, a, sa, b, sb, "f32").cpu()
    assert bool(torch.isnan(out[1:3]).all())
    assert bool((out[3, :128] == 0).all())
    assert_near(out[4:, :128], want[4:, :128], tol[4:, :128])
    assert_near(out[4:, 256:], want[4:, 256:], tol[4:, 256:])


# ------------------------------------------------------------------------------------------------ head norms and rotation
ROPE = [([1], [5001], 64, 8, 128, 128, False, True, "f16", 0), ([1], [1], 1, 1, 8, 8, False, True, "bf16", 0),
        ([3, 0, 5], [3, 9, 5], 8, 2, 64, 64, True, True, "f16", 2), ([2, 1, 4, 1], [1000000, 70001, 33, 1], 5, 5, 72, 72, False, True, "bf16", 1),
        ([7, 1], [4097, 2], 12, 4, 80, 40, False, False, "f16", 0), ([1] * 70, list(range(1, 71)), 32, 1, 96, 96, True, True, "bf16", 0),
        ([33], [2 ** 20 + 77], 40, 40, 128, 64, True, True, "bf16", 5), ([4, 6], [100, 7], 4, 2, 256, 256, False, True, "f16", 0),
        ([5], [3], 3, 1, 16, 16, False, False, "f16", 0), ([9], [9000], 16, 2, 112, 112, False, True, "f16", 0),
        ([2, 3], [77, 78], 6, 6, 48, 0, False, True, "bf16", 1), ([300, 1, 45], [5000, 60000, 45], 7, 1, 128, 128, False, True, "f16", 3),
        ([1, 1], [2 ** 24 + 3, 2 ** 30 + 12345], 2, 2, 32, 32, False, True, "f16", 0), ([11], [12], 3, 3, 24, 16, True, True, "f16", 0)]


def freqs(rot, base=10000.0):
    return (base ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)).float() if rot else None


@pytest.mark.parametrize("ns,ps,Hq,Hk,d,rot,inter,norm,ty,pad", ROPE)
def test_rope(gpu_ready, ns, ps, Hq, Hk, d, rot, inter, norm, ty, pad):
    dev, N = gpu_ready, sum(ns)
    g = torch.Generator().manual_seed(N + d)
    wide = (torch.randn((N + pad, (Hq + 2 * Hk) * d), generator=g) * 2).to(DT[ty])
    wq, wk = (1 + 0.3 * torch.randn(d, generator=g) for _ in range(2))
    if not norm:
        wq = wk = None
    fr, eps = freqs(rot), 1e-6 if norm else None
    cu = torch.tensor([0] + [sum(ns[:i + 1]) for i in range(len(ns))], dtype=torch.int32)
    pos = torch.cat([torch.arange(p - n, p) for n, p in zip(ns, ps)])
    q, k = wide[:, :Hq * d].unflatten(1, (Hq, d)), wide[:, Hq * d:(Hq + Hk) * d].unflatten(1, (Hk, d))
    wants = [head_rows(x[:N], w, eps, pos, fr, inter, ty) for x, w in ((q, wq), (k, wk))]
    cg, lg = cu.to(dev), torch.tensor(ps, dtype=torch.int32, device=dev)
    args = [None if w is None else w.to(dev) for w in (wq, wk)] + [eps, cg, lg, None if fr is None else fr.to(dev)]
    # to other tensors
    gw = wide.to(dev)
    gq, gk = gw[:, :Hq * d].unflatten(1, (Hq, d)), gw[:, Hq * d:(Hq + Hk) * d].unflatten(1, (Hk, d))
    qo, ko = torch.full((N + pad, Hq, d), 7.0, dtype=DT[ty], device=dev), torch.full((N + pad, Hk, d), 7.0, dtype=DT[ty], device=dev)
    say(f"[rope {ns[:4]} {ps[:4]} {Hq} {Hk} {d} {rot} {inter} {norm} {ty}]")
    _lib.qk_norm_rope(gq, gk, *args, qo, ko, interleaved=inter)
    torch.cuda.synchronize()
    for o, (w, t) in zip((qo, ko), wants):
        say("  ", assert_near(o[:N], w, t))
        assert bool((o[N:] == 7).all())
    # in place, and queries alone
    alone = torch.empty_like(qo)
    _lib.qk_norm_rope(gq, None, *args, alone, None, interleaved=inter)
    _lib.qk_norm_rope(gq, gk, *args, gq, gk, interleaved=inter)
    torch.cuda.synchronize()
    assert torch.equal(alone[:N], qo[:N]) and torch.equal(gq[:N], qo[:N]) and torch.equal(gk[:N], ko[:N])
    assert torch.equal(gw[N:].cpu(), wide[N:]) and torch.equal(gw[:, (Hq + Hk) * d:].cpu(), wide[:, (Hq + Hk) * d:])


def test_rope_extremes(gpu_ready):
    """Heads whose squares leave fp32's range, zeros without and with eps, infinities and NaN only in their own head; tokens
    before a sequence's first (negative positions)."""
    dev, d = gpu_ready, 64
    x = torch.randn((6, 3, d), generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    x[0, 0] *= 2.0 ** 70
    x[1, 1] *= 2.0 ** -75
    x[2, 2] = 0
    x[3, 0, 5], x[3, 1, 6] = math.inf, math.nan
    cu, ln = torch.tensor([0, 6], dtype=torch.int32, device=dev), torch.tensor([2], dtype=torch.int32, device=dev)
    o = torch.zeros_like(x, device=dev)
    fr = freqs(d)
    for eps in (1e-5, 0.0):
        _lib.qk_norm_rope(x.to(dev), None, None, None, eps, cu, ln, fr.to(dev), o, None)
        w, t = head_rows(x, None, eps, torch.arange(-4, 2), fr, False, "bf16")
        got = o.cpu()
        bad = ~torch.isfinite(w).all(-1)
        assert bool(bad[3, 0]) and bool(bad[3, 1]) and int(bad.sum()) == (2 if eps else 3)
        assert bool(torch.isnan(got[3, :2]).any(-1).all())
        ok = ~bad
        assert_near(got[ok], w[ok], t[ok])


# ------------------------------------------------------------------------------------------------ attention mass
MASS = [([1], [1], 1, 1, 16, 16, "f16", "f16", 0, 0, 0), ([1], [500], 64, 8, 128, 16, "f16", "f16", 0, 0, 0),
        ([1, 1, 1], [33, 1, 700], 8, 8, 64, 32, "bf16", "bf16", 0, 0, 1), ([1, 0, 2], [129, 64, 40], 5, 5, 80, 16, "f16", "i8", 0, 0, 0),
        ([3, 4, 1], [3, 100, 17], 8, 2, 96, 64, "bf16", "i8", 0, 0, 2), ([2, 1], [300, 31], 32, 1, 112, 16, "bf16", "e4m3", 0, 0, 0),
        ([4, 4], [900, 64], 16, 1, 256, 32, "f16", "e4m3", 100, 4, 0), ([5], [515], 14, 2, 48, 16, "bf16", "bf16", 64, 0, 0),
        ([70], [70], 2, 2, 64, 16, "f16", "f16", 0, 0, 0), ([100, 33], [300, 33], 8, 2, 128, 64, "bf16", "bf16", 0, 0, 3),
        ([257, 1, 0, 90], [600, 5, 40, 300], 12, 4, 80, 32, "f16", "f16", 0, 0, 1), ([150], [1000], 8, 1, 128, 128, "f16", "i8", 200, 16, 0),
        ([150, 20], [700, 333], 4, 4, 256, 64, "bf16", "e4m3", 0, 0, 0), ([200], [900], 8, 2, 72, 16, "bf16", "bf16", 33, 5, 2),
        ([1000], [1000], 16, 2, 64, 32, "f16", "f16", 0, 0, 0), ([40, 40], [2000, 40], 16, 8, 16, 16, "bf16", "e4m3", 0, 0, 0),
        ([300], [520], 8, 1, 160, 16, "f16", "i8", 0, 0, 0), ([64], [64], 1, 1, 256, 16, "f16", "f16", 7, 2, 0),
        ([300], [900], 24, 2, 128, 16, "bf16", "i8", 0, 0, 0), ([130, 400], [500, 700], 9, 3, 64, 32, "f16", "e4m3", 0, 0, 2),
        ([333], [1200], 20, 4, 96, 16, "bf16", "bf16", 300, 9, 0), ([600], [600], 8, 8, 112, 16, "f16", "e4m3", 0, 0, 0)]


def mass_call(dev, b, q, lse, Hq, scale, old, window, sinks, max_q, max_kv, plen=None, in_place=False):
    kv, cu, kl, tab = b.gpu(dev)
    W = old.shape[2]
    m = old.to(dev)
    out = m if in_place else torch.full_like(m, 7.0)
    pos = torch.full(old.shape, -5, dtype=torch.int32, device=dev)
    need = _lib.attn_mass_workspace_size(b.S, Hq, b.Hkv, b.d, max_q, max_kv, W)
    ws = torch.full((need,), 255, dtype=torch.uint8, device=dev) if need else None
    _lib.attn_mass(q.to(dev), kv, cu, kl, tab, max_q, max_kv, lse.to(dev), m, pos, ws, seq_len=plen, mass_out=out, scale=scale,
                   window=window, sinks=sinks)
    torch.cuda.synchronize()
    return out, pos


@pytest.mark.parametrize("ns,ks,Hq,Hkv,d,page,qt,kvt,window,sinks,pad", MASS)
def test_mass(gpu_ready, ns, ks, Hq, Hkv, d, page, qt, kvt, window, sinks, pad):
    dev = gpu_ready
    b = Paged(ns, ks, Hkv, d, page, qt, kvt, seed=d, pad=pad)
    q = torch.randn((b.T, Hq, d), generator=b.g).to(DT[qt])
    scale = d ** -0.5
    _, lse, _, _ = attention(b, q, Hq, scale, window, sinks)
    lse = lse.float()                                                                  # NaN in rows of no sequence
    W = b.cols * page + 3
    old = torch.rand((b.S, Hkv, W), generator=b.g) * 5
    want, tol = mass(b, q, lse, Hq, scale, old, window, sinks)
    plen = torch.tensor([k + 1000 for k in ks], dtype=torch.int32, device=dev)
    for max_kv, in_place in ((max(ks), False), (17, False), (1 << 20, True)):
        say(f"[mass {ns} {ks} {Hq} {Hkv} {d} {page} {qt} {kvt} {window} {sinks} hint {max_kv}]")
        out, pos = mass_call(dev, b, q, lse, Hq, scale, old, window, sinks, max(ns), max_kv, plen, in_place)
        got, stay = out.cpu().double(), torch.isnan(want)
        assert torch.equal(got[stay], (old.double() if in_place else torch.full_like(got, 7.0))[stay])
        say("  ", assert_near(torch.where(stay, torch.zeros_like(got), got), torch.where(stay, torch.zeros_like(want), want), tol))
        wp = torch.full(old.shape, -5, dtype=torch.int32)
        for s, (n, k) in enumerate(zip(ns, ks)):
            wp[s, :, k - n:k] = torch.arange(k - n, k, dtype=torch.int32) + 1000
        assert torch.equal(pos.cpu(), wp)
        again, _ = mass_call(dev, b, q, lse, Hq, scale, old, window, sinks, max(ns), max_kv, plen, in_place)
        assert torch.equal(out, again)
    # every row's weights sum to 1 where nothing was there before
    if not window:
        zero, _ = mass_call(dev, b, q, lse, Hq, scale, torch.zeros_like(old), window, sinks, max(ns), max(ks), plen, True)
        for s, n in enumerate(ns):
            total = zero[s].double().sum().item()
            assert abs(total - n * Hq) <= 1e-3 * max(1, n * Hq)


@pytest.mark.parametrize("n,qt,kvt", [(1, "f16", "f16"), (1, "bf16", "i8"), (1, "f16", "e4m3"), (90, "f16", "f16"), (90, "bf16", "i8"), (90, "bf16", "bf16")])
def test_mass_masked_places(gpu_ready, n, qt, kvt):
    """Infinities and NaN in slots that no row sees, bad pages, a table row shorter than the sequence, rows without a sum, rows past
    max_q, W inside the sequence."""
    dev, Hq, d, page = gpu_ready, 4, 64, 16
    ns, ks = [n, n + 4, 1], [n + 150, 90 + n, 1]
    b = Paged(ns, ks, 2, d, page, qt, kvt, seed=n, pad=2)
    # the slots behind each sequence's end, in its last page
    x = torch.randn((2, b.n_pages, 2, page, d), generator=b.g)
    for s, k in enumerate(ks):
        if k % page:
            x[:, b.table[s, k // page].long(), :, k % page:] = math.nan
    b.set_values(x.to(DT[qt]))
    b.table[0, 3] = 1 << 20                                                            # a page that does not exist
    b.table[0, 5] = -7
    q = torch.randn((b.T, Hq, d), generator=b.g).to(DT[qt])
    _, lse, _, _ = attention(b, q, Hq, 0.2)
    lse = lse.float()
    lse[0, 1] = -math.inf                                                              # a row that saw nothing
    lse[n + 1, 2] = math.nan
    q[n + 2, 3, 7] = math.inf
    for W in (b.cols * page, 100):
        old = torch.rand((3, 2, W), generator=b.g)
        for max_q in (n + 4, n):
            want, tol = mass(b, q, lse, Hq, 0.2, old, max_q=max_q)
            say(f"[masked {n} {qt} {kvt} W {W} max_q {max_q}]")
            out, pos = mass_call(dev, b, q, lse, Hq, 0.2, old, 0, 0, max_q, max(ks))
            held = torch.tensor([min(k, b.cols * page, W) for k in ks]).view(3, 1, 1)
            want = torch.where(torch.arange(W) < held, want, 7.0)
            odd = int(torch.isnan(want).sum()), int(torch.isinf(want).sum())
            assert max_q == n or min(odd) > 0
            assert_near(out, want, tol)


def test_mass_after_attn(gpu_ready):
    """With the log-sum-exp that attn wrote: weights of every row sum to 1, on a stream of its own."""
    dev = gpu_ready
    for ns, ks, Hq, Hkv, kvt in (([1, 1], [4000, 77], 16, 4, "i8"), ([120, 5], [400, 9], 8, 8, "f16")):
        b = Paged(ns, ks, Hkv, 128, 32, "f16", kvt, seed=3)
        kv, cu, kl, tab = b.gpu(dev)
        q = torch.randn((b.T, Hq, 128), generator=b.g).half().to(dev)
        out, lse = torch.zeros_like(q), torch.zeros((b.T, Hq), device=dev)
        W = b.cols * 32
        m, pos = torch.full((2, Hkv, W), 3.0, device=dev), torch.zeros((2, Hkv, W), dtype=torch.int32, device=dev)
        m[:, :, :] = 0
        need = _lib.attn_workspace_size(b.T, 2, Hq, Hkv, 128, max(ns), max(ks))
        ws = torch.empty(max(need, 256), dtype=torch.uint8, device=dev)
        need = _lib.attn_mass_workspace_size(2, Hq, Hkv, 128, max(ns), max(ks), W)
        wm = torch.empty(max(need, 256), dtype=torch.uint8, device=dev)
        st = torch.cuda.Stream()
        st.wait_stream(torch.cuda.current_stream())
        _lib.attn(q, kv, cu, kl, tab, max(ns), max(ks), out, ws, lse=lse, stream=st)
        _lib.attn_mass(q, kv, cu, kl, tab, max(ns), max(ks), lse, m, pos, wm, stream=st)
        st.synchronize()
        for s in range(2):
            G = Hq // Hkv
            per = m[s].double().sum(-1).cpu()
            assert bool(((per - ns[s] * G).abs() <= 1e-3 * ns[s] * G).all())


@pytest.mark.parametrize("Hq,Hkv,d,kvt", [(16, 2, 128, "bf16"), (6, 2, 64, "i8"), (4, 1, 256, "e4m3")])
def test_mass_strided_rows(gpu_ready, Hq, Hkv, d, kvt):
    """Queries that are a part of wider rows, whose other parts hold NaN: the bits of the call on their copy."""
    dev = gpu_ready
    for ns, ks in (([1, 3], [70, 90]), ([200, 37], [500, 300])):
        b = Paged(ns, ks, Hkv, d, 16, "bf16", kvt, seed=d)
        wide = torch.full((b.T, Hq + 3, d), math.nan, dtype=DT["bf16"])
        wide[:, 2:2 + Hq] = torch.randn((b.T, Hq, d), generator=b.g).to(DT["bf16"])
        _, lse, _, _ = attention(b, wide[:, 2:2 + Hq], Hq, 0.1)
        kv, cu, kl, tab = b.gpu(dev)
        old = torch.rand((2, Hkv, b.cols * 16), generator=b.g).to(dev)
        q, l = wide.to(dev)[:, 2:2 + Hq], lse.float().to(dev)
        need = _lib.attn_mass_workspace_size(2, Hq, Hkv, d, max(ns), max(ks), old.shape[2])
        ws = torch.full((need,), 255, dtype=torch.uint8, device=dev) if need else None
        got = []
        for x in (q, q.contiguous()):
            out, pos = old.clone(), torch.zeros(old.shape, dtype=torch.int32, device=dev)
            say(f"[strided {Hq} {Hkv} {d} {kvt} {ns} {x.stride(0)}]")
            _lib.attn_mass(x, kv, cu, kl, tab, max(ns), max(ks), l, out, pos, ws, scale=0.1)
            torch.cuda.synchronize()
            got.append(out)
        assert torch.equal(*got) and bool(torch.isfinite(got[0]).all())


def test_mass_far_max_q(gpu_ready):
    """max_q is an upper bound, up to the largest int: also where its product with the shared heads passes 32 bits."""
    dev, Hq, Hkv, d = gpu_ready, 8, 2, 64
    for n in (9, 70):
        b = Paged([n], [200], Hkv, d, 16, "f16", "f16", seed=n)
        q = torch.randn((b.T, Hq, d), generator=b.g).to(DT["f16"])
        _, lse, _, _ = attention(b, q, Hq, 0.1)
        lse = lse.float()
        old = torch.rand((1, Hkv, b.cols * 16), generator=b.g)
        want, tol = mass(b, q, lse, Hq, 0.1, old)
        for max_q in (1 << 29, 1 << 30, (1 << 30) + 1, (1 << 31) - 1):
            say(f"[far {n} {max_q}]")
            out, _ = mass_call(dev, b, q, lse, Hq, 0.1, old, 0, 0, max_q, 200)
            assert_near(torch.where(torch.isnan(want), 0.0, out.cpu().double()), torch.nan_to_num(want), tol)


# ------------------------------------------------------------------------------------------------ eviction
EVICT = [([40, 16, 7], 16, 4, 2, 1, 16, 16, "f16"), ([1100, 1024, 1025, 30], 1024, 256, 4, 8, 128, 16, "f16"),
         ([300], 1, 0, 0, 2, 64, 32, "i8"), ([300, 299], 100, 1, 0, 3, 80, 16, "e4m3"), ([5000], 4999, 0, 0, 1, 32, 64, "bf16"),
         ([9000, 8193], 3000, 500, 16, 2, 48, 128, "i8"), ([70000], 30000, 1000, 4, 1, 16, 1024, "f16"), ([64] * 20, 32, 8, 0, 2, 256, 16, "e4m3"),
         ([600000], 250000, 70000, 5, 1, 16, 1024, "i8"), ([20000, 8200, 9000], 8500, 8000, 500, 2, 16, 64, "f16"), ([200], 200, 50, 4, 1, 24, 16, "f16"), ([130], 129, 64, 65, 2, 112, 16, "i8"),
         # enough rows that several are moved at a time
         ([20000], 9000, 100, 2, 4, 256, 16, "f16"), ([30000, 12001], 12000, 0, 0, 6, 128, 64, "bf16"),
         ([40000, 30001], 12000, 100, 4, 6, 96, 32, "e4m3")]


def evict_case(ks, keep, Hkv, d, page, kvt, seed=0, kind="mixed", extra=0):
    b = Paged([0] * len(ks), ks, Hkv, d, page, "bf16" if kvt == "bf16" else "f16", kvt, seed=seed)
    W = b.cols * page + extra
    g = torch.Generator().manual_seed(seed + 1)
    m = torch.exp(2 * torch.randn((b.S, Hkv, W), generator=g))
    if kind == "mixed":
        m = torch.where(torch.rand(m.shape, generator=g) < 0.2, (m * 2).round() / 2, m)   # ties, zeros among them
    elif kind == "same":
        m[:] = 0.5
    elif kind == "zero":
        m[:] = 0
    elif kind == "odd":
        r = torch.rand(m.shape, generator=g)
        m = torch.where(r < 0.1, torch.full_like(m, math.nan), m)
        m = torch.where((r > 0.1) & (r < 0.2), -m, m)
        m = torch.where((r > 0.2) & (r < 0.25), torch.full_like(m, math.inf), m)
        m = torch.where((r > 0.25) & (r < 0.3), m * 2.0 ** -140, m)
    pos = torch.stack([torch.stack([torch.randperm(3 * W, generator=g)[:W] for _ in range(Hkv)]) for _ in ks]).to(torch.int32)
    plen = torch.full((b.S,), 3 * W, dtype=torch.int32)
    return b, W, m, pos, plen


def evict_call(dev, b, m, pos, plen, keep, sinks, recent, in_place):
    kv, _, kl, tab = b.gpu(dev)
    gm, gp, gl = m.to(dev), pos.to(dev), plen.to(dev)
    src = torch.full((b.S, b.Hkv, keep), -9, dtype=torch.int32, device=dev)
    out = (None, None, None) if in_place else (torch.full_like(kl, -3), torch.full_like(gm, 7.0), torch.full_like(gp, -7))
    ws = torch.empty(_lib.kv_evict_workspace_size(b.S, b.Hkv, m.shape[2], keep), dtype=torch.uint8, device=dev)
    _lib.kv_evict(kv, kl, tab, gm, gp, keep, src, ws, seq_len=gl, sinks=sinks, recent=recent, kv_len_out=out[0], mass_out=out[1], pos_out=out[2])
    torch.cuda.synchronize()
    return kv, src.cpu(), (kl if in_place else out[0]).cpu(), (gm if in_place else out[1]).cpu(), (gp if in_place else out[2]).cpu()


def check_evict(dev, b, W, m, pos, plen, keep, sinks, recent, in_place):
    kv, src, kl, mo, po = evict_call(dev, b, m, pos, plen, keep, sinks, recent, in_place)
    before = [b.codes[0], b.codes[1]] + ([] if b.scales is None else [b.scales[0], b.scales[1]])
    want = [t.view(torch.uint8).clone().view(t.dtype) if t.dtype == E4M3 else t.clone() for t in before]
    wm, wp = (m.clone(), pos.clone()) if in_place else (torch.full_like(m, 7.0), torch.full_like(pos, -7))
    for s in range(b.S):
        raw = int(b.kv_len[s])
        n = max(0, min(raw, b.cols * b.page, W))
        held = [0 <= int(b.table[s, j // b.page]) < b.n_pages for j in range(n)]
        for h in range(b.Hkv):
            ws = evicted(n, int(plen[s]), held, m[s, h].tolist(), pos[s, h].tolist(), keep, sinks, recent)
            assert src[s, h].tolist() == ws, (s, h)
            w = min(n, keep)
            frm = torch.tensor(ws[:w], dtype=torch.long)
            wm[s, h, :w], wp[s, h, :w] = m[s, h][frm], pos[s, h][frm]
            for j, f in enumerate(ws):
                if f != j and held[j] and held[f]:
                    pj, pf = int(b.table[s, j // b.page]), int(b.table[s, f // b.page])
                    for x, y in zip(want, before):
                        x, y = (t.view(torch.uint8) if t.dtype == E4M3 else t for t in (x, y))
                        x[pj, h, j % b.page] = y[pf, h, f % b.page]
        assert int(kl[s]) == (keep if n > keep else raw)
    assert torch.equal(mo.view(torch.int32), wm.view(torch.int32)) and torch.equal(po, wp)
    for x, y in zip(kv, want):
        bits = torch.uint8 if y.element_size() == 1 else torch.int16 if y.element_size() == 2 else torch.int32
        assert torch.equal(x.view(bits).cpu(), y.view(bits))


@pytest.mark.parametrize("ks,keep,recent,sinks,Hkv,d,page,kvt", EVICT)
def test_evict(gpu_ready, ks, keep, recent, sinks, Hkv, d, page, kvt):
    for kind in ("mixed", "same") if max(ks) < 20000 else ("mixed",):
        for in_place in (False, True):
            say(f"[evict {ks[:4]} {keep} {recent} {sinks} {Hkv} {d} {page} {kvt} {kind} {in_place}]")
            b, W, m, pos, plen = evict_case(ks, keep, Hkv, d, page, kvt, seed=keep, kind=kind, extra=5 if in_place else 0)
            check_evict(gpu_ready, b, W, m, pos, plen, keep, sinks, recent, in_place)


def test_evict_odd(gpu_ready):
    """NaN, negative, infinite and tiny weights; all zero; more protected tokens than places; bad pages; lengths past the table row,
    past W, negative."""
    for kind in ("odd", "zero", "mixed"):
        b, W, m, pos, plen = evict_case([250, 100, 260], 90, 2, 32, 16, "i8", seed=5, kind=kind)
        say(f"[evict odd {kind}]")
        check_evict(gpu_ready, b, W, m, pos, plen, 90, 3, 20, False)
        check_evict(gpu_ready, b, W, m, torch.zeros_like(pos), plen, 90, 3, 20, False)             # everything protected
        check_evict(gpu_ready, b, W, m, pos, plen, 90, 0, 0, True)
    for kind in ("odd", "zero"):                                                                   # the same over several workgroups
        b, W, m, pos, plen = evict_case([17000, 9000, 100], 8300, 1, 16, 256, "i8", seed=6, kind=kind)
        say(f"[evict odd long {kind}]")
        check_evict(gpu_ready, b, W, m, pos, plen, 8300, 3, 20, False)
        check_evict(gpu_ready, b, W, m, torch.zeros_like(pos), plen, 8300, 3, 20, True)
        b.table[0, 40:44], b.table[0, 3] = -1, b.n_pages
        check_evict(gpu_ready, b, W, m, pos, plen, 8300, 0, 0, False)
        check_evict(gpu_ready, b, W, m, pos, plen, 100, 0, 0, False)
    b, W, m, pos, plen = evict_case([250, 100, 260], 90, 2, 32, 16, "i8", seed=5, kind="mixed")
    b.table[0, 2], b.table[0, 12], b.table[2, 0] = -1, b.n_pages, 1 << 30
    check_evict(gpu_ready, b, W, m, pos, plen, 90, 3, 20, False)
    b.kv_len = torch.tensor([100000, -5, 0], dtype=torch.int32)
    check_evict(gpu_ready, b, W, m, pos, plen, 90, 3, 20, False)
    check_evict(gpu_ready, b, 120, m[..., :120].contiguous(), pos[..., :120].contiguous(), plen, 90, 3, 20, True)
    plen[:] = -2147483648
    check_evict(gpu_ready, b, W, m, pos, plen, 90, 3, 20, False)


# ------------------------------------------------------------------------------------------------ all of them, in graphs
def test_graphs_and_streams(gpu_ready):
    """A pass through all of them, eager, on a stream of its own, and in two captured graphs that share their workspaces, replayed
    in turn with eager work between: the same bits every time."""
    dev = gpu_ready
    Hq, Hkv, d, page, D, S, W = 16, 4, 64, 16, 512, 3, 640
    width = (Hq + 2 * Hkv) * d
    g = torch.Generator().manual_seed(4)
    wq = torch.randn((width, D), generator=g) / D ** 0.5
    codes_w, sc_w = torch.empty((width, D), dtype=E4M3, device=dev), torch.empty((blocks(width), blocks(D)), device=dev)
    _lib.quant128(wq.to(dev), codes_w, sc_w, rows=128)
    fr = freqs(d).to(dev)

    class Pass:
        """One pass for ns new tokens of sequences that hold ks with them."""
        def __init__(self, ns, ks, seed, shared):
            gg = torch.Generator().manual_seed(seed)
            b = Paged(ns, ks, Hkv, d, page, "f16", "i8", seed=seed, cols=W // page)
            b.table = torch.arange(S * (W // page), dtype=torch.int32).view(S, -1) % b.n_pages
            b.n_pages = S * (W // page)
            b.table = torch.randperm(b.n_pages, generator=gg).to(torch.int32).view(S, -1)
            x = torch.randn((2, b.n_pages, Hkv, page, d), generator=gg)
            b.set_values(x.half())
            self.kv, self.cu, self.kl, self.tab = b.gpu(dev)
            self.kv0 = [t.clone() for t in self.kv]
            self.ns, self.T = ns, sum(ns)
            self.x = torch.randn((self.T, D), generator=gg).half().to(dev)
            self.xq, self.xs = torch.empty((self.T, D), dtype=E4M3, device=dev), torch.empty((self.T, blocks(D)), device=dev)
            self.qkv = torch.empty((self.T, width), dtype=torch.float16, device=dev)
            self.o, self.lse = torch.empty((self.T, Hq, d), dtype=torch.float16, device=dev), torch.empty((self.T, Hq), device=dev)
            self.mass0 = torch.rand((S, Hkv, W), generator=gg).to(dev)
            self.pos0 = torch.arange(W, dtype=torch.int32, device=dev).expand(S, Hkv, W).contiguous()
            self.mass, self.pos, self.len2 = self.mass0.clone(), self.pos0.clone(), torch.zeros_like(self.kl)
            self.src = torch.zeros((S, Hkv, 100), dtype=torch.int32, device=dev)
            self.ws = shared

        def __call__(self):
            for t, t0 in zip(self.kv, self.kv0):
                t.copy_(t0)
            self.mass.copy_(self.mass0)
            self.pos.copy_(self.pos0)
            _lib.quant128(self.x, self.xq, self.xs)
            _lib.mm_e4m3(self.xq, self.xs, codes_w, sc_w, self.qkv, self.ws)
            q, k, v = self.qkv.unflatten(1, (-1, d)).split([Hq, Hkv, Hkv], dim=1)
            _lib.qk_norm_rope(q, k, None, None, 1e-6, self.cu, self.kl, fr, q, k)
            _lib.kv_write(k, v, self.kv, self.cu, self.kl, self.tab)
            _lib.attn(q, self.kv, self.cu, self.kl, self.tab, max(self.ns), W, self.o, self.ws, lse=self.lse)
            _lib.attn_mass(q, self.kv, self.cu, self.kl, self.tab, max(self.ns), W, self.lse, self.mass, self.pos, self.ws)
            _lib.kv_evict(self.kv, self.kl, self.tab, self.mass, self.pos, 100, self.src, self.ws, sinks=2, recent=20, kv_len_out=self.len2)
            return [t.clone() for t in (self.qkv, self.o, self.lse, self.mass, self.pos, self.src, self.len2) + tuple(self.kv)]

    def same(a, b, what):
        for i, (x, y) in enumerate(zip(a, b)):
            bits = {1: torch.uint8, 2: torch.int16, 4: torch.int32}[x.element_size()]
            assert torch.equal(x.view(bits), y.view(bits)), (what, i)
    need = max([_lib.mm_workspace_size(T, width, D) for T in (3, 150)] + [_lib.kv_evict_workspace_size(S, Hkv, W, 100)]
               + [f for n in (1, 90) for f in (_lib.attn_workspace_size(150, S, Hq, Hkv, d, n, W), _lib.attn_workspace_size(3, S, Hq, Hkv, d, n, W),
                                               _lib.attn_mass_workspace_size(S, Hq, Hkv, d, n, W, W))])
    ws = torch.zeros(need, dtype=torch.uint8, device=dev)
    a, b = Pass([1, 1, 1], [600, 99, 300], 1, ws), Pass([90, 1, 59], [500, 120, 59], 2, ws)
    want = [a(), b()]
    torch.cuda.synchronize()
    assert want[0][6].tolist() == [100, 99, 100] and want[1][6].tolist() == [100, 100, 59]
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        same(a(), want[0], "stream")
    torch.cuda.synchronize()
    graphs, outs = [], []
    for p in (a, b):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            out = p()
        graphs.append(gr)
        outs.append(out)
    for rep in range(4):
        for gr, out, w in zip(graphs, outs, want):
            gr.replay()
            torch.cuda.synchronize()
            same(out, w, f"replay {rep}")
            same(b() if w is want[0] else a(), want[1] if w is want[0] else want[0], "eager between")
            torch.cuda.synchronize()


def test_nothing_to_do(gpu_ready):
    """No tokens, empty sequences, and rows behind the last one."""
    dev = gpu_ready
    e = torch.empty((0, 256), device=dev)
    _lib.quant128(e, e.to(E4M3), torch.empty((0, 2), device=dev))
    out = torch.empty((0, 64), device=dev)
    _lib.mm_e4m3(e.to(E4M3), torch.empty((0, 2), device=dev), torch.zeros((64, 256), device=dev).to(E4M3), torch.zeros((1, 2), device=dev), out)
    b = Paged([0, 0], [30, 0], 2, 64, 16, "f16", "f16", seed=1, pad=4)
    kv, cu, kl, tab = b.gpu(dev)
    q, k = torch.ones((4, 4, 64), dtype=torch.float16, device=dev), torch.ones((4, 2, 64), dtype=torch.float16, device=dev)
    _lib.qk_norm_rope(q, k, None, None, 1e-6, cu, kl, freqs(64).to(dev), q, k)
    m, pos = torch.full((2, 2, 40), 3.0, device=dev), torch.full((2, 2, 40), 5, dtype=torch.int32, device=dev)
    _lib.attn_mass(q, kv, cu, kl, tab, 1, 30, torch.zeros((4, 4), device=dev), m, pos)
    _lib.attn_mass(q[:0], kv, cu, kl, tab, 1, 30, torch.zeros((0, 4), device=dev), m, pos)
    torch.cuda.synchronize()
    assert bool((q == 1).all()) and bool((k == 1).all()) and bool((m == 3).all()) and bool((pos == 5).all())
