"""Paged K/V cache, attention over it and residual norm on the GPU against their 64-bit definitions."""
import math

import pytest
import torch

from activation_sparse_ffn_predictor_amd import _lib
from attn_util import DT, TOP, Paged, assert_near, attention, half_step, quant_rows

pytestmark = pytest.mark.gpu


def say(*a):
    print(*a, flush=True)


def f64(t):
    """CPU float64 values of a device tensor of any type."""
    if t.dtype == torch.float8_e4m3fn:
        t = t.view(torch.uint8).cpu().view(torch.float8_e4m3fn)
    return t.cpu().float().double() if t.dtype != torch.float64 else t.cpu()


# ------------------------------------------------------------------------------------------------ residual norm
NORM = [(1, 8, "f32", "f32", "f32"), (1, 4096, "f16", "f32", "f16"), (3, 4096, "bf16", "bf16", "bf16"),
        (5, 512, "f16", "f16", "f32"), (7, 520, "f32", "f16", "bf16"), (2, 2048, "f32", None, "f16"),
        (3, 2056, "f32", "f32", "f32"), (2, 8192, "bf16", "f32", "f16"), (2, 16384, "f16", "bf16", "f32"),
        (9, 64, "f32", "f32", "i8"), (1, 4096, "f32", "f32", "i8"), (3, 5128, "bf16", "bf16", "i8"),
        (2, 16384, "f32", "f32", "i8"), (33, 72, "f16", "f32", "e4m3"), (2, 1000, "f32", None, "e4m3"),
        (3, 8192, "f16", "f16", "e4m3"), (2, 12288, "bf16", "f32", "e4m3"), (65, 200, "bf16", "f16", "i8")]


def norm_case(T, D, xt, rt, seed):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn((T, D), generator=g) * 3).to(DT[xt])
    r = None if rt is None else torch.randn((T, D), generator=g).to(DT[rt])
    w = 1 + 0.3 * torch.randn(D, generator=g)
    return x, r, w


def norm_ref(x, r, w, eps):
    h = x.float() if r is None else x.float() + r.float()
    hd = h.double()
    y = hd / torch.sqrt(hd.square().mean(-1, keepdim=True) + eps)
    return h, y if w is None else y * w.double()


@pytest.mark.parametrize("T,D,xt,rt,yt", NORM)
def test_norm(gpu_ready, T, D, xt, rt, yt):
    dev, eps = gpu_ready, 1e-5
    x, r, w = norm_case(T, D, xt, rt, T * D)
    h, y = norm_ref(x, r, w, eps)
    say(f"[norm {T} {D} {xt} {rt} {yt}]")
    # rows apart by more than D, guard rows behind
    big = torch.full((T + 1, D + 16), 7.0).to(DT[xt]).to(dev)
    big[:T, :D] = x.to(dev)
    yo = torch.full((T + 1, D + 8), 5.0).to(DT[yt]).to(dev)
    ys = torch.full((T + 1,), -1.0, device=dev)
    ro = None if rt is None else torch.full((T, D), 9.0).to(DT[rt]).to(dev)
    _lib.add_rmsnorm(big[:T, :D], None if r is None else r.to(dev), w.to(dev), eps, yo[:T, :D], res_out=ro,
                     y_scale=ys[:T] if yt in TOP else None)
    torch.cuda.synchronize()
    if ro is not None:
        assert torch.equal(ro.cpu(), h.to(DT[rt]))
    got = f64(yo)
    assert (got[T] == 5.0).all() and (got[:, D:] == 5.0).all() and ys[T].item() == -1.0
    if yt in TOP:
        c, s = quant_rows(y, yt, floor=0.0)
        assert torch.equal(ys[:T].cpu(), s)
        assert torch.equal(got[:T, :D], c)
    else:
        # fp32: sum of D squares, square root, division, two products: (D / 2 + 8) steps of 2^-24; then one rounding,
        # which below the type's smallest normal value is off by half of that value's step: tiny * half_step (fp16:
        # values below 2^-14 lie 2^-24 apart, so up to 2^-25)
        tol = (D / 2 + 8) * 2.0 ** -24 * y.abs() + half_step(yt) * y.abs() * 1.01
        assert_near(yo[:T, :D].float(), y, tol + torch.finfo(DT[yt]).tiny * half_step(yt) * 1.01, "y")


@pytest.mark.parametrize("yt", ["f16", "i8", "e4m3"])
def test_norm_edges(gpu_ready, yt):
    """In-place residual, no weights, zero rows, infinities and NaN, the same bits in every run."""
    dev, T, D = gpu_ready, 6, 640
    x, r, _ = norm_case(T, D, "f32", "f32", 3)
    x[1], r[1] = 0, 0
    x[2, 5] = math.inf
    x[3, 7] = math.nan
    x[4], r[4] = 1e-30, 0
    h, y = norm_ref(x, r, None, 0.0)
    outs = []
    for _ in range(2):
        rg, yo = r.to(dev), torch.zeros((T, D), device=dev).to(DT[yt])
        ys = torch.full((T,), -1.0, device=dev)
        _lib.add_rmsnorm(x.to(dev), rg, None, 0.0, yo, res_out=rg, y_scale=ys if yt in TOP else None)
        torch.cuda.synchronize()
        assert torch.equal(torch.nan_to_num(rg.cpu(), nan=-5.0), torch.nan_to_num(h, nan=-5.0))
        outs.append((f64(yo), ys.cpu()))
    assert torch.equal(torch.nan_to_num(outs[0][0], nan=-5.0), torch.nan_to_num(outs[1][0], nan=-5.0))
    if yt in TOP:
        c, s = quant_rows(y, yt, floor=0.0)
        for row in (0, 4, 5):
            assert torch.equal(outs[0][0][row], c[row]) and outs[0][1][row] == s[row]
        for row in (1, 2, 3):      # 0 / 0, an infinity, a NaN: no scale
            assert (outs[0][0][row] == 0).all() and math.isnan(outs[0][1][row].item())


@pytest.mark.parametrize("xt", ["f32", "bf16"])
@pytest.mark.parametrize("D", [64, 640, 4096, 8192, 16384])
def test_norm_of_any_finite_size(gpu_ready, D, xt):
    """Rows whose squares leave fp32's range at either end, beside ordinary ones."""
    dev = gpu_ready
    size = torch.tensor([1.0, 1e25, 3e36, 1e18, 1e-12, 1e-18, 1e-25, 1e-36], dtype=torch.float64)
    x = (torch.randn((8, D), generator=torch.Generator().manual_seed(D), dtype=torch.float64) * size[:, None]).to(DT[xt])
    w = 1 + 0.3 * torch.randn(D, generator=torch.Generator().manual_seed(1))
    for eps in (0.0, 1e-6, 1e-40):
        _, y = norm_ref(x, None, w, eps)
        for yt in ("f32", "bf16"):
            yo = torch.zeros((8, D), device=dev).to(DT[yt])
            _lib.add_rmsnorm(x.to(dev), None, w.to(dev), eps, yo)
            torch.cuda.synchronize()
            # as above; values below the smallest normal one may be flushed
            tol = (D / 2 + 8) * 2.0 ** -24 * y.abs() + half_step(yt) * y.abs() * 1.01
            assert_near(yo.float(), y, tol + torch.finfo(DT[yt]).tiny, f"y {xt} {yt} {eps}")


def test_norm_of_more_rows_than_a_launch_holds(gpu_ready):
    T, D = (1 << 22) + 5, 4104
    if torch.cuda.mem_get_info(gpu_ready)[0] < T * D * 4:
        pytest.skip("needs 70 GB")
    x = torch.empty((T, D), device=gpu_ready, dtype=torch.float16).fill_(0.25)
    y, ys = torch.empty((T, D), device=gpu_ready, dtype=torch.int8), torch.zeros(T, device=gpu_ready)
    rows = [0, 1, (1 << 21) - 1, 1 << 21, (1 << 22) - 1, 1 << 22, T - 1]
    for r in rows:
        x[r, ::2] = -0.5 * (1 + r % 7)
    _lib.add_rmsnorm(x, None, None, 1e-5, y, y_scale=ys)
    torch.cuda.synchronize()
    for r in rows + [7, T - 2]:
        c, s = quant_rows(norm_ref(x[r:r + 1].cpu(), None, None, 1e-5)[1], "i8", floor=0.0)
        assert torch.equal(f64(y[r:r + 1]), c) and ys[r].item() == s.item(), r
    del x, y
    torch.cuda.empty_cache()


# ------------------------------------------------------------------------------------------------ write and read
CACHES = [("f16", "f16", 128, 8, 16), ("bf16", "bf16", 64, 1, 64), ("f16", "i8", 128, 3, 16), ("bf16", "i8", 16, 2, 32),
          ("f16", "e4m3", 80, 5, 128), ("bf16", "e4m3", 256, 2, 16), ("f16", "f16", 24, 2, 16), ("bf16", "i8", 112, 40, 32),
          ("f16", "e4m3", 32, 1, 1024), ("bf16", "bf16", 200, 2, 16)]
BATCHES = [([1], [1]), ([1] * 8, [5, 16, 17, 1, 64, 33, 100, 31]), ([0, 37, 1, 0, 64, 3], [40, 37, 200, 0, 70, 65]),
           ([300], [333]), ([1, 0] * 70, [3 + i for i in range(140)])]


@pytest.mark.parametrize("qt,kvt,d,Hkv,page", CACHES)
@pytest.mark.parametrize("bi", range(len(BATCHES)))
def test_write_then_read(gpu_ready, qt, kvt, d, Hkv, page, bi):
    dev = gpu_ready
    ns, ks = BATCHES[bi]
    b = Paged(ns, ks, Hkv, d, page, qt, kvt, seed=bi, pad=3)
    g = torch.Generator().manual_seed(7)
    qkv = torch.randn((b.T, 4 * Hkv * d), generator=g)
    qkv[0, 2 * Hkv * d:2 * Hkv * d + d] = 0                       # a row of zeros
    if b.T > 4:
        qkv[1] *= 2.0 ** -12                                      # small rows (subnormal in fp16)
        qkv[2] = torch.round(qkv[2] * 4) / 4                      # many ties and equal values
    qkv = qkv.to(DT[qt])
    k, v = (qkv[:, i * Hkv * d:(i + 1) * Hkv * d].unflatten(1, (Hkv, d)) for i in (2, 3))
    say(f"[write {qt} {kvt} d={d} H={Hkv} page={page} batch {bi}]")
    kv, cu, kl, tab = b.gpu(dev)
    before = [f64(t) for t in kv]
    qg = qkv.to(dev)
    kg, vg = (qg[:, i * Hkv * d:(i + 1) * Hkv * d].unflatten(1, (Hkv, d)) for i in (2, 3))
    _lib.kv_write(kg, vg, kv, cu, kl, tab)
    torch.cuda.synchronize()
    want = [t.clone() for t in before]
    for s in range(b.S):
        for i in range(ns[s]):
            p, t = ks[s] - ns[s] + i, int(b.cu[s]) + i
            pid, slot = int(b.table[s, p // page]), p % page
            for m, x in enumerate((k, v)):
                if kvt in TOP:
                    c, sc = quant_rows(x[t].double(), kvt)
                    want[m][pid, :, slot], want[2 + m][pid, :, slot] = c, sc.double()
                else:
                    want[m][pid, :, slot] = x[t].double()
    for m, t in enumerate(kv):
        assert torch.equal(f64(t), want[m]), f"part {m}"
    # back: the written tokens, rows behind the last sequence untouched
    out = torch.full((2, b.T, Hkv, d), 3.0).to(DT[qt]).to(dev)
    _lib.kv_read(kv, cu, kl, tab, out[0], out[1])
    torch.cuda.synchronize()
    for m in range(2):
        for s in range(b.S):
            for i in range(ns[s]):
                p, t = ks[s] - ns[s] + i, int(b.cu[s]) + i
                val = want[m][int(b.table[s, p // page]), :, p % page]
                if kvt in TOP:
                    val = (val.float() * want[2 + m][int(b.table[s, p // page]), :, p % page].float()[:, None])
                assert torch.equal(out[m, t].cpu(), val.to(DT[qt]))
        assert (out[m, b.N:] == 3.0).all()


@pytest.mark.parametrize("qt", ["f16", "bf16"])
@pytest.mark.parametrize("kvt", ["i8", "e4m3"])
def test_write_rounds_exact_quotients(gpu_ready, qt, kvt):
    """Every mantissa under largest values of many, at sizes from a row's largest value to a 2^-12th of it: quotients
    on the middle of two codes and a few 2^-30ths beside it are among them."""
    dev = gpu_ready
    bits = 7 if qt == "bf16" else 10
    man = 1 + torch.arange(2 ** bits, dtype=torch.float64) / 2 ** bits
    big = man[::1 if qt == "bf16" else 37]
    x = man.view(-1, 128).repeat(len(big) * 13, 1)                # [row, 128]
    per = len(x) // (len(big) * 13)
    e = torch.arange(13).repeat_interleave(per).repeat(len(big))
    b = big.repeat_interleave(13 * per)
    x = x * torch.pow(torch.tensor(2.0, dtype=torch.float64), -e.double())[:, None]
    x = torch.where(x > b[:, None], x / 2, x)
    x[:, ::2] *= -1
    x[:, 5] = b
    for size in ([1.0] if qt == "f16" else [1.0, 2.0 ** 126, 2.0 ** -50]):
        v = (x * size).to(DT[qt]).view(-1, 1, 128)
        assert torch.equal(v.double().view(-1, 128), x * size)
        T, page = len(v), 64
        n = -(-T // page)
        kv = tuple(torch.zeros((n, 1, page, 128), device=dev).to(DT[kvt]) for _ in range(2))
        kv += tuple(torch.zeros((n, 1, page), device=dev) for _ in range(2))
        cu, kl, tab = (torch.tensor(t, dtype=torch.int32, device=dev) for t in ([0, T], [T], [list(range(n))]))
        _lib.kv_write(v.to(dev), v.to(dev), kv, cu, kl, tab)
        torch.cuda.synchronize()
        c, sc = quant_rows(v.double().view(-1, 128), kvt)
        for m in range(2):
            assert torch.equal(f64(kv[m]).view(-1, 128)[:T], c), f"part {m} size {size}"
            assert torch.equal(kv[2 + m].cpu().view(-1)[:T], sc)


@pytest.mark.parametrize("kvt", ["f16", "i8", "e4m3"])
def test_write_nothing_to_bad_places(gpu_ready, kvt):
    """Pages outside the cache, positions outside the table row and before the first token: nothing is written there
    or read from there, and nothing else is touched."""
    dev, page = gpu_ready, 16
    b = Paged([4, 20, 3, 2], [40, 50, 30, 1], 2, 64, page, "f16", kvt, seed=4, cols=3)
    b.table[0, 2] = b.n_pages                       # tokens 36 .. 39 of sequence 0
    b.table[1, 2] = -7                              # 32 .. 47 of sequence 1; 48, 49 lie past the row
    b.table[2, 1] = 2 ** 31 - 1
    kv, cu, kl, tab = b.gpu(dev)
    before = [f64(t) for t in kv]
    x = torch.randn((2, b.T, 2, 64), generator=torch.Generator().manual_seed(1)).half().to(dev)
    _lib.kv_write(x[0], x[1], kv, cu, kl, tab)
    out = torch.full((2, b.T, 2, 64), 3.0).half().to(dev)
    _lib.kv_read(kv, cu, kl, tab, out[0], out[1])
    torch.cuda.synchronize()
    live = torch.zeros(b.T, dtype=torch.bool)
    live[4:6] = True                                # positions 30, 31 of sequence 1
    live[28] = True                                 # the second token of sequence 3 (position 0)
    changed = sum(int((f64(t) != w).flatten(2).any(-1).any(1).sum()) if i < 2 else 0 for i, (t, w) in enumerate(zip(kv, before)))
    assert changed <= 2 * 2                         # two pages, K and V
    assert bool(((out != 3.0).flatten(2).any(-1).all(0).cpu() == live).all())
    if kvt == "f16":
        assert torch.equal(out[:, live.to(dev)], x[:, live.to(dev)])


@pytest.mark.parametrize("qt", ["f16", "bf16"])
@pytest.mark.parametrize("kvt", ["i8", "e4m3"])
def test_write_nonfinite_and_tiny_rows(gpu_ready, qt, kvt):
    dev = gpu_ready
    b = Paged([6], [6], 1, 64, 16, qt, kvt)
    x = torch.randn((6, 1, 64), generator=torch.Generator().manual_seed(2))
    x[1, 0, 3], x[2, 0, 5], x[3, 0, 7] = math.inf, -math.inf, math.nan
    x[4] *= 1e-37 if qt == "bf16" else 1e-7
    x[5] = torch.finfo(DT[qt]).max
    x = x.to(DT[qt])
    kv, cu, kl, tab = b.gpu(dev)
    _lib.kv_write(x.to(dev), x.to(dev), kv, cu, kl, tab)
    out = torch.zeros((2, 6, 1, 64), device=dev, dtype=DT[qt])
    _lib.kv_read(kv, cu, kl, tab, out[0], out[1])
    torch.cuda.synchronize()
    c, s = quant_rows(x.double(), kvt)
    pid = int(b.table[0, 0])
    for m in range(2):
        assert torch.equal(f64(kv[m])[pid, :, :6].transpose(0, 1), c)
        got = kv[2 + m].cpu()[pid, :, :6].transpose(0, 1)
        assert torch.equal(torch.nan_to_num(got, nan=-1.0), torch.nan_to_num(s, nan=-1.0))
        assert out[m, 1:4].isnan().all() and out[m, [0, 5]].isfinite().all()


# ------------------------------------------------------------------------------------------------ attention
def run_attn(b, q, Hq, dev, scale=None, window=0, sinks=0, max_q=None, max_kv=None, poison=None, lse=True):
    kv, cu, kl, tab = b.gpu(dev)
    max_q, max_kv = max_q or max(1, max(b.ns)), max_kv or max(1, max(b.ks))
    out = torch.full((b.T, Hq, b.d), 3.0, device=dev).to(DT[b.qt])
    ls = torch.full((b.T, Hq), 3.0, device=dev) if lse else None
    need = _lib.attn_workspace_size(b.T, b.S, Hq, b.Hkv, b.d, max_q, max_kv, window, sinks)
    ws = torch.full((need + 256,), 255, dtype=torch.uint8, device=dev)          # NaN everywhere
    _lib.attn(q.to(dev), kv, cu, kl, tab, max_q, max_kv, out, ws[:need], scale=scale, window=window, sinks=sinks, lse=ls)
    torch.cuda.synchronize()
    assert (ws[need:] == 255).all()
    return out, ls


def check_attn(b, Hq, dev, scale=None, window=0, sinks=0, q=None, q_scale=1.0, **kw):
    if q is None:
        q = (torch.randn((b.T, Hq, b.d), generator=b.g) * q_scale).to(DT[b.qt])
    out, lse = run_attn(b, q, Hq, dev, scale, window, sinks, **kw)
    o, l, to, tl = attention(b, q, Hq, b.d ** -0.5 if scale is None else scale, window, sinks)
    r = assert_near(out[:b.N], o[:b.N], to[:b.N], "out")
    r2 = assert_near(lse[:b.N], l[:b.N], tl[:b.N], "lse")
    assert (out[b.N:] == 3.0).all() and (lse[b.N:] == 3.0).all()
    return r, r2


TYPES = [("f16", "f16"), ("bf16", "bf16"), ("f16", "i8"), ("bf16", "i8"), ("f16", "e4m3"), ("bf16", "e4m3")]
# (new tokens, cached tokens) of each sequence, K/V heads, query heads, head size, page, window, sinks
ATTN = {
    "one key": ([1], [1], 1, 1, 64, 16, 0, 0),
    "single tokens": ([1, 1, 1, 1], [5, 31, 32, 33], 2, 8, 128, 16, 0, 0),
    "no shared heads": ([1, 1], [64, 129], 3, 3, 128, 32, 0, 0),
    "16 shared": ([1, 1, 1], [257, 1, 700], 2, 32, 64, 64, 0, 0),
    "17 shared": ([1, 1], [100, 40], 1, 17, 128, 16, 0, 0),
    "71 shared": ([1, 1], [130, 40], 1, 71, 64, 16, 0, 0),
    "drafts": ([3, 4, 1, 2], [90, 4, 300, 257], 2, 14, 128, 16, 0, 0),
    "odd head sizes": ([1, 2], [77, 130], 2, 4, 80, 16, 0, 0),
    "small heads": ([1, 5], [20, 300], 2, 6, 16, 16, 0, 0),
    "wide heads": ([1, 3], [200, 99], 2, 4, 256, 16, 0, 0),
    "wide odd heads, chunk": ([40, 9], [200, 99], 2, 4, 208, 16, 0, 0),
    "chunk": ([130], [200], 2, 4, 128, 16, 0, 0),
    "whole prompt": ([257], [257], 1, 8, 64, 64, 0, 0),
    "chunk, no shared heads": ([70, 200], [70, 333], 3, 3, 128, 32, 0, 0),
    "mixed": ([1, 0, 64, 33, 1, 129], [500, 10, 64, 100, 2, 190], 2, 10, 128, 16, 0, 0),
    "mixed small heads": ([1, 50, 3], [70, 90, 300], 4, 12, 48, 128, 0, 0),
    "chunk 112": ([90, 20], [300, 20], 1, 5, 112, 16, 0, 0),
    "window 1": ([1, 1], [100, 3], 2, 4, 64, 16, 1, 0),
    "window": ([1, 2, 1], [500, 300, 20], 2, 8, 128, 16, 70, 0),
    "window sinks": ([1, 2, 4], [500, 300, 20], 2, 8, 128, 16, 70, 5),
    "window many sinks": ([1, 1], [900, 600], 1, 4, 64, 32, 33, 100),
    "sinks meet window": ([1, 3], [130, 129], 1, 4, 64, 16, 64, 66),
    "chunk window": ([150, 80], [400, 80], 2, 4, 128, 16, 50, 0),
    "chunk window sinks": ([150, 200, 1], [600, 200, 333], 2, 4, 128, 16, 50, 20),
    "chunk window sinks 64": ([100], [1000], 1, 16, 64, 64, 129, 65),
    "long, split": ([1, 2], [5000, 37], 1, 8, 128, 64, 0, 0),
    "chunk, split": ([20], [3000], 1, 16, 128, 64, 0, 0),
    "chunk window, split": ([33, 40], [4000, 2500], 1, 8, 64, 16, 1500, 9),
}


@pytest.mark.parametrize("qt,kvt", TYPES)
@pytest.mark.parametrize("name", ATTN)
def test_attention(gpu_ready, name, qt, kvt):
    ns, ks, Hkv, Hq, d, page, window, sinks = ATTN[name]
    say(f"[attn {name} {qt} {kvt}]")
    b = Paged(ns, ks, Hkv, d, page, qt, kvt, seed=len(name), pad=2, v_scale=0.37)
    r = check_attn(b, Hq, gpu_ready, window=window, sinks=sinks)
    say("   of the bounds: out %.2f lse %.2f" % r)


@pytest.mark.parametrize("qt,kvt", TYPES)
@pytest.mark.parametrize("d", [16, 64, 80, 96, 112, 128, 144, 192, 208, 256])
def test_chunks_of_every_padding(gpu_ready, d, qt, kvt):
    """Head sizes at both ends of each padded one; columns past a head hold NaN or another head's values."""
    say(f"[chunk d={d} {qt} {kvt}]")
    b = Paged([70, 3], [150, 90], 2, d, 16, qt, kvt, seed=d, pad=1, v_scale=0.5)
    check_attn(b, 6, gpu_ready, window=100, sinks=3)
    q = (torch.randn((b.T, 6, d), generator=b.g)).to(DT[qt])
    wide = torch.full((b.T, 6 * d + 64), math.nan).to(DT[qt]).to(gpu_ready)
    wide[:, :6 * d] = q.flatten(1).to(gpu_ready)
    kv, cu, kl, tab = b.gpu(gpu_ready)
    out = torch.full((b.T, 6 * d + 64), 3.0).to(DT[qt]).to(gpu_ready)
    need = _lib.attn_workspace_size(b.T, b.S, 6, 2, d, 70, 150)
    ws = torch.full((need + 256,), 255, dtype=torch.uint8, device=gpu_ready)
    _lib.attn(wide[:, :6 * d].unflatten(1, (6, d)), kv, cu, kl, tab, 70, 150, out[:, :6 * d].unflatten(1, (6, d)), ws)
    torch.cuda.synchronize()
    o, l, to, tl = attention(b, q, 6, d ** -0.5)
    assert_near(out[:b.N, :6 * d].unflatten(1, (6, d)), o[:b.N], to[:b.N], "out")
    assert (out[:, 6 * d:] == 3.0).all() and (out[b.N:] == 3.0).all()


@pytest.mark.parametrize("qt,kvt", TYPES)
def test_attention_sizes_of_values(gpu_ready, qt, kvt):
    """Values and queries far from 1: small ones keep their relative precision, one row is far larger than its
    neighbours, another holds only zeros."""
    for v_scale, q_scale in ((2.0 ** -10, 1.0), (1000.0, 1.0), (1.0, 30.0), (1.0, 2.0 ** -12)):
        for ns, ks in (([1, 1], [90, 300]), ([50, 1], [90, 300])):
            b = Paged(ns, ks, 2, 128, 16, qt, kvt, seed=5, v_scale=v_scale)
            x = torch.randn((2, b.n_pages, 2, 16, 128), generator=b.g)
            x[1] *= v_scale
            x[1, :, :, 3] *= 60.0
            x[1, :, :, 5] = 0
            x[0, :, :, 7] = 0
            b.set_values(x.to(DT[qt]))
            check_attn(b, 8, gpu_ready, q_scale=q_scale)


@pytest.mark.parametrize("qt", ["f16", "bf16"])
@pytest.mark.parametrize("ns,ks,window,sinks", [([1], [40], 0, 0), ([4, 2], [40, 33], 0, 0), ([2, 1], [300, 100], 40, 3),
                                                ([100], [180], 0, 0), ([150, 1], [300, 90], 40, 3)])
def test_nothing_comes_from_masked_places(gpu_ready, qt, ns, ks, window, sinks):
    """Infinities and NaN behind a sequence's end, in later tokens and before the window change nothing; where a row
    sees one, that row alone shows it."""
    dev = gpu_ready
    b = Paged(ns, ks, 2, 64, 16, qt, qt, seed=11)
    x = torch.randn((2, b.n_pages, 2, 16, 64), generator=b.g).to(DT[qt])
    used = torch.zeros((b.n_pages, 16), dtype=torch.bool)
    for s, k in enumerate(ks):
        for p in range(k):
            used[int(b.table[s, p // 16]), p % 16] = True
    x.transpose(2, 3)[:, ~used] = math.nan                       # slots that hold no token
    vals = [math.inf, -math.inf, math.nan]
    for i, p in enumerate([ks[0] - 1, ks[0] - ns[0], 7, ks[0] // 2]):
        x[1, int(b.table[0, p // 16]), i % 2, p % 16, 10 * i:10 * i + 3] = torch.tensor(vals).to(DT[qt])
    b.set_values(x)
    check_attn(b, 4, dev, window=window, sinks=sinks)
    x[0, int(b.table[0, (ks[0] - 1) // 16]), :, (ks[0] - 1) % 16, 3] = math.nan      # a key: its viewers' rows are NaN
    b.set_values(x)
    check_attn(b, 4, dev, window=window, sinks=sinks)


@pytest.mark.parametrize("kvt", ["i8", "e4m3"])
@pytest.mark.parametrize("n", [1, 70])
def test_rows_without_a_scale(gpu_ready, kvt, n):
    """8-bit rows whose tokens held an infinity: NaN for the rows that see them, nothing for the others."""
    b = Paged([n], [150], 2, 64, 16, "f16", kvt, seed=3)
    x = torch.randn((2, b.n_pages, 2, 16, 64), generator=b.g).half()
    for p in (148, 149):
        x[1, int(b.table[0, p // 16]), 0, p % 16, 1] = math.inf
    b.set_values(x)
    q = torch.randn((n, 4, 64), generator=b.g).half()
    out, lse = run_attn(b, q, 4, gpu_ready)
    bad = torch.zeros((n, 4), dtype=torch.bool)
    bad[max(0, n - 2):, :2] = True
    assert torch.equal(out.isnan().all(-1).cpu(), bad) and torch.equal(out.isnan().any(-1).cpu(), bad)
    o, l, to, tl = attention(b, q, 4, 64 ** -0.5)
    ok = ~bad
    assert_near(out[ok.to(out.device)], o[ok], to[ok])
    assert_near(lse[ok.to(out.device)], l[ok], tl[ok])


@pytest.mark.parametrize("qt,kvt", [("f16", "f16"), ("bf16", "i8")])
def test_bad_pages_and_empty_rows(gpu_ready, qt, kvt):
    """Bad page ids hold no tokens; rows before a sequence's first token, and rows whose window holds nothing, are 0
    with the sum's logarithm -infinity."""
    for n in (2, 90):
        b = Paged([n, n, n, n], [200, 150, n - 1, 0], 2, 64, 16, qt, kvt, seed=n, pad=1)
        b.table[0, 1], b.table[0, 3] = -1, b.n_pages
        b.table[0, 12] = 2 ** 31 - 1                 # the newest tokens' own page: with a window of 3 nothing is left
        b.table[1, :] = -(2 ** 31)
        check_attn(b, 4, gpu_ready)
        check_attn(b, 4, gpu_ready, window=3)
        out, lse = run_attn(b, torch.ones((b.T, 4, 64)).to(DT[qt]), 4, gpu_ready, window=3)
        assert (out[n:2 * n] == 0).all() and (lse[n:2 * n] == -math.inf).all()      # no page at all
        assert (out[2 * n] == 0).all() and (lse[2 * n] == -math.inf).all()          # position -1
        assert (out[3 * n:4 * n] == 0).all()


def test_lengths_past_the_table(gpu_ready):
    """kv_len beyond what a table row holds counts as what it holds; cu past T as T; max_q bounds the tokens."""
    b = Paged([1, 1], [48, 40], 1, 64, 16, "f16", "f16", cols=3)
    b.kv_len = torch.tensor([2 ** 31 - 1, 40], dtype=torch.int32)
    check_attn(b, 4, gpu_ready)
    b = Paged([40, 3], [48, 40], 1, 64, 16, "f16", "f16")
    q = torch.randn((43, 4, 64), generator=b.g).half()
    out, lse = run_attn(b, q, 4, gpu_ready, max_q=30)
    o, l, to, tl = attention(b, q, 4, 0.125)
    keep = [i for i in range(43) if i < 30 or i >= 40]
    assert_near(out[keep], o[keep], to[keep])
    assert (out[30:40] == 3.0).all() and (lse[30:40] == 3.0).all()
    b.cu = torch.tensor([0, 40, 1000], dtype=torch.int32)
    b.ns = [40, 3]
    out, lse = run_attn(b, q, 4, gpu_ready)
    assert_near(out[:40], o[:40], to[:40])


def test_split_hint_changes_only_the_split(gpu_ready):
    """max_kv decides over the number of parts: results agree within their bounds, and repeat bit for bit."""
    for ns in ([1, 2], [40, 3]):
        b = Paged(ns, [3000, 700], 1, 128, 16, "f16", "f16", seed=9)
        q = torch.randn((b.T, 8, 128), generator=b.g).half()
        o, l, to, tl = attention(b, q, 8, 128 ** -0.5)
        for max_kv in (1, 700, 3000, 10 ** 6):
            first = run_attn(b, q, 8, gpu_ready, max_kv=max_kv)
            again = run_attn(b, q, 8, gpu_ready, max_kv=max_kv)
            assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
            assert_near(first[0], o, to)
            assert_near(first[1], l, tl)
        no_lse = run_attn(b, q, 8, gpu_ready, lse=False)
        assert torch.equal(no_lse[0], run_attn(b, q, 8, gpu_ready)[0])


SPREAD = {
    "single wide": ([1, 1], [2500, 700], 1, 4, 256, 16, 0, 0),
    "drafts 48": ([3, 2], [3000, 900], 2, 8, 48, 32, 0, 0),
    "drafts 208, window": ([2, 1], [5000, 4000], 1, 3, 208, 16, 3000, 5),
    "chunk 80": ([50], [4000], 1, 4, 80, 64, 0, 0),
    "chunk wide": ([20], [2500], 1, 4, 208, 16, 0, 0),
    "chunk wide, window": ([33, 7], [3000, 2200], 1, 4, 256, 16, 1500, 9),
}


@pytest.mark.parametrize("qt,kvt", TYPES)
@pytest.mark.parametrize("name", SPREAD)
def test_keys_spread_over_workgroups(gpu_ready, name, qt, kvt):
    """Keys in several parts, then with pages missing from whole parts, then with infinities and NaN where no row
    looks (16-bit caches: and where one does)."""
    ns, ks, Hkv, Hq, d, page, window, sinks = SPREAD[name]
    assert _lib.attn_workspace_size(sum(ns), len(ns), Hq, Hkv, d, max(ns), max(ks), window, sinks) > 0
    say(f"[spread {name} {qt} {kvt}]")
    b = Paged(ns, ks, Hkv, d, page, qt, kvt, seed=len(name), pad=1)
    check_attn(b, Hq, gpu_ready, window=window, sinks=sinks)
    table = b.table.clone()
    b.table[0, 600 // page:(ks[0] - 300) // page] = -1
    check_attn(b, Hq, gpu_ready, window=window, sinks=sinks)
    b.table = table
    x = torch.randn((2, b.n_pages, Hkv, page, d), generator=b.g).to(DT[qt])
    used = torch.zeros((b.n_pages, page), dtype=torch.bool)
    for s, k in enumerate(ks):
        for p in range(k):
            used[int(table[s, p // page]), p % page] = True
    x.transpose(2, 3)[:, ~used] = math.nan
    if kvt == qt:
        for i, p in enumerate([ks[0] - 1, 600, ks[0] - 700]):
            x[1, int(table[0, p // page]), 0, p % page, 10 * i] = (math.inf, -math.inf, math.nan)[i]
    b.set_values(x)
    check_attn(b, Hq, gpu_ready, window=window, sinks=sinks)


def test_strided_queries_and_outputs(gpu_ready):
    dev = gpu_ready
    for n in (1, 60):
        b = Paged([n, n], [100, 130], 2, 64, 16, "bf16", "bf16", seed=2)
        kv, cu, kl, tab = b.gpu(dev)
        wide = torch.randn((b.T, 6 * 64 + 8), generator=b.g).bfloat16()
        q = wide[:, 8:8 + 4 * 64].unflatten(1, (4, 64))
        wg = wide.to(dev)
        og = torch.full((b.T, 10, 64), 3.0, device=dev, dtype=torch.bfloat16)
        tabs = torch.full((b.S, b.cols + 5), -1, dtype=torch.int32, device=dev)
        tabs[:, :b.cols] = tab
        _lib.attn(wg[:, 8:8 + 4 * 64].unflatten(1, (4, 64)), kv, cu, kl, tabs[:, :b.cols], n, 130, og[:, 2:6],
                  torch.empty(1 << 24, dtype=torch.uint8, device=dev), scale=0.2)
        torch.cuda.synchronize()
        o, l, to, tl = attention(b, q, 4, 0.2)
        assert_near(og[:, 2:6], o, to)
        assert (og[:, :2] == 3.0).all() and (og[:, 6:] == 3.0).all()


def test_far_pages(gpu_ready):
    """Pages whose byte offsets pass 32 bits."""
    dev, d, page, H = gpu_ready, 128, 64, 8
    n_pages = 40000                                  # 40000 * 8 * 64 * 256 bytes: 5.2 GB each of K and V
    K = torch.empty((n_pages, H, page, d), dtype=torch.float16, device=dev)
    V = torch.empty_like(K)
    for n in (1, 80):
        b = Paged([n, n], [200, 150], H, d, page, "f16", "f16", seed=n)
        far = torch.arange(b.n_pages) * 1000 + n_pages - 1000 * b.n_pages
        kv, cu, kl, tab = b.gpu(dev)
        K[far.to(dev)], V[far.to(dev)] = kv[0], kv[1]
        ftab = torch.where(tab >= 0, far.to(dev).int()[tab.clamp(min=0).long()], tab)
        q = torch.randn((b.T, 16, d), generator=b.g).half()
        out = torch.zeros((b.T, 16, d), dtype=torch.float16, device=dev)
        ws = torch.empty(_lib.attn_workspace_size(b.T, 2, 16, H, d, n, 200), dtype=torch.uint8, device=dev)
        _lib.attn(q.to(dev), (K, V), cu, kl, ftab, n, 200, out, ws)
        back = torch.zeros((2, b.T, H, d), dtype=torch.float16, device=dev)
        _lib.kv_read((K, V), cu, kl, ftab, back[0], back[1])
        _lib.kv_write(back[0], back[1], (K, V), cu, kl, ftab)
        torch.cuda.synchronize()
        o, l, to, tl = attention(b, q, 16, d ** -0.5)
        assert_near(out, o, to)
        assert torch.equal(K[far.to(dev)], kv[0]) and torch.equal(V[far.to(dev)], kv[1])
        t = 0
        for s in range(2):
            r, _ = b.rows(0, s, b.ks[s])
            assert torch.equal(back[0, t:t + n].cpu().double(), r[:, -n:].transpose(0, 1))
            t += n


# ------------------------------------------------------------------------------------------------ as they are used
@pytest.mark.parametrize("kvt", ["f16", "i8"])
def test_chunks_equal_single_tokens(gpu_ready, kvt):
    """A prompt entered in one chunk, in uneven chunks and token by token: the same cache bit for bit, outputs within
    twice the bound of one."""
    dev, Hq, Hkv, d, page, n = gpu_ready, 8, 2, 64, 16, 75
    g = torch.Generator().manual_seed(1)
    x = torch.randn((n, (Hq + 2 * Hkv) * d), generator=g).half()
    res = []
    for cuts in ([n], [40, 1, 34], [1] * n):
        b = Paged([n], [n], Hkv, d, page, "f16", kvt)
        kv, _, _, tab = b.gpu(dev)
        for t in kv:
            t.view(torch.uint8).zero_()
        xg, out, done = x.to(dev), torch.zeros((n, Hq, d), dtype=torch.float16, device=dev), 0
        for m in cuts:
            cu = torch.tensor([0, m], dtype=torch.int32, device=dev)
            kl = torch.tensor([done + m], dtype=torch.int32, device=dev)
            part = xg[done:done + m].unflatten(1, (Hq + 2 * Hkv, d))
            _lib.kv_write(part[:, Hq:Hq + Hkv], part[:, Hq + Hkv:], kv, cu, kl, tab)
            ws = torch.empty(_lib.attn_workspace_size(m, 1, Hq, Hkv, d, m, done + m), dtype=torch.uint8, device=dev)
            _lib.attn(part[:, :Hq], kv, cu, kl, tab, m, done + m, out[done:done + m], ws)
            done += m
        torch.cuda.synchronize()
        b.codes = torch.stack([t.view(torch.uint8).cpu().view(t.dtype) for t in kv[:2]])
        b.val = b.codes.float().double()
        if kvt != "f16":
            b.scales = torch.stack([t.cpu() for t in kv[2:]])
            b.val = b.val * b.scales.double()[..., None]
        o, _, to, _ = attention(b, x[:, :Hq * d].unflatten(1, (Hq, d)), Hq, d ** -0.5)
        assert_near(out, o, to)
        res.append((b.codes, b.scales, out))
    for codes, scales, out in res[1:]:
        assert torch.equal(codes.view(torch.uint8), res[0][0].view(torch.uint8))
        assert scales is None or torch.equal(scales, res[0][1])
        assert ((out - res[0][2]).abs().cpu().double() <= 2 * to).all()


def test_graph_replays_and_other_streams(gpu_ready):
    """Write and attention captured into one graph, replayed while lengths and inputs change in place, with eager work
    between; and the same calls on two streams at once, each with its own workspace."""
    dev, Hq, Hkv, d, page, S = gpu_ready, 8, 2, 64, 16, 3
    b = Paged([1] * S, [900, 130, 40], Hkv, d, page, "f16", "i8", seed=6)
    kv, cu, kl, tab = b.gpu(dev)
    need = _lib.attn_workspace_size(S, S, Hq, Hkv, d, 1, 1024)
    assert need > 0                                  # the join runs too

    class Job:
        def __init__(self):
            self.x = torch.randn((S, Hq + 2 * Hkv, d), device=dev).half()
            self.kv = tuple(t.clone() for t in kv)
            self.kl, self.out = kl.clone(), torch.zeros((S, Hq, d), dtype=torch.float16, device=dev)
            self.ws = torch.empty(need, dtype=torch.uint8, device=dev)

        def step(self):
            _lib.kv_write(self.x[:, Hq:Hq + Hkv], self.x[:, Hq + Hkv:], self.kv, cu, self.kl, tab)
            _lib.attn(self.x[:, :Hq], self.kv, cu, self.kl, tab, 1, 1024, self.out, self.ws)

    j = Job()
    j.step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        j.step()
    for rep in range(3):
        j.x.copy_(torch.randn((S, Hq + 2 * Hkv, d), device=dev).half())
        j.kl.copy_(torch.tensor([900 - 5 * rep, 130 + rep, 3 + rep], dtype=torch.int32))
        j.out.fill_(float("nan"))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        got = j.out.clone()
        j.out.fill_(float("nan"))
        j.step()
        torch.cuda.synchronize()
        assert torch.equal(got, j.out)
    jobs, streams = [Job(), Job()], [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(20):
        for job, st in zip(jobs, streams):
            with torch.cuda.stream(st):
                job.step()
    torch.cuda.synchronize()
    for job in jobs:
        got = job.out.clone()
        job.step()
        torch.cuda.synchronize()
        assert torch.equal(got, job.out)
    a = jobs[0]
    got = a.out.clone()
    a.out.zero_()
    torch.cuda.synchronize()
    _lib.attn(a.x[:, :Hq], a.kv, cu, a.kl, tab, 1, 1024, a.out, a.ws, stream=streams[1])
    torch.cuda.synchronize()
    assert torch.equal(got, a.out)


@pytest.mark.parametrize("qt,kvt", [("f16", "f16"), ("bf16", "bf16"), ("f16", "i8"), ("bf16", "e4m3")])
@pytest.mark.parametrize("scale", [0.0, -0.125, 1e-42, 3.0])
def test_any_finite_scale(gpu_ready, qt, kvt, scale):
    for ns, ks in (([1, 2], [90, 40]), ([70, 3], [90, 40])):
        b = Paged(ns, ks, 2, 64, 16, qt, kvt, seed=8)
        check_attn(b, 4, gpu_ready, scale=scale, q_scale=0.2)


@pytest.mark.parametrize("kvt", ["bf16", "i8"])
def test_queries_with_infinities_touch_only_their_rows(gpu_ready, kvt):
    for n in (2, 80):
        b = Paged([n], [150], 1, 64, 16, "bf16", kvt, seed=4)
        q = (torch.randn((n, 4, 64), generator=b.g) * 1000).bfloat16()
        clean = q.clone()
        q[0, 1, 3], q[n - 1, 2, 7] = math.inf, math.nan
        out, lse = run_attn(b, q, 4, gpu_ready)
        o, l, to, tl = attention(b, clean, 4, 0.125)
        ok = torch.ones((n, 4), dtype=torch.bool)
        ok[0, 1] = ok[n - 1, 2] = False
        assert_near(out[ok.to(out.device)], o[ok], to[ok])
        assert_near(lse[ok.to(out.device)], l[ok], tl[ok])
        assert out[~ok.to(out.device)].isnan().all()


def test_shared_pages(gpu_ready):
    """Sequences whose tables share the pages of a common beginning."""
    for n in (1, 60):
        b = Paged([n, n, n], [160, 200, 170], 2, 64, 16, "f16", "f16", seed=n)
        b.table[1, :4] = b.table[0, :4]
        b.table[2, :4] = b.table[0, :4]
        check_attn(b, 8, gpu_ready)


def test_many_sequences(gpu_ready):
    """More sequences than any lookup step takes at once: single tokens, and a few longer ones among them."""
    dev = gpu_ready
    for S, long in ((5000, 0), (700, 9)):
        ns = [1] * S
        ks = [1 + (7 * i) % 40 for i in range(S)]
        for i in range(long):
            ns[71 * i] = ks[71 * i] = 20 + i
        b = Paged(ns, ks, 1, 16, 16, "f16", "f16", seed=3)
        q = torch.randn((b.T, 4, 16), generator=b.g).half()
        kv, cu, kl, tab = b.gpu(dev)
        back = torch.zeros((2, b.T, 1, 16), dtype=torch.float16, device=dev)
        _lib.kv_read(kv, cu, kl, tab, back[0], back[1])
        _lib.kv_write(back[0], back[1], kv, cu, kl, tab)
        out, lse = run_attn(b, q, 4, dev)
        assert torch.equal(kv[0].cpu(), b.codes[0])
        pick = sorted({0, 1, S // 2, S - 2, S - 1, *(71 * i for i in range(long))})
        for s in pick:
            one = Paged([ns[s]], [ks[s]], 1, 16, 16, "f16", "f16")
            one.table, one.n_pages, one.cols, one.val = b.table[s:s + 1], b.n_pages, b.cols, b.val
            t = int(b.cu[s])
            o, l, to, tl = attention(one, q[t:t + ns[s]], 4, 0.25)
            assert_near(out[t:t + ns[s]], o, to, f"sequence {s}")
            assert torch.equal(back[0, t:t + ns[s]].cpu().double(), one.rows(0, 0, ks[s])[0][:, -ns[s]:].transpose(0, 1))


def test_graphs_of_chunks_share_a_workspace(gpu_ready):
    """Two graphs (a chunk with split keys, single tokens) that use one workspace in turn, with a norm and a read among
    their nodes, replayed alternately with eager work between: each replay gives the eager bits."""
    dev, Hq, Hkv, d = gpu_ready, 16, 2, 64
    b = Paged([40, 1], [2000, 900], Hkv, d, 16, "bf16", "bf16", seed=12)
    kv, cu, kl, tab = b.gpu(dev)
    sizes = [_lib.attn_workspace_size(41, 2, Hq, Hkv, d, 40, 2000), _lib.attn_workspace_size(2, 2, Hq, Hkv, d, 1, 2000)]
    assert min(sizes) > 0
    ws = torch.empty(max(sizes), dtype=torch.uint8, device=dev)
    x = torch.randn((41, Hq * d), device=dev)
    w = torch.ones(Hq * d, device=dev)

    class Job:
        def __init__(self, T, cu, max_q):
            self.cu, self.max_q, self.x = cu, max_q, x[:T].clone()
            self.xn = torch.zeros((T, Hq * d), dtype=torch.bfloat16, device=dev)
            self.out = torch.zeros((T, Hq, d), dtype=torch.bfloat16, device=dev)
            self.back = torch.zeros((2, T, Hkv, d), dtype=torch.bfloat16, device=dev)

        def step(self):
            _lib.add_rmsnorm(self.x, None, w, 1e-5, self.xn)
            _lib.attn(self.xn.view(-1, Hq, d), kv, self.cu, kl, tab, self.max_q, 2000, self.out, ws)
            _lib.kv_read(kv, self.cu, kl, tab, self.back[0], self.back[1])

    jobs = [Job(41, cu, 40), Job(2, torch.tensor([0, 1, 2], dtype=torch.int32, device=dev), 1)]
    graphs = []
    for j in jobs:
        j.step()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            j.step()
        graphs.append(g)
    for rep in range(3):
        for j, g in zip(jobs, graphs):
            j.x.normal_()
            j.out.fill_(float("nan"))
            j.back.zero_()
            g.replay()
            torch.cuda.synchronize()
            got = [t.clone() for t in (j.xn, j.out, j.back)]
            j.out.fill_(float("nan"))
            j.step()
            torch.cuda.synchronize()
            assert all(torch.equal(a, c) for a, c in zip(got, (j.xn, j.out, j.back))), rep


def test_no_tokens(gpu_ready):
    dev = gpu_ready
    b = Paged([0, 0], [5, 0], 1, 64, 16, "f16", "f16")
    kv, cu, kl, tab = b.gpu(dev)
    e = torch.zeros((0, 1, 64), dtype=torch.float16, device=dev)
    _lib.kv_write(e, e, kv, cu, kl, tab)
    _lib.kv_read(kv, cu, kl, tab, e, e)
    q = torch.zeros((0, 4, 64), dtype=torch.float16, device=dev)
    _lib.attn(q, kv, cu, kl, tab, 1, 5, q, None)
    x = torch.zeros((0, 64), device=dev)
    _lib.add_rmsnorm(x, x, None, 1e-5, x)
    torch.cuda.synchronize()
