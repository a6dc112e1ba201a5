"""The resident stack with 8-bit projections, norms of heads, rotary positions and a bounded cache: what a layer's calls hand to
each other, checked from the buffers they worked on; evictions on the way; eager steps and replays give the same bits."""
import dataclasses

import pytest
import torch

import synthgen as sg
from activation_sparse_ffn_predictor_amd import SffnError, _lib
from activation_sparse_ffn_predictor_amd.stack import AttnConfig, SparseFFNStack
from attn_util import TOP, Paged, assert_near, attention
from layer_def import evicted, head_rows, mass, product, quant_blocks

pytestmark = pytest.mark.gpu
BASE = AttnConfig(8, 2, 64, "i8", page=16, max_len=60, sinks=2, qk_norm=True, rope_base=10000.0, rope_dim=32, rope_interleaved=True,
                  weights="e4m3", keep=40, recent=8)
CASES = [BASE, dataclasses.replace(BASE, kv_type="f16", rope_dim=0, rope_interleaved=False, weights="f16", sinks=0, recent=0),
         dataclasses.replace(BASE, kv_type="e4m3", qk_norm=False, keep=0, recent=0, window=20, sinks=3)]


def toy(dev, c, max_batch=12, layers=2):
    return SparseFFNStack(sg.custom(sg.workload("toy_relu"), L=layers), dev, max_batch=max_batch, attn=c)


def f64(t):
    return (t.view(torch.uint8).cpu().view(t.dtype) if t.dtype == torch.float8_e4m3fn else t.cpu()).float().double()


def cached(st, i, ns, lens, rows):
    """The sequences `rows` of layer i's cache."""
    c, t = st.attn, st.layers[i]
    b = Paged(ns, lens, c.n_kv_heads, c.head_dim, c.page, "f16", c.kv_type, cols=st.table.shape[1])
    b.table, b.n_pages = st.table.cpu()[rows], t["kv"][0].shape[0]
    b.val = torch.stack([f64(x) for x in t["kv"][:2]])
    if c.kv_type in TOP:
        b.val = b.val * torch.stack([x.cpu() for x in t["kv"][2:]]).double()[..., None]
    return b


def project(st, x, w):
    """x W^T through calls of their own."""
    if st.attn.weights == "f16":
        return torch.mm(x, w.t())
    out = torch.zeros((x.shape[0], w[0].shape[0]), dtype=torch.float16, device=x.device)
    q, s = st._quantised(x.contiguous(), 1)
    wq, ws = quant_blocks(x.cpu(), 1)
    assert torch.equal(f64(q), wq) and torch.equal(s.cpu(), ws)
    _lib.mm_e4m3(q, s, *w, out, st.ws_mm)
    torch.cuda.synchronize()
    assert_near(out, *product(wq, ws, f64(w[0]), w[1].cpu(), "f16"), "projection")
    return out


@pytest.mark.parametrize("c", CASES)
def test_layers(gpu_ready, c):
    dev = gpu_ready
    st = toy(dev, c)
    g = torch.Generator().manual_seed(1)

    def run(T, x, cu, first, ns):
        """One pass by hand over sequences first, first + 1, ... with ns new tokens each."""
        rows = slice(first, first + len(ns))
        ids = list(range(first, first + len(ns)))
        lens, seqs = [st.lens[r] for r in ids], st.seq_len[rows].tolist()
        for i, t in enumerate(st.layers):
            old = t["mass"][rows].clone() if c.keep else None
            st.attn_layer(i, x, T, cu, st.kv_len[rows], st.table[rows], max(ns), st.seq_len[rows], rows)
            torch.cuda.synchronize()
            before = project(st, st.xn[:T], t["W_qkv"]).cpu().unflatten(1, (-1, c.head_dim))
            q0, k0, v0 = before.split([c.n_heads, c.n_kv_heads, c.n_kv_heads], dim=1)
            q, k, v = st.qkv[:T].cpu().unflatten(1, (-1, c.head_dim)).split([c.n_heads, c.n_kv_heads, c.n_kv_heads], dim=1)
            pos = torch.cat([torch.arange(p - n, p) for n, p in zip(ns, seqs)])
            fr = None if st.freq is None else st.freq.cpu()
            for a, b0, w in ((q, q0, "w_q"), (k, k0, "w_k")):
                wt = t[w].cpu() if c.qk_norm else None
                assert_near(a, *head_rows(b0, wt, c.eps if c.qk_norm else None, pos, fr, c.rope_interleaved, "f16"), w)
            assert torch.equal(v, v0)
            b = cached(st, i, ns, lens, ids)
            o, lse, to, tl = attention(b, q, c.n_heads, c.head_dim ** -0.5, c.window, c.sinks)
            assert_near(st.o[:T], o, to, "attention")
            if c.keep:
                assert_near(st.lse[:T], lse, tl, "log-sum-exp")
                want, tol = mass(b, q, st.lse[:T].cpu(), c.n_heads, c.head_dim ** -0.5, old.cpu())
                held = ~torch.isnan(want)
                assert_near(t["mass"][rows].cpu()[held], want[held], tol[held], "mass")
                for s, (n, ln, p) in enumerate(zip(ns, lens, seqs)):
                    assert t["pos"][first + s, 0, ln - n:ln].tolist() == list(range(p - n, p))
            assert torch.equal(st.ao[:T], project(st, st.o[:T].flatten(1), t["W_o"]))
            st.layer_call(i, st.xf[:T], False, st.y[i, :T])
            x = st.y[i, :T].clone()

    def grow(rows, n):
        st.kv_len[rows] += n
        st.seq_len[rows] += n
        st.lens[rows] = [m + n for m in st.lens[rows]]
    for s, T in ((0, 12), (1, 7), (0, 12), (1, 1)):
        grow(slice(s, s + 1), T)
        run(T, torch.randn((T, 512), generator=g).to(dev), torch.tensor([0, T], dtype=torch.int32, device=dev), s, [T])
    for _ in range(2):
        grow(slice(0, 2), 1)
        run(2, torch.randn((2, 512), generator=g).to(dev), st.cu_step[:3], 0, [1, 1])
    if not c.keep:
        return
    # the sequence runs full; the next token cuts it down first
    while st.lens[0] + 12 <= c.max_len:
        st.prompt(0, torch.randn((12, 512), generator=g).to(dev))
    while st.lens[0] < c.max_len:
        st.x_in[:1] = torch.randn((1, 512), generator=g).to(dev)
        st.step(1)
    torch.cuda.synchronize()
    for turn in range(2):
        snap = [(t["mass"][0].cpu(), t["pos"][0].cpu(), cached(st, i, [0], [st.lens[0]], [0])) for i, t in enumerate(st.layers)]
        n, total, other = st.lens[0], int(st.seq_len[0]), st.lens[1]
        if turn == 0:
            st.x_in[:1] = torch.randn((1, 512), generator=g).to(dev)
            st.evict(0)
        else:
            for _ in range(3):
                st.prompt(0, torch.randn((7, 512), generator=g).to(dev))          # past max_len on the way
            assert c.keep < st.lens[0] <= c.max_len
            assert int(st.seq_len[0]) == total + 21 and st.lens[1] == other
            break
        torch.cuda.synchronize()
        assert st.lens[0] == c.keep == int(st.kv_len[0]) and int(st.seq_len[0]) == total and st.lens[1] == other
        for i, t in enumerate(st.layers):
            m, p, b = snap[i]
            now = cached(st, i, [0], [c.keep], [0])
            (was_k, _), (was_v, _) = b.rows(0, 0, n), b.rows(1, 0, n)
            (k, _), (v, _) = now.rows(0, 0, c.keep), now.rows(1, 0, c.keep)
            for h in range(c.n_kv_heads):
                src = torch.tensor(evicted(n, total, [True] * n, m[h].tolist(), p[h].tolist(), c.keep, c.sinks, c.recent))
                assert torch.equal(t["mass"][0, h, :c.keep].cpu(), m[h][src]) and torch.equal(t["pos"][0, h, :c.keep].cpu(), p[h][src])
                assert torch.equal(k[h], was_k[h][src]) and torch.equal(v[h], was_v[h][src])
                got = set(t["pos"][0, h, :c.keep].tolist())
                assert set(range(c.sinks)) <= got and set(range(total - c.recent, total)) <= got
        st.step(1)
        torch.cuda.synchronize()
        assert st.lens[0] == c.keep + 1 and st.out[:1].isfinite().all()


@pytest.mark.parametrize("c", CASES[:2])
def test_steps_and_replays_agree(gpu_ready, c):
    """Eager steps in one stack, graph replays in another, with evictions on the way and eager work between: the same bits."""
    dev, B = gpu_ready, 3
    a, b = toy(dev, c), toy(dev, c)
    g = torch.Generator().manual_seed(2)
    for s, n in ((0, 12), (1, 5), (2, 9), (0, 12), (0, 12), (0, 12)):
        x = torch.randn((n, 512), generator=g).to(dev)
        for st in (a, b):
            st.prompt(s, x)
    b.x_in.normal_()
    gr = b.capture(B)
    assert b.lens == a.lens and torch.equal(a.kv_len, b.kv_len) and torch.equal(a.seq_len, b.seq_len)
    for rep in range(60):
        x = torch.randn((B, 512), generator=g).to(dev)
        a.x_in[:B] = x
        b.x_in[:B] = x
        a.step(B)
        b.replay(B)
        if rep % 20 == 19:
            torch.cuda.synchronize()
            assert torch.equal(a.out[:B], b.out[:B]) and a.out[:B].isfinite().all(), rep
            torch.mm(b.xn.float(), b.xn.float().t())
    torch.cuda.synchronize()
    assert a.lens == b.lens and torch.equal(a.kv_len, b.kv_len) and torch.equal(a.seq_len, b.seq_len)
    assert a.seq_len[:3].tolist() == [108, 65, 69] and max(a.lens) <= c.max_len and a.lens[0] < 60 + 1
    for ta, tb in zip(a.layers, b.layers):
        for s in range(B):
            n = a.lens[s]
            assert torch.equal(ta["mass"][s, :, :n], tb["mass"][s, :, :n]) and torch.equal(ta["pos"][s, :, :n], tb["pos"][s, :, :n])
    a.reset()
    assert a.lens == [0] * 12 and a.seq_len.tolist() == [0] * 12 and a.kv_len.tolist() == [0] * 12
    del gr


def test_state(gpu_ready, monkeypatch):
    """A prompt that would not fit after an eviction either, a refused call below, and sequences that have nothing to give."""
    st = toy(gpu_ready, dataclasses.replace(BASE, max_len=48), layers=1)
    x = torch.randn((12, 512), device=gpu_ready)
    for _ in range(4):
        st.prompt(1, x)
    with pytest.raises(ValueError):
        st.prompt(1, x)                                        # 40 + 12 > 48
    assert st.lens[1] == 48 and st.seq_len.tolist()[1] == 48
    st.evict(0)
    assert st.lens[0] == 0
    good = st.layers[0]["kv"]
    st.prompt(1, x[:8])
    st.layers[0]["kv"] = tuple(t[:, :, :12].contiguous() for t in good)
    with pytest.raises(SffnError):
        st.step(1)
    torch.cuda.synchronize()
    assert st.lens[:2] == [0, 48] and st.seq_len.tolist()[:2] == [0, 56] and st.kv_len.tolist()[:2] == [0, 48]
    st.layers[0]["kv"] = good
    st.step(2)
    assert st.lens[:2] == [1, 41]
    for s in (-1, 12):
        with pytest.raises(ValueError):
            st.evict(s)
    with pytest.raises(ValueError):
        toy(gpu_ready, CASES[2], layers=1).evict(0)
