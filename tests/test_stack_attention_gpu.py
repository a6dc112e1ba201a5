"""The resident stack with attention: prompts in chunks, decode steps eager and replayed, each layer's attention half
checked from the buffers it worked on (its input is the GPU's own)."""
import numpy as np
import pytest
import torch

import synthgen as sg
from activation_sparse_ffn_predictor_amd.stack import AttnConfig, SparseFFNStack
from attn_util import DT, TOP, Paged, assert_near, attention, half_step, quant_rows

pytestmark = pytest.mark.gpu


def toy(dev, kv_type, max_batch=12, window=0, sinks=0, max_len=100, layers=2):
    wl = sg.custom(sg.workload("toy_relu"), L=layers)
    return SparseFFNStack(wl, dev, max_batch=max_batch,
                          attn=AttnConfig(8, 2, 64, kv_type, page=16, max_len=max_len, window=window, sinks=sinks))


def check_half(st, i, x, before, T, ns, lens, rows):
    """Layer i's attention half, run for T tokens (ns new ones of the sequences `rows`, whose lengths are `lens` with them),
    from its input x and the residual `before`."""
    c, t = st.attn, st.layers[i]
    kt = c.kv_type
    h0 = x.cpu().float() + (before.cpu() if before is not None else 0)
    xn = h0.double() / torch.sqrt(h0.double().square().mean(-1, keepdim=True) + c.eps) * t["w_attn"].cpu().double()
    D = h0.shape[1]
    f32 = (D / 2 + 8) * 2.0 ** -24
    tiny = torch.finfo(torch.float16).tiny * half_step("f16") * 1.01
    assert_near(st.xn[:T], xn, (f32 + half_step("f16") * 1.01) * xn.abs() + tiny, "norm")
    qkv = st.qkv[:T].cpu().unflatten(1, (-1, c.head_dim))
    q, k, v = qkv.split([c.n_heads, c.n_kv_heads, c.n_kv_heads], dim=1)
    b = Paged(ns, lens, c.n_kv_heads, c.head_dim, c.page, "f16", kt, cols=st.table.shape[1])
    b.table = st.table.cpu()[rows]
    b.n_pages = t["kv"][0].shape[0]
    codes = torch.stack([x.view(torch.uint8).cpu().view(x.dtype).float() for x in t["kv"][:2]])
    b.val = codes.double()
    if kt in TOP:
        scales = torch.stack([x.cpu() for x in t["kv"][2:]])
        b.val = b.val * scales.double()[..., None]
    # the new tokens' rows are in their places
    r = 0
    for s, (n, ln) in enumerate(zip(ns, lens)):
        for p in range(ln - n, ln):
            pid, slot = int(b.table[s, p // c.page]), p % c.page
            for m, src in enumerate((k, v)):
                if kt in TOP:
                    cc, sc = quant_rows(src[r].double(), kt)
                    assert torch.equal(codes[m][pid, :, slot].double(), cc) and torch.equal(scales[m][pid, :, slot], sc)
                else:
                    assert torch.equal(codes[m][pid, :, slot].half(), src[r])
            r += 1
    o, _, to, _ = attention(b, q, c.n_heads, c.head_dim ** -0.5, c.window, c.sinks)
    assert_near(st.o[:T], o, to, "attention")
    h1 = h0 + st.ao[:T].cpu().float()
    assert torch.equal(st.h[:T].cpu(), h1)
    xf = h1.double() / torch.sqrt(h1.double().square().mean(-1, keepdim=True) + c.eps) * t["w_ffn"].cpu().double()
    assert_near(st.xf[:T], xf, f32 * xf.abs() + 1e-30, "second norm")


@pytest.mark.parametrize("kv_type,window,sinks", [("f16", 0, 0), ("i8", 0, 0), ("e4m3", 20, 3)])
def test_layers(gpu_ready, kv_type, window, sinks):
    dev = gpu_ready
    st = toy(dev, kv_type, window=window, sinks=sinks)
    g = torch.Generator().manual_seed(1)

    def run(T, x, cu, rows, ns, max_q):
        kl, tab = st.kv_len[rows], st.table[rows].contiguous()
        for i in range(2):
            before = st.h[:T].clone() if i else None
            st.attn_layer(i, x, T, cu, kl, tab, max_q)
            torch.cuda.synchronize()
            check_half(st, i, x, before, T, ns, [st.lens[r] for r in rows], rows)
            st.layer_call(i, st.xf[:T], False, st.y[i, :T])
            x = st.y[i, :T].clone()

    for s, T in ((0, 12), (1, 7), (0, 12), (1, 1)):            # chunks of two prompts
        st.kv_len[s] += T
        st.lens[s] += T
        run(T, torch.randn((T, 512), generator=g).to(dev), torch.tensor([0, T], dtype=torch.int32, device=dev), [s], [T], T)
    for _ in range(2):                                         # both decode
        st.kv_len[:2] += 1
        st.lens[:2] = [n + 1 for n in st.lens[:2]]
        run(2, torch.randn((2, 512), generator=g).to(dev), st.cu_step[:3], [0, 1], [1, 1], 1)


@pytest.mark.parametrize("kv_type", ["f16", "i8"])
def test_prompt_steps_and_replays_agree(gpu_ready, kv_type):
    """The same tokens by prompts and eager steps in one stack, and by prompts and graph replays in another, with
    eager work between: the same bits; a window of one stack's tokens entered step by step gives the same cache."""
    dev, B = gpu_ready, 3
    a, b = toy(dev, kv_type), toy(dev, kv_type)
    g = torch.Generator().manual_seed(2)
    xs = [torch.randn((n, 512), generator=g).to(dev) for n in (12, 5, 9)]
    for st in (a, b):
        for s, x in enumerate(xs):
            st.prompt(s, x)
    b.x_in.normal_()
    gr = b.capture(B)
    assert b.lens[:B] == [12, 5, 9] and b.kv_len[:B].tolist() == [12, 5, 9]
    for rep in range(4):
        x = torch.randn((B, 512), generator=g).to(dev)
        a.x_in[:B] = x
        b.x_in[:B] = x
        a.step(B)
        b.replay(B)
        torch.cuda.synchronize()
        assert torch.equal(a.out[:B], b.out[:B]) and torch.equal(a.y[:, :B], b.y[:, :B]), rep
        assert a.out[:B].isfinite().all() and a.kv_len.tolist() == b.kv_len.tolist()
        torch.mm(b.xn.float(), b.xn.float().t())               # eager work between replays
        torch.cuda.synchronize()
    for i in range(2):
        for s in range(B):
            n, pages = a.lens[s], a.table[s].cpu()
            for p in range(n):
                pid, slot = int(pages[p // 16]), p % 16
                for ta, tb in zip(a.layers[i]["kv"], b.layers[i]["kv"]):
                    assert torch.equal(ta[pid, :, slot].float(), tb[pid, :, slot].float())
    a.reset()
    assert a.lens == [0] * 12 and a.kv_len.tolist() == [0] * 12
    del gr


def test_no_room_is_refused(gpu_ready):
    st = toy(gpu_ready, "f16", max_batch=4, max_len=6, layers=1)
    x = torch.zeros((4, 512), device=gpu_ready)
    st.prompt(0, x)
    with pytest.raises(ValueError):
        st.prompt(0, x)
    with pytest.raises(ValueError):
        st.prompt(4, x)
    with pytest.raises(ValueError):
        st.prompt(0, torch.zeros((5, 512), device=gpu_ready))
    st.step(1)
    st.step(1)
    with pytest.raises(ValueError):
        st.step(1)
    assert st.lens == [6, 0, 0, 0]
    plain = SparseFFNStack(sg.workload("toy_relu"), gpu_ready)
    with pytest.raises(ValueError):
        plain.prompt(0, x[:1])


def test_prompt_checks_its_input_first(gpu_ready):
    """A refused prompt leaves the sequence as it was; rows need not be dense."""
    st = toy(gpu_ready, "f16", max_batch=4, max_len=16, layers=1)
    wide = torch.randn((4, 1032), device=gpu_ready, generator=torch.Generator(gpu_ready).manual_seed(2))
    for x in (wide, wide[:, :504], wide[:, :512].half(), wide[:, :512].cpu(), wide[0, :512][None, None]):
        with pytest.raises(ValueError):
            st.prompt(0, x)
    assert st.lens == [0, 0, 0, 0] and (st.kv_len == 0).all()
    st.prompt(0, wide[:, 3:515])
    a = st.out.clone()
    st.prompt(1, wide[:, 3:515].contiguous())
    assert torch.equal(a, st.out) and st.lens == [4, 4, 0, 0]
