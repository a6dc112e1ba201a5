"""A stack that keeps the attended tokens: a step, prompt, capture or eviction that is refused in a later layer leaves every layer's
weights, positions and cache as they were, so what follows has the bits of a stack that never saw it."""
import dataclasses

import pytest
import torch

import synthgen as sg
from activation_sparse_ffn_predictor_amd import SffnError
from activation_sparse_ffn_predictor_amd.stack import AttnConfig, SparseFFNStack

pytestmark = pytest.mark.gpu
BASE = AttnConfig(8, 2, 64, "i8", page=16, max_len=48, sinks=2, rope_base=10000.0, weights="e4m3", keep=30, recent=6)


def toy(dev, c):
    return SparseFFNStack(sg.custom(sg.workload("toy_relu"), L=3), dev, max_batch=8, attn=c)


def held(st):
    """Lengths, and what every layer holds below them."""
    torch.cuda.synchronize()
    out = [list(st.lens), st.kv_len.tolist(), st.seq_len.tolist()]
    page = st.attn.page
    for t in st.layers:
        for s, n in enumerate(st.lens):
            out += [t["mass"][s, :, :n].tolist(), t["pos"][s, :, :n].tolist()]
            for x in t["kv"]:
                x = x.view(torch.uint8) if x.element_size() == 1 else x
                out += [x[st.table[s, j // page].item(), :, j % page].tolist() for j in range(0, n, 5)]
    return out


def spoil(st, layer, what):
    """Makes calls of a layer refused: a cache whose page the library does not take (before its weights change), an output projection
    of the wrong size (after they did)."""
    t = st.layers[layer]
    good = t[what]
    if what == "kv":
        t[what] = tuple(x[:, :, :12].contiguous() for x in good)
    elif isinstance(good, tuple):
        t[what] = (good[0][:, :-16].contiguous(), good[1])
    else:
        t[what] = good[:, :-16].contiguous()
    return lambda: t.__setitem__(what, good)


@pytest.mark.parametrize("what", ["kv", "W_o"])
@pytest.mark.parametrize("c", [BASE, dataclasses.replace(BASE, kv_type="f16", weights="f16")])
def test_refused_calls(gpu_ready, c, what):
    dev = gpu_ready
    a, b = toy(dev, c), toy(dev, c)
    g = torch.Generator().manual_seed(3)

    def both(f):
        f(a)
        f(b)
    for s, n in ((0, 8), (1, 5), (0, 8), (0, 8)):
        x = torch.randn((n, 512), generator=g).to(dev)
        both(lambda st: st.prompt(s, x))
    x = torch.randn((8, 512), generator=g).to(dev)
    for layer in (1, 2):
        before = held(b)
        undo = spoil(b, layer, what)
        b.x_in.normal_()
        for call in (lambda: b.step(2), lambda: b.prompt(0, x), lambda: b.prompt(2, x[:3]), lambda: b.capture(3)):
            with pytest.raises((SffnError, ValueError, RuntimeError)):
                call()
            undo()
            assert held(b) == before
            undo = spoil(b, layer, what)
        undo()
        y = torch.randn((2, 512), generator=g).to(dev)
        for st in (a, b):
            st.x_in[:2] = y
            st.step(2)
        assert held(a) == held(b) and torch.equal(a.out[:2], b.out[:2])


def test_refused_evictions(gpu_ready):
    dev = gpu_ready
    st = toy(dev, BASE)
    g = torch.Generator().manual_seed(4)
    for _ in range(6):
        st.prompt(1, torch.randn((8, 512), generator=g).to(dev))
    before = held(st)
    assert st.lens[1] == 48
    for call in (lambda: st.evict(1), lambda: st.prompt(1, torch.randn((4, 512), generator=g).to(dev))):
        undo = spoil(st, 2, "kv")
        with pytest.raises(SffnError):
            call()
        undo()
        assert held(st) == before
    st.evict(1)
    assert st.lens[1] == 30 and st.kv_len.tolist()[1] == 30 and st.seq_len.tolist()[1] == 48
