"""What a stack with attention keeps between calls: a refused call leaves its sequences as they were."""
import pytest
import torch

import synthgen as sg
from activation_sparse_ffn_predictor_amd import SffnError
from activation_sparse_ffn_predictor_amd.stack import AttnConfig, SparseFFNStack

pytestmark = pytest.mark.gpu


def toy(dev, max_batch=4, max_len=40, **kw):
    c = dict(n_heads=8, n_kv_heads=2, head_dim=64, kv_type="f16", page=16, max_len=max_len)
    c.update(kw)
    return SparseFFNStack(sg.custom(sg.workload("toy_relu"), L=1), dev, max_batch=max_batch, attn=AttnConfig(**c))


def state(st):
    torch.cuda.synchronize()
    return list(st.lens), st.kv_len.tolist()


def test_replay_of_an_uncaptured_batch(gpu_ready):
    st = toy(gpu_ready)
    st.x_in.normal_()
    st.prompt(0, torch.randn((3, 512), device=gpu_ready))
    g = st.capture(2)
    before = state(st)
    for B in (1, 3, 4):
        with pytest.raises((KeyError, ValueError)):
            st.replay(B)
        assert state(st) == before
    st.replay(2)
    assert state(st) == ([4, 1, 0, 0], [4, 1, 0, 0])
    del g


@pytest.mark.parametrize("B", [0, -1, 5])
def test_batches_out_of_range(gpu_ready, B):
    st = toy(gpu_ready)
    before = state(st)
    for call in (st.step, st.capture, st.replay):
        with pytest.raises((KeyError, ValueError)):
            call(B)
        assert state(st) == before


def test_a_call_refused_below_leaves_the_sequences(gpu_ready, monkeypatch):
    """The library turns a layer's call away (here: a cache whose page size it does not take)."""
    st = toy(gpu_ready)
    st.prompt(1, torch.randn((2, 512), device=gpu_ready))
    before = state(st)
    good = st.layers[0]["kv"]
    st.layers[0]["kv"] = tuple(t[:, :, :12].contiguous() for t in good)
    for call in (lambda: st.step(2), lambda: st.prompt(1, torch.randn((3, 512), device=gpu_ready)), lambda: st.capture(3)):
        with pytest.raises(SffnError):
            call()
        assert state(st) == before
    st.layers[0]["kv"] = good
    st.step(2)
    assert state(st) == ([1, 3, 0, 0], [1, 3, 0, 0])


def test_prompts_longer_than_the_ffn_takes(gpu_ready):
    """The sparse FFN takes up to 64 tokens a call, so a prompt of more is refused, and changes nothing."""
    st = toy(gpu_ready, max_batch=70, max_len=100)
    st.prompt(2, torch.randn((64, 512), device=gpu_ready))
    before = state(st)
    for call in (lambda: st.prompt(2, torch.randn((65, 512), device=gpu_ready)[:, :512]), lambda: st.step(66)):
        with pytest.raises((ValueError, SffnError)):
            call()
        assert state(st) == before
    st.prompt(2, torch.randn((30, 512), device=gpu_ready))
    assert st.lens[2] == 94


def test_prompt_uploads_nothing_it_has(gpu_ready):
    """A prompt of a length that was entered before builds no new tensor of its boundaries (one is kept for each length)."""
    st = toy(gpu_ready)
    st.prompt(0, torch.randn((3, 512), device=gpu_ready))
    kept = st.cu_prompt[3]
    real, made = torch.tensor, []

    def spy(*a, **kw):
        made.append(a)
        return real(*a, **kw)
    torch.tensor = spy
    try:
        st.prompt(1, torch.randn((3, 512), device=gpu_ready))
    finally:
        torch.tensor = real
    assert not made and st.cu_prompt[3] is kept


@pytest.mark.parametrize("kw", [dict(n_kv_heads=0), dict(n_heads=0), dict(head_dim=60), dict(head_dim=0), dict(page=24), dict(page=8),
                                dict(kv_type="i8", head_dim=72), dict(kv_type="bf16"), dict(max_len=0), dict(window=-1), dict(sinks=-1),
                                dict(n_heads=7), dict(eps=-1.0)])
def test_configurations_are_checked_at_the_start(gpu_ready, kw):
    with pytest.raises(ValueError):
        toy(gpu_ready, **kw)
