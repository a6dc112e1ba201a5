"""What a stack with attention keeps between calls: a refused call leaves its sequences as they were."""
import pytest
import torch

import synthgen as sg
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
