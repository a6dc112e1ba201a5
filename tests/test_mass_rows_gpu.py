"""Attention mass where the device arrays name more tokens than the call has: no access leaves the tensors, and what the tokens' places
say stands in the results."""
import pytest
import torch

from activation_sparse_ffn_predictor_amd import _lib
from attn_util import Paged

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("end", [1 << 26, 1 << 30, (1 << 31) - 1])
@pytest.mark.parametrize("Hq,Hkv,d,kvt", [(64, 1, 64, "f16"), (128, 1, 256, "e4m3"), (8, 1, 128, "f16")])
def test_rows_past_the_call(gpu_ready, Hq, Hkv, d, kvt, end):
    """A sequence whose rows end far behind the call's: its tokens stand before its first one and see nothing, and every slot that it
    holds is one of its new tokens'."""
    dev, T, n = gpu_ready, 100, 600
    b = Paged([T], [n], Hkv, d, 16, "f16", kvt, seed=d)
    kv, _, kl, tab = b.gpu(dev)
    cu = torch.tensor([0, end], dtype=torch.int32, device=dev)
    q, lse = torch.randn((T, Hq, d), generator=b.g).half().to(dev), torch.zeros((T, Hq), device=dev)
    W = b.cols * 16
    old = torch.rand((1, Hkv, W), generator=b.g).to(dev)
    for max_q in (1, T):
        m, pos = old.clone(), torch.full((1, Hkv, W), -5, dtype=torch.int32, device=dev)
        need = _lib.attn_mass_workspace_size(1, Hq, Hkv, d, max_q, n, W)
        ws = torch.empty(max(need, 256), dtype=torch.uint8, device=dev)
        print(f"[rows past the call {Hq} {d} {kvt} {end} {max_q}]", flush=True)
        _lib.attn_mass(q, kv, cu, kl, tab, max_q, n, lse, m, pos, ws, seq_len=kl + 1000)
        torch.cuda.synchronize()
        assert bool((m[..., :n] == 0).all()) and torch.equal(m[..., n:], old[..., n:])
        assert torch.equal(pos[0, 0, :n].cpu(), torch.arange(1000, 1000 + n, dtype=torch.int32)) and bool((pos[..., n:] == -5).all())
