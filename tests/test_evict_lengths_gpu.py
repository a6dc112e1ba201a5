"""An eviction's lengths: kv_len counts the sequence's tokens where seq_len is left out, if the new lengths go elsewhere."""
import pytest
import torch

from activation_sparse_ffn_predictor_amd import SffnError, _lib
from attn_util import Paged
from layer_def import evicted

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("ks,keep", [([70, 32, 9], 32), ([9000, 5000], 4500)])
def test_lengths_left_out(gpu_ready, ks, keep):
    dev, Hkv = gpu_ready, 2
    b = Paged([0] * len(ks), ks, Hkv, 16, 16, "f16", "f16", seed=keep)
    W = b.cols * 16
    m = torch.rand((b.S, Hkv, W), generator=b.g)
    pos = torch.arange(W, dtype=torch.int32).expand(b.S, Hkv, W).contiguous()
    ws = torch.empty(_lib.kv_evict_workspace_size(b.S, Hkv, W, keep), dtype=torch.uint8, device=dev)

    def run(**kw):
        kv, _, kl, tab = b.gpu(dev)
        gm, gp = m.to(dev), pos.to(dev)
        src = torch.full((b.S, Hkv, keep), -9, dtype=torch.int32, device=dev)
        before = [t.clone() for t in (kl, gm, gp, src) + tuple(kv)]
        kw = {k: v(kl) for k, v in kw.items()}
        try:
            _lib.kv_evict(kv, kl, tab, gm, gp, keep, src, ws, sinks=2, recent=7, **kw)
        except SffnError as e:
            torch.cuda.synchronize()
            assert "kv_len_out" in str(e) and "seq_len" in str(e)
            assert all(torch.equal(x, y) for x, y in zip((kl, gm, gp, src) + tuple(kv), before))
            return None
        torch.cuda.synchronize()
        return src.cpu(), (kw["kv_len_out"] if "kv_len_out" in kw else kl).cpu()
    assert run() is None                                        # both left out: the count would be lost
    want = torch.tensor([[evicted(k, k, [True] * k, m[s, h].tolist(), pos[s, h].tolist(), keep, 2, 7) for h in range(Hkv)] for s, k in enumerate(ks)])
    for got in (run(seq_len=torch.clone), run(kv_len_out=torch.zeros_like), run(seq_len=torch.clone, kv_len_out=torch.zeros_like)):
        assert torch.equal(got[0].long(), want) and got[1].tolist() == [min(k, keep) for k in ks]
