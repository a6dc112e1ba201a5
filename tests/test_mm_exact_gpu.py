"""The block-scaled product where nothing may be lost, for every kernel that a call can take: results bit for bit.

Codes from 1 to 3.75 (either sign) and zeros: a product has a leading bit of 2^0 to 2^3 and no bit below 2^-6, so none lies 2^-13
under the largest of its neighbours, and the 8-bit instruction keeps all of them as the fp16 one does. Scales are powers of two from
1/2 to 2: every term is a multiple of 2^-8, and where the terms' magnitudes add up to less than 2^16 every partial sum has at most 24
bits, exact in fp32 in any order. What is left is one rounding to the result's type."""
import math

import pytest
import torch

from activation_sparse_ffn_predictor_amd import _lib
from attn_util import DT
from layer_def import blocks, spread
from test_layer_ops_gpu import mm, say

pytestmark = pytest.mark.gpu

# T, N, K, results: each kernel with k in one share and in several, tokens and rows that end inside tiles, blocks and shares
EXACT = [(1, 136, 16, "bf16"), (13, 264, 1040, "f16"), (2, 1032, 4112, "f32"),
         (21, 264, 1856, "f16"), (31, 24584, 640, "bf16"), (18, 2056, 4112, "f32"),
         (38, 136, 4032, "bf16"), (60, 16392, 912, "f16"), (47, 2056, 2064, "f32"),
         (65, 136, 272, "f16"), (79, 264, 4064, "bf16"), (70, 4104, 2064, "f16"), (129, 648, 528, "bf16"), (264, 2064, 2720, "f32"), (100, 1032, 400, "f32"),
         (259, 8200, 1040, "bf16"), (153, 1384, 4912, "f16"), (66, 8832, 3248, "bf16"), (130, 1416, 4752, "f32"), (273, 5512, 272, "f32"),
         (1064, 7248, 272, "bf16"), (131, 5688, 7648, "f16"), (513, 10248, 8208, "f16"), (1000, 10248, 8208, "bf16"), (4095, 8192, 1040, "f16"),
         (1025, 8200, 528, "bf16")]
# one product a result, of every code with every code
VALUES = [(5, 264, 256, "f16"), (19, 264, 256, "bf16"), (40, 264, 256, "f16"), (200, 264, 256, "bf16"), (70, 264, 256, "f16"), (259, 8200, 272, "bf16"),
          (133, 9704, 272, "f16"), (1064, 7248, 272, "bf16"), (1025, 8200, 528, "f16")]


def exact_case(T, N, K):
    g = torch.Generator().manual_seed(T * 11 + N * 3 + K)

    def some(rows, dense):
        m = 1 + torch.randint(0, 8, (rows, K), generator=g).double() / 8
        v = m * 2.0 ** torch.randint(0, 2, (rows, K), generator=g) * (1 - 2.0 * torch.randint(0, 2, (rows, K), generator=g))
        return torch.where(torch.rand((rows, K), generator=g) < dense, v, torch.zeros((), dtype=torch.float64))
    scale = [2.0 ** torch.randint(-1, 2, s, generator=g).float() for s in ((T, blocks(K)), (blocks(N), blocks(K)))]
    return some(T, min(1.0, 700 / K)), scale[0], some(N, 1.0), scale[1]


@pytest.mark.parametrize("T,N,K,ot", EXACT)
def test_exact(gpu_ready, T, N, K, ot):
    dev = gpu_ready
    a, sa, b, sb = exact_case(T, N, K)
    x, w = (a * spread(sa, 1, T, K)).to(dev), (b * spread(sb, 128, N, K)).to(dev)
    assert (x.abs() @ w.abs().t().contiguous()).amax().item() < 2.0 ** 16
    want = x @ w.t().contiguous()                                                      # (exact in 64 bits)
    assert want.abs().amax().item() < 65504 and torch.equal(want.float().double(), want)
    want = want.float().to(DT[ot])
    for pad in (0, 8):
        say(f"[exact {T} {N} {K} {ot} pad {pad}]")
        out = mm(dev, a, sa, b, sb, ot, pad)
        assert torch.equal(out, want), (out != want).nonzero()[:4].tolist()


@pytest.mark.parametrize("T,N,K,ot", VALUES)
def test_values(gpu_ready, T, N, K, ot):
    """Every code times every code, one product a result: a 4 x 4 bit mantissa, exact in every type once 1/4 keeps 448 * 448 in fp16's
    range. Then NaN codes and scales, an infinite and a zero scale, which change the results that they enter and no others."""
    dev = gpu_ready
    every = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float().double()
    every = every[~torch.isnan(every)]                                                 # 254
    t, n = torch.arange(T), torch.arange(N)
    ka = (7 * t) % K
    av, bv = every[(53 * t) % 254], every[n % 254]
    a, b = torch.zeros((T, K), dtype=torch.float64), bv[:, None].expand(N, K).clone()
    a[t, ka] = av
    sa, sb = torch.full((T, blocks(K)), 0.5), torch.full((blocks(N), blocks(K)), 0.5)
    want = (av[:, None] * bv[None] * 0.25).to(dev)
    assert torch.equal(want.to(DT[ot]).double(), want)
    say(f"[values {T} {N} {K} {ot}]")
    assert torch.equal(mm(dev, a, sa, b, sb, ot).double(), want)

    a[1, 3] = math.nan
    sa[2, blocks(K) - 1] = math.nan
    sa[3] = 0
    b[200, 5] = math.nan
    sb[0, 0] = math.inf
    out = mm(dev, a, sa, b, sb, ot).double()
    bad = torch.zeros((T, N), dtype=torch.bool, device=dev)
    bad[1:3] = True
    bad[:, 200] = True
    assert bool(torch.isnan(out[bad]).all())
    first = (ka < 128).to(dev)[:, None] & (av != 0).to(dev)[:, None] & (bv[:128] != 0).to(dev)[None]
    inf = torch.where(first, want[:, :128].sign() * math.inf, math.nan)                # (0 times infinity elsewhere)
    inf[3] = math.nan
    keep = ~bad[:, :128]
    assert torch.equal(torch.isnan(out[:, :128])[keep], torch.isnan(inf)[keep])
    assert torch.equal(torch.nan_to_num(out[:, :128])[keep], torch.nan_to_num(inf)[keep])
    want[3] = 0
    keep = ~bad[:, 128:]
    assert torch.equal(out[:, 128:][keep], want[:, 128:][keep])
