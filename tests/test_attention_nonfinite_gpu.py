"""Infinities and NaN in the cache: in places that a row does not see they change nothing, where it sees them it shows them,
however small their weight. 8-bit caches may hold e4m3's NaN codes (0x7F, 0xFF), which no write stores."""
import math

import pytest
import torch

from attn_def import definition
from attn_util import DT, Paged, assert_near
from test_attention_gpu import run_attn

pytestmark = pytest.mark.gpu

# new tokens, cached tokens, window, sinks, positions of sequence 0 that hold NaN codes
CODES = {
    "draft: the last token": ([3, 1], [90, 40], 0, 0, [89]),
    "drafts: later tokens": ([4], [70], 0, 0, [67, 69]),
    "before the window": ([1, 2], [200, 90], 40, 0, [150, 131, 3]),
    "between sinks and window": ([2], [300], 64, 5, [5, 100, 236]),
    "seen by all": ([2], [300], 0, 0, [10]),
    "chunk: later tokens": ([70], [150], 0, 0, [149, 120, 81]),
    "chunk: before windows": ([90, 20], [300, 60], 50, 3, [3, 170, 250, 240]),
    "chunk: seen by all": ([60], [300], 0, 0, [0]),
    "spread": ([2], [3000], 1000, 2, [2, 1995, 2000, 2999]),
    "chunk, spread": ([20], [3000], 1500, 9, [9, 1485, 2990]),
}


@pytest.mark.parametrize("qt", ["f16", "bf16"])
@pytest.mark.parametrize("d", [64, 128, 208])
@pytest.mark.parametrize("name", CODES)
def test_nan_codes(gpu_ready, name, d, qt):
    ns, ks, window, sinks, at = CODES[name]
    print(f"[nan codes {name} {qt} d={d}]", flush=True)
    b = Paged(ns, ks, 2, d, 16, qt, "e4m3", seed=len(name) + d, pad=1)
    for i, p in enumerate(at):                       # element 3 i of V, and an element of K's next head
        pid, slot = int(b.table[0, p // 16]), p % 16
        b.codes.view(torch.uint8)[1, pid, i % 2, slot, 3 * i] = 0x7F if i % 2 else 0xFF
        b.val[1, pid, i % 2, slot, 3 * i] = math.nan
    last = ks[0] - 1                                 # slots behind the sequence's end
    if last % 16 != 15:
        b.codes.view(torch.uint8)[:, int(b.table[0, last // 16]), :, last % 16 + 1:] = 0x7F
        b.val[:, int(b.table[0, last // 16]), :, last % 16 + 1:] = math.nan
    q = torch.randn((b.T, 8, d), generator=b.g).to(DT[qt])
    out, lse = run_attn(b, q, 8, gpu_ready, window=window, sinks=sinks)
    o, l, to, tl = definition(b, q, 8, d ** -0.5, window, sinks)
    assert bool(o[:b.N].isnan().any()) == (name != "before the window") and not o[:b.N].isnan().all()
    assert_near(out[:b.N], o[:b.N], to[:b.N], "out")
    assert_near(lse[:b.N], l[:b.N], tl[:b.N], "lse")


@pytest.mark.parametrize("d", [64, 128, 256])
def test_nan_key_codes(gpu_ready, d):
    """Keys with a NaN code: NaN for the rows that see them, nothing for the others."""
    for n, window in ((3, 0), (3, 30), (60, 0), (60, 30)):
        b = Paged([n], [150], 1, d, 16, "f16", "e4m3", seed=d)
        for p in (149, 60):
            b.codes.view(torch.uint8)[0, int(b.table[0, p // 16]), 0, p % 16, 5] = 0x7F
            b.val[0, int(b.table[0, p // 16]), 0, p % 16, 5] = math.nan
        q = torch.randn((n, 4, d), generator=b.g).half()
        out, lse = run_attn(b, q, 4, gpu_ready, window=window)
        p = 150 - n + torch.arange(n)
        bad = (p == 149) | ((p >= 60) & ((p < 90) if window else True))
        assert torch.equal(out.isnan().all(-1).all(-1).cpu(), bad) and torch.equal(lse.isnan().all(-1).cpu(), bad)
        b.val = torch.nan_to_num(b.val)
        o, l, to, tl = definition(b, q, 4, d ** -0.5, window)
        assert_near(out.cpu()[~bad], o[~bad], to[~bad])
        assert_near(lse.cpu()[~bad], l[~bad], tl[~bad])


@pytest.mark.parametrize("qt", ["f16", "bf16"])
@pytest.mark.parametrize("n,d", [(1, 64), (2, 128), (1, 256), (60, 64), (60, 128), (40, 256)])
def test_infinities_under_vanishing_weights(gpu_ready, n, d, qt):
    """An infinity whose weight is far below what 16 bits, or 32, hold: the output is that infinity in a unit of keys that
    every row sees as in one that some row sees in part; one of each sign, or a NaN: NaN."""
    for k, gap in ((200, 30.0), (200, 300.0), (3000, 60.0)):
        b = Paged([n], [k], 1, d, 16, qt, qt, seed=n + d)
        x = torch.randn((2, b.n_pages, 1, 16, d), generator=b.g)
        x[0] *= 0.1
        x[0, ..., 0] = 0

        def put(p, el, v):
            x[1, int(b.table[0, p // 16]), 0, p % 16, el] = v
        for s in range(0, k, 32):                    # in every part of the keys
            x[0, int(b.table[0, s // 16]), 0, s % 16, 0] = 8.0
        put(33, 1, math.inf)
        put(34, 2, -math.inf)
        put(35, 3, math.inf)
        put(70, 3, -math.inf)
        put(36, 4, math.nan)
        put(k - n, 5, math.inf)
        put(k - 1, 6, -math.inf)
        put(k // 2 + 3, 9, math.inf)
        b.set_values(x.to(DT[qt]))
        q = torch.randn((n, 4, d), generator=b.g)
        q[..., 0] = gap * d ** 0.5 / 8
        q = q.to(DT[qt])
        out, lse = run_attn(b, q, 4, gpu_ready)
        o, l, to, tl = definition(b, q, 4, d ** -0.5)
        assert (o[:, :, 1] == math.inf).all() and (o[:, :, 9] == math.inf).all() and o[:, :, 3].isnan().all()
        assert_near(out, o, to, f"out {k} {gap}")
        assert_near(lse, l, tl, f"lse {k} {gap}")
