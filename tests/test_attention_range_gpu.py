"""Keys that outweigh all others but hold nothing where they do: the output there is the many small weights' alone.

fp16 weights refer to a power of two that leaves the largest one between 2^7 and 2^15, so that weights down to 2^-21 of it
are normal numbers, and the definition's bound (attn_def) has keys * 2^-32 * max|v| over the weights' sum for those below.
With one key in 32 that outweighs, and the others' weights at 2^-24.5 of it, the output is 31 * 2^-24.5 times a mean of
theirs: weights that were lost, or held in the few bits of a subnormal number, are seen at many times the bound."""
import math

import pytest
import torch

from attn_def import definition
from attn_util import DT, Paged, assert_near
from test_attention_gpu import TYPES, run_attn

pytestmark = pytest.mark.gpu


def dominated(ns, ks, Hkv, Hq, d, qt, kvt, gap, tail, seed, every, size):
    """A batch in which one key in `every` has a score `gap` nats over the others' (which vary by `tail`), and a value in
    element 0 alone, a large one (a row's scale in an 8-bit cache); queries [T, Hq, d]."""
    b = Paged(ns, ks, Hkv, d, 16, qt, kvt, seed=seed)
    x = torch.randn((2, b.n_pages, Hkv, 16, d), generator=b.g)
    x[0, ..., 0] = 0
    x[0, ..., 1:] *= tail
    x[1] = (x[1] + 2) * size
    for s in range(b.S):
        for j in range(0, ks[s], every):
            p, slot = int(b.table[s, j // 16]), j % 16
            x[0, p, :, slot] = 0
            x[0, p, :, slot, 0] = 4.0
            x[1, p, :, slot] = 0
            x[1, p, :, slot, 0] = 16 * size
    b.set_values(x.to(DT[qt]))
    q = torch.randn((b.T, Hq, d), generator=b.g)
    q[..., 0] = gap * d ** 0.5 / 4
    return b, q.to(DT[qt])


@pytest.mark.parametrize("qt,kvt", TYPES)
@pytest.mark.parametrize("n,d,Hq", [(1, 128, 8), (3, 64, 16), (1, 256, 4), (60, 128, 4), (60, 64, 4), (40, 256, 4)])
def test_small_weights_count(gpu_ready, n, d, Hq, qt, kvt):
    for gap, every in ((12.0, 32), (24.5 * math.log(2), 32), (25.5 * math.log(2), 32), (24.5 * math.log(2), 4000)):
        b, q = dominated([n], [4000], 2, Hq, d, qt, kvt, gap, 0.0, n + d, every, 100.0)
        out, lse = run_attn(b, q, Hq, gpu_ready)
        o, l, to, tl = definition(b, q, Hq, d ** -0.5)
        assert_near(out, o, to, f"out, gap {gap:.1f} every {every}")
        assert_near(lse, l, tl, f"lse, gap {gap:.1f} every {every}")


@pytest.mark.parametrize("qt,kvt", [("f16", "f16"), ("bf16", "i8"), ("f16", "e4m3"), ("bf16", "bf16")])
def test_small_weights_that_differ(gpu_ready, qt, kvt):
    """Tails of normally distributed scores, one of 131072 keys among them; windows and sinks."""
    for ns, ks, gap, window, sinks, every in (([1, 1], [3000, 700], 18.0, 0, 0, 32), ([1], [131072], 18.0, 0, 0, 32),
                                              ([1], [131072], 18.0, 0, 0, 131072), ([4], [6000], 16.0, 4096, 4, 6000),
                                              ([4], [6000], 16.0, 4096, 4, 32), ([50], [3000], 17.0, 0, 0, 32),
                                              ([30], [5000], 17.0, 2000, 1, 64)):
        b, q = dominated(ns, ks, 1, 2, 64, qt, kvt, gap, 0.5, 3, every, 100.0)
        out, lse = run_attn(b, q, 2, gpu_ready, window=window, sinks=sinks)
        o, l, to, tl = definition(b, q, 2, 0.125, window, sinks)
        assert_near(out, o, to, f"out {ks} {window}")
        assert_near(lse, l, tl, f"lse {ks} {window}")


@pytest.mark.parametrize("qt,kvt", TYPES)
@pytest.mark.parametrize("n", [2, 50])
def test_maxima_that_grow(gpu_ready, n, qt, kvt):
    """Scores that rise along the keys, by steps under and over what moves the reference: largest weights stay in range."""
    for step in (0.02, 0.15, 3.0):
        b = Paged([n], [800], 1, 64, 16, qt, kvt, seed=n)
        x = torch.randn((2, b.n_pages, 1, 16, 64), generator=b.g)
        x[0] = 0
        for p in range(800):
            x[0, int(b.table[0, p // 16]), 0, p % 16, 0] = step * p
        b.set_values(x.to(DT[qt]))
        q = torch.zeros((b.T, 4, 64))
        q[..., 0] = 1
        out, lse = run_attn(b, q.to(DT[qt]), 4, gpu_ready, scale=1.0)
        o, l, to, tl = definition(b, q.to(DT[qt]), 4, 1.0)
        assert_near(out, o, to, f"out, step {step}")
        assert_near(lse, l, tl, f"lse, step {step}")


@pytest.mark.parametrize("qt", ["f16", "bf16"])
@pytest.mark.parametrize("kvt", ["i8", "e4m3"])
def test_value_scales_far_apart(gpu_ready, qt, kvt):
    """V rows of sizes 2^-40 to 2^40 side by side (cache contents given as codes and scales): the large ones are the output,
    and the small ones count in the sum."""
    for n in (2, 60):
        b = Paged([n], [300], 2, 64, 16, "f16", kvt, seed=n)
        b.qt = qt
        size = torch.tensor([2.0 ** -40, 1.0, 2.0 ** 40, 2.0 ** -20])[torch.arange(16) % 4]
        b.scales = b.scales.clone()
        b.scales[1] *= size
        b.val[1] *= size.double()[:, None]
        if qt == "f16":                              # outputs within fp16's range
            b.scales[1] *= 2.0 ** -42
            b.scales[1] = b.scales[1].clamp(min=2.0 ** -60)
            b.val[1] = b.codes[1].double() * b.scales[1].double()[..., None]
        q = (torch.randn((n, 4, 64), generator=b.g) * 2).to(DT[qt])
        out, lse = run_attn(b, q, 4, gpu_ready)
        o, l, to, tl = definition(b, q, 4, 0.125)
        assert_near(out, o, to, "out")
        assert_near(lse, l, tl, "lse")
