"""The kernels that serve large calls, just past the sizes that choose them: the few-row kernel's four-wave workgroups (more
than 256 workgroups), with and without shares of the keys, and the write's and the read's two tokens a thread (from 16384
workgroups of one token)."""
import pytest
import torch

from activation_sparse_ffn_predictor_amd import _lib
from attn_def import definition
from attn_util import DT, TOP, Paged, assert_near, quant_rows
from test_attention_gpu import CACHES, TYPES, f64, run_attn

pytestmark = pytest.mark.gpu


def shares(T, S, Hq, Hkv, d, max_q, max_kv):
    """Shares of the keys, from the workspace that they need: (d + 2) fp32 a row and share, each part rounded up to 256."""
    need = _lib.attn_workspace_size(T, S, Hq, Hkv, d, max_q, max_kv)
    return max(1, round(need / (T * Hq * (d + 2) * 4)))


# head size, query heads a K/V head, most new tokens: row tiles of 16, of one, two and four
ROWS = [(64, 4, 1), (64, 8, 3), (64, 16, 4), (48, 1, 40), (128, 8, 1), (128, 8, 4), (112, 16, 2), (128, 5, 3), (256, 8, 1), (208, 4, 4)]


@pytest.mark.parametrize("qt,kvt", TYPES)
@pytest.mark.parametrize("d,G,n", ROWS)
def test_many_workgroups_of_few_rows(gpu_ready, d, G, n, qt, kvt):
    """Over 256 sequences and heads: one share each, window and sinks too; sequences with fewer tokens among them."""
    S, Hkv = 70, 4
    assert _lib.attn_path(G * Hkv, Hkv, d, n) == _lib.ATTN_FEW and S * Hkv > 256
    ns = [n if i % 3 == 0 else (i * 7) % (n + 1) for i in range(S)]
    ks = [max(ns[i], 1 + (37 * i) % 130) for i in range(S)]
    assert shares(sum(ns), S, G * Hkv, Hkv, d, n, max(ks)) == 1
    print(f"[few, many workgroups d={d} G={G} n={n} {qt} {kvt}]", flush=True)
    for window, sinks in ((0, 0), (45, 3)):
        b = Paged(ns, ks, Hkv, d, 16, qt, kvt, seed=d + G, pad=1, v_scale=0.6)
        q = torch.randn((b.T, G * Hkv, d), generator=b.g).to(DT[qt])
        out, lse = run_attn(b, q, G * Hkv, gpu_ready, window=window, sinks=sinks)
        o, l, to, tl = definition(b, q, G * Hkv, d ** -0.5, window, sinks)
        assert_near(out[:b.N], o[:b.N], to[:b.N], "out")
        assert_near(lse[:b.N], l[:b.N], tl[:b.N], "lse")
        assert (out[b.N:] == 3.0).all()


@pytest.mark.parametrize("qt,kvt", TYPES)
@pytest.mark.parametrize("d,G,n", ROWS)
def test_many_workgroups_with_shares(gpu_ready, d, G, n, qt, kvt):
    """Few sequences whose keys are spread until there are over 256 workgroups; short ones use fewer shares."""
    S, Hkv, most = 8, 6, 100000
    ns, ks = [n, 1, n, 0, n, n, 1, n], [1300, 700, 520, 90, 1000, 60, 1, 513]
    ks = [max(a, b) for a, b in zip(ns, ks)]
    parts = shares(sum(ns), S, G * Hkv, Hkv, d, n, most)
    assert _lib.attn_path(G * Hkv, Hkv, d, n) == _lib.ATTN_FEW and parts > 1 and parts * S * Hkv > 256
    print(f"[few, many shares d={d} G={G} n={n} {qt} {kvt}]", flush=True)
    b = Paged(ns, ks, Hkv, d, 32, qt, kvt, seed=d + G, pad=1, v_scale=0.6)
    q = torch.randn((b.T, G * Hkv, d), generator=b.g).to(DT[qt])
    out, lse = run_attn(b, q, G * Hkv, gpu_ready, max_kv=most)
    o, l, to, tl = definition(b, q, G * Hkv, d ** -0.5)
    assert_near(out[:b.N], o[:b.N], to[:b.N], "out")
    assert_near(lse[:b.N], l[:b.N], tl[:b.N], "lse")
    assert (out[b.N:] == 3.0).all()


@pytest.mark.parametrize("qt,kvt,d", [(c[0], c[1], c[2]) for c in CACHES] + [("f16", "f16", 64), ("bf16", "bf16", 16), ("f16", "i8", 64),
                                      ("f16", "i8", 256), ("bf16", "e4m3", 128), ("f16", "e4m3", 16)])
def test_two_tokens_a_thread(gpu_ready, qt, kvt, d):
    """Ragged sequences that begin and end between a thread's two tokens, rows behind the last one, a bad page and a position
    before the first token among them."""
    dev, page = gpu_ready, 16
    lanes = 4 if d <= 32 else 8 if d <= 64 else 16 if d <= 128 else 32
    tok = 256 // lanes                               # tokens of a workgroup that takes one a thread
    ns = [tok // 2 + 1, 0, 3, tok, 1, tok // 2, 5]
    pad = 2
    T = sum(ns) + pad
    Hkv = -(-(16384 + 64) // (-(-T // tok)))
    assert -(-T // tok) * Hkv >= 16384 and T % (2 * tok)
    ks = [n + 11 for n in ns]
    ks[6] = 3                                        # the first two of five tokens lie before the sequence
    g = torch.Generator(device=dev).manual_seed(d)
    need = [-(-max(k, 1) // page) for k in ks]
    n_pages, cols = sum(need) + 1, max(need)
    ids = torch.randperm(n_pages, generator=g, device=dev).int().cpu().tolist()
    table, at = torch.full((len(ns), cols), -1, dtype=torch.int32), 0
    for s, m in enumerate(need):
        table[s, :m] = torch.tensor(ids[at:at + m], dtype=torch.int32)
        at += m
    table[3, 1] = n_pages                            # sequence 3's positions 16 .. 31 have no page
    cu = torch.tensor([0] + [sum(ns[:i + 1]) for i in range(len(ns))], dtype=torch.int32)
    print(f"[two tokens a thread {qt} {kvt} d={d} heads={Hkv} T={T}]", flush=True)
    x = torch.randn((2, T, Hkv, d), generator=g, device=dev).to(DT[qt])
    kv = [torch.zeros((n_pages, Hkv, page, d), device=dev).to(DT[kvt]) for _ in range(2)]
    if kvt in TOP:
        kv += [torch.full((n_pages, Hkv, page), -1.0, device=dev) for _ in range(2)]
    gpu = cu.to(dev), torch.tensor(ks, dtype=torch.int32, device=dev), table.to(dev)
    _lib.kv_write(x[0], x[1], tuple(kv), *gpu)
    back = torch.full((2, T, Hkv, d), 3.0, device=dev).to(DT[qt])
    _lib.kv_read(tuple(kv), *gpu, back[0], back[1])
    torch.cuda.synchronize()
    place = {}                                       # page and slot of each token that has one
    for s, n in enumerate(ns):
        for i in range(n):
            p = ks[s] - n + i
            if p >= 0 and 0 <= int(table[s, p // page]) < n_pages:
                place[int(cu[s]) + i] = (int(table[s, p // page]), p % page)
    assert len(place) < sum(ns) - 2
    lone = torch.ones((n_pages, page), dtype=torch.bool)
    for t in range(T):
        if t not in place:
            assert (back[:, t] == 3.0).all(), t
            continue
        pid, slot = place[t]
        lone[pid, slot] = False
        for m in range(2):
            if kvt in TOP:
                c, sc = quant_rows(x[m, t].double().cpu(), kvt)
                assert torch.equal(f64(kv[m][pid, :, slot]), c) and torch.equal(kv[2 + m][pid, :, slot].cpu(), sc), (t, m)
                assert torch.equal(back[m, t].cpu(), (c.float() * sc[:, None]).to(DT[qt])), (t, m)
            else:
                assert torch.equal(kv[m][pid, :, slot], x[m, t]) and torch.equal(back[m, t], x[m, t]), (t, m)
    for m in range(2):                               # no other slot was written
        raw = kv[m].view(torch.uint8) if kvt == "e4m3" else kv[m]
        assert bool((raw.transpose(1, 2)[lone.to(dev)] == 0).all())
        if kvt in TOP:
            assert bool((kv[2 + m].transpose(1, 2)[lone.to(dev)] == -1.0).all())
