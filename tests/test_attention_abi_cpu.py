"""Refusals of the cache, attention and norm entry points: bad arguments are turned away on the host before anything is
enqueued (fake pointers that are never followed), and the binding checks what the C ABI cannot see. No GPU."""
import math
import os
import subprocess
import sys

import pytest
import torch

from activation_sparse_ffn_predictor_amd import _lib

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A = 0x10000
KV = dict(k=A, v=A, k_scale=A, v_scale=A, type=1, n_pages=4, page=16, n_kv_heads=2, head_dim=64)
SQ = dict(cu=A, kv_len=A, table=A, S=2, T=5, max_pages=3, table_stride=3)


def kv(**kw):
    return _lib._KV(**{**KV, **kw})


def sq(**kw):
    return _lib._Seqs(**{**SQ, **kw})


def attn(c=None, s=None, **kw):
    a = dict(type=1, q=A, q_stride=512, Hq=8, max_q=4, max_kv=40, scale=0.1, window=0, sinks=0, out=A, out_stride=512,
             lse=None, ws=None, ws_bytes=0, stream=None)
    a.update(kw)
    return _lib.lib().sffn_attn(c or kv(), s or sq(), *a.values())


def move(fn, c=None, s=None, **kw):
    a = dict(type=1, k=A, k_stride=128, v=A, v_stride=128, stream=None)
    a.update(kw)
    return getattr(_lib.lib(), fn)(c or kv(), s or sq(), *a.values())


CACHE_BAD = [(dict(k=None), 1), (dict(v=None), 1), (dict(type=3, k_scale=None), 1), (dict(type=4, v_scale=None), 1),
             (dict(type=0), 6), (dict(type=2), 6), (dict(type=9), 6), (dict(head_dim=8), 2), (dict(head_dim=60), 2),
             (dict(head_dim=264), 2), (dict(type=3, head_dim=72), 2), (dict(page=8), 2), (dict(page=24), 2),
             (dict(page=2048), 2), (dict(n_pages=0), 2), (dict(n_kv_heads=0), 2),
             (dict(n_pages=1 << 20, n_kv_heads=128), 2), (dict(n_kv_heads=1 << 17), 2), (dict(k=A + 8), 3),
             (dict(type=3, k_scale=A + 4), 3)]
SEQ_BAD = [(dict(cu=None), 1), (dict(kv_len=None), 1), (dict(table=None), 1), (dict(S=0), 2), (dict(S=65536), 2),
           (dict(T=-1), 2), (dict(T=(1 << 24) + 1), 2), (dict(max_pages=0), 2), (dict(max_pages=1 << 27, table_stride=1 << 27), 2),
           (dict(table_stride=2), 2), (dict(cu=A + 2), 3)]


@pytest.mark.parametrize("fn", ["sffn_kv_write", "sffn_kv_read"])
def test_write_and_read_reject(fn):
    for kw, st in CACHE_BAD:
        assert move(fn, c=kv(**kw)) == st, kw
        assert _lib.lib().sffn_last_error().decode() != ""
    for kw, st in SEQ_BAD:
        assert move(fn, s=sq(**kw)) == st, kw
    for kw, st in [(dict(type=0), 6), (dict(type=3), 6), (dict(k=None), 1), (dict(v=None), 1), (dict(k_stride=120), 2),
                   (dict(v_stride=132), 2), (dict(k_stride=-128), 2), (dict(k=A + 8), 3), (dict(v=A + 2), 3)]:
        assert move(fn, **kw) == st, kw
    assert move(fn, s=sq(T=0), k=None, v=None) == 0           # nothing to do
    assert _lib.lib().sffn_last_error().decode() == ""


def test_attn_rejects():
    for kw, st in CACHE_BAD:
        assert attn(c=kv(**kw)) == st, kw
    for kw, st in SEQ_BAD:
        assert attn(s=sq(**kw)) == st, kw
    for kw, st in [(dict(type=0), 6), (dict(Hq=7), 2), (dict(Hq=1), 2), (dict(Hq=0), 2), (dict(max_q=0), 2),
                   (dict(scale=math.nan), 6), (dict(scale=math.inf), 6), (dict(window=-1), 6), (dict(sinks=-1), 6),
                   (dict(q=None), 1), (dict(out=None), 1), (dict(q_stride=504), 2), (dict(out_stride=516), 2),
                   (dict(q=A + 2), 3), (dict(out=A + 8), 3), (dict(lse=A + 2), 3)]:
        assert attn(**kw) == st, kw
    long = dict(max_kv=4096)                                  # spread: a workspace is needed
    assert attn(**long) == 1 and attn(ws=A + 16, ws_bytes=1 << 30, **long) == 3 and attn(ws=A, ws_bytes=64, **long) == 4
    assert attn(s=sq(T=1 << 24), c=kv(n_kv_heads=2), Hq=256, q_stride=1 << 14, out_stride=1 << 14) == 2
    assert attn(s=sq(T=0), q=None, out=None) == 0


def test_attn_sizes():
    f, ws = _lib.attn_path, _lib.attn_workspace_size
    assert f(64, 8, 128, 1) == _lib.ATTN_FEW and f(64, 8, 128, 4) == _lib.ATTN_FEW
    assert f(64, 8, 128, 5) == _lib.ATTN_MANY
    assert f(64, 8, 256, 2) == _lib.ATTN_FEW and f(64, 8, 256, 3) == _lib.ATTN_MANY
    assert f(7, 2, 128, 1) == -1 and f(8, 8, 12, 1) == -1 and f(8, 0, 64, 1) == -1 and f(8, 8, 64, 0) == -1
    assert ws(64, 64, 64, 32, 128, 1, 100) == 0               # enough sequences: no parts
    a = ws(1, 1, 64, 8, 128, 1, 131072)
    assert a > 0 and a % 256 == 0
    assert ws(1, 1, 64, 8, 128, 1, 131072, 100, 4) < a        # a window: fewer keys, fewer parts
    assert ws(4, 4, 64, 8, 128, 4, 4096) == ws(4, 4, 64, 8, 128, 400, 4096)   # max_q counts up to T
    assert ws(0, 1, 8, 8, 64, 1, 10) == 0 and ws(1, 1, 8, 3, 64, 1, 10) == 0 and ws(1, 1, 8, 8, 64, 1, 10, -1) == 0


def test_launch_limits():
    """More threads than one launch holds: refused, or (partial results of that many rows) not asked for."""
    wide = dict(n_kv_heads=64, head_dim=256)
    for fn in ("sffn_kv_write", "sffn_kv_read"):
        assert move(fn, c=kv(**wide), s=sq(T=1 << 24), k_stride=64 * 256, v_stride=64 * 256) == 2
        assert "too many" in _lib.lib().sffn_last_error().decode()
    assert attn(c=kv(n_kv_heads=126, head_dim=16), s=sq(T=1 << 24, S=65535), Hq=126, max_q=1 << 20, q_stride=126 * 16,
                out_stride=126 * 16) == 2
    assert "too many" in _lib.lib().sffn_last_error().decode()
    assert _lib.attn_workspace_size(1 << 17, 1, 64, 8, 128, 1, 131072) > 0
    assert _lib.attn_workspace_size(1 << 18, 1, 64, 8, 128, 1, 131072) == 0


def norm(**kw):
    a = dict(xt=0, x=A, ldx=64, rt=0, res=2 * A, ldr=64, w=A, eps=1e-5, T=3, D=64, yt=1, y=3 * A, ldy=64, ys=None, ro=None,
             ldro=0, stream=None)
    a.update(kw)
    return _lib.lib().sffn_add_rmsnorm(*a.values())


@pytest.mark.parametrize("kw,st", [
    (dict(xt=3), 6), (dict(rt=4), 6), (dict(yt=5), 6), (dict(T=-1), 2), (dict(T=(1 << 24) + 1), 2), (dict(D=4), 2),
    (dict(D=60), 2), (dict(D=16392), 2), (dict(eps=-1.0), 6), (dict(eps=math.nan), 6), (dict(eps=math.inf), 6),
    (dict(x=None), 1), (dict(y=None), 1), (dict(ldx=56), 2), (dict(ldr=68), 2), (dict(ldy=60), 2), (dict(yt=3), 1),
    (dict(x=A + 4), 3), (dict(res=A + 4), 3), (dict(y=3 * A + 8), 3), (dict(w=A + 4), 3), (dict(yt=3, ys=A + 2), 3),
    (dict(y=A), 6), (dict(y=2 * A), 6), (dict(ro=3 * A, ldro=64), 6), (dict(ro=A, ldro=64), 6), (dict(ro=2 * A, ldro=72), 6), (dict(ro=4 * A, ldro=8), 2),
    (dict(T=0, x=None, y=None), 0)])
def test_norm_rejects(kw, st):
    assert norm(**kw) == st


def test_binding_rejects():
    """Types, shapes, layouts and devices are checked before the library is called (CPU tensors would be refused last)."""
    h = torch.float16
    c = (torch.zeros((4, 2, 16, 64), dtype=h), torch.zeros((4, 2, 16, 64), dtype=h))
    cu, kl, tab = torch.tensor([0, 1, 3], dtype=torch.int32), torch.tensor([4, 5], dtype=torch.int32), torch.zeros((2, 3), dtype=torch.int32)
    k = torch.zeros((3, 2, 64), dtype=h)
    q, o, ws = torch.zeros((3, 8, 64), dtype=h), torch.zeros((3, 8, 64), dtype=h), torch.zeros(256, dtype=torch.uint8)

    def write(k=k, v=k, c=c, cu=cu, kl=kl, tab=tab):
        _lib.kv_write(k, v, c, cu, kl, tab)

    def attn(q=q, o=o, c=c, cu=cu, kl=kl, tab=tab, **kw):
        _lib.attn(q, c, cu, kl, tab, 2, 5, o, ws, **kw)

    c8 = tuple(t.to(torch.int8) for t in c)
    sc = torch.zeros((4, 2, 16))
    bad = [lambda: write(k=k.float()), lambda: write(k=k[:, :1]), lambda: write(k=k[:2]), lambda: write(k=k.transpose(1, 2)),
           lambda: write(k=torch.zeros((3, 2, 128), dtype=h)[:, :, ::2], v=torch.zeros((3, 2, 128), dtype=h)[:, :, ::2]),
           lambda: write(v=k.bfloat16()), lambda: write(c=(c[0], c[1][:2])), lambda: write(c=(c[0], c[1].bfloat16())),
           lambda: write(c=tuple(t.transpose(1, 2) for t in c)), lambda: write(c=c8), lambda: write(c=c8 + (sc, None)),
           lambda: write(c=c8 + (sc, sc.half())), lambda: write(c=c8 + (sc, sc[:2])), lambda: write(cu=cu.long()),
           lambda: write(cu=cu[:2]), lambda: write(kl=kl.float()), lambda: write(tab=tab[:1]), lambda: write(tab=tab.t()),
           lambda: write(cu=torch.zeros(6, dtype=torch.int32)[::2]), lambda: write(k=k.to("meta"), v=k.to("meta")),
           lambda: attn(q=q.float()), lambda: attn(o=o.bfloat16()), lambda: attn(o=o[:2]), lambda: attn(q=q[0], o=o[0]),
           lambda: attn(lse=torch.zeros((3, 7))), lambda: attn(lse=torch.zeros((3, 8), dtype=h)),
           lambda: attn(q=q[..., :32], o=o[..., :32]), lambda: attn(lse=torch.zeros((3, 8)).to("meta")),
           lambda: _lib.add_rmsnorm(q, None, None, 1e-5, o), lambda: _lib.add_rmsnorm(k[0], None, None, 1e-5, k[1].long()),
           lambda: _lib.add_rmsnorm(k[0], None, k[1, 0], 1e-5, k[1]), lambda: _lib.add_rmsnorm(k[0], k[1, :1], None, 1e-5, k[2]),
           lambda: _lib.add_rmsnorm(k[0], None, None, 1e-5, k[1].to(torch.int8)),
           lambda: _lib.add_rmsnorm(k[0], k[1], None, 1e-5, k[2], res_out=k[2].float()),
           lambda: _lib.add_rmsnorm(k[0].t(), None, None, 1e-5, k[2].t()),
           lambda: write(), lambda: attn(), lambda: _lib.add_rmsnorm(k[0], None, None, 1e-5, k[1])]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            print("accepted:", i)


def test_refusals_under_host_sanitizers():
    """The checks above once more against a library whose host code is instrumented, in a child process."""
    if os.environ.get("SFFN_LIB_PATH"):
        pytest.skip("this is the child")
    if subprocess.run(["which", "hipcc"], capture_output=True).returncode != 0:
        pytest.skip("hipcc is not installed")
    from activation_sparse_ffn_predictor_amd import build_sanitized as bs
    bs.build()
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-p", "no:cacheprovider", os.path.abspath(__file__)],
                       env=bs.sanitizer_env(), cwd=ROOT, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout[-4000:] + r.stderr[-4000:]
    assert "passed" in r.stdout and "AddressSanitizer" not in r.stderr and "runtime error" not in r.stderr
