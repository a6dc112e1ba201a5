"""Each check of the C++ binding by its own message (types, shapes, layouts, devices: what stands between a wrong tensor and
a raw pointer). CPU tensors throughout, so a call that passes every check is refused last, for being off the GPU."""
import re

import pytest
import torch

from activation_sparse_ffn_predictor_amd import _lib

H, I32 = torch.float16, torch.int32
KV = (torch.zeros((4, 2, 16, 64), dtype=H), torch.zeros((4, 2, 16, 64), dtype=H))
KV8 = tuple(t.to(torch.int8) for t in KV)
SC = torch.zeros((4, 2, 16))
CU, KL, TAB = torch.tensor([0, 1, 3], dtype=I32), torch.tensor([4, 5], dtype=I32), torch.zeros((2, 3), dtype=I32)
K = torch.zeros((3, 2, 64), dtype=H)
Q, O = torch.zeros((3, 8, 64), dtype=H), torch.zeros((3, 8, 64), dtype=H)
X, Y = torch.zeros((3, 64)), torch.zeros((3, 64))
LAST = "the tensors must be on the GPU"


def write(k=K, v=K, c=KV, cu=CU, kl=KL, tab=TAB, **kw):
    _lib.kv_write(k, v, c, cu, kl, tab, **kw)


def read(k=K, v=K, c=KV, cu=CU, kl=KL, tab=TAB):
    _lib.kv_read(c, cu, kl, tab, k, v)


def attn(q=Q, o=O, c=KV, cu=CU, kl=KL, tab=TAB, ws=None, max_q=2, max_kv=5, **kw):
    _lib.attn(q, c, cu, kl, tab, max_q, max_kv, o, ws, **kw)


def norm(x=X, r=None, w=None, y=Y, eps=1e-5, **kw):
    _lib.add_rmsnorm(x, r, w, eps, y, **kw)


META = torch.device("meta")
CACHES = [
    (dict(c=KV[0]), "the cache is a tuple"), (dict(c=KV[:1]), "the cache is a tuple"), (dict(c=KV + (SC,)), "the cache is a tuple"),
    (dict(c=(KV[0], None)), "V is not a tensor"), (dict(c=tuple(t.double() for t in KV)), "K: this type is not supported here"),
    (dict(c=tuple(t.float() for t in KV)), "K: this type is not supported here"),
    (dict(c=(KV[0], KV[1][:2])), "K and V are contiguous"), (dict(c=(KV[0], KV[1].bfloat16())), "K and V are contiguous"),
    (dict(c=tuple(t.transpose(1, 2) for t in KV)), "K and V are contiguous"), (dict(c=tuple(t[0] for t in KV)), "K and V are contiguous"),
    (dict(c=KV8), "an 8-bit cache needs contiguous fp32 scales"), (dict(c=KV8 + (SC, None)), "an 8-bit cache needs contiguous fp32 scales"),
    (dict(c=KV8 + (SC.half(), SC)), "an 8-bit cache needs contiguous fp32 scales"),
    (dict(c=KV8 + (SC, SC[:2])), "an 8-bit cache needs contiguous fp32 scales"),
    (dict(c=KV8 + (SC.transpose(0, 2).contiguous().transpose(0, 2), SC)), "an 8-bit cache needs contiguous fp32 scales"),
    (dict(c=KV8 + (SC, SC.to(META))), "the tensors are on different devices"), (dict(c=(KV[0], KV[1].to(META))), "the tensors are on different devices"),
]
SEQS = [
    (dict(cu=[0, 1, 3]), "cu is not a tensor"), (dict(kl=None), "kv_len is not a tensor"), (dict(tab=3), "table is not a tensor"),
    (dict(cu=CU.long()), "cu, kv_len and table are int32"), (dict(kl=KL.float()), "cu, kv_len and table are int32"),
    (dict(tab=TAB.short()), "cu, kv_len and table are int32"), (dict(cu=CU[:2]), "need cu [S + 1], kv_len [S], table [S, max_pages]"),
    (dict(tab=TAB[:1]), "need cu [S + 1], kv_len [S], table [S, max_pages]"), (dict(tab=TAB[0]), "need cu [S + 1], kv_len [S], table [S, max_pages]"),
    (dict(kl=KL[:, None]), "need cu [S + 1], kv_len [S], table [S, max_pages]"),
    (dict(cu=torch.zeros(6, dtype=I32)[::2]), "cu, kv_len and the rows of table must be dense"),
    (dict(kl=torch.zeros(4, dtype=I32)[::2]), "cu, kv_len and the rows of table must be dense"),
    (dict(tab=torch.zeros((3, 2), dtype=I32).t()), "cu, kv_len and the rows of table must be dense"),
    (dict(cu=CU.to(META)), "the tensors are on different devices"), (dict(kl=KL.to(META)), "the tensors are on different devices"),
    (dict(tab=TAB.to(META)), "the tensors are on different devices"),
]
ROWS = [
    (dict(k=None), "k is not a tensor"), (dict(v=1.0), "v is not a tensor"), (dict(k=K.float(), v=K.float()), "k: this type is not supported here"),
    (dict(k=K.to(torch.int8), v=K.to(torch.int8)), "k: this type is not supported here"), (dict(v=K.bfloat16()), "k and v differ in type or shape"),
    (dict(k=K[:2]), "k and v differ in type or shape"), (dict(k=K[:, :1], v=K[:, :1]), "k is not [tokens, 2, 64]"),
    (dict(k=K[..., :32], v=K[..., :32]), "k is not [tokens, 2, 64]"), (dict(k=K.flatten(1), v=K.flatten(1)), "k is not [tokens, 2, 64]"),
    (dict(k=torch.zeros((3, 2, 128), dtype=H)[:, :, ::2]), "k: the heads of a token must be dense"),
    (dict(v=torch.zeros((3, 4, 64), dtype=H)[:, ::2]), "v: the heads of a token must be dense"),
    (dict(k=torch.zeros((3, 64, 2), dtype=H).transpose(1, 2)), "k: the heads of a token must be dense"),
    (dict(k=K.to(META)), "the tensors are on different devices"), (dict(v=K.to(META)), "the tensors are on different devices"),
    (dict(), LAST), (dict(c=KV8 + (SC, SC)), LAST),
]
ATTN = [
    (dict(q=None), "q is not a tensor"), (dict(o=7), "out is not a tensor"), (dict(ws=b""), "ws is not a tensor"), (dict(lse=1), "lse is not a tensor"),
    (dict(q=Q.float(), o=O.float()), "q: this type is not supported here"), (dict(o=O.bfloat16()), "q and out are [tokens, heads, head size] of one type"),
    (dict(o=O[:2]), "q and out are [tokens, heads, head size] of one type"), (dict(q=Q[0], o=O[0]), "q and out are [tokens, heads, head size] of one type"),
    (dict(q=Q[..., :32], o=O[..., :32]), "q is not [tokens, 8, 64]"),
    (dict(q=torch.zeros((3, 8, 128), dtype=H)[..., ::2]), "q: the heads of a token must be dense"),
    (dict(o=torch.zeros((3, 16, 64), dtype=H)[:, ::2]), "out: the heads of a token must be dense"),
    (dict(lse=torch.zeros((3, 7))), "lse is contiguous fp32 [tokens, heads]"), (dict(lse=torch.zeros((3, 8), dtype=H)), "lse is contiguous fp32 [tokens, heads]"),
    (dict(lse=torch.zeros((8, 3)).t()), "lse is contiguous fp32 [tokens, heads]"), (dict(lse=torch.zeros(24)), "lse is contiguous fp32 [tokens, heads]"),
    (dict(ws=torch.zeros(512, dtype=torch.uint8)[::2]), "the workspace must be contiguous"),
    (dict(lse=torch.zeros((3, 8), device=META)), "the tensors are on different devices"), (dict(o=O.to(META)), "the tensors are on different devices"),
    (dict(q=Q.to(META)), "the tensors are on different devices"), (dict(ws=torch.zeros(8, device=META)), "the tensors are on different devices"),
    (dict(), LAST), (dict(lse=torch.zeros((3, 8)), ws=torch.zeros(256, dtype=torch.uint8), window=3, sinks=1, scale=0.5), LAST),
]
NORM = [
    (dict(x=None), "x is not a tensor"), (dict(y=None), "y is not a tensor"), (dict(x=Q, y=O), "x is [tokens, D]"), (dict(x=X[0]), "x is [tokens, D]"),
    (dict(x=X.double()), "x: this type is not supported here"), (dict(x=X.to(torch.int8)), "x: this type is not supported here"),
    (dict(y=Y.long()), "y: this type is not supported here"), (dict(r=X.to(torch.int8)), "res: this type is not supported here"),
    (dict(res_out=X.double()), "res_out: this type is not supported here"), (dict(r=X, res_out=Y.half()), "res and res_out differ in type"),
    (dict(x=torch.zeros((3, 128))[:, ::2]), "x is not [3, 64] with dense rows"), (dict(y=Y[:2]), "y is not [3, 64] with dense rows"),
    (dict(y=torch.zeros((64, 3)).t()), "y is not [3, 64] with dense rows"), (dict(r=X[:, :32]), "res is not [3, 64] with dense rows"),
    (dict(res_out=X[:2]), "res_out is not [3, 64] with dense rows"), (dict(w=torch.zeros(63)), "w is contiguous fp32 [D]"),
    (dict(w=torch.zeros(64, dtype=H)), "w is contiguous fp32 [D]"), (dict(w=torch.zeros((1, 64))), "w is contiguous fp32 [D]"),
    (dict(w=torch.zeros(128)[::2]), "w is contiguous fp32 [D]"), (dict(y=Y.to(torch.int8)), "an 8-bit y needs y_scale"),
    (dict(y=Y.to(torch.int8), y_scale=torch.zeros(2)), "an 8-bit y needs y_scale"), (dict(y=Y.to(torch.int8), y_scale=torch.zeros(3, dtype=H)), "an 8-bit y needs y_scale"),
    (dict(y=Y.to(torch.int8), y_scale=torch.zeros(6)[::2]), "an 8-bit y needs y_scale"), (dict(y=Y.to(META)), "the tensors are on different devices"),
    (dict(w=torch.zeros(64, device=META)), "the tensors are on different devices"), (dict(r=X.to(META)), "the tensors are on different devices"),
    (dict(res_out=X.to(META)), "the tensors are on different devices"),
    (dict(y=Y.to(torch.int8), y_scale=torch.zeros(3, device=META)), "the tensors are on different devices"),
    (dict(), LAST), (dict(r=X.half(), w=torch.zeros(64), res_out=X.half(), y=Y.to(torch.float8_e4m3fn), y_scale=torch.zeros(3)), LAST),
]
CASES = [(f, n, *c) for f, n, cs in ((write, "sffn_kv_write", CACHES + SEQS + ROWS), (read, "sffn_kv_read", CACHES + SEQS + ROWS),
                                     (attn, "sffn_attn", CACHES + SEQS + ATTN), (norm, "sffn_add_rmsnorm", NORM)) for c in cs]


@pytest.mark.parametrize("i", range(len(CASES)))
def test_refused_for_its_reason(i):
    call, name, kw, text = CASES[i]
    with pytest.raises(ValueError, match="^" + re.escape(f"{name}: {text}")):
        call(**kw)


def test_numbers_that_are_none():
    for kw in (dict(max_q="2"), dict(max_kv=None), dict(window=1.5), dict(sinks=[]), dict(scale="x")):
        with pytest.raises(TypeError):
            attn(**kw)
    with pytest.raises(TypeError):
        norm(eps="small")
    with pytest.raises(OverflowError):
        attn(max_kv=1 << 70)
