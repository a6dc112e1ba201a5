"""ctypes binding of libsffn.so: argument marshalling only, every computation runs in the HIP library.

Names and argument order follow include/sffn.h. Tensors are torch tensors on the GPU (device pointers are
taken with ``data_ptr()``); the stream is torch's current stream unless one is given.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

HERE = os.path.dirname(os.path.abspath(__file__))
# SFFN_LIB_PATH selects another build of the same library (the host-sanitized one of the CPU checks)
LIB_PATH = os.environ.get("SFFN_LIB_PATH") or os.path.join(HERE, "libsffn.so")

ACT_RELU, ACT_REGLU, ACT_SQRELU = 0, 1, 2
ACTS = {"relu": ACT_RELU, "reglu": ACT_REGLU, "sqrelu": ACT_SQRELU}

EXPORTS = ("sffn_status_string", "sffn_last_error", "sffn_workspace_size", "sffn_mask_words", "sffn_predict",
           "sffn_predict_hot", "sffn_forward", "sffn_forward_q4", "sffn_profile_begin", "sffn_profile_end",
           "sffn_forward_path", "sffn_decode", "sffn_decode_path", "sffn_decode_noalloc",
           "sffn_noalloc_scratch_bytes", "sffn_kv_write", "sffn_kv_read", "sffn_attn", "sffn_attn_path",
           "sffn_attn_workspace_size", "sffn_add_rmsnorm", "sffn_quant128", "sffn_mm_e4m3", "sffn_mm_workspace_size",
           "sffn_qk_norm_rope", "sffn_attn_mass", "sffn_attn_mass_workspace_size", "sffn_kv_evict",
           "sffn_kv_evict_workspace_size")
K_PRED_H, K_PRED_Z, K_ROWS, K_COLS = 0, 1, 2, 3


class SffnError(RuntimeError):
    def __init__(self, status: int, where: str, detail: str):
        super().__init__(f"{where}: status {status} ({detail})")
        self.status = status


class _Q4(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("s", ctypes.c_void_p)]


class _KV(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("type", ctypes.c_int), ("n_pages", ctypes.c_int), ("page", ctypes.c_int),
                ("n_kv_heads", ctypes.c_int), ("head_dim", ctypes.c_int)]


class _Seqs(ctypes.Structure):
    _fields_ = [("cu", ctypes.c_void_p), ("kv_len", ctypes.c_void_p), ("table", ctypes.c_void_p), ("S", ctypes.c_int),
                ("T", ctypes.c_int), ("max_pages", ctypes.c_int), ("table_stride", ctypes.c_int)]


_handle = None


def lib() -> ctypes.CDLL:
    """The loaded HIP library; raises if it has not been built (there is no fallback path)."""
    global _handle
    if _handle is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with __graft_entry__.build() "
                               "(the sparse FFN has no non-HIP implementation)")
        h = ctypes.CDLL(LIB_PATH)
        vp, i32, f32, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
        h.sffn_status_string.argtypes, h.sffn_status_string.restype = [i32], ctypes.c_char_p
        h.sffn_last_error.argtypes, h.sffn_last_error.restype = [], ctypes.c_char_p
        h.sffn_workspace_size.argtypes, h.sffn_workspace_size.restype = [i32, i32, i32, i32], sz
        h.sffn_mask_words.argtypes, h.sffn_mask_words.restype = [i32], i32
        h.sffn_predict.argtypes = [vp, vp, vp, vp, i32, i32, i32, i32, i32, f32, vp, vp, vp, sz, vp]
        h.sffn_predict.restype = i32
        h.sffn_predict_hot.argtypes = [vp, vp, vp, vp, i32, i32, i32, i32, i32, f32, i32, vp, vp, vp, sz, vp]
        h.sffn_predict_hot.restype = i32
        h.sffn_forward.argtypes = [i32, vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, vp, vp, vp, vp, vp, sz, vp]
        h.sffn_forward.restype = i32
        h.sffn_forward_q4.argtypes = [i32, _Q4, vp, _Q4, vp, _Q4, vp, i32, i32, i32, i32, vp, vp, vp, vp, vp, sz, vp]
        h.sffn_forward_q4.restype = i32
        h.sffn_decode.argtypes = [i32, vp, vp, vp, f32, i32, vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, vp, vp, vp, vp,
                                  vp, vp, sz, vp]
        h.sffn_decode.restype = i32
        h.sffn_decode_noalloc.argtypes = [i32, vp, vp, vp, f32, i32, vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, vp, vp,
                                          vp, vp, vp, vp]
        h.sffn_decode_noalloc.restype = i32
        h.sffn_noalloc_scratch_bytes.argtypes, h.sffn_noalloc_scratch_bytes.restype = [], sz
        h.sffn_decode_path.argtypes, h.sffn_decode_path.restype = [i32, i32, i32, i32, i32], i32
        h.sffn_profile_begin.argtypes, h.sffn_profile_begin.restype = [i32, i32], i32
        h.sffn_forward_path.argtypes, h.sffn_forward_path.restype = [i32, i32, i32, i32, i32], i32
        h.sffn_profile_end.argtypes, h.sffn_profile_end.restype = [ctypes.POINTER(ctypes.c_float), i32], i32
        i64, f64 = ctypes.c_int64, ctypes.c_double
        h.sffn_kv_write.argtypes, h.sffn_kv_write.restype = [_KV, _Seqs, i32, vp, i64, vp, i64, vp], i32
        h.sffn_kv_read.argtypes, h.sffn_kv_read.restype = [_KV, _Seqs, i32, vp, i64, vp, i64, vp], i32
        h.sffn_attn_path.argtypes, h.sffn_attn_path.restype = [i32] * 4, i32
        h.sffn_attn_workspace_size.argtypes, h.sffn_attn_workspace_size.restype = [i32] * 9, sz
        h.sffn_attn.argtypes = [_KV, _Seqs, i32, vp, i64, i32, i32, i32, f32, i32, i32, vp, i64, vp, vp, sz, vp]
        h.sffn_attn.restype = i32
        h.sffn_add_rmsnorm.argtypes = [i32, vp, i64, i32, vp, i64, vp, f64, i32, i32, i32, vp, i64, vp, vp, i64, vp]
        h.sffn_add_rmsnorm.restype = i32
        h.sffn_quant128.argtypes, h.sffn_quant128.restype = [i32, vp, i64, i32, i32, i32, vp, i64, vp, vp], i32
        h.sffn_mm_workspace_size.argtypes, h.sffn_mm_workspace_size.restype = [i32] * 3, sz
        h.sffn_mm_e4m3.argtypes = [vp, i64, vp, vp, i64, vp, i32, i32, i32, i32, vp, i64, vp, sz, vp]
        h.sffn_mm_e4m3.restype = i32
        h.sffn_qk_norm_rope.argtypes = [i32, vp, vp, i32, i32, vp, i64, i32, vp, i64, i32, i32, i32, vp, vp, f64, vp, i32, i32, vp,
                                        i64, vp, i64, vp]
        h.sffn_qk_norm_rope.restype = i32
        h.sffn_attn_mass_workspace_size.argtypes, h.sffn_attn_mass_workspace_size.restype = [i32] * 7, sz
        h.sffn_attn_mass.argtypes = [_KV, _Seqs, vp, i32, vp, i64, i32, i32, i32, f32, i32, i32, vp, vp, vp, vp, i32, vp, sz, vp]
        h.sffn_attn_mass.restype = i32
        h.sffn_kv_evict_workspace_size.argtypes, h.sffn_kv_evict_workspace_size.restype = [i32] * 4, sz
        h.sffn_kv_evict.argtypes = [_KV, vp, vp, vp, i32, i32, i32, vp, vp, i32, i32, i32, i32, vp, vp, vp, vp, vp, sz, vp]
        h.sffn_kv_evict.restype = i32
        _handle = h
    return _handle


def _p(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _nbytes(t) -> int:
    return t.numel() * t.element_size()


def _stream(stream, ref):
    if stream is not None:
        return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    import torch
    return torch.cuda.current_stream(ref.device).cuda_stream


def _check(rc: int, where: str):
    if rc != 0:
        h = lib()
        raise SffnError(rc, where, f"{h.sffn_status_string(rc).decode()}: {h.sffn_last_error().decode()}")


def status_string(s: int) -> str:
    return lib().sffn_status_string(s).decode()


def workspace_size(B: int, D: int, F: int, r: int) -> int:
    return int(lib().sffn_workspace_size(B, D, F, r))


def mask_words(F: int) -> int:
    return int(lib().sffn_mask_words(F))


def predict(P1, P2, c, x, t: float, mask, ws, logits=None, x_norm: bool = False, stream=None, n_hot: int = 0):
    """sffn_predict (n_hot = 0) or sffn_predict_hot (stored neurons 0 .. n_hot-1 always active). P1 [r, D] fp16,
    P2 [F, r] fp16, c [F] fp32 or None, x [B, D] fp32, mask [ceil(F/64)] int64 (bit pattern), ws uint8
    workspace, logits [B, F] fp32 or None."""
    B, D = x.shape
    F, r = P2.shape
    if n_hot:
        rc = lib().sffn_predict_hot(_p(P1), _p(P2), _p(c), _p(x), int(bool(x_norm)), B, D, F, r, float(t), int(n_hot),
                                    _p(mask), _p(logits), _p(ws), _nbytes(ws), _stream(stream, x))
        _check(rc, "sffn_predict_hot")
        return
    rc = lib().sffn_predict(_p(P1), _p(P2), _p(c), _p(x), int(bool(x_norm)), B, D, F, r, float(t), _p(mask), _p(logits),
                            _p(ws), _nbytes(ws), _stream(stream, x))
    _check(rc, "sffn_predict")


def forward(act, W_gate, b_gate, W_up, b_up, W_downT, x, mask, active, n_active, y, ws, x_norm: bool = False,
            stream=None):
    """sffn_forward. W_gate/W_up/W_downT [F, D] fp16 in stored order, biases [F] fp32 or None,
    active [F] int32 and n_active [1] int32 outputs, y [B, D] fp32 output."""
    B, D = x.shape
    F = W_up.shape[0]
    rc = lib().sffn_forward(ACTS.get(act, act), _p(W_gate), _p(b_gate), _p(W_up), _p(b_up), _p(W_downT), _p(x),
                            int(bool(x_norm)), B, D, F, _p(mask), _p(active), _p(n_active), _p(y), _p(ws), _nbytes(ws),
                            _stream(stream, x))
    _check(rc, "sffn_forward")


def forward_q4(act, W_gate, b_gate, W_up, b_up, W_downT, x, mask, active, n_active, y, ws, x_norm: bool = False,
               stream=None):
    """sffn_forward_q4. Each W is a pair (q [F, D/2] uint8, s [F, D/32] fp16) or None (W_gate for ReLU)."""
    B, D = x.shape
    F = W_up[0].shape[0]
    g = _Q4(*(map(_p, W_gate))) if W_gate is not None else _Q4(None, None)
    rc = lib().sffn_forward_q4(ACTS.get(act, act), g, _p(b_gate), _Q4(*map(_p, W_up)), _p(b_up),
                               _Q4(*map(_p, W_downT)), _p(x), int(bool(x_norm)), B, D, F, _p(mask), _p(active),
                               _p(n_active), _p(y), _p(ws), _nbytes(ws), _stream(stream, x))
    _check(rc, "sffn_forward_q4")


def decode(act, P1, P2, c, t: float, W_gate, b_gate, W_up, b_up, W_downT, x, mask, active, n_active, y, ws,
           x_norm: bool = False, n_hot: int = 0, logits=None, stream=None):
    """sffn_decode: predictor and sparse FFN of one layer for one token (x [1, D]); fp16 weights as in forward."""
    B, D = x.shape
    F, r = P2.shape
    rc = lib().sffn_decode(ACTS.get(act, act), _p(P1), _p(P2), _p(c), float(t), int(n_hot), _p(W_gate), _p(b_gate),
                           _p(W_up), _p(b_up), _p(W_downT), _p(x), int(bool(x_norm)), D, F, r, _p(mask), _p(active),
                           _p(n_active), _p(y), _p(logits), _p(ws), _nbytes(ws), _stream(stream, x))
    _check(rc, "sffn_decode")


def decode_noalloc(act, P1, P2, c, t: float, W_gate, b_gate, W_up, b_up, W_downT, x, mask, active, n_active, y,
                   x_norm: bool = False, n_hot: int = 0, logits=None, stream=None):
    """sffn_decode_noalloc: sffn_decode with the library's own per-GPU device scratch as its workspace (no
    allocation; calls that overlap in time on one GPU race on the scratch)."""
    B, D = x.shape
    F, r = P2.shape
    rc = lib().sffn_decode_noalloc(ACTS.get(act, act), _p(P1), _p(P2), _p(c), float(t), int(n_hot), _p(W_gate),
                                   _p(b_gate), _p(W_up), _p(b_up), _p(W_downT), _p(x), int(bool(x_norm)), D, F, r,
                                   _p(mask), _p(active), _p(n_active), _p(y), _p(logits), _stream(stream, x))
    _check(rc, "sffn_decode_noalloc")


def noalloc_scratch_bytes() -> int:
    return int(lib().sffn_noalloc_scratch_bytes())


DECODE_SEPARATE, DECODE_FOLDED = 0, 1


def decode_path(act, q4: bool, D: int, F: int, r: int) -> int:
    """Which kernels sffn_decode runs for these sizes: DECODE_FOLDED (h, then the predictor's second stage inside
    the fused gather, then the sum of partials) or DECODE_SEPARATE (the sffn_predict and sffn_forward calls)."""
    return int(lib().sffn_decode_path(ACTS.get(act, act), int(bool(q4)), D, F, r))


PATH_DECODE, PATH_FUSED, PATH_UNION = 0, 1, 2


def forward_path(act, q4: bool, B: int, D: int, F: int) -> int:
    """Which kernels a forward call of these sizes runs (PATH_DECODE, PATH_FUSED or PATH_UNION)."""
    return int(lib().sffn_forward_path(ACTS.get(act, act), int(bool(q4)), B, D, F))


def profile_begin(kernel: int, max_launches: int):
    """Time every launch of `kernel` (K_PRED_H, K_PRED_Z, K_ROWS, K_COLS) with the kernel's own device timestamps
    (eager launches only)."""
    _check(lib().sffn_profile_begin(int(kernel), int(max_launches)), "sffn_profile_begin")


def _profile_times(fn, name, max_launches):
    buf = (ctypes.c_float * max(1, max_launches))()
    n = fn(buf, max_launches)
    if n < 0:
        _check(-n, name)
    return [float(buf[i]) for i in range(min(n, max_launches))]


def profile_end(max_launches: int):
    """Per-launch elapsed milliseconds of the bracketed launches (list of floats); frees the events."""
    return _profile_times(lib().sffn_profile_end, "sffn_profile_end", max_launches)


# ------------------------------------------------------------- residual norm, paged K/V cache, attention over it
# These go through the C++ binding _bind.so (csrc/bind.cpp), which takes types, sizes and strides from the tensors and
# checks what the C entry points cannot see: devices, dtypes and layouts. A bad argument raises ValueError, one that the
# library turns away SffnError, before anything is enqueued. Work goes to the current stream of the tensors' own
# device, whichever device is current.
_bound = None


def _fast():
    """The C++ binding, given the loaded library's entry points."""
    global _bound
    if _bound is None:
        import torch  # noqa: F401  (its libraries have to be loaded first)
        from . import _bind
        h = lib()
        _bind.bind(*(ctypes.cast(getattr(h, n), ctypes.c_void_p).value
                     for n in ("sffn_kv_write", "sffn_kv_read", "sffn_attn", "sffn_add_rmsnorm", "sffn_quant128",
                               "sffn_mm_e4m3", "sffn_qk_norm_rope", "sffn_attn_mass", "sffn_kv_evict")))
        _bound = _bind
    return _bound


def _handle_of(stream):
    return stream if stream is None or isinstance(stream, int) else stream.cuda_stream


def kv_write(k, v, kv, cu, kv_len, table, stream=None):
    """sffn_kv_write: new tokens' K and V [T, heads, head size] (fp16 or bf16, any token stride that is a multiple of
    8) into the paged cache kv = (K, V) of the same type, or (K, V, K_scale, V_scale) in int8 or float8_e4m3fn.
    K, V [pages, heads, page, head size]; scales [pages, heads, page] fp32. cu [S + 1], kv_len [S] (with the new
    tokens) and table [S, max_pages] int32 name the places."""
    rc = (_bound or _fast()).kv_write(k, v, kv, cu, kv_len, table, _handle_of(stream))
    if rc:
        _check(rc, "sffn_kv_write")


def kv_read(kv, cu, kv_len, table, k, v, stream=None):
    """sffn_kv_read: the newest cu[s + 1] - cu[s] cached tokens of every sequence into k, v [T, heads, head size]."""
    rc = (_bound or _fast()).kv_read(k, v, kv, cu, kv_len, table, _handle_of(stream))
    if rc:
        _check(rc, "sffn_kv_read")


ATTN_FEW, ATTN_MANY = 0, 1


def attn_path(Hq: int, n_kv_heads: int, head_dim: int, max_q: int) -> int:
    """Which kernel sffn_attn runs for these sizes (ATTN_FEW or ATTN_MANY; -1 for bad sizes)."""
    return int(lib().sffn_attn_path(Hq, n_kv_heads, head_dim, max_q))


def attn_workspace_size(T: int, S: int, Hq: int, n_kv_heads: int, head_dim: int, max_q: int, max_kv: int,
                        window: int = 0, sinks: int = 0) -> int:
    """Bytes of workspace that attn needs for these sizes (0: none)."""
    return int(lib().sffn_attn_workspace_size(T, S, Hq, n_kv_heads, head_dim, max_q, max_kv, window, sinks))


def attn(q, kv, cu, kv_len, table, max_q: int, max_kv: int, out, ws, scale: Optional[float] = None, window: int = 0,
         sinks: int = 0, lse=None, stream=None):
    """sffn_attn: attention of the new tokens q [T, Hq, head size] (fp16 or bf16) over the cache (see kv_write), causal,
    with an optional window and always-visible first tokens. out as q; lse [T, Hq] fp32 or None; ws a uint8 tensor of
    attn_workspace_size bytes (or None if that is 0); scale: 1 / sqrt(head size) unless given."""
    rc = (_bound or _fast()).attn(q, kv, cu, kv_len, table, max_q, max_kv, out, ws, scale, window, sinks, lse,
                                  _handle_of(stream))
    if rc:
        _check(rc, "sffn_attn")


def add_rmsnorm(x, res, w, eps: float, y, res_out=None, y_scale=None, stream=None):
    """sffn_add_rmsnorm: h = x + res, res_out = h, y = h / sqrt(mean(h^2) + eps) * w for rows of [T, D]. x, res (None:
    0) and res_out (None, or as res, also res itself) fp32, fp16 or bf16; w [D] fp32 or None (1); y any of these or
    int8 / float8_e4m3fn with y_scale [T] fp32."""
    rc = (_bound or _fast()).add_rmsnorm(x, res, w, eps, y, res_out, y_scale, _handle_of(stream))
    if rc:
        _check(rc, "sffn_add_rmsnorm")


# ------------------------------------------------------------- 8-bit products, head norms with rotation, eviction
def quant128(x, y, scale, rows: int = 1, stream=None):
    """sffn_quant128: x [T, D] fp32, fp16 or bf16 as codes y [T, D] float8_e4m3fn with one scale for each block of `rows` (1:
    activations, 128: weights) x 128 columns, scale [ceil(T / rows), ceil(D / 128)] fp32."""
    rc = (_bound or _fast()).quant128(x, y, scale, rows, _handle_of(stream))
    if rc:
        _check(rc, "sffn_quant128")


def mm_workspace_size(T: int, N: int, K: int) -> int:
    """Bytes of workspace that mm_e4m3 needs for these sizes (0: none)."""
    return int(lib().sffn_mm_workspace_size(T, N, K))


def mm_e4m3(a, a_scale, b, b_scale, out, ws=None, stream=None):
    """sffn_mm_e4m3: out [T, N] = a [T, K] b [N, K]^T for float8_e4m3fn codes with scales of blocks of 128 columns of a row
    (a_scale [T, ceil(K / 128)]) and of 128 x 128 (b_scale [ceil(N / 128), ceil(K / 128)]); out fp32, fp16 or bf16; ws a uint8
    tensor of mm_workspace_size bytes (or None if that is 0)."""
    rc = (_bound or _fast()).mm_e4m3(a, a_scale, b, b_scale, out, ws, _handle_of(stream))
    if rc:
        _check(rc, "sffn_mm_e4m3")


def qk_norm_rope(q, k, w_q, w_k, eps: Optional[float], cu, seq_len, freq, q_out, k_out, interleaved: bool = False, stream=None):
    """sffn_qk_norm_rope: norms of every head of q [T, Hq, head size] and k [T, K/V heads, head size] (eps None: no norm; w_q,
    w_k [head size] fp32 or None: 1), then the rotation of the first 2 * len(freq) elements (freq None: none) by positions
    seq_len[s] - n + i, in halves or in neighbouring pairs. k and k_out may be None; q_out may be q, k_out k."""
    rc = (_bound or _fast()).qk_norm_rope(q, k, w_q, w_k, eps, cu, seq_len, freq, q_out, k_out, interleaved, _handle_of(stream))
    if rc:
        _check(rc, "sffn_qk_norm_rope")


def attn_mass_workspace_size(S: int, Hq: int, n_kv_heads: int, head_dim: int, max_q: int, max_kv: int, W: int) -> int:
    """Bytes of workspace that attn_mass needs for these sizes (0: none)."""
    return int(lib().sffn_attn_mass_workspace_size(S, Hq, n_kv_heads, head_dim, max_q, max_kv, W))


def attn_mass(q, kv, cu, kv_len, table, max_q: int, max_kv: int, lse, mass, pos, ws=None, seq_len=None, mass_out=None,
              scale: Optional[float] = None, window: int = 0, sinks: int = 0, stream=None):
    """sffn_attn_mass: the attention weight that every cached token got in the attn call with these arguments (lse as it wrote
    it), added to mass [S, K/V heads, slots] fp32 (mass_out None: in place); new tokens begin at 0 and enter their positions in
    pos (int32, same sizes), counted by seq_len [S] (None: kv_len)."""
    rc = (_bound or _fast()).attn_mass(q, kv, cu, kv_len, table, max_q, max_kv, lse, mass, pos, ws, seq_len, mass_out, scale,
                                       window, sinks, _handle_of(stream))
    if rc:
        _check(rc, "sffn_attn_mass")


def kv_evict_workspace_size(S: int, n_kv_heads: int, W: int, keep: int) -> int:
    """Bytes of workspace that kv_evict needs for these sizes."""
    return int(lib().sffn_kv_evict_workspace_size(S, n_kv_heads, W, keep))


def kv_evict(kv, kv_len, table, mass, pos, keep: int, src, ws, seq_len=None, sinks: int = 0, recent: int = 0, kv_len_out=None,
             mass_out=None, pos_out=None, stream=None):
    """sffn_kv_evict: cuts every sequence with more than `keep` cached tokens down to them: those at positions below `sinks` or
    among the last `recent` (of seq_len tokens; None: kv_len), then those with the largest mass. src [S, K/V heads, keep] int32
    tells which slot each came from. kv_len_out, mass_out, pos_out None: in place. seq_len or kv_len_out has to be given: with both
    left out the cached length would overwrite the sequence's own, which is refused."""
    rc = (_bound or _fast()).kv_evict(kv, kv_len, table, mass, pos, keep, src, ws, seq_len, sinks, recent, kv_len_out, mass_out,
                                      pos_out, _handle_of(stream))
    if rc:
        _check(rc, "sffn_kv_evict")
