"""A resident sparse-FFN stack on one GPU: every layer's predictor and weights in HBM, one decode step =
sffn_predict + sffn_forward (or sffn_forward_q4) per layer, layer l+1 reading layer l's output through the
library's normalise-on-load option (a parameter-free LayerNorm). A step can be captured once into a HIP graph and replayed.

The pages' decode touches the whole model for every token (Turkish article, motivation section); the stack
is the FFN part of that, with the neuron order of every layer chosen hot-first (pack.hot_first_perm).

Layers may differ in predictor rank (Turkish article, "Adaptive sparsity predictors": the predictor is sized per
layer), and with ``hot_prefix`` each layer's saturated neurons, stored first, are declared always active so the
predictor reads no rows for them (sffn_predict_hot).

With ``attn`` the layers have both halves: a residual stream in fp32, and before each sparse FFN a residual norm
(sffn_add_rmsnorm), the Q/K/V product, the new tokens' K and V into the layer's paged cache (sffn_kv_write), attention
over it (sffn_attn) and the output product; the FFN reads a second residual norm's output. Every sequence owns a row of
the page table from the start (its pages are reserved for max_len tokens). ``step`` decodes one token of each of the
first B sequences, ``prompt`` enters a chunk of one sequence's tokens (at most max_batch, and at most the 64 that a sparse
FFN call takes). No positions are encoded: queries and keys are used as they are projected, which is not what models with
rotary positions do.
"""
from __future__ import annotations

import contextlib
import dataclasses
import math
from typing import Dict, List, Optional

import numpy as np
import torch

import synthgen as sg

from . import _lib
from .pack import hot_first_perm, pack_layer


KV_TYPES = {"f16": torch.float16, "i8": torch.int8, "e4m3": torch.float8_e4m3fn}
PAGES = tuple(1 << b for b in range(4, 11))


@dataclasses.dataclass(frozen=True)
class AttnConfig:
    """Attention of a stack's layers: head layout, cache type ("f16", "i8" or "e4m3") and room, window and sinks; norms of heads,
    rotary positions (rope_base > 0; of the first rope_dim elements of a head, 0: all), type of the projections' weights ("f16" or
    "e4m3"). keep > 0: a sequence that would grow past max_len is cut down to `keep` cached tokens for each K/V head, the first
    `sinks`, the last `recent` and those with the most attention (no window then: it would count slots)."""
    n_heads: int
    n_kv_heads: int
    head_dim: int
    kv_type: str = "f16"
    page: int = 64
    max_len: int = 4096
    window: int = 0
    sinks: int = 0
    eps: float = 1e-5
    qk_norm: bool = False
    rope_base: float = 0.0
    rope_dim: int = 0
    rope_interleaved: bool = False
    weights: str = "f16"
    keep: int = 0
    recent: int = 0

    def __post_init__(self):
        rot = self.rope_dim or self.head_dim
        if (not (self.rope_base >= 0 and math.isfinite(self.rope_base)) or not 8 <= rot <= self.head_dim or rot % 8
                or self.weights not in ("f16", "e4m3") or not 0 <= self.keep < max(self.max_len, 1) or self.recent < 0
                or (self.keep and (self.window or self.sinks + self.recent > self.keep)) or (self.recent and not self.keep)):
            raise ValueError(f"attention: {self}")
        if (self.kv_type not in KV_TYPES or min(self.max_len, self.n_kv_heads, self.n_heads) < 1
                or self.n_heads % self.n_kv_heads or not 16 <= self.head_dim <= 256
                or self.head_dim % (8 if self.kv_type == "f16" else 16) or self.page not in PAGES
                or min(self.window, self.sinks) < 0 or not (self.eps >= 0 and math.isfinite(self.eps))):
            raise ValueError(f"attention: {self}")


class SparseFFNStack:
    def __init__(self, wl: sg.Workload, device="cuda:0", layers: Optional[List[int]] = None, with_c: bool = True,
                 max_batch: int = 1, seed: int = sg.MASTER_SEED, hot_prefix: bool = False, fold_predictor: bool = True,
                 attn: Optional[AttnConfig] = None):
        self.wl = wl
        self.device = torch.device(device)
        self.layer_ids = list(range(wl.L)) if layers is None else list(layers)
        self.q4 = wl.wdtype == "q4"
        self.with_c = with_c
        self.max_batch = max_batch
        self.fold_predictor = fold_predictor
        self.ranks = [wl.rank(l) for l in self.layer_ids]
        self.n_hot = [sg.saturated_count(wl, l, seed) if hot_prefix else 0 for l in self.layer_ids]
        self.layers: List[Dict[str, torch.Tensor]] = []
        for l in self.layer_ids:
            logical = sg.layer_device(wl, l, self.device, seed=seed, with_c=with_c)
            perm = hot_first_perm(sg.neuron_probs(wl, l, seed))
            self.layers.append(pack_layer(logical, perm))
            del logical
        torch.cuda.synchronize(self.device)
        L, F, D = len(self.layer_ids), wl.F, wl.D
        self.nw = _lib.mask_words(F)
        self.mask = torch.zeros((L, self.nw), dtype=torch.int64, device=self.device)
        self.active = torch.zeros((L, F), dtype=torch.int32, device=self.device)
        self.n_active = torch.zeros((L,), dtype=torch.int32, device=self.device)
        self.y = torch.zeros((L, max_batch, D), dtype=torch.float32, device=self.device)
        # one token needs more than a few (a partial sum of y per workgroup), so the largest need is not max_batch's
        need = max(_lib.workspace_size(b, D, F, max(self.ranks)) for b in range(1, max_batch + 1))
        self.ws = torch.zeros(need, dtype=torch.uint8, device=self.device)
        self.x_in = torch.zeros((max_batch, D), dtype=torch.float32, device=self.device)
        self.graphs = {}
        self.attn = attn
        if attn is not None:
            self._attn_setup(seed)

    # ------------------------------------------------------------------ attention half
    def _attn_setup(self, seed: int):
        """Projections and norm weights (synthetic, normal), caches, page table and buffers of the attention half."""
        c, D, B, dev = self.attn, self.wl.D, self.max_batch, self.device
        width, cols = (c.n_heads + 2 * c.n_kv_heads) * c.head_dim, -(-c.max_len // c.page)
        kt, cache = KV_TYPES[c.kv_type], (B * cols, c.n_kv_heads, c.page, c.head_dim)
        heads, slots, e8 = c.n_heads * c.head_dim, cols * c.page, c.weights == "e4m3"
        if e8 and (D % 16 or heads % 16 or width % 8):
            raise ValueError(f"e4m3 projections: d_model = {D}, heads of {heads} together: need multiples of 16")
        for l, t in zip(self.layer_ids, self.layers):
            g = torch.Generator(device=dev)
            g.manual_seed((seed * 1000003 + l) % (1 << 63))
            t["W_qkv"] = (torch.randn((width, D), generator=g, device=dev) / D ** 0.5).half()
            t["W_o"] = (torch.randn((D, heads), generator=g, device=dev) / heads ** 0.5).half()
            if e8:
                for name in ("W_qkv", "W_o"):
                    t[name] = self._quantised(t[name], 128)
            t["w_attn"], t["w_ffn"] = (1 + 0.1 * torch.randn(D, generator=g, device=dev) for _ in range(2))
            kv = [torch.zeros(cache, device=dev).to(kt) for _ in range(2)]
            if c.kv_type != "f16":
                kv += [torch.zeros(cache[:3], device=dev) for _ in range(2)]
            t["kv"] = tuple(kv)
            if c.qk_norm:
                t["w_q"], t["w_k"] = (1 + 0.1 * torch.randn(c.head_dim, generator=g, device=dev) for _ in range(2))
            if c.keep:
                t["pos"] = torch.zeros((B, c.n_kv_heads, slots), dtype=torch.int32, device=dev)
        if c.keep:
            self.mass = torch.zeros((len(self.layers), B, c.n_kv_heads, slots), device=dev)
            for t, m in zip(self.layers, self.mass):
                t["mass"] = m
        self.w_out = torch.ones(D, device=dev)
        self.table = torch.arange(B * cols, dtype=torch.int32, device=dev).view(B, cols)
        self.kv_len = torch.zeros(B, dtype=torch.int32, device=dev)
        self.lens = [0] * B                                    # the same on the host, to refuse what does not fit
        self.seq_len = torch.zeros(B, dtype=torch.int32, device=dev)   # tokens entered, evicted ones with them
        self.cu_step = torch.arange(B + 1, dtype=torch.int32, device=dev)
        self.cu_prompt = {}
        self.h = torch.zeros((B, D), device=dev)               # residual stream
        self.xn = torch.zeros((B, D), dtype=torch.float16, device=dev)
        self.qkv = torch.zeros((B, width), dtype=torch.float16, device=dev)
        self.o = torch.zeros((B, c.n_heads, c.head_dim), dtype=torch.float16, device=dev)
        self.ao = torch.zeros((B, D), dtype=torch.float16, device=dev)
        self.xf = torch.zeros((B, D), device=dev)
        self.out = torch.zeros((B, D), device=dev)             # the last layer's normalised output
        sizes = [_lib.attn_workspace_size(T, S, c.n_heads, c.n_kv_heads, c.head_dim, T // S, c.max_len, c.window, c.sinks)
                 for T in range(1, B + 1) for S in (1, T)]
        self.ws_attn = torch.zeros(max([256] + sizes), dtype=torch.uint8, device=dev)
        rot = c.rope_dim or c.head_dim
        self.freq = (c.rope_base ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)).float().to(dev) if c.rope_base else None
        if e8:
            self.xq, self.xs = self._quantised(self.xn, 1)
            self.oq, self.os = self._quantised(self.o.flatten(1), 1)
            need = max(_lib.mm_workspace_size(T, *n_k) for T in range(1, B + 1) for n_k in ((width, D), (D, heads)))
            self.ws_mm = torch.zeros(max(256, need), dtype=torch.uint8, device=dev)
        if c.keep:
            self.lse = torch.zeros((B, c.n_heads), device=dev)
            need = max(_lib.attn_mass_workspace_size(S, c.n_heads, c.n_kv_heads, c.head_dim, T // S, c.max_len, slots)
                       for T in range(1, B + 1) for S in (1, T))
            self.ws_mass = torch.zeros(max(256, need), dtype=torch.uint8, device=dev)
            self.ws_evict = torch.zeros(_lib.kv_evict_workspace_size(1, c.n_kv_heads, slots, c.keep), dtype=torch.uint8, device=dev)
            self.src = torch.zeros((1, c.n_kv_heads, c.keep), dtype=torch.int32, device=dev)
            self.no_len, self.cut_len = (torch.zeros(1, dtype=torch.int32, device=dev) for _ in range(2))

    @staticmethod
    def _quantised(x, rows: int):
        """(codes, scales) of x [T, K] in blocks of `rows` x 128."""
        T, K = x.shape
        q = torch.empty((T, K), dtype=torch.float8_e4m3fn, device=x.device)
        s = torch.empty((-(-T // rows), -(-K // 128)), device=x.device)
        _lib.quant128(x, q, s, rows=rows)
        return q, s

    def _project(self, x, xq, xs, w, out):
        """out = x W^T: fp16, or x quantised into xq, xs and 8-bit weights."""
        if self.attn.weights == "f16":
            torch.mm(x, w.t(), out=out)
            return
        _lib.quant128(x, xq, xs)
        _lib.mm_e4m3(xq, xs, *w, out, self.ws_mm)

    def attn_layer(self, i: int, x, B: int, cu, kv_len, table, max_q: int, seq_len=None, rows: slice = slice(0, None)):
        """Attention half of stored layer i for B tokens: x (the FFN output before it, or the input with i = 0) joins the
        residual stream self.h; leaves the FFN's input in self.xf. The call's sequences are rows `rows` of the stack's, which
        count seq_len tokens (None: kv_len)."""
        c, t = self.attn, self.layers[i]
        e8 = c.weights == "e4m3"
        h, xn, qkv, o, ao = self.h[:B], self.xn[:B], self.qkv[:B], self.o[:B], self.ao[:B]
        _lib.add_rmsnorm(x, h if i else None, t["w_attn"], c.eps, xn, res_out=h)
        self._project(xn, self.xq[:B] if e8 else None, self.xs[:B] if e8 else None, t["W_qkv"], qkv)
        parts = qkv.unflatten(1, (-1, c.head_dim))
        q, k, v = parts.split([c.n_heads, c.n_kv_heads, c.n_kv_heads], dim=1)
        if c.qk_norm or self.freq is not None:
            _lib.qk_norm_rope(q, k, t.get("w_q"), t.get("w_k"), c.eps if c.qk_norm else None, cu, kv_len if seq_len is None else seq_len,
                              self.freq, q, k, interleaved=c.rope_interleaved)
        _lib.kv_write(k, v, t["kv"], cu, kv_len, table)
        # the keys are split for max_len however long the sequences are yet, so that eager and replayed steps give the same
        # bits (one sequence of 500 tokens, 64 heads on 8 of 128: 12.2 us with max_len 4096, 9.7 where the hint is 500)
        lse = self.lse[:B] if c.keep else None
        _lib.attn(q, t["kv"], cu, kv_len, table, max_q, c.max_len, o, self.ws_attn, window=c.window, sinks=c.sinks, lse=lse)
        if c.keep:
            mine = slice(rows.start, rows.start + table.shape[0])
            _lib.attn_mass(q, t["kv"], cu, kv_len, table, max_q, c.max_len, lse, t["mass"][mine], t["pos"][mine], self.ws_mass,
                           seq_len=seq_len)
        self._project(o.flatten(1), self.oq[:B] if e8 else None, self.os[:B] if e8 else None, t["W_o"], ao)
        _lib.add_rmsnorm(ao, h, t["w_ffn"], c.eps, self.xf[:B], res_out=h)

    def _layers(self, x, B: int, cu, rows: slice, max_q: int):
        kv_len, seq_len, table = self.kv_len[rows], self.seq_len[rows], self.table[rows]
        for i in range(len(self.layers)):
            self.attn_layer(i, x, B, cu, kv_len, table, max_q, seq_len, rows)
            x = self.y[i, :B]
            self.layer_call(i, self.xf[:B], False, x)
        _lib.add_rmsnorm(x, self.h[:B], self.w_out, self.attn.eps, self.out[:B], res_out=self.h[:B])

    def evict(self, s: int):
        """Cut sequence s down to the configuration's `keep` cached tokens if it holds more, in every layer, or in none if a layer's
        call is refused."""
        c = self.attn
        if c is None or not c.keep or not 0 <= s < self.max_batch:
            raise ValueError(f"evict: sequence {s} (the stack needs attention with keep > 0)")
        if self.lens[s] <= c.keep:
            return
        one = slice(s, s + 1)
        # what is moved cannot be put back, so every layer's call goes through the library once with no tokens held, which moves none
        for held in (self.no_len, self.kv_len[one]):
            for t in self.layers:
                _lib.kv_evict(t["kv"], held, self.table[one], t["mass"][one], t["pos"][one], c.keep, self.src, self.ws_evict,
                              seq_len=self.seq_len[one], sinks=c.sinks, recent=c.recent, kv_len_out=self.cut_len)
        self.kv_len[one] = self.cut_len
        self.lens[s] = c.keep

    @contextlib.contextmanager
    def _grown(self, rows: slice, n: int):
        """The sequences `rows` longer by n tokens for the calls inside; as they were if one of these is refused, with the attention
        weight of their tokens (not while a graph is captured: see capture; sequences that were cut down to make room stay so)."""
        # (the copy costs an eager step about 10 us whatever its layers; replays have none)
        before, mass = self.lens[rows], None
        if self.attn.keep and not torch.cuda.is_current_stream_capturing():
            mass = self.mass[:, rows, :, :max(before)]
            seen = mass.clone()
        self.lens[rows] = [m + n for m in before]
        self.kv_len[rows] += n
        self.seq_len[rows] += n
        try:
            yield
        except Exception:
            self.lens[rows] = before
            self.kv_len[rows] -= n
            self.seq_len[rows] -= n
            if mass is not None:
                mass.copy_(seen)
            raise

    def _batch(self, B: int):
        if not 1 <= B <= self.max_batch:
            raise ValueError(f"{B} sequences: need 1 to max_batch = {self.max_batch}")

    def _room(self, s: int, n: int):
        """Refuse what does not fit (and with `keep` would not after an eviction either)."""
        held = min(self.lens[s], self.attn.keep) if self.attn.keep else self.lens[s]
        if held + n > self.attn.max_len:
            raise ValueError(f"sequence {s}: {self.lens[s]} + {n} tokens exceed max_len = {self.attn.max_len}")

    def _make_room(self, rows, n: int):
        """Refuse what does not fit; evict from the sequences that would grow past max_len."""
        for s in rows:
            self._room(s, n)
        for s in rows:
            if self.lens[s] + n > self.attn.max_len:
                self.evict(s)

    def prompt(self, s: int, x: torch.Tensor):
        """Enter x [T, D] fp32 (T <= max_batch), the next tokens of sequence s; results in self.out[:T]."""
        T = x.shape[0]
        if self.attn is None or not 0 <= s < self.max_batch or not 1 <= T <= self.max_batch:
            raise ValueError(f"prompt: sequence {s}, {T} tokens (at most {self.max_batch}; the stack needs attention)")
        if x.dim() != 2 or x.shape[1] != self.wl.D or x.dtype != torch.float32 or x.device != self.out.device:
            raise ValueError(f"prompt: x is fp32 [T, {self.wl.D}] on {self.out.device}")
        x = x.contiguous()
        self._make_room([s], T)
        if T not in self.cu_prompt:
            self.cu_prompt[T] = torch.tensor([0, T], dtype=torch.int32, device=self.device)
        one = slice(s, s + 1)
        with self._grown(one, T):
            self._layers(x, T, self.cu_prompt[T], one, T)

    def reset(self):
        """Forget every sequence's tokens."""
        self.kv_len.zero_()
        self.seq_len.zero_()
        self.lens = [0] * self.max_batch

    # ------------------------------------------------------------------ one layer
    def layer_call(self, i: int, x: torch.Tensor, x_norm: bool, y: torch.Tensor, logits=None):
        """Predict + forward of stored layer i on input x [B, D]; writes self.mask[i], active[i], n_active[i], y."""
        t, wl = self.layers[i], self.wl
        if self.fold_predictor and x.shape[0] == 1 and not self.q4:
            # one token, fp16: sffn_decode (predictor stage 2 folded into the row gather where it applies)
            _lib.decode(wl.act, t["P1"], t["P2"], t.get("c"), wl.t, t.get("W_gate"), t.get("b_gate"), t["W_up"],
                        t.get("b_up"), t["W_downT"], x, self.mask[i], self.active[i], self.n_active[i:i + 1], y,
                        self.ws, x_norm=x_norm, n_hot=self.n_hot[i], logits=logits)
            return
        _lib.predict(t["P1"], t["P2"], t.get("c"), x, wl.t, self.mask[i], self.ws, logits=logits, x_norm=x_norm,
                     n_hot=self.n_hot[i])
        if self.q4:
            g = (t["Q_gate"], t["S_gate"]) if wl.act == "reglu" else None
            _lib.forward_q4(wl.act, g, t.get("b_gate"), (t["Q_up"], t["S_up"]), t.get("b_up"),
                            (t["Q_downT"], t["S_downT"]), x, self.mask[i], self.active[i], self.n_active[i:i + 1], y,
                            self.ws, x_norm=x_norm)
        else:
            _lib.forward(wl.act, t.get("W_gate"), t.get("b_gate"), t["W_up"], t.get("b_up"), t["W_downT"], x,
                         self.mask[i], self.active[i], self.n_active[i:i + 1], y, self.ws, x_norm=x_norm)

    def decode_path(self, i: int, B: int) -> int:
        """The kernels of layer i's call for B tokens: _lib.DECODE_FOLDED when sffn_decode runs the predictor's
        second stage inside the row gather, else DECODE_SEPARATE (sffn_predict, then the forward call)."""
        if not (self.fold_predictor and B == 1 and not self.q4):
            return _lib.DECODE_SEPARATE
        return _lib.decode_path(self.wl.act, False, self.wl.D, self.wl.F, self.ranks[i])

    def folded(self, i: int, B: int) -> bool:
        """Whether layer i's call for B tokens runs the predictor's second stage in the row-gather kernel."""
        return self.decode_path(i, B) != _lib.DECODE_SEPARATE

    # ------------------------------------------------------------------ decode step
    def step(self, B: int = 1):
        """One pass through every layer for the B tokens in self.x_in[:B]; outputs land in self.y[:, :B]. With
        attention: the next token of each of the first B sequences, the last layer's output in self.out[:B] too."""
        x = self.x_in[:B]
        if self.attn is not None:
            self._batch(B)
            self._make_room(range(B), 1)
            with self._grown(slice(0, B), 1):
                self._layers(x, B, self.cu_step[:B + 1], slice(0, B), 1)
            return
        for i in range(len(self.layers)):
            y = self.y[i, :B]
            self.layer_call(i, x, i > 0, y)
            x = y

    def capture(self, B: int = 1):
        """Capture step(B) into a HIP graph (after one eager warm-up). With attention the warm-up's tokens are taken
        back: the sequences are as long afterwards as before (unless one had to be cut down for it)."""
        lens = None
        if self.attn is not None:
            self._batch(B)
            self._make_room(range(B), 1)
            seen = [(t["mass"][:B].clone(), t["pos"][:B].clone()) for t in self.layers] if self.attn.keep else []
            lens = (list(self.lens), self.kv_len.clone(), self.seq_len.clone())
        try:
            self.step(B)
            torch.cuda.synchronize(self.device)
            if lens is not None:
                self.lens = list(lens[0])
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                self.step(B)
        finally:
            if lens is not None:
                self.lens = lens[0]
                self.kv_len.copy_(lens[1])
                self.seq_len.copy_(lens[2])
                for t, (mass, pos) in zip(self.layers, seen):
                    t["mass"][:B] = mass
                    t["pos"][:B] = pos
        self.graphs[B] = g
        return g

    def replay(self, B: int = 1):
        graph = self.graphs[B]                                 # (before any length grows)
        if self.attn is not None:
            self._make_room(range(B), 1)
            self.lens[:B] = [n + 1 for n in self.lens[:B]]
        graph.replay()

    # ------------------------------------------------------------------ accounting
    def active_weight_bytes_per_row(self) -> int:
        wl = self.wl
        row = (wl.D // 2 + 2 * (wl.D // 32)) if self.q4 else 2 * wl.D
        return wl.n_mats * row

    def predictor_bytes(self) -> int:
        """Predictor bytes one step reads over the whole stack: P1, and the rows of P2 outside the always-active
        prefix."""
        wl = self.wl
        return sum(2 * (r * wl.D + (wl.F - h) * r) for r, h in zip(self.ranks, self.n_hot))
