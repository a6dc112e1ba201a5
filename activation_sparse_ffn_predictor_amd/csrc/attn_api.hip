// C ABI of the residual norm, the paged K/V cache, the attention, the block-scaled products, the head norms with rotation and
// the eviction: argument checks and dispatch (host only).
#include <math.h>
#include <stdarg.h>
#include <stdio.h>

#include <algorithm>

#include "../../include/sffn.h"
#include "attn.h"
#include "evict.h"
#include "mass.h"
#include "mm.h"

namespace {

int fail(int status, const char* fmt, ...) {
  char text[400];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(text, sizeof(text), fmt, ap);
  va_end(ap);
  return sffn_err_set(status, text);
}

bool al(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }
bool is16(int t) { return t == SFFN_F16 || t == SFFN_BF16; }
bool is8(int t) { return t == SFFN_I8 || t == SFFN_E4M3; }
size_t align256(size_t v) { return (v + 255) & ~(size_t)255; }

constexpr int MAX_T = 1 << 24, MAX_POS = 1 << 30, MAX_S = 65535;

int check_cache(const sffn_kv& c, int type) {
  if (!is16(type)) return fail(SFFN_ERR_ARG, "type %d is not a 16-bit type", type);
  if (!is8(c.type) && c.type != type) return fail(SFFN_ERR_ARG, "cache type %d does not go with type %d", c.type, type);
  if (!c.k || !c.v) return fail(SFFN_ERR_NULL, "cache: k and v are required");
  if (is8(c.type) && (!c.k_scale || !c.v_scale)) return fail(SFFN_ERR_NULL, "an 8-bit cache needs k_scale and v_scale");
  const int step = is8(c.type) ? 16 : 8;
  if (c.head_dim < 16 || c.head_dim > 256 || c.head_dim % step)
    return fail(SFFN_ERR_SHAPE, "head_dim=%d: need 16 <= head_dim <= 256, head_dim %% %d == 0", c.head_dim, step);
  if (c.page < 16 || c.page > 1024 || (c.page & (c.page - 1)))
    return fail(SFFN_ERR_SHAPE, "page=%d: need a power of two in [16, 1024]", c.page);
  if (c.n_pages < 1 || c.n_kv_heads < 1 || c.n_kv_heads > 65535 ||
      (long double)c.n_pages * c.n_kv_heads * c.page >= 2147483648.0L)
    return fail(SFFN_ERR_SHAPE, "n_pages=%d, n_kv_heads=%d, page=%d", c.n_pages, c.n_kv_heads, c.page);
  if (!al(c.k, 16) || !al(c.v, 16) || (is8(c.type) && (!al(c.k_scale, 16) || !al(c.v_scale, 16))))
    return fail(SFFN_ERR_ALIGN, "cache: misaligned pointer");
  return SFFN_OK;
}

int check_seqs(const sffn_seqs& q, int page) {
  if (!q.cu || !q.kv_len || !q.table) return fail(SFFN_ERR_NULL, "cu, kv_len and table are required");
  if (q.S < 1 || q.S > MAX_S) return fail(SFFN_ERR_SHAPE, "S=%d outside [1, %d]", q.S, MAX_S);
  if (q.T < 0 || q.T > MAX_T) return fail(SFFN_ERR_SHAPE, "T=%d outside [0, %d]", q.T, MAX_T);
  if (q.max_pages < 1 || (int64_t)q.max_pages * page > MAX_POS)
    return fail(SFFN_ERR_SHAPE, "max_pages=%d: need 1 <= max_pages, max_pages * page <= %d", q.max_pages, MAX_POS);
  if (q.table_stride < q.max_pages) return fail(SFFN_ERR_SHAPE, "table_stride=%d < max_pages=%d", q.table_stride, q.max_pages);
  if (!al(q.cu, 4) || !al(q.kv_len, 4) || !al(q.table, 4)) return fail(SFFN_ERR_ALIGN, "cu, kv_len or table misaligned");
  return SFFN_OK;
}

int check_rows(const char* what, const void* p, int64_t stride, int64_t width) {
  if (!p) return fail(SFFN_ERR_NULL, "%s is required", what);
  if (stride < width || stride % 8 || stride > ((int64_t)1 << 40))
    return fail(SFFN_ERR_SHAPE, "%s: stride %lld: need a multiple of 8, at least %lld", what, (long long)stride, (long long)width);
  if (!al(p, 16)) return fail(SFFN_ERR_ALIGN, "%s: not 16-byte aligned", what);
  return SFFN_OK;
}

// kv_write, kv_read: fewer than 2^32 threads, a thread taking 8 elements of two tokens
int check_move(const sffn_kv& c, const sffn_seqs& q) {
  const int lanes = c.head_dim <= 32 ? 4 : c.head_dim <= 64 ? 8 : c.head_dim <= 128 ? 16 : 32, tokens = 2 * 256 / lanes;
  if ((int64_t)((q.T + tokens - 1) / tokens) * c.n_kv_heads >= ((int64_t)1 << 24))
    return fail(SFFN_ERR_SHAPE, "T=%d, n_kv_heads=%d, head_dim=%d: too many elements", q.T, c.n_kv_heads, c.head_dim);
  return SFFN_OK;
}

sffn::Kv kv_of(const sffn_kv& c) {
  return {(char*)c.k, (char*)c.v, c.k_scale, c.v_scale, c.n_pages, __builtin_ctz(c.page), c.n_kv_heads, c.head_dim};
}
sffn::Seqs seqs_of(const sffn_seqs& q) { return {q.cu, q.kv_len, q.table, q.S, q.T, q.max_pages, q.table_stride}; }

bool attn_sizes_ok(int Hq, int Hkv, int d, int max_q) {
  return Hkv >= 1 && Hkv <= 65535 && Hq >= Hkv && Hq % Hkv == 0 && d >= 16 && d <= 256 && d % 8 == 0 && max_q >= 1;
}
bool few_rows(int G, int d, int max_q) { return (int64_t)max_q * G <= sffn_attn_few_rows(d); }

// Over how many workgroups the keys of one sequence (few rows) or of one row tile are spread, at most one per few_least
// (MANY_LEAST) units of the keys that the longest sequence can see. Shares fill the chip, but their partial results are
// written, read again and joined by a second kernel.
int shares(int T, int S, int Hkv, int G, int d, int max_q, int max_kv, int window, int sinks) {
  const bool few = few_rows(G, d, max_q);
  int64_t see = std::max(1, std::min(max_kv, MAX_POS));
  if (window > 0) {
    const int64_t rows = few ? max_q : sffn::MANY_ROWS / G + 2;      // tokens of one tile
    see = std::min(see, (int64_t)window + rows + std::min<int64_t>(sinks, see) + 128);
  }
  const int unit = few ? 1 << sffn::FEW_USH : 1 << sffn::many_ush(d), least = few ? sffn::few_least(d) : sffn::MANY_LEAST;
  const int64_t chunk = (int64_t)unit * least;     // keys of the smallest share
  const int64_t most = std::min<int64_t>((see + chunk - 1) / chunk, sffn::MAX_SHARES);
  // workgroups without shares; row tiles: the whole ones, and half a tile more for each further sequence's end
  const int64_t tiles = ((int64_t)T * G + sffn::MANY_ROWS - 1) / sffn::MANY_ROWS + (std::min(S, T) - 1) / 2;
  const int64_t blocks = (few ? (int64_t)S : tiles) * Hkv;
  const int64_t places = 512;                      // workgroups that run at once: two a compute unit
  if ((int64_t)T * Hkv * G >= ((int64_t)1 << 24)) return 1;          // one launch joins: fewer than 2^32 threads
  if (few) {
    // Up to one and a half of the smallest share the join costs more than it saves (16 sequences of 700 on 8 K/V heads,
    // fp16: one share 12.7 us, two 16.3; one sequence of 513: 9.9 and 12.5, of 1000: 14.2 and 13.1).
    if (2 * see <= 3 * chunk) return 1;
    // As many shares as fill one round; with many rows partial results weigh as much as the keys (48 sequences of 4
    // drafts on 128 heads of 64 over a window of 4096, bf16: one share 86 us, six 121; two sequences of 131072 on 8 K/V
    // heads, e4m3: 32 shares 105 us, 64 109). Few rows and most places taken already: shares of half a round's work even
    // out sequences of different lengths (32 sequences to 6000 tokens on 40 heads, int8: one share 187 us, two 169).
    int64_t ns = max_q * G > 16 || 2 * blocks <= places ? places / blocks : (3 * places + blocks - 1) / blocks;
    ns = std::min(ns, most);
    // Past one workgroup a compute unit shares of 1024 keys are enough (60 sequences of 2200 on 8 K/V heads, fp16: four
    // shares 113 us, two 106; 32 of 1100: two 32, one 25; size 256, 64 of 1000: two 116, one 103).
    if (ns * blocks > places / 2)
      ns = std::max(std::min(ns, places / 2 / blocks), std::min(ns, (see + 512) / 1024));
    return (int)std::max<int64_t>(1, ns);
  }
  // Row tiles: one share, a round of one workgroup a compute unit or a round of two, whichever a sum of measured costs
  // puts first: a key takes a tile of head size 128 about 20 ns, half as much again where two share a compute unit; a join
  // starts in 4 us and moves each partial result out and in at 4 TB/s. 64 heads of 128 on 8, fp16: 300 tokens over 300:
  // one share 14 us, two 23; over 1000 one 29, three 35; over 2500 one 59, three 51; 100 tokens over 4000: four shares
  // 36 us, nine 41; over 100000: nine 424, ten 511 (more than a round).
  int64_t best = 1;
  double cost = 0;
  for (const int64_t wgs : {(int64_t)0, places / 2, places}) {
    const int64_t ns = std::max<int64_t>(1, std::min(most, wgs / blocks));
    double t = (double)see / ns * (d + 64) * 0.104 * (ns * blocks > places / 2 ? 1.5 : 1.0);
    if (ns > 1) t += 4000.0 + 0.002 * ns * T * Hkv * G * d;
    if (wgs == 0 || t < cost) best = ns, cost = t;
  }
  return (int)best;
}
int check_workspace(const void* ws, size_t have, size_t need) {
  if (!need) return SFFN_OK;
  if (!ws) return fail(SFFN_ERR_NULL, "workspace is NULL");
  if (!al(ws, 256)) return fail(SFFN_ERR_ALIGN, "workspace not 256-byte aligned");
  if (have < need) return fail(SFFN_ERR_WORKSPACE, "workspace %zu bytes < %zu needed", have, need);
  return SFFN_OK;
}
bool mm_sizes_ok(int N, int K) { return N >= 8 && N <= (1 << 22) && N % 8 == 0 && K >= 16 && K <= 65536 && K % 16 == 0; }
// mass and pos [S, n_kv_heads, W]
int check_track(int S, int Hkv, int W) {
  if (W < 1 || (int64_t)S * Hkv >= (1 << 22) || (long double)S * Hkv * W >= 2147483648.0L) return fail(SFFN_ERR_SHAPE, "S=%d, n_kv_heads=%d, W=%d", S, Hkv, W);
  return SFFN_OK;
}
// Workgroups of an attn_mass call along the keys, and the shares of its rows
struct MassPlan {
  int tiles, rs, wp;
};
MassPlan mass_plan(int S, int Hkv, int G, int d, int max_q, int max_kv, int W) {
  const int64_t keys = std::max(1, std::min(max_kv, W)), rows = (int64_t)max_q * G, seqs = (int64_t)S * Hkv;
  MassPlan p{1, 1, 0};
  if (sffn::mass_few(rows, d)) {
    // Workgroups of 1024 keys, eight units a wave; of fewer where that leaves places free (32 sequences to 6000 tokens on 40 heads,
    // int8: of 512 keys 102 us, 1024 100, 2048 109): up to 4096 workgroups, or 2048 where each has more than 16 rows to load first (16
    // sequences of 5000, 4 heads of 256: 2048 workgroups 24 us, 4096 19.6; 48 of 4000, 8 heads of 64 and 32 rows: 27 and 31.5)
    const int64_t places = rows <= 16 ? 4096 : 2048;
    p.tiles = (int)std::min((keys + 127) / 128, std::max((keys + 1023) / 1024, (places + seqs - 1) / seqs));
    p.tiles = std::max(1, std::min(p.tiles, (1 << 22) / (int)seqs));
    return p;
  }
  const int tile = sffn::mass_tile(d);
  p.tiles = (int)std::min<int64_t>((keys + tile - 1) / tile, std::max<int64_t>(1, (1 << 20) / seqs));
  const int64_t blocks = seqs * p.tiles;
  // Shares of the rows: about 2048 workgroups, four times what runs at once, since early keys have more rows than late ones (2048
  // tokens over 6144, 64 heads on 8: 6 shares 262 us, 8 255, 11 245, 22 262), of 512 rows or more; up to 1024 workgroups of 256 or
  // more (700 tokens over 2000, 12 heads of 80 on 4: 5 shares 33 us, 9 24; 40 heads of 96 on 8: 7 shares 42.5, 14 37.8)
  const int64_t fill = std::min({(2047 + blocks) / blocks, (rows + 511) / 512, (int64_t)16}),
                few = std::min({(1023 + blocks) / blocks, (rows + 255) / 256, (int64_t)32});
  if (blocks < 2048) p.rs = (int)std::max<int64_t>(1, std::max(fill, few));
  p.wp = p.tiles * tile;
  return p;
}
size_t po_bytes(int T, int Hq, int d, int ns) { return align256((size_t)T * Hq * ns * d * sizeof(float)); }

}  // namespace

extern "C" {

int sffn_kv_write(sffn_kv c, sffn_seqs q, int type, const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                  void* stream) {
  sffn_err_clear();
  int s = check_cache(c, type);
  if (!s) s = check_seqs(q, c.page);
  if (!s && q.T) s = check_rows("k", k, k_stride, (int64_t)c.n_kv_heads * c.head_dim);
  if (!s && q.T) s = check_rows("v", v, v_stride, (int64_t)c.n_kv_heads * c.head_dim);
  if (s || q.T == 0) return s;
  if ((s = check_move(c, q))) return s;
  const hipError_t e = sffn_launch_kv_write(kv_of(c), c.type, seqs_of(q), k, v, type, k_stride, v_stride, (hipStream_t)stream);
  return e == hipSuccess ? SFFN_OK : sffn_err_hip(e, "kv_write launch");
}

int sffn_kv_read(sffn_kv c, sffn_seqs q, int type, void* k, int64_t k_stride, void* v, int64_t v_stride, void* stream) {
  sffn_err_clear();
  int s = check_cache(c, type);
  if (!s) s = check_seqs(q, c.page);
  if (!s && q.T) s = check_rows("k", k, k_stride, (int64_t)c.n_kv_heads * c.head_dim);
  if (!s && q.T) s = check_rows("v", v, v_stride, (int64_t)c.n_kv_heads * c.head_dim);
  if (s || q.T == 0) return s;
  if ((s = check_move(c, q))) return s;
  const hipError_t e = sffn_launch_kv_read(kv_of(c), c.type, seqs_of(q), k, v, type, k_stride, v_stride, (hipStream_t)stream);
  return e == hipSuccess ? SFFN_OK : sffn_err_hip(e, "kv_read launch");
}

int sffn_attn_path(int Hq, int n_kv_heads, int head_dim, int max_q) {
  if (!attn_sizes_ok(Hq, n_kv_heads, head_dim, max_q)) return -1;
  return few_rows(Hq / n_kv_heads, head_dim, max_q) ? SFFN_ATTN_FEW : SFFN_ATTN_MANY;
}

size_t sffn_attn_workspace_size(int T, int S, int Hq, int n_kv_heads, int head_dim, int max_q, int max_kv, int window,
                                int sinks) {
  if (!attn_sizes_ok(Hq, n_kv_heads, head_dim, max_q) || T < 1 || S < 1 || window < 0 || sinks < 0) return 0;
  max_q = std::min(max_q, T);
  const int ns = shares(T, S, n_kv_heads, Hq / n_kv_heads, head_dim, max_q, max_kv, window, sinks);
  return ns > 1 ? po_bytes(T, Hq, head_dim, ns) + align256((size_t)T * Hq * ns * 2 * sizeof(float)) : 0;
}

int sffn_attn(sffn_kv c, sffn_seqs q, int type, const void* qp, int64_t q_stride, int Hq, int max_q, int max_kv,
              float scale, int window, int sinks, void* out, int64_t out_stride, float* lse, void* ws, size_t ws_bytes,
              void* stream) {
  sffn_err_clear();
  int s = check_cache(c, type);
  if (!s) s = check_seqs(q, c.page);
  if (s) return s;
  if (Hq < c.n_kv_heads || Hq % c.n_kv_heads) return fail(SFFN_ERR_SHAPE, "Hq=%d is not a multiple of n_kv_heads=%d", Hq, c.n_kv_heads);
  if ((int64_t)q.T * Hq >= ((int64_t)1 << 31)) return fail(SFFN_ERR_SHAPE, "T=%d, Hq=%d: T * Hq reaches 2^31", q.T, Hq);
  if (max_q < 1) return fail(SFFN_ERR_SHAPE, "max_q=%d < 1", max_q);
  if (!isfinite(scale)) return fail(SFFN_ERR_ARG, "scale is not finite");
  if (window < 0 || sinks < 0) return fail(SFFN_ERR_ARG, "window=%d, sinks=%d: need both >= 0", window, sinks);
  if (q.T == 0) return SFFN_OK;
  s = check_rows("q", qp, q_stride, (int64_t)Hq * c.head_dim);
  if (!s) s = check_rows("out", out, out_stride, (int64_t)Hq * c.head_dim);
  if (s) return s;
  if (lse && !al(lse, 4)) return fail(SFFN_ERR_ALIGN, "lse misaligned");
  max_q = std::min(max_q, q.T);
  const int G = Hq / c.n_kv_heads;
  const int ns = shares(q.T, q.S, c.n_kv_heads, G, c.head_dim, max_q, max_kv, window, sinks);
  const size_t need = sffn_attn_workspace_size(q.T, q.S, Hq, c.n_kv_heads, c.head_dim, max_q, max_kv, window, sinks);
  if (need) {
    if (!ws) return fail(SFFN_ERR_NULL, "workspace is NULL");
    if (!al(ws, 256)) return fail(SFFN_ERR_ALIGN, "workspace not 256-byte aligned");
    if (ws_bytes < need) return fail(SFFN_ERR_WORKSPACE, "workspace %zu bytes < %zu needed", ws_bytes, need);
  }
  const bool few = few_rows(G, c.head_dim, max_q);
  // fewer than 2^32 threads a launch
  if (!few && ((int64_t)q.T * G / sffn::MANY_ROWS + std::min(q.S, q.T)) * c.n_kv_heads >= ((int64_t)1 << 24))
    return fail(SFFN_ERR_SHAPE, "T=%d, S=%d, Hq=%d: too many row tiles", q.T, q.S, Hq);
  sffn::AttnArgs a;
  a.q = (const char*)qp;
  a.out = (char*)out;
  a.lse = lse;
  a.kv = kv_of(c);
  a.sq = seqs_of(q);
  a.hq = Hq;
  a.G = G;
  a.max_q = max_q;
  a.window = std::min(window, sffn::MOST_LEN);                    // every position is below it
  a.sinks = std::min(sinks, MAX_POS);
  a.ns = ns;
  a.ldq = q_stride;
  a.ldo = out_stride;
  a.c = std::max(fabsf(scale) * 1.4426950408889634f, 1.2e-38f);   // not 0: masked scores are -infinity times it
  a.neg = scale < 0.f;
  a.po = (float*)ws;
  a.pml = (float2*)((char*)ws + (ns > 1 ? po_bytes(q.T, Hq, c.head_dim, ns) : 0));
  hipStream_t st = (hipStream_t)stream;
  hipError_t e = few ? sffn_launch_attn_few(a, type, c.type, st) : sffn_launch_attn_many(a, type, c.type, st);
  if (e == hipSuccess && ns > 1) e = sffn_launch_attn_join(a, type, few, st);
  return e == hipSuccess ? SFFN_OK : sffn_err_hip(e, "attn launch");
}

int sffn_add_rmsnorm(int x_type, const void* x, int64_t x_stride, int res_type, const void* res, int64_t res_stride,
                     const float* w, double eps, int T, int D, int y_type, void* y, int64_t y_stride, float* y_scale,
                     void* res_out, int64_t res_out_stride, void* stream) {
  sffn_err_clear();
  if ((x_type != SFFN_F32 && !is16(x_type)) || ((res || res_out) && res_type != SFFN_F32 && !is16(res_type)) ||
      (y_type != SFFN_F32 && !is16(y_type) && !is8(y_type)))
    return fail(SFFN_ERR_ARG, "add_rmsnorm: types %d, %d, %d", x_type, res_type, y_type);
  if (T < 0 || T > MAX_T) return fail(SFFN_ERR_SHAPE, "T=%d outside [0, %d]", T, MAX_T);
  if (D < 8 || D > 16384 || D % 8) return fail(SFFN_ERR_SHAPE, "D=%d: need 8 <= D <= 16384, D %% 8 == 0", D);
  if (!(eps >= 0.0) || !isfinite(eps)) return fail(SFFN_ERR_ARG, "eps=%g: need a finite eps >= 0", eps);
  if (T == 0) return SFFN_OK;
  int s = check_rows("x", x, x_stride, D);
  if (!s && res) s = check_rows("res", res, res_stride, D);
  if (!s && res_out) s = check_rows("res_out", res_out, res_out_stride, D);
  if (!s) s = check_rows("y", y, y_stride, D);
  if (s) return s;
  if (is8(y_type) && !y_scale) return fail(SFFN_ERR_NULL, "an 8-bit y needs y_scale");
  if ((w && !al(w, 16)) || (y_scale && !al(y_scale, 4))) return fail(SFFN_ERR_ALIGN, "add_rmsnorm: misaligned pointer");
  if (res && res == res_out && res_stride != res_out_stride)
    return fail(SFFN_ERR_ARG, "add_rmsnorm: res_out is res with another stride");
  if (y == x || y == res || y == res_out || x == res_out) return fail(SFFN_ERR_ARG, "add_rmsnorm: y or res_out overlaps an input");
  const hipError_t e = sffn_launch_add_rmsnorm(x, x_type, res, res_type, w, eps, T, D, x_stride, res_stride, y, y_type,
                                               y_scale, res_out, y_stride, res_out_stride, (hipStream_t)stream);
  return e == hipSuccess ? SFFN_OK : sffn_err_hip(e, "add_rmsnorm launch");
}

int sffn_quant128(int x_type, const void* x, int64_t x_stride, int T, int D, int rows, void* y, int64_t y_stride, float* scale,
                  void* stream) {
  sffn_err_clear();
  if (x_type != SFFN_F32 && !is16(x_type)) return fail(SFFN_ERR_ARG, "quant128: type %d", x_type);
  if (rows != 1 && rows != 128) return fail(SFFN_ERR_ARG, "quant128: rows=%d: need 1 or 128", rows);
  if (T < 0 || T > MAX_T) return fail(SFFN_ERR_SHAPE, "T=%d outside [0, %d]", T, MAX_T);
  if (D < 8 || D > 65536 || D % 8) return fail(SFFN_ERR_SHAPE, "D=%d: need 8 <= D <= 65536, D %% 8 == 0", D);
  if (T == 0) return SFFN_OK;
  int s = check_rows("x", x, x_stride, D);
  if (!s) s = check_rows("y", y, y_stride, D);
  if (s) return s;
  if (!scale) return fail(SFFN_ERR_NULL, "scale is required");
  if (!al(scale, 4)) return fail(SFFN_ERR_ALIGN, "scale misaligned");
  if (x == y || x == scale || y == (void*)scale) return fail(SFFN_ERR_ARG, "quant128: an output overlaps another tensor");
  const hipError_t e = sffn_launch_quant128(x, x_type, x_stride, T, D, rows, y, y_stride, scale, (hipStream_t)stream);
  return e == hipSuccess ? SFFN_OK : sffn_err_hip(e, "quant128 launch");
}

size_t sffn_mm_workspace_size(int T, int N, int K) {
  if (T < 1 || T > MAX_T || !mm_sizes_ok(N, K)) return 0;
  return align256(sffn_mm_workspace(T, N, K));
}

int sffn_mm_e4m3(const void* a, int64_t a_stride, const float* a_scale, const void* b, int64_t b_stride, const float* b_scale,
                 int T, int N, int K, int out_type, void* out, int64_t out_stride, void* ws, size_t ws_bytes, void* stream) {
  sffn_err_clear();
  if (out_type != SFFN_F32 && !is16(out_type)) return fail(SFFN_ERR_ARG, "mm_e4m3: type %d", out_type);
  if (T < 0 || T > MAX_T) return fail(SFFN_ERR_SHAPE, "T=%d outside [0, %d]", T, MAX_T);
  if (!mm_sizes_ok(N, K))
    return fail(SFFN_ERR_SHAPE, "N=%d, K=%d: need N %% 8 == 0, 8 <= N <= 2^22, K %% 16 == 0, 16 <= K <= 65536", N, K);
  if ((int64_t)((T + 127) / 128) * ((N + 127) / 128) >= ((int64_t)1 << 24)) return fail(SFFN_ERR_SHAPE, "T=%d, N=%d: too many tiles", T, N);
  if (T == 0) return SFFN_OK;
  int s = check_rows("a", a, a_stride, K);
  if (!s) s = check_rows("b", b, b_stride, K);
  if (!s) s = check_rows("out", out, out_stride, N);
  if (s) return s;
  if (a_stride % 16 || b_stride % 16 || a_stride > (1 << 22) || b_stride > (1 << 22))
    return fail(SFFN_ERR_SHAPE, "mm_e4m3: strides %lld, %lld: need multiples of 16, at most 2^22", (long long)a_stride, (long long)b_stride);
  if (!a_scale || !b_scale) return fail(SFFN_ERR_NULL, "a_scale and b_scale are required");
  if (!al(a_scale, 4) || !al(b_scale, 4)) return fail(SFFN_ERR_ALIGN, "a_scale or b_scale misaligned");
  if (out == a || out == b || out == a_scale || out == b_scale) return fail(SFFN_ERR_ARG, "mm_e4m3: out overlaps an input");
  const size_t need = sffn_mm_workspace_size(T, N, K);
  if ((s = check_workspace(ws, ws_bytes, need))) return s;
  const sffn::MmArgs g{(const char*)a, (const char*)b, a_scale, b_scale, out, (char*)ws, (long)a_stride, (long)b_stride, (long)out_stride, T, N, K};
  const hipError_t e = sffn_launch_mm(g, out_type, (hipStream_t)stream);
  return e == hipSuccess ? SFFN_OK : sffn_err_hip(e, "mm_e4m3 launch");
}

int sffn_qk_norm_rope(int type, const int32_t* cu, const int32_t* seq_len, int S, int T, const void* q, int64_t q_stride, int Hq,
                      const void* k, int64_t k_stride, int n_kv_heads, int head_dim, int norm, const float* w_q, const float* w_k,
                      double eps, const float* freq, int rot, int interleaved, void* q_out, int64_t q_out_stride, void* k_out,
                      int64_t k_out_stride, void* stream) {
  sffn_err_clear();
  if (!is16(type)) return fail(SFFN_ERR_ARG, "type %d is not a 16-bit type", type);
  if (!cu || !seq_len) return fail(SFFN_ERR_NULL, "cu and seq_len are required");
  if (S < 1 || S > MAX_S) return fail(SFFN_ERR_SHAPE, "S=%d outside [1, %d]", S, MAX_S);
  if (T < 0 || T > MAX_T) return fail(SFFN_ERR_SHAPE, "T=%d outside [0, %d]", T, MAX_T);
  if (head_dim < 8 || head_dim > 256 || head_dim % 8)
    return fail(SFFN_ERR_SHAPE, "head_dim=%d: need 8 <= head_dim <= 256, head_dim %% 8 == 0", head_dim);
  if (rot < 0 || rot > head_dim || rot % 8) return fail(SFFN_ERR_SHAPE, "rot=%d: need 0 <= rot <= head_dim=%d, rot %% 8 == 0", rot, head_dim);
  if (Hq < 1 || Hq > 65535 || (k && (n_kv_heads < 1 || n_kv_heads > 65535)))
    return fail(SFFN_ERR_SHAPE, "Hq=%d, n_kv_heads=%d outside [1, 65535]", Hq, n_kv_heads);
  if (norm && (!(eps >= 0.0) || !isfinite(eps))) return fail(SFFN_ERR_ARG, "eps=%g: need a finite eps >= 0", eps);
  if (rot && !freq) return fail(SFFN_ERR_NULL, "freq is required");
  if (!al(cu, 4) || !al(seq_len, 4) || !al(freq, 4) || !al(w_q, 4) || !al(w_k, 4)) return fail(SFFN_ERR_ALIGN, "qk_norm_rope: misaligned pointer");
  if (T == 0) return SFFN_OK;
  int s = check_rows("q", q, q_stride, (int64_t)Hq * head_dim);
  if (!s) s = check_rows("q_out", q_out, q_out_stride, (int64_t)Hq * head_dim);
  if (!s && k) s = check_rows("k", k, k_stride, (int64_t)n_kv_heads * head_dim);
  if (!s && k) s = check_rows("k_out", k_out, k_out_stride, (int64_t)n_kv_heads * head_dim);
  if (s) return s;
  if ((q == q_out && q_stride != q_out_stride) || (k && k == k_out && k_stride != k_out_stride))
    return fail(SFFN_ERR_ARG, "qk_norm_rope: an output is its input with another stride");
  if (k && (q_out == k || k_out == q || k_out == q_out)) return fail(SFFN_ERR_ARG, "qk_norm_rope: an output overlaps another tensor");
  const hipError_t e = sffn_launch_rope(type, cu, seq_len, S, T, q, q_stride, Hq, k, k_stride, n_kv_heads, head_dim, norm, w_q, w_k,
                                        eps, freq, rot, interleaved, q_out, q_out_stride, k_out, k_out_stride, (hipStream_t)stream);
  return e == hipSuccess ? SFFN_OK : sffn_err_hip(e, "qk_norm_rope launch");
}

size_t sffn_attn_mass_workspace_size(int S, int Hq, int n_kv_heads, int head_dim, int max_q, int max_kv, int W) {
  if (!attn_sizes_ok(Hq, n_kv_heads, head_dim, max_q) || S < 1 || S > MAX_S || W < 1) return 0;
  const MassPlan p = mass_plan(S, n_kv_heads, Hq / n_kv_heads, head_dim, max_q, max_kv, W);
  return p.rs > 1 ? align256((size_t)S * n_kv_heads * p.rs * p.wp * sizeof(float)) : 0;
}

int sffn_attn_mass(sffn_kv c, sffn_seqs q, const int32_t* seq_len, int type, const void* qp, int64_t q_stride, int Hq, int max_q,
                   int max_kv, float scale, int window, int sinks, const float* lse, const float* mass, float* mass_out,
                   int32_t* pos, int W, void* ws, size_t ws_bytes, void* stream) {
  sffn_err_clear();
  int s = check_cache(c, type);
  if (!s) s = check_seqs(q, c.page);
  if (s) return s;
  if (!seq_len || !mass || !mass_out || !pos) return fail(SFFN_ERR_NULL, "seq_len, mass, mass_out and pos are required");
  if (Hq < c.n_kv_heads || Hq % c.n_kv_heads) return fail(SFFN_ERR_SHAPE, "Hq=%d is not a multiple of n_kv_heads=%d", Hq, c.n_kv_heads);
  if ((int64_t)q.T * Hq >= ((int64_t)1 << 31)) return fail(SFFN_ERR_SHAPE, "T=%d, Hq=%d: T * Hq reaches 2^31", q.T, Hq);
  if (max_q < 1) return fail(SFFN_ERR_SHAPE, "max_q=%d < 1", max_q);
  if ((s = check_track(q.S, c.n_kv_heads, W))) return s;
  if (!isfinite(scale)) return fail(SFFN_ERR_ARG, "scale is not finite");
  if (window < 0 || sinks < 0) return fail(SFFN_ERR_ARG, "window=%d, sinks=%d: need both >= 0", window, sinks);
  if (!al(seq_len, 4) || !al(lse, 4) || !al(mass, 4) || !al(mass_out, 4) || !al(pos, 4))
    return fail(SFFN_ERR_ALIGN, "attn_mass: misaligned pointer");
  if ((const void*)pos == mass || (void*)pos == mass_out) return fail(SFFN_ERR_ARG, "attn_mass: pos overlaps mass");
  if (q.T == 0) return SFFN_OK;
  if ((s = check_rows("q", qp, q_stride, (int64_t)Hq * c.head_dim))) return s;
  if (!lse) return fail(SFFN_ERR_NULL, "lse is required");
  const size_t need = sffn_attn_mass_workspace_size(q.S, Hq, c.n_kv_heads, c.head_dim, max_q, max_kv, W);
  if ((s = check_workspace(ws, ws_bytes, need))) return s;
  const MassPlan p = mass_plan(q.S, c.n_kv_heads, Hq / c.n_kv_heads, c.head_dim, max_q, max_kv, W);
  sffn::MassArgs a;
  a.q = (const char*)qp;
  a.lse = lse;
  a.mass = mass;
  a.out = mass_out;
  a.pos = pos;
  a.plen = seq_len;
  a.kv = kv_of(c);
  a.sq = seqs_of(q);
  a.hq = Hq;
  a.G = Hq / c.n_kv_heads;
  a.max_q = max_q;
  a.window = std::min(window, sffn::MOST_LEN);
  a.sinks = std::min(sinks, MAX_POS);
  a.W = W;
  a.ldq = q_stride;
  a.c = scale * 1.4426950408889634f;
  a.rs = p.rs;
  a.wp = p.wp;
  a.part = (float*)ws;
  const hipError_t e = sffn_launch_mass(a, type, c.type, p.tiles, (hipStream_t)stream);
  return e == hipSuccess ? SFFN_OK : sffn_err_hip(e, "attn_mass launch");
}

size_t sffn_kv_evict_workspace_size(int S, int n_kv_heads, int W, int keep) {
  if (S < 1 || S > MAX_S || n_kv_heads < 1 || n_kv_heads > 65535 || keep < 1 || keep > W) return 0;
  sffn::EvictArgs a{};
  a.S = S, a.W = W, a.keep = keep;
  return sffn::evict_plan(a, n_kv_heads, nullptr);
}

int sffn_kv_evict(sffn_kv c, const int32_t* kv_len, const int32_t* seq_len, const int32_t* table, int S, int max_pages,
                  int table_stride, const float* mass, const int32_t* pos, int W, int keep, int sinks, int recent, int32_t* src,
                  float* mass_out, int32_t* pos_out, int32_t* kv_len_out, void* ws, size_t ws_bytes, void* stream) {
  sffn_err_clear();
  int s = check_cache(c, is16(c.type) ? c.type : SFFN_F16);
  // (the table's checks ask for a cu array too, which an eviction has none of)
  if (!s) s = check_seqs({kv_len, kv_len, table, S, 0, max_pages, table_stride}, c.page);
  if (s) return s;
  if (!seq_len || !mass || !pos || !src || !mass_out || !pos_out || !kv_len_out)
    return fail(SFFN_ERR_NULL, "seq_len, mass, pos, src, mass_out, pos_out and kv_len_out are required");
  if ((s = check_track(S, c.n_kv_heads, W))) return s;
  if (keep < 1 || keep > W) return fail(SFFN_ERR_SHAPE, "keep=%d outside [1, W=%d]", keep, W);
  if (sinks < 0 || recent < 0 || (int64_t)sinks + recent > keep)
    return fail(SFFN_ERR_ARG, "sinks=%d, recent=%d: need both >= 0, their sum at most keep=%d", sinks, recent, keep);
  if (!al(seq_len, 4) || !al(mass, 4) || !al(pos, 4) || !al(src, 4) || !al(mass_out, 4) || !al(pos_out, 4) || !al(kv_len_out, 4))
    return fail(SFFN_ERR_ALIGN, "kv_evict: misaligned pointer");
  if (kv_len_out == seq_len)
    return fail(SFFN_ERR_ARG, "kv_evict: kv_len_out is seq_len, so the sequences would forget how many tokens they count: one of them has to be a tensor of its own");
  const void* all[] = {mass, pos, src, mass_out, pos_out, kv_len, seq_len, kv_len_out, table};
  for (int i = 0; i < 9; ++i)
    for (int j = 0; j < i; ++j)
      if (all[i] == all[j] && !(j == 0 && i == 3) && !(j == 1 && i == 4) && !(j == 5 && (i == 6 || i == 7)))
        return fail(SFFN_ERR_ARG, "kv_evict: an output overlaps another tensor");
  if ((s = check_workspace(ws, ws_bytes, sffn_kv_evict_workspace_size(S, c.n_kv_heads, W, keep)))) return s;
  // fewer than 2^32 threads a launch, 8 slots a workgroup at least, and 256 of weights and positions
  if ((int64_t)((keep + 7) / 8 + (keep + 255) / 256) * S * c.n_kv_heads >= ((int64_t)1 << 24))
    return fail(SFFN_ERR_SHAPE, "S=%d, n_kv_heads=%d, keep=%d: too many slots", S, c.n_kv_heads, keep);
  sffn::EvictArgs a{kv_of(c), kv_len, seq_len, table, mass, pos, mass_out, pos_out, kv_len_out, src, S, max_pages, table_stride, W, keep,
                    sinks, recent};
  sffn::evict_plan(a, c.n_kv_heads, ws);
  const hipError_t e = sffn_launch_evict(a, c.type, (hipStream_t)stream);
  return e == hipSuccess ? SFFN_OK : sffn_err_hip(e, "kv_evict launch");
}

}  // extern "C"
