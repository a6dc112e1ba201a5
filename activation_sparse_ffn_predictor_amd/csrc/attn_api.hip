// C ABI of the residual norm, the paged K/V cache and the attention: argument checks and dispatch (host only).
#include <math.h>
#include <stdarg.h>
#include <stdio.h>

#include <algorithm>

#include "../../include/sffn.h"
#include "attn.h"

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

}  // extern "C"
