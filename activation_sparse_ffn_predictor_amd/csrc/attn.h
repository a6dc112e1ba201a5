// Shared declarations of the paged K/V cache, the attention over it and the residual norm (gfx950, wave64).
#pragma once
#include "common.h"

namespace sffn {

enum { T_F32 = 0, T_F16 = 1, T_BF16 = 2, T_I8 = 3, T_E4M3 = 4 };   // sffn_type

// Rows whose scale would be below this are stored as zeros with scale 0, so that quotients by it have exact remainders and the attention can work with the
// scales' logarithms and reciprocals in normal fp32 numbers.
constexpr float KV_MIN_SCALE = 8.673617379884035e-19f;   // 2^-60

// A cache as the kernels take it: pages [n_pages, hkv, 1 << psh, d], scales [n_pages, hkv, 1 << psh].
struct Kv {
  char* k;
  char* v;
  float* ks;
  float* vs;
  int n_pages, psh, hkv, d;
};
// The sequences of a call (cu [S + 1], len [S], table rows of `cols` entries, ldt apart).
struct Seqs {
  const int* cu;
  const int* len;
  const int* table;
  int S, T, cols, ldt;
};
// The position of row t of a sequence whose rows end at `end` and whose length is `len`: len - n + (t - first). It comes from
// the caller's numbers as they are, whatever the table row or the call's rows hold (only accesses are bounded by those), so
// the attention and the write agree on it. Lengths count up to MOST_LEN, which puts every one of the up to 2^24 new tokens of
// a longer sequence behind the largest table row. 0 <= t < end. In 32 bits (64 cost a large write 3%): the two limits keep the
// difference from wrapping, and change only positions that are below 0 with them and without.
constexpr int MOST_LEN = (1 << 30) + (1 << 24);
__host__ __device__ __forceinline__ int token_pos(int len, int end, int t) {
  return min(max(len, -(1 << 24)), MOST_LEN) - min(end - t, 0x7F000000);
}

// One sequence, clamped so that nothing read from device memory can lead an access out of the caller's tensors:
// its first row of the token tensors, its new tokens, its cached tokens (at most what its table row can hold); and the first
// row's position, which is not clamped by those.
struct Seq {
  int q0, n, len, p0;
};
__host__ __device__ __forceinline__ Seq load_seq(const Seqs& q, int s, int psh) {
  Seq r;
  const int a = q.cu[s], b = q.cu[s + 1], l = q.len[s];
  r.q0 = min(max(a, 0), q.T);
  r.n = min(max(b, r.q0), q.T) - r.q0;
  r.len = min(max(l, 0), q.cols << psh);
  r.p0 = token_pos(l, max(b, r.q0), r.q0);
  return r;
}

// The sequence of token t: how many of cu[1 .. S] are at most t, counted over a group of G lanes (G-ary search, the
// same t in every lane of a group). S: t lies behind the last sequence.
template <int G>
__device__ __forceinline__ int find_seq(const int* __restrict__ cu, int S, int t) {
  int lo = 0, hi = S;                          // the answer is in lo .. hi
  const int lane = threadIdx.x & (G - 1);
  while (__any(lo < hi)) {
    const int step = (hi - lo + G) / G;        // lane i looks at entry lo + i * step (< hi)
    const int e = lo + lane * step;
    const bool in = lo < hi && e < hi;
    const bool le = in && cu[e + 1] <= t;
    const int c = (int)group_sum<G>(le ? 1.f : 0.f);
    if (lo < hi) {
      const int nlo = c ? lo + (c - 1) * step + 1 : lo;
      const int nhi = c ? min(hi, lo + c * step) : lo;
      lo = nlo;
      hi = max(nhi, nlo);
    }
  }
  return lo;
}

// The key units (1 << ush keys each) that a tile of rows at positions p_lo .. p_hi reads, as one list: first the
// units of the always-visible first tokens that lie before the window, then those of the window itself.
struct Units {
  int sink, w0, tot;        // units before the window; first window unit; all
  __host__ __device__ __forceinline__ int key0(int u, int ush) const { return (u < sink ? u : u - sink + w0) << ush; }
};
__host__ __device__ __forceinline__ Units key_units(int p_lo, int p_hi, int len, int window, int sinks, int ush) {
  const int end = min(len, p_hi + 1);          // keys at or after it are visible to no row
  Units u{0, 0, 0};
  if (end <= 0) return u;
  const int lo = window > 0 ? min(max(0, p_lo - window + 1), end) : 0;   // past the end: tokens past the table row
  u.w0 = lo >> ush;
  u.sink = min((min(sinks, lo) + (1 << ush) - 1) >> ush, u.w0);
  u.tot = u.sink + ((end + (1 << ush) - 1) >> ush) - u.w0;
  return u;
}
// Units of each share when a list of `tot` is split into at most ns shares of at least `least` units, whole
// multiples of `step`.
__host__ __device__ __forceinline__ int share_units(int tot, int ns, int least, int step) {
  const int per = max(least, (tot + ns - 1) / ns);
  return (per + step - 1) / step * step;
}

// Arguments of an attention call. Rows of one K/V head: r = i * G + g for new token i and query head hk * G + g.
struct AttnArgs {
  const char* q;
  char* out;
  float* lse;
  Kv kv;
  Seqs sq;
  int hq, G, max_q, window, sinks, ns;
  long ldq, ldo;            // elements between tokens
  float c;                  // |softmax scale| * log2(e)
  int neg;                  // the scale is negative: the queries' signs are turned as they are loaded
  float* po;                // partial outputs [T * hq][ns][d], used when ns > 1
  float2* pml;              // their references (log2 domain) and sums [T * hq][ns]
};

// few-row kernel: units of 32 keys; a share has at least few_least of them and a multiple of FEW_STEP. (Head sizes over
// 128, whose rows take twice the time: one sequence of 1000 keys, 64 heads on 8 of 256, fp16: 22.1 us in two shares, 15.6
// in four; of 300: 14.5 in one or two.)
constexpr int FEW_USH = 5, FEW_STEP = 4;
__host__ __device__ constexpr int few_least(int d) { return d <= 128 ? 16 : 8; }
// tile kernel: units of 64 keys (32 for head sizes over 128: the accumulators leave no registers for more), 128 rows
__host__ __device__ constexpr int many_ush(int d) { return d <= 128 ? 6 : 5; }
constexpr int MANY_LEAST = 4, MANY_ROWS = 128;
constexpr int MAX_SHARES = 64;

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __bf16 bf8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf2 __attribute__((ext_vector_type(2)));
typedef _Float16 half2v __attribute__((ext_vector_type(2)));
typedef __fp16 fp16x4 __attribute__((ext_vector_type(4)));
typedef int i32x2 __attribute__((ext_vector_type(2)));

// 16-bit operands are kept as raw bits; BF says which of the two types they are.
template <bool BF>
__device__ __forceinline__ f32x4 mfma16(const uint4& a, const uint4& b, f32x4 c) {
  if constexpr (BF) return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf8, a), __builtin_bit_cast(bf8, b), c, 0, 0, 0);
  else return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(half8, a), __builtin_bit_cast(half8, b), c, 0, 0, 0);
}
template <bool BF>
__device__ __forceinline__ f32x16 mfma32(const uint4& a, const uint4& b, f32x16 c) {
  if constexpr (BF) return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf8, a), __builtin_bit_cast(bf8, b), c, 0, 0, 0);
  else return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(half8, a), __builtin_bit_cast(half8, b), c, 0, 0, 0);
}
// buffer load at voff + soff (a wave-uniform part): voff = OOB still reads zeros
__device__ __forceinline__ uint4 ld16(const Buf& b, uint32_t voff, uint32_t soff) {
  const v4u32 v = __builtin_amdgcn_raw_buffer_load_b128(b.r, (int)voff, (int)soff, 0);
  return make_uint4(v.x, v.y, v.z, v.w);
}
// two fp32 values as 16 bits each, rounded to nearest even
template <bool BF>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  if constexpr (BF) return __builtin_bit_cast(uint32_t, bf2{(__bf16)a, (__bf16)b});
  else return __builtin_bit_cast(uint32_t, half2v{(_Float16)a, (_Float16)b});
}
template <bool BF>
__device__ __forceinline__ float lo16(uint32_t u) {
  if constexpr (BF) return __uint_as_float(u << 16);
  else return (float)__builtin_bit_cast(half2v, u).x;
}
template <bool BF>
__device__ __forceinline__ float hi16(uint32_t u) {
  if constexpr (BF) return __uint_as_float(u & 0xFFFF0000u);
  else return (float)__builtin_bit_cast(half2v, u).y;
}
// a bit pattern that is nonzero iff one of the two 16-bit values is infinite or NaN (all exponent bits set: adding
// the lowest exponent bit carries into the sign's place exactly then)
template <bool BF>
__device__ __forceinline__ uint32_t nonfinite2(uint32_t u) {
  constexpr uint32_t E = BF ? 0x7F807F80u : 0x7C007C00u, L = BF ? 0x00800080u : 0x04000400u;
  return ((u & E) + L) & 0x80008000u;
}

// eight 16-bit values: signs turned; largest magnitude; infinities and NaN replaced by 0
__device__ __forceinline__ uint4 flip_signs(const uint4& t) {
  return make_uint4(t.x ^ 0x80008000u, t.y ^ 0x80008000u, t.z ^ 0x80008000u, t.w ^ 0x80008000u);
}
template <bool BF>
__device__ __forceinline__ float absmax8(const uint4& t) {
  const uint32_t u[4] = {t.x, t.y, t.z, t.w};
  float big = 0.f;
#pragma unroll
  for (int k = 0; k < 4; ++k) big = fmaxf(big, fmaxf(fabsf(lo16<BF>(u[k])), fabsf(hi16<BF>(u[k]))));
  return big;
}
template <bool BF>
__device__ __forceinline__ uint4 finite_only(const uint4& t) {
  constexpr uint32_t E = BF ? 0x7F80u : 0x7C00u;
  uint32_t u[4] = {t.x, t.y, t.z, t.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint32_t a = u[k] & 0xFFFFu, b = u[k] >> 16;
    u[k] = ((a & E) != E ? a : 0u) | ((b & E) != E ? b << 16 : 0u);
  }
  return make_uint4(u[0], u[1], u[2], u[3]);
}
// e4m3's two NaN codes, 0x7F and 0xFF (no write stores them): a bit pattern with a byte's top bit where four codes hold one;
// and the codes with those replaced by 0
__device__ __forceinline__ uint32_t nan_codes(uint32_t u) { return ((u & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u; }
__device__ __forceinline__ uint32_t finite_codes(uint32_t u) {
  const uint32_t n = nan_codes(u);
  return u & ~(n | (n - (n >> 7)));
}
__device__ __forceinline__ uint32_t nan_codes4(const uint4& t) { return nan_codes(t.x) | nan_codes(t.y) | nan_codes(t.z) | nan_codes(t.w); }
__device__ __forceinline__ uint4 finite_codes4(const uint4& t) {
  return make_uint4(finite_codes(t.x), finite_codes(t.y), finite_codes(t.z), finite_codes(t.w));
}
// bf16 queries for fp16 products: all times one power of two that takes the largest, `big`, to 2^14 .. 2^15 (exact but for
// elements below 2^-31 of it, rounded to fp16's smallest step: 2^-38 of it or less; the factor ends at 2^126, so under 2^-112 the
// largest comes out smaller and the step is 2^-150 of the elements as they were); c takes the factor back.
__device__ __forceinline__ float to_f16_range(float big, float& c) {
  const int e = big > 0.f && big < 3.4e38f ? 14 - ((int)((__float_as_uint(big) >> 23) & 255) - 127) : 0;
  const int e1 = min(max(e, -126), 126);
  c = c * __uint_as_float((uint32_t)(127 - e1) << 23);
  return __uint_as_float((uint32_t)(e1 + 127) << 23);
}
__device__ __forceinline__ uint4 bf16_to_f16(const uint4& t, float f) {
  const uint32_t u[4] = {t.x, t.y, t.z, t.w};
  uint32_t o[4];
#pragma unroll
  for (int k = 0; k < 4; ++k)
    o[k] = __builtin_bit_cast(uint32_t, half2v{(_Float16)(lo16<true>(u[k]) * f), (_Float16)(hi16<true>(u[k]) * f)});
  return make_uint4(o[0], o[1], o[2], o[3]);
}

// Four 8-bit codes as four fp16 values (exact). int8: the code + 128 in the low byte of 0x64xx is 1024 + code + 128;
// one packed subtraction leaves the code.
template <bool E4M3>
__device__ __forceinline__ uint2 codes4(uint32_t u) {
  if constexpr (E4M3) {
    const half2v a = __builtin_bit_cast(half2v, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)u, 1.0f, false));
    const half2v b = __builtin_bit_cast(half2v, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)u, 1.0f, true));
    return make_uint2(__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b));
  } else {
    u ^= 0x80808080u;
    const half2v k = {(_Float16)-1152.f, (_Float16)-1152.f};
    const half2v a = __builtin_bit_cast(half2v, __builtin_amdgcn_perm(0x64646464u, u, 0x07010700u)) + k;
    const half2v b = __builtin_bit_cast(half2v, __builtin_amdgcn_perm(0x64646464u, u, 0x07030702u)) + k;
    return make_uint2(__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b));
  }
}

// What the softmax takes from a key's scales. With 8-bit V rows the weights p_j s_j that multiply the codes must not
// leave fp16's range whatever the scales are, so the running maximum is taken over x_j + log2 s_j (x: scores in
// log2 units): P_j = 2^(x_j + log2 s_j - m) multiplies the codes, and the softmax's own sum is that of P_j / s_j.
// A row with scale 0 has codes 0, so any scale serves; one with scale NaN counts in the sum as if it had scale 0, and
// its weight in the second product is NaN for the rows that see it.
struct VScale {
  float lg, inv;
};
__device__ __forceinline__ VScale v_scale(float s) {
  const float t = s >= KV_MIN_SCALE ? s : KV_MIN_SCALE;
  return {__builtin_amdgcn_logf(t), __builtin_amdgcn_rcpf(t)};
}
// What weights refer to. P_j = 2^(x_j - m) enters the second product in 16 bits. The reference m follows a row's maximum (lazily:
// it moves only when the maximum has grown by 2^8, so that most tiles leave the sums alone) and lies WEIGHT_UP powers of two
// under it: the largest P_j is 2^WEIGHT_UP .. 2^(WEIGHT_UP + 8). fp16 holds normal numbers from 2^-14 to 2^16, so with 7 weights
// down to 2^-21 of the largest keep its 11 bits and those below are off by at most 2^-25, 2^-32 of the largest; with 0 a flat tail
// of weights under 2^-17 of a dominant key lost its bits, under 2^-25 itself, though its sum may be the output (4000 keys at
// 2^-24.5: 41% off). bf16 has fp32's exponents and needs none (and headroom for values near its largest).
template <bool CB>
constexpr float WEIGHT_UP = CB ? 0.f : 7.f;
template <bool CB>
__device__ __forceinline__ bool outgrown(float top, float m) { return top > m + (WEIGHT_UP<CB> + 8.f); }
template <bool CB>
__device__ __forceinline__ float new_reference(float top, float m) { return fmaxf(m, top - WEIGHT_UP<CB>); }

// Factor of what was accumulated under the reference m when the reference becomes `to` (finite): never 0 where something
// was, so that an infinity or NaN stays one however small its weight has become.
__device__ __forceinline__ float fade(float m, float to) {
  return m == -INFINITY ? 0.f : fmaxf(__builtin_amdgcn_exp2f(m - to), 1.1754944e-38f);
}

// An accumulator that an infinity under a weight of 0 (what 16 bits hold of a small one) has made NaN is set to LOST, a small
// number that stays as it is when 0 is added and is gone with the first infinity or NaN that its row sees; what is still LOST
// after them all was NaN for another reason and is put back.
constexpr float LOST = 1.17549449e-38f;            // one step over the smallest normal number
__device__ __forceinline__ float lose_nan(float o) { return o == o ? o : LOST; }
__device__ __forceinline__ float find_lost(float o) { return o == LOST ? __uint_as_float(0x7FC00000u) : o; }

// natural logarithm of L * 2^M (-infinity for a row without visible keys)
__device__ __forceinline__ float log_sum(float M, float L) {
  return L == 0.f ? -INFINITY : (M + __builtin_amdgcn_logf(L)) * 0.6931471805599453f;
}

// v of this lane and of the one 32 (16) lanes away, combined: lanes of both halves (of neighbouring rows of 16) change
// places in registers, without the LDS crossbar
template <bool MAX>
__device__ __forceinline__ float over32(float v) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  const float a = __uint_as_float(r[0]), b = __uint_as_float(r[1]);
  return MAX ? fmaxf(a, b) : a + b;
}
template <bool MAX>
__device__ __forceinline__ float over16(float v) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  const float a = __uint_as_float(r[0]), b = __uint_as_float(r[1]);
  return MAX ? fmaxf(a, b) : a + b;
}

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

}  // namespace sffn

// error text of the calling thread (api.hip)
void sffn_err_clear();
int sffn_err_set(int status, const char* text);
int sffn_err_hip(hipError_t e, const char* what);

// Launches. Types are sffn_type values; host code has checked every argument.
hipError_t sffn_launch_add_rmsnorm(const void* x, int xt, const void* res, int rt, const float* w, double eps, int T,
                                   int D, long ldx, long ldr, void* y, int yt, float* y_scale, void* res_out, long ldy,
                                   long ldro, hipStream_t st);
hipError_t sffn_launch_kv_write(const sffn::Kv& kv, int kvt, const sffn::Seqs& sq, const void* k, const void* v, int xt,
                                long ldk, long ldv, hipStream_t st);
hipError_t sffn_launch_kv_read(const sffn::Kv& kv, int kvt, const sffn::Seqs& sq, void* k, void* v, int xt, long ldk,
                               long ldv, hipStream_t st);
// rows of one K/V head per sequence that the few-row kernel takes (0: none)
int sffn_attn_few_rows(int d);
hipError_t sffn_launch_attn_few(const sffn::AttnArgs& a, int qt, int kvt, hipStream_t st);
hipError_t sffn_launch_attn_many(const sffn::AttnArgs& a, int qt, int kvt, hipStream_t st);
hipError_t sffn_launch_attn_join(const sffn::AttnArgs& a, int qt, bool few, hipStream_t st);
