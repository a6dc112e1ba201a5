// Paged K/V cache: new tokens written (as they are or quantised to 8 bits), and a range of tokens read back.
//
// Both are bound by memory, each byte moved once; a row of a head is a few lanes' work, so that its maximum needs no LDS
// and neighbouring tokens of a head fill neighbouring slots. Measured: 4000 tokens of 40 heads of 128 written in 32.5 us as
// bf16 (5.0 TB/s) and in 28 to 31 as e4m3 (4.0 to 4.4 TB/s; 24.7 us without the encoding, which is what then bounds it); 54000 tokens
// read from e4m3 to bf16, 703 MB in 134 to 143 us (box to box; 5.0 to 5.3 TB/s).
#include "attn.h"

using namespace sffn;

namespace {

// max over aligned groups of G lanes
template <int CTRL>
__device__ __forceinline__ uint32_t dpp_u(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, true);
}
template <int G>
__device__ __forceinline__ uint32_t group_max(uint32_t v) {
  if (G >= 2) v = max(v, dpp_u<0xB1>(v));
  if (G >= 4) v = max(v, dpp_u<0x4E>(v));
  if (G >= 8) v = max(v, dpp_u<0x141>(v));
  if (G >= 16) v = max(v, dpp_u<0x140>(v));
  if (G >= 32) v = max(v, (uint32_t)__shfl_xor((int)v, 16, WAVE));
  return v;
}

// b / TOP, correctly rounded (shown for every mantissa of 11 bits by exact arithmetic; below 2^-60 it does not matter)
template <int TOP>
__device__ __forceinline__ float over_top(float b) {
  constexpr float R = 1.f / TOP;
  const float q = b * R;
  return fmaf(fmaf(-q, (float)TOP, b), R, q);
}

// four codes of x * f, rounded to nearest even
template <bool E4M3>
__device__ __forceinline__ uint32_t encode4(const float* x, float f) {
  if constexpr (E4M3) {
    const int u = __builtin_amdgcn_cvt_pk_fp8_f32(x[0] * f, x[1] * f, 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(x[2] * f, x[3] * f, u, true);
  } else {
    uint32_t b[4];                                           // x f + 1.5 * 2^23 has the rounded x f in its low byte
#pragma unroll
    for (int i = 0; i < 4; ++i) b[i] = __float_as_uint(fmaf(x[i], f, 12582912.f));
    return __builtin_amdgcn_perm(__builtin_amdgcn_perm(b[3], b[2], 0x0C0C0400u),
                                 __builtin_amdgcn_perm(b[1], b[0], 0x0C0C0400u), 0x05040100u);
  }
}
// A value that rounds to the same code as the exact quotient x / s. inv: 1 / s to within a few steps. A code or the middle
// between two of them has at most 5 significant bits (e4m3) or is a multiple of 1/2 (int8): h is the one nearest to the
// quotient, and the sign of the remainder x - h s (one rounding: exact) tells on which side of it the quotient lies.
template <bool E4M3>
__device__ __forceinline__ float beside(float x, float s, float inv) {
  const float h = E4M3 ? __uint_as_float((__float_as_uint(x * inv) + 0x40000u) & 0xFFF80000u)
                       : fmaf(x, inv, 6291456.f) - 6291456.f;      // 1.5 * 2^22: steps of 1/2
  constexpr float T = E4M3 ? 0x1p-15f : 0x1p-8f;   // 2^-15 is one step at 448; what is nearer to 0 than 2^-10 is 0
  return h + __builtin_amdgcn_fmed3f(fmaf(-h, s, x) * 0x1p100f, -T, T);
}
// Codes of x[0 .. 8) / s, rounded to nearest even from the exact quotients. 1 / s lies between two fp32 factors; where
// both give the same codes, these are the quotients' codes, else (in one of the wave's rows) remainders decide. A value
// with the largest one's mantissa is a middle or within a step of one, which every second wave of bf16 rows holds: those
// go to the remainders at once (4000 tokens of 40 heads of 128, bf16 to e4m3: 31.9 -> 30.0 us; 3300 from fp16 to int8:
// with the factors 21.2 us, without 22.6). Quotients are at most top (1 + 2^-23) by the scale's making: nothing needs a
// limit.
template <bool E4M3, bool BF>
__device__ __forceinline__ uint2 encode8(const float* x, float s) {
  const float inv = __builtin_amdgcn_rcpf(s);
  uint2 c = make_uint2(0, 0);
  bool same = false;
  if constexpr (!BF) {
    const float lo = inv * (1.f - 0x1p-20f), hi = inv * (1.f + 0x1p-20f);
    c = make_uint2(encode4<E4M3>(x, lo), encode4<E4M3>(x + 4, lo));
    same = !__any(((c.x ^ encode4<E4M3>(x, hi)) | (c.y ^ encode4<E4M3>(x + 4, hi))) != 0);
  }
  if (!same) {
    float q[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = beside<E4M3>(x[i], s, inv);
    c = make_uint2(encode4<E4M3>(q, 1.f), encode4<E4M3>(q + 4, 1.f));
  }
  return c;
}

// The rows (cache row index of head 0's copy, or -1) of the PASS tokens t0, t0 + step, ...: neighbours mostly belong to
// one sequence, so it is searched for once.
template <int LPR, int PASS>
__device__ __forceinline__ void find_rows(const Kv& kv, const Seqs& sq, int h, int t0, int step, long (&row)[PASS]) {
  int s = 0, a = 0, end = -1, shift = 0;           // sequence, its tokens a .. end - 1, their positions less their rows
#pragma unroll
  for (int p = 0; p < PASS; ++p) {
    const int t = t0 + p * step;
    row[p] = -1;
    if (t >= sq.T) continue;
    if (t >= end || t < a) {
      s = find_seq<LPR>(sq.cu, sq.S, t);
      if (s >= sq.S) continue;                     // behind the last sequence
      a = sq.cu[s];
      end = sq.cu[s + 1];
      shift = token_pos(sq.len[s], max(end, 0), 0);
    }
    const int pos = shift + t;
    if (t < a || t >= end || pos < 0 || (pos >> kv.psh) >= sq.cols) continue;
    const int pid = sq.table[(long)s * sq.ldt + (pos >> kv.psh)];
    if ((unsigned)pid >= (unsigned)kv.n_pages) continue;
    row[p] = (((long)pid * kv.hkv + h) << kv.psh) + (pos & ((1 << kv.psh) - 1));
  }
}

// LPR lanes a row, 8 elements each (16 bytes of input); a block takes PASS * 256 / LPR consecutive tokens of one head,
// whose slots and scales are neighbours. KVM 0: same 16-bit type, 1: int8, 2: e4m3.
template <int LPR, int KVM, bool BF, int PASS>
__global__ __launch_bounds__(256) void k_kv_write(Kv kv, Seqs sq, const char* __restrict__ k,
                                                  const char* __restrict__ v, long ldk, long ldv) {
  constexpr int RPB = 256 / LPR;
  const int h = blockIdx.x % kv.hkv, lane = threadIdx.x % LPR;
  const int t0 = (blockIdx.x / kv.hkv) * (RPB * PASS) + threadIdx.x / LPR;
  const bool act = lane * 8 < kv.d;
  uint4 x[PASS][2];
#pragma unroll
  for (int p = 0; p < PASS; ++p) {
    const int t = t0 + p * RPB;
    x[p][0] = x[p][1] = make_uint4(0, 0, 0, 0);
    if (t < sq.T && act) {
      x[p][0] = *reinterpret_cast<const uint4*>(k + ((long)t * ldk + (long)h * kv.d + lane * 8) * 2);
      x[p][1] = *reinterpret_cast<const uint4*>(v + ((long)t * ldv + (long)h * kv.d + lane * 8) * 2);
    }
  }
  long row[PASS];
  find_rows<LPR, PASS>(kv, sq, h, t0, RPB, row);
#pragma unroll
  for (int p = 0; p < PASS; ++p)
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      char* dst = m ? kv.v : kv.k;
      const uint4 xv = x[p][m];
      if constexpr (KVM == 0) {
        if (row[p] >= 0 && act) *reinterpret_cast<uint4*>(dst + (row[p] * kv.d + lane * 8) * 2) = xv;
      } else {
        // the largest magnitude, as a bit pattern: those of 16-bit values ascend with them, infinity and NaN on top
        typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
        const uint32_t u[4] = {xv.x, xv.y, xv.z, xv.w};
        float f[8];
        u16x2 mx = {0, 0};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          f[2 * i] = lo16<BF>(u[i]);
          f[2 * i + 1] = hi16<BF>(u[i]);
          mx = __builtin_elementwise_max(mx, __builtin_bit_cast(u16x2, u[i] & 0x7FFF7FFFu));
        }
        const uint32_t big = group_max<LPR>((uint32_t)max(mx.x, mx.y));
        // a row that holds an infinity or NaN has no scale: it is stored as NaN (scale NaN, codes 0)
        const bool fin = big < (BF ? 0x7F80u : 0x7C00u);
        float sc = over_top<KVM == 1 ? 127 : 448>(lo16<BF>(big));
        if (sc < KV_MIN_SCALE) sc = 0.f;
        const bool some = fin && sc > 0.f;
        uint2 c = encode8<KVM == 2, BF>(f, some ? sc : 1.f);
        if (!some) c = make_uint2(0, 0);
        if (row[p] >= 0 && act) {
          *reinterpret_cast<uint2*>(dst + row[p] * kv.d + lane * 8) = c;
          if (lane == 0) (m ? kv.vs : kv.ks)[row[p]] = fin ? sc : __uint_as_float(0x7FC00000u);
        }
      }
    }
}

// The other way: value = code * scale in fp32, rounded once to the 16-bit type (16-bit caches: copied).
template <int LPR, int KVM, bool BF, int PASS>
__global__ __launch_bounds__(256) void k_kv_read(Kv kv, Seqs sq, char* __restrict__ k, char* __restrict__ v, long ldk,
                                                 long ldv) {
  constexpr int RPB = 256 / LPR;
  const int h = blockIdx.x % kv.hkv, lane = threadIdx.x % LPR;
  const int t0 = (blockIdx.x / kv.hkv) * (RPB * PASS) + threadIdx.x / LPR;
  const bool act = lane * 8 < kv.d;
  long row[PASS];
  find_rows<LPR, PASS>(kv, sq, h, t0, RPB, row);
  uint4 x[PASS][2];
  float sc[PASS][2];
#pragma unroll
  for (int p = 0; p < PASS; ++p)
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      const char* src = m ? kv.v : kv.k;
      x[p][m] = make_uint4(0, 0, 0, 0);
      sc[p][m] = 0.f;
      if (row[p] < 0 || !act) continue;
      if constexpr (KVM == 0) {
        x[p][m] = *reinterpret_cast<const uint4*>(src + (row[p] * kv.d + lane * 8) * 2);
      } else {
        const uint2 c = *reinterpret_cast<const uint2*>(src + row[p] * kv.d + lane * 8);
        x[p][m].x = c.x;
        x[p][m].y = c.y;
        sc[p][m] = (m ? kv.vs : kv.ks)[row[p]];
      }
    }
#pragma unroll
  for (int p = 0; p < PASS; ++p)
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      if (row[p] < 0 || !act) continue;
      uint4 o = x[p][m];
      if constexpr (KVM != 0) {
        const uint2 a = codes4<KVM == 2>(o.x), b = codes4<KVM == 2>(o.y);
        const float g = sc[p][m];
        o.x = pack2<BF>(lo16<false>(a.x) * g, hi16<false>(a.x) * g);
        o.y = pack2<BF>(lo16<false>(a.y) * g, hi16<false>(a.y) * g);
        o.z = pack2<BF>(lo16<false>(b.x) * g, hi16<false>(b.x) * g);
        o.w = pack2<BF>(lo16<false>(b.y) * g, hi16<false>(b.y) * g);
      }
      const int t = t0 + p * RPB;
      *reinterpret_cast<uint4*>((m ? v : k) + ((long)t * (m ? ldv : ldk) + (long)h * kv.d + lane * 8) * 2) = o;
    }
}

template <int LPR>
hipError_t go(bool write, const Kv& kv, int kvm, bool bf, const Seqs& sq, char* k, char* v, long ldk, long ldv,
              hipStream_t st) {
  constexpr int RPB = 256 / LPR;
  // two tokens a thread where that still leaves 32 workgroups a compute unit (54000 tokens of 40 heads read from e4m3:
  // 155 -> 134 us; 4000 tokens written to e4m3 in 10000 workgroups: 28.1 us, in 5000 28.6, 6400 in 16000 47.3, in 8000 50.3)
  const long one = (long)((sq.T + RPB - 1) / RPB) * kv.hkv;
  const bool two = one >= 2 * 32 * 256;
  const int per = two ? 2 * RPB : RPB;
  const dim3 grid((unsigned)((sq.T + per - 1) / per) * kv.hkv);
#define GO(K, KVM, BF)                                                                                        \
  do {                                                                                                        \
    if (two) hipLaunchKernelGGL((K<LPR, KVM, BF, 2>), grid, dim3(256), 0, st, kv, sq, k, v, ldk, ldv);        \
    else hipLaunchKernelGGL((K<LPR, KVM, BF, 1>), grid, dim3(256), 0, st, kv, sq, k, v, ldk, ldv);            \
  } while (0)
#define PICK(K)                                    \
  if (kvm == 0) GO(K, 0, false);                   \
  else if (kvm == 1 && !bf) GO(K, 1, false);       \
  else if (kvm == 1) GO(K, 1, true);               \
  else if (!bf) GO(K, 2, false);                   \
  else GO(K, 2, true);
  if (write) { PICK(k_kv_write) } else { PICK(k_kv_read) }
#undef PICK
#undef GO
  return hipGetLastError();
}

hipError_t pick(bool write, const Kv& kv, int kvt, const Seqs& sq, void* k, void* v, int xt, long ldk, long ldv,
                hipStream_t st) {
  const int kvm = kvt == T_I8 ? 1 : kvt == T_E4M3 ? 2 : 0;
  const bool bf = xt == T_BF16;
  char *kc = (char*)k, *vc = (char*)v;
  if (kv.d <= 32) return go<4>(write, kv, kvm, bf, sq, kc, vc, ldk, ldv, st);
  if (kv.d <= 64) return go<8>(write, kv, kvm, bf, sq, kc, vc, ldk, ldv, st);
  if (kv.d <= 128) return go<16>(write, kv, kvm, bf, sq, kc, vc, ldk, ldv, st);
  return go<32>(write, kv, kvm, bf, sq, kc, vc, ldk, ldv, st);
}

}  // namespace

hipError_t sffn_launch_kv_write(const Kv& kv, int kvt, const Seqs& sq, const void* k, const void* v, int xt, long ldk,
                                long ldv, hipStream_t st) {
  return pick(true, kv, kvt, sq, const_cast<void*>(k), const_cast<void*>(v), xt, ldk, ldv, st);
}
hipError_t sffn_launch_kv_read(const Kv& kv, int kvt, const Seqs& sq, void* k, void* v, int xt, long ldk, long ldv,
                               hipStream_t st) {
  return pick(false, kv, kvt, sq, k, v, xt, ldk, ldv, st);
}
