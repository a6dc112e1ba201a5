// Paged K/V cache: new tokens written (as they are or quantised to 8 bits), and a range of tokens read back.
#include "attn.h"

using namespace sffn;

namespace {

constexpr int TOK = 16;     // consecutive tokens of one head that a block takes: their slots and scales are neighbours

// x / s rounded so that a later rounding to fewer bits is that of the exact quotient: the fp32 quotient is cut
// towards zero and its last bit set if anything was cut off (s > 0, quotient far from overflow).
__device__ __forceinline__ float div_sticky(float x, float s) {
  float q = x / s;
  const float e = fmaf(-q, s, x);                            // exact remainder of the rounded quotient
  if (e != 0.f && q != 0.f) {
    uint32_t b = __float_as_uint(q);
    if ((e < 0.f) != (q < 0.f)) b -= 1;                      // |q| was rounded up: back to the value below
    q = __uint_as_float(b | 1u);
  }
  return q;
}

template <bool E4M3>
__device__ __forceinline__ uint32_t encode4(const float* v) {
  if constexpr (E4M3) {
    int u = __builtin_amdgcn_cvt_pk_fp8_f32(v[0], v[1], 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(v[2], v[3], u, true);
  } else {
    uint32_t u = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) u |= (uint32_t)((int)rintf(v[i]) & 255) << (8 * i);
    return u;
  }
}

// The slot of token t in the cache (row index of head 0's slot 0 of its page is pid * hkv << psh), or false.
__device__ __forceinline__ bool find_slot(const Kv& kv, const Seqs& sq, int s, int t, int& pid, int& slot) {
  if (s >= sq.S) return false;
  const int a = sq.cu[s], n = sq.cu[s + 1] - a, pos = sq.len[s] - n + (t - a);
  if (t < a || pos < 0 || (pos >> kv.psh) >= sq.cols) return false;
  pid = sq.table[(long)s * sq.ldt + (pos >> kv.psh)];
  slot = pos & ((1 << kv.psh) - 1);
  return (unsigned)pid < (unsigned)kv.n_pages;
}

// LPR lanes a row, 8 elements each (16 bytes of input). KVM 0: same 16-bit type, 1: int8, 2: e4m3.
template <int LPR, int KVM, bool BF>
__global__ __launch_bounds__(256) void k_kv_write(Kv kv, Seqs sq, const char* __restrict__ k,
                                                  const char* __restrict__ v, long ldk, long ldv) {
  constexpr int RPB = 256 / LPR, PASS = RPB < TOK ? TOK / RPB : 1;   // rows a block holds at once
  const int h = blockIdx.x % kv.hkv, lane = threadIdx.x % LPR;
  const bool act = lane * 8 < kv.d;
#pragma unroll
  for (int ps = 0; ps < PASS; ++ps) {
    const int row = ps * RPB + threadIdx.x / LPR;
    const int t = (blockIdx.x / kv.hkv) * (RPB < TOK ? TOK : RPB) + row;
    const bool in = t < sq.T && act;
    uint4 x[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
    if (in) {
      x[0] = *reinterpret_cast<const uint4*>(k + ((long)t * ldk + (long)h * kv.d + lane * 8) * 2);
      x[1] = *reinterpret_cast<const uint4*>(v + ((long)t * ldv + (long)h * kv.d + lane * 8) * 2);
    }
    const int s = find_seq<LPR>(sq.cu, sq.S, t);
    int pid = 0, slot = 0;
    const bool ok = find_slot(kv, sq, s, t, pid, slot) && t < sq.T;
    const long r = (((long)pid * kv.hkv + h) << kv.psh) + slot;
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      char* dst = m ? kv.v : kv.k;
      if constexpr (KVM == 0) {
        if (ok && in) *reinterpret_cast<uint4*>(dst + (r * kv.d + lane * 8) * 2) = x[m];
      } else {
        const uint32_t u[4] = {x[m].x, x[m].y, x[m].z, x[m].w};
        float f[8], big = 0.f;
        bool bad = false;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          f[2 * i] = lo16<BF>(u[i]);
          f[2 * i + 1] = hi16<BF>(u[i]);
          big = fmaxf(big, fmaxf(fabsf(f[2 * i]), fabsf(f[2 * i + 1])));
          bad |= nonfinite2<BF>(u[i]) != 0;
        }
        if (bad) big = __uint_as_float(0x7F800000u);
#pragma unroll
        for (int o = 1; o < LPR; o <<= 1) big = fmaxf(big, __shfl_xor(big, o, WAVE));
        // a row that holds an infinity or NaN has no scale: it is stored as NaN (scale NaN, codes 0)
        const bool fin = big < __uint_as_float(0x7F800000u);
        float sc = big / (KVM == 1 ? 127.f : 448.f);
        if (sc < KV_MIN_SCALE) sc = 0.f;
        uint2 c = make_uint2(0, 0);
        if (fin && sc > 0.f) {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            f[i] = fminf(fmaxf(div_sticky(f[i], sc), KVM == 1 ? -127.f : -448.f), KVM == 1 ? 127.f : 448.f);
          c = make_uint2(encode4<KVM == 2>(f), encode4<KVM == 2>(f + 4));
        }
        if (ok && in) {
          *reinterpret_cast<uint2*>(dst + r * kv.d + lane * 8) = c;
          if (lane == 0) (m ? kv.vs : kv.ks)[r] = fin ? sc : __uint_as_float(0x7FC00000u);
        }
      }
    }
  }
}

// The other way: value = code * scale in fp32, rounded once to the 16-bit type (16-bit caches: copied).
template <int LPR, int KVM, bool BF>
__global__ __launch_bounds__(256) void k_kv_read(Kv kv, Seqs sq, char* __restrict__ k, char* __restrict__ v, long ldk,
                                                 long ldv) {
  constexpr int RPB = 256 / LPR, PASS = RPB < TOK ? TOK / RPB : 1;
  const int h = blockIdx.x % kv.hkv, lane = threadIdx.x % LPR;
  const bool act = lane * 8 < kv.d;
#pragma unroll
  for (int ps = 0; ps < PASS; ++ps) {
    const int t = (blockIdx.x / kv.hkv) * (RPB < TOK ? TOK : RPB) + ps * RPB + threadIdx.x / LPR;
    const int s = find_seq<LPR>(sq.cu, sq.S, t);
    int pid = 0, slot = 0;
    if (!find_slot(kv, sq, s, t, pid, slot) || t >= sq.T || !act) continue;
    const long r = (((long)pid * kv.hkv + h) << kv.psh) + slot;
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      const char* src = m ? kv.v : kv.k;
      uint4 o;
      if constexpr (KVM == 0) {
        o = *reinterpret_cast<const uint4*>(src + (r * kv.d + lane * 8) * 2);
      } else {
        const uint2 c = *reinterpret_cast<const uint2*>(src + r * kv.d + lane * 8);
        const float sc = (m ? kv.vs : kv.ks)[r];
        const uint2 a = codes4<KVM == 2>(c.x), b = codes4<KVM == 2>(c.y);
        o.x = pack2<BF>(lo16<false>(a.x) * sc, hi16<false>(a.x) * sc);
        o.y = pack2<BF>(lo16<false>(a.y) * sc, hi16<false>(a.y) * sc);
        o.z = pack2<BF>(lo16<false>(b.x) * sc, hi16<false>(b.x) * sc);
        o.w = pack2<BF>(lo16<false>(b.y) * sc, hi16<false>(b.y) * sc);
      }
      *reinterpret_cast<uint4*>((m ? v : k) + ((long)t * (m ? ldv : ldk) + (long)h * kv.d + lane * 8) * 2) = o;
    }
  }
}

template <int LPR>
hipError_t go(bool write, const Kv& kv, int kvm, bool bf, const Seqs& sq, char* k, char* v, long ldk, long ldv,
              hipStream_t st) {
  constexpr int PER = 256 / LPR < TOK ? TOK : 256 / LPR;
  const dim3 grid((unsigned)((sq.T + PER - 1) / PER) * kv.hkv);
#define GO(K, KVM, BF) hipLaunchKernelGGL((K<LPR, KVM, BF>), grid, dim3(256), 0, st, kv, sq, k, v, ldk, ldv)
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
