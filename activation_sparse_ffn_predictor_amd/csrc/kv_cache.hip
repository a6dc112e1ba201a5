// Paged K/V cache: new tokens written (as they are or quantised to 8 bits), and a range of tokens read back.
//
// Both are bound by memory, each byte moved once; a row of a head is a few lanes' work, so that its maximum needs no LDS
// and neighbouring tokens of a head fill neighbouring slots. Measured: 4000 tokens of 40 heads of 128 written in 32.5 us as
// bf16 (5.0 TB/s) and in 28 to 31 as e4m3 (4.0 to 4.4 TB/s; 24.7 us without the encoding, which is what then bounds it); 54000 tokens
// read from e4m3 to bf16, 703 MB in 134 to 143 us (box to box; 5.0 to 5.3 TB/s).
#include "codes.h"

using namespace sffn;

namespace {

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
