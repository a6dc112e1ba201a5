// Attention over the paged cache for few rows a K/V head (single tokens, a few drafted ones).
//
// S^T = K Q^T and O^T = V^T P^T on the matrix cores (16x16x32): a lane's column is one row of Q in both products, so
// a row's maximum and sum live in the lanes that hold its scores, and the scores of a lane are, as they are, its part
// of the next product's operand (the order of the keys within a product is free, V is read in the same one).
//
// Bound by the cache's bytes: a row of K or V is loaded once for all query heads that share it. Each wave runs through
// its own units of 32 keys (no barrier in the loop), K from registers, V through the wave's own LDS tile, read transposed;
// the next unit's loads run under this one's softmax. Occupancy (two or three waves a SIMD) hides the rest, so nothing
// may be spilled: a spilled value's load would wait for the cache loads in flight. Measured: one token of two sequences
// of 131072, 64 heads on 8 of 128, e4m3, 554 MB in 104 us with the join (5.3 TB/s; a large read reaches 5.9); fp16, 1.07 GB
// in 187 us (5.7 TB/s); 32 ragged sequences to 6000 tokens, 40 heads, int8, 892 MB in 169 to 176 us; 48 sequences of up to 4
// drafts, 128 heads on 8 of 64, bf16, window 4096, 385 MB in 80 us (4.8 TB/s). One sequence of 500 tokens, 2 MB: 9.6 us,
// of which 5 are a call on 32 tokens: the rest is one compute unit's loads of a head's 256 KB. From 769 keys on (385
// for sizes over 128) the keys are spread and joined (13 us up to 4000; in one workgroup 700 take 11.7, 1000 take 14.2).
#include "attn.h"

using namespace sffn;

namespace {

// A 16-byte slot of V's tile in LDS: key's 16-byte chunk c goes to slot c ^ few_swz(key), so that the 16 (32) rows
// that a transposing read touches at one column spread over the banks.
template <int RB>   // bytes of a tile row
__device__ __forceinline__ int few_swz(int key, bool codes) {
  if (codes) return RB >= 256 ? key & 15 : RB == 128 ? (key >> 1) & 7 : (key >> 2) & 3;
  return RB >= 256 ? (key & 7) << 1 : ((key >> 1) & 3) << 1;
}

// The sequence and share of a block.
struct Place {
  Seq sq;
  Units un;
  int n, rows, p0, p1, hk, s, split, used, u0, u1;
};

// KVM 0: cache of the query's 16-bit type, 1: int8, 2: e4m3 (both computed in fp16: codes are exact there, and bf16
// queries are scaled by one power of two into fp16's range). DP: head size padded to 64, 128 or 256. QB: 16-row tiles.
template <bool BF, int KVM, int DP, int QB, int NW>
__device__ __forceinline__ void few_rows(const AttnArgs& a, const Place& pl, char* lds, float (*mlw)[2], uint4* qlds) {
  constexpr int NT = NW * 64;
  constexpr bool C8 = KVM != 0, CB = BF && !C8;
  constexpr int EB = C8 ? 1 : 2, RB = DP * EB, KS = DP / 32, DB = DP / 16, CPR = RB / 16;   // chunks a row
  constexpr int KL = RB / 64;                      // 16-byte K loads of a lane per 16 keys
  constexpr int RPI = 64 / CPR, VL = 16 / RPI;     // V rows a load instruction covers; V loads per 16 keys
  constexpr int VT = 32 * RB, OS = DP + 4;         // V tile of a wave; row stride of the merge (floats)
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), l = threadIdx.x & 63, g4 = l >> 4, ql = l & 15;
  const int d = a.kv.d, G = a.G, hk = pl.hk, s = pl.s, rows = pl.rows, p0 = pl.p0, p1 = pl.p1, used = pl.used;
  const int split = pl.split, u1 = pl.u1;
  const Seq sq = pl.sq;
  const Units un = pl.un;

  // queries: 8 consecutive elements of row ql per product step
  uint4 qf[QB][KS];
  int pos[QB];
  float c = a.c;
#pragma unroll
  for (int qb = 0; qb < QB; ++qb) {
    const int r = qb * 16 + ql, i = r / G, g = r - i * G;
    pos[qb] = r < rows ? p0 + i : p1;              // rows past the last compute along and are dropped
    const char* qp = a.q + ((long)(sq.q0 + i) * a.ldq + (long)(hk * G + g) * d) * 2;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      const int ch = C8 ? ((ks >> 1) * 4 + g4) * 2 + (ks & 1) : ks * 4 + g4;
      qf[qb][ks] = r < rows && ch * 8 < d ? *reinterpret_cast<const uint4*>(qp + ch * 16) : make_uint4(0, 0, 0, 0);
      if (a.neg) qf[qb][ks] = flip_signs(qf[qb][ks]);
    }
  }
  if constexpr (C8 && BF) {
    float big = 0.f;
#pragma unroll
    for (int qb = 0; qb < QB; ++qb)
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) big = fmaxf(big, absmax8<true>(finite_only<true>(qf[qb][ks])));
    const float up = to_f16_range(wave_max(big), c);
#pragma unroll
    for (int qb = 0; qb < QB; ++qb)
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) qf[qb][ks] = bf16_to_f16(qf[qb][ks], up);
  }

  // Many rows: the query operands (the same in every wave) wait in LDS, 16 bytes a lane, instead of registers. Kept in
  // registers they are spilled, and a spilled value's load waits for the cache loads in flight before it.
  constexpr bool QL = QB * DP >= 256 && QB > 1;
  if constexpr (QL) {
    if (w == 0) {
#pragma unroll
      for (int qb = 0; qb < QB; ++qb)
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) qlds[(qb * KS + ks) * 64 + l] = qf[qb][ks];
    }
    __syncthreads();
  }
  auto q_frag = [&](int qb, int ks) { return QL ? qlds[(qb * KS + ks) * 64 + l] : qf[qb][ks]; };

  float m[QB], ls[QB];
  f32x4 o[QB][DB];
#pragma unroll
  for (int qb = 0; qb < QB; ++qb) {
    m[qb] = -INFINITY;
    ls[qb] = 0.f;
#pragma unroll
    for (int db = 0; db < DB; ++db) o[qb][db] = f32x4{0.f, 0.f, 0.f, 0.f};
  }
  char* vt = lds + w * VT;
  const int* trow = a.sq.table + (long)s * a.sq.ldt;
  const uint32_t dB = (uint32_t)d * EB;

  // One unit's loads. 16 keys share a page; what does not exist (behind the sequence, a bad page) reads as zeros.
  uint4 kr[2][KL], vr[2][VL];
  float4 ksc[2], vsc[2];
  int have[2], page[2];                            // keys of each 16 that exist; page ids of the next unit to load
  auto pages = [&](int u) {
    const int t0 = un.key0(u, FEW_USH);
#pragma unroll
    for (int kb = 0; kb < 2; ++kb) page[kb] = trow[min((t0 + kb * 16) >> a.kv.psh, a.sq.cols - 1)];
  };
  auto load = [&](int u) {
    const int t0 = un.key0(u, FEW_USH);
    int lx = l;                                    // places worked out anew per unit: registers are short
    asm volatile("" : "+v"(lx));
    const uint32_t ko = (lx & 15) * dB + (lx >> 4) * 16, vc = lx % CPR;
    const uint32_t vo = boff(vc * 16 < dB, (lx / CPR) * dB + vc * 16);
#pragma unroll
    for (int kb = 0; kb < 2; ++kb) {
      const int t = t0 + kb * 16, pid = __builtin_amdgcn_readfirstlane(page[kb]);
      have[kb] = (unsigned)pid < (unsigned)a.kv.n_pages ? min(16, max(0, sq.len - t)) : 0;
      const long r = (((long)(have[kb] ? pid : 0) * a.kv.hkv + hk) << a.kv.psh) + (t & ((1 << a.kv.psh) - 1));
      const Buf bk(a.kv.k + r * dB, have[kb] * dB), bv(a.kv.v + r * dB, have[kb] * dB);
#pragma unroll
      for (int i = 0; i < KL; ++i) kr[kb][i] = bk.ld16(boff((i * 4 + (lx >> 4)) * 16 < (int)dB, ko) + i * 64);
#pragma unroll
      for (int i = 0; i < VL; ++i) vr[kb][i] = ld16(bv, vo, i * RPI * dB);
      if constexpr (C8) {
        const Buf sk(a.kv.ks + r, have[kb] * 4), sv(a.kv.vs + r, have[kb] * 4);
        ksc[kb] = sk.ldf4(g4 * 16);
        vsc[kb] = sv.ldf4(g4 * 16);
      }
    }
  };

  bool left_out = false;
  int u = pl.u0 + w;
  if (u < u1) {
    pages(u);
    load(u);
    if (u + NW < u1) pages(u + NW);
  }
  for (; u < u1; u += NW) {
    const int t0 = un.key0(u, FEW_USH), h0 = have[0], h1 = have[1];
    // every key of the unit visible to every row?
    const bool full = h0 + h1 == 32 && t0 + 31 <= p0 && (a.window <= 0 || t0 > p1 - a.window || t0 + 32 <= a.sinks);
    // scores: element (kb, i) is key kb * 16 + 4 * g4 + i of row ql
    f32x4 sc[QB][2];
#pragma unroll
    for (int qb = 0; qb < QB; ++qb)
#pragma unroll
      for (int kb = 0; kb < 2; ++kb) sc[qb][kb] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < KL; ++i)
#pragma unroll
      for (int kb = 0; kb < 2; ++kb) {
        if constexpr (C8) {
          const uint4 t = kr[kb][i];
          const uint2 x0 = codes4<KVM == 2>(t.x), x1 = codes4<KVM == 2>(t.y), x2 = codes4<KVM == 2>(t.z),
                      x3 = codes4<KVM == 2>(t.w);
          const uint4 ka = make_uint4(x0.x, x0.y, x1.x, x1.y), kc = make_uint4(x2.x, x2.y, x3.x, x3.y);
#pragma unroll
          for (int qb = 0; qb < QB; ++qb) {
            sc[qb][kb] = mfma16<false>(ka, q_frag(qb, 2 * i), sc[qb][kb]);
            sc[qb][kb] = mfma16<false>(kc, q_frag(qb, 2 * i + 1), sc[qb][kb]);
          }
        } else {
#pragma unroll
          for (int qb = 0; qb < QB; ++qb) sc[qb][kb] = mfma16<CB>(kr[kb][i], q_frag(qb, i), sc[qb][kb]);
        }
      }
    // V through the wave's own LDS tile (the LDS pipe keeps a wave's accesses in order). Infinities and NaN (NaN codes) in a
    // unit that some row sees only in part are left out here and added where they are seen after the last unit.
    if constexpr (KVM == 2) {
      if (!full) {
        uint32_t n = 0;
#pragma unroll
        for (int kb = 0; kb < 2; ++kb)
#pragma unroll
          for (int i = 0; i < VL; ++i) n |= nan_codes4(vr[kb][i]);
        if (__any(n != 0)) {
          left_out = true;
#pragma unroll
          for (int kb = 0; kb < 2; ++kb)
#pragma unroll
            for (int i = 0; i < VL; ++i) vr[kb][i] = finite_codes4(vr[kb][i]);
        }
      }
    }
    int lv = l;                                    // as in load: worked out anew
    asm volatile("" : "+v"(lv));
#pragma unroll
    for (int kb = 0; kb < 2; ++kb)
#pragma unroll
      for (int i = 0; i < VL; ++i) {
        const int key = kb * 16 + i * RPI + lv / CPR, ch = lv % CPR;
        uint4 t = vr[kb][i];
        if (!C8 && !full) {
          left_out |= (nonfinite2<CB>(t.x) | nonfinite2<CB>(t.y) | nonfinite2<CB>(t.z) | nonfinite2<CB>(t.w)) != 0;
          t = finite_only<CB>(t);
        }
        *reinterpret_cast<uint4*>(vt + key * RB + ((ch ^ few_swz<RB>(key, C8)) << 4)) = t;
      }
    f32x4 inv[2];
    uint32_t vnan = 0;                             // bit kb * 4 + i: the key's V row has no scale
    if constexpr (C8) {
#pragma unroll
      for (int kb = 0; kb < 2; ++kb) {
        const float ka[4] = {ksc[kb].x, ksc[kb].y, ksc[kb].z, ksc[kb].w};
        const float va[4] = {vsc[kb].x, vsc[kb].y, vsc[kb].z, vsc[kb].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const VScale v = v_scale(va[i]);
          inv[kb][i] = v.inv;
          vnan |= va[i] != va[i] ? 1u << (kb * 4 + i) : 0u;
          const float kf = ka[i] * c;
#pragma unroll
          for (int qb = 0; qb < QB; ++qb) sc[qb][kb][i] = fmaf(sc[qb][kb][i], kf, v.lg);
        }
      }
    }
    // the next unit's loads run under the rest of this one (not earlier: both units' registers would be alive)
    __builtin_amdgcn_sched_barrier(0);
    if (u + NW < u1) {
      load(u + NW);
      if (u + 2 * NW < u1) pages(u + 2 * NW);
    }
    const bool slow = C8 && __any(vnan != 0);
    uint4 pf[QB];
#pragma unroll
    for (int qb = 0; qb < QB; ++qb) {
      if (!full) {
        const int hi = pos[qb] - t0 - 4 * g4;
#pragma unroll
        for (int kb = 0; kb < 2; ++kb)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const bool see = (kb * 16 + i <= hi) & (4 * g4 + i < (kb ? h1 : h0));
            sc[qb][kb][i] = see ? sc[qb][kb][i] : -INFINITY;
          }
        if (a.window > 0) {
          const int lo = hi - a.window, sk = a.sinks - t0 - 4 * g4;
#pragma unroll
          for (int kb = 0; kb < 2; ++kb)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              sc[qb][kb][i] = ((kb * 16 + i > lo) | (kb * 16 + i < sk)) ? sc[qb][kb][i] : -INFINITY;
        }
      }
      float top = -INFINITY;
#pragma unroll
      for (int kb = 0; kb < 2; ++kb)
#pragma unroll
        for (int i = 0; i < 4; ++i) top = fmaxf(top, sc[qb][kb][i]);
      top = over32<true>(over16<true>(top));
      if constexpr (!C8) top *= c;
      if (__any(outgrown<CB>(top, m[qb]))) {
        const float mn = new_reference<CB>(top, m[qb]), f = fade(m[qb], mn);
        ls[qb] *= f;
#pragma unroll
        for (int db = 0; db < DB; ++db) o[qb][db] *= f;
        m[qb] = mn;
      }
      const float ms = m[qb] == -INFINITY ? 0.f : m[qb];
      float p[2][4];
#pragma unroll
      for (int kb = 0; kb < 2; ++kb)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          p[kb][i] = exp2_fast(C8 ? sc[qb][kb][i] - ms : fmaf(sc[qb][kb][i], c, -ms));
          ls[qb] = C8 ? fmaf(p[kb][i], inv[kb][i], ls[qb]) : ls[qb] + p[kb][i];
        }
      if (slow) {                            // a V row without a scale: NaN for the rows that see it
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (sc[qb][e >> 2][e & 3] != -INFINITY && (vnan >> e & 1)) p[e >> 2][e & 3] = __uint_as_float(0x7FC00000u);
      }
      // weights of one rounding (half a step of the type each) enter the second product
      pf[qb] = make_uint4(pack2<CB>(p[0][0], p[0][1]), pack2<CB>(p[0][2], p[0][3]), pack2<CB>(p[1][0], p[1][1]),
                          pack2<CB>(p[1][2], p[1][3]));
      if (QL) __builtin_amdgcn_sched_barrier(0);   // one row tile after the other: registers are short
    }
    asm volatile("" ::: "memory");
    auto v_frag = [&](int db) {
      if constexpr (C8) {
        const int j = ql >> 1, key = (j < 4 ? 0 : 12) + g4 * 4 + j;   // rows 0-3: keys g4*4.., 4-7: 16 + g4*4..
        const i32x2 t = __builtin_amdgcn_ds_read_tr8_b64_v2i32((__attribute__((address_space(3))) i32x2*)(
            vt + key * RB + ((db ^ few_swz<RB>(key, true)) << 4) + (ql & 1) * 8));
        const uint2 x0 = codes4<KVM == 2>((uint32_t)t.x), x1 = codes4<KVM == 2>((uint32_t)t.y);
        return make_uint4(x0.x, x0.y, x1.x, x1.y);
      } else {
        const int key = g4 * 4 + (ql >> 2), ch = db * 2 + ((ql & 3) >> 1);
        const int at = ((ch ^ few_swz<RB>(key, false)) << 4) + (ql & 1) * 8;   // keys 16 apart: the same slot
        const fp16x4 t0v = __builtin_amdgcn_ds_read_tr16_b64_v4f16(
            (__attribute__((address_space(3))) fp16x4*)(vt + key * RB + at));
        const fp16x4 t1v = __builtin_amdgcn_ds_read_tr16_b64_v4f16(
            (__attribute__((address_space(3))) fp16x4*)(vt + (key + 16) * RB + at));
        const uint2 y0 = __builtin_bit_cast(uint2, t0v), y1 = __builtin_bit_cast(uint2, t1v);
        return make_uint4(y0.x, y0.y, y1.x, y1.y);
      }
    };
#pragma unroll
    for (int db = 0; db < DB; ++db) {
      const uint4 vf = v_frag(db);
#pragma unroll
      for (int qb = 0; qb < QB; ++qb) o[qb][db] = mfma16<CB>(vf, pf[qb], o[qb][db]);
    }
    asm volatile("" ::: "memory");
  }

  if (KVM != 1 && __any(left_out)) {
    // once more through the keys of the units that some row sees only in part
#pragma unroll 1
    for (u = pl.u0 + w; u < u1; u += NW) {
      const int t0 = un.key0(u, FEW_USH);
      int hv[2], pid[2];
#pragma unroll
      for (int kb = 0; kb < 2; ++kb) {
        pid[kb] = trow[min((t0 + kb * 16) >> a.kv.psh, a.sq.cols - 1)];
        hv[kb] = (unsigned)pid[kb] < (unsigned)a.kv.n_pages ? min(16, max(0, sq.len - (t0 + kb * 16))) : 0;
      }
      if (hv[0] + hv[1] == 32 && t0 + 31 <= p0 && (a.window <= 0 || t0 > p1 - a.window || t0 + 32 <= a.sinks)) continue;
#pragma unroll
      for (int kb = 0; kb < 2; ++kb)
#pragma unroll 1
        for (int kk = 0; kk < hv[kb]; ++kk) {
          const int j = t0 + kb * 16 + kk;
          const char* row = a.kv.v + ((((long)pid[kb] * a.kv.hkv + hk) << a.kv.psh) + (j & ((1 << a.kv.psh) - 1))) * dB;
#pragma unroll
          for (int db = 0; db < DB; ++db) {
            const int d0 = db * 16 + g4 * 4;
            if (d0 >= d) continue;
            float f[4];
            if constexpr (C8) {
              const uint32_t v = nan_codes(*reinterpret_cast<const uint32_t*>(row + d0));
#pragma unroll
              for (int i = 0; i < 4; ++i) f[i] = v >> (8 * i + 7) & 1 ? __uint_as_float(0x7FC00000u) : 0.f;
            } else {
              const uint2 v = *reinterpret_cast<const uint2*>(row + d0 * 2);
              f[0] = lo16<CB>(v.x), f[1] = hi16<CB>(v.x), f[2] = lo16<CB>(v.y), f[3] = hi16<CB>(v.y);
            }
#pragma unroll
            for (int qb = 0; qb < QB; ++qb) {
              const bool see = j <= pos[qb] && (a.window <= 0 || j > pos[qb] - a.window || j < a.sinks);
#pragma unroll
              for (int i = 0; i < 4; ++i) o[qb][db][i] += see && !(fabsf(f[i]) < INFINITY) ? f[i] : 0.f;
            }
          }
        }
    }
  }

  // the waves' parts joined in wave order
  __syncthreads();
  float* om = reinterpret_cast<float*>(lds);
#pragma unroll
  for (int qb = 0; qb < QB; ++qb) {
    const float t = over32<false>(over16<false>(ls[qb]));
    if (g4 == 0) {
      mlw[w * QB * 16 + qb * 16 + ql][0] = m[qb];
      mlw[w * QB * 16 + qb * 16 + ql][1] = t;
    }
#pragma unroll
    for (int db = 0; db < DB; ++db)
      *reinterpret_cast<f32x4*>(om + ((w * QB + qb) * 16 + ql) * OS + db * 16 + g4 * 4) = o[qb][db];
  }
  __syncthreads();
  for (int e = threadIdx.x; e < rows * (DP / 8); e += NT) {
    const int r = e / (DP / 8), d0 = (e % (DP / 8)) * 8, i = r / G, g = r - i * G;
    if (d0 >= d) continue;
    float M = -INFINITY, L = 0.f, acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int k = 0; k < NW; ++k) M = fmaxf(M, mlw[k * QB * 16 + r][0]);
    const float ms = M == -INFINITY ? 0.f : M;
#pragma unroll
    for (int k = 0; k < NW; ++k) {
      const float f = fade(mlw[k * QB * 16 + r][0], ms);
      L = fmaf(mlw[k * QB * 16 + r][1], f, L);
      const float* src = om + ((k * QB) * 16 + r) * OS + d0;
#pragma unroll
      for (int j = 0; j < 8; ++j) acc[j] = fmaf(src[j], f, acc[j]);
    }
    if constexpr (!C8) {
      const float all = ((acc[0] + acc[1]) + (acc[2] + acc[3])) + ((acc[4] + acc[5]) + (acc[6] + acc[7]));
      if (all != all && L == L) {                  // perhaps a lost infinity: once more through what the row sees
        const int pr = p0 + i;
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[j] = lose_nan(acc[j]);
#pragma unroll 1
        for (int t = pl.u0; t < u1; ++t) {
          const int t0 = un.key0(t, FEW_USH);
#pragma unroll 1
          for (int j = t0; j < min(t0 + 32, min(sq.len, pr + 1)); ++j) {
            const int pid = trow[min(j >> a.kv.psh, a.sq.cols - 1)];
            if ((unsigned)pid >= (unsigned)a.kv.n_pages || !(a.window <= 0 || j > pr - a.window || j < a.sinks)) continue;
            const uint4 v = *reinterpret_cast<const uint4*>(
                a.kv.v + ((((long)pid * a.kv.hkv + hk) << a.kv.psh) + (j & ((1 << a.kv.psh) - 1))) * dB + d0 * 2);
            const uint32_t x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const float f = k & 1 ? hi16<CB>(x[k >> 1]) : lo16<CB>(x[k >> 1]);
              acc[k] += fabsf(f) < INFINITY ? 0.f : f;
            }
          }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[j] = find_lost(acc[j]);
      }
    }
    const long row = (long)(sq.q0 + i) * a.hq + hk * G + g;
    if (used == 1) {
      const float iv = L == 0.f ? 0.f : 1.f / L;   // no key was visible: 0
#pragma unroll
      for (int j = 0; j < 8; ++j) acc[j] *= iv;
      *reinterpret_cast<uint4*>(a.out + ((long)(sq.q0 + i) * a.ldo + (long)(hk * G + g) * d + d0) * 2) =
          make_uint4(pack2<BF>(acc[0], acc[1]), pack2<BF>(acc[2], acc[3]), pack2<BF>(acc[4], acc[5]),
                     pack2<BF>(acc[6], acc[7]));
      if (a.lse && d0 == 0) a.lse[row] = log_sum(M, L);
    } else {
      float* po = a.po + (row * a.ns + split) * d + d0;
      reinterpret_cast<float4*>(po)[0] = make_float4(acc[0], acc[1], acc[2], acc[3]);
      reinterpret_cast<float4*>(po)[1] = make_float4(acc[4], acc[5], acc[6], acc[7]);
      if (d0 == 0) a.pml[row * a.ns + split] = make_float2(M, L);
    }
  }
}

// One sequence, K/V head and share of the keys; a sequence with fewer rows than the call's most takes fewer tiles.
template <bool BF, int KVM, int DP, int QB, int NW>
__global__ __launch_bounds__(NW * 64, DP <= 128 ? 2 : 1) void k_attn_few(AttnArgs a) {
  constexpr int VT = NW * 32 * DP * (KVM ? 1 : 2), MG = NW * QB * 16 * (DP + 4) * 4;
  __shared__ __align__(16) char lds[VT > MG ? VT : MG];
  __shared__ float mlw[NW * QB * 16][2];
  __shared__ uint4 qlds[QB * DP >= 256 && QB > 1 ? QB * DP * 2 : 1];   // QB * DP / 32 operands of 64 lanes
  Place pl;
  pl.split = blockIdx.x;
  pl.hk = blockIdx.y;
  pl.s = blockIdx.z;
  pl.sq = load_seq(a.sq, pl.s, a.kv.psh);
  pl.n = min(pl.sq.n, a.max_q);
  pl.rows = pl.n * a.G;
  if (pl.rows == 0) return;
  pl.p0 = pl.sq.p0;                                // positions of the first and last new token
  pl.p1 = pl.p0 + pl.n - 1;
  pl.un = key_units(pl.p0, pl.p1, pl.sq.len, a.window, a.sinks, FEW_USH);
  const int per = share_units(pl.un.tot, a.ns, few_least(DP), FEW_STEP);
  pl.used = max(1, (pl.un.tot + per - 1) / per);
  if (pl.split >= pl.used) return;
  pl.u0 = pl.split * per;
  pl.u1 = min(pl.un.tot, pl.u0 + per);
  if (QB >= 4 && pl.rows > 32) few_rows<BF, KVM, DP, QB >= 4 ? 4 : 1, NW>(a, pl, lds, mlw, qlds);
  else if (QB >= 2 && pl.rows > 16) few_rows<BF, KVM, DP, QB >= 2 ? 2 : 1, NW>(a, pl, lds, mlw, qlds);
  else few_rows<BF, KVM, DP, 1, NW>(a, pl, lds, mlw, qlds);
}

}  // namespace

// Up to as many rows as the accumulators leave registers for (the tile kernel on 64 rows of size 64, bf16, 48 windowed
// sequences of 4 drafts: 142 us, this one 86).
int sffn_attn_few_rows(int d) { return d <= 64 ? 64 : d <= 128 ? 32 : 16; }

hipError_t sffn_launch_attn_few(const AttnArgs& a, int qt, int kvt, hipStream_t st) {
  const dim3 grid(a.ns, a.kv.hkv, a.sq.S);
  const bool bf = qt == T_BF16;
  const int kvm = kvt == T_I8 ? 1 : kvt == T_E4M3 ? 2 : 0;
  const int rows = a.max_q * a.G;
  // eight waves a workgroup where there is at most one workgroup a compute unit (500 keys, 64 heads on 8: 12.2 us with four
  // waves, two shares and a join, 9.6 with eight and no join); four otherwise, two workgroups a compute unit. Four for
  // 16-bit rows of head sizes over 128 too: eight leave a wave too few registers there (30 sequences of 700, size 256, fp16:
  // 50 us with eight, 39.5 with four; int8, 16 of 1000: 21 and 23)
  const bool wide = (a.kv.d <= 128 || kvm) && (long)grid.x * grid.y * grid.z <= 256;
#define GO(BF, KVM, DP, QB, NW) hipLaunchKernelGGL((k_attn_few<BF, KVM, DP, QB, NW>), grid, dim3(NW * 64), 0, st, a)
#define TYPES(DP, QB, NW)                                                                                          \
  if (bf) {                                                                                                        \
    if (kvm == 0) GO(true, 0, DP, QB, NW); else if (kvm == 1) GO(true, 1, DP, QB, NW); else GO(true, 2, DP, QB, NW); \
  } else {                                                                                                         \
    if (kvm == 0) GO(false, 0, DP, QB, NW); else if (kvm == 1) GO(false, 1, DP, QB, NW); else GO(false, 2, DP, QB, NW); \
  }
#define WAVES(DP, QB) if (wide) { TYPES(DP, QB, 8) } else { TYPES(DP, QB, 4) }
  if (a.kv.d <= 64) { if (rows > 32) { WAVES(64, 4) } else if (rows > 16) { WAVES(64, 2) } else { WAVES(64, 1) } }
  else if (a.kv.d <= 128) { if (rows > 16) { WAVES(128, 2) } else { WAVES(128, 1) } }
  else if (wide) {
    if (bf) { if (kvm == 1) GO(true, 1, 256, 1, 8); else GO(true, 2, 256, 1, 8); }
    else { if (kvm == 1) GO(false, 1, 256, 1, 8); else GO(false, 2, 256, 1, 8); }
  } else { TYPES(256, 1, 4) }
#undef WAVES
#undef TYPES
#undef GO
  return hipGetLastError();
}
