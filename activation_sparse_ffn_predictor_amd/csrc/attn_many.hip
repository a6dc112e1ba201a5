// Attention over the paged cache for many rows a K/V head (chunks of a prompt), and the join of split results.
//
// As the few-row kernel, S^T = K Q^T and O^T = V^T P^T, with 32x32x16 products: a lane's column is one of the wave's
// 32 rows, its 16 scores per 32 keys are that row's, and they are the second product's operand as they are. Four
// waves (128 rows of one K/V head, the query heads of a token next to each other) share tiles of 64 keys in LDS.
//
// Bound by the matrix cores and the power they draw: 4096 tokens of 64 heads on 8 of 128 over 8192, 825 GFLOP, take 850 to
// 960 us in fp16 (box to box; 859 to 970 TFLOP/s where a large fp16 product reaches 1221 to 1289) and 807 to 850 in bf16 (970
// to 1022, where one of bf16 reaches 1376 to 1389), with the matrix cores busy 48% of the time at a mean clock of about 1.8 GHz and no LDS conflicts. Wave priorities around the
// products, reading operands further ahead, and computing the next tile's scores under this one's softmax changed that by
// -2 to +2%. int8 and e4m3: 1.0 to 1.2 ms, with the codes widened once a workgroup on their way into LDS. What was worth it: tiles
// straight to LDS, a maximum that seldom moves, no second copy of the product loops (2557 -> 870 us).
#include "attn.h"

using namespace sffn;

namespace {

constexpr int NT = 256, NW = 4;
constexpr int NOT_DS = 0x41E;    // scheduling barrier that LDS accesses do not cross, anything else may

template <int DP>
__device__ __forceinline__ int swz_k(int key) {   // slot of K's 16-byte chunk c: c ^ swz (16 rows, one column: all banks)
  return DP >= 128 ? key & 15 : (key >> 1) & 7;
}
template <int DP>
__device__ __forceinline__ int swz_v(int key) {   // V: 4 rows x 64 bytes of a transposing read on all banks
  return DP >= 128 ? (key & 3) << 2 : ((key >> 1) & 1) << 2;
}

// Row tile -> sequence: tiles of the sequences in order, each ceil(n * G / MANY_ROWS). Every wave searches for
// itself, 64 sequences at a step.
__device__ __forceinline__ bool find_tile(const AttnArgs& a, int want, int& s, int& tile, int& ntiles) {
  int before = 0;
  const int l = threadIdx.x & 63;
  for (int s0 = 0; s0 < a.sq.S; s0 += 64) {
    int nt = 0;
    if (s0 + l < a.sq.S) {
      const int x = min(max(a.sq.cu[s0 + l], 0), a.sq.T), y = min(a.sq.cu[s0 + l + 1], a.sq.T);
      nt = (int)(((long)min(max(y - x, 0), a.max_q) * a.G + MANY_ROWS - 1) / MANY_ROWS);
    }
    int inc = nt;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int t = __shfl_up(inc, o, WAVE);
      if (l >= o) inc += t;
    }
    const int all = __builtin_amdgcn_readlane(inc, 63);
    if (want < before + all) {
      const uint64_t hit = __ballot(before + inc > want);
      const int k = __ffsll((unsigned long long)hit) - 1;
      s = s0 + k;
      ntiles = __builtin_amdgcn_readlane(nt, k);
      tile = want - (before + __builtin_amdgcn_readlane(inc, k) - ntiles);
      return true;
    }
    before += all;
  }
  return false;
}

// One 16-byte direct load per lane from `off` (a lane past the descriptor's bytes gets zeros) to LDS at dst + 16 * lane.
__device__ __forceinline__ void load_lds(const Buf& b, char* dst, uint32_t off) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(b.r, (__attribute__((address_space(3))) void*)dst, 16, (int)off, 0, 0, 0);
}

// Barrier after which every wave's direct loads to LDS have arrived: each wave waits for its own first. (A plain barrier
// waits for LDS accesses, not for loads on their way there.)
__device__ __forceinline__ void arrive() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0x0F70);              // vmcnt(0); the other counters at their maximum (no wait)
  __syncthreads();
}

// LDS of one tile of keys. The two tiles of a block are separate objects: the compiler then sees that the loads on
// their way into one do not concern the reads of the other.
template <int DP, bool C8>
struct Tile {
  static constexpr int TK = 1 << many_ush(DP);
  alignas(16) char k[TK * DP * 2];
  alignas(16) char v[TK * DP * 2];
  alignas(16) float kf[C8 ? TK : 4], lg[C8 ? TK : 4], inv[C8 ? TK : 4];   // see VScale; kf: K scale * softmax scale
  int have[NW];                                  // keys of each 16 that exist
  int odd;                                       // the last unit with an infinity or NaN in V that was stored here
  uint8_t vnan[C8 ? TK : 4];
};

// DP: columns of an LDS row, a power of two; DU <= DP: the columns that are multiplied, at least the head size.
template <bool BF, int KVM, int DP, int DU>
__global__ __launch_bounds__(NT, DP <= 128 ? 2 : 1) void k_attn_many(AttnArgs a) {
  constexpr bool C8 = KVM != 0, CB = BF && !C8;
  constexpr int EB = C8 ? 1 : 2, RB = DP * 2, KS = DU / 16, DB = DU / 32;
  constexpr int CPR = DP * EB / 16, RPI = 64 / CPR, LD = 16 / RPI;   // 16-byte chunks a cached row; rows, loads of a wave
  // Operands of one group of products are read while the group before is multiplied. With one wave a SIMD (head sizes
  // over 128) that has to be said: 4096 tokens of 64 heads of 256 over 8192, fp16, 3324 -> 2890 us. With two the order is
  // left to the compiler (said there too: 482 -> 492 us at size 64, 961 -> 981 at 128).
  constexpr bool AHEAD = DP > 128;
  constexpr int USH = many_ush(DP), TK = 1 << USH, KB = TK / 32, NG = TK / 16;   // keys of a tile, by 32 and by 16
  __shared__ Tile<DP, C8> tile0, tile1;
  __shared__ float big_[NW];
  __shared__ int nan_code;                         // e4m3: a tile that some row may see only in part held a NaN code of V
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), l = threadIdx.x & 63, h = l >> 5, ql = l & 31;
  const int hk = blockIdx.x % a.kv.hkv, d = a.kv.d, G = a.G, split = blockIdx.y;
  int s, tile, ntiles;
  if (!find_tile(a, blockIdx.x / a.kv.hkv, s, tile, ntiles)) return;
  tile = ntiles - 1 - tile;                        // the longest first
  const Seq sq = load_seq(a.sq, s, a.kv.psh);
  const int n = min(sq.n, a.max_q), r0 = tile * MANY_ROWS, rows = min(MANY_ROWS, n * G - r0);
  const int p0 = sq.p0;
  const int b_lo = p0 + r0 / G, b_hi = p0 + (r0 + rows - 1) / G;
  const Units un = key_units(b_lo, b_hi, sq.len, a.window, a.sinks, USH);
  const int per = share_units(un.tot, a.ns, MANY_LEAST, 1), used = max(1, (un.tot + per - 1) / per);
  if (split >= used) return;
  const int u0 = split * per, u1 = min(un.tot, u0 + per);

  // this lane's row, and the wave's range of positions
  const int r = r0 + w * 32 + ql, ri = r / G, rg = r - ri * G;
  const bool mine = w * 32 + ql < rows;
  const bool wave_on = w * 32 < rows;
  const int p_lo = p0 + (r0 + w * 32) / G, p_hi = p0 + (r0 + min(w * 32 + 32, rows) - 1) / G;
  const int pos = mine ? p0 + ri : p_hi;
  uint4 qf[KS];
  {
    const char* qp = a.q + ((long)(sq.q0 + ri) * a.ldq + (long)(hk * G + rg) * d) * 2;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      const int ch = ks * 2 + h;
      qf[ks] = mine && ch * 8 < d ? *reinterpret_cast<const uint4*>(qp + ch * 16) : make_uint4(0, 0, 0, 0);
      if (a.neg) qf[ks] = flip_signs(qf[ks]);
    }
  }
  float c = a.c;
  if constexpr (C8 && BF) {   // bf16 queries into fp16's range, as in the few-row kernel
    float big = 0.f;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) big = fmaxf(big, absmax8<true>(finite_only<true>(qf[ks])));
    big = wave_max(big);
    if (l == 0) big_[w] = big;
    __syncthreads();
    const float up = to_f16_range(fmaxf(fmaxf(big_[0], big_[1]), fmaxf(big_[2], big_[3])), c);
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) qf[ks] = bf16_to_f16(qf[ks], up);
  }
  if (threadIdx.x == 0) { tile0.odd = -1; tile1.odd = -1; nan_code = 0; }
  __syncthreads();

  const int* trow = a.sq.table + (long)s * a.sq.ldt;
  const uint32_t dB = (uint32_t)d * EB;
  // A wave brings K and V of 16 keys of a 64-key tile (they share a page), of a 32-key tile one of the two; what does
  // not exist reads as zeros. 16-bit rows go straight to LDS: the lane for slot l % CPR of a row loads the chunk that
  // belongs there. 8-bit codes pass through registers and are widened once a block.
  const int grp = w & (NG - 1);
  const bool do_k = NG == NW || w < NG, do_v = NG == NW || w >= NG;
  uint4 kr[C8 ? LD : 1], vr[C8 ? LD : 1];
  float sk1 = 0.f, sv1 = 0.f;
  int have = 0;
  uint32_t ko[LD], vo[LD];
#pragma unroll
  for (int i = 0; i < LD; ++i) {
    const uint32_t key = i * RPI + l / CPR, slot = l % CPR;
    const uint32_t kc = C8 ? slot : slot ^ swz_k<DP>(key), vc = C8 ? slot : slot ^ swz_v<DP>(key);
    ko[i] = boff(kc * 16 < dB, key * dB + kc * 16);
    vo[i] = boff(vc * 16 < dB, key * dB + vc * 16);
  }
  auto page_of = [&](int t0) { return trow[min((t0 + grp * 16) >> a.kv.psh, a.sq.cols - 1)]; };
  auto fetch = [&](Tile<DP, C8>& tl, int t0, int page) {
    const int t = t0 + grp * 16;
    const int pid = __builtin_amdgcn_readfirstlane(page);
    have = (unsigned)pid < (unsigned)a.kv.n_pages ? min(16, max(0, sq.len - t)) : 0;
    const long row = (((long)(have ? pid : 0) * a.kv.hkv + hk) << a.kv.psh) + (t & ((1 << a.kv.psh) - 1));
    const Buf bk(a.kv.k + row * dB, have * dB), bv(a.kv.v + row * dB, have * dB);
#pragma unroll
    for (int i = 0; i < LD; ++i) {
      if constexpr (C8) {
        if (do_k) kr[i] = bk.ld16(ko[i]);
        if (do_v) vr[i] = bv.ld16(vo[i]);
      } else {
        if (do_k) load_lds(bk, tl.k + (grp * 16 + i * RPI) * RB, ko[i]);
        if (do_v) load_lds(bv, tl.v + (grp * 16 + i * RPI) * RB, vo[i]);
      }
    }
    if constexpr (C8) {
      const Buf sk(a.kv.ks + row, have * 4), sv(a.kv.vs + row, have * 4);
      sk1 = sk.ldf((l & 15) * 4);
      sv1 = sv.ldf((l & 15) * 4);
    }
    if (!C8 && l == 0) tl.have[grp] = have;
  };
  // whether every row of the block sees every key that exists of the TK keys from t0 on
  auto by_all = [&](int t0) {
    return t0 + TK - 1 <= b_lo && (a.window <= 0 || t0 > b_hi - a.window || t0 + TK <= a.sinks);
  };
  // 8-bit: the fetched codes into the tile
  auto store = [&](Tile<DP, C8>& tl, int u) {
    if constexpr (C8) {
      int lx = l;                                  // places worked out anew per tile: registers are short
      asm volatile("" : "+v"(lx));
#pragma unroll
      for (int i = 0; i < LD; ++i) {
        const int key = grp * 16 + i * RPI + lx / CPR, ch = lx % CPR;
        const uint2 k0 = codes4<KVM == 2>(kr[i].x), k1 = codes4<KVM == 2>(kr[i].y), k2 = codes4<KVM == 2>(kr[i].z),
                    k3 = codes4<KVM == 2>(kr[i].w);
        if (do_k) {
          *reinterpret_cast<uint4*>(&tl.k[key * RB + (((2 * ch) ^ swz_k<DP>(key)) << 4)]) = make_uint4(k0.x, k0.y, k1.x, k1.y);
          *reinterpret_cast<uint4*>(&tl.k[key * RB + (((2 * ch + 1) ^ swz_k<DP>(key)) << 4)]) = make_uint4(k2.x, k2.y, k3.x, k3.y);
        }
      }
      if constexpr (KVM == 2) {
        // NaN codes are left out and added after the last tile, see look(). (Here, behind K's codes: before them a chunk of
        // head size 256 takes 279 us instead of 269.)
        if (do_v && !by_all(un.key0(u, USH))) {
          uint32_t bad = 0;
#pragma unroll
          for (int i = 0; i < LD; ++i) {
            bad |= nan_codes4(vr[i]);
            vr[i] = finite_codes4(vr[i]);
          }
          if (bad != 0) nan_code = 1;
        }
      }
#pragma unroll
      for (int i = 0; i < LD; ++i) {
        const int key = grp * 16 + i * RPI + lx / CPR, ch = lx % CPR;
        const uint2 v0 = codes4<KVM == 2>(vr[i].x), v1 = codes4<KVM == 2>(vr[i].y), v2 = codes4<KVM == 2>(vr[i].z),
                    v3 = codes4<KVM == 2>(vr[i].w);
        if (do_v) {
          *reinterpret_cast<uint4*>(&tl.v[key * RB + (((2 * ch) ^ swz_v<DP>(key)) << 4)]) = make_uint4(v0.x, v0.y, v1.x, v1.y);
          *reinterpret_cast<uint4*>(&tl.v[key * RB + (((2 * ch + 1) ^ swz_v<DP>(key)) << 4)]) = make_uint4(v2.x, v2.y, v3.x, v3.y);
        }
      }
      if (l < 16) {
        const VScale v = v_scale(sv1);
        tl.kf[grp * 16 + l] = sk1 * c;
        tl.lg[grp * 16 + l] = v.lg;
        tl.inv[grp * 16 + l] = v.inv;
        tl.vnan[grp * 16 + l] = sv1 != sv1 ? 1 : 0;
        if (sv1 != sv1) tl.odd = u;
      }
      if (l == 0) tl.have[grp] = have;
    }
  };

  float m = -INFINITY, ls = 0.f;
  f32x16 o[DB];
#pragma unroll
  for (int db = 0; db < DB; ++db)
#pragma unroll
    for (int i = 0; i < 16; ++i) o[db][i] = 0.f;

  // Operand places: a row's base with the swizzle of its key, and one exclusive or for the 16-byte column. The bases
  // are made opaque once a tile, or the loop's invariants (one address a column) would be kept in registers that are
  // not there; their spilled values' loads would wait for the tile loads in flight.
  const int kb0 = ql * RB + ((h ^ swz_k<DP>(ql)) << 4);
  const int vkey = 4 * h + ((l & 15) >> 2);
  const int vb0 = vkey * RB + (((((l >> 4) & 1) * 2 + ((l & 3) >> 1)) ^ swz_v<DP>(vkey)) << 4) + (l & 1) * 8;
  auto v_frag = [&](const Tile<DP, C8>& tl, int vb, int kk, int db) {
    const char* at = tl.v + (vb ^ (db * 64));      // keys 8 and 16 apart: the same slot
    const fp16x4 y0 = __builtin_amdgcn_ds_read_tr16_b64_v4f16((__attribute__((address_space(3))) fp16x4*)(at + kk * 16 * RB));
    const fp16x4 y1 = __builtin_amdgcn_ds_read_tr16_b64_v4f16((__attribute__((address_space(3))) fp16x4*)(at + (kk * 16 + 8) * RB));
    const uint2 z0 = __builtin_bit_cast(uint2, y0), z1 = __builtin_bit_cast(uint2, y1);
    return make_uint4(z0.x, z0.y, z1.x, z1.y);
  };

  bool left_out = false;
  // one tile: scores, softmax, weighted sum
  auto work = [&](const Tile<DP, C8>& tl, int u, int t0) {
    int kb_ = kb0, vb = vb0;
    asm volatile("" : "+v"(kb_), "+v"(vb));
    f32x16 sc[KB];
#pragma unroll
    for (int kb = 0; kb < KB; ++kb)
#pragma unroll
      for (int i = 0; i < 16; ++i) sc[kb][i] = 0.f;
    auto k_frag = [&](int ks, int kb) { return *reinterpret_cast<const uint4*>(tl.k + (kb_ ^ (ks * 32)) + kb * 32 * RB); };
    if constexpr (AHEAD) {
      uint4 kf[2][2 * KB];
      auto group = [&](int g) {
#pragma unroll
        for (int j = 0; j < 2 * KB; ++j) kf[g & 1][j] = k_frag(g * 2 + j / KB, j % KB);
      };
      group(0);
#pragma unroll
      for (int g = 0; g < KS / 2; ++g) {
        if (g + 1 < KS / 2) group(g + 1);
        __builtin_amdgcn_sched_barrier(NOT_DS);
#pragma unroll
        for (int j = 0; j < 2 * KB; ++j) sc[j % KB] = mfma32<CB>(kf[g & 1][j], qf[g * 2 + j / KB], sc[j % KB]);
      }
    } else {
#pragma unroll
      for (int ks = 0; ks < KS; ++ks)
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) sc[kb] = mfma32<CB>(k_frag(ks, kb), qf[ks], sc[kb]);
    }
    if constexpr (C8) {
#pragma unroll
      for (int kb = 0; kb < KB; ++kb)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const f32x4 kf = *reinterpret_cast<const f32x4*>(&tl.kf[kb * 32 + 8 * e + 4 * h]);
          const f32x4 lg = *reinterpret_cast<const f32x4*>(&tl.lg[kb * 32 + 8 * e + 4 * h]);
#pragma unroll
          for (int i = 0; i < 4; ++i) sc[kb][e * 4 + i] = fmaf(sc[kb][e * 4 + i], kf[i], lg[i]);
        }
    }
    const int hv0 = tl.have[0], hv1 = tl.have[1], hv2 = NG > 2 ? tl.have[2] : 0, hv3 = NG > 2 ? tl.have[3] : 0, nv = hv0 + hv1 + hv2 + hv3;
    const bool full = nv == TK && t0 + TK - 1 <= p_lo &&
                      (a.window <= 0 || t0 > p_hi - a.window || t0 + TK <= a.sinks);
    if (!full) {
      // element (kb, e, i) is key kb * 32 + 8 e + i of those that start at 4 h
      const bool holes = (hv0 < 16 && hv1 + hv2 + hv3) || (hv1 < 16 && hv2 + hv3) || (hv2 < 16 && hv3);
      const int hi = min(pos - t0, holes ? TK - 1 : nv - 1) - 4 * h;
#pragma unroll
      for (int kb = 0; kb < KB; ++kb)
#pragma unroll
        for (int i = 0; i < 16; ++i) sc[kb][i] = kb * 32 + 8 * (i >> 2) + (i & 3) <= hi ? sc[kb][i] : -INFINITY;
      if (a.window > 0) {
        const int lo = pos - a.window - t0 - 4 * h, sk = a.sinks - t0 - 4 * h;
#pragma unroll
        for (int kb = 0; kb < KB; ++kb)
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int kk = kb * 32 + 8 * (i >> 2) + (i & 3);
            sc[kb][i] = ((kk > lo) | (kk < sk)) ? sc[kb][i] : -INFINITY;
          }
      }
      if (holes) {
#pragma unroll
        for (int kb = 0; kb < KB; ++kb)
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int hv = kb == 0 ? (i < 8 ? hv0 : hv1) : (i < 8 ? hv2 : hv3);
            sc[kb][i] = 8 * ((i >> 2) & 1) + (i & 3) + 4 * h < hv ? sc[kb][i] : -INFINITY;
          }
      }
    }
    float top = -INFINITY;
#pragma unroll
    for (int kb = 0; kb < KB; ++kb)
#pragma unroll
      for (int i = 0; i < 16; ++i) top = fmaxf(top, sc[kb][i]);
    top = over32<true>(top);
    if constexpr (!C8) top *= c;
    if (__any(outgrown<CB>(top, m))) {
      const float mn = new_reference<CB>(top, m), f = fade(m, mn);
      ls *= f;
#pragma unroll
      for (int db = 0; db < DB; ++db) o[db] *= f;
      m = mn;
    }
    const float ms = m == -INFINITY ? 0.f : m;
    uint4 vf[2][AHEAD ? DB : 1];
    auto v_group = [&](int kk) {
#pragma unroll
      for (int db = 0; db < DB; ++db) vf[kk & 1][AHEAD ? db : 0] = v_frag(tl, vb, kk, db);
    };
    if constexpr (AHEAD) {
      v_group(0);
      __builtin_amdgcn_sched_barrier(NOT_DS);
    }
    uint4 pf[NG];
    const bool slow = C8 && tl.odd == u;
    uint32_t vis = 0;
    if (slow) {                              // which elements are seen: bit kb * 16 + i
#pragma unroll
      for (int kb = 0; kb < KB; ++kb)
#pragma unroll
        for (int i = 0; i < 16; ++i) vis |= sc[kb][i] != -INFINITY ? 1u << (kb * 16 + i) : 0u;
    }
#pragma unroll
    for (int kb = 0; kb < KB; ++kb)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float p[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          p[i] = exp2_fast(C8 ? sc[kb][e * 4 + i] - ms : fmaf(sc[kb][e * 4 + i], c, -ms));
        if constexpr (C8) {
          const f32x4 iv = *reinterpret_cast<const f32x4*>(&tl.inv[kb * 32 + 8 * e + 4 * h]);
#pragma unroll
          for (int i = 0; i < 4; ++i) ls = fmaf(p[i], iv[i], ls);
        } else {
          ls += (p[0] + p[1]) + (p[2] + p[3]);
        }
        const uint32_t a0 = pack2<CB>(p[0], p[1]), a1 = pack2<CB>(p[2], p[3]);
        if (e & 1) { pf[kb * 2 + (e >> 1)].z = a0; pf[kb * 2 + (e >> 1)].w = a1; }
        else { pf[kb * 2 + (e >> 1)].x = a0; pf[kb * 2 + (e >> 1)].y = a1; }
      }
    if (slow) {                                    // a V row without a scale: NaN for the rows that see it
#pragma unroll
      for (int kk = 0; kk < NG; ++kk) {
        uint32_t nan[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          nan[k] = 0;
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int e = kk * 8 + k * 2 + j, kb = e >> 4, i = e & 15;
            if ((vis >> e & 1) && tl.vnan[kb * 32 + 8 * (i >> 2) + 4 * h + (i & 3)]) nan[k] |= 0x7E00u << (16 * j);
          }
        }
        pf[kk] = make_uint4(pf[kk].x | nan[0], pf[kk].y | nan[1], pf[kk].z | nan[2], pf[kk].w | nan[3]);
      }
    }
    if constexpr (AHEAD) {
#pragma unroll
      for (int kk = 0; kk < NG; ++kk) {
        if (kk + 1 < NG) v_group(kk + 1);
        __builtin_amdgcn_sched_barrier(NOT_DS);
#pragma unroll
        for (int db = 0; db < DB; ++db) o[db] = mfma32<CB>(vf[kk & 1][db], pf[kk], o[db]);
      }
    } else {
#pragma unroll
      for (int kk = 0; kk < NG; ++kk)
#pragma unroll
        for (int db = 0; db < DB; ++db) o[db] = mfma32<CB>(v_frag(tl, vb, kk, db), pf[kk], o[db]);
    }
  };
  // Infinities and NaN in a 16-bit tile that some row may see only in part: set to 0 in LDS, and added after the last
  // tile where they are seen. (NaN codes of e4m3: in store().)
  auto inside = [&](int t0, int have) { return by_all(t0) && have == TK; };
  auto look = [&](Tile<DP, C8>& tl, int u, int t0) {
    if (C8 || inside(t0, tl.have[0] + tl.have[1] + (NG > 2 ? tl.have[2] + tl.have[3] : 0))) return;   // the same in every wave
#pragma unroll
    for (int i = 0; i < TK * RB / (NT * 16); ++i) {
      uint4* p = reinterpret_cast<uint4*>(&tl.v[(i * NT + threadIdx.x) * 16]);
      const uint4 v = *p;
      if (nonfinite2<CB>(v.x) | nonfinite2<CB>(v.y) | nonfinite2<CB>(v.z) | nonfinite2<CB>(v.w)) {
        *p = finite_only<CB>(v);
        tl.odd = u;
      }
    }
    lds_barrier();                                 // the next tile's loads stay in flight
    left_out |= tl.odd == u;
  };

  if (u0 < u1) {
    const int t0 = un.key0(u0, USH);
    fetch(tile0, t0, page_of(t0));
    store(tile0, u0);
  }
  int page = u0 + 1 < u1 ? page_of(un.key0(u0 + 1, USH)) : 0;
  auto step = [&](Tile<DP, C8>& cur, Tile<DP, C8>& nxt, int u) {
    const int t0 = un.key0(u, USH);
    arrive();                                      // cur is there, nxt is free
    if (u + 1 < u1) {
      fetch(nxt, un.key0(u + 1, USH), page);
      if (u + 2 < u1) page = page_of(un.key0(u + 2, USH));
    }
    look(cur, u, t0);
    if (wave_on && t0 <= p_hi) work(cur, u, t0);
    if (u + 1 < u1) store(nxt, u + 1);
  };
  for (int u = u0; u < u1; u += 2) {
    step(tile0, tile1, u);
    if (u + 1 < u1) step(tile1, tile0, u + 1);
  }

  if constexpr (KVM == 2) {
    __syncthreads();
    left_out = nan_code;
  }
  if (!wave_on) return;
  ls = over32<false>(ls);
  bool again = false;                              // NaN though the row's sum is none: it may be an infinity's (see LOST)
  if constexpr (!C8) {
#pragma unroll
    for (int db = 0; db < DB; ++db)
#pragma unroll
      for (int i = 0; i < 16; ++i) again |= ls == ls && o[db][i] != o[db][i];
    again = __any(again);
    if (again) {
#pragma unroll
      for (int db = 0; db < DB; ++db)
#pragma unroll
        for (int i = 0; i < 16; ++i) o[db][i] = lose_nan(o[db][i]);
    }
  }
  if (KVM != 1 && (again || left_out)) {
    // once more through the keys of those tiles (of all, for lost infinities)
#pragma unroll 1
    for (int u = u0; u < u1; ++u) {
      const int t0 = un.key0(u, USH);
      int have[NG], pid[NG], nv = 0;
#pragma unroll
      for (int k = 0; k < NG; ++k) {
        pid[k] = trow[min((t0 + k * 16) >> a.kv.psh, a.sq.cols - 1)];
        have[k] = (unsigned)pid[k] < (unsigned)a.kv.n_pages ? min(16, max(0, sq.len - (t0 + k * 16))) : 0;
        nv += have[k];
      }
      if (!again && (C8 ? by_all(t0) : inside(t0, nv))) continue;
#pragma unroll
      for (int k = 0; k < NG; ++k)
#pragma unroll 1
        for (int kk = 0; kk < have[k]; ++kk) {
          const int j = t0 + k * 16 + kk;
          const bool see = j <= pos && (a.window <= 0 || j > pos - a.window || j < a.sinks);
          const char* row = a.kv.v + ((((long)pid[k] * a.kv.hkv + hk) << a.kv.psh) + (j & ((1 << a.kv.psh) - 1))) * dB;
#pragma unroll
          for (int db = 0; db < DB; ++db)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int d0 = db * 32 + e * 8 + h * 4;
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
              for (int i = 0; i < 4; ++i) o[db][e * 4 + i] += see && !(fabsf(f[i]) < INFINITY) ? f[i] : 0.f;
            }
        }
    }
    if (again) {
#pragma unroll
      for (int db = 0; db < DB; ++db)
#pragma unroll
        for (int i = 0; i < 16; ++i) o[db][i] = find_lost(o[db][i]);
    }
  }
  if (!mine) return;
  const long row = (long)(sq.q0 + ri) * a.hq + hk * G + rg;
  if (used == 1) {
    const float iv = ls == 0.f ? 0.f : 1.f / ls;   // no key was visible: 0
    char* op = a.out + ((long)(sq.q0 + ri) * a.ldo + (long)(hk * G + rg) * d) * 2;
#pragma unroll
    for (int db = 0; db < DB; ++db)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int d0 = db * 32 + e * 8 + h * 4;
        if (d0 < d)
          *reinterpret_cast<uint2*>(op + d0 * 2) = make_uint2(pack2<BF>(o[db][e * 4] * iv, o[db][e * 4 + 1] * iv),
                                                              pack2<BF>(o[db][e * 4 + 2] * iv, o[db][e * 4 + 3] * iv));
      }
    if (a.lse && h == 0) a.lse[row] = log_sum(m, ls);
  } else {
    float* po = a.po + (row * a.ns + split) * d;
#pragma unroll
    for (int db = 0; db < DB; ++db)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int d0 = db * 32 + e * 8 + h * 4;
        if (d0 < d)
          *reinterpret_cast<f32x4*>(po + d0) = f32x4{o[db][e * 4], o[db][e * 4 + 1], o[db][e * 4 + 2], o[db][e * 4 + 3]};
      }
    if (h == 0) a.pml[row * a.ns + split] = make_float2(m, ls);
  }
}

// Split results of a row added in a fixed order. WPR waves a row: lanes hold 4 elements each, the lanes that are left
// take the shares in turn (groups of shares are summed, then the groups). Which shares exist follows from the same
// rule as in the kernels above.
template <bool BF, int DP, int WPR>
__global__ __launch_bounds__(NT) void k_attn_join(AttnArgs a, int few) {
  constexpr int LE = DP / 4, GR = WPR * 64 / LE;   // lanes of a row's elements; groups
  __shared__ f32x4 part[WPR > 1 ? WPR : 1][64];
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), l = threadIdx.x & 63;
  const long row = WPR > 1 ? (long)blockIdx.x : (long)blockIdx.x * NW + w;
  if (row >= (long)a.sq.T * a.hq) return;
  const int t = (int)(row / a.hq), hq = (int)(row - (long)t * a.hq), g = hq % a.G, d = a.kv.d;
  const int s = __builtin_amdgcn_readfirstlane(find_seq<64>(a.sq.cu, a.sq.S, t));
  if (s >= a.sq.S) return;
  const Seq sq = load_seq(a.sq, s, a.kv.psh);
  const int n = min(sq.n, a.max_q), i = t - sq.q0, p0 = sq.p0;
  if (i < 0 || i >= n) return;
  int lo, hi;                                      // positions of the row's tile
  if (few) {
    lo = p0;
    hi = p0 + n - 1;
  } else {
    const int r0 = (i * a.G + g) / MANY_ROWS * MANY_ROWS;
    lo = p0 + r0 / a.G;
    hi = p0 + (min(n * a.G, r0 + MANY_ROWS) - 1) / a.G;
  }
  const Units un = key_units(lo, hi, sq.len, a.window, a.sinks, few ? FEW_USH : many_ush(d));
  const int per = share_units(un.tot, a.ns, few ? few_least(d) : MANY_LEAST, few ? FEW_STEP : 1);
  const int used = (un.tot + per - 1) / per;       // at most MAX_SHARES
  if (used <= 1) return;                           // the row's only block has written it
  const float2 ml = l < used ? a.pml[row * a.ns + l] : make_float2(-INFINITY, 0.f);
  const float M = wave_max(ml.x), f = fade(ml.x, M == -INFINITY ? 0.f : M), L = wave_sum(ml.y * f);
  const float iv = L == 0.f ? 0.f : 1.f / L;
  const int e = (l % LE) * 4, gr = (w % WPR) * (64 / LE) + l / LE;
  const float* po = a.po + row * a.ns * d + e;
  f32x4 acc = {0.f, 0.f, 0.f, 0.f};
  for (int k0 = 0; k0 < used; k0 += 4 * GR) {
    f32x4 x[4];
    float fk[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int k = k0 + j * GR + gr;
      const bool in = k < used && e < d;
      x[j] = in ? *reinterpret_cast<const f32x4*>(po + (long)k * d) : f32x4{0.f, 0.f, 0.f, 0.f};
      fk[j] = __shfl(f, k, WAVE);                  // k < 64 wherever x is not 0
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) acc += x[j] * (k0 + j * GR + gr < used ? fk[j] : 0.f);
  }
#pragma unroll
  for (int x = LE; x < 64; x <<= 1)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[j] += __shfl_xor(acc[j], x, WAVE);
  if constexpr (WPR > 1) {
    part[w][l] = acc;
    __syncthreads();
    if (w) return;
#pragma unroll
    for (int k = 1; k < WPR; ++k) acc += part[k][l];
  }
  if (l < LE && e < d)
    *reinterpret_cast<uint2*>(a.out + ((long)t * a.ldo + (long)hq * d + e) * 2) =
        make_uint2(pack2<BF>(acc[0] * iv, acc[1] * iv), pack2<BF>(acc[2] * iv, acc[3] * iv));
  if (a.lse && l == 0) a.lse[row] = log_sum(M, L);
}

}  // namespace

hipError_t sffn_launch_attn_many(const AttnArgs& a, int qt, int kvt, hipStream_t st) {
  // at most T * G / MANY_ROWS whole tiles, and one that is not whole for each sequence
  const long tiles = (long)a.sq.T * a.G / MANY_ROWS + (a.sq.S < a.sq.T ? a.sq.S : a.sq.T);
  const dim3 grid((unsigned)(tiles * a.kv.hkv), a.ns);
  const bool bf = qt == T_BF16;
  const int kvm = kvt == T_I8 ? 1 : kvt == T_E4M3 ? 2 : 0;
#define GO(BF, KVM, DP, DU) hipLaunchKernelGGL((k_attn_many<BF, KVM, DP, DU>), grid, dim3(NT), 0, st, a)
#define TYPES(DP, DU)                                                                           \
  if (bf) {                                                                                     \
    if (kvm == 0) GO(true, 0, DP, DU); else if (kvm == 1) GO(true, 1, DP, DU); else GO(true, 2, DP, DU);    \
  } else {                                                                                      \
    if (kvm == 0) GO(false, 0, DP, DU); else if (kvm == 1) GO(false, 1, DP, DU); else GO(false, 2, DP, DU); \
  }
  // Head sizes that leave a quarter of the padded columns are multiplied without it (4096 tokens of 64 heads on 8 over
  // 8192, fp16: size 96 846 -> 750 us, 80 804 -> 712; 1000 tokens: 192 900 -> 763, 144 897 -> 764).
  if (a.kv.d <= 64) { TYPES(64, 64) }
  else if (a.kv.d <= 96) { TYPES(128, 96) }
  else if (a.kv.d <= 128) { TYPES(128, 128) }
  else if (a.kv.d <= 192) { TYPES(256, 192) }
  else { TYPES(256, 256) }
#undef TYPES
#undef GO
  return hipGetLastError();
}

hipError_t sffn_launch_attn_join(const AttnArgs& a, int qt, bool few, hipStream_t st) {
  const long rows = (long)a.sq.T * a.hq;
  const bool bf = qt == T_BF16, wide = a.ns > 8;   // four waves a row from 9 shares on
  const dim3 grid((unsigned)(wide ? rows : (rows + NW - 1) / NW));
#define GO(BF, DP, WPR) hipLaunchKernelGGL((k_attn_join<BF, DP, WPR>), grid, dim3(NT), 0, st, a, (int)few)
#define PICK(DP) \
  if (bf) { if (wide) GO(true, DP, 4); else GO(true, DP, 1); } else { if (wide) GO(false, DP, 4); else GO(false, DP, 1); }
  if (a.kv.d <= 64) { PICK(64) } else if (a.kv.d <= 128) { PICK(128) } else { PICK(256) }
#undef PICK
#undef GO
  return hipGetLastError();
}
