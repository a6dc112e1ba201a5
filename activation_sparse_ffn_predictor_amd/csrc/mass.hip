// Attention weight that each cached token gets from a call's new tokens, summed over them and the query heads that share its
// K/V head, and added to what it had:
//   out[s, h, j] = (mass[s, h, j], or 0 for a new token) + sum over rows (i, g) that see j of exp(scale q . K_j - lse)
// with the attention's own log-sum-exp, so no maximum is sought and no row waits for another: one product and one exponential
// a score. New tokens' positions in the sequence are entered beside it. Every sum has one order, whatever runs beside it.
#include "mass.h"

using namespace sffn;

namespace {

constexpr float LOG2E = 1.4426950408889634f;

// The sequence of a workgroup: its clamped numbers, how far its tokens' positions are ahead of their slots, the keys that have a place.
struct MassSeq {
  Seq q;
  int n, rows, p1, ahead, keys;
};
__device__ __forceinline__ MassSeq mass_seq(const MassArgs& a, int s) {
  MassSeq m;
  m.q = load_seq(a.sq, s, a.kv.psh);
  m.ahead = token_pos(a.plen[s], max(a.sq.cu[s + 1], m.q.q0), m.q.q0) - m.q.p0;
  m.q.p0 = max(m.q.p0, -(1 << 25));                  // (below it no token of a call can see anything)
  m.n = min(m.q.n, a.max_q);
  m.rows = m.n * a.G;
  m.p1 = m.q.p0 + m.n - 1;
  m.keys = min(m.q.len, a.W);
  return m;
}
// one key's sum to its place
__device__ __forceinline__ void give(const MassArgs& a, const MassSeq& m, long base, int j, float old, float sum) {
  const bool fresh = j >= m.q.p0;
  a.out[base + j] = (fresh ? 0.f : old) + sum;
  if (fresh) a.pos[base + j] = j + m.ahead;
}
// does any (every) row at positions pa .. pb see any (every one) of the keys k0 .. k1?
__device__ __forceinline__ bool some_seen(const MassArgs& a, int pa, int pb, int k0, int k1) {
  return k0 <= pb && (a.window <= 0 || k1 > pa - a.window || k0 < a.sinks);
}
__device__ __forceinline__ bool all_seen(const MassArgs& a, int pa, int pb, int k0, int k1) {
  return k1 <= pa && (a.window <= 0 || k0 > pb - a.window || k1 < a.sinks);
}
__device__ __forceinline__ bool seen(const MassArgs& a, int p, int j) {
  return (j <= p) & ((a.window <= 0) | (j > p - a.window) | (j < a.sinks));
}
// 8-bit codes (8 of them) as bf16, exactly
template <bool E4M3>
__device__ __forceinline__ uint4 codes8_bf16(uint2 c) {
  const uint2 x = codes4<E4M3>(c.x), y = codes4<E4M3>(c.y);
  return make_uint4(pack2<true>(lo16<false>(x.x), hi16<false>(x.x)), pack2<true>(lo16<false>(x.y), hi16<false>(x.y)),
                    pack2<true>(lo16<false>(y.x), hi16<false>(y.x)), pack2<true>(lo16<false>(y.y), hi16<false>(y.y)));
}

// ------------------------------------------------------------------------------------------------ few rows
// Up to 16 * QB rows (single tokens, drafts): the queries stay in registers, every wave runs through its own units of 32 keys.
// S = Q K^T (16x16x32): a lane's column is a key, its registers are rows, so a key's sum needs two exchanges for 16 keys.
// Bound by K's bytes (32 sequences to 6000 tokens on 40 heads, int8, 467 MB: 98 us, 4.8 TB/s; a large copy reaches 5.55, reading alone
// 5.9; page ids ahead of the loads that need them: 130 -> 113). KVM 0: cache of the queries' type, 1: int8, 2: e4m3 (products in fp16, bf16 queries brought into its
// range by one power of two). DP: head size padded.
template <bool BF, int KVM, int DP, int QB>
__global__ __launch_bounds__(256) void k_mass_few(MassArgs a) {
  constexpr bool C8 = KVM != 0, CB = BF && !C8;
  constexpr int EB = C8 ? 1 : 2, KS = DP / 32, KL = DP * EB / 64;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), l = threadIdx.x & 63, g4 = l >> 4, ql = l & 15;
  const int hk = blockIdx.y, s = blockIdx.z, d = a.kv.d, G = a.G;
  const MassSeq m = mass_seq(a, s);
  if (m.q.n == 0 || m.rows == 0 || m.keys <= 0) return;
  const bool copy = a.out != a.mass;                 // also what no row sees
  const int* trow = a.sq.table + (long)s * a.sq.ldt;
  const long base = ((long)s * a.kv.hkv + hk) * a.W;
  const uint32_t dB = (uint32_t)d * EB, ko = (uint32_t)ql * dB + g4 * 16;
  const int units = (m.keys + 31) >> 5, step = gridDim.x * 4;

  // page ids are read a unit ahead of the loads that need them, which would wait for everything on its way otherwise
  int page[2];
  auto pages = [&](int u) {
#pragma unroll
    for (int kb = 0; kb < 2; ++kb) page[kb] = trow[min((u * 32 + kb * 16) >> a.kv.psh, a.sq.cols - 1)];
  };
  int u = blockIdx.x * 4 + w;
  if (u >= units) return;
  pages(u);

  float c = a.c;
  uint4 qf[QB][KS];
  float L[QB][4];
  int pr[QB][4];
#pragma unroll
  for (int qb = 0; qb < QB; ++qb) {
    const int r = qb * 16 + ql, i = r / G, g = r - i * G;
    const char* qp = a.q + ((long)(m.q.q0 + i) * a.ldq + (long)(hk * G + g) * d) * 2;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      const int ch = C8 ? ((ks >> 1) * 4 + g4) * 2 + (ks & 1) : ks * 4 + g4;
      qf[qb][ks] = r < m.rows && ch * 8 < d ? *reinterpret_cast<const uint4*>(qp + ch * 16) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int rr = qb * 16 + 4 * g4 + e, ii = rr / G;
      const float x = rr < m.rows ? a.lse[(long)(m.q.q0 + ii) * a.hq + hk * G + rr - ii * G] : -INFINITY;
      pr[qb][e] = m.q.p0 + ii;
      L[qb][e] = x;
    }
  }
  struct Unit {
    uint4 kr[2][KL];
    float ksc[2], old;
    int have[2];
  };
  auto visible = [&](int u) { return some_seen(a, m.q.p0, m.p1, u * 32, u * 32 + 31); };
  auto load = [&](int u, const int (&pg)[2], Unit& x) {
    const int t0 = u * 32;
    x.old = 0.f;
    if (l < 32 && t0 + l < m.keys) x.old = a.mass[base + t0 + l];
#pragma unroll
    for (int kb = 0; kb < 2; ++kb) {
      const int t = t0 + kb * 16, pid = __builtin_amdgcn_readfirstlane(pg[kb]);
      x.have[kb] = visible(u) && (unsigned)pid < (unsigned)a.kv.n_pages ? min(16, max(0, m.q.len - t)) : 0;
      const long r = (((long)(x.have[kb] ? pid : 0) * a.kv.hkv + hk) << a.kv.psh) + (t & ((1 << a.kv.psh) - 1));
      const Buf bk(a.kv.k + r * dB, x.have[kb] * dB);
#pragma unroll
      for (int i = 0; i < KL; ++i) x.kr[kb][i] = bk.ld16(boff((uint32_t)((i * 4 + g4) * 16) < dB, ko + i * 64));
      if constexpr (C8) x.ksc[kb] = Buf(a.kv.ks + r, x.have[kb] * 4).ldf(ql * 4);
    }
  };
  // A unit's registers are free once its products are made: the next one's loads are on their way under its exponentials and under
  // other waves' work (two units in turn, with registers for fewer waves, take as long over long caches, 26 us for 24 over 16
  // sequences of 5000 with 4 heads of 256)
  auto fetch = [&](int v, Unit& x) {
    if (v >= units) return;
    const int pg[2] = {page[0], page[1]};
    pages(v + step);
    load(v, pg, x);
  };
  auto work = [&](int u, Unit& now) {
    const int t0 = u * 32, h0 = now.have[0], h1 = now.have[1];
    const float old = now.old, sk[2] = {C8 ? now.ksc[0] : 0.f, C8 ? now.ksc[1] : 0.f};
    float sum[2] = {0.f, 0.f};
    const bool some = visible(u);
    f32x4 sc[QB][2];
    if (some) {
#pragma unroll
      for (int qb = 0; qb < QB; ++qb)
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) sc[qb][kb] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < KL; ++i)
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) {
          if constexpr (C8) {
            const uint4 t = now.kr[kb][i];
            const uint2 x0 = codes4<KVM == 2>(t.x), x1 = codes4<KVM == 2>(t.y), x2 = codes4<KVM == 2>(t.z), x3 = codes4<KVM == 2>(t.w);
            const uint4 ka = make_uint4(x0.x, x0.y, x1.x, x1.y), kc = make_uint4(x2.x, x2.y, x3.x, x3.y);
#pragma unroll
            for (int qb = 0; qb < QB; ++qb) {
              sc[qb][kb] = mfma16<false>(qf[qb][2 * i], ka, sc[qb][kb]);
              sc[qb][kb] = mfma16<false>(qf[qb][2 * i + 1], kc, sc[qb][kb]);
            }
          } else {
#pragma unroll
            for (int qb = 0; qb < QB; ++qb) sc[qb][kb] = mfma16<CB>(qf[qb][i], now.kr[kb][i], sc[qb][kb]);
          }
        }
    }
    fetch(u + step, now);
    if (some) {
      // most units are seen whole by every row: then rows alone decide
      const bool full = h0 + h1 == 32 && all_seen(a, m.q.p0, m.p1, t0, t0 + 31);
#pragma unroll
      for (int kb = 0; kb < 2; ++kb) {
        const float f = C8 ? sk[kb] * c : c;
        const int j = t0 + kb * 16 + ql;
        const bool held = ql < (kb ? h1 : h0);
#pragma unroll
        for (int qb = 0; qb < QB; ++qb)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float x = exp2_fast(fmaf(sc[qb][kb][e], f, -L[qb][e]));
            bool see = pr[qb][e] >= 0;
            if (!full) see = held & seen(a, pr[qb][e], j);
            sum[kb] += see ? x : 0.f;
          }
        sum[kb] = over32<false>(over16<false>(sum[kb]));
      }
    }
    const int j = t0 + l;
    if (l < 32 && j < m.keys && (copy || j >= m.q.p0 || some)) give(a, m, base, j, old, l < 16 ? sum[0] : sum[1]);
  };
  Unit x0;
  fetch(u, x0);
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
#pragma unroll
  for (int qb = 0; qb < QB; ++qb)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (L[qb][e] == -INFINITY) pr[qb][e] = -1;       // rows without a sum see nothing
      L[qb][e] *= LOG2E;
    }
  for (; u < units; u += step) work(u, x0);
}

// ------------------------------------------------------------------------------------------------ many rows
// K stays in registers (KT tiles of 32 keys a wave), the queries stream through LDS, 64 rows at a time, shared by the waves.
// S^T = K Q^T (32x32x16): a lane's column is a row, so it holds one log-sum-exp a tile, and keys' sums stay in its registers
// until the rows are through; 32 lanes are joined once. 8-bit codes are widened once, exactly, to the queries' type.
// Bound by exponentials and matrix products together: for 64 scores the vector unit needs 16 cycles (a multiply-add, an exponential, an
// addition), and so does the matrix core for products of 128 elements; what each leaves idle the other cannot wholly use (a step of
// one matrix instruction, two exponentials and four others takes 24 ns where the instruction alone takes 18.6). 2048 tokens over 6144,
// 64 heads on 8, 172 GFLOP: 205 to 252 us on different cards; with KT = 1, before they overlapped, 313 for 298. No vector registers spill;
// 71 to 115 scalar ones do: written to lanes of vector registers at the start, read back where K is loaded and the sums are given, not
// in the loops of products (k_mass_few: 28 to 32 with four blocks of rows, none with fewer).
constexpr int MROWS = 64;
template <bool BF, int KVM, int DP, int KT>
__global__ __launch_bounds__(256, 2) void k_mass_many(MassArgs a) {
  constexpr bool C8 = KVM != 0;
  constexpr int KS = DP / 16, CPR = DP / 8, RB = DP * 2, WG = 4 * KT * 32, LOADS = MROWS * CPR / 256;
  __shared__ __align__(16) char qs[2][MROWS * RB];
  __shared__ float Ls[2][MROWS];
  __shared__ int ps[2][MROWS];
  __shared__ __align__(16) float fk[C8 ? 4 : 1][KT * 32];    // 8-bit: scales of the waves' keys times the softmax scale
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), l = threadIdx.x & 63, hi = l >> 5, lc = l & 31;
  const int d = a.kv.d, G = a.G, tiles = a.wp / WG;  // (keys' tiles: 0 .. tiles - 1 shared out)
  // early keys have the most rows: theirs go first. K/V heads are neighbours: with 8 of them an XCD reads one head's rows
  uint32_t id = blockIdx.x;
  const int hk = id % a.kv.hkv;
  id /= a.kv.hkv;
  const int share = id % a.rs;
  id /= a.rs;
  const int s = id % a.sq.S, first = id / a.sq.S;
  const MassSeq m = mass_seq(a, s);
  if (m.q.n == 0 || m.rows == 0 || m.keys <= 0) return;
  const int* trow = a.sq.table + (long)s * a.sq.ldt;
  const long base = ((long)s * a.kv.hkv + hk) * a.W;

  for (int kt = first; (long)kt * WG < m.keys; kt += tiles) {
    // tiles past the expected longest sequence are not shared out: the first share takes all rows
    const bool split = a.rs > 1 && kt < tiles;
    if (a.rs > 1 && !split && share) break;
    const int wk = kt * WG + w * KT * 32;            // the wave's first key
    // K: lane holds key lc of each tile, 8 elements at 16 ks + 8 hi
    uint4 kf[KT][KS];
    uint32_t held[KT];
#pragma unroll
    for (int t = 0; t < KT; ++t) {
      const int j = wk + t * 32 + lc, pid = trow[min(j >> a.kv.psh, a.sq.cols - 1)];
      const bool ok = j < m.q.len && (unsigned)pid < (unsigned)a.kv.n_pages;
      held[t] = (uint32_t)__ballot(ok);
      const long r = (((long)(ok ? pid : 0) * a.kv.hkv + hk) << a.kv.psh) + (j & ((1 << a.kv.psh) - 1));
      const char* kp = a.kv.k + r * d * (C8 ? 1 : 2);
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        const int e = ks * 16 + hi * 8;
        kf[t][ks] = make_uint4(0, 0, 0, 0);
        if (ok && e < d) {
          if constexpr (!C8) kf[t][ks] = *reinterpret_cast<const uint4*>(kp + e * 2);
          else {
            const uint2 cd = *reinterpret_cast<const uint2*>(kp + e);
            if constexpr (BF) kf[t][ks] = codes8_bf16<KVM == 2>(cd);
            else {
              const uint2 x = codes4<KVM == 2>(cd.x), y = codes4<KVM == 2>(cd.y);
              kf[t][ks] = make_uint4(x.x, x.y, y.x, y.y);
            }
          }
        }
      }
      if (C8 && hi == 0) fk[w][t * 32 + lc] = ok ? a.kv.ks[r] * a.c : 0.f;
    }
    // factors of the scores 4 j .. 4 j + 3 of a lane and tile (written by this wave, and read behind the barrier below)
    auto factors = [&](int t, int j) {
      if constexpr (C8) return *reinterpret_cast<const f32x4*>(fk[w] + t * 32 + 8 * j + 4 * hi);
      else return f32x4{a.c, a.c, a.c, a.c};
    };
    bool every = true;                               // are all of the wave's keys held?
#pragma unroll
    for (int t = 0; t < KT; ++t) every &= held[t] == 0xFFFFFFFFu;
    float sum[KT][16];
#pragma unroll
    for (int t = 0; t < KT; ++t)
#pragma unroll
      for (int i = 0; i < 16; ++i) sum[t][i] = 0.f;

    // rows that see some key of the workgroup's, and this share of them
    const int k0 = kt * WG, k1 = min(k0 + WG, m.keys) - 1;
    const Tokens tk = tokens_of_keys(m.q.p0, m.n, k0, k1, a.window, a.sinks);
    const int r0 = tk.first * G, r1 = tk.end * G;
    int n_t = r1 > r0 ? (r1 - r0 + MROWS - 1) / MROWS : 0, t_0 = 0;
    if (split) {
      const int per = (n_t + a.rs - 1) / a.rs;
      t_0 = min(n_t, share * per);
      n_t = min(n_t, t_0 + per);
    }

    // A thread's rows of a tile: a load of the workgroup covers RPL of them. Where the query heads divide that, a thread's place in a
    // token is the same in all, and loads differ by a number of tokens only (the wave's own arithmetic); else token and head of
    // its first row are moved on a tile at a time.
    constexpr int RPL = 256 / CPR;
    const int ch = threadIdx.x % CPR, row = threadIdx.x / CPR, r_0 = r0 + t_0 * MROWS, step_i = MROWS / G, step_g = MROWS - step_i * G;
    const bool even = RPL % G == 0 && a.ldq <= 1 << 24, chunk = ch * 8 < d;
    int ti = (r_0 + row) / G, tg = r_0 + row - ti * G, si = (r_0 + (int)(threadIdx.x % MROWS)) / G, sg = r_0 + threadIdx.x % MROWS - si * G,
        left = r1 - r_0;
    // positions of a tile's first and last row
    int pa_i = m.q.p0 + r_0 / G, pa_g = r_0 % G, pb_i = m.q.p0 + (r_0 + MROWS - 1) / G, pb_g = (r_0 + MROWS - 1) % G;
    const char* qb = a.q + ((long)m.q.q0 * a.ldq + (long)hk * G * d) * 2;
    const char* qt = qb + (long)(r_0 / G) * (a.ldq * 2);
    const long step_t = (long)(RPL / G) * (a.ldq * 2);
    const uint32_t mine = (uint32_t)(row / G) * (uint32_t)(a.ldq * 2) + (uint32_t)(row % G * d * 2 + ch * 16);
    const float* lb = a.lse + (long)m.q.q0 * a.hq + hk * G;
    auto on = [&](int& i, int& g) {
      g += step_g;
      i += step_i + (g >= G);
      g -= g >= G ? G : 0;
    };
    uint4 st[LOADS];
#pragma unroll
    for (int i = 0; i < LOADS; ++i) st[i] = make_uint4(0, 0, 0, 0);
    float sl = 0.f;
    int sp = 0;
    // the next tile's (rows behind the last one keep what was there: they see nothing)
    auto fetch = [&] {
      if (chunk) {
        if (even && left >= MROWS) {
#pragma unroll
          for (int i = 0; i < LOADS; ++i) st[i] = *reinterpret_cast<const uint4*>(qt + i * step_t + mine);
        } else {
#pragma unroll
          for (int i = 0; i < LOADS; ++i) {
            int g = tg + i * RPL % G, n = ti + i * RPL / G;
            n += g >= G;
            g -= g >= G ? G : 0;
            if (i * RPL + row < left) st[i] = *reinterpret_cast<const uint4*>(qb + (long)n * (a.ldq * 2) + g * d * 2 + ch * 16);
          }
        }
      }
      if (even) {
        qt += LOADS * step_t;
        ti += step_i;
      } else {
        on(ti, tg);
      }
      if (threadIdx.x < MROWS) {
        sl = (int)threadIdx.x < left ? lb[(long)si * a.hq + sg] : -INFINITY;
        sp = sl == -INFINITY ? -1 : m.q.p0 + si;
        on(si, sg);
      }
      left -= MROWS;
    };
    auto put = [&](int b) {
#pragma unroll
      for (int i = 0; i < LOADS; ++i) {
        const int to = i * RPL + row;
        *reinterpret_cast<uint4*>(qs[b] + to * RB + ((ch ^ (to & (CPR - 1))) << 4)) = st[i];
      }
      if (threadIdx.x < MROWS) {
        Ls[b][threadIdx.x] = sl * LOG2E;
        ps[b][threadIdx.x] = sp;
      }
    };
    if (t_0 < n_t) {
      fetch();
      __syncthreads();                               // (a former tile's readers are through)
      put(0);
    }
    int t = t_0, b = 0;
    bool whole = false;
    // tile t is in LDS, the next one is fetched; is it one that every row sees whole?
    auto next = [&] {
      __syncthreads();
      if (t + 1 < n_t) fetch();
      whole = DP <= 128 && every && all_seen(a, pa_i, pb_i, wk, wk + KT * 32 - 1) && __all(ps[b][l] >= 0);
      on(pa_i, pa_g);
      on(pb_i, pb_g);
    };
    if (t < n_t) next();
    while (t < n_t) {
      // Such a tile: a product of 32 x 32 scores runs on the matrix core under the former one's exponentials (a loop of its own, so that
      // the sums stay in their registers). 2048 tokens over 6144, 64 heads on 8: 262 -> 235 us; head sizes over 128 have no registers
      // left for it (32 on 4 of 256: 268 -> 293).
      while (whole) {
        constexpr int N = MROWS / 32 * KT * KS, EL = 16 / KS;  // steps of one matrix instruction; scores a step
        uint4 qv[KS];
        f32x16 sc[2];
        f32x4 fc = factors(0, 0), fn = fc;           // this step's factors and the next ones
        float L[MROWS / 32], z[EL], e[EL];
        auto q16 = [&](int h, int ks) {
          const int row = h * 32 + lc;
          return *reinterpret_cast<const uint4*>(qs[b] + row * RB + (((ks * 2 + hi) ^ (row & (CPR - 1))) << 4));
        };
        auto product = [&](int n) {
          const int ks = n % KS, x = n / KS % KT, h = n / (KS * KT);
          f32x16& now = sc[n / KS & 1];
          if (ks == 0) {
#pragma unroll
            for (int i = 0; i < 16; ++i) now[i] = 0.f;
          }
          now = mfma32<BF>(kf[x][ks], qv[ks], now);
          if (x == KT - 1 && h + 1 < MROWS / 32) qv[ks] = q16(h + 1, ks);
        };
#pragma unroll
        for (int h = 0; h < MROWS / 32; ++h) L[h] = Ls[b][h * 32 + lc];
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) qv[ks] = q16(0, ks);
#pragma unroll
        for (int n = 0; n < KS; ++n) product(n);
        // step n adds the scores of step n - 3, takes the exponentials of those of n - 2, finds the exponents of those of n - 1 (the
        // empty statements keep a step's instructions together)
#pragma unroll
        for (int n = 0; n < N + 3; ++n) {
#pragma unroll
          for (int i = 0; i < EL; ++i) {
            if (n > 2) {
              float& to = sum[(n - 3) / KS % KT][(n - 3) % KS * EL + i];
              to += e[i];
              asm volatile("" : "+v"(to));
            }
            if (n > 1 && n < N + 2) {
              e[i] = exp2_fast(z[i]);
              asm volatile("" : "+v"(e[i]));
            }
            if (n > 0 && n < N + 1) {
              const int x = (n - 1) / KS, c = (n - 1) % KS * EL + i;
              if (c % 4 == 0) {
                fc = fn;
                fn = factors((x + c / 12) % KT, (c / 4 + 1) % 4);
              }
              z[i] = fmaf(sc[x & 1][c], fc[c % 4], -L[x / KT]);
              asm volatile("" : "+v"(z[i]));
            }
          }
          if (n + KS < N) product(n + KS);
          __builtin_amdgcn_sched_barrier(0);
        }
        if (t + 1 < n_t) put(b ^ 1);
        whole = false;
        if (++t < n_t) {
          b ^= 1;
          next();
        }
      }
      if (t >= n_t) break;
#pragma unroll
      for (int h = 0; h < MROWS / 32; ++h) {
        const int row = h * 32 + lc;
        const float L = Ls[b][row];
        const int p = ps[b][row], pa = m.q.p0 + (r0 + t * MROWS + h * 32) / G, pb = m.q.p0 + (r0 + t * MROWS + h * 32 + 31) / G;
        const bool lines = __all(p >= 0);
        f32x16 sc[KT];
#pragma unroll
        for (int x = 0; x < KT; ++x)
#pragma unroll
          for (int i = 0; i < 16; ++i) sc[x][i] = 0.f;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
          const uint4 qv = *reinterpret_cast<const uint4*>(qs[b] + row * RB + (((ks * 2 + hi) ^ (row & (CPR - 1))) << 4));
#pragma unroll
          for (int x = 0; x < KT; ++x) sc[x] = mfma32<BF>(kf[x][ks], qv, sc[x]);
        }
#pragma unroll
        for (int x = 0; x < KT; ++x) {
          const int ka = wk + x * 32;
          if (lines && held[x] == 0xFFFFFFFFu && all_seen(a, pa, pb, ka, ka + 31)) {
#pragma unroll
            for (int i = 0; i < 16; ++i) sum[x][i] += exp2_fast(fmaf(sc[x][i], factors(x, i >> 2)[i & 3], -L));
          } else if (some_seen(a, pa, pb, ka, ka + 31)) {
            // this lane's row sees its keys up to `last`, from `from` on or before `sink`, where they are held (the numbers are hidden
            // from the compiler, which would keep 32 comparisons' results over the loop)
            int last = p - ka - 4 * hi, from = last - a.window, sink = a.sinks - ka - 4 * hi;
            if (a.window <= 0) from = -1000;
            uint32_t have = held[x] >> (4 * hi);
            asm volatile("" : "+v"(last), "+v"(from), "+v"(sink), "+v"(have));
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const int kk = 8 * (i >> 2) + (i & 3);
              const float e = exp2_fast(fmaf(sc[x][i], factors(x, i >> 2)[i & 3], -L));
              const bool see = (kk <= last) & ((kk > from) | (kk < sink)) & (((have >> kk) & 1) != 0);
              sum[x][i] += see ? e : 0.f;
            }
          }
        }
      }
      if (t + 1 < n_t) put(b ^ 1);
      if (++t < n_t) {
        b ^= 1;
        next();
      }
    }
    // over the 32 lanes of each half; lane i (of 16) of a half then takes key register i
#pragma unroll
    for (int x = 0; x < KT; ++x) {
      float mine = 0.f;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float v = over16<false>(row16_sum(sum[x][i]));
        mine = (l & 15) == i ? v : mine;
      }
      const int i = l & 15, j = wk + x * 32 + 8 * (i >> 2) + 4 * hi + (i & 3);
      if ((l & 31) < 16 && j < m.keys) {
        if (split) a.part[(((long)s * a.kv.hkv + hk) * a.rs + share) * a.wp + j] = mine;
        else give(a, m, base, j, a.mass[base + j], mine);
      }
    }
  }
}

// The shares' sums in their order.
__global__ __launch_bounds__(256) void k_mass_join(MassArgs a) {
  const int hk = blockIdx.y, s = blockIdx.z, j = blockIdx.x * 256 + threadIdx.x;
  const MassSeq m = mass_seq(a, s);
  if (m.q.n == 0 || m.rows == 0 || j >= m.keys || j >= a.wp) return;
  const long base = ((long)s * a.kv.hkv + hk) * a.W, at = ((long)s * a.kv.hkv + hk) * a.rs * a.wp + j;
  float sum = 0.f;
  for (int i = 0; i < a.rs; ++i) sum += a.part[at + (long)i * a.wp];
  give(a, m, base, j, a.mass[base + j], sum);
}

template <int DP, int QB>
hipError_t few(const MassArgs& a, bool bf, int kvm, dim3 grid, hipStream_t st) {
#define GO(BF, KVM) hipLaunchKernelGGL((k_mass_few<BF, KVM, DP, QB>), grid, dim3(256), 0, st, a)
  if (bf) { if (kvm == 0) GO(true, 0); else if (kvm == 1) GO(true, 1); else GO(true, 2); }
  else { if (kvm == 0) GO(false, 0); else if (kvm == 1) GO(false, 1); else GO(false, 2); }
#undef GO
  return hipGetLastError();
}
template <int DP, int KT>
hipError_t many(const MassArgs& a, bool bf, int kvm, dim3 grid, hipStream_t st) {
#define GO(BF, KVM) hipLaunchKernelGGL((k_mass_many<BF, KVM, DP, KT>), grid, dim3(256), 0, st, a)
  if (bf) { if (kvm == 0) GO(true, 0); else if (kvm == 1) GO(true, 1); else GO(true, 2); }
  else { if (kvm == 0) GO(false, 0); else if (kvm == 1) GO(false, 1); else GO(false, 2); }
#undef GO
  return hipGetLastError();
}

}  // namespace

hipError_t sffn_launch_mass(const MassArgs& a, int qt, int kvt, int tiles, hipStream_t st) {
  const bool bf = qt == T_BF16;
  const int kvm = kvt == T_I8 ? 1 : kvt == T_E4M3 ? 2 : 0, d = a.kv.d;
  const long rows = (long)a.max_q * a.G;             // (max_q may be far over what the sequences have)
  if (mass_few(rows, d)) {
    const dim3 grid(tiles, a.kv.hkv, a.sq.S);
    if (d <= 64) return rows > 32 ? few<64, 4>(a, bf, kvm, grid, st) : rows > 16 ? few<64, 2>(a, bf, kvm, grid, st) : few<64, 1>(a, bf, kvm, grid, st);
    if (d <= 128) return rows > 32 ? few<128, 4>(a, bf, kvm, grid, st) : rows > 16 ? few<128, 2>(a, bf, kvm, grid, st) : few<128, 1>(a, bf, kvm, grid, st);
    return rows > 16 ? few<256, 2>(a, bf, kvm, grid, st) : few<256, 1>(a, bf, kvm, grid, st);
  }
  const dim3 grid((unsigned)tiles * a.rs * a.kv.hkv * a.sq.S);
  const hipError_t e = d <= 64 ? many<64, 2>(a, bf, kvm, grid, st) : d <= 128 ? many<128, 2>(a, bf, kvm, grid, st) : many<256, 1>(a, bf, kvm, grid, st);
  if (e != hipSuccess || a.rs == 1) return e;
  hipLaunchKernelGGL(k_mass_join, dim3((a.wp + 255) / 256, a.kv.hkv, a.sq.S), dim3(256), 0, st, a);
  return hipGetLastError();
}
