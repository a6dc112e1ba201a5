// Root-mean-square norms of queries and keys for each head and the position rotation, in one pass over them.
//   y = x / sqrt(mean(x^2) + eps) * w            (norm; else y = x)
//   (y_a, y_b) <- (y_a cos - y_b sin, y_b cos + y_a sin), angle = position * freq[i], for the pairs of the first `rot` elements
//
// Bound by memory: q and k read and written once. Measured: 4500 tokens of 80 heads of 128, bf16, 182 MB in 40.5 us (4.5 TB/s; a large
// copy reaches 5.55; two to eight tokens a workgroup, or fewer registers, are slower); one token of 72 heads 3.5 us on the device, a
// launch and a chain of three loads. Angles: position * freq and its reduction to turns in 64 bits, so that far positions keep what
// fp32 would lose (at 10^6 an fp32 angle is off by 0.03), then sine and cosine of the fraction in 32; each is worked out once for a
// token and shared by its heads through LDS.
#include "attn.h"

using namespace sffn;

namespace {

struct RopeArgs {
  const char *q, *k;
  char *qo, *ko;
  const float *wq, *wk, *freq;
  const int *cu, *len;
  long ldq, ldk, ldqo, ldko;
  double eps;
  int S, T, hq, hk, d, rot, inter, norm;
};

constexpr int ROPE_TOKENS = 8;                     // of a workgroup, at most

__device__ __forceinline__ double shfl_xor_d(double v, int o) {
  return __hiloint2double(__shfl_xor(__double2hiint(v), o, WAVE), __shfl_xor(__double2loint(v), o, WAVE));
}

// P consecutive 16-bit values (4 or 8) as they lie in memory
template <int P>
struct Piece {
  uint32_t u[P / 2];
  __device__ __forceinline__ void load(const char* p) {
    if constexpr (P == 8) {
      const uint4 v = *reinterpret_cast<const uint4*>(p);
      u[0] = v.x; u[1] = v.y; u[2] = v.z; u[3] = v.w;
    } else {
      const uint2 v = *reinterpret_cast<const uint2*>(p);
      u[0] = v.x; u[1] = v.y;
    }
  }
  template <bool BF>
  __device__ __forceinline__ void values(float* f) const {
#pragma unroll
    for (int i = 0; i < P / 2; ++i) {
      f[2 * i] = lo16<BF>(u[i]);
      f[2 * i + 1] = hi16<BF>(u[i]);
    }
  }
};
template <int P, bool BF>
__device__ __forceinline__ void store_piece(char* p, const float* f) {
  if constexpr (P == 8)
    *reinterpret_cast<uint4*>(p) = make_uint4(pack2<BF>(f[0], f[1]), pack2<BF>(f[2], f[3]), pack2<BF>(f[4], f[5]), pack2<BF>(f[6], f[7]));
  else
    *reinterpret_cast<uint2*>(p) = make_uint2(pack2<BF>(f[0], f[1]), pack2<BF>(f[2], f[3]));
}

// LPH lanes hold a head, two pieces of P elements each: the two halves of P pairs (rotated in halves), or places half a head apart,
// so that what neighbouring lanes load lies side by side. A
// workgroup takes `tokens` tokens and, of each, a share of the heads; a thread's next row loads while positions and angles are
// found and while its present one is worked on (more rows ahead leave fewer waves: 4500 tokens of 80 heads 42 us with one, 45 with two,
// 50 with three).
template <int P, int LPH, bool BF>
__global__ __launch_bounds__(256) void k_rope(RopeArgs a, int tokens, int shares, int first) {
  __shared__ float2 turn[ROPE_TOKENS * 128];
  __shared__ int where[ROPE_TOKENS];
  __shared__ __align__(16) float gain[2][256];       // (in LDS: loads of them would wait for the rows' that are on their way)
  constexpr int SLOTS = 256 / LPH;
  const int t0 = first + blockIdx.x / shares * tokens, sh = blockIdx.x % shares;
  const int heads = a.hq + a.hk, per = (heads + shares - 1) / shares, h0 = sh * per, nh = min(per, heads - h0);
  const int here = min(tokens, min(a.T, max(a.cu[a.S], 0)) - t0);      // rows behind the last sequence stay as they are
  if (here <= 0 || nh <= 0) return;
  const int m = a.rot >> 1, items = here * nh;
  const float over_d = 1.f / (float)a.d, eps = (float)a.eps;
  const int slot = threadIdx.x / LPH, l = threadIdx.x % LPH;
  // rotated in halves, the pieces behind the rotated part are neighbours instead
  const bool halves = !a.inter && m > 0, half = halves && l * P < m, act = l * 2 * P < a.d;
  const int e0 = halves && !half ? l * 2 * P : l * P, e1 = half ? e0 + m : halves ? e0 + P : e0 + (a.d >> 1);

  Piece<P> raw[2] = {};
  auto fetch = [&](int i) {
    if (!act || i >= items) return;
    const int tt = i / nh, hh = h0 + i - tt * nh, t = t0 + tt;
    const char* p = hh < a.hq ? a.q + (t * a.ldq + (long)hh * a.d) * 2 : a.k + (t * a.ldk + (long)(hh - a.hq) * a.d) * 2;
    raw[0].load(p + e0 * 2);
    raw[1].load(p + e1 * 2);
  };
  fetch(slot);
  if (a.norm)
    for (int i = threadIdx.x; i < 2 * a.d; i += 256) {
      const int k = i >= a.d, e = i - k * a.d;
      const float* w = k ? a.wk : a.wq;
      gain[k][e] = w ? w[e] : 1.f;
    }
  if (m)
    for (int tt = threadIdx.x >> 6; tt < here; tt += 4) {
      const int s = min(find_seq<64>(a.cu, a.S, t0 + tt), a.S - 1);
      if ((threadIdx.x & 63) == 0) where[tt] = token_pos(a.len[s], max(a.cu[s + 1], 0), t0 + tt);
    }
  __syncthreads();
  if (m) {
    for (int i = threadIdx.x; i < here * m; i += 256) {
      const int tt = i / m;
      const double turns = (double)where[tt] * (double)a.freq[i - tt * m] * 0.15915494309189535;
      float s, c;
      sincospif(2.f * (float)(turns - rint(turns)), &s, &c);
      turn[i] = make_float2(c, s);
    }
    __syncthreads();
  }

  for (int i = slot; i < items; i += SLOTS) {
    const int tt = i / nh, hh = h0 + i - tt * nh, t = t0 + tt;
    float x[2][P];
    raw[0].template values<BF>(x[0]);
    raw[1].template values<BF>(x[1]);
    fetch(i + SLOTS);
    if (a.norm) {
      const float* w = gain[hh < a.hq ? 0 : 1];
      float g[2][P], sum = 0.f;
#pragma unroll
      for (int j = 0; j < P; ++j) {
        g[0][j] = act ? w[e0 + j] : 1.f;
        g[1][j] = act ? w[e1 + j] : 1.f;
      }
#pragma unroll
      for (int j = 0; j < P; ++j) sum = fmaf(x[0][j], x[0][j], fmaf(x[1][j], x[1][j], sum));
      sum = group_sum<LPH>(sum);
      const float mean = fmaf(sum, over_d, eps);
      if (mean >= 1e-30f && mean < INFINITY) {
        // the unit's estimate and one step of Newton's method (a division and a root in full: 41.2 us for 40.5 of the tokens above)
        const float near = __builtin_amdgcn_rsqf(mean), rs = fmaf(0.5f * near, fmaf(-mean * near, near, 1.f), near);
#pragma unroll
        for (int j = 0; j < P; ++j) {
          x[0][j] = x[0][j] * rs * g[0][j];
          x[1][j] = x[1][j] * rs * g[1][j];
        }
      } else {                                     // squares outside fp32's range (or a zero head without eps): in 64 bits
        double q = 0.0;
#pragma unroll
        for (int j = 0; j < P; ++j) q = fma((double)x[0][j], (double)x[0][j], fma((double)x[1][j], (double)x[1][j], q));
#pragma unroll
        for (int o = LPH / 2; o; o >>= 1) q += shfl_xor_d(q, o);
        const double rs = 1.0 / sqrt(q / (double)a.d + a.eps);
#pragma unroll
        for (int j = 0; j < P; ++j) {
          x[0][j] = (float)((double)x[0][j] * rs * (double)g[0][j]);
          x[1][j] = (float)((double)x[1][j] * rs * (double)g[1][j]);
        }
      }
    }
    if (half) {
      const float2* cs = turn + tt * m + e0;
#pragma unroll
      for (int j = 0; j < P; ++j) {
        const float2 v = cs[j];
        const float p = x[0][j], r = x[1][j];
        x[0][j] = p * v.x - r * v.y;
        x[1][j] = r * v.x + p * v.y;
      }
    } else if (a.inter) {
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const int e = b ? e1 : e0;
        if (e >= a.rot) continue;
        const float2* cs = turn + tt * m + (e >> 1);
#pragma unroll
        for (int j = 0; j < P; j += 2) {
          const float2 v = cs[j / 2];
          const float p = x[b][j], r = x[b][j + 1];
          x[b][j] = p * v.x - r * v.y;
          x[b][j + 1] = r * v.x + p * v.y;
        }
      }
    }
    if (act) {
      char* to = hh < a.hq ? a.qo + (t * a.ldqo + (long)hh * a.d) * 2 : a.ko + (t * a.ldko + (long)(hh - a.hq) * a.d) * 2;
      store_piece<P, BF>(to + e0 * 2, x[0]);
      store_piece<P, BF>(to + e1 * 2, x[1]);
    }
  }
}

template <int P, int LPH>
hipError_t go(const RopeArgs& a, bool bf, hipStream_t st) {
  constexpr int SLOTS = 256 / LPH;
  const int heads = a.hq + a.hk;
  // several tokens a workgroup where one has few heads; a token's heads over several workgroups where tokens are few
  const int tokens = heads >= SLOTS ? 1 : SLOTS / heads < ROPE_TOKENS ? SLOTS / heads : ROPE_TOKENS;
  const int groups = (a.T + tokens - 1) / tokens, most = (heads + SLOTS - 1) / SLOTS;
  int shares = groups >= 1024 ? 1 : (1024 + groups - 1) / groups;
  shares = shares < most ? shares : most;
  constexpr int MOST = 1 << 22;                    // a launch holds fewer than 2^32 threads: more tokens go in several
  hipError_t e = hipSuccess;
  for (int g = 0; g < groups && e == hipSuccess; g += MOST) {
    const dim3 grid((unsigned)(groups - g < MOST ? groups - g : MOST) * shares);
    if (bf) hipLaunchKernelGGL((k_rope<P, LPH, true>), grid, dim3(256), 0, st, a, tokens, shares, g * tokens);
    else hipLaunchKernelGGL((k_rope<P, LPH, false>), grid, dim3(256), 0, st, a, tokens, shares, g * tokens);
    e = hipGetLastError();
  }
  return e;
}

}  // namespace

hipError_t sffn_launch_rope(int type, const int* cu, const int* len, int S, int T, const void* q, long ldq, int hq,
                            const void* k, long ldk, int hk, int d, int norm, const float* wq, const float* wk, double eps,
                            const float* freq, int rot, int inter, void* qo, long ldqo, void* ko, long ldko, hipStream_t st) {
  const RopeArgs a{(const char*)q, (const char*)k, (char*)qo, (char*)ko, wq, wk, freq, cu, len, ldq, ldk, ldqo, ldko, eps,
                   S, T, hq, k ? hk : 0, d, rot, inter, norm};
  const bool bf = type == T_BF16;
  // 16-byte pieces where halves and heads are whole numbers of them, else pieces of 8 bytes
  if (d % 16 == 0 && rot % 16 == 0) {
    if (d <= 16) return go<8, 1>(a, bf, st);
    if (d <= 32) return go<8, 2>(a, bf, st);
    if (d <= 64) return go<8, 4>(a, bf, st);
    if (d <= 128) return go<8, 8>(a, bf, st);
    return go<8, 16>(a, bf, st);
  }
  if (d <= 16) return go<4, 2>(a, bf, st);
  if (d <= 32) return go<4, 4>(a, bf, st);
  if (d <= 64) return go<4, 8>(a, bf, st);
  if (d <= 128) return go<4, 16>(a, bf, st);
  return go<4, 32>(a, bf, st);
}
