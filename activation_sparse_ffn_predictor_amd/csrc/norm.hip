// Root-mean-square norm with the residual's addition.
//   h = x + res (fp32), res_out = h rounded to the residual's type, y = h / sqrt(mean(h^2) + eps) * w
// y as 32 or 16 bits, or as int8 / e4m3 codes with one fp32 scale per row (max|y| / 127 or / 448).
//
// Bound by memory: x, res read, h, y written, once each. Measured: 4099 rows of 8192, fp32 + fp32 to int8, 437 MB in 81 us
// (5.4 TB/s; a large copy reaches 5.55); one row of 4096 2.2 us on the device, a launch and one round trip.
#include "attn.h"

using namespace sffn;

namespace {

// 8 consecutive elements of a row, widened; nothing past D is read (D % 8 == 0)
__device__ __forceinline__ void load8(const void* p, int type, long i, float* f) {
  if (type == T_F32) {
    const float4 a = reinterpret_cast<const float4*>((const float*)p + i)[0];
    const float4 b = reinterpret_cast<const float4*>((const float*)p + i)[1];
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
    return;
  }
  const uint4 u = *reinterpret_cast<const uint4*>((const char*)p + 2 * i);
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    f[2 * k] = type == T_F16 ? lo16<false>(w[k]) : lo16<true>(w[k]);
    f[2 * k + 1] = type == T_F16 ? hi16<false>(w[k]) : hi16<true>(w[k]);
  }
}
__device__ __forceinline__ void store8(void* p, int type, long i, const float* f) {
  if (type == T_F32) {
    reinterpret_cast<float4*>((float*)p + i)[0] = make_float4(f[0], f[1], f[2], f[3]);
    reinterpret_cast<float4*>((float*)p + i)[1] = make_float4(f[4], f[5], f[6], f[7]);
  } else if (type == T_F16) {
    *reinterpret_cast<uint4*>((char*)p + 2 * i) = make_uint4(pack2<false>(f[0], f[1]), pack2<false>(f[2], f[3]),
                                                             pack2<false>(f[4], f[5]), pack2<false>(f[6], f[7]));
  } else {
    *reinterpret_cast<uint4*>((char*)p + 2 * i) = make_uint4(pack2<true>(f[0], f[1]), pack2<true>(f[2], f[3]),
                                                             pack2<true>(f[4], f[5]), pack2<true>(f[6], f[7]));
  }
}

__device__ __forceinline__ double shfl_xor_d(double v, int o) {
  return __hiloint2double(__shfl_xor(__double2hiint(v), o, WAVE), __shfl_xor(__double2loint(v), o, WAVE));
}

// code of a value on the 8-bit grid, from 64 bits: int8 by rint; e4m3 through an fp32 value with a sticky last bit,
// whose rounding to 4 significant bits is that of the 64-bit value
template <bool E4M3>
__device__ __forceinline__ uint32_t code4(const double* v) {
  if constexpr (E4M3) {
    float f[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const double c = fmin(fmax(v[i], -448.0), 448.0);
      float q = (float)c;
      if ((double)q != c) {
        uint32_t b = __float_as_uint(q);
        if (fabs((double)q) > fabs(c)) b -= 1;
        q = __uint_as_float(b | 1u);
      }
      f[i] = v[i] == v[i] ? q : 0.f;
    }
    int u = __builtin_amdgcn_cvt_pk_fp8_f32(f[0], f[1], 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(f[2], f[3], u, true);
  } else {
    uint32_t u = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const double c = fmin(fmax(rint(v[i]), -127.0), 127.0);
      u |= (uint32_t)((v[i] == v[i] ? (int)c : 0) & 255) << (8 * i);
    }
    return u;
  }
}

// sum of a row's squares in 64 bits, the same in every thread (part: LDS of a double a wave)
template <int WPR, int CH>
__device__ __forceinline__ double square_sum(const float (&h)[CH][8], double* part, int wv, int lane) {
  double q = 0.0;
#pragma unroll
  for (int c = 0; c < CH; ++c)
#pragma unroll
    for (int k = 0; k < 8; ++k) q = fma((double)h[c][k], (double)h[c][k], q);
#pragma unroll
  for (int o = 32; o; o >>= 1) q += shfl_xor_d(q, o);
  if (WPR > 1) {
    if (lane == 0) part[wv] = q;
    __syncthreads();
    q = part[0];
#pragma unroll
    for (int k = 1; k < WPR; ++k) q += part[k];
  }
  return q;
}

// WPR waves a row, CH chunks of 8 elements per lane: D <= 512 * WPR * CH. One chunk a lane wherever 1024 threads hold a
// row (4099 rows of 8192 to int8: 97 us on 4 waves, 93 on 8, 81 on 16). The row stays in registers
// between its sum and its output, so every byte is read and written once. YQ: 0 = 16 / 32 bits out, 1 = int8,
// 2 = e4m3. An 8-bit output is computed in 64 bits from the fp32 sums h on (the fp64 units are idle in a kernel that
// waits for memory): codes are then those of the formula, whatever the order of the sum, but for quotients within
// 1e-15 of a border.
template <int WPR, int CH, int YQ>
__global__ __launch_bounds__(WPR > 4 ? WPR * 64 : 256) void k_add_rmsnorm(const void* __restrict__ x, int xt, const void* res, int rt,
                                                     const float* __restrict__ w, double eps, int T, int D, long ldx,
                                                     long ldr, void* __restrict__ y, int yt, float* __restrict__ ys,
                                                     void* res_out, long ldy, long ldro) {
  __shared__ double red[2][WPR > 1 ? WPR : 1];
  const int wv = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int row = WPR == 1 ? blockIdx.x * 4 + wv : blockIdx.x;
  if (WPR == 1 && row >= T) return;
  const int t = WPR == 1 ? lane : threadIdx.x;
  float h[CH][8], g[CH][8];
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int i = (c * WPR * 64 + t) * 8;
    if (i < D) load8(x, xt, row * ldx + i, h[c]);
    else
#pragma unroll
      for (int k = 0; k < 8; ++k) h[c][k] = 0.f;
  }
  if (res) {
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int i = (c * WPR * 64 + t) * 8;
      if (i < D) load8(res, rt, row * ldr + i, g[c]);
      else
#pragma unroll
        for (int k = 0; k < 8; ++k) g[c][k] = 0.f;
    }
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
      for (int k = 0; k < 8; ++k) h[c][k] += g[c][k];
  }
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int i = (c * WPR * 64 + t) * 8;
    if (w && i < D) load8(w, T_F32, i, g[c]);
    else
#pragma unroll
      for (int k = 0; k < 8; ++k) g[c][k] = 1.f;
  }
  if (res_out) {
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int i = (c * WPR * 64 + t) * 8;
      if (i < D) store8(res_out, rt, row * ldro + i, h[c]);
    }
  }
  if constexpr (YQ == 0) {
    float q = 0.f;
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
      for (int k = 0; k < 8; ++k) q = fmaf(h[c][k], h[c][k], q);
    q = wave_sum(q);
    if (WPR > 1) {
      float* r = reinterpret_cast<float*>(red[0]);
      if (lane == 0) r[wv] = q;
      __syncthreads();
      q = r[0];
#pragma unroll
      for (int k = 1; k < WPR; ++k) q += r[k];
    }
    const float mean = q / (float)D + (float)eps;
    if (mean >= 1e-30f && mean < INFINITY) {
      const float rs = 1.0f / sqrtf(mean);
#pragma unroll
      for (int c = 0; c < CH; ++c)
#pragma unroll
        for (int k = 0; k < 8; ++k) h[c][k] = h[c][k] * rs * g[c][k];
    } else {                                // squares outside fp32's range (or a zero row without eps): again in 64 bits
      const double rs = 1.0 / sqrt(square_sum<WPR, CH>(h, red[1], wv, lane) / (double)D + eps);
#pragma unroll
      for (int c = 0; c < CH; ++c)
#pragma unroll
        for (int k = 0; k < 8; ++k) h[c][k] = (float)((double)h[c][k] * rs * (double)g[c][k]);
    }
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int i = (c * WPR * 64 + t) * 8;
      if (i < D) store8(y, yt, row * ldy + i, h[c]);
    }
  } else {
    const double q = square_sum<WPR, CH>(h, red[0], wv, lane);
    const double rs = 1.0 / sqrt(q / (double)D + eps);
    double big = 0.0;                       // largest |h w| (times rs below); NaN is looked for apart
    bool bad = false;
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const double v = fabs((double)h[c][k] * (double)g[c][k]);
        bad |= !(v < 1.7e308);
        big = fmax(big, v);
      }
    bad |= !(rs < 1.7e308);
#pragma unroll
    for (int o = 32; o; o >>= 1) big = fmax(big, shfl_xor_d(big, o));
    bad = __any(bad);
    if (WPR > 1) {
      if (lane == 0) red[1][wv] = bad ? __longlong_as_double(0x7FF0000000000000ll) : big;
      __syncthreads();
#pragma unroll
      for (int k = 0; k < WPR; ++k) big = fmax(big, red[1][k]);
      bad = !(big < 1.7e308);
    }
    // the scale is the fp32 rounding of max|y| / top; a row with an infinity or NaN gets the scale NaN and codes 0
    const float sc = bad ? __uint_as_float(0x7FC00000u) : (float)(big * rs / (YQ == 1 ? 127.0 : 448.0));
    const double f = sc > 0.f ? rs / (double)sc : 0.0;
    if (t == 0) ys[row] = sc;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int i = (c * WPR * 64 + t) * 8;
      double v[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = bad ? 0.0 : (double)h[c][k] * (double)g[c][k] * f;
      if (i < D) *reinterpret_cast<uint2*>((char*)y + row * ldy + i) = make_uint2(code4<YQ == 2>(v), code4<YQ == 2>(v + 4));
    }
  }
}

}  // namespace

hipError_t sffn_launch_add_rmsnorm(const void* x, int xt, const void* res, int rt, const float* w, double eps, int T,
                                   int D, long ldx, long ldr, void* y, int yt, float* ys, void* res_out, long ldy,
                                   long ldro, hipStream_t st) {
  const int yq = yt == T_I8 ? 1 : yt == T_E4M3 ? 2 : 0;
  // a launch holds fewer than 2^32 threads, 4 million rows of 1024: more rows go in several
  constexpr int MOST = 1 << 21;
  if (T > MOST) {
    auto size = [](int t) { return t == T_F32 ? 4 : t == T_I8 || t == T_E4M3 ? 1 : 2; };
    hipError_t e = hipSuccess;
    for (int r = 0; r < T && e == hipSuccess; r += MOST) {
      const long o = r;
      e = sffn_launch_add_rmsnorm((const char*)x + o * ldx * size(xt), xt, res ? (const char*)res + o * ldr * size(rt) : nullptr, rt,
                                  w, eps, T - r < MOST ? T - r : MOST, D, ldx, ldr, (char*)y + o * ldy * size(yt), yt,
                                  ys ? ys + o : nullptr, res_out ? (char*)res_out + o * ldro * size(rt) : nullptr, ldy, ldro, st);
    }
    return e;
  }
#define GO(WPR, CH, YQ)                                                                                           \
  hipLaunchKernelGGL((k_add_rmsnorm<WPR, CH, YQ>), dim3(WPR == 1 ? (T + 3) / 4 : T), dim3(WPR > 4 ? WPR * 64 : 256), 0, st, x, xt, \
                     res, rt, \
                     w, eps, T, D, ldx, ldr, y, yt, ys, res_out, ldy, ldro)
#define PICK(WPR, CH) \
  if (yq == 0) GO(WPR, CH, 0); else if (yq == 1) GO(WPR, CH, 1); else GO(WPR, CH, 2)
  if (D <= 512) { PICK(1, 1); }
  else if (D <= 2048) { PICK(4, 1); }
  else if (D <= 4096) { PICK(8, 1); }
  else if (D <= 8192) { PICK(16, 1); }
  else { PICK(16, 2); }
#undef PICK
#undef GO
  return hipGetLastError();
}
