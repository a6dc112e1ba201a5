// Blocks of 128 columns (of one row, or of 128 rows) as e4m3 codes with one fp32 scale each:
//   scale = fp32(max|x| / 448),  code = x / scale to nearest even, from the exact quotient
// A scale below 2^-60 becomes 0 (codes 0), a block with an infinity or NaN gets the scale NaN (codes 0), as in the cache.
//
// Bound by memory: x read and the codes written, once each (a block stays in registers between its maximum and its codes).
// Measured: 10184 x 8192 fp32 in blocks of 128 rows, 417 MB, 73 us (5.7 TB/s; a large copy reaches 5.55); 4099 x 8192 bf16 rows, 101 MB,
// 21 us (4.8); one row 3.9 us a call, its host side.
#include "codes.h"

using namespace sffn;

namespace {

// 8 elements as they lie in memory, their values and the bit pattern of their largest magnitude (those of floats ascend with
// them, infinities and NaN on top)
template <int XT>
struct Eight {
  uint4 a, b;                                     // b: fp32 only
  __device__ __forceinline__ void load(const char* p, long i) {
    const uint4* s = reinterpret_cast<const uint4*>(p + i * (XT == T_F32 ? 4 : 2));
    a = s[0];
    if (XT == T_F32) b = s[1];
  }
  __device__ __forceinline__ void clear() { a = b = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void values(float* f) const {
    if constexpr (XT == T_F32) {
      f[0] = __uint_as_float(a.x); f[1] = __uint_as_float(a.y); f[2] = __uint_as_float(a.z); f[3] = __uint_as_float(a.w);
      f[4] = __uint_as_float(b.x); f[5] = __uint_as_float(b.y); f[6] = __uint_as_float(b.z); f[7] = __uint_as_float(b.w);
    } else {
      const uint32_t u[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        f[2 * k] = lo16<XT == T_BF16>(u[k]);
        f[2 * k + 1] = hi16<XT == T_BF16>(u[k]);
      }
    }
  }
  __device__ __forceinline__ uint32_t largest() const {
    if constexpr (XT == T_F32) {
      const uint32_t m = 0x7FFFFFFFu;
      return max(max(max(a.x & m, a.y & m), max(a.z & m, a.w & m)), max(max(b.x & m, b.y & m), max(b.z & m, b.w & m)));
    } else {
      typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
      const uint32_t u[4] = {a.x, a.y, a.z, a.w};
      u16x2 mx = {0, 0};
#pragma unroll
      for (int i = 0; i < 4; ++i) mx = __builtin_elementwise_max(mx, __builtin_bit_cast(u16x2, u[i] & 0x7FFF7FFFu));
      return (uint32_t)max(mx.x, mx.y);
    }
  }
};
// scale of a block from its largest magnitude's bit pattern; NaN where that is none of a finite value
template <int XT>
__device__ __forceinline__ float block_scale(uint32_t big) {
  if (big >= (XT == T_F32 ? 0x7F800000u : XT == T_F16 ? 0x7C00u : 0x7F80u)) return __uint_as_float(0x7FC00000u);
  float s;
  if constexpr (XT == T_F32) s = __fdiv_rn(__uint_as_float(big), 448.f);
  else s = over_top<448>(lo16<XT == T_BF16>(big));
  return s < KV_MIN_SCALE ? 0.f : s;
}
template <int XT>
__device__ __forceinline__ uint2 block_codes(const Eight<XT>& x, float s) {
  float f[8];
  x.values(f);
  const bool some = s > 0.f;                      // (not NaN)
  const uint2 c = encode8<true, XT != T_F16>(f, some ? s : 1.f);
  return some ? c : make_uint2(0, 0);
}

// One row a block: 16 lanes hold one, 8 elements each. A workgroup takes 1 << lc blocks of columns of 16 >> lc rows at a time.
template <int XT>
__global__ __launch_bounds__(256) void k_quant_rows(const char* __restrict__ x, long ldx, int T, int D, int lc, int nc,
                                                    long tiles, char* __restrict__ y, long ldy, float* __restrict__ ys) {
  const int cb = (D + 127) >> 7, g = threadIdx.x >> 4, lane = threadIdx.x & 15;
  for (long i = blockIdx.x; i < tiles; i += gridDim.x) {
    const int c = (int)(i % nc) << lc | (g & ((1 << lc) - 1)), col = c * 128 + lane * 8;
    const long row = (i / nc) * (16 >> lc) + (g >> lc);
    const bool have = row < T && col < D;
    Eight<XT> e;
    e.clear();
    if (have) e.load(x, row * ldx + col);
    const float s = block_scale<XT>(group_max<16>(e.largest()));
    const uint2 code = block_codes<XT>(e, s);
    if (have) *reinterpret_cast<uint2*>(y + row * ldy + col) = code;
    if (row < T && c < cb && lane == 0) ys[row * cb + c] = s;
  }
}

// 128 rows a block: one workgroup, 8 rows a thread, which stay in registers.
template <int XT>
__global__ __launch_bounds__(256) void k_quant_tile(const char* __restrict__ x, long ldx, int T, int D, long tiles,
                                                    char* __restrict__ y, long ldy, float* __restrict__ ys) {
  __shared__ uint32_t part[2][4];
  const int cb = (D + 127) >> 7, r0 = threadIdx.x >> 4, lane = threadIdx.x & 15;
  int turn = 0;
  for (long i = blockIdx.x; i < tiles; i += gridDim.x, turn ^= 1) {
    const int c = (int)(i % cb), col = c * 128 + lane * 8;
    const long row = (i / cb) * 128 + r0;
    Eight<XT> e[8];
    uint32_t big = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      e[k].clear();
      if (row + 16 * k < T && col < D) e[k].load(x, (row + 16 * k) * ldx + col);
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) big = max(big, e[k].largest());
    big = group_max<16>(big);
    big = max(big, (uint32_t)__shfl_xor((int)big, 16, WAVE));
    big = max(big, (uint32_t)__shfl_xor((int)big, 32, WAVE));
    if ((threadIdx.x & 63) == 0) part[turn][threadIdx.x >> 6] = big;
    __syncthreads();                              // (the other turn's places are read before this one)
    big = max(max(part[turn][0], part[turn][1]), max(part[turn][2], part[turn][3]));
    const float s = block_scale<XT>(big);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const uint2 code = block_codes<XT>(e[k], s);
      if (row + 16 * k < T && col < D) *reinterpret_cast<uint2*>(y + (row + 16 * k) * ldy + col) = code;
    }
    if (threadIdx.x == 0) ys[i] = s;
  }
}

}  // namespace

hipError_t sffn_launch_quant128(const void* x, int xt, long ldx, int T, int D, int rows, void* y, long ldy, float* ys,
                                hipStream_t st) {
  constexpr long MOST = 1 << 20;                  // workgroups of a launch; more tiles are taken in turn
  const int cb = (D + 127) >> 7;
  const char* xc = (const char*)x;
  if (rows == 1) {
    int lc = 0;                                   // as many of the 16 blocks beside each other as there are columns for
    while (lc < 4 && (1 << lc) < cb) ++lc;
    const int nc = (cb + (1 << lc) - 1) >> lc, rpt = 16 >> lc;
    const long tiles = ((long)T + rpt - 1) / rpt * nc;
    const dim3 grid((unsigned)(tiles < MOST ? tiles : MOST));
    if (xt == T_F32) hipLaunchKernelGGL(k_quant_rows<T_F32>, grid, dim3(256), 0, st, xc, ldx, T, D, lc, nc, tiles, (char*)y, ldy, ys);
    else if (xt == T_F16) hipLaunchKernelGGL(k_quant_rows<T_F16>, grid, dim3(256), 0, st, xc, ldx, T, D, lc, nc, tiles, (char*)y, ldy, ys);
    else hipLaunchKernelGGL(k_quant_rows<T_BF16>, grid, dim3(256), 0, st, xc, ldx, T, D, lc, nc, tiles, (char*)y, ldy, ys);
  } else {
    const long tiles = ((long)T + 127) / 128 * cb;
    const dim3 grid((unsigned)(tiles < MOST ? tiles : MOST));
    if (xt == T_F32) hipLaunchKernelGGL(k_quant_tile<T_F32>, grid, dim3(256), 0, st, xc, ldx, T, D, tiles, (char*)y, ldy, ys);
    else if (xt == T_F16) hipLaunchKernelGGL(k_quant_tile<T_F16>, grid, dim3(256), 0, st, xc, ldx, T, D, tiles, (char*)y, ldy, ys);
    else hipLaunchKernelGGL(k_quant_tile<T_BF16>, grid, dim3(256), 0, st, xc, ldx, T, D, tiles, (char*)y, ldy, ys);
  }
  return hipGetLastError();
}
