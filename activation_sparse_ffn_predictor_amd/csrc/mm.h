// Arguments of the block-scaled product's kernels (mm.hip), where their lanes read, and which of them a call takes.
#pragma once
#include <math.h>

#include <algorithm>

#include "attn.h"

namespace sffn {

struct MmArgs {
  const char *a, *b;        // codes [T, K], [N, K], rows lda, ldb apart
  const float *sa, *sb;     // [T, ceil(K / 128)], [ceil(N / 128), ceil(K / 128)]
  void* out;                // [T, N], rows ldo apart
  char* ws;
  long lda, ldb, ldo;
  int T, N, K;
};

// Memory that a buffer descriptor covers; `from`: without the first `off` bytes, nothing past the end. A load's scalar offset may or
// may not count in the range check, so nothing here hangs on it: rows that do not exist are turned away by the lane's offset alone,
// and the scalar one never exceeds the descriptor's bytes.
struct Span {
  const char* p;
  uint32_t bytes;
  __host__ __device__ __forceinline__ Span from(uint32_t off) const {
    const uint32_t o = off < bytes ? off : bytes;
    return {p + o, bytes - o};
  }
};
// rows r0 .. r0 + n - 1 of a matrix of codes, as far as they exist
__host__ __device__ __forceinline__ Span rows_of(const char* p, long ld, long r0, long rows, int n, int K) {
  const long have = rows - r0 < n ? rows - r0 : n;
  return {p + (have > 0 ? r0 * ld : 0), have > 0 ? (uint32_t)((have - 1) * ld + K) : 0u};
}
// Direct loads of 128 columns of a tile's rows: W waves beside each other take 8 rows each and turn, a lane 16 columns, from the row
// and column below. LDS holds a row's 16-byte chunk c in slot c ^ ((row >> 1) & 7); W is even, so a lane's swizzle is the same in
// every turn and one offset serves all.
__host__ __device__ __forceinline__ int lane_row(int w, int l) { return w * 8 + (l >> 3); }
__host__ __device__ __forceinline__ int lane_col(int row, int l) { return ((l & 7) ^ ((row >> 1) & 7)) << 4; }
// The rows of turn i. One without rows reads the tile's first ones (of which there are some) in their place: what it brings belongs to
// results that nobody stores. Descriptors of a whole turn each, once for all blocks: with the block's columns in them too, at nine
// scalar instructions a load, 1024 x 10240 x 8192 took 125 us for 119, 4096 tokens 365 for 352.
__host__ __device__ __forceinline__ Span turn_of(const Span& s, int i, int W, long ld) {
  const uint32_t off = (uint32_t)(i * W * 8) * (uint32_t)ld;
  return off < s.bytes ? s.from(off) : s;
}
// Block kb of them: the wave's offset (the last block's behind it), and whether the lane's column exists (`some`: is there such a block?)
struct Cols {
  uint32_t at;
  bool in;
};
__host__ __device__ __forceinline__ Cols cols_of(int kb, int KB, int K, int col, bool some) {
  return {(uint32_t)(kb < KB ? kb : KB - 1) * 128u, (bool)(some & ((kb < KB - 1) | ((KB - 1) * 128 + col < K)))};
}
// Factors of a tile's tokens (rows of KB): in slice p & 7 (SL tokens) of the 8 blocks behind those of block p, counted from k0 on, that
// of the slice's token ft and block fk. All of it in the lane's offset: descriptors of what a wave's part leaves would put a chain of
// scalar instructions before a block's first products (4096 x 10240 x 8192: 342 us for 339, 1024 tokens 114 for 111).
__host__ __device__ __forceinline__ uint32_t factor_at(int p, int SL, int KB, int k0, int ft, int fk) {
  return (uint32_t)(ft * KB + fk) * 4u + (uint32_t)(((p & 7) * SL * KB + (p & ~7) + 8 + k0) * 4);
}

// Which kernel, and over how many workgroups k is spread: the sum of measured costs decides. Workgroups take a block of k in `one`
// us when a compute unit has one of them and in `all` when it has as many as fit, at least a round of them; a join starts in 4 us and
// moves each partial result out and in at 5 TB/s. 10240 rows of K = 8192, us: 64 tokens SOME64 41, in three shares 30; 128 tokens
// SOME128 40, TILE128 in three shares 31; 256 tokens TILE128 59, in three shares 45; 512 tokens TILE128 82, TILE256 in three shares 63;
// 1024 tokens TILE128 128, TILE256 109; 2048 tokens 204 and 218; 4096 TILE256 340. Beside every other kernel and share that fits, for 20
// to 2048 tokens: of 10240 x 8192, 15360 x 5120, 8192 x 8192, 5120 x 5120, 2048 x 2048, 1024 x 8192 and 32768 x 4096 the choice is within
// 4% of the fastest in 55 of 63 calls and within 11% in all (512 x 5120 x 5120: 35.2 us, 31.7 with TILE128 in one share).
enum MmKernel { FEW, SOME32, SOME64, SOME128, TILE128, TILE256 };
struct MmShape {
  int n, t, fit;                                   // rows and tokens of a workgroup, workgroups a compute unit
  double one, all;
};
constexpr MmShape MM_SHAPES[] = {{16, 16, 4, 0, 0},        {64, 32, 3, 0.42, 0.75},   {64, 64, 2, 0.62, 0.9},
                            {64, 128, 1, 0.6, 0.6},   {128, 128, 2, 0.92, 1.28}, {256, 256, 1, 1.75, 1.75}};
struct MmPlan {
  int how, ks;
};
inline MmPlan mm_plan(int T, int N, int K, bool f32) {
  // few tokens' rows go to registers; past 4 tokens and 16 MB their loads outweigh what LDS costs (10240 x 8192: 16 tokens 31 us, by
  // LDS 22; 512 x 1024, 8 tokens: 4.9 and 5.6)
  if (T <= 4 || (T <= 16 && (long)N * K <= 1 << 24)) return {FEW, 1};
  const int KB = (K + 127) / 128, from = T <= 32 ? SOME32 : T <= 64 ? SOME64 : SOME128,
            to = T <= 32 ? SOME32 : T <= 64 ? SOME64 : f32 ? TILE128 : TILE256;
  MmPlan best{from, 1};
  double least = 0;
  for (int how = from; how <= to; ++how) {
    const MmShape& c = MM_SHAPES[how];
    const double tiles = (double)((N + c.n - 1) / c.n) * ((T + c.t - 1) / c.t);
    for (const int ks : {1, 2, 3, 4, 6, 8}) {
      if (ks > 1 && (KB < 4 * ks || tiles * ks > 512)) break;
      const double wgs = tiles * ks, fit = 256.0 * c.fit, turns = c.fit == 1 ? ceil(wgs / fit) : std::max({1.0, wgs / fit, ceil(wgs / fit) - 0.4});
      double us = turns * ((KB + ks - 1) / ks) * (wgs <= 256 ? c.one : c.all);
      if (ks > 1) us += 4.0 + (double)ks * T * N * 8 / 5e6;
      if (least == 0 || us < least) best = {how, ks}, least = us;
    }
  }
  return best;
}

}  // namespace sffn

size_t sffn_mm_workspace(int T, int N, int K);
hipError_t sffn_launch_mm(const sffn::MmArgs& a, int ot, hipStream_t st);
