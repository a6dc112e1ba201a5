// Arguments of the block-scaled product's kernels (mm.hip), and where their lanes read.
#pragma once
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
// Block kb of them: the wave's offset, and whether the lane's column exists (`some`: is there such a block?)
struct Cols {
  uint32_t at;
  bool in;
};
__host__ __device__ __forceinline__ Cols cols_of(int kb, int KB, int K, int col, bool some) {
  return {some ? (uint32_t)kb * 128u : 0u, (bool)(some & ((kb < KB - 1) | ((KB - 1) * 128 + col < K)))};
}
// Factors of a tile's tokens (rows of KB): in slice p & 7 (SL tokens) of the 8 blocks behind those of block p, counted from k0 on
__host__ __device__ __forceinline__ Span factors_of(const Span& s, int p, int SL, int KB, int k0) {
  return s.from((uint32_t)(((p & 7) * SL * KB + (p & ~7) + 8 + k0) * 4));
}

}  // namespace sffn

size_t sffn_mm_workspace(int T, int N, int K);
hipError_t sffn_launch_mm(const sffn::MmArgs& a, int ot, hipStream_t st);
