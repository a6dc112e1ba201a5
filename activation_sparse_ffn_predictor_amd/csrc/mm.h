// Arguments of the block-scaled product's kernels (mm.hip).
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

}  // namespace sffn

size_t sffn_mm_workspace(int T, int N, int K);
hipError_t sffn_launch_mm(const sffn::MmArgs& a, int ot, hipStream_t st);
