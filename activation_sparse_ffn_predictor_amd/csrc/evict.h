// Arguments of the eviction kernels (evict.hip).
#pragma once
#include "attn.h"

namespace sffn {

struct EvictArgs {
  Kv kv;
  const int* len;           // cached tokens [S]; plen: the sequences' tokens
  const int* plen;
  const int* table;
  const float* mass;        // mass, pos and their outputs (which may be themselves) [S, hkv, W]
  const int* pos;
  float* mass_out;
  int* pos_out;
  int* len_out;             // may be len
  int* src;                 // [S, hkv, keep]: the slot that each kept token stood in
  int* line;                // workspace [S, hkv, keep]
  int S, cols, ldt, W, keep, sinks, recent;
};

}  // namespace sffn

hipError_t sffn_launch_evict(const sffn::EvictArgs& a, int kvt, hipStream_t st);
