// Arguments of the eviction kernels (evict.hip).
#pragma once
#include "attn.h"

namespace sffn {

constexpr int EVICT_ONE = 8192;      // slots that one workgroup takes
constexpr int EVICT_CHUNKS = 64;     // workgroups of more, at most (and one for the end on either side of `keep`)
constexpr int EVICT_BINS = 2048;

struct EvictFound {
  uint32_t cut;
  int ties;
};
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
  int S, cols, ldt, W, keep, sinks, recent;
  // workspace: rows that move [S, hkv], the slots they leave and take [S, hkv, keep]
  int *moves, *from, *to;
  // more than EVICT_ONE slots: chunks of `chunk` slots, chunks_lo of them below `keep` (chunks = 0: one workgroup); keys [S, hkv, W],
  // counts [3, S, hkv, chunks, EVICT_BINS], protected tokens and keys over the cut's digits [S, hkv, chunks], what was found [S, hkv, 3]
  int chunks, chunks_lo, chunk;
  uint32_t* keys;
  int *hist, *tops, *over;
  EvictFound* found;
};

// Sets a's chunks and, given the workspace, its pointers; returns the workspace's bytes.
inline size_t evict_plan(EvictArgs& a, int hkv, void* ws) {
  const int most = a.W;
  a.chunks = a.chunks_lo = a.chunk = 0;
  if (most > EVICT_ONE) {
    const long each = EVICT_ONE, per = (most + (EVICT_CHUNKS - 2) * each - 1) / ((EVICT_CHUNKS - 2) * each);
    a.chunk = (int)(per * each);
    a.chunks_lo = (a.keep + a.chunk - 1) / a.chunk;
    a.chunks = a.chunks_lo + (most > a.keep ? (most - a.keep + a.chunk - 1) / a.chunk : 0);
  }
  size_t at = 0;
  const size_t sh = (size_t)a.S * hkv;
  auto take = [&](size_t n) {
    const uintptr_t p = (uintptr_t)ws + at;
    at += (n * 4 + 255) / 256 * 256;
    return p;
  };
  a.moves = (int*)take(sh);
  a.from = (int*)take(sh * a.keep);
  a.to = (int*)take(sh * a.keep);
  if (a.chunks) {
    a.keys = (uint32_t*)take(sh * a.W);
    a.hist = (int*)take(3 * sh * a.chunks * EVICT_BINS);
    a.tops = (int*)take(sh * a.chunks);
    a.over = (int*)take(sh * a.chunks);
    a.found = (EvictFound*)take(sh * 3 * 2);
  }
  return at;
}

}  // namespace sffn

hipError_t sffn_launch_evict(const sffn::EvictArgs& a, int kvt, hipStream_t st);
