// Arguments and sizes of the attention-mass kernels (mass.hip), which the host side decides on.
#pragma once
#include "attn.h"

namespace sffn {

// mass, out, pos [S, hkv, W]; rows of one K/V head: r = i * G + g for new token i and query head hk * G + g.
struct MassArgs {
  const char* q;
  const float* lse;         // [T, hq]
  const float* mass;
  float* out;               // may be mass
  int* pos;
  const int* plen;          // tokens of the sequences [S]
  Kv kv;
  Seqs sq;
  int hq, G, max_q, window, sinks, W;
  long ldq;
  float c;                  // softmax scale * log2(e)
  int rs, wp;               // shares of the rows (tile kernel); keys whose sums are shared out
  float* part;              // [S, hkv, rs, wp], used when rs > 1
};

// the few-row kernel keeps the queries in registers
__host__ __device__ constexpr bool mass_few(long rows, int d) { return rows <= (d <= 128 ? 64 : 32); }
// New tokens first .. end - 1 of a sequence's n (at positions p0, p0 + 1, ...): outside them no token sees any of the keys k0 .. k1.
// Always tokens that there are, however far p0 lies from them, so that their rows' numbers keep to 32 bits.
struct Tokens {
  int first, end;
};
__host__ __device__ __forceinline__ Tokens tokens_of_keys(int p0, int n, int k0, int k1, int window, int sinks) {
  const int a = k0 - p0;                           // (k0 < 2^30, p0 >= -2^25)
  const long b = (long)k1 + window - p0;
  return {a < 0 ? 0 : a < n ? a : n, window > 0 && k0 >= sinks ? (int)(b < 0 ? 0 : b < n ? b : n) : n};
}
// keys of a workgroup of the tile kernel
__host__ __device__ constexpr int mass_tile(int d) { return d <= 128 ? 256 : 128; }

}  // namespace sffn

hipError_t sffn_launch_mass(const sffn::MassArgs& a, int qt, int kvt, int tiles, hipStream_t st);
