// Eviction: of each sequence and K/V head the `keep` cached tokens that come first in this order stay:
//   those among the sequence's first `sinks` tokens or its last `recent` ones (by their positions), then by the attention weight
//   they have accumulated; ties: the lowest slot.
// What stays in a slot at or behind `keep` moves, in order, into the slots below it that are given up, in order: nothing that
// may stay where it is is moved, no row is both read and written, so all moves run at once.
//
// Selection: one workgroup a sequence and head. A token's place in the order is a 32-bit key; the key of the last one that stays
// is found digit by digit (11, 11 and 10 bits) with counts in LDS. Bound by memory: weights and positions once, then the moved
// rows in and out.
#include "evict.h"

using namespace sffn;

namespace {

constexpr int NT = 1024, BINS = 2048;

// Order of a slot's token: 0 holds none, 1 no weight (what is negative or NaN counts as none), then by weight, protected last
struct Keys {
  const float* mass;
  const int* pos;
  const int* trow;
  int psh, n_pages, cols, sinks, late;
  __device__ __forceinline__ uint32_t operator()(int j) const {
    const float m = mass[j];
    const int p = pos[j], pid = trow[j >> psh];
    if ((unsigned)pid >= (unsigned)n_pages) return 0;
    if (p < sinks || p >= late) return 0xFFFFFFFFu;
    return m > 0.f ? 1u + __float_as_uint(m) : 1u;
  }
};

// KPT keys a thread stay in registers (0: they are worked out again each time). Wave w owns slots w * seg .. (w + 1) * seg - 1.
template <int KPT>
__global__ __launch_bounds__(NT) void k_select(EvictArgs a) {
  __shared__ int hist[BINS];
  __shared__ int tmp[NT / 64 + 1];
  __shared__ int found[2];
  const int hk = blockIdx.x, s = blockIdx.y, w = threadIdx.x >> 6, l = threadIdx.x & 63, keep = a.keep;
  const long sh = (long)s * a.kv.hkv + hk;
  int* src = a.src + sh * keep;
  const int n = min(max(a.len[s], 0), min(a.cols << a.kv.psh, a.W));
  if (n <= keep) {
    for (int j = threadIdx.x; j < keep; j += NT) src[j] = j;
    return;
  }
  const Keys key{a.mass + sh * a.W, a.pos + sh * a.W, a.table + (long)s * a.ldt, a.kv.psh, a.kv.n_pages, a.cols, a.sinks,
                 a.recent ? (int)max((long)a.plen[s] - a.recent, -2147483648l) : 2147483647};
  const int steps = (n + NT - 1) / NT, j0 = w * steps * 64 + l;      // slots j0, j0 + 64, ... of this lane
  uint32_t k[KPT ? KPT : 1];
#pragma unroll
  for (int i = 0; i < KPT; ++i) k[i] = i < steps && j0 + i * 64 < n ? key(j0 + i * 64) : 0;
  auto each = [&](auto f) {                        // f(slot, key, does it exist) in every lane of the wave
    if constexpr (KPT > 0) {
#pragma unroll
      for (int i = 0; i < KPT; ++i)
        if (i < steps) f(j0 + i * 64, k[i], j0 + i * 64 < n);
    } else {
      for (int i = 0; i < steps; ++i) f(j0 + i * 64, j0 + i * 64 < n ? key(j0 + i * 64) : 0u, j0 + i * 64 < n);
    }
  };
  int total;
  // protected ones, which would all count in one place
  int c = 0;
  each([&](int, uint32_t x, bool in) { c += __popcll(__ballot(in && x == 0xFFFFFFFFu)); });
  block_exclusive_scan<NT>(l == 0 ? c : 0, tmp, total);
  __syncthreads();
  uint32_t cut = 0xFFFFFFFFu;                      // the last key that stays, and how many of those do
  int ties = keep;
  if (total < keep) {
    ties = keep - total;
    cut = 0;
    // digits: bits 31 .. 21, 20 .. 10, 9 .. 0
#pragma unroll 1
    for (int d = 0; d < 3; ++d) {
      const int low = d == 0 ? 21 : d == 1 ? 10 : 0;
      hist[threadIdx.x] = hist[threadIdx.x + NT] = 0;
      __syncthreads();
      int ones = 0;                                // tokens without weight, which would all count in one place too
      each([&](int, uint32_t x, bool in) {
        const bool mine = in && x != 0xFFFFFFFFu && (d == 0 || (x >> (low + (d == 1 ? 11 : 10))) == (cut >> (low + (d == 1 ? 11 : 10))));
        ones += __popcll(__ballot(mine && x == 1u));
        if (mine && x != 1u) atomicAdd(&hist[(x >> low) & (d == 2 ? 1023 : 2047)], 1);
      });
      if (l == 0 && ones) atomicAdd(&hist[(1u >> low) & 2047], ones);
      __syncthreads();
      // from the largest digit down: thread t has 2047 - 2 t and the one below it
      const int b1 = BINS - 1 - 2 * threadIdx.x, n1 = hist[b1], n0 = hist[b1 - 1];
      const int above = block_exclusive_scan<NT>(n1 + n0, tmp, total);
      if (above < ties && ties <= above + n1) { found[0] = b1; found[1] = ties - above; }
      else if (above + n1 < ties && ties <= above + n1 + n0) { found[0] = b1 - 1; found[1] = ties - above - n1; }
      __syncthreads();
      cut |= (uint32_t)found[0] << low;
      ties = found[1];
      __syncthreads();
    }
  }
  // keys over `cut` stay, and of those equal to it the first `ties`
  const uint64_t below = l ? ~0ull >> (64 - l) : 0ull;
  c = 0;
  each([&](int, uint32_t x, bool in) { c += __popcll(__ballot(in && x == cut)); });
  int run = __shfl(block_exclusive_scan<NT>(l == 0 ? c : 0, tmp, total), 0, WAVE);
  __syncthreads();
  const int tie0 = run;
  int movers = 0, holes = 0;
  each([&](int j, uint32_t x, bool in) {
    const uint64_t eq = __ballot(in && x == cut);
    const bool stay = in && (x > cut || (x == cut && run + __popcll(eq & below) < ties));
    run += __popcll(eq);
    movers += __popcll(__ballot(stay && j >= keep));
    holes += __popcll(__ballot(in && !stay && j < keep));
  });
  const int m0 = __shfl(block_exclusive_scan<NT>(l == 0 ? movers : 0, tmp, total), 0, WAVE);
  __syncthreads();
  const int h0 = __shfl(block_exclusive_scan<NT>(l == 0 ? holes : 0, tmp, total), 0, WAVE);
  int* line = a.line + sh * keep;                  // the movers' slots in order
  run = tie0;
  int m = m0;
  each([&](int j, uint32_t x, bool in) {
    const uint64_t eq = __ballot(in && x == cut);
    const bool stay = in && (x > cut || (x == cut && run + __popcll(eq & below) < ties));
    run += __popcll(eq);
    const uint64_t mv = __ballot(stay && j >= keep);
    if (stay && j >= keep) line[m + __popcll(mv & below)] = j;
    m += __popcll(mv);
  });
  __syncthreads();                                 // (orders the workgroup's own writes of the list before its reads)
  run = tie0;
  int h = h0;
  each([&](int j, uint32_t x, bool in) {
    const uint64_t eq = __ballot(in && x == cut);
    const bool stay = in && (x > cut || (x == cut && run + __popcll(eq & below) < ties));
    run += __popcll(eq);
    const bool hole = in && !stay && j < keep;
    const uint64_t hv = __ballot(hole);
    if (in && j < keep) src[j] = hole ? line[h + __popcll(hv & below)] : j;
    h += __popcll(hv);
  });
}

// The moves: LPR lanes a slot, 16 bytes each of K and V; weights, positions and scales with them.
template <int LPR>
__global__ __launch_bounds__(256) void k_move(EvictArgs a, int eb, int groups) {
  const int hk = blockIdx.x % a.kv.hkv, g = blockIdx.x / a.kv.hkv % groups, s = blockIdx.x / a.kv.hkv / groups;
  const int lane = threadIdx.x % LPR, j = g * (256 / LPR) + threadIdx.x / LPR;
  const long sh = (long)s * a.kv.hkv + hk;
  const int n = min(max(a.len[s], 0), min(a.cols << a.kv.psh, a.W));
  // (the lengths may be updated in place while other workgroups read them: n, cut off at keep, is the same before and after)
  if (g == 0 && hk == 0 && threadIdx.x == 0) {
    const int old = a.len[s];
    a.len_out[s] = n > a.keep ? a.keep : old;
  }
  if (j >= min(n, a.keep)) return;
  const int from = a.src[sh * a.keep + j];
  if (lane == 0) {
    if (from != j || a.mass_out != a.mass) a.mass_out[sh * a.W + j] = a.mass[sh * a.W + from];
    if (from != j || a.pos_out != a.pos) a.pos_out[sh * a.W + j] = a.pos[sh * a.W + from];
  }
  if (from == j) return;
  const int* trow = a.table + (long)s * a.ldt;
  const int mask = (1 << a.kv.psh) - 1, pf = trow[from >> a.kv.psh], pt = trow[j >> a.kv.psh];
  if ((unsigned)pf >= (unsigned)a.kv.n_pages || (unsigned)pt >= (unsigned)a.kv.n_pages) return;
  const long rf = (((long)pf * a.kv.hkv + hk) << a.kv.psh) + (from & mask), rt = (((long)pt * a.kv.hkv + hk) << a.kv.psh) + (j & mask);
  const int row = a.kv.d * eb;
  if (lane * 16 < row) {
    const uint4 k = *reinterpret_cast<const uint4*>(a.kv.k + rf * row + lane * 16);
    const uint4 v = *reinterpret_cast<const uint4*>(a.kv.v + rf * row + lane * 16);
    *reinterpret_cast<uint4*>(a.kv.k + rt * row + lane * 16) = k;
    *reinterpret_cast<uint4*>(a.kv.v + rt * row + lane * 16) = v;
  }
  if (eb == 1 && lane == 0) {
    a.kv.ks[rt] = a.kv.ks[rf];
    a.kv.vs[rt] = a.kv.vs[rf];
  }
}

}  // namespace

hipError_t sffn_launch_evict(const EvictArgs& a, int kvt, hipStream_t st) {
  const dim3 grid(a.kv.hkv, a.S);
  const int most = a.W < a.cols << a.kv.psh ? a.W : a.cols << a.kv.psh;
  if (most <= 8 * NT) hipLaunchKernelGGL(k_select<8>, grid, dim3(NT), 0, st, a);
  else if (most <= 64 * NT) hipLaunchKernelGGL(k_select<64>, grid, dim3(NT), 0, st, a);
  else hipLaunchKernelGGL(k_select<0>, grid, dim3(NT), 0, st, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int eb = kvt == T_I8 || kvt == T_E4M3 ? 1 : 2, row = a.kv.d * eb;
  const int lpr = row <= 64 ? 4 : row <= 128 ? 8 : row <= 256 ? 16 : 32, groups = (a.keep + 256 / lpr - 1) / (256 / lpr);
  const dim3 moves((unsigned)groups * a.kv.hkv * a.S);
  if (lpr == 4) hipLaunchKernelGGL(k_move<4>, moves, dim3(256), 0, st, a, eb, groups);
  else if (lpr == 8) hipLaunchKernelGGL(k_move<8>, moves, dim3(256), 0, st, a, eb, groups);
  else if (lpr == 16) hipLaunchKernelGGL(k_move<16>, moves, dim3(256), 0, st, a, eb, groups);
  else hipLaunchKernelGGL(k_move<32>, moves, dim3(256), 0, st, a, eb, groups);
  return hipGetLastError();
}
