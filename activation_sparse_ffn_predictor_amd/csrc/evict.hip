// Eviction: of each sequence and K/V head the `keep` cached tokens that come first in this order stay:
//   those among the sequence's first `sinks` tokens or its last `recent` ones (by their positions), then by the attention weight
//   they have accumulated; ties: the lowest slot.
// What stays in a slot at or behind `keep` moves, in order, into the slots below it that are given up, in order: nothing that
// may stay where it is is moved, no row is both read and written, so all moves run at once.
//
// Selection: a token's place in the order is a 32-bit key; the key of the last one that stays is found digit by digit (11, 11 and
// 10 bits) with counts in LDS. Up to 8192 slots one workgroup does all of it with the keys in registers; more slots are spread
// over workgroups, a kernel a digit, since one workgroup's passes are bound by its instructions (6 x 8 heads of 40001 slots in
// 48 workgroups: 69 us; by kernels of a digit 10.3 + 6.2 + 6.2, what moves 11.4). Each of them is a chain of dependent loads and
// barriers rather than bytes. The moves are bound by memory: the moved rows in and out (115 MB with rows of 128 bytes: 20 to 27
// us). 4 x 8 heads of 1100 slots: 9.1 to 10.7 and 2.1 to 4.1 us.
#include "evict.h"

using namespace sffn;

namespace {

constexpr int NT = 1024, BINS = 2048;
constexpr int REGS = 8;                            // keys that a thread keeps in registers

// Order of a slot's token: 0 holds none, 1 no weight (what is negative or NaN counts as none), then by weight, protected last
struct Keys {
  const float* mass;
  const int* pos;
  const int* trow;
  int psh, n_pages, sinks, late;
  __device__ __forceinline__ uint32_t operator()(int j) const {
    const float m = mass[j];
    const int p = pos[j], pid = trow[j >> psh];    // (no branches, so that the loads of several slots are under way at once)
    const uint32_t held = ((p < sinks) | (p >= late)) ? 0xFFFFFFFFu : 1u + (m > 0.f ? __float_as_uint(m) : 0u);
    return (unsigned)pid < (unsigned)n_pages ? held : 0u;
  }
};

// inclusive sum over the wave's lanes (row shifts and broadcasts of DPP: no LDS crossbar)
template <int CTRL, int ROWS>
__device__ __forceinline__ int shift_add(int v) {
  return v + __builtin_amdgcn_update_dpp(0, v, CTRL, ROWS, 0xF, true);
}
__device__ __forceinline__ int row_scan(int v) {
  v = shift_add<0x111, 0xF>(v);
  v = shift_add<0x112, 0xF>(v);
  v = shift_add<0x114, 0xF>(v);
  return shift_add<0x118, 0xF>(v);
}
__device__ __forceinline__ int wave_scan(int v) {
  v = row_scan(v);
  v = shift_add<0x142, 0xA>(v);
  return shift_add<0x143, 0xC>(v);
}
// a wave's number before it among the workgroup's (tmp: one a wave, written and synchronised), and all of them together
__device__ __forceinline__ int before_wave(const int* tmp, int& total) {
  const int l = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), c = row_scan(tmp[l & 15]);
  total = __builtin_amdgcn_readlane(c, 15);
  return w ? __builtin_amdgcn_readlane(c, w - 1) : 0;
}

// Counts of one digit of the keys (bits 31 .. 21, 20 .. 10, 9 .. 0) among those that share the cut's digits above it. Protected
// tokens, and those without weight, would all count in one place: those are counted by the wave. In every lane of the wave.
struct Digit {
  int low, up, mask;
  uint32_t over;
  __device__ __forceinline__ Digit(int d, uint32_t cut) : low(d == 0 ? 21 : d == 1 ? 10 : 0), up(low + (d == 2 ? 10 : 11)), mask(d == 2 ? 1023 : 2047), over(d ? cut >> up : 0) {}
  __device__ __forceinline__ void count(int* hist, uint32_t x, bool in, int& tops, int& ones) const {
    const bool top = in && x == 0xFFFFFFFFu, mine = in && !top && (low == 21 || x >> up == over);
    tops += __popcll(__ballot(top));
    ones += __popcll(__ballot(mine && x == 1u));
    if (mine && x != 1u) atomicAdd(&hist[(x >> low) & mask], 1);
  }
  __device__ __forceinline__ int of_ones() const { return low ? 0 : 1; }
};
// The digit of the last key that stays, and how many of its keys do, where `need` of the counted ones stay: thread t has the
// counts n1 and n0 of the digits 2047 - 2 t and the one below it. found: of LDS; synchronised afterwards.
__device__ __forceinline__ void find_digit(int n1, int n0, int need, int* tmp, int* found) {
  int total;
  const int b1 = BINS - 1 - 2 * threadIdx.x, inc = wave_scan(n1 + n0);
  if ((threadIdx.x & 63) == 63) tmp[threadIdx.x >> 6] = inc;
  __syncthreads();
  const int above = before_wave(tmp, total) + inc - n1 - n0;
  if (above < need && need <= above + n1) { found[0] = b1; found[1] = need - above; }
  else if (above + n1 < need && need <= above + n1 + n0) { found[0] = b1 - 1; found[1] = need - above - n1; }
  __syncthreads();
}
// A workgroup's slots j0, j0 + 64, ... of this lane, `steps` of them, below `end`; wave w owns (w * steps .. (w + 1) * steps - 1) * 64, so
// that ranks in slot order need one prefix over the waves. Keys are in registers or, where a lane has more than REGS, read again (WS).
template <bool WS>
struct Slots {
  int j0, steps, end;
  const uint32_t* kept;
  uint32_t k[REGS];
  __device__ __forceinline__ void read(int i0) {
#pragma unroll
    for (int i = 0; i < REGS; ++i) k[i] = kept[max(0, min(j0 + (i0 + i) * 64, end - 1))];
  }
  template <class F>
  __device__ __forceinline__ void each(F f) {      // f(slot, key, does it exist) in every lane of the wave
    for (int i0 = 0; i0 < steps; i0 += REGS) {
      if (WS && steps > REGS) read(i0);
#pragma unroll
      for (int i = 0; i < REGS; ++i) {
        const int j = j0 + (i0 + i) * 64;
        if (i0 + i < steps) f(j, k[i], j < end);
      }
    }
  }
};
// Keys over `cut` stay, and of those equal to it the first `ties` in slot order, `rank` of which stand before this workgroup's. Writes
// the slots below `keep` that are given up to to[holes ...], those at or behind it that stay to from[movers ...], in order, and the
// others' src (given-up ones: -1, until the move). tmp: three of an int a wave.
template <bool WS>
__device__ __forceinline__ void emit(Slots<WS>& sl, const EvictArgs& a, long sh, uint32_t cut, int ties, int rank, int movers, int holes,
                                     int (*tmp)[NT / 64], int* moves) {
  const int l = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), keep = a.keep;
  const uint64_t below = l ? ~0ull >> (64 - l) : 0ull;
  int eq_lo = 0, eq_hi = 0, gt_lo = 0, gt_hi = 0, lows = 0, total;
  sl.each([&](int j, uint32_t x, bool in) {
    const uint64_t lo = __ballot(in && j < keep), e = __ballot(in && x == cut), g = __ballot(in && x > cut);
    lows += __popcll(lo);
    eq_lo += __popcll(e & lo);
    eq_hi += __popcll(e & ~lo);
    gt_lo += __popcll(g & lo);
    gt_hi += __popcll(g & ~lo);
  });
  if (l == 0) tmp[0][w] = eq_lo + eq_hi;
  __syncthreads();
  rank += before_wave(tmp[0], total);              // of the wave's first key equal to `cut`
  const int left = max(0, ties - rank), stay_lo = min(eq_lo, left), stay_hi = min(eq_hi, left - stay_lo);
  if (l == 0) {
    tmp[1][w] = gt_hi + stay_hi;                   // the wave's movers and holes
    tmp[2][w] = lows - gt_lo - stay_lo;
  }
  __syncthreads();
  int h = holes + before_wave(tmp[2], total), m = movers + before_wave(tmp[1], total);
  if (moves && threadIdx.x == 0) *moves = total;   // (as many move as there are holes)
  int *src = a.src + sh * keep, *from = a.from + sh * keep, *to = a.to + sh * keep;
  sl.each([&](int j, uint32_t x, bool in) {
    const uint64_t e = __ballot(in && x == cut);
    const bool stay = in && (x > cut || (x == cut && rank + __popcll(e & below) < ties));
    rank += __popcll(e);
    const uint64_t mv = __ballot(stay && j >= keep), hv = __ballot(in && !stay && j < keep);
    if (stay && j >= keep) from[m + __popcll(mv & below)] = j;
    if (in && j < keep) {
      src[j] = stay ? j : -1;
      if (!stay) to[h + __popcll(hv & below)] = j;
    }
    m += __popcll(mv);
    h += __popcll(hv);
  });
}

__device__ __forceinline__ int slots_of(const EvictArgs& a, int s) { return min(max(a.len[s], 0), min(a.cols << a.kv.psh, a.W)); }
__device__ __forceinline__ Keys keys_of(const EvictArgs& a, int s, long sh) {
  return {a.mass + sh * a.W, a.pos + sh * a.W, a.table + (long)s * a.ldt, a.kv.psh, a.kv.n_pages, a.sinks,
          a.recent ? (int)max((long)a.plen[s] - a.recent, -2147483648l) : 2147483647};
}
__device__ __forceinline__ void keep_all(const EvictArgs& a, long sh, int first, int step) {
  for (int j = first; j < a.keep; j += step) a.src[sh * a.keep + j] = j;
  if (first == 0) a.moves[sh] = 0;
}

// up to REGS * NT slots: one workgroup
__global__ __launch_bounds__(NT) void k_select(EvictArgs a) {
  __shared__ int hist[BINS];
  __shared__ int tmp[3][NT / 64];
  __shared__ int prot, found[3][2];
  const int hk = blockIdx.x, s = blockIdx.y, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), l = threadIdx.x & 63;
  const long sh = (long)s * a.kv.hkv + hk;
  const int n = slots_of(a, s);
  if (n <= a.keep) return keep_all(a, sh, threadIdx.x, NT);
  const Keys key = keys_of(a, s, sh);
  Slots<false> sl;
  sl.steps = (n + NT - 1) / NT;
  sl.j0 = w * sl.steps * 64 + l;
  sl.end = n;
#pragma unroll
  for (int i = 0; i < REGS; ++i)
    if (i < sl.steps) sl.k[i] = key(min(sl.j0 + i * 64, n - 1));
  hist[threadIdx.x] = hist[threadIdx.x + NT] = 0;
  if (threadIdx.x == 0) prot = 0;
  __syncthreads();
  uint32_t cut = 0;                                // the last key that stays, and how many of those do
  int ties = a.keep;
#pragma unroll 1
  for (int d = 0; d < 3; ++d) {
    const Digit g(d, cut);
    int tops = 0, ones = 0;
    sl.each([&](int, uint32_t x, bool in) { g.count(hist, x, in, tops, ones); });
    if (l == 0 && ones) atomicAdd(&hist[g.of_ones()], ones);
    if (l == 0 && tops && d == 0) atomicAdd(&prot, tops);
    __syncthreads();
    if (d == 0) {
      if (prot >= a.keep) {
        cut = 0xFFFFFFFFu;
        break;
      }
      ties -= prot;
    }
    const int b1 = BINS - 1 - 2 * threadIdx.x, n1 = hist[b1], n0 = hist[b1 - 1];
    hist[b1] = hist[b1 - 1] = 0;
    find_digit(n1, n0, ties, tmp[d], found[d]);
    cut |= (uint32_t)found[d][0] << g.low;
    ties = found[d][1];
  }
  emit<false>(sl, a, sh, cut, ties, 0, 0, 0, tmp, a.moves + sh);
}

// More slots: chunks of them a workgroup each, which never reach over `keep`. Three kernels count a digit each and hand the counts
// on; each begins with the sum of the former's over the chunks.
struct Chunk {
  int c, n, begin, end;
  long sh;
  __device__ __forceinline__ Chunk(const EvictArgs& a, int s) {
    c = blockIdx.x % a.chunks;
    sh = (long)s * a.kv.hkv + blockIdx.x / a.chunks;
    n = slots_of(a, s);
    const long b = c < a.chunks_lo ? (long)c * a.chunk : a.keep + (long)(c - a.chunks_lo) * a.chunk;
    begin = (int)min(b, (long)n);
    end = (int)min(b + a.chunk, (long)(c < a.chunks_lo ? a.keep : n));
    end = max(end, begin);
  }
};
// f(chunk, the thread's two counts (digits b1 - 1 and b1)) for every chunk; eight chunks' are read at once
template <class F>
__device__ __forceinline__ void each_chunk(const int* counts, int chunks, int b1, F f) {
  for (int c0 = 0; c0 < chunks; c0 += 8) {
    int2 v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = *reinterpret_cast<const int2*>(counts + (long)min(c0 + i, chunks - 1) * BINS + b1 - 1);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c0 + i < chunks) f(c0 + i, v[i]);
  }
}
template <int D>
__global__ __launch_bounds__(NT) void k_digit(EvictArgs a) {
  __shared__ int hist[BINS];
  __shared__ int tmp[NT / 64], prot, found[2], more;
  const int s = blockIdx.y, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), l = threadIdx.x & 63;
  const Chunk ch(a, s);
  const long sh = ch.sh, at = sh * a.chunks + ch.c;
  if (ch.n <= a.keep) {
    if (D == 0) keep_all(a, sh, ch.c * NT + threadIdx.x, a.chunks * NT);
    return;
  }
  EvictFound* state = a.found + sh * 3;
  Slots<true> sl;
  sl.steps = (ch.end - ch.begin + NT - 1) / NT;
  sl.j0 = ch.begin + w * sl.steps * 64 + l;
  sl.end = ch.end;
  sl.kept = a.keys + sh * a.W;
  if (D > 0) sl.read(0);                           // (ahead of what the digit's count waits for)
  uint32_t cut = 0;
  int need = a.keep;
  hist[threadIdx.x] = hist[threadIdx.x + NT] = 0;
  if (threadIdx.x == 0) prot = more = 0;
  __syncthreads();
  const int b1 = BINS - 1 - 2 * threadIdx.x;
  if constexpr (D > 0) {
    // the digit before this one, from the counts of all chunks; and how many of this chunk's keys lie over it
    const int* before = a.hist + ((long)(D - 1) * a.kv.hkv * a.S + sh) * a.chunks * BINS;
    int n1 = 0, n0 = 0;
    each_chunk(before, a.chunks, b1, [&](int, int2 v) { n0 += v.x, n1 += v.y; });
    if (D == 1) {
      if (l < 64) {
        int p = 0;
        for (int c = l; c < a.chunks; c += 64) p += a.tops[sh * a.chunks + c];
        need -= __builtin_amdgcn_readlane(wave_scan(p), 63);
      }
    } else {
      cut = state[D - 2].cut;
      need = state[D - 2].ties;
    }
    const bool full = D == 1 ? need <= 0 : cut == 0xFFFFFFFFu;       // protected tokens alone take every place
    if (full) {
      cut = 0xFFFFFFFFu;
      need = a.keep;
    } else {
      find_digit(n1, n0, need, tmp, found);
      cut |= (uint32_t)found[0] << Digit(D - 1, 0).low;
      need = found[1];
      const int2 v = *reinterpret_cast<const int2*>(before + (long)ch.c * BINS + b1 - 1);
      const int mine = (b1 > found[0] ? v.y : 0) + (b1 - 1 > found[0] ? v.x : 0), sum = wave_scan(mine);
      if (l == 63 && sum) atomicAdd(&more, sum);
      __syncthreads();
    }
    if (threadIdx.x == 0) {
      a.over[at] = full ? 0 : (D == 1 ? a.tops[at] : a.over[at]) + more;
      if (ch.c == 0) state[D - 1] = {cut, need};
    }
    if (full) return;
  }
  const Digit g(D, cut);
  int tops = 0, ones = 0;
  if constexpr (D == 0) {
    const Keys key = keys_of(a, s, sh);
    uint32_t* kept = a.keys + sh * a.W;
    for (int i0 = 0; i0 < sl.steps; i0 += REGS) {
#pragma unroll
      for (int i = 0; i < REGS; ++i) sl.k[i] = key(min(sl.j0 + (i0 + i) * 64, ch.end - 1));
#pragma unroll
      for (int i = 0; i < REGS; ++i) {
        const int j = sl.j0 + (i0 + i) * 64;
        const bool in = i0 + i < sl.steps && j < ch.end;
        if (in) kept[j] = sl.k[i];
        if (i0 + i < sl.steps) g.count(hist, sl.k[i], in, tops, ones);
      }
    }
  } else {
    sl.each([&](int, uint32_t x, bool in) { g.count(hist, x, in, tops, ones); });
  }
  if (l == 0 && ones) atomicAdd(&hist[g.of_ones()], ones);
  if (D == 0 && l == 0 && tops) atomicAdd(&prot, tops);
  __syncthreads();
  int* out = a.hist + ((long)D * a.kv.hkv * a.S * a.chunks + at) * BINS;
  *reinterpret_cast<int2*>(out + b1 - 1) = make_int2(hist[b1 - 1], hist[b1]);
  if (D == 0 && threadIdx.x == 0) a.tops[at] = prot;
}
__global__ __launch_bounds__(NT) void k_emit(EvictArgs a) {
  __shared__ int tmp[3][NT / 64], found[2], over[EVICT_CHUNKS], eq[EVICT_CHUNKS], start[3];
  const int s = blockIdx.y, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), l = threadIdx.x & 63;
  const Chunk ch(a, s);
  const long sh = ch.sh;
  if (ch.n <= a.keep) return;
  Slots<true> sl;
  sl.steps = (ch.end - ch.begin + NT - 1) / NT;
  sl.j0 = ch.begin + w * sl.steps * 64 + l;
  sl.end = ch.end;
  sl.kept = a.keys + sh * a.W;
  sl.read(0);
  uint32_t cut = a.found[sh * 3 + 1].cut;
  int ties = a.found[sh * 3 + 1].ties;
  const bool full = cut == 0xFFFFFFFFu;            // then the protected ones are the ties
  const int* before = a.hist + ((long)2 * a.kv.hkv * a.S + sh) * a.chunks * BINS;
  const int b1 = BINS - 1 - 2 * threadIdx.x;
  for (int c = threadIdx.x; c < a.chunks; c += NT) {
    over[c] = full ? 0 : a.over[sh * a.chunks + c];
    eq[c] = full ? a.tops[sh * a.chunks + c] : 0;
  }
  __syncthreads();
  if (!full) {
    int n1 = 0, n0 = 0;
    each_chunk(before, a.chunks, b1, [&](int, int2 v) { n0 += v.x, n1 += v.y; });
    find_digit(n1, n0, ties, tmp[0], found);
    cut |= (uint32_t)found[0];
    ties = found[1];
    each_chunk(before, a.chunks, b1, [&](int c, int2 v) {
      const int sum = wave_scan((b1 > found[0] ? v.y : 0) + (b1 - 1 > found[0] ? v.x : 0));
      if (l == 63 && sum) atomicAdd(&over[c], sum);
      if (b1 == found[0]) eq[c] = v.y;
      if (b1 - 1 == found[0]) eq[c] = v.x;
    });
    __syncthreads();
  }
  // where this chunk's ties, movers and holes begin
  if (threadIdx.x == 0) {
    int rank = 0, m = 0, h = 0;
    for (int c = 0; c < a.chunks; ++c) {
      if (c == ch.c) start[0] = rank, start[1] = m, start[2] = h;
      const int stay = over[c] + min(eq[c], max(0, ties - rank));
      rank += eq[c];
      if (c < a.chunks_lo) h += min(a.chunk, a.keep - c * a.chunk) - stay;
      else m += stay;
    }
    if (ch.c == 0) a.moves[sh] = m;
  }
  __syncthreads();
  if (ch.end > ch.begin) emit<true>(sl, a, sh, cut, ties, start[0], start[1], start[2], tmp, nullptr);
}

// The moves, `rest` workgroups a sequence and head: LPR lanes a row, 16 bytes each of K and V; its scales, weight and position. ROWS rows
// at a time, since each waits for a chain of four loads (6 x 8 heads, 115 MB: one row 23 us, four 20), one where that leaves places
// free (4 x 8 heads, up to 76 rows each: one 3.0 us, four 4.0).
// Behind them workgroups for the weights and positions of tokens that stay where they are, a thread a slot, and the lengths.
template <int LPR, int ROWS>
__global__ __launch_bounds__(256) void k_move(EvictArgs a, int eb, int rest) {
  const int hk = blockIdx.x % a.kv.hkv, s = blockIdx.x / a.kv.hkv % a.S, g = blockIdx.x / a.kv.hkv / a.S;
  const long sh = (long)s * a.kv.hkv + hk;
  if (g >= rest) {
    const int j = (g - rest) * 256 + threadIdx.x, old = a.len[s], n = slots_of(a, s);
    // (lengths may be updated in place while other workgroups read them: n, cut off at keep, is the same before and after)
    if (j == 0 && hk == 0) a.len_out[s] = n > a.keep ? a.keep : old;
    if (j >= min(n, a.keep) || a.src[sh * a.keep + j] != j) return;
    if (a.mass_out != a.mass) a.mass_out[sh * a.W + j] = a.mass[sh * a.W + j];
    if (a.pos_out != a.pos) a.pos_out[sh * a.W + j] = a.pos[sh * a.W + j];
    return;
  }
  const int lane = threadIdx.x % LPR, first = g * (ROWS * (256 / LPR)), n = a.moves[sh];
  if (first >= n) return;
  const int* trow = a.table + (long)s * a.ldt;
  const int mask = (1 << a.kv.psh) - 1, row = a.kv.d * eb;
  int f[ROWS], t[ROWS], pf[ROWS], pt[ROWS];
  bool in[ROWS];
#pragma unroll
  for (int r = 0; r < ROWS; ++r) {
    const int i = first + r * (256 / LPR) + threadIdx.x / LPR;
    in[r] = i < n;
    f[r] = a.from[sh * a.keep + min(i, n - 1)];
    t[r] = a.to[sh * a.keep + min(i, n - 1)];
  }
#pragma unroll
  for (int r = 0; r < ROWS; ++r) {
    pf[r] = trow[f[r] >> a.kv.psh];
    pt[r] = trow[t[r] >> a.kv.psh];
  }
  long rf[ROWS], rt[ROWS];
  bool held[ROWS];
  uint4 k[ROWS], v[ROWS];
#pragma unroll
  for (int r = 0; r < ROWS; ++r) {
    held[r] = in[r] && (unsigned)pf[r] < (unsigned)a.kv.n_pages && (unsigned)pt[r] < (unsigned)a.kv.n_pages;
    rf[r] = (((long)(held[r] ? pf[r] : 0) * a.kv.hkv + hk) << a.kv.psh) + (f[r] & mask);
    rt[r] = (((long)(held[r] ? pt[r] : 0) * a.kv.hkv + hk) << a.kv.psh) + (t[r] & mask);
    k[r] = v[r] = make_uint4(0, 0, 0, 0);
    if (held[r] && lane * 16 < row) {
      k[r] = *reinterpret_cast<const uint4*>(a.kv.k + rf[r] * row + lane * 16);
      v[r] = *reinterpret_cast<const uint4*>(a.kv.v + rf[r] * row + lane * 16);
    }
  }
  // lane r takes what row r has besides
  int mf = f[0], mt = t[0];
  long mrf = rf[0], mrt = rt[0];
  bool mine = in[0], mheld = held[0];
#pragma unroll
  for (int r = 1; r < ROWS; ++r)
    if (lane == r) mf = f[r], mt = t[r], mrf = rf[r], mrt = rt[r], mine = in[r], mheld = held[r];
  if (lane < ROWS && mine) {
    const float mass = a.mass[sh * a.W + mf];
    const int pos = a.pos[sh * a.W + mf];
    a.src[sh * a.keep + mt] = mf;
    if (eb == 1 && mheld) {
      const float ks = a.kv.ks[mrf], vs = a.kv.vs[mrf];
      a.kv.ks[mrt] = ks;
      a.kv.vs[mrt] = vs;
    }
    a.mass_out[sh * a.W + mt] = mass;
    a.pos_out[sh * a.W + mt] = pos;
  }
#pragma unroll
  for (int r = 0; r < ROWS; ++r)
    if (held[r] && lane * 16 < row) {
      *reinterpret_cast<uint4*>(a.kv.k + rt[r] * row + lane * 16) = k[r];
      *reinterpret_cast<uint4*>(a.kv.v + rt[r] * row + lane * 16) = v[r];
    }
}

}  // namespace

hipError_t sffn_launch_evict(const EvictArgs& a, int kvt, hipStream_t st) {
  const int most = a.W < a.cols << a.kv.psh ? a.W : a.cols << a.kv.psh;
  if (a.chunks == 0) hipLaunchKernelGGL(k_select, dim3(a.kv.hkv, a.S), dim3(NT), 0, st, a);
  else {
    const dim3 grid(a.chunks * a.kv.hkv, a.S);
    hipLaunchKernelGGL(k_digit<0>, grid, dim3(NT), 0, st, a);
    hipLaunchKernelGGL(k_digit<1>, grid, dim3(NT), 0, st, a);
    hipLaunchKernelGGL(k_digit<2>, grid, dim3(NT), 0, st, a);
    hipLaunchKernelGGL(k_emit, grid, dim3(NT), 0, st, a);
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int eb = kvt == T_I8 || kvt == T_E4M3 ? 1 : 2, row = a.kv.d * eb;
  // at most as many rows move as there are slots on either side of `keep`
  const int lpr = row <= 64 ? 4 : row <= 128 ? 8 : row <= 256 ? 16 : 32, rows = most - a.keep < a.keep ? most - a.keep : a.keep;
  const int slots = 256 / lpr, each = (long)rows * a.kv.hkv * a.S > 4096l * slots ? 4 * slots : slots,
            rest = rows > 0 ? (rows + each - 1) / each : 0, groups = rest + (a.keep + 255) / 256;
  const dim3 moves((unsigned)groups * a.kv.hkv * a.S);
#define GO(LPR)                                                                                 \
  do {                                                                                          \
    if (each > slots) hipLaunchKernelGGL((k_move<LPR, 4>), moves, dim3(256), 0, st, a, eb, rest); \
    else hipLaunchKernelGGL((k_move<LPR, 1>), moves, dim3(256), 0, st, a, eb, rest);            \
  } while (0)
  if (lpr == 4) GO(4);
  else if (lpr == 8) GO(8);
  else if (lpr == 16) GO(16);
  else GO(32);
#undef GO
  return hipGetLastError();
}
