// out = A B^T for e4m3 matrices with one fp32 scale for each 128 columns of a row of A and each 128 x 128 block of B:
//   out[t, n] = sum over blocks kb of sa[t, kb] sb[n / 128, kb] * (sum over k in kb of A[t, k] B[n, k])
// Rows of B are the matrix instructions' rows, tokens their columns: a lane's results belong to one token, so its factor is one
// register, and sb is the same for the whole tile. Blocks are scaled and added in fp32.
//
// A block's own sum: the 8-bit instruction (16x16x128, a block at once) brings each 8 products to the largest one's exponent (the
// sum of its factors') and drops, towards zero, what lies 2^-13 under it; the fp16 instruction on widened codes (exact) adds in fp32,
// at half the rate (599 us for 340 at 4096 x 10240 x 8192). Few tokens wait for memory, so they take the fp16 one, as do fp32 results;
// 16-bit results of many tokens take the 8-bit one, fewer than 32 bits by choice: measured at K = 1024 and 8192, the dropped bits are
// 1.8e-5 of the results (root mean squares, their mean 1e-6 or less), fp16's own rounding 2.1e-4, bf16's 1.7e-3.
#include "mm.h"

using namespace sffn;

namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
// A lane's 32 codes of a block (two 16-byte chunks), as they are or as fp16 operands of four products
template <bool EXACT>
struct Codes {
  uint4 v[EXACT ? 4 : 2];
  __device__ __forceinline__ void set(const uint4& a, const uint4& b) {
    if constexpr (EXACT) {
      const uint32_t u[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint2 p = codes4<true>(u[2 * i]), q = codes4<true>(u[2 * i + 1]);
        v[i] = make_uint4(p.x, p.y, q.x, q.y);
      }
    } else {
      v[0] = a;
      v[1] = b;
    }
  }
};
// the block's sums for 16 rows and 16 tokens
__device__ __forceinline__ f32x4 block_sum(const Codes<false>& a, const Codes<false>& b) {
  const i32x8 x = {(int)a.v[0].x, (int)a.v[0].y, (int)a.v[0].z, (int)a.v[0].w, (int)a.v[1].x, (int)a.v[1].y, (int)a.v[1].z, (int)a.v[1].w};
  const i32x8 y = {(int)b.v[0].x, (int)b.v[0].y, (int)b.v[0].z, (int)b.v[0].w, (int)b.v[1].x, (int)b.v[1].y, (int)b.v[1].z, (int)b.v[1].w};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x, y, f32x4{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 0, 0, 0);
}
__device__ __forceinline__ f32x4 block_sum(const Codes<true>& a, const Codes<true>& b) {
  f32x4 p = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < 4; ++i) p = mfma16<false>(a.v[i], b.v[i], p);
  return p;
}
template <int OT>
__device__ __forceinline__ void store4(void* p, long i, f32x4 v) {
  if constexpr (OT == T_F32) *reinterpret_cast<f32x4*>((float*)p + i) = v;
  else *reinterpret_cast<uint2*>((char*)p + 2 * i) = make_uint2(pack2<OT == T_BF16>(v[0], v[1]), pack2<OT == T_BF16>(v[2], v[3]));
}
// what lies past a span's end reads as zeros
__device__ __forceinline__ Buf buf(const Span& s) { return Buf(s.p, s.bytes); }
__device__ __forceinline__ void load_lds(const Span& s, uint32_t off, uint32_t at, char* to) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(buf(s).r, (__attribute__((address_space(3))) void*)to, 16, (int)off, (int)at, 0, 0);
}

// ------------------------------------------------------------------------------------------------ few tokens
// Up to 16 tokens: 16 rows of B a workgroup, whose NW waves take blocks of k in turn and are added up in LDS. Bound by B's bytes;
// a wave has U blocks on their way beside the one it multiplies, the next waves of a compute unit theirs: 1 x 10240 x 8192, 84 MB, on
// one card: U = 4 22.2 us, 2 21.4, 1 19.8 (4.2 TB/s with its launch), with registers for twice the waves.
template <int OT, int NW>
__global__ __launch_bounds__(NW * 64) void k_mm_few(MmArgs a) {
  __shared__ f32x4 part[NW][64];
  constexpr int U = 1;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), l = threadIdx.x & 63, g4 = l >> 4, ql = l & 15;
  const int n0 = blockIdx.x * 16, KB = (a.K + 127) >> 7;
  const Buf bb = buf(rows_of(a.b, a.ldb, n0, a.N, 16, a.K)), ba = buf(rows_of(a.a, a.lda, 0, a.T, 16, a.K)), bs(a.sa, (uint32_t)a.T * KB * 4),
      bw(a.sb + (long)(n0 >> 7) * KB, (uint32_t)KB * 4);
  const uint32_t vb = ql * (uint32_t)a.ldb + g4 * 16, va = ql * (uint32_t)a.lda + g4 * 16, vs = boff(ql < a.T, ql * (uint32_t)KB * 4);
  uint4 x[U][2], y[U][2];
  float f[U], s[U];
  // workgroups begin at different blocks: rows are often a power of two apart, and those that read the same columns of theirs wait
  // for the same memory channels (1 x 10240 x 8192 with four blocks ahead: 25 us, so 22; with one ahead 19.5 either way)
  const int turn = blockIdx.x * 5 % KB;
  auto load = [&](int u, int i) {                  // (past the end nothing is loaded)
    int kb = i + turn;
    kb = kb >= KB ? kb - KB : kb;
    const bool some = i < KB;
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const uint32_t col = kb * 128 + c * 64;
      const bool in = some & (col + g4 * 16 < (uint32_t)a.K);
      x[u][c] = bb.ld16(boff(in, vb + col));
      y[u][c] = ba.ld16(boff(in, va + col));
    }
    f[u] = bs.ldf(boff(some, vs + kb * 4));
    s[u] = bw.ldf(boff(some, kb * 4));
  };
  f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int u = 0; u < U; ++u) load(u, w + u * NW);
  for (int k0 = w; k0 < KB; k0 += NW * U) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      Codes<true> c, z;
      c.set(x[u][0], x[u][1]);
      z.set(y[u][0], y[u][1]);
      const float g = f[u] * s[u];
      load(u, k0 + (U + u) * NW);
      const f32x4 p = block_sum(c, z);
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[i] = fmaf(p[i], g, acc[i]);
    }
  }
  part[w][l] = acc;
  __syncthreads();
  if (threadIdx.x < 64) {
    const int n = n0 + 4 * g4;
    f32x4 v = part[0][l];
#pragma unroll
    for (int i = 1; i < NW; ++i) v += part[i][l];
    if (ql < a.T && n < a.N) store4<OT>(a.out, ql * a.ldo + n, v);
  }
}

// ------------------------------------------------------------------------------------------------ some tokens
// BN rows of B x BT tokens a workgroup of WN x WT waves, for calls that B's bytes or a few tiles bound: four blocks of k in LDS,
// three of them on their way (direct loads) while one is multiplied; k may be spread over workgroups, whose fp32 partial results
// a second kernel adds up in order. Swizzle as below. 37 x 15360 x 5120, 80 MB: 22 to 23 us (20.6 of them before the join, 4.1 TB/s; the operands' way through LDS and
// their widening to fp16 do not wholly hide behind the loads); 10240 rows of K = 8192: 16 tokens 22.5 us, 64 30.
template <int OT, bool EXACT, int BN, int BT, int WN, int WT>
__global__ __launch_bounds__(WN * WT * 64) void k_mm_some(MmArgs a, int ks) {
  constexpr int W = WN * WT, MI = BN / WN / 16, NI = BT / WT / 16, FC = 32;   // FC: blocks whose factors LDS holds
  constexpr int LB = BN / 8 / W, LA = BT / 8 / W, L = LB + LA;
  static_assert(LB * 8 * W == BN && LA * 8 * W == BT && BN <= 128 && W % 2 == 0, "whole direct loads, one block of 128 rows");
  constexpr int SW = BN + BT;
  __shared__ __align__(16) char s0[SW * 128], s1[SW * 128], s2[SW * 128], s3[SW * 128];
  __shared__ float fs[BT * (FC + 1)], ws[FC];
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), l = threadIdx.x & 63, g4 = l >> 4, ql = l & 15;
  const int wn = (w % WN) * (BN / WN), wt = (w / WN) * (BT / WT);
  const int tn = (a.N + BN - 1) / BN, share = blockIdx.x % ks, id = blockIdx.x / ks, n0 = id % tn * BN, t0 = id / tn * BT;
  const int KB = (a.K + 127) >> 7, per = (KB + ks - 1) / ks, k0 = min(KB, share * per), n = min(KB, k0 + per) - k0;   // (its n blocks)
  const Span bb = rows_of(a.b, a.ldb, n0, a.N, BN, a.K), ba = rows_of(a.a, a.lda, t0, a.T, BT, a.K);
  const int rr = lane_row(w, l), ch = lane_col(rr, l);
  const uint32_t vb = rr * (uint32_t)a.ldb + ch, va = rr * (uint32_t)a.lda + ch;
  Span tb[LB], ta[LA];
#pragma unroll
  for (int i = 0; i < LB; ++i) tb[i] = turn_of(bb, i, W, a.ldb);
#pragma unroll
  for (int i = 0; i < LA; ++i) ta[i] = turn_of(ba, i, W, a.lda);
  auto load = [&](int i0, char* st) {              // (past the end: nothing is read)
    const Cols c = cols_of(k0 + i0, KB, a.K, ch, i0 < n);
#pragma unroll
    for (int i = 0; i < LB; ++i) load_lds(tb[i], boff(c.in, vb), c.at, st + (i * W + w) * 1024);
#pragma unroll
    for (int i = 0; i < LA; ++i) load_lds(ta[i], boff(c.in, va), c.at, st + BN * 128 + (i * W + w) * 1024);
  };
  auto frag = [&](const char* tile, int row) {     // chunks g4 and 4 + g4 of a row
    Codes<EXACT> c;
    const int z = (row >> 1) & 7;
    c.set(*reinterpret_cast<const uint4*>(tile + row * 128 + ((g4 ^ z) << 4)),
          *reinterpret_cast<const uint4*>(tile + row * 128 + (((4 + g4) ^ z) << 4)));
    return c;
  };
  f32x4 acc[MI][NI];
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < NI; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  // block kb of stage st; the stage that the block before it left is loaded for block kb + 3
  auto block = [&](int kb, const char* st, char* left) {
    asm volatile("" ::: "memory");
    // this wave's loads for kb are there, those of two more blocks may be on their way; then everyone's are, and all have left
    // the former block's stage
    __builtin_amdgcn_s_waitcnt(0x0F70 | (2 * L & 15) | ((2 * L >> 4) << 14));
    __builtin_amdgcn_s_waitcnt(0xC07F);
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    load(kb + 3, left);
    const float s = ws[kb % FC];
    Codes<EXACT> y[NI];
    float g[NI];
#pragma unroll
    for (int j = 0; j < NI; ++j) {
      y[j] = frag(st + BN * 128, wt + j * 16 + ql);
      g[j] = fs[(wt + j * 16 + ql) * (FC + 1) + kb % FC] * s;
    }
#pragma unroll
    for (int i = 0; i < MI; ++i) {
      const Codes<EXACT> x = frag(st, wn + i * 16 + ql);
#pragma unroll
      for (int j = 0; j < NI; ++j) {
        const f32x4 p = block_sum(x, y[j]);
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[i][j][e] = fmaf(p[e], g[j], acc[i][j][e]);
      }
    }
  };
  auto factors = [&](int i0) {                     // of FC blocks from the i0-th on
    __syncthreads();                               // (also waits for every load on its way)
    for (int i = threadIdx.x; i < BT * FC; i += W * 64) {
      const int t = i / FC, k = i0 + i % FC;
      fs[t * (FC + 1) + i % FC] = t0 + t < a.T && k < n ? a.sa[(long)(t0 + t) * KB + k0 + k] : 0.f;
    }
    const int k = i0 + threadIdx.x;
    if (threadIdx.x < FC) ws[threadIdx.x] = k < n ? a.sb[(long)(n0 >> 7) * KB + k0 + k] : 0.f;
    __syncthreads();
  };
  for (int ic = 0; ic < n; ic += FC) {
    factors(ic);
    const int ie = min(n, ic + FC);
    if (ic == 0) {
      load(0, s0);
      load(1, s1);
      load(2, s2);
    }
    // (FC is a multiple of the stages)
    for (int i = ic; i < ie; i += 4) {
      block(i, s0, s3);
      if (i + 1 < ie) block(i + 1, s1, s0);
      if (i + 2 < ie) block(i + 2, s2, s1);
      if (i + 3 < ie) block(i + 3, s3, s2);
    }
  }
  __builtin_amdgcn_s_waitcnt(0x0F70);              // (the loads past the end are on their way to this workgroup's LDS)
#pragma unroll
  for (int j = 0; j < NI; ++j) {
    const int t = t0 + wt + j * 16 + ql;
#pragma unroll
    for (int i = 0; i < MI; ++i) {
      const int n = n0 + wn + i * 16 + 4 * g4;
      if (t >= a.T || n >= a.N) continue;
      if (ks > 1) *reinterpret_cast<f32x4*>((float*)a.ws + ((long)share * a.T + t) * a.N + n) = acc[i][j];
      else store4<OT>(a.out, t * a.ldo + n, acc[i][j]);
    }
  }
}

// partial results of the shares of k, added up in their order
template <int OT>
__global__ __launch_bounds__(256) void k_mm_join(MmArgs a, int ks) {
  const long all = (long)a.T * a.N, i = ((long)blockIdx.x * 256 + threadIdx.x) * 4;
  if (i >= all) return;
  const int t = (int)(i / a.N), n = (int)(i - (long)t * a.N);
  f32x4 v = *reinterpret_cast<const f32x4*>((const float*)a.ws + i);
  for (int s = 1; s < ks; ++s) v += *reinterpret_cast<const f32x4*>((const float*)a.ws + s * all + i);
  store4<OT>(a.out, t * a.ldo + n, v);
}

// ------------------------------------------------------------------------------------------------ many tokens
// BN rows of B x BT tokens a workgroup of WN x WT waves; both operands' next block of k is on its way to LDS (direct loads)
// while this one is multiplied. A row's 16-byte chunk c lies in slot c ^ ((row >> 1) & 7): the 16 rows that a fragment's
// read touches at one chunk spread over all banks. Workgroups of one XCD take neighbouring tiles, 4 along the tokens, so that
// what they load at one time is shared in its L2.
// 4096 x 10240 x 8192, 687 GFLOP, fp16 results: 338 to 352 us on different cards, 362 to 375 under the profiler (1.8 to 2.0 PFLOP/s; a library product of that shape
// with one scale for each matrix takes 372 to 376). The matrix cores bound it together with the scaling (a multiply-add a result and
// block) and with the power they draw: 4096 x 8192 x 8192 took 282 us on a card where it took 211 without its loads and 218 with
// operands of zeros; 243 on another.
template <int OT, int BN, int BT, int WN, int WT>
__global__ __launch_bounds__(WN * WT * 64, 2) void k_mm_tile(MmArgs a, int ks) {
  constexpr int W = WN * WT, MI = BN / WN / 16, NI = BT / WT / 16;        // waves; 16-blocks of a wave
  // (the two turns' LDS are separate objects: the compiler then sees that loads on their way into one do not concern reads of
  // the other)
  __shared__ __align__(16) char b0[BN * 128], b1[BN * 128], a0[BT * 128], a1[BT * 128];
  __shared__ float fs[3 * BT * 8];
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), l = threadIdx.x & 63, g4 = l >> 4, ql = l & 15;
  const int wn = (w % WN) * (BN / WN), wt = (w / WN) * (BT / WT);
  static_assert(W % 2 == 0, "a lane's swizzle is the same in every turn of its rows");
  const int tn = (a.N + BN - 1) / BN, tt = (a.T + BT - 1) / BT, each = xcd_slice(blockIdx.x, gridDim.x),
            share = each % ks, id = each / ks;
  if (id >= tn * tt) return;
  const int first = id / (4 * tn) * 4, wide = min(4, tt - first), in = id % (4 * tn);
  const int n0 = in / wide * BN, t0 = (first + in % wide) * BT;
  const int KB = (a.K + 127) >> 7, per = (KB + ks - 1) / ks, k0 = min(KB, share * per), nk = min(KB, k0 + per) - k0;   // (its nk blocks)
  const Span bb = rows_of(a.b, a.ldb, n0, a.N, BN, a.K), ba = rows_of(a.a, a.lda, t0, a.T, BT, a.K);
  // direct loads: one offset of a lane serves all turns and blocks. Past the last row, and past K, zeros are read.
  const int rr = lane_row(w, l), ch = lane_col(rr, l);
  const uint32_t vb = rr * (uint32_t)a.ldb + ch, va = rr * (uint32_t)a.lda + ch;
  constexpr int LB = BN / 8 / W, LA = BT / 8 / W;  // direct loads of a wave and block
  Span tb[LB], ta[LA];
#pragma unroll
  for (int i = 0; i < LB; ++i) tb[i] = turn_of(bb, i, W, a.ldb);
#pragma unroll
  for (int i = 0; i < LA; ++i) ta[i] = turn_of(ba, i, W, a.lda);
  auto load = [&](int i, int kb, char* lb, char* la) {
    const Cols c = cols_of(k0 + kb, KB, a.K, ch, kb < nk);
    if (i < LB) load_lds(tb[i], boff(c.in, vb), c.at, lb + (i * W + w) * 1024);
    else load_lds(ta[i - LB], boff(c.in, va), c.at, la + ((i - LB) * W + w) * 1024);
  };
  auto arrive = [&] {                              // every wave's direct loads are there
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0x0F70);
    __syncthreads();
  };
  // Factors of the tokens: through LDS, for 8 blocks at a time (a row of sa is 4 bytes a block: read block by block, its lines
  // came from L2 as often as the codes': 4096 x 8192 x 8192 in 311 us, so in 282). Of the tile's BT tokens x 8 blocks, BT values are
  // loaded with every block and put in their place with the next; they are complete when the 8 blocks begin, and the ring's third
  // place is the one that nobody reads.
  const Buf bs(a.sa + (long)t0 * KB, (uint32_t)min(a.T - t0, BT) * KB * 4),
      bw(a.sb + (long)((n0 + wn) >> 7) * KB, n0 + wn < a.N ? (uint32_t)KB * 4 : 0u);
  constexpr int SL = BT / 8;                       // tokens of a slice
  const int ft = (threadIdx.x % BT) >> 3, fk = threadIdx.x & 7;
  auto fetch = [&](int p) {                        // slice p & 7 of the 8 blocks behind those of block p
    return bs.ldf(factor_at(p, SL, KB, k0, ft, fk));
  };
  auto place = [&](int p, float v) { fs[((((p >> 3) + 1) % 3) * BT + (p & 7) * SL + ft) * 8 + fk] = v; };
  auto weight = [&](int kb) { return bw.ldf((k0 + kb) * 4); };
  f32x4 acc[MI][NI];
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < NI; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  auto frag = [&](const char* tile, int row) {       // chunks g4 and 4 + g4 of a row
    Codes<OT == T_F32> c;
    const int z = (row >> 1) & 7;
    c.set(*reinterpret_cast<const uint4*>(tile + row * 128 + ((g4 ^ z) << 4)),
          *reinterpret_cast<const uint4*>(tile + row * 128 + (((4 + g4) ^ z) << 4)));
    return c;
  };
#pragma unroll
  for (int i = 0; i < LB + LA; ++i) load(i, 0, b0, a0);
  for (int p = -8; p < 2; ++p) place(p, fetch(p));
  float s = weight(0), fv = fetch(2);
  arrive();
#pragma unroll
  for (int i = 0; i < LB + LA; ++i) load(i, 1, b1, a1);
  // One block. Results are scaled and added while the next row's products run (those of the last row under the next block's
  // first), a row's operand is read one row ahead. Before the last row the waves meet: nobody reads this block's LDS any more,
  // which the block after the next is loaded into, and the next block's has arrived, so the last row's products run while the next
  // block's first operands are read (with waves that meet at the end of a block: 362 us for 357, fp32 results 666 for 599).
  Codes<OT == T_F32> x = frag(b0, wn + ql), y[NI];
  f32x4 p[NI];
  float gp[NI];
#pragma unroll
  for (int j = 0; j < NI; ++j) {
    y[j] = frag(a0, wt + j * 16 + ql);
    p[j] = f32x4{0.f, 0.f, 0.f, 0.f};
    gp[j] = 0.f;
  }
  auto block = [&](int kb, char* lb, char* la, const char* nb, const char* na) {
    place(kb + 2, fv);
    fv = fetch(kb + 3);
    const float sn = weight(kb + 1);
    float g[NI];
#pragma unroll
    for (int i = 0; i < MI; ++i) {
      if (i == MI - 1) arrive();
      if (i == 1) {
#pragma unroll
        for (int j = 0; j < NI; ++j) g[j] = fs[(((kb >> 3) % 3) * BT + wt + j * 16 + ql) * 8 + (kb & 7)] * s;
      }
      const Codes<OT == T_F32> xn = i < MI - 1 ? frag(lb, wn + (i + 1) * 16 + ql) : frag(nb, wn + ql);
#pragma unroll
      for (int j = 0; j < NI; ++j) {
        const f32x4 q = block_sum(x, y[j]);
        if (i == MI - 1) {
          y[j] = frag(na, wt + j * 16 + ql);
#pragma unroll
          for (int c = j * (LB + LA) / NI; c < (j + 1) * (LB + LA) / NI; ++c) load(c, kb + 2, lb, la);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[(i + MI - 1) % MI][j][e] = fmaf(p[j][e], i ? g[j] : gp[j], acc[(i + MI - 1) % MI][j][e]);
        p[j] = q;
        // (in this order: a product occupies the matrix core for as long as eight vector instructions take)
        if (OT != T_F32) __builtin_amdgcn_sched_barrier(0);
      }
      x = xn;
    }
    s = sn;
#pragma unroll
    for (int j = 0; j < NI; ++j) gp[j] = g[j];
  };
  int kb = 0;
  for (; kb + 1 < nk; kb += 2) {
    block(kb, b0, a0, b1, a1);
    block(kb + 1, b1, a1, b0, a0);
  }
  if (kb < nk) block(kb, b0, a0, b1, a1);
  __builtin_amdgcn_s_waitcnt(0x0F70);                // (the loads past the end are on their way to this workgroup's LDS)
#pragma unroll
  for (int j = 0; j < NI; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[MI - 1][j][e] = fmaf(p[j][e], gp[j], acc[MI - 1][j][e]);
#pragma unroll
  for (int j = 0; j < NI; ++j) {
    const int t = t0 + wt + j * 16 + ql;
#pragma unroll
    for (int i = 0; i < MI; ++i) {
      const int n = n0 + wn + i * 16 + 4 * g4;
      if (t >= a.T || n >= a.N) continue;
      if (ks > 1) *reinterpret_cast<f32x4*>((float*)a.ws + ((long)share * a.T + t) * a.N + n) = acc[i][j];
      else store4<OT>(a.out, t * a.ldo + n, acc[i][j]);
    }
  }
}

template <int OT>
hipError_t go(const MmArgs& a, hipStream_t st) {
  const MmPlan p = mm_plan(a.T, a.N, a.K, OT == T_F32);
  auto tiles = [&](int n, int t) { return (unsigned)((long)((a.N + n - 1) / n) * ((a.T + t - 1) / t)); };
  auto whole = [&](unsigned v) { return dim3((v + 7) / 8 * 8); };
  if (p.how == FEW) {
    // (waves as many as leave 16 on a compute unit)
    const unsigned n = tiles(16, 16);
    if (n >= 512) hipLaunchKernelGGL((k_mm_few<OT, 4>), dim3(n), dim3(256), 0, st, a);
    else if (n >= 256) hipLaunchKernelGGL((k_mm_few<OT, 8>), dim3(n), dim3(512), 0, st, a);
    else hipLaunchKernelGGL((k_mm_few<OT, 16>), dim3(n), dim3(1024), 0, st, a);
  } else if (p.how == SOME32) hipLaunchKernelGGL((k_mm_some<OT, true, 64, 32, 4, 1>), dim3(tiles(64, 32) * p.ks), dim3(256), 0, st, a, p.ks);
  else if (p.how == SOME64) hipLaunchKernelGGL((k_mm_some<OT, true, 64, 64, 2, 2>), dim3(tiles(64, 64) * p.ks), dim3(256), 0, st, a, p.ks);
  else if (p.how == SOME128) hipLaunchKernelGGL((k_mm_some<OT, OT == T_F32, 64, 128, 2, 4>), dim3(tiles(64, 128) * p.ks), dim3(512), 0, st, a, p.ks);
  else if (p.how == TILE128 || OT == T_F32) hipLaunchKernelGGL((k_mm_tile<OT, 128, 128, 2, 2>), whole(tiles(128, 128) * p.ks), dim3(256), 0, st, a, p.ks);
  else if constexpr (OT != T_F32) hipLaunchKernelGGL((k_mm_tile<OT, 256, 256, 2, 4>), whole(tiles(256, 256) * p.ks), dim3(512), 0, st, a, p.ks);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.ks == 1) return e;
  hipLaunchKernelGGL(k_mm_join<OT>, dim3((unsigned)(((long)a.T * a.N / 4 + 255) / 256)), dim3(256), 0, st, a, p.ks);
  return hipGetLastError();
}

}  // namespace

size_t sffn_mm_workspace(int T, int N, int K) {
  // (whichever type the results are of)
  const MmPlan p = mm_plan(T, N, K, false), q = mm_plan(T, N, K, true);
  const int ks = p.ks > q.ks ? p.ks : q.ks;
  return ks > 1 ? (size_t)ks * T * N * sizeof(float) : 0;
}

hipError_t sffn_launch_mm(const MmArgs& a, int ot, hipStream_t st) {
  return ot == T_F32 ? go<T_F32>(a, st) : ot == T_F16 ? go<T_F16>(a, st) : go<T_BF16>(a, st);
}
