// decay_tc.cuh -- the recurrence of decay.cuh on the sm_100a tensor cores
// (tcgen05 + TMEM, operands staged by TMA), bf16 in, fp32 accumulate, for
// widths up to 128 (narrower ones are zero-filled to 64 or 128 by the loads).
//
// Per tile of C = 128 tokens, rows r and columns c in memory order, with P and
// the powers of decay.cuh:
//   Sc = Q K^T                       M = C,  N = C,  K = DK
//   O2 = Q X^T                       M = C,  N = DV, K = DK
//   D  = V^T K~ , K~_c = w_c k_c     M = DV, N = DK, K = C
//   O1 = P V , P = weights * Sc      M = C,  N = DV, K = C
//   o_r = O1 + (read power of r) O2 ,  X <- gamma^n X + D
// The state X stays in registers in fp32: D is a fresh product every tile, so
// the decay between tiles is one FMA and the tensor memory is only read.  The
// read power multiplies O2 in fp32 in the epilogue, so Q is used as loaded.
//
// Three launches where a sequence has several segments or its final state is
// wanted:
//   decay_tc_total_kernel   every segment's own contribution to the state, by
//       tiles of 64 or 128 tokens whose products are added in fp32 registers, K~ as
//       three bf16 parts whose sum it is: the states that the caller sees are
//       fp32 sums of unrounded products.
//   decay_scan_kernel       contributions -> start states and final states.
//   decay_tc_out_kernel     the outputs.  P, the state where it is read for O2
//       and K~ are two bf16 parts each, which carry them to 2^-14, so that an
//       output is off by its own rounding, 1.66e-3 of its norm.  With one part
//       of P and of the state it was 2.35e-3, at 196 us for 1 x 8 x 65536 x 128
//       where two take 210 (227 and 254 at the power cap's clock), and 281 us
//       for the gradient of 2 x 16 x 8192 x 128 where two take 303 (313, 356).
//
// Weights gamma^(r-c) <= 1 come as products of a row's and a column's power,
// each with a distance >= 0 to the edge of a 32-column block, so no power
// overflows however strong the decay: an underflow is a weight below 2^-126.
//
// Waits are bounded as in chunked_tc.cuh: a thread whose wait runs out stops
// waiting, and issues no more copies or MMAs, but keeps arriving, so that the
// block drains and exits with nothing of its own in flight.
#pragma once
#include "chunked_tc.cuh"
#include "chunked_tc_mom.cuh"
#include "common.cuh"
#include "decay.cuh"

namespace ttt {

__device__ __forceinline__ void tma_load_4d(const CUtensorMap* m, uint64_t* bar, void* dst, int x, int y, int z, int w,
                                            uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint "
      "[%0], [%1, {%3, %4, %5, %6}], [%2], %7;" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z), "r"(w), "l"(policy)
      : "memory");
}
__device__ __forceinline__ void tma_store_4d(const CUtensorMap* m, const void* src, int x, int y, int z, int w) {
  asm volatile("cp.async.bulk.tensor.4d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4, %5}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(m)),
               "r"(smem_u32(src)), "r"(x), "r"(y), "r"(z), "r"(w)
               : "memory");
}
// tmem_ld32 with 16 columns.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]), "r"(r[1]),
               "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
// After tmem_ld_wait: what is made of r stays behind it.
__device__ __forceinline__ void tmem_ld_done(uint32_t (&r)[16]) {
  asm volatile("" : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                    "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]));
}
// tmem_ld_half32 with 16 columns a thread.
__device__ __forceinline__ void tmem_ld_half16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x32bx2.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16], 16;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}

constexpr int kDecayTcC = 128;      // tokens per tile of the outputs
// Tokens per tile of the totals, for keys of d features (padded): 64 where three
// parts of 128 tokens would leave no room to load ahead.
__host__ __device__ constexpr int decay_total_tile(int d) { return d <= 64 ? 128 : 64; }
constexpr int kDecayTcRuns = 3;     // the most runs in one launch
constexpr int kDecayTcMaps = 11;

// One run: indices of its tensors' maps, and the recurrence's parameters.
struct DecayTcRun {
  int q, k, v, o;           // indices into DecayTcArgs::map
  int kt, vt;               // k and v in the totals' tiles
  int dk, dv;
  int rev;
  float sP, sR, sU;
  const float* s_in;        // start states of sequences that are one segment (ws_all: of none)
  int s_in_t;               // they are [dk][dv]
  float* s_out;             // total kernel: final states of sequences that are one segment, or nullptr
  float* ws;                // per segment: contributions, then start states; nullptr: one segment each
  int ws_t;                 // start states there are [dk][dv] (they are another run's)
  int ws_all;               // sequences of one segment go through ws too
  int total_last;           // total kernel: contributions of the last segment in walking order as well
  // outputs of tiles that end inside the tensor's rows
  __nv_bfloat16* op;
  long long ob, oh, ot;
};
struct alignas(64) DecayTcArgs {
  CUtensorMap map[kDecayTcMaps];
  DecayGeom g;
  DecayTcRun run[kDecayTcRuns];
  int nrun;
  int clear;                // zeros for the first run's rows of o in no (packed) sequence
  const float* log_decay;
  uint64_t limit_ns;
};

// decay_span by all threads of the block (at most 768), where there are more
// sequences than a warp sees at once; sh: 64 ints of shared memory on 8 bytes.
__device__ __forceinline__ DecaySpan decay_span_block(const DecayGeom& g, int s, int* sh) {
  if (!g.cu || g.N <= 32) return decay_span(g, s);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nw = blockDim.x >> 5;
  if (tid == 0) sh[48] = -1;
  int before = 0, single = 0;
  for (int n0 = 0; n0 < g.N; n0 += static_cast<int>(blockDim.x)) {
    const int n = n0 + tid;
    int a = 0, b = 0, c = 0;
    if (n < g.N) {
      decay_rows(g, n, a, b);
      c = decay_segments(b - a, g.S);
    }
    int incl = c;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, off);
      if (lane >= off) incl += y;
    }
    const unsigned one = __ballot_sync(0xffffffffu, c == 1 && !g.all);
    int2* sums = reinterpret_cast<int2*>(sh);
    if (lane == 31) sums[warp] = make_int2(incl, __popc(one));
    __syncthreads();
    int below = before, all = before, none = single + __popc(one & ((1u << lane) - 1u));
    for (int w = 0; w < nw; ++w) {
      const int2 x = sums[w];
      if (w < warp) {
        below += x.x;
        none += x.y;
      }
      all += x.x;
      single += x.y;
    }
    incl += below;
    if (incl > s && incl - c <= s && c > 0) {  // exactly one thread, if any
      sh[48] = n;
      sh[49] = a;
      sh[50] = b;
      sh[51] = s - (incl - c);
      sh[52] = c;
      sh[53] = s - none;
    }
    before = all;
    __syncthreads();
    if (sh[48] >= 0) break;
  }
  DecaySpan r;
  r.seq = sh[48];
  r.batch = 0;
  r.row0 = r.len = r.j = r.nseg = r.slot = 0;
  if (r.seq >= 0) {
    r.j = sh[51];
    r.nseg = sh[52];
    r.row0 = sh[49] + r.j * g.S;
    r.len = min(g.S, sh[50] - r.row0);
    r.slot = sh[53];
    if ((r.nseg > 1 || g.all) && r.slot >= g.slots) r.seq = -1;
  }
  return r;
}

template <int DK, int DV>
struct DecayTcCfg {
  static constexpr int C = kDecayTcC;
  static constexpr int TK = C * DK * 2, TV = C * DV * 2;   // bytes of a tile
  static constexpr int STAGE = 2 * TK + TV;                // Q, K, V
  static constexpr int WBF = DK * DV * 2;
  // the second parts of K~ and of the state have places of their own where two stages still fit beside them (LSEP);
  // else K~'s goes over the state's first part, which has been read by then, and the state's over the Q of the tile
  // before, which then is loaded anew one tile later than K and V
  static constexpr bool LSEP = 2 * STAGE + 2 * WBF + TK <= 232448 - 2048;
  static constexpr int LO = LSEP ? TK + WBF : 0, ROOM = (232448 - 2048 - WBF - LO) / STAGE;
  static constexpr int NST = ROOM > 4 ? 4 : ROOM;
  static constexpr int BIG = NST * STAGE + WBF + LO;
  static constexpr int SMEM = BIG + 1024 + 1024;           // + barriers and tables, + alignment
  static_assert((5 * NST + 18) * 8 + 98 * 4 + 64 * 4 <= 1024, "barriers, tables and decay_span_block's");
  static constexpr int THREADS = 608;                      // TMA, MMA, 8 warps P and outputs, 8 warps state, MMA
  static constexpr int NW = DK * DV / 256;                 // elements of X per state thread
  // tensor memory: Sc (P over it; twice where it fits), O1, O2, D
  static constexpr int NSB = DV == 64 ? 2 : 1;
  static constexpr int T_O1 = NSB * C, T_O2 = T_O1 + DV, T_D = T_O2 + DV;
  static_assert(DV * (DK + 4) * 4 <= STAGE, "the start state's buffer");
  static_assert(NST >= 2 && T_D + DK <= 512, "shared and tensor memory");
  // total kernel: K (then its first part) and V per stage; the other two parts twice
  static constexpr int CT = decay_total_tile(DK), A_TK = CT * DK * 2, A_TV = CT * DV * 2, A_STAGE = A_TK + A_TV;
  static constexpr int A_NST = (232448 - 2048 - 4 * A_TK) / A_STAGE > 8 ? 8 : (232448 - 2048 - 4 * A_TK) / A_STAGE;
  static constexpr int A_SMEM = A_NST * A_STAGE + 4 * A_TK + 1024 + 1024;
  static constexpr int A_THREADS = 576;                    // TMA, MMA, 8 warps that split K~, 8 that add products
  static_assert(A_SMEM <= 232448, "shared memory");
};

// The elements of the DV x DK state that thread (w = 0..7, lane) of the state
// warps owns: row `row`, columns col .. col + NW.  DV = 128: a TMEM lane a row.
// DV = 64: an M = 64 accumulator fills lanes 0-15 of each quadrant, read in two
// column halves by the two halves of the warp.  Warp w must be on quadrant w & 3.
template <int DK, int DV>
__device__ __forceinline__ void decay_state_at(int quad, int half, int lane, int& row, int& col) {
  if constexpr (DV == 128) {
    row = quad * 32 + lane;
    col = half * (DK / 2);
  } else {
    row = quad * 16 + (lane & 15);
    col = half * (DK / 2) + (lane >> 4) * (DK / 4);
  }
}
// Elements [i, i + N) of them (DV = 64: i = 0, N = NW).
template <int DK, int DV, int N>
__device__ __forceinline__ void decay_state_ld(uint32_t t_d, int quad, int half, int i, uint32_t (&r)[N]) {
  const uint32_t at = t_d + (static_cast<uint32_t>(quad * 32) << 16) + half * (DK / 2) + i;
  static_assert(DV == 128 ? N == 16 : N == DK / 4, "");
  if constexpr (DV == 128)
    tmem_ld16(at, r);
  else if constexpr (DK == 128)
    tmem_ld_half32(at, r);
  else
    tmem_ld_half16(at, r);
}

// Takes the leading bf16 of each of two values off x and returns the pair of
// them.  The upper halves of the words, not the nearest values: a part then is a
// byte permutation, and what is left is exact with 8 of 24 bits less, so three
// parts are the value itself.
__device__ __forceinline__ uint32_t take_bf16x2(f2& x) {
  const uint32_t a = __float_as_uint(lo_of(x)), b = __float_as_uint(hi_of(x));
  x = add2(x, pair((a & 0xffff0000u) ^ 0x80000000u, (b & 0xffff0000u) ^ 0x80000000u));
  return __byte_perm(a, b, 0x7632);
}
// x as the sum of two bf16 values, to 2^-14 of it.
__device__ __forceinline__ void split_bf16x2(f2 x, uint32_t& hi, uint32_t& lo) {
  hi = take_bf16x2(x);
  lo = take_bf16x2(x);
}
// Splits a K tile (64-column blocks of C rows of 128 bytes) scaled by w[i], the
// weight of row (t >> 3) + 32 i, for thread t of 256, into three bf16 tiles of
// decreasing size whose sum it is: the first over the tile itself, the others
// at `rest`, `rest` + one tile.  (A unit's place in its row does not matter
// here, so the swizzle is left alone.)
template <int DK, int C>
__device__ __forceinline__ void decay_scale_tile(uint8_t* kt, uint8_t* rest, int t, const float (&w)[C / 32]) {
#pragma unroll 1
  for (int b = 0; b < DK / 64; ++b)
#pragma unroll
  for (int i = 0; i < C / 32; ++i) {
    const int u = (b * (C / 32) + i) * 256 + t;
    const uint4 x = *reinterpret_cast<const uint4*>(kt + u * 16);
    const uint32_t xs[4] = {x.x, x.y, x.z, x.w};
    uint32_t out[3][4];
    const f2 wt = pair(w[i], w[i]);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      f2 y = mul2(pair(xs[e] << 16, xs[e] & 0xffff0000u), wt);
#pragma unroll
      for (int r = 0; r < 3; ++r) out[r][e] = take_bf16x2(y);
    }
    *reinterpret_cast<uint4*>(kt + u * 16) = make_uint4(out[0][0], out[0][1], out[0][2], out[0][3]);
#pragma unroll
    for (int r = 1; r < 3; ++r)
      *reinterpret_cast<uint4*>(rest + (r - 1) * (C * DK * 2) + u * 16) = make_uint4(out[r][0], out[r][1], out[r][2], out[r][3]);
  }
}
// The same in two parts for the rows [64 y, 64 y + 64) of a tile: the first over
// the tile, the second into registers, and from there to `rest`.
template <int DK, int C>
__device__ __forceinline__ void decay_scale_half(uint8_t* kt, int t, int y, float w0, float w1, uint4 (&lo)[DK / 32]) {
#pragma unroll
  for (int i = 0; i < DK / 32; ++i) {
    uint4* at = reinterpret_cast<uint4*>(kt + (((i >> 1) * (C / 32) + 2 * y + (i & 1)) * 256 + t) * 16);
    const uint4 x = *at;
    const f2 wt = i & 1 ? pair(w1, w1) : pair(w0, w0);
    uint4 hi;
    split_bf16x2(mul2(pair(x.x << 16, x.x & 0xffff0000u), wt), hi.x, lo[i].x);
    split_bf16x2(mul2(pair(x.y << 16, x.y & 0xffff0000u), wt), hi.y, lo[i].y);
    split_bf16x2(mul2(pair(x.z << 16, x.z & 0xffff0000u), wt), hi.z, lo[i].z);
    split_bf16x2(mul2(pair(x.w << 16, x.w & 0xffff0000u), wt), hi.w, lo[i].w);
    *at = hi;
  }
}
template <int DK, int C>
__device__ __forceinline__ void decay_store_half(uint8_t* rest, int t, int y, const uint4 (&lo)[DK / 32]) {
#pragma unroll
  for (int i = 0; i < DK / 32; ++i)
    *reinterpret_cast<uint4*>(rest + (((i >> 1) * (C / 32) + 2 * y + (i & 1)) * 256 + t) * 16) = lo[i];
}
// Zeroes the rows >= n of a tile of D features: what is in memory behind a
// segment's end, whatever it holds, then enters no sum.
template <int D, int C>
__device__ __forceinline__ void decay_zero_rows(uint8_t* tile, int n, int t) {
  const uint4 z = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll 1
  for (int u = t; u < C * D / 8; u += 256)
    if (((u >> 3) & (C - 1)) >= n) *reinterpret_cast<uint4*>(tile + u * 16) = z;
}

// The start state into registers through shared memory: 256 threads read whole
// rows (a thread's own row would be a line of its own in each load: measured
// 7 us for 128 x 128 where this takes 1), `buf` holds [DV][DK + 4] floats.
template <int DK, int DV, int NW>
__device__ __forceinline__ void decay_state_in(float* buf, const float* src, bool transposed, int dk, int dv, int t,
                                               int row, int col, float (&w)[NW]) {
  constexpr int LD = DK + 4;
  const int wp = t >> 5, lane = t & 31;
  if (transposed) {  // [dk][dv]
#pragma unroll 4
    for (int c = wp; c < DK; c += 8)
#pragma unroll
      for (int v = 0; v < DV; v += 32)
        buf[(v + lane) * LD + c] = c < dk && v + lane < dv ? ld_after(src + static_cast<size_t>(c) * dv + v + lane) : 0.f;
  } else {
    constexpr int PER = 128 / DK;  // rows a warp reads at once
    const int c = (lane % (DK / 4)) * 4;
#pragma unroll 8
    for (int r = wp * PER + lane / (DK / 4); r < DV; r += 8 * PER) {
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
      if (r < dv && c < dk) x = ld_after(reinterpret_cast<const float4*>(src + static_cast<size_t>(r) * dk + c));
      *reinterpret_cast<float4*>(buf + r * LD + c) = x;
    }
  }
  asm volatile("bar.sync 2, 256;" ::: "memory");
#pragma unroll
  for (int e = 0; e < NW; e += 4) {
    const float4 x = *reinterpret_cast<const float4*>(buf + row * LD + col + e);
    w[e] = x.x, w[e + 1] = x.y, w[e + 2] = x.z, w[e + 3] = x.w;
  }
}

// A suspending wait; nothing once `dead`.
__device__ __forceinline__ void decay_wait(bool& dead, uint64_t* bar, uint32_t parity, uint64_t lim) {
  if (!dead) dead = !mbar_wait_suspended(bar, parity, lim);
}
// This warp's writes (and tensor memory reads) before one arrival for it.
__device__ __forceinline__ void warp_arrive(uint64_t* bar, int lane) {
  tc_fence_before();
  __syncwarp();
  if (lane == 0) mbar_arrive(bar);
}

// ------------------------------------------------------------- totals ----
// One block per (segment, head, run).  Tiles are walked from the far end of
// the walking order to its start, so that the tiles the output kernel reads
// first are the ones last left in L2.  Warps 0 load, 1 issues, 2-9 split K~ into
// its parts, 10-17 add the products.  Bound by shared memory, through which 192
// KB pass for 64 tokens of 128 x 128 (three products, K read and three parts
// written).  Measured: 1 x 8 x 65536 x 128 73 us (268 MB read, 3.7 TB/s; 54 us
// with two parts, 82 with one set of warps for both), 4 x 16 x 4096 x 64 27 us
// (33 with tiles of 64 tokens).
template <int DK, int DV>
__global__ void __launch_bounds__(576, 1) decay_tc_total_kernel(const __grid_constant__ DecayTcArgs A) {
  using Cfg = DecayTcCfg<DK, DV>;
  constexpr int C = Cfg::CT, NST = Cfg::A_NST, STAGE = Cfg::A_STAGE, TK = Cfg::A_TK, TV = Cfg::A_TV, NW = Cfg::NW;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* rest = smem + NST * STAGE;  // [2][2] second and third parts of K~
  uint64_t* bars = reinterpret_cast<uint64_t*>(rest + 4 * TK);
  uint64_t* full = bars;               // [NST] tile landed
  uint64_t* ready = bars + NST;        // [NST] K~ written
  uint64_t* empty = bars + 2 * NST;    // [NST] stage read
  uint64_t* dfull = bars + 3 * NST;    // [2] product complete
  uint64_t* lofree = dfull + 2;        // [2] second and third parts read
  uint64_t* dfree = dfull + 4;         // [2] product read out
  uint64_t* drain = dfull + 6;
  uint32_t* holder = reinterpret_cast<uint32_t*>(drain + 1);
  int* sh = reinterpret_cast<int*>(holder + 2);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const DecayGeom& g = A.g;
  const int b = blockIdx.x, ri = b % A.nrun, h = (b / A.nrun) % g.H, s = b / A.nrun / g.H;
  const DecayTcRun& p = A.run[ri];
  const DecaySpan sp = decay_span_block(g, s, sh);
  launch_next();
  if (sp.seq < 0 || (!p.total_last && sp.j == (p.rev ? 0 : sp.nseg - 1))) {
    wait_before();
    return;
  }
  const uint64_t lim = A.limit_ns;
  const int nt = (sp.len + C - 1) / C;
  auto tile_at = [&](int i) { return p.rev ? i : nt - 1 - i; };

  if (threadIdx.x == 0) {
    for (int i = 0; i < NST; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&ready[i], 8);
      mbar_init(&empty[i], 1);
    }
    mbar_init(&dfull[0], 1);
    mbar_init(&dfull[1], 1);
    mbar_init(&dfree[0], 8);
    mbar_init(&dfree[1], 8);
    mbar_init(&lofree[0], 1);
    mbar_init(&lofree[1], 1);
    mbar_init(drain, 1);
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(holder, 2 * DK);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *holder;

  if (warp == 0) {
    if (lane == 0) {
      bool dead = false;
      int sent = 0;
      const uint64_t pol = l2_policy_evict_last();
      for (int i = 0; i < nt; ++i) {
        const int st = i % NST, y = sp.row0 + tile_at(i) * C;
        if (i >= NST) decay_wait(dead, &empty[st], (i / NST - 1) & 1, lim);
        if (dead) break;
        mbar_arrive_expect_tx(&full[st], TK + TV);
        uint8_t* d = smem + st * STAGE;
#pragma unroll
        for (int x = 0; x < DK / 64; ++x) tma_load_4d(&A.map[p.kt], &full[st], d + x * C * 128, x * 64, y, h, sp.batch, pol);
#pragma unroll
        for (int x = 0; x < DV / 64; ++x)
          tma_load_4d(&A.map[p.vt], &full[st], d + TK + x * C * 128, x * 64, y, h, sp.batch, pol);
        sent = i + 1;
      }
      for (int i = max(0, sent - NST); i < sent; ++i) mbar_wait(&full[i % NST], (i / NST) & 1, lim);
    }
  } else if (warp == 1) {
    if (lane == 0) {
      bool dead = false;
      constexpr uint32_t ID = idesc_bf16_f32(DV, DK, true, true);
      for (int i = 0; i < nt; ++i) {
        const int st = i % NST;
        const uint32_t base = smem_u32(smem) + st * STAGE;
        const uint64_t dk = sdesc_sw128(base, C * 128, 1024), dv = sdesc_sw128(base + TK, C * 128, 1024);
        // the smallest part first, so that the sums lose least
        const uint64_t parts[3] = {sdesc_sw128(smem_u32(rest) + ((i & 1) * 2 + 1) * TK, C * 128, 1024),
                                   sdesc_sw128(smem_u32(rest) + (i & 1) * 2 * TK, C * 128, 1024), dk};
        decay_wait(dead, &ready[st], (i / NST) & 1, lim);
        if (i > 1) decay_wait(dead, &dfree[i & 1], ((i >> 1) - 1) & 1, lim);
        tc_fence_after();
#pragma unroll
        for (int r = 0; r < 3; ++r) {
          if (!dead) {
#pragma unroll
            for (int kk = 0; kk < C / 16; ++kk)
              mma_bf16_ss(tmem + (i & 1) * DK, dv + mn_step(kk), parts[r] + mn_step(kk), ID, r > 0 || kk > 0);
          }
          if (r == 1) tc_commit(&lofree[i & 1]);
        }
        tc_commit(&empty[st]);
        tc_commit(&dfull[i & 1]);
      }
      tc_commit(drain);
      mbar_wait(drain, 0, lim);
    }
  } else if (warp < 10) {
    // K~ in three parts
    bool dead = false;
    const int t = static_cast<int>(threadIdx.x) - 64;
    const float l = decay_log(A.log_decay, h);
    // row weights inside a tile: distance to its end (reverse: to before its start)
    float wgt[C / 32];
    auto weights = [&](int n) {
#pragma unroll
      for (int x = 0; x < C / 32; ++x) {
        const int r = (t >> 3) + 32 * x;
        wgt[x] = p.sU * expf(l * static_cast<float>(p.rev ? r + 1 : max(n - 1 - r, 0)));
      }
    };
    weights(C);
    for (int i = 0; i < nt; ++i) {
      const int st = i % NST, n = min(C, sp.len - tile_at(i) * C);
      decay_wait(dead, &full[st], (i / NST) & 1, lim);
      uint8_t* d = smem + st * STAGE;
      if (n < C) weights(n);
      if (i > 1) decay_wait(dead, &lofree[i & 1], ((i >> 1) - 1) & 1, lim);
      __syncwarp();
      uint8_t* parts = rest + (i & 1) * 2 * TK;
      decay_scale_tile<DK, C>(d, parts, t, wgt);
      if (n < C) {
        // (a thread zeroes the units that it scaled itself)
        decay_zero_rows<DK, C>(d, n, t);
        decay_zero_rows<DK, C>(parts, n, t);
        decay_zero_rows<DK, C>(parts + TK, n, t);
        decay_zero_rows<DV, C>(d + TK, n, t);
        weights(C);
      }
      fence_async_smem();
      warp_arrive(&ready[st], lane);
    }
  } else {
    // the sum of the tiles' products, each weighted by its tile's distance
    bool dead = false;
    const int quad = warp & 3, half = (warp - 10) >> 2;
    const float l = decay_log(A.log_decay, h);
    float acc[NW];
#pragma unroll
    for (int e = 0; e < NW; ++e) acc[e] = 0.f;
    for (int i = 0; i < nt; ++i) {
      const int at = tile_at(i) * C, n = min(C, sp.len - at);
      const float f = expf(l * static_cast<float>(p.rev ? at : sp.len - at - n));
      decay_wait(dead, &dfull[i & 1], (i >> 1) & 1, lim);
      __syncwarp();
      tc_fence_after();
      constexpr int PIECE = DV == 128 ? 16 : NW;
#pragma unroll
      for (int x = 0; x < NW; x += PIECE) {
        uint32_t r[PIECE];
        decay_state_ld<DK, DV>(tmem + (i & 1) * DK, quad, half, x, r);
        tmem_ld_wait();
        if (x + PIECE == NW) warp_arrive(&dfree[i & 1], lane);
#pragma unroll
        for (int e = 0; e < PIECE; ++e) acc[x + e] = fmaf(f, __uint_as_float(r[e]), acc[x + e]);
      }
    }
    int row, col;
    decay_state_at<DK, DV>(quad, half, lane, row, col);
    const size_t dd = static_cast<size_t>(p.dk) * p.dv, off = static_cast<size_t>(row) * p.dk;
    // a sequence of one segment: its final state is made here
    const bool direct = sp.nseg == 1 && !p.ws_all;
    float* dst = (direct ? p.s_out + (static_cast<size_t>(sp.seq) * g.H + h) * dd
                         : p.ws + (static_cast<size_t>(sp.slot) * g.H + h) * dd) + off;
    const float* src = direct && p.s_in ? p.s_in + (static_cast<size_t>(sp.seq) * g.H + h) * dd + off : nullptr;
    const float gl = expf(l * static_cast<float>(sp.len));
#pragma unroll
    for (int e = 0; e < NW; e += 4) {
      const int c = col + e;
      if (row >= p.dv || c >= p.dk) continue;
      float4 x = make_float4(acc[e], acc[e + 1], acc[e + 2], acc[e + 3]);
      if (src) {
        const float4 y = *reinterpret_cast<const float4*>(src + c);
        x.x = fmaf(gl, y.x, x.x);
        x.y = fmaf(gl, y.y, x.y);
        x.z = fmaf(gl, y.z, x.z);
        x.w = fmaf(gl, y.w, x.w);
      }
      *reinterpret_cast<float4*>(dst + c) = x;
    }
    tc_fence_before();
  }
  wait_before();  // (nothing here depends on the launch before)
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 2 * DK);
  }
}

// ------------------------------------------------------------ outputs ----
// One block per (segment, head, run), one per SM.  19 warps: 0 TMA loads, 1
// issues Sc, O2 and O1, 2-9 P and the outputs, 10-17 the state and K~, 18
// issues D.  P lies over the scores, as the MMA's operand in tensor memory.
// Where tensor memory has room for one set of score columns, Sc of tile i + 1
// follows O1 of tile i; where it has two, it comes before O1 and the warps
// write P of tile i + 1 before they read the output of tile i.  Q and K are
// free once O2 and D are done (Q, where it then holds a part of the state, once
// the next tile's O2 is), V once the output, staged over it, is stored.
//
// A barrier's next phase must not complete before each waiter has seen this
// one (two phases look like none).  Each single barrier below has that from the
// order of the steps: its next arrival needs, directly or through another
// barrier, something that every waiter does after its wait.  Scores and P,
// which run a tile ahead, have two.
//
// The kernel starts before the launch before it has ended, and only the state
// warps need that launch's results. The limit of a wait is to measure this
// block's own pipeline, so each role calls wait_before (which has no limit)
// ahead of its first wait that the state warps have a part in; what comes
// earlier, the first loads and the scores and P of a whole first tile, overlaps
// that launch.
//
// A tile's time is the state's chain before HBM: its parts written, O2, the
// second part of K~ (which takes the place of the state's first), D, the state
// read and updated: 7400 cycles for 128 x 128 x 128, with about 750 KB through
// shared memory meanwhile, of which an MMA reads 128 bytes a clock for both
// operands.  K~ is written and multiplied in two halves of the tokens, and its
// first half's second part is made before O2 is done (8000 cycles without).
// 64 wide it is the chain of P and outputs, 4250 cycles.  Measured, of calls of
// 210 and 72 us: 1 x 8 x 65536 x 128 130 us (537 MB, 4.1 TB/s), 4 x 16 x 4096 x
// 64 42 us, the gradient's three runs of 2 x 16 x 8192 x 128 200 us.
template <int DK, int DV>
__global__ void __launch_bounds__(608, 1) decay_tc_out_kernel(const __grid_constant__ DecayTcArgs A) {
  using Cfg = DecayTcCfg<DK, DV>;
  constexpr int C = Cfg::C, NST = Cfg::NST, STAGE = Cfg::STAGE, TK = Cfg::TK, TV = Cfg::TV, NW = Cfg::NW;
  constexpr int NSB = Cfg::NSB;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const uint32_t sbase = smem_u32(smem);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Cfg::BIG);
  uint64_t* full = bars;                // [NST] K and Q landed
  uint64_t* fullv = bars + NST;         // [NST] V landed
  uint64_t* free_qk = bars + 2 * NST;   // [NST] O2 and D complete: Q and K read for the last time, V by D
  uint64_t* empty = bars + 3 * NST;     // [NST] V's slot free: the output has left
  uint64_t* sfull = bars + 4 * NST;     // [2] scores complete
  uint64_t* kready = sfull + 15;        // [2] K~ of the tile's first, of its last 64 tokens written; D before read out
  uint64_t* qdone = sfull + 3;          // O2 complete: Q and the state's parts have been read
  uint64_t* pready = sfull + 13;        // [2] P written over the scores
  uint64_t* dfull = sfull + 5;          // D complete
  uint64_t* wready = sfull + 6;         // the state's parts written
  uint64_t* ofull = sfull + 7;          // O1 complete
  uint64_t* ofree = sfull + 8;          // O1 and O2 read out
  uint64_t* drain = sfull + 9;
  uint64_t* drain2 = sfull + 11;
  uint64_t* cut = sfull + 12;           // rows past the segment's end zeroed in K and V (its last tile, if it has such)
  uint64_t* sread = sfull + 10;         // start state read: the last stage, its buffer, is free
  uint64_t* wfree = sfull + 17;         // [NST] not LSEP: O2 complete that read the state's second part in Q's place there
  float* colp = reinterpret_cast<float*>(bars + 5 * NST + 18);  // [32] gamma^(31-t), reverse gamma^t
  float* diag = colp + 32;                                      // [64] sP gamma^(x-31) at x >= 31
  uint32_t* holder = reinterpret_cast<uint32_t*>(diag + 64);
  int* sh = reinterpret_cast<int*>(holder + 2);                 // [64]

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const DecayGeom& g = A.g;
  const int b = blockIdx.x, ri = b % A.nrun, h = (b / A.nrun) % g.H, s = b / A.nrun / g.H;
  const DecayTcRun& p = A.run[ri];
  const DecaySpan sp = decay_span_block(g, s, sh);
  launch_next();
  if (A.clear) decay_clear_rest(g, A.run[0].op, A.run[0].oh, A.run[0].ot, A.run[0].dv);
  if (sp.seq < 0 || sp.len <= 0) {
    wait_before();
    return;
  }
  const uint64_t lim = A.limit_ns;
  const bool rev = p.rev != 0;
  const int nt = (sp.len + C - 1) / C;
  auto tile_at = [&](int i) { return (rev ? nt - 1 - i : i) * C; };  // first token of the i-th tile walked
  const float l = decay_log(A.log_decay, h);

  if (threadIdx.x == 0) {
    for (int i = 0; i < NST; ++i) {
      mbar_init(&full[i], 2);
      mbar_init(&wfree[i], 1);
      mbar_init(&fullv[i], 1);
      mbar_init(&free_qk[i], 2);
      mbar_init(&empty[i], 1);
    }
    mbar_init(&sfull[0], 1);
    mbar_init(&sfull[1], 1);
    mbar_init(&kready[0], 8);
    mbar_init(&kready[1], 8);
    mbar_init(qdone, 1);
    mbar_init(&pready[0], 8);
    mbar_init(&pready[1], 8);
    mbar_init(dfull, 1);
    mbar_init(wready, 8);
    mbar_init(ofull, 1);
    mbar_init(ofree, 8);
    mbar_init(drain, 1);
    mbar_init(drain2, 1);
    mbar_init(cut, 8);
    mbar_init(sread, 8);
    fence_mbar_init();
  }
  if (threadIdx.x < 32) {
    colp[lane] = expf(l * static_cast<float>(rev ? lane : 31 - lane));
    diag[lane] = lane == 31 ? p.sP : 0.f;
    diag[32 + lane] = p.sP * expf(l * static_cast<float>(lane + 1));
  }
  if (warp == 1) {
    tmem_alloc(holder, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *holder;
  // offset of the state's second part for tile i
  auto second_of = [&](int i) { return Cfg::LSEP ? NST * STAGE + Cfg::WBF : (i + NST - 1) % NST * STAGE; };
  const uint32_t t_o1 = tmem + Cfg::T_O1, t_o2 = tmem + Cfg::T_O2, t_d = tmem + Cfg::T_D;

  if (warp == 0) {
    // ------------------------------------------------------------ loads --
    if (lane == 0) {
      bool dead = false;
      int sent = 0, sentv = 0;
      const uint64_t pol = l2_policy_evict_first();
      for (int i = 0; i < nt; ++i) {
        const int st = i % NST, y = sp.row0 + tile_at(i);
        uint8_t* d = smem + st * STAGE;
        if (i >= NST) decay_wait(dead, &free_qk[st], (i / NST - 1) & 1, lim);
        if (i == NST - 1) {
          wait_before();
          decay_wait(dead, sread, 0, lim);
        }
        if (dead) break;
        mbar_arrive_expect_tx(&full[st], TK);
#pragma unroll
        for (int x = 0; x < DK / 64; ++x)
          tma_load_4d(&A.map[p.k], &full[st], d + TK + x * C * 128, x * 64, y, h, sp.batch, pol);
        sent = i + 1;
        // (the state's second part for tile j lies in stage (j - 1) % NST: j = i - NST + 1, the last one's uses first)
        if (!Cfg::LSEP && i >= NST - 1) decay_wait(dead, &wfree[st], (st == NST - 1 ? i / NST : i / NST - 1) & 1, lim);
        if (dead) {
          mbar_arrive(&full[st]);  // complete when K has landed
          break;
        }
        mbar_arrive_expect_tx(&full[st], TK);
#pragma unroll
        for (int x = 0; x < DK / 64; ++x)
          tma_load_4d(&A.map[p.q], &full[st], d + x * C * 128, x * 64, y, h, sp.batch, pol);
        if (i >= NST) decay_wait(dead, &empty[st], (i / NST - 1) & 1, lim);
        if (dead) break;
        mbar_arrive_expect_tx(&fullv[st], TV);
#pragma unroll
        for (int x = 0; x < DV / 64; ++x)
          tma_load_4d(&A.map[p.v], &fullv[st], d + 2 * TK + x * C * 128, x * 64, y, h, sp.batch, pol);
        sentv = i + 1;
      }
      for (int i = max(0, sent - NST); i < sent; ++i) mbar_wait(&full[i % NST], (i / NST) & 1, lim);
      for (int i = max(0, sentv - NST); i < sentv; ++i) mbar_wait(&fullv[i % NST], (i / NST) & 1, lim);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------- MMAs --
    if (lane == 0) {
      bool dead = false;
      constexpr uint32_t ID_S = idesc_bf16_f32(C, C, false, false), ID_Q = idesc_bf16_f32(C, DV, false, false);
      constexpr uint32_t ID_P = idesc_bf16_f32(C, DV, false, true);
      const uint64_t d_w = sdesc_sw128(sbase + NST * STAGE, 16, 1024);
      auto ragged = [&](int i) { return sp.len - tile_at(i) < C; };
      auto scores = [&](int i) {  // its tile has landed
        if (ragged(i)) decay_wait(dead, cut, 0, lim);
        const uint32_t base = sbase + (i % NST) * STAGE;
        const uint64_t dq = sdesc_sw128(base, 16, 1024), dk = sdesc_sw128(base + TK, 16, 1024);
        tc_fence_after();
        if (!dead) {
#pragma unroll
          for (int kk = 0; kk < DK / 16; ++kk)
            mma_bf16_ss(tmem + (i % NSB) * C, dq + k_step(C, kk), dk + k_step(C, kk), ID_S, kk > 0);
        }
        tc_commit(&sfull[i & 1]);
      };
      decay_wait(dead, &full[0], 0, lim);
      if (ragged(0)) wait_before();
      scores(0);
      wait_before();
      for (int i = 0; i < nt; ++i) {
        const uint32_t base = sbase + (i % NST) * STAGE, par = i & 1;
        const uint64_t dq = sdesc_sw128(base, 16, 1024), dvm = sdesc_sw128(base + 2 * TK, C * 128, 1024);
        const int j = i + 1;
        // the state at tile i: its warps are done with tile i - 1, its scores' barrier among that
        decay_wait(dead, wready, par, lim);
        bool ahead = false;
        if (NSB == 2) {  // (the other score columns were last P of tile i - 1, read by the O1 before)
          ahead = j < nt && !dead && !ragged(j) && mbar_try_wait(smem_u32(&full[j % NST]), (j / NST) & 1);
          if (ahead) scores(j);
        }
        if (i > 0) decay_wait(dead, ofree, (i - 1) & 1, lim);
        tc_fence_after();
        if (!dead) {
#pragma unroll
          for (int kk = 0; kk < DK / 16; ++kk)
            mma_bf16_ss(t_o2, dq + k_step(C, kk), d_w + k_step(DV, kk), ID_Q, kk > 0);
          const uint64_t d_wl = sdesc_sw128(sbase + second_of(i), 16, 1024);
#pragma unroll
          for (int kk = 0; kk < DK / 16; ++kk)
            mma_bf16_ss(t_o2, dq + k_step(C, kk), d_wl + k_step(DV, kk), ID_Q, 1);
        }
        tc_commit(qdone);
        if (!Cfg::LSEP) tc_commit(&wfree[(i + NST - 1) % NST]);
        tc_commit(&free_qk[i % NST]);
        decay_wait(dead, &fullv[i % NST], (i / NST) & 1, lim);
        decay_wait(dead, &pready[par], (i >> 1) & 1, lim);
        tc_fence_after();
        const uint32_t t_p = tmem + (i % NSB) * C;
        if (!dead) {
#pragma unroll
          for (int kk = 0; kk < C / 16; ++kk)
            mma_bf16_ts(t_o1, t_p + 16 * kk + 8, dvm + mn_step(kk), ID_P, kk > 0);
#pragma unroll
          for (int kk = 0; kk < C / 16; ++kk)
            mma_bf16_ts(t_o1, t_p + 16 * kk, dvm + mn_step(kk), ID_P, 1);
        }
        tc_commit(ofull);
        if (j < nt && !ahead) {
          decay_wait(dead, &full[j % NST], (j / NST) & 1, lim);
          scores(j);
        }
      }
      tc_commit(drain);
      mbar_wait(drain, 0, lim);
    }
  } else if (warp == 18) {
    if (lane == 0) {
      bool dead = false;
      constexpr uint32_t ID_D = idesc_bf16_f32(DV, DK, true, true);
      wait_before();
      for (int i = 0; i < nt; ++i) {
        if (i + 1 < nt) {
          const uint32_t base = sbase + (i % NST) * STAGE;
          const uint64_t dkm = sdesc_sw128(base + TK, C * 128, 1024), dvm = sdesc_sw128(base + 2 * TK, C * 128, 1024);
          const uint64_t dlm = sdesc_sw128(sbase + NST * STAGE + (Cfg::LSEP ? 2 * Cfg::WBF : 0), C * 128, 1024);
          decay_wait(dead, &fullv[i % NST], (i / NST) & 1, lim);
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            decay_wait(dead, &kready[y], i & 1, lim);
            tc_fence_after();
            if (!dead) {
#pragma unroll
              for (int kk = y * C / 32; kk < (y + 1) * C / 32; ++kk)
                mma_bf16_ss(t_d, dvm + mn_step(kk), dlm + mn_step(kk), ID_D, kk > 0);
#pragma unroll
              for (int kk = y * C / 32; kk < (y + 1) * C / 32; ++kk)
                mma_bf16_ss(t_d, dvm + mn_step(kk), dkm + mn_step(kk), ID_D, 1);
            }
          }
          tc_commit(dfull);
        }
        tc_commit(&free_qk[i % NST]);
      }
      tc_commit(drain2);
      mbar_wait(drain2, 0, lim);
    }
  } else if (warp < 10) {
    // --------------------------------------------------- P and outputs --
    // Warp (quad, half): rows 32 quad + lane; of P the columns 64 half + [0, 64),
    // of the output DV / 2 columns from half DV / 2.
    bool dead = false;
    const int quad = warp & 3, half = (warp - 2) >> 2, r = quad * 32 + lane;
    const uint32_t lanes = static_cast<uint32_t>(quad * 32) << 16;
    // for each of its two 32-column blocks: how many blocks the rows are past it (0: the diagonal, below 0: zeros),
    // and the row's power to the block's near edge
    int dist[2];
    float edge[2];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      dist[x] = rev ? 2 * half + x - quad : quad - 2 * half - x;
      edge[x] = p.sP * expf(l * static_cast<float>(max(rev ? 32 * dist[x] - lane : lane + 32 * dist[x] - 31, 0)));
    }
    const float read_full = p.sR * expf(l * static_cast<float>(rev ? C - 1 - r : r + 1));
    auto scores_to_p = [&](int i) {
      decay_wait(dead, &sfull[i & 1], (i >> 1) & 1, lim);
      __syncwarp();
      tc_fence_after();
      const uint32_t ts = tmem + lanes + (i % NSB) * C + 64 * half;
      // P's two parts of 16 scores, 8 columns each, go over those scores; the next 16 are read meanwhile.  One loop
      // body for all four: what these warps do for a tile is bound by fetching it, not by its arithmetic (4 x 16 x
      // 4096 x 64: 75 us a call, 78 with two bodies, 91 with four).
      uint32_t x[16], next[16];
      if (dist[0] >= 0) tmem_ld16(ts, next);
#pragma unroll 1
      for (int c = 0; c < 64; c += 16) {
        const int d = c < 32 ? dist[0] : dist[1], t0 = c & 31;
        uint32_t pk[16];
        tmem_ld_wait();
        tmem_ld_done(next);
#pragma unroll
        for (int y = 0; y < 16; ++y) x[y] = next[y];
        if (c < 48 && (c < 16 ? dist[0] : dist[1]) >= 0) tmem_ld16(ts + c + 16, next);
        if (d > 0) {
          const f2 rp = c < 32 ? pair(edge[0], edge[0]) : pair(edge[1], edge[1]);
#pragma unroll
          for (int y = 0; y < 16; y += 4) {
            const float4 cp = *reinterpret_cast<const float4*>(colp + t0 + y);
            split_bf16x2(mul2(mul2(rp, pair(cp.x, cp.y)), pair(x[y], x[y + 1])), pk[y / 2], pk[8 + y / 2]);
            split_bf16x2(mul2(mul2(rp, pair(cp.z, cp.w)), pair(x[y + 2], x[y + 3])), pk[y / 2 + 1], pk[8 + y / 2 + 1]);
          }
        } else if (d == 0) {
          const float* at = rev ? diag + 31 - lane + t0 : diag + 31 + lane - t0;
          const int step = rev ? 1 : -1;
#pragma unroll
          for (int y = 0; y < 16; y += 2)
            split_bf16x2(mul2(pair(at[y * step], at[(y + 1) * step]), pair(x[y], x[y + 1])), pk[y / 2], pk[8 + y / 2]);
        } else {
#pragma unroll
          for (int y = 0; y < 16; ++y) pk[y] = 0u;
        }
        tmem_st16(ts + c, pk);
      }
      tmem_st_wait();
      warp_arrive(&pready[i & 1], lane);
    };
    auto output = [&](int i) {
      const int at = tile_at(i), n = min(C, sp.len - at), y = sp.row0 + at;
      float rp = read_full;
      if (rev && n < C) rp = r < n ? p.sR * expf(l * static_cast<float>(n - 1 - r)) : 0.f;
      const f2 rp2 = pair(rp, rp);
      const uint32_t stage = sbase + (i % NST) * STAGE + 2 * TK;
      // a tile that ends inside the tensor's rows is stored row by row: a box would reach the rows behind
      const bool whole = n == C || y + n == g.T;
      decay_wait(dead, ofull, i & 1, lim);
      decay_wait(dead, &free_qk[i % NST], (i / NST) & 1, lim);
      __syncwarp();
      tc_fence_after();
#pragma unroll(DV == 64 ? 2 : 1)
      for (int x = 0; x < DV / 2; x += 16) {
        const int c0 = half * (DV / 2) + x;
        uint32_t a[16], q[16], pk[8];
        tmem_ld16(t_o1 + lanes + c0, a);
        tmem_ld16(t_o2 + lanes + c0, q);
        tmem_ld_wait();
        if (x + 16 == DV / 2) warp_arrive(ofree, lane);
#pragma unroll
        for (int e = 0; e < 8; ++e)
          pk[e] = pack_bf16x2(fma2(rp2, pair(q[2 * e], q[2 * e + 1]), pair(a[2 * e], a[2 * e + 1])));
        if (whole) {
#pragma unroll
          for (int e = 0; e < 2; ++e)
            st_shared_v4(stage + (c0 >> 6) * C * 128 + sw128_off(r, ((c0 & 63) >> 3) + e), pk[4 * e], pk[4 * e + 1],
                         pk[4 * e + 2], pk[4 * e + 3]);
        } else if (r < n) {
          __nv_bfloat16* out = p.op + static_cast<size_t>(sp.batch) * p.ob + static_cast<size_t>(h) * p.oh +
                               static_cast<size_t>(y + r) * p.ot;
#pragma unroll
          for (int e = 0; e < 2; ++e)
            if (c0 + 8 * e < p.dv)
              *reinterpret_cast<uint4*>(out + c0 + 8 * e) = make_uint4(pk[4 * e], pk[4 * e + 1], pk[4 * e + 2], pk[4 * e + 3]);
        }
      }
      if (whole) {
        fence_async_smem();
        asm volatile("bar.sync 1, 256;" ::: "memory");
        if (threadIdx.x == 2 * 32) {
#pragma unroll
          for (int x = 0; x < (dead ? 0 : DV / 64); ++x)
            tma_store_4d(&A.map[p.o], smem + (i % NST) * STAGE + 2 * TK + x * C * 128, x * 64, y, h, sp.batch);
          bulk_commit();
          bulk_wait_read0();
          mbar_arrive(&empty[i % NST]);
        }
      } else if (threadIdx.x == 2 * 32) {
        mbar_arrive(&empty[i % NST]);
      }
    };
    if (sp.len - tile_at(0) < C) wait_before();
#pragma unroll 1
    for (int i = 0; i < nt + NSB - 1; ++i) {
      if (i < nt) scores_to_p(i);
      if (i == 0) wait_before();
      if (i >= NSB - 1) output(i - (NSB - 1));
    }
    if (threadIdx.x == 2 * 32) bulk_wait0();
  } else {
    // ------------------------------------------------------------ state --
    bool dead = false;
    const int t = static_cast<int>(threadIdx.x) - 320, quad = warp & 3, half = (warp - 10) >> 2;
    int row, col;
    decay_state_at<DK, DV>(quad, half, lane, row, col);
    float w[NW];
    {
      const size_t dd = static_cast<size_t>(p.dk) * p.dv;
      wait_before();  // the scan's states
      const bool via = p.ws && (sp.nseg > 1 || p.ws_all);
      const float* src = via ? p.ws + (static_cast<size_t>(sp.slot) * g.H + h) * dd
                             : p.s_in ? p.s_in + (static_cast<size_t>(sp.seq) * g.H + h) * dd : nullptr;
      const bool tr = via ? p.ws_t != 0 : p.s_in_t != 0;
      if (src) {
        decay_state_in<DK, DV>(reinterpret_cast<float*>(smem + (NST - 1) * STAGE), src, tr, p.dk, p.dv, t, row, col, w);
      } else {
#pragma unroll
        for (int e = 0; e < NW; ++e) w[e] = 0.f;
      }
      fence_async_smem();
      warp_arrive(sread, lane);
      // the state's second part goes over the buffer
      if (!Cfg::LSEP && src) asm volatile("bar.sync 2, 256;" ::: "memory");
    }
    const uint32_t wtile = sbase + NST * STAGE;
    // the state's two bf16 parts as O2 reads them
    auto put_w = [&](uint32_t second) {
#pragma unroll
      for (int e = 0; e < NW; e += 8) {
        const uint32_t at = ((col + e) >> 6) * (DV * 128) + sw128_off(row, ((col + e) & 63) >> 3);
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int y = 0; y < 4; ++y) split_bf16x2(pair(w[e + 2 * y], w[e + 2 * y + 1]), hi[y], lo[y]);
        st_shared_v4(wtile + at, hi[0], hi[1], hi[2], hi[3]);
        st_shared_v4(second + at, lo[0], lo[1], lo[2], lo[3]);
      }
      fence_async_smem();
      warp_arrive(wready, lane);
    };
    float wgt[4];
    auto weights = [&](int n) {
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const int r = (t >> 3) + 32 * x;
        wgt[x] = p.sU * expf(l * static_cast<float>(rev ? r + 1 : max(n - 1 - r, 0)));
      }
    };
    weights(C);
    const float g_full = expf(l * static_cast<float>(C));
    for (int i = 0; i < nt; ++i) {
      const int st = i % NST, n = min(C, sp.len - tile_at(i));
      const bool more = i + 1 < nt;
      put_w(sbase + second_of(i));
      decay_wait(dead, &full[st], (i / NST) & 1, lim);
      uint8_t* d = smem + st * STAGE;
      if (n < C) {
        // what lies behind the segment's end may be anything: with zeros for keys and values it enters no sum, and the
        // scores need no mask there (queries behind the end make rows that are not stored)
        decay_wait(dead, &fullv[st], (i / NST) & 1, lim);
        __syncwarp();
        decay_zero_rows<DK, C>(d + TK, n, t);
        decay_zero_rows<DV, C>(d + 2 * TK, n, t);
        fence_async_smem();
        warp_arrive(cut, lane);
      }
      decay_wait(dead, &sfull[i & 1], (i >> 1) & 1, lim);  // K has been read for the scores
      __syncwarp();
      float gn = g_full;
      if (n < C) {
        weights(n);
        gn = expf(l * static_cast<float>(n));
      }
      if (!more) break;
      // 64 tokens at a time, so that D starts on the first of them; without a place of its own K~'s second part of
      // those waits in registers for the state's first part to have been read
#pragma unroll(Cfg::LSEP ? 1 : 2)
      for (int y = 0; y < 2; ++y) {
        uint4 lo[DK / 32];
        decay_scale_half<DK, C>(d + TK, t, y, y ? wgt[2] : wgt[0], y ? wgt[3] : wgt[1], lo);
        if (!Cfg::LSEP && y == 0) {
          decay_wait(dead, qdone, i & 1, lim);
          __syncwarp();
        }
        decay_store_half<DK, C>(smem + NST * STAGE + (Cfg::LSEP ? 2 * Cfg::WBF : 0), t, y, lo);
        fence_async_smem();
        warp_arrive(&kready[y], lane);
      }
      if (n < C) weights(C);
      decay_wait(dead, dfull, i & 1, lim);
      __syncwarp();
      tc_fence_after();
      constexpr int PIECE = DV == 128 ? 16 : NW;
#pragma unroll
      for (int x = 0; x < NW; x += PIECE) {
        uint32_t y[PIECE];
        decay_state_ld<DK, DV>(t_d, quad, half, x, y);
        tmem_ld_wait();
#pragma unroll
        for (int e = 0; e < PIECE; ++e) w[x + e] = fmaf(gn, w[x + e], __uint_as_float(y[e]));
      }
      if (Cfg::LSEP) {
        decay_wait(dead, qdone, i & 1, lim);  // the state's parts have been read
        __syncwarp();
      }
    }
    tc_fence_before();
  }
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

}  // namespace ttt
