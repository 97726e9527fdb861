// group_norm.cuh -- group norm over channels-last data with a silu, or a gate,
// in its epilogue, and its gradient.
//
// x is [N, L, C]: N samples of L positions of C channels, G groups of
// cg = C / G adjacent channels.  Per (sample, group), over its L cg values:
//   mean, rstd = 1 / sqrt(var + eps) ;  hat = (x - mean) rstd ;  t = hat w + b
//   y = act(t)  or, with a gate,  y = t act(gate) ,   act = silu or identity.
// The norm of every head's output of the layer is L = 1 (one token a sample),
// G = heads.
//
// Gradient, with dt = dL/dt and dh = dt w, the means over the (sample, group):
//   dx = rstd (dh - mean(dh) - hat mean(dh hat)) ,  dw = sum dt hat ,  db = sum dt.
//
// All of it is bound by memory: values come in 16-byte units through a ring of
// bulk copies (below), and the statistics are taken in fp32 from registers, mean
// first and then squares around it (of a channel over a batch of positions;
// batches, channels, threads and blocks are joined by the exact two-set
// formula), so a mean far from zero costs no digits.  Every sum has a fixed
// order: the same call gives the same bits.
#pragma once
#include <type_traits>

#include "common.cuh"

namespace ttt {

// V consecutive values of T as pairs of floats: 16 bytes, or one value (its
// pair's other half is 0) where rows do not start on 16 bytes.
template <typename T, int V>
struct Unit {
  static constexpr int P = V > 1 ? V / 2 : 1;
  f2 v[P];
};
template <typename T, int V>
__device__ __forceinline__ void st_unit(T* p, const Unit<T, V>& x) {
  if constexpr (V == 1) {
    *p = from_f<T>(lo_of(x.v[0]));
  } else if constexpr (sizeof(T) == 2) {
    *reinterpret_cast<uint4*>(p) =
        make_uint4(pack_bf16x2(x.v[0]), pack_bf16x2(x.v[1]), pack_bf16x2(x.v[2]), pack_bf16x2(x.v[3]));
  } else {
    *reinterpret_cast<float4*>(p) = make_float4(lo_of(x.v[0]), hi_of(x.v[0]), lo_of(x.v[1]), hi_of(x.v[1]));
  }
}
// A bulk copy's units as they lie in shared memory.
template <typename T, int V>
__device__ __forceinline__ Unit<T, V> unit_of(const uint4 u) {
  Unit<T, V> r;
  if constexpr (sizeof(T) == 2) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) r.v[i] = pair(w[i] << 16, w[i] & 0xffff0000u);
  } else {
    r.v[0] = pair(u.x, u.y);
    r.v[1] = pair(u.z, u.w);
  }
  return r;
}
// The same from memory, or one value.
template <typename T, int V>
__device__ __forceinline__ Unit<T, V> ld_unit(const T* p) {
  if constexpr (V == 1) {
    Unit<T, V> r;
    r.v[0] = pair(to_f<T>(__ldg(p)), 0.f);
    return r;
  } else {
    return unit_of<T, V>(__ldg(reinterpret_cast<const uint4*>(p)));
  }
}
__device__ __forceinline__ f2 both(float x) { return pair(x, x); }
__device__ __forceinline__ float sum_of(f2 x) { return lo_of(x) + hi_of(x); }

struct GnParams {
  int N, L, C, G, cg;
  const void *x, *gate;
  const void *weight, *bias;  // [C] or nullptr
  int pbf;                    // weight and bias are bf16 (else fp32)
  float eps;
  void* y;
  float *mean, *rstd;         // [N][G]
  float* part;                // partial statistics
  int splits, rows;           // parts of a sample for the statistics and the gradient's sums, positions in each
  int parts, part_rows;       // the same for the passes that write y or dx
  int width, slots;           // one-position kernels: units of a row in a block, rows at a time
  int per;                    // of those: rows in a block
  uint64_t limit_ns;
  // gradient
  const void* gy;
  void *gx, *ggate;
  void *gw, *gb;              // [C] or nullptr
};

__device__ __forceinline__ float gn_param(const void* p, int pbf, int c, float none) {
  if (!p) return none;
  return pbf ? __bfloat162float(__ldg(static_cast<const __nv_bfloat16*>(p) + c)) : __ldg(static_cast<const float*>(p) + c);
}
// 1 / (1 + exp(-x)): the approximate exponential and reciprocal are off by a
// few steps and the rounded exponent by |x| of them relative to the result, which
// falls off faster where x is negative: silu is off by a few 2^-24 at most, its
// slope too.  Below x = -87, where the result passes 2^-126, it is 0.
__device__ __forceinline__ float gn_sigmoid1(float e) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(e));
  return r;
}
__device__ __forceinline__ f2 gn_sigmoid(f2 x) {
  const f2 e = mul2(x, both(-1.4426950408889634f));
  const f2 d = add2(pair(gn_sigmoid1(lo_of(e)), gn_sigmoid1(hi_of(e))), both(1.f));
  float a, b;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(a) : "f"(lo_of(d)));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(b) : "f"(hi_of(d)));
  return pair(a, b);
}

// y of two values; ACT: silu, else identity.
template <bool GATE, bool ACT>
__device__ __forceinline__ f2 gn_out(f2 t, f2 z) {
  if constexpr (GATE) return mul2(t, ACT ? mul2(z, gn_sigmoid(z)) : z);
  return ACT ? mul2(t, gn_sigmoid(t)) : t;
}
// dL/dt of two values; dz: dL/dgate.  silu(z) = z s, silu'(z) = s + z s (1 - s).
template <bool GATE, bool ACT>
__device__ __forceinline__ f2 gn_grad(f2 g, f2 t, f2 z, f2& dz) {
  if constexpr (GATE) {
    if constexpr (!ACT) {
      dz = mul2(g, t);
      return mul2(g, z);
    }
    const f2 s = gn_sigmoid(z), zs = mul2(z, s);
    dz = mul2(mul2(g, t), fma2(zs, fma2(s, both(-1.f), both(1.f)), s));
    return mul2(g, zs);
  }
  dz = both(0.f);
  if constexpr (!ACT) return g;
  const f2 s = gn_sigmoid(t);
  return mul2(g, fma2(mul2(t, s), fma2(s, both(-1.f), both(1.f)), s));
}

// Count, mean and variance; joined exactly.  The variance instead of the sum of
// squares, and the means' distance weighted before it is squared: neither
// passes the largest number before the variance itself does.  (With nothing on
// one side that distance is the other's mean.)
struct Moments {
  float n, mean, var;
};
__device__ __forceinline__ Moments join(const Moments& a, const Moments& b) {
  const float n = a.n + b.n;
  if (n == 0.f) return a;
  const float r = __fdividef(1.f, n), f = b.n * r, d = b.mean - a.mean;  // (counts: far from the division's limits)
  return Moments{n, fmaf(d, f, a.mean), fmaf(d * (f * (a.n * r)), d, fmaf(f, b.var - a.var, a.var))};
}
__device__ __forceinline__ Moments shfl_xor(const Moments& a, int off) {
  return Moments{__shfl_xor_sync(0xffffffffu, a.n, off), __shfl_xor_sync(0xffffffffu, a.mean, off),
                 __shfl_xor_sync(0xffffffffu, a.var, off)};
}

// A variance past the largest number is infinite or, joined on, NaN, and stays
// so: beside a mean that is a number rstd is 0 then, as of an infinite variance.
__device__ __forceinline__ float gn_rstd(float mean, float var, float eps) {
  return isnan(var) && isfinite(mean) ? 0.f : rsqrtf(var + eps);
}

// Walks rows of C values in memory, `slots` rows at a time, a thread one unit of
// each: thread slot * units + u has unit u of row `slot`.  What a step reads of
// the block's units is contiguous (narrow rows are held whole, a wide one
// alone), so it is one bulk copy (cp.async.bulk) of up to 4 KB a tensor into a
// ring of S steps, issued S steps ahead by one thread: memory stays busy
// without registers or occupancy.  Measured (gated rows 16384 x 2048 bf16): 55
// us with two rows of plain loads a thread, 46 us with the ring, 50 us with
// steps of two rows a thread; their gradient 114, 76 and 100 us.
// Waits are bounded; after one runs out nothing more is copied or waited for.
constexpr int kGnStage = 4096, kGnRingBytes = 12 * kGnStage;
template <int NT>
struct GnRing {
  static constexpr int S = 12 / NT;
  uint8_t* buf;       // [S][NT][4096]
  uint64_t* full;     // [S]
  uint64_t limit_ns;
  int used;           // steps so far
  bool dead;

  __device__ __forceinline__ void init(uint8_t* smem, uint64_t* bars, uint64_t limit) {
    buf = smem, full = bars, limit_ns = limit, used = 0, dead = false;
    if (threadIdx.x == 0) {
      for (int i = 0; i < S; ++i) mbar_init(&full[i], 1);
      fence_mbar_init();
    }
    __syncthreads();
  }

  // f(row, units[NT], ok) for this thread's rows of every step, by all threads.
  // src: row 0's first unit of the block's; `units`: the block's of a row.
  template <typename T, int V, typename F>
  __device__ __forceinline__ void walk(const T* const (&src)[NT], int rows, int C, int units, int slots, F&& f) {
    const int tid = threadIdx.x, slot = tid / units, u = tid % units;
    const bool on = slot < slots;
    if constexpr (V == 1) {  // rows at any address: plain loads
      const int steps = (rows + slots - 1) / slots;
      for (int k = 0; k < steps; ++k) {
        const int row = k * slots + slot;
        const bool ok = on && row < rows;
        Unit<T, V> x[NT];
#pragma unroll
        for (int i = 0; i < NT; ++i)
          x[i].v[0] = pair(ok ? to_f<T>(__ldg(src[i] + static_cast<size_t>(row) * C + u)) : 0.f, 0.f);
        f(row, x, ok);
      }
    } else {
      const int steps = (rows + slots - 1) / slots;
      auto issue = [&](int k) {
        const int st = (used + k) % S, n = min(slots, rows - k * slots);
        const uint32_t bytes = static_cast<uint32_t>(n * units) * 16u;
        mbar_arrive_expect_tx(&full[st], bytes * NT);
#pragma unroll
        for (int i = 0; i < NT; ++i)
          bulk_load(buf + (st * NT + i) * kGnStage, src[i] + static_cast<size_t>(k) * slots * C, bytes, &full[st]);
      };
      int sent = 0;
      if (tid == 0 && !dead)
        for (; sent < min(S, steps); ++sent) issue(sent);
      for (int k = 0; k < steps; ++k) {
        const int st = (used + k) % S;
        if (!dead) dead = !mbar_wait_suspended(&full[st], ((used + k) / S) & 1, limit_ns);
        uint4 raw[NT];
#pragma unroll
        for (int i = 0; i < NT; ++i) raw[i] = ld_shared_v4(smem_u32(buf) + (st * NT + i) * kGnStage + tid * 16);
        // read by all, the reads ordered before the copy into the same place S steps later
        fence_async_smem();
        __syncthreads();
        if (tid == 0 && !dead && sent < steps) issue(sent++);
        const int row = k * slots + slot;
        Unit<T, V> x[NT];
#pragma unroll
        for (int i = 0; i < NT; ++i) x[i] = unit_of<T, V>(raw[i]);
        f(row, x, on && row < rows);
      }
      if (dead && tid == 0)  // what is still on its way lands before the block ends
        for (int k = max(0, sent - S); k < sent; ++k) mbar_wait(&full[(used + k) % S], ((used + k) / S) & 1, limit_ns);
      used += steps;
    }
  }
};

// weight and bias of V channels from c.
template <int V>
struct GnParam {
  static constexpr int P = V > 1 ? V / 2 : 1;
  f2 w[P], b[P];
  __device__ __forceinline__ GnParam(const GnParams& p, int c, bool on) {
    float x[2 * P], y[2 * P];
#pragma unroll
    for (int e = 0; e < 2 * P; ++e) {
      const bool has = on && (V > 1 || e == 0);
      x[e] = has ? gn_param(p.weight, p.pbf, c + e, 1.f) : 1.f;
      y[e] = has ? gn_param(p.bias, p.pbf, c + e, 0.f) : 0.f;
    }
#pragma unroll
    for (int e = 0; e < P; ++e) {
      w[e] = pair(x[2 * e], x[2 * e + 1]);
      b[e] = pair(y[2 * e], y[2 * e + 1]);
    }
  }
};

// ------------------------------------------------- one position a sample ----
// L = 1 and a group of 1, 2, 4 .. 32 units: the lanes of a group hold it in
// registers, one unit a thread, so the values are read once.  A thread keeps
// its channels over all its rows, with weight and bias in registers.  Block
// (x, y): units [x width, (x + 1) width) of rows [y per, (y + 1) per).
// 16384 x 2048 bf16 gated: 44 us (201 MB, 4.6 TB/s), bound by instruction issue.
template <typename T, int V, bool GATE, bool ACT>
__global__ void __launch_bounds__(256, 4) gn_row_kernel(const GnParams p, int lanes) {
  constexpr int P = V / 2, NT = GATE ? 2 : 1;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(8) uint64_t bars[12];
  const int tid = threadIdx.x, u0 = blockIdx.x * p.width, units = min(p.width, p.C / V - u0);
  const int row0 = blockIdx.y * p.per, rows = min(p.per, p.N - row0);
  const bool on = tid < units * p.slots;
  const int c = (u0 + (on ? tid % units : 0)) * V, g = c / p.cg;
  const GnParam<V> par(p, c, on);
  const float inv = 1.f / static_cast<float>(p.cg);
  const bool first = c % p.cg == 0;
  const size_t base = static_cast<size_t>(row0) * p.C;
  T* yp = static_cast<T*>(p.y) + base + c;
  float *mp = p.mean + static_cast<size_t>(row0) * p.G + g, *rp = p.rstd + static_cast<size_t>(row0) * p.G + g;
  GnRing<NT> ring;
  ring.init(smem, bars, p.limit_ns);
  const T* src[NT];
  src[0] = static_cast<const T*>(p.x) + base + u0 * V;
  if constexpr (GATE) src[1] = static_cast<const T*>(p.gate) + base + u0 * V;
  ring.template walk<T, V>(src, rows, p.C, units, p.slots, [&](int row, Unit<T, V>(&in)[NT], bool ok) {
    Unit<T, V>& x = in[0];
    f2 s = x.v[0];
#pragma unroll
    for (int e = 1; e < P; ++e) s = add2(s, x.v[e]);
    float mean = sum_of(s);
    for (int off = lanes >> 1; off > 0; off >>= 1) mean += __shfl_xor_sync(0xffffffffu, mean, off);
    mean *= inv;
    s = both(0.f);
#pragma unroll
    for (int e = 0; e < P; ++e) {
      x.v[e] = add2(x.v[e], both(-mean));
      s = fma2(x.v[e], x.v[e], s);
    }
    float q = sum_of(s);
    for (int off = lanes >> 1; off > 0; off >>= 1) q += __shfl_xor_sync(0xffffffffu, q, off);
    if (!ok) return;
    const float rstd = rsqrtf(fmaf(q, inv, p.eps));
    Unit<T, V> y;
#pragma unroll
    for (int e = 0; e < P; ++e)
      y.v[e] = gn_out<GATE, ACT>(fma2(mul2(x.v[e], both(rstd)), par.w[e], par.b[e]), in[NT - 1].v[e]);
    st_unit<T, V>(yp + static_cast<size_t>(row) * p.C, y);
    if (first) {
      mp[static_cast<size_t>(row) * p.G] = mean;
      rp[static_cast<size_t>(row) * p.G] = rstd;
    }
  });
}

// Its gradient: dw and db gather in registers over the thread's rows; the
// block's sums go to part[2][gridDim.y][C].  The same rows: 69 us (336 MB, 4.9
// TB/s) and 8 for the parameters' sums.
template <typename T, int V, bool GATE, bool ACT>
__global__ void __launch_bounds__(256, 3) gn_row_grad_kernel(const GnParams p, int lanes) {
  constexpr int P = V / 2, NT = GATE ? 3 : 2;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(8) uint64_t bars[12];
  __shared__ float red[2][256][V + 1];
  const int tid = threadIdx.x, u0 = blockIdx.x * p.width, units = min(p.width, p.C / V - u0);
  const int row0 = blockIdx.y * p.per, rows = min(p.per, p.N - row0);
  const bool on = tid < units * p.slots;
  const int c = (u0 + (on ? tid % units : 0)) * V, g = c / p.cg;
  const GnParam<V> par(p, c, on);
  f2 dw[P], db[P];
#pragma unroll
  for (int e = 0; e < P; ++e) dw[e] = db[e] = both(0.f);
  const float inv = 1.f / static_cast<float>(p.cg);
  const size_t base = static_cast<size_t>(row0) * p.C;
  T *gxp = static_cast<T*>(p.gx) + base + c, *gzp = static_cast<T*>(p.ggate) + base + c;
  const float *mp = p.mean + static_cast<size_t>(row0) * p.G + g, *rp = p.rstd + static_cast<size_t>(row0) * p.G + g;
  // the next row's statistics, a step ahead
  auto stat = [&](const float* q, int row) { return on && row < rows ? __ldg(q + static_cast<size_t>(row) * p.G) : 0.f; };
  float mean = stat(mp, tid / units), rstd = stat(rp, tid / units);
  launch_next();
  GnRing<NT> ring;
  ring.init(smem, bars, p.limit_ns);
  const T* src[NT];
  src[0] = static_cast<const T*>(p.x) + base + u0 * V;
  src[1] = static_cast<const T*>(p.gy) + base + u0 * V;
  if constexpr (GATE) src[2] = static_cast<const T*>(p.gate) + base + u0 * V;
  ring.template walk<T, V>(src, rows, p.C, units, p.slots, [&](int row, Unit<T, V>(&in)[NT], bool ok) {
    const f2 m2 = both(-mean), r2 = both(rstd);
    mean = stat(mp, row + p.slots), rstd = stat(rp, row + p.slots);
    Unit<T, V> dz;
    f2 a = both(0.f), b = both(0.f);
#pragma unroll
    for (int e = 0; e < P; ++e) {
      const f2 hat = mul2(add2(in[0].v[e], m2), r2);
      f2 dt = gn_grad<GATE, ACT>(in[1].v[e], fma2(hat, par.w[e], par.b[e]), in[NT - 1].v[e], dz.v[e]);
      if (!ok) dt = both(0.f);
      dw[e] = fma2(dt, ok ? hat : both(0.f), dw[e]);
      db[e] = add2(db[e], dt);
      in[0].v[e] = hat;
      in[1].v[e] = mul2(dt, par.w[e]);
      a = add2(a, in[1].v[e]);
      b = fma2(in[1].v[e], hat, b);
    }
    float s1 = sum_of(a), s2 = sum_of(b);
    for (int off = lanes >> 1; off > 0; off >>= 1) {
      s1 += __shfl_xor_sync(0xffffffffu, s1, off);
      s2 += __shfl_xor_sync(0xffffffffu, s2, off);
    }
    if (!ok) return;
    if constexpr (GATE) st_unit<T, V>(gzp + static_cast<size_t>(row) * p.C, dz);
    Unit<T, V> dx;
#pragma unroll
    for (int e = 0; e < P; ++e)
      dx.v[e] = mul2(r2, fma2(in[0].v[e], both(-s2 * inv), add2(in[1].v[e], both(-s1 * inv))));
    st_unit<T, V>(gxp + static_cast<size_t>(row) * p.C, dx);
  });
  if (!p.part) return;
#pragma unroll
  for (int e = 0; e < P; ++e) {
    red[0][tid][2 * e] = lo_of(dw[e]);
    red[0][tid][2 * e + 1] = hi_of(dw[e]);
    red[1][tid][2 * e] = lo_of(db[e]);
    red[1][tid][2 * e + 1] = hi_of(db[e]);
  }
  __syncthreads();
  for (int i = tid; i < 2 * units * V; i += blockDim.x) {
    const int which = i / (units * V), ch = i % (units * V), un = ch / V, e = ch % V;
    float s = 0.f;
    for (int k = 0; k < p.slots; ++k) s += red[which][k * units + un][e];
    p.part[(static_cast<size_t>(which) * gridDim.y + blockIdx.y) * p.C + u0 * V + ch] = s;
  }
}

// dw (which = 0) or db (1) of channels 32 b .. 32 b + 31: the sum of `count`
// rows of part[2][count][C] in a fixed order, eight strands over the block's
// warps, each with eight loads in flight.
__device__ __forceinline__ void gn_param_sum(const float* __restrict__ part, int count, int C, void* dst, int pbf, int b,
                                             int which) {
  __shared__ float red[8][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = b * 32 + lane;
  float s = 0.f;
  if (c < C) {
    const float* at = part + static_cast<size_t>(which) * count * C + c;
    for (int k = warp; k < count; k += 64) {
      float t[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) t[i] = ld_after(at + static_cast<size_t>(min(k + 8 * i, count - 1)) * C);
#pragma unroll
      for (int i = 0; i < 8; ++i) s += k + 8 * i < count ? t[i] : 0.f;
    }
  }
  red[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && c < C && dst) {
    float t = 0.f;
    for (int k = 0; k < 8; ++k) t += red[k][lane];
    if (pbf)
      static_cast<__nv_bfloat16*>(dst)[c] = __float2bfloat16_rn(t);
    else
      static_cast<float*>(dst)[c] = t;
  }
}
__global__ void __launch_bounds__(256) gn_param_grad_kernel(const float* __restrict__ part, int count, int C, void* gw,
                                                            void* gb, int pbf) {
  wait_before();
  gn_param_sum(part, count, C, blockIdx.y ? gb : gw, pbf, blockIdx.x, blockIdx.y);
}

// ------------------------------------------------------ any L and width ----
// A thread keeps one unit of channels (whose channels may lie in two groups)
// and walks positions: rows [k rows, (k + 1) rows) of a sample are part k.
// (L may be 2^31 - 1: a position with a step past the last one is unsigned.)
__device__ __forceinline__ void gn_rows(int L, int rows, int k, int& l0, int& l1) {
  l0 = static_cast<int>(min(static_cast<long long>(L), static_cast<long long>(k) * rows));
  l1 = static_cast<int>(min(static_cast<long long>(L), static_cast<long long>(l0) + rows));
}

// Statistics of one split of one sample: part[N][splits][G] of (mean, variance), or,
// where a sample is one split, mean and rstd.  Plain loads, a batch of eight
// positions in flight a thread (6 x 4225 x 320 fp32: 15 us cold, of a call of 30
// to 34; through the ring, whose steps cost a barrier, 18).  Dynamic shared memory: G Moments.
template <typename T, int V>
__global__ void __launch_bounds__(256, 3) gn_stats_kernel(const GnParams p) {
  constexpr int P = Unit<T, V>::P, U = 8;  // U: positions in a batch
  extern __shared__ __align__(16) uint8_t smem[];
  Moments* group = reinterpret_cast<Moments*>(smem);  // [G]
  __shared__ float each[2][256][V + 1];
  __shared__ float counts[256];
  const int tid = threadIdx.x, n = blockIdx.x / p.splits, part = blockIdx.x % p.splits, cv = p.C / V;
  int l0, l1;
  gn_rows(p.L, p.rows, part, l0, l1);
  for (int g = tid; g < p.G; g += 256) group[g] = Moments{0.f, 0.f, 0.f};
  const T* x = static_cast<const T*>(p.x) + static_cast<size_t>(n) * p.L * p.C;
  launch_next();
  for (int u0 = 0; u0 < cv; u0 += 256) {
    const int width = min(cv - u0, 256), slots = cv > 256 ? 1 : 256 / width, slot = tid / width;
    float cnt = 0.f;
    f2 mean[P], var[P];
#pragma unroll
    for (int e = 0; e < P; ++e) mean[e] = var[e] = both(0.f);
    // `have` units from l: their sums relative to the first, joined to the mean and variance so far
    auto batch = [&](unsigned l, int have, bool all) {
      using Raw = std::conditional_t<V == 1, T, uint4>;
      const T* at = x + static_cast<size_t>(l) * p.C + (u0 + tid % width) * V;
      const size_t step = static_cast<size_t>(slots) * p.C;
      Raw raw[U];
#pragma unroll
      for (int i = 0; i < U; ++i)
        if (all || i < have) raw[i] = __ldg(reinterpret_cast<const Raw*>(at + i * step));
      auto unit = [&](int i) {
        if constexpr (V == 1) {
          Unit<T, V> r;
          r.v[0] = pair(to_f<T>(raw[i]), 0.f);
          return r;
        } else {
          return unit_of<T, V>(raw[i]);
        }
      };
      const Unit<T, V> first = unit(0);
      f2 s[P], q[P];
#pragma unroll
      for (int e = 0; e < P; ++e) s[e] = q[e] = both(0.f);
#pragma unroll
      for (int i = 1; i < U; ++i)
        if (all || i < have) {
          const Unit<T, V> y = unit(i);
#pragma unroll
          for (int e = 0; e < P; ++e) {
            const f2 d = fma2(first.v[e], both(-1.f), y.v[e]);
            s[e] = add2(s[e], d);
            q[e] = fma2(d, d, q[e]);
          }
        }
      const float h = static_cast<float>(have), inv = all ? 1.f / U : __fdividef(1.f, h), r = __fdividef(1.f, cnt + h);
      const float f = h * r, cf = f * (cnt * r);
#pragma unroll
      for (int e = 0; e < P; ++e) {
        const f2 d0 = mul2(s[e], both(inv));  // the batch's mean - its first value
        const f2 more = fma2(fma2(mul2(s[e], both(-1.f)), d0, q[e]), both(inv), mul2(var[e], both(-1.f)));
        const f2 d = fma2(mean[e], both(-1.f), add2(first.v[e], d0));
        mean[e] = fma2(d, both(f), mean[e]);
        var[e] = add2(fma2(more, both(f), var[e]), mul2(mul2(d, both(cf)), d));
      }
      cnt += h;
    };
    if (slot < slots) {
      unsigned l = static_cast<unsigned>(l0) + slot;
      const unsigned end = l1;
      for (; l + (U - 1) * slots < end; l += U * slots) batch(l, U, true);
      if (l < end) batch(l, (end - l - 1) / slots + 1, false);
    }
    __syncthreads();
    counts[tid] = cnt;
#pragma unroll
    for (int e = 0; e < V; ++e) {
      each[0][tid][e] = e & 1 ? hi_of(mean[e / 2]) : lo_of(mean[e / 2]);
      each[1][tid][e] = e & 1 ? hi_of(var[e / 2]) : lo_of(var[e / 2]);
    }
    __syncthreads();
    // a warp for each group that these channels touch
    const int c0 = u0 * V, c1 = c0 + width * V, g0 = c0 / p.cg, g1 = (c1 - 1) / p.cg;
    for (int g = g0 + (tid >> 5); g <= g1; g += 8) {
      const int a = max(g * p.cg, c0) - c0, w = min((g + 1) * p.cg, c1) - c0 - a;  // its channels here
      Moments t{0.f, 0.f, 0.f};
      for (int i = tid & 31; i < slots * w; i += 32) {
        const int k = i / w, ch = a + i % w, at = k * width + ch / V;
        t = join(t, Moments{counts[at], each[0][at][ch % V], each[1][at][ch % V]});
      }
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) t = join(t, shfl_xor(t, off));
      if ((tid & 31) == 0) group[g] = join(group[g], t);
    }
  }
  __syncthreads();
  for (int g = tid; g < p.G; g += 256) {
    if (p.splits == 1) {
      const size_t at = static_cast<size_t>(n) * p.G + g;
      p.mean[at] = group[g].mean;
      p.rstd[at] = gn_rstd(group[g].mean, group[g].var, p.eps);
    } else {
      float2* d = reinterpret_cast<float2*>(p.part) + (static_cast<size_t>(n) * p.splits + part) * p.G + g;
      *d = make_float2(group[g].mean, group[g].var);
    }
  }
}

// mean and rstd from the splits' statistics, a warp per (sample, group).
__global__ void __launch_bounds__(256) gn_join_kernel(const GnParams p) {
  const long long i = (static_cast<long long>(blockIdx.x) * 256 + threadIdx.x) >> 5;
  launch_next();
  wait_before();
  if (i >= static_cast<long long>(p.N) * p.G) return;
  const long long n = i / p.G;
  const int g = static_cast<int>(i % p.G);
  const float2* d = reinterpret_cast<const float2*>(p.part) + n * p.splits * p.G + g;
  Moments m{0.f, 0.f, 0.f};
  for (int k0 = threadIdx.x & 31; k0 < p.splits; k0 += 128) {
    float2 x[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (k0 + 32 * j < p.splits) x[j] = ld_after(d + static_cast<size_t>(k0 + 32 * j) * p.G);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      int a, b;
      gn_rows(p.L, p.rows, k0 + 32 * j, a, b);
      if (b > a) m = join(m, Moments{static_cast<float>(b - a) * static_cast<float>(p.cg), x[j].x, x[j].y});
    }
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) m = join(m, shfl_xor(m, off));
  if ((threadIdx.x & 31) == 0) {
    p.mean[i] = m.mean;
    p.rstd[i] = gn_rstd(m.mean, m.var, p.eps);
  }
}

// A sample's statistics for V channels from c, whose groups may differ.
template <int V>
struct GnStat {
  static constexpr int P = V > 1 ? V / 2 : 1;
  f2 v[P];
  __device__ __forceinline__ GnStat(const float* s, int stride, int c, int cg) {
#pragma unroll
    for (int e = 0; e < P; ++e)
      v[e] = pair(ld_after(s + stride * ((c + 2 * e) / cg)), V > 1 ? ld_after(s + stride * ((c + 2 * e + 1) / cg)) : 0.f);
  }
};

// y from mean and rstd.  x is in L2 from the statistics where it fits, and a
// step's work is small: plain loads, four in flight a thread (measured, 6 x
// 4225 x 320 fp32: 12 us; through the ring, whose steps cost a barrier, 18).
template <typename T, int V, bool GATE, bool ACT>
__global__ void __launch_bounds__(256) gn_apply_kernel(const GnParams p) {
  constexpr int P = Unit<T, V>::P;
  const int tid = threadIdx.x, n = blockIdx.x / p.parts, part = blockIdx.x % p.parts, cv = p.C / V;
  int l0, l1;
  gn_rows(p.L, p.part_rows, part, l0, l1);
  const size_t base = static_cast<size_t>(n) * p.L * p.C;
  wait_before();
  for (int u0 = 0; u0 < cv; u0 += 256) {
    const int width = min(cv - u0, 256), slots = 256 / width, slot = tid / width, u = u0 + tid % width;
    if (slot >= slots) continue;
    const int c = u * V;
    GnParam<V> par(p, c, true);  // t = (x - mean) w + b, rstd in w
    const GnStat<V> mean(p.mean + static_cast<size_t>(n) * p.G, 1, c, p.cg), rstd(p.rstd + static_cast<size_t>(n) * p.G, 1, c, p.cg);
    f2 neg[P];
#pragma unroll
    for (int e = 0; e < P; ++e) {
      neg[e] = mul2(mean.v[e], both(-1.f));
      par.w[e] = mul2(par.w[e], rstd.v[e]);
    }
#pragma unroll 4
    for (unsigned l = static_cast<unsigned>(l0) + slot; l < static_cast<unsigned>(l1); l += slots) {
      const size_t at = base + static_cast<size_t>(l) * p.C + c;
      const Unit<T, V> x = ld_unit<T, V>(static_cast<const T*>(p.x) + at);
      Unit<T, V> z = x, y;
      if constexpr (GATE) z = ld_unit<T, V>(static_cast<const T*>(p.gate) + at);
#pragma unroll
      for (int e = 0; e < P; ++e) y.v[e] = gn_out<GATE, ACT>(fma2(add2(x.v[e], neg[e]), par.w[e], par.b[e]), z.v[e]);
      st_unit<T, V>(static_cast<T*>(p.y) + at, y);
    }
  }
}

// Gradient, first pass: part[2][N][splits][C], the sums of dt hat and of dt
// over a split's positions; also dgate.  8 x 4096 x 512 bf16: 27 us, the third
// pass as long.
template <typename T, int V, bool GATE, bool ACT>
__global__ void __launch_bounds__(256, 3) gn_grad_sums_kernel(const GnParams p) {
  constexpr int P = Unit<T, V>::P, NT = GATE ? 3 : 2;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(8) uint64_t bars[12];
  __shared__ float red[2][256][V + 1];
  const int tid = threadIdx.x, n = blockIdx.x / p.splits, part = blockIdx.x % p.splits, cv = p.C / V;
  int l0, l1;
  gn_rows(p.L, p.rows, part, l0, l1);
  const size_t base = (static_cast<size_t>(n) * p.L + l0) * p.C, all = static_cast<size_t>(p.N) * p.splits * p.C;
  launch_next();
  GnRing<NT> ring;
  ring.init(smem, bars, p.limit_ns);
  for (int u0 = 0; u0 < cv; u0 += 256) {
    const int width = min(cv - u0, 256), slots = cv > 256 ? 1 : 256 / width, c = (u0 + tid % width) * V;
    f2 dw[P], db[P];
#pragma unroll
    for (int e = 0; e < P; ++e) dw[e] = db[e] = both(0.f);
    const GnParam<V> par(p, c, true);
    const GnStat<V> mean(p.mean + static_cast<size_t>(n) * p.G, 1, c, p.cg), rstd(p.rstd + static_cast<size_t>(n) * p.G, 1, c, p.cg);
    const T* src[NT];
    src[0] = static_cast<const T*>(p.x) + base + u0 * V;
    src[1] = static_cast<const T*>(p.gy) + base + u0 * V;
    if constexpr (GATE) src[2] = static_cast<const T*>(p.gate) + base + u0 * V;
    T* gzp = static_cast<T*>(p.ggate) + base + c;
    ring.template walk<T, V>(src, l1 - l0, p.C, width, slots, [&](int row, Unit<T, V>(&in)[NT], bool ok) {
      if (!ok) return;
      Unit<T, V> dz;
#pragma unroll
      for (int e = 0; e < P; ++e) {
        const f2 hat = mul2(fma2(mean.v[e], both(-1.f), in[0].v[e]), rstd.v[e]);
        const f2 dt = gn_grad<GATE, ACT>(in[1].v[e], fma2(hat, par.w[e], par.b[e]), in[NT - 1].v[e], dz.v[e]);
        dw[e] = fma2(dt, hat, dw[e]);
        db[e] = add2(db[e], dt);
      }
      if constexpr (GATE) st_unit<T, V>(gzp + static_cast<size_t>(row) * p.C, dz);
    });
    __syncthreads();
#pragma unroll
    for (int e = 0; e < V; ++e) {
      red[0][tid][e] = e & 1 ? hi_of(dw[e / 2]) : lo_of(dw[e / 2]);
      red[1][tid][e] = e & 1 ? hi_of(db[e / 2]) : lo_of(db[e / 2]);
    }
    __syncthreads();
    for (int i = tid; i < 2 * width * V; i += 256) {
      const int which = i / (width * V), ch = i % (width * V), un = ch / V, e = ch % V;
      float s = 0.f;
      for (int k = 0; k < slots; ++k) s += red[which][k * width + un][e];
      p.part[which * all + (static_cast<size_t>(n) * p.splits + part) * p.C + u0 * V + ch] = s;
    }
  }
}

// Gradient, second pass.  The first `warp_blocks` blocks: sums[N][G] of (mean
// dh, mean dh hat), a warp each, from the channel sums: over the group w db and
// w dw.  The others: dw, then db, 32 channels a block.
__global__ void __launch_bounds__(256) gn_grad_groups_kernel(const GnParams p, float* __restrict__ sums,
                                                             int warp_blocks) {
  launch_next();
  wait_before();
  if (static_cast<int>(blockIdx.x) >= warp_blocks) {
    const int b = blockIdx.x - warp_blocks, per = (p.C + 31) / 32;
    gn_param_sum(p.part, p.N * p.splits, p.C, b / per ? p.gb : p.gw, p.pbf, b % per, b / per);
    return;
  }
  const long long i = (static_cast<long long>(blockIdx.x) * 256 + threadIdx.x) >> 5;
  if (i >= static_cast<long long>(p.N) * p.G) return;
  const long long n = i / p.G;
  const int g = static_cast<int>(i % p.G), lane = threadIdx.x & 31;
  const size_t all = static_cast<size_t>(p.N) * p.splits * p.C;
  const float* at = p.part + n * p.splits * p.C + g * p.cg;
  float s1 = 0.f, s2 = 0.f;
  // lanes over the group's channels and, where those are few, over the splits
  const int across = min(p.cg, 32), per = 32 / across, k0 = lane / across;
  if (k0 < per)
    for (int c = lane % across; c < p.cg; c += across) {
      float t1 = 0.f, t2 = 0.f;
      for (int k = k0; k < p.splits; k += 8 * per) {
        float x[8], y[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float* q = at + static_cast<size_t>(min(k + j * per, p.splits - 1)) * p.C + c;
          x[j] = ld_after(q);
          y[j] = ld_after(q + all);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          t2 += k + j * per < p.splits ? x[j] : 0.f;
          t1 += k + j * per < p.splits ? y[j] : 0.f;
        }
      }
      const float w = gn_param(p.weight, p.pbf, g * p.cg + c, 1.f);
      s1 = fmaf(w, t1, s1);
      s2 = fmaf(w, t2, s2);
    }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
    s1 += __shfl_xor_sync(0xffffffffu, s1, off);
    s2 += __shfl_xor_sync(0xffffffffu, s2, off);
  }
  if (lane == 0) {
    const float inv = 1.f / (static_cast<float>(p.L) * static_cast<float>(p.cg));
    sums[i * 2] = s1 * inv;
    sums[i * 2 + 1] = s2 * inv;
  }
}

// Gradient, third pass: dx.
template <typename T, int V, bool GATE, bool ACT>
__global__ void __launch_bounds__(256, 3) gn_grad_apply_kernel(const GnParams p, const float* __restrict__ sums) {
  constexpr int P = Unit<T, V>::P, NT = GATE ? 3 : 2;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(8) uint64_t bars[12];
  const int tid = threadIdx.x, n = blockIdx.x / p.parts, part = blockIdx.x % p.parts, cv = p.C / V;
  int l0, l1;
  gn_rows(p.L, p.part_rows, part, l0, l1);
  const size_t base = (static_cast<size_t>(n) * p.L + l0) * p.C, ng = static_cast<size_t>(n) * p.G;
  GnRing<NT> ring;
  ring.init(smem, bars, p.limit_ns);
  wait_before();
  for (int u0 = 0; u0 < cv; u0 += 256) {
    const int width = min(cv - u0, 256), slots = cv > 256 ? 1 : 256 / width, c = (u0 + tid % width) * V;
    const GnParam<V> par(p, c, true);
    const GnStat<V> mean(p.mean + ng, 1, c, p.cg), rstd(p.rstd + ng, 1, c, p.cg);
    GnStat<V> s1(sums + 2 * ng, 2, c, p.cg), s2(sums + 2 * ng + 1, 2, c, p.cg);
#pragma unroll
    for (int e = 0; e < P; ++e) {
      s1.v[e] = mul2(s1.v[e], both(-1.f));
      s2.v[e] = mul2(s2.v[e], both(-1.f));
    }
    const T* src[NT];
    src[0] = static_cast<const T*>(p.x) + base + u0 * V;
    src[1] = static_cast<const T*>(p.gy) + base + u0 * V;
    if constexpr (GATE) src[2] = static_cast<const T*>(p.gate) + base + u0 * V;
    T* gxp = static_cast<T*>(p.gx) + base + c;
    ring.template walk<T, V>(src, l1 - l0, p.C, width, slots, [&](int row, Unit<T, V>(&in)[NT], bool ok) {
      if (!ok) return;
      Unit<T, V> dx;
#pragma unroll
      for (int e = 0; e < P; ++e) {
        const f2 hat = mul2(fma2(mean.v[e], both(-1.f), in[0].v[e]), rstd.v[e]);
        f2 dz;
        const f2 dt = gn_grad<GATE, ACT>(in[1].v[e], fma2(hat, par.w[e], par.b[e]), in[NT - 1].v[e], dz);
        dx.v[e] = mul2(rstd.v[e], fma2(hat, s2.v[e], fma2(dt, par.w[e], s1.v[e])));
      }
      st_unit<T, V>(gxp + static_cast<size_t>(row) * p.C, dx);
    });
  }
}

}  // namespace ttt
