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
// All of it is bound by memory: values are read in 16-byte units, several in
// flight a thread, and the statistics are taken in fp32 from registers, mean
// first and then squares around it (of a channel over a batch of positions;
// batches, channels, threads and blocks are joined by the exact two-set
// formula), so a mean far from zero costs no digits.  Every sum has a fixed
// order: the same call gives the same bits.
#pragma once
#include "common.cuh"

namespace ttt {

// 16 bytes of T as floats.
template <typename T, int V>
struct Unit {
  float v[V];
};
template <typename T, int V>
__device__ __forceinline__ Unit<T, V> ld_unit(const T* p) {
  static_assert(sizeof(T) * V == 16, "");
  Unit<T, V> r;
  const uint4 u = __ldg(reinterpret_cast<const uint4*>(p));
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (sizeof(T) == 2) {
      r.v[2 * i] = __uint_as_float(w[i] << 16);
      r.v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    } else {
      r.v[i] = __uint_as_float(w[i]);
    }
  }
  return r;
}
template <typename T, int V>
__device__ __forceinline__ void st_unit(T* p, const Unit<T, V>& x) {
  uint4 u;
  if constexpr (sizeof(T) == 2)
    u = make_uint4(pack_bf16x2(x.v[0], x.v[1]), pack_bf16x2(x.v[2], x.v[3]), pack_bf16x2(x.v[4], x.v[5]),
                   pack_bf16x2(x.v[6], x.v[7]));
  else
    u = make_uint4(__float_as_uint(x.v[0]), __float_as_uint(x.v[1]), __float_as_uint(x.v[2]), __float_as_uint(x.v[3]));
  *reinterpret_cast<uint4*>(p) = u;
}

struct GnParams {
  int N, L, C, G, cg;
  const void *x, *gate;
  const void *weight, *bias;  // [C] or nullptr
  int pbf;                    // weight and bias are bf16 (else fp32)
  int act;                    // 0 identity, 1 silu
  float eps;
  void* y;
  float *mean, *rstd;         // [N][G]
  float* part;                // partial statistics
  int splits, rows;           // parts of a sample for the statistics and the gradient's sums, positions in each
  int parts, part_rows;       // the same for the passes that write y or dx
  int width, slots;           // one-position kernels: units of a row in a block, rows at a time
  // gradient
  const void* gy;
  void *gx, *ggate;
  void *gw, *gb;              // [C] or nullptr
};

__device__ __forceinline__ float gn_param(const void* p, int pbf, int c, float none) {
  if (!p) return none;
  return pbf ? __bfloat162float(__ldg(static_cast<const __nv_bfloat16*>(p) + c)) : __ldg(static_cast<const float*>(p) + c);
}
// (the approximate division is off by two steps at most and gives 0 for the infinite exp(-x) of x < -88)
__device__ __forceinline__ float gn_sigmoid(float x) { return __fdividef(1.f, 1.f + __expf(-x)); }

// y for one value.
template <bool GATE>
__device__ __forceinline__ float gn_out(float t, float z, int act) {
  if constexpr (GATE) return t * (act ? z * gn_sigmoid(z) : z);
  return act ? t * gn_sigmoid(t) : t;
}
// dL/dt for one value; dz: dL/dgate.
template <bool GATE>
__device__ __forceinline__ float gn_grad(float g, float t, float z, int act, float& dz) {
  if constexpr (GATE) {
    if (!act) {
      dz = g * t;
      return g * z;
    }
    const float s = gn_sigmoid(z);
    dz = g * t * s * (1.f + z * (1.f - s));
    return g * z * s;
  }
  dz = 0.f;
  if (!act) return g;
  const float s = gn_sigmoid(t);
  return g * s * (1.f + t * (1.f - s));
}

// Count, mean and sum of squares around it; joined exactly.
struct Moments {
  float n, mean, m2;
};
__device__ __forceinline__ Moments join(const Moments& a, const Moments& b) {
  const float n = a.n + b.n;
  if (n == 0.f) return a;
  const float f = b.n / n, d = b.mean - a.mean;
  return Moments{n, fmaf(d, f, a.mean), a.m2 + b.m2 + d * d * a.n * f};
}
__device__ __forceinline__ Moments shfl_xor(const Moments& a, int off) {
  return Moments{__shfl_xor_sync(0xffffffffu, a.n, off), __shfl_xor_sync(0xffffffffu, a.mean, off),
                 __shfl_xor_sync(0xffffffffu, a.m2, off)};
}

// ------------------------------------------------- one position a sample ----
// L = 1 and a group of 1, 2, 4 .. 32 units: the lanes of a group hold it in
// registers, one unit a thread, so the values are read once.  A thread keeps
// its channels over all its rows (weight and bias in registers) and has R rows
// in flight.  Block x: units [x width, (x + 1) width) of a row, `slots` rows at
// a time where a row is narrow.
// Measured (B200, 16384 x 2048 bf16 with a gate): 33 us, 6.1 TB/s.
template <typename T, int V>
struct GnParam {
  float w[V], b[V];
  __device__ __forceinline__ GnParam(const GnParams& p, int c, bool on) {
#pragma unroll
    for (int e = 0; e < V; ++e) {
      w[e] = on ? gn_param(p.weight, p.pbf, c + e, 1.f) : 1.f;
      b[e] = on ? gn_param(p.bias, p.pbf, c + e, 0.f) : 0.f;
    }
  }
};

template <typename T, int V, bool GATE>
__global__ void __launch_bounds__(256) gn_row_kernel(const GnParams p, int lanes) {
  constexpr int R = GATE ? 4 : 6;
  const int tid = threadIdx.x, slot = tid / p.width, u = blockIdx.x * p.width + tid % p.width;
  const bool on = slot < p.slots && u < p.C / V;
  const int c = on ? u * V : 0;
  const GnParam<T, V> par(p, c, on);
  const float inv = 1.f / static_cast<float>(p.cg);
  const long long step = static_cast<long long>(gridDim.y) * p.slots;
  const long long rounds = (p.N + step - 1) / step;  // the same for the whole block: warps meet in the shuffles
  for (long long k0 = 0; k0 < rounds; k0 += R) {
    Unit<T, V> x[R], z[R];
    long long n[R];
    bool ok[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
      n[i] = (k0 + i) * step + static_cast<long long>(blockIdx.y) * p.slots + slot;
      ok[i] = on && n[i] < p.N;
      if (ok[i]) {
        x[i] = ld_unit<T, V>(static_cast<const T*>(p.x) + n[i] * p.C + c);
        if constexpr (GATE) z[i] = ld_unit<T, V>(static_cast<const T*>(p.gate) + n[i] * p.C + c);
      } else {
#pragma unroll
        for (int e = 0; e < V; ++e) x[i].v[e] = z[i].v[e] = 0.f;
      }
    }
    float mean[R], q[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
      mean[i] = 0.f;
#pragma unroll
      for (int e = 0; e < V; ++e) mean[i] += x[i].v[e];
    }
    for (int off = lanes >> 1; off > 0; off >>= 1)
#pragma unroll
      for (int i = 0; i < R; ++i) mean[i] += __shfl_xor_sync(0xffffffffu, mean[i], off);
#pragma unroll
    for (int i = 0; i < R; ++i) {
      mean[i] *= inv;
      q[i] = 0.f;
#pragma unroll
      for (int e = 0; e < V; ++e) {
        x[i].v[e] -= mean[i];
        q[i] = fmaf(x[i].v[e], x[i].v[e], q[i]);
      }
    }
    for (int off = lanes >> 1; off > 0; off >>= 1)
#pragma unroll
      for (int i = 0; i < R; ++i) q[i] += __shfl_xor_sync(0xffffffffu, q[i], off);
#pragma unroll
    for (int i = 0; i < R; ++i) {
      if (!ok[i]) continue;
      const float rstd = rsqrtf(fmaf(q[i], inv, p.eps));
      Unit<T, V> y;
#pragma unroll
      for (int e = 0; e < V; ++e)
        y.v[e] = gn_out<GATE>(fmaf(x[i].v[e] * rstd, par.w[e], par.b[e]), z[i].v[e], p.act);
      st_unit<T, V>(static_cast<T*>(p.y) + n[i] * p.C + c, y);
      if (c % p.cg == 0) {
        p.mean[n[i] * p.G + c / p.cg] = mean[i];
        p.rstd[n[i] * p.G + c / p.cg] = rstd;
      }
    }
  }
}

// Its gradient: dw and db gather in registers over the thread's rows; the
// block's sums go to part[2][gridDim.y][C].
template <typename T, int V, bool GATE>
__global__ void __launch_bounds__(256) gn_row_grad_kernel(const GnParams p, int lanes) {
  constexpr int R = 2;
  __shared__ float red[2][256][V + 1];
  const int tid = threadIdx.x, slot = tid / p.width, u = blockIdx.x * p.width + tid % p.width;
  const bool on = slot < p.slots && u < p.C / V;
  const int c = on ? u * V : 0;
  const GnParam<T, V> par(p, c, on);
  float dw[V], db[V];
#pragma unroll
  for (int e = 0; e < V; ++e) dw[e] = db[e] = 0.f;
  const int g = c / p.cg;
  const float inv = 1.f / static_cast<float>(p.cg);
  const long long step = static_cast<long long>(gridDim.y) * p.slots;
  const long long rounds = (p.N + step - 1) / step;
  for (long long k0 = 0; k0 < rounds; k0 += R) {
    Unit<T, V> x[R], z[R], gy[R];
    float mean[R], rstd[R], s1[R], s2[R];
    long long n[R];
    bool ok[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
      n[i] = (k0 + i) * step + static_cast<long long>(blockIdx.y) * p.slots + slot;
      ok[i] = on && n[i] < p.N;
      mean[i] = rstd[i] = s1[i] = s2[i] = 0.f;
      if (ok[i]) {
        const long long at = n[i] * p.C + c;
        x[i] = ld_unit<T, V>(static_cast<const T*>(p.x) + at);
        gy[i] = ld_unit<T, V>(static_cast<const T*>(p.gy) + at);
        if constexpr (GATE) z[i] = ld_unit<T, V>(static_cast<const T*>(p.gate) + at);
        mean[i] = __ldg(p.mean + n[i] * p.G + g);
        rstd[i] = __ldg(p.rstd + n[i] * p.G + g);
      } else {
#pragma unroll
        for (int e = 0; e < V; ++e) x[i].v[e] = gy[i].v[e] = z[i].v[e] = 0.f;
      }
    }
#pragma unroll
    for (int i = 0; i < R; ++i) {
      Unit<T, V> dz;
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float hat = (x[i].v[e] - mean[i]) * rstd[i];
        const float dt = gn_grad<GATE>(gy[i].v[e], fmaf(hat, par.w[e], par.b[e]), z[i].v[e], p.act, dz.v[e]);
        dw[e] = fmaf(dt, hat, dw[e]);
        db[e] += dt;
        x[i].v[e] = hat;
        gy[i].v[e] = dt * par.w[e];
        s1[i] += gy[i].v[e];
        s2[i] = fmaf(gy[i].v[e], hat, s2[i]);
      }
      if (GATE && ok[i]) st_unit<T, V>(static_cast<T*>(p.ggate) + n[i] * p.C + c, dz);
    }
    for (int off = lanes >> 1; off > 0; off >>= 1)
#pragma unroll
      for (int i = 0; i < R; ++i) {
        s1[i] += __shfl_xor_sync(0xffffffffu, s1[i], off);
        s2[i] += __shfl_xor_sync(0xffffffffu, s2[i], off);
      }
#pragma unroll
    for (int i = 0; i < R; ++i) {
      if (!ok[i]) continue;
      Unit<T, V> dx;
#pragma unroll
      for (int e = 0; e < V; ++e) dx.v[e] = rstd[i] * (gy[i].v[e] - s1[i] * inv - x[i].v[e] * (s2[i] * inv));
      st_unit<T, V>(static_cast<T*>(p.gx) + n[i] * p.C + c, dx);
    }
  }
  if (!p.part) return;
#pragma unroll
  for (int e = 0; e < V; ++e) {
    red[0][tid][e] = dw[e];
    red[1][tid][e] = db[e];
  }
  __syncthreads();
  for (int i = tid; i < 2 * p.width * V; i += blockDim.x) {
    const int which = i / (p.width * V), ch = i % (p.width * V), un = ch / V, e = ch % V;
    const int at = blockIdx.x * p.width * V + ch;
    if (at >= p.C) continue;
    float s = 0.f;
    for (int k = 0; k < p.slots; ++k) s += red[which][k * p.width + un][e];
    p.part[(static_cast<size_t>(which) * gridDim.y + blockIdx.y) * p.C + at] = s;
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
    int k = warp;
    for (; k + 56 < count; k += 64) {
      float t[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) t[i] = __ldg(at + static_cast<size_t>(k + 8 * i) * C);
#pragma unroll
      for (int i = 0; i < 8; ++i) s += t[i];
    }
    for (; k < count; k += 8) s += __ldg(at + static_cast<size_t>(k) * C);
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
  gn_param_sum(part, count, C, blockIdx.y ? gb : gw, pbf, blockIdx.x, blockIdx.y);
}

// ------------------------------------------------------ any L and width ----
// A thread keeps one unit of channels (whose channels may lie in two groups)
// and walks positions: rows [k rows, (k + 1) rows) of a sample are part k.
__device__ __forceinline__ void gn_rows(int L, int rows, int k, int& l0, int& l1) {
  l0 = static_cast<int>(min(static_cast<long long>(L), static_cast<long long>(k) * rows));
  l1 = static_cast<int>(min(static_cast<long long>(L), static_cast<long long>(l0) + rows));
}

// Statistics of one split of one sample: part[N][splits][G] of (mean, m2), or,
// where a sample is one split, mean and rstd.  Dynamic shared memory: G
// Moments.
template <typename T, int V>
__global__ void __launch_bounds__(256) gn_stats_kernel(const GnParams p) {
  extern __shared__ Moments group[];  // [G]
  __shared__ float each[2][256][V + 1];
  __shared__ float counts[256];
  const int tid = threadIdx.x, n = blockIdx.x / p.splits, part = blockIdx.x % p.splits, cv = p.C / V;
  int l0, l1;
  gn_rows(p.L, p.rows, part, l0, l1);
  for (int g = tid; g < p.G; g += 256) group[g] = Moments{0.f, 0.f, 0.f};
  const T* x = static_cast<const T*>(p.x) + static_cast<size_t>(n) * p.L * p.C;
  for (int u0 = 0; u0 < cv; u0 += 256) {
    const int width = min(cv - u0, 256), slots = 256 / width, slot = tid / width, u = u0 + tid % width;
    float cnt = 0.f, mean[V], m2[V];
#pragma unroll
    for (int e = 0; e < V; ++e) mean[e] = m2[e] = 0.f;
    if (slot < slots) {
      constexpr int U = 32 / V;  // positions per batch: 128 bytes a thread in flight (fp32), 64 (bf16)
      for (int l = l0 + slot; l < l1; l += U * slots) {
        Unit<T, V> b[U];
        int have = 0;
#pragma unroll
        for (int i = 0; i < U; ++i)
          if (l + i * slots < l1) {
            b[i] = ld_unit<T, V>(x + static_cast<size_t>(l + i * slots) * p.C + u * V);
            ++have;
          }
        const float h = static_cast<float>(have), inv = 1.f / h, f = h / (cnt + h);
#pragma unroll
        for (int e = 0; e < V; ++e) {
          float s = 0.f, q = 0.f;
#pragma unroll
          for (int i = 0; i < U; ++i)
            if (i < have) s += b[i].v[e];
          s *= inv;
#pragma unroll
          for (int i = 0; i < U; ++i)
            if (i < have) q = fmaf(b[i].v[e] - s, b[i].v[e] - s, q);
          const float d = s - mean[e];
          mean[e] = fmaf(d, f, mean[e]);
          m2[e] += q + d * d * cnt * f;
        }
        cnt += h;
      }
    }
    __syncthreads();
    counts[tid] = cnt;
#pragma unroll
    for (int e = 0; e < V; ++e) {
      each[0][tid][e] = mean[e];
      each[1][tid][e] = m2[e];
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
      p.rstd[at] = rsqrtf(group[g].m2 / group[g].n + p.eps);
    } else {
      float2* d = reinterpret_cast<float2*>(p.part) + (static_cast<size_t>(n) * p.splits + part) * p.G + g;
      *d = make_float2(group[g].mean, group[g].m2);
    }
  }
}

// mean and rstd from the splits' statistics, a warp per (sample, group).
__global__ void __launch_bounds__(256) gn_join_kernel(const GnParams p) {
  const long long i = (static_cast<long long>(blockIdx.x) * 256 + threadIdx.x) >> 5;
  if (i >= static_cast<long long>(p.N) * p.G) return;
  const long long n = i / p.G;
  const int g = static_cast<int>(i % p.G);
  const float2* d = reinterpret_cast<const float2*>(p.part) + n * p.splits * p.G + g;
  Moments m{0.f, 0.f, 0.f};
#pragma unroll 4
  for (int k = threadIdx.x & 31; k < p.splits; k += 32) {
    const float2 x = __ldg(d + static_cast<size_t>(k) * p.G);
    int a, b;
    gn_rows(p.L, p.rows, k, a, b);
    if (b > a) m = join(m, Moments{static_cast<float>(b - a) * static_cast<float>(p.cg), x.x, x.y});
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) m = join(m, shfl_xor(m, off));
  if ((threadIdx.x & 31) == 0) {
    p.mean[i] = m.mean;
    p.rstd[i] = rsqrtf(m.m2 / m.n + p.eps);
  }
}

// y from mean and rstd.
template <typename T, int V, bool GATE>
__global__ void __launch_bounds__(256) gn_apply_kernel(const GnParams p) {
  const int tid = threadIdx.x, n = blockIdx.x / p.parts, part = blockIdx.x % p.parts, cv = p.C / V;
  int l0, l1;
  gn_rows(p.L, p.part_rows, part, l0, l1);
  const size_t base = static_cast<size_t>(n) * p.L * p.C;
  for (int u0 = 0; u0 < cv; u0 += 256) {
    const int width = min(cv - u0, 256), slots = 256 / width, slot = tid / width, u = u0 + tid % width;
    if (slot >= slots) continue;
    const int c = u * V;
    const GnParam<T, V> par(p, c, true);
    float k[V], mean[V];  // t = (x - mean) k + b
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const size_t at = static_cast<size_t>(n) * p.G + (c + e) / p.cg;
      mean[e] = __ldg(p.mean + at);
      k[e] = __ldg(p.rstd + at) * par.w[e];
    }
#pragma unroll 4
    for (int l = l0 + slot; l < l1; l += slots) {
      const size_t at = base + static_cast<size_t>(l) * p.C + c;
      const Unit<T, V> x = ld_unit<T, V>(static_cast<const T*>(p.x) + at);
      Unit<T, V> z = x, y;
      if constexpr (GATE) z = ld_unit<T, V>(static_cast<const T*>(p.gate) + at);
#pragma unroll
      for (int e = 0; e < V; ++e) y.v[e] = gn_out<GATE>(fmaf(x.v[e] - mean[e], k[e], par.b[e]), z.v[e], p.act);
      st_unit<T, V>(static_cast<T*>(p.y) + at, y);
    }
  }
}

// Gradient, first pass: part[2][N][splits][C], the sums of dt hat and of dt
// over a split's positions; also dgate.
template <typename T, int V, bool GATE>
__global__ void __launch_bounds__(256) gn_grad_sums_kernel(const GnParams p) {
  __shared__ float red[2][256][V + 1];
  const int tid = threadIdx.x, n = blockIdx.x / p.splits, part = blockIdx.x % p.splits, cv = p.C / V;
  int l0, l1;
  gn_rows(p.L, p.rows, part, l0, l1);
  const size_t base = static_cast<size_t>(n) * p.L * p.C, all = static_cast<size_t>(p.N) * p.splits * p.C;
  for (int u0 = 0; u0 < cv; u0 += 256) {
    const int width = min(cv - u0, 256), slots = 256 / width, slot = tid / width, u = u0 + tid % width;
    float dw[V], db[V];
#pragma unroll
    for (int e = 0; e < V; ++e) dw[e] = db[e] = 0.f;
    if (slot < slots) {
      const int c = u * V;
      const GnParam<T, V> par(p, c, true);
      float mean[V], rstd[V];
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const size_t at = static_cast<size_t>(n) * p.G + (c + e) / p.cg;
        mean[e] = __ldg(p.mean + at);
        rstd[e] = __ldg(p.rstd + at);
      }
#pragma unroll 4
      for (int l = l0 + slot; l < l1; l += slots) {
        const size_t at = base + static_cast<size_t>(l) * p.C + c;
        const Unit<T, V> x = ld_unit<T, V>(static_cast<const T*>(p.x) + at);
        const Unit<T, V> gy = ld_unit<T, V>(static_cast<const T*>(p.gy) + at);
        Unit<T, V> z = x, dz;
        if constexpr (GATE) z = ld_unit<T, V>(static_cast<const T*>(p.gate) + at);
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const float hat = (x.v[e] - mean[e]) * rstd[e];
          const float dt = gn_grad<GATE>(gy.v[e], fmaf(hat, par.w[e], par.b[e]), z.v[e], p.act, dz.v[e]);
          dw[e] = fmaf(dt, hat, dw[e]);
          db[e] += dt;
        }
        if constexpr (GATE) st_unit<T, V>(static_cast<T*>(p.ggate) + at, dz);
      }
    }
    __syncthreads();
#pragma unroll
    for (int e = 0; e < V; ++e) {
      red[0][tid][e] = dw[e];
      red[1][tid][e] = db[e];
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
  const long long items = static_cast<long long>(p.splits) * p.cg;
#pragma unroll 8
  for (long long e = lane; e < items; e += 32) {
    const int k = static_cast<int>(e / p.cg), c = static_cast<int>(e % p.cg);
    const float w = gn_param(p.weight, p.pbf, g * p.cg + c, 1.f);
    const float* q = at + static_cast<size_t>(k) * p.C + c;
    s2 = fmaf(w, __ldg(q), s2);
    s1 = fmaf(w, __ldg(q + all), s1);
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
template <typename T, int V, bool GATE>
__global__ void __launch_bounds__(256) gn_grad_apply_kernel(const GnParams p, const float* __restrict__ sums) {
  const int tid = threadIdx.x, n = blockIdx.x / p.parts, part = blockIdx.x % p.parts, cv = p.C / V;
  int l0, l1;
  gn_rows(p.L, p.part_rows, part, l0, l1);
  const size_t base = static_cast<size_t>(n) * p.L * p.C;
  for (int u0 = 0; u0 < cv; u0 += 256) {
    const int width = min(cv - u0, 256), slots = 256 / width, slot = tid / width, u = u0 + tid % width;
    if (slot >= slots) continue;
    const int c = u * V;
    const GnParam<T, V> par(p, c, true);
    float mean[V], rstd[V], s1[V], s2[V];
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const size_t ng = static_cast<size_t>(n) * p.G + (c + e) / p.cg;
      mean[e] = __ldg(p.mean + ng);
      rstd[e] = __ldg(p.rstd + ng);
      s1[e] = __ldg(sums + 2 * ng);
      s2[e] = __ldg(sums + 2 * ng + 1);
    }
#pragma unroll 2
    for (int l = l0 + slot; l < l1; l += slots) {
      const size_t at = base + static_cast<size_t>(l) * p.C + c;
      const Unit<T, V> x = ld_unit<T, V>(static_cast<const T*>(p.x) + at);
      const Unit<T, V> gy = ld_unit<T, V>(static_cast<const T*>(p.gy) + at);
      Unit<T, V> z = x, dx;
      if constexpr (GATE) z = ld_unit<T, V>(static_cast<const T*>(p.gate) + at);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float hat = (x.v[e] - mean[e]) * rstd[e];
        float dz;
        const float dt = gn_grad<GATE>(gy.v[e], fmaf(hat, par.w[e], par.b[e]), z.v[e], p.act, dz);
        dx.v[e] = rstd[e] * (fmaf(dt, par.w[e], -s1[e]) - hat * s2[e]);
      }
      st_unit<T, V>(static_cast<T*>(p.gx) + at, dx);
    }
  }
}

}  // namespace ttt
