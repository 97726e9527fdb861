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
// All of it is bound by memory: the values are read in 16-byte units and the
// statistics are taken in fp32 from registers, mean first and then squares
// around it (per thread over a batch of units; batches, threads and blocks are
// joined by the exact two-set formula), so a mean far from zero costs no
// digits.  Every sum has a fixed order: the same call gives the same bits.
#pragma once
#include "common.cuh"

namespace ttt {

// 16 bytes of T as floats, and smaller units where the group width asks for them.
template <typename T, int V>
struct Unit {
  float v[V];
};
template <typename T, int V>
__device__ __forceinline__ Unit<T, V> ld_unit(const T* p) {
  Unit<T, V> r;
  if constexpr (sizeof(T) * V == 16) {
    const uint4 u = __ldg(reinterpret_cast<const uint4*>(p));
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    if constexpr (sizeof(T) == 2) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        r.v[2 * i] = __uint_as_float(w[i] << 16);
        r.v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) r.v[i] = __uint_as_float(w[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) r.v[i] = to_f<T>(__ldg(p + i));
  }
  return r;
}
template <typename T, int V>
__device__ __forceinline__ void st_unit(T* p, const Unit<T, V>& x) {
  if constexpr (sizeof(T) * V == 16) {
    uint4 u;
    if constexpr (sizeof(T) == 2)
      u = make_uint4(pack_bf16x2(x.v[0], x.v[1]), pack_bf16x2(x.v[2], x.v[3]), pack_bf16x2(x.v[4], x.v[5]),
                     pack_bf16x2(x.v[6], x.v[7]));
    else
      u = make_uint4(__float_as_uint(x.v[0]), __float_as_uint(x.v[1]), __float_as_uint(x.v[2]), __float_as_uint(x.v[3]));
    *reinterpret_cast<uint4*>(p) = u;
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) p[i] = from_f<T>(x.v[i]);
  }
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
  int splits, rows;           // parts of a sample, positions in each
  // gradient
  const void* gy;
  void *gx, *ggate;
  void *gw, *gb;              // [C] or nullptr
  int blocks;                 // row blocks of the one-position gradient (partials in `part`)
};

__device__ __forceinline__ float gn_param(const void* p, int pbf, int c, float none) {
  if (!p) return none;
  return pbf ? __bfloat162float(__ldg(static_cast<const __nv_bfloat16*>(p) + c)) : __ldg(static_cast<const float*>(p) + c);
}
__device__ __forceinline__ float gn_sigmoid(float x) { return 1.f / (1.f + __expf(-x)); }

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
// L = 1 and cg / V a power of two up to 32: the lanes of a group hold it in
// registers, one unit a thread, so the values are read once.
template <typename T, int V, bool GATE>
__global__ void __launch_bounds__(256) gn_row_kernel(const GnParams p, int lanes) {
  const int cv = p.C / V;
  const long long total = static_cast<long long>(p.N) * cv, stride = static_cast<long long>(gridDim.x) * blockDim.x;
  const long long padded = (total + 31) / 32 * 32;  // whole warps take part in the shuffles
  for (long long i = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x; i < padded; i += stride) {
    const bool ok = i < total;
    const long long n = ok ? i / cv : 0;
    const int c = ok ? static_cast<int>(i - n * cv) * V : 0;
    Unit<T, V> x, z;
#pragma unroll
    for (int e = 0; e < V; ++e) x.v[e] = z.v[e] = 0.f;
    if (ok) {
      x = ld_unit<T, V>(static_cast<const T*>(p.x) + n * p.C + c);
      if constexpr (GATE) z = ld_unit<T, V>(static_cast<const T*>(p.gate) + n * p.C + c);
    }
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < V; ++e) s += x.v[e];
    for (int off = lanes >> 1; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
    const float mean = s / static_cast<float>(p.cg);
    float q = 0.f;
#pragma unroll
    for (int e = 0; e < V; ++e) q = fmaf(x.v[e] - mean, x.v[e] - mean, q);
    for (int off = lanes >> 1; off > 0; off >>= 1) q += __shfl_xor_sync(0xffffffffu, q, off);
    const float rstd = rsqrtf(q / static_cast<float>(p.cg) + p.eps);
    if (!ok) continue;
    Unit<T, V> y;
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const float t = fmaf((x.v[e] - mean) * rstd, gn_param(p.weight, p.pbf, c + e, 1.f), gn_param(p.bias, p.pbf, c + e, 0.f));
      y.v[e] = gn_out<GATE>(t, z.v[e], p.act);
    }
    st_unit<T, V>(static_cast<T*>(p.y) + n * p.C + c, y);
    if (c % p.cg == 0) {
      p.mean[n * p.G + c / p.cg] = mean;
      p.rstd[n * p.G + c / p.cg] = rstd;
    }
  }
}

// Its gradient: a thread keeps one unit of channels and walks samples, so dw
// and db gather in registers; the block's sums go to part[2][blocks][C].
template <typename T, int V, bool GATE>
__global__ void __launch_bounds__(256) gn_row_grad_kernel(const GnParams p, int lanes) {
  __shared__ float red[2][256][V + 1];
  const int cv = p.C / V;
  const int width = min(cv, 256), slots = 256 / width;  // units of channels in this block, samples at a time
  const int tid = threadIdx.x, slot = tid / width, u = blockIdx.x * 256 + tid % width;
  const bool on = slot < slots && u < cv;
  const int c = on ? u * V : 0;
  float w[V], b[V], dw[V], db[V];
#pragma unroll
  for (int e = 0; e < V; ++e) {
    w[e] = gn_param(p.weight, p.pbf, c + e, 1.f);
    b[e] = gn_param(p.bias, p.pbf, c + e, 0.f);
    dw[e] = db[e] = 0.f;
  }
  const int g = c / p.cg;
  const float inv = 1.f / static_cast<float>(p.cg);
  // (the trip count is the block's, so whole warps meet in the shuffles)
  for (long long n0 = static_cast<long long>(blockIdx.y) * slots; n0 < p.N; n0 += static_cast<long long>(gridDim.y) * slots) {
    const long long n = n0 + slot;
    const bool ok = on && n < p.N;
    Unit<T, V> x, z, gy;
    float mean = 0.f, rstd = 0.f;
#pragma unroll
    for (int e = 0; e < V; ++e) x.v[e] = z.v[e] = gy.v[e] = 0.f;
    if (ok) {
      const long long at = n * p.C + c;
      x = ld_unit<T, V>(static_cast<const T*>(p.x) + at);
      gy = ld_unit<T, V>(static_cast<const T*>(p.gy) + at);
      if constexpr (GATE) z = ld_unit<T, V>(static_cast<const T*>(p.gate) + at);
      mean = __ldg(p.mean + n * p.G + g);
      rstd = __ldg(p.rstd + n * p.G + g);
    }
    float dh[V], s1 = 0.f, s2 = 0.f;
    Unit<T, V> dz;
#pragma unroll
    for (int e = 0; e < V; ++e) {
      x.v[e] = (x.v[e] - mean) * rstd;  // hat
      const float dt = gn_grad<GATE>(gy.v[e], fmaf(x.v[e], w[e], b[e]), z.v[e], p.act, dz.v[e]);
      dw[e] = fmaf(dt, x.v[e], dw[e]);
      db[e] += dt;
      dh[e] = dt * w[e];
      s1 += dh[e];
      s2 = fmaf(dh[e], x.v[e], s2);
    }
    for (int off = lanes >> 1; off > 0; off >>= 1) {
      s1 += __shfl_xor_sync(0xffffffffu, s1, off);
      s2 += __shfl_xor_sync(0xffffffffu, s2, off);
    }
    if (!ok) continue;
    s1 *= inv, s2 *= inv;
    Unit<T, V> dx;
#pragma unroll
    for (int e = 0; e < V; ++e) dx.v[e] = rstd * (dh[e] - s1 - x.v[e] * s2);
    st_unit<T, V>(static_cast<T*>(p.gx) + n * p.C + c, dx);
    if constexpr (GATE) st_unit<T, V>(static_cast<T*>(p.ggate) + n * p.C + c, dz);
  }
  if (!p.part) return;
#pragma unroll
  for (int e = 0; e < V; ++e) {
    red[0][tid][e] = dw[e];
    red[1][tid][e] = db[e];
  }
  __syncthreads();
  for (int i = tid; i < 2 * width * V; i += 256) {
    const int which = i / (width * V), ch = i % (width * V), un = ch / V, e = ch % V;
    const int at = blockIdx.x * 256 * V + ch;
    if (at >= p.C) continue;
    float s = 0.f;
    for (int k = 0; k < slots; ++k) s += red[which][k * width + un][e];
    p.part[(static_cast<size_t>(which) * gridDim.y + blockIdx.y) * p.C + at] = s;
  }
}

// dw[c] and db[c]: the sum of `count` rows of part[2][count][C] in order, 8 at
// a time over the block's warps, then the warps in order.
__global__ void __launch_bounds__(256) gn_param_grad_kernel(const float* __restrict__ part, int count, int C, void* gw,
                                                            void* gb, int pbf) {
  __shared__ float red[8][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = blockIdx.x * 32 + lane, which = blockIdx.y;
  float s = 0.f;
  if (c < C)
    for (int k = warp; k < count; k += 8) s += __ldg(part + (static_cast<size_t>(which) * count + k) * C + c);
  red[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && c < C) {
    float t = 0.f;
    for (int k = 0; k < 8; ++k) t += red[k][lane];
    void* dst = which ? gb : gw;
    if (dst) {
      if (pbf)
        static_cast<__nv_bfloat16*>(dst)[c] = __float2bfloat16_rn(t);
      else
        static_cast<float*>(dst)[c] = t;
    }
  }
}

// ------------------------------------------------------ any L and width ----
// Positions of sample n that split k covers.
__device__ __forceinline__ void gn_rows(const GnParams& p, int k, int& l0, int& l1) {
  l0 = static_cast<int>(min(static_cast<long long>(p.L), static_cast<long long>(k) * p.rows));
  l1 = static_cast<int>(min(static_cast<long long>(p.L), static_cast<long long>(l0) + p.rows));
}

// Statistics of one split of one sample: part[N][splits][G] of (mean, m2).
// V divides cg, so that a thread's unit lies in one group.  dynamic shared
// memory: G Moments.
template <typename T, int V>
__global__ void __launch_bounds__(256) gn_stats_kernel(const GnParams p) {
  extern __shared__ Moments group[];  // [G]
  __shared__ Moments each[256];
  const int tid = threadIdx.x, n = blockIdx.x / p.splits, part = blockIdx.x % p.splits, cv = p.C / V, gv = p.cg / V;
  int l0, l1;
  gn_rows(p, part, l0, l1);
  for (int g = tid; g < p.G; g += 256) group[g] = Moments{0.f, 0.f, 0.f};
  const T* x = static_cast<const T*>(p.x) + static_cast<size_t>(n) * p.L * p.C;
  for (int u0 = 0; u0 < cv; u0 += 256) {
    const int width = min(cv - u0, 256), slots = 256 / width, slot = tid / width, u = u0 + tid % width;
    Moments m{0.f, 0.f, 0.f};
    if (slot < slots) {
      constexpr int U = (V >= 4) ? 4 : 8;  // positions per batch
      for (int l = l0 + slot; l < l1; l += U * slots) {
        Unit<T, V> b[U];
        int have = 0;
#pragma unroll
        for (int i = 0; i < U; ++i)
          if (l + i * slots < l1) {
            b[i] = ld_unit<T, V>(x + static_cast<size_t>(l + i * slots) * p.C + u * V);
            ++have;
          }
        float s = 0.f, q = 0.f;
#pragma unroll
        for (int i = 0; i < U; ++i)
          if (i < have)
#pragma unroll
            for (int e = 0; e < V; ++e) s += b[i].v[e];
        const float cnt = static_cast<float>(have * V), mean = s / cnt;
#pragma unroll
        for (int i = 0; i < U; ++i)
          if (i < have)
#pragma unroll
            for (int e = 0; e < V; ++e) q = fmaf(b[i].v[e] - mean, b[i].v[e] - mean, q);
        m = join(m, Moments{cnt, mean, q});
      }
    }
    __syncthreads();
    each[tid] = m;
    __syncthreads();
    // a warp for each group that these units touch
    const int g0 = u0 / gv, g1 = (u0 + width - 1) / gv;
    for (int g = g0 + (tid >> 5); g <= g1; g += 8) {
      const int a = max(g * gv, u0) - u0, b = min((g + 1) * gv, u0 + width) - u0;  // its units here
      Moments t{0.f, 0.f, 0.f};
      for (int i = tid & 31; i < slots * (b - a); i += 32) t = join(t, each[(i / (b - a)) * width + a + i % (b - a)]);
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) t = join(t, shfl_xor(t, off));
      if ((tid & 31) == 0) group[g] = join(group[g], t);
    }
  }
  __syncthreads();
  for (int g = tid; g < p.G; g += 256) {
    float* d = p.part + ((static_cast<size_t>(n) * p.splits + part) * p.G + g) * 2;
    d[0] = group[g].mean;
    d[1] = group[g].m2;
  }
}

// y from the splits' statistics.  Dynamic shared memory: 2 G floats.
template <typename T, int V, bool GATE>
__global__ void __launch_bounds__(256) gn_apply_kernel(const GnParams p) {
  extern __shared__ float st[];  // mean[G], rstd[G]
  const int tid = threadIdx.x, n = blockIdx.x / p.splits, part = blockIdx.x % p.splits, cv = p.C / V, gv = p.cg / V;
  for (int g = tid; g < p.G; g += 256) {
    Moments m{0.f, 0.f, 0.f};
    for (int k = 0; k < p.splits; ++k) {
      int a, b;
      gn_rows(p, k, a, b);
      const float* d = p.part + ((static_cast<size_t>(n) * p.splits + k) * p.G + g) * 2;
      if (b > a) m = join(m, Moments{static_cast<float>(b - a) * static_cast<float>(p.cg), d[0], d[1]});
    }
    const float rstd = rsqrtf(m.m2 / m.n + p.eps);
    st[g] = m.mean;
    st[p.G + g] = rstd;
    if (part == 0) {
      p.mean[static_cast<size_t>(n) * p.G + g] = m.mean;
      p.rstd[static_cast<size_t>(n) * p.G + g] = rstd;
    }
  }
  __syncthreads();
  int l0, l1;
  gn_rows(p, part, l0, l1);
  const size_t base = static_cast<size_t>(n) * p.L * p.C;
  for (int u0 = 0; u0 < cv; u0 += 256) {
    const int width = min(cv - u0, 256), slots = 256 / width, slot = tid / width, u = u0 + tid % width;
    if (slot >= slots) continue;
    const int c = u * V, g = u / gv;
    float k[V], b[V];  // t = x k + b
#pragma unroll
    for (int e = 0; e < V; ++e) {
      k[e] = st[p.G + g] * gn_param(p.weight, p.pbf, c + e, 1.f);
      b[e] = gn_param(p.bias, p.pbf, c + e, 0.f);
    }
    const float mean = st[g];
#pragma unroll 4
    for (int l = l0 + slot; l < l1; l += slots) {
      const size_t at = base + static_cast<size_t>(l) * p.C + c;
      const Unit<T, V> x = ld_unit<T, V>(static_cast<const T*>(p.x) + at);
      Unit<T, V> z = x, y;
      if constexpr (GATE) z = ld_unit<T, V>(static_cast<const T*>(p.gate) + at);
#pragma unroll
      for (int e = 0; e < V; ++e) y.v[e] = gn_out<GATE>(fmaf(x.v[e] - mean, k[e], b[e]), z.v[e], p.act);
      st_unit<T, V>(static_cast<T*>(p.y) + at, y);
    }
  }
}

// Gradient, first pass: part[2][N][splits][C], the sums of dt hat and of dt
// over a split's positions; also dgate.
template <typename T, int V, bool GATE>
__global__ void __launch_bounds__(256) gn_grad_sums_kernel(const GnParams p) {
  __shared__ float red[2][256][V + 1];
  const int tid = threadIdx.x, n = blockIdx.x / p.splits, part = blockIdx.x % p.splits, cv = p.C / V, gv = p.cg / V;
  int l0, l1;
  gn_rows(p, part, l0, l1);
  const size_t base = static_cast<size_t>(n) * p.L * p.C, all = static_cast<size_t>(p.N) * p.splits * p.C;
  for (int u0 = 0; u0 < cv; u0 += 256) {
    const int width = min(cv - u0, 256), slots = 256 / width, slot = tid / width, u = u0 + tid % width;
    float dw[V], db[V];
#pragma unroll
    for (int e = 0; e < V; ++e) dw[e] = db[e] = 0.f;
    if (slot < slots) {
      const int c = u * V, g = u / gv;
      const float mean = __ldg(p.mean + static_cast<size_t>(n) * p.G + g), rstd = __ldg(p.rstd + static_cast<size_t>(n) * p.G + g);
      float w[V], b[V];
#pragma unroll
      for (int e = 0; e < V; ++e) {
        w[e] = gn_param(p.weight, p.pbf, c + e, 1.f);
        b[e] = gn_param(p.bias, p.pbf, c + e, 0.f);
      }
#pragma unroll 2
      for (int l = l0 + slot; l < l1; l += slots) {
        const size_t at = base + static_cast<size_t>(l) * p.C + c;
        const Unit<T, V> x = ld_unit<T, V>(static_cast<const T*>(p.x) + at);
        const Unit<T, V> gy = ld_unit<T, V>(static_cast<const T*>(p.gy) + at);
        Unit<T, V> z = x, dz;
        if constexpr (GATE) z = ld_unit<T, V>(static_cast<const T*>(p.gate) + at);
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const float hat = (x.v[e] - mean) * rstd;
          const float dt = gn_grad<GATE>(gy.v[e], fmaf(hat, w[e], b[e]), z.v[e], p.act, dz.v[e]);
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

// Gradient, second pass: sums[N][G] of (mean dh, mean dh hat), one warp each,
// from the first pass's channel sums: sum over the group of w db and w dw.
__global__ void __launch_bounds__(256) gn_grad_groups_kernel(const GnParams p, float* __restrict__ sums) {
  const long long i = (static_cast<long long>(blockIdx.x) * 256 + threadIdx.x) >> 5;
  if (i >= static_cast<long long>(p.N) * p.G) return;
  const long long n = i / p.G;
  const int g = static_cast<int>(i % p.G), lane = threadIdx.x & 31;
  const size_t all = static_cast<size_t>(p.N) * p.splits * p.C;
  float s1 = 0.f, s2 = 0.f;
  const int items = p.splits * p.cg;
  for (int e = lane; e < items; e += 32) {
    const int k = e / p.cg, c = g * p.cg + e % p.cg;
    const float w = gn_param(p.weight, p.pbf, c, 1.f);
    const size_t at = (static_cast<size_t>(n) * p.splits + k) * p.C + c;
    s2 = fmaf(w, p.part[at], s2);
    s1 = fmaf(w, p.part[all + at], s1);
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
  const int tid = threadIdx.x, n = blockIdx.x / p.splits, part = blockIdx.x % p.splits, cv = p.C / V, gv = p.cg / V;
  int l0, l1;
  gn_rows(p, part, l0, l1);
  const size_t base = static_cast<size_t>(n) * p.L * p.C;
  for (int u0 = 0; u0 < cv; u0 += 256) {
    const int width = min(cv - u0, 256), slots = 256 / width, slot = tid / width, u = u0 + tid % width;
    if (slot >= slots) continue;
    const int c = u * V, g = u / gv;
    const size_t ng = static_cast<size_t>(n) * p.G + g;
    const float mean = __ldg(p.mean + ng), rstd = __ldg(p.rstd + ng), s1 = __ldg(sums + 2 * ng), s2 = __ldg(sums + 2 * ng + 1);
    float w[V], b[V];
#pragma unroll
    for (int e = 0; e < V; ++e) {
      w[e] = gn_param(p.weight, p.pbf, c + e, 1.f);
      b[e] = gn_param(p.bias, p.pbf, c + e, 0.f);
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
        const float hat = (x.v[e] - mean) * rstd;
        float dz;
        const float dt = gn_grad<GATE>(gy.v[e], fmaf(hat, w[e], b[e]), z.v[e], p.act, dz);
        dx.v[e] = rstd * (fmaf(dt, w[e], -s1) - hat * s2);
      }
      st_unit<T, V>(static_cast<T*>(p.gx) + at, dx);
    }
  }
}

}  // namespace ttt
