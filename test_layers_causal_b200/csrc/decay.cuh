// decay.cuh -- the fast-weight layer with a decay for each head: geometry,
// state scan, fp32-FMA chunked kernel and single-token step.
//
//   W_t = gamma_h W_{t-1} + a v_t k_t^T ,  o_t = W_t q_t ,  gamma_h = exp(log_decay[h]),  a = sigma * eta
//
// Everything below runs one recurrence in one of two directions over the
// tokens of a sequence, so that the gradient needs no kernels of its own.
// For a tile of n consecutive tokens, rows r, c = 0 .. n-1 in memory order,
// and the state X carried in (rows: features of v, columns: features of k):
//
//   forward   P_rc = sP gamma^(r-c) (q_r . k_c)  for c <= r, else 0
//             o_r  = sum_c P_rc v_c + sR gamma^(r+1) X q_r
//             X'   = gamma^n X + sU sum_c gamma^(n-1-c) v_c k_c^T
//   reverse   P_rc = sP gamma^(c-r) (q_r . k_c)  for c >= r, else 0
//             o_r  = sum_c P_rc v_c + sR gamma^(n-1-r) X q_r
//             X'   = gamma^n X + sU sum_c gamma^(c+1) v_c k_c^T
//
// The layer is (q, k, v) forward with (sP, sR, sU) = (a, 1, a) from W_0.  Its
// gradient, with G_t = dL/dW_t = gamma G_{t+1} + do_t q_t^T:
//   dq_t = W_t^T do_t    (do, v, k) forward, (a, 1, a), from W_0^T
//   dv_t = a G_t k_t     (k, q, do) reverse, (a, a, 1), from dL/dW_T; ends in dL/dW_0
//   dk_t = a G_t^T v_t   (v, do, q) reverse, (a, a, 1), from (dL/dW_T)^T
//
// A sequence is cut into segments of S tokens.  Where a sequence has more than
// one, three launches share the work: every segment's own contribution to the
// state (from zero), the scan of those over the segments, and the outputs of
// every segment from its start state.  No block waits for another.
#pragma once
#include "common.cuh"

namespace ttt {

// Sequences and their segments.  cu == nullptr: N sequences of T tokens each,
// else the sequences lie one behind another in T rows, sequence n in rows
// [cu[n], cu[n+1]) (values outside [0, T] are clamped to it, so no access
// leaves the tensors whatever cu holds).  Every sequence has at least one
// segment, an empty one too, whose block hands its state on.
//
// The workspace has a slot for each segment of the sequences that have several
// (`all`: of every sequence), numbered like the segments.  Many short sequences
// so need no more of it than the tokens do.  (Offsets that overlap make more
// segments than there are slots: those without one are not worked on.)
struct DecayGeom {
  int N, H, T, S;
  int nseg;         // upper bound of the segments over all sequences
  int slots;        // of the workspace
  int all;
  const int* cu;
};

struct DecaySpan {
  int seq;     // -1: no such segment
  int batch;   // index of the outer dimension
  int row0;    // first token row
  int len;     // tokens in the segment
  int j, nseg; // segment j of the sequence's nseg
  int slot;    // its place in the workspace, where it has one
};

__device__ __forceinline__ int decay_segments(int len, int S) { return len > 0 ? (len - 1) / S + 1 : 1; }

// Rows of sequence n.
__device__ __forceinline__ void decay_rows(const DecayGeom& g, int n, int& a, int& b) {
  if (!g.cu) {
    a = 0;
    b = g.T;
    return;
  }
  a = min(max(__ldg(g.cu + n), 0), g.T);
  b = min(max(__ldg(g.cu + n + 1), a), g.T);
}

// Zeros for the rows of o in no sequence, those before the first one and behind
// the last; the grid's blocks share them.  Inside the output kernels, so that
// rows which are there to be written once cost no launch, and none are cleared
// that the layer writes.
template <typename T>
__device__ __forceinline__ void decay_clear_rest(const DecayGeom& g, T* o, long long oh, long long ot, int dv) {
  constexpr int unit = 16 / sizeof(T);
  const int a = min(max(__ldg(g.cu), 0), g.T), b = min(max(__ldg(g.cu + g.N), a), g.T);
  const long long units = dv / unit, per = g.H * units, n = (a + static_cast<long long>(g.T - b)) * per;
  for (long long i = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x; i < n;
       i += static_cast<long long>(gridDim.x) * blockDim.x) {
    const long long row = i / per, at = i - row * per, h = at / units;
    *reinterpret_cast<uint4*>(o + h * oh + (row < a ? row : row - a + b) * ot + (at - h * units) * unit) =
        make_uint4(0u, 0u, 0u, 0u);
  }
}

// Segment s counted over all sequences; called by whole warps.
__device__ __forceinline__ DecaySpan decay_span(const DecayGeom& g, int s) {
  DecaySpan r;
  r.seq = -1;
  r.batch = r.row0 = r.len = r.j = r.nseg = 0;
  r.slot = s;
  if (!g.cu) {
    const int per = decay_segments(g.T, g.S);
    if (s >= g.N * per) return r;
    r.seq = r.batch = s / per;
    r.j = s % per;
    r.nseg = per;
    r.row0 = r.j * g.S;
    r.len = min(g.S, g.T - r.row0);
    return r;
  }
  const int lane = threadIdx.x & 31;
  int before = 0;  // segments of the sequences before n0
  int single = 0;  // sequences among them that are one segment, which has no slot
  for (int n0 = 0; n0 < g.N; n0 += 32) {
    const int n = n0 + lane;
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
    const unsigned hit = __ballot_sync(0xffffffffu, before + incl > s), one = __ballot_sync(0xffffffffu, c == 1 && !g.all);
    if (hit) {
      const int f = __ffs(hit) - 1;
      r.slot = s - single - __popc(one & ((1u << f) - 1u));
      a = __shfl_sync(0xffffffffu, a, f);
      b = __shfl_sync(0xffffffffu, b, f);
      c = __shfl_sync(0xffffffffu, c, f);
      incl = __shfl_sync(0xffffffffu, incl, f);
      r.seq = n0 + f;
      r.j = s - (before + incl - c);
      r.nseg = c;
      r.row0 = a + r.j * g.S;
      r.len = min(g.S, b - r.row0);
      if ((c > 1 || g.all) && r.slot >= g.slots) r.seq = -1;
      return r;
    }
    before += __shfl_sync(0xffffffffu, incl, 31);
    single += __popc(one);
  }
  return r;
}

// The first slot of sequence n, at most `slots`; whole warps.
__device__ __forceinline__ int decay_first_slot(const DecayGeom& g, int n) {
  if (!g.cu) return n * decay_segments(g.T, g.S);
  int c = 0;
  for (int m = threadIdx.x & 31; m < n; m += 32) {
    int a, b;
    decay_rows(g, m, a, b);
    const int x = decay_segments(b - a, g.S);
    if (x > 1 || g.all) c = min(c + x, g.slots);  // (at most 2^25 each: no overflow whatever the offsets)
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) c = min(c + __shfl_xor_sync(0xffffffffu, c, off), g.slots);
  return c;
}

// log gamma of head h.  -inf (gamma = 0: every token forgets all earlier ones)
// is taken as -1e4, whose powers are 0 in fp32 from the first on while the
// power 0 stays 1, where -inf * 0 would be NaN.
__device__ __forceinline__ float decay_log(const float* log_decay, int h) {
  const float x = __ldg(log_decay + h);
  return x < -1e4f ? -1e4f : x;
}

struct DecayTensor {
  const void* p;
  long long sb, sh, st;  // elements between sequences, heads, tokens
};

// One run of the recurrence over every (segment, head).
struct DecayRun {
  DecayTensor q, k, v, o;
  int dk, dv;              // features of k (and q), of v (and o)
  int rev;
  float sP, sR, sU;
  const float* s_in;       // [N][H][dv][dk], or [N][H][dk][dv] where s_in_t; nullptr: zeros
  int s_in_t;
  float* s_out;            // [N][H][dv][dk] or nullptr
  float* ws;               // [slots][H][dv][dk]: segments' contributions, then start states; nullptr: one segment each
  int clear;               // zeros for o's rows in no (packed) sequence
};

// The state that a segment's block starts from: the caller's where the
// sequence is a single segment, else the scan's.
__device__ __forceinline__ const float* decay_start(const DecayRun& p, const DecaySpan& sp, int H, int h,
                                                    bool* transposed) {
  const size_t dd = static_cast<size_t>(p.dv) * p.dk;
  *transposed = false;
  if (sp.nseg > 1) return p.ws + (static_cast<size_t>(sp.slot) * H + h) * dd;
  if (!p.s_in) return nullptr;
  *transposed = p.s_in_t != 0;
  return p.s_in + (static_cast<size_t>(sp.seq) * H + h) * dd;
}

// --------------------------------------------------------------- scan ----
// In place over ws: the contribution of each segment of a sequence becomes the
// state the segment starts from.  One thread per 4 elements of a (sequence,
// head)'s state, all segments in order (reverse runs: last to first); four
// loads are in flight at a time, since each is a round trip to L2.  FINAL: the
// last segment walked has left its contribution too, and the state behind it
// goes to s_out; `all` takes in sequences of one segment.
struct DecayScan {
  DecayGeom g;
  int dk, dv, rev;
  const float* s_in;  // [N][H][dv][dk], or [N][H][dk][dv] where s_in_t; nullptr: zeros
  int s_in_t;
  float* s_out;       // or nullptr
  float* ws;
  int all;
};
struct DecayScans {
  DecayScan s[2];  // one per blockIdx.y
};

template <bool FINAL>
__global__ void __launch_bounds__(256) decay_scan_kernel(const DecayScans ps, const float* __restrict__ log_decay) {
  const DecayScan& p = ps.s[blockIdx.y];
  const DecayGeom& g = p.g;
  launch_next();
  wait_before();
  const size_t dd = static_cast<size_t>(p.dv) * p.dk;
  const int slices = static_cast<int>((dd / 4 + blockDim.x - 1) / blockDim.x);
  const int h = (blockIdx.x / slices) % g.H, n = blockIdx.x / slices / g.H;
  int a, b;
  decay_rows(g, n, a, b);
  const int len = b - a, nseg = decay_segments(len, g.S);
  if (nseg <= 1 && !p.all) return;
  const int first = decay_first_slot(g, n);
  const size_t e = (static_cast<size_t>(blockIdx.x % slices) * blockDim.x + threadIdx.x) * 4;
  if (e >= dd) return;
  const float l = decay_log(log_decay, h);
  const float gS = expf(l * static_cast<float>(g.S));
  const float gL = expf(l * static_cast<float>(len - (nseg - 1) * g.S));  // the last segment's
  float4 run = make_float4(0.f, 0.f, 0.f, 0.f);
  if (p.s_in) {
    const float* s = p.s_in + (static_cast<size_t>(n) * g.H + h) * dd;
    if (p.s_in_t) {
      const size_t r = e / p.dk, c = e % p.dk;
      run = make_float4(s[c * p.dv + r], s[(c + 1) * p.dv + r], s[(c + 2) * p.dv + r], s[(c + 3) * p.dv + r]);
    } else {
      run = *reinterpret_cast<const float4*>(s + e);
    }
  }
  const size_t pitch = static_cast<size_t>(g.H) * dd;
  float* w = p.ws + (static_cast<size_t>(first) * g.H + h) * dd + e;
  const int sums = FINAL && p.s_out ? nseg : nseg - 1;  // contributions that are there
  constexpr int U = 4;
  for (int i0 = 0; i0 < nseg; i0 += U) {
    float4 t[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u, j = p.rev ? nseg - 1 - i : i;
      if (i < sums && first + j < g.slots) t[u] = ld_after(reinterpret_cast<const float4*>(w + j * pitch));
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u, j = p.rev ? nseg - 1 - i : i;
      if (i < nseg && first + j < g.slots) {
        __stcg(reinterpret_cast<float4*>(w + j * pitch), run);
        if (i < sums) {
          const float f = (j == nseg - 1) ? gL : gS;
          run.x = fmaf(f, run.x, t[u].x);
          run.y = fmaf(f, run.y, t[u].y);
          run.z = fmaf(f, run.z, t[u].z);
          run.w = fmaf(f, run.w, t[u].w);
        }
      }
    }
  }
  if (FINAL && p.s_out) *reinterpret_cast<float4*>(p.s_out + (static_cast<size_t>(n) * g.H + h) * dd + e) = run;
}

// ---------------------------------------------------------- fp32 FMA ----
// The run in fp32 FMA, for fp32 inputs and for widths that the tensor-core
// kernel does not have.  A block owns 32 rows of the state (features of v) of
// one (segment, head) and walks the segment in tiles of 32 tokens: Q, K, V,
// the weighted scores and the state stay in shared memory, products are taken
// in 2 x 2 and RT x 4 register tiles over 16-byte shared loads (rows padded by
// 4 floats: 8 rows cover the 32 banks).  Bound by FMA issue, not by memory: 1 x
// 2 x 256 x 32 takes 25 us in four segments a head, launches and host included.
// TOT: only the segment's contribution to the state, into ws.
constexpr int kDecayC = 32, kDecayVT = 32;
inline int decay_simt_smem(int dk) {
  const int ld = dk + 4;
  return (2 * kDecayC * ld + kDecayVT * ld + kDecayC * (kDecayVT + 4) + kDecayC * (kDecayC + 1) + kDecayC + 1) * 4;
}

__device__ __forceinline__ float dot4(float4 a, float4 b, float c) {
  return fmaf(a.x, b.x, fmaf(a.y, b.y, fmaf(a.z, b.z, fmaf(a.w, b.w, c))));
}

template <int N>
struct Rows {
  static constexpr int value = N;
};

template <typename T, bool TOT>
__global__ void __launch_bounds__(256) decay_simt_kernel(const DecayGeom g, const DecayRun p,
                                                         const float* __restrict__ log_decay) {
  constexpr int C = kDecayC, VT = kDecayVT, LDV = VT + 4, LDP = C + 1;
  extern __shared__ __align__(16) float sm[];
  const int dk = p.dk, dv = p.dv, ld = dk + 4;
  float* Qs = sm;
  float* Ks = Qs + C * ld;
  float* Ws = Ks + C * ld;
  float* Vs = Ws + VT * ld;
  float* Ps = Vs + C * LDV;
  float* gp = Ps + C * LDP;  // gamma^0 .. gamma^C

  const int nvt = (dv + VT - 1) / VT;
  const int vt = blockIdx.x % nvt, h = (blockIdx.x / nvt) % g.H, s = blockIdx.x / nvt / g.H;
  if (!TOT && p.clear) decay_clear_rest(g, static_cast<T*>(const_cast<void*>(p.o.p)), p.o.sh, p.o.st, dv);
  const DecaySpan sp = decay_span(g, s);
  if (sp.seq < 0) return;
  if (TOT && (sp.nseg <= 1 || sp.j == (p.rev ? 0 : sp.nseg - 1))) return;
  const int v0 = vt * VT, nv0 = min(VT, dv - v0);  // rows of the state here
  const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
  const size_t dd = static_cast<size_t>(dv) * dk;
  const float l = decay_log(log_decay, h);

  if (tid <= C) gp[tid] = expf(l * static_cast<float>(tid));
  bool tr = false;
  const float* s0 = TOT ? nullptr : decay_start(p, sp, g.H, h, &tr);
  for (int i = tid; i < VT * dk; i += 256) {
    const int r = i / dk, c = i % dk;
    float x = 0.f;
    if (s0 && r < nv0) x = tr ? s0[static_cast<size_t>(c) * dv + v0 + r] : s0[static_cast<size_t>(v0 + r) * dk + c];
    Ws[r * ld + c] = x;
  }
  auto base = [&](const DecayTensor& t) {
    return static_cast<const T*>(t.p) + static_cast<size_t>(sp.batch) * t.sb + static_cast<size_t>(h) * t.sh +
           static_cast<size_t>(sp.row0) * t.st;
  };
  const T *qg = base(p.q), *kg = base(p.k), *vg = base(p.v) + v0;
  T* og = const_cast<T*>(base(p.o)) + v0;

  const int tiles = (sp.len + C - 1) / C;
  auto tile_at = [&](int it) { return (p.rev ? tiles - 1 - it : it) * C; };
  // up to 64 wide, the next tile's loads are in flight while this one is worked on
  const bool ahead = dk <= 64;
  float4 nk[2], nq[2], nv;
  const int k4 = dk / 4;
  auto fetch = [&](int it) {
    const int t0 = tile_at(it), n = min(C, sp.len - t0);
    const float4 z = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int i = tid + 256 * x, r = i / k4, c = (i - r * k4) * 4;
      nk[x] = nq[x] = z;
      if (i < C * k4 && r < n) {
        nk[x] = load4(kg + static_cast<size_t>(t0 + r) * p.k.st + c);
        if (!TOT) nq[x] = load4(qg + static_cast<size_t>(t0 + r) * p.q.st + c);
      }
    }
    const int r = tid >> 3, c = (tid & 7) * 4;
    nv = r < n && c < nv0 ? load4(vg + static_cast<size_t>(t0 + r) * p.v.st + c) : z;
  };
  if (ahead && tiles > 0) fetch(0);
  for (int it = 0; it < tiles; ++it) {
    const int t0 = tile_at(it), n = min(C, sp.len - t0);
    __syncthreads();
    if (ahead) {
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int i = tid + 256 * x, r = i / k4, c = (i - r * k4) * 4;
        if (i < C * k4) {
          *reinterpret_cast<float4*>(Ks + r * ld + c) = nk[x];
          if (!TOT) *reinterpret_cast<float4*>(Qs + r * ld + c) = nq[x];
        }
      }
      *reinterpret_cast<float4*>(Vs + (tid >> 3) * LDV + (tid & 7) * 4) = nv;
      if (it + 1 < tiles) fetch(it + 1);
    } else {
      for (int i = tid; i < C * k4; i += 256) {
        const int r = i / k4, c = (i % k4) * 4;
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f), y = x;
        if (r < n) {
          x = load4(kg + static_cast<size_t>(t0 + r) * p.k.st + c);
          if (!TOT) y = load4(qg + static_cast<size_t>(t0 + r) * p.q.st + c);
        }
        *reinterpret_cast<float4*>(Ks + r * ld + c) = x;
        if (!TOT) *reinterpret_cast<float4*>(Qs + r * ld + c) = y;
      }
      const int r = tid >> 3, c = (tid & 7) * 4;
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
      if (r < n && c < nv0) x = load4(vg + static_cast<size_t>(t0 + r) * p.v.st + c);
      *reinterpret_cast<float4*>(Vs + r * LDV + c) = x;
    }
    __syncthreads();
    if (!TOT) {
      // scores, masked and weighted; rows ty, ty + 16, columns tx, tx + 16
      float a00 = 0.f, a01 = 0.f, a10 = 0.f, a11 = 0.f;
      for (int c = 0; c < dk; c += 4) {
        const float4 q0 = *reinterpret_cast<const float4*>(Qs + ty * ld + c);
        const float4 q1 = *reinterpret_cast<const float4*>(Qs + (ty + 16) * ld + c);
        const float4 k0 = *reinterpret_cast<const float4*>(Ks + tx * ld + c);
        const float4 k1 = *reinterpret_cast<const float4*>(Ks + (tx + 16) * ld + c);
        a00 = dot4(q0, k0, a00);
        a01 = dot4(q0, k1, a01);
        a10 = dot4(q1, k0, a10);
        a11 = dot4(q1, k1, a11);
      }
      auto weigh = [&](int r, int c, float x) {
        const int d = p.rev ? c - r : r - c;
        Ps[r * LDP + c] = d >= 0 ? p.sP * gp[d] * x : 0.f;
      };
      weigh(ty, tx, a00);
      weigh(ty, tx + 16, a01);
      weigh(ty + 16, tx, a10);
      weigh(ty + 16, tx + 16, a11);
      __syncthreads();
      float o00 = 0.f, o01 = 0.f, o10 = 0.f, o11 = 0.f;
      for (int c = 0; c < dk; c += 4) {
        const float4 q0 = *reinterpret_cast<const float4*>(Qs + ty * ld + c);
        const float4 q1 = *reinterpret_cast<const float4*>(Qs + (ty + 16) * ld + c);
        const float4 w0 = *reinterpret_cast<const float4*>(Ws + tx * ld + c);
        const float4 w1 = *reinterpret_cast<const float4*>(Ws + (tx + 16) * ld + c);
        o00 = dot4(q0, w0, o00);
        o01 = dot4(q0, w1, o01);
        o10 = dot4(q1, w0, o10);
        o11 = dot4(q1, w1, o11);
      }
      // (rows past n have no read-out power: n - 1 - r would be negative)
      auto read_power = [&](int r) { return r < n ? p.sR * gp[p.rev ? n - 1 - r : r + 1] : 0.f; };
      const float r0 = read_power(ty), r1 = read_power(ty + 16);
      o00 *= r0, o01 *= r0, o10 *= r1, o11 *= r1;
#pragma unroll 8
      for (int c = 0; c < C; ++c) {
        const float x0 = Ps[ty * LDP + c], x1 = Ps[(ty + 16) * LDP + c];
        const float y0 = Vs[c * LDV + tx], y1 = Vs[c * LDV + tx + 16];
        o00 = fmaf(x0, y0, o00);
        o01 = fmaf(x0, y1, o01);
        o10 = fmaf(x1, y0, o10);
        o11 = fmaf(x1, y1, o11);
      }
      auto put = [&](int r, int c, float x) {
        if (r < n && c < nv0) og[static_cast<size_t>(t0 + r) * p.o.st + c] = from_f<T>(x);
      };
      put(ty, tx, o00);
      put(ty, tx + 16, o01);
      put(ty + 16, tx, o10);
      put(ty + 16, tx + 16, o11);
      __syncthreads();  // the state is read above
    }
    // state: RT rows x 4 columns a thread, so that all threads have work at every width
    const float gn = gp[n];
    auto update = [&](auto rows) {
      constexpr int RT = decltype(rows)::value;
      for (int e = tid; e < (VT / RT) * k4; e += 256) {
        const int r = e / k4 * RT, c = (e % k4) * 4;
        float4 w[RT];
#pragma unroll
        for (int i = 0; i < RT; ++i) w[i] = f4_scale(gn, *reinterpret_cast<const float4*>(Ws + (r + i) * ld + c));
#pragma unroll 8
        for (int j = 0; j < n; ++j) {
          const float u = p.sU * gp[p.rev ? j + 1 : n - 1 - j];
          const float4 kk = f4_scale(u, *reinterpret_cast<const float4*>(Ks + j * ld + c));
#pragma unroll
          for (int i = 0; i < RT; ++i) {
            const float va = Vs[j * LDV + r + i];
            w[i].x = fmaf(va, kk.x, w[i].x);
            w[i].y = fmaf(va, kk.y, w[i].y);
            w[i].z = fmaf(va, kk.z, w[i].z);
            w[i].w = fmaf(va, kk.w, w[i].w);
          }
        }
#pragma unroll
        for (int i = 0; i < RT; ++i) *reinterpret_cast<float4*>(Ws + (r + i) * ld + c) = w[i];
      }
    };
    if (dk <= 32)
      update(Rows<1>{});
    else if (dk <= 64)
      update(Rows<2>{});
    else
      update(Rows<4>{});
  }
  __syncthreads();
  float* dst = nullptr;
  if (TOT)
    dst = p.ws + (static_cast<size_t>(sp.slot) * g.H + h) * dd;
  else if (p.s_out && sp.j == (p.rev ? 0 : sp.nseg - 1))
    dst = p.s_out + (static_cast<size_t>(sp.seq) * g.H + h) * dd;
  if (dst)
    for (int i = tid; i < nv0 * dk; i += 256) {
      const int r = i / dk, c = i % dk;
      dst[static_cast<size_t>(v0 + r) * dk + c] = Ws[r * ld + c];
    }
}

// ---------------------------------------------------------- one token ----
// The step for one new token of each of N sequences, the state in place.
// As in decode.cuh the rows of all states form one list of N H d_v rows of d_k
// floats, a row owned by d_k / 4 consecutive lanes; W is read once and written
// once in 16-byte streaming accesses, U of them in flight per lane.  Where a
// warp's U accesses lie in one (sequence, head), as they do for every d_v that
// is a multiple of their rows, q, k and gamma are fetched once for all of them.
// Bound by HBM: 83 us for 544 MB (256 sequences x 16 heads x 128 x 128), the
// measured copy rate.
struct DecayStep {
  int N, H, dk, dv;
  DecayTensor q, k, v, o;  // sb: between sequences, sh: between heads
  const float* log_decay;
  float a;
  float* S;
};

template <int DK, typename T, int U>
__global__ void __launch_bounds__(256) decay_step_kernel(const DecayStep p) {
  constexpr int TPR = DK / 4, RPW = 32 / TPR, STEP = RPW * U;
  const int lane = threadIdx.x & 31, sub = lane / TPR, c4 = lane % TPR;
  const int rows = p.N * p.H * p.dv;  // host guarantees < 2^31 - 2^20, so `base` does not wrap
  const int base = static_cast<int>((static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5) * STEP;
  if (base >= rows) return;
  struct Head {
    float4 k, q;
    float g;
    const T* v;
    T* o;
  };
  auto head_of = [&](int nh) {
    const int n = nh / p.H, h = nh - n * p.H;
    Head x;
    x.k = load4(static_cast<const T*>(p.k.p) + n * p.k.sb + h * p.k.sh + 4 * c4);
    x.q = load4(static_cast<const T*>(p.q.p) + n * p.q.sb + h * p.q.sh + 4 * c4);
    x.v = static_cast<const T*>(p.v.p) + n * p.v.sb + h * p.v.sh;
    x.o = static_cast<T*>(const_cast<void*>(p.o.p)) + n * p.o.sb + h * p.o.sh;
    x.g = decay_log(p.log_decay, h);
    return x;
  };
  // one row: the state's new values and their share of o
  auto step = [&](const Head& x, float gamma, float v, float4& s) {
    const float a = p.a * v;
    s.x = fmaf(gamma, s.x, a * x.k.x);
    s.y = fmaf(gamma, s.y, a * x.k.y);
    s.z = fmaf(gamma, s.z, a * x.k.z);
    s.w = fmaf(gamma, s.w, a * x.k.w);
    return dot4(s, x.q, 0.f);
  };
  float4 w[U];
  float4* W = reinterpret_cast<float4*>(p.S) + static_cast<size_t>(base + sub) * TPR + c4;
  const int nh = base / p.dv, f = base - nh * p.dv;
  if (f + STEP <= p.dv) {  // (then every row is there, too)
#pragma unroll
    for (int u = 0; u < U; ++u) w[u] = __ldcs(W + u * 32);
    const Head x = head_of(nh);
    float v[U], dot[U];
#pragma unroll
    for (int u = 0; u < U; ++u) v[u] = to_f(x.v[f + u * RPW + sub]);
    const float gamma = expf(x.g);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      dot[u] = step(x, gamma, v[u], w[u]);
      __stcs(W + u * 32, w[u]);
    }
#pragma unroll
    for (int off = TPR / 2; off > 0; off >>= 1)
#pragma unroll
      for (int u = 0; u < U; ++u) dot[u] += __shfl_xor_sync(0xffffffffu, dot[u], off);
    if (c4 == 0)
#pragma unroll
      for (int u = 0; u < U; ++u) x.o[f + u * RPW + sub] = from_f<T>(dot[u]);
  } else {
#pragma unroll 1
    for (int u = 0; u < U; ++u) {
      const int row = base + u * RPW + sub;
      float dot = 0.f;
      T* dst = nullptr;
      if (row < rows) {
        const int m = row / p.dv, e = row - m * p.dv;
        const Head x = head_of(m);
        w[0] = __ldcs(W + u * 32);
        dot = step(x, expf(x.g), to_f(x.v[e]), w[0]);
        __stcs(W + u * 32, w[0]);
        dst = x.o + e;
      }
#pragma unroll
      for (int off = TPR / 2; off > 0; off >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, off);
      if (row < rows && c4 == 0) *dst = from_f<T>(dot);
    }
  }
}

}  // namespace ttt
