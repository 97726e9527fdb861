// group_norm_host.cuh -- C ABI of the group norm (ttt_la_group_norm,
// ttt_la_group_norm_backward): checks, plan, launches.  Included by ttt_la.cu,
// whose host helpers it uses.
#pragma once

namespace {

// Values per thread unit: the most of 16 bytes that lie in one group.
int gn_unit(int cg, int dtype) {
  for (int v = dtype == TTT_LA_F32 ? 4 : 8; v > 1; v /= 2)
    if (cg % v == 0) return v;
  return 1;
}
// One position a sample and a group of at most a warp's units, a power of two
// of them: the registers-only kernels.
int gn_row_lanes(int L, int cg, int dtype) {
  const int v = gn_unit(cg, dtype), lanes = cg / v;
  return L == 1 && v == (dtype == TTT_LA_F32 ? 4 : 8) && lanes <= 32 && (lanes & (lanes - 1)) == 0 ? lanes : 0;
}

struct GnPlan {
  int lanes;         // > 0: the one-position kernels
  int splits, rows;  // parts of a sample and the positions in each
  int blocks;        // row blocks of the one-position gradient
  size_t floats;     // workspace
};

// Enough parts that all samples together fill the SMs a few times over, none
// with so few positions that a block's joins cost more than its reads.
void gn_split(GnPlan* p, int N, int L, int C, int dtype) {
  const long long want = std::max(1ll, (static_cast<long long>(sm_count()) * 8 + N - 1) / N);
  const long long row_bytes = static_cast<long long>(C) * (dtype == TTT_LA_F32 ? 4 : 2);
  const long long least = std::max(1ll, 16384 / row_bytes);
  p->rows = static_cast<int>(std::max(least, (L + want - 1) / want));
  p->rows = std::min(p->rows, L);
  p->splits = (L - 1) / p->rows + 1;
}

GnPlan gn_plan_forward(int N, int L, int C, int G, int dtype) {
  GnPlan p = {};
  p.lanes = gn_row_lanes(L, C / G, dtype);
  if (p.lanes) return p;
  gn_split(&p, N, L, C, dtype);
  p.floats = static_cast<size_t>(N) * p.splits * G * 2;
  return p;
}
GnPlan gn_plan_backward(int N, int L, int C, int G, int dtype, bool params) {
  GnPlan p = {};
  p.lanes = gn_row_lanes(L, C / G, dtype);
  if (p.lanes) {
    const int cv = C / gn_unit(C / G, dtype), cols = (cv + 255) / 256, slots = cv < 256 ? 256 / cv : 1;
    p.blocks = static_cast<int>(std::min<long long>((N + slots - 1) / slots, std::max(1, sm_count() * 4 / cols)));
    p.floats = params ? static_cast<size_t>(2) * p.blocks * C : 0;
    return p;
  }
  gn_split(&p, N, L, C, dtype);
  p.floats = static_cast<size_t>(2) * N * p.splits * C + static_cast<size_t>(2) * N * G;
  return p;
}

ttt_la_status check_gn(int N, int L, int C, int G, int dtype, int param_dtype, int act) {
  if (N < 1 || L < 1 || C < 1 || G < 1 || C % G) return TTT_LA_ERR_INVALID_ARG;
  if ((dtype != TTT_LA_F32 && dtype != TTT_LA_BF16) || (param_dtype != TTT_LA_F32 && param_dtype != TTT_LA_BF16))
    return TTT_LA_ERR_INVALID_ARG;
  if (act != 0 && act != 1) return TTT_LA_ERR_INVALID_ARG;
  if (static_cast<long long>(N) * L > (1ll << 40) / C) return TTT_LA_ERR_INVALID_ARG;
  // rows of a sample start on 16 bytes, and a block's table of the groups fits in shared memory
  if (C % (dtype == TTT_LA_F32 ? 4 : 8) || G > 4096) return TTT_LA_ERR_UNSUPPORTED;
  return TTT_LA_OK;
}

bool gn_aligned(const void* p, int dtype) { return reinterpret_cast<uintptr_t>(p) % (dtype == TTT_LA_F32 ? 4 : 2) == 0; }

template <typename F>
ttt_la_status gn_dispatch(int dtype, int v, bool gate, F&& f) {
  // f(type tag, unit, gate)
  auto by_gate = [&](auto t, auto u) {
    return gate ? f(t, u, std::true_type{}) : f(t, u, std::false_type{});
  };
  if (dtype == TTT_LA_F32) {
    if (v == 4) return by_gate(float{}, std::integral_constant<int, 4>{});
    if (v == 2) return by_gate(float{}, std::integral_constant<int, 2>{});
    return by_gate(float{}, std::integral_constant<int, 1>{});
  }
  using bf = __nv_bfloat16;
  if (v == 8) return by_gate(bf{}, std::integral_constant<int, 8>{});
  if (v == 4) return by_gate(bf{}, std::integral_constant<int, 4>{});
  if (v == 2) return by_gate(bf{}, std::integral_constant<int, 2>{});
  return by_gate(bf{}, std::integral_constant<int, 1>{});
}

}  // namespace

extern "C" {

size_t ttt_la_group_norm_workspace_size(const ttt_la_group_norm_args* a) {
  if (!a || check_gn(a->N, a->L, a->C, a->G, a->dtype, a->param_dtype, a->activation) != TTT_LA_OK) return 0;
  return gn_plan_forward(a->N, a->L, a->C, a->G, a->dtype).floats * sizeof(float);
}

ttt_la_status ttt_la_group_norm(const ttt_la_group_norm_args* a, void* stream) {
  NvtxRange range("ttt_la_group_norm");
  if (!a) return TTT_LA_ERR_INVALID_ARG;
  ttt_la_status s = check_gn(a->N, a->L, a->C, a->G, a->dtype, a->param_dtype, a->activation);
  if (s != TTT_LA_OK) return s;
  if (!a->x || !a->y || !a->mean || !a->rstd || !aligned16(a->x) || !aligned16(a->y) || !aligned16(a->gate) ||
      !gn_aligned(a->weight, a->param_dtype) || !gn_aligned(a->bias, a->param_dtype) ||
      !gn_aligned(a->mean, TTT_LA_F32) || !gn_aligned(a->rstd, TTT_LA_F32))
    return TTT_LA_ERR_INVALID_ARG;
  if (!(a->eps >= 0.f) || a->y == a->x || a->y == a->gate) return TTT_LA_ERR_INVALID_ARG;
  const GnPlan pl = gn_plan_forward(a->N, a->L, a->C, a->G, a->dtype);
  if (pl.floats && (!a->workspace || !aligned16(a->workspace) || a->workspace_bytes < pl.floats * sizeof(float)))
    return TTT_LA_ERR_INVALID_ARG;
  ttt::GnParams p = {};
  p.N = a->N, p.L = a->L, p.C = a->C, p.G = a->G, p.cg = a->C / a->G;
  p.x = a->x, p.gate = a->gate, p.weight = a->weight, p.bias = a->bias;
  p.pbf = a->param_dtype == TTT_LA_BF16;
  p.act = a->activation, p.eps = a->eps;
  p.y = a->y, p.mean = a->mean, p.rstd = a->rstd;
  p.part = static_cast<float*>(a->workspace);
  p.splits = pl.splits, p.rows = pl.rows;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int v = gn_unit(p.cg, a->dtype);
  return gn_dispatch(a->dtype, v, a->gate != nullptr, [&](auto t, auto u, auto gate) -> ttt_la_status {
    using T = decltype(t);
    constexpr int V = decltype(u)::value;
    constexpr bool GATE = decltype(gate)::value;
    if (pl.lanes) {
      const long long units = static_cast<long long>(a->N) * (a->C / V);
      const int blocks = static_cast<int>(std::min<long long>((units + 255) / 256, static_cast<long long>(sm_count()) * 32));
      return launch_kernel(ttt::gn_row_kernel<T, V, GATE>, blocks, 256, 0, st, false, p, pl.lanes);
    }
    const long long blocks = static_cast<long long>(a->N) * pl.splits;
    if (blocks >= (1ll << 31)) return TTT_LA_ERR_UNSUPPORTED;
    const int sm1 = a->G * static_cast<int>(sizeof(ttt::Moments)), sm2 = a->G * 8;
    if (!grant_smem(reinterpret_cast<const void*>(ttt::gn_stats_kernel<T, V>), sm1)) return TTT_LA_ERR_CUDA;
    const ttt_la_status r = launch_kernel(ttt::gn_stats_kernel<T, V>, static_cast<int>(blocks), 256, sm1, st, false, p);
    if (r != TTT_LA_OK) return r;
    return launch_kernel(ttt::gn_apply_kernel<T, V, GATE>, static_cast<int>(blocks), 256, sm2, st, false, p);
  });
}

size_t ttt_la_group_norm_backward_workspace_size(const ttt_la_group_norm_grad_args* a) {
  if (!a || check_gn(a->N, a->L, a->C, a->G, a->dtype, a->param_dtype, a->activation) != TTT_LA_OK) return 0;
  return gn_plan_backward(a->N, a->L, a->C, a->G, a->dtype, a->grad_weight || a->grad_bias).floats * sizeof(float);
}

ttt_la_status ttt_la_group_norm_backward(const ttt_la_group_norm_grad_args* a, void* stream) {
  NvtxRange range("ttt_la_group_norm_backward");
  if (!a) return TTT_LA_ERR_INVALID_ARG;
  ttt_la_status s = check_gn(a->N, a->L, a->C, a->G, a->dtype, a->param_dtype, a->activation);
  if (s != TTT_LA_OK) return s;
  const void* ptr[] = {a->grad_y, a->x, a->gate, a->weight, a->bias, a->mean, a->rstd, a->grad_x, a->grad_gate,
                       a->grad_weight, a->grad_bias};
  const int per[] = {-1, -1, -1, a->param_dtype, a->param_dtype, TTT_LA_F32, TTT_LA_F32, -1, -1, a->param_dtype,
                     a->param_dtype};  // read or written one value at a time, in this type
  for (int i = 0; i < 11; ++i)
    if (per[i] < 0 ? !aligned16(ptr[i]) : !gn_aligned(ptr[i], per[i])) return TTT_LA_ERR_INVALID_ARG;
  if (!a->grad_y || !a->x || !a->mean || !a->rstd || !a->grad_x || (a->gate && !a->grad_gate))
    return TTT_LA_ERR_INVALID_ARG;
  for (int i = 7; i < 11; ++i)  // an output is neither an input nor another output
    for (int j = 0; j < i; ++j)
      if (ptr[i] && ptr[i] == ptr[j]) return TTT_LA_ERR_INVALID_ARG;
  const bool params = a->grad_weight || a->grad_bias;
  const GnPlan pl = gn_plan_backward(a->N, a->L, a->C, a->G, a->dtype, params);
  if (pl.floats && (!a->workspace || !aligned16(a->workspace) || a->workspace_bytes < pl.floats * sizeof(float)))
    return TTT_LA_ERR_INVALID_ARG;
  ttt::GnParams p = {};
  p.N = a->N, p.L = a->L, p.C = a->C, p.G = a->G, p.cg = a->C / a->G;
  p.x = a->x, p.gate = a->gate, p.weight = a->weight, p.bias = a->bias;
  p.pbf = a->param_dtype == TTT_LA_BF16;
  p.act = a->activation;
  p.mean = const_cast<float*>(a->mean), p.rstd = const_cast<float*>(a->rstd);
  p.gy = a->grad_y, p.gx = a->grad_x, p.ggate = a->grad_gate;
  p.part = pl.floats ? static_cast<float*>(a->workspace) : nullptr;
  p.splits = pl.splits, p.rows = pl.rows, p.blocks = pl.blocks;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int v = gn_unit(p.cg, a->dtype);
  return gn_dispatch(a->dtype, v, a->gate != nullptr, [&](auto t, auto u, auto gate) -> ttt_la_status {
    using T = decltype(t);
    constexpr int V = decltype(u)::value;
    constexpr bool GATE = decltype(gate)::value;
    ttt_la_status r = TTT_LA_OK;
    int count = 0;
    if (pl.lanes) {
      const dim3 grid((a->C / V + 255) / 256, pl.blocks);
      ttt::gn_row_grad_kernel<T, V, GATE><<<grid, 256, 0, st>>>(p, pl.lanes);
      if ((r = launched()) != TTT_LA_OK) return r;
      count = pl.blocks;
    } else {
      const long long blocks = static_cast<long long>(a->N) * pl.splits;
      if (blocks >= (1ll << 31)) return TTT_LA_ERR_UNSUPPORTED;
      float* sums = p.part + static_cast<size_t>(2) * blocks * a->C;
      r = launch_kernel(ttt::gn_grad_sums_kernel<T, V, GATE>, static_cast<int>(blocks), 256, 0, st, false, p);
      if (r != TTT_LA_OK) return r;
      const long long warps = static_cast<long long>(a->N) * a->G;
      r = launch_kernel(ttt::gn_grad_groups_kernel, static_cast<int>((warps * 32 + 255) / 256), 256, 0, st, false, p, sums);
      if (r != TTT_LA_OK) return r;
      r = launch_kernel(ttt::gn_grad_apply_kernel<T, V, GATE>, static_cast<int>(blocks), 256, 0, st, false, p, sums);
      if (r != TTT_LA_OK) return r;
      count = static_cast<int>(blocks);
    }
    if (params) {
      ttt::gn_param_grad_kernel<<<dim3((a->C + 31) / 32, 2), 256, 0, st>>>(p.part, count, a->C, a->grad_weight,
                                                                          a->grad_bias, p.pbf);
      r = launched();
    }
    return r;
  });
}

}  // extern "C"
