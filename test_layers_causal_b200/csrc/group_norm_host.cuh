// group_norm_host.cuh -- C ABI of the group norm (ttt_la_group_norm,
// ttt_la_group_norm_backward): checks, plan, launches.  Included by ttt_la.cu,
// whose host helpers it uses.
#pragma once

namespace {

// Values a thread reads at once: 16 bytes, or one where rows do not all start
// on 16 bytes.
int gn_unit(int C, int dtype) {
  const int v = dtype == TTT_LA_F32 ? 4 : 8;
  return C % v == 0 ? v : 1;
}

// One position a sample and a group of 1, 2, 4 .. 32 units: the kernels that
// hold a group in registers.
int gn_row_lanes(int L, int cg, int dtype) {
  const int v = dtype == TTT_LA_F32 ? 4 : 8, lanes = cg / v;
  return L == 1 && cg % v == 0 && lanes <= 32 && (lanes & (lanes - 1)) == 0 ? lanes : 0;
}

struct GnPlan {
  int lanes;               // > 0: the one-position kernels
  int width, slots;        // of those: units of a row in a block, rows at a time
  int columns, blocks;     // and their grid
  int per;                 // rows of a block
  int splits, rows;        // parts of a sample and the positions in each: sums
  int parts, part_rows;    // the same: writing passes
  size_t floats;           // workspace
};

// `per_sm` parts for each SM over all samples, none with so few positions that
// a block's sums cost more than its reads (16 KB).
void gn_split(int N, int L, int C, int dtype, int per_sm, int* parts, int* rows) {
  const long long want = std::max(1ll, static_cast<long long>(sm_count()) * per_sm / N);  // (one wave of blocks)
  const long long least = std::max(1ll, 16384 / (static_cast<long long>(C) * (dtype == TTT_LA_F32 ? 4 : 2)));
  *rows = static_cast<int>(std::min<long long>(std::max(least, (L + want - 1) / want), L));
  *parts = (L - 1) / *rows + 1;
}

// Blocks of up to 256 threads over the units of a row (wide rows in equal
// columns, narrow ones several at a time) and `per_sm` of them for each SM.
void gn_row_plan(GnPlan* p, int N, int C, int dtype, int per_sm) {
  const int cv = C / gn_unit(C, dtype);
  p->columns = (cv + 255) / 256;
  // (whole warps, so that a group's lanes stay in one)
  p->width = p->columns == 1 ? cv : ((cv + p->columns - 1) / p->columns + 31) / 32 * 32;
  p->columns = (cv + p->width - 1) / p->width;
  p->slots = std::max(1, 256 / p->width);
  // rows of a block: whole steps of `slots`, in one wave of `per_sm` blocks a SM
  const long long steps = (static_cast<long long>(N) + p->slots - 1) / p->slots;
  const long long want = std::max(1, sm_count() * per_sm / p->columns);
  p->per = static_cast<int>(std::min<long long>((steps + want - 1) / want * p->slots, N));
  p->blocks = (N - 1) / p->per + 1;
}

GnPlan gn_plan_forward(int N, int L, int C, int G, int dtype) {
  GnPlan p = {};
  p.lanes = gn_row_lanes(L, C / G, dtype);
  if (p.lanes) {
    gn_row_plan(&p, N, C, dtype, 4);
    return p;
  }
  gn_split(N, L, C, dtype, 3, &p.splits, &p.rows);
  gn_split(N, L, C, dtype, 6, &p.parts, &p.part_rows);
  p.floats = p.splits > 1 ? static_cast<size_t>(N) * p.splits * G * 2 : 0;
  return p;
}
GnPlan gn_plan_backward(int N, int L, int C, int G, int dtype, bool params) {
  GnPlan p = {};
  p.lanes = gn_row_lanes(L, C / G, dtype);
  if (p.lanes) {
    gn_row_plan(&p, N, C, dtype, 3);
    p.floats = params ? static_cast<size_t>(2) * p.blocks * C : 0;
    return p;
  }
  gn_split(N, L, C, dtype, 3, &p.splits, &p.rows);
  gn_split(N, L, C, dtype, 3, &p.parts, &p.part_rows);
  p.floats = static_cast<size_t>(2) * N * p.splits * C + static_cast<size_t>(2) * N * G;
  return p;
}

ttt_la_status check_gn(int N, int L, int C, int G, int dtype, int param_dtype, int act) {
  if (N < 1 || L < 1 || C < 1 || G < 1 || C % G) return TTT_LA_ERR_INVALID_ARG;
  if ((dtype != TTT_LA_F32 && dtype != TTT_LA_BF16) || (param_dtype != TTT_LA_F32 && param_dtype != TTT_LA_BF16))
    return TTT_LA_ERR_INVALID_ARG;
  if (act != 0 && act != 1) return TTT_LA_ERR_INVALID_ARG;
  if (static_cast<long long>(N) * L > (1ll << 40) / C) return TTT_LA_ERR_INVALID_ARG;
  if (G > 4096) return TTT_LA_ERR_UNSUPPORTED;  // a block's table of the groups fits in shared memory
  return TTT_LA_OK;
}

bool gn_aligned(const void* p, int dtype) { return reinterpret_cast<uintptr_t>(p) % (dtype == TTT_LA_F32 ? 4 : 2) == 0; }

template <typename F>
ttt_la_status gn_dispatch(int dtype, int unit, bool gate, bool act, F&& f) {
  // f(type tag, values of a unit, gate, silu)
  auto with = [&](auto t, auto u) {
    if (gate) return act ? f(t, u, std::true_type{}, std::true_type{}) : f(t, u, std::true_type{}, std::false_type{});
    return act ? f(t, u, std::false_type{}, std::true_type{}) : f(t, u, std::false_type{}, std::false_type{});
  };
  if (dtype == TTT_LA_F32)
    return unit > 1 ? with(float{}, std::integral_constant<int, 4>{}) : with(float{}, std::integral_constant<int, 1>{});
  using bf = __nv_bfloat16;
  return unit > 1 ? with(bf{}, std::integral_constant<int, 8>{}) : with(bf{}, std::integral_constant<int, 1>{});
}

void gn_fill(ttt::GnParams* p, const GnPlan& pl) {
  p->splits = pl.splits, p->rows = pl.rows, p->parts = pl.parts, p->part_rows = pl.part_rows;
  p->width = pl.width, p->slots = pl.slots, p->per = pl.per;
  p->limit_ns = g_limit_ns;
}
constexpr int kGnRing = ttt::kGnRingBytes;
// (granted with the kernels' own tables of up to 20 KB in mind, which count towards the 48 KB that need none)
template <typename K>
bool gn_grant(K kern, int bytes = kGnRing) {
  return grant_smem(reinterpret_cast<const void*>(kern), std::max(bytes, 49 * 1024));
}
int gn_row_threads(const GnPlan& pl) { return (pl.width * pl.slots + 31) / 32 * 32; }

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
  p.eps = a->eps;
  p.y = a->y, p.mean = a->mean, p.rstd = a->rstd;
  p.part = static_cast<float*>(a->workspace);
  gn_fill(&p, pl);
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  return gn_dispatch(a->dtype, gn_unit(a->C, a->dtype), a->gate != nullptr, a->activation == 1,
                     [&](auto t, auto u, auto gate, auto act) -> ttt_la_status {
    using T = decltype(t);
    constexpr int V = decltype(u)::value;
    constexpr bool GATE = decltype(gate)::value, ACT = decltype(act)::value;
    if constexpr (V > 1)
      if (pl.lanes) {
        if (!gn_grant(ttt::gn_row_kernel<T, V, GATE, ACT>)) return TTT_LA_ERR_CUDA;
        ttt::gn_row_kernel<T, V, GATE, ACT>
            <<<dim3(pl.columns, pl.blocks), gn_row_threads(pl), kGnRing, st>>>(p, pl.lanes);
        return launched();
      }
    const long long sums = static_cast<long long>(a->N) * pl.splits, parts = static_cast<long long>(a->N) * pl.parts;
    if (parts >= (1ll << 31) || sums >= (1ll << 31)) return TTT_LA_ERR_UNSUPPORTED;
    const int sm = a->G * static_cast<int>(sizeof(ttt::Moments));
    if (sm > 28 * 1024 && !gn_grant(ttt::gn_stats_kernel<T, V>, sm)) return TTT_LA_ERR_CUDA;
    ttt_la_status r = launch_kernel(ttt::gn_stats_kernel<T, V>, static_cast<int>(sums), 256, sm, st, false, p);
    if (r != TTT_LA_OK) return r;
    if (pl.splits > 1) {
      const long long warps = static_cast<long long>(a->N) * a->G;
      r = launch_after(ttt::gn_join_kernel, dim3(static_cast<unsigned>((warps + 7) / 8)), 256, 0, st, p);
      if (r != TTT_LA_OK) return r;
    }
    return launch_after(ttt::gn_apply_kernel<T, V, GATE, ACT>, dim3(static_cast<unsigned>(parts)), 256, 0, st, p);
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
  p.mean = const_cast<float*>(a->mean), p.rstd = const_cast<float*>(a->rstd);
  p.gy = a->grad_y, p.gx = a->grad_x, p.ggate = a->grad_gate;
  p.gw = a->grad_weight, p.gb = a->grad_bias;
  p.part = pl.floats ? static_cast<float*>(a->workspace) : nullptr;
  gn_fill(&p, pl);
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  return gn_dispatch(a->dtype, gn_unit(a->C, a->dtype), a->gate != nullptr, a->activation == 1,
                     [&](auto t, auto u, auto gate, auto act) -> ttt_la_status {
    using T = decltype(t);
    constexpr int V = decltype(u)::value;
    constexpr bool GATE = decltype(gate)::value, ACT = decltype(act)::value;
    if constexpr (V > 1)
      if (pl.lanes) {
        if (!gn_grant(ttt::gn_row_grad_kernel<T, V, GATE, ACT>)) return TTT_LA_ERR_CUDA;
        ttt::gn_row_grad_kernel<T, V, GATE, ACT>
            <<<dim3(pl.columns, pl.blocks), gn_row_threads(pl), kGnRing, st>>>(p, pl.lanes);
        const ttt_la_status r = launched();
        if (r != TTT_LA_OK || !params) return r;
        return launch_after(ttt::gn_param_grad_kernel, dim3((a->C + 31) / 32, 2), 256, 0, st,
                            static_cast<const float*>(p.part), pl.blocks, static_cast<int>(a->C), a->grad_weight,
                            a->grad_bias, p.pbf);
      }
    const long long rows = static_cast<long long>(a->N) * pl.splits, parts = static_cast<long long>(a->N) * pl.parts;
    if (parts >= (1ll << 31) || rows >= (1ll << 31)) return TTT_LA_ERR_UNSUPPORTED;
    float* sums = p.part + static_cast<size_t>(2) * rows * a->C;
    if (!gn_grant(ttt::gn_grad_sums_kernel<T, V, GATE, ACT>) || !gn_grant(ttt::gn_grad_apply_kernel<T, V, GATE, ACT>))
      return TTT_LA_ERR_CUDA;
    ttt_la_status r = launch_kernel(ttt::gn_grad_sums_kernel<T, V, GATE, ACT>, static_cast<int>(rows), 256, kGnRing, st, false, p);
    if (r != TTT_LA_OK) return r;
    const long long warp_blocks = (static_cast<long long>(a->N) * a->G + 7) / 8;
    const long long blocks = warp_blocks + (params ? 2 * ((a->C + 31) / 32) : 0);
    if (blocks >= (1ll << 31)) return TTT_LA_ERR_UNSUPPORTED;
    r = launch_after(ttt::gn_grad_groups_kernel, dim3(static_cast<unsigned>(blocks)), 256, 0, st, p, sums,
                     static_cast<int>(warp_blocks));
    if (r != TTT_LA_OK) return r;
    return launch_after(ttt::gn_grad_apply_kernel<T, V, GATE, ACT>, dim3(static_cast<unsigned>(parts)), 256, kGnRing, st, p,
                        static_cast<const float*>(sums));
  });
}

}  // extern "C"
