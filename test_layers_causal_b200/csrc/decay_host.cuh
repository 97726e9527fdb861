// decay_host.cuh -- C ABI of the decayed layer (ttt_la_forward_decay,
// ttt_la_backward_decay, ttt_la_decode_step_decay): checks, plan, launches.
// Included by ttt_la.cu, whose host helpers it uses.
#pragma once

namespace {

// Tokens per segment.  `rows` tokens of `heads` independent (sequence, head)
// runs are cut so that the launch fills the device's `slots` blocks: a wave
// takes as long as its longest segment, and cutting at all costs a pass over
// k and v for the segments' contributions (about half of the output pass, as
// it moves half the bytes) and a scan (about the time of kDecayScanTiles
// tiles).  Packed sequences are planned as one of their total length, since
// the host does not see where they end.
constexpr int kDecayTile = 64;
constexpr double kDecayTotalCost = 0.5, kDecayScanTiles = 0.75;
int decay_plan_tokens(long long heads, int rows, int slots) {
  const int tiles = (rows + kDecayTile - 1) / kDecayTile;
  int best = tiles;
  double cost = 1e30;
  for (int ns = 1; ns <= tiles && ns <= 1024; ++ns) {
    const int per = (tiles + ns - 1) / ns;
    const long long n = (tiles + per - 1) / per;
    auto waves = [&](long long blocks) { return static_cast<double>((blocks + slots - 1) / slots); };
    double c = waves(heads * n) * per;
    if (n > 1) c += waves(heads * (n - 1)) * per * kDecayTotalCost + kDecayScanTiles;
    if (c < cost) {
      cost = c;
      best = per;
    }
    if (heads * n > 4ll * slots) break;
  }
  return static_cast<int>(std::min<long long>(static_cast<long long>(best) * kDecayTile, 1 << 30));
}

struct DecayLayout {
  ttt::DecayGeom g;
  size_t run_floats;  // workspace of one run (0: one segment per sequence)
};

bool decay_fits(int d, int dtype) { return d >= 4 && d <= 256 && d % (dtype == TTT_LA_F32 ? 4 : 8) == 0; }

// `tokens`: of a segment; `every`: one state per segment even where no
// sequence has two.
DecayLayout decay_layout(const int32_t* cu, int N, int H, int T, int dk, int dv, int tokens, bool every) {
  DecayLayout l;
  l.g.N = N;
  l.g.H = H;
  l.g.T = T;
  l.g.cu = cu;
  l.g.S = tokens;
  const bool multi = tokens < T;
  const long long nseg = cu ? (multi ? T / tokens : 0) + static_cast<long long>(N)
                            : static_cast<long long>(N) * (T > 0 ? (T - 1) / tokens + 1 : 1);
  l.g.nseg = nseg < (1ll << 31) ? static_cast<int>(nseg) : -1;
  // packed: each sequence of several segments is longer than one and has at most one that is not whole
  long long slots = 0;
  if (every || (multi && !cu))
    slots = nseg;
  else if (multi)
    slots = T / tokens + std::min<long long>(N, T / (static_cast<long long>(tokens) + 1));
  l.g.slots = slots < (1ll << 31) ? static_cast<int>(slots) : 0;  // (nseg, which is no less, is refused then)
  l.g.all = every;
  l.run_floats = static_cast<size_t>(slots) * H * dk * dv;
  return l;
}

ttt::DecayTensor decay_tensor(const void* p, const int64_t* stride) {
  return ttt::DecayTensor{p, stride[0], stride[1], stride[2]};
}

template <typename T>
ttt_la_status decay_simt_run(const ttt::DecayGeom& g, const ttt::DecayRun& r, const float* log_decay, bool totals,
                             cudaStream_t st) {
  const long long blocks = static_cast<long long>(g.nseg) * g.H * ((r.dv + ttt::kDecayVT - 1) / ttt::kDecayVT);
  if (blocks >= (1ll << 31)) return TTT_LA_ERR_UNSUPPORTED;
  const int smem = ttt::decay_simt_smem(r.dk);
  auto kern = totals ? ttt::decay_simt_kernel<T, true> : ttt::decay_simt_kernel<T, false>;
  if (!grant_smem(reinterpret_cast<const void*>(kern), smem)) return TTT_LA_ERR_CUDA;
  return launch_kernel(kern, static_cast<int>(blocks), 256, smem, st, false, g, r, log_decay);
}

// One scan per entry of `p` (at most two), all over the same sequences.
ttt_la_status decay_scan(const ttt::DecayScans& p, int n, bool final, const float* log_decay, cudaStream_t st) {
  long long blocks = 0;
  for (int i = 0; i < n; ++i) {
    const long long dd = static_cast<long long>(p.s[i].dk) * p.s[i].dv, slices = (dd / 4 + 255) / 256;
    blocks = std::max(blocks, slices * p.s[i].g.N * p.s[i].g.H);
  }
  if (blocks >= (1ll << 31)) return TTT_LA_ERR_UNSUPPORTED;
  const dim3 grid(static_cast<unsigned>(blocks), static_cast<unsigned>(n));
  return launch_after(final ? ttt::decay_scan_kernel<true> : ttt::decay_scan_kernel<false>, grid, 256, 0, st, p, log_decay);
}

ttt::DecayScan decay_scan_of(const ttt::DecayGeom& g, const ttt::DecayRun& r) {
  return ttt::DecayScan{g, r.dk, r.dv, r.rev, r.s_in, r.s_in_t, nullptr, r.ws, 0};
}

// `n` runs of the recurrence over the same tokens, in fp32 FMA.
ttt_la_status decay_simt_runs(const ttt::DecayGeom& g, const ttt::DecayRun* r, int n, int dtype, const float* log_decay,
                              cudaStream_t st) {
  for (int i = 0; i < n; ++i) {
    ttt_la_status s = TTT_LA_OK;
    for (int pass = r[i].ws ? 0 : 2; pass < 3 && s == TTT_LA_OK; ++pass) {
      if (pass == 1)
        s = decay_scan(ttt::DecayScans{{decay_scan_of(g, r[i])}}, 1, false, log_decay, st);
      else
        s = dtype == TTT_LA_F32 ? decay_simt_run<float>(g, r[i], log_decay, pass == 0, st)
                                : decay_simt_run<__nv_bfloat16>(g, r[i], log_decay, pass == 0, st);
    }
    if (s != TTT_LA_OK) return s;
  }
  return TTT_LA_OK;
}

// ------------------------------------------------- tensor-core kernels ----
// Prompts from 64 rows on, and every gradient.  T counts all rows of the call,
// those of packed sequences together.  Measured, us here and in fp32 FMA, whose
// outputs are as exact: gradients of 1 to 63 tokens 28 to 29 and 30 to 93 for up
// to 48 (sequence, head)s, 124 to 134 and 269 to 606 for 32 x 16 x 128, 167 to 175
// and 177 to 388 for 64 x 16 x 64.  Prompts of one token 22 and 19 for few, 96 and
// 70 for 64 x 16 x 64, 86 and 111 for 32 x 16 x 128; of 63 tokens 23 and 19 to 35,
// 97 and 138, 91 and 258.  Of many short packed ones, which come here, 64 x 16
// heads x 128 of 1, 15, 46 tokens: prompts 126, 154, 160 and 184, 250, 417,
// gradients 241, 316, 320 and 493, 682, 1181.
bool decay_on_tc(int dtype, int T, int dk, int dv, bool gradient) {
  return dtype == TTT_LA_BF16 && T >= (gradient ? 1 : 64) && dk <= 128 && dv <= 128;
}

// Tokens per segment of the tensor-core kernels, whose blocks have an SM each.
// `heads` sequences of `rows` tokens, `runs` outputs of each.  In units of one
// tile's outputs: a block costs kDecayBlock more than its tiles (its start
// state, filling and draining its pipeline), the totals' pass kDecayTotal of
// that, and cutting the scan.  Whether the final state is asked for plays no
// part, so that the outputs' bits do not depend on it.
constexpr double kDecayBlock = 2.0, kDecayTotal = 0.5, kDecayScan = 2.0;
int decay_tc_plan_tokens(long long heads, int rows, int runs, bool packed, int slots) {
  const int tiles = (rows + ttt::kDecayTcC - 1) / ttt::kDecayTcC;
  int best = tiles;
  double cost = 1e30;
  auto waves = [&](long long blocks) { return static_cast<double>((blocks + slots - 1) / slots); };
  for (int ns = 1; ns <= tiles && ns <= 4096; ++ns) {
    const int per = (tiles + ns - 1) / ns;
    const long long n = (tiles + per - 1) / per;
    double c = waves(heads * n * runs) * (per + kDecayBlock);
    c += waves(heads * n * (runs > 1 ? 2 : 1)) * (per + kDecayBlock) * kDecayTotal;
    if (n > 1) c += kDecayScan;
    if (c < cost) {
      cost = c;
      best = per;
    }
    if (heads * n * runs > 8ll * slots) break;
  }
  // Packed sequences end where they end, and what fills the SMs evenly as one long one leaves them waiting for the
  // longest: at least 1.3 blocks for each SM, but no segment below 512 tokens for that.  The host does not see the
  // lengths, and the rule pays where they differ: us with the even split, then with the rule, of 10 sequences of 1 to
  // 3999 tokens, gradient of 4 heads x 128 106 and 97, of 12 x 64 152 and 136; 30 of 1 to 2000, prompt of 4 x 128 119
  // and 107; no difference for 16 heads x 128 of either, 200 of 1 to 120, 64 of 256.  It costs where a few are equally
  // long or one is nearly all: 2 of 6000, prompt of 16 x 128 98 and 123, gradient of 4 x 128 86 and 98; 12000 tokens
  // and 20 of 20, gradient of 4 x 128 95 and 104.
  if (packed) {
    const long long even = static_cast<long long>(rows) * heads * runs * 10 / (13ll * slots) / ttt::kDecayTcC;
    best = static_cast<int>(std::min<long long>(best, std::max<long long>(even, 512 / ttt::kDecayTcC)));
  }
  return static_cast<int>(std::min<long long>(static_cast<long long>(best) * ttt::kDecayTcC, 1 << 30));
}

// [N][H][T][d] bf16 in the order of `t`'s strides, boxes of 64 features x 128
// tokens (or `rows`); features behind d read as zeros and are not written.
bool decay_map(CUtensorMap* m, const ttt::DecayTensor& t, int N, int H, int T, int d, int rows = ttt::kDecayTcC) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[4] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(T), static_cast<cuuint64_t>(H),
                        static_cast<cuuint64_t>(N)};
  // (the stride of a dimension of size 1 is the caller's to leave out)
  const long long s[3] = {T > 1 ? t.st : d, H > 1 ? t.sh : d, N > 1 ? t.sb : d};
  cuuint64_t strides[3];
  for (int i = 0; i < 3; ++i) strides[i] = static_cast<cuuint64_t>(s[i]) * 2;
  cuuint32_t box[4] = {64, static_cast<cuuint32_t>(rows), 1, 1}, es[4] = {1, 1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(t.p), dims, strides, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int DK, int DV>
ttt_la_status decay_tc_launch(const ttt::DecayTcArgs& a, bool totals, bool first, cudaStream_t st) {
  using Cfg = ttt::DecayTcCfg<DK, DV>;
  const long long blocks = static_cast<long long>(a.g.nseg) * a.g.H * a.nrun;
  if (blocks >= (1ll << 31)) return TTT_LA_ERR_UNSUPPORTED;
  auto kern = totals ? ttt::decay_tc_total_kernel<DK, DV> : ttt::decay_tc_out_kernel<DK, DV>;
  const int smem = totals ? Cfg::A_SMEM : Cfg::SMEM;
  if (!grant_smem(reinterpret_cast<const void*>(kern), smem)) return TTT_LA_ERR_CUDA;
  const int threads = totals ? Cfg::A_THREADS : Cfg::THREADS;
  if (first) return launch_kernel(kern, static_cast<int>(blocks), threads, smem, st, false, a);
  return launch_after(kern, dim3(static_cast<unsigned>(blocks)), threads, smem, st, a);
}
// Launches the runs r[0 .. n) of `a`, those of equal tile widths together.
// `first`: nothing of this call was launched before.
ttt_la_status decay_tc_group(ttt::DecayTcArgs& a, const ttt::DecayTcRun* r, int n, bool totals, bool first,
                             cudaStream_t st) {
  auto wide = [](int d) { return d > 64; };
  for (int shape = 0; shape < 4; ++shape) {
    a.nrun = 0;
    for (int i = 0; i < n; ++i)
      if ((wide(r[i].dk) ? 1 : 0) + (wide(r[i].dv) ? 2 : 0) == shape) a.run[a.nrun++] = r[i];
    if (!a.nrun) continue;
    const ttt_la_status s = shape == 0   ? decay_tc_launch<64, 64>(a, totals, first, st)
                            : shape == 1 ? decay_tc_launch<128, 64>(a, totals, first, st)
                            : shape == 2 ? decay_tc_launch<64, 128>(a, totals, first, st)
                                         : decay_tc_launch<128, 128>(a, totals, first, st);
    if (s != TTT_LA_OK) return s;
    first = false;
  }
  return TTT_LA_OK;
}

ttt::DecayTcRun decay_tc_run(int q, int k, int v, int o, int kt, int vt, const ttt::DecayRun& r) {
  ttt::DecayTcRun t = {};
  t.q = q, t.k = k, t.v = v, t.o = o, t.kt = kt, t.vt = vt;
  t.dk = r.dk, t.dv = r.dv, t.rev = r.rev;
  t.sP = r.sP, t.sR = r.sR, t.sU = r.sU;
  t.s_in = r.s_in, t.s_in_t = r.s_in_t, t.s_out = r.s_out, t.ws = r.ws;
  t.op = static_cast<__nv_bfloat16*>(const_cast<void*>(r.o.p));
  t.ob = r.o.sb, t.oh = r.o.sh, t.ot = r.o.st;
  t.total_last = r.s_out != nullptr;
  return t;
}

// Sizes and strides that the forward and the backward share.
bool decay_strides_ok(const int64_t* s, int N, int H, int T, bool packed, int dtype) {
  const int unit = dtype == TTT_LA_F32 ? 4 : 8;
  const long long size[3] = {packed ? 1 : N, H, T};
  for (int i = 0; i < 3; ++i)
    if (size[i] > 1 && (s[i] < unit || s[i] % unit || s[i] > (1ll << 36))) return false;
  return true;
}

ttt_la_status check_decay_shape(int N, int H, int T, int dk, int dv, int dtype, const int32_t* cu, const float* log_decay,
                                int segment_tokens) {
  if (N < 1 || H < 1 || T < 0 || dk < 1 || dv < 1 || (T == 0 && !cu)) return TTT_LA_ERR_INVALID_ARG;
  if (dtype != TTT_LA_F32 && dtype != TTT_LA_BF16) return TTT_LA_ERR_INVALID_ARG;
  if (!log_decay || (reinterpret_cast<uintptr_t>(log_decay) & 3) || (reinterpret_cast<uintptr_t>(cu) & 3))
    return TTT_LA_ERR_INVALID_ARG;
  if (segment_tokens < 0 || segment_tokens % kDecayTile) return TTT_LA_ERR_INVALID_ARG;
  if (static_cast<long long>(N) * H > (1ll << 24) || T > (1 << 30)) return TTT_LA_ERR_INVALID_ARG;
  if (!decay_fits(dk, dtype) || !decay_fits(dv, dtype)) return TTT_LA_ERR_UNSUPPORTED;
  return TTT_LA_OK;
}

// The layer in its forward direction, as one run.
ttt::DecayRun decay_forward_run(const ttt_la_decay_args* a) {
  ttt::DecayRun r = {};
  r.q = decay_tensor(a->q, a->q_stride);
  r.k = decay_tensor(a->k, a->k_stride);
  r.v = decay_tensor(a->v, a->v_stride);
  r.o = decay_tensor(a->o, a->o_stride);
  r.dk = a->d_k;
  r.dv = a->d_v;
  r.sP = r.sU = a->ascent ? -a->eta_const : a->eta_const;
  r.sR = 1.f;
  r.s_in = a->state_in;
  r.s_out = a->state_out;
  r.clear = a->cu_seqlens && a->clear_rest;
  return r;
}

// The final states overwrite the start states, which the outputs are read
// from: those go through the workspace.
bool decay_in_place(const ttt_la_decay_args* a) {
  return a->state_in && a->state_in == a->state_out && decay_on_tc(a->dtype, a->T, a->d_k, a->d_v, false);
}

int decay_segment_tokens(int asked, const int32_t* cu, int N, int H, int T, int dk, int dv, int dtype, int runs) {
  if (asked > 0) return asked;
  const int rows = std::max(1, T);
  const long long seqs = cu ? 1 : N;
  if (decay_on_tc(dtype, T, dk, dv, runs > 1)) return decay_tc_plan_tokens(seqs * H, rows, runs, cu != nullptr, sm_count());
  const int widest = runs > 1 ? std::max(dk, dv) : dv;
  return decay_plan_tokens(seqs * H * ((widest + ttt::kDecayVT - 1) / ttt::kDecayVT), rows, sm_count() * 2);
}

DecayLayout decay_forward_layout(const ttt_la_decay_args* a) {
  const int tokens = decay_segment_tokens(a->segment_tokens, a->cu_seqlens, a->N, a->H, a->T, a->d_k, a->d_v, a->dtype,
                                          1);
  return decay_layout(a->cu_seqlens, a->N, a->H, a->T, a->d_k, a->d_v, tokens, decay_in_place(a));
}
// Workspaces of one run each, dq's, dv's and dk's states; on the tensor cores
// dk reads dv's.
DecayLayout decay_backward_layout(const ttt_la_decay_grad_args* a, size_t* floats) {
  const int tokens = decay_segment_tokens(a->segment_tokens, a->cu_seqlens, a->N, a->H, a->T, a->d_k, a->d_v, a->dtype,
                                          3);
  const DecayLayout l = decay_layout(a->cu_seqlens, a->N, a->H, a->T, a->d_k, a->d_v, tokens, false);
  *floats = (decay_on_tc(a->dtype, a->T, a->d_k, a->d_v, true) ? 2 : 3) * l.run_floats;
  return l;
}

}  // namespace

extern "C" {

size_t ttt_la_decay_workspace_size(const ttt_la_decay_args* a) {
  if (!a || check_decay_shape(a->N, a->H, a->T, a->d_k, a->d_v, a->dtype, a->cu_seqlens, a->log_decay,
                              a->segment_tokens) != TTT_LA_OK)
    return 0;
  return decay_forward_layout(a).run_floats * sizeof(float);
}

ttt_la_status ttt_la_forward_decay(const ttt_la_decay_args* a, void* stream) {
  NvtxRange range("ttt_la_forward_decay");
  if (!a) return TTT_LA_ERR_INVALID_ARG;
  const ttt_la_status s = check_decay_shape(a->N, a->H, a->T, a->d_k, a->d_v, a->dtype, a->cu_seqlens, a->log_decay,
                                            a->segment_tokens);
  if (s != TTT_LA_OK) return s;
  if (a->clear_rest != 0 && a->clear_rest != 1) return TTT_LA_ERR_INVALID_ARG;
  const bool packed = a->cu_seqlens != nullptr;
  const void* t[4] = {a->q, a->k, a->v, a->o};
  const int64_t* stride[4] = {a->q_stride, a->k_stride, a->v_stride, a->o_stride};
  for (int i = 0; i < 4; ++i)
    if ((a->T > 0 && !t[i]) || !aligned16(t[i]) || !decay_strides_ok(stride[i], a->N, a->H, a->T, packed, a->dtype))
      return TTT_LA_ERR_INVALID_ARG;
  if (!aligned16(a->state_in) || !aligned16(a->state_out)) return TTT_LA_ERR_INVALID_ARG;
  if (a->T > 0 && (a->o == a->q || a->o == a->k || a->o == a->v)) return TTT_LA_ERR_INVALID_ARG;
  const DecayLayout l = decay_forward_layout(a);
  if (l.g.nseg < 0) return TTT_LA_ERR_UNSUPPORTED;
  const size_t need = l.run_floats * sizeof(float);
  if (need && (!a->workspace || !aligned16(a->workspace) || a->workspace_bytes < need)) return TTT_LA_ERR_INVALID_ARG;
  ttt::DecayRun r = decay_forward_run(a);
  r.ws = need ? static_cast<float*>(a->workspace) : nullptr;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (!decay_on_tc(a->dtype, a->T, a->d_k, a->d_v, false))
    return decay_simt_runs(l.g, &r, 1, a->dtype, a->log_decay, st);
  ttt::DecayTcArgs m = {};
  const int batch = packed ? 1 : a->N;
  if (!decay_map(&m.map[0], r.q, batch, a->H, a->T, a->d_k) || !decay_map(&m.map[1], r.k, batch, a->H, a->T, a->d_k) ||
      !decay_map(&m.map[2], r.v, batch, a->H, a->T, a->d_v) || !decay_map(&m.map[3], r.o, batch, a->H, a->T, a->d_v) ||
      !decay_map(&m.map[4], r.k, batch, a->H, a->T, a->d_k, ttt::decay_total_tile(a->d_k)) ||
      !decay_map(&m.map[5], r.v, batch, a->H, a->T, a->d_v, ttt::decay_total_tile(a->d_k)))
    return TTT_LA_ERR_CUDA;
  m.g = l.g, m.log_decay = a->log_decay, m.limit_ns = g_limit_ns, m.clear = r.clear;
  ttt::DecayTcRun run = decay_tc_run(0, 1, 2, 3, 4, 5, r);
  run.ws_all = decay_in_place(a);
  if (r.ws || r.s_out) {
    const ttt_la_status e = decay_tc_group(m, &run, 1, true, true, st);
    if (e != TTT_LA_OK) return e;
  }
  if (r.ws) {
    ttt::DecayScan sc = decay_scan_of(l.g, r);
    sc.s_out = r.s_out, sc.all = run.ws_all;
    const ttt_la_status e = decay_scan(ttt::DecayScans{{sc}}, 1, true, a->log_decay, st);
    if (e != TTT_LA_OK) return e;
  }
  return decay_tc_group(m, &run, 1, false, !(r.ws || r.s_out), st);
}

size_t ttt_la_backward_decay_workspace_size(const ttt_la_decay_grad_args* a) {
  if (!a || check_decay_shape(a->N, a->H, a->T, a->d_k, a->d_v, a->dtype, a->cu_seqlens, a->log_decay,
                              a->segment_tokens) != TTT_LA_OK)
    return 0;
  size_t floats = 0;
  decay_backward_layout(a, &floats);
  return floats * sizeof(float);
}

ttt_la_status ttt_la_backward_decay(const ttt_la_decay_grad_args* a, void* stream) {
  NvtxRange range("ttt_la_backward_decay");
  if (!a) return TTT_LA_ERR_INVALID_ARG;
  const ttt_la_status s = check_decay_shape(a->N, a->H, a->T, a->d_k, a->d_v, a->dtype, a->cu_seqlens, a->log_decay,
                                            a->segment_tokens);
  if (s != TTT_LA_OK) return s;
  const bool packed = a->cu_seqlens != nullptr;
  const void* t[7] = {a->q, a->k, a->v, a->grad_o, a->grad_q, a->grad_k, a->grad_v};
  const int64_t* stride[7] = {a->q_stride,      a->k_stride,      a->v_stride,     a->grad_o_stride,
                              a->grad_q_stride, a->grad_k_stride, a->grad_v_stride};
  for (int i = 0; i < 7; ++i) {
    if ((a->T > 0 && !t[i]) || !aligned16(t[i]) || !decay_strides_ok(stride[i], a->N, a->H, a->T, packed, a->dtype))
      return TTT_LA_ERR_INVALID_ARG;
    for (int j = std::max(4, i + 1); j < 7; ++j)  // an output is neither an input nor another output
      if (a->T > 0 && t[i] == t[j]) return TTT_LA_ERR_INVALID_ARG;
  }
  if (!aligned16(a->state_in) || !aligned16(a->grad_state) || !aligned16(a->grad_state_in))
    return TTT_LA_ERR_INVALID_ARG;
  if (a->grad_state_in && (a->grad_state_in == a->grad_state || a->grad_state_in == a->state_in))
    return TTT_LA_ERR_INVALID_ARG;
  size_t need = 0;
  const DecayLayout l = decay_backward_layout(a, &need);
  if (l.g.nseg < 0) return TTT_LA_ERR_UNSUPPORTED;
  need *= sizeof(float);
  if (need && (!a->workspace || !aligned16(a->workspace) || a->workspace_bytes < need)) return TTT_LA_ERR_INVALID_ARG;
  const ttt::DecayTensor q = decay_tensor(a->q, a->q_stride), k = decay_tensor(a->k, a->k_stride),
                         v = decay_tensor(a->v, a->v_stride), dO = decay_tensor(a->grad_o, a->grad_o_stride);
  const float c = a->ascent ? -a->eta_const : a->eta_const;
  ttt::DecayRun r[3] = {};
  // dq: W^T read with do
  r[0].q = dO, r[0].k = v, r[0].v = k, r[0].o = decay_tensor(a->grad_q, a->grad_q_stride);
  r[0].dk = a->d_v, r[0].dv = a->d_k;
  r[0].sP = r[0].sU = c, r[0].sR = 1.f;
  r[0].s_in = a->state_in, r[0].s_in_t = 1;
  // dk: (dL/dW)^T read with v, last token to first
  r[1].q = v, r[1].k = dO, r[1].v = q, r[1].o = decay_tensor(a->grad_k, a->grad_k_stride);
  r[1].dk = a->d_v, r[1].dv = a->d_k;
  r[1].rev = 1, r[1].sP = r[1].sR = c, r[1].sU = 1.f;
  r[1].s_in = a->grad_state, r[1].s_in_t = 1;
  // dv: dL/dW read with k; where it ends is dL/dW_0
  r[2].q = k, r[2].k = q, r[2].v = dO, r[2].o = decay_tensor(a->grad_v, a->grad_v_stride);
  r[2].dk = a->d_k, r[2].dv = a->d_v;
  r[2].rev = 1, r[2].sP = r[2].sR = c, r[2].sU = 1.f;
  r[2].s_in = a->grad_state, r[2].s_out = a->grad_state_in;
  if (need) {
    r[0].ws = static_cast<float*>(a->workspace);
    r[2].ws = r[0].ws + l.run_floats;
  }
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (!decay_on_tc(a->dtype, a->T, a->d_k, a->d_v, true)) {
    if (need) r[1].ws = r[2].ws + l.run_floats;
    return decay_simt_runs(l.g, r, 3, a->dtype, a->log_decay, st);
  }
  ttt::DecayTcArgs m = {};
  const ttt::DecayTensor x[7] = {q, k, v, dO, r[0].o, r[1].o, r[2].o};
  const bool values[7] = {false, false, true, true, false, false, true};  // d_v wide
  for (int i = 0; i < 11; ++i) {  // the inputs once more in the totals' tiles: q and do for dv's run, k and v for dq's
    const int j = i < 7 ? i : i - 7;
    if (!decay_map(&m.map[i], x[j], packed ? 1 : a->N, a->H, a->T, values[j] ? a->d_v : a->d_k,
                   i < 7 ? ttt::kDecayTcC : ttt::decay_total_tile(j == 0 || j == 3 ? a->d_k : a->d_v)))
      return TTT_LA_ERR_CUDA;
  }
  m.g = l.g, m.log_decay = a->log_decay, m.limit_ns = g_limit_ns;
  // dk reads the transpose of dv's states
  ttt::DecayTcRun run[3] = {decay_tc_run(3, 2, 1, 4, 9, 8, r[0]), decay_tc_run(1, 0, 3, 6, 7, 10, r[2]),
                            decay_tc_run(2, 3, 0, 5, 10, 7, r[1])};
  run[2].ws = run[1].ws, run[2].ws_t = 1;
  if (need || a->grad_state_in) {
    // (without segments only dL/dW_0 is wanted)
    const ttt_la_status e = decay_tc_group(m, need ? run : run + 1, need ? 2 : 1, true, true, st);
    if (e != TTT_LA_OK) return e;
  }
  if (need) {
    ttt::DecayScans sc = {{decay_scan_of(l.g, r[0]), decay_scan_of(l.g, r[2])}};
    sc.s[1].s_out = a->grad_state_in;
    const ttt_la_status e = decay_scan(sc, 2, true, a->log_decay, st);
    if (e != TTT_LA_OK) return e;
  }
  return decay_tc_group(m, run, 3, false, !(need || a->grad_state_in), st);
}

}  // extern "C"

namespace {
template <int DK, typename T>
ttt_la_status launch_decay_step(const ttt::DecayStep& p, cudaStream_t st) {
  // Accesses per lane: 8 where that leaves every SM 16 warps or more, 2 where
  // those do, else 1 (latency counts: small blocks over all SMs).  A warp takes
  // its rows and ends.  Measured (256 sequences x 16 heads x 128 x 128, 544 MB):
  // 8 a lane 83 us, 4 a lane 99, 2 a lane 95; resident blocks that walk on 87
  // to 113.
  constexpr int RPW = 32 / (DK / 4);
  const long long groups = (static_cast<long long>(p.N) * p.H * p.dv + RPW - 1) / RPW;  // of one access a lane
  const long long enough = static_cast<long long>(sm_count()) * 16;
  if (groups / 8 >= enough)
    ttt::decay_step_kernel<DK, T, 8><<<static_cast<int>((groups + 63) / 64), 256, 0, st>>>(p);
  else if (groups / 2 >= enough)
    ttt::decay_step_kernel<DK, T, 2><<<static_cast<int>((groups + 15) / 16), 256, 0, st>>>(p);
  else
    ttt::decay_step_kernel<DK, T, 1><<<static_cast<int>((groups + 3) / 4), 128, 0, st>>>(p);
  return launched();
}
template <typename T>
ttt_la_status decay_step_dk(const ttt::DecayStep& p, cudaStream_t st) {
  switch (p.dk) {
    case 32: return launch_decay_step<32, T>(p, st);
    case 64: return launch_decay_step<64, T>(p, st);
    case 128: return launch_decay_step<128, T>(p, st);
    default: return TTT_LA_ERR_UNSUPPORTED;
  }
}
}  // namespace

extern "C" ttt_la_status ttt_la_decode_step_decay(const ttt_la_decay_decode_args* a, void* stream) {
  NvtxRange range("ttt_la_decode_step_decay");
  if (!a || a->N < 1 || a->H < 1 || a->d_k < 1 || a->d_v < 1) return TTT_LA_ERR_INVALID_ARG;
  if (a->dtype != TTT_LA_F32 && a->dtype != TTT_LA_BF16) return TTT_LA_ERR_INVALID_ARG;
  if (!a->log_decay || (reinterpret_cast<uintptr_t>(a->log_decay) & 3) || !a->state || !aligned16(a->state))
    return TTT_LA_ERR_INVALID_ARG;
  if (static_cast<long long>(a->N) * a->H * a->d_v >= (1ll << 31) - (1 << 20)) return TTT_LA_ERR_INVALID_ARG;
  const void* t[4] = {a->q, a->k, a->v, a->o};
  const int64_t* stride[4] = {a->q_stride, a->k_stride, a->v_stride, a->o_stride};
  const int unit = a->dtype == TTT_LA_F32 ? 4 : 8;
  ttt::DecayTensor x[4];
  for (int i = 0; i < 4; ++i) {
    if (!t[i] || !aligned16(t[i])) return TTT_LA_ERR_INVALID_ARG;
    const long long size[2] = {a->N, a->H};
    const int step = i < 2 ? unit : 1;  // q and k are read in 16-byte pieces, v and o one value at a time
    for (int j = 0; j < 2; ++j)
      if (size[j] > 1 && (stride[i][j] < step || stride[i][j] % step || stride[i][j] > (1ll << 36)))
        return TTT_LA_ERR_INVALID_ARG;
    x[i] = ttt::DecayTensor{t[i], stride[i][0], stride[i][1], 0};
  }
  if (a->o == a->q || a->o == a->k || a->o == a->v) return TTT_LA_ERR_INVALID_ARG;
  ttt::DecayStep p = {};
  p.N = a->N, p.H = a->H, p.dk = a->d_k, p.dv = a->d_v;
  p.q = x[0], p.k = x[1], p.v = x[2], p.o = x[3];
  p.log_decay = a->log_decay;
  p.a = a->ascent ? -a->eta_const : a->eta_const;
  p.S = a->state;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  return a->dtype == TTT_LA_F32 ? decay_step_dk<float>(p, st) : decay_step_dk<__nv_bfloat16>(p, st);
}
