// qlora_mlp_host.cuh -- host side of the gated MLP and of the linear layer with bias, activation and
// residual: argument checks, launches and entry points (included by qlora.cu).
#pragma once

namespace qlora {
namespace {

const float* ts_of(const qlora_weight_t* W) {
  return W->fmt == QLORA_FMT_NVFP4 ? W->tensor_scale : nullptr;
}

bool act_valid(int act) { return act >= QLORA_ACT_NONE && act <= QLORA_ACT_GELU_TANH; }

template <int FMT, bool DX, int EPI, bool SPLIT, int RB>
qlora_status_t launch_fused_ex_s(const FusedExParams& p, int grid, bool early, cudaStream_t st) {
  const size_t smem = fused::smem_bytes(1, RB);
  if (!set_smem(qlora_fused_gemm_kernel<FMT, DX, EPI, SPLIT, RB>, smem)) return QLORA_ERR_CUDA;
  LaunchScope scope(EPI == kEpiAct ? (DX ? kKindFusedDx : kKindActFwd) : (DX ? kKindGatedDx : kKindGatedFwd), st);
  if (launch_pdl(qlora_fused_gemm_kernel<FMT, DX, EPI, SPLIT, RB>, dim3(grid), dim3(fused::threads(RB)), smem, st, p,
                 early) != cudaSuccess)
    return QLORA_ERR_CUDA;
  return cudaGetLastError() == cudaSuccess ? QLORA_OK : QLORA_ERR_CUDA;
}

template <int FMT, bool DX, int EPI>
qlora_status_t launch_fused_ex_t(const FusedExParams& p, int grid, bool early, cudaStream_t st) {
  if (p.splits == 1) return launch_fused_ex_s<FMT, DX, EPI, false, 2>(p, grid, early, st);
  return p.M <= 2 * fused::HM ? launch_fused_ex_s<FMT, DX, EPI, true, 1>(p, grid, early, st)
                              : launch_fused_ex_s<FMT, DX, EPI, true, 2>(p, grid, early, st);
}

// early: the launch may start beside the kernel before it (which must then not write this
// one's activations).
template <bool DX, int EPI>
qlora_status_t launch_fused_ex(int fmt, const FusedExParams& p, int grid, bool early, cudaStream_t st) {
  switch (fmt) {
    case QLORA_FMT_NF4: return launch_fused_ex_t<kFmtNF4, DX, EPI>(p, grid, early, st);
    case QLORA_FMT_MXFP4: return launch_fused_ex_t<kFmtMXFP4, DX, EPI>(p, grid, early, st);
    case QLORA_FMT_NVFP4: return launch_fused_ex_t<kFmtNVFP4, DX, EPI>(p, grid, early, st);
    default: return launch_fused_ex_t<kFmtNF4DQ, DX, EPI>(p, grid, early, st);
  }
}

bool tmap_codes(CUtensorMap* m, const qlora_weight_t* W, bool dx) {
  const uint64_t kb = uint64_t(W->K / 2);
  return dx ? tmap_2d(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, W->codes, kb, uint64_t(W->N), kb, 64, 64,
                      CU_TENSOR_MAP_SWIZZLE_64B)
            : tmap_2d(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, W->codes, kb, uint64_t(W->N), kb, 32, 128,
                      CU_TENSOR_MAP_SWIZZLE_32B);
}

// The members of FusedParams that every variant of one layer shares: `act` and the weight Wg, Zs
// [M, zr], `out`, and a grid of pair tiles of `tile_cols` output columns.
qlora_status_t fill_fused(FusedExParams& p, const qlora_weight_t* W, bool dx, const void* act,
                          const void* zs, int zr, const void* lora_up, void* out, int64_t M, int r,
                          int tile_cols, int* status, const SplitPlan& split, float* split_out,
                          int& grid) {
  const int64_t Kc = dx ? W->N : W->K;
  if (!tmap_2d(&p.tm_act, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, act, uint64_t(Kc), uint64_t(M),
               uint64_t(Kc) * 2, 64, 128, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !tmap_codes(&p.tm_codes, W, dx) ||
      !tmap_2d(&p.tm_zs, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, zs, uint64_t(zr), uint64_t(M),
               uint64_t(zr) * 2, 64, 128, CU_TENSOR_MAP_SWIZZLE_128B))
    return QLORA_ERR_CUDA;
  p.scales = W->scales;
  p.scales2 = W->fmt == QLORA_FMT_NF4_DQ ? W->scales2 : nullptr;
  p.tensor_scale = W->fmt == QLORA_FMT_NVFP4 ? W->tensor_scale : nullptr;
  p.lora_up = static_cast<const __nv_bfloat16*>(lora_up);
  p.out = static_cast<__nv_bfloat16*>(out);
  p.status = status;
  p.ticket = reinterpret_cast<unsigned*>(status + 1);
  p.M = int(M);
  p.N = int(W->N);
  p.K = int(W->K);
  p.r = r;
  p.E = 1;
  p.num_n = int(((dx ? W->K : W->N) + tile_cols - 1) / tile_cols);
  p.num_k = int((Kc + fused::BK - 1) / fused::BK);
  // as launch_fused: one CTA pair per two SMs, a short last wave in half tiles (unless split)
  int64_t tiles = row_tiles(M) * p.num_n;
  const int64_t most = num_sms() / 2;
  p.splits = split.S;
  p.split_out = split_out;
  if (split.S == 1) {
    int64_t pairs = tiles < most ? tiles : most;
    const int64_t rem = tiles % pairs;
    if (rem > 0 && 2 * rem <= pairs && tiles > pairs) p.tail_split = int(rem);
  }
  const int64_t items = (tiles + p.tail_split) * split.S;
  const int64_t pairs = items < most ? items : most;
  grid = int(2 * pairs);
  return QLORA_OK;
}

// The sums and the epilogue of a split contraction whose accumulators `p` has written.
qlora_status_t launch_split(const FusedExParams& p, int n, bool gated, cudaStream_t st) {
  SplitParams q{};
  q.part = p.split_out;
  q.bias = p.bias;
  q.residual = p.residual;
  q.out = p.out;
  q.save0 = p.save0;
  q.save1 = p.save1;
  q.groups = (long long)p.M * (n / 8);
  q.S = p.splits;
  q.n = n;
  q.width = gated ? 2 * n : n;
  q.gated = gated ? 1 : 0;
  q.act = p.act;
  if (!set_smem(qlora_split_kernel, 0)) return QLORA_ERR_CUDA;
  LaunchScope scope(kKindSplit, st);
  if (launch_pdl(qlora_split_kernel, dim3(unsigned((q.groups + 255) / 256)), dim3(256), 0, st, q) != cudaSuccess ||
      cudaGetLastError() != cudaSuccess)
    return QLORA_ERR_CUDA;
  return QLORA_OK;
}

template <int NB, int ACT, bool LO>
qlora_status_t launch_act_down_lo(const ActDownParams& p, unsigned grid, cudaStream_t st) {
  const size_t smem = actdown::smem_bytes(NB, LO);
  auto kern = qlora_act_down_kernel<NB, ACT, LO>;
  if (!set_smem(kern, smem)) return QLORA_ERR_CUDA;
  LaunchScope scope(kKindActDown, st);
  if (launch_pdl(kern, dim3(grid), dim3(actdown::kThreads), smem, st, p) != cudaSuccess) return QLORA_ERR_CUDA;
  return cudaGetLastError() == cudaSuccess ? QLORA_OK : QLORA_ERR_CUDA;
}
// dZ of no activation is dY itself: no rounding.
template <int NB, int ACT>
qlora_status_t launch_act_down_t(const ActDownParams& p, unsigned grid, cudaStream_t st) {
  if constexpr (NB == 2 || ACT != act::kNone) {
    if (p.M <= actdown::BM) return launch_act_down_lo<NB, ACT, true>(p, grid, st);
  }
  return launch_act_down_lo<NB, ACT, false>(p, grid, st);
}

// Gradients of the pre-activations and their projections (nb = 1 or 2 streams): grad, U as u + u_lo, Zs.
qlora_status_t launch_act_down(int nb, int act, const void* dy, const void* a0, const void* a1,
                               const void* const* B, const float* const* ts, void* const* grad,
                               void* const* u, void* const* u_lo, void* zs, float* bias_part, int64_t M,
                               int64_t N, int r, float s, float zs_mul, void* sums, void* ws,
                               cudaStream_t st) {
  ActDownParams p{};
  const int rpad = rank_pad(r);
  const ActDownPlan dp = act_down_plan(M, N, num_sms());
  for (int b = 0; b < nb; ++b) {
    if (!tmap_3d(&p.tm_r[b], B[b], uint64_t(r), uint64_t(N), 1, uint32_t(rpad), 64,
                 swizzle_for_bytes(uint32_t(rpad) * 2)))
      return QLORA_ERR_CUDA;
    p.grad[b] = static_cast<__nv_bfloat16*>(grad[b]);
  }
  p.dy = static_cast<const __nv_bfloat16*>(dy);
  p.a0 = static_cast<const __nv_bfloat16*>(a0);
  p.a1 = static_cast<const __nv_bfloat16*>(a1);
  p.part = static_cast<float*>(sums);
  p.ts0 = ts[0];
  p.ts1 = nb == 2 ? ts[1] : nullptr;
  p.bias_part = bias_part;
  p.status = ws_status(ws);
  p.M = int(M);
  p.N = int(N);
  p.r = r;
  p.rpad = rpad;
  p.num_k = dp.num_k;
  p.S = dp.S;
  p.sps = dp.sps;
  const unsigned grid = unsigned(int64_t(dp.tiles) * dp.S);
  qlora_status_t rc;
  switch ((nb - 1) * act::kNumActs + act) {
    case 0: rc = launch_act_down_t<1, act::kNone>(p, grid, st); break;
    case 1: rc = launch_act_down_t<1, act::kSilu>(p, grid, st); break;
    case 2: rc = launch_act_down_t<1, act::kGelu>(p, grid, st); break;
    case 3: rc = launch_act_down_t<1, act::kGeluTanh>(p, grid, st); break;
    case 4: rc = launch_act_down_t<2, act::kNone>(p, grid, st); break;
    case 5: rc = launch_act_down_t<2, act::kSilu>(p, grid, st); break;
    case 6: rc = launch_act_down_t<2, act::kGelu>(p, grid, st); break;
    default: rc = launch_act_down_t<2, act::kGeluTanh>(p, grid, st); break;
  }
  if (rc != QLORA_OK) return rc;
  DownSumParams q{};
  q.part = p.part;
  for (int b = 0; b < nb; ++b) {
    q.hi[b] = static_cast<__nv_bfloat16*>(u[b]);
    q.lo[b] = static_cast<__nv_bfloat16*>(u_lo[b]);
  }
  q.zs = static_cast<__nv_bfloat16*>(zs);
  q.ts = ts[0];
  q.width = nb * r;
  q.groups = (long long)M * (q.width / 4);
  q.S = dp.S;
  q.r = r;
  q.s = s;
  q.zs_mul = zs_mul;
  if (!set_smem(qlora_down_sum_kernel, 0)) return QLORA_ERR_CUDA;
  LaunchScope scope(kKindDownSum, st);
  if (launch_pdl(qlora_down_sum_kernel, dim3(unsigned((q.groups + 31) / 32)), dim3(256), 0, st, q) != cudaSuccess ||
      cudaGetLastError() != cudaSuccess)
    return QLORA_ERR_CUDA;
  return QLORA_OK;
}

// Up to this many rows the adapter gradients run ahead of dX on the same stream: a few microseconds,
// after which dX may be launched early (its predecessor has waited for the gradients it reads), and
// no events.  Longer batches run them beside dX.  Measured: gated, 77 rows of 2 x 2048 from 7168, 44 us ahead
// and 48 beside; one weight, 1021 rows of 8192 x 2048, 87 ahead and 78 beside.
constexpr int64_t kWgradFirstRows = 256;

// Runs `side_work` on the device's side stream beside `main_work` on `s`, joined into `s` again.  The
// first kernel of main_work reads what the kernels before on `s` have only just written, so it is
// launched without the permission to start early; launched early, it would also hold back the fork
// event and with it side_work, until its own end (measured).
template <class F, class G>
qlora_status_t fork_join(cudaStream_t s, F&& side_work, G&& main_work) {
  SideStream* side = side_stream();
  if (!side) {
    const qlora_status_t st = main_work();
    return st != QLORA_OK ? st : side_work(s);
  }
  const int slot = side->next.fetch_add(1, std::memory_order_relaxed) % SideStream::kEvents;
  if (cudaEventRecord(side->fork[slot], s) != cudaSuccess ||
      cudaStreamWaitEvent(side->stream, side->fork[slot], 0) != cudaSuccess)
    return QLORA_ERR_CUDA;
  // main_work first: its kernel takes the SMs it needs, side_work the ones it leaves idle
  qlora_status_t st = main_work();
  const qlora_status_t st2 = side_work(side->stream);
  if (st == QLORA_OK) st = st2;
  if (cudaEventRecord(side->join[slot], side->stream) != cudaSuccess) return QLORA_ERR_CUDA;
  if (cudaStreamWaitEvent(s, side->join[slot], 0) != cudaSuccess) return QLORA_ERR_CUDA;
  return st;
}

// ------------------------------------------------------------------------- batches of up to 16 rows
template <int NB>
qlora_status_t launch_narrow_down_t(const NarrowDownParams& p, unsigned groups, cudaStream_t st) {
  if (!set_smem(qlora_narrow_down_kernel<NB>, 0)) return QLORA_ERR_CUDA;
  LaunchScope scope(kKindNarrowDown, st);
  const dim3 grid(groups * unsigned(p.S), unsigned((p.M + 8 * NB - 1) / (8 * NB)));
  if (launch_pdl_cluster(qlora_narrow_down_kernel<NB>, grid, dim3(narrow::kDownWarps * 32), 0, st, p,
                         unsigned(p.S)) != cudaSuccess)
    return QLORA_ERR_CUDA;
  return cudaGetLastError() == cudaSuccess ? QLORA_OK : QLORA_ERR_CUDA;
}

template <int FMT, bool GATED, int NB>
qlora_status_t launch_narrow_t(const NarrowParams& p, unsigned grid, cudaStream_t st) {
  const size_t smem = narrow::smem_bytes(NB);
  auto kern = qlora_narrow_kernel<FMT, GATED, NB>;
  if (!set_smem(kern, smem)) return QLORA_ERR_CUDA;
  LaunchScope scope(GATED ? kKindGatedFwd : kKindActFwd, st);
  if (launch_pdl(kern, dim3(grid), dim3(narrow::kThreads), smem, st, p) != cudaSuccess) return QLORA_ERR_CUDA;
  return cudaGetLastError() == cudaSuccess ? QLORA_OK : QLORA_ERR_CUDA;
}

template <bool GATED, int NB>
qlora_status_t launch_narrow_f(int fmt, const NarrowParams& p, unsigned grid, cudaStream_t st) {
  switch (fmt) {
    case QLORA_FMT_NF4: return launch_narrow_t<kFmtNF4, GATED, NB>(p, grid, st);
    case QLORA_FMT_MXFP4: return launch_narrow_t<kFmtMXFP4, GATED, NB>(p, grid, st);
    case QLORA_FMT_NVFP4: return launch_narrow_t<kFmtNVFP4, GATED, NB>(p, grid, st);
    default: return launch_narrow_t<kFmtNF4DQ, GATED, NB>(p, grid, st);
  }
}

NarrowWeight narrow_weight(const qlora_weight_t* W, const void* B) {
  return NarrowWeight{W->scales, W->fmt == QLORA_FMT_NF4_DQ ? W->scales2 : nullptr,
                      W->fmt == QLORA_FMT_NVFP4 ? W->tensor_scale : nullptr,
                      static_cast<const __nv_bfloat16*>(B)};
}

// Blocks of 8 batch rows, as the kernels are compiled for.
int narrow_blocks(int64_t M) { return M <= 8 ? 1 : 2; }

// T [nw][M, r] and Zs [M, nw r] of one or two adapters (Wu, Au null: one).
qlora_status_t narrow_down(const qlora_weight_t* Wg, const qlora_weight_t* Wu, const void* X, const void* Ag,
                           const void* Au, void* T, void* Zs, int64_t M, int r, float scale, cudaStream_t st) {
  const int64_t K = Wg->K;
  const int nw = Wu ? 2 : 1, nb = narrow_blocks(M);
  NarrowDownParams d{};
  d.a0 = static_cast<const __nv_bfloat16*>(Ag);
  d.a1 = static_cast<const __nv_bfloat16*>(Au);
  d.x = static_cast<const __nv_bfloat16*>(X);
  d.ts0 = ts_of(Wg);
  d.ts1 = Wu ? ts_of(Wu) : nullptr;
  d.t = static_cast<__nv_bfloat16*>(T);
  d.zs = static_cast<__nv_bfloat16*>(Zs);
  d.M = int(M);
  d.K = int(K);
  d.r = r;
  d.nw = nw;
  d.ldzs = nw * r;
  // CTAs per row group: beside the narrow kernel, which wants every SM, half as many for one depth as
  // beside the split one (one token of 2 x 14336 from 4096: 36 us with 8, 33 with 4)
  const int64_t deep = M <= narrow::kMaxRows ? 2 : 1;
  d.S = K >= 4096 * deep ? 8 : (K >= 1024 * deep ? 4 : 1);
  d.s = scale;
  const unsigned groups = unsigned((nw * r + 15) / 16);
  return nb == 1 ? launch_narrow_down_t<1>(d, groups, st) : launch_narrow_down_t<2>(d, groups, st);
}

// T and Zs by the kernels of the batch size: in the forward, and in a backward call that was not
// given T (the forward's T bit for bit).
qlora_status_t project_t(const qlora_weight_t* Wg, const qlora_weight_t* Wu, const void* X, const void* Ag,
                           const void* Au, uint8_t* T, uint8_t* Zs, int64_t M, int r, float scale, void* ws,
                           cudaStream_t s) {
  if (M <= narrow::kMaxDownRows) return narrow_down(Wg, Wu, X, Ag, Au, T, Zs, M, r, scale, s);
  const int nw = Wu ? 2 : 1;
  for (int i = 0; i < nw; ++i) {
    const qlora_status_t st = launch_lora_down(
        false, X, M, Wg->K, i ? Au : Ag, r, scale, ts_of(i ? Wu : Wg), T + size_t(i) * M * r * 2,
        Zs + size_t(i) * r * 2, ws_status(ws), nullptr, 1, false, kDownCtasBesidePair, s, 1.0f, 0, nullptr,
        nullptr, nw * r);
    if (st != QLORA_OK) return st;
  }
  return QLORA_OK;
}

// The whole forward of a batch of at most 16 rows (Wu: the up weight of a gated MLP, else null).  p
// holds the epilogue's members; T [nw][M, r] and Zs [M, nw r] are written first.
qlora_status_t run_narrow(const qlora_weight_t* Wg, const qlora_weight_t* Wu, const void* X, const void* Ag,
                          const void* Bg, const void* Au, const void* Bu, void* T, void* Zs, int64_t M, int r,
                          float scale, NarrowParams p, void* ws, float* partial, size_t partial_bytes,
                          cudaStream_t st) {
  const int64_t N = Wg->N, K = Wg->K;
  const int nw = Wu ? 2 : 1;
  const int nb = narrow_blocks(M);
  const int cols = Wu ? narrow::kRows / 2 : narrow::kRows;
  const int64_t tiles = (N + cols - 1) / cols, chunks = (K + narrow::CK - 1) / narrow::CK, units = tiles * chunks;
  if (units > INT32_MAX) return QLORA_ERR_UNSUPPORTED;
  const qlora_status_t rc = narrow_down(Wg, Wu, X, Ag, Au, T, Zs, M, r, scale, st);
  if (rc != QLORA_OK) return rc;
  p.w[0] = narrow_weight(Wg, Bg);
  if (Wu) p.w[1] = narrow_weight(Wu, Bu);
  for (int i = 0; i < nw; ++i)
    if (!tmap_2d(&p.tm_codes[i], CU_TENSOR_MAP_DATA_TYPE_UINT8, (i ? Wu : Wg)->codes, uint64_t(K / 2), uint64_t(N),
                 uint64_t(K / 2), narrow::CK / 2, narrow::kRows / nw, CU_TENSOR_MAP_SWIZZLE_128B))
      return QLORA_ERR_CUDA;
  p.x = static_cast<const __nv_bfloat16*>(X);
  p.zs = static_cast<const __nv_bfloat16*>(Zs);
  p.M = int(M);
  p.N = int(N);
  p.K = int(K);
  p.r = r;
  p.ldzs = nw * r;
  p.tiles = int(tiles);
  p.chunks = int(chunks);
  p.one = 1u;
  // Equal ranges of (tile, chunk) units over the SMs; without room for the partials, or with more
  // tiles than counters, whole tiles.
  p.status = ws_status(ws);
  p.counters = reinterpret_cast<unsigned*>(static_cast<uint8_t*>(ws) + kCounterOffset);
  p.partial = partial;
  const int64_t sms = num_sms();
  const bool split = p.tiles <= narrow::kMaxCounters && partial_bytes >= narrow_partial_bytes(M, sms);
  const int64_t iters = split ? (units + sms - 1) / sms : (p.tiles + sms - 1) / sms * p.chunks;
  p.iters = int(iters);
  const unsigned grid = unsigned((units + iters - 1) / iters);
  if (Wu)
    return nb == 1 ? launch_narrow_f<true, 1>(Wg->fmt, p, grid, st) : launch_narrow_f<true, 2>(Wg->fmt, p, grid, st);
  return nb == 1 ? launch_narrow_f<false, 1>(Wg->fmt, p, grid, st) : launch_narrow_f<false, 2>(Wg->fmt, p, grid, st);
}

qlora_status_t check_gated(const qlora_weight_t* Wg, const qlora_weight_t* Wu, int act, int64_t M, int r) {
  qlora_status_t st = check_common(Wg, M, r);
  if (st != QLORA_OK) return st;
  if ((st = check_weight(Wu)) != QLORA_OK) return st;
  if (Wg->N != Wu->N || Wg->K != Wu->K || !act_valid(act)) return QLORA_ERR_INVALID_ARG;
  return Wg->fmt == Wu->fmt ? QLORA_OK : QLORA_ERR_UNSUPPORTED;
}


}  // namespace
}  // namespace qlora

extern "C" {

qlora_status_t qlora_gated_mlp_fwd(const qlora_weight_t* Wg, const qlora_weight_t* Wu, int act,
                                   const void* X, const void* Ag, const void* Bg, const void* Au,
                                   const void* Bu, void* H, void* G, void* U, void* T_save, int64_t M,
                                   int r, float scale, void* ws, size_t ws_bytes,
                                   qlora_stream_t stream) {
  qlora_status_t st = check_gated(Wg, Wu, act, M, r);
  if (st != QLORA_OK) return st;
  if (!act_ok(X, M) || !ptr_ok(Ag) || !ptr_ok(Bg) || !ptr_ok(Au) || !ptr_ok(Bu) || !act_ok(H, M) ||
      !opt_ok(G) || !opt_ok(U) || !opt_ok(T_save))
    return QLORA_ERR_INVALID_ARG;
  const MlpLayout L = mlp_layout(Wg->N, Wg->K, M, r, 2, false, num_sms());
  if (!ws || !aligned16(ws) || ws_bytes < L.partial) return QLORA_ERR_WORKSPACE;
  if (M == 0) return QLORA_OK;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  uint8_t* w = static_cast<uint8_t*>(ws);
  uint8_t* T = T_save ? static_cast<uint8_t*>(T_save) : w + L.t;
  if (M <= narrow::kMaxRows) {
    NarrowParams p{};
    p.out = static_cast<__nv_bfloat16*>(H);
    p.save0 = static_cast<__nv_bfloat16*>(G);
    p.save1 = static_cast<__nv_bfloat16*>(U);
    p.act = act;
    return run_narrow(Wg, Wu, X, Ag, Bg, Au, Bu, T, w + L.zs, M, r, scale, p, ws,
                      reinterpret_cast<float*>(w + L.partial), ws_bytes - L.partial, s);
  }
  st = project_t(Wg, Wu, X, Ag, Au, T, w + L.zs, M, r, scale, ws, s);
  if (st != QLORA_OK) return st;
  FusedExParams p{};
  int grid = 0;
  const SplitPlan sp = split_fwd(Wg->N, Wg->K, M, r, 2, num_sms(), ws_bytes - L.partial);
  st = fill_fused(p, Wg, false, X, w + L.zs, 2 * r, Bg, H, M, r, fused::HN, ws_status(ws), sp,
                  reinterpret_cast<float*>(w + L.partial), grid);
  if (st != QLORA_OK) return st;
  if (!tmap_codes(&p.tm_codes_up, Wu, false)) return QLORA_ERR_CUDA;
  p.scales_up = Wu->scales;
  p.scales2_up = Wu->scales2;
  p.tensor_scale_up = ts_of(Wu);
  p.lora_up_up = static_cast<const __nv_bfloat16*>(Bu);
  p.save0 = static_cast<__nv_bfloat16*>(G);
  p.save1 = static_cast<__nv_bfloat16*>(U);
  p.act = act;
  st = launch_fused_ex<false, kEpiGated>(Wg->fmt, p, grid, true, s);
  return st != QLORA_OK || sp.S == 1 ? st : launch_split(p, p.N, true, s);
}

qlora_status_t qlora_gated_mlp_bwd(const qlora_weight_t* Wg, const qlora_weight_t* Wu, int act,
                                   const void* X, const void* Ag, const void* Bg, const void* Au,
                                   const void* Bu, const void* T, const void* G, const void* U,
                                   const void* dH, void* dX, void* dAg, void* dBg, void* dAu, void* dBu,
                                   int64_t M, int r, float scale, void* ws, size_t ws_bytes,
                                   qlora_stream_t stream) {
  qlora_status_t st = check_gated(Wg, Wu, act, M, r);
  if (st != QLORA_OK) return st;
  if (!act_ok(X, M) || !ptr_ok(Ag) || !ptr_ok(Bg) || !ptr_ok(Au) || !ptr_ok(Bu) || !opt_ok(T) ||
      !act_ok(G, M) || !act_ok(U, M) || !act_ok(dH, M) || !opt_ok(dX) || !ptr_ok(dAg) || !ptr_ok(dBg) ||
      !ptr_ok(dAu) || !ptr_ok(dBu))
    return QLORA_ERR_INVALID_ARG;
  const int64_t N = Wg->N, K = Wg->K;
  const MlpLayout L = mlp_layout(N, K, M, r, 2, true, num_sms());
  if (!ws || !aligned16(ws) || ws_bytes < L.partial) return QLORA_ERR_WORKSPACE;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (M == 0) {
    for (void* d : {dAg, dAu})
      if (cudaMemsetAsync(d, 0, size_t(r) * K * 2, s) != cudaSuccess) return QLORA_ERR_CUDA;
    for (void* d : {dBg, dBu})
      if (cudaMemsetAsync(d, 0, size_t(N) * r * 2, s) != cudaSuccess) return QLORA_ERR_CUDA;
    return QLORA_OK;
  }
  uint8_t* w = static_cast<uint8_t*>(ws);
  const size_t mr = size_t(M) * size_t(r) * 2, mn = size_t(M) * size_t(N) * 2;
  const uint8_t* Ts = static_cast<const uint8_t*>(T);
  if (!T) {   // recomputed with the forward's plan: the forward's T bit for bit
    st = project_t(Wg, Wu, X, Ag, Au, w + L.t, w + L.zs, M, r, scale, ws, s);
    if (st != QLORA_OK) return st;
    Ts = w + L.t;
  }
  void* const grad[2] = {w + L.grad, w + L.grad + mn};
  void* const z[2] = {w + L.u, w + L.u + mr};
  void* const z_lo[2] = {w + L.u_lo, w + L.u_lo + mr};
  const void* const Bs[2] = {Bg, Bu};
  const float* const ts[2] = {ts_of(Wg), ts_of(Wu)};
  st = launch_act_down(2, act, dH, G, U, Bs, ts, grad, z, z_lo, w + L.zs, nullptr, M, N, r, scale, 1.0f,
                       w + L.sums, ws, s);
  if (st != QLORA_OK) return st;
  auto wgrads = [&](cudaStream_t q) {
    const WgradSecond up{grad[1], Ts + mr, z[1], z_lo[1], dAu, dBu, ts[1], ts[0]};
    return launch_wgrad(X, grad[0], Ts, z[0], M, N, K, r, scale, dAg, dBg, ws, nullptr, 1, false, q, z_lo[0],
                        &up);
  };
  if (!dX) return wgrads(s);
  const bool beside = M > kWgradFirstRows;
  if (!beside && (st = wgrads(s)) != QLORA_OK) return st;
  auto run_dx = [&]() {
    FusedExParams p{};
    int grid = 0;
    const SplitPlan sp = split_dx(N, K, M, r, 2, num_sms(), ws_bytes - L.partial);
    qlora_status_t e = fill_fused(p, Wg, true, grad[0], w + L.zs, 2 * r, Ag, dX, M, r, fused::BN,
                                  ws_status(ws), sp, reinterpret_cast<float*>(w + L.partial), grid);
    if (e != QLORA_OK) return e;
    if (!tmap_codes(&p.tm_codes_up, Wu, true) ||
        !tmap_2d(&p.tm_act_up, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, grad[1], uint64_t(N), uint64_t(M),
                 uint64_t(N) * 2, 64, 128, CU_TENSOR_MAP_SWIZZLE_128B))
      return QLORA_ERR_CUDA;
    p.scales_up = Wu->scales;
    p.scales2_up = Wu->scales2;
    p.lora_up_up = static_cast<const __nv_bfloat16*>(Au);
    e = launch_fused_ex<true, kEpiGated>(Wg->fmt, p, grid, !beside, s);
    return e != QLORA_OK || sp.S == 1 ? e : launch_split(p, p.K, false, s);
  };
  return beside ? fork_join(s, wgrads, run_dx) : run_dx();
}

qlora_status_t qlora_linear_act_fwd(const qlora_weight_t* W, const void* X, const void* A, const void* B,
                                    const void* bias, int act, const void* residual, void* Y,
                                    void* Z_save, void* T_save, int64_t M, int r, float scale, void* ws,
                                    size_t ws_bytes, qlora_stream_t stream) {
  qlora_status_t st = check_common(W, M, r);
  if (st != QLORA_OK) return st;
  if (!act_valid(act) || !act_ok(X, M) || !ptr_ok(A) || !ptr_ok(B) || !opt_ok(bias) || !opt_ok(residual) ||
      !act_ok(Y, M) || !opt_ok(Z_save) || !opt_ok(T_save))
    return QLORA_ERR_INVALID_ARG;
  const MlpLayout L = mlp_layout(W->N, W->K, M, r, 1, false, num_sms());
  if (!ws || !aligned16(ws) || ws_bytes < L.partial) return QLORA_ERR_WORKSPACE;
  if (M == 0) return QLORA_OK;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  uint8_t* w = static_cast<uint8_t*>(ws);
  if (M <= narrow::kMaxRows) {
    NarrowParams p{};
    p.out = static_cast<__nv_bfloat16*>(Y);
    p.save0 = static_cast<__nv_bfloat16*>(Z_save);
    p.bias = static_cast<const __nv_bfloat16*>(bias);
    p.residual = static_cast<const __nv_bfloat16*>(residual);
    p.act = act;
    return run_narrow(W, nullptr, X, A, B, nullptr, nullptr, T_save ? T_save : w + L.t, w + L.zs, M, r, scale, p,
                      ws, reinterpret_cast<float*>(w + L.partial), ws_bytes - L.partial, s);
  }
  st = project_t(W, nullptr, X, A, nullptr, T_save ? static_cast<uint8_t*>(T_save) : w + L.t, w + L.zs, M, r,
                   scale, ws, s);
  if (st != QLORA_OK) return st;
  FusedExParams p{};
  int grid = 0;
  const SplitPlan sp = split_fwd(W->N, W->K, M, r, 1, num_sms(), ws_bytes - L.partial);
  st = fill_fused(p, W, false, X, w + L.zs, r, B, Y, M, r, fused::BN, ws_status(ws), sp,
                  reinterpret_cast<float*>(w + L.partial), grid);
  if (st != QLORA_OK) return st;
  p.bias = static_cast<const __nv_bfloat16*>(bias);
  p.residual = static_cast<const __nv_bfloat16*>(residual);
  p.save0 = static_cast<__nv_bfloat16*>(Z_save);
  p.act = act;
  st = launch_fused_ex<false, kEpiAct>(W->fmt, p, grid, true, s);
  return st != QLORA_OK || sp.S == 1 ? st : launch_split(p, p.N, false, s);
}

qlora_status_t qlora_linear_act_bwd(const qlora_weight_t* W, const void* X, const void* A, const void* B,
                                    const void* T, const void* Z, int act, const void* dY, void* dX,
                                    void* dA, void* dB, void* dbias, int64_t M, int r, float scale,
                                    void* ws, size_t ws_bytes, qlora_stream_t stream) {
  qlora_status_t st = check_common(W, M, r);
  if (st != QLORA_OK) return st;
  if (!act_valid(act) || !opt_ok(Z) || (act != QLORA_ACT_NONE && !act_ok(Z, M)) || !opt_ok(dbias))
    return QLORA_ERR_INVALID_ARG;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (act == QLORA_ACT_NONE && !dbias)   // dZ is dY: the layer's own backward pass
    return run_bwd(W, 1, nullptr, false, X, A, B, T, dY, dX, dA, dB, M, r, scale, ws, ws_bytes, s);
  if (!act_ok(X, M) || !ptr_ok(A) || !ptr_ok(B) || !opt_ok(T) || !act_ok(dY, M) || !opt_ok(dX) ||
      !ptr_ok(dA) || !ptr_ok(dB))
    return QLORA_ERR_INVALID_ARG;
  const int64_t N = W->N, K = W->K;
  const MlpLayout L = mlp_layout(N, K, M, r, 1, true, num_sms());
  if (!ws || !aligned16(ws) || ws_bytes < L.partial) return QLORA_ERR_WORKSPACE;
  if (M == 0) {
    if (cudaMemsetAsync(dA, 0, size_t(r) * K * 2, s) != cudaSuccess ||
        cudaMemsetAsync(dB, 0, size_t(N) * r * 2, s) != cudaSuccess ||
        (dbias && cudaMemsetAsync(dbias, 0, size_t(N) * 2, s) != cudaSuccess))
      return QLORA_ERR_CUDA;
    return QLORA_OK;
  }
  uint8_t* w = static_cast<uint8_t*>(ws);
  float* part = reinterpret_cast<float*>(w + L.partial);
  const size_t region = ws_bytes - L.partial;
  const bool short_dx = dX && short_fits(W, M, 1, true, region);
  const bool stream_dx = dX && !short_dx && stream_fits(W, M, 1, true, region);
  if (!T) {
    st = project_t(W, nullptr, X, A, nullptr, w + L.t, w + L.zs, M, r, scale, ws, s);
    if (st != QLORA_OK) return st;
    T = w + L.t;
  }
  void* const grad[1] = {act == QLORA_ACT_NONE ? nullptr : w + L.grad};
  void* const z[1] = {w + L.u};
  void* const z_lo[1] = {w + L.u_lo};
  const void* const Bs[1] = {B};
  const float* const ts[1] = {ts_of(W)};
  float* bias_part = dbias ? reinterpret_cast<float*>(w + L.bias) : nullptr;
  st = launch_act_down(1, act, dY, act == QLORA_ACT_NONE ? nullptr : Z, nullptr, Bs, ts, grad, z, z_lo,
                       w + L.zs, bias_part, M, N, r, scale, short_dx ? short_zs_mul(W) : 1.0f, w + L.sums, ws, s);
  if (st != QLORA_OK) return st;
  const void* dZ = act == QLORA_ACT_NONE ? dY : grad[0];
  auto side_work = [&](cudaStream_t q) {
    const qlora_status_t e = launch_wgrad(X, dZ, T, z[0], M, N, K, r, scale, dA, dB, ws, nullptr, 1, false, q, z_lo[0]);
    if (e != QLORA_OK || !dbias) return e;
    BiasSumParams b{bias_part, static_cast<__nv_bfloat16*>(dbias), int((M + 127) / 128), int(N)};
    LaunchScope scope(kKindBiasSum, q);
    if (launch_pdl(qlora_bias_sum_kernel, dim3(unsigned((N + 255) / 256)), dim3(256), 0, q, b) != cudaSuccess ||
        cudaGetLastError() != cudaSuccess)
      return QLORA_ERR_CUDA;
    return QLORA_OK;
  };
  if (!dX) return side_work(s);
  const bool early = M <= kWgradFirstRows;
  if (early && (st = side_work(s)) != QLORA_OK) return st;
  auto run_dx = [&]() {
    if (short_dx) return launch_short(W, true, dZ, w + L.zs, A, dX, M, r, ws, part, region, s, early);
    if (stream_dx)
      return launch_stream(W, true, dZ, w + L.zs, A, dX, M, r, ws_status(ws), part, region, s, early);
    FusedExParams p{};
    int grid = 0;
    const SplitPlan sp = split_dx(N, K, M, r, 1, num_sms(), region);
    qlora_status_t e = fill_fused(p, W, true, dZ, w + L.zs, r, A, dX, M, r, fused::BN, ws_status(ws), sp, part, grid);
    if (e != QLORA_OK) return e;
    e = launch_fused_ex<true, kEpiAct>(W->fmt, p, grid, early, s);
    return e != QLORA_OK || sp.S == 1 ? e : launch_split(p, p.K, false, s);
  };
  return early ? run_dx() : fork_join(s, side_work, run_dx);
}

}  // extern "C"
