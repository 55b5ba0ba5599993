// qlora_norm_host.cuh -- launch plans of the RMS norm kernels (included by qlora.cu).
#pragma once

namespace qlora {
namespace {

// G threads per row, V vectors of 8 elements each: V is kept at most `want` where 1024 threads
// allow it.
struct NormPlan {
  int G, V, threads, groups;
};

NormPlan norm_plan(int64_t K, int want) {
  NormPlan p{};
  const int nv = int(K / 8);
  p.G = 32;
  while (p.G < 1024 && nv > want * p.G) p.G *= 2;
  p.V = (nv + p.G - 1) / p.G;
  p.threads = norm::cta_threads(p.G);
  p.groups = p.threads / p.G;
  return p;
}

// Vectors a thread should hold.  Groups of 1024 threads leave one CTA per SM, whose barriers stop all
// its loads: they are for rows that nothing smaller holds.  Up to there fewer vectors shorten the way
// from the load to the store, more of them keep more rows per SM in flight.  Measured, microseconds
// with 1 / 2 / 4 vectors: forward 592 x 4096 6.6 / 5.1 / 5.1, 148 x 7168 3.6 / 2.8 / 2.8, 300 x 7168
// 9.7 / 6.2 / 5.5, 300 x 1024 2.0 / 2.1 / 2.2; backward with 1 / 2 (it holds the dgamma sums as well
// and stops there) 592 x 7168 13.3 / 9.9, 64 x 4096 2.9 / 2.4, 64 x 1024 2.1 / 2.4.
int norm_vectors(int64_t M, int64_t K, int sms, bool bwd) {
  if (K <= 2048 && M <= (bwd ? 2 : 4) * int64_t(sms)) return 1;
  if (bwd) return 2;
  return (K <= 4096 && M <= 4 * int64_t(sms)) || (K <= 8192 && M <= sms) ? 2 : 4;
}

// The (V, T) that norm_plan makes of those.
template <bool MX, int V, int T>
cudaError_t launch_norm_fwd_t(unsigned grid, const NormFwdParams& p, cudaStream_t st) {
  return launch_pdl(qlora_norm_fwd_kernel<V, MX, T>, dim3(grid), dim3(T), 0, st, p);
}

template <bool MX>
cudaError_t launch_norm_fwd(const NormPlan& np, unsigned grid, const NormFwdParams& p, cudaStream_t st) {
  switch (np.threads * 8 + np.V) {
    case 256 * 8 + 1: return launch_norm_fwd_t<MX, 1, 256>(grid, p, st);
    case 256 * 8 + 2: return launch_norm_fwd_t<MX, 2, 256>(grid, p, st);
    case 256 * 8 + 3: return launch_norm_fwd_t<MX, 3, 256>(grid, p, st);
    case 256 * 8 + 4: return launch_norm_fwd_t<MX, 4, 256>(grid, p, st);
    case 512 * 8 + 2: return launch_norm_fwd_t<MX, 2, 512>(grid, p, st);
    case 512 * 8 + 3: return launch_norm_fwd_t<MX, 3, 512>(grid, p, st);
    case 512 * 8 + 4: return launch_norm_fwd_t<MX, 4, 512>(grid, p, st);
    case 1024 * 8 + 3: return launch_norm_fwd_t<MX, 3, 1024>(grid, p, st);
    default: return launch_norm_fwd_t<MX, 4, 1024>(grid, p, st);
  }
}

template <bool DG, int V, int T>
cudaError_t launch_norm_bwd_t(unsigned grid, const NormBwdParams& p, cudaStream_t st) {
  // the ring; with several groups of at most 2 vectors it is larger than their sums [groups - 1][K]
  const size_t smem = size_t(norm::bwd_stages(V, T)) * norm::bwd_stage_bytes(V, T);
  if (!set_smem(qlora_norm_bwd_kernel<V, DG, T>, smem)) return cudaErrorInvalidValue;
  return launch_pdl(qlora_norm_bwd_kernel<V, DG, T>, dim3(grid), dim3(T), smem, st, p);
}

template <bool DG>
cudaError_t launch_norm_bwd(const NormPlan& np, unsigned grid, const NormBwdParams& p, cudaStream_t st) {
  switch (np.threads * 8 + np.V) {
    case 256 * 8 + 1: return launch_norm_bwd_t<DG, 1, 256>(grid, p, st);
    case 256 * 8 + 2: return launch_norm_bwd_t<DG, 2, 256>(grid, p, st);
    case 512 * 8 + 2: return launch_norm_bwd_t<DG, 2, 512>(grid, p, st);
    case 1024 * 8 + 2: return launch_norm_bwd_t<DG, 2, 1024>(grid, p, st);
    case 1024 * 8 + 3: return launch_norm_bwd_t<DG, 3, 1024>(grid, p, st);
    default: return launch_norm_bwd_t<DG, 4, 1024>(grid, p, st);
  }
}

// CTAs of the backward kernel: every row has a group, and no more than the SMs hold at once.  Each CTA
// writes one partial row of dgamma, so the count also sizes the workspace.
int64_t norm_bwd_ctas(const NormPlan& np, int64_t M, int sms) {
  const int64_t need = (M + np.groups - 1) / np.groups;
  const int64_t most = int64_t(sms) * norm::bwd_per_sm(np.threads);
  return need < most ? need : most;
}

qlora_status_t check_norm(int64_t M, int64_t K, float eps) {
  if (M < 0 || M > (int64_t(1) << 31) - 512 || K < 8 || K % 8 != 0) return QLORA_ERR_INVALID_ARG;
  if (!(eps >= 0.0f) || !(eps <= 3.0e38f)) return QLORA_ERR_INVALID_ARG;
  return K > norm::kMaxK ? QLORA_ERR_UNSUPPORTED : QLORA_OK;
}

bool opt_ok(const void* p) { return p == nullptr || aligned16(p); }

}  // namespace
}  // namespace qlora

extern "C" {

size_t qlora_rmsnorm_workspace_size(int64_t M, int64_t K) {
  if (check_norm(M, K, 0.0f) != QLORA_OK) return 0;
  const int sms = num_sms();
  const NormPlan np = norm_plan(K, norm_vectors(M, K, sms, true));
  const int64_t rows = norm_bwd_ctas(np, M, sms);
  return align_up(size_t(rows > 0 ? rows : 1) * size_t(K) * 4, 256);
}

qlora_status_t qlora_rmsnorm_fwd(const void* X, const void* R, const void* gamma, float eps, void* S,
                                 void* Y, void* codes, void* scales, float* rstd, int64_t M,
                                 int64_t K, qlora_stream_t stream) {
  const qlora_status_t st = check_norm(M, K, eps);
  if (st != QLORA_OK) return st;
  if (!act_ok(X, M) || !opt_ok(R) || !opt_ok(gamma) || !opt_ok(S) || !opt_ok(Y) || !opt_ok(codes) ||
      !opt_ok(scales) || !opt_ok(rstd))
    return QLORA_ERR_INVALID_ARG;
  if ((codes == nullptr) != (scales == nullptr) || (S && (!R || S == Y)) || (codes && K % 32 != 0))
    return QLORA_ERR_INVALID_ARG;
  if (M == 0) return QLORA_OK;
  if (!Y && !codes) return QLORA_ERR_INVALID_ARG;
  const NormPlan np = norm_plan(K, norm_vectors(M, K, num_sms(), false));
  NormFwdParams p{};
  p.x = static_cast<const __nv_bfloat16*>(X);
  p.res = static_cast<const __nv_bfloat16*>(R);
  p.gamma = static_cast<const __nv_bfloat16*>(gamma);
  p.s = static_cast<__nv_bfloat16*>(S);
  p.y = static_cast<__nv_bfloat16*>(Y);
  p.codes = static_cast<uint8_t*>(codes);
  p.scales = static_cast<uint8_t*>(scales);
  p.rstd = rstd;
  p.M = M;
  p.K = int(K);
  p.G = np.G;
  p.eps = eps;
  const unsigned grid = unsigned((M + np.groups - 1) / np.groups);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  LaunchScope scope(kKindNormFwd, s);
  const cudaError_t e = codes ? launch_norm_fwd<true>(np, grid, p, s) : launch_norm_fwd<false>(np, grid, p, s);
  if (e != cudaSuccess) return QLORA_ERR_CUDA;
  return cudaGetLastError() == cudaSuccess ? QLORA_OK : QLORA_ERR_CUDA;
}

qlora_status_t qlora_rmsnorm_bwd(const void* S, const float* rstd, const void* gamma, float eps,
                                 const void* dY, const void* dS_in, void* dS, void* dgamma, int64_t M,
                                 int64_t K, void* ws, size_t ws_bytes, qlora_stream_t stream) {
  const qlora_status_t st = check_norm(M, K, eps);
  if (st != QLORA_OK) return st;
  if (!act_ok(S, M) || !act_ok(dY, M) || !act_ok(dS, M) || !opt_ok(rstd) || !opt_ok(gamma) ||
      !opt_ok(dS_in) || !opt_ok(dgamma))
    return QLORA_ERR_INVALID_ARG;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const int sms = num_sms();
  const NormPlan np = norm_plan(K, norm_vectors(M, K, sms, true));
  const int64_t ctas = norm_bwd_ctas(np, M, sms);
  if (dgamma && (!ws || !aligned16(ws) || ws_bytes < size_t(ctas) * size_t(K) * 4))
    return QLORA_ERR_WORKSPACE;
  if (M == 0) {
    if (dgamma && cudaMemsetAsync(dgamma, 0, size_t(K) * 2, s) != cudaSuccess) return QLORA_ERR_CUDA;
    return QLORA_OK;
  }
  NormBwdParams p{};
  p.s = static_cast<const __nv_bfloat16*>(S);
  p.gamma = static_cast<const __nv_bfloat16*>(gamma);
  p.dy = static_cast<const __nv_bfloat16*>(dY);
  p.ds_in = static_cast<const __nv_bfloat16*>(dS_in);
  p.rstd = rstd;
  p.ds = static_cast<__nv_bfloat16*>(dS);
  p.part = static_cast<float*>(ws);
  p.M = M;
  p.K = int(K);
  p.G = np.G;
  p.eps = eps;
  {
    LaunchScope scope(kKindNormBwd, s);
    const cudaError_t e = dgamma ? launch_norm_bwd<true>(np, unsigned(ctas), p, s)
                                 : launch_norm_bwd<false>(np, unsigned(ctas), p, s);
    if (e != cudaSuccess || cudaGetLastError() != cudaSuccess) return QLORA_ERR_CUDA;
  }
  if (dgamma) {
    NormDgammaParams q{};
    q.part = static_cast<const float*>(ws);
    q.dgamma = static_cast<__nv_bfloat16*>(dgamma);
    q.P = int(ctas);
    q.K = int(K);
    LaunchScope scope(kKindNormDgamma, s);
    if (launch_pdl(qlora_norm_dgamma_kernel, dim3(unsigned((K + 31) / 32)), dim3(512), 0, s, q) !=
            cudaSuccess ||
        cudaGetLastError() != cudaSuccess)
      return QLORA_ERR_CUDA;
  }
  return QLORA_OK;
}

}  // extern "C"
