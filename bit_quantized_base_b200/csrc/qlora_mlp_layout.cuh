// qlora_mlp_layout.cuh -- workspace of the gated MLP and the linear layer with an epilogue (included
// by qlora.cu before qlora_workspace_size).
#pragma once

namespace qlora {
namespace {

// Work items a pair tile's contraction is split into (1: not).  A pair takes about 0.5 us for a step
// of a 512-row tile and 0.35 us for one of at most 256 rows; a split costs its fp32 accumulators,
// written and read once, and a launch.  Items for more than nine tenths of the pairs count as another
// round: the last pairs wait for SMs that the kernel before still holds (128 x 2048, 14336 deep: 72
// items 40 us, 64 items 32).  Measured on whole calls against the best of 1..16 items: within 4 % for
// 33 x 2 x 2048 from 7168 (1: 72 us, best 4: 34), 1021 x 2048 from 8192 (119, best 3: 78), 300 x 4096
// from 4096 (71, best 3: 33), 200 x 2 x 14336 from 4096 (best 1: 89; 2: 106).
// `room`: bytes for the accumulators.
struct SplitPlan {
  int S;
  size_t bytes;
};
SplitPlan split_plan(int64_t M, int64_t tiles, int64_t steps, int64_t width, int sms, size_t room) {
  SplitPlan best{1, 0};
  if (M <= 0) return best;
  const int64_t pairs = sms / 2;
  const int64_t filled = pairs * 9 / 10;
  const double step_us = M > 256 ? 0.5 : 0.35;
  double cost = double((tiles + pairs - 1) / pairs) * double(steps) * step_us;
  for (int S = 2; S <= 16 && steps / S >= 4; ++S) {
    const size_t bytes = size_t(S) * size_t(M) * size_t(width) * 4;
    if (bytes > room) break;
    const double c = double((tiles * S + filled - 1) / filled) * double((steps + S - 1) / S) * step_us + 5.0 +
                     double(bytes) * 2 / 4.0e6;
    if (c < 0.95 * cost) {
      cost = c;
      best = SplitPlan{S, bytes};
    }
  }
  return best;
}
int64_t row_tiles(int64_t M) { return (M + fused::BM - 1) / fused::BM; }
// The fused kernel's tiles and steps: forward of n weights, dX of n weights.
SplitPlan split_fwd(int64_t N, int64_t K, int64_t M, int r, int n, int sms, size_t room) {
  const int64_t cols = n == 2 ? fused::HN : fused::BN;
  return split_plan(M, row_tiles(M) * ((N + cols - 1) / cols), (K + 63) / 64 + (n * r + 63) / 64, n * N, sms, room);
}
SplitPlan split_dx(int64_t N, int64_t K, int64_t M, int r, int n, int sms, size_t room) {
  return split_plan(M, row_tiles(M) * ((K + fused::BN - 1) / fused::BN), n * ((N + 63) / 64) + (n * r + 63) / 64, K,
                    sms, room);
}

// The plan of the act_down kernel: S CTAs a 128-row tile, about two CTAs per SM in all (one for a
// single row tile, whose CTAs hold twice the operand tiles), at least two 64-column chunks each.
struct ActDownPlan {
  int tiles, S, sps, num_k;
};
ActDownPlan act_down_plan(int64_t M, int64_t N, int sms) {
  ActDownPlan p{};
  p.tiles = int((M + 127) / 128);
  p.num_k = int((N + 63) / 64);
  const int most = std::max(1, std::min(p.tiles > 1 ? 2 * sms / p.tiles : sms, p.num_k / 2));
  p.sps = (p.num_k + most - 1) / most;
  p.S = (p.num_k + p.sps - 1) / p.sps;                          // no split is empty
  return p;
}
// Bytes that its sums take at most, for M rows and any fewer: S M <= 128 * 2 SMs, and S <= chunks / 2.
size_t act_down_sum_bytes(int64_t M, int64_t N, int nb, int r, int sms) {
  const int64_t num_k = (N + 63) / 64;
  const int64_t rows = std::max(M, std::min(std::max<int64_t>(1, num_k / 2) * M, int64_t(256) * sms));
  return size_t(rows > 0 ? rows : 0) * size_t(nb) * size_t(r) * 4;
}

// fp32 partials of the narrow kernel (batches of up to 16 rows): two pieces per CTA.
size_t narrow_partial_bytes(int64_t M, int64_t sms) {
  return M > 0 && M <= narrow::kMaxRows ? size_t(sms) * 2 * narrow::partial_floats(int(M)) * 4 : 0;
}

// n = 2 (gated) or 1 weights.  header | Zs [M, n r] | T [n][M, r] | backward: U [n][M, r] and the rest
// of its rounding [n][M, r], gradients of the pre-activations [n][M, N] bf16, the splits' fp32 sums of
// U, bias partials [ceil(M/128)][N] fp32 (n = 1) | fp32 partials or accumulators of the product.
struct MlpLayout {
  size_t zs, t, u, u_lo, grad, sums, bias, partial, total;
};

MlpLayout mlp_layout(int64_t N, int64_t K, int64_t M, int r, int n, bool bwd, int sms) {
  MlpLayout L{};
  const size_t m = size_t(M > 0 ? M : 0);
  size_t off = kHeaderBytes;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off += align_up(bytes, 256);
    return at;
  };
  L.zs = take(m * size_t(n) * r * 2);
  L.t = take(m * size_t(n) * r * 2);
  if (bwd) {
    L.u = take(m * size_t(n) * r * 2);
    L.u_lo = take(m * size_t(n) * r * 2);
    L.grad = take(m * size_t(n) * size_t(N) * 2);
    L.sums = take(act_down_sum_bytes(M, N, n, r, sms));
    L.bias = take(n == 1 ? (m + 127) / 128 * size_t(N) * 4 : 0);
  }
  L.partial = off;
  size_t pb = narrow_partial_bytes(M, sms);
  if (bwd && n == 1 && M > 0 && M <= shortk::kMaxRows) pb = std::max(pb, short_plan(N, K, M, true, sms).partial_bytes);
  if (bwd && n == 1 && use_stream(M, 1)) pb = std::max(pb, stream_plan(N, K, M, true, sms).partial_bytes);
  // (a batch the narrow, short-batch or streaming kernels take needs no split accumulators)
  const size_t any = ~size_t(0);
  if (M > narrow::kMaxRows) pb = std::max(pb, split_fwd(N, K, M, r, n, sms, any).bytes);
  if (bwd) pb = std::max(pb, split_dx(N, K, M, r, n, sms, any).bytes);
  take(pb);
  L.total = off;
  return L;
}

size_t mlp_workspace(int op, const qlora_weight_t* W, int64_t M, int r) {
  const bool gated = op == QLORA_OP_GATED_MLP_FWD || op == QLORA_OP_GATED_MLP_BWD;
  const bool bwd = op == QLORA_OP_GATED_MLP_BWD || op == QLORA_OP_ACT_BWD;
  size_t n = mlp_layout(W->N, W->K, M, r, gated ? 2 : 1, bwd, num_sms()).total;
  // without an activation and a bias the backward pass is the layer's own
  if (op == QLORA_OP_ACT_BWD) n = std::max(n, ws_layout(W->N, W->K, M, r, true, 1, num_sms()).total);
  return n;
}

}  // namespace
}  // namespace qlora
