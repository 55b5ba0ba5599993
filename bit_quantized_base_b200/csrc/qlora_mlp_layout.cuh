// qlora_mlp_layout.cuh -- workspace of the gated MLP and the linear layer with an epilogue (included
// by qlora.cu before qlora_workspace_size).
#pragma once

namespace qlora {
namespace {

// n = 2 (gated) or 1 weights.  header | Zs [M, n r] | T [n][M, r] | backward: U [n][M, r],
// gradients of the pre-activations [n][M, N] bf16, the projection's cluster sums, bias partials
// [ceil(M/128)][N] fp32 (n = 1), and the short-batch kernels' fp32 partials.
// fp32 partials of the narrow kernel (batches of up to 16 rows): two pieces per CTA.
size_t narrow_partial_bytes(int64_t M, int64_t sms) {
  return M > 0 && M <= narrow::kMaxRows ? size_t(sms) * 2 * narrow::partial_floats(int(M)) * 4 : 0;
}

struct MlpLayout {
  size_t zs, t, u, grad, sums, bias, partial, total;
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
    L.grad = take(m * size_t(n) * size_t(N) * 2);
    L.sums = take(size_t(n) * down_sum_bytes(r));
    L.bias = take(n == 1 ? (m + 127) / 128 * size_t(N) * 4 : 0);
  }
  L.partial = off;
  size_t pb = narrow_partial_bytes(M, sms);
  if (bwd && n == 1 && M > 0 && M <= shortk::kMaxRows) pb = std::max(pb, short_plan(N, K, M, true, sms).partial_bytes);
  if (bwd && n == 1 && use_stream(M, 1)) pb = std::max(pb, stream_plan(N, K, M, true, sms).partial_bytes);
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
