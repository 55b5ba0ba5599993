// qlora_act_down.cuh -- the first step of the backward pass behind an activation: the gradient of
// the pre-activations and its rank-r projection, in one pass over the saved tensors.
//
//   gated (NB = 2): dG = dH U act'(G), dU = dH act(G);   Ug = dG Bg, Uu = dU Bu
//   plain (NB = 1): dZ = dY act'(Z);                      U  = dZ B;  dbias partials sum_m dZ
//
// The gradients (bf16, the operands of the dX and adapter-gradient products) are written once; the
// projection multiplies them while they are on the chip.  Memory bound: 3 reads and 2 writes (NB =
// 2) of an [M, N] bf16 tensor, which a separate elementwise kernel would follow with 2 more reads.
//
// The projection takes each gradient as the sum of two bf16 values (the rounded gradient and the
// rest of its binary32 value), two MMAs into one accumulator: U then carries no rounding of the
// gradient, and dA = s U^T X, a product of U, only U's own.
//
// Work split: 128-row tiles; the N columns of a tile are split over S CTAs of one cluster (partial
// sums added in split order through distributed shared memory) times C clusters, whose sums go to
// the workspace and are added in cluster order by the last to arrive.  S C tiles fill the SMs twice:
// two CTAs share an SM, so that one computes while the other waits for its loads or its MMAs (one CTA
// per SM with two operand stages took 176 us where this one takes 110, at 4096 x 14336; 91 us of
// traffic at the copy rate).
//
// 256 threads: all load (one 64-column chunk ahead, in registers), differentiate, and write the
// gradients and the swizzled operand tiles; one thread also copies the chunks' rows of B (TMA) and
// issues the MMAs; at the end four warps drain the accumulators.
#pragma once
#include <cuda_bf16.h>
#include "qlora_ptx.cuh"
#include "qlora_act.cuh"
#include "qlora_lora.cuh"

namespace qlora {
namespace actdown {
constexpr int BM = 128, BK = 64;
constexpr int T_BYTES = BM * BK * 2;            // one operand tile: 16 KB
constexpr int R_BYTES = 64 * 128;               // 64 rows of B, up to 64 wide
constexpr int kWarps = 8, kThreads = kWarps * 32;
constexpr int kRowStep = kWarps * 4;            // rows between two vectors of a thread
constexpr int kTmemCols = 128;                  // accumulator of stream b at column 64 b
constexpr int kVec = BM * BK / 8 / kThreads;    // 16-byte vectors a thread holds per tensor
constexpr int kMaxTilesSplit = 240;             // counters: [tiles][S] of them when C > 1
// operand tiles of one chunk, two chunks' rows of B, barriers, bias partials
__host__ __device__ constexpr size_t smem_bytes(int nb) {
  return 1024 + size_t(nb) * (2 * T_BYTES + 2 * R_BYTES) + 256 + kWarps * 256;
}

// What rounding x0, x1 to the bf16 pair `hi` left out, as a bf16 pair (0 where `hi` is infinite or NaN:
// the value is all there).
__device__ __forceinline__ uint32_t rest2(uint32_t hi, float x0, float x1) {
  const uint32_t lo = ptx::cvt_bf16x2(x0 - __uint_as_float(hi << 16), x1 - __uint_as_float(hi & 0xFFFF0000u));
  const uint32_t top = ((hi & 0x7F807F80u) + 0x00800080u) & 0x80008000u;   // halves with a full exponent
  if (top == 0u) return lo;
  return lo & ~((top >> 15) * 0xFFFFu);
}
}  // namespace actdown

struct ActDownParams {
  CUtensorMap tm_r[2];               // B of each stream: [1, N, r], box {rpad, 64, 1}
  const __nv_bfloat16 *dy, *a0, *a1; // gated: dH, G, U; plain: dY, Z (or null: act none)
  __nv_bfloat16* grad[2];            // [M, N] out: dG, dU / dZ (or null: dZ is dY itself)
  __nv_bfloat16* z[2];               // [M, r] out: U of each stream
  __nv_bfloat16* zs;                 // [M, ldzs] out: the dX kernel's LoRA operand, stream b at column b r
  const float *ts0, *ts1;            // NVFP4: tensor scales of the streams' weights, else null
  float* bias_part;                  // NB = 1: [tiles][N] partial column sums, or null
  int* status;
  float* cpart;                      // C > 1: [tiles][C][NB][128][rpad] fp32
  unsigned* ccount;                  // C > 1: [tiles][S] arrival counters, zero between launches
  int M, N, r, rpad, ldzs, num_k, S, C, sps;
  float s;
  float zs_mul;                      // as DownParams
};

template <int NB, int ACT>
__global__ void __launch_bounds__(actdown::kThreads, 2)
qlora_act_down_kernel(const __grid_constant__ ActDownParams p) {
  using namespace actdown;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  uint8_t* tail = smem + size_t(NB) * (2 * T_BYTES + 2 * R_BYTES);
  uint64_t* bars = reinterpret_cast<uint64_t*>(tail);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 6);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile unsigned* s_ticket = reinterpret_cast<volatile unsigned*>(tmem_slot + 2);
  float* s_bias = reinterpret_cast<float*>(tail + 256);          // [kWarps][64]
  const uint32_t b0 = ptx::smem_u32(bars);
  const uint32_t full = b0, empty = b0 + 8u, acc_full = b0 + 16u;    // operand tiles written / multiplied
  auto b_full = [&](int q) { return b0 + 24u + 8u * uint32_t(q); };   // rows of B of an even / odd chunk
  // stream b's rounded tile, the rest's tile; its rows of B
  auto tile = [&](int b, int lo) { return ptx::smem_u32(smem) + uint32_t(2 * b + lo) * T_BYTES; };
  auto rtile = [&](int q, int b) {
    return ptx::smem_u32(smem) + uint32_t(2 * NB) * T_BYTES + uint32_t(q * NB + b) * R_BYTES;
  };

  const int per_tile = p.S * p.C;
  const int mt = int(blockIdx.x) / per_tile, gs = int(blockIdx.x) % per_tile;
  const int split = gs % p.S, cg = gs / p.S;
  const int m0 = mt * BM;
  const int ks0 = min(gs * p.sps, p.num_k), ks1 = min(ks0 + p.sps, p.num_k);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    ptx::mbar_init(full, kWarps);
    ptx::mbar_init(empty, 1);
    ptx::mbar_init(acc_full, 1);
    ptx::mbar_init(b_full(0), 1);
    ptx::mbar_init(b_full(1), 1);
    *abort_flag = 0;
    ptx::fence_mbarrier_init();
  }
  if (warp == 0) {
    ptx::tmem_alloc(ptx::smem_u32(tmem_slot), kTmemCols);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  const uint32_t rowb = uint32_t(p.rpad) * 2u;
  const uint32_t r_bytes = uint32_t(p.rpad) * 128u;
  const float ts0 = p.ts0 ? __ldg(p.ts0) : 1.0f;
  // dX has one accumulator, scaled by the first weight's tensor scale at the end
  const float up_ratio = NB == 2 && p.ts1 ? __ldg(p.ts1) / ts0 : 1.0f;
  const float zscale = p.s / ts0 * p.zs_mul;
  auto write8 = [&](int b, int rw, int c, const float (&v)[8]) {
    if (c >= p.r) return;
    if (!ptx::dcheck(rw >= 0 && rw < p.M, p.status)) return;
    uint4 z, zs;
    z.x = ptx::cvt_bf16x2(v[0], v[1]); z.y = ptx::cvt_bf16x2(v[2], v[3]);
    z.z = ptx::cvt_bf16x2(v[4], v[5]); z.w = ptx::cvt_bf16x2(v[6], v[7]);
    zs.x = ptx::cvt_bf16x2(v[0] * zscale, v[1] * zscale);
    zs.y = ptx::cvt_bf16x2(v[2] * zscale, v[3] * zscale);
    zs.z = ptx::cvt_bf16x2(v[4] * zscale, v[5] * zscale);
    zs.w = ptx::cvt_bf16x2(v[6] * zscale, v[7] * zscale);
    *reinterpret_cast<uint4*>(p.z[b] + size_t(rw) * p.r + c) = z;
    *reinterpret_cast<uint4*>(p.zs + size_t(rw) * p.ldzs + size_t(b) * p.r + c) = zs;
  };

  auto copy_b = [&](int ks) {
    const int q = (ks - ks0) & 1;
    ptx::mbar_arrive_expect_tx(b_full(q), uint32_t(NB) * r_bytes);
    for (int b = 0; b < NB; ++b) ptx::tma_load_3d(rtile(q, b), &p.tm_r[b], b_full(q), 0, ks * BK, 0);
  };
  const uint32_t idesc = ptx::idesc_bf16(128, uint32_t(p.rpad), 0u, 1u);
  const uint32_t rsw = swz_mode_for_row_bytes(rowb);
  if (threadIdx.x == 0 && ks1 > ks0) copy_b(ks0);
  {
    // ---------------------------------------------------------------- gradients and operand tiles
    // Vector i of this thread: row vr + kRowStep i of the tile, columns 8 vc .. 8 vc + 7 of the chunk (a
    // warp covers 4 rows of 128 contiguous bytes).
    const int vc = int(threadIdx.x) & 7, vr = int(threadIdx.x) >> 3;
    uint4 d[kVec], g[kVec], u[NB == 2 ? kVec : 1];
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
    auto load = [&](int ks, int i) {
      const int col = ks * BK + vc * 8;
      const int row = m0 + vr + kRowStep * i;
      const bool ok = row < p.M && col < p.N && ks < ks1;
      const size_t off = size_t(row) * p.N + col;
      d[i] = ok ? ptx::ldg_stream_v4(p.dy + off) : zero;
      g[i] = ok && p.a0 ? ptx::ldg_stream_v4(p.a0 + off) : zero;
      if constexpr (NB == 2) u[i] = ok ? ptx::ldg_stream_v4(p.a1 + off) : zero;
    };
    auto pair_grad = [&](float dd, float gg, float uu, float& o0, float& o1) {
      float a, da;
      act::value_grad<ACT>(gg, a, da);
      o0 = NB == 2 ? dd * uu * da : dd * da;
      o1 = dd * a;
    };
#pragma unroll
    for (int i = 0; i < kVec; ++i) load(ks0, i);
    for (int ks = ks0; ks < ks1; ++ks) {
      const uint32_t n = uint32_t(ks - ks0);
      // the chunk before has been multiplied: its operand tiles and its rows of B are free  (a wait
      // that gave up skips the shared-memory writes but not the barriers below, which all warps
      // must reach)
      const bool stage_ok = ptx::mbar_wait(empty, (n & 1u) ^ 1u, p.status, abort_flag);
      if (threadIdx.x == 0 && stage_ok && ks + 1 < ks1) copy_b(ks + 1);
      float bsum[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) bsum[j] = 0.0f;
#pragma unroll
      for (int i = 0; i < kVec; ++i) {
        const uint32_t wd[4] = {d[i].x, d[i].y, d[i].z, d[i].w};
        const uint32_t wg[4] = {g[i].x, g[i].y, g[i].z, g[i].w};
        uint32_t wu[4] = {0u, 0u, 0u, 0u};
        if constexpr (NB == 2) { wu[0] = u[i].x; wu[1] = u[i].y; wu[2] = u[i].z; wu[3] = u[i].w; }
        uint32_t hi[NB][4], lo[NB][4], out1[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float x0, x1, y0, y1;
          pair_grad(__uint_as_float(wd[j] << 16), __uint_as_float(wg[j] << 16),
                    __uint_as_float(wu[j] << 16), x0, y0);
          pair_grad(__uint_as_float(wd[j] & 0xFFFF0000u), __uint_as_float(wg[j] & 0xFFFF0000u),
                    __uint_as_float(wu[j] & 0xFFFF0000u), x1, y1);
          if constexpr (NB == 1) { bsum[2 * j] += x0; bsum[2 * j + 1] += x1; }
          hi[0][j] = ptx::cvt_bf16x2(x0, x1);
          lo[0][j] = rest2(hi[0][j], x0, x1);
          if constexpr (NB == 2) {
            hi[1][j] = ptx::cvt_bf16x2(y0, y1);
            lo[1][j] = rest2(hi[1][j], y0, y1);
            out1[j] = p.ts1 ? ptx::cvt_bf16x2(y0 * up_ratio, y1 * up_ratio) : hi[1][j];
          }
        }
        load(ks + 1, i);                         // the vector's place in the next chunk, as soon as it is free
        const int lr = vr + kRowStep * i, row = m0 + lr, col = ks * BK + vc * 8;
        const uint32_t off = uint32_t(lr) * 128u + ((uint32_t(vc) ^ (uint32_t(lr) & 7u)) << 4);
#pragma unroll
        for (int b = 0; b < NB && stage_ok; ++b) {
          ptx::st_shared_v4(tile(b, 0) + off, hi[b][0], hi[b][1], hi[b][2], hi[b][3]);
          ptx::st_shared_v4(tile(b, 1) + off, lo[b][0], lo[b][1], lo[b][2], lo[b][3]);
        }
        if (row < p.M && col < p.N) {
          const size_t o = size_t(row) * p.N + col;
          if (p.grad[0])
            *reinterpret_cast<uint4*>(p.grad[0] + o) = make_uint4(hi[0][0], hi[0][1], hi[0][2], hi[0][3]);
          if constexpr (NB == 2)
            *reinterpret_cast<uint4*>(p.grad[1] + o) = make_uint4(out1[0], out1[1], out1[2], out1[3]);
        }
      }
      ptx::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0 && stage_ok) ptx::mbar_arrive(full);
      if (threadIdx.x == 0 && stage_ok && ptx::mbar_wait(full, n & 1u, p.status, abort_flag) &&
          ptx::mbar_wait(b_full(int(n & 1u)), (n >> 1) & 1u, p.status, abort_flag)) {
        ptx::tc_fence_after();
        for (int b = 0; b < NB; ++b)
          for (int lo = 0; lo < 2; ++lo)
            for (int kk = 0; kk < BK / 16; ++kk) {
              const uint64_t ad = ptx::smem_desc(tile(b, lo) + kk * 32, 16, 1024, ptx::kSw128);
              const uint64_t bd =
                  ptx::smem_desc(rtile(int(n & 1u), b) + kk * 16 * rowb, 64 * rowb, 8 * rowb, rsw);
              ptx::mma_bf16(tmem + uint32_t(b) * 64u, ad, bd, idesc, (n > 0 || lo > 0 || kk > 0) ? 1u : 0u);
            }
        ptx::mma_commit(empty);
        if (ks + 1 == ks1) ptx::mma_commit(acc_full);
      }
      __syncwarp();
      if constexpr (NB == 1) {
        if (p.bias_part) {
          // column sums of the tile: over the warp's 4 rows by shuffles, over the warps in order
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            bsum[j] += __shfl_xor_sync(0xFFFFFFFFu, bsum[j], 8);
            bsum[j] += __shfl_xor_sync(0xFFFFFFFFu, bsum[j], 16);
          }
          ptx::named_bar_sync(1, kWarps * 32);
          if (lane < 8)
#pragma unroll
            for (int j = 0; j < 8; ++j) s_bias[warp * 64 + lane * 8 + j] = bsum[j];
          ptx::named_bar_sync(1, kWarps * 32);
          if (threadIdx.x < 64) {
            const int col = ks * BK + int(threadIdx.x);
            float t = 0.0f;
            for (int w = 0; w < kWarps; ++w) t += s_bias[w * 64 + threadIdx.x];
            if (col < p.N) p.bias_part[size_t(mt) * p.N + col] = t;
          }
        }
      }
    }
  }

  // ------------------------------------------------------------------ accumulators to U and Zs
  const bool have = ks1 > ks0;
  const int nrows = min(BM, p.M - m0);
  const uint32_t part = ptx::smem_u32(smem);       // the operand tiles are free by then: stream b at
  constexpr uint32_t PART = 32768u;                // b * PART
  if (warp < 4) {
    if (have) ptx::mbar_wait(acc_full, 0, p.status, abort_flag);
    ptx::named_bar_sync(2, 128);
    if (*abort_flag == 0) {
#pragma unroll 1
      for (int b = 0; b < NB; ++b) {
        float acc[64];
        if (have) {
          ptx::tc_fence_after();
          load_acc_row(tmem + (uint32_t(warp * 32) << 16) + uint32_t(b) * 64u, p.rpad, acc);
        } else {
#pragma unroll
          for (int c = 0; c < 64; ++c) acc[c] = 0.0f;
        }
        if (p.S == 1 && p.C == 1) {
          const int lr = warp * 32 + lane;
          if (lr < nrows) {
#pragma unroll
            for (int c = 0; c < 64; c += 8) {
              float v[8];
#pragma unroll
              for (int q = 0; q < 8; ++q) v[q] = acc[c + q];
              write8(b, m0 + lr, c, v);
            }
          }
        } else {
          store_partial_row(part + uint32_t(b) * PART, warp * 32 + lane, acc, p.rpad);
        }
      }
    }
  }
  if (p.S > 1 || p.C > 1) {
    float* const csum = p.cpart + (size_t(mt) * p.C + cg) * NB * BM * p.rpad;
    ptx::cluster_sync();
    if (warp < 4 && *abort_flag == 0) {
#pragma unroll 1
      for (int b = 0; b < NB; ++b) {
        if (p.C == 1)
          cluster_sum(part + uint32_t(b) * PART, p.rpad, p.S, split, nrows, int(threadIdx.x),
                      [&](int lr, int c, const float (&v)[8]) { write8(b, m0 + lr, c, v); });
        else
          cluster_sum(part + uint32_t(b) * PART, p.rpad, p.S, split, nrows, int(threadIdx.x),
                      [&](int lr, int c, const float (&v)[8]) {
                        float4* dst = reinterpret_cast<float4*>(csum + (size_t(b) * BM + lr) * p.rpad + c);
                        __stcg(dst, make_float4(v[0], v[1], v[2], v[3]));
                        __stcg(dst + 1, make_float4(v[4], v[5], v[6], v[7]));
                      });
      }
    }
    ptx::cluster_sync();
    if (p.C > 1 && warp < 4) {
      unsigned* const counter = p.ccount + mt * p.S + split;
      __threadfence();
      ptx::named_bar_sync(2, 128);
      if (threadIdx.x == 0) *s_ticket = atomicAdd(counter, 1u);
      ptx::named_bar_sync(2, 128);
      if (*s_ticket == unsigned(p.C - 1)) {
        __threadfence();
        const int rows_per = (BM + p.S - 1) / p.S;
        const int r0 = split * rows_per, r1 = min(nrows, r0 + rows_per);
        const int g8 = p.rpad / 8;
        const int items = r1 > r0 ? (r1 - r0) * g8 * NB : 0;
        for (int it = int(threadIdx.x); it < items && *abort_flag == 0; it += 128) {
          const int b = it / ((r1 - r0) * g8), q = it % ((r1 - r0) * g8);
          const int lr = r0 + q / g8, c = (q % g8) * 8;
          float v[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) v[k] = 0.0f;
          for (int k = 0; k < p.C; ++k) {
            const float4* src = reinterpret_cast<const float4*>(
                p.cpart + (((size_t(mt) * p.C + k) * NB + b) * BM + lr) * p.rpad + c);
            const float4 x = __ldcg(src), y = __ldcg(src + 1);
            v[0] += x.x; v[1] += x.y; v[2] += x.z; v[3] += x.w;
            v[4] += y.x; v[5] += y.y; v[6] += y.z; v[7] += y.w;
          }
          write8(b, m0 + lr, c, v);
        }
        if (threadIdx.x == 0) *counter = 0u;
      }
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  if (warp == 0) ptx::tmem_dealloc(tmem, kTmemCols);
}

// dbias[n] = the sum over the row tiles of their partial column sums, in tile order.
struct BiasSumParams {
  const float* part;       // [tiles][N]
  __nv_bfloat16* dbias;    // [N]
  int tiles, N;
};
__global__ void __launch_bounds__(256) qlora_bias_sum_kernel(const __grid_constant__ BiasSumParams p) {
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  const int n = int(blockIdx.x) * 256 + int(threadIdx.x);
  if (n >= p.N) return;
  float a = 0.0f;
#pragma unroll 4
  for (int t = 0; t < p.tiles; ++t) a += __ldcg(p.part + size_t(t) * p.N + n);
  p.dbias[n] = __float2bfloat16_rn(a);
}

}  // namespace qlora
