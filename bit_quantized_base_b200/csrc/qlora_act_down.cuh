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
// U leaves as the sum of two bf16 tensors, its rounded value and the rest: dA = s U^T X multiplies both
// (qlora_lora_wgrad_kernel<true>), so that the roundings of dA are the gradient's and its own.
//
// Batches of one row tile (LO): the gradients too enter U in two bf16 terms, the second from operand tiles
// of its own.  U of a few rows is so few values that a rounding of dU is not averaged out: dA of one row
// and rank 8 was off by up to 1.9 times its own rounding.  More rows have thousands of values, whose
// error the square root of two bounds, and are not latency bound.
//
// Work split: 128-row tiles, the N columns of a tile over S CTAs (about two per SM in all, at least
// two 64-column chunks each); every CTA writes its binary32 sums to the workspace and
// qlora_down_sum_kernel adds them in split order.  (Clusters of CTAs adding through distributed
// shared memory took 6 to 10 us for that at rank 64, most of a short batch's time.)
//
// 256 threads, two CTAs per SM: all load (one 64-column chunk ahead, in registers), differentiate, and
// write the gradients and the swizzled operand tiles (two stages); one thread also copies the chunks'
// rows of B (TMA) and issues the MMAs, a chunk behind so that it never waits for the other warps; at
// the end four warps drain the accumulators.
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
// two stages of operand tiles (lo: and as many of their roundings) and rows of B, barriers, bias partials
__host__ __device__ constexpr size_t smem_bytes(int nb, bool lo) {
  return 1024 + size_t(2 * nb) * ((lo ? 2 : 1) * T_BYTES + R_BYTES) + 256 + kWarps * 256;
}

}  // namespace actdown

struct ActDownParams {
  CUtensorMap tm_r[2];               // B of each stream: [1, N, r], box {rpad, 64, 1}
  const __nv_bfloat16 *dy, *a0, *a1; // gated: dH, G, U; plain: dY, Z (or null: act none)
  __nv_bfloat16* grad[2];            // [M, N] out: dG, dU / dZ (or null: dZ is dY itself)
  float* part;                       // [S][M][NB r] out: the splits' sums, stream b at column b r
  const float *ts0, *ts1;            // NVFP4: tensor scales of the streams' weights, else null
  float* bias_part;                  // NB = 1: [tiles][N] partial column sums, or null
  int* status;
  int M, N, r, rpad, num_k, S, sps;
};

template <int NB, int ACT, bool LO>
__global__ void __launch_bounds__(actdown::kThreads, LO ? 1 : 2)
qlora_act_down_kernel(const __grid_constant__ ActDownParams p) {
  using namespace actdown;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  constexpr int NT = LO ? 2 * NB : NB;           // operand tiles of a stage: NB, then their roundings
  uint8_t* tail = smem + size_t(2 * NT) * T_BYTES + size_t(2 * NB) * R_BYTES;
  uint64_t* bars = reinterpret_cast<uint64_t*>(tail);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 8);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  float* s_bias = reinterpret_cast<float*>(tail + 256);          // [kWarps][64]
  const uint32_t b0 = ptx::smem_u32(bars);
  // per stage q = chunk % 2: operand tiles written, multiplied; rows of B there
  auto full = [&](uint32_t q) { return b0 + 8u * q; };
  auto empty = [&](uint32_t q) { return b0 + 16u + 8u * q; };
  auto b_full = [&](uint32_t q) { return b0 + 32u + 8u * q; };
  const uint32_t acc_full = b0 + 48u;
  auto tile = [&](uint32_t q, int b) { return ptx::smem_u32(smem) + (q * NT + uint32_t(b)) * uint32_t(T_BYTES); };
  auto rtile = [&](uint32_t q, int b) {
    return ptx::smem_u32(smem) + uint32_t(2 * NT * T_BYTES) + (q * NB + uint32_t(b)) * uint32_t(R_BYTES);
  };

  const int mt = int(blockIdx.x) / p.S, split = int(blockIdx.x) % p.S;
  const int m0 = mt * BM;
  const int ks0 = split * p.sps, ks1 = min(ks0 + p.sps, p.num_k);   // never empty
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (uint32_t q = 0; q < 2; ++q) {
      ptx::mbar_init(full(q), kWarps);
      ptx::mbar_init(empty(q), 1);
      ptx::mbar_init(b_full(q), 1);
    }
    ptx::mbar_init(acc_full, 1);
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
  auto copy_b = [&](int ks) {
    const uint32_t q = uint32_t(ks - ks0) & 1u;
    ptx::mbar_arrive_expect_tx(b_full(q), uint32_t(NB) * r_bytes);
    for (int b = 0; b < NB; ++b) ptx::tma_load_3d(rtile(q, b), &p.tm_r[b], b_full(q), 0, ks * BK, 0);
  };
  const uint32_t idesc = ptx::idesc_bf16(128, uint32_t(p.rpad), 0u, 1u);
  const uint32_t rsw = swz_mode_for_row_bytes(rowb);
  // thread 0: the MMAs of chunk n, whose tiles every warp has written or is about to
  auto multiply = [&](uint32_t n) {
    const uint32_t q = n & 1u, ph = (n >> 1) & 1u;
    if (!ptx::mbar_wait(full(q), ph, p.status, abort_flag) || !ptx::mbar_wait(b_full(q), ph, p.status, abort_flag))
      return;
    ptx::tc_fence_after();
    for (int b = 0; b < NB; ++b)
      for (int kk = 0; kk < BK / 16; ++kk) {
        const uint64_t ad = ptx::smem_desc(tile(q, b) + kk * 32, 16, 1024, ptx::kSw128);
        const uint64_t bd = ptx::smem_desc(rtile(q, b) + kk * 16 * rowb, 64 * rowb, 8 * rowb, rsw);
        ptx::mma_bf16(tmem + uint32_t(b) * 64u, ad, bd, idesc, (n > 0 || kk > 0) ? 1u : 0u);
        if constexpr (LO)
          ptx::mma_bf16(tmem + uint32_t(b) * 64u, ptx::smem_desc(tile(q, NB + b) + kk * 32, 16, 1024, ptx::kSw128),
                        bd, idesc, 1u);
      }
    ptx::mma_commit(empty(q));
  };
  if (threadIdx.x == 0) {
    copy_b(ks0);
    if (ks0 + 1 < ks1) copy_b(ks0 + 1);
  }
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
      const uint32_t q = n & 1u;
      // the chunk before last has been multiplied: its operand tiles and rows of B are free (a wait
      // that gave up skips the shared-memory writes but not the barriers below, which all warps must
      // reach)
      const bool stage_ok = ptx::mbar_wait(empty(q), ((n >> 1) & 1u) ^ 1u, p.status, abort_flag);
      if (threadIdx.x == 0 && stage_ok && n >= 2) copy_b(ks);
      float bsum[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) bsum[j] = 0.0f;
#pragma unroll
      for (int i = 0; i < kVec; ++i) {
        const uint32_t wd[4] = {d[i].x, d[i].y, d[i].z, d[i].w};
        const uint32_t wg[4] = {g[i].x, g[i].y, g[i].z, g[i].w};
        uint32_t wu[4] = {0u, 0u, 0u, 0u};
        if constexpr (NB == 2) { wu[0] = u[i].x; wu[1] = u[i].y; wu[2] = u[i].z; wu[3] = u[i].w; }
        uint32_t hi[NB][4], out1[4];
        [[maybe_unused]] uint32_t lo[NB][4];
        auto rest = [](float x0, float x1, uint32_t h) {   // what the rounding to h left
          return ptx::cvt_bf16x2(x0 - __uint_as_float(h << 16), x1 - __uint_as_float(h & 0xFFFF0000u));
        };
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float x0, x1, y0, y1;
          pair_grad(__uint_as_float(wd[j] << 16), __uint_as_float(wg[j] << 16),
                    __uint_as_float(wu[j] << 16), x0, y0);
          pair_grad(__uint_as_float(wd[j] & 0xFFFF0000u), __uint_as_float(wg[j] & 0xFFFF0000u),
                    __uint_as_float(wu[j] & 0xFFFF0000u), x1, y1);
          if constexpr (NB == 1) { bsum[2 * j] += x0; bsum[2 * j + 1] += x1; }
          hi[0][j] = ptx::cvt_bf16x2(x0, x1);
          if constexpr (LO) lo[0][j] = rest(x0, x1, hi[0][j]);
          if constexpr (NB == 2) {
            hi[1][j] = ptx::cvt_bf16x2(y0, y1);
            if constexpr (LO) lo[1][j] = rest(y0, y1, hi[1][j]);
            out1[j] = p.ts1 ? ptx::cvt_bf16x2(y0 * up_ratio, y1 * up_ratio) : hi[1][j];
          }
        }
        load(ks + 1, i);                         // the vector's place in the next chunk, as soon as it is free
        const int lr = vr + kRowStep * i, row = m0 + lr, col = ks * BK + vc * 8;
        const uint32_t off = uint32_t(lr) * 128u + ((uint32_t(vc) ^ (uint32_t(lr) & 7u)) << 4);
#pragma unroll
        for (int b = 0; b < NB && stage_ok; ++b) {
          ptx::st_shared_v4(tile(q, b) + off, hi[b][0], hi[b][1], hi[b][2], hi[b][3]);
          if constexpr (LO) ptx::st_shared_v4(tile(q, NB + b) + off, lo[b][0], lo[b][1], lo[b][2], lo[b][3]);
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
      if (lane == 0 && stage_ok) ptx::mbar_arrive(full(q));
      if (threadIdx.x == 0 && n > 0) multiply(n - 1);
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

  // ------------------------------------------------------------------ sums of this split
  if (threadIdx.x == 0) {
    multiply(uint32_t(ks1 - ks0 - 1));
    ptx::mma_commit(acc_full);
  }
  __syncwarp();
  if (warp < 4) {
    const bool ok = ptx::mbar_wait(acc_full, 0, p.status, abort_flag);
    __syncwarp();
    ptx::tc_fence_after();
    const int row = m0 + warp * 32 + lane;
    float* dst = p.part + (size_t(split) * p.M + size_t(row)) * size_t(NB * p.r);
#pragma unroll 1
    for (int b = 0; b < NB; ++b) {
      float acc[64];
      load_acc_row(tmem + (uint32_t(warp * 32) << 16) + uint32_t(b) * 64u, p.rpad, acc);
      if (ok && row < p.M && *abort_flag == 0) {
#pragma unroll
        for (int c = 0; c < 64; c += 4)
          if (c < p.r)
            *reinterpret_cast<float4*>(dst + b * p.r + c) = make_float4(acc[c], acc[c + 1], acc[c + 2], acc[c + 3]);
      }
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  if (warp == 0) ptx::tmem_dealloc(tmem, kTmemCols);
}

// U of each stream from the splits' sums, in split order: 32 groups of 4 columns a CTA, 8 slices of
// the splits each, added in slice order.  Writes U as hi + lo and the dX kernel's operand Zs.
struct DownSumParams {
  const float* part;                 // [S][M][width], stream b at column b r
  __nv_bfloat16 *hi[2], *lo[2];      // [M, r] each
  __nv_bfloat16* zs;                 // [M, width] = bf16(U s zs_mul / ts)
  const float* ts;                   // the first weight's tensor scale, or null
  long long groups;                  // M * width / 4
  int S, r, width;
  float s, zs_mul;                   // zs_mul: as DownParams
};
__global__ void __launch_bounds__(256) qlora_down_sum_kernel(const __grid_constant__ DownSumParams p) {
  __shared__ float4 sm[8][32];
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  const int c = int(threadIdx.x) & 31, sl = int(threadIdx.x) >> 5;
  const long long q = (long long)blockIdx.x * 32 + c;
  const int per = (p.S + 7) / 8;
  float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  if (q < p.groups) {
    const float4* src = reinterpret_cast<const float4*>(p.part) + q;
    const int s1 = min(p.S, (sl + 1) * per);
#pragma unroll 4
    for (int k = sl * per; k < s1; ++k) {
      const float4 v = __ldcg(src + size_t(k) * size_t(p.groups));
      a.x += v.x; a.y += v.y; a.z += v.z; a.w += v.w;
    }
  }
  sm[sl][c] = a;
  __syncthreads();
  if (sl != 0 || q >= p.groups) return;
  for (int k = 1; k < 8 && k * per < p.S; ++k) {
    const float4 v = sm[k][c];
    a.x += v.x; a.y += v.y; a.z += v.z; a.w += v.w;
  }
  const long long row = q * 4 / p.width;
  const int col = int(q * 4 - row * p.width);
  const int b = col >= p.r ? 1 : 0;
  const size_t o = size_t(row) * p.r + (col - b * p.r);
  const uint32_t h0 = ptx::cvt_bf16x2(a.x, a.y), h1 = ptx::cvt_bf16x2(a.z, a.w);
  // (an infinite or NaN sum is all in hi)
  auto rest = [](float x, uint32_t h16) {
    const float d = x - __uint_as_float(h16 << 16);
    return d - d == 0.0f ? d : 0.0f;
  };
  *reinterpret_cast<uint2*>(p.hi[b] + o) = make_uint2(h0, h1);
  *reinterpret_cast<uint2*>(p.lo[b] + o) =
      make_uint2(ptx::cvt_bf16x2(rest(a.x, h0 & 0xFFFFu), rest(a.y, h0 >> 16)),
                 ptx::cvt_bf16x2(rest(a.z, h1 & 0xFFFFu), rest(a.w, h1 >> 16)));
  const float zs = p.s / (p.ts ? __ldg(p.ts) : 1.0f) * p.zs_mul;
  *reinterpret_cast<uint2*>(p.zs + size_t(row) * p.width + col) =
      make_uint2(ptx::cvt_bf16x2(a.x * zs, a.y * zs), ptx::cvt_bf16x2(a.z * zs, a.w * zs));
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
