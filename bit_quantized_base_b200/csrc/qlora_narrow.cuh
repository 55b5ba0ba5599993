// qlora_narrow.cuh -- forward of the gated MLP and of the linear layer with an epilogue for batches of
// at most 64 rows (single tokens, decoding batches): each pass streams the 4-bit weights once.
//
//   qlora_narrow_down_kernel   T = X A^T of one or two adapters in one launch, and Zs = bf16(T s / ts)
//   qlora_narrow_kernel        G and U, or Z, and the whole epilogue in one kernel
//
// What bounds it: reading the weights (one token of a 14336 x 4096 NF4 gate and up: 66 MB, 10 us) and
// the SMs' decode (about 3 integer operations a weight, 20-30 weights a clock and SM).  Here a decoded
// pair of weights goes from the register it was decoded in straight into a warp-level m16n8k16
// tensor-core product (weights the 16-row operand, batch rows the 8 columns), with no barrier, copy
// or hand-off between decode and product: the tcgen05 path has to place every decoded operand in
// shared or tensor memory and synchronise with the issuing thread once per tile, which costs it half
// of the decode rate at these batch sizes.  The warp product's own rate (about 1000 multiply-adds a
// clock and SM) is above the decode's up to about 32 rows.
//
// The order of the contraction is free as long as both operands agree: lane t of a quad takes the
// 64-element block 4 j + t of its two weight rows (32 contiguous code bytes, one block scale), and
// step i of a block multiplies its elements 4 i .. 4 i + 3, so the operand registers are the decoded
// pairs as they come, and the batch operand is a 16-byte piece of X for every two steps.
//
// Work split: a CTA (8 warps) owns 128 columns of the gate and of the up weight (gated; the two
// accumulators of an output sit in the same thread) or 256 columns; S CTAs of a cluster share a
// tile's depth in contiguous ranges of 256-deep chunks and add their sums in rank order through
// distributed shared memory, each finishing a part of the outputs.  Deterministic.
#pragma once
#include <cuda_bf16.h>
#include "qlora_ptx.cuh"
#include "qlora_dequant.cuh"
#include "qlora_fused.cuh"
#include "qlora_act.cuh"

namespace qlora {
namespace narrow {
constexpr int kMaxRows = 64;
constexpr int kWarps = 8, kThreads = kWarps * 32;
constexpr int CK = 256;                    // contraction elements of one chunk: 4 blocks of 64
constexpr int NSTAGE = 3;                  // chunks of X in shared memory
constexpr int RG = 2;                      // 16-row groups per warp (gated: one gate, one up)
constexpr int kRows = kWarps * RG * 16;    // 256 weight rows per CTA tile
constexpr int ROWP = kRows + 4;            // pitch of the fp32 tile in shared memory (no conflicts)
constexpr int kMaxSplit = 8;
// bytes: X chunks (nb blocks of 8 batch rows), then the fp32 tile [8 nb][ROWP]
__host__ __device__ constexpr size_t x_bytes(int nb) { return size_t(nb) * 8 * CK * 2; }
__host__ __device__ constexpr size_t smem_bytes(int nb) {
  return NSTAGE * x_bytes(nb) + size_t(nb) * 8 * ROWP * 4;
}

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// 16-byte asynchronous copy global -> shared; `bytes` 0 writes zeros instead.
__device__ __forceinline__ void cp_async_16(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
// The 32 code bytes of one block.  wide: the address is a multiple of 32.
__device__ __forceinline__ void load_block(uint32_t (&w)[8], const uint8_t* p, bool wide) {
  if (wide) {
    asm volatile("ld.global.nc.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
                 : "l"(p));
  } else {
    const uint4 a = __ldg(reinterpret_cast<const uint4*>(p)), b = __ldg(reinterpret_cast<const uint4*>(p) + 1);
    w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
    w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
  }
}

// One 64-element block's decoder: its table (NF4) or packed scales, then 8 codes at a time.
template <int FMT>
struct BlockDecoder {
  Lut16 lut;
  __device__ __forceinline__ void init(uint32_t raw) { lut = nf4_lut(__uint_as_float(raw)); }
  __device__ __forceinline__ void word(int, uint32_t w, const DecodeMul& k, uint32_t (&o)[4]) const {
    nf4_lookup8_mul(lut, w, k, o);
  }
};
// MXFP4: bit placement times 2^(e-1) for e <= 128, else in two exact multiplies (see qlora_dequant.cuh).
template <>
struct BlockDecoder<kFmtMXFP4> {
  uint32_t s0, s1;
  bool slow;
  __device__ __forceinline__ void init(uint32_t raw) {
    const uint32_t e0 = raw & 0xFFu, e1 = (raw >> 8) & 0xFFu;
    slow = e0 > 128u || e1 > 128u;
    s0 = slow ? mx_exact_scale(e0) : mx_fast_scale(e0);
    s1 = slow ? mx_exact_scale(e1) : mx_fast_scale(e1);
  }
  __device__ __forceinline__ void word(int j, uint32_t w, const DecodeMul& k, uint32_t (&o)[4]) const {
    e2m1_pattern8(w, k, o);
    const uint32_t s = j < 4 ? s0 : s1;
    if (slow) {
#pragma unroll
      for (int i = 0; i < 4; ++i) o[i] = ptx::mul_bf16x2(o[i], kBf16x2Pow126);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = ptx::mul_bf16x2(o[i], s);
  }
};
// NVFP4: elements times 2^-8 (the epilogue multiplies by 2^8 ts; Zs carries the same 2^-8).
template <>
struct BlockDecoder<kFmtNVFP4> {
  uint32_t s[4];
  __device__ __forceinline__ void init(uint32_t raw) {
#pragma unroll
    for (int q = 0; q < 4; ++q) s[q] = nv_shifted_scale((raw >> (8 * q)) & 0xFFu);
  }
  __device__ __forceinline__ void word(int j, uint32_t w, const DecodeMul& k, uint32_t (&o)[4]) const {
    e2m1_pattern8(w, k, o);
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = ptx::mul_bf16x2(o[i], s[j >> 1]);
  }
};
}  // namespace narrow

struct NarrowWeight {
  const uint8_t* codes;              // [N, K/2]
  const void* scales;
  const float *scales2, *tensor_scale;
  const __nv_bfloat16* lora_up;      // B [N, r]
};

struct NarrowParams {
  NarrowWeight w[2];                 // gated: gate, up; else w[0]
  const __nv_bfloat16 *x, *zs;       // [M, K]; [M, ldzs], weight i at column i r
  const __nv_bfloat16 *bias, *residual;
  __nv_bfloat16 *out, *save0, *save1;
  int M, N, K, r, ldzs;
  int tiles, chunks, S, act;
  float ts_mul;                      // 2^8 for NVFP4, else 1
  uint32_t one;                      // 1 (see decode_mul)
  int wide;                          // codes are 32-byte aligned
};

template <int FMT, bool GATED, int NB>
__global__ void __launch_bounds__(narrow::kThreads, 1)
qlora_narrow_kernel(const __grid_constant__ NarrowParams p) {
  using namespace narrow;
  constexpr int COLS = GATED ? kRows / 2 : kRows;      // output columns of a tile
  extern __shared__ __align__(128) uint8_t smem[];
  const uint32_t xs = ptx::smem_u32(smem);
  float* tile = reinterpret_cast<float*>(smem + NSTAGE * x_bytes(NB));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int rank = int(blockIdx.x) % p.S, cluster = int(blockIdx.x) / p.S, clusters = int(gridDim.x) / p.S;
  const int c0 = int((long long)p.chunks * rank / p.S), c1 = int((long long)p.chunks * (rank + 1) / p.S);
  const int blocks = p.K / 64;
  const DecodeMul km = decode_mul(p.one);
  ptx::griddep_launch_dependents();

  // X chunk c into stage s: piece (nb, i, lane) = 8 elements of batch row 8 nb + lane / 4 at block
  // 4 c + lane % 4, element 8 i -- the order in which the products read them
  auto stage_x = [&](int c, int s) {
#pragma unroll
    for (int q = 0; q < NB; ++q) {
      const int v = int(threadIdx.x) + q * kThreads;   // nb = q, i = warp
      const int row = 8 * q + g, blk = 4 * c + t;
      const bool ok = row < p.M && blk < blocks;
      const __nv_bfloat16* src = p.x + (ok ? size_t(row) * p.K + size_t(blk) * 64 + warp * 8 : 0);
      cp_async_16(xs + uint32_t(s) * uint32_t(x_bytes(NB)) + uint32_t(v) * 16u, src, ok ? 16u : 0u);
    }
    ptx::cp_async_commit();
  };
  // Weight rows of this lane: groups q = 0, 1, rows g and g + 8 of each (h), clamped to the weight (a
  // clamped row's results are dropped).
  auto row_of = [&](int tl, int q, int h) {
    const int n = GATED ? tl * COLS + warp * 16 + g + 8 * h : tl * COLS + warp * 32 + q * 16 + g + 8 * h;
    return min(n, p.N - 1);
  };
  auto load_codes_of = [&](int tl, int c, uint32_t (&w)[RG][2][8], uint32_t (&sc)[RG][2]) {
    const int blk = 4 * c + t;
#pragma unroll
    for (int q = 0; q < RG; ++q)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const NarrowWeight& W = p.w[GATED ? q : 0];
        if (blk < blocks) {
          const int n = row_of(tl, q, h);
          load_block(w[q][h], W.codes + (size_t(n) * p.K + size_t(blk) * 64) / 2, p.wide != 0);
          if constexpr (FMT == kFmtNF4DQ)
            sc[q][h] = load_item_scale_dq(W.scales, W.scales2, 0, p.N, n, blk * 64, p.K).raw;
          else
            sc[q][h] = load_item_scale<FMT>(W.scales, n, blk * 64, p.K).raw;
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) w[q][h][i] = 0u;
          sc[q][h] = 0u;
        }
      }
  };

  uint32_t nw[RG][2][8], nsc[RG][2];
  if (cluster < p.tiles && c0 < c1) load_codes_of(cluster, c0, nw, nsc);
  for (int tl = cluster; tl < p.tiles; tl += clusters) {
    float acc[RG][NB][4];
#pragma unroll
    for (int q = 0; q < RG; ++q)
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[q][b][i] = 0.0f;
    for (int s = 0; s < NSTAGE - 1; ++s) {
      if (c0 + s < c1) stage_x(c0 + s, s);
      else ptx::cp_async_commit();
    }
    for (int c = c0; c < c1; ++c) {
      const int s = (c - c0) % NSTAGE;
      uint32_t w[RG][2][8], sc[RG][2];
#pragma unroll
      for (int q = 0; q < RG; ++q)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
          for (int i = 0; i < 8; ++i) w[q][h][i] = nw[q][h][i];
          sc[q][h] = nsc[q][h];
        }
      if (c + 1 < c1) load_codes_of(tl, c + 1, nw, nsc);
      else if (tl + clusters < p.tiles) load_codes_of(tl + clusters, c0, nw, nsc);
      ptx::cp_async_wait<NSTAGE - 2>();
      __syncthreads();                       // chunk c is in place; everyone is done with chunk c - 1
      if (c + NSTAGE - 1 < c1) stage_x(c + NSTAGE - 1, (c - c0 + NSTAGE - 1) % NSTAGE);
      else ptx::cp_async_commit();
      BlockDecoder<FMT> dec[RG][2];
#pragma unroll
      for (int q = 0; q < RG; ++q)
#pragma unroll
        for (int h = 0; h < 2; ++h) dec[q][h].init(sc[q][h]);
      const uint32_t xb = xs + uint32_t(s) * uint32_t(x_bytes(NB)) + uint32_t(lane) * 16u;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        uint32_t a[RG][2][4];
#pragma unroll
        for (int q = 0; q < RG; ++q)
#pragma unroll
          for (int h = 0; h < 2; ++h) dec[q][h].word(i, w[q][h][i], km, a[q][h]);
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          const uint4 x = ptx::ld_shared_v4(xb + uint32_t(b * 8 + i) * 512u);
#pragma unroll
          for (int q = 0; q < RG; ++q) {
            mma16816(acc[q][b], a[q][0][0], a[q][1][0], a[q][0][1], a[q][1][1], x.x, x.y);
            mma16816(acc[q][b], a[q][0][2], a[q][1][2], a[q][0][3], a[q][1][3], x.z, x.w);
          }
        }
      }
    }
    // The LoRA term: rows of B times Zs, by the last rank (Zs comes from the kernel before).
    ptx::griddep_wait();
    if (rank == p.S - 1) {
      for (int k = 0; k < p.r; k += 16) {
        const int ka = k + 2 * t, kb = ka + 8;
#pragma unroll
        for (int q = 0; q < RG; ++q) {
          const NarrowWeight& W = p.w[GATED ? q : 0];
          uint32_t a[2][2];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const __nv_bfloat16* br = W.lora_up + size_t(row_of(tl, q, h)) * p.r;
            a[h][0] = __ldg(reinterpret_cast<const uint32_t*>(br + ka));
            a[h][1] = kb < p.r ? __ldg(reinterpret_cast<const uint32_t*>(br + kb)) : 0u;
          }
#pragma unroll
          for (int b = 0; b < NB; ++b) {
            const int m = 8 * b + g;
            const __nv_bfloat16* zr = p.zs + size_t(m) * p.ldzs + (GATED ? q * p.r : 0);
            const uint32_t z0 = m < p.M ? __ldcg(reinterpret_cast<const uint32_t*>(zr + ka)) : 0u;
            const uint32_t z1 = m < p.M && kb < p.r ? __ldcg(reinterpret_cast<const uint32_t*>(zr + kb)) : 0u;
            mma16816(acc[q][b], a[0][0], a[1][0], a[0][1], a[1][1], z0, z1);
          }
        }
      }
    }
    // fp32 tile [batch row][weight row] (gated: 128 gate rows, then 128 up rows)
#pragma unroll
    for (int q = 0; q < RG; ++q) {
      const int row = GATED ? q * COLS + warp * 16 + g : warp * 32 + q * 16 + g;
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        float* d = tile + size_t(8 * b + 2 * t) * ROWP + row;
        d[0] = acc[q][b][0];
        d[ROWP] = acc[q][b][1];
        d[8] = acc[q][b][2];
        d[ROWP + 8] = acc[q][b][3];
      }
    }
    if (p.S > 1) ptx::cluster_sync();
    else __syncthreads();
    // 8 columns at a time: the ranks' sums in rank order, then the epilogue
    const float ts0 = (p.w[0].tensor_scale ? __ldg(p.w[0].tensor_scale) : 1.0f) * p.ts_mul;
    const float ts1 = GATED ? (p.w[1].tensor_scale ? __ldg(p.w[1].tensor_scale) : 1.0f) * p.ts_mul : 1.0f;
    const uint32_t tile_a = ptx::smem_u32(tile);
    constexpr int G8 = COLS / 8;
    for (int it = rank * kThreads + int(threadIdx.x); it < p.M * G8; it += p.S * kThreads) {
      const int m = it / G8, cc = (it % G8) * 8, n = tl * COLS + cc;
      if (n >= p.N) continue;
      float v[GATED ? 2 : 1][8];
#pragma unroll
      for (int q = 0; q < (GATED ? 2 : 1); ++q) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[q][i] = 0.0f;
        const uint32_t off = tile_a + uint32_t(m * ROWP + q * COLS + cc) * 4u;
        for (int k = 0; k < p.S; ++k) {
          const uint32_t ra = p.S > 1 ? ptx::mapa(off, uint32_t(k)) : off;
          const float4 a = ptx::ld_dsmem_f4(ra), b = ptx::ld_dsmem_f4(ra + 16u);
          v[q][0] += a.x; v[q][1] += a.y; v[q][2] += a.z; v[q][3] += a.w;
          v[q][4] += b.x; v[q][5] += b.y; v[q][6] += b.z; v[q][7] += b.w;
        }
      }
      const size_t o = size_t(m) * p.N + n;
      auto put = [&](__nv_bfloat16* dst, const float (&y)[8]) {
        *reinterpret_cast<uint4*>(dst + o) =
            make_uint4(ptx::cvt_bf16x2(y[0], y[1]), ptx::cvt_bf16x2(y[2], y[3]), ptx::cvt_bf16x2(y[4], y[5]),
                       ptx::cvt_bf16x2(y[6], y[7]));
      };
      uint32_t z[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        v[0][i] *= ts0;
        if constexpr (GATED) v[1][i] *= ts1;
        z[i] = __float_as_uint(v[0][i]);
      }
      if constexpr (!GATED) {
        if (p.bias) act::add8(z, __ldg(reinterpret_cast<const uint4*>(p.bias + n)));
#pragma unroll
        for (int i = 0; i < 8; ++i) v[0][i] = __uint_as_float(z[i]);
      }
      if (p.save0) put(p.save0, v[0]);
      if constexpr (GATED) {
        if (p.save1) put(p.save1, v[1]);
      }
      act::apply<8>(p.act, z);
      if constexpr (!GATED) {
        if (p.residual) act::add8(z, *reinterpret_cast<const uint4*>(p.residual + o));
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) v[0][i] = GATED ? __uint_as_float(z[i]) * v[GATED ? 1 : 0][i] : __uint_as_float(z[i]);
      put(p.out, v[0]);
    }
    if (p.S > 1) ptx::cluster_sync();        // the tile is reused only after every rank has read it
    else __syncthreads();
  }
}

// T = X A^T and Zs for nw adapters of rank r: the 16-row operand is 16 rows of the adapters stacked
// (row j < r: A0, else A1), the 8-wide one the batch rows.  8 warps split the depth of a CTA, S CTAs of
// a cluster that of a row group; the sums meet in shared memory in warp and rank order.
struct NarrowDownParams {
  const __nv_bfloat16 *a0, *a1, *x;   // [r, K] each (a1 null: one adapter); [M, K]
  const float *ts0, *ts1;             // tensor scales, or null
  __nv_bfloat16 *t, *zs;              // [nw][M, r]; [M, ldzs]
  int M, K, r, nw, ldzs, S;
  float s, zs_mul;
};

template <int NB>
__global__ void __launch_bounds__(narrow::kThreads)
qlora_narrow_down_kernel(const __grid_constant__ NarrowDownParams p) {
  using namespace narrow;
  __shared__ float part[kWarps][16][NB * 8 + 1];
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int rank = int(blockIdx.x) % p.S, grp = int(blockIdx.x) / p.S;
  const int rows = p.nw * p.r;
  const __nv_bfloat16* ar[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int j = min(grp * 16 + g + 8 * h, rows - 1);   // a clamped row's results are dropped
    ar[h] = j < p.r ? p.a0 + size_t(j) * p.K : p.a1 + size_t(j - p.r) * p.K;
  }
  float acc[NB][4];
#pragma unroll
  for (int b = 0; b < NB; ++b)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[b][i] = 0.0f;
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
  // pieces of 32 elements: lane t of a quad takes 8 of them; piece index strides over warps and ranks
  const int pieces = p.K / 32;
#pragma unroll 4
  for (int q = rank * kWarps + warp; q < pieces; q += p.S * kWarps) {
    const size_t k = size_t(q) * 32 + t * 8;
    const uint4 a = __ldg(reinterpret_cast<const uint4*>(ar[0] + k)), c = __ldg(reinterpret_cast<const uint4*>(ar[1] + k));
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const int m = 8 * b + g;
      const uint4 x = m < p.M ? __ldg(reinterpret_cast<const uint4*>(p.x + size_t(m) * p.K + k)) : zero;
      mma16816(acc[b], a.x, c.x, a.y, c.y, x.x, x.y);
      mma16816(acc[b], a.z, c.z, a.w, c.w, x.z, x.w);
    }
  }
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    part[warp][g][8 * b + 2 * t] = acc[b][0];
    part[warp][g][8 * b + 2 * t + 1] = acc[b][1];
    part[warp][g + 8][8 * b + 2 * t] = acc[b][2];
    part[warp][g + 8][8 * b + 2 * t + 1] = acc[b][3];
  }
  __syncthreads();
  // the warps' sums into part[0], in warp order
  for (int e = int(threadIdx.x); e < 16 * NB * 8; e += kThreads) {
    float v = part[0][e / (NB * 8)][e % (NB * 8)];
    for (int w = 1; w < kWarps; ++w) v += part[w][e / (NB * 8)][e % (NB * 8)];
    part[0][e / (NB * 8)][e % (NB * 8)] = v;
  }
  if (p.S > 1) ptx::cluster_sync();
  else __syncthreads();
  if (rank == 0) {
    for (int e = int(threadIdx.x); e < 16 * p.M; e += kThreads) {
      const int jj = e % 16, m = e / 16, j = grp * 16 + jj;
      if (j >= rows) continue;
      float v = 0.0f;
      const uint32_t at = ptx::smem_u32(&part[0][jj][m]);
      for (int k = 0; k < p.S; ++k) {
        float f;
        asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(f) : "r"(p.S > 1 ? ptx::mapa(at, uint32_t(k)) : at) : "memory");
        v += f;
      }
      const int i = j >= p.r ? 1 : 0;
      const float* ts = i ? p.ts1 : p.ts0;
      const float zs = p.s / (ts ? __ldg(ts) : 1.0f) * p.zs_mul;
      p.t[(size_t(i) * p.M + m) * p.r + (j - i * p.r)] = __float2bfloat16_rn(v);
      p.zs[size_t(m) * p.ldzs + j] = __float2bfloat16_rn(v * zs);
    }
  }
  if (p.S > 1) ptx::cluster_sync();          // every rank's sums stay until they are read
}

}  // namespace qlora
