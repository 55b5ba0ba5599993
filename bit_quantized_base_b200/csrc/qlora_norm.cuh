// qlora_norm.cuh -- RMS norm with the residual's addition, and its backward pass.
//
//   S = bf16(X + R)        rstd = (mean_k S^2 + eps)^(-1/2)        Y = bf16(S rstd gamma)
//   v = gamma dY           dS = dS_in + rstd (v - S rstd^2 mean_k(v S))
//   dgamma[k] = sum_m dY[m,k] S[m,k] rstd[m]
//
// Y leaves as bf16, as MXFP8 (E4M3 codes and one E8M0 scale per 32 along K: bit for bit what
// qlora_mxfp8_quantize makes of the bf16 Y) or as both.
//
// Both kernels are memory bound: each input element is read once and each output written once,
// with 5 to 20 operations in between.  A group of G threads (a power of two, 32..1024) holds one
// row in registers, V vectors of 8 elements a thread (vector j of thread t is vector j G + t of
// the row, so a warp's accesses are contiguous); the row's sum crosses the group by shuffles and
// one pass through shared memory.  4 adjacent lanes hold one 32-element MXFP8 block.
#pragma once
#include <cuda_bf16.h>
#include "qlora_ptx.cuh"
#include "qlora_w4a8.cuh"

namespace qlora {
namespace norm {
constexpr int kMaxV = 4;                     // 16-byte vectors of a row per thread
constexpr int kMaxK = 1024 * kMaxV * 8;      // widest row: 1024 threads
constexpr int kCta = 256;                    // threads per CTA for groups of up to 256
__host__ __device__ constexpr int cta_threads(int G) { return G > kCta ? G : kCta; }

// The two bf16 halves of a word as binary32.
__device__ __forceinline__ float lo_f32(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_f32(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
__device__ __forceinline__ uint4 ld_v4(const __nv_bfloat16* p) {
  return __ldcs(reinterpret_cast<const uint4*>(p));
}
__device__ __forceinline__ void st_v4(__nv_bfloat16* p, const uint4& v) {
  *reinterpret_cast<uint4*>(p) = v;
}

// Sum of `v` over the group's G threads, the same in each of them.  Groups of more than a warp
// pass through `red` (one slot per warp of the CTA); every thread of the CTA calls.
template <typename T>
__device__ __forceinline__ T group_sum(T v, int G, T* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  if (G > 32) {
    const int warp = threadIdx.x >> 5, wpg = G >> 5, w0 = warp & ~(wpg - 1);
    __syncthreads();                          // the slots' readers of the row before are done
    if ((threadIdx.x & 31) == 0) red[warp] = v;
    __syncthreads();
    v = T(0);
    for (int w = 0; w < wpg; ++w) v += red[w0 + w];
  }
  return v;
}

// (mean + eps)^(-1/2) as hi + lo: the binary32 estimate and one Newton step in binary64.  An
// infinite or NaN mean keeps the estimate (0 or NaN).
__device__ __forceinline__ void rstd_pair(double ms, float& hi, float& lo) {
  const float r0 = rsqrtf(float(ms));
  hi = r0;
  lo = 0.0f;
  if (r0 > 0.0f && r0 < INFINITY) {
    const double r = double(r0) * (1.5 - 0.5 * ms * double(r0) * double(r0));
    hi = float(r);
    lo = float(r - double(hi));
  }
}

// Whether a product's binary32 estimate (at most 3 units of its last place off: two roundings and
// rstd's) lies so near the border of two bf16 values that they could decide: its low 16 bits within 8
// of the middle.  Returned as a value to take the minimum of: at most kNearBorder if so.
constexpr uint32_t kNearBorder = 16u << 16;
__device__ __forceinline__ uint32_t border(float y) { return (__float_as_uint(y) << 16) + (0x8008u << 16); }

// bf16(s rstd gamma) as if computed exactly, up to about 2^-44 of the value: the two products'
// rounding errors are carried (fused multiply-adds return them exactly), and a binary32 sum that
// lands on the border between two bf16 values goes to the side its error points to.  An 8-bit
// code that depends on a bf16 border is then that of the definition, not of the order of rounding.
__device__ __forceinline__ uint32_t product_bf16(float s, float hi, float lo, float g) {
  const float p = __fmul_rn(s, hi);           // _rn: not to be contracted into the additions
  const float pe = fmaf(s, lo, fmaf(s, hi, -p));
  const float q = __fmul_rn(p, g);
  const float qe = fmaf(pe, g, fmaf(p, g, -q));
  const float y = __fadd_rn(q, qe);
  const float ye = __fadd_rn(qe, -__fadd_rn(y, -q));
  uint32_t b = __float_as_uint(y);
  if ((b & 0xFFFFu) == 0x8000u && ye != 0.0f) b += ((ye > 0.0f) == (y > 0.0f)) ? 1u : 0xFFFFFFFFu;
  return __bfloat16_as_ushort(__float2bfloat16_rn(__uint_as_float(b)));
}
}  // namespace norm

struct NormFwdParams {
  const __nv_bfloat16 *x, *res, *gamma;   // res, gamma: may be null
  __nv_bfloat16 *s, *y;                   // may be null
  uint8_t *codes, *scales;                // may be null
  float* rstd;                            // may be null
  long long M;
  int K, G;
  float eps;
};

// V: vectors a thread holds; MX: the MXFP8 output is wanted (Y then goes through product_bf16); T:
// threads per CTA.  Registers for at least 1024 threads per SM: 4096 x 8192 to MXFP8 took 56 us with
// the 67 a thread that the compiler took by itself, 47 with 64 (one CTA more per SM).
template <int V, bool MX, int T>
__global__ void __launch_bounds__(T, 1024 / T) qlora_norm_fwd_kernel(const __grid_constant__ NormFwdParams p) {
  using namespace norm;
  __shared__ double red[32];
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  const int groups = int(blockDim.x) / p.G;
  const int t = int(threadIdx.x) & (p.G - 1);
  const int nv = p.K / 8;
  const long long row = (long long)blockIdx.x * groups + int(threadIdx.x) / p.G;
  const bool live = row < p.M;
  const size_t base = size_t(live ? row : 0) * size_t(p.K);
  uint4 s[V];
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int v = j * p.G + t;
    s[j] = make_uint4(0u, 0u, 0u, 0u);
    if (live && v < nv) s[j] = ld_v4(p.x + base + size_t(v) * 8);
  }
  if (p.res) {
    uint4 r[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int v = j * p.G + t;
      r[j] = make_uint4(0u, 0u, 0u, 0u);
      if (live && v < nv) r[j] = ld_v4(p.res + base + size_t(v) * 8);
    }
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const uint32_t a[4] = {s[j].x, s[j].y, s[j].z, s[j].w}, b[4] = {r[j].x, r[j].y, r[j].z, r[j].w};
      uint32_t o[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        o[i] = ptx::cvt_bf16x2(lo_f32(a[i]) + lo_f32(b[i]), hi_f32(a[i]) + hi_f32(b[i]));
      s[j] = make_uint4(o[0], o[1], o[2], o[3]);
      const int v = j * p.G + t;
      if (p.s && live && v < nv) st_v4(p.s + base + size_t(v) * 8, s[j]);
    }
  }
  // at most 32 squares (exact in binary32) per thread in two binary32 sums (MX: with the rounding
  // error of every addition, which a two-sum returns exactly, summed beside), then binary64
  float2 sq = make_float2(0.0f, 0.0f), comp = sq;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const uint32_t a[4] = {s[j].x, s[j].y, s[j].z, s[j].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = make_float2(lo_f32(a[i]), hi_f32(a[i]));
      if constexpr (MX) {
        const float2 q = ptx::mul2(f, f), n = ptx::add2(sq, q), b = ptx::sub2(n, sq);
        comp = ptx::add2(comp, ptx::add2(ptx::sub2(sq, ptx::sub2(n, b)), ptx::sub2(q, b)));
        sq = n;
      } else {
        sq.x = fmaf(f.x, f.x, sq.x);
        sq.y = fmaf(f.y, f.y, sq.y);
      }
    }
  }
  const double sum = group_sum((double(sq.x) + double(sq.y)) + (double(comp.x) + double(comp.y)), p.G, red);
  float hi, lo;
  rstd_pair(sum / double(p.K) + double(p.eps), hi, lo);
  if (p.rstd && live && t == 0) p.rstd[row] = hi;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int v = j * p.G + t;
    const bool ok = live && v < nv;
    const uint32_t a[4] = {s[j].x, s[j].y, s[j].z, s[j].w};
    uint4 gv = make_uint4(0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u);
    if (p.gamma && ok) gv = __ldg(reinterpret_cast<const uint4*>(p.gamma) + v);
    const uint32_t g[4] = {gv.x, gv.y, gv.z, gv.w};
    uint32_t o[4], near = 0xFFFFFFFFu;
    [[maybe_unused]] uint2 e[4];               // MX: how near a border each product is
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 y = ptx::mul2(ptx::mul2(make_float2(lo_f32(a[i]), hi_f32(a[i])), make_float2(hi, hi)),
                                 make_float2(lo_f32(g[i]), hi_f32(g[i])));
      o[i] = ptx::cvt_bf16x2(y.x, y.y);
      if constexpr (MX) {
        e[i] = make_uint2(border(y.x), border(y.y));
        near = min(near, min(e[i].x, e[i].y));
      }
    }
    if constexpr (MX) {
      if (near <= kNearBorder) {               // about one element in 4000
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (e[i].x <= kNearBorder)
            o[i] = (o[i] & 0xFFFF0000u) | product_bf16(lo_f32(a[i]), hi, lo, lo_f32(g[i]));
          if (e[i].y <= kNearBorder)
            o[i] = (o[i] & 0xFFFFu) | (product_bf16(hi_f32(a[i]), hi, lo, hi_f32(g[i])) << 16);
        }
      }
    }
    if (p.y && ok) st_v4(p.y + base + size_t(v) * 8, make_uint4(o[0], o[1], o[2], o[3]));
    if constexpr (MX) {
      uint32_t amax = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) amax = __vmaxu2(amax, o[i] & 0x7FFF7FFFu);
      amax = max(amax & 0xFFFFu, amax >> 16);
      amax = max(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
      amax = max(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 2));
      const int ex = mxfp8_exponent(amax);
      const float inv = mxfp8_inverse(ex);
      if (ok) {
        const uint2 c = make_uint2(mxfp8_encode4(o[0], o[1], inv), mxfp8_encode4(o[2], o[3], inv));
        *reinterpret_cast<uint2*>(p.codes + base + size_t(v) * 8) = c;
        if ((v & 3) == 0) p.scales[(base + size_t(v) * 8) / 32] = uint8_t(ex);
      }
    }
  }
}

struct NormBwdParams {
  const __nv_bfloat16 *s, *gamma, *dy, *ds_in;   // gamma, ds_in: may be null
  const float* rstd;                              // may be null: recomputed from S and eps
  __nv_bfloat16* ds;
  float* part;                                    // dgamma partials [gridDim.x][K] (DG)
  long long M;
  int K, G;
  float eps;
};

// CTAs per SM and, per CTA, the rows a group keeps in flight or in shared memory.
namespace norm {
__host__ __device__ constexpr int bwd_per_sm(int T) { return T > 512 ? 1 : (T > 256 ? 2 : 3); }
__host__ __device__ constexpr size_t bwd_stage_bytes(int V, int T) { return size_t(3) * V * T * 16; }
__host__ __device__ constexpr int bwd_stages(int V, int T) {
  const int n = int(size_t(225) * 1024 / bwd_per_sm(T) / bwd_stage_bytes(V, T));
  return n < 1 ? 1 : (n > 4 ? 4 : n);
}
}  // namespace norm

// Persistent over rows: group g of the grid takes rows g, g + groups, ...  Every thread copies the
// vectors of S, dY and dS_in that it will work on into its own slots of a ring in shared memory,
// up to four rows ahead (asynchronously, so no registers hold them and no barrier guards them: the
// slots are the thread's own).  With DG each thread keeps its columns' dgamma sums in registers over
// all its rows; the CTA's groups add theirs in group order through shared memory and write one
// partial row, which qlora_norm_dgamma_kernel sums.
template <int V, bool DG, int T>
__global__ void __launch_bounds__(T, norm::bwd_per_sm(T)) qlora_norm_bwd_kernel(const __grid_constant__ NormBwdParams p) {
  using namespace norm;
  constexpr int S = bwd_stages(V, T);
  __shared__ float red[32], red2[32];
  extern __shared__ __align__(16) uint8_t ring[];   // [S][S, dY, dS_in][V][T] vectors
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  const int groups = T / p.G;
  const int grp = int(threadIdx.x) / p.G;
  const int t = int(threadIdx.x) & (p.G - 1);
  const int nv = p.K / 8;
  const float inv_k = 1.0f / float(p.K);
  const uint4 one4 = make_uint4(0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u);
  // gamma stays in registers, but for 3 and 4 vectors a thread, which have none left
  auto load_gamma = [&](int j) {
    const int v = j * p.G + t;
    return p.gamma && v < nv ? __ldg(reinterpret_cast<const uint4*>(p.gamma) + v) : one4;
  };
  uint4 gam[V];
#pragma unroll
  for (int j = 0; j < V; ++j) gam[j] = V <= 2 ? load_gamma(j) : one4;
  float acc[DG ? V * 8 : 1];
#pragma unroll
  for (int i = 0; i < (DG ? V * 8 : 1); ++i) acc[i] = 0.0f;
  const uint4* slots = reinterpret_cast<const uint4*>(ring) + threadIdx.x;
  const uint32_t slot0 = ptx::smem_u32(slots);
  const long long step = (long long)gridDim.x * groups;
  // one row's vectors into stage sg; past the last row or the row's end: zeros
  auto fetch = [&](long long row, int sg) {
    const bool live = row < p.M;
    const size_t base = size_t(live ? row : 0) * size_t(p.K);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int v = j * p.G + t;
      const uint32_t bytes = live && v < nv ? 16u : 0u;
      const size_t at = base + size_t(v < nv ? v : 0) * 8;
      const uint32_t dst = slot0 + uint32_t((sg * 3 * V + j) * T) * 16u;
      ptx::cp_async_16(dst, p.s + at, bytes);
      ptx::cp_async_16(dst + uint32_t(V * T) * 16u, p.dy + at, bytes);
      if (p.ds_in) ptx::cp_async_16(dst + uint32_t(2 * V * T) * 16u, p.ds_in + at, bytes);
    }
  };
  long long row = (long long)blockIdx.x * groups + grp;
  // the CTA's groups run the same number of rows (the last may be past the end)
  const long long first = (long long)blockIdx.x * groups;
  const int count = first < p.M ? int((p.M - first + step - 1) / step) : 0;
#pragma unroll
  for (int i = 0; i < S - 1; ++i) {
    fetch(row + i * step, i);
    ptx::cp_async_commit();
  }
  int sg = 0, pf = S - 1;
  for (int it = 0; it < count; ++it, row += step) {
    fetch(row + (S - 1) * step, pf);
    ptx::cp_async_commit();
    ptx::cp_async_wait<S - 1>();
    const bool live = row < p.M;
    const size_t base = size_t(live ? row : 0) * size_t(p.K);
    const uint4* my = slots + sg * 3 * V * T;
    pf = sg;
    sg = sg + 1 == S ? 0 : sg + 1;
    float dot = 0.0f, sq = 0.0f;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const uint4 sv = my[j * T], dv = my[(V + j) * T];
      const uint32_t a[4] = {sv.x, sv.y, sv.z, sv.w}, b[4] = {dv.x, dv.y, dv.z, dv.w};
      const uint4 gv = V <= 2 ? gam[j] : load_gamma(j);
      const uint32_t g[4] = {gv.x, gv.y, gv.z, gv.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        dot = fmaf(lo_f32(b[i]) * lo_f32(g[i]), lo_f32(a[i]), dot);
        dot = fmaf(hi_f32(b[i]) * hi_f32(g[i]), hi_f32(a[i]), dot);
        if (!p.rstd) {
          sq = fmaf(lo_f32(a[i]), lo_f32(a[i]), sq);
          sq = fmaf(hi_f32(a[i]), hi_f32(a[i]), sq);
        }
      }
    }
    dot = group_sum(dot, p.G, red);
    float rstd;
    if (p.rstd) {
      rstd = live ? __ldg(p.rstd + row) : 0.0f;
    } else {
      float lo;
      rstd_pair(double(group_sum(sq, p.G, red2)) * double(inv_k) + double(p.eps), rstd, lo);
      if (!live) rstd = 0.0f;                  // no row: with eps = 0 it would be infinite, and 0 rstd NaN
    }
    const float c = dot * inv_k * rstd * rstd;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int v = j * p.G + t;
      const uint4 sv = my[j * T], dv = my[(V + j) * T];
      const uint32_t a[4] = {sv.x, sv.y, sv.z, sv.w}, b[4] = {dv.x, dv.y, dv.z, dv.w};
      const uint4 gv = V <= 2 ? gam[j] : load_gamma(j);
      const uint32_t g[4] = {gv.x, gv.y, gv.z, gv.w};
      uint4 iv = make_uint4(0u, 0u, 0u, 0u);
      if (p.ds_in) iv = my[(2 * V + j) * T];
      const uint32_t in[4] = {iv.x, iv.y, iv.z, iv.w};
      uint32_t o[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float s0 = lo_f32(a[i]), s1 = hi_f32(a[i]), d0 = lo_f32(b[i]), d1 = hi_f32(b[i]);
        const float v0 = rstd * (d0 * lo_f32(g[i]) - s0 * c) + lo_f32(in[i]);
        const float v1 = rstd * (d1 * hi_f32(g[i]) - s1 * c) + hi_f32(in[i]);
        o[i] = ptx::cvt_bf16x2(v0, v1);
        if constexpr (DG) {
          acc[j * 8 + 2 * i] = fmaf(d0, s0 * rstd, acc[j * 8 + 2 * i]);
          acc[j * 8 + 2 * i + 1] = fmaf(d1, s1 * rstd, acc[j * 8 + 2 * i + 1]);
        }
      }
      if (live && v < nv) st_v4(p.ds + base + size_t(v) * 8, make_uint4(o[0], o[1], o[2], o[3]));
    }
  }
  if constexpr (DG) {
    float* gsum = reinterpret_cast<float*>(ring);   // [groups - 1][K]
    if (groups > 1) {
      ptx::cp_async_wait<0>();
      __syncthreads();                         // the ring is every thread's from here
      if (grp > 0) {
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const int v = j * p.G + t;
          if (v < nv)
#pragma unroll
            for (int i = 0; i < 8; ++i) gsum[size_t(grp - 1) * p.K + v * 8 + i] = acc[j * 8 + i];
        }
      }
      __syncthreads();
    }
    if (grp == 0) {
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int v = j * p.G + t;
        if (v >= nv) continue;
        for (int q = 1; q < groups; ++q)
#pragma unroll
          for (int i = 0; i < 8; ++i) acc[j * 8 + i] += gsum[size_t(q - 1) * p.K + v * 8 + i];
        float4* dst = reinterpret_cast<float4*>(p.part + size_t(blockIdx.x) * p.K + size_t(v) * 8);
        dst[0] = make_float4(acc[j * 8], acc[j * 8 + 1], acc[j * 8 + 2], acc[j * 8 + 3]);
        dst[1] = make_float4(acc[j * 8 + 4], acc[j * 8 + 5], acc[j * 8 + 6], acc[j * 8 + 7]);
      }
    }
  }
}

struct NormDgammaParams {
  const float* part;        // [P][K]
  __nv_bfloat16* dgamma;    // [K]
  int P, K;
};

// dgamma[k] = the sum of the P partial rows: 32 columns per CTA, 16 slices of the rows, each summed
// in row order and then in slice order (a fixed order: the same result every run).
__global__ void __launch_bounds__(512) qlora_norm_dgamma_kernel(const __grid_constant__ NormDgammaParams p) {
  __shared__ float sm[16][33];
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  const int c = int(threadIdx.x) & 31, sl = int(threadIdx.x) >> 5;
  const int k = int(blockIdx.x) * 32 + c;
  const int per = (p.P + 15) / 16;
  float a = 0.0f;
  if (k < p.K) {
    const int r1 = min(p.P, (sl + 1) * per);
#pragma unroll 4
    for (int r = sl * per; r < r1; ++r) a += __ldcg(p.part + size_t(r) * p.K + k);
  }
  sm[sl][c] = a;
  __syncthreads();
  if (sl == 0 && k < p.K) {
    for (int q = 1; q < 16; ++q) a += sm[q][c];
    p.dgamma[k] = __float2bfloat16_rn(a);
  }
}

}  // namespace qlora
