// qlora_narrow.cuh -- forward of the gated MLP and of the linear layer with an epilogue for batches of
// at most 16 rows (single tokens, small decoding batches): each pass streams the 4-bit weights once.
//
//   qlora_narrow_down_kernel   T = X A^T of one or two adapters in one launch, and Zs = bf16(T s / ts)
//   qlora_narrow_kernel        G and U, or Z, and the whole epilogue in one kernel
//
// What bounds it: reading the weights (one token of a 14336 x 4096 NF4 gate and up: 66 MB, 10 us) and
// the SMs' decode.  A decoded pair of weights goes from the register it was decoded in straight into a
// warp-level m16n8k16 tensor-core product (weights the 16-row operand, batch rows the 8 columns), with
// no copy or hand-off between decode and product: the tcgen05 path has to place every decoded operand
// in shared or tensor memory and synchronise with the issuing thread.  The warp product's rate sets
// the limit of 16 rows: measured 8 clocks a sub-partition, so 8 rows allow 128 weights a clock and SM,
// but a decoded register serves only 8 rows per product.
//
// Decode: one code byte (two weights) indexes a 256-entry table in shared memory, replicated so that
// every lane reads its own banks.  MXFP4 / NVFP4: the pair of E2M1 values in bf16, times the block's
// scale in one packed multiply (exact).  NF4: the pair of levels in binary32, each times the absmax,
// rounded to bf16 (the definition).  NF4's entries are 8 bytes, which makes the shared-memory reads
// the limit (2 clocks a warp and pair), while the table-in-registers decode of qlora_dequant.cuh is
// limited by the byte permutes (2 clocks each a sub-partition, measured, and 2.6 a weight); kNfRegWords
// of every 8 words go the second way, which balances the two.
//
// The order of the contraction is free as long as both operands agree: lane t of a quad takes the
// 64-element block 4 j + t of its two weight rows (32 contiguous code bytes, one block scale), and
// two steps of a block multiply 8 consecutive elements, so the operand registers are the decoded pairs
// as they come, and the batch operand is a 16-byte piece of X for every two steps.
//
// Work split: a tile is 256 weight rows (gated: 128 of the gate and the same 128 of the up weight, one
// row group of 16 per warp), a unit of work one 256-deep chunk of a tile.  The flat space of units is
// cut into equal contiguous ranges, one per CTA and one CTA per SM.  A tile that one CTA covers is
// finished from its shared memory; the pieces of a split tile go to fp32 partials in the workspace
// and the CTA that counts in last adds them in piece order (deterministic) and finishes the tile.
// (Splitting over clusters instead, with the sums in distributed shared memory, left SMs idle: only
// 15 clusters of 8 or 33 of 4 fit beside each other on 148 SMs.)
//
// 20 warps, so that none waits for another's latency: 16 decode and multiply; one brings each unit's
// codes (one TMA box per weight: copies issued by the decoding warps stalled them whenever the memory
// pushed back) and its chunk of X through a ring of 4 units; 3 finish tiles (partials, arrival, epilogue) from one
// of two fp32 tile buffers while the others go on with the next tile.
#pragma once
#include <cuda_bf16.h>
#include "qlora_ptx.cuh"
#include "qlora_dequant.cuh"
#include "qlora_fused.cuh"
#include "qlora_act.cuh"

namespace qlora {
namespace narrow {
constexpr int kMaxRows = 16;
constexpr int kMaxDownRows = 64;           // of the down-projection
constexpr int kWarps = 16;                 // decoding warps
constexpr int kXWarps = 1;                 // brings X
constexpr int kEpiWarps = 3;               // finish tiles
constexpr int kThreads = (kWarps + kXWarps + kEpiWarps) * 32;
constexpr int CK = 256;                    // contraction elements of one chunk: 4 blocks of 64
constexpr int NS = 4;                      // units in shared memory
constexpr int C_BYTES = 256 * CK / 2;      // one unit's codes: 256 rows x 128 bytes, 128-byte swizzle
constexpr int kRows = kWarps * 16;         // 256 weight rows per tile
constexpr int ROWP = kRows + 4;            // pitch of the fp32 tile in shared memory (no conflicts)
constexpr int kDownWarps = 8;              // warps of a down-projection CTA
constexpr int kMaxCounters = 1984;         // arrival counters in the workspace header, one per tile
// fp32 partials: at most two pieces of split tiles per CTA, [8 nb rows][kRows] each
__host__ __device__ constexpr size_t partial_floats(int M) { return size_t(M) * kRows; }
__host__ __device__ constexpr size_t x_bytes(int nb) { return size_t(nb) * 8 * CK * 2; }
constexpr int kLoraDelay = 6;              // units (see lora_at)
constexpr int kTableBytes = 256 * 128;     // 256 entries x 32 lanes x 4 bytes, or x 16 lanes x 8
constexpr int kNfRegWords = 3;             // NF4: words of each 8 decoded from registers
__host__ __device__ constexpr size_t stage_bytes(int nb) { return C_BYTES + x_bytes(nb); }
// unit ring (1024-byte aligned), decode table, two fp32 tiles [8 nb][ROWP], barriers
__host__ __device__ constexpr size_t smem_bytes(int nb) {
  return 1024 + NS * stage_bytes(nb) + kTableBytes + size_t(2) * nb * 8 * ROWP * 4 + 256;
}

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Arrive on `bar` once this thread's asynchronous copies so far have landed (counted among the
// arrivals the barrier was initialised with).
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
// 16-byte asynchronous copy global -> shared; `bytes` 0 writes zeros instead.
__device__ __forceinline__ void cp_async_16(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
// Entries warp, warp + warps, ... of the decode table, every lane its own copy.
template <int FMT>
__device__ __forceinline__ void fill_table(uint32_t table, int warp, int warps, int lane) {
  if constexpr (FMT == kFmtNF4 || FMT == kFmtNF4DQ) {
    float mine = 0.0f;                        // the level of code lane % 16
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if ((lane & 15) == i) mine = nf4_level_dev(i);
    for (int e = warp; e < 256; e += warps) {
      const float lo = __shfl_sync(0xFFFFFFFFu, mine, e & 15), hi = __shfl_sync(0xFFFFFFFFu, mine, e >> 4);
      if (lane < 16)
        asm volatile("st.shared.v2.f32 [%0], {%1, %2};" ::"r"(table + uint32_t(e * 128 + lane * 8)), "f"(lo), "f"(hi) : "memory");
    }
  } else {
    for (int e = warp; e < 256; e += warps) {
      uint32_t o[4];
      e2m1_decode8(uint32_t(e), o);           // codes 0 and 1 of the word
      asm volatile("st.shared.b32 [%0], %1;" ::"r"(table + uint32_t(e * 128 + lane * 4)), "r"(o[0]) : "memory");
    }
  }
}
// Where this lane reads the decode table.  x128 is 128 in a form the compiler cannot see through (a
// kernel argument times 128): the address of byte b's entry then is a multiply-add, on a pipe that the
// decode leaves idle, and not a shift and add on the one that limits it.
struct Table {
  uint32_t base, x128;
  __device__ __forceinline__ uint32_t addr(uint32_t w, int b) const {
    return ptx::prmt(w, 0u, 0x4440u + uint32_t(b)) * x128 + base;
  }
};

// One 64-element block's decoder: its scales, then 8 codes (a word) at a time into pairs 2 i, 2 i + 1.
template <int FMT>
struct BlockDecoder {                         // NF4, NF4DQ
  Lut16 t;
  uint64_t absmax2;                           // the absmax twice
  __device__ __forceinline__ static uint32_t lane_base(uint32_t table, int lane) {
    return table + uint32_t(lane & 15) * 8u;
  }
  __device__ __forceinline__ void init(uint32_t raw) {
    absmax2 = (uint64_t(raw) << 32) | raw;
    t = nf4_lut(__uint_as_float(raw));
  }
  __device__ __forceinline__ void word(int j, uint32_t w, const Table& tab, uint32_t (&o)[4]) const {
    if (j >= kNfRegWords) {
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        uint64_t v;
        asm volatile("ld.shared.b64 %0, [%1];" : "=l"(v) : "r"(tab.addr(w, b)));
        asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(v) : "l"(v), "l"(absmax2));
        o[b] = ptx::cvt_bf16x2(__uint_as_float(uint32_t(v)), __uint_as_float(uint32_t(v >> 32)));
      }
    } else {
      // As lut16_lookup8, with the halves of the table chosen by a third permute whose selector is
      // the identity plus 4 where the code is above 7.
      const uint32_t sel3 = w & 0x77777777u;                        // low 3 bits of each code
      const uint32_t pick = ((w >> 1) & 0x44444444u) | 0x32103210u;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t s = h ? sel3 >> 16 : sel3, q = h ? pick >> 16 : pick;
        const uint32_t lo = ptx::prmt(ptx::prmt(t.lo[0], t.lo[1], s), ptx::prmt(t.lo[2], t.lo[3], s), q);
        const uint32_t hi = ptx::prmt(ptx::prmt(t.hi[0], t.hi[1], s), ptx::prmt(t.hi[2], t.hi[3], s), q);
        o[2 * h] = ptx::prmt(lo, hi, 0x5140u);
        o[2 * h + 1] = ptx::prmt(lo, hi, 0x7362u);
      }
    }
  }
};
// MXFP4 and NVFP4: table pair times the block's scale, exact (at most 2 x 4 significant bits).
template <int FMT>
struct E2m1Decoder {
  uint32_t s[4];                              // packed scale of words 2 q, 2 q + 1
  __device__ __forceinline__ static uint32_t lane_base(uint32_t table, int lane) { return table + uint32_t(lane) * 4u; }
  __device__ __forceinline__ void init(uint32_t raw) {
    if constexpr (FMT == kFmtMXFP4) {
      s[0] = s[1] = mx_exact_scale(raw);
      s[2] = s[3] = mx_exact_scale(raw >> 8);
    } else {
      // E4M3 to bf16, two at a time: exponent and mantissa placed in the low bits of the bf16 fields
      // are the value times 2^-120 (E4M3's subnormals are bf16's there); a NaN byte takes the slow way
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t x = ptx::prmt(raw, 0u, h ? 0x4342u : 0x4140u);
        const uint32_t v = ptx::mul_bf16x2(((x & 0x007F007Fu) << 4) | ((x & 0x00800080u) << 8), 0x7B807B80u);
        s[2 * h] = ptx::prmt(v, 0u, 0x1010u);
        s[2 * h + 1] = ptx::prmt(v, 0u, 0x3232u);
      }
      if ((((raw & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u) != 0u) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const uint32_t v = e4m3_bf16(raw >> (8 * q));
          s[q] = v | (v << 16);
        }
      }
    }
  }
  __device__ __forceinline__ void word(int j, uint32_t w, const Table& tab, uint32_t (&o)[4]) const {
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      uint32_t v;
      asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(tab.addr(w, b)));
      o[b] = ptx::mul_bf16x2(v, s[j >> 1]);
    }
  }
};
template <>
struct BlockDecoder<kFmtMXFP4> : E2m1Decoder<kFmtMXFP4> {};
template <>
struct BlockDecoder<kFmtNVFP4> : E2m1Decoder<kFmtNVFP4> {};
}  // namespace narrow

struct NarrowWeight {
  const void* scales;
  const float *scales2, *tensor_scale;
  const __nv_bfloat16* lora_up;      // B [N, r]
};

struct NarrowParams {
  CUtensorMap tm_codes[2];           // codes [N, K/2] u8 of each weight, box {128, 256} (gated: {128, 128}), SW128
  NarrowWeight w[2];                 // gated: gate, up; else w[0]
  const __nv_bfloat16 *x, *zs;       // [M, K]; [M, ldzs], weight i at column i r
  const __nv_bfloat16 *bias, *residual;
  __nv_bfloat16 *out, *save0, *save1;
  float* partial;                    // [gridDim.x][2][M][kRows]
  unsigned* counters;                // [tiles], zero between launches (split tiles only)
  int* status;
  int M, N, K, r, ldzs;
  int tiles, chunks, iters, act;     // iters: units per CTA
  uint32_t one;                      // 1 (see narrow::Table)
};

template <int FMT, bool GATED, int NB>
__global__ void __launch_bounds__(narrow::kThreads, 1)
qlora_narrow_kernel(const __grid_constant__ NarrowParams p) {
  using namespace narrow;
  using Dec = BlockDecoder<FMT>;
  constexpr int COLS = GATED ? kRows / 2 : kRows;      // output columns of a tile
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  constexpr uint32_t STAGE = uint32_t(stage_bytes(NB));   // codes, then X
  const uint32_t ring = ptx::smem_u32(smem);
  const uint32_t table = ring + NS * STAGE;
  constexpr int TILE = NB * 8 * ROWP;                  // floats of one tile buffer
  float* tiles = reinterpret_cast<float*>(smem + NS * STAGE + kTableBytes);
  uint64_t* bars = reinterpret_cast<uint64_t*>(tiles + 2 * TILE);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(bars + 2 * NS + 4);
  volatile unsigned* s_last = reinterpret_cast<volatile unsigned*>(abort_flag + 1);
  const uint32_t b0 = ptx::smem_u32(bars);
  auto full = [&](uint32_t s) { return b0 + 8u * s; };
  auto empty = [&](uint32_t s) { return b0 + 8u * (NS + s); };
  auto tile_full = [&](uint32_t b) { return b0 + 8u * (2 * NS + b); };
  auto tile_empty = [&](uint32_t b) { return b0 + 8u * (2 * NS + 2 + b); };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int total = p.tiles * p.chunks;
  const int u0 = int(blockIdx.x) * p.iters, u1 = min(u0 + p.iters, total);
  const int blocks = p.K / 64;
  if (threadIdx.x == 0) {
    for (int s = 0; s < NS; ++s) {
      ptx::mbar_init(full(s), 1 + 32);        // the codes' bytes; every lane's copies of X
      ptx::mbar_init(empty(s), kWarps);
    }
    for (int b = 0; b < 2; ++b) {
      ptx::mbar_init(tile_full(b), kWarps);
      ptx::mbar_init(tile_empty(b), kEpiWarps);
    }
    *abort_flag = 0;
    ptx::fence_mbarrier_init();
  }
  __syncthreads();
  ptx::griddep_launch_dependents();

  if (warp >= kWarps && warp < kWarps + kXWarps) {
    // ------------------------------------------------------------------ codes and X
    // piece (b, i, lane) = 8 elements of batch row 8 b + lane / 4 at block 4 c + lane % 4, element 8 i
    // -- the order in which the products read them; zeros past M and K
    uint32_t s = 0, ph = 0;
    int c = u0 % p.chunks, tl = u0 / p.chunks;
    for (int u = u0; u < u1; ++u) {
      if (!ptx::mbar_wait(empty(s), ph ^ 1u, p.status, abort_flag)) break;
      const uint32_t st = ring + s * STAGE;
      if (lane == 0) {
        ptx::mbar_arrive_expect_tx(full(s), uint32_t(C_BYTES));
        if (ptx::dcheck(ptx::tma_x_ok(c * (CK / 2), 1) && tl < p.tiles, p.status)) {
          ptx::tma_load_2d(st, &p.tm_codes[0], full(s), c * (CK / 2), tl * COLS);
          if constexpr (GATED) ptx::tma_load_2d(st + C_BYTES / 2, &p.tm_codes[1], full(s), c * (CK / 2), tl * COLS);
        }
      }
      __syncwarp();
      const uint32_t at = st + uint32_t(C_BYTES) + uint32_t(lane) * 16u;
      const int blk = 4 * c + t;
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const int row = 8 * b + g;
        const uint32_t bytes = row < p.M && blk < blocks ? 16u : 0u;
        const __nv_bfloat16* src = bytes ? p.x + size_t(row) * p.K + size_t(blk) * 64 : p.x;
#pragma unroll
        for (int i = 0; i < 8; ++i) cp_async_16(at + uint32_t(b * 8 + i) * 512u, src + (bytes ? i * 8 : 0), bytes);
      }
      cp_async_arrive(full(s));
      if (++s == uint32_t(NS)) { s = 0; ph ^= 1u; }
      if (++c == p.chunks) { c = 0; ++tl; }
    }
    ptx::cp_async_wait<0>();
    return;
  }

  if (warp >= kWarps + kXWarps) {
    // ------------------------------------------------------------------ tiles
    const int et = int(threadIdx.x) - (kWarps + kXWarps) * 32;
    // first, the adapter rows of the tiles whose LoRA term this CTA adds, into L2
    for (int tl = (u0 + p.chunks - 1) / p.chunks; tl * p.chunks < u1; ++tl) {
      const size_t row0 = size_t(tl) * COLS;
      const size_t bytes = size_t(min(COLS, p.N - int(row0))) * size_t(p.r) * 2;
      for (int i = 0; i < (GATED ? 2 : 1); ++i)
        for (size_t o = size_t(et) * 128; o < bytes; o += kEpiWarps * 32 * 128)
          asm volatile("prefetch.global.L2 [%0];" ::"l"(reinterpret_cast<const char*>(p.w[i].lora_up + row0 * p.r) + o));
    }
    ptx::griddep_wait();
    uint32_t nt = 0;
    for (int u = u0; u < u1; ++nt) {
      const int tl = u / p.chunks;
      u = min((tl + 1) * p.chunks, u1);
      ptx::mbar_wait(tile_full(nt & 1u), (nt >> 1) & 1u, p.status, abort_flag);
      const float* tile = tiles + (nt & 1u) * TILE;
      // the CTAs that share this tile
      const int first = (tl * p.chunks) / p.iters, last = (tl * p.chunks + p.chunks - 1) / p.iters;
      const size_t piece = partial_floats(p.M);
      bool finish = first == last && *abort_flag == 0;
      if (first != last) {
        float* mine = p.partial + (size_t(blockIdx.x) * 2 + (u0 / p.chunks == tl ? 0 : 1)) * piece;
        for (int e = et; e < p.M * (kRows / 4); e += kEpiWarps * 32) {
          const int m = e / (kRows / 4), q = e % (kRows / 4);
          __stcg(reinterpret_cast<float4*>(mine) + e, *reinterpret_cast<const float4*>(tile + size_t(m) * ROWP + 4 * q));
        }
        ptx::named_bar_sync(1, kEpiWarps * 32);
        if (et == 0) {
          __threadfence();                    // the piece (all threads' stores, ordered by the barrier)
          const unsigned n = atomicAdd(p.counters + tl, 1u);
          *s_last = n == unsigned(last - first) ? 1u : 0u;
          if (*s_last) p.counters[tl] = 0u;   // every piece has counted: back to zero for the next launch
          __threadfence();
        }
        ptx::named_bar_sync(1, kEpiWarps * 32);
        finish = *s_last != 0u && *abort_flag == 0;
      }
      if (finish) {
        // 8 columns at a time: the pieces in order, then the epilogue
        const float ts0 = p.w[0].tensor_scale ? __ldg(p.w[0].tensor_scale) : 1.0f;
        const float ts1 = GATED && p.w[1].tensor_scale ? __ldg(p.w[1].tensor_scale) : 1.0f;
        constexpr int G8 = COLS / 8;
        for (int it = et; it < p.M * G8; it += kEpiWarps * 32) {
          const int m = it / G8, cc = (it % G8) * 8, n = tl * COLS + cc;
          if (n >= p.N) continue;
          float v[GATED ? 2 : 1][8];
#pragma unroll
          for (int q = 0; q < (GATED ? 2 : 1); ++q) {
            const int col = q * COLS + cc;
            if (first == last) {
#pragma unroll
              for (int i = 0; i < 8; ++i) v[q][i] = tile[size_t(m) * ROWP + col + i];
            } else {
#pragma unroll
              for (int i = 0; i < 8; ++i) v[q][i] = 0.0f;
#pragma unroll 8
              for (int k = first; k <= last; ++k) {
                const float* src = p.partial + (size_t(k) * 2 + ((k * p.iters) / p.chunks == tl ? 0 : 1)) * piece +
                                   size_t(m) * kRows + col;
                const float4 a = __ldcg(reinterpret_cast<const float4*>(src)),
                             b = __ldcg(reinterpret_cast<const float4*>(src) + 1);
                v[q][0] += a.x; v[q][1] += a.y; v[q][2] += a.z; v[q][3] += a.w;
                v[q][4] += b.x; v[q][5] += b.y; v[q][6] += b.z; v[q][7] += b.w;
              }
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
          for (int i = 0; i < 8; ++i)
            v[0][i] = GATED ? __uint_as_float(z[i]) * v[GATED ? 1 : 0][i] : __uint_as_float(z[i]);
          put(p.out, v[0]);
        }
      }
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(tile_empty(nt & 1u));
    }
    return;
  }

  // ------------------------------------------------------------------ decode and multiply
  const Table lane_table{Dec::lane_base(table, lane), p.one * 128u};
  // this warp's weight and its first row in the tile's columns
  const int wi = GATED && warp >= kWarps / 2 ? 1 : 0;
  const void* scales = p.w[wi].scales;
  const float* scales2 = p.w[wi].scales2;
  const __nv_bfloat16* lora_up = p.w[wi].lora_up;
  const int wrow = (GATED ? warp % (kWarps / 2) : warp) * 16;
  // Row j of the warp's group in tile tl, clamped to the weight (a clamped row's results are dropped).
  auto row_of = [&](int tl, int j) { return min(tl * COLS + wrow + j, p.N - 1); };
  // Code bytes of this lane's blocks: 16-byte piece q of row j of a unit is at q ^ (j % 8).
  const uint32_t code_off = uint32_t(warp * 16 + g) * 128u;
  // Block scales: a cursor one unit ahead.
  int tl = u0 / p.chunks, c = u0 % p.chunks;
  int stl = tl, sc_c = c;
  const uint8_t* sptr[2];
  constexpr int SB = FMT == kFmtMXFP4 ? 2 : 4;          // scale bytes of a block (NF4DQ: see below)
  auto scale_tile = [&](int tl_, int c_) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
      sptr[h] = static_cast<const uint8_t*>(scales) + (size_t(row_of(tl_, g + 8 * h)) * blocks + 4 * c_ + t) * SB;
  };
  if constexpr (FMT != kFmtNF4DQ) scale_tile(stl, sc_c);
  auto next_scales = [&](uint32_t (&out)[2]) {
    const bool ok = 4 * sc_c + t < blocks;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      out[h] = 0u;
      if (ok) {
        if constexpr (FMT == kFmtNF4DQ)
          out[h] = load_item_scale_dq(scales, scales2, 0, p.N, row_of(stl, g + 8 * h), (4 * sc_c + t) * 64, p.K).raw;
        else if constexpr (FMT == kFmtMXFP4)
          out[h] = __ldg(reinterpret_cast<const uint16_t*>(sptr[h]));
        else
          out[h] = __ldg(reinterpret_cast<const uint32_t*>(sptr[h]));
      }
      if constexpr (FMT != kFmtNF4DQ) sptr[h] += 4 * SB;
    }
    if (++sc_c == p.chunks) {
      sc_c = 0;
      ++stl;
      if constexpr (FMT != kFmtNF4DQ) scale_tile(stl, 0);
    }
  };
  uint32_t sc[2], nsc[2] = {0u, 0u};
  next_scales(sc);
  fill_table<FMT>(table, warp, kWarps, lane);   // while the first codes are on their way
  float acc[NB][4];
#pragma unroll
  for (int b = 0; b < NB; ++b)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[b][i] = 0.0f;
  uint32_t st = 0, ph = 0, nt = 0;
  // The LoRA term of a tile belongs to the CTA with its chunk 0.  It needs Zs, which the kernel before
  // (launched just ahead of this one) writes, so it is added after the CTA's first few units, or with
  // its last unit of the tile: waiting earlier held CTAs back by 5 us.
  auto lora_unit = [&](int u) { return max(u, min(u0 + kLoraDelay, min(u + p.chunks, u1) - 1)); };
  int lora_at = c == 0 ? lora_unit(u0) : -1;
  ptx::named_bar_sync(2, kWarps * 32);          // the decode table is complete
  for (int u = u0; u < u1; ++u) {
    const bool tile_done = c + 1 == p.chunks;
    if (c == 0) lora_at = lora_unit(u);
    if (u == lora_at) {
      // rows of B times Zs: a lane takes the same r / 4 (r = 64: twice 8) rank elements of both, in the
      // widest pieces they come in, all on their way before the first product
      ptx::griddep_wait();
      uint4 la[2][2], lz[2][NB];
      const uint4 none = make_uint4(0u, 0u, 0u, 0u);
      auto piece = [&](const __nv_bfloat16* row, int k) {
        if (p.r >= 32) return k < p.r ? __ldcg(reinterpret_cast<const uint4*>(row + k + 8 * t)) : none;
        if (k > 0) return none;
        if (p.r == 16) {
          const uint2 v = __ldcg(reinterpret_cast<const uint2*>(row + 4 * t));
          return make_uint4(v.x, v.y, 0u, 0u);
        }
        return make_uint4(__ldcg(reinterpret_cast<const uint32_t*>(row + 2 * t)), 0u, 0u, 0u);
      };
#pragma unroll
      for (int k = 0; k < 2; ++k) {
#pragma unroll
        for (int h = 0; h < 2; ++h) la[k][h] = piece(lora_up + size_t(row_of(tl, g + 8 * h)) * p.r, 32 * k);
#pragma unroll
        for (int b = 0; b < NB; ++b)
          lz[k][b] = 8 * b + g < p.M ? piece(p.zs + size_t(8 * b + g) * p.ldzs + wi * p.r, 32 * k) : none;
      }
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          mma16816(acc[b], la[k][0].x, la[k][1].x, la[k][0].y, la[k][1].y, lz[k][b].x, lz[k][b].y);
          mma16816(acc[b], la[k][0].z, la[k][1].z, la[k][0].w, la[k][1].w, lz[k][b].z, lz[k][b].w);
        }
    }
    ptx::mbar_wait(full(st), ph, p.status, abort_flag);     // giving up is seen at the tile's end
    const uint32_t stage = ring + st * STAGE;
    uint32_t w[2][8];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const uint4 v = ptx::ld_shared_v4(stage + code_off + uint32_t(h) * 1024u + ((uint32_t(2 * t + q) ^ uint32_t(g)) << 4));
        w[h][4 * q] = v.x; w[h][4 * q + 1] = v.y; w[h][4 * q + 2] = v.z; w[h][4 * q + 3] = v.w;
      }
    Dec dec[2];
    dec[0].init(sc[0]);
    dec[1].init(sc[1]);
    if (u + 1 < u1) next_scales(nsc);
    const uint32_t xb = stage + uint32_t(C_BYTES) + uint32_t(lane) * 16u;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      uint32_t a[2][4];
      dec[0].word(i, w[0][i], lane_table, a[0]);
      dec[1].word(i, w[1][i], lane_table, a[1]);
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const uint4 x = ptx::ld_shared_v4(xb + uint32_t(b * 8 + i) * 512u);
        mma16816(acc[b], a[0][0], a[1][0], a[0][1], a[1][1], x.x, x.y);
        mma16816(acc[b], a[0][2], a[1][2], a[0][3], a[1][3], x.z, x.w);
      }
    }
    __syncwarp();
    // (every shared-memory read of the unit has returned: the products that took them have been issued)
    if (lane == 0) ptx::mbar_arrive(empty(st));
    if (++st == uint32_t(NS)) { st = 0; ph ^= 1u; }
    sc[0] = nsc[0];
    sc[1] = nsc[1];
    if (tile_done || u + 1 == u1) {
      // fp32 tile [batch row][weight row] (gated: 128 gate rows, then 128 up rows)
      ptx::mbar_wait(tile_empty(nt & 1u), ((nt >> 1) & 1u) ^ 1u, p.status, abort_flag);
      float* dst = tiles + (nt & 1u) * TILE + warp * 16 + g;
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        float* d = dst + size_t(8 * b + 2 * t) * ROWP;
        d[0] = acc[b][0];
        d[ROWP] = acc[b][1];
        d[8] = acc[b][2];
        d[ROWP + 8] = acc[b][3];
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[b][i] = 0.0f;
      }
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(tile_full(nt & 1u));
      ++nt;
    }
    if (tile_done) { ++tl; c = 0; }
    else ++c;
  }
}

// T = X A^T and Zs for nw adapters of rank r: the 16-row operand is 16 rows of the adapters stacked
// (row j < r: A0, else A1), the 8-wide one the batch rows (blockIdx.y: a block of 8 NB of them).  8
// warps split the depth of a CTA, S CTAs of a cluster that of a row group; the sums meet in shared memory in warp and rank order.
struct NarrowDownParams {
  const __nv_bfloat16 *a0, *a1, *x;   // [r, K] each (a1 null: one adapter); [M, K]
  const float *ts0, *ts1;             // tensor scales, or null
  __nv_bfloat16 *t, *zs;              // [nw][M, r]; [M, ldzs]
  int M, K, r, nw, ldzs, S;
  float s;
};

template <int NB>
__global__ void __launch_bounds__(narrow::kDownWarps * 32)
qlora_narrow_down_kernel(const __grid_constant__ NarrowDownParams p) {
  using namespace narrow;
  __shared__ float part[kDownWarps][16][NB * 8 + 1];
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int rank = int(blockIdx.x) % p.S, grp = int(blockIdx.x) / p.S;
  const int m0 = int(blockIdx.y) * NB * 8, mrows = min(NB * 8, p.M - m0);
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
  for (int q = rank * kDownWarps + warp; q < pieces; q += p.S * kDownWarps) {
    const size_t k = size_t(q) * 32 + t * 8;
    const uint4 a = __ldg(reinterpret_cast<const uint4*>(ar[0] + k)), c = __ldg(reinterpret_cast<const uint4*>(ar[1] + k));
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const int m = m0 + 8 * b + g;
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
  for (int e = int(threadIdx.x); e < 16 * NB * 8; e += kDownWarps * 32) {
    float v = part[0][e / (NB * 8)][e % (NB * 8)];
    for (int w = 1; w < kDownWarps; ++w) v += part[w][e / (NB * 8)][e % (NB * 8)];
    part[0][e / (NB * 8)][e % (NB * 8)] = v;
  }
  if (p.S > 1) ptx::cluster_sync();
  else __syncthreads();
  if (rank == 0) {
    for (int e = int(threadIdx.x); e < 16 * mrows; e += kDownWarps * 32) {
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
      const float zs = p.s / (ts ? __ldg(ts) : 1.0f);
      p.t[(size_t(i) * p.M + m0 + m) * p.r + (j - i * p.r)] = __float2bfloat16_rn(v);
      p.zs[size_t(m0 + m) * p.ldzs + j] = __float2bfloat16_rn(v * zs);
    }
  }
  if (p.S > 1) ptx::cluster_sync();          // every rank's sums stay until they are read
}

}  // namespace qlora
