// gemm_epilogue.cu -- C = act(A W^T + bias) + residual on the 5th-generation
// tensor cores, for bf16 operands and for e4m3 operands with a scale per row
// of A and of W.
//
// Batch invariance: as in the plain GEMM every shape runs one instruction
// family (tcgen05.mma kind::f16 with K = 16 or kind::f8f6f4 with K = 32) and
// accumulates the k-blocks of 128 bytes in increasing k into one fp32
// accumulator.  What an element's sum is does not depend on how many rows (64,
// 128, or 128 and 256 over two SMs) and columns (16 .. 256) the instruction takes: every
// shape that a batch size leads to gives a row the same bytes (tests compare
// them, and those of the plain GEMM), and the epilogue is element-wise.  So a
// row of C depends only on its rows of A and of the residual, W and the bias,
// and the tile may be chosen from the shape (fused_plan).
//
// Epilogue, every step one fp32 operation rounded once (activations aside):
//   z = acc (bf16), (acc * a_scale) * w_scale (e4m3);  z += bias;  z = act(z);
//   z += residual;  C = bf16(z).
//
// Structure: persistent blocks, one per SM, 10 warps: a TMA producer, one thread
// that issues the MMAs into one of two accumulators in tensor memory, eight
// epilogue warps of 32 accumulator rows and half the tile's columns each.  Four
// forms: up to 64 rows of A (MMAs of 64 rows, narrow tiles, plain stores; a
// weight is streamed), one CTA with 128 rows, and pairs of CTAs with 256 or 128 rows,
// whose one MMA reads half of W's rows from each SM.  Tile width, k-blocks per
// stage and stages are run-time values.  Every wait is bounded; a wait that runs
// out records BI_ERR_TIMEOUT, tells the other roles to stop, waits (bounded) for
// its copies and MMAs in flight, frees tensor memory and returns.
//
// What bounds it (one GB300, a few calls in a loop; rates are of the measured 1957
// TFLOP/s bf16, twice that for e4m3, and 6777 GB/s): with many rows the tensor
// cores and the power they draw (8192 x 28672 x 4096 e4m3 with SwiGLU 493 us =
// 3.9 PFLOP/s, 1.00; bf16 2048 x 4096 x 14336 with the residual 131 us, 0.94; in a
// run of seconds, which draws the power limit, 572 to 594 us, 0.83 to 0.86, and 154 to
// 160, 0.77 to 0.80); with few the weight's bytes (64 x 28672 x 4096 e4m3 21.5 us,
// 0.82) and for short ones start and end, some 3 us, and some 50 cycles an MMA,
// whatever its width (16 x 6144 x 4096 e4m3 5.9 us with the weight in L2, 8.0 from
// memory, 0.47).  Those 50 cycles are the same with two accumulators taking turns,
// so they are not one accumulator's chain, but the issuing thread's instructions or
// the MMA's own least time.  Short K: C's way out through the epilogue (8192 x 14336 x
// 256 e4m3 89 us, 2.6 TB/s; x 1024 99, with GELU 152, with a residual too 193).
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>

#include "bi_internal.h"
#include "device_common.cuh"
#include "f32x2.cuh"
#include "tcgen05.cuh"

namespace bi {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int BM = 128;                      // rows of a CTA's tile
constexpr int kEpiWarps = 8;                 // two per quarter of the accumulator's lanes
constexpr int kThreads = 64 + 32 * kEpiWarps;
constexpr int kBlockBytes = 128;             // bytes of a row in one k-block
constexpr int kMaxStages = 24;
constexpr int kChunk = 32;                   // columns of C that a warp stores at once
constexpr int kChunkBytes = 32 * kChunk * 2; // of 32 rows of them
constexpr int kBufs = 2;                     // buffers of that size a warp has
constexpr int kPadBytes = 1024;              // to the ring's alignment
constexpr int kColumnBytes = 2 * 256 * (4 + 2);  // a tile's w_scale and bias, twice
// the operand ring and the epilogue's buffers share the rest (less than 1 KB
// of barriers is static)
constexpr int kPoolBytes = 227 * 1024 - 1024 - kPadBytes - kColumnBytes;
static_assert(kPoolBytes % 1024 == 0, "the buffers behind the ring are aligned as it is");
constexpr size_t kSmemBytes = kPadBytes + kPoolBytes + kColumnBytes;
constexpr uint32_t kAccCols = 256;           // columns between the two accumulators
constexpr int kLongBlocks = 32;              // k-blocks from which a tile's MMAs outlast its epilogue
constexpr int kSwigluBlock = 16;             // gate (then up) rows of a block of W
constexpr int kDirectRows = 64;              // at most this many rows of A: MMAs of 64, plain stores

// Division of 0 <= n < 2^31 by d >= 1 as a product: with s = ceil(log2 d) and
// m = ceil(2^(31 + s) / d), n / d is the high word of n m, s - 1 places down
// (a divide takes some 150 cycles, and a tile's place three of them).
struct Divisor {
  int d;
  uint32_t m, shift;
  Divisor() = default;
  explicit Divisor(int64_t by) : d(static_cast<int>(by)), m(0), shift(0) {
    int s = 0;
    while ((int64_t(1) << s) < by) ++s;
    if (s == 0) return;  // by 1: n itself
    m = static_cast<uint32_t>(((uint64_t(1) << (31 + s)) + by - 1) / by);
    shift = s - 1;
  }
  __device__ __forceinline__ int of(int n) const {
    return d == 1 ? n : static_cast<int>(__umulhi(static_cast<uint32_t>(n), m) >> shift);
  }
};

struct FusedParams {
  __nv_bfloat16* C;
  const __nv_bfloat16* bias;      // [N] or null
  const __nv_bfloat16* residual;  // C's shape or null (may be C)
  const float* a_scale;           // [M] (e4m3)
  const float* w_scale;           // [N] (e4m3)
  int* err;
  int M, N, n_out;                // n_out: columns of C
  int act;
  int bn, a_rows, kg, stages;     // tile width, rows of A and k-blocks per stage
  int deep;                       // a stage's k-blocks come by one copy
  int mma_rows;                   // rows of an MMA in this CTA
  int ring, staged;               // the ring's bytes; whether C goes through shared memory
  int m_tiles, n_tiles, kb_total; // m_tiles: of the pair's 256 rows where kCtas is 2
  int m_fast;                     // raster, as in the plain GEMM: 1: M's tiles in groups
  Divisor by_per, by_group, by_last;  // tiles of a group times the others, a group, the last
  uint32_t idesc;
};

__device__ __forceinline__ void prefetch_l2(const void* p) {
  asm volatile("prefetch.global.L2 [%0];" ::"l"(p));
}

struct Tile {
  int m, n;
};
// Tile order (it only decides which block runs a tile and when): the smaller
// operand is kept resident in L2 in groups of `group` tiles while the other
// one streams past it once per group.
__device__ __forceinline__ Tile tile_of(int u, const FusedParams& p) {
  const int span = p.m_fast ? p.m_tiles : p.n_tiles;
  const int g = p.by_per.of(u), r = u - g * p.by_per.d;
  const int first = g * p.by_group.d;
  const bool whole = span - first >= p.by_group.d;  // the last group may be smaller
  const int slow = whole ? p.by_group.of(r) : p.by_last.of(r);
  const int fast = first + r - slow * (whole ? p.by_group.d : p.by_last.d);
  return p.m_fast ? Tile{fast, slow} : Tile{slow, fast};
}

// The activations take the special-function unit's exponential and reciprocal
// (2^-22 relative, results below 2^-126 flushed to zero) instead of expf and a
// division, whose path for special cases kept a warp from interleaving its 32
// values (100 cycles a value: 330 us at 8192 x 14336 x 1024 e4m3 with SiLU, where
// this takes 20), and the result is rounded to 2^-9.  Everything else goes two
// values at a time (f32x2).
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ f32x2 ex2_2(f32x2 x) {
  const float2 f = halves(x);
  return pair(ex2(f.x), ex2(f.y));
}
__device__ __forceinline__ f32x2 rcp_2(f32x2 x) {
  const float2 f = halves(x);
  return pair(rcp(f.x), rcp(f.y));
}
constexpr float kLog2e = 1.4426950408889634f;

// z / (1 + 2^e)
__device__ __forceinline__ f32x2 z_sigmoid(f32x2 z, f32x2 e) {
  return mul2(z, rcp_2(add2(ex2_2(e), both(1.0f))));
}
__device__ __forceinline__ f32x2 silu(f32x2 z) { return z_sigmoid(z, mul2(z, both(-kLog2e))); }
// z/2 (1 + tanh u) = z / (1 + exp(-2 u)), u = sqrt(2/pi) (z + 0.044715 z^3)
__device__ __forceinline__ f32x2 gelu_tanh(f32x2 z) {
  const f32x2 c = mul2(mul2(z, z), both(0.044715f));
  return z_sigmoid(z, mul2(fma2(z, c, z), both(-1.5957691216057308f * kLog2e)));
}
// max(z, 0), a NaN where z is one
__device__ __forceinline__ f32x2 relu(f32x2 z) {
  float2 f = halves(z);
  asm("max.NaN.f32 %0, %0, 0f00000000;" : "+f"(f.x));
  asm("max.NaN.f32 %0, %0, 0f00000000;" : "+f"(f.y));
  return pair(f.x, f.y);
}
// z/2 (1 + erf(z / sqrt 2)) = max(z, 0) - |z|/2 erfcx(x) exp(-x^2), x = |z| / sqrt 2,
// with -erfcx(x)/2 as t times a polynomial in t = 1 / (1 + x/2): the least
// largest relative error of degree 6 over 0 <= x <= 11.4, by linear
// programming; 2^-18.8 in fp32.  Both tails keep their digits.  Past |z| = 16
// the second term is 0.  One reciprocal, of the product of both denominators
// (1 .. 6.7), serves the two values.
__device__ __forceinline__ f32x2 gelu(f32x2 z) {
  const float2 f = halves(z);
  const f32x2 m = pair(fminf(fabsf(f.x), 16.0f), fminf(fabsf(f.y), 16.0f));
  const float2 d = halves(fma2(m, both(0.35355339059327376f), both(1.0f)));
  const f32x2 t = mul2(both(rcp(d.x * d.y)), pair(d.y, d.x));
  f32x2 s = both(-0.0429137014f);
  s = fma2(s, t, both(0.174213769f));
  s = fma2(s, t, both(-0.188846613f));
  s = fma2(s, t, both(-0.0229806649f));
  s = fma2(s, t, both(-0.139260697f));
  s = fma2(s, t, both(-0.139064864f));
  s = fma2(s, t, both(-0.141146311f));
  const f32x2 e = ex2_2(mul2(mul2(m, m), both(-0.5f * kLog2e)));
  return fma2(mul2(s, mul2(t, m)), e, relu(z));
}

// In 32 values, one activation; the choice is the same for the whole call.
__device__ __forceinline__ void activate(f32x2 (&z)[16], int act) {
  switch (act) {
    case BI_ACT_RELU:
#pragma unroll
      for (int i = 0; i < 16; ++i) z[i] = relu(z[i]);
      break;
    case BI_ACT_GELU:
#pragma unroll
      for (int i = 0; i < 16; ++i) z[i] = gelu(z[i]);
      break;
    case BI_ACT_GELU_TANH:
#pragma unroll
      for (int i = 0; i < 16; ++i) z[i] = gelu_tanh(z[i]);
      break;
    case BI_ACT_SILU:
#pragma unroll
      for (int i = 0; i < 16; ++i) z[i] = silu(z[i]);
      break;
    default:
      break;
  }
}

// 32 accumulator columns of this lane's row times the scales and with the
// bias; ws and bias: those columns' values in shared memory.
template <bool kQ8>
__device__ __forceinline__ void load_z(f32x2 (&z)[16], uint32_t taddr, const float* ws,
                                       const __nv_bfloat16* bias, bool add_bias, f32x2 a_scale) {
  uint32_t v[32];
  __syncwarp();
  tmem_ld32(taddr, v);
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    f32x2 x = pair(__uint_as_float(v[4 * q]), __uint_as_float(v[4 * q + 1]));
    f32x2 y = pair(__uint_as_float(v[4 * q + 2]), __uint_as_float(v[4 * q + 3]));
    if constexpr (kQ8) {
      const float4 w4 = reinterpret_cast<const float4*>(ws)[q];
      x = mul2(mul2(x, a_scale), pair(w4.x, w4.y));
      y = mul2(mul2(y, a_scale), pair(w4.z, w4.w));
    }
    if (add_bias) {
      const uint2 b2 = reinterpret_cast<const uint2*>(bias)[q];
      x = add2(x, widen2(b2.x));
      y = add2(y, widen2(b2.y));
    }
    z[2 * q] = x;
    z[2 * q + 1] = y;
  }
}

// z + residual for eight columns, rounded
__device__ __forceinline__ uint4 add_pack8(const f32x2* z, bool add, const uint4& r) {
  const uint32_t rw[4] = {r.x, r.y, r.z, r.w};
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = halves(add ? add2(z[i], widen2(rw[i])) : z[i]);
    o[i] = pack_bf16x2(f.x, f.y);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

// An epilogue warp's chunks (32 rows by 32 columns of C) of one tile: the first
// or the second half of the tile's columns, none where its rows are past M.
struct Span {
  int c, end;
};
template <int kUnit, bool kSides>
__device__ __forceinline__ Span span_of(const Tile& t, const FusedParams& p, int bn_out,
                                        int row_in_unit, int half, int side) {
  if (t.m * kUnit + row_in_unit >= p.M) return Span{0, 0};
  const int n = (min(bn_out, p.n_out - t.n * bn_out) + kChunk - 1) / kChunk;
  if constexpr (kSides) {  // a lane has its row's columns of one side
    const int per = bn_out / (2 * kChunk), first = side * per, mid = first + ((per + 1) >> 1);
    return half == 0 ? Span{min(first, n), min(mid, n)} : Span{min(mid, n), min(first + per, n)};
  }
  const int mid = (n + 1) >> 1;
  return half == 0 ? Span{0, mid} : Span{mid, n};
}

struct Ring {
  uint64_t *full, *empty, *tfull, *tempty, *drain;
  uint32_t a, b;     // the operands' tiles
  int a_sub, b_sub;  // bytes of one k-block's
  uint32_t tmem;
};

// The MMAs of all of a block's tiles, by one thread, kKG k-blocks a stage.
// This loop is what a narrow tile waits for (some 50 cycles an MMA, the loop's
// instructions or the MMA's own least time, and 150 around a stage; with the
// k-blocks of a stage counted at run time and the addresses formed anew 100 more:
// 256 x 4096 x 14336 e4m3 21 us in place of 27), so nothing is recomputed in it, and
// the next stage's barrier is looked at while the MMAs are on their way.
template <bool kQ8, bool kPair, int kKG>
__device__ __forceinline__ void issue_mmas(const FusedParams& p, const Ring& r, int first,
                                           int units, int step, volatile int* abort_flag) {
  // K-major tiles, 128-byte swizzle: rows of 128 bytes, 8-row groups 1024
  // bytes apart; an instruction takes 32 bytes of each row, the next ones
  // start 32 bytes (two units of a descriptor) further on
  const uint64_t ad0 = umma_desc_sw128(r.a, 16, 1024), bd0 = umma_desc_sw128(r.b, 16, 1024);
  const uint32_t a_step = r.a_sub >> 4, b_step = r.b_sub >> 4;
  const int stages = p.stages, kb_total = p.kb_total;
  const uint32_t idesc = p.idesc;
  int* err = p.err;
  uint64_t ad = ad0, bd = bd0;
  int stage = 0, acc = 0;
  uint32_t phase = 0, acc_phase = 0;
  bool ok = true, there = false;
  for (int u = first; u < units && ok; u += step) {
    if (!mbar_wait(&r.tempty[acc], acc_phase ^ 1u, err, abort_flag)) {
      ok = false;
      break;
    }
    tc_fence_after();
    const uint32_t d = r.tmem + static_cast<uint32_t>(acc) * kAccCols;
    uint32_t add = 0;  // 0: the tile's first MMA
    for (int left = kb_total; left > 0; left -= kKG) {
      if (!there && !mbar_wait(&r.full[stage], phase, err, abort_flag)) {
        ok = false;
        break;
      }
      tc_fence_after();
#pragma unroll
      for (int g = 0; g < kKG; ++g) {
        if (g > 0 && g >= left) continue;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          tc_mma_any<kQ8, kPair>(d, ad + g * a_step + 2u * k, bd + g * b_step + 2u * k, idesc, add);
          add = 1;
        }
      }
      uint64_t* done = &r.empty[stage];
      ad += kKG * a_step;
      bd += kKG * b_step;
      if (++stage == stages) {
        stage = 0;
        phase ^= 1u;
        ad = ad0;
        bd = bd0;
      }
      there = mbar_test(&r.full[stage], phase);
      tc_commit_any<kPair, true>(done);
    }
    if (!ok) break;
    tc_commit_any<kPair, true>(&r.tfull[acc]);
    acc ^= 1;
    if (acc == 0) acc_phase ^= 1u;
  }
  if (!ok) {  // all issued MMAs done before tensor memory is freed
    tc_commit_any<kPair, false>(r.drain);
    mbar_wait(r.drain, 0, nullptr);
  }
}

// kCtas = 2: a pair of CTAs computes 256 x bn tiles with one MMA over both
// SMs; each loads its 128 rows of A and half of the tile's rows of W, which
// both read.  kSides: the pair's MMA has 128 rows instead of 256, each CTA 64 of
// them, their first half of the columns in the first half of the accumulator's
// lanes and the second in the second.
template <bool kQ8, int kCtas, bool kSides>
__global__ void __launch_bounds__(kThreads, 1) gemm_fused_kernel(
    const __grid_constant__ CUtensorMap ta, const __grid_constant__ CUtensorMap tb,
    const __grid_constant__ CUtensorMap tc, const FusedParams p) {
  constexpr bool kPair = kCtas == 2;
  constexpr int kCtaRows = kSides ? 64 : BM;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  __shared__ uint64_t full[kMaxStages], empty[kMaxStages], tfull[2], tempty[2], drain;
  __shared__ uint32_t tmem_slot;
  __shared__ volatile int abort_flag;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  const int b_rows = p.bn / kCtas;
  const int a_sub = p.a_rows * kBlockBytes, b_sub = b_rows * kBlockBytes;  // of one k-block
  uint8_t* sA = smem;
  uint8_t* sB = smem + p.stages * p.kg * a_sub;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = kPair ? static_cast<int>(cluster_rank()) : 0;
  const int units = p.m_tiles * p.n_tiles;
  const int first = blockIdx.x / kCtas, step = gridDim.x / kCtas;

  if (threadIdx.x == 0) {
    prefetch_tmap(&ta);
    prefetch_tmap(&tb);
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&tfull[a], 1);
      mbar_init(&tempty[a], kCtas * kEpiWarps);  // one arrival per epilogue warp of the pair
    }
    mbar_init(&drain, 1);
    abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    if constexpr (kPair) tmem_alloc_pair(&tmem_slot, 2 * kAccCols);
    else tmem_alloc(&tmem_slot, 2 * kAccCols);
  }
  tc_fence_before();
  if constexpr (kPair) cluster_sync();
  else __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = tmem_slot;
  // past the wait this kernel's inputs are there and nobody reads its output any
  // more (it may have started while the one before it in the stream drains)
  grid_dependency_wait();

  if (warp == 0) {
    if (elect_one()) {
      // ------------------------------------------------------------ producer
      const int a_stage = p.kg * a_sub, b_stage = p.kg * b_sub;
      // both CTAs' bytes are counted on the even one's barriers
      const uint32_t bytes = static_cast<uint32_t>(kCtas * (a_stage + b_stage));
      const uint32_t full0 = kPair ? cluster_addr(full, 0) : 0u;
      int stage = 0, issued = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int u = first; u < units && ok; u += step) {
        const Tile t = tile_of(u, p);
        const int ra = (t.m * kCtas + rank) * kCtaRows, rb = t.n * p.bn + rank * b_rows;
        for (int kb = 0; kb < p.kb_total; kb += p.kg) {
          if (!mbar_wait(&empty[stage], phase ^ 1u, p.err, &abort_flag)) {
            ok = false;
            break;
          }
          uint8_t* a = sA + stage * a_stage;
          uint8_t* b = sB + stage * b_stage;
          if (rank == 0) mbar_arrive_expect_tx(&full[stage], bytes);
          if (!kPair && p.deep) {  // k-blocks past the last read as zero and are not used
            tma_load_3d(a, &ta, 0, ra, kb, &full[stage]);
            tma_load_3d(b, &tb, 0, rb, kb, &full[stage]);
          } else {
            for (int g = 0; g < p.kg; ++g) {
              const int x = (kb + g) * kBlockBytes;
              if constexpr (kPair) {
                tma_load_2d_pair(a + g * a_sub, &ta, x, ra, full0 + stage * 8);
                tma_load_2d_pair(b + g * b_sub, &tb, x, rb, full0 + stage * 8);
              } else {
                tma_load_2d(a + g * a_sub, &ta, x, ra, &full[stage]);
                tma_load_2d(b + g * b_sub, &tb, x, rb, &full[stage]);
              }
            }
          }
          ++issued;
          if (++stage == p.stages) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      const int last = issued > p.stages ? issued - p.stages : 0;
      if (!ok) {
        // let the copies already issued land before the block goes away
        if (rank == 0)
          for (int i = last; i < issued; ++i)
            mbar_wait(&full[i % p.stages], (i / p.stages) & 1, nullptr);
      } else if (kPair) {
        // the even CTA's MMAs arrive on this CTA's barriers: none is left to
        for (int i = last; i < issued; ++i)
          if (!mbar_wait(&empty[i % p.stages], (i / p.stages) & 1, p.err, &abort_flag)) break;
      }
    }
  } else if (warp == 1) {
    if (elect_one() && rank == 0) {
      const Ring ring{full, empty, tfull, tempty, &drain, smem_u32(sA), smem_u32(sB), a_sub, b_sub,
                      tmem_base};
      if (p.kg == 1) issue_mmas<kQ8, kPair, 1>(p, ring, first, units, step, &abort_flag);
      else if (p.kg == 2) issue_mmas<kQ8, kPair, 2>(p, ring, first, units, step, &abort_flag);
      else issue_mmas<kQ8, kPair, 4>(p, ring, first, units, step, &abort_flag);
    }
  } else {
    // ------------------------------------------------------------- epilogue
    const int ew = warp - 2, wq = warp & 3;  // this warp may access accumulator lanes 32*wq ..
    const int half = ew >> 2;
    const bool swiglu = p.act == BI_ACT_SWIGLU, add_bias = p.bias != nullptr;
    const int bn_out = swiglu ? p.bn / 2 : p.bn, acc_chunk = swiglu ? 2 * kChunk : kChunk;
    // (an MMA of 64 rows leaves rows 16 q .. 16 q + 15 in the first half of the
    // q-th quarter of the lanes)
    const int side = wq >> 1;  // (kSides)
    const int row_in_unit = kSides ? rank * kCtaRows + (wq & 1) * 32
                                   : rank * BM + wq * (p.mma_rows == 64 ? 16 : 32);
    const bool mine_too = p.mma_rows != 64 || lane < 16;
    const bool staged = p.staged != 0;
    uint8_t* buf = smem + p.ring + ew * kBufs * kChunkBytes;
    float* columns = reinterpret_cast<float*>(smem + kPoolBytes);  // [2][256] scales, then biases
    const uint32_t row_off = static_cast<uint32_t>(lane) * 64;
    const uint32_t swz = (static_cast<uint32_t>(lane) >> 1) & 3;

    int acc = 0, b = 0;
    uint32_t acc_phase = 0;
    bool ok = true;  // the same in every lane
    for (int u = first; u < units && ok; u += step) {
      const Tile t = tile_of(u, p);
      const int row0 = t.m * (kCtaRows * kCtas) + row_in_unit, row = row0 + lane;
      const Span span = span_of<kCtaRows * kCtas, kSides>(t, p, bn_out, row_in_unit, half, side);
      // this half's scales and biases, four columns a lane (N % 8 == 0)
      const int col0 = span.c * acc_chunk + 4 * lane, col = t.n * p.bn + col0;
      float4 ws = make_float4(0.f, 0.f, 0.f, 0.f);
      uint2 bs = make_uint2(0, 0);
      float row_scale = 1.0f;
      // (plain loads: the kernel before, which may write them, can still run when
      // this one starts, and read-only loads are for what no one writes meanwhile)
      if (span.c < span.end && col < p.N) {
        if constexpr (kQ8) ws = *reinterpret_cast<const float4*>(p.w_scale + col);
        if (add_bias) bs = *reinterpret_cast<const uint2*>(p.bias + col);
      }
      if (kQ8 && row < p.M && mine_too) row_scale = p.a_scale[row];
      // the residual of the first chunk, while the tile's MMAs run; each further
      // one as soon as the one before is used, and, unless the epilogue is what
      // the blocks wait for (fetching twice then costs more than it hides), all
      // of them into L2 now
      const int out0 = t.n * bn_out, cols = min(bn_out, p.n_out - out0);
      const bool adds = p.residual != nullptr && row < p.M && mine_too;
      const __nv_bfloat16* res = p.residual + static_cast<int64_t>(row) * p.n_out + out0;
      uint4 r[4];
      auto load_residual = [&](int c) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          r[q] = make_uint4(0, 0, 0, 0);
          if (adds && c < span.end && c * kChunk + 8 * q < cols)
            r[q] = *reinterpret_cast<const uint4*>(res + c * kChunk + 8 * q);
        }
      };
      load_residual(span.c);
      if (adds && (p.kb_total >= kLongBlocks || units <= step))
        for (int c = span.c + 1; c < span.end; ++c) prefetch_l2(res + c * kChunk);
      // (the one wait that lasts for a whole tile: a microsecond more for each
      // k-block, which takes 0.06 to 0.2)
      ok = __all_sync(kFull, mbar_wait(&tfull[acc], acc_phase, p.err, &abort_flag,
                                       kWaitNs + static_cast<uint64_t>(p.kb_total) * 1000));
      if (!ok) break;
      tc_fence_after();
      const f32x2 a_scale = both(row_scale);
      // (the four warps of a half write the same values; the accumulator's
      // last use, whose columns these replace, is over)
      float* cw = columns + acc * 256;
      __nv_bfloat16* cb = reinterpret_cast<__nv_bfloat16*>(columns + 512) + acc * 256;
      if (span.c < span.end && col0 < 256) {
        if constexpr (kQ8) *reinterpret_cast<float4*>(cw + col0) = ws;
        if (add_bias) *reinterpret_cast<uint2*>(cb + col0) = bs;
      }
      const uint32_t tbase = tmem_base + (static_cast<uint32_t>(wq * 32) << 16) +
                             static_cast<uint32_t>(acc) * kAccCols -
                             (kSides ? static_cast<uint32_t>(side * (p.bn / 2)) : 0u);
      for (int c = span.c; c < span.end; ++c) {
        uint8_t* mine = buf + b * kChunkBytes;
        // (here, and not between the values and their stores, where a branch on
        // one lane cost the values 400 cycles a chunk)
        if (staged && lane == 0) bulk_wait_read<kBufs - 1>();
        f32x2 z[16];
        if (swiglu) {
          // two blocks of 16 gate columns and the 16 up columns of the same
          // features; the second may lie past the tile
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if (c * kChunk + h * kSwigluBlock >= cols) {
#pragma unroll
              for (int i = 0; i < 8; ++i) z[h * 8 + i] = 0;
              continue;
            }
            f32x2 g[16];
            const int ac = c * 2 * kChunk + h * 32;
            load_z<kQ8>(g, tbase + static_cast<uint32_t>(ac), cw + ac, cb + ac, add_bias, a_scale);
#pragma unroll
            for (int i = 0; i < 8; ++i) z[h * 8 + i] = mul2(silu(g[i]), g[8 + i]);
          }
        } else {
          const int ac = c * kChunk;
          load_z<kQ8>(z, tbase + static_cast<uint32_t>(ac), cw + ac, cb + ac, add_bias, a_scale);
          activate(z, p.act);
        }
        if (staged) {
          __syncwarp();  // (lane 0's wait for the buffer holds for the warp)
#pragma unroll
          for (uint32_t q = 0; q < 4; ++q)
            *reinterpret_cast<uint4*>(mine + row_off + ((q ^ swz) << 4)) =
                add_pack8(z + 4 * q, p.residual != nullptr, r[q]);
          load_residual(c + 1);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            tma_store_2d(&tc, mine, out0 + c * kChunk, row0);
            bulk_commit();
          }
          b ^= 1;
        } else {
          __nv_bfloat16* out = p.C + static_cast<int64_t>(row) * p.n_out + out0 + c * kChunk;
#pragma unroll
          for (int q = 0; q < 4; ++q)
            if (row < p.M && mine_too && c * kChunk + 8 * q < cols)
              *reinterpret_cast<uint4*>(out + 8 * q) =
                  add_pack8(z + 4 * q, p.residual != nullptr, r[q]);
          load_residual(c + 1);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if constexpr (kPair) mbar_arrive_cluster(cluster_addr(&tempty[acc], 0));
        else mbar_arrive(&tempty[acc]);
      }
      acc ^= 1;
      if (acc == 0) acc_phase ^= 1u;
    }
    if (staged && lane == 0) bulk_wait_all();
  }
  tc_fence_before();
  if constexpr (kPair) cluster_sync();
  else __syncthreads();
  tc_fence_after();
  if (warp == 1) {
    __syncwarp();
    if constexpr (kPair) tmem_dealloc_pair(tmem_base, 2 * kAccCols);
    else tmem_dealloc(tmem_base, 2 * kAccCols);
  }
}

// How a call's work is cut up.
struct Plan {
  int ctas, bn;      // CTAs of a tile (1: 128 rows, 2: 256) and its width
  int cta_rows;      // rows of a CTA's tile: 128, or 64 of a pair whose MMA has 128
  int a_rows;        // rows of A per stage
  int kg, stages;    // k-blocks per stage, stages
  bool deep;         // one copy per operand and stage
  bool staged;       // C goes through shared memory and TMA stores, not plain ones
  int ring;          // the operand ring's bytes
};

// k-blocks per stage: the more, the fewer instructions around them (a narrow
// tile waits for those: 4 x 1088 x 12824 bf16 38 us with one, 18 with four;
// 256 x 4096 x 4096 13.6 and 12.5 with one and two), as long as enough stages
// are in flight.  Rows that are whole k-blocks come by one copy of kg * 128
// contiguous bytes of each row; other rows, and pairs, take a copy per k-block
// and more stages (128-row tiles of 64 columns: 99 x 8296 x 10176 bf16 41 us
// with one, 44 with two).
bool whole_blocks(uint64_t row_bytes, int ctas) {
  return ctas == 1 && row_bytes % kBlockBytes == 0;
}
int stage_blocks(const Plan& q, bool few, int64_t kb, uint64_t row_bytes) {
  const int sub = (q.a_rows + q.bn / q.ctas) * kBlockBytes;
  const int stages = whole_blocks(row_bytes, q.ctas) ? 3 : q.ctas == 2 ? 4 : 5;
  for (int g = few ? 4 : 2; g > 1; g /= 2)
    if (g <= kb && stages * g * sub <= q.ring) return g;
  return 1;
}

// The tile with the least cost: rounds of as many tiles as the device runs at
// once, each as long as its k-blocks or its epilogue, then one epilogue.  The cost is a
// ranking of one shape's tiles, not a time: its numbers were fitted so that the tile
// with the least cost is a fast one, over 19000 timings of 447 shapes (both types, every
// form and width; M, N and K from 72, 80 and 256 to 8192, 28672 and 14336; the tile
// chosen takes 1.011 times the best one's time on average), and e4m3 8192 x 28672 x
// 4096 comes out at 260000 and takes 493 us, 16 x 6144 x 4096 at 23600 and takes 6.  A
// k-block counts 40 to 55 for the MMA thread and 100 a stage, 6 and 0.6 a row for the
// copies into the SM, 0.65 a column that a warp's lanes have for a pair's MMAs; an
// epilogue 900 and 6 such a column; starting a pair 2200, or 700 with the smaller
// tile.  Pairs load half the rows of W for the same MMAs (8192 x
// 28672 x 4096 e4m3 526 us against 621), and with 64 rows a CTA half the rows of A (128
// x 4096 x 14336 bf16 31 us, 40 with one CTA, 43 with 128; 384 of them 44, 56, 53;
// 1024 100, 87, 67); short K's epilogues wait for one another in a pair (8192 x
// 14336 x 1024 e4m3 117 us, 100 with one CTA).  Up to 64 rows of A a k-block's time
// hardly goes by the width.  Below 128 rows one CTA loads only the rows there are, where a
// pair would fill its second half up with zeros: 4096 x 14336 bf16 65 rows 27.6 us, 32.1
// in a pair of 64 each, 80 29.9 and 32.2, 96 33.4 and 32.2, 112 33.7 and 32.3; e4m3 15.5
// and 18.7, 16.5 and 18.8, 18.2 and 18.8, 18.3 and 18.8; 28672 x 4096 bf16 41.4 to 42.2
// and 43.1 to 43.7.  The last rows before 128 would gain by a pair (127 rows 39.8 us,
// 32.3), and do not get one.
Plan fused_plan(int64_t M, int64_t N, uint64_t row_bytes, int sms, bool swiglu) {
  const int64_t kb = static_cast<int64_t>((row_bytes + kBlockBytes - 1) / kBlockBytes);
  const bool few = M <= kDirectRows;
  Plan q{};
  // The MMA always reads a window of 128 rows (64 up to 64 rows and in the smaller
  // pair), whose rows past A's tile reach accumulator rows that are never stored.
  // Only the rows that there are get loaded, in eights (the swizzle's groups): rows
  // that a copy fills with zeros cost more than rows of data, as if all of them came
  // from one place (1 x 6144 x 4096 e4m3 8.7 us with 31 such rows, 6.0 with 7).
  const int rows_there = M >= BM ? BM : static_cast<int>((M + 7) / 8 * 8);
  q.staged = !few;
  q.ring = kPoolBytes - (q.staged ? kEpiWarps * kBufs * kChunkBytes : 0);
  struct Form {
    int ctas, cta_rows;
    double mma, start;
  };
  const Form forms[3] = {{1, BM, 55.0, 0.0}, {2, BM, 40.0, 2200.0}, {2, 64, 50.0, 700.0}};
  Plan best{};
  double least = 1e300;
  for (int f = 0; f < (M >= BM ? 3 : 1); ++f) {
    q.ctas = forms[f].ctas;
    q.cta_rows = forms[f].cta_rows;
    q.a_rows = std::min(rows_there, q.cta_rows);
    const int sides = BM / q.cta_rows;  // into which a tile's columns are cut
    const int step = (few ? 16 : 32) * (swiglu ? 2 : 1) * sides;
    // (with few rows a second round of narrow tiles streams a long K better than
    // one of wide tiles: with widths up to 128 and up to 256 e4m3 64 x 28672 x 4096 22.2
    // and 23.8 us, 1 x 28672 x 4096 21.1, 22.3, bf16 1 x 28672 x 1536 16.9, 17.8, 64 x
    // 28672 x 2048 22.3, 23.7, but 32 x 20000 x 4096 30.3, 28.9; short K e4m3 7 x 19848 x
    // 1136 10.3, 9.1, 64 rows 11.4, 9.7, but 64 x 28672 x 2048 12.7, 13.8)
    for (q.bn = few && kb >= 24 ? 128 : 256; q.bn >= step; q.bn -= step) {
      q.kg = stage_blocks(q, few, kb, row_bytes);
      const int64_t rows = q.cta_rows * q.ctas;
      const int64_t tiles = (M + rows - 1) / rows * ((N + q.bn - 1) / q.bn);
      const int64_t rounds = (tiles + sms / q.ctas - 1) / (sms / q.ctas);
      const double block =
          few ? 700.0 + 0.25 * q.bn
              : std::max({forms[f].mma + 100.0 / q.kg, 6.0 + 0.6 * (q.a_rows + q.bn / q.ctas),
                          q.ctas == 2 ? 0.65 * q.bn / sides : 0.0});
      const double epilogue = few ? 500.0 + 7.0 * q.bn : 900.0 + 6.0 * q.bn / sides;
      const double cost = forms[f].start +
                          static_cast<double>(rounds) * std::max(kb * block, epilogue) + epilogue;
      if (cost < least) {
        least = cost;
        best = q;
      }
    }
  }
  best.deep = best.kg > 1 && whole_blocks(row_bytes, best.ctas);
  const int sub = (best.a_rows + best.bn / best.ctas) * kBlockBytes;
  best.stages = std::min(kMaxStages, best.ring / (best.kg * sub));
  // the last window of A stays inside the ring
  while (best.stages * best.kg * best.a_rows + best.cta_rows - best.a_rows >
         best.ring / kBlockBytes)
    --best.stages;
  return best;
}

// Pairs of CTAs that fit on the device at once (0 on failure); the same for
// all of the kernel's pairs, asked once per device.
int resident_pairs() {
  constexpr int kMaxDevices = 64;
  static std::atomic<int> known[kMaxDevices];
  int d = -1;
  if (cudaGetDevice(&d) != cudaSuccess || d < 0 || d >= kMaxDevices) return 0;
  int n = known[d].load(std::memory_order_relaxed);
  if (n == 0) {
    const auto kernel = gemm_fused_kernel<true, 2, false>;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(kSmemBytes)) != cudaSuccess)
      return 0;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = 2;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(2);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmemBytes;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess || n < 0) return 0;
    known[d].store(n, std::memory_order_relaxed);
  }
  return n;
}

template <bool kQ8, int kCtas, bool kSides>
bi_status launch(const CUtensorMap& ta, const CUtensorMap& tb, const CUtensorMap& tc,
                 const FusedParams& p, int grid, cudaStream_t s) {
  const auto kernel = gemm_fused_kernel<kQ8, kCtas, kSides>;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           static_cast<int>(kSmemBytes)) != cudaSuccess)
    return BI_ERR_CUDA;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = kCtas;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = kCtas == 1 ? 1 : 2;
  return cuda_status(cudaLaunchKernelEx(&cfg, kernel, ta, tb, tc, p));
}

template <bool kQ8>
bi_status launch(const Plan& plan, const CUtensorMap& ta, const CUtensorMap& tb,
                 const CUtensorMap& tc, const FusedParams& p, int grid, cudaStream_t s) {
  if (plan.ctas == 1) return launch<kQ8, 1, false>(ta, tb, tc, p, grid, s);
  return plan.cta_rows == BM ? launch<kQ8, 2, false>(ta, tb, tc, p, grid, s)
                             : launch<kQ8, 2, true>(ta, tb, tc, p, grid, s);
}

}  // namespace

bi_status launch_gemm_fused(const void* A, const float* a_scale, const void* W,
                            const float* w_scale, const void* bias, const void* residual, void* C,
                            int64_t M, int64_t N, int64_t K, int act, bool q8, int* err,
                            cudaStream_t s) {
  const int sms = device_sm_count();
  if (sms <= 0) return BI_ERR_CUDA;
  const bool swiglu = act == BI_ACT_SWIGLU;
  const uint64_t row_bytes = static_cast<uint64_t>(K) * (q8 ? 1 : 2);
  const Plan plan = fused_plan(M, N, row_bytes, sms, swiglu);
  FusedParams p{};
  p.C = static_cast<__nv_bfloat16*>(C);
  p.bias = static_cast<const __nv_bfloat16*>(bias);
  p.residual = static_cast<const __nv_bfloat16*>(residual);
  p.a_scale = a_scale;
  p.w_scale = w_scale;
  p.err = err;
  p.M = static_cast<int>(M);
  p.N = static_cast<int>(N);
  p.n_out = static_cast<int>(swiglu ? N / 2 : N);
  p.act = act;
  p.bn = plan.bn;
  p.a_rows = plan.a_rows;
  p.kg = plan.kg;
  p.deep = plan.deep;
  p.stages = plan.stages;
  p.staged = plan.staged;
  p.ring = plan.ring;
  p.kb_total = static_cast<int>((row_bytes + kBlockBytes - 1) / kBlockBytes);
  const int rows = plan.cta_rows * plan.ctas;
  p.m_tiles = static_cast<int>((M + rows - 1) / rows);
  p.n_tiles = static_cast<int>((N + p.bn - 1) / p.bn);
  // (a block's tile index passes the last one by at most a grid)
  if (static_cast<int64_t>(p.m_tiles) * p.n_tiles > 0x7fffffff - sms) return BI_ERR_UNSUPPORTED;
  // raster: the smaller operand whole where it leaves half of L2 (2048 x 4096 x 14336
  // bf16, A 56 MiB: 137 us in two groups, 133 in one), else in even groups of up to
  // 40 MiB of it (8192 x 28672 x 4096 bf16, A 64 MiB, in a run of a second: 1100 us in
  // two groups, 1167 whole)
  p.m_fast = M <= N ? 1 : 0;
  const int64_t tile_bytes = static_cast<int64_t>(p.m_fast ? rows : p.bn) * row_bytes;
  const int64_t span = p.m_fast ? p.m_tiles : p.n_tiles, all = span * tile_bytes;
  const int64_t groups = all <= int64_t(60) << 20 ? 1 : (all - 1) / (int64_t(40) << 20) + 1;
  const int64_t group = (span + groups - 1) / groups;
  p.by_per = Divisor(group * (p.m_fast ? p.n_tiles : p.m_tiles));
  p.by_group = Divisor(group);
  p.by_last = Divisor(span % group ? span % group : group);
  // up to 64 rows the MMA takes 64 (an element's sum is the same): below some
  // 100 columns its time goes by its rows, not by them
  p.mma_rows = M <= kDirectRows ? 64 : BM;
  const int mma = plan.ctas == 2 ? rows : p.mma_rows;
  p.idesc = q8 ? umma_idesc_e4m3(mma, p.bn) : umma_idesc_bf16(mma, p.bn, false, false);
  CUtensorMap ta, tb, tc{};
  const uint64_t ra = static_cast<uint64_t>(M), rb = static_cast<uint64_t>(N);
  if (!make_tmap_rows(&ta, A, ra, row_bytes, plan.a_rows, plan.deep ? plan.kg : 1) ||
      !make_tmap_rows(&tb, W, rb, row_bytes, p.bn / plan.ctas, plan.deep ? plan.kg : 1))
    return BI_ERR_CUDA;
  if (plan.staged && !make_tmap_chunks(&tc, C, ra, static_cast<uint64_t>(p.n_out)))
    return BI_ERR_CUDA;
  const int units = p.m_tiles * p.n_tiles;
  int blocks = sms;
  if (plan.ctas == 2) {
    blocks = resident_pairs();
    if (blocks <= 0) return BI_ERR_CUDA;
  }
  const int grid = std::min(units, blocks) * plan.ctas;
  return q8 ? launch<true>(plan, ta, tb, tc, p, grid, s)
            : launch<false>(plan, ta, tb, tc, p, grid, s);
}

}  // namespace bi
