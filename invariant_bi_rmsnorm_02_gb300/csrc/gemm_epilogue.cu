// gemm_epilogue.cu -- C = act(A W^T + bias) + residual on the 5th-generation
// tensor cores, for bf16 operands and for e4m3 operands with a scale per row
// of A and of W.
//
// Batch invariance: as in the plain GEMM every shape runs one instruction
// (tcgen05.mma.cta_group::1, kind::f16 with K = 16 or kind::f8f6f4 with K = 32,
// M = 128) and accumulates the k-blocks of 128 bytes in increasing k into one
// fp32 accumulator; what an element's sum is does not depend on the
// instruction's N, and the epilogue is element-wise.  So a row of C depends
// only on its rows of A and of the residual, W and the bias, and the tile's
// width may be chosen from the shape (fused_plan).
//
// Epilogue, every step one fp32 operation rounded once:
//   z = acc (bf16), (acc * a_scale) * w_scale (e4m3);  z += bias;  z = act(z);
//   z += residual;  C = bf16(z).
//
// Structure: persistent blocks (one per SM), 6 warps: a TMA producer, an MMA
// issuer with two accumulators in tensor memory, four epilogue warps of 32
// accumulator rows each.  A tile is 128 rows by 16 .. 256 columns, a stage of
// the operand ring one, two or four k-blocks.  All of these are run-time
// values: the same code serves every shape.  Every wait is bounded; a wait
// that runs out records BI_ERR_TIMEOUT, tells the other roles to stop, waits
// (bounded) for its copies and MMAs in flight, frees tensor memory and
// returns.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "bi_internal.h"
#include "device_common.cuh"
#include "tcgen05.cuh"

namespace bi {
namespace {

constexpr int BM = 128;
constexpr int kThreads = 192;
constexpr int kBlockBytes = 128;             // bytes of a row in one k-block
constexpr int kMaxStages = 8;
constexpr int kRingBytes = 208 * 1024;
constexpr size_t kSmemBytes = 1024 + kRingBytes;
constexpr uint32_t kAccCols = 256;           // columns between the two accumulators
constexpr int kSwigluBlock = 16;             // gate (then up) rows of a block of W

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
  int m_tiles, n_tiles, kb_total;
  int group, m_fast;              // raster, as in the plain GEMM
  uint32_t idesc;
};

struct Tile {
  int m, n;
};
// Tile order (it only decides which block runs a tile and when): the smaller
// operand is kept resident in L2 in groups of `group` tiles while the other
// one streams past it once per group.
__device__ __forceinline__ Tile tile_of(int u, const FusedParams& p) {
  const int span = p.m_fast ? p.m_tiles : p.n_tiles, other = p.m_fast ? p.n_tiles : p.m_tiles;
  const int per = p.group * other;
  const int g = u / per, r = u - g * per;
  const int gs = min(p.group, span - g * p.group);
  const int fast = g * p.group + r % gs, slow = r / gs;
  return p.m_fast ? Tile{fast, slow} : Tile{slow, fast};
}

// D (tmem) = A B (+ D if accumulate), one CTA, e4m3 operands.
__device__ __forceinline__ void tc_mma_f8(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc,
                                          uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// silu(z) = z / (1 + exp(-z)), as silu_mul_f32 forms it.
__device__ __forceinline__ float silu_f32(float z) {
  return __fdiv_rn(z, __fadd_rn(1.0f, expf(-z)));
}

// In 32 values, one activation; the choice is the same for the whole call.
__device__ __forceinline__ void activate(float (&z)[32], int act) {
  switch (act) {
    case BI_ACT_RELU:  // a NaN stays one
#pragma unroll
      for (int i = 0; i < 32; ++i) z[i] = z[i] <= 0.0f ? 0.0f : z[i];
      break;
    case BI_ACT_GELU:  // z/2 (1 + erf(z / sqrt 2)), by erfc so that the left tail keeps its digits
#pragma unroll
      for (int i = 0; i < 32; ++i)
        z[i] = __fmul_rn(__fmul_rn(0.5f, z[i]), erfcf(__fmul_rn(z[i], -0.70710678118654752f)));
      break;
    case BI_ACT_GELU_TANH:  // z/2 (1 + tanh u) = z / (1 + exp(-2u)), u = sqrt(2/pi) (z + 0.044715 z^3)
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        const float c = __fmul_rn(__fmul_rn(z[i], z[i]), 0.044715f);
        const float u2 = __fmul_rn(__fmaf_rn(z[i], c, z[i]), -1.5957691216057308f);
        z[i] = __fdiv_rn(z[i], __fadd_rn(1.0f, expf(u2)));
      }
      break;
    case BI_ACT_SILU:
#pragma unroll
      for (int i = 0; i < 32; ++i) z[i] = silu_f32(z[i]);
      break;
    default:
      break;
  }
}

template <bool kQ8>
__global__ void __launch_bounds__(kThreads, 1) gemm_fused_kernel(
    const __grid_constant__ CUtensorMap ta, const __grid_constant__ CUtensorMap tb,
    const FusedParams p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  __shared__ uint64_t full[kMaxStages], empty[kMaxStages], tfull[2], tempty[2], drain;
  __shared__ uint32_t tmem_slot;
  __shared__ volatile int abort_flag;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  const int a_sub = p.a_rows * kBlockBytes, b_sub = p.bn * kBlockBytes;  // of one k-block
  uint8_t* sA = smem;
  uint8_t* sB = smem + p.stages * p.kg * a_sub;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int units = p.m_tiles * p.n_tiles;

  if (threadIdx.x == 0) {
    prefetch_tmap(&ta);
    prefetch_tmap(&tb);
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&tfull[a], 1);
      mbar_init(&tempty[a], 4);  // one arrival per epilogue warp
    }
    mbar_init(&drain, 1);
    abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) tmem_alloc(&tmem_slot, 2 * kAccCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = tmem_slot;

  if (warp == 0) {
    if (lane == 0) {
      // ------------------------------------------------------------ producer
      int stage = 0, issued = 0;
      uint32_t phase = 0;
      bool ok = true;
      const uint32_t bytes = static_cast<uint32_t>(p.kg * (a_sub + b_sub));
      for (int u = blockIdx.x; u < units && ok; u += gridDim.x) {
        const Tile t = tile_of(u, p);
        for (int kb = 0; kb < p.kb_total; kb += p.kg) {
          if (!mbar_wait(&empty[stage], phase ^ 1u, p.err, &abort_flag)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(&full[stage], bytes);
          uint8_t* a = sA + stage * p.kg * a_sub;
          uint8_t* b = sB + stage * p.kg * b_sub;
          if (p.kg == 1) {
            tma_load_2d(a, &ta, kb * kBlockBytes, t.m * BM, &full[stage]);
            tma_load_2d(b, &tb, kb * kBlockBytes, t.n * p.bn, &full[stage]);
          } else {  // k-blocks past the last read as zero and are not used
            tma_load_3d(a, &ta, 0, t.m * BM, kb, &full[stage]);
            tma_load_3d(b, &tb, 0, t.n * p.bn, kb, &full[stage]);
          }
          ++issued;
          if (++stage == p.stages) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      if (!ok) {
        // let the copies already issued land before the block goes away
        const int first = issued > p.stages ? issued - p.stages : 0;
        for (int i = first; i < issued; ++i)
          mbar_wait(&full[i % p.stages], (i / p.stages) & 1, nullptr);
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      // ----------------------------------------------------------- MMA issuer
      int stage = 0, acc = 0;
      uint32_t phase = 0, acc_phase = 0;
      bool ok = true;
      for (int u = blockIdx.x; u < units && ok; u += gridDim.x) {
        if (!mbar_wait(&tempty[acc], acc_phase ^ 1u, p.err, &abort_flag)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t d = tmem_base + static_cast<uint32_t>(acc) * kAccCols;
        for (int kb0 = 0; kb0 < p.kb_total; kb0 += p.kg) {
          if (!mbar_wait(&full[stage], phase, p.err, &abort_flag)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const int here = min(p.kg, p.kb_total - kb0);
          for (int g = 0; g < here; ++g) {
            // K-major tiles, 128-byte swizzle: rows of 128 bytes, 8-row groups
            // 1024 bytes apart; an instruction takes 32 bytes of each row
            const uint64_t ad =
                umma_desc_sw128(smem_u32(sA + (stage * p.kg + g) * a_sub), 16, 1024);
            const uint64_t bd =
                umma_desc_sw128(smem_u32(sB + (stage * p.kg + g) * b_sub), 16, 1024);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const uint32_t add = (kb0 + g > 0 || k > 0) ? 1u : 0u;
              if constexpr (kQ8)
                tc_mma_f8(d, ad + 2u * k, bd + 2u * k, p.idesc, add);
              else
                tc_mma(d, ad + 2u * k, bd + 2u * k, p.idesc, add);
            }
          }
          tc_commit(&empty[stage]);
          if (++stage == p.stages) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (!ok) break;
        tc_commit(&tfull[acc]);
        acc ^= 1;
        if (acc == 0) acc_phase ^= 1u;
      }
      if (!ok) {
        tc_commit(&drain);  // all issued MMAs done before tensor memory is freed
        mbar_wait(&drain, 0, nullptr);
      }
    }
  } else {
    // ------------------------------------------------------------- epilogue
    const int wq = warp & 3;  // this warp may access accumulator lanes 32*wq ..
    const bool swiglu = p.act == BI_ACT_SWIGLU;
    int acc = 0;
    uint32_t acc_phase = 0;
    for (int u = blockIdx.x; u < units; u += gridDim.x) {
      const Tile t = tile_of(u, p);
      if (!mbar_wait(&tfull[acc], acc_phase, p.err, &abort_flag)) break;
      __syncwarp();
      tc_fence_after();
      const int row0 = t.m * BM + wq * 32, row = row0 + lane;
      const int n0 = t.n * p.bn, n_end = min(n0 + p.bn, p.N);
      const uint32_t tbase = tmem_base + (static_cast<uint32_t>(wq * 32) << 16) +
                             static_cast<uint32_t>(acc) * kAccCols;
      float a_scale = 1.0f;
      if (kQ8 && row < p.M) a_scale = __ldg(p.a_scale + row);
      // 32 accumulator columns at a time (the last chunk of a tile may have
      // 16: its other columns are read and not stored)
      for (int col = n0; row0 < p.M && col < n_end; col += 32) {
        uint32_t v[32];
        __syncwarp();
        tmem_ld32(tbase + static_cast<uint32_t>(col - n0), v);
        if (row >= p.M) continue;
        float z[32];
#pragma unroll
        for (int q = 0; q < 4; ++q) {  // eight columns: N % 8 == 0
          const bool in = col + 8 * q < n_end;
          float ws[8];
          if constexpr (kQ8) {
            const float4* src = reinterpret_cast<const float4*>(p.w_scale + col + 8 * q);
            const float4 x = in ? __ldg(src) : make_float4(0, 0, 0, 0);
            const float4 y = in ? __ldg(src + 1) : make_float4(0, 0, 0, 0);
            ws[0] = x.x; ws[1] = x.y; ws[2] = x.z; ws[3] = x.w;
            ws[4] = y.x; ws[5] = y.y; ws[6] = y.z; ws[7] = y.w;
          }
          uint4 b = make_uint4(0, 0, 0, 0);
          if (p.bias && in) b = __ldg(reinterpret_cast<const uint4*>(p.bias + col + 8 * q));
          const uint32_t bw[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            float x = __uint_as_float(v[8 * q + e]);
            if constexpr (kQ8) x = __fmul_rn(__fmul_rn(x, a_scale), ws[e]);
            if (p.bias) x = __fadd_rn(x, e & 1 ? bf16_hi(bw[e >> 1]) : bf16_lo(bw[e >> 1]));
            z[8 * q + e] = x;
          }
        }
        int groups = 4;  // of eight columns
        int64_t at = static_cast<int64_t>(row) * p.n_out + col;
        if (swiglu) {  // 16 gate columns, then the 16 up columns of the same features
#pragma unroll
          for (int i = 0; i < kSwigluBlock; ++i) z[i] = silu_mul_f32(z[i], z[kSwigluBlock + i]);
          groups = 2;
          at = static_cast<int64_t>(row) * p.n_out + col / 2;
        } else {
          activate(z, p.act);
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          if (q >= groups || (!swiglu && col + 8 * q >= n_end)) continue;
          if (p.residual) {  // may be C: read before it is written, by the same thread
            const uint4 r = *reinterpret_cast<const uint4*>(p.residual + at + 8 * q);
            const uint32_t rw[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
            for (int e = 0; e < 8; ++e)
              z[8 * q + e] = __fadd_rn(z[8 * q + e],
                                       e & 1 ? bf16_hi(rw[e >> 1]) : bf16_lo(rw[e >> 1]));
          }
          *reinterpret_cast<uint4*>(p.C + at + 8 * q) = make_uint4(
              pack_bf16x2(z[8 * q], z[8 * q + 1]), pack_bf16x2(z[8 * q + 2], z[8 * q + 3]),
              pack_bf16x2(z[8 * q + 4], z[8 * q + 5]), pack_bf16x2(z[8 * q + 6], z[8 * q + 7]));
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&tempty[acc]);
      acc ^= 1;
      if (acc == 0) acc_phase ^= 1u;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) {
    __syncwarp();
    tmem_dealloc(tmem_base, 2 * kAccCols);
  }
}

// The tile width: rounds of #SM tiles times what a tile costs.  A tile's
// k-block takes the MMA 2 bn cycles, or as long as its operands take to come,
// in proportion to bn plus the rows of A; widths are multiples of 16 (32 with
// SwiGLU, whose blocks of 16 gate and 16 up rows stay together).
int tile_width(int64_t M, int64_t N, int sms, bool swiglu) {
  const int step = swiglu ? 32 : 16;
  const int64_t mt = (M + BM - 1) / BM;
  const int64_t rows = std::min<int64_t>(M, BM);
  int best = 256;
  int64_t best_cost = INT64_MAX;
  for (int bn = 256; bn >= step; bn -= step) {
    const int64_t tiles = mt * ((N + bn - 1) / bn);
    const int64_t cost = (tiles + sms - 1) / sms * std::max<int64_t>(2 * bn, bn + rows);
    if (cost < best_cost) {
      best_cost = cost;
      best = bn;
    }
  }
  return best;
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
  p.bn = tile_width(M, N, sms, swiglu);
  // rows of A per stage: the MMA always reads a window of 128 rows, whose
  // rows past M reach accumulator rows that are never stored
  p.a_rows = M <= 32 ? 32 : M <= 64 ? 64 : BM;
  p.kb_total = static_cast<int>((row_bytes + kBlockBytes - 1) / kBlockBytes);
  // k-blocks per stage: one copy then reads kg * 128 contiguous bytes of each
  // row; at least four stages
  const int sub = (p.a_rows + p.bn) * kBlockBytes;
  p.kg = 1;
  if (row_bytes % kBlockBytes == 0)
    for (int g = 4; g > 1; g /= 2)
      if (g <= p.kb_total && 4 * g * sub <= kRingBytes) {
        p.kg = g;
        break;
      }
  // (the last window of A stays inside the ring: with stages of at most four
  // k-blocks A takes at most 8 * 4 of its tiles, and W's follow them)
  p.stages = std::min(kMaxStages, kRingBytes / (p.kg * sub));
  while (p.stages * p.kg * p.a_rows + BM - p.a_rows > kRingBytes / kBlockBytes) --p.stages;
  p.m_tiles = static_cast<int>((M + BM - 1) / BM);
  p.n_tiles = static_cast<int>((N + p.bn - 1) / p.bn);
  // (a block's tile index passes the last one by at most a grid)
  if (static_cast<int64_t>(p.m_tiles) * p.n_tiles > 0x7fffffff - sms) return BI_ERR_UNSUPPORTED;
  // raster: about 40 MB of the smaller operand stay in L2 per group
  p.m_fast = M <= N ? 1 : 0;
  const int64_t tile_bytes = static_cast<int64_t>(p.m_fast ? BM : p.bn) * row_bytes;
  const int64_t span = p.m_fast ? p.m_tiles : p.n_tiles;
  p.group = static_cast<int>(
      std::min(span, std::max<int64_t>(1, (int64_t(40) << 20) / std::max<int64_t>(1, tile_bytes))));
  p.idesc = q8 ? umma_idesc_e4m3(BM, p.bn) : umma_idesc_bf16(BM, p.bn, false, false);
  CUtensorMap ta, tb;
  const uint64_t ra = static_cast<uint64_t>(M), rb = static_cast<uint64_t>(N);
  if (!make_tmap_rows(&ta, A, ra, row_bytes, p.a_rows, p.kg) ||
      !make_tmap_rows(&tb, W, rb, row_bytes, p.bn, p.kg))
    return BI_ERR_CUDA;
  const int units = p.m_tiles * p.n_tiles;
  const int grid = std::min(units, sms);
  const auto kernel = q8 ? gemm_fused_kernel<true> : gemm_fused_kernel<false>;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           static_cast<int>(kSmemBytes)) != cudaSuccess)
    return BI_ERR_CUDA;
  kernel<<<grid, kThreads, kSmemBytes, s>>>(ta, tb, p);
  return cuda_status(cudaGetLastError());
}

}  // namespace bi
