// quant_rows.cu -- rows held as e4m3 with one fp32 scale each: RMSNorm (after
// the residual's addition) with that output, and rows of a bf16 matrix.
//
//   t = max(max_j |v_j|, 448 * 2^-126),  scale = t / 448,
//   y_j = e4m3(448 v_j / t)
//
// so that y * scale stands for v and the largest magnitude is stored as 448,
// the largest e4m3 number.  A row with an infinity or a NaN gets the scale NaN
// and zeros.  Rows of a bf16 matrix take the quotient of 448 v and t rounded
// once to fp32 (exact where it lies midway between two e4m3 numbers, so ties,
// which such quotients do hit, go to the even one); the norm's fp32 values v,
// which hit no ties but by chance, take v times the rounded 448 / t.
//
// Each row is a function of its own elements only, in an order fixed by its
// length: the norm's reduction is the batch-invariant RMSNorm's
// (rmsnorm_row.cuh; v is exactly that kernel's fp32 value), and a maximum does
// not depend on its order.
//
// A row is read once and kept in registers; one row per block, or one per warp
// (eight a block) where the row's shape is one warp.  Bound by memory for many
// rows (8192 of 14336 quantised 56 us = 6.3 TB/s, 0.93 of the measured rate; the
// norm of 8192 of 4096 with a residual 36 us, 0.96, without one 16.5), by the launch for
// few (64 of 4096: 1.5 and 1.9 us among others).  With one value an
// instruction it was instructions that bounded it (33 million elements at 16 each
// are 15 us of issue slots, against 15 of memory); products and quotients are
// formed two at a time (f32x2).
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "bi_internal.h"
#include "device_common.cuh"
#include "f32x2.cuh"
#include "rmsnorm_row.cuh"

namespace bi {
namespace {

constexpr float kTop = 448.0f;                    // the largest e4m3 number
constexpr float kLeastTop = 448.0f * 0x1p-126f;   // a scale is never below 2^-126
constexpr int kRowsPerBlock = 8;                  // of rows of one warp each

// max(a, |b|), a NaN where either is one
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(fabsf(b)));
  return r;
}

// The largest magnitude's bits over the row (fp32 magnitudes order as
// integers, NaN above infinity above the rest).
template <bool kWarpRow>
__device__ __forceinline__ uint32_t row_max(uint32_t v, uint32_t* red) {
  v = __reduce_max_sync(kFull, v);
  if (kWarpRow) return v;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (lane == 0) red[warp] = v;
  __syncthreads();
  const int nw = (blockDim.x + 31) >> 5;
  return __reduce_max_sync(kFull, lane < nw ? red[lane] : 0u);
}

// What a row's largest magnitude (bits) gives: whether it is finite, and t.
// The row's first thread stores the scale.
struct RowTop {
  bool fine;
  float t;
  __device__ RowTop(uint32_t top, bool first, float* scale) {
    fine = top < 0x7f800000u;
    t = fmaxf(__uint_as_float(top), kLeastTop);
    if (first) *scale = fine ? __fdiv_rn(t, kTop) : __uint_as_float(0x7fffffffu);
  }
};

__device__ __forceinline__ uint32_t e4m3x4(f32x2 a, f32x2 b) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(halves(a), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(halves(b), __NV_SATFINITE, __NV_E4M3);
  return lo | hi << 16;
}

// kAdd: h = bf16(x + res) first, written to h (which may be x or res: a
// thread reads its elements of both before it writes any).  64 registers a
// thread; with 48, of which one more block of 256 threads fits an SM, values
// were spilled (64 rows of 4096 2.4 us where 64 registers took 1.8, 8192 17.3 and
// 16.9, before the weight's loads went ahead of the sum's barrier).
template <int VPT, bool kAdd, bool kWarpRow>
__global__ void __launch_bounds__(1024) rmsnorm_q8_kernel(
    const uint4* x, const uint4* res, const uint4* w, uint4* h, uint2* __restrict__ y,
    float* __restrict__ scale, int64_t M, int nvec, float inv_h, float eps) {
  __shared__ float red[32];
  __shared__ uint32_t red_max[32];
  const int first = kWarpRow ? threadIdx.x & 31 : threadIdx.x;
  const int stride = kWarpRow ? 32 : blockDim.x;
  const int64_t row =
      kWarpRow ? blockIdx.x * (int64_t)kRowsPerBlock + (threadIdx.x >> 5) : blockIdx.x;
  grid_dependency_wait();  // (these kernels may start while the one before drains)
  if (kWarpRow && row >= M) return;
  // (the sums in a loop of their own: one between the loads waits for those before it)
  constexpr int kGroup = VPT < 4 ? VPT : 4;
  uint4 hv[VPT];
#pragma unroll
  for (int k0 = 0; k0 < VPT; k0 += kGroup) {
    uint4 rv[kGroup];
#pragma unroll
    for (int g = 0; g < kGroup; ++g) {
      const int i = first + (k0 + g) * stride;
      hv[k0 + g] = rv[g] = make_uint4(0, 0, 0, 0);
      if (i < nvec) {
        hv[k0 + g] = __ldcs(x + row * nvec + i);
        if (kAdd) rv[g] = __ldcs(res + row * nvec + i);
      }
    }
    if (kAdd) {
#pragma unroll
      for (int g = 0; g < kGroup; ++g) {
        const int i = first + (k0 + g) * stride;
        hv[k0 + g] = add_bf16x8(hv[k0 + g], rv[g]);
        if (i < nvec) __stcs(h + row * nvec + i, hv[k0 + g]);
      }
    }
  }
  // blocks of 1024 threads have registers for the row, not for its values too:
  // they form them twice (1024 x 65536 with a residual 95 us when kept, 87 when not)
  constexpr bool kKeep = VPT <= 4;
  // The weight by ordinary loads (read-only ones are for what no one writes while
  // the kernel lives, and the kernel before may write w while this one starts),
  // which have to go out before the sum's barrier: 8192 x 4096 16.5 us, 17.8 behind it.
  auto weight = [&](int k) {
    const int i = first + k * stride;
    return i < nvec ? w[i] : make_uint4(0, 0, 0, 0);
  };
  uint4 wk[kKeep ? VPT : 1];
  if constexpr (kKeep) {
#pragma unroll
    for (int k = 0; k < VPT; ++k) wk[k] = weight(k);
  }
  float ss = 0.0f;
#pragma unroll
  for (int k = 0; k < VPT; ++k) ss = sum_squares8(hv[k], ss);
  // (a row of one warp: block_sum's second butterfly adds zeros)
  const float r = inv_rms(kWarpRow ? warp_sum(ss) : block_sum(ss, red), inv_h, eps);
  const f32x2 r2 = both(r);
  auto values = [&](int k, f32x2 (&v)[4]) {
    uint4 wv;
    if constexpr (kKeep) wv = wk[k];
    else wv = weight(k);
    const uint32_t hw[4] = {hv[k].x, hv[k].y, hv[k].z, hv[k].w}, ww[4] = {wv.x, wv.y, wv.z, wv.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = mul2(mul2(widen2(hw[e]), r2), widen2(ww[e]));
  };
  f32x2 v[kKeep ? VPT : 1][4];
  float top = 0.0f;
#pragma unroll
  for (int k = 0; k < VPT; ++k) {
    f32x2(&vk)[4] = v[kKeep ? k : 0];
    values(k, vk);
    if (first + k * stride >= nvec) continue;  // (0 times an infinite r is no element's value)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 f = halves(vk[e]);
      top = max_nan(max_nan(top, f.x), f.y);
    }
  }
  const RowTop t(row_max<kWarpRow>(__float_as_uint(top), red_max), first == 0, scale + row);
  // (t is between 2^-117.2 and 2^128, so 448 / t is a normal number)
  const f32x2 q = both(__fdiv_rn(kTop, t.t));
#pragma unroll
  for (int k = 0; k < VPT; ++k) {
    const int i = first + k * stride;
    if (i >= nvec) continue;
    uint2 o = make_uint2(0u, 0u);
    if (t.fine) {
      f32x2(&vk)[4] = v[kKeep ? k : 0];
      if (!kKeep) {
        asm volatile("" : "+r"(hv[k].x), "+r"(hv[k].y), "+r"(hv[k].z), "+r"(hv[k].w));
        values(k, vk);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) vk[e] = mul2(vk[e], q);
      o = make_uint2(e4m3x4(vk[0], vk[1]), e4m3x4(vk[2], vk[3]));
    }
    __stcs(y + row * nvec + i, o);
  }
}

// kAhead: a block takes every gridDim.x-th row, the next one on its way while
// this one is quantised and stored.  For rows that leave two or three blocks to
// an SM, which load and store in step (8192 rows of 14336 66 -> 58 us in a loop);
// with eight blocks an SM they cover for one another and the copies of a row
// ahead cost more (28672 rows of 4096 53 -> 57).
template <int VPT, bool kWarpRow, bool kAhead>
__global__ void __launch_bounds__(kAhead ? 512 : 1024) quantize_q8_kernel(
    const uint4* __restrict__ x, uint2* __restrict__ y, float* __restrict__ scale, int64_t M,
    int nvec) {
  __shared__ uint32_t red_max[2][32];  // of rows in turn: a warp may be a row ahead
  const int first = kWarpRow ? threadIdx.x & 31 : threadIdx.x;
  const int stride = kWarpRow ? 32 : blockDim.x;
  int64_t row =
      kWarpRow ? blockIdx.x * (int64_t)kRowsPerBlock + (threadIdx.x >> 5) : blockIdx.x;
  grid_dependency_wait();
  uint4 xv[VPT];
  auto load = [&](int64_t r) {
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      const int i = first + k * stride;
      xv[k] = i < nvec && r < M ? __ldcs(x + r * nvec + i) : make_uint4(0, 0, 0, 0);
    }
  };
  load(row);
  for (int turn = 0; row < M; row += gridDim.x, turn ^= 1) {
    uint4 cur[VPT];
#pragma unroll
    for (int k = 0; k < VPT; ++k) cur[k] = xv[k];
    if (kAhead) load(row + gridDim.x);
    // bf16 magnitudes order as integers, two at a time
    uint32_t top2 = 0;
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      const uint32_t w[4] = {cur[k].x, cur[k].y, cur[k].z, cur[k].w};
#pragma unroll
      for (int e = 0; e < 4; ++e)
        asm("max.u16x2 %0, %0, %1;" : "+r"(top2) : "r"(w[e] & 0x7fff7fffu));
    }
    const uint32_t top = max(top2 & 0xffffu, top2 >> 16) << 16;
    const RowTop t(row_max<kWarpRow>(top, red_max[turn]), first == 0, scale + row);
    // (448 v) / t: a quotient q = RN(u r), r = RN(1 / t), corrected by its exact
    // remainder is the correctly rounded u / t (Markstein, IBM J. Res. Dev. 34,
    // 1990) while no step over- or underflows; so both are taken times a power of
    // two p that brings t between 2^-53 and 2^64 (quotients whose remainder
    // underflows all the same are far below the least e4m3 number).  u = 448 v is
    // exact for a bf16 v.
    const float p = t.t < 0x1p-40f ? 0x1p64f : t.t > 0x1p60f ? 0x1p-64f : 1.0f;
    const float d = __fmul_rn(t.t, p), inv = __fdiv_rn(1.0f, d), top_p = __fmul_rn(kTop, p);
    const f32x2 c = both(top_p), minus_c = both(-top_p), d2 = both(d), r2 = both(inv),
                minus_r2 = both(-inv);
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      const int i = first + k * stride;
      if (i >= nvec) continue;
      uint2 o = make_uint2(0u, 0u);
      if (t.fine) {
        const uint32_t w[4] = {cur[k].x, cur[k].y, cur[k].z, cur[k].w};
        f32x2 q[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const f32x2 v = widen2(w[e]);
          q[e] = mul2(mul2(v, c), r2);
          // (the remainder's sign the way round that keeps a zero's sign)
          q[e] = fma2(fma2(q[e], d2, mul2(v, minus_c)), minus_r2, q[e]);
        }
        o = make_uint2(e4m3x4(q[0], q[1]), e4m3x4(q[2], q[3]));
      }
      __stcs(y + row * nvec + i, o);
    }
    if (!kAhead) break;
  }
}

// Launch with programmatic stream serialisation: the blocks may be set up while
// the previous kernel in the stream drains, and wait for it in the kernel.
template <typename... KArgs, typename... Args>
bi_status launch(void (*kernel)(KArgs...), int64_t grid, int threads, cudaStream_t s,
                 Args... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.stream = s;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cuda_status(cudaLaunchKernelEx(&cfg, kernel, static_cast<KArgs>(args)...));
}

template <int VPT, bool kAdd>
bi_status launch_norm(const void* x, const void* res, const void* w, void* h, void* y,
                      float* scale, int64_t M, int64_t H, int threads, float eps,
                      cudaStream_t s) {
  const int nvec = static_cast<int>(H / 8);
  const float inv_h = 1.0f / static_cast<float>(H);
  const auto* xp = static_cast<const uint4*>(x);
  const auto* rp = static_cast<const uint4*>(res);
  const auto* wp = static_cast<const uint4*>(w);
  auto* hp = static_cast<uint4*>(h);
  auto* yp = static_cast<uint2*>(y);
  if constexpr (VPT <= 2) {  // a row of one warp has at most 64 vectors
    if (threads == 32)
      return launch(rmsnorm_q8_kernel<VPT, kAdd, true>, (M + kRowsPerBlock - 1) / kRowsPerBlock,
                    32 * kRowsPerBlock, s, xp, rp, wp, hp, yp, scale, M, nvec, inv_h, eps);
  }
  return launch(rmsnorm_q8_kernel<VPT, kAdd, false>, M, threads, s, xp, rp, wp, hp, yp,
                scale, M, nvec, inv_h, eps);
}

template <int VPT>
bi_status launch_rows(const void* x, void* y, float* scale, int64_t M, int64_t K, int threads,
                      cudaStream_t s) {
  const int nvec = static_cast<int>(K / 8);
  const auto* xp = static_cast<const uint4*>(x);
  auto* yp = static_cast<uint2*>(y);
  if constexpr (VPT <= 2) {
    if (threads == 32)
      return launch(quantize_q8_kernel<VPT, true, false>, (M + kRowsPerBlock - 1) / kRowsPerBlock,
                    32 * kRowsPerBlock, s, xp, yp, scale, M, nvec);
  }
  if constexpr (VPT == 4) {
    const int sms = device_sm_count();
    if (sms <= 0) return BI_ERR_CUDA;
    const int64_t most = static_cast<int64_t>(sms) * (1024 / threads);
    if (threads > 256 && threads <= 512 && M > most)
      return launch(quantize_q8_kernel<VPT, false, true>, most, threads, s, xp, yp, scale, M,
                    nvec);
  }
  return launch(quantize_q8_kernel<VPT, false, false>, M, threads, s, xp, yp, scale, M, nvec);
}

}  // namespace

bi_status launch_rmsnorm_q8(const void* x, const void* res, const void* w, void* h, void* y,
                            float* scale, int64_t M, int64_t H, float eps, cudaStream_t s) {
  const RowShape sh = row_shape(H);
  switch (sh.vpt) {
#define BI_NORM(V)                                                                             \
  case V:                                                                                      \
    return res ? launch_norm<V, true>(x, res, w, h, y, scale, M, H, sh.threads, eps, s)        \
               : launch_norm<V, false>(x, res, w, h, y, scale, M, H, sh.threads, eps, s);
    BI_NORM(1) BI_NORM(2) BI_NORM(4) BI_NORM(8)
#undef BI_NORM
    default: return BI_ERR_UNSUPPORTED;
  }
}

bi_status launch_quantize_q8(const void* x, void* y, float* scale, int64_t M, int64_t K,
                             cudaStream_t s) {
  const RowShape sh = row_shape(K);
  switch (sh.vpt) {
    case 1: return launch_rows<1>(x, y, scale, M, K, sh.threads, s);
    case 2: return launch_rows<2>(x, y, scale, M, K, sh.threads, s);
    case 4: return launch_rows<4>(x, y, scale, M, K, sh.threads, s);
    case 8: return launch_rows<8>(x, y, scale, M, K, sh.threads, s);
    default: return BI_ERR_UNSUPPORTED;
  }
}

}  // namespace bi
