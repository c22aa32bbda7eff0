// quant_rows.cu -- rows held as e4m3 with one fp32 scale each: RMSNorm (after
// the residual's addition) with that output, and rows of a bf16 matrix.
//
//   t = max(max_j |v_j|, 448 * 2^-126),  scale = t / 448,
//   y_j = e4m3(448 v_j / t)
//
// so that y * scale stands for v and the largest magnitude is stored as 448,
// the largest e4m3 number.  The quotient is formed from v and t directly,
// rounded once to fp32, and not from the rounded scale: for a bf16 row it is
// exact wherever it lies midway between two e4m3 numbers, so ties go to the
// even one as the formula says.  A row with an infinity or a NaN gets the
// scale NaN and zeros.
//
// Each row is a function of its own elements only, in an order fixed by its
// length: the norm's reduction is the batch-invariant RMSNorm's
// (rmsnorm_row.cuh; v is exactly that kernel's fp32 value), and a maximum does
// not depend on its order.
//
// Bound by memory: a row is read once and kept in registers.  One row per
// block, or one per warp (eight a block) where the row's shape is one warp.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "bi_internal.h"
#include "device_common.cuh"
#include "rmsnorm_row.cuh"

namespace bi {
namespace {

constexpr float kTop = 448.0f;                    // the largest e4m3 number
constexpr float kLeastTop = 448.0f * 0x1p-126f;   // a scale is never below 2^-126
constexpr int kRowsPerBlock = 8;                  // of rows of one warp each

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

// 448 v / t of a row's values.  A quotient q = RN(u r), r = RN(1 / t),
// corrected by its exact remainder is the correctly rounded u / t (Markstein,
// IBM J. Res. Dev. 34, 1990) while no step over- or underflows; so u and t are
// taken times a power of two that brings t between 2^-53 and 2^64 (quotients
// whose remainder still underflows are far below the least e4m3 number).
struct RowDivisor {
  float c, t, r;
  __device__ explicit RowDivisor(float top) {
    const float p = top < 0x1p-40f ? 0x1p64f : top > 0x1p60f ? 0x1p-64f : 1.0f;
    c = 0.875f * p;  // 448 / 512
    t = top * p;
    r = __fdiv_rn(1.0f, t);
  }
  __device__ __forceinline__ float operator()(float v) const {
    const float u = __fmul_rn(v, c);
    const float q = __fmul_rn(u, r);
    // (the remainder's sign the way round that keeps a zero's sign)
    return __fmul_rn(__fmaf_rn(__fmaf_rn(q, t, -u), -r, q), 512.0f);
  }
};

__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
  return lo | hi << 16;
}

__device__ __forceinline__ uint32_t magnitude(float v) {
  return __float_as_uint(v) & 0x7fffffffu;
}

__device__ __forceinline__ void widen8(const uint4& x, float (&v)[8]) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = bf16_lo(w[i]);
    v[2 * i + 1] = bf16_hi(w[i]);
  }
}

// One row's vectors of 8 values as this thread holds them: vector
// first + k * stride of the row, k < VPT.  `values(k, i, v)` gives the 8
// values of vector i (again in the second pass: a few products cost less than
// the registers that would hold them).
template <int VPT, bool kWarpRow, typename Values>
__device__ __forceinline__ void quantise_row(const Values& values, uint32_t* red,
                                             uint2* __restrict__ y, float* __restrict__ scale,
                                             int64_t row, int nvec, int first, int stride) {
  uint32_t top = 0;
#pragma unroll
  for (int k = 0; k < VPT; ++k) {
    const int i = first + k * stride;
    if (i >= nvec) continue;
    float v[8];
    values(k, i, v);
#pragma unroll
    for (int e = 0; e < 8; ++e) top = max(top, magnitude(v[e]));
  }
  top = row_max<kWarpRow>(top, red);
  const bool fine = top < 0x7f800000u;
  const float t = fmaxf(__uint_as_float(top), kLeastTop);
  if (first == 0) scale[row] = fine ? __fdiv_rn(t, kTop) : __uint_as_float(0x7fffffffu);
  const RowDivisor part(t);
#pragma unroll
  for (int k = 0; k < VPT; ++k) {
    const int i = first + k * stride;
    if (i >= nvec) continue;
    uint2 o = make_uint2(0u, 0u);
    if (fine) {
      float v[8];
      values(k, i, v);
      o = make_uint2(e4m3x4(part(v[0]), part(v[1]), part(v[2]), part(v[3])),
                     e4m3x4(part(v[4]), part(v[5]), part(v[6]), part(v[7])));
    }
    __stcs(y + row * nvec + i, o);
  }
}

// kAdd: h = bf16(x + res) first, written to h (which may be x or res: a
// thread reads its elements of both before it writes any).
template <int VPT, bool kAdd, bool kWarpRow>
__global__ void __launch_bounds__(1024) rmsnorm_q8_kernel(
    const uint4* x, const uint4* res, const uint4* __restrict__ w, uint4* h,
    uint2* __restrict__ y, float* __restrict__ scale, int64_t M, int nvec, float inv_h,
    float eps) {
  __shared__ float red[32];
  __shared__ uint32_t red_max[32];
  const int first = kWarpRow ? threadIdx.x & 31 : threadIdx.x;
  const int stride = kWarpRow ? 32 : blockDim.x;
  const int64_t row =
      kWarpRow ? blockIdx.x * (int64_t)kRowsPerBlock + (threadIdx.x >> 5) : blockIdx.x;
  if (kWarpRow && row >= M) return;
  uint4 hv[VPT];
#pragma unroll
  for (int k = 0; k < VPT; ++k) {
    const int i = first + k * stride;
    hv[k] = make_uint4(0, 0, 0, 0);
    if (i < nvec) {
      hv[k] = __ldcs(x + row * nvec + i);
      if (kAdd) hv[k] = add_bf16x8(hv[k], __ldcs(res + row * nvec + i));
    }
  }
  if (kAdd) {
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      const int i = first + k * stride;
      if (i < nvec) __stcs(h + row * nvec + i, hv[k]);
    }
  }
  float ss = 0.0f;
#pragma unroll
  for (int k = 0; k < VPT; ++k) ss = sum_squares8(hv[k], ss);
  // (a row of one warp: block_sum's second butterfly adds zeros)
  const float r = inv_rms(kWarpRow ? warp_sum(ss) : block_sum(ss, red), inv_h, eps);
  quantise_row<VPT, kWarpRow>(
      [&](int k, int i, float (&v)[8]) {
        float g[8];
        widen8(__ldg(w + i), g);
        widen8(hv[k], v);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = __fmul_rn(__fmul_rn(v[e], r), g[e]);
      },
      red_max, y, scale, row, nvec, first, stride);
}

template <int VPT, bool kWarpRow>
__global__ void __launch_bounds__(1024) quantize_q8_kernel(const uint4* __restrict__ x,
                                                           uint2* __restrict__ y,
                                                           float* __restrict__ scale, int64_t M,
                                                           int nvec) {
  __shared__ uint32_t red_max[32];
  const int first = kWarpRow ? threadIdx.x & 31 : threadIdx.x;
  const int stride = kWarpRow ? 32 : blockDim.x;
  const int64_t row =
      kWarpRow ? blockIdx.x * (int64_t)kRowsPerBlock + (threadIdx.x >> 5) : blockIdx.x;
  if (kWarpRow && row >= M) return;
  uint4 xv[VPT];
#pragma unroll
  for (int k = 0; k < VPT; ++k) {
    const int i = first + k * stride;
    xv[k] = i < nvec ? __ldcs(x + row * nvec + i) : make_uint4(0, 0, 0, 0);
  }
  quantise_row<VPT, kWarpRow>([&](int k, int, float (&v)[8]) { widen8(xv[k], v); }, red_max, y,
                              scale, row, nvec, first, stride);
}

template <int VPT, bool kAdd>
void launch_norm(const void* x, const void* res, const void* w, void* h, void* y, float* scale,
                 int64_t M, int64_t H, int threads, float eps, cudaStream_t s) {
  const int nvec = static_cast<int>(H / 8);
  const float inv_h = 1.0f / static_cast<float>(H);
  const auto* xp = static_cast<const uint4*>(x);
  const auto* rp = static_cast<const uint4*>(res);
  const auto* wp = static_cast<const uint4*>(w);
  auto* hp = static_cast<uint4*>(h);
  auto* yp = static_cast<uint2*>(y);
  if constexpr (VPT <= 2) {  // a row of one warp has at most 64 vectors
    if (threads == 32) {
      rmsnorm_q8_kernel<VPT, kAdd, true>
          <<<static_cast<unsigned>((M + kRowsPerBlock - 1) / kRowsPerBlock), 32 * kRowsPerBlock, 0,
             s>>>(xp, rp, wp, hp, yp, scale, M, nvec, inv_h, eps);
      return;
    }
  }
  rmsnorm_q8_kernel<VPT, kAdd, false><<<static_cast<unsigned>(M), threads, 0, s>>>(
      xp, rp, wp, hp, yp, scale, M, nvec, inv_h, eps);
}

template <int VPT>
void launch_rows(const void* x, void* y, float* scale, int64_t M, int64_t K, int threads,
                 cudaStream_t s) {
  const int nvec = static_cast<int>(K / 8);
  const auto* xp = static_cast<const uint4*>(x);
  auto* yp = static_cast<uint2*>(y);
  if constexpr (VPT <= 2) {
    if (threads == 32) {
      quantize_q8_kernel<VPT, true>
          <<<static_cast<unsigned>((M + kRowsPerBlock - 1) / kRowsPerBlock), 32 * kRowsPerBlock, 0,
             s>>>(xp, yp, scale, M, nvec);
      return;
    }
  }
  quantize_q8_kernel<VPT, false>
      <<<static_cast<unsigned>(M), threads, 0, s>>>(xp, yp, scale, M, nvec);
}

}  // namespace

bi_status launch_rmsnorm_q8(const void* x, const void* res, const void* w, void* h, void* y,
                            float* scale, int64_t M, int64_t H, float eps, cudaStream_t s) {
  const RowShape sh = row_shape(H);
  switch (sh.vpt) {
#define BI_NORM(V)                                                                    \
  case V:                                                                             \
    if (res) launch_norm<V, true>(x, res, w, h, y, scale, M, H, sh.threads, eps, s);  \
    else launch_norm<V, false>(x, res, w, h, y, scale, M, H, sh.threads, eps, s);     \
    break;
    BI_NORM(1) BI_NORM(2) BI_NORM(4) BI_NORM(8)
#undef BI_NORM
    default: return BI_ERR_UNSUPPORTED;
  }
  return cuda_status(cudaGetLastError());
}

bi_status launch_quantize_q8(const void* x, void* y, float* scale, int64_t M, int64_t K,
                             cudaStream_t s) {
  const RowShape sh = row_shape(K);
  switch (sh.vpt) {
    case 1: launch_rows<1>(x, y, scale, M, K, sh.threads, s); break;
    case 2: launch_rows<2>(x, y, scale, M, K, sh.threads, s); break;
    case 4: launch_rows<4>(x, y, scale, M, K, sh.threads, s); break;
    case 8: launch_rows<8>(x, y, scale, M, K, sh.threads, s); break;
    default: return BI_ERR_UNSUPPORTED;
  }
  return cuda_status(cudaGetLastError());
}

}  // namespace bi
