// rmsnorm_row.cuh -- the in-row reduction of the batch-invariant RMSNorm,
// shared by the kernels that have to give its bytes (bf16 output, e4m3
// output): the block shape, the order of the sum of squares and the fused
// residual add.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "device_common.cuh"

namespace bi {

constexpr unsigned kFull = 0xffffffffu;

__device__ __forceinline__ float sum_squares8(const uint4& v, float acc) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float a = bf16_lo(w[i]), b = bf16_hi(w[i]);
    acc = __fmaf_rn(a, a, acc);
    acc = __fmaf_rn(b, b, acc);
  }
  return acc;
}

// Fixed xor-butterfly over the 32 lanes; every lane ends with the same sum
// (fp32 addition is commutative, so lane i and lane i^o add the same pair).
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) v = __fadd_rn(v, __shfl_xor_sync(kFull, v, o));
  return v;
}

// Sum of one value per thread over the block, in a fixed order: warp
// butterflies, then the same butterfly over the warp sums (missing warps
// contribute +0, which leaves a sum of squares unchanged).
__device__ __forceinline__ float block_sum(float v, float* red) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  v = warp_sum(v);
  if (lane == 0) red[warp] = v;
  __syncthreads();
  const int nw = (blockDim.x + 31) >> 5;
  float t = lane < nw ? red[lane] : 0.0f;
  return warp_sum(t);
}

__device__ __forceinline__ float inv_rms(float sum_sq, float inv_h, float eps) {
  return rsqrtf(__fadd_rn(__fmul_rn(sum_sq, inv_h), eps));
}

// bf16(a + b) of 8 elements, each an fp32 add rounded once.
__device__ __forceinline__ uint4 add_bf16x8(const uint4& a, const uint4& b) {
  const uint32_t as[4] = {a.x, a.y, a.z, a.w}, bs[4] = {b.x, b.y, b.z, b.w};
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    o[i] = pack_bf16x2(__fadd_rn(bf16_lo(as[i]), bf16_lo(bs[i])),
                       __fadd_rn(bf16_hi(as[i]), bf16_hi(bs[i])));
  return make_uint4(o[0], o[1], o[2], o[3]);
}

// Block shape as a function of H only: VPT vectors of 8 elements per thread,
// T threads (a multiple of 32, at most 1024).
struct RowShape {
  int vpt, threads;
};
inline RowShape row_shape(int64_t H) {
  const int nvec = static_cast<int>(H / 8);
  int vpt = nvec >= 256 ? 4 : (nvec >= 64 ? 2 : 1);
  while ((nvec + vpt - 1) / vpt > 1024) vpt *= 2;
  int t = (nvec + vpt - 1) / vpt;
  t = (t + 31) / 32 * 32;
  return {vpt, t};
}

}  // namespace bi
