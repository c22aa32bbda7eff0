// rope.cu -- rotary positions in the forms long-context decoders use, fused
// with the split of the QKV projection like bi_rope_qkv: a table of rotation
// frequencies (scaled or not, made on the host by bi_rope_frequencies), the
// rotate-half or the interleaved arrangement, and a rotation of the first
// rot_dim elements of a head with the rest passed through.
//
// Every output element is a function of its own head and position only, so
// the result does not depend on the batch.
#include <cuda_runtime.h>
#include <math.h>

#include "bi_internal.h"
#include "device_common.cuh"

namespace bi {
namespace {

constexpr int kThreads = 256;

// The fraction of a turn that one position adds, freq / (2 pi) mod 1, in
// units of 2^-64.  An angle is then a 64-bit product that wraps at whole
// turns by itself, with an error of pos * 2^-65 turns beside the table's own
// 53 bits: exact enough at any 32-bit position with no range reduction.
__device__ __forceinline__ uint64_t turn_fraction(double freq) {
  double t = freq * 0.15915494309189533576888376337251;  // 1 / (2 pi)
  t -= floor(t);
  return __double2ull_rn(t * 18446744073709551616.0);  // 2^64
}
// Cosine and sine of phase 2^-64 turns.  The signed phase is converted with
// its own relative precision, so small angles keep theirs.
__device__ __forceinline__ void cos_sin(uint64_t phase, float& c, float& s) {
  const float half_turns = __ll2float_rn(static_cast<int64_t>(phase)) * 0x1p-63f;
  sincospif(half_turns, &s, &c);
}

// One thread per pair of elements of a head: pair p < rot / 2 is rotated, the
// others are the head's remaining elements, copied.
__global__ void __launch_bounds__(kThreads) rope_pairs_kernel(
    const uint16_t* __restrict__ qkv, const int32_t* __restrict__ pos, int64_t T, int Hq, int Hkv,
    int D, int rot, bool interleaved, const double* __restrict__ freqs, float attn_scale,
    uint16_t* __restrict__ q, uint16_t* __restrict__ k, uint16_t* __restrict__ v) {
  const int heads = Hq + 2 * Hkv, half = D / 2;
  const int64_t total = T * heads * half;
  for (int64_t e = blockIdx.x * (int64_t)kThreads + threadIdx.x; e < total;
       e += (int64_t)gridDim.x * kThreads) {
    const int64_t th = e / half;
    const int p = (int)(e - th * half);
    const int64_t t = th / heads;
    const int h = (int)(th - t * heads);
    const uint16_t* src = qkv + th * D;
    uint16_t* dst = h < Hq         ? q + (t * Hq + h) * D
                    : h < Hq + Hkv ? k + (t * Hkv + (h - Hq)) * D
                                   : v + (t * Hkv + (h - Hq - Hkv)) * D;
    if (h >= Hq + Hkv || p >= rot / 2) {
      dst[2 * p] = src[2 * p];
      dst[2 * p + 1] = src[2 * p + 1];
      continue;
    }
    const double f = freqs[p];
    float c, s;
    cos_sin(static_cast<uint64_t>(static_cast<int64_t>(pos[t])) * turn_fraction(f), c, s);
    if (!isfinite(f)) c = s = __int_as_float(0x7fffffff);
    c *= attn_scale;
    s *= attn_scale;
    const int i0 = interleaved ? 2 * p : p, i1 = interleaved ? 2 * p + 1 : p + rot / 2;
    const float x0 = __uint_as_float((uint32_t)src[i0] << 16);
    const float x1 = __uint_as_float((uint32_t)src[i1] << 16);
    const uint32_t y =
        pack_bf16x2(__fsub_rn(__fmul_rn(x0, c), __fmul_rn(x1, s)),
                    __fadd_rn(__fmul_rn(x1, c), __fmul_rn(x0, s)));
    dst[i0] = (uint16_t)y;
    dst[i1] = (uint16_t)(y >> 16);
  }
}

}  // namespace

bi_status launch_rope_qkv_scaled(const void* qkv, const int32_t* pos, int64_t T, int Hq, int Hkv,
                                 int D, int rot_dim, bool interleaved, const double* freqs,
                                 float attn_scale, void* q, void* k, void* v, cudaStream_t s) {
  const int64_t pairs = T * (Hq + 2 * Hkv) * (D / 2);
  int64_t blocks = (pairs + kThreads - 1) / kThreads;
  if (blocks > 152 * 32) blocks = 152 * 32;
  rope_pairs_kernel<<<static_cast<unsigned>(blocks), kThreads, 0, s>>>(
      static_cast<const uint16_t*>(qkv), pos, T, Hq, Hkv, D, rot_dim, interleaved, freqs,
      attn_scale, static_cast<uint16_t*>(q), static_cast<uint16_t*>(k), static_cast<uint16_t*>(v));
  return cuda_status(cudaGetLastError());
}

}  // namespace bi
