// rope.cu -- rotary positions in the forms long-context decoders use, fused
// with the split of the QKV projection like bi_rope_qkv: a table of rotation
// frequencies (scaled or not, made on the host by bi_rope_frequencies), the
// rotate-half or the interleaved arrangement, and a rotation of the first
// rot_dim elements of a head with the rest passed through.
//
// Every output element is a function of its own head and position only, so
// the result does not depend on the batch.
#include <cuda_runtime.h>
#include <math_constants.h>

#include <type_traits>

#include "bi_internal.h"
#include "device_common.cuh"

namespace bi {
namespace {

// The fraction of a turn that one position adds, freq / (2 pi) mod 1, in
// units of 2^-64.  An angle is then a 64-bit product that wraps at whole
// turns by itself, with no range reduction.  1 / (2 pi) and the product with
// it are rounded to 53 bits each and the fraction to 2^-65, so an angle is off
// by less than pos * (freq * 2^-52 + 2^-62) radians: below half a unit of its
// rounding to fp32 up to positions of some 2^27, and 2^-21 at the last one.
__device__ __forceinline__ uint64_t turn_fraction(double freq) {
  double t = freq * 0.15915494309189533576888376337251;  // 1 / (2 pi)
  t -= floor(t);
  return __double2ull_rn(t * 18446744073709551616.0);  // 2^64
}
// attn_scale times cosine and sine of pos * frac turns.  The signed phase is
// converted with its own relative precision, so small angles keep theirs.
__device__ __forceinline__ float2 cos_sin(int32_t pos, uint64_t frac, float attn_scale) {
  const uint64_t phase = static_cast<uint64_t>(static_cast<int64_t>(pos)) * frac;
  const float half_turns = __ll2float_rn(static_cast<int64_t>(phase)) * 0x1p-63f;
  float s, c;
  sincospif(half_turns, &s, &c);
  return make_float2(__fmul_rn(c, attn_scale), __fmul_rn(s, attn_scale));
}
// (x0, x1) turned: both elements of a pair, rounded once to bf16 (low, high).
__device__ __forceinline__ uint32_t rotate(float x0, float x1, float2 cs) {
  return pack_bf16x2(__fsub_rn(__fmul_rn(x0, cs.x), __fmul_rn(x1, cs.y)),
                     __fadd_rn(__fmul_rn(x1, cs.x), __fmul_rn(x0, cs.y)));
}

struct RopeArgs {
  const void* qkv;
  const int32_t* pos;
  const double* freqs;
  void *q, *k, *v;
  int64_t T;
  int Hq, Hkv, D, rot;
  float attn_scale;
  int tokens;                 // per step of a block
  uint32_t inv_heads, inv_D, inv_half;  // reciprocals for div_by
};

// n / d for n * d < 2^32 through m = ceil(2^32 / d), exact there (m = 0: d = 1).
__device__ __forceinline__ int div_by(int n, uint32_t m) {
  return m ? static_cast<int>(__umulhi(static_cast<uint32_t>(n), m)) : n;
}

// A block takes `tokens` tokens a step, in chunks of kItems items per thread.
// Its threads first make the step's cosines and sines, each (token, pair) once
// for all heads, in shared memory (the frequencies' turn fractions, the only
// fp64 work, once per block); then every item of 16 elements, two 16-byte
// vectors, is turned or passed through and written by one thread, which at
// once loads its item of the next chunk into the same registers: loads are in
// flight through the stores and the next step's table.
// Bound by memory: 8192 tokens of 32 + 2 * 8 heads of 128 move 201 MB in 35 us
// (5.7 TB/s, 0.85 of the measured copy rate; 37 us with the loads issued at the
// head of their own step and three items, 47 and more with the items staged in
// shared memory by cp.async).
// A step takes whole tokens, so what a block's slots (kItems per thread) hold
// of them goes by the heads and their width; the launch takes the block of 192
// or 256 threads that they fill better.  8192 tokens, us with 192 and 256
// threads (and the share of the slots filled):
//   32 + 2*8 of 128: 35.4, 39.7 (100, 75%)   28 + 2*4 of 128: 31.5, 33.9 (75, 56%)
//   40 + 2*8 of 128: 45.2, 43.5 (58, 88%)    16 + 2*16 of 256: 65.7, 68.8 (100, 75%)
//   24 + 2*8 of 80:  24.3, 21.7 (52, 78%)    32 + 2*8 of 80:  27.9, 24.0 (62, 94%)
// 128 and 384 threads are between the two or behind both in most shapes, and 4%
// ahead at best (64 + 2 * 8 heads of 128, 128 threads).
// A width that is no multiple of 16 is bound by its 2-byte loads and the pairs
// turned twice instead: 24 + 2 * 8 heads of 80, 20 of them rotated, take 45 us
// (rotate-half) and 37 (interleaved) where 80 rotated take 22.
constexpr int kItems = 2;  // items in flight per thread

// kAligned: rot_dim % 16 == 0, so that rotated items are whole vectors of
// either half of the rotated part (rotate-half) or of pairs.  Otherwise the
// items that hold rotated elements gather their pairs one by one; the head's
// other items stay vectors.
template <int kThreads, bool kInterleaved, bool kAligned>
__global__ void __launch_bounds__(kThreads) rope_kernel(const RopeArgs a) {
  constexpr int kChunk = kItems * kThreads;
  const int heads = a.Hq + 2 * a.Hkv, half = a.rot / 2;
  extern __shared__ __align__(16) uint8_t smem[];
  float2* table = reinterpret_cast<float2*>(smem);                       // [tokens][rot / 2]
  uint64_t* frac = reinterpret_cast<uint64_t*>(table + a.tokens * half);  // [rot / 2]
  float* amp = reinterpret_cast<float*>(frac + half);                    // [rot / 2]
  const int per_head = a.D / 16, per_token = heads * per_head;
  const int rot_items = (a.rot + 15) / 16;
  const int chunks = (a.tokens * per_token + kChunk - 1) / kChunk;  // of a step
  const int64_t step = static_cast<int64_t>(gridDim.x) * a.tokens;
  const uint4* src = static_cast<const uint4*>(a.qkv);
  struct Item {
    int tok, head, sub;
    bool turn, apart;  // rotated; a vector of the first half and its partner
  };
  auto item_at = [&](int i) {
    Item it;
    const int th = div_by(i, a.inv_D);  // (token, head) of the step
    it.sub = i - th * per_head;
    it.tok = div_by(th, a.inv_heads);
    it.head = th - it.tok * heads;
    it.turn = it.head < a.Hq + a.Hkv && it.sub < rot_items;
    it.apart = kAligned && !kInterleaved && it.turn;
    return it;
  };
  auto items_of = [&](int64_t t0) {
    return static_cast<int>(a.T - t0 < a.tokens ? a.T - t0 : a.tokens) * per_token;
  };
  uint4 x[kItems][2];
  auto load = [&](int u, int64_t t0, int chunk, int items) {
    const int i = chunk * kChunk + u * kThreads + threadIdx.x;
    if (i >= items) return;
    const Item it = item_at(i);
    if (!kAligned && it.turn) return;
    const uint4* row = src + ((t0 + it.tok) * heads + it.head) * (a.D / 8);
    x[u][0] = __ldcs(row + (it.apart ? it.sub : 2 * it.sub));
    x[u][1] = __ldcs(row + (it.apart ? it.sub + rot_items : 2 * it.sub + 1));
  };
  int64_t t0 = static_cast<int64_t>(blockIdx.x) * a.tokens;
  int chunk = 0;
  if (t0 < a.T) {
#pragma unroll
    for (int u = 0; u < kItems; ++u) load(u, t0, 0, items_of(t0));
  }
  for (int p = threadIdx.x; p < half; p += kThreads) {
    const double f = a.freqs[p];
    frac[p] = turn_fraction(f);
    amp[p] = isfinite(f) ? a.attn_scale : CUDART_NAN_F;
  }
  while (t0 < a.T) {
    const int items = items_of(t0);
    if (chunk == 0) {
      __syncthreads();  // the fractions are there, the last step's table has been read
      for (int e = threadIdx.x; e < (items / per_token) * half; e += kThreads) {
        const int t = div_by(e, a.inv_half), p = e - t * half;
        table[e] = cos_sin(a.pos[t0 + t], frac[p], amp[p]);
      }
      __syncthreads();
    }
    const int next_chunk = chunk + 1 == chunks ? 0 : chunk + 1;
    const int64_t next_t0 = next_chunk ? t0 : t0 + step;
    const int next_items = next_t0 < a.T ? items_of(next_t0) : 0;
#pragma unroll
    for (int u = 0; u < kItems; ++u) {
      const int i = chunk * kChunk + u * kThreads + threadIdx.x;
      if (i < items) {
        const Item it = item_at(i);
        uint4 y0 = x[u][0], y1 = x[u][1];
        if (!kAligned && it.turn) {
          const uint16_t* row = static_cast<const uint16_t*>(a.qkv) +
                                ((t0 + it.tok) * heads + it.head) * a.D;
          auto element = [&](int e) { return __uint_as_float((uint32_t)row[e] << 16); };
          auto turned = [&](int e) -> uint32_t {  // element e of the head's output
            if (e >= a.rot) return row[e];
            const int p = kInterleaved ? e >> 1 : e < half ? e : e - half;
            const uint32_t y = rotate(element(kInterleaved ? 2 * p : p),
                                      element(kInterleaved ? 2 * p + 1 : p + half),
                                      table[it.tok * half + p]);
            return (kInterleaved ? (e & 1) : e >= half) ? y >> 16 : y & 0xffffu;
          };
          uint32_t r[8];
#pragma unroll
          for (int w = 0; w < 8; ++w)
            r[w] = turned(16 * it.sub + 2 * w) | turned(16 * it.sub + 2 * w + 1) << 16;
          y0 = make_uint4(r[0], r[1], r[2], r[3]);
          y1 = make_uint4(r[4], r[5], r[6], r[7]);
        } else if (it.turn) {
          const float4* cs4 =
              reinterpret_cast<const float4*>(table + it.tok * half + 8 * it.sub);
          uint32_t r0[4] = {y0.x, y0.y, y0.z, y0.w}, r1[4] = {y1.x, y1.y, y1.z, y1.w};
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const float4 c = cs4[w];  // pairs 2w and 2w + 1 of the item's eight
            const float2 ca = make_float2(c.x, c.y), cb = make_float2(c.z, c.w);
            if (kInterleaved) {
              uint32_t& lo = w < 2 ? r0[2 * w] : r1[2 * w - 4];
              uint32_t& hi = w < 2 ? r0[2 * w + 1] : r1[2 * w - 3];
              lo = rotate(bf16_lo(lo), bf16_hi(lo), ca);
              hi = rotate(bf16_lo(hi), bf16_hi(hi), cb);
            } else {
              const uint32_t ya = rotate(bf16_lo(r0[w]), bf16_lo(r1[w]), ca);
              const uint32_t yb = rotate(bf16_hi(r0[w]), bf16_hi(r1[w]), cb);
              r0[w] = __byte_perm(ya, yb, 0x5410);
              r1[w] = __byte_perm(ya, yb, 0x7632);
            }
          }
          y0 = make_uint4(r0[0], r0[1], r0[2], r0[3]);
          y1 = make_uint4(r1[0], r1[1], r1[2], r1[3]);
        }
        const int64_t t = t0 + it.tok;
        const int h = it.head;
        uint4* dst = (h < a.Hq ? static_cast<uint4*>(a.q) + (t * a.Hq + h) * (a.D / 8)
                      : h < a.Hq + a.Hkv
                          ? static_cast<uint4*>(a.k) + (t * a.Hkv + h - a.Hq) * (a.D / 8)
                          : static_cast<uint4*>(a.v) + (t * a.Hkv + h - a.Hq - a.Hkv) * (a.D / 8));
        dst += it.apart ? it.sub : 2 * it.sub;
        dst[0] = y0;
        dst[it.apart ? rot_items : 1] = y1;
      }
      load(u, next_t0, next_chunk, next_items);
    }
    t0 = next_t0;
    chunk = next_chunk;
  }
}

}  // namespace

bi_status launch_rope_qkv_scaled(const void* qkv, const int32_t* pos, int64_t T, int Hq, int Hkv,
                                 int D, int rot_dim, bool interleaved, const double* freqs,
                                 float attn_scale, void* q, void* k, void* v, cudaStream_t s) {
  RopeArgs a{qkv, pos, freqs, q, k, v, T, Hq, Hkv, D, rot_dim, attn_scale, 0, 0, 0, 0};
  const int sms = device_sm_count();
  if (sms <= 0) return BI_ERR_CUDA;
  const int heads = Hq + 2 * Hkv;
  const int per_token = heads * (D / 16), half = rot_dim / 2;
  // the share of a block's slots that whole tokens fill, out of 2^20
  auto filled = [&](int threads) {
    const int64_t slots = kItems * threads;
    return per_token <= slots ? (slots / per_token * per_token << 20) / slots
                              : (int64_t(per_token) << 20) /
                                    ((per_token + slots - 1) / slots * slots);
  };
  const int threads = filled(256) > filled(192) ? 256 : 192;
  // enough tokens to give every thread its kItems items, no more than the
  // default 48 KB of shared memory hold, and no fewer blocks than two an SM
  int tokens = kItems * threads / per_token;
  const int room = (49152 - half * 12) / (half * 8);
  if (tokens > room) tokens = room;
  while (tokens > 1 && T / tokens < 2 * sms) --tokens;
  if (tokens < 1) tokens = 1;
  a.tokens = tokens;
  auto inv = [](uint32_t d) { return static_cast<uint32_t>(((uint64_t(1) << 32) + d - 1) / d); };
  a.inv_D = inv(D / 16);
  a.inv_heads = inv(heads);
  a.inv_half = inv(half);
  int64_t blocks = (T + tokens - 1) / tokens;
  if (blocks > 16 * sms) blocks = 16 * sms;
  const size_t sm = static_cast<size_t>(half) * (8 * tokens + 12);
  const bool aligned = rot_dim % 16 == 0;
  auto form = [&](auto t) {
    constexpr int n = decltype(t)::value;
    return interleaved ? (aligned ? rope_kernel<n, true, true> : rope_kernel<n, true, false>)
                       : (aligned ? rope_kernel<n, false, true> : rope_kernel<n, false, false>);
  };
  auto kernel = threads == 256 ? form(std::integral_constant<int, 256>())
                               : form(std::integral_constant<int, 192>());
  kernel<<<static_cast<unsigned>(blocks), threads, sm, s>>>(a);
  return cuda_status(cudaGetLastError());
}

}  // namespace bi
