// cache_q8.cu -- the quantised paged KV cache: K/V rows of new tokens
// quantised as they are written, and cached pages read back as bf16.
//
// One scale per row (token, kv head, K or V): the least power of two, within
// 2^-124 .. 2^7, that brings the row's largest magnitude to 448 or less (the
// largest e4m3 number).  A power of two costs nothing against a general scale
// (e4m3's relative step is the same in every binade) and makes every stored
// value exact in bf16, so the attention on this cache is the bf16 attention
// on the pages read back, bit for bit.  Each row is a function of its own
// elements only, whatever the batch around it.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "bi_internal.h"
#include "device_common.cuh"
#include "e4m3.cuh"

namespace bi {
namespace {

constexpr int kPage = 16;
constexpr int kThreads = 256;
constexpr unsigned kFull = 0xffffffffu;

// ------------------------------------------------------------------ write
// D/16 lanes per row, 32 bytes of bf16 each: the K row of a (token, head) and
// its V row on neighbouring lanes, kRows such pairs in flight per thread (a
// step of `stride` apart), since a pair is only loads behind one another
// (sequence and position, page id, then the stores).  Bound by instructions
// more than by memory: a row's bookkeeping is shared by few lanes, and the
// 8192-token prompt of 8 heads of 128 (50 MB, in L2) went from 14.9 to 8.8 us with
// 16 elements a lane in place of 8.
constexpr int kRows = 2;

template <int D>
__global__ void __launch_bounds__(kThreads) kv_write_q8_kernel(
    const uint4* __restrict__ k_new, const uint4* __restrict__ v_new,
    const int32_t* __restrict__ seq, const int32_t* __restrict__ pos, uint32_t pairs, uint32_t Hkv,
    uint8_t* __restrict__ cache, const int32_t* __restrict__ bt, int num_seqs, int num_pages,
    int max_blocks, int* err) {
  constexpr uint32_t kLanes = D / 16;
  constexpr uint32_t kPerWarp = 32 / (2 * kLanes);  // pairs of a warp
  const uint32_t warp = (blockIdx.x * kThreads + threadIdx.x) / 32;
  const uint32_t stride = gridDim.x * (kThreads / 32) * kPerWarp;
  const uint32_t mine = (threadIdx.x % 32) / (2 * kLanes);
  const uint32_t c = threadIdx.x % kLanes;
  const bool is_v = (threadIdx.x / kLanes) & 1;
  const uint4* src = (is_v ? v_new : k_new) + 2 * c;
  // a warp's lanes stay together: it goes on while its first pair exists
  // (pairs < 2^31 and a step is far below it, so 32 bits hold every index)
  for (uint32_t base = warp * kPerWarp; base < pairs; base += kRows * stride) {
    uint4 x[kRows][2];
    uint32_t head[kRows];
    int page[kRows], slot[kRows];
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
      const uint32_t th = base + mine + u * stride;  // token * Hkv + head
      x[u][0] = x[u][1] = make_uint4(0, 0, 0, 0);
      page[u] = -2;  // no pair
      if (th >= pairs) continue;
      const uint32_t tok = th / Hkv;
      head[u] = th - tok * Hkv;
      x[u][0] = src[(uint64_t)th * (2 * kLanes)];
      x[u][1] = src[(uint64_t)th * (2 * kLanes) + 1];
      const int s = seq[tok], ps = pos[tok];
      slot[u] = ps % kPage;
      page[u] = -1;  // out of range
      if (s >= 0 && s < num_seqs && ps >= 0 && ps / kPage < max_blocks)
        page[u] = bt[(int64_t)s * max_blocks + ps / kPage];
      if (page[u] < 0 || page[u] >= num_pages) page[u] = -1;
    }
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
      // the largest magnitude bits of the row: bf16 magnitudes order as integers
      const uint32_t w[8] = {x[u][0].x, x[u][0].y, x[u][0].z, x[u][0].w,
                             x[u][1].x, x[u][1].y, x[u][1].z, x[u][1].w};
      uint32_t top2 = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i)
        asm("max.u16x2 %0, %0, %1;" : "+r"(top2) : "r"(w[i] & 0x7fff7fffu));
      uint32_t top = max(top2 & 0xffffu, top2 >> 16);
#pragma unroll
      for (int o = kLanes / 2; o >= 1; o >>= 1) top = max(top, __shfl_xor_sync(kFull, top, o));
      if (page[u] < 0) {
        if (page[u] == -1 && c == 0) record_error(err, BI_ERR_DEVICE_BOUNDS);
        continue;
      }
      // least e with amax 2^-e <= 448 = 1.75 * 2^8
      int e = kQ8MinExp;
      if (top >= 0x80) {  // a normal number: 1.f * 2^(exponent - 127)
        e = (int)(top >> 7) - 127 - 8 + ((top & 0x7f) > 0x60 ? 1 : 0);
        e = max(kQ8MinExp, min(kQ8MaxExp, e));
      }
      const bool fine = top < 0x7f80;
      const float inv = __uint_as_float((uint32_t)(127 - e) << 23);
      uint32_t q[4] = {0, 0, 0, 0};
      if (fine) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float2 f = make_float2(bf16_lo(w[i]) * inv, bf16_hi(w[i]) * inv);
          const uint32_t p = __nv_cvt_float2_to_fp8x2(f, __NV_SATFINITE, __NV_E4M3);
          q[i >> 1] |= p << (16 * (i & 1));
        }
      }
      uint8_t* rec = cache + (uint64_t)((uint32_t)page[u] * Hkv + head[u]) *
                                 (uint32_t)kv_q8_record_bytes(D);
      *reinterpret_cast<uint4*>(rec + (is_v ? kPage * D : 0) + slot[u] * D + 16 * c) =
          make_uint4(q[0], q[1], q[2], q[3]);
      if (c == 0)
        rec[2 * kPage * D + (is_v ? kPage : 0) + slot[u]] =
            (uint8_t)(fine ? e + kQ8ScaleBias : kQ8NonFinite);
    }
  }
}

// ------------------------------------------------------------------- read
// 32 bytes (32-byte aligned) in one store, so that a warp whose lanes write
// neighbouring 32-byte pieces fills whole sectors with each instruction (two
// 16-byte stores per lane leave every sector half written twice).
__device__ __forceinline__ void store32(void* dst, const uint4& a, const uint4& b) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(a.x),
               "r"(a.y), "r"(a.z), "r"(a.w), "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w)
               : "memory");
}

// One warp per (page, kv head) of the batch's pages: the warp finds its pages
// from a running sum of the sequences' page counts.  Bound by memory (a third
// read, two thirds written): 64 sequences, 94,100 tokens of 8 kv heads of 128
// (580 MB) take 90 us = 6.4 TB/s, 0.95 of the measured copy rate; with two
// 16-byte stores per lane instead of one of 32 bytes and half the blocks,
// 115 us.
template <int D>
__global__ void __launch_bounds__(kThreads) kv_read_q8_kernel(
    const uint8_t* __restrict__ cache, const int32_t* __restrict__ bt,
    const int32_t* __restrict__ kv_lens, int B, int Hkv, int64_t num_pages, int max_blocks,
    __nv_bfloat16* __restrict__ k_out, __nv_bfloat16* __restrict__ v_out,
    const int32_t* __restrict__ out_bt, int64_t num_out, int max_out_blocks, int max_kv_len,
    int* err) {
  const int lane = threadIdx.x & 31;
  const int64_t warps = (int64_t)gridDim.x * (kThreads / 32);
  int64_t u = (blockIdx.x * (int64_t)kThreads + threadIdx.x) / 32;  // this warp's next unit
  int64_t base = 0;                                                 // units before the slab
  for (int b0 = 0; b0 < B; b0 += 32) {
    const int bl = b0 + lane;
    int L = bl < B ? kv_lens[bl] : 0;
    if (L < 0 || L > max_kv_len || L > max_blocks * (int64_t)kPage ||
        L > max_out_blocks * (int64_t)kPage) {
      record_error(err, BI_ERR_DEVICE_BOUNDS);
      L = 0;
    }
    const int64_t mine = (int64_t)((L + kPage - 1) / kPage) * Hkv;
    int64_t incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t t = __shfl_up_sync(kFull, incl, o);
      if (lane >= o) incl += t;
    }
    const int64_t total = __shfl_sync(kFull, incl, 31);
    for (; u < base + total; u += warps) {
      const int64_t r = u - base;
      const int w = __popc(__ballot_sync(kFull, incl <= r));
      const int64_t in_seq = r - __shfl_sync(kFull, incl - mine, w);
      const int len = __shfl_sync(kFull, L, w);
      const int j = (int)(in_seq / Hkv), h = (int)(in_seq - (int64_t)j * Hkv);
      const int64_t b = b0 + w;
      const int64_t page = bt[b * max_blocks + j], outp = out_bt[b * max_out_blocks + j];
      if (page < 0 || page >= num_pages || outp < 0 || outp >= num_out) {
        if (lane == 0) record_error(err, BI_ERR_DEVICE_BOUNDS);
        continue;
      }
      const uint8_t* rec = cache + (page * Hkv + h) * kv_q8_record_bytes(D);
      const uint32_t scale = rec[2 * kPage * D + lane];
      const int64_t out = (outp * Hkv + h) * kPage * D;
      const int valid = min(kPage, len - j * kPage);
      constexpr int kChunks = 2 * kPage * D / 16 / 32;  // 16-byte chunks per lane
      uint4 x[kChunks];
#pragma unroll
      for (int i = 0; i < kChunks; ++i)
        x[i] = reinterpret_cast<const uint4*>(rec)[32 * i + lane];
#pragma unroll
      for (int i = 0; i < kChunks; ++i) {
        const int c = 32 * i + lane;
        const int row = c / (D / 16);  // 0..15 of K, then of V
        const uint32_t f = q8_factor2(__shfl_sync(kFull, scale, row));
        if ((row & 15) >= valid) continue;
        const uint32_t in[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
        uint32_t o[8];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t ev = mul_bf16x2(e4m3_even(in[k]), f), od = mul_bf16x2(e4m3_odd(in[k]), f);
          o[2 * k] = __byte_perm(ev, od, 0x5410);
          o[2 * k + 1] = __byte_perm(ev, od, 0x7632);
        }
        uint4* dst = reinterpret_cast<uint4*>((row < 16 ? k_out : v_out) + out + (row & 15) * D +
                                              (c % (D / 16)) * 16);
        store32(dst, make_uint4(o[0], o[1], o[2], o[3]), make_uint4(o[4], o[5], o[6], o[7]));
      }
    }
    base += total;
  }
}

template <int D>
bi_status write_impl(const void* k_new, const void* v_new, const int32_t* seq, const int32_t* pos,
                     int64_t n_tokens, void* cache, const int32_t* bt, int num_seqs, int Hkv,
                     int64_t num_pages, int max_blocks, int* err, cudaStream_t s) {
  const int sms = device_sm_count();
  if (sms <= 0) return BI_ERR_CUDA;
  const int64_t pairs = n_tokens * Hkv, per_block = kThreads / (2 * D / 16);
  // a pair per thread while that leaves SMs idle, kRows behind each other after
  int64_t blocks = (pairs + per_block - 1) / per_block;
  if (blocks > 4 * sms) blocks = std::max<int64_t>(4 * sms, (blocks + kRows - 1) / kRows);
  if (blocks > 32 * sms) blocks = 32 * sms;
  kv_write_q8_kernel<D><<<static_cast<unsigned>(blocks), kThreads, 0, s>>>(
      static_cast<const uint4*>(k_new), static_cast<const uint4*>(v_new), seq, pos,
      static_cast<uint32_t>(pairs), static_cast<uint32_t>(Hkv), static_cast<uint8_t*>(cache), bt,
      num_seqs, static_cast<int>(num_pages), max_blocks, err);
  return cuda_status(cudaGetLastError());
}

template <int D>
bi_status read_impl(const void* cache, const int32_t* bt, const int32_t* kv_lens, int B, int Hkv,
                    int64_t num_pages, int max_blocks, void* k_out, void* v_out,
                    const int32_t* out_bt, int64_t num_out, int max_out_blocks, int max_kv_len,
                    int* err, cudaStream_t s) {
  const int sms = device_sm_count();
  if (sms <= 0) return BI_ERR_CUDA;
  const int64_t most = static_cast<int64_t>(B) * ((max_kv_len + kPage - 1) / kPage) * Hkv;
  const int64_t want = (most + kThreads / 32 - 1) / (kThreads / 32);
  const int64_t cap = static_cast<int64_t>(sms) * 8;
  kv_read_q8_kernel<D><<<static_cast<unsigned>(want < cap ? want : cap), kThreads, 0, s>>>(
      static_cast<const uint8_t*>(cache), bt, kv_lens, B, Hkv, num_pages, max_blocks,
      static_cast<__nv_bfloat16*>(k_out), static_cast<__nv_bfloat16*>(v_out), out_bt, num_out,
      max_out_blocks, max_kv_len, err);
  return cuda_status(cudaGetLastError());
}

}  // namespace

bi_status launch_kv_write_q8(const void* k_new, const void* v_new, const int32_t* seq,
                             const int32_t* pos, int64_t n_tokens, void* cache,
                             const int32_t* block_table, int num_seqs, int Hkv, int D,
                             int64_t num_pages, int max_blocks, int* err, cudaStream_t s) {
  return D == 64 ? write_impl<64>(k_new, v_new, seq, pos, n_tokens, cache, block_table, num_seqs,
                                  Hkv, num_pages, max_blocks, err, s)
                 : write_impl<128>(k_new, v_new, seq, pos, n_tokens, cache, block_table, num_seqs,
                                   Hkv, num_pages, max_blocks, err, s);
}

bi_status launch_kv_read_q8(const void* cache, const int32_t* block_table, const int32_t* kv_lens,
                            int B, int Hkv, int D, int64_t num_pages, int max_blocks, void* k_out,
                            void* v_out, const int32_t* out_table, int64_t num_out_pages,
                            int max_out_blocks, int max_kv_len, int* err, cudaStream_t s) {
  return D == 64 ? read_impl<64>(cache, block_table, kv_lens, B, Hkv, num_pages, max_blocks, k_out,
                                 v_out, out_table, num_out_pages, max_out_blocks, max_kv_len, err, s)
                 : read_impl<128>(cache, block_table, kv_lens, B, Hkv, num_pages, max_blocks,
                                  k_out, v_out, out_table, num_out_pages, max_out_blocks,
                                  max_kv_len, err, s);
}

}  // namespace bi
