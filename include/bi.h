/*
 * bi.h -- C ABI of libbi: batch-invariant reduction kernels for GB300 (sm_103a).
 *
 * The three reductions of an LLM forward pass -- RMSNorm, the linear-layer
 * GEMM and attention over a paged KV cache -- written so that every output
 * row is a function of its own inputs only: the same bytes whatever the batch
 * size, the row's position in the batch, the neighbouring rows, the KV-cache
 * length of other requests or the way a prompt is cut into prefill chunks.
 *
 * Pages this interface follows:
 *   [P1] "Reproducible LLM Inference - Batch Invariance, the Cost of
 *        Determinism, and Where Bitwise Identity Is Actually Required"
 *        (hidekazu-konishi.com)
 *   [P3] "Your Answer Depends on Who Else Is in the Batch" (praveentn.live)
 * Batch invariance is defined in P1 §5.1: the result for one element of a
 * batch does not change when the batch changes.  P1 §5.3-5.5 name the three
 * operations and the freedom each kernel must give up.
 *
 * Conventions (all entry points):
 *   - Tensor pointers are DEVICE pointers owned by the caller; bf16 means IEEE
 *     bfloat16 (passed as void*), row-major, densely packed unless a stride is
 *     given.  Every tensor pointer must be 16-byte aligned.
 *   - `stream` is a cudaStream_t passed as void* (NULL = the legacy default
 *     stream).  Calls are asynchronous on that stream; they never synchronise
 *     and never allocate device memory.  Scratch space ("workspace") is
 *     provided by the caller; its size comes from the matching *_workspace_size
 *     query, which is pure host arithmetic except where noted.
 *   - Return: BI_OK, or an error code; on an argument error nothing is
 *     launched.  Errors found on the device (a page id outside the pool, a
 *     kv length beyond the page table, a bounded wait that ran out) do not
 *     fault the GPU: the kernel skips the access, records the code in a
 *     per-device error word and returns; bi_check_device_errors reads it.
 *   - Modes: BI_MODE_INVARIANT is the batch-invariant kernel.  BI_MODE_VARIANT
 *     is the same arithmetic with the reduction split chosen from the batch
 *     shape (split-K for the GEMM, a split row for RMSNorm, a fixed split
 *     COUNT for attention), i.e. what a shape-tuned kernel does; it is
 *     deterministic run to run but not batch-invariant, and exists to measure
 *     the cost of invariance (P1 §8).
 *   - Only the current CUDA device is used.
 */
#ifndef BI_H
#define BI_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum bi_status {
  BI_OK = 0,
  BI_ERR_INVALID_ARG = 1,   /* null pointer, negative size, misaligned pointer */
  BI_ERR_UNSUPPORTED = 2,   /* shape outside what the kernels implement */
  BI_ERR_WORKSPACE = 3,     /* workspace missing or smaller than required */
  BI_ERR_CUDA = 4,          /* a CUDA runtime/driver call failed */
  BI_ERR_DEVICE_BOUNDS = 5, /* device-side check: index outside a buffer */
  BI_ERR_TIMEOUT = 6        /* device-side bounded wait ran out */
} bi_status;

typedef enum bi_mode {
  BI_MODE_INVARIANT = 0,
  BI_MODE_VARIANT = 1
} bi_mode;

/* ------------------------------------------------------------------------ */
/* RMSNorm  (P1 §5.3-5.4; P3 "Where the reductions are", "A Concrete Example") */
/* ------------------------------------------------------------------------ */
/* y[i,:] = x[i,:] * (mean_j x[i,j]^2 + eps)^(-1/2) * w
 *   x [M,H] bf16, w [H] bf16, y [M,H] bf16 (y may not alias x).
 *   y_f32 (may be NULL): [M,H] fp32, the same values before the final
 *   rounding to bf16.
 *   Sum of squares in fp32; one rounding to bf16 at the end.
 * INVARIANT: one row per thread block; the block shape and the order of the
 *   in-row reduction depend on H only (P1 §5.3: more rows only means more
 *   rows per core).  Needs no workspace.
 * VARIANT: when M is small the row is cut into s chunks reduced by separate
 *   blocks and combined in a second pass (P1 §5.3; P3's 32-block example);
 *   s is chosen from M and the SM count.  Workspace: see below.
 * Requirements: H % 8 == 0, 8 <= H <= 65536, M >= 0 (M == 0 is a no-op).
 * Errors: BI_ERR_INVALID_ARG (null/misaligned), BI_ERR_UNSUPPORTED (H),
 *   BI_ERR_WORKSPACE, BI_ERR_CUDA. */
bi_status bi_rmsnorm(const void* x, const void* w, void* y, float* y_f32, int64_t M,
                     int64_t H, float eps, bi_mode mode, void* workspace,
                     size_t workspace_bytes, void* stream);

/* Residual add fused with RMSNorm (the pre-norm step of a decoder layer).
 * The pages define only RMSNorm ("Your Answer Depends on Who Else Is in the
 * Batch", "A Concrete Example"); the fused add is this library's addition:
 *   h = bf16(x + residual)   (each element: fp32 add, rounded once to bf16),
 *       written over residual (the updated residual stream);
 *   y = RMSNorm(h) * w        exactly as bi_rmsnorm(h, w, y, ...).
 * The bytes equal a bf16 add followed by bi_rmsnorm, in both modes; the
 * invariant mode reads x and residual once (one row per CTA, the RMSNorm
 * row reduction above).  Layouts, alignment and errors as bi_rmsnorm; x and
 * residual must not overlap.  BI_MODE_VARIANT runs the add, then the split
 * RMSNorm, and needs bi_rmsnorm_workspace_size(M, H, BI_MODE_VARIANT)
 * bytes. */
bi_status bi_add_rmsnorm(const void* x, void* residual, const void* w, void* y, float* y_f32,
                         int64_t M, int64_t H, float eps, bi_mode mode, void* workspace,
                         size_t workspace_bytes, void* stream);

/* Bytes of workspace bi_rmsnorm needs: 0 for BI_MODE_INVARIANT; for
 * BI_MODE_VARIANT an upper bound (M * 64 * 4).  Host arithmetic only. */
size_t bi_rmsnorm_workspace_size(int64_t M, int64_t H, bi_mode mode);

/* ------------------------------------------------------------------------ */
/* GEMM  (P1 §3.3, §5.4; P3 "Where the reductions are")                     */
/* ------------------------------------------------------------------------ */
/* C[i,n] = sum_k A[i,k] * W[n,k]
 *   A [M,K] bf16 (activations, K contiguous), W [N,K] bf16 (a Linear weight,
 *   K contiguous), C [M,N] bf16.  fp32 accumulation in tensor memory, one
 *   rounding to bf16 at the end.
 * INVARIANT: one tensor-core instruction family (tcgen05.mma kind::f16,
 *   M=128, K=16) and one K order (k-blocks of 64 in increasing k) for every
 *   M; no split-K, no stream-K (P1 §5.4: the instruction and the split are
 *   the two freedoms to give up).  Output tiles are 128 x 64 (instruction
 *   N=64) for M <= 64 when ceil(N/64) tiles fit in one wave of the device's
 *   SMs, K % 64 == 0 and K >= 256 (more blocks then stream the weight);
 *   otherwise 128 x 192 above 32 rows when its tiles fill the SMs' rounds
 *   better (rounds of #SM tiles times the width, 192's weighted by 10/9),
 *   else 128 x 256.  The instruction's N does not change any output
 *   element's sum (every element has the same bytes at N = 64, 192 and 256
 *   on sm_103a), so a row's bytes do not depend on M.  Needs no
 *   workspace.
 * VARIANT: same tiles and instruction, but K is split into s slices chosen
 *   from M, N and the SM count (split-K, P1 §5.4: only when the output tiles
 *   cover at most a quarter of the SMs, then doubling until the slices cover
 *   them, at least 4 k-blocks per slice); fp32 slice results are
 *   summed in slice order by a second kernel.  s = variant_splits if > 0.
 * Requirements: M >= 0, N >= 1, K >= 1, N % 8 == 0, K % 8 == 0 (16-byte rows
 *   for the tensor-memory-access engine), all dims < 2^31.
 * Errors: as bi_rmsnorm. */
bi_status bi_gemm(const void* A, const void* W, void* C, int64_t M, int64_t N, int64_t K,
                  bi_mode mode, int variant_splits, void* workspace,
                  size_t workspace_bytes, void* stream);

/* Bytes of workspace bi_gemm needs: 0 for BI_MODE_INVARIANT.  For
 * BI_MODE_VARIANT it queries the current device's SM count (so it needs a
 * GPU) and returns splits * M * N * 4 for the split count bi_gemm will use;
 * (size_t)-1 if the device cannot be queried. */
size_t bi_gemm_workspace_size(int64_t M, int64_t N, int64_t K, bi_mode mode,
                              int variant_splits);

/* Split count bi_gemm uses in BI_MODE_VARIANT for this shape on a device
 * with num_sms SMs (1 = no split), counted over the tiles bi_gemm runs for
 * it (above); bi_gemm_swiglu uses the count of its [M, 2F] shape.  Host
 * arithmetic only. */
int bi_gemm_variant_splits(int64_t M, int64_t N, int64_t K, int num_sms);

/* Gate/up projection with the SwiGLU product in the GEMM epilogue (P1 §5.4:
 * element-wise work is batch-invariant by nature, so fusing it into the
 * invariant GEMM keeps every row's bytes).
 *   out[i,j] = bf16( silu(g) * u ),  silu(x) = x / (1 + exp(-x)) in fp32,
 *   g = bf16((A W^T)[i, 256*(j/128) + j%128]),
 *   u = bf16((A W^T)[i, 256*(j/128) + 128 + j%128]).
 *   A [M,K] bf16, W [2F,K] bf16 with the gate and up rows stacked in blocks
 *   of 128 features (rows 256b .. 256b+127: gate of features 128b ..
 *   128b+127; rows 256b+128 .. 256b+255: up of the same features), out [M,F]
 *   bf16.  The GEMM arithmetic (instruction, K order, split count in both
 *   modes) is bi_gemm's on (M, 2F, K), always with 128 x 256 tiles (a tile
 *   holds the gate and up rows of 128 features), so out holds exactly the
 *   bytes of bi_gemm into a [M,2F] buffer followed by bi_silu_mul with
 *   block = 128, with no [M,2F] tensor written.
 * Workspace: bi_gemm_workspace_size(M, 2F, K, mode, variant_splits) bytes.
 * Requirements: F % 128 == 0, K % 8 == 0, 2F and K < 2^31; pointers 16-byte
 *   aligned.  Errors: as bi_gemm. */
bi_status bi_gemm_swiglu(const void* A, const void* W, void* out, int64_t M, int64_t F,
                         int64_t K, bi_mode mode, int variant_splits, void* workspace,
                         size_t workspace_bytes, void* stream);

/* ------------------------------------------------------------------------ */
/* Attention over a paged KV cache  (P1 §5.5; P3 "The attention detail that */
/* gets missed")                                                            */
/* ------------------------------------------------------------------------ */
/* Common layout:
 *   k_cache, v_cache [num_pages][Hkv][page_size][D] bf16.  Token t of
 *     sequence b lives in page block_table[b*max_blocks_per_seq + t/page_size]
 *     at slot t % page_size.  The caller writes the K/V of new tokens into
 *     the cache and extends block_table / kv_lens BEFORE calling attention,
 *     so cached and new tokens are read from one layout and reduced alike
 *     (P1 §5.5).
 *   block_table [B][max_blocks_per_seq] int32, kv_lens [B] int32: device.
 *   Grouped-query attention: q-head h reads kv-head h / (Hq/Hkv).
 *   scores = sm_scale * q.k (pass 1/sqrt(D) for the usual scale; sm_scale
 *   must be positive and finite, else BI_ERR_INVALID_ARG); softmax over the
 *   visible keys; out = sum softmax * v.
 *   out is bf16; out_f32 (may be NULL) receives the same values before the
 *   final rounding, in fp32, same layout.
 * Split plan (BI_MODE_INVARIANT, P1 §5.5 fixed split SIZE): the keys
 *   0..L-1 of a query are cut at multiples of split_size; each chunk is
 *   reduced with an online softmax over key tiles of 64 in increasing order
 *   (partial max m, sum l, unnormalised o), and the chunks are merged by a
 *   left fold in chunk order with the log-sum-exp rule, then o times the
 *   correctly rounded 1/l is rounded.
 *   Boundaries depend on absolute key indices only, never on L, B, the grid
 *   or the chunking of a prompt.
 * BI_MODE_VARIANT (a split plan sized from the batch, the kind of plan the
 *   pages name as not batch-invariant): one chunk size C for the call,
 *   C = 64 * max(ceil(Hkv * T / U), ceil(T_max / c)), where T is the sum and
 *   T_max the largest of the sequences' 64-key tile counts ceil(L/64),
 *   U = 4 * (resident split-kernel blocks on the device) the target number
 *   of work units, and c = variant_splits if > 0, else
 *   c = min(128, ceil(max_kv_len / 256)) the largest number of chunks a
 *   sequence may get (it sizes the workspace);
 *   sequence b is cut at multiples of C into ceil(L_b / C) chunks.  Every
 *   boundary moves with the lengths of the other sequences in the call.
 * A sequence with L == 0 produces zeros, and so does a row whose every score
 *   is -inf.  A NaN score makes its row NaN, and a value of V that is not
 *   finite the rows that attend to its position, whatever its weight.  (Two
 *   differences where values are not finite: decode passes over those of a
 *   split whose scores are all -inf; and a prefill chunk takes tiles of 64 keys
 *   for up to 128 rows at once, so that one up to 190 positions behind a row
 *   may make that row NaN as well.)
 * Requirements: D in {64, 128}; Hq % Hkv == 0 and Hq/Hkv <= 16;
 *   page_size == 16; split_size a positive multiple of 64; num_pages >= 1;
 *   max_blocks_per_seq >= 1.
 * Device checks: a page id outside [0, num_pages) or a kv length above
 *   max_blocks_per_seq*page_size (or above max_kv_len) is recorded as
 *   BI_ERR_DEVICE_BOUNDS and the offending sequence is skipped. */

/* Decode: one new query token per sequence.
 *   q [B][Hq][D] bf16, out [B][Hq][D] bf16.
 *   max_kv_len: host-side upper bound on kv_lens (sizes the grid only); here
 *   and in the other calls a bound above 2^30 counts as 2^30.
 *   Workspace: bi_attn_decode_workspace_size(...) bytes. */
bi_status bi_attn_decode(const void* q, const void* k_cache, const void* v_cache,
                         const int32_t* block_table, const int32_t* kv_lens, void* out,
                         float* out_f32, int B, int Hq, int Hkv, int D, int page_size,
                         int64_t num_pages, int max_blocks_per_seq, int max_kv_len,
                         int split_size, float sm_scale, bi_mode mode,
                         int variant_splits, void* workspace, size_t workspace_bytes,
                         void* stream);

/* Bytes of workspace bi_attn_decode needs: the unit list of the split plan
 * (16 bytes per (sequence, split)) and the split partials m, l, o in fp32,
 * i.e. 256 + up256(16*B*S_max) + up256(8*B*Hq*E) + 4*B*Hq*S_max*D with
 * S_max = ceil(max_kv_len / split_size) (the variant's count in
 * BI_MODE_VARIANT), E = S_max rounded up to an even number and up256
 * rounding up to a multiple of 256.
 * Host arithmetic, except that BI_MODE_VARIANT with variant_splits <= 0
 * queries the current device's SM count ((size_t)-1 if that fails). */
size_t bi_attn_decode_workspace_size(int B, int Hq, int Hkv, int D, int max_kv_len,
                                     int split_size, bi_mode mode, int variant_splits);

/* Decode without a caller workspace, for callers that cannot allocate device
 * memory (an engine that has given all of HBM to its KV-cache pool and
 * forbids further allocations, a plugin whose host framework owns the
 * allocator).  The pages describe no such entry point; it is a convenience of
 * this library.
 * Same arguments, layout and result as bi_attn_decode in BI_MODE_INVARIANT
 * (bit-identical output), minus mode and workspace.  The scratch comes from a
 * fixed array of BI_NOALLOC_SCRATCH_BYTES inside the library, reserved on
 * every GPU that loads this code until the process exits; the call itself
 * allocates nothing.
 * Limit: bi_attn_decode_workspace_size(B, Hq, Hkv, D, max_kv_len, split_size,
 *   BI_MODE_INVARIANT, 0) must not exceed BI_NOALLOC_SCRATCH_BYTES, else the
 *   call returns BI_ERR_WORKSPACE and launches nothing.
 * The first call on a device looks up the array's device address (once per
 * device, with that device current); make that first call before any stream
 * capture begins.
 * The looked-up address is kept for the life of the process: after a
 * cudaDeviceReset of that device it is stale, so do not call this entry
 * point again on a device that has been reset.
 * All calls share the array: calls whose kernels overlap on the GPU race with
 * each other, so order them (e.g. issue them on one stream).
 * Errors: as bi_attn_decode, plus BI_ERR_WORKSPACE for the size limit. */
#define BI_NOALLOC_SCRATCH_BYTES ((size_t)32 << 20)
bi_status bi_attn_decode_noalloc(const void* q, const void* k_cache, const void* v_cache,
                                 const int32_t* block_table, const int32_t* kv_lens, void* out,
                                 float* out_f32, int B, int Hq, int Hkv, int D, int page_size,
                                 int64_t num_pages, int max_blocks_per_seq, int max_kv_len,
                                 int split_size, float sm_scale, void* stream);

/* Causal prefill of one chunk per sequence (P1 §5.5, §6.4: a prompt may
 * arrive in chunks; every token's reduction must not depend on the chunking).
 *   q [total_q][Hq][D] bf16: the chunk tokens of all sequences, sequence b
 *     owning rows cu_q[b] .. cu_q[b+1]-1 (cu_q [B+1] int32, device).
 *   q_start_pos [B] int32 (device): absolute position of sequence b's first
 *     chunk token; token i of the chunk sits at position q_start_pos[b]+i and
 *     attends to keys 0..q_start_pos[b]+i.  kv_lens[b] must be at least
 *     q_start_pos[b] + chunk length (the cache already holds the chunk).
 *   out [total_q][Hq][D] bf16 (+ optional out_f32).
 *   max_q_len: host bound on the chunk lengths; max_kv_len: host bound on
 *     kv_lens.  Both size the grid only.
 * In BI_MODE_INVARIANT the result at every position is bit-identical to
 * bi_attn_decode in BI_MODE_INVARIANT with L = position + 1 and the same
 * split_size.  BI_MODE_VARIANT sizes the chunks from max_kv_len and c
 * (split size = 64 * ceil(max_kv_len / (64 c))), so results move with the
 * chunking.  Needs no workspace (pass NULL, 0).
 * Errors: as bi_attn_decode; a block whose sequence has a page id outside
 *   the pool (among the pages its keys use) or a chunk past kv_lens records
 *   BI_ERR_DEVICE_BOUNDS before any copy and leaves its rows unwritten. */
bi_status bi_attn_prefill_chunk(const void* q, const int32_t* cu_q,
                                const int32_t* q_start_pos, const void* k_cache,
                                const void* v_cache, const int32_t* block_table,
                                const int32_t* kv_lens, void* out, float* out_f32, int B,
                                int Hq, int Hkv, int D, int page_size, int64_t num_pages,
                                int max_blocks_per_seq, int64_t total_q, int max_q_len,
                                int max_kv_len, int split_size, float sm_scale,
                                bi_mode mode, int variant_splits, void* workspace,
                                size_t workspace_bytes, void* stream);

/* Write K/V rows of new tokens into the paged cache (the precondition of
 * both attention calls, P1 §5.5).  k_new, v_new [n_tokens][Hkv][D] bf16;
 * token i goes to sequence seq[i] at absolute position pos[i] (int32 device
 * arrays), i.e. page block_table[seq*max_blocks + pos/page_size], slot
 * pos % page_size.  Pure data movement, no arithmetic.  Bounds are checked
 * on the device as for attention. */
bi_status bi_kv_write(const void* k_new, const void* v_new, const int32_t* seq,
                      const int32_t* pos, int64_t n_tokens, void* k_cache, void* v_cache,
                      const int32_t* block_table, int Hkv, int D, int page_size,
                      int64_t num_pages, int max_blocks_per_seq, void* stream);

/* ------------------------------------------------------------------------ */
/* Quantised paged KV cache (about half the bytes of the bf16 one)          */
/* ------------------------------------------------------------------------ */
/* The pages define no quantised cache; this is the library's addition.
 * cache [num_pages][Hkv][BI_KV_Q8_RECORD_BYTES(D)] bytes: the record of one
 * page and kv head holds
 *   K [16][D] e4m3, V [16][D] e4m3, K scales [16], V scales [16].
 * Page tables and lengths are those of the bf16 cache.  A row (one token's K
 * or V of one head) has one scale byte c that stands for 2^(c - 127):
 *   amax = the row's largest magnitude,
 *   e = the least integer in -124 .. 7 with amax * 2^-e <= 448 (7 if none),
 *   c = e + 127, element = e4m3(x * 2^-e), rounded to nearest even, magnitudes
 *   above 448 (only where amax > 448 * 2^7 = 57344) stored as 448.
 * A row with an infinity or a NaN is stored as zeros with c = 135 and reads
 * back as NaN throughout.  Every other stored value e4m3 * 2^e is a bf16
 * number, so reading back is exact, and an element is off by at most 2^-4 of
 * its magnitude or 2^(e - 10), whichever is larger.
 * Records written by other means: scale bytes outside 3 .. 135 and the bytes
 * 0x7f and 0xff (read as 480 and -480, not NaN) give unspecified values, but
 * no access outside the buffers.
 * Requirements of all three calls: D in {64, 128}; page_size == 16;
 * num_pages * Hkv * 16 < 2^31; cache 16-byte aligned. */
#define BI_KV_Q8_RECORD_BYTES(D) (32 * (D) + 32)

/* Quantise the K/V rows of new tokens and write them into the cache: as
 * bi_kv_write, with the same arguments but one cache.  A (sequence, position)
 * given twice in one call, or two sequences' positions in one shared slot,
 * leaves that slot's rows unspecified (its scale may be one row's and its
 * elements the other's); no other slot is touched.  num_seqs: the rows of
 * block_table.  A token whose sequence (outside 0 .. num_seqs-1), position
 * or page is out of range is recorded as BI_ERR_DEVICE_BOUNDS and skipped.
 * Further requirement: n_tokens * Hkv < 2^31. */
bi_status bi_kv_write_q8(const void* k_new, const void* v_new, const int32_t* seq,
                         const int32_t* pos, int64_t n_tokens, void* cache,
                         const int32_t* block_table, int num_seqs, int Hkv, int D,
                         int page_size, int64_t num_pages, int max_blocks_per_seq,
                         void* stream);

/* Read the tokens 0 .. kv_lens[b]-1 of each sequence back as bf16 pages
 * k_out, v_out [num_out_pages][Hkv][16][D], the layout of the bf16 cache:
 * block j of sequence b goes to page out_table[b][j] (out_table int32
 * [B][max_out_blocks], device), so that bi_attn_prefill_chunk can run on the
 * result.  out_table may be block_table itself (the same page ids in a pool
 * of the same size).  Slots behind a sequence's last token and other pages
 * are left as they were.  Two sequences may share a page (and an out page)
 * whose tokens they agree on.
 * k_out and v_out must be 32-byte aligned and overlap neither each other nor
 * the cache.
 * max_kv_len: host bound on kv_lens (sizes the grid).  A length outside
 * 0 .. max_kv_len or past either table is recorded as BI_ERR_DEVICE_BOUNDS
 * and its sequence skipped; a page id outside its pool likewise skips that
 * page.  B <= 65535. */
bi_status bi_kv_read_q8(const void* cache, const int32_t* block_table, const int32_t* kv_lens,
                        int B, int Hkv, int D, int page_size, int64_t num_pages,
                        int max_blocks_per_seq, int max_kv_len, void* k_out, void* v_out,
                        const int32_t* out_table, int64_t num_out_pages, int max_out_blocks,
                        void* stream);

/* Decode over the quantised cache: bi_attn_decode with one cache in place of
 * two (same modes, split plan, workspace size, checks and errors).  The
 * result in BI_MODE_INVARIANT has exactly the bytes of bi_attn_decode on the
 * pages that bi_kv_read_q8 gives, and so those of bi_attn_prefill_chunk on
 * them at every position, wherever
 *   - the elements of q and the stored values are zero or at least 2^-126 in
 *     magnitude (an MMA aligns subnormal numbers apart), and no element of q is
 *     2^64 or more (bi_attn_decode's unscaled sums q . k become infinite from
 *     2^128 on, where these need not);
 *   - every partial sum of an output element, over its row's first keys, is zero
 *     or above 2^-100 both in magnitude and beside the largest value of V in the
 *     row's keys (the two kernels hold their sums times different powers of two,
 *     and smaller ones lose low bits).
 * Past the second bound an element is off by less than 2^-120 of the largest
 * value of V beside the usual error.  NaN results are NaN in both.
 * BI_MODE_VARIANT sizes its chunks from this kernel's resident blocks, so its
 * plan may differ from bi_attn_decode's. */
bi_status bi_attn_decode_q8(const void* q, const void* cache, const int32_t* block_table,
                            const int32_t* kv_lens, void* out, float* out_f32, int B, int Hq,
                            int Hkv, int D, int page_size, int64_t num_pages,
                            int max_blocks_per_seq, int max_kv_len, int split_size,
                            float sm_scale, bi_mode mode, int variant_splits, void* workspace,
                            size_t workspace_bytes, void* stream);

/* ------------------------------------------------------------------------ */
/* Element-wise decoder-layer steps (P1 §5.4: batch-invariant by nature)    */
/* ------------------------------------------------------------------------ */
/* Row gather: dst[i, :] = src[idx[i], :] for i < n (token embedding lookup,
 * or picking the rows that need logits).  src [rows][H] bf16, idx int32 [n]
 * (device), dst [n][H] bf16.  H % 8 == 0.  An index outside [0, rows) is
 * recorded in the device error word (BI_ERR_DEVICE_BOUNDS) and its row is
 * written as zeros.  Pure data movement. */
bi_status bi_gather_rows(const void* src, int64_t rows, int64_t H, const int32_t* idx, int64_t n,
                         void* dst, void* stream);

/* Rotary position embedding fused with the split of a QKV projection.
 *   qkv [T][(Hq + 2 Hkv) D] bf16: per token the Hq query heads, then the Hkv
 *   key heads, then the Hkv value heads, D elements each (the output of
 *   bi_gemm with the stacked q/k/v weight); pos int32 [T] (device): each
 *   token's absolute position.
 *   q [T][Hq][D], k [T][Hkv][D]: rotated; v [T][Hkv][D]: copied.
 * Rotation (the rotate-half arrangement): for pair i < D/2 of a head,
 *   angle = pos * theta^(-2i/D),
 *   y[i] = x[i] cos - x[i + D/2] sin,  y[i + D/2] = x[i + D/2] cos + x[i] sin.
 * The angle is formed in fp64 and reduced modulo 2 pi; sine, cosine and the
 * rotation are fp32, rounded once to bf16.  The pages fix no positional
 * encoding; this is the one of the Llama family.
 * Requirements: D % 16 == 0, D <= 1024, theta > 1.  Errors: as bi_rmsnorm. */
bi_status bi_rope_qkv(const void* qkv, const int32_t* pos, int64_t T, int Hq, int Hkv, int D,
                      double theta, void* q, void* k, void* v, void* stream);

/* Rotation frequencies of rotary positions stretched for long contexts, on
 * the host: freqs [rot_dim / 2] (a HOST array; copy it to the device for
 * bi_rope_qkv_scaled) and the factor on cosine and sine.  With
 * f_i = theta^(-2i/rot_dim):
 *   BI_ROPE_NONE     f_i
 *   BI_ROPE_LINEAR   f_i / factor (position interpolation)
 *   BI_ROPE_NTK      f_i with theta * factor^(rot_dim / (rot_dim - 2))
 *   BI_ROPE_LLAMA3   (1 - w) f_i / factor + w f_i, w = clamp((n_i - low_turns)
 *                    / (high_turns - low_turns), 0, 1), n_i = trained_len f_i
 *                    / (2 pi) the turns of pair i over the trained length
 *   BI_ROPE_YARN     the same mix with w = 1 - clamp((i - a) / (b - a), 0, 1),
 *                    a = max(floor(p(high_turns)), 0), b = min(ceil(
 *                    p(low_turns)), rot_dim - 1) (b - a at least 0.001),
 *                    p(n) = rot_dim ln(trained_len / (2 pi n)) / (2 ln theta);
 *                    *attn_scale = 0.1 ln(factor) + 1 (1 in the other cases)
 * The published ramps run from 4 turns (high_turns) to 1 (low_turns) for
 * LLAMA3 and from 32 to 1 for YARN.
 * theta > 1; factor >= 1 (not read for NONE); trained_len >= 1 and
 * 0 < low_turns < high_turns (read for LLAMA3 and YARN only); rot_dim even,
 * at most 1024 (NTK: above 2).  Touches no device. */
typedef enum bi_rope_scaling {
  BI_ROPE_NONE = 0,
  BI_ROPE_LINEAR = 1,
  BI_ROPE_NTK = 2,
  BI_ROPE_LLAMA3 = 3,
  BI_ROPE_YARN = 4
} bi_rope_scaling;
bi_status bi_rope_frequencies(int rot_dim, double theta, bi_rope_scaling scaling, double factor,
                              double trained_len, double low_turns, double high_turns,
                              double* freqs, float* attn_scale);

/* bi_rope_qkv with a table of frequencies, either pair arrangement and a
 * rotation of part of the head.  qkv, pos, q, k, v as bi_rope_qkv; freqs
 * [rot_dim / 2] double (device, 16-byte aligned; finite values, a NaN or
 * infinity makes its pairs NaN).  For pair i < rot_dim / 2 of a query or key
 * head, with a = pos * freqs[i], c = attn_scale cos a, s = attn_scale sin a:
 *   interleaved = 0: x0 = x[i], x1 = x[i + rot_dim / 2];
 *   interleaved = 1: x0 = x[2i], x1 = x[2i + 1];
 *   y0 = x0 c - x1 s, y1 = x1 c + x0 s in their places.
 * Elements rot_dim .. D-1 and the value heads are copied.  The angle is kept
 * in turns as a 64-bit fraction: beside the error of freqs it is off by less
 * than |pos| (|freqs[i]| 2^-52 + 2^-62) radians (2^-35 at position 131072 and
 * 2^-21 at the last int32 position for a frequency of 1; negative positions
 * alike), and is rounded to fp32 within half a turn of 0.  Cosine, sine and the
 * rotation are fp32, rounded once to bf16.
 * q, k and v must not overlap qkv or one another (BI_ERR_INVALID_ARG).
 * Requirements: D % 16 == 0, D <= 1024, rot_dim even and at most D,
 *   attn_scale positive and finite, T < 2^31.  Errors: as bi_rmsnorm. */
bi_status bi_rope_qkv_scaled(const void* qkv, const int32_t* pos, int64_t T, int Hq, int Hkv,
                             int D, int rot_dim, int interleaved, const double* freqs,
                             float attn_scale, void* q, void* k, void* v, void* stream);

/* SwiGLU product: out[t, j] = bf16(silu(g) * u), silu(g) = g / (1 + exp(-g))
 * in fp32, out [T][F] bf16, from the gate and up projections stacked in one
 * GEMM output gate_up [T][2F] bf16 in blocks of `block` features:
 *   g = gate_up[t, 2*block*(j/block) + j%block],  u = the element block
 *   columns further on.
 * block = F: all gate columns, then all up columns.  block = 128: the layout
 * bi_gemm writes with bi_gemm_swiglu's weight, so that this kernel after
 * bi_gemm gives the bytes of bi_gemm_swiglu.
 * Requirements: F % block == 0, block % 8 == 0, F < 2^31.  Errors: as bi_rmsnorm. */
bi_status bi_silu_mul(const void* gate_up, int64_t T, int64_t F, int64_t block, void* out,
                      void* stream);

/* ------------------------------------------------------------------------ */
/* Next-token selection  (P1 §9.2, §9.3)                                    */
/* ------------------------------------------------------------------------ */
/* One token per request from its row of logits, deterministic for given
 * (logits row, temperature, seed, step) whatever the batch around it.
 *   logits [B][V] bf16 (row-major, e.g. the LM-head output of bi_gemm);
 *   temperature [B] float, seed [B] and step [B] uint64, tokens [B] int32:
 *   all device pointers, caller-owned; logits aligned to 2 bytes, the
 *   others to their element size.
 * temperature[b] > 0: Gumbel-max sampling (P1 §9.3: the logits perturbed by
 *   Gumbel noise from a seeded hash), tokens[b] = argmax_v z_v / T + G_v with
 *   G_v = -log(-log(u_v)), computed in fp32 (z * (1/T), then + G).  u_v is
 *   drawn by Philox4x64-10 (Salmon et al., SC 2011) under key {seed[b], 0}
 *   at counter {v / 8, step[b], 0, 0}: 32-bit half v % 2 (low half first) of
 *   output word (v / 2) % 4, top 23 bits k, u = (k + 1/2) 2^-23.  The draw
 *   follows softmax(z / T); step is the caller's per-request counter (e.g.
 *   the position of the token being chosen), so successive tokens of one
 *   request get fresh noise.
 * temperature[b] <= 0 (or NaN): greedy, tokens[b] = argmax_v z_v (P1 §9.2).
 * Ties go to the lowest index; -0 equals +0; a NaN score counts as -inf (it
 *   is chosen only when no entry scores above -inf, lowest index first: an
 *   all-NaN or all -inf row gives token 0).
 * The argmax is a reduction under a total order, so its result does not
 *   depend on how the row is split; one launch: a cluster of 8 CTAs per row
 *   below 128 rows (one row keeps several SMs busy), one CTA per row above.
 * Requirements: 0 <= B <= 65535, 1 <= V < 2^31.  Needs no workspace.
 * Errors: BI_ERR_INVALID_ARG (null, misaligned, B < 0, V < 1),
 *   BI_ERR_UNSUPPORTED (B or V too large), BI_ERR_CUDA (launch). */
bi_status bi_sample(const void* logits, int64_t B, int64_t V, const float* temperature,
                    const uint64_t* seed, const uint64_t* step, int32_t* tokens, void* stream);

/* ------------------------------------------------------------------------ */
/* Errors and introspection                                                 */
/* ------------------------------------------------------------------------ */
/* Synchronises `stream`, then reads and clears the current device's error
 * word.  Returns BI_OK, the first recorded device error, or BI_ERR_CUDA. */
bi_status bi_check_device_errors(void* stream);

/* Diagnostic of the failure path: launches one thread that waits on a
 * barrier nothing arrives on, with the bounded wait every kernel of this
 * library uses, given up after timeout_us microseconds (1 .. 2,000,000).
 * The kernel records BI_ERR_TIMEOUT in the device error word and returns;
 * the context stays usable.  Returns the launch status (BI_ERR_INVALID_ARG
 * for an out-of-range timeout); read the recorded status with
 * bi_check_device_errors. */
bi_status bi_selftest_wait_timeout(uint32_t timeout_us, void* stream);

/* Static English description of a status code (never NULL). */
const char* bi_status_string(bi_status status);

/* Library version, "major.minor.patch". */
const char* bi_version(void);

#ifdef __cplusplus
}
#endif
#endif /* BI_H */
