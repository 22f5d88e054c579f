// Internal launchers behind the C ABI (mars_api.cu). Arguments are validated there;
// every launcher enqueues on `stream` and returns the cudaError_t of its launches.
#pragma once

#include <cuda_runtime.h>

#include <atomic>
#include <stddef.h>
#include <stdint.h>

namespace mars {

// Host-side count of kernels enqueued by the library (read by mars_launch_count()).
void count_launches(int n);

// ---- KV commit ([notes] Key design 4): one CTA per sequence.
cudaError_t launch_kv_commit(const uint16_t* k_blk, const uint16_t* v_blk,
                             const int32_t* n_accept, int32_t* seq_lens,
                             const int32_t* block_table, int max_pages, uint16_t* k_pool,
                             uint16_t* v_pool, int num_pages, int32_t* commit_slots,
                             int batch, int B, int hkv, int d, bool batch_sync,
                             int32_t* status, cudaStream_t stream);

// ---- Block-level commit with a B_cache boundary (block buffer, batch-wide flush).
cudaError_t launch_kv_commit_block(const uint16_t* k_blk, const uint16_t* v_blk,
                                   const int32_t* n_accept, int32_t* seq_lens, int32_t* fill,
                                   uint16_t* k_stage, uint16_t* v_stage, int B_cache,
                                   int32_t* sync, const int32_t* block_table, int max_pages,
                                   uint16_t* k_pool, uint16_t* v_pool, int num_pages,
                                   int32_t* commit_slots, int batch, int B, int hkv, int d,
                                   int32_t* status, cudaStream_t stream);

// ---- Decode attention: split-KV partials then a combine pass.
struct DecodePlan {
  int split_len;   // keys per split (multiple of 128)
  int nsplit;      // splits per (sequence, kv head)
  int rows;        // query rows per (sequence, kv head) = (hq / hkv) * B
  bool ordered;    // CTAs take the sequences longest first (order array in the workspace)
  size_t order_bytes;
  size_t ws_bytes;
};
DecodePlan plan_decode(int batch, int B, int hq, int hkv, int d, int max_len);

cudaError_t launch_decode_attn(const uint16_t* q, const uint16_t* k_blk,
                               const uint16_t* v_blk, const uint16_t* k_pool,
                               const uint16_t* v_pool, int num_pages,
                               const int32_t* block_table, int max_pages,
                               const int32_t* seq_lens, const DecodePlan& plan, float* o,
                               int batch, int B, int hq, int hkv, int d, float scale,
                               void* workspace, int32_t* status, cudaStream_t stream,
                               const uint16_t* k_stage = nullptr,
                               const uint16_t* v_stage = nullptr,
                               const int32_t* stage_fill = nullptr, int B_cache = 0);

// ---- LM head + max-prob/argmax + acceptance.
size_t head_workspace_bytes(int batch, int B, int vocab);
// taus: one threshold per sequence (device, [batch]), or NULL to use tau for all.
cudaError_t launch_head_accept(const uint16_t* h, const uint16_t* w, int batch, int B,
                               int hidden, int vocab, float tau, const float* taus,
                               int32_t* tokens, float* maxprob, int32_t* n_accept,
                               void* workspace, int32_t* status, cudaStream_t stream);

// ---- Gradient of the dual-stream attention: a statistics-only forward run, then the
// tcgen05 dK/dV kernel over key tiles and the row-parallel tcgen05 dQ kernel.
size_t dual_grad_workspace_bytes(int batch, int L, int B, int hq, int hkv, int d);
cudaError_t launch_dual_stream_grad(const uint16_t* q, const uint16_t* k, const uint16_t* v,
                                    const float* o, const float* d_o, int batch, int L, int B,
                                    int hq, int hkv, int d, float scale, float* dq, float* dk,
                                    float* dv, void* workspace, int32_t* status,
                                    cudaStream_t stream, const float* lse = nullptr);

// ---- Dual-stream training loss (L_mask + L_AR) over the 2L rows of each sequence.
size_t ce_workspace_bytes(int batch, int L, int vocab);
cudaError_t launch_ce_loss(const uint16_t* h, const uint16_t* w, const int32_t* targets,
                           int batch, int L, int hidden, int vocab, float* loss,
                           float* row_ce, float* row_lse, void* workspace, int32_t* status,
                           cudaStream_t stream);
size_t ce_grad_workspace_bytes(int batch, int L, int vocab);
cudaError_t launch_ce_loss_grad(const uint16_t* h, const uint16_t* w, const int32_t* targets,
                                const float* row_lse, int batch, int L, int hidden, int vocab,
                                float* dh, float* dw, void* workspace, int32_t* status,
                                cudaStream_t stream);

// Streaming multiprocessors of the current device (cached per device).
int num_sms();

// Function attributes belong to the device they were set on: raise a kernel's dynamic
// shared-memory limit once per device (flags indexed by device ordinal).
template <class Kernel>
cudaError_t set_smem_limit_once(Kernel* fn, int bytes, std::atomic<int> (&done)[64]) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 0 && dev < 64 && done[dev].load(std::memory_order_acquire)) return cudaSuccess;
  e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && dev >= 0 && dev < 64) done[dev].store(1, std::memory_order_release);
  return e;
}

// Launch of a kernel that calls wait_for_previous (sm100.cuh) before all else that touches memory.
template <class... Params, class... Args>
cudaError_t launch_early(void (*fn)(Params...), dim3 grid, unsigned threads, size_t smem,
                         cudaStream_t stream, const Args&... args) {
  cudaLaunchAttribute early{};
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t c{};
  c.gridDim = grid;
  c.blockDim = dim3(threads);
  c.dynamicSmemBytes = smem;
  c.stream = stream;
  c.attrs = &early;
  c.numAttrs = 1;
  return cudaLaunchKernelEx(&c, fn, Params(args)...);
}

// ---- One CTA waiting on an mbarrier that nothing completes (the wait-limit self-check).
cudaError_t launch_wait_timeout_check(int32_t* status, cudaStream_t stream);

// ---- Dual-stream attention under mask M. o may be null when lse is given (the row
// statistics alone: lse[b][h][stream][t], t < Lp = L rounded up to 128, = log2 of the
// softmax denominator in units of scale*log2(e)*score; pad rows are written as 0).
cudaError_t launch_dual_stream(const uint16_t* q, const uint16_t* k, const uint16_t* v,
                               float* o, int batch, int L, int B, int hq, int hkv, int d,
                               float scale, int32_t* status, cudaStream_t stream,
                               float* lse = nullptr);

// dQ of the dual-stream attention gradient from the forward's row statistics: lse and
// D = rowsum(dO * O) as [b][hq][2][Lp] fp32, dO in bf16 like q. Writes every row of dq.
cudaError_t launch_dual_stream_dq(const uint16_t* q, const uint16_t* k, const uint16_t* v,
                                  const uint16_t* do_bf, const float* lse, const float* drow,
                                  float* dq, int batch, int L, int B, int hq, int hkv, int d,
                                  float scale, int32_t* status, cudaStream_t stream);

// ---- Packed sequences: causal attention, without a cache or after a paged prefix.
struct PackedAttn {
  const uint16_t *q, *k, *v;            // [total][heads][d], row pitches in elements
  long long q_stride, k_stride, v_stride;
  const int32_t* cu;                    // [batch + 1]
  const uint16_t *k_pool, *v_pool;      // with a cache
  const int32_t *block_table, *seq_lens;   // seq_lens NULL: no cache
  int num_pages, max_pages;
  uint16_t* o;                          // [total][hq][d] bf16
  float* lse;                           // [hq][total] or NULL
  int batch, total, hq, hkv, d;
  float scale;
  int32_t* status;
};
struct PackedPlan {
  bool pair;               // persistent CTAs over equal parts of the work
  int rows;                // tokens of an item (pair)
  bool can_split;          // items may be divided among CTAs (pair)
  size_t ticket_bytes;
  int gp, tpt;             // heads and tokens of a row tile
  int nsplit, split_tiles; // splits of a key list, 128-key tiles per split
  long long items, ctas;
  size_t ws_bytes;
};
// max_len: upper bound of a sequence's keys (cached and own) for which the splits are sized.
PackedPlan plan_packed(int batch, int total, int hq, int hkv, int d, int max_len);
cudaError_t launch_packed_attn(const PackedAttn& p, const PackedPlan& plan, void* workspace,
                               cudaStream_t stream);

// ---- Gradient of the packed attention without a cache.
struct PackedGrad {
  const uint16_t *q, *k, *v, *o, *d_o;
  long long q_stride, k_stride, v_stride, dq_stride, dk_stride, dv_stride;
  const float* lse;
  const int32_t* cu;
  uint16_t *dq, *dk, *dv;
  int batch, total, hq, hkv, d;
  float scale;
  int32_t* status;
};
// The largest count of items or CTAs, which are 32-bit numbers.
long long packed_grad_items(int batch, int total, int hq);
size_t packed_grad_workspace_bytes(int batch, int total, int hq, int hkv, int d);
cudaError_t launch_packed_grad(const PackedGrad& p, void* workspace, cudaStream_t stream);

// ---- K/V rows of packed sequences into the paged cache.
cudaError_t launch_kv_append(const uint16_t* k, const uint16_t* v, long long k_stride,
                             long long v_stride, const int32_t* cu, const int32_t* seq_lens,
                             int32_t* new_lens, const int32_t* block_table, int max_pages,
                             uint16_t* k_pool, uint16_t* v_pool, int num_pages, int32_t* slots,
                             int batch, int total, int hkv, int d, int32_t* status,
                             cudaStream_t stream);

// ---- Rotary positions of packed rows.
struct Rotary {
  const uint16_t *q, *k;
  uint16_t *q_out, *k_out;
  long long q_stride, k_stride, qo_stride, ko_stride;
  const int32_t *cu, *seq_lens;         // seq_lens NULL: all 0
  const float* inv_freq;                // [rot / 2]
  int batch, total, hq, hkv, d, rot;
  float factor;
  bool inverse, in_place;               // in place: what is not rotated is not copied
  int32_t* status;
};
long long rotary_ctas(int batch, int total);
cudaError_t launch_rotary(const Rotary& a, bool interleaved, cudaStream_t stream);

// ---- K/V rows of packed sequences into the 8-bit paged cache.
struct AppendQ8 {
  const uint16_t *k, *v;
  long long k_stride, v_stride;
  const int32_t *cu, *seq_lens, *counts, *block_table;
  int32_t *new_lens, *slots, *status;
  uint8_t *k_pool, *v_pool, *k_scale, *v_scale;
  int num_pages, max_pages, batch, total, hkv;
};
long long append_q8_ctas(int batch, int total);
cudaError_t launch_kv_append_q8(const AppendQ8& a, int d, cudaStream_t stream);

// ---- Attention of new tokens over the 8-bit paged cache.
struct ChunkQ8 {
  PackedAttn attn;                      // its pools stay NULL
  const uint8_t *k_pool, *v_pool, *k_scale, *v_scale;
};
struct ChunkQ8Plan {
  int gp, tpt;             // heads and tokens of a row tile
  int ctas;
  bool can_split;          // items may be divided among CTAs
  int few;                 // rows of an item of chunk_q8_few.cu's kernel (0: not that)
  int pages;               // the wide form's pages per sequence (0: without it)
  long long tiles;         // of own rows and pages that come before the attention
  PackedPlan wide;
  size_t least, ws_bytes;  // what has to be there; what the call makes use of
};
// ws_bytes: what there is for the wide form's pages and all else.
ChunkQ8Plan plan_chunk_q8(int batch, int total, int hq, int hkv, int d, int max_len, size_t ws_bytes = SIZE_MAX);
cudaError_t launch_chunk_q8(const ChunkQ8& p, const ChunkQ8Plan& plan, void* workspace,
                            cudaStream_t stream);

}  // namespace mars
