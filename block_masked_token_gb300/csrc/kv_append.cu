// Append of the K/V rows of packed sequences (a prompt, a chunk of one) to the paged cache:
// row i of sequence s goes to position seq_lens[s] + i, i.e. slot pos % 16 of page
// block_table[s][pos / 16]. An unmapped page ends the append of its sequence.
//
// A pure copy: 4 hkv d bytes read and written per row. 43 MB in all take 12 us, of which the chain
// of boundary, length, page and row loads is about 3 and the launch 2 (with the rows loaded before
// the pages are known, at the registers that takes, it is no faster). A CTA takes kRows rows of
// one sequence. It first finds the sequence's first unmapped page at or before its rows (a scan
// of the block-table row, which stays in L2), then copies with 16-byte vectors.
#include <climits>

#include "common.cuh"
#include "internal.h"
#include "packed.cuh"

namespace mars {

namespace {

constexpr int kRows = 16;
constexpr int kThreads = 256;
constexpr int kAhead = 4;

struct AppendArgs {
  const uint16_t *k, *v;
  long long k_stride, v_stride;
  const int32_t *cu, *seq_lens, *block_table;
  int32_t *new_lens, *slots, *status;
  uint16_t *k_pool, *v_pool;
  int num_pages, max_pages, batch, total, hkv, d;
};

__global__ void __launch_bounds__(kThreads) kv_append_kernel(AppendArgs a) {
  __shared__ int s_bad;                  // first logical page that is not mapped
  __shared__ int s_slot[kRows];
  bool bad;
  const packed::Seq sq =
      packed::find_tile(a.cu, a.batch, a.total, kRows, 1, (long long)blockIdx.x, bad, a.seq_lens);
  if (threadIdx.x == 0) {
    s_bad = INT_MAX;
    if (bad && a.status) atomicOr(a.status, MARS_ST_BADSEQ);
  }
  if (sq.s < 0) return;
  __syncthreads();
  const int r0 = sq.tile * kRows, nr = min(kRows, sq.n - r0);
  const long long P = sq.len;
  const int32_t* bt = a.block_table + (size_t)sq.s * a.max_pages;
  // pages of positions P .. P + r0 + nr - 1
  const long long first = P / kPageSize;
  const long long last = P < 0 || nr <= 0 ? -1 : (P + r0 + nr - 1) / kPageSize;
  for (long long lp = first + threadIdx.x; lp <= last; lp += kThreads) {
    const int e = lp < a.max_pages ? bt[lp] : -1;
    if (e < 0 || e >= a.num_pages) {
      atomicMin(&s_bad, (int)min(lp, (long long)INT_MAX - 1));
      break;
    }
  }
  __syncthreads();
  // rows of the sequence before the first position that cannot be written
  const long long stop = P < 0 ? 0 : s_bad == INT_MAX ? sq.n : max(0LL, (long long)s_bad * kPageSize - P);
  if (threadIdx.x == 0) {
    if (a.new_lens && r0 + kRows >= sq.n) a.new_lens[sq.s] = (int)(P + min(stop, (long long)sq.n));
    if (a.status && stop < r0 + nr)
      atomicOr(a.status, P < 0 || s_bad >= a.max_pages ? MARS_ST_OVERFLOW : MARS_ST_NOPAGE);
  }
  if (threadIdx.x < nr) {
    const long long pos = P + r0 + threadIdx.x;
    int slot = -1;
    if (r0 + (long long)threadIdx.x < stop)
      slot = bt[pos / kPageSize] * kPageSize + (int)(pos % kPageSize);
    s_slot[threadIdx.x] = slot;
    if (a.slots) a.slots[sq.base + r0 + threadIdx.x] = slot;
  }
  __syncthreads();
  const int n = (int)max(0LL, min((long long)nr, stop - r0));
  const int vph = a.d / 8, per = a.hkv * vph;       // 16-byte vectors per head row, per row
  // all loads of kAhead vectors of k and v before the stores: one after another they left an SM
  // with a few KB in flight, and 21.7 MB took 14 us
  for (int i0 = threadIdx.x; i0 < n * per; i0 += kAhead * kThreads) {
    uint4 xk[kAhead], xv[kAhead];
    size_t dst[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int i = min(i0 + u * kThreads, n * per - 1);
      const int r = i / per, rem = i - r * per, h = rem / vph, c = rem - h * vph;
      const size_t row = (size_t)sq.base + r0 + r;
      const int gs = s_slot[r];
      dst[u] = (((size_t)(gs / kPageSize) * a.hkv + h) * kPageSize + gs % kPageSize) * a.d +
               (size_t)c * 8;
      xk[u] = *reinterpret_cast<const uint4*>(a.k + row * a.k_stride + rem * 8);
      xv[u] = *reinterpret_cast<const uint4*>(a.v + row * a.v_stride + rem * 8);
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
      if (i0 + u * kThreads < n * per) {
        *reinterpret_cast<uint4*>(a.k_pool + dst[u]) = xk[u];
        *reinterpret_cast<uint4*>(a.v_pool + dst[u]) = xv[u];
      }
  }
}

}  // namespace

cudaError_t launch_kv_append(const uint16_t* k, const uint16_t* v, long long k_stride,
                             long long v_stride, const int32_t* cu, const int32_t* seq_lens,
                             int32_t* new_lens, const int32_t* block_table, int max_pages,
                             uint16_t* k_pool, uint16_t* v_pool, int num_pages, int32_t* slots,
                             int batch, int total, int hkv, int d, int32_t* status,
                             cudaStream_t stream) {
  AppendArgs a{k,        v,     k_stride, v_stride, cu,        seq_lens,  block_table,
               new_lens, slots, status,   k_pool,   v_pool,    num_pages, max_pages,
               batch,    total, hkv,      d};
  const long long ctas = packed::max_tiles(batch, total, kRows);
  kv_append_kernel<<<(unsigned)ctas, kThreads, 0, stream>>>(a);
  count_launches(1);
  return cudaGetLastError();
}

}  // namespace mars
