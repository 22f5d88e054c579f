// Append of the K/V rows of packed sequences to the 8-bit paged cache (cache_q8.cuh): row i of
// sequence s goes to position seq_lens[s] + i, as in kv_append.cu, as codes over the page's scale.
//
//   A page's scale is the smallest power of two under which its largest magnitude needs no code
//   beyond 448; a page that held tokens before keeps its scale unless the new rows need a larger
//   one, and then its old codes are formed again over that.
//
// A CTA takes one page of a sequence's new rows, a warp at a time one KV head of K or V there: it
// loads the rows, finds their largest magnitude and writes their codes, so that each element is
// read once. 2 bytes read and 1 written per element.
//
// Prompts of 9,055 rows of 4 heads of 128 (28 MB): 8.3 us, 0.49 of the copy bandwidth: the launch (2 us)
// and the chain of boundary, length, page and row reads (some 4) come before the first byte. It was
// 9.5 with the old codes read ahead of the scales (128 registers, two waves of CTAs; now one), 12.2
// when it did not start while the kernel before it ended. A few rows: 6.5 us, the host's and the launch's.
#include <climits>

#include "cache_q8.cuh"
#include "internal.h"
#include "packed.cuh"
#include "sm100.cuh"

namespace mars {

namespace {

constexpr int kThreads = 256;

// Rows of a sequence to append, and the pages that they fall on (at least one: it writes the new
// length, and the slots of rows that are not appended).
MARS_DEV int rows_of(const AppendQ8& a, int s, int n, int len) {
  if (len < 0) return 0;
  return a.counts ? min(max(a.counts[s], 0), n) : n;
}
MARS_DEV int pages_of(int rows, int len) {
  return rows > 0 ? (int)((len % kPageSize + (long long)rows + kPageSize - 1) / kPageSize) : 1;
}

template <int D>
MARS_DEV void append_head(const uint16_t* __restrict__ rows, long long stride, uint8_t* codes,
                          uint8_t* scale, int held, int end) {
  constexpr int kChunks = D / 8, kStep = 32 / kChunks, kIts = kPageSize / kStep;
  const int lane = threadIdx.x & 31, c = lane % kChunks, r0 = lane / kChunks;
  // slots [held, end) get rows[0 ..], slots below held keep their tokens
  uint4 x[kIts];
  // lane 0 alone reads and writes the scale
  int byte0 = lane == 0 && held > 0 ? q8::scale_byte(*scale) : q8::kLeast;
#pragma unroll
  for (int i = 0; i < kIts; ++i) {
    const int slot = r0 + i * kStep;
    x[i] = make_uint4(0, 0, 0, 0);
    if (slot >= held && slot < end)
      x[i] = *reinterpret_cast<const uint4*>(rows + (long long)(slot - held) * stride + c * 8);
  }
  uint32_t top = 0, endless = 0;                 // largest finite magnitude, in each half; infinities, NaN
#pragma unroll
  for (int i = 0; i < kIts; ++i) {
    const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t m = w[e] & 0x7fff7fffu, no = __vcmpgeu2(m, 0x7f807f80u);
      top = __vmaxu2(top, m & ~no);
      endless |= no;
    }
  }
  byte0 = __shfl_sync(0xffffffffu, byte0, 0);
  top = __reduce_max_sync(0xffffffffu, max(top >> 16, top & 0xffffu));
  const int byte = max(byte0, top ? q8::scale_for(top) : q8::kLeast);
  if (lane == 0) *scale = (uint8_t)byte;
  const float f = q8::inverse_power(byte);
  const float g = q8::power(q8::kBias - (byte - byte0));
#pragma unroll
  for (int i = 0; i < kIts; ++i) {
    const int slot = r0 + i * kStep;
    float e[8];
    if (slot >= held && slot < end) {
      unpack8(x[i], e);
      if (endless) {                             // an infinity becomes NaN, which stays
#pragma unroll
        for (int k = 0; k < 8; ++k) e[k] = fmaf(e[k], 0.f, e[k]);
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) e[k] *= f;
    } else if (slot < held && byte > byte0) {
      const uint2 old = *reinterpret_cast<const uint2*>(codes + slot * D + c * 8);
      const uint32_t w[2] = {old.x, old.y};
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        uint32_t lo, hi;
        q8::decode4(w[k], lo, hi);
        const float2 a = q8::halves(lo), b = q8::halves(hi);
        e[4 * k] = a.x * g;
        e[4 * k + 1] = a.y * g;
        e[4 * k + 2] = b.x * g;
        e[4 * k + 3] = b.y * g;
      }
    } else {
      continue;
    }
    *reinterpret_cast<uint2*>(codes + slot * D + c * 8) =
        make_uint2(q8::encode2(e[0], e[1]) | (q8::encode2(e[2], e[3]) << 16),
                   q8::encode2(e[4], e[5]) | (q8::encode2(e[6], e[7]) << 16));
  }
}

template <int D>
__global__ void __launch_bounds__(kThreads, 4) kv_append_q8_kernel(AppendQ8 a) {
  __shared__ int s_bad;                  // first logical page that is not mapped
  bool bad;
  sm100::let_next_start();
  sm100::wait_for_previous();
  const packed::Seq sq = packed::find_tile_by(
      a.cu, a.batch, a.total, (long long)blockIdx.x, bad, a.seq_lens,
      [&](int s, int n, int len) { return pages_of(rows_of(a, s, n, len), len); });
  if (threadIdx.x == 0) {
    s_bad = INT_MAX;
    if (bad && a.status) atomicOr(a.status, MARS_ST_BADSEQ);
  }
  if (sq.s < 0) return;
  __syncthreads();
  const long long P = sq.len;
  const int n = rows_of(a, sq.s, sq.n, sq.len);
  const int32_t* bt = a.block_table + (size_t)sq.s * a.max_pages;
  const long long first = P / kPageSize, lp = first + sq.tile;
  const bool last = sq.tile == pages_of(n, sq.len) - 1;
  for (long long p = first + threadIdx.x; n > 0 && p <= lp; p += kThreads) {
    const int e = p < a.max_pages ? bt[p] : -1;
    if (e < 0 || e >= a.num_pages) {
      atomicMin(&s_bad, (int)min(p, (long long)INT_MAX - 1));
      break;
    }
  }
  __syncthreads();
  // rows [i0, i1) of the sequence fall on this page; those before `stop` can be written
  const long long i0 = n > 0 ? max(0LL, lp * kPageSize - P) : 0;
  const long long i1 = min((long long)n, (lp + 1) * kPageSize - P);
  const bool mapped = n > 0 && s_bad == INT_MAX;
  const long long stop = s_bad == INT_MAX ? n : max(0LL, (long long)s_bad * kPageSize - P);
  if (threadIdx.x == 0) {
    if (a.new_lens && last) a.new_lens[sq.s] = (int)(P + min(stop, (long long)n));
    if (a.status && ((P < 0 && sq.n > 0) || (n > 0 && !mapped)))
      atomicOr(a.status, P < 0 || s_bad >= a.max_pages ? MARS_ST_OVERFLOW : MARS_ST_NOPAGE);
  }
  const int page = mapped ? bt[lp] : 0;
  if (a.slots) {
    // the last page's CTA also marks the rows that are not to be appended
    const long long end = last ? sq.n : i1;
    for (long long i = i0 + threadIdx.x; i < end; i += kThreads)
      a.slots[sq.base + i] =
          mapped && i < i1 ? page * kPageSize + (int)((P + i) % kPageSize) : -1;
  }
  if (!mapped) return;
  const int held = sq.tile == 0 ? (int)(P % kPageSize) : 0;
  const int end = (int)(P + i1 - lp * kPageSize);
  for (int w = threadIdx.x >> 5; w < 2 * a.hkv; w += kThreads / 32) {
    const bool is_v = w >= a.hkv;
    const int h = is_v ? w - a.hkv : w;
    const size_t at = (size_t)page * a.hkv + h;
    const long long stride = is_v ? a.v_stride : a.k_stride;
    append_head<D>((is_v ? a.v : a.k) + ((size_t)sq.base + i0) * stride + h * D, stride,
                   (is_v ? a.v_pool : a.k_pool) + at * (kPageSize * D),
                   (is_v ? a.v_scale : a.k_scale) + at, held, end);
  }
}

}  // namespace

// Rows over at most two more pages than they fill, and a page of each sequence.
long long append_q8_ctas(int batch, int total) { return (long long)total / kPageSize + 2LL * batch; }

cudaError_t launch_kv_append_q8(const AppendQ8& a, int d, cudaStream_t stream) {
  const unsigned ctas = (unsigned)append_q8_ctas(a.batch, a.total);
  count_launches(1);
  return launch_early(d == 64 ? kv_append_q8_kernel<64> : kv_append_q8_kernel<128>, ctas, kThreads, 0, stream, a);
}

}  // namespace mars
