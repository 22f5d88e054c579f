// What the kernels of the attention over the 8-bit paged cache share: the line of items that their
// CTAs divide evenly, and the join of divided items.
//
// An item is a tile of (token, query head) rows of one sequence that share a KV head, with the 128-key
// tiles that its rows see: the sequence's own keys first, then the cached ones. The items of all
// sequences are laid out on a line, each as long as its work; CTA c of E takes the part from c/E to
// (c + 1)/E of it. A cut inside an item leaves partials (m', l, O), which are joined in the order of the keys:
// by merge_kernel, or in chunk_q8_few.cu by the CTA that is the last to leave one.
//
// With V = 2^e c (a scale and a code), a weight's power goes the other way: P' = 2^(s + e - m') is what
// multiplies the codes, m' the running maximum of s + e instead of s, and the row sum takes P' 2^-e. P' is
// then as large as what it contributes, whatever the pages' scales are, and in f16, which holds every code
// exactly (bf16 would too, but takes five instructions for what one conversion does), 2^7 P' keeps the
// bits of small ones.
#pragma once

#include <cuda.h>

#include <climits>

#include "cache_q8.cuh"
#include "flash_tc.cuh"
#include "internal.h"
#include "packed.cuh"

namespace mars {
namespace q8 {

constexpr int kTile = 128;           // keys of a tile
constexpr int kPagesPerTile = kTile / kPageSize;
constexpr long long kUnit = 8;       // work of a key tile
constexpr int kMinPart = 2;          // key tiles of a part of a divided item
// Work of an item's start and end, in chunk_q8.cu (8 positions, 28 query over 4 KV heads, 32 sequences of
// 512 .. 2,048 keys: 40.2 us at 4, 39.4 at 24, 41.9 at 48, 44.7 at 64; 16 positions, 128 sequences of
// 2,048 .. 8,192: 256, 246, 244, 247) and in chunk_q8_few.cu (single tokens, 32 sequences of 2,048 .. 8,192:
// 45.6 at 12, 42.7 at 32, 41.5 at 64, 41.6 at 80)
constexpr int kItemWork = 24, kFewItemWork = 64;
constexpr float kLift = 7.f;         // log2 of what P' is multiplied by
constexpr float kNoKeys = -1.f;      // l of a part without keys, which has no O

// float4 of a partial: D / 4 columns of an item's kRows rows, then m' and l of each.
template <int D, int kRows>
constexpr int kPartial = kRows * D / 4 + kRows / 2;

// Largest finite magnitude, as bf16 bits, of the halves of a word and `top`, in both halves.
MARS_DEV uint32_t finite_max(uint32_t top, uint32_t word) {
  const uint32_t m = word & 0x7fff7fffu;
  return __vmaxu2(top, m & ~__vcmpgeu2(m, 0x7f807f80u));
}

// Rows in f16 stand over a power of two that brings their largest finite magnitude into [2^kTop,
// 2^(kTop + 1)).
constexpr int kTop = 14;
// Own values from 2^88 on count as the largest bf16 below (infinities and NaN stay), so that their powers
// end at 2^73. P' = 2^(s + e - m' + 7) with m' at most that of the largest weight times 2^73; a key over
// the smallest scale, 2^-40, then keeps its part of the row sum, P' 2^40, while its weight is above 2^-20 of
// the largest: below that P' leaves the range of 32 bits. (Without a cap that began at weights as large as
// any, and f16 values beyond the range became infinite, NaN with the weight 0 of a row that does not see them.)
constexpr uint32_t kMostValue = 0x6b7f;            // bf16
MARS_DEV uint32_t cap_values(uint32_t word) {
  const uint32_t m = word & 0x7fff7fffu, most = kMostValue << 16 | kMostValue;
  const uint32_t beyond = __vcmpgtu2(m, most) & ~__vcmpgeu2(m, 0x7f807f80u) & 0x7fff7fffu;
  return (word & ~beyond) | (most & beyond);
}
MARS_DEV uint4 cap_values(const uint4& x) {
  return make_uint4(cap_values(x.x), cap_values(x.y), cap_values(x.z), cap_values(x.w));
}

// Wait of one thread for the phase with `parity`. Gives up (false) after 2^20 attempts of a
// microsecond at most.
MARS_DEV bool wait_bounded(uint64_t* b, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .u32 n;\n\t"
      "mov.u32 n, 0;\n\t"
      "TRY:\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, 1000;\n\t"
      "@p bra DONE;\n\t"
      "add.u32 n, n, 1;\n\t"
      "setp.lt.u32 p, n, 1048576;\n\t"
      "@p bra TRY;\n\t"
      "setp.ne.u32 p, n, n;\n\t"
      "DONE:\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(sm100::smem_u32(b)), "r"(parity)
      : "memory");
  return ok != 0;
}

// ---------------------------------------------------------------------------- the line of items

struct Args {
  const uint16_t *q, *k, *v;
  long long q_stride, k_stride, v_stride;
  const int32_t *cu, *seq_lens, *block_table;
  const uint8_t *k_pool, *v_pool, *k_scale, *v_scale;
  int num_pages, max_pages, batch, total, hq, hkv, gp, tpt, heads;   // heads: KV heads x groups
  bool can_split;
  int item_work;                     // work of an item's start and end
  int skip_pages;                    // sequences of more than tpt rows and at most so many pages
                                     // are left to the wide form (-1: none)
  float scale_log2;
  uint16_t* o;
  // for chunk_q8.cu, what its first kernel makes: scale bytes of Q's rows, of groups of 16 own rows, and of
  // the rows of those that share none
  const uint8_t *q_byte, *own_k_byte, *own_v_byte, *own_k_bytes, *own_v_bytes;
  int own_groups;
  struct Record* rec;                // [CTA], for merge_kernel
  uint32_t* arrived;                 // [CTA], parts of the item that it begins (chunk_q8_few.cu)
  float4* part;                      // [CTA][2], see kPartial
  int32_t* status;
};

// What merge_kernel needs of a CTA: the item that it begins and does not end, if any, and whether
// all of its part lies inside an item that goes on in the next CTA.
struct Record {
  int begins, inside, base, tok0, tokens, h0, pad[2];
};

struct Row {
  int s, base, n, P;
  long long pre;                     // work before the sequence
  MARS_DEV int own() const { return (n + kTile - 1) / kTile; }
  // own and cached tiles of every item of the sequence (an item's own tiles behind its last
  // token, which it skips, counted too)
  MARS_DEV int tiles() const { return own() + packed::key_tiles(P); }
  MARS_DEV long long unit(const Args& a) const { return kUnit * tiles() + a.item_work; }
};

// Number of the first group of 16 of a sequence's own rows, among those of all sequences.
MARS_DEV int own_group(int base, int s) { return base / kPageSize + s; }
inline long long own_groups(int batch, int total) { return (long long)total / kPageSize + batch; }

MARS_DEV bool left_out(int skip_pages, int tpt, int n, int P) {
  return n > tpt && P / kPageSize + (P % kPageSize != 0) <= skip_pages;
}
MARS_DEV int cached(const Args& a, int len) {
  return (int)max(0LL, min((long long)len, (long long)a.max_pages * kPageSize));
}
MARS_DEV int items_of(const Args& a, const Row& q) {
  if (q.n <= 0 || left_out(a.skip_pages, a.tpt, q.n, q.P)) return 0;
  return (q.n + a.tpt - 1) / a.tpt * a.heads;
}

template <int kThreads>
struct Scan {
  long long sum[kThreads / 32], count[kThreads / 32];
  int top[kThreads / 32];
  Row at[2];
  long long total, ctas, p0, p1;
};

// Every thread of the CTA: the work of all, how many CTAs share it, and the sequences where this
// CTA's part begins and ends. A thread takes ceil(batch / threads) sequences.
template <int kThreads>
MARS_DEV void find_part(const Args& a, Scan<kThreads>& sc) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = a.batch / kThreads + (a.batch % kThreads != 0);
  const int lo = (int)min((long long)tid * per, (long long)a.batch), hi = min(lo + per, a.batch);
  auto clamped = [&](int s) { return min(max(a.cu[s], 0), a.total); };
  int bad = 0, m = 0;
  // the first sequence's, read at once: each trip to memory before the first copy is time lost
  const int first_end = lo < hi ? a.cu[lo + 1] : 0, first_len = lo < hi ? a.seq_lens[lo] : 0;
  const int zeroth = a.cu[0];
  for (int s = lo; s < hi; ++s) m = max(m, s == lo ? min(max(first_end, 0), a.total) : clamped(s + 1));
#pragma unroll 1
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, m, o);
    if (lane >= o) m = max(m, v);
  }
  if (lane == 31) sc.top[warp] = m;
  __syncthreads();
  int lead = min(max(zeroth, 0), a.total);           // the boundary before this thread's sequences
  if (tid == 0 && lead != zeroth) bad = MARS_ST_BADSEQ;
  for (int w = 0; w < warp; ++w) lead = max(lead, sc.top[w]);
  m = __shfl_up_sync(0xffffffffu, m, 1);
  if (lane > 0) lead = max(lead, m);
  // pass 0 sums up, pass 1 finds the sequences of the ends
  long long mine = 0, pre = 0, p0 = -1, p1 = -1;
#pragma unroll 1
  for (int pass = 0; pass < 2; ++pass) {
    long long count = 0;
    Row q{};
    q.base = lead;
    q.pre = pre;
#pragma unroll 1
    for (int s = lo; s < hi; ++s) {
      const int given = s == lo ? first_end : a.cu[s + 1], len = s == lo ? first_len : a.seq_lens[s];
      const int end = max(min(max(given, 0), a.total), q.base);
      q.s = s;
      q.n = end - q.base;
      q.P = cached(a, len);
      if (end != given) bad |= MARS_ST_BADSEQ;
      if (q.P != len && q.n > 0) bad |= MARS_ST_OVERFLOW;
      const int items = items_of(a, q);
      const long long work = items * q.unit(a);
      if (p0 >= q.pre && p0 < q.pre + work) sc.at[0] = q;
      if (p1 >= q.pre && p1 < q.pre + work) sc.at[1] = q;
      count += items;
      q.pre += work;
      q.base = end;
    }
    if (pass) break;
    mine = q.pre;
    long long incl = mine, sum = count;
#pragma unroll 1
    for (int o = 1; o < 32; o <<= 1) {
      const long long v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
      sum += __shfl_xor_sync(0xffffffffu, sum, o);
    }
    if (lane == 31) {
      sc.sum[warp] = incl;
      sc.count[warp] = sum;
    }
    __syncthreads();
    pre = incl - mine;
    long long total = 0, items = 0;
#pragma unroll 1
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < warp) pre += sc.sum[w];
      total += sc.sum[w];
      items += sc.count[w];
    }
    // as many CTAs as there are, unless that leaves less than a part each and there are fewer items
    const long long ctas =
        min((long long)gridDim.x, max(items, total / (kUnit * kMinPart + a.item_work)));
    if (tid == 0) {
      sc.total = total;
      sc.ctas = ctas;
    }
    if ((long long)blockIdx.x >= ctas) break;
    const int n = (int)ctas;
    const long long share = total / n;
    const int rest = (int)(total - share * n);       // cuts at floor(x total / n)
    p0 = blockIdx.x * share + blockIdx.x * rest / n;
    p1 = (blockIdx.x + 1) * share + (blockIdx.x + 1) * rest / n;
    if (tid == 0) {
      sc.p0 = p0;
      sc.p1 = p1;
    }
  }
  if (bad && blockIdx.x == 0 && a.status) atomicOr(a.status, bad);
  __syncthreads();
}

// Item i of the sequence and its tile j at which position `pos` of the line cuts; not within
// kMinPart tiles of an item's ends.
MARS_DEV void cut_at(const Args& a, const Row& q, long long pos, int& i, int& j) {
  const long long rem = pos - q.pre;
  i = (int)(rem / q.unit(a));
  const int tiles = q.tiles();
  j = (int)min(max((rem - i * q.unit(a) - a.item_work / 2) / kUnit, 0LL), (long long)tiles);
  const int least = a.can_split ? kMinPart : tiles / 2;
  if (j < least || !a.can_split) {
    const bool up = j >= least && j > 0;
    i += up;
    j = 0;
  } else if (tiles - j < kMinPart) {
    ++i;
    j = 0;
  }
}

// Sequences one after another, 32 of them read at once. Whole warp.
struct Window {
  const Args& a;
  int s0, begin, end, len;           // first sequence; this lane's
  MARS_DEV explicit Window(const Args& a_) : a(a_), s0(INT_MIN / 2), begin(0), end(0), len(0) {}
  MARS_DEV void load(int s, int base) {
    const int lane = threadIdx.x & 31;
    s0 = s;
    const int mine = s + lane;
    end = mine < a.batch ? min(max(a.cu[mine + 1], 0), a.total) : 0;
    len = mine < a.batch ? a.seq_lens[mine] : 0;
    end = max(end, base);
#pragma unroll 1
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, end, o);
      if (lane >= o) end = max(end, v);
    }
    begin = __shfl_up_sync(0xffffffffu, end, 1);
    if (lane == 0) begin = base;
  }
  // the sequence after q, which is not the last one
  MARS_DEV Row after(const Row& q) {
    const int s = q.s + 1;
    if (s >= s0 + 32) load(s, q.base + q.n);
    const int l = s - s0;
    Row r{};
    r.s = s;
    r.base = __shfl_sync(0xffffffffu, begin, l);
    r.n = __shfl_sync(0xffffffffu, end, l) - r.base;
    r.P = cached(a, __shfl_sync(0xffffffffu, len, l));
    return r;
  }
};

// Factor of a row's O. l is 0 where every score is -infinity (O is then 0), NaN where one is NaN or
// +infinity.
MARS_DEV float reciprocal(float l) { return l == 0.f ? 0.f : 1.f / l; }

// Joins the parts of a divided item, the k-th of which is at part(k): four columns of a row at a time.
template <int D, int kRows, int kAtOnce, class Part>
MARS_DEV void join(const Args& a, Part part, int parts, int rows, size_t tok, int h0, int from, int step) {
  for (int i = from; i < rows * (D / 4); i += step) {
    const int row = i % rows, c = i / rows;
    float m = -INFINITY, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    // kAtOnce at a time: a trip to the L2 cache each
#pragma unroll 1
    for (int k0 = 0; k0 < parts; k0 += kAtOnce) {
      float2 ml[kAtOnce];
      float4 v[kAtOnce];
      float top = m;
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k) {
        ml[k] = make_float2(-INFINITY, kNoKeys);
        v[k] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (k0 + k >= parts) continue;
        ml[k] = __ldcg(reinterpret_cast<const float2*>(part(k0 + k) + kRows * D / 4) + row);
        v[k] = __ldcg(part(k0 + k) + c * kRows + row);
      }
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k) top = fmaxf(top, ml[k].x);
      const float w0 = m > -INFINITY ? exp2f(m - top) : 0.f;        // (+infinity gives NaN)
      m = top;
      l *= w0;
      o = make_float4(o.x * w0, o.y * w0, o.z * w0, o.w * w0);
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k) {
        if (ml[k].y == kNoKeys) continue;
        const float w = ml[k].x > -INFINITY ? exp2f(ml[k].x - top) : 0.f;
        l = fmaf(ml[k].y, w, l);
        o = make_float4(fmaf(v[k].x, w, o.x), fmaf(v[k].y, w, o.y), fmaf(v[k].z, w, o.z), fmaf(v[k].w, w, o.w));
      }
    }
    const float inv = reciprocal(l);
    *reinterpret_cast<uint2*>(a.o + ((tok + row / a.gp) * a.hq + h0 + row % a.gp) * D + 4 * c) =
        make_uint2(flash::pack_bf16x2(o.x * inv, o.y * inv), flash::pack_bf16x2(o.z * inv, o.w * inv));
  }
}

// Joins the parts of divided items. Block (x, y): the item that CTA x begins and does not end, a
// thread per (row, four columns).
template <int D, int kRows>
__global__ void __launch_bounds__(256, 6) merge_kernel(Args a, int ctas) {
  constexpr int PART = kPartial<D, kRows>;
  sm100::wait_for_previous();
  const int x = blockIdx.x, lane = threadIdx.x & 31;
  const Record rec = a.rec[x];
  if (!rec.begins) return;
  // its parts: CTA x's, those that lie inside it, and the one that ends it
  int parts = 2;
  for (int c = x + 1;; c += 32) {
    const bool inside = c + lane < ctas && a.rec[c + lane].inside;
    const uint32_t out = __ballot_sync(0xffffffffu, !inside);
    parts += out ? __ffs(out) - 1 : 32;
    if (out) break;
  }
  const float4* first = a.part + ((size_t)x * 2 + 1) * PART;
  auto part = [&](int k) { return k == 0 ? first : a.part + (size_t)(x + k) * 2 * PART; };
  join<D, kRows, 2>(a, part, parts, rec.tokens * a.gp, (size_t)rec.base + rec.tok0, rec.h0,
                 blockIdx.y * 256 + threadIdx.x, gridDim.y * 256);
}

}  // namespace q8

// chunk_q8_few.cu, for items of kRows rows, 8 or 16; k and v map the pools, a page of a KV head as a box.
template <int D, int kRows>
cudaError_t launch_chunk_q8_few(const q8::Args& a, int ctas, const CUtensorMap& k, const CUtensorMap& v,
                                cudaStream_t stream);

}  // namespace mars
