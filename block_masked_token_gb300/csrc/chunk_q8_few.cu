// Attention over the 8-bit paged cache for few rows: single tokens, and blocks whose (token, query
// head) rows of a KV head are 16 at most (or more, where there is little to do: plan_chunk_q8).
//
// With so few rows the work is the reading of the cache: 2 D bytes per key and KV head against
// 4 * rows * D flops. chunk_q8.cu's roles and its 128-row tiles cost more there than the reading.
// Here a CTA's warps are alike and do not wait for each other: warp w takes pages w, w + kWarps, ..
// of the CTA's part of an item (chunk_q8.cuh), copies them by TMA through a ring of its own, and
// keeps its own running maximum, sum and O in registers, which the CTA joins at the part's end. A
// page is a step: S^T = K Q^T and O^T += V^T P^T by mma.sync, with 16 keys and 16 of d as its 16 rows
// and 8 rows of the item as its 8 columns. (The other way round half of each product would be empty
// for the 7 or 8 rows of a single token.) Codes are converted (e4m3 to f16, exactly) where they are
// used and never stored again, and one warp's conversion runs beside another's products. The order
// of d inside a product is free, and of O's rows too; both are taken so that a lane's operands are
// whole 16-byte reads of shared memory, without bank conflicts:
//   K: lane (g, t) = (lane / 4, lane % 4) of keys g and 8 + g holds d = t D/4 .. of them; four
//      consecutive d are its part of a step of 16.
//   V: lane (g, t) holds d = g D/8 .. of keys 2t, 2t + 1, 2t + 8, 2t + 9; byte permutations pair the
//      codes of two keys. Rows g and 8 + g of product j are then d = g D/8 + 2j and the next.
// A lane has the scores of keys g and 8 + g for rows 2t and 2t + 1; movmatrix turns the weights.
//
// Single tokens of 32 sequences of 2,048 .. 8,192 keys (28 query over 4 KV heads of 128): 42 us, 0.62 of
// the copy bandwidth (the first form, rows as the 16 rows of a product, 55.4; chunk_kernel 87.8). From
// 4,096 to 16,384 keys each it gains on them at 7 TB/s, the memory's rate; what is left is the launches
// (3 us), 6 us before the first copy (boundaries, the part, a page's entry, its scales, in turn) and
// some 5 at the end, where parts are joined and CTAs of two items come in later than those of one.
// 12 warps with a ring of 2 stages: 41.5, 8 with 4: 46.8, 16 with 2 (128 registers): 50. One token of
// one sequence: 7.7 us.
#include <algorithm>
#include <atomic>

#include "chunk_q8.cuh"

namespace mars {
namespace {

using namespace q8;

constexpr int kList = 32;            // parts found at a time

// A part of an item: which rows, which own keys and which cached pages.
struct Part {
  int s, base, tok0, tokens, h0, kvh, slot;
  int own0, own1, page0, page1, keys;               // keys: cached ones of the sequence
  long long cuts0, cuts1;                           // of a divided item: where its cuts lie
  // units of work: cached pages, then 16 own keys each
  MARS_DEV int pages() const { return page1 - page0; }
  MARS_DEV int units() const { return pages() + (own1 - own0 + kPageSize - 1) / kPageSize; }
};

// The parts of this CTA, one after another. Whole warp; where it is stays in shared memory.
struct Place {
  Row q;                             // at item i, tile j of it; before the end, items and tiles too
  int i, j, es, ei, ej;
  long long end_pre;                 // work before sequence es
  bool more;
};
template <int kThreads>
MARS_DEV Place first_place(const Args& a, const Scan<kThreads>& sc) {
  Place w{sc.at[0], 0, 0, a.batch, 0, 0, 0, true};
  if (sc.p1 < sc.total) {
    w.es = sc.at[1].s;
    w.end_pre = sc.at[1].pre;
    cut_at(a, sc.at[1], sc.p1, w.ei, w.ej);
  }
  cut_at(a, w.q, sc.p0, w.i, w.j);
  return w;
}
MARS_DEV bool next_part(const Args& a, Place& w, Window& window, Part& p) {
  if (!w.more) return false;
  Row& q = w.q;
  if (w.i >= items_of(a, q)) {
    w.i = w.j = 0;
    do {
      w.more = q.s + 1 < a.batch && q.s + 1 <= w.es;
      if (w.more) q = window.after(q);
    } while (w.more && items_of(a, q) == 0);
  }
  w.more = w.more && !(q.s > w.es || (q.s == w.es && (w.i > w.ei || (w.i == w.ei && w.j >= w.ej))));
  if (!w.more) return false;
  const int tiles = q.tiles(), jb = q.s == w.es && w.i == w.ei ? w.ej : tiles;
  const int hg = w.i % a.heads, last_tok = min((w.i / a.heads + 1) * a.tpt, q.n) - 1;
  p.s = q.s;
  p.base = q.base;
  p.tok0 = w.i / a.heads * a.tpt;
  p.tokens = last_tok + 1 - p.tok0;
  p.h0 = hg * a.gp;
  p.kvh = hg / (a.heads / a.hkv);
  p.slot = w.j > 0 ? 0 : jb < tiles ? 1 : -1;
  if (p.slot >= 0) {
    // a cut divides the item if it lies in [cuts0, cuts1) (cut_at)
    p.cuts0 = (w.j > 0 ? q.pre : w.end_pre) + w.i * q.unit(a) + a.item_work / 2 + kUnit * kMinPart;
    p.cuts1 = p.cuts0 + kUnit * (tiles - 2 * kMinPart + 1);
  }
  // own tiles [j, own), cached tiles from behind them
  const int own = q.own();
  p.own0 = min(min(w.j, own) * kTile, last_tok + 1);
  p.own1 = jb < own ? min(jb * kTile, last_tok + 1) : last_tok + 1;
  p.page0 = max(w.j - own, 0) * kPagesPerTile;
  p.keys = q.P;
  p.page1 = min(max(jb - own, 0) * kPagesPerTile, q.P / kPageSize + (q.P % kPageSize != 0));
  ++w.i;
  w.j = 0;
  return true;
}

template <int D, int kRows>
struct Shared {
  static constexpr int kWarps = kRows == 8 ? 12 : 8, kThreads = 32 * kWarps, kStages = kRows == 8 ? 2 : 4;
  static constexpr int kPage = kPageSize * D;
  static constexpr int kVec = kRows * D / 128;       // float4 of O per lane
  uint8_t ring[kWarps][kStages][2][kPage];           // codes of K and V
  float4 o[kWarps][kVec][32];
  float2 ml[kWarps][kRows];
  uint64_t full[kWarps][kStages];
  Part parts[kList];
  Place place;
  Scan<kThreads> scan;
  int first, pieces;                                // CTAs of the divided item in work
  int found, joins;
};

// 8 x 8 halves, two of a row to a lane, transposed.
MARS_DEV uint32_t transposed(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
// D += A B: 16 x 8, of depth 16, f16 operands.
MARS_DEV void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// bf16 rows as f16 (kTop): what f16 loses lies below 2^-39 of the largest magnitude.
MARS_DEV uint32_t word_max(const uint4& x, uint32_t top) {
  return finite_max(finite_max(finite_max(finite_max(top, x.x), x.y), x.z), x.w);
}
// The power's exponent, from `least` on, by the largest magnitude (either half of `top`).
MARS_DEV int row_exponent(uint32_t top, int least) {
  return max((int)(max(top >> 16, top & 0xffffu) >> 7) - kBias - kTop, least);
}
MARS_DEV uint32_t to_f16(uint32_t word, float f) {
  return pack_f16x2(__uint_as_float(word << 16) * f, __uint_as_float(word & 0xffff0000u) * f);
}
// A read that stays where it stands among the copies, and a read to come.
MARS_DEV uint4 load_once(const uint16_t* p) {
  uint4 x;
  asm volatile("ld.global.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w) : "l"(p));
  return x;
}
MARS_DEV void prefetch(const uint16_t* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }
// One more has arrived: what the CTA wrote before is there for whoever arrives later. Returns how many
// were there.
MARS_DEV uint32_t arrive(uint32_t* count) {
  uint32_t n;
  asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], 1;" : "=r"(n) : "l"(count) : "memory");
  return n;
}
constexpr int kLeastRow = -126;      // Q and K: 2^126 is the largest factor
constexpr int kLeastV = -40;         // V: as low as the pages' scales (and to 2^73: cap_values)

template <int D, int kRows>
__global__ void __launch_bounds__(Shared<D, kRows>::kThreads, 1)
few_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v, Args a) {
  using namespace sm100;
  using Sh = Shared<D, kRows>;
  constexpr int kWarps = Sh::kWarps, kStages = Sh::kStages;
  constexpr int kCols = kRows / 8, kSteps = D / 16;  // products next to each other; along d
  constexpr int kQuads = D / 32;                     // 16-byte reads of D/4 bf16
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  Sh& sh = *reinterpret_cast<Sh*>(smem_raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  if (smem_u32(smem_raw) % 1024) {                   // the ring's swizzle goes by address
    if (a.status) atomicOr(a.status, MARS_ST_TIMEOUT);
    return;
  }
  if (lane < kStages) mbar_init(&sh.full[warp][lane], 1);
  fence_barrier_init();
  if (threadIdx.x < 2) prefetch_tmap(threadIdx.x ? &tm_v : &tm_k);
  let_next_start();
  wait_for_previous();
  find_part(a, sh.scan);
  if ((long long)blockIdx.x >= sh.scan.ctas) return;
  if (threadIdx.x == 0) sh.place = first_place(a, sh.scan);
  uint64_t* full = sh.full[warp];
  bool ok = true;
  int flags = 0;
  uint32_t issued = 0, used = 0;                     // stages, counted on
  uint32_t meta = 0;                                 // of stage `lane`: scale bytes of K and V, and keys
  for (;;) {
    if (warp == 0) {
      __syncwarp();
      Place place = sh.place;
      Window window(a);
      Part p;
      int n = 0;
      while (n < kList && next_part(a, place, window, p)) {
        if (lane == 0) sh.parts[n] = p;
        ++n;
      }
      __syncwarp();
      if (lane == 0) {
        sh.place = place;
        sh.found = n;
      }
    }
    __syncthreads();
    const int found = sh.found;
    if (found == 0) break;
    // ---- the copies' place: page cu of part cp, and of the 32 pages 8 apart from `from` on this
    // lane's table entry and scale bytes
    int cp = -1, cu = 0, cend = 0, from = 0, entry = -1;
    uint32_t bytes = 0;
    int seq = 0, kvh = 0, keys = 0;
    auto issue = [&]() {
      while (cu >= cend) {
        if (cp + 1 >= found) return;
        const Part& p = sh.parts[++cp];
        cu = p.page0 + warp;
        cend = p.page1;
        from = INT_MIN;
        seq = p.s;
        kvh = p.kvh;
        keys = p.keys;
        // its rows, for when it begins: behind the copies in flight they would take 2 us
        const int row = lane >> 1, half = (lane & 1) * (D / 2);
        if (cp > 0 && row < p.tokens * a.gp)
          prefetch(a.q + ((size_t)p.base + p.tok0 + row / a.gp) * a.q_stride + (p.h0 + row % a.gp) * D + half);
        if (cp > 0 && p.own0 + row < p.own1) {
          const size_t key = (size_t)p.base + p.own0 + row;
          prefetch(a.k + key * a.k_stride + kvh * D + half);
          prefetch(a.v + key * a.v_stride + kvh * D + half);
        }
      }
      if (from == INT_MIN || cu >= from + 32 * kWarps) {
        from = cu;
        const int mine = cu + lane * kWarps;
        entry = mine < cend && mine >= cu ? a.block_table[(size_t)seq * a.max_pages + mine] : -1;
        const bool readable = entry >= 0 && entry < a.num_pages;
        if (mine < cend && mine >= cu && !readable) flags |= MARS_ST_NOPAGE;
        bytes = 0;
        if (readable) {
          const size_t at = (size_t)entry * a.hkv + kvh;
          bytes = (uint32_t)scale_byte(a.k_scale[at]) | (uint32_t)scale_byte(a.v_scale[at]) << 8;
        }
      }
      const int from_lane = (cu - from) / kWarps, st = issued % kStages;
      const int page = __shfl_sync(0xffffffffu, entry, from_lane);
      const uint32_t b = __shfl_sync(0xffffffffu, bytes, from_lane);
      const uint32_t count = (uint32_t)min(keys - cu * kPageSize, kPageSize);
      if (lane == st) meta = b | count << 16;
      if (lane == 0) {
        if (b) {
          mbar_arrive_expect_tx(&full[st], 2 * Sh::kPage);
          const int row = (int)(((long long)page * a.hkv + kvh) * kPageSize);
          tma_load_2d(sh.ring[warp][st][0], &tm_k, &full[st], 0, row);
          tma_load_2d(sh.ring[warp][st][1], &tm_v, &full[st], 0, row);
        } else {
          mbar_arrive(&full[st]);                    // an unreadable page: nothing to copy
        }
      }
      ++issued;
      cu += kWarps;
    };

#pragma unroll 1
    for (int part = 0; part < found; ++part) {
      const Part& p = sh.parts[part];
      const int pages = p.pages(), units = p.units();
      // ---- Q: row 8n + g, d = t D/4 .. ; factors and tokens of rows 8n + 2t, 8n + 2t + 1
      uint2 qb[kCols][kSteps];
      float factor[kCols][2];
      int tok[kCols][2], ex[kCols];
      uint4 x[kCols][kQuads];
#pragma unroll
      for (int n = 0; n < kCols; ++n) {
        const int row = 8 * n + g;
        const uint16_t* from_q = a.q + ((size_t)p.base + p.tok0 + row / a.gp) * a.q_stride +
                                 (p.h0 + row % a.gp) * D + t * (D / 4);
#pragma unroll
        for (int e = 0; e < kQuads; ++e)
          x[n][e] = row < p.tokens * a.gp ? load_once(from_q + 8 * e) : make_uint4(0, 0, 0, 0);
      }
      if (part == 0 && ok) {                         // the first copies, behind these reads
#pragma unroll 1
        for (int k = 0; k < kStages; ++k) issue();
      }
#pragma unroll
      for (int n = 0; n < kCols; ++n) {
        uint32_t top = 0;
#pragma unroll
        for (int e = 0; e < kQuads; ++e) top = word_max(x[n][e], top);
        top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, 2));
        ex[n] = row_exponent(top, kLeastRow);
        const float f = power(kBias - ex[n]);
#pragma unroll
        for (int e = 0; e < kQuads; ++e) {
          qb[n][2 * e] = make_uint2(to_f16(x[n][e].x, f), to_f16(x[n][e].y, f));
          qb[n][2 * e + 1] = make_uint2(to_f16(x[n][e].z, f), to_f16(x[n][e].w, f));
        }
      }
#pragma unroll
      for (int n = 0; n < kCols; ++n)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          factor[n][r] = a.scale_log2 * power(kBias + __shfl_sync(0xffffffffu, ex[n], 8 * t + 4 * r));
          tok[n][r] = p.tok0 + (8 * n + 2 * t + r) / a.gp;
        }
      float o[kCols][kSteps][4], m[kCols][2], l[kCols][2];
#pragma unroll
      for (int n = 0; n < kCols; ++n) {
        m[n][0] = m[n][1] = -INFINITY;
        l[n][0] = l[n][1] = 0.f;
#pragma unroll
        for (int j = 0; j < kSteps; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[n][j][e] = 0.f;
      }
      // Scores y (s + e; of key g and rows 8n + 2t, 8n + 2t + 1, then of key 8 + g) to weights, in pb
      // as the right operand of V^T P^T. inv: 2^-e of the two keys.
      auto weights = [&](float (&y)[kCols][4], float inv0, float inv1, uint32_t (&pb)[kCols][2]) {
        // the maxima of rows are only brought together where one outgrows the running one
        bool grows = false;
#pragma unroll
        for (int n = 0; n < kCols; ++n)
#pragma unroll
          for (int r = 0; r < 2; ++r) grows |= fmaxf(y[n][r], y[n][2 + r]) > m[n][r] + flash::kRescaleLog2;
        if (__any_sync(0xffffffffu, grows)) {
#pragma unroll
          for (int n = 0; n < kCols; ++n)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              float top = fmaxf(y[n][r], y[n][2 + r]);
#pragma unroll
              for (int x = 4; x < 32; x <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
              if (!(top > m[n][r] + flash::kRescaleLog2)) continue;
              if (m[n][r] != -INFINITY) {
                const float alpha = flash::ex2_approx(m[n][r] - top);
                l[n][r] *= alpha;
#pragma unroll
                for (int j = 0; j < kSteps; ++j) {
                  o[n][j][r] *= alpha;
                  o[n][j][2 + r] *= alpha;
                }
              }
              m[n][r] = top;
            }
        }
#pragma unroll
        for (int n = 0; n < kCols; ++n) {
          float w[4];
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const float shift = kLift - (m[n][r] == -INFINITY ? 0.f : m[n][r]);
            w[r] = flash::ex2_approx(y[n][r] + shift);
            w[2 + r] = flash::ex2_approx(y[n][2 + r] + shift);
            l[n][r] = fmaf(w[r], inv0, fmaf(w[2 + r], inv1, l[n][r]));
          }
          pb[n][0] = transposed(pack_f16x2(w[0], w[1]));
          pb[n][1] = transposed(pack_f16x2(w[2], w[3]));
        }
      };
#pragma unroll 1
      for (int u = warp; u < units; u += kWarps) {
        float y[kCols][4] = {};
        uint32_t pb[kCols][2];
        if (u < pages) {
          const int st = used % kStages;
          ok = ok && __all_sync(0xffffffffu, wait_bounded(&full[st], (used / kStages) & 1));
          if (!ok) break;
          ++used;
          const uint32_t info = __shfl_sync(0xffffffffu, meta, st);
          const int kb = info & 255, vb = (info >> 8) & 255, count = info >> 16;
          if (vb) {
            const uint8_t* k = sh.ring[warp][st][0];
            const uint8_t* v = sh.ring[warp][st][1];
            // 16-byte chunk c of row r, as the copies swizzle it
            auto chunk = [](int r, int c) { return r * D + ((c ^ (D == 128 ? r & 7 : (r >> 1) & 3)) << 4); };
            uint4 kx[2][D / 64];
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
              for (int c = 0; c < D / 64; ++c)
                kx[h][c] = *reinterpret_cast<const uint4*>(k + chunk(8 * h + g, t * (D / 64) + c));
            uint32_t x[4][D / 32];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const int row = 2 * t + (r & 1) + 4 * (r & 2);
              if (D == 128) {
                *reinterpret_cast<uint4*>(x[r]) = *reinterpret_cast<const uint4*>(v + chunk(row, g));
              } else {
                *reinterpret_cast<uint2*>(x[r]) =
                    *reinterpret_cast<const uint2*>(v + chunk(row, g >> 1) + (g & 1) * 8);
              }
            }
#pragma unroll
            for (int c = 0; c < D / 64; ++c) {
              const uint32_t w0[4] = {kx[0][c].x, kx[0][c].y, kx[0][c].z, kx[0][c].w};
              const uint32_t w1[4] = {kx[1][c].x, kx[1][c].y, kx[1][c].z, kx[1][c].w};
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                uint32_t a0, a1, a2, a3;
                decode4(w0[e], a0, a2);
                decode4(w1[e], a1, a3);
#pragma unroll
                for (int n = 0; n < kCols; ++n) {
                  const uint2 b = qb[n][4 * c + e];
                  mma(y[n], a0, a1, a2, a3, b.x, b.y);
                }
              }
            }
            __syncwarp();
            const float e = (float)(vb - kBias), inv = inverse_power(vb);
#pragma unroll
            for (int n = 0; n < kCols; ++n)
#pragma unroll
              for (int r = 0; r < 2; ++r) {
                // (never 0 or infinite: it meets infinite scores)
                const float mul = fminf(fmaxf(factor[n][r] * power(kb), 1e-38f), 3e38f);
                y[n][r] = fmaf(y[n][r], mul, e);
                y[n][2 + r] = fmaf(y[n][2 + r], mul, e);
              }
            if (count < kPageSize) {                 // free slots, which may hold anything
#pragma unroll
              for (int n = 0; n < kCols; ++n)
#pragma unroll
                for (int c = 0; c < 4; ++c)
                  if (g + 4 * (c & 2) >= count) y[n][c] = -INFINITY;
#pragma unroll
              for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int w = 0; w < D / 32; ++w)
                  if (2 * t + (r & 1) + 4 * (r & 2) >= count) x[r][w] = 0;
            }
            weights(y, inv, inv, pb);
#pragma unroll
            for (int w = 0; w < D / 32; ++w) {
#pragma unroll
              for (int half = 0; half < 2; ++half) {
                const uint32_t pick = half ? 0x7362 : 0x5140;       // bytes of two keys in turn
                uint32_t a0, a1, a2, a3;
                decode4(__byte_perm(x[0][w], x[1][w], pick), a0, a1);
                decode4(__byte_perm(x[2][w], x[3][w], pick), a2, a3);
#pragma unroll
                for (int n = 0; n < kCols; ++n) mma(o[n][2 * w + half], a0, a1, a2, a3, pb[n][0], pb[n][1]);
              }
            }
          }
          issue();
        } else {
          // ---- 16 own keys, each over powers of two of its own
          const int k0 = p.own0 + (u - pages) * kPageSize, count = min(p.own1 - k0, kPageSize);
          uint4 kx[2][kQuads];
          float of_key[2], e[4];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int key = 8 * h + g;
            const uint16_t* row = a.k + ((size_t)p.base + k0 + key) * a.k_stride + p.kvh * D + t * (D / 4);
            uint32_t top = 0;
#pragma unroll
            for (int c = 0; c < kQuads; ++c) {
              kx[h][c] = key < count ? reinterpret_cast<const uint4*>(row)[c] : make_uint4(0, 0, 0, 0);
              top = word_max(kx[h][c], top);
            }
            top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, 2));
            const int ex = row_exponent(top, kLeastRow);
            const float f = power(kBias - ex);
            of_key[h] = power(kBias + ex);
#pragma unroll
            for (int c = 0; c < kQuads; ++c)
              kx[h][c] = make_uint4(to_f16(kx[h][c].x, f), to_f16(kx[h][c].y, f), to_f16(kx[h][c].z, f),
                                    to_f16(kx[h][c].w, f));
          }
#pragma unroll
          for (int c = 0; c < kQuads; ++c)
#pragma unroll
            for (int n = 0; n < kCols; ++n) {
              const uint2 b0 = qb[n][2 * c], b1 = qb[n][2 * c + 1];
              mma(y[n], kx[0][c].x, kx[1][c].x, kx[0][c].y, kx[1][c].y, b0.x, b0.y);
              mma(y[n], kx[0][c].z, kx[1][c].z, kx[0][c].w, kx[1][c].w, b1.x, b1.y);
            }
          uint32_t x[4][D / 16];
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int key = 2 * t + (r & 1) + 4 * (r & 2);
            const uint16_t* row = a.v + ((size_t)p.base + k0 + key) * a.v_stride + p.kvh * D + g * (D / 8);
            uint32_t top = 0;
#pragma unroll
            for (int c = 0; c < D / 64; ++c) {
              const uint4 in =
                  key < count ? cap_values(reinterpret_cast<const uint4*>(row)[c]) : make_uint4(0, 0, 0, 0);
              *reinterpret_cast<uint4*>(&x[r][4 * c]) = in;
              top = word_max(in, top);
            }
#pragma unroll
            for (int s = 4; s < 32; s <<= 1) top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, s));
            const int ex = row_exponent(top, kLeastV);
            const float f = power(kBias - ex);
            e[r] = (float)ex;
#pragma unroll
            for (int w = 0; w < D / 16; ++w) x[r][w] = to_f16(x[r][w], f);
          }
          float of_v[2];                             // exponents of keys g and 8 + g
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float even = __shfl_sync(0xffffffffu, e[2 * h], g >> 1);
            const float odd = __shfl_sync(0xffffffffu, e[2 * h + 1], g >> 1);
            of_v[h] = g & 1 ? odd : even;
          }
#pragma unroll
          for (int n = 0; n < kCols; ++n)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const int key = g + 4 * (c & 2);
              const float mul = fminf(fmaxf(factor[n][c & 1] * of_key[c >> 1], 1e-38f), 3e38f);
              const bool sees = key < count && k0 + key <= tok[n][c & 1];
              y[n][c] = sees ? fmaf(y[n][c], mul, of_v[c >> 1]) : -INFINITY;
            }
          weights(y, power(kBias - (int)of_v[0]), power(kBias - (int)of_v[1]), pb);
#pragma unroll
          for (int w = 0; w < D / 16; ++w)
#pragma unroll
            for (int n = 0; n < kCols; ++n)
              mma(o[n][w], __byte_perm(x[0][w], x[1][w], 0x5410), __byte_perm(x[0][w], x[1][w], 0x7632),
                  __byte_perm(x[2][w], x[3][w], 0x5410), __byte_perm(x[2][w], x[3][w], 0x7632), pb[n][0],
                  pb[n][1]);
        }
      }
      // ---- the warps' maxima, sums and O together
      __syncthreads();                               // the part before is out
      if (p.slot >= 0 && threadIdx.x == 0) {
        // cut x of n lies at floor(x total / n)
        const long long n = sh.scan.ctas, total = sh.scan.total;
        sh.first = (int)((p.cuts0 * n + total - 1) / total) - 1;
        sh.pieces = (int)((p.cuts1 * n + total - 1) / total) - sh.first;
      }
#pragma unroll
      for (int n = 0; n < kCols; ++n)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
#pragma unroll
          for (int x = 4; x < 32; x <<= 1) l[n][r] += __shfl_xor_sync(0xffffffffu, l[n][r], x);
          if (g == 0) sh.ml[warp][8 * n + 2 * t + r] = make_float2(m[n][r], l[n][r]);
          // vector (n, r, w): row 8n + 2t + r, d = g D/8 + 4w ..
#pragma unroll
          for (int w = 0; w < D / 32; ++w)
            sh.o[warp][(2 * n + r) * (D / 32) + w][lane] = make_float4(
                o[n][2 * w][r], o[n][2 * w][2 + r], o[n][2 * w + 1][r], o[n][2 * w + 1][2 + r]);
        }
      __syncthreads();
      float4* to_part = a.part + ((size_t)blockIdx.x * 2 + p.slot) * kPartial<D, kRows>;
#pragma unroll 1
      for (int i = warp; i < Sh::kVec; i += kWarps) {
        const int nr = i / (D / 32), row = 8 * (nr >> 1) + 2 * t + (nr & 1), d = g * (D / 8) + i % (D / 32) * 4;
        float top = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) top = fmaxf(top, sh.ml[w][row].x);
        float sum = 0.f;
        float4 r = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          const float2 ml = sh.ml[w][row];
          const float f = ml.x > -INFINITY ? flash::ex2_approx(ml.x - top) : 0.f;    // top = +infinity: NaN
          const float4 v = sh.o[w][i][lane];
          sum = fmaf(ml.y, f, sum);
          r = make_float4(fmaf(v.x, f, r.x), fmaf(v.y, f, r.y), fmaf(v.z, f, r.z), fmaf(v.w, f, r.w));
        }
        if (p.slot >= 0) {
          to_part[d / 4 * kRows + row] = r;
          if (d == 0)
            reinterpret_cast<float2*>(to_part + kRows * D / 4)[row] =
                make_float2(top, units ? sum : kNoKeys);
        } else if (row < p.tokens * a.gp) {
          const float inv = reciprocal(sum);
          const size_t to = ((size_t)p.base + p.tok0 + row / a.gp) * a.hq + p.h0 + row % a.gp;
          *reinterpret_cast<uint2*>(a.o + to * D + d) =
              make_uint2(flash::pack_bf16x2(r.x * inv, r.y * inv), flash::pack_bf16x2(r.z * inv, r.w * inv));
        }
      }
      if (p.slot >= 0) {                             // whoever comes last joins the item's parts
        __syncthreads();
        if (threadIdx.x == 0) sh.joins = arrive(&a.arrived[sh.first]) == (uint32_t)sh.pieces - 1;
        __syncthreads();
        if (sh.joins) {
          constexpr int PART = kPartial<D, kRows>;
          const float4* first = a.part + (size_t)sh.first * 2 * PART;
          auto at = [&](int k) { return first + (k == 0 ? PART : (size_t)k * 2 * PART); };
          join<D, kRows, 4>(a, at, sh.pieces, p.tokens * a.gp, (size_t)p.base + p.tok0, p.h0, threadIdx.x,
                         Sh::kThreads);
        }
      }
    }
    __syncthreads();                                 // the list is free again
  }
  if (!ok) {                                         // a wait gave up: what is in flight ends first
    for (; used != issued; ++used) wait_bounded(&full[used % kStages], (used / kStages) & 1);
    flags |= MARS_ST_TIMEOUT;
  }
  flags = __reduce_or_sync(0xffffffffu, (unsigned)flags);
  if (lane == 0 && flags && a.status) atomicOr(a.status, flags);
}

// No part of an item has arrived yet.
__global__ void clear_kernel(uint32_t* arrived, int n) {
  sm100::let_next_start();
  sm100::wait_for_previous();
  for (int i = threadIdx.x; i < n; i += blockDim.x) arrived[i] = 0;
}

}  // namespace

template <int D, int kRows>
cudaError_t launch_chunk_q8_few(const q8::Args& a, int ctas, const CUtensorMap& k, const CUtensorMap& v,
                                cudaStream_t stream) {
  using Sh = Shared<D, kRows>;
  static_assert(sizeof(Sh) <= 227 * 1024, "shared memory of a CTA");
  static std::atomic<int> attr[64];
  cudaError_t e = set_smem_limit_once(few_kernel<D, kRows>, sizeof(Sh), attr);
  if (e != cudaSuccess) return e;
  if (a.can_split) {
    count_launches(1);
    e = launch_early(clear_kernel, 1, 256, 0, stream, a.arrived, ctas);
    if (e != cudaSuccess) return e;
  }
  count_launches(1);
  return launch_early(few_kernel<D, kRows>, ctas, Sh::kThreads, sizeof(Sh), stream, k, v, a);
}
#define MARS_FEW(D, R) \
  template cudaError_t launch_chunk_q8_few<D, R>(const q8::Args&, int, const CUtensorMap&, const CUtensorMap&, cudaStream_t)
MARS_FEW(64, 8);
MARS_FEW(64, 16);
MARS_FEW(128, 8);
MARS_FEW(128, 16);

}  // namespace mars
