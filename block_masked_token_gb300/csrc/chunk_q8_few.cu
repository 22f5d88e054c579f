// Attention over the 8-bit paged cache for few rows: single tokens, and blocks whose (token, query
// head) rows of a KV head are 16 at most.
//
// With so few rows the work is the reading of the cache: 2 D bytes per key and KV head against
// 4 * rows * D flops. chunk_q8.cu's roles and its 128-row tiles cost more there than the reading.
// Here a CTA's eight warps are alike and do not wait for each other: warp w takes pages w, w + 8, ..
// of the CTA's part of an item (chunk_q8.cuh), copies them by TMA through a ring of its own, and
// keeps its own running maximum, sum and O in registers, which the CTA joins at the part's end. A
// page is a step: S = Q K^T is 16 x 16 of it, P V one product of depth 16, by mma.sync, whose
// operands come from registers: codes are converted (e4m3 to f16, exactly) where they are used and
// never stored again, and one warp's conversion runs beside another's products. The order of d
// inside a product is free, and of O's columns too; both are taken so that a lane's operands are
// whole 16-byte reads of shared memory, without bank conflicts:
//   K: lane (g, t) of key g (and 8 + g) holds d = t D/4 .. of it; four consecutive d are its part
//      of a step of 16.
//   V: lane (g, t) holds d = g D/8 .. of keys 2t, 2t + 1, 2t + 8, 2t + 9; byte permutations pair
//      the codes of two keys. Column g of product j is then d = g D/8 + j.
#include <algorithm>
#include <atomic>

#include "chunk_q8.cuh"

namespace mars {
namespace {

using namespace q8;

constexpr int kRows = kFewRows, kWarps = 8, kThreads = 32 * kWarps, kStages = 4;
constexpr int kList = 32;            // parts found at a time
static_assert(kRows == 16, "a product's");

// A part of an item: which rows, which own keys and which cached pages.
struct Part {
  int s, base, tok0, tokens, h0, kvh, slot;
  int own0, own1, page0, page1, keys;               // keys: cached ones of the sequence
  // units of work: cached pages, then 16 own keys each
  MARS_DEV int pages() const { return page1 - page0; }
  MARS_DEV int units() const { return pages() + (own1 - own0 + kPageSize - 1) / kPageSize; }
};

template <int D>
struct Shared {
  static constexpr int kPage = kPageSize * D, kVec = D / 8;        // kVec: float4 of O per lane
  uint8_t ring[kWarps][kStages][2][kPage];           // codes of K and V
  float4 o[kWarps][kVec][32];
  float2 ml[kWarps][kRows];
  uint64_t full[kWarps][kStages];
  Part parts[kList];
  Scan<kThreads> scan;
  int found, abort;
};

// The parts of this CTA, one after another. Whole warp.
struct Walk {
  const Args& a;
  Row q, last;
  int i, j, es, ei, ej;
  bool more;
  Window window;
  Record rec;
  MARS_DEV Walk(const Args& a_, const Scan<kThreads>& sc)
      : a(a_), q(sc.at[0]), i(0), j(0), es(a_.batch), ei(0), ej(0), more(true), window(a_), rec{} {
    if (sc.p1 < sc.total) {
      es = sc.at[1].s;
      cut_at(a, sc.at[1], sc.p1, ei, ej);
    }
    cut_at(a, q, sc.p0, i, j);
  }
  MARS_DEV bool next(Part& p) {
    if (!more) return false;
    if (i >= items_of(a, q)) {
      i = j = 0;
      do {
        more = q.s + 1 < a.batch && q.s + 1 <= es;
        if (more) q = window.after(q);
      } while (more && items_of(a, q) == 0);
    }
    more = more && !(q.s > es || (q.s == es && (i > ei || (i == ei && j >= ej))));
    if (!more) return false;
    const int tiles = q.tiles(), jb = q.s == es && i == ei ? ej : tiles;
    const int hg = i % a.heads, last_tok = min((i / a.heads + 1) * a.tpt, q.n) - 1;
    p.s = q.s;
    p.base = q.base;
    p.tok0 = i / a.heads * a.tpt;
    p.tokens = last_tok + 1 - p.tok0;
    p.h0 = hg * a.gp;
    p.kvh = hg / (a.heads / a.hkv);
    p.slot = j > 0 ? 0 : jb < tiles ? 1 : -1;
    if (p.slot == 1) rec = Record{1, rec.inside, p.base, p.tok0, p.tokens, p.h0, {0, 0}};
    if (p.slot == 0 && jb < tiles) rec.inside = 1;
    // own tiles [j, own), cached tiles from behind them
    const int own = q.own();
    p.own0 = min(min(j, own) * kTile, last_tok + 1);
    p.own1 = jb < own ? min(jb * kTile, last_tok + 1) : last_tok + 1;
    p.page0 = max(j - own, 0) * kPagesPerTile;
    p.keys = q.P;
    p.page1 = min(max(jb - own, 0) * kPagesPerTile, q.P / kPageSize + (q.P % kPageSize != 0));
    ++i;
    j = 0;
    return true;
  }
};

// D += A B: 16 x 8, of depth 16, f16 operands.
MARS_DEV void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// bf16 rows as f16 over a power of two that brings the largest finite magnitude into
// [2^14, 2^15): what f16 then loses lies below 2^-39 of that.
constexpr int kTop = 14;
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
constexpr int kLeastRow = -126;      // Q and K: 2^126 is the largest factor
constexpr int kLeastV = -60;         // V: the sums of P' 2^-e stay far from the ends of the range

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
few_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v, Args a) {
  using namespace sm100;
  using Sh = Shared<D>;
  constexpr int kSteps = D / 16, kTiles = D / 8;     // products of S along d, and of O
  constexpr int kQuads = D / 32;                     // 16-byte reads of D/4 bf16
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  Sh& sh = *reinterpret_cast<Sh*>(smem_raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  if (smem_u32(smem_raw) % 1024) {                   // the ring's swizzle goes by address
    if (a.status) atomicOr(a.status, MARS_ST_TIMEOUT);
    return;
  }
  if (lane < kStages) mbar_init(&sh.full[warp][lane], 1);
  if (threadIdx.x == 0) sh.abort = 0;
  fence_barrier_init();
  find_part(a, sh.scan);
  if ((long long)blockIdx.x >= sh.scan.ctas) {
    if (threadIdx.x == 0 && a.rec) a.rec[blockIdx.x] = Record{};
    return;
  }
  Walk walk(a, sh.scan);                             // warp 0's is used
  uint64_t* full = sh.full[warp];
  bool ok = true;
  int flags = 0;
  uint32_t issued = 0, used = 0;                     // stages, counted on
  uint32_t meta = 0;                                 // of stage `lane`: scale bytes of K and V, and keys
  for (bool first = true;; first = false) {
    if (warp == 0) {
      int n = 0;
      Part p;
      while (n < kList && walk.next(p)) {
        if (lane == 0) sh.parts[n] = p;
        ++n;
      }
      if (lane == 0) sh.found = n;
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
    for (int k = 0; k < kStages; ++k) issue();

#pragma unroll 1
    for (int part = 0; part < found; ++part) {
      const Part& p = sh.parts[part];
      const int pages = p.pages(), units = p.units();
      // ---- Q: rows g and 8 + g, d = t D/4 ..
      uint32_t qa[kSteps][4];
      float factor[2];
      int tok[2];
      bool has[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int row = g + 8 * h;
        tok[h] = p.tok0 + row / a.gp;
        has[h] = row < p.tokens * a.gp;
        uint4 x[kQuads];
        const uint16_t* from_q = a.q + ((size_t)p.base + tok[h]) * a.q_stride + (p.h0 + row % a.gp) * D + t * (D / 4);
        uint32_t top = 0;
#pragma unroll
        for (int e = 0; e < kQuads; ++e) {
          x[e] = has[h] ? reinterpret_cast<const uint4*>(from_q)[e] : make_uint4(0, 0, 0, 0);
          top = word_max(x[e], top);
        }
        top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const int ex = row_exponent(top, kLeastRow);
        const float f = power(kBias - ex);
        factor[h] = a.scale_log2 * power(kBias + ex);
#pragma unroll
        for (int e = 0; e < kQuads; ++e) {
          qa[2 * e][h] = to_f16(x[e].x, f);
          qa[2 * e][2 + h] = to_f16(x[e].y, f);
          qa[2 * e + 1][h] = to_f16(x[e].z, f);
          qa[2 * e + 1][2 + h] = to_f16(x[e].w, f);
        }
      }
      float o[kTiles][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
      for (int j = 0; j < kTiles; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[j][e] = 0.f;
      // Scores y (s + e; of keys 2t, 2t + 1 of row g, then of row 8 + g; then of the keys 8 on) to
      // weights, in pa as the left operand of P V. inv: 2^-e of the lane's keys.
      auto weights = [&](float (&y)[2][4], const float (&inv)[4], uint32_t (&pa)[4]) {
        float top[2];
#pragma unroll
        for (int h = 0; h < 2; ++h)
          top[h] = fmaxf(fmaxf(y[0][2 * h], y[0][2 * h + 1]), fmaxf(y[1][2 * h], y[1][2 * h + 1]));
        // the maxima of rows are only brought together where one outgrows the running one
        const float limit0 = m[0] + flash::kRescaleLog2, limit1 = m[1] + flash::kRescaleLog2;
        if (__any_sync(0xffffffffu, top[0] > limit0 || top[1] > limit1)) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            top[h] = fmaxf(top[h], __shfl_xor_sync(0xffffffffu, top[h], 1));
            top[h] = fmaxf(top[h], __shfl_xor_sync(0xffffffffu, top[h], 2));
            if (!(top[h] > m[h] + flash::kRescaleLog2)) continue;
            if (m[h] != -INFINITY) {
              const float alpha = flash::ex2_approx(m[h] - top[h]);
              l[h] *= alpha;
#pragma unroll
              for (int j = 0; j < kTiles; ++j) {
                o[j][2 * h] *= alpha;
                o[j][2 * h + 1] *= alpha;
              }
            }
            m[h] = top[h];
          }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float shift = kLift - (m[h] == -INFINITY ? 0.f : m[h]);
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            const float w0 = flash::ex2_approx(y[n][2 * h] + shift), w1 = flash::ex2_approx(y[n][2 * h + 1] + shift);
            l[h] = fmaf(w0, inv[2 * n], fmaf(w1, inv[2 * n + 1], l[h]));
            pa[2 * n + h] = pack_f16x2(w0, w1);
          }
        }
      };
#pragma unroll 1
      for (int u = warp; u < units; u += kWarps) {
        float y[2][4] = {};
        uint32_t pa[4];
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
#pragma unroll
            for (int n = 0; n < 2; ++n) {
#pragma unroll
              for (int c = 0; c < D / 64; ++c) {
                const uint4 x = *reinterpret_cast<const uint4*>(k + chunk(8 * n + g, t * (D / 64) + c));
                const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  uint32_t b0, b1;
                  decode4(w[e], b0, b1);
                  mma(y[n], qa[4 * c + e], b0, b1);
                }
              }
            }
            // V's words early: their reading is done by the time that the weights are
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
            __syncwarp();
            const float e = (float)(vb - kBias), inv = inverse_power(vb);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              // (never 0 or infinite: it meets infinite scores)
              const float mul = fminf(fmaxf(factor[h] * power(kb), 1e-38f), 3e38f);
#pragma unroll
              for (int n = 0; n < 2; ++n) {
                y[n][2 * h] = fmaf(y[n][2 * h], mul, e);
                y[n][2 * h + 1] = fmaf(y[n][2 * h + 1], mul, e);
              }
            }
            if (count < kPageSize) {                 // free slots, which may hold anything
#pragma unroll
              for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int c = 0; c < 4; ++c)
                  if (8 * n + 2 * t + (c & 1) >= count) y[n][c] = -INFINITY;
#pragma unroll
              for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int w = 0; w < D / 32; ++w)
                  if (2 * t + (r & 1) + 4 * (r & 2) >= count) x[r][w] = 0;
            }
            weights(y, {inv, inv, inv, inv}, pa);
#pragma unroll
            for (int w = 0; w < D / 32; ++w) {
#pragma unroll
              for (int half = 0; half < 2; ++half) {
                const uint32_t pick = half ? 0x7362 : 0x5140;       // bytes of two keys in turn
                uint32_t b0[2], b1[2];
                decode4(__byte_perm(x[0][w], x[1][w], pick), b0[0], b0[1]);
                decode4(__byte_perm(x[2][w], x[3][w], pick), b1[0], b1[1]);
                mma(o[4 * w + 2 * half], pa, b0[0], b1[0]);
                mma(o[4 * w + 2 * half + 1], pa, b0[1], b1[1]);
              }
            }
          }
          issue();
        } else {
          // ---- 16 own keys, each over powers of two of its own
          const int k0 = p.own0 + (u - pages) * kPageSize, count = min(p.own1 - k0, kPageSize);
          float mul[2][2][2], e[4], inv[4];          // mul: [row][8 keys][key 2t, 2t + 1]
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            const int key = 8 * n + g;
            const uint16_t* row = a.k + ((size_t)p.base + k0 + key) * a.k_stride + p.kvh * D + t * (D / 4);
            uint4 x[kQuads];
            uint32_t top = 0;
#pragma unroll
            for (int c = 0; c < kQuads; ++c) {
              x[c] = key < count ? reinterpret_cast<const uint4*>(row)[c] : make_uint4(0, 0, 0, 0);
              top = word_max(x[c], top);
            }
            top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, 2));
            const int ex = row_exponent(top, kLeastRow);
            const float f = power(kBias - ex);
#pragma unroll
            for (int c = 0; c < kQuads; ++c) {
              mma(y[n], qa[2 * c], to_f16(x[c].x, f), to_f16(x[c].y, f));
              mma(y[n], qa[2 * c + 1], to_f16(x[c].z, f), to_f16(x[c].w, f));
            }
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              const float of_key = power(kBias + __shfl_sync(0xffffffffu, ex, 8 * t + 4 * c));
#pragma unroll
              for (int h = 0; h < 2; ++h) mul[h][n][c] = fminf(fmaxf(factor[h] * of_key, 1e-38f), 3e38f);
            }
          }
          uint32_t x[4][D / 16];
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int key = 2 * t + (r & 1) + 4 * (r & 2);
            const uint16_t* row = a.v + ((size_t)p.base + k0 + key) * a.v_stride + p.kvh * D + g * (D / 8);
            uint32_t top = 0;
#pragma unroll
            for (int c = 0; c < D / 64; ++c) {
              const uint4 in = key < count ? reinterpret_cast<const uint4*>(row)[c] : make_uint4(0, 0, 0, 0);
              *reinterpret_cast<uint4*>(&x[r][4 * c]) = in;
              top = word_max(in, top);
            }
#pragma unroll
            for (int s = 4; s < 32; s <<= 1) top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, s));
            const int ex = row_exponent(top, kLeastV);
            const float f = power(kBias - ex);
            e[r] = (float)ex;
            inv[r] = f;
#pragma unroll
            for (int w = 0; w < D / 16; ++w) x[r][w] = to_f16(x[r][w], f);
          }
#pragma unroll
          for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const int key = 8 * n + 2 * t + (c & 1);
              const bool sees = key < count && k0 + key <= tok[c >> 1];
              y[n][c] = sees ? fmaf(y[n][c], mul[c >> 1][n][c & 1], e[2 * n + (c & 1)]) : -INFINITY;
            }
          weights(y, inv, pa);
#pragma unroll
          for (int w = 0; w < D / 16; ++w) {
            mma(o[2 * w], pa, __byte_perm(x[0][w], x[1][w], 0x5410), __byte_perm(x[2][w], x[3][w], 0x5410));
            mma(o[2 * w + 1], pa, __byte_perm(x[0][w], x[1][w], 0x7632), __byte_perm(x[2][w], x[3][w], 0x7632));
          }
        }
      }
      // ---- the warps' maxima, sums and O together
      __syncthreads();                               // the part before is out
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
        l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
        if (t == 0) sh.ml[warp][g + 8 * h] = make_float2(m[h], l[h]);
      }
      // vector (w, h, c): row 8h + g, d = (2t + c) D/8 + 4w ..
#pragma unroll
      for (int w = 0; w < D / 32; ++w)
#pragma unroll
        for (int hc = 0; hc < 4; ++hc)
          sh.o[warp][4 * w + hc][lane] =
              make_float4(o[4 * w][hc], o[4 * w + 1][hc], o[4 * w + 2][hc], o[4 * w + 3][hc]);
      __syncthreads();
      float4* to_part = a.part + ((size_t)blockIdx.x * 2 + p.slot) * kPartial<D, kRows>;
#pragma unroll 1
      for (int i = warp; i < Sh::kVec; i += kWarps) {
        const int row = g + 4 * (i & 2), d = (2 * t + (i & 1)) * (D / 8) + (i >> 2) * 4;
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
    }
    __syncthreads();                                 // the list is free again
  }
  if (!ok) {                                         // a wait gave up: what is in flight ends first
    for (; used != issued; ++used) wait_bounded(&full[used % kStages], (used / kStages) & 1);
    flags |= MARS_ST_TIMEOUT;
  }
  flags = __reduce_or_sync(0xffffffffu, (unsigned)flags);
  if (lane == 0 && flags && a.status) atomicOr(a.status, flags);
  if (threadIdx.x == 0 && a.rec) a.rec[blockIdx.x] = walk.rec;
}

}  // namespace

template <int D>
cudaError_t launch_chunk_q8_few(const q8::Args& a, int ctas, const CUtensorMap& k, const CUtensorMap& v,
                                cudaStream_t stream) {
  static_assert(sizeof(Shared<D>) <= 227 * 1024, "shared memory of a CTA");
  static std::atomic<int> attr[64];
  cudaError_t e = set_smem_limit_once(few_kernel<D>, sizeof(Shared<D>), attr);
  if (e != cudaSuccess) return e;
  few_kernel<D><<<ctas, kThreads, sizeof(Shared<D>), stream>>>(k, v, a);
  count_launches(1);
  e = cudaGetLastError();
  if (e != cudaSuccess || !a.can_split) return e;
  merge_kernel<D, kRows><<<dim3(ctas, D / 64), 256, 0, stream>>>(a, ctas);
  count_launches(1);
  return cudaGetLastError();
}
template cudaError_t launch_chunk_q8_few<64>(const q8::Args&, int, const CUtensorMap&, const CUtensorMap&, cudaStream_t);
template cudaError_t launch_chunk_q8_few<128>(const q8::Args&, int, const CUtensorMap&, const CUtensorMap&, cudaStream_t);

}  // namespace mars
