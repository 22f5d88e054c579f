// Attention of new tokens over the 8-bit paged cache (cache_q8.cuh).
//
//   O_i = sum_u softmax_u(scale q_i . k_u) v_u over the keys row i of its sequence sees: the
//   P = seq_lens[s] cached keys, each its code times its page's scale, and the sequence's own keys
//   0 .. i in bf16.
//
// Three forms, by rows per sequence (plan_chunk_q8): chunk_q8_few.cu for the fewest, chunk_kernel here,
// and the wide form for many (packed_attn.cu over pages that ready_kernel unpacks).
//
// chunk_kernel works on the codes. A persistent CTA per SM takes an equal part of all key tiles of
// all items (chunk_q8.cuh); an item is a tile of up to 128 (token, query head) rows that share a KV
// head, as in packed_attn.cu, with the 128-key tiles that its rows see: the sequence's own keys
// first, then the cached ones.
//   - S = Q K^T takes K's codes as they are, in 8 bits. A row of Q, over a power of two that brings
//     its largest magnitude into [128, 256), is the sum of two e4m3 numbers (bf16 has 8 significant
//     bits, e4m3 4): exactly down to 2^-10 of that magnitude, to 2^-17 of it below. Own keys are two
//     such numbers too, over a power of two per 16 tokens. ready_kernel, before this one, makes both.
//   - Scores get the row's power and the K scale of their 16 keys as one factor in 32 bits.
//   - O += P V runs on f16 (chunk_q8.cuh says over what), and own values over a power of two per 16
//     tokens.
//   - Where 16 own rows differ much in size (kApartK, kApartV), each has a power of its own: one for all
//     would go by rows that a row may not see (a key 2^10 times the 15 before it took 0.8 % of
//     their rows' results, from 2^20 on everything). The converter warps then take those into an own
//     tile's scores, before the softmax sees them. (With the code for it in the softmax, although not
//     run, the 128 blocks of 16 took 254 to 278 us; so 245, and 240 without any of it.)
// Shared memory moves 128 bytes per cycle: the copies of a tile's codes take 256 cycles, S 512, the
// conversion of V 384, P V 256. (With K converted to f16 as well, 1,800 cycles per tile.)
//
// What bounds it: a tile takes 2,500 cycles, 1.7 times what its copies take at the rate of the memory. S
// of tile t + 2 waits for P V of tile t, whose P lies in its buffer, so that the chain S (1,000 with its
// waits), softmax (2,300), P V (700), waits (1,000) takes 5,000 cycles for each of the two buffers; TMEM
// has no room for a third beside two O of 128 columns.
//
// Blocks of 16 positions (28 query over 4 KV heads of 128, 128 sequences of 2,048 .. 8,192 keys): 246 us,
// 0.45 of the copy bandwidth; of 8, 32 sequences of 512 .. 2,048 keys: 39 us, of which the three
// launches and the start and end of every CTA are about 25.
//
// Roles (640 threads): warp 0 walks the items and reads block table and scales ahead of the others
// (infos); warp 1 copies K and Q; warps 12..15 copy V of even tiles, 16..19 of odd ones, two pages each
// into a ring of their own, and turn them into 32 rows of a swizzled f16 tile, zero where no key may be
// read; warps 2 and 3 issue S and O += P' V; warps 4..7 run the softmax of even tiles, 8..11 that of odd
// ones, a thread per row, each with an S buffer, an O, a maximum and a sum of its own, which are joined
// at an item's end. (With half of every tile's keys each, the exchange of maxima and the waits took
// longer than the softmax.) What a warp runs per tile is kept short: the code of all roles has to stay
// in some 32 KB of instruction cache. When it did not, a tile took 5,000 cycles; and what runs once per
// item costs some 40 cycles per instruction. (Hence ready_kernel; with Q and own rows turned into
// operands here, an item's start took 17,000 cycles instead of 9,000.)
//
// merge_kernel joins the parts of divided items. (Joined by the warps that come last, as
// chunk_q8_few.cu does it, blocks of 8 took 44 us: more of that code.)
#include <algorithm>
#include <climits>

#include "chunk_q8.cuh"

namespace mars {

namespace {

using flash::BKV;
using flash::BQ;
using namespace q8;

constexpr int kThreads = 640;
constexpr int kSoftmaxWarp = 4, kSoftmaxWarps = 8, kConvertWarp = 12, kConvertWarps = 8;
constexpr int kControlRegs = 72, kSoftmaxRegs = 136, kConvertRegs = 64;
static_assert(128 * (kControlRegs + 2 * kSoftmaxRegs + 2 * kConvertRegs) <=
                  kThreads * (65536 / kThreads / 8 * 8),
              "the register split fits the launch's register pool");
constexpr int kGroupWarps = kConvertWarps / 2, kPages = kPagesPerTile / kGroupWarps;   // of even or odd
                                     // tiles; pages of a warp
constexpr int kRaw = 2;              // ring of a converter warp's raw pages, kPages at a time
constexpr int kSlots = 4;            // ring of tiles of K's codes; an own tile takes two slots
constexpr int kAhead = 2;            // tiles that copies may be ahead of the conversion
constexpr int kTiles = 2;            // f16 tiles of V
constexpr int kBufs = 2;             // S buffers, and O's, in TMEM: of even and odd tiles
// Tiles that the walk may be ahead. It publishes up to four at once, the converters wait for up to
// kAhead more than they have released, and with this many the slots that it then needs belong to
// tiles that every converter has released.
constexpr int kInfos = 8;
static_assert(kInfos > kAhead + 4, "the walk and the converters do not wait for each other");

// 16 own rows share a power while the exponents of their largest magnitudes differ by at most so much.
constexpr int kApartK = 3, kApartV = 10;
// What the scores of an own tile with more powers than that become (own_scores): s + e, over a V of this
// scale byte. Its 2^-e is 0 in 32 bits, so that the row sum takes nothing from these weights.
constexpr int kMixedByte = 254;

// --------------------------------------------------------------------------------- the pipeline

enum : int { kFirst = 1, kLast = 2, kOwn = 4, kEnd = 8, kHoles = 16, kSecond = 32, kMixed = 64, kMixedEven = 128, kMixedOdd = 256 };

// A key tile as the walk hands it to the other warps.
struct alignas(16) Info {
  int flags;
  int base, n, tok0, h0, kvh;        // its item
  int slot;                          // of the partial, -1: the item is whole
  int k0, count;                     // first key (own: token of the sequence), keys that there are
  int item;                          // of this CTA
  int again;                         // mixed: not the first such of the even or odd tiles of its item
  int pad;
  alignas(16) int page[kPagesPerTile];         // own tiles: groups of own rows; -1: not to be read
  alignas(8) uint8_t k_byte[kPagesPerTile];    // scale bytes
  alignas(8) uint8_t v_byte[kPagesPerTile];    // 0: no such keys
};

struct Bar {
  uint64_t info_full[kInfos], info_empty[kInfos];
  uint64_t raw_full[kConvertWarps][kRaw];              // of a warp's pages
  uint64_t k_full[kSlots], k_empty[kSlots];
  uint64_t v_full[kTiles], v_empty[kTiles];
  uint64_t s_full[kBufs], p_full[kBufs], pv_done[kBufs];
  uint64_t s_raw[kBufs], own_done[kBufs];              // of mixed tiles, before s_full
  uint64_t q_full, q_free, o_free, drain[2];
  uint64_t pair[4];                  // the two warps of 32 rows
  uint32_t tmem_base;
  int abort;
};

// All that is not a tile. Its size keeps what follows, the tiles, aligned to 1024 bytes: they leave
// no room for aligning them at run time.
struct alignas(1024) Shared {
  Bar bar;
  Info infos[kInfos];
  union {
    Scan<kThreads> scan;             // until the walk has published its first tile
    float exchange[2][BQ];           // [even or odd tiles][row], at the end of items (and see own_scores)
  };
};
static_assert(sizeof(Shared) <= 3 * 1024, "with the tiles, the shared memory of a CTA");

template <int D>
struct Layout {
  static constexpr int RAW = BKV * D, TILE = BKV * D * 2, PAGE = kPageSize * D;
  // both parts of Q; K's codes; f16 tiles of V; raw ones
  static constexpr int OFF_Q = 0, OFF_K = 2 * RAW, OFF_V = OFF_K + kSlots * RAW;
  static constexpr int OFF_RAW = OFF_V + kTiles * TILE;
  static constexpr int TOTAL = OFF_RAW + 2 * kRaw * RAW;
  static constexpr int TM_S = 0, TM_O = kBufs * BKV, P_OFF = BKV / 2;    // O: D columns each
  static constexpr int PART = kPartial<D, BQ>;
  // 8-bit operands: rows of D bytes, 16-byte chunk c of row r, swizzled over D bytes
  static MARS_DEV uint32_t code_at(int r, int c) {
    return r * D + ((c ^ (D == 128 ? r & 7 : (r >> 1) & 3)) << 4);
  }
  static MARS_DEV uint64_t code_desc(const uint8_t* at) {
    return D == 128 ? sm100::sdesc_sw128(sm100::smem_u32(at), 16, 1024)
                    : sm100::sdesc_sw64(sm100::smem_u32(at), 16, 512);
  }
};

struct Pipe {
  const Args& a;
  Bar& bar;
  Info* infos;
  float (&exchange)[2][BQ];
  uint8_t* smem;
  uint32_t tmem;

  // Waits of one thread, and of a whole warp (by all lanes: behind a test of the lane a wait that is
  // over takes 250 cycles instead of 100). Where one gives up, the kernel's end sets the status.
  MARS_DEV bool wait(uint64_t* b, uint32_t parity) const {
    const bool ok = wait_bounded(b, parity);
    if (!ok) *(volatile int*)&bar.abort = 1;
    return ok;
  }
  MARS_DEV bool warp_wait(uint64_t* b, uint32_t parity) const {
    return __all_sync(0xffffffffu, wait(b, parity));
  }
  // the same for what a thread has in flight when it ends
  MARS_DEV void drain(uint64_t* b, uint32_t parity) const { wait(b, parity); }
  MARS_DEV Info& info(int t) const { return infos[t % kInfos]; }
  MARS_DEV uint64_t* info_full(int t, uint32_t& parity) const {
    parity = (t / kInfos) & 1;
    return &bar.info_full[t % kInfos];
  }
  MARS_DEV bool wait_info(int t) const {
    uint32_t p;
    uint64_t* b = info_full(t, p);
    return wait(b, p);
  }
  MARS_DEV bool warp_wait_info(int t) const {
    uint32_t p;
    uint64_t* b = info_full(t, p);
    return warp_wait(b, p);
  }
  MARS_DEV void warp_done(int t) const {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) sm100::mbar_arrive(&bar.info_empty[t % kInfos]);
  }
};

// Warp 0: this CTA's tiles, one after another.
template <int D>
MARS_DEV void walk(const Pipe& p, const Scan<kThreads>& sc) {
  using namespace sm100;
  const Args& a = p.a;
  const int lane = threadIdx.x & 31;
  Record rec{};
  int t = 0, flags = 0, items = 0;
  bool ok = true;
  // wait until `n` entries from t on are free
  auto room = [&](int n) {
    int good = 1;
    if (lane < n) good = p.wait(&p.bar.info_empty[(t + lane) % kInfos], (((t + lane) / kInfos) & 1) ^ 1);
    return __all_sync(0xffffffffu, good) != 0;
  };
  auto publish = [&](int n) {
    __syncwarp();
    if (lane < n) mbar_arrive(&p.bar.info_full[(t + lane) % kInfos]);
    t += n;
  };
  Row q = sc.at[0];
  int i = 0, j = 0, es = a.batch, ei = 0, ej = 0;
  if (sc.p1 < sc.total) es = sc.at[1].s;
#pragma unroll 1
  for (int end = es < a.batch; end >= 0; --end) {    // the end, if it is not that of all, then the start
    cut_at(a, sc.at[end], end ? sc.p1 : sc.p0, i, j);
    if (end) {
      ei = i;
      ej = j;
    }
  }
  Window window(a);
  for (;; ++i, j = 0) {
    if (i >= items_of(a, q)) {
      i = 0;
      j = 0;
      bool more;
      do {
        more = q.s + 1 < a.batch && q.s + 1 <= es;
        if (more) q = window.after(q);
      } while (more && items_of(a, q) == 0);
      if (!more) break;
    }
    if (q.s > es || (q.s == es && (i > ei || (i == ei && j >= ej)))) break;
    const int tiles = q.tiles(), jb = q.s == es && i == ei ? ej : tiles;
    const int rt = i / a.heads, hg = i % a.heads;
    const int tok0 = rt * a.tpt, last_tok = min(tok0 + a.tpt, q.n) - 1;
    const int slot = j > 0 ? 0 : jb < tiles ? 1 : -1;
    const int kvh = hg / (a.heads / a.hkv), h0 = hg * a.gp;
    if (slot == 1) rec = Record{1, rec.inside, q.base, tok0, last_tok + 1 - tok0, h0, {0, 0}};
    if (slot == 0 && jb < tiles) rec.inside = 1;
    // own tiles [j, own), cached tiles [c0, c1)
    const int own = min(min(jb, q.own()), last_tok / BKV + 1);
    const int c0 = max(j - q.own(), 0), c1 = max(jb - q.own(), 0);
    int left = max(own - j, 0) + c1 - c0;
    if (left == 0) {                                 // its own tiles here are behind the last token
      float2* ml = reinterpret_cast<float2*>(a.part + ((size_t)blockIdx.x * 2 + slot) * Layout<D>::PART +
                                             BQ * D / 4);
      for (int r = lane; r < BQ; r += 32) ml[r] = make_float2(-INFINITY, kNoKeys);
      continue;
    }
    int first = kFirst, last = kLast;
    const int item = items++;
    auto entry = [&](Info& e, int k0, int count, int f) {
      e.item = item;
      e.flags = f;
      e.base = q.base;
      e.n = q.n;
      e.tok0 = tok0;
      e.h0 = h0;
      e.kvh = kvh;
      e.slot = slot;
      e.k0 = k0;
      e.count = count;
    };
    for (int x = j; x < own && ok; ++x) {
      const int count = min(last_tok + 1 - x * BKV, BKV);
      const bool needed = lane < kPagesPerTile && lane * kPageSize < count;
      const int group = own_group(q.base, q.s) + x * kPagesPerTile + lane;
      uint8_t kb = kBias, vb = 0;
      if (needed) {
        const size_t at = (size_t)group * a.hkv + kvh;
        kb = a.own_k_byte[at];
        vb = a.own_v_byte[at];
      }
      const bool mixed = __any_sync(0xffffffffu, needed && (kb == 0 || vb == 0));
      if (!(ok = room(1))) break;
      Info& f = p.info(t);
      if (lane < kPagesPerTile) {
        f.page[lane] = needed ? group : -1;
        f.k_byte[lane] = mixed ? kBias : kb;
        f.v_byte[lane] = mixed && needed ? kMixedByte : vb;
      }
      const int bit = t & 1 ? kMixedOdd : kMixedEven;
      if (lane == 0) f.again = (last & bit) != 0;
      if (mixed) last |= bit;
      if (lane == 0) entry(f, x * BKV, count, kOwn | first | (left == 1 ? last : 0) | (mixed ? kMixed : 0));
      first = first & kFirst ? kSecond : 0;
      --left;
      publish(1);
    }
    // four cached tiles at a time, a page per lane; table entries are read a step ahead
    const int32_t* table = a.block_table + (size_t)q.s * a.max_pages;
    auto page_of = [&](int x) {
      const long long lp = (long long)x * kPagesPerTile + lane;
      return x + lane / kPagesPerTile < c1 && lp * kPageSize < q.P ? table[lp] : -1;
    };
    int next = page_of(c0);
    for (int x = c0; x < c1 && ok; x += 4) {
      const int n = min(4, c1 - x), e = next, mine = x + lane / kPagesPerTile;
      next = page_of(x + 4);
      const bool needed = mine < c1 && (mine * kPagesPerTile + lane % kPagesPerTile) * (long long)kPageSize < q.P;
      const bool readable = needed && e >= 0 && e < a.num_pages;
      if (needed && !readable) flags |= MARS_ST_NOPAGE;
      const uint32_t holes = __ballot_sync(0xffffffffu, needed && !readable);
      uint8_t kb = 127, vb = 0;
      if (readable) {
        const size_t at = (size_t)e * a.hkv + kvh;
        kb = (uint8_t)q8::scale_byte(a.k_scale[at]);
        vb = (uint8_t)q8::scale_byte(a.v_scale[at]);
      }
      if (!(ok = room(n))) break;
      if (lane < n * kPagesPerTile) {
        const int g = lane % kPagesPerTile, u = lane / kPagesPerTile;
        Info& f = p.info(t + u);
        f.page[g] = readable ? e : -1;
        f.k_byte[g] = kb;
        f.v_byte[g] = vb;
        if (g == 0)
          entry(f, mine * BKV, min(q.P - mine * BKV, BKV),
                (u == 0 ? first : u == 1 && first == kFirst ? kSecond : 0) | (u + 1 == left ? last : 0) |
                    (((holes >> lane) & 0xffu) ? kHoles : 0));
      }
      first = first & kFirst && n == 1 ? kSecond : 0;
      left -= n;
      publish(n);
    }
    if (!ok) break;
  }
  if (ok && room(2)) {                               // for the converters of even and of odd tiles
    if (lane < 2) p.info(t + lane).flags = kEnd;
    publish(2);
  }
  if (lane == 0 && a.rec) a.rec[blockIdx.x] = rec;
  if (flags && a.status) atomicOr(a.status, flags);
}

// Factor of a row's scores (one of 1e-30 makes them 0; own_scores divides by it).
MARS_DEV float row_factor(const Args& a, const Info& f, int tok, int row) {
  return fmaxf(a.scale_log2 * q8::power(a.q_byte[((size_t)f.base + tok) * a.hq + f.h0 + row % a.gp]), 1e-30f);
}

// Converter warps, a row per thread: the scores of a mixed own tile, whose keys and values have powers of
// their own, to what softmax() takes like a cached tile's: (s + e - 127) / factor in place, for a V of
// kMixedByte. The row sum cannot come from these weights, no 16 of which share an e: log2 of the sum of
// 2^s is left in exchange, where the softmax's thread finds it at the item's end. `uses`: mixed tiles before.
template <int D>
MARS_DEV bool own_scores(const Pipe& p, const Info& f, int t, int uses) {
  using namespace sm100;
  using L = Layout<D>;
  const Args& a = p.a;
  const int odd = t & 1, quad = (threadIdx.x >> 5) & 3, row = quad * 32 + (int)(threadIdx.x & 31);
  const uint32_t s_addr = p.tmem + L::TM_S + odd * BKV + ((uint32_t)(quad * 32) << 16);
  const int tok = f.tok0 + row / a.gp;
  const bool has = row < a.gp * a.tpt && tok < f.n;
  const int limit = min(f.count, tok + 1 - f.k0);
  const float factor = has ? row_factor(a, f, tok, row) : 1.f, inv = 1.f / factor;
  float* const kept = &p.exchange[odd][row];
  // The softmax has left the item before, and this tile's scores are there. (The P V of the tile before has
  // waited for the softmax to leave the item before its own: o_free is at most one phase behind then.)
  if (f.item > 0 && !(p.warp_wait(&p.bar.pv_done[odd ^ 1], ((t - 1) / kBufs) & 1) &&
                      p.warp_wait(&p.bar.o_free, (f.item - 1) & 1)))
    return false;
  if (!p.warp_wait(&p.bar.s_raw[odd], uses & 1)) return false;
  tc_fence_after();
  float top = -INFINITY, sum = 0.f;
  if (f.again) {                                     // the sum so far
    top = *kept;
    sum = 1.f;
  }
#pragma unroll 1
  for (int c = 0; c < f.count; c += 4) {
    uint32_t r[4];
    tmem_ld4(s_addr + c, r);
    // a group's byte, or where that is 0 those of its rows
    const int group = f.page[0] + c / kPageSize;
    const size_t at = (size_t)group * a.hkv + f.kvh, of_rows = ((size_t)f.kvh * a.own_groups + group) * kPageSize + c % kPageSize;
    uint32_t kb = a.own_k_byte[at] * 0x01010101u, vb = a.own_v_byte[at] * 0x01010101u;
    if (!kb) kb = *reinterpret_cast<const uint32_t*>(a.own_k_bytes + of_rows);
    if (!vb) vb = *reinterpret_cast<const uint32_t*>(a.own_v_bytes + of_rows);
    tmem_ld_wait();
    float s[4], m = top;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      s[e] = __uint_as_float(r[e]) * fminf(factor * power((int)(kb >> (8 * e) & 255u)), 3e38f);
      if (c + e >= limit) s[e] = -INFINITY;
      r[e] = __float_as_uint((s[e] + (float)((int)(vb >> (8 * e) & 255u) - kMixedByte)) * inv);
      m = fmaxf(m, s[e]);
    }
    tmem_st4(s_addr + c, r);
    const float base = m == -INFINITY ? 0.f : m;     // (+infinity gives NaN)
    sum *= flash::ex2_approx(top - base);
#pragma unroll
    for (int e = 0; e < 4; ++e) sum += flash::ex2_approx(s[e] - base);
    top = m;
  }
  tmem_st_wait();
  *kept = (top == -INFINITY ? 0.f : top) + log2f(sum);
  tc_fence_before();
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(&p.bar.own_done[odd]);
  if (quad == 0) {
    if (!p.warp_wait(&p.bar.own_done[odd], uses & 1)) return false;
    if ((threadIdx.x & 31) == 0) mbar_arrive(&p.bar.s_full[odd]);
  }
  return true;
}

// 16 bytes of an f16 tile: chunk c (8 elements) of row r. Regions of 64 elements, 128-byte swizzle.
MARS_DEV uint8_t* chunk_at(uint8_t* tile, int r, int c) {
  return tile + (c >> 3) * (BKV * 128) + flash::sw_off(r, c & 7);
}

// Warp 1: K's codes, a copy per page, an own tile's in two parts; and an item's Q, once every S of the
// item before is done.
template <int D>
MARS_DEV void load_k(const Pipe& p, const CUtensorMap& map, const CUtensorMap& map_q,
                     const CUtensorMap& map_own) {
  using namespace sm100;
  using L = Layout<D>;
  const Args& a = p.a;
  const int lane = threadIdx.x & 31;
  int c = 0, items = 0;                              // slots taken
  bool ok = true;
  for (int t = 0; ok && p.warp_wait_info(t); ++t) {
    const Info& f = p.info(t);
    const int flags = f.flags;
    if (flags & kEnd) break;
    const bool own = flags & kOwn;
    const int page = lane < kPagesPerTile ? f.page[lane] : -1;
    const int pages = __popc(__ballot_sync(0xffffffffu, page >= 0));
    int row = (max(page, 0) * a.hkv + f.kvh) * kPageSize;
#pragma unroll 1
    for (int i = 0; i <= own; ++i, ++c, row += a.own_groups * a.hkv * kPageSize) {
      const int st = c % kSlots;
      if (!(ok = p.warp_wait(&p.bar.k_empty[st], ((c / kSlots) & 1) ^ 1))) break;
      if (lane == 0) mbar_arrive_expect_tx(&p.bar.k_full[st], pages * L::PAGE);
      __syncwarp();
      if (page >= 0)
        tma_load_2d(p.smem + L::OFF_K + st * L::RAW + lane * L::PAGE, own ? &map_own : &map, &p.bar.k_full[st], 0, row);
    }
    if (!ok) break;
    if (flags & kFirst) {
      if (items > 0 && !(ok = p.warp_wait(&p.bar.q_free, (items - 1) & 1))) break;
      if (lane == 0) {
        mbar_arrive_expect_tx(&p.bar.q_full, 2 * a.gp * a.tpt * D);
#pragma unroll 1
        for (int i = 0; i < 2; ++i)
          tma_load_3d(p.smem + L::OFF_Q + i * L::RAW, &map_q, &p.bar.q_full, 0, f.h0, i * a.total + f.base + f.tok0);
      }
      ++items;
    }
    p.warp_done(t);
  }
  // no copy is in flight when the CTA ends
  if (lane == 0) {
#pragma unroll 1
    for (int i = max(0, c - kSlots); i < c; ++i)
      p.drain(&p.bar.k_full[i % kSlots], (i / kSlots) & 1);
    if (items > 0) p.drain(&p.bar.q_full, (items - 1) & 1);
  }
  __syncwarp();
}

// A raw page as rows r0 .. r0 + 15 of an f16 tile, zero from row `valid` of the page on.
template <int D>
MARS_DEV void convert_raw(const uint8_t* raw, uint8_t* tile, int r0, int valid) {
  constexpr int kLanes = D / 16, kStep = 32 / kLanes, kIts = kPageSize / kStep;
  const int lane = threadIdx.x & 31, c = lane % kLanes;
  // lanes of the second region store their chunks in the other order: the eight lanes of a row
  // then hit eight different chunks
  const int up = D == 128 ? c >> 2 : 0;
#pragma unroll 2
  for (int i = 0; i < kIts; ++i) {
    const int r = lane / kLanes + i * kStep;
    uint4 x = make_uint4(0, 0, 0, 0);
    if (r < valid)
      x = *reinterpret_cast<const uint4*>(raw + Layout<D>::code_at(r, c));
    uint32_t h[8];
    q8::decode4(x.x, h[0], h[1]);
    q8::decode4(x.y, h[2], h[3]);
    q8::decode4(x.z, h[4], h[5]);
    q8::decode4(x.w, h[6], h[7]);
    const uint4 lo = make_uint4(h[0], h[1], h[2], h[3]), hi = make_uint4(h[4], h[5], h[6], h[7]);
    *reinterpret_cast<uint4*>(chunk_at(tile, r0 + r, 2 * c + up)) = up ? hi : lo;
    *reinterpret_cast<uint4*>(chunk_at(tile, r0 + r, 2 * c + 1 - up)) = up ? lo : hi;
  }
}

// Warps 12 ..: copies of their pages of V and f16 tiles from them; own V is in f16.
template <int D>
MARS_DEV void convert(const Pipe& p, const CUtensorMap& map, const CUtensorMap& map_own) {
  using namespace sm100;
  using L = Layout<D>;
  const Args& a = p.a;
  const int lane = threadIdx.x & 31, warp = (threadIdx.x >> 5) - kConvertWarp;
  // of every other tile: pages page0 ..
  const int odd = warp / kGroupWarps, page0 = warp % kGroupWarps * kPages;
  uint64_t* const full = p.bar.raw_full[warp];
  uint8_t* const ring = p.smem + L::OFF_RAW + warp * kRaw * kPages * L::PAGE;
  // the next copies: their number and tile; `converted`: those that have left the ring
  int copies = 0, next = odd, converted = 0, own_copies = -1, mixed = 0;
  bool more = true, ok = true;
  auto copy_ahead = [&](int t) {
    while (more && next <= t + kAhead && copies < converted + kRaw) {
      if (!(ok = p.warp_wait_info(next))) break;
      const Info& f = p.info(next);
      const int flags = f.flags;
      next += 2;
      if (flags & kEnd) more = false;
      if (flags & (kEnd | kOwn)) continue;
      const int st = copies % kRaw, page = lane < kPages ? f.page[page0 + lane] : -1;
      const int pages = __popc(__ballot_sync(0xffffffffu, page >= 0));
      if (lane == 0) mbar_arrive_expect_tx(&full[st], pages * L::PAGE);
      __syncwarp();
      if (page >= 0)
        tma_load_2d(ring + (st * kPages + lane) * L::PAGE, &map, &full[st], 0, (page * a.hkv + f.kvh) * kPageSize);
      ++copies;
    }
  };
  for (int t = odd;; t += 2) {
    copy_ahead(t);                                   // has waited for tile t, if not earlier
    if (!ok) break;
    Info& f = p.info(t);
    const int flags = f.flags;
    static_assert(kTiles == 2, "of even and odd tiles");
    if (flags & kEnd) break;
    uint8_t* tile = p.smem + L::OFF_V + odd * L::TILE;
    if (!(ok = p.warp_wait(&p.bar.v_empty[odd], ((t / kTiles) & 1) ^ 1))) break;
    uint32_t bytes = 0;                              // that a copy puts there
    if (flags & kOwn) {
#pragma unroll 1
      for (int g = page0; g < page0 + kPages; ++g) {
        if (f.page[g] >= 0) bytes += 2 * L::PAGE;
        else convert_raw<D>(ring, tile, g * kPageSize, 0);
      }
    } else {
      const int st = converted % kRaw;
      if (!(ok = p.warp_wait(&full[st], (converted / kRaw) & 1))) break;
#pragma unroll 1
      for (int g = 0; g < kPages; ++g)
        convert_raw<D>(ring + (st * kPages + g) * L::PAGE, tile, (page0 + g) * kPageSize,
                       f.page[page0 + g] >= 0 ? f.count - (page0 + g) * kPageSize : 0);
      ++converted;
    }
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
      mbar_arrive_expect_tx(&p.bar.v_full[odd], bytes);
#pragma unroll 1
      for (int g = page0; bytes && g < page0 + kPages; ++g)
        for (int x = 0; x < D / 64 && f.page[g] >= 0; ++x)
          tma_load_2d(tile + x * (BKV * 128) + g * kPageSize * 128, &map_own, &p.bar.v_full[odd], x * 64,
                      (f.page[g] * a.hkv + f.kvh) * kPageSize);
      own_copies = bytes ? t : own_copies;
    }
    if ((flags & kMixed) && !(ok = own_scores<D>(p, f, t, mixed++))) break;
    p.warp_done(t);
  }
  // no copy is in flight when the CTA ends
  __syncwarp();
  if (lane == 0)
#pragma unroll 1
    for (int i = converted; i < copies; ++i) p.drain(&full[i % kRaw], (i / kRaw) & 1);
  // (where all went well, the last P V has waited for own ones)
  if (lane == 0 && !ok && own_copies >= 0) p.drain(&p.bar.v_full[odd], (own_copies / kTiles) & 1);
  __syncwarp();
}

// One thread: S_t = Q K_t^T, the sum over the parts of Q and K.
template <int D>
MARS_DEV void issue_s(const Pipe& p) {
  using namespace sm100;
  using L = Layout<D>;
  const uint32_t idesc = idesc_e4m3_f32(BQ, BKV);
  const uint64_t qd = L::code_desc(p.smem + L::OFF_Q);
  int slots = 0, items = 0;
  for (int t = 0; p.wait_info(t); ++t) {
    const int flags = p.info(t).flags;
    if (flags & kEnd) break;
    mbar_arrive(&p.bar.info_empty[t % kInfos]);
    const int sb = t % kBufs;
    if ((flags & kFirst) && !p.wait(&p.bar.q_full, items++ & 1)) break;
    // S buffer sb last held tile t - 2, whose P the PV of that tile read from it
    if (t >= kBufs && !p.wait(&p.bar.pv_done[sb], (t / kBufs - 1) & 1)) break;
    const int parts = flags & kOwn ? 2 : 1;
    bool ok = true;
#pragma unroll 1
    for (int i = 0; i < parts; ++i, ++slots) {
      const int st = slots % kSlots;
      if (!(ok = p.wait(&p.bar.k_full[st], (slots / kSlots) & 1))) break;
      tc_fence_after();
      const uint64_t kd = L::code_desc(p.smem + L::OFF_K + st * L::RAW);
#pragma unroll 2
      for (int k = 0; k < 2 * (D / 32); ++k) {
        const uint32_t off = k % (D / 32) * 32;
        mma_f8_ss(p.tmem + L::TM_S + sb * BKV, sdesc_advance(qd, off + k / (D / 32) * L::RAW),
                  sdesc_advance(kd, off), idesc, k != 0 || i != 0);
      }
      mma_commit(&p.bar.k_empty[st]);
    }
    if (!ok) break;
    mma_commit(flags & kMixed ? &p.bar.s_raw[sb] : &p.bar.s_full[sb]);
    if (flags & kLast) mma_commit(&p.bar.q_free);
  }
  mma_commit(&p.bar.drain[0]);
  p.drain(&p.bar.drain[0], 0);
}

// One thread: O += P'_t V_t.
template <int D>
MARS_DEV void issue_pv(const Pipe& p) {
  using namespace sm100;
  using L = Layout<D>;
  const uint32_t idesc = idesc_f16_f32(BQ, D, true);
  for (int t = 0, items = 0; p.wait_info(t); ++t) {
    const int flags = p.info(t).flags;
    if (flags & kEnd) break;
    mbar_arrive(&p.bar.info_empty[t % kInfos]);
    const int pb = t % kBufs;
    // the O of the item before have been read
    if ((flags & kFirst) && items++ && !p.wait(&p.bar.o_free, items & 1)) break;
    if (!p.wait(&p.bar.v_full[t % kTiles], (t / kTiles) & 1)) break;
    if (!p.wait(&p.bar.p_full[pb], (t / kBufs) & 1)) break;
    tc_fence_after();
    const uint64_t vd =
        sdesc_sw128(smem_u32(p.smem + L::OFF_V + t % kTiles * L::TILE), BKV * 128, 1024);
#pragma unroll 2
    for (int k = 0; k < BKV / 16; ++k)
      mma_bf16_ts(p.tmem + L::TM_O + pb * D, p.tmem + L::TM_S + pb * BKV + L::P_OFF + k * 8,
                  sdesc_advance(vd, k * 2048), idesc, k != 0 || !(flags & (kFirst | kSecond)));
    mma_commit(&p.bar.pv_done[pb]);
    mma_commit(&p.bar.v_empty[t % kTiles]);
  }
  mma_commit(&p.bar.drain[1]);
  p.drain(&p.bar.drain[1], 0);
}

// Factor of the scores of 16 keys (never 0 or infinite: it meets infinite scores), and the exponent
// of their V; by their scale bytes, the low ones of k and v.
MARS_DEV float k_factor(float factor, uint32_t k) {
  return fminf(fmaxf(factor * q8::power((int)(k & 255u)), 1e-38f), 3e38f);
}
MARS_DEV float v_exponent(uint32_t v) {              // 2^23 + byte is exact
  return (v & 255u) ? __int_as_float(0x4b000000 | (int)(v & 255u)) - (8388608.f + q8::kBias) : -INFINITY;
}

// Softmax and output.
template <int D>
MARS_DEV void softmax(const Pipe& p) {
  using namespace sm100;
  using L = Layout<D>;
  constexpr int kKeys = BKV / 2, kGroups = kPagesPerTile / 2;       // at a time
  const Args& a = p.a;
  const int warp = (threadIdx.x >> 5) - kSoftmaxWarp, quad = warp & 3, odd = warp >> 2;
  const int row = quad * 32 + (int)(threadIdx.x & 31);
  const uint32_t lane_off = (uint32_t)(quad * 32) << 16;
  const uint32_t s_addr = p.tmem + L::TM_S + odd * BKV + lane_off;
  const uint32_t o_addr = p.tmem + L::TM_O + lane_off;              // of even tiles
  float factor = 0.f, m = -INFINITY, l = 0.f;
  int tok = 0, tiles = 0, flags = 0, uses = 0;
  bool has = false, busy = false;
  // The two warps of 32 rows meet; what either wrote before is there after.
  auto meet = [&]() -> bool {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(&p.bar.pair[quad]);
    return p.warp_wait(&p.bar.pair[quad], uses++ & 1);
  };
  for (int t = -1;;) {                               // before the first tile t = -1
    const bool mine = t >= 0 && (t & 1) == odd;
    if (mine) {
      if (!p.warp_wait(&p.bar.s_full[t & 1], (t / kBufs) & 1)) return;
      tc_fence_after();
    }
    const Info& f = p.info(max(t, 0));
    if (mine && busy) {
      // keys that the row sees
      const int limit = (flags & kOwn) ? min(f.count, tok + 1 - f.k0) : f.count;
      const uint2 kbs = *reinterpret_cast<const uint2*>(f.k_byte);
      const uint2 vbs = *reinterpret_cast<const uint2*>(f.v_byte);
      const bool masked = __any_sync(0xffffffffu, limit < BKV) || (flags & kHoles);
      // Halves of the tile, the second first: its P' lies over its scores and makes room for the other's
#pragma unroll 1
      for (int h = 1; h >= 0; --h) {
        const uint32_t kb = h ? kbs.y : kbs.x, vb = h ? vbs.y : vbs.x;
        uint32_t r[kKeys], packed[kKeys / 2];
#pragma unroll
        for (int c = 0; c < kKeys / 32; ++c)
          tmem_ld32(s_addr + h * kKeys + c * 32, *reinterpret_cast<uint32_t(*)[32]>(r + c * 32));
        tmem_ld_wait();
        if (masked) {
#pragma unroll
          for (int g = 0; g < kGroups; ++g) {
            const int seen = ((vb >> (8 * g)) & 255) ? limit - h * kKeys - 16 * g : 0;
#pragma unroll
            for (int e = 0; e < 16; ++e)
              if (e >= seen) r[16 * g + e] = 0xff800000u;
          }
        }
        float sum, part;                             // of the P', and of P' 2^-e
#pragma unroll 1
        for (bool again = false;; again = true) {
          const float shift = kLift - (m == -INFINITY ? 0.f : m);
          sum = part = 0.f;
#pragma unroll
          for (int g = 0; g < kGroups; ++g) {
            const float mul = k_factor(factor, kb >> (8 * g)), add = v_exponent(vb >> (8 * g)) + shift;
            const float2 mul2 = make_float2(mul, mul), add2 = make_float2(add, add);
            float2 acc = make_float2(0.f, 0.f);
#pragma unroll
            for (int e = 16 * g; e < 16 * g + 16; e += 2) {
              const float2 x = __ffma2_rn(make_float2(__uint_as_float(r[e]), __uint_as_float(r[e + 1])), mul2, add2);
              const float2 w = make_float2(flash::ex2_approx(x.x), flash::ex2_approx(x.y));
              packed[e / 2] = q8::pack_f16x2(w.x, w.y);
              acc = __fadd2_rn(acc, w);
            }
            sum += acc.x + acc.y;
            // 2^-e; where there are no keys, the bits of some finite number, times 0
            part = fmaf(acc.x + acc.y, q8::inverse_power((vb >> (8 * g)) & 255), part);
          }
          // A maximum is only looked for where there is none as yet, or where it has been outgrown by so
          // much that f16 might end: the P' of a half are 2^15 together at most. (Looked for in every
          // half it took a fifth of the softmax.)
          if (again || !__any_sync(0xffffffffu, has && (m == -INFINITY || sum > 32768.f))) break;
          float top = -INFINITY;                     // the largest s + e
#pragma unroll
          for (int g = 0; g < kGroups; ++g) {
            float x[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) x[e] = __uint_as_float(r[16 * g + e]);
            const float y = flash::max3f(flash::max3f(x[0], x[1], x[2]), flash::max3f(x[3], x[4], x[5]),
                                         flash::max3f(x[6], x[7], x[8]));
            const float z = flash::max3f(flash::max3f(x[9], x[10], x[11]), flash::max3f(x[12], x[13], x[14]), x[15]);
            top = fmaxf(top, fmaf(fmaxf(y, z), k_factor(factor, kb >> (8 * g)), v_exponent(vb >> (8 * g))));
          }
          // O (the PV of its last tile came before S of this one; an item's first two tiles find none)
          // and the other half's P' go over the new maximum
          const bool raise = top > m;
          if (__any_sync(0xffffffffu, raise && m != -INFINITY)) {
            const float alpha = raise && m != -INFINITY ? flash::ex2_approx(m - top) : 1.f;
            l *= alpha;
            if (!(flags & (kFirst | kSecond))) {
#pragma unroll 1
              for (int c = odd * D; c < odd * D + D; c += 16) {
                uint32_t o[16];
                tmem_ld16(o_addr + c, o);
                tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                tmem_st16(o_addr + c, o);
              }
            }
            tmem_st_wait();
            if (h == 0) {
#pragma unroll 1
              for (int c = kKeys / 2; c < kKeys; c += 16) {
                uint32_t o[16];
                tmem_ld16(s_addr + L::P_OFF + c, o);
                tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                  const float2 w = q8::halves(o[e]);
                  o[e] = q8::pack_f16x2(w.x * alpha, w.y * alpha);
                }
                tmem_st16(s_addr + L::P_OFF + c, o);
              }
            }
          }
          if (raise) m = top;
        }
        l += part;
        tmem_st32(s_addr + L::P_OFF + h * (kKeys / 2), packed);
      }
      tmem_st_wait();
    }
    if (mine) {
      tc_fence_before();
      mbar_arrive_warp(&p.bar.p_full[odd]);
    }
    if (t >= 0 && (flags & kLast)) {
      if (busy) {
        // maxima and sums of the row's even and odd tiles, once both have left the item before
        float (&x)[2][BQ] = p.exchange;
        if (flags & (kMixedEven << odd)) l += flash::ex2_approx(x[odd][row] + kLift - (m == -INFINITY ? 0.f : m));
        if (!meet()) return;
        x[odd][row] = m;
        if (!meet()) return;
        const float other = x[odd ^ 1][row], top = fmaxf(m, other);
        // (m = +infinity gives NaN)
        float w = m > -INFINITY ? flash::ex2_approx(m - top) : 0.f;
        float w_other = other > -INFINITY ? flash::ex2_approx(other - top) : 0.f;
        if (!meet()) return;
        x[odd][row] = l * w;
        if (!meet()) return;
        l = x[0][row] + x[1][row];
        m = top;
        // the last two PVs, this thread's own first: the other's is known by what that one implies
        const bool two = tiles > 1;
        const int first = two && !mine ? t - 1 : t;
        if (!p.warp_wait(&p.bar.pv_done[first & 1], (first / kBufs) & 1)) return;
        const int second = 2 * t - 1 - first;
        if (two && !p.warp_wait(&p.bar.pv_done[second & 1], (second / kBufs) & 1)) return;
        tc_fence_after();
        // the row's O, half of the columns each: over its sum to where the row is, or into a partial
        // (without tiles of its own, an O is not there: the other one takes its place, times 0)
        const int slot = f.slot;
        const float inv = slot < 0 ? reciprocal(l) : 1.f;
        const uint32_t mine_at = o_addr + (two ? odd : t & 1) * D, other_at = o_addr + (two ? odd ^ 1 : t & 1) * D;
        w *= inv;
        w_other *= inv;
        float4* part = a.part + ((size_t)blockIdx.x * 2 + slot) * L::PART;
        if (slot >= 0 && has && odd == 0) reinterpret_cast<float2*>(part + BQ * D / 4)[row] = make_float2(m, l);
        uint16_t* to = a.o + (((size_t)f.base + tok) * a.hq + f.h0 + row % a.gp) * D;
#pragma unroll 1
        for (int c = odd * (D / 2); c < (odd + 1) * (D / 2); c += 16) {
          uint32_t u[16], v[16];
          tmem_ld16(mine_at + c, u);
          tmem_ld16(other_at + c, v);
          tmem_ld_wait();
          float o[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) o[e] = fmaf(__uint_as_float(u[e]), w, __uint_as_float(v[e]) * w_other);
          if (!has) continue;
          if (slot < 0) {
#pragma unroll
            for (int e = 0; e < 16; e += 8)
              *reinterpret_cast<uint4*>(to + c + e) =
                  make_uint4(flash::pack_bf16x2(o[e], o[e + 1]), flash::pack_bf16x2(o[e + 2], o[e + 3]),
                             flash::pack_bf16x2(o[e + 4], o[e + 5]), flash::pack_bf16x2(o[e + 6], o[e + 7]));
          } else {
#pragma unroll
            for (int e = 0; e < 16; e += 4)
              part[(c + e) / 4 * BQ + row] = make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
          }
        }
        tc_fence_before();
      }
      __syncwarp();
      if ((threadIdx.x & 31) == 0) mbar_arrive(&p.bar.o_free);
    }
    if (t >= 0) p.warp_done(t);
    ++t;
    if (!p.warp_wait_info(t)) return;
    const Info& n = p.info(t);
    flags = n.flags;
    if (flags & kEnd) return;
    ++tiles;
    if (flags & kFirst) {
      m = -INFINITY;
      l = 0.f;
      tiles = 1;
      tok = n.tok0 + row / a.gp;
      has = row < a.gp * a.tpt && tok < n.n;
      busy = __any_sync(0xffffffffu, has);       // warps without rows only keep step
      factor = 1.f;
      if (has) factor = row_factor(a, n, tok, row);
    }
  }
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
chunk_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
             const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_own_k,
             const __grid_constant__ CUtensorMap tm_own_v, Args a) {
  using namespace sm100;
  using L = Layout<D>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  __shared__ Shared shared;
  Bar& bar = shared.bar;
  Scan<kThreads>& scan = shared.scan;
  const int warp = threadIdx.x >> 5;
  if (smem_u32(smem_raw) % 1024) {                   // see Shared
    if (a.status) atomicOr(a.status, MARS_ST_TIMEOUT);
    return;
  }
  if (threadIdx.x == 0) {
    bar.abort = 0;
    for (int i = 0; i < kInfos; ++i) {
      mbar_init(&bar.info_full[i], 1);
      // the copies of K, both issuers, the tile's converters, the softmax's warps
      mbar_init(&bar.info_empty[i], 3 + kGroupWarps + kSoftmaxWarps);
    }
    for (int i = 0; i < kConvertWarps * kRaw; ++i) mbar_init(&bar.raw_full[i / kRaw][i % kRaw], 1);
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(&bar.k_full[i], 1);
      mbar_init(&bar.k_empty[i], 1);
    }
    for (int i = 0; i < kTiles; ++i) {
      mbar_init(&bar.v_full[i], kGroupWarps);
      mbar_init(&bar.v_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) mbar_init(&bar.drain[i], 1);
    for (int i = 0; i < kBufs; ++i) {
      mbar_init(&bar.s_full[i], 1);
      mbar_init(&bar.s_raw[i], 1);
      mbar_init(&bar.own_done[i], kGroupWarps);
      mbar_init(&bar.p_full[i], 128);
      mbar_init(&bar.pv_done[i], 1);
    }
    mbar_init(&bar.q_full, 1);
    mbar_init(&bar.q_free, 1);
    mbar_init(&bar.o_free, kSoftmaxWarps);
    for (int i = 0; i < 4; ++i) mbar_init(&bar.pair[i], 2);
    fence_barrier_init();
  }
  let_next_start();
  wait_for_previous();
  find_part(a, scan);
  if ((long long)blockIdx.x >= scan.ctas) {
    if (threadIdx.x == 0 && a.rec) a.rec[blockIdx.x] = Record{};
    return;
  }
  if (warp == 2) {
    tmem_alloc(&bar.tmem_base, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const Pipe p{a, bar, shared.infos, shared.exchange, smem_raw, __shfl_sync(0xffffffffu, bar.tmem_base, 0)};
  if (warp < kSoftmaxWarp) {
    regs_lower<kControlRegs>();
    if (warp == 0) {
      walk<D>(p, scan);
    } else if (warp == 1) {
      load_k<D>(p, tm_k, tm_q, tm_own_k);
    } else if (elect_one()) {
      if (warp == 2) issue_s<D>(p); else issue_pv<D>(p);
    }
  } else if (warp < kConvertWarp) {
    regs_raise<kSoftmaxRegs>();
    softmax<D>(p);
  } else {
    regs_lower<kConvertRegs>();
    convert<D>(p, tm_v, tm_own_v);
  }
  tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0 && bar.abort && a.status) atomicOr(a.status, MARS_ST_TIMEOUT);
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc(p.tmem, 512);
  }
}

// ------------------------------------------------------------------------- what comes before
//
// A kernel before chunk_kernel turns Q and the sequences' own rows into what its products take: it
// would otherwise do so at the start of every item, with the code for it out of the instruction cache
// (17,000 cycles an item, in which nothing else ran).
//
// Where the rows are many, a sequence's pages are written out in bf16 (exact too), once, and
// attended to by packed_attn.cu, whose CTAs would otherwise each convert them again (the wide form).

struct ReadyArgs {
  const uint16_t *q, *k, *v;
  long long q_stride, k_stride, v_stride;
  const int32_t *cu, *seq_lens, *block_table;
  const uint8_t *k_pool, *v_pool, *k_scale, *v_scale;
  int num_pages, max_pages, pages, tpt, batch, total, hq, hkv, own_groups;
  long long tiles;
  // the wide form's pages, lengths and table
  uint16_t *k_out, *v_out;
  int32_t *lens, *table;
  // chunk_kernel's: Q as [2][total][hq][D], scale bytes [total][hq]; groups of 16 own rows, K as
  // [2][groups][hkv][16][D] and V in f16 as [groups][hkv][16][D], scale bytes [groups][hkv] each, 0 where
  // the rows have their own, [hkv][groups][16]
  uint8_t *q_parts, *q_byte, *k_parts, *k_byte, *v_byte, *k_bytes, *v_bytes;
  uint16_t* v_half;
};
constexpr int kReadyThreads = 256;
// CTAs per SM where sequences may be unpacked. A hint may be far above what is cached: with a CTA for each tile
// that there could be, 12 chunks of up to 700 rows over 2,048 keys took 205 us at a hint of 131,072, 132 at 2,380.
constexpr int kReadyCtas = 16;
constexpr size_t kWideBytes = (size_t)1 << 31;       // pages of the wide form

// Eight bf16 times f as two e4m3 numbers each: the nearest, and the nearest to what that leaves. An
// infinity becomes NaN (a finite value's second product adds nothing).
MARS_DEV void split8(const uint4& x, float f, uint2& first, uint2& second) {
  float e[8];
  unpack8(x, e);
  uint32_t u[2], v[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    float* w = e + 4 * i;
#pragma unroll
    for (int k = 0; k < 4; ++k) w[k] = fmaf(w[k], 0.f, w[k] * f);
    u[i] = q8::encode2(w[0], w[1]) | (q8::encode2(w[2], w[3]) << 16);
    uint32_t lo, hi;
    q8::decode4(u[i], lo, hi);
    const float2 p = q8::halves(lo), q = q8::halves(hi);
    v[i] = q8::encode2(w[0] - p.x, w[1] - p.y) | (q8::encode2(w[2] - q.x, w[3] - q.y) << 16);
  }
  first = make_uint2(u[0], u[1]);
  second = make_uint2(v[0], v[1]);
}

// Head w of q, k and v for 16 rows from r0 on of a sequence, rows of k and v from nr on zero. Whole warp.
template <int D>
MARS_DEV void split_rows(const ReadyArgs& a, const packed::Seq& sq, int r0, int nr, int w) {
  constexpr int kLanes = D / 8, kRows = 32 / kLanes, kIts = kPageSize / kRows;     // rows at a time
  const int lane = threadIdx.x & 31, c = lane % kLanes, r = lane / kLanes;
  const bool is_q = w < a.hq, is_v = w >= a.hq + a.hkv;
  const int h = is_q ? w : is_v ? w - a.hq - a.hkv : w - a.hq;
  const long long stride = is_q ? a.q_stride : is_v ? a.v_stride : a.k_stride;
  const size_t row0 = (size_t)sq.base + r0;
  const uint16_t* from = (is_q ? a.q : is_v ? a.v : a.k) + row0 * stride + h * D + c * 8;
  uint4 x[kIts];
#pragma unroll
  for (int i = 0; i < kIts; ++i)
    x[i] = r + i * kRows < nr ? *reinterpret_cast<const uint4*>(from + (r + i * kRows) * stride)
                              : make_uint4(0, 0, 0, 0);
  // largest finite magnitude of row i, as bf16 bits: this lane's part, in both halves, and all of it
  auto row_max = [&](int i) {
    return finite_max(finite_max(finite_max(finite_max(0, x[i].x), x[i].y), x[i].z), x[i].w);
  };
  auto top_of = [&](int i) {
    uint32_t top = row_max(i);
    top = max(top >> 16, top & 0xffffu);
#pragma unroll
    for (int o = 1; o < kLanes; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
    return top;
  };
  // q, k: the row's largest magnitude into [128, 256) (a row of next to nothing: 2^-53)
  auto byte_of = [](uint32_t top) { return top ? min(max((int)(top >> 7), 74), 253) - 7 : kBias; };
  if (is_q) {
#pragma unroll
    for (int i = 0; i < kIts; ++i) {
      const int byte = byte_of(top_of(i));
      if (r + i * kRows >= nr) continue;
      uint2 u, v;
      split8(x[i], inverse_power(byte), u, v);
      const size_t at = (row0 + r + i * kRows) * a.hq + h;
      *reinterpret_cast<uint2*>(a.q_parts + at * D + c * 8) = u;
      *reinterpret_cast<uint2*>(a.q_parts + ((size_t)a.total * a.hq + at) * D + c * 8) = v;
      if (c == 0) a.q_byte[at] = (uint8_t)byte;
    }
    return;
  }
  // the same of rows i and i + 1 in the halves of tops[i / 2]; rows of zeros go by any power
  uint32_t tops[kIts / 2] = {}, most = 0, least = UINT_MAX;
#pragma unroll
  for (int i = 0; i < kIts; ++i) {
    if (is_v) x[i] = cap_values(x[i]);
    const uint32_t top = row_max(i);
    tops[i / 2] |= max(top >> 16, top & 0xffffu) << (i % 2 * 16);
  }
#pragma unroll
  for (int i = 0; i < kIts / 2; ++i) {
#pragma unroll
    for (int o = 1; o < kLanes; o <<= 1) tops[i] = __vmaxu2(tops[i], __shfl_xor_sync(0xffffffffu, tops[i], o));
    most = __vmaxu2(most, tops[i]);
    least = __vminu2(least, __vsub2(tops[i], 0x00010001u));
  }
  most = __reduce_max_sync(0xffffffffu, max(most >> 16, most & 0xffffu));
  least = __reduce_min_sync(0xffffffffu, min(least >> 16, least & 0xffffu)) + 1;
  // V's largest magnitude as high as f16 lets it: what is far below it keeps its bits
  auto of = [&](uint32_t top) { return is_v ? max((int)(top >> 7) - kTop, kLeast) : byte_of(top); };
  const bool mixed = most && (int)(most >> 7) - (int)(least >> 7) > (is_v ? kApartV : kApartK);
  const int shared = of(most), group = own_group(sq.base, sq.s) + sq.tile;
  if (lane == 0) (is_v ? a.v_byte : a.k_byte)[(size_t)group * a.hkv + h] = mixed ? 0 : (uint8_t)shared;
  const size_t second = (size_t)a.own_groups * a.hkv * kPageSize * D;
  size_t to = (((size_t)group * a.hkv + h) * kPageSize + r) * D + c * 8;
  uint8_t* bytes = (is_v ? a.v_bytes : a.k_bytes) + ((size_t)h * a.own_groups + group) * kPageSize + r;
#pragma unroll
  for (int i = 0; i < kIts; ++i, to += kRows * D, bytes += kRows) {
    const int byte = mixed ? of(tops[i / 2] >> (i % 2 * 16) & 0xffffu) : shared;
    const float f = inverse_power(byte);
    if (is_v) {
      float e[8];
      unpack8(x[i], e);
      *reinterpret_cast<uint4*>(a.v_half + to) =
          make_uint4(pack_f16x2(e[0] * f, e[1] * f), pack_f16x2(e[2] * f, e[3] * f),
                     pack_f16x2(e[4] * f, e[5] * f), pack_f16x2(e[6] * f, e[7] * f));
    } else {
      uint2 u, v;
      split8(x[i], f, u, v);
      *reinterpret_cast<uint2*>(a.k_parts + to) = u;
      *reinterpret_cast<uint2*>(a.k_parts + second + to) = v;
    }
    if (mixed && c == 0) *bytes = (uint8_t)byte;
  }
}

// A tile: 16 own rows of a sequence of P cached keys, or where it is left to the wide form a page of it (page j
// of sequence s becomes page s * pages + j); every gridDim.y-th eight heads. Sequences that chunk_kernel takes have no
// keys in the wide form, and what that then makes of their rows is written over.
template <int D>
MARS_DEV void ready_tile(const ReadyArgs& a, const packed::Seq& sq, int P, bool wide) {
  if (a.pages && sq.tile == 0 && blockIdx.y == 0 && threadIdx.x == 0) a.lens[sq.s] = wide ? P : 0;
  if (!wide) {
    const int r0 = sq.tile * kPageSize;
    if (r0 >= sq.n) return;
#pragma unroll 1
    for (int w = (blockIdx.y * kReadyThreads + threadIdx.x) / 32; w < a.hq + 2 * a.hkv;
         w += gridDim.y * (kReadyThreads / 32))
      split_rows<D>(a, sq, r0, min(sq.n - r0, kPageSize), w);
    return;
  }
  if (sq.tile * kPageSize >= P) return;
  const int page = a.block_table[(size_t)sq.s * a.max_pages + sq.tile];
  const bool mapped = page >= 0 && page < a.num_pages;
  const size_t out_page = (size_t)sq.s * a.pages + sq.tile;
  if (threadIdx.x == 0 && blockIdx.y == 0) a.table[out_page] = mapped ? (int)out_page : -1;
  if (!mapped) return;
  constexpr int kVectors = kPageSize * D / 16;     // of 16 codes, per head
  for (int i = blockIdx.y * kReadyThreads + threadIdx.x; i < 2 * a.hkv * kVectors; i += gridDim.y * kReadyThreads) {
    const int w = i / kVectors, c = i % kVectors;
    const bool is_v = w >= a.hkv;
    const int h = is_v ? w - a.hkv : w;
    const size_t at = (size_t)page * a.hkv + h, to = out_page * a.hkv + h;
    const uint4 x = reinterpret_cast<const uint4*>((is_v ? a.v_pool : a.k_pool) + at * (kPageSize * D))[c];
    const float f = power(scale_byte((is_v ? a.v_scale : a.k_scale)[at]));
    const uint32_t in[4] = {x.x, x.y, x.z, x.w};
    uint32_t out[8];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      uint32_t h[2];
      decode4(in[e], h[0], h[1]);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const float2 v = halves(h[k]);
        out[2 * e + k] = flash::pack_bf16x2(v.x * f, v.y * f);
      }
    }
    uint4* dst = reinterpret_cast<uint4*>((is_v ? a.v_out : a.k_out) + to * (kPageSize * D)) + 2 * c;
    dst[0] = make_uint4(out[0], out[1], out[2], out[3]);
    dst[1] = make_uint4(out[4], out[5], out[6], out[7]);
  }
}

// Block (x, y): tiles x, x + gridDim.x, .. of those that there are, of `a.tiles` that there could be by the hint.
template <int D>
__global__ void __launch_bounds__(kReadyThreads, 4) ready_kernel(ReadyArgs a) {
  sm100::let_next_start();
  sm100::wait_for_previous();
  const int skip = a.pages ? a.pages : -1;
  auto cut = [&](int len) { return (int)max(0LL, min((long long)len, (long long)a.max_pages * kPageSize)); };
  auto tiles = [](int rows) { return rows / kPageSize + (rows % kPageSize != 0); };
  __shared__ packed::Seq found;
#pragma unroll 1
  for (long long i = blockIdx.x; i < a.tiles; i += gridDim.x) {
    if (threadIdx.x < 32) {                          // (by every warp it was a third of all instructions)
      bool bad;
      const packed::Seq sq = packed::find_tile_by(
          a.cu, a.batch, a.total, i, bad, a.seq_lens, [&](int, int n, int len) {
            const int P = cut(len);
            return max(left_out(skip, a.tpt, n, P) ? tiles(P) : tiles(n), a.pages ? 1 : 0);
          });
      if (threadIdx.x == 0) found = sq;
    }
    __syncthreads();
    const packed::Seq sq = found;
    if (sq.s < 0) return;
    const int P = cut(sq.len);
    ready_tile<D>(a, sq, P, left_out(skip, a.tpt, sq.n, P));
    __syncthreads();                                 // `found` is free again
  }
}

// Parts of the workspace, in bytes from its start: what ready_kernel makes, what divided items leave, and
// the wide form's.
struct Places {
  size_t wide, lens, table, k, v, q_parts, q_byte, k_parts, k_byte, v_half, v_byte, k_bytes, v_bytes, rec, part, end;
};
Places places(const ChunkQ8Plan& plan, int batch, int total, int hq, int hkv, int d) {
  Places l{};
  size_t end = 0;
  auto take = [&](size_t& at, size_t bytes) {
    at = end;
    end += packed::align256(bytes);
  };
  if (!plan.few) {
    const size_t groups = (size_t)own_groups(batch, total) * hkv, rows = (size_t)total * hq;
    take(l.q_parts, 2 * rows * d);
    take(l.q_byte, rows);
    take(l.k_parts, 2 * groups * kPageSize * d);
    take(l.k_byte, groups);
    take(l.v_half, groups * kPageSize * d * 2);
    take(l.v_byte, groups);
    take(l.k_bytes, groups * kPageSize);
    take(l.v_bytes, groups * kPageSize);
  }
  if (plan.can_split) {
    const int rows = plan.few ? plan.few : BQ;       // of a partial
    take(l.rec, plan.ctas * (plan.few ? sizeof(uint32_t) : sizeof(Record)));
    take(l.part, (size_t)plan.ctas * 2 * rows * (d + 2) * sizeof(float));
  }
  if (plan.pages) {
    end = std::max(end, plan.least);                 // (where the other forms' parts may end)
    const size_t bytes = (size_t)batch * plan.pages * hkv * kPageSize * d * 2;
    take(l.wide, plan.wide.ws_bytes);
    take(l.lens, (size_t)batch * sizeof(int32_t));
    take(l.table, (size_t)batch * plan.pages * sizeof(int32_t));
    take(l.k, bytes);
    take(l.v, bytes);
  }
  l.end = end;
  return l;
}

template <int D>
cudaError_t launch(const ChunkQ8& p, const ChunkQ8Plan& plan, uint8_t* ws, cudaStream_t stream) {
  const PackedAttn& t = p.attn;
  const Places l = places(plan, t.batch, t.total, t.hq, t.hkv, D);
  cudaError_t e;
  if (!plan.few) {
    ReadyArgs u{};
    u.q = t.q;
    u.k = t.k;
    u.v = t.v;
    u.q_stride = t.q_stride;
    u.k_stride = t.k_stride;
    u.v_stride = t.v_stride;
    u.cu = t.cu;
    u.seq_lens = t.seq_lens;
    u.block_table = t.block_table;
    u.k_pool = p.k_pool;
    u.v_pool = p.v_pool;
    u.k_scale = p.k_scale;
    u.v_scale = p.v_scale;
    u.num_pages = t.num_pages;
    u.max_pages = t.max_pages;
    u.pages = plan.pages;
    u.tpt = plan.tpt;
    u.batch = t.batch;
    u.total = t.total;
    u.hq = t.hq;
    u.hkv = t.hkv;
    u.own_groups = (int)own_groups(t.batch, t.total);
    u.tiles = plan.tiles;
    u.k_out = reinterpret_cast<uint16_t*>(ws + l.k);
    u.v_out = reinterpret_cast<uint16_t*>(ws + l.v);
    u.lens = reinterpret_cast<int32_t*>(ws + l.lens);
    u.table = reinterpret_cast<int32_t*>(ws + l.table);
    u.q_parts = ws + l.q_parts;
    u.q_byte = ws + l.q_byte;
    u.k_parts = ws + l.k_parts;
    u.k_byte = ws + l.k_byte;
    u.v_byte = ws + l.v_byte;
    u.k_bytes = ws + l.k_bytes;
    u.v_bytes = ws + l.v_bytes;
    u.v_half = reinterpret_cast<uint16_t*>(ws + l.v_half);
    count_launches(1);
    // (where there are many tiles, one CTA for each: mixed rows 148 us with five, 133 with one)
    const unsigned y = plan.pages ? 1 : (t.hq + 2 * t.hkv + 7) / 8;
    const long long most = plan.pages ? (long long)num_sms() * kReadyCtas : plan.tiles;
    e = launch_early(ready_kernel<D>, dim3((unsigned)std::min(plan.tiles, most), y), kReadyThreads, 0, stream, u);
    if (e != cudaSuccess) return e;
    if (plan.pages) {
      PackedAttn wide = t;
      wide.k_pool = u.k_out;
      wide.v_pool = u.v_out;
      wide.seq_lens = u.lens;
      wide.block_table = u.table;
      wide.num_pages = t.batch * plan.pages;
      wide.max_pages = plan.pages;
      e = launch_packed_attn(wide, plan.wide, ws + l.wide, stream);
      if (e != cudaSuccess) return e;
    }
  }
  Args a{};
  a.q = t.q;
  a.k = t.k;
  a.v = t.v;
  a.q_stride = t.q_stride;
  a.k_stride = t.k_stride;
  a.v_stride = t.v_stride;
  a.cu = t.cu;
  a.seq_lens = t.seq_lens;
  a.block_table = t.block_table;
  a.k_pool = p.k_pool;
  a.v_pool = p.v_pool;
  a.k_scale = p.k_scale;
  a.v_scale = p.v_scale;
  a.num_pages = t.num_pages;
  a.max_pages = t.max_pages;
  a.batch = t.batch;
  a.total = t.total;
  a.hq = t.hq;
  a.hkv = t.hkv;
  a.gp = plan.gp;
  a.tpt = plan.tpt;
  a.heads = t.hq / plan.gp;
  a.can_split = plan.can_split;
  a.skip_pages = plan.pages ? plan.pages : -1;
  a.scale_log2 = t.scale * 1.4426950408889634f;
  a.o = t.o;
  a.item_work = plan.few ? kFewItemWork : kItemWork;
  if (plan.can_split && plan.few) a.arrived = reinterpret_cast<uint32_t*>(ws + l.rec);
  if (!plan.few) {
    a.q_byte = ws + l.q_byte;
    a.own_k_byte = ws + l.k_byte;
    a.own_v_byte = ws + l.v_byte;
    a.own_k_bytes = ws + l.k_bytes;
    a.own_v_bytes = ws + l.v_bytes;
    a.own_groups = (int)own_groups(t.batch, t.total);
  }
  if (plan.can_split && !plan.few) a.rec = reinterpret_cast<Record*>(ws + l.rec);
  a.part = plan.can_split ? reinterpret_cast<float4*>(ws + l.part) : nullptr;
  a.status = t.status;
  // a page and KV head is 16 rows of the maps; an empty pool is never read (one page over q)
  CUtensorMap map_k, map_v, map_q, map_own_k, map_own_v;
  const bool any = t.num_pages > 0;
  const uint64_t dims[2] = {(uint64_t)D, (any ? (uint64_t)t.num_pages * t.hkv : 1) * kPageSize};
  const uint64_t pitch[1] = {(uint64_t)D};
  const uint32_t box[2] = {(uint32_t)D, (uint32_t)kPageSize};
  const void* none = t.q;
  if (!encode_tmap_u8(&map_k, any ? p.k_pool : none, 2, dims, pitch, box) ||
      !encode_tmap_u8(&map_v, any ? p.v_pool : none, 2, dims, pitch, box))
    return cudaErrorInvalidValue;
  if (plan.few == 8) return launch_chunk_q8_few<D, 8>(a, plan.ctas, map_k, map_v, stream);
  if (plan.few == 16) return launch_chunk_q8_few<D, 16>(a, plan.ctas, map_k, map_v, stream);
  using L = Layout<D>;
  static_assert(L::TOTAL + sizeof(Shared) <= 227 * 1024,
                "layout fits shared memory");
  static std::atomic<int> attr[64];
  e = set_smem_limit_once(chunk_kernel<D>, L::TOTAL, attr);
  if (e != cudaSuccess) return e;
  // groups of 16 own rows as pages: a KV head is 16 rows of these maps too
  const uint64_t own_rows = (uint64_t)a.own_groups * t.hkv * kPageSize;
  const uint64_t dims_k[2] = {(uint64_t)D, 2 * own_rows}, dims_v[2] = {(uint64_t)D, own_rows};
  const uint64_t pitch_v[1] = {(uint64_t)D * 2};
  const uint32_t box_v[2] = {64, (uint32_t)kPageSize};
  const uint64_t dims_q[3] = {(uint64_t)D, (uint64_t)t.hq, 2 * (uint64_t)t.total};
  const uint64_t pitch_q[2] = {(uint64_t)D, (uint64_t)t.hq * D};
  const uint32_t box_q[3] = {(uint32_t)D, (uint32_t)plan.gp, (uint32_t)plan.tpt};
  if (!encode_tmap_u8(&map_q, ws + l.q_parts, 3, dims_q, pitch_q, box_q) ||
      !encode_tmap_u8(&map_own_k, ws + l.k_parts, 2, dims_k, pitch, box) ||
      !encode_tmap_bf16(&map_own_v, ws + l.v_half, 2, dims_v, pitch_v, box_v))
    return cudaErrorInvalidValue;
  e = launch_early(chunk_kernel<D>, plan.ctas, kThreads, L::TOTAL, stream, map_k, map_v, map_q, map_own_k,
                   map_own_v, a);
  count_launches(1);
  if (e != cudaSuccess || !plan.can_split) return e;
  const int most = std::min(plan.gp * std::min(plan.tpt, t.total), BQ);      // rows of an item
  count_launches(1);
  return launch_early(merge_kernel<D, BQ>, dim3(plan.ctas, (most * (D / 4) + 255) / 256), 256, 0, stream, a,
                      plan.ctas);
}

}  // namespace

ChunkQ8Plan plan_chunk_q8(int batch, int total, int hq, int hkv, int d, int max_len, size_t ws_bytes) {
  ChunkQ8Plan p{};
  p.wide = plan_packed(batch, total, hq, hkv, d, max_len);
  p.gp = p.wide.gp;
  p.tpt = p.wide.tpt;
  const int group = hq / hkv;
  // chunk_q8_few.cu where a sequence's rows make one of its tiles, on average (28 query over 4 KV heads of 128, 32
  // sequences of 2,048 keys and 2 tokens each: 31 us against 44 here; with 4 tokens each, two tiles, 48 and 45); or
  // several, each of which reads the cache again, where neither are they more than the SMs nor their keys many:
  // 4 tokens of 8 sequences over 512 keys 17.2 us against 25.3 here, 64 of 1 17.5 and 26.9, 16 of 4 over 1,024
  // 26.3 and 26.9, over 2,000 30.8 and 26.5, 16 of 2 over 2,000 23.8 and 25.4, 8 of 1 over 8,192 24.7 and 28.8 (which
  // the bound on the keys leaves here).
  for (int rows : {16, 8}) {
    if (group > rows) continue;
    const long long mine = packed::max_tiles(batch, total, rows / group) * hkv;
    if (total <= (long long)batch * (rows / group) ||
        (rows == 16 && mine <= num_sms() && max_len <= 2048 && mine * max_len <= num_sms() * 1024LL))
      p.few = rows;
  }
  if (p.few) {
    p.gp = group;
    p.tpt = p.few / group;
  }
  // CTAs: as many as the items and their parts can keep busy, by the hint
  const int tiles = packed::key_tiles(max_len) + 1;
  auto ctas = [&](int gp, int tpt) {
    const long long items = packed::max_tiles(batch, total, tpt) * (hq / gp);
    return (int)std::min<long long>(num_sms(), items * std::max(1, tiles / kMinPart));
  };
  p.can_split = tiles >= 2 * kMinPart;
  p.ctas = ctas(p.gp, p.tpt);
  // What every form but the wide one can do with. Each of these grows with batch, total and max_len, so that
  // a workspace for the largest call is enough for all, whatever forms they take.
  for (int rows : {0, 8, 16}) {
    if (rows && group > rows) continue;
    ChunkQ8Plan f{};
    f.few = rows;
    f.can_split = p.can_split;
    f.ctas = rows ? ctas(group, rows / group) : ctas(p.wide.gp, p.wide.tpt);
    p.least = std::max(p.least, places(f, batch, total, hq, hkv, d).end);
  }
  // The wide form where packed_attn.cu would take pairs of row tiles (plan_packed) and sequences have more
  // than ten row tiles on average. 28 query over 4 KV heads of 128, 2,048 cached keys, chunk_kernel against
  // the wide form: 50 rows of 16 sequences (3 tiles) 61 and 82 us, 120 of 32 (7) 199 and 190, 200 of 8 (11) 99
  // and 92, 300 of 32 (17) 475 and 335, 1,400 of 1 (78) 106 and 79; 14 over 2 of 64: 120 of 32 (7) 87 and 91, 300
  // of 32 (17) 199 and 157. Its pages: by the hint, in kWideBytes and in what the workspace has beyond
  // the rest (sequences of more keys are left to chunk_kernel).
  if (p.wide.pair && !p.few && total > 10LL * batch * p.tpt) {
    const long long pages = std::max(1, max_len / kPageSize + (max_len % kPageSize != 0));
    const long long per_page = (long long)batch * (hkv * kPageSize * d * 4LL + (long long)sizeof(int32_t));
    const size_t besides = p.least + packed::align256(p.wide.ws_bytes) + 4 * 256 + (size_t)batch * sizeof(int32_t);
    const long long room = ws_bytes > besides ? (long long)std::min(ws_bytes - besides, kWideBytes) : 0;
    p.pages = (int)std::min(pages, room / per_page);
  }
  p.tiles = (long long)batch * p.pages + own_groups(batch, total);
  p.ws_bytes = std::max(p.least, places(p, batch, total, hq, hkv, d).end);
  return p;
}

cudaError_t launch_chunk_q8(const ChunkQ8& p, const ChunkQ8Plan& plan, void* workspace,
                            cudaStream_t stream) {
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  return p.attn.d == 64 ? launch<64>(p, plan, ws, stream) : launch<128>(p, plan, ws, stream);
}

}  // namespace mars
