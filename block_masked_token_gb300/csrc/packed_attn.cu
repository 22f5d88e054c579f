// Causal attention over packed sequences, without a cache (prompts) or after a paged prefix
// (a chunk of new tokens over the cache).
//
//   O_i = sum_u softmax_u(scale q_i . k_u) v_u over the keys row i of its sequence sees: the
//   P = seq_lens[s] cached keys (none without a cache) and the sequence's own keys 0 .. i;
//   lse_i = log2 sum_u exp2(scale log2(e) q_i . k_u).
//
// A CTA takes a tile of up to 128 (token, query head) rows that share one KV head: row r is
// token r / gp of the tile and head r % gp of the group, so that K and V are read once for the
// group. It runs the tcgen05 flash engine (flash_tc.cuh) over the 128-key tiles its rows see:
// prefix tiles gathered page by page from the pool, then tiles of the sequence's own keys,
// the last of which are causal. Keys past a sequence's end (rows of the next sequence, free
// slots of the last page, unmapped pages) are masked, and their V rows cleared, so that
// whatever they hold stays out.
//
// With few tiles and long key lists the list is cut into splits (plan_packed): each CTA writes
// an unnormalised partial (m in log2 units, l, O) and a second kernel merges them. One token for
// each of 32 sequences (28 heads over 4 of 128, 158,000 cached keys, 325 MB) takes 67 us, 0.72
// of the copy bandwidth; one SM takes in 16-token pages at 27 bytes per cycle, so a CTA that is
// left alone with a long list bounds it.
//
// Where the rows are many, pair_kernel takes two row tiles per CTA instead (see there).

#include <algorithm>
#include <climits>

#include "common.cuh"
#include "flash_tc.cuh"
#include "internal.h"
#include "packed.cuh"

namespace mars {

namespace {

using flash::BKV;
using flash::BQ;

constexpr int kPagesPerTile = BKV / kPageSize;   // 8
static_assert(BKV == 128, "packed::key_tiles");
constexpr int kVStages = 3;                      // as in the decode kernel: no O staging area
constexpr int kMinSplitTiles = 4;                // key tiles a split takes at least
constexpr int kEvenSplitTiles = 16;              // where splits only even lengths out

struct AttnArgs {
  const int32_t* cu;
  const int32_t* seq_lens;     // NULL: no cache
  const int32_t* block_table;
  int num_pages, max_pages;
  int batch, total, hq, hkv, gp, tpt, ngrp, nsplit, split_tiles;
  int rows;                    // pair kernel: tokens of an item
  bool can_split;              // and whether items may be divided
  float scale_log2;
  uint16_t* o;                 // [total][hq][D] bf16
  float* lse;                  // [hq][total] or NULL
  float* part;                 // [nsplit][total][hq][D + 4]; pair kernel: partial()
  int32_t* tickets;            // pair kernel: [ctas][2], zero at its start
  int32_t* status;
};

// lse of a row, and the factor of its O. l is 0 where every score is -infinity (O is then 0), and
// NaN where a score is NaN or +infinity: such a row is NaN in lse and, through the factor, in O,
// whatever a merge of partials made of its O.
MARS_DEV float statistic(float m, float l) { return l == 0.f ? -INFINITY : m + log2f(l); }
MARS_DEV float reciprocal(float l) { return l == 0.f ? 0.f : 1.f / l; }

// l of a split without keys, which writes no O.
constexpr float kNoKeys = -1.f;

template <int D>
struct RowsPolicy {
  static constexpr bool kHandOff = false;
  static constexpr bool kRowStats = false;
  static constexpr bool kClearRows = true;
  static constexpr int kVStages = mars::kVStages;
  const AttnArgs* a;
  const int32_t* bt_row;
  int base, n, tok0;           // sequence rows [base, base + n); first token of the tile
  int P, np;                   // cached keys, prefix tiles
  int h0;                      // first query head
  int j0, split;               // first key tile of this split
  int last_tok;                // last token of the tile

  struct Tile {
    int k0;              // first key: cached position, or token of the sequence
    uint32_t pmask;      // 16-key groups that may be read
    int count;           // keys that may be read
    bool prefix, full, clear;
  };
  int trow, hrow;              // token and head of this thread's row inside the tile
  MARS_DEV void set_row(int row) {
    trow = row / a->gp;
    hrow = row - trow * a->gp;
  }
  MARS_DEV int token(int row) const { return tok0 + row / a->gp; }
  // A row without a token (the tile's last rows, the tokens past the sequence) computes
  // something that is not stored; masking it would cost its whole warp the masks of every tile
  // (550 of 3900 cycles per key tile with 7 heads x 18 tokens = 126 rows).
  MARS_DEV bool row_valid(int) const { return true; }
  MARS_DEV bool has_token(int row) const { return row < a->gp * a->tpt && token(row) < n; }
  MARS_DEV flash::RowVis row_vis(int row) const { return {token(row) + 1, 0, -1}; }
  MARS_DEV Tile tile(int jl) const {
    Tile t;
    const int j = j0 + jl;
    t.prefix = j < np;
    if (t.prefix) {
      t.k0 = j * BKV;
      t.count = min(P - t.k0, BKV);
      // one page per lane (the call is warp-uniform)
      const int lp = t.k0 / kPageSize + (threadIdx.x & (kPagesPerTile - 1));
      const int e = lp < a->max_pages ? bt_row[lp] : -1;
      t.pmask = __ballot_sync(0xffffffffu, e >= 0 && e < a->num_pages) & 0xffu;
      t.full = t.count == BKV && t.pmask == 0xffu;
      t.clear = !t.full;
    } else {
      t.k0 = (j - np) * BKV;
      t.count = min(last_tok + 1 - t.k0, BKV);
      t.pmask = 0xffu;
      t.full = t.k0 + BKV <= tok0 + 1;
      t.clear = t.count < BKV;
    }
    return t;
  }
  MARS_DEV bool key_read(const Tile& t, int key) const {
    return key < t.count && ((t.pmask >> (key / kPageSize)) & 1u);
  }
  MARS_DEV flash::ColRange cols(const flash::RowVis& v, const Tile& t) const {
    return {t.prefix ? t.count : min(v.end1 - t.k0, t.count), BKV, -1, t.pmask};
  }
  MARS_DEV void store_chunk(int row, int col, const uint32_t (&r)[32], float inv, float m,
                            float l) const {
    if (!has_token(row)) return;
    const size_t tok = (size_t)base + token(row);
    const int h = h0 + row % a->gp;
    if (a->nsplit == 1) {
      if (col == 0 && a->lse)
        a->lse[(size_t)h * a->total + tok] = statistic(m, l);
      uint4* dst = reinterpret_cast<uint4*>(a->o + (tok * a->hq + h) * D + col);
#pragma unroll
      for (int e = 0; e < 32; e += 8) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          w[i] = flash::pack_bf16x2(__uint_as_float(r[e + 2 * i]) * inv,
                                    __uint_as_float(r[e + 2 * i + 1]) * inv);
        dst[e / 8] = make_uint4(w[0], w[1], w[2], w[3]);
      }
      return;
    }
    float* rec = a->part + (((size_t)split * a->total + tok) * a->hq + h) * (D + 4);
    if (col == 0) {
      rec[0] = m;
      rec[1] = l;
    }
#pragma unroll
    for (int e = 0; e < 32; e += 4)
      *reinterpret_cast<float4*>(rec + 4 + col + e) =
          make_float4(__uint_as_float(r[e]), __uint_as_float(r[e + 1]),
                      __uint_as_float(r[e + 2]), __uint_as_float(r[e + 3]));
  }
};

template <int D>
__global__ void __launch_bounds__(flash::NUM_THREADS, 1)
packed_rows_kernel(const __grid_constant__ CUtensorMap tm_q,
                   const __grid_constant__ CUtensorMap tm_k,
                   const __grid_constant__ CUtensorMap tm_v,
                   const __grid_constant__ CUtensorMap tm_kp,
                   const __grid_constant__ CUtensorMap tm_vp, AttnArgs a) {
  using namespace sm100;
  using S = flash::Smem<D, 0, kVStages>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ flash::Barriers bar;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int id = blockIdx.x;
  const int sp = id % a.nsplit;
  id /= a.nsplit;
  const int grp = id % a.ngrp;
  id /= a.ngrp;
  const int kvh = id % a.hkv;
  id /= a.hkv;
  bool bad;
  const packed::Seq sq =
      packed::find_tile(a.cu, a.batch, a.total, a.tpt, 0, id, bad, a.seq_lens);
  if (bad && threadIdx.x == 0 && a.status) atomicOr(a.status, MARS_ST_BADSEQ);
  if (sq.s < 0) return;

  RowsPolicy<D> pol;
  pol.a = &a;
  pol.base = sq.base;
  pol.n = sq.n;
  pol.tok0 = sq.tile * a.tpt;
  // cached keys; a length that the table cannot hold is cut to what it can
  const int cached = sq.len;
  pol.P = (int)max(0LL, min((long long)cached, (long long)a.max_pages * kPageSize));
  if (pol.P != cached && threadIdx.x == 0 && a.status) atomicOr(a.status, MARS_ST_OVERFLOW);
  pol.np = packed::key_tiles(pol.P);
  pol.bt_row = a.block_table ? a.block_table + (size_t)sq.s * a.max_pages : nullptr;
  pol.h0 = (kvh * a.ngrp + grp) * a.gp;
  pol.last_tok = min(pol.tok0 + a.tpt, sq.n) - 1;
  const int all = pol.np + pol.last_tok / BKV + 1;
  pol.split = sp;
  pol.j0 = sp * a.split_tiles;
  const int end = sp == a.nsplit - 1 ? all : min(all, pol.j0 + a.split_tiles);
  const int n_total = end - pol.j0;
  if (n_total <= 0) {                  // no keys in this split: empty partials
    for (int r = threadIdx.x; r < BQ; r += blockDim.x)
      if (pol.has_token(r)) {
        float* rec = a.part + (((size_t)sp * a.total + sq.base + pol.token(r)) * a.hq + pol.h0 +
                               r % a.gp) * (D + 4);
        rec[0] = -INFINITY;
        rec[1] = kNoKeys;
      }
    return;
  }

  const uint32_t raw = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + (((raw + 1023u) & ~1023u) - raw);
  if (threadIdx.x == 0) flash::init_barriers(bar);
  if (warp == 1) {
    tmem_alloc(&bar.tmem_base, S::TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, bar.tmem_base, 0);

  if (warp == 0 || warp == flash::V_LOADER_WARP) {
    const bool is_v = warp == flash::V_LOADER_WARP;
    if (!is_v && lane == 0) {
      mbar_arrive_expect_tx(&bar.q_full, a.gp * a.tpt * 128 * (D / 64));
      for (int x = 0; x < D / 64; ++x)
        tma_load_3d(smem + S::OFF_Q + x * (BQ * 128), &tm_q, &bar.q_full, x * 64, pol.h0,
                    sq.base + pol.tok0);
    }
    int st_flags = 0;
    const CUtensorMap* tm_pool = is_v ? &tm_vp : &tm_kp;
    const CUtensorMap* tm_new = is_v ? &tm_v : &tm_k;
    // block-table entry of this lane's page in key tile jl (-1 past the table), read one tile
    // ahead of its use
    auto entry = [&](int jl) -> int {
      const int j = pol.j0 + jl;
      if (jl >= n_total || j >= pol.np || lane >= kPagesPerTile) return 0;
      const int lp = j * kPagesPerTile + lane;
      return lp < a.max_pages ? pol.bt_row[lp] : -1;
    };
    int next_entry = entry(0);
    auto issue = [&](int jl, uint8_t* dst, uint64_t* b) {
      const int e = next_entry;
      next_entry = entry(jl + 1);
      const int j = pol.j0 + jl;
      if (j < pol.np) {
        if (lane < kPagesPerTile) {
          // a page that may not be read loads page 0 (masked, V rows cleared), or with an empty
          // pool the zeros past the end of its one-page map
          int page = 0;
          if (e >= 0 && e < a.num_pages)
            page = e;
          else if (j * BKV + lane * kPageSize < pol.P)
            st_flags |= MARS_ST_NOPAGE;
          const int row = a.num_pages > 0 ? (page * a.hkv + kvh) * kPageSize : kPageSize;
          for (int x = 0; x < D / 64; ++x)
            tma_load_2d(dst + x * (BKV * 128) + lane * (kPageSize * 128), tm_pool, b, x * 64, row);
        }
      } else if (lane == 0) {
        for (int x = 0; x < D / 64; ++x)
          tma_load_3d(dst + x * (BKV * 128), tm_new, b, x * 64, kvh, sq.base + (j - pol.np) * BKV);
      }
    };
    flash::load_ring<D, kVStages>(bar, smem, n_total, a.status, is_v, issue);
    if (!is_v && lane == 0) mbar_wait(&bar.q_full, 0, nullptr, a.status);
    if (st_flags && a.status) atomicOr(a.status, st_flags);
  } else if (warp == 1 || warp == flash::PV_ISSUER_WARP) {
    if (warp == 1 && elect_one())
      flash::single_issuer<D, kVStages>(bar, smem, n_total, tmem, a.status);
  } else {
    flash::softmax_loop<D>(bar, smem, pol, n_total, tmem, a.scale_log2, a.status);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, S::TMEM_COLS);
  }
}

// One warp per (row, query head): merge the partials of the splits.
template <int D>
__global__ void __launch_bounds__(256) packed_merge_kernel(AttnArgs a) {
  const long long gw = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  const long long tok = gw / a.hq;
  const int h = (int)(gw - tok * a.hq);
  if (tok >= a.total) return;
  const size_t rec = D + 4, step = (size_t)a.total * a.hq * rec;
  const float* base = a.part + ((size_t)tok * a.hq + h) * rec;
  auto stats = [&](int sp) {
    return sp < a.nsplit ? *reinterpret_cast<const float2*>(base + sp * step)
                         : make_float2(-INFINITY, kNoKeys);
  };
  float2 ml = stats(lane);                           // on its way while the boundaries are read
  bool bad;
  // rows behind the last sequence have no partials and stay as they are
  const packed::Seq sq = packed::find_tile(a.cu, a.batch, a.total, 1, 0, INT_MAX, bad);
  const int first_row = min(max(a.cu[0], 0), a.total);
  if (tok < first_row || tok >= sq.base) return;
  // m and l of 32 splits at a time, a lane each
  float m = -INFINITY, l = 0.f;
  float2 acc[D / 64];
#pragma unroll
  for (int i = 0; i < D / 64; ++i) acc[i] = make_float2(0.f, 0.f);
  for (int s0 = 0; s0 < a.nsplit; s0 += 32) {
    const int n = min(32, a.nsplit - s0);
    const float* first = base + s0 * step;
    if (s0) ml = stats(s0 + lane);
    float mx = fmaxf(m, ml.x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    const float old = m > -INFINITY ? exp2f(m - mx) : 0.f;
    // kNoKeys also marks the weight of a split that wrote no O; m = +infinity gives NaN
    const float w = ml.y == kNoKeys ? kNoKeys : ml.x > -INFINITY ? exp2f(ml.x - mx) : 0.f;
    float sum = w == kNoKeys ? 0.f : ml.y * w;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    m = mx;
    l = l * old + sum;
#pragma unroll
    for (int i = 0; i < D / 64; ++i) acc[i] = make_float2(acc[i].x * old, acc[i].y * old);
#pragma unroll 4
    for (int sp = 0; sp < n; ++sp) {
      const float ws = __shfl_sync(0xffffffffu, w, sp);
#pragma unroll
      for (int i = 0; i < D / 64; ++i) {
        const float2 v =
            *reinterpret_cast<const float2*>(first + sp * step + 4 + 2 * lane + 64 * i);
        acc[i].x += ws == kNoKeys ? 0.f : v.x * ws;
        acc[i].y += ws == kNoKeys ? 0.f : v.y * ws;
      }
    }
  }
  const float inv = reciprocal(l);
  if (a.lse && lane == 0) a.lse[(size_t)h * a.total + tok] = statistic(m, l);
  uint32_t* orow = reinterpret_cast<uint32_t*>(a.o + ((size_t)tok * a.hq + h) * D);
#pragma unroll
  for (int i = 0; i < D / 64; ++i)
    orow[lane + 32 * i] = flash::pack_bf16x2(acc[i].x * inv, acc[i].y * inv);
}

// ------------------------------------------------------------------------ pair kernel
//
// A persistent CTA per SM takes items of two row tiles (x = 0, 1) of the same sequence and KV
// head over one key list, each with a softmax warpgroup of its own, so that the tensor pipe
// works for one tile while the other's softmax runs, and each K and V tile is loaded once for
// both.
//   warp 0  loader: V_0, K_0, V_1, K_1, ... into a ring for K and one for V. Every warp that waits
//           on a ring waits for each of its tiles, needed or not: a wait for a phase whose
//           predecessor is still open would pass at once, on the one before
//   warps 1 (TMEM owner), 3  load Q_x and issue S_x = Q_x K_j^T for x = 0, 1. One thread for
//           both was the bottleneck: a step's wait, eight MMAs, commit and loop took it about
//           800 cycles, four times per key tile
//   warp 2  issues O_x += P_x V_j for both
//   warps 4..7, 8..11  softmax and output of row tile 0, 1 (thread = row)
// They work in steps of 64 keys. One step's chain, S, its softmax, PV and the hand-offs
// between them, takes about 1,700 cycles, of which the tensor pipe works a third: four steps
// have to be in flight, two per row tile, and TMEM holds just that many (two S buffers of 64
// columns per row tile, P in bf16 over the upper half of each, and two O of 128). With 128-key
// steps, one in flight per row tile, a pair of tiles took 4,000 cycles instead of 2,870.
// What bounds those 2,870 is shared memory at 128 bytes per cycle: an S MMA of 64 keys reads 6 KB
// for its 32 cycles of arithmetic, S 192 KB per pair, PV 64 KB, the copies write 64 KB: 2,500
// cycles. One sequence of 8,191 rows (28 heads over 4) runs at 1.35 PFLOP/s, 0.69 of the GEMM rate.
// The start and output of an item take about 7,000 cycles, which bounds short sequences.
// A row tile's first P of an item also says that its warps have read the O of the item before.
//
// CTAs take whole items by falling cost (list_items) or, where that would not come out even,
// equal parts of the work: the items of all sequences are laid out on a line, each as long as its
// work (its key tiles and a constant), and CTA c of E takes the part from c/E to (c+1)/E of it. A
// cut inside an item with many key tiles splits its key list there (cut_at); the CTAs then write
// partials (m, l, O) and the last of them to finish, known by a ticket, merges them in the order
// of the keys, so that results do not depend on which one it was. Nothing waits for another CTA.
// Each CTA finds its items from the boundaries by itself (find_part), for 3 to 7 us of the
// launch; a separate kernel that listed them took 9.
constexpr int kKSlots = 2, kVSlots = 3;          // ring depths, in tiles
constexpr int kStep = 64;                        // keys per step
constexpr int PAIR_THREADS = 384;
constexpr int PAIR_WG0_REGS = 88, PAIR_SOFTMAX_REGS = 208;
static_assert(128 * (PAIR_WG0_REGS + 2 * PAIR_SOFTMAX_REGS) <=
                  PAIR_THREADS * (65536 / PAIR_THREADS / 8 * 8),
              "the register split fits the launch's register pool");

template <int D>
struct PairSmem {
  static constexpr int TILE = BKV * D * 2;             // a Q, K or V tile
  static constexpr int OFF_Q = 0, OFF_K = 2 * TILE, OFF_V = OFF_K + kKSlots * TILE;
  static constexpr int TOTAL = OFF_V + kVSlots * TILE + 1024;
  static constexpr int TM_S = 0, TM_O = 2 * BKV, P_OFF = kStep / 2;
};

// An item as the loader hands it to the other warps.
struct PairItem {
  int s, base, n, P, np, tok0, h0;
  int tiles, ja, jb;                 // key tiles; this CTA's [ja, jb) (jb = 0: no more items)
  int all[2], steps[2];              // steps of the row tiles: over all key tiles, in this CTA
  int c1, cuts;                      // a divided item: CTAs c1 .. c1 + cuts - 1 start inside it
};
constexpr int kItems = 3;            // items handed over and not yet taken by every warp

struct PairBar {
  uint64_t k_full[kKSlots], k_empty[kKSlots], v_full[kVSlots], v_empty[kVSlots];
  uint64_t q_full[2], q_empty[2];
  uint64_t s_full[2][2], p_full[2][2], pv_done[2][2];     // [row tile][buffer]
  uint64_t drain[3];
  uint32_t tmem_base;
  int abort;
  uint64_t stored[2], told[2];       // a partial has been written; `last` has been set
  int last[2][4];                    // whether this CTA merges: per row tile, two questions for
                                     // each of at most two divided items
  uint64_t item_full[kItems], item_empty[kItems];
  PairItem items[kItems];
};

// Work of an item in units of 1/128 key tile: its key tiles, nearly, and kItemWork for its
// start and output. Linear in the tile index t, so that sums have a closed form.
constexpr long long kItemWork = 400;
constexpr int kMinPart = 4;                      // key tiles of a part of a split item

// A sequence as the line of items sees it.
struct Row {
  int s, base, n, P;
  long long pre;                     // work before the sequence

  MARS_DEV int tiles_of(const AttnArgs& a) const { return (n + a.rows - 1) / a.rows; }
  MARS_DEV int prefix() const { return packed::key_tiles(P); }
  // work of one head's first t items
  MARS_DEV long long upto(const AttnArgs& a, long long t) const {
    return t * (128LL * prefix() + kItemWork) + a.rows * (t * (t + 1) / 2);
  }
};

// Cached keys of a sequence: a length that the table cannot hold is cut to what it can.
MARS_DEV int cached_keys(const AttnArgs& a, int s) {
  if (!a.seq_lens) return 0;
  return (int)max(0LL, min((long long)a.seq_lens[s], (long long)a.max_pages * kPageSize));
}

// Key tiles of item t of a sequence.
MARS_DEV int key_tiles(const AttnArgs& a, const Row& q, int t) {
  return q.prefix() + (int)((min((long long)(t + 1) * a.rows, (long long)q.n) - 1) / BKV) + 1;
}

// Where position `pos` cuts an item of `tiles` key tiles at [s0, s0 + work): before its key
// tile j (0: before the item, tiles: after it). Items that are small beside a CTA's part, or
// too short to split, are cut at the nearer end.
MARS_DEV int cut_at(const AttnArgs& a, long long pos, long long s0, long long work, int tiles,
                    long long part) {
  const long long rem = pos - s0;
  if (!a.can_split || tiles < 2 * kMinPart || 8 * work <= part) return 2 * rem >= work ? tiles : 0;
  const int j = (int)(rem * tiles / work);
  return j < kMinPart ? 0 : tiles - j < kMinPart ? tiles : j;
}

// A CTA's part of the line: from key tile j of item (q, g, t), to key tile end_j of the item
// that starts at end_s0.
struct PairPart {
  Row q;
  int g, t, j;
  long long end_s0;
  int end_j;
  long long total, ctas;             // all work, CTAs that share it (0: none for this CTA)
};

// An undivided item of a CTA: token tile and (KV head, group) tg = t * heads + g.
struct ListItem {
  int s, base, n, tg;
};
constexpr int kListItems = 32;       // of a CTA
constexpr int kListMax = 1024;       // (sequence, token tile) entries

// What find_part leaves: `count` undivided items, or (count < 0) a part of the line; and its
// scan scratch.
struct PartScan {
  long long sum[PAIR_THREADS / 32];
  int top[PAIR_THREADS / 32];
  long long work;
  int tops, items, count;
  Row at[2];
  PairPart part;
  ListItem list[kListItems];
};

// Whole items, in turn by falling cost, where no CTA then has 15 % more than the average; false
// otherwise, or with so many items that their ends hardly matter. Every CTA ranks all (sequence,
// tile) entries for itself, alike, in `scratch`. Equal parts of the line are off by a few tiles
// where they meet between items, and a divided item takes 5,000 cycles more on either side: twelve
// prompts of 150 to 2,048 rows took 145 us so and take 137, chunks of 1 to 700 tokens over a cache
// 109 and 100.
struct ListScratch {
  int off[PAIR_THREADS + 1], base[PAIR_THREADS], n[PAIR_THREADS], P[PAIR_THREADS];
  alignas(16) int key[kListMax];
  int entry[kListMax], sorted_key[kListMax], sorted_entry[kListMax];
  long long most[PAIR_THREADS / 32], all[PAIR_THREADS / 32];
};

MARS_DEV bool list_items(const AttnArgs& a, PartScan& sc, const Row& q, ListScratch& w) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int heads = a.hkv * a.ngrp, ctas = gridDim.x, total = sc.items, n = total / heads;
  const int rounds = (total + ctas - 1) / ctas;
  if (a.batch > PAIR_THREADS || n == 0 || n > kListMax || rounds > kListItems) return false;
  // entries of the sequences, one after another
  const int mine = tid < a.batch ? q.tiles_of(a) : 0;
  int incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  __syncthreads();
  if (lane == 31) sc.top[warp] = incl;
  __syncthreads();
  for (int i = 0; i < warp; ++i) incl += sc.top[i];
  w.off[tid] = incl - mine;
  w.base[tid] = q.base;
  w.n[tid] = q.n;
  w.P[tid] = q.P;
  if (tid == 0) w.off[PAIR_THREADS] = n;
  __syncthreads();
  const int padded = (n + 3) / 4 * 4;
  for (int e = tid; e < padded; e += PAIR_THREADS) {
    int lo = 0, hi = PAIR_THREADS;                 // off[lo] <= e < off[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (w.off[mid] <= e) lo = mid; else hi = mid;
    }
    const Row r{lo, w.base[lo], w.n[lo], w.P[lo], 0};
    const int t = e - w.off[lo];
    // key tiles, and the entry's number so that no two are equal
    const int tiles = min(key_tiles(a, r, t), INT_MAX / kListMax - 1);
    w.key[e] = e < n ? tiles * kListMax + kListMax - 1 - e : -1;
    if (e < n) w.entry[e] = lo << 16 | t;
  }
  __syncthreads();
  for (int e = tid; e < n; e += PAIR_THREADS) {
    const int k = w.key[e];
    int rank = 0;
#pragma unroll 4
    for (int j = 0; j < padded; j += 4) {
      const int4 v = *reinterpret_cast<const int4*>(w.key + j);
      rank += (v.x > k) + (v.y > k) + (v.z > k) + (v.w > k);
    }
    w.sorted_key[rank] = k / kListMax;
    w.sorted_entry[rank] = w.entry[e];
  }
  __syncthreads();
  // item of CTA c in round r; rounds run forwards and backwards
  auto item = [&](int c, int r) { return r * ctas + ((r & 1) ? ctas - 1 - c : c); };
  long long most = 0, all = 0;
  for (int c = tid; c < ctas; c += PAIR_THREADS) {
    long long sum = 0;
    for (int r = 0; r < rounds; ++r) {
      const int i = item(c, r);
      if (i < total) sum += kItemWork - 64 + 128LL * w.sorted_key[i / heads];
    }
    most = max(most, sum);
    all += sum;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    most = max(most, __shfl_xor_sync(0xffffffffu, most, o));
    all += __shfl_xor_sync(0xffffffffu, all, o);
  }
  if (lane == 0) {
    w.most[warp] = most;
    w.all[warp] = all;
  }
  __syncthreads();
  for (int i = 0; i < PAIR_THREADS / 32; ++i) {
    most = max(most, w.most[i]);
    all = i == 0 ? w.all[0] : all + w.all[i];
  }
  if (most * ctas * 20 > all * 23) return false;
  if (tid < rounds) {
    const int i = item(blockIdx.x, tid);
    if (i < total) {
      const int e = w.sorted_entry[i / heads], s = e >> 16;
      sc.list[tid] = ListItem{s, w.base[s], w.n[s], (e & 0xffff) * heads + i % heads};
    }
    if (tid == rounds - 1) sc.count = rounds - (i >= total);
  }
  __syncthreads();
  return true;
}

// Every thread of the CTA: fill sc.list or sc.part.
MARS_DEV void find_part(const AttnArgs& a, PartScan& sc, ListScratch& scratch) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const long long heads = a.hkv * a.ngrp;
  int bad = 0;
  Row q{};
  long long mine = 0;
  // one chunk of sequences: q (with its work before it) and mine for this thread's
  auto chunk = [&](int s0) {
    const int s = s0 + tid, top0 = sc.tops;
    const long long before = sc.work;
    const int c = s < a.batch ? a.cu[s + 1] : top0;
    q.P = s < a.batch ? cached_keys(a, s) : 0;
    if (s < a.batch && a.seq_lens && q.P != a.seq_lens[s]) bad |= MARS_ST_OVERFLOW;
    int end = max(min(max(c, 0), a.total), top0);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, end, o);
      if (lane >= o) end = max(end, v);
    }
    if (lane == 31) sc.top[warp] = end;
    __syncthreads();
    int lead = top0;                               // the boundary before this warp
    for (int w = 0; w < warp; ++w) lead = max(lead, sc.top[w]);
    end = max(end, lead);
    if (s < a.batch && c != end) bad |= MARS_ST_BADSEQ;
    int begin = __shfl_up_sync(0xffffffffu, end, 1);
    if (lane == 0) begin = lead;
    q.s = s;
    q.base = begin;
    q.n = end - begin;
    const int tiles = s < a.batch ? q.tiles_of(a) : 0;
    mine = heads * q.upto(a, tiles);
    long long incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    if (lane == 31) sc.sum[warp] = incl;
    if (tiles) atomicAdd(&sc.items, (int)(tiles * heads));
    __syncthreads();
    q.pre = before + incl - mine;
    for (int w = 0; w < warp; ++w) q.pre += sc.sum[w];
    __syncthreads();
    if (tid == PAIR_THREADS - 1) {
      sc.tops = end;
      sc.work = q.pre + mine;
    }
    __syncthreads();
  };
  auto begin = [&] {
    if (tid == 0) {
      const int c0 = a.cu[0];
      sc.tops = min(max(c0, 0), a.total);
      if (c0 != sc.tops) bad |= MARS_ST_BADSEQ;
      sc.work = 0;
      sc.items = 0;
      sc.count = -1;
    }
    __syncthreads();
  };
  begin();
  for (int s0 = 0; s0 < a.batch; s0 += PAIR_THREADS) chunk(s0);
  if (bad && blockIdx.x == 0 && a.status) atomicOr(a.status, bad);
  if (list_items(a, sc, q, scratch)) return;
  const long long total = sc.work;
  // CTAs that share the work: as many as there are, unless that leaves less than a part each
  // and there are fewer items
  const long long ctas = min((long long)gridDim.x,
                             max((long long)sc.items, total / (160 * kMinPart)));
  if ((long long)blockIdx.x >= ctas) {
    if (tid == 0) sc.part.ctas = 0;
    __syncthreads();
    return;
  }
  const long long p0 = blockIdx.x * total / ctas, p1 = (blockIdx.x + 1) * total / ctas;
  auto locate = [&] {
    if (mine > 0 && p0 >= q.pre && p0 < q.pre + mine) sc.at[0] = q;
    if (mine > 0 && p1 >= q.pre && p1 < q.pre + mine) sc.at[1] = q;
  };
  if (a.batch <= PAIR_THREADS) {
    locate();
  } else {
    __syncthreads();                               // the totals have been read
    begin();
    for (int s0 = 0; s0 < a.batch; s0 += PAIR_THREADS) {
      chunk(s0);
      locate();
    }
  }
  __syncthreads();
  if (lane == 0 && warp < 2) {                     // warp 0: the start, warp 1: the end
    const long long pos = warp ? p1 : p0;
    PairPart& r = sc.part;
    if (pos >= total) {
      r.end_s0 = total;
      r.end_j = 0;
    } else {
      const Row& f = sc.at[warp];
      const long long one = f.upto(a, f.tiles_of(a));
      const int g = (int)((pos - f.pre) / one);
      const long long rem = (pos - f.pre) - g * one;
      int lo = 0, hi = f.tiles_of(a);              // the item: upto(lo) <= rem < upto(hi)
      while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (f.upto(a, mid) <= rem) lo = mid; else hi = mid;
      }
      const long long s0 = f.pre + g * one + f.upto(a, lo);
      const long long work = f.upto(a, lo + 1) - f.upto(a, lo);
      const int tiles = key_tiles(a, f, lo);
      const int j = cut_at(a, pos, s0, work, tiles, total / ctas);
      if (warp == 0) {
        r.q = f;
        r.g = g;
        r.t = lo;
        r.j = j;
        r.total = total;
        r.ctas = ctas;
      } else {
        r.end_s0 = j == tiles ? s0 + work : s0;
        r.end_j = j == tiles ? 0 : j;
      }
    }
  }
  __syncthreads();
}

// The items of a CTA's part, one after another: row tiles at tokens tok0 and tok0 + tpt, the
// steps of 64 keys that each takes (the last is left out where a tile's own keys end in the
// first half of a key tile), and the key tiles [ja, jb) of the item's `tiles` that this CTA
// visits. The loader walks and hands the items to the other warps.
struct PairWalk {
  const AttnArgs& a;
  const PartScan& sc;
  const PairPart& p;
  Row q;
  int i, g, t, tok0, kvh, h0, np, tiles, ja, jb;
  long long s0, work;
  bool more;

  MARS_DEV PairWalk(const AttnArgs& a_, const PartScan& sc_)
      : a(a_), sc(sc_), p(sc_.part), q(p.q), i(0), g(p.g), t(p.t) {
    if (sc.count >= 0) {
      listed();
      return;
    }
    item();
    ja = p.j;
    if (ja == tiles) next(); else end();
  }
  MARS_DEV void item() {
    np = q.prefix();
    tiles = key_tiles(a, q, t);
    tok0 = t * a.rows;
    kvh = g / a.ngrp;
    h0 = g * a.gp;
    ja = 0;
  }
  MARS_DEV void end() {
    const long long one = q.upto(a, q.tiles_of(a)), off = q.upto(a, t);
    s0 = q.pre + g * one + off;
    work = q.upto(a, t + 1) - off;
    jb = s0 == p.end_s0 ? p.end_j : tiles;
    more = s0 < p.end_s0 || (s0 == p.end_s0 && p.end_j > ja);
  }
  MARS_DEV void listed() {
    more = i < sc.count;
    if (!more) return;
    const ListItem l = sc.list[i];
    q = Row{l.s, l.base, l.n, cached_keys(a, l.s), 0};
    t = l.tg / (a.hkv * a.ngrp);
    g = l.tg % (a.hkv * a.ngrp);
    item();
    jb = tiles;
  }
  MARS_DEV void next() {
    if (sc.count >= 0) {
      ++i;
      listed();
      return;
    }
    if (++t == q.tiles_of(a)) {
      t = 0;
      if (++g == a.hkv * a.ngrp) {
        g = 0;
        const long long after = q.pre + (long long)a.hkv * a.ngrp * q.upto(a, q.tiles_of(a));
        q.pre = after;
        do {                                       // the next sequence with rows
          if (++q.s >= a.batch || after >= p.end_s0 + (p.end_j > 0)) {
            more = false;
            return;
          }
          q.base += q.n;
          q.n = max(min(max(a.cu[q.s + 1], 0), a.total), q.base) - q.base;
        } while (q.n == 0);
        q.P = cached_keys(a, q.s);
      }
    }
    item();
    end();
  }
  MARS_DEV int first_token(int x) const { return tok0 + x * a.tpt; }
  // steps of row tile x over all the item's key tiles; 0 if it has no rows
  MARS_DEV int all_steps(int x) const {
    if (first_token(x) >= q.n) return 0;
    return 2 * np + (min(first_token(x) + a.tpt, q.n) - 1) / kStep + 1;
  }
  // its steps [first, last) in this CTA's key tiles
  MARS_DEV int steps(int x) const { return max(min(all_steps(x), 2 * jb) - 2 * ja, 0); }
  MARS_DEV PairItem describe() const {
    PairItem d{q.s, q.base, q.n, q.P, np, tok0, h0, tiles, ja, jb,
               {all_steps(0), all_steps(1)}, {steps(0), steps(1)}, 0, 0};
    if (ja > 0 || jb < tiles) {
      const long long part = p.total / p.ctas;
      auto cut = [&](long long c) {
        return cut_at(a, c * p.total / p.ctas, s0, work, tiles, part);
      };
      long long c1 = s0 * p.ctas / p.total;
      while (c1 * p.total / p.ctas <= s0 || cut(c1) == 0) ++c1;
      d.c1 = (int)c1;
      d.cuts = 1;
      while (c1 + d.cuts < p.ctas && (c1 + d.cuts) * p.total / p.ctas < s0 + work &&
             cut(c1 + d.cuts) < tiles)
        ++d.cuts;
    }
    return d;
  }
};

template <int D>
constexpr int PART4 = BQ * D / 4 + BQ / 2;       // float4 of a partial

// Partials: [CTA][0: a part that starts inside its item, 1: at its start][row tile], each D / 4
// rows of 128 float4 (a thread per row of the tile: its loads and stores are coalesced) and 128
// pairs of m and l.
template <int D>
MARS_DEV float4* partial(const AttnArgs& a, int cta, bool inside, int x) {
  return reinterpret_cast<float4*>(a.part) +
         (((size_t)cta * 2 + (inside ? 0 : 1)) * 2 + x) * PART4<D>;
}

// The next item of the loader's queue (number i), copied; false if the wait gave up. The
// caller then arrives on item_empty, once per warp.
MARS_DEV bool take_item(PairBar& bar, int i, PairItem& it, volatile int* ab, int32_t* status) {
  if (!sm100::mbar_wait(&bar.item_full[i % kItems], (i / kItems) & 1, ab, status)) return false;
  it = bar.items[i % kItems];
  return true;
}

template <int D>
__global__ void __launch_bounds__(PAIR_THREADS, 1)
pair_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
            const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_kp,
            const __grid_constant__ CUtensorMap tm_vp, AttnArgs a) {
  using namespace sm100;
  using S = PairSmem<D>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ PairBar bar;
  __shared__ PartScan scan;
  const uint32_t raw = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + (((raw + 1023u) & ~1023u) - raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int* ab = &bar.abort;
  if (threadIdx.x == 0) {
    bar.abort = 0;
    for (int i = 0; i < kKSlots; ++i) {
      mbar_init(&bar.k_full[i], 1);
      mbar_init(&bar.k_empty[i], 2);
    }
    for (int i = 0; i < kVSlots; ++i) {
      mbar_init(&bar.v_full[i], 1);
      mbar_init(&bar.v_empty[i], 1);
    }
    mbar_init(&bar.drain[2], 1);
    for (int i = 0; i < kItems; ++i) {
      mbar_init(&bar.item_full[i], 1);
      mbar_init(&bar.item_empty[i], 3 + 8);        // both S issuers, the PV issuer, softmax warps
    }
    for (int x = 0; x < 2; ++x) {
      mbar_init(&bar.q_full[x], 1);
      mbar_init(&bar.q_empty[x], 1);
      for (int i = 0; i < 2; ++i) {
        mbar_init(&bar.s_full[x][i], 1);
        mbar_init(&bar.p_full[x][i], 128);
        mbar_init(&bar.pv_done[x][i], 1);
      }
      mbar_init(&bar.drain[x], 1);
      mbar_init(&bar.stored[x], 128);
      mbar_init(&bar.told[x], 1);
    }
    fence_barrier_init();
  }
  static_assert(sizeof(ListScratch) <= S::TOTAL - 1024, "the scratch fits the tiles' place");
  find_part(a, scan, *reinterpret_cast<ListScratch*>(smem));
  if (scan.count == 0 || (scan.count < 0 && scan.part.ctas == 0)) return;
  fence_proxy_async_smem();                            // before copies into the scratch's place
  if (warp == 1) {
    tmem_alloc(&bar.tmem_base, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, bar.tmem_base, 0);

  if (warp < 4) {
    regs_lower<PAIR_WG0_REGS>();
    if (warp == 0) {
      // ------------------------------------------------------------------- loader
      int g = 0, flags = 0;                            // key tiles loaded
      bool ok = true;
      int ni = 0, nk = 0, nv = 0;                      // items handed over; K and V tiles issued
      auto publish = [&](const PairItem& d) {
        int good = 1;
        if (lane == 0) {
          good = mbar_wait(&bar.item_empty[ni % kItems], ((ni / kItems) & 1) ^ 1, ab, a.status);
          if (good) {
            bar.items[ni % kItems] = d;
            mbar_arrive(&bar.item_full[ni % kItems]);
          }
        }
        ++ni;
        return __shfl_sync(0xffffffffu, good, 0) != 0;
      };
      for (PairWalk it(a, scan); it.more && ok; it.next()) {
        if (!(ok = publish(it.describe()))) break;
        const int32_t* bt = a.block_table ? a.block_table + (size_t)it.q.s * a.max_pages : nullptr;
        // this lane's page of prefix tile j, read one tile ahead
        auto entry = [&](int j) -> int {
          const int lp = j * kPagesPerTile + lane;
          return j < it.np && lane < kPagesPerTile && lp < a.max_pages ? bt[lp] : -1;
        };
        int next = entry(it.ja);
        for (int j = it.ja; j < it.jb && ok; ++j) {
          const int e = next;
          next = entry(j + 1);
          for (int v = 1; v >= 0; --v) {                 // V first, see the softmax warps' clearing
            const int n = v ? kVSlots : kKSlots, st = g % n;
            uint64_t* full = v ? &bar.v_full[st] : &bar.k_full[st];
            uint64_t* empty = v ? &bar.v_empty[st] : &bar.k_empty[st];
            int good = 1;
            if (lane == 0) {
              good = mbar_wait(empty, ((g / n) & 1) ^ 1, ab, a.status);
              if (good) mbar_arrive_expect_tx(full, S::TILE);
            }
            ok = __shfl_sync(0xffffffffu, good, 0) != 0;
            if (!ok) break;
            (v ? nv : nk) = g + 1;
            uint8_t* dst = smem + (v ? S::OFF_V : S::OFF_K) + st * S::TILE;
            if (j < it.np) {
              if (lane < kPagesPerTile) {
                // as in packed_rows_kernel: a page that may not be read loads page 0
                int page = 0;
                if (e >= 0 && e < a.num_pages)
                  page = e;
                else if (j * BKV + lane * kPageSize < it.q.P)
                  flags |= MARS_ST_NOPAGE;
                const int row = a.num_pages > 0 ? (page * a.hkv + it.kvh) * kPageSize : kPageSize;
                for (int x = 0; x < D / 64; ++x)
                  tma_load_2d(dst + x * (BKV * 128) + lane * (kPageSize * 128), v ? &tm_vp : &tm_kp,
                              full, x * 64, row);
              }
            } else if (lane == 0) {
              for (int x = 0; x < D / 64; ++x)
                tma_load_3d(dst + x * (BKV * 128), v ? &tm_v : &tm_k, full, x * 64, it.kvh,
                            it.q.base + (j - it.np) * BKV);
            }
          }
          ++g;
        }
      }
      if (ok) publish(PairItem{});                     // no more items
      if (flags && a.status) atomicOr(a.status, flags);
      // wait (bounded) for the copies still in flight, and for every arrival that releases a slot
      if (lane == 0) {
        for (int k = nk - 1; k >= max(nk - kKSlots, 0); --k) {
          mbar_wait(&bar.k_full[k % kKSlots], (k / kKSlots) & 1, nullptr, a.status);
          if (ok) mbar_wait(&bar.k_empty[k % kKSlots], (k / kKSlots) & 1, ab, a.status);
        }
        for (int k = nv - 1; k >= max(nv - kVSlots, 0); --k) {
          mbar_wait(&bar.v_full[k % kVSlots], (k / kVSlots) & 1, nullptr, a.status);
          if (ok) mbar_wait(&bar.v_empty[k % kVSlots], (k / kVSlots) & 1, ab, a.status);
        }
      }
      __syncwarp();
    } else if (warp != 2) {
      // ------------------------------- warp 1, 3: Q_x loads, S_x = Q_x K^T for x = 0, 1
      const int x = warp >> 1;
      if (elect_one()) {
        const uint32_t idesc = idesc_bf16_f32(BQ, kStep, false);
        const uint64_t qd = sdesc_sw128(smem_u32(smem + S::OFF_Q + x * S::TILE), 16, 1024);
        const uint32_t ts = tmem + S::TM_S + x * BKV;
        int g = 0, c = 0, items = 0;                   // key tiles; steps and items of x
        bool ok = true;
        PairItem it;
        for (int i = 0; ok && (ok = take_item(bar, i, it, ab, a.status)) && it.jb; ++i) {
          mbar_arrive(&bar.item_empty[i % kItems]);
          const int steps = x ? it.steps[1] : it.steps[0];
          if (steps) {
            // Q_x is replaced once the S MMAs of its previous item have completed
            if (items && !(ok = mbar_wait(&bar.q_empty[x], (items - 1) & 1, ab, a.status))) break;
            mbar_arrive_expect_tx(&bar.q_full[x], a.gp * a.tpt * 128 * (D / 64));
            for (int cc = 0; cc < D / 64; ++cc)
              tma_load_3d(smem + S::OFF_Q + x * S::TILE + cc * (BQ * 128), &tm_q, &bar.q_full[x],
                          cc * 64, it.h0, it.base + it.tok0 + x * a.tpt);
            if (!(ok = mbar_wait(&bar.q_full[x], items & 1, ab, a.status))) break;
            ++items;
          }
          for (int j = 0; j < it.jb - it.ja && ok; ++j, ++g) {
            const int st = g % kKSlots;
            if (!(ok = mbar_wait(&bar.k_full[st], (g / kKSlots) & 1, ab, a.status))) break;
            const uint64_t kd = sdesc_sw128(smem_u32(smem + S::OFF_K + st * S::TILE), 16, 1024);
            for (int u = 2 * j; u < min(2 * j + 2, steps); ++u, ++c) {
              const int b = c & 1;
              // the PV of two steps before has read P out of the buffer
              if (c >= 2 && !(ok = mbar_wait(&bar.pv_done[x][b], ((c >> 1) - 1) & 1, ab, a.status)))
                break;
              tc_fence_after();
              const uint64_t kh = sdesc_advance(kd, (u & 1) * (kStep * 128));
#pragma unroll
              for (int k = 0; k < D / 16; ++k) {
                const uint32_t off = (k >> 2) * (BQ * 128) + (k & 3) * 32;
                mma_bf16_ss(ts + b * kStep, sdesc_advance(qd, off), sdesc_advance(kh, off), idesc,
                            k != 0);
              }
              mma_commit(&bar.s_full[x][b]);
              if (u == steps - 1) mma_commit(&bar.q_empty[x]);
            }
            if (!ok) break;
            // one of the two arrivals for a K slot: by a commit only where this thread's MMAs read
            // it (a commit with nothing before it to wait for could arrive after the CTA has ended)
            if (2 * j < steps)
              mma_commit(&bar.k_empty[st]);
            else
              mbar_arrive(&bar.k_empty[st]);
          }
        }
        // wait (bounded) for this thread's MMAs and Q copies
        if (c > 0) {
          mma_commit(&bar.drain[x]);
          mbar_wait(&bar.drain[x], 0, nullptr, a.status);
        }
        if (items) {
          mbar_wait(&bar.q_full[x], (items - 1) & 1, nullptr, a.status);
          if (ok) mbar_wait(&bar.q_empty[x], (items - 1) & 1, nullptr, a.status);
        }
      }
    } else {
      // ------------------------------------------------------------------ O += P V
      if (elect_one()) {
        const uint32_t idesc = idesc_bf16_f32(BQ, D, true);
        int g = 0, done[2] = {0, 0};
        bool ok = true;
        PairItem it;
        for (int i = 0; ok && (ok = take_item(bar, i, it, ab, a.status)) && it.jb; ++i) {
          mbar_arrive(&bar.item_empty[i % kItems]);
          const int steps[2] = {it.steps[0], it.steps[1]};
          for (int j = 0; j < it.jb - it.ja && ok; ++j, ++g) {
            const int st = g % kVSlots;
            if (!(ok = mbar_wait(&bar.v_full[st], (g / kVSlots) & 1, ab, a.status))) break;
            const uint64_t vd =
                sdesc_sw128(smem_u32(smem + S::OFF_V + st * S::TILE), BKV * 128, 1024);
            for (int hx = 0; hx < 4; ++hx) {
              const int h = hx >> 1, x = hx & 1, u = 2 * j + h;
              if (u >= (x ? steps[1] : steps[0])) continue;
              const int c = done[x], b = c & 1;
              if (!(ok = mbar_wait(&bar.p_full[x][b], (c >> 1) & 1, ab, a.status))) break;
              tc_fence_after();
#pragma unroll
              for (int k = 0; k < kStep / 16; ++k)
                mma_bf16_ts(tmem + S::TM_O + x * BKV,
                            tmem + S::TM_S + x * BKV + b * kStep + S::P_OFF + k * 8,
                            sdesc_advance(vd, h * (kStep * 128) + k * 2048), idesc, (u | k) != 0);
              mma_commit(&bar.pv_done[x][b]);
              ++done[x];
            }
            if (!ok) break;
            mma_commit(&bar.v_empty[st]);
          }
        }
        if (done[0] + done[1] > 0) {                     // wait (bounded) for this thread's MMAs
          mma_commit(&bar.drain[2]);
          mbar_wait(&bar.drain[2], 0, nullptr, a.status);
        }
      }
    }
  } else {
    // -------------------------------------------------------------- softmax, output
    regs_raise<PAIR_SOFTMAX_REGS>();
    const int x = warp >= 8, quad = warp & 3, row = quad * 32 + lane;
    const uint32_t lane_off = (uint32_t)(quad * 32) << 16;
    auto warp_wait = [&](uint64_t* b, uint32_t parity) -> bool {
      return __all_sync(0xffffffffu, mbar_wait(b, parity, ab, a.status));
    };
    const uint32_t s_addr = tmem + S::TM_S + x * BKV + lane_off;
    const uint32_t o_addr = tmem + S::TM_O + x * BKV + lane_off;
    int g = 0, done = 0, parts = 0, tells = 0;
    bool ok = true;
    RowsPolicy<D> pol;
    pol.a = &a;
    pol.set_row(row);
    pol.j0 = pol.split = 0;
    PairItem it;
    for (int i = 0; ok; ++i) {
      if (!(ok = __all_sync(0xffffffffu, take_item(bar, i, it, ab, a.status)))) break;
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar.item_empty[i % kItems]);
      if (!it.jb) break;
      const int steps = x ? it.steps[1] : it.steps[0];
      if ((x ? it.all[1] : it.all[0]) == 0) {
        g += it.jb - it.ja;
        continue;
      }
      pol.bt_row = a.block_table ? a.block_table + (size_t)it.s * a.max_pages : nullptr;
      pol.base = it.base;
      pol.n = it.n;
      pol.tok0 = it.tok0 + x * a.tpt;
      pol.P = it.P;
      pol.np = it.np;
      pol.h0 = it.h0;
      pol.j0 = it.ja;
      pol.last_tok = min(it.tok0 + a.rows, it.n) - 1;   // of the item: neither tile reads on
      const int tok = pol.tok0 + pol.trow;              // this thread's token
      const flash::RowVis vis{tok + 1, 0, -1};
      float m = -INFINITY, l = 0.f;
      typename RowsPolicy<D>::Tile tile, next = pol.tile(0);
#pragma unroll 1
      for (int u = 0; u < steps; ++u, ++done) {
        const int h = u & 1, b = done & 1;
        if (h == 0) {
          tile = next;
          if (u + 2 < steps) next = pol.tile(u / 2 + 1);
        }
        const uint32_t sb = s_addr + b * kStep;
        if (!(ok = warp_wait(&bar.s_full[x][b], (done >> 1) & 1))) break;
        tc_fence_after();
        uint32_t v[kStep];
#pragma unroll
        for (int c = 0; c < kStep / 32; ++c)
          tmem_ld32(sb + c * 32, *reinterpret_cast<uint32_t(*)[32]>(v + c * 32));
        tmem_ld_wait();
        if (!tile.full) {
          const flash::ColRange cr = pol.cols(vis, tile);
#pragma unroll
          for (int c = 0; c < kStep / 32; ++c) {
            const uint32_t mk = flash::chunk_mask(cr, 2 * h + c);
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (!((mk >> e) & 1u)) v[c * 32 + e] = 0xff800000u;
          }
        }
        // P with the maximum so far, while the step's own maximum is being found; only where
        // that one is larger by more than 2^8 (the lazy rescale of flash_tc.cuh) is it formed
        // again
        float2 acc[2];
        uint32_t packed[32];
        acc[0] = acc[1] = make_float2(0.f, 0.f);
        flash::exp2_pack64(v, 0, a.scale_log2, m == -INFINITY ? 0.f : -m, packed, acc);
        const float tmax = flash::row_max_log2(v, a.scale_log2);
        const bool raise = tmax > m + flash::kRescaleLog2;
        if (__any_sync(0xffffffffu, raise)) {
          const bool rescale = raise && m != -INFINITY;
          if (__any_sync(0xffffffffu, rescale)) {
            // the PV of the step before must have landed in O
            if (!(ok = warp_wait(&bar.pv_done[x][b ^ 1], ((done - 1) >> 1) & 1))) break;
            tc_fence_after();
            const float alpha = rescale ? flash::ex2_approx(m - tmax) : 1.f;
            l *= alpha;
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
              uint32_t o[32];
              tmem_ld32(o_addr + c * 32, o);
              tmem_ld_wait();
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
              tmem_st32(o_addr + c * 32, o);
            }
            tmem_st_wait();
          }
          if (raise) m = tmax;
          acc[0] = acc[1] = make_float2(0.f, 0.f);
          flash::exp2_pack64(v, 0, a.scale_log2, m == -INFINITY ? 0.f : -m, packed, acc);
        }
        if (tile.clear) {
          // V rows that no row of the item may read (flash_tc.cuh, kClearRows), the step's half
          // of the tile; both row tiles' threads write the same zeros. K of this tile has
          // landed, so V's copy, issued before it, is in this phase of its slot or later.
          const int gv = g + u / 2, st = gv % kVSlots;
          if (!(ok = warp_wait(&bar.v_full[st], (gv / kVSlots) & 1))) break;
          if (row / kStep == h && !pol.key_read(tile, row)) {
            uint8_t* vr = smem + S::OFF_V + st * S::TILE + row * 128;
#pragma unroll
            for (int c = 0; c < D / 64; ++c)
#pragma unroll
              for (int q = 0; q < 8; ++q)
                *reinterpret_cast<uint4*>(vr + c * (BKV * 128) + q * 16) = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
        }
        tmem_st32(sb + S::P_OFF, packed);
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive_warp(&bar.p_full[x][b]);
        l += (acc[0].x + acc[0].y) + (acc[1].x + acc[1].y);
      }
      if (!ok) break;
      g += it.jb - it.ja;
      // there were steps: a part has four key tiles or more, and begins as many before the end of
      // the item, which is at most one behind that of either row tile
      if (!(ok = warp_wait(&bar.pv_done[x][(done - 1) & 1], ((done - 1) >> 1) & 1))) break;
      tc_fence_after();
      // where this thread's row goes, in elements (-1: no token)
      const long long at =
          pol.trow < a.tpt && tok < it.n
              ? (((long long)it.base + tok) * a.hq + it.h0 + pol.hrow) * D : -1;
      const bool whole = it.ja == 0 && it.jb == it.tiles;
      const int own = blockIdx.x - (it.c1 - 1);        // this part of a divided item
      bool write = true;
      if (!whole) {
        // A divided item: its last part to finish merges. A part that finds all others finished
        // does so without writing its own partial; the others write theirs and count it.
        int32_t* ticket = a.tickets + 2 * it.c1 + x;
        auto tell = [&](auto f) {                      // one thread's answer for all 128
          if (quad == 0 && lane == 0) {
            bar.last[x][tells] = f();
            mbar_arrive(&bar.told[x]);
          }
          ok = warp_wait(&bar.told[x], tells & 1);
          const bool last = ok && *reinterpret_cast<volatile int*>(&bar.last[x][tells]) != 0;
          ++tells;
          return last;
        };
        write = tell([&] { return *reinterpret_cast<volatile int32_t*>(ticket) == it.cuts; });
        if (!ok) break;
        if (!write) {
          float4* rec = partial<D>(a, blockIdx.x, it.ja > 0, x);
          reinterpret_cast<float2*>(rec + BQ * D / 4)[row] = make_float2(m, l);
#pragma unroll 1
          for (int c = 0; c < D / 32; ++c) {
            uint32_t o[32];
            tmem_ld32(o_addr + c * 32, o);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 32; e += 4)
              rec[(c * 8 + e / 4) * BQ + row] =
                  make_float4(__uint_as_float(o[e]), __uint_as_float(o[e + 1]),
                              __uint_as_float(o[e + 2]), __uint_as_float(o[e + 3]));
          }
          __threadfence();
          mbar_arrive_warp(&bar.stored[x]);
          if (quad == 0 && !(ok = warp_wait(&bar.stored[x], parts & 1))) break;
          ++parts;
          write = tell([&] { return atomicAdd(ticket, 1) == it.cuts; });
          if (!ok) break;
        }
        if (write) __threadfence();
      }
      if (write) {
        auto rec_of = [&](int k) { return partial<D>(a, it.c1 - 1 + k, k > 0, x); };
        auto ml_of = [&](int k) {
          if (k == own) return make_float2(m, l);
          return __ldcg(reinterpret_cast<const float2*>(rec_of(k) + BQ * D / 4) + row);
        };
        // weights of the parts' O; those of the first two are kept, an item has rarely more
        float mw = m, lw = l, w0 = 1.f, w1 = 0.f;
        auto weight = [&](float mk) { return mk > -INFINITY ? exp2f(mk - mw) : 0.f; };
        if (!whole) {
          const float2 a0 = ml_of(0), a1 = ml_of(1);
          mw = fmaxf(a0.x, a1.x);
          for (int k = 2; k <= it.cuts; ++k) mw = fmaxf(mw, ml_of(k).x);
          w0 = weight(a0.x);
          w1 = weight(a1.x);
          lw = a0.y * w0 + a1.y * w1;
          for (int k = 2; k <= it.cuts; ++k) {
            const float2 r = ml_of(k);
            lw += r.y * weight(r.x);
          }
        }
        const float inv = reciprocal(lw);
        if (a.lse && at >= 0)
          a.lse[(size_t)(it.h0 + pol.hrow) * a.total + it.base + tok] = statistic(mw, lw);
        // 64 columns at a time, exchanged in groups of 8 lanes so that these write 128 bytes of a
        // row (a thread writing its own row took 5,000 cycles per item; staging in shared memory
        // would take a fifth of the ring, which costs 9 %)
#pragma unroll 1
        for (int c = 0; c < D / 64; ++c) {
          float o[64];
          if (whole) {
#pragma unroll
            for (int k = 0; k < 2; ++k)
              tmem_ld32(o_addr + c * 64 + 32 * k, *reinterpret_cast<uint32_t(*)[32]>(o + 32 * k));
            tmem_ld_wait();
          } else {
#pragma unroll
            for (int e = 0; e < 64; ++e) o[e] = 0.f;
            for (int k = 0; k <= it.cuts; ++k) {
              const float wt = k == 0 ? w0 : k == 1 ? w1 : weight(ml_of(k).x);
              if (k == own) {
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                  uint32_t v[32];
                  tmem_ld32(o_addr + c * 64 + 32 * q, v);
                  tmem_ld_wait();
#pragma unroll
                  for (int e = 0; e < 32; ++e) o[32 * q + e] += __uint_as_float(v[e]) * wt;
                }
                continue;
              }
              const float4* r = rec_of(k) + c * 16 * BQ + row;
#pragma unroll
              for (int e = 0; e < 64; e += 4) {
                const float4 v4 = __ldcg(r + (e / 4) * BQ);
                o[e] += v4.x * wt;
                o[e + 1] += v4.y * wt;
                o[e + 2] += v4.z * wt;
                o[e + 3] += v4.w * wt;
              }
            }
          }
          packed::store_rows<64>(a.o + c * 64, at, lane, [&](int e) { return o[e] * inv; });
        }
      }
      tc_fence_before();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Tensor map of [total][heads][D] rows with a row pitch of `stride` elements.
bool map_rows(CUtensorMap* m, const void* base, int d, int heads, int total, long long stride,
              uint32_t box_heads, uint32_t box_rows) {
  const uint64_t dims[3] = {(uint64_t)d, (uint64_t)heads, (uint64_t)total};
  const uint64_t str[2] = {(uint64_t)d * 2, (uint64_t)stride * 2};
  const uint32_t box[3] = {64, box_heads, box_rows};
  return encode_tmap_bf16(m, base, 3, dims, str, box);
}

template <int D>
cudaError_t launch_rows(const PackedAttn& p, const PackedPlan& plan, AttnArgs& a,
                        void* workspace, cudaStream_t stream) {
  using S = flash::Smem<D, 0, kVStages>;
  static_assert(S::TOTAL + sizeof(flash::Barriers) <= 227 * 1024, "layout fits shared memory");
  CUtensorMap tq, tk, tv, tkp, tvp;
  if (!map_rows(&tq, p.q, D, p.hq, p.total, p.q_stride, a.gp, a.tpt) ||
      !map_rows(&tk, p.k, D, p.hkv, p.total, p.k_stride, 1, BKV) ||
      !map_rows(&tv, p.v, D, p.hkv, p.total, p.v_stride, 1, BKV))
    return cudaErrorInvalidValue;
  tkp = tk;
  tvp = tv;
  if (p.seq_lens) {
    // an empty pool is never read: one page over q, and the loader's boxes start past its end
    const bool any = p.num_pages > 0;
    const uint64_t dims[2] = {(uint64_t)D, any ? (uint64_t)p.num_pages * p.hkv * kPageSize
                                               : (uint64_t)kPageSize};
    const uint64_t str[1] = {(uint64_t)D * 2};
    const uint32_t box[2] = {64, (uint32_t)kPageSize};
    if (!encode_tmap_bf16(&tkp, any ? p.k_pool : p.q, 2, dims, str, box) ||
        !encode_tmap_bf16(&tvp, any ? p.v_pool : p.q, 2, dims, str, box))
      return cudaErrorInvalidValue;
  }
  if (plan.pair) {
    using SP = PairSmem<D>;
    static_assert(SP::TOTAL + sizeof(PairBar) + sizeof(PartScan) <= 227 * 1024,
                  "pair layout fits shared memory");
    static std::atomic<int> attr_pair[64];
    cudaError_t e = set_smem_limit_once(pair_kernel<D>, SP::TOTAL, attr_pair);
    if (e != cudaSuccess) return e;
    if (a.can_split) {
      e = cudaMemsetAsync(a.tickets, 0, plan.ctas * 2 * sizeof(int32_t), stream);
      if (e != cudaSuccess) return e;
    }
    pair_kernel<D><<<(unsigned)plan.ctas, PAIR_THREADS, SP::TOTAL, stream>>>(tq, tk, tv, tkp,
                                                                             tvp, a);
    count_launches(1);
    return cudaGetLastError();
  }
  static std::atomic<int> attr[64];
  const cudaError_t ea = set_smem_limit_once(packed_rows_kernel<D>, S::TOTAL, attr);
  if (ea != cudaSuccess) return ea;
  packed_rows_kernel<D><<<(unsigned)plan.ctas, flash::NUM_THREADS, S::TOTAL, stream>>>(
      tq, tk, tv, tkp, tvp, a);
  count_launches(1);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || plan.nsplit == 1) return e;
  const long long warps = (long long)p.total * p.hq;
  packed_merge_kernel<D><<<(unsigned)((warps + 7) / 8), 256, 0, stream>>>(a);
  count_launches(1);
  return cudaGetLastError();
}

}  // namespace

PackedPlan plan_packed(int batch, int total, int hq, int hkv, int d, int max_len) {
  PackedPlan p{};
  const int G = hq / hkv;
  p.gp = G <= BQ ? G : 1;
  p.tpt = BQ / p.gp;
  const long long items = packed::max_tiles(batch, total, p.tpt) * hkv * (G / p.gp);
  const int tiles = packed::key_tiles(max_len) + 1;
  // Two row tiles per item where sequences have more rows than one on average and the items
  // fill the GPU. Both forms, in us, 28 heads over 4 of 128 (rows | pair; the rule's border is at
  // about 1,330 rows): one prompt of 512 rows 16 | 23, 1,024: 27 | 31, 1,300: 33 | 34, 1,400: 37 | 36,
  // 2,048: 51 | 43; six and eight prompts of 200: 22.5 | 23.6 and 28.7 | 27.6; chunks of 100 over
  // 1,000 cached, ten and fourteen: 37 | 46 and 49 | 50; one chunk over 8,192 cached of 256 rows 47 |
  // 62, 512: 90 | 77, 1,024: 131 | 118, 1,300: 137 | 136, 1,400: 195 | 146. 14 heads over 2 of 64
  // (border at about 2,700 rows): prompts of 2,600 rows 39 | 42, 2,800: 45 | 45, 4,096: 70 | 63; one chunk
  // over 8,192 cached of 512 rows 45 | 50, 2,800: 199 | 144.
  const long long pairs = packed::max_tiles(batch, total, 2 * p.tpt) * hkv * (G / p.gp);
  if (total > (long long)batch * p.tpt && pairs >= num_sms()) {
    p.pair = true;
    p.rows = 2 * p.tpt;
    p.nsplit = 1;
    p.split_tiles = tiles;
    p.items = pairs;
    p.can_split = tiles >= 2 * kMinPart;
    p.ctas = num_sms();
    p.ticket_bytes = packed::align256(p.ctas * 2 * sizeof(int32_t));
    if (p.can_split)
      p.ws_bytes = p.ticket_bytes + (size_t)p.ctas * 4 * (BQ * (d + 2)) * sizeof(float);
    return p;
  }
  // Splits: with few items as many as fill the SMs once; with about as many as SMs, or more, so
  // that there are two to three CTAs per SM, each with a good part of a list, to even lengths out
  // (132 items of 16 to 61 key tiles, whole: 82 us, in 2, 3, 4 parts: 85, 74, 78).
  const long long once = std::min<long long>(num_sms() / items, tiles / kMinSplitTiles);
  const long long even = items <= num_sms() / 2 ? 1
      : std::min<long long>(3LL * num_sms() / items, tiles / kEvenSplitTiles);
  const long long nsplit = std::max(1LL, std::max(once, even));
  p.split_tiles = (int)((tiles + nsplit - 1) / nsplit);
  p.nsplit = (tiles + p.split_tiles - 1) / p.split_tiles;
  p.items = p.ctas = items * p.nsplit;
  p.ws_bytes =
      p.nsplit > 1 ? (size_t)p.nsplit * total * hq * (size_t)(d + 4) * sizeof(float) : 0;
  return p;
}

cudaError_t launch_packed_attn(const PackedAttn& p, const PackedPlan& plan, void* workspace,
                               cudaStream_t stream) {
  AttnArgs a{};
  a.cu = p.cu;
  a.seq_lens = p.seq_lens;
  a.block_table = p.block_table;
  a.num_pages = p.num_pages;
  a.max_pages = p.max_pages;
  a.batch = p.batch;
  a.total = p.total;
  a.hq = p.hq;
  a.hkv = p.hkv;
  a.gp = plan.gp;
  a.tpt = plan.tpt;
  a.ngrp = p.hq / p.hkv / plan.gp;
  a.nsplit = plan.nsplit;
  a.split_tiles = plan.split_tiles;
  a.scale_log2 = p.scale * 1.4426950408889634f;
  a.o = p.o;
  a.lse = p.lse;
  a.rows = plan.rows;
  a.can_split = plan.can_split;
  a.tickets = static_cast<int32_t*>(workspace);
  a.part = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + plan.ticket_bytes);
  a.status = p.status;
  return p.d == 64 ? launch_rows<64>(p, plan, a, workspace, stream)
                   : launch_rows<128>(p, plan, a, workspace, stream);
}

}  // namespace mars
