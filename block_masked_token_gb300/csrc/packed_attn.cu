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
// With few tiles and long key lists the list is cut into splits: each CTA writes an
// unnormalised partial (m in log2 units, l, O) and a second kernel merges them.
//
// Where the rows are many, pair_kernel takes two row tiles per CTA instead (see there).
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
constexpr int kVStages = 3;                      // as in the decode kernel: no O staging area
constexpr int kMinSplitTiles = 4;                // key tiles a split takes at least

struct AttnArgs {
  const int32_t* cu;
  const int32_t* seq_lens;     // NULL: no cache
  const int32_t* block_table;
  int num_pages, max_pages;
  int batch, total, hq, hkv, gp, tpt, ngrp, nsplit, split_tiles;
  float scale_log2;
  uint16_t* o;                 // [total][hq][D] bf16
  float* lse;                  // [hq][total] or NULL
  float* part;                 // [nsplit][total][hq][D + 4] with several splits
  int32_t* status;
};

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
      if (col == 0 && a->lse) a->lse[(size_t)h * a->total + tok] = l > 0.f ? m + log2f(l) : -INFINITY;
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
  const packed::Seq sq = packed::find_tile(a.cu, a.batch, a.total, a.tpt, 0, id, bad);
  if (bad && threadIdx.x == 0 && a.status) atomicOr(a.status, MARS_ST_BADSEQ);
  if (sq.s < 0) return;

  RowsPolicy<D> pol;
  pol.a = &a;
  pol.base = sq.base;
  pol.n = sq.n;
  pol.tok0 = sq.tile * a.tpt;
  // cached keys; a length that the table cannot hold is cut to what it can
  const int cached = a.seq_lens ? a.seq_lens[sq.s] : 0;
  pol.P = (int)max(0LL, min((long long)cached, (long long)a.max_pages * kPageSize));
  if (pol.P != cached && threadIdx.x == 0 && a.status) atomicOr(a.status, MARS_ST_OVERFLOW);
  pol.np = (pol.P + BKV - 1) / BKV;
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
        rec[1] = 0.f;
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
    if (warp == 1 && lane == 0)
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
  bool bad;
  // rows behind the last sequence have no partials and stay as they are
  const packed::Seq sq = packed::find_tile(a.cu, a.batch, a.total, 1, 0, INT_MAX, bad);
  const int first = min(max(a.cu[0], 0), a.total);
  if (tok < first || tok >= sq.base) return;
  const size_t rec = D + 4, step = (size_t)a.total * a.hq * rec;
  const float* base = a.part + ((size_t)tok * a.hq + h) * rec;
  float m = -INFINITY;
  for (int sp = 0; sp < a.nsplit; ++sp) m = fmaxf(m, base[sp * step]);
  float l = 0.f;
  float2 acc[D / 64];
#pragma unroll
  for (int i = 0; i < D / 64; ++i) acc[i] = make_float2(0.f, 0.f);
  for (int sp = 0; sp < a.nsplit; ++sp) {
    const float* pr = base + sp * step;
    const float ms = pr[0];
    if (ms == -INFINITY) continue;
    const float w = exp2f(ms - m);
    l += pr[1] * w;
#pragma unroll
    for (int i = 0; i < D / 64; ++i) {
      const float2 v = *reinterpret_cast<const float2*>(pr + 4 + 2 * lane + 64 * i);
      acc[i].x += v.x * w;
      acc[i].y += v.y * w;
    }
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
  if (a.lse && lane == 0)
    a.lse[(size_t)h * a.total + tok] = l > 0.f ? m + log2f(l) : -INFINITY;
  uint32_t* orow = reinterpret_cast<uint32_t*>(a.o + ((size_t)tok * a.hq + h) * D);
#pragma unroll
  for (int i = 0; i < D / 64; ++i)
    orow[lane + 32 * i] = flash::pack_bf16x2(acc[i].x * inv, acc[i].y * inv);
}

// ------------------------------------------------------------------------ pair kernel
//
// Compute-bound calls: a persistent CTA per SM runs items of two row tiles (x = 0, 1) of the
// same sequence and KV head over one key list, each with a softmax warpgroup of its own, so
// that the tensor pipe works for one tile while the other's softmax runs, and each K and V
// tile is loaded once for both. Items come from a plan (packed_plan.cu), costliest first.
//   warp 0  loader: K_0, V_0, K_1, V_1, ... through one ring of kSlots tiles
//   warps 1 (TMEM owner), 3  load Q_x and issue S_x = Q_x K_j^T for x = 0, 1. One thread for
//           both was the bottleneck: a step's wait, eight MMAs, commit and loop took it about
//           800 cycles, four times per key tile
//   warp 2  issues O_x += P_x V_j for both
//   warps 4..7, 8..11  softmax and output of row tile 0, 1 (thread = row)
// They work in steps of 64 keys. One step's chain, S, its softmax, PV and the hand-offs
// between them, takes about 1,700 cycles, of which the tensor pipe works a third: four steps
// have to be in flight, two per row tile, and TMEM holds just that many (two S buffers of 64
// columns per row tile, P in bf16 over the upper half of each, and two O of 128). With 128-key
// steps, one in flight per row tile, a pair of tiles took 4,000 cycles instead of 2,048.
// A row tile's first P of an item also says that its warps have read the O of the item before.
constexpr int kSlots = 5;
constexpr int kStep = 64;                        // keys per step
constexpr int PAIR_THREADS = 384;
constexpr int PAIR_WG0_REGS = 80, PAIR_SOFTMAX_REGS = 208;
static_assert(128 * (PAIR_WG0_REGS + 2 * PAIR_SOFTMAX_REGS) <=
                  PAIR_THREADS * (65536 / PAIR_THREADS / 8 * 8),
              "the register split fits the launch's register pool");

template <int D>
struct PairSmem {
  static constexpr int TILE = BKV * D * 2;             // a Q, K or V tile
  static constexpr int OFF_Q = 0, OFF_RING = 2 * TILE;
  static constexpr int TOTAL = OFF_RING + kSlots * TILE + 1024;
  static constexpr int TM_S = 0, TM_O = 2 * BKV, P_OFF = kStep / 2;
};

struct PairBar {
  uint64_t full[kSlots], empty[kSlots];
  uint64_t q_full[2], q_empty[2];
  uint64_t s_full[2][2], p_full[2][2], pv_done[2][2];     // [row tile][buffer]
  uint64_t drain[3];
  uint32_t tmem_base;
  int abort;
};

// An item: row tiles at tokens tok0 and tok0 + tpt of a sequence, the steps that each takes (0:
// no rows; the last step is left out where a tile's own keys end in the first half of a key
// tile), and the key tiles that are loaded.
struct PairItem {
  int base, n, seq, tok0, h0, kvh, P, np, steps[2], tiles;
};

MARS_DEV PairItem pair_item(const AttnArgs& a, const packed::Plan& plan, int id) {
  PairItem it;
  const int heads = a.hkv * a.ngrp, g = id % heads;
  const packed::Tile t = plan.first[id / heads];
  it.base = t.base;
  it.n = t.n;
  it.seq = t.id;
  it.kvh = g / a.ngrp;
  it.h0 = g * a.gp;
  it.tok0 = t.tile * 2 * a.tpt;
  const long long cached = a.seq_lens ? a.seq_lens[t.id] : 0;
  it.P = (int)max(0LL, min(cached, (long long)a.max_pages * kPageSize));
  it.np = (it.P + BKV - 1) / BKV;
  for (int x = 0; x < 2; ++x) {
    const int first = it.tok0 + x * a.tpt;
    it.steps[x] = first < it.n ? 2 * it.np + (min(first + a.tpt, it.n) - 1) / kStep + 1 : 0;
  }
  it.tiles = (max(it.steps[0], it.steps[1]) + 1) / 2;
  return it;
}

template <int D>
__global__ void __launch_bounds__(PAIR_THREADS, 1)
pair_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
            const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_kp,
            const __grid_constant__ CUtensorMap tm_vp, AttnArgs a, packed::Plan plan) {
  using namespace sm100;
  using S = PairSmem<D>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ PairBar bar;
  const packed::Turns turns(*plan.count * a.hkv * a.ngrp);
  if (turns.at(0) < 0) return;                         // more CTAs than items
  const uint32_t raw = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + (((raw + 1023u) & ~1023u) - raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int* ab = &bar.abort;
  if (threadIdx.x == 0) {
    bar.abort = 0;
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(&bar.full[i], 1);
      mbar_init(&bar.empty[i], 2);
    }
    mbar_init(&bar.drain[2], 1);
    for (int x = 0; x < 2; ++x) {
      mbar_init(&bar.q_full[x], 1);
      mbar_init(&bar.q_empty[x], 1);
      for (int i = 0; i < 2; ++i) {
        mbar_init(&bar.s_full[x][i], 1);
        mbar_init(&bar.p_full[x][i], 128);
        mbar_init(&bar.pv_done[x][i], 1);
      }
      mbar_init(&bar.drain[x], 1);
    }
    fence_barrier_init();
  }
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
      int g = 0, flags = 0;                            // tiles loaded (K and V counted apart)
      bool ok = true;
      for (int r = 0; r < turns.rounds && ok; ++r) {
        const int id = turns.at(r);
        if (id < 0) continue;
        const PairItem it = pair_item(a, plan, id);
        if (a.seq_lens && a.seq_lens[it.seq] != it.P) flags |= MARS_ST_OVERFLOW;
        const int32_t* bt = a.block_table ? a.block_table + (size_t)it.seq * a.max_pages : nullptr;
        // this lane's page of prefix tile j, read one tile ahead
        auto entry = [&](int j) -> int {
          const int lp = j * kPagesPerTile + lane;
          return j < it.np && lane < kPagesPerTile && lp < a.max_pages ? bt[lp] : -1;
        };
        int next = entry(0);
        for (int j = 0; j < it.tiles && ok; ++j) {
          const int e = next;
          next = entry(j + 1);
          for (int v = 0; v < 2; ++v, ++g) {
            const int st = g % kSlots;
            int good = 1;
            if (lane == 0) {
              good = mbar_wait(&bar.empty[st], ((g / kSlots) & 1) ^ 1, ab, a.status);
              if (good) mbar_arrive_expect_tx(&bar.full[st], S::TILE);
            }
            ok = __shfl_sync(0xffffffffu, good, 0) != 0;
            if (!ok) break;
            uint8_t* dst = smem + S::OFF_RING + st * S::TILE;
            if (j < it.np) {
              if (lane < kPagesPerTile) {
                // as in packed_rows_kernel: a page that may not be read loads page 0
                int page = 0;
                if (e >= 0 && e < a.num_pages)
                  page = e;
                else if (j * BKV + lane * kPageSize < it.P)
                  flags |= MARS_ST_NOPAGE;
                const int row = a.num_pages > 0 ? (page * a.hkv + it.kvh) * kPageSize : kPageSize;
                for (int x = 0; x < D / 64; ++x)
                  tma_load_2d(dst + x * (BKV * 128) + lane * (kPageSize * 128), v ? &tm_vp : &tm_kp,
                              &bar.full[st], x * 64, row);
              }
            } else if (lane == 0) {
              for (int x = 0; x < D / 64; ++x)
                tma_load_3d(dst + x * (BKV * 128), v ? &tm_v : &tm_k, &bar.full[st], x * 64, it.kvh,
                            it.base + (j - it.np) * BKV);
            }
          }
        }
      }
      if (flags && a.status) atomicOr(a.status, flags);
      // wait (bounded) for the copies still in flight
      if (lane == 0)
        for (int k = 1; k <= kSlots && g - k >= 0; ++k)
          mbar_wait(&bar.full[(g - k) % kSlots], ((g - k) / kSlots) & 1, nullptr, a.status);
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
        for (int r = 0; r < turns.rounds && ok; ++r) {
          const int id = turns.at(r);
          if (id < 0) continue;
          const PairItem it = pair_item(a, plan, id);
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
          for (int j = 0; j < it.tiles && ok; ++j, ++g) {
            const int st = (2 * g) % kSlots;
            if (!(ok = mbar_wait(&bar.full[st], (2 * g / kSlots) & 1, ab, a.status))) break;
            const uint64_t kd = sdesc_sw128(smem_u32(smem + S::OFF_RING + st * S::TILE), 16, 1024);
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
            mma_commit(&bar.empty[st]);                // one of the two arrivals for a K slot
          }
        }
        mma_commit(&bar.drain[x]);
        mbar_wait(&bar.drain[x], 0, nullptr, a.status);
        if (items) mbar_wait(&bar.q_full[x], (items - 1) & 1, nullptr, a.status);
      }
    } else {
      // ------------------------------------------------------------------ O += P V
      if (elect_one()) {
        const uint32_t idesc = idesc_bf16_f32(BQ, D, true);
        int g = 0, done[2] = {0, 0};
        bool ok = true;
        for (int r = 0; r < turns.rounds && ok; ++r) {
          const int id = turns.at(r);
          if (id < 0) continue;
          const PairItem it = pair_item(a, plan, id);
          for (int j = 0; j < it.tiles && ok; ++j, ++g) {
            const int st = (2 * g + 1) % kSlots;
            if (!(ok = mbar_wait(&bar.full[st], ((2 * g + 1) / kSlots) & 1, ab, a.status))) break;
            const uint64_t vd = sdesc_sw128(smem_u32(smem + S::OFF_RING + st * S::TILE), BKV * 128, 1024);
            for (int hx = 0; hx < 4; ++hx) {
              const int h = hx >> 1, x = hx & 1, u = 2 * j + h;
              if (u >= it.steps[x]) continue;
              const int c = done[x], b = c & 1;
              if (!(ok = mbar_wait(&bar.p_full[x][b], (c >> 1) & 1, ab, a.status))) break;
              tc_fence_after();
#pragma unroll
              for (int k = 0; k < kStep / 16; ++k)
                mma_bf16_ts(tmem + S::TM_O + x * BKV, tmem + S::TM_S + x * BKV + b * kStep + S::P_OFF + k * 8,
                            sdesc_advance(vd, h * (kStep * 128) + k * 2048), idesc, (u | k) != 0);
              mma_commit(&bar.pv_done[x][b]);
              ++done[x];
            }
            if (!ok) break;
            mma_commit(&bar.empty[st]);                // both arrivals for a V slot
            mma_commit(&bar.empty[st]);
          }
        }
        mma_commit(&bar.drain[2]);
        mbar_wait(&bar.drain[2], 0, nullptr, a.status);
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
    int g = 0, done = 0;
    bool ok = true;
    for (int r = 0; r < turns.rounds && ok; ++r) {
      const int id = turns.at(r);
      if (id < 0) continue;
      const PairItem it = pair_item(a, plan, id);
      const int steps = it.steps[x];
      if (steps == 0) {
        g += it.tiles;
        continue;
      }
      RowsPolicy<D> pol;
      pol.a = &a;
      pol.bt_row = a.block_table ? a.block_table + (size_t)it.seq * a.max_pages : nullptr;
      pol.base = it.base;
      pol.n = it.n;
      pol.tok0 = it.tok0 + x * a.tpt;
      pol.P = it.P;
      pol.np = it.np;
      pol.h0 = it.h0;
      pol.j0 = 0;
      pol.split = 0;
      pol.last_tok = min(it.tok0 + 2 * a.tpt, it.n) - 1;   // of the item: V rows that neither tile reads
      const flash::RowVis vis = pol.row_vis(row);
      float m = -INFINITY, l = 0.f;
      typename RowsPolicy<D>::Tile tile, next = pol.tile(0);
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
        // that one is larger by more than 2^8 (the lazy rescale of flash_tc.cuh, always on an
        // item's first step) is it formed again
        float2 acc[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
        uint32_t packed[32];
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
          // of the tile; both row tiles' threads write the same zeros
          const int gv = 2 * (g + u / 2) + 1, st = gv % kSlots;
          if (!(ok = warp_wait(&bar.full[st], (gv / kSlots) & 1))) break;
          if (row / kStep == h && !pol.key_read(tile, row)) {
            uint8_t* vr = smem + S::OFF_RING + st * S::TILE + row * 128;
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
      g += it.tiles;
      const float inv = l > 0.f ? 1.f / l : 0.f;
      if (!(ok = warp_wait(&bar.pv_done[x][(done - 1) & 1], ((done - 1) >> 1) & 1))) break;
      tc_fence_after();
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {
        uint32_t o[32];
        tmem_ld32(o_addr + c * 32, o);
        tmem_ld_wait();
        pol.store_chunk(row, c * 32, o, inv, m, l);
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
    static_assert(SP::TOTAL + sizeof(PairBar) <= 227 * 1024, "pair layout fits shared memory");
    static std::atomic<int> attr_pair[64];
    cudaError_t e = set_smem_limit_once(pair_kernel<D>, SP::TOTAL, attr_pair);
    if (e != cudaSuccess) return e;
    size_t off = 0;
    const packed::Plan list =
        packed::carve_plan(workspace, off, p.batch, p.total, 2 * plan.tpt, false);
    e = packed::launch_plan(list, p.cu, p.seq_lens, a.max_pages, p.batch, p.total, 2 * plan.tpt,
                            p.status, stream);
    if (e != cudaSuccess) return e;
    pair_kernel<D><<<(unsigned)plan.ctas, PAIR_THREADS, SP::TOTAL, stream>>>(tq, tk, tv, tkp, tvp,
                                                                             a, list);
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
  const int tiles = (max_len + BKV - 1) / BKV + 1;
  // Two row tiles per item where sequences have more rows than one on average and the items
  // fill the GPU.
  const long long pairs = packed::max_tiles(batch, total, 2 * p.tpt) * hkv * (G / p.gp);
  if (total > (long long)batch * p.tpt && pairs >= num_sms()) {
    p.pair = true;
    p.nsplit = 1;
    p.split_tiles = tiles;
    p.items = pairs;
    p.ctas = num_sms();
    packed::carve_plan(nullptr, p.ws_bytes, batch, total, 2 * p.tpt, false);
    return p;
  }
  long long nsplit = 1;
  if (items < num_sms()) {
    nsplit = num_sms() / items;
    nsplit = nsplit < tiles / kMinSplitTiles ? nsplit : tiles / kMinSplitTiles;
    if (nsplit < 1) nsplit = 1;
  }
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
  a.part = static_cast<float*>(workspace);
  a.status = p.status;
  return p.d == 64 ? launch_rows<64>(p, plan, a, workspace, stream)
                   : launch_rows<128>(p, plan, a, workspace, stream);
}

}  // namespace mars
