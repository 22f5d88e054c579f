// Gradient of the causal attention of packed sequences (packed_attn.cu).
//
// With S = Q K^T, P = exp2(scale log2(e) S - lse) on the visible pairs (u <= t, same
// sequence), dP = dO V^T and D_t = sum_c dO_tc O_tc:
//   dV = P^T dO,   dS = P (dP - D),   dQ = scale dS K,   dK = scale dS^T Q.
// Row 0 of a sequence sees one key, whose weight is 1 whatever the score: its dS is 0, and is
// set so instead of being left to the cancellation of dP and D, unless it is infinite or NaN.
//
// Two tcgen05 pipelines over 128-row tiles, neither storing a score block, each a persistent CTA
// per SM, in one launch:
//   - dkdv: an item is a key tile and a KV head. Per pair of it with a query head of the group
//     and a query tile at or after it: S^T = K Q^T and dP^T = V dO^T (keys on TMEM lanes), then
//     dV += P^T dO and dK += dS^T Q with P^T and dS^T as bf16 operands in TMEM, all in two
//     halves of 64 queries with their own barriers. dV and dK stay in TMEM over the item.
//     The pairs of all items are divided evenly among the CTAs, whatever the lengths (KWalk):
//     an item that is cut leaves partials, and the last of its CTAs to finish adds them up in
//     the order of the pairs, so that the result is the same from run to run. With whole items
//     in turn, 4096 rows (28 heads over 4) kept the SMs busy for 44 % of the time, with an
//     item's heads divided in three for 76 %.
//   - dq: an item is a query tile and a query head, taken in turn by falling cost; S, dP and
//     dQ += dS K per key tile.
// P and dS are rounded to bf16 as MMA operands; dS is formed from the unrounded P, and D from O as
// the forward rounded it (sum P dP in 32 bits would take a further pass over all pairs). The error
// of dQ and dK against 64 bits is 0.0024 to 0.0028 of their norm, where rounding the exact result
// gives 0.0017; in sequences of a handful of rows, whose weights are large, D's share makes it up to
// 0.0044. prep_kernel computes D, lays lse and D out in 128-row blocks per (head, tile), for bulk
// copies, and lists the tiles.
//
// What bounds both is shared memory at 128 bytes per cycle (d = 128): a pair of dkdv reads 96 KB
// each for S^T and dP^T (with halves of 64 queries an MMA reads its 4 KB of K or V again), 32 KB
// each for dV and dK, and 64 KB are copied in: 2,500 cycles of the 2,900 measured; a tile of dq
// 64 + 64 + 32 KB and 64 KB in: 1,750 of 1,850. Whole S^T and dP^T would save 64 KB a pair, but
// then S^T of the next pair waits for all of dV: 5 % slower. 4096 rows (28 heads over 4) take 275
// us: 1.1 PFLOP/s counting each product once, 1.5 (0.78 of the GEMM rate) as computed.
//
// A pair's tile can reach past its sequence: scores there are masked, and the rows of dO, Q
// (dkdv) or K (dq) that the masked weights of 0 would multiply are cleared in shared memory, so
// that other sequences' rows have no effect whatever they hold.
#include <cuda_bf16.h>

#include <algorithm>
#include <atomic>

#include "common.cuh"
#include "flash_tc.cuh"
#include "internal.h"
#include "packed.cuh"
#include "packed_plan.cuh"

namespace mars {

namespace {

using namespace sm100;
using packed::Tile;
using packed::Walk;

constexpr int GT = 128;                 // rows per key tile and per query tile
constexpr int MATH_WARPS = 8;           // two per TMEM lane quadrant, 64 columns each
constexpr int MATH_THREADS = 32 * MATH_WARPS;
constexpr int NSTAGE = 2;               // Q / dO ring depth of dkdv

struct GradArgs {
  packed::Plan plan;
  int total, hq, hkv, G;
  int k_ctas, q_ctas;                   // CTAs for dK / dV and for dQ
  long long pad;                        // padded rows per head: 128 * the bound of the tiles
  float scale, scale_log2;
  const uint16_t *o, *d_o;              // [total][hq][D]
  const float* lse;                     // [hq][total]
  float *lse_p, *d_p;                   // [hq][pad]
  uint16_t *dq, *dk, *dv;
  long long dq_stride, dk_stride, dv_stride;
  float* part;                          // partial()
  int32_t* status;
};

// ------------------------------------------------------------------------------ prep

// Block 0 lists the tiles. Each of the others computes D and lse of PREP_ROWS rows of a tile and
// up to PREP_HEADS heads, in 128-row blocks per head; rows past the sequence get zeros. D / 8
// lanes per (row, head), heads fastest, as O and dO lie in memory; the results go out over shared
// memory with the rows fastest, as lse lies. It reads O and dO once, which bounds it.
constexpr int PREP_ROWS = 8, PREP_HEADS = 64;

template <int D>
__global__ void __launch_bounds__(packed::kPlanThreads, 5)
prep_kernel(GradArgs a, packed::PlanArgs plan) {
  if (blockIdx.x == 0) {
    packed::make_plan(plan);
    return;
  }
  __shared__ float s_d[PREP_HEADS][PREP_ROWS + 1];
  constexpr int LANES = D / 8, PER = packed::kPlanThreads / LANES;
  constexpr int CHUNKS = GT / PREP_ROWS;
  const int hchunks = (a.hq + PREP_HEADS - 1) / PREP_HEADS;
  int id = blockIdx.x - 1;
  const int h0 = id % hchunks * PREP_HEADS;
  id /= hchunks;
  const int chunk = id % CHUNKS;
  id /= CHUNKS;
  bool bad;                                            // reported with the plan
  const packed::Seq t = packed::find_tile(plan.cu, plan.batch, a.total, GT, 0, id, bad);
  if (t.s < 0) return;
  const int sub = threadIdx.x / LANES, lane = threadIdx.x % LANES;
  const int nh = min(PREP_HEADS, a.hq - h0), row0 = t.tile * GT + chunk * PREP_ROWS;
  const int n = PREP_ROWS * nh;
  constexpr int AHEAD = 4;                             // loads in flight per thread: 2 * AHEAD
  for (int i0 = sub; i0 - sub < n; i0 += AHEAD * PER) {
    uint4 x[AHEAD], y[AHEAD];
#pragma unroll
    for (int u = 0; u < AHEAD; ++u) {
      // past the end or the sequence: some row, whose result is not used
      const int i = min(i0 + u * PER, n - 1), r = i / nh, h = i - r * nh;
      const int row = min(row0 + r, t.n - 1);
      const size_t at = ((size_t)(t.base + row) * a.hq + h0 + h) * D + lane * 8;
      x[u] = *reinterpret_cast<const uint4*>(a.o + at);
      y[u] = *reinterpret_cast<const uint4*>(a.d_o + at);
    }
#pragma unroll
    for (int u = 0; u < AHEAD; ++u) {
      float xf[8], yf[8], acc = 0.f;
      unpack8(x[u], xf);
      unpack8(y[u], yf);
#pragma unroll
      for (int e = 0; e < 8; ++e) acc += xf[e] * yf[e];
#pragma unroll
      for (int o = LANES / 2; o > 0; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
      const int i = i0 + u * PER;
      if (lane == 0 && i < n) s_d[i % nh][i / nh] = acc;
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < PREP_ROWS * nh; i += packed::kPlanThreads) {
    const int r = i % PREP_ROWS, h = i / PREP_ROWS;
    const size_t p = (size_t)(h0 + h) * a.pad + (size_t)id * GT + chunk * PREP_ROWS + r;
    a.d_p[p] = row0 + r < t.n ? s_d[h][r] : 0.f;
    a.lse_p[p] = row0 + r < t.n ? a.lse[(size_t)(h0 + h) * a.total + t.base + row0 + r] : 0.f;
  }
}

// ---------------------------------------------------------------------------- shared

MARS_DEV uint32_t bits(int lo, int hi) { return flash::bit_range(lo, hi); }

// Two bf16, the low one set to 0 if it is finite.
MARS_DEV uint32_t clear_low(uint32_t w) { return (~w & 0x7f80u) ? w & 0xffff0000u : w; }

// Rows [first, 128) of a [128][D] operand tile (D / 64 swizzled regions) set to zero, by
// `threads` threads of which this is number `id`; rows [lo, hi) of the tile are theirs.
template <int D>
MARS_DEV void clear_rows(uint8_t* tile, int first, int lo, int hi, int id, int threads) {
  constexpr int VECS = D / 8;                       // 16-byte vectors per row
  for (int i = max(first, lo) * VECS + id; i < hi * VECS; i += threads) {
    const int r = i / VECS, c = i % VECS;
    *reinterpret_cast<uint4*>(tile + (c >> 3) * (GT * 128) + r * 128 + (c & 7) * 16) =
        make_uint4(0, 0, 0, 0);
  }
}

// ---------------------------------------------------------------------- dK and dV

template <int D>
struct KSmem {
  static constexpr int T_BYTES = GT * D * 2;
  static constexpr int OFF_K = 0, OFF_V = T_BYTES, OFF_RING = 2 * T_BYTES;
  // a stage: Q and dO [128][D], lse and D of its 128 rows
  static constexpr int ST_Q = 0, ST_DO = T_BYTES, ST_LSE = 2 * T_BYTES, ST_D = ST_LSE + GT * 4;
  static constexpr int STAGE = (ST_D + GT * 4 + 1023) / 1024 * 1024;
  static constexpr int TOTAL = OFF_RING + NSTAGE * STAGE + 1024;
  static constexpr int TM_S = 0, TM_DP = 128, TM_DV = 256, TM_DK = 256 + D, TM_COLS = 512;
};

// Part [pa, pb) of the `all` pairs of key tile t and a KV head: pair p is query head
// kvh * G + p / nq and query tile t.tile + p % nq of its sequence.
struct KItem {
  Tile t;
  int kvh, nq, all, pa, pb;
  int first, cuts;                      // a divided item: CTAs first .. first + cuts share it
};

constexpr int K_ITEMS = 3;              // items handed over by the loader and not yet finished

struct KBar {
  uint64_t kv_full, kv_empty;
  uint64_t full[NSTAGE], empty[NSTAGE];
  uint64_t s_full[2], dp_full[2], p_full[2], ds_full[2], dv_done[2], dk_done[2];
  uint64_t acc_full, acc_free, drain, drain_ts;
  uint64_t stored, told;                // partials written; `last` set
  uint64_t item_full[K_ITEMS], item_empty[K_ITEMS];
  KItem items[K_ITEMS];
  uint32_t tmem_base;
  int abort;
  int last;                             // whether this CTA adds up an item's partials
};

constexpr int kMinPart = 2;             // pairs of a part of a divided item, at least
// Work of a part of the line, at least. An item's pairs take more than half of its work (with
// kMinPart pairs or more), so that two cuts of an item are at least a pair apart.
constexpr int kMinWork = kMinPart * packed::kPairWork + packed::kTileWork;

// The line of all items, KV head by KV head, tile by tile, each as long as its work; CTA c of
// `parts` takes the part of it from cut(c) to cut(c + 1). (Cutting it so that the CTAs stay
// near one another, for Q and dO in L2, saved as much as the further cuts cost.)
struct KLine {
  long long head, total;                // work of one KV head and of all
  int parts;
  MARS_DEV explicit KLine(const GradArgs& a)
      : head(a.plan.before[*a.plan.count]), total(head * a.hkv) {
    parts = (int)max(1LL, min((long long)a.k_ctas, total / kMinWork));
  }
  MARS_DEV long long cut(int i) const { return i * total / parts; }
  // The pair before which position pos cuts an item of `pairs` pairs and `work` at s0: 0 before
  // the item, `pairs` after it.
  MARS_DEV int inside(long long pos, long long s0, int work, int pairs) const {
    const int j = (int)((pos - s0) * pairs / work);
    return j < kMinPart ? 0 : pairs - j < kMinPart ? pairs : j;
  }
};

// Where a part begins: pair pa of tile i of a KV head.
struct KStart {
  int kvh, i, pa;
};

// Query tiles at or after a key tile.
MARS_DEV int after(const Tile& t) { return (t.n + GT - 1) / GT - t.tile; }

// Every thread of the CTA; the caller synchronises.
MARS_DEV void find_start(const GradArgs& a, const KLine& line, KStart& st) {
  const long long p0 = line.cut(blockIdx.x);
  const int kvh = (int)(p0 / line.head), n = *a.plan.count;
  const long long x = p0 - kvh * line.head;
  for (int i = threadIdx.x; i < n; i += blockDim.x)
    if (a.plan.before[i] <= x && x < a.plan.before[i + 1]) {
      const int nq = after(a.plan.in_order[i]);
      st = KStart{kvh, i, line.inside(p0, kvh * line.head + a.plan.before[i],
                                      packed::tile_work(a.G, nq), a.G * nq)};
    }
}

// The items of a CTA's part. A tile is read while the item before it is worked on.
struct KWalk {
  const GradArgs& a;
  long long s0, end;
  int kvh, i, n, pa;
  Tile tile;
  MARS_DEV KWalk(const GradArgs& a_, const KLine& line, const KStart& st)
      : a(a_), s0(st.kvh * line.head + a_.plan.before[st.i]), end(line.cut(blockIdx.x + 1)),
        kvh(st.kvh), i(st.i), n(*a_.plan.count), pa(st.pa), tile(a_.plan.in_order[st.i]) {}
  MARS_DEV void next(int work) {
    s0 += work;
    pa = 0;
    if (++i == n) {
      i = 0;
      ++kvh;
    }
    if (s0 < end) tile = a.plan.in_order[i];
  }
  MARS_DEV bool take(const KLine& line, KItem& it) {
    if (s0 >= end) return false;
    int nq = after(tile);
    if (pa == a.G * nq) {                // the part begins behind this item
      next(packed::tile_work(a.G, nq));
      if (s0 >= end) return false;
      nq = after(tile);
    }
    const int all = a.G * nq, work = packed::tile_work(a.G, nq);
    const int pb = end >= s0 + work ? all : line.inside(end, s0, work, all);
    it = KItem{tile, kvh, nq, all, pa, pb, 0, 0};
    if (pb - pa < all) {
      int c = (int)(s0 * line.parts / line.total);
      while (line.cut(c) <= s0 || line.inside(line.cut(c), s0, work, all) == 0) ++c;
      it.first = c - 1;
      while (c < line.parts && line.cut(c) < s0 + work &&
             line.inside(line.cut(c), s0, work, all) < all)
        ++c;
      it.cuts = c - 1 - it.first;
    }
    next(work);
    return pb > pa;
  }
};

// dkdv: warps 0 loader, 1 S / dP issuer and TMEM owner, 2 dV / dK issuer, 4 .. 11 math.
// The first four give registers to the math warps, which hold 200 values in the sums.
constexpr int K_THREADS = 128 + MATH_THREADS;
constexpr int K_WG0_REGS = 88, K_MATH_REGS = 208;
static_assert(128 * (K_WG0_REGS + 2 * K_MATH_REGS) <= K_THREADS * (65536 / K_THREADS / 8 * 8),
              "the register split fits the launch's register pool");

// Partial dV (and D / 4 x 128 float4 further on dK) of the item that a CTA's part starts inside
// of, or of the one that it ends inside of and has the start of: [column / 4][row], so that the
// lanes of a warp, a row each, access consecutive places.
template <int D>
MARS_DEV float4* partial(const GradArgs& a, int cta, bool inside) {
  return reinterpret_cast<float4*>(a.part) +
         ((size_t)cta * 2 + (inside ? 0 : 1)) * (2 * GT * D / 4);
}

// TMEM column of K-step k (16 queries) of P^T or dS^T: queries [0, 64) over columns [0, 32),
// [64, 128) over [64, 96), the first half of each half's own fp32 columns.
MARS_DEV uint32_t p_col(int k) { return (uint32_t)(8 * k + (k >= 4 ? 32 : 0)); }

template <int D>
MARS_DEV void dkdv(const CUtensorMap& tm_q, const CUtensorMap& tm_do, const CUtensorMap& tm_k,
                   const CUtensorMap& tm_v, const GradArgs& a, uint8_t* smem_raw) {
  using S = KSmem<D>;
  __shared__ KBar bar;
  const uint32_t raw = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + (((raw + 1023u) & ~1023u) - raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int* ab = &bar.abort;
  if (*a.plan.count == 0) return;
  const KLine line(a);
  if ((int)blockIdx.x >= line.parts) return;
  __shared__ KStart start;
  find_start(a, line, start);

  if (threadIdx.x == 0) {
    bar.abort = 0;
    mbar_init(&bar.kv_full, 1);
    mbar_init(&bar.kv_empty, 1);
    for (int i = 0; i < NSTAGE; ++i) {
      mbar_init(&bar.full[i], 1);
      mbar_init(&bar.empty[i], 1);
    }
    for (int h = 0; h < 2; ++h) {
      mbar_init(&bar.s_full[h], 1);
      mbar_init(&bar.dp_full[h], 1);
      mbar_init(&bar.p_full[h], MATH_THREADS / 2);
      mbar_init(&bar.ds_full[h], MATH_THREADS / 2);
      mbar_init(&bar.dv_done[h], 1);
      mbar_init(&bar.dk_done[h], 1);
    }
    mbar_init(&bar.acc_full, 1);
    mbar_init(&bar.acc_free, MATH_THREADS);
    mbar_init(&bar.drain, 1);
    mbar_init(&bar.drain_ts, 1);
    mbar_init(&bar.stored, MATH_THREADS);
    for (int i = 0; i < K_ITEMS; ++i) {
      mbar_init(&bar.item_full[i], 1);
      mbar_init(&bar.item_empty[i], 2 + MATH_WARPS);   // both issuers, the math warps
    }
    mbar_init(&bar.told, 1);
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(&bar.tmem_base, S::TM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, bar.tmem_base, 0);

  if (warp < 4) {
    regs_lower<K_WG0_REGS>();
    if (warp == 0) {
      // ---------------------------------------------------------------- loads
      if (lane == 0) {
        int gp = 0, ii = 0, nkv = 0;
        bool ok = true;
        KItem it;
        int ni = 0;                                    // items handed over
        auto publish = [&](const KItem& d) {
          if (!mbar_wait(&bar.item_empty[ni % K_ITEMS], ((ni / K_ITEMS) & 1) ^ 1, ab, a.status))
            return false;
          bar.items[ni % K_ITEMS] = d;
          mbar_arrive(&bar.item_full[ni % K_ITEMS]);
          ++ni;
          return true;
        };
        for (KWalk walk(a, line, start); ok && walk.take(line, it);) {
          if (!(ok = publish(it))) break;
          if (ii > 0 && !(ok = mbar_wait(&bar.kv_empty, (ii - 1) & 1, ab, a.status))) break;
          mbar_arrive_expect_tx(&bar.kv_full, 2 * S::T_BYTES);
          const int z = it.t.base + GT * it.t.tile;
          for (int x = 0; x < D / 64; ++x) {
            tma_load_3d(smem + S::OFF_K + x * (GT * 128), &tm_k, &bar.kv_full, x * 64, it.kvh, z);
            tma_load_3d(smem + S::OFF_V + x * (GT * 128), &tm_v, &bar.kv_full, x * 64, it.kvh, z);
          }
          ++nkv;
          for (int p = it.pa; p < it.pb; ++p, ++gp) {
            const int st = gp % NSTAGE;
            uint8_t* stage = smem + S::OFF_RING + st * S::STAGE;
            if (!(ok = mbar_wait(&bar.empty[st], ((gp / NSTAGE) & 1) ^ 1, ab, a.status))) break;
            const int h = it.kvh * a.G + p / it.nq, qi = p % it.nq;
            const size_t rb = (size_t)h * a.pad + (size_t)(it.t.id + qi) * GT;
            mbar_arrive_expect_tx(&bar.full[st], 2 * S::T_BYTES + 2 * GT * 4);
            bulk_load(stage + S::ST_LSE, a.lse_p + rb, GT * 4, &bar.full[st]);
            bulk_load(stage + S::ST_D, a.d_p + rb, GT * 4, &bar.full[st]);
            const int zq = z + GT * qi;
            for (int x = 0; x < D / 64; ++x) {
              uint8_t* to = stage + x * (GT * 128);
              tma_load_3d(to + S::ST_Q, &tm_q, &bar.full[st], x * 64, h, zq);
              tma_load_3d(to + S::ST_DO, &tm_do, &bar.full[st], x * 64, h, zq);
            }
          }
          ++ii;
        }
        if (ok) publish(KItem{});                      // no more items
        // wait (bounded) for the copies still in flight
        if (nkv > 0) mbar_wait(&bar.kv_full, (nkv - 1) & 1, nullptr, a.status);
        for (int k = 1; k <= NSTAGE && gp - k >= 0; ++k)
          mbar_wait(&bar.full[(gp - k) % NSTAGE], ((gp - k) / NSTAGE) & 1, nullptr, a.status);
      }
      __syncwarp();
    } else if (warp == 1) {
      // ------------------------------------------------------- S^T and dP^T MMAs
      if (elect_one()) {
        const uint32_t id_qk = idesc_bf16_f32(GT, GT / 2, false);
        const uint64_t kd = sdesc_sw128(smem_u32(smem + S::OFF_K), 16, 1024);
        const uint64_t vd = sdesc_sw128(smem_u32(smem + S::OFF_V), 16, 1024);
        // half h of S^T = K Q^T (or dP^T = V dO^T) of pair gp, once `done` says that the MMAs
        // that read the buffer's previous P^T (dS^T) have completed
        auto issue = [&](int gp, uint64_t ad, int st_off, int col, uint64_t* done, uint64_t* full) {
          const uint32_t sb = smem_u32(smem + S::OFF_RING + (gp % NSTAGE) * S::STAGE);
          const uint64_t bd = sdesc_sw128(sb + st_off, 16, 1024);
          for (int h = 0; h < 2; ++h) {
            if (gp > 0 && !mbar_wait(&done[h], (gp - 1) & 1, ab, a.status)) return false;
            tc_fence_after();
  #pragma unroll
            for (int k = 0; k < D / 16; ++k) {
              const uint32_t off = (k >> 2) * (GT * 128) + (k & 3) * 32;
              mma_bf16_ss(tmem + col + (GT / 2) * h, sdesc_advance(ad, off),
                          sdesc_advance(bd, off + h * (GT / 2) * 128), id_qk, k != 0);
            }
            mma_commit(&full[h]);
          }
          return true;
        };
        int gp = 0, ii = 0, items = 0;
        bool ok = true;
        // pairs of the next item, 0 at the end
        auto next_pairs = [&](int& np) {
          const int q = items % K_ITEMS;
          if (!mbar_wait(&bar.item_full[q], (items / K_ITEMS) & 1, ab, a.status)) return false;
          np = bar.items[q].pb - bar.items[q].pa;
          mbar_arrive(&bar.item_empty[q]);
          ++items;
          return true;
        };
        int np;
        while (ok && (ok = next_pairs(np)) && np) {
          if (!(ok = mbar_wait(&bar.kv_full, ii & 1, ab, a.status))) break;
          for (int p = 0; p < np && ok; ++p, ++gp)
            ok = mbar_wait(&bar.full[gp % NSTAGE], (gp / NSTAGE) & 1, ab, a.status) &&
                 issue(gp, kd, S::ST_Q, S::TM_S, bar.dv_done, bar.s_full) &&
                 issue(gp, vd, S::ST_DO, S::TM_DP, bar.dk_done, bar.dp_full);
          if (!ok) break;
          mma_commit(&bar.kv_empty);                     // only these MMAs read K and V
          ++ii;
        }
        mma_commit(&bar.drain);
        mbar_wait(&bar.drain, 0, nullptr, a.status);
      }
    } else if (warp == 2) {
      // -------------------------------------------------------- dV and dK MMAs
      if (elect_one()) {
        const uint32_t id_acc = idesc_bf16_f32(GT, D, true);     // A from TMEM, B MN-major
        int gp = 0, ii = 0, items = 0;
        bool ok = true;
        // pairs of the next item, 0 at the end
        auto next_pairs = [&](int& np) {
          const int q = items % K_ITEMS;
          if (!mbar_wait(&bar.item_full[q], (items / K_ITEMS) & 1, ab, a.status)) return false;
          np = bar.items[q].pb - bar.items[q].pa;
          mbar_arrive(&bar.item_empty[q]);
          ++items;
          return true;
        };
        int np;
        while (ok && (ok = next_pairs(np)) && np) {
          for (int p = 0; p < np; ++p, ++gp) {
            const int st = gp % NSTAGE;
            const uint32_t sb = smem_u32(smem + S::OFF_RING + st * S::STAGE);
            if (!(ok = mbar_wait(&bar.full[st], (gp / NSTAGE) & 1, ab, a.status))) break;
            // the accumulators start from zero: the previous item's must have been read
            if (p == 0 && ii > 0 && !(ok = mbar_wait(&bar.acc_free, (ii - 1) & 1, ab, a.status)))
              break;
            auto accumulate = [&](uint64_t* ready, uint64_t* done, int st_off, int src, int dst) {
              const uint64_t bd = sdesc_sw128(sb + st_off, GT * 128, 1024);
              for (int h = 0; h < 2; ++h) {
                if (!mbar_wait(&ready[h], gp & 1, ab, a.status)) return false;
                tc_fence_after();
  #pragma unroll
                for (int kq = 0; kq < GT / 32; ++kq) {
                  const int k = (GT / 32) * h + kq;
                  mma_bf16_ts(tmem + dst, tmem + src + p_col(k), sdesc_advance(bd, k * 2048),
                              id_acc, (p | k) != 0);
                }
                mma_commit(&done[h]);
              }
              return true;
            };
            if (!(ok = accumulate(bar.p_full, bar.dv_done, S::ST_DO, S::TM_S, S::TM_DV) &&
                       accumulate(bar.ds_full, bar.dk_done, S::ST_Q, S::TM_DP, S::TM_DK)))
              break;
            // S^T and dP^T completed before the math warps formed dS^T, and those have read
            // the stage's lse and D: the stage is free after dK
            mma_commit(&bar.empty[st]);
          }
          if (!ok) break;
          mma_commit(&bar.acc_full);
          ++ii;
        }
        mma_commit(&bar.drain_ts);
        mbar_wait(&bar.drain_ts, 0, nullptr, a.status);
      }
    }
  } else {
    regs_raise<K_MATH_REGS>();
    // ------------------------------------------------------- math (two warps per quadrant)
    const int quad = warp & 3, half = (warp - 4) >> 2;
    const int row = quad * 32 + lane;                  // TMEM lane = key row of the tile
    const uint32_t lane_off = (uint32_t)(quad * 32) << 16;
    constexpr int HC = GT / 2, HD = D / 2;
    auto warp_wait = [&](uint64_t* b, uint32_t parity) -> bool {
      return __all_sync(0xffffffffu, mbar_wait(b, parity, ab, a.status));
    };
    int gp = 0, ii = 0, cut_items = 0;
    bool ok = true;
    for (;; ++ii) {
      // read where it is: a copy of the item would cost the key loop its registers
      const volatile KItem& it = bar.items[ii % K_ITEMS];
      if (!(ok = warp_wait(&bar.item_full[ii % K_ITEMS], (ii / K_ITEMS) & 1))) break;
      const int pb = it.pb, nq = it.nq, n = it.t.n, tile0 = it.t.tile;
      if (!pb) break;
      const int kk = GT * tile0 + row;                 // key position in its sequence
      for (int p = it.pa; p < pb; ++p, ++gp) {
        const int st = gp % NSTAGE;
        uint8_t* stage = smem + S::OFF_RING + st * S::STAGE;
        const float* ls = reinterpret_cast<const float*>(stage + S::ST_LSE) + HC * half;
        const float* dsv = reinterpret_cast<const float*>(stage + S::ST_D) + HC * half;
        const int q0 = GT * (tile0 + p % nq);   // first query position
        // query columns [lo, hi) of this half that see the key; none for a key past the end
        const int live = n - q0;                  // query rows of the tile
        const int lo = kk - q0 - HC * half;
        const int hi = kk < n ? live - HC * half : -1;
        const bool ragged = live < GT;                 // uniform over the CTA
        if (!(ok = warp_wait(&bar.s_full[half], gp & 1))) break;
        tc_fence_after();
        uint32_t v[HC];
#pragma unroll
        for (int q = 0; q < HC / 32; ++q)
          tmem_ld32(tmem + S::TM_S + HC * half + q * 32 + lane_off,
                    *reinterpret_cast<uint32_t(*)[32]>(v + q * 32));
        tmem_ld_wait();
        if (ragged) {
          // the half's rows of Q and dO past the sequence, once the MMAs that read them as S^T
          // and dP^T operands have completed
          if (!(ok = warp_wait(&bar.dp_full[half], gp & 1))) break;
          const int tid = quad * 32 + lane;
          clear_rows<D>(stage + S::ST_Q, live, HC * half, HC * half + HC, tid, 128);
          clear_rows<D>(stage + S::ST_DO, live, HC * half, HC * half + HC, tid, 128);
          fence_proxy_async_smem();
        }
        const bool whole = lo <= 0 && hi >= HC;
        uint32_t mk[2] = {0xffffffffu, 0xffffffffu};
        if (!whole) {
#pragma unroll
          for (int q = 0; q < HC / 32; ++q) {
            mk[q] = bits(lo - 32 * q, hi - 32 * q);
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (!((mk[q] >> e) & 1u)) v[32 * q + e] = 0xff800000u;
          }
        }
        float pf[HC];
        uint32_t pp[HC / 2];
        const float2 sc2 = make_float2(a.scale_log2, a.scale_log2);
#pragma unroll
        for (int e = 0; e < HC; e += 4) {
          const float4 l4 = *reinterpret_cast<const float4*>(ls + e);
          const float2 s01 = make_float2(__uint_as_float(v[e]), __uint_as_float(v[e + 1]));
          const float2 t01 = __ffma2_rn(s01, sc2, make_float2(-l4.x, -l4.y));
          const float2 s23 = make_float2(__uint_as_float(v[e + 2]), __uint_as_float(v[e + 3]));
          const float2 t23 = __ffma2_rn(s23, sc2, make_float2(-l4.z, -l4.w));
          pf[e] = flash::ex2_approx(t01.x);
          pf[e + 1] = flash::ex2_approx(t01.y);
          pf[e + 2] = flash::ex2_approx(t23.x);
          pf[e + 3] = flash::ex2_approx(t23.y);
          pp[e / 2] = flash::pack_bf16x2(pf[e], pf[e + 1]);
          pp[e / 2 + 1] = flash::pack_bf16x2(pf[e + 2], pf[e + 3]);
        }
        tmem_st32(tmem + S::TM_S + HC * half + lane_off, *reinterpret_cast<uint32_t(*)[32]>(pp));
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive_warp(&bar.p_full[half]);
        if (!(ok = warp_wait(&bar.dp_full[half], gp & 1))) break;
        tc_fence_after();
#pragma unroll
        for (int q = 0; q < HC / 32; ++q)
          tmem_ld32(tmem + S::TM_DP + HC * half + q * 32 + lane_off,
                    *reinterpret_cast<uint32_t(*)[32]>(v + q * 32));
        tmem_ld_wait();
        if (!whole) {                                  // masked dP may hold anything
#pragma unroll
          for (int q = 0; q < HC / 32; ++q)
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (!((mk[q] >> e) & 1u)) v[32 * q + e] = 0u;
        }
#pragma unroll
        for (int e = 0; e < HC; e += 4) {
          const float4 d4 = *reinterpret_cast<const float4*>(dsv + e);
          const float2 s01 = __fmul2_rn(make_float2(pf[e], pf[e + 1]),
                                        __fadd2_rn(make_float2(__uint_as_float(v[e]),
                                                               __uint_as_float(v[e + 1])),
                                                   make_float2(-d4.x, -d4.y)));
          const float2 s23 = __fmul2_rn(make_float2(pf[e + 2], pf[e + 3]),
                                        __fadd2_rn(make_float2(__uint_as_float(v[e + 2]),
                                                               __uint_as_float(v[e + 3])),
                                                   make_float2(-d4.z, -d4.w)));
          pp[e / 2] = flash::pack_bf16x2(s01.x, s01.y);
          pp[e / 2 + 1] = flash::pack_bf16x2(s23.x, s23.y);
        }
        if (q0 == 0 && half == 0) pp[0] = clear_low(pp[0]);   // dS of row 0 is 0
        tmem_st32(tmem + S::TM_DP + HC * half + lane_off, *reinterpret_cast<uint32_t(*)[32]>(pp));
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive_warp(&bar.ds_full[half]);
      }
      if (!ok) break;
      // the item's dV and dK rows, this thread's half of the columns
      if (!(ok = warp_wait(&bar.acc_full, ii & 1))) break;
      tc_fence_after();
      uint32_t dvr[HD], dkr[HD];
#pragma unroll
      for (int q = 0; q < HD / 32; ++q) {
        tmem_ld32(tmem + S::TM_DV + HD * half + q * 32 + lane_off,
                  *reinterpret_cast<uint32_t(*)[32]>(dvr + q * 32));
        tmem_ld32(tmem + S::TM_DK + HD * half + q * 32 + lane_off,
                  *reinterpret_cast<uint32_t(*)[32]>(dkr + q * 32));
      }
      tmem_ld_wait();
      tc_fence_before();
      mbar_arrive_warp(&bar.acc_free);
      bool write = it.pb - it.pa == it.all;
      if (!write) {
        // a part of the item: its partial, and the sum by the last part to arrive
        float4* pv = partial<D>(a, blockIdx.x, it.pa > 0) + (HD / 4) * half * GT + row;
#pragma unroll
        for (int e = 0; e < HD; e += 4) {
          pv[(e / 4) * GT] = make_float4(__uint_as_float(dvr[e]), __uint_as_float(dvr[e + 1]),
                                         __uint_as_float(dvr[e + 2]), __uint_as_float(dvr[e + 3]));
          pv[(D + e) / 4 * GT] =
              make_float4(__uint_as_float(dkr[e]), __uint_as_float(dkr[e + 1]),
                          __uint_as_float(dkr[e + 2]), __uint_as_float(dkr[e + 3]));
        }
        const int first = it.first, cuts = it.cuts;
        __threadfence();
        mbar_arrive_warp(&bar.stored);
        if (warp == 4) {
          if (!(ok = warp_wait(&bar.stored, cut_items & 1))) break;
          if (lane == 0) {
            bar.last = atomicAdd(a.plan.tickets + first, 1) == cuts;
            mbar_arrive(&bar.told);
          }
        }
        if (!(ok = warp_wait(&bar.told, cut_items & 1))) break;
        ++cut_items;
        write = *reinterpret_cast<volatile int*>(&bar.last) != 0;
        if (write) {
          __threadfence();
#pragma unroll
          for (int e = 0; e < HD; ++e) dvr[e] = dkr[e] = 0u;
#pragma unroll 1
          for (int k = 0; k <= cuts; ++k) {
            const float4* r = partial<D>(a, first + k, k > 0) + (HD / 4) * half * GT + row;
            auto add = [&](uint32_t* acc, const float4* from) {
#pragma unroll
              for (int e = 0; e < HD; e += 4) {
                const float4 u = __ldcg(from + (e / 4) * GT);
                acc[e] = __float_as_uint(__uint_as_float(acc[e]) + u.x);
                acc[e + 1] = __float_as_uint(__uint_as_float(acc[e + 1]) + u.y);
                acc[e + 2] = __float_as_uint(__uint_as_float(acc[e + 2]) + u.z);
                acc[e + 3] = __float_as_uint(__uint_as_float(acc[e + 3]) + u.w);
              }
            };
            add(dvr, r);
            add(dkr, r + D / 4 * GT);
          }
        }
      }
      if (write) {
        const long long tok = (long long)it.t.base + kk;
        const int col = it.kvh * D + HD * half;
        const bool rv = kk < n;
        packed::store_rows<HD>(a.dv, rv ? tok * a.dv_stride + col : -1, lane,
                               [&](int e) { return __uint_as_float(dvr[e]); });
        packed::store_rows<HD>(a.dk, rv ? tok * a.dk_stride + col : -1, lane,
                               [&](int e) { return __uint_as_float(dkr[e]) * a.scale; });
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar.item_empty[ii % K_ITEMS]);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, S::TM_COLS);
  }
}

// -------------------------------------------------------------------------------- dQ

// K ring and V ring of flash_tc.cuh, Q and dO tiles; TMEM: S at 0, dP at 128, dQ at 256, dS
// (bf16 pairs, 64 columns) at 384. Warps: 0 K loader, 1 TMEM owner and S/dP issuer (it also
// loads Q and dO), 2..9 math, 10 V loader, 11 dQ issuer.
constexpr int Q_THREADS = 32 * (4 + MATH_WARPS);
constexpr int Q_V_WARP = 2 + MATH_WARPS, Q_TS_WARP = 3 + MATH_WARPS;

struct QBar {
  uint64_t s_full, dp_full, s_free, dp_free, ds_full, dq_done, acc_free;
};

struct QItem {
  Tile t;
  int h, n;      // query head, key tiles
};

MARS_DEV Walk q_walk(const GradArgs& a) { 
  return Walk(a.plan.count, a.plan.by_cost, a.hq, blockIdx.x - a.k_ctas, a.q_ctas);
}

MARS_DEV bool take(Walk& w, QItem& it) {
  if (!w.take(it.t, it.h)) return false;
  it.n = it.t.tile + 1;
  return true;
}

template <int D>
MARS_DEV void dq(const CUtensorMap& tm_q, const CUtensorMap& tm_do, const CUtensorMap& tm_k,
                 const CUtensorMap& tm_v, const GradArgs& a, uint8_t* smem_raw) {
  using S = flash::Smem<D, D / 64>;                 // the dO tile over the staging area
  static_assert(D * GT * 2 <= (D / 64) * GT * 128, "dO tile fits the staging area");
  constexpr int TM_S = 0, TM_DP = GT, TM_DQ = 2 * GT, TM_DS = 3 * GT;
  __shared__ flash::Barriers bar;
  __shared__ QBar qb;
  const uint32_t raw = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + (((raw + 1023u) & ~1023u) - raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  Walk walk = q_walk(a);
  if (walk.id < 0) return;                             // more CTAs than items
  if (threadIdx.x == 0) {
    mbar_init(&qb.s_full, 1);
    mbar_init(&qb.dp_full, 1);
    mbar_init(&qb.dq_done, 1);
    mbar_init(&qb.s_free, MATH_THREADS);
    mbar_init(&qb.dp_free, MATH_THREADS);
    mbar_init(&qb.ds_full, MATH_THREADS);
    mbar_init(&qb.acc_free, MATH_THREADS);
    flash::init_barriers(bar);
  }
  if (warp == 1) {
    tmem_alloc(&bar.tmem_base, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, bar.tmem_base, 0);
  volatile int* ab = &bar.abort;

  if (warp == 0 || warp == Q_V_WARP) {
    const bool is_v = warp != 0;
    int last_k[flash::K_STAGES], last_v[flash::V_STAGES];
    for (int i = 0; i < flash::K_STAGES; ++i) last_k[i] = -1;
    for (int i = 0; i < flash::V_STAGES; ++i) last_v[i] = -1;
    int j0 = 0, z = 0, kvh = 0;
    auto issue = [&](int j, uint8_t* dst, uint64_t* b) {
      if (lane == 0)
        for (int x = 0; x < D / 64; ++x)
          tma_load_3d(dst + x * (GT * 128), is_v ? &tm_v : &tm_k, b, x * 64, kvh, z + j * GT);
    };
    auto ring = [&](int n, bool drain) {
      return is_v ? flash::load_ring_item<D, flash::V_STAGES>(bar, smem, n, j0, last_v, drain,
                                                              a.status, true, issue)
                  : flash::load_ring_item<D, flash::K_STAGES>(bar, smem, n, j0, last_k, drain,
                                                              a.status, false, issue);
    };
    QItem it;
    while (take(walk, it)) {
      z = it.t.base;
      kvh = it.h / a.G;
      if (!ring(it.n, false)) break;
      j0 += it.n;
    }
    ring(0, true);                                   // wait (bounded) for copies in flight
  } else if (warp == 1) {
    if (elect_one()) {
      const uint32_t id_s = idesc_bf16_f32(GT, GT, false);
      const uint64_t qd = sdesc_sw128(smem_u32(smem + S::OFF_Q), 16, 1024);
      const uint64_t dd = sdesc_sw128(smem_u32(smem + S::OFF_STAGE), 16, 1024);
      int jg = 0, i = 0, nq = 0;
      bool ok = true;
      auto product = [&](uint64_t ad, int off_b, int col, uint64_t* full) {
        const uint64_t bd = sdesc_sw128(smem_u32(smem + off_b), 16, 1024);
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint32_t off = (k >> 2) * (GT * 128) + (k & 3) * 32;
          mma_bf16_ss(tmem + col, sdesc_advance(ad, off), sdesc_advance(bd, off), id_s, k != 0);
        }
        mma_commit(full);
      };
      QItem it;
      while (ok && take(walk, it)) {
        // Q and dO are replaced once the previous item's S and dP MMAs have completed
        if (i > 0 && !(ok = mbar_wait(&bar.q_empty, (i - 1) & 1, ab, a.status))) break;
        mbar_arrive_expect_tx(&bar.q_full, 2 * S::Q_BYTES);
        const int z = it.t.base + GT * it.t.tile;
        for (int x = 0; x < D / 64; ++x) {
          tma_load_3d(smem + S::OFF_Q + x * (GT * 128), &tm_q, &bar.q_full, x * 64, it.h, z);
          tma_load_3d(smem + S::OFF_STAGE + x * (GT * 128), &tm_do, &bar.q_full, x * 64, it.h, z);
        }
        ++nq;
        if (!(ok = mbar_wait(&bar.q_full, i & 1, ab, a.status))) break;
        for (int j = 0; j < it.n && ok; ++j, ++jg) {
          const int sk = jg % flash::K_STAGES, sv = jg % flash::V_STAGES;
          // S and dP of the previous tile have been loaded by the math warps
          ok = mbar_wait(&bar.k_full[sk], (jg / flash::K_STAGES) & 1, ab, a.status) &&
               (jg == 0 || mbar_wait(&qb.s_free, (jg - 1) & 1, ab, a.status));
          if (!ok) break;
          tc_fence_after();
          product(qd, S::OFF_K + sk * S::KV_BYTES, TM_S, &qb.s_full);
          ok = mbar_wait(&bar.v_full[sv], (jg / flash::V_STAGES) & 1, ab, a.status) &&
               (jg == 0 || mbar_wait(&qb.dp_free, (jg - 1) & 1, ab, a.status));
          if (!ok) break;
          tc_fence_after();
          product(dd, S::OFF_V + sv * S::KV_BYTES, TM_DP, &qb.dp_full);
          mma_commit(&bar.v_empty[sv]);
        }
        if (!ok) break;
        mma_commit(&bar.q_empty);
        ++i;
      }
      mma_commit(&bar.drain);
      mbar_wait(&bar.drain, 0, nullptr, a.status);
      if (nq > 0) mbar_wait(&bar.q_full, (nq - 1) & 1, nullptr, a.status);
    }
  } else if (warp == Q_TS_WARP) {
    if (elect_one()) {
      const uint32_t id_q = idesc_bf16_f32(GT, D, true);       // A from TMEM, B MN-major
      int jg = 0, i = 0;
      bool ok = true;
      QItem it;
      while (ok && take(walk, it)) {
        for (int j = 0; j < it.n; ++j, ++jg) {
          const int st = jg % flash::K_STAGES;
          // the previous item's accumulator has been read out
          ok = (j > 0 || i == 0 || mbar_wait(&qb.acc_free, (i - 1) & 1, ab, a.status)) &&
               mbar_wait(&bar.k_full[st], (jg / flash::K_STAGES) & 1, ab, a.status) &&
               mbar_wait(&qb.ds_full, jg & 1, ab, a.status);
          if (!ok) break;
          tc_fence_after();
          const uint64_t kd =
              sdesc_sw128(smem_u32(smem + S::OFF_K + st * S::KV_BYTES), GT * 128, 1024);
#pragma unroll
          for (int k = 0; k < GT / 16; ++k)
            mma_bf16_ts(tmem + TM_DQ, tmem + TM_DS + 8 * k, sdesc_advance(kd, k * 2048), id_q,
                        (j | k) != 0);
          mma_commit(&qb.dq_done);
          // S, which also read this stage, completed before the math warps wrote dS
          mma_commit(&bar.k_empty[st]);
        }
        if (!ok) break;
        mma_commit(&bar.o_final);
        ++i;
      }
      mma_commit(&bar.drain_pv);
      mbar_wait(&bar.drain_pv, 0, nullptr, a.status);
    }
  } else {
    // math: thread = query row (TMEM lane), 64 key columns per warp
    const int quad = warp & 3, half = (warp - 2) >> 2;
    const int row = quad * 32 + lane;
    const uint32_t lane_off = (uint32_t)(quad * 32) << 16;
    auto warp_wait = [&](uint64_t* b, uint32_t parity) -> bool {
      return __all_sync(0xffffffffu, mbar_wait(b, parity, ab, a.status));
    };
    int jg = 0, i = 0;
    bool ok = true;
    // lse and D of this thread's row of an item (zeros past the sequence), read ahead
    auto stats = [&](const Tile& t, int h) {
      const size_t at = (size_t)h * a.pad + (size_t)t.id * GT + row;
      return make_float2(a.lse_p[at], a.d_p[at]);
    };
    float2 ahead = stats(walk.tile, walk.id % a.hq);
    QItem it;
    while (ok && take(walk, it)) {
      const int live = it.t.n - GT * it.t.tile;         // query rows of the tile
      const bool rv = row < live;
      const float lse = ahead.x, dd = ahead.y;
      for (int j = 0; j < it.n; ++j, ++jg) {
        const bool diag = j == it.t.tile;
        if (!(ok = warp_wait(&qb.s_full, jg & 1))) break;
        tc_fence_after();
        uint32_t sv[64];
#pragma unroll
        for (int q = 0; q < 2; ++q)
          tmem_ld32(tmem + TM_S + 64 * half + 32 * q + lane_off,
                    *reinterpret_cast<uint32_t(*)[32]>(sv + 32 * q));
        tmem_ld_wait();
        tc_fence_before();
        mbar_arrive_warp(&qb.s_free);
        // keys this row sees among the warp's columns: on the diagonal tile 0 .. row
        uint32_t mk[2] = {0xffffffffu, 0xffffffffu};
        if (diag || !rv) {
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            mk[q] = rv ? bits(0, row + 1 - 64 * half - 32 * q) : 0u;
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (!((mk[q] >> e) & 1u)) sv[32 * q + e] = 0xff800000u;
          }
        }
        float pf[64];
        const float2 sc2 = make_float2(a.scale_log2, a.scale_log2);
        const float2 nl2 = make_float2(-lse, -lse), nd2 = make_float2(-dd, -dd);
#pragma unroll
        for (int e = 0; e < 64; e += 2) {
          const float2 s2 = make_float2(__uint_as_float(sv[e]), __uint_as_float(sv[e + 1]));
          const float2 t = __ffma2_rn(s2, sc2, nl2);
          pf[e] = flash::ex2_approx(t.x);
          pf[e + 1] = flash::ex2_approx(t.y);
        }
        if (!(ok = warp_wait(&qb.dp_full, jg & 1))) break;
        tc_fence_after();
#pragma unroll
        for (int q = 0; q < 2; ++q)
          tmem_ld32(tmem + TM_DP + 64 * half + 32 * q + lane_off,
                    *reinterpret_cast<uint32_t(*)[32]>(sv + 32 * q));
        tmem_ld_wait();
        tc_fence_before();
        mbar_arrive_warp(&qb.dp_free);
        if (diag || !rv) {                             // masked dP may hold anything
#pragma unroll
          for (int q = 0; q < 2; ++q)
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (!((mk[q] >> e) & 1u)) sv[32 * q + e] = 0u;
        }
        if (diag && live < GT) {
          // K rows past the sequence, which the MMA of S has read
          clear_rows<D>(smem + S::OFF_K + (jg % flash::K_STAGES) * S::KV_BYTES, live, 0, GT,
                        (warp - 2) * 32 + lane, MATH_THREADS);
          fence_proxy_async_smem();
        }
        uint32_t ds[32];
#pragma unroll
        for (int e = 0; e < 64; e += 2) {
          const float2 x = __fmul2_rn(make_float2(pf[e], pf[e + 1]),
                                      __fadd2_rn(make_float2(__uint_as_float(sv[e]),
                                                             __uint_as_float(sv[e + 1])), nd2));
          ds[e / 2] = flash::pack_bf16x2(x.x, x.y);
        }
        if (it.t.tile == 0 && row == 0 && half == 0) ds[0] = clear_low(ds[0]);   // dS of row 0 is 0
        // dS has one buffer: the previous tile's dQ MMA must have read it
        if (jg > 0 && !(ok = warp_wait(&qb.dq_done, (jg - 1) & 1))) break;
        tc_fence_after();
        tmem_st32(tmem + TM_DS + 32 * half + lane_off, ds);
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive_warp(&qb.ds_full);
      }
      if (!ok) break;
      if (walk.id >= 0) ahead = stats(walk.tile, walk.id % a.hq);
      if (!(ok = warp_wait(&bar.o_final, i & 1))) break;
      tc_fence_after();
      constexpr int HD = D / 2;
      uint32_t o[HD];
#pragma unroll
      for (int q = 0; q < HD / 32; ++q)
        tmem_ld32(tmem + TM_DQ + HD * half + 32 * q + lane_off,
                  *reinterpret_cast<uint32_t(*)[32]>(o + 32 * q));
      tmem_ld_wait();
      tc_fence_before();
      mbar_arrive_warp(&qb.acc_free);
      const long long tok = (long long)it.t.base + GT * it.t.tile + row;
      const long long at = rv ? tok * a.dq_stride + it.h * D + HD * half : -1;
      packed::store_rows<HD>(a.dq, at, lane,
                             [&](int e) { return __uint_as_float(o[e]) * a.scale; });
      ++i;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// The first k_ctas CTAs compute dK and dV, the others dQ: one launch, so that dQ's CTAs take over
// the SMs as they become free, and small problems run side by side.
template <int D>
__global__ void __launch_bounds__(K_THREADS, 1)
grad_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_do,
            const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
            GradArgs a) {
  extern __shared__ uint8_t smem_raw[];
  static_assert(K_THREADS == Q_THREADS, "one launch for both");
  if ((int)blockIdx.x < a.k_ctas)
    dkdv<D>(tm_q, tm_do, tm_k, tm_v, a, smem_raw);
  else
    dq<D>(tm_q, tm_do, tm_k, tm_v, a, smem_raw);
}

// ------------------------------------------------------------------------------- host

// CTAs of dkdv: one per SM, or as many as the most work that `total` rows can make (one
// sequence) feeds.
int k_ctas(int batch, int total, int hq, int hkv) {
  const long long tiles = packed::max_tiles(batch, total, GT);
  const long long work = hq * (packed::kPairWork * (tiles * (tiles + 1) / 2) + tiles) +
                         hkv * packed::kTileWork * tiles;
  return (int)std::max(1LL, std::min<long long>(num_sms(), work / kMinWork));
}

long long prep_ctas(long long tiles, int hq) {
  return 1 + tiles * (GT / PREP_ROWS) * ((hq + PREP_HEADS - 1) / PREP_HEADS);
}

struct GradSpace {
  packed::Plan plan;
  float *lse_p, *d_p, *part;
  size_t bytes;
};

GradSpace carve(void* base, int batch, int total, int hq, int hkv, int d) {
  GradSpace g{};
  size_t off = 0;
  const int ctas = k_ctas(batch, total, hq, hkv);
  g.plan = packed::carve_plan(base, off, batch, total, ctas);
  uint8_t* p = static_cast<uint8_t*>(base);
  auto take = [&](size_t n) {
    float* at = p ? reinterpret_cast<float*>(p + off) : nullptr;
    off += packed::align256(n * sizeof(float));
    return at;
  };
  const size_t rows = (size_t)packed::max_tiles(batch, total, GT) * GT;
  g.lse_p = take(rows * hq);
  g.d_p = take(rows * hq);
  g.part = take((size_t)ctas * 4 * GT * d);
  g.bytes = off;
  return g;
}

bool map3(CUtensorMap* m, const void* base, int d, int heads, int total, long long stride) {
  const uint64_t dims[3] = {(uint64_t)d, (uint64_t)heads, (uint64_t)total};
  const uint64_t str[2] = {(uint64_t)d * 2, (uint64_t)stride * 2};
  const uint32_t box[3] = {64, 1, GT};
  return encode_tmap_bf16(m, base, 3, dims, str, box);
}

template <int D>
cudaError_t launch_grad(const PackedGrad& p, GradArgs& a, cudaStream_t stream) {
  CUtensorMap tq, tdo, tk, tv;
  if (!map3(&tq, p.q, D, p.hq, p.total, p.q_stride) ||
      !map3(&tdo, p.d_o, D, p.hq, p.total, (long long)p.hq * D) ||
      !map3(&tk, p.k, D, p.hkv, p.total, p.k_stride) ||
      !map3(&tv, p.v, D, p.hkv, p.total, p.v_stride))
    return cudaErrorInvalidValue;
  using SK = KSmem<D>;
  using SQ = flash::Smem<D, D / 64>;
  constexpr int kSmem = std::max<int>(SK::TOTAL, SQ::TOTAL);
  static_assert(kSmem + sizeof(KBar) + sizeof(KStart) + sizeof(flash::Barriers) + sizeof(QBar) <=
                    227 * 1024,
                "both layouts fit shared memory");
  static std::atomic<int> attr[64];
  const cudaError_t e = set_smem_limit_once(grad_kernel<D>, kSmem, attr);
  if (e != cudaSuccess) return e;
  const long long tiles = packed::max_tiles(p.batch, p.total, GT);
  prep_kernel<D><<<(unsigned)prep_ctas(tiles, p.hq), packed::kPlanThreads, 0, stream>>>(
      a, packed::PlanArgs{a.plan, p.cu, p.batch, p.total, a.G, a.k_ctas, p.status});
  grad_kernel<D><<<(unsigned)(a.k_ctas + a.q_ctas), K_THREADS, kSmem, stream>>>(tq, tdo, tk, tv, a);
  count_launches(2);
  return cudaGetLastError();
}

}  // namespace

long long packed_grad_items(int batch, int total, int hq) {
  const long long tiles = packed::max_tiles(batch, total, GT);
  return std::max(tiles * hq, prep_ctas(tiles, hq));
}

size_t packed_grad_workspace_bytes(int batch, int total, int hq, int hkv, int d) {
  return carve(nullptr, batch, total, hq, hkv, d).bytes;
}

cudaError_t launch_packed_grad(const PackedGrad& p, void* workspace, cudaStream_t stream) {
  const GradSpace g = carve(workspace, p.batch, p.total, p.hq, p.hkv, p.d);
  GradArgs a{};
  a.plan = g.plan;
  a.total = p.total;
  a.hq = p.hq;
  a.hkv = p.hkv;
  a.G = p.hq / p.hkv;
  const long long tiles = packed::max_tiles(p.batch, p.total, GT);
  a.pad = tiles * GT;
  a.k_ctas = k_ctas(p.batch, p.total, p.hq, p.hkv);
  a.q_ctas = (int)std::min<long long>(num_sms(), tiles * p.hq);
  a.scale = p.scale;
  a.scale_log2 = p.scale * 1.4426950408889634f;
  a.o = p.o;
  a.d_o = p.d_o;
  a.lse = p.lse;
  a.lse_p = g.lse_p;
  a.d_p = g.d_p;
  a.dq = p.dq;
  a.dk = p.dk;
  a.dv = p.dv;
  a.dq_stride = p.dq_stride;
  a.dk_stride = p.dk_stride;
  a.dv_stride = p.dv_stride;
  a.part = g.part;
  a.status = p.status;
  return p.d == 64 ? launch_grad<64>(p, a, stream) : launch_grad<128>(p, a, stream);
}

}  // namespace mars
