// Tile lists of a packed batch for its gradient: one CTA reads the sequence boundaries, counts
// the 128-row tiles of each sequence and writes them out in their order, with the work before
// each, and in the order of falling cost (a counting sort over kBuckets cost classes, so that
// the list is sorted to about a five-hundredth of the largest cost). Entries of one class come
// in any order: that moves work between CTAs, not results.
#pragma once

#include "common.cuh"
#include "packed.cuh"

namespace mars {
namespace packed {

constexpr int kPlanThreads = 256;
constexpr int kBuckets = 2 * kPlanThreads;

struct PlanArgs {
  Plan plan;
  const int32_t* cu;
  int batch, total, groups, ntickets;
  int32_t* status;
};

// Inclusive scan over the CTA of a sum or a maximum; s_warp holds one value per warp.
template <bool kMax, class T>
MARS_DEV T scan(T v, T* s_warp) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  auto join = [](T a, T b) { return kMax ? max(a, b) : a + b; };
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v = join(v, u);
  }
  if (lane == 31) s_warp[warp] = v;
  __syncthreads();
  for (int w = 0; w < warp; ++w) v = join(v, s_warp[w]);
  __syncthreads();
  return v;
}

// One CTA of kPlanThreads threads: fill a.plan.
MARS_DEV void make_plan(const PlanArgs& a) {
  __shared__ int s_warp[kPlanThreads / 32];
  __shared__ long long s_warp64[kPlanThreads / 32];
  __shared__ int s_hist[kBuckets];
  __shared__ int s_base[kPlanThreads], s_n[kPlanThreads], s_off[kPlanThreads];
  __shared__ long long s_pre[kPlanThreads], s_work;
  __shared__ int s_top, s_tiles, s_cost;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  bool bad = false;
  const auto tiles_of = [](int n) { return (n + kTileRows - 1) / kTileRows; };

  // A pass over the sequences, kPlanThreads at a time, calls f(base, n, first tile, tiles, work
  // before) with one warp per sequence. The chunk's arrays are kept for the next pass where
  // there is one chunk only.
  auto each = [&](bool first, auto f) {
    if (tid == 0 && (first || a.batch > kPlanThreads)) {
      const int c0 = a.cu[0];
      s_top = min(max(c0, 0), a.total);
      s_tiles = 0;
      s_work = 0;
      bad |= c0 != s_top;
    }
    __syncthreads();
    for (int s0 = 0; s0 < a.batch; s0 += kPlanThreads) {
      if (first || a.batch > kPlanThreads) {
        const int s = s0 + tid, top = s_top, tiles0 = s_tiles;
        const long long work0 = s_work;
        const int c = s < a.batch ? a.cu[s + 1] : top;
        const int end = scan<true>(max(min(max(c, 0), a.total), top), s_warp);
        if (s < a.batch && c != end) bad = true;
        s_n[tid] = end;
        __syncthreads();
        const int begin = tid ? s_n[tid - 1] : top;
        __syncthreads();
        const int n = end - begin, mine = s < a.batch ? tiles_of(n) : 0;
        const int incl = scan<false>(mine, s_warp);
        const long long work = work_before(a.groups, mine, mine);
        const long long sum = scan<false>(work, s_warp64);
        s_base[tid] = begin;
        s_n[tid] = n;
        s_off[tid] = tiles0 + incl - mine;
        s_pre[tid] = work0 + sum - work;
        if (tid == kPlanThreads - 1) {
          s_top = end;
          s_tiles = tiles0 + incl;
          s_work = work0 + sum;
        }
        __syncthreads();
      }
      for (int i = warp; i < min(kPlanThreads, a.batch - s0); i += kPlanThreads / 32)
        f(s_base[i], s_n[i], s_off[i], tiles_of(s_n[i]), s_pre[i]);
      __syncthreads();
    }
  };

  for (int i = tid; i < kBuckets; i += kPlanThreads) s_hist[i] = 0;
  for (int i = tid; i < a.ntickets; i += kPlanThreads) a.plan.tickets[i] = 0;
  if (tid == 0) s_cost = 1;
  __syncthreads();
  each(true, [&](int, int, int, int tiles, long long) {
    if (lane == 0) atomicMax(&s_cost, tiles);
  });
  const int most = s_cost;
  // class of a tile that sees t + 1 key tiles
  auto bucket = [&](int t) {
    return kBuckets - 1 - (int)((long long)(t + 1) * (kBuckets - 1) / most);
  };
  each(false, [&](int, int, int, int tiles, long long) {
    for (int t = lane; t < tiles; t += 32) atomicAdd(&s_hist[bucket(t)], 1);
  });
  int* h = s_hist + 2 * tid;                           // first place of each class
  const int v0 = h[0], v1 = h[1];
  const int before = scan<false>(v0 + v1, s_warp) - v0 - v1;
  h[0] = before;
  h[1] = before + v0;
  __syncthreads();
  each(false, [&](int base, int n, int off, int tiles, long long pre) {
    for (int t = lane; t < tiles; t += 32) {
      const Tile e{base, n, t, off + t};
      a.plan.by_cost[atomicAdd(&s_hist[bucket(t)], 1)] = e;
      a.plan.in_order[off + t] = e;
      a.plan.before[off + t] = pre + work_before(a.groups, tiles, t);
    }
  });
  if (tid == 0) {
    a.plan.before[s_tiles] = s_work;
    *a.plan.count = s_tiles;
  }
  if (bad && a.status) atomicOr(a.status, MARS_ST_BADSEQ);
}

}  // namespace packed
}  // namespace mars
