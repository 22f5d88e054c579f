// Tile lists of a packed batch (packed.cuh): one CTA reads the sequence boundaries, counts the
// tiles of each sequence and writes them out in the order of falling cost (a counting sort
// over kBuckets cost classes, so that the list is sorted to about a two-thousandth of the
// largest cost). Entries of one class come in any order: that moves work between CTAs, not
// results.
#include "common.cuh"
#include "internal.h"
#include "packed.cuh"

namespace mars {
namespace packed {

namespace {

constexpr int kThreads = 1024;
constexpr int kBuckets = 2048;
constexpr int kTile = 128;

struct PlanArgs {
  Plan plan;
  const int32_t *cu, *seq_lens;
  int max_pages, batch, total, rows;
  int32_t* status;
};

// Inclusive scan over the CTA of a sum or a maximum; s_warp holds one value per warp.
template <bool kMax>
MARS_DEV int scan(int v, int* s_warp) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  auto join = [](int a, int b) { return kMax ? max(a, b) : a + b; };
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v = join(v, u);
  }
  if (lane == 31) s_warp[warp] = v;
  __syncthreads();
  if (warp == 0) {
    int w = s_warp[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w = join(w, u);
    }
    s_warp[lane] = w;
  }
  __syncthreads();
  if (warp > 0) v = join(v, s_warp[warp - 1]);
  __syncthreads();
  return v;
}

__global__ void __launch_bounds__(kThreads) plan_kernel(PlanArgs a) {
  __shared__ int s_warp[32];
  __shared__ int s_hist[2][kBuckets];
  __shared__ int s_base[kThreads], s_n[kThreads], s_off[kThreads], s_old[kThreads];
  __shared__ int s_top, s_tiles, s_cost;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const bool grad = a.plan.second != nullptr;
  bool bad = false;

  // A pass over the sequences, kThreads at a time, calls f(sequence, base, n, first global
  // tile, tiles, cached key tiles) with one warp per sequence.
  auto each = [&](auto f) {
    if (tid == 0) {
      const int c0 = a.cu[0];
      s_top = min(max(c0, 0), a.total);
      s_tiles = 0;
      bad |= c0 != s_top;
    }
    __syncthreads();
    for (int s0 = 0; s0 < a.batch; s0 += kThreads) {
      const int s = s0 + tid, top = s_top, tiles0 = s_tiles;
      const int c = s < a.batch ? a.cu[s + 1] : top;
      const int end = scan<true>(max(min(max(c, 0), a.total), top), s_warp);
      if (s < a.batch && c != end) bad = true;
      s_n[tid] = end;
      __syncthreads();
      const int begin = tid ? s_n[tid - 1] : top;
      __syncthreads();
      const int n = end - begin, mine = s < a.batch ? (n + a.rows - 1) / a.rows : 0;
      const int incl = scan<false>(mine, s_warp);
      s_base[tid] = begin;
      s_n[tid] = n;
      s_off[tid] = tiles0 + incl - mine;
      int old = 0;
      if (a.seq_lens && s < a.batch) {
        const long long p = min((long long)a.seq_lens[s], (long long)a.max_pages * kPageSize);
        old = p > 0 ? (int)((p + kTile - 1) / kTile) : 0;
      }
      s_old[tid] = old;
      if (tid == kThreads - 1) {
        s_top = end;
        s_tiles = tiles0 + incl;
      }
      __syncthreads();
      for (int i = warp; i < min(kThreads, a.batch - s0); i += kThreads / 32)
        f(s0 + i, s_base[i], s_n[i], s_off[i], (s_n[i] + a.rows - 1) / a.rows, s_old[i]);
      __syncthreads();
    }
  };
  // key tiles that tile t's rows see
  auto cost = [&](int n, int t, int old) {
    const int last = min((long long)(t + 1) * a.rows, (long long)n) - 1;
    return old + last / kTile + 1;
  };

  for (int i = tid; i < 2 * kBuckets; i += kThreads) (&s_hist[0][0])[i] = 0;
  if (tid == 0) s_cost = 1;
  __syncthreads();
  each([&](int, int, int n, int, int tiles, int old) {
    if (lane == 0 && tiles > 0) atomicMax(&s_cost, cost(n, tiles - 1, old));
  });
  const int most = s_cost;
  auto bucket = [&](int c) { return kBuckets - 1 - (int)((long long)c * (kBuckets - 1) / most); };
  each([&](int, int, int n, int, int tiles, int old) {
    for (int t = lane; t < tiles; t += 32) {
      atomicAdd(&s_hist[0][bucket(cost(n, t, old))], 1);
      if (grad) atomicAdd(&s_hist[1][bucket(tiles - t)], 1);
    }
  });
  for (int l = 0; l < (grad ? 2 : 1); ++l) {           // first place of each class
    int2* h = reinterpret_cast<int2*>(s_hist[l]) + tid;
    const int2 v = *h;
    const int before = scan<false>(v.x + v.y, s_warp) - v.x - v.y;
    *h = make_int2(before, before + v.x);
  }
  static_assert(kBuckets == 2 * kThreads, "two classes per thread");
  __syncthreads();
  each([&](int s, int base, int n, int off, int tiles, int old) {
    for (int t = lane; t < tiles; t += 32) {
      const Tile e{base, n, t, grad ? off + t : s};
      a.plan.first[atomicAdd(&s_hist[0][bucket(cost(n, t, old))], 1)] = e;
      if (grad) {
        a.plan.second[atomicAdd(&s_hist[1][bucket(tiles - t)], 1)] = e;
        a.plan.in_order[off + t] = e;
      }
    }
  });
  if (tid == 0) *a.plan.count = s_tiles;
  if (bad && a.status) atomicOr(a.status, MARS_ST_BADSEQ);
}

}  // namespace

cudaError_t launch_plan(const Plan& plan, const int32_t* cu, const int32_t* seq_lens,
                        int max_pages, int batch, int total, int rows, int32_t* status,
                        cudaStream_t stream) {
  plan_kernel<<<1, kThreads, 0, stream>>>(
      PlanArgs{plan, cu, seq_lens, max_pages, batch, total, rows, status});
  count_launches(1);
  return cudaGetLastError();
}

}  // namespace packed
}  // namespace mars
