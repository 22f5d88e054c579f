// Packed batches: the rows of `batch` sequences stand one after another in [total] rows, and
// sequence s owns rows cu[s] .. cu[s+1] - 1. The kernels never trust cu for addresses:
// boundaries are clamped to [0, total] and made non-decreasing (a running maximum), so that
// every sequence lies inside the tensors and the sequences' tiles number at most
// total / rows_per_tile + batch, which sizes the grids on the host.
#pragma once

#include "common.cuh"

namespace mars {
namespace packed {

struct Seq {
  int s;          // sequence, or -1: no such tile
  int tile;       // tile index inside the sequence
  int base, n;    // first row and number of rows of the sequence
};

inline long long max_tiles(int batch, int total, int rows_per_tile) {
  return (long long)total / rows_per_tile + batch;
}

// The sequence and tile of global tile index i (tiles of the sequences in order, each of
// `rows` rows and at least `least` tiles per sequence). Whole warp; the result is uniform.
// end = the last boundary, bad = whether cu was malformed (only where the scan got to).
MARS_DEV Seq find_tile(const int32_t* __restrict__ cu, int batch, int total, int rows, int least,
                       long long i, bool& bad) {
  const int lane = threadIdx.x & 31;
  long long tiles = 0;                         // tiles of the sequences before this group
  const int c0 = cu[0];
  int top = min(max(c0, 0), total);            // running maximum of the boundaries
  bad = c0 != top;
  for (int s0 = 0; s0 < batch; s0 += 32) {
    const int s = s0 + lane;
    const int c = s < batch ? cu[s + 1] : top;
    int e = min(max(c, 0), total);
    int m = max(e, top);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, m, o);
      if (lane >= o) m = max(m, v);
    }
    bad |= __any_sync(0xffffffffu, s < batch && c != m) != 0;
    int begin = __shfl_up_sync(0xffffffffu, m, 1);
    if (lane == 0) begin = top;
    const int n = m - begin;
    const int mine = s < batch ? max((n + rows - 1) / rows, least) : 0;
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    const uint32_t hit = __ballot_sync(0xffffffffu, i < tiles + incl);
    if (hit) {
      const int l = __ffs(hit) - 1;
      Seq q;
      q.s = s0 + l;
      q.tile = (int)(i - tiles) - __shfl_sync(0xffffffffu, incl - mine, l);
      q.base = __shfl_sync(0xffffffffu, begin, l);
      q.n = __shfl_sync(0xffffffffu, n, l);
      return q;
    }
    tiles += __shfl_sync(0xffffffffu, incl, 31);
    top = __shfl_sync(0xffffffffu, m, 31);
  }
  return Seq{-1, 0, top, 0};
}

// A tile of a sequence in a plan's lists.
struct alignas(16) Tile {
  int base, n;    // first row and number of rows of its sequence
  int tile;       // tile index inside the sequence
  int id;         // sequence (by_cost of a forward plan) or global tile index (a gradient's)
};

// Lists of the tiles of a packed batch, made on the device (the boundaries are there), for
// kernels that run many tiles per CTA: CTAs take a list's entries in turn, so each is sorted
// by falling cost, the number of 128-key (or 128-row) tiles that an entry visits.
struct Plan {
  int32_t* count;     // number of tiles
  Tile* first;        // by the keys a tile's rows see (forward, dQ)
  Tile* second;       // gradient: by the rows that see a tile's keys (dK, dV)
  Tile* in_order;     // gradient: by global tile index
};

// The items of a persistent CTA, by round: rounds run forwards and backwards over the CTAs, so that the costs even out.
struct Turns {
  int total, rounds;
  MARS_DEV explicit Turns(int n) : total(n), rounds((n + (int)gridDim.x - 1) / (int)gridDim.x) {}
  MARS_DEV int at(int r) const {
    const int g = gridDim.x, c = blockIdx.x;
    const int id = r * g + ((r & 1) ? g - 1 - c : c);
    return id < total ? id : -1;
  }
};

inline size_t align256(size_t x) { return (x + 255) / 256 * 256; }

// Carve a plan out of a workspace at `off` (base may be null to size it).
inline Plan carve_plan(void* base, size_t& off, int batch, int total, int rows, bool grad) {
  uint8_t* p = static_cast<uint8_t*>(base);
  auto take = [&](size_t bytes) {
    uint8_t* at = p ? p + off : nullptr;
    off += align256(bytes);
    return at;
  };
  const size_t list = (size_t)max_tiles(batch, total, rows) * sizeof(Tile);
  Plan r{};
  r.count = reinterpret_cast<int32_t*>(take(sizeof(int32_t)));
  r.first = reinterpret_cast<Tile*>(take(list));
  if (grad) {
    r.second = reinterpret_cast<Tile*>(take(list));
    r.in_order = reinterpret_cast<Tile*>(take(list));
  }
  return r;
}

// Fill a plan. rows: rows per tile (128 for a gradient); seq_lens: cached keys per sequence
// (NULL: none), cut to what max_pages pages hold.
cudaError_t launch_plan(const Plan& plan, const int32_t* cu, const int32_t* seq_lens,
                        int max_pages, int batch, int total, int rows, int32_t* status,
                        cudaStream_t stream);

}  // namespace packed
}  // namespace mars
