// Packed batches: the rows of `batch` sequences stand one after another in [total] rows, and
// sequence s owns rows cu[s] .. cu[s+1] - 1. The kernels never trust cu for addresses:
// boundaries are clamped to [0, total] and made non-decreasing (a running maximum), so that
// every sequence lies inside the tensors and the sequences' tiles number at most
// total / rows_per_tile + batch, which sizes the grids on the host.
#pragma once

#include <cuda_bf16.h>

#include "common.cuh"

namespace mars {
namespace packed {

struct Seq {
  int s;          // sequence, or -1: no such tile
  int tile;       // tile index inside the sequence
  int base, n;    // first row and number of rows of the sequence
  int len;        // lens[s]
};

// 128-key tiles of `keys` keys. Rounding up by adding 127 first would pass 31 bits for the last 127
// counts that an int holds, which a max_len_hint ("no bound") or a length may have.
__host__ __device__ constexpr int key_tiles(int keys) { return keys / 128 + (keys % 128 != 0); }
static_assert(key_tiles(0x7fffffff) == 1 << 24 && key_tiles(0x7fffff80) == (1 << 24) - 1 &&
                  key_tiles(1) == 1 && key_tiles(0) == 0,
              "tiles of any int");

inline long long max_tiles(int batch, int total, int rows_per_tile) {
  return (long long)total / rows_per_tile + batch;
}

// The sequence and tile of global tile index i (tiles of the sequences in order, each of
// `rows` rows and at least `least` tiles per sequence). Whole warp; the result is uniform.
// bad = whether cu was malformed (only where the scan got to). lens [batch] or NULL is read with
// the boundaries: after them it would be a further trip to memory before the tile can start.
MARS_DEV Seq find_tile(const int32_t* __restrict__ cu, int batch, int total, int rows, int least,
                       long long i, bool& bad, const int32_t* lens = nullptr) {
  const int lane = threadIdx.x & 31;
  long long tiles = 0;                         // tiles of the sequences before this group
  const int c0 = cu[0];
  int top = min(max(c0, 0), total);            // running maximum of the boundaries
  bad = c0 != top;
  for (int s0 = 0; s0 < batch; s0 += 32) {
    const int s = s0 + lane;
    const int c = s < batch ? cu[s + 1] : top;
    const int len = lens && s < batch ? lens[s] : 0;
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
      q.len = __shfl_sync(0xffffffffu, len, l);
      return q;
    }
    tiles += __shfl_sync(0xffffffffu, incl, 31);
    top = __shfl_sync(0xffffffffu, m, 31);
  }
  return Seq{-1, 0, top, 0, 0};
}

constexpr int kTileRows = 128;

// A 128-row tile of a sequence in a plan's lists.
struct alignas(16) Tile {
  int base, n;    // first row and number of rows of its sequence
  int tile;       // tile index inside the sequence
  int id;         // index among all tiles, in the order of the sequences
};

// Lists of the tiles of a packed batch, made on the device (the boundaries are there), for the
// gradient's kernels, which run many tiles per CTA.
struct Plan {
  int32_t* count;     // number of tiles
  Tile* by_cost;      // by falling number of keys that a tile's rows see (dQ)
  Tile* in_order;     // by id
  long long* before;  // [count + 1]: dK / dV work of one KV head before each tile, and of all
  int32_t* tickets;   // zeroed
};

// Work of dK and dV of a key tile and a KV head with `groups` query heads: kPairWork for each
// (query head, query tile) pair, 1 more for each on the diagonal (its masks), and kTileWork for
// the tile's start and output; a unit is about 900 cycles.
constexpr int kPairWork = 3, kTileWork = 6;

// That of a tile with `after` query tiles, and of the first t of a sequence's tiles.
MARS_DEV int tile_work(int groups, int after) {
  return groups * (kPairWork * after + 1) + kTileWork;
}
MARS_DEV long long work_before(int groups, long long tiles, long long t) {
  return groups * (kPairWork * (t * tiles - t * (t - 1) / 2) + t) + kTileWork * t;
}

// The items (tile of a list, head) of a persistent CTA. Rounds run forwards and backwards over
// the CTAs, so that the costs even out. The next item's tile is read while the current one is
// worked on: at its turn the read cost 800 cycles and more.
struct Walk {
  const Tile* list;
  int heads, total, cta, ctas;         // items per tile, items; CTA and CTAs
  int round, id;                       // the next item (id -1: none)
  Tile tile;                           // and its tile
  MARS_DEV Walk(const int32_t* count, const Tile* l, int heads_per_tile, int cta_, int ctas_)
      : list(l), heads(heads_per_tile), total(*count * heads_per_tile), cta(cta_), ctas(ctas_),
        round(0), id(-1) {
    fetch();
  }
  MARS_DEV void fetch() {
    id = round * ctas + ((round & 1) ? ctas - 1 - cta : cta);
    if (id >= total) id = -1;
    if (id >= 0) tile = list[id / heads];
  }
  // The next item's tile and its number among the tile's items.
  MARS_DEV bool take(Tile& t, int& head) {
    if (id < 0) return false;
    t = tile;
    head = id % heads;
    ++round;
    fetch();
    return true;
  }
};

// Transpose chunks of 16 bytes within groups of N lanes: before, lane i of the group holds the
// N chunks of row i in w; after, w[4k ..] is chunk i of row k.
template <int N>
MARS_DEV void transpose_chunks(uint32_t (&w)[4 * N], int lane) {
#pragma unroll
  for (int s = N / 2; s > 0; s >>= 1) {
    const bool up = (lane & s) != 0;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (i & s) continue;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        uint32_t &lo = w[4 * i + e], &hi = w[4 * (i | s) + e];
        const uint32_t got = __shfl_xor_sync(0xffffffffu, up ? lo : hi, s);
        lo = up ? got : lo;
        hi = up ? hi : got;
      }
    }
  }
}

// Store COLS values per lane, get(0) .. get(COLS - 1), as bf16 to out + at (at < 0: nowhere).
// Whole warp. Lanes exchange chunks first, so that a store instruction writes runs of 2 COLS
// bytes: with a row per lane it touched 32 lines for 512 bytes, and the output of a 128 x 128
// tile by eight warps took about 2,500 cycles.
template <int COLS, class F>
MARS_DEV void store_rows(uint16_t* out, long long at, int lane, F get) {
  constexpr int N = COLS / 8;                      // chunks per row
  uint32_t w[COLS / 2];
#pragma unroll
  for (int e = 0; e < COLS / 2; ++e) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(get(2 * e), get(2 * e + 1));
    w[e] = *reinterpret_cast<const uint32_t*>(&v);
  }
  transpose_chunks<N>(w, lane);
#pragma unroll
  for (int k = 0; k < N; ++k) {
    const long long to = __shfl_sync(0xffffffffu, at, (lane & (32 - N)) + k);
    if (to >= 0)
      *reinterpret_cast<uint4*>(out + to + (lane & (N - 1)) * 8) =
          make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
  }
}

inline size_t align256(size_t x) { return (x + 255) / 256 * 256; }

// Carve a plan out of a workspace at `off` (base may be null to size it).
inline Plan carve_plan(void* base, size_t& off, int batch, int total, int ntickets) {
  uint8_t* p = static_cast<uint8_t*>(base);
  auto take = [&](size_t bytes) {
    uint8_t* at = p ? p + off : nullptr;
    off += align256(bytes);
    return at;
  };
  const size_t tiles = (size_t)max_tiles(batch, total, kTileRows);
  Plan r{};
  r.count = reinterpret_cast<int32_t*>(take(sizeof(int32_t)));
  r.by_cost = reinterpret_cast<Tile*>(take(tiles * sizeof(Tile)));
  r.in_order = reinterpret_cast<Tile*>(take(tiles * sizeof(Tile)));
  r.before = reinterpret_cast<long long*>(take((tiles + 1) * sizeof(long long)));
  r.tickets = reinterpret_cast<int32_t*>(take(ntickets * sizeof(int32_t)));
  return r;
}

}  // namespace packed
}  // namespace mars
