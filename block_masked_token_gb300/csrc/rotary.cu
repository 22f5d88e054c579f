// Rotary positions of the queries and keys of packed sequences: pair j of a head, (a, b), of a
// row at position p becomes factor * (a cos t - b sin t, a sin t + b cos t) with t = p f_j. The
// map is orthogonal up to its factor, so its gradient is the same with -t (`inverse`).
//
// A pass over memory: 4 (hq + hkv) d bytes per row, read and written once. A CTA takes kRows rows
// of one sequence; the sines and cosines of its rows, the same for every head, are formed once
// into shared memory. t reaches far beyond what 32 bits resolve (position 131,072 at f = 1 is off
// by 0.008 in fp32), so f / 2 pi is kept as a 64-bit fraction of a turn, off by 2^-52 of f / 2 pi at most:
// its product with the position is modulo 1 by itself. sincospi gets the upper 32 bits as a float
// of half turns in [-1, 1), which keeps 24 of them: pi 2^-25 off at most, to which a position adds itself times
// f 2^-52 radians.
//
// Prompts of 10,586 rows of 28 + 4 heads of 128 (173 MB moved): 31.1 us, 0.82 of the copy bandwidth; the
// gradient over 8,191 long rows 24.7 us, 0.80. With 8 rows per CTA 31.2 and 27.6 (fewer CTAs to even out
// at the end), with 16 32.7 and 26.9, with 4 and 128 threads 30.5 and 26.0.
#include "common.cuh"
#include "internal.h"
#include "packed.cuh"
#include "sm100.cuh"

namespace mars {

namespace {

constexpr int kRows = 4;
constexpr int kThreads = 256;
constexpr int kUnit = 16;            // elements that a thread takes at a time: eight pairs
constexpr int kMaxPairs = 64;        // pairs of a head

// Fraction of a turn, in 2^-64, that frequency f (radians per position) advances by.
MARS_DEV uint64_t turn_of(float f) {
  double t = (double)f * 0.15915494309189533577;
  t -= floor(t);
  return t < 1.0 ? (uint64_t)(t * 18446744073709551616.0) : 0;     // NaN too: see poison
}

template <bool kInterleaved>
__global__ void __launch_bounds__(kThreads) rotary_kernel(Rotary a) {
  // cosines and sines of pairs 8u .. 8u + 7 as four 16-byte vectors (cos, sin, cos, sin), vector v
  // of unit u at v * units + u: the lanes of a head then read consecutive vectors
  __shared__ float4 turns[kRows][kMaxPairs / 2];
  bool bad;
  sm100::let_next_start();
  sm100::wait_for_previous();
  const packed::Seq sq = packed::find_tile(a.cu, a.batch, a.total, kRows, 0, (long long)blockIdx.x,
                                           bad, a.seq_lens);
  if (bad && threadIdx.x == 0 && a.status) atomicOr(a.status, MARS_ST_BADSEQ);
  if (sq.s < 0) return;
  if (sq.len < 0 && threadIdx.x == 0 && a.status) atomicOr(a.status, MARS_ST_OVERFLOW);
  const int r0 = sq.tile * kRows, nr = min(kRows, sq.n - r0);

  // thread = unit u of an item (row, head); in place, what is not rotated stays where it is
  const int rot_units = a.rot / kUnit, units = a.in_place ? rot_units : a.d / kUnit;
  const int slots = kThreads / units, slot = threadIdx.x / units, u = threadIdx.x - slot * units;
  const int heads = a.hq + a.hkv;
  const bool turned = u < rot_units;
  const int lo = (kInterleaved || !turned) ? u * kUnit : u * 8;
  const int hi = (kInterleaved || !turned) ? lo + 8 : lo + a.rot / 2;
  struct Item {
    int row, head;
  };
  auto advance = [&](Item& it, int by) {
    it.head += by;
    while (it.head >= heads) {
      it.head -= heads;
      ++it.row;
    }
  };
  auto live = [&](const Item& it) { return slot < slots && it.row < nr; };
  auto load = [&](const Item& it, uint4& x, uint4& y) {
    const size_t row = (size_t)sq.base + r0 + it.row;
    const uint16_t* p = it.head < a.hq ? a.q + row * a.q_stride + it.head * a.d
                                       : a.k + row * a.k_stride + (it.head - a.hq) * a.d;
    x = *reinterpret_cast<const uint4*>(p + lo);
    y = *reinterpret_cast<const uint4*>(p + hi);
  };
  Item it{0, 0};
  advance(it, slot);
  uint4 x = {}, y = {};
  if (live(it)) load(it, x, y);                  // on its way while the angles are formed

  {
    const int pairs = a.rot / 2, j = threadIdx.x % pairs;
    const float f = a.inv_freq[j];
    const uint64_t turn = turn_of(f);
    // a frequency that is no number gives outputs that are none
    const float factor = isfinite(f) ? a.factor : __int_as_float(0x7fc00000);
    const long long first = (long long)max(sq.len, 0) + r0;
    for (int r = threadIdx.x / pairs; r < nr; r += kThreads / pairs) {
      if (threadIdx.x >= (kThreads / pairs) * pairs) break;
      const uint64_t t = (uint64_t)(first + r) * turn;
      float s, c;
      sincospif((float)(int32_t)(t >> 32) * 4.656612873077393e-10f, &s, &c);     // 2^-31
      float* at = reinterpret_cast<float*>(&turns[r][((j & 7) >> 1) * rot_units + (j >> 3)]);
      at[(j & 1) * 2] = c * factor;
      at[(j & 1) * 2 + 1] = (a.inverse ? -s : s) * factor;
    }
  }
  __syncthreads();

  while (live(it)) {
    const Item now = it;
    const uint4 vx = x, vy = y;
    advance(it, slots);
    if (live(it)) load(it, x, y);
    uint4 ox = vx, oy = vy;
    if (turned) {
      float e[16];
      unpack8(vx, e);
      unpack8(vy, e + 8);
      uint32_t w[8];
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const float4 t = turns[now.row][v * rot_units + u];
        float p[4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int j = 2 * v + h;
          const float c = h ? t.z : t.x, s = h ? t.w : t.y;
          const float e0 = kInterleaved ? e[2 * j] : e[j], e1 = kInterleaved ? e[2 * j + 1] : e[8 + j];
          p[2 * h] = e0 * c - e1 * s;
          p[2 * h + 1] = e0 * s + e1 * c;
        }
        const __nv_bfloat162 w0 = kInterleaved ? __floats2bfloat162_rn(p[0], p[1])
                                               : __floats2bfloat162_rn(p[0], p[2]);
        const __nv_bfloat162 w1 = kInterleaved ? __floats2bfloat162_rn(p[2], p[3])
                                               : __floats2bfloat162_rn(p[1], p[3]);
        w[kInterleaved ? 2 * v : v] = *reinterpret_cast<const uint32_t*>(&w0);
        w[kInterleaved ? 2 * v + 1 : 4 + v] = *reinterpret_cast<const uint32_t*>(&w1);
      }
      ox = make_uint4(w[0], w[1], w[2], w[3]);
      oy = make_uint4(w[4], w[5], w[6], w[7]);
    }
    const size_t row = (size_t)sq.base + r0 + now.row;
    uint16_t* p = now.head < a.hq ? a.q_out + row * a.qo_stride + now.head * a.d
                                  : a.k_out + row * a.ko_stride + (now.head - a.hq) * a.d;
    *reinterpret_cast<uint4*>(p + lo) = ox;
    *reinterpret_cast<uint4*>(p + hi) = oy;
  }
}

}  // namespace

long long rotary_ctas(int batch, int total) { return packed::max_tiles(batch, total, kRows); }

cudaError_t launch_rotary(const Rotary& a, bool interleaved, cudaStream_t stream) {
  const unsigned ctas = (unsigned)rotary_ctas(a.batch, a.total);
  count_launches(1);
  return launch_early(interleaved ? rotary_kernel<true> : rotary_kernel<false>, ctas, kThreads, 0, stream, a);
}

}  // namespace mars
