// Attention of new tokens over the 8-bit paged cache (cache_q8.cuh): the pages that the sequences
// read are written out in bf16, which holds every code times its scale exactly, and attended to by
// packed_attn.cu.
#include <algorithm>

#include "cache_q8.cuh"
#include "internal.h"
#include "packed.cuh"

namespace mars {

namespace {

constexpr int kThreads = 256;

struct UnpackArgs {
  const int32_t *cu, *seq_lens, *block_table;
  const uint8_t *k_pool, *v_pool, *k_scale, *v_scale;
  uint16_t *k_out, *v_out;
  int32_t *lens, *table, *status;
  int num_pages, max_pages, pages, batch, total, hkv;
};

// A CTA writes one page of a sequence out: page j of sequence s becomes page s * pages + j.
template <int D>
__global__ void __launch_bounds__(kThreads) unpack_kernel(UnpackArgs a) {
  const int s = blockIdx.x / a.pages, j = blockIdx.x % a.pages;
  const int len = a.seq_lens[s];
  const int P = (int)max(0LL, min((long long)len, (long long)a.max_pages * kPageSize));
  if (j == 0 && threadIdx.x == 0) {
    a.lens[s] = min(P, a.pages * kPageSize);
    if (a.status && P != len) atomicOr(a.status, MARS_ST_OVERFLOW);
  }
  if (j * kPageSize >= P) return;
  const int page = a.block_table[(size_t)s * a.max_pages + j];
  const bool mapped = page >= 0 && page < a.num_pages;
  if (threadIdx.x == 0) a.table[(size_t)s * a.pages + j] = mapped ? (int)blockIdx.x : -1;
  if (!mapped) return;
  constexpr int kVectors = kPageSize * D / 16;     // of 16 codes, per head
  for (int i = threadIdx.x; i < 2 * a.hkv * kVectors; i += kThreads) {
    const int w = i / kVectors, c = i - w * kVectors;
    const bool is_v = w >= a.hkv;
    const int h = is_v ? w - a.hkv : w;
    const size_t at = (size_t)page * a.hkv + h, to = (size_t)blockIdx.x * a.hkv + h;
    const uint4 x = reinterpret_cast<const uint4*>((is_v ? a.v_pool : a.k_pool) + at * (kPageSize * D))[c];
    const float f = q8::power(q8::scale_byte((is_v ? a.v_scale : a.k_scale)[at]));
    const uint32_t in[4] = {x.x, x.y, x.z, x.w};
    uint32_t out[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float2 v = q8::decode2_f32((in[e >> 1] >> (16 * (e & 1))) & 0xffffu);
      const __nv_bfloat162 b = __floats2bfloat162_rn(v.x * f, v.y * f);
      out[e] = *reinterpret_cast<const uint32_t*>(&b);
    }
    uint4* dst = reinterpret_cast<uint4*>((is_v ? a.v_out : a.k_out) + to * (kPageSize * D)) + 2 * c;
    dst[0] = make_uint4(out[0], out[1], out[2], out[3]);
    dst[1] = make_uint4(out[4], out[5], out[6], out[7]);
  }
}

// Parts of the workspace, in bytes from its start.
struct Layout {
  size_t lens, table, k, v, end;
};
Layout layout(const ChunkQ8Plan& plan, int batch, int hkv, int d) {
  Layout l;
  l.lens = packed::align256(plan.wide.ws_bytes);
  l.table = l.lens + packed::align256((size_t)batch * sizeof(int32_t));
  l.k = l.table + packed::align256((size_t)batch * plan.pages * sizeof(int32_t));
  l.v = l.k + (size_t)batch * plan.pages * hkv * kPageSize * d * 2;
  l.end = l.v + (l.v - l.k);
  return l;
}

}  // namespace

ChunkQ8Plan plan_chunk_q8(int batch, int total, int hq, int hkv, int d, int max_len) {
  ChunkQ8Plan p{};
  p.wide = plan_packed(batch, total, hq, hkv, d, max_len);
  p.pages = std::max(1, max_len / kPageSize + (max_len % kPageSize != 0));
  p.ws_bytes = layout(p, batch, hkv, d).end;
  return p;
}

cudaError_t launch_chunk_q8(const ChunkQ8& p, const ChunkQ8Plan& plan, void* workspace,
                            cudaStream_t stream) {
  const PackedAttn& t = p.attn;
  const Layout l = layout(plan, t.batch, t.hkv, t.d);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  UnpackArgs a{t.cu, t.seq_lens, t.block_table, p.k_pool, p.v_pool, p.k_scale, p.v_scale,
               reinterpret_cast<uint16_t*>(ws + l.k), reinterpret_cast<uint16_t*>(ws + l.v),
               reinterpret_cast<int32_t*>(ws + l.lens), reinterpret_cast<int32_t*>(ws + l.table),
               t.status, t.num_pages, t.max_pages, plan.pages, t.batch, t.total, t.hkv};
  const unsigned ctas = (unsigned)((long long)t.batch * plan.pages);
  if (t.d == 64)
    unpack_kernel<64><<<ctas, kThreads, 0, stream>>>(a);
  else
    unpack_kernel<128><<<ctas, kThreads, 0, stream>>>(a);
  count_launches(1);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  PackedAttn wide = t;
  wide.k_pool = a.k_out;
  wide.v_pool = a.v_out;
  wide.seq_lens = a.lens;
  wide.block_table = a.table;
  wide.num_pages = t.batch * plan.pages;
  wide.max_pages = plan.pages;
  return launch_packed_attn(wide, plan.wide, workspace, stream);
}

}  // namespace mars
