// Parts the attention kernels over the 4-bit cache share: which rows and pages a
// CTA takes, the nodes' ancestor masks, and the join of the chunks' results.
#pragma once
#include <cmath>

#include "gdn_kv4.cuh"

namespace gdn {

struct KvItem {
  int b, l, h, bl, tile;
};
__device__ __forceinline__ KvItem kv_item(const KvAttnParams& p, unsigned x) {
  KvItem it;
  it.tile = x % p.row_tiles;
  x /= p.row_tiles;
  it.h = x % p.Hkv;
  it.bl = x / p.Hkv;
  it.b = it.bl / p.layers;
  it.l = it.bl % p.layers;
  return it;
}

// The request's nodes and length, and the pages of one chunk.  Every chunk has the planned number of pages;
// a request longer than the host expected gets longer chunks instead of more.
struct KvSpan {
  bool ok;
  int bit;                     // error bit where not ok
  int n, len, chunks, page_lo, page_hi;
};
__device__ __forceinline__ KvSpan kv_span(const KvAttnParams& p, const KvItem& it, int chunk) {
  KvSpan s{};
  s.n = p.words ? p.words[static_cast<size_t>(it.b) * SchedLayout{p.n_max}.words()] : 1;
  s.len = p.c.seq_len[it.b];
  s.bit = (s.n < 1 || s.n > p.n_max) ? GDN_DEVERR_SCHEDULE : GDN_DEVERR_CACHE;
  s.ok = s.n >= 1 && s.n <= p.n_max && s.len >= 0 && s.len <= static_cast<long long>(p.c.pages_max) * kPage;
  const int pages = (s.len + kPage - 1) / kPage;
  const int each = max(p.chunk_pages, (pages + p.chunks - 1) / p.chunks);
  s.chunks = max(1, (pages + each - 1) / each);
  s.page_lo = min(pages, chunk * each);
  s.page_hi = min(pages, s.page_lo + each);
  return s;
}

// see[i], bit j: node j is i or an ancestor of i.  The CTA's threads call it; false if the parents are no tree.
__device__ __forceinline__ bool kv_ancestors(const KvAttnParams& p, int b, int n, unsigned long long* see) {
  bool ok = true;
  const int32_t* parent = p.words ? p.words + static_cast<size_t>(b) * SchedLayout{p.n_max}.words() + SchedLayout{p.n_max}.parent()
                                  : nullptr;
  for (int i = threadIdx.x; i < n; i += blockDim.x) {
    unsigned long long m = 1ull << i;
    int a = parent ? parent[i] : -1, prev = i;
    while (a >= 0 && a < prev) {
      m |= 1ull << a;
      prev = a;
      a = parent[a];
    }
    ok = ok && a < 0;
    see[i] = m;
  }
  return __syncthreads_and(ok);
}

// Partial result of a row tile over one chunk: rows of D outputs, maximum, sum.
__device__ __forceinline__ float* kv_part(const KvAttnParams& p, size_t tile, int chunk, int tile_rows, int D) {
  return p.part + (tile * p.chunks + chunk) * static_cast<size_t>(tile_rows) * (D + 2);
}
// True in the CTA that finishes the tile's chunks last, with every chunk's partial result visible.
__device__ __forceinline__ bool kv_last_chunk(const KvAttnParams& p, size_t tile, int chunks, int* flag) {
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) {
    const int prev = atomicAdd(&p.done[tile], 1);
    *flag = prev == chunks - 1;
    if (prev == chunks - 1) p.done[tile] = 0;
  }
  __syncthreads();
  __threadfence();
  return *flag != 0;
}
__device__ __forceinline__ void kv_store(float* p, float x) { *p = x; }
__device__ __forceinline__ void kv_store(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

// One warp joins a row's chunks, in chunk order: out = sum_c 2^{m_c - m} O_c / sum_c 2^{m_c - m} l_c (maxima are
// kept in base 2).
template <typename T, int D>
__device__ __forceinline__ void kv_join_row(const KvAttnParams& p, size_t tile, int chunks, int tile_rows, int r, T* out) {
  const int lane = threadIdx.x & 31;
  float m = -INFINITY;
  for (int c = lane; c < chunks; c += 32) m = fmaxf(m, __ldcg(kv_part(p, tile, c, tile_rows, D) + r * (D + 2) + D));
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  float acc[D / 32], sum = 0.f;
#pragma unroll
  for (int i = 0; i < D / 32; ++i) acc[i] = 0.f;
  for (int c = 0; c < chunks; ++c) {
    const float* part = kv_part(p, tile, c, tile_rows, D) + r * (D + 2);
    const float2 ml = __ldcg(reinterpret_cast<const float2*>(part + D));
    if (ml.x == -INFINITY && ml.y == 0.f) continue;         // the chunk held nothing this row sees
    const float w = exp2f(ml.x - m);
    sum = fmaf(w, ml.y, sum);
#pragma unroll
    for (int i = 0; i < D / 64; ++i) {
      const float2 v = __ldcg(reinterpret_cast<const float2*>(part + 64 * i + 2 * lane));
      acc[2 * i] = fmaf(w, v.x, acc[2 * i]);
      acc[2 * i + 1] = fmaf(w, v.y, acc[2 * i + 1]);
    }
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
  for (int i = 0; i < D / 64; ++i) {
    kv_store(out + 64 * i + 2 * lane, acc[2 * i] * inv);
    kv_store(out + 64 * i + 2 * lane + 1, acc[2 * i + 1] * inv);
  }
}

}  // namespace gdn
