// Parts the attention kernels over the 4-bit cache share: which rows and pages a
// CTA takes, the nodes' root paths, and the join of partial results.
#pragma once
#include <cmath>

#include "gdn_kv4.cuh"

namespace gdn {

// ---- A schedule without waves.  The pages of all work items, one after another, are one sequence of units; CTA c
// of N takes units [c T / N, (c + 1) T / N), whatever items they belong to, so that ragged lengths cost no idle
// SMs and a CTA starts once.  An item is (request, layer, kv head, row tile), its units its request's pages (one,
// where there are none: its own rows are still owed).  An item that several CTAs share is joined by the last of
// them to finish; a CTA shares at most its first and its last item, so two partial results per CTA are enough.
struct KvRequest {
  bool ok;                     // lengths and schedule in range
  int n, len, pages, units, tiles;
  int weight;                  // items of the request: layers * Hkv * tiles
};
__device__ __forceinline__ KvRequest kv_request(const KvAttnParams& p, int b, int tile_rows) {
  KvRequest r;
  r.n = p.words ? p.words[static_cast<size_t>(b) * SchedLayout{p.n_max}.words()] : 1;
  r.len = p.c.seq_len[b];
  r.ok = r.n >= 1 && r.n <= p.n_max && r.len >= 0 && r.len <= static_cast<long long>(p.c.pages_max) * kPage;
  r.pages = r.ok ? (r.len + kPage - 1) / kPage : 0;
  r.units = r.pages > 0 ? r.pages : 1;
  r.tiles = r.ok ? (r.n * p.G + tile_rows - 1) / tile_rows : 1;
  r.weight = p.layers * p.Hkv * r.tiles;
  return r;
}
// Quotients of unit counts: 32-bit where they fit, since a 64-bit division costs about a hundred instructions.
__device__ __forceinline__ long long kv_div(long long a, long long b) {
  if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
  return a / b;
}
__device__ __forceinline__ long long kv_unit_of(long long cta, long long total, int n) { return kv_div(cta * total, n); }
__device__ __forceinline__ int kv_cta_of(long long x, long long total, int n) {
  return static_cast<int>(kv_div((x + 1) * n - 1, total));
}
// The launch's units, the CTAs that take them (few units go to few CTAs), this CTA's units [at, end), the request
// that `at` falls into and the units before that.  All threads of the CTA call it; `sh` holds 35 values.
struct KvPlace {
  long long total, before, at, end;
  int b, ctas;
};
__device__ __forceinline__ KvPlace kv_place(const KvAttnParams& p, int tile_rows, long long* sh) {
  KvPlace r;
  auto share = [&](long long total) {
    r.total = total;
    r.ctas = static_cast<int>(min(static_cast<long long>(p.ctas), kv_div(total + p.least - 1, p.least)));
    const int cta = min(static_cast<int>(blockIdx.x), r.ctas);      // the others have no units
    r.at = kv_unit_of(cta, total, r.ctas);
    r.end = cta < r.ctas ? kv_unit_of(cta + 1, total, r.ctas) : r.at;
  };
  if (p.bn == 1) {
    // one request's items are alike: the same number of CTAs for each, so that none starts twice
    const KvRequest q = kv_request(p, p.b0, tile_rows);
    r.total = static_cast<long long>(q.weight) * q.units;
    r.before = 0;
    r.b = p.b0;
    if (q.weight <= p.ctas) {
      const int each = max(1, min(p.each, (q.units + p.least - 1) / p.least));
      r.ctas = q.weight * each;
      const int cta = min(static_cast<int>(blockIdx.x), r.ctas), item = cta / each, k = cta - item * each;
      r.at = static_cast<long long>(item) * q.units + kv_div(static_cast<long long>(k) * q.units, each);
      r.end = cta < r.ctas ? static_cast<long long>(item) * q.units + kv_div(static_cast<long long>(k + 1) * q.units, each)
                           : r.at;
    } else {
      share(r.total);
    }
    return r;
  }
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  long long w = 0, sum = 0, off = 0, carry = 0;
  // pass 0 sums; pass 1 finds the request.  Requests of the last block of pass 0 stay in registers for a single block
  for (int pass = 0; pass < 2; ++pass) {
    if (pass == 1 && p.bn > static_cast<int>(blockDim.x)) carry = 0;
    for (int base = 0; base < p.bn; base += blockDim.x) {
      const int i = base + threadIdx.x;
      if (pass == 0 || p.bn > static_cast<int>(blockDim.x)) {
        w = 0;
        if (i < p.bn) {
          const KvRequest q = kv_request(p, p.b0 + i, tile_rows);
          w = static_cast<long long>(q.weight) * q.units;
        }
        sum = w;
        for (int o = 1; o < 32; o <<= 1) {
          const long long y = __shfl_up_sync(0xffffffffu, sum, o);
          if (lane >= o) sum += y;
        }
        if (lane == 31) sh[warp] = sum;
        __syncthreads();
        off = carry;
        for (int k = 0; k < warps; ++k) {
          if (k < warp) off += sh[k];
          carry += sh[k];
        }
      }
      if (pass == 1) {
        const long long end = off + sum;
        if (w > 0 && r.at >= end - w && r.at < end) {
          sh[33] = end - w;
          sh[34] = p.b0 + i;
        }
      }
      __syncthreads();
    }
    if (pass == 0) share(carry);
  }
  r.before = r.at < r.end ? sh[33] : 0;
  r.b = r.at < r.end ? static_cast<int>(sh[34]) : p.b0;
  __syncthreads();
  return r;
}
// A CTA's run of pages inside one item.
struct KvSegment {
  KvRequest r;
  int b, l, h, bl, tile;
  int item;                    // counter of the item
  int page_lo, pages;          // pages taken here
  bool first, whole;           // the item's first pages; all of them
  long long start;             // the item's first unit
};
__device__ __forceinline__ KvSegment kv_segment(const KvAttnParams& p, int tile_rows, long long x, long long end,
                                                KvPlace& at, long long* next) {
  KvSegment s;
  s.r = kv_request(p, at.b, tile_rows);
  while (x >= at.before + static_cast<long long>(s.r.weight) * s.r.units) {
    at.before += static_cast<long long>(s.r.weight) * s.r.units;
    s.r = kv_request(p, ++at.b, tile_rows);
  }
  const long long off = x - at.before;
  const int idx = static_cast<int>(kv_div(off, s.r.units));
  const int lo = static_cast<int>(off - static_cast<long long>(idx) * s.r.units);
  const int take = static_cast<int>(min(static_cast<long long>(s.r.units - lo), end - x));
  s.b = at.b;
  s.tile = idx % s.r.tiles;
  const int lh = idx / s.r.tiles;
  s.h = lh % p.Hkv;
  s.l = lh / p.Hkv;
  s.bl = s.b * p.layers + s.l;
  s.item = (((s.b - p.b0) * p.layers + s.l) * p.Hkv + s.h) * p.row_tiles + s.tile;
  s.page_lo = lo;
  s.pages = max(0, min(s.r.pages, lo + take) - lo);
  s.first = lo == 0;
  s.whole = lo == 0 && take == s.r.units;
  s.start = x - lo;
  *next = x + take;
  return s;
}
// Partial result of an item in a CTA -- the first one that the CTA holds, or its last, which starts inside it: the
// rows' outputs [tile_rows][D], then their maxima and sums [tile_rows][2].
__device__ __forceinline__ float* kv_stream_part(const KvAttnParams& p, int c, bool starts_inside, int tile_rows, int D) {
  return p.part + (2 * static_cast<size_t>(c) + (starts_inside ? 1 : 0)) * tile_rows * (D + 2);
}

// The request's parents, and the nodes on the root path of node i (itself included) as a bit mask; false if the
// parents are no tree (the mask then ends at the fault).
__device__ __forceinline__ const int32_t* kv_parents(const KvAttnParams& p, int b) {
  const SchedLayout lay{p.n_max};
  return p.words + static_cast<size_t>(b) * lay.words() + lay.parent();
}
__device__ __forceinline__ bool kv_root_path(const int32_t* parent, int i, unsigned long long* mask) {
  unsigned long long m = 1ull << i;
  int a = parent ? parent[i] : -1, prev = i;
  while (a >= 0 && a < prev) {
    m |= 1ull << a;
    prev = a;
    a = parent[a];
  }
  *mask = m;
  return a < 0;
}

// True in the CTA that finishes an item last of `count`, with every partial result visible.
__device__ __forceinline__ bool kv_last(const KvAttnParams& p, size_t item, int count, int* flag) {
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) {
    const int prev = atomicAdd(&p.done[item], 1);
    *flag = prev == count - 1;
    if (prev == count - 1) p.done[item] = 0;
  }
  __syncthreads();
  __threadfence();
  return *flag != 0;
}
__device__ __forceinline__ void kv_store(float* p, float x) { *p = x; }
__device__ __forceinline__ void kv_store(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

// The join of all rows of a tile by the whole CTA, in order: out = sum_c 2^{m_c - m} O_c / sum_c 2^{m_c - m} l_c (maxima
// are kept in base 2), from partial results with the layout of kv_stream_part.  Reads of what other SMs just wrote take
// a microsecond and more, so the loads of a step are all in flight together: a row's maxima and sums by one warp, then
// four channels of a row per thread, kAhead parts at a time.  `sh` holds
// (count + 1) * rows floats; row r of the item is query head r % G of node r / G, counted from out0.
struct KvJoin {
  int c0, count, rows, inside;     // first CTA, CTAs, rows; the item starts inside its first CTA
  int b, l, h, row0;
};
template <typename T, int D>
__device__ __forceinline__ void kv_join_rows(const float* part, const KvJoin& t, int tile_rows, T* out0, int G,
                                             long long out_node, float* sh) {
  const int c0 = t.c0, count = t.count, rows = t.rows;
  const bool inside = t.inside != 0;
  constexpr int kAhead = 16;
  const size_t size = static_cast<size_t>(tile_rows) * (D + 2);
  auto part_of = [&](int c) { return part + (2 * static_cast<size_t>(c0 + c) + (c == 0 && inside ? 1 : 0)) * size; };
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  for (int r = warp; r < rows; r += warps) {
    float m = -INFINITY, sum = 0.f;
    for (int b = 0; b < count; b += 32) {
      const int c = b + lane;
      const float2 ml = c < count ? __ldcg(reinterpret_cast<const float2*>(part_of(c) + tile_rows * D + 2 * r))
                                  : make_float2(-INFINITY, 0.f);
      if (c < count) sh[c * rows + r] = ml.x;
      float top = fmaxf(m, ml.x);
      for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      // a part that held nothing this row sees has maximum -inf, sum 0 and zeros
      const float w = (ml.x == -INFINITY && ml.y == 0.f) ? 0.f : exp2f(ml.x - top) * ml.y;
      sum = (m == -INFINITY ? 0.f : sum * exp2f(m - top)) + w;
      m = top;
    }
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    __syncwarp();
    for (int c = lane; c < count; c += 32) {
      const float mc = sh[c * rows + r];
      sh[c * rows + r] = mc == -INFINITY ? 0.f : exp2f(mc - m) * inv;
    }
    if (lane == 0) sh[count * rows + r] = sum == sum ? 0.f : sum;       // a NaN reaches every channel
  }
  __syncthreads();
  for (int i = threadIdx.x; i < rows * (D / 4); i += blockDim.x) {
    const int r = i / (D / 4), d = 4 * (i % (D / 4));
    const float bad = sh[count * rows + r];
    float4 acc = make_float4(bad, bad, bad, bad);
    const float* at = part_of(0) + r * D + d;
    const float* from1 = part + 2 * static_cast<size_t>(c0) * size + r * D + d;       // part c > 0: + 2 c size
#pragma unroll 1
    for (int b = 0; b < count; b += kAhead) {
      float4 v[kAhead];
#pragma unroll
      for (int k = 0; k < kAhead; ++k)
        if (b + k < count) {
          v[k] = __ldcg(reinterpret_cast<const float4*>(at));
          at = from1 + 2 * static_cast<size_t>(b + k + 1) * size;
        }
#pragma unroll
      for (int k = 0; k < kAhead; ++k)
        if (b + k < count) {
          const float w = sh[(b + k) * rows + r];
          acc.x = fmaf(w, v[k].x, acc.x);
          acc.y = fmaf(w, v[k].y, acc.y);
          acc.z = fmaf(w, v[k].z, acc.z);
          acc.w = fmaf(w, v[k].w, acc.w);
        }
    }
    const int x = t.row0 + r;
    T* out = out0 + (x / G) * out_node + (x % G) * D + d;
    kv_store(out, acc.x);
    kv_store(out + 1, acc.y);
    kv_store(out + 2, acc.z);
    kv_store(out + 3, acc.w);
  }
}

}  // namespace gdn
