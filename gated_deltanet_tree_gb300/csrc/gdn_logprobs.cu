// Log-probabilities of rows of logits: of a given token, of the best ones, and the entropy.
//
// One pass over a row keeps, relative to the running maximum m, s = sum e^(z - m) and
// t = sum e^(z - m) (z - m); then log p_i = z_i - m - log s and the entropy is log s - t / s.
//
// The best `top` tokens (larger logit first, lower index on ties) come from the same pass.  A tile
// of 4096 entries lies in the CTA's registers; the top-th largest of 32 group maxima of the first
// one bounds its top-th largest entry from below, so a handful of entries pass and are put on a list
// in shared memory.  Its exact best are picked by counting, and the worst of them is the bound of
// later tiles; it is renewed after ever more of them, and the warps need no barrier in between.  Where
// more entries pass than the list holds the best are found tile by tile, one after another, in a second
// pass: long ties, rising rows, and rows whose first 4096 entries hold fewer than `top` groups with one
// that is not masked (the bound is -inf then, which masked entries pass).  That is some 4 times as slow
// at ten rows and 14 times at 320 (us, 131072 entries of bf16, 8 best): 300 entries not masked 48 and 476,
// equal entries 45 and 461, the first 4096 masked 62 and 652, against 11 and 33.
//
// A cluster of up to eight CTAs shares a row where rows are few; each puts its sums and its list into
// the first one's shared memory.
//
// The bytes, read once, are the floor.  Instruction issue is nearer, half its slots taken (by the counters
// 12 to 22 instructions an entry, tiles' and rows' starts and ends among them, for clocks of 1440 to
// 2070 MHz), and, where a row has few tiles, the latencies of its start and end.
// Measured (us): 10 rows of 131072 bf16 7.8, 320 of them 33 (floor 12), 1500 rows of 65537 fp32 with
// 20 best 92 (floor 58).  Two CTAs a row where there are 320 took 37; a warp's entries that pass, taken
// in unrolled code, cost the ten rows 1.4 us more, because code that runs once is fetched slowly.
// Four CTAs an SM for bf16 (64 registers), three for fp32: 92 against 106 us with spills.
#include <cooperative_groups.h>
#include <cuda_bf16.h>

#include "gdn_logprobs.cuh"

namespace cg = cooperative_groups;

namespace gdn {
namespace {

typedef unsigned long long u64;
constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kVals = 16;                    // entries of a tile in a thread's registers
constexpr int kCap = 1024;                   // candidates
constexpr int kMaxCluster = 8;
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float max_nan(float a, float b) {   // a NaN stays
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
// packed pairs of fp32
__device__ __forceinline__ u64 pack2(float lo, float hi) {
  u64 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 unpack2(u64 v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ u64 add2(u64 a, u64 b) {
  u64 d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ u64 mul2(u64 a, u64 b) {
  u64 d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ u64 fma2(u64 a, u64 b, u64 c) {
  u64 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}

template <typename T>
struct Vec;
template <>
struct Vec<float> {
  static constexpr int N = 4;
  static __device__ __forceinline__ void unpack(uint4 v, float* x) {
    x[0] = __uint_as_float(v.x), x[1] = __uint_as_float(v.y), x[2] = __uint_as_float(v.z), x[3] = __uint_as_float(v.w);
  }
  static __device__ __forceinline__ float one(const float* p) { return *p; }
  // the largest of the sixteen bytes' entries, a NaN if one is
  static __device__ __forceinline__ float most(uint4 v) {
    return max_nan(max_nan(__uint_as_float(v.x), __uint_as_float(v.y)), max_nan(__uint_as_float(v.z), __uint_as_float(v.w)));
  }
};
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int N = 8;
  static __device__ __forceinline__ void unpack(uint4 v, float* x) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
  static __device__ __forceinline__ float one(const __nv_bfloat16* p) { return __bfloat162float(*p); }
  static __device__ __forceinline__ float most(uint4 v) {        // (two entries an instruction)
    auto pair = [](uint32_t w) { return *reinterpret_cast<__nv_bfloat162*>(&w); };
    const __nv_bfloat162 m = __hmax2_nan(__hmax2_nan(pair(v.x), pair(v.y)), __hmax2_nan(pair(v.z), pair(v.w)));
    return max_nan(__low2float(m), __high2float(m));
  }
};

// A value's bits in an order that integers have; not 0 for a value that is not NaN.
__device__ __forceinline__ uint32_t ordered(float v) {
  const uint32_t u = __float_as_uint(v + 0.f);     // -0 counts as +0
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t o) {
  return __uint_as_float((o & 0x80000000u) ? (o & 0x7FFFFFFFu) : ~o);
}
// Order-preserving key of (value, lowest index wins).
__device__ __forceinline__ u64 key_of(float v, int idx) {
  return (static_cast<u64>(ordered(v)) << 32) | (0xFFFFFFFFu - static_cast<uint32_t>(idx));
}
__device__ __forceinline__ float key_value(u64 k) { return unordered(static_cast<uint32_t>(k >> 32)); }
__device__ __forceinline__ int key_index(u64 k) { return static_cast<int>(0xFFFFFFFFu - static_cast<uint32_t>(k)); }

__device__ __forceinline__ float exp2_fast(float x) {   // results below 2^-126 are zero
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

struct Sums {
  float m, s, t;
};
__device__ __forceinline__ float finite_ref(float m) { return m == -INFINITY ? 0.f : m; }
__device__ __forceinline__ Sums join(const Sums& a, const Sums& b) {
  Sums r;
  r.m = max_nan(a.m, b.m);
  const float ref = finite_ref(r.m);
  // a side that saw nothing has s = t = 0 and m = -inf: its difference only must not be infinite
  const float da = fmaxf(a.m - ref, -1e4f), db = fmaxf(b.m - ref, -1e4f);
  const float ea = exp2_fast(da * kLog2e), eb = exp2_fast(db * kLog2e);
  r.s = fmaf(a.s, ea, b.s * eb);
  r.t = fmaf(ea, fmaf(a.s, da, a.t), eb * fmaf(b.s, db, b.t));
  return r;
}

struct Shared {
  u64 cand[kCap];
  u64 sorted[kLogprobTop];
  u64 best[kWarps];
  float groups[32];
  Sums sums[kWarps];
  int count;
};

// The best min(n, top) of the first n candidates, in order, at the front of the list; n is uniform.  Returns how many.
__device__ __forceinline__ int pick(Shared& sh, int n, int top) {
  const int tid = threadIdx.x;
  for (int i = tid; i < n; i += kThreads) {
    const u64 k = sh.cand[i];
    int r = 0;
#pragma unroll 4
    for (int j = 0; j < n; ++j) r += sh.cand[j] > k;
    if (r < top) sh.sorted[r] = k;
  }
  __syncthreads();
  n = min(n, top);
  if (tid < n) sh.cand[tid] = sh.sorted[tid];
  if (tid == 0) sh.count = n;
  __syncthreads();
  return n;
}

// A tile of a row in a thread's registers: entry i is index_of(at, i) of the row; entries outside [0, V) and the CTA's blocks
// are -inf.
template <typename T>
struct Tile {
  static constexpr int N = Vec<T>::N, kLoads = kVals / N;
  const T* z;
  int skew, V, hi;
  __device__ __forceinline__ int index_of(int at, int i) const {
    return (at + i / N * kThreads + static_cast<int>(threadIdx.x)) * N - skew + i % N;
  }
  __device__ __forceinline__ bool has(int at, int i) const {
    const int blk = at + i / N * kThreads + static_cast<int>(threadIdx.x), e = index_of(at, i);
    return blk < hi && e >= 0 && e < V;
  }
  __device__ __forceinline__ bool whole(int at) const {        // no entry of the tile is outside
    const int last = at + kThreads * kLoads;
    return at * N - skew >= 0 && last <= hi && last * N - skew <= V;
  }
  __device__ __forceinline__ void fetch(int at, uint4 (&raw)[kLoads]) const {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) raw[i] = __ldcs(reinterpret_cast<const uint4*>(z - skew) + at + i * kThreads + threadIdx.x);
  }
  static __device__ __forceinline__ void unpack(const uint4 (&raw)[kLoads], float (&v)[kVals]) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) Vec<T>::unpack(raw[i], v + i * N);
  }
  __device__ __forceinline__ void load(int at, float (&v)[kVals]) const {
    if (whole(at)) {
      uint4 raw[kLoads];
      fetch(at, raw);
      unpack(raw, v);
      return;
    }
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int blk = at + i * kThreads + threadIdx.x, e = blk * N - skew;
      if (blk < hi && e >= 0 && e + N <= V) {
        Vec<T>::unpack(__ldcs(reinterpret_cast<const uint4*>(z - skew) + blk), v + i * N);
      } else {
#pragma unroll
        for (int j = 0; j < N; ++j) v[i * N + j] = blk < hi && e + j >= 0 && e + j < V ? Vec<T>::one(z + e + j) : -INFINITY;
      }
    }
  }
};

// The exact best `top` of a CTA's blocks, tile by tile, for rows whose entries pass the bound in too large a number.
template <typename T>
__device__ __noinline__ int best_slowly(Shared& sh, const Tile<T>& tile, int lo, int top) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int n = 0;
  for (int at = lo; at < tile.hi; at += kThreads * Tile<T>::kLoads) {
    float v[kVals];
    tile.load(at, v);
    u64 last = ~0ull;
    for (int r = 0; r < top; ++r) {
      u64 best = 0;
#pragma unroll
      for (int i = 0; i < kVals; ++i) {
        const u64 k = key_of(v[i], tile.index_of(at, i));
        if (v[i] == v[i] && k < last && k > best && tile.has(at, i)) best = k;
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        const u64 k = __shfl_xor_sync(~0u, best, o);
        best = k > best ? k : best;
      }
      __syncthreads();
      if (lane == 0) sh.best[warp] = best;
      __syncthreads();
      best = 0;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) best = sh.best[w] > best ? sh.best[w] : best;
      if (best == 0) break;
      last = best;
      if (tid == 0) sh.cand[n] = best;
      ++n;
    }
    __syncthreads();
    n = pick(sh, n, top);
  }
  return n;
}

template <typename T>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 4 ? 3 : 4) logprob_kernel(const LogprobParams p) {
  constexpr int N = Vec<T>::N, kLoads = kVals / N;
  __shared__ Shared sh;
  __shared__ u64 lists[kMaxCluster * kLogprobTop];
  __shared__ Sums parts[kMaxCluster];
  cg::cluster_group cluster = cg::this_cluster();
  const int CL = cluster.num_blocks(), rank = cluster.block_rank();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int row = blockIdx.x / CL, top = p.top;
  // here, so that the others know that this CTA runs: they write into the first one's memory
  if (CL > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;");
  const T* z = static_cast<const T*>(p.logits) + row * p.v_stride;
  // blocks of sixteen aligned bytes; the row begins `skew` entries into block 0
  const int skew = static_cast<int>((reinterpret_cast<uintptr_t>(z) & 15u) / sizeof(T));
  const int blocks = (p.V + skew + N - 1) / N;
  const int per = ((blocks + CL - 1) / CL + 31) / 32 * 32;
  const int lo = min(rank * per, blocks);
  const Tile<T> tile{z, skew, p.V, min(lo + per, blocks)};
  if (tid == 0) sh.count = 0;

  Sums a{-INFINITY, 0.f, 0.f};
  float bound = -INFINITY;
  bool strict = false, fetched = false;
  uint4 raw[kLoads];                                   // of the next tile
  int number = 0, pick_at = 0;
  for (int at = lo; at < tile.hi; at += kThreads * kLoads, ++number) {
    float v[kVals], most;
    if (fetched) {
      most = Vec<T>::most(raw[0]);
#pragma unroll
      for (int i = 1; i < kLoads; ++i) most = max_nan(most, Vec<T>::most(raw[i]));
      Tile<T>::unpack(raw, v);
    } else {
      tile.load(at, v);
      most = v[0];
#pragma unroll
      for (int i = 1; i < kVals; ++i) most = max_nan(most, v[i]);
    }
    const int next = at + kThreads * kLoads;
    fetched = next < tile.hi && tile.whole(next);
    if (fetched) tile.fetch(next, raw);
    // the sums; a masked entry's difference must not be infinite (its exponential is 0), and a NaN is in the maximum
    if (!(most <= a.m)) a = join(a, Sums{most, 0.f, 0.f});
    const float ref = finite_ref(a.m);
    u64 s2 = 0ull, t2 = 0ull;
#pragma unroll
    for (int i = 0; i < kVals; i += 2) {
      const float2 f = unpack2(add2(pack2(v[i], v[i + 1]), pack2(-ref, -ref)));
      const u64 d = pack2(fmaxf(f.x, -1e4f), fmaxf(f.y, -1e4f));
      const float2 x = unpack2(mul2(d, pack2(kLog2e, kLog2e)));
      const u64 e = pack2(exp2_fast(x.x), exp2_fast(x.y));
      s2 = add2(s2, e);
      t2 = fma2(e, d, t2);
    }
    const float2 s = unpack2(s2), ts = unpack2(t2);
    a.s += s.x + s.y;
    a.t += ts.x + ts.y;
    // candidates
    if (number == 0) {
      float g = most;
#pragma unroll
      for (int o = 1; o < kWarps; o <<= 1) g = fmaxf(g, __shfl_xor_sync(~0u, g, o));
      if (tid % kWarps == 0) sh.groups[tid / kWarps] = g;     // (as many threads a group as there are warps)
      __syncthreads();
      // the top-th largest of the 32: one after another is taken out
      uint32_t left = ordered(sh.groups[lane]), m = 0;
      for (int r = 0; r < top; ++r) {
        m = __reduce_max_sync(~0u, left);
        if (lane == __ffs(__ballot_sync(~0u, left == m)) - 1) left = 0;
      }
      bound = unordered(m);
    }
    if (strict ? most > bound : most >= bound) {
      // which entries pass; then one after another, in little code (what runs seldom is fetched slowly)
      uint32_t in = 0;
#pragma unroll
      for (int i = 0; i < kVals; ++i) in |= (strict ? v[i] > bound : v[i] >= bound) ? 1u << i : 0u;
#pragma unroll 1
      while (in) {
        const int i = __ffs(in) - 1;
        in &= in - 1;
        float x = v[0];
#pragma unroll
        for (int k = 1; k < kVals; ++k) x = k == i ? v[k] : x;
        if (tile.has(at, i)) {
          const int pos = atomicAdd(&sh.count, 1);
          if (pos < kCap) sh.cand[pos] = key_of(x, tile.index_of(at, i));
        }
      }
    }
    if (number == pick_at) {
      // the best so far are the bound of later tiles; after tiles 0, 3, 15, 63, ... few pass it, and there is no barrier between
      __syncthreads();
      const int n = sh.count;
      __syncthreads();
      if (n <= kCap) {
        strict = pick(sh, n, top) == top;              // later entries lose ties
        bound = strict ? key_value(sh.cand[top - 1]) : -INFINITY;
        __syncthreads();
      }
      pick_at = 4 * pick_at + 3;
    }
  }
  __syncthreads();
  int n = sh.count;
  if (n > kCap) n = best_slowly<T>(sh, tile, lo, top);
  else n = pick(sh, n, top);

  // the CTA's sums, relative to its largest entry, then the cluster's
  {
    float m = a.m;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(~0u, m, o));
    if (lane == 0) sh.sums[warp].m = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWarps; ++w) m = max_nan(m, sh.sums[w].m);
    a = join(a, Sums{m, 0.f, 0.f});
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) a.s += __shfl_xor_sync(~0u, a.s, o), a.t += __shfl_xor_sync(~0u, a.t, o);
    if (lane == 0) sh.sums[warp].s = a.s, sh.sums[warp].t = a.t;
    __syncthreads();
    a.s = a.t = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) a.s += sh.sums[w].s, a.t += sh.sums[w].t;
  }
  const u64* list = sh.cand;
  if (CL > 1) {
    // every CTA puts its list and sums into the first one's memory
    asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
    if (tid < top) cluster.map_shared_rank(lists, 0)[rank * top + tid] = tid < n ? sh.cand[tid] : 0ull;
    if (tid == 0) cluster.map_shared_rank(parts, 0)[rank] = a;
    cluster.sync();
    if (rank != 0) return;
    a = parts[0];
#pragma unroll
    for (int c = 1; c < kMaxCluster; ++c)
      if (c < CL) a = join(a, parts[c]);
    {
      for (int i = tid; i < CL * top; i += kThreads) {
        const u64 k = lists[i];
        int r = 0;
#pragma unroll 4
        for (int j = 0; j < CL * top; ++j) r += lists[j] > k;
        if (k != 0 && r < top) sh.sorted[r] = k;
      }
      __syncthreads();
    }
    list = sh.sorted;
  }
  // no distribution: a NaN or +inf (in the maximum), or nothing finite (the sum is 0)
  const bool bad = !(a.s > 0.f) || !(a.m < INFINITY);
  const float log_s = logf(a.s), none = __int_as_float(0x7fc00000);
  if (tid < top) {
    const u64 k = list[tid];
    p.top_logp[static_cast<long long>(row) * top + tid] = bad ? none : (key_value(k) - a.m) - log_s;
    p.top_token[static_cast<long long>(row) * top + tid] = bad ? -1 : key_index(k);
  }
  if (tid == 0) {
    if (bad) device_error(p.err, GDN_DEVERR_LOGITS, row);
    if (p.entropy) p.entropy[row] = bad ? none : log_s - a.t / a.s;
    if (p.tokens) {
      const int token = p.tokens[row];
      p.given[row] = bad || token < 0 || token >= p.V ? none : (Vec<T>::one(z + token) - a.m) - log_s;
    }
  }
}

template <typename T>
cudaError_t launch_t(const LogprobParams& p, cudaStream_t s) {
  int CL = 1;
  while (CL < kMaxCluster && p.rows * CL < 304 && p.V / (2 * CL) >= 16384) CL *= 2;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(p.rows) * CL);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = CL, at[0].val.clusterDim.y = 1, at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, logprob_kernel<T>, p);
}
}  // namespace

cudaError_t launch_logprobs(const LogprobParams& p, cudaStream_t s) {
  return p.dtype == GDN_DTYPE_BF16 ? launch_t<__nv_bfloat16>(p, s) : launch_t<float>(p, s);
}

}  // namespace gdn
