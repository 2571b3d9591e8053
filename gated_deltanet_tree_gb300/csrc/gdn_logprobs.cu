// Log-probabilities of rows of logits: of a given token, of the best ones, and the entropy.
//
// One pass over a row keeps, relative to the running maximum m, s = sum e^(z - m) and
// t = sum e^(z - m) (z - m); then log p_i = z_i - m - log s and the entropy is log s - t / s.
//
// The best `top` tokens (larger logit first, lower index on ties) come from the same pass.  A tile
// of 4096 entries lies in the CTA's registers; the top-th largest of 32 group maxima of the first
// one bounds its top-th largest entry from below, so a handful of entries pass and are put on a list
// in shared memory.  Its exact best are picked by counting, and the worst of them is the bound of
// later tiles; it is renewed after ever more of them, and the warps need no barrier in between.  Where more entries pass than the list holds
// (long ties, rising rows) the best are found tile by tile, one after another, in a second pass.
//
// A cluster of up to eight CTAs shares a row where rows are few, joined through distributed
// shared memory.  The bound is the row's bytes, read once.
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

template <typename T>
struct Vec;
template <>
struct Vec<float> {
  static constexpr int N = 4;
  static __device__ __forceinline__ void unpack(uint4 v, float* x) {
    x[0] = __uint_as_float(v.x), x[1] = __uint_as_float(v.y), x[2] = __uint_as_float(v.z), x[3] = __uint_as_float(v.w);
  }
  static __device__ __forceinline__ float one(const float* p) { return *p; }
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
};

// Order-preserving key of (value, lowest index wins); never 0 for a value that is not NaN.
__device__ __forceinline__ u64 key_of(float v, int idx) {
  const uint32_t u = __float_as_uint(v + 0.f);     // -0 counts as +0
  const uint32_t o = (u & 0x80000000u) ? ~u : (u | 0x80000000u);
  return (static_cast<u64>(o) << 32) | (0xFFFFFFFFu - static_cast<uint32_t>(idx));
}
__device__ __forceinline__ float key_value(u64 k) {
  const uint32_t o = static_cast<uint32_t>(k >> 32);
  return __uint_as_float((o & 0x80000000u) ? (o & 0x7FFFFFFFu) : ~o);
}
__device__ __forceinline__ int key_index(u64 k) { return static_cast<int>(0xFFFFFFFFu - static_cast<uint32_t>(k)); }

__device__ __forceinline__ float exp2_fast(float x) {   // results below 2^-126 are zero
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float max_nan(float a, float b) {   // a NaN stays
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
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
__global__ void __launch_bounds__(kThreads, 4) logprob_kernel(const LogprobParams p) {
  constexpr int N = Vec<T>::N, kLoads = kVals / N;
  __shared__ Shared sh;
  __shared__ u64 lists[kMaxCluster * kLogprobTop];
  cg::cluster_group cluster = cg::this_cluster();
  const int CL = cluster.num_blocks(), rank = cluster.block_rank();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int row = blockIdx.x / CL, top = p.top;
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
    float v[kVals];
    if (fetched) Tile<T>::unpack(raw, v);
    else tile.load(at, v);
    const int next = at + kThreads * kLoads;
    fetched = next < tile.hi && tile.whole(next);
    if (fetched) tile.fetch(next, raw);
    float most = v[0];
#pragma unroll
    for (int i = 1; i < kVals; ++i) most = max_nan(most, v[i]);
    // the sums; a masked entry's difference must not be infinite (its exponential is 0), and a NaN is in the maximum
    if (!(most <= a.m)) a = join(a, Sums{most, 0.f, 0.f});
    const float ref = finite_ref(a.m);
    float s0 = 0.f, s1 = 0.f, t0 = 0.f, t1 = 0.f;
#pragma unroll
    for (int i = 0; i < kVals; i += 2) {
      const float d0 = fmaxf(v[i] - ref, -1e4f), d1 = fmaxf(v[i + 1] - ref, -1e4f);
      const float e0 = exp2_fast(d0 * kLog2e), e1 = exp2_fast(d1 * kLog2e);
      s0 += e0, s1 += e1;
      t0 = fmaf(e0, d0, t0), t1 = fmaf(e1, d1, t1);
    }
    a.s += s0 + s1;
    a.t += t0 + t1;
    // candidates
    if (number == 0) {
      float g = most;
#pragma unroll
      for (int o = 1; o < kWarps; o <<= 1) g = fmaxf(g, __shfl_xor_sync(~0u, g, o));
      if (tid % kWarps == 0) sh.groups[tid / kWarps] = g;     // (as many threads a group as there are warps)
      __syncthreads();
      g = sh.groups[lane];
      int r = 0;
#pragma unroll
      for (int j = 0; j < 32; ++j) {
        const float o = __shfl_sync(~0u, g, j);
        r += o > g || (o == g && j < lane);
      }
      bound = __shfl_sync(~0u, g, __ffs(__ballot_sync(~0u, r == top - 1)) - 1);
    }
    if (strict ? most > bound : !(most < bound)) {
#pragma unroll
      for (int i = 0; i < kVals; ++i)
        if ((strict ? v[i] > bound : v[i] >= bound) && tile.has(at, i)) {
          const int pos = atomicAdd(&sh.count, 1);
          if (pos < kCap) sh.cand[pos] = key_of(v[i], tile.index_of(at, i));
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
    __syncthreads();
    if (tid == 0) sh.sums[0] = a, sh.count = n;
    cluster.sync();
    if (rank == 0) {
      for (int c = 1; c < CL; ++c) a = join(a, cluster.map_shared_rank(&sh, c)->sums[0]);
      for (int i = tid; i < CL * kLogprobTop; i += kThreads) {
        const Shared* other = cluster.map_shared_rank(&sh, i / kLogprobTop);
        lists[i] = (i % kLogprobTop) < other->count ? other->cand[i % kLogprobTop] : 0ull;
      }
      __syncthreads();
      // each list is in order: an entry's rank is its place and how many of the others' are larger
      for (int i = tid; i < CL * kLogprobTop; i += kThreads) {
        const u64 k = lists[i];
        int r = i % kLogprobTop;
        for (int c = 0; c < CL; ++c) {
          if (c == i / kLogprobTop) continue;
          int larger = 0;
#pragma unroll
          for (int step = kLogprobTop / 2; step > 0; step >>= 1)
            if (lists[c * kLogprobTop + larger + step - 1] > k) larger += step;
          if (lists[c * kLogprobTop + larger] > k) ++larger;
          r += larger;
        }
        if (k != 0 && r < top) sh.sorted[r] = k;
      }
      __syncthreads();
    }
    cluster.sync();                                    // the others' lists have been read
    if (rank != 0) return;
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
  while (CL < kMaxCluster && p.rows * CL < 304 && p.V / (2 * CL) >= 8192) CL *= 2;
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
