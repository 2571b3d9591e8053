// Acceptance of drafted tokens: the walk down a request's tree, from given random
// numbers (the rule is stated in gdn_tree.h).
//
// One thread-block cluster walks one request; its CTAs share every row of logits
// by slices of the vocabulary and exchange their partial sums through distributed
// shared memory, so a step costs one read of one row, one cluster barrier and no
// launch: only the rows on the accepted path are read.  Every CTA takes each
// decision itself from the same numbers in the same order.  The bound is the
// bytes of the visited rows when many requests share the GPU, and the latency of
// a step (a row's loads, two block barriers, one cluster barrier) when few do.
//
// Sums and probabilities are fp32.  Scores of the next token are z / T + gumbel
// with each operation rounded once, so that the choice does not depend on how the
// compiler contracts it.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cmath>

#include "gdn_accept.cuh"

namespace cg = cooperative_groups;

namespace gdn {
namespace {

constexpr int kThreads = 512;
constexpr int kMaxCluster = 8;
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }

// Sixteen bytes of a row as fp32.
template <typename T>
struct Vec;
template <>
struct Vec<float> {
  static constexpr int N = 4;
  static __device__ __forceinline__ void load(const float* p, float (&x)[4]) {
    const float4 v = __ldg(reinterpret_cast<const float4*>(p));
    x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
  }
};
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int N = 8;
  static __device__ __forceinline__ void load(const __nv_bfloat16* p, float (&x)[8]) {
    const uint4 v = __ldg(reinterpret_cast<const uint4*>(p));
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
};

// Order-preserving key of (value, lowest index wins); values are not NaN.
__device__ __forceinline__ unsigned long long key_of(float v, int idx) {
  const uint32_t u = __float_as_uint(v + 0.f);     // -0 counts as +0
  const uint32_t o = (u & 0x80000000u) ? ~u : (u | 0x80000000u);
  return (static_cast<unsigned long long>(o) << 32) | (0xFFFFFFFFu - static_cast<uint32_t>(idx));
}
__device__ __forceinline__ float key_value(unsigned long long k) {
  const uint32_t o = static_cast<uint32_t>(k >> 32);
  return __uint_as_float((o & 0x80000000u) ? (o & 0x7FFFFFFFu) : ~o);
}
__device__ __forceinline__ int key_index(unsigned long long k) {
  return static_cast<int>(0xFFFFFFFFu - static_cast<uint32_t>(k));
}

// What a CTA's slice of a row contributes.
struct Partial {
  float m, s;                 // running maximum (of z log2 e / T), sum of 2^(. - m)
  unsigned long long top;     // best (value, index)
};
__device__ __forceinline__ Partial join(Partial a, Partial b) {
  Partial r;
  r.m = fmaxf(a.m, b.m);
  const float ref = r.m == -INFINITY ? 0.f : r.m;
  r.s = a.s * exp2f(a.m - ref) + b.s * exp2f(b.m - ref);
  r.top = a.top > b.top ? a.top : b.top;
  return r;
}
__device__ __forceinline__ Partial empty_partial() { return Partial{-INFINITY, 0.f, 0ull}; }

struct Shared {
  Partial warp[kThreads / 32];
  Partial slot[2][kMaxCluster];      // written by the cluster's CTAs, alternating by step
  int parent[GDN_MAX_NODES], token[GDN_MAX_NODES];
  float zc[GDN_MAX_NODES];           // children's logits of the current row
  float qc[GDN_MAX_NODES];           // and their draft probabilities
  int node, child, more, path_len, n_tried;
  int tried[GDN_MAX_NODES];
  float c, mass;
};

// The cluster's join of every thread's partial, known to all threads.  `step` alternates the slots: a slot is
// written again only after the barrier of the step in between.
__device__ Partial cluster_join(cg::cluster_group& cl, Shared& sh, Partial x, int& step) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int o = 16; o > 0; o >>= 1) {
    Partial y;
    y.m = __shfl_xor_sync(0xffffffffu, x.m, o);
    y.s = __shfl_xor_sync(0xffffffffu, x.s, o);
    y.top = __shfl_xor_sync(0xffffffffu, x.top, o);
    // the lower lane's part first, so that all lanes round alike
    x = (lane & o) ? join(y, x) : join(x, y);
  }
  if (lane == 0) sh.warp[warp] = x;
  __syncthreads();
  const int n = cl.num_blocks(), rank = cl.block_rank(), par = step & 1;
  if (threadIdx.x < n) {
    Partial t = sh.warp[0];
    for (int i = 1; i < kThreads / 32; ++i) t = join(t, sh.warp[i]);
    Shared* there = cl.map_shared_rank(&sh, threadIdx.x);
    there->slot[par][rank] = t;
  }
  cl.sync();
  Partial r = sh.slot[par][0];
  for (int i = 1; i < n; ++i) r = join(r, sh.slot[par][i]);
  ++step;
  return r;
}

template <typename TL, typename TQ>
__global__ void __launch_bounds__(kThreads) accept_walk_kernel(AcceptParams p) {
  cg::cluster_group cl = cg::this_cluster();
  __shared__ Shared sh;
  const int ranks = cl.num_blocks(), rank = cl.block_rank();
  const int b = blockIdx.x / ranks, tid = threadIdx.x;
  const SchedLayout lay{p.n_max};
  const int32_t* rec = p.words + static_cast<size_t>(b) * lay.words();
  const int n = rec[0];
  int32_t* path = p.path + static_cast<size_t>(b) * p.n_max;
  if (n < 1 || n > p.n_max) {           // the whole cluster reads the same record
    if (rank == 0) {
      if (tid == 0) {
        device_error(p.err, GDN_DEVERR_SCHEDULE, b);
        p.len[b] = 0;
        p.next[b] = -1;
      }
      if (tid < p.n_max) path[tid] = -1;
    }
    return;
  }
  const float T = p.temperature ? p.temperature[b] : 0.f;
  const bool cold = T == 0.f;
  bool bad = !(T >= 0.f) || T == INFINITY;
  if (tid < n) {
    sh.parent[tid] = rec[lay.parent() + tid];
    sh.token[tid] = p.tokens[static_cast<size_t>(b) * p.n_max + tid];
  }
  if (tid == 0) {
    sh.node = 0;
    sh.path_len = 0;
  }
  if (rank == 0 && tid < p.n_max) path[tid] = -1;
  cl.sync();                            // every CTA runs before its shared memory is written from outside

  const TL* logits = static_cast<const TL*>(p.logits);
  const TQ* draft = static_cast<const TQ*>(p.draft);
  const size_t row_of_b = static_cast<size_t>(b) * p.n_max;
  const float scale2 = cold ? kLog2e : kLog2e / T;
  const int V = p.V;
  int step = 0, pick = -1;

  while (!bad) {
    const int node = sh.node;
    const TL* z = logits + (row_of_b + node) * p.v_stride;
    const TQ* q = draft ? draft + (row_of_b + node) * p.v_stride : nullptr;
    if (tid < n) {                      // the children's entries, ahead of the row
      const int t = sh.token[tid];
      const bool kid = tid > 0 && sh.parent[tid] == node && t >= 0 && t < V;
      sh.zc[tid] = kid ? to_f(z[t]) : -INFINITY;
      sh.qc[tid] = (kid && q) ? to_f(q[t]) : 0.f;
    }
    if (tid == 0) {
      if (rank == 0) path[sh.path_len] = node;
      ++sh.path_len;
    }
    // ---- the row: maximum and sum, or the first largest logit
    Partial x = empty_partial();
    bool nan = false;
    constexpr int N = Vec<TL>::N;
    const int head = min(V, static_cast<int>(((16 - (reinterpret_cast<uintptr_t>(z) & 15)) & 15) / sizeof(TL)));
    const int vecs = (V - head) / N;
    auto take = [&](const float* v, int base, int count) {
      if (cold) {
        for (int i = 0; i < count; ++i) {
          nan = nan || v[i] != v[i];
          const unsigned long long k = key_of(v[i] != v[i] ? -INFINITY : v[i], base + i);
          x.top = x.top > k ? x.top : k;
        }
      } else {
        float m = x.m;
        for (int i = 0; i < count; ++i) m = fmaxf(m, v[i] * scale2);
        const float ref = m == -INFINITY ? 0.f : m;
        float s = x.s * exp2f(x.m - ref);
        for (int i = 0; i < count; ++i) s += exp2f(fmaf(v[i], scale2, -ref));
        x.m = m;
        x.s = s;
      }
    };
    for (int i = rank * kThreads + tid; i < vecs; i += ranks * kThreads) {
      float v[N];
      Vec<TL>::load(z + head + static_cast<size_t>(i) * N, v);
      take(v, head + i * N, N);
    }
    if (rank == 0) {                    // what the aligned vectors leave: fewer than 2 N values
      const int rest = V - vecs * N;
      if (tid < rest) {
        const int at = tid < head ? tid : head + vecs * N + (tid - head);
        const float v[1] = {to_f(z[at])};
        take(v, at, 1);
      }
    }
    if (nan) x.top = key_of(INFINITY, 0);      // a NaN reads as the infinity that ends the walk
    x = cluster_join(cl, sh, x, step);
    const float mx = x.m, total = x.s;
    // a NaN or +inf makes the sum NaN; a row of -inf leaves it 0
    if (cold ? !(fabsf(key_value(x.top)) < INFINITY) : !(total > 0.f && total < INFINITY)) {
      bad = true;
      break;
    }
    // ---- the children, in index order
    auto prob = [&](float zv) { return exp2f(fmaf(zv, scale2, -mx)) / total; };
    if (tid == 0) {
      sh.child = -1;
      sh.more = -1;
      sh.n_tried = 0;
      sh.c = 0.f;
      sh.mass = 1.f;
      float left = 1.f;
      for (int j = node + 1; j < n; ++j) {
        if (sh.parent[j] != node) continue;
        const int t = sh.token[j];
        const bool in = t >= 0 && t < V;
        bool yes;
        if (cold) {
          yes = in && t == key_index(x.top);
        } else if (!q) {
          float w = in ? prob(sh.zc[j]) : 0.f;
          for (int k = 0; k < sh.n_tried; ++k)
            if (sh.tried[k] == t) w = 0.f;
          yes = p.uniform[row_of_b + j] * left < w;
          if (!yes) {
            left -= w;
            sh.tried[sh.n_tried++] = t;
          }
        } else {
          yes = in && p.uniform[row_of_b + j] * sh.qc[j] < prob(sh.zc[j]);
          if (!yes) {                   // later siblings need what is left of the whole row
            sh.c = 1.f;
            sh.more = j;
          }
        }
        if (yes) {
          sh.child = j;
          break;
        }
        if (sh.more >= 0) break;
      }
    }
    __syncthreads();
    int child = sh.child;
    float c = sh.c;
    if (q && !cold) {
      int j = sh.more;                  // the last rejected child
      while (child < 0 && j >= 0) {
        int k = j + 1;                  // the next sibling
        while (k < n && sh.parent[k] != node) ++k;
        if (k >= n) break;
        // N = sum (p - c q)+
        Partial y = empty_partial();
        y.m = 0.f;
        for (int i = rank * kThreads + tid; i < V; i += ranks * kThreads)
          y.s += fmaxf(prob(to_f(z[i])) - c * to_f(q[i]), 0.f);
        y = cluster_join(cl, sh, y, step);
        const float mass = y.s;
        const int t = sh.token[k];
        const float r = fmaxf(prob(sh.zc[k]) - c * sh.qc[k], 0.f);
        const bool yes = t >= 0 && t < V && p.uniform[row_of_b + k] * sh.qc[k] * mass < r;
        if (yes) {
          child = k;
        } else {
          c += mass;
        }
        j = k;
      }
    }
    __syncthreads();                    // sh is read above by every thread
    if (child >= 0) {
      if (tid == 0) sh.node = child;
      __syncthreads();
      continue;
    }
    // ---- the stop: the next token from what is left of this row
    if (cold) {
      pick = key_index(x.top);
      break;
    }
    for (int whole = 0; whole < 2 && pick < 0; ++whole) {   // p itself where nothing is left
      Partial y = empty_partial();
      const float* g = p.gumbel + static_cast<size_t>(b) * V;
      const float use = whole ? 0.f : c;
      for (int i = rank * kThreads + tid; i < V; i += ranks * kThreads) {
        const float zv = to_f(z[i]);
        float score;
        if (!q) {
          score = __fadd_rn(__fdiv_rn(zv, T), g[i]);
        } else {
          const float r = prob(zv) - use * to_f(q[i]);
          if (!(r > 0.f)) continue;
          score = __fadd_rn(logf(r), g[i]);
        }
        const unsigned long long k = key_of(score, i);
        if (score > -INFINITY && k > y.top) {
          bool out = false;
          if (!q && !whole)
            for (int e = 0; e < sh.n_tried; ++e) out = out || sh.tried[e] == i;
          if (!out) y.top = k;
        }
      }
      y = cluster_join(cl, sh, y, step);
      if (y.top != 0ull) pick = key_index(y.top);
    }
    break;
  }
  if (rank == 0 && tid == 0) {
    if (bad) device_error(p.err, GDN_DEVERR_LOGITS, b);
    if (bad && sh.path_len == 0) path[sh.path_len++] = 0;    // a bad temperature: the root alone
    p.len[b] = sh.path_len;
    p.next[b] = pick;
  }
  cl.sync();                            // no CTA leaves while others may still write to it
}

template <typename TL, typename TQ>
cudaError_t walk_t(const AcceptParams& p, cudaStream_t s) {
  cudaLaunchConfig_t cfg{};
  const int ranks = p.V >= 8192 ? kMaxCluster : 1;
  cfg.gridDim = dim3(static_cast<unsigned>(p.B) * ranks);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ranks;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, accept_walk_kernel<TL, TQ>, p);
}

}  // namespace

cudaError_t launch_accept(const AcceptParams& p, cudaStream_t s) {
  const bool qf = p.draft_dtype == GDN_DTYPE_F32;
  if (p.logits_dtype == GDN_DTYPE_BF16)
    return qf ? walk_t<__nv_bfloat16, float>(p, s) : walk_t<__nv_bfloat16, __nv_bfloat16>(p, s);
  return qf ? walk_t<float, float>(p, s) : walk_t<float, __nv_bfloat16>(p, s);
}

}  // namespace gdn
