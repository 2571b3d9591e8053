// Acceptance of drafted tokens: the walk down a request's tree, from given random
// numbers (the rule is stated in gdn_tree.h).
//
// What the walk needs of a row of logits is three numbers -- its maximum, its sum
// of exponentials, or its first largest entry -- and the children's entries.  Two
// ways to get them:
//  - all rows at once (accept_rows_kernel): every node's row is reduced by slices,
//    the whole GPU busy, and the walk then only looks numbers up.  Its bound is the
//    bytes of all rows, read once;
//  - along the walk: a request's cluster reads the rows on its path, one after
//    another.  Few bytes, but every step waits for a row's latency and a cluster
//    barrier.
// The first is taken while all rows are few (kRowsAtOnce entries, twice as many with
// draft probabilities, where the walk's steps cost more).  Its time goes with the
// entries, of either type; the walk's with the nodes it visits, which nothing knows
// beforehand.  Measured (us, at once : along the walk, by nodes visited):
//   B x n x V                  M entries   1          3          6          9
//   4 x 22 x 131072, bf16        12     19 : 15    19 : 19    21 : 26    23 : 33
//   8 x 22 x 131072              23     23 : 15    24 : 19    25 : 26    27 : 33
//   12 x 22 x 131072             35     27 : 15    27 : 19    29 : 27    31 : 33
//   24 x 22 x 131072             69     47 : 17    47 : 23    49 : 33    50 : 43
//   64 x 22 x 32000              45     37 : 19    38 : 29    41 : 42    44 : 56
//   chains of 9 with draft probabilities, fp32 (visited   1.7       3.5       6.5       7.5)
//   32 x 9 x 65537               19     27 : 23    27 : 31    29 : 35    29 : 39
//   96 x 9 x 65537               57     83 : 60    87 : 83    90 : 110   92 : 125
// The limits lie where a walk of six nodes costs the same.  The walk of 32 trees of 22
// such rows, 2.5 of them visited on average, reads 44 MB in 44 us (1.0 TB/s): its bound
// is the latency of the steps, not the bytes.  The reduction of 64 chains' rows reads
// its 151 MB at 4.5 TB/s.
//
// One thread-block cluster walks one request.  Its CTAs share each row they read by
// slices and exchange their partial results through distributed shared memory;
// every CTA takes each decision itself from the same numbers in the same order.
//
// Sums and probabilities are fp32.  Exponents are (z - row's maximum) / T, the difference
// first: z / T alone would round to steps larger than 1 at small temperatures, and a
// product that the subtraction sees unrounded would leave that step in the exponent.
// Scores of the next token are (z - maximum) / T + gumbel with each operation rounded
// once, so that the choice does not depend on how the compiler contracts it.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cmath>
#include <type_traits>

#include "gdn_accept.cuh"

namespace cg = cooperative_groups;

namespace gdn {
namespace {

constexpr int kThreads = 512;
constexpr int kMaxCluster = 8;
constexpr int kRowThreads = 256;
constexpr double kRowsAtOnce = 1 << 25;      // entries
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }

// Sixteen bytes of a row as fp32.
template <typename T>
struct Vec;
template <>
struct Vec<float> {
  static constexpr int N = 4;
  static __device__ __forceinline__ void unpack(uint4 v, float (&x)[4]) {
    x[0] = __uint_as_float(v.x); x[1] = __uint_as_float(v.y); x[2] = __uint_as_float(v.z); x[3] = __uint_as_float(v.w);
  }
};
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int N = 8;
  static __device__ __forceinline__ void unpack(uint4 v, float (&x)[8]) {
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

// What a slice of a row contributes.
struct __align__(16) Partial {
  float m, s;                 // maximum, sum of 2^((z - m) log2 e / T)
  unsigned long long top;     // best (value, index)
};
__device__ __forceinline__ Partial empty_partial() { return Partial{-INFINITY, 0.f, 0ull}; }
__device__ __forceinline__ float exp2_fast(float x) {   // results below 2^-126 are zero
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// The warp's join, the same in every lane: of maxima and sums (the sums rescaled once, to the warp's maximum), or of
// the best entries.
__device__ __forceinline__ Partial warp_join_sum(Partial x, float scale2) {
  float m = x.m;
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  float s = x.s * exp2_fast((x.m - (m == -INFINITY ? 0.f : m)) * scale2);
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return Partial{m, s, 0ull};
}
__device__ __forceinline__ Partial warp_join_top(Partial x) {
  unsigned long long top = x.top;
  for (int o = 16; o > 0; o >>= 1) {
    const unsigned long long y = __shfl_xor_sync(0xffffffffu, top, o);
    top = top > y ? top : y;
  }
  return Partial{-INFINITY, 0.f, top};
}
__device__ __forceinline__ Partial warp_join(Partial x, bool top, float scale2) {
  return top ? warp_join_top(x) : warp_join_sum(x, scale2);
}
// log2 e / T and 1 / T, finite for the smallest temperatures too (0 times them is 0).
__device__ __forceinline__ float over_temperature(float x, float T) { return fminf(x / T, 3.402823466e38f); }

// This thread's share of part `part` of `parts` of a row: every parts * threads-th 16-byte vector, kAhead loads in
// flight, and what the aligned vectors leave (part 0).  A NaN makes the sum NaN, or the first largest +inf.
template <typename TL>
__device__ __forceinline__ Partial scan_row(const TL* z, int V, float scale2, bool cold, int part, int parts) {
  constexpr int N = Vec<TL>::N, kAhead = 4;
  Partial x = empty_partial();
  float best = -INFINITY;              // (greedy) the first largest entry of this thread's, whose indices ascend
  int at_best = -1;
  bool nan = false;
  const int head = min(V, static_cast<int>(((16 - (reinterpret_cast<uintptr_t>(z) & 15)) & 15) / sizeof(TL)));
  const int vecs = (V - head) / N;
  auto take = [&](const float* v, int base, int count) {
    if (cold) {
#pragma unroll
      for (int i = 0; i < count; ++i) {
        nan = nan || v[i] != v[i];
        if (v[i] > best || at_best < 0) {
          best = v[i];
          at_best = base + i;
        }
      }
    } else {
      float m = x.m;
#pragma unroll
      for (int i = 0; i < count; ++i) m = fmaxf(m, v[i]);
      const float ref = m == -INFINITY ? 0.f : m;
      float s = x.s * exp2_fast((x.m - ref) * scale2);
#pragma unroll
      for (int i = 0; i < count; ++i) s += exp2_fast((v[i] - ref) * scale2);
      x.m = m;
      x.s = s;
    }
  };
  const uint4* body = reinterpret_cast<const uint4*>(z + head);
  const int stride = parts * static_cast<int>(blockDim.x);
  for (int i = part * static_cast<int>(blockDim.x) + threadIdx.x; i < vecs; i += kAhead * stride) {
    uint4 raw[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
      if (i + k * stride < vecs) raw[k] = __ldg(body + i + k * stride);
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
      if (i + k * stride < vecs) {
        float v[N];
        Vec<TL>::unpack(raw[k], v);
        take(v, head + (i + k * stride) * N, N);
      }
  }
  if (at_best >= 0) x.top = key_of(best, at_best);
  if (part == 0) {                      // fewer than 2 N values, of any index
    const int rest = V - vecs * N, tid = threadIdx.x;
    if (tid < rest) {
      const int at = tid < head ? tid : head + vecs * N + (tid - head);
      const float v[1] = {to_f(z[at])};
      const unsigned long long before = x.top;
      best = -INFINITY;
      at_best = -1;
      take(v, at, 1);
      if (cold) {
        const unsigned long long k = key_of(best, at_best);
        x.top = before > k ? before : k;
      }
    }
  }
  if (nan) x.top = key_of(INFINITY, 0);
  return x;
}

// Every node's row, a slice a CTA.
template <typename TL>
__global__ void __launch_bounds__(kRowThreads) accept_rows_kernel(AcceptParams p) {
  __shared__ Partial part[kRowThreads / 32];
  const int row = blockIdx.y, b = row / p.n_max, node = row % p.n_max;
  const int n = p.words[static_cast<size_t>(b) * SchedLayout{p.n_max}.words()];
  if (node >= n || n > p.n_max) return;
  const float T = p.temperature ? p.temperature[b] : 0.f;
  const bool cold = T == 0.f;
  if (!(T >= 0.f) || T == INFINITY) return;             // the walk reports it
  const TL* z = static_cast<const TL*>(p.logits) + static_cast<size_t>(row) * p.v_stride;
  const int lane = threadIdx.x & 31;
  const float scale2 = cold ? kLog2e : over_temperature(kLog2e, T);
  Partial x = warp_join(scan_row<TL>(z, p.V, scale2, cold, blockIdx.x, gridDim.x), cold, scale2);
  if (lane == 0) part[threadIdx.x >> 5] = x;
  __syncthreads();
  if (threadIdx.x < 32) {
    x = warp_join(lane < kRowThreads / 32 ? part[lane] : empty_partial(), cold, scale2);
    if (lane == 0) static_cast<Partial*>(p.slices)[static_cast<size_t>(row) * gridDim.x + blockIdx.x] = x;
  }
}

struct Shared {
  Partial warp[kThreads / 32];
  Partial slot[2][kMaxCluster];      // written by the cluster's CTAs, alternating by step
  Partial row[GDN_MAX_NODES];        // each node's row, where all were reduced at once
  int parent[GDN_MAX_NODES], token[GDN_MAX_NODES];
  float uniform[GDN_MAX_NODES];
  float zc[GDN_MAX_NODES];           // each node's entry in its parent's row of logits
  float qc[GDN_MAX_NODES];           // and of draft probabilities
  unsigned long long kids[GDN_MAX_NODES];
  int child, more, n_tried;
  int tried[GDN_MAX_NODES];
};

// The cluster's join of every thread's partial, known to all threads.  `step` alternates the slots: a slot is
// written again only after the barrier of the step in between.
__device__ __forceinline__ Partial cluster_join(cg::cluster_group& cl, Shared& sh, Partial x, int& step, bool top,
                                                float scale2) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  x = warp_join(x, top, scale2);
  if (lane == 0) sh.warp[warp] = x;
  __syncthreads();
  const int n = cl.num_blocks(), rank = cl.block_rank(), par = step & 1;
  if (warp == 0) {
    const Partial t = warp_join(lane < kThreads / 32 ? sh.warp[lane] : empty_partial(), top, scale2);
    if (lane < n) cl.map_shared_rank(&sh, lane)->slot[par][rank] = t;
  }
  cl.sync();
  ++step;
  return warp_join(lane < n ? sh.slot[par][lane] : empty_partial(), top, scale2);
}

// TQ: the type of the draft probabilities, void without them.
template <typename TL, typename TQ, bool kAtOnce>
__global__ void __launch_bounds__(kThreads) accept_walk_kernel(AcceptParams p) {
  cg::cluster_group cl = cg::this_cluster();
  __shared__ Shared sh;
  const int ranks = cl.num_blocks(), rank = cl.block_rank();
  const int b = blockIdx.x / ranks, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
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
  const TL* logits = static_cast<const TL*>(p.logits);
  constexpr bool kDraft = !std::is_void_v<TQ>;
  using Q = std::conditional_t<kDraft, TQ, float>;
  const Q* draft = static_cast<const Q*>(p.draft);
  const size_t row_of_b = static_cast<size_t>(b) * p.n_max;
  const float scale2 = cold ? kLog2e : over_temperature(kLog2e, T);
  const int V = p.V;
  // everything the decisions look up, for every node at once
  if (tid < n) {
    const int parent = rec[lay.parent() + tid], t = p.tokens[row_of_b + tid];
    sh.parent[tid] = tid > 0 && parent >= 0 && parent < tid ? parent : -1;
    sh.token[tid] = t;
    sh.uniform[tid] = cold ? 0.f : p.uniform[row_of_b + tid];
    float zc = -INFINITY, qc = 0.f;
    if (sh.parent[tid] >= 0 && t >= 0 && t < V) {
      zc = to_f(logits[(row_of_b + parent) * p.v_stride + t]);
      if (kDraft) qc = to_f(draft[(row_of_b + parent) * p.v_stride + t]);
    }
    sh.zc[tid] = zc;
    sh.qc[tid] = qc;
  }
  if (rank == 0 && tid < p.n_max) path[tid] = -1;
  __syncthreads();
  if (tid < n) {
    unsigned long long kids = 0;
    for (int j = tid + 1; j < n; ++j) kids |= static_cast<unsigned long long>(sh.parent[j] == tid) << j;
    sh.kids[tid] = kids;
  }
  if constexpr (kAtOnce) {
    asm volatile("griddepcontrol.wait;" ::: "memory");   // launched ahead of the rows' kernel's end
    const Partial* slices = static_cast<const Partial*>(p.slices);
    for (int i = warp; i < n; i += kThreads / 32) {
      // (a row of any size: 32 slices at a time, with what they make in lane 0's place)
      Partial x = empty_partial();
      for (int k0 = 0; !bad && k0 < p.n_slices; k0 += 31) {
        const int k = k0 + lane - 1;
        if (lane > 0) x = k < p.n_slices ? slices[(row_of_b + i) * p.n_slices + k] : empty_partial();
        x = warp_join(x, cold, scale2);
      }
      if (lane == 0) sh.row[i] = x;
    }
  }
  cl.sync();                            // every CTA runs before its shared memory is written from outside

  int step = 0, pick = -1, node = 0, path_len = 0;
  while (!bad) {
    const TL* z = logits + (row_of_b + node) * p.v_stride;
    const Q* q = kDraft ? draft + (row_of_b + node) * p.v_stride : nullptr;
    if (rank == 0 && tid == 0) path[path_len] = node;
    ++path_len;
    const Partial x =
        kAtOnce ? sh.row[node] : cluster_join(cl, sh, scan_row<TL>(z, V, scale2, cold, rank, ranks), step, cold, scale2);
    const float mx = x.m, total = x.s;
    // a NaN or +inf makes the sum NaN; a row of -inf leaves it 0
    if (cold ? !(fabsf(key_value(x.top)) < INFINITY) : !(total > 0.f && total < INFINITY)) {
      bad = true;
      break;
    }
    // ---- the children, in index order: by one thread
    auto prob = [&](float zv) { return exp2f(__fmul_rn(__fsub_rn(zv, mx), scale2)) / total; };
    if (tid == 0) {
      sh.child = -1;
      sh.more = -1;
      sh.n_tried = 0;
      float left = 1.f;
      for (unsigned long long kids = sh.kids[node]; kids; kids &= kids - 1) {
        const int j = __ffsll(static_cast<long long>(kids)) - 1, t = sh.token[j];
        const bool in = t >= 0 && t < V;
        bool yes;
        if (cold) {
          yes = in && t == key_index(x.top);
        } else if constexpr (!kDraft) {
          float w = in ? prob(sh.zc[j]) : 0.f;
          for (int k = 0; k < sh.n_tried; ++k)
            if (sh.tried[k] == t) w = 0.f;
          yes = sh.uniform[j] * left < w;
          if (!yes) {
            left -= w;
            sh.tried[sh.n_tried++] = t;
          }
        } else {
          yes = in && sh.uniform[j] * sh.qc[j] < prob(sh.zc[j]);
          if (!yes) sh.more = j;        // later siblings need what is left of the whole row
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
    // what is left after the last rejection is (p - next q)+; where that is empty, it stays what it was, (p - c q)+ of sum N
    float c = 0.f, N = 1.f, next = 0.f;
    if (kDraft && !cold && sh.more >= 0) {
      next = 1.f;
      // the rejected child's later siblings
      for (unsigned long long kids = sh.kids[node] & ~((2ull << sh.more) - 1); child < 0 && kids; kids &= kids - 1) {
        const int k = __ffsll(static_cast<long long>(kids)) - 1;
        Partial y = empty_partial();
        y.m = 0.f;
        for (int i = rank * kThreads + tid; i < V; i += ranks * kThreads)
          y.s += fmaxf(prob(to_f(z[i])) - next * to_f(q[i]), 0.f);
        const float mass = cluster_join(cl, sh, y, step, false, scale2).s;
        if (mass > 0.f) {
          c = next;
          N = mass;
        }
        const int t = sh.token[k];
        const float r = fmaxf(prob(sh.zc[k]) - c * sh.qc[k], 0.f);
        if (t >= 0 && t < V && sh.uniform[k] * sh.qc[k] * N < r)
          child = k;
        else
          next = c + N;
      }
    }
    if (child >= 0) {
      __syncthreads();                  // sh.child is read above by every thread
      node = child;
      continue;
    }
    // ---- the stop: the next token from what is left of this row
    if (cold) {
      pick = key_index(x.top);
      break;
    }
    const float rT = over_temperature(1.f, T), rtotal = 1.f / total;
    for (int whole = 0; whole < 2 && pick < 0; ++whole) {   // what there was before where nothing is left
      constexpr int kAhead = 8;
      Partial y = empty_partial();
      const float* g = p.gumbel + static_cast<size_t>(b) * V;
      const float use = whole ? c : next;
      const int stride = ranks * kThreads;
      float best = -INFINITY, floor = -INFINITY;            // this thread's best score, of ascending indices; the warp's bound
#pragma unroll 1
      for (int i0 = rank * kThreads + tid; i0 - lane < V; i0 += kAhead * stride) {      // by whole warps
        float zv[kAhead], gv[kAhead], qv[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
          const int i = i0 + k * stride;
          zv[k] = i < V ? to_f(z[i]) : -INFINITY;
          gv[k] = i < V ? __ldg(g + i) : 0.f;
          if (kDraft) qv[k] = i < V ? to_f(q[i]) : 0.f;
        }
        // the tried tokens among them (the stride is a power of two)
        unsigned skip = 0;
        if (!kDraft && !whole)
          for (int x = 0; x < sh.n_tried; ++x) {
            const unsigned d = static_cast<unsigned>(sh.tried[x] - i0);
            if (sh.tried[x] >= i0 && d < static_cast<unsigned>(kAhead * stride) && (d & (stride - 1)) == 0)
              skip |= 1u << (d / stride);
          }
        // Screening: each score within bounds of a few roundings, the warp's largest lower bound so far, and the entries
        // whose upper bound reaches it -- one or two a warp and step, which then are scored exactly
        float low = -INFINITY;
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
          float t, slack = 0.f;                             // the log weight from above, and how far below it may be
          if constexpr (!kDraft) {
            t = (zv[k] - mx) * rT;
          } else {
            // (the difference may cancel)
            const float pk = exp2_fast((zv[k] - mx) * scale2) * rtotal, qk = use * qv[k];
            const float up = fmaf(pk, 1.0001f, -0.9999f * qk), dn = fmaf(pk, 0.9999f, -1.0001f * qk);
            t = up > 0.f ? __logf(up) + 1e-3f : -INFINITY;
            slack = dn > 0.f ? t - __logf(dn) + 1e-3f : INFINITY;
          }
          const float a = t + gv[k], e = 1e-6f * (fabsf(t) + fabsf(gv[k]));
          zv[k] = (skip >> k & 1) || !(t > -INFINITY) ? -INFINITY : a + e;
          low = fmaxf(low, (skip >> k & 1) || !(t > -INFINITY) ? -INFINITY : a - e - slack);
        }
        for (int o = 16; o > 0; o >>= 1) low = fmaxf(low, __shfl_xor_sync(0xffffffffu, low, o));
        floor = fmaxf(floor, low);
        unsigned may = 0;
#pragma unroll
        for (int k = 0; k < kAhead; ++k) may |= static_cast<unsigned>(zv[k] >= floor && zv[k] > -INFINITY) << k;
        while (may) {
          const int k = __ffs(static_cast<int>(may)) - 1, i = i0 + k * stride;
          may &= may - 1;
          const float zi = to_f(z[i]), gi = __ldg(g + i);
          float score;
          if constexpr (!kDraft) {
            score = __fadd_rn(__fdiv_rn(__fsub_rn(zi, mx), T), gi);
          } else {
            const float r = prob(zi) - use * to_f(q[i]);
            score = r > 0.f ? __fadd_rn(logf(r), gi) : -INFINITY;
          }
          if (score > best) {
            best = score;
            y.top = key_of(score, i);
          }
        }
      }
      y = cluster_join(cl, sh, y, step, true, scale2);
      if (y.top != 0ull) pick = key_index(y.top);
    }
    break;
  }
  if (rank == 0 && tid == 0) {
    if (bad) device_error(p.err, GDN_DEVERR_LOGITS, b);
    if (bad && path_len == 0) path[path_len++] = 0;         // a bad temperature: the root alone
    p.len[b] = path_len;
    p.next[b] = pick;
  }
  cl.sync();                            // no CTA leaves while others may still write to it
}

template <typename TL, typename TQ, bool kAtOnce>
cudaError_t walk_t(const AcceptParams& p, cudaStream_t s) {
  cudaLaunchConfig_t cfg{};
  const int ranks = p.V >= 8192 ? kMaxCluster : 1;
  cfg.gridDim = dim3(static_cast<unsigned>(p.B) * ranks);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ranks;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = kAtOnce ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, accept_walk_kernel<TL, TQ, kAtOnce>, p);
}

template <typename TL, typename TQ>
cudaError_t accept_t(const AcceptParams& p, cudaStream_t s) {
  if (!p.n_slices) return walk_t<TL, TQ, false>(p, s);
  accept_rows_kernel<TL><<<dim3(p.n_slices, p.B * p.n_max), kRowThreads, 0, s>>>(p);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? walk_t<TL, TQ, true>(p, s) : e;
}

}  // namespace

// All rows at once while they are few; slices of 8192 entries, which a CTA of the rows' kernel reads in one go.
int accept_slices(int B, int n_max, int V, bool draft) {
  const double entries = static_cast<double>(B) * n_max * V;
  if (n_max < 2 || entries > (draft ? 2.0 : 1.0) * kRowsAtOnce || static_cast<long long>(B) * n_max > 65535) return 0;
  return (V + 8191) / 8192;
}

cudaError_t launch_accept(const AcceptParams& p, cudaStream_t s) {
  const bool bf = p.logits_dtype == GDN_DTYPE_BF16;
  if (!p.draft) return bf ? accept_t<__nv_bfloat16, void>(p, s) : accept_t<float, void>(p, s);
  if (p.draft_dtype == GDN_DTYPE_F32) return bf ? accept_t<__nv_bfloat16, float>(p, s) : accept_t<float, float>(p, s);
  return bf ? accept_t<__nv_bfloat16, __nv_bfloat16>(p, s) : accept_t<float, __nv_bfloat16>(p, s);
}

}  // namespace gdn
