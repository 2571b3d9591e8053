// Sequences through one GDN layer, token by token: single tokens (decoding) and short prompts.
//
// Per v-head with T = S^T [dk][dv]:  T <- g T;  u = beta (v - T^T k);  T <- T + k u^T;  o = T^T q.
// With the decayed tile g T both products need only what is known before u:
//   p = (g T)^T k,  r = (g T)^T q,  u = beta (v - p),  o = r + (q . k) u,
// so a token costs one pass over the tile, one reduction and one barrier.
//
// A CTA holds the tile of one v-head, or NS of its columns (columns do not depend on each
// other), in registers: each thread RPT adjacent rows of four columns.  The CTAs that share a
// k-head form a cluster: all of them read the q and k channels of the conv window, which a call
// in place overwrites, so they meet before one of them does.
//
// For a single token the bound is the state, read once and written once.
// Conv, SiLU, the norms and the order of their operations are those of the conv-window kernel.
#include <cooperative_groups.h>
#include <cuda_bf16.h>

#include "gdn_seq.cuh"

namespace cg = cooperative_groups;

namespace gdn {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kMaxCluster = 6;   // (6 CTAs a k-head's cluster: 9.8 us a token of 48 heads, 8: 10.4, 3: 12.7)

__device__ __forceinline__ float load_f(const float* p) { return __ldg(p); }
__device__ __forceinline__ float load_f(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ float silu(float y) { return __fdividef(y, 1.f + __expf(-y)); }
__device__ __forceinline__ void store4(float* p, const float (&v)[4]) {
  *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ void store4(__nv_bfloat16* p, const float (&v)[4]) {
  __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]), b = __floats2bfloat162_rn(v[2], v[3]);
  *reinterpret_cast<uint2*>(p) = make_uint2(*reinterpret_cast<uint32_t*>(&a), *reinterpret_cast<uint32_t*>(&b));
}

struct SeqOne {   // requests 0 .. n - 1, one row each
  int n;
};
__device__ __forceinline__ void request(const SeqOne&, int i, int& b, int& start, int& len) { b = start = i, len = 1; }
__device__ __forceinline__ void request(const SeqReqs& r, int i, int& b, int& start, int& len) {
  b = r.b[i], start = r.start[i], len = r.len[i];
}

// KT: taps, filled up with zeros in front (4 or 8).  TB: tokens convolved at once.
template <typename InT, typename Reqs, int DK, int NS, int KT, int TB>
__global__ void __launch_bounds__(kThreads) seq_rec_kernel(const SeqParams p, const __grid_constant__ Reqs reqs) {
  constexpr int kQuads = NS / 4, kGroups = kThreads / kQuads, RPT = DK / kGroups;
  constexpr int NC = 2 * DK + NS;                      // channels: q, k, the v slice
  static_assert(RPT >= 1, "a thread holds a row at least");
  __shared__ __align__(16) float ys[TB][NC];           // q, k (normalised), v of the block's tokens
  __shared__ float gates[TB][2];                       // beta, g
  __shared__ float qk[TB];                             // q . k
  __shared__ __align__(16) float2 part[2][kWarps][NS];
  cg::cluster_group cluster = cg::this_cluster();
  const int CL = cluster.num_blocks(), rank = cluster.block_rank();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int group = blockIdx.x / CL;
  const int kh = group % p.Hk;
  int b, start, len;
  request(reqs, group / p.Hk, b, start, len);
  if (p.live && p.live[b] == 0) return;                // the whole cluster's answer
  const int R = p.Hv / p.Hk, slices = p.dv / NS, items = R * slices;
  const int K = p.conv_mode == 1 ? p.K : 1, kq = p.Hk * DK;
  const InT* x = static_cast<const InT*>(p.x) + static_cast<long long>(start) * p.x_row;
  const float* win = p.conv_in ? p.conv_in + b * p.conv_stride : nullptr;
  const bool aborted = launch_aborted(p.err);

  const int c0 = 4 * (tid % kQuads), r0 = (tid / kQuads) * RPT;
  for (int item = rank; item < items; item += CL) {
    const int h = kh * R + item / slices, col0 = (item % slices) * NS;
    const long long tile = static_cast<long long>(h) * DK * p.dv + static_cast<long long>(r0) * p.dv + col0 + c0;
    float T[RPT][4];
    if (p.state_in) {
      const float* src = p.state_in + b * p.state_stride + tile;
#pragma unroll
      for (int i = 0; i < RPT; ++i) {
        const float4 t = __ldcs(reinterpret_cast<const float4*>(src + static_cast<long long>(i) * p.dv));
        T[i][0] = t.x, T[i][1] = t.y, T[i][2] = t.z, T[i][3] = t.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < RPT; ++i) T[i][0] = T[i][1] = T[i][2] = T[i][3] = 0.f;
    }
    for (int t0 = 0; t0 < len; t0 += TB) {
      const int nt = min(TB, len - t0);
      // conv and activation: a thread takes a channel through the block's tokens
      for (int c = tid; c < NC; c += kThreads) {
        const int ch = c < DK ? kh * DK + c : c < 2 * DK ? kq + kh * DK + c - DK : 2 * kq + h * p.dv + col0 + c - 2 * DK;
        float xr[TB + KT - 1], w[KT];
        // the rows, all in flight at once: those outside the request are read at its nearest row, and not used
#pragma unroll
        for (int i = 0; i < TB + KT - 1; ++i)
          xr[i] = load_f(x + static_cast<long long>(min(max(t0 + i - (KT - 1), 0), len - 1)) * p.x_row + ch);
#pragma unroll
        for (int j = 0; j < KT; ++j) {
          w[j] = j == KT - 1 && p.conv_mode != 1 ? 1.f : 0.f;
          if (p.conv_mode == 1) {
            const float f = __ldg(p.conv_w + static_cast<long long>(ch) * K + max(j - (KT - K), 0));
            w[j] = j >= KT - K ? f : 0.f;
          }
        }
        if (t0 == 0) {                                 // rows before the first: the window's, zeros where there is none
          float old[KT - 1];
#pragma unroll
          for (int i = 0; i < KT - 1; ++i)
            old[i] = win ? win[static_cast<long long>(max(i - (KT - K), 0)) * p.C + ch] : 0.f;
#pragma unroll
          for (int i = 0; i < KT - 1; ++i) xr[i] = i >= KT - K ? old[i] : 0.f;
        }
#pragma unroll
        for (int t = 0; t < TB; ++t) {
          float y = w[KT - 1] * xr[t + KT - 1];
#pragma unroll
          for (int i = 1; i < KT; ++i)
            if (i < K) y = fmaf(w[KT - 1 - i], xr[t + KT - 1 - i], y);
          if (p.act == 1) y = silu(y);
          if (t < nt) ys[t][c] = y;
        }
      }
      if (tid < nt) {
        const long long at = static_cast<long long>(start + t0 + tid) * p.gate_row + h;
        gates[tid][0] = load_f(static_cast<const InT*>(p.beta) + at);
        gates[tid][1] = expf(load_f(static_cast<const InT*>(p.log_g) + at));
      }
      if (__syncthreads_or(aborted)) {
        if (K > 1 && p.conv_out == p.conv_in && CL > 1) cluster.sync();   // as the others, at the end
        return;
      }
      for (int t = warp; t < nt; t += kWarps) {        // a warp normalises a token's q and k
        float q[DK / 32], k[DK / 32], sq = 0.f, sk = 0.f, d = 0.f;
#pragma unroll
        for (int i = 0; i < DK / 32; ++i) {
          q[i] = ys[t][lane + 32 * i], k[i] = ys[t][DK + lane + 32 * i];
          sq = fmaf(q[i], q[i], sq), sk = fmaf(k[i], k[i], sk);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sq += __shfl_xor_sync(~0u, sq, o), sk += __shfl_xor_sync(~0u, sk, o);
        const float nq = rsqrtf(sq + p.l2_eps) * p.q_scale, nk = rsqrtf(sk + p.l2_eps);
#pragma unroll
        for (int i = 0; i < DK / 32; ++i) {
          q[i] *= nq, k[i] *= nk;
          d = fmaf(q[i], k[i], d);
          ys[t][lane + 32 * i] = q[i], ys[t][DK + lane + 32 * i] = k[i];
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) d += __shfl_xor_sync(~0u, d, o);
        if (lane == 0) qk[t] = d;
      }
      __syncthreads();
      for (int t = 0; t < nt; ++t) {
        const float beta = gates[t][0], g = gates[t][1];
        float kr[RPT], pk[4] = {0.f, 0.f, 0.f, 0.f}, pq[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < RPT; ++i) {
          const float qi = ys[t][r0 + i];
          kr[i] = ys[t][DK + r0 + i];
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            T[i][c] *= g;
            pk[c] = fmaf(kr[i], T[i][c], pk[c]);
            pq[c] = fmaf(qi, T[i][c], pq[c]);
          }
        }
#pragma unroll
        for (int o = kQuads; o < 32; o <<= 1)          // the warp's row groups
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            pk[c] += __shfl_xor_sync(~0u, pk[c], o);
            pq[c] += __shfl_xor_sync(~0u, pq[c], o);
          }
        if (lane < kQuads) {
          float4* dst = reinterpret_cast<float4*>(&part[t & 1][warp][c0]);
          dst[0] = make_float4(pk[0], pq[0], pk[1], pq[1]);
          dst[1] = make_float4(pk[2], pq[2], pk[3], pq[3]);
        }
        __syncthreads();
        float sk[4] = {0.f, 0.f, 0.f, 0.f}, sq[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          const float4* src = reinterpret_cast<const float4*>(&part[t & 1][w][c0]);
          const float4 a = src[0], e = src[1];
          sk[0] += a.x, sq[0] += a.y, sk[1] += a.z, sq[1] += a.w;
          sk[2] += e.x, sq[2] += e.y, sk[3] += e.z, sq[3] += e.w;
        }
        float u[4];
        const float4 v = *reinterpret_cast<const float4*>(&ys[t][2 * DK + c0]);
        u[0] = beta * (v.x - sk[0]), u[1] = beta * (v.y - sk[1]);
        u[2] = beta * (v.z - sk[2]), u[3] = beta * (v.w - sk[3]);
#pragma unroll
        for (int i = 0; i < RPT; ++i)
#pragma unroll
          for (int c = 0; c < 4; ++c) T[i][c] = fmaf(kr[i], u[c], T[i][c]);
        if (tid < kQuads) {
          const float d = qk[t], o[4] = {fmaf(d, u[0], sq[0]), fmaf(d, u[1], sq[1]), fmaf(d, u[2], sq[2]), fmaf(d, u[3], sq[3])};
          const long long at = (static_cast<long long>(start + t0 + t) * p.Hv + h) * p.dv + col0 + c0;
          if (p.out_dtype == GDN_DTYPE_BF16) store4(static_cast<__nv_bfloat16*>(p.out) + at, o);
          else store4(static_cast<float*>(p.out) + at, o);
        }
      }
      if (t0 + TB < len || item + CL < items) __syncthreads();   // ys, gates and part are written again
    }
    float* dst = p.state_out + b * p.state_stride + tile;
#pragma unroll
    for (int i = 0; i < RPT; ++i)
      __stcs(reinterpret_cast<float4*>(dst + static_cast<long long>(i) * p.dv), make_float4(T[i][0], T[i][1], T[i][2], T[i][3]));
  }

  // The window after the last token: its last K - 1 rows, old ones among them where it has fewer tokens.
  if (K == 1) return;
  if (p.conv_out == p.conv_in) {
    if (CL > 1) cluster.sync();
    else __syncthreads();
  }
  float* wout = p.conv_out + b * p.conv_stride;
  const int nv = R * p.dv;
  for (int c = rank * kThreads + tid; c < 2 * DK + nv; c += CL * kThreads) {
    const int ch = c < DK ? kh * DK + c : c < 2 * DK ? kq + kh * DK + c - DK : 2 * kq + kh * nv + c - 2 * DK;
    for (int j = 0; j < K - 1; ++j) {                  // ascending: row j takes row j + len, which is not yet written
      const int t = len - (K - 1) + j;
      wout[static_cast<long long>(j) * p.C + ch] =
          t >= 0 ? load_f(x + t * p.x_row + ch) : win ? win[static_cast<long long>(K - 1 + t) * p.C + ch] : 0.f;
    }
  }
}

template <typename InT, typename Reqs, int DK, int NS, int KT>
cudaError_t launch_k(const SeqParams& p, const Reqs& reqs, cudaStream_t s) {
  constexpr int TB = sizeof(Reqs) == sizeof(SeqOne) ? 1 : 16;
  const int items = (p.Hv / p.Hk) * (p.dv / NS), CL = items < kMaxCluster ? items : kMaxCluster;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(reqs.n) * p.Hk * CL);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = CL, at[0].val.clusterDim.y = 1, at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, seq_rec_kernel<InT, Reqs, DK, NS, KT, TB>, p, reqs);
}
template <typename InT, typename Reqs, int DK>
cudaError_t launch_n(const SeqParams& p, const Reqs& reqs, cudaStream_t s) {
  if (p.conv_mode == 1 && p.K > 4) return launch_k<InT, Reqs, DK, 32, 8>(p, reqs, s);
  // a quarter of the columns a CTA where whole heads would leave SMs idle
  if (p.dv == 128 && static_cast<long long>(reqs.n) * p.Hv >= 152) return launch_k<InT, Reqs, DK, 128, 4>(p, reqs, s);
  return launch_k<InT, Reqs, DK, 32, 4>(p, reqs, s);
}
template <typename InT, typename Reqs>
cudaError_t launch_d(const SeqParams& p, const Reqs& reqs, cudaStream_t s) {
  if (p.dk == 128) return launch_n<InT, Reqs, 128>(p, reqs, s);
  if (p.dk == 64) return launch_n<InT, Reqs, 64>(p, reqs, s);
  return launch_n<InT, Reqs, 32>(p, reqs, s);
}
template <typename Reqs>
cudaError_t launch_r(const SeqParams& p, const Reqs& reqs, cudaStream_t s) {
  return p.in_dtype == GDN_DTYPE_BF16 ? launch_d<__nv_bfloat16>(p, reqs, s) : launch_d<float>(p, reqs, s);
}

}  // namespace

cudaError_t launch_seq_rec(const SeqParams& p, const SeqReqs* reqs, int n, cudaStream_t s) {
  if (reqs) return launch_r(p, *reqs, s);
  return launch_r(p, SeqOne{n}, s);
}

}  // namespace gdn
