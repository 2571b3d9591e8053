// Single tokens of many requests through one GDN layer: a stream of state tiles.
//
// The states are read and written once, 128 KB a v-head of 128 x 128, and that is the bound.  One CTA an SM walks the
// (request, k-head) pairs; a warp of it keeps the bulk copies going -- a tile on its way in, one being worked on, one on
// its way out -- and the others take each tile through registers and back into its place.  A pair's raw rows and conv
// window come the same way, a pair ahead.  All channels of a k-head's group belong to one CTA, so a window that is written
// in place has been read by then.
//
// Measured (us a call, this kernel : the one of gdn_seq_rec.cu, which the others go to), 16 k-heads and 48 v-heads: 4 requests
// 13.0 : 10.4, 8 15.6 : 18.4, 16 26.6 : 34.8, 32 47 : 66, 128 154 : 246 (5.3 TB/s, 0.78 of measured).  Heads of 64 x 64 gain a
// tenth at 128 requests, heads of 64 x 128 nothing: their tiles are too small for one CTA an SM.  With fp32 rows or many v-heads
// a k-head the rows may leave no room for three tiles.  (At its 168 registers the kernel spills 24 bytes a thread.)
//
// The arithmetic is that of gdn_seq_rec.cu: p = (g T)^T k and r = (g T)^T q in one pass, u = beta (v - p),
// o = r + (q . k) u, T' = g T + k u^T.
#include <cuda_bf16.h>

#include "gdn_seq.cuh"

namespace gdn {
namespace {

constexpr int kWork = 256, kWorkWarps = kWork / 32, kThreads = kWork + 32;
constexpr int kTaps = 4;
constexpr int kSmem = 226 * 1024;

__device__ __forceinline__ float load_f(const float* p) { return __ldg(p); }
__device__ __forceinline__ float load_f(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ float as_f(float x) { return x; }
__device__ __forceinline__ float as_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float silu(float y) { return __fdividef(y, 1.f + __expf(-y)); }
__device__ __forceinline__ void store4(float* p, const float (&v)[4]) {
  *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ void store4(__nv_bfloat16* p, const float (&v)[4]) {
  __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]), b = __floats2bfloat162_rn(v[2], v[3]);
  *reinterpret_cast<uint2*>(p) = make_uint2(*reinterpret_cast<uint32_t*>(&a), *reinterpret_cast<uint32_t*>(&b));
}
__device__ __forceinline__ bool wait_quiet(uint64_t* bar, uint32_t parity) {
  const long long t0 = clock64();
  while (!mbar_ready(bar, parity))
    if (clock64() - t0 > kWaitCycles) return false;
  return true;
}
__device__ __forceinline__ void init_n(uint64_t* bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_addr(bar)), "r"(count) : "memory");
}
__device__ __forceinline__ void bulk_s2g(void* dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(smem_addr(src)), "r"(bytes) : "memory");
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
__device__ __forceinline__ void stores_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }

constexpr int kStagesMost = 8;
struct StepPlan {
  int stages, pairs;       // tiles in shared memory; (request, k-head) pairs
  int row_bytes;           // a pair's raw rows and window in shared memory, twice
};
template <int DK, int DV>
__host__ __device__ constexpr int tile_bytes() { return DK * DV * 4; }
// ys [channels] | part [8][DV] float2 | q.k | barriers, behind the rows and tiles
template <int DV>
__host__ __device__ constexpr int fixed_bytes(int channels) { return channels * 4 + kWorkWarps * DV * 8 + 16 + 8 * (2 * kStagesMost + 4); }

template <typename InT, int DK, int DV>
__global__ void __launch_bounds__(kThreads, 1) seq_step_kernel(const SeqParams p, const StepPlan plan) {
  constexpr int kQuads = DV / 4, kGroups = kWork / kQuads, RPT = DK / kGroups;
  extern __shared__ __align__(128) char sm[];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int R = p.Hv / p.Hk, K = p.conv_mode == 1 ? p.K : 1, nc = 2 * DK + R * DV, kq = p.Hk * DK, stages = plan.stages;
  char* const rows_sm = sm + stages * tile_bytes<DK, DV>();
  float* const ys = reinterpret_cast<float*>(rows_sm + 2 * plan.row_bytes);
  float2* const part = reinterpret_cast<float2*>(ys + nc);
  float* const qk = reinterpret_cast<float*>(part + kWorkWarps * DV);
  uint64_t* const bar = reinterpret_cast<uint64_t*>(qk + 4);
  uint64_t *const full = bar, *const done = bar + kStagesMost, *const rows_full = bar + 2 * kStagesMost, *const rows_done = rows_full + 2;
  const bool aborted = launch_aborted(p.err);
  if (tid == 0) {
    for (int i = 0; i < stages; ++i) init_n(full + i, 1), init_n(done + i, kWorkWarps);
    for (int i = 0; i < 2; ++i) init_n(rows_full + i, 1), init_n(rows_done + i, kWorkWarps);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  if (__syncthreads_or(aborted)) return;
  bool late = false;
  auto wait = [&](uint64_t* b, int n) {                        // for the n-th completion of b
    if (!late && !wait_quiet(b, n & 1)) late = true;
  };
  auto tile = [&](int i) { return reinterpret_cast<float*>(sm + (i % stages) * tile_bytes<DK, DV>()); };
  auto takes_part = [&](int pair) { return !p.live || p.live[pair / p.Hk] != 0; };
  // raw rows in shared memory: q, k, v as they come, then K - 1 window rows of all channels
  auto x_row = [&](int n) { return reinterpret_cast<InT*>(rows_sm + (n & 1) * plan.row_bytes); };
  auto window = [&](int n) { return reinterpret_cast<float*>(rows_sm + (n & 1) * plan.row_bytes + nc * sizeof(InT)); };

  if (warp == kWorkWarps) {
    if (lane == 0) {
      // tile number t of this CTA: head t % R of its pair number t / R
      auto load_rows = [&](int n, int pair) {
        if (n >= 2) wait(rows_done + (n & 1), (n >> 1) - 1);
        if (late) return;
        const int b = pair / p.Hk, kh = pair % p.Hk;
        uint64_t* const f = rows_full + (n & 1);
        const bool win = K > 1 && p.conv_in;
        mbar_expect(f, nc * sizeof(InT) + (win ? (K - 1) * nc * 4 : 0));
        const InT* x = static_cast<const InT*>(p.x) + b * p.x_row;
        bulk_g2s(x_row(n), x + kh * DK, DK * sizeof(InT), f);
        bulk_g2s(x_row(n) + DK, x + kq + kh * DK, DK * sizeof(InT), f);
        bulk_g2s(x_row(n) + 2 * DK, x + 2 * kq + kh * R * DV, R * DV * sizeof(InT), f);
        if (win)
          for (int j = 0; j < K - 1; ++j) {
            const float* w = p.conv_in + b * p.conv_stride + static_cast<long long>(j) * p.C;
            bulk_g2s(window(n) + j * nc, w + kh * DK, DK * 4, f);
            bulk_g2s(window(n) + j * nc + DK, w + kq + kh * DK, DK * 4, f);
            bulk_g2s(window(n) + j * nc + 2 * DK, w + 2 * kq + kh * R * DV, R * DV * 4, f);
          }
      };
      auto offset = [&](int pair, int r) {
        return (pair / p.Hk) * p.state_stride + static_cast<long long>((pair % p.Hk) * R + r) * DK * DV;
      };
      int t = 0, n = 0, ahead = blockIdx.x, n_ahead = 0;       // the tile and pair to load; rows are a pair ahead
      int out_pair = blockIdx.x, out_r = 0, out_t = 0;         // the tile to store next
      auto next_pair = [&](int pair) {
        do pair += gridDim.x;
        while (pair < plan.pairs && !takes_part(pair));
        return pair;
      };
      if (ahead < plan.pairs && !takes_part(ahead)) ahead = next_pair(ahead);
      out_pair = ahead;
      int pair = ahead;
      auto store_one = [&]() {
        wait(done + out_t % stages, out_t / stages);
        if (!late) bulk_s2g(p.state_out + offset(out_pair, out_r), tile(out_t), tile_bytes<DK, DV>());
        ++out_t;
        if (++out_r == R) out_r = 0, out_pair = next_pair(out_pair);
      };
      if (ahead < plan.pairs) load_rows(n_ahead++, ahead), ahead = next_pair(ahead);
      for (; pair < plan.pairs && !late; pair = next_pair(pair), ++n) {
        for (int r = 0; r < R && !late; ++r, ++t) {
          if (t >= stages) stores_read();                      // of tile t - stages
          mbar_expect(full + t % stages, tile_bytes<DK, DV>());
          bulk_g2s(tile(t), p.state_in + offset(pair, r), tile_bytes<DK, DV>(), full + t % stages);
          if (r == 0 && ahead < plan.pairs) load_rows(n_ahead++, ahead), ahead = next_pair(ahead);
          if (t + 1 >= stages) store_one();                    // tile t + 1 - stages
        }
      }
      while (out_t < t && !late) store_one();
      stores_read();
      if (late)                                                // what was in flight has had twice the time
        for (int i = 0; i < 2 * kStagesMost + 4; ++i)
          if (i < stages || (i >= 2 * kStagesMost && i < 2 * kStagesMost + 2)) mbar_wait(bar + i, 0), mbar_wait(bar + i, 1);
      asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    }
    __syncwarp();
  } else {
    auto barrier = [] { asm volatile("bar.sync 1, %0;" ::"n"(kWork) : "memory"); };
    const int c0 = 4 * (tid % kQuads), r0 = (tid / kQuads) * RPT;
    int t = 0, n = 0;
    for (int pair = blockIdx.x; pair < plan.pairs; pair += gridDim.x) {
      if (!takes_part(pair)) continue;
      const int b = pair / p.Hk, kh = pair % p.Hk;
      wait(rows_full + (n & 1), n >> 1);
      const InT* x = x_row(n);
      const float* win = K > 1 && p.conv_in ? window(n) : nullptr;
      for (int c = tid; c < nc; c += kWork) {
        const int ch = c < DK ? kh * DK + c : c < 2 * DK ? kq + kh * DK + c - DK : 2 * kq + kh * R * DV + c - 2 * DK;
        float xr[kTaps], w[kTaps];
#pragma unroll
        for (int j = 0; j < kTaps; ++j) {
          xr[j] = w[j] = 0.f;
          if (j >= kTaps - K) {
            if (j == kTaps - 1) xr[j] = as_f(x[c]);
            else if (win) xr[j] = win[(j - (kTaps - K)) * nc + c];
            w[j] = p.conv_mode == 1 ? __ldg(p.conv_w + static_cast<long long>(ch) * K + j - (kTaps - K)) : 1.f;
          }
        }
        float y = w[kTaps - 1] * xr[kTaps - 1];
#pragma unroll
        for (int i = 1; i < kTaps; ++i) y = fmaf(w[kTaps - 1 - i], xr[kTaps - 1 - i], y);
        if (p.act == 1) y = silu(y);
        ys[c] = y;
        if (K > 1) {
          float* wo = p.conv_out + b * p.conv_stride + ch;
#pragma unroll
          for (int j = 1; j < kTaps; ++j)
            if (j > kTaps - K) wo[static_cast<long long>(j - 1 - (kTaps - K)) * p.C] = xr[j];
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(rows_done + (n & 1));
      ++n;
      barrier();
      if (warp == 0) {                                         // norms and q . k
        float q[DK / 32], k[DK / 32], sq = 0.f, sk = 0.f, d = 0.f;
#pragma unroll
        for (int i = 0; i < DK / 32; ++i) {
          q[i] = ys[lane + 32 * i], k[i] = ys[DK + lane + 32 * i];
          sq = fmaf(q[i], q[i], sq), sk = fmaf(k[i], k[i], sk);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sq += __shfl_xor_sync(~0u, sq, o), sk += __shfl_xor_sync(~0u, sk, o);
        const float nq = rsqrtf(sq + p.l2_eps) * p.q_scale, nk = rsqrtf(sk + p.l2_eps);
#pragma unroll
        for (int i = 0; i < DK / 32; ++i) {
          q[i] *= nq, k[i] *= nk;
          d = fmaf(q[i], k[i], d);
          ys[lane + 32 * i] = q[i], ys[DK + lane + 32 * i] = k[i];
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) d += __shfl_xor_sync(~0u, d, o);
        if (lane == 0) *qk = d;
      }
      barrier();
      const float dot = *qk;
      float kr[RPT], qr[RPT];
#pragma unroll
      for (int i = 0; i < RPT; ++i) qr[i] = ys[r0 + i], kr[i] = ys[DK + r0 + i];
      for (int r = 0; r < R; ++r, ++t) {
        const int h = kh * R + r;
        const long long gate = b * p.gate_row + h;
        const float beta = load_f(static_cast<const InT*>(p.beta) + gate), g = expf(load_f(static_cast<const InT*>(p.log_g) + gate));
        const float4 v = *reinterpret_cast<const float4*>(ys + 2 * DK + r * DV + c0);
        wait(full + t % stages, t / stages);
        float* const T0 = tile(t) + r0 * DV + c0;
        float T[RPT][4], pk[4] = {0.f, 0.f, 0.f, 0.f}, pq[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < RPT; ++i) {
          const float4 f = *reinterpret_cast<const float4*>(T0 + i * DV);
          T[i][0] = f.x * g, T[i][1] = f.y * g, T[i][2] = f.z * g, T[i][3] = f.w * g;
#pragma unroll
          for (int c = 0; c < 4; ++c) pk[c] = fmaf(kr[i], T[i][c], pk[c]), pq[c] = fmaf(qr[i], T[i][c], pq[c]);
        }
#pragma unroll
        for (int o = kQuads; o < 32; o <<= 1)
#pragma unroll
          for (int c = 0; c < 4; ++c) pk[c] += __shfl_xor_sync(~0u, pk[c], o), pq[c] += __shfl_xor_sync(~0u, pq[c], o);
        if (lane < kQuads) {
          float4* dst = reinterpret_cast<float4*>(part + warp * DV + c0);
          dst[0] = make_float4(pk[0], pq[0], pk[1], pq[1]);
          dst[1] = make_float4(pk[2], pq[2], pk[3], pq[3]);
        }
        barrier();
        float sk[4] = {0.f, 0.f, 0.f, 0.f}, sq[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int w = 0; w < kWorkWarps; ++w) {
          const float4* src = reinterpret_cast<const float4*>(part + w * DV + c0);
          const float4 a = src[0], e = src[1];
          sk[0] += a.x, sq[0] += a.y, sk[1] += a.z, sq[1] += a.w;
          sk[2] += e.x, sq[2] += e.y, sk[3] += e.z, sq[3] += e.w;
        }
        const float u[4] = {beta * (v.x - sk[0]), beta * (v.y - sk[1]), beta * (v.z - sk[2]), beta * (v.w - sk[3])};
#pragma unroll
        for (int i = 0; i < RPT; ++i)
          *reinterpret_cast<float4*>(T0 + i * DV) = make_float4(fmaf(kr[i], u[0], T[i][0]), fmaf(kr[i], u[1], T[i][1]),
                                                                fmaf(kr[i], u[2], T[i][2]), fmaf(kr[i], u[3], T[i][3]));
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) mbar_arrive(done + t % stages);
        if (tid < kQuads) {
          const float o[4] = {fmaf(dot, u[0], sq[0]), fmaf(dot, u[1], sq[1]), fmaf(dot, u[2], sq[2]), fmaf(dot, u[3], sq[3])};
          const long long at = (static_cast<long long>(b) * p.Hv + h) * DV + c0;
          if (p.out_dtype == GDN_DTYPE_BF16) store4(static_cast<__nv_bfloat16*>(p.out) + at, o);
          else store4(static_cast<float*>(p.out) + at, o);
        }
        barrier();                                             // part and, after the last head, ys are written again
      }
    }
  }
  if (__syncthreads_or(late) && tid == 0) device_error(p.err, GDN_DEVERR_TIMEOUT, 0);
}

template <typename InT, int DK, int DV>
cudaError_t launch_t(const SeqParams& p, const StepPlan& plan, int smem, int ctas, cudaStream_t s) {
  auto k = seq_step_kernel<InT, DK, DV>;
  const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  k<<<ctas, kThreads, smem, s>>>(p, plan);
  return cudaGetLastError();
}
}  // namespace

bool launch_seq_step(const SeqParams& p, int n, cudaStream_t s, cudaError_t& e) {
  constexpr int kTile = tile_bytes<128, 128>();
  const long long pairs = static_cast<long long>(n) * p.Hk;
  if (p.dk != 128 || p.dv != 128 || (p.conv_mode == 1 && p.K > kTaps) || !p.state_in || static_cast<long long>(n) * p.Hv < 304)
    return false;
  const int nc = 2 * p.dk + p.Hv / p.Hk * p.dv, in = p.in_dtype == GDN_DTYPE_BF16 ? 2 : 4;
  StepPlan plan{};
  plan.pairs = static_cast<int>(pairs);
  plan.row_bytes = nc * (in + 4 * (kTaps - 1));
  const int rest = 2 * plan.row_bytes + fixed_bytes<128>(nc);
  plan.stages = (kSmem - rest) / kTile < kStagesMost ? (kSmem - rest) / kTile : kStagesMost;
  if (rest > kSmem || plan.stages < 3) return false;
  const int smem = plan.stages * kTile + rest, ctas = pairs < 152 ? static_cast<int>(pairs) : 152;
  e = p.in_dtype == GDN_DTYPE_BF16 ? launch_t<__nv_bfloat16, 128, 128>(p, plan, smem, ctas, s)
                                   : launch_t<float, 128, 128>(p, plan, smem, ctas, s);
  return true;
}

}  // namespace gdn
