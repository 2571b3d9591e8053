// Prompts through one GDN layer in chunks of 64 tokens, on tcgen05.
//
// With c_i the cumulated log gates of a chunk, rows k_i, q_i, v_i and the state T before it:
//   A = (beta_i e^(c_i - c_j) k_i.k_j)_{j < i},   M = (1 + A)^-1 diag(beta),   N = (e^(c_i - c_j) q_i.k_j)_{j <= i} M,
//   w_i = v_i - e^(c_i) T^T k_i,   u = M w,   o_i = e^(c_i) T^T q_i + (N w)_i,
//   T' = e^(c_63) T + sum_i k_i (e^(c_63 - c_i) u_i)^T.
// Everything in the first line is independent of T: seq_prepare_kernel computes it for many chunks at once, with the conv,
// the activation and the norms.  seq_chain_kernel then walks each head's chunks:
//   D1 = [K; Q] T   ->   w   ->   D2 = [M; N] w   ->   u, o   ->   D3 = K^T u   ->   T'
// with T in fp32 in registers, a row of d_k and 32 columns a thread.  Columns of d_v do not depend on each other.
//
// Precision: operands enter the products as two fp16 terms, x = hi + lo, and hi hi + hi lo + lo hi is accumulated in fp32:
// 22 bits of every element, half the tensor-core time of a tf32 split in three.  fp16's range is met by powers of two: k
// and q are normalised (2^12), M, N and T scaled by their largest entry, w and u by bounds that follow from those of T
// and v:  |w| <= max v + max e^c sqrt(dk) max T,  |u| <= max_i sum_j |M_ij| max w.  An element keeps 2^-23 of itself or
// 2^-40 of the bound, and the bounds lie some 2^6 above the values.  Where they lie 2^17 above the largest entry of T' or of
// the chunk's o (values that shrink or grow by that much within 64 tokens), the chunk is taken again token by token.
//
// Operands in shared memory have no swizzle: 8 rows x 16 bytes are 128 contiguous bytes.  With 16 bytes of d_k per
// token, a core matrix of K serves as K-major operand of D1 and as M-major operand of D3.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "gdn_seq.cuh"
#include "gdn_umma.cuh"

namespace gdn {
namespace {

constexpr float kUnit = 4096.f;            // scale of k and q
constexpr float kGateFloor = -1.0e4f;      // e to this is 0; keeps differences of sums finite
constexpr float kLog2e = 1.4426950408889634f;

// ---- operands ----
__host__ __device__ constexpr uint32_t idesc_f16(int n, bool a_mn, bool b_mn) {   // M = 128, fp32 accumulator
  return (1u << 4) | (a_mn ? 1u << 15 : 0u) | (b_mn ? 1u << 16 : 0u) | (static_cast<uint32_t>(n >> 3) << 17) | (8u << 24);
}
__device__ __forceinline__ void umma_f16_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, int accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
// D = A B in two-term operands, K elements deep: `steps` instructions of 16 each, three times.  Descriptors of the high
// terms; the low ones lie a_lo and b_lo bytes behind.  a_step, b_step: bytes from one instruction's operands to the next.
template <int kSteps>
__device__ __forceinline__ void product(uint32_t d, uint64_t a, uint64_t b, uint32_t a_lo, uint32_t b_lo, uint32_t a_step,
                                        uint32_t b_step, uint32_t idesc) {
  const uint64_t al = a_lo >> 4, bl = b_lo >> 4, as = a_step >> 4, bs = b_step >> 4;
#pragma unroll
  for (int i = 0; i < kSteps; ++i) umma_f16_ss(d, a + i * as, b + i * bs, idesc, i > 0);
#pragma unroll
  for (int i = 0; i < kSteps; ++i) umma_f16_ss(d, a + i * as, b + bl + i * bs, idesc, 1);
#pragma unroll
  for (int i = 0; i < kSteps; ++i) umma_f16_ss(d, a + al + i * as, b + i * bs, idesc, 1);
}
// Two values as fp16 pairs of their high and low terms.
__device__ __forceinline__ void split2(float x, float y, uint32_t& hi, uint32_t& lo) {
  const __half2 h = __floats2half2_rn(x, y);
  const float2 f = __half22float2(h);
  const __half2 l = __floats2half2_rn(x - f.x, y - f.y);
  hi = *reinterpret_cast<const uint32_t*>(&h);
  lo = *reinterpret_cast<const uint32_t*>(&l);
}
__device__ __forceinline__ void split8(const float* x, uint4& hi, uint4& lo) {
  split2(x[0], x[1], hi.x, lo.x);
  split2(x[2], x[3], hi.y, lo.y);
  split2(x[4], x[5], hi.z, lo.z);
  split2(x[6], x[7], hi.w, lo.w);
}
// The power of two that brings values up to `bound` below 2^15, and its inverse.
__device__ __forceinline__ float scale_for(float bound, float& inverse) {
  const int e = static_cast<int>(__float_as_uint(bound) >> 23 & 0xFF);     // bound < 2^(e - 126)
  const int f = min(max(127 + 14 + 126 - e, 2), 252);
  inverse = __uint_as_float(static_cast<uint32_t>(254 - f) << 23);
  return __uint_as_float(static_cast<uint32_t>(f) << 23);
}
__device__ __forceinline__ float warp_max(float x) {     // x >= 0 (or NaN, which counts as larger than all)
  return __uint_as_float(__reduce_max_sync(~0u, __float_as_uint(x)));
}
__device__ __forceinline__ float abs_bits_max(float a, float b) {
  return __uint_as_float(max(__float_as_uint(a), __float_as_uint(b) & 0x7FFFFFFFu));
}
__device__ __forceinline__ void mbar_init_n(uint64_t* bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_addr(bar)), "r"(count) : "memory");
}

// ---- loads of raw rows ----
__device__ __forceinline__ float4 raw4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ float4 raw4(const __nv_bfloat16* p) {
  const uint2 u = *reinterpret_cast<const uint2*>(p);
  return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xFFFF0000u), __uint_as_float(u.y << 16),
                     __uint_as_float(u.y & 0xFFFF0000u));
}
__device__ __forceinline__ float load_f(const float* p) { return __ldg(p); }
__device__ __forceinline__ float load_f(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ float silu(float y) { return __fdividef(y, 1.f + __expf(-y)); }

// Conv and activation of four channels (the first is ch) for kTok tokens from t0 of a request; zeros past its end.
template <typename InT, int KT, int kTok>
__device__ __forceinline__ void conv_tokens(const SeqParams& p, const InT* x, const float* win, int t0, int len, int ch,
                                            float4 (&y)[kTok]) {
  float4 r[kTok + KT - 1], w[KT];
  const int K = p.K;
#pragma unroll
  for (int i = 0; i < kTok + KT - 1; ++i) {
    const int t = t0 + i - (KT - 1);
    r[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (i >= KT - K && t < len) {
      if (t >= 0) r[i] = raw4(x + t * p.x_row + ch);
      else if (win) r[i] = raw4(win + static_cast<long long>(K - 1 + t) * p.C + ch);
    }
  }
#pragma unroll
  for (int j = 0; j < KT; ++j) {
    w[j] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (j >= KT - K) {
      if (p.conv_mode == 1) {
        const float* cw = p.conv_w + static_cast<long long>(ch) * K + j - (KT - K);
        w[j] = make_float4(__ldg(cw), __ldg(cw + K), __ldg(cw + 2 * K), __ldg(cw + 3 * K));
      } else {
        w[j] = make_float4(1.f, 1.f, 1.f, 1.f);
      }
    }
  }
#pragma unroll
  for (int t = 0; t < kTok; ++t) {
    float4 a = r[t + KT - 1];
    a = make_float4(w[KT - 1].x * a.x, w[KT - 1].y * a.y, w[KT - 1].z * a.z, w[KT - 1].w * a.w);
#pragma unroll
    for (int i = 1; i < KT; ++i) {
      const float4 b = r[t + KT - 1 - i], c = w[KT - 1 - i];
      a = make_float4(fmaf(c.x, b.x, a.x), fmaf(c.y, b.y, a.y), fmaf(c.z, b.z, a.z), fmaf(c.w, b.w, a.w));
    }
    if (p.act == 1) a = make_float4(silu(a.x), silu(a.y), silu(a.z), silu(a.w));
    if (t0 + t >= len) a = make_float4(0.f, 0.f, 0.f, 0.f);
    y[t] = a;
  }
}

// ---- what does not depend on the state ------------------------------------------------------------------------------

constexpr int kPrepThreads = 256, kPrepWarps = kPrepThreads / 32;
constexpr int kLd = 68;                    // floats a row of the 64-wide matrices

template <int DK>
struct Prep {
  static constexpr int kImage = kChunk * DK * 2;              // one fp16 image of K or Q
  static constexpr int kYLd = DK + 4;
  // G and H (128 rows), in the place of the rows of q or k before the split
  static constexpr int kGram = 0;
  static constexpr int kGramBytes = 128 * kLd * 4;
  static_assert(kChunk * kYLd * 4 <= kGramBytes, "rows fit the Gram matrices' place");
  // Kh Qh Kl Ql; after the Gram product A, X, C (hi, lo), M (hi, lo)
  static constexpr int kImages = kGram + kGramBytes;
  static constexpr int kA = kImages, kX = kA + kChunk * kLd * 4;
  static constexpr int kSq = kChunk * kChunk * 2;             // an fp16 image of a 64 x 64 matrix
  static constexpr int kC = kX + kChunk * kLd * 4, kM = kC + 2 * kSq;
  static constexpr int kEnd = (kImages + 4 * kImage > kM + 2 * kSq ? kImages + 4 * kImage : kM + 2 * kSq);   // (C is read as 128 rows: its lower terms and M lie behind)
  static constexpr int kGate = kEnd;                          // float [64] x { beta, c hi, c lo }
  static constexpr int kRed = kGate + 3 * kChunk * 4;         // float [64]
  static constexpr int kBar = kRed + 64 * 4;
  static constexpr int kTotal = kBar + 64;
};

// 16-byte places of an fp16 image of `width` columns: row r, columns 8 c ..
__device__ __forceinline__ int image_at(int r, int c, int width) { return (r >> 3) * width * 16 + c * 128 + (r & 7) * 16; }

template <typename InT, int DK, int KT>
__global__ void __launch_bounds__(kPrepThreads, 2)
seq_prepare_kernel(const SeqParams p, const __grid_constant__ Segment seg, char* ws) {
  using P = Prep<DK>;
  extern __shared__ __align__(128) char sm[];
  float* gram = reinterpret_cast<float*>(sm + P::kGram);
  float* A = reinterpret_cast<float*>(sm + P::kA);
  float* X = reinterpret_cast<float*>(sm + P::kX);
  float* gate = reinterpret_cast<float*>(sm + P::kGate);
  float* red = reinterpret_cast<float*>(sm + P::kRed);
  uint64_t* bar = reinterpret_cast<uint64_t*>(sm + P::kBar);
  uint32_t* tmem_at = reinterpret_cast<uint32_t*>(bar + 1);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int kh = blockIdx.x, slot = blockIdx.y;
  int ri = 0;
  while (ri + 1 < seg.n && slot >= seg.r[ri + 1].slot0) ++ri;
  const SegReq req = seg.r[ri];
  const int chunk = req.c0 + slot - req.slot0, t0 = chunk * kChunk, len = req.len;
  const int R = p.Hv / p.Hk, dv = p.dv;
  const InT* x = static_cast<const InT*>(p.x) + static_cast<long long>(req.start) * p.x_row;
  const float* win = p.conv_in ? p.conv_in + req.b * p.conv_stride : nullptr;
  char* const slot_ws = ws + slot * (p.Hk * seq_kq_bytes(DK) + p.Hv * seq_v_bytes(dv));
  char* const kq_ws = slot_ws + kh * seq_kq_bytes(DK);
  const bool aborted = launch_aborted(p.err);

  if (warp == 0) tmem_alloc(tmem_at, 128);
  if (tid == 0) mbar_init(bar);
  if (__syncthreads_or(aborted)) {
    if (warp == 0) {
      tmem_relinquish();
      tmem_dealloc(*tmem_at, 128);
    }
    return;
  }
  if (warp == 0) tmem_relinquish();
  const uint32_t tmem = *tmem_at;
  int phase = 0;
  bool late = false;

  // q and k: conv, activation, norm; then the two-term images, here and in the workspace
  constexpr int kLanes = DK / 4, kRowsWarp = 32 / kLanes, kTok = 8 / kRowsWarp;   // lanes a token, tokens at once and in turn
#pragma unroll 1
  for (int kind = 1; kind >= 0; --kind) {          // 1: k, 0: q
    {
      const int tl = warp * 8 + (lane / kLanes) * kTok, cl = (lane % kLanes) * 4;
      float4 y[kTok];
      conv_tokens<InT, KT, kTok>(p, x, win, t0 + tl, len, kind * p.Hk * DK + kh * DK + cl, y);
#pragma unroll
      for (int t = 0; t < kTok; ++t) {
        float ss = fmaf(y[t].x, y[t].x, fmaf(y[t].y, y[t].y, fmaf(y[t].z, y[t].z, y[t].w * y[t].w)));
#pragma unroll
        for (int o = kLanes / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(~0u, ss, o);
        const float f = t0 + tl + t < len ? rsqrtf(ss + p.l2_eps) * kUnit : 0.f;
        *reinterpret_cast<float4*>(gram + (tl + t) * P::kYLd + cl) = make_float4(y[t].x * f, y[t].y * f, y[t].z * f, y[t].w * f);
      }
    }
    __syncthreads();
    const int t = tid & 63;
    char* const hi_sm = sm + P::kImages + (kind ? 0 : 1) * P::kImage;
    char* const hi_ws = kq_ws + (kind ? 0 : 2) * P::kImage;
    for (int c = tid >> 6; c < DK / 8; c += kPrepThreads / 64) {
      uint4 hi, lo;
      split8(gram + t * P::kYLd + 8 * c, hi, lo);
      const int at = image_at(t, c, DK);
      *reinterpret_cast<uint4*>(hi_sm + at) = hi;
      *reinterpret_cast<uint4*>(hi_sm + 2 * P::kImage + at) = lo;
      *reinterpret_cast<uint4*>(hi_ws + at) = hi;
      *reinterpret_cast<uint4*>(hi_ws + P::kImage + at) = lo;
    }
    fence_proxy_async();
    __syncthreads();
  }

  // G = K K^T (lanes 0 to 63) and H = Q K^T
  if (tid == 0) {
    const uint64_t a = umma_desc(smem_addr(sm + P::kImages), 128, DK * 16);
    product<DK / 16>(tmem, a, a, 2 * P::kImage, 2 * P::kImage, 256, 256, idesc_f16(kChunk, false, false));
    umma_commit(bar);
  }
  // meanwhile the values
  for (int h = 0; h < R; ++h) {
    // a lane takes four channels of four adjacent tokens, twice where a row takes the whole warp
    const int vh = kh * R + h, lanes = dv / 4, sub = lane / lanes, cl = (lane % lanes) * 4;
    char* const v_ws = slot_ws + p.Hk * seq_kq_bytes(DK) + vh * seq_v_bytes(dv);
    float* const V = reinterpret_cast<float*>(v_ws + 4 * 128 * kChunk);
    float most = 0.f;
    for (int t = 4 * sub; t < 8; t += lanes == 32 ? 4 : 8) {
      const int first = warp * 8 + t;
      float4 y[4];
      conv_tokens<InT, KT, 4>(p, x, win, t0 + first, len, 2 * p.Hk * DK + vh * dv + cl, y);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        *reinterpret_cast<float4*>(V + (first + i) * dv + cl) = y[i];
        most = abs_bits_max(abs_bits_max(abs_bits_max(abs_bits_max(most, y[i].x), y[i].y), y[i].z), y[i].w);
      }
    }
    __syncwarp();
    most = warp_max(most);
    if (lane == 0) red[(h & 3) * kPrepWarps + warp] = most;
    __syncthreads();
    if (tid == 0) {
      most = 0.f;
      for (int w = 0; w < kPrepWarps; ++w) most = abs_bits_max(most, red[(h & 3) * kPrepWarps + w]);
      reinterpret_cast<float*>(v_ws + 4 * 128 * kChunk + kChunk * dv * 4)[2 * kChunk + 3] = most;
    }
  }
  if (!late && !mbar_wait(bar, phase & 1)) late = true;
  ++phase;
  tmem_fence_after();
  const int trow = (warp & 3) * 32 + lane, tcol = (warp >> 2) * 32;
  const uint32_t ta = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
  {
    float v[16];
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      tmem_ld16(ta + tcol + 16 * half, v);
      tmem_wait_ld();
#pragma unroll
      for (int i = 0; i < 16; i += 4)
        *reinterpret_cast<float4*>(gram + trow * kLd + tcol + 16 * half + i) =
            make_float4(v[i] * (1.f / (kUnit * kUnit)), v[i + 1] * (1.f / (kUnit * kUnit)), v[i + 2] * (1.f / (kUnit * kUnit)),
                        v[i + 3] * (1.f / (kUnit * kUnit)));
    }
  }

#pragma unroll 1
  for (int h = 0; h < R; ++h) {
    const int vh = kh * R + h;
    char* const v_ws = slot_ws + p.Hk * seq_kq_bytes(DK) + vh * seq_v_bytes(dv);
    float* const meta = reinterpret_cast<float*>(v_ws + 4 * 128 * kChunk + kChunk * dv * 4);
    __syncthreads();                               // the head before is done with gates and matrices; the Gram matrices are there
    // gates: cumulated in 64 bits, kept as two floats
    if (warp == 0) {
      double c[2];
      float rise = 0.f;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int t = t0 + 2 * lane + i;
        float g = 0.f, b = 0.f;
        if (t < len) {
          const long long at = (req.start + static_cast<long long>(t)) * p.gate_row + vh;
          b = load_f(static_cast<const InT*>(p.beta) + at);
          g = load_f(static_cast<const InT*>(p.log_g) + at);
          g = g < kGateFloor ? kGateFloor : g;
        }
        rise += fmaxf(g, 0.f);
        c[i] = g;
        gate[2 * lane + i] = b;
      }
      c[1] += c[0];
      double sum = c[1];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const double s = __shfl_up_sync(~0u, sum, o);
        if (lane >= o) sum += s;
      }
      const double before = sum - c[1], total = __shfl_sync(~0u, sum, 31);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) rise += __shfl_xor_sync(~0u, rise, o);
      float most = 0.f;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const double s = before + c[i];
        const float hi = static_cast<float>(s), first = expf(hi) * (1.f + static_cast<float>(s - hi));
        const float left = expf(static_cast<float>(total - s));
        gate[kChunk + 2 * lane + i] = hi;
        gate[2 * kChunk + 2 * lane + i] = static_cast<float>(s - hi);
        meta[2 * lane + i] = first;
        meta[kChunk + 2 * lane + i] = left;
        red[2 * lane + i] = left;
        most = fmaxf(most, first);
      }
      most = warp_max(most);
      if (lane == 31) {
        meta[2 * kChunk] = expf(static_cast<float>(total));
        meta[2 * kChunk + 5] = most;
      }
      // no product of gates is above e^rise (1 unless a log gate is above 0): C's scale
      if (lane == 0) reinterpret_cast<float*>(bar)[4] = exp2f(floorf(11.f - rise * kLog2e));
    }
    __syncthreads();
    const float unit = reinterpret_cast<float*>(bar)[4];
    // A = beta_i e^(c_i - c_j) G_ij below the diagonal;  C = e^(c_i - c_j) H_ij up to it, as two-term image
    {
      const int i = tid >> 2, j0 = (tid & 3) * 16;
      const float ci = gate[kChunk + i], di = gate[2 * kChunk + i], bi = gate[i];
#pragma unroll
      for (int jj = 0; jj < 16; jj += 8) {
        float c[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int j = j0 + jj + k;
          const float e = j <= i ? expf((ci - gate[kChunk + j]) + (di - gate[2 * kChunk + j])) : 0.f;
          A[i * kLd + j] = j < i ? bi * e * gram[i * kLd + j] : 0.f;
          c[k] = j <= i ? e * gram[(kChunk + i) * kLd + j] * unit : 0.f;
        }
        uint4 hi, lo;
        split8(c, hi, lo);
        const int at = image_at(i, (j0 + jj) >> 3, kChunk);
        *reinterpret_cast<uint4*>(sm + P::kC + at) = hi;
        *reinterpret_cast<uint4*>(sm + P::kC + P::kSq + at) = lo;
      }
    }
    __syncthreads();
    // X = (1 + A)^-1: diagonal blocks of 16 by substitution, then of 32 and 64 by products
    {
      const int blk = warp >> 1, j = lane & 15, r0 = blk * 16;
      if ((warp & 1) == 0 && lane < 16) {
        float xc[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          float s = i == j ? 1.f : 0.f;
#pragma unroll
          for (int k = 0; k < 16; ++k)
            if (k < i) s = fmaf(-A[(r0 + i) * kLd + r0 + k], xc[k], s);
          xc[i] = s;
          X[(r0 + i) * kLd + r0 + j] = s;
        }
      }
    }
    __syncthreads();
#pragma unroll 1
    for (int n = 16; n <= 32; n *= 2) {
      // for each pair of diagonal blocks: X21 = -X22 (A21 X11); the inner product is kept in X21's mirror place
      const int per = n * n, pairs = kChunk / (2 * n);
      float s[4];
      for (int pass = 0; pass < 2; ++pass) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int idx = tid + e * kPrepThreads;
          s[e] = 0.f;
          if (idx < pairs * per) {
            const int b = idx / per * 2 * n, i = idx % per / n, j = idx % n;
            float a = 0.f;
            if (pass == 0) {
              for (int k = j & ~3; k < n; ++k) a = fmaf(A[(b + n + i) * kLd + b + k], X[(b + k) * kLd + b + j] * (k >= j ? 1.f : 0.f), a);
            } else {
              for (int k = 0; k <= i; ++k) a = fmaf(X[(b + n + i) * kLd + b + n + k], X[(b + k) * kLd + b + n + j], a);
              a = -a;
            }
            s[e] = a;
          }
        }
        __syncthreads();
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int idx = tid + e * kPrepThreads;
          if (idx < pairs * per) {
            const int b = idx / per * 2 * n, i = idx % per / n, j = idx % n;
            if (pass == 0) X[(b + i) * kLd + b + n + j] = s[e];
            else X[(b + n + i) * kLd + b + j] = s[e];
          }
        }
        __syncthreads();
      }
    }
    // M = X diag(beta): its largest entry, its largest row sum times the gates behind it, its image
    const int i = tid >> 2, j0 = (tid & 3) * 16;
    float m[16], big = 0.f, row = 0.f;
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      const int j = j0 + k;
      m[k] = j <= i ? X[i * kLd + j] * gate[j] : 0.f;
      big = abs_bits_max(big, m[k]);
      row += fabsf(m[k]);
    }
    row += __shfl_xor_sync(~0u, row, 1);
    row += __shfl_xor_sync(~0u, row, 2);
    row *= red[i];
    big = warp_max(big);
    row = warp_max(row);
    __syncthreads();
    if (lane == 0) red[warp] = big, red[kPrepWarps + warp] = row;
    __syncthreads();
    big = row = 0.f;
#pragma unroll
    for (int w = 0; w < kPrepWarps; ++w) big = abs_bits_max(big, red[w]), row = abs_bits_max(row, red[kPrepWarps + w]);
    float inv_m;
    const float sc_m = scale_for(big, inv_m);
    // rows of [M; N] change places with every chunk of the request, as those of [K; Q] do
    const int m_row = (chunk & 1) * kChunk, n_row = kChunk - m_row;
#pragma unroll
    for (int k = 0; k < 16; ++k) m[k] *= sc_m;
#pragma unroll
    for (int k = 0; k < 16; k += 8) {
      uint4 hi, lo;
      split8(m + k, hi, lo);
      const int at = image_at(i, (j0 + k) >> 3, kChunk);
      *reinterpret_cast<uint4*>(sm + P::kM + at) = hi;
      *reinterpret_cast<uint4*>(sm + P::kM + P::kSq + at) = lo;
      *reinterpret_cast<uint4*>(v_ws + m_row * 128 + at) = hi;
      *reinterpret_cast<uint4*>(v_ws + 128 * 128 + m_row * 128 + at) = lo;
    }
    fence_proxy_async();
    __syncthreads();
    // N = C M
    if (tid == 0) {
      tmem_fence_after();
      product<kChunk / 16>(tmem + 64, umma_desc(smem_addr(sm + P::kC), 128, 1024), umma_desc(smem_addr(sm + P::kM), 1024, 128),
                           P::kSq, P::kSq, 256, 2048, idesc_f16(kChunk, false, true));
      umma_commit(bar);
    }
    if (!late && !mbar_wait(bar, phase & 1)) late = true;
    ++phase;
    tmem_fence_after();
    const bool mine = (warp & 3) < 2;              // N is in lanes 0 to 63
    float v[32];
    tmem_ld16(ta + 64 + tcol, *reinterpret_cast<float(*)[16]>(v));
    tmem_ld16(ta + 64 + tcol + 16, *reinterpret_cast<float(*)[16]>(v + 16));
    tmem_wait_ld();
    tmem_fence_before();
    big = 0.f;
    float row_n = 0.f;
    const float back = inv_m / unit;
#pragma unroll
    for (int k = 0; k < 32; ++k) {
      v[k] *= back;
      big = abs_bits_max(big, v[k]);
      row_n += fabsf(v[k]);
    }
    big = warp_max(big);
    row_n = warp_max(row_n);
    if (lane == 0) red[2 * kPrepWarps + warp] = mine ? big : 0.f, red[3 * kPrepWarps + warp] = mine ? row_n : 0.f;
    __syncthreads();
    big = 0.f;
    float half[2] = {0.f, 0.f};                    // the rows' halves lie in two warps
#pragma unroll
    for (int w = 0; w < kPrepWarps; ++w) {
      big = abs_bits_max(big, red[2 * kPrepWarps + w]);
      half[w >> 2] = abs_bits_max(half[w >> 2], red[3 * kPrepWarps + w]);
    }
    float inv_n;
    const float sc_n = scale_for(big, inv_n);
    if (mine) {
#pragma unroll
      for (int k = 0; k < 32; ++k) v[k] *= sc_n;
#pragma unroll
      for (int k = 0; k < 32; k += 8) {
        uint4 hi, lo;
        split8(v + k, hi, lo);
        const int at = image_at(trow, (tcol + k) >> 3, kChunk);
        *reinterpret_cast<uint4*>(v_ws + n_row * 128 + at) = hi;
        *reinterpret_cast<uint4*>(v_ws + 128 * 128 + n_row * 128 + at) = lo;
      }
    }
    if (tid == 0) {
      meta[2 * kChunk + 1] = inv_m;
      meta[2 * kChunk + 2] = inv_n;
      meta[2 * kChunk + 4] = row;
      meta[2 * kChunk + 6] = half[0] + half[1];
    }
  }
  if (__syncthreads_or(late) && tid == 0) device_error(p.err, GDN_DEVERR_TIMEOUT, req.b);
  if (warp == 0) tmem_dealloc(tmem, 128);
}

// ---- the chunks of a head, one after another ------------------------------------------------------------------------

template <int DK, int NB>
struct Chain {
  static constexpr int kGroups = NB / 32;                      // warpgroups, 32 columns each
  static constexpr int kSoft = 128 * kGroups, kThreads = kSoft + 32;
  static constexpr int kImage = kChunk * DK * 2;               // K or Q, one term
  static constexpr int kKq = 0, kKqLo = 3 * kImage;            // K of even chunks | Q | K of odd chunks
  static constexpr int kMn = 6 * kImage, kMnLo = 128 * kChunk * 2;
  static constexpr int kS = kMn + 2 * kMnLo, kSLo = DK * NB * 2;
  static constexpr int kW = kS + 2 * kSLo, kWLo = kChunk * NB * 2;
  static constexpr int kBar = kW + 2 * kWLo;
  static constexpr int kMax = kBar + 8 * 10;                   // float [2][4 kGroups]: largest entries of T, of o
  // K^T is read as 128 rows of d_k: from its last core matrices up to 1536 bytes past the image, into the next place
  static constexpr int kTotal = kMax + 2 * 4 * kGroups * 4;
  static constexpr uint32_t kCols = 3 * NB <= 128 ? 128 : 3 * NB <= 256 ? 256 : 512;
};
enum ChainBar { kKqFull, kMnFull, kSReady, kD1, kWReady, kD2, kUReady, kD3, kTmemAt };

constexpr float kRange = 0x1p-17f;   // bounds this far above the largest value still leave 2^-22 of it

// A chunk by the rule itself, with fp32 sums, from the state in its operand (S / scale, 22 bits): its outputs are written
// again and S is the state after it.  All threads of the warpgroups; rare and slow (some 0.1 ms).
template <int DK, int NB>
__device__ __noinline__ void again_by_token(const SeqParams& p, const SegReq& req, int vh, int row, bool has_row, int c0,
                                            int col0, int t0, float inv_s, const char* kq, const float* V, char* sm,
                                            float (&S)[32]) {
  using L = Chain<DK, NB>;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  auto barrier = [] { asm volatile("bar.sync 1, %0;" ::"n"(L::kSoft) : "memory"); };
  auto term = [](const char* at) { return __half2float(*reinterpret_cast<const __half*>(at)); };
  float* const part = reinterpret_cast<float*>(sm + L::kW);     // [warps][p, r: 32 each] and [warps] q.k
  float* const dots = part + 4 * L::kGroups * 64;
#pragma unroll
  for (int j = 0; j < 32; ++j) {
    const char* at = sm + L::kS + ((c0 + j) >> 3) * DK * 16 + row * 16 + (j & 7) * 2;
    S[j] = has_row ? (term(at) + term(at + L::kSLo)) * inv_s : 0.f;
  }
  for (int t = 0; t < kChunk && t0 + t < req.len; ++t) {
    const long long gate = (req.start + static_cast<long long>(t0 + t)) * p.gate_row + vh;
    const bool bf16 = p.in_dtype == GDN_DTYPE_BF16;
    const float beta = bf16 ? load_f(static_cast<const __nv_bfloat16*>(p.beta) + gate) : load_f(static_cast<const float*>(p.beta) + gate);
    const float g = expf(bf16 ? load_f(static_cast<const __nv_bfloat16*>(p.log_g) + gate) : load_f(static_cast<const float*>(p.log_g) + gate));
    float k = 0.f, q = 0.f;
    if (has_row) {
      const char* at = kq + image_at(t, row >> 3, DK) + (row & 7) * 2;
      k = (term(at) + term(at + L::kImage)) * (1.f / kUnit);
      q = (term(at + 2 * L::kImage) + term(at + 3 * L::kImage)) * (1.f / kUnit);
    }
    float mine_p = 0.f, mine_r = 0.f, qk = k * q;
#pragma unroll
    for (int j = 0; j < 32; ++j) {
      S[j] *= g;
      float a = k * S[j], b = q * S[j];
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) a += __shfl_xor_sync(~0u, a, o), b += __shfl_xor_sync(~0u, b, o);
      if (lane == j) mine_p = a, mine_r = b;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) qk += __shfl_xor_sync(~0u, qk, o);
    part[warp * 64 + lane] = mine_p;
    part[warp * 64 + 32 + lane] = mine_r;
    if (lane == 0) dots[warp] = qk;
    barrier();
    const float* mine = part + (warp & ~3) * 64;
    qk = (dots[0] + dots[1]) + (dots[2] + dots[3]);
    const float* v = V + t * p.dv + col0 + c0;
    {
      const float pj = (mine[lane] + mine[64 + lane]) + (mine[128 + lane] + mine[192 + lane]);
      const float rj = (mine[32 + lane] + mine[96 + lane]) + (mine[160 + lane] + mine[224 + lane]);
      const float u = beta * (v[lane] - pj), o = p.q_scale * fmaf(qk, u, rj);
#pragma unroll
      for (int j = 0; j < 32; ++j) S[j] = fmaf(k, __shfl_sync(~0u, u, j), S[j]);
      if ((warp & 3) == 0) {
        const long long at = ((req.start + static_cast<long long>(t0 + t)) * p.Hv + vh) * p.dv + col0 + c0 + lane;
        if (p.out_dtype == GDN_DTYPE_BF16) static_cast<__nv_bfloat16*>(p.out)[at] = __float2bfloat16_rn(o);
        else static_cast<float*>(p.out)[at] = o;
      }
    }
    barrier();
  }
}

template <int DK, int NB>
__global__ void __launch_bounds__(Chain<DK, NB>::kThreads, 1)
seq_chain_kernel(const SeqParams p, const __grid_constant__ Segment seg, const char* ws) {
  using L = Chain<DK, NB>;
  extern __shared__ __align__(128) char sm[];
  uint64_t* bar = reinterpret_cast<uint64_t*>(sm + L::kBar);
  float* maxima = reinterpret_cast<float*>(sm + L::kMax);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int slices = p.dv / NB;
  const int vh = blockIdx.x / slices, col0 = blockIdx.x % slices * NB;
  const SegReq req = seg.r[blockIdx.y];
  const int R = p.Hv / p.Hk, kh = vh / R;
  const size_t slot_bytes = p.Hk * seq_kq_bytes(DK) + p.Hv * seq_v_bytes(p.dv);
  const char* const kq_ws = ws + req.slot0 * slot_bytes + kh * seq_kq_bytes(DK);
  const char* const v_ws = ws + req.slot0 * slot_bytes + p.Hk * seq_kq_bytes(DK) + vh * seq_v_bytes(p.dv);
  const bool aborted = launch_aborted(p.err);

  if (warp == 4 * L::kGroups) tmem_alloc(reinterpret_cast<uint32_t*>(bar + kTmemAt), L::kCols);
  if (tid == 0) {
    mbar_init_n(bar + kKqFull, 1);
    mbar_init_n(bar + kMnFull, 1);
    mbar_init_n(bar + kSReady, 4 * L::kGroups);
    mbar_init_n(bar + kD1, 1);
    mbar_init_n(bar + kWReady, 2 * L::kGroups);
    mbar_init_n(bar + kD2, 1);
    mbar_init_n(bar + kUReady, 2 * L::kGroups);
    mbar_init_n(bar + kD3, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    fence_proxy_async();
  }
  const bool stop = __syncthreads_or(aborted);
  const uint32_t tmem = *reinterpret_cast<uint32_t*>(bar + kTmemAt);
  if (warp == 4 * L::kGroups) tmem_relinquish();
  bool late = false;
  // A wait that gave up is not repeated: the loops run to their end, the results are reported as lost.
  auto wait = [&](int which, int parity) {
    if (!late && !mbar_wait(bar + which, parity)) late = true;
  };

  if (stop) {
    // an earlier launch gave up: nothing is done
  } else if (warp == 4 * L::kGroups) {
    if (lane == 0) {
      auto load_k = [&](int i) {       // chunk i of the segment
        const int place = (req.c0 + i) & 1 ? 2 : 0;
        const char* src = kq_ws + i * slot_bytes;
        mbar_expect(bar + kKqFull, 4 * L::kImage);
        bulk_g2s(sm + L::kKq + place * L::kImage, src, L::kImage, bar + kKqFull);
        bulk_g2s(sm + L::kKq + L::kKqLo + place * L::kImage, src + L::kImage, L::kImage, bar + kKqFull);
      };
      auto load_q = [&](int i) {
        const char* src = kq_ws + i * slot_bytes + 2 * L::kImage;
        bulk_g2s(sm + L::kKq + L::kImage, src, L::kImage, bar + kKqFull);
        bulk_g2s(sm + L::kKq + L::kKqLo + L::kImage, src + L::kImage, L::kImage, bar + kKqFull);
      };
      auto load_mn = [&](int i) {
        mbar_expect(bar + kMnFull, 2 * L::kMnLo);
        bulk_g2s(sm + L::kMn, v_ws + i * slot_bytes, 2 * L::kMnLo, bar + kMnFull);
      };
      load_k(0);
      load_q(0);
      load_mn(0);
      const uint64_t s_b = umma_desc(smem_addr(sm + L::kS), 128, DK * 16);
      const uint64_t w_b = umma_desc(smem_addr(sm + L::kW), 128, kChunk * 16);
      const uint64_t mn_a = umma_desc(smem_addr(sm + L::kMn), 128, 1024);
      for (int i = 0; i < req.nc; ++i) {
        const int odd = (req.c0 + i) & 1, ph = i & 1;
        wait(kKqFull, ph);
        wait(kSReady, ph);
        if (late) break;
        tmem_fence_after();
        // rows 0 to 127: [K; Q], or [Q; K] in odd chunks
        product<DK / 16>(tmem, umma_desc(smem_addr(sm + L::kKq + odd * L::kImage), 128, DK * 16), s_b, L::kKqLo, L::kSLo, 256,
                         256, idesc_f16(NB, false, true));
        umma_commit(bar + kD1);
        if (i + 1 < req.nc) load_k(i + 1);
        wait(kD1, ph);
        if (i + 1 < req.nc) load_q(i + 1);
        wait(kMnFull, ph);
        wait(kWReady, ph);
        if (late) break;
        tmem_fence_after();
        product<kChunk / 16>(tmem + NB, mn_a, w_b, L::kMnLo, L::kWLo, 256, 256, idesc_f16(NB, false, true));
        umma_commit(bar + kD2);
        wait(kD2, ph);
        if (i + 1 < req.nc) load_mn(i + 1);
        wait(kUReady, ph);
        if (late) break;
        tmem_fence_after();
        product<kChunk / 16>(tmem + 2 * NB, umma_desc(smem_addr(sm + L::kKq + odd * 2 * L::kImage), DK * 16, 128), w_b, L::kKqLo,
                             L::kWLo, 2 * DK * 16, 256, idesc_f16(NB, true, true));
        umma_commit(bar + kD3);
      }
      wait(kD3, (req.nc - 1) & 1);
      if (late) {      // whatever was in flight has had twice the time that a wait gives it
        mbar_wait(bar + kKqFull, 0), mbar_wait(bar + kKqFull, 1), mbar_wait(bar + kMnFull, 0), mbar_wait(bar + kMnFull, 1);
      }
    }
    __syncwarp();
  } else {
    const int row = (warp & 3) * 32 + lane, cg = warp >> 2, c0 = cg * 32;     // lane of tensor memory, columns of the slice
    const uint32_t ta = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + c0;
    const bool has_row = row < DK;
    auto soft_barrier = [] { asm volatile("bar.sync 1, %0;" ::"n"(L::kSoft) : "memory"); };
    float S[32];
    // the state before the segment: the call's, or what the segment before left
    {
      const float* src = req.c0 == 0 ? p.state_in : p.state_out;
      if (src && has_row) {
        src += req.b * p.state_stride + (static_cast<long long>(vh) * DK + row) * p.dv + col0 + c0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float4 t = *reinterpret_cast<const float4*>(src + 4 * j);
          S[4 * j] = t.x, S[4 * j + 1] = t.y, S[4 * j + 2] = t.z, S[4 * j + 3] = t.w;
        }
      } else {
#pragma unroll
        for (int j = 0; j < 32; ++j) S[j] = 0.f;
      }
    }
    float smax, omax = 0.f, inv_s;
    // the largest entry of T, and of the chunk's o, over all threads
    auto find_maxima = [&]() {
      float big = 0.f;
#pragma unroll
      for (int j = 0; j < 32; ++j) big = abs_bits_max(big, S[j]);
      big = warp_max(big);
      const float bigo = warp_max(omax);
      if (lane == 0) maxima[warp] = big, maxima[4 * L::kGroups + warp] = bigo;
      soft_barrier();
      smax = omax = 0.f;
#pragma unroll
      for (int w = 0; w < 4 * L::kGroups; ++w) {
        smax = abs_bits_max(smax, maxima[w]);
        omax = abs_bits_max(omax, maxima[4 * L::kGroups + w]);
      }
    };
    // T into its two-term operand
    auto put_state = [&]() {
      const float sc = scale_for(smax, inv_s);
      if (has_row) {
#pragma unroll
        for (int j = 0; j < 32; j += 8) {
          float v[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) v[k] = S[j + k] * sc;
          uint4 hi, lo;
          split8(v, hi, lo);
          char* at = sm + L::kS + ((c0 + j) >> 3) * DK * 16 + row * 16;
          *reinterpret_cast<uint4*>(at) = hi;
          *reinterpret_cast<uint4*>(at + L::kSLo) = lo;
        }
      }
      fence_proxy_async();
      tmem_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar + kSReady);
    };
    find_maxima();
    put_state();
    for (int i = 0; i < req.nc; ++i) {
      const int odd = (req.c0 + i) & 1, ph = i & 1;
      const bool k_row = (row >> 6) == odd;                    // this thread's row is a token's k (else its q)
      const int t = row & 63, tok = (req.c0 + i) * kChunk + t;
      const float* meta = reinterpret_cast<const float*>(v_ws + i * slot_bytes + 4 * 128 * kChunk + kChunk * p.dv * 4);
      const float first = __ldg(meta + t), left = __ldg(meta + kChunk + t), whole = __ldg(meta + 2 * kChunk);
      const float inv_m = __ldg(meta + 2 * kChunk + 1), inv_n = __ldg(meta + 2 * kChunk + 2), vmax = __ldg(meta + 2 * kChunk + 3);
      const float mbound = __ldg(meta + 2 * kChunk + 4), fmax_ = __ldg(meta + 2 * kChunk + 5), nbound = __ldg(meta + 2 * kChunk + 6);
      float a[32];                                             // v of a k row; later the first part of o of a q row
      if (k_row) {
        const float* V = reinterpret_cast<const float*>(v_ws + i * slot_bytes + 4 * 128 * kChunk) + t * p.dv + col0 + c0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float4 f = __ldg(reinterpret_cast<const float4*>(V) + j);
          a[4 * j] = f.x, a[4 * j + 1] = f.y, a[4 * j + 2] = f.z, a[4 * j + 3] = f.w;
        }
      }
      wait(kD1, ph);
      tmem_fence_after();
      const float w_bound = (vmax + fmax_ * (DK == 128 ? 11.32f : DK == 64 ? 8.001f : 5.657f) * smax) * 1.001f;
      const float u_bound = mbound * w_bound * 1.001f;
      float inv_w, inv_u;
      const float sc_w = scale_for(w_bound, inv_w), sc_u = scale_for(u_bound, inv_u);
      const float f1 = first * (inv_s * (1.f / kUnit));
      if (k_row) {
#pragma unroll
        for (int j = 0; j < 32; j += 16) {
          float d[16];
          tmem_ld16(ta + j, d);
          tmem_wait_ld();
#pragma unroll
          for (int k = 0; k < 16; ++k) d[k] = fmaf(-f1, d[k], a[j + k]) * sc_w;
#pragma unroll
          for (int k = 0; k < 16; k += 8) {
            uint4 hi, lo;
            split8(d + k, hi, lo);
            char* at = sm + L::kW + ((c0 + j + k) >> 3) * kChunk * 16 + t * 16;
            *reinterpret_cast<uint4*>(at) = hi;
            *reinterpret_cast<uint4*>(at + L::kWLo) = lo;
          }
        }
        fence_proxy_async();
        tmem_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar + kWReady);
      } else {
        const float f = f1 * p.q_scale;
        tmem_ld16(ta, *reinterpret_cast<float(*)[16]>(a));
        tmem_ld16(ta + 16, *reinterpret_cast<float(*)[16]>(a + 16));
        tmem_wait_ld();
#pragma unroll
        for (int j = 0; j < 32; ++j) a[j] *= f;
      }
      wait(kD2, ph);
      tmem_fence_after();
      if (k_row) {
        const float f = left * inv_m * inv_w * sc_u;
#pragma unroll
        for (int j = 0; j < 32; j += 16) {
          float d[16];
          tmem_ld16(ta + NB + j, d);
          tmem_wait_ld();
#pragma unroll
          for (int k = 0; k < 16; ++k) d[k] *= f;
#pragma unroll
          for (int k = 0; k < 16; k += 8) {
            uint4 hi, lo;
            split8(d + k, hi, lo);
            char* at = sm + L::kW + ((c0 + j + k) >> 3) * kChunk * 16 + t * 16;
            *reinterpret_cast<uint4*>(at) = hi;
            *reinterpret_cast<uint4*>(at + L::kWLo) = lo;
          }
        }
        fence_proxy_async();
        tmem_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar + kUReady);
      } else {
        const float f = inv_n * inv_w * p.q_scale;
#pragma unroll
        for (int j = 0; j < 32; j += 16) {
          float d[16];
          tmem_ld16(ta + NB + j, d);
          tmem_wait_ld();
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            a[j + k] = fmaf(f, d[k], a[j + k]);
            omax = abs_bits_max(omax, a[j + k]);
          }
        }
        if (tok < req.len) {
          const long long at = ((req.start + static_cast<long long>(tok)) * p.Hv + vh) * p.dv + col0 + c0;
          if (p.out_dtype == GDN_DTYPE_BF16) {
            uint4* o = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.out) + at);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              __nv_bfloat162 b[4];
#pragma unroll
              for (int k = 0; k < 4; ++k) b[k] = __floats2bfloat162_rn(a[8 * j + 2 * k], a[8 * j + 2 * k + 1]);
              o[j] = *reinterpret_cast<uint4*>(b);
            }
          } else {
            float4* o = reinterpret_cast<float4*>(static_cast<float*>(p.out) + at);
#pragma unroll
            for (int j = 0; j < 8; ++j) o[j] = make_float4(a[4 * j], a[4 * j + 1], a[4 * j + 2], a[4 * j + 3]);
          }
        }
      }
      wait(kD3, ph);
      tmem_fence_after();
      const float f3 = inv_u * (1.f / kUnit);
#pragma unroll
      for (int j = 0; j < 32; j += 16) {
        float d[16];
        tmem_ld16(ta + 2 * NB + j, d);
        tmem_wait_ld();
#pragma unroll
        for (int k = 0; k < 16; ++k) S[j + k] = has_row ? fmaf(whole, S[j + k], f3 * d[k]) : 0.f;
      }
      find_maxima();
      // Values far below what the bounds allow have lost their bits: the chunk is taken again, token by token.
      const float o_bound = nbound * w_bound * fabsf(p.q_scale);
      if (u_bound * kRange > smax || o_bound * kRange > omax) {
        again_by_token<DK, NB>(p, req, vh, row, has_row, c0, col0, (req.c0 + i) * kChunk, inv_s, kq_ws + i * slot_bytes,
                               reinterpret_cast<const float*>(v_ws + i * slot_bytes + 4 * 128 * kChunk), sm, S);
        find_maxima();
      }
      omax = 0.f;
      if (i + 1 < req.nc) put_state();
    }
    if (has_row) {
      float* dst = p.state_out + req.b * p.state_stride + (static_cast<long long>(vh) * DK + row) * p.dv + col0 + c0;
#pragma unroll
      for (int j = 0; j < 8; ++j)
        *reinterpret_cast<float4*>(dst + 4 * j) = make_float4(S[4 * j], S[4 * j + 1], S[4 * j + 2], S[4 * j + 3]);
    }
  }
  // The window after the prompt: its last K - 1 rows (the launch before has read the old ones).
  if (!stop && p.K > 1 && (req.c0 + req.nc) * kChunk >= req.len) {
    const float* win = p.conv_in ? p.conv_in + req.b * p.conv_stride : nullptr;
    float* wout = p.conv_out + req.b * p.conv_stride;
    const int kq = p.Hk * DK, extra = vh % R == 0 && col0 == 0 ? 2 * DK : 0;
    for (int c = tid; c < NB + extra; c += L::kThreads) {
      const int ch = c < NB ? 2 * kq + vh * p.dv + col0 + c : c - NB < DK ? kh * DK + c - NB : kq + kh * DK + c - NB - DK;
      for (int j = 0; j < p.K - 1; ++j) {
        const int t = req.len - (p.K - 1) + j;
        const long long at = (req.start + static_cast<long long>(t)) * p.x_row + ch;
        wout[static_cast<long long>(j) * p.C + ch] =
            t < 0 ? (win ? win[static_cast<long long>(p.K - 1 + t) * p.C + ch] : 0.f)
                  : p.in_dtype == GDN_DTYPE_BF16 ? load_f(static_cast<const __nv_bfloat16*>(p.x) + at)
                                                 : load_f(static_cast<const float*>(p.x) + at);
      }
    }
  }
  if (__syncthreads_or(late) && tid == 0) device_error(p.err, GDN_DEVERR_TIMEOUT, req.b);
  if (warp == 4 * L::kGroups) tmem_dealloc(tmem, L::kCols);
}

template <typename F>
cudaError_t with_smem(F kernel, int bytes) {
  return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
}
template <typename InT, int DK, int KT>
cudaError_t launch_prepare(const SeqParams& p, const Segment& seg, char* ws, cudaStream_t s) {
  auto k = seq_prepare_kernel<InT, DK, KT>;
  cudaError_t e = with_smem(k, Prep<DK>::kTotal);
  if (e != cudaSuccess) return e;
  k<<<dim3(p.Hk, seg.slots), kPrepThreads, Prep<DK>::kTotal, s>>>(p, seg, ws);
  return cudaGetLastError();
}
template <int DK, int NB>
cudaError_t launch_chain(const SeqParams& p, const Segment& seg, const char* ws, cudaStream_t s) {
  auto k = seq_chain_kernel<DK, NB>;
  cudaError_t e = with_smem(k, Chain<DK, NB>::kTotal);
  if (e != cudaSuccess) return e;
  k<<<dim3(p.Hv * (p.dv / NB), seg.n), Chain<DK, NB>::kThreads, Chain<DK, NB>::kTotal, s>>>(p, seg, ws);
  return cudaGetLastError();
}
template <int DK>
cudaError_t launch_d(const SeqParams& p, const Segment& seg, char* ws, cudaStream_t s) {
  using bf16 = __nv_bfloat16;
  const bool wide = p.K > 4;
  cudaError_t e = p.in_dtype == GDN_DTYPE_BF16
                      ? (wide ? launch_prepare<bf16, DK, 8>(p, seg, ws, s) : launch_prepare<bf16, DK, 4>(p, seg, ws, s))
                      : (wide ? launch_prepare<float, DK, 8>(p, seg, ws, s) : launch_prepare<float, DK, 4>(p, seg, ws, s));
  if (e != cudaSuccess) return e;
  // whole heads a CTA, or half ones where the other half of the GPU would be idle
  if (p.dv == 128 && seg.n * p.Hv > 76) return launch_chain<DK, 128>(p, seg, ws, s);
  if (p.dv >= 64 && seg.n * p.Hv * (p.dv / 64) > 38) return launch_chain<DK, 64>(p, seg, ws, s);
  return launch_chain<DK, 32>(p, seg, ws, s);
}

}  // namespace

int seq_requests_at_once(int Hv) { return Hv >= 152 ? 1 : 152 / Hv < kSegReqs ? 152 / Hv : kSegReqs; }

cudaError_t launch_seq_chunks(const SeqParams& p, const Segment& seg, void* workspace, cudaStream_t s) {
  char* ws = static_cast<char*>(workspace);
  if (p.dk == 128) return launch_d<128>(p, seg, ws, s);
  if (p.dk == 64) return launch_d<64>(p, seg, ws, s);
  return launch_d<32>(p, seg, ws, s);
}

}  // namespace gdn
