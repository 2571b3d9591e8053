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
__device__ __forceinline__ void umma_f16_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, int accumulate) {   // A in tensor memory
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ bool elect_one() {
  uint32_t yes;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(yes));
  return yes != 0;
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
// Four packed pairs as eight fp16 high terms and eight low ones.
__device__ __forceinline__ void split_pair(u64 x, uint32_t& hi, uint32_t& lo) {
  const float2 f = unpack2(x);
  const __half2 h = __floats2half2_rn(f.x, f.y);
  const float2 b = __half22float2(h);
  const float2 r = unpack2(fma2(pack2(b.x, b.y), pack2(-1.f, -1.f), x));
  const __half2 l = __floats2half2_rn(r.x, r.y);
  hi = *reinterpret_cast<const uint32_t*>(&h);
  lo = *reinterpret_cast<const uint32_t*>(&l);
}
__device__ __forceinline__ void split_pairs(const u64* x, uint4& hi, uint4& lo) {
  split_pair(x[0], hi.x, lo.x);
  split_pair(x[1], hi.y, lo.y);
  split_pair(x[2], hi.z, lo.z);
  split_pair(x[3], hi.w, lo.w);
}
__device__ __forceinline__ float abs_max(float m, u64 x) {
  const float2 f = unpack2(x);
  return fmaxf(m, fmaxf(fabsf(f.x), fabsf(f.y)));
}

// A bounded wait that leaves the issue slots to the working warps.
__device__ __forceinline__ bool mbar_wait_quiet(uint64_t* bar, uint32_t parity) {
  const long long t0 = clock64();
  while (!mbar_ready(bar, parity))
    if (clock64() - t0 > kWaitCycles) return false;
  return true;
}

// Sixteen columns of this thread's lane as packed pairs; the wait is inside, so they are defined when the statement ends.
__device__ __forceinline__ void tmem_pairs(uint32_t ta, u64 (&v)[8]) {
  asm volatile(
      "{\n"
      " .reg .b32 t<16>;\n"
      " tcgen05.ld.sync.aligned.32x32b.x16.b32 {t0, t1, t2, t3, t4, t5, t6, t7, t8, t9, t10, t11, t12, t13, t14, t15}, [%8];\n"
      " tcgen05.wait::ld.sync.aligned;\n"
      " mov.b64 %0, {t0, t1};\n"
      " mov.b64 %1, {t2, t3};\n"
      " mov.b64 %2, {t4, t5};\n"
      " mov.b64 %3, {t6, t7};\n"
      " mov.b64 %4, {t8, t9};\n"
      " mov.b64 %5, {t10, t11};\n"
      " mov.b64 %6, {t12, t13};\n"
      " mov.b64 %7, {t14, t15};\n"
      "}"
      : "=l"(v[0]), "=l"(v[1]), "=l"(v[2]), "=l"(v[3]), "=l"(v[4]), "=l"(v[5]), "=l"(v[6]), "=l"(v[7])
      : "r"(ta)
      : "memory");
}
__device__ __forceinline__ float exp2_fast(float x) {   // results below 2^-126 are zero
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
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
  u64 r[kTok + KT - 1][2], w[KT][2];
  const int K = p.K;
  // The rows, all in flight at once: those outside the request are read at its nearest row, and replaced after.
  float4 f[kTok + KT - 1];
#pragma unroll
  for (int i = 0; i < kTok + KT - 1; ++i)
    f[i] = raw4(x + static_cast<long long>(min(max(t0 + i - (KT - 1), 0), len - 1)) * p.x_row + ch);
#pragma unroll
  for (int j = 0; j < KT; ++j) w[j][0] = w[j][1] = 0ull;
  if (p.conv_mode != 1) {
    w[KT - 1][0] = w[KT - 1][1] = pack2(1.f, 1.f);
  } else if (KT == 4 && K == 4) {
    const float4* cw = reinterpret_cast<const float4*>(p.conv_w + static_cast<long long>(ch) * 4);
    const float4 c0 = __ldg(cw), c1 = __ldg(cw + 1), c2 = __ldg(cw + 2), c3 = __ldg(cw + 3);
    w[0][0] = pack2(c0.x, c1.x), w[0][1] = pack2(c2.x, c3.x);
    w[1][0] = pack2(c0.y, c1.y), w[1][1] = pack2(c2.y, c3.y);
    w[KT - 2][0] = pack2(c0.z, c1.z), w[KT - 2][1] = pack2(c2.z, c3.z);
    w[KT - 1][0] = pack2(c0.w, c1.w), w[KT - 1][1] = pack2(c2.w, c3.w);
  } else {
#pragma unroll
    for (int j = 0; j < KT; ++j)
      if (j >= KT - K) {
        const float* cw = p.conv_w + static_cast<long long>(ch) * K + j - (KT - K);
        w[j][0] = pack2(__ldg(cw), __ldg(cw + K)), w[j][1] = pack2(__ldg(cw + 2 * K), __ldg(cw + 3 * K));
      }
  }
  if (t0 < KT - 1) {                               // rows before the first: the window's, where it has them
#pragma unroll
    for (int i = 0; i < KT - 1; ++i) {
      const int t = t0 + i - (KT - 1);
      if (t < 0) {
        f[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (i >= KT - K && win) f[i] = raw4(win + static_cast<long long>(K - 1 + t) * p.C + ch);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < kTok + KT - 1; ++i) r[i][0] = pack2(f[i].x, f[i].y), r[i][1] = pack2(f[i].z, f[i].w);
#pragma unroll
  for (int t = 0; t < kTok; ++t) {
    u64 a = mul2(w[KT - 1][0], r[t + KT - 1][0]), b = mul2(w[KT - 1][1], r[t + KT - 1][1]);
#pragma unroll
    for (int i = 1; i < KT; ++i)
      if (i < K) {
        a = fma2(w[KT - 1 - i][0], r[t + KT - 1 - i][0], a);
        b = fma2(w[KT - 1 - i][1], r[t + KT - 1 - i][1], b);
      }
    const float2 lo = unpack2(a), hi = unpack2(b);
    float4 o = make_float4(lo.x, lo.y, hi.x, hi.y);
    if (p.act == 1) o = make_float4(silu(o.x), silu(o.y), silu(o.z), silu(o.w));
    y[t] = o;
  }
  if (t0 + kTok > len) {
#pragma unroll
    for (int t = 0; t < kTok; ++t)
      if (t0 + t >= len) y[t] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
}

// ---- what does not depend on the state ------------------------------------------------------------------------------

constexpr int kPrepThreads = 256, kPrepWarps = kPrepThreads / 32;
constexpr int kHeads = 3;                  // v-heads of a k-head in work together
constexpr int kLd = 68;                    // floats a row of A and X
constexpr int kRowLd = 132;                // of rows of q, k or v

template <int DK>
struct Prep {
  static constexpr int kImage = kChunk * DK * 2;              // one fp16 image of K or Q
  static constexpr int kImages = 0;                           // Kh Qh Kl Ql
  static constexpr int kRows = 4 * kImage;                    // rows of q, k or v in 32 bits
  static constexpr int kRowBytes = kChunk * kRowLd * 4;
  // later, in the images' place: A and X of kHeads heads, images (high, low) of their M
  static constexpr int kSq = kChunk * kChunk * 2;             // an fp16 image of a 64 x 64 matrix
  static constexpr int kAx = 0, kAxBytes = kChunk * kLd * 4;
  static constexpr int kM = kHeads * kAxBytes;
  static constexpr int kEnd = kRows + kRowBytes > kM + kHeads * 2 * kSq ? kRows + kRowBytes : kM + kHeads * 2 * kSq;
  static constexpr int kGate = kEnd;                          // a head: float2 [64] log2 of the cumulated gates (high, low part), beta [64], left [64]
  static constexpr int kRed = kGate + kHeads * 4 * kChunk * 4;  // float [128]
  static constexpr int kBar = kRed + 128 * 4;                 // Gram product, N
  static constexpr int kTotal = kBar + 64;
};
// Columns of tensor memory: the Gram product, later N | C of the heads
constexpr uint32_t kTmGram = 0, kTmC = 64, kTmPrep = 256;

// 16-byte places of an fp16 image of `width` columns: row r, columns 8 c ..
__device__ __forceinline__ int image_at(int r, int c, int width) { return (r >> 3) * width * 16 + c * 128 + (r & 7) * 16; }

// X = (1 + A)^-1 for strictly lower A, columns 32 half ..: lane = column, forward substitution by blocks of 16 rows.
// ax[j][i] (kLd floats a row) holds A_ij in i > j; X_kj goes to ax[k][j], j <= k, which A leaves free.
__device__ __forceinline__ void solve_columns(float* ax, int half, int lane) {
  const int col = half * 32 + lane;
#pragma unroll 1
  for (int bi = 2 * half; bi < 4; ++bi) {                      // blocks above the columns' own are zero
    const int r0 = 16 * bi;
    u64 acc[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) acc[q] = pack2(r0 + 2 * q == col ? 1.f : 0.f, r0 + 2 * q + 1 == col ? 1.f : 0.f);
#pragma unroll 1
    for (int k = 32 * half; k < r0; k += 4) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float* a = ax + (k + e) * kLd;
        const float x = col <= k + e ? -a[col] : 0.f;
        const u64 x2 = pack2(x, x);
#pragma unroll
        for (int q = 0; q < 8; q += 2) {
          const ulonglong2 v = *reinterpret_cast<const ulonglong2*>(a + r0 + 2 * q);
          acc[q] = fma2(x2, v.x, acc[q]);
          acc[q + 1] = fma2(x2, v.y, acc[q + 1]);
        }
      }
    }
    // row i of the diagonal block, read one step ahead of the store into it
    ulonglong2 now[4], next[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) now[q] = *reinterpret_cast<const ulonglong2*>(ax + r0 * kLd + r0 + 4 * q);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float* a = ax + (r0 + i) * kLd;
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (i + 1 < 15 && 4 * q + 3 > i + 1) next[q] = *reinterpret_cast<const ulonglong2*>(a + kLd + r0 + 4 * q);
      const float2 f = unpack2(acc[i / 2]);
      const float x = i & 1 ? f.y : f.x;
      const u64 x2 = pack2(-x, -x);
      // rows behind row i (their neighbours in a pair are done with and may take anything)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        if (4 * q + 1 > i) acc[2 * q] = fma2(x2, now[q].x, acc[2 * q]);
        if (4 * q + 3 > i) acc[2 * q + 1] = fma2(x2, now[q].y, acc[2 * q + 1]);
      }
      if (col <= r0 + i) a[col] = x;
#pragma unroll
      for (int q = 0; q < 4; ++q) now[q] = next[q];
    }
    __syncwarp();
  }
}

template <typename InT, int DK, int KT>
__global__ void __launch_bounds__(kPrepThreads, 2)
seq_prepare_kernel(const SeqParams p, const __grid_constant__ Segment seg, char* ws) {
  using P = Prep<DK>;
  extern __shared__ __align__(128) char sm[];
  float* rows = reinterpret_cast<float*>(sm + P::kRows);
  float* red = reinterpret_cast<float*>(sm + P::kRed);
  uint64_t* bar = reinterpret_cast<uint64_t*>(sm + P::kBar);
  uint32_t* tmem_at = reinterpret_cast<uint32_t*>(bar + 3);
  float* unit = reinterpret_cast<float*>(bar + 4);             // [2 kHeads] scales of C, inverse ones of M
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
  const int h0 = blockIdx.z * kHeads, nh = min(kHeads, R - h0);      // the k-head's v-heads this CTA takes
  auto head_ws = [&](int h) { return slot_ws + p.Hk * seq_kq_bytes(DK) + (kh * R + h0 + h) * seq_v_bytes(dv); };
  auto head_meta = [&](int h) { return reinterpret_cast<float*>(head_ws(h) + 4 * 128 * kChunk + kChunk * dv * 4); };
  auto gates_of = [&](int h) { return reinterpret_cast<float*>(sm + P::kGate) + h * 4 * kChunk; };
  const bool aborted = launch_aborted(p.err);

  if (warp == 0) tmem_alloc(tmem_at, kTmPrep);
  if (tid == 0)
    for (int i = 0; i < 2; ++i) mbar_init(bar + i);
  if (__syncthreads_or(aborted)) {
    if (warp == 0) {
      tmem_relinquish();
      tmem_dealloc(*tmem_at, kTmPrep);
    }
    return;
  }
  if (warp == 0) tmem_relinquish();
  const uint32_t tmem = *tmem_at;
  bool late = false;
  auto wait = [&](int which, int parity) {
    if (!late && !mbar_wait_quiet(bar + which, parity)) late = true;
  };

  if (tid < kChunk + 3) {                          // the raw rows on their way into L2
    const int t = t0 + tid - 3;
    if (t >= 0 && t < len) {
      const InT* r = x + static_cast<long long>(t) * p.x_row;
      prefetch_l2(r + kh * DK, DK * sizeof(InT));
      prefetch_l2(r + (p.Hk + kh) * DK, DK * sizeof(InT));
      prefetch_l2(r + 2 * p.Hk * DK + (kh * R + h0) * dv, nh * dv * sizeof(InT));
    }
  }
  // gates, a warp a head: cumulated in 64 bits and base 2, kept as two floats
  if (warp < nh) {
    float* const gate = gates_of(warp);
    float* const meta = head_meta(warp);
    double c[2];
    float rise = 0.f;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int t = t0 + 2 * lane + k;
      float lg = 0.f, b = 0.f;
      if (t < len) {
        const long long at = (req.start + static_cast<long long>(t)) * p.gate_row + kh * R + h0 + warp;
        b = load_f(static_cast<const InT*>(p.beta) + at);
        lg = load_f(static_cast<const InT*>(p.log_g) + at);
        lg = lg < kGateFloor ? kGateFloor : lg;
      }
      rise += fmaxf(lg, 0.f);
      c[k] = static_cast<double>(lg) * 1.4426950408889634;
      gate[2 * kChunk + 2 * lane + k] = b;
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
    for (int k = 0; k < 2; ++k) {
      const double s = before + c[k];
      const float hi = static_cast<float>(s), lo = static_cast<float>(s - hi);
      const float first = exp2f(hi) * fmaf(lo, 0.69314718f, 1.f), left = exp2f(static_cast<float>(total - s));
      reinterpret_cast<float2*>(gate)[2 * lane + k] = make_float2(hi, lo);
      gate[3 * kChunk + 2 * lane + k] = left;
      meta[2 * lane + k] = first;
      meta[kChunk + 2 * lane + k] = left;
      most = fmaxf(most, first);
    }
    most = warp_max(most);
    if (lane == 0) {
      meta[2 * kChunk] = exp2f(static_cast<float>(total));
      meta[2 * kChunk + 5] = most;
      // no product of gates is above e^rise (1 unless a log gate is above 0)
      unit[warp] = exp2f(floorf(11.f - rise * kLog2e));
    }
  }

  // k, q, then the heads' v: conv and activation (k and q: norm) into rows; from there k and q as two-term images, here and
  // in the workspace, and v four columns of all tokens together, [dv / 4][64][4].
  // A lane takes four channels of kTok adjacent tokens, a warp eight tokens.
  constexpr int kTok = DK == 128 ? 8 : 4;
#pragma unroll 1
  for (int kind = 0; kind < 2 + nh; ++kind) {
    const int width = kind < 2 ? DK : dv, lanes = width / 4, sub = lane / lanes, cl = (lane % lanes) * 4;
    const int ch = kind == 0 ? (p.Hk + kh) * DK : kind == 1 ? kh * DK : 2 * p.Hk * DK + (kh * R + h0 + kind - 2) * dv;
    float most = 0.f;
#pragma unroll 1
    for (int t = kTok * sub; t - kTok * sub < 8; t += lanes == 32 ? kTok : 8) {
      const int first = warp * 8 + t;
      float4 y[kTok];
      if (t < 8) conv_tokens<InT, KT, kTok>(p, x, win, t0 + first, len, ch + cl, y);
#pragma unroll
      for (int i = 0; i < kTok; ++i) {
        if (kind < 2) {
          float ss = fmaf(y[i].x, y[i].x, fmaf(y[i].y, y[i].y, fmaf(y[i].z, y[i].z, y[i].w * y[i].w)));
#pragma unroll
          for (int o = DK / 8; o > 0; o >>= 1) ss += __shfl_xor_sync(~0u, ss, o);
          const float f = t0 + first + i < len ? rsqrtf(ss + p.l2_eps) * kUnit : 0.f;
          y[i] = make_float4(y[i].x * f, y[i].y * f, y[i].z * f, y[i].w * f);
        }
        if (t < 8) {
          *reinterpret_cast<float4*>(rows + (first + i) * kRowLd + cl) = y[i];
          most = fmaxf(most, fmaxf(fmaxf(fabsf(y[i].x), fabsf(y[i].y)), fmaxf(fabsf(y[i].z), fabsf(y[i].w))));
        }
      }
    }
    __syncwarp();
    most = warp_max(most);
    if (lane == 0) red[warp] = most;
    __syncthreads();
    const int t = tid & 63;
    if (kind < 2) {
      char* const hi_sm = sm + P::kImages + kind * P::kImage;
      char* const hi_ws = kq_ws + 2 * kind * P::kImage;
#pragma unroll
      for (int c = 0; c < DK / 8; c += kPrepThreads / 64) {
        const int cc = c + (tid >> 6);
        const ulonglong2* src = reinterpret_cast<const ulonglong2*>(rows + t * kRowLd + 8 * cc);
        const ulonglong2 v0 = src[0], v1 = src[1];
        const u64 v[4] = {v0.x, v0.y, v1.x, v1.y};
        uint4 hi, lo;
        split_pairs(v, hi, lo);
        const int at = image_at(t, cc, DK);
        *reinterpret_cast<uint4*>(hi_sm + at) = hi;
        *reinterpret_cast<uint4*>(hi_sm + 2 * P::kImage + at) = lo;
        if (h0 == 0) {
          *reinterpret_cast<uint4*>(hi_ws + at) = hi;
          *reinterpret_cast<uint4*>(hi_ws + P::kImage + at) = lo;
        }
      }
      fence_proxy_async();
    } else {
      float4* const V = reinterpret_cast<float4*>(head_ws(kind - 2) + 4 * 128 * kChunk);
#pragma unroll 4
      for (int c = tid >> 6; c < dv / 4; c += kPrepThreads / 64)
        V[c * kChunk + t] = *reinterpret_cast<const float4*>(rows + t * kRowLd + 4 * c);
      if (tid == 0) {
        most = 0.f;
        for (int w = 0; w < kPrepWarps; ++w) most = fmaxf(most, red[w]);
        head_meta(kind - 2)[2 * kChunk + 3] = most;
      }
    }
    __syncthreads();
    if (kind == 1 && warp == 0) {
      // G = K K^T (lanes 0 to 63) and H = Q K^T
      if (elect_one()) {
        const uint64_t a = umma_desc(smem_addr(sm + P::kImages), 128, DK * 16);
        product<DK / 16>(tmem + kTmGram, a, a, 2 * P::kImage, 2 * P::kImage, 256, 256, idesc_f16(kChunk, false, false));
        umma_commit(bar);
      }
      __syncwarp();
    }
  }
  wait(0, 0);
  tmem_fence_after();
  __syncthreads();                                 // A takes the Gram operands' place

  // A thread has 32 entries of a row of G (warps 0, 1, 4, 5) or H (the others).
  const int trow = (warp & 3) * 32 + lane, tcol = (warp >> 2) * 32, i = trow & 63;
  const bool q_row = trow >= kChunk;
  const uint32_t ta = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
  {
    u64 g[16];
    tmem_pairs(ta + kTmGram + tcol, *reinterpret_cast<u64(*)[8]>(g));
    tmem_pairs(ta + kTmGram + tcol + 16, *reinterpret_cast<u64(*)[8]>(g + 8));
#pragma unroll 1
    for (int h = 0; h < nh; ++h) {
      const float* const gate = gates_of(h);
      const float4* const c = reinterpret_cast<const float4*>(gate) + tcol / 2;     // two tokens' sums
      const float2 ci = reinterpret_cast<const float2*>(gate)[i];
      const float f = (q_row ? unit[h] : gate[2 * kChunk + i]) * (1.f / (kUnit * kUnit));
      float* const ax = reinterpret_cast<float*>(sm + P::kAx + h * P::kAxBytes) + tcol * kLd + i;
      float hi[16], lo[16];
      // e^(c_i - c_j) times the row: the sums in base 2, their low parts apart
#pragma unroll
      for (int k = 0; k < 16; ++k) {
        const int j = tcol + 2 * k;
        const float4 cj = c[k];
        const float2 e = unpack2(g[k]);
        const float a = exp2_fast((ci.x - cj.x) + (ci.y - cj.y)) * (f * e.x);
        const float b = exp2_fast((ci.x - cj.z) + (ci.y - cj.w)) * (f * e.y);
        if (q_row) {
          // C = e^(c_i - c_j) H_ij up to the diagonal: A operand in tensor memory, in two terms, two columns of C a cell
          uint32_t x0, x1;
          split2(j <= i ? a : 0.f, j + 1 <= i ? b : 0.f, x0, x1);
          hi[k] = __uint_as_float(x0), lo[k] = __uint_as_float(x1);
        } else {
          // A = beta_i e^(c_i - c_j) G_ij below it, transposed
          if (j < i) ax[2 * k * kLd] = a;
          if (j + 1 < i) ax[(2 * k + 1) * kLd] = b;
        }
      }
      if (q_row) {
        tmem_st16(ta + kTmC + h * 64 + tcol / 2, hi);
        tmem_st16(ta + kTmC + h * 64 + 32 + tcol / 2, lo);
      }
    }
    tmem_wait_st();
    tmem_fence_before();
  }
  __syncthreads();
  if (warp < 2 * nh) solve_columns(reinterpret_cast<float*>(sm + P::kAx + (warp >> 1) * P::kAxBytes), warp & 1, lane);
  __syncthreads();
  // M = X diag(beta): its largest entry, a bound of its rows' sums times the gates behind them, its image.
  // A thread has sixteen columns of row mi.  Rows of [M; N] change places with every chunk of the request, as [K; Q] do.
  const int mi = tid & 63, j0 = (tid >> 6) * 16;
  const int m_row = (chunk & 1) * kChunk, n_row = kChunk - m_row;
#pragma unroll 1
  for (int h = 0; h < nh; ++h) {
    const float* const ax = reinterpret_cast<const float*>(sm + P::kAx + h * P::kAxBytes) + mi * kLd + j0;
    const float* const beta = gates_of(h) + 2 * kChunk + j0;
    float m[16], big = 0.f, sum = 0.f;
#pragma unroll
    for (int k = 0; k < 16; k += 4) {
      const float4 a = *reinterpret_cast<const float4*>(ax + k), b = *reinterpret_cast<const float4*>(beta + k);
      m[k] = j0 + k <= mi ? a.x * b.x : 0.f;
      m[k + 1] = j0 + k + 1 <= mi ? a.y * b.y : 0.f;
      m[k + 2] = j0 + k + 2 <= mi ? a.z * b.z : 0.f;
      m[k + 3] = j0 + k + 3 <= mi ? a.w * b.w : 0.f;
    }
#pragma unroll
    for (int k = 0; k < 16; ++k) big = fmaxf(big, fabsf(m[k])), sum += fabsf(m[k]);
    big = warp_max(big);
    sum = warp_max(sum * gates_of(h)[3 * kChunk + mi]);
    if (lane == 0) red[h * 16 + warp] = big, red[h * 16 + 8 + warp] = sum;
    __syncthreads();
    big = sum = 0.f;
#pragma unroll
    for (int w = 0; w < kPrepWarps; w += 2) {
      big = fmaxf(big, fmaxf(red[h * 16 + w], red[h * 16 + w + 1]));
      sum += fmaxf(red[h * 16 + 8 + w], red[h * 16 + 8 + w + 1]);
    }
    float inv;
    const float sc = scale_for(big, inv);
    char* const ws_h = head_ws(h);
#pragma unroll
    for (int k = 0; k < 16; k += 8) {
      u64 v[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = mul2(pack2(m[k + 2 * e], m[k + 2 * e + 1]), pack2(sc, sc));
      uint4 hi, lo;
      split_pairs(v, hi, lo);
      const int at = image_at(mi, (j0 + k) >> 3, kChunk);
      char* const dst = sm + P::kM + h * 2 * P::kSq + at;
      *reinterpret_cast<uint4*>(dst) = hi;
      *reinterpret_cast<uint4*>(dst + P::kSq) = lo;
      *reinterpret_cast<uint4*>(ws_h + m_row * 128 + at) = hi;
      *reinterpret_cast<uint4*>(ws_h + 128 * 128 + m_row * 128 + at) = lo;
    }
    if (tid == 0) head_meta(h)[2 * kChunk + 1] = inv, head_meta(h)[2 * kChunk + 4] = sum, unit[kHeads + h] = inv;
  }
  fence_proxy_async();
  __syncthreads();
  // N = C M, by the warps that hold the rows of H
  if (q_row) {
    auto q_barrier = [] { asm volatile("bar.sync 1, 128;" ::: "memory"); };
#pragma unroll 1
    for (int h = 0; h < nh; ++h) {
      if (warp == 2 && elect_one()) {
        tmem_fence_after();
        const uint32_t d = tmem + kTmGram, a = tmem + kTmC + h * 64;
        const uint64_t b = umma_desc(smem_addr(sm + P::kM + h * 2 * P::kSq), 1024, 128), lo = P::kSq >> 4;
        const uint32_t id = idesc_f16(kChunk, false, true);
#pragma unroll
        for (int k = 0; k < 4; ++k) umma_f16_ts(d, a + 8 * k, b + k * (2048 >> 4), id, k > 0);
#pragma unroll
        for (int k = 0; k < 4; ++k) umma_f16_ts(d, a + 8 * k, b + lo + k * (2048 >> 4), id, 1);
#pragma unroll
        for (int k = 0; k < 4; ++k) umma_f16_ts(d, a + 32 + 8 * k, b + k * (2048 >> 4), id, 1);
        umma_commit(bar + 1);
      }
      __syncwarp();
      wait(1, h & 1);
      tmem_fence_after();
      u64 v[16];
      tmem_pairs(ta + kTmGram + tcol, *reinterpret_cast<u64(*)[8]>(v));
      tmem_pairs(ta + kTmGram + tcol + 16, *reinterpret_cast<u64(*)[8]>(v + 8));
      tmem_fence_before();
      float big = 0.f, sum = 0.f;
#pragma unroll
      for (int k = 0; k < 16; ++k) {
        const float2 f = unpack2(v[k]);
        big = fmaxf(big, fmaxf(fabsf(f.x), fabsf(f.y)));
        sum += fabsf(f.x) + fabsf(f.y);
      }
      big = warp_max(big);
      sum = warp_max(sum);
      if (lane == 0) red[64 + h * 16 + warp] = big, red[64 + h * 16 + 8 + warp] = sum;
      q_barrier();                                             // also: N of this head has been read
      const float* const rb = red + 64 + h * 16;
      big = fmaxf(fmaxf(rb[2], rb[3]), fmaxf(rb[6], rb[7]));
      sum = fmaxf(rb[10], rb[11]) + fmaxf(rb[14], rb[15]);     // the rows' halves lie in two warps
      const float inv = unit[kHeads + h] / unit[h];            // what N is known times
      float inv_n;
      const float sc = scale_for(big, inv_n);
      char* const ws_h = head_ws(h);
#pragma unroll
      for (int k = 0; k < 16; k += 4) {
#pragma unroll
        for (int e = 0; e < 4; ++e) v[k + e] = mul2(v[k + e], pack2(sc, sc));
        uint4 hi, lo;
        split_pairs(v + k, hi, lo);
        const int at = image_at(i, (tcol + 2 * k) >> 3, kChunk);
        *reinterpret_cast<uint4*>(ws_h + n_row * 128 + at) = hi;
        *reinterpret_cast<uint4*>(ws_h + 128 * 128 + n_row * 128 + at) = lo;
      }
      if (tid == 64) head_meta(h)[2 * kChunk + 2] = inv_n * inv, head_meta(h)[2 * kChunk + 6] = sum * inv;
    }
  }
  if (__syncthreads_or(late) && tid == 0) device_error(p.err, GDN_DEVERR_TIMEOUT, req.b);
  if (warp == 0) tmem_dealloc(tmem, kTmPrep);
}

// ---- the chunks of a head, one after another ------------------------------------------------------------------------

template <int DK, int NB>
struct Chain {
  // columns of a thread: with 16, twice as many warps share a step's latencies (32 warps and the issuing one would be
  // more than a CTA's 1024 threads)
  static constexpr int kCols = NB == 128 ? 32 : 16;
  static constexpr int kGroups = NB / kCols;                   // warpgroups
  static constexpr int kSoft = 128 * kGroups, kThreads = kSoft + 32, kWarps = 4 * kGroups;
  static constexpr int kImage = kChunk * DK * 2;               // K or Q, one term
  static constexpr int kKq = 0, kKqLo = 3 * kImage;            // K of even chunks | Q | K of odd chunks
  static constexpr int kMn = 6 * kImage, kMnLo = 128 * kChunk * 2;
  static constexpr int kS = kMn + 2 * kMnLo, kSLo = DK * NB * 2;
  static constexpr int kW = kS + 2 * kSLo, kWLo = kChunk * NB * 2;
  static constexpr int kBar = kW + 2 * kWLo;
  static constexpr int kMax = kBar + 8 * 10;                   // float [2][kWarps]: largest entries of T, of o
  // K^T is read as 128 rows of d_k: from its last core matrices up to 1536 bytes past the image, into the next place
  static constexpr int kTotal = kMax + 2 * kWarps * 4;
  static constexpr uint32_t kTmem = 3 * NB <= 128 ? 128 : 3 * NB <= 256 ? 256 : 512;
};
enum ChainBar { kKqFull, kMnFull, kSReady, kD1, kWReady, kD2, kUReady, kD3, kTmemAt };

constexpr float kRange = 0x1p-17f;   // bounds this far above the largest value still leave 2^-22 of it

// A chunk by the rule itself, with fp32 sums, from the state in its operand (S / scale, 22 bits): its outputs are written
// again and S is the state after it.  All threads of the warpgroups; rare and slow (some 0.1 ms).
template <int DK, int NB>
__device__ __noinline__ void again_by_token(const SeqParams& p, const SegReq& req, int vh, int row, bool has_row, int c0,
                                            int col0, int t0, float inv_s, const char* kq, const float* V, char* sm,
                                            float* S) {
  using L = Chain<DK, NB>;
  constexpr int CP = L::kCols;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  auto barrier = [] { asm volatile("bar.sync 1, %0;" ::"n"(L::kSoft) : "memory"); };
  auto term = [](const char* at) { return __half2float(*reinterpret_cast<const __half*>(at)); };
  float* const part = reinterpret_cast<float*>(sm + L::kW);     // [warps][p, r: CP each], then [warps] q.k
  float* const dots = part + L::kWarps * 2 * CP;
  for (int j = 0; j < CP; ++j) {
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
    for (int j = 0; j < CP; ++j) {
      S[j] *= g;
      float a = k * S[j], b = q * S[j];
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) a += __shfl_xor_sync(~0u, a, o), b += __shfl_xor_sync(~0u, b, o);
      if (lane == j) mine_p = a, mine_r = b;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) qk += __shfl_xor_sync(~0u, qk, o);
    if (lane < CP) {
      part[warp * 2 * CP + lane] = mine_p;
      part[warp * 2 * CP + CP + lane] = mine_r;
    }
    if (lane == 0) dots[warp] = qk;
    barrier();
    const int j = lane % CP;                                    // this lane's column
    const float* mine = part + (warp & ~3) * 2 * CP + j;
    qk = (dots[0] + dots[1]) + (dots[2] + dots[3]);
    const float pj = (mine[0] + mine[2 * CP]) + (mine[4 * CP] + mine[6 * CP]);
    const float rj = (mine[CP] + mine[3 * CP]) + (mine[5 * CP] + mine[7 * CP]);
    const float u = beta * (V[((col0 + c0 + j) / 4 * kChunk + t) * 4 + (j & 3)] - pj), o = p.q_scale * fmaf(qk, u, rj);
    for (int i = 0; i < CP; ++i) S[i] = fmaf(k, __shfl_sync(~0u, u, i), S[i]);
    if ((warp & 3) == 0 && lane < CP) {
      const long long at = ((req.start + static_cast<long long>(t0 + t)) * p.Hv + vh) * p.dv + col0 + c0 + j;
      if (p.out_dtype == GDN_DTYPE_BF16) static_cast<__nv_bfloat16*>(p.out)[at] = __float2bfloat16_rn(o);
      else static_cast<float*>(p.out)[at] = o;
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

  if (warp == L::kWarps) tmem_alloc(reinterpret_cast<uint32_t*>(bar + kTmemAt), L::kTmem);
  if (tid == 0) {
    mbar_init_n(bar + kKqFull, 1);
    mbar_init_n(bar + kMnFull, 1);
    mbar_init_n(bar + kSReady, L::kWarps);
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
  if (warp == L::kWarps) tmem_relinquish();
  bool late = false;
  // A wait that gave up is not repeated: the loops run to their end, the results are reported as lost.
  auto wait = [&](int which, int parity) {
    if (!late && !mbar_wait_quiet(bar + which, parity)) late = true;
  };

  if (stop) {
    // an earlier launch gave up: nothing is done
  } else if (warp == L::kWarps) {
    // The whole warp walks the loop and one elected lane issues: descriptors stay in uniform registers.
    auto load_k = [&](int i) {         // chunk i of the segment
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
    auto given_up = [&]() { return late = __any_sync(~0u, late); };
    if (elect_one()) {
      load_k(0);
      load_q(0);
      load_mn(0);
    }
    __syncwarp();
    const uint64_t s_b = umma_desc(smem_addr(sm + L::kS), 128, DK * 16);
    const uint64_t w_b = umma_desc(smem_addr(sm + L::kW), 128, kChunk * 16);
    const uint64_t mn_a = umma_desc(smem_addr(sm + L::kMn), 128, 1024);
    for (int i = 0; i < req.nc; ++i) {
      const int odd = (req.c0 + i) & 1, ph = i & 1;
      wait(kKqFull, ph);
      wait(kSReady, ph);
      if (given_up()) break;
      tmem_fence_after();
      if (elect_one()) {
        // rows 0 to 127: [K; Q], or [Q; K] in odd chunks
        product<DK / 16>(tmem, umma_desc(smem_addr(sm + L::kKq + odd * L::kImage), 128, DK * 16), s_b, L::kKqLo, L::kSLo, 256,
                         256, idesc_f16(NB, false, true));
        umma_commit(bar + kD1);
        if (i + 1 < req.nc) load_k(i + 1);
      }
      __syncwarp();
      wait(kD1, ph);
      if (i + 1 < req.nc && elect_one()) load_q(i + 1);
      __syncwarp();
      wait(kMnFull, ph);
      wait(kWReady, ph);
      if (given_up()) break;
      tmem_fence_after();
      if (elect_one()) {
        product<kChunk / 16>(tmem + NB, mn_a, w_b, L::kMnLo, L::kWLo, 256, 256, idesc_f16(NB, false, true));
        umma_commit(bar + kD2);
      }
      __syncwarp();
      wait(kD2, ph);
      if (i + 1 < req.nc && elect_one()) load_mn(i + 1);
      __syncwarp();
      wait(kUReady, ph);
      if (given_up()) break;
      tmem_fence_after();
      if (elect_one()) {
        product<kChunk / 16>(tmem + 2 * NB, umma_desc(smem_addr(sm + L::kKq + odd * 2 * L::kImage), DK * 16, 128), w_b, L::kKqLo,
                             L::kWLo, 2 * DK * 16, 256, idesc_f16(NB, true, true));
        umma_commit(bar + kD3);
      }
      __syncwarp();
    }
    wait(kD3, (req.nc - 1) & 1);
    if (late) {        // whatever was in flight has had twice the time that a wait gives it
      mbar_wait(bar + kKqFull, 0), mbar_wait(bar + kKqFull, 1), mbar_wait(bar + kMnFull, 0), mbar_wait(bar + kMnFull, 1);
    }
    __syncwarp();
  } else {
    constexpr int CP = L::kCols, kPairs = CP / 2;
    const int row = (warp & 3) * 32 + lane, c0 = (warp >> 2) * CP;            // lane of tensor memory, columns of the slice
    const uint32_t ta = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + c0;
    const bool has_row = row < DK;
    auto soft_barrier = [] { asm volatile("bar.sync 1, %0;" ::"n"(L::kSoft) : "memory"); };
    u64 S[kPairs];
    // the state before the segment: the call's, or what the segment before left
    {
      const float* src = req.c0 == 0 ? p.state_in : p.state_out;
#pragma unroll
      for (int j = 0; j < kPairs; ++j) S[j] = 0ull;
      if (src && has_row) {
        src += req.b * p.state_stride + (static_cast<long long>(vh) * DK + row) * p.dv + col0 + c0;
#pragma unroll
        for (int j = 0; j < kPairs; j += 2) {
          const float4 t = *reinterpret_cast<const float4*>(src + 2 * j);
          S[j] = pack2(t.x, t.y), S[j + 1] = pack2(t.z, t.w);
        }
      }
    }
    float smax, omax = 0.f, inv_s;
    // the largest entry of T, and of the chunk's o, over all threads
    auto find_maxima = [&]() {
      float big = 0.f;
#pragma unroll
      for (int j = 0; j < kPairs; ++j) big = abs_max(big, S[j]);
      big = warp_max(big);
      const float bigo = warp_max(omax);
      if (lane == 0) maxima[warp] = big, maxima[L::kWarps + warp] = bigo;
      soft_barrier();
      smax = warp_max(lane < L::kWarps ? maxima[lane] : 0.f);
      omax = warp_max(lane < L::kWarps ? maxima[L::kWarps + lane] : 0.f);
    };
    // packed pairs, scaled, into a two-term operand at `at`, whose groups of eight columns lie `step` bytes apart
    auto put = [&](const u64* x, float sc, char* at, int step, int lo_at) {
      const u64 sc2 = pack2(sc, sc);
#pragma unroll
      for (int j = 0; j < 8; j += 4) {
        u64 v[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = mul2(x[j + k], sc2);
        uint4 hi, lo;
        split_pairs(v, hi, lo);
        *reinterpret_cast<uint4*>(at + j / 4 * step) = hi;
        *reinterpret_cast<uint4*>(at + j / 4 * step + lo_at) = lo;
      }
    };
    auto put_state = [&]() {
      const float sc = scale_for(smax, inv_s);
      if (has_row) {
#pragma unroll
        for (int j = 0; j < CP; j += 16) put(S + j / 2, sc, sm + L::kS + ((c0 + j) >> 3) * DK * 16 + row * 16, DK * 16, L::kSLo);
      }
      fence_proxy_async();
      tmem_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar + kSReady);
    };
    u64 a[kPairs];                                             // v of a k row; the first part of o of a q row
    auto load_v = [&](int i) {
      const float4* V = reinterpret_cast<const float4*>(v_ws + i * slot_bytes + 4 * 128 * kChunk) + (col0 + c0) / 4 * kChunk + (row & 63);
#pragma unroll
      for (int j = 0; j < kPairs; j += 2) {
        const float4 f = __ldg(V + j / 2 * kChunk);
        a[j] = pack2(f.x, f.y), a[j + 1] = pack2(f.z, f.w);
      }
    };
    // Writes the warp's 32 rows of o from token t0 on.  Sixteen bytes of a row go to place row ^ unit of their unit's 512
    // bytes, so that neither rows nor units share banks; the units are the places of w that this warp itself writes.
    auto store_out = [&](int t0) {
      auto place = [&](int unit, int r) {                      // units: eight columns, high and low terms
        return sm + L::kW + (unit & 1) * L::kWLo + ((c0 >> 3) + (unit >> 1)) * kChunk * 16 + (row & 32) * 16 + (r ^ unit) * 16;
      };
      const bool bf16 = p.out_dtype == GDN_DTYPE_BF16;
      if (bf16) {
#pragma unroll
        for (int j = 0; j < kPairs; j += 4) {
          __nv_bfloat162 b[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float2 x = unpack2(a[j + k]);
            b[k] = __floats2bfloat162_rn(x.x, x.y);
          }
          *reinterpret_cast<uint4*>(place(j / 4, lane)) = *reinterpret_cast<uint4*>(b);
        }
      } else {
#pragma unroll
        for (int j = 0; j < kPairs; j += 2) {
          const float2 x = unpack2(a[j]), y = unpack2(a[j + 1]);
          *reinterpret_cast<float4*>(place(j / 2, lane)) = make_float4(x.x, x.y, y.x, y.y);
        }
      }
      __syncwarp();
      const int units = bf16 ? CP / 8 : CP / 4, size = bf16 ? 2 : 4;
      const int rows = 32 / units, unit = lane % units;
      for (int r = lane / units; r < 32; r += rows) {
        if (t0 + r < req.len) {
          const long long at = ((req.start + static_cast<long long>(t0 + r)) * p.Hv + vh) * p.dv + col0 + c0;
          *reinterpret_cast<uint4*>(static_cast<char*>(p.out) + at * size + unit * 16) = *reinterpret_cast<const uint4*>(place(unit, r));
        }
      }
      __syncwarp();
    };
    if ((row >> 6) == (req.c0 & 1)) load_v(0);
    find_maxima();
    put_state();
    for (int i = 0; i < req.nc; ++i) {
      const int odd = (req.c0 + i) & 1, ph = i & 1;
      const bool k_row = (row >> 6) == odd;                    // this thread's row is a token's k (else its q)
      const int t = row & 63;
      const float* meta = reinterpret_cast<const float*>(v_ws + i * slot_bytes + 4 * 128 * kChunk + kChunk * p.dv * 4);
      const float first = __ldg(meta + t), left = __ldg(meta + kChunk + t);
      const float4 m0 = __ldg(reinterpret_cast<const float4*>(meta + 2 * kChunk));
      const float4 m1 = __ldg(reinterpret_cast<const float4*>(meta + 2 * kChunk + 4));
      const float whole = m0.x, inv_m = m0.y, inv_n = m0.z, vmax = m0.w, mbound = m1.x, fmax_ = m1.y, nbound = m1.z;
      const float w_bound = (vmax + fmax_ * (DK == 128 ? 11.32f : DK == 64 ? 8.001f : 5.657f) * smax) * 1.001f;
      const float u_bound = mbound * w_bound * 1.001f;
      float inv_w, inv_u;
      const float sc_w = scale_for(w_bound, inv_w), sc_u = scale_for(u_bound, inv_u);
      const float f1 = first * (inv_s * (1.f / kUnit));
      char* const w_at = sm + L::kW + (c0 >> 3) * kChunk * 16 + t * 16;
      wait(kD1, ph);
      tmem_fence_after();
      if (k_row) {
        const u64 f = pack2(-f1, -f1);
#pragma unroll
        for (int j = 0; j < CP; j += 16) {
          u64 d[8];
          tmem_pairs(ta + j, d);
#pragma unroll
          for (int k = 0; k < 8; ++k) d[k] = fma2(f, d[k], a[j / 2 + k]);
          put(d, sc_w, w_at + (j >> 3) * kChunk * 16, kChunk * 16, L::kWLo);
        }
        fence_proxy_async();
        tmem_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar + kWReady);
      } else {
        const u64 f = pack2(f1 * p.q_scale, f1 * p.q_scale);
#pragma unroll
        for (int j = 0; j < CP; j += 16) {
          u64 d[8];
          tmem_pairs(ta + j, d);
#pragma unroll
          for (int k = 0; k < 8; ++k) a[j / 2 + k] = mul2(d[k], f);
        }
      }
      wait(kD2, ph);
      tmem_fence_after();
      if (k_row) {
        const float f = left * inv_m * inv_w * sc_u;
#pragma unroll
        for (int j = 0; j < CP; j += 16) {
          u64 d[8];
          tmem_pairs(ta + NB + j, d);
          put(d, f, w_at + (j >> 3) * kChunk * 16, kChunk * 16, L::kWLo);
        }
        fence_proxy_async();
        tmem_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar + kUReady);
      } else {
        const u64 f = pack2(inv_n * inv_w * p.q_scale, inv_n * inv_w * p.q_scale);
#pragma unroll
        for (int j = 0; j < CP; j += 16) {
          u64 d[8];
          tmem_pairs(ta + NB + j, d);
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            a[j / 2 + k] = fma2(f, d[k], a[j / 2 + k]);
            omax = abs_max(omax, a[j / 2 + k]);
          }
        }
      }
      wait(kD3, ph);
      tmem_fence_after();
      const u64 f3 = pack2(inv_u * (1.f / kUnit), inv_u * (1.f / kUnit)), whole2 = pack2(whole, whole);
#pragma unroll
      for (int j = 0; j < CP; j += 16) {
        u64 d[8];
        tmem_pairs(ta + 2 * NB + j, d);
#pragma unroll
        for (int k = 0; k < 8; ++k) S[j / 2 + k] = has_row ? fma2(whole2, S[j / 2 + k], mul2(f3, d[k])) : 0ull;
      }
      find_maxima();
      // Values far below what the bounds allow have lost their bits: the chunk is taken again, token by token.
      const float o_bound = nbound * w_bound * fabsf(p.q_scale);
      const bool again = u_bound * kRange > smax || o_bound * kRange > omax;
      if (again) {
        float s[CP];
        again_by_token<DK, NB>(p, req, vh, row, has_row, c0, col0, (req.c0 + i) * kChunk, inv_s, kq_ws + i * slot_bytes,
                               reinterpret_cast<const float*>(v_ws + i * slot_bytes + 4 * 128 * kChunk), sm, s);
#pragma unroll
        for (int j = 0; j < kPairs; ++j) S[j] = pack2(s[2 * j], s[2 * j + 1]);
        find_maxima();
      }
      omax = 0.f;
      if (i + 1 < req.nc) put_state();
      if (!k_row) {
        // o, in rows again: through the warp's own part of w's operand, which D3 was the last to read
        if (!again) store_out((req.c0 + i) * kChunk + (row & 32));
        if (i + 1 < req.nc) load_v(i + 1);                     // a q row is the next chunk's k row
      }
    }
    if (has_row) {
      float* dst = p.state_out + req.b * p.state_stride + (static_cast<long long>(vh) * DK + row) * p.dv + col0 + c0;
#pragma unroll
      for (int j = 0; j < kPairs; j += 2) {
        const float2 x = unpack2(S[j]), y = unpack2(S[j + 1]);
        *reinterpret_cast<float4*>(dst + 2 * j) = make_float4(x.x, x.y, y.x, y.y);
      }
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
  if (warp == L::kWarps) tmem_dealloc(tmem, L::kTmem);
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
  k<<<dim3(p.Hk, seg.slots, (p.Hv / p.Hk + kHeads - 1) / kHeads), kPrepThreads, Prep<DK>::kTotal, s>>>(p, seg, ws);
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
