// Prompts through one GDN layer in chunks of 64 tokens, on tcgen05.
//
// With c_i the cumulated log gates of a chunk, rows k_i, q_i, v_i and the state T before it:
//   A = (beta_i e^(c_i - c_j) k_i.k_j)_{j < i},   M = (1 + A)^-1 diag(beta),   N = (e^(c_i - c_j) q_i.k_j)_{j <= i} M,
//   w_i = v_i - e^(c_i) T^T k_i,   u = M w,   o_i = e^(c_i) T^T q_i + (N w)_i,
//   T' = e^(c_63) T + sum_i k_i (e^(c_63 - c_i) u_i)^T.
// Everything in the first line is independent of T: seq_keys_kernel (k, q and their products, once a k-head) and
// seq_values_kernel (gates, v, M and N of a v-head) compute it for many chunks at once, with the conv, the activation and the
// norms.  seq_chain_kernel then walks each head's chunks:
//   D1 = [K; Q] T   ->   w   ->   D2 = [M; N] w   ->   u, o   ->   D3 = K^T u   ->   T'
// with T in fp32 in registers, a row of d_k and 32 columns a thread.  Columns of d_v do not depend on each other.
//
// Precision: operands enter the products as two fp16 terms, x = hi + lo, and hi hi + hi lo + lo hi is accumulated in fp32:
// 22 bits of every element, half the tensor-core time of a tf32 split in three.  fp16's range is met by powers of two: k
// and q are normalised (2^12), M and N scaled by their largest entry, w and u by bounds that follow from those of T
// and v:  |w| <= max v + max e^c sqrt(dk) max T,  |u| <= max_i sum_j |M_ij| max w.  An element keeps 2^-23 of itself or
// 2^-40 of the bound, and the bounds lie some 2^6 above the values.  T' is handed on scaled by a bound as well,
// |T'| <= e^c max T + 64 max u, some 2^11 above it, and the largest entry is looked at afterwards: no warp waits for the
// others'.  Where a bound turns out to lie 2^17 above the largest entry of T' or of the chunk's o (values that shrink or grow
// by that much within 64 tokens), T' is handed on again, or the chunk is taken again, token by token; so are chunks in which
// products of gates, or M, grow (kMostGrowth).  Entries of T and v that are not finite count for no bound: they stay in their
// own column of d_v, as in the rule.
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
// What grows within a chunk and shrinks again keeps its rounding errors, in the triangular system's fp32 and in operands that
// are scaled by their largest entry, where the rule forgets them.  Chunks in which a product of gates or an entry of M is above
// this are taken token by token.  Gates up to 1 and beta in [0, 2] stay at 4 and below (u_i depends on w_j through
// beta_i k_i^T (1 - beta k k^T) .. k_j beta_j, whose factors have norms up to 1).  It costs four bits of fp32's 24.
constexpr float kMostGrowth = 4.f;         // log2

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
// D = A B in two-term operands, K elements deep: `kSteps` instructions of 16 each, three times.  Descriptors of the high
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
// The same where b's low terms are its columns n .. 2 n - 1: one instruction takes both (the high terms of A are read once
// instead of twice; an instruction of 64 columns is bound by those reads).  D is columns 0 .. n - 1 plus n .. 2 n - 1.
template <int kSteps, int n>
__device__ __forceinline__ void product_wide(uint32_t d, uint64_t a, uint64_t b, uint32_t a_lo, uint32_t a_step, uint32_t b_step,
                                             bool a_mn) {
  const uint64_t al = a_lo >> 4, as = a_step >> 4, bs = b_step >> 4;
#pragma unroll
  for (int i = 0; i < kSteps; ++i) umma_f16_ss(d, a + i * as, b + i * bs, idesc_f16(2 * n, a_mn, true), i > 0);
#pragma unroll
  for (int i = 0; i < kSteps; ++i) umma_f16_ss(d, a + al + i * as, b + i * bs, idesc_f16(n, a_mn, true), 1);
}
// Two values as fp16 pairs of their high and low terms.
__device__ __forceinline__ void split2(float x, float y, uint32_t& hi, uint32_t& lo) {
  const __half2 h = __floats2half2_rn(x, y);
  const float2 f = __half22float2(h);
  const __half2 l = __floats2half2_rn(x - f.x, y - f.y);
  hi = *reinterpret_cast<const uint32_t*>(&h);
  lo = *reinterpret_cast<const uint32_t*>(&l);
}
__device__ __forceinline__ u64 add2(u64 a, u64 b) {
  u64 d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
// Sixteen columns at `ta` and sixteen at `tb`, added.
__device__ __forceinline__ void tmem_sum_pairs(uint32_t ta, uint32_t tb, u64 (&v)[8]) {
  u64 w[8];
  asm volatile(
      "{\n"
      " .reg .b32 t<16>;\n"
      " .reg .b32 s<16>;\n"
      " tcgen05.ld.sync.aligned.32x32b.x16.b32 {t0, t1, t2, t3, t4, t5, t6, t7, t8, t9, t10, t11, t12, t13, t14, t15}, [%16];\n"
      " tcgen05.ld.sync.aligned.32x32b.x16.b32 {s0, s1, s2, s3, s4, s5, s6, s7, s8, s9, s10, s11, s12, s13, s14, s15}, [%17];\n"
      " tcgen05.wait::ld.sync.aligned;\n"
      " mov.b64 %0, {t0, t1};\n"
      " mov.b64 %1, {t2, t3};\n"
      " mov.b64 %2, {t4, t5};\n"
      " mov.b64 %3, {t6, t7};\n"
      " mov.b64 %4, {t8, t9};\n"
      " mov.b64 %5, {t10, t11};\n"
      " mov.b64 %6, {t12, t13};\n"
      " mov.b64 %7, {t14, t15};\n"
      " mov.b64 %8, {s0, s1};\n"
      " mov.b64 %9, {s2, s3};\n"
      " mov.b64 %10, {s4, s5};\n"
      " mov.b64 %11, {s6, s7};\n"
      " mov.b64 %12, {s8, s9};\n"
      " mov.b64 %13, {s10, s11};\n"
      " mov.b64 %14, {s12, s13};\n"
      " mov.b64 %15, {s14, s15};\n"
      "}"
      : "=l"(v[0]), "=l"(v[1]), "=l"(v[2]), "=l"(v[3]), "=l"(v[4]), "=l"(v[5]), "=l"(v[6]), "=l"(v[7]), "=l"(w[0]), "=l"(w[1]),
        "=l"(w[2]), "=l"(w[3]), "=l"(w[4]), "=l"(w[5]), "=l"(w[6]), "=l"(w[7])
      : "r"(ta), "r"(tb)
      : "memory");
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = add2(v[i], w[i]);
}
__device__ __forceinline__ void tmem_put_pairs(uint32_t ta, const u64* v) {   // complete at tmem_wait_st()
  float f[16];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float2 x = unpack2(v[i]);
    f[2 * i] = x.x, f[2 * i + 1] = x.y;
  }
  tmem_st16(ta, f);
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
constexpr float kInf = __builtin_huge_valf();
__device__ __forceinline__ float finite_max(float m, float x) { return fabsf(x) < kInf ? fmaxf(m, fabsf(x)) : m; }

// The same, where zeros count as something: 0 stays where nothing is finite.
__device__ __forceinline__ float finite_some(float m, float x) { return fabsf(x) < kInf ? fmaxf(m, fmaxf(fabsf(x), 0x1p-149f)) : m; }

// A bounded wait that leaves the issue slots to the working warps.
__device__ __forceinline__ bool mbar_wait_quiet(uint64_t* bar, uint32_t parity) {
  if (mbar_ready(bar, parity)) return true;
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
__device__ __forceinline__ void tmem_st8(uint32_t ta, const float (&v)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(ta), "f"(v[0]), "f"(v[1]),
               "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
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
__device__ __forceinline__ float warp_max(float x) {     // x >= 0 (a NaN counts as larger than all)
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
  if (t0 >= KT - 1 && t0 + kTok <= len) {
    const InT* at = x + static_cast<long long>(t0 - (KT - 1)) * p.x_row + ch;
#pragma unroll
    for (int i = 0; i < kTok + KT - 1; ++i, at += p.x_row) f[i] = raw4(at);
  } else {
#pragma unroll
    for (int i = 0; i < kTok + KT - 1; ++i)
      f[i] = raw4(x + static_cast<long long>(min(max(t0 + i - (KT - 1), 0), len - 1)) * p.x_row + ch);
  }
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

// Programmatic dependent launches: a kernel may start while the last CTAs of the one before finish, and waits for it (and all
// it waited for) where it reads that one's results.
__device__ __forceinline__ void start_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
// (Those are read by loads that the wait orders: not __ldg, which may be moved before it.)
__device__ __forceinline__ void wait_for_primary() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// ---- what does not depend on the state ------------------------------------------------------------------------------

constexpr int kPrepThreads = 256, kPrepWarps = kPrepThreads / 32;
constexpr int kLd = 68;                    // floats a row of A and X
constexpr int kRowLd = 132;                // of rows of q, k or v
constexpr int kRowBytes = kChunk * kRowLd * 4;
constexpr int kSq = kChunk * kChunk * 2;   // an fp16 image of a 64 x 64 matrix

// What a chunk and k-head's kernel holds: Kh Qh Kl Ql | rows | barrier
template <int DK>
struct PrepK {
  static constexpr int kImage = kChunk * DK * 2;              // one fp16 image of K or Q
  static constexpr int kRows = 4 * kImage, kBar = kRows + kRowBytes, kTotal = kBar + 32;
};
// A chunk and v-head's: rows of v, later A and X, and the images (high, low) of M in their place | gates | maxima | barrier
struct PrepV {
  static constexpr int kAx = 0, kM = kChunk * kLd * 4;
  static constexpr int kEnd = kRowBytes > kM + 2 * kSq ? kRowBytes : kM + 2 * kSq;
  static constexpr int kGate = kEnd;                          // float2 [64] log2 of the cumulated gates (high, low part), beta [64], left [64]
  static constexpr int kRed = kGate + 4 * kChunk * 4;         // float [48]
  static constexpr int kBar = kRed + 48 * 4, kTotal = kBar + 32;
  static constexpr uint32_t kTmN = 0, kTmC = 64, kTmem = 128;   // columns of tensor memory: N | C
};

// 16-byte places of an fp16 image of `width` columns: row r, columns 8 c ..
__device__ __forceinline__ int image_at(int r, int c, int width) { return (r >> 3) * width * 16 + c * 128 + (r & 7) * 16; }

// Where a CTA's chunk is: request, rows, window, and the chunk's places in the workspace.
template <typename InT>
struct Place {
  SegReq req;
  int chunk, t0, len;
  const InT* x;
  const float* win;
  char* kq;       // of k-head 0; seq_kq_bytes apart
  char* v;        // of v-head 0; seq_v_bytes apart
  __device__ __forceinline__ Place(const SeqParams& p, const Segment& seg, char* ws, int slot) {
    int ri = 0;
    while (ri + 1 < seg.n && slot >= seg.r[ri + 1].slot0) ++ri;
    req = seg.r[ri];
    chunk = req.c0 + slot - req.slot0, t0 = chunk * kChunk, len = req.len;
    x = static_cast<const InT*>(p.x) + static_cast<long long>(req.start) * p.x_row;
    win = p.conv_in ? p.conv_in + req.b * p.conv_stride : nullptr;
    kq = ws + slot * seq_slot_bytes(p.Hk, p.Hv, p.dk, p.dv);
    v = kq + p.Hk * seq_kq_bytes(p.dk);
  }
};

// Conv and activation of the chunk's 64 tokens in `width` channels from ch on, into rows; norm as well where kNorm.
// A lane takes four channels of kTok adjacent tokens, a warp eight tokens.  Returns the warp's largest entry.
template <bool kNorm, int kTok, int KT, typename InT>
__device__ __forceinline__ float conv_rows(const SeqParams& p, const Place<InT>& at, int width, int ch, float* rows) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, lanes = width / 4, sub = lane / lanes, cl = (lane % lanes) * 4;
  float most = 0.f;
#pragma unroll 1
  for (int t = kTok * sub; t - kTok * sub < 8; t += lanes == 32 ? kTok : 8) {
    const int first = warp * 8 + t;
    float4 y[kTok];
#pragma unroll
    for (int i = 0; i < kTok; ++i) y[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (t < 8) conv_tokens<InT, KT, kTok>(p, at.x, at.win, at.t0 + first, at.len, ch + cl, y);
#pragma unroll
    for (int i = 0; i < kTok; ++i) {
      if (kNorm) {
        float ss = fmaf(y[i].x, y[i].x, fmaf(y[i].y, y[i].y, fmaf(y[i].z, y[i].z, y[i].w * y[i].w)));
        for (int o = lanes / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(~0u, ss, o);
        const float f = at.t0 + first + i < at.len ? rsqrtf(ss + p.l2_eps) * kUnit : 0.f;
        y[i] = make_float4(y[i].x * f, y[i].y * f, y[i].z * f, y[i].w * f);
      }
      if (t < 8) {
        *reinterpret_cast<float4*>(rows + (first + i) * kRowLd + cl) = y[i];
        if (!kNorm) most = fmaxf(most, fmaxf(fmaxf(fabsf(y[i].x), fabsf(y[i].y)), fmaxf(fabsf(y[i].z), fabsf(y[i].w))));
      }
    }
  }
  if (!kNorm && most == kInf) {
    most = 0.f;
    for (int t = kTok * sub; t < 8; t += lanes == 32 ? kTok : 8)
      for (int i = 0; i < 4 * kTok; ++i) most = finite_max(most, rows[(warp * 8 + t + i / 4) * kRowLd + cl + i % 4]);
  }
  __syncwarp();
  return kNorm ? 0.f : warp_max(most);
}

// X = (1 + A)^-1 for strictly lower A.  ax[j][i] (kLd floats a row) holds A_ij in i > j; X_kj goes to ax[k][j], j <= k,
// which A leaves free.  First the diagonal blocks of 32, a warp each: lane = column, forward substitution by blocks of 16
// rows; then X21 = -X22 (A21 X11) by all warps, a tile of 16 x 8 each, through T = A21 X11 in tmp (its own memory).
__device__ __forceinline__ void solve_block(float* ax, int half, int lane) {
  const int col = half * 32 + lane;
#pragma unroll 1
  for (int bi = 2 * half; bi < 2 * half + 2; ++bi) {
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
// c (16 x 8) += a (16 x 8) b (8 x 8) with both in two tf32 terms: a tile of 1024 multiply-adds is too small for tcgen05, whose
// operands would have to be laid out and results fetched from tensor memory.
__device__ __forceinline__ void mma_tf32(float (&c)[4], const uint32_t (&a)[4], const uint32_t (&b)[2]) {
  asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}
__device__ __forceinline__ void mma_exact(float (&c)[4], const float (&a)[4], const float (&b)[2]) {
  uint32_t ah[4], al[4], bh[2], bl[2];
#pragma unroll
  for (int i = 0; i < 4; ++i) ah[i] = __float_as_uint(tf32_hi(a[i])), al[i] = __float_as_uint(tf32_lo(a[i]));
#pragma unroll
  for (int i = 0; i < 2; ++i) bh[i] = __float_as_uint(tf32_hi(b[i])), bl[i] = __float_as_uint(tf32_lo(b[i]));
  mma_tf32(c, al, bl);             // (the terms are cut off, not rounded: their product has a sign and counts)
  mma_tf32(c, al, bh);
  mma_tf32(c, ah, bl);
  mma_tf32(c, ah, bh);
}
__device__ __forceinline__ void solve(float* ax, float* tmp, int warp, int lane) {
  if (warp < 2) solve_block(ax, warp, lane);
  __syncthreads();
  // a warp takes rows m0 .. and columns n0 .. of the lower left block
  const int m0 = 16 * (warp & 1), n0 = 8 * (warp >> 1), g = lane >> 2, q = lane & 3;
  float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int k = 0; k < 32; k += 8) {                // T = A21 X11
    if (k + 7 < n0) continue;                      // above X11's diagonal
    const float* a = ax + (k + q) * kLd;
    const float av[4] = {a[32 + m0 + g], a[32 + m0 + g + 8], a[4 * kLd + 32 + m0 + g], a[4 * kLd + 32 + m0 + g + 8]};
    const float bv[2] = {n0 + g <= k + q ? a[n0 + g] : 0.f, n0 + g <= k + q + 4 ? a[4 * kLd + n0 + g] : 0.f};
    mma_exact(c, av, bv);
  }
  constexpr int kT = 40;                           // floats a row of T: the reads below touch all banks once
  *reinterpret_cast<float2*>(tmp + (m0 + g) * kT + n0 + 2 * q) = make_float2(c[0], c[1]);
  *reinterpret_cast<float2*>(tmp + (m0 + g + 8) * kT + n0 + 2 * q) = make_float2(c[2], c[3]);
  __syncthreads();
  c[0] = c[1] = c[2] = c[3] = 0.f;
#pragma unroll
  for (int k = 0; k < 32; k += 8) {                // X22 T
    if (k > m0 + 15) continue;                     // above X22's diagonal
    const float* a = ax + (32 + m0 + g) * kLd + 32 + k + q;
    const int d = m0 + g - k - q;                  // how far the first entry is below the diagonal
    const float av[4] = {d >= 0 ? a[0] : 0.f, d + 8 >= 0 ? a[8 * kLd] : 0.f, d - 4 >= 0 ? a[4] : 0.f, d + 4 >= 0 ? a[8 * kLd + 4] : 0.f};
    const float bv[2] = {tmp[(k + q) * kT + n0 + g], tmp[(k + q + 4) * kT + n0 + g]};
    mma_exact(c, av, bv);
  }
  float* const x = ax + (32 + m0 + g) * kLd + n0 + 2 * q;
  *reinterpret_cast<float2*>(x) = make_float2(-c[0], -c[1]);
  *reinterpret_cast<float2*>(x + 8 * kLd) = make_float2(-c[2], -c[3]);
  __syncthreads();
}

// k and q of a chunk and k-head: rows, two-term images, Gram matrices (K K^T and Q K^T in one 128 x 64 product).
//
// Bound: the latencies of a CTA's five steps (rows from memory, conv, images, product, results) with two CTAs an SM, whose
// shared memory the images and the rows in 32 bits fill; 128 chunks of 16 heads of 128 take 86 us, 2.4 TB/s, 41% of the issue
// slots.  (Rows in the places of images that are not written yet leave room for three CTAs, at 80 registers: 3% off 32 prompts,
// but 4% more for a prompt of 70 tokens and 6% for heads of 64.)
template <typename InT, int DK, int KT>
__global__ void __launch_bounds__(kPrepThreads, 2)
seq_keys_kernel(const SeqParams p, const __grid_constant__ Segment seg, char* ws) {
  using P = PrepK<DK>;
  extern __shared__ __align__(128) char sm[];
  float* rows = reinterpret_cast<float*>(sm + P::kRows);
  uint64_t* bar = reinterpret_cast<uint64_t*>(sm + P::kBar);
  uint32_t* tmem_at = reinterpret_cast<uint32_t*>(bar + 1);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, kh = blockIdx.x;
  const Place<InT> at(p, seg, ws, blockIdx.y);
  char* const out = at.kq + kh * seq_kq_bytes(DK);
  const bool aborted = launch_aborted(p.err);
  if (warp == 0) tmem_alloc(tmem_at, kChunk);
  if (tid == 0) mbar_init(bar);
  const bool stop = __syncthreads_or(aborted);
  if (warp == 0) tmem_relinquish();
  start_dependents();
  const uint32_t tmem = *tmem_at;
  bool late = false;
  if (!stop) {
#pragma unroll 1
    for (int kind = 0; kind < 2; ++kind) {         // k, q
      conv_rows<true, DK == 128 ? 8 : 4, KT>(p, at, DK, ((kind == 0 ? p.Hk : 0) + kh) * DK, rows);
      __syncthreads();
      const int t = tid & 63;
#pragma unroll
      for (int c = 0; c < DK / 8; c += kPrepThreads / 64) {
        const int cc = c + (tid >> 6);
        const ulonglong2* src = reinterpret_cast<const ulonglong2*>(rows + t * kRowLd + 8 * cc);
        const ulonglong2 v0 = src[0], v1 = src[1];
        const u64 v[4] = {v0.x, v0.y, v1.x, v1.y};
        uint4 hi, lo;
        split_pairs(v, hi, lo);
        const int to = image_at(t, cc, DK);
        *reinterpret_cast<uint4*>(sm + kind * P::kImage + to) = hi;
        *reinterpret_cast<uint4*>(sm + (kind + 2) * P::kImage + to) = lo;
        *reinterpret_cast<uint4*>(out + 2 * kind * P::kImage + to) = hi;
        *reinterpret_cast<uint4*>(out + (2 * kind + 1) * P::kImage + to) = lo;
      }
      fence_proxy_async();
      __syncthreads();
    }
    // G = K K^T (lanes 0 to 63) and H = Q K^T
    if (warp == 0) {
      if (elect_one()) {
        const uint64_t a = umma_desc(smem_addr(sm), 128, DK * 16);
        product<DK / 16>(tmem, a, a, 2 * P::kImage, 2 * P::kImage, 256, 256, idesc_f16(kChunk, false, false));
        umma_commit(bar);
      }
      __syncwarp();
    }
    late = !mbar_wait_quiet(bar, 0);
    tmem_fence_after();
    // four columns of all rows together, [16][64][4]: G, then H
    const int row = (warp & 3) * 32 + lane, col = (warp >> 2) * 32;
    float4* const gram = reinterpret_cast<float4*>(out + 4 * P::kImage) + (row >> 6) * (kChunk / 4 * kChunk) + (row & 63);
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      u64 v[8];
      tmem_pairs(tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + col + 16 * half, v);
#pragma unroll
      for (int k = 0; k < 8; k += 2) {
        const float2 a = unpack2(v[k]), b = unpack2(v[k + 1]);
        constexpr float f = 1.f / (kUnit * kUnit);
        gram[((col + 16 * half) / 4 + k / 2) * kChunk] = make_float4(a.x * f, a.y * f, b.x * f, b.y * f);
      }
    }
    tmem_fence_before();
  }
  if (__syncthreads_or(late) && tid == 0) device_error(p.err, GDN_DEVERR_TIMEOUT, at.req.b);
  if (warp == 0) tmem_dealloc(tmem, kChunk);
}

// v, the gates, M and N of a chunk and v-head.
//
// (1 + A)^-1 by substitution in blocks: two 32 x 32 triangles, a warp each, and the block below them as a product of three on
// mma.sync: tiles of 16 x 8 straight from and into A's rows in shared memory, where tcgen05 would want images, tensor memory
// and two barriers for two products of 32 x 32 x 32.  N = C M is on tcgen05.  Bound: instruction issue (57% of the slots; the
// rest goes with the barriers between the steps); 128 chunks of 48 heads take 201 us.  The 64 registers that let four CTAs share
// an SM spill some 110 bytes a thread, with more than four taps 540 to 680.
template <typename InT, int KT>
__global__ void __launch_bounds__(kPrepThreads, 4)
seq_values_kernel(const SeqParams p, const __grid_constant__ Segment seg, char* ws) {
  using P = PrepV;
  extern __shared__ __align__(128) char sm[];
  float* rows = reinterpret_cast<float*>(sm);
  float* ax = reinterpret_cast<float*>(sm + P::kAx);
  float* gate = reinterpret_cast<float*>(sm + P::kGate);
  float* red = reinterpret_cast<float*>(sm + P::kRed);
  uint64_t* bar = reinterpret_cast<uint64_t*>(sm + P::kBar);
  uint32_t* tmem_at = reinterpret_cast<uint32_t*>(bar + 1);
  float* unit = reinterpret_cast<float*>(bar + 2);             // scale of C, log2 of the largest product of gates
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, vh = blockIdx.x, dv = p.dv;
  const Place<InT> at(p, seg, ws, blockIdx.y);
  const float* const grams = reinterpret_cast<const float*>(at.kq + vh / (p.Hv / p.Hk) * seq_kq_bytes(p.dk) + 4 * kChunk * p.dk * 2);
  char* const out = at.v + vh * seq_v_bytes(dv);
  float4* const V = reinterpret_cast<float4*>(out + 4 * 128 * kChunk);
  float* const meta = reinterpret_cast<float*>(V + dv / 4 * kChunk);
  const bool aborted = launch_aborted(p.err);
  if (warp == 0) tmem_alloc(tmem_at, P::kTmem);
  if (tid == 0) mbar_init(bar);
  const bool stop = __syncthreads_or(aborted);
  if (warp == 0) tmem_relinquish();
  start_dependents();
  const uint32_t tmem = *tmem_at;
  bool late = false;
  if (!stop) {
    // The raw rows on their way into L2, and two tokens' gates for each lane of the last warp.
    if (tid < kChunk + 3) {
      const int t = at.t0 + tid - 3;
      if (t >= 0 && t < at.len) prefetch_l2(at.x + static_cast<long long>(t) * p.x_row + 2 * p.Hk * p.dk + vh * dv, dv * sizeof(InT));
    }
    float lg[2] = {0.f, 0.f}, be[2] = {0.f, 0.f};
    if (warp == kPrepWarps - 1) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int t = at.t0 + 2 * lane + k;
        if (t < at.len) {
          const long long from = (at.req.start + static_cast<long long>(t)) * p.gate_row + vh;
          be[k] = load_f(static_cast<const InT*>(p.beta) + from);
          lg[k] = load_f(static_cast<const InT*>(p.log_g) + from);
          lg[k] = lg[k] < kGateFloor ? kGateFloor : lg[k];
        }
      }
    }
    // v: rows, then four columns of all tokens together, [dv / 4][64][4]
    {
      float most = conv_rows<false, 4, KT>(p, at, dv, 2 * p.Hk * p.dk + vh * dv, rows);
      if (lane == 0) red[warp] = most;
    }
    __syncthreads();
    if (warp == kPrepWarps - 1) {
      // the gates meanwhile: cumulated in 64 bits and base 2, kept as two floats
      double c[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        c[k] = static_cast<double>(lg[k]) * 1.4426950408889634;
        gate[2 * kChunk + 2 * lane + k] = be[k];
      }
      c[1] += c[0];
      double sum = c[1];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const double s = __shfl_up_sync(~0u, sum, o);
        if (lane >= o) sum += s;
      }
      const double before = sum - c[1], total = __shfl_sync(~0u, sum, 31);
      // the largest product of gates in a row: how far a sum lies above the least one before it
      const float s0 = static_cast<float>(before + c[0]), s1 = static_cast<float>(sum);
      float least = fminf(s0, s1);
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const float s = __shfl_up_sync(~0u, least, o);
        if (lane >= o) least = fminf(least, s);
      }
      least = __shfl_up_sync(~0u, least, 1);
      least = lane == 0 ? 0.f : fminf(least, 0.f);
      const float growth = warp_max(fmaxf(fmaxf(s0 - least, s1 - fminf(least, s0)), 0.f));
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
        // no product of gates is above 2^growth (1 unless a log gate is above 0)
        unit[0] = exp2f(floorf(11.f - fminf(growth, kMostGrowth)));
        unit[1] = growth;
      }
    } else {
#pragma unroll 4
      for (int c = tid; c < dv / 4 * kChunk; c += kPrepThreads - 32)
        V[c] = *reinterpret_cast<const float4*>(rows + (c & 63) * kRowLd + (c >> 6) * 4);
      if (tid == 0) {
        float most = 0.f;
        for (int w = 0; w < kPrepWarps; ++w) most = fmaxf(most, red[w]);
        meta[2 * kChunk + 3] = most;
      }
    }
    __syncthreads();                               // A takes the rows' place
    wait_for_primary();                            // the Gram matrices
    // A thread has 32 entries of a row of G (warps 0, 1, 4, 5) or H (the others).
    const int trow = (warp & 3) * 32 + lane, tcol = (warp >> 2) * 32, i = trow & 63;
    const bool q_row = trow >= kChunk;
    const uint32_t ta = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    {
      const float4* g = reinterpret_cast<const float4*>(grams) + (q_row ? kChunk / 4 * kChunk : 0) + tcol / 4 * kChunk + i;
      const float4* const c = reinterpret_cast<const float4*>(gate) + tcol / 2;     // two tokens' sums
      const float2 ci = reinterpret_cast<const float2*>(gate)[i];
      const float f = q_row ? *unit : gate[2 * kChunk + i];
      // e^(c_i - c_j) times the row: the sums in base 2, their low parts apart
      auto decayed = [&](float4 cj, float x, float y, float& a, float& b) {
        a = exp2_fast((ci.x - cj.x) + (ci.y - cj.y)) * (f * x);
        b = exp2_fast((ci.x - cj.z) + (ci.y - cj.w)) * (f * y);
      };
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        float4 e[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) e[k] = __ldcg(g + (4 * half + k) * kChunk);
        float hi[8], lo[8];
        if (tcol + 16 * half > ((warp & 1) * 32 + 31)) {       // all above the diagonal
#pragma unroll
          for (int k = 0; k < 8; ++k) hi[k] = lo[k] = 0.f;
        } else
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int j = tcol + 16 * half + 4 * k;
          float a[4];
          decayed(c[8 * half + 2 * k], e[k].x, e[k].y, a[0], a[1]);
          decayed(c[8 * half + 2 * k + 1], e[k].z, e[k].w, a[2], a[3]);
          if (q_row) {
            // C = e^(c_i - c_j) H_ij up to the diagonal: A operand in tensor memory, in two terms, two columns of C a cell
#pragma unroll
            for (int n = 0; n < 2; ++n) {
              uint32_t x0, x1;
              split2(j + 2 * n <= i ? a[2 * n] : 0.f, j + 2 * n + 1 <= i ? a[2 * n + 1] : 0.f, x0, x1);
              hi[2 * k + n] = __uint_as_float(x0), lo[2 * k + n] = __uint_as_float(x1);
            }
          } else {
            // A = beta_i e^(c_i - c_j) G_ij below it, transposed
#pragma unroll
            for (int n = 0; n < 4; ++n)
              if (j + n < i) ax[(j + n) * kLd + i] = a[n];
          }
        }
        if (q_row) {
          tmem_st8(ta + P::kTmC + tcol / 2 + 8 * half, hi);
          tmem_st8(ta + P::kTmC + 32 + tcol / 2 + 8 * half, lo);
        }
      }
      tmem_wait_st();
      tmem_fence_before();
    }
    __syncthreads();
    solve(ax, reinterpret_cast<float*>(sm + P::kM), warp, lane);
    // M = X diag(beta): its largest entry, a bound of its rows' sums times the gates behind them, its image.
    // A thread has sixteen columns of row mi.  Rows of [M; N] change places with every chunk of the request, as [K; Q] do.
    const int mi = tid & 63, j0 = (tid >> 6) * 16;
    const int m_row = (at.chunk & 1) * kChunk, n_row = kChunk - m_row;
    float inv_m;
    {
      float m[16], big = 0.f, sum = 0.f;
#pragma unroll
      for (int k = 0; k < 16; k += 4) {
        const float4 a = *reinterpret_cast<const float4*>(ax + mi * kLd + j0 + k), b = *reinterpret_cast<const float4*>(gate + 2 * kChunk + j0 + k);
        m[k] = j0 + k <= mi ? a.x * b.x : 0.f;
        m[k + 1] = j0 + k + 1 <= mi ? a.y * b.y : 0.f;
        m[k + 2] = j0 + k + 2 <= mi ? a.z * b.z : 0.f;
        m[k + 3] = j0 + k + 3 <= mi ? a.w * b.w : 0.f;
      }
#pragma unroll
      for (int k = 0; k < 16; ++k) big = fmaxf(big, fabsf(m[k])), sum += fabsf(m[k]);
      big = warp_max(big);
      sum = warp_max(sum * gate[3 * kChunk + mi]);
      if (lane == 0) red[8 + warp] = big, red[16 + warp] = sum;
      __syncthreads();
      big = sum = 0.f;
#pragma unroll
      for (int w = 0; w < kPrepWarps; w += 2) {
        big = fmaxf(big, fmaxf(red[8 + w], red[9 + w]));
        sum += fmaxf(red[16 + w], red[17 + w]);
      }
      const float sc = scale_for(big, inv_m);
#pragma unroll
      for (int k = 0; k < 16; k += 8) {
        u64 v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = mul2(pack2(m[k + 2 * e], m[k + 2 * e + 1]), pack2(sc, sc));
        uint4 hi, lo;
        split_pairs(v, hi, lo);
        const int to = image_at(mi, (j0 + k) >> 3, kChunk);
        *reinterpret_cast<uint4*>(sm + P::kM + to) = hi;
        *reinterpret_cast<uint4*>(sm + P::kM + kSq + to) = lo;
        *reinterpret_cast<uint4*>(out + m_row * 128 + to) = hi;
        *reinterpret_cast<uint4*>(out + 128 * 128 + m_row * 128 + to) = lo;
      }
      if (tid == 0) {
        meta[2 * kChunk + 1] = inv_m, meta[2 * kChunk + 4] = sum;
        meta[2 * kChunk + 7] = unit[1] > kMostGrowth || big > exp2f(kMostGrowth) ? 1.f : 0.f;
      }
    }
    fence_proxy_async();
    __syncthreads();
    // N = C M
    if (warp == 0) {
      if (elect_one()) {
        tmem_fence_after();
        const uint32_t d = tmem + P::kTmN, a = tmem + P::kTmC;
        const uint64_t b = umma_desc(smem_addr(sm + P::kM), 1024, 128), lo = kSq >> 4;
        const uint32_t id = idesc_f16(kChunk, false, true);
#pragma unroll
        for (int k = 0; k < 4; ++k) umma_f16_ts(d, a + 8 * k, b + k * (2048 >> 4), id, k > 0);
#pragma unroll
        for (int k = 0; k < 4; ++k) umma_f16_ts(d, a + 8 * k, b + lo + k * (2048 >> 4), id, 1);
#pragma unroll
        for (int k = 0; k < 4; ++k) umma_f16_ts(d, a + 32 + 8 * k, b + k * (2048 >> 4), id, 1);
        umma_commit(bar);
      }
      __syncwarp();
    }
    late = !mbar_wait_quiet(bar, 0);
    tmem_fence_after();
    if (q_row) {                                   // N is in the lanes of H's rows
      u64 v[16];
      tmem_pairs(ta + P::kTmN + tcol, *reinterpret_cast<u64(*)[8]>(v));
      tmem_pairs(ta + P::kTmN + tcol + 16, *reinterpret_cast<u64(*)[8]>(v + 8));
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
      if (lane == 0) red[24 + warp] = big, red[32 + warp] = sum;
      asm volatile("bar.sync 1, 128;" ::: "memory");
      big = fmaxf(fmaxf(red[26], red[27]), fmaxf(red[30], red[31]));
      sum = fmaxf(red[34], red[35]) + fmaxf(red[38], red[39]);   // the rows' halves lie in two warps
      const float inv = inv_m / *unit;             // what N is known times
      float inv_n;
      const float sc = scale_for(big, inv_n);
#pragma unroll
      for (int k = 0; k < 16; k += 4) {
#pragma unroll
        for (int e = 0; e < 4; ++e) v[k + e] = mul2(v[k + e], pack2(sc, sc));
        uint4 hi, lo;
        split_pairs(v + k, hi, lo);
        const int to = image_at(i, (tcol + 2 * k) >> 3, kChunk);
        *reinterpret_cast<uint4*>(out + n_row * 128 + to) = hi;
        *reinterpret_cast<uint4*>(out + 128 * 128 + n_row * 128 + to) = lo;
      }
      if (tid == 64) meta[2 * kChunk + 2] = inv_n * inv, meta[2 * kChunk + 6] = sum * inv;
    }
  }
  if (stop) wait_for_primary();
  if (__syncthreads_or(late) && tid == 0) device_error(p.err, GDN_DEVERR_TIMEOUT, at.req.b);
  if (warp == 0) tmem_dealloc(tmem, P::kTmem);
}

// ---- the chunks of a head, one after another ------------------------------------------------------------------------

// Bound: the way from one chunk to the next.  Its three products, T's and w's conversion to operands and the six hand-overs
// between tensor cores and threads take 3.1 us for 64 columns (tensor pipe 45% busy by the two groups together: a product with
// few columns runs at the rate at which A, 128 rows, is read from shared memory; issue 35%).  All 128 columns of a head in a CTA
// would halve the reading of K, Q, M and N, but take 9.3 us a chunk and leave half the SMs without work where requests are few.
template <int DK, int NB>
struct Chain {
  // Two groups of columns take turns at the tensor cores: one's products run while the other's threads work.
  static constexpr int kTurns = 2, kN = NB / kTurns;           // columns of a group
  static constexpr int kCols = 16;                             // of a thread
  static constexpr int kGroups = NB / kCols;                   // warpgroups
  static constexpr int kThreads = 128 * kGroups, kWarps = 4 * kGroups;
  static constexpr int kTurnWarps = kWarps / kTurns;
  static constexpr int kImage = kChunk * DK * 2;               // K or Q, one term
  static constexpr int kKq = 0, kKqLo = 3 * kImage;            // K of even chunks | Q | K of odd chunks
  static constexpr int kMn = 6 * kImage, kMnLo = 128 * kChunk * 2;
  // operands of a group: T [high | low], w or u [high | low]
  static constexpr int kS = kMn + 2 * kMnLo, kSLo = DK * kN * 2, kSTurn = 2 * kSLo;
  static constexpr int kW = kS + kTurns * kSTurn, kWLo = kChunk * kN * 2, kWTurn = 2 * kWLo;
  static constexpr int kMeta = kW + kTurns * kWTurn;           // two chunks' gates and bounds
  static constexpr int kMetaBytes = kSeqMeta * 4;
  static constexpr int kBar = kMeta + 2 * kMetaBytes;
  static constexpr int kCount = kBar + 8 * 16;                 // int [16]: arrivals
  static constexpr int kMax = kCount + 4 * 16;                 // float [2 chunks][groups][T, o][kTurnWarps]: largest entries
  // K^T is read as 128 rows of d_k: from its last core matrices up to 1536 bytes past the image, into the next place
  static constexpr int kTotal = kMax + 2 * 2 * kWarps * 4;
  // tensor memory of a group: D1 and later D3 | D2, high and low terms' products side by side
  static constexpr uint32_t kD = 2 * kN, kTmem = kTurns * 2 * kD < 32 ? 32 : kTurns * 2 * kD;
};

// kMetaFull: one for even and one for odd chunks (the copy for a chunk may be under way while the other group has still to look
// at the chunk before); the others from kD1 on: one a group of columns
enum ChainBar { kKqFull, kMnFull, kTmemAt, kMetaFull = 4, kD1 = 6, kD2 = 8, kD3 = 10, kMeet = 12 };
enum ChainCount { kSDone = 0, kWDone = 2, kUDone = 4 };                               // warps of a group
constexpr float kRange = 0x1p-17f;   // bounds this far above the largest value still leave 2^-22 of it

// A chunk by the rule itself, with fp32 sums, from the state S before it: its outputs are written again and S is the state
// after it.  All threads of a group; rare and slow (some 0.1 ms).
template <int DK, int NB>
__device__ __noinline__ void again_by_token(const SeqParams& p, const SegReq& req, int vh, int row, bool has_row, int g,
                                            int gw, int c0, int t0, const char* kq, const float* V,
                                            char* sm, float* S, int& meetings, bool& late) {
  using L = Chain<DK, NB>;
  constexpr int CP = L::kCols;
  const int lane = threadIdx.x & 31;
  uint64_t* const meet = reinterpret_cast<uint64_t*>(sm + L::kBar) + kMeet + g;
  auto barrier = [&] {
    __syncwarp();
    if (lane == 0) mbar_arrive(meet);
    if (!late && !mbar_wait_quiet(meet, meetings & 1)) late = true;
    ++meetings;
  };
  auto term = [](const char* at) { return __half2float(*reinterpret_cast<const __half*>(at)); };
  float* const part = reinterpret_cast<float*>(sm + L::kW + g * L::kWTurn);   // [warps][p, r: CP each], then [warps] q.k
  float* const dots = part + L::kTurnWarps * 2 * CP;
  barrier();                                                    // the group's o are written, w's place is free
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
      part[gw * 2 * CP + lane] = mine_p;
      part[gw * 2 * CP + CP + lane] = mine_r;
    }
    if (lane == 0) dots[gw] = qk;
    barrier();
    const int j = lane % CP;                                    // this lane's column
    const float* mine = part + (gw & ~3) * 2 * CP + j;
    qk = (dots[0] + dots[1]) + (dots[2] + dots[3]);
    const float pj = (mine[0] + mine[2 * CP]) + (mine[4 * CP] + mine[6 * CP]);
    const float rj = (mine[CP] + mine[3 * CP]) + (mine[5 * CP] + mine[7 * CP]);
    const float u = beta * (V[((c0 + j) / 4 * kChunk + t) * 4 + (j & 3)] - pj), o = p.q_scale * fmaf(qk, u, rj);
    for (int i = 0; i < CP; ++i) S[i] = fmaf(k, __shfl_sync(~0u, u, i), S[i]);
    if ((gw & 3) == 0 && lane < CP) {
      const long long at = ((req.start + static_cast<long long>(t0 + t)) * p.Hv + vh) * p.dv + c0 + j;
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

  if (warp == 0) tmem_alloc(reinterpret_cast<uint32_t*>(bar + kTmemAt), L::kTmem);
  if (tid == 0) {
    mbar_init_n(bar + kKqFull, 1);
    mbar_init_n(bar + kMnFull, 1);
    for (int g = 0; g < L::kTurns; ++g) {
      mbar_init_n(bar + kMetaFull + g, 1);
      mbar_init_n(bar + kD1 + g, 1), mbar_init_n(bar + kD2 + g, 1), mbar_init_n(bar + kD3 + g, 1);
      mbar_init_n(bar + kMeet + g, L::kTurnWarps);
    }
    static_assert(L::kTurns == 2, "two of each");
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    fence_proxy_async();
  }
  int* const count = reinterpret_cast<int*>(sm + L::kCount);
  if (tid < 16) count[tid] = 0;
  const bool stop = __syncthreads_or(aborted);
  const uint32_t tmem = *reinterpret_cast<uint32_t*>(bar + kTmemAt);
  if (warp == 0) tmem_relinquish();
  bool late = false;
  // A wait that gave up is not repeated: the loops run to their end, the results are reported as lost.
  auto wait = [&](int which, int parity) {
    if (!late && !mbar_wait_quiet(bar + which, parity)) late = true;
  };
  // k, q and [M; N] of chunk i of the segment, by a warp: a lane a copy
  auto load_chunk = [&](int i) {
    if (lane == 0) {
      mbar_expect(bar + kKqFull, 4 * L::kImage);
      mbar_expect(bar + kMnFull, 2 * L::kMnLo);
    }
    __syncwarp();
    if (lane < 5) {
      const int place = lane >= 2 ? 1 : (req.c0 + i) & 1 ? 2 : 0;              // lanes 0 to 3: Kh Kl Qh Ql
      const char* src = kq_ws + i * slot_bytes + lane * L::kImage;
      char* dst = sm + L::kKq + (lane & 1) * L::kKqLo + place * L::kImage;
      if (lane == 4) src = v_ws + i * slot_bytes, dst = sm + L::kMn;
      bulk_g2s(dst, src, lane == 4 ? 2 * L::kMnLo : L::kImage, bar + (lane == 4 ? kMnFull : kKqFull));
    }
    __syncwarp();
  };
  auto load_meta = [&](int i) {        // gates and bounds, by a thread
    mbar_expect(bar + kMetaFull + (i & 1), L::kMetaBytes);
    bulk_g2s(sm + L::kMeta + (i & 1) * L::kMetaBytes, v_ws + i * slot_bytes + 2 * L::kMnLo + kChunk * p.dv * 4, L::kMetaBytes,
             bar + kMetaFull + (i & 1));
  };

  if (!stop) {
    if (warp == 0) {
      wait_for_primary();
      if (lane == 0) load_meta(0);
      __syncwarp();
      load_chunk(0);
    }
    constexpr int CP = L::kCols, kPairs = CP / 2;
    const int row = (warp & 3) * 32 + lane, c0 = (warp >> 2) * CP;            // lane of tensor memory, columns of the slice
    const int g = c0 / L::kN, cg = c0 % L::kN;                                // group, columns in it
    const uint32_t ta = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + 2 * g * L::kD + cg;
    char* const s_op = sm + L::kS + g * L::kSTurn + (cg >> 3) * DK * 16;
    char* const w_op = sm + L::kW + g * L::kWTurn + (cg >> 3) * kChunk * 16;
    float* const most = maxima + g * 2 * L::kTurnWarps;                      // [2][2 groups][T, o][warps]
    const int gw = warp - g * L::kTurnWarps;                                  // warp of the group
    const bool has_row = DK == 128 || row < DK;
    const bool copies = g == L::kTurns - 1 && (gw & 1) == 0 && gw < 4;        // of these two warps that with q rows issues the copies
    // The warp that arrives last of n issues what the others have made ready: no warp is kept for it (a seventeenth would
    // leave each thread 96 registers), and no other has to be woken.
    auto last_of = [&](int which, int n) {
      int last = 0;
      __syncwarp();
      if (lane == 0) {
        int old;
        asm volatile("atom.acq_rel.cta.shared::cta.add.u32 %0, [%1], 1;" : "=r"(old) : "r"(smem_addr(count + which)) : "memory");
        last = old == n - 1;
        if (last) count[which] = 0;
      }
      return __shfl_sync(~0u, last, 0) != 0;
    };
    auto issue_d1 = [&](int i) {                   // rows 0 to 127: [K; Q], or [Q; K] in odd chunks
      wait(kKqFull, i & 1);
      tmem_fence_after();
      if (elect_one()) {
        product_wide<DK / 16, L::kN>(tmem + 2 * g * L::kD, umma_desc(smem_addr(sm + L::kKq + ((req.c0 + i) & 1) * L::kImage), 128, DK * 16),
                                     umma_desc(smem_addr(sm + L::kS + g * L::kSTurn), 128, DK * 16), L::kKqLo, 256, 256, false);
        umma_commit(bar + kD1 + g);
      }
      __syncwarp();
    };
    auto issue_d2 = [&](int i) {
      wait(kMnFull, i & 1);
      tmem_fence_after();
      if (elect_one()) {
        product_wide<kChunk / 16, L::kN>(tmem + 2 * g * L::kD + L::kD, umma_desc(smem_addr(sm + L::kMn), 128, 1024),
                                         umma_desc(smem_addr(sm + L::kW + g * L::kWTurn), 128, kChunk * 16), L::kMnLo, 256, 256, false);
        umma_commit(bar + kD2 + g);
      }
      __syncwarp();
    };
    auto issue_d3 = [&](int i) {
      tmem_fence_after();
      if (elect_one()) {
        product_wide<kChunk / 16, L::kN>(tmem + 2 * g * L::kD, umma_desc(smem_addr(sm + L::kKq + ((req.c0 + i) & 1) * 2 * L::kImage), DK * 16, 128),
                                         umma_desc(smem_addr(sm + L::kW + g * L::kWTurn), 128, kChunk * 16), L::kKqLo, 2 * DK * 16, 256, true);
        umma_commit(bar + kD3 + g);
      }
      __syncwarp();
    };
// the group's warps meet; bounded like every other wait (what the warps decide on may be garbage once one has given up)
    int meetings = 0;
    auto group_barrier = [&] {
      __syncwarp();
      if (lane == 0) mbar_arrive(bar + kMeet + g);
      wait(kMeet + g, meetings++ & 1);
    };
    // sixteen columns of a product, its two parts added
    auto product_at = [&](uint32_t at, u64 (&d)[8]) { tmem_sum_pairs(at, at + L::kN, d); };
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
    float smax = 0.f, omax = 0.f, inv_s;
    // The largest entries of T and of the chunk's o (0: none is finite): each warp notes its own when it hands T on, in the half
    // of the table that the chunk's number gives, and all read them once D1 is there.
    auto note_maxima = [&](int half) {
      float big = 0.f;
#pragma unroll
      for (int j = 0; j < kPairs; ++j) big = abs_max(big, S[j]);
      if (has_row && (big == kInf || big == 0.f)) {
        big = 0.f;
#pragma unroll
        for (int j = 0; j < kPairs; ++j) {
          const float2 f = unpack2(S[j]);
          big = finite_some(finite_some(big, f.x), f.y);
        }
      }
      big = warp_max(big);
      const float bigo = warp_max(omax);
      if (lane == 0) most[half * 2 * L::kWarps + gw] = big, most[half * 2 * L::kWarps + L::kTurnWarps + gw] = bigo;
      omax = 0.f;
    };
    auto read_maxima = [&](int half, float& s, float& o) {
      const float* m = most + half * 2 * L::kWarps;
      s = warp_max(lane < L::kTurnWarps ? m[lane] : 0.f);
      o = warp_max(lane < L::kTurnWarps ? m[L::kTurnWarps + lane] : 0.f);
    };
    // A bound lies far above the values that it was for.  Where none of these is finite there is nothing to take again; a chunk
    // that has to be, whatever it came to, has infinite bounds.
    auto too_far = [](float bound, float most) { return bound * kRange > most && (most > 0.f || bound == kInf); };
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
    // T, whose entries are at most `bound`, into its operand for chunk i
    auto put_state = [&](int i, float bound) {
      const float sc = scale_for(bound, inv_s);
      if (has_row) {
#pragma unroll
        for (int j = 0; j < CP; j += 16) put(S + j / 2, sc, s_op + (j >> 3) * DK * 16 + row * 16, DK * 16, L::kSLo);
      }
      note_maxima(i & 1);
      fence_proxy_async();
      tmem_fence_before();
      if (last_of(kSDone + g, L::kTurnWarps)) issue_d1(i);
    };
    // T once more with the scale that its largest entry allows, by all warps of the group (D1 of chunk i is done)
    auto put_again = [&](int i) {
      group_barrier();                             // all have read the maxima
      note_maxima(i & 1);
      group_barrier();
      float unused;
      read_maxima(i & 1, smax, unused);
      put_state(i, smax);
    };
    // Chunk i once more, token by token: T before it lies in D2's place.
    auto take_again = [&](int i) {
      float s[CP];
#pragma unroll
      for (int j = 0; j < CP; j += 16) {
        u64 d[8];
        tmem_pairs(ta + L::kD + j, d);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float2 f = unpack2(d[k]);
          s[j + 2 * k] = f.x, s[j + 2 * k + 1] = f.y;
        }
      }
      again_by_token<DK, NB>(p, req, vh, row, has_row, g, gw, col0 + c0, (req.c0 + i) * kChunk, kq_ws + i * slot_bytes,
                             reinterpret_cast<const float*>(v_ws + i * slot_bytes + 4 * 128 * kChunk), sm, s, meetings, late);
#pragma unroll
      for (int j = 0; j < kPairs; ++j) S[j] = pack2(s[2 * j], s[2 * j + 1]);
    };
    u64 a[kPairs];                                             // v of a k row; the first part of o of a q row
    u64 ahead[kPairs];                                         // v of the next chunk
    auto load_v = [&](int i, u64* a) {
      const float4* V = reinterpret_cast<const float4*>(v_ws + i * slot_bytes + 4 * 128 * kChunk) + (col0 + c0) / 4 * kChunk + (row & 63);
#pragma unroll
      for (int j = 0; j < kPairs; j += 2) {
        const float4 f = __ldcg(V + j / 2 * kChunk);
        a[j] = pack2(f.x, f.y), a[j + 1] = pack2(f.z, f.w);
      }
    };
    // Writes the warp's 32 rows of o from token t0 on.  Sixteen bytes of a row go to place row ^ unit of their unit's 512
    // bytes, so that neither rows nor units share banks; the units are the places of w that this warp itself writes.
    auto store_out = [&](int t0) {
      auto place = [&](int unit, int r) {                      // units: eight columns, high and low terms
        return w_op + (unit & 1) * L::kWLo + (unit >> 1) * kChunk * 16 + (row & 32) * 16 + (r ^ unit) * 16;
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
    wait_for_primary();
    if ((row >> 6) == (req.c0 & 1)) load_v(0, a);
    // the first T's scale: its largest entry
    int d1_done = 0;                               // D1's so far: one a chunk, and those taken again
    note_maxima(1);
    group_barrier();
    {
      float unused;
      read_maxima(1, smax, unused);
    }
    put_state(0, smax);
    // While D1 runs: the window after the prompt, its last K - 1 rows (the launches before have read the old ones).
    if ((req.c0 + req.nc) * kChunk >= req.len) {
      float* wout = p.conv_out + req.b * p.conv_stride;
      const int kq = p.Hk * DK, extra = vh % R == 0 && col0 == 0 ? 2 * DK : 0;
      for (int c = tid; c < NB + extra; c += L::kThreads) {
        const int ch = c < NB ? 2 * kq + vh * p.dv + col0 + c : c - NB < DK ? kh * DK + c - NB : kq + kh * DK + c - NB - DK;
        for (int j = 0; j < p.K - 1; ++j) {
          const long long at = (req.start + static_cast<long long>(req.len - (p.K - 1) + j)) * p.x_row + ch;
          wout[static_cast<long long>(j) * p.C + ch] = p.in_dtype == GDN_DTYPE_BF16 ? load_f(static_cast<const __nv_bfloat16*>(p.x) + at)
                                                                                    : load_f(static_cast<const float*>(p.x) + at);
        }
      }
    }
    float s_bound = smax, u_bound = 0.f, o_bound = 0.f, omax_before;   // of the chunk before
    for (int i = 0; i < req.nc; ++i) {
      const int odd = (req.c0 + i) & 1, ph = i & 1;
      const bool k_row = (row >> 6) == odd;                    // this thread's row is a token's k (else its q)
      const int t = row & 63;
      const float* meta = reinterpret_cast<const float*>(sm + L::kMeta + ph * L::kMetaBytes);
      wait(kMetaFull + ph, (i >> 1) & 1);
      const float first = meta[t], left = meta[kChunk + t];
      const float4 m0 = *reinterpret_cast<const float4*>(meta + 2 * kChunk);
      const float4 m1 = *reinterpret_cast<const float4*>(meta + 2 * kChunk + 4);
      const float whole = m0.x, inv_m = m0.y, inv_n = m0.z, vmax = m0.w, mbound = m1.x, fmax_ = m1.y, nbound = m1.z;
      if (!k_row && i + 1 < req.nc) load_v(i + 1, ahead);      // a q row is the next chunk's k row
      wait(kD1 + g, d1_done++ & 1);
      tmem_fence_after();
      read_maxima(ph, smax, omax_before);
      // Bounds far above the values have cost these their bits.  T itself is exact: its operand is made again.  u and o are
      // not: the chunk before is taken again, token by token.
      if (i > 0 && (too_far(s_bound, smax) || too_far(o_bound, omax_before))) {
        if (too_far(u_bound, smax) || too_far(o_bound, omax_before)) take_again(i - 1);
        put_again(i);
        wait(kD1 + g, d1_done++ & 1);
        tmem_fence_after();
      }
      const float w_bound = (vmax + fmax_ * (DK == 128 ? 11.32f : DK == 64 ? 8.001f : 5.657f) * smax) * 1.001f;
      float inv_w, inv_u;
      const float sc_w = scale_for(w_bound, inv_w);
      const float f1 = first * (inv_s * (1.f / kUnit));
      char* const w_at = w_op + t * 16;
      if (k_row) {
        const u64 f = pack2(-f1, -f1);
#pragma unroll
        for (int j = 0; j < CP; j += 16) {
          u64 d[8];
          product_at(ta + j, d);
#pragma unroll
          for (int k = 0; k < 8; ++k) d[k] = fma2(f, d[k], a[j / 2 + k]);
          put(d, sc_w, w_at + (j >> 3) * kChunk * 16, kChunk * 16, L::kWLo);
        }
        fence_proxy_async();
        tmem_fence_before();
      } else {
        const u64 f = pack2(f1 * p.q_scale, f1 * p.q_scale);
#pragma unroll
        for (int j = 0; j < CP; j += 16) {
          u64 d[8];
          product_at(ta + j, d);
#pragma unroll
          for (int k = 0; k < 8; ++k) a[j / 2 + k] = mul2(d[k], f);
        }
        tmem_fence_before();                                   // D3 takes D1's place
      }
      if (last_of(kWDone + g, L::kTurnWarps)) issue_d2(i);
      u_bound = mbound * w_bound * 1.001f;
      o_bound = nbound * w_bound * fabsf(p.q_scale);
      s_bound = (whole * smax + 64.f * u_bound) * 1.001f;
      if (m1.w != 0.f) u_bound = s_bound = kInf;               // to be taken again, whatever the chunk came to
      const float sc_u = scale_for(u_bound, inv_u);
      // (the other group has read the gates of the chunk before: it took part in D2 there, without which nobody is here)
      if (!k_row && copies && i + 1 < req.nc && elect_one()) load_meta(i + 1);
      __syncwarp();
      wait(kD2 + g, ph);
      tmem_fence_after();
      if (!k_row && copies && i + 1 < req.nc) {
        // A warp of q rows fetches the next chunk: with D2 of both groups done nothing reads Q or [M; N] any more, and D3 of
        // the chunk before, the last to read the other K, was done before T went to D1.
        wait(kD2, ph);
        load_chunk(i + 1);
      }
      if (k_row) {
        const float f = left * inv_m * inv_w * sc_u;
#pragma unroll
        for (int j = 0; j < CP; j += 16) {
          u64 d[8];
          product_at(ta + L::kD + j, d);
          put(d, f, w_at + (j >> 3) * kChunk * 16, kChunk * 16, L::kWLo);
        }
        fence_proxy_async();
        tmem_fence_before();
        if (last_of(kUDone + g, L::kTurnWarps / 2)) issue_d3(i);
      } else {
        const u64 f = pack2(inv_n * inv_w * p.q_scale, inv_n * inv_w * p.q_scale);
#pragma unroll
        for (int j = 0; j < CP; j += 16) {
          u64 d[8];
          product_at(ta + L::kD + j, d);
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            a[j / 2 + k] = fma2(f, d[k], a[j / 2 + k]);
            omax = abs_max(omax, a[j / 2 + k]);
          }
        }
        if (omax == 0.f)
#pragma unroll
          for (int j = 0; j < kPairs; ++j) {
            const float2 f = unpack2(a[j]);
            omax = finite_some(finite_some(omax, f.x), f.y);
          }
      }
      // T before the chunk is kept in D2's place, of which this thread has read its part
#pragma unroll
      for (int j = 0; j < CP; j += 16) tmem_put_pairs(ta + L::kD + j, S + j / 2);
      wait(kD3 + g, ph);
      tmem_fence_after();
      const u64 f3 = pack2(inv_u * (1.f / kUnit), inv_u * (1.f / kUnit)), whole2 = pack2(whole, whole);
#pragma unroll
      for (int j = 0; j < CP; j += 16) {
        u64 d[8];
        product_at(ta + j, d);
#pragma unroll
        for (int k = 0; k < 8; ++k) S[j / 2 + k] = has_row ? fma2(whole2, S[j / 2 + k], mul2(f3, d[k])) : 0ull;
      }
      tmem_wait_st();
      if (i + 1 < req.nc) put_state(i + 1, s_bound);
      if (!k_row) {
        // o, in rows again: through the warp's own part of w's operand, which D3 was the last to read
        store_out((req.c0 + i) * kChunk + (row & 32));
#pragma unroll
        for (int j = 0; j < kPairs; ++j) a[j] = ahead[j];
      }
    }
    note_maxima(req.nc & 1);
    group_barrier();
    read_maxima(req.nc & 1, smax, omax_before);
    if (too_far(u_bound, smax) || too_far(o_bound, omax_before)) take_again(req.nc - 1);
    if (has_row) {
      float* dst = p.state_out + req.b * p.state_stride + (static_cast<long long>(vh) * DK + row) * p.dv + col0 + c0;
#pragma unroll
      for (int j = 0; j < kPairs; j += 2) {
        const float2 x = unpack2(S[j]), y = unpack2(S[j + 1]);
        *reinterpret_cast<float4*>(dst + 2 * j) = make_float4(x.x, x.y, y.x, y.y);
      }
    }
  }
  if (__syncthreads_or(late) && tid == 0) {
    // whatever was in flight has had twice the time that a wait gives it
    mbar_wait(bar + kKqFull, 0), mbar_wait(bar + kKqFull, 1), mbar_wait(bar + kMnFull, 0), mbar_wait(bar + kMnFull, 1);
    device_error(p.err, GDN_DEVERR_TIMEOUT, req.b);
  }
  __syncthreads();
  if (warp == 0) tmem_dealloc(tmem, L::kTmem);
}

template <typename F>
cudaError_t with_smem(F kernel, int bytes) {
  return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
}
// A launch that may start before the one before it has ended.
template <typename F, typename... A>
cudaError_t launch_after(F kernel, dim3 grid, int threads, int smem, cudaStream_t s, const A&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}
template <typename InT, int DK, int KT>
cudaError_t launch_prepare(const SeqParams& p, const Segment& seg, char* ws, cudaStream_t s) {
  auto keys = seq_keys_kernel<InT, DK, KT>;
  auto values = seq_values_kernel<InT, KT>;
  cudaError_t e = with_smem(keys, PrepK<DK>::kTotal);
  if (e == cudaSuccess) e = with_smem(values, PrepV::kTotal);
  if (e != cudaSuccess) return e;
  keys<<<dim3(p.Hk, seg.slots), kPrepThreads, PrepK<DK>::kTotal, s>>>(p, seg, ws);
  e = cudaGetLastError();
  return e != cudaSuccess ? e : launch_after(values, dim3(p.Hv, seg.slots), kPrepThreads, PrepV::kTotal, s, p, seg, ws);
}
template <int DK, int NB>
cudaError_t launch_chain(const SeqParams& p, const Segment& seg, const char* ws, bool right_after, cudaStream_t s) {
  auto k = seq_chain_kernel<DK, NB>;
  cudaError_t e = with_smem(k, Chain<DK, NB>::kTotal);
  if (e != cudaSuccess) return e;
  const dim3 grid(p.Hv * (p.dv / NB), seg.n);
  if (right_after) return launch_after(k, grid, Chain<DK, NB>::kThreads, Chain<DK, NB>::kTotal, s, p, seg, ws);
  k<<<grid, Chain<DK, NB>::kThreads, Chain<DK, NB>::kTotal, s>>>(p, seg, ws);
  return cudaGetLastError();
}
template <int DK>
cudaError_t launch_prepare_d(const SeqParams& p, const Segment& seg, char* ws, cudaStream_t s) {
  using bf16 = __nv_bfloat16;
  if (p.in_dtype == GDN_DTYPE_BF16)
    return p.K > 4 ? launch_prepare<bf16, DK, 8>(p, seg, ws, s) : launch_prepare<bf16, DK, 4>(p, seg, ws, s);
  return p.K > 4 ? launch_prepare<float, DK, 8>(p, seg, ws, s) : launch_prepare<float, DK, 4>(p, seg, ws, s);
}
template <int DK>
cudaError_t launch_chain_d(const SeqParams& p, const Segment& seg, const char* ws, bool right_after, cudaStream_t s) {
  // 64 columns a CTA, or 32 where the other half of the GPU would be idle.
  if (p.dv >= 64 && seg.n * p.Hv * (p.dv / 64) > 76) return launch_chain<DK, 64>(p, seg, ws, right_after, s);
  return launch_chain<DK, 32>(p, seg, ws, right_after, s);
}

}  // namespace

cudaError_t launch_seq_prepare(const SeqParams& p, const Segment& seg, void* workspace, cudaStream_t s) {
  char* ws = static_cast<char*>(workspace);
  if (p.dk == 128) return launch_prepare_d<128>(p, seg, ws, s);
  if (p.dk == 64) return launch_prepare_d<64>(p, seg, ws, s);
  return launch_prepare_d<32>(p, seg, ws, s);
}
cudaError_t launch_seq_chain(const SeqParams& p, const Segment& seg, const void* workspace, bool right_after, cudaStream_t s) {
  const char* ws = static_cast<const char*>(workspace);
  if (p.dk == 128) return launch_chain_d<128>(p, seg, ws, right_after, s);
  if (p.dk == 64) return launch_chain_d<64>(p, seg, ws, right_after, s);
  return launch_chain_d<32>(p, seg, ws, right_after, s);
}

}  // namespace gdn
