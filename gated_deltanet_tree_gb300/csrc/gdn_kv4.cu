// Append to and read from the paged 4-bit key/value cache (format: gdn_tree.h).
//
// Append.  One CTA per (request and layer, page it touches, kv head): it owns
// every word of that page's block, so the value words -- eight tokens of one
// channel each -- are merged with tokens written earlier without atomics.  Four
// lanes share a group of 32 channels: eight channels each, the group's largest
// magnitude by two shuffles, one code word per lane.  Keys go straight to their
// words; value codes pass through shared memory ([token][channel] bytes) and are
// regrouped into words of eight tokens.  The work is the rows read once and
// 1.125 D bytes a row and head written.
//
// The lengths are read by every CTA and advanced by the request's last one to
// finish (a ticket per request), so a call is one launch.
//
// Measured: two prompts of 20001 and 15001 bf16 rows, 4 kv heads of 256, appended in
// 57 us (3.2 TB/s; issue slots, 73% taken, bound it: about 19 instructions an element,
// most of them rounding) and read back to fp32 in 62 us (6.0 TB/s, 0.88 of a plain
// copy's rate).  fp32 rows, with a division an element: 94 us.
#include "gdn_kv4.cuh"

namespace gdn {
namespace {

constexpr int kAppendThreads = 128;

// Eight consecutive elements, as they lie and as fp32.
template <typename T>
struct Raw8;
template <>
struct Raw8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = __ldg(reinterpret_cast<const float4*>(p));
    b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  }
};
template <>
struct Raw8<__nv_bfloat16> {
  uint4 u;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { u = __ldg(reinterpret_cast<const uint4*>(p)); }
};
__device__ __forceinline__ void unpack(const Raw8<float>& r, float (&x)[8]) {
  x[0] = r.a.x; x[1] = r.a.y; x[2] = r.a.z; x[3] = r.a.w;
  x[4] = r.b.x; x[5] = r.b.y; x[6] = r.b.z; x[7] = r.b.w;
}
__device__ __forceinline__ void unpack(const Raw8<__nv_bfloat16>& r, float (&x)[8]) {
  const uint32_t w[4] = {r.u.x, r.u.y, r.u.z, r.u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

// The element of largest magnitude of a group held by four adjacent lanes (eight channels each), the lowest channel's on
// ties.  All 32 lanes of the warp call it.
__device__ __forceinline__ float largest_of(const float (&x)[8]) {
  float big = 0.f, m = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float a = fabsf(x[i]);
    if (a > big) { big = a; m = x[i]; }        // the first of equals stays
  }
#pragma unroll
  for (int o = 1; o < 4; o <<= 1) {
    const float ob = __shfl_xor_sync(0xffffffffu, big, o), om = __shfl_xor_sync(0xffffffffu, m, o);
    const bool other_first = (threadIdx.x & o) != 0;   // the partner holds the lower channels
    if (ob > big || (ob == big && other_first)) { big = ob; m = om; }
  }
  return m;
}
// The group's scale from that element; 0 where it is left out (d: what elements are divided by).
__device__ __forceinline__ __half scale_of(float m, float* d) {
  const float x = fminf(fmaxf(__bfloat162float(__float2bfloat16_rn(m * -0.125f)), -kScaleMax), kScaleMax);
  const __half h = __float2half_rn(x);
  *d = __half2float(h);
  return h;
}

// Quantises a group: codes 0..15 of this lane's channels 2i and 2i + 1 in the halves of code[i], and the group's scale.
// code = rint(x / d) + 8, clamped.
__device__ __forceinline__ __half quantise8(const Raw8<float>& r, uint32_t (&code)[4]) {
  float x[8], d;
  unpack(r, x);
  bool bad = false;
#pragma unroll
  for (int i = 0; i < 8; ++i) bad |= !(fabsf(x[i]) <= 3.402823466e38f);
  const float m = largest_of(x);
  const unsigned quad = 0xFu << (threadIdx.x & 28);
  bad = (__ballot_sync(0xffffffffu, bad) & quad) != 0;
  const __half h = scale_of(m, &d);
  const bool none = bad || d == 0.f;
  uint32_t c[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float q = none ? 0.f : __fdiv_rn(x[i], d);
    // adding 1.5 2^23 rounds to an integer, ties to even, in the low bits; 8 more makes it the code
    c[i] = __float_as_uint(fminf(fmaxf(q, -8.f), 7.f) + 12582920.f) & 15u;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) code[i] = c[2 * i] | c[2 * i + 1] << 16;
  return bad ? __ushort_as_half(0x7FFF) : h;
}

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.u16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t min_u16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("min.u16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t max_s16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.s16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
// The same of bf16 elements, on as few integer instructions as the format allows: they are what bounds the kernel.
//
// The largest magnitude: a bf16 number's bits are its magnitude's order, so two packed maxima of the words as they lie,
// one signed (the largest positive element) and one unsigned (the most negative one, if any), find it and its sign;
// only where both magnitudes are equal does the order of the channels decide.  Infinities and NaN are the largest.
//
// x and d have eight significant bits, so x / d is a tie or at least 2^-11 away from one: a product with 1 / d,
// corrected once by its remainder (exact, and ties come out exact), rounds like the quotient, and so does that number
// over 16 plus 1/2, saturated to [0, 1]: 24 bits hold a tie exactly, and move the others by 2^-21 of a code at most.
__device__ __forceinline__ __half quantise8(const Raw8<__nv_bfloat16>& r, uint32_t (&code)[4]) {
  float x[8], d;
  unpack(r, x);
  uint32_t pos = max_s16x2(max_s16x2(r.u.x, r.u.y), max_s16x2(r.u.z, r.u.w));
  uint32_t neg = max_u16x2(max_u16x2(r.u.x, r.u.y), max_u16x2(r.u.z, r.u.w));
#pragma unroll
  for (int o = 1; o < 4; o <<= 1) {
    pos = max_s16x2(pos, __shfl_xor_sync(0xffffffffu, pos, o));
    neg = max_u16x2(neg, __shfl_xor_sync(0xffffffffu, neg, o));
  }
  pos = max_s16x2(pos, pos >> 16);
  neg = max_u16x2(neg, neg >> 16);
  const int p = static_cast<int16_t>(pos & 0xFFFFu), n = static_cast<int>(neg & 0xFFFFu) - 0x8000;   // < 0: none
  const int big = max(p, n);
  float m = __uint_as_float(static_cast<uint32_t>(big) << 16 | (n > max(p, 0) ? 0x80000000u : 0u));
  if (__any_sync(0xffffffffu, p == n)) m = largest_of(x);
  const bool bad = big >= 0x7F80;
  const __half h = scale_of(m, &d);
  float inv;                                   // within an ulp or two: the remainder makes up for it
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(d));
  if (bad || d == 0.f) inv = 0.f;
  uint32_t c[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float q = x[i] * inv;
    q = fmaf(fmaf(-q, d, x[i]), inv, q);
    // 1.5 2^23 more rounds to an integer, ties to even, in the low bits
    c[i] = __float_as_uint(fmaf(__saturatef(fmaf(q, 0.0625f, 0.5f)), 16.f, 12582912.f));
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) code[i] = min_u16x2(__byte_perm(c[2 * i], c[2 * i + 1], 0x5410), 0x000F000Fu);
  return bad ? __ushort_as_half(0x7FFF) : h;
}

template <typename T, int D>
__global__ void __launch_bounds__(kAppendThreads) kv4_append_kernel(KvAppendParams p) {
  using Blk = KvBlock<D>;
  constexpr int kLanesPerRow = D / 8;                       // lanes that hold one row
  constexpr int kRowsPerPass = kAppendThreads / kLanesPerRow;
  __shared__ __align__(16) uint8_t codes[kPage][D];         // value codes of the rows written here
  const int bl = blockIdx.x, b = bl / p.c.layers, l = bl % p.c.layers;
  const int h = blockIdx.z, tid = threadIdx.x;

  const int len = p.c.seq_len[b], cnt = p.count[b];
  const long long cap = static_cast<long long>(p.c.pages_max) * kPage;
  bool ok = len >= 0 && cnt >= 0 && cnt <= p.n_rows && len + static_cast<long long>(cnt) <= cap;
  const int32_t* table = p.c.page_table + static_cast<size_t>(b) * p.c.pages_max;
  const int32_t* path = p.path ? p.path + static_cast<size_t>(b) * p.n_rows : nullptr;
  const int page0 = len / kPage;
  if (ok && cnt > 0) {
    const int pages = (len + cnt - 1) / kPage - page0 + 1;
    bool mine = true;
    for (int i = tid; i < pages; i += kAppendThreads) {
      const int g = table[page0 + i];
      mine = mine && g >= 0 && g < p.c.n_pages;
    }
    if (path)
      for (int i = tid; i < cnt; i += kAppendThreads) mine = mine && path[i] >= 0 && path[i] < p.n_rows;
    ok = __syncthreads_and(mine);
  }
  if (!ok && tid == 0) device_error(p.c.err, GDN_DEVERR_CACHE, b);

#pragma unroll 1
  for (int y = blockIdx.y; ok && y * kPage < len % kPage + cnt; y += gridDim.y) {
    // rows [lo, hi) of the page are written; row r holds appended row first + r
    const int first = (page0 + y) * kPage - len;
    const int lo = max(0, -first), hi = min(kPage, cnt - first);
    if (lo >= hi) break;
    if (y >= static_cast<int>(gridDim.y)) __syncthreads();     // the page before has left `codes`
    char* blk = kv_block<D>(p.c, p.Hkv, table[page0 + y], l, h);
    const size_t row0 = static_cast<size_t>(bl) * p.n_rows;
    const T* kn = static_cast<const T*>(p.k_new) + h * D;
    const T* vn = static_cast<const T*>(p.v_new) + h * D;
    const int w = tid % kLanesPerRow;                       // word of the row this lane holds
    constexpr int kAhead = sizeof(T) == 2 ? 4 : 2;          // rows in flight
#pragma unroll 1
    for (int r0 = lo + tid / kLanesPerRow; r0 - tid / kLanesPerRow < hi; r0 += kAhead * kRowsPerPass) {
      Raw8<T> rk[kAhead], rv[kAhead];
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const int r = min(r0 + k * kRowsPerPass, hi - 1);   // (rows past the last repeat it and are not stored)
        const size_t at = (row0 + (path ? path[first + r] : first + r)) * p.kv_row + 8 * w;
        rk[k].load(kn + at);
        rv[k].load(vn + at);
      }
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const int r = r0 + k * kRowsPerPass;
        uint32_t c[4];
        const __half dk = quantise8(rk[k], c);
        const uint32_t word = c[0] | c[1] << 4 | c[2] << 8 | c[3] << 12;      // nibble_of's order
        const __half dv = quantise8(rv[k], c);
        if (r < hi) {
          reinterpret_cast<uint32_t*>(blk)[Blk::key_word(r, w)] = word;
          *reinterpret_cast<uint2*>(&codes[r][8 * w]) =
              make_uint2(__byte_perm(c[0], c[1], 0x6420), __byte_perm(c[2], c[3], 0x6420));
          if ((w & 3) == 0) {
            reinterpret_cast<__half*>(blk + Blk::kKeyScales)[r * Blk::kGroups + (w >> 2)] = dk;
            reinterpret_cast<__half*>(blk + Blk::kValScales)[(w >> 2) * kPage + r] = dv;
          }
        }
      }
    }
    __syncthreads();
    // value words: (four channels, eight tokens) per thread and step
    const int o_lo = lo >> 3, o_hi = (hi + 7) >> 3;
    uint4* out = reinterpret_cast<uint4*>(blk + Blk::kValCodes);
    for (int i = tid; i < (o_hi - o_lo) * (D / 4); i += kAppendThreads) {
      const int cq = i % (D / 4), o = o_lo + i / (D / 4);
      uint32_t q[8], keep = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int r = 8 * o + e;
        const bool in = r >= lo && r < hi;
        q[e] = in ? *reinterpret_cast<const uint32_t*>(&codes[r][4 * cq]) : 0u;
        if (!in) keep |= 0xFu << (4 * nibble_of(e));
      }
      // two tokens a byte, then a transpose of four by four bytes: nibble_of's order
      const uint32_t a0 = q[0] | q[2] << 4, a1 = q[4] | q[6] << 4, a2 = q[1] | q[3] << 4, a3 = q[5] | q[7] << 4;
      const uint32_t b0 = __byte_perm(a0, a1, 0x5140), b1 = __byte_perm(a0, a1, 0x7362);
      const uint32_t b2 = __byte_perm(a2, a3, 0x5140), b3 = __byte_perm(a2, a3, 0x7362);
      uint32_t v[4] = {__byte_perm(b0, b2, 0x5410), __byte_perm(b0, b2, 0x7632), __byte_perm(b1, b3, 0x5410),
                       __byte_perm(b1, b3, 0x7632)};
      uint4* dst = out + Blk::val_word(4 * cq, o) / 4;
      if (keep) {
        const uint4 old = *dst;
        v[0] |= old.x & keep;
        v[1] |= old.y & keep;
        v[2] |= old.z & keep;
        v[3] |= old.w & keep;
      }
      *dst = make_uint4(v[0], v[1], v[2], v[3]);
    }
  }
  // the request's last CTA advances its length: every other one has read it before taking its ticket
  __syncthreads();
  if (tid == 0) {
    __threadfence();
    const int all = static_cast<int>(gridDim.y * gridDim.z) * p.c.layers;
    if (atomicAdd(&p.c.ticket[b], 1) == all - 1) {
      p.c.ticket[b] = 0;
      if (ok) p.c.seq_len[b] = len + cnt;
    }
  }
}

__device__ __forceinline__ void store4(float* p, const float (&x)[4]) {
  __stcs(reinterpret_cast<float4*>(p), make_float4(x[0], x[1], x[2], x[3]));
}
__device__ __forceinline__ void store4(__nv_bfloat16* p, const float (&x)[4]) {
  reinterpret_cast<__nv_bfloat162*>(p)[0] = __floats2bfloat162_rn(x[0], x[1]);
  reinterpret_cast<__nv_bfloat162*>(p)[1] = __floats2bfloat162_rn(x[2], x[3]);
}

// One CTA per (request and layer, page of the range, kv head).
template <typename T, int D>
__global__ void __launch_bounds__(kAppendThreads) kv4_read_kernel(KvReadParams p) {
  using Blk = KvBlock<D>;
  const int bl = blockIdx.x, b = bl / p.c.layers, l = bl % p.c.layers;
  const int h = blockIdx.z, tid = threadIdx.x;
  const int len = p.c.seq_len[b], t0 = p.start ? p.start[b] : 0;
  const bool ok = t0 >= 0 && len >= 0 && len <= static_cast<long long>(p.c.pages_max) * kPage;
  if (!ok && tid == 0) device_error(p.c.err, GDN_DEVERR_CACHE, b);
  // tokens of this page, as offsets from t0: [lo, hi); those past the length are zeros
  const long long base = (ok ? t0 / kPage + static_cast<long long>(blockIdx.y) : blockIdx.y) * kPage;
  const long long first = base - (ok ? t0 : 0);
  const int lo = static_cast<int>(max(0ll, first)) , hi = static_cast<int>(min(static_cast<long long>(p.n_rows), first + kPage));
  if (lo >= hi) return;
  const int rl = static_cast<int>(lo - first), rh = static_cast<int>(hi - first);   // rows of the page
  int live = ok && len > base ? static_cast<int>(min(static_cast<long long>(kPage), len - base)) : 0;
  const char* blk = nullptr;
  if (live > 0) {
    const int g = p.c.page_table[static_cast<size_t>(b) * p.c.pages_max + base / kPage];
    if (g >= 0 && g < p.c.n_pages) {
      blk = kv_block<D>(p.c, p.Hkv, g, l, h);
    } else {
      if (tid == 0) device_error(p.c.err, GDN_DEVERR_CACHE, b);
      live = 0;
    }
  }
  const size_t row = static_cast<size_t>(p.Hkv) * D;
  const size_t out0 = (static_cast<size_t>(bl) * p.n_rows) * row + static_cast<size_t>(h) * D;
  T* ko = static_cast<T*>(p.k_out) + out0;
  T* vo = static_cast<T*>(p.v_out) + out0;
  // four channels a lane: half a word of codes, 16 (or 8) adjacent bytes out
#pragma unroll 4
  for (int i = tid; i < (rh - rl) * (D / 4); i += kAppendThreads) {
    const int r = rl + i / (D / 4), q = i % (D / 4);
    float x[4] = {0.f, 0.f, 0.f, 0.f};
    if (r < live) {
      const uint32_t word = reinterpret_cast<const uint32_t*>(blk)[Blk::key_word(r, q >> 1)] >> (8 * (q & 1));
      const float d = __half2float(reinterpret_cast<const __half*>(blk + Blk::kKeyScales)[r * Blk::kGroups + (q >> 3)]);
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] = static_cast<float>(static_cast<int>((word >> (4 * nibble_of(e))) & 15u) - 8) * d;
    }
    store4(ko + (first + r) * static_cast<long long>(row) + 4 * q, x);
  }
  // values: four channels, eight tokens a lane
#pragma unroll 1
  for (int i = tid; i < 2 * D; i += kAppendThreads) {
    const int cq = i % (D / 4), o = i / (D / 4);
    if (8 * o + 8 <= rl || 8 * o >= rh) continue;
    uint4 word = make_uint4(0, 0, 0, 0), scale = make_uint4(0, 0, 0, 0);
    if (8 * o < live) {
      word = *(reinterpret_cast<const uint4*>(blk + Blk::kValCodes) + Blk::val_word(4 * cq, o) / 4);
      scale = *reinterpret_cast<const uint4*>(blk + Blk::kValScales + 2 * ((cq >> 3) * kPage + 8 * o));
    }
    const uint32_t w[4] = {word.x, word.y, word.z, word.w}, sc[4] = {scale.x, scale.y, scale.z, scale.w};
    T* dst = vo + (first + 8 * o) * static_cast<long long>(row) + 4 * cq;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int r = 8 * o + e;
      const float d = __half2float(__ushort_as_half(static_cast<unsigned short>(sc[e >> 1] >> (16 * (e & 1)))));
      float x[4];
#pragma unroll
      for (int c = 0; c < 4; ++c)
        x[c] = r < live ? static_cast<float>(static_cast<int>((w[c] >> (4 * nibble_of(e))) & 15u) - 8) * d : 0.f;
      if (r >= rl && r < rh) store4(dst + e * static_cast<long long>(row), x);
    }
  }
}

template <typename T, int D>
cudaError_t append_t(const KvAppendParams& p, cudaStream_t s) {
  // pages that n_rows rows can touch, at any offset; up to a page of rows, which mostly touch one, a CTA takes both: the
  // second one's CTAs would find no work (32 requests, 16 layers, up to 11 rows, with the lengths' reset and the rows read
  // back in one graph: 31.9 us with them, 30.5 without)
  const dim3 grid(p.c.B * p.c.layers, p.n_rows <= kPage ? 1 : (p.n_rows + kPage - 2) / kPage + 1, p.Hkv);
  kv4_append_kernel<T, D><<<grid, kAppendThreads, 0, s>>>(p);
  return cudaGetLastError();
}
template <typename T, int D>
cudaError_t read_t(const KvReadParams& p, cudaStream_t s) {
  const dim3 grid(p.c.B * p.c.layers, (p.n_rows + kPage - 2) / kPage + 1, p.Hkv);
  kv4_read_kernel<T, D><<<grid, kAppendThreads, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace

#define GDN_KV4_BY_SIZE(fn, T, p, s) \
  ((p).D == 256 ? fn<T, 256>(p, s) : (p).D == 128 ? fn<T, 128>(p, s) : fn<T, 64>(p, s))

cudaError_t launch_kv4_append(const KvAppendParams& p, cudaStream_t s) {
  return p.dtype == GDN_DTYPE_BF16 ? GDN_KV4_BY_SIZE(append_t, __nv_bfloat16, p, s) : GDN_KV4_BY_SIZE(append_t, float, p, s);
}
cudaError_t launch_kv4_read(const KvReadParams& p, cudaStream_t s) {
  return p.out_dtype == GDN_DTYPE_BF16 ? GDN_KV4_BY_SIZE(read_t, __nv_bfloat16, p, s) : GDN_KV4_BY_SIZE(read_t, float, p, s);
}

}  // namespace gdn
