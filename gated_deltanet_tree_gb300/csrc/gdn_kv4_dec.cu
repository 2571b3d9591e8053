// Attention over the paged 4-bit cache for few rows: tiles of eight (node, query
// head) pairs that share a kv head -- plain decoding, and small trees of models
// with few query heads per kv head; and every fp32 call.
//
// With so few rows the cache's bytes are the bound, so the kernel is built around
// moving and unpacking them.  A pair of warps takes a page: one bulk copy brings
// its block (72 D bytes) into a ring of stages, each warp takes 32 of its tokens.
// The products run on mma.m16n8k16 with the cache on the 16-wide side, which
// wastes nothing on absent rows: S^T = K Q^T (tokens x 8 rows) and O^T = V^T P^T
// (channels x 8 rows).  A code pair becomes two fp16 values by one mask-or -- the
// four code bits as the top mantissa bits of 1 + n/16 -- and one fused
// multiply-add with 16 d and -24 d, which gives (n - 8) d exactly.  The page
// format puts a lane's codes of 32 channels (keys) or 4 channels x 8 tokens
// (values) into one 16-byte word, in the order the fragments want; the order of
// the tokens inside 32 is the values' and the keys follow it.
//
// Every warp keeps its own maximum, sum and output (fp32) and the CTA's warps
// meet once, at the end, where the nodes' own rows are added in fp32 from
// each row's ancestor list.  Weights are carried as 2^(x - m + 6), m the largest
// score when the output was last rescaled, which happens only where a score passes
// it by more than 8: weights down to 2^-30 of the largest stay above fp16's
// smallest value and none passes its largest.
//
// fp32 calls run the same products on values split in two fp16 terms each: q = hi +
// lo keeps 22 bits of a row's largest, hi + 2^-12 lo 22 bits of a weight, or 2^-43 of the
// largest one, the unpacked codes are exact as they are, and a product costs two MMAs
// instead of one.  An MMA's additions truncate, so
// its sums are kept short -- 16 channels of a score, 32 tokens of an output -- and
// added in fp32 outside: 24 query heads of 256 over 50000 tokens have a relative
// error of 9e-7 that way (3.7e-6 with the sums left in the MMAs), for a tenth of the
// time (86 -> 95 us).
//
// Measured: 32 requests of 16640 to 32768 tokens, 24 query and 4 kv heads of 256, one bf16
// token each: 912 MB in 192 us, 4.8 TB/s, 0.70 of a plain copy's rate.  No unit is full
// (issue slots 55%, ALU 46%): the latencies of a warp's chain of scores, shuffles and
// output, with two pages in flight a pair of warps, set the pace, and the schedule gives
// every CTA the same number of pages.  One request of 4096 tokens: 17 us, latencies.
// The same 32 requests in fp32: 397 us (one CTA of D = 256 fits an SM).
#include "gdn_kv4_attn.cuh"
#include "gdn_umma.cuh"

namespace gdn {
namespace {

constexpr int kStages = 2;
// Warps of a CTA; two CTAs share an SM, so that one computes while the other starts or ends.  The register file
// holds 12 warps with the 160 registers D = 256 takes, or 16 with 128.
template <int D>
constexpr int kWarpsOf = D == 256 ? 6 : 8;
constexpr int kRows = kKvDecRows;
constexpr float kLift = 6.f;          // weights are scaled by 2^kLift ...
constexpr float kSlack = 8.f;         // ... against a maximum that may lag by up to 2^kSlack: 2^14 at most in fp16
// (fp32) the low terms of the weights, at most 2^2, are scaled by this: unscaled, fp16's smallest value would cut them
// off at 2^-31 of the reference, which 200,000 tokens behind one that dominates make 9e-5 of the output.
constexpr float kLowScale = 4096.f;
// Pages that are added to one output and one sum: a segment is taken in runs, joined in the place of its partial result.
// fp32 sums lose up to 2^-24 an addition, one a page in each pair of warps, behind a token that dominates: 2e-5 of the
// output at 1024 pages (1.5e-4 over a million tokens at once).  The MMAs of bf16 calls truncate, 2^-23 an addition and two
// a page: 2^-13 at 2048.
template <typename T>
constexpr int kRun = sizeof(T) == 4 ? 1024 : 2048;
constexpr float kLog2e = 1.4426950408889634f;

template <int D, typename T>
struct Smem {   // bf16: twice this fits the 228 KB of an SM
  static constexpr int kTerms = sizeof(T) == 4 ? 2 : 1;            // fp16 terms of a query or a weight
  static constexpr int kWarps = kWarpsOf<D>, kPairs = kWarps / 2;
  static constexpr int kStage = KvBlock<D>::kBytes;
  static constexpr int kQ = kPairs * kStages * kStage;             // fp16 [8][D + 8]
  static constexpr int kQRow = D + 8;
  static constexpr int kStat = kQ + kTerms * kRows * kQRow * 2;    // float [kWarps][8][2], scale [8]
  static constexpr int kSee = kStat + (kWarps * kRows * 2 + kRows) * 4;
  static constexpr int kBar = kSee + kRows * 8;                    // each row's ancestors; full, empty [kPairs][kStages]
  static constexpr int kTotal = kBar + 2 * kPairs * kStages * 8 + 16;
};

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}
__device__ __forceinline__ float exp2_fast(float x) {   // results below 2^-126 are zero
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float exp2i(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }   // |e| < 127
__device__ __forceinline__ float2 load2(const __nv_bfloat16* p) {
  return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(p));
}
__device__ __forceinline__ float2 load2(const float* p) { return *reinterpret_cast<const float2*>(p); }
__device__ __forceinline__ void store2(__nv_bfloat16* p, float x, float y) {
  *reinterpret_cast<__nv_bfloat162*>(p) = __floats2bfloat162_rn(x, y);
}
__device__ __forceinline__ void store2(float* p, float x, float y) { *reinterpret_cast<float2*>(p) = make_float2(x, y); }
__device__ __forceinline__ uint32_t h2u(__half2 h) { return *reinterpret_cast<uint32_t*>(&h); }
__device__ __forceinline__ __half2 u2h(uint32_t u) { return *reinterpret_cast<__half2*>(&u); }

template <int D, typename T>
__global__ void __launch_bounds__(32 * kWarpsOf<D>, 2) kv4_attn_dec_kernel(KvAttnParams p) {
  using Blk = KvBlock<D>;
  using Sm = Smem<D, T>;
  constexpr int kTerms = Sm::kTerms;
  constexpr int kWarps = Sm::kWarps, kPairs = Sm::kPairs;
  extern __shared__ __align__(128) char smem_dec[];
  __shared__ int last;
  __shared__ KvJoin joins[2];      // shared items that this CTA finished last
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, pair = warp >> 1, kb = warp & 1;
  const int m8 = lane >> 2, j = lane & 3;
  const bool aborted = launch_aborted(p.c.err);
  // this CTA's units; the stages serve as scratch until the first copy
  KvPlace where = kv_place(p, kRows, reinterpret_cast<long long*>(smem_dec));
  if (__syncthreads_or(aborted) || where.at == where.end) return;
  const int cta = blockIdx.x, ctas = where.ctas;
  const long long total = where.total, begin = where.at, end = where.end;
  long long at = begin;

  uint64_t* full = reinterpret_cast<uint64_t*>(smem_dec + Sm::kBar);
  uint64_t* empty = full + kPairs * kStages;
  if (tid == 0) {
    for (int i = 0; i < kPairs * kStages; ++i) {
      mbar_init(&full[i]);
      asm volatile("mbarrier.init.shared::cta.b64 [%0], 2;" ::"r"(smem_addr(&empty[i])) : "memory");
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  fence_proxy_async();
  __syncthreads();

  __half* qs = reinterpret_cast<__half*>(smem_dec + Sm::kQ);
  float* st_ml = reinterpret_cast<float*>(smem_dec + Sm::kStat);
  float* st_c = st_ml + kWarps * kRows * 2;
  unsigned long long* see = reinterpret_cast<unsigned long long*>(smem_dec + Sm::kSee);
  float* po = reinterpret_cast<float*>(smem_dec);                // the warps' outputs, over the stages
  char* stages = smem_dec + pair * kStages * Sm::kStage;
  const T* q = static_cast<const T*>(p.q);
  T* out = static_cast<T*>(p.out);
  const __half2 k16 = __float2half2_rn(16.f), k24 = __float2half2_rn(-24.f);
  auto valid = [&](int g) { return g >= 0 && g < p.c.n_pages; };
  int n_joins = 0;
  int used = 0;          // pages this pair has put through its stages: stage used % kStages, phase used / kStages
  bool alive = true;
  int done = 0;          // pages of the segment in its partial result, from runs before this one

  while (at < end) {
    long long next;
    KvSegment it = kv_segment(p, kRows, at, end, where, &next);
    const bool folded = done > 0, over = it.pages - done <= kRun<T>;
    it.page_lo += done;
    it.pages = min(it.pages - done, kRun<T>);
    done = over ? 0 : done + kRun<T>;
    if (over) at = next;
    if (!it.r.ok) {
      if (tid == 0 && it.first)
        device_error(p.c.err, it.r.n < 1 || it.r.n > p.n_max ? GDN_DEVERR_SCHEDULE : GDN_DEVERR_CACHE, it.b);
      continue;
    }
    const int row0 = it.tile * kRows, rows = min(kRows, it.r.n * p.G - row0);
    const size_t node0 = static_cast<size_t>(it.bl) * p.n_max;
    auto q_row = [&](int r) {
      const int x = row0 + r;
      return q + (node0 + x / p.G) * p.q_row + static_cast<size_t>(it.h * p.G + x % p.G) * D;
    };
    // queries: loaded first, used below
    constexpr int kMine = (kRows + kWarps - 1) / kWarps;     // rows of a warp, loaded together
    float2 v[kMine][D / 64];
#pragma unroll
    for (int k = 0; k < kMine; ++k)
#pragma unroll
      for (int i = 0; i < D / 64; ++i) {
        const int r = warp + k * kWarps;
        v[k][i] = r < rows ? load2(q_row(r) + 64 * i + 2 * lane) : make_float2(0.f, 0.f);
      }
    // this pair's pages: page_lo + pair, + kPairs, ...; a lane holds the page numbers of 32 of them at a time
    const int mine = it.pages > pair ? (it.pages - pair + kPairs - 1) / kPairs : 0;
    const int32_t* table = p.c.page_table + static_cast<size_t>(it.b) * p.c.pages_max + it.page_lo + pair;
    auto page_no = [&](int i) { return i < mine ? table[i * kPairs] : -1; };
    int tbl = page_no(lane), tbl_next = page_no(32 + lane);       // iterations [32 k, 32 k + 32) and the next 32
    // one lane: page of iteration i into its stage; a page number out of range completes the stage with nothing,
    // so that the stages' phases count pages whatever they are
    auto fetch = [&](int i, int g) {
      const int st = (used + i) % kStages;
      uint64_t* bar = &full[pair * kStages + st];
      if (valid(g)) {
        mbar_expect(bar, Sm::kStage);
        bulk_g2s(stages + st * Sm::kStage, kv_block<D>(p.c, p.Hkv, g, it.l, it.h), Sm::kStage, bar);
      } else {
        mbar_arrive(bar);
        device_error(p.c.err, GDN_DEVERR_CACHE, it.b);
      }
    };
    const bool was_alive = alive;
    if (kb == 0 && alive) {
      for (int i = 0; i < kStages; ++i) {
        const int g = __shfl_sync(0xffffffffu, tbl, i);
        if (lane == 0 && i < mine) fetch(i, g);
      }
    }

    const bool with_new = it.first && over && p.k_new;
    if (with_new && lane == 0)      // the nodes' own rows are wanted last, from nearby
      for (int t = warp; t < it.r.n; t += kWarps) {
        const size_t row = (node0 + t) * p.kv_row + static_cast<size_t>(it.h) * D;
        prefetch_l2(static_cast<const T*>(p.k_new) + row, sizeof(T) * D);
        prefetch_l2(static_cast<const T*>(p.v_new) + row, sizeof(T) * D);
      }
    // queries: fp16, each row scaled by a power of two that brings its largest value to [2^13, 2^14)
    {
#pragma unroll
      for (int k = 0; k < kMine; ++k) {
        const int r = warp + k * kWarps;
        if (r >= kRows) break;
        float big = 0.f;
#pragma unroll
        for (int i = 0; i < D / 64; ++i) big = fmaxf(big, fmaxf(fabsf(v[k][i].x), fabsf(v[k][i].y)));
        for (int o = 16; o > 0; o >>= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, o));
        // 2^e <= big < 2^(e + 1); a zero or non-finite row stays as it is
        const int ex = static_cast<int>(__float_as_uint(big) >> 23);
        const int e = (big > 0.f && ex < 255) ? ex - 127 - 13 : 0;
        const float f0 = exp2i(-(e / 2)), f1 = exp2i(-(e - e / 2));
#pragma unroll
        for (int i = 0; i < D / 64; ++i) {
          const float x = v[k][i].x * f0 * f1, y = v[k][i].y * f0 * f1;
          const __half2 hi = __floats2half2_rn(x, y);
          __half2* at = reinterpret_cast<__half2*>(qs + r * Sm::kQRow + 64 * i + 2 * lane);
          at[0] = hi;
          if (kTerms == 2) at[kRows * Sm::kQRow / 2] = __floats2half2_rn(x - __low2float(hi), y - __high2float(hi));
        }
        if (lane == 0) st_c[r] = p.scale * kLog2e * exp2i(e / 2) * exp2i(e - e / 2);
      }
    }
    if (with_new && tid < rows) {
      const int32_t* parent = p.words ? kv_parents(p, it.b) : nullptr;
      if (!kv_root_path(parent, (row0 + tid) / p.G, &see[tid])) device_error(p.c.err, GDN_DEVERR_SCHEDULE, it.b);
    }
    __syncthreads();
    // B fragments of Q^T: step (hh, w, u) holds channels 128 hh + 32 j + 8 w + 4 u + {0,1} and {2,3} of row m8
    constexpr int kHalves = D == 256 ? 2 : 1;
    constexpr int kWords = D == 64 ? 2 : 4;        // words of a key chunk that this lane takes
    auto query = [&](int hh, int w, int u, int term) {       // read where they are used: registers go to the output
      const int c = D == 64 ? 16 * j + 8 * w + 4 * u : 128 * hh + 32 * j + 8 * w + 4 * u;
      return *reinterpret_cast<const uint2*>(qs + (term * kRows + m8) * Sm::kQRow + c);
    };
    const float c0 = st_c[2 * j], c1 = st_c[2 * j + 1];    // of rows 2j and 2j + 1, whose scores this lane holds

    float o[D / 32][2][4];
#pragma unroll
    for (int g = 0; g < D / 32; ++g)
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[g][x][i] = 0.f;
    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
    // a word's pair i (0..3) as values: code bits at 6..9 of each half
    auto pair_of = [&](uint32_t w, int i, __half2 a, __half2 b) {
      const uint32_t s = i == 0 ? w << 6 : i == 1 ? w << 2 : i == 2 ? w >> 2 : w >> 6;
      uint32_t v;                               // (s & mask) | one, in one operation
      asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(v) : "r"(s), "r"(0x03C003C0u), "r"(0x3C003C00u));
      return h2u(__hfma2(u2h(v), a, b));
    };

    for (int i = 0; i < mine && alive; ++i) {
      if (i > 0 && (i & 31) == 0) {
        tbl = tbl_next;
        tbl_next = page_no(i + 32 + lane);
      }
      const int g = __shfl_sync(0xffffffffu, tbl, i & 31);
      const int k = used + i, st = k % kStages;
      const int toks = min(32, it.r.len - (it.page_lo + pair + i * kPairs) * kPage - 32 * kb);
      if (!__all_sync(0xffffffffu, mbar_wait(&full[pair * kStages + st], (k / kStages) & 1))) {
        alive = false;
        break;
      }
      // refill the stage of the iteration before this one: the pair's other warp has most likely left it
      const int next = i - 1 + kStages;
      if (kb == 0 && i > 0 && next < mine) {
        const int at = next - (i & ~31);      // 32 at most: within the two tables held
        const int ga = __shfl_sync(0xffffffffu, tbl, at & 31), gb = __shfl_sync(0xffffffffu, tbl_next, at & 31);
        if (lane == 0) {
          if (mbar_wait(&empty[pair * kStages + (k - 1) % kStages], ((k - 1) / kStages) & 1))
            fetch(next, at < 32 ? ga : gb);
          else
            alive = false;
        }
        alive = __shfl_sync(0xffffffffu, alive, 0);
      }
      if (valid(g) && toks > 0) {
        const char* blk = stages + st * Sm::kStage;
        const uint32_t* kw = reinterpret_cast<const uint32_t*>(blk);
        const __half* kd = reinterpret_cast<const __half*>(blk + Blk::kKeyScales);
        // ---- S^T: M tile u holds tokens tok(2u, m8) in rows 0-7 and tok(2u + 1, m8) in rows 8-15
        auto tok = [&](int t) { return 32 * kb + 8 * (m8 >> 1) + 2 * t + (m8 & 1); };
        float s[2][4];
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int x = 0; x < 4; ++x) s[u][x] = 0.f;
#pragma unroll
        for (int hh = 0; hh < kHalves; ++hh) {
          uint32_t ww[4][kWords];
          __half2 d16[4], d24[4];
#pragma unroll
          for (int t = 0; t < 4; ++t) {
            int grp;
            if constexpr (D == 64) {
              const uint2 v = *reinterpret_cast<const uint2*>(kw + Blk::key_word(tok(t), 2 * j));
              ww[t][0] = v.x; ww[t][1] = v.y;
              grp = j >> 1;
            } else {
              const uint4 v = *reinterpret_cast<const uint4*>(kw + Blk::key_word(tok(t), 16 * hh + 4 * j));
              ww[t][0] = v.x; ww[t][1] = v.y; ww[t][2] = v.z; ww[t][3] = v.w;
              grp = 4 * hh + j;
            }
            const __half2 d = __half2half2(kd[tok(t) * Blk::kGroups + grp]);
            d16[t] = __hmul2(d, k16);
            d24[t] = __hmul2(d, k24);
          }
#pragma unroll
          for (int w = 0; w < kWords; ++w)
#pragma unroll
            for (int v = 0; v < 2; ++v) {
              const uint2 qv = query(hh, w, v, 0);
#pragma unroll
              for (int u = 0; u < 2; ++u) {
                const uint32_t a0 = pair_of(ww[2 * u][w], 2 * v, d16[2 * u], d24[2 * u]),
                               a1 = pair_of(ww[2 * u + 1][w], 2 * v, d16[2 * u + 1], d24[2 * u + 1]),
                               a2 = pair_of(ww[2 * u][w], 2 * v + 1, d16[2 * u], d24[2 * u]),
                               a3 = pair_of(ww[2 * u + 1][w], 2 * v + 1, d16[2 * u + 1], d24[2 * u + 1]);
                if constexpr (kTerms == 1) {
                  mma16816(s[u], a0, a1, a2, a3, qv.x, qv.y);
                } else {               // sixteen channels at a time, summed outside: the MMA's own additions truncate
                  const uint2 ql = query(hh, w, v, 1);
                  float t[4] = {0.f, 0.f, 0.f, 0.f};
                  mma16816(t, a0, a1, a2, a3, ql.x, ql.y);
                  mma16816(t, a0, a1, a2, a3, qv.x, qv.y);
#pragma unroll
                  for (int x = 0; x < 4; ++x) s[u][x] += t[x];
                }
              }
            }
        }
        // ---- weights: this lane holds rows 2j (x = 0, 2) and 2j + 1 (x = 1, 3)
        float n0 = m0, n1 = m1;
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int x = 0; x < 4; ++x) s[u][x] *= (x & 1) ? c1 : c0;
        if (toks < 32) {
#pragma unroll
          for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int x = 0; x < 4; ++x)
              if (tok(2 * u + (x >> 1)) - 32 * kb >= toks) s[u][x] = -INFINITY;
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          n0 = fmaxf(n0, fmaxf(s[u][0], s[u][2]));
          n1 = fmaxf(n1, fmaxf(s[u][1], s[u][3]));
        }
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) {
          n0 = fmaxf(n0, __shfl_xor_sync(0xffffffffu, n0, off));
          n1 = fmaxf(n1, __shfl_xor_sync(0xffffffffu, n1, off));
        }
        if (__any_sync(0xffffffffu, n0 - m0 > kSlack || n1 - m1 > kSlack)) {       // (the sums would round)
          const float f0 = m0 == -INFINITY ? 0.f : exp2f(m0 - n0), f1 = m1 == -INFINITY ? 0.f : exp2f(m1 - n1);
          m0 = n0;
          m1 = n1;
          l0 *= f0;
          l1 *= f1;
#pragma unroll
          for (int gg = 0; gg < D / 32; ++gg)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              o[gg][x][0] *= f0;
              o[gg][x][1] *= f1;
              o[gg][x][2] *= f0;
              o[gg][x][3] *= f1;
            }
        }
        // a row whose scores so far are all -inf keeps weight 0 (its maximum is not subtracted)
        // (rounded down: where the scores' own steps are larger than kLift, no weight passes fp16's largest number)
        const float r0 = m0 == -INFINITY ? kLift : __fsub_rd(kLift, m0), r1 = m1 == -INFINITY ? kLift : __fsub_rd(kLift, m1);
        uint32_t pf[kTerms][2][2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
#pragma unroll
          for (int x = 0; x < 4; ++x) s[u][x] = exp2_fast(s[u][x] + ((x & 1) ? r1 : r0));
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const __half2 hi = __floats2half2_rn(s[u][2 * x], s[u][2 * x + 1]);
            pf[0][u][x] = transpose8x8(h2u(hi));
            if constexpr (kTerms == 2)
              pf[1][u][x] = transpose8x8(
                  h2u(__floats2half2_rn((s[u][2 * x] - __low2float(hi)) * kLowScale, (s[u][2 * x + 1] - __high2float(hi)) * kLowScale)));
          }
        }
        l0 += (s[0][0] + s[0][2]) + (s[1][0] + s[1][2]);
        l1 += (s[0][1] + s[0][3]) + (s[1][1] + s[1][3]);
        // ---- O^T: tile (gg, x) holds channel 32 gg + 4 m8 + 2x in rows 0-7 and the next one in rows 8-15; step u
        // takes tokens 8j + 4u .. + 3 of the 32
        const uint4* vw = reinterpret_cast<const uint4*>(blk + Blk::kValCodes) + kb * D;
        const __half* vd = reinterpret_cast<const __half*>(blk + Blk::kValScales) + 32 * kb + 8 * j;
#pragma unroll
        for (int gg = 0; gg < D / 32; ++gg) {
          const uint4 wv = vw[(8 * gg + m8) * 4 + j];
          uint4 dv = *reinterpret_cast<const uint4*>(vd + gg * kPage);
          uint32_t dd[4] = {dv.x, dv.y, dv.z, dv.w};
          if (toks < 32) {                        // scales past the length are whatever the page held
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const int left = toks - (8 * j + 2 * x);
              dd[x] = left <= 0 ? 0u : left == 1 ? dd[x] & 0xFFFFu : dd[x];
            }
          }
          const uint32_t ww[4] = {wv.x, wv.y, wv.z, wv.w};
          // fp32 calls: these tokens' products with the two terms of the weights, summed outside like the scores'
          float page[2][4] = {}, low[2][4] = {};
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const __half2 e0 = u2h(dd[2 * u]), e1 = u2h(dd[2 * u + 1]);
            const __half2 a0 = __hmul2(e0, k16), b0 = __hmul2(e0, k24), a1 = __hmul2(e1, k16), b1 = __hmul2(e1, k24);
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const uint32_t f0 = pair_of(ww[2 * x], 2 * u, a0, b0), f1 = pair_of(ww[2 * x + 1], 2 * u, a0, b0),
                             f2 = pair_of(ww[2 * x], 2 * u + 1, a1, b1), f3 = pair_of(ww[2 * x + 1], 2 * u + 1, a1, b1);
              if constexpr (kTerms == 1) {
                mma16816(o[gg][x], f0, f1, f2, f3, pf[0][u][0], pf[0][u][1]);
              } else {
                mma16816(low[x], f0, f1, f2, f3, pf[kTerms - 1][u][0], pf[kTerms - 1][u][1]);
                mma16816(page[x], f0, f1, f2, f3, pf[0][u][0], pf[0][u][1]);
              }
            }
          }
          if constexpr (kTerms == 2) {
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
              for (int y = 0; y < 4; ++y) o[gg][x][y] += fmaf(low[x][y], 1.f / kLowScale, page[x][y]);
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[pair * kStages + st]);
    }
    used += mine;
    if (was_alive && !alive) {
      if (lane == 0) device_error(p.c.err, GDN_DEVERR_TIMEOUT, it.b);
      // let this pair's copies land before the CTA exits
      for (int st = 0; st < kStages; ++st)
        for (int par = 0; par < 2; ++par) mbar_wait(&full[pair * kStages + st], par);
    }
#pragma unroll
    for (int off = 4; off < 32; off <<= 1) {
      l0 += __shfl_xor_sync(0xffffffffu, l0, off);
      l1 += __shfl_xor_sync(0xffffffffu, l1, off);
    }
    // ---- the CTA's warps meet: outputs [warp][row][D] over the stages, maxima and sums beside them
    __syncthreads();
#pragma unroll
    for (int gg = 0; gg < D / 32; ++gg)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int c = 32 * gg + 4 * m8 + 2 * x;
        *reinterpret_cast<float2*>(po + (warp * kRows + 2 * j) * D + c) = make_float2(o[gg][x][0], o[gg][x][2]);
        *reinterpret_cast<float2*>(po + (warp * kRows + 2 * j + 1) * D + c) = make_float2(o[gg][x][1], o[gg][x][3]);
      }
    if (lane < 4) {
      *reinterpret_cast<float2*>(st_ml + (warp * kRows + 2 * j) * 2) = make_float2(m0, l0);
      *reinterpret_cast<float2*>(st_ml + (warp * kRows + 2 * j + 1) * 2) = make_float2(m1, l1);
    }
    __syncthreads();

    auto out_row = [&](int r) {
      const int x = row0 + r;
      return out + (node0 + x / p.G) * (static_cast<size_t>(p.Hq) * D) + static_cast<size_t>(it.h * p.G + x % p.G) * D;
    };
    // (an item that the CTA holds whole has no partial result of its own, and its place is free)
    float* slot = kv_stream_part(p, cta, it.start > begin, kRows, D);
    float* part = it.whole && over ? nullptr : slot;
    for (int r = warp; r < rows; r += kWarps) {
      float m = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) m = fmaxf(m, st_ml[(w * kRows + r) * 2]);
      float acc[D / 32], l = 0.f;
#pragma unroll
      for (int i = 0; i < D / 32; ++i) acc[i] = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float mw = st_ml[(w * kRows + r) * 2], lw = st_ml[(w * kRows + r) * 2 + 1];
        if (mw == -INFINITY && lw == 0.f) continue;
        const float f = exp2f(mw - m);
        l = fmaf(f, lw, l);
#pragma unroll
        for (int i = 0; i < D / 64; ++i) {
          const float2 v = *reinterpret_cast<const float2*>(po + (w * kRows + r) * D + 64 * i + 2 * lane);
          acc[2 * i] = fmaf(f, v.x, acc[2 * i]);
          acc[2 * i + 1] = fmaf(f, v.y, acc[2 * i + 1]);
        }
      }
      if (folded) {                      // (a warp's own rows, written by the same lanes)
        const float2 before = *reinterpret_cast<const float2*>(slot + kRows * D + 2 * r);
        const float mn = fmaxf(m, before.x);
        const float fo = m == -INFINITY ? 0.f : exp2f(m - mn), fs = before.x == -INFINITY ? 0.f : exp2f(before.x - mn);
        m = mn;
        l = fmaf(l, fo, before.y * fs);
#pragma unroll
        for (int i = 0; i < D / 64; ++i) {
          const float2 v = *reinterpret_cast<const float2*>(slot + r * D + 64 * i + 2 * lane);
          acc[2 * i] = fmaf(acc[2 * i], fo, v.x * fs);
          acc[2 * i + 1] = fmaf(acc[2 * i + 1], fo, v.y * fs);
        }
        __syncwarp();                    // read by all lanes before one writes the sums
      }
      if (with_new) {
        // the row's own ancestors, one at a time in fp32: what it does not see is not read
        const T* kn = static_cast<const T*>(p.k_new) + static_cast<size_t>(it.h) * D + 2 * lane;
        const T* vn = static_cast<const T*>(p.v_new) + static_cast<size_t>(it.h) * D + 2 * lane;
        float2 qv[D / 64];
#pragma unroll
        for (int i = 0; i < D / 64; ++i) qv[i] = load2(q_row(r) + 64 * i + 2 * lane);
        unsigned long long left = see[r];
        while (left) {
          const int t = __ffsll(static_cast<long long>(left)) - 1;
          left &= left - 1;
          const size_t at = (node0 + t) * p.kv_row;
          float x = 0.f;
          float2 vv[D / 64];
#pragma unroll
          for (int i = 0; i < D / 64; ++i) {
            const float2 kv = load2(kn + at + 64 * i);
            vv[i] = load2(vn + at + 64 * i);
            x = fmaf(qv[i].x, kv.x, fmaf(qv[i].y, kv.y, x));
          }
          for (int off = 16; off > 0; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
          x *= p.scale * kLog2e;
          const float mn = fmaxf(m, x);
          const float f = m == -INFINITY ? 0.f : exp2f(m - mn);
          const float wt = x == -INFINITY ? 0.f : exp2f(x - mn + kLift);
          m = mn;
          l = fmaf(l, f, wt);
#pragma unroll
          for (int i = 0; i < D / 64; ++i) {
            acc[2 * i] = fmaf(acc[2 * i], f, wt == 0.f ? 0.f : wt * vv[i].x);
            acc[2 * i + 1] = fmaf(acc[2 * i + 1], f, wt == 0.f ? 0.f : wt * vv[i].y);
          }
        }
      }
      if (part) {
#pragma unroll
        for (int i = 0; i < D / 64; ++i)
          *reinterpret_cast<float2*>(part + r * D + 64 * i + 2 * lane) = make_float2(acc[2 * i], acc[2 * i + 1]);
        if (lane == 0) *reinterpret_cast<float2*>(part + kRows * D + 2 * r) = make_float2(m, l);
      } else {
        const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
        for (int i = 0; i < D / 64; ++i)
          store2(out_row(r) + 64 * i + 2 * lane, acc[2 * i] * inv, acc[2 * i + 1] * inv);
      }
    }
    if (over && !it.whole) {
      const int c0 = kv_cta_of(it.start, total, ctas), c1 = kv_cta_of(it.start + it.r.units - 1, total, ctas);
      if (kv_last(p, it.item, c1 - c0 + 1, &last)) {     // joined after the loop: at most two
        if (tid == 0)
          joins[n_joins] = {c0, c1 - c0 + 1, rows, it.start > kv_unit_of(c0, total, ctas), it.b, it.l, it.h, row0};
        ++n_joins;
      }
    }
    // the next item's copies go where the outputs were just read; a timeout ends the CTA's work, not its count
    fence_proxy_async();
    if (__syncthreads_or(!alive)) alive = false;
  }
  for (int i = 0; i < n_joins; ++i) {
    const KvJoin t = joins[i];
    const size_t node = (static_cast<size_t>(t.b) * p.layers + t.l) * p.n_max;
    kv_join_rows<T, D>(p.part, t, kRows, out + (node * p.Hq + t.h * p.G) * D, p.G, static_cast<long long>(p.Hq) * D, po);
    __syncthreads();
  }
}

template <int D, typename T>
cudaError_t dec_t(KvAttnParams p, cudaStream_t s) {
  auto k = kv4_attn_dec_kernel<D, T>;
  cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, Smem<D, T>::kTotal);
  if (e != cudaSuccess) return e;
  // as many requests a launch as have counters
  const int items = p.layers * p.Hkv * p.row_tiles, per = kKvCounters / items;
  p.each = p.ctas / items;
  for (p.b0 = 0; p.b0 < p.c.B; p.b0 += per) {
    p.bn = p.c.B - p.b0 < per ? p.c.B - p.b0 : per;
    k<<<p.ctas, 32 * kWarpsOf<D>, Smem<D, T>::kTotal, s>>>(p);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace

cudaError_t launch_kv4_attention_dec(const KvAttnParams& p, cudaStream_t s) {
  if (p.dtype == GDN_DTYPE_F32)
    return p.D == 256 ? dec_t<256, float>(p, s) : p.D == 128 ? dec_t<128, float>(p, s) : dec_t<64, float>(p, s);
  return p.D == 256   ? dec_t<256, __nv_bfloat16>(p, s)
         : p.D == 128 ? dec_t<128, __nv_bfloat16>(p, s)
                      : dec_t<64, __nv_bfloat16>(p, s);
}

}  // namespace gdn
