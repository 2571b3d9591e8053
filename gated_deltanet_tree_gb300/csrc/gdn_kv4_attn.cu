// Attention over the paged 4-bit cache on the CUDA cores, in fp32 throughout, and
// the plan of the work's split that all attention kernels share.
//
// One CTA takes a tile of 16 rows -- (node, query head) pairs that share a kv
// head -- over one chunk of the request's pages.  Tiles of 32 tokens are unpacked
// to fp32 in shared memory; scores, the running maximum and sum of the softmax
// and the output stay in fp32 (registers).  The nodes' own rows are one more
// token tile, taken by chunk 0, with each row's ancestors as its mask: a masked
// weight is not multiplied at all there, so that a NaN in a row that is not seen
// stays out.  Chunks write an unnormalised output with its maximum and sum; the
// last chunk of a tile to finish joins them in chunk order, so the result does
// not depend on which one that was.
#include "gdn_kv4_attn.cuh"

namespace gdn {
namespace {

constexpr int kThreads = 128;
constexpr int kRows = 16;      // rows of a tile
constexpr int kToks = 32;      // tokens of a tile

template <typename T>
__device__ __forceinline__ float to_f(T x) { return static_cast<float>(x); }
template <>
__device__ __forceinline__ float to_f<__nv_bfloat16>(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void from_f(float* p, float x) { *p = x; }
__device__ __forceinline__ void from_f(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

// shared: qs [16][D] | ks [32][D + 4] | vs [32][D] | pt [32][16] | stat [3][16] (max, sum, rescale)
template <int D>
constexpr size_t simt_smem() {
  return sizeof(float) * (kRows * D + kToks * (D + 4) + kToks * D + kToks * kRows + 3 * kRows) + 64 * 8;
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) kv4_attn_simt_kernel(KvAttnParams p) {
  using Blk = KvBlock<D>;
  extern __shared__ float smem_simt[];
  float* qs = smem_simt;
  float* ks = qs + kRows * D;
  float* vs = ks + kToks * (D + 4);
  float* pt = vs + kToks * D;
  float* st_m = pt + kToks * kRows;
  float* st_l = st_m + kRows;
  float* st_s = st_l + kRows;
  unsigned long long* see = reinterpret_cast<unsigned long long*>(st_s + kRows);
  __shared__ int last;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const KvItem it = kv_item(p, blockIdx.x);
  const int chunk = blockIdx.y;
  const KvSpan sp = kv_span(p, it, chunk);
  if (!sp.ok) {
    if (tid == 0 && chunk == 0) device_error(p.c.err, sp.bit, it.b);
    return;
  }
  const int row0 = it.tile * kRows, rows = min(kRows, sp.n * p.G - row0);
  if (rows <= 0 || chunk >= sp.chunks) return;

  const size_t node0 = static_cast<size_t>(it.bl) * p.n_max;
  const T* q = static_cast<const T*>(p.q);
  for (int i = tid; i < kRows * D; i += kThreads) {
    const int r = i / D, d = i % D, row = row0 + r;
    qs[i] = r < rows ? to_f(q[(node0 + row / p.G) * p.q_row + (it.h * p.G + row % p.G) * D + d]) * (p.scale * 1.4426950408889634f) : 0.f;
  }
  if (tid < kRows) {
    st_m[tid] = -INFINITY;
    st_l[tid] = 0.f;
  }
  // output: thread owns two channels of kRows / kSlices rows
  constexpr int kSlices = 2 * kThreads / D, kOwn = kRows / kSlices;
  const int oc = 2 * (tid % (D / 2)), or0 = (tid / (D / 2)) * kOwn;
  float o0[kOwn], o1[kOwn];
#pragma unroll
  for (int i = 0; i < kOwn; ++i) o0[i] = o1[i] = 0.f;

  // one tile of `toks` tokens in ks / vs; kNew: masked by the rows' ancestors (nodes t0 ..)
  auto tile = [&](int toks, int t0, bool is_new) {
    // scores: two rows x two tokens per thread
    {
      const int r = 2 * (tid & 7), t = 2 * (tid >> 3);
      float s00 = 0.f, s01 = 0.f, s10 = 0.f, s11 = 0.f;
      const float *qa = qs + r * D, *ka = ks + t * (D + 4);
#pragma unroll 8
      for (int d = 0; d < D; d += 4) {
        const float4 a = *reinterpret_cast<const float4*>(qa + d), b = *reinterpret_cast<const float4*>(qa + D + d);
        const float4 c = *reinterpret_cast<const float4*>(ka + d),
                     e = *reinterpret_cast<const float4*>(ka + D + 4 + d);
        s00 = fmaf(a.x, c.x, fmaf(a.y, c.y, fmaf(a.z, c.z, fmaf(a.w, c.w, s00))));
        s01 = fmaf(a.x, e.x, fmaf(a.y, e.y, fmaf(a.z, e.z, fmaf(a.w, e.w, s01))));
        s10 = fmaf(b.x, c.x, fmaf(b.y, c.y, fmaf(b.z, c.z, fmaf(b.w, c.w, s10))));
        s11 = fmaf(b.x, e.x, fmaf(b.y, e.y, fmaf(b.z, e.z, fmaf(b.w, e.w, s11))));
      }
      const float s[2][2] = {{s00, s01}, {s10, s11}};
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          bool vis = t + j < toks;
          if (is_new && vis) vis = r + i < rows && (see[(row0 + r + i) / p.G] >> (t0 + t + j)) & 1;
          pt[(t + j) * kRows + r + i] = vis ? s[i][j] : -INFINITY;
        }
    }
    __syncthreads();
    // softmax: warp w holds rows 4w .. 4w + 3, a lane a token
#pragma unroll
    for (int i = 0; i < kRows / 4; ++i) {
      const int r = warp * (kRows / 4) + i;
      const float x = pt[lane * kRows + r];
      float mx = x;
      // a NaN score has to reach the result: fmaxf drops it, so it is carried by the weight below
      for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      const float m0 = st_m[r], m1 = fmaxf(m0, mx);
      const float w = (x == -INFINITY) ? 0.f : exp2f(x - m1);
      float sum = w;
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      pt[lane * kRows + r] = w;
      if (lane == 0) {
        const float c = m0 == -INFINITY ? 0.f : exp2f(m0 - m1);
        st_m[r] = m1;
        st_l[r] = st_l[r] * c + sum;
        st_s[r] = c;
      }
      __syncwarp();
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kOwn; ++i) {
      o0[i] *= st_s[or0 + i];
      o1[i] *= st_s[or0 + i];
    }
    for (int t = 0; t < toks; ++t) {
      const float2 v = *reinterpret_cast<const float2*>(vs + t * D + oc);
#pragma unroll
      for (int i = 0; i < kOwn; ++i) {
        const float w = pt[t * kRows + or0 + i];
        if (is_new && w == 0.f) continue;
        o0[i] = fmaf(w, v.x, o0[i]);
        o1[i] = fmaf(w, v.y, o1[i]);
      }
    }
    __syncthreads();
  };

  if (chunk == 0 && p.k_new) {
    if (!kv_ancestors(p, it.b, sp.n, see)) {
      if (tid == 0) device_error(p.c.err, GDN_DEVERR_SCHEDULE, it.b);
    }
    const T* kn = static_cast<const T*>(p.k_new);
    const T* vn = static_cast<const T*>(p.v_new);
    for (int t0 = 0; t0 < sp.n; t0 += kToks) {
      const int toks = min(kToks, sp.n - t0);
      for (int i = tid; i < kToks * D; i += kThreads) {
        const int t = i / D, d = i % D;
        const size_t at = (node0 + t0 + t) * p.kv_row + it.h * D + d;
        ks[t * (D + 4) + d] = t < toks ? to_f(kn[at]) : 0.f;
        vs[t * D + d] = t < toks ? to_f(vn[at]) : 0.f;
      }
      __syncthreads();
      tile(toks, t0, true);
    }
  }
  const int32_t* table = p.c.page_table + static_cast<size_t>(it.b) * p.c.pages_max;
  for (int pg = sp.page_lo; pg < sp.page_hi; ++pg) {
    const int g = table[pg];
    if (g < 0 || g >= p.c.n_pages) {     // the whole CTA reads the same number
      if (tid == 0) device_error(p.c.err, GDN_DEVERR_CACHE, it.b);
      continue;
    }
    const char* blk = kv_block<D>(p.c, p.Hkv, g, it.l, it.h);
    const uint32_t* kw = reinterpret_cast<const uint32_t*>(blk);
    const uint32_t* vw = reinterpret_cast<const uint32_t*>(blk + Blk::kValCodes);
    const __half* kd = reinterpret_cast<const __half*>(blk + Blk::kKeyScales);
    const __half* vd = reinterpret_cast<const __half*>(blk + Blk::kValScales);
    for (int half = 0; half < 2; ++half) {
      const int toks = min(kToks, sp.len - pg * kPage - half * kToks);
      if (toks <= 0) break;
      for (int i = tid; i < kToks * (D / 8); i += kThreads) {
        const int t = i / (D / 8), w = i % (D / 8), r = half * kToks + t;
        const uint32_t word = kw[Blk::key_word(r, w)];
        const float d = t < toks ? __half2float(kd[r * Blk::kGroups + (w >> 2)]) : 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e)
          ks[t * (D + 4) + 8 * w + e] = static_cast<float>(static_cast<int>((word >> (4 * nibble_of(e))) & 15u) - 8) * d;
      }
      for (int i = tid; i < 4 * D; i += kThreads) {
        const int c = i % D, o = i / D;
        const uint32_t word = vw[Blk::val_word(c, half * 4 + o)];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int t = 8 * o + e;
          const float d = t < toks ? __half2float(vd[(c / kGroup) * kPage + half * kToks + t]) : 0.f;
          vs[t * D + c] = static_cast<float>(static_cast<int>((word >> (4 * nibble_of(e))) & 15u) - 8) * d;
        }
      }
      __syncthreads();
      tile(toks, 0, false);
    }
  }

  // result of this chunk; the last chunk of the tile joins all of them
  T* out = static_cast<T*>(p.out);
  auto out_at = [&](int row) {
    return (node0 + row / p.G) * (static_cast<size_t>(p.Hq) * D) + static_cast<size_t>(it.h * p.G + row % p.G) * D;
  };
  if (sp.chunks == 1) {
#pragma unroll
    for (int i = 0; i < kOwn; ++i) {
      const int r = or0 + i;
      if (r >= rows) break;
      const float l = st_l[r], inv = l == 0.f ? 0.f : 1.f / l;
      from_f(out + out_at(row0 + r) + oc, o0[i] * inv);
      from_f(out + out_at(row0 + r) + oc + 1, o1[i] * inv);
    }
    return;
  }
  float* part = kv_part(p, blockIdx.x, chunk, kRows, D);
#pragma unroll
  for (int i = 0; i < kOwn; ++i) {
    const int r = or0 + i;
    if (r >= rows) break;
    *reinterpret_cast<float2*>(part + r * (D + 2) + oc) = make_float2(o0[i], o1[i]);
    if (oc == 0) *reinterpret_cast<float2*>(part + r * (D + 2) + D) = make_float2(st_m[r], st_l[r]);
  }
  if (!kv_last_chunk(p, blockIdx.x, sp.chunks, &last)) return;
  for (int r = warp; r < rows; r += kThreads / 32)
    kv_join_row<T, D>(p, blockIdx.x, sp.chunks, kRows, r, out + out_at(row0 + r));
}

template <typename T, int D>
cudaError_t simt_t(const KvAttnParams& p, cudaStream_t s) {
  auto k = kv4_attn_simt_kernel<T, D>;
  if (simt_smem<D>() > 48 * 1024) {
    cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(simt_smem<D>()));
    if (e != cudaSuccess) return e;
  }
  const dim3 grid(static_cast<unsigned>(p.c.B) * p.layers * p.Hkv * p.row_tiles, p.chunks);
  k<<<grid, kThreads, simt_smem<D>(), s>>>(p);
  return cudaGetLastError();
}

}  // namespace

// Which kernel takes a call, and how its tokens are split.  Up to eight rows a kv head in bf16 the cache's bytes are
// the bound and kv4_attn_dec_kernel moves them best; with more rows kv4_attn_tree_kernel shares the unpacking among
// them.  fp32 calls (and more layers and heads than a launch has records for) go to the CUDA cores.
//
// On the CUDA cores the tokens are split in as many chunks as fill the GPU, so that a lone request is spread over it,
// but none so short that its own start and join cost more than its pages.
KvAttnPlan plan_kv4_attention(int Hq, int Hkv, int D, int dtype, int B, int layers, int n_max, int pages) {
  KvAttnPlan pl{};
  const long long rows = static_cast<long long>(n_max) * (Hq / Hkv);
  pl.done_bytes = kKvCounters * sizeof(int32_t) + kKvItems * sizeof(int4);
  if (dtype == GDN_DTYPE_BF16 && rows <= kKvDecRows && static_cast<long long>(layers) * Hkv <= kKvCounters) {
    // units: two CTAs an SM, and at least a page for each of a CTA's pairs of warps
    pl.kernel = kKvDec;
    pl.tile_rows = kKvDecRows;
    pl.row_tiles = 1;
    pl.least = D == 256 ? 3 : 4;
    pl.ctas = 152 * 2;
    pl.bytes = pl.done_bytes + static_cast<size_t>(pl.ctas) * 2 * pl.tile_rows * (D + 2) * sizeof(float);
    return pl;
  }
  pl.tile_rows = kKvTreeRows;
  pl.row_tiles = static_cast<int>((rows + pl.tile_rows - 1) / pl.tile_rows);
  if (dtype == GDN_DTYPE_BF16 && static_cast<long long>(layers) * Hkv * pl.row_tiles <= kKvItems) {
    pl.kernel = kKvTree;
    pl.least = 2;
    pl.ctas = 152;
    pl.bytes = pl.done_bytes + static_cast<size_t>(pl.ctas) * 2 * pl.tile_rows * (D + 2) * sizeof(float);
    return pl;
  }
  pl.kernel = kKvSimt;
  pl.tile_rows = kRows;
  const int want = 152 * 6, least = 2;      // CTAs that fill the GPU; pages a chunk has at least
  pl.row_tiles = static_cast<int>((rows + pl.tile_rows - 1) / pl.tile_rows);
  const long long tiles = static_cast<long long>(B) * layers * Hkv * pl.row_tiles;
  long long chunks = (want + tiles - 1) / tiles;
  const long long most = (pages + least - 1) / least;
  chunks = tiles > kKvCounters ? 1 : chunks > most ? most : chunks;
  chunks = chunks < 1 ? 1 : chunks;
  pl.chunk_pages = static_cast<int>((pages + chunks - 1) / chunks);
  pl.chunk_pages = pl.chunk_pages < 1 ? 1 : pl.chunk_pages;
  pl.chunks = static_cast<int>(chunks);
  pl.bytes = pl.done_bytes;
  if (chunks > 1) pl.bytes += static_cast<size_t>(tiles) * chunks * pl.tile_rows * (D + 2) * sizeof(float);
  return pl;
}

cudaError_t launch_kv4_attention_simt(const KvAttnParams& p, cudaStream_t s) {
  if (p.dtype == GDN_DTYPE_BF16)
    return p.D == 256 ? simt_t<__nv_bfloat16, 256>(p, s) : p.D == 128 ? simt_t<__nv_bfloat16, 128>(p, s) : simt_t<__nv_bfloat16, 64>(p, s);
  return p.D == 256 ? simt_t<float, 256>(p, s) : p.D == 128 ? simt_t<float, 128>(p, s) : simt_t<float, 64>(p, s);
}

}  // namespace gdn
