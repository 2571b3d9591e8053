// Attention over the paged 4-bit cache for trees: up to 128 (node, query head)
// pairs that share a kv head per tile, on tcgen05.  bf16 calls.
//
// With tens of rows per kv head the two products are the bound (4 D operations a
// row and token), so the rows fill a 128-row tile and the cache is unpacked to
// fp16 in shared memory for the fifth-generation tensor cores, one page (64
// tokens) a step, or two where D is 128 or less (their halved work a page left the
// step's fixed costs standing: 16 trees of 8 nodes, 32 rows a head, 76 us against 70).
// Tensor memory (512 columns) holds everything else: the output O[128][D] in fp32,
// the queries as the A operand of S = Q K^T, and two score buffers; the weights
// overwrite the scores they came from and are the A operand of O += P V.  The scores
// of one step are computed while the step before it goes through the softmax.
//
// Roles (18 warps, one CTA an SM): eight softmax warps, two threads a row that take
// the steps in turn and hand each other the row's reference maximum; four warps
// unpack keys and four values (codes to fp16: see gdn_kv4_dec.cu); one warp issues
// the bulk copies of the pages, one the MMAs.  They meet at mbarriers only; every
// wait is bounded.  CTAs take equal runs of the requests' pages (KvPlace); items that
// two or more CTAs share are joined by a second kernel, spread over the GPU.
//
// The nodes' own rows are one more step of an item, the last; their values are
// fetched while the pages go by.  They are fp16 like the rest, each key row scaled
// to fp16's range by a power of two, the row's ancestors as its mask.  A masked weight is 0, which would still turn a NaN or an infinity
// in an unseen row into NaN inside a product; if any such value (or one outside
// fp16's range) is among the rows, that step is left out of the products and each row
// adds its own ancestors in fp32 at the end.
//
// Measured: trees of 64 and 48 nodes over 200001 and 150001 tokens (three tiles each),
// 24 query and 4 kv heads of 256: 497 to 515 us from run to run, 0.94 to 0.97 PFLOP/s of
// useful products, about half of cuBLAS' bf16 rate.  A 64-token step takes about 1.9
// times its MMAs' 1024 cycles; issue slots
// (60%) and the latencies of tensor memory share the rest.
#include "gdn_kv4_attn.cuh"
#include "gdn_umma.cuh"

namespace gdn {
namespace {

constexpr int kSoftWarps = 8, kKeyWarps = 4, kUnpackWarps = 8;      // of the latter, kKeyWarps for the keys
constexpr int kCopyWarp = kSoftWarps + kUnpackWarps, kMmaWarp = kCopyWarp + 1;
constexpr int kThreads = 32 * (kMmaWarp + 1);
constexpr int kRows = kKvTreeRows;
constexpr int kStages = 3;
// Weights are scaled by 2^kLift against a reference that the largest may pass by 2^kSlack: 2^15 at most in fp16.  Its
// rounding error is then 2^-31 of the reference at most, what T tokens' weights lose together T 2^-31 (5e-4 at a million
// tokens, a quarter of bf16's own rounding).  Two more for the lift and less for the slack has the output rescaled more
// often (32 22-node trees 155 -> 160 us, 64-node trees over 200k tokens 513 -> 522); 2 and 13 gains nothing over these.
constexpr float kLift = 6.f;
constexpr float kSlack = 9.f;
// Additions into the output in tensor memory truncate: 16 tokens at a time, each by up to 2^-23 of what is there, which
// a million tokens behind one that dominates make 2^-7 of the output.  A segment is therefore taken in runs of pages,
// joined in fp32 in the place of its partial result: 131072 tokens a run leave 2^-10, and cost a start and an end
// (some 10 us of 2 ms).
constexpr int kRun = 2048;
constexpr float kLarge = 0x1p22f;     // scores (base 2) whose steps are 1/2 or more
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kTooLarge = 6.0e4f;   // new values beyond this take the fp32 path,
constexpr float kTooSmall = 0x1p-12f; // as do those that fp16 rounds (below 2^-17) where eight nodes' channel has none this large

// kScored: scores written, which also frees the key operand; kAdded: product added to the output, which also frees the
// value operand (a commit costs the issuing thread some two hundred cycles, so there is one for each)
enum Bar { kStFull = 0, kStEmpty = 3, kKFull = 6, kVFull = 8, kScored = 10, kPFull = 12, kAdded = 14, kOFree = 16,
           kQReady = 17, kNewFull = 18, kDrain = 19, kPair = 20, kDecided = 24, kItem = 28, kSoft = 29,
           kKeyMeet = 30, kValMeet = 31, kBars = 32 };

template <int D>
struct Smem {
  static constexpr int kPages = D == 256 ? 1 : 2, kTok = kPages * kPage;      // pages and tokens of a step
  static constexpr int kBlock = KvBlock<D>::kBytes, kStage = kPages * kBlock;
  // operands without swizzle: 8 rows x 16 bytes contiguous; adjacent row groups 128 bytes apart, adjacent groups of
  // eight elements along K `kKeyK` / `kValK` bytes (the values' 16 bytes more spread the unpackers' stores over all banks)
  static constexpr int kKeyK = kTok * 16, kValK = D * 16 + 16;
  static constexpr int kKeyTile = (D / 8) * kKeyK, kValTile = (kTok / 8) * kValK;
  static constexpr int kKeys = kStages * kStage;
  static constexpr int kVals = kKeys + 2 * kKeyTile;
  static constexpr int kSee = kVals + 2 * kValTile;                // u64 [64]
  static constexpr int kColScale = kSee + GDN_MAX_NODES * 8;       // float [kTok]
  static constexpr int kBar = kColScale + kTok * 4;
  static constexpr int kTmem = kBar + kBars * 8;                   // tensor-memory address, flags
  static constexpr int kSwap = kTmem + 32;                         // float [2][2][128]: what the two threads of a row tell each other
  static constexpr int kRef = kSwap + 4 * kRows * 4;               // float [128]: each row's reference maximum
  static constexpr int kRawVal = kRef + kRows * 4;                 // bf16 [64][D]: the nodes' own value rows as they came
  static constexpr int kTotal = kRawVal + GDN_MAX_NODES * D * 2;
  // tensor-memory columns
  static constexpr int kO = 0, kQ = D, kS = D + D / 2;
  static constexpr int kCols = 512;
  static_assert(kS + 2 * kTok <= kCols, "output, queries and two score buffers");
};

__host__ __device__ constexpr uint32_t idesc_f16(int m, int n) {
  return (1u << 4) | (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(m >> 4) << 24);
}
// D = A B^T or D += A B^T, kind::f16 (K = 16), A in tensor memory.
template <bool kAdd>
__device__ __forceinline__ void umma_f16_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "n"(kAdd ? 1 : 0)
      : "memory");
}
// Sixteen bytes of global memory to shared memory, asynchronously; complete after copy16_wait() in the thread that issued
// it.  Code that runs once an item is kept small -- rolled loops of such copies instead of loads unrolled into registers:
// an SM fetches cold code at some twenty cycles an instruction.
__device__ __forceinline__ void copy16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_addr(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void copy16_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }
__device__ __forceinline__ bool elect_one() {
  uint32_t yes;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(yes));
  return yes != 0;
}
// 32 columns of this thread's lane; defined after tmem_wait_ld().
__device__ __forceinline__ void tmem_ld32(uint32_t ta, float (&v)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]),
        "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]), "=f"(v[16]),
        "=f"(v[17]), "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]), "=f"(v[24]),
        "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
      : "r"(ta)
      : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t ta, const float (&v)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
      "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(ta),
      "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]), "f"(v[8]), "f"(v[9]),
      "f"(v[10]), "f"(v[11]), "f"(v[12]), "f"(v[13]), "f"(v[14]), "f"(v[15]), "f"(v[16]), "f"(v[17]), "f"(v[18]),
      "f"(v[19]), "f"(v[20]), "f"(v[21]), "f"(v[22]), "f"(v[23]), "f"(v[24]), "f"(v[25]), "f"(v[26]), "f"(v[27]),
      "f"(v[28]), "f"(v[29]), "f"(v[30]), "f"(v[31])
      : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t ta, const float (&v)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(ta), "f"(v[0]),
               "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
               : "memory");
}
__device__ __forceinline__ u64 add2(u64 a, u64 b) {
  u64 d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint32_t h2u(__half2 h) { return *reinterpret_cast<uint32_t*>(&h); }
__device__ __forceinline__ __half2 u2h(uint32_t u) { return *reinterpret_cast<__half2*>(&u); }
__device__ __forceinline__ float exp2i(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Exponent that brings 2^e <= big < 2^(e + 1) to [2^13, 2^14); 0 for zero and non-finite rows.
__device__ __forceinline__ int row_exponent(float big) {
  const int ex = static_cast<int>(__float_as_uint(big) >> 23);
  return (big > 0.f && ex < 255) ? ex - 127 - 13 : 0;
}
// Eight codes as fp16: pairs (elements 2i, 2i + 1) with scale constants 16 d and -24 d of each pair.
__device__ __forceinline__ uint32_t pair_of(uint32_t w, int i, __half2 a, __half2 b) {
  const uint32_t s = i == 0 ? w << 6 : i == 1 ? w << 2 : i == 2 ? w >> 2 : w >> 6;
  uint32_t v;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(v) : "r"(s), "r"(0x03C003C0u), "r"(0x3C003C00u));
  return h2u(__hfma2(u2h(v), a, b));
}
__device__ __forceinline__ void unpack8(float (&x)[8], uint4 u) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) kv4_attn_tree_kernel(KvAttnParams p) {
  using Blk = KvBlock<D>;
  using Sm = Smem<D>;
  constexpr int kTok = Sm::kTok;
  extern __shared__ __align__(1024) char sm[];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const bool aborted = launch_aborted(p.c.err);
  const KvPlace place = kv_place(p, kRows, reinterpret_cast<long long*>(sm));
  if (__syncthreads_or(aborted)) return;
  if (place.at == place.end) {
    if (threadIdx.x == 0 && !p.by_item) p.desc[blockIdx.x] = make_int4(0, 0, 0, 0);
    return;
  }

  uint64_t* bar = reinterpret_cast<uint64_t*>(sm + Sm::kBar);
  volatile int* gave_up = reinterpret_cast<volatile int*>(sm + Sm::kTmem + 8);
  volatile int* odd = reinterpret_cast<volatile int*>(sm + Sm::kTmem + 16);      // [2], alternating by new-row step
  unsigned long long* see = reinterpret_cast<unsigned long long*>(sm + Sm::kSee);
  float* colscale = reinterpret_cast<float*>(sm + Sm::kColScale);
  if (tid == 0) {
    auto init = [&](int i, int count) {
      asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_addr(&bar[i])), "r"(count) : "memory");
    };
    for (int i = 0; i < kBars; ++i) init(i, 1);
    for (int i = 0; i < kStages; ++i) init(kStEmpty + i, kUnpackWarps);
    for (int i = 0; i < 2; ++i) {
      init(kKFull + i, kKeyWarps);
      init(kVFull + i, kUnpackWarps - kKeyWarps);
      init(kPFull + i, kSoftWarps / 2);
    }
    init(kOFree, kSoftWarps);
    init(kQReady, kSoftWarps);
    init(kNewFull, kUnpackWarps);
    for (int i = 0; i < 4; ++i) init(kPair + i, 2);
    init(kSoft, kSoftWarps);
    init(kKeyMeet, kKeyWarps);
    init(kValMeet, kUnpackWarps - kKeyWarps);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    *gave_up = 0;
    odd[0] = odd[1] = 0;
  }
  uint32_t* tslot = reinterpret_cast<uint32_t*>(sm + Sm::kTmem);
  if (warp == kMmaWarp) {
    tmem_alloc(tslot, Sm::kCols);
    tmem_relinquish();
  }
  fence_proxy_async();
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();
  const uint32_t tmem = *tslot;

  // Bounded wait; once any wait of the CTA has given up, all of them return at once.
  auto wait = [&](int b, uint32_t parity) {
    if (mbar_ready(&bar[b], parity & 1)) return true;
    const long long t0 = clock64();
    while (!*gave_up && clock64() - t0 <= kWaitCycles)
      if (mbar_ready(&bar[b], parity & 1)) return true;
    if (*gave_up) return false;
    *gave_up = 1;
    device_error(p.c.err, GDN_DEVERR_TIMEOUT, place.b);
    return false;
  };
  auto wait_all = [&](int b, uint32_t parity) { return __all_sync(0xffffffffu, wait(b, parity)) != 0; };   // by a whole warp
  auto arrive_warp = [&](int b) {
    __syncwarp();
    if (lane == 0) mbar_arrive(&bar[b]);
  };

  long long at = place.at;
  KvPlace where = place;
  int step = 0, pages = 0, segs = 0, news = 0;      // steps, pages, segments with steps and new-row steps so far
  int swaps = 0, decisions = 0;                     // exchanges between the two threads of a row, reference maxima so far
  int meets = 0;                                    // meetings of the softmax warps so far
  bool alive = true;
  int done = 0;                                     // pages of the segment in its partial result, from runs before this one
  while (at < place.end && alive) {
    long long next;
    KvSegment it = kv_segment(p, kRows, at, place.end, where, &next);
    const bool folded = done > 0, over = it.pages - done <= kRun;
    it.page_lo += done;
    it.pages = min(it.pages - done, kRun);
    done = over ? 0 : done + kRun;
    if (over) at = next;
    if (!it.r.ok) {
      if (tid == 0 && it.first) {
        device_error(p.c.err, it.r.n < 1 || it.r.n > p.n_max ? GDN_DEVERR_SCHEDULE : GDN_DEVERR_CACHE, it.b);
        if (p.by_item)
          for (int t = 0; t < p.row_tiles; ++t) p.desc[it.item + t] = make_int4(0, 0, 0, 0);
      }
      if (tid == 0 && !p.by_item) p.desc[blockIdx.x] = make_int4(0, 0, 0, 0);
      continue;
    }
    const bool with_new = it.first && over && p.k_new;
    const int psteps = (it.pages + Sm::kPages - 1) / Sm::kPages;
    const int steps = psteps + (with_new ? 1 : 0);        // the new rows last: a page sets better first references
    const int seg_toks = min(it.r.len - it.page_lo * kPage, it.pages * kPage);
    const int row0 = it.tile * kRows, rows = min(kRows, it.r.n * p.G - row0);
    const size_t node0 = static_cast<size_t>(it.bl) * p.n_max;

    if (warp < kSoftWarps) {
      // ================= softmax: two threads a row take steps in turn (half = step & 1), so that the latencies of one
      // step run beside those of the next, and half of the channels each of queries and output
      const int quarter = warp & 3, half = warp >> 2, r = 32 * quarter + lane;     // lane r of tensor memory
      const uint32_t lanes = tmem + (static_cast<uint32_t>(quarter) << 21);
      const bool busy = 32 * quarter < rows;               // a warp without rows only keeps the barriers going
      const int row = row0 + min(r, rows - 1);             // rows past the tile repeat its last one
      const int node = row / p.G, head = it.h * p.G + row % p.G;
      const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(p.q) + (node0 + node) * p.q_row + static_cast<size_t>(head) * D;
      float* swap = reinterpret_cast<float*>(sm + Sm::kSwap);
      // a value to the row's other thread, and its value
      auto exchange = [&](float x, bool* ok) {
        float* to = swap + (swaps & 1) * 2 * kRows;
        to[half * kRows + r] = x;
        arrive_warp(kPair + quarter);
        *ok = wait_all(kPair + quarter, swaps);
        ++swaps;
        return to[(half ^ 1) * kRows + r];
      };
      // the softmax warps' meeting point; what they wrote to shared memory before it is seen by all of them
      auto meet = [&]() {
        arrive_warp(kSoft);
        const bool ok = wait_all(kSoft, meets);
        ++meets;
        return ok;
      };
      // 16-byte chunk i of row x in a staging tile of `chunks` chunks a row, spread over the banks
      char* stage = sm + Sm::kKeys;
      auto staged = [&](int x, int i, int chunks) { return reinterpret_cast<uint4*>(stage) + x * chunks + (i ^ (x & 7)); };
      // the queries' tile lies in the values' operands, so that the keys of the first page are unpacked meanwhile
      auto query = [&](int x, int i) { return reinterpret_cast<uint4*>(sm + Sm::kVals) + x * (D / 8) + (i ^ (x & 7)); };
      float c = 0.f;
      if (steps > 0) {
        // the rows' queries, whole rows at a time, into the operands' space, which is free once the item before is out
        alive = wait_all(kOFree, segs + 1);
        constexpr int kChunks = D / 8;
        const __nv_bfloat16* q0 = static_cast<const __nv_bfloat16*>(p.q) + node0 * p.q_row + static_cast<size_t>(it.h) * p.G * D;
#pragma unroll 1
        for (int i = tid; alive && i < rows * kChunks; i += 32 * kSoftWarps) {
          const int x = row0 + i / kChunks, nd = x / p.G;
          copy16(query(i / kChunks, i % kChunks), q0 + nd * p.q_row + (x - nd * p.G) * D + 8 * (i % kChunks));
        }
        copy16_wait();
        alive = alive && meet();
      }
      if (busy && steps > 0 && alive) {
        // a thread half a row: largest value, then fp16, scaled by a power of two, in tensor memory
        const int x0 = min(r, rows - 1);
        float big = 0.f;
#pragma unroll 2
        for (int i = 0; i < D / 16; ++i) {
          float x[8];
          unpack8(x, *query(x0, half * (D / 16) + i));
#pragma unroll
          for (int e = 0; e < 8; ++e) big = fmaxf(big, fabsf(x[e]));
        }
        big = fmaxf(big, exchange(big, &alive));
        const int e = row_exponent(big);
        const float f0 = exp2i(-(e / 2)), f1 = (p.scale < 0.f ? -1.f : 1.f) * exp2i(-(e - e / 2));
        // the scores' factor; never 0, so that a masked score stays -inf
        c = fmaxf(fabsf(p.scale) * kLog2e * exp2i(e / 2) * exp2i(e - e / 2), 1.2e-38f);
#pragma unroll 1
        for (int i = 0; i < D / 32; ++i) {
          float w[8];
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            float x[8];
            unpack8(x, *query(x0, half * (D / 16) + 2 * i + k));
#pragma unroll
            for (int z = 0; z < 4; ++z)
              w[4 * k + z] = __uint_as_float(h2u(__floats2half2_rn(x[2 * z] * f0 * f1, x[2 * z + 1] * f0 * f1)));
          }
          tmem_st8(lanes + Sm::kQ + half * (D / 4) + 8 * i, w);
        }
        tmem_wait_st();
      }
      if (steps > 0) {
        tmem_fence_before();
        arrive_warp(kQReady);
      }
      float m = -INFINITY, l = 0.f;      // l is relative to m, the row's reference when this thread last looked
      float* ref = reinterpret_cast<float*>(sm + Sm::kRef) + r;
      // the row's reference after decision n, and l in its terms
      auto follow = [&](float mn) {
        if (mn != m) l *= m == -INFINITY ? 0.f : exp2f(m - mn);
        m = mn;
      };
      for (int i = 0; i < steps && alive; ++i) {
        const int k = step + i, buf = k & 1;
        if (buf != half) continue;
        alive = wait_all(kScored + buf, k >> 1);
        if (alive && i == psteps) alive = wait_all(kNewFull, news);
        if (!alive) break;
        tmem_fence_after();
        if (busy) {
          const uint32_t ts = lanes + Sm::kS + kTok * buf;
          const bool is_new = i == psteps;
          const int toks = seg_toks - i * kTok;               // tokens of this step
          if (is_new || toks < kTok) {
            // scale and mask in place, apart from the common path (whose code is better small: the roles of an SM share
            // its instruction caches)
#pragma unroll 1
            for (int x = 0; x < kTok; x += 16) {
              float t[16];
              tmem_ld16(ts + x, t);
              tmem_wait_ld();
              // which of the 16 columns the row sees
              uint32_t vis = toks - x >= 16 ? 0xFFFFu : toks > x ? (1u << (toks - x)) - 1 : 0u;
              if (is_new) vis = odd[news & 1] || x >= GDN_MAX_NODES ? 0u : static_cast<uint32_t>(see[node] >> x);
#pragma unroll
              for (int y = 0; y < 16; ++y) {
                if (is_new) t[y] *= colscale[x + y];
                if (!((vis >> y) & 1)) t[y] = -INFINITY;
              }
              tmem_st16(ts + x, t);
            }
            tmem_wait_st();
          }
          float top = -INFINITY;
#pragma unroll 1
          for (int h = 0; h < kTok; h += 32) {
            float x[32];
            tmem_ld32(ts + h, x);
            tmem_wait_ld();
            float t0 = x[0], t1 = x[1];
#pragma unroll
            for (int y = 2; y < 32; y += 4) {          // (three-input maxima)
              t0 = fmaxf(t0, fmaxf(x[y], x[y + 1]));
              if (y + 3 < 32) t1 = fmaxf(t1, fmaxf(x[y + 2], x[y + 3]));
            }
            top = fmaxf(top, fmaxf(t0, t1));
          }
          // rounded up, so that no score times c passes it; large scores' products are rounded themselves (below)
          top = fabsf(top) * c < kLarge ? __fmul_ru(top, c) : __fmul_rn(top, c);
          // the reference: the other thread's of the page before, raised where this page passes it by too much
          float before = -INFINITY;
          if (i > 0) {
            alive = wait_all(kDecided + quarter, decisions + i - 1);
            if (!alive) break;
            before = *const_cast<volatile float*>(ref);
          }
          const float now = top - before > kSlack ? top : before;       // (the sum would round)
          *ref = now;
          arrive_warp(kDecided + quarter);
          follow(now);
          const bool raised = i > 0 && now != before, large = fabsf(now) >= kLarge && now > -INFINITY;
          float times = c;
          if (__any_sync(0xffffffffu, raised || large)) {          // (one vote for both, which are rare)
            if (__any_sync(0xffffffffu, raised)) {
              // rescale the output: the product of the step before has to be in it first
              const float f = before == -INFINITY ? 0.f : exp2f(before - now);
              alive = wait_all(kAdded + (buf ^ 1), (k - 1) >> 1);
              if (!alive) break;
              tmem_fence_after();
#pragma unroll 1
              for (int x = 0; x < D; x += 32) {
                float o[32];
                tmem_ld32(lanes + Sm::kO + x, o);
                tmem_wait_ld();
#pragma unroll
                for (int y = 0; y < 32; ++y) o[y] *= f;
                tmem_st32(lanes + Sm::kO + x, o);
              }
              tmem_wait_st();
            }
            if (__any_sync(0xffffffffu, large)) {
              // the products' own rounding has to be the reference's: a fused multiply-add would leave it in the exponent
              if (large) times = 1.f;
#pragma unroll 1
              for (int x = 0; x < kTok; x += 16) {
                float t[16];
                tmem_ld16(ts + x, t);
                tmem_wait_ld();
#pragma unroll
                for (int y = 0; y < 16; ++y) t[y] = large ? __fmul_rn(t[y], c) : t[y];
                tmem_st16(ts + x, t);
              }
              tmem_wait_st();
            }
          }
          // (rounded down: where the scores' own steps are larger than kLift, no weight passes fp16's largest number)
          const float base = m == -INFINITY ? kLift : __fsub_rd(kLift, m);
          const u64 c2 = pack2(times, times), b2 = pack2(base, base);
          u64 sum[2] = {0, 0};
#pragma unroll 1
          for (int h = 0; h < kTok; h += 32) {
            float x[32], w[16];
            tmem_ld32(ts + h, x);
            tmem_wait_ld();
#pragma unroll
            for (int y = 0; y < 16; ++y) {
              const float2 e = unpack2(fma2(pack2(x[2 * y], x[2 * y + 1]), c2, b2));
              const float e0 = exp2_fast(e.x), e1 = exp2_fast(e.y);
              sum[y & 1] = add2(sum[y & 1], pack2(e0, e1));
              w[y] = __uint_as_float(h2u(__floats2half2_rn(e0, e1)));
            }
            // the weights of 32 tokens go over the scores they came from: columns h .. h + 15
            tmem_st16(ts + h, w);
          }
          const float2 total = unpack2(add2(sum[0], sum[1]));
          l += total.x + total.y;
          tmem_wait_st();
        }
        tmem_fence_before();
        arrive_warp(kPFull + buf);
      }
      // ---- the item's rows (or this CTA's part of them)
      bool own = false;                                    // the row adds its own ancestors
      if (steps > 0 && alive) {
        // every product of the item (a barrier of its own, once an item: a wait tells a phase from the one before and
        // the one after only)
        alive = wait_all(kItem, segs);
        tmem_fence_after();
        own = with_new && odd[news & 1];
        if (alive && busy) {
          alive = wait_all(kDecided + quarter, decisions + steps - 1);
          follow(*ref);
        }
      }
      if (busy) decisions += steps;
      // (an item that the CTA holds whole has no partial result of its own, and its place is free)
      float* slot = kv_stream_part(p, blockIdx.x, it.start > place.at, kRows, D);
      float* part = it.whole ? nullptr : slot;
      // channels x .. x + 3 of the row in a partial result (laid out as the staging tile)
      auto partial = [&](int x) { return reinterpret_cast<float4*>(slot) + r * (D / 4) + ((x / 4) ^ (r & 7)); };
      if (alive && busy && (folded || !over)) {
        // one of several runs: this one's output and the earlier ones', in the place of the partial result, in terms of
        // their common reference; back to tensor memory from the last run
        float fo = 1.f, fs = 0.f;
        if (folded) {
          const float2 before = *reinterpret_cast<const float2*>(slot + kRows * D + 2 * r);
          const float mn = fmaxf(m, before.x);
          fo = m == -INFINITY ? 0.f : exp2f(m - mn);
          fs = before.x == -INFINITY ? 0.f : exp2f(before.x - mn);
          m = mn;
          l = fmaf(l, fo, half == 0 ? before.y * fs : 0.f);
        }
#pragma unroll 1
        for (int x = half * (D / 2); x < (half + 1) * (D / 2); x += 32) {
          float o[32];
          tmem_ld32(lanes + Sm::kO + x, o);
          tmem_wait_ld();
#pragma unroll
          for (int y = 0; y < 32; y += 4) {
            float4* at = partial(x + y);
            if (folded) {
              const float4 b = *at;
              o[y] = fmaf(o[y], fo, b.x * fs);
              o[y + 1] = fmaf(o[y + 1], fo, b.y * fs);
              o[y + 2] = fmaf(o[y + 2], fo, b.z * fs);
              o[y + 3] = fmaf(o[y + 3], fo, b.w * fs);
            }
            if (!over) *at = make_float4(o[y], o[y + 1], o[y + 2], o[y + 3]);
          }
          if (over) tmem_st32(lanes + Sm::kO + x, o);
        }
        if (over) {
          tmem_wait_st();
        } else {
          l += exchange(l, &alive);                        // (both threads of the row have read the earlier sums before)
          if (half == 0) *reinterpret_cast<float2*>(slot + kRows * D + 2 * r) = make_float2(m, l);
        }
      }
      if (alive && busy && over) {
        const bool mine = r < rows;
        float f = 1.f;
        // the row's ancestors' weights, in the operands' space (every product has completed)
        float* ps = reinterpret_cast<float*>(sm + Sm::kKeys) + r * GDN_MAX_NODES;
        const unsigned long long anc = own ? see[node] : 0ull;
        if (own) {
          if (half == 0) {
            const float sc = p.scale * kLog2e;
            float mn = m;
            for (unsigned long long left = anc; left; left &= left - 1) {
              const int t = __ffsll(static_cast<long long>(left)) - 1;
              const __nv_bfloat16* kr = static_cast<const __nv_bfloat16*>(p.k_new) + (node0 + t) * p.kv_row + static_cast<size_t>(it.h) * D;
              float x = 0.f;
#pragma unroll 1
              for (int i = 0; i < D / 8; ++i) {
                float a[8], b[8];
                unpack8(a, __ldg(reinterpret_cast<const uint4*>(q) + i));
                unpack8(b, __ldg(reinterpret_cast<const uint4*>(kr) + i));
#pragma unroll
                for (int e = 0; e < 8; ++e) x = fmaf(a[e], b[e], x);
              }
              x *= sc;
              ps[t] = x;
              mn = fmaxf(mn, x);
            }
            f = m == -INFINITY ? 0.f : exp2f(m - mn);
            m = mn;
            l *= f;
            for (unsigned long long left = anc; left; left &= left - 1) {
              const int t = __ffsll(static_cast<long long>(left)) - 1;
              const float w = ps[t] == -INFINITY ? 0.f : exp2f(ps[t] - m + kLift);
              ps[t] = w;
              l += w;
            }
          }
          const float g = exchange(f, &alive);      // and the weights with it
          if (half == 1) {
            f = g;
            l *= f;
          }
        }
        l += exchange(l, &alive);
        const float inv = !it.whole ? 1.f : (l == 0.f ? 0.f : 1.f / l);
        __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.out) + (node0 + node) * (static_cast<size_t>(p.Hq) * D) + static_cast<size_t>(head) * D;
        if (!own && steps > 0) {
#pragma unroll 1
          for (int x = half * (D / 2); x < (half + 1) * (D / 2); x += 32) {
            float o[32];
            tmem_ld32(lanes + Sm::kO + x, o);
            tmem_wait_ld();
            if (part) {
#pragma unroll
              for (int y = 0; y < 8; ++y)
                *reinterpret_cast<float4*>(staged(r, x / 4 + y, D / 4)) = make_float4(o[4 * y], o[4 * y + 1], o[4 * y + 2], o[4 * y + 3]);
            } else {
#pragma unroll
              for (int y = 0; y < 4; ++y) {
                __nv_bfloat162 b[4];
#pragma unroll
                for (int z = 0; z < 4; ++z) b[z] = __floats2bfloat162_rn(o[8 * y + 2 * z] * inv, o[8 * y + 2 * z + 1] * inv);
                *staged(r, x / 8 + y, D / 8) = *reinterpret_cast<uint4*>(b);
              }
            }
          }
        } else {                       // rare: straight to global memory (the loads of tensor memory take the whole warp)
#pragma unroll 1
          for (int x = half * (D / 2); x < (half + 1) * (D / 2); x += 4) {
            float o[4] = {0.f, 0.f, 0.f, 0.f};
            __syncwarp();
            if (own) {
              tmem_ld4(lanes + Sm::kO + x, o);
              tmem_wait_ld();
#pragma unroll
              for (int y = 0; y < 4; ++y) o[y] = f == 0.f ? 0.f : o[y] * f;
              for (unsigned long long left = mine ? anc : 0ull; left; left &= left - 1) {
                const int t = __ffsll(static_cast<long long>(left)) - 1;
                if (ps[t] == 0.f) continue;
                const __nv_bfloat16* vr = static_cast<const __nv_bfloat16*>(p.v_new) + (node0 + t) * p.kv_row + static_cast<size_t>(it.h) * D + x;
#pragma unroll
                for (int y = 0; y < 4; ++y) o[y] = fmaf(ps[t], __bfloat162float(vr[y]), o[y]);
              }
            }
            if (mine && part) {
              *partial(x) = make_float4(o[0], o[1], o[2], o[3]);
            } else if (mine) {
              *reinterpret_cast<__nv_bfloat162*>(out + x) = __floats2bfloat162_rn(o[0] * inv, o[1] * inv);
              *reinterpret_cast<__nv_bfloat162*>(out + x + 2) = __floats2bfloat162_rn(o[2] * inv, o[3] * inv);
            }
            __syncwarp();
          }
        }
        if (part && mine && half == 0) *reinterpret_cast<float2*>(part + kRows * D + 2 * r) = make_float2(m, l);
      }
      if (steps > 0 && alive && over && !own) {
        // from the staging tile to global memory, whole rows at a time
        if (part) fence_proxy_async();
        alive = meet();
        if (alive && part && tid == 0) {
          asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(part), "r"(smem_addr(stage)),
                       "r"(static_cast<uint32_t>(rows * D * 4))
                       : "memory");
          asm volatile("cp.async.bulk.commit_group;" ::: "memory");
          asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
        }
        if (alive && !part) {
          constexpr int kChunks = D / 8;
          __nv_bfloat16* o0 = static_cast<__nv_bfloat16*>(p.out) + (node0 * p.Hq + it.h * p.G) * D;
#pragma unroll 4
          for (int i = tid; i < rows * kChunks; i += 32 * kSoftWarps) {
            const int x = row0 + i / kChunks;
            *(reinterpret_cast<uint4*>(o0 + static_cast<size_t>(x / p.G) * p.Hq * D + (x % p.G) * D) + i % kChunks) =
                *staged(i / kChunks, i % kChunks, kChunks);
          }
        }
      }
      if (tid == 0 && (it.first || !p.by_item)) {
        const int c0 = kv_cta_of(it.start, place.total, place.ctas);
        const int c1 = kv_cta_of(it.start + it.r.units - 1, place.total, place.ctas);
        // what the join reads: item, CTAs (none to join: 0), the first one and whether the item starts inside it, rows.
        // A CTA's last item is the only one that can both start in it and pass its end
        const int inside = it.start > kv_unit_of(c0, place.total, place.ctas);
        p.desc[p.by_item ? it.item : blockIdx.x] = make_int4(it.item, it.whole || !it.first ? 0 : c1 - c0 + 1, 2 * c0 + inside, rows);
        if (p.by_item && it.tile == 0)          // tiles that this request does not fill
          for (int t = it.r.tiles; t < p.row_tiles; ++t) p.desc[it.item + t] = make_int4(0, 0, 0, 0);
      }
      if (steps > 0) {
        tmem_fence_before();
        arrive_warp(kOFree);
      }
    } else if (warp < kCopyWarp) {
      // ================= unpacking: four warps the keys, four the values
      // (warps of one kind on two of the four schedulers: warp % 4 is a warp's scheduler, with instruction caches of its own)
      const bool keys = (warp & 2) == 0;
      const int uw = (warp & 1) + 2 * ((warp - kSoftWarps) >> 2);
      // 32 x 16-byte units of a page's keys, and of its values; a warp takes units uw, uw + 4, ...
      constexpr int kUnits = Sm::kPages * D / 16, kShare = kUnits / kKeyWarps, kValWarps = kUnpackWarps - kKeyWarps;
      static_assert(kKeyWarps == 4 && kUnpackWarps == 8, "units are dealt to four warps");
      constexpr bool kTwo = Sm::kPages == 2;
      const __half2 k16 = __float2half2_rn(16.f), k24 = __float2half2_rn(-24.f);
      // keys: one page: unit uw + 4 y is chunk uw / 2 + 2 y of token 32 (uw & 1) + lane; two pages: a warp takes all
      // chunks of tokens 32 uw + lane
      constexpr int kChunkStep = kTwo ? 1 : 2;
      const int kt_tok = 32 * (uw & 1) + lane, kt_turn = Blk::turn(kt_tok), kt_at = kTwo ? 32 * uw + lane : kt_tok;
      const int kt_ch = kTwo ? 0 : uw >> 1;
      // values: one page: unit uw + 4 y holds units (of 16 bytes) 32 uw + lane + 128 y; two pages: two warps a page,
      // 64 units apart.  The first one's octet and channel quad
      constexpr int kUnitStep = kTwo ? 64 : 128, kPerHalf = D / kUnitStep;      // steps a half (32 tokens) of a page
      const int vt_page = kTwo ? uw >> 1 : 0, vt_unit = 32 * (kTwo ? uw & 1 : uw) + lane;
      const int vt_oct = (vt_unit / D) * 4 + (vt_unit & 3), vt_quad = (vt_unit % D) >> 2;
      const int block = kTwo ? (uw >> 1) * Sm::kBlock : 0;                     // the warp's page in a stage
      // the operands' space, the ancestor masks and the scales belong to the item before until its output is released
      // (the values' also to this one's queries, on their way to tensor memory)
      if (steps > 0) alive = wait_all(kOFree, segs + 1);
      if (!keys && steps > 0 && alive) {
        if (with_new) {          // the nodes' own values, on their way while the pages go by
          const __nv_bfloat16* from = static_cast<const __nv_bfloat16*>(p.v_new) + node0 * p.kv_row + static_cast<size_t>(it.h) * D;
#pragma unroll 1
          for (int x = 32 * uw + lane; x < it.r.n * (D / 8); x += 32 * kValWarps) {
            const int t = x / (D / 8), ch = x % (D / 8);
            copy16(sm + Sm::kRawVal + t * (2 * D) + 16 * (ch ^ (t & 7)), from + t * p.kv_row + 8 * ch);
          }
        }
        alive = wait_all(kQReady, segs);
      }
      for (int i = 0; i < steps && alive; ++i) {
        const int k = step + i, buf = k & 1;
        char* kt = sm + Sm::kKeys + buf * Sm::kKeyTile;
        char* vt = sm + Sm::kVals + buf * Sm::kValTile;
        const int free_bar = keys ? kScored + buf : kAdded + buf, full_bar = keys ? kKFull + buf : kVFull + buf;
        if (i == psteps) {
          // the nodes' own rows, straight from global memory; the keys pass through the space of the other operand
          // buffer, so the step before has to be done with it
          alive = wait_all(free_bar, (k >> 1) + 1);
          if (keys && alive && k > 0) alive = wait_all(kScored + (buf ^ 1), (k - 1) >> 1);
          if (!alive) break;
          if (keys && uw == 0 && lane == 0) odd[(news + 1) & 1] = 0;      // the next one's, which nobody uses now
          bool strange = false;
          if (keys) {
            const int32_t* parent = p.words ? kv_parents(p, it.b) : nullptr;
            const int ut = 32 * uw + lane;
            if (ut < it.r.n) {
              unsigned long long mask;
              if (!kv_root_path(parent, ut, &mask)) device_error(p.c.err, GDN_DEVERR_SCHEDULE, it.b);
              see[ut] = mask;
            }
          }
          char* raw = keys ? sm + Sm::kKeys + (buf ^ 1) * Sm::kKeyTile : sm + Sm::kRawVal;
          if (keys) {
            const __nv_bfloat16* from = static_cast<const __nv_bfloat16*>(p.k_new) + node0 * p.kv_row + static_cast<size_t>(it.h) * D;
#pragma unroll 1
            for (int x = 32 * uw + lane; x < it.r.n * (D / 8); x += 32 * kKeyWarps) {
              const int t = x / (D / 8), ch = x % (D / 8);
              copy16(raw + t * (2 * D) + 16 * (ch ^ (t & 7)), from + t * p.kv_row + 8 * ch);
            }
          }
          copy16_wait();
          arrive_warp(keys ? kKeyMeet : kValMeet);
          alive = keys ? wait_all(kKeyMeet, 2 * news) : wait_all(kValMeet, news);
          if (!alive) break;
          if (keys) {
            // two to eight threads a row: its largest value, then fp16, scaled by a power of two.  Rows past the nodes
            // stay as they are: their scores are masked
            const int parts = it.r.n > 32 ? 2 : it.r.n > 16 ? 4 : 8, share = (D / 8) / parts;
            const int ut = 32 * uw + lane, t = ut / parts, ch0 = (ut % parts) * share;
            const bool in = t < it.r.n;
            float big = 0.f, sum = 0.f;
#pragma unroll 2
            for (int ch = ch0; in && ch < ch0 + share; ++ch) {
              float x[8];
              unpack8(x, *reinterpret_cast<const uint4*>(raw + t * (2 * D) + 16 * (ch ^ (t & 7))));
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                big = fmaxf(big, fabsf(x[e]));
                sum = fmaf(0.f, x[e], sum);
              }
            }
            strange = sum != 0.f;                    // a NaN or infinity times 0 is NaN
            for (int o = 1; o < parts; o <<= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, o));
            const int e = row_exponent(big);
            const float f0 = exp2i(-(e / 2)), f1 = exp2i(-(e - e / 2));
            if (in && ch0 == 0) colscale[t] = exp2i(e / 2) * exp2i(e - e / 2);
#pragma unroll 2
            for (int ch = ch0; in && ch < ch0 + share; ++ch) {
              float x[8];
              uint32_t w[4];
              unpack8(x, *reinterpret_cast<const uint4*>(raw + t * (2 * D) + 16 * (ch ^ (t & 7))));
#pragma unroll
              for (int z = 0; z < 4; ++z) w[z] = h2u(__floats2half2_rn(x[2 * z] * f0 * f1, x[2 * z + 1] * f0 * f1));
              *reinterpret_cast<uint4*>(kt + ch * Sm::kKeyK + (t >> 3) * 128 + (t & 7) * 16) = make_uint4(w[0], w[1], w[2], w[3]);
            }
          } else {
            // eight tokens of a channel a thread
#pragma unroll 1
            for (int x = 32 * uw + lane; x < (kTok / 8) * D; x += 32 * kValWarps) {
              const int ch = x % D, o = x / D;
              uint32_t w[4] = {0, 0, 0, 0};
              if (8 * o < it.r.n) {
                float y[8], sum = 0.f, big = 0.f;
                bool cut = false;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                  const int t = 8 * o + e;
                  const char* at = raw + t * (2 * D) + 16 * ((ch >> 3) ^ e) + 2 * (ch & 7);
                  y[e] = t < it.r.n ? __bfloat162float(*reinterpret_cast<const __nv_bfloat16*>(at)) : 0.f;
                  sum = fmaf(0.f, y[e], sum);
                  big = fmaxf(big, fabsf(y[e]));
                  cut = cut || __half2float(__float2half_rn(y[e])) != y[e];
                }
                const bool bad = sum != 0.f || big > kTooLarge || (cut && big < kTooSmall);
                strange = strange || bad;
#pragma unroll
                for (int z = 0; z < 4; ++z) w[z] = bad ? 0u : h2u(__floats2half2_rn(y[2 * z], y[2 * z + 1]));
              }
              *reinterpret_cast<uint4*>(vt + o * Sm::kValK + (ch >> 3) * 128 + (ch & 7) * 16) = make_uint4(w[0], w[1], w[2], w[3]);
            }
          }
          if (strange) odd[news & 1] = 1;
          fence_proxy_async();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&bar[full_bar]);
            mbar_arrive(&bar[kNewFull]);
            if (keys) mbar_arrive(&bar[kKeyMeet]);
          }
          // the raw keys' space is the next step's operand: every warp has to be done with them (the raw values' next
          // user waits for this item's output)
          if (keys) alive = wait_all(kKeyMeet, 2 * news + 1);
          continue;
        }
        const int pg = pages + i, st = pg % kStages;
        alive = wait_all(kStFull + st, pg / kStages);
        if (!alive) break;
        const char* blk = sm + st * Sm::kStage + block;
        const int toks = seg_toks - i * kTok;                     // tokens past them read as zeros
        // rolled loops: the roles of an SM share its instruction caches, and unrolled they do not fit
        if (keys) {                    // a unit: a chunk of 32 channels of a token a lane
          const char* from = blk + kt_tok * (D / 2);
          const __half* scale = reinterpret_cast<const __half*>(blk + Blk::kKeyScales) + kt_tok * Blk::kGroups + kt_ch;
          char* dst = kt + 4 * kt_ch * Sm::kKeyK + (kt_at >> 3) * 128 + (kt_at & 7) * 16;
          int ch = kt_ch;
          uint4 cw = *reinterpret_cast<const uint4*>(from + ((ch ^ kt_turn) << 4));
          __half d = *scale;
          alive = wait_all(free_bar, (k >> 1) + 1);
          if (!alive) break;
#pragma unroll 1
          for (int y = 0; y < kShare; ++y) {
            if (kt_at >= toks) d = __ushort_as_half(0);            // scales past the length are whatever the page held
            const __half2 d2 = __half2half2(d), a = __hmul2(d2, k16), b = __hmul2(d2, k24);
            const uint32_t w[4] = {cw.x, cw.y, cw.z, cw.w};
            ch += kChunkStep;
            scale += kChunkStep;
            if (y + 1 < kShare) {
              cw = *reinterpret_cast<const uint4*>(from + ((ch ^ kt_turn) << 4));
              d = *scale;
            }
#pragma unroll
            for (int z = 0; z < 4; ++z)
              *reinterpret_cast<uint4*>(dst + z * Sm::kKeyK) =
                  make_uint4(pair_of(w[z], 0, a, b), pair_of(w[z], 1, a, b), pair_of(w[z], 2, a, b), pair_of(w[z], 3, a, b));
            dst += 4 * kChunkStep * Sm::kKeyK;
          }
        } else {                       // a unit: four channels, eight tokens a lane
          const char* from = blk + Blk::kValCodes + 16 * vt_unit;
          const char* scale = blk + Blk::kValScales + (vt_quad >> 3) * (2 * kPage) + 16 * vt_oct;
          char* dst = vt + (8 * vt_page + vt_oct) * Sm::kValK + (vt_quad >> 1) * 128 + (vt_quad & 1) * 64;
          int left = toks - kPage * vt_page - 8 * vt_oct;                             // tokens of the octet inside the length
          uint4 cw = *reinterpret_cast<const uint4*>(from), sd = *reinterpret_cast<const uint4*>(scale);
          alive = wait_all(free_bar, (k >> 1) + 1);
          if (!alive) break;
#pragma unroll 1
          for (int y = 0; y < kShare; ++y) {
            const uint32_t w[4] = {cw.x, cw.y, cw.z, cw.w};
            uint32_t dd[4] = {sd.x, sd.y, sd.z, sd.w};
            if (left < 8) {
#pragma unroll
              for (int z = 0; z < 4; ++z)
                if (left - 2 * z < 2) dd[z] = left - 2 * z == 1 ? dd[z] & 0xFFFFu : 0u;
            }
            __half2 a[4], b[4];
#pragma unroll
            for (int z = 0; z < 4; ++z) {
              a[z] = __hmul2(u2h(dd[z]), k16);
              b[z] = __hmul2(u2h(dd[z]), k24);
            }
            char* to = dst;
            // the next unit: as many channels further (where a half page takes two steps, the odd ones), or the next
            // 32 tokens
            constexpr int kScaleStep = (kUnitStep / 32) * (2 * kPage), kChanStep = (kUnitStep / 8) * 128;
            from += kUnitStep * 16;
            if (kPerHalf == 2 && (y & 1) == 0) {
              scale += kScaleStep;
              dst += kChanStep;
            } else {
              scale += 64 - (kPerHalf == 2 ? kScaleStep : 0);
              dst += 4 * Sm::kValK - (kPerHalf == 2 ? kChanStep : 0);
              left -= 32;
            }
            if (y + 1 < kShare) {
              cw = *reinterpret_cast<const uint4*>(from);
              sd = *reinterpret_cast<const uint4*>(scale);
            }
#pragma unroll
            for (int z = 0; z < 4; ++z)
              *reinterpret_cast<uint4*>(to + 16 * z) = make_uint4(pair_of(w[z], 0, a[0], b[0]), pair_of(w[z], 1, a[1], b[1]),
                                                                  pair_of(w[z], 2, a[2], b[2]), pair_of(w[z], 3, a[3], b[3]));
          }
        }
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&bar[full_bar]);
          mbar_arrive(&bar[kStEmpty + st]);
        }
      }
    } else if (warp == kCopyWarp) {
      // ================= bulk copies of the pages; a lane holds the numbers of 32 of them at a time
      const int32_t* table = p.c.page_table + static_cast<size_t>(it.b) * p.c.pages_max + it.page_lo;
      for (int base = 0; base < it.pages && alive; base += 32) {
        const int mine = base + lane < it.pages ? table[base + lane] : -1;
        for (int i = base; i < min(it.pages, base + 32) && alive; i += Sm::kPages) {
          const int pg = pages + i / Sm::kPages, st = pg % kStages;
          int g[Sm::kPages];
#pragma unroll
          for (int x = 0; x < Sm::kPages; ++x) g[x] = __shfl_sync(0xffffffffu, mine, (i - base + x) & 31);
          if (lane == 0) {
            alive = wait(kStEmpty + st, pg / kStages + 1);
            if (alive) {
              int good = 0;
#pragma unroll
              for (int x = 0; x < Sm::kPages; ++x) {
                // whatever the stage holds is unpacked in a bad page's place; the request is reported.  A page past the
                // segment's last reads as zeros
                const bool in = i + x < it.pages, ok = in && g[x] >= 0 && g[x] < p.c.n_pages;
                if (in && !ok) device_error(p.c.err, GDN_DEVERR_CACHE, it.b);
                if (!ok) g[x] = -1;
                good += ok;
              }
              if (good)
                mbar_expect(&bar[kStFull + st], good * Sm::kBlock);
              else
                mbar_arrive(&bar[kStFull + st]);
#pragma unroll
              for (int x = 0; x < Sm::kPages; ++x)
                if (g[x] >= 0)
                  bulk_g2s(sm + st * Sm::kStage + x * Sm::kBlock, kv_block<D>(p.c, p.Hkv, g[x], it.l, it.h), Sm::kBlock,
                           &bar[kStFull + st]);
            }
          }
          alive = __shfl_sync(0xffffffffu, alive, 0);
        }
      }
      if (!alive && lane == 0)          // let the copies in flight land before the CTA exits
        for (int st = 0; st < kStages; ++st)
          for (int par = 0; par < 2; ++par) mbar_wait(&bar[kStFull + st], par);
    } else if (steps > 0) {
      // ================= MMAs: scores of step i, then the product of step i - 1.  The warp runs the loop together
      // and one elected thread issues: operand descriptors stay in uniform registers that way, and an issue takes a
      // few instructions (in a lane-0 branch the 20 issues of a step took three times as long as the MMAs themselves)
      const bool leader = elect_one();
      alive = wait_all(kQReady, segs);
      tmem_fence_after();
      for (int i = 0; i <= steps && alive; ++i) {
        if (i < steps) {
          const int k = step + i, buf = k & 1;
          alive = wait_all(kKFull + buf, k >> 1);
          if (!alive) break;
          tmem_fence_after();
          const uint64_t b0 = umma_desc(smem_addr(sm + Sm::kKeys + buf * Sm::kKeyTile), Sm::kKeyK, 128);
          const uint32_t d = tmem + Sm::kS + kTok * buf;
          if (leader) {
            umma_f16_ts<false>(d, tmem + Sm::kQ, b0, idesc_f16(128, kTok));
#pragma unroll
            for (int x = 1; x < D / 16; ++x)
              umma_f16_ts<true>(d, tmem + Sm::kQ + 8 * x, b0 + static_cast<uint64_t>(x) * (2 * Sm::kKeyK / 16),
                                idesc_f16(128, kTok));
            umma_commit(&bar[kScored + buf]);
          }
          __syncwarp();
        }
        if (i > 0) {
          const int k = step + i - 1, buf = k & 1;
          // the first product of an item overwrites the output of the one before it
          alive = (i > 1 || wait_all(kOFree, segs + 1)) && wait_all(kPFull + buf, k >> 1) && wait_all(kVFull + buf, k >> 1);
          if (!alive) break;
          tmem_fence_after();
          const uint64_t b0 = umma_desc(smem_addr(sm + Sm::kVals + buf * Sm::kValTile), Sm::kValK, 128);
          const uint32_t a0 = tmem + Sm::kS + kTok * buf;    // weights of 16 tokens in columns 0, 8, 32, 40, ...
          if (leader) {
            if (i == 1)
              umma_f16_ts<false>(tmem + Sm::kO, a0, b0, idesc_f16(128, D));
            else
              umma_f16_ts<true>(tmem + Sm::kO, a0, b0, idesc_f16(128, D));
#pragma unroll
            for (int x = 1; x < kTok / 16; ++x)
              umma_f16_ts<true>(tmem + Sm::kO, a0 + 16 * x - 8 * (x & 1), b0 + static_cast<uint64_t>(x) * (2 * Sm::kValK / 16),
                                idesc_f16(128, D));
            umma_commit(&bar[kAdded + buf]);
            if (i == steps) umma_commit(&bar[kItem]);
          }
          __syncwarp();
        }
      }
      if (!alive) {                     // MMAs in flight read shared and tensor memory: wait for them
        if (leader) {
          umma_commit(&bar[kDrain]);
          mbar_wait(&bar[kDrain], 0);
        }
        __syncwarp();
      }
    }
    step += steps;
    pages += psteps;
    segs += steps > 0 ? 1 : 0;
    news += with_new ? 1 : 0;
    alive = __shfl_sync(0xffffffffu, alive, 0);
  }
  copy16_wait();
  if (tid == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
  tmem_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) tmem_dealloc(tmem, Sm::kCols);
}

// Joins the items that several CTAs share: a thread four channels of a row, kPass rows one after another with all their
// loads in flight together.  Two forms, since blocks cost time where there are many and loads where there are few:
// records by CTA (its last item, if that goes on in the next; four rows a thread, so that 152 CTAs' 128-row items are
// 2,432 blocks) where items are many, and records by item (one row a thread) where a few items have many parts.  With
// one row a thread and a block row for all 128 rows everywhere, the join of 32 requests' 22-node trees took 16 us.
constexpr int kJoinThreads = 128;
template <int D, int kPass>
__global__ void __launch_bounds__(kJoinThreads) kv4_join_kernel(KvAttnParams p) {
  constexpr int kQuads = D / 4, kPer = kJoinThreads / kQuads, kAhead = kPass == 1 ? 8 : 2;
  asm volatile("griddepcontrol.wait;" ::: "memory");      // launched ahead: everything below reads the first kernel's results
  if (launch_aborted(p.c.err)) return;  // the records may be an earlier call's
  const int lane = threadIdx.x & 31, r0 = blockIdx.y * (kPer * kPass) + threadIdx.x / kQuads, i = threadIdx.x % kQuads;
  const int4 t = p.desc[blockIdx.x];
  const int count = t.y, rows = t.w;
  if (count < 2 || static_cast<int>(blockIdx.y) * (kPer * kPass) >= rows) return;
  constexpr size_t kSize = static_cast<size_t>(kRows) * (D + 2);
  const float* parts = p.part + 2 * static_cast<size_t>(t.z >> 1) * kSize;
  auto part_of = [&](int c) { return parts + (2 * static_cast<size_t>(c) + (c == 0 ? t.z & 1 : 0)) * kSize; };
  // maxima and sums of 32 parts a time, a lane a part (the lanes of a warp share a row, or, for D = 64, two rows: a
  // half-warp then takes 16 parts a time)
  constexpr int kLanes = kQuads < 32 ? kQuads : 32;
  const int sub = lane % kLanes;
  float m[kPass], sum[kPass];
  float2 ml[kPass];
  float4 acc[kPass];
  auto load = [&](int b) {
#pragma unroll
    for (int k = 0; k < kPass; ++k) {
      const int r = r0 + k * kPer;
      ml[k] = make_float2(-INFINITY, 0.f);
      if (r < rows && b + sub < count) ml[k] = *reinterpret_cast<const float2*>(part_of(b + sub) + kRows * D + 2 * r);
    }
  };
#pragma unroll
  for (int k = 0; k < kPass; ++k) {
    m[k] = -INFINITY;
    sum[k] = 0.f;
    acc[k] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  for (int b = 0; b < count; b += kLanes) {
    load(b);
#pragma unroll
    for (int k = 0; k < kPass; ++k) {
      float top = fmaxf(m[k], ml[k].x);
      for (int o = kLanes / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      m[k] = top;
    }
  }
  for (int b = 0; b < count; b += kLanes) {
    if (count > kLanes) load(b);
    float wt[kPass], wl[kPass];
#pragma unroll
    for (int k = 0; k < kPass; ++k) {
      // a part that held nothing this row sees has maximum -inf, sum 0 and zeros
      wt[k] = (ml[k].x == -INFINITY && ml[k].y == 0.f) ? 0.f : exp2f(ml[k].x - m[k]);
      wl[k] = wt[k] * ml[k].y;
    }
    for (int c0 = b; c0 < min(count, b + kLanes); c0 += kAhead) {
      float4 v[kPass][kAhead];
#pragma unroll
      for (int k = 0; k < kPass; ++k)
#pragma unroll
        for (int a = 0; a < kAhead; ++a) {
          const int r = r0 + k * kPer;
          if (r < rows && c0 + a < count)
            v[k][a] = *(reinterpret_cast<const float4*>(part_of(c0 + a)) + static_cast<size_t>(r) * kQuads + (i ^ (r & 7)));
        }
#pragma unroll
      for (int k = 0; k < kPass; ++k)
#pragma unroll
        for (int a = 0; a < kAhead; ++a) {
          const float w = __shfl_sync(0xffffffffu, wt[k], c0 + a - b, kLanes);
          const float s = __shfl_sync(0xffffffffu, wl[k], c0 + a - b, kLanes);
          if (r0 + k * kPer < rows && c0 + a < count) {
            sum[k] += s;
            acc[k].x = fmaf(w, v[k][a].x, acc[k].x);
            acc[k].y = fmaf(w, v[k][a].y, acc[k].y);
            acc[k].z = fmaf(w, v[k][a].z, acc[k].z);
            acc[k].w = fmaf(w, v[k][a].w, acc[k].w);
          }
        }
    }
  }
  const int tile = t.x % p.row_tiles, lh = t.x / p.row_tiles, h = lh % p.Hkv, bl = p.b0 * p.layers + lh / p.Hkv;
#pragma unroll
  for (int k = 0; k < kPass; ++k) {
    const int r = r0 + k * kPer;
    if (r >= rows) continue;
    const int row = tile * kRows + r, node = row / p.G;
    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.out) +
                         ((static_cast<size_t>(bl) * p.n_max + node) * p.Hq + h * p.G + row - node * p.G) * D + 4 * i;
    const float inv = sum[k] == 0.f ? 0.f : 1.f / sum[k];
    __nv_bfloat162 o[2] = {__floats2bfloat162_rn(acc[k].x * inv, acc[k].y * inv),
                           __floats2bfloat162_rn(acc[k].z * inv, acc[k].w * inv)};
    *reinterpret_cast<uint2*>(out) = *reinterpret_cast<const uint2*>(o);
  }
}

template <int D>
cudaError_t tree_t(KvAttnParams p, cudaStream_t s) {
  auto k = kv4_attn_tree_kernel<D>;
  cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, Smem<D>::kTotal);
  if (e != cudaSuccess) return e;
  const int items = p.layers * p.Hkv * p.row_tiles, per = kKvItems / items;      // requests a launch
  p.each = p.ctas / items;
  for (p.b0 = 0; p.b0 < p.c.B; p.b0 += per) {
    p.bn = p.c.B - p.b0 < per ? p.c.B - p.b0 : per;
    p.by_item = p.bn * items <= p.ctas / 4;
    k<<<p.ctas, kThreads, Smem<D>::kTotal, s>>>(p);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    const int at_once = (p.by_item ? 1 : 4) * kJoinThreads / (D / 4);                 // rows a block
    const int most = p.n_max * p.G < kRows ? p.n_max * p.G : kRows;
    cfg.gridDim = dim3(static_cast<unsigned>(p.by_item ? p.bn * items : p.ctas),
                       static_cast<unsigned>((most + at_once - 1) / at_once));
    cfg.blockDim = dim3(kJoinThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = p.by_item ? cudaLaunchKernelEx(&cfg, kv4_join_kernel<D, 1>, p) : cudaLaunchKernelEx(&cfg, kv4_join_kernel<D, 4>, p);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace

cudaError_t launch_kv4_attention_tree(const KvAttnParams& p, cudaStream_t s) {
  return p.D == 256 ? tree_t<256>(p, s) : p.D == 128 ? tree_t<128>(p, s) : tree_t<64>(p, s);
}

}  // namespace gdn
