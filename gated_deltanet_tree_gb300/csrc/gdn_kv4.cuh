// The paged 4-bit key/value cache as the kernels address it: block layout, the
// checks of lengths and page numbers, and parameters shared by the append, read
// and attention kernels.  The format is documented in gdn_tree.h.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "gdn_internal.h"

namespace gdn {

constexpr int kPage = GDN_KV4_PAGE;
constexpr int kGroup = 32;              // channels that share a scale
constexpr float kScaleMax = 2720.f;     // 24 d stays below fp16's largest value

// Offsets (bytes) inside one (page, kv head) block.
template <int D>
struct KvBlock {
  static constexpr int kGroups = D / kGroup;
  static constexpr int kKeyCodes = 0;
  static constexpr int kKeyScales = 32 * D;
  static constexpr int kValCodes = 36 * D;
  static constexpr int kValScales = 68 * D;
  static constexpr int kBytes = 72 * D;
  // place of 16-byte key chunk j of token r among the token's chunks
  static __host__ __device__ constexpr int turn(int r) {
    return D == 256 ? (((r & 1) << 2) | ((r >> 1) & 3)) : D == 128 ? ((r >> 1) & 3) : ((r >> 2) & 1);
  }
  // 32-bit word of channels 8w .. 8w + 7 of token r's key, from the block's start
  static __host__ __device__ constexpr int key_word(int r, int w) {
    return r * (D / 8) + (((w >> 2) ^ turn(r)) << 2) + (w & 3);
  }
  // 32-bit word of tokens 8o .. 8o + 7 of value channel c, from the start of the value codes
  static __host__ __device__ constexpr int val_word(int c, int o) {
    return (((o >> 2) * (D / 4) + (c >> 2)) * 4 + (o & 3)) * 4 + (c & 3);
  }
};
// Nibble of element e of a word.
__host__ __device__ constexpr int nibble_of(int e) { return (e >> 1) + 4 * (e & 1); }

struct KvCacheView {
  char* pool;
  const int32_t* page_table;
  int32_t* seq_len;
  int32_t* ticket;
  int32_t* err;
  int B, layers, pages_max;
  long long n_pages;
};

struct KvAppendParams {
  KvCacheView c;
  int Hkv, D, dtype, n_rows;
  long long kv_row;
  const void* k_new;
  const void* v_new;
  const int32_t* path;
  const int32_t* count;
};
struct KvReadParams {
  KvCacheView c;
  int Hkv, D, out_dtype, n_rows;
  const int32_t* start;
  void* k_out;
  void* v_out;
};
cudaError_t launch_kv4_append(const KvAppendParams& p, cudaStream_t s);
cudaError_t launch_kv4_read(const KvReadParams& p, cudaStream_t s);

#ifdef __CUDACC__
// Block of page `page` (already checked), layer l, kv head h.
template <int D>
__device__ __forceinline__ char* kv_block(const KvCacheView& c, int Hkv, long long page, int l, int h) {
  return c.pool + ((static_cast<long long>(l) * c.n_pages + page) * Hkv + h) * KvBlock<D>::kBytes;
}
#endif

// The attention call, whichever kernel takes it.  The rows of a (request, layer, kv head) are its (node, query head of
// the group) pairs, row = node * G + g, taken in tiles.
struct KvAttnParams {
  KvCacheView c;
  int layers, n_max, Hq, Hkv, D, dtype, G;
  float scale;
  long long q_row, kv_row;
  const int32_t* words;        // packed schedules; nullptr: one node per request
  const void* q;
  const void* k_new;           // nullptr: the cache alone
  const void* v_new;
  void* out;
  int b0, bn;                  // requests of this launch (the kernels that take units)
  int ctas, least;             // CTAs launched, and the units one takes at least where there are few
  int each;                    // CTAs an item of a lone request can have: ctas / (layers * Hkv * row_tiles)
  int row_tiles;               // row tiles of a (request, layer, kv head), at most
  float* part;                 // partial results, rows of D + 2: unnormalised output, maximum (base 2), sum
  int4* desc;                  // [kKvItems] what the join reads (tree kernel), by item or by CTA
  int by_item;
  int32_t* done;               // [kKvCounters] CTAs that have finished an item, zero between calls
};
struct KvAttnPlan {
  int kernel;                  // kKvDec or kKvTree; 0: no kernel takes the call
  int ctas, least;
  int tile_rows, row_tiles;
  size_t done_bytes, bytes;    // workspace: counters and records, then partial results
};
constexpr int kKvDec = 1;       // tiles of kKvDecRows rows
constexpr int kKvDecRows = 8;
constexpr int kKvTree = 2;      // tiles of kKvTreeRows rows
constexpr int kKvTreeRows = 128;
// Counters lead every workspace at a fixed size, so that one workspace serves calls of different shapes.
constexpr int kKvCounters = 16384;
constexpr int kKvItems = 4096;  // items of a launch of the tree kernel; their join records follow the counters
KvAttnPlan plan_kv4_attention(int Hq, int Hkv, int D, int dtype, int B, int layers, int n_max, int max_pages);
cudaError_t launch_kv4_attention_dec(const KvAttnParams& p, cudaStream_t s);
cudaError_t launch_kv4_attention_tree(const KvAttnParams& p, cudaStream_t s);

}  // namespace gdn
