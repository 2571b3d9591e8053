// Which kernel takes an attention call over the 4-bit cache, and how much of the GPU it gets.
//
// kv4_attn_dec_kernel unpacks the cache once for each tile of eight rows: while the rows of a kv head are few, the
// cache's bytes are the bound and it moves them best.  kv4_attn_tree_kernel unpacks it once for 128 rows.  They cross
// at (microseconds, the first kernel : the second; 4 kv heads of 256 or 8 smaller ones, bf16):
//                       1 request, 5000 tokens  4 of 5000     16 of 5000    32 of up to 16384
//   D = 256:   8 rows       20.7 : 22.7        33.0 : 33.0   39.5 : 53.9      113 : 200
//             16 rows       24.8 : 22.7        34.7 : 33.3   52.9 : 54.0      203 : 201
//             18 rows       24.7 : 22.8        37.1 : 34.8   65.8 : 55.1      289 : 203
//   D = 128:  20 rows       18.6 : 22.7        30.5 : 35.1   59.1 : 68.0      253 : 250
//             24 rows       18.6 : 22.7        31.0 : 35.6   62.5 : 67.9      274 : 250
//             32 rows       20.7 : 22.7        35.0 : 36.5   76.1 : 69.7      348 : 252
//   D =  64:  24 rows       16.6 : 20.7        26.8 : 33.0   47.3 : 61.7      187 : 222
//             28 rows       16.6 : 20.7        28.1 : 33.0   55.5 : 62.0      225 : 222
//             32 rows       18.0 : 20.7        28.8 : 33.0   56.9 : 63.0      238 : 222
// fp32 calls run in kv4_attn_dec_kernel at any size.
#include "gdn_kv4_attn.cuh"

namespace gdn {

namespace {
int dec_rows(int D) { return D == 64 ? 28 : D == 128 ? 20 : 16; }      // rows of a kv head
}

// max_pages: the longest request's pages where the host knows a bound, else 0; with it no more CTAs are launched than
// can have work.
KvAttnPlan plan_kv4_attention(int Hq, int Hkv, int D, int dtype, int B, int layers, int n_max, int max_pages) {
  KvAttnPlan pl{};
  const int rows = n_max * (Hq / Hkv);
  const int dec_tiles = (rows + kKvDecRows - 1) / kKvDecRows, tree_tiles = (rows + kKvTreeRows - 1) / kKvTreeRows;
  const long long heads = static_cast<long long>(layers) * Hkv;
  pl.done_bytes = kKvCounters * sizeof(int32_t) + kKvItems * sizeof(int4);
  if (dtype == GDN_DTYPE_BF16 && rows > dec_rows(D) && heads * tree_tiles <= kKvItems) {
    pl.kernel = kKvTree;
    pl.tile_rows = kKvTreeRows;
    pl.row_tiles = tree_tiles;
    pl.least = 2;
    pl.ctas = 152;                // one an SM
  } else if (heads * dec_tiles <= kKvCounters) {
    pl.kernel = kKvDec;
    pl.tile_rows = kKvDecRows;
    pl.row_tiles = dec_tiles;
    pl.least = D == 256 ? 3 : 4;  // a page for each of a CTA's pairs of warps
    pl.ctas = 152 * 2;            // two an SM (fp32 calls of D = 256 have room for one: two rounds)
  } else {
    return pl;                    // more items a request than a launch has counters for
  }
  if (max_pages > 0) {
    const long long most = heads * B * pl.row_tiles * ((max_pages + pl.least - 1) / pl.least);
    pl.ctas = most < pl.ctas ? static_cast<int>(most) : pl.ctas;
  }
  pl.bytes = pl.done_bytes + static_cast<size_t>(pl.ctas) * 2 * pl.tile_rows * (D + 2) * sizeof(float);
  return pl;
}

}  // namespace gdn
