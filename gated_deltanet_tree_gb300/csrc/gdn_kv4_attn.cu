// Which kernel takes an attention call over the 4-bit cache, and how much of the GPU it gets.
//
// kv4_attn_dec_kernel unpacks the cache once for each tile of eight rows: while the rows of a kv head are few, the
// cache's bytes are the bound and it moves them best.  kv4_attn_tree_kernel unpacks it once for 128 rows.  They cross
// at (microseconds, the first kernel against the second; 16 requests of 5000 tokens | 4 of 5000):
//   D = 256:   8 rows  53 :  66 |  31 :  39     16 rows  72 :  68 | 44 : 39 (tiles of 12 to 16 rows: even)
//   D = 128:  16 rows  61 :  72 |  35 :  40     24 rows  84 :  74 | 39 : 41     32 rows  96 :  74
//   D =  64:  24 rows  61 :  66 |  31 :  36     32 rows  76 :  66 | 35 : 35
// fp32 calls run in kv4_attn_dec_kernel at any size.
#include "gdn_kv4_attn.cuh"

namespace gdn {

namespace {
int dec_rows(int D) { return D == 64 ? 24 : 16; }      // rows of a kv head
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
    pl.ctas = 152 * 2;            // two an SM
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
