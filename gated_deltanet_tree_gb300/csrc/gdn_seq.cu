// Which kernels take a batch of prompts.
#include "gdn_seq.cuh"

namespace gdn {

size_t seq_workspace_bytes(const gdn_dims&) { return 256; }

cudaError_t launch_prefill(const SeqParams& p, const int32_t* lens, int B, void*, cudaStream_t s) {
  SeqReqs r{};
  int start = 0;
  for (int b = 0; b < B; ++b) {
    if (lens[b] > 0) {
      r.b[r.n] = b, r.start[r.n] = start, r.len[r.n] = lens[b];
      ++r.n;
    }
    start += lens[b];
    if (r.n == kSeqReqs || (b == B - 1 && r.n > 0)) {
      const cudaError_t e = launch_seq_rec(p, &r, r.n, s);
      if (e != cudaSuccess) return e;
      r.n = 0;
    }
  }
  return cudaSuccess;
}

}  // namespace gdn
