// Parameters of the acceptance kernels.
#pragma once
#include "gdn_internal.h"

namespace gdn {

struct AcceptParams {
  int B, n_max, V, logits_dtype, draft_dtype;
  long long v_stride;
  const int32_t* words;
  const void* logits;
  const int32_t* tokens;
  const void* draft;           // nullptr: the drafted tokens were chosen, not sampled
  const float* uniform;
  const float* gumbel;
  const float* temperature;    // nullptr: all 0
  int32_t* path;
  int32_t* len;
  int32_t* next;
  int32_t* err;
  int n_slices;                // > 0: every row is reduced at once, in this many slices
  void* slices;                // [B][n_max][n_slices] partial results of 16 bytes (workspace)
};
constexpr int kMaxVocab = 1 << 30;   // the kernels' indices pass V by up to a cluster's step of 2^15 before they are compared with it
// Slices of a row where all rows are reduced at once, 0 where the walk reads the ones on its path; the most a call needs
// is with draft probabilities.
int accept_slices(int B, int n_max, int V, bool draft);
cudaError_t launch_accept(const AcceptParams& p, cudaStream_t s);

}  // namespace gdn
