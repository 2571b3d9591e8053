// Parameters of the log-probability kernel.
#pragma once
#include "gdn_internal.h"

namespace gdn {

struct LogprobParams {
  int rows, V, top, dtype;
  long long v_stride;
  const void* logits;
  const int32_t* tokens;       // nullptr: no given tokens
  float* top_logp;             // [rows][top]
  int32_t* top_token;
  float* given;                // [rows]
  float* entropy;              // [rows], may be nullptr
  int32_t* err;
};
constexpr int kLogprobTop = GDN_MAX_TOP;  // best tokens a row at most (the kernel's bound comes from 32 groups)
constexpr int kLogprobVocab = 1 << 30;    // the kernel's indices pass V by up to a cluster's step of 2^16
cudaError_t launch_logprobs(const LogprobParams& p, cudaStream_t s);

}  // namespace gdn
