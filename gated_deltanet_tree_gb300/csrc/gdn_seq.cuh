// Parameters of the kernels that take sequences (prompts, single tokens) through one GDN layer.
#pragma once
#include "gdn_internal.h"

namespace gdn {

struct SeqParams {
  int Hk, Hv, dk, dv, K, C, conv_mode, act, in_dtype, out_dtype;
  float q_scale, l2_eps;
  long long x_row, gate_row;            // elements from one token's row to the next
  const void* x;                        // [rows][C]
  const float* conv_w;                  // [C][K], the layer's
  const void* beta;                     // [rows][Hv]
  const void* log_g;
  const float* state_in;                // the layer's, request 0; nullptr: zero states
  const float* conv_in;                 // nullptr: zero windows
  float* state_out;
  float* conv_out;
  long long state_stride, conv_stride;  // floats from one request to the next
  void* out;                            // [rows][Hv][dv] out_dtype
  const int32_t* live;                  // [requests] (single tokens only): 0 leaves the request as it is; nullptr: all
  int32_t* err;
};
// The requests of one launch: where their rows begin and how many there are.
constexpr int kSeqReqs = 128;
struct SeqReqs {
  int n;
  int b[kSeqReqs], start[kSeqReqs], len[kSeqReqs];
};

// Token by token; reqs nullptr: requests 0 .. n - 1 with one row each.
cudaError_t launch_seq_rec(const SeqParams& p, const SeqReqs* reqs, int n, cudaStream_t s);

// One token each of requests 0 .. n - 1, as a stream of tiles; false where that form does not apply or does not pay.
bool launch_seq_step(const SeqParams& p, int n, cudaStream_t s, cudaError_t& e);

// ---- the chunked form: 64 tokens at a time ----
constexpr int kChunk = 64;
// Bytes of one chunk's operands in the workspace (see gdn_seq_chunk.cu), for one k-head and for one v-head.
__host__ __device__ constexpr size_t seq_kq_bytes(int dk) { return 4ull * kChunk * dk * 2 + 2ull * kChunk * kChunk * 4; }
constexpr int kSeqMeta = 2 * kChunk + 16;                      // floats
__host__ __device__ constexpr size_t seq_v_bytes(int dv) { return 2ull * 128 * kChunk * 2 + kChunk * dv * 4ull + kSeqMeta * 4ull; }
__host__ __device__ constexpr size_t seq_slot_bytes(int Hk, int Hv, int dk, int dv) {
  return Hk * seq_kq_bytes(dk) + Hv * seq_v_bytes(dv);
}
// A stretch of chunks of several requests, prepared and then run through.
constexpr int kSegReqs = 64;
struct SegReq {
  int b, start, len;           // request, its first row, its rows
  int c0, nc, slot0;           // first chunk, chunks, place of the first in the workspace
};
struct Segment {
  int n, slots;
  SegReq r[kSegReqs];
};
cudaError_t launch_seq_prepare(const SeqParams& p, const Segment& seg, void* workspace, cudaStream_t s);
// right_after: the launch before it on the stream is that segment's preparation, whose end it may overlap
cudaError_t launch_seq_chain(const SeqParams& p, const Segment& seg, const void* workspace, bool right_after, cudaStream_t s);

// A ragged batch of prompts: lens[b] rows of each of B requests, one after another.
size_t seq_workspace_bytes(const gdn_dims& d);
cudaError_t launch_prefill(const SeqParams& p, const int32_t* lens, int B, void* workspace, cudaStream_t s);

}  // namespace gdn
