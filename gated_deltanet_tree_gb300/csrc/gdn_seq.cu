// Which kernels take a batch of prompts, and in which order.
//
// Prompts of more than kTokenByToken rows go through the chunked form, 64 tokens at a time.  (The two take the same time, of
// one request and of 32, at 13 and 27 rows with 48 heads of 128 x 128, at 24 and 24 with small heads.)  Up to kSegReqs requests are in
// work together, the longest first; a segment is the next chunks of each, as many as the workspace has places for.  Its
// operands are prepared, then run through; the next segment finds the states where this one left them.
// The workspace is large rather than kept in L2: every segment pays three launches, rounds of CTAs that do not fill the GPU
// and the states' way through memory.  8191 tokens of 48 heads took 858 us with 104 MB, 801 with 300 and 735 with 1000; 32
// prompts of up to 500 tokens 1447, 1323 and 1237.
#include <algorithm>
#include <new>

#include "gdn_seq.cuh"

namespace gdn {
namespace {

constexpr int kTokenByToken = 16;
constexpr size_t kWorkspace = 1000u << 20;

int workspace_slots(const gdn_dims& d) {
  const size_t n = kWorkspace / seq_slot_bytes(d.Hk, d.Hv, d.dk, d.dv);
  return n < kSegReqs ? kSegReqs : n > 1024 ? 1024 : static_cast<int>(n);
}

}  // namespace

size_t seq_workspace_bytes(const gdn_dims& d) {
  return workspace_slots(d) * seq_slot_bytes(d.Hk, d.Hv, d.dk, d.dv);
}

cudaError_t launch_prefill(const SeqParams& p, const int32_t* lens, int B, void* workspace, cudaStream_t s) {
  SeqReqs few{};
  gdn_dims d{};
  d.Hk = p.Hk, d.Hv = p.Hv, d.dk = p.dk, d.dv = p.dv;
  const int slots = workspace_slots(d);
  SegReq* todo = new (std::nothrow) SegReq[B];
  if (!todo) return cudaErrorMemoryAllocation;
  int n = 0, start = 0;
  cudaError_t e = cudaSuccess;
  for (int b = 0; b < B; ++b) {
    if (lens[b] > kTokenByToken) {
      todo[n++] = SegReq{b, start, lens[b], 0, 0, 0};
    } else if (lens[b] > 0) {
      few.b[few.n] = b, few.start[few.n] = start, few.len[few.n] = lens[b];
      ++few.n;
    }
    start += lens[b];
    if (few.n == kSeqReqs || (b == B - 1 && few.n > 0)) {
      if (e == cudaSuccess) e = launch_seq_rec(p, &few, few.n, s);
      few.n = 0;
    }
  }
  std::sort(todo, todo + n, [](const SegReq& a, const SegReq& c) { return a.len != c.len ? a.len > c.len : a.b < c.b; });
  Segment seg{};
  int active[kSegReqs], n_active = 0, next = 0;
  while (e == cudaSuccess && (n_active > 0 || next < n)) {
    while (n_active < kSegReqs && next < n) active[n_active++] = next++;
    // the longest one's chunks in even parts (the others' follow from its)
    int most = 0;
    for (int i = 0; i < n_active; ++i) {
      const SegReq& r = todo[active[i]];
      most = std::max(most, (r.len + kChunk - 1) / kChunk - (r.c0 + r.nc));
    }
    const int parts = (most + slots / n_active - 1) / (slots / n_active), share = (most + parts - 1) / parts;
    seg.n = seg.slots = 0;
    for (int i = 0; i < n_active; ++i) {
      SegReq& r = todo[active[i]];
      r.c0 += r.nc;
      r.nc = std::min(share, (r.len + kChunk - 1) / kChunk - r.c0);
      r.slot0 = seg.slots;
      seg.slots += r.nc;
      seg.r[seg.n++] = r;
    }
    e = launch_seq_chunks(p, seg, workspace, s);
    int left = 0;
    for (int i = 0; i < n_active; ++i) {
      const SegReq& r = todo[active[i]];
      if ((r.c0 + r.nc) * kChunk < r.len) active[left++] = active[i];
    }
    n_active = left;
  }
  delete[] todo;
  return e;
}

}  // namespace gdn
