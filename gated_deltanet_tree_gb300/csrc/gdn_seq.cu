// Which kernels take a batch of prompts, and in which order.
//
// Prompts of more than kTokenByToken rows go through the chunked form, 64 tokens at a time.  (The two take the same time, of
// one request and of 32, at 13 and 27 rows with 48 heads of 128 x 128, at 24 and 24 with small heads.)  Up to kSegReqs requests are in
// work together, the longest first; a segment is the next chunks of each, as many as the workspace has places for.  Its
// operands are prepared, then run through; the next segment finds the states where this one left them.  A chain's CTA takes
// some 5 us besides its chunks (3 us each), so no more requests are begun than fill the GPU: once they have kManyCtas CTAs, four
// an SM, another has to fit in whole.  Where few requests leave SMs idle, the next segment is prepared beside it: the workspace's
// halves take turns, and the chains go to a stream of the library's own, which has the higher priority and which the caller's
// stream waits for at the end.
// The workspace is large rather than kept in L2: every segment pays three launches, rounds of CTAs that do not fill the GPU
// and the states' way through memory.  8191 tokens of 48 heads took 858 us with 104 MB, 801 with 300 and 735 with 1000 (before
// the halves took turns).
//
// Measured, 16 k-heads and 48 v-heads of 128 x 128, bf16 (us): 70 tokens 31, 1024 104, 8191 651, 20001 and 15001 together 2535,
// 32 prompts of 250 to 500 tokens 1022, 128 of 50 to 100 1505.
#include <algorithm>
#include <initializer_list>
#include <mutex>
#include <new>

#include "gdn_seq.cuh"

namespace gdn {
namespace {

constexpr int kTokenByToken = 16;
// 32 prompts of 1000 to 2000 rows: 3681 us, with 32 at a time 3900; 64 of 125 to 250 1300 and 1543; with 304 CTAs six of 1500 to
// 3000 took 1133 us instead of 1065.
constexpr int kManyCtas = 608;
constexpr size_t kWorkspace = 1000u << 20;

// As many chunks as kWorkspace holds; two at least (a half each of the workspace), which fit it up to some 2000 heads.
int workspace_slots(const gdn_dims& d) {
  const size_t n = kWorkspace / seq_slot_bytes(d.Hk, d.Hv, d.dk, d.dv);
  return n < 2 ? 2 : n > 1024 ? 1024 : static_cast<int>(n);
}

// The segments of a batch of prompts, one after another.
struct Planner {
  SegReq* todo;                // the longest first
  int n, ctas;                 // ctas: of one request's chains
  int active[kSegReqs];
  int n_active = 0, begun = 0;
  Planner(SegReq* t, int count, int c) : todo(t), n(count), ctas(c) {}
  static int left(const SegReq& r) { return (r.len + kChunk - 1) / kChunk - (r.c0 + r.nc); }
  // The next chunks of some requests, at most `slots` in all; false when there are none.
  bool next(Segment& seg, int slots) {
    int kept = 0, sum = 0, most = 0;
    for (int i = 0; i < n_active; ++i)
      if (const int c = left(todo[active[i]])) active[kept++] = active[i], sum += c, most = std::max(most, c);
    n_active = kept;
    while (n_active < std::min(kSegReqs, slots) && begun < n) {
      const int c = left(todo[begun]);
      if (n_active * ctas >= kManyCtas && sum + c > slots) break;
      active[n_active++] = begun++, sum += c, most = std::max(most, c);
    }
    if (n_active == 0) return false;
    // at most `share` chunks of each: as many as there are places for, the longest one's in even parts
    int share = most, low = slots / n_active;
    for (int high = most; low < high;) {
      const int mid = low + (high - low + 1) / 2;
      int total = 0;
      for (int i = 0; i < n_active; ++i) total += std::min(mid, left(todo[active[i]]));
      if (total <= slots) low = mid; else high = mid - 1;
      share = low;
    }
    const int parts = (most + share - 1) / share;
    share = (most + parts - 1) / parts;
    seg.n = seg.slots = 0;
    for (int i = 0; i < n_active; ++i) {
      SegReq& r = todo[active[i]];
      const int c = std::min(share, left(r));
      r.c0 += r.nc;
      r.nc = c;
      r.slot0 = seg.slots;
      seg.slots += r.nc;
      seg.r[seg.n++] = r;
    }
    return true;
  }
};

// A stream and events for the chains that run beside the next segment's preparation.  They are made when first needed, kept
// for the process, and lent to one call at a time: a set still at work is lent on to the same stream only, whose order it keeps,
// so that no stream waits for another one's work.
struct Side {
  int state = 0;               // 0: not made, 1: there, 2: cannot be made
  bool lent = false;
  unsigned long long user = 0; // the number of the stream it was lent to last
  cudaStream_t stream;
  cudaEvent_t ready[2], go[2], done[2];
};
constexpr int kDevices = 64, kSides = 8;
std::mutex side_lock;
Side sides[kDevices][kSides];

bool make_side(Side& side) {
  int least = 0, greatest = 0;
  cudaError_t e = cudaDeviceGetStreamPriorityRange(&least, &greatest);
  if (e == cudaSuccess) e = cudaStreamCreateWithPriority(&side.stream, cudaStreamNonBlocking, greatest);
  for (int i = 0; i < 2; ++i)
    for (cudaEvent_t* v : {&side.ready[i], &side.go[i], &side.done[i]})
      if (e == cudaSuccess) e = cudaEventCreateWithFlags(v, cudaEventDisableTiming);
  if (e != cudaSuccess) cudaGetLastError();
  side.state = e == cudaSuccess ? 1 : 2;
  return side.state == 1;
}
bool capturing(cudaStream_t s) {
  cudaStreamCaptureStatus capture = cudaStreamCaptureStatusNone;
  if (cudaStreamIsCapturing(s, &capture) == cudaSuccess) return capture != cudaStreamCaptureStatusNone;
  cudaGetLastError();
  return true;
}
// nullptr: none is free, and the caller's stream does all of the work.
Side* borrow_side(cudaStream_t s) {
  int device = 0;
  unsigned long long user = 0;
  if (cudaGetDevice(&device) != cudaSuccess || device >= kDevices) {
    cudaGetLastError();
    return nullptr;
  }
  // another thread's capture is no concern of these calls, which put nothing on a stream
  cudaStreamCaptureMode mode = cudaStreamCaptureModeRelaxed;
  cudaThreadExchangeStreamCaptureMode(&mode);
  Side* found = nullptr;
  if (cudaStreamGetId(s, &user) == cudaSuccess) {
    std::lock_guard<std::mutex> hold(side_lock);
    for (Side& side : sides[device])
      if (!found && side.state == 1 && !side.lent && side.user == user) found = &side;
    for (Side& side : sides[device])
      if (!found && side.state == 1 && !side.lent && cudaEventQuery(side.done[0]) == cudaSuccess) found = &side;
    for (Side& side : sides[device])
      if (!found && side.state == 0 && make_side(side)) found = &side;
    if (found) found->lent = true, found->user = user;
  }
  cudaGetLastError();          // (among others: a set's work is not done yet)
  cudaThreadExchangeStreamCaptureMode(&mode);
  return found;
}
void return_side(Side* side) {
  std::lock_guard<std::mutex> hold(side_lock);
  side->lent = false;
}
// Chains of at most kFewCtas CTAs, of at least kAheadLeast chunks, in segments of kAheadChunks chunks a request: 8191 tokens of
// one request 741 -> 675 us (16 chunks 757, 32 689, 64 677), 20001 and 15001 tokens 3018 -> 2620 us; three requests (288 CTAs)
// gain nothing.
constexpr int kFewCtas = 240, kAheadLeast = 48, kAheadChunks = 48;

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
  const int ctas = p.Hv * (p.dv / 64 ? p.dv / 64 : 1);
  Planner plan{todo, n, ctas};
  const int chunks = n ? (todo[0].len + kChunk - 1) / kChunk : 0;
  // Few requests leave SMs to the next segment's preparation; several segments are needed for that.  The segments are the same
  // whether there is a stream for it or not, and with them the results.
  const bool ahead = n > 0 && n * ctas <= kFewCtas && chunks >= kAheadLeast && !capturing(s);
  Side* const side = ahead ? borrow_side(s) : nullptr;
  char* const ws = static_cast<char*>(workspace);
  const size_t half = ahead ? slots / 2 * seq_slot_bytes(p.Hk, p.Hv, p.dk, p.dv) : 0;
  const int most = ahead ? std::min(slots / 2, std::max(n * kAheadChunks, 1)) : slots;
  Segment seg{};
  int i = 0;
  if (!side) {
    for (; e == cudaSuccess && plan.next(seg, most); ++i) {
      e = launch_seq_prepare(p, seg, ws + (i & 1) * half, s);
      if (e == cudaSuccess) e = launch_seq_chain(p, seg, ws + (i & 1) * half, true, s);
    }
  } else {
    auto step = [&](cudaError_t r) {
      if (e == cudaSuccess) e = r;
    };
    for (; e == cudaSuccess && plan.next(seg, most); ++i) {
      if (i >= 2) step(cudaStreamWaitEvent(s, side->done[i & 1], 0));            // who used this half before
      if (i >= 1) step(cudaStreamWaitEvent(s, side->go[(i - 1) & 1], 0));        // the chain before takes its SMs first
      step(launch_seq_prepare(p, seg, ws + (i & 1) * half, s));
      step(cudaEventRecord(side->ready[i & 1], s));
      step(cudaStreamWaitEvent(side->stream, side->ready[i & 1], 0));
      step(cudaEventRecord(side->go[i & 1], side->stream));
      step(launch_seq_chain(p, seg, ws + (i & 1) * half, false, side->stream));
      step(cudaEventRecord(side->done[i & 1], side->stream));
    }
    // whatever has been launched there comes before what follows on the caller's stream
    if (i > 0) {
      const cudaError_t r = cudaEventRecord(side->done[0], side->stream);
      step(r);
      if (r == cudaSuccess) step(cudaStreamWaitEvent(s, side->done[0], 0));
    }
    return_side(side);
  }
  delete[] todo;
  return e;
}

}  // namespace gdn
