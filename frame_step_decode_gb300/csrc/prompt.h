// prompt.h -- what the calls on packed prompts share: the batch of sequences
// as a kernel parameter and its checks on the host.
#pragma once
#include <stdint.h>

#include "../../include/wave.h"
#include "ctx.h"

namespace wave {

// The sequences of one call that have tokens and a session, in the caller's
// order.  Passed to kernels by value (2 KB of parameters): nothing is copied
// to the device first, and a captured launch keeps the batch it was made with.
struct SeqBatch {
  int n;
  int32_t cum[WAVE_MAX_SEQS + 1];  // tokens before sequence i, sequences with nothing to do left out
  int32_t begin[WAVE_MAX_SEQS];    // its first row in the packed buffers
  int32_t slot[WAVE_MAX_SEQS];     // its session
  int32_t start[WAVE_MAX_SEQS];    // the position of its first token
  __host__ __device__ int len(int i) const { return cum[i + 1] - cum[i]; }
};

// Whether cu_seqlens is a packed layout: 1 <= n_seq <= WAVE_MAX_SEQS, starts
// at 0 or later and never decreases.
inline bool cu_ok(int n_seq, const int32_t* cu) {
  if (!cu || n_seq < 1 || n_seq > WAVE_MAX_SEQS || cu[0] < 0) return false;
  for (int i = 0; i < n_seq; ++i)
    if (cu[i + 1] < cu[i]) return false;
  return true;
}

// The batch of (cu_seqlens, slots, starts), empty slots (negative) and empty
// sequences left out.  WAVE_EINVAL for a bad layout, a slot at or beyond
// S_max, a negative start or a session named twice.
inline int make_batch(SeqBatch* b, int n_seq, const int32_t* cu, const int32_t* slots, const int32_t* starts,
                      int S_max) {
  if (!cu_ok(n_seq, cu) || !slots || !starts) return WAVE_EINVAL;
  bool seen[WAVE_MAX_SEQS] = {false};
  b->n = 0;
  b->cum[0] = 0;
  for (int i = 0; i < n_seq; ++i) {
    if (slots[i] < 0) continue;
    if (slots[i] >= S_max || starts[i] < 0 || seen[slots[i]]) return WAVE_EINVAL;
    seen[slots[i]] = true;
    const int len = cu[i + 1] - cu[i];
    if (len == 0) continue;
    b->begin[b->n] = cu[i];
    b->slot[b->n] = slots[i];
    b->start[b->n] = starts[i];
    b->cum[b->n + 1] = b->cum[b->n] + len;
    ++b->n;
  }
  return WAVE_OK;
}

// The sequence of kept token t (the last i with cum[i] <= t).
__device__ __forceinline__ int seq_of(const SeqBatch& b, int t) {
  int lo = 0, hi = b.n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (b.cum[mid] <= t)
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo;
}

constexpr int64_t kMaxStride = (1LL << 31) - 1;  // elements between rows: what a tensor map can describe

inline bool aligned16(const void* p) { return ((uintptr_t)p & 15) == 0; }

// Whether the handle's device is the current one (a launch elsewhere would
// read the workspace and the caller's tensors of another GPU).
inline bool on_device(const wave_ctx* h) {
  int dev = -1;
  return cudaGetDevice(&dev) == cudaSuccess && dev == h->device;
}

}  // namespace wave
