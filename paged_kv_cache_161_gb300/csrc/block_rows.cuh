// Shared by the block-sparse kernels: the request and position of a query token, found on
// the device from query_start_loc and seq_lens.
#pragma once

#include "common.cuh"
#include "launch.h"

namespace pa {
namespace {

struct QueryRow {
  int s;    // the request, or -1: the token belongs to no request (padding behind the last)
  int pos;  // the token's position: seq_lens[s] - q_len + index among the request's queries
};

// The last request whose query_start_loc is <= t, by a 32-way search of the warp (all 32
// lanes call it with one t): one dependent load up to 31 requests, two up to 991, ...
// A decode batch answers with its first load.
__device__ __forceinline__ QueryRow find_row(const BatchArgs& b, int t) {
  const int lane = threadIdx.x & 31, S = b.num_seqs;
  const int32_t* qsl = b.query_start_loc;
  int s = -1;
  if (t < S && __ldg(qsl + t) == t && __ldg(qsl + t + 1) == t + 1) {
    s = t;
  } else {
    int lo = 0, n = S + 1;  // the wanted entry is in [lo, lo + n): entries [0, S], non-decreasing
    while (n > 1) {
      const int step = (n + 31) / 32;
      const int at = lo + lane * step;
      const bool le = at < lo + n && __ldg(qsl + at) <= t;
      const unsigned m = __ballot_sync(0xffffffffu, le);
      if (m == 0) break;  // t < qsl[0]: only with a malformed query_start_loc
      const int k = 31 - __clz(m);
      const int next = lo + k * step;
      n = min(step, lo + n - next);
      lo = next;
    }
    if (lo < S && __ldg(qsl + lo) <= t && t < __ldg(qsl + lo + 1)) s = lo;
  }
  if (s < 0) return {-1, -1};
  const int q0 = __ldg(qsl + s), q1 = __ldg(qsl + s + 1), L = __ldg(b.seq_lens + s);
  const int64_t cap = int64_t(b.max_blocks_per_seq) * b.block_size;
  if (L > cap || q1 - q0 > L) {
    if (lane == 0) raise_error(b.err, PA_DEVERR_SEQ_RANGE);
    return {-1, -1};
  }
  return {s, L - (q1 - q0) + (t - q0)};
}

}  // namespace
}  // namespace pa
