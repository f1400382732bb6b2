// Shared by the block-sparse kernels: the request and position of a query token, found on
// the device from query_start_loc and seq_lens.
//
// These kernels start before the one in front of them has ended, and read what it wrote behind
// griddep_wait(): none of their pointers is __restrict__, which would let the compiler take the
// wait's memory clobber as not meant for them and move a load above it.
#pragma once

#include "common.cuh"
#include "launch.h"

namespace pa {
namespace {

struct QueryRow {
  int s;    // the request, or -1: the token belongs to no request (padding behind the last)
  int pos;  // the token's position: seq_lens[s] - q_len + index among the request's queries
};

// The request of token t (all 32 lanes of a warp call it with one t). A decode batch (request t
// is token t) and batches of up to 31 requests answer after one round of loads; others search
// query_start_loc 32 ways: two more rounds up to 991 requests, three up to 31743.
__device__ __forceinline__ QueryRow find_row(const BatchArgs& b, int t) {
  const int lane = threadIdx.x & 31, S = b.num_seqs;
  const int32_t* qsl = b.query_start_loc;
  const bool few = S <= 31;
  const int mine = min(few ? lane : t, S), mine_len = __ldg(b.seq_lens + min(mine, S - 1));
  int q0 = __ldg(qsl + mine), q1 = few ? 0 : __ldg(qsl + min(t + 1, S)), L = mine_len, s = -1;
  if (few) {
    const unsigned m = __ballot_sync(0xffffffffu, lane <= S && q0 <= t);  // non-decreasing: the lowest lanes
    const int at = m ? 31 - __clz(m) : 0;
    const int a = __shfl_sync(0xffffffffu, q0, at), z = __shfl_sync(0xffffffffu, q0, min(at + 1, S));
    L = __shfl_sync(0xffffffffu, mine_len, at);
    q0 = a;
    q1 = z;
    if (m && at < S && t < q1) s = at;
  } else if (t < S && q0 == t && q1 == t + 1) {
    s = t;
  } else {
    int lo = 0, n = S + 1;  // the last entry <= t is in [lo, lo + n): entries [0, S], non-decreasing
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
    if (lo < S) {
      q0 = __ldg(qsl + lo);
      q1 = __ldg(qsl + lo + 1);
      L = __ldg(b.seq_lens + lo);
      if (q0 <= t && t < q1) s = lo;
    }
  }
  if (s < 0) return {-1, -1};
  const int64_t cap = int64_t(b.max_blocks_per_seq) * b.block_size;
  if (L > cap || q1 - q0 > L) {
    if (lane == 0) raise_error(b.err, PA_DEVERR_SEQ_RANGE);
    return {-1, -1};
  }
  return {s, L - (q1 - q0) + (t - q0)};
}

}  // namespace
}  // namespace pa
