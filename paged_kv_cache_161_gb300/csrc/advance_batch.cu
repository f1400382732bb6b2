// pa_advance_batch: the metadata of a step (block tables, slot mapping, positions, query
// offsets) from request lengths, on the device (vLLM 0.10.0 flow page, 3.3 KV Manager and
// 3.5 Attention: slot_mapping, block_table, query_start_loc; "vLLM" docs page, algorithm
// flow: a token that must go into a full block takes a new one; ceil(n / B) blocks for n
// tokens).
//
// With c_s cached and q_s new tokens, request s takes need_s = ceil((c_s + q_s) / B) -
// ceil(c_s / B) blocks from the free list, in request order: two exclusive prefix sums
// (of q for the token offsets, of need for the list offsets), then every token on its own:
// its request by binary search in the offsets, its block from the table or the free list.
// The first token of a new block also stores the block's id in the table.
//
// Bound by latency, not bytes (about 28 bytes a request and token): one launch of one
// cluster of up to 16 CTAs. Each CTA scans all requests itself (1024 at a time, from L2),
// which costs less than handing the offsets over, and takes every C-th batch of tokens.
// The cluster barrier before the last writes lets seq_lens_out and free_head_out be the
// input arrays, so that one captured graph can be replayed step after step.
#include "common.cuh"
#include "launch.h"

namespace pa {
namespace {

struct AdvanceParams {
  int32_t* table;
  const int32_t* seq_lens;
  const int32_t* query_lens;
  const int32_t* free_blocks;
  const int32_t* free_head;
  int32_t* seq_lens_out;
  int32_t* free_head_out;
  int32_t* qsl;
  int64_t* slots;
  int32_t* positions;
  unsigned int* err;
  int64_t num_blocks;
  int num_seqs, num_tokens, width, block_size, num_free;
};

struct Request {
  int ctx, q, need;
  bool bad;
};

__device__ __forceinline__ Request load_request(const AdvanceParams& p, int s) {
  Request r;
  r.ctx = p.seq_lens[s];  // not __ldg: seq_lens_out may be the same array
  r.q = p.query_lens[s];
  r.bad = r.ctx < 0 || r.q < 0 || int64_t(r.ctx) + r.q > int64_t(p.width) * p.block_size || r.q > p.num_tokens;
  if (r.bad) r.ctx = r.q = 0;
  const int B = p.block_size;
  r.need = (r.ctx + r.q) / B - r.ctx / B + ((r.ctx + r.q) % B != 0) - (r.ctx % B != 0);
  return r;
}

// Inclusive scan over the block of (need << 32 | q): neither half overflows, since the totals
// have been checked.
template <int kThreads>
__device__ uint64_t block_inclusive_scan(uint64_t x, uint64_t* red) {
  constexpr int kWarps = kThreads / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const uint64_t y = __shfl_up_sync(0xffffffffu, x, d);
    if (lane >= d) x += y;
  }
  if (lane == 31) red[warp] = x;
  __syncthreads();
  if (warp == 0) {
    uint64_t w = lane < kWarps ? red[lane] : 0;
#pragma unroll
    for (int d = 1; d < kWarps; d <<= 1) {
      const uint64_t y = __shfl_up_sync(0xffffffffu, w, d);
      if (lane >= d) w += y;
    }
    if (lane < kWarps) red[lane] = w;
  }
  __syncthreads();
  return x + (warp ? red[warp - 1] : 0);
}

// Sum over the warp of values below 2^48, in two parts of 24 bits, whose sums cannot overflow.
__device__ __forceinline__ uint64_t warp_sum(uint64_t x) {
  const uint64_t lo = __reduce_add_sync(0xffffffffu, unsigned(x & 0xffffff));
  const uint64_t hi = __reduce_add_sync(0xffffffffu, unsigned(x >> 24));
  return lo + (hi << 24);
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}

// kRun: tokens of a lane whose loads are in flight together.
template <int kThreads, int kRun>
__global__ void __launch_bounds__(kThreads) advance_batch_kernel(const AdvanceParams p) {
  __shared__ uint64_t red[kThreads / 32];
  __shared__ int qoff[kThreads + 1], noff[kThreads + 1], ctx[kThreads];
  __shared__ unsigned long long total_q, total_need;
  griddep_wait();
  griddep_launch_dependents();
  const int tid = threadIdx.x, S = p.num_seqs, B = p.block_size;
  const int rank = int(cluster_rank()), ranks = int(cluster_size());
  const int head = *p.free_head;  // every thread, before the barrier: free_head_out may be the same word

  // Totals and checks first: a step that cannot be built changes nothing.
  bool bad = false;
  uint64_t sq = 0, sn = 0;
  Request mine = {0, 0, 0, false};  // of the first tile, kept
  for (int s = tid; s < S; s += kThreads) {
    const Request r = load_request(p, s);
    if (s == tid) mine = r;
    bad |= r.bad;
    sq += r.q;
    sn += r.need;
  }
  bad |= sq > uint64_t(p.num_tokens);  // so that the sums below stay small (a block needs a token)
  if (tid == 0) total_q = total_need = 0;
  bad = __syncthreads_or(bad);
  sq = warp_sum(sq);
  sn = warp_sum(sn);
  if ((tid & 31) == 0) {
    atomicAdd(&total_q, sq);
    atomicAdd(&total_need, sn);
  }
  __syncthreads();
  const uint64_t need_all = total_need;
  const bool range = bad || total_q > uint64_t(p.num_tokens);
  const bool blocks = head < 0 || uint64_t(max(head, 0)) + need_all > uint64_t(p.num_free);
  const bool fail = range || blocks;
  if (fail && rank == 0 && tid == 0) {
    if (range) raise_error(p.err, PA_DEVERR_SEQ_RANGE);
    if (blocks) raise_error(p.err, PA_DEVERR_NO_BLOCKS);
  }
  const int tokens = fail ? 0 : int(total_q);

  int q_base = 0, n_base = head;  // of the tile
  for (int base = 0; base < S; base += kThreads) {
    const int s = base + tid;
    if (base > 0 && s < S) mine = load_request(p, s);
    const bool have = s < S && !fail;
    const uint64_t x = have ? (uint64_t(mine.need) << 32 | uint32_t(mine.q)) : 0;
    const uint64_t inc = block_inclusive_scan<kThreads>(x, red), ex = inc - x;
    qoff[tid] = q_base + int(uint32_t(ex));
    noff[tid] = n_base + int(ex >> 32);
    ctx[tid] = mine.ctx;
    if (tid == kThreads - 1) {
      qoff[kThreads] = q_base + int(uint32_t(inc));
      noff[kThreads] = n_base + int(inc >> 32);
    }
    if (rank == 0 && s < S) p.qsl[s + 1] = q_base + int(uint32_t(inc));
    __syncthreads();
    const int n = min(kThreads, S - base), t_end = qoff[kThreads];
    // the last request of the tile whose offset is <= t (requests without tokens come before it)
    auto request_of = [&](int t, int lo) {
      int hi = n - 1;
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (qoff[mid] <= t)
          lo = mid;
        else
          hi = mid - 1;
      }
      return lo;
    };
    // A warp takes 32 x kRun consecutive tokens: mostly one request's (a prompt chunk) or one
    // each of consecutive requests (decodes); other tokens search.
    const int warp = tid >> 5, lane = tid & 31, stride = ranks * kThreads * kRun;
    for (int t0 = q_base + (rank * (kThreads / 32) + warp) * (32 * kRun); t0 < t_end; t0 += stride) {
      int first = request_of(t0, 0);
      int pos[kRun], from[kRun];  // from >= 0: the request's from-th new block
      int32_t id[kRun];
      int32_t* entry[kRun];
#pragma unroll
      for (int k = 0; k < kRun; ++k) {
        const int t = min(t0 + k * 32 + lane, t_end - 1);
        int r = first;
        if (t >= (r + 1 < n ? qoff[r + 1] : t_end)) {
          r = min(first + lane, n - 1);
          if (t < qoff[r] || t >= (r + 1 < n ? qoff[r + 1] : t_end)) r = request_of(t, first);
        }
        first = __shfl_sync(0xffffffffu, r, 31);
        const int c = ctx[r];
        pos[k] = c + (t - qoff[r]);
        const int b = pos[k] / B, first_new = c / B + (c % B != 0);
        from[k] = b - first_new;
        entry[k] = p.table + int64_t(base + r) * p.width + b;
        id[k] = from[k] >= 0 ? __ldg(p.free_blocks + noff[r] + from[k]) : *entry[k];
      }
#pragma unroll
      for (int k = 0; k < kRun; ++k) {
        const int t = t0 + k * 32 + lane, in = pos[k] % B;
        if (t >= t_end) break;
        if (from[k] >= 0 && in == 0) *entry[k] = id[k];
        const bool ok = id[k] >= 0 && id[k] < p.num_blocks;
        if (!ok) raise_error(p.err, PA_DEVERR_BLOCK_RANGE);
        p.slots[t] = ok ? int64_t(id[k]) * B + in : -1;
        p.positions[t] = pos[k];
      }
    }
    q_base = t_end;
    n_base = noff[kThreads];
    __syncthreads();
  }
  if (rank == 0 && tid == 0) p.qsl[0] = 0;
  for (int t = tokens + rank * kThreads + tid; t < p.num_tokens; t += ranks * kThreads) {
    p.slots[t] = -1;
    p.positions[t] = 0;
  }
  // every CTA has read the lengths and the head: they may now be overwritten
  cluster_barrier();
  if (rank != 0) return;
  for (int s = tid; s < S; s += kThreads) p.seq_lens_out[s] = p.seq_lens[s] + (fail ? 0 : p.query_lens[s]);
  if (tid == 0) *p.free_head_out = fail ? head : head + int(need_all);
}

// Whether the device runs clusters of 16 CTAs of the kernel for long chunks: they need the opt-in
// and 16 SMs of one GPC to themselves, which a process given part of the GPU may not have. Asked
// once per device; an answer that cannot be had counts as no.
bool cluster_of_16_fits() {
  static std::mutex mu;
  static int known[64] = {};  // 1: yes, -1: no
  constexpr auto kern = advance_batch_kernel<1024, 4>;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return false;
  std::lock_guard<std::mutex> lock(mu);
  if (!known[dev]) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(16);
    cfg.blockDim = dim3(1024);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 16;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int clusters = 0;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess ||
        cudaOccupancyMaxActiveClusters(&clusters, kern, &cfg) != cudaSuccess) {
      cudaGetLastError();  // answered here: the launch's status is its own
      clusters = 0;
    }
    known[dev] = clusters > 0 ? 1 : -1;
  }
  return known[dev] > 0;
}

}  // namespace

cudaError_t launch_advance_batch(int32_t* block_table, int width, const int32_t* seq_lens, const int32_t* query_lens,
                                 const int32_t* free_blocks, int num_free, const int32_t* free_head,
                                 int32_t* seq_lens_out, int32_t* free_head_out, int32_t* query_start_loc,
                                 int64_t* slot_mapping, int32_t* positions, int num_seqs, int num_tokens,
                                 int block_size, int64_t num_blocks, unsigned int* err, cudaStream_t stream) {
  AdvanceParams p = {block_table, seq_lens,      query_lens,      free_blocks,  free_head, seq_lens_out,
                     free_head_out, query_start_loc, slot_mapping, positions,    err,       num_blocks,
                     num_seqs,    num_tokens,    width,           block_size,   num_free};
  // A small step in one CTA of 256 threads (256 decodes: 3.8 us, 5.4 with 1024 threads). Else one
  // token a lane up to 8 CTAs (the portable cluster size), beyond that four at once and, from
  // two rounds of 8 on, 16 CTAs where they fit (480 decodes and 32 chunks of 2048 tokens: 8.5 us, 11.2 with 8).
  constexpr int kFull = 1024;
  const bool small = num_seqs <= 256 && num_tokens <= 256;
  int ctas = 1;
  while (ctas < 8 && int64_t(ctas) * kFull < num_tokens) ctas *= 2;
  if (num_tokens > 8 * kFull * 4 && cluster_of_16_fits()) ctas = 16;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(ctas));
  cfg.blockDim = dim3(small ? 256 : kFull);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = unsigned(ctas);
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = ctas > 1 ? 2 : 1;  // (a CTA without the attribute is a cluster of its own)
  return cudaLaunchKernelEx(&cfg,
                            small                                    ? advance_batch_kernel<256, 1>
                            : int64_t(ctas) * kFull < num_tokens ? advance_batch_kernel<1024, 4>
                                                                     : advance_batch_kernel<1024, 1>,
                            p);
}

}  // namespace pa
