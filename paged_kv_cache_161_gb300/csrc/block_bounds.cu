// pa_block_bounds: the smallest and largest cached key of each block that holds new tokens,
// per KV head and dimension: the summary from which pa_block_scores bounds a block's logits.
//
//   bounds[id, g, 0, d] = min_i K_i[g, d],  bounds[id, g, 1, d] = max_i K_i[g, d]
//
// over the positions of the block below the request's length (rows past it are never read).
// Recomputed from the cache, not updated in place: a call may be repeated, a block that was
// reused, copied or swapped in needs no special case, and nothing depends on the order in
// which tokens arrived. Minimum and maximum round nothing (E4M3 codes' values are bf16
// values), and a NaN key gives NaN bounds.
//
// Bound by the bytes of the touched blocks' keys. A thread owns one 16-byte column of a
// block's rows, loads kBatch rows at a time and keeps the packed minimum and maximum in
// registers; a warp's loads are 512 consecutive bytes of a row.
#include <algorithm>

#include "block_rows.cuh"

namespace pa {
namespace {

constexpr int kThreads = 256;
constexpr int kBatch = 8;  // rows loaded before the first is used

template <typename KV>
struct Column;
// Packed min / max over the rows of a 16-byte column.
template <>
struct Column<__nv_bfloat16> {
  __nv_bfloat162 lo[4], hi[4];
  __device__ __forceinline__ void add(const uint4& u, bool first) {
    const __nv_bfloat162* w = reinterpret_cast<const __nv_bfloat162*>(&u);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      lo[i] = first ? w[i] : __hmin2_nan(lo[i], w[i]);
      hi[i] = first ? w[i] : __hmax2_nan(hi[i], w[i]);
    }
  }
  __device__ __forceinline__ void store(__nv_bfloat16* plo, __nv_bfloat16* phi) const {
    *reinterpret_cast<uint4*>(plo) = *reinterpret_cast<const uint4*>(lo);
    *reinterpret_cast<uint4*>(phi) = *reinterpret_cast<const uint4*>(hi);
  }
};
template <>
struct Column<Fp8E4M3> {
  __half2 lo[8], hi[8];  // E4M3 values are f16 values
  __device__ __forceinline__ void add(const uint4& u, bool first) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t c[2];
      asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
          : "=r"(c[0]), "=r"(c[1])
          : "r"(w[i]));
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const __half2 h = *reinterpret_cast<const __half2*>(&c[j]);
        lo[2 * i + j] = first ? h : __hmin2_nan(lo[2 * i + j], h);
        hi[2 * i + j] = first ? h : __hmax2_nan(hi[2 * i + j], h);
      }
    }
  }
  __device__ __forceinline__ void store(__nv_bfloat16* plo, __nv_bfloat16* phi) const {
    float f[16], h[16];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 a = __half22float2(lo[i]), b = __half22float2(hi[i]);
      f[2 * i] = a.x, f[2 * i + 1] = a.y, h[2 * i] = b.x, h[2 * i + 1] = b.y;
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      reinterpret_cast<uint4*>(plo)[i] = Elem<__nv_bfloat16>::pack(f + 8 * i);
      reinterpret_cast<uint4*>(phi)[i] = Elem<__nv_bfloat16>::pack(h + 8 * i);
    }
  }
};

// Touched blocks of request s: logical blocks [first, first + count).
struct Touched {
  int first, count, len;
};
__device__ __forceinline__ Touched touched(const BatchArgs& b, int s) {
  const int q = __ldg(b.query_start_loc + s + 1) - __ldg(b.query_start_loc + s), L = __ldg(b.seq_lens + s);
  if (q <= 0) return {0, 0, 0};
  if (q > L || L > int64_t(b.max_blocks_per_seq) * b.block_size) {
    raise_error(b.err, PA_DEVERR_SEQ_RANGE);
    return {0, 0, 0};
  }
  const int first = (L - q) / b.block_size;
  return {first, (L - 1) / b.block_size - first + 1, L};
}

template <typename KV>
__device__ __forceinline__ void reduce_column(const BatchArgs& b, __nv_bfloat16* bounds, const uint4* cache, int vec,
                                              int vecs, int head_dim, int s, int blk, int len) {
  constexpr int kElems = 16 / sizeof(KV);
  const int id = __ldg(b.block_table + int64_t(s) * b.max_blocks_per_seq + blk);
  if (id < 0 || id >= b.num_blocks) {
    if (vec == 0) raise_error(b.err, PA_DEVERR_BLOCK_RANGE);
    return;
  }
  const int rows = min(b.block_size, len - blk * b.block_size);
  const uint4* src = cache + int64_t(id) * b.block_size * vecs + vec;
  Column<KV> col;
  for (int r0 = 0; r0 < rows; r0 += kBatch) {
    uint4 u[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) u[i] = __ldg(src + int64_t(min(r0 + i, rows - 1)) * vecs);  // the last row again: harmless
#pragma unroll
    for (int i = 0; i < kBatch; ++i) col.add(u[i], r0 + i == 0);
  }
  const int e = vec * kElems, head = e / head_dim, d = e % head_dim;
  __nv_bfloat16* dst = bounds + (int64_t(id) * (vecs * kElems / head_dim) + head) * 2 * head_dim + d;
  col.store(dst, dst + head_dim);
}

// A decode batch: request s touches one block; one thread per (request, column).
template <typename KV>
__global__ void __launch_bounds__(kThreads) bounds_decode_kernel(const __grid_constant__ BatchArgs b,
                                                                __nv_bfloat16* bounds, const uint4* cache, int vecs,
                                                                int head_dim) {
  griddep_wait();
  griddep_launch_dependents();
  const int64_t i = int64_t(blockIdx.x) * kThreads + threadIdx.x;
  const int s = int(i / vecs), vec = int(i % vecs);
  if (s >= b.num_seqs) return;
  const Touched w = touched(b, s);
  for (int j = 0; j < w.count; ++j)
    reduce_column<KV>(b, bounds, cache, vec, vecs, head_dim, s, w.first + j, w.len);
}

// Any batch: the touched blocks of all requests, request-major, are split evenly over the
// CTAs; each CTA scans the requests' counts (1024 at a time) to find its own.
template <typename KV>
__global__ void __launch_bounds__(kThreads) bounds_kernel(const __grid_constant__ BatchArgs b, __nv_bfloat16* bounds,
                                                         const uint4* cache, int vecs, int head_dim) {
  constexpr int kPer = 4, kTile = kThreads * kPer;  // requests per thread and tile
  __shared__ int warp_sum[kThreads / 32];
  __shared__ int start[kTile + 1];
  __shared__ unsigned long long all;
  griddep_wait();
  griddep_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) all = 0;
  __syncthreads();
  unsigned long long mine = 0;
  for (int s = tid; s < b.num_seqs; s += kThreads) mine += touched(b, s).count;
#pragma unroll
  for (int m = 16; m >= 1; m >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, m);
  if (lane == 0 && mine) atomicAdd(&all, mine);
  __syncthreads();
  const int64_t total = int64_t(all);
  const int64_t u0 = total * blockIdx.x / gridDim.x, u1 = total * (blockIdx.x + 1) / gridDim.x;
  int64_t base = 0;  // blocks of the tiles before
  for (int s0 = 0; s0 < b.num_seqs && base < u1; s0 += kTile) {
    int c[kPer], sum = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int s = s0 + tid * kPer + i;
      c[i] = s < b.num_seqs ? touched(b, s).count : 0;
      sum += c[i];
    }
    int inc = sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, inc, d);
      if (lane >= d) inc += y;
    }
    if (lane == 31) warp_sum[warp] = inc;
    __syncthreads();
    int ex = inc - sum;
    for (int w = 0; w < warp; ++w) ex += warp_sum[w];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      start[tid * kPer + i] = ex;
      ex += c[i];
    }
    if (tid == kThreads - 1) start[kTile] = ex;
    __syncthreads();
    const int64_t a0 = max(u0 - base, int64_t(0)), a1 = min(u1 - base, int64_t(start[kTile]));
    for (int64_t i = a0 * vecs + tid; i < a1 * vecs; i += kThreads) {
      const int u = int(i / vecs), vec = int(i % vecs);
      int lo = 0, hi = kTile - 1;  // the last request that starts at or before block u
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (start[mid] <= u)
          lo = mid;
        else
          hi = mid - 1;
      }
      const Touched w = touched(b, s0 + lo);
      reduce_column<KV>(b, bounds, cache, vec, vecs, head_dim, s0 + lo, w.first + u - start[lo], w.len);
    }
    base += start[kTile];
    __syncthreads();
  }
}

template <typename KV>
cudaError_t launch(const BatchArgs& b, void* bounds, const void* k_cache, int num_kv_heads, int head_dim,
                   cudaStream_t stream) {
  const int vecs = num_kv_heads * head_dim * int(sizeof(KV)) / 16;
  auto* out = static_cast<__nv_bfloat16*>(bounds);
  auto* in = static_cast<const uint4*>(k_cache);
  if (b.max_query_len <= 1) {
    const int64_t ctas = (int64_t(b.num_seqs) * vecs + kThreads - 1) / kThreads;
    return launch_pdl(bounds_decode_kernel<KV>, dim3(unsigned(ctas)), dim3(kThreads), 0, stream, b, out, in, vecs,
                      head_dim);
  }
  // a request touches at most (max_query_len - 1) / B + 2 blocks
  const int64_t items = int64_t(b.num_seqs) * ((b.max_query_len - 1) / b.block_size + 2) * vecs;
  const int64_t ctas = std::min<int64_t>((items + kThreads - 1) / kThreads, 152 * 8);
  return launch_pdl(bounds_kernel<KV>, dim3(unsigned(ctas)), dim3(kThreads), 0, stream, b, out, in, vecs, head_dim);
}

}  // namespace

cudaError_t launch_block_bounds(const BatchArgs& b, void* bounds, const void* k_cache, int num_kv_heads, int head_dim,
                                pa_dtype cache_dtype, cudaStream_t stream) {
  return cache_dtype == PA_FP8_E4M3 ? launch<Fp8E4M3>(b, bounds, k_cache, num_kv_heads, head_dim, stream)
                                    : launch<__nv_bfloat16>(b, bounds, k_cache, num_kv_heads, head_dim, stream);
}

}  // namespace pa
