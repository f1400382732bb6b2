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
// Bound by the bytes of the touched blocks' keys. A warp owns 32 consecutive 16-byte columns of
// a block and keeps the packed minimum and maximum in registers (a warp's loads: 512
// consecutive bytes of a row, 8 rows in flight). Its block a warp finds by a 32-way search: no
// scan over the requests, no barrier before the first load. Where that leaves SMs empty -- a
// decode step over wide blocks -- up to 8 warps of a CTA take a block's rows between them and
// merge through shared memory; 16 prompts of 8192 tokens in blocks of 64 E4M3 keys take 26.4 us
// with one warp a column chunk (5.4 TB/s), 28.7 with two, 30.1 with four.
#include "block_rows.cuh"

namespace pa {
namespace {

constexpr int kWarps = 8;
constexpr int kBatch = 8;      // rows loaded before the first is used
constexpr int kWarpRows = 16;  // a block's rows are shared only in parts of this many

template <typename KV>
struct Column;
// Packed min / max over the rows of a 16-byte column.
template <>
struct Column<__nv_bfloat16> {
  __nv_bfloat162 lo[4], hi[4];
  __device__ __forceinline__ void merge(const Column& o) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      lo[i] = __hmin2_nan(lo[i], o.lo[i]);
      hi[i] = __hmax2_nan(hi[i], o.hi[i]);
    }
  }
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
  __device__ __forceinline__ void merge(const Column& o) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      lo[i] = __hmin2_nan(lo[i], o.lo[i]);
      hi[i] = __hmax2_nan(hi[i], o.hi[i]);
    }
  }
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

// The first place of request s among the batch's blocks: no scan is needed, since 2 s + (tokens
// before it) / B leaves room for every request's partial first and last block. A decode batch
// needs one place a request.
__device__ __forceinline__ int64_t place(const BatchArgs& b, int s) {
  return b.max_query_len <= 1 ? s : int64_t(__ldg(b.query_start_loc + s)) / b.block_size + 2 * int64_t(s);
}

// `share` warps of the CTA per (block, 32 columns).
template <typename KV>
__global__ void __launch_bounds__(kWarps * 32, 4) block_bounds_kernel(const __grid_constant__ BatchArgs b,
                                                                  __nv_bfloat16* bounds, const uint4* cache, int vecs,
                                                                  int head_dim, int share, int64_t items) {
  __shared__ Column<KV> merged[kWarps][32];
  griddep_wait();
  griddep_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // more tokens than announced: blocks of the last requests have no place in the grid
  if (b.max_query_len > 1 && blockIdx.x == 0 && threadIdx.x == 0 && __ldg(b.query_start_loc + b.num_seqs) > b.num_tokens)
    raise_error(b.err, PA_DEVERR_SEQ_RANGE);
  const int chunks = (vecs + 31) / 32, part = warp % share;
  const int64_t item = int64_t(blockIdx.x) * (kWarps / share) + warp / share;
  bool have = item < items;
  const int64_t at = item / chunks;
  const int vec = int(item - at * chunks) * 32 + lane;
  // ---- the request: the last whose first place is <= at
  int s = 0;
  if (b.max_query_len <= 1) {
    s = int(at);
  } else {
    int n = b.num_seqs;
    while (n > 1) {
      const int step = (n + 31) / 32, probe = s + lane * step;
      const unsigned m = __ballot_sync(0xffffffffu, probe < s + n && place(b, probe) <= at);
      const int k = m ? 31 - __clz(m) : 0, next = s + k * step;
      n = min(step, s + n - next);
      s = next;
    }
  }
  have = have && s < b.num_seqs;
  Column<KV> col;
  int id = -1, rows = 0;
  if (have) {
    const Touched w = touched(b, s);
    const int64_t i = at - place(b, s);
    have = i >= 0 && i < w.count;
    if (b.max_query_len <= 1 && w.count > 1) raise_error(b.err, PA_DEVERR_SEQ_RANGE);  // more queries than announced
    if (have) {
      const int blk = w.first + int(i);
      id = __ldg(b.block_table + int64_t(s) * b.max_blocks_per_seq + blk);
      rows = min(b.block_size, w.len - blk * b.block_size);
      if (id < 0 || id >= b.num_blocks) {
        if (lane == 0) raise_error(b.err, PA_DEVERR_BLOCK_RANGE);
        have = false;
      }
    }
  }
  // ---- this warp's rows: batches part, part + share, ..
  have = have && vec < vecs;
  bool any = false;
  if (have) {
    const uint4* src = cache + int64_t(id) * b.block_size * vecs + vec;
    for (int r0 = part * kBatch; r0 < rows; r0 += share * kBatch) {
      uint4 u[kBatch];
      const uint4* at_row = src + int64_t(r0) * vecs;
      if (r0 + kBatch <= rows) {
#pragma unroll
        for (int k = 0; k < kBatch; ++k) u[k] = __ldg(at_row + k * vecs);
      } else {  // past the last row: that row again, harmless
#pragma unroll
        for (int k = 0; k < kBatch; ++k) u[k] = __ldg(at_row + min(k, rows - 1 - r0) * vecs);
      }
#pragma unroll
      for (int k = 0; k < kBatch; ++k) col.add(u[k], !any && k == 0);
      any = true;
    }
  }
  if (share > 1) {
    if (any && part > 0) merged[warp][lane] = col;
    __syncthreads();
    if (part > 0) return;
    for (int k = 1; k < share && k * kBatch < rows; ++k)
      if (any) col.merge(merged[warp + k][lane]);
  }
  if (!any) return;
  constexpr int kElems = 16 / sizeof(KV);
  const int e = vec * kElems, head = e / head_dim, d = e % head_dim;
  __nv_bfloat16* dst = bounds + (int64_t(id) * (vecs * kElems / head_dim) + head) * 2 * head_dim + d;
  col.store(dst, dst + head_dim);
}

template <typename KV>
cudaError_t launch(const BatchArgs& b, void* bounds, const void* k_cache, int num_kv_heads, int head_dim,
                   cudaStream_t stream) {
  const int vecs = num_kv_heads * head_dim * int(sizeof(KV)) / 16, chunks = (vecs + 31) / 32;
  const int64_t places = b.max_query_len <= 1 ? b.num_seqs : int64_t(b.num_tokens) / b.block_size + 2 * int64_t(b.num_seqs);
  const int64_t items = places * chunks;
  int share = 1;
  while (share < kWarps && share * kWarpRows < b.block_size && items * share < 152 * 16) share *= 2;
  const int64_t per_cta = kWarps / share, ctas = (items + per_cta - 1) / per_cta;
  if (ctas > 0x7fffffff) return cudaErrorInvalidConfiguration;
  return launch_pdl(block_bounds_kernel<KV>, dim3(unsigned(ctas)), dim3(kWarps * 32), 0, stream, b,
                    static_cast<__nv_bfloat16*>(bounds), static_cast<const uint4*>(k_cache), vecs, head_dim, share, items);
}

}  // namespace

cudaError_t launch_block_bounds(const BatchArgs& b, void* bounds, const void* k_cache, int num_kv_heads, int head_dim,
                                pa_dtype cache_dtype, cudaStream_t stream) {
  return cache_dtype == PA_FP8_E4M3 ? launch<Fp8E4M3>(b, bounds, k_cache, num_kv_heads, head_dim, stream)
                                    : launch<__nv_bfloat16>(b, bounds, k_cache, num_kv_heads, head_dim, stream);
}

}  // namespace pa
