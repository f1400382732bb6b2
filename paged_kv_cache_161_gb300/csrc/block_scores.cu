// pa_block_scores: for each query token, KV head and block of the request's context, an
// upper bound of the logits (before the softmax scale) of the head's query group:
//
//   score[t, g, b] = max_h sum_d max(q_hd lo_d, q_hd hi_d),   (lo, hi) = bounds of block b
//
// With q- = min(q, 0) and q+ = max(q, 0) the sum is one dot product of length 2 D,
// <[q-, q+], [lo, hi]>: a matrix product of the blocks' bounds (rows) with the query heads
// (columns), whose products of bf16 values are exact in fp32 and whose sums are fp32.
//
// Decode is bound by the bytes of the bounds (1/16 of the keys at 16 tokens a block and bf16):
// a warp loads 16 blocks of one KV head straight into MMA fragments -- the order of the
// product's terms is free, so a lane takes 16 consecutive bytes of a row as the k slots of two
// MMA steps, and no shared memory is needed. The 8 warps of a CTA take (tile, KV head) pairs in
// order, so the KV heads of a block, which are adjacent in memory, are read together.
#include "block_rows.cuh"
#include "mma.cuh"

namespace pa {
namespace {

constexpr int kWarps = 8;
constexpr int kPairs = 4;  // (tile, head) pairs a warp takes

__device__ __forceinline__ uint32_t bf16x2_neg_part(uint32_t x) {
  const __nv_bfloat162 z = __floats2bfloat162_rn(0.f, 0.f);
  const __nv_bfloat162 r = __hmin2_nan(*reinterpret_cast<const __nv_bfloat162*>(&x), z);
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t bf16x2_pos_part(uint32_t x) {
  const __nv_bfloat162 z = __floats2bfloat162_rn(0.f, 0.f);
  const __nv_bfloat162 r = __hmax2_nan(*reinterpret_cast<const __nv_bfloat162*>(&x), z);
  return *reinterpret_cast<const uint32_t*>(&r);
}

template <int D>
__global__ void __launch_bounds__(kWarps * 32, 2)
    block_scores_kernel(const __grid_constant__ BatchArgs b, float* __restrict__ scores, int width,
                        const __nv_bfloat16* __restrict__ q, const __nv_bfloat16* __restrict__ bounds, int Hkv, int G,
                        int ctas_per_seq) {
  constexpr int CH = D / 32;  // 32-element chunks of a row: 16 bytes a lane, two MMA steps
  griddep_wait();
  griddep_launch_dependents();
  const int s = blockIdx.x / ctas_per_seq, part = blockIdx.x % ctas_per_seq;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int q0 = __ldg(b.query_start_loc + s), q_len = __ldg(b.query_start_loc + s + 1) - q0;
  const int L = __ldg(b.seq_lens + s);
  if (q_len <= 0) return;
  if (q_len > L || L > int64_t(b.max_blocks_per_seq) * b.block_size || (L - 1) / b.block_size >= width) {
    if (threadIdx.x == 0) raise_error(b.err, PA_DEVERR_SEQ_RANGE);
    return;
  }
  const int tiles = (width + 15) / 16, blocks = (L - 1) / b.block_size + 1;
  const int32_t* table = b.block_table + int64_t(s) * b.max_blocks_per_seq;
  const int cols = q_len * G;  // column = token * G + query head of the group
  const float ninf = -INFINITY;

  for (int i = 0; i < kPairs; ++i) {
    const int64_t pair = (int64_t(part) * kPairs + i) * kWarps + warp;
    if (pair >= int64_t(tiles) * Hkv) return;
    const int tile = int(pair / Hkv), head = int(pair % Hkv);
    uint4 lo[2][CH], hi[2][CH];  // rows g and g + 8 of the tile
    bool have[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int blk = tile * 16 + g + 8 * r;
      int id = blk < blocks ? __ldg(table + blk) : -1;
      have[r] = id >= 0 && id < b.num_blocks;
      if (blk < blocks && !have[r]) raise_error(b.err, PA_DEVERR_BLOCK_RANGE);
      const __nv_bfloat16* row = bounds + (int64_t(have[r] ? id : 0) * Hkv + head) * 2 * D + t * 8;
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        lo[r][c] = have[r] ? __ldg(reinterpret_cast<const uint4*>(row + 32 * c)) : make_uint4(0, 0, 0, 0);
        hi[r][c] = have[r] ? __ldg(reinterpret_cast<const uint4*>(row + D + 32 * c)) : make_uint4(0, 0, 0, 0);
      }
    }
    for (int n0 = 0; n0 < cols; n0 += 8) {
      const int col = n0 + g;  // this lane's B column
      float acc[4] = {0.f, 0.f, 0.f, 0.f}, acc2[4] = {0.f, 0.f, 0.f, 0.f};
      const __nv_bfloat16* qp =
          q + ((int64_t(q0) + (col < cols ? col / G : 0)) * (Hkv * G) + head * G + (col < cols ? col % G : 0)) * D + t * 8;
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const uint4 u = col < cols ? __ldg(reinterpret_cast<const uint4*>(qp + 32 * c)) : make_uint4(0, 0, 0, 0);
        mma_16816(acc, lo[0][c].x, lo[1][c].x, lo[0][c].y, lo[1][c].y, bf16x2_neg_part(u.x), bf16x2_neg_part(u.y), false);
        mma_16816(acc2, hi[0][c].x, hi[1][c].x, hi[0][c].y, hi[1][c].y, bf16x2_pos_part(u.x), bf16x2_pos_part(u.y), false);
        mma_16816(acc, lo[0][c].z, lo[1][c].z, lo[0][c].w, lo[1][c].w, bf16x2_neg_part(u.z), bf16x2_neg_part(u.w), false);
        mma_16816(acc2, hi[0][c].z, hi[1][c].z, hi[0][c].w, hi[1][c].w, bf16x2_pos_part(u.z), bf16x2_pos_part(u.w), false);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[e] += acc2[e];
      // accumulators: rows g (e 0, 1) and g + 8 (e 2, 3), columns n0 + 2t and n0 + 2t + 1
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int blk = tile * 16 + g + 8 * r;
        float x = acc[2 * r], y = acc[2 * r + 1];
        auto put = [&](int column, float v) {
          if (column >= cols || blk >= width) return;
          const int j = column / G, last = (L - q_len + j) / b.block_size;
          scores[((int64_t(q0) + j) * Hkv + head) * width + blk] = blk <= last && have[r] ? v : ninf;
        };
        if (G == 1) {
          put(n0 + 2 * t, x);
          put(n0 + 2 * t + 1, y);
        } else {
          float m = fmaxf(x, y);
          if (G >= 4) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
          if (G >= 8) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
          if ((2 * t) % G == 0) put(n0 + 2 * t, m);
        }
      }
    }
  }
}

}  // namespace

cudaError_t launch_block_scores(const BatchArgs& b, float* scores, int score_width, const void* q, const void* bounds,
                                int num_heads, int num_kv_heads, int head_dim, cudaStream_t stream) {
  const int64_t pairs = int64_t((score_width + 15) / 16) * num_kv_heads;
  const int ctas_per_seq = int((pairs + kWarps * kPairs - 1) / (kWarps * kPairs));
  const dim3 grid(unsigned(int64_t(b.num_seqs) * ctas_per_seq));
  const auto* qp = static_cast<const __nv_bfloat16*>(q);
  const auto* bp = static_cast<const __nv_bfloat16*>(bounds);
  const int G = num_heads / num_kv_heads;
  if (head_dim == 64)
    return launch_pdl(block_scores_kernel<64>, grid, dim3(kWarps * 32), 0, stream, b, scores, score_width, qp, bp,
                      num_kv_heads, G, ctas_per_seq);
  return launch_pdl(block_scores_kernel<128>, grid, dim3(kWarps * 32), 0, stream, b, scores, score_width, qp, bp,
                    num_kv_heads, G, ctas_per_seq);
}

}  // namespace pa
