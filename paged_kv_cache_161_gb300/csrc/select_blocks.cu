// pa_select_blocks: for each query token and KV head, the num_select blocks to attend, in
// ascending order: always the first `init` and the last `local` blocks of the token's context,
// then the blocks of the largest scores (equal scores: the lowest block first).
//
// Exact selection without a sort: scores become unsigned keys of the same order, and a
// bisection finds the largest threshold that at least `need` keys reach, by counting. Each
// step halves the interval of values (not of bit patterns: the scores are spread evenly
// enough that about ten steps isolate the threshold among a thousand), and ends as soon as
// exactly `need` keys reach it; bit patterns are halved when values no longer separate, so
// ties end it too. The chosen blocks are then written in order by ballots and prefix counts.
//
// Bound by instructions, not bytes (one read of the scores, then a compare and an add per key
// and step): a row's keys stay in registers, spread over one warp up to 1024 blocks and over
// 4, 16 or 32 warps beyond; rows of more than 32768 blocks are read again from L2 each step.
#include "block_rows.cuh"

namespace pa {
namespace {

constexpr int kPer = 32;  // keys per lane

// Order-preserving: larger score, larger key. 0: never selected (-inf, NaN, not a block of the
// context); 0xffffffff: always selected. -0 and +0 are one value.
__device__ __forceinline__ uint32_t key_of(float x) {
  if (!(x > -INFINITY)) return 0u;
  const uint32_t u = __float_as_uint(x + 0.f);
  return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t k) {
  return __uint_as_float((k >> 31) ? k ^ 0x80000000u : ~k);
}

// WARPS warps per row; RELOAD: keys are computed from global memory each time.
template <int WARPS, bool RELOAD>
__global__ void __launch_bounds__(WARPS == 1 ? 128 : WARPS * 32)
    select_blocks_kernel(const __grid_constant__ BatchArgs b, int32_t* __restrict__ block_idx, int num_select,
                         const float* __restrict__ scores, int width, int Hkv, int init, int local, int64_t rows) {
  constexpr int kRowsPerCta = WARPS == 1 ? 4 : 1;
  __shared__ int sums[2][WARPS == 1 ? 1 : 32];
  __shared__ int gt_of[WARPS == 1 ? 1 : 32], eq_of[WARPS == 1 ? 1 : 32];
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int wr = WARPS == 1 ? 0 : warp;  // the warp's part of the row
  const int64_t row = int64_t(blockIdx.x) * kRowsPerCta + (WARPS == 1 ? warp : 0);
  if (row >= rows) return;
  const QueryRow qr = find_row(b, int(row / Hkv));
  if (qr.s < 0) return;
  const int last = qr.pos / b.block_size;
  if (last >= width) {
    if (lane == 0) raise_error(b.err, PA_DEVERR_SEQ_RANGE);
    return;
  }
  const int n = last + 1;
  const float* src = scores + row * width;
  int32_t* dst = block_idx + row * num_select;
  // warp wr holds blocks [seg, seg + per * 32), lane l block seg + 32 j + l
  const int per = RELOAD ? (n + WARPS * 32 - 1) / (WARPS * 32) : kPer;
  const int seg = wr * per * 32;
  auto fetch = [&](int j) -> uint32_t {
    const int i = seg + j * 32 + lane;
    if (i >= n) return 0u;
    if (i < init || i > last - local) return 0xffffffffu;
    return key_of(__ldg(src + i));
  };
  uint32_t keys[RELOAD ? 1 : kPer];
  const int steps = min(per, (max(n - seg, 0) + 31) / 32);  // j beyond holds no block
  if constexpr (!RELOAD) {
#pragma unroll
    for (int j = 0; j < kPer; ++j) keys[j] = fetch(j);
  }
  // calls f(j, key) for the warp's keys
  auto each = [&](auto f) {
    if constexpr (RELOAD) {
      for (int j = 0; j < steps; ++j) f(j, fetch(j));
    } else {
#pragma unroll
      for (int j = 0; j < kPer; ++j)
        if (j < steps) f(j, keys[j]);
    }
  };
  int flip = 0;
  auto row_sum = [&](int x) {  // over the row's warps; every thread gets it
    x = __reduce_add_sync(0xffffffffu, x);
    if constexpr (WARPS > 1) {
      if (lane == 0) sums[flip][warp] = x;
      __syncthreads();
      x = __reduce_add_sync(0xffffffffu, lane < WARPS ? sums[flip][lane] : 0);
      flip ^= 1;
    }
    return x;
  };
  auto count_ge = [&](uint32_t k) {
    int c = 0;
    each([&](int, uint32_t key) { c += key >= k; });
    return row_sum(c);
  };

  const int eligible = count_ge(1u);
  const int need = min(num_select, eligible);
  uint32_t thr = 1u;
  if (need < eligible) {
    // keys: at least `need` reach lo, fewer reach hi
    uint32_t lo = 1u, hi = 0xffffffffu;
    if (count_ge(hi) >= need) {  // the always-selected alone (init + local <= num_select)
      thr = hi;
    } else {
      uint32_t mn = 0xffffffffu, mx = 0u;  // of the scored keys
      each([&](int, uint32_t key) {
        if (key != 0u && key != 0xffffffffu) {
          mn = min(mn, key);
          mx = max(mx, key);
        }
      });
      mn = __reduce_min_sync(0xffffffffu, mn);
      mx = __reduce_max_sync(0xffffffffu, mx);
      if constexpr (WARPS > 1) {
        __syncthreads();
        if (lane == 0) gt_of[warp] = int(mn), eq_of[warp] = int(mx);
        __syncthreads();
        mn = __reduce_min_sync(0xffffffffu, lane < WARPS ? uint32_t(gt_of[lane]) : 0xffffffffu);
        mx = __reduce_max_sync(0xffffffffu, lane < WARPS ? uint32_t(eq_of[lane]) : 0u);
        __syncthreads();
      }
      lo = mn;
      hi = mx + 1;  // mx < 0xffffffff
      for (int it = 0; hi - lo > 1; ++it) {
        uint32_t mid = lo + (hi - lo) / 2;
        if (it < 24) {  // halve the values; infinities and neighbours fall back to the patterns
          const float v = 0.5f * value_of(lo) + 0.5f * value_of(hi - 1);
          const uint32_t k = key_of(v);
          if (k > lo && k < hi) mid = k;
        }
        const int c = count_ge(mid);
        if (c >= need) {
          lo = mid;
          if (c == need) break;
        } else {
          hi = mid;
        }
      }
      thr = lo;
    }
  }
  // Selected: keys > thr, and the first `ties` keys equal to it.
  int gt = 0, eq = 0;
  each([&](int, uint32_t key) {
    gt += key > thr;
    eq += key == thr;
  });
  gt = __reduce_add_sync(0xffffffffu, gt);
  eq = __reduce_add_sync(0xffffffffu, eq);
  int gt_before = 0, eq_before = 0, gt_all = gt;
  if constexpr (WARPS > 1) {
    __syncthreads();
    if (lane == 0) gt_of[warp] = gt, eq_of[warp] = eq;
    __syncthreads();
    const int a = lane < WARPS ? gt_of[lane] : 0, e = lane < WARPS ? eq_of[lane] : 0;
    gt_all = __reduce_add_sync(0xffffffffu, a);
    gt_before = __reduce_add_sync(0xffffffffu, lane < warp ? a : 0);
    eq_before = __reduce_add_sync(0xffffffffu, lane < warp ? e : 0);
  }
  const int ties = need - gt_all;
  const unsigned below = (1u << lane) - 1u;
  each([&](int j, uint32_t key) {
    const unsigned mg = __ballot_sync(0xffffffffu, key > thr), me = __ballot_sync(0xffffffffu, key == thr);
    const int eq_rank = eq_before + __popc(me & below);
    if (key > thr || (key == thr && eq_rank < ties))
      dst[gt_before + __popc(mg & below) + min(eq_rank, ties)] = seg + j * 32 + lane;
    gt_before += __popc(mg);
    eq_before += __popc(me);
  });
  for (int i = need + wr * 32 + lane; i < num_select; i += WARPS * 32) dst[i] = -1;
}

template <int WARPS, bool RELOAD>
cudaError_t launch(const BatchArgs& b, int32_t* block_idx, int num_select, const float* scores, int width, int Hkv,
                   int init, int local, cudaStream_t stream) {
  const int64_t rows = int64_t(b.num_tokens) * Hkv;
  constexpr int per_cta = WARPS == 1 ? 4 : 1;
  return launch_pdl(select_blocks_kernel<WARPS, RELOAD>, dim3(unsigned((rows + per_cta - 1) / per_cta)),
                    dim3(WARPS == 1 ? 128 : WARPS * 32), 0, stream, b, block_idx, num_select, scores, width, Hkv, init,
                    local, rows);
}

}  // namespace

cudaError_t launch_select_blocks(const BatchArgs& b, int32_t* block_idx, int num_select, const float* scores,
                                 int score_width, int num_kv_heads, int init_blocks, int local_blocks,
                                 cudaStream_t stream) {
  auto go = [&](auto f) { return f(b, block_idx, num_select, scores, score_width, num_kv_heads, init_blocks, local_blocks, stream); };
  if (score_width <= 1 * 32 * kPer) return go(launch<1, false>);
  if (score_width <= 4 * 32 * kPer) return go(launch<4, false>);
  if (score_width <= 16 * 32 * kPer) return go(launch<16, false>);
  if (score_width <= 32 * 32 * kPer) return go(launch<32, false>);
  return go(launch<32, true>);
}

}  // namespace pa
