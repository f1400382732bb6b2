// pa_select_blocks: for each query token and KV head, the num_select blocks to attend, in
// ascending order: always the first `init` and the last `local` blocks of the token's context,
// then the blocks of the largest scores (equal scores: the lowest block first).
//
// Exact selection without a sort: the score that exactly as many reach as are wanted is found
// in two steps. A histogram in shared memory, 256 bins even over the range of a sample of the
// row's scores (any monotone binning is right; this one spreads them), gives the bin of the
// wanted score and its rank there; the bin's few scores are then compared with one another. A
// bin of more than 32 -- equal scores, or values of very different magnitudes -- is bisected by
// counting instead: 24 halvings of the value, then of bit patterns, so that it ends. Of scores
// equal to the border the lowest blocks are taken. The chosen blocks are written in order by
// ballots and prefix counts.
//
// Bound by instructions, not bytes: 1200 a row of 512 blocks (16384 rows 24.5 us, 1.5 TB/s; by
// bisection alone 35.6 us). A row's scores stay in registers, spread evenly over one warp up to
// 1024 blocks -- no barrier, many rows a CTA -- and over 8 or 32 warps beyond (512 rows of 2048:
// 7.1 us; one warp each 20.6); rows of more than 32768 blocks are read again from L2 by each
// pass. Blocks that are always selected or behind the context, and scores of -inf, are treated
// as NaN is: no comparison counts them. The scores are fetched before the row's request is
// known: only their use depends on it.
#include <cfloat>

#include "block_rows.cuh"

namespace pa {
namespace {

// Floats in order as signed integers, and back (adding 0 makes -0 the same as +0).
__device__ __forceinline__ int order_of(float x) {
  const int u = __float_as_int(x + 0.f);
  return u ^ ((u >> 31) & 0x7fffffff);
}
__device__ __forceinline__ float value_of(int k) { return __int_as_float(k ^ ((k >> 31) & 0x7fffffff)) + 0.f; }

// Minimum and maximum that keep a NaN.
__device__ __forceinline__ float min_nan(float a, float b) {
  float d;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

constexpr int kRowsPerCta = 4;  // of one warp each
constexpr int kBins = 256;

// WARPS warps per row, PER scores per lane (0: read from global memory each time).
template <int WARPS, int PER>
__global__ void __launch_bounds__(WARPS == 1 ? kRowsPerCta * 32 : WARPS * 32)
    select_blocks_kernel(const __grid_constant__ BatchArgs b, int32_t* block_idx, int num_select,
                         const float* scores, int width, int Hkv, int init, int local, int rows) {
  constexpr bool kReload = PER == 0;
  constexpr int kGroup = 4;  // scores handled without a test of their number
  static_assert(PER % kGroup == 0, "whole groups");
  constexpr int kRows = WARPS == 1 ? kRowsPerCta : 1;
  __shared__ __align__(16) int hist_all[kRows][kBins];
  __shared__ float cand_all[kRows][32];
  __shared__ int ncand_all[kRows];
  __shared__ int sums[2][WARPS], part_a[WARPS], part_b[WARPS];
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31, warp = WARPS == 1 ? 0 : threadIdx.x >> 5;  // the warp's part of the row
  const int slot = WARPS == 1 ? threadIdx.x >> 5 : 0;
  int* hist = hist_all[slot];
  float* cand = cand_all[slot];
  const int row = WARPS == 1 ? int(blockIdx.x) * kRowsPerCta + (threadIdx.x >> 5) : int(blockIdx.x);
  if (row >= rows) return;
  const float* src = scores + int64_t(row) * width;
  // warp w holds blocks [seg, seg + 32 per), lane l block seg + 32 j + l as its score j
  const int per = (width + WARPS * 32 - 1) / (WARPS * 32), seg = warp * per * 32;
  float x[kReload ? 1 : PER];
  if constexpr (!kReload) {
    const int end = min(width, seg + per * 32);
#pragma unroll
    for (int j = 0; j < PER; ++j) x[j] = seg + j * 32 + lane < end ? __ldg(src + seg + j * 32 + lane) : 0.f;
  }
  const QueryRow qr = find_row(b, row / Hkv);
  if (qr.s < 0) return;
  const int last = qr.pos / b.block_size;
  if (last >= width) {
    if (lane == 0) raise_error(b.err, PA_DEVERR_SEQ_RANGE);
    return;
  }
  const int n = last + 1, end = min(n, seg + per * 32);
  int32_t* dst = block_idx + int64_t(row) * num_select;
  const int steps = (max(end - seg, 0) + 31) / 32;  // scores j >= steps are no blocks
  // always selected: blocks [0, head) and [tail, n); the scores that count are those between
  const int head = min(init, n), tail = max(n - local, head), forced = head + n - tail;
  const int from = head - seg, to = min(tail, end) - seg;  // within the warp's part
  // i: within the warp's part; NaN: not to be counted (outside, NaN or -inf)
  auto mask = [&](int i, float v) { return i >= from && i < to && v > -INFINITY ? v : NAN; };
  // calls f(j, score) for the warp's scores
  auto each = [&](auto f) {
    if constexpr (kReload) {
      for (int j = 0; j < steps; ++j) {
        const int i = j * 32 + lane;
        f(j, mask(i, seg + i < end ? __ldg(src + seg + i) : 0.f));
      }
    } else {
#pragma unroll
      for (int j0 = 0; j0 < PER; j0 += kGroup) {
        if (j0 < steps) {
#pragma unroll
          for (int j = j0; j < j0 + kGroup; ++j) f(j, x[j]);
        }
      }
    }
  };
  int flip = 0;
  auto row_sum = [&](int c) {  // over the row's warps; every thread gets it
    c = __reduce_add_sync(0xffffffffu, c);
    if constexpr (WARPS > 1) {
      if (lane == 0) sums[flip][warp] = c;
      __syncthreads();
      c = __reduce_add_sync(0xffffffffu, lane < WARPS ? sums[flip][lane] : 0);
      flip ^= 1;  // the other buffer next: no second barrier
    }
    return c;
  };
  auto count_ge = [&](float v) {
    int c = 0;
    each([&](int, float s) { c += s >= v; });
    return row_sum(c);
  };

  auto sync_row = [&]() {
    if constexpr (WARPS == 1)
      __syncwarp();
    else
      __syncthreads();
  };
  // smallest and largest over the row of what the lanes hold
  auto row_range = [&](float& lo, float& hi) {
    int a = __reduce_min_sync(0xffffffffu, order_of(lo)), z = __reduce_max_sync(0xffffffffu, order_of(hi));
    if constexpr (WARPS > 1) {
      if (lane == 0) part_a[warp] = a, part_b[warp] = z;
      __syncthreads();
      a = __reduce_min_sync(0xffffffffu, lane < WARPS ? part_a[lane] : 0x7fffffff);
      z = __reduce_max_sync(0xffffffffu, lane < WARPS ? part_b[lane] : int(0x80000000));
      __syncthreads();
    }
    lo = value_of(a);
    hi = value_of(z);
  };
  // ---- the range of a sample: up to kSample of each lane's scores
  constexpr int kSample = 8;
  float mn = INFINITY, mx = -INFINITY;
  auto sample = [&](float v) {
    const float w = v < INFINITY ? v : NAN;  // fmaxf and fminf pass NaN over
    mx = fmaxf(mx, w);
    mn = fminf(mn, w);
  };
  if constexpr (kReload) {
    for (int k = 0; k < min(kSample, steps); ++k) {
      const int i = int(int64_t(k) * steps / kSample) * 32 + lane;
      sample(mask(i, seg + i < end ? __ldg(src + seg + i) : 0.f));
    }
  } else {
#pragma unroll
    for (int j0 = 0; j0 < PER; j0 += kGroup) {
      if (j0 < steps) {
#pragma unroll
        for (int j = j0; j < j0 + kGroup; ++j) {
          x[j] = mask(j * 32 + lane, x[j]);
          if (j % (PER > kSample ? PER / kSample : 1) == 0) sample(x[j]);
        }
      }
    }
  }
  for (int i = (WARPS == 1 ? lane : int(threadIdx.x)); i < kBins / 4; i += WARPS * 32)
    reinterpret_cast<int4*>(hist)[i] = make_int4(0, 0, 0, 0);
  if (lane == 0 && warp == 0) ncand_all[slot] = 0;
  if (WARPS == 1) __syncwarp();
  row_range(mn, mx);  // (with several warps its barriers also order the zeroing)
  // ---- the histogram: bin 0 for what does not count, the scores in bins 1 (below the sample's
  // range) to 255 (above it)
  const float ratio = (kBins - 3) / (mx - mn);
  // (without a usable range a scale that keeps infinities and their order)
  const bool flat = !(ratio > 0.f && ratio < INFINITY) || !(fabsf(mn * ratio) < INFINITY);
  const float scale = flat ? 2e-38f : ratio, off = flat ? 1.f : 2.f - mn * ratio;
  auto bin_of = [&](float v) {
    return __float2int_rz(min_nan(max_nan(fmaf(v, scale, off), 1.f), float(kBins - 1)));  // NaN: 0
  };
  // the lane's bins, four to a word, so that the border bin's scores are found without another
  // computation of them
  uint32_t bins[kReload ? 1 : PER / 4];
  if constexpr (kReload) {
    each([&](int, float s) { atomicAdd(hist + bin_of(s), 1); });
  } else {
#pragma unroll
    for (int j0 = 0; j0 < PER; j0 += kGroup) {
      if (j0 < steps) {
#pragma unroll
        for (int j = j0; j < j0 + kGroup; j += 4) {
          uint32_t word = 0;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int bin = bin_of(x[j + e]);
            atomicAdd(hist + bin, 1);
            word |= uint32_t(bin) << (8 * e);
          }
          bins[j / 4] = word;
        }
      }
    }
  }
  // calls f(score) for the warp's scores in a bin
  auto each_in = [&](int bin, auto f) {
    if constexpr (kReload) {
      each([&](int, float s) {
        if (bin_of(s) == bin) f(s);
      });
    } else {
      const uint32_t want = uint32_t(bin) * 0x01010101u;
#pragma unroll
      for (int j0 = 0; j0 < PER; j0 += kGroup) {
        if (j0 < steps) {
#pragma unroll
          for (int j = j0; j < j0 + kGroup; j += 4) {
            const uint32_t d = bins[j / 4] ^ want;
            if ((d - 0x01010101u) & ~d & 0x80808080u) {  // a byte of d is 0
#pragma unroll
              for (int e = 0; e < 4; ++e)
                if (((d >> (8 * e)) & 0xffu) == 0) f(x[j + e]);
            }
          }
        }
      }
    }
  };
  sync_row();
  // lane l holds bins 255 - 8 l .. 248 - 8 l: from the top down
  int c[8], mine = 0;
  {
    const int4 u = reinterpret_cast<const int4*>(hist)[63 - 2 * lane], v = reinterpret_cast<const int4*>(hist)[62 - 2 * lane];
    c[0] = u.w, c[1] = u.z, c[2] = u.y, c[3] = u.x, c[4] = v.w, c[5] = v.z, c[6] = v.y, c[7] = v.x;
    if (lane == 31) c[7] = 0;  // bin 0
#pragma unroll
    for (int i = 0; i < 8; ++i) mine += c[i];
  }
  int upto = mine;  // scores in this lane's bins and above
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, upto, d);
    if (lane >= d) upto += y;
  }
  const int scored = __shfl_sync(0xffffffffu, upto, 31);  // scores above -inf
  // ---- the threshold: scores >= thr are selected, of those equal to it perhaps only the first
  const int need = min(num_select - forced, scored);  // init + local <= num_select
  float thr = NAN;  // none
  int ge = 0;       // scores >= thr
  if (need == scored && need > 0) {
    thr = -FLT_MAX;
    ge = scored;
  } else if (need > 0) {
    const int owner = __ffs(__ballot_sync(0xffffffffu, upto >= need)) - 1;
    int bin = 0, above = upto - mine, in_bin = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (in_bin == 0 && above + c[i] >= need) {
        bin = kBins - 1 - 8 * lane - i;
        in_bin = c[i];
      }
      if (in_bin == 0) above += c[i];
    }
    bin = __shfl_sync(0xffffffffu, bin, owner);
    above = __shfl_sync(0xffffffffu, above, owner);  // scores in the bins above
    in_bin = __shfl_sync(0xffffffffu, in_bin, owner);
    if (in_bin <= 32) {
      each_in(bin, [&](float s) { cand[atomicAdd(&ncand_all[slot], 1)] = s; });
      sync_row();
      // the (need - above)-th largest of them, by counting (in any order: only values matter)
      const float v = lane < in_bin ? cand[lane] : -INFINITY;
      const int rank = need - above;
      int more = 0, same = 0;
      for (int i = 0; i < in_bin; ++i) {
        const float o = __shfl_sync(0xffffffffu, v, i);
        more += o > v;
        same += o == v;
      }
      const int at = __ffs(__ballot_sync(0xffffffffu, lane < in_bin && more < rank && rank <= more + same)) - 1;
      thr = __shfl_sync(0xffffffffu, v, at);
      ge = above + __shfl_sync(0xffffffffu, more + same, at);
    } else {
      float hi = -INFINITY;
      thr = INFINITY;
      each_in(bin, [&](float s) {
        thr = fminf(thr, s);
        hi = fmaxf(hi, s);
      });
      row_range(thr, hi);
      ge = above + in_bin;  // scores >= thr, the bin's lowest
      const int at_max = count_ge(hi);
      if (at_max >= need) {
        thr = hi;
        ge = at_max;
      } else {  // at least `need` scores reach thr, fewer hi
        for (int it = 0; ge != need; ++it) {
          float mid = 0.5f * thr + 0.5f * hi;
          if (it >= 24 || !(mid > thr && mid < hi)) {
            const uint32_t lo = uint32_t(order_of(thr)), up = uint32_t(order_of(hi));
            mid = value_of(int(lo + (up - lo) / 2));
            if (!(mid > thr && mid < hi)) break;  // neighbours
          }
          const int reach = count_ge(mid);
          if (reach >= need) {
            thr = mid;
            ge = reach;
          } else {
            hi = mid;
          }
        }
      }
    }
  }
  // ---- the selected blocks, in order
  const unsigned below = (1u << lane) - 1u;
  // sum over the warps before this one, and over all
  auto before = [&](int mine, int* parts, int* all) {
    mine = __reduce_add_sync(0xffffffffu, mine);
    if constexpr (WARPS == 1) {
      *all = mine;
      return 0;
    } else {
      __syncthreads();  // earlier reads of parts
      if (lane == 0) parts[warp] = mine;
      __syncthreads();
      const int v = lane < WARPS ? parts[lane] : 0;
      *all = __reduce_add_sync(0xffffffffu, v);
      return __reduce_add_sync(0xffffffffu, lane < warp ? v : 0);
    }
  };
  int all;
  int32_t* out = dst + head;
  if (ge == need) {  // every score that reaches thr
    int at = 0;
    if constexpr (WARPS > 1) {
      int mine = 0;
      each([&](int, float s) { mine += s >= thr; });
      at = before(mine, part_a, &all);
    }
    each([&](int j, float s) {
      const unsigned m = __ballot_sync(0xffffffffu, s >= thr);
      if (s >= thr) out[at + __popc(m & below)] = seg + j * 32 + lane;
      at += __popc(m);
    });
  } else {  // equal scores at thr: the lowest blocks of them
    int gt = 0, eq = 0;
    each([&](int, float s) {
      gt += s > thr;
      eq += s == thr;
    });
    int gt_before = before(gt, part_a, &all);
    const int ties = need - all;
    int eq_before = before(eq, part_b, &all);
    each([&](int j, float s) {
      const unsigned mg = __ballot_sync(0xffffffffu, s > thr), me = __ballot_sync(0xffffffffu, s == thr);
      const int eq_rank = eq_before + __popc(me & below);
      if (s > thr || (s == thr && eq_rank < ties))
        out[gt_before + __popc(mg & below) + min(eq_rank, ties)] = seg + j * 32 + lane;
      gt_before += __popc(mg);
      eq_before += __popc(me);
    });
  }
  const int tid = warp * 32 + lane;
  for (int i = tid; i < head; i += WARPS * 32) dst[i] = i;
  for (int i = tail + tid; i < n; i += WARPS * 32) out[need + i - tail] = i;
  for (int i = need + forced + tid; i < num_select; i += WARPS * 32) dst[i] = -1;
}

template <int WARPS, int PER>
cudaError_t launch(const BatchArgs& b, int32_t* block_idx, int num_select, const float* scores, int width, int Hkv,
                   int init, int local, cudaStream_t stream) {
  const int64_t rows = int64_t(b.num_tokens) * Hkv;
  constexpr int per_cta = WARPS == 1 ? kRowsPerCta : 1;
  return launch_pdl(select_blocks_kernel<WARPS, PER>, dim3(unsigned((rows + per_cta - 1) / per_cta)),
                    dim3(WARPS == 1 ? kRowsPerCta * 32 : WARPS * 32), 0, stream, b, block_idx, num_select, scores, width,
                    Hkv, init, local, int(rows));
}

}  // namespace

cudaError_t launch_select_blocks(const BatchArgs& b, int32_t* block_idx, int num_select, const float* scores,
                                 int score_width, int num_kv_heads, int init_blocks, int local_blocks,
                                 cudaStream_t stream) {
  auto go = [&](auto f) { return f(b, block_idx, num_select, scores, score_width, num_kv_heads, init_blocks, local_blocks, stream); };
  if (score_width <= 256) return go(launch<1, 8>);
  if (score_width <= 512) return go(launch<1, 16>);
  if (score_width <= 768) return go(launch<1, 24>);
  if (score_width <= 1024) return go(launch<1, 32>);
  if (score_width <= 2048) return go(launch<8, 8>);
  if (score_width <= 4096) return go(launch<8, 16>);
  if (score_width <= 8192) return go(launch<8, 32>);
  if (score_width <= 32768) return go(launch<32, 32>);
  return go(launch<32, 0>);
}

}  // namespace pa
