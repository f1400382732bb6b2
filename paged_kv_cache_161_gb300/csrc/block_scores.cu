// pa_block_scores: for each query token, KV head and block of the request's context, an
// upper bound of the logits (before the softmax scale) of the head's query group:
//
//   score[t, g, b] = max_h sum_d max(q_hd lo_d, q_hd hi_d),   (lo, hi) = bounds of block b
//
// With q- = min(q, 0) and q+ = max(q, 0) the sum is one dot product of length 2 D,
// <[q-, q+], [lo, hi]>: a matrix product of the blocks' bounds (rows) with the query heads
// (columns), whose products of bf16 values are exact in fp32 and whose sums are fp32.
//
// Few query rows (decode, drafts): bound by the bytes of the bounds (1/16 of the keys at 16
// tokens a block and bf16). A warp streams tiles of 16 blocks of one KV head through a private
// ring of kRing stages of 16-byte asynchronous copies, as pa_attention_sparse streams keys
// (loads straight into MMA fragments, in bursts of 8 KB a warp, reached 0.81 of the copy rate).
// Many query rows (prompt chunks): a tcgen05 product, below.
#include "block_rows.cuh"
#include "mma.cuh"
#include "tcgen05.cuh"

namespace pa {
namespace {

constexpr int kWarps = 4;
// Stages of a warp's ring: 64 x 32768 positions, 8 heads: 85.5 us with 2 (three CTAs a SM), 99.8
// with 3 (two): more warps hide the products' latency better than deeper rings.
constexpr int kRing = 2;
constexpr int kTiles = 8;  // tiles of 16 blocks a warp takes

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool real) {
  const int n = real ? 16 : 0;  // 0: nothing is read, 16 zero bytes are written
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

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

// Requests with more query rows than this (columns of the product) go to the tcgen05 kernel.
constexpr int kMaxFewCols = 32;
__device__ __forceinline__ bool is_chunk(int q_len, int G) { return int64_t(q_len) * G > kMaxFewCols; }
__device__ __forceinline__ bool fits(const BatchArgs& b, int q0, int q_len, int L, int width) {
  return q0 >= 0 && q0 <= b.num_tokens - q_len && q_len <= L && L <= int64_t(b.max_blocks_per_seq) * b.block_size &&
         (L - 1) / b.block_size < width;
}

// ---------------------------------------------------------------- few query rows: mma.sync
// How a CTA's warps share the KV heads and tiles: with at least kWarps heads each warp has its
// own head (kWarps consecutive ones a CTA: adjacent in memory); with fewer, `lanes` warps per
// head take every `lanes`-th tile.
struct Sharing {
  int groups, lanes, tiles;  // head groups, warps per head, tiles per CTA and head
};
__host__ __device__ inline Sharing sharing(int Hkv) {
  if (Hkv >= kWarps) return {(Hkv + kWarps - 1) / kWarps, 1, kTiles};
  return {1, kWarps / Hkv, kTiles * (kWarps / Hkv)};
}

template <int D>
__global__ void __launch_bounds__(kWarps * 32)
    block_scores_kernel(const __grid_constant__ BatchArgs b, float* scores, int width,
                        const __nv_bfloat16* q, const __nv_bfloat16* bounds, int Hkv, int G,
                        int ctas_per_seq, bool after_chunks) {
  constexpr int KC = D / 16;            // MMA steps of lo (and of hi)
  constexpr int RB = 4 * D;             // bytes of a block's row: lo, hi
  constexpr int PPR = RB / 16;          // 16-byte pieces of it
  constexpr int kStage = 16 * RB;
  extern __shared__ __align__(128) unsigned char smem[];
  // Behind the chunk kernel of the same call, which this grid needs nothing of: it starts once
  // every CTA of that kernel has (each of which then has waited for the grids before), runs
  // beside its last ones, and waits for it only before it ends, so that what follows this grid
  // follows both.
  struct Ending {
    bool wait;
    __device__ ~Ending() {
      if (wait) griddep_wait();
    }
  } ending{after_chunks};
  if (!after_chunks) griddep_wait();
  griddep_launch_dependents();
  const Sharing sh = sharing(Hkv);
  const int s = blockIdx.x / ctas_per_seq, part = blockIdx.x % ctas_per_seq;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int q0 = __ldg(b.query_start_loc + s), q_len = __ldg(b.query_start_loc + s + 1) - q0;
  const int L = __ldg(b.seq_lens + s);
  if (q_len <= 0) return;
  if (is_chunk(q_len, G)) {  // the other kernel's, which max_query_len must have called for
    if (!after_chunks && threadIdx.x == 0) raise_error(b.err, PA_DEVERR_SEQ_RANGE);
    return;
  }
  if (!fits(b, q0, q_len, L, width)) {
    if (threadIdx.x == 0) raise_error(b.err, PA_DEVERR_SEQ_RANGE);
    return;
  }
  const int tiles = (width + 15) / 16, blocks = (L - 1) / b.block_size + 1;
  const int32_t* table = b.block_table + int64_t(s) * b.max_blocks_per_seq;
  const int lg = __ffs(G) - 1, cols = q_len << lg;  // column = token * G + query head of the group

  // ---- this warp's head and tiles first_tile, first_tile + sh.lanes, ..
  const int head = sh.lanes == 1 ? part % sh.groups * kWarps + warp : warp % Hkv;
  const int lane_of = sh.lanes == 1 ? 0 : warp / Hkv;
  const int tile0 = part / sh.groups * sh.tiles;
  const int first_tile = tile0 + lane_of, end_tile = min(tile0 + sh.tiles, tiles);
  if (head >= Hkv || lane_of >= sh.lanes || first_tile >= end_tile) return;
  const int n = (end_tile - first_tile + sh.lanes - 1) / sh.lanes;
  // lane l < 16 looks up row l's block of a tile one tile ahead of its copies
  auto look_up = [&](int i) {
    const int blk = (first_tile + i * sh.lanes) * 16 + (lane & 15);
    if (i >= n || blk >= blocks) return -1;
    const int id = __ldg(table + blk);
    if (id >= 0 && id < b.num_blocks) return id;
    raise_error(b.err, PA_DEVERR_BLOCK_RANGE);
    return -1;
  };
  const uint32_t ring = smem_u32(smem) + uint32_t(warp * kRing * kStage);
  int next = look_up(0);
  uint32_t have_ring[kRing];  // bit r: row r of the tile in that stage exists
  auto issue = [&](int i) {
    const int my = next;
    next = look_up(i + 1);
    const unsigned have = __ballot_sync(0xffffffffu, my >= 0) & 0xffffu;
#pragma unroll
    for (int st = 0; st < kRing; ++st)
      if (i % kRing == st) have_ring[st] = have;
    if (have) {
      const uint32_t dst = ring + uint32_t(i % kRing * kStage);
#pragma unroll
      for (int k = 0; k < 16 * PPR / 32; ++k) {
        const int r = (k * 32 + lane) / PPR, piece = (k * 32 + lane) % PPR;
        const int id = __shfl_sync(0xffffffffu, my, r);
        const char* src = reinterpret_cast<const char*>(bounds) + (int64_t(max(id, 0)) * Hkv + head) * RB + piece * 16;
        cp_async16(dst + uint32_t(r * RB + ((piece ^ (r & 7)) << 4)), src, id >= 0);
      }
    }
    cp_async_commit();  // one group a tile, empty ones too
  };

  // ---- the columns' values as B fragments (k slots 2t, 2t + 1 and 2t + 8, 2t + 9 of column g)
  uint32_t qneg[KC][2], qpos[KC][2];  // of q- and q+
  auto load_q = [&](int n0) {
    const int col = n0 + g;
    const bool in = col < cols;
    const __nv_bfloat16* row =
        q + ((int64_t(q0) + (in ? col >> lg : 0)) * (Hkv << lg) + (head << lg) + (in ? col & (G - 1) : 0)) * D;
#pragma unroll
    for (int kc = 0; kc < KC; ++kc) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t x = in ? __ldg(reinterpret_cast<const uint32_t*>(row + 16 * kc + 8 * h + 2 * t)) : 0u;
        qneg[kc][h] = bf16x2_neg_part(x);
        qpos[kc][h] = bf16x2_pos_part(x);
      }
    }
  };
#pragma unroll
  for (int i = 0; i < kRing - 1; ++i) issue(i);
  load_q(0);
  const int64_t pitch = int64_t(Hkv) * width;  // between tokens
  float* out = scores + (int64_t(q0) * Hkv + head) * width;
  const int pos0 = L - q_len;
  for (int i = 0; i < n; ++i) {
    issue(i + kRing - 1);
    cp_async_wait<kRing - 1>();
    __syncwarp();  // every lane's copies of tile i have landed
    uint32_t have = 0;
#pragma unroll
    for (int st = 0; st < kRing; ++st)
      if (i % kRing == st) have = have_ring[st];
    const int tile = first_tile + i * sh.lanes;
    const uint32_t at = ring + uint32_t(i % kRing * kStage);
    for (int n0 = 0; n0 < cols; n0 += 8) {
      if (cols > 8) load_q(n0);
      float acc[4][4] = {};  // four chains of MMAs
      if (have) {
        const int row = lane & 15, half = lane >> 4;  // ldmatrix: rows 0-7, 8-15 of k 0-7, then of k 8-15
#pragma unroll
        for (int kc = 0; kc < KC; ++kc) {
          uint32_t a0, a1, a2, a3;
          const int piece = 2 * kc + half;
          ldsm_x4(at + uint32_t(row * RB + ((piece ^ (row & 7)) << 4)), a0, a1, a2, a3);
          mma_16816(acc[kc & 1], a0, a1, a2, a3, qneg[kc][0], qneg[kc][1], false);
          ldsm_x4(at + uint32_t(row * RB + (((piece + 2 * KC) ^ (row & 7)) << 4)), a0, a1, a2, a3);
          mma_16816(acc[2 + (kc & 1)], a0, a1, a2, a3, qpos[kc][0], qpos[kc][1], false);
        }
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[0][e] += acc[1][e] + acc[2][e] + acc[3][e];
      // accumulators: rows g (e 0, 1) and g + 8 (e 2, 3), columns n0 + 2t and n0 + 2t + 1
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int blk = tile * 16 + g + 8 * r;
        const bool is = (have >> (g + 8 * r)) & 1u;
        auto put = [&](int column, float v) {
          if (column >= cols || blk >= width) return;
          const int j = column >> lg;
          out[j * pitch + blk] = is && blk * b.block_size <= pos0 + j ? v : -INFINITY;
        };
        const float x = acc[0][2 * r], y = acc[0][2 * r + 1];
        if (G == 1) {
          put(n0 + 2 * t, x);
          put(n0 + 2 * t + 1, y);
        } else {
          float m = fmaxf(x, y);
          if (G >= 4) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
          if (G >= 8) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
          if (((2 * t) & (G - 1)) == 0) put(n0 + 2 * t, m);
        }
      }
    }
    __syncwarp();  // the stage may be refilled
  }
  cp_async_wait<0>();
}

template <int D>
cudaError_t launch_few(const BatchArgs& b, float* scores, int width, const __nv_bfloat16* q,
                       const __nv_bfloat16* bounds, int Hkv, int G, bool after_chunks, cudaStream_t stream) {
  constexpr auto kern = block_scores_kernel<D>;
  constexpr size_t smem = size_t(kWarps) * kRing * 16 * 4 * D;
  const cudaError_t e = ensure_smem<kern>(smem);
  if (e != cudaSuccess) return e;
  const Sharing sh = sharing(Hkv);
  const int per_seq = ((width + 15) / 16 + sh.tiles - 1) / sh.tiles * sh.groups;
  return launch_pdl(kern, dim3(unsigned(int64_t(b.num_seqs) * per_seq)), dim3(kWarps * 32), smem, stream, b, scores,
                    width, q, bounds, Hkv, G, per_seq, after_chunks);
}

// ---------------------------------------------------------------- chunks: tcgen05
// Requests of many query rows: a matrix product of 128 blocks (rows of TMEM) with up to 256
// columns (query heads of consecutive tokens of one KV head), K = 2 D.
//
// A CTA keeps its columns' [q-, q+] in shared memory -- split from q once, 128 KB at D = 128 --
// and streams the request's blocks past them: 128 rows of lo, then 128 of hi, gathered by 16-byte
// asynchronous copies (a block's row is 2 D contiguous bytes per half) into a ring of 3 stages.
// With 256 columns a tile's copies (64 KB at D = 128, arriving at about 30 bytes a clock and SM) and
// its MMAs (2050 clocks at the measured bf16 rate) take about the same time; with 128 the copies
// would take twice the MMAs'. Blocks are the M side so that the maximum over a group's
// heads runs over a thread's own accumulator columns, and 32 lanes store 32 consecutive blocks.
// Two accumulators of 256 columns: the epilogue of one tile runs beside the next tile's MMAs.
// Clock stamps of four 512-token chunks against 8192 positions (28.5 us): a CTA's 26 k clocks are 6 k
// until its request is known and its query loads are under way, 6 k more until the first tile's
// products are there, then a tile every 2.6 to 3.1 k; 256 such CTAs run on 152 SMs as two waves.
// Warps 0-7: the columns' split, then the epilogue (TMEM lanes 32 (w % 4) .., every second 32
// columns), 8-11: producers, 12: MMA issue.
constexpr int kChunkCols = 256;
constexpr int kTileBlocks = 128;
constexpr int kStages = 3;
constexpr int kEpiWarps = 8, kProdWarps = 4, kMmaWarp = kEpiWarps + kProdWarps;
constexpr int kChunkThreads = (kMmaWarp + 1) * 32;

template <int D>
struct ChunkLayout {
  static constexpr uint32_t kHalfA = kTileBlocks * 128;          // 128 rows x 64 elements, 128-byte swizzle
  static constexpr uint32_t kHalfB = kChunkCols * 128;
  static constexpr int kHalves = D / 64;
  static constexpr uint32_t B = 0;                               // q- halves, then q+ halves
  static constexpr uint32_t A = B + 2 * kHalves * kHalfB;        // kStages x (lo or hi)
  static constexpr uint32_t kStageBytes = kHalves * kHalfA;
  static constexpr uint32_t BAR = A + kStages * kStageBytes;     // full[3], empty[3], acc_full[2], acc_empty[2], done, b_full
  static constexpr uint32_t MISC = BAR + 12 * 8;                 // TMEM address
  static constexpr uint32_t BYTES = MISC + 8;
  static constexpr uint32_t SMEM = BYTES + 1024;                 // + alignment slack
};

// The first column tile of request s in the grid: no scan is needed, since (columns before it) /
// 256 and one more tile for every request, or for every kMaxFewCols + 1 columns where those are
// fewer, leaves room for every request's last, partial tile: a request of this kernel has more
// than kMaxFewCols columns. (480 decodes and a chunk of 512 tokens, contexts of 1024: 38 us, 55 with
// one more tile for every request; contexts of 8192: 167 and 187.)
__host__ __device__ __forceinline__ int64_t tiles_before(int64_t columns, int requests) {
  const int64_t partial = columns / (kMaxFewCols + 1);
  return columns / kChunkCols + (partial < requests ? partial : requests);
}
__device__ __forceinline__ int64_t tile_base(const BatchArgs& b, int G, int s) {
  return tiles_before(int64_t(__ldg(b.query_start_loc + s)) * G, s);
}

template <int D, int G>
__global__ void __launch_bounds__(kChunkThreads, 1)
    block_scores_chunk_kernel(const __grid_constant__ BatchArgs b, float* scores, int width,
                              const __nv_bfloat16* q, const __nv_bfloat16* bounds, int Hkv,
                              int tiles_per_cta) {
  using LY = ChunkLayout<D>;
  constexpr int NH = LY::kHalves;
  constexpr int kTokens = kChunkCols / G;
  extern __shared__ unsigned char smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;  // 128-byte swizzle atoms need 1024-byte alignment
  unsigned char* sm = smem_raw + (base - raw);
  const uint32_t full0 = base + LY::BAR, empty0 = full0 + 8 * kStages, acc_full0 = empty0 + 8 * kStages,
                 acc_empty0 = acc_full0 + 16, done = acc_empty0 + 16, b_full = done + 8;
  griddep_wait();
  griddep_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  // ---- this CTA's request and columns
  const int head = blockIdx.x % Hkv;
  const int64_t id = blockIdx.x / Hkv;
  int lo = 0, n = b.num_seqs;  // the last request whose first tile is <= id, as in find_row
  while (n > 1) {
    const int step = (n + 31) / 32, at = lo + lane * step;
    const unsigned m = __ballot_sync(0xffffffffu, at < lo + n && tile_base(b, G, at) <= id);
    const int k = m ? 31 - __clz(m) : 0, next = lo + k * step;
    n = min(step, lo + n - next);
    lo = next;
  }
  const int s = lo;
  const int q0 = __ldg(b.query_start_loc + s), q_len = __ldg(b.query_start_loc + s + 1) - q0;
  const int L = __ldg(b.seq_lens + s);
  const int64_t tile64 = id - tile_base(b, G, s);
  if (!is_chunk(q_len, G) || tile64 < 0 || tile64 * kTokens >= q_len) return;
  if (!fits(b, q0, q_len, L, width)) {
    if (threadIdx.x == 0) raise_error(b.err, PA_DEVERR_SEQ_RANGE);
    return;
  }
  const int j0 = int(tile64) * kTokens, ntok = min(kTokens, q_len - j0), cols = ntok * G;
  const int pos0 = L - q_len + j0;                                  // position of the first token
  const int last_max = (pos0 + ntok - 1) / b.block_size;            // the last token's last block
  const int tile_begin = blockIdx.y * tiles_per_cta, tiles = (width + kTileBlocks - 1) / kTileBlocks;
  const int tile_end = min(tile_begin + tiles_per_cta, tiles);
  const int live_end = min(tile_end, last_max / kTileBlocks + 1);   // tiles behind it are all -inf
  const int32_t* table = b.block_table + int64_t(s) * b.max_blocks_per_seq;

  // ---- setup: the query rows' loads (the epilogue warps'; 16 bytes a piece), barriers, TMEM
  constexpr int PPR = D / 8, kEpiThreads = kEpiWarps * 32, kPieces = kChunkCols * PPR / kEpiThreads;
  uint4 qv[kPieces];
  if (warp < kEpiWarps) {
    const __nv_bfloat16* qp = q + ((int64_t(q0) + j0) * (Hkv * G) + head * G) * D + int(threadIdx.x) % PPR * 8;
#pragma unroll
    for (int k = 0; k < kPieces; ++k) {
      const int c = (int(threadIdx.x) + k * kEpiThreads) / PPR;
      qv[k] = c < cols ? __ldg(reinterpret_cast<const uint4*>(qp + (int64_t(c / G) * (Hkv * G) + c % G) * D))
                       : make_uint4(0, 0, 0, 0);
    }
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(full0 + 8 * i, kProdWarps);
      mbar_init(empty0 + 8 * i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(acc_full0 + 8 * i, 1);
      mbar_init(acc_empty0 + 8 * i, kEpiWarps);
    }
    mbar_init(done, 1);
    mbar_init(b_full, kEpiWarps);
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    tc::tmem_alloc(base + LY::MISC, 512);
    tc::tmem_relinquish();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(sm + LY::MISC);

  if (warp >= kEpiWarps && warp < kMmaWarp) {
    // =========================== producers: 32 rows each ===========================
    const int pw = warp - kEpiWarps;
    int stage = 0, it = 0;
    bool ok = true;
    auto hand_over = [&](int st) {  // this warp's rows of stage st have landed
      tc::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(full0 + 8 * st);
    };
    auto look_up = [&](int tile) {  // lane i: row i's block
      const int blk = tile * kTileBlocks + pw * 32 + lane;
      return tile < live_end && blk <= last_max ? __ldg(table + blk) : -1;
    };
    int next = look_up(tile_begin);
    for (int tile = tile_begin; tile < live_end && ok; ++tile) {
      int my = next;
      next = look_up(tile + 1);
      if (tile * kTileBlocks + pw * 32 + lane <= last_max && (my < 0 || my >= b.num_blocks)) {
        raise_error(b.err, PA_DEVERR_BLOCK_RANGE);
        my = -1;
      }
      for (int part = 0; part < 2; ++part, ++it) {
        ok = mbar_wait(empty0 + 8 * stage, ((it / kStages) & 1) ^ 1);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        const uint32_t dst = base + LY::A + uint32_t(stage) * LY::kStageBytes;
        constexpr int RPI = 32 / PPR;              // rows per instruction
#pragma unroll 4
        for (int r0 = 0; r0 < 32; r0 += RPI) {
          const int sub = r0 + lane / PPR, piece = lane % PPR;
          const int idr = __shfl_sync(0xffffffffu, my, sub);
          const int r = pw * 32 + sub;
          const __nv_bfloat16* row = bounds + ((int64_t(max(idr, 0)) * Hkv + head) * 2 + part) * D + piece * 8;
          cp_async16(dst + (piece / 8) * LY::kHalfA + uint32_t(r * 128) + uint32_t(((piece & 7) ^ (r & 7)) << 4), row, idr >= 0);
        }
        cp_async_commit();
        if (it > 0) {  // one stage behind: its copies have had the time of this one's issue
          cp_async_wait<1>();
          hand_over(stage == 0 ? kStages - 1 : stage - 1);
        }
        if (++stage == kStages) stage = 0;
      }
    }
    cp_async_wait<0>();
    if (ok && it > 0) hand_over(stage == 0 ? kStages - 1 : stage - 1);
    if (!ok && lane == 0) raise_error(b.err, PA_DEVERR_TIMEOUT);
  } else if (warp == kMmaWarp) {
    // =========================== MMA issue (one thread) ===========================
    if (lane == 0) {
      const uint32_t idesc = tc::idesc_bf16_f32(kTileBlocks, (cols + 15) / 16 * 16, 0);
      int stage = 0, it = 0;
      bool ok = mbar_wait(b_full, 0);
      for (int tile = tile_begin; tile < live_end && ok; ++tile) {
        const int i = tile - tile_begin, buf = i & 1;
        ok = mbar_wait(acc_empty0 + 8 * buf, ((i >> 1) & 1) ^ 1);
        for (int part = 0; part < 2 && ok; ++part, ++it) {
          ok = mbar_wait(full0 + 8 * stage, (it / kStages) & 1);
          if (!ok) break;
          tc::fence_after_sync();
          const uint64_t a = tc::smem_desc_sw128(base + LY::A + uint32_t(stage) * LY::kStageBytes, 16, 1024);
          const uint64_t c = tc::smem_desc_sw128(base + LY::B + uint32_t(part * NH) * LY::kHalfB, 16, 1024);
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            const uint32_t ko = uint32_t(k % 4) * 32;  // bytes within a 64-element half
            tc::mma_f16(tmem + uint32_t(buf) * kChunkCols, a + ((uint32_t(k / 4) * LY::kHalfA + ko) >> 4),
                        c + ((uint32_t(k / 4) * LY::kHalfB + ko) >> 4), idesc, (part > 0 || k > 0) ? 1u : 0u);
          }
          tc::mma_commit(empty0 + 8 * stage);
          if (++stage == kStages) stage = 0;
        }
        if (ok) tc::mma_commit(acc_full0 + 8 * buf);
      }
      tc::mma_commit(done);  // nothing may still write TMEM when it is freed
      if (!mbar_wait(done, 0)) ok = false;
      if (!ok) raise_error(b.err, PA_DEVERR_TIMEOUT);
    }
    __syncwarp();
  } else {
    // =========================== columns, then epilogue ===========================
    // the columns' [q-, q+], beside the producers' first copies
#pragma unroll
    for (int k = 0; k < kPieces; ++k) {
      const int i = threadIdx.x + k * kEpiThreads, c = i / PPR, piece = i % PPR;
      if (c >= (cols + 15) / 16 * 16) break;  // the MMA does not read them
      unsigned char* at = sm + LY::B + (piece / 8) * LY::kHalfB + c * 128 + (((piece & 7) ^ (c & 7)) << 4);
      *reinterpret_cast<uint4*>(at) = make_uint4(bf16x2_neg_part(qv[k].x), bf16x2_neg_part(qv[k].y),
                                                 bf16x2_neg_part(qv[k].z), bf16x2_neg_part(qv[k].w));
      *reinterpret_cast<uint4*>(at + NH * LY::kHalfB) =
          make_uint4(bf16x2_pos_part(qv[k].x), bf16x2_pos_part(qv[k].y), bf16x2_pos_part(qv[k].z),
                     bf16x2_pos_part(qv[k].w));
    }
    tc::fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(b_full);
    const int quarter = warp & 3, c_first = (warp >> 2) * 32;
    const int64_t pitch = int64_t(Hkv) * width;  // between tokens
    float* out = scores + ((int64_t(q0) + j0) * Hkv + head) * width;
    for (int tile = tile_begin; tile < tile_end; ++tile) {
      const int blk = tile * kTileBlocks + quarter * 32 + lane;
      const bool live = tile < live_end;
      bool have = false;
      const int i = tile - tile_begin, buf = i & 1;
      if (live) {
        if (blk <= last_max) {
          const int id_ = __ldg(table + blk);
          have = id_ >= 0 && id_ < b.num_blocks;
        }
        if (!__all_sync(0xffffffffu, mbar_wait(acc_full0 + 8 * buf, (i >> 1) & 1))) {
          if (lane == 0) raise_error(b.err, PA_DEVERR_TIMEOUT);
          break;
        }
        tc::fence_after_sync();
      }
      // token j sees this thread's block from position blk * B on
      const int first_j = have ? blk * b.block_size - pos0 : 0x7fffffff;
      for (int c0 = c_first; c0 < cols; c0 += kEpiWarps / 4 * 32) {
        float v[32] = {};
        if (live) {
          tc::tmem_ld32(tmem + uint32_t(buf) * kChunkCols + uint32_t(c0) + (uint32_t(quarter * 32) << 16), v);
          tc::tmem_wait_ld();
        }
        const int jc = c0 / G, nj = min(32 / G, ntok - jc);
        float* at = out + jc * pitch + blk;
#pragma unroll
        for (int x = 0; x < 32 / G; ++x) {
          float m = v[x * G];
#pragma unroll
          for (int h = 1; h < G; ++h) m = fmaxf(m, v[x * G + h]);
          if (!(live && jc + x >= first_j)) m = -INFINITY;
          if (x < nj && blk < width) *at = m;
          at += pitch;
        }
      }
      if (live) {
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(acc_empty0 + 8 * buf);
      }
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  if (warp == kMmaWarp) tc::tmem_dealloc(tmem, 512);
}

template <int D, int G>
cudaError_t launch_chunk(const BatchArgs& b, float* scores, int width, const __nv_bfloat16* q,
                         const __nv_bfloat16* bounds, int Hkv, cudaStream_t stream) {
  using LY = ChunkLayout<D>;
  constexpr auto kern = block_scores_chunk_kernel<D, G>;
  const cudaError_t e = ensure_smem<kern>(LY::SMEM);
  if (e != cudaSuccess) return e;
  const int64_t x = tiles_before(int64_t(b.num_tokens) * G, b.num_seqs) * Hkv;
  // Blocks per CTA: a CTA's setup (its request, the columns' split, the pipeline's filling) costs
  // about as much as kSetup tiles, and one CTA runs on a SM at a time: the fewest waves x (setup
  // + tiles). Four 512-token chunks (288 column tiles of 5 block tiles): 38.0 us in parts of 3 and
  // 2 tiles, 29.5 us whole.
  constexpr int64_t kSetup = 2;
  const int tiles = (width + kTileBlocks - 1) / kTileBlocks;
  int per = tiles;
  int64_t best = INT64_MAX;
  for (int split = 1; split <= tiles && split <= 2 * 152; ++split) {
    const int p = (tiles + split - 1) / split;
    const int64_t ctas = x * ((tiles + p - 1) / p), cost = (ctas + 151) / 152 * (kSetup + p);
    if (cost < best) {
      best = cost;
      per = p;
    }
  }
  return launch_pdl(kern, dim3(unsigned(x), unsigned((tiles + per - 1) / per)), dim3(kChunkThreads), LY::SMEM, stream, b,
                    scores, width, q, bounds, Hkv, per);
}

template <int D>
cudaError_t dispatch_chunk(const BatchArgs& b, float* scores, int width, const __nv_bfloat16* q,
                           const __nv_bfloat16* bounds, int Hkv, int G, cudaStream_t stream) {
  switch (G) {
    case 1: return launch_chunk<D, 1>(b, scores, width, q, bounds, Hkv, stream);
    case 2: return launch_chunk<D, 2>(b, scores, width, q, bounds, Hkv, stream);
    case 4: return launch_chunk<D, 4>(b, scores, width, q, bounds, Hkv, stream);
    default: return launch_chunk<D, 8>(b, scores, width, q, bounds, Hkv, stream);
  }
}

}  // namespace

cudaError_t launch_block_scores(const BatchArgs& b, float* scores, int score_width, const void* q, const void* bounds,
                                int num_heads, int num_kv_heads, int head_dim, cudaStream_t stream) {
  const auto* qp = static_cast<const __nv_bfloat16*>(q);
  const auto* bp = static_cast<const __nv_bfloat16*>(bounds);
  const int G = num_heads / num_kv_heads;
  const bool chunks = int64_t(min(b.max_query_len, b.num_tokens)) * G > kMaxFewCols;
  if (chunks) {
    const cudaError_t e = head_dim == 64
                              ? dispatch_chunk<64>(b, scores, score_width, qp, bp, num_kv_heads, G, stream)
                              : dispatch_chunk<128>(b, scores, score_width, qp, bp, num_kv_heads, G, stream);
    if (e != cudaSuccess) return e;
  }
  return head_dim == 64 ? launch_few<64>(b, scores, score_width, qp, bp, num_kv_heads, G, chunks, stream)
                        : launch_few<128>(b, scores, score_width, qp, bp, num_kv_heads, G, chunks, stream);
}

}  // namespace pa
