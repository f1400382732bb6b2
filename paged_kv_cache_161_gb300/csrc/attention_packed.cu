// Causal attention of whole prompts over packed rows (pa_attention_packed): [docs] PagedAttention
// (the prompt's own attention, before its rows are only in blocks); [flow] 3.2 Scheduler (prefill is
// compute-bound); [intro] 2.1 (causal mask). Token j of a request with Q query and K key rows sits at
// position K - Q + j and sees keys 0 .. K - Q + j.
//
// Bound: the tensor cores, 4 head_dim operations a visible (query row, key) pair. Tile: 128 rows =
// 128 / G query tokens x the G query heads of one KV head; steps of 128 keys:
//   S = Q.K^T        8 tcgen05.mma 128 x 128 x 16 (bf16, f32 sums in TMEM)
//   P = 2^(S scale log2 e - m), a thread a row; m moves (and O is scaled) only when a row's maximum
//                    passes it by 2^8; rounded to bf16 for the second product (2^-8 a numerator at most, averaged
//                    over the keys: below the output's own rounding)
//   O += P.V         8 tcgen05.mma 128 x D x 16, P from TMEM, V from shared memory as it lies
// The products must not wait for the softmax. TMEM holds two S (2 x 128 columns), two P (2 x 64) and
// one O (128): the softmax of a step lasts up to two steps' products, on two warpgroups that take the
// steps in turn, while Q.K of the step after next fills the S that was read. With P in its own columns, S is
// free as soon as it is in registers: nothing but P(n) stands between P.V(n - 1) and P.V(n).
// The two warpgroups' row maxima form a chain, step n's from step n - 1's, through shared memory,
// known long before the numerators; each keeps its own sums of numerators, joined at the tile's end.
//
// Roles (16 warps, one CTA a SM): warps 0-3 and 4-7 the warpgroups of even and odd steps (counted over
// all the CTA's tiles); warp 8 the tiles, Q (two buffers) and K (two); warp 9 TMEM and Q.K; warp 10 V (two);
// warp 11 P.V (a thread that issues both waits out the products it has queued before it turns to the
// other, and the tensor cores idle meanwhile: one prompt of 16384 tokens took 1971 us, with two threads 1494);
// warps 12-15 the output. The softmax goes on to the next tiles while P.V and the output follow, up to a ring's
// length of tiles behind.
// Measured (GB300, 32 / 8 heads x 128): one prompt of 16384 tokens 1240 us in a short burst, 1770 TFLOP/s, 0.91
// of the measured burst bf16 rate, and 1420 to 1490 us repeated for long, 0.86 to 0.90 of the sustained one; four chunks
// of 512 behind 8192 keys 172 us, 1450 TFLOP/s, and 182 to 190 us repeated; 16 prompts of 1024 125 us. With heads of 64 a step
// has half the products and the same softmax, which bounds it: one prompt of 16384 1126 us, 977 TFLOP/s.
// Tiles: requests with the most keys first (up to kThreads of them), a request's last tiles first; a running CTA
// takes the tiles of CTAs that have not started (clusterlaunchcontrol), so no counter lives in memory between
// calls.
//
// Every wait is bounded; on a timeout the kernel sets an error bit and leaves after its copies and
// products in flight have landed, freeing TMEM. All waits are for what takes a few steps, but for the output's, for a
// whole tile: its bound grows with the tile's steps (0.3 % of one prompt of 16384 tokens).
#include <cuda.h>
#include <cudaTypedefs.h>

#include "common.cuh"
#include "launch.h"
#include "tcgen05.cuh"

namespace pa {
namespace {

constexpr int kBM = 128;           // rows of a tile
constexpr int kBN = 128;           // keys of a step
constexpr int kMaxSeqs = 4096;     // requests of a call
constexpr int kThreads = 16 * 32;
constexpr int kWarpLoad = 8, kWarpQK = 9, kWarpV = 10, kWarpPV = 11, kWarpOut = 12;
// Registers: 512 threads x 128 at launch = 65536 = 256 x 184 (a row's 128 logits in registers) + 128 x 56 + 128 x 88.
constexpr int kRegsSoftmax = 184, kRegsOther = 56, kRegsOut = 88;
static_assert(256 * kRegsSoftmax + 128 * kRegsOther + 128 * kRegsOut <= 512 * 128, "setmaxnreg waits for registers the launch has");
constexpr uint32_t kHalf = 128 * 128;  // bytes of 128 rows x 64 bf16
constexpr uint32_t kS = 0, kP = 256, kO = 384;  // TMEM columns

struct PackedParams {
  __nv_bfloat16* out;
  const int32_t* qsl;
  const int32_t* ksl;
  unsigned int* err;
  int num_seqs, num_q_rows, num_k_rows, max_query_len, num_heads, num_kv_heads;
  int log_group;     // query heads of a KV head: 2^log_group
  float scale_log2;  // softmax scale x log2(e)
  int out_v8;        // out is 32-byte aligned
};

// A tile as warp 8 hands it to the other roles; t < 0: no more.
struct Tile {
  int t, hk, row0, nq, k0, pos0, leff, nt;
};
constexpr int kSlots = 4;
// Steps of a tile (4 million keys) for which the output waits once more, as long as a wait may last: 20 ms at
// the 0.62 us of a step of 128 keys (120 million keys of 64 elements 579 ms)
constexpr int kWaitSteps = 1 << 15;

template <int D>
struct Layout {
  static constexpr int NH = D / 64;
  static constexpr uint32_t Q = 0;                    // 2 buffers
  static constexpr uint32_t K = Q + 2 * NH * kHalf;   // 2
  static constexpr uint32_t V = K + 2 * NH * kHalf;   // 2
  static constexpr uint32_t M = V + 2 * NH * kHalf;   // float[2][128]: row maxima of the steps
  static constexpr uint32_t X = M + 2 * 128 * 4;      // float2[kSlots][2][128]: the tiles' maxima and sums
  static constexpr uint32_t RING = X + kSlots * 2 * 128 * 8;  // Tile[kSlots]
  static constexpr uint32_t CLC = RING + kSlots * 32; // 16 bytes: the answer of a try_cancel
  static constexpr uint32_t BAR = CLC + 16;
  static constexpr int NBAR = 56;
  static constexpr uint32_t MISC = BAR + NBAR * 8;    // TMEM address
  static constexpr uint32_t PLAN = MISC + 16;         // int[n + 8], uint16[n + 8]: prefix of the tiles, order of the requests
};
static_assert(sizeof(Tile) == 32, "a ring slot");

enum : int {
  bQ0 = 0, bQ1,        // a tile's queries are in shared memory
  bK0, bK1, bV0, bV1,  // a step's keys, values
  bQK0, bQK1,          // Q.K of a step has landed: S is there, the K stage is free
  bSFree0, bSFree1,    // S is in registers (4 warps)
  bP0, bP1,            // P is in TMEM (4 warps)
  bPV0, bPV1,          // P.V of a step has landed: P and the V stage are free, O holds it
  bOFree,              // O of a tile has been read (4 warps)
  bEnd0, bEnd1,        // every Q.K, every P.V has landed
  bClc,
  bRingFull0, bRingEmpty0 = bRingFull0 + kSlots,
  bM0 = bRingEmpty0 + kSlots,  // [4 warps][2]: a warp's row maxima of a step are in shared memory
  bX0 = bM0 + 8,               // [kSlots][4]: both warps of a tile's 32 rows have left their sums
  kBars = bX0 + 4 * kSlots
};
static_assert(kBars <= Layout<128>::NBAR, "barriers in the layout");
constexpr uint32_t kTakers = 15;  // of a ring slot: V, Q.K, P.V, 8 softmax warps, 4 of the output

// 16 columns of the warp's lanes (tc::tmem_ld32 with half the registers)
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float (&v)[16]) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const float (&v)[16]) {
  uint32_t r[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) r[i] = __float_as_uint(v[i]);
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::
          "r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

__device__ __forceinline__ void store32(void* dst, const uint4 a, const uint4 b, bool wide) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(a.x), "r"(a.y), "r"(a.z),
                 "r"(a.w), "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w)
                 : "memory");
  } else {
    static_cast<uint4*>(dst)[0] = a;
    static_cast<uint4*>(dst)[1] = b;
  }
}

template <int N>
__device__ __forceinline__ void regs_up() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void regs_down() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }

// One thread: asks for a CTA that has not started; 16 bytes arrive at `dst`.
__device__ __forceinline__ void clc_try_cancel(uint32_t dst, uint32_t bar) {
  asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(dst),
               "r"(bar)
               : "memory");
}
// The index of the CTA taken over, or -1.
__device__ __forceinline__ int clc_answer(uint32_t src) {
  uint32_t ok, x;
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b128 r;\n\t"
      "ld.shared.b128 r, [%2];\n\t"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t"
      "mov.u32 %1, 0;\n\t"
      "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, r;\n\t}"
      : "=r"(ok), "=r"(x)
      : "r"(src)
      : "memory");
  return ok ? int(x) : -1;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) attention_packed_kernel(const __grid_constant__ PackedParams p,
                                                                       const __grid_constant__ CUtensorMap qmap,
                                                                       const __grid_constant__ CUtensorMap kmap,
                                                                       const __grid_constant__ CUtensorMap vmap) {
  using LY = Layout<D>;
  constexpr int NH = LY::NH;
  extern __shared__ unsigned char smem_raw[];
  __shared__ int wsum[kThreads / 32];
  __shared__ volatile int failed;  // P.V gave up, which waits for all the other roles up to a tile's last step
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;  // swizzle atoms
  unsigned char* sm = smem_raw + (base - raw);
  auto bar = [&](int i) { return base + LY::BAR + 8u * uint32_t(i); };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int S = p.num_seqs, lg = p.log_group, TOK = kBM >> lg;

  griddep_wait();

  // ---- the plan: requests with queries, most keys first, and the prefix of their tiles
  int* pfx = reinterpret_cast<int*>(sm + LY::PLAN);
  uint16_t* ord = reinterpret_cast<uint16_t*>(pfx + S + 8);
  auto tiles_of = [&](int s, bool report) -> int {  // a KV head's; 0: no queries, or a malformed request
    const int q0 = p.qsl[s], q1 = p.qsl[s + 1], k0 = p.ksl[s], k1 = p.ksl[s + 1];
    if (q0 < 0 || q1 < q0 || q1 > p.num_q_rows || k0 < 0 || k1 < k0 || k1 > p.num_k_rows || q1 - q0 > p.max_query_len) {
      if (report) raise_error(p.err, PA_DEVERR_SEQ_RANGE);
      return 0;
    }
    return (q1 - q0 + TOK - 1) / TOK;
  };
  // Exclusive, in thread order. Sums stop at 2^31 - 1, which only requests that lie over one another in
  // q_start_loc can reach: their tiles end there.
  auto add = [](int a, int b) { return int(min(uint32_t(a) + uint32_t(b), 0x7fffffffu)); };
  auto block_scan = [&](int x, int* tot) {
    int inc = x;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, inc, d);
      if (lane >= d) inc = add(inc, y);
    }
    const int before = __shfl_up_sync(0xffffffffu, inc, 1);
    if (lane == 31) wsum[warp] = inc;
    __syncthreads();
    int off = 0, t = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < warp) off = add(off, wsum[w]);
      t = add(t, wsum[w]);
    }
    __syncthreads();
    *tot = t;
    return lane ? add(off, before) : off;
  };
  int P = 0;
  for (int b0 = 0; b0 < S; b0 += kThreads) {
    const int s = b0 + threadIdx.x;
    const int flag = s < S && tiles_of(s, blockIdx.x == 0) > 0;
    int tot;
    const int at = P + block_scan(flag, &tot);
    if (flag) {
      ord[at] = uint16_t(s);
      pfx[at] = p.ksl[s + 1] - p.ksl[s];
    }
    P += tot;
  }
  __syncthreads();
  if (P <= kThreads) {  // ranked by keys, then batch order; more requests: batch order
    int s = 0, key = 0, rank = 0;
    if (int(threadIdx.x) < P) {
      s = ord[threadIdx.x];
      key = pfx[threadIdx.x];
      for (int i = 0; i < P; ++i) rank += pfx[i] > key || (pfx[i] == key && i < int(threadIdx.x));
    }
    __syncthreads();
    if (int(threadIdx.x) < P) ord[rank] = uint16_t(s);
    __syncthreads();
  }
  int total = 0;
  for (int b0 = 0; b0 <= P; b0 += kThreads) {
    const int i = b0 + threadIdx.x;
    int tot;
    const int ex = block_scan(i < P ? tiles_of(ord[i], false) * p.num_kv_heads : 0, &tot);
    if (i <= P) pfx[i] = add(total, ex);
    total = add(total, tot);
  }
  __syncthreads();
  if (int(blockIdx.x) >= total) return;

  // Tile t: a request's KV heads fastest, its tiles from the last one back. For warp 8's thread, whose tiles
  // mostly ascend: the request is stepped along.
  int at_p = -1, at_q0 = 0, at_Q = 0, at_k0 = 0, at_K = 0;
  auto tile_info = [&](int t) {
    if (at_p < 0 || pfx[at_p + 1] <= t || t < pfx[at_p]) {
      if (at_p < 0 || t < pfx[at_p]) at_p = 0;
      while (pfx[at_p + 1] <= t) ++at_p;
      const int s = ord[at_p];
      at_q0 = p.qsl[s];
      at_Q = p.qsl[s + 1] - at_q0;
      at_k0 = p.ksl[s];
      at_K = p.ksl[s + 1] - at_k0;
    }
    const int r = t - pfx[at_p], back = r / p.num_kv_heads;
    const int q = (((at_Q + TOK - 1) >> (7 - lg)) - 1 - back) << (7 - lg);
    Tile x;
    x.t = t;
    x.hk = r - back * p.num_kv_heads;
    x.row0 = at_q0 + q;
    x.nq = min(TOK, at_Q - q);
    x.k0 = at_k0;
    x.pos0 = at_K - at_Q + q;
    x.leff = max(0, x.pos0 + x.nq);  // keys that its rows see
    x.nt = (x.leff + kBN - 1) / kBN;
    return x;
  };
  volatile Tile* ring = reinterpret_cast<volatile Tile*>(sm + LY::RING);
  // The CTA's i-th tile, for one thread / for a warp; false: a wait ran out.
  auto read_slot = [&](int i, Tile& x) {
    const volatile Tile& y = ring[i % kSlots];
    x.t = y.t, x.hk = y.hk, x.row0 = y.row0, x.nq = y.nq, x.k0 = y.k0, x.pos0 = y.pos0, x.leff = y.leff, x.nt = y.nt;
  };
  auto take = [&](int i, Tile& x) -> bool {
    if (!mbar_wait(bar(bRingFull0 + i % kSlots), uint32_t(i / kSlots) & 1u)) return false;
    read_slot(i, x);
    mbar_arrive(bar(bRingEmpty0 + i % kSlots));
    return true;
  };
  auto take_warp = [&](int i, Tile& x) -> bool {
    if (!__all_sync(0xffffffffu, mbar_wait(bar(bRingFull0 + i % kSlots), uint32_t(i / kSlots) & 1u))) return false;
    read_slot(i, x);
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(bRingEmpty0 + i % kSlots));
    return true;
  };

  if (threadIdx.x == 0) {
    failed = 0;
    for (int i = 0; i < kBars; ++i) {
      uint32_t n = 1;
      if (i == bSFree0 || i == bSFree1 || i == bP0 || i == bP1) n = 4;
      if (i == bOFree) n = 4;
      if (i >= bRingEmpty0 && i < bRingEmpty0 + kSlots) n = kTakers;
      if (i >= bX0) n = 2;
      mbar_init(bar(i), n);
    }
    fence_mbar_init();
  }
  if (warp == kWarpQK) {
    tc::tmem_alloc(base + LY::MISC, 512);
    tc::tmem_relinquish();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(sm + LY::MISC);
  auto fail = [&]() { raise_error(p.err, PA_DEVERR_TIMEOUT); };
  // Step n (counted over the CTA's tiles) uses S, P, K and V number n & 1; phase n >> 1 of their barriers.
  // No waiter can be two phases behind: the next phase of each barrier needs something of the waiter's.
  auto wait_step = [&](int b0, int n) { return mbar_wait(bar(b0 + (n & 1)), uint32_t(n >> 1) & 1u); };

  if (warp >= 8 && warp < kWarpOut) {
    regs_down<kRegsOther>();
    if (warp == kWarpLoad && lane == 0) {
      // =========================== tiles, Q, K ===========================
      tc::prefetch_tensormap(&qmap);
      tc::prefetch_tensormap(&kmap);
      bool ok = true;
      int n = 0, nq = 0, asked = 0, t = int(blockIdx.x);
      for (int i = 0;; ++i) {
        const bool last = t < 0 || t >= total;
        const bool again = !last && t < total - int(gridDim.x);  // a CTA's index stands for every gridDim-th tile from there
        if (!last && !again) {  // the next CTA is asked for while this tile's rows are fetched
          mbar_arrive_expect_tx(bar(bClc), 16);
          clc_try_cancel(base + LY::CLC, bar(bClc));
        }
        Tile x = {};
        x.t = -1;
        if (!last) x = tile_info(t);
        if (!mbar_wait(bar(bRingEmpty0 + i % kSlots), (uint32_t(i / kSlots) & 1u) ^ 1u)) ok = false;
        if (ok) {
          volatile Tile& y = ring[i % kSlots];
          y.t = x.t, y.hk = x.hk, y.row0 = x.row0, y.nq = x.nq, y.k0 = x.k0, y.pos0 = x.pos0, y.leff = x.leff, y.nt = x.nt;
          mbar_arrive(bar(bRingFull0 + i % kSlots));
        }
        if (last) break;
        for (int kb = 0; ok && kb < x.nt; ++kb, ++n) {
          // Q.K of step n - 2 frees the stage; no later step reads the queries of the tile before the last
          if (n >= 2 && !wait_step(bQK0, n - 2)) {
            ok = false;
            break;
          }
          if (kb == 0) {
            mbar_arrive_expect_tx(bar(bQ0 + (nq & 1)), uint32_t(kBM * D * 2));
#pragma unroll
            for (int h = 0; h < NH; ++h)
              tc::tma_load_3d(base + LY::Q + uint32_t((nq & 1) * NH + h) * kHalf, &qmap, 64 * h, x.hk << lg, x.row0,
                              bar(bQ0 + (nq & 1)));
            ++nq;
          }
          mbar_arrive_expect_tx(bar(bK0 + (n & 1)), uint32_t(kBN * D * 2));
#pragma unroll
          for (int h = 0; h < NH; ++h)
            tc::tma_load_3d(base + LY::K + uint32_t((n & 1) * NH + h) * kHalf, &kmap, 64 * h, x.hk, x.k0 + kb * kBN,
                            bar(bK0 + (n & 1)));
        }
        if (again) {
          if (!ok) break;
          t += int(gridDim.x);
          continue;
        }
        // (waited for even when a wait ran out: the answer must not arrive after the CTA has left)
        if (!mbar_wait(bar(bClc), uint32_t(asked++) & 1u)) ok = false;
        if (!ok) break;
        t = clc_answer(base + LY::CLC);
        tc::fence_proxy_async_smem();  // read before the next answer is written there
      }
      if (!ok) {  // the copies under way land before the CTA leaves
        fail();
        if (nq > 0) mbar_wait(bar(bQ0 + ((nq - 1) & 1)), uint32_t((nq - 1) >> 1) & 1u);
        for (int j = n > 2 ? n - 2 : 0; j < n; ++j) wait_step(bK0, j);
      }
    } else if (warp == kWarpV && lane == 0) {
      // =========================== V ===========================
      tc::prefetch_tensormap(&vmap);
      bool ok = true;
      int n = 0;
      for (int i = 0; ok; ++i) {
        Tile x;
        if (!take(i, x)) ok = false;
        if (!ok || x.t < 0) break;
        for (int kb = 0; kb < x.nt; ++kb, ++n) {
          if (n >= 2 && !wait_step(bPV0, n - 2)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(bar(bV0 + (n & 1)), uint32_t(kBN * D * 2));
#pragma unroll
          for (int h = 0; h < NH; ++h)
            tc::tma_load_3d(base + LY::V + uint32_t((n & 1) * NH + h) * kHalf, &vmap, 64 * h, x.hk, x.k0 + kb * kBN,
                            bar(bV0 + (n & 1)));
        }
      }
      if (!ok) {
        fail();
        for (int j = n > 2 ? n - 2 : 0; j < n; ++j) wait_step(bV0, j);
      }
    } else if (warp == kWarpQK && lane == 0) {
      // =========================== Q.K ===========================
      constexpr uint32_t idesc = tc::idesc_bf16_f32(kBM, kBN, 0);
      const uint64_t dq0 = tc::smem_desc_sw128(base + LY::Q, 16, 1024);
      const uint64_t dk0 = tc::smem_desc_sw128(base + LY::K, 16, 1024);
      bool ok = true;
      int n = 0, nq = 0;
      for (int i = 0; ok; ++i) {
        Tile x;
        if (!take(i, x)) ok = false;
        if (!ok || x.t < 0) break;
        if (x.nt == 0) continue;
        if (!mbar_wait(bar(bQ0 + (nq & 1)), uint32_t(nq >> 1) & 1u)) {
          ok = false;
          break;
        }
        const uint64_t a0 = dq0 + uint64_t((uint32_t((nq & 1) * NH) * kHalf) >> 4);
        ++nq;
        for (int kb = 0; kb < x.nt; ++kb, ++n) {
          if ((n >= 2 && !wait_step(bSFree0, n - 2)) || !wait_step(bK0, n)) {
            ok = false;
            break;
          }
          tc::fence_after_sync();
          const uint64_t b0 = dk0 + uint64_t((uint32_t((n & 1) * NH) * kHalf) >> 4);
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            const uint32_t off = uint32_t(k / 4) * kHalf + uint32_t(k % 4) * 32;
            tc::mma_f16(tmem + kS + uint32_t((n & 1) * kBN), a0 + (off >> 4), b0 + (off >> 4), idesc, k > 0 ? 1u : 0u);
          }
          tc::mma_commit(bar(bQK0 + (n & 1)));
        }
      }
      if (!ok) fail();
      tc::mma_commit(bar(bEnd0));  // every product has landed before TMEM is released
      mbar_wait(bar(bEnd0), 0);
    } else if (warp == kWarpPV && lane == 0) {
      // =========================== P.V ===========================
      constexpr uint32_t idesc = tc::idesc_bf16_f32(kBM, D, 1);
      const uint64_t dv0 = tc::smem_desc_sw128(base + LY::V, kHalf, 1024);
      bool ok = true;
      int n = 0, live = 0;
      for (int i = 0; ok; ++i) {
        Tile x;
        if (!take(i, x)) ok = false;
        if (!ok || x.t < 0) break;
        if (x.nt == 0) continue;
        if (live > 0 && !mbar_wait(bar(bOFree), uint32_t(live - 1) & 1u)) {  // O of the tile before
          ok = false;
          break;
        }
        ++live;
        for (int kb = 0; kb < x.nt; ++kb, ++n) {
          if (!wait_step(bP0, n) || !wait_step(bV0, n)) {
            ok = false;
            break;
          }
          tc::fence_after_sync();
          const uint64_t b0 = dv0 + uint64_t((uint32_t((n & 1) * NH) * kHalf) >> 4);
          auto pv = [&](int k) {
            tc::mma_f16_ts(tmem + kO, tmem + kP + uint32_t((n & 1) * 64 + k * 8), b0 + uint64_t((uint32_t(k) * 2048) >> 4),
                           idesc, (kb == 0 && k == 0) ? 0u : 1u);
          };
          if (kb + 1 < x.nt) {
#pragma unroll
            for (int k = 0; k < kBN / 16; ++k) pv(k);
          } else {  // the sixteens that hold visible keys
            const int sixteens = (x.leff - kb * kBN + 15) >> 4;
#pragma unroll 1
            for (int k = 0; k < sixteens; ++k) pv(k);
          }
          tc::mma_commit(bar(bPV0 + (n & 1)));
        }
      }
      if (!ok) {
        failed = 1;
        fail();
      }
      tc::mma_commit(bar(bEnd1));
      mbar_wait(bar(bEnd1), 0);
    }
  } else if (warp < 8) {
    regs_up<kRegsSoftmax>();
    // =========================== softmax ===========================
    const int w = warp >> 2, wr = warp & 3;  // warpgroup; its warp: TMEM lanes 32 wr ..
    const int r = wr * 32 + lane;
    const uint32_t trow = tmem + (uint32_t(wr * 32) << 16);
    float* m_sh = reinterpret_cast<float*>(sm + LY::M);
    float2* x_sh = reinterpret_cast<float2*>(sm + LY::X);
    const float sc = p.scale_log2;
    int n = 0;  // steps of the tiles before
    bool ok = true;
    Tile x;
    int kb = 0, mypos = 0;  // this warpgroup's next step of the tile
    bool active = false;
    float m = -INFINITY, l = 0.f;  // reference maximum at this warpgroup's last step, its sum of numerators
    auto next_tile = [&](int i) {
      if (!take_warp(i, x)) {
        ok = false;
        return;
      }
      kb = (n & 1) == w ? 0 : 1;
      active = (r >> lg) < x.nq;
      mypos = active ? x.pos0 + (r >> lg) : x.leff - 1;
      m = -INFINITY;
      l = 0.f;
    };
    next_tile(0);
    for (int i = 0; ok; ++i) {
      if (x.t < 0) break;
      for (; kb < x.nt; kb += 2) {
        const int at = n + kb, key0 = kb * kBN;
        if (!__all_sync(0xffffffffu, wait_step(bQK0, at))) {
          ok = false;
          break;
        }
        tc::fence_after_sync();
        float s[128];
#pragma unroll
        for (int c = 0; c < 4; ++c)
          tc::tmem_ld32(trow + kS + uint32_t(w * kBN + c * 32), *reinterpret_cast<float(*)[32]>(s + c * 32));
        tc::tmem_wait_ld();
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(bSFree0 + w));
        if (key0 + kBN - 1 > x.pos0) {  // keys past this row's position
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int k = min(max(mypos - key0 + 1 - q * 32, 0), 32);
            const uint32_t seen = k == 32 ? 0xffffffffu : (1u << k) - 1u;
#pragma unroll
            for (int c = 0; c < 32; ++c) s[q * 32 + c] = (seen >> c & 1u) ? s[q * 32 + c] : -INFINITY;
          }
        }
        float mx[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const float* y = s + 32 * c;
          float a = fmax3(y[0], y[1], y[2]), b = fmax3(y[3], y[4], y[5]);
#pragma unroll
          for (int e = 6; e < 30; e += 4) {
            a = fmax3(a, y[e], y[e + 1]);
            b = fmax3(b, y[e + 2], y[e + 3]);
          }
          mx[c] = fmax3(fmaxf(a, b), y[30], y[31]);
        }
        const float mt = fmaxf(fmax3(mx[0], mx[1], mx[2]), mx[3]);
        // ---- the maximum's chain: from the step before (the other warpgroup's), on to the next
        float m_prev = -INFINITY;
        if (at > 0) {
          if (!__all_sync(0xffffffffu, mbar_wait(bar(bM0 + wr * 2 + (w ^ 1)), uint32_t((at - 1) >> 1) & 1u))) {
            ok = false;
            break;
          }
          if (kb > 0) m_prev = m_sh[(w ^ 1) * 128 + r];
        }
        const float m_new = fmaxf(m_prev, mt);
        const bool grow = (m_new - m_prev) * sc > 8.f;
        const float m_use = grow ? m_new : m_prev;
        m_sh[w * 128 + r] = m_use;
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(bM0 + wr * 2 + w));
        if (kb > 0 && __any_sync(0xffffffffu, grow)) {  // O holds the steps before: scaled once they all landed
          if (!__all_sync(0xffffffffu, wait_step(bPV0, at - 1))) {
            ok = false;
            break;
          }
          tc::fence_after_sync();
          const float a = grow ? exp2f((m_prev - m_new) * sc) : 1.f;
#pragma unroll 1
          for (int c = 0; c < D / 16; ++c) {
            float o[16];
            tmem_ld16(trow + kO + uint32_t(c * 16), o);
            tc::tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] *= a;
            tmem_st16(trow + kO + uint32_t(c * 16), o);
          }
        }
        l *= m == m_use ? 1.f : exp2f((m - m_use) * sc);
        m = m_use;
        const float ref = m_use == -INFINITY ? 0.f : m_use;  // a row that has seen no key yet
        const float2 sc2 = make_float2(sc, sc), bias2 = make_float2(-ref * sc, -ref * sc);
        float2 rs[4] = {};
        float pk[64];
#pragma unroll
        for (int c = 0; c < 128; c += 2) {
          const float2 y = ffma2v(make_float2(s[c], s[c + 1]), sc2, bias2);
          const float2 e = make_float2(ex2_ftz(y.x), ex2_ftz(y.y));
          rs[(c >> 1) & 3] = fadd2(rs[(c >> 1) & 3], e);
          const __nv_bfloat162 h = __floats2bfloat162_rn(e.x, e.y);
          pk[c / 2] = __uint_as_float(*reinterpret_cast<const uint32_t*>(&h));
        }
        if (at >= 2 && !__all_sync(0xffffffffu, wait_step(bPV0, at - 2))) {  // P's columns, read by that step's P.V
          ok = false;
          break;
        }
        tc::fence_after_sync();
        tc::tmem_st32(trow + kP + uint32_t(w * 64), *reinterpret_cast<float(*)[32]>(pk));
        tc::tmem_st32(trow + kP + uint32_t(w * 64 + 32), *reinterpret_cast<float(*)[32]>(pk + 32));
        const float2 r01 = fadd2(rs[0], rs[1]), r23 = fadd2(rs[2], rs[3]);
        l += (r01.x + r01.y) + (r23.x + r23.y);
        // V rows behind the last key any row sees (of later tokens, or another request's) may hold NaN: P is
        // 0 there, and 0 * NaN is not. P.V ends with the sixteen rows that hold the last key; what they hold
        // behind it becomes zeros before.
        const int used = x.leff - key0;
        if (used < kBN && (used & 15)) {
          if (!__all_sync(0xffffffffu, wait_step(bV0, at))) {
            ok = false;
            break;
          }
          if (r >= used && r < ((used + 15) & ~15)) {
#pragma unroll
            for (int h = 0; h < NH; ++h)
#pragma unroll
              for (int ch = 0; ch < 8; ++ch)
                *reinterpret_cast<uint4*>(sm + LY::V + uint32_t(w * NH + h) * kHalf + uint32_t(r) * 128 + ch * 16) =
                    make_uint4(0, 0, 0, 0);
          }
          tc::fence_proxy_async_smem();
        }
        tc::tmem_wait_st();
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(bP0 + w));
      }
      if (!ok) break;
      // ---- the tile's steps are done: this warpgroup's last maximum and its sum for the output's warps
      x_sh[((i & (kSlots - 1)) * 2 + w) * 128 + r] = make_float2(m, l);
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(bX0 + (i & (kSlots - 1)) * 4 + wr));
      n += x.nt;
      next_tile(i + 1);
    }
    if (!ok) fail();
  } else {
    regs_down<kRegsOut>();
    // =========================== output ===========================
    // O / l -> out, beside the next tiles' softmax (by the softmax's own warps, behind a tile's first step, every
    // tile's P.V waited 4000 clocks for them: 16 prompts of 1024 tokens 139 -> 124 us, 64 of 256 88 -> 72 us)
    const int wr = warp & 3, r = wr * 32 + lane;
    const uint32_t trow = tmem + (uint32_t(wr * 32) << 16);
    const float2* x_sh = reinterpret_cast<const float2*>(sm + LY::X);
    bool ok = true;
    int n = 0;
    for (int i = 0;; ++i) {
      const int slot = i & (kSlots - 1);
      Tile x;
      // (the slot is given back behind the sums' reading, so the softmax is never more than kSlots tiles ahead)
      if (!__all_sync(0xffffffffu, mbar_wait(bar(bRingFull0 + slot), uint32_t(i / kSlots) & 1u))) ok = false;
      if (!ok) break;
      read_slot(i, x);
      if (x.t < 0) break;
      const int end = n + x.nt - 1;  // the tile's last step
      n += x.nt;
      bool done = false;
      for (int tries = x.nt / kWaitSteps; !done && tries >= 0; --tries) {
        done = __all_sync(0xffffffffu, mbar_wait(bar(bX0 + slot * 4 + wr), uint32_t(i / kSlots) & 1u));
        if (__any_sync(0xffffffffu, failed)) break;  // what is waited for may not come
      }
      if (!done || (x.nt > 0 && !__all_sync(0xffffffffu, wait_step(bPV0, end)))) {
        ok = false;
        break;
      }
      const float2 z = x_sh[(slot * 2 + (end & 1)) * 128 + r], y = x_sh[(slot * 2 + ((end & 1) ^ 1)) * 128 + r];
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(bRingEmpty0 + slot));
      float sum = z.y;  // z of the last step's warpgroup, y of the other
      if (y.y != 0.f) sum += y.y * (y.x == z.x ? 1.f : exp2f((y.x - z.x) * p.scale_log2));
      const float inv = x.nt == 0 ? 0.f : sum > 0.f ? 1.f / sum : (sum == 0.f ? 0.f : sum);
      tc::fence_after_sync();
      // A thread its row, 32 dimensions at a time: little code, which the softmax's does not leave much room for in
      // the instruction cache. (O packed at once and P.V let go earlier, 16 prompts of 1024 tokens: 138 us against 124;
      // rows through shared memory, so that a store writes longer runs: 128.)
      __nv_bfloat16* out = p.out + (int64_t(x.row0 + (r >> lg)) * p.num_heads + (x.hk << lg) + (r & ((1 << lg) - 1))) * D;
      const bool row = (r >> lg) < x.nq;  // else the request has no such row
#pragma unroll 1
      for (int c = 0; c < D; c += 32) {
        float o[32] = {};
        if (x.nt > 0) {
          tc::tmem_ld32(trow + kO + uint32_t(c), o);
          tc::tmem_wait_ld();
        }
        if (c + 32 == D && x.nt > 0) {
          tc::fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(bOFree));
        }
        uint4 v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float y[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) y[j] = o[8 * e + j] * inv;
          v[e] = Elem<__nv_bfloat16>::pack(y);
          if (inv == 0.f) v[e] = make_uint4(0, 0, 0, 0);  // a row that sees no key
        }
        if (row) {
#pragma unroll
          for (int e = 0; e < 4; e += 2) store32(out + c + 8 * e, v[e], v[e + 1], p.out_v8);
        }
      }
    }
    if (!ok) fail();
  }

  tc::fence_before_sync();
  __syncthreads();
  if (warp == kWarpQK) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, 512);
  }
}

// ---------------------------------------------------------------- host side
PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      return static_cast<PFN_cuTensorMapEncodeTiled_v12000>(nullptr);
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  }();
  return fn;
}

// Rows [rows][heads][D] of bf16, `stride` elements between rows; boxes of 64 dimensions, b1 heads, b2 rows.
bool row_map(CUtensorMap* m, const void* ptr, int D, int heads, int rows, int64_t stride, uint32_t b1, uint32_t b2) {
  const auto fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[3] = {cuuint64_t(D), cuuint64_t(heads), cuuint64_t(rows > 0 ? rows : 1)};
  const cuuint64_t strides[2] = {cuuint64_t(D) * 2, cuuint64_t(stride) * 2};
  const cuuint32_t box[3] = {64, b1, b2}, one[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(ptr), dims, strides, box, one,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D>
constexpr size_t plan_smem(int num_seqs) { return Layout<D>::PLAN + 6 * (size_t(num_seqs) + 8) + 1024; }
static_assert(plan_smem<128>(kMaxSeqs) + 128 <= 232448, "shared memory of a CTA");

template <int D>
cudaError_t run_packed(const PackedArgs& a, cudaStream_t stream) {
  const int G = a.num_heads / a.num_kv_heads, tok = kBM / G;
  CUtensorMap qm, km, vm;
  // no key rows at all: nothing is loaded through the maps, which then describe the queries
  const void* k = a.num_k_rows > 0 ? a.k : a.q;
  const void* v = a.num_k_rows > 0 ? a.v : a.q;
  if (!row_map(&qm, a.q, D, a.num_heads, a.num_q_rows, a.q_stride, G, tok) ||
      !row_map(&km, k, D, a.num_kv_heads, a.num_k_rows, a.k_stride, 1, kBN) ||
      !row_map(&vm, v, D, a.num_kv_heads, a.num_k_rows, a.v_stride, 1, kBN))
    return cudaErrorInvalidValue;
  int lg = 0;
  while ((1 << lg) < G) ++lg;
  const PackedParams p = {static_cast<__nv_bfloat16*>(a.out), a.q_start_loc, a.k_start_loc, a.err, a.num_seqs, a.num_q_rows,
                          a.num_k_rows, a.max_query_len, a.num_heads, a.num_kv_heads, lg,
                          a.scale * 1.4426950408889634f, reinterpret_cast<uintptr_t>(a.out) % 32 == 0 ? 1 : 0};
  const cudaError_t e = ensure_smem<attention_packed_kernel<D>>(plan_smem<D>(kMaxSeqs));
  if (e != cudaSuccess) return e;
  // At most a tile for every 128 / G tokens, and one more a request; but no more CTAs than the first
  // number and two a SM: each CTA makes the plan, and the batch may hold many requests without queries (one of 500
  // tokens among 4096: a CTA for every tile there may be takes 1340 us, so 23)
  const int64_t by_rows = int64_t(a.num_q_rows) / tok + a.num_seqs;
  const int64_t by_len = int64_t(a.num_seqs) * ((a.max_query_len + tok - 1) / tok);
  const int64_t tiles = (by_rows < by_len ? by_rows : by_len) * a.num_kv_heads;
  const int64_t most = int64_t(a.num_q_rows) / tok * a.num_kv_heads + 2 * 152;
  return launch_pdl(attention_packed_kernel<D>, dim3(unsigned(tiles < most ? tiles : most)), dim3(kThreads), plan_smem<D>(a.num_seqs), stream, p,
                    qm, km, vm);
}

}  // namespace

bool attention_packed_fits(const PackedArgs& a) {
  const int G = a.num_heads / a.num_kv_heads;
  return a.num_seqs <= kMaxSeqs && a.max_query_len <= 0x7fffffff - kBM &&
         a.num_q_rows <= 0x7fffffff - 2 * kBM && a.num_k_rows <= 0x7fffffff - 2 * kBN &&  // row numbers a tile further
         (int64_t(a.num_q_rows) * G / kBM + a.num_seqs) * a.num_kv_heads <= 0x7fffffff;
}

cudaError_t launch_attention_packed(const PackedArgs& a, cudaStream_t stream) {
  return a.head_dim == 64 ? run_packed<64>(a, stream) : run_packed<128>(a, stream);
}

}  // namespace pa
