// pa_attention_sparse: attention of each query token over the blocks listed for it and its
// KV head (the list pa_select_blocks writes), through the request's block table.
//
//   out[t, h] = sum_i softmax_i(scale <q[t, h], K_i>) V_i,  i over the listed blocks' positions <= p
//
// A unit of work is (token, KV head): its G query heads are the 8 columns of the MMAs, its keys
// come in chunks of 16 tokens (one listed block is block_size / 16 of them): S^T = K Q^T with the
// tokens as rows, O^T += V^T P^T with the dims as rows. (With the heads as the 16 rows, of which
// G are used, the same takes twice the MMAs and accumulators.) Units share no keys by
// construction -- every head of every token may have chosen other blocks -- so the kernel is
// bound by the bytes of K and V, as decode attention is.
//
// Each warp streams its own chunks (every C x NW-th of the list) through a private ring of
// STAGES chunks filled by 16-byte asynchronous copies: K and V rows of one head are 2 D-byte
// segments scattered over the pool, which a warp's lanes gather directly (no tensor map, no
// barrier between warps; rows past the causal limit are zero-filled, never read). Running
// maximum, sum and O stay in fp32 registers; the reference maximum moves only when a score
// exceeds it by more than 8 (log2 units), so most chunks need no reduction over their tokens
// and no rescaling of O, and numerators stay below 2^8.
//
// Few units (a small batch, a draft of some tokens): a cluster of C = 2, 4 or 8 CTAs shares
// one unit's list. Each CTA sends its partial result to the CTAs that write the outputs,
// through distributed shared memory, so the split needs no workspace and no second launch.
// The merge runs in a fixed order: same bits every time.
//
// Precision: bf16 caches multiply in bf16; E4M3 caches in f16, which holds every code's value, and
// queries of magnitudes from 2^-14 to 65504 exactly. Everything is summed in fp32. A numerator goes
// into the second product as two 16-bit parts, the rounded value and what the rounding left: 2^-16
// relative with bf16 parts, 2^-22 with f16 (below 2^-14: 2^-25 of the reference), where one part
// alone (2^-8, 2^-11) shows in sums that cancel. 256 tokens of 64 blocks: bf16 161.1 us, 160.2 with
// one part; E4M3 100.7, 96.4; 2 x 4 tokens, E4M3: 10.7, 10.3. (The rests in the columns that four
// heads leave, without a second set of MMAs, measured the same.)
#include "block_rows.cuh"
#include "mma.cuh"

namespace pa {
namespace {

constexpr int kTok = 16;  // tokens per chunk

template <typename KV, int D, int NW, int STAGES>
struct SparseCfg {
  static constexpr int EL = sizeof(KV);
  static constexpr bool kF16 = EL == 1;
  static constexpr int RB = D * EL;       // bytes of one head's row
  static constexpr int CPR = RB / 16;     // 16-byte pieces of a row
  static constexpr int KC = D / 16;        // MMA steps of S^T, tiles of O^T
  static constexpr int kTile = kTok * RB;  // bytes of a chunk's K (or V)
  static constexpr int kWarpBytes = STAGES * 2 * kTile;
  static constexpr int kPartOff = NW * kWarpBytes;         // O from the cluster's CTAs, for this one's outputs
  static constexpr int kMlOff = kPartOff + 8 * D * 4 + 64;  // per warp, then per CTA of the cluster: m[8], l[8]
  static constexpr int kSmem = kMlOff + (NW + 8) * 16 * 4;
  static_assert(8 * D * 4 <= kWarpBytes, "a warp's O goes where its ring was");
  // Byte offset of 16-byte piece c of row r: the piece index is XORed with the row so that
  // the 8 rows of an ldmatrix fall in 8 different bank groups.
  static __device__ __forceinline__ uint32_t at(int r, int c) {
    if constexpr (RB >= 128) return uint32_t(r * RB + ((c ^ (r & 7)) << 4));
    return uint32_t(r * RB + ((c ^ ((r >> 1) & 3)) << 4));  // two 64-byte rows per 128 bytes
  }
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool real) {
  const int n = real ? 16 : 0;  // 0: nothing is read, 16 zero bytes are written
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.aligned;" ::: "memory"); }
// The address in CTA `rank` of the cluster of what is at `addr` in this one.
__device__ __forceinline__ uint32_t cluster_addr(uint32_t addr, uint32_t rank) {
  uint32_t a;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(addr), "r"(rank));
  return a;
}
__device__ __forceinline__ void st_cluster(uint32_t addr, float x) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(x) : "memory");
}
__device__ __forceinline__ void st_cluster2(uint32_t addr, float x, float y) {
  asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(addr), "f"(x), "f"(y) : "memory");
}
// An 8 x 8 matrix of 16-bit elements, transposed: lane (g, t) gives row g, columns 2t, 2t + 1.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
// Two floats as a packed pair of 16-bit values and the pair of what that rounding left.
template <bool F16>
__device__ __forceinline__ void two_parts(float a, float b, uint32_t& value, uint32_t& rest) {
  if constexpr (F16) {
    value = pack_f16(a, b);
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&value));
    rest = pack_f16(a - f.x, b - f.y);
  } else {
    value = pack_bf16(a, b);
    rest = pack_bf16(a - __uint_as_float(value << 16), b - __uint_as_float(value & 0xffff0000u));
  }
}

// ONE: a unit per warp; else a unit per CTA or cluster of csplit CTAs.
template <typename KV, int D, int NW, int STAGES, bool ONE>
__global__ void __launch_bounds__(NW * 32)
    attention_sparse_kernel(const __grid_constant__ BatchArgs b, const __grid_constant__ SparseAttnArgs a, int csplit) {
  using C = SparseCfg<KV, D, NW, STAGES>;
  extern __shared__ __align__(128) unsigned char smem[];
  griddep_wait();
  griddep_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int unit = ONE ? int(blockIdx.x) * NW + warp : int(blockIdx.x) / csplit, rank = ONE ? 0 : int(blockIdx.x) % csplit;
  const int Hkv = a.num_kv_heads, Hq = a.num_heads, G = Hq / Hkv;
  const int tok = unit / Hkv, head = unit % Hkv;
  if (ONE && tok >= b.num_tokens) return;
  const int g = lane >> 2, t = lane & 3;
  const int B = b.block_size, CB = B / kTok;
  const int nchunks = a.num_select * CB;
  const int first = ONE ? 0 : rank * NW + warp, step = ONE ? 1 : csplit * NW;
  const int n = nchunks > first ? (nchunks - first + step - 1) / step : 0;  // this warp's chunks
  const uint32_t ring = smem_u32(smem) + uint32_t(warp * C::kWarpBytes);
  const int32_t* list = a.block_idx + int64_t(unit) * a.num_select;
  // lane i's entry of the window of 32 chunks from k0 on: read before the token's request is known
  auto entry = [&](int k0) { return k0 + lane < n ? __ldg(list + (first + (k0 + lane) * step) / CB) : -1; };
  const int entry0 = entry(0);
  const QueryRow row = find_row(b, tok);
  if (row.s < 0) return;  // the whole cluster: one unit
  if (!ONE && csplit > 1) cluster_arrive();
  const int32_t* table = b.block_table + int64_t(row.s) * b.max_blocks_per_seq;

  // ---- the G query heads as B fragments: lane (g, t) holds dims of head g (0 from G on)
  uint32_t qb[C::KC][2];
  {
    const __nv_bfloat16* qp = static_cast<const __nv_bfloat16*>(a.q) + (int64_t(tok) * Hq + head * G + (g < G ? g : 0)) * D;
#pragma unroll
    for (int kc = 0; kc < C::KC; ++kc) {
      if constexpr (C::kF16) {  // k slots 2t, 2t+1, 2t+8, 2t+9 hold dims 4t .. 4t+3, as K's codes do below
        const uint2 w = g < G ? __ldg(reinterpret_cast<const uint2*>(qp + 16 * kc + 4 * t)) : make_uint2(0u, 0u);
        qb[kc][0] = pack_f16(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u));
        qb[kc][1] = pack_f16(__uint_as_float(w.y << 16), __uint_as_float(w.y & 0xffff0000u));
      } else {
        qb[kc][0] = g < G ? __ldg(reinterpret_cast<const uint32_t*>(qp + 16 * kc + 2 * t)) : 0u;
        qb[kc][1] = g < G ? __ldg(reinterpret_cast<const uint32_t*>(qp + 16 * kc + 8 + 2 * t)) : 0u;
      }
    }
  }

  // ---- chunks: lane i of a window of 32 looks up the warp's chunk k0 + i
  int64_t win_row = 0;  // cache row (block * B + offset) of the chunk's first token
  int win_valid = 0;    // tokens of it at positions <= p
  auto load_window = [&](int k0) {
    win_valid = 0;
    if (k0 + lane < n) {
      const int sub = (first + (k0 + lane) * step) % CB, blk = k0 == 0 ? entry0 : entry(k0);
      if (blk >= b.max_blocks_per_seq) {
        raise_error(b.err, PA_DEVERR_BLOCK_RANGE);
      } else if (blk >= 0) {
        win_valid = min(max(row.pos + 1 - (blk * B + sub * kTok), 0), kTok);
        if (win_valid > 0) {
          const int id = __ldg(table + blk);
          if (id < 0 || id >= b.num_blocks) {
            raise_error(b.err, PA_DEVERR_BLOCK_RANGE);
            win_valid = 0;
          } else {
            win_row = int64_t(id) * B + sub * kTok;
          }
        }
      }
    }
  };
  constexpr int kPieces = kTok * C::CPR / 32;  // 16-byte copies per lane, for K and for V
  const int64_t pitch = int64_t(Hkv) * C::RB;
  uint64_t vring = 0;  // 8 bits a stage: valid tokens of the chunk in flight there
  static_assert(STAGES <= 8, "a byte each");
  auto issue = [&](int k) {
    if (k < n) {
      if ((k & 31) == 0) load_window(k);
      const int64_t r0 = __shfl_sync(0xffffffffu, win_row, k & 31);
      const int valid = __shfl_sync(0xffffffffu, win_valid, k & 31);
      const int st = k % STAGES;
      vring = (vring & ~(uint64_t(0xff) << (8 * st))) | uint64_t(valid) << (8 * st);
      if (valid > 0) {
        const int64_t off = r0 * pitch + int64_t(head) * C::RB;
        const char* kp = static_cast<const char*>(a.k_cache) + off;
        const char* vp = static_cast<const char*>(a.v_cache) + off;
        const uint32_t kd = ring + uint32_t(st * 2 * C::kTile), vd = kd + C::kTile;
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
          const int piece = i * 32 + lane, r = piece / C::CPR, c = piece % C::CPR;
          const bool real = r < valid;
          const int64_t o = real ? r * pitch + c * 16 : 0;
          cp_async16(kd + C::at(r, c), kp + o, real);
          cp_async16(vd + C::at(r, c), vp + o, real);
        }
      }
    }
    cp_async_commit();  // one group a step, empty ones too
  };

  // O^T: lane (g, t) holds dims 16 i + g (e 0, 1) and 16 i + 8 + g (e 2, 3) of heads 2t, 2t + 1
  float o[C::KC][4];
#pragma unroll
  for (int i = 0; i < C::KC; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
  float mrun[2] = {-INFINITY, -INFINITY}, lpart[2] = {0.f, 0.f};  // of heads 2t, 2t + 1
  const float cscale = a.scale * 1.4426950408889634f * a.k_scale;
  const int lm = lane >> 3, lr = lane & 7;
  // this lane's rows g and g + 8 of S^T as tokens of the chunk (E4M3: in the order in which the
  // transposed codes of V pair tokens, 0 1 4 5 8 9 12 13 | 2 3 6 7 ..)
  const int tok0 = C::kF16 ? 4 * (g >> 1) + (g & 1) : g, tok1 = C::kF16 ? tok0 + 2 : g + 8;

#pragma unroll
  for (int k = 0; k < STAGES - 1; ++k) issue(k);
  for (int k = 0; k < n; ++k) {
    issue(k + STAGES - 1);
    cp_async_wait<STAGES - 1>();
    __syncwarp();  // every lane's copies of chunk k have landed
    const int st = k % STAGES;
    const int valid = int(vring >> (8 * st)) & 0xff;
    if (valid > 0) {
      const uint32_t kb = ring + uint32_t(st * 2 * C::kTile), vb = kb + C::kTile;
      // S^T = K Q^T, in four chains
      float acc[4][4] = {};
#pragma unroll
      for (int kc = 0; kc < C::KC; ++kc) {
        uint32_t r0, r1, r2, r3;
        if constexpr (C::kF16) {
          if ((kc & 1) == 0) {  // 16-byte pieces kc, kc + 1 (16 codes each) of rows g and g + 8
            ldsm_x4(kb + C::at(4 * (lr >> 1) + (lr & 1) + 2 * (lm & 1), kc + (lm >> 1)), r0, r1, r2, r3);
            uint32_t a0, a1, a2, a3;
            e4m3x4_to_f16x2x2(r0, a0, a2);
            e4m3x4_to_f16x2x2(r1, a1, a3);
            mma_16816(acc[kc & 2], a0, a1, a2, a3, qb[kc][0], qb[kc][1], true);
            e4m3x4_to_f16x2x2(r2, a0, a2);
            e4m3x4_to_f16x2x2(r3, a1, a3);
            mma_16816(acc[(kc & 2) + 1], a0, a1, a2, a3, qb[kc + 1][0], qb[kc + 1][1], true);
          }
        } else {
          ldsm_x4(kb + C::at((lm & 1) * 8 + lr, 2 * kc + (lm >> 1)), r0, r1, r2, r3);
          mma_16816(acc[kc & 3], r0, r1, r2, r3, qb[kc][0], qb[kc][1], false);
        }
      }
      // numerators: x[e] token tok0 of heads 2t, 2t + 1; x[2 + e] token tok1
      float x[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float v = (acc[0][e] + acc[1][e]) + (acc[2][e] + acc[3][e]);
        x[e] = (e < 2 ? tok0 : tok1) < valid ? v * cscale : -INFINITY;
      }
      float mx[2] = {fmaxf(x[0], x[2]), fmaxf(x[1], x[3])};
      if (__any_sync(0xffffffffu, mx[0] > mrun[0] + 8.f || mx[1] > mrun[1] + 8.f)) {
        float alpha[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
          for (int m = 4; m <= 16; m *= 2) mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], m));
          const float mnew = mx[e] > mrun[e] + 8.f ? mx[e] : mrun[e];
          alpha[e] = mnew == mrun[e] ? 1.f : ex2_ftz(mrun[e] - mnew);
          mrun[e] = mnew;
          lpart[e] *= alpha[e];
        }
#pragma unroll
        for (int i = 0; i < C::KC; ++i) {
          o[i][0] *= alpha[0];
          o[i][1] *= alpha[1];
          o[i][2] *= alpha[0];
          o[i][3] *= alpha[1];
        }
      }
      float pv[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float m = mrun[e & 1];
        pv[e] = ex2_ftz(x[e] - (m == -INFINITY ? 0.f : m));
        lpart[e & 1] += pv[e];
      }
      // O^T += V^T P^T (rows of V past the causal limit are zeros in shared memory), P as p + rest
      uint32_t p0, p1, rest0, rest1;
      two_parts<C::kF16>(pv[0], pv[1], p0, rest0);
      two_parts<C::kF16>(pv[2], pv[3], p1, rest1);
      p0 = transpose8x8(p0), p1 = transpose8x8(p1);
      rest0 = transpose8x8(rest0), rest1 = transpose8x8(rest1);
      if constexpr (C::kF16) {
#pragma unroll
        for (int c2 = 0; c2 < C::KC / 2; ++c2) {
          uint32_t r0, r1, r2, r3;
          ldsm_b8_x2_trans(vb + C::at(lane & 15, 2 * c2 + (lane >> 4)), r0, r1, r2, r3);
          uint32_t a0, a1, a2, a3;
          e4m3x4_to_f16x2x2(r0, a0, a2);
          e4m3x4_to_f16x2x2(r1, a1, a3);
          mma_16816(o[2 * c2], a0, a1, a2, a3, p0, p1, true);
          mma_16816(o[2 * c2], a0, a1, a2, a3, rest0, rest1, true);
          e4m3x4_to_f16x2x2(r2, a0, a2);
          e4m3x4_to_f16x2x2(r3, a1, a3);
          mma_16816(o[2 * c2 + 1], a0, a1, a2, a3, p0, p1, true);
          mma_16816(o[2 * c2 + 1], a0, a1, a2, a3, rest0, rest1, true);
        }
      } else {
#pragma unroll
        for (int i = 0; i < C::KC; ++i) {
          uint32_t r0, r1, r2, r3;  // (tokens 0-7 | 8-15) x (dims 16 i .. | + 8 ..), transposed
          ldsm_x4_trans(vb + C::at((lm >> 1) * 8 + lr, 2 * i + (lm & 1)), r0, r1, r2, r3);
          mma_16816(o[i], r0, r1, r2, r3, p0, p1, false);
          mma_16816(o[i], r0, r1, r2, r3, rest0, rest1, false);
        }
      }
    }
    __syncwarp();  // the stage may be refilled
  }
  cp_async_wait<0>();

  // ---- merge the warps' pieces (each holds O relative to its own reference maximum)
#pragma unroll
  for (int e = 0; e < 2; ++e)
#pragma unroll
    for (int m = 4; m <= 16; m *= 2) lpart[e] += __shfl_xor_sync(0xffffffffu, lpart[e], m);
  float* ml = reinterpret_cast<float*>(smem + C::kMlOff);
  __syncwarp();
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int h = 2 * t + e;
    if (h < G) {
      float* po = reinterpret_cast<float*>(smem + warp * C::kWarpBytes) + h * D + g;
#pragma unroll
      for (int i = 0; i < C::KC; ++i) {
        po[16 * i] = o[i][e];
        po[16 * i + 8] = o[i][2 + e];
      }
      if (g == 0) {
        ml[warp * 16 + h] = mrun[e];
        ml[warp * 16 + 8 + h] = lpart[e];
      }
    }
  }
  if (!ONE && csplit > 1) cluster_wait();  // every CTA of the cluster has started: its shared memory may be written
  if constexpr (ONE)
    __syncwarp();
  else
    __syncthreads();
  // Outputs in pairs of dims; of a split unit CTA r writes pairs [r share, (r + 1) share), from the
  // pieces that every CTA sends it. A piece without keys has m = -inf and weight 0.
  const int pairs = G * D / 2, share = (pairs + csplit - 1) / csplit;
  const uint32_t part_at = smem_u32(smem + C::kPartOff), ml_at = smem_u32(ml + NW * 16);
  auto write = [&](int e, float l, float x, float y) {
    const float inv = l == 0.f ? 0.f : a.v_scale / l;  // no keys: zeros
    *reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(a.out) + (int64_t(tok) * Hq + head * G) * D + 2 * e) =
        pack_bf16(x * inv, y * inv);
  };
  if constexpr (ONE) {
    for (int e = lane; e < pairs; e += 32) {
      const float2 v = *reinterpret_cast<const float2*>(smem + warp * C::kWarpBytes + e * 8);
      write(e, ml[warp * 16 + 8 + 2 * e / D], v.x, v.y);
    }
    return;
  }
  for (int e = threadIdx.x; e < pairs; e += NW * 32) {
    const int r = 2 * e / D;
    float M = -INFINITY;
#pragma unroll
    for (int w = 0; w < NW; ++w) M = fmaxf(M, ml[w * 16 + r]);
    const float Ms = M == -INFINITY ? 0.f : M;
    float l = 0.f, x = 0.f, y = 0.f;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      const float wt = ex2_ftz(ml[w * 16 + r] - Ms);
      const float2 v = *reinterpret_cast<const float2*>(smem + w * C::kWarpBytes + e * 8);
      l = fmaf(wt, ml[w * 16 + 8 + r], l);
      x = fmaf(wt, v.x, x);
      y = fmaf(wt, v.y, y);
    }
    if (csplit == 1) {
      write(e, l, x, y);
    } else {
      const int owner = e / share;
      st_cluster2(cluster_addr(part_at + uint32_t(rank * share + e - owner * share) * 8, owner), x, y);
      if (2 * e % D == 0) {  // the row's maximum and sum, to every CTA
        for (int c = 0; c < csplit; ++c) {
          st_cluster(cluster_addr(ml_at + uint32_t(rank * 16 + r) * 4, c), M);
          st_cluster(cluster_addr(ml_at + uint32_t(rank * 16 + 8 + r) * 4, c), l);
        }
      }
    }
  }
  if (csplit == 1) return;
  cluster_arrive();  // (release: what was sent is visible after the wait)
  cluster_wait();
  const float2* part = reinterpret_cast<const float2*>(smem + C::kPartOff);
  for (int i = threadIdx.x; i < min(share, pairs - rank * share); i += NW * 32) {
    const int e = rank * share + i, r = 2 * e / D;
    const float* from = ml + NW * 16 + r;
    float M = -INFINITY;
    for (int c = 0; c < csplit; ++c) M = fmaxf(M, from[c * 16]);
    const float Ms = M == -INFINITY ? 0.f : M;
    float l = 0.f, x = 0.f, y = 0.f;
    for (int c = 0; c < csplit; ++c) {
      const float wt = ex2_ftz(from[c * 16] - Ms);
      const float2 v = part[c * share + i];
      l = fmaf(wt, from[c * 16 + 8], l);
      x = fmaf(wt, v.x, x);
      y = fmaf(wt, v.y, y);
    }
    write(e, l, x, y);
  }
}

template <typename KV, int D>
cudaError_t launch(const BatchArgs& b, const SparseAttnArgs& a, cudaStream_t stream) {
  constexpr int NW = 4, STAGES = sizeof(KV) == 1 ? 6 : 3;
  using C = SparseCfg<KV, D, NW, STAGES>;
  const int64_t units = int64_t(b.num_tokens) * a.num_kv_heads;
  const int chunks = a.num_select * (b.block_size / kTok);
  // A warp per unit (nothing is merged) or a CTA: 2 CTAs of NW warps fit a SM either way, so the
  // time goes with the waves of warps (of CTAs) x (chunks a warp takes + what a unit costs
  // beside them, 2.5 and 5 chunks' time). 256 x 8 units: of 4 blocks 17.6 us by warps, 30.8 by
  // CTAs, of 32 blocks 82.4 and 87.9; 160 x 8 units (two waves of warps, the second almost
  // empty) of 128 blocks 251.5 and 196.6.
  const int64_t slots = 2 * 152, warps_t = (units + slots * NW - 1) / (slots * NW) * (2 * int64_t(chunks) + 5),
                ctas_t = (units + slots - 1) / slots * (2 * ((int64_t(chunks) + NW - 1) / NW) + 10);
  if (units >= slots && warps_t < ctas_t) {
    constexpr auto kern = attention_sparse_kernel<KV, D, NW, STAGES, true>;
    const cudaError_t e = ensure_smem<kern>(C::kSmem);
    if (e != cudaSuccess) return e;
    return launch_pdl(kern, dim3(unsigned((units + NW - 1) / NW)), dim3(NW * 32), C::kSmem, stream, b, a, 1);
  }
  constexpr auto kern = attention_sparse_kernel<KV, D, NW, STAGES, false>;
  cudaError_t e = ensure_smem<kern>(C::kSmem);
  if (e != cudaSuccess) return e;
  // CTAs per unit: one a SM at least, while each warp still has two chunks. (Two requests of
  // four tokens, 64 units of 128 blocks, E4M3: 10.7 us with 256 CTAs in clusters of 4, 13.5 with
  // 128 in clusters of 2, 15.3 with 512 in clusters of 8.)
  int split = 1;
  while (split < 8 && units * split < 152 && chunks >= split * 2 * NW * 2) split *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(units * split));
  cfg.blockDim = dim3(NW * 32);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = unsigned(split);
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = split > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, b, a, split);
}

}  // namespace

cudaError_t launch_attention_sparse(const BatchArgs& b, const SparseAttnArgs& a, cudaStream_t stream) {
  if (a.cache_dtype == PA_FP8_E4M3)
    return a.head_dim == 64 ? launch<Fp8E4M3, 64>(b, a, stream) : launch<Fp8E4M3, 128>(b, a, stream);
  return a.head_dim == 64 ? launch<__nv_bfloat16, 64>(b, a, stream) : launch<__nv_bfloat16, 128>(b, a, stream);
}

}  // namespace pa
