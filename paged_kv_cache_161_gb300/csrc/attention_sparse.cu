// pa_attention_sparse: attention of each query token over the blocks listed for it and its
// KV head (the list pa_select_blocks writes), through the request's block table.
//
//   out[t, h] = sum_i softmax_i(scale <q[t, h], K_i>) V_i,  i over the listed blocks' positions <= p
//
// A unit of work is (token, KV head): its G query heads are rows of a 16-row MMA, its keys
// come in chunks of 16 tokens (one listed block is block_size / 16 of them). Units share no
// keys by construction -- every head of every token may have chosen other blocks -- so the
// kernel streams G x 16-row products against keys read once per unit: bound by the bytes of
// K and V, as decode attention is.
//
// Each warp streams its own chunks (every C x NW-th of the list) through a private ring of
// STAGES chunks filled by 16-byte asynchronous copies: K and V rows of one head are 2 D-byte
// segments scattered over the pool, which a warp's lanes gather directly (no tensor map, no
// barrier between warps; rows past the causal limit are zero-filled, never read). Running
// maximum, sum and O stay in fp32 registers.
//
// Few units (a small batch, a draft of some tokens): a cluster of C = 2, 4 or 8 CTAs shares
// one unit's list, and merges its partial results through distributed shared memory, so the
// split needs no workspace and no second launch. The merge runs in a fixed order: same bits
// every time.
//
// Precision as the decode kernel: bf16 caches multiply in bf16 with P rounded to bf16; E4M3
// caches in f16 (codes exact, P rounded to f16); everything summed in fp32.
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
  static constexpr int KC = D / 16;
  static constexpr int NT = D / 8;
  static constexpr int kTile = kTok * RB;  // bytes of a chunk's K (or V)
  static constexpr int kWarpBytes = STAGES * 2 * kTile;
  static constexpr int kPartOff = NW * kWarpBytes;         // the CTA's merged O, for the cluster
  static constexpr int kMlOff = kPartOff + 8 * D * 4;      // per warp: m[8], l[8]; then the CTA's
  static constexpr int kSmem = kMlOff + (NW + 1) * 16 * 4;
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

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}
__device__ __forceinline__ float ld_cluster(uint32_t addr, uint32_t rank) {
  float v;
  asm volatile("{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %1, %2;\n\tld.shared::cluster.f32 %0, [a];\n\t}"
               : "=f"(v)
               : "r"(addr), "r"(rank)
               : "memory");
  return v;
}

template <typename KV, int D, int NW, int STAGES>
__global__ void __launch_bounds__(NW * 32)
    attention_sparse_kernel(const __grid_constant__ BatchArgs b, const __grid_constant__ SparseAttnArgs a, int csplit) {
  using C = SparseCfg<KV, D, NW, STAGES>;
  extern __shared__ __align__(128) unsigned char smem[];
  griddep_wait();
  griddep_launch_dependents();
  const int unit = blockIdx.x / csplit, rank = blockIdx.x % csplit;
  const int Hkv = a.num_kv_heads, Hq = a.num_heads, G = Hq / Hkv;
  const int tok = unit / Hkv, head = unit % Hkv;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int B = b.block_size, CB = B / kTok;
  const int nchunks = a.num_select * CB;
  const int first = rank * NW + warp, step = csplit * NW;
  const int n = nchunks > first ? (nchunks - first + step - 1) / step : 0;  // this warp's chunks
  const uint32_t ring = smem_u32(smem) + uint32_t(warp * C::kWarpBytes);
  const int32_t* list = a.block_idx + int64_t(unit) * a.num_select;
  // lane i's entry of the window of 32 chunks from k0 on: read before the token's request is known
  auto entry = [&](int k0) { return k0 + lane < n ? __ldg(list + (first + (k0 + lane) * step) / CB) : -1; };
  const int entry0 = entry(0);
  const QueryRow row = find_row(b, tok);
  if (row.s < 0) return;  // the whole cluster: one unit
  const int32_t* table = b.block_table + int64_t(row.s) * b.max_blocks_per_seq;

  // ---- the G query rows as A fragments (rows g >= G are zero)
  uint32_t qa0[C::KC], qa2[C::KC];
  {
    const __nv_bfloat16* qp = static_cast<const __nv_bfloat16*>(a.q) + (int64_t(tok) * Hq + head * G + (g < G ? g : 0)) * D;
#pragma unroll
    for (int kc = 0; kc < C::KC; ++kc) {
      if constexpr (C::kF16) {  // k slots 2t, 2t+1, 2t+8, 2t+9 hold dims 4t .. 4t+3, as K's codes do below
        const uint2 w = g < G ? __ldg(reinterpret_cast<const uint2*>(qp + 16 * kc + 4 * t)) : make_uint2(0u, 0u);
        qa0[kc] = pack_f16(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u));
        qa2[kc] = pack_f16(__uint_as_float(w.y << 16), __uint_as_float(w.y & 0xffff0000u));
      } else {
        qa0[kc] = g < G ? __ldg(reinterpret_cast<const uint32_t*>(qp + 16 * kc + 2 * t)) : 0u;
        qa2[kc] = g < G ? __ldg(reinterpret_cast<const uint32_t*>(qp + 16 * kc + 8 + 2 * t)) : 0u;
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
  uint32_t vring = 0;  // 8 bits a stage: valid tokens of the chunk in flight there
  auto issue = [&](int k) {
    if (k < n) {
      if ((k & 31) == 0) load_window(k);
      const int64_t r0 = __shfl_sync(0xffffffffu, win_row, k & 31);
      const int valid = __shfl_sync(0xffffffffu, win_valid, k & 31);
      const int st = k % STAGES;
      vring = (vring & ~(0xffu << (8 * st))) | uint32_t(valid) << (8 * st);
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

  float o[C::NT][4];
#pragma unroll
  for (int i = 0; i < C::NT; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
  float mrun = -INFINITY, lpart = 0.f;
  const float cscale = a.scale * 1.4426950408889634f * a.k_scale;

#pragma unroll
  for (int k = 0; k < STAGES - 1; ++k) issue(k);
  for (int k = 0; k < n; ++k) {
    issue(k + STAGES - 1);
    cp_async_wait<STAGES - 1>();
    __syncwarp();  // every lane's copies of chunk k have landed
    const int st = k % STAGES;
    const int valid = (vring >> (8 * st)) & 0xff;
    if (valid > 0) {
      const uint32_t kb = ring + uint32_t(st * 2 * C::kTile), vb = kb + C::kTile;
      // S = Q K^T: two tiles of 8 tokens, two accumulators each (even / odd k steps)
      float sacc[2][4], sacc2[2][4];
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) sacc[j][e] = sacc2[j][e] = 0.f;
      const int lm = lane >> 3, lr = lane & 7;
#pragma unroll
      for (int kc = 0; kc < C::KC; ++kc) {
        uint32_t r0, r1, r2, r3;
        if constexpr (C::kF16) {
          if ((kc & 1) == 0) {  // 16-byte pieces kc, kc + 1 (16 codes each) of the two token tiles
            ldsm_x4(kb + C::at(4 * (lr >> 1) + (lr & 1) + 2 * (lm & 1), kc + (lm >> 1)), r0, r1, r2, r3);
            uint32_t a0, a1, b0, b1, c0, c1, d0, d1;
            e4m3x4_to_f16x2x2(r0, a0, a1);
            e4m3x4_to_f16x2x2(r1, b0, b1);
            e4m3x4_to_f16x2x2(r2, c0, c1);
            e4m3x4_to_f16x2x2(r3, d0, d1);
            mma_16816(sacc[0], qa0[kc], 0u, qa2[kc], 0u, a0, a1, true);
            mma_16816(sacc[1], qa0[kc], 0u, qa2[kc], 0u, b0, b1, true);
            mma_16816(sacc2[0], qa0[kc + 1], 0u, qa2[kc + 1], 0u, c0, c1, true);
            mma_16816(sacc2[1], qa0[kc + 1], 0u, qa2[kc + 1], 0u, d0, d1, true);
          }
        } else {
          ldsm_x4(kb + C::at((lm & 1) * 8 + lr, 2 * kc + (lm >> 1)), r0, r1, r2, r3);
          mma_16816((kc & 1) ? sacc2[0] : sacc[0], qa0[kc], 0u, qa2[kc], 0u, r0, r2, false);
          mma_16816((kc & 1) ? sacc2[1] : sacc[1], qa0[kc], 0u, qa2[kc], 0u, r1, r3, false);
        }
      }
      // online softmax of row g over the chunk; the quad's lanes share the row. The reference
      // maximum moves only when a score exceeds it by more than 8 (log2 units), so O is
      // rescaled only then and numerators stay below 2^8.
      float x[2][2], mx = -INFINITY;
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const bool in = (C::kF16 ? 4 * t + 2 * j + e : 8 * j + 2 * t + e) < valid;
          x[j][e] = in ? (sacc[j][e] + sacc2[j][e]) * cscale : -INFINITY;
          mx = fmaxf(mx, x[j][e]);
        }
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      const float mnew = mx > mrun + 8.f ? mx : mrun;
      const float ms = mnew == -INFINITY ? 0.f : mnew;
      const float alpha = mnew == mrun ? 1.f : ex2_ftz(mrun - ms);
      float pv[2][2], psum = 0.f;
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          pv[j][e] = ex2_ftz(x[j][e] - ms);
          psum += pv[j][e];
        }
      lpart = lpart * alpha + psum;
      mrun = mnew;
      if (__any_sync(0xffffffffu, alpha != 1.f)) {
#pragma unroll
        for (int i = 0; i < C::NT; ++i) {
          o[i][0] *= alpha;
          o[i][1] *= alpha;
        }
      }
      // O += P V (rows of V past the causal limit are zeros in shared memory)
      if constexpr (C::kF16) {
        const uint32_t p0 = pack_f16(pv[0][0], pv[0][1]), p2 = pack_f16(pv[1][0], pv[1][1]);
#pragma unroll
        for (int c2 = 0; c2 < C::KC / 2; ++c2) {
          uint32_t r0, r1, r2, r3;
          ldsm_b8_x2_trans(vb + C::at(lane & 15, 2 * c2 + (lane >> 4)), r0, r1, r2, r3);
          uint32_t a0, a1, b0, b1, c0, c1, d0, d1;
          e4m3x4_to_f16x2x2(r0, a0, a1);
          e4m3x4_to_f16x2x2(r1, b0, b1);
          e4m3x4_to_f16x2x2(r2, c0, c1);
          e4m3x4_to_f16x2x2(r3, d0, d1);
          mma_16816(o[4 * c2 + 0], p0, 0u, p2, 0u, a0, a1, true);
          mma_16816(o[4 * c2 + 1], p0, 0u, p2, 0u, b0, b1, true);
          mma_16816(o[4 * c2 + 2], p0, 0u, p2, 0u, c0, c1, true);
          mma_16816(o[4 * c2 + 3], p0, 0u, p2, 0u, d0, d1, true);
        }
      } else {
        const uint32_t p0 = pack_bf16(pv[0][0], pv[0][1]), p2 = pack_bf16(pv[1][0], pv[1][1]);
#pragma unroll
        for (int i2 = 0; i2 < C::NT / 2; ++i2) {
          uint32_t r0, r1, r2, r3;
          ldsm_x4_trans(vb + C::at((lm & 1) * 8 + lr, 2 * i2 + (lm >> 1)), r0, r1, r2, r3);
          mma_16816(o[2 * i2], p0, 0u, p2, 0u, r0, r1, false);
          mma_16816(o[2 * i2 + 1], p0, 0u, p2, 0u, r2, r3, false);
        }
      }
    }
    __syncwarp();  // the stage may be refilled
  }
  cp_async_wait<0>();

  // ---- merge the warps' pieces (each holds O relative to its own reference maximum)
  lpart += __shfl_xor_sync(0xffffffffu, lpart, 1);
  lpart += __shfl_xor_sync(0xffffffffu, lpart, 2);
  float* ml = reinterpret_cast<float*>(smem + C::kMlOff);
  __syncwarp();
  if (g < G) {
    float* po = reinterpret_cast<float*>(smem + warp * C::kWarpBytes) + g * D + 2 * t;
#pragma unroll
    for (int i = 0; i < C::NT; ++i) *reinterpret_cast<float2*>(po + 8 * i) = make_float2(o[i][0], o[i][1]);
    if (t == 0) {
      ml[warp * 16 + g] = mrun;
      ml[warp * 16 + 8 + g] = lpart;
    }
  }
  __syncthreads();
  // (m, l, O) of `parts` pieces of row r, dims d, d + 1; a piece without keys has m = -inf
  float* part = reinterpret_cast<float*>(smem + C::kPartOff);
  for (int e = threadIdx.x; e < G * D / 2; e += NW * 32) {
    const int r = 2 * e / D, d = 2 * e % D;
    float M = -INFINITY;
#pragma unroll
    for (int w = 0; w < NW; ++w) M = fmaxf(M, ml[w * 16 + r]);
    const float Ms = M == -INFINITY ? 0.f : M;
    float l = 0.f, x = 0.f, y = 0.f;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      const float wt = ex2_ftz(ml[w * 16 + r] - Ms);
      const float2 v = *reinterpret_cast<const float2*>(smem + w * C::kWarpBytes + (r * D + d) * 4);
      l = fmaf(wt, ml[w * 16 + 8 + r], l);
      x = fmaf(wt, v.x, x);
      y = fmaf(wt, v.y, y);
    }
    if (csplit == 1) {
      const float inv = l == 0.f ? 0.f : a.v_scale / l;  // no keys: zeros
      *reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(a.out) + (int64_t(tok) * Hq + head * G + r) * D + d) =
          pack_bf16(x * inv, y * inv);
    } else {
      *reinterpret_cast<float2*>(part + r * D + d) = make_float2(x, y);
      if (d == 0) {
        ml[NW * 16 + r] = M;
        ml[NW * 16 + 8 + r] = l;
      }
    }
  }
  if (csplit == 1) return;
  // ---- merge the cluster's CTAs: CTA `rank` writes its share of the outputs
  cluster_sync();
  const uint32_t part_at = smem_u32(part), ml_at = smem_u32(ml + NW * 16);
  const int share = (G * D / 2 + csplit - 1) / csplit;
  for (int e = rank * share + threadIdx.x; e < min(rank * share + share, G * D / 2); e += NW * 32) {
    const int r = 2 * e / D, d = 2 * e % D;
    float M = -INFINITY;
    for (int c = 0; c < csplit; ++c) M = fmaxf(M, ld_cluster(ml_at + r * 4, c));
    const float Ms = M == -INFINITY ? 0.f : M;
    float l = 0.f, x = 0.f, y = 0.f;
    for (int c = 0; c < csplit; ++c) {
      const float wt = ex2_ftz(ld_cluster(ml_at + r * 4, c) - Ms);
      l = fmaf(wt, ld_cluster(ml_at + (8 + r) * 4, c), l);
      x = fmaf(wt, ld_cluster(part_at + (r * D + d) * 4, c), x);
      y = fmaf(wt, ld_cluster(part_at + (r * D + d + 1) * 4, c), y);
    }
    const float inv = l == 0.f ? 0.f : a.v_scale / l;
    *reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(a.out) + (int64_t(tok) * Hq + head * G + r) * D + d) =
        pack_bf16(x * inv, y * inv);
  }
  cluster_sync();  // no CTA leaves while another reads its shared memory
}

template <typename KV, int D>
cudaError_t launch(const BatchArgs& b, const SparseAttnArgs& a, cudaStream_t stream) {
  constexpr int NW = 4, STAGES = 3;
  using C = SparseCfg<KV, D, NW, STAGES>;
  constexpr auto kern = attention_sparse_kernel<KV, D, NW, STAGES>;
  cudaError_t e = ensure_smem<kern>(C::kSmem);
  if (e != cudaSuccess) return e;
  // CTAs per unit: one a SM at least, while each warp still has two chunks. (Two requests of
  // four tokens, 64 units of 128 blocks, E4M3: 12.3 us with 256 CTAs in clusters of 4, 17.5 with
  // 512 in clusters of 8.)
  const int64_t units = int64_t(b.num_tokens) * a.num_kv_heads;
  const int chunks = a.num_select * (b.block_size / kTok);
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
