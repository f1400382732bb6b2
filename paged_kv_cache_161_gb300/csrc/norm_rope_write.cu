// pa_norm_rope_write: RMS norm of each query and key head, rotary positions, and the cache
// write of the step's tokens, in one pass over the projection's rows.
//
//   y = x / sqrt(mean(x^2) + eps) * w                        (per head row; skipped without w)
//   a' = a cos - b sin,  b' = b cos + a sin                  for each rotated pair (a, b)
//   q_out[t] = q',  k_cache[slot] = k',  v_cache[slot] = v   (E4M3 caches: x / scale, rounded)
//
// One read of q, k, v and one write of each result: HBM-bound for long prompts, latency-bound
// for a decode step. All arithmetic is fp32 with a single rounding to the output type: the
// norm's result is not rounded before the rotation, which costs nothing in registers.
//
// A head row is D / 8 lanes of 8 elements: 4 elements of each half of the rotated part, so that
// every pair lies in one lane and only the sum of squares travels by shuffles (8-byte accesses,
// each half's contiguous over the lanes). With g the partners of the elements f, a row is
//   y' = inv (f P + g Q),  P = w cos,  Q = -/+ (the partner's w) sin
// in packed fp32 instructions, P and Q computed once per token: instructions, not bytes, bound
// the first version of this kernel (shuffled partners, scalar arithmetic).
//
// Two kernels. Few tokens: a warp loads up to kRows x 256 / D rows of one kind (query, key or
// value heads) of one token into registers and finishes: as many loads at once as there are
// rows. Many tokens: a CTA streams whole tokens through a ring in shared memory, filled by bulk
// copies (a token's q, k, v are contiguous, and so is each angle row), so that loads stay in
// flight while rows are turned and each warp's setup is paid once.
#include <type_traits>

#include "common.cuh"
#include "launch.h"

namespace pa {
namespace {

constexpr int kWarps = 4;
constexpr int kRows = 4;

__device__ __forceinline__ float2 mul2(const float2 a, const float2 b) {
  unsigned long long d;
  const unsigned long long aa = (static_cast<unsigned long long>(__float_as_uint(a.y)) << 32) | __float_as_uint(a.x);
  const unsigned long long bb = (static_cast<unsigned long long>(__float_as_uint(b.y)) << 32) | __float_as_uint(b.x);
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(aa), "l"(bb));
  return make_float2(__uint_as_float(static_cast<uint32_t>(d)), __uint_as_float(static_cast<uint32_t>(d >> 32)));
}

// 4 consecutive elements, as loaded.
template <typename T>
struct Quad;
template <>
struct Quad<__nv_bfloat16> {
  uint2 u;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { u = *reinterpret_cast<const uint2*>(p); }
  __device__ __forceinline__ void copy(__nv_bfloat16* p) const { *reinterpret_cast<uint2*>(p) = u; }
  __device__ __forceinline__ void unpack(float2* f) const {
    f[0] = make_float2(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u));
    f[1] = make_float2(__uint_as_float(u.y << 16), __uint_as_float(u.y & 0xffff0000u));
  }
};
template <>
struct Quad<float> {
  float4 u;
  __device__ __forceinline__ void load(const float* p) { u = *reinterpret_cast<const float4*>(p); }
  __device__ __forceinline__ void copy(float* p) const { *reinterpret_cast<float4*>(p) = u; }
  __device__ __forceinline__ void unpack(float2* f) const {
    f[0] = make_float2(u.x, u.y);
    f[1] = make_float2(u.z, u.w);
  }
};

__device__ __forceinline__ void store4(__nv_bfloat16* p, const float2* f, float) {
  const __nv_bfloat162 a = __floats2bfloat162_rn(f[0].x, f[0].y), b = __floats2bfloat162_rn(f[1].x, f[1].y);
  *reinterpret_cast<uint2*>(p) = make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}
__device__ __forceinline__ void store4(float* p, const float2* f, float) {
  *reinterpret_cast<float4*>(p) = make_float4(f[0].x, f[0].y, f[1].x, f[1].y);
}
// E4M3(x / scale): one binary32 division, round to nearest even, saturating (as pa_kv_write_fp8)
__device__ __forceinline__ void store4(Fp8E4M3* p, const float2* f, float scale) {
  *reinterpret_cast<uint32_t*>(p) = float2_to_fp8x2(__fdiv_rn(f[0].x, scale), __fdiv_rn(f[0].y, scale)) |
                                    float2_to_fp8x2(__fdiv_rn(f[1].x, scale), __fdiv_rn(f[1].y, scale)) << 16;
}

// What a lane does with a row. T: type of q, k, v, weights and q_out; KV: cache type.
template <typename T, typename KV, int D>
struct Turn {
  static constexpr int LPR = D / 8;     // lanes per row
  static constexpr int RPW = 32 / LPR;  // rows a warp holds per step
  bool rotated, interleaved, partial;
  int l, a, b;  // elements [a, a + 4) and [b, b + 4) of the row
  float2 cs[2], sn[2];  // the lane's 4 pairs

  __device__ __forceinline__ Turn(const NormRopeArgs& p, int lane) : interleaved(p.interleaved), partial(p.rot_dim < D), l(lane % LPR) {
    rotated = l < p.rot_dim / 8;
    const bool adjacent = interleaved || !rotated;
    a = adjacent ? 8 * l : 4 * l;
    b = adjacent ? a + 4 : p.rot_dim / 2 + a;
    cs[0] = cs[1] = make_float2(1.f, 1.f);
    sn[0] = sn[1] = make_float2(0.f, 0.f);
  }
  // The angles from the table rows of the axes' positions: row(axis) is the row's address.
  template <typename F>
  __device__ __forceinline__ void angles(const NormRopeArgs& p, F row) {
    if (!rotated) return;
    const int pair = 4 * l, half = p.rot_dim / 2;
    int first = 0, last = 0;  // the axes of the lane's first and last pair
#pragma unroll
    for (int x = 1; x < kMaxAxes; ++x) {
      if (pair >= p.section_start[x]) first = x;
      if (pair + 3 >= p.section_start[x]) last = x;
    }
    if (first == last) {
      const float* at = row(first) + pair;
      const float4 c = *reinterpret_cast<const float4*>(at), s = *reinterpret_cast<const float4*>(at + half);
      cs[0] = make_float2(c.x, c.y), cs[1] = make_float2(c.z, c.w);
      sn[0] = make_float2(s.x, s.y), sn[1] = make_float2(s.z, s.w);
    } else {  // a section ends inside
      float c[4], s[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        int axis = 0;
#pragma unroll
        for (int x = 1; x < kMaxAxes; ++x)
          if (pair + e >= p.section_start[x]) axis = x;
        c[e] = row(axis)[pair + e];
        s[e] = row(axis)[half + pair + e];
      }
      cs[0] = make_float2(c[0], c[1]), cs[1] = make_float2(c[2], c[3]);
      sn[0] = make_float2(s[0], s[1]), sn[1] = make_float2(s[2], s[3]);
    }
  }
  // The lane's weights (1 without a norm).
  __device__ __forceinline__ void weights(const void* w, float2 (&wt)[4]) const {
#pragma unroll
    for (int e = 0; e < 4; ++e) wt[e] = make_float2(1.f, 1.f);
    if (w) {
      Quad<T> x;
      x.load(static_cast<const T*>(w) + a);
      x.unpack(wt);
      x.load(static_cast<const T*>(w) + b);
      x.unpack(wt + 2);
    }
  }
  __device__ __forceinline__ void coefficients(const float2 (&wt)[4], float2 (&P)[4], float2 (&Q)[4]) const {
    if (interleaved) {
      const float c[4] = {cs[0].x, cs[0].y, cs[1].x, cs[1].y}, z[4] = {sn[0].x, sn[0].y, sn[1].x, sn[1].y};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        P[e] = make_float2(wt[e].x * c[e], wt[e].y * c[e]);
        Q[e] = make_float2(-wt[e].y * z[e], wt[e].x * z[e]);
      }
    } else {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        P[e] = mul2(wt[e], cs[e]);
        P[e + 2] = mul2(wt[e + 2], cs[e]);
        Q[e] = mul2(wt[e + 2], make_float2(-sn[e].x, -sn[e].y));
        Q[e + 2] = mul2(wt[e], sn[e]);
      }
    }
  }
  // One row per LPR lanes (all lanes of the warp call it).
  __device__ __forceinline__ void row(const Quad<T> (&in)[2], const float2 (&P)[4], const float2 (&Q)[4], bool norm, float eps,
                                      float2 (&y)[4]) const {
    float2 f[4];
    in[0].unpack(f);
    in[1].unpack(f + 2);
    if (interleaved) {
#pragma unroll
      for (int e = 0; e < 4; ++e) y[e] = ffma2v(f[e], P[e], mul2(make_float2(f[e].y, f[e].x), Q[e]));
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) y[e] = ffma2v(f[e], P[e], mul2(f[e ^ 2], Q[e]));
    }
    if (partial && !rotated) {  // nothing of a "partner", which may be infinite
#pragma unroll
      for (int e = 0; e < 4; ++e) y[e] = mul2(f[e], P[e]);
    }
    if (norm) {
      float2 q2 = mul2(f[0], f[0]);
#pragma unroll
      for (int e = 1; e < 4; ++e) q2 = ffma2v(f[e], f[e], q2);
      float ss = q2.x + q2.y;
#pragma unroll
      for (int m = LPR / 2; m >= 1; m >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, m);
      const float inv = rsqrtf(ss * (1.f / D) + eps);
#pragma unroll
      for (int e = 0; e < 4; ++e) y[e] = mul2(y[e], make_float2(inv, inv));
    }
  }
  template <typename Out>
  __device__ __forceinline__ void store(Out* dst, const float2 (&y)[4], float scale) const {
    store4(dst + a, y, scale);
    store4(dst + b, y + 2, scale);
  }
  // V: its bytes as they are, or encoded
  __device__ __forceinline__ void store_v(KV* dst, const Quad<T> (&in)[2], float scale) const {
    if constexpr (std::is_same<T, KV>::value) {
      in[0].copy(dst + a);
      in[1].copy(dst + b);
    } else {
      float2 f[4];
      in[0].unpack(f);
      in[1].unpack(f + 2);
      store(dst, f, scale);
    }
  }
};

// ---------------------------------------------------------------- few tokens
template <typename T, typename KV, int D>
__global__ void __launch_bounds__(kWarps * 32, 7)
    norm_rope_write_kernel(const __grid_constant__ NormRopeArgs p, int q_warps, int kv_warps) {
  using Lane = Turn<T, KV, D>;
  constexpr int RPW = Lane::RPW;
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31, sub = lane / Lane::LPR;
  const unsigned w = blockIdx.x * kWarps + (threadIdx.x >> 5), per_token = q_warps + 2 * kv_warps;
  const int64_t t = w / per_token;
  if (t >= p.num_tokens) return;
  const int part = int(w % per_token);
  const bool is_q = part < q_warps, is_v = part >= q_warps + kv_warps;
  const int heads = is_q ? p.num_heads : p.num_kv_heads;
  const int row0 = (is_q ? part : is_v ? part - q_warps - kv_warps : part - q_warps) * (RPW * kRows);
  Lane turn(p, lane);
  const T* src = is_q   ? static_cast<const T*>(p.q) + t * p.q_stride
                 : is_v ? static_cast<const T*>(p.v) + t * p.v_stride
                        : static_cast<const T*>(p.k) + t * p.k_stride;
  Quad<T> in[kRows][2];
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int r = min(row0 + sub + i * RPW, heads - 1);  // past the last: that row again, not stored
    in[i][0].load(src + r * D + turn.a);
    in[i][1].load(src + r * D + turn.b);
  }
  int64_t slot = 0;
  if (!is_q) slot = __ldg(p.slot_mapping + t);
  // every part of the token checks its positions: a bad one skips the token
  int pos[kMaxAxes] = {};
  bool bad = false;
#pragma unroll
  for (int x = 0; x < kMaxAxes; ++x) {
    if (x < p.num_axes) {
      pos[x] = __ldg(p.positions + x * p.num_tokens + t);
      bad |= pos[x] < 0 || pos[x] >= p.max_position;
    }
  }
  if (bad) {  // the whole warp: one token
    if (lane == 0) raise_error(p.err, PA_DEVERR_POSITION);
    return;
  }
  if (!is_q) {
    if (slot >= p.num_slots && row0 == 0 && lane == 0) raise_error(p.err, PA_DEVERR_SLOT_RANGE);
    if (slot < 0 || slot >= p.num_slots) return;  // nothing is cached
  }
  KV* cache = static_cast<KV*>(is_v ? p.v_cache : p.k_cache) + slot * p.num_kv_heads * D;
  if (is_v) {
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const int r = row0 + sub + i * RPW;
      if (r < heads) turn.store_v(cache + r * D, in[i], p.v_scale);
    }
    return;
  }
  turn.angles(p, [&](int axis) {
    int at = pos[0];
#pragma unroll
    for (int x = 1; x < kMaxAxes; ++x)
      if (axis == x) at = pos[x];
    return p.cos_sin + int64_t(at) * p.rot_dim;
  });
  const void* weight = is_q ? p.q_weight : p.k_weight;
  float2 wt[4], P[4], Q[4];
  turn.weights(weight, wt);
  turn.coefficients(wt, P, Q);
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int r = row0 + sub + i * RPW;
    if (r - sub >= heads) break;  // no row of this step
    float2 y[4];
    turn.row(in[i], P, Q, weight != nullptr, p.eps, y);
    if (r >= heads) continue;
    if (is_q)
      turn.store(static_cast<T*>(p.q_out) + (t * heads + r) * D, y, 1.f);
    else
      turn.store(cache + r * D, y, p.k_scale);
  }
}

// ---------------------------------------------------------------- many tokens
// Warps 0 .. kTurners - 1 turn a token's rows, step by step (steps of RPW rows of one kind);
// the last warp fills the ring: token t of the CTA's tokens blockIdx.x, + gridDim.x, .. .
constexpr int kTurners = 4;
constexpr int kStreamCtas = 3;                 // per SM
constexpr size_t kRingBytes = 72 * 1024;       // of a CTA
constexpr int kMaxStages = 8;
constexpr int64_t kStreamBytes = 40 << 20;

struct StageHead {
  int64_t token, slot;  // slot < 0: nothing is cached
};

struct StreamLayout {
  uint32_t k, v, angles, bytes;  // offsets in a stage, and its size
  int stages;
};
inline __host__ __device__ StreamLayout stream_layout(const NormRopeArgs& p, int row_bytes) {
  StreamLayout s;
  s.k = uint32_t(p.num_heads * row_bytes);
  s.v = s.k + uint32_t(p.num_kv_heads * row_bytes);
  s.angles = s.v + uint32_t(p.num_kv_heads * row_bytes);
  s.bytes = s.angles + uint32_t(p.num_axes * p.rot_dim * 4);
  const int n = int(kRingBytes / s.bytes);
  s.stages = n < kMaxStages ? n : kMaxStages;
  return s;
}

template <typename T, typename KV, int D>
__global__ void __launch_bounds__((kTurners + 1) * 32, kStreamCtas)
    norm_rope_stream_kernel(const __grid_constant__ NormRopeArgs p) {
  using Lane = Turn<T, KV, D>;
  constexpr int RPW = Lane::RPW, kRow = D * int(sizeof(T));
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ StageHead heads[kMaxStages];
  __shared__ __align__(8) uint64_t bars[2 * kMaxStages];
  const StreamLayout lay = stream_layout(p, kRow);
  const uint32_t full0 = smem_u32(bars), empty0 = full0 + 8 * kMaxStages;
  griddep_wait();
  griddep_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < lay.stages; ++i) {
      mbar_init(full0 + 8 * i, 1);
      mbar_init(empty0 + 8 * i, kTurners);
    }
    fence_mbar_init();
  }
  __syncthreads();
  const int64_t first = blockIdx.x, step = gridDim.x;
  int stage = 0;
  uint32_t phase = 0;
  auto advance = [&]() {
    if (++stage == lay.stages) {
      stage = 0;
      phase ^= 1;
    }
  };

  if (warp == kTurners) {
    // =========================== producer ===========================
    // lane l looks up the CTA's token k0 + l: its slot and its positions
    int64_t slot = -1;
    int pos[kMaxAxes] = {};
    bool bad = false;
    // The turners have stopped (every stage was filled): nothing may land behind the CTA's end.
    auto give_up = [&]() {
      raise_error(p.err, PA_DEVERR_TIMEOUT);
      for (int i = 0; i < lay.stages; ++i) mbar_wait(full0 + 8 * i, i < stage ? phase : phase ^ 1);
    };
    for (int64_t k = 0;; ++k) {
      if (first + k * step >= p.num_tokens) break;
      if ((k & 31) == 0) {
        const int64_t t = first + (k + lane) * step;
        bad = false;
        if (t < p.num_tokens) {
          slot = __ldg(p.slot_mapping + t);
#pragma unroll
          for (int x = 0; x < kMaxAxes; ++x) {
            if (x < p.num_axes) {
              pos[x] = __ldg(p.positions + x * p.num_tokens + t);
              bad |= pos[x] < 0 || pos[x] >= p.max_position;
            }
          }
          if (bad) raise_error(p.err, PA_DEVERR_POSITION);
          if (!bad && slot >= p.num_slots) raise_error(p.err, PA_DEVERR_SLOT_RANGE);
          if (slot >= p.num_slots) slot = -1;
        }
      }
      const int from = int(k & 31);
      const int64_t t = first + k * step, at_slot = __shfl_sync(0xffffffffu, slot, from);
      if (__shfl_sync(0xffffffffu, int(bad), from)) continue;  // a bad position skips the token
      int at[kMaxAxes];
#pragma unroll
      for (int x = 0; x < kMaxAxes; ++x) at[x] = __shfl_sync(0xffffffffu, pos[x], from);
      int ok = 1;
      if (lane == 0) {
        ok = mbar_wait(empty0 + 8 * stage, phase ^ 1) ? 1 : 0;
        if (ok) {
          heads[stage] = {t, at_slot};
          const uint32_t dst = smem_u32(smem) + uint32_t(stage) * lay.bytes, bar = full0 + 8 * stage;
          const bool kv = at_slot >= 0;
          mbar_arrive_expect_tx(bar, kv ? lay.bytes : lay.bytes - (lay.angles - lay.k));
          bulk_g2s(dst, static_cast<const T*>(p.q) + t * p.q_stride, lay.k, bar);
          if (kv) {
            bulk_g2s(dst + lay.k, static_cast<const T*>(p.k) + t * p.k_stride, lay.v - lay.k, bar);
            bulk_g2s(dst + lay.v, static_cast<const T*>(p.v) + t * p.v_stride, lay.angles - lay.v, bar);
          }
          for (int x = 0; x < p.num_axes; ++x)
            bulk_g2s(dst + lay.angles + uint32_t(x * p.rot_dim * 4), p.cos_sin + int64_t(at[x]) * p.rot_dim,
                     uint32_t(p.rot_dim * 4), bar);
        }
      }
      if (!__shfl_sync(0xffffffffu, ok, 0)) {
        if (lane == 0) give_up();
        return;
      }
      advance();
    }
    // one more stage without a token ends the others
    if (lane == 0) {
      if (mbar_wait(empty0 + 8 * stage, phase ^ 1)) {
        heads[stage] = {-1, -1};
        mbar_arrive(full0 + 8 * stage);
      } else {
        give_up();
      }
    }
    return;
  }

  // =========================== turners ===========================
  Lane turn(p, lane);
  const int sub = lane / Lane::LPR;
  float2 wq[4], wk[4];
  turn.weights(p.q_weight, wq);
  turn.weights(p.k_weight, wk);
  const int q_steps = (p.num_heads + RPW - 1) / RPW, kv_steps = (p.num_kv_heads + RPW - 1) / RPW;
  while (true) {
    if (!mbar_wait(full0 + 8 * stage, phase)) {
      raise_error(p.err, PA_DEVERR_TIMEOUT);
      return;
    }
    const StageHead head = heads[stage];
    if (head.token < 0) return;
    const unsigned char* at = smem + uint32_t(stage) * lay.bytes;
    const float* table = reinterpret_cast<const float*>(at + lay.angles);
    turn.angles(p, [&](int axis) { return table + axis * p.rot_dim; });
    auto load = [&](uint32_t base, int r, int n, Quad<T> (&in)[2]) {
      const T* row = reinterpret_cast<const T*>(at + base) + min(r, n - 1) * D;
      in[0].load(row + turn.a);
      in[1].load(row + turn.b);
    };
    float2 P[4], Q[4];
    turn.coefficients(wq, P, Q);
    T* out = static_cast<T*>(p.q_out) + head.token * p.num_heads * D;
    int i = warp;
#pragma unroll 4
    for (; i < q_steps; i += kTurners) {
      const int r = i * RPW + sub;
      Quad<T> in[2];
      float2 y[4];
      load(0, r, p.num_heads, in);
      turn.row(in, P, Q, p.q_weight != nullptr, p.eps, y);
      if (r < p.num_heads) turn.store(out + r * D, y, 1.f);
    }
    if (head.slot >= 0) {
      const int64_t to = head.slot * p.num_kv_heads * D;
      if (i - q_steps < kv_steps) turn.coefficients(wk, P, Q);
      for (; i < q_steps + kv_steps; i += kTurners) {
        const int r = (i - q_steps) * RPW + sub;
        Quad<T> in[2];
        float2 y[4];
        load(lay.k, r, p.num_kv_heads, in);
        turn.row(in, P, Q, p.k_weight != nullptr, p.eps, y);
        if (r < p.num_kv_heads) turn.store(static_cast<KV*>(p.k_cache) + to + r * D, y, p.k_scale);
      }
      for (; i < q_steps + 2 * kv_steps; i += kTurners) {
        const int r = (i - q_steps - kv_steps) * RPW + sub;
        Quad<T> in[2];
        load(lay.v, r, p.num_kv_heads, in);
        if (r < p.num_kv_heads) turn.store_v(static_cast<KV*>(p.v_cache) + to + r * D, in, p.v_scale);
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(empty0 + 8 * stage);
    advance();
  }
}

template <typename T, typename KV, int D>
cudaError_t launch(const NormRopeArgs& p, cudaStream_t stream) {
  constexpr int per_warp = 256 / D * kRows;
  const int q_warps = (p.num_heads + per_warp - 1) / per_warp, kv_warps = (p.num_kv_heads + per_warp - 1) / per_warp;
  // The stream for 40 MB of input rows or more, with at least three tokens in its ring. 32 / 8
  // heads of 128, bf16: 4096 tokens 22.3 us against 23.6, 16384 71.6 against 79.4, but 2048 14.4
  // against 13.3; 8 / 1 heads: 8192 tokens (20 MB) 20.8 against 19.3.
  const StreamLayout lay = stream_layout(p, D * int(sizeof(T)));
  if (p.num_tokens * int64_t(lay.angles) >= kStreamBytes && lay.stages >= 3) {
    constexpr auto kern = norm_rope_stream_kernel<T, KV, D>;
    const cudaError_t e = ensure_smem<kern>(kRingBytes);
    if (e != cudaSuccess) return e;
    return launch_pdl(kern, dim3(152 * kStreamCtas), dim3((kTurners + 1) * 32), size_t(lay.stages) * lay.bytes, stream, p);
  }
  const int64_t ctas = (p.num_tokens * (q_warps + 2 * kv_warps) + kWarps - 1) / kWarps;
  return launch_pdl(norm_rope_write_kernel<T, KV, D>, dim3(unsigned(ctas)), dim3(kWarps * 32), 0, stream, p, q_warps,
                    kv_warps);
}

template <int D>
cudaError_t dispatch(const NormRopeArgs& p, pa_dtype dtype, pa_dtype cache, cudaStream_t stream) {
  if (dtype == PA_BF16)
    return cache == PA_BF16 ? launch<__nv_bfloat16, __nv_bfloat16, D>(p, stream)
                            : launch<__nv_bfloat16, Fp8E4M3, D>(p, stream);
  return cache == PA_F32 ? launch<float, float, D>(p, stream) : launch<float, Fp8E4M3, D>(p, stream);
}

}  // namespace

cudaError_t launch_norm_rope_write(const NormRopeArgs& p, int head_dim, pa_dtype dtype, pa_dtype cache_dtype,
                                   cudaStream_t stream) {
  return head_dim == 64 ? dispatch<64>(p, dtype, cache_dtype, stream)
                        : dispatch<128>(p, dtype, cache_dtype, stream);
}

}  // namespace pa
