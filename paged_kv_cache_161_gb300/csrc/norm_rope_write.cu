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
// each half's contiguous over the lanes). A warp takes up to kRows x 256 / D rows of one kind
// (query, key or value heads) of one token, whose loads are all issued before the first is
// used; the token's cosines and sines and the weights stay in registers over them. Arithmetic
// on pairs of fp32 values (packed instructions): instructions, not bytes, were the bound of
// the kernel with shuffled partners and scalar arithmetic.
#include <type_traits>

#include "common.cuh"
#include "launch.h"

namespace pa {
namespace {

constexpr int kWarps = 4;
constexpr int kRows = 4;
constexpr int kBatches = 2;
constexpr int64_t kFill = 152 * 32 * 4;  // warps

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

// T: type of q, k, v, weights and q_out; KV: cache type.
template <typename T, typename KV, int D>
__global__ void __launch_bounds__(kWarps * 32, 7) norm_rope_write_kernel(const __grid_constant__ NormRopeArgs p, int q_warps,
                                                                        int kv_warps, int batches) {
  constexpr int LPR = D / 8;     // lanes per row
  constexpr int RPW = 32 / LPR;  // rows a warp holds per step
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31, sub = lane / LPR, l = lane % LPR;
  const unsigned w = blockIdx.x * kWarps + (threadIdx.x >> 5), per_token = q_warps + 2 * kv_warps;
  const int64_t t = w / per_token;
  if (t >= p.num_tokens) return;
  const int part = int(w % per_token);
  const bool is_q = part < q_warps, is_v = part >= q_warps + kv_warps;
  const int heads = is_q ? p.num_heads : p.num_kv_heads;
  // the warp's rows: `batches` times RPW x kRows of them
  const int row_begin = (is_q ? part : is_v ? part - q_warps - kv_warps : part - q_warps) * (batches * RPW * kRows);
  const int row_end = min(row_begin + batches * RPW * kRows, heads);

  // this lane's elements: [a, a + 4) and [b, b + 4)
  const int rot = p.rot_dim, half = rot / 2;
  const bool rotated = l < rot / 8;
  const int a = p.interleaved || !rotated ? 8 * l : 4 * l, b = p.interleaved || !rotated ? a + 4 : half + a;
  const T* src = is_q   ? static_cast<const T*>(p.q) + t * p.q_stride
                 : is_v ? static_cast<const T*>(p.v) + t * p.v_stride
                        : static_cast<const T*>(p.k) + t * p.k_stride;
  Quad<T> in[kRows][2];
  auto load_rows = [&](int row0) {
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const int r = min(row0 + sub + i * RPW, heads - 1);  // past the last: that row again, not stored
      in[i][0].load(src + r * D + a);
      in[i][1].load(src + r * D + b);
    }
  };
  load_rows(row_begin);
  int64_t slot = 0;
  if (!is_q) slot = __ldg(p.slot_mapping + t);
  // ---- positions (every part of the token checks them: a bad one skips the token)
  int pos[kMaxAxes];
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
    if (slot >= p.num_slots && row_begin == 0 && lane == 0) raise_error(p.err, PA_DEVERR_SLOT_RANGE);
    if (slot < 0 || slot >= p.num_slots) return;  // nothing is cached
  }
  KV* cache = static_cast<KV*>(is_v ? p.v_cache : p.k_cache) + slot * p.num_kv_heads * D;
  if (is_v) {
    for (int row0 = row_begin;;) {
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const int r = row0 + sub + i * RPW;
      if (r >= heads) break;
      if constexpr (std::is_same<T, KV>::value) {  // V's bytes as they are
        in[i][0].copy(cache + r * D + a);
        in[i][1].copy(cache + r * D + b);
      } else {
        float2 f[4];
        in[i][0].unpack(f);
        in[i][1].unpack(f + 2);
        store4(cache + r * D + a, f, p.v_scale);
        store4(cache + r * D + b, f + 2, p.v_scale);
      }
    }
    row0 += RPW * kRows;
    if (row0 >= row_end) return;
    load_rows(row0);
    }
  }
  // ---- the lane's 4 pairs: cosines and sines
  float2 cs[2] = {make_float2(1.f, 1.f), make_float2(1.f, 1.f)}, sn[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
  if (rotated) {
    const int pair = 4 * l;
    int first = pos[0], last = pos[0];  // the positions of the lane's first and last pair
#pragma unroll
    for (int x = 1; x < kMaxAxes; ++x) {
      if (x < p.num_axes && pair >= p.section_start[x]) first = pos[x];
      if (x < p.num_axes && pair + 3 >= p.section_start[x]) last = pos[x];
    }
    if (first == last) {
      const float* at = p.cos_sin + int64_t(first) * rot + pair;
      const float4 c = __ldg(reinterpret_cast<const float4*>(at)), s = __ldg(reinterpret_cast<const float4*>(at + half));
      cs[0] = make_float2(c.x, c.y), cs[1] = make_float2(c.z, c.w);
      sn[0] = make_float2(s.x, s.y), sn[1] = make_float2(s.z, s.w);
    } else {  // a section ends inside
      float c[4], s[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        int at = pos[0];
#pragma unroll
        for (int x = 1; x < kMaxAxes; ++x)
          if (x < p.num_axes && pair + e >= p.section_start[x]) at = pos[x];
        c[e] = __ldg(p.cos_sin + int64_t(at) * rot + pair + e);
        s[e] = __ldg(p.cos_sin + int64_t(at) * rot + half + pair + e);
      }
      cs[0] = make_float2(c[0], c[1]), cs[1] = make_float2(c[2], c[3]);
      sn[0] = make_float2(s[0], s[1]), sn[1] = make_float2(s[2], s[3]);
    }
  }
  // ---- a row is then y' = inv (f P + g Q), g the partners of f: P = w cos, Q = -/+ (the
  // partner's w) sin (w = inv = 1 without a norm)
  const T* weight = static_cast<const T*>(is_q ? p.q_weight : p.k_weight);
  float2 P[4], Q[4];
  {
    float2 wt[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) wt[e] = make_float2(1.f, 1.f);
    if (weight) {
      Quad<T> x;
      x.load(weight + a);
      x.unpack(wt);
      x.load(weight + b);
      x.unpack(wt + 2);
    }
    if (p.interleaved) {
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

  for (int row0 = row_begin;;) {
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int r = row0 + sub + i * RPW;
    if (r - sub >= heads) break;  // no row of this step
    float2 f[4], y[4];
    in[i][0].unpack(f);
    in[i][1].unpack(f + 2);
    if (!rotated) {  // (no product with a partner: it may be infinite)
#pragma unroll
      for (int e = 0; e < 4; ++e) y[e] = mul2(f[e], P[e]);
    } else if (p.interleaved) {
#pragma unroll
      for (int e = 0; e < 4; ++e) y[e] = ffma2v(f[e], P[e], mul2(make_float2(f[e].y, f[e].x), Q[e]));
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) y[e] = ffma2v(f[e], P[e], mul2(f[e ^ 2], Q[e]));
    }
    if (weight) {
      float2 q2 = mul2(f[0], f[0]);
#pragma unroll
      for (int e = 1; e < 4; ++e) q2 = ffma2v(f[e], f[e], q2);
      float ss = q2.x + q2.y;
#pragma unroll
      for (int m = LPR / 2; m >= 1; m >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, m);
      const float inv = rsqrtf(ss * (1.f / D) + p.eps);
#pragma unroll
      for (int e = 0; e < 4; ++e) y[e] = mul2(y[e], make_float2(inv, inv));
    }
    if (r >= heads) continue;
    if (is_q) {
      T* dst = static_cast<T*>(p.q_out) + (t * heads + r) * D;
      store4(dst + a, y, 1.f);
      store4(dst + b, y + 2, 1.f);
    } else {
      store4(cache + r * D + a, y, p.k_scale);
      store4(cache + r * D + b, y + 2, p.k_scale);
    }
  }
  row0 += RPW * kRows;
  if (row0 >= row_end) return;
  load_rows(row0);
  }
}

template <typename T, typename KV, int D>
cudaError_t launch(const NormRopeArgs& p, cudaStream_t stream) {
  // one batch of rows a warp while that is needed to fill the SMs, then up to kBatches: a warp's
  // setup (positions, angles, weights) costs about as much as one batch
  const int64_t once = p.num_tokens * ((p.num_heads + 2 * p.num_kv_heads) / (256 / D * kRows));
  const int batches = once > kFill ? kBatches : 1;
  const int per_warp = 256 / D * kRows * batches;
  const int q_warps = (p.num_heads + per_warp - 1) / per_warp, kv_warps = (p.num_kv_heads + per_warp - 1) / per_warp;
  const int64_t ctas = (p.num_tokens * (q_warps + 2 * kv_warps) + kWarps - 1) / kWarps;
  return launch_pdl(norm_rope_write_kernel<T, KV, D>, dim3(unsigned(ctas)), dim3(kWarps * 32), 0, stream, p, q_warps,
                    kv_warps, batches);
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
