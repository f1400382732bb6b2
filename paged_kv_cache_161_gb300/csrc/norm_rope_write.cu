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
// A head row is D / 8 lanes of 8 elements, so a warp takes 256 / D rows at a time; the
// sum of squares and the rotation's partner elements travel by shuffles. A warp keeps one
// token's cos and sin in registers over kRows rows of that token, whose loads are all issued
// before the first is used.
#include <type_traits>

#include "common.cuh"
#include "launch.h"

namespace pa {
namespace {

constexpr int kWarps = 8;

// 8 consecutive elements -> fp32, as one or two 16-byte loads.
template <typename T>
struct Vec8;
template <>
struct Vec8<__nv_bfloat16> {
  uint4 a;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { a = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void unpack(float* f) const { Elem<__nv_bfloat16>::unpack(a, f); }
  __device__ __forceinline__ void copy(__nv_bfloat16* p) const { *reinterpret_cast<uint4*>(p) = a; }
  static __device__ __forceinline__ void store(__nv_bfloat16* p, const float* f, float) {
    *reinterpret_cast<uint4*>(p) = Elem<__nv_bfloat16>::pack(f);
  }
};
template <>
struct Vec8<float> {
  uint4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = reinterpret_cast<const uint4*>(p)[0];
    b = reinterpret_cast<const uint4*>(p)[1];
  }
  __device__ __forceinline__ void unpack(float* f) const {
    Elem<float>::unpack(a, f);
    Elem<float>::unpack(b, f + 4);
  }
  __device__ __forceinline__ void copy(float* p) const {
    reinterpret_cast<uint4*>(p)[0] = a;
    reinterpret_cast<uint4*>(p)[1] = b;
  }
  static __device__ __forceinline__ void store(float* p, const float* f, float) {
    reinterpret_cast<uint4*>(p)[0] = Elem<float>::pack(f);
    reinterpret_cast<uint4*>(p)[1] = Elem<float>::pack(f + 4);
  }
};
template <>
struct Vec8<Fp8E4M3> {
  // E4M3(x / scale): one binary32 division, round to nearest even, saturating (as pa_kv_write_fp8)
  static __device__ __forceinline__ void store(Fp8E4M3* p, const float* f, float scale) {
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
      w[i] = float2_to_fp8x2(__fdiv_rn(f[4 * i], scale), __fdiv_rn(f[4 * i + 1], scale)) |
             float2_to_fp8x2(__fdiv_rn(f[4 * i + 2], scale), __fdiv_rn(f[4 * i + 3], scale)) << 16;
    *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
  }
};

// T: type of q, k, v, weights and q_out; KV: cache type; kRows: rows a lane holds at once.
template <typename T, typename KV, int D, int kRows>
__global__ void __launch_bounds__(kWarps * 32) norm_rope_write_kernel(const __grid_constant__ NormRopeArgs p,
                                                                     int warps_per_token) {
  constexpr int LPR = D / 8;      // lanes per row
  constexpr int RPW = 32 / LPR;   // rows a warp holds per step
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int64_t w = int64_t(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  const int64_t t = w / warps_per_token;
  if (t >= p.num_tokens) return;
  const int sub = lane / LPR, l = lane % LPR, d0 = l * 8;
  const int Hq = p.num_heads, Hkv = p.num_kv_heads, R = Hq + 2 * Hkv;
  const int row0 = int(w - t * warps_per_token) * (RPW * kRows) + sub;

  Vec8<T> in[kRows];
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int r = row0 + i * RPW;
    if (r < R) {
      const T* src = r < Hq ? static_cast<const T*>(p.q) + t * p.q_stride + int64_t(r) * D
                     : r < Hq + Hkv ? static_cast<const T*>(p.k) + t * p.k_stride + int64_t(r - Hq) * D
                                    : static_cast<const T*>(p.v) + t * p.v_stride + int64_t(r - Hq - Hkv) * D;
      in[i].load(src + d0);
    }
  }
  const int64_t slot = __ldg(p.slot_mapping + t);

  // the token's cos and sin for this lane's 8 elements: of pairs pair0 .. (interleaved: 4 of them)
  const int rot = p.rot_dim, half = rot / 2;
  const bool rotated = d0 < rot;
  float cs[8], sn[8];
  bool bad = false;
#pragma unroll
  for (int e = 0; e < 8; ++e) cs[e] = 1.f, sn[e] = 0.f;
  {
    const int pair0 = p.interleaved ? d0 / 2 : d0 % half;
    if (p.num_axes == 1) {
      const int pos = __ldg(p.positions + t);
      bad = pos < 0 || pos >= p.max_position;
      if (rotated && !bad) {
        const float* row = p.cos_sin + int64_t(pos) * rot + pair0;
        const float4 c0 = __ldg(reinterpret_cast<const float4*>(row));
        const float4 s0 = __ldg(reinterpret_cast<const float4*>(row + half));
        cs[0] = c0.x, cs[1] = c0.y, cs[2] = c0.z, cs[3] = c0.w;
        sn[0] = s0.x, sn[1] = s0.y, sn[2] = s0.z, sn[3] = s0.w;
        if (!p.interleaved) {
          const float4 c1 = __ldg(reinterpret_cast<const float4*>(row + 4));
          const float4 s1 = __ldg(reinterpret_cast<const float4*>(row + half + 4));
          cs[4] = c1.x, cs[5] = c1.y, cs[6] = c1.z, cs[7] = c1.w;
          sn[4] = s1.x, sn[5] = s1.y, sn[6] = s1.z, sn[7] = s1.w;
        }
      }
    } else {
      int pos[kMaxAxes];
#pragma unroll
      for (int a = 0; a < kMaxAxes; ++a) {
        pos[a] = a < p.num_axes ? __ldg(p.positions + int64_t(a) * p.num_tokens + t) : 0;
        bad |= pos[a] < 0 || pos[a] >= p.max_position;
      }
      if (rotated && !bad) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          if (e >= 4 && p.interleaved) break;
          const int pair = pair0 + e;
          int at = pos[0];
#pragma unroll
          for (int a = 1; a < kMaxAxes; ++a)
            if (pair >= p.section_start[a]) at = pos[a];
          const float* row = p.cos_sin + int64_t(at) * rot + pair;
          cs[e] = __ldg(row);
          sn[e] = __ldg(row + half);
        }
      }
    }
  }
  if (bad) {  // the whole warp: one token
    if (lane == 0) raise_error(p.err, PA_DEVERR_POSITION);
    return;
  }
  const bool write = slot >= 0 && slot < p.num_slots;
  if (slot >= p.num_slots && row0 == 0 && l == 0) raise_error(p.err, PA_DEVERR_SLOT_RANGE);
  // the lane holding the partner elements (half-split pairs), or this lane
  const int hop = half / 8, partner = p.interleaved || !rotated ? lane : d0 < half ? lane + hop : lane - hop;
  const float sign = d0 < half ? -1.f : 1.f;

#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int r = row0 + i * RPW;
    if (r - sub >= R) break;  // warp-uniform: no row of this step
    float f[8];
    if (r < R) {
      in[i].unpack(f);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = 0.f;
    }
    const bool is_q = r < Hq, is_v = r >= Hq + Hkv;
    const T* weight = static_cast<const T*>(is_q ? p.q_weight : p.k_weight);
    float ss = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) ss = fmaf(f[e], f[e], ss);
#pragma unroll
    for (int m = LPR / 2; m >= 1; m >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, m);
    if (!is_v && weight) {
      const float inv = rsqrtf(ss * (1.f / D) + p.eps);
      Vec8<T> wv;
      wv.load(weight + d0);
      float wf[8];
      wv.unpack(wf);
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = f[e] * inv * wf[e];
    }
    if (p.interleaved) {
      if (!is_v && rotated) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float a = f[2 * e], b = f[2 * e + 1];
          f[2 * e] = a * cs[e] - b * sn[e];
          f[2 * e + 1] = b * cs[e] + a * sn[e];
        }
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float o = __shfl_sync(0xffffffffu, f[e], partner);
        if (!is_v && rotated) f[e] = f[e] * cs[e] + sign * o * sn[e];
      }
    }
    if (r >= R) continue;
    if (is_q) {
      Vec8<T>::store(static_cast<T*>(p.q_out) + (t * Hq + r) * D + d0, f, 1.f);
    } else if (write) {
      const int h = is_v ? r - Hq - Hkv : r - Hq;
      KV* dst = static_cast<KV*>(is_v ? p.v_cache : p.k_cache) + (slot * Hkv + h) * D + d0;
      if constexpr (std::is_same<T, KV>::value) {
        if (is_v) {  // V's bytes as they are
          in[i].copy(dst);
          continue;
        }
      }
      Vec8<KV>::store(dst, f, is_v ? p.v_scale : p.k_scale);
    }
  }
}

template <typename T, typename KV, int D>
cudaError_t launch(const NormRopeArgs& p, cudaStream_t stream) {
  constexpr int kRows = 4;
  const int rows = p.num_heads + 2 * p.num_kv_heads, per_warp = 32 / (D / 8) * kRows;
  const int wpt = (rows + per_warp - 1) / per_warp;
  const int64_t ctas = (p.num_tokens * wpt + kWarps - 1) / kWarps;
  return launch_pdl(norm_rope_write_kernel<T, KV, D, kRows>, dim3(unsigned(ctas)), dim3(kWarps * 32), 0, stream, p,
                    wpt);
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
