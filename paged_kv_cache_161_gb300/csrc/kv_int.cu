// Integer-coded caches: pa_kv_write_int quantises rows as they are written, pa_kv_read_int gives
// rows back as the values their codes stand for. [docs] PagedAttention, algorithm flow (store each
// new token's KV in its physical block); the codes have no counterpart in the pages.
//
// Both are bound by the bytes they move; a row's arithmetic is a few instructions an element.
//
// These kernels may start before the one in front of them has ended, where that one lets them (these do not), and
// read what it wrote behind griddep_wait(): none of their pointers is __restrict__ or read through __ldg.
#include "int_codes.cuh"
#include "launch.h"

namespace pa {
namespace {

// ---------------------------------------------------------------- write
// x -> the largest bfloat16 not above it / the smallest not below it (x >= 0), as float
__device__ __forceinline__ float bf16_down(float x) {
  const uint32_t u = __float_as_uint(x), t = u & 0xffff0000u;
  return __uint_as_float((u >> 31) && t != u ? t + 0x10000u : t);
}
__device__ __forceinline__ float bf16_up(float x) {
  const uint32_t u = __float_as_uint(x), t = u & 0xffff0000u;
  return __uint_as_float(t != u ? t + 0x10000u : t);
}

// NaN if either is NaN
__device__ __forceinline__ uint32_t max2_nan(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t min2_nan(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

// Eight consecutive elements of a row, and the largest and smallest of several (over LANES lanes).
template <typename T>
struct Eight;

template <>
struct Eight<__nv_bfloat16> {
  using Most = uint32_t;  // {max, -min} in one register: one shuffle and one maximum a step reduce both
  uint4 r;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { r = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ Most most() const {
    const uint32_t hi = max2_nan(max2_nan(r.x, r.y), max2_nan(r.z, r.w));
    const uint32_t lo = min2_nan(min2_nan(r.x, r.y), min2_nan(r.z, r.w)) ^ 0x80008000u;
    return max2_nan(__byte_perm(hi, lo, 0x5410), __byte_perm(hi, lo, 0x7632));
  }
  static __device__ __forceinline__ Most join(Most a, Most b) { return max2_nan(a, b); }
  template <int LANES>
  static __device__ __forceinline__ float2 range(Most m) {
#pragma unroll
    for (int d = 1; d < LANES; d <<= 1) m = max2_nan(m, __shfl_xor_sync(0xffffffffu, m, d));
    return make_float2(__uint_as_float(m << 16), -__uint_as_float(m & 0xffff0000u));
  }
  __device__ __forceinline__ void get(float* f) const { Elem<__nv_bfloat16>::unpack(r, f); }
};

template <>
struct Eight<float> {
  using Most = float2;  // {max, -min}
  float f8[8];
  __device__ __forceinline__ void load(const float* p) {
    Elem<float>::unpack(reinterpret_cast<const uint4*>(p)[0], f8);
    Elem<float>::unpack(reinterpret_cast<const uint4*>(p)[1], f8 + 4);
  }
  __device__ __forceinline__ Most most() const {
    float hi = f8[0], lo = -f8[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) {
      hi = max_nan(hi, f8[i]);
      lo = max_nan(lo, -f8[i]);
    }
    return make_float2(hi, lo);
  }
  static __device__ __forceinline__ Most join(Most a, Most b) { return make_float2(max_nan(a.x, b.x), max_nan(a.y, b.y)); }
  template <int LANES>
  static __device__ __forceinline__ float2 range(Most m) {
#pragma unroll
    for (int d = 1; d < LANES; d <<= 1) {
      m.x = max_nan(m.x, __shfl_xor_sync(0xffffffffu, m.x, d));
      m.y = max_nan(m.y, __shfl_xor_sync(0xffffffffu, m.y, d));
    }
    return make_float2(m.x, -m.y);
  }
  __device__ __forceinline__ void get(float* f) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = f8[i];
  }
};

struct WriteParams {
  const void* k;
  const void* v;
  unsigned char* k_cache;
  unsigned char* v_cache;
  const int64_t* slot_mapping;
  unsigned int* err;
  int64_t k_stride, v_stride, num_tokens, num_slots;
  uint32_t units;
  int block_size, num_kv_heads;
  int log_block;  // of a block size that is a power of two, else -1
};

// What a row's codes are made with, from its largest and smallest element: lo and step as they are stored,
// and 1 / step. With N = 2^bits - 1 (binary32 operations, rounded to nearest):
//   lo = bf16_down(min x), step = max(2^-126, bf16_up((max x - lo) / N)), inv = 1 / step,
//   code = rint((x - lo) inv)       (the product not rounded before rint: one FMA with 1.5 2^23)
// (max x - lo) inv <= N (1 + 2^-22), so no code leaves its range. A NaN or an infinity in the row,
// or a spread past the largest float, makes lo and step NaN: the row then reads back as NaN.
constexpr uint32_t kBadRow = 0x7fc07fc0u;
template <int BITS>
__device__ __forceinline__ void row_params(float2 range, uint32_t& param, float& inv) {
  const float lo = bf16_down(range.y);
  const float step = fmaxf(bf16_up(__fdiv_rn(range.x - lo, float((1 << BITS) - 1))), 1.17549435e-38f);
  const bool bad = !(fabsf(lo) < INFINITY) || !(range.x - lo < INFINITY) || !(step < INFINITY);
  param = bad ? kBadRow : (__float_as_uint(lo) >> 16) | __float_as_uint(step);
  inv = __frcp_rn(step);
}

// A warp takes U rows of one (K or V, head) a lane group: D / (8 P) lanes hold a row, each P pieces of eight
// elements, D / P apart. With U > 1 each lane makes the parameters of one of its group's rows, and the group
// shares them: the divisions are a third of a row's instructions otherwise. Instructions bound the kernel
// (16384 tokens of 8 heads x 128, 4 / 8 bits: parameters in every lane, P = 1, 25.4 / 27.7 us; shared 22.2 / 23.4;
// P = 2 16.6 / 19.1).
template <typename T, int BITS, int D, int P, int U>
__global__ void __launch_bounds__(256) kv_write_int_kernel(const WriteParams p) {
  griddep_wait();
  constexpr int LANES = D / (8 * P), ROWS = 32 / LANES, ROW = code_row_bytes<D, BITS>();
  static_assert(U <= LANES, "a lane for every row's parameters");
  constexpr uint32_t kMagic = 0x4B400000u;  // 1.5 * 2^23: adding it leaves the rounded code in the low bits
  const int lane = threadIdx.x & 31, sub = lane % LANES;
  const uint32_t unit = blockIdx.x * 8u + (threadIdx.x >> 5);
  if (unit >= p.units) return;
  const uint32_t kinds = 2u * uint32_t(p.num_kv_heads);  // heads of K, then heads of V; fastest, as in the rows' memory
  const int kind = int(unit % kinds);
  const int64_t t0 = int64_t(unit / kinds) * (ROWS * U) + lane / LANES;
  const bool is_v = kind >= p.num_kv_heads;
  const int head = is_v ? kind - p.num_kv_heads : kind;
  const int64_t stride = is_v ? p.v_stride : p.k_stride;
  const T* src = static_cast<const T*>(is_v ? p.v : p.k) + int64_t(head) * D + sub * 8 + t0 * stride;
  const int64_t rec_bytes = int64_t(p.block_size) * (ROW + 4), block_bytes = rec_bytes * p.num_kv_heads;
  unsigned char* cache = (is_v ? p.v_cache : p.k_cache) + head * rec_bytes;

  Eight<T> x[U][P];
  int64_t slot[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    slot[u] = -1;
    if (t0 + u * ROWS < p.num_tokens) {
      slot[u] = p.slot_mapping[t0 + u * ROWS];
#pragma unroll
      for (int i = 0; i < P; ++i) x[u][i].load(src + u * ROWS * stride + i * (D / P));
    } else {
#pragma unroll
      for (int i = 0; i < P; ++i) x[u][i] = {};
    }
  }
  float2 mine = make_float2(0.f, 0.f);
#pragma unroll
  for (int u = 0; u < U; ++u) {
    auto most = x[u][0].most();
#pragma unroll
    for (int i = 1; i < P; ++i) most = Eight<T>::join(most, x[u][i].most());
    const float2 r = Eight<T>::template range<LANES>(most);
    if (sub % U == u) mine = r;
  }
  uint32_t my_param;
  float my_inv;
  row_params<BITS>(mine, my_param, my_inv);
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const uint32_t param = U == 1 ? my_param : __shfl_sync(0xffffffffu, my_param, u, LANES);
    const float inv = U == 1 ? my_inv : __shfl_sync(0xffffffffu, my_inv, u, LANES);
    uint32_t w[P][2];
    // the magic's bits add up to a constant beside the shifted codes
    const float2 lo2 = make_float2(-param_lo(param), -param_lo(param)), inv2 = make_float2(inv, inv),
                 magic2 = make_float2(__uint_as_float(kMagic), __uint_as_float(kMagic));
    constexpr uint32_t kSum = BITS == 8 ? kMagic * 0x01010101u : kMagic * 0x11111111u;
#pragma unroll
    for (int i = 0; i < P; ++i) {
      float f[8];
      x[u][i].get(f);
      w[i][0] = w[i][1] = 0u;
#pragma unroll
      for (int e = 6; e >= 0; e -= 2) {
        const float2 c = ffma2v(fadd2(make_float2(f[e], f[e + 1]), lo2), inv2, magic2);
        uint32_t& to = w[i][BITS == 8 ? e / 4 : 0];
        to = (((to << BITS) + __float_as_uint(c.y)) << BITS) + __float_as_uint(c.x);
      }
      w[i][0] = param == kBadRow ? 0u : w[i][0] - kSum;
      w[i][1] = param == kBadRow ? 0u : w[i][1] - kSum;
    }
    if (slot[u] < 0) continue;
    if (slot[u] >= p.num_slots) {
      if (sub == 0) raise_error(p.err, PA_DEVERR_SLOT_RANGE);
      continue;
    }
    int64_t block;
    int at;
    if (p.log_block >= 0) {
      block = slot[u] >> p.log_block;
      at = int(slot[u]) & (p.block_size - 1);
    } else {
      block = slot[u] / p.block_size;
      at = int(slot[u] - block * p.block_size);
    }
    unsigned char* rec = cache + block * block_bytes;
    unsigned char* dst = rec + int64_t(at) * ROW + sub * BITS;
#pragma unroll
    for (int i = 0; i < P; ++i, dst += ROW / P) {
      if (BITS == 8)
        *reinterpret_cast<uint2*>(dst) = make_uint2(w[i][0], w[i][1]);
      else
        *reinterpret_cast<uint32_t*>(dst) = w[i][0];
    }
    if (sub == 0) *reinterpret_cast<uint32_t*>(rec + int64_t(p.block_size) * ROW + int64_t(at) * 4) = param;
  }
}

// ---------------------------------------------------------------- read
struct ReadParams {
  void* k_out;
  void* v_out;
  const unsigned char* k_cache;
  const unsigned char* v_cache;
  const int32_t* block_table;
  const int32_t* start_pos;  // or null: 0
  const int32_t* seq_lens;
  const int32_t* row_start_loc;
  unsigned int* err;
  int64_t num_rows, num_blocks, units;
  unsigned row_ctas;  // CTAs of the rows; those behind them check the requests
  int max_blocks_per_seq, num_seqs, block_size, num_kv_heads;
  int wide;  // the outputs are 32-byte aligned
};

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

// Sixteen codes -> values (exact but for the one rounding of the sum: step has 8 significant bits, a
// code at most 8).
template <int BITS>
__device__ __forceinline__ void decode16(const uint32_t* w, uint32_t param, float* f) {
  const float lo = param_lo(param), step = param_step(param);
  const float2 s2 = make_float2(step, step), l2 = make_float2(lo, lo), m2 = make_float2(-8388608.f, -8388608.f);
#pragma unroll
  for (int i = 0; i < 16; i += 2) {
    uint32_t a, b;  // a code over the exponent of 2^23
    if (BITS == 8) {
      a = __byte_perm(w[i / 4], 0x4B000000u, 0x7440 + i % 4);
      b = __byte_perm(w[i / 4], 0x4B000000u, 0x7440 + i % 4 + 1);
    } else {
      a = (w[i / 8] >> (4 * (i % 8)) & 15u) | 0x4B000000u;
      b = (w[i / 8] >> (4 * (i % 8) + 4) & 15u) | 0x4B000000u;
    }
    const float2 c = fadd2(make_float2(__uint_as_float(a), __uint_as_float(b)), m2);
    const float2 y = ffma2v(c, s2, l2);
    f[i] = y.x;
    f[i + 1] = y.y;
  }
}

// Whether a request's positions start .. L - 1 fit its table and its rows r0 .. r1 - 1 (of num_rows).
__device__ __forceinline__ bool fits(const ReadParams& p, int64_t r0, int64_t r1, int start, int L) {
  if (r0 < 0 || start < 0 || L < 0 || L > int64_t(p.max_blocks_per_seq) * p.block_size) return false;
  return L <= start || int64_t(L) - start <= min(r1, p.num_rows) - r0;
}

// A warp takes 32 / (head_dim / 16) consecutive output rows and COMBOS of the 2 num_kv_heads (K
// or V, head) rows of each: sixteen elements a lane. The lane's row is found once for all of them.
template <typename T, int BITS, int D, int COMBOS>
__global__ void __launch_bounds__(256) kv_read_int_kernel(const ReadParams p) {
  griddep_wait();
  constexpr int LANES = D / 16, ROWS = 32 / LANES, ROW = code_row_bytes<D, BITS>(), WORDS = BITS / 2;
  // A request that does not fit may have no row that would tell: CTAs of their own look at all of them.
  if (blockIdx.x >= p.row_ctas) {
    const int64_t s = int64_t(blockIdx.x - p.row_ctas) * 256 + threadIdx.x;
    if (s < p.num_seqs && !fits(p, p.row_start_loc[s], p.row_start_loc[s + 1], p.start_pos ? p.start_pos[s] : 0, p.seq_lens[s]))
      raise_error(p.err, PA_DEVERR_SEQ_RANGE);
    return;
  }
  const int lane = threadIdx.x & 31, sub = lane % LANES;
  const int64_t unit = int64_t(blockIdx.x) * 8 + (threadIdx.x >> 5);
  if (unit >= p.units) return;
  const int kinds = 2 * p.num_kv_heads, parts = (kinds + COMBOS - 1) / COMBOS;
  const int kind0 = int(unit % parts) * COMBOS;
  const int64_t r = unit / parts * ROWS + lane / LANES;
  if (r >= p.num_rows) return;
  // the last request that starts at or before row r (row_start_loc does not decrease)
  int s = 0, n = p.num_seqs;
  if (r < n && p.row_start_loc[r] == r && p.row_start_loc[r + 1] == r + 1) s = int(r), n = 1;  // a row a request
  while (n > 1) {
    const int half = n >> 1;
    if (p.row_start_loc[s + half] <= r) s += half, n -= half;
    else n = half;
  }
  const int64_t r0 = p.row_start_loc[s], r1 = p.row_start_loc[s + 1];
  if (r < r0 || r >= r1) return;  // a row of no request
  const int L = p.seq_lens[s], start = p.start_pos ? p.start_pos[s] : 0, B = p.block_size;
  if (!fits(p, r0, r1, start, L)) return;
  const int64_t pos = start + (r - r0);
  if (pos >= L) return;  // behind the positions asked for: left as it is
  const int64_t block = p.block_table[int64_t(s) * p.max_blocks_per_seq + pos / B];
  const int64_t at = pos % B;
  if (block < 0 || block >= p.num_blocks) {
    if (sub == 0) raise_error(p.err, PA_DEVERR_BLOCK_RANGE);
    return;
  }
  const int64_t rec_bytes = int64_t(B) * (ROW + 4), base = block * p.num_kv_heads * rec_bytes;
  uint32_t w[COMBOS][WORDS], param[COMBOS];
#pragma unroll
  for (int i = 0; i < COMBOS; ++i) {
    const int kind = kind0 + i;
    if (kind >= kinds) break;
    const bool is_v = kind >= p.num_kv_heads;
    const unsigned char* rec = (is_v ? p.v_cache : p.k_cache) + base + (is_v ? kind - p.num_kv_heads : kind) * rec_bytes;
    const unsigned char* src = rec + at * ROW + sub * (2 * BITS);
    if constexpr (BITS == 8) {
      const uint4 x = *reinterpret_cast<const uint4*>(src);
      w[i][0] = x.x, w[i][1] = x.y, w[i][2] = x.z, w[i][3] = x.w;
    } else {
      const uint2 x = *reinterpret_cast<const uint2*>(src);
      w[i][0] = x.x, w[i][1] = x.y;
    }
    param[i] = *reinterpret_cast<const uint32_t*>(rec + int64_t(B) * ROW + at * 4);
  }
#pragma unroll
  for (int i = 0; i < COMBOS; ++i) {
    const int kind = kind0 + i;
    if (kind >= kinds) break;
    const bool is_v = kind >= p.num_kv_heads;
    T* dst = static_cast<T*>(is_v ? p.v_out : p.k_out) +
             (r * p.num_kv_heads + (is_v ? kind - p.num_kv_heads : kind)) * D + sub * 16;
    float f[16];
    decode16<BITS>(w[i], param[i], f);
    if (sizeof(T) == 2) {
      store32(dst, Elem<__nv_bfloat16>::pack(f), Elem<__nv_bfloat16>::pack(f + 8), p.wide);
    } else {
      store32(dst, Elem<float>::pack(f), Elem<float>::pack(f + 4), p.wide);
      store32(dst + 8, Elem<float>::pack(f + 8), Elem<float>::pack(f + 12), p.wide);
    }
  }
}

template <typename T, int BITS, int D>
cudaError_t write_as(WriteParams p, cudaStream_t stream) {
  // several rows and pieces a lane keep more loads in flight, one spreads few rows over the SMs: from 8 warps a SM on
  constexpr int P = 2, U = sizeof(T) == 2 ? 4 : 2, MANY = 32 / (D / (8 * P)) * U, FEW = 32 / (D / 8);
  const int64_t kinds = 2 * int64_t(p.num_kv_heads);
  const bool many = p.num_tokens * kinds / MANY >= 152 * 8;
  const int64_t rows = many ? MANY : FEW;
  p.units = uint32_t((p.num_tokens + rows - 1) / rows * kinds);
  const dim3 grid((p.units + 7) / 8);
  return many ? launch_pdl(kv_write_int_kernel<T, BITS, D, P, U>, grid, dim3(256), 0, stream, p)
              : launch_pdl(kv_write_int_kernel<T, BITS, D, 1, 1>, grid, dim3(256), 0, stream, p);
}

template <typename T, int BITS, int D>
cudaError_t read_as(ReadParams p, cudaStream_t stream) {
  constexpr int ROWS = 32 / (D / 16);
  const int64_t groups = (p.num_rows + ROWS - 1) / ROWS, kinds = 2 * int64_t(p.num_kv_heads);
  // eight (K or V, head) rows a lane where that leaves 8 warps a SM, else four (8 heads x 128, 4 bits: 16384 rows 15.8
  // against 17.1 us, 256 rows 3.75 against 3.1 us)
  const bool many = groups * ((kinds + 7) / 8) >= 152 * 8;
  p.units = groups * (many ? (kinds + 7) / 8 : (kinds + 3) / 4);
  p.row_ctas = unsigned((p.units + 7) / 8);
  const dim3 grid(p.row_ctas + (unsigned(p.num_seqs) + 255u) / 256u);
  return many ? launch_pdl(kv_read_int_kernel<T, BITS, D, 8>, grid, dim3(256), 0, stream, p)
              : launch_pdl(kv_read_int_kernel<T, BITS, D, 4>, grid, dim3(256), 0, stream, p);
}

// f<T, BITS, D>(args) for the call's type, width and head_dim (checked before)
#define PA_INT_DISPATCH(f, dtype, bits, D, ...)                                                                \
  (dtype == PA_BF16                                                                                            \
       ? (bits == 4 ? (D == 64 ? f<__nv_bfloat16, 4, 64>(__VA_ARGS__) : f<__nv_bfloat16, 4, 128>(__VA_ARGS__)) \
                    : (D == 64 ? f<__nv_bfloat16, 8, 64>(__VA_ARGS__) : f<__nv_bfloat16, 8, 128>(__VA_ARGS__))) \
       : (bits == 4 ? (D == 64 ? f<float, 4, 64>(__VA_ARGS__) : f<float, 4, 128>(__VA_ARGS__))                 \
                    : (D == 64 ? f<float, 8, 64>(__VA_ARGS__) : f<float, 8, 128>(__VA_ARGS__))))

}  // namespace

cudaError_t launch_kv_write_int(const KvIntArgs& a, const void* k, const void* v, int64_t k_stride, int64_t v_stride,
                                void* k_cache, void* v_cache, const int64_t* slot_mapping, int64_t num_tokens,
                                cudaStream_t stream) {
  int log_block = -1;
  if ((a.block_size & (a.block_size - 1)) == 0)
    for (log_block = 0; (1 << log_block) < a.block_size;) ++log_block;
  const WriteParams p = {k, v, static_cast<unsigned char*>(k_cache), static_cast<unsigned char*>(v_cache), slot_mapping,
                         a.err, k_stride, v_stride, num_tokens, a.num_blocks * a.block_size, 0u, a.block_size,
                         a.num_kv_heads, log_block};
  return PA_INT_DISPATCH(write_as, a.dtype, a.bits, a.head_dim, p, stream);
}

cudaError_t launch_kv_read_int(const KvIntArgs& a, void* k_out, void* v_out, const void* k_cache, const void* v_cache,
                               const int32_t* block_table, int max_blocks_per_seq, const int32_t* start_pos,
                               const int32_t* seq_lens, const int32_t* row_start_loc, int num_seqs, int64_t num_rows,
                               cudaStream_t stream) {
  const bool wide = (reinterpret_cast<uintptr_t>(k_out) | reinterpret_cast<uintptr_t>(v_out)) % 32 == 0;
  const ReadParams p = {k_out, v_out, static_cast<const unsigned char*>(k_cache),
                        static_cast<const unsigned char*>(v_cache), block_table, start_pos, seq_lens, row_start_loc,
                        a.err, num_rows, a.num_blocks, 0, 0u, max_blocks_per_seq, num_seqs, a.block_size, a.num_kv_heads,
                        wide ? 1 : 0};
  return PA_INT_DISPATCH(read_as, a.dtype, a.bits, a.head_dim, p, stream);
}

}  // namespace pa
