// Attention of a few new tokens over integer-coded caches (pa_attention_int): [docs] PagedAttention
// (attention over a block table); [flow] 3.5. The codes have no counterpart in the pages.
//
// With key row j = lo_j + step_j c_j and value row j = lo'_j + step'_j c'_j (codes c, c'):
//   s_j = scale q.k_j = scale (step_j (q.c_j) + lo_j sum(q)),     p_j = 2^(s_j log2 e - m)
//   out = (sum_j (p_j step'_j) (c'_j - mid) + sum_j p_j (lo'_j + mid step'_j)) / sum_j p_j
// so the tensor cores multiply whole codes, and a row's two parameters cost a few instructions a
// logit instead of one an element. mid is half the codes' range: the codes enter the second product as
// small whole numbers around 0, so that an average over many rows does not come out as the
// difference of two large sums.
//
// Bound: the cache's bytes (68 a row and head at 128 elements of 4 bits), and the instructions that turn
// codes into 16-bit operands, about one an element of K and V. So: one pass, and every element converted once
// for up to 8 or 16 query rows. Measured (GB300, 32 / 8 heads x 128): 64 requests of 32768 keys, 8 bits,
// 648 to 670 us, 6640 GB/s of cache or more, 0.98 of the measured copy rate; 256 requests of 16 to 8192 keys around
// 1024, 4 bits, 99 us, 4770 GB/s (4 bits are bound by instructions, latency and what comes before and behind the stream).
//
// Work: a unit is unit_keys keys of one segment (request, KV head, tile of 8 or 16 query rows: query tokens
// x the head's query heads). The units of all segments, in order, are dealt to the grid's warps in
// equal runs; a warp streams its run through a ring of its own in shared memory, and no warp waits for
// another while it streams. Segments cut between warps leave pieces (m, l, unnormalised output), the one
// that ends a run where the warp's ring was (in the workspace like the others: one request of 2000 keys
// took 15.8 us, so 12.3): a CTA joins those of its warps, a second kernel those cut between CTAs, which are in the
// workspace.
//
// Operands (mma.sync m16n8k16, keys as the 16 rows, query rows as the 8 columns): a code under the
// bits of the f16 1024 is that number plus the code (or 1024 + 16 c, a nibble higher), one logic
// instruction for two, and half an addition more where the 1024 has to go before the products. Which
// dimension sits where in a contraction is free as long as both sides agree, so a lane takes 16-byte pieces
// of rows as they lie; so is which key is which row.
//
// The kernels may start before the one in front of them has ended, where that one lets them (these do not), and
// read what it wrote behind griddep_wait(): none of their pointers is __restrict__ or read through __ldg.
#include <type_traits>

#include "int_codes.cuh"
#include "launch.h"
#include "mma.cuh"

namespace pa {
namespace {

// A tile of query rows is NT times the 8 columns of an MMA. NT = 2 where a request has more than 8 rows a KV
// head: the codes are converted once for 16, with 8 warps a CTA (their sums take 250 registers a thread)
// instead of 12 (two requests of four drafted tokens, 40000 keys: 4 bits 45 us with two tiles of 8, 43 us with
// one of 16, 8 bits 52 and 45 us; 160000 keys: 132 and 113 us, 162 and 120 us).
template <int NT>
__host__ __device__ constexpr int num_warps() { return NT == 1 ? 12 : 8; }
template <int NT>
__host__ __device__ constexpr int num_rows() { return 8 * NT; }
constexpr float kNoMax = -1e30f;  // running maximum before any key: finite, so that differences are not NaN

constexpr int kPart = 32;  // keys of a copy at most
template <int BITS>
__host__ __device__ constexpr int unit_keys() { return BITS == 4 ? 64 : 32; }
// A segment's start in units of keys, by the time it takes (256 requests of 16 to 8192 keys around 1024, 4
// bits: 0 units 122 us, 1 108, 2 99, 4 105; 8 bits: 0 units 170 us, 1 161, 2 158, 4 159)
template <int KU>
__host__ __device__ constexpr int start_units() { return 2; }
template <int D, int NT>
__host__ __device__ constexpr int num_stages() { return D == 128 && NT == 1 ? 2 : 3; }  // of a warp's ring
template <int D, int BITS>
__host__ __device__ constexpr int stage_bytes() { return unit_keys<BITS>() * 2 * (code_row_bytes<D, BITS>() + 4); }
// a piece: a tile's rows of D sums, then their maxima and their sums of numerators
template <int D, int NT>
__host__ __device__ constexpr int piece_floats() { return num_rows<NT>() * (D + 2); }

struct IntParams {
  __nv_bfloat16* out;
  const __nv_bfloat16* q;
  const unsigned char* k_cache;
  const unsigned char* v_cache;
  const int32_t* block_table;
  const int32_t* seq_lens;
  const int32_t* qsl;
  unsigned int* err;
  float* pieces;  // [grid * kWarps] of the warps, then [grid * 2] of the CTAs
  int4* descs;    // [grid * 2]: a CTA's pieces, {first unit of the segment or -1, its last + 1, rows_of's two}
  int* total;     // units of the call
  int64_t num_blocks;
  int max_blocks_per_seq, num_seqs, num_tokens, max_query_len, max_seq_len;
  int num_heads, num_kv_heads, group, block_size;
  int part;    // keys a copy of codes covers: the largest power of two in block_size, at most kPart
  float scale_log2;
};

// What a request contributes: `tiles` tiles of rows, each a segment of `span` units a KV head: start_units
// that stand for a segment's start (its queries, table, sums: none of them is work of its own), then
// those of its keys.
struct Request {
  int q0, q_len, L, tiles, span;
};

template <int KU, int NT>
__device__ __forceinline__ bool request_of(const IntParams& p, int s, Request& r) {
  r.q0 = p.qsl[s];
  const int q1 = p.qsl[s + 1];
  r.L = p.seq_lens[s];
  r.tiles = r.span = r.q_len = 0;
  if (r.q0 < 0 || q1 < r.q0 || q1 > p.num_tokens) return false;
  r.q_len = q1 - r.q0;
  if (r.q_len == 0) return true;
  if (r.q_len > p.max_query_len || r.q_len > r.L || r.L > p.max_seq_len) return false;
  r.tiles = int((int64_t(r.q_len) * p.group + num_rows<NT>() - 1) / num_rows<NT>());
  r.span = start_units<KU>() + (r.L + KU - 1) / KU;
  return true;
}

// The segment that holds unit u of the whole call: request s by search in the units' prefix.
struct Segment {
  int s, head, tile, begin, end;  // units [begin, end) of the call
};
template <int KU, int NT>
__device__ __forceinline__ Segment segment_of(const IntParams& p, const int* prefix, int u) {
  int s = 0, n = p.num_seqs;
  while (n > 1) {
    const int half = n >> 1;
    if (prefix[s + half] <= u) s += half, n -= half;
    else n = half;
  }
  Request r;
  request_of<KU, NT>(p, s, r);
  const int seg = (u - prefix[s]) / r.span;
  Segment g;
  g.s = s;
  g.head = seg / r.tiles;
  g.tile = seg - g.head * r.tiles;  // tiles fastest: neighbours read the same keys
  g.begin = prefix[s] + seg * r.span;
  g.end = g.begin + r.span;
  return g;
}

// Words of a stage, read as ordinary memory: the compiler may move them between the waits.
__device__ __forceinline__ uint32_t shared_word(const unsigned char* p) { return *reinterpret_cast<const uint32_t*>(p); }
template <int N>
__device__ __forceinline__ void shared_words(const unsigned char* p, uint32_t* w) {
  if constexpr (N == 4) {
    const uint4 x = *reinterpret_cast<const uint4*>(p);
    w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
  } else if constexpr (N == 2) {
    const uint2 x = *reinterpret_cast<const uint2*>(p);
    w[0] = x.x, w[1] = x.y;
  } else {
    w[0] = shared_word(p);
  }
}

// The first unit of warp w: runs of two sizes, one unit apart, spread evenly over the grid; with fewer units
// than warps, one for each of the first warps (only runs behind the last are empty: the joins rely on it).
struct Deal {
  int each, rest, warps;
  __device__ __forceinline__ Deal(int total, int n) : each(total / n), rest(total % n), warps(n) {}
  __device__ __forceinline__ int operator()(int w) const {
    return each == 0 ? min(w, rest) : w * each + int(uint32_t(w) * uint32_t(rest) / uint32_t(warps));
  }
};

__device__ __forceinline__ void copy16(uint32_t dst, const unsigned char* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>  // all but the last N groups have landed
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }
__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }
// (x & mask) | bits in one instruction: two immediates take two, so `bits` comes in a register.
__device__ __forceinline__ uint32_t and_or(uint32_t x, uint32_t mask, uint32_t bits) {
  uint32_t d;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(d) : "r"(x), "r"(mask), "r"(bits));
  return d;
}

__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return ffma2v(a, b, make_float2(0.f, 0.f)); }
__device__ __forceinline__ uint32_t movm(uint32_t x) {
  uint32_t d;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(x));
  return d;
}
__device__ __forceinline__ uint32_t h2(uint32_t x, __half2 mul, __half2 add) {
  const __half2 r = __hfma2(*reinterpret_cast<const __half2*>(&x), mul, add);
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t h2(uint32_t x, __half2 add) {
  const __half2 r = __hadd2(*reinterpret_cast<const __half2*>(&x), add);
  return *reinterpret_cast<const uint32_t*>(&r);
}

// The key of a 16-key tile that is row r of the contraction: even r < 8 the keys 0 .. 3, odd ones 5, 4, 7,
// 6, and 8 more from r = 8 on. A quarter warp's 16-byte loads of key rows then meet rows of both
// parities, and so do the half warps' 8-byte loads of value rows.
__device__ __forceinline__ int key_of(int r) {
  const int h = (r & 7) >> 1;
  return (r & 8) + ((r & 1) ? (h ^ 1) + 4 : h);
}

// Where a tile's rows go: {token of its first row, that row's query head << 5 | number of rows}.
template <int NT>
__device__ __forceinline__ int2 rows_of(const IntParams& p, const Request& r, const Segment& sg) {
  const int rr = sg.tile * num_rows<NT>(), rows = min(num_rows<NT>(), r.q_len * p.group - rr);
  return make_int2(r.q0 + rr / p.group, int(uint32_t(sg.head * p.group + rr % p.group) << 5 | uint32_t(rows)));
}
__device__ __forceinline__ __nv_bfloat16* out_row(const IntParams& p, int2 where, int row, int D) {
  const int head = int(uint32_t(where.y) >> 5), first = head % p.group, rr = first + row;
  return p.out + (int64_t(where.x + rr / p.group) * p.num_heads + head - first + rr % p.group) * D;
}

// Joins `count` pieces, piece k at at(k), of one row of a tile for every G lanes of the warp: into the
// output, or into the piece `to`. The pieces' maxima and sums come a lane a piece, then the rows, a few pieces
// at a time: little code, which is met cold, and few waits.
template <int D, int G, int NT, typename At>
__device__ __forceinline__ void join_rows(const IntParams& p, int2 where, int row, int lane, int count, At at, float* to) {
  constexpr int kRows = num_rows<NT>();
  constexpr int E = D / G;  // a lane's elements, four (two) at a time
  constexpr int V = E >= 4 ? 4 : 2;
  const int sub = lane % G;
  const bool mine = row < (where.y & 31);  // a row of the request
  float m = kNoMax, l = 0.f, o[E];
#pragma unroll
  for (int e = 0; e < E; ++e) o[e] = 0.f;
#pragma unroll 1
  for (int k0 = 0; k0 < count; k0 += G) {
    const int k = k0 + sub;
    const bool live = mine && k < count;
    const float* ml = at(live ? k : 0) + kRows * D + row;
    const float mk = live ? ml[0] : kNoMax, lk = live ? ml[kRows] : 0.f;
    float top = lk == 0.f ? kNoMax : mk;  // an empty piece: its other sums were never written
#pragma unroll
    for (int x = 1; x < G; x <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
    top = fmaxf(top, m);
    const float w = lk == 0.f ? 0.f : exp2f(mk - top), before = exp2f(m - top);
    float sum = lk * w;
#pragma unroll
    for (int x = 1; x < G; x <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
    l = l * before + sum;
    m = top;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] *= before;
#pragma unroll(G == 32 ? 4 : 2)
    for (int j = 0; j < min(G, count - k0); ++j) {
      const float e0 = __shfl_sync(0xffffffffu, w, j, G);
      const float* x = at(k0 + j) + row * D + sub * V;
#pragma unroll
      for (int e = 0; e < E; e += V) {
        float y[V];
        if constexpr (V == 4) {
          const float4 f = *reinterpret_cast<const float4*>(x + e * G);
          y[0] = f.x, y[1] = f.y, y[V - 2] = f.z, y[V - 1] = f.w;
        } else {
          const float2 f = *reinterpret_cast<const float2*>(x + e * G);
          y[0] = f.x, y[1] = f.y;
        }
#pragma unroll
        for (int i = 0; i < V; ++i) o[e + i] = e0 == 0.f ? o[e + i] : fmaf(e0, y[i], o[e + i]);
      }
    }
  }
  if (!mine) return;
  if (to) {
    if (sub == 0) {
      to[kRows * D + row] = m;
      to[kRows * D + kRows + row] = l;
    }
#pragma unroll
    for (int e = 0; e < E; ++e) to[row * D + sub * V + e / V * (V * G) + e % V] = o[e];
  } else {
    __nv_bfloat16* out = out_row(p, where, row, D) + sub * V;
    const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
#pragma unroll
    for (int e = 0; e < E; e += V) {
      if constexpr (V == 4)
        *reinterpret_cast<uint2*>(out + e * G) = make_uint2(pack_bf16(o[e] * inv, o[e + 1] * inv), pack_bf16(o[e + 2] * inv, o[e + 3] * inv));
      else
        *reinterpret_cast<uint32_t*>(out + e * G) = pack_bf16(o[e] * inv, o[e + 1] * inv);
    }
  }
}

// B16: blocks of 16 tokens, whose copies are all of one known size (256 requests of 1024 keys, 4 bits: 81 us
// without, 70 us with; two requests of four drafts, 40000 keys, 8 bits: 50, 45 us). In other blocks, 4 / 8 bits: of 8 98 / 108 us, of
// 32 to 128 74 to 76 / 102 us.
template <int D, int BITS, bool B16, int NT>
__global__ void __launch_bounds__(num_warps<NT>() * 32, 1) attention_int_kernel(const IntParams p) {
  constexpr int kWarps = num_warps<NT>(), kRows = num_rows<NT>();
  constexpr int KU = unit_keys<BITS>(), ROW = code_row_bytes<D, BITS>();
  constexpr int STAGE = stage_bytes<D, BITS>(), STAGES = num_stages<D, NT>();
  static_assert(STAGE % 16 == 0 && STAGES * STAGE >= piece_floats<D, NT>() * 4, "a warp's last piece takes its ring's place");
  constexpr int HALF = STAGE / 2;                   // keys' part of a stage, then the values'
  constexpr int NK = D / 16;                        // contraction steps of q.c, and tiles of 16 value dimensions
  constexpr float kMid = BITS == 4 ? 8.f : 128.f;
  // the codes in q.c are c (4 bits, even nibbles), 64 + c (odd ones), or 1024 + c: 64 or 1024 times the sum of
  // their q leaves again in fp32
  constexpr float kOffset = BITS == 4 ? 64.f : 1024.f;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ int wsum[kWarps];
  __shared__ int4 desc[kWarps * 2];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int S = p.num_seqs;
  // shared memory: the warps' rings, the units' prefix over the requests
  unsigned char* ring = smem + warp * STAGES * STAGE;
  int* prefix = reinterpret_cast<int*>(smem + kWarps * STAGES * STAGE);
  if (threadIdx.x < kWarps * 2) desc[threadIdx.x] = make_int4(-1, 0, 0, 0);
  griddep_wait();

  // ---- the plan: units of every request, their prefix, this warp's run. Sums stop at 2^31 - 1, which only
  // requests that lie over one another in query_start_loc can reach.
  auto add = [](int a, int b) { return int(min(uint32_t(a) + uint32_t(b), 0x7fffffffu)); };
  int total = 0;
  for (int b = 0; b < S; b += kWarps * 32) {
    const int s = b + threadIdx.x;
    int x = 0;
    if (s < S) {
      Request r;
      if (!request_of<KU, NT>(p, s, r) && blockIdx.x == 0) raise_error(p.err, PA_DEVERR_SEQ_RANGE);
      x = r.tiles * r.span * p.num_kv_heads;
    }
    int inc = x;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, inc, d);
      if (lane >= d) inc = add(inc, y);
    }
    const int before = __shfl_up_sync(0xffffffffu, inc, 1);
    if (lane == 31) wsum[warp] = inc;
    __syncthreads();
    int off = total, sum = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) off = add(off, wsum[w]);
      sum = add(sum, wsum[w]);
    }
    if (s < S) prefix[s] = lane ? add(off, before) : off;
    total = add(total, sum);
    __syncthreads();
  }
  if (total == 0x7fffffff) {
    if (blockIdx.x == 0 && threadIdx.x == 0) raise_error(p.err, PA_DEVERR_SEQ_RANGE);
    total = 0;
  }
  const int num_warps = gridDim.x * kWarps;
  const int w0 = blockIdx.x * kWarps;
  const Deal first(total, num_warps);
  const int u0 = first(w0 + warp), u1 = first(w0 + warp + 1);
  if (blockIdx.x == 0 && threadIdx.x == 0) *p.total = total;
  const int64_t rec_bytes = int64_t(p.block_size) * (ROW + 4);

  // ---- the run's units of keys in order, each into the next stage of the ring: asynchronous copies of 16
  // bytes a lane, one group a unit (an empty one behind the last). Every `part` keys come as the records of K
  // and V, or as their codes and parameters where a block holds more than that. Block and offset are
  // stepped along: no division a unit. (One bulk copy a record instead took 25 to 45 instructions each for
  // its uniform operands, a fifth of all.)
  struct {
    int u, seg_end = 0, x = 0, units = 0, blocks = 0, b0 = 0, ent = 0, ent_next = 0;
    int b = 0, in = 0;  // block and offset of the next piece
    int stage = 0;
    bool any_missing = false;  // a block id out of range has been met
    const int32_t* row = nullptr;
    int64_t head_off = 0;
  } pr;
  pr.u = u0;
  const bool fused = p.part == p.block_size;  // a record is one run of bytes
  const int part = B16 ? 16 : p.part, part_bytes = part * (ROW + 4);
  const int64_t block_bytes = int64_t(p.num_kv_heads) * rec_bytes;
  auto entry = [&](int b) { return b < pr.blocks ? pr.row[b] : -1; };
  // the next 32 table entries, read a batch ahead; -1 for a block that is not there
  auto next_entries = [&](int b0) {
    pr.b0 = b0;
    pr.ent = pr.ent_next;
    pr.ent_next = entry(b0 + 32 + lane);
    const bool bad = b0 + lane < pr.blocks && (pr.ent < 0 || pr.ent >= p.num_blocks);
    if (bad) {
      raise_error(p.err, PA_DEVERR_BLOCK_RANGE);
      pr.ent = -1;
    }
    if (__any_sync(0xffffffffu, bad)) pr.any_missing = true;
  };
  auto locate = [&]() {  // the segment of pr.u, past its start; false: the run ends before its keys
    const Segment sg = segment_of<KU, NT>(p, prefix, pr.u);
    pr.u = max(pr.u, sg.begin + start_units<KU>());
    if (pr.u >= u1) return false;
    Request r;
    request_of<KU, NT>(p, sg.s, r);
    // keys the tile's last row sees, and the blocks and units that hold them
    const int rows = min(kRows, r.q_len * p.group - sg.tile * kRows), last = (sg.tile * kRows + rows - 1) / p.group;
    const int n = r.L - r.q_len + last + 1;
    pr.seg_end = sg.end;
    pr.x = pr.u - sg.begin - start_units<KU>();
    pr.units = (n + KU - 1) / KU;
    pr.blocks = (n + p.block_size - 1) / p.block_size;
    pr.row = p.block_table + int64_t(sg.s) * p.max_blocks_per_seq;
    pr.head_off = int64_t(sg.head) * rec_bytes;
    pr.b = pr.x * KU / p.block_size;
    pr.in = pr.x * KU - pr.b * p.block_size;
    pr.ent_next = entry(pr.b + lane);
    next_entries(pr.b);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {  // the queries, read when the segment's turn comes
      const int rr = sg.tile * kRows + min(g + 8 * nt, rows - 1);
      prefetch_l2(p.q + (int64_t(r.q0 + rr / p.group) * p.num_heads + sg.head * p.group + rr % p.group) * D + t * (D / 4));
    }
    return true;
  };
  // bytes (a multiple of 16, at most a piece's) of K and of V, 512 a step, of which all but the last are full
  auto copy = [&](unsigned char* dst, const unsigned char* k_src, const unsigned char* v_src, int bytes) {
    constexpr int STEPS = (kPart * (ROW + 4) + 511) / 512;
    const uint32_t to = smem_u32(dst) + lane * 16;
    k_src += lane * 16;
    v_src += lane * 16;
#pragma unroll
    for (int j = 0; j < STEPS; ++j) {
      if (j * 512 >= bytes) break;
      if (j * 512 + lane * 16 < bytes) {
        copy16(to + j * 512, k_src + j * 512);
        copy16(to + HALF + j * 512, v_src + j * 512);
      }
    }
  };
  auto fill = [&]() {
    if (pr.u < u1 && (pr.u < pr.seg_end || locate())) {
      if (pr.x < pr.units) {
        unsigned char* dst = ring + pr.stage * STAGE;
        if (B16) {
          if (pr.b >= pr.b0 + 32) next_entries(pr.b0 + 32);  // (batches begin and end with a unit)
#pragma unroll
          for (int k = 0; k < KU / 16; ++k) {
            const int block = __shfl_sync(0xffffffffu, pr.ent, pr.b - pr.b0 + k);
            const int64_t off = int64_t(block) * block_bytes + pr.head_off;
            if (block >= 0) copy(dst + k * 16 * (ROW + 4), p.k_cache + off, p.v_cache + off, 16 * (ROW + 4));
          }
          pr.b += KU / 16;
        } else {
#pragma unroll 1
          for (int k = 0; k < KU; k += p.part, dst += part_bytes) {
            if (pr.b >= pr.b0 + 32) next_entries(pr.b0 + 32);
            const int block = __shfl_sync(0xffffffffu, pr.ent, pr.b - pr.b0);
            if (block >= 0) {
              const int64_t off = int64_t(block) * block_bytes + pr.head_off;
              const unsigned char *k_rec = p.k_cache + off, *v_rec = p.v_cache + off;
              const int c = pr.in * ROW;
              copy(dst, k_rec + c, v_rec + c, fused ? part_bytes : p.part * ROW);
              if (!fused && lane * 4 < p.part) {  // the rows' parameters lie behind all the block's codes
                const int w = p.block_size * ROW + pr.in * 4 + lane * 16;  // (blocks of 2^20 tokens at most)
                const uint32_t to = smem_u32(dst) + p.part * ROW + lane * 16;
                copy16(to, k_rec + w);
                copy16(to + HALF, v_rec + w);
              }
            }
            pr.in += p.part;
            if (pr.in == p.block_size) {
              pr.in = 0;
              ++pr.b;
            }
          }
        }
      }
      ++pr.x;
      ++pr.u;
      if (++pr.stage == STAGES) pr.stage = 0;
    }
    copies_commit();
  };

  // ---- where a lane's rows lie in a stage: keys key_of(g), key_of(g + 8) of a tile as rows of K,
  // keys key_of(2t), (2t + 1), (2t + 8), (2t + 9) as rows of V; the second tile `next` bytes on
  auto code_at = [&](int key) { return key / part * part_bytes + key % part * ROW; };
  auto param_at = [&](int key) { return key / part * part_bytes + part * ROW + key % part * 4; };
  constexpr int kLane = BITS == 4 ? D / 8 : 16;  // bytes of a key row a lane takes at once
  int k_at[2], v_at[4], par_at[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    k_at[i] = code_at(key_of(g + 8 * i)) + t * kLane;
    par_at[i] = param_at(key_of(g + 8 * i));
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) v_at[i] = HALF + code_at(key_of(2 * t + (i & 1) + 8 * (i >> 1))) + g * (ROW / 8);
  const int next_code = B16 ? 16 * (ROW + 4) : part >= 32 ? 16 * ROW : 16 / min(part, 16) * part_bytes;
  const int next_param = !B16 && part >= 32 ? 64 : next_code;

  uint32_t C;  // two f16 1024s
  asm volatile("mov.b32 %0, 0x64006400;" : "=r"(C));
  // The last free stage is filled before the next unit, behind a segment's end and the next one's queries: the
  // first units come sooner than with a filling behind each unit (256 requests of 16 to 8192 keys, 4 bits: 99.3 us, 98.5
  // so; two requests of four drafts, 160000 keys: 112.7 both ways).
  int stage = 0;
  bool filled = false;
  for (int u = u0; u < u1;) {
    // ---- a segment of the run: units x0 .. x1 - 1 of its keys
    const Segment sg = segment_of<KU, NT>(p, prefix, u);
    Request r;
    request_of<KU, NT>(p, sg.s, r);
    const int rows = min(kRows, r.q_len * p.group - sg.tile * kRows);
    const int x0 = max(u - sg.begin - start_units<KU>(), 0), x1 = min(sg.end, u1) - sg.begin - start_units<KU>();
    const bool whole = u <= sg.begin && u1 >= sg.end;
    const int slot = u == u0 ? 0 : 1;
    u = min(sg.end, u1);
    const int2 where = rows_of<NT>(p, r, sg);
    if (!whole && lane == 0) desc[warp * 2 + slot] = make_int4(sg.begin, sg.end, where.x, where.y);
    // a piece that ends the run goes where the ring was, else (the first of a run that goes on) to memory
    float* piece = u == u1 ? reinterpret_cast<float*>(ring) : p.pieces + int64_t(w0 + warp) * piece_floats<D, NT>();
    if (x1 <= x0) {  // nothing but the start, which ends the run: an empty piece
      if (lane < 2 * kRows) piece[kRows * D + lane] = lane < kRows ? kNoMax : 0.f;  // (32 at most)
      continue;
    }
    const int j_first = sg.tile * kRows / p.group, j_last = (sg.tile * kRows + rows - 1) / p.group;
    const int n_min = r.L - r.q_len + j_first + 1, n_max = r.L - r.q_len + j_last + 1;  // keys the rows see
    // Query row g (g + 8) of the tile as f16 with its largest element in [2^14, 2^15): a power of two, so exact
    // but for elements 2^24 times smaller than the row's largest. Its factor goes back in with the logits' scale
    // before the row parameters do: q.c scale and sum(q) scale have the logits' own range, however
    // large the keys and small the queries.
    uint32_t qb[NT][NK][2];
    // of query rows 2t and 2t + 1 (and 8 on), whose logits this lane holds
    float qs[NT][2], off[NT][2], fac[NT][2], m[NT][2], l[NT][2], mid[NT][2];
    int lim[NT][2];
    uint4 raw[NT][D / 32];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int rr = sg.tile * kRows + min(g + 8 * nt, rows - 1);
      const __nv_bfloat16* src = p.q + (int64_t(r.q0 + rr / p.group) * p.num_heads + sg.head * p.group + rr % p.group) * D;
#pragma unroll
      for (int i = 0; i < D / 32; ++i)  // the dimensions of the key row's pieces that this lane takes
        raw[nt][i] = *reinterpret_cast<const uint4*>(src + (BITS == 4 ? t * (D / 4) + 8 * i : (i / 2) * 64 + t * 16 + (i & 1) * 8));
    }
    if (!filled) {  // behind the first queries' loads, which would wait for all the copies otherwise
      filled = true;
#pragma unroll 1
      for (int i = 0; i < STAGES - 1; ++i) fill();
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int row = g + 8 * nt;
      float f[D / 4], qsum = 0.f, qoff = 0.f, big = 0.f;
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        Elem<__nv_bfloat16>::unpack(raw[nt][i], f + 8 * i);
#pragma unroll
        for (int e = 0; e < 8; ++e) big = fmaxf(big, fabsf(f[8 * i + e]));
      }
      big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
      big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
      // the biased exponent; 255: left unscaled. 2^113 turns the smallest bfloat16 into 16 times the smallest
      // f16 (odd elements of 4-bit rows are divided by 16 below), so no row needs more, and the factor's inverse
      // stays a normal number.
      const int ex = int(__float_as_uint(big) >> 23);
      const int shift = (ex == 255 || row >= rows) ? 0 : min(113, 14 - (ex - 127));
      const float mul = row >= rows ? 0.f : __uint_as_float(uint32_t(shift + 127) << 23);
      const float qfactor = p.scale_log2 * exp2f(float(-shift));
#pragma unroll
      for (int i = 0; i < D / 4; ++i) {
        f[i] = __half2float(__float2half_rn(f[i] * mul));
        qsum += f[i];
        if (BITS == 8 || (i & 1)) qoff += f[i];
      }
      if (row >= rows) qsum = qoff = 0.f;
#pragma unroll
      for (int d = 1; d < 4; d <<= 1) {
        qoff += __shfl_xor_sync(0xffffffffu, qoff, d);
        qsum += __shfl_xor_sync(0xffffffffu, qsum, d);
      }
#pragma unroll
      for (int k = 0; k < NK; ++k) {
        if (BITS == 4) {  // word k / 2 of the lane's piece: elements (0, 4), (1, 5), then (2, 6), (3, 7)
          const float* e = f + 8 * (k / 2) + 2 * (k & 1);
          qb[nt][k][0] = pack_f16(e[0], e[4]);
          qb[nt][k][1] = pack_f16(e[1] * 0.0625f, e[5] * 0.0625f);  // their codes come 16-fold
        } else {
          qb[nt][k][0] = pack_f16(f[4 * k], f[4 * k + 1]);
          qb[nt][k][1] = pack_f16(f[4 * k + 2], f[4 * k + 3]);
        }
        if (row >= rows) qb[nt][k][0] = qb[nt][k][1] = 0u;
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        fac[nt][h] = __shfl_sync(0xffffffffu, qfactor, (2 * t + h) * 4);
        qs[nt][h] = __shfl_sync(0xffffffffu, qsum, (2 * t + h) * 4) * fac[nt][h];
        off[nt][h] = -kOffset * __shfl_sync(0xffffffffu, qoff, (2 * t + h) * 4);
        m[nt][h] = kNoMax;
        l[nt][h] = mid[nt][h] = 0.f;
        lim[nt][h] = r.L - r.q_len + (sg.tile * kRows + min(8 * nt + 2 * t + h, rows - 1)) / p.group + 1;
      }
    }
    float o[NT][NK][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < NK; ++i) o[nt][i][0] = o[nt][i][1] = o[nt][i][2] = o[nt][i][3] = 0.f;
    // Numerators times value steps enter the second product as f16 (rounded to 2^-11 relative at most: an
    // eighth of the output's own rounding), scaled by a power of two a query row, wscale, that keeps the products
    // below 2^15 and the largest of them so far at 2^3 or more: what rounds to nothing is 2^-28 of that one,
    // whatever the steps of rows without weight.
    float wscale[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) wscale[nt][0] = wscale[nt][1] = __uint_as_float(253u << 23);

    // tiles tile0 .. of a stage whose keys start at key0: all of a whole unit's, or one with masks (small
    // code: the two together have to stay in the instruction cache) or blocks to look up
    auto unit = [&](const unsigned char* st, int key0, int tile0, auto tail_c) {
      constexpr bool kTail = decltype(tail_c)::value;
      constexpr int TILES = kTail ? 1 : NT == 1 ? KU / 16 : 2;
      // ---- q.c of 16 keys x 8 NT query rows a tile, all tiles before their logits: independent chains, two a
      // product with NT = 1
      float s[TILES][NT][4], s1[TILES][4];
      uint32_t pk[TILES][2], pv[TILES][2];
#pragma unroll
      for (int tile = 0; tile < TILES; ++tile) {
        const int at = tile0 + tile;
        const unsigned char* two = st + (at >> 1) * (32 * (ROW + 4));  // pieces are at most 32 keys
        const unsigned char *base = two + (at & 1) * next_code, *pbase = two + (at & 1) * next_param;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          s1[tile][i] = 0.f;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) s[tile][nt][i] = 0.f;
        }
        // one step of the contraction: A of 16 keys, for every query row
        auto step = [&](int k, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            mma_16816(NT == 1 && (k & 1) ? s1[tile] : s[tile][nt], a0, a1, a2, a3, qb[nt][k][0], qb[nt][k][1], true);
        };
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          pk[tile][i] = lds32(smem_u32(pbase + par_at[i]));  // (a plain load is made again at every use)
          pv[tile][i] = lds32(smem_u32(pbase + HALF + par_at[i]));
        }
        if constexpr (BITS == 4) {
          uint32_t a[2][D / 32];
#pragma unroll
          for (int i = 0; i < 2; ++i) shared_words<D / 32>(base + k_at[i], a[i]);
          constexpr uint32_t M = 0x000f000fu, N = 0x00f000f0u;
          const __half2 low = __half2half2(__float2half_rn(-1024.f));
#pragma unroll
          for (int w = 0; w < D / 32; ++w) {  // c of even nibbles, 16 (64 + c) of odd ones
            const uint32_t x = a[0][w], y = a[1][w];
            step(2 * w, h2(and_or(x, M, C), low), h2(and_or(y, M, C), low), and_or(x, N, C), and_or(y, N, C));
            step(2 * w + 1, h2(and_or(x >> 8, M, C), low), h2(and_or(y >> 8, M, C), low), and_or(x >> 8, N, C),
                 and_or(y >> 8, N, C));
          }
        } else {
#pragma unroll
          for (int c = 0; c < D / 64; ++c) {
            uint32_t x[4], y[4];
            shared_words<4>(base + k_at[0] + 64 * c, x);
            shared_words<4>(base + k_at[1] + 64 * c, y);
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              const uint32_t H = 0x64646464u;
              step(4 * c + w, __byte_perm(x[w], H, 0x4140), __byte_perm(y[w], H, 0x4140), __byte_perm(x[w], H, 0x4342),
                   __byte_perm(y[w], H, 0x4342));
            }
          }
        }
      }
      // ---- logits (in powers of two), numerators: [0], [1] key_of(g), [2], [3] key_of(g + 8)
      float x[TILES][NT][4], ws[TILES][2];
      bool hidden[TILES][NT][4];
#pragma unroll
      for (int tile = 0; tile < TILES; ++tile)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int key = key0 + (tile0 + tile) * 16 + key_of(g + 8 * i);
          bool gone = false;  // a key of a block that is not there, whose place in the stage holds anything
          if (kTail && pr.any_missing && key < n_max) {
            const int id = p.block_table[int64_t(sg.s) * p.max_blocks_per_seq + key / p.block_size];
            gone = id < 0 || id >= p.num_blocks;
          }
          // a row behind the last, or of no block: whatever it holds
          if (kTail && (key >= n_max || gone)) pk[tile][i] = pv[tile][i] = 0u;
          const float step = param_step(pk[tile][i]), lo = param_lo(pk[tile][i]);
          ws[tile][i] = param_step(pv[tile][i]);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            float2 c = make_float2(s[tile][nt][2 * i], s[tile][nt][2 * i + 1]);
            if (NT == 1) c = fadd2(c, make_float2(s1[tile][2 * i], s1[tile][2 * i + 1]));
            c = mul2(fadd2(c, make_float2(off[nt][0], off[nt][1])), make_float2(fac[nt][0], fac[nt][1]));
            c = ffma2v(c, make_float2(step, step), mul2(make_float2(lo, lo), make_float2(qs[nt][0], qs[nt][1])));
            x[tile][nt][2 * i] = c.x, x[tile][nt][2 * i + 1] = c.y;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int e = 2 * i + h;
              hidden[tile][nt][e] = kTail && (key >= lim[nt][h] || gone);
              if (hidden[tile][nt][e]) x[tile][nt][e] = -INFINITY;
            }
          }
        }
      // The reference maximum (a whole number, so that moves are exact) moves only when a logit passes it by
      // 2^8, a row's wscale when its maximum does or a step comes over 2^7: then the sums so far are scaled.
      float top[NT][2], big = fmaxf(ws[0][0], ws[0][1]);
      bool move = false;
#pragma unroll
      for (int tile = 1; tile < TILES; ++tile) big = fmax3(big, ws[tile][0], ws[tile][1]);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          top[nt][h] = fmaxf(x[0][nt][h], x[0][nt][2 + h]);
#pragma unroll
          for (int tile = 1; tile < TILES; ++tile) top[nt][h] = fmax3(top[nt][h], x[tile][nt][h], x[tile][nt][2 + h]);
          move = move || top[nt][h] - m[nt][h] > 8.f || big * wscale[nt][h] > 128.f;
        }
      if (__any_sync(0xffffffffu, move)) {
        // The power that brings the unit's largest step to [2^6, 2^7): small enough for every product (numerators
        // are at most 2^8). NaN steps (of rows that hold NaN) do not count.
        const uint32_t bits = __float_as_uint(big);
        const uint32_t most = __reduce_max_sync(0xffffffffu, bits <= 0x7f800000u ? bits : 0u);
        const int by_step = 6 - (int(most >> 23) - 126);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float beta[2];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float up = top[nt][h];
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) up = fmaxf(up, __shfl_xor_sync(0xffffffffu, up, d));
            up = up - m[nt][h] > 8.f ? ceilf(up) : m[nt][h];
            // the power that brings the row's largest product of the unit to [2^3, 2^4): the larger of the two,
            // but not so large that the largest product of the units before passes where it was
            float peak = 0.f;
#pragma unroll
            for (int tile = 0; tile < TILES; ++tile)
#pragma unroll
              for (int i = 0; i < 2; ++i) peak = fmaxf(peak, ex2_ftz(x[tile][nt][2 * i + h] - up) * ws[tile][i]);
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) peak = fmaxf(peak, __shfl_xor_sync(0xffffffffu, peak, d));
            const int by_product = 3 - (int(__float_as_uint(peak) >> 23) - 126);
            const int old = int(__float_as_uint(wscale[nt][h]) >> 23) - 127;
            const int want = min(min(126, old + int(fminf(up - m[nt][h], 300.f))), max(by_step, by_product));
            wscale[nt][h] = __uint_as_float(uint32_t(want + 127) << 23);
            beta[h] = exp2f(float(want - old) + (m[nt][h] - up));  // at most 1
            const float alpha = exp2f(m[nt][h] - up);
            m[nt][h] = up;
            l[nt][h] *= alpha;
            mid[nt][h] *= alpha;
          }
#pragma unroll
          for (int i = 0; i < NK; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[nt][i][e] *= beta[e & 1];
        }
      }
      uint32_t pb[TILES][NT][2];
#pragma unroll
      for (int tile = 0; tile < TILES; ++tile)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          asm volatile("" : "+r"(pv[tile][i]));  // unpacked here, not above: fewer registers over the move
          const float step = param_step(pv[tile][i]), middle = fmaf(step, kMid, param_lo(pv[tile][i]));
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            float w[2], e2[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) e2[h] = ex2_ftz(x[tile][nt][2 * i + h] - m[nt][h]);
            // (a step times wscale alone may pass the largest float where the numerator is 0)
            const float2 scaled = mul2(mul2(make_float2(e2[0], e2[1]), make_float2(step, step)),
                                       make_float2(wscale[nt][0], wscale[nt][1]));
            w[0] = scaled.x, w[1] = scaled.y;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const float e = e2[h];
              l[nt][h] += e;
              if (hidden[tile][nt][2 * i + h]) {
                w[h] = 0.f;  // not 0 * NaN
              } else {
                mid[nt][h] = fmaf(e, middle, mid[nt][h]);
              }
            }
            pb[tile][nt][i] = movm(pack_f16(w[0], w[1]));
          }
        }
      // ---- 16 value dimensions x 8 NT query rows a step: rows of the tile of codes - mid, dimensions
      // (D / 8) g + 2 i in rows 0 .. 7 and the next in rows 8 .. 15
#pragma unroll
      for (int tile = 0; tile < TILES; ++tile) {
        const int at = tile0 + tile;
        const unsigned char* base = st + (at >> 1) * (32 * (ROW + 4)) + (at & 1) * next_code;
        auto step = [&](int i, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) mma_16816(o[nt][i], a0, a1, a2, a3, pb[tile][nt][0], pb[tile][nt][1], true);
        };
        if constexpr (BITS == 4) {
          const __half2 low = __half2half2(__float2half_rn(-1032.f)), high = __half2half2(__float2half_rn(-72.f)),
                        six = __half2half2(__float2half_rn(0.0625f));
          uint32_t v[4][D / 64];
#pragma unroll
          for (int i = 0; i < 4; ++i) shared_words<D / 64>(base + v_at[i], v[i]);
          constexpr uint32_t M = 0x000f000fu, N = 0x00f000f0u;
#pragma unroll
          for (int w = 0; w < D / 64; ++w)
#pragma unroll
            for (int half = 0; half < 2; ++half) {  // elements 0 .. 3, 4 .. 7 of the words
              const uint32_t sel = half ? 0x7632 : 0x5410;
              const uint32_t a = __byte_perm(v[0][w], v[1][w], sel), b = __byte_perm(v[2][w], v[3][w], sel);
              step(4 * w + 2 * half, h2(and_or(a, M, C), low), h2(and_or(a, N, C), six, high), h2(and_or(b, M, C), low),
                   h2(and_or(b, N, C), six, high));
              step(4 * w + 2 * half + 1, h2(and_or(a >> 8, M, C), low), h2(and_or(a >> 8, N, C), six, high),
                   h2(and_or(b >> 8, M, C), low), h2(and_or(b >> 8, N, C), six, high));
            }
        } else {
          const __half2 sub = __half2half2(__float2half_rn(-1152.f));
          const uint32_t H = 0x64646464u;
          uint32_t v[4][D / 32];
#pragma unroll
          for (int i = 0; i < 4; ++i) shared_words<D / 32>(base + v_at[i], v[i]);
#pragma unroll
          for (int w = 0; w < D / 32; ++w)
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              const uint32_t sel = half ? 0x7362 : 0x5140;
              const uint32_t a = __byte_perm(v[0][w], v[1][w], sel), b = __byte_perm(v[2][w], v[3][w], sel);
              step(2 * w + half, h2(__byte_perm(a, H, 0x4140), sub), h2(__byte_perm(a, H, 0x4342), sub),
                   h2(__byte_perm(b, H, 0x4140), sub), h2(__byte_perm(b, H, 0x4342), sub));
            }
        }
      }
    };

    for (int x = x0; x < x1; ++x) {
      fill();
      copies_wait<STAGES - 1>();
      __syncwarp();
      const int key0 = x * KU;
      const unsigned char* st = ring + stage * STAGE;
      if (key0 + KU <= n_min && !pr.any_missing) {
#pragma unroll 1
        for (int tile = 0; tile < KU / 16; tile += NT == 1 ? KU / 16 : 2) unit(st, key0, tile, std::false_type{});
      } else {
#pragma unroll 1
        for (int tile = 0; tile < KU / 16 && key0 + tile * 16 < n_max; ++tile) unit(st, key0, tile, std::true_type{});
      }
      __syncwarp();
      if (++stage == STAGES) stage = 0;
    }
    // ---- the segment's end in this run: sums over the lanes that share a query row, then out or a piece
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float sum = l[nt][h], add = mid[nt][h];
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) {
          sum += __shfl_xor_sync(0xffffffffu, sum, d);
          add += __shfl_xor_sync(0xffffffffu, add, d);
        }
        const int row = 8 * nt + 2 * t + h;
        if (row >= rows) continue;
        const float unscale = __uint_as_float((254u << 23) - __float_as_uint(wscale[nt][h]));
        float f[D / 8];
#pragma unroll
        for (int i = 0; i < NK; ++i) {
          f[2 * i] = fmaf(o[nt][i][h], unscale, add);
          f[2 * i + 1] = fmaf(o[nt][i][2 + h], unscale, add);
        }
        if (whole) {
          const float inv = sum > 0.f ? 1.f / sum : (sum == 0.f ? 0.f : sum);
          __nv_bfloat16* dst = out_row(p, where, row, D) + g * (D / 8);
#pragma unroll
          for (int i = 0; i < D / 8; ++i) f[i] *= inv;
#pragma unroll
          for (int i = 0; i < D / 64; ++i) reinterpret_cast<uint4*>(dst)[i] = Elem<__nv_bfloat16>::pack(f + 8 * i);
        } else {
#pragma unroll
          for (int i = 0; i < D / 32; ++i)
            reinterpret_cast<float4*>(piece + row * D + g * (D / 8))[i] =
                make_float4(f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3]);
          if (g == 0) {
            piece[kRows * D + row] = m[nt][h];
            piece[kRows * D + kRows + row] = sum;
          }
        }
      }
  }
  __syncthreads();

  // ---- pieces of segments cut between this CTA's warps, or between CTAs. A leader is a CTA's first
  // piece of a segment; the leaders' rows are dealt to the warps, one by one where there are few leaders.
  const int c0 = first(w0), c1 = first(w0 + kWarps);
  float* cta_pieces = p.pieces + int64_t(num_warps) * piece_floats<D, NT>();
  const int4 mine = lane < kWarps * 2 ? desc[lane] : make_int4(-1, 0, 0, 0);
  if (warp == 0) {
    // slot 0: a segment from before c0, or one from c0 to past c1; slot 1: one that goes on behind c1
    const unsigned tail = __ballot_sync(0xffffffffu, mine.x > c0 && mine.y > c1);
    if (lane == (tail ? __ffs(tail) - 1 : 1)) p.descs[blockIdx.x * 2 + 1] = tail ? mine : make_int4(-1, 0, 0, 0);
    if (lane == 0) p.descs[blockIdx.x * 2] = mine.x >= 0 && (mine.x < c0 || mine.y > c1) ? mine : make_int4(-1, 0, 0, 0);
  }
  const unsigned leaders =
      __ballot_sync(0xffffffffu, mine.x >= 0 && ((lane & 1) || lane == 0 || mine.x == first(w0 + (lane >> 1))));
  const int num = __popc(leaders);
  const int at_once = num * kRows <= kWarps ? 1 : 4;
  for (int task = warp; task < num * (kRows / at_once); task += kWarps) {
    const int at = __fns(leaders, 0, task / (kRows / at_once) + 1), row0 = task % (kRows / at_once) * at_once, w = at >> 1;
    const int4 d = desc[at];
    int count = 1;
    while (w + count < kWarps && first(w0 + w + count) < d.y) ++count;
    float* whole = d.x >= c0 && d.y <= c1 ? nullptr
                                          : cta_pieces + int64_t(blockIdx.x * 2 + (d.x <= c0 ? 0 : 1)) * piece_floats<D, NT>();
    // the last one may be the first piece of a run that goes on
    const bool goes_on = first(w0 + w + count) > d.y;
    auto piece = [&](int k) -> const float* {
      return goes_on && k == count - 1 ? p.pieces + int64_t(w0 + w + k) * piece_floats<D, NT>()
                                       : reinterpret_cast<const float*>(smem + (w + k) * STAGES * STAGE);
    };
    const int2 where = make_int2(d.z, d.w);
    if (at_once == 1)
      join_rows<D, 32, NT>(p, where, row0, lane, count, piece, whole);
    else
      join_rows<D, 8, NT>(p, where, row0 + lane / 8, lane, count, piece, whole);
  }
}

// Segments cut between CTAs: CTA c joins those whose first piece is c's, several warps a row: 4 elements a
// lane of several pieces at once, so that up to 16 (8) pieces are on their way together (one request of 32000
// keys, 4 bits, 8 heads of 19 pieces: with a warp a row and 4 pieces the call takes 26.0 us, so 22.7; with
// 1024 threads 23.1, and every other call 0.5 us more).
constexpr int kJoinThreads = 512;
template <int D, int NT>
__global__ void __launch_bounds__(kJoinThreads, 1) attention_int_join_kernel(const IntParams p, int num_ctas) {
  constexpr int kWarps = num_warps<NT>(), kRows = num_rows<NT>();
  constexpr int PARTS = kJoinThreads / 32 / kRows, LANES = D / PARTS / 4, GROUPS = 32 / LANES;  // warps a row, lanes a piece, pieces a load
  griddep_wait();
  const int c = blockIdx.x, row = int(threadIdx.x >> 5) / PARTS, part = int(threadIdx.x >> 5) % PARTS, lane = threadIdx.x & 31;
  const int d0 = part * (D / PARTS) + lane % LANES * 4, group = lane / LANES;
  const Deal first(*p.total, num_ctas * kWarps);
  const float* pieces = p.pieces + int64_t(num_ctas) * kWarps * piece_floats<D, NT>() + row * D + d0;
#pragma unroll 1
  for (int slot = 0; slot < 2; ++slot) {
    const int4 d = p.descs[c * 2 + slot];
    if (d.x < 0 || (slot == 0 && d.x != first(c * kWarps)) || row >= (d.w & 31)) continue;
    int count = 1;
    while (c + count < num_ctas && first((c + count) * kWarps) < d.y) ++count;
    auto piece = [&](int k) { return pieces + int64_t(k == 0 ? c * 2 + slot : (c + k) * 2) * piece_floats<D, NT>(); };
    float m = kNoMax, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
    for (int k0 = 0; k0 < count; k0 += 32) {
      const bool live = k0 + lane < count;
      const float* ml = piece(live ? k0 + lane : 0) + (kRows - row) * D - d0 + row;
      const float mk = ml[0], lk = live ? ml[kRows] : 0.f;
      float top = lk == 0.f ? kNoMax : mk;  // an empty piece: its other sums were never written
#pragma unroll
      for (int x = 1; x < 32; x <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
      top = fmaxf(top, m);
      const float w = lk == 0.f ? 0.f : exp2f(mk - top), before = exp2f(m - top);
      float sum = lk * w;
#pragma unroll
      for (int x = 1; x < 32; x <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
      l = l * before + sum;
      m = top;
      o.x *= before, o.y *= before, o.z *= before, o.w *= before;
#pragma unroll 8
      for (int j = group; j < 32; j += GROUPS) {
        if (k0 + j - group >= count) break;
        const float e = __shfl_sync(0xffffffffu, w, j);
        const float4 y = *reinterpret_cast<const float4*>(piece(k0 + j < count ? k0 + j : 0));
        if (e != 0.f) o = make_float4(fmaf(e, y.x, o.x), fmaf(e, y.y, o.y), fmaf(e, y.z, o.z), fmaf(e, y.w, o.w));
      }
    }
#pragma unroll
    for (int x = LANES; x < 32; x <<= 1) {
      o.x += __shfl_xor_sync(0xffffffffu, o.x, x);
      o.y += __shfl_xor_sync(0xffffffffu, o.y, x);
      o.z += __shfl_xor_sync(0xffffffffu, o.z, x);
      o.w += __shfl_xor_sync(0xffffffffu, o.w, x);
    }
    const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
    if (group == 0)
      *reinterpret_cast<uint2*>(out_row(p, make_int2(d.z, d.w), row, D) + d0) =
          make_uint2(pack_bf16(o.x * inv, o.y * inv), pack_bf16(o.z * inv, o.w * inv));
  }
}

constexpr size_t align_up(size_t x) { return (x + 255) & ~size_t(255); }

template <int D, int BITS, int NT>
cudaError_t run_int(IntParams p, const AttnIntArgs& a, cudaStream_t stream) {
  constexpr size_t rings = size_t(num_warps<NT>()) * num_stages<D, NT>() * stage_bytes<D, BITS>(),
                   most = rings + kIntMaxSeqs * 4;
  static_assert(most + 1024 <= 232448, "shared memory of a CTA");
  const bool b16 = a.block_size == 16;
  const cudaError_t e = b16 ? ensure_smem<attention_int_kernel<D, BITS, true, NT>>(most)
                            : ensure_smem<attention_int_kernel<D, BITS, false, NT>>(most);
  if (e != cudaSuccess) return e;
  const cudaError_t l = launch_pdl(b16 ? attention_int_kernel<D, BITS, true, NT> : attention_int_kernel<D, BITS, false, NT>,
                                   dim3(a.num_ctas), dim3(num_warps<NT>() * 32), rings + size_t(a.num_seqs) * 4, stream, p);
  if (l != cudaSuccess) return l;
  return launch_pdl(attention_int_join_kernel<D, NT>, dim3(a.num_ctas), dim3(kJoinThreads), 0, stream, p,
                    a.num_ctas);
}
template <int D, int BITS>
cudaError_t run_rows(const IntParams& p, const AttnIntArgs& a, cudaStream_t stream) {
  return int64_t(a.max_query_len) * p.group > num_rows<1>() ? run_int<D, BITS, 2>(p, a, stream)
                                                            : run_int<D, BITS, 1>(p, a, stream);
}

}  // namespace

// descs, total, pieces of the CTAs' warps and of the CTAs
size_t attention_int_workspace_bytes(int head_dim, int num_ctas) {
  const size_t row = (size_t(head_dim) + 2) * 4;
  const size_t one = num_rows<1>() * (num_warps<1>() + 2), two = num_rows<2>() * (num_warps<2>() + 2);
  return align_up(size_t(num_ctas) * 2 * sizeof(int4)) + 256 + size_t(num_ctas) * (one > two ? one : two) * row;
}

bool attention_int_fits(const AttnIntArgs& a) {
  const int group = a.num_heads / a.num_kv_heads;
  const bool two = int64_t(a.max_query_len) * group > num_rows<1>();
  const int ku = a.bits == 4 ? unit_keys<4>() : unit_keys<8>();
  const int64_t tiles = int64_t(a.num_tokens) * group / (two ? num_rows<2>() : num_rows<1>()) + 1 + a.num_seqs;
  const int64_t units = (int64_t(a.max_seq_len) + ku - 1) / ku + 2;
  // units are counted in 32 bits (a step of all warps past the end, too)
  return a.num_seqs <= kIntMaxSeqs && a.num_heads < (1 << 27) && a.max_seq_len <= 0x7fffffff - 128 && tiles <= 0x7fffffff / a.num_kv_heads &&
         tiles * a.num_kv_heads <= (0x7fffffff - (1 << 20)) / units;
}

cudaError_t launch_attention_int(const AttnIntArgs& a, cudaStream_t stream) {
  IntParams p = {};
  p.out = static_cast<__nv_bfloat16*>(a.out);
  p.q = static_cast<const __nv_bfloat16*>(a.q);
  p.k_cache = static_cast<const unsigned char*>(a.k_cache);
  p.v_cache = static_cast<const unsigned char*>(a.v_cache);
  p.block_table = a.block_table;
  p.seq_lens = a.seq_lens;
  p.qsl = a.query_start_loc;
  p.err = a.err;
  unsigned char* ws = static_cast<unsigned char*>(a.workspace);
  p.descs = reinterpret_cast<int4*>(ws);
  ws += align_up(size_t(a.num_ctas) * 2 * sizeof(int4));
  p.total = reinterpret_cast<int*>(ws);
  p.pieces = reinterpret_cast<float*>(ws + 256);
  p.num_blocks = a.num_blocks;
  p.max_blocks_per_seq = a.max_blocks_per_seq;
  p.num_seqs = a.num_seqs;
  p.num_tokens = a.num_tokens;
  p.max_query_len = a.max_query_len;
  p.max_seq_len = a.max_seq_len;
  p.num_heads = a.num_heads;
  p.num_kv_heads = a.num_kv_heads;
  p.group = a.num_heads / a.num_kv_heads;
  p.block_size = a.block_size;
  p.scale_log2 = a.scale * 1.4426950408889634f;
  p.part = a.block_size & -a.block_size;
  if (p.part > kPart) p.part = kPart;
  if (a.bits == 4) return a.head_dim == 64 ? run_rows<64, 4>(p, a, stream) : run_rows<128, 4>(p, a, stream);
  return a.head_dim == 64 ? run_rows<64, 8>(p, a, stream) : run_rows<128, 8>(p, a, stream);
}

}  // namespace pa
