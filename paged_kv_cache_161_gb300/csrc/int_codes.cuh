// The integer-coded cache: what a block holds, shared by the kernels that write, read and attend
// to it (kv_int.cu, attention_int.cu).
//
// A row x of head_dim elements (one token, one KV head) is held as `bits`-bit codes c with
// x ~ lo + step c. Per block and KV head one record: the block's rows of codes, row after row
// (element 2 i in the low half of byte i when bits = 4), then a 32-bit word a row, the
// bfloat16 lo in its low half and the bfloat16 step in its high half.
//   - One record is what a decode warp streams: at 16 tokens x 128 elements x 4 bits it is 1088
//     contiguous bytes, one bulk copy, where [block_size, heads, head_dim] order would scatter it
//     over pieces of 64 bytes.
//   - One scale for a row and not for parts of it: it then leaves the inner products (q.x = step
//     q.c + lo sum q), so that attention multiplies whole codes.
//   - lo and step in 16 bits (4 bytes a row: 6 % of a 4-bit row; 8 bytes would be 12 %): lo is
//     rounded down and step up, so every element stays within the codes' range and only the resolution
//     suffers: the step by 2^-7, the spread by 2^-7 of lo where a float32 row's smallest element is no
//     bfloat16 (a bfloat16 row's is its lo exactly).
#pragma once

#include "common.cuh"

namespace pa {
namespace {

template <int D, int BITS>
__host__ __device__ constexpr int code_row_bytes() { return D * BITS / 8; }

__device__ __forceinline__ float param_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float param_step(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

}  // namespace
}  // namespace pa
