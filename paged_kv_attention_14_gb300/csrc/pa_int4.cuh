// pa_int4.cuh -- layout and arithmetic of the 4-bit cache.
//
// A page of one kv head is 9 head_dim bytes: the codes of its 16 rows
// (head_dim / 2 bytes a row, the even dim in the low half of a byte), then
// the rows' (scale, minimum) pairs in fp16, one pair per 64 dims.  A dim reads
// as scale * code + minimum.
#pragma once

#include "pa_device.cuh"

namespace pa {
namespace i4 {

constexpr int kGroup = 64;  // dims that share a scale and a minimum

__host__ __device__ constexpr int tile_bytes(int d) { return 9 * d; }
__host__ __device__ constexpr int code_bytes(int d) { return 8 * d; }  // the codes of a tile, before its pairs
__host__ __device__ constexpr int groups(int d) { return d / kGroup; }

}  // namespace i4
}  // namespace pa
