// pa_int4.cuh -- the 4-bit cache format (PA_INT4) shared by the kernels that
// write, read back and attend over it.
//
// A (block, KV head) chunk of a pool holds 16 token rows of D / 2 code bytes
// (element 2i in the low nibble of byte i) and then, for each row, two bf16
// numbers (scale, low): element = code * scale + low.  The chunk is
// 8 D + 64 bytes, a multiple of the 64 bytes that DRAM delivers at once for
// D = 64 and 128, so no chunk shares such a piece with its neighbour and
// every chunk starts where a bulk copy may start.  An offset beside the
// scale (instead of a symmetric code) costs 2 bytes per row of 64 and takes
// the step from 2 max|x| / 15 to (max - min) / 15.
#pragma once

#include "pa_common.cuh"

namespace pa {

__host__ __device__ constexpr int int4_chunk_bytes(int D) { return 8 * D + 64; }
__host__ __device__ constexpr int int4_ends_offset(int D) { return 8 * D; }

// The (scale, low) pair of a row, widened (scale in the low half).
__device__ __forceinline__ float2 int4_ends(uint32_t bits) {
    return make_float2(__uint_as_float(bits << 16), __uint_as_float(bits & 0xffff0000u));
}

}  // namespace pa
