// dpg_fp4.h -- 4-bit quantised matrices: layout and checks shared by the
// quantisation (dpg_fp4.cu) and the products (dpg_fp4_product.cu).
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "dpg_internal.h"

namespace dpg {

constexpr int64_t kFp4MaxSide = int64_t(1) << 30;
constexpr int kFp4TileRows = 128;       // of a scale tile
constexpr int kFp4TileBytes = 512;      // 128 rows x 4 scales

__host__ __device__ constexpr int fp4_block(int format) { return format == DPG_MXFP4 ? 32 : 16; }
// bytes from a row of codes to the next: whole 16-byte pieces
__host__ __device__ constexpr int64_t fp4_pitch(int64_t cols) { return (cols + 31) / 32 * 16; }
// scale tiles in a row of tiles: 4 blocks each
__host__ __device__ constexpr int64_t fp4_tiles(int64_t cols, int format) {
    return (cols + 4 * fp4_block(format) - 1) / (4 * fp4_block(format));
}

// The exponent e of the matrix's power of two: the least with amax <= 6 * 448 *
// 2^e = 1.3125 * 2^(e + 11), from -126 on.
__host__ __device__ __forceinline__ int fp4_exponent(uint32_t amax_bits) {
    const int e = int(amax_bits >> 23) - 127 - 11 + ((amax_bits & 0x7FFFFFu) > 0x280000u ? 1 : 0);
    return e < -126 ? -126 : e;
}

// null, alignment and range checks of one quantised matrix; `name` is "by_row", ...
int fp4_check(const dpg_fp4* q, const char* name, const char* who);

}  // namespace dpg
