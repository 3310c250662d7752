// Launchers behind the 8-bit floating-point format with a scale for each block
// of 128 and the grouped product over it.
#pragma once

#include "grouped.h"

namespace moeq {

constexpr int kFp8Block = MOEQ_FP8_BLOCKSIZE;
__host__ __device__ constexpr int32_t fp8_blocks(int32_t n) { return (int32_t)(((int64_t)n + kFp8Block - 1) / kFp8Block); }

// tile: one scale for 128 rows by 128 columns of an expert, otherwise for 128
// columns of a row.
hipError_t launch_quantize_fp8(const uint16_t* w, uint8_t* q, float* scales, int32_t E, int32_t rows, int32_t cols, bool tile,
                               hipStream_t s);
hipError_t launch_dequantize_fp8(const uint8_t* q, const float* scales, uint16_t* out, int32_t E, int32_t rows, int32_t cols,
                                 bool tile, hipStream_t s);

// g: x [M][kc] and w [E][nout][kc] codes, out bf16 [M][nout]; x_scales
// [M][ceil(kc / 128)], w_scales [E][ceil(nout / 128)][ceil(kc / 128)].
hipError_t launch_grouped_mm_fp8(const GroupedArgs& g, const float* x_scales, const float* w_scales, hipStream_t s);

}  // namespace moeq
