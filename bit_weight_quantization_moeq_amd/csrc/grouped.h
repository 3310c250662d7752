// Launchers behind the grouped products, the MXFP4 format and the gradient
// clipping (their C entry points are in api_grouped.hip).
#pragma once

#include "moeq_internal.h"

namespace moeq {

hipError_t launch_quantize_mxfp4(const uint16_t* w, uint8_t* q, uint8_t* scales, int64_t nblocks, hipStream_t s);
hipError_t launch_dequantize_mxfp4(const uint8_t* q, const uint8_t* scales, uint16_t* out, int64_t nblocks,
                                   hipStream_t s);

// One grouped product over rows sorted by expert.
//   forward:      x [M][kc], w [E][nout][kc], out [M][nout]
//   grad_input:   x = dy [M][kc], w [E][kc][nout], out = dx [M][nout]
//   grad_weight:  x [M][kc], w = dy [M][nout], out = dw [E][nout][kc]
// MXFP4 operands: codes in x / w and one scale byte per 32 values.
struct GroupedArgs {
  const void* x;
  const void* w;
  const uint8_t* x_scales;
  const uint8_t* w_scales;
  const int32_t* offsets;  // [E + 1], on the device
  void* out;
  int32_t M, E, nout, kc;
  // grad_weight: rows per segment, and room for the fp32 sums of the segments
  // of experts that have several
  int32_t segment = 0, slots = 0;
  float* partial = nullptr;
};

// The rows of an expert between two offsets, which can hold anything: both are
// clamped to [0, M], and the expert has no rows where they do not ascend.
struct RowRange {
  int32_t lo, n;
};
__host__ __device__ inline RowRange row_range(int32_t from, int32_t to, int32_t M) {
  const int32_t lo = from < 0 ? 0 : from < M ? from : M, hi = to < 0 ? 0 : to < M ? to : M;
  return {lo, hi > lo ? hi - lo : 0};
}

int32_t grad_weight_segment(int32_t M, int32_t N, int32_t K);
int64_t grad_weight_slots(int32_t M, int32_t segment);   // [N][K] slots of the workspace
hipError_t launch_grouped_mm(const GroupedArgs& g, hipStream_t s);
hipError_t launch_grouped_mm_mxfp4(const GroupedArgs& g, hipStream_t s);
hipError_t launch_grouped_mm_grad_input(const GroupedArgs& g, hipStream_t s);
hipError_t launch_grouped_mm_grad_weight(const GroupedArgs& g, bool fp32, hipStream_t s);

// Gradient clipping.  partial: kClipHead + clip_partials(count) fp64.
constexpr int kClipPartials = 768;  // partial sums per launch, at most
constexpr int kClipHead = 2;        // room for the factor, in front of the partial sums
int64_t clip_partials(int32_t count);
hipError_t launch_clip(const moeq_grad* g, int32_t count, double max_norm, float* norm, double* partial, hipStream_t s);

}  // namespace moeq
