// FP8 in and out of bf16 (gfx950): E4M3 codes (OCP, 448 the largest) with one
// fp32 scale for each 128 columns of a row, or for each 128 x 128 tile.
//
//   amax = the block's largest magnitude     scale = fp32(amax / 448)
//   code = E4M3 nearest to 448 w / amax, ties to even;  w' = bf16(fp32(code scale))
//
// The quotient is taken of w itself rather than by the rounded scale, so that
// a tie is a tie: 448 w (11 bits) is exact in fp32, and a quotient of 11 by 8
// bits is either halfway between two codes exactly or off by more than 2^-17
// relative, so that rounding it to fp32 first decides nothing.  It is formed as
// q = 448 w r, r = 1 / amax, with one correction q + r fma(-q, amax, 448 w) (a
// Newton step), which is exact where the quotient fits fp32, and within two
// units elsewhere.  Blocks whose amax lies far from 1 are taken times 2^64 or
// 2^-64 first, so that none of this leaves fp32's normal range.
//
// Bound by memory: bf16 in (or out) 2 bytes and codes 1 byte a value.  Measured,
// [32, 5760, 2880] in tiles: 287 us there (5.6 TB/s, part of the input from the
// memory-side cache) and 356 back (4.5 TB/s); a copy reaches 4.7 to 4.9.  64 rows
// of 2880: 3 us each, a launch's latency.
#include "fp8.h"

namespace moeq {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));

constexpr uint32_t kInf = 0x7f80;   // bf16 magnitudes from here on are infinities and NaNs

__device__ __forceinline__ uint32_t max16x2(uint32_t a, uint32_t b) {
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, a), __builtin_bit_cast(u16x2, b)));
}
template <int CTRL>
__device__ __forceinline__ uint32_t max_dpp(uint32_t v) {
  return max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, false));
}

// The largest magnitude (bf16 bits) of 16 values.
__device__ __forceinline__ uint32_t magnitude(const u32x4 (&v)[2]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) m = max16x2(m, v[i][j] & 0x7fff7fffu);
  return max(m & 0xffffu, m >> 16);
}
// Of 8 lanes, in all of them: neighbours, pairs, halves.
__device__ __forceinline__ uint32_t max8(uint32_t m) {
  return max_dpp<0x141>(max_dpp<0x4E>(max_dpp<0xB1>(m)));
}

// What a block's codes are made with; a block with an infinity or a NaN has
// the scale NaN and zero codes, one of zeros the scale 0.
struct Quantizer {
  float amax, inv, times, scale;
  bool finite;
  __device__ __forceinline__ explicit Quantizer(uint32_t bits) {
    const float a = __builtin_bit_cast(float, bits << 16);
    const float by = a < 0x1p-60f ? 0x1p64f : a > 0x1p60f ? 0x1p-64f : 1.0f;
    finite = bits < kInf;
    scale = finite ? a / 448.0f : __builtin_nanf("");
    amax = bits ? a * by : 1.0f;
    inv = 1.0f / amax;
    times = 448.0f * by;
  }
  __device__ __forceinline__ float quotient(uint32_t bits) const {
    const float w = times * __builtin_bit_cast(float, bits);
    const float q = w * inv;
    return __builtin_copysignf(__builtin_fmaf(__builtin_fmaf(-q, amax, w), inv, q), w);
  }
  // the codes of four values (two dwords of bf16 pairs)
  __device__ __forceinline__ uint32_t four(uint32_t lo, uint32_t hi) const {
    int c = __builtin_amdgcn_cvt_pk_fp8_f32(quotient(lo << 16), quotient(lo & 0xffff0000u), 0, false);
    c = __builtin_amdgcn_cvt_pk_fp8_f32(quotient(hi << 16), quotient(hi & 0xffff0000u), c, true);
    return finite ? (uint32_t)c : 0u;
  }
  __device__ __forceinline__ u32x4 sixteen(const u32x4 (&v)[2]) const {
    return u32x4{four(v[0].x, v[0].y), four(v[0].z, v[0].w), four(v[1].x, v[1].y), four(v[1].z, v[1].w)};
  }
};

// 16 values a lane, 8 lanes a block.  Index: 32 bits where everything fits.
template <typename Index>
__global__ __launch_bounds__(256) void quantize_rows_kernel(const uint16_t* __restrict__ w, uint8_t* __restrict__ q,
                                                            float* __restrict__ scales, Index blocks, int32_t cols,
                                                            uint32_t row_blocks) {
  const int lane = threadIdx.x & 7;
  for (Index b = (Index)blockIdx.x * 32 + (threadIdx.x >> 3); b < blocks; b += (Index)gridDim.x * 32) {
    const Index row = b / row_blocks;
    const int c = (int)(b - row * row_blocks) * kFp8Block + 16 * lane;
    const int64_t at = (int64_t)row * cols + c;
    u32x4 v[2] = {};
    if (c < cols) {
      v[0] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(w + at));
      v[1] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(w + at) + 1);
    }
    const Quantizer z(max8(magnitude(v)));
    if (c < cols) *reinterpret_cast<u32x4*>(q + at) = z.sixteen(v);
    if (lane == 0) scales[b] = z.scale;
  }
}

// A workgroup a tile: 64 values a lane, in registers from the one read to the
// codes.
__global__ __launch_bounds__(256) void quantize_tiles_kernel(const uint16_t* __restrict__ w, uint8_t* __restrict__ q,
                                                             float* __restrict__ scales, int64_t tiles, int32_t rows,
                                                             int32_t cols, int32_t row_tiles, int32_t col_tiles) {
  __shared__ uint32_t part[2][4];
  const int t = threadIdx.x, r0 = t >> 3, c0 = 16 * (t & 7);
  int turn = 0;
  for (int64_t i = blockIdx.x; i < tiles; i += gridDim.x, turn ^= 1) {
    const int64_t strip = i / col_tiles, e = strip / row_tiles;
    const int c = (int)(i - strip * col_tiles) * kFp8Block + c0, r = (int)(strip - e * row_tiles) * kFp8Block + r0;
    const int64_t at = (e * rows + r) * cols + c;
    u32x4 v[4][2] = {};
    uint32_t m = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (c < cols && r + 32 * k < rows) {
        const u32x4* p = reinterpret_cast<const u32x4*>(w + at + (int64_t)(32 * k) * cols);
        v[k][0] = __builtin_nontemporal_load(p);
        v[k][1] = __builtin_nontemporal_load(p + 1);
      }
#pragma unroll
    for (int k = 0; k < 4; ++k) m = max(m, magnitude(v[k]));
    m = max8(m);
    m = max(m, (uint32_t)__shfl_xor((int)m, 8));
    m = max(m, (uint32_t)__shfl_xor((int)m, 16));
    m = max(m, (uint32_t)__shfl_xor((int)m, 32));
    if ((t & 63) == 0) part[turn][t >> 6] = m;
    __syncthreads();   // (the other turn's values were read before this one's barrier)
    const Quantizer z(max(max(part[turn][0], part[turn][1]), max(part[turn][2], part[turn][3])));
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (c < cols && r + 32 * k < rows) *reinterpret_cast<u32x4*>(q + at + (int64_t)(32 * k) * cols) = z.sixteen(v[k]);
    if (t == 0) scales[i] = z.scale;
  }
}

__device__ __forceinline__ uint32_t pack(f32x2 v) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));
}

// 16 values a lane.
template <typename Index, bool kTile>
__global__ __launch_bounds__(256) void dequantize_kernel(const uint8_t* __restrict__ q, const float* __restrict__ scales,
                                                         uint16_t* __restrict__ out, Index groups, uint32_t row_groups,
                                                         uint32_t rows, uint32_t row_tiles) {
  const uint32_t row_blocks = (row_groups + 7) / 8;
  for (Index i = (Index)blockIdx.x * 256 + threadIdx.x; i < groups; i += (Index)gridDim.x * 256) {
    const Index row = i / row_groups;
    const uint32_t block = (uint32_t)(i - row * row_groups) / 8;
    Index strip = row;
    if constexpr (kTile) {
      const Index e = row / rows;
      strip = e * row_tiles + (row - e * rows) / kFp8Block;
    }
    const float s = scales[(int64_t)strip * row_blocks + block];
    const u32x4 c = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(q) + i);
    u32x4 o[2];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const f32x2 lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)c[k], false), hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)c[k], true);
      o[k / 2][2 * (k & 1)] = pack(f32x2{lo.x * s, lo.y * s});
      o[k / 2][2 * (k & 1) + 1] = pack(f32x2{hi.x * s, hi.y * s});
    }
    u32x4* p = reinterpret_cast<u32x4*>(out) + 2 * (int64_t)i;
    __builtin_nontemporal_store(o[0], p);
    __builtin_nontemporal_store(o[1], p + 1);
  }
}

constexpr int64_t kMaxGrid = 1 << 20;   // workgroups; larger tensors take several turns
unsigned grid_of(int64_t n) { return (unsigned)(n < kMaxGrid ? n : kMaxGrid); }

}  // namespace

hipError_t launch_quantize_fp8(const uint16_t* w, uint8_t* q, float* scales, int32_t E, int32_t rows, int32_t cols, bool tile,
                               hipStream_t s) {
  const int32_t cb = fp8_blocks(cols), rb = fp8_blocks(rows);
  if (tile) {
    const int64_t tiles = (int64_t)E * rb * cb;
    quantize_tiles_kernel<<<grid_of(tiles), 256, 0, s>>>(w, q, scales, tiles, rows, cols, rb, cb);
  } else {
    const int64_t blocks = (int64_t)E * rows * cb;
    // (an index of the last turn stays below 2^32: blocks + a grid's 2^25)
    if (blocks < int64_t(1) << 31)
      quantize_rows_kernel<uint32_t><<<grid_of((blocks + 31) / 32), 256, 0, s>>>(w, q, scales, (uint32_t)blocks, cols, cb);
    else
      quantize_rows_kernel<uint64_t><<<grid_of((blocks + 31) / 32), 256, 0, s>>>(w, q, scales, blocks, cols, cb);
  }
  return hipGetLastError();
}

hipError_t launch_dequantize_fp8(const uint8_t* q, const float* scales, uint16_t* out, int32_t E, int32_t rows, int32_t cols,
                                 bool tile, hipStream_t s) {
  const uint32_t row_groups = cols / 16, rb = fp8_blocks(rows);
  const int64_t groups = (int64_t)E * rows * row_groups;
  const unsigned grid = grid_of((groups + 255) / 256);
  const bool narrow = groups < int64_t(1) << 31;
  if (tile && narrow)
    dequantize_kernel<uint32_t, true><<<grid, 256, 0, s>>>(q, scales, out, (uint32_t)groups, row_groups, rows, rb);
  else if (tile)
    dequantize_kernel<uint64_t, true><<<grid, 256, 0, s>>>(q, scales, out, groups, row_groups, rows, rb);
  else if (narrow)
    dequantize_kernel<uint32_t, false><<<grid, 256, 0, s>>>(q, scales, out, (uint32_t)groups, row_groups, rows, rb);
  else
    dequantize_kernel<uint64_t, false><<<grid, 256, 0, s>>>(q, scales, out, groups, row_groups, rows, rb);
  return hipGetLastError();
}

}  // namespace moeq
