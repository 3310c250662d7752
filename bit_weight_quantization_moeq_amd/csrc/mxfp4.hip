// MXFP4 quantize and dequantize kernels for expert tensors and activations
// (gfx950).
//
// The format is the microscaled 4-bit floating point of the OCP
// Microscaling specification: 32 consecutive columns of a row share one
// power-of-two scale 2^(s - 127) (one byte s, E8M0), each value is E2M1: a
// sign, and one of the magnitudes 0, 1/2, 1, 3/2, 2, 3, 4, 6.
//
//   s    = max(floor(log2(largest |w| of the block)) - 2, -127) + 127
//   code = the E2M1 value nearest to w * 2^(127 - s), ties to the even code,
//          at most 6 in magnitude
//
// so the largest |w| of a block lands in [4, 8).  bf16 has an 8-bit exponent
// biased by 127: with E the exponent field of the largest magnitude,
// s = max(E - 2, 0).  E = 255 (an infinity or a NaN in the block) gives
// s = 255, which stands for NaN, and codes 0.  w * 2^(127 - s) is exact in
// fp32 wherever it can round to a non-zero code, and so is the way back.
//
// Both kernels stream HBM: a block is read by four lanes (8 bf16, 16 B each),
// its largest magnitude comes from integer maxima (the order of magnitudes is
// that of their bit patterns) and two DPP steps, and v_cvt_scalef32_pk_*
// round two values an instruction.  Since a block never straddles a row, a
// tensor is a flat array of blocks.  [32, 5760, 2880]: quantize 229 us (5.9
// TB/s of 2.53 B a value), dequantize 268 us (5.0 TB/s).
#include "moeq_internal.h"

namespace moeq {
namespace {

constexpr int kThreads = 256;

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));

template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t x) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, CTRL, 0xF, 0xF, false);
}

// maxima of the low and of the high halves
__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, a), __builtin_bit_cast(u16x2, b)));
}

// Codes of two bf16 (the low half in the low nibble) into byte B of `old`.
template <int B>
__device__ __forceinline__ uint32_t codes2(uint32_t old, uint32_t w, float scale) {
  return __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(old, __builtin_bit_cast(bf16x2, w), scale, B);
}

constexpr int kUnroll = 4;

__global__ __launch_bounds__(kThreads) void mxfp4_quantize_kernel(const u32x4* __restrict__ w, uint32_t* __restrict__ q,
                                                                 uint8_t* __restrict__ scales, int64_t nchunks) {
  // chunk: 8 values, a quarter of a block.  A wave takes kUnroll groups of 64
  // consecutive chunks a trip, the loads of all of them first.
  const int lane = threadIdx.x & 63;
  const int64_t wave = ((int64_t)blockIdx.x * kThreads + threadIdx.x) >> 6;
  const int64_t nwaves = ((int64_t)gridDim.x * kThreads) >> 6;
  for (int64_t base = wave * (64 * kUnroll); base < nchunks; base += nwaves * (64 * kUnroll)) {
    u32x4 v[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      int64_t c = base + 64 * u + lane;
      c = c < nchunks ? c : nchunks - 1;  // every lane loads, only valid ones store
      v[u] = __builtin_nontemporal_load(&w[c]);
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int64_t c = base + 64 * u + lane;
      uint32_t m = max_u16x2(max_u16x2(v[u].x & 0x7fff7fffu, v[u].y & 0x7fff7fffu),
                             max_u16x2(v[u].z & 0x7fff7fffu, v[u].w & 0x7fff7fffu));
      m = max_u16x2(m, dpp<0xB1>(m));  // quad_perm [1,0,3,2]
      m = max_u16x2(m, dpp<0x4E>(m));  // quad_perm [2,3,0,1]
      m = max(m & 0xffffu, m >> 16);   // magnitude bits of the block's largest value
      const uint32_t e = m >> 7;
      const bool finite = e < 255u;
      const uint32_t s = finite ? (e > 2u ? e - 2u : 0u) : 255u;
      uint32_t word = 0;
      if (__all(s >= 8u)) {
        const float scale = __uint_as_float(s << 23);  // 2^(s - 127)
        word = codes2<0>(word, v[u].x, scale);
        word = codes2<1>(word, v[u].y, scale);
        word = codes2<2>(word, v[u].z, scale);
        word = codes2<3>(word, v[u].w, scale);
      } else {
        // Some block's scale is (nearly) no normal fp32, so that subnormal
        // values can round to a non-zero code: its values, all below
        // 2^-116, go up by 2^100 first, which is exact.
        const float up = s < 8u ? 0x1p100f : 1.0f;
        const float scale = __uint_as_float((s < 8u ? s + 100u : s) << 23);
        const uint32_t in[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const f32x2 f = {__uint_as_float(in[k] << 16) * up, __uint_as_float(in[k] & 0xffff0000u) * up};
          const uint32_t b = codes2<0>(0u, __builtin_bit_cast(uint32_t, __builtin_convertvector(f, bf16x2)), scale);
          word |= (b & 0xffu) << (8 * k);
        }
      }
      if (c < nchunks) {
        __builtin_nontemporal_store(finite ? word : 0u, &q[c]);
        if ((lane & 3) == 0) scales[c >> 2] = (uint8_t)s;
      }
    }
  }
}

// out = E2M1 value * 2^(s - 127), exact in fp32; the rounding to bf16 only
// acts where that leaves bf16's range (s >= 253, which the quantizer never
// writes, gives infinities for the magnitudes that overflow).
__global__ __launch_bounds__(kThreads) void mxfp4_dequantize_kernel(const uint32_t* __restrict__ q,
                                                                   const uint8_t* __restrict__ scales,
                                                                   u32x4* __restrict__ out, int64_t nchunks) {
  const int64_t stride = (int64_t)gridDim.x * kThreads;
  for (int64_t c = (int64_t)blockIdx.x * kThreads + threadIdx.x; c < nchunks; c += stride) {
    const uint32_t word = __builtin_nontemporal_load(&q[c]);
    const uint32_t s = scales[c >> 2];
    const float scale = s == 255u ? __uint_as_float(0x7fc00000u) : __uint_as_float(s ? s << 23 : 0x00400000u);
    u32x4 r;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(word >> (8 * k), 1.0f, 0);
      const uint32_t u = __builtin_bit_cast(uint32_t, b);
      const f32x2 f = {__uint_as_float(u << 16) * scale, __uint_as_float(u & 0xffff0000u) * scale};
      r[k] = __builtin_bit_cast(uint32_t, __builtin_convertvector(f, bf16x2));
    }
    __builtin_nontemporal_store(r, &out[c]);
  }
}

int grid_for(int64_t items, int64_t per_block, int64_t cap) {
  const int64_t g = (items + per_block - 1) / per_block;
  return (int)(g < cap ? g : cap);
}

}  // namespace

hipError_t launch_quantize_mxfp4(const uint16_t* w, uint8_t* q, uint8_t* scales, int64_t nblocks, hipStream_t s) {
  const int64_t nchunks = nblocks * 4;
  mxfp4_quantize_kernel<<<grid_for(nchunks, kThreads * kUnroll, 8192), kThreads, 0, s>>>(
      reinterpret_cast<const u32x4*>(w), reinterpret_cast<uint32_t*>(q), scales, nchunks);
  return hipGetLastError();
}

hipError_t launch_dequantize_mxfp4(const uint8_t* q, const uint8_t* scales, uint16_t* out, int64_t nblocks,
                                   hipStream_t s) {
  const int64_t nchunks = nblocks * 4;
  mxfp4_dequantize_kernel<<<grid_for(nchunks, kThreads, 16384), kThreads, 0, s>>>(
      reinterpret_cast<const uint32_t*>(q), scales, reinterpret_cast<u32x4*>(out), nchunks);
  return hipGetLastError();
}

}  // namespace moeq
