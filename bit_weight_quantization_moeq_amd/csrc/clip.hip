// Norm of the gradients of a training step and their clipping (gfx950):
//
//   norm = sqrt(sum of g^2 over every tensor)
//   dst  = src * min(1, max_norm / norm)
//
// for any number of bf16 and fp32 tensors ("MoE Expert Quantization", Axolotl
// docs, Expert LoRA targeting: adapters and routers train beside the frozen
// experts).  Two passes over the data, both bound by HBM, each in one launch
// per kTable tensors, with a small kernel between them:
//   sum_kernel    adds the squares of its chunks (a chunk lies in one tensor)
//                 in fp64; one partial sum per workgroup;
//   norm_kernel   one workgroup adds the partial sums in a fixed order and
//                 leaves the norm and the factor;
//   scale_kernel  one workgroup per chunk.
// A square of an fp32 or bf16 value is exact in fp64 and cannot overflow it,
// so the norm is right to fp32 for every finite gradient; one past fp32's range
// is an infinity in the result alone, the factor comes from its fp64 value.
//
// Measured, 2.0 GB of fp32 into another buffer: sum 371-383 us (5.3 TB/s), norm
// 4.6 us, scale 870-900 us (4.5 TB/s, the rate of an elementwise product of
// the same tensors).  One workgroup per chunk of 32 KB in the scaling: a
// persistent grid took 1.01 ms.
//
// The tensors' addresses travel in the kernel arguments: nothing is copied to
// the device, and a call can be captured into a graph.
#include "grouped.h"

namespace moeq {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef u32x4 u32x4a __attribute__((aligned(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

constexpr int kThreads = 256;
constexpr int kTable = 96;            // tensors per launch (the kernel arguments hold the table)
constexpr int kMaxGrid = kClipPartials;
constexpr int kUnroll = 8;             // 16-byte vectors of a thread in flight
constexpr int64_t kChunkBytes = 16 * kThreads * kUnroll;

struct Entry {
  const void* src;
  void* dst;
  int64_t n;
  int64_t first;  // chunks before this tensor's
};
struct Table {
  Entry e[kTable];
  uint32_t fp32[kTable / 32];  // bit i: tensor i is fp32, else bf16
  int32_t count;
  int64_t chunks;
};

__device__ __forceinline__ bool is_fp32(const Table& t, int i) { return (t.fp32[i >> 5] >> (i & 31)) & 1u; }

// elements per chunk
__host__ __device__ __forceinline__ int64_t chunk_of(bool fp32) { return kChunkBytes / (fp32 ? 4 : 2); }

// Tensor that holds chunk c: the lanes look at all of the table at once.
__device__ __forceinline__ int tensor_of(const Table& t, int64_t c) {
  const int lane = threadIdx.x & 63;
  int n = 0;
#pragma unroll
  for (int i = 0; i < kTable; i += 64)
    n += __popcll(__ballot(i + lane < t.count && t.e[min(i + lane, kTable - 1)].first <= c));
  return __builtin_amdgcn_readfirstlane(n - 1);
}

// 16 bytes of a tensor as fp32 and back.  Tensors are aligned to their
// elements only; the hardware takes 16-byte accesses at any address.
template <typename T>
struct Vec;
template <>
struct Vec<float> {
  static constexpr int kN = 4;
  static __device__ __forceinline__ void unpack(const u32x4& v, float (&f)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = __uint_as_float(v[i]);
  }
  static __device__ __forceinline__ u32x4 pack(const float (&f)[4]) {
    return u32x4{__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3])};
  }
};
template <>
struct Vec<uint16_t> {
  static constexpr int kN = 8;
  static __device__ __forceinline__ void unpack(const u32x4& v, float (&f)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(v[i] << 16);
      f[2 * i + 1] = __uint_as_float(v[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ u32x4 pack(const float (&f)[8]) {
    u32x4 v;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const f32x2 p = {f[2 * i], f[2 * i + 1]};
      v[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(p, bf16x2));
    }
    return v;
  }
};
__device__ __forceinline__ float to_float(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }
__device__ __forceinline__ float to_float(float v) { return v; }
__device__ __forceinline__ void from_float(float v, uint16_t& o) { o = __builtin_bit_cast(uint16_t, (__bf16)v); }
__device__ __forceinline__ void from_float(float v, float& o) { o = v; }

// Calls vec(u, i) for the n / kN whole vectors of a chunk, kUnroll at a time
// with all their loads first, and one(i) for the elements behind them.
template <typename T, typename V, typename O>
__device__ __forceinline__ void each(const T* p, int n, V vec, O one) {
  constexpr int kN = Vec<T>::kN;
  const int nv = n / kN;
  int i = threadIdx.x;
  for (; i + (kUnroll - 1) * kThreads < nv; i += kUnroll * kThreads) {
    u32x4 v[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) v[u] = __builtin_nontemporal_load(reinterpret_cast<const u32x4a*>(p + (int64_t)(i + u * kThreads) * kN));
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) vec(v[u], i + u * kThreads);
  }
  for (; i < nv; i += kThreads) {
    u32x4 v;
    __builtin_memcpy(&v, p + (int64_t)i * kN, 16);
    vec(v, i);
  }
  const int r = nv * kN + (int)threadIdx.x;
  if (r < n) one(r);
}

// Sum over the workgroup, in a fixed order; every thread gets it.
__device__ __forceinline__ double block_sum(double v) {
  __shared__ double part[kThreads / 64];
#pragma unroll
  for (int o = 32; o; o >>= 1) v += __shfl_xor(v, o, 64);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
  __syncthreads();
  double s = part[0];
#pragma unroll
  for (int i = 1; i < kThreads / 64; ++i) s += part[i];
  return s;
}

template <typename T>
__device__ __forceinline__ double chunk_squares(const T* p, int n) {
  double s = 0.0;
  each(
      p, n,
      [&](const u32x4& v, int) {
        float f[Vec<T>::kN];
        Vec<T>::unpack(v, f);
#pragma unroll
        for (int k = 0; k < Vec<T>::kN; ++k) s = __builtin_fma((double)f[k], (double)f[k], s);
      },
      [&](int i) {
        const double g = (double)to_float(p[i]);
        s = __builtin_fma(g, g, s);
      });
  return s;
}

__global__ __launch_bounds__(kThreads) void sum_kernel(Table t, double* __restrict__ partial) {
  double s = 0.0;
  for (int64_t c = blockIdx.x; c < t.chunks; c += gridDim.x) {
    const int i = tensor_of(t, c);
    const int64_t chunk = chunk_of(is_fp32(t, i)), at = (c - t.e[i].first) * chunk;
    const int n = (int)min(chunk, t.e[i].n - at);
    s += is_fp32(t, i) ? chunk_squares(static_cast<const float*>(t.e[i].src) + at, n)
                       : chunk_squares(static_cast<const uint16_t*>(t.e[i].src) + at, n);
  }
  s = block_sum(s);
  if (threadIdx.x == 0) partial[blockIdx.x] = s;
}

// max_norm / norm as m * 2^e, with e = 0 where fp32 holds the quotient as a
// normal number.  Below that (large gradients, a small max_norm) fp32 keeps few
// of its bits or none, but the gradients it scales can come out as normal
// numbers: the product with m is rounded, and 2^e exact where they do.
struct Factor {
  float m;
  int32_t e;
  __device__ __forceinline__ static Factor of(double k) {
    if (!(k < 0x1p-126) || k == 0.0) return {(float)k, 0};
    int e;
    const double m = frexp(k, &e);
    return {(float)m, e};
  }
  __device__ __forceinline__ float times(float g) const { return __builtin_ldexpf(g * m, e); }
};

template <typename T>
__device__ __forceinline__ void chunk_scale(const T* src, T* dst, int n, Factor k) {
  each(
      src, n,
      [&](const u32x4& v, int i) {
        float f[Vec<T>::kN];
        Vec<T>::unpack(v, f);
#pragma unroll
        for (int j = 0; j < Vec<T>::kN; ++j) f[j] = k.times(f[j]);
        const u32x4 o = Vec<T>::pack(f);
        __builtin_nontemporal_store(o, reinterpret_cast<u32x4a*>(dst + (int64_t)i * Vec<T>::kN));
      },
      [&](int i) { from_float(k.times(to_float(src[i])), dst[i]); });
}

// The norm and the factor of every gradient: 1 when there is nothing to clip,
// also for a norm that is no finite number in fp64 (then some gradient is none).
__global__ __launch_bounds__(kThreads) void norm_kernel(const double* __restrict__ partial, int32_t partials,
                                                       double max_norm, float* __restrict__ norm_out,
                                                       Factor* __restrict__ factor) {
  double s = 0.0;
  for (int i = threadIdx.x; i < partials; i += kThreads) s += partial[i];
  const double norm = sqrt(block_sum(s));
  if (threadIdx.x == 0) {
    *norm_out = (float)norm;
    *factor = Factor::of(norm > max_norm && norm < __builtin_inf() ? max_norm / norm : 1.0);
  }
}

__global__ __launch_bounds__(kThreads) void scale_kernel(Table t, const Factor* __restrict__ factor) {
  // from the back: what the sum read last may still be cached
  const int64_t c = t.chunks - 1 - blockIdx.x;
  const int i = tensor_of(t, c);
  const Factor k = *factor;
  if (k.m == 1.0f && k.e == 0 && t.e[i].src == t.e[i].dst) return;  // nothing to change in place
  const int64_t chunk = chunk_of(is_fp32(t, i)), at = (c - t.e[i].first) * chunk;
  const int n = (int)min(chunk, t.e[i].n - at);
  if (is_fp32(t, i))
    chunk_scale(static_cast<const float*>(t.e[i].src) + at, static_cast<float*>(t.e[i].dst) + at, n, k);
  else
    chunk_scale(static_cast<const uint16_t*>(t.e[i].src) + at, static_cast<uint16_t*>(t.e[i].dst) + at, n, k);
}

// Table of the tensors from `from` on; empty tensors take no place.
int32_t fill(Table& t, const moeq_grad* g, int32_t count, int32_t from) {
  t = Table{};
  int32_t i = from;
  for (; i < count && t.count < kTable; ++i) {
    if (g[i].numel == 0) continue;
    Entry& e = t.e[t.count];
    e.src = g[i].src;
    e.dst = g[i].dst;
    e.n = g[i].numel;
    e.first = t.chunks;
    const int64_t chunk = chunk_of(g[i].dtype == MOEQ_DTYPE_FP32);
    t.chunks += (e.n + chunk - 1) / chunk;
    if (g[i].dtype == MOEQ_DTYPE_FP32) t.fp32[t.count >> 5] |= 1u << (t.count & 31);
    ++t.count;
  }
  return i;
}

}  // namespace

int64_t clip_partials(int32_t count) { return ((int64_t)count + kTable - 1) / kTable * kMaxGrid; }

hipError_t launch_clip(const moeq_grad* g, int32_t count, double max_norm, float* norm, double* partial, hipStream_t s) {
  Table t;
  int32_t partials = 0;
  static_assert(sizeof(Factor) <= kClipHead * sizeof(double), "the factor lies in front of the partial sums");
  Factor* factor = reinterpret_cast<Factor*>(partial);
  partial += kClipHead;
  for (int32_t i = 0; i < count;) {
    i = fill(t, g, count, i);
    if (t.count == 0) break;
    const int grid = (int)(t.chunks < kMaxGrid ? t.chunks : kMaxGrid);
    sum_kernel<<<grid, kThreads, 0, s>>>(t, partial + partials);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    partials += grid;
  }
  norm_kernel<<<1, kThreads, 0, s>>>(partial, partials, max_norm, norm, factor);
  hipError_t e = hipGetLastError();
  for (int32_t i = 0; i < count && e == hipSuccess;) {
    i = fill(t, g, count, i);
    if (t.count == 0) break;
    scale_kernel<<<(unsigned)t.chunks, kThreads, 0, s>>>(t, factor);
    e = hipGetLastError();
  }
  return e;
}

}  // namespace moeq
