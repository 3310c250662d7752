// Norm of the gradients of a training step and their clipping (gfx950):
//
//   norm = sqrt(sum of g^2 over every tensor)
//   dst  = src * min(1, max_norm / norm)
//
// for any number of bf16 and fp32 tensors ("MoE Expert Quantization", Axolotl
// docs, Expert LoRA targeting: adapters and routers train beside the frozen
// experts).  Two passes over the data, both bound by HBM, in one launch each
// per kTable tensors:
//   sum_kernel    every workgroup adds the squares of its chunks (a chunk lies
//                 in one tensor) in fp64 and writes one partial sum;
//   scale_kernel  every workgroup adds all partial sums in the same fixed
//                 order (at most a few thousand, from L2), so all of them and
//                 every run get the same norm bits, then scales its chunks.
// A square of an fp32 or bf16 value is exact in fp64 and cannot overflow it,
// so the norm is right to fp32 for every finite gradient.
//
// The tensors' addresses travel in the kernel arguments: nothing is copied to
// the device, and a call can be captured into a graph.
#include "grouped.h"

namespace moeq {
namespace {

constexpr int kThreads = 256;
constexpr int kTable = 96;            // tensors per launch (the kernel arguments hold the table)
constexpr int kMaxGrid = kClipPartials;
constexpr int64_t kChunk = 1 << 14;   // elements per chunk

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

// Tensor that holds chunk c.
__device__ __forceinline__ int tensor_of(const Table& t, int64_t c) {
  int lo = 0, hi = t.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (t.e[mid].first <= c) lo = mid; else hi = mid - 1;
  }
  return lo;
}

__device__ __forceinline__ float get(const uint16_t* p, int64_t i) { return __uint_as_float((uint32_t)p[i] << 16); }
__device__ __forceinline__ float get(const float* p, int64_t i) { return p[i]; }
__device__ __forceinline__ void put(uint16_t* p, int64_t i, float v) {
  p[i] = __builtin_bit_cast(uint16_t, (__bf16)v);
}
__device__ __forceinline__ void put(float* p, int64_t i, float v) { p[i] = v; }

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
__device__ __forceinline__ double chunk_squares(const T* p, int64_t n) {
  double s = 0.0;
  for (int64_t i = threadIdx.x; i < n; i += kThreads) {
    const double g = (double)get(p, i);
    s += g * g;
  }
  return s;
}

__global__ __launch_bounds__(kThreads) void sum_kernel(Table t, double* __restrict__ partial) {
  double s = 0.0;
  for (int64_t c = blockIdx.x; c < t.chunks; c += gridDim.x) {
    const int i = tensor_of(t, c);
    const int64_t at = (c - t.e[i].first) * kChunk, n = min(kChunk, t.e[i].n - at);
    s += is_fp32(t, i) ? chunk_squares(static_cast<const float*>(t.e[i].src) + at, n)
                       : chunk_squares(static_cast<const uint16_t*>(t.e[i].src) + at, n);
  }
  s = block_sum(s);
  if (threadIdx.x == 0) partial[blockIdx.x] = s;
}

template <typename T>
__device__ __forceinline__ void chunk_scale(const T* src, T* dst, int64_t n, float k) {
  for (int64_t i = threadIdx.x; i < n; i += kThreads) put(dst, i, get(src, i) * k);
}

__global__ __launch_bounds__(kThreads) void scale_kernel(Table t, const double* __restrict__ partial, int32_t partials,
                                                        double max_norm, float* __restrict__ norm_out) {
  double s = 0.0;
  for (int i = threadIdx.x; i < partials; i += kThreads) s += partial[i];
  const double norm = sqrt(block_sum(s));
  if (norm_out && blockIdx.x == 0 && threadIdx.x == 0) *norm_out = (float)norm;
  // a norm that is no finite number scales nothing
  const bool clip = norm > max_norm && norm < __builtin_inf();
  const float k = clip ? (float)(max_norm / norm) : 1.0f;
  for (int64_t c = blockIdx.x; c < t.chunks; c += gridDim.x) {
    const int i = tensor_of(t, c);
    if (!clip && t.e[i].src == t.e[i].dst) continue;  // nothing to change in place
    const int64_t at = (c - t.e[i].first) * kChunk, n = min(kChunk, t.e[i].n - at);
    if (is_fp32(t, i))
      chunk_scale(static_cast<const float*>(t.e[i].src) + at, static_cast<float*>(t.e[i].dst) + at, n, k);
    else
      chunk_scale(static_cast<const uint16_t*>(t.e[i].src) + at, static_cast<uint16_t*>(t.e[i].dst) + at, n, k);
  }
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
    t.chunks += (e.n + kChunk - 1) / kChunk;
    if (g[i].dtype == MOEQ_DTYPE_FP32) t.fp32[t.count >> 5] |= 1u << (t.count & 31);
    ++t.count;
  }
  return i;
}

int grid_of(const Table& t) { return (int)(t.chunks < kMaxGrid ? t.chunks : kMaxGrid); }

}  // namespace

int64_t clip_partials(int32_t count) { return ((int64_t)count + kTable - 1) / kTable * kMaxGrid; }

hipError_t launch_clip(const moeq_grad* g, int32_t count, double max_norm, float* norm, double* partial, hipStream_t s) {
  Table t;
  int32_t partials = 0;
  for (int32_t i = 0; i < count;) {
    i = fill(t, g, count, i);
    if (t.count == 0) break;
    const int grid = grid_of(t);
    sum_kernel<<<grid, kThreads, 0, s>>>(t, partial + partials);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    partials += grid;
  }
  int32_t i = 0;
  do {  // (no tensor at all, or only empty ones: one workgroup writes the norm, 0)
    i = fill(t, g, count, i);
    const int grid = t.count ? grid_of(t) : 1;
    scale_kernel<<<grid, kThreads, 0, s>>>(t, partial, partials, max_norm, norm);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    norm = nullptr;  // written by the first launch
  } while (i < count && t.count);
  return hipSuccess;
}

}  // namespace moeq
