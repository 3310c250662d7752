// Orthogonalised updates (gfx950): for each of a batch of matrices G, the
// Newton-Schulz steps that move its singular values towards 1 and keep its
// singular vectors,
//
//   X = G / |G|_F,   A = X X^T,   P = a I + b A + c A A,   X <- P X
//
// (A = X^T X and X <- X P where G is taller than wide, so that A has the
// shorter side).  Three products a step, on the tile engine of
// grouped_tile.h; the polynomial is the second one's epilogue.
//
// Precision.  X, A and P are kept in fp16, not in bf16: all three are bounded
// (singular values up to about 1.2, |G|_F = 1 at the start), so fp16's range is
// enough, its eight times smaller rounding shows in the result (Gaussian 512 x
// 1024, five steps: 1.3e-3 off before the output's rounding, bf16 working
// matrices 1.1e-2), and its products run at the same rate.  Powers of two keep
// the entries in fp16's normal range: X times 2^s, s = floor(log2(sqrt(m))) with
// m the longer side, so that entries of an orthogonal matrix are around 1, A times
// 2^8, and P times 2^8 or less (Poly).  Sums are fp32, the norm's fp64.  What the
// rounding adds to directions that the matrix lacks grows by a from step to step as
// small singular values do.  Off after five steps with a = 3.4445, [512, 1024]: rank
// one 15 %, two and four 7 %, eight and sixteen 4.3 %, 64 2.2 %, 256 0.75 %, full rank
// 0.21 %; [512, 512] and [1024, 2048] within a third of that.
//
// Measured, median us of a product, five steps each: 8 matrices of [4096, 14336]
// A 1850, P 590, P X 3010 (1.28 PFLOP/s, matrix cores 81 % busy at 1.49 GHz, which
// the card's power leaves; half of A and P is computed), start 650.  64 of [2048,
// 1024] 190, 122, 270 (1.0 PFLOP/s): 640 tiles of half the products and 1024 of the
// whole ones, of 16 to 32 steps, whose first copies and stores nothing covers.
#include <cmath>

#include "grouped_tile.h"

#include "ortho.h"

namespace moeq {
namespace {

constexpr int kShift = 8;   // A is stored times 2^kShift

// A step's polynomial as its kernels take it: P times 2^k from A times 2^8, and
// what takes a product with it back.  No entry of P is larger than its 2-norm, the
// largest |a + b s^2 + c s^4| of a singular value s (0 among them): at most |a| + |b|
// + |c| up to s = 1, and beyond 1, where the step's result keeps s below 16, below
// 16 itself.  k = 8 as long as 2^8 (|a| + |b| + |c|) <= 2^15, half of fp16's range;
// past that, which a alone reaches at 128, as much less as it takes, so that an entry
// is off by 2^-11 of itself or by 2^-39 (|a| + |b| + |c|).
struct Poly {
  float a, b, c, down;
};
Poly poly_of(const float* abc) {
  const double sum = std::fabs((double)abc[0]) + std::fabs((double)abc[1]) + std::fabs((double)abc[2]);
  int k = kShift;
  while (std::ldexp(sum, k) > 0x1p15) --k;
  return {std::ldexp(abc[0], k), std::ldexp(abc[1], k - kShift), std::ldexp(abc[2], k - 2 * kShift), std::ldexp(1.0f, -k)};
}

__device__ __forceinline__ float bf16_value(uint16_t b) { return __builtin_bit_cast(float, (uint32_t)b << 16); }
__device__ __forceinline__ float value(const uint16_t* p) { return bf16_value(*p); }
__device__ __forceinline__ float value(const float* p) { return *p; }

// Eight values from p on: those before `n`, zeros behind.
template <typename T>
__device__ __forceinline__ void load8(const T* p, int64_t n, bool wide, float (&v)[8]) {
  if (wide) {
    if constexpr (sizeof(T) == 4) {
      const float4 lo = reinterpret_cast<const float4*>(p)[0], hi = reinterpret_cast<const float4*>(p)[1];
      v[0] = lo.x; v[1] = lo.y; v[2] = lo.z; v[3] = lo.w;
      v[4] = hi.x; v[5] = hi.y; v[6] = hi.z; v[7] = hi.w;
    } else {
      const u32x4 b = *reinterpret_cast<const u32x4*>(p);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[2 * i] = __builtin_bit_cast(float, b[i] << 16);
        v[2 * i + 1] = __builtin_bit_cast(float, b[i] & 0xffff0000u);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < n ? value(p + i) : 0.0f;
  }
}

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int d = 1; d < 64; d *= 2) v += __shfl_xor(v, d);
  return v;
}

// Sum of squares of chunk blockIdx.x of matrix blockIdx.y, in a fixed order.
template <typename T>
__global__ __launch_bounds__(256) void ortho_squares_kernel(const T* g, int64_t size, bool wide, double* partial) {
  __shared__ double part[4];
  const int64_t per = ((size + gridDim.x - 1) / gridDim.x + 7) / 8 * 8;
  const int64_t lo = per * blockIdx.x, hi = min(lo + per, size);
  const T* p = g + size * blockIdx.y;
  double s = 0.0;
  for (int64_t i = lo + 8 * threadIdx.x; i < hi; i += 8 * 256) {
    float v[8];
    load8(p + i, hi - i, wide, v);
#pragma unroll
    for (int j = 0; j < 8; ++j) s += (double)v[j] * (double)v[j];
  }
  s = wave_sum(s);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = s;
  __syncthreads();
  if (threadIdx.x == 0) partial[(int64_t)blockIdx.y * gridDim.x + blockIdx.x] = part[0] + part[1] + part[2] + part[3];
}

// X = G 2^s / |G| of matrix blockIdx.y, columns padded with zeros to xc.  A
// matrix of zeros stays one.
template <typename T>
__global__ __launch_bounds__(256) void ortho_scale_kernel(const T* g, int32_t N, int32_t K, int32_t xc, bool wide,
                                                          const double* partial, int32_t chunks, double times, _Float16* x) {
  static_assert(kOrthoMaxChunks == 64, "a partial sum a lane");
  const int lane = threadIdx.x & 63;
  const double sum = wave_sum(lane < chunks ? partial[(int64_t)blockIdx.y * chunks + lane] : 0.0);
  const double f = sum == 0.0 ? 0.0 : times / sqrt(sum);   // (an infinity or a NaN of G: NaN or 0 times inf below)
  // in fp32 where it can hold the factor (the same to fp16's rounding), which is quicker
  const bool narrow = f > 0x1p-100 && f < 0x1p100;
  const float f32 = (float)f;
  const T* p = g + (int64_t)N * K * blockIdx.y;
  _Float16* o = x + (int64_t)N * xc * blockIdx.y;
  const uint32_t groups = xc / 8;
  const int64_t total = (int64_t)N * groups;   // (fits 32 bits: N K < 2^34, and N <= 2^20)
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
    const int64_t r = (uint32_t)i / groups;
    const int c = 8 * (int)(i - r * groups);
    float v[8];
    load8(p + r * K + c, K - c, wide, v);
    f16x8 h;
#pragma unroll
    for (int j = 0; j < 8; ++j) h[j] = (_Float16)(narrow ? v[j] * f32 : (float)((double)v[j] * f));
    *reinterpret_cast<f16x8*>(o + r * xc + c) = h;
  }
}

// One batched product: out [rows][cols] of each matrix from the columns' operand
// w and the rows' operand x, contraction kc.  Pitches ld* in elements (a
// multiple of 8), matrices [strides] apart.  Which layouts w and x have, and what
// becomes of the sums, the kernel's parameters say.
enum class Then { kGram, kPoly, kApply, kOut };
struct OrthoProduct {
  const _Float16 *w, *x;
  void* out;
  int32_t E, rows, cols, kc, ldw, ldx, ldo;
  int64_t sw, sx, so;
  const _Float16* a16 = nullptr;   // kPoly: A
  float a = 0.f, b = 0.f, c = 0.f, times = 1.f;
};

// A and P are symmetric: of those the tiles on and below the diagonal are
// computed, and stored on both sides.
constexpr bool symmetric(Then t) { return t == Then::kGram || t == Then::kPoly; }
constexpr int64_t triangle(int64_t n) { return n * (n + 1) / 2; }

typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
struct ScaledF16 {
  float times;
  __device__ __forceinline__ uint32_t operator()(float lo, float hi) const {
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{lo * times, hi * times}), f16x2));
  }
};
struct ScaledBf16 {
  float times;
  __device__ __forceinline__ uint32_t operator()(float lo, float hi) const { return pack_bf16x2(lo * times, hi * times); }
};

// Tile q of a matrix's nr x nc, row tiles in groups that go through the column
// tiles together.
template <bool kTriangle>
__device__ __forceinline__ void tile_at(int q, int nr, int nc, int& rt, int& ct) {
  if constexpr (!kTriangle) {
    const int grp = q / (kTileGroup * nc), gt = min(kTileGroup, nr - grp * kTileGroup), rr = q - grp * kTileGroup * nc;
    ct = rr / gt;
    rt = grp * kTileGroup + rr % gt;
  } else {
    int first = 0;   // row of the group
    while (first + kTileGroup < nr && q >= (int)triangle(first + kTileGroup)) first += kTileGroup;
    const int gt = min(kTileGroup, nr - first);
    int r = q - (int)triangle(first);
    if (r < (first + 1) * gt) {   // columns that all of its rows have
      ct = r / gt;
      rt = first + r % gt;
    } else {                      // then one row less each
      r -= (first + 1) * gt;
      int k = 1;
      while (r >= gt - k) r -= gt - k++;
      ct = first + k;
      rt = ct + r;
    }
  }
}

template <Then kThen, bool kAT, bool kBT, int kNWN, int kNWM, int kTN, int kTM, int kBufsA, int kBufsB>
__global__ __launch_bounds__(64 * kNWN * kNWM, kNWN * kNWM / 4) void ortho_kernel(OrthoProduct g) {
  using T = Tile<Op::kF16, kAT, kBT, kNWN, kNWM, kTN, kTM, kBufsA, kBufsB>;
  constexpr bool kMirror = symmetric(kThen);
  static_assert(!kMirror || T::kRows == T::kCols, "square tiles");
  // the wave's piece of LDS: 32 rows in fp32, and the same turned in fp16
  constexpr int kPitch = 128 * kTN + 16, kTurned = 64 + 16, kPiece = 32 * kPitch + 32 * kTN * kTurned;
  __shared__ __attribute__((aligned(16))) char smem[imax(T::kLds, kMirror ? T::kNW * kPiece : T::out_bytes(4))];
  const int nc = (g.cols + T::kCols - 1) / T::kCols, nr = (g.rows + T::kRows - 1) / T::kRows;
  const int tiles = kMirror ? (int)triangle(nr) : nr * nc;
  const int at = work_item(g.E * tiles, kTileGroup * nc);
  if (at >= g.E * tiles) return;
  const int e = at / tiles;
  int rt, ct;
  tile_at<kMirror>(at - e * tiles, nr, nc, rt, ct);
  const int c0 = ct * T::kCols, r0 = rt * T::kRows;
  const int t = threadIdx.x, lane = t & 63, wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const int nrows = min(T::kRows, g.rows - r0), ncols = min(T::kCols, g.cols - c0);
  const char* w = reinterpret_cast<const char*>(g.w + g.sw * e);
  const char* x = reinterpret_cast<const char*>(g.x + g.sx * e);
  typename T::A a;
  typename T::B b;
  const int kbytes = (g.kc + 7) / 8 * 16;   // (a row's padding is zeros)
  if constexpr (kAT)
    a.init(w + 2 * c0, (int64_t)g.kc * g.ldw * 2 - 2 * c0, 2 * g.ldw, 0, wave, lane);
  else
    a.init(w + (int64_t)c0 * g.ldw * 2, (int64_t)ncols * g.ldw * 2, 2 * g.ldw, kbytes, wave, lane);
  if constexpr (kBT)
    b.init(x + 2 * r0, (int64_t)g.kc * g.ldx * 2 - 2 * r0, 2 * g.ldx, 0, wave, lane);
  else
    b.init(x + (int64_t)r0 * g.ldx * 2, (int64_t)nrows * g.ldx * 2, 2 * g.ldx, kbytes, wave, lane);
  f32x16 acc[kTN][kTM];
#pragma unroll
  for (int n = 0; n < kTN; ++n)
#pragma unroll
    for (int m = 0; m < kTM; ++m) acc[n][m] = (f32x16){};
  T::run(smem, a, b, nullptr, 0, (g.kc + 63) / 64, acc);

  const int64_t base = g.so * e;
  if constexpr (kMirror) {
    // Rows and columns up to the pitch: what lies behind the matrix is sums of
    // zeros, and fills the padding.
    const _Float16* a16 = g.a16 + base;
    _Float16* out = static_cast<_Float16*>(g.out) + base;
    constexpr int kLanes = 4 * kTN, kRowsAt = 64 / kLanes;
    const int wn = wave % kNWN, wm = wave / kNWN, l32 = lane & 31, h = lane >> 5;
    char *buf = smem + wave * kPiece, *turned = buf + 32 * kPitch;
    const int lc = 8 * (lane % kLanes), c = c0 + 32 * kTN * wn + lc, cw = c0 + 32 * kTN * wn;
#pragma unroll
    for (int m = 0; m < kTM; ++m) {
      const int rw = r0 + 32 * (kTM * wm + m);
      if (rw >= g.ldo) break;
#pragma unroll
      for (int n = 0; n < kTN; ++n)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const f32x16& v = acc[n][m];
          *reinterpret_cast<float4*>(buf + l32 * kPitch + 4 * (32 * n + 8 * q + 4 * h)) =
              make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
        }
      // (a wave's LDS accesses are done in order)
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront", "local");
      __builtin_amdgcn_wave_barrier();
#pragma unroll
      for (int u = 0; u < 32 / kRowsAt; ++u) {
        const int lr = u * kRowsAt + lane / kLanes, r = rw + lr;
        const float4 lo = *reinterpret_cast<const float4*>(buf + lr * kPitch + 4 * lc);
        const float4 hi = *reinterpret_cast<const float4*>(buf + lr * kPitch + 4 * lc + 16);
        const float v[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
        f16x8 o;
        if constexpr (kThen == Then::kPoly) {
          f16x8 in = {};
          if (r < g.rows && c < g.ldo) in = *reinterpret_cast<const f16x8*>(a16 + (int64_t)r * g.ldo + c);
#pragma unroll
          for (int i = 0; i < 8; ++i)
            o[i] = (_Float16)((r == c + i && r < g.rows ? g.a : 0.f) + (g.b * (float)in[i] + g.c * v[i]));
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) o[i] = (_Float16)(v[i] * g.times);
        }
        if (r < g.rows && c < g.ldo) *reinterpret_cast<f16x8*>(out + (int64_t)r * g.ldo + c) = o;
        if (rt != ct)
#pragma unroll
          for (int i = 0; i < 8; ++i) *reinterpret_cast<_Float16*>(turned + (lc + i) * kTurned + 2 * lr) = o[i];
      }
      if (rt != ct) {
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront", "local");
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int k = 0; k < 2 * kTN; ++k) {
          const int lr = 16 * k + lane / 4, r = cw + lr, cc = rw + 8 * (lane & 3);
          const f16x8 o = *reinterpret_cast<const f16x8*>(turned + lr * kTurned + 16 * (lane & 3));
          if (r < g.rows && cc < g.ldo) *reinterpret_cast<f16x8*>(out + (int64_t)r * g.ldo + cc) = o;
        }
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront", "local");
      __builtin_amdgcn_wave_barrier();
    }
  } else {
    // (columns up to the pitch: sums of zeros fill the padding)
    const int width = min(T::kCols, (kThen == Then::kOut ? g.cols : g.ldo) - c0);
    uint16_t* out = static_cast<uint16_t*>(g.out) + base + (int64_t)r0 * g.ldo + c0;
    if constexpr (kThen == Then::kApply)
      T::store(smem, acc, out, g.ldo, nrows, width, ScaledF16{g.times});
    else if (g.ldo % 8 == 0)
      T::store(smem, acc, out, g.ldo, nrows, width, ScaledBf16{g.times});
    else
      T::each8(
          smem, acc, nrows, width, [](int, int) { return 0; },
          [&](int r, int c, const float (&v)[8], int) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
              if (c + i < width) out[(int64_t)r * g.ldo + c + i] = (uint16_t)pack_bf16x2(v[i] * g.times, 0.f);
          });
  }
}

template <Then kThen, bool kAT, bool kBT, int kNWN, int kNWM, int kTN, int kTM, int kBufsA, int kBufsB>
hipError_t launch_shape(const OrthoProduct& g, hipStream_t s) {
  using T = Tile<Op::kF16, kAT, kBT, kNWN, kNWM, kTN, kTM, kBufsA, kBufsB>;
  const int64_t nr = (g.rows + T::kRows - 1) / T::kRows, tiles = symmetric(kThen) ? triangle(nr) : nr * ((g.cols + T::kCols - 1) / T::kCols);
  ortho_kernel<kThen, kAT, kBT, kNWN, kNWM, kTN, kTM, kBufsA, kBufsB>
      <<<(unsigned)items_grid(g.E * tiles), 64 * kNWN * kNWM, 0, s>>>(g);
  return hipGetLastError();
}

// The largest tiles of 256, 128 or 64 that give each of 256 compute units one.
// us of five steps with tiles of 64, of 128, of 256 throughout:
//   1 x [1024, 1024] 140, 267, 428      16 x [1024, 1024]  797,  634,  585
//   1 x [2048, 2048] 422, 474, 677      4 x [2048, 4096]  2105, 1749, 1450
//   32 x [512, 512]  303, 270, 336      64 x [1024, 2048] 5098, 3827, 3203
//   1 x [3000, 3000] 1372, 1081, 1094   1 x [4096, 4096]  2329, 1938, 1596
// For tiles of 128 a symmetric product's half is counted (1 x [2048, 2048], all of
// them and half, 474 and 410, 4 x [1024, 1024] 294 and 260), for tiles of 256 all:
// their half is 160 for 16 x [1024, 1024], where tiles of 128 take longer (602, 580).
template <Then kThen, bool kAT, bool kBT>
hipError_t launch_product(const OrthoProduct& g, hipStream_t s) {
  auto tiles = [&](int size, bool half) {
    const int64_t nr = (g.rows + size - 1) / size;
    return g.E * (half ? triangle(nr) : nr * ((g.cols + size - 1) / size));
  };
  if (g.rows <= 64 || g.cols <= 64 || tiles(128, symmetric(kThen)) < 256)
    return launch_shape<kThen, kAT, kBT, 2, 2, 1, 1, 3, 3>(g, s);
  if (tiles(256, false) < 256) return launch_shape<kThen, kAT, kBT, 2, 2, 2, 2, 2, 2>(g, s);
  return launch_shape<kThen, kAT, kBT, 4, 2, 2, 4, 3, 2>(g, s);
}

// ---------------------------------------------------------------------------
// Few rows (adapters): one workgroup takes a matrix through all steps. X stays in
// registers (in the forms of 8 waves, past 2048 columns, which take all 256, 14 to
// 32 of a lane's others go through scratch memory), in blocks of 16 x 16 as
// v_mfma_f32_16x16x16_f16 leaves its result (lane (c, g): rows 4 g .. + 3 of column
// c), which is also the layout of its second operand, and of its first for a
// symmetric matrix. So A A, the polynomial and X <- P X need no exchange; A = X X^T
// sums over columns, for which a block is turned on its way through the wave's own
// piece of LDS (written in columns, read with ds_read_b64_tr_b16), and the waves'
// sums are added through LDS. One launch instead of three a step: 64 matrices of
// [16, 2048] 124 us in tiles, 21 us here (1024 of them 769 and 68; 64 of [32, 4096]
// 218 and 87).
// ---------------------------------------------------------------------------
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

struct OrthoSteps {
  Poly poly[kOrthoMaxSteps];
};
constexpr int kBatch = 4;

// kNW waves; kNB blocks of 16 rows, kCB of 16 columns a wave.
template <typename T, bool kTall, int kNW, int kNB, int kCB>
__global__ __launch_bounds__(64 * kNW) void ortho_few_kernel(const T* g, int32_t n, int32_t m, bool wide, int32_t steps,
                                                                   OrthoSteps table, float scale, uint16_t* out) {
  __shared__ __attribute__((aligned(16))) char turn[kNW][kBatch * kNB * 512];
  __shared__ __attribute__((aligned(16))) f32x4 part[kNW][kNB * kNB][64];
  __shared__ double sums[kNW];
  const int t = threadIdx.x, lane = t & 63, wave = __builtin_amdgcn_readfirstlane(t >> 6), l16 = lane & 15, grp = lane >> 4;
  const int64_t size = (int64_t)n * m;
  g += size * blockIdx.x;
  out += size * blockIdx.x;

  double s = 0.0;
  for (int64_t i = 8 * t; i < size; i += 8 * 64 * kNW) {
    float v[8];
    load8(g + i, size - i, wide, v);
#pragma unroll
    for (int j = 0; j < 8; ++j) s += (double)v[j] * (double)v[j];
  }
  s = wave_sum(s);
  if (lane == 0) sums[wave] = s;
  __syncthreads();
  double sum = 0.0;
  for (int i = 0; i < kNW; ++i) sum += sums[i];
  const double f = sum == 0.0 ? 0.0 : (double)scale / sqrt(sum);

  // element (r, c) of X is at r m + c of a wide matrix and at c n + r of a tall one
  const bool four = wide && n % 4 == 0;   // a lane's four rows of a tall matrix are one access
  auto column = [&](int b) { return 16 * (kNW * b + wave) + l16; };
  const bool narrow = f > 0x1p-100 && f < 0x1p100;   // (as ortho_scale_kernel)
  const float f32 = (float)f;
  const __amdgpu_buffer_rsrc_t from = buffer(reinterpret_cast<const char*>(g), size * (int64_t)sizeof(T));
  f16x4 x[kNB][kCB];
#pragma unroll
  for (int b = 0; b < kCB; ++b) {
    const int c = column(b);
#pragma unroll
    for (int i = 0; i < kNB; ++i) {
      float v[4];
      if (kTall && four) {
        const int r = 16 * i + 4 * grp, off = (int)(r < n && c < m ? sizeof(T) * (uint32_t)(c * n + r) : kPast);
        if constexpr (sizeof(T) == 2) {
          const auto q = __builtin_bit_cast(uint2, __builtin_amdgcn_raw_buffer_load_b64(from, off, 0, 0));
          v[0] = __builtin_bit_cast(float, q.x << 16);
          v[1] = __builtin_bit_cast(float, q.x & 0xffff0000u);
          v[2] = __builtin_bit_cast(float, q.y << 16);
          v[3] = __builtin_bit_cast(float, q.y & 0xffff0000u);
        } else {
          const float4 q = __builtin_bit_cast(float4, buffer_load16(from, (uint32_t)off));
          v[0] = q.x;
          v[1] = q.y;
          v[2] = q.z;
          v[3] = q.w;
        }
      } else
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int r = 16 * i + 4 * grp + j;
        const uint32_t at = sizeof(T) * (kTall ? (uint32_t)(c * n + r) : (uint32_t)(r * m + c));
        const int off = (int)(r < n && c < m ? at : kPast);   // (past the end: 0)
        if constexpr (sizeof(T) == 2)
          v[j] = bf16_value((uint16_t)__builtin_amdgcn_raw_buffer_load_b16(from, off, 0, 0));
        else
          v[j] = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(from, off, 0, 0));
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) x[i][b][j] = (_Float16)(narrow ? v[j] * f32 : (float)((double)v[j] * f));
      asm volatile("" : "+v"(x[i][b]));   // (in two registers from here on)
    }
    if (b % 4 == 3) __builtin_amdgcn_sched_barrier(0);   // (all loads at once would not fit the registers)
  }
  const float gram_times = (float)(1 << kShift) / scale / scale;
  char* mine = turn[wave];
  f16x4 p16[kNB][kNB];
  // P X of column block b
  auto apply = [&](int b, f32x4 (&y)[kNB]) {
#pragma unroll
    for (int i = 0; i < kNB; ++i) {
      y[i] = (f32x4){0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int q = 0; q < kNB; ++q) y[i] = __builtin_amdgcn_mfma_f32_16x16x16f16(p16[q][i], x[q][b], y[i], 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < kNB; ++i) mfma_done(y[i]);
  };
  for (int k = 0;; ++k) {
    f32x4 a[kNB][kNB];
#pragma unroll
    for (int i = 0; i < kNB; ++i)
#pragma unroll
      for (int j = 0; j < kNB; ++j) a[i][j] = (f32x4){0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int b0 = 0; b0 < kCB; b0 += kBatch) {
#pragma unroll
      for (int b = 0; b < kBatch; ++b)
#pragma unroll
        for (int i = 0; i < kNB; ++i)
          *reinterpret_cast<f16x4*>(mine + (b * kNB + i) * 512 + 32 * l16 + 8 * grp) = x[i][b0 + b];
      // (a wave's LDS accesses are done in order)
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront", "local");
      __builtin_amdgcn_wave_barrier();
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        f16x4 rows[kNB];
#pragma unroll
        for (int i = 0; i < kNB; ++i)
          rows[i] = __builtin_bit_cast(f16x4, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                                                  (lds_v4i16*)(mine + (b * kNB + i) * 512 + 8 * lane)));
#pragma unroll
        for (int i = 0; i < kNB; ++i)
#pragma unroll
          for (int j = 0; j < kNB; ++j)
            a[i][j] = __builtin_amdgcn_mfma_f32_16x16x16f16(rows[i], rows[j], a[i][j], 0, 0, 0);
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront", "local");
      __builtin_amdgcn_wave_barrier();
      __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int i = 0; i < kNB; ++i)
#pragma unroll
      for (int j = 0; j < kNB; ++j) {
        mfma_done(a[i][j]);
        part[wave][i * kNB + j][lane] = a[i][j];
      }
    __syncthreads();
    f16x4 a16[kNB][kNB];
#pragma unroll
    for (int i = 0; i < kNB; ++i)
#pragma unroll
      for (int j = 0; j < kNB; ++j) {
        f32x4 v = part[0][i * kNB + j][lane];
#pragma unroll 5
        for (int w = 1; w < kNW; ++w) {
          const f32x4 q = part[w][i * kNB + j][lane];
#pragma unroll
          for (int z = 0; z < 4; ++z) v[z] += q[z];
        }
#pragma unroll
        for (int z = 0; z < 4; ++z) a16[i][j][z] = (_Float16)(v[z] * gram_times);
      }
    __syncthreads();   // (before the next step's sums)
    // (2^8 A)(2^8 A): a symmetric matrix's block (k, i) is the first operand's (i, k)
    const Poly c = table.poly[k];
#pragma unroll
    for (int i = 0; i < kNB; ++i)
#pragma unroll
      for (int j = 0; j < kNB; ++j) {
        f32x4 v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int q = 0; q < kNB; ++q) v = __builtin_amdgcn_mfma_f32_16x16x16f16(a16[q][i], a16[q][j], v, 0, 0, 0);
        mfma_done(v);
#pragma unroll
        for (int z = 0; z < 4; ++z)
          p16[i][j][z] = (_Float16)((i == j && 4 * grp + z == l16 ? c.a : 0.f) + (c.b * (float)a16[i][j][z] + c.c * v[z]));
      }
    if (k + 1 >= steps) break;
#pragma unroll
    for (int b = 0; b < kCB; ++b) {   // (blocks behind the last are zeros, and stay so)
      f32x4 y[kNB];
      apply(b, y);
#pragma unroll
      for (int i = 0; i < kNB; ++i)
#pragma unroll
        for (int z = 0; z < 4; ++z) x[i][b][z] = (_Float16)(y[i][z] * c.down);
#pragma unroll
      for (int i = 0; i < kNB; ++i) asm volatile("" : "+v"(x[i][b]));
      if (b % 4 == 3) __builtin_amdgcn_sched_barrier(0);
    }
  }
  // (addresses made anew, not kept from the loads through all steps)
  const __amdgpu_buffer_rsrc_t to = buffer(reinterpret_cast<const char*>(out), size * 2);
  const float last = table.poly[steps - 1].down / scale;
  int c0 = 16 * wave + l16, r0 = 4 * grp;
  asm volatile("" : "+v"(c0), "+v"(r0));
#pragma unroll
  for (int b = 0; b < kCB; ++b) {
    f32x4 y[kNB];
    apply(b, y);
    const int c = c0 + 16 * kNW * b;
#pragma unroll
    for (int i = 0; i < kNB; ++i)
      if (kTall && four) {
        const int r = 16 * i + r0, off = (int)(r < n && c < m ? 2u * (uint32_t)(c * n + r) : kPast);
        const uint2 q = make_uint2(pack_bf16x2(y[i][0] * last, y[i][1] * last), pack_bf16x2(y[i][2] * last, y[i][3] * last));
        __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(u32x2, q), to, off, 0, 0);
      } else
#pragma unroll
      for (int z = 0; z < 4; ++z) {
        const int r = 16 * i + r0 + z;
        const uint32_t at = 2u * (kTall ? (uint32_t)(c * n + r) : (uint32_t)(r * m + c));
        __builtin_amdgcn_raw_buffer_store_b16((short)pack_bf16x2(y[i][z] * last, 0.f), to, (int)(r < n && c < m ? at : kPast), 0,
                                              0);
      }
    __builtin_amdgcn_sched_barrier(0);
  }
}

// Whether a matrix fits a workgroup's registers: up to 16 waves of 8 column
// blocks, or 8 waves, which have twice the registers, of 64 (for two row blocks 32).
bool few(const OrthoPlan& p) { return p.n <= 32 && p.m <= (p.n <= 16 ? 8192 : 4096); }

template <typename T, bool kTall>
hipError_t launch_few(const T* g, const OrthoPlan& p, const OrthoSteps& table, int32_t steps, float scale, uint16_t* out,
                      hipStream_t s) {
  const bool wide = reinterpret_cast<uintptr_t>(g) % 16 == 0 && (int64_t)p.n * p.m % 8 == 0;
  auto go = [&](auto kernel, int waves) {
    kernel<<<(unsigned)p.E, 64 * waves, 0, s>>>(g, p.n, p.m, wide, steps, table, scale, out);
  };
  if (p.n <= 16 && p.m <= 2048)
    go(ortho_few_kernel<T, kTall, 16, 1, 8>, 16);
  else if (p.n <= 16)
    go(ortho_few_kernel<T, kTall, 8, 1, 64>, 8);
  else if (p.m <= 2048)
    go(ortho_few_kernel<T, kTall, 16, 2, 8>, 16);
  else
    go(ortho_few_kernel<T, kTall, 8, 2, 32>, 8);
  return hipGetLastError();
}

template <typename T>
hipError_t launch_start(const T* g, const OrthoPlan& p, double times, double* partial, _Float16* x, hipStream_t s) {
  const int64_t size = (int64_t)p.N * p.K;
  const bool aligned = reinterpret_cast<uintptr_t>(g) % 16 == 0;
  ortho_squares_kernel<T><<<dim3(p.chunks, p.E), 256, 0, s>>>(g, size, aligned && size % 8 == 0, partial);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  // (a workgroup takes several turns: each begins with the norm)
  const int64_t blocks = ((int64_t)p.N * (p.xc / 8) + 255) / 256, most = std::max<int64_t>(1, 8192 / p.E);
  ortho_scale_kernel<T><<<dim3((unsigned)std::min(blocks, most), p.E), 256, 0, s>>>(
      g, p.N, p.K, p.xc, aligned && p.K % 8 == 0, partial, p.chunks, times, x);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_orthogonalize(const void* grad, bool fp32, const OrthoPlan& p, const float* coefficients, int32_t steps,
                                uint16_t* out, void* workspace, hipStream_t s) {
  int shift = 0;
  while (shift < 15 && (int64_t(1) << (2 * (shift + 1))) <= p.m) ++shift;
  if (few(p)) {
    OrthoSteps table = {};
    for (int i = 0; i < steps; ++i) table.poly[i] = poly_of(coefficients + 3 * i);
    const float scale = (float)(1 << shift);
    const uint16_t* g16 = static_cast<const uint16_t*>(grad);
    const float* g32 = static_cast<const float*>(grad);
    if (p.tall)
      return fp32 ? launch_few<float, true>(g32, p, table, steps, scale, out, s)
                  : launch_few<uint16_t, true>(g16, p, table, steps, scale, out, s);
    return fp32 ? launch_few<float, false>(g32, p, table, steps, scale, out, s)
                : launch_few<uint16_t, false>(g16, p, table, steps, scale, out, s);
  }
  char* ws = static_cast<char*>(workspace);
  double* partial = reinterpret_cast<double*>(ws + p.partial);
  _Float16 *x = reinterpret_cast<_Float16*>(ws + p.x), *y = reinterpret_cast<_Float16*>(ws + p.y);
  _Float16 *a = reinterpret_cast<_Float16*>(ws + p.a), *poly = reinterpret_cast<_Float16*>(ws + p.p);
  hipError_t e = fp32 ? launch_start(static_cast<const float*>(grad), p, (double)(1 << shift), partial, x, s)
                      : launch_start(static_cast<const uint16_t*>(grad), p, (double)(1 << shift), partial, x, s);
  const int64_t sx = (int64_t)p.N * p.xc, sa = (int64_t)p.n * p.nc;
  for (int i = 0; i < steps && e == hipSuccess; ++i) {
    const Poly c = poly_of(coefficients + 3 * i);
    OrthoProduct gram = {x, x, a, p.E, p.n, p.n, p.m, p.xc, p.xc, p.nc, sx, sx, sa};
    gram.times = (float)(1 << kShift) / (float)(1 << shift) / (float)(1 << shift);
    e = p.tall ? launch_product<Then::kGram, true, true>(gram, s) : launch_product<Then::kGram, false, false>(gram, s);
    if (e != hipSuccess) break;
    // (2^8 A)(2^8 A): A is symmetric, so its rows serve as its columns
    OrthoProduct square = {a, a, poly, p.E, p.n, p.n, p.n, p.nc, p.nc, p.nc, sa, sa, sa};
    square.a16 = a;
    square.a = c.a;
    square.b = c.b;
    square.c = c.c;
    e = launch_product<Then::kPoly, false, false>(square, s);
    if (e != hipSuccess) break;
    const bool last = i + 1 == steps;
    OrthoProduct apply = {poly, x, y, p.E, p.N, p.K, p.n, p.nc, p.xc, p.xc, sa, sx, sx};   // tall: X P, P symmetric
    if (!p.tall) {
      apply.w = x;
      apply.x = poly;
      apply.ldw = p.xc;
      apply.ldx = p.nc;
      apply.sw = sx;
      apply.sx = sa;
    }
    apply.times = c.down;
    if (last) {
      apply.out = out;
      apply.ldo = p.K;
      apply.so = (int64_t)p.N * p.K;
      apply.times = c.down / (float)(1 << shift);
      e = p.tall ? launch_product<Then::kOut, false, false>(apply, s) : launch_product<Then::kOut, true, false>(apply, s);
    } else {
      e = p.tall ? launch_product<Then::kApply, false, false>(apply, s) : launch_product<Then::kApply, true, false>(apply, s);
      std::swap(x, y);
    }
  }
  return e;
}

}  // namespace moeq
