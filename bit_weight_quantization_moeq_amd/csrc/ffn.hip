// The gated feed-forward block of experts over rows sorted by expert (gfx950),
// bf16 weights ("MoE Expert Quantization", Axolotl docs, Expert LoRA
// targeting: experts that are trained rather than frozen and packed):
//
//   g | u  = gate_up[e] x[p]            h = silu(g) u         out = down[e] h
//   dh     = down[e]^T dout[p]          s = 1 / (1 + exp(-g))
//   dg     = dh u s (1 + g (1 - s))     du = dh g s
//
// Two kernels here carry the activation in the epilogue of a product: the
// gate_up product stores h (and, for training, g and u in fp32), the down
// product's input gradient stores dg | du and h again.  The other products of
// the block are those of grouped.hip on what these store.  A tile of the
// gate_up product holds the same columns of the gate and of the up projection,
// 32 of each in turn, so that a wave has g and u of a value in the same lane.
//
// Roundings: g, u and dh are fp32 sums, and g and u are kept so for the backward
// pass (in bf16, half the bytes, their rounding would be as large again as the
// gradients' own: 3.5e-3 of grad_down instead of 2.4e-3).  h, dg and du are
// rounded to bf16, because the next product's matrix instructions take bf16.
//
// Measured (median us of a kernel): 16384 rows, E = 8, H = 4096, I = 14336:
// gate_up with silu(g) u 3340 (1.15 PFLOP/s, matrix cores 70 % busy at the 1.59
// GHz that the card's power leaves), down 1690.  32768 rows, E = 64, H = 2048,
// I = 1024, for training: gate_up 320 (0.86 PFLOP/s, 47 % busy at 2.0 GHz; 8 to
// 32 steps of contraction a tile, whose first copies and stores nothing covers),
// down's input gradient 230 (its epilogue reads and writes 580 MB), the rest of
// the backward pass 270 + 170 + 280.  One token over 64 experts: 100 MB of weights in
// 21 us, 4.6 TB/s.
#include "grouped_tile.h"

#include "ffn.h"

namespace moeq {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ float sigmoid(float g) { return __builtin_amdgcn_rcpf(1.0f + __expf(-g)); }
// (u last: g u may leave fp32's range where silu(g) u does not)
__device__ __forceinline__ float glu(float g, float u) { return g * sigmoid(g) * u; }

// gate_up product of a tile: rows row0 .. + nrows, columns c0 .. of h.
template <int kNWN, int kNWM, int kTM, int kBufsA, int kBufsB>
struct GluTile {
  using T = Tile<Op::kBf16, false, false, kNWN, kNWM, 2, kTM, kBufsA, kBufsB, true>;
  static constexpr int kCols = T::kCols / 2;
  // 32 rows of 32 columns of h in bf16, and of g and u in fp32
  static constexpr int kPitch = 64 + 16, kWide = 128 + 16, kPiece = 32 * (kPitch + 2 * kWide);
  static constexpr int kLds = imax(T::kLds, T::kNW * kPiece);

  __device__ __forceinline__ static void run(char* smem, const GroupedArgs& g, float* gu, int e, int row0, int nrows,
                                             int c0) {
    const int t = threadIdx.x, lane = t & 63, wave = __builtin_amdgcn_readfirstlane(t >> 6);
    const int kbytes = 2 * g.kc, I = g.nout;
    typename T::A a;
    typename T::B b;
    // (rows past the gate's last are the up projection's first: their columns are not stored)
    a.init_pair(static_cast<const char*>(g.w) + ((int64_t)e * 2 * I + c0) * kbytes, (int64_t)(2 * I - c0) * kbytes, kbytes,
                kbytes, I, wave, lane);
    b.init(static_cast<const char*>(g.x) + (int64_t)row0 * kbytes, (int64_t)nrows * kbytes, kbytes, kbytes, wave, lane);
    f32x16 acc[2][kTM];
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int m = 0; m < kTM; ++m) acc[n][m] = (f32x16){};
    T::run(smem, a, b, nullptr, 0, (kbytes + kStepBytes - 1) / kStepBytes, acc);

    const int wn = wave % kNWN, wm = wave / kNWN, l32 = lane & 31, h = lane >> 5;
    char* buf = smem + wave * kPiece;
    const int c = c0 + 32 * wn + 8 * (lane & 3);
    char* wide = buf + 32 * kPitch;
    const int cw = c0 + 32 * wn + 4 * (lane & 7);
#pragma unroll
    for (int m = 0; m < kTM; ++m) {
      const int r0 = 32 * (kTM * wm + m);
      if (r0 >= nrows) break;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        float gv[4], uv[4], hv[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          gv[i] = acc[0][m][4 * q + i];
          uv[i] = acc[1][m][4 * q + i];
          hv[i] = glu(gv[i], uv[i]);
        }
        *reinterpret_cast<uint2*>(buf + l32 * kPitch + 2 * (8 * q + 4 * h)) =
            make_uint2(pack_bf16x2(hv[0], hv[1]), pack_bf16x2(hv[2], hv[3]));
        if (gu) {
          char* p = wide + l32 * kWide + 4 * (8 * q + 4 * h);
          *reinterpret_cast<float4*>(p) = make_float4(gv[0], gv[1], gv[2], gv[3]);
          *reinterpret_cast<float4*>(p + 32 * kWide) = make_float4(uv[0], uv[1], uv[2], uv[3]);
        }
      }
      // (a wave's LDS accesses are done in order)
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront", "local");
      __builtin_amdgcn_wave_barrier();
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int r = 16 * k + lane / 4;
        if (r0 + r < nrows && c < I)
          __builtin_nontemporal_store(
              *reinterpret_cast<const u32x4*>(buf + r * kPitch + 16 * (lane & 3)),
              reinterpret_cast<u32x4*>(static_cast<uint16_t*>(g.out) + (int64_t)(row0 + r0 + r) * I + c));
      }
      if (gu)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int r = 8 * k + lane / 8;
          if (r0 + r < nrows && cw < I) {
            float* to = gu + (int64_t)(row0 + r0 + r) * 2 * I + cw;
            const char* from = wide + r * kWide + 16 * (lane & 7);
            __builtin_nontemporal_store(*reinterpret_cast<const u32x4*>(from), reinterpret_cast<u32x4*>(to));
            __builtin_nontemporal_store(*reinterpret_cast<const u32x4*>(from + 32 * kWide), reinterpret_cast<u32x4*>(to + I));
          }
        }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront", "local");
      __builtin_amdgcn_wave_barrier();
    }
  }
};

template <int kNWN, int kNWM, int kTM, int kBufsA, int kBufsB>
__global__ __launch_bounds__(64 * kNWN * kNWM, kNWN * kNWM / 4) void glu_kernel(GroupedArgs g, float* gu) {
  using Big = GluTile<kNWN, kNWM, kTM, kBufsA, kBufsB>;
  __shared__ __attribute__((aligned(16))) char smem[Big::kLds];
  int e, row0, nrows, ct;
  if (!find_tile(g, Big::T::kRows, (g.nout + Big::kCols - 1) / Big::kCols, e, row0, nrows, ct)) return;
  const int c0 = ct * Big::kCols;
  // blocks of 32 rows per wave: as few as the tile's rows need
  if constexpr (kTM > 3)
    if (nrows > 3 * 32 * kNWM) return GluTile<kNWN, kNWM, 4, kBufsA, kBufsB>::run(smem, g, gu, e, row0, nrows, c0);
  if constexpr (kTM > 2)
    if (nrows > 2 * 32 * kNWM) return GluTile<kNWN, kNWM, 3, kBufsA, kBufsB>::run(smem, g, gu, e, row0, nrows, c0);
  if constexpr (kTM > 1)
    if (nrows > 32 * kNWM) return GluTile<kNWN, kNWM, 2, kBufsA, kBufsB>::run(smem, g, gu, e, row0, nrows, c0);
  GluTile<kNWN, kNWM, 1, kBufsA, kBufsB>::run(smem, g, gu, e, row0, nrows, c0);
}

// dh of a tile, and from it and g | u: dg | du and h.
template <int kNWN, int kNWM, int kTN, int kTM, int kBufsA, int kBufsB>
__device__ __forceinline__ void glu_backward_tile(char* smem, const GroupedArgs& g, const float* gu, uint16_t* dgu, int e,
                                                  int row0, int nrows, int c0) {
  using T = Tile<Op::kBf16, true, false, kNWN, kNWM, kTN, kTM, kBufsA, kBufsB>;
  const int t = threadIdx.x, lane = t & 63, wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const int kbytes = 2 * g.kc, I = g.nout;
  const int64_t expert = (int64_t)g.kc * I * 2;
  typename T::A a;
  typename T::B b;
  a.init(static_cast<const char*>(g.w) + e * expert + 2 * c0, expert - 2 * c0, 2 * I, 0, wave, lane);
  b.init(static_cast<const char*>(g.x) + (int64_t)row0 * kbytes, (int64_t)nrows * kbytes, kbytes, kbytes, wave, lane);
  f32x16 acc[kTN][kTM];
#pragma unroll
  for (int n = 0; n < kTN; ++n)
#pragma unroll
    for (int m = 0; m < kTM; ++m) acc[n][m] = (f32x16){};
  T::run(smem, a, b, nullptr, 0, (kbytes + kStepBytes - 1) / kStepBytes, acc);

  struct Pair {
    float4 g[2], u[2];
  };
  gu += (int64_t)row0 * 2 * I + c0;
  dgu += (int64_t)row0 * 2 * I + c0;
  uint16_t* h = static_cast<uint16_t*>(g.out) + (int64_t)row0 * I + c0;
  T::each8(
      smem, acc, nrows, min(T::kCols, I - c0),
      [&](int r, int c) {
        const float4* p = reinterpret_cast<const float4*>(gu + (int64_t)r * 2 * I + c);
        const float4* q = reinterpret_cast<const float4*>(gu + (int64_t)r * 2 * I + I + c);
        return Pair{{p[0], p[1]}, {q[0], q[1]}};
      },
      [&](int r, int c, const float (&dh)[8], const Pair& in) {
        u32x4 dgv, duv, hv;
        const float gs[8] = {in.g[0].x, in.g[0].y, in.g[0].z, in.g[0].w, in.g[1].x, in.g[1].y, in.g[1].z, in.g[1].w};
        const float us[8] = {in.u[0].x, in.u[0].y, in.u[0].z, in.u[0].w, in.u[1].x, in.u[1].y, in.u[1].z, in.u[1].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float o[3][2];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float gv = gs[2 * i + j], uv = us[2 * i + j];
            const float s = sigmoid(gv), d = dh[2 * i + j];
            o[0][j] = d * (s * (1.0f + gv * (1.0f - s))) * uv;   // (u last, as in glu)
            o[1][j] = d * (gv * s);
            o[2][j] = gv * s * uv;
          }
          dgv[i] = pack_bf16x2(o[0][0], o[0][1]);
          duv[i] = pack_bf16x2(o[1][0], o[1][1]);
          hv[i] = pack_bf16x2(o[2][0], o[2][1]);
        }
        uint16_t* q = dgu + (int64_t)r * 2 * I + c;
        __builtin_nontemporal_store(dgv, reinterpret_cast<u32x4*>(q));
        __builtin_nontemporal_store(duv, reinterpret_cast<u32x4*>(q + I));
        __builtin_nontemporal_store(hv, reinterpret_cast<u32x4*>(h + (int64_t)r * I + c));
      });
}

template <int kNWN, int kNWM, int kTN, int kTM, int kBufsA, int kBufsB>
__global__ __launch_bounds__(64 * kNWN * kNWM, kNWN * kNWM / 4) void glu_backward_kernel(GroupedArgs g, const float* gu,
                                                                                       uint16_t* dgu) {
  using Big = Tile<Op::kBf16, true, false, kNWN, kNWM, kTN, kTM, kBufsA, kBufsB>;
  __shared__ __attribute__((aligned(16))) char smem[imax(Big::kLds, Big::out_bytes(4))];
  int e, row0, nrows, ct;
  if (!find_tile(g, Big::kRows, (g.nout + Big::kCols - 1) / Big::kCols, e, row0, nrows, ct)) return;
  const int c0 = ct * Big::kCols;
  if constexpr (kTM > 3)
    if (nrows > 3 * 32 * kNWM)
      return glu_backward_tile<kNWN, kNWM, kTN, 4, kBufsA, kBufsB>(smem, g, gu, dgu, e, row0, nrows, c0);
  if constexpr (kTM > 2)
    if (nrows > 2 * 32 * kNWM)
      return glu_backward_tile<kNWN, kNWM, kTN, 3, kBufsA, kBufsB>(smem, g, gu, dgu, e, row0, nrows, c0);
  if constexpr (kTM > 1)
    if (nrows > 32 * kNWM)
      return glu_backward_tile<kNWN, kNWM, kTN, 2, kBufsA, kBufsB>(smem, g, gu, dgu, e, row0, nrows, c0);
  glu_backward_tile<kNWN, kNWM, kTN, 1, kBufsA, kBufsB>(smem, g, gu, dgu, e, row0, nrows, c0);
}

// Few rows per expert (decode): gate and up columns stream past at most 16 rows
// straight into the matrix instructions' operands, as in the other products'
// form: 16 columns of h a work item, a unit of 256 B of their two weight rows
// and of the token rows at a time, one unit ahead.
constexpr int kUnitBytes = 256, kFewWaves = 4;

template <bool kSplit>
__global__ __launch_bounds__(64 * kFewWaves) void glu_few_rows_kernel(GroupedArgs g, float* gu) {
  constexpr int kCols = kSplit ? 16 : 16 * kFewWaves;   // of a workgroup
  __shared__ __attribute__((aligned(16))) f32x4 part[kSplit ? kFewWaves : 1][2][64];
  int e, row0, nrows, ct;
  if (!find_tile(g, 16, (g.nout + kCols - 1) / kCols, e, row0, nrows, ct)) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l16 = lane & 15, grp = lane >> 4, kbytes = 2 * g.kc, I = g.nout;
  const int c0 = ct * kCols + (kSplit ? 0 : 16 * wave), ncols = min(16, I - c0);
  if (!kSplit && ncols <= 0) return;   // (no barrier there)
  const __amdgpu_buffer_rsrc_t rx = buffer(static_cast<const char*>(g.x) + (int64_t)row0 * kbytes, (int64_t)nrows * kbytes);
  const char* w = static_cast<const char*>(g.w) + ((int64_t)e * 2 * I + c0) * kbytes;
  const __amdgpu_buffer_rsrc_t rw[2] = {buffer(w, (int64_t)ncols * kbytes),
                                        buffer(w + (int64_t)I * kbytes, (int64_t)ncols * kbytes)};
  struct Unit {
    u32x4 w[2][4], x[4];
  };
  // unit u (what is out of range loads zeros)
  auto load = [&](Unit& v, int u) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int at = u * kUnitBytes + 64 * j + 16 * grp;
      const uint32_t off = at < kbytes ? (uint32_t)l16 * (uint32_t)kbytes + (uint32_t)at : kPast;
      v.w[0][j] = buffer_load16(rw[0], off);
      v.w[1][j] = buffer_load16(rw[1], off);
      v.x[j] = buffer_load16(rx, off);
    }
  };
  f32x4 acc[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
  auto use = [&](const Unit& v) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int k = 0; k < 2; ++k)
        acc[k] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, v.w[k][j]),
                                                         __builtin_bit_cast(bf16x8, v.x[j]), acc[k], 0, 0, 0);
    mfma_done(acc[0]);
    mfma_done(acc[1]);
  };
  const int units = (kbytes + kUnitBytes - 1) / kUnitBytes;
  constexpr int kStep = kSplit ? kFewWaves : 1;
  Unit va, vb;
  int u = kSplit ? wave : 0;
  if (u < units) load(va, u);
  while (u < units) {
    if (u + kStep < units) load(vb, u + kStep);
    use(va);
    u += kStep;
    if (u >= units) break;
    if (u + kStep < units) load(va, u + kStep);
    use(vb);
    u += kStep;
  }
  if constexpr (kSplit) {
    part[wave][0][lane] = acc[0];
    part[wave][1][lane] = acc[1];
    __syncthreads();
    if (wave) return;
#pragma unroll
    for (int v = 1; v < kFewWaves; ++v)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const f32x4 q = part[v][k][lane];
        acc[k].x += q.x; acc[k].y += q.y; acc[k].z += q.z; acc[k].w += q.w;
      }
  }
  // the lane holds columns 4 (lane / 16) .. +3 of row lane % 16
  if (l16 < nrows && 4 * grp < ncols) {
    const int64_t p = row0 + l16;
    const int c = c0 + 4 * grp;
    const f32x4 a = acc[0], b = acc[1];
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(g.out) + p * I + c) =
        make_uint2(pack_bf16x2(glu(a.x, b.x), glu(a.y, b.y)), pack_bf16x2(glu(a.z, b.z), glu(a.w, b.w)));
    if (gu) {
      *reinterpret_cast<f32x4*>(gu + p * 2 * I + c) = a;
      *reinterpret_cast<f32x4*>(gu + p * 2 * I + I + c) = b;
    }
  }
}

hipError_t launch_glu_few_rows(const GroupedArgs& g, float* gu, hipStream_t s) {
  const int64_t tiles = (g.nout + 15) / 16, slots = (int64_t)g.M / 16 + std::min(g.E, g.M);
  const int64_t units = (2 * (int64_t)g.kc + kUnitBytes - 1) / kUnitBytes;
  if (units >= 2 * kFewWaves || slots * tiles < 4096)
    glu_few_rows_kernel<true><<<(unsigned)items_grid(slots * tiles), 64 * kFewWaves, 0, s>>>(g, gu);
  else
    glu_few_rows_kernel<false>
        <<<(unsigned)items_grid(slots * ((tiles + kFewWaves - 1) / kFewWaves)), 64 * kFewWaves, 0, s>>>(g, gu);
  return hipGetLastError();
}

// Whether the weights stream past the rows.  us of the whole block here and in
// tiles, the same number of rows for each expert, other weights from call to call (a
// GB and more):
//   rows an expert                       1         8        16        24
//     E = 64, H = 2048, I = 1024   151, 179  166, 191  156, 177  223, 179
//     E = 8, H = I = 4096          157, 177  161, 184  169, 190  226, 191
//     E = 32, H = I = 2880         263, 267  283, 283  299, 283  426, 284
//     E = 128, H = 2048, I = 768   208, 234  226, 251  230, 246  325, 249
// so up to 16 rows, which are one pass over the weights.  Where the rows lie the
// host does not know.  At 8 rows an expert on average, even, by Zipf's law (exponent
// 1.1) and all in one expert, whose weights then pass many times:
//     E = 64, H = 2048, I = 1024   166, 191  178, 189   92,  82
//     E = 8, H = I = 4096          162, 185  167, 191   80,  66
//     E = 32, H = I = 2880         283, 283  332, 315  158, 117
//     E = 128, H = 2048, I = 768   220, 246  249, 266  123,  90
// At 4 on average the stream is ahead by Zipf's law everywhere, and behind for one
// expert's 32 rows of H = I = 2880 and more (86, 67).
// A grid holds less than 2^32 threads; beyond that the tiles serve.
bool streams(const GroupedArgs& g) {
  const int64_t items = ((int64_t)g.M / 16 + std::min(g.E, g.M)) * ((g.nout + 15) / 16);
  return g.M <= 8 * (int64_t)g.E && items_grid(items) * 64 * kFewWaves < (int64_t(1) << 32);
}

// Whether tiles of `cols` columns (128 of h, 256 of dh) leave compute units without
// work: those of half the columns then do better.  us of the whole block, then of the
// whole backward pass, in small and in large tiles, with the number of large ones:
//   E = 1, 512 rows, H = 2048, I = 1024       16: 47, 61       8: 94, 110
//   E = 8, 64 rows each, H = 2048, I = 1024   64: 38, 45      32: 83, 92
//   E = 8, 512 each, H = 2048, I = 1024      128: 64, 76      64: 158, 173
//   E = 4, 100 each, H = I = 4096            128: 110, 118    64: 267, 282
//   E = 64, 64 each, H = 2048, I = 256       128: 58, 61      64: 126, 134
//   E = 8, 256 each, H = I = 4096            256: 232, 219   128: 582, 593
//   E = 16, 64 each, H = I = 2048            256: 104, 108   128: 204, 212
//   E = 64, 256 each, H = 2048, I = 512      256: 143, 136   128: 372, 367
//   E = 64, 64 each, H = 2048, I = 1024      512: 186, 186   256: 391, 385
bool few_tiles(const GroupedArgs& g, int32_t cols) {
  const int64_t experts = std::min(g.E, g.M), rows = std::max<int64_t>(1, (g.M / experts + 255) / 256) * experts;
  return rows * ((g.nout + cols - 1) / cols) <= 128;
}

template <int kNWN, int kNWM, int kTM, int kBufsA, int kBufsB>
hipError_t launch_glu_tiles(const GroupedArgs& g, float* gu, hipStream_t s) {
  using Big = GluTile<kNWN, kNWM, kTM, kBufsA, kBufsB>;
  const int64_t ncol = (g.nout + Big::kCols - 1) / Big::kCols;
  const int64_t grid = items_grid(((int64_t)g.M / Big::T::kRows + std::min(g.E, g.M)) * ncol);
  glu_kernel<kNWN, kNWM, kTM, kBufsA, kBufsB><<<(unsigned)grid, 64 * kNWN * kNWM, 0, s>>>(g, gu);
  return hipGetLastError();
}

template <int kNWN, int kNWM, int kTN, int kTM, int kBufsA, int kBufsB>
hipError_t launch_backward_tiles(const GroupedArgs& g, const float* gu, uint16_t* dgu, hipStream_t s) {
  using Big = Tile<Op::kBf16, true, false, kNWN, kNWM, kTN, kTM, kBufsA, kBufsB>;
  const int64_t ncol = (g.nout + Big::kCols - 1) / Big::kCols;
  const int64_t grid = items_grid(((int64_t)g.M / Big::kRows + std::min(g.E, g.M)) * ncol);
  glu_backward_kernel<kNWN, kNWM, kTN, kTM, kBufsA, kBufsB><<<(unsigned)grid, 64 * kNWN * kNWM, 0, s>>>(g, gu, dgu);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_glu(const GroupedArgs& g, float* gu, hipStream_t s) {
  if (streams(g)) return launch_glu_few_rows(g, gu, s);
  if (few_tiles(g, 128)) return launch_glu_tiles<2, 4, 2, 3, 3>(g, gu, s);
  return launch_glu_tiles<4, 2, 4, 3, 2>(g, gu, s);
}

hipError_t launch_glu_backward(const GroupedArgs& g, const float* gu, uint16_t* dgu, hipStream_t s) {
  if (few_tiles(g, 256)) return launch_backward_tiles<4, 2, 1, 4, 3, 3>(g, gu, dgu, s);
  return launch_backward_tiles<4, 2, 2, 4, 3, 2>(g, gu, dgu, s);
}

}  // namespace moeq
