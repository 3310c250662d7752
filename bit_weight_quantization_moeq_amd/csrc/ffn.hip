// The gated feed-forward block of experts over rows sorted by expert (gfx950),
// bf16 weights ("MoE Expert Quantization", Axolotl docs, Expert LoRA
// targeting: experts that are trained rather than frozen and packed):
//
//   g | u  = gate_up[e] x[p]            h = silu(g) u         out = down[e] h
//   dh     = down[e]^T dout[p]          s = 1 / (1 + exp(-g))
//   dg     = dh u s (1 + g (1 - s))     du = dh g s
//
// Two kernels here carry the activation in the epilogue of a product: the
// gate_up product stores h (and, for training, g and u in bf16), the down
// product's input gradient stores dg | du and h again.  The other products of
// the block are those of grouped.hip on what these store.  A tile of the
// gate_up product holds the same columns of the gate and of the up projection,
// 32 of each in turn, so that a wave has g and u of a value in the same lane.
//
// Roundings: g, u and dh are fp32 sums.  h, dg and du are rounded to bf16
// because the next product's matrix instructions take bf16; g and u are kept
// in bf16 for the backward pass, which doubles the rounding of h, dg and du
// (2^-9 relative each) and halves what training has to hold and move.
#include "grouped_tile.h"

#include "ffn.h"

namespace moeq {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ float sigmoid(float g) { return __builtin_amdgcn_rcpf(1.0f + __expf(-g)); }
__device__ __forceinline__ float glu(float g, float u) { return g * u * sigmoid(g); }

// gate_up product of a tile: rows row0 .. + nrows, columns c0 .. of h.
template <int kNWN, int kNWM, int kTM, int kBufsA, int kBufsB>
struct GluTile {
  using T = Tile<Op::kBf16, false, false, kNWN, kNWM, 2, kTM, kBufsA, kBufsB, true>;
  static constexpr int kCols = T::kCols / 2;
  static constexpr int kPitch = 64 + 16, kPiece = 3 * 32 * kPitch;   // 32 rows of 32 columns of h, g and u
  static constexpr int kLds = imax(T::kLds, T::kNW * kPiece);

  __device__ __forceinline__ static void run(char* smem, const GroupedArgs& g, uint16_t* gu, int e, int row0, int nrows,
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
    auto put = [&](int plane, int q, const float (&v)[4]) {
      *reinterpret_cast<uint2*>(buf + (32 * plane + l32) * kPitch + 2 * (8 * q + 4 * h)) =
          make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
    };
    auto get = [&](int plane, int r) {
      return *reinterpret_cast<const u32x4*>(buf + (32 * plane + r) * kPitch + 16 * (lane & 3));
    };
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
        put(0, q, hv);
        if (gu) {
          put(1, q, gv);
          put(2, q, uv);
        }
      }
      // (a wave's LDS accesses are done in order)
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront", "local");
      __builtin_amdgcn_wave_barrier();
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int r = 16 * k + lane / 4;
        if (r0 + r < nrows && c < I) {
          const int64_t p = row0 + r0 + r;
          __builtin_nontemporal_store(get(0, r), reinterpret_cast<u32x4*>(static_cast<uint16_t*>(g.out) + p * I + c));
          if (gu) {
            __builtin_nontemporal_store(get(1, r), reinterpret_cast<u32x4*>(gu + p * 2 * I + c));
            __builtin_nontemporal_store(get(2, r), reinterpret_cast<u32x4*>(gu + p * 2 * I + I + c));
          }
        }
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront", "local");
      __builtin_amdgcn_wave_barrier();
    }
  }
};

template <int kNWN, int kNWM, int kTM, int kBufsA, int kBufsB>
__global__ __launch_bounds__(64 * kNWN * kNWM, kNWN * kNWM / 4) void glu_kernel(GroupedArgs g, uint16_t* gu) {
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
__device__ __forceinline__ void glu_backward_tile(char* smem, const GroupedArgs& g, const uint16_t* gu, uint16_t* dgu, int e,
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
    u32x4 g, u;
  };
  gu += (int64_t)row0 * 2 * I + c0;
  dgu += (int64_t)row0 * 2 * I + c0;
  uint16_t* h = static_cast<uint16_t*>(g.out) + (int64_t)row0 * I + c0;
  T::each8(
      smem, acc, nrows, min(T::kCols, I - c0),
      [&](int r, int c) {
        const uint16_t* p = gu + (int64_t)r * 2 * I + c;
        return Pair{*reinterpret_cast<const u32x4*>(p), *reinterpret_cast<const u32x4*>(p + I)};
      },
      [&](int r, int c, const float (&dh)[8], const Pair& in) {
        u32x4 dgv, duv, hv;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float o[3][2];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float gv = __builtin_bit_cast(float, j ? in.g[i] & 0xffff0000u : in.g[i] << 16);
            const float uv = __builtin_bit_cast(float, j ? in.u[i] & 0xffff0000u : in.u[i] << 16);
            const float s = sigmoid(gv), d = dh[2 * i + j];
            o[0][j] = d * uv * (s * (1.0f + gv * (1.0f - s)));
            o[1][j] = d * (gv * s);
            o[2][j] = gv * uv * s;
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
__global__ __launch_bounds__(64 * kNWN * kNWM, kNWN * kNWM / 4) void glu_backward_kernel(GroupedArgs g, const uint16_t* gu,
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

template <int kNWN, int kNWM, int kTM, int kBufsA, int kBufsB>
hipError_t launch_glu_tiles(const GroupedArgs& g, uint16_t* gu, hipStream_t s) {
  using Big = GluTile<kNWN, kNWM, kTM, kBufsA, kBufsB>;
  const int64_t ncol = (g.nout + Big::kCols - 1) / Big::kCols;
  const int64_t grid = items_grid(((int64_t)g.M / Big::T::kRows + std::min(g.E, g.M)) * ncol);
  glu_kernel<kNWN, kNWM, kTM, kBufsA, kBufsB><<<(unsigned)grid, 64 * kNWN * kNWM, 0, s>>>(g, gu);
  return hipGetLastError();
}

template <int kNWN, int kNWM, int kTN, int kTM, int kBufsA, int kBufsB>
hipError_t launch_backward_tiles(const GroupedArgs& g, const uint16_t* gu, uint16_t* dgu, hipStream_t s) {
  using Big = Tile<Op::kBf16, true, false, kNWN, kNWM, kTN, kTM, kBufsA, kBufsB>;
  const int64_t ncol = (g.nout + Big::kCols - 1) / Big::kCols;
  const int64_t grid = items_grid(((int64_t)g.M / Big::kRows + std::min(g.E, g.M)) * ncol);
  glu_backward_kernel<kNWN, kNWM, kTN, kTM, kBufsA, kBufsB><<<(unsigned)grid, 64 * kNWN * kNWM, 0, s>>>(g, gu, dgu);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_glu(const GroupedArgs& g, uint16_t* gu, hipStream_t s) {
  return launch_glu_tiles<4, 2, 4, 3, 2>(g, gu, s);
}

hipError_t launch_glu_backward(const GroupedArgs& g, const uint16_t* gu, uint16_t* dgu, hipStream_t s) {
  return launch_backward_tiles<4, 2, 2, 4, 3, 2>(g, gu, dgu, s);
}

}  // namespace moeq
