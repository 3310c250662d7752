// The tile engine of the products grouped by expert: an output tile's operands
// staged through LDS by DMA, the matrix instructions over them, and the tile's
// way back to memory; the experts' row ranges and the order of the tiles.
#pragma once

#include <algorithm>
#include <type_traits>

#include "grouped.h"

namespace moeq {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef short v4i16 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) v4i16 lds_v4i16;

constexpr int kXcds = 8;
constexpr int kStepBytes = 128;  // contraction bytes of a row per step
constexpr int kSub = 4;          // MFMA steps per step
constexpr int kTileGroup = 4;    // row tiles that run side by side over the column tiles
constexpr uint32_t kPast = 0x80000000u;  // a buffer offset past every resource's end

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  const f32x2 v = {lo, hi};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));
}

struct PackBf16 {
  __device__ __forceinline__ uint32_t operator()(float lo, float hi) const { return pack_bf16x2(lo, hi); }
};

// s_waitcnt immediate: at most N vector-memory loads outstanding and every LDS
// access of this wave done (gfx9 encoding: vmcnt in bits 3:0 and 15:14, expcnt
// 6:4, lgkmcnt 11:8).
template <int N>
constexpr int kWaitLoads = (N & 0xF) | ((N >> 4) << 14) | (0x7 << 4);

// Resource of `bytes` bytes at p (none if negative).
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer(const char* p, int64_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(p), 0, bytes > 0 ? (int)bytes : 0, 0x00020000);
}
// 16 bytes per lane at byte off, zeros past the resource's end: into registers,
__device__ __forceinline__ u32x4 buffer_load16(__amdgpu_buffer_rsrc_t r, uint32_t off) {
  return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, (int)off, 0, 0));
}
// or into LDS at lds + 16 * lane.  The address is a bare number: with a
// pointer to the array the compiler would make later LDS reads wait for all
// copies in flight; the waits before the barriers order them instead.  For
// ds_read_b64_tr_b16 the compiler waits all the same, so the bf16 kernels
// copy through inline assembly (with no register output), which it does not
// look into; the MXFP4 kernel has loads of its own between the copies, whose
// waits it counts right only if it sees both.  The DMA reads M0 one wait state
// after its write.
template <bool kSeen>
__device__ __forceinline__ void dma16(const char* p, int64_t bytes, uint32_t off, uint32_t lds) {
  if constexpr (kSeen) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(buffer(p, bytes), (__attribute__((address_space(3))) void*)(size_t)lds, 16,
                                             (int)off, 0, 0, 0);
  } else {
    const uint64_t a = (uint64_t)p;
    const u32x4 r = {(uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)a),
                     (uint32_t)__builtin_amdgcn_readfirstlane((int)((uint32_t)(a >> 32) & 0xffffu)),
                     (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)(bytes > 0 ? bytes : 0)), 0x00020000u};
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"s"(lds), "v"(off), "s"(r)
                 : "memory", "m0");
  }
}

// The wait states between an MFMA and the first other use of its result, by
// hand: where that use stands behind a branch, the compiler has been seen to
// leave them out (and the use to read the sums of two MFMAs before).
template <typename V>
__device__ __forceinline__ void mfma_done(V& acc) {
  asm volatile("s_nop 15\n\ts_nop 3" : "+v"(acc));
}

// What a tile multiplies: bf16, MXFP4 or fp16 values.
enum class Op { kBf16, kMxfp4, kF16 };

// One operand's side of a tile: kC rows (contraction-contiguous, !kT) or
// columns (output-contiguous, kT), staged by kNW waves.  kPair: rows of two
// matrices one behind the other, in turn, 32 of the first at 64 b of the tile
// and the same 32 of the second at 64 b + 32.
template <bool kT, int kC, int kNW, bool kPair = false>
struct Side {
  static constexpr int kBytes = kC * kStepBytes;
  static constexpr int kInstr = kC / 8 / kNW;      // DMA instructions per wave per step
  static constexpr int kLpr = kT ? kC / 8 : 8;     // lanes per LDS row
  static constexpr int kRpi = 64 / kLpr;           // LDS rows per instruction
  static constexpr int kPitch = kT ? 2 * kC : kStepBytes;
  static_assert(kC % (8 * kNW) == 0, "whole instructions per wave");
  static_assert(!kT || kC == 64 || kC == 128 || kC == 256, "transposed widths");
  static_assert(!kPair || (!kT && kRpi * kNW == 64), "an instruction's rows are 32 of each matrix");

  // slot swizzle of LDS row r (the same for every row a lane stages)
  __device__ __forceinline__ static int swz(int r) {
    if (!kT) return (r >> 1) & 7;   // 16 rows read at one chunk: 16 distinct 16-B banks of 256 B
    if (kC == 64) return ((r >> 1) & 1) << 2;
    return (r & 3) << 2;            // 4 rows of 64 B read together: 4 distinct quarters of 256 B
  }

  const char* base;   // !kT: the tile's first row; kT: the matrix's first row, at the tile's first column
  int64_t bytes;      // from base to the end of what may be read
  int32_t stride;     // bytes per row
  int32_t kbytes;     // !kT: contraction bytes of a row
  uint32_t voff;      // lane's offset of instruction 0
  int32_t chunk16;    // byte of the lane's chunk within its row

  __device__ __forceinline__ void init(const void* p, int64_t size, int32_t stride_, int32_t kbytes_, int wave, int lane) {
    base = static_cast<const char*>(p);
    bytes = size;
    stride = stride_;
    kbytes = kbytes_;
    const int r = kRpi * wave + lane / kLpr;
    chunk16 = 16 * ((lane % kLpr) ^ swz(r));
    voff = (uint32_t)r * (uint32_t)stride + (uint32_t)chunk16;
  }
  // kPair: the second matrix's first row is `second` rows behind the first's
  __device__ __forceinline__ void init_pair(const void* p, int64_t size, int32_t stride_, int32_t kbytes_, int32_t second,
                                            int wave, int lane) {
    init(p, size, stride_, kbytes_, wave, lane);
    if (wave >= kNW / 2) voff += (uint32_t)(second - 32) * (uint32_t)stride;
  }
  // instruction i of step ks into the LDS tile at lds
  template <bool kSeen>
  __device__ __forceinline__ void dma(int ks, int i, int wave, uint32_t lds) const {
    uint32_t off = voff + (uint32_t)(i * (kPair ? 32 : kRpi * kNW)) * (uint32_t)stride;
    const char* p = base;
    int64_t n = bytes;
    if constexpr (kT) {
      p += (int64_t)ks * 64 * stride;
      n = min(n - (int64_t)ks * 64 * stride, (int64_t)64 * stride);
    } else {
      off += (uint32_t)ks * kStepBytes;
      off = ks * kStepBytes + chunk16 < kbytes ? off : kPast;
    }
    dma16<kSeen>(p, n, off, lds + (uint32_t)(i * kNW + wave) * 1024u);
  }
  // Operand fragment of the 32 rows / columns from c0 on at MFMA step s:
  // lane (l32, h) gets contraction chunk 4 h + s (8 bf16, or one MXFP4 block).
  __device__ __forceinline__ static u32x4 frag(const char* tile, int c0, int s, int lane) {
    const int l32 = lane & 31, h = lane >> 5;
    if constexpr (!kT) {
      const int slot = (4 * h + s) ^ swz(l32);
      return *reinterpret_cast<const u32x4*>(tile + (c0 + l32) * kStepBytes + 16 * slot);
    } else {
      const int L = lane & 15, g = (lane >> 4) & 1;
      const int r = 8 * (4 * h + s) + (L >> 2);
      const int slot = (c0 / 8 + 2 * g + ((L & 3) >> 1)) ^ swz(L >> 2);
      const char* p = tile + r * kPitch + 16 * slot + 8 * (L & 1);
      const uint2 lo = __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4i16*)(p)));
      const uint2 hi = __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4i16*)(p + 4 * kPitch)));
      return u32x4{lo.x, lo.y, hi.x, hi.y};
    }
  }
};

// Scale bytes of an MXFP4 row, sixteen (those of two steps) at a time, zeros
// past its end.  The loads have no branch around them: past the row's last
// sixteen bytes those are read and shifted down, and a row that is not there
// (or shorter than sixteen blocks, whose only pair first() loads) reads zeros.
__device__ const uint64_t kNoScales[2] = {0, 0};
struct ScaleRow {
  typedef __attribute__((address_space(1))) const uint8_t* Ptr;   // global, so that no load is a flat one
  Ptr p;
  int32_t n, lim;   // scales of the row; the last offset to load from
  __device__ __forceinline__ void init(const uint8_t* row, int n_) {
    const bool in = row && n_ >= 16;
    p = (Ptr)(in ? row : reinterpret_cast<const uint8_t*>(kNoScales));
    n = n_;
    lim = in ? n_ - 16 : 0;
  }
  __device__ __forceinline__ u32x4 load(int pair) const {
    typedef u32x4 u32x4a __attribute__((aligned(1)));
    return *(__attribute__((address_space(1))) const u32x4a*)(p + min(16 * pair, lim));
  }
  // what load(pair) returned, in place
  __device__ __forceinline__ u32x4 use(u32x4 v, int pair) const {
    const int half = 4 * min(max(16 * pair + 16 - n, 0), 16);
    unsigned __int128 b = __builtin_bit_cast(unsigned __int128, v);
    b = (b >> half) >> half;
    return __builtin_bit_cast(u32x4, b);
  }
  __device__ __forceinline__ static u32x4 first(const uint8_t* row, int n) {
    uint64_t lo = 0, hi = 0;
    if (row) {
      for (int i = 0; i < min(n, 8); ++i) lo |= (uint64_t)row[i] << (8 * i);
      for (int i = 8; i < min(n, 16); ++i) hi |= (uint64_t)row[i] << (8 * (i - 8));
    }
    return u32x4{(uint32_t)lo, (uint32_t)(lo >> 32), (uint32_t)hi, (uint32_t)(hi >> 32)};
  }
};

// Shape of a tile: kNWN x kNWM waves, each kTN blocks of 32 columns by kTM
// blocks of 32 rows; kBufsA and kBufsB LDS buffers of the columns' and of the
// rows' operand.
template <Op kOp, bool kAT, bool kBT, int kNWN, int kNWM, int kTN, int kTM, int kBufsA, int kBufsB, bool kPairA = false>
struct Tile {
  static constexpr bool kMX = kOp == Op::kMxfp4;
  static constexpr int kNW = kNWN * kNWM;
  static constexpr int kCols = 32 * kTN * kNWN, kRows = 32 * kTM * kNWM;
  using A = Side<kAT, kCols, kNW, kPairA>;
  using B = Side<kBT, kRows, kNW>;
  static constexpr int kBytesB = kBufsA * A::kBytes;   // where the rows' buffers start
  static constexpr int kScaleBuf = kMX ? 16 * 64 * kNW : 0;   // every thread stores a row's
  static_assert(!kMX || kCols + kRows <= 64 * kNW, "a thread per scale row");
  static constexpr int kInstr = A::kInstr + B::kInstr;
  static constexpr int kScales = kBytesB + kBufsB * B::kBytes;   // and the scales'
  static constexpr int kLds = kScales + 2 * kScaleBuf;

  __device__ __forceinline__ static f32x16 mfma(u32x4 a, u32x4 b, f32x16 c) {
    if constexpr (kOp == Op::kF16)
      return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
    else
      return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0,
                                                     0);
  }

  // acc[n][m]: 32 columns x 32 rows each
  __device__ __forceinline__ static void run(char* smem, const A& a, const B& b, const uint8_t* scales, int nscale, int nks,
                                             f32x16 (&acc)[kTN][kTM]) {
    const int t = threadIdx.x, lane = t & 63;
    const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
    const int wn = wave % kNWN, wm = wave / kNWN;
    uint32_t lds0 = (uint32_t)(size_t)(__attribute__((address_space(3))) char*)smem;
    asm volatile("" : "+s"(lds0));  // opaque, so that it is not folded back into a pointer to the array
    char* sc = smem + kScales;   // MX: two buffers of two steps, each step kCols then kRows rows of 8 B
    constexpr int kScaleStep = kScaleBuf / 2;

    // instruction i of step ks's copies into ring slot `slot`
    auto dma_a = [&](int ks, int slot, int i) { a.template dma<kMX>(ks, i, wave, lds0 + (uint32_t)(slot * A::kBytes)); };
    auto dma_b = [&](int ks, int slot, int i) {
      b.template dma<kMX>(ks, i, wave, lds0 + (uint32_t)(kBytesB + slot * B::kBytes));
    };
    auto scale_store = [&](int pair, u32x4 v) {
      char* p = sc + (pair & 1) * kScaleBuf + 8 * t;
      *reinterpret_cast<uint2*>(p) = make_uint2(v.x, v.y);
      *reinterpret_cast<uint2*>(p + kScaleStep) = make_uint2(v.z, v.w);
    };
    // the MFMA order is column block by column block: operand j of kOps is
    // the j-th that it needs (a 0, the b's, the other a's)
    constexpr int kOps = kTN + kTM, kMfmas = kTN * kTM;
    auto frag = [&](const char* ta, const char* tb, int s, int j, u32x4 (&fa)[kTN], u32x4 (&fb)[kTM]) {
      if (j >= 1 && j <= kTM) {
        fb[j - 1] = B::frag(tb, 32 * (kTM * wm + j - 1), s, lane);
      } else {
        const int n = j == 0 ? 0 : j - kTM;
        fa[n] = A::frag(ta, 32 * (kTN * wn + n), s, lane);
      }
    };
    // the dwords of step ks: scales 4 h .. 4 h + 3 of the lane's rows
    auto load_scales = [&](int ks, uint32_t (&sa)[kTN], uint32_t (&sb)[kTM]) {
      const char* s0 = sc + (ks & 3) * kScaleStep + 8 * (lane & 31) + 4 * (lane >> 5);
#pragma unroll
      for (int n = 0; n < kTN; ++n) sa[n] = *reinterpret_cast<const uint32_t*>(s0 + 8 * 32 * (kTN * wn + n));
#pragma unroll
      for (int m = 0; m < kTM; ++m) sb[m] = *reinterpret_cast<const uint32_t*>(s0 + 8 * (kCols + 32 * (kTM * wm + m)));
    };
    // The step loop.  The barrier stands before the last MFMA step: by then
    // every wave holds that step's operands in registers, so that the LDS
    // buffer is free for a later step's copies, and the next step's first
    // operands are read during the last MFMAs, so that the matrix cores need
    // not wait at the turn of a step.  In step ks the columns' copies of step
    // ks + kBufsA - 1 are spread over the MFMAs before the barrier and the
    // rows' of step ks + kBufsB over those behind it, one at a time, as are
    // the operand reads: issued together, the copies hold the wave up at the
    // memory pipeline.  Loads complete in order, so the barrier's wait can
    // leave in flight whatever was issued after the next step's copies.
    constexpr int kInFlight = (kBufsA - 2) * A::kInstr + (kBufsB - 2) * B::kInstr;
    ScaleRow sr;
    u32x4 sv = {0u, 0u, 0u, 0u};   // scales on their way to LDS: the next pair of steps'
    uint32_t sa[2][kTN], sb[2][kTM];
    if constexpr (kMX) {
      sr.init(scales, nscale);
      scale_store(0, nscale < 16 ? ScaleRow::first(scales, nscale) : sr.use(sr.load(0), 0));
    }
    auto fill_a = [&](int p) {
#pragma unroll
      for (int i = 0; i < A::kInstr; ++i) dma_a(p, p, i);
    };
    auto fill_b = [&](int p) {
#pragma unroll
      for (int i = 0; i < B::kInstr; ++i) dma_b(p, p, i);
    };
    // in the order of the loop
#pragma unroll
    for (int p = 0; p < kBufsA || p < kBufsB; ++p) {
      if (kBufsA > kBufsB && p < kBufsA - 1) fill_a(p);
      if (p < kBufsB) fill_b(p);
      if (kBufsA <= kBufsB && p < kBufsA - 1) fill_a(p);
    }
    __builtin_amdgcn_s_waitcnt(kWaitLoads<kInFlight + B::kInstr>);
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
    u32x4 fa[2][kTN], fb[2][kTM];
#pragma unroll
    for (int j = 0; j < kOps; ++j) frag(smem, smem + kBytesB, 0, j, fa[0], fb[0]);
    if constexpr (kMX) load_scales(0, sa[0], sb[0]);

    int sa0 = 0, sb0 = 0;   // this step's ring slots
    auto step = [&](auto parity, int ks) {   // parity: ks & 1 (MXFP4 only)
      constexpr int kOdd = decltype(parity)::value;
      const int sa1 = sa0 + 1 == kBufsA ? 0 : sa0 + 1, sb1 = sb0 + 1 == kBufsB ? 0 : sb0 + 1;
      const int sap = sa0 == 0 ? kBufsA - 1 : sa0 - 1;
      if constexpr (kMX && !kOdd) sv = sr.load((ks >> 1) + 1);
#pragma unroll
      for (int s = 0; s < kSub; ++s) {
        if (s + 1 == kSub) {
          if constexpr (kMX && kOdd) scale_store((ks + 1) >> 1, sr.use(sv, (ks + 1) >> 1));
          __builtin_amdgcn_s_waitcnt(kWaitLoads<kInFlight>);
          __builtin_amdgcn_s_barrier();
          __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
          if constexpr (kMX) {
            load_scales(ks + 1, sa[kOdd ^ 1], sb[kOdd ^ 1]);
          }
        }
        const char* ta = smem + (s + 1 < kSub ? sa0 : sa1) * A::kBytes;
        const char* tb = smem + kBytesB + (s + 1 < kSub ? sb0 : sb1) * B::kBytes;
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int n = 0; n < kTN; ++n)
#pragma unroll
          for (int m = 0; m < kTM; ++m) {
            if constexpr (kMX) {
              const u32x4 x = fa[s & 1][n], y = fb[s & 1][m];
              const i32x8 xa = {(int)x.x, (int)x.y, (int)x.z, (int)x.w, 0, 0, 0, 0};
              const i32x8 yb = {(int)y.x, (int)y.y, (int)y.z, (int)y.w, 0, 0, 0, 0};
              // operand formats 4: E2M1; scale byte s of the lanes' dwords
              if (s == 0)
                acc[n][m] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
                    xa, yb, acc[n][m], 4, 4, 0, sa[kOdd][n], 0, sb[kOdd][m]);
              else if (s == 1)
                acc[n][m] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
                    xa, yb, acc[n][m], 4, 4, 1, sa[kOdd][n], 1, sb[kOdd][m]);
              else if (s == 2)
                acc[n][m] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
                    xa, yb, acc[n][m], 4, 4, 2, sa[kOdd][n], 2, sb[kOdd][m]);
              else
                acc[n][m] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
                    xa, yb, acc[n][m], 4, 4, 3, sa[kOdd][n], 3, sb[kOdd][m]);
            } else {
              acc[n][m] = mfma(fa[s & 1][n], fb[s & 1][m], acc[n][m]);
            }
            const int i = n * kTM + m;
#pragma unroll
            for (int j = i * kOps / kMfmas; j < (i + 1) * kOps / kMfmas; ++j)
              frag(ta, tb, (s + 1) % kSub, j, fa[(s + 1) & 1], fb[(s + 1) & 1]);
            // (past the last step everything is out of range)
            if (s + 1 < kSub) {
              constexpr int kSlots = (kSub - 1) * kMfmas;
#pragma unroll
              for (int d = 0; d < A::kInstr; ++d)
                if (s * kMfmas + i == d * kSlots / A::kInstr) dma_a(ks + kBufsA - 1, sap, d);
            } else {
#pragma unroll
              for (int d = 0; d < B::kInstr; ++d)
                if (i == d * kMfmas / B::kInstr) dma_b(ks + kBufsB, sb0, d);
            }
            __builtin_amdgcn_sched_barrier(0);
          }
      }
      sa0 = sa1;
      sb0 = sb1;
    };
    int ks = 0;
    if constexpr (kMX)
      for (; ks + 1 < nks; ks += 2) {
        step(std::integral_constant<int, 0>{}, ks);
        step(std::integral_constant<int, 1>{}, ks + 1);
      }
    for (; ks < nks; ++ks) step(std::integral_constant<int, 0>{}, ks);
    __builtin_amdgcn_s_waitcnt(0);   // copies of steps past the end
    __syncthreads();
    mfma_done(acc[kTN - 1][kTM - 1]);   // (the last one's; the barrier stands behind them all)
  }

  // The same for a contraction of one step at most (bf16, one buffer each):
  // the product moves its output and little else, so the tile is kept small
  // enough for four workgroups per compute unit, whose copies, products and
  // stores overlap.  E = 64, 512 rows each, N = 2048, inputs from HBM: K = 16
  // 29 us and 37 in the large tiles, K = 32 31 and 37, K = 64 43 and 41 (grad_input
  // alike); K = 72 and 128, which take more than one step, 47-49 in those.
  // Rank-16 grad_input over 128 experts 11-12 us, 27 in tiles of 128 rows.
  __device__ __forceinline__ static void run_short(char* smem, const A& a, const B& b, int kbytes, f32x16 (&acc)[kTN][kTM]) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wn = wave % kNWN, wm = wave / kNWN;
    uint32_t lds0 = (uint32_t)(size_t)(__attribute__((address_space(3))) char*)smem;
    asm volatile("" : "+s"(lds0));
#pragma unroll
    for (int i = 0; i < A::kInstr; ++i) a.template dma<false>(0, i, wave, lds0);
#pragma unroll
    for (int i = 0; i < B::kInstr; ++i) b.template dma<false>(0, i, wave, lds0 + (uint32_t)kBytesB);
    __builtin_amdgcn_s_waitcnt(0);
    __syncthreads();
    // MFMA step s covers chunks s and 4 + s: none behind the contraction's end
    const int steps = min(kSub, kbytes / 16);
    for (int s = 0; s < steps; ++s) {
      u32x4 fa[kTN], fb[kTM];
#pragma unroll
      for (int n = 0; n < kTN; ++n) fa[n] = A::frag(smem, 32 * (kTN * wn + n), s, lane);
#pragma unroll
      for (int m = 0; m < kTM; ++m) fb[m] = B::frag(smem + kBytesB, 32 * (kTM * wm + m), s, lane);
#pragma unroll
      for (int n = 0; n < kTN; ++n)
#pragma unroll
        for (int m = 0; m < kTM; ++m)
          acc[n][m] = mfma(fa[n], fb[m], acc[n][m]);
    }
    __syncthreads();
    mfma_done(acc[kTN - 1][kTM - 1]);
  }

  // Stores the tile: rows r < nrows, columns c < ncols (a multiple of 8) of
  // out, ld elements a row.  From the accumulator layout one instruction would
  // touch 32 rows, so every wave takes its blocks of 32 rows through a piece of
  // LDS of its own (two in turn, no barrier) and stores 64 to 256 B of a row
  // at a time, past the caches, which hold the operands.
  template <typename T>
  static constexpr int kOutPitch = 32 * kTN * (int)sizeof(T) + 16;
  static constexpr int kOutBufs = kTM > 1 ? 2 : 1;
  // Values of two bytes are made by pack, two at a time.
  template <typename T, typename Pack = PackBf16>
  __device__ __forceinline__ static void store(char* smem, const f32x16 (&acc)[kTN][kTM], T* out, int64_t ld, int nrows,
                                               int ncols, Pack pack = Pack()) {
    constexpr int kPer = 16 / (int)sizeof(T), kLanes = 32 * kTN / kPer;   // lanes per row
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wn = wave % kNWN, wm = wave / kNWN, l32 = lane & 31, h = lane >> 5;
    char* piece = smem + wave * (kOutBufs * 32 * kOutPitch<T>);
    const int c = 32 * kTN * wn + kPer * (lane % kLanes);
#pragma unroll
    for (int m = 0; m < kTM; ++m) {
      const int r0 = 32 * (kTM * wm + m);
      if (r0 >= nrows) break;
      char* buf = piece + (m & 1) * (32 * kOutPitch<T>);
#pragma unroll
      for (int n = 0; n < kTN; ++n)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          char* p = buf + l32 * kOutPitch<T> + (int)sizeof(T) * (32 * n + 8 * q + 4 * h);
          const f32x16& v = acc[n][m];
          if constexpr (sizeof(T) == 4)
            *reinterpret_cast<float4*>(p) = make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
          else
            *reinterpret_cast<uint2*>(p) =
                make_uint2(pack(v[4 * q], v[4 * q + 1]), pack(v[4 * q + 2], v[4 * q + 3]));
        }
      // (a wave's LDS accesses are done in order)
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront", "local");
      __builtin_amdgcn_wave_barrier();
#pragma unroll
      for (int u = 0; u < kLanes / 2; ++u) {
        const int r = u * (64 / kLanes) + lane / kLanes;
        const u32x4 v = *reinterpret_cast<const u32x4*>(buf + r * kOutPitch<T> + 16 * (lane % kLanes));
        if (r0 + r < nrows && c < ncols)
          __builtin_nontemporal_store(v, reinterpret_cast<u32x4*>(out + (int64_t)(r0 + r) * ld + c));
      }
    }
  }
  // Hands the tile over by rows, in fp32 and through the waves' pieces of LDS as
  // store does: use(r, c, v, read(r, c)) for columns c .. c + 7 of row r, r <
  // nrows and c < ncols.  The reads of 32 rows are under way before the first use.
  template <typename Read, typename Use>
  __device__ __forceinline__ static void each8(char* smem, const f32x16 (&acc)[kTN][kTM], int nrows, int ncols, Read read,
                                               Use use) {
    constexpr int kLanes = 4 * kTN, kRowsAt = 64 / kLanes, kTimes = 32 / kRowsAt, kPitch = kOutPitch<float>;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wn = wave % kNWN, wm = wave / kNWN, l32 = lane & 31, h = lane >> 5;
    char* piece = smem + wave * (kOutBufs * 32 * kPitch);
    const int lc = 8 * (lane % kLanes), c = 32 * kTN * wn + lc;
#pragma unroll
    for (int m = 0; m < kTM; ++m) {
      const int r0 = 32 * (kTM * wm + m);
      if (r0 >= nrows) break;
      char* buf = piece + (m & 1) * (32 * kPitch);
      decltype(read(0, 0)) in[kTimes];
#pragma unroll
      for (int u = 0; u < kTimes; ++u) {
        const int r = r0 + u * kRowsAt + lane / kLanes;
        if (r < nrows && c < ncols) in[u] = read(r, c);
      }
#pragma unroll
      for (int n = 0; n < kTN; ++n)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const f32x16& v = acc[n][m];
          *reinterpret_cast<float4*>(buf + l32 * kPitch + 4 * (32 * n + 8 * q + 4 * h)) =
              make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
        }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront", "local");
      __builtin_amdgcn_wave_barrier();
#pragma unroll
      for (int u = 0; u < kTimes; ++u) {
        const int lr = u * kRowsAt + lane / kLanes;
        const float4 lo = *reinterpret_cast<const float4*>(buf + lr * kPitch + 4 * lc);
        const float4 hi = *reinterpret_cast<const float4*>(buf + lr * kPitch + 4 * lc + 16);
        const float v[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
        if (r0 + lr < nrows && c < ncols) use(r0 + lr, c, v, in[u]);
      }
    }
  }
  static constexpr int out_bytes(int size) { return kNW * kOutBufs * 32 * (32 * kTN * size + 16); }
};

constexpr int imax(int a, int b) { return a > b ? a : b; }

template <int CTRL, int ROWS>
__device__ __forceinline__ int add_dpp(int v) {
  return v + __builtin_amdgcn_update_dpp(0, v, CTRL, ROWS, 0xF, false);
}
// Inclusive prefix sum over the wave, in six DPP additions.
__device__ __forceinline__ int wave_scan(int v) {
  v = add_dpp<0x111, 0xF>(v);   // row_shr:1, 2, 4, 8 within rows of 16 lanes
  v = add_dpp<0x112, 0xF>(v);
  v = add_dpp<0x114, 0xF>(v);
  v = add_dpp<0x118, 0xF>(v);
  v = add_dpp<0x142, 0xA>(v);   // row_bcast:15 into rows 1 and 3
  return add_dpp<0x143, 0xC>(v);  // row_bcast:31 into rows 2 and 3
}

// The experts' row ranges, 64 experts at a time, one per lane.  The first 256
// are loaded together (one memory latency for all that is needed of them);
// visit(f) calls f(first expert of the 64, lo, rows) in order until it returns
// true, and says whether it did.
struct ExpertRows {
  static constexpr int kKept = 4;
  const int32_t* offsets;
  int32_t E, M;
  int lo[kKept], n[kKept];
  __device__ __forceinline__ void rows(int i, int& l, int& c) const {   // none past the last expert
    const RowRange r = row_range(offsets[min(i, E)], offsets[min(i + 1, E)], M);
    l = r.lo;
    c = r.n;
  }
  __device__ __forceinline__ ExpertRows(const GroupedArgs& g) : offsets(g.offsets), E(g.E), M(g.M) {
#pragma unroll
    for (int c = 0; c < kKept; ++c) rows(64 * c + (threadIdx.x & 63), lo[c], n[c]);
  }
  template <typename F>
  __device__ __forceinline__ bool visit(F f) const {
#pragma unroll
    for (int c = 0; c < kKept; ++c)
      if (64 * c < E && f(64 * c, lo[c], n[c])) return true;
    for (int i = 64 * kKept; i < E; i += 64) {
      int l, c;
      rows(i + (threadIdx.x & 63), l, c);
      if (f(i, l, c)) return true;
    }
    return false;
  }
};

// Work item of this workgroup, of `total` in an order in which neighbours
// share operands (total if there is none for it).  Runs of up to `run` items
// go to the XCDs in turn, so that neighbours share an L2, but an expert with
// many rows does not leave its work to one XCD (contiguous eighths: rank-16
// grad_weight over Zipf-distributed experts 31 instead of 22 us, square
// products 3 % slower); at most total / 32, so that every XCD has several.
// Needs a grid of at least items_grid(total) workgroups.
__device__ __forceinline__ int work_item(int total, int run) {
  run = max(min(run, total / (4 * kXcds)), 1);
  const int slot = blockIdx.x / kXcds, q = slot / run;
  return min((q * kXcds + (int)(blockIdx.x % kXcds)) * run + slot - q * run, total);
}
int64_t items_grid(int64_t total) { return (total + total / 4 + 2 * kXcds - 1) / kXcds * kXcds; }

// The (expert, row tile, column tile) triples, expert-major.  An expert's rows
// are cut into ceil(rows / max_rows) tiles, whole ones and a rest where equal
// ones would be nearly whole (16384 ragged rows over 8 experts through the
// feed-forward block 4.81 ms in equal tiles, 4.72 so), otherwise equal ones (bf16
// products of 320 and 384 rows an expert 383 and 398 us, with whole tiles and a
// rest 400 and 432), taken in groups of kTileGroup that go through the column
// tiles together.  Each wave scans the
// experts by itself, 64 at a time.
__device__ __forceinline__ bool find_tile(const GroupedArgs& g, int max_rows, int ncol, int& e, int& row0, int& nrows,
                                          int& ct) {
  const ExpertRows x(g);
  int total = 0;
  x.visit([&](int, int, int n) {
    total += __builtin_amdgcn_readlane(wave_scan((n + max_rows - 1) / max_rows), 63);
    return false;
  });
  total *= ncol;
  const int w = work_item(total, kTileGroup * ncol);
  if (w >= total) return false;
  int before = 0;
  nrows = 0;
  x.visit([&](int i, int lo, int n) {
    const int nt = (n + max_rows - 1) / max_rows, incl = wave_scan(nt);
    const int first = before + incl - nt;
    const uint64_t hit = __ballot(w >= first * ncol && w < (first + nt) * ncol);
    before += __builtin_amdgcn_readlane(incl, 63);
    if (!hit) return false;
    const int src = __builtin_ctzll(hit);
    e = i + src;
    const int f = __builtin_amdgcn_readlane(first, src), k = __builtin_amdgcn_readlane(nt, src);
    const int r0 = __builtin_amdgcn_readlane(lo, src), c = __builtin_amdgcn_readlane(n, src);
    const int r = w - f * ncol, grp = r / (kTileGroup * ncol), gt = min(kTileGroup, k - grp * kTileGroup);
    const int rr = r - grp * kTileGroup * ncol;
    ct = rr / gt;
    const int mt = grp * kTileGroup + (rr - ct * gt);
    if (mt >= k) return true;   // (only offsets that do not ascend come here)
    int a = (int)((int64_t)mt * c / k), b = (int)((int64_t)(mt + 1) * c / k);
    if (4 * ((c + k - 1) / k) > 3 * max_rows) {   // equal tiles would cost as much as whole ones
      a = mt * max_rows;
      b = min(a + max_rows, c);
    }
    row0 = r0 + a;
    nrows = b - a;
    return true;
  });
  return nrows > 0;
}

}  // namespace
}  // namespace moeq
