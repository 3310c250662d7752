// Matrix products grouped by expert over rows sorted by expert (gfx950):
//
//   forward       y[p]  = w[e] x[p]                    bf16 or MXFP4 operands
//   grad_input    dx[p] = w[e]^T dy[p]                 bf16
//   grad_weight   dw[e] = sum over p of dy[p] x[p]^T   bf16 operands
//
// with offsets[e] <= p < offsets[e + 1] the rows of expert e (the layout that
// moeq_route_buckets and moeq_router_route produce; "MoE Expert
// Quantization", Axolotl docs, Expert LoRA targeting: adapters and trainable
// experts beside the frozen packed ones).
//
// One kernel body serves the three.  A workgroup owns an output tile: its
// columns are the MFMA A operand (so a lane ends up with four consecutive
// output columns of one row) and its rows the B operand.  Each contraction
// step takes 128 bytes of contraction of every tile row and column through
// LDS, in two or three buffers, copied by the LDS DMA of buffer_load ... lds:
//   * an operand that is contiguous along the contraction (x, w and dy of the
//     first two products) lies in LDS as rows of 128 B whose 16-B slots are
//     XOR-swizzled by the row, and is read with ds_read_b128;
//   * an operand that is contiguous along the output (w in grad_input, both
//     in grad_weight) lies in LDS as 64 contraction rows of the tile's
//     columns, and is read with ds_read_b64_tr_b16, which hands each lane of
//     16 one column of a 4 x 16 block.
// The buffer resource of a copy ends where the expert's data (or the tile's
// rows) end, and chunks past the contraction get an offset past that end, so
// everything out of range arrives in LDS as zeros: rows of the next expert,
// rows behind the last one and column tails can hold anything.
//
// MXFP4: a step of 128 B holds 256 values, eight blocks a row.  The order of
// the contraction is free as long as both operands agree: MFMA s of a step
// gives lane half h block 4 h + s of its row, which is 16 B (one LDS slot,
// as for bf16) and one scale byte, byte s of the dword of scales that the
// lane holds for the step.  v_mfma_scale_f32_32x32x64_f8f6f4 applies the
// scales of both operands in the product, with an fp32 sum.
//
// offsets are data on the device: row_range clamps them to [0, M], and no tile
// leaves the arrays whatever they hold.
//
// Measured, E = 8 with 4096 rows each, N = K = 4096, call after call: bf16 840-
// 860 us (1.28-1.31 PFLOP/s), MXFP4 285-325 us (3.4-3.9 PFLOP/s).  Single
// dispatches under the profiler's counters: bf16 938 us (1.17 PFLOP/s), the
// matrix cores 77 % busy at 1.46 GHz; MXFP4 306 us (3.6 PFLOP/s), 50 % busy at
// 1.71 GHz: a step's copies take two thirds of it, and a tile's first copies
// and its stores overlap with nothing.  256 x 256 tiles, because their operands
// are read from L2 least often, with LDS for one workgroup per compute unit.
#include <algorithm>
#include <type_traits>

#include "grouped.h"

namespace moeq {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
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

// One operand's side of a tile: kC rows (contraction-contiguous, !kT) or
// columns (output-contiguous, kT), staged by kNW waves.
template <bool kT, int kC, int kNW>
struct Side {
  static constexpr int kBytes = kC * kStepBytes;
  static constexpr int kInstr = kC / 8 / kNW;      // DMA instructions per wave per step
  static constexpr int kLpr = kT ? kC / 8 : 8;     // lanes per LDS row
  static constexpr int kRpi = 64 / kLpr;           // LDS rows per instruction
  static constexpr int kPitch = kT ? 2 * kC : kStepBytes;
  static_assert(kC % (8 * kNW) == 0, "whole instructions per wave");
  static_assert(!kT || kC == 64 || kC == 128 || kC == 256, "transposed widths");

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
  // instruction i of step ks into the LDS tile at lds
  template <bool kSeen>
  __device__ __forceinline__ void dma(int ks, int i, int wave, uint32_t lds) const {
    uint32_t off = voff + (uint32_t)(i * kRpi * kNW) * (uint32_t)stride;
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
template <bool kMX, bool kAT, bool kBT, int kNWN, int kNWM, int kTN, int kTM, int kBufsA, int kBufsB>
struct Tile {
  static constexpr int kNW = kNWN * kNWM;
  static constexpr int kCols = 32 * kTN * kNWN, kRows = 32 * kTM * kNWM;
  using A = Side<kAT, kCols, kNW>;
  using B = Side<kBT, kRows, kNW>;
  static constexpr int kBytesB = kBufsA * A::kBytes;   // where the rows' buffers start
  static constexpr int kScaleBuf = kMX ? 16 * 64 * kNW : 0;   // every thread stores a row's
  static_assert(!kMX || kCols + kRows <= 64 * kNW, "a thread per scale row");
  static constexpr int kInstr = A::kInstr + B::kInstr;
  static constexpr int kScales = kBytesB + kBufsB * B::kBytes;   // and the scales'
  static constexpr int kLds = kScales + 2 * kScaleBuf;

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
              acc[n][m] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, fa[s & 1][n]),
                                                                  __builtin_bit_cast(bf16x8, fb[s & 1][m]),
                                                                  acc[n][m], 0, 0, 0);
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
          acc[n][m] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, fa[n]),
                                                              __builtin_bit_cast(bf16x8, fb[m]), acc[n][m], 0, 0, 0);
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
  template <typename T>
  __device__ __forceinline__ static void store(char* smem, const f32x16 (&acc)[kTN][kTM], T* out, int64_t ld, int nrows,
                                               int ncols) {
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
                make_uint2(pack_bf16x2(v[4 * q], v[4 * q + 1]), pack_bf16x2(v[4 * q + 2], v[4 * q + 3]));
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
// are cut into ceil(rows / max_rows) near-equal tiles, taken in groups of
// kTileGroup that go through the column tiles together.  Each wave scans the
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
    const int a = (int)((int64_t)mt * c / k), b = (int)((int64_t)(mt + 1) * c / k);
    row0 = r0 + a;
    nrows = b - a;
    return true;
  });
  return nrows > 0;
}

// forward (kAT = false, kMX or not) and grad_input (kAT = true).
//   x [M][kc], w [E][..], out [M][nout]: kc contraction length, nout columns.
template <bool kMX, bool kAT, int kNWN, int kNWM, int kTN, int kTM, int kBufsA, int kBufsB>
__device__ __forceinline__ void rows_tile(char* smem, const GroupedArgs& g, int e, int row0, int nrows, int c0) {
  using T = Tile<kMX, kAT, false, kNWN, kNWM, kTN, kTM, kBufsA, kBufsB>;
  const int t = threadIdx.x, lane = t & 63, wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const int kbytes = kMX ? g.kc / 2 : 2 * g.kc;
  typename T::A a;
  typename T::B b;
  const char* w = static_cast<const char*>(g.w);
  const int ncols = min(T::kCols, g.nout - c0);
  if constexpr (kAT) {
    const int64_t expert = (int64_t)g.kc * g.nout * 2;
    a.init(w + e * expert + 2 * c0, expert - 2 * c0, 2 * g.nout, 0, wave, lane);
  } else {
    a.init(w + ((int64_t)e * g.nout + c0) * kbytes, (int64_t)ncols * kbytes, kbytes, kbytes, wave, lane);
  }
  b.init(static_cast<const char*>(g.x) + (int64_t)row0 * kbytes, (int64_t)nrows * kbytes, kbytes, kbytes, wave, lane);
  const int nscale = g.kc / 32;
  const uint8_t* scales = nullptr;   // of this thread's row of the tile: the columns, then the rows
  if constexpr (kMX) {
    if (t < T::kCols) {
      if (t < ncols) scales = g.w_scales + ((int64_t)e * g.nout + c0 + t) * nscale;
    } else if (t - T::kCols < nrows) {
      scales = g.x_scales + (int64_t)(row0 + t - T::kCols) * nscale;
    }
  }
  f32x16 acc[kTN][kTM];
#pragma unroll
  for (int n = 0; n < kTN; ++n)
#pragma unroll
    for (int m = 0; m < kTM; ++m) acc[n][m] = (f32x16){};
  if constexpr (kBufsA == 1)
    T::run_short(smem, a, b, kbytes, acc);
  else
    T::run(smem, a, b, scales, nscale, (kbytes + kStepBytes - 1) / kStepBytes, acc);
  T::store(smem, acc, static_cast<uint16_t*>(g.out) + (int64_t)row0 * g.nout + c0, g.nout, nrows, ncols);
}

template <bool kMX, bool kAT, int kNWN, int kNWM, int kTN, int kTM, int kBufsA, int kBufsB>
__global__ __launch_bounds__(64 * kNWN * kNWM, kBufsA == 1 ? 4 : kNWN * kNWM / 4) void rows_kernel(GroupedArgs g) {
  using Big = Tile<kMX, kAT, false, kNWN, kNWM, kTN, kTM, kBufsA, kBufsB>;
  __shared__ __attribute__((aligned(16))) char smem[imax(Big::kLds, Big::out_bytes(2))];
  int e, row0, nrows, ct;
  if (!find_tile(g, Big::kRows, (g.nout + Big::kCols - 1) / Big::kCols, e, row0, nrows, ct)) return;
  const int c0 = ct * Big::kCols;
  // blocks of 32 rows per wave: as few as the tile's rows need
  if constexpr (kTM > 3)
    if (nrows > 3 * 32 * kNWM) return rows_tile<kMX, kAT, kNWN, kNWM, kTN, 4, kBufsA, kBufsB>(smem, g, e, row0, nrows, c0);
  if constexpr (kTM > 2)
    if (nrows > 2 * 32 * kNWM) return rows_tile<kMX, kAT, kNWN, kNWM, kTN, 3, kBufsA, kBufsB>(smem, g, e, row0, nrows, c0);
  if constexpr (kTM > 1)
    if (nrows > 32 * kNWM) return rows_tile<kMX, kAT, kNWN, kNWM, kTN, 2, kBufsA, kBufsB>(smem, g, e, row0, nrows, c0);
  rows_tile<kMX, kAT, kNWN, kNWM, kTN, 1, kBufsA, kBufsB>(smem, g, e, row0, nrows, c0);
}

// grad_weight.  An expert's rows are cut into segments of g.segment rows (one
// at least, also for an expert without rows, whose result is zeros), so that a
// long expert is not one workgroup's chain of steps.  The only segment of an
// expert writes dw; several write fp32 partial sums, one [N][K] slot of the
// workspace each, which sum_segments_kernel adds in order.

// The (segment, tile) pairs, `tiles` a segment: the expert, its rows
// [lo, lo + n), tile r, segment k of the expert's nseg, and the slots before
// the expert's.  Experts of one segment have no slots.
struct Segment {
  int e, lo, n, r, k, nseg, slot;
};
__device__ __forceinline__ bool find_segment(const GroupedArgs& g, int tiles, Segment& o) {
  const ExpertRows x(g);
  const int lane = threadIdx.x & 63;
  auto segments = [&](int i, int n) { return i + lane < g.E ? max((n + g.segment - 1) / g.segment, 1) : 0; };
  int total = 0;
  x.visit([&](int i, int, int n) {
    total += __builtin_amdgcn_readlane(wave_scan(segments(i, n)), 63);
    return false;
  });
  total *= tiles;
  const int w = work_item(total, tiles);
  if (w >= total) return false;
  const int at = w / tiles;
  o.r = w - at * tiles;
  int before = 0, slots = 0;
  return x.visit([&](int i, int lo, int n) {
    const int ns = segments(i, n), sl = ns > 1 ? ns : 0;
    const int incl = wave_scan(ns), slot_incl = wave_scan(sl), first = before + incl - ns;
    const uint64_t hit = __ballot(at >= first && at < first + ns);
    if (hit) {
      const int src = __builtin_ctzll(hit);
      o.e = i + src;
      o.k = at - __builtin_amdgcn_readlane(first, src);
      o.nseg = __builtin_amdgcn_readlane(ns, src);
      o.slot = slots + __builtin_amdgcn_readlane(slot_incl - sl, src);
      o.lo = __builtin_amdgcn_readlane(lo, src) + o.k * g.segment;
      o.n = min(__builtin_amdgcn_readlane(n, src) - o.k * g.segment, g.segment);
      return true;
    }
    before += __builtin_amdgcn_readlane(incl, 63);
    slots += __builtin_amdgcn_readlane(slot_incl, 63);
    return false;
  });
}

// Tile of a segment's product [N][K]: rows n (dy columns, B), columns k (x
// columns, A), contraction over the segment's rows.
template <typename Out, int kNWN, int kNWM, int kTN, int kTM, int kBufsA, int kBufsB>
__global__ __launch_bounds__(64 * kNWN * kNWM, kNWN * kNWM / 4) void weight_kernel(GroupedArgs g) {
  using T = Tile<false, true, true, kNWN, kNWM, kTN, kTM, kBufsA, kBufsB>;
  __shared__ __attribute__((aligned(16))) char smem[imax(T::kLds, T::out_bytes(4))];
  const int N = g.nout, K = g.kc;
  const int nk = (K + T::kCols - 1) / T::kCols, nn = (N + T::kRows - 1) / T::kRows;
  Segment sg;
  if (!find_segment(g, nn * nk, sg)) return;
  const int lo = sg.lo, cnt = sg.n, r = sg.r;
  // row tiles in groups, as in find_tile
  const int grp = r / (kTileGroup * nk), gt = min(kTileGroup, nn - grp * kTileGroup), rr = r - grp * kTileGroup * nk;
  const int k0 = (rr / gt) * T::kCols, n0 = (grp * kTileGroup + rr % gt) * T::kRows;
  const int t = threadIdx.x, lane = t & 63, wave = __builtin_amdgcn_readfirstlane(t >> 6);
  typename T::A a;
  typename T::B b;
  a.init(static_cast<const char*>(g.x) + ((int64_t)lo * K + k0) * 2, (int64_t)cnt * K * 2 - 2 * k0, 2 * K, 0, wave, lane);
  b.init(static_cast<const char*>(g.w) + ((int64_t)lo * N + n0) * 2, (int64_t)cnt * N * 2 - 2 * n0, 2 * N, 0, wave, lane);
  f32x16 acc[kTN][kTM];
#pragma unroll
  for (int n = 0; n < kTN; ++n)
#pragma unroll
    for (int m = 0; m < kTM; ++m) acc[n][m] = (f32x16){};
  T::run(smem, a, b, nullptr, 0, (cnt + 63) / 64, acc);
  const int nrows = min(T::kRows, N - n0), ncols = min(T::kCols, K - k0);
  if (sg.nseg == 1)
    T::store(smem, acc, static_cast<Out*>(g.out) + ((int64_t)sg.e * N + n0) * K + k0, K, nrows, ncols);
  else if (sg.slot + sg.nseg <= g.slots)
    T::store(smem, acc, g.partial + ((int64_t)(sg.slot + sg.k) * N + n0) * K + k0, K, nrows, ncols);
}

// dw of the blockIdx.y-th expert of several segments: their sums, in order.
template <typename Out>
__global__ __launch_bounds__(256) void sum_segments_kernel(GroupedArgs g) {
  const ExpertRows x(g);
  int e = -1, nseg = 0, slot = 0, many = 0, slots = 0;
  x.visit([&](int i, int, int n) {
    const int ns = (n + g.segment - 1) / g.segment, sl = ns > 1 ? ns : 0;
    const int rank = wave_scan(ns > 1 ? 1 : 0), slot_incl = wave_scan(sl);
    const uint64_t hit = __ballot(ns > 1 && many + rank - 1 == (int)blockIdx.y);
    if (hit) {
      const int src = __builtin_ctzll(hit);
      e = i + src;
      nseg = __builtin_amdgcn_readlane(ns, src);
      slot = slots + __builtin_amdgcn_readlane(slot_incl - sl, src);
      return true;
    }
    many += __builtin_amdgcn_readlane(rank, 63);
    slots += __builtin_amdgcn_readlane(slot_incl, 63);
    return false;
  });
  if (e < 0 || slot + nseg > g.slots) return;
  const int64_t nk4 = (int64_t)g.nout * g.kc / 4;   // (K % 8 == 0)
  const float4* p = reinterpret_cast<const float4*>(g.partial) + slot * nk4;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < nk4; i += (int64_t)gridDim.x * 256) {
    float4 s = p[i];
    for (int k = 1; k < nseg; ++k) {
      const float4 v = p[k * nk4 + i];
      s.x += v.x; s.y += v.y; s.z += v.z; s.w += v.w;
    }
    if constexpr (sizeof(Out) == 4)
      reinterpret_cast<float4*>(g.out)[e * nk4 + i] = s;
    else
      reinterpret_cast<uint2*>(g.out)[e * nk4 + i] = make_uint2(pack_bf16x2(s.x, s.y), pack_bf16x2(s.z, s.w));
  }
}

// ---------------------------------------------------------------------------
// Few rows per expert (decode): the product streams the weights once and the
// matrix cores have time to spare, so a work item is at most 16 rows of an
// expert by 16 columns, and belongs to the four waves of a workgroup, which
// split the contraction and add their sums in wave order through LDS (kSplit),
// or to one wave.  A wave reads units of 256 B of its weight rows straight
// into MFMA operands (16x16x32 bf16 / 16x16x128 MXFP4), one unit ahead, lane
// group g = lane / 16 holding chunk 4 j + g of the unit for MFMA j, so that 64
// consecutive bytes of 16 rows are read at a time.  Bound by HBM: 5.2 TB/s for
// two rows over eight experts of N = 28672, K = 4096, 5.5 TB/s for 256 rows
// over 64 experts of N = K = 2048 (bf16).
// ---------------------------------------------------------------------------
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef int i32x4 __attribute__((ext_vector_type(4)));

constexpr int kUnitBytes = 256;

// Sixteen scale bytes of a row: those of unit u, zeros past the row's end
// (where the last sixteen of the row are read and shifted down).
__device__ __forceinline__ u32x4 unit_scales(const uint8_t* p, int n, int u) {
  uint64_t v[2] = {0, 0};
  const int at = 16 * u;
  if (p && at < n) {
    const int over = at + 16 - n;   // the same for all lanes
    if (n < 16) {
      for (int i = 0; i < min(n, 8); ++i) v[0] |= (uint64_t)p[i] << (8 * i);
      for (int i = 8; i < n; ++i) v[1] |= (uint64_t)p[i] << (8 * (i - 8));
    } else {
      __builtin_memcpy(v, p + (over > 0 ? n - 16 : at), 16);
      if (over >= 8) {
        v[0] = v[1] >> (8 * (over - 8));
        v[1] = 0;
      } else if (over > 0) {
        v[0] = v[0] >> (8 * over) | v[1] << (64 - 8 * over);
        v[1] >>= 8 * over;
      }
    }
  }
  return u32x4{(uint32_t)v[0], (uint32_t)(v[0] >> 32), (uint32_t)v[1], (uint32_t)(v[1] >> 32)};
}

constexpr int kFewWaves = 4;

template <bool kMX, bool kSplit>
__global__ __launch_bounds__(64 * kFewWaves) void few_rows_kernel(GroupedArgs g) {
  constexpr int kCols = kSplit ? 16 : 16 * kFewWaves;   // of a workgroup
  __shared__ __attribute__((aligned(16))) f32x4 part[kSplit ? kFewWaves : 1][64];
  int e, row0, nrows, ct;
  if (!find_tile(g, 16, (g.nout + kCols - 1) / kCols, e, row0, nrows, ct)) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l16 = lane & 15, grp = lane >> 4;
  const int kbytes = kMX ? g.kc / 2 : 2 * g.kc;
  const int c0 = ct * kCols + (kSplit ? 0 : 16 * wave), ncols = min(16, g.nout - c0);
  if (!kSplit && ncols <= 0) return;   // (no barrier there)
  const __amdgpu_buffer_rsrc_t rx = buffer(static_cast<const char*>(g.x) + (int64_t)row0 * kbytes, (int64_t)nrows * kbytes);
  const __amdgpu_buffer_rsrc_t rw =
      buffer(static_cast<const char*>(g.w) + ((int64_t)e * g.nout + c0) * kbytes, (int64_t)ncols * kbytes);
  const int nscale = g.kc / 32;
  const uint8_t *xs = nullptr, *ws = nullptr;
  if constexpr (kMX) {
    if (l16 < nrows) xs = g.x_scales + (int64_t)(row0 + l16) * nscale;
    if (l16 < ncols) ws = g.w_scales + ((int64_t)e * g.nout + c0 + l16) * nscale;
  }

  struct Unit {
    u32x4 w[4], x[4], sw, sx;
  };
  // unit u (what is out of range loads zeros)
  auto load = [&](Unit& v, int u) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int at = u * kUnitBytes + 64 * j + 16 * grp;
      const uint32_t off = at < kbytes ? (uint32_t)l16 * (uint32_t)kbytes + (uint32_t)at : kPast;
      v.w[j] = buffer_load16(rw, off);
      v.x[j] = buffer_load16(rx, off);
    }
    if constexpr (kMX) {
      v.sx = unit_scales(xs, nscale, u);
      v.sw = unit_scales(ws, nscale, u);
    }
  };
  f32x4 acc = {0.f, 0.f, 0.f, 0.f};
  auto use = [&](const Unit& v) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (kMX) {
        const u32x4 a = v.w[j], b = v.x[j];
        const i32x8 xa = {(int)a.x, (int)a.y, (int)a.z, (int)a.w, 0, 0, 0, 0};
        const i32x8 xb = {(int)b.x, (int)b.y, (int)b.z, (int)b.w, 0, 0, 0, 0};
        acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(xa, xb, acc, 4, 4, 0, v.sw[j] >> (8 * grp), 0,
                                                               v.sx[j] >> (8 * grp));
      } else {
        acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, v.w[j]),
                                                      __builtin_bit_cast(bf16x8, v.x[j]), acc, 0, 0, 0);
      }
    }
    mfma_done(acc);
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
    part[wave][lane] = acc;
    __syncthreads();
    if (wave) return;
#pragma unroll
    for (int v = 1; v < kFewWaves; ++v) {
      const f32x4 q = part[v][lane];
      acc.x += q.x; acc.y += q.y; acc.z += q.z; acc.w += q.w;
    }
  }
  // the lane holds columns 4 (lane / 16) .. +3 of row lane % 16
  if (l16 < nrows && 4 * grp < ncols)
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(g.out) + (int64_t)(row0 + l16) * g.nout + c0 + 4 * grp) =
        make_uint2(pack_bf16x2(acc.x, acc.y), pack_bf16x2(acc.z, acc.w));
}

template <bool kMX>
hipError_t launch_few_rows(const GroupedArgs& g, hipStream_t s) {
  const int64_t tiles = (g.nout + 15) / 16, slots = (int64_t)g.M / 16 + (g.E < g.M ? g.E : g.M);
  // Long rows are split over the waves (bf16, K = 2048, 512 rows over 128
  // experts: 143 us, 154 whole); rows of less than two units a wave are not,
  // where there are tiles enough for every wave to have its own (MXFP4, K =
  // 2880, 64 rows over 32 experts: 60 us, 73 split).
  const int64_t units = ((kMX ? g.kc / 2 : 2 * g.kc) + kUnitBytes - 1) / kUnitBytes;
  if (units >= 2 * kFewWaves || slots * tiles < 4096)
    few_rows_kernel<kMX, true><<<(unsigned)items_grid(slots * tiles), 64 * kFewWaves, 0, s>>>(g);
  else
    few_rows_kernel<kMX, false>
        <<<(unsigned)items_grid(slots * ((tiles + kFewWaves - 1) / kFewWaves)), 64 * kFewWaves, 0, s>>>(g);
  return hipGetLastError();
}

template <bool kMX, bool kAT, int kNWN, int kNWM, int kTN, int kTM, int kBufsA, int kBufsB>
hipError_t launch_rows(const GroupedArgs& g, hipStream_t s) {
  using Big = Tile<kMX, kAT, false, kNWN, kNWM, kTN, kTM, kBufsA, kBufsB>;
  const int64_t ncol = (g.nout + Big::kCols - 1) / Big::kCols;
  const int64_t tiles = (int64_t)g.M / Big::kRows + (g.E < g.M ? g.E : g.M);
  const int64_t grid = items_grid(tiles * ncol);
  rows_kernel<kMX, kAT, kNWN, kNWM, kTN, kTM, kBufsA, kBufsB><<<(unsigned)grid, 64 * kNWN * kNWM, 0, s>>>(g);
  return hipGetLastError();
}

template <typename Out, int kNWN, int kNWM, int kTN, int kTM, int kBufsA, int kBufsB>
hipError_t launch_weight(const GroupedArgs& g, hipStream_t s) {
  using T = Tile<false, true, true, kNWN, kNWM, kTN, kTM, kBufsA, kBufsB>;
  const int64_t tiles = (int64_t)((g.nout + T::kRows - 1) / T::kRows) * ((g.kc + T::kCols - 1) / T::kCols);
  const int64_t grid = items_grid((g.E + g.M / g.segment) * tiles);
  weight_kernel<Out, kNWN, kNWM, kTN, kTM, kBufsA, kBufsB><<<(unsigned)grid, 64 * kNWN * kNWM, 0, s>>>(g);
  return hipGetLastError();
}

// Whether the product does little more than stream one operand past the
// other, row by row or column by column.  us here and in tiles, inputs from HBM:
//   few rows per expert (the weights stream)       rows  here  tiles
//     bf16, E = 64, N = K = 2048                      8   106    123
//                                                    12   118    125
//                                                    16   131    124
//     bf16, E = 8, N = K = 4096                       8    55     61
//                                                    16    64     61
//     MXFP4, E = 32, N = 5760, K = 2880            1, 2 65, 66 71, 71
//                                                  3, 4 67, 68 72, 72
//     MXFP4, E = 8, N = K = 4096                   1, 2 20, 21 18, 18
//                                                  3, 4     22     18
//   few output columns (the rows stream), bf16,       N
//     E = 64, K = 2048, 64 rows each             16, 32  9, 12 18, 18
//     512 rows each                              24, 32 58, 61 38, 38
// so MXFP4, with as many loads of scales for half the bytes, stops at two rows,
// where the one layer gains as much as the other loses.
// A grid holds less than 2^32 threads; beyond that the tiles serve.
bool streams(const GroupedArgs& g, bool mx) {
  const int64_t items = ((int64_t)g.M / 16 + std::min(g.E, g.M)) * ((g.nout + 15) / 16);
  return (g.M <= (mx ? 2 : 8) * g.E || g.nout <= 16) && items_grid(items) * 64 * kFewWaves < (int64_t(1) << 32);
}

// Whether tiles of 256 x 256 would leave compute units without work; those of
// half the columns then do better (and have room for a third buffer).  us in
// tiles of 128 and of 256 columns, E = 8, 256 rows each, contraction 4096:
//   tiles of 256 columns   bf16     grad_input    MXFP4
//     64                  61,  88    59,  78     26, 37
//    128                  80,  95    78,  82     33, 38
//    144                 123,  99   118,  90     50, 39
//    192                 131, 114   125, 106     54, 43
// 128 rows each, 4096 outputs, contraction 14336 (128): bf16 191-208 and 232-270,
// grad_input 178 and 215, MXFP4 71 and 98.
bool few_tiles(const GroupedArgs& g) {
  const int64_t experts = std::min(g.E, g.M), rows = std::max<int64_t>(1, (g.M / experts + 255) / 256) * experts;
  return rows * ((g.nout + 255) / 256) <= 128;
}

template <bool kMX>
hipError_t launch_forward(const GroupedArgs& g, hipStream_t s) {
  if (streams(g, kMX)) return launch_few_rows<kMX>(g, s);
  if constexpr (!kMX)
    if (g.kc <= 64) return launch_rows<false, false, 4, 1, 1, 2, 1, 1>(g, s);
  if (few_tiles(g)) return launch_rows<kMX, false, 4, 2, 1, 4, 3, 3>(g, s);
  // (three buffers of the columns' operand leave no room for the scales)
  return launch_rows<kMX, false, 4, 2, 2, 4, kMX ? 2 : 3, 2>(g, s);
}

}  // namespace

hipError_t launch_grouped_mm(const GroupedArgs& g, hipStream_t s) { return launch_forward<false>(g, s); }

hipError_t launch_grouped_mm_mxfp4(const GroupedArgs& g, hipStream_t s) { return launch_forward<true>(g, s); }

hipError_t launch_grouped_mm_grad_input(const GroupedArgs& g, hipStream_t s) {
  if (g.kc <= 64) return launch_rows<false, true, 4, 1, 1, 2, 1, 1>(g, s);
  if (few_tiles(g)) return launch_rows<false, true, 4, 2, 1, 4, 3, 3>(g, s);
  return launch_rows<false, true, 4, 2, 2, 4, 3, 2>(g, s);
}

namespace {

// Tile shapes of grad_weight: narrow outputs take tiles that are narrow, too
// (and more of them on a compute unit).  us in narrow and in square tiles, E =
// 64, 512 rows each, bf16, the other side 2048, inputs from HBM:
//   narrow side      16      64      72      96     128     192     256
//     few rows   38, 45  45, 49  48, 49  51, 50  52, 54  65, 61  79, 67
//     few cols   31, 46  37, 49  48, 49  51, 51  53, 53  65, 60  80, 67
enum class WeightTile { kSquare, kFewRows, kFewCols };
WeightTile weight_tile(int32_t N, int32_t K) {
  return N <= 64 ? WeightTile::kFewRows : K <= 64 ? WeightTile::kFewCols : WeightTile::kSquare;
}

template <typename Out>
hipError_t launch_weight_for(const GroupedArgs& g, hipStream_t s) {
  hipError_t e;
  switch (weight_tile(g.nout, g.kc)) {
    case WeightTile::kFewRows: e = launch_weight<Out, 2, 2, 2, 1, 2, 2>(g, s); break;
    case WeightTile::kFewCols: e = launch_weight<Out, 2, 2, 1, 4, 2, 2>(g, s); break;
    default: e = launch_weight<Out, 4, 2, 2, 4, 3, 2>(g, s);
  }
  const int32_t many = g.M / (g.segment + 1);   // experts of more than one segment, at most
  if (e != hipSuccess || many == 0) return e;
  const int64_t blocks = ((int64_t)g.nout * g.kc / 4 + 255) / 256;
  sum_segments_kernel<Out><<<dim3((unsigned)std::min<int64_t>(blocks, 1024), (unsigned)many), 256, 0, s>>>(g);
  return hipGetLastError();
}

}  // namespace

int32_t grad_weight_segment(int32_t M, int32_t N, int32_t K) {
  // Enough segments to fill the card when every expert had one (1024 narrow
  // or 256 square tiles), of at least 512 rows: eight steps, so that a slot's
  // traffic stays below that of the rows.
  const WeightTile w = weight_tile(N, K);
  const int64_t rows = w == WeightTile::kFewRows ? 64 : 256, cols = w == WeightTile::kFewRows ? 128 : w == WeightTile::kFewCols ? 64 : 256;
  const int64_t tiles = ((N + rows - 1) / rows) * ((K + cols - 1) / cols);
  const int64_t want = std::max<int64_t>(1, (w == WeightTile::kSquare ? 256 : 1024) / tiles);
  const int64_t len = std::max<int64_t>(512, (M + want - 1) / want);
  return (int32_t)((len + 63) / 64 * 64);
}

int64_t grad_weight_slots(int32_t M, int32_t segment) {
  const int64_t many = M / (segment + 1);   // experts of more than one segment, each with at most one not full
  return many ? M / segment + many : 0;
}

hipError_t launch_grouped_mm_grad_weight(const GroupedArgs& g, bool fp32, hipStream_t s) {
  return fp32 ? launch_weight_for<float>(g, s) : launch_weight_for<uint16_t>(g, s);
}

}  // namespace moeq
