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
#include "grouped_tile.h"

namespace moeq {
namespace {

// forward (kAT = false, kMX or not) and grad_input (kAT = true).
//   x [M][kc], w [E][..], out [M][nout]: kc contraction length, nout columns.
template <bool kMX, bool kAT, int kNWN, int kNWM, int kTN, int kTM, int kBufsA, int kBufsB>
__device__ __forceinline__ void rows_tile(char* smem, const GroupedArgs& g, int e, int row0, int nrows, int c0) {
  using T = Tile<kMX ? Op::kMxfp4 : Op::kBf16, kAT, false, kNWN, kNWM, kTN, kTM, kBufsA, kBufsB>;
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
  using Big = Tile<kMX ? Op::kMxfp4 : Op::kBf16, kAT, false, kNWN, kNWM, kTN, kTM, kBufsA, kBufsB>;
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
  using T = Tile<Op::kBf16, true, true, kNWN, kNWM, kTN, kTM, kBufsA, kBufsB>;
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
  using Big = Tile<kMX ? Op::kMxfp4 : Op::kBf16, kAT, false, kNWN, kNWM, kTN, kTM, kBufsA, kBufsB>;
  const int64_t ncol = (g.nout + Big::kCols - 1) / Big::kCols;
  const int64_t tiles = (int64_t)g.M / Big::kRows + (g.E < g.M ? g.E : g.M);
  const int64_t grid = items_grid(tiles * ncol);
  rows_kernel<kMX, kAT, kNWN, kNWM, kTN, kTM, kBufsA, kBufsB><<<(unsigned)grid, 64 * kNWN * kNWM, 0, s>>>(g);
  return hipGetLastError();
}

template <typename Out, int kNWN, int kNWM, int kTN, int kTM, int kBufsA, int kBufsB>
hipError_t launch_weight(const GroupedArgs& g, hipStream_t s) {
  using T = Tile<Op::kBf16, true, true, kNWN, kNWM, kTN, kTM, kBufsA, kBufsB>;
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
