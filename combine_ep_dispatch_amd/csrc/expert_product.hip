// The experts' products on the dispatched rows: y[r, :] = act(W[e(r)] a[r]),
// W in MXFP4, rows in MXFP4 or in FP8 with one binary32 scale per 128
// channels.  The contract is ep_expert_product's in include/ep.h.
//
// gfx950's scaled MFMA takes the codes as they are and multiplies each
// 32-channel block by both operands' E8M0 scales.  The weights are its A
// operand (16 channels of y), the rows its B operand (16 rows), so a lane
// ends up with four consecutive channels of one row.

#include "ep_device.h"
#include "ep_internal.h"
#include "mx_device.h"

namespace ep {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kFp4 = 4, kFp8 = 0;  // operand formats of the scaled MFMA
constexpr int kThreads = 256;
constexpr int kMaxExperts = 1024;

// Rows of expert e: [first, first + count), clamped to the buffer.
__device__ __forceinline__ void rows_of(const int32_t* __restrict__ expert_rows, int e, int capacity, int num_rows,
                                        int& first, int& count) {
  if (capacity > 0) {
    first = e * capacity;
    count = min(max(expert_rows[e], 0), capacity);
  } else {
    first = min(max(expert_rows[e], 0), num_rows);
    count = max(min(expert_rows[e + 1], num_rows) - first, 0);
  }
}

__device__ __forceinline__ float silu_mul(float g, float u) { return g / (1.0f + __expf(-g)) * u; }

template <bool FP8, bool GATED>
__global__ __launch_bounds__(kThreads) void product_kernel(const uint8_t* __restrict__ a,
                                                           const uint8_t* __restrict__ a_scale,
                                                           const uint8_t* __restrict__ w,
                                                           const uint8_t* __restrict__ w_scale,
                                                           const int32_t* __restrict__ expert_rows, int32_t num_rows,
                                                           int32_t E, int32_t capacity, int32_t H, int32_t N,
                                                           uint16_t* __restrict__ y) {
  constexpr int BM = 16, BN = 64;
  __shared__ int start[kMaxExperts + 1];  // row tiles before each expert
  const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave;
  for (int e = tid; e < E; e += kThreads) {
    int first, count;
    rows_of(expert_rows, e, capacity, num_rows, first, count);
    start[e] = (count + BM - 1) / BM;
  }
  if (tid == 0) start[E] = 0;
  __syncthreads();
  block_exclusive_scan(start, E + 1);
  const int O = GATED ? N / 2 : N;  // channels of y
  const int nt = (O + BN - 1) / BN;
  const int64_t tiles = static_cast<int64_t>(start[E]) * nt;
  const int grp = lane >> 4, col = lane & 15;
  for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    const int q = static_cast<int>(tile / nt);
    int lo = 0, hi = E;  // the expert with start[lo] <= q < start[lo + 1]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (start[mid] <= q) lo = mid; else hi = mid;
    }
    int first, count;
    rows_of(expert_rows, lo, capacity, num_rows, first, count);
    const int te = start[lo + 1] - start[lo];
    const int64_t local = tile - static_cast<int64_t>(start[lo]) * nt;
    const int m0 = static_cast<int>(local % te) * BM, n0 = static_cast<int>(local / te) * BN + wave * 16;
    const int m = m0 + col;
    const size_t row = static_cast<size_t>(first) + min(m, count - 1);
    const uint8_t* ap = a + row * (FP8 ? H : H / 2);
    const uint8_t* as = a_scale + row * (H / 32);
    const size_t wrow = static_cast<size_t>(lo) * N + min(n0 + col, O - 1);
    f32x4 acc[GATED ? 2 : 1];
#pragma unroll
    for (auto& c : acc) c = f32x4{0, 0, 0, 0};
    for (int k = 0; k < H; k += 128) {
      i32x8 b = {0, 0, 0, 0, 0, 0, 0, 0};
      int sb = 127;
      if constexpr (FP8) {
        *reinterpret_cast<u32x4*>(&b) = *reinterpret_cast<const u32x4*>(ap + k + 16 * grp);
        *(reinterpret_cast<u32x4*>(&b) + 1) = *reinterpret_cast<const u32x4*>(ap + k + 64 + 16 * grp);
      } else {
        *reinterpret_cast<u32x4*>(&b) = *reinterpret_cast<const u32x4*>(ap + k / 2 + 16 * grp);
        sb = as[k / 32 + grp];
      }
#pragma unroll
      for (int h = 0; h < (GATED ? 2 : 1); ++h) {
        const size_t wr = wrow + (h == 1 ? O : 0);
        i32x8 v = {0, 0, 0, 0, 0, 0, 0, 0};
        *reinterpret_cast<u32x4*>(&v) = *reinterpret_cast<const u32x4*>(w + wr * (H / 2) + k / 2 + 16 * grp);
        const int sw = w_scale[wr * (H / 32) + k / 32 + grp];
        if constexpr (FP8) {
          const f32x4 d = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(v, b, f32x4{0, 0, 0, 0}, kFp4, kFp8, 0, sw,
                                                                           0, sb);
          const float s = reinterpret_cast<const float*>(as)[k / 128];
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[h][i] = __builtin_fmaf(s, d[i], acc[h][i]);
        } else {
          acc[h] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(v, b, acc[h], kFp4, kFp4, 0, sw, 0, sb);
        }
      }
    }
    const int n = n0 + 4 * grp;  // this lane's four channels; O is a multiple of 8
    if (m < count && n < O) {
      __bf16 o[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        o[i] = static_cast<__bf16>(GATED ? silu_mul(acc[0][i], acc[GATED ? 1 : 0][i]) : acc[0][i]);
      *reinterpret_cast<uint2*>(y + row * O + n) = *reinterpret_cast<uint2*>(o);
    }
  }
}

// ---- the tiled kernel --------------------------------------------------------
//
// Workgroup tile: BN weight rows (with GATED half gate, half up, of the same
// BN/2 channels of y) times BM token rows, over all of H in stages of 256
// channels.  A stage's codes go from global memory straight to LDS (16 bytes a
// lane), into one of two buffers while the other one is multiplied.  LDS rows
// are 128 bytes (FP8 rows 256) and hold their 16-byte pieces in the order
// piece ^ (row & 7) (& 15), so that eight lanes reading one piece of eight
// rows meet all banks.  Scales go along 16 bytes a row (512 channels) at a
// time, every second stage.

typedef float f32x16 __attribute__((ext_vector_type(16)));

__device__ __forceinline__ void wait_loads() {
  __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0): the copies to LDS count there
}

typedef __amdgpu_buffer_rsrc_t Rsrc;
typedef __attribute__((address_space(3))) void LdsVoid;

__device__ __forceinline__ Rsrc make_rsrc(const void* p, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, static_cast<int>(bytes), 0x00027000);
}

// 64 lanes x 16 bytes: lane l's piece lands at dst + 16 l.
__device__ __forceinline__ void copy16(Rsrc src, uint8_t* dst, uint32_t lane_off, uint32_t off) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(src, (LdsVoid*)dst, 16, lane_off, off, 0, 0);
}

__device__ __forceinline__ i32x8 widen(u32x4 lo) {
  return i32x8{static_cast<int>(lo[0]), static_cast<int>(lo[1]), static_cast<int>(lo[2]), static_cast<int>(lo[3]), 0, 0, 0, 0};
}

template <bool FP8, bool GATED, int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(WM* WN* kWave) void product_tiled(
    const uint8_t* __restrict__ a, const uint8_t* __restrict__ a_scale, const uint8_t* __restrict__ w,
    const uint8_t* __restrict__ w_scale, const int32_t* __restrict__ expert_rows, int32_t num_rows, int32_t E,
    int32_t capacity, int32_t H, int32_t N, uint16_t* __restrict__ y) {
  constexpr int NW = WM * WN, kThr = NW * kWave;
  constexpr int TM = BM / WM, TN = BN / WN;    // a wave's rows and weight rows
  constexpr int FM = TM / 32, FN = TN / 32;
  constexpr int AB = FP8 ? 256 : 128;          // bytes of a token row in a stage
  constexpr int LW = BN / 8 / NW;              // copies per wave and stage: 8 weight rows each
  constexpr int LA = BM * AB / 1024 / NW;      // (1024 / AB token rows each)
  static_assert(LW * 8 * NW == BN && LA * 1024 * NW == BM * AB && FM * 32 * WM == BM && FN * 32 * WN == BN, "tile");
  static_assert(!GATED || FN % 2 == 0, "a wave holds both halves of its channels");
  constexpr int SR = BN + (BM < 64 ? 64 : BM);  // rows of scales, in copies of 64
  constexpr int LS = (SR / 64 + NW - 1) / NW;   // those per wave
  __shared__ __align__(16) uint8_t w0[BN * 128];
  __shared__ __align__(16) uint8_t w1[BN * 128];
  __shared__ __align__(16) uint8_t a0[BM * AB];
  __shared__ __align__(16) uint8_t a1[BM * AB];
  __shared__ __align__(16) uint8_t sc[2][SR * 16 + 16];
  __shared__ int start[kMaxExperts + 1];
  const int tid = threadIdx.x, lane = tid & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int half = lane >> 5, col = lane & 31;
  const int wm = wave % WM, wn = wave / WM;
  for (int e = tid; e < E; e += kThr) {
    int first, count;
    rows_of(expert_rows, e, capacity, num_rows, first, count);
    start[e] = (count + BM - 1) / BM;
  }
  if (tid == 0) start[E] = 0;
  __syncthreads();
  block_exclusive_scan(start, E + 1);
  const int O = GATED ? N / 2 : N;
  constexpr int BO = GATED ? BN / 2 : BN;  // channels of y per tile
  const int nt = (O + BO - 1) / BO;
  const uint32_t wrow_bytes = H / 2, arow_bytes = FP8 ? H : H / 2, srow_bytes = H / 32;
  const int stages = (H + 255) / 256;
  const bool tail = (H & 255) != 0;  // the last stage holds 128 channels
  const uint32_t tiles = static_cast<uint32_t>(start[E]) * nt;

  // tiles in eight runs, one per XCD (workgroups go to the XCDs in turn)
  const uint32_t run = (tiles + 7) / 8, step = gridDim.x / 8;
  for (uint32_t t = blockIdx.x / 8; t < run; t += step) {
    const uint32_t tile = (blockIdx.x & 7) * run + t;
    if (tile >= tiles) break;
    const int q = static_cast<int>(tile / nt);
    int lo = 0, hi = E;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (start[mid] <= q) lo = mid; else hi = mid;
    }
    const int e = __builtin_amdgcn_readfirstlane(lo);
    int first, count;
    rows_of(expert_rows, e, capacity, num_rows, first, count);
    const uint32_t before = start[e], te = start[e + 1] - before;
    const uint32_t local = tile - before * nt;
    const int m0 = __builtin_amdgcn_readfirstlane(static_cast<int>(local % te) * BM);
    const int n0 = __builtin_amdgcn_readfirstlane(static_cast<int>(local / te) * BO);
    first = __builtin_amdgcn_readfirstlane(first);
    const int rows = __builtin_amdgcn_readfirstlane(min(count - m0, BM));  // >= 1
    const size_t row0 = static_cast<size_t>(first) + m0;

    const Rsrc wr = make_rsrc(w + static_cast<size_t>(e) * N * wrow_bytes, static_cast<uint32_t>(N) * wrow_bytes);
    const Rsrc ar = make_rsrc(a + row0 * arow_bytes, static_cast<uint32_t>(rows) * arow_bytes);
    const Rsrc wsr = make_rsrc(w_scale + static_cast<size_t>(e) * N * srow_bytes, static_cast<uint32_t>(N) * srow_bytes);
    const Rsrc asr = make_rsrc(a_scale + row0 * srow_bytes, static_cast<uint32_t>(rows) * srow_bytes);

    // this lane's pieces: rows past the end repeat the last one
    const auto weight_row = [&](int r) -> uint32_t {
      if (!GATED) return min(n0 + r, O - 1);
      return r < BO ? min(n0 + r, O - 1) : O + min(n0 + r - BO, O - 1);
    };
    uint32_t woff[LW], aoff[LA], soff[LS];
    const uint32_t wpiece = (lane & 7) ^ (lane >> 3);
    const uint32_t wcut = tail ? (wpiece & 4) * 16 : 0;  // in a last stage of 128 channels, stay inside the row
#pragma unroll
    for (int i = 0; i < LW; ++i) woff[i] = weight_row((wave * LW + i) * 8 + (lane >> 3)) * wrow_bytes + wpiece * 16;
    uint32_t apiece, acut;
#pragma unroll
    for (int i = 0; i < LA; ++i) {
      constexpr int per = 1024 / AB;
      const int r = (wave * LA + i) * per + lane / (AB / 16);
      apiece = (lane % (AB / 16)) ^ (r & (AB / 16 - 1));
      aoff[i] = min(r, rows - 1) * arow_bytes + apiece * 16;
    }
    // FP8: the piece depends on the copy (4 rows each); cut per copy below
    acut = tail ? (AB == 128 ? (wpiece & 4) * 16 : 0) : 0;
#pragma unroll
    for (int i = 0; i < LS; ++i) {
      const int c = wave + i * NW;  // copy c: 64 rows of scales
      soff[i] = (c < BN / 64 ? weight_row(c * 64 + lane) : min((c - BN / 64) * 64 + lane, rows - 1)) * srow_bytes;
    }

    const auto copy_stage = [&](int st, uint8_t* wb, uint8_t* ab) {
      const bool cut = tail && st == stages - 1;
#pragma unroll
      for (int i = 0; i < LW; ++i)
        copy16(wr, wb + (wave * LW + i) * 1024, woff[i] - (cut ? wcut : 0), st * 128);
#pragma unroll
      for (int i = 0; i < LA; ++i) {
        uint32_t c = acut;
        if (AB == 256) {
          const int r = (wave * LA + i) * 4 + lane / 16;
          c = (((lane % 16) ^ (r & 15)) & 8) * 16;
        }
        copy16(ar, ab + (wave * LA + i) * 1024, aoff[i] - (cut ? c : 0), st * AB);
      }
    };
    const auto scale_at = [&](int pair) { return min(static_cast<uint32_t>(pair) * 16, srow_bytes - 16); };
    const auto copy_scales = [&](int pair) {
#pragma unroll
      for (int i = 0; i < LS; ++i) {
        const int c = wave + i * NW;
        uint8_t* dst = sc[pair & 1] + c * 1024;
        if (c < BN / 64) copy16(wsr, dst, soff[i], scale_at(pair));
        else if (c < SR / 64) copy16(asr, dst, soff[i], scale_at(pair));
      }
    };

    f32x16 acc[FN][FM];
#pragma unroll
    for (int i = 0; i < FN; ++i)
#pragma unroll
      for (int j = 0; j < FM; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;

    // the wave's frag i of weight rows starts at this row of the tile
    const auto frag_row = [&](int i) {
      if (!GATED) return wn * TN + i * 32;
      return i < FN / 2 ? wn * (TN / 2) + i * 32 : BO + wn * (TN / 2) + (i - FN / 2) * 32;
    };

    const auto multiply = [&](int st, const uint8_t* wb, const uint8_t* ab, const uint2 (&sw)[FN], const uint2 (&sa)[FM]) {
      const int ksteps = tail && st == stages - 1 ? 2 : 4;
#pragma unroll
      for (int ks = 0; ks < 4; ++ks) {
        if (ks >= ksteps) break;
        i32x8 av[FM], wv[FN];
#pragma unroll
        for (int i = 0; i < FN; ++i) {
          const int r = frag_row(i) + col;
          wv[i] = widen(*reinterpret_cast<const u32x4*>(wb + r * 128 + (((ks * 2 + half) ^ (r & 7)) * 16)));
        }
#pragma unroll
        for (int j = 0; j < FM; ++j) {
          const int r = wm * TM + j * 32 + col;
          if constexpr (FP8) {
            const u32x4 lo4 = *reinterpret_cast<const u32x4*>(ab + r * 256 + (((ks * 4 + half) ^ (r & 15)) * 16));
            const u32x4 hi4 = *reinterpret_cast<const u32x4*>(ab + r * 256 + (((ks * 4 + 2 + half) ^ (r & 15)) * 16));
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              av[j][x] = static_cast<int>(lo4[x]);
              av[j][4 + x] = static_cast<int>(hi4[x]);
            }
          } else {
            av[j] = widen(*reinterpret_cast<const u32x4*>(ab + r * 128 + (((ks * 2 + half) ^ (r & 7)) * 16)));
          }
        }
#pragma unroll
        for (int i = 0; i < FN; ++i)
#pragma unroll
          for (int j = 0; j < FM; ++j) {
            const int sx = ks < 2 ? sw[i].x : sw[i].y;
            if constexpr (FP8) {
              // handled per 128 channels in multiply_fp8
            } else {
              const int sy = ks < 2 ? sa[j].x : sa[j].y;
              if (ks % 2 == 0)
                acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(wv[i], av[j], acc[i][j], kFp4, kFp4, 0, sx, 0, sy);
              else
                acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(wv[i], av[j], acc[i][j], kFp4, kFp4, 2, sx, 2, sy);
            }
          }
      }
    };
    const auto multiply_fp8 = [&](int st, const uint8_t* wb, const uint8_t* ab, const uint2 (&sw)[FN], const uint2 (&sa)[FM]) {
      const int groups = tail && st == stages - 1 ? 1 : 2;
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        if (g >= groups) break;
        i32x8 av[2][FM], wv[2][FN];
#pragma unroll
        for (int k2 = 0; k2 < 2; ++k2) {
          const int ks = g * 2 + k2;
#pragma unroll
          for (int i = 0; i < FN; ++i) {
            const int r = frag_row(i) + col;
            wv[k2][i] = widen(*reinterpret_cast<const u32x4*>(wb + r * 128 + (((ks * 2 + half) ^ (r & 7)) * 16)));
          }
#pragma unroll
          for (int j = 0; j < FM; ++j) {
            const int r = wm * TM + j * 32 + col;
            const u32x4 lo4 = *reinterpret_cast<const u32x4*>(ab + r * 256 + (((ks * 4 + half) ^ (r & 15)) * 16));
            const u32x4 hi4 = *reinterpret_cast<const u32x4*>(ab + r * 256 + (((ks * 4 + 2 + half) ^ (r & 15)) * 16));
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              av[k2][j][x] = static_cast<int>(lo4[x]);
              av[k2][j][4 + x] = static_cast<int>(hi4[x]);
            }
          }
        }
#pragma unroll
        for (int i = 0; i < FN; ++i)
#pragma unroll
          for (int j = 0; j < FM; ++j) {
            const int sx = g == 0 ? sw[i].x : sw[i].y;
            const float s = __uint_as_float(g == 0 ? sa[j].x : sa[j].y);
            f32x16 d;
#pragma unroll
            for (int r = 0; r < 16; ++r) d[r] = 0.0f;
            d = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(wv[0][i], av[0][j], d, kFp4, kFp8, 0, sx, 0, 127);
            d = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(wv[1][i], av[1][j], d, kFp4, kFp8, 2, sx, 0, 127);
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[i][j][r] = __builtin_fmaf(s, d[r], acc[i][j][r]);
          }
      }
    };

    // one stage: read its scales, start the next stage's copies, multiply
    const auto stage = [&](int st, uint8_t* wb, uint8_t* ab, uint8_t* wnext, uint8_t* anext) {
      uint2 sw[FN], sa[FM];
      const int pair = st >> 1;
      const uint32_t at = static_cast<uint32_t>(pair) * 16 - scale_at(pair) + (st & 1) * 8;
      const uint8_t* sb = sc[pair & 1] + at;
#pragma unroll
      for (int i = 0; i < FN; ++i) {
        const uint32_t* p = reinterpret_cast<const uint32_t*>(sb + (frag_row(i) + col) * 16);
        sw[i] = uint2{p[0] >> (8 * half), p[1] >> (8 * half)};
      }
#pragma unroll
      for (int j = 0; j < FM; ++j) {
        const uint32_t* p = reinterpret_cast<const uint32_t*>(sb + (BN + wm * TM + j * 32 + col) * 16);
        sa[j] = FP8 ? uint2{p[0], p[1]} : uint2{p[0] >> (8 * half), p[1] >> (8 * half)};
      }
      if (st + 1 < stages) {
        if ((st & 1) == 0 && st + 2 < stages) copy_scales(pair + 1);
        copy_stage(st + 1, wnext, anext);
      }
      if (wm * TM < rows) {  // else this wave's rows are all past the end
        if constexpr (FP8) multiply_fp8(st, wb, ab, sw, sa); else multiply(st, wb, ab, sw, sa);
      }
      wait_loads();
      __syncthreads();
    };

    copy_scales(0);
    copy_stage(0, w0, a0);
    wait_loads();
    __syncthreads();
    for (int st = 0; st < stages; st += 2) {
      stage(st, w0, a0, w1, a1);
      if (st + 1 < stages) stage(st + 1, w1, a1, w0, a0);
    }

#pragma unroll
    for (int j = 0; j < FM; ++j) {
      const int m = wm * TM + j * 32 + col;
      if (m >= rows) continue;
      uint16_t* yrow = y + (row0 + m) * O;
#pragma unroll
      for (int i = 0; i < (GATED ? FN / 2 : FN); ++i)
#pragma unroll
        for (int r4 = 0; r4 < 4; ++r4) {
          const int n = n0 + frag_row(i) + 8 * r4 + 4 * half;
          if (n >= O) continue;
          __bf16 o[4];
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const float v = acc[i][j][4 * r4 + x];
            o[x] = static_cast<__bf16>(GATED ? silu_mul(v, acc[GATED ? i + FN / 2 : i][j][4 * r4 + x]) : v);
          }
          *reinterpret_cast<uint2*>(yrow + n) = *reinterpret_cast<uint2*>(o);
        }
    }
  }
}

}  // namespace

hipError_t launch_expert_product(const void* a, const void* a_scale, bool fp8, const void* w, const void* w_scale,
                                 const int32_t* expert_rows, int32_t num_rows, int32_t E, int32_t capacity,
                                 int32_t H, int32_t N, bool gated, uint16_t* y, hipStream_t stream) {
  const uint8_t* ap = static_cast<const uint8_t*>(a);
  const uint8_t* as = static_cast<const uint8_t*>(a_scale);
  const uint8_t* wp = static_cast<const uint8_t*>(w);
  const uint8_t* ws = static_cast<const uint8_t*>(w_scale);
  const auto with = [&](auto kernel, int grid, int threads) {
    hipLaunchKernelGGL(kernel, dim3(grid), dim3(threads), 0, stream, ap, as, wp, ws, expert_rows, num_rows, E,
                       capacity, H, N, y);
    return hipGetLastError();
  };
  const auto pick = [&](auto f, auto g) {
    constexpr bool F = decltype(f)::value, G = decltype(g)::value;
    if (H < 512) return with(product_kernel<F, G>, 2048, kThreads);
    const int64_t avg = num_rows / E;
    if (avg <= 48 || capacity > 0) return with(product_tiled<F, G, 32, 128, 1, 2>, 768, 128);
    if constexpr (!F) {
      if (avg > 192) return with(product_tiled<F, G, 256, 256, 2, 4>, 256, 512);
    }
    return with(product_tiled<F, G, 128, 256, 2, 4>, 256, 512);
  };
  if (fp8) return gated ? pick(std::true_type{}, std::true_type{}) : pick(std::true_type{}, std::false_type{});
  return gated ? pick(std::false_type{}, std::true_type{}) : pick(std::false_type{}, std::false_type{});
}

}  // namespace ep
