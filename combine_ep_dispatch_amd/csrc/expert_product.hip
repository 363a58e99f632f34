// The experts' products on the dispatched rows: y[r, :] = act(W[e(r)] a[r]),
// W in MXFP4, rows in MXFP4 or in FP8 with one binary32 scale per 128
// channels.  The contract is ep_expert_product's in include/ep.h.
//
// gfx950's scaled MFMA takes the codes as they are and multiplies each
// 32-channel block by both operands' E8M0 scales.  The weights are its A
// operand (channels of y), the rows its B operand, so a lane ends up with four
// consecutive channels of one row.  FP8 rows go through it with a scale of 1
// and 128 channels at a time, whose sums are scaled on the vector unit; codes
// below 2 and the others go through it apart, see split_codes.
//
// With E 256, H 7168, N 4096 gated and 8 experts a token, MXFP4 rows: 1 token
// 23 us; 128 tokens 550 (the weights at 7.1 TB/s); 4096 tokens 930 (4.6 TB/s,
// 2.1 PFLOP/s), up to 1120 on slower cards, bounded by copies into LDS that end
// at each stage's barrier (without products 846 of 1120, without the rows'
// copies as well 724); 32768 tokens 4560 to 4640 (3.4 PFLOP/s; the matrix unit
// reaches 6.1 on such operands alone).  FP8 rows take twice the LDS and, split,
// four times the matrix cycles: 42, 700, 2190 and 13900.

#include "ep_device.h"
#include "ep_internal.h"
#include "expert_device.h"
#include "mx_device.h"

namespace ep {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));

constexpr int kFp4 = 4, kFp8 = 0;  // operand formats of the scaled MFMA
constexpr int kThreads = 256;

// FP8 codes below 2 in magnitude, and those of 2 and more; zeros elsewhere.
// The matrix unit adds the products of eight neighbouring channels in one step
// and drops what lies more than 13 binades below the largest one's exponent
// (measured: beside 448 x 6, a product below 2^-3 is lost).  E4M3 x E2M1 spans
// 21 binades; split at 2 each half spans 13, so that all products count in
// full: those below 2 are multiples of 2^-10 with exponents up to 2, the others
// multiples of 2^-3 with exponents up to 10.  (MXFP4 rows need none of this:
// eight of their products share a scale and span 8 binades.)
__device__ __forceinline__ void split_codes(i32x8 x, i32x8& low, i32x8& high) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t v = x[i];
    // bit 6 of each byte, the exponent's highest, spread over the byte
    const uint32_t m = __builtin_amdgcn_perm(v << 9, v << 1, 0x090B080A);
    high[i] = static_cast<int>(v & m);
    low[i] = static_cast<int>(v & ~m);
  }
}

template <bool FP8, bool GATED>
__global__ __launch_bounds__(kThreads) void product_kernel(const uint8_t* __restrict__ a,
                                                           const uint8_t* __restrict__ a_scale,
                                                           const uint8_t* __restrict__ w,
                                                           const uint8_t* __restrict__ w_scale,
                                                           const int32_t* __restrict__ expert_rows, int32_t num_rows,
                                                           int32_t E, int32_t capacity, int32_t H, int32_t N,
                                                           uint16_t* __restrict__ y) {
  constexpr int BM = 16, BN = 64;
  __shared__ RowTiles start[kMaxExperts + 1];  // row tiles before each expert
  const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave;
  for (int e = tid; e < E; e += kThreads) {
    int first, count;
    rows_of(expert_rows, e, capacity, num_rows, first, count);
    start[e] = (count + BM - 1) / BM;
  }
  if (tid == 0) start[E] = 0;
  __syncthreads();
  tiles_before(start, E);
  const int O = GATED ? N / 2 : N;  // channels of y
  const int nt = (O + BN - 1) / BN;
  const int64_t tiles = start[E] * nt;
  const int grp = lane >> 4, col = lane & 15;
  for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    const int e = expert_of_tile(start, E, tile / nt);
    int first, count;
    rows_of(expert_rows, e, capacity, num_rows, first, count);
    const int64_t te = start[e + 1] - start[e];
    const int64_t local = tile - start[e] * nt;
    const int m0 = static_cast<int>(local % te) * BM, n0 = static_cast<int>(local / te) * BN + wave * 16;
    const int m = m0 + col;
    const size_t row = static_cast<size_t>(first) + min(m, count - 1);
    const uint8_t* ap = a + row * (FP8 ? H : H / 2);
    const uint8_t* as = a_scale + row * (H / 32);
    const size_t wrow = static_cast<size_t>(e) * N + min(n0 + col, O - 1);
    f32x4 acc[GATED ? 2 : 1];
#pragma unroll
    for (auto& c : acc) c = f32x4{0, 0, 0, 0};
    for (int k = 0; k < H; k += 128) {
      i32x8 b = {0, 0, 0, 0, 0, 0, 0, 0}, low, high;
      int sb = 127;
      if constexpr (FP8) {
        *reinterpret_cast<u32x4*>(&b) = *reinterpret_cast<const u32x4*>(ap + k + 16 * grp);
        *(reinterpret_cast<u32x4*>(&b) + 1) = *reinterpret_cast<const u32x4*>(ap + k + 64 + 16 * grp);
        split_codes(b, low, high);
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
          f32x4 d = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(v, low, f32x4{0, 0, 0, 0}, kFp4, kFp8, 0, sw, 0, sb);
          d = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(v, high, d, kFp4, kFp8, 0, sw, 0, sb);
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
// lane): rows into one of two buffers while the other one is multiplied,
// weights into one of two or three, so one or two stages ahead; the copies run
// on over the end of a tile into the next one.  LDS rows are 128 bytes (FP8
// rows 256) and hold their 16-byte pieces permuted (piece ^ swizzle(row)), so
// that the 16 lanes served together meet different banks.  Scales are copied
// 64 bytes a weight row (eight stages) and 32 bytes a token row (four) at a
// time: short pieces of many rows are what a copy costs most.  It is 32 for
// both in the largest tile, which has no registers left (4642 against 4951
// us), and where three stages of 256 weight rows leave no LDS.

__device__ __forceinline__ uint32_t swizzle8(uint32_t row) { return (row & 7) ^ ((row >> 3) & 1); }
__device__ __forceinline__ uint32_t swizzle16(uint32_t row) { return row & 15; }

__device__ __forceinline__ i32x8 widen(u32x4 lo) {
  return i32x8{static_cast<int>(lo[0]), static_cast<int>(lo[1]), static_cast<int>(lo[2]), static_cast<int>(lo[3]),
               0, 0, 0, 0};
}

// An offset past the end of every operand (at most 2^31 bytes of one expert's
// weights, 2^24 of a tile's rows): buffer loads from there give 0.
constexpr uint32_t kNone = 0x80000000u;

// BM x BN: the tile; WM x WN: its waves; WR: stages of weights kept; NT: the
// weights are read non-temporally.
template <bool FP8, bool GATED, int BM, int BN, int WM, int WN, int WR, bool NT>
__global__ __launch_bounds__(WM* WN* kWave) void product_tiled(
    const uint8_t* __restrict__ a, const uint8_t* __restrict__ a_scale, const uint8_t* __restrict__ w,
    const uint8_t* __restrict__ w_scale, const int32_t* __restrict__ expert_rows, int32_t num_rows, int32_t E,
    int32_t capacity, int32_t H, int32_t N, uint16_t* __restrict__ y) {
  constexpr int NW = WM * WN;
  constexpr int TN = BN / WN;                       // a wave's weight rows
  constexpr int FM = BM / WM / 32, FN = TN / 32;    // its fragments of 32 rows
  constexpr int AB = FP8 ? 256 : 128;               // bytes of a token row in a stage
  constexpr int LW = BN / 8 / NW;                   // copies per wave and stage: 8 weight rows each
  constexpr int LA = BM * AB / 1024 / NW;           // 1024 / AB token rows each
  static_assert(LW * 8 * NW == BN && LA * 1024 * NW == BM * AB && FM * 32 * WM == BM && FN * 32 * WN == BN, "tile");
  static_assert(!GATED || FN % 2 == 0, "a wave holds both halves of its channels");
  constexpr int SW = BM > 192 || (WR == 3 && BN > 128) ? 32 : 64;  // bytes of a weight row's scales copied at a time
  constexpr int NQ = SW / 32;                       // quads of stages in SW bytes of a weight row's scales
  constexpr int LSW = BN * SW / 1024 / NW;          // copies per wave for those: 1024 / SW rows each
  constexpr int LSA = (BM / 32 + NW - 1) / NW;      // token rows' scales, a quad's (32 bytes): 32 rows each
  static_assert(LSW * 1024 * NW == BN * SW && BM * AB >= 2048 * NW, "scales, and y's fragments");
  constexpr int BO = GATED ? BN / 2 : BN;           // channels of y per tile
  __shared__ __align__(16) uint8_t w0[BN * 128];
  __shared__ __align__(16) uint8_t w1[BN * 128];
  __shared__ __align__(16) uint8_t w2[WR == 3 ? BN * 128 : 16];
  __shared__ __align__(16) uint8_t a0[BM * AB];
  __shared__ __align__(16) uint8_t a1[BM * AB];
  __shared__ __align__(16) uint8_t scw[BN * SW];
  __shared__ __align__(16) uint8_t sca[BM * 32 + 16];
  const int tid = threadIdx.x, lane = tid & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int half = lane >> 5, col = lane & 31;
  const int wm = wave % WM, wn = wave / WM;
  const int O = GATED ? N / 2 : N;
  const uint32_t nt = (O + BO - 1) / BO;
  const uint32_t wrow_bytes = H / 2, arow_bytes = FP8 ? H : H / 2, srow_bytes = H / 32;
  const int stages = (H + 255) / 256;  // >= 2
  const bool tail = (H & 255) != 0;    // the last stage holds 128 channels

  // Tiles in eight runs, one per XCD (workgroups go to the XCDs in turn), so
  // that neighbouring tiles, which share weights or rows, meet in one L2.
  // Each wavefront finds the first one from sums over E / 64 experts a lane; from
  // there on it walks over the experts.
  const auto row_tiles = [&](int e) -> uint32_t {
    int first, count;
    rows_of(expert_rows, e, capacity, num_rows, first, count);
    return (count + BM - 1) / BM;
  };
  int mine = 0;
  const int per = (E + kWave - 1) / kWave;  // experts of a lane
  for (int i = 0; i < per; i += 4) {
    int n[4];  // (loaded for any lane, so that the four loads overlap)
#pragma unroll
    for (int x = 0; x < 4; ++x) n[x] = row_tiles(min(lane * per + i + x, E - 1));
#pragma unroll
    for (int x = 0; x < 4; ++x) mine += i + x < per && lane * per + i + x < E ? n[x] : 0;
  }
  const int upto = wave_inclusive_scan(mine);
  const uint32_t tiles = static_cast<uint32_t>(__builtin_amdgcn_readlane(upto, kWave - 1)) * nt;
  const uint32_t run = (tiles + 7) / 8, step = gridDim.x / 8;
  const uint32_t end = min((blockIdx.x & 7) * run + run, tiles);
  uint32_t tile = (blockIdx.x & 7) * run + blockIdx.x / 8;
  if (tile >= end) return;
  // the first lane that ends beyond this tile's row tile holds its expert
  const int at = __builtin_ctzll(wave_ballot(static_cast<uint32_t>(upto) > tile / nt));
  uint32_t before = __builtin_amdgcn_readlane(upto - mine, at);  // row tiles before expert `walk`
  int walk = at * per;
  uint32_t te = __builtin_amdgcn_readfirstlane(row_tiles(walk));  // and its own

  // The tile whose stages are being copied: its operands and this lane's
  // pieces.  Rows past the end repeat the last one.
  int n0, rows, row0, m0, first, count;
  Rsrc wr, ar, wsr, asr;
  uint32_t woff[LW], aoff[LA], swoff[LSW], saoff[LSA];
  const auto weight_row = [&](int r0, int r) -> uint32_t {  // r0: wave-uniform, of the same half as r
    const uint32_t n = min(n0 + (GATED && r0 >= BO ? r - BO : r), O - 1);
    return GATED && r0 >= BO ? n + O : n;
  };
  const auto open_weights = [&]() {
    const uint32_t q = tile / nt;
    while (q >= before + te) {  // ends at the expert of tile q
      before += te;
      te = __builtin_amdgcn_readfirstlane(row_tiles(++walk));
    }
    rows_of(expert_rows, walk, capacity, num_rows, first, count);
    const uint32_t local = tile - before * nt;
    m0 = static_cast<int>(local % te) * BM;
    n0 = static_cast<int>(local / te) * BO;
    wr = make_rsrc(w + static_cast<size_t>(walk) * N * wrow_bytes, static_cast<uint32_t>(N) * wrow_bytes);
#pragma unroll
    for (int i = 0; i < LW; ++i) {
      const int r0 = (i * NW + wave) * 8, r = r0 + (lane >> 3);
      woff[i] = weight_row(r0, r) * wrow_bytes + ((lane & 7) ^ swizzle8(r)) * 16;
    }
  };
  const auto open_rows = [&]() {
    rows = __builtin_amdgcn_readfirstlane(min(count - m0, BM));  // >= 1
    row0 = __builtin_amdgcn_readfirstlane(first) + m0;
    ar = make_rsrc(a + static_cast<size_t>(row0) * arow_bytes, static_cast<uint32_t>(rows) * arow_bytes);
    wsr = make_rsrc(w_scale + static_cast<size_t>(walk) * N * srow_bytes, static_cast<uint32_t>(N) * srow_bytes);
    asr = make_rsrc(a_scale + static_cast<size_t>(row0) * srow_bytes, static_cast<uint32_t>(rows) * srow_bytes);
#pragma unroll
    for (int i = 0; i < LA; ++i) {
      const int r = (i * NW + wave) * (1024 / AB) + lane / (AB / 16);
      aoff[i] = min(r, rows - 1) * arow_bytes + (FP8 ? (lane & 15) ^ swizzle16(r) : (lane & 7) ^ swizzle8(r)) * 16;
    }
#pragma unroll
    for (int i = 0; i < LSW; ++i) {
      const int r0 = (i * NW + wave) * (1024 / SW);
      swoff[i] = weight_row(r0, r0 + lane / (SW / 16)) * srow_bytes;
    }
#pragma unroll
    for (int i = 0; i < LSA; ++i) saoff[i] = min((i * NW + wave) * 32 + (lane >> 1), rows - 1) * srow_bytes;
  };
  // A stage's copies.  In a last stage of 128 channels the pieces of the
  // missing half are read past the end of the buffer resource (kNone), which
  // gives zero codes.
  const auto copy_weights = [&](int i, int s, bool none, uint8_t* wb) {
    const int r0 = (i * NW + wave) * 8;
    uint32_t off = woff[i];
    // (no branches here: they would hide from the compiler how many copies are under way)
    const uint32_t cut = tail && s == stages - 1 ? 4 : 0;
    off |= none || (((lane & 7) ^ swizzle8(r0 + (lane >> 3))) & cut) ? kNone : 0;
    if constexpr (NT) copy16_once(wr, wb + r0 * 128, off, s * 128); else copy16(wr, wb + r0 * 128, off, s * 128);
  };
  const auto copy_rows = [&](int s, uint8_t* ab) {
    const bool cut = tail && s == stages - 1;
#pragma unroll
    for (int i = 0; i < LA; ++i) {
      const int r0 = (i * NW + wave) * (1024 / AB), r = r0 + lane / (AB / 16);
      uint32_t off = aoff[i];
      if (cut && (FP8 ? ((lane & 15) ^ swizzle16(r)) & 8 : ((lane & 7) ^ swizzle8(r)) & 4)) off = kNone;
      if (r0 < rows) copy16(ar, ab + r0 * AB, off, s * AB);
    }
  };
  // 16 bytes of scales from 512-channel group g on, or the row's last 16
  const auto scale_at = [&](uint32_t g) { return min(g * 16, srow_bytes - 16); };
  // piece p of weight row r's SW bytes lies at
  const auto scale_place = [](uint32_t r, uint32_t p) {
    return r * SW + ((SW == 64 ? p ^ ((r >> 1) & 3) ^ ((r >> 3) & 1) : p) * 16);
  };
  const auto copy_scales = [&](int quad) {
    if (quad % NQ == 0) {
#pragma unroll
      for (int i = 0; i < LSW; ++i) {
        const int r0 = (i * NW + wave) * (1024 / SW), r = r0 + lane / (SW / 16);
        const uint32_t p = (scale_place(r, lane % (SW / 16)) - r * SW) / 16;  // (its own inverse)
        copy16(wsr, scw + r0 * SW, swoff[i] + scale_at(quad * 2 + p), 0);
      }
    }
    const uint32_t at = scale_at(quad * 2 + (lane & 1));
#pragma unroll
    for (int i = 0; i < LSA; ++i) {
      const int r0 = (i * NW + wave) * 32;
      if (r0 < BM && r0 < rows) copy16(asr, sca + r0 * 32, saoff[i] + at, 0);
    }
  };

  // the wave's fragment i of weight rows, and j of token rows, in the tile
  const auto weight_frag = [&](int i) {
    if (!GATED) return wn * TN + i * 32;
    return i < FN / 2 ? wn * (TN / 2) + i * 32 : BO + wn * (TN / 2) + (i - FN / 2) * 32;
  };
  const auto row_frag = [&](int j) { return (j * WM + wm) * 32; };  // in turn, so that short tiles keep all waves busy

  f32x16 acc[FN][FM];
  uint32_t sw[FN][4], sa[FM][4];  // scales of a pair of stages: one 32-bit word per 128 channels
  const auto read_scales = [&](int pair) {
    // A row that is no multiple of 512 channels ends inside a pair: its last 16
    // bytes were copied, and the missing words, for zero codes, are a scale of 1.
    const int skip = (pair * 16 - static_cast<int>(scale_at(pair))) / 4;
    const auto read4 = [&](const u32x4 q, uint32_t one, uint32_t(&v)[4]) {
      if (skip == 0) {
#pragma unroll
        for (int x = 0; x < 4; ++x) v[x] = q[x];
      } else {
        const uint32_t q1 = q[1], q2 = q[2], q3 = q[3];
        v[0] = skip == 1 ? q1 : (skip == 2 ? q2 : q3);
        v[1] = skip == 1 ? q2 : (skip == 2 ? q3 : one);
        v[2] = skip == 1 ? q3 : one;
        v[3] = one;
      }
    };
#pragma unroll
    for (int i = 0; i < FN; ++i) {
      read4(*reinterpret_cast<const u32x4*>(scw + scale_place(weight_frag(i) + col, pair % (2 * NQ))), 0x7F7F7F7Fu, sw[i]);
#pragma unroll
      for (int x = 0; x < 4; ++x) sw[i][x] >>= 8 * half;
    }
#pragma unroll
    for (int j = 0; j < FM; ++j) {
      read4(*reinterpret_cast<const u32x4*>(sca + ((row_frag(j) + col) * 32 + (pair & 1) * 16)), FP8 ? 0x3F800000u : 0x7F7F7F7Fu, sa[j]);
#pragma unroll
      for (int x = 0; x < 4; ++x) sa[j][x] >>= FP8 ? 0 : 8 * half;
    }
  };

  const auto weight_piece = [&](int ks, int i, const uint8_t* wb) {
    return widen(*reinterpret_cast<const u32x4*>(
        wb + ((weight_frag(i) + col) * 128 + (((ks * 2 + half) ^ swizzle8(col)) * 16))));
  };
  const auto token_piece = [&](int ks, int j, const uint8_t* ab) {
    const uint32_t r = row_frag(j) + col;
    if constexpr (FP8) {
      // this half-wave's 32 channels of a 64-channel step: 16 of each 32
      const uint32_t p = ks * 4 + half;
      const u32x4 lo4 = *reinterpret_cast<const u32x4*>(ab + (r * 256 + ((p ^ swizzle16(col)) * 16)));
      const u32x4 hi4 = *reinterpret_cast<const u32x4*>(ab + (r * 256 + (((p + 2) ^ swizzle16(col)) * 16)));
      return i32x8{static_cast<int>(lo4[0]), static_cast<int>(lo4[1]), static_cast<int>(lo4[2]), static_cast<int>(lo4[3]),
                   static_cast<int>(hi4[0]), static_cast<int>(hi4[1]), static_cast<int>(hi4[2]), static_cast<int>(hi4[3])};
    } else {
      return widen(*reinterpret_cast<const u32x4*>(ab + (r * 128 + (((ks * 2 + half) ^ swizzle8(col)) * 16))));
    }
  };
  // A stage's products: four steps of 64 channels times FM row fragments, in
  // an order that keeps an FP8 fragment's two steps of one scale together;
  // each is read two places ahead of its use.
  constexpr int U = 4 * FM;
  const auto step_of = [](int u) { return FP8 ? u / (2 * FM) * 2 + u % 2 : u / FM; };
  const auto frag_of = [](int u) { return FP8 ? u / 2 % FM : u % FM; };
  const auto multiply = [&](auto xc, const uint8_t* wb, const uint8_t* ab) {
    constexpr int X = decltype(xc)::value;  // first word of the stage's scales
    i32x8 wv[4][FN], av[U];
#pragma unroll
    for (int i = 0; i < FN; ++i) wv[0][i] = weight_piece(0, i, wb);
    av[0] = token_piece(0, 0, ab);
    if constexpr (FP8) {
#pragma unroll
      for (int i = 0; i < FN; ++i) wv[1][i] = weight_piece(1, i, wb);
    }
    av[1] = token_piece(step_of(1), frag_of(1), ab);
    f32x16 d[FN];
    i32x8 lowv[U], highv[U];
    // The next place's split goes under this one's products (64 x 256, 4096
    // tokens: 2174 against 2236 us); with two row fragments it would spill.
    constexpr bool kAhead = FP8 && FM == 1;
    if constexpr (kAhead) split_codes(av[0], lowv[0], highv[0]);
    static_for<0, U>([&](auto uc) {
      constexpr int u = decltype(uc)::value;
      constexpr int ks = step_of(u), j = frag_of(u);
      if constexpr (u + 2 < U) {
        av[u + 2] = token_piece(step_of(u + 2), frag_of(u + 2), ab);
      }
      // the next step's weights (FP8: the next two steps')
      if constexpr (!FP8 && u % FM == 0 && ks < 3) {
#pragma unroll
        for (int i = 0; i < FN; ++i) wv[ks + 1][i] = weight_piece(ks + 1, i, wb);
      }
      if constexpr (FP8 && u == FM) {
#pragma unroll
        for (int i = 0; i < FN; ++i) {
          wv[2][i] = weight_piece(2, i, wb);
          wv[3][i] = weight_piece(3, i, wb);
        }
      }
      __builtin_amdgcn_sched_barrier(0);
      constexpr int sel = ks % 2 * 2;
      if constexpr (FP8) {
        if constexpr (!kAhead) split_codes(av[u], lowv[u], highv[u]);
        else if constexpr (u + 1 < U) split_codes(av[u + 1], lowv[u + 1], highv[u + 1]);
        const i32x8 low = lowv[u], high = highv[u];
#pragma unroll
        for (int i = 0; i < FN; ++i) {
          if (ks % 2 == 0) {
#pragma unroll
            for (int r = 0; r < 16; ++r) d[i][r] = 0.0f;
          }
          d[i] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(wv[ks][i], low, d[i], kFp4, kFp8, sel,
                                                                 static_cast<int>(sw[i][X + ks / 2]), 0, 127);
        }
#pragma unroll
        for (int i = 0; i < FN; ++i)
          d[i] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(wv[ks][i], high, d[i], kFp4, kFp8, sel,
                                                                 static_cast<int>(sw[i][X + ks / 2]), 0, 127);
        if constexpr (kAhead && u + 1 < U) {  // one product, then its share of the next split's vector work, and so on
#pragma unroll
          for (int i = 0; i < 2 * FN; ++i) {
            __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);
            __builtin_amdgcn_sched_group_barrier(0x2, 40 / (2 * FN), 0);
          }
        }
        if constexpr (ks % 2 == 1) {
          const float f = __uint_as_float(sa[j][X + ks / 2]);
#pragma unroll
          for (int i = 0; i < FN; ++i)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[i][j][r] = __builtin_fmaf(f, d[i][r], acc[i][j][r]);
        }
      } else {
#pragma unroll
        for (int i = 0; i < FN; ++i)
          acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(wv[ks][i], av[u], acc[i][j], kFp4, kFp4, sel,
                                                                     static_cast<int>(sw[i][X + ks / 2]), sel,
                                                                     static_cast<int>(sa[j][X + ks / 2]));
      }
    });
  };

  // A tile's stages, and none or more without products that make them a
  // multiple of WR, so that each tile starts with the same buffers.
  const int padded = (stages + WR - 1) / WR * WR;
  const auto start_rows = [&]() {
    open_rows();
    copy_scales(0);
    copy_rows(0, a0);
  };
  open_weights();
  start_rows();
#pragma unroll
  for (int x = 0; x < WR - 1; ++x) {
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < LW; ++i) copy_weights(i, x, false, x == 0 ? w0 : w1);
  }
  for (;;) {
    const int c_n0 = n0, c_rows = rows, c_row0 = row0;  // the tile being multiplied
    bool last = false, early = false;
#pragma unroll
    for (int i = 0; i < FN; ++i)
#pragma unroll
      for (int j = 0; j < FM; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;
    const bool live = wm * 32 < c_rows;  // else this wave's rows are all past the end
    const auto stage = [&](int st, auto pc) {
      constexpr int P = decltype(pc)::value, X = P % 4, PW = P % WR, PN = (P + WR - 1) % WR;
      const uint8_t* wb = PW == 0 ? w0 : (PW == 1 ? w1 : w2);
      uint8_t* wnext = PN == 0 ? w0 : (PN == 1 ? w1 : w2);
      const uint8_t* ab = P % 2 == 0 ? a0 : a1;
      uint8_t* anext = P % 2 == 0 ? a1 : a0;
      // all has arrived but (WR 3) the next stage's weights, which were copied last
      wait_and_sync<(WR - 2) * LW>();
      if (X % 2 == 0 && st < stages) read_scales(st >> 1);
      if (P % WR == 1 && st + WR - 1 == padded) {  // from here on the weights are the next tile's
        tile += step;
        last = tile >= end;
        if (!last) open_weights();
      }
      if (st + 1 < stages) {
        if (X == 3) copy_scales((st >> 2) + 1);
        copy_rows(st + 1, anext);
      } else if (P % WR == WR - 1 && X % 2 == 1 && st + 1 == padded && !last) {  // nothing reads a0 and the scales now
        early = true;
        start_rows();
      }
      __builtin_amdgcn_sched_barrier(0);
      asm volatile("" ::: "memory");  // the weights are the last ones: the wait above counts on it
      int s = st + WR - 1;
      bool none = s >= stages;
      if (s >= padded) {
        s -= padded;
        none = last;
      }
#pragma unroll
      for (int i = 0; i < LW; ++i) copy_weights(i, s, none, wnext);
      __builtin_amdgcn_sched_barrier(0);
      if (live && st < stages) multiply(std::integral_constant<int, X % 2 * 2>{}, wb, ab);
    };
    constexpr int kRing = WR == 3 ? 12 : 4;  // stages after which buffers and scales repeat
    // (leaving the loop inside a round, not passing over the stages left of it:
    // the compiler follows the copies under way along every path)
    for (int first = 0;; first += kRing)
      if (!static_while<0, kRing>([&](auto pc) {
            constexpr int P = decltype(pc)::value;
            stage(first + P, pc);
            return (P + 1) % WR != 0 || first + P + 1 < padded;
          }))
        break;

    // y: a fragment's 32 rows of 32 channels go through LDS, so that four lanes
    // store 64 bytes of a row (from the accumulators' layout it would be 16).
    // a1 is free: nothing is copied there before the next tile's first barrier.
    wait_reads();
    uint8_t* const yb = a1 + wave * 2048;
    // 16-byte piece p of the fragment's row r lies at
    const auto y_place = [](uint32_t r, uint32_t p) { return r * 64 + (p ^ ((r >> 2) & 3)) * 16; };
#pragma unroll
    for (int j = 0; j < FM; ++j)
#pragma unroll
      for (int i = 0; i < (GATED ? FN / 2 : FN); ++i) {
        if (row_frag(j) >= c_rows) continue;
#pragma unroll
        for (int r4 = 0; r4 < 4; ++r4) {
          __bf16 o[4];
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const float v = acc[i][j][4 * r4 + x];
            o[x] = static_cast<__bf16>(GATED ? silu_mul(v, acc[GATED ? i + FN / 2 : i][j][4 * r4 + x]) : v);
          }
          *reinterpret_cast<uint2*>(yb + (y_place(col, r4) + half * 8)) = *reinterpret_cast<uint2*>(o);
        }
        asm volatile("" ::: "memory");
        const int n = c_n0 + weight_frag(i) + (lane & 3) * 8;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int r = x * 16 + (lane >> 2), m = row_frag(j) + r;
          const u32x4 v = *reinterpret_cast<const u32x4*>(yb + y_place(r, lane & 3));
          if (m < c_rows && n < O) *reinterpret_cast<u32x4*>(y + static_cast<size_t>(c_row0 + m) * O + n) = v;
        }
        asm volatile("" ::: "memory");
      }
    if (last) break;
    if (!early) {
      start_rows();
      __builtin_amdgcn_s_waitcnt(15 << 8 | 7 << 4);  // vmcnt(0): the first wait counts on the weights being last
    }
  }
  __builtin_amdgcn_s_waitcnt(15 << 8 | 7 << 4);  // vmcnt(0): no copy outlives the workgroup's LDS
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
    // rows too short for 16-byte pieces of scales
    if (H < 512) return with(product_kernel<F, G>, 2048, kThreads);
    // Tile by the mean rows of an expert (the padded layout tells nothing about
    // them: as for few).  Few rows: the weights' stream decides, and small
    // workgroups keep it up, two on a CU; many rows: tiles that reuse what they
    // read, one workgroup on a CU.  Measured with E 256, H 7168, N 4096 gated
    // (down: 4096 tokens, H 2048, N 7168), rows spread evenly, in microseconds;
    // x3: three stages of weights are kept, else two; * as the rule picks:
    //   tokens                1   128   512  1024  2048  4096  8192  32768  down
    //   MXFP4 rows
    //   64 x 128 x3         *23  *548  *577  *653  1073  1661  3016  11824   881
    //   64 x 128             33   587   621   701  1109  1648  2886  11833   898
    //   128 x 128            35   607   636   728  *821  1286  1923   7078   731
    //   192 x 256 x3         39   661   673   765   866  *945  1925   5207  *525
    //   192 x 256            44   699   730   813   888   970  2000   5358   523
    //   256 x 256            47   808   837   918  1038  1121 *1777  *4637   622
    //   FP8 rows
    //   64 x 128            *42  *702  *739   942  1465  2476  4710  17683  1250
    //   64 x 128 x3          42  1108  1130  1147  1742  2889  5194  19204  1537
    //   64 x 256 x3          53   783   813  *912 *1392 *2189 *3957  14654 *1140
    //   128 x 256            93  1436  1455  1472  1673  2510  3975 *13884  1315
    // (64 x 128 x3 of FP8 rows: one workgroup fits a CU.)
    // Weights of an expert with one row tile are read once and non-temporally
    // (576 against 595 at 128 tokens); where more row tiles read them, that
    // would keep them out of L2 (192 x 256 at 32768 tokens: 5419 against 4922).
    // Two or three row tiles do not mind, though more is read (64 x 256, FP8
    // rows, 4096 tokens: 4.7 GB for 3.9 of weights).
    const int64_t avg = capacity > 0 ? 0 : num_rows / E;
    if constexpr (F) {
      if (avg <= 16) return with(product_tiled<F, G, 64, 128, 2, 2, 2, true>, 512, 256);
      if (avg <= 320) return with(product_tiled<F, G, 64, 256, 2, 4, 3, true>, 256, 512);
      return with(product_tiled<F, G, 128, 256, 2, 4, 2, false>, 256, 512);
    } else {
      if (avg <= 32) return with(product_tiled<F, G, 64, 128, 2, 2, 3, true>, 512, 256);
      if (avg <= 64) return with(product_tiled<F, G, 128, 128, 2, 2, 2, true>, 512, 256);
      if (avg <= 170) return with(product_tiled<F, G, 192, 256, 2, 4, 3, true>, 256, 512);
      return with(product_tiled<F, G, 256, 256, 2, 4, 2, false>, 256, 512);
    }
  };
  if (fp8) return gated ? pick(std::true_type{}, std::true_type{}) : pick(std::true_type{}, std::false_type{});
  return gated ? pick(std::false_type{}, std::true_type{}) : pick(std::false_type{}, std::false_type{});
}

}  // namespace ep
