// The tiled product of the experts' bf16 layers (internal header): forward,
// the rows' gradient and the weights' gradient are one kernel, whose operands
// lie differently in memory.
//
// A tile of the result is BM rows x BN channels.  Its channels' operand (X) is
// the MFMA's A operand, its rows' (R) the B operand; both pass through LDS in
// stages of 64 summed elements, copied straight from global memory some stages
// ahead.
//
//            result            X                          R            summed over
//   kForward y [row][n]        w [n][h], along h          a [row][h]   h
//   kRows    grad_a [row][h]   w [n][h], across n         g [row][n]   n
//   kWeights grad_w [n][h]     a [row][h], across rows    g [row][n]   an expert's rows
//
// An operand whose rows run along the summed index lies in LDS as rows of 128
// bytes and is read 16 bytes (eight elements) a lane.  One that runs across
// it lies as 64 rows of BN (BM) elements and is read through gfx950's
// transposing LDS load: sixteen lanes read four rows of sixteen elements, and
// each gets the four of its column.  Both kinds hold their 16-byte pieces
// permuted, so that lanes served together meet different banks (counted: 1 to 6
// conflicts in 100 LDS cycles).
//
// Sums are binary32: the bf16 MFMA keeps them (products exact, a term 2^-23 below
// the sum counts in full, subnormals kept), and every result is rounded once.
//
// What bounds it: 8192^3 takes 803 to 840 us in all three kinds (1310 to 1370
// TFLOP/s; the matrix unit is busy 84% of the time, at 1.4 GHz: the card's power
// limit).  With 256 experts of 7168 to 4096 (gated) the weights stream in at 7.1
// TB/s where an expert has few rows; at 128 rows an expert both bounds meet (5.3
// TB/s, 650 TFLOP/s, 1.4 to 1.5 GHz); at 1024 rows 1100 to 1200 TFLOP/s (by the card).  Measured without gain:
// half a tile's products where an expert's last rows fit that (3% at 128 rows, but
// tiles that drift apart lose their shared lines in L2: 14.6 against 13.0 ms at 1024
// rows), four waves of 128 x 128, all of a stage's fragments read at once,
// non-temporal stores of the result.
#pragma once

#include "ep_internal.h"
#include "expert_device.h"

namespace ep {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef float f32x8 __attribute__((ext_vector_type(8)));

enum Kind { kForward, kRows, kWeights };

struct LinearArgs {
  const __bf16* x;         // w (kForward, kRows) or a
  const __bf16* r;         // a, or the output's gradient
  const __bf16* bias;      // or null (kForward)
  const __bf16* residual;  // or null (kForward); may be y
  const int32_t* expert_rows;
  int32_t num_rows, E, capacity;
  int32_t C;  // summed channels (not kWeights)
  int32_t O;  // channels of the result (kForward gated: of y; kRows gated: of d)
  int32_t M;  // rows of the result of one expert (kWeights: out channels)
  bool add;   // kWeights: add to what is there
  __bf16* p;  // kForward gated: out or null; kRows gated: in, may be y
  void* y;
  void* sums;  // kWeights: sums of r's columns (the biases' gradient) out, or null
};

// A value that is the same in every lane, kept where the compiler knows it (a
// branch on anything else is taken for one that lanes take apart, and then the
// copies of both its sides are waited for).
__device__ __forceinline__ int64_t uniform(int64_t v) {
  const uint32_t lo = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(v));
  const uint32_t hi = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(v >> 32));
  return static_cast<int64_t>(static_cast<uint64_t>(hi) << 32 | lo);
}
template <typename T>
__device__ __forceinline__ T* uniform(T* p) {
  return reinterpret_cast<T*>(uniform(reinterpret_cast<int64_t>(p)));
}

// Rows of expert e; without expert_rows every row is expert 0's.
__device__ __forceinline__ void span_of(const int32_t* __restrict__ expert_rows, int e, int capacity, int num_rows,
                                        int& first, int& count) {
  if (expert_rows == nullptr) {
    first = 0;
    count = num_rows;
  } else {
    rows_of(expert_rows, e, capacity, num_rows, first, count);
  }
}

// The same for an expert that is one for the wavefront, through the scalar cache:
// a load that the copies under way are not waited for with.
__device__ __forceinline__ void span_of_one(const int32_t* expert_rows, int e, int capacity, int num_rows, int& first,
                                            int& count) {
  typedef __attribute__((address_space(4))) const int32_t Constant;
  Constant* rows = (Constant*)(uintptr_t)uniform(expert_rows);
  e = __builtin_amdgcn_readfirstlane(e);
  if (expert_rows == nullptr) {
    first = 0;
    count = num_rows;
  } else if (capacity > 0) {
    first = e * capacity;
    count = min(max(rows[e], 0), capacity);
  } else {
    span_rows(rows[e], rows[e + 1], num_rows, first, count);
  }
}

// The gate's sigmoid s = 1 / (1 + exp(-g)) as two factors s1 s2, and n = 1 - s,
// each without cancellation.  (Two, each with half the exponent, so that s
// keeps its accuracy below 2^-126, where a large u or d makes it count: to g =
// -174, where each factor ends.)
struct Gate {
  float s1, s2, n;
};
__device__ __forceinline__ Gate gate(float g) {
  const float h = __expf(-0.5f * __builtin_fabsf(g)), e = h * h;
  const float r = __builtin_amdgcn_rcpf(1.0f + e);
  const bool low = g < 0.0f;
  return Gate{low ? h : 1.0f, low ? h * r : r, low ? r : e * r};
}
__device__ __forceinline__ float silu_times(float g, float u) {
  const Gate k = gate(g);
  return (g * k.s1) * (u * k.s2);
}

// Until at most N of this wave's copies are under way (they finish in order)
// and its LDS reads are done; then the workgroup's barrier.
template <int N>
__device__ __forceinline__ void wait_copies() {
  static_assert(N < 64, "vmcnt");
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt((N & 15) | 7 << 4 | (N >> 4) << 14);  // vmcnt(N) lgkmcnt(0)
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// 16-byte pieces of 128-byte rows: eight rows, and the eight beyond, differ.
__device__ __forceinline__ uint32_t along_swizzle(uint32_t row) { return (row & 7) ^ ((row >> 3) & 1); }
// Pairs of pieces of the rows that a transposing load reads together.
__device__ __forceinline__ uint32_t across_swizzle(uint32_t k) { return ((k & 3) | (k & 1) << 2) * 2; }

template <bool ONCE>
__device__ __forceinline__ void copy_piece(Rsrc src, uint8_t* dst, uint32_t lane_off, uint32_t off) {
  if constexpr (ONCE) copy16_once(src, dst, lane_off, off);
  else copy16(src, dst, lane_off, off);
}

// A lane offset past the end of every buffer resource: loads from there give 0,
// and stores are dropped.  Needs resources of at most 2^31 bytes, and offsets added
// to it of less.  Here a tile's rows reach 2^26 bytes (256 rows of 2 x 65536 bf16
// channels of p, or of 65536 binary32 gradients), linear_few's matrix of one expert
// nearly 2^31.
constexpr uint32_t kNone = 0x80000000u;

// WM x WN: the tile's waves; XS, RS: stages of X and of R kept; PER: workgroups
// of a CU; ONCE: X is read non-temporally; G: groups of WM x WN waves, each with
// buffers of its own, that take a part of the summed channels each (where there are
// fewer tiles than CUs: a stage's waits then serve G of them).
template <Kind KIND, bool GATED, typename T, int BM, int BN, int WM, int WN, int XS, int RS, int PER, bool ONCE, int G>
__global__ __launch_bounds__(G* WM* WN* kWave, (G * WM * WN * PER + 3) / 4) void linear_tiled(const LinearArgs g) {
  constexpr int NW = WM * WN;
  constexpr bool kPair = KIND == kForward && GATED;  // X holds gate and up rows of the same BO channels
  constexpr bool kXAlong = KIND == kForward, kRAlong = KIND != kWeights;
  constexpr int BO = kPair ? BN / 2 : BN;
  constexpr int TN = BN / WN, FN = TN / 32, FM = BM / WM / 32;  // fragments of 32
  constexpr int LX = BN / 8 / NW, LR = BM / 8 / NW;             // copies per wave and stage, 1 KB each
  static_assert(LX * 8 * NW == BN && LR * 8 * NW == BM && FM * 32 * WM == BM && FN * 32 * WN == BN && NW % 2 == 0, "tile");
  static_assert(!kPair || (FN % 2 == 0 && LX % 2 == 0), "a wave holds, and copies, both halves of its channels");
  static_assert((kXAlong || BN >= 128) && (kRAlong || BM >= 128), "across_swizzle permutes 16 pieces");
  static_assert(BN * 128 >= NW * 4096, "y's fragments");
  static_assert(KIND != kWeights || NW * kWave >= BM, "a lane for each column's sum");
  static_assert(XS == RS || XS == RS + 1, "the order of the copies");
  constexpr int kRing = XS == RS ? XS : XS * RS;  // stages after which the buffers repeat
  static_assert(XS <= 6 && RS <= 6, "buffers");
  static_assert(G == 1 || KIND != kWeights, "the column sums are one group's");
#define EP_BUFFER(name, i, n, rows) __shared__ __align__(16) uint8_t name##i[(n) > i ? G * (rows) * 128 : 16]
  EP_BUFFER(x, 0, XS, BN);  // (arrays of their own: the compiler tells copies into one from reads of another)
  EP_BUFFER(x, 1, XS, BN);
  EP_BUFFER(x, 2, XS, BN);
  EP_BUFFER(x, 3, XS, BN);
  EP_BUFFER(x, 4, XS, BN);
  EP_BUFFER(x, 5, XS, BN);
  EP_BUFFER(r, 0, RS, BM);
  EP_BUFFER(r, 1, RS, BM);
  EP_BUFFER(r, 2, RS, BM);
  EP_BUFFER(r, 3, RS, BM);
  EP_BUFFER(r, 4, RS, BM);
  EP_BUFFER(r, 5, RS, BM);
#undef EP_BUFFER
  const int tid = threadIdx.x, lane = tid & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave) % NW;  // of its group
  const int group = G == 1 ? 0 : __builtin_amdgcn_readfirstlane(tid / kWave) / NW;
  const auto x_buf = [&](auto qc) -> uint8_t* {
    constexpr int q = decltype(qc)::value % XS;
    const int mine = group * BN * 128;
    if constexpr (q == 0) return x0 + mine;
    else if constexpr (q == 1) return x1 + mine;
    else if constexpr (q == 2) return x2 + mine;
    else if constexpr (q == 3) return x3 + mine;
    else if constexpr (q == 4) return x4 + mine;
    else return x5 + mine;
  };
  const auto r_buf = [&](auto qc) -> uint8_t* {
    constexpr int q = decltype(qc)::value % RS;
    const int mine = group * BM * 128;
    if constexpr (q == 0) return r0 + mine;
    else if constexpr (q == 1) return r1 + mine;
    else if constexpr (q == 2) return r2 + mine;
    else if constexpr (q == 3) return r3 + mine;
    else if constexpr (q == 4) return r4 + mine;
    else return r5 + mine;
  };
  const int half = lane >> 5, col = lane & 31;
  const int wm = wave % WM, wn = wave / WM;
  const int O = g.O;
  const uint32_t nt = (O + BO - 1) / BO;
  const int E = g.E;

  // ---- tiles ----
  // Neighbouring tiles share weights or rows, and are to meet in one XCD's L2
  // (workgroups go to the XCDs in turn).  They are dealt out in turns of one a
  // workgroup, 32 of an XCD next to one another; or, where few rows an expert make
  // all of them streams of weights, in eight runs, one per XCD (128 tokens, 8 of 256
  // experts: 2191 against 2227 us; but 4096 tokens with popular experts, whose
  // tiles differ: 4028 against 3825).
  // kForward, kRows: the row tiles of each expert times nt; each wavefront finds
  // its first one from sums over E / 64 experts a lane, and walks on from there.
  constexpr bool kRuns = KIND != kWeights && BM <= 128;
  // kWeights: every expert has the same tiles, but sums of its own length.  The
  // experts go by falling length, and every other turn is dealt backwards, so that
  // no workgroup is left with a long sum at the end (32 experts, popular ones: 1309
  // against 1349 us).  order: this lane's experts in that order, the 64 i-th on,
  // two in a register.
  uint32_t order[KIND == kWeights ? kMaxExperts / kWave / 2 : 1];
  if constexpr (KIND == kWeights) {
    int32_t* const counts = reinterpret_cast<int32_t*>(x0);
    uint16_t* const sorted = reinterpret_cast<uint16_t*>(x0 + kMaxExperts * 4);
    static_assert(BN * 128 >= kMaxExperts * 6, "the experts' order");
    for (int e = tid; e < E; e += NW * kWave) {
      int first, count;
      span_of(g.expert_rows, e, g.capacity, g.num_rows, first, count);
      counts[e] = count;
    }
    __syncthreads();
    for (int e = tid; e < E; e += NW * kWave) {
      const int mine = counts[e];
      int rank = 0;
      for (int o = 0; o < E; ++o) rank += counts[o] > mine || (counts[o] == mine && o < e);
      sorted[rank] = static_cast<uint16_t>(e);
    }
    __syncthreads();
    static_for<0, kMaxExperts / kWave / 2>([&](auto ic) {
      const int lo = 128 * decltype(ic)::value + lane, hi = lo + 64;
      order[decltype(ic)::value] = (lo < E ? sorted[lo] : 0) | static_cast<uint32_t>(hi < E ? sorted[hi] : 0) << 16;
    });
    __syncthreads();
  }
  const auto expert_at = [&](uint32_t rank) -> int {
    uint32_t pair = 0;  // (added up: chosen from, the registers would go to scratch memory)
    static_for<0, KIND == kWeights ? kMaxExperts / kWave / 2 : 1>([&](auto ic) {
      pair |= rank / 128 == decltype(ic)::value ? order[decltype(ic)::value] : 0;
    });
    pair = __builtin_amdgcn_readlane(pair, rank % 64);
    return rank & 64 ? pair >> 16 : pair & 0xFFFF;
  };
  const auto row_tiles = [&](int e) -> uint32_t {
    int first, count;
    span_of(g.expert_rows, e, g.capacity, g.num_rows, first, count);
    return (static_cast<uint32_t>(count) + BM - 1) / BM;
  };
  const auto row_tiles_of_one = [&](int e) -> uint32_t {
    int first, count;
    span_of_one(g.expert_rows, e, g.capacity, g.num_rows, first, count);
    return (static_cast<uint32_t>(count) + BM - 1) / BM;
  };
  uint32_t tile, end, step, te = 0;
  uint32_t before = 0;  // row tiles before expert `walk`
  int walk = 0;
  if constexpr (KIND == kWeights) {
    te = (g.M + BM - 1) / BM;
    end = te * nt * E;  // at most 2^9 * 2^9 * 2^10
    step = gridDim.x;
    tile = (blockIdx.x & 7) * (gridDim.x / 8) + blockIdx.x / 8;
    if (tile >= end) return;
  } else {
    uint32_t mine = 0, upto = 0, total, high = 0;
    const int per = (E + kWave - 1) / kWave;  // experts of a lane
    if (g.expert_rows == nullptr) {
      total = te = row_tiles_of_one(0);
    } else {
      for (int i = 0; i < per; i += 4) {
        uint32_t n[4];  // (loaded for any lane, so that the four loads overlap)
#pragma unroll
        for (int x = 0; x < 4; ++x) n[x] = row_tiles(min(lane * per + i + x, E - 1));
#pragma unroll
        for (int x = 0; x < 4; ++x) mine += i + x < per && lane * per + i + x < E ? n[x] : 0;
      }
      upto = wave_inclusive_scan(mine);
      total = __builtin_amdgcn_readlane(upto, kWave - 1);
      high = __builtin_amdgcn_readlane(wave_inclusive_scan(mine >> 16), kWave - 1);
    }
    const uint32_t tiles = tiles_or_none(total, high, nt);
    if constexpr (kRuns) {
      const uint32_t run = (tiles + 7) / 8;
      step = gridDim.x / 8;
      end = min((blockIdx.x & 7) * run + run, tiles);
      tile = (blockIdx.x & 7) * run + blockIdx.x / 8;
    } else {
      end = tiles;
      step = gridDim.x;
      tile = (blockIdx.x & 7) * (gridDim.x / 8) + blockIdx.x / 8;
    }
    if (tile >= end) return;
    if (g.expert_rows != nullptr) {
      // the first lane that ends beyond this tile's row tile holds its expert
      const int at = __builtin_ctzll(wave_ballot(upto > tile / nt));
      before = __builtin_amdgcn_readlane(upto - mine, at);
      walk = at * per;
      te = row_tiles_of_one(walk);
    }
  }

  // ---- the tile whose stages are being copied ----
  struct Place {
    int e, first, count, m0, n0;  // expert, its rows, the tile's first row and channel
  } at;
  // An expert's tiles go in bands of eight row tiles, channel by channel, so that
  // the 32 workgroups of an XCD read 8 + 4 operands' tiles at a time, not 32 + 1
  // (8192^3: 870 against 1009 us).
  const auto place = [&](uint32_t local) {
    const uint32_t band = local / (8 * nt), rest = local - band * 8 * nt, width = min(te - band * 8, 8u);
    at.m0 = static_cast<int>(band * 8 + rest % width) * BM;
    at.n0 = static_cast<int>(rest / width) * BO;
  };
  const auto open_tile = [&]() {
    if constexpr (KIND == kWeights) {
      const uint32_t each = te * nt, turn = tile / gridDim.x;
      // (not the last, incomplete turn)
      const uint32_t q = (turn & 1) != 0 && (turn + 1) * gridDim.x <= end ? (2 * turn + 1) * gridDim.x - 1 - tile : tile;
      const uint32_t rank = q / each;
      at.e = expert_at(rank);
      place(q - rank * each);
    } else {
      const uint32_t q = tile / nt;
      while (q >= before + te) {  // ends at the expert of tile q
        before += te;
        te = row_tiles_of_one(++walk);
      }
      at.e = walk;
      const uint32_t local = tile - before * nt;
      place(local);
    }
    span_of_one(g.expert_rows, at.e, g.capacity, g.num_rows, at.first, at.count);
  };
  const auto stages_of = [&](const Place& t) { return stages_of_sum(KIND == kWeights ? t.count : g.C); };  // of all groups
  const auto share = [&](int stages) { return G == 1 ? stages : (stages + G - 1) / G; };
  const int ahead = G == 1 ? 0 : group * share(stages_of_sum(g.C));  // stages of the groups before
  const auto rows_in = [&](const Place& t) { return min((KIND == kWeights ? g.M : t.count) - t.m0, BM); };

  // An operand's copies.  Along: piece (lane & 7) of row lane / 8 of eight, and
  // the last stage's pieces past the end are read past the end of the buffer
  // resource (kNone), which gives zeros.  Across: a stage is a buffer resource of
  // its own, which ends with its last row.
  const uint32_t along_piece = (lane & 7) ^ along_swizzle((wave & 1) * 8 + (lane >> 3));
  const bool along_cut = ((g.C - 1) / 64) * 64 + along_piece * 8 >= static_cast<uint32_t>(g.C);
  const __bf16 *xbase, *rbase;  // the tile's first element
  Rsrc xr, xr2, rr;
  uint32_t xoff[LX], roff[LR];
  int x_stages = 0, r_stages = 0, x_left = 0, r_left = 0;
  uint32_t x_bytes = 0, r_bytes = 0;  // across: bytes of a row, and (_cols) before the tile's first element
  uint32_t x_cols = 0, r_cols = 0;
  const auto across_off = [&](int i, int width, uint32_t row_bytes, int valid) -> uint32_t {
    const uint32_t k = (i * NW + wave) * (512 / width) + lane / (width / 8);
    const uint32_t piece = (lane % (width / 8)) ^ across_swizzle(k);
    return static_cast<int>(piece * 8) < valid ? k * row_bytes + piece * 16 : kNone;
  };
  const auto open_x = [&]() {
    x_stages = stages_of(at);
    const int valid = min(O - at.n0, BO);
    if constexpr (kXAlong) {
      const __bf16* we = g.x + (static_cast<size_t>(at.e) * (kPair ? 2 * O : O) + at.n0) * g.C;
      const uint32_t bytes = static_cast<uint32_t>(g.C) * 2;
      xr = make_rsrc(uniform(we), valid * bytes);
      if constexpr (kPair) xr2 = make_rsrc(uniform(we + static_cast<size_t>(O) * g.C), valid * bytes);
#pragma unroll
      for (int i = 0; i < LX; ++i) {
        const int r = ((kPair ? i % (LX / 2) : i) * NW + wave) * 8 + (lane >> 3);
        xoff[i] = r < valid ? r * bytes + along_piece * 16 : kNone;
      }
    } else {
      x_bytes = static_cast<uint32_t>(O) * 2;
      x_cols = at.n0 * 2;
      x_left = KIND == kWeights ? at.count : g.C;
      xbase = uniform(g.x + (KIND == kWeights ? static_cast<size_t>(at.first) : static_cast<size_t>(at.e) * g.C) * O + at.n0);
#pragma unroll
      for (int i = 0; i < LX; ++i) xoff[i] = across_off(i, BN, x_bytes, valid);
    }
  };
  const auto open_r = [&]() {
    r_stages = stages_of(at);
    const int valid = rows_in(at);
    if constexpr (kRAlong) {
      const uint32_t bytes = static_cast<uint32_t>(g.C) * 2;
      rr = make_rsrc(uniform(g.r + (static_cast<size_t>(at.first) + at.m0) * g.C), valid * bytes);
#pragma unroll
      for (int i = 0; i < LR; ++i) {
        const int r = (i * NW + wave) * 8 + (lane >> 3);
        roff[i] = r < valid ? r * bytes + along_piece * 16 : kNone;
      }
    } else {
      r_bytes = static_cast<uint32_t>(g.M) * 2;
      r_cols = at.m0 * 2;
      r_left = at.count;
      rbase = uniform(g.r + static_cast<size_t>(at.first) * g.M + at.m0);
#pragma unroll
      for (int i = 0; i < LR; ++i) roff[i] = across_off(i, BM, r_bytes, valid);
    }
  };
  const auto copy_x = [&](int s, bool none, uint8_t* buf) {
    none = none || s >= share(x_stages) || (G > 1 && s + ahead >= x_stages);
    s += ahead;
    if constexpr (kXAlong) {
      const uint32_t gone = none || (s == x_stages - 1 && along_cut) ? kNone : 0;
#pragma unroll
      for (int i = 0; i < LX; ++i)
        copy_piece<ONCE>(kPair && i >= LX / 2 ? xr2 : xr, buf + (i * NW + wave) * 1024, xoff[i] | gone, s * 128);
    } else {
      const int rows = none ? 0 : min(x_left - s * 64, 64);
      const Rsrc src = make_rsrc(xbase + static_cast<size_t>(none ? 0 : s) * 64 * O, rows > 0 ? rows * x_bytes - x_cols : 0);
#pragma unroll
      for (int i = 0; i < LX; ++i) copy_piece<ONCE>(src, buf + (i * NW + wave) * 1024, xoff[i], 0);
    }
  };
  const auto copy_r = [&](int s, bool none, uint8_t* buf) {
    none = none || s >= share(r_stages) || (G > 1 && s + ahead >= r_stages);
    s += ahead;
    if constexpr (kRAlong) {
      const uint32_t gone = none || (s == r_stages - 1 && along_cut) ? kNone : 0;
#pragma unroll
      for (int i = 0; i < LR; ++i) copy16(rr, buf + (i * NW + wave) * 1024, roff[i] | gone, s * 128);
    } else {
      const int rows = none ? 0 : min(r_left - s * 64, 64);
      const Rsrc src = make_rsrc(rbase + static_cast<size_t>(none ? 0 : s) * 64 * g.M, rows > 0 ? rows * r_bytes - r_cols : 0);
#pragma unroll
      for (int i = 0; i < LR; ++i) copy16(src, buf + (i * NW + wave) * 1024, roff[i], 0);
    }
  };

  // ---- fragments ----
  const auto x_frag = [&](int i) {  // the wave's fragment i of X, in the tile
    if (!kPair) return wn * TN + i * 32;
    return i < FN / 2 ? wn * (TN / 2) + i * 32 : BO + wn * (TN / 2) + (i - FN / 2) * 32;
  };
  const auto r_frag = [&](int j) { return (j * WM + wm) * 32; };  // in turn, so that short tiles keep all waves busy
  // Where this lane reads: along, of fragment 0 by 16-element step; across, of
  // step 0 by fragment.  (Opaque to the compiler: it would split them into sums of
  // many terms, at the end of which it loses which buffer an address is in and waits
  // for every copy: across, 8192^3 took 929 us, and 840 so.)
  uint32_t xa[kXAlong ? 4 : FN], ra[kRAlong ? 4 : FM];
  const auto lane_along = [&](int row, int ks) {
    uint32_t v = (row + col) * 128 + ((ks * 2 + half) ^ along_swizzle(col)) * 16;
    asm volatile("" : "+v"(v));
    return v;
  };
  const auto lane_across = [&](int row, int width) {
    const int j = lane & 15, b = (lane >> 4) & 1;
    const uint32_t piece = (row / 8 + 2 * b + ((j & 3) >> 1)) ^ across_swizzle(j >> 2);
    uint32_t v = (8 * half + (j >> 2)) * width * 2 + piece * 16 + (j & 1) * 8;
    asm volatile("" : "+v"(v));
    return v;
  };
  static_for<0, kXAlong ? 4 : FN>([&](auto ic) {
    constexpr int i = decltype(ic)::value;
    xa[i] = kXAlong ? lane_along(x_frag(0), i) : lane_across(x_frag(i), BN);
  });
  static_for<0, kRAlong ? 4 : FM>([&](auto jc) {
    constexpr int j = decltype(jc)::value;
    ra[j] = kRAlong ? lane_along(r_frag(0), j) : lane_across(r_frag(j), BM);
  });
  const auto along = [&](const uint8_t* p) { return *reinterpret_cast<const bf16x8*>(p); };
  const auto across = [&](const uint8_t* p, int width) {
    typedef __attribute__((address_space(3))) s16x4 Lds;
    const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((Lds*)p);
    const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((Lds*)(p + 4 * width * 2));
    return __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
  };
  bf16x8 xv[2][FN], rv[2][FM];
  const auto read = [&](int set, int ks, const uint8_t* xb, const uint8_t* rb) {
#pragma unroll
    for (int i = 0; i < FN; ++i) {
      const int row = x_frag(i) - x_frag(0);  // a constant
      xv[set][i] = kXAlong ? along(xb + xa[kXAlong ? ks : 0] + row * 128) : across(xb + xa[kXAlong ? 0 : i] + ks * 32 * BN, BN);
    }
#pragma unroll
    for (int j = 0; j < FM; ++j) {
      const int row = r_frag(j) - r_frag(0);
      rv[set][j] = kRAlong ? along(rb + ra[kRAlong ? ks : 0] + row * 128) : across(rb + ra[kRAlong ? 0 : j] + ks * 32 * BM, BM);
    }
  };
  f32x16 acc[FN][FM];
  const auto multiply = [&](int set) {
#pragma unroll
    for (int i = 0; i < FN; ++i)
#pragma unroll
      for (int j = 0; j < FM; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(xv[set][i], rv[set][j], acc[i][j], 0, 0, 0);
  };
  // One product, then its share of the next fragments' reads and of the copies,
  // and so on: copies issued together would keep the wave from its products (8192^3:
  // 1050 to 1060 us, and 883 to 1009 spread out).
  constexpr int kReads = FN * (kXAlong ? 1 : 2) + FM * (kRAlong ? 1 : 2), kMul = FN * FM;
  const auto interleave = [&](auto copies) {
    constexpr int kCopies = decltype(copies)::value;
    static_for<0, kMul>([&](auto ic) {
      constexpr int i = decltype(ic)::value;
      constexpr int reads = kReads * (i + 1) / kMul - kReads * i / kMul, some = kCopies * (i + 1) / kMul - kCopies * i / kMul;
      __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);
      if constexpr (reads > 0) __builtin_amdgcn_sched_group_barrier(0x100, reads, 0);
      if constexpr (some > 0) __builtin_amdgcn_sched_group_barrier(0x10, some, 0);
    });
  };

  open_tile();
  open_x();
  open_r();
  // In the loop R of stage st + RS follows stage st, and X of stage st + XS - 1
  // goes before its end, so that behind both operands of the next stage there are
  // kAhead copies under way.
  constexpr int kAhead = XS == RS ? (RS - 2) * (LX + LR) : (RS - 1) * LX + (RS - 2) * LR;
  static_for<0, RS>([&](auto qc) {
    constexpr int q = decltype(qc)::value;
    if constexpr (q < XS - 1) copy_x(q, false, x_buf(qc));
    copy_r(q, false, r_buf(qc));
    asm volatile("" ::: "memory");
  });
  wait_copies<(XS - 2) * LX + (RS - 1) * LR>();
  read(0, 0, x_buf(std::integral_constant<int, 0>{}), r_buf(std::integral_constant<int, 0>{}));
  for (;;) {
    const Place c = at;  // the tile being multiplied
    const int c_rows = rows_in(c), c_stages = share(stages_of(c));
    // its stages, and none or more without products, so that each tile starts with the same buffers
    const int c_all = max((c_stages + kRing - 1) / kRing, 1) * kRing;
    const bool live = wm * 32 < c_rows;  // else this wave's rows are all past the end
    // The tiles of the first channels sum R's columns as well, from the stages in
    // LDS: each lane eight columns of every kAtOnce-th row.  (32768 rows of 7168: 866 us
    // in all, and 961 with a kernel that reads R again.)
    constexpr int kPieces = BM / 8, kAtOnce = NW * kWave / kPieces;
    const bool c_sums = KIND == kWeights && g.sums != nullptr && c.n0 == 0;
    f32x8 columns = {0, 0, 0, 0, 0, 0, 0, 0};
    const auto add_columns = [&](const uint8_t* rb) {
#pragma unroll
      for (int i = 0; i < 64 / kAtOnce; ++i)
        columns += __builtin_convertvector(*reinterpret_cast<const bf16x8*>(rb + (tid * 16 + i * NW * 1024)), f32x8);
    };
    bool last = false;
#pragma unroll
    for (int i = 0; i < FN; ++i)
#pragma unroll
      for (int j = 0; j < FM; ++j)
#pragma unroll
        for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.0f;
    // A stage; without products (`idle`) past the last one.
    const auto stage = [&](int st, auto pc, auto idle) {
      constexpr int P = decltype(pc)::value;
      const uint8_t *xb = x_buf(pc), *rb = r_buf(pc);
      constexpr std::integral_constant<int, P + 1> after{};
      if (st + RS == c_all) {  // from here on R's copies are the next tile's, and X's with it or a stage later
        tile += step;
        last = tile >= end;
        if (!last) {
          open_tile();
          open_r();
        }
      }
      if (st + XS - 1 == c_all && !last) open_x();
      const int sx = st + XS - 1 >= c_all ? st + XS - 1 - c_all : st + XS - 1;  // the stages to copy
      const int sr = st + RS >= c_all ? st + RS - c_all : st + RS;
      const bool no_x = last && st + XS - 1 >= c_all, no_r = last && st + RS >= c_all;
      if constexpr (!decltype(idle)::value) {
        __builtin_amdgcn_sched_barrier(0);
        copy_x(sx, no_x, x_buf(std::integral_constant<int, P + XS - 1>{}));
        read(1, 1, xb, rb);
        multiply(0);
        interleave(std::integral_constant<int, LX>{});
        __builtin_amdgcn_sched_barrier(0);
        read(0, 2, xb, rb);
        multiply(1);
        interleave(std::integral_constant<int, 0>{});
        __builtin_amdgcn_sched_barrier(0);
        read(1, 3, xb, rb);
        multiply(0);
        interleave(std::integral_constant<int, 0>{});
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (KIND == kWeights) {
          if (c_sums) add_columns(rb);
        }
        // the next stage has arrived, and this one's buffers are read
        wait_copies<kAhead>();
        __builtin_amdgcn_sched_barrier(0);
        copy_r(sr, no_r, r_buf(pc));
        read(0, 0, x_buf(after), r_buf(after));
        multiply(1);
        interleave(std::integral_constant<int, LR>{});
        __builtin_amdgcn_sched_barrier(0);
      } else {
        copy_x(sx, no_x, x_buf(std::integral_constant<int, P + XS - 1>{}));
        wait_copies<kAhead>();
        copy_r(sr, no_r, r_buf(pc));
        if constexpr (P + 1 == kRing) read(0, 0, x_buf(after), r_buf(after));
      }
      asm volatile("" ::: "memory");  // the copies' order stays: the wait above counts on it
    };
    // Rounds of the buffers, and a last one that is not all products (written out a
    // second time, and with a wait for all copies at its end, so that no path leads
    // from an idle stage's copies to products: the compiler would wait for them
    // there, on every path).
    const int whole = c_stages / kRing * kRing;
    for (int first = 0; first < whole; first += kRing)
      static_for<0, kRing>([&](auto pc) { stage(first + decltype(pc)::value, pc, std::false_type{}); });
    if (whole < c_all) {
      static_while<0, kRing - 1>([&](auto pc) {
        constexpr int P = decltype(pc)::value;
        if (whole + P >= c_stages) return false;
        stage(whole + P, pc, std::false_type{});
        return true;
      });
      static_for<0, kRing>([&](auto pc) {
        constexpr int P = decltype(pc)::value;
        if (whole + P >= c_stages) stage(whole + P, pc, std::true_type{});
      });
      __builtin_amdgcn_s_waitcnt(7 << 4 | 15 << 8);  // vmcnt(0)
    }

    // ---- the result ----
    const size_t row0 = KIND == kWeights ? static_cast<size_t>(c.e) * g.M + c.m0 : static_cast<size_t>(c.first) + c.m0;
    if constexpr (KIND == kWeights) {
      if (c_sums) {
        float* const part = reinterpret_cast<float*>(x_buf(std::integral_constant<int, XS - 1>{}));
        static_assert(BN * 128 >= kAtOnce * BM * 4, "the column sums");
        const int k = tid / kPieces, n = ((tid % kPieces) ^ across_swizzle(k)) * 8;  // (a row's pieces lie permuted)
        f32x4* const mine = reinterpret_cast<f32x4*>(part + (k * BM + n));
        mine[0] = f32x4{columns[0], columns[1], columns[2], columns[3]};
        mine[1] = f32x4{columns[4], columns[5], columns[6], columns[7]};
        wait_reads();
        if (tid < c_rows && !(g.add && c_stages == 0)) {
          float sum = 0.0f;
          for (int i = 0; i < kAtOnce; ++i) sum += part[i * BM + tid];
          T* const to = static_cast<T*>(g.sums) + (row0 + tid);
          *to = static_cast<T>(g.add ? sum + static_cast<float>(*to) : sum);
        }
        wait_reads();
      }
    }
    // A fragment goes through LDS (the last stage's X buffer, where the next copy of
    // X goes, behind the barrier below), so that four lanes hold 32 channels of a
    // row and store 64 bytes (from the accumulators' layout it would be 8).  What a
    // fragment needs from memory is read before the one before it is stored: a
    // wait for loads is one for the stores ahead of them (4096 rows of 2048 to 7168 with
    // a residual: 121 against 131 us).  Not so an old gradient (g.add), which is read
    // where it is added: 32 matrices of 7168 x 2048 in binary32 take 1455 us so and 1069
    // without, where a read of them alone takes some 310.  Rows and channels past the
    // end are past the end of the buffer resources, where nothing is read or written.
    uint8_t* const yb = x_buf(std::integral_constant<int, XS - 1>{}) + wave * 4096;
    const auto y_place = [](uint32_t row, uint32_t piece) { return row * 128 + ((piece ^ (row & 7)) * 16); };
    const auto lay = [&](const f32x16& v) {
#pragma unroll
      for (int q = 0; q < 4; ++q)
        *reinterpret_cast<f32x4*>(yb + y_place(col, 2 * q + half)) = f32x4{v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]};
      asm volatile("" ::: "memory");
    };
    const auto turn = [&](const f32x16& v, f32x8(&out)[2]) {  // rows lane / 4 and 16 + lane / 4 of a fragment
      lay(v);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t row = h * 16 + (lane >> 2), q = (lane & 3) * 2;
        const f32x4 lo = *reinterpret_cast<const f32x4*>(yb + y_place(row, q));
        const f32x4 hi = *reinterpret_cast<const f32x4*>(yb + y_place(row, q + 1));
        out[h] = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
      }
      asm volatile("" ::: "memory");
    };
    constexpr bool kDouble = KIND == kRows && GATED;  // rows of 2 O channels
    constexpr uint32_t kSize = sizeof(T);
    const uint32_t y_bytes = (kDouble ? 2 : 1) * static_cast<uint32_t>(O) * kSize, p_bytes = 2 * static_cast<uint32_t>(O) * 2;
    const Rsrc yr = make_rsrc(uniform(static_cast<T*>(g.y) + row0 * (kDouble ? 2 * O : O)), c_rows * y_bytes);
    Rsrc pr = yr, resr = yr, br = yr;
    if (kPair || kDouble) pr = make_rsrc(uniform(g.p + row0 * 2 * O), g.p != nullptr ? c_rows * p_bytes : 0);
    if (KIND == kForward) {
      resr = make_rsrc(uniform(g.residual + row0 * O), g.residual != nullptr ? c_rows * y_bytes : 0);
      br = make_rsrc(uniform(g.bias + static_cast<size_t>(c.e) * (kPair ? 2 * O : O)), g.bias != nullptr ? (kPair ? 4 : 2) * O : 0);
    }
    const auto get = [](Rsrc from, uint32_t off) {
      return __builtin_bit_cast(bf16x8, __builtin_amdgcn_raw_buffer_load_b128(from, off, 0, 0));
    };
    const auto put = [](Rsrc to, uint32_t off, const f32x8& v) {
      __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, __builtin_convertvector(v, bf16x8)), to, off, 0, 0);
    };
    const auto wide = [](const bf16x8& v) { return __builtin_convertvector(v, f32x8); };
    // Fragment f: rows f / kAcross, channels f % kAcross.
    constexpr int kAcross = kPair ? FN / 2 : FN, kFragments = kAcross * FM;
    const auto channel = [&](int f) -> uint32_t { return c.n0 + x_frag(f % kAcross) + (lane & 3) * 8; };
    // its offset, for rows of so many bytes and elements of so many, of channel + more
    const auto offset = [&](int f, int h, uint32_t bytes, uint32_t size, uint32_t more) -> uint32_t {
      const uint32_t m = r_frag(f / kAcross) + h * 16 + (lane >> 2), n = channel(f);
      return n < static_cast<uint32_t>(O) ? m * bytes + (n + more) * size : kNone;
    };
    bf16x8 bias[2][2], old[2][kDouble ? 4 : 2];
    const bool adds = KIND == kWeights && g.add;
    const auto fetch = [&](int f) {
      const int b = f & 1;
      if constexpr (KIND == kForward) {
        const uint32_t n = channel(f);
        if (g.bias != nullptr) {
          bias[b][0] = get(br, n < static_cast<uint32_t>(O) ? n * 2 : kNone);
          if constexpr (kPair) bias[b][1] = get(br, n < static_cast<uint32_t>(O) ? (n + O) * 2 : kNone);
        }
        if (g.residual != nullptr) {
#pragma unroll
          for (int h = 0; h < 2; ++h) old[b][h] = get(resr, offset(f, h, y_bytes, 2, 0));
        }
      } else if constexpr (kDouble) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          old[b][2 * h] = get(pr, offset(f, h, p_bytes, 2, 0));
          old[b][2 * h + 1] = get(pr, offset(f, h, p_bytes, 2, O));
        }
      }
    };
    const auto finish = [&](auto fc) {
      constexpr int f = decltype(fc)::value, b = f & 1, i = f % kAcross, j = f / kAcross;
      f32x8 v[2], u[2];
      if constexpr (kSize == 4) lay(acc[i][j]);
      else turn(acc[i][j], v);
      if constexpr (kPair) turn(acc[i + FN / 2][j], u);
      if constexpr (KIND == kForward) {
        if (g.bias != nullptr) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            v[h] += wide(bias[b][0]);
            if constexpr (kPair) u[h] += wide(bias[b][1]);
          }
        }
        if constexpr (kPair) {
          if (g.p != nullptr) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              put(pr, offset(f, h, p_bytes, 2, 0), v[h]);
              put(pr, offset(f, h, p_bytes, 2, O), u[h]);
            }
          }
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int x = 0; x < 8; ++x) v[h][x] = silu_times(v[h][x], u[h][x]);
        }
        if (g.residual != nullptr) {
#pragma unroll
          for (int h = 0; h < 2; ++h) v[h] += wide(old[b][h]);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) put(yr, offset(f, h, y_bytes, 2, 0), v[h]);
      } else if constexpr (kDouble) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const f32x8 gv = wide(old[b][2 * h]), uv = wide(old[b][2 * h + 1]);
          f32x8 dg, du;
#pragma unroll
          for (int x = 0; x < 8; ++x) {
            const Gate k = gate(gv[x]);
            dg[x] = (v[h][x] * k.s1) * (uv[x] * k.s2) * (1.0f + gv[x] * k.n);
            du[x] = (v[h][x] * k.s1) * (gv[x] * k.s2);
          }
          put(yr, offset(f, h, y_bytes, 2, 0), dg);
          put(yr, offset(f, h, y_bytes, 2, O), du);
        }
      } else if constexpr (kSize == 4) {
#pragma unroll
        for (int h = 0; h < 4; ++h) {  // whole lines of 32 channels, eight rows at a time
          const uint32_t row = h * 8 + (lane >> 3), m = r_frag(j) + row, n = c.n0 + x_frag(i) + (lane & 7) * 4;
          const uint32_t at = n < static_cast<uint32_t>(O) ? m * y_bytes + n * 4 : kNone;
          f32x4 w = *reinterpret_cast<const f32x4*>(yb + y_place(row, lane & 7));
          if (adds) w += __builtin_bit_cast(f32x4, get(yr, at));
          __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, w), yr, at, 0, 0);
        }
        asm volatile("" ::: "memory");
      } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (adds) v[h] += wide(get(yr, offset(f, h, y_bytes, 2, 0)));
          put(yr, offset(f, h, y_bytes, 2, 0), v[h]);
        }
      }
    };
    if constexpr (G > 1) {  // the groups' sums, in their order, a fragment at a time
      static_for<0, FN * FM>([&](auto fc) {
        constexpr int i = decltype(fc)::value % FN, j = decltype(fc)::value / FN;
        if (group != 0) {
#pragma unroll
          for (int q = 0; q < 4; ++q)
            *reinterpret_cast<f32x4*>(yb + q * 1024 + lane * 16) =
                f32x4{acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
        }
        wait_reads();
        if (group == 0) {
#pragma unroll
          for (int o = 1; o < G; ++o)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const f32x4 v = *reinterpret_cast<const f32x4*>(yb + o * BN * 128 + q * 1024 + lane * 16);
#pragma unroll
              for (int x = 0; x < 4; ++x) acc[i][j][4 * q + x] += v[x];
            }
        }
        wait_reads();
      });
    }
    if (live && group == 0 && !(adds && c_stages == 0)) {
      fetch(0);
      static_while<0, kFragments>([&](auto fc) {
        constexpr int f = decltype(fc)::value;
        if (f % kAcross == 0 && r_frag(f / kAcross) >= c_rows) return false;  // (nor have those behind it)
        if constexpr (f + 1 < kFragments) fetch(f + 1);
        finish(fc);
        return true;
      });
    }
    if (last) break;
    wait_reads();  // every wave's fragments have left LDS
  }
  __builtin_amdgcn_s_waitcnt(7 << 4);  // vmcnt(0) lgkmcnt(0): no copy outlives the workgroup's LDS
}

template <typename Kernel>
hipError_t launch_linear(Kernel kernel, int threads, int per_cu, const LinearArgs& g, hipStream_t stream) {
  const int grid = max(device_cu_count() / 8, 1) * 8 * per_cu;
  hipLaunchKernelGGL(kernel, dim3(grid), dim3(threads), 0, stream, g);
  return hipGetLastError();
}
template <Kind KIND, bool GATED, typename T, int BM, int BN, int WM, int WN, int XS, int RS, int PER, bool ONCE = false, int G = 1>
hipError_t launch_tiles(const LinearArgs& g, hipStream_t stream) {
  return launch_linear(linear_tiled<KIND, GATED, T, BM, BN, WM, WN, XS, RS, PER, ONCE, G>, G * WM * WN * kWave, PER, g, stream);
}

// What the choice of a tile goes by.  The rows of each expert are on the device;
// the host knows their number, and for the padded layout no more than the
// capacity, which stands for some 64 rows at most (32 experts of 7168 to 4096, gated,
// capacity 1024 with 128 rows each: 346 us, and 371 packed; capacity 4096 with 1024
// rows each: 1816, and 1509 packed).
struct LinearShape {
  int64_t rows, hit;  // and experts that have any, at most
  int64_t avg;        // rows of an expert
  int64_t cus;
  int64_t tiles(int bm, int o, int bo) const {  // of bm rows and bo of o channels
    return max(hit, (rows + bm - 1) / bm) * ((o + bo - 1) / bo);
  }
  bool fill(int bm, int o, int bo) const { return tiles(bm, o, bo) * 8 >= 7 * cus; }  // the chip, or nearly
};
inline LinearShape linear_shape(const LinearArgs& g) {
  const int64_t each = g.capacity > 0 ? min(g.capacity, 64) : g.num_rows / g.E;
  const int64_t rows = g.capacity > 0 ? each * g.E : g.num_rows;
  return LinearShape{rows, min(static_cast<int64_t>(g.E), rows), each, max(device_cu_count(), 1)};
}

inline const __bf16* b16(const uint16_t* p) { return reinterpret_cast<const __bf16*>(p); }
inline __bf16* b16(uint16_t* p) { return reinterpret_cast<__bf16*>(p); }

}  // namespace ep
