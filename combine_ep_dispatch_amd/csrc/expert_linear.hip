// The experts' bf16 layers: y[r, :] = act(W[e(r)] a[r] + b[e(r)]) (+ residual).
// The contract is ep_expert_linear's in include/ep.h.

#include "linear_tile.h"

namespace ep {
namespace {

// Few rows an expert: the weights' stream is all there is.  A workgroup takes 16
// rows of a and 16 of w (the gates and ups of 8 channels, or 16 channels); its
// eight waves split the summed channels, read their share straight into
// registers, eight loads of 16 rows by 64 bytes ahead, and add their sums in LDS
// in a fixed order.  16 rows of 7168 to 4096, gated: 16.5 us (3.6 TB/s, bounded by
// the latency of few loads a wave), against 23 in 64 x 64 tiles, which leave half of
// the CUs idle; 7 rows of 2048 to 7168: 10.6.  Where tiles fill the chip they are
// faster (1 token of 8 of 256 experts: 73 against 88 us; 128 tokens 2090 against 2900).
constexpr int kFewWaves = 8;

template <bool GATED>
__global__ __launch_bounds__(kFewWaves* kWave, 4) void linear_few(const LinearArgs g) {
  constexpr int U = 4;  // steps of 32 channels read together
  constexpr int BM = 16, BO = GATED ? 8 : 16;
  __shared__ RowTiles start[kMaxExperts + 1];  // row tiles before each expert
  __shared__ __align__(16) float part[kFewWaves][16][16];
  const int tid = threadIdx.x, lane = tid & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int grp = lane >> 4, col = lane & 15;
  const int E = g.E, C = g.C, O = g.O;
  if (g.expert_rows != nullptr) {
    for (int e = tid; e < E; e += kFewWaves * kWave) {
      int first, count;
      span_of(g.expert_rows, e, g.capacity, g.num_rows, first, count);
      start[e] = (static_cast<int64_t>(count) + BM - 1) / BM;
    }
    if (tid == 0) start[E] = 0;
    __syncthreads();
    tiles_before(start, E);
  }
  const uint32_t nt = (O + BO - 1) / BO;
  const int64_t all_rows = g.expert_rows != nullptr ? uniform(start[E]) : (static_cast<int64_t>(g.num_rows) + BM - 1) / BM;
  const int64_t tiles = all_rows * nt;
  const int slice = ((C + kFewWaves - 1) / kFewWaves + 31) / 32 * 32;  // this wave's channels
  const int k0 = min(wave * slice, C), k1 = min(k0 + slice, C);
  const uint32_t bytes = static_cast<uint32_t>(C) * 2;
  const uint32_t wbytes = (GATED ? 2 : 1) * static_cast<uint32_t>(O) * bytes;  // of an expert's matrix: below 2^31
  for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    int e = 0, first = 0, count = g.num_rows;
    int64_t te = all_rows, local = tile;
    if (g.expert_rows != nullptr) {
      e = __builtin_amdgcn_readfirstlane(expert_of_tile(start, E, tile / nt));
      span_of(g.expert_rows, e, g.capacity, g.num_rows, first, count);
      te = start[e + 1] - start[e];
      local = tile - start[e] * nt;
    }
    const int m0 = __builtin_amdgcn_readfirstlane(static_cast<int>(local % te)) * BM;
    const int n0 = __builtin_amdgcn_readfirstlane(static_cast<int>(local / te)) * BO;
    const int rows = __builtin_amdgcn_readfirstlane(min(count - m0, BM)), valid = min(O - n0, BO);
    const size_t row0 = static_cast<size_t>(__builtin_amdgcn_readfirstlane(first)) + m0;
    const Rsrc wr = make_rsrc(uniform(g.x + static_cast<size_t>(e) * (GATED ? 2 : 1) * O * C), wbytes);
    const Rsrc rr = make_rsrc(uniform(g.r + row0 * C), rows * bytes);
    const int ch = col % BO;
    const uint32_t woff = ch < valid ? (n0 + ch + (col < BO ? 0 : O)) * bytes : kNone;
    const uint32_t roff = col < rows ? col * bytes : kNone;
    f32x4 acc = {0, 0, 0, 0};
    bf16x8 w[2][U], a[2][U];
    const auto load = [&](int set, int k) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int kk = k + u * 32 + grp * 8;
        const bool in = kk < k1;
        w[set][u] = __builtin_bit_cast(bf16x8, __builtin_amdgcn_raw_buffer_load_b128(wr, in ? woff + kk * 2 : kNone, 0, 0));
        a[set][u] = __builtin_bit_cast(bf16x8, __builtin_amdgcn_raw_buffer_load_b128(rr, in ? roff + kk * 2 : kNone, 0, 0));
      }
      __builtin_amdgcn_sched_barrier(0);
    };
    const auto multiply = [&](int set) {
#pragma unroll
      for (int u = 0; u < U; ++u) acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w[set][u], a[set][u], acc, 0, 0, 0);
      __builtin_amdgcn_sched_barrier(0);
    };
    load(0, k0);
    for (int k = k0; k < k1; k += 64 * U) {
      load(1, k + 32 * U);
      multiply(0);
      load(0, k + 64 * U);
      multiply(1);
    }
    __syncthreads();  // the last tile's sums are read
    *reinterpret_cast<f32x4*>(&part[wave][col][grp * 4]) = acc;
    __syncthreads();
    if (tid < 16 * BO) {
      const int m = tid / BO, o = tid % BO, n = n0 + o;
      if (m < rows && o < valid) {
        float v = 0.0f, u = 0.0f;
#pragma unroll
        for (int x = 0; x < kFewWaves; ++x) {
          v += part[x][m][o];
          if (GATED) u += part[x][m][o + 8];
        }
        const size_t at = (row0 + m) * O + n;
        if (g.bias != nullptr) {
          const __bf16* be = g.bias + static_cast<size_t>(e) * (GATED ? 2 : 1) * O + n;
          v += static_cast<float>(be[0]);
          if (GATED) u += static_cast<float>(be[O]);
        }
        if (GATED && g.p != nullptr) {
          __bf16* p = g.p + (row0 + m) * 2 * O + n;
          p[0] = static_cast<__bf16>(v);
          p[O] = static_cast<__bf16>(u);
        }
        if (GATED) v = silu_times(v, u);
        if (g.residual != nullptr) v += static_cast<float>(g.residual[at]);
        static_cast<__bf16*>(g.y)[at] = static_cast<__bf16>(v);
      }
    }
  }
}

// The tile, by the mean rows of an expert, and smaller where larger ones would
// leave CUs without any.  Measured in microseconds, * as the rule picks, "once":
// weights read non-temporally; with E 256, H 7168, N 4096 gated, 8 experts a token,
//   tokens (mean rows)  128 (4)  512 (16)  2048 (64)  3000 (94)  4096 (128)  32768 (1024)
//   64 x 128 once         *2088     *2234       3614
//   64 x 128               2350      2403       3601       3789        4380
//   128 x 256 once         2106      2256      *2397      *2571         4308
//   128 x 256              2450      2512       2606       2656        3655        15890
//   192 x 256              2414      2469       2671       2749       *3016        15510
//   256 x 256              2531      2652       2880       2969        3216       *13230
// With popular experts (1.2 in Zipf's law) as the rule picks: 512 tokens 2350 us and
// 2165 evenly, 2048 3080 and 2475, 4096 3680 and 2976.
// And for one matrix of the same sizes (its rows), where few tiles are idle CUs:
//   rows                  16    64   128   256   384   512   768  1024  2048
//   few rows           *16.2          109   214         425         847  1688
//   64 x 64, 2 groups   23.2 *24.7 *24.9 *26.0  46.6  48.4  70.4
//   64 x 64             31.3  31.6  31.8  32.6  41.2  42.8  72.9  83.4   163
//   64 x 128, 2 groups  31.4  33.9  33.8  34.2 *35.2 *39.4  70.1
//   64 x 128            35.5        36.2  37.5  41.6  41.4 *75.2  82.2   160
//   128 x 128           41.4        43.4  43.5        47.4       *58.7   113
//   128 x 256           65.4        69.2  69.5        70.2        74.5  *103
//   256 x 256            112         113   117         117         119   137
// Three and four groups, of fewer stages each, take 25.7 and 33.3 us at 128 rows.
// Two groups need a long sum (the second one's way to the first costs 2 us):
//   summed channels                256   512  1024  2048  4096
//   128 rows, N 1024:
//     64 x 64, 2 groups            6.2   6.1  *7.3  *9.9 *15.5
//     64 x 64                     *4.6  *5.6   7.6  11.5  19.8
//   384 rows, N 4096 gated:
//     64 x 128, 2 groups           7.2   8.4  10.5  14.9 *23.0
//     64 x 64                     *6.1  *7.2 *10.0 *14.8  24.5
// With many rows on one matrix L2 serves the weights, two stages of them do, and
// more stages cost more idle ones at a tile's end (16384 rows of 2048 to 7168: two
// 371, three 391; 1024 rows an expert as above: 13880 and 13090).
template <bool GATED>
hipError_t launch(const LinearArgs& g, hipStream_t stream) {
  constexpr Kind F = kForward;
  const LinearShape s = linear_shape(g);
  const auto fill = [&](int bm, int bn) { return s.fill(bm, g.O, GATED ? bn / 2 : bn); };
  if (s.avg > 170 && fill(256, 256)) {
    if (s.avg > 2048) return launch_tiles<F, GATED, __bf16, 256, 256, 4, 2, 2, 2, 1>(g, stream);
    return launch_tiles<F, GATED, __bf16, 256, 256, 4, 2, 3, 2, 1>(g, stream);
  }
  if (s.avg > 100 && fill(192, 256)) return launch_tiles<F, GATED, __bf16, 192, 256, 2, 4, 3, 2, 1>(g, stream);
  if (s.avg > 32 && fill(128, 256)) {
    if (s.avg <= 100) return launch_tiles<F, GATED, __bf16, 128, 256, 2, 4, 3, 3, 1, true>(g, stream);
    return launch_tiles<F, GATED, __bf16, 128, 256, 2, 4, 3, 3, 1>(g, stream);
  }
  if (s.avg > 32 && fill(128, 128)) return launch_tiles<F, GATED, __bf16, 128, 128, 2, 2, 4, 4, 1>(g, stream);
  if (s.avg <= 64 && fill(64, 128)) return launch_tiles<F, GATED, __bf16, 64, 128, 2, 2, 6, 6, 1, true>(g, stream);
  if (s.avg <= 16 && static_cast<int64_t>(g.O) * g.C < (GATED ? int64_t(1) << 29 : int64_t(1) << 30))
    return launch_linear(linear_few<GATED>, kFewWaves * kWave, 2, g, stream);
  if (g.C > 768 && s.tiles(64, g.O, GATED ? 32 : 64) <= s.cus)
    return launch_tiles<F, GATED, __bf16, 64, 64, 2, 1, 4, 4, 1, false, 2>(g, stream);
  if (s.tiles(64, g.O, GATED ? 64 : 128) <= s.cus) {
    if (g.C > 2048) return launch_tiles<F, GATED, __bf16, 64, 128, 2, 2, 3, 3, 1, false, 2>(g, stream);
    return launch_tiles<F, GATED, __bf16, 64, 64, 2, 1, 4, 4, 2>(g, stream);
  }
  return launch_tiles<F, GATED, __bf16, 64, 128, 2, 2, 6, 6, 1>(g, stream);
}

}  // namespace

hipError_t launch_expert_linear(const uint16_t* a, const uint16_t* w, const uint16_t* bias, const uint16_t* residual,
                                const int32_t* expert_rows, int32_t num_rows, int32_t E, int32_t capacity, int32_t H,
                                int32_t N, bool gated, uint16_t* p, uint16_t* y, hipStream_t stream) {
  const LinearArgs g{b16(w), b16(a), b16(bias), b16(residual), expert_rows, num_rows, E, capacity, H,
                     gated ? N / 2 : N, 0, false, b16(p), y, nullptr};
  return gated ? launch<true>(g, stream) : launch<false>(g, stream);
}

}  // namespace ep
