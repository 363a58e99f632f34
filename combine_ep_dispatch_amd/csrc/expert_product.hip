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

}  // namespace

hipError_t launch_expert_product(const void* a, const void* a_scale, bool fp8, const void* w, const void* w_scale,
                                 const int32_t* expert_rows, int32_t num_rows, int32_t E, int32_t capacity,
                                 int32_t H, int32_t N, bool gated, uint16_t* y, hipStream_t stream) {
  const auto launch = [&](auto f, auto g) {
    hipLaunchKernelGGL((product_kernel<decltype(f)::value, decltype(g)::value>), dim3(2048), dim3(kThreads), 0, stream,
                       static_cast<const uint8_t*>(a), static_cast<const uint8_t*>(a_scale),
                       static_cast<const uint8_t*>(w), static_cast<const uint8_t*>(w_scale), expert_rows, num_rows, E,
                       capacity, H, N, y);
  };
  if (fp8) {
    if (gated) launch(std::true_type{}, std::true_type{}); else launch(std::true_type{}, std::false_type{});
  } else {
    if (gated) launch(std::false_type{}, std::true_type{}); else launch(std::false_type{}, std::false_type{});
  }
  return hipGetLastError();
}

}  // namespace ep
