// The gradients of the experts' bf16 layers with respect to their weights and
// biases.  The contract is ep_expert_linear_backward_weights' in include/ep.h.

#include "linear_tile.h"

namespace ep {
namespace {

// grad_b[e, n] = sum over e's rows of g[r, n]: a workgroup takes COLS columns of
// one expert; COLS / 8 lanes hold a row's, 16 bytes each, the others every so
// many rows beyond, and their sums are added in LDS in a fixed order.
constexpr int kSumThreads = 1024;

template <typename T, int COLS>
__global__ __launch_bounds__(kSumThreads) void column_sums(const __bf16* __restrict__ g,
                                                           const int32_t* __restrict__ expert_rows, int32_t num_rows,
                                                           int32_t capacity, int32_t N, bool add,
                                                           T* __restrict__ grad_b) {
  constexpr int L = COLS / 8, S = kSumThreads / L;  // lanes of a row, and rows read at once
  __shared__ float part[S][COLS + 1];
  const int groups = (N + COLS - 1) / COLS;
  const int e = blockIdx.x / groups, n0 = blockIdx.x % groups * COLS;
  const int lane = threadIdx.x % L, s = threadIdx.x / L, n = n0 + lane * 8;
  int first, count;
  span_of(expert_rows, e, capacity, num_rows, first, count);
  f32x8 sum = {0, 0, 0, 0, 0, 0, 0, 0};
  if (n < N) {
    const __bf16* p = g + static_cast<size_t>(first) * N + n;
    int r = s;
    for (; r + 3 * S < count; r += 4 * S) {
      bf16x8 v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = *reinterpret_cast<const bf16x8*>(p + static_cast<size_t>(r + i * S) * N);
#pragma unroll
      for (int i = 0; i < 4; ++i) sum += __builtin_convertvector(v[i], f32x8);
    }
    for (; r < count; r += S) sum += __builtin_convertvector(*reinterpret_cast<const bf16x8*>(p + static_cast<size_t>(r) * N), f32x8);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) part[s][lane * 8 + i] = sum[i];
  for (int d = S / 2; d > 0; d /= 2) {
    __syncthreads();
    for (int i = threadIdx.x; i < d * COLS; i += kSumThreads) part[i / COLS][i % COLS] += part[i / COLS + d][i % COLS];
  }
  __syncthreads();
  const int c = threadIdx.x;
  if (c < COLS && n0 + c < N) {
    T* to = grad_b + static_cast<size_t>(e) * N + n0 + c;
    *to = static_cast<T>(add ? part[0][c] + static_cast<float>(*to) : part[0][c]);
  }
}

template <typename T>
hipError_t launch(const LinearArgs& g, hipStream_t stream) {
  const int64_t cus = max(device_cu_count(), 1);
  const auto fill = [&](int bm, int bn) {
    return static_cast<int64_t>(g.E) * ((g.M + bm - 1) / bm) * ((g.O + bn - 1) / bn) * 8 >= 7 * cus;
  };
  if (linear_shape(g).avg > 400 && fill(256, 256)) return launch_tiles<kWeights, false, T, 256, 256, 2, 4, 3, 2, 1>(g, stream);
  if (fill(128, 256)) return launch_tiles<kWeights, false, T, 128, 256, 2, 4, 3, 3, 1>(g, stream);
  return launch_tiles<kWeights, false, T, 128, 128, 2, 2, 4, 4, 1>(g, stream);
}

}  // namespace

hipError_t launch_expert_linear_backward_weights(const uint16_t* grad_y, const uint16_t* a, const int32_t* expert_rows,
                                                 int32_t num_rows, int32_t E, int32_t capacity, int32_t H, int32_t N,
                                                 bool bf16, bool add, void* grad_w, void* grad_bias,
                                                 hipStream_t stream) {
  const LinearArgs args{b16(a), b16(grad_y), nullptr, nullptr, expert_rows, num_rows, E, capacity, 0,
                        H, N, add, nullptr, grad_w};
  const auto run = [&](auto t) {
    using T = decltype(t);
    const hipError_t err = launch<T>(args, stream);
    if (err != hipSuccess || grad_bias == nullptr) return err;
    const auto sums = [&](auto kernel, int cols) {
      hipLaunchKernelGGL(kernel, dim3(E * ((N + cols - 1) / cols)), dim3(kSumThreads), 0, stream, args.r, expert_rows,
                         num_rows, capacity, N, add, static_cast<T*>(grad_bias));
    };
    // whole lines where that gives every CU a workgroup, else half lines
    if (static_cast<int64_t>(E) * N >= 64 * 512) sums(column_sums<T, 64>, 64);
    else sums(column_sums<T, 32>, 32);
    return hipGetLastError();
  };
  return bf16 ? run(__bf16{}) : run(float{});
}

}  // namespace ep
