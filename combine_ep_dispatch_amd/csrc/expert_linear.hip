// The experts' linear layers in bf16: y[r, :] = act(W[e(r)] a[r] + b[e(r)])
// (+ residual), and the gradients of the rows and of the weights.  The
// contracts are ep_expert_linear's, ep_expert_linear_backward's and
// ep_expert_linear_backward_weights' in include/ep.h.
//
// Each is a product per expert on gfx950's bf16 MFMA, whose sums are binary32
// (products exact, subnormals kept; measured: a term 2^-23 below the sum counts
// in full).  An output's channels are the A operand and its rows the B operand,
// so a lane ends up with four consecutive channels of one row.

#include "ep_internal.h"
#include "expert_device.h"

namespace ep {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));

constexpr int kThreads = 256;

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

// The gate's sigmoid s = 1 / (1 + exp(-g)) as two factors s1 s2, and n = 1 - s,
// each without cancellation.  (Two, each with half the exponent, so that s
// keeps its accuracy below 2^-126, where a large g or d makes it count.)
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

// What a product is for: the layer itself, or the gradient of its rows.
enum Kind { kForward, kRows };

// C: the summed channels, O: channels of the result (before GATED doubles or
// halves them): kForward sums over w's last dimension, kRows over its middle one.
template <Kind KIND, bool GATED>
__global__ __launch_bounds__(kThreads) void linear_simple(const __bf16* __restrict__ a, const __bf16* __restrict__ w,
                                                          const __bf16* __restrict__ bias, const __bf16* residual,
                                                          const int32_t* __restrict__ expert_rows, int32_t num_rows,
                                                          int32_t E, int32_t capacity, int32_t C, int32_t O,
                                                          __bf16* p, __bf16* y) {
  constexpr int BM = 16, BN = 64;
  constexpr bool kPair = KIND == kForward && GATED;
  __shared__ RowTiles start[kMaxExperts + 1];  // row tiles before each expert
  const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave;
  for (int e = tid; e < E; e += kThreads) {
    int first, count;
    span_of(expert_rows, e, capacity, num_rows, first, count);
    start[e] = (static_cast<int64_t>(count) + BM - 1) / BM;
  }
  if (tid == 0) start[E] = 0;
  __syncthreads();
  tiles_before(start, E);
  const int nt = (O + BN - 1) / BN;
  const int64_t tiles = start[E] * nt;
  const int grp = lane >> 4, col = lane & 15;
  const int rows_w = kPair ? 2 * O : O;  // rows of w (kForward)
  for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    const int e = expert_of_tile(start, E, tile / nt);
    int first, count;
    span_of(expert_rows, e, capacity, num_rows, first, count);
    const int64_t te = start[e + 1] - start[e];
    const int64_t local = tile - start[e] * nt;
    const int m = static_cast<int>(local % te) * BM + col, n0 = static_cast<int>(local / te) * BN + wave * 16;
    const size_t row = static_cast<size_t>(first) + min(m, count - 1);
    const __bf16* ap = a + row * C;
    const int wn = min(n0 + col, O - 1);
    const __bf16* we = w + static_cast<size_t>(e) * (KIND == kForward ? rows_w : O) * C;
    f32x4 acc[kPair ? 2 : 1];
#pragma unroll
    for (auto& c : acc) c = f32x4{0, 0, 0, 0};
    for (int k0 = 0; k0 < C; k0 += 32) {
      const int k = k0 + 8 * grp;
      const bool in = k < C;  // C is a multiple of 8
      bf16x8 b = {};
      if (in) b = *reinterpret_cast<const bf16x8*>(ap + k);
#pragma unroll
      for (int h = 0; h < (kPair ? 2 : 1); ++h) {
        bf16x8 v = {};
        if (in) {
          if constexpr (KIND == kForward) {
            v = *reinterpret_cast<const bf16x8*>(we + static_cast<size_t>(h * O + wn) * C + k);
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = we[static_cast<size_t>(k + i) * O + wn];
          }
        }
        acc[h] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v, b, acc[h], 0, 0, 0);
      }
    }
    const int n = n0 + 4 * grp;  // this lane's four channels; O is a multiple of 8
    if (m < count && n < O) {
      if constexpr (KIND == kForward) {
        bf16x4 o;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float g = acc[0][i], v = kPair ? acc[kPair ? 1 : 0][i] : 0.0f;
          if (bias != nullptr) {
            const __bf16* be = bias + static_cast<size_t>(e) * rows_w;
            g += static_cast<float>(be[n + i]);
            if (kPair) v += static_cast<float>(be[O + n + i]);
          }
          if (kPair && p != nullptr) {
            p[row * rows_w + n + i] = static_cast<__bf16>(g);
            p[row * rows_w + O + n + i] = static_cast<__bf16>(v);
          }
          float r = kPair ? silu_times(g, v) : g;
          if (residual != nullptr) r += static_cast<float>(residual[row * O + n + i]);
          o[i] = static_cast<__bf16>(r);
        }
        *reinterpret_cast<bf16x4*>(y + row * O + n) = o;
      } else if constexpr (GATED) {
        const bf16x4 g = *reinterpret_cast<const bf16x4*>(p + row * 2 * O + n);
        const bf16x4 u = *reinterpret_cast<const bf16x4*>(p + row * 2 * O + O + n);
        bf16x4 dg, du;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float gi = static_cast<float>(g[i]), d = acc[0][i];
          const Gate k = gate(gi);
          dg[i] = static_cast<__bf16>((d * k.s1) * (static_cast<float>(u[i]) * k.s2) * (1.0f + gi * k.n));
          du[i] = static_cast<__bf16>((d * k.s1) * (gi * k.s2));
        }
        *reinterpret_cast<bf16x4*>(y + row * 2 * O + n) = dg;
        *reinterpret_cast<bf16x4*>(y + row * 2 * O + O + n) = du;
      } else {
        bf16x4 o;
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = static_cast<__bf16>(acc[0][i]);
        *reinterpret_cast<bf16x4*>(y + row * O + n) = o;
      }
    }
  }
}

// grad_w[e, n, h] = sum over e's rows of g[r, n] a[r, h]: h is the A operand.
template <typename T>
__global__ __launch_bounds__(kThreads) void weights_simple(const __bf16* __restrict__ g, const __bf16* __restrict__ a,
                                                           const int32_t* __restrict__ expert_rows, int32_t num_rows,
                                                           int32_t E, int32_t capacity, int32_t H, int32_t N,
                                                           bool add, T* __restrict__ grad_w) {
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
  const int grp = lane >> 4, col = lane & 15;
  const int nt = (N + 15) / 16, ht = (H + 63) / 64;
  const int64_t tiles = static_cast<int64_t>(E) * nt * ht;
  for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    const int e = static_cast<int>(tile / (static_cast<int64_t>(nt) * ht));
    const int64_t local = tile - static_cast<int64_t>(e) * nt * ht;
    const int n = static_cast<int>(local / ht) * 16 + col, h0 = static_cast<int>(local % ht) * 64 + wave * 16;
    int first, count;
    span_of(expert_rows, e, capacity, num_rows, first, count);
    const __bf16* gp = g + static_cast<size_t>(first) * N + min(n, N - 1);
    const __bf16* ap = a + static_cast<size_t>(first) * H + min(h0 + col, H - 1);
    f32x4 acc = {0, 0, 0, 0};
    for (int k0 = 0; k0 < count; k0 += 32) {
      bf16x8 u = {}, v = {};
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int k = k0 + 8 * grp + i;
        if (k < count) {
          u[i] = ap[static_cast<size_t>(k) * H];
          v[i] = gp[static_cast<size_t>(k) * N];
        }
      }
      acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(u, v, acc, 0, 0, 0);
    }
    const int h = h0 + 4 * grp;
    if (n < N && h < H) {
      T* out = grad_w + (static_cast<size_t>(e) * N + n) * H + h;
#pragma unroll
      for (int i = 0; i < 4; ++i) out[i] = static_cast<T>(add ? acc[i] + static_cast<float>(out[i]) : acc[i]);
    }
  }
}

// grad_b[e, n] = sum over e's rows of g[r, n].
template <typename T>
__global__ __launch_bounds__(kThreads) void bias_simple(const __bf16* __restrict__ g,
                                                        const int32_t* __restrict__ expert_rows, int32_t num_rows,
                                                        int32_t E, int32_t capacity, int32_t N, bool add,
                                                        T* __restrict__ grad_b) {
  const int64_t items = static_cast<int64_t>(E) * N;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; i < items;
       i += static_cast<int64_t>(gridDim.x) * kThreads) {
    const int e = static_cast<int>(i / N), n = static_cast<int>(i % N);
    int first, count;
    span_of(expert_rows, e, capacity, num_rows, first, count);
    float sum = 0.0f;
    for (int r = 0; r < count; ++r) sum += static_cast<float>(g[(static_cast<size_t>(first) + r) * N + n]);
    grad_b[i] = static_cast<T>(add ? sum + static_cast<float>(grad_b[i]) : sum);
  }
}

}  // namespace

hipError_t launch_expert_linear(const uint16_t* a, const uint16_t* w, const uint16_t* bias, const uint16_t* residual,
                                const int32_t* expert_rows, int32_t num_rows, int32_t E, int32_t capacity, int32_t H,
                                int32_t N, bool gated, uint16_t* p, uint16_t* y, hipStream_t stream) {
  const auto with = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3(2048), dim3(kThreads), 0, stream, reinterpret_cast<const __bf16*>(a),
                       reinterpret_cast<const __bf16*>(w), reinterpret_cast<const __bf16*>(bias),
                       reinterpret_cast<const __bf16*>(residual), expert_rows, num_rows, E, capacity, H,
                       gated ? N / 2 : N, reinterpret_cast<__bf16*>(p), reinterpret_cast<__bf16*>(y));
    return hipGetLastError();
  };
  return gated ? with(linear_simple<kForward, true>) : with(linear_simple<kForward, false>);
}

hipError_t launch_expert_linear_backward(const uint16_t* grad_y, const uint16_t* w, const uint16_t* p,
                                         const int32_t* expert_rows, int32_t num_rows, int32_t E, int32_t capacity,
                                         int32_t H, int32_t N, uint16_t* grad_a, hipStream_t stream) {
  const auto with = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3(2048), dim3(kThreads), 0, stream, reinterpret_cast<const __bf16*>(grad_y),
                       reinterpret_cast<const __bf16*>(w), static_cast<const __bf16*>(nullptr),
                       static_cast<const __bf16*>(nullptr), expert_rows, num_rows, E, capacity, N, H,
                       const_cast<__bf16*>(reinterpret_cast<const __bf16*>(p)), reinterpret_cast<__bf16*>(grad_a));
    return hipGetLastError();
  };
  return p != nullptr ? with(linear_simple<kRows, true>) : with(linear_simple<kRows, false>);
}

hipError_t launch_expert_linear_backward_weights(const uint16_t* grad_y, const uint16_t* a, const int32_t* expert_rows,
                                                 int32_t num_rows, int32_t E, int32_t capacity, int32_t H, int32_t N,
                                                 bool bf16, bool add, void* grad_w, void* grad_bias,
                                                 hipStream_t stream) {
  const __bf16* g = reinterpret_cast<const __bf16*>(grad_y);
  const auto run = [&](auto t) {
    using T = decltype(t);
    hipLaunchKernelGGL(weights_simple<T>, dim3(2048), dim3(kThreads), 0, stream, g, reinterpret_cast<const __bf16*>(a),
                       expert_rows, num_rows, E, capacity, H, N, add, static_cast<T*>(grad_w));
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess || grad_bias == nullptr) return err;
    hipLaunchKernelGGL(bias_simple<T>, dim3(2048), dim3(kThreads), 0, stream, g, expert_rows, num_rows, E, capacity, N,
                       add, static_cast<T*>(grad_bias));
    return hipGetLastError();
  };
  return bf16 ? run(__bf16{}) : run(float{});
}

}  // namespace ep
