// Routing: router logits to the expert ids and weights the dispatch takes,
// and the gradient of those weights.  The rule is stated at ep_route in
// include/ep.h.
//
// One wavefront per token.

#include <hip/hip_runtime.h>

#include "ep_device.h"
#include "ep_internal.h"

namespace ep {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / kWave;
constexpr float kNegInf = -__builtin_inff();

__device__ __forceinline__ float load_logit(const float* p) { return *p; }
__device__ __forceinline__ float load_logit(const uint16_t* p) { return bf16_lo(*p); }

// z of ep_route: NaN counts as -inf, +inf as the largest finite binary32.
__device__ __forceinline__ float clean_logit(float z) {
  z = z != z ? kNegInf : z;
  return fminf(z, __FLT_MAX__);
}

__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) v = fmaxf(v, __shfl_xor(v, d));
  return v;
}

template <typename T>
__device__ __forceinline__ T wave_sum(T v) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) v += __shfl_xor(v, d);
  return v;
}

// The lane holding the largest (key, lowest index) of the wavefront.
__device__ __forceinline__ void wave_argmax(double& key, int& idx) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) {
    const double k = __shfl_xor(key, d);
    const int i = __shfl_xor(idx, d);
    if (k > key || (k == key && i < idx)) {
      key = k;
      idx = i;
    }
  }
}

// Lane l holds experts l, l + 64, ..; EPL of them.
template <typename Z, int EPL>
__global__ __launch_bounds__(kThreads) void route_kernel(const Z* __restrict__ logits, const float* __restrict__ bias,
                                                         int32_t T, int32_t E, int32_t K, int32_t n_group,
                                                         int32_t topk_group, int32_t score, int32_t renorm,
                                                         float scale, int32_t* __restrict__ ids,
                                                         float* __restrict__ weights) {
  extern __shared__ double route_lds[];  // per wave: v [E]
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
  const int t = blockIdx.x * kWaves + wave;
  if (t >= T) return;  // no barrier below: the wavefronts are independent
  const double ninf = -__builtin_inf();
  double* v_lds = route_lds + static_cast<size_t>(wave) * E;
  float z[EPL];
  float zmax = kNegInf;
#pragma unroll
  for (int j = 0; j < EPL; ++j) {
    const int e = j * kWave + lane;
    z[j] = e < E ? clean_logit(load_logit(logits + static_cast<size_t>(t) * E + e)) : kNegInf;
    if (bias != nullptr && e < E && !(bias[e] > kNegInf)) z[j] = kNegInf;
    zmax = fmaxf(zmax, z[j]);
  }
  zmax = wave_max(zmax);
  double s[EPL], key[EPL], total = 0.0;
#pragma unroll
  for (int j = 0; j < EPL; ++j) {
    const bool on = z[j] > kNegInf;
    if (score == 1)
      s[j] = on ? 1.0 / (1.0 + exp(-static_cast<double>(z[j]))) : 0.0;
    else
      s[j] = on ? exp(static_cast<double>(z[j]) - static_cast<double>(zmax)) : 0.0;
    total += s[j];
  }
  if (score == 0) {
    total = wave_sum(total);
#pragma unroll
    for (int j = 0; j < EPL; ++j) s[j] = total > 0.0 ? s[j] / total : 0.0;
  }
#pragma unroll
  for (int j = 0; j < EPL; ++j) {
    const int e = j * kWave + lane;
    const bool on = z[j] > kNegInf;
    const double v = s[j] + (bias != nullptr && e < E ? static_cast<double>(bias[e]) : 0.0);
    key[j] = !on ? ninf : (bias != nullptr ? v : static_cast<double>(z[j]));
    if (e < E) v_lds[e] = on ? v : ninf;
  }
  if (n_group > 1) {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    const int n = E / n_group;
    double gs = ninf;
    if (lane < n_group) {
      double a = ninf, b = ninf;
      for (int i = 0; i < n; ++i) {
        const double v = v_lds[lane * n + i];
        if (v > a) {
          b = a;
          a = v;
        } else if (v > b) {
          b = v;
        }
      }
      if (a > ninf) gs = rint((b > ninf ? a + b : a) * 0x1p40);
    }
    int above = 0;
    for (int g = 0; g < n_group; ++g) {
      const double o = __shfl(gs, g);
      above += o > gs || (o == gs && g < lane);
    }
    const uint64_t kept = wave_ballot(lane < n_group && above < topk_group);
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
      const int e = j * kWave + lane;
      if (e < E && !((kept >> (e / n)) & 1)) key[j] = ninf;
    }
  }
  // the K best, one after the other; lane k keeps entry k
  int my_id = -1;
  float my_z = kNegInf;
  double my_s = 0.0;
  for (int k = 0; k < K; ++k) {
    double best = ninf;
    int at = 1 << 30;
#pragma unroll
    for (int j = 0; j < EPL; ++j)
      if (key[j] > best) {
        best = key[j];
        at = j * kWave + lane;
      }
    wave_argmax(best, at);
    if (!(best > ninf)) break;
    float bz = 0.0f;
    double bs = 0.0;
#pragma unroll
    for (int j = 0; j < EPL; ++j)
      if (j * kWave + lane == at) {
        key[j] = ninf;
        bz = z[j];
        bs = s[j];
      }
    bz = __shfl(bz, at & (kWave - 1));
    bs = __shfl(bs, at & (kWave - 1));
    if (lane == k) {
      my_id = at;
      my_z = bz;
      my_s = bs;
    }
  }
  if (renorm) {
    // q = s / sum s, each s divided by exp(min(zmax of the chosen, 0)) first
    // so that very negative logits do not underflow together
    const double m = wave_max(my_z);
    double u = 0.0;
    if (my_id >= 0) {
      const double zz = my_z;
      u = score == 1 ? exp(fmin(zz, 0.0) - fmin(m, 0.0)) / (1.0 + exp(-fabs(zz))) : exp(zz - m);
    }
    my_s = u;
    const double sum = wave_sum(u);
    if (sum > 0.0) my_s = u / sum;
  }
  if (lane < K) {
    ids[static_cast<size_t>(t) * K + lane] = my_id;
    weights[static_cast<size_t>(t) * K + lane] = my_id >= 0 ? static_cast<float>(scale * my_s) : 0.0f;
  }
}

__device__ __forceinline__ void store_grad(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_grad(uint16_t* p, float v) {
  *p = __builtin_bit_cast(uint16_t, static_cast<__bf16>(v));
}

template <typename Z, int EPL>
__global__ __launch_bounds__(kThreads) void route_backward_kernel(
    const float* __restrict__ grad_w, const Z* __restrict__ logits, const int32_t* __restrict__ ids, int32_t T,
    int32_t E, int32_t K, int32_t score, int32_t renorm, float scale, Z* __restrict__ grad) {
  const int lane = threadIdx.x & (kWave - 1);
  const int t = blockIdx.x * kWaves + threadIdx.x / kWave;
  if (t >= T) return;
  const Z* zrow = logits + static_cast<size_t>(t) * E;
  int id = lane < K ? ids[static_cast<size_t>(t) * K + lane] : -1;
  if (id >= E) id = -1;
  const float zk = id >= 0 ? clean_logit(load_logit(zrow + id)) : kNegInf;
  const bool on = zk > kNegInf;
  const float g = on ? grad_w[static_cast<size_t>(t) * K + lane] : 0.0f;
  const bool dense = score == 0 && !renorm;
  float p[EPL], zmax = kNegInf, inv = 0.0f;
  if (dense) {
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
      const int e = j * kWave + lane;
      p[j] = e < E ? clean_logit(load_logit(zrow + e)) : kNegInf;
      zmax = fmaxf(zmax, p[j]);
    }
    zmax = wave_max(zmax);
    float sum = 0.0f;
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
      p[j] = p[j] > kNegInf ? expf(p[j] - zmax) : 0.0f;
      sum += p[j];
    }
    sum = wave_sum(sum);
    inv = sum > 0.0f ? 1.0f / sum : 0.0f;
  }
  float d = 0.0f, dsum = 0.0f;
  if (renorm) {
    const float m = wave_max(zk);
    float u = 0.0f, rest = 1.0f;
    if (on) {
      if (score == 1) {
        const float e = expf(-fabsf(zk));
        u = expf(fminf(zk, 0.0f) - fminf(m, 0.0f)) / (1.0f + e);
        rest = (zk > 0.0f ? e : 1.0f) / (1.0f + e);  // 1 - s
      } else {
        u = expf(zk - m);
      }
    }
    const float sum = wave_sum(u);
    const float q = on ? u / sum : 0.0f;
    dsum = wave_sum(g * q);
    d = on ? scale * q * rest * (g - dsum) : 0.0f;
  } else if (score == 1) {
    if (on) {
      const float e = expf(-fabsf(zk));
      d = scale * g * e / ((1.0f + e) * (1.0f + e));
    }
  } else {
    const float pk = on ? expf(zk - zmax) * inv : 0.0f;
    d = scale * g;
    dsum = wave_sum(scale * g * pk);
  }
  float o[EPL];
#pragma unroll
  for (int j = 0; j < EPL; ++j) o[j] = 0.0f;
  for (int k = 0; k < K; ++k) {
    const int e = __shfl(on ? id : -1, k);
    const float dk = __shfl(d, k);
#pragma unroll
    for (int j = 0; j < EPL; ++j)
      if (j * kWave + lane == e) o[j] += dk;
  }
#pragma unroll
  for (int j = 0; j < EPL; ++j) {
    const int e = j * kWave + lane;
    if (e < E) store_grad(grad + static_cast<size_t>(t) * E + e, dense ? p[j] * inv * (o[j] - dsum) : o[j]);
  }
}

template <typename Z>
hipError_t route(const Z* logits, const float* bias, int32_t T, int32_t E, int32_t K, int32_t n_group,
                 int32_t topk_group, int32_t score, int32_t renorm, float scale, int32_t* ids, float* weights,
                 hipStream_t stream) {
  const dim3 grid((T + kWaves - 1) / kWaves), block(kThreads);
  const size_t lds = static_cast<size_t>(kWaves) * E * sizeof(double);
  const auto launch = [&](auto epl) {
    hipLaunchKernelGGL((route_kernel<Z, decltype(epl)::value>), grid, block, lds, stream, logits, bias, T, E, K,
                       n_group, topk_group, score, renorm, scale, ids, weights);
  };
  if (E <= 64) launch(std::integral_constant<int, 1>{});
  else if (E <= 128) launch(std::integral_constant<int, 2>{});
  else if (E <= 256) launch(std::integral_constant<int, 4>{});
  else if (E <= 512) launch(std::integral_constant<int, 8>{});
  else launch(std::integral_constant<int, 16>{});
  return hipGetLastError();
}

template <typename Z>
hipError_t route_backward(const float* grad_w, const Z* logits, const int32_t* ids, int32_t T, int32_t E, int32_t K,
                          int32_t score, int32_t renorm, float scale, Z* grad, hipStream_t stream) {
  const dim3 grid((T + kWaves - 1) / kWaves), block(kThreads);
  const auto launch = [&](auto epl) {
    hipLaunchKernelGGL((route_backward_kernel<Z, decltype(epl)::value>), grid, block, 0, stream, grad_w, logits, ids,
                       T, E, K, score, renorm, scale, grad);
  };
  if (E <= 64) launch(std::integral_constant<int, 1>{});
  else if (E <= 128) launch(std::integral_constant<int, 2>{});
  else if (E <= 256) launch(std::integral_constant<int, 4>{});
  else if (E <= 512) launch(std::integral_constant<int, 8>{});
  else launch(std::integral_constant<int, 16>{});
  return hipGetLastError();
}

}  // namespace

hipError_t launch_route(const void* logits, bool bf16, const float* bias, int32_t T, int32_t E, int32_t K,
                        int32_t n_group, int32_t topk_group, int32_t score, bool renorm, float scale, int32_t* ids,
                        float* weights, hipStream_t stream) {
  if (T == 0) return hipSuccess;
  return bf16 ? route(static_cast<const uint16_t*>(logits), bias, T, E, K, n_group, topk_group, score, renorm, scale,
                      ids, weights, stream)
              : route(static_cast<const float*>(logits), bias, T, E, K, n_group, topk_group, score, renorm, scale,
                      ids, weights, stream);
}

hipError_t launch_route_backward(const float* grad_w, const void* logits, bool bf16, const int32_t* ids, int32_t T,
                                 int32_t E, int32_t K, int32_t score, bool renorm, float scale, void* grad,
                                 hipStream_t stream) {
  if (T == 0) return hipSuccess;
  return bf16 ? route_backward(grad_w, static_cast<const uint16_t*>(logits), ids, T, E, K, score, renorm, scale,
                               static_cast<uint16_t*>(grad), stream)
              : route_backward(grad_w, static_cast<const float*>(logits), ids, T, E, K, score, renorm, scale,
                               static_cast<float*>(grad), stream);
}

}  // namespace ep
