// Routing: router logits to the expert ids and weights the dispatch takes,
// and the gradient of those weights.  The rule is stated at ep_route in
// include/ep.h.
//
// The choice is defined on binary64 scores, the work is done in binary32: see
// "the binary32 path" below.

#include <hip/hip_runtime.h>

#include "../../include/ep.h"
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

struct RouteArgs {
  const float* bias;
  int32_t* ids;
  float* weights;
  int32_t T, E, K, n_group, topk_group, score, renorm;
  float scale;
};

// One token in binary64, by a whole wavefront: the rule as it stands.  Lane l
// holds experts l, l + 64, ..; EPL of them.  v_lds: E doubles of the wavefront.
template <typename Z, int EPL>
__device__ __attribute__((noinline)) void route_token(const Z* __restrict__ logits, const RouteArgs A, int t,
                                                      double* v_lds) {
  const float* bias = A.bias;
  const int E = A.E, K = A.K, n_group = A.n_group, topk_group = A.topk_group, score = A.score;
  const int lane = threadIdx.x & (kWave - 1);
  const double ninf = -__builtin_inf();
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
  if (A.renorm) {
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
    A.ids[static_cast<size_t>(t) * K + lane] = my_id;
    A.weights[static_cast<size_t>(t) * K + lane] = my_id >= 0 ? static_cast<float>(A.scale * my_s) : 0.0f;
  }
}

// ---- the binary32 path --------------------------------------------------------
//
// LPT lanes per token (two tokens in a wavefront up to 256 experts), EPL
// neighbouring experts in each lane, sorted there once; the K best are then
// taken one by one: the largest head over the lanes (a butterfly of DPP and
// lane swaps), and its lane drops it.  A lane holds neighbours in index order,
// so the lowest lane among equal heads is the lowest index.
//
// Without a bias experts are compared by their logits, which is exact.  Group
// scores, and scores with a bias, are compared in binary32; where two that
// matter lie nearer than their rounding errors, the token is done again by
// route_token.

// Largest value of the LPT lanes, in all of them.
template <int LPT>
__device__ __forceinline__ uint32_t lanes_max(uint32_t v) {
  const auto dpp = [](uint32_t x, auto ctrl) {
    return static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(x), decltype(ctrl)::value, 0xF, 0xF, false));
  };
  v = max(v, dpp(v, std::integral_constant<int, 0xB1>{}));   // neighbour
  v = max(v, dpp(v, std::integral_constant<int, 0x4E>{}));   // neighbouring pair
  v = max(v, dpp(v, std::integral_constant<int, 0x141>{}));  // half row mirrored
  v = max(v, dpp(v, std::integral_constant<int, 0x140>{}));  // row mirrored
  const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
  v = max(r[0], r[1]);
  if (LPT == 64) {
    const auto q = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    v = max(q[0], q[1]);
  }
  return v;
}

template <int LPT>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
  for (int d = 1; d < LPT; d <<= 1) v += __shfl_xor(v, d);
  return v;
}

// Binary32 values as unsigned numbers of the same order (0 below all of them).
__device__ __forceinline__ uint32_t order_bits(float z) {
  const uint32_t u = __float_as_uint(z + 0.0f);  // -0 counts as +0
  return u ^ (static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float from_order(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}

// e^z with a relative error of a few units of binary32's last place.
__device__ __forceinline__ float sigmoid32(float z) {
  const float e = expf(-fabsf(z));
  return (z >= 0.0f ? 1.0f : e) / (1.0f + e);
}

template <int EPL>
__device__ __forceinline__ void sort_desc(uint64_t (&k)[EPL]) {
  const auto ce = [&](int i, int j) {
    const bool sw = k[j] > k[i];
    const uint64_t hi = sw ? k[j] : k[i], lo = sw ? k[i] : k[j];
    k[i] = hi;
    k[j] = lo;
  };
  // odd-even merge sort, unrolled
#pragma unroll
  for (int p = 1; p < EPL; p <<= 1)
#pragma unroll
    for (int q = p; q >= 1; q >>= 1)
#pragma unroll
      for (int j = q % p; j + q < EPL; j += 2 * q)
#pragma unroll
        for (int i = 0; i < q; ++i)
          if (i + j + q < EPL && (i + j) / (2 * p) == (i + j + q) / (2 * p)) ce(i + j, i + j + q);
}

// EPL neighbouring logits from p on (those below n of the row).
template <int EPL>
__device__ __forceinline__ void load_logits(const float* p, int n, bool vec, float (&z)[EPL]) {
  if (EPL >= 4 && vec) {  // rows and pieces aligned to 16 bytes, EPL divides E
    if (n <= 0) return;
#pragma unroll
    for (int i = 0; i < EPL / 4; ++i) {
      const float4 v = reinterpret_cast<const float4*>(p)[i];
      z[4 * i % EPL] = v.x;
      z[(4 * i + 1) % EPL] = v.y;
      z[(4 * i + 2) % EPL] = v.z;
      z[(4 * i + 3) % EPL] = v.w;
    }
  } else {
#pragma unroll
    for (int j = 0; j < EPL; ++j)
      if (j < n) z[j] = p[j];
  }
}
template <int EPL>
__device__ __forceinline__ void load_logits(const uint16_t* p, int n, bool vec, float (&z)[EPL]) {
  if (EPL >= 8 && vec) {
    if (n <= 0) return;
#pragma unroll
    for (int i = 0; i < EPL / 8; ++i) {
      const u32x4 v = reinterpret_cast<const u32x4*>(p)[i];
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        z[(8 * i + 2 * x) % EPL] = bf16_lo(v[x]);
        z[(8 * i + 2 * x + 1) % EPL] = bf16_hi(v[x]);
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < EPL; ++j)
      if (j < n) z[j] = bf16_lo(p[j]);
  }
}

template <typename Z, int EPL, int LPT, bool BIAS>
__global__ __launch_bounds__(kThreads) void route_kernel(const Z* __restrict__ logits, RouteArgs A, bool vec) {
  extern __shared__ double route_lds[];  // per wave: E doubles (route_token; the groups' scan of binary32 keys)
  constexpr int TPW = kWave / LPT;       // tokens per wavefront
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
  const int sub = lane & (LPT - 1), half = TPW == 2 ? lane >> 5 : 0;
  const int E = A.E, K = A.K;
  const int t0 = (blockIdx.x * kWaves + wave) * TPW;
  if (t0 >= A.T) return;  // no barrier below: the wavefronts are independent
  const int t = min(t0 + half, A.T - 1);  // (the last token twice where T is odd)
  double* v_lds = route_lds + static_cast<size_t>(wave) * E;
  const int e0 = sub * EPL;
  float z[EPL];
#pragma unroll
  for (int j = 0; j < EPL; ++j) z[j] = kNegInf;
  load_logits<EPL>(logits + static_cast<size_t>(t) * E + e0, E - e0, vec, z);
  bool near = false;  // a comparison that binary32 cannot decide
  float zmax = kNegInf, inv = 0.0f;
#pragma unroll
  for (int j = 0; j < EPL; ++j) {
    z[j] = clean_logit(z[j]);
    if (BIAS && e0 + j < E && !(A.bias[e0 + j] > kNegInf)) z[j] = kNegInf;
    zmax = fmaxf(zmax, z[j]);
  }
  const bool softmax = A.score == 0;
  if (softmax) {  // the sum over all experts that are on
    zmax = from_order(max(lanes_max<LPT>(order_bits(zmax)), 0x00800000u));
    float sum = 0.0f;
#pragma unroll
    for (int j = 0; j < EPL; ++j) sum += z[j] > kNegInf ? expf(z[j] - zmax) : 0.0f;
    sum = lanes_sum<LPT>(sum);
    inv = sum > 0.0f ? 1.0f / sum : 0.0f;
  }
  const auto score_of = [&](float x) {
    return !(x > kNegInf) ? 0.0f : (softmax ? expf(x - zmax) * inv : sigmoid32(x));
  };
  // (key, index from behind): largest first, ties to the lower index; 0: off
  uint64_t k[EPL];
#pragma unroll
  for (int j = 0; j < EPL; ++j) {
    const float v = BIAS && e0 + j < E ? score_of(z[j]) + A.bias[e0 + j] : z[j];
    k[j] = z[j] > kNegInf ? static_cast<uint64_t>(order_bits(v)) << 32 | static_cast<uint32_t>(EPL - 1 - j) : 0;
  }

  if (A.n_group > 1) {
    // two largest of each group, by the lanes of a token in turn over groups
    const int n = E / A.n_group;
    uint32_t* key_lds = reinterpret_cast<uint32_t*>(v_lds) + half * E;  // 2 E words a wavefront
#pragma unroll
    for (int j = 0; j < EPL; ++j)
      if (e0 + j < E) key_lds[e0 + j] = static_cast<uint32_t>(k[j] >> 32);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    // P lanes per group, P a power of two; rounds where LPT lanes are too few
    float mine = 0.0f;   // the score of group `sub` (and of sub + LPT where LPT < n_group)
    float mine2 = 0.0f;
    float mag = 1.0f;    // largest magnitude that goes into a score
    bool any = false, any2 = false;
    int P = 1;
    while (P * 2 * A.n_group <= LPT && P < 16) P *= 2;
    for (int g0 = 0; g0 < A.n_group; g0 += LPT / P) {
      const int g = g0 + sub / P;
      uint32_t b0 = 0, b1 = 0;
      if (g < A.n_group)
        for (int i = sub & (P - 1); i < n; i += P) {
          const uint32_t x = key_lds[g * n + i];
          b1 = max(b1, min(b0, x));
          b0 = max(b0, x);
        }
      for (int d = 1; d < P; d <<= 1) {
        const uint32_t o0 = __shfl_xor(b0, d), o1 = __shfl_xor(b1, d);
        b1 = max(max(b1, o1), min(b0, o0));
        b0 = max(b0, o0);
      }
      float gs = 0.0f;
      if (b0) gs += BIAS ? from_order(b0) : score_of(from_order(b0));
      if (b1) gs += BIAS ? from_order(b1) : score_of(from_order(b1));
      if (BIAS) {
        if (b0) mag = fmaxf(mag, fabsf(from_order(b0)));
        if (b1) mag = fmaxf(mag, fabsf(from_order(b1)));
      }
      // group g's score to lane g (of the token)
      const int src = (lane & ~(LPT - 1)) + ((sub - g0) * P & (LPT - 1));
      const float got = __shfl(gs, src);
      const bool on = __shfl(static_cast<int>(b0 != 0), src) != 0;
      if (sub >= g0 && sub < g0 + LPT / P && sub < A.n_group) {
        mine = got;
        any = on;
      }
      if (LPT < 64 && sub + LPT >= g0 && sub + LPT < g0 + LPT / P && sub + LPT < A.n_group) {
        mine2 = got;
        any2 = on;
      }
    }
    // each lane ranks its group (its two groups)
    int above = 0, above2 = 0;
    const auto beats = [](float a, bool ao, int ai, float b, bool bo, int bi) {
      return ao && (!bo || a > b || (a == b && ai < bi));
    };
    for (int g = 0; g < A.n_group; ++g) {
      const int src = (lane & ~(LPT - 1)) + (g & (LPT - 1));
      const float o = g < LPT ? __shfl(mine, src) : __shfl(mine2, src);
      const bool oo = (g < LPT ? __shfl(static_cast<int>(any), src) : __shfl(static_cast<int>(any2), src)) != 0;
      above += beats(o, oo, g, mine, any, sub);
      above2 += beats(o, oo, g, mine2, any2, sub + LPT);
    }
    const bool keep = sub < A.n_group && any && above < A.topk_group;
    const bool keep2 = LPT < 64 && sub + LPT < A.n_group && any2 && above2 < A.topk_group;
    const uint64_t m1 = wave_ballot(keep), m2 = wave_ballot(keep2);
    const uint64_t kept = LPT == 64 ? m1 : ((m1 >> (half * 32)) & 0xFFFFFFFFull) | (m2 >> (half * 32)) << 32;
    // the last kept score against the first dropped one
    const uint32_t low_bits = ~0u;
    uint32_t worst = 0, best = 0;  // order bits; the smallest kept as the largest complement
    if (sub < A.n_group && any) (keep ? worst : best) = keep ? low_bits - order_bits(mine) : order_bits(mine);
    if (LPT < 64 && sub + LPT < A.n_group && any2) {
      if (keep2) worst = max(worst, low_bits - order_bits(mine2));
      else best = max(best, order_bits(mine2));
    }
    worst = lanes_max<LPT>(worst);
    best = lanes_max<LPT>(best);
    if (best != 0) {
      const float lo = from_order(low_bits - worst), hi = from_order(best);
      // binary32 is off by a few units of 2^-24 of what is added up, the rule's
      // own rounding by half of 2^-40
      if (BIAS) mag = from_order(lanes_max<LPT>(order_bits(mag)));
      near = lo - hi <= (BIAS ? 0x1p-19f * mag : 0x1p-19f * fmaxf(lo, hi) + 0x1p-38f);
    }
#pragma unroll
    for (int j = 0; j < EPL; ++j)
      if (e0 + j < E && !((kept >> ((e0 + j) / n)) & 1)) k[j] = 0;
  }

  sort_desc(k);

  // the K best (with a bias one more, for the last comparison); lane i of the
  // token keeps entry i's key, the winner's lane writes its index
  int* id_lds = reinterpret_cast<int*>(route_lds + static_cast<size_t>(kWaves) * E) + (wave * 2 + half) * EP_MAX_TOPK;
  if (sub < K && sub < EP_MAX_TOPK) id_lds[sub] = -1;
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  uint32_t my_key = 0, before = 0;
  bool tie = false;
  for (int i = 0; i < K + (BIAS ? 1 : 0); ++i) {
    const uint32_t head = static_cast<uint32_t>(k[0] >> 32);
    const uint32_t m = lanes_max<LPT>(head);
    const bool eq = head == m && m != 0;
    const uint64_t mask = wave_ballot(eq);
    const uint32_t lower = LPT == 64 ? lanes_below(mask)
                                     : (half ? __builtin_amdgcn_mbcnt_hi(static_cast<uint32_t>(mask >> 32), 0u)
                                             : __builtin_amdgcn_mbcnt_lo(static_cast<uint32_t>(mask), 0u));
    const bool win = eq && lower == 0;
    if (BIAS && i > 0 && m != 0 && before != 0) {
      const float hi = from_order(before), lo = from_order(m);
      tie = tie || hi - lo <= 0x1p-20f * fmaxf(1.0f, fmaxf(fabsf(hi), fabsf(lo)));
    }
    before = m;
    if (i == K) break;
    if (win) {
      id_lds[i] = e0 + EPL - 1 - static_cast<int>(static_cast<uint32_t>(k[0]));
#pragma unroll
      for (int j = 0; j + 1 < EPL; ++j) k[j] = k[j + 1];
      k[EPL - 1] = 0;
    }
    my_key = sub == i ? m : my_key;
  }
  near = near || tie;
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");

  const int id = sub < K && sub < EP_MAX_TOPK ? id_lds[sub] : -1;
  float zk = kNegInf;
  if (id >= 0) zk = BIAS ? clean_logit(load_logit(logits + static_cast<size_t>(t) * E + id)) : from_order(my_key);
  float q = 0.0f;
  if (A.renorm) {
    // s / sum s, each s divided by exp(min(largest chosen logit, 0)) first so
    // that very negative logits do not underflow together
    const float m = from_order(max(lanes_max<LPT>(order_bits(zk)), 0x00800000u));
    if (id >= 0) q = softmax ? expf(zk - m) : expf(fminf(zk, 0.0f) - fminf(m, 0.0f)) / (1.0f + expf(-fabsf(zk)));
    const float sum = lanes_sum<LPT>(q);
    if (sum > 0.0f) q /= sum;
  } else if (id >= 0) {
    q = score_of(zk);
  }
  if (sub < K && t0 + half < A.T && !near) {
    A.ids[static_cast<size_t>(t) * K + sub] = id;
    A.weights[static_cast<size_t>(t) * K + sub] = A.scale * q;
  }
  // tokens that binary32 could not decide
  uint64_t again = wave_ballot(near);
  for (int h = 0; h < TPW; ++h) {
    if (((again >> (h * 32)) & 1) == 0 || t0 + h >= A.T) continue;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    route_token<Z, (EPL * LPT + kWave - 1) / kWave>(logits, A, t0 + h, v_lds);
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
hipError_t route(const Z* logits, const RouteArgs& A, hipStream_t stream) {
  // per wave: E doubles, and the ids of its tokens
  const size_t lds = static_cast<size_t>(kWaves) * (A.E * sizeof(double) + 2 * EP_MAX_TOPK * sizeof(int));
  const auto launch = [&](auto epl, auto lpt) {
    constexpr int EPL = decltype(epl)::value, LPT = decltype(lpt)::value, tokens = kWaves * (kWave / LPT);
    const dim3 grid((A.T + tokens - 1) / tokens), block(kThreads);
    const bool vec = A.E % EPL == 0 && A.E * sizeof(Z) % 16 == 0 && (reinterpret_cast<uintptr_t>(logits) & 15) == 0;
    if (A.bias != nullptr)
      hipLaunchKernelGGL((route_kernel<Z, EPL, LPT, true>), grid, block, lds, stream, logits, A, vec);
    else
      hipLaunchKernelGGL((route_kernel<Z, EPL, LPT, false>), grid, block, lds, stream, logits, A, vec);
    return hipGetLastError();
  };
  const std::integral_constant<int, 32> two{};
  const std::integral_constant<int, 64> one{};
  if (A.E <= 64) return launch(std::integral_constant<int, 2>{}, two);
  if (A.E <= 128) return launch(std::integral_constant<int, 4>{}, two);
  if (A.E <= 256) return launch(std::integral_constant<int, 8>{}, two);
  if (A.E <= 512) return launch(std::integral_constant<int, 8>{}, one);
  return launch(std::integral_constant<int, 16>{}, one);
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
  const RouteArgs A{bias, ids, weights, T, E, K, n_group, topk_group, score, renorm, scale};
  return bf16 ? route(static_cast<const uint16_t*>(logits), A, stream)
              : route(static_cast<const float*>(logits), A, stream);
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
