// Routing: router logits to the expert ids and weights the dispatch takes,
// and the gradient of those weights.  The rule is stated at ep_route in
// include/ep.h.
//
// The choice is defined on binary64 scores, the work is done in binary32: see
// "the binary32 path" below.
//
// A wavefront takes two tokens up to 256 experts (one beyond), each lane
// holding consecutive experts in registers: memory is read once, in order, and
// the choice is vector work between lanes, which is what bounds it.  32768
// tokens of 256 experts in BF16, sigmoid, 4 of 8 groups, top 8: 28.1 us
// (17 MB in, 2 MB out: 3 us at the rate of a copy; softmax 31.4, with a bias
// 33 and 36); wholly in binary64, with one token a wavefront, it was 94.  128 tokens are as fast as the host calls
// (11 us).

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

template <int LPT, typename T>
__device__ __forceinline__ T lanes_sum(T v) {
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

struct RouteArgs {
  const float* bias;
  int32_t* ids;
  float* weights;
  int32_t T, E, K, n_group, topk_group, score, renorm;
  float scale;
};

// Binary64 values as unsigned numbers of the same order (0 below all of them).
__device__ __forceinline__ uint64_t order_bits(double v) {
  const int64_t u = __double_as_longlong(v + 0.0);
  return static_cast<uint64_t>(u ^ ((u >> 63) | static_cast<int64_t>(0x8000000000000000ull)));
}

// Largest of the wavefront's values, in all lanes.
__device__ __forceinline__ uint64_t wave_max_u64(uint64_t v) {
  const uint32_t hi = lanes_max<64>(static_cast<uint32_t>(v >> 32));
  const uint32_t lo = lanes_max<64>(static_cast<uint32_t>(v >> 32) == hi ? static_cast<uint32_t>(v) : 0u);
  return static_cast<uint64_t>(hi) << 32 | lo;
}

// A group's score: the sum of its two largest v, a >= b (b = -inf: of its only
// one), to 40 binary places below the larger one's magnitude, so that sums
// that are equal in exact arithmetic tie whatever the exponentials' last bits.
__device__ __forceinline__ double group_score(double a, double b) {
  const bool two = b > -__builtin_inf();
  const double sum = two ? a + b : a, m = fmax(fabs(a), two ? fabs(b) : 0.0);
  if (!(m < __builtin_inf())) return sum;
  int e;
  frexp(m, &e);  // 2^(e-1) <= m < 2^e
  return ldexp(rint(ldexp(sum, 41 - e)), e - 41);
}

// One token in binary64, by a whole wavefront: the rule as it stands.  Lane l
// holds experts l * EPL ..; v_lds: E doubles of the wavefront, sum_lds: room
// for EP_MAX_GROUPS doubles.
template <typename Z, int EPL>
__device__ __attribute__((noinline)) void route_token(const Z* __restrict__ logits, const RouteArgs A, int t,
                                                      double* v_lds, double* sum_lds) {
  const int lane = threadIdx.x & (kWave - 1), E = A.E, e0 = lane * EPL;
  const double ninf = -__builtin_inf();
  float z[EPL], zmax = kNegInf;
#pragma unroll
  for (int j = 0; j < EPL; ++j) {
    const int e = e0 + j;
    z[j] = e < E ? clean_logit(load_logit(logits + static_cast<size_t>(t) * E + e)) : kNegInf;
    zmax = fmaxf(zmax, z[j]);
  }
  double s[EPL], total = 0.0;
  if (A.score == 0) zmax = wave_max(zmax);
#pragma unroll
  for (int j = 0; j < EPL; ++j) {
    const double zz = z[j];
    s[j] = !(z[j] > kNegInf) ? 0.0 : (A.score == 1 ? 1.0 / (1.0 + exp(-zz)) : exp(zz - static_cast<double>(zmax)));
    total += s[j];
  }
  if (A.score == 0) {
    total = wave_sum(total);
#pragma unroll
    for (int j = 0; j < EPL; ++j) s[j] = total > 0.0 ? s[j] / total : 0.0;
  }
  uint64_t key[EPL];
#pragma unroll
  for (int j = 0; j < EPL; ++j) {
    const float bias = A.bias != nullptr && e0 + j < E ? A.bias[e0 + j] : 0.0f;
    const bool on = z[j] > kNegInf && bias > kNegInf;
    const double v = s[j] + static_cast<double>(bias);
    key[j] = !on ? 0 : order_bits(A.bias != nullptr ? v : static_cast<double>(z[j]));
    if (e0 + j < E) v_lds[e0 + j] = on ? v : ninf;
  }
  if (A.n_group > 1) {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    const int n = E / A.n_group;
    int P = 1;  // lanes per group
    while (P * 2 * A.n_group <= kWave) P *= 2;
    double a = ninf, b = ninf;
    const int g = lane / P;
    if (g < A.n_group)
      for (int i = lane & (P - 1); i < n; i += P) {
        const double v = v_lds[g * n + i];
        b = fmax(b, fmin(a, v));
        a = fmax(a, v);
      }
    for (int d = 1; d < P; d <<= 1) {
      const double oa = __shfl_xor(a, d), ob = __shfl_xor(b, d);
      b = fmax(fmax(b, ob), fmin(a, oa));
      a = fmax(a, oa);
    }
    const double gs = a > ninf ? group_score(a, b) : ninf;
    if (g < A.n_group && (lane & (P - 1)) == 0) sum_lds[g] = gs;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    const double mine = lane < A.n_group ? sum_lds[lane] : ninf;
    int above = 0;
    for (int o = 0; o < A.n_group; ++o) {
      const double x = sum_lds[o];
      above += x > mine || (x == mine && o < lane);
    }
    const uint64_t kept = wave_ballot(lane < A.n_group && mine > ninf && above < A.topk_group);
    int ge = e0 / n, r = e0 - ge * n;
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
      if (!((kept >> (ge & 63)) & 1)) key[j] = 0;
      if (++r == n) {
        r = 0;
        ++ge;
      }
    }
  }
  // the K best, one after the other; the winner's lane hands its values to
  // lane k (a lane holds neighbours in index order: the lowest lane among
  // equal keys is the lowest index)
  int my_id = -1;
  float my_z = kNegInf;
  double my_s = 0.0;
  for (int k = 0; k < A.K; ++k) {
    uint64_t best = 0;
    int at = 0;
    float bz = 0.0f;
    double bs = 0.0;
#pragma unroll
    for (int j = 0; j < EPL; ++j)
      if (key[j] > best) {
        best = key[j];
        at = j;
        bz = z[j];
        bs = s[j];
      }
    const uint64_t m = wave_max_u64(best);
    if (m == 0) break;
    const int w = __builtin_ctzll(wave_ballot(best == m));
    if (lane == w) {
#pragma unroll
      for (int j = 0; j < EPL; ++j)
        if (j == at) key[j] = 0;
    }
    const int id = __shfl(e0 + at, w);
    bz = __shfl(bz, w);
    bs = __shfl(bs, w);
    if (lane == k) {
      my_id = id;
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
      u = A.score == 1 ? exp(fmin(zz, 0.0) - fmin(m, 0.0)) / (1.0 + exp(-fabs(zz))) : exp(zz - m);
    }
    my_s = u;
    const double sum = wave_sum(u);
    if (sum > 0.0) my_s = u / sum;
  }
  if (lane < A.K) {
    A.ids[static_cast<size_t>(t) * A.K + lane] = my_id;
    A.weights[static_cast<size_t>(t) * A.K + lane] = my_id >= 0 ? static_cast<float>(A.scale * my_s) : 0.0f;
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

// Errors below are relative, in units of 2^-24, at most; those of the helpers
// were measured over every binary32 argument of their range.

// e^(z + rest), |rest| <= 2^-17, 0 where it leaves the normal range: exp2 of
// z log2(e), whose rounding error is put back with rest.  2.9 units.
__device__ __forceinline__ float exp32(float z, float rest = 0.0f) {
  const float y = z * 0x1.715476p+0f;
  const float r = __builtin_fmaf(z, 0x1.4ae0bep-26f, __builtin_fmaf(z, 0x1.715476p+0f, -y));
  const float e = __builtin_amdgcn_exp2f(y);
  return __builtin_fmaf(e * __builtin_fmaf(rest, 0x1.715476p+0f, r), 0x1.62e430p-1f, e);
}

// e^(x - m), x <= m: the difference's rounding error, up to 2^-18 for logits
// 64 to 128 apart, goes into the exponential with it.  2.9 units; 0 for x =
// -inf and below e^-150.
__device__ __forceinline__ float exp32_diff(float x, float m) {
  const float d = x - m;
  const float b = d - x;
  const float rest = (x - (d - b)) + (-m - b);
  return d > -150.0f ? exp32(d, rest) : 0.0f;
}

// 1 / (1 + e^-z).  4.3 units.
__device__ __forceinline__ float sigmoid32(float z) {
  const float e = exp32(fmaxf(-fabsf(z), -150.0f));
  return (z >= 0.0f ? 1.0f : e) * __builtin_amdgcn_rcpf(1.0f + e);
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
__global__ __launch_bounds__(kThreads) void route_kernel(const Z* __restrict__ logits, RouteArgs A, bool vec, bool vec_bias) {
  extern __shared__ double route_lds[];  // per wave: E doubles (route_token; the groups' scan of binary32 keys)
  constexpr int TPW = kWave / LPT;       // tokens per wavefront
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
  const int sub = lane & (LPT - 1), half = TPW == 2 ? lane >> 5 : 0;
  const int E = A.E, K = A.K;
  const int t0 = (blockIdx.x * kWaves + wave) * TPW;
  if (t0 >= A.T) return;  // no barrier below: the wavefronts are independent
  const int t = min(t0 + half, A.T - 1);  // (the last token twice where T is odd)
  double* v_lds = route_lds + static_cast<size_t>(wave) * E;
  // ids of the wave's tokens, 2 x EP_MAX_TOPK (before that their groups' sums, 2 x EP_MAX_GROUPS)
  int* id_lds = reinterpret_cast<int*>(route_lds + static_cast<size_t>(kWaves) * E) + wave * 2 * EP_MAX_GROUPS + half * EP_MAX_TOPK;
  const int e0 = sub * EPL;
  float z[EPL];
#pragma unroll
  for (int j = 0; j < EPL; ++j) z[j] = kNegInf;
  load_logits<EPL>(logits + static_cast<size_t>(t) * E + e0, E - e0, vec, z);
  float bias[EPL];
  if constexpr (BIAS) {
#pragma unroll
    for (int j = 0; j < EPL; ++j) bias[j] = 0.0f;
    load_logits<EPL>(A.bias + e0, E - e0, vec_bias, bias);
  }
  bool near = false;  // a comparison that binary32 cannot decide
  float zmax = kNegInf, inv = 0.0f;
#pragma unroll
  for (int j = 0; j < EPL; ++j) {
    z[j] = clean_logit(z[j]);
    zmax = fmaxf(zmax, z[j]);
  }
  const bool softmax = A.score == 0;
  if (softmax) {  // the sum over all experts, those that the bias switches off among them
    zmax = from_order(max(lanes_max<LPT>(order_bits(zmax)), 0x00800000u));
    double sum = 0.0;  // (in binary32 up to 21 additions would each be off by 2^-24 of the sum)
#pragma unroll
    for (int j = 0; j < EPL; ++j) sum += exp32_diff(z[j], zmax);  // (0 for -inf)
    sum = lanes_sum<LPT>(sum);
    inv = sum > 0.0 ? 1.0f / static_cast<float>(sum) : 0.0f;
  }
  const auto score_of = [&](float x) {
    return softmax ? exp32_diff(x, zmax) * inv : sigmoid32(x);
  };
  // (key, index from behind): largest first, ties to the lower index; 0: off
  uint64_t k[EPL];
#pragma unroll
  for (int j = 0; j < EPL; ++j) {
    const float v = BIAS ? score_of(z[j]) + bias[j] : z[j];
    k[j] = z[j] > kNegInf && (!BIAS || bias[j] > kNegInf) ? static_cast<uint64_t>(order_bits(v)) << 32 | static_cast<uint32_t>(EPL - 1 - j) : 0;
  }

  // Groups of whole lanes, a power of two of them, have their two largest in
  // the sorted lanes' heads; others go through LDS and are sorted afterwards.
  const int n = A.n_group > 1 ? E / A.n_group : E;
  const int lanes = n / EPL;  // lanes per group
  const bool whole = n % EPL == 0 && (lanes & (lanes - 1)) == 0 && lanes <= 16;
  if (whole || A.n_group == 1) sort_desc(k);
  if (A.n_group > 1) {
    uint32_t* sum_lds = reinterpret_cast<uint32_t*>(id_lds) - half * EP_MAX_TOPK + half * EP_MAX_GROUPS;
    for (int g = sub; g < EP_MAX_GROUPS; g += LPT) sum_lds[g] = 0;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    float mag = 1.0f;  // largest magnitude that goes into a sum
    // the sum of a group's two largest, as order bits (0: nobody to choose)
    const auto add_up = [&](uint32_t b0, uint32_t b1) {
      const float v0 = from_order(b0), v1 = from_order(b1);
      float gs = BIAS ? v0 : score_of(v0);
      if (b1 != 0) gs += BIAS ? v1 : score_of(v1);
      if (BIAS && b0 != 0) mag = fmaxf(fmaxf(mag, fabsf(v0)), b1 != 0 ? fabsf(v1) : 0.0f);
      return b0 != 0 ? order_bits(gs) : 0u;
    };
    uint32_t b0 = 0, b1 = 0;
    const auto merge = [&](auto ctrl) {
      constexpr int C = decltype(ctrl)::value;
      const uint32_t o0 = __builtin_amdgcn_update_dpp(0, static_cast<int>(b0), C, 0xF, 0xF, false);
      const uint32_t o1 = __builtin_amdgcn_update_dpp(0, static_cast<int>(b1), C, 0xF, 0xF, false);
      b1 = max(max(b1, o1), min(b0, o0));
      b0 = max(b0, o0);
    };
    if (whole) {
      b0 = static_cast<uint32_t>(k[0] >> 32);
      b1 = EPL > 1 ? static_cast<uint32_t>(k[EPL > 1 ? 1 : 0] >> 32) : 0;
      if (lanes >= 2) merge(std::integral_constant<int, 0xB1>{});
      if (lanes >= 4) merge(std::integral_constant<int, 0x4E>{});
      if (lanes >= 8) merge(std::integral_constant<int, 0x141>{});
      if (lanes >= 16) merge(std::integral_constant<int, 0x140>{});
      const uint32_t sum = add_up(b0, b1);
      if (e0 < E && (sub & (lanes - 1)) == 0) sum_lds[sub / lanes] = sum;
    } else {
      uint32_t* key_lds = reinterpret_cast<uint32_t*>(v_lds) + half * E;  // 2 E words a wavefront
#pragma unroll
      for (int j = 0; j < EPL; ++j)
        if (e0 + j < E) key_lds[e0 + j] = static_cast<uint32_t>(k[j] >> 32);
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      // P neighbouring lanes per group, in rounds where a token's lanes are too few
      const int P = A.n_group * 4 <= LPT ? 4 : (A.n_group * 2 <= LPT ? 2 : 1);
      for (int g0 = 0; g0 < A.n_group; g0 += LPT / P) {
        const int g = g0 + sub / P;
        b0 = b1 = 0;
        if (g < A.n_group)
          for (int i = sub & (P - 1); i < n; i += P) {
            const uint32_t x = key_lds[g * n + i];
            b1 = max(b1, min(b0, x));
            b0 = max(b0, x);
          }
        if (P >= 2) merge(std::integral_constant<int, 0xB1>{});
        if (P >= 4) merge(std::integral_constant<int, 0x4E>{});
        const uint32_t sum = add_up(b0, b1);
        if (g < A.n_group && (sub & (P - 1)) == 0) sum_lds[g] = sum;
      }
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    // each lane ranks group `sub` (and sub + LPT): how many come before it
    const bool more = LPT < EP_MAX_GROUPS && A.n_group > LPT;
    const uint32_t mine = sum_lds[sub], mine2 = more ? sum_lds[(sub + LPT) % EP_MAX_GROUPS] : 0;
    int above = 0, above2 = 0;
    for (int g = 0; g < A.n_group; g += 4) {  // (sums past the last group are 0)
      const u32x4 o = *reinterpret_cast<const u32x4*>(sum_lds + g);
#pragma unroll
      for (int x = 0; x < 4; ++x) {  // a tie goes to the lower group
        above += o[x] > mine - (g + x < sub ? 1u : 0u);
        if (more) above2 += o[x] > mine2 - (g + x < sub + LPT ? 1u : 0u);
      }
    }
    const bool keep = mine != 0 && above < A.topk_group;
    const bool keep2 = mine2 != 0 && above2 < A.topk_group;
    const uint64_t m1 = wave_ballot(keep), m2 = more ? wave_ballot(keep2) : 0;
    const uint64_t kept = LPT == 64 ? m1 : ((m1 >> (half * 32)) & 0xFFFFFFFFull) | (m2 >> (half * 32)) << 32;
    // the last kept sum against the first dropped one: the smallest kept as
    // the largest complement
    const uint32_t worst = lanes_max<LPT>(max(keep ? ~mine : 0u, keep2 ? ~mine2 : 0u));
    const uint32_t best = lanes_max<LPT>(max(keep ? 0u : mine, keep2 ? 0u : mine2));
    if (BIAS) mag = from_order(lanes_max<LPT>(order_bits(mag)));
    if (best != 0) {
      const float lo = from_order(~worst), hi = from_order(best);
      // a score is off by at most 8.8 units of itself (softmax: its exponential,
      // the sum's, and three roundings; sigmoid 4.3), a sum of two by one more,
      // with a bias by 13 of mag in all (two additions to it, and their sum):
      // 32 units part them; the rule's own rounding is 2^-41.  Scores that
      // leave the normal range are off by up to 2^-126; sums that leave it
      // (huge biases) say nothing.
      const float gap = lo - hi;
      near = !(gap > (BIAS ? 0x1p-19f * mag : 0x1p-19f * fmaxf(lo, hi) + 0x1p-120f) && gap < __builtin_inff());
    }
    if (whole) {
      if (!((kept >> (sub / lanes & 63)) & 1)) {
#pragma unroll
        for (int j = 0; j < EPL; ++j) k[j] = 0;
      }
    } else {
      int g = e0 / n, r = e0 - g * n;
#pragma unroll
      for (int j = 0; j < EPL; ++j) {
        if (!((kept >> (g & 63)) & 1)) k[j] = 0;
        if (++r == n) {
          r = 0;
          ++g;
        }
      }
      sort_desc(k);
    }
  }

  // the K best (with a bias one more, for the last comparison); lane i of the
  // token keeps entry i's key, the winner's lane writes its index
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  if (sub < K) id_lds[sub] = -1;
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  uint32_t my_key = 0, before = 0;
  bool tie = false;
  uint32_t head[EPL];  // the sorted keys, and their places in the lane, four bits each
  uint64_t place = 0;
#pragma unroll
  for (int j = 0; j < EPL; ++j) {
    head[j] = static_cast<uint32_t>(k[j] >> 32);
    place |= static_cast<uint64_t>((EPL - 1 - static_cast<uint32_t>(k[j])) & 15) << (4 * j);
  }
  for (int i = 0; i < K + (BIAS ? 1 : 0); ++i) {
    const uint32_t m = lanes_max<LPT>(head[0]);
    const bool eq = head[0] == m && m != 0;
    const uint64_t mask = wave_ballot(eq);
    const uint32_t lower = LPT == 64 ? lanes_below(mask)
                                     : (half ? __builtin_amdgcn_mbcnt_hi(static_cast<uint32_t>(mask >> 32), 0u)
                                             : __builtin_amdgcn_mbcnt_lo(static_cast<uint32_t>(mask), 0u));
    if (BIAS && i > 0 && m != 0 && before != 0) {
      const float hi = from_order(before), lo = from_order(m);
      // two scores of a token are off by at most 8.8 units together (softmax:
      // of their sum, at most 1; sigmoid: 4.3 of each), and each by one more
      // for the bias: 16 units part them
      tie = tie || hi - lo <= 0x1p-20f * fmaxf(1.0f, fmaxf(fabsf(hi), fabsf(lo)));
    }
    before = m;
    if (i == K) break;
    if (eq && lower == 0) {
      id_lds[i] = e0 + static_cast<int>(static_cast<uint32_t>(place) & 15);
#pragma unroll
      for (int j = 0; j + 1 < EPL; ++j) head[j] = head[j + 1];
      head[EPL - 1] = 0;
      if (EPL <= 8) place = static_cast<uint32_t>(place) >> 4; else place >>= 4;
    }
    my_key = sub == i ? m : my_key;
  }
  near = near || tie;
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");

  const int id = sub < K ? id_lds[sub] : -1;
  float zk = kNegInf;
  if (id >= 0) zk = BIAS ? clean_logit(load_logit(logits + static_cast<size_t>(t) * E + id)) : from_order(my_key);
  float q = 0.0f;
  if (A.renorm) {
    // s / sum s, each s divided by exp(min(largest chosen logit, 0)) first so
    // that very negative logits do not underflow together
    const float m = from_order(max(lanes_max<LPT>(order_bits(zk)), 0x00800000u));
    // 6.4 units each (the exponential, 1 + e, the division), as many again in
    // their sum, and three roundings: within 16
    if (id >= 0) {
      q = softmax ? exp32_diff(zk, m) : exp32_diff(fminf(zk, 0.0f), fminf(m, 0.0f));
      if (!softmax) q /= 1.0f + exp32(fmaxf(-fabsf(zk), -150.0f));
    }
    const float sum = static_cast<float>(lanes_sum<LPT>(static_cast<double>(q)));
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
    route_token<Z, (EPL * LPT + kWave - 1) / kWave>(logits, A, t0 + h, v_lds,
                                                    reinterpret_cast<double*>(id_lds - half * EP_MAX_TOPK));
  }
}

__device__ __forceinline__ void store_grad(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_grad(uint16_t* p, float v) {
  *p = __builtin_bit_cast(uint16_t, static_cast<__bf16>(v));
}

// e^(x - m) with the difference's rounding error, up to 2^-18, put back.
__device__ __forceinline__ float exp_diff(float x, float m) {
  const float d = x - m;
  const float b = d - x;
  const float rest = (x - (d - b)) + (-m - b);
  const float e = expf(d);
  return d > -150.0f ? __builtin_fmaf(e, rest, e) : 0.0f;
}

// A wavefront per token; a lane holds experts 64 apart, so that a row leaves in
// whole runs, and picks the K entries' terms out of the other lanes in order of
// k: an id that occurs twice is added up the same way every time, without
// atomics.  Sums are binary32 (softmax's over all experts binary64); a BF16
// gradient is rounded once, as it is stored.  Bounded by vector work and by its stores: 32768 tokens of 256
// experts in binary32, sigmoid, top 8: 18 us for 34 MB written (6 us at the
// rate of a fill); softmax without renormalisation, which reads them all, 26.
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
    double sum = 0.0;
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
      p[j] = p[j] > kNegInf ? exp_diff(p[j], zmax) : 0.0f;
      sum += p[j];
    }
    sum = wave_sum(sum);
    inv = sum > 0.0 ? 1.0f / static_cast<float>(sum) : 0.0f;
  }
  float d = 0.0f, dsum = 0.0f;
  if (renorm) {
    const float m = wave_max(zk);
    float u = 0.0f, rest = 1.0f;
    if (on) {
      if (score == 1) {
        const float e = expf(-fabsf(zk));
        u = exp_diff(fminf(zk, 0.0f), fminf(m, 0.0f)) / (1.0f + e);
        rest = (zk > 0.0f ? e : 1.0f) / (1.0f + e);  // 1 - s
      } else {
        u = exp_diff(zk, m);
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
    const float pk = on ? exp_diff(zk, zmax) * inv : 0.0f;
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
  // per wave: E doubles, and the groups' sums or the ids of its tokens
  const size_t lds = static_cast<size_t>(kWaves) * (A.E * sizeof(double) + 2 * EP_MAX_GROUPS * sizeof(int));
  static_assert(EP_MAX_TOPK <= EP_MAX_GROUPS && EP_MAX_TOPK <= 32, "a lane per entry");
  const auto launch = [&](auto epl, auto lpt) {
    constexpr int EPL = decltype(epl)::value, LPT = decltype(lpt)::value, tokens = kWaves * (kWave / LPT);
    const dim3 grid((A.T + tokens - 1) / tokens), block(kThreads);
    const bool vec = A.E % EPL == 0 && A.E * sizeof(Z) % 16 == 0 && (reinterpret_cast<uintptr_t>(logits) & 15) == 0;
    const bool vec_bias = A.E % EPL == 0 && EPL % 4 == 0 && (reinterpret_cast<uintptr_t>(A.bias) & 15) == 0;
    if (A.bias != nullptr)
      hipLaunchKernelGGL((route_kernel<Z, EPL, LPT, true>), grid, block, lds, stream, logits, A, vec, vec_bias);
    else
      hipLaunchKernelGGL((route_kernel<Z, EPL, LPT, false>), grid, block, lds, stream, logits, A, vec, vec_bias);
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
