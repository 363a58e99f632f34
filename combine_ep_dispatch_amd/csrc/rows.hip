// Rows in microscaled 4-bit floating point: quantisation, dequantisation,
// and the dispatch that quantises tokens as it copies them to their experts.
// Also the FP8 rows of ep_quantize_rows / ep_dequantize_rows (the dispatch's
// own quantiser, on rows in their own order).
//
// MXFP4 (OCP microscaling formats v1.0): 32 channels share a power-of-two
// scale 2^e, e = floor(log2 amax) - 2, and each is E2M1_RNE(x / 2^e),
// saturating at 6.  Data movement only: 2 bytes read and 0.53 written per
// channel (per copy, for the dispatch).  The dispatch holds a whole group in
// one lane, so that a copy is one 16-byte store: 4096 tokens of 7168 to 8
// experts in 34 us, 5.4 TB/s (30 at best).

#include "ep_device.h"
#include "ep_internal.h"
#include "mx_device.h"

namespace ep {
namespace {

constexpr int kThreads = 256;

// Rows larger than the 256 MB Infinity Cache are read with non-temporal loads
// (65536 x 7168: 206 -> 178 us); what may still lie in it is not (32747 x 2048:
// 24 us against 27).  Dequantised rows that do not fit the L2s leave with
// non-temporal stores (65536 x 7168: 208 -> 162 us, 7.3 TB/s).
constexpr int64_t kReadOnceBytes = int64_t(256) << 20;
constexpr int64_t kWriteOnceBytes = int64_t(32) << 20;

template <bool ONCE, typename V>
__device__ __forceinline__ V load_row(const V* p) {
  return ONCE ? __builtin_nontemporal_load(p) : *p;
}
template <bool ONCE, typename V>
__device__ __forceinline__ void store_row(V v, V* p) {
  if (ONCE) __builtin_nontemporal_store(v, p); else *p = v;
}

// Four neighbouring lanes hold a group, 8 channels each, so that every load
// is a whole wavefront's run of memory.
constexpr int kQuantItems = 4;  // 8-channel items per lane, a workgroup apart

template <bool ONCE>
__global__ __launch_bounds__(kThreads) void quantize_mxfp4_kernel(const u32x4* __restrict__ x, uint32_t n_items,
                                                                  uint32_t* __restrict__ q, uint8_t* __restrict__ scale) {
  const uint32_t first = blockIdx.x * (kThreads * kQuantItems) + threadIdx.x;
  u32x4 a[kQuantItems];
#pragma unroll
  for (int i = 0; i < kQuantItems; ++i) {
    const uint32_t item = first + i * kThreads;
    a[i] = u32x4{0, 0, 0, 0};
    if (item < n_items) a[i] = load_row<ONCE>(x + item);  // n_items is a multiple of 4: whole groups
  }
#pragma unroll
  for (int i = 0; i < kQuantItems; ++i) {
    const uint32_t item = first + i * kThreads;
    uint32_t s;
    const uint32_t c = quantize8_mxfp4(a[i], s);
    if (item < n_items) {
      q[item] = c;
      if ((item & 3) == 0) scale[item >> 2] = static_cast<uint8_t>(s);
    }
  }
}

// Work item = (row, 16 channels); 8 lanes share a 128-channel group.
__global__ __launch_bounds__(kThreads) void quantize_fp8_kernel(const uint16_t* __restrict__ x, uint32_t n_items,
                                                                u32x4* __restrict__ q, float* __restrict__ scale) {
  const uint32_t item = blockIdx.x * kThreads + threadIdx.x;
  const bool active = item < n_items;  // n_items is a multiple of 8: whole groups
  u32x4 a = {0, 0, 0, 0}, b = {0, 0, 0, 0};
  if (active) {
    const u32x4* src = reinterpret_cast<const u32x4*>(x) + static_cast<size_t>(item) * 2;
    a = src[0];
    b = src[1];
  }
  float s;
  const u32x4 c = quantize16_e4m3(a, b, s);
  if (!active) return;
  q[item] = c;
  if ((item & 7) == 0) scale[item >> 3] = s;
}

// Work item = 8 channels: 4 bytes of codes in, 16 bytes of BF16 out.
template <bool ONCE>
__global__ __launch_bounds__(kThreads) void dequantize_mxfp4_kernel(const uint32_t* __restrict__ q,
                                                                    const uint8_t* __restrict__ scale,
                                                                    uint32_t n_items, u32x4* __restrict__ x) {
  const uint32_t item = blockIdx.x * kThreads + threadIdx.x;
  if (item >= n_items) return;
  const uint32_t w = q[item];
  const float s = e8m0_to_f32(scale[item >> 2]);
  u32x4 o;
  o[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 0));
  o[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 1));
  o[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 2));
  o[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 3));
  store_row<ONCE>(o, x + item);
}

// Work item = 8 channels: 8 bytes of codes in, 16 bytes of BF16 out.
template <bool ONCE>
__global__ __launch_bounds__(kThreads) void dequantize_fp8_kernel(const uint2* __restrict__ q,
                                                                  const float* __restrict__ scale, uint32_t n_items,
                                                                  u32x4* __restrict__ x) {
  const uint32_t item = blockIdx.x * kThreads + threadIdx.x;
  if (item >= n_items) return;
  const uint2 w = q[item];
  const float s = scale[item >> 4];
  float f[8];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int v = static_cast<int>(h == 0 ? w.x : w.y);
    f[4 * h + 0] = __builtin_amdgcn_cvt_f32_fp8(v, 0);
    f[4 * h + 1] = __builtin_amdgcn_cvt_f32_fp8(v, 1);
    f[4 * h + 2] = __builtin_amdgcn_cvt_f32_fp8(v, 2);
    f[4 * h + 3] = __builtin_amdgcn_cvt_f32_fp8(v, 3);
  }
  u32x4 o;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const bf16x2 p = {static_cast<__bf16>(f[2 * i] * s), static_cast<__bf16>(f[2 * i + 1] * s)};
    o[i] = __builtin_bit_cast(uint32_t, p);
  }
  store_row<ONCE>(o, x + item);
}

// Dispatch: work item = (token, 32 channels), quantised once and written to
// the token's K rows.
__global__ __launch_bounds__(kThreads) void dispatch_mxfp4_kernel(
    const uint16_t* __restrict__ x, uint32_t n_items, uint32_t vpt, int32_t K, const int32_t* __restrict__ slot,
    const float* __restrict__ w, u32x4* __restrict__ recv, uint8_t* __restrict__ recv_scale,
    float* __restrict__ recv_weight) {
  const uint32_t item = blockIdx.x * kThreads + threadIdx.x;
  if (item >= n_items) return;
  const uint32_t t = item / vpt;
  const uint32_t v = item - t * vpt;
  const u32x4* src = reinterpret_cast<const u32x4*>(x) + static_cast<size_t>(item) * 4;
  u32x4 a[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) a[i] = src[i];
  uint32_t s;
  const u32x4 q = quantize32_mxfp4(a, s);
  const int32_t* srow = slot + static_cast<size_t>(t) * K;
  for (int k = 0; k < K; ++k) {
    const int32_t r = srow[k];
    if (r < 0) continue;
    const size_t at = static_cast<size_t>(r) * vpt + v;
    recv[at] = q;
    recv_scale[at] = static_cast<uint8_t>(s);
    if (recv_weight != nullptr && v == 0) recv_weight[r] = w[static_cast<size_t>(t) * K + k];
  }
}

dim3 grid_of(uint32_t items) { return dim3((items + kThreads - 1) / kThreads); }

}  // namespace

hipError_t launch_dispatch_mxfp4(const uint16_t* x, int32_t T, int32_t H, int32_t K, const int32_t* slot,
                                 const float* w, uint8_t* recv, uint8_t* recv_scale, float* recv_weight,
                                 hipStream_t stream) {
  const uint32_t vpt = static_cast<uint32_t>(H) / kMxGroup;
  const uint32_t n = static_cast<uint32_t>(T) * vpt;
  if (n == 0) return hipSuccess;
  hipLaunchKernelGGL(dispatch_mxfp4_kernel, grid_of(n), dim3(kThreads), 0, stream, x, n, vpt, K, slot, w,
                     reinterpret_cast<u32x4*>(recv), recv_scale, recv_weight);
  return hipGetLastError();
}

hipError_t launch_quantize_rows(const uint16_t* x, int64_t rows, int32_t H, bool fp8, void* q, void* scale,
                                hipStream_t stream) {
  const uint32_t n = static_cast<uint32_t>(rows * (H / (fp8 ? 16 : 8)));
  if (n == 0) return hipSuccess;
  if (fp8) {
    hipLaunchKernelGGL(quantize_fp8_kernel, grid_of(n), dim3(kThreads), 0, stream, x, n, static_cast<u32x4*>(q),
                       static_cast<float*>(scale));
    return hipGetLastError();
  }
  const dim3 grid((n + kThreads * kQuantItems - 1) / (kThreads * kQuantItems));
  const auto kernel = rows * H * 2 >= kReadOnceBytes ? quantize_mxfp4_kernel<true> : quantize_mxfp4_kernel<false>;
  hipLaunchKernelGGL(kernel, grid, dim3(kThreads), 0, stream, reinterpret_cast<const u32x4*>(x), n,
                     static_cast<uint32_t*>(q), static_cast<uint8_t*>(scale));
  return hipGetLastError();
}

hipError_t launch_dequantize_rows(const void* q, const void* scale, int64_t rows, int32_t H, bool fp8, uint16_t* x,
                                  hipStream_t stream) {
  const uint32_t n = static_cast<uint32_t>(rows * (H / 8));
  if (n == 0) return hipSuccess;
  const bool once = rows * H * 2 >= kWriteOnceBytes;
  u32x4* out = reinterpret_cast<u32x4*>(x);
  if (fp8) {
    const auto kernel = once ? dequantize_fp8_kernel<true> : dequantize_fp8_kernel<false>;
    hipLaunchKernelGGL(kernel, grid_of(n), dim3(kThreads), 0, stream, static_cast<const uint2*>(q),
                       static_cast<const float*>(scale), n, out);
  } else {
    const auto kernel = once ? dequantize_mxfp4_kernel<true> : dequantize_mxfp4_kernel<false>;
    hipLaunchKernelGGL(kernel, grid_of(n), dim3(kThreads), 0, stream, static_cast<const uint32_t*>(q),
                       static_cast<const uint8_t*>(scale), n, out);
  }
  return hipGetLastError();
}

}  // namespace ep
