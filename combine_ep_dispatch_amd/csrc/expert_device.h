// Device-side helpers shared by the experts' kernels: the rows of an expert,
// copies straight to LDS, waits (gfx950, wave64).  Internal header.
#pragma once

#include "ep_device.h"
#include "expert_rows.h"

namespace ep {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr int kMaxExperts = 1024;

// Rows of expert e: [first, first + count), clamped to the buffer.
__device__ __forceinline__ void rows_of(const int32_t* __restrict__ expert_rows, int e, int capacity, int num_rows,
                                        int& first, int& count) {
  if (capacity > 0) {
    first = e * capacity;
    count = min(max(expert_rows[e], 0), capacity);
  } else {
    span_rows(expert_rows[e], expert_rows[e + 1], num_rows, first, count);
  }
}

__device__ __forceinline__ float silu_mul(float g, float u) { return g / (1.0f + __expf(-g)) * u; }

// start[0 .. E] to the sums before each, by the workgroup's first wavefront;
// every thread must call it.
__device__ __forceinline__ void tiles_before(RowTiles* start, int E) {
  if (threadIdx.x < kWave) {
    const int per = E / kWave + 1, beg = threadIdx.x * per, end = min(beg + per, E + 1);
    RowTiles mine = 0;
    for (int e = beg; e < end; ++e) mine += start[e];
    RowTiles run = mine;
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) {
      const RowTiles o = __shfl_up(run, d);
      if (static_cast<int>(threadIdx.x) >= d) run += o;
    }
    run -= mine;
    for (int e = beg; e < end; ++e) {
      const RowTiles n = start[e];
      start[e] = run;
      run += n;
    }
  }
  __syncthreads();
}

typedef __amdgpu_buffer_rsrc_t Rsrc;
typedef __attribute__((address_space(3))) void LdsVoid;

__device__ __forceinline__ Rsrc make_rsrc(const void* p, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, static_cast<int>(bytes), 0x00027000);
}

// 64 lanes x 16 bytes: lane l's piece lands at dst + 16 l.
__device__ __forceinline__ void copy16(Rsrc src, uint8_t* dst, uint32_t lane_off, uint32_t off) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(src, (LdsVoid*)dst, 16, lane_off, off, 0, 0);
}
// The same, non-temporal.
__device__ __forceinline__ void copy16_once(Rsrc src, uint8_t* dst, uint32_t lane_off, uint32_t off) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(src, (LdsVoid*)dst, 16, lane_off, off, 0, 2);
}

// Until at most N of this wave's copies are under way (they finish in order)
// and its LDS reads are done; then the workgroup's barrier.
template <int N>
__device__ __forceinline__ void wait_and_sync() {
  static_assert(N < 16, "vmcnt");
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(N | 7 << 4);  // vmcnt(N) lgkmcnt(0)
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// The workgroup's barrier once this wave's LDS reads are done.
__device__ __forceinline__ void wait_reads() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(15 | 7 << 4 | 3 << 14);  // lgkmcnt(0)
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// f(0) && f(1) && ...
template <int I, int N, typename F>
__device__ __forceinline__ bool static_while(F&& f) {
  if constexpr (I < N) {
    if (!f(std::integral_constant<int, I>{})) return false;
    return static_while<I + 1, N>(f);
  }
  return true;
}

}  // namespace ep
