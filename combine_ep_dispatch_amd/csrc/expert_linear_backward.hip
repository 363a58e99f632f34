// The gradient of the experts' bf16 layers with respect to their rows, and on
// through the gated activation that made them.  The contract is
// ep_expert_linear_backward's in include/ep.h.

#include "linear_tile.h"

namespace ep {
namespace {

template <bool GATED>
hipError_t launch(const LinearArgs& g, hipStream_t stream) {
  const LinearShape s = linear_shape(g);
  if (s.avg > 170 && s.fill(256, g.O, 256)) {
    if (s.avg > 2048) return launch_tiles<kRows, GATED, __bf16, 256, 256, 4, 2, 2, 2, 1>(g, stream);
    return launch_tiles<kRows, GATED, __bf16, 256, 256, 4, 2, 3, 2, 1>(g, stream);
  }
  if (s.fill(192, g.O, 256)) return launch_tiles<kRows, GATED, __bf16, 192, 256, 2, 4, 3, 2, 1>(g, stream);
  if (s.fill(128, g.O, 256)) return launch_tiles<kRows, GATED, __bf16, 128, 256, 2, 4, 3, 3, 1>(g, stream);
  if (s.fill(128, g.O, 128)) return launch_tiles<kRows, GATED, __bf16, 128, 128, 2, 2, 4, 4, 1>(g, stream);
  return launch_tiles<kRows, GATED, __bf16, 64, 128, 2, 2, 6, 6, 1>(g, stream);
}

}  // namespace

hipError_t launch_expert_linear_backward(const uint16_t* grad_y, const uint16_t* w, const uint16_t* p,
                                         const int32_t* expert_rows, int32_t num_rows, int32_t E, int32_t capacity,
                                         int32_t H, int32_t N, uint16_t* grad_a, hipStream_t stream) {
  const LinearArgs g{b16(w), b16(grad_y), nullptr, nullptr, expert_rows, num_rows, E, capacity, N,
                     H, 0, false, const_cast<__bf16*>(b16(p)), grad_a, nullptr};
  return p != nullptr ? launch<true>(g, stream) : launch<false>(g, stream);
}

}  // namespace ep
