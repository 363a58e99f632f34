// The gradients of the experts' bf16 layers with respect to their weights and
// biases.  The contract is ep_expert_linear_backward_weights' in include/ep.h.

#include "linear_tile.h"

namespace ep {
namespace {

template <typename T>
hipError_t launch(const LinearArgs& g, hipStream_t stream) {
  const int64_t cus = max(device_cu_count(), 1);
  const auto fill = [&](int bm, int bn) {
    return static_cast<int64_t>(g.E) * ((g.M + bm - 1) / bm) * ((g.O + bn - 1) / bn) * 8 >= 7 * cus;
  };
  if (linear_shape(g).avg > 400 && fill(256, 256)) return launch_tiles<kWeights, false, T, 256, 256, 4, 2, 3, 2, 1>(g, stream);
  if (fill(128, 256)) return launch_tiles<kWeights, false, T, 128, 256, 2, 4, 3, 3, 1>(g, stream);
  return launch_tiles<kWeights, false, T, 128, 128, 2, 2, 4, 4, 1>(g, stream);
}

}  // namespace

hipError_t launch_expert_linear_backward_weights(const uint16_t* grad_y, const uint16_t* a, const int32_t* expert_rows,
                                                 int32_t num_rows, int32_t E, int32_t capacity, int32_t H, int32_t N,
                                                 bool bf16, bool add, void* grad_w, void* grad_bias,
                                                 hipStream_t stream) {
  const LinearArgs args{b16(a), b16(grad_y), nullptr, nullptr, expert_rows, num_rows, E, capacity, 0,
                        H, N, add, nullptr, grad_w, grad_bias};
  return bf16 ? launch<__bf16>(args, stream) : launch<float>(args, stream);
}

}  // namespace ep
