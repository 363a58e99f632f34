// The gradients of the experts' bf16 layers with respect to their weights and
// biases.  The contract is ep_expert_linear_backward_weights' in include/ep.h.

#include "linear_tile.h"

namespace ep {
namespace {

// The tile, by the mean rows of an expert and by how many tiles there are (in
// microseconds, * as the rule picks, bf16):
//   experts x rows, N x H   256 x 128, 1024 x 2048   64 x 512, same   32 x 1024, 4096 x 7168   1 x 8192, 2048 x 2048
//   128 x 128                                  530              272                     2424                     *75
//   128 x 256                                 *426              206                     2010                     113
//   256 x 256                                  485             *210                    *1841                     206
// Few tiles of a long sum are not split: 512 x 512 over 32768 rows keeps 16
// workgroups busy for 205 us.
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
