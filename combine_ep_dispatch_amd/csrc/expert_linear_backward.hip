// The gradient of the experts' bf16 layers with respect to their rows, and on
// through the gated activation that made them.  The contract is
// ep_expert_linear_backward's in include/ep.h.

#include "linear_tile.h"

namespace ep {
namespace {

// The tile, as for the layer itself; microseconds, * as the rule picks, with E 256,
// N 4096 to H 7168, 8 experts a token (p: N 7168 to H 2048 through the activation):
//   tokens (mean rows)  512 (16)  1024 (32)  2048 (64)  3000 (94)  4096 (128) p  4096 popular
//   64 x 128                2711       2854       3385       4226          2583          5351
//   128 x 128               2655       2827       3148       3364          2590          4505
//   128 x 256               2635       2771       2934       3038          2492          4052
//   192 x 256              *2518      *2616      *2761      *2947         *1593         *3846
//   256 x 256               2730       2844       3027       3145          1760          4023
// and for one matrix:
//   rows                 128   512  1024  2048  4096
//   64 x 128, 2 groups *24.0  45.3
//   64 x 128            25.3  47.4  93.8   177   330
//   128 x 128           30.7 *35.1  66.4   128   240
//   128 x 256           45.8  48.2 *58.1   115   224
//   256 x 256           74.0  76.6  79.3  *102  *202
// (7168 to 2048, through the activation, 64 x 128: 128 rows 35.0 in two groups and 40.8
// in one, 1024 rows 41.9 and 46.6; 256 to 256: 7.9 both ways.)
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
  if (s.tiles(64, g.O, 128) <= s.cus)
    return launch_tiles<kRows, GATED, __bf16, 64, 128, 2, 2, 3, 3, 1, false, 2>(g, stream);
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
