// Attention over a paged cache, head dimension 64.
#include "attend_kernel.hpp"

namespace misa {

hipError_t launch_attend_d64(const AttendArgs& a, int R, bool half, unsigned blocks, hipStream_t st) {
  return attend::launch_dim<64>(a, R, half, blocks, st);
}

}  // namespace misa
