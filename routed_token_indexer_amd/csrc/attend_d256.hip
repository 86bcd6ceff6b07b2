// Attention over a paged cache, head dimension 256.
#include "attend_kernel.hpp"

namespace misa {

hipError_t launch_attend_d256(const AttendArgs& a, int R, bool half, unsigned blocks, hipStream_t st) {
  return attend::launch_dim<256>(a, R, half, blocks, st);
}

}  // namespace misa
