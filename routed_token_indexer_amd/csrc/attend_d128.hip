// Attention over a paged cache, head dimension 128.
#include "attend_kernel.hpp"

namespace misa {

hipError_t launch_attend_d128(const AttendArgs& a, int R, bool half, unsigned blocks, hipStream_t st) {
  return attend::launch_dim<128>(a, R, half, blocks, st);
}

}  // namespace misa
