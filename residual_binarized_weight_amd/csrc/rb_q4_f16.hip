// rb_q4_f16.hip -- the 4-bit product for fp16 activations.
#include "rb_q4_kernel.hpp"

namespace rb {
namespace q4 {

hipError_t launch_f16(const Args& a, int group, bool pair, hipStream_t s) {
  return pair ? launch_group<_Float16, true>(a, group, s) : launch_group<_Float16, false>(a, group, s);
}

}  // namespace q4
}  // namespace rb
