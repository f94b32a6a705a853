// rb_q4_bf16.hip -- the 4-bit product for bf16 activations.
#include "rb_q4_kernel.hpp"

namespace rb {
namespace q4 {

hipError_t launch_bf16(const Args& a, int group, bool pair, hipStream_t s) {
  return pair ? launch_group<__bf16, true>(a, group, s) : launch_group<__bf16, false>(a, group, s);
}

}  // namespace q4
}  // namespace rb
