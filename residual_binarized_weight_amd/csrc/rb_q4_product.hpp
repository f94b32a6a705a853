// rb_q4_product.hpp -- products with 4-bit weights for decode batches; compiled once per type of x.
//
// A block owns 16 weight rows (of both weights of a pair); its waves take the 128-column tiles in turn and join in
// LDS in their order. A code becomes a number of x's type by a shift and a mask: in the top four fraction bits above 16,
// it reads 16 + q. So a group's sum of products is s (D - 24 S), or s D + (z - 16 s) S with offsets, with D the matrix
// instructions' sum over 16 + q and S the sum of the group's x, which an instruction with ones for weights gives in
// the same lanes. All sums are fp32; 16 + q against q - 8 costs about two bits of them.
#pragma once

#include "rb_act.hpp"
#include "rb_internal.h"
#include "rb_tile.hpp"

namespace rb {
namespace q4 {

struct Weights {
  const uint32_t* codes;
  const _Float16 *s, *z;
};
struct Args {
  Weights w[2];
  const void* x;
  void* y;
  int64_t ldx, ldy, N, first;
  int M, K, steps, act;
  bool wide;  // y is fp32, else of x's type
};
// group 32, 64 or 128; M up to 16
hipError_t launch_f16(const Args& a, int group, bool pair, hipStream_t s);
hipError_t launch_bf16(const Args& a, int group, bool pair, hipStream_t s);

}  // namespace q4
}  // namespace rb
