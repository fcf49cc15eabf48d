// The joint's kernels for blocks of fp16.
#include "block_norm.hpp"

const ssim_train::NormTable& ssim_train::norm_table_f16() {
  static const NormTable table = make_table<F16>();
  return table;
}
