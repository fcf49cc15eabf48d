// The joint's kernels for blocks of bf16.
#include "block_norm.hpp"

const ssim_train::NormTable& ssim_train::norm_table_bf16() {
  static const NormTable table = make_table<BF16>();
  return table;
}
