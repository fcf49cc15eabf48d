// The joint's kernels for blocks of fp32.
#include "block_norm.hpp"

const ssim_train::NormTable& ssim_train::norm_table_f32() {
  static const NormTable table = make_table<F32>();
  return table;
}
