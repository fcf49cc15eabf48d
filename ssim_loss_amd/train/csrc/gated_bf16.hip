// The gated layer's kernels for bf16.
#include "gated.hpp"

const ssim_train::GatedTable& ssim_train::gated_table_bf16() {
  static const GatedTable table = make_gated_table<BF16>();
  return table;
}
