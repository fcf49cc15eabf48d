// The gated layer's kernels for fp16.
#include "gated.hpp"

const ssim_train::GatedTable& ssim_train::gated_table_f16() {
  static const GatedTable table = make_gated_table<F16>();
  return table;
}
