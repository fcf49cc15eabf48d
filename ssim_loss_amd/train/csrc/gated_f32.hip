// The gated layer's kernels for fp32.
#include "gated.hpp"

const ssim_train::GatedTable& ssim_train::gated_table_f32() {
  static const GatedTable table = make_gated_table<F32>();
  return table;
}
