// Attention's kernels for fp32.
#include "attention.hpp"

const ssim_train::AttentionTable& ssim_train::attention_table_f32() {
  static const AttentionTable table = make_attention_table<F32>();
  return table;
}
