// Attention's kernels for fp16.
#include "attention.hpp"

const ssim_train::AttentionTable& ssim_train::attention_table_f16() {
  static const AttentionTable table = make_attention_table<F16>();
  return table;
}
