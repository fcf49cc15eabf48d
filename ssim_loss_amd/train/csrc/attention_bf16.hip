// Attention's kernels for bf16.
#include "attention.hpp"

const ssim_train::AttentionTable& ssim_train::attention_table_bf16() {
  static const AttentionTable table = make_attention_table<BF16>();
  return table;
}
