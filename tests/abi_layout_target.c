/* Sizes and field offsets of the structures of the target's side (include/dflash2.h), one
 * "name value" per line, for the binding's layout test. */
#include <stddef.h>
#include <stdio.h>

#include "dflash2.h"

#define OFF(T, f) printf(#T "." #f " %zu\n", offsetof(T, f))
#define SIZE(T) printf(#T " %zu\n", sizeof(T))

int main(void) {
  SIZE(dflash2_paged_config);
  OFF(dflash2_paged_config, kv_format);
  SIZE(dflash2_paged_cache);
  OFF(dflash2_paged_cache, page_table);
  OFF(dflash2_paged_cache, page_stride);
  OFF(dflash2_paged_cache, scale_head_stride);
  OFF(dflash2_paged_cache, table_stride);
  OFF(dflash2_paged_cache, max_pages);
  SIZE(dflash2_rows);
  OFF(dflash2_rows, type);
  SIZE(dflash2_paged_attention_args);
  OFF(dflash2_paged_attention_args, scale);
  OFF(dflash2_paged_attention_args, token_begin);
  OFF(dflash2_paged_attention_args, out);
  OFF(dflash2_paged_attention_args, tree_mask);
  OFF(dflash2_paged_attention_args, status);
  SIZE(dflash2_sample_args);
  OFF(dflash2_sample_args, logits);
  OFF(dflash2_sample_args, temperature);
  OFF(dflash2_sample_args, kept);
  OFF(dflash2_sample_args, status);
  return 0;
}
