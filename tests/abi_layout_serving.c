/* Sizes and field offsets of the structures of the calls for many samples of one prompt (include/dflash2.h), one
 * "name value" per line, for the binding's layout test. */
#include <stddef.h>
#include <stdio.h>

#include "dflash2.h"

#define OFF(T, f) printf(#T "." #f " %zu\n", offsetof(T, f))
#define SIZE(T) printf(#T " %zu\n", sizeof(T))

int main(void) {
  SIZE(dflash2_rope_config);
  OFF(dflash2_rope_config, theta);
  OFF(dflash2_rope_config, amplitude);
  OFF(dflash2_rope_config, table);
  SIZE(dflash2_rotation);
  OFF(dflash2_rotation, amplitude);
  OFF(dflash2_rotation, turns);
  SIZE(dflash2_page_pool);
  OFF(dflash2_page_pool, table_stride);
  OFF(dflash2_page_pool, n_pages);
  OFF(dflash2_page_pool, page_size);
  SIZE(dflash2_paged_shared_args);
  OFF(dflash2_paged_shared_args, n_groups);
  OFF(dflash2_paged_shared_args, group_begin);
  OFF(dflash2_paged_shared_args, workspace);
  OFF(dflash2_paged_shared_args, workspace_bytes);
  return 0;
}
