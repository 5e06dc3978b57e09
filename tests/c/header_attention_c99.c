/* Compile-and-link check of the rotary table, norm-and-rotation and attention
 * entry points of include/convrot.h from plain C99: each is referenced with
 * arguments of the declared types. Nothing here is executed. */
#include <stddef.h>
#include <stdint.h>

#include "convrot.h"

int convrot_header_attention_c99_check(void* p, int i) {
  convrot_status s = CONVROT_OK;
  convrot_qk_args h = {0};
  convrot_attention_args a = {0};
  const int32_t dims[3] = {16, 56, 56};
  size_t n = 0;
  if (i == 1) {
    s = convrot_rope_table(p, CONVROT_POSITION_I64, 3, 1, 1, 3, dims, 10000.0, 0, (float*)p, p);
    h.q = p;
    h.norm = CONVROT_NORM_RMS;
    h.dtype = CONVROT_DTYPE_F16;
    h.eps = 1e-6f;
    s = convrot_qk_norm_rope(&h, p);
    a.q = p;
    a.q_offsets = a.k_offsets = a.k_lens = (const int32_t*)p;
    a.lse = (float*)p;
    a.scale = 0.125f;
    a.dtype = CONVROT_DTYPE_BF16;
    n = convrot_attention_workspace_size(&a);
    s = convrot_attention(&a, p, n, p);
  }
  return (int)s + (int)n;
}
