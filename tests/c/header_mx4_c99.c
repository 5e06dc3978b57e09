/* Compile-and-link check of the MXFP4 and norm entry points of
 * include/convrot.h from plain C99: each is referenced with arguments of the
 * declared types. Nothing here is executed. */
#include <stddef.h>
#include <stdint.h>

#include "convrot.h"

int convrot_header_mx4_c99_check(void* p, int i) {
  convrot_status s = CONVROT_OK;
  uint8_t* c = (uint8_t*)p;
  convrot_norm_args a = {0};
  convrot_launch_plan plan;
  size_t n = convrot_mx4_scales_size(16, 256);
  if (i == 1) {
    s = convrot_quantize_mx4(p, CONVROT_DTYPE_BF16, 1, 256, 256, 1u, c, c, p);
    s = convrot_dequant_mx4(c, c, 1, 256, 1, 1u, p, CONVROT_DTYPE_F16, p);
    s = convrot_gemm_mx4(c, c, c, c, p, 1, 16, 256, p, CONVROT_DTYPE_BF16, 0, p);
    n += convrot_linear_mx4_workspace_for_rows(1, 256);
    n += convrot_linear_mx4_workspace_size(1, 16, 256);
    s = convrot_linear_mx4(p, c, c, p, 1, 16, 256, 256, 1u, p, CONVROT_DTYPE_BF16, p, n, p);
    a.x = p;
    a.h_codes = c;
    a.h_scales = c;
    a.m = 1;
    a.k = 256;
    a.g = 256;
    a.rows_per_mod = 1;
    a.gate_stride = a.scale_stride = a.shift_stride = 0;
    a.post_norm = CONVROT_NORM_NONE;
    a.norm = CONVROT_NORM_LAYER;
    a.dtype = CONVROT_DTYPE_F16;
    a.eps = 1e-6f;
    s = convrot_norm_residual(&a, p);
    s = convrot_plan_launch(CONVROT_KERNEL_GEMM_MX4, 1, 16, 256, 1, 0, &plan);
  }
  return (int)s + (int)n;
}
