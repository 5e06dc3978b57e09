// C ABI of the microscaled 4-bit layers and the gated residual norm: argument
// checks and slicing. Every check runs before any HIP call.

#include "api_common.h"
#include "mx4.h"

using namespace convrot;

namespace {

constexpr int64_t kMaxMx4K = 131072;
constexpr int64_t kMaxNormK = 16384;
constexpr int64_t kDefaultWorkspace = (int64_t)64 << 20;

size_t codes_bytes(int64_t rows, int64_t k) { return (size_t)(rows * (k / 2)); }
size_t scales_bytes(int64_t rows, int64_t k) {
  return (size_t)((k + kMx4Tile - 1) / kMx4Tile * mx4_pad_rows(rows) * 8);
}

// dimensions that some call takes
bool valid_size(int64_t rows, int64_t k) {
  return rows > 0 && rows < kMaxDim && k > 0 && k % kMx4Block == 0 && k <= kMaxMx4K;
}

bool valid_mx4_group(int g) { return g == 1 || valid_group(g); }

// rows x k quantized in groups of g (1: not rotated)
convrot_status check_mx4(const char* fn, int64_t rows, int64_t k, int g) {
  if (rows < 0 || k <= 0)
    return fail(CONVROT_E_INVALID_ARG, "%s: bad dims rows=%lld k=%lld", fn, (long long)rows,
                (long long)k);
  if (!valid_mx4_group(g))
    return fail(CONVROT_E_UNSUPPORTED_GROUP, "%s: g=%d not in {1,4,16,64,256}", fn, g);
  if (k % g)
    return fail(CONVROT_E_UNSUPPORTED_GROUP, "%s: k=%lld not a multiple of g=%d", fn,
                (long long)k, g);
  if (k % kMx4Block || k > kMaxMx4K || rows >= kMaxDim || !mx4_grid_fits(rows, k))
    return fail(CONVROT_E_UNSUPPORTED_SHAPE,
                "%s: need k %% 32 == 0, k <= %lld, ceil(rows/8) * ceil(k/256) < 2^26 "
                "(rows=%lld k=%lld)", fn, (long long)kMaxMx4K, (long long)rows, (long long)k);
  return CONVROT_OK;
}

}  // namespace

namespace convrot {

convrot_status check_mx4_gemm(const char* fn, int64_t m, int64_t n, int64_t k) {
  if (m < 0 || n <= 0 || k <= 0)
    return fail(CONVROT_E_INVALID_ARG, "%s: bad dims m=%lld n=%lld k=%lld", fn, (long long)m,
                (long long)n, (long long)k);
  if (k % kMx4Block || n % 16 || k > kMaxMx4K || m >= kMaxDim || n >= kMaxDim)
    return fail(CONVROT_E_UNSUPPORTED_SHAPE,
                "%s: need k %% 32 == 0, n %% 16 == 0, k <= %lld (m=%lld n=%lld k=%lld)", fn,
                (long long)kMaxMx4K, (long long)m, (long long)n, (long long)k);
  // grids: the tiles that the choice is left with fit far beyond this, 16 columns a block of
  // eight waves for few rows; the kernels' row indices run up to a tile beyond m and n
  if (((m + 63) / 64) * ((n + 63) / 64) * 4 > kMaxLaunchWaves || n / 16 * 8 > kMaxLaunchWaves ||
      m > kMaxDim - 1024)
    return fail(CONVROT_E_UNSUPPORTED_SHAPE, "%s: output too large (m=%lld n=%lld)", fn,
                (long long)m, (long long)n);
  return CONVROT_OK;
}

}  // namespace convrot

extern "C" {

size_t convrot_mx4_scales_size(int64_t rows, int64_t k) {
  if (!valid_size(rows, k)) return 0;
  return scales_bytes(rows, k);
}

convrot_status convrot_quantize_mx4(const void* x, convrot_dtype dtype, int64_t rows, int64_t k,
                                    int g, uint64_t rot_seed, uint8_t* codes, uint8_t* scales,
                                    void* stream) {
  const char* fn = "convrot_quantize_mx4";
  DType dt;
  if (!dtype_of(dtype, &dt)) return fail(CONVROT_E_INVALID_ARG, "%s: dtype=%d", fn, (int)dtype);
  if (convrot_status s = check_mx4(fn, rows, k, g)) return s;
  if (rows == 0) return ok();  // the buffers may be null
  if (!x || !codes || !scales) return fail(CONVROT_E_INVALID_ARG, "%s: null pointer", fn);
  if (!aligned(x, 16) || !aligned(codes, 16) || !aligned(scales, 16))
    return fail(CONVROT_E_MISALIGNED, "%s: misaligned pointer", fn);
  const size_t nx = (size_t)(rows * k) * 2, nc = codes_bytes(rows, k), ns = scales_bytes(rows, k);
  if (overlap(x, nx, codes, nc) || overlap(x, nx, scales, ns) || overlap(codes, nc, scales, ns))
    return fail(CONVROT_E_INVALID_ARG, "%s: overlapping buffers", fn);
  return hip_status(launch_mx4_quantize(static_cast<const uint16_t*>(x), rows, (int)k, g,
                                        make_signs(rot_seed, g), dt, codes, scales,
                                        (hipStream_t)stream),
                    fn);
}

convrot_status convrot_dequant_mx4(const uint8_t* codes, const uint8_t* scales, int64_t rows,
                                   int64_t k, int g, uint64_t rot_seed, void* out,
                                   convrot_dtype out_dtype, void* stream) {
  const char* fn = "convrot_dequant_mx4";
  DType dt;
  if (!dtype_of(out_dtype, &dt))
    return fail(CONVROT_E_INVALID_ARG, "%s: out_dtype=%d", fn, (int)out_dtype);
  if (convrot_status s = check_mx4(fn, rows, k, g)) return s;
  if (rows == 0) return ok();
  if (!codes || !scales || !out) return fail(CONVROT_E_INVALID_ARG, "%s: null pointer", fn);
  if (!aligned(codes, 16) || !aligned(scales, 16) || !aligned(out, 16))
    return fail(CONVROT_E_MISALIGNED, "%s: misaligned pointer", fn);
  const size_t no = (size_t)(rows * k) * 2;
  if (overlap(out, no, codes, codes_bytes(rows, k)) ||
      overlap(out, no, scales, scales_bytes(rows, k)))
    return fail(CONVROT_E_INVALID_ARG, "%s: overlapping buffers", fn);
  return hip_status(launch_mx4_dequant(codes, scales, rows, (int)k, g, make_signs(rot_seed, g),
                                       static_cast<uint16_t*>(out), dt, (hipStream_t)stream),
                    fn);
}

convrot_status convrot_gemm_mx4(const uint8_t* x_codes, const uint8_t* x_scales,
                                const uint8_t* w_codes, const uint8_t* w_scales,
                                const void* bias, int64_t m, int64_t n, int64_t k, void* y,
                                convrot_dtype dtype, int tile, void* stream) {
  const char* fn = "convrot_gemm_mx4";
  DType dt;
  if (!dtype_of(dtype, &dt)) return fail(CONVROT_E_INVALID_ARG, "%s: dtype=%d", fn, (int)dtype);
  if (tile != 0 && tile != 16 && tile != 40 && tile != 64 && tile != 96 && tile != 128 &&
      tile != 160 && tile != 192 && tile != 256 && tile != 384)
    return fail(CONVROT_E_INVALID_ARG, "%s: tile=%d not supported", fn, tile);
  if (tile == 16 && m > 64)
    return fail(CONVROT_E_INVALID_ARG, "%s: tile=16 takes at most 64 rows (m=%lld)", fn,
                (long long)m);
  if (convrot_status s = check_mx4_gemm(fn, m, n, k)) return s;
  if (tile != 0 && !mx4_gemm_grid_fits(m, n, tile))
    return fail(CONVROT_E_UNSUPPORTED_SHAPE, "%s: too many tiles for tile=%d (m=%lld n=%lld)", fn,
                tile, (long long)m, (long long)n);
  if (!w_codes || !w_scales) return fail(CONVROT_E_INVALID_ARG, "%s: null pointer", fn);
  if (m == 0) return ok();  // the M-sized buffers may be null
  if (!x_codes || !x_scales || !y) return fail(CONVROT_E_INVALID_ARG, "%s: null pointer", fn);
  if (!aligned(x_codes, 16) || !aligned(x_scales, 16) || !aligned(w_codes, 16) ||
      !aligned(w_scales, 16) || !aligned(y, 16) || (bias && !aligned(bias, 8)))
    return fail(CONVROT_E_MISALIGNED, "%s: misaligned pointer", fn);
  const size_t ny = (size_t)(m * n) * 2;
  if (overlap(y, ny, x_codes, codes_bytes(m, k)) || overlap(y, ny, x_scales, scales_bytes(m, k)) ||
      overlap(y, ny, w_codes, codes_bytes(n, k)) || overlap(y, ny, w_scales, scales_bytes(n, k)) ||
      overlap(y, ny, bias, (size_t)n * 2))
    return fail(CONVROT_E_INVALID_ARG, "%s: overlapping buffers", fn);
  return hip_status(launch_mx4_gemm(x_codes, x_scales, w_codes, w_scales,
                                    static_cast<const uint16_t*>(bias), m, n, k,
                                    static_cast<uint16_t*>(y), tile, dt, (hipStream_t)stream),
                    fn);
}

size_t convrot_linear_mx4_workspace_for_rows(int64_t rows, int64_t k) {
  if (!valid_size(rows, k)) return 0;
  return align_up(codes_bytes(rows, k), 256) + scales_bytes(rows, k);
}

size_t convrot_linear_mx4_workspace_size(int64_t m, int64_t n, int64_t k) {
  if (m < 0 || m >= kMaxDim || n % 16 || !valid_size(n, k)) return 0;
  // at least what 64 MiB hold: a narrow layer's short slices are bound by their
  // launches (5518 x 144 x 6080 in 13 slices of 432 rows 298 us, in one 30;
  // 21017 x 304 x 768 in 3 slices of 8192 rows 41 us, in one 23)
  const int64_t per_row = k / 2 + (k + kMx4Tile - 1) / kMx4Tile * 8;
  const int64_t held = kDefaultWorkspace / per_row;
  int64_t rows = 3 * n > held ? 3 * n : held;
  if (rows > m) rows = m < 1 ? 1 : m;
  return convrot_linear_mx4_workspace_for_rows(rows, k);
}

convrot_status convrot_linear_mx4(const void* x, const uint8_t* w_codes, const uint8_t* w_scales,
                                  const void* bias, int64_t m, int64_t n, int64_t k, int g,
                                  uint64_t rot_seed, void* y, convrot_dtype dtype,
                                  void* workspace, size_t workspace_bytes, void* stream) {
  const char* fn = "convrot_linear_mx4";
  DType dt;
  if (!dtype_of(dtype, &dt)) return fail(CONVROT_E_INVALID_ARG, "%s: dtype=%d", fn, (int)dtype);
  if (!w_codes || !w_scales) return fail(CONVROT_E_INVALID_ARG, "%s: null pointer", fn);
  if (convrot_status s = check_mx4(fn, m, k, g)) return s;
  if (convrot_status s = check_mx4_gemm(fn, m, n, k)) return s;
  if (m == 0) return ok();
  if (!x || !y || !workspace) return fail(CONVROT_E_INVALID_ARG, "%s: null pointer", fn);
  if (!aligned(x, 16) || !aligned(w_codes, 16) || !aligned(w_scales, 16) || !aligned(y, 16) ||
      (bias && !aligned(bias, 8)) || !aligned(workspace, 256))
    return fail(CONVROT_E_MISALIGNED, "%s: misaligned pointer", fn);
  // the largest slice that fits: whole 256-row GEMM tiles where there are several
  int64_t slice = m;
  if (convrot_linear_mx4_workspace_for_rows(m, k) > workspace_bytes) {
    // rounding up costs at most 256 bytes of codes and 15 padding rows of scales
    const size_t per_row = (size_t)(k / 2 + (k + kMx4Tile - 1) / kMx4Tile * 8);
    slice = (int64_t)(workspace_bytes / per_row);
    if (slice > m) slice = m;
    while (slice > 0 && convrot_linear_mx4_workspace_for_rows(slice, k) > workspace_bytes) --slice;
    if (slice < 1)
      return fail(CONVROT_E_WORKSPACE, "%s: %zu bytes hold no row (need %zu)", fn, workspace_bytes,
                  convrot_linear_mx4_workspace_for_rows(1, k));
    if (slice >= 256) slice -= slice % 256;
  }
  const size_t nx = (size_t)(m * k) * 2, ny = (size_t)(m * n) * 2;
  const size_t nc = codes_bytes(n, k), ns = scales_bytes(n, k);
  if (overlap(y, ny, x, nx) || overlap(y, ny, w_codes, nc) || overlap(y, ny, w_scales, ns) ||
      overlap(y, ny, bias, (size_t)n * 2) || overlap(y, ny, workspace, workspace_bytes) ||
      overlap(workspace, workspace_bytes, x, nx) ||
      overlap(workspace, workspace_bytes, w_codes, nc) ||
      overlap(workspace, workspace_bytes, w_scales, ns) ||
      overlap(workspace, workspace_bytes, bias, (size_t)n * 2))
    return fail(CONVROT_E_INVALID_ARG, "%s: overlapping buffers", fn);
  const SignMask sm = make_signs(rot_seed, g);
  uint8_t* codes = static_cast<uint8_t*>(workspace);
  uint8_t* scales = codes + align_up(codes_bytes(slice, k), 256);
  hipStream_t st = (hipStream_t)stream;
  for (int64_t r0 = 0; r0 < m; r0 += slice) {
    const int64_t rows = m - r0 < slice ? m - r0 : slice;
    hipError_t e = launch_mx4_quantize(static_cast<const uint16_t*>(x) + r0 * k, rows, (int)k, g,
                                       sm, dt, codes, scales, st);
    if (e != hipSuccess) return hip_status(e, fn);
    e = launch_mx4_gemm(codes, scales, w_codes, w_scales, static_cast<const uint16_t*>(bias), rows,
                        n, k, static_cast<uint16_t*>(y) + r0 * n,
                        mx4_gemm_tile(rows, n, k, m, compute_units()), dt, st);
    if (e != hipSuccess) return hip_status(e, fn);
  }
  return ok();
}

convrot_status convrot_norm_residual(const convrot_norm_args* args, void* stream) {
  const char* fn = "convrot_norm_residual";
  if (!args) return fail(CONVROT_E_INVALID_ARG, "%s: null arguments", fn);
  const convrot_norm_args& a = *args;
  DType dt;
  if (!dtype_of(a.dtype, &dt)) return fail(CONVROT_E_INVALID_ARG, "%s: dtype=%d", fn, (int)a.dtype);
  auto kind = [](int v, bool none) {
    return v == CONVROT_NORM_RMS || v == CONVROT_NORM_LAYER || (none && v == CONVROT_NORM_NONE);
  };
  if (!kind(a.norm, false) || !kind(a.post_norm, true))
    return fail(CONVROT_E_INVALID_ARG, "%s: norm=%d post_norm=%d", fn, (int)a.norm,
                (int)a.post_norm);
  if (!(a.eps >= 0.0f) || a.eps > 3.0e38f)
    return fail(CONVROT_E_INVALID_ARG, "%s: eps=%g", fn, (double)a.eps);
  const int64_t m = a.m, k = a.k;
  if (m < 0 || k <= 0)
    return fail(CONVROT_E_INVALID_ARG, "%s: bad dims m=%lld k=%lld", fn, (long long)m,
                (long long)k);
  const bool quantized = a.h_codes || a.h_scales;
  if (quantized) {
    if (convrot_status s = check_mx4(fn, m, k, a.g)) return s;
  }
  if (k % 8 || k > kMaxNormK || m >= kMaxDim || !norm_grid_fits(m, k))
    return fail(CONVROT_E_UNSUPPORTED_SHAPE,
                "%s: need k %% 8 == 0, k <= %lld, m * ceil(k/2048) < 2^26 (m=%lld k=%lld)", fn,
                (long long)kMaxNormK, (long long)m, (long long)k);
  const bool mods = a.gate || a.scale || a.shift;
  if (mods && a.rows_per_mod < 1)
    return fail(CONVROT_E_INVALID_ARG, "%s: rows_per_mod=%lld", fn, (long long)a.rows_per_mod);
  if (!a.o && (a.x_out || a.gate || a.post_weight || a.post_norm != CONVROT_NORM_NONE))
    return fail(CONVROT_E_INVALID_ARG, "%s: x_out, gate and the post norm need o", fn);
  if (a.post_weight && a.post_norm == CONVROT_NORM_NONE)
    return fail(CONVROT_E_INVALID_ARG, "%s: a post weight without a post norm", fn);
  if (m == 0) return ok();
  if (!a.x || (a.o && !a.x_out) || (!a.h && !quantized) || (quantized && !(a.h_codes && a.h_scales)))
    return fail(CONVROT_E_INVALID_ARG, "%s: null pointer", fn);
  const void* wide[] = {a.x, a.o, a.x_out, a.post_weight, a.weight, a.gate, a.scale, a.shift,
                        a.h, a.h_codes, a.h_scales};
  for (const void* p : wide)
    if (!aligned(p, 16)) return fail(CONVROT_E_MISALIGNED, "%s: misaligned pointer", fn);
  // modulation rows: rows_per_mod beyond m (any value) means one for all
  const int64_t rows_per_mod = mods && a.rows_per_mod < m ? a.rows_per_mod : m;
  const int64_t samples = (m - 1) / rows_per_mod + 1;
  const struct {
    const void* p;
    int64_t stride;
  } mod[] = {{a.gate, a.gate_stride}, {a.scale, a.scale_stride}, {a.shift, a.shift_stride}};
  for (const auto& t : mod) {
    if (!t.p) continue;
    // no range of 2^62 bytes: byte counts below stay inside 64 bits
    if (t.stride < 0 || t.stride > ((int64_t)1 << 40) ||
        (samples > 1 && t.stride > ((int64_t)1 << 60) / (samples - 1)))
      return fail(CONVROT_E_INVALID_ARG, "%s: modulation stride %lld", fn, (long long)t.stride);
    if (t.stride % 8)
      return fail(CONVROT_E_MISALIGNED, "%s: modulation stride %lld is not a multiple of 8", fn,
                  (long long)t.stride);
  }
  const size_t nx = (size_t)(m * k) * 2, nw = (size_t)k * 2;
  const struct {
    const void* p;
    size_t bytes;
  } out[] = {{a.x_out, nx}, {a.h, nx}, {a.h_codes, quantized ? codes_bytes(m, k) : 0},
             {a.h_scales, quantized ? scales_bytes(m, k) : 0}};
  for (int i = 0; i < 4; ++i) {
    bool bad = false;
    for (int j = i + 1; j < 4; ++j) bad |= overlap(out[i].p, out[i].bytes, out[j].p, out[j].bytes);
    // x may be updated in place
    if (!(i == 0 && a.x_out == a.x)) bad |= overlap(out[i].p, out[i].bytes, a.x, nx);
    bad |= overlap(out[i].p, out[i].bytes, a.o, nx) ||
           overlap(out[i].p, out[i].bytes, a.post_weight, nw) ||
           overlap(out[i].p, out[i].bytes, a.weight, nw);
    for (const auto& t : mod)
      bad |= overlap(out[i].p, out[i].bytes, t.p, (size_t)((samples - 1) * t.stride + k) * 2);
    if (bad) return fail(CONVROT_E_INVALID_ARG, "%s: overlapping buffers", fn);
  }
  auto p16 = [](const void* p) { return static_cast<const uint16_t*>(p); };
  NormArgs n;
  n.x = p16(a.x);
  n.o = p16(a.o);
  n.post_weight = p16(a.post_weight);
  n.weight = p16(a.weight);
  n.gate = p16(a.gate);
  n.scale = p16(a.scale);
  n.shift = p16(a.shift);
  n.gate_stride = a.gate_stride;
  n.scale_stride = a.scale_stride;
  n.shift_stride = a.shift_stride;
  n.x_out = static_cast<uint16_t*>(a.x_out);
  n.h = static_cast<uint16_t*>(a.h);
  n.h_codes = a.h_codes;
  n.h_scales = a.h_scales;
  n.m = m;
  n.rows_per_mod = rows_per_mod;
  n.k = (int)k;
  n.post_norm = (NormKind)a.post_norm;
  n.norm = (NormKind)a.norm;
  n.eps = a.eps;
  const int g = quantized ? a.g : 0;
  return hip_status(launch_norm_residual(n, g, g ? make_signs(a.rot_seed, g) : SignMask{}, dt,
                                         (hipStream_t)stream),
                    fn);
}

}  // extern "C"
