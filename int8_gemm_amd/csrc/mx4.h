// Device side of the microscaled 4-bit (MXFP4) form, shared by the kernels
// that write it (mx4.hip, norm.hip) and read it back.
//
// A [rows, K] tensor is held as
//   codes  [rows, K / 2]: one byte per two elements, the even one in the low
//          nibble; a code is a sign bit and one of 0, 0.5, 1, 1.5, 2, 3, 4, 6;
//   scales [ceil(K / 256)][R16][8], R16 = rows rounded up to 16: the biased
//          exponent of the 2^e that 32 consecutive elements of a row share
//          (255: the block is NaN). Eight blocks of a row are one K-step of
//          the GEMM; with the rows innermost a tile's scales of a K-step are
//          one contiguous run, and the padding aligns every K-step's run.
//
// Rotation. A tile is 256 elements of one row, held by 8 lanes (a wave holds
// 8 tiles). Lane j of the 8 keeps label c = j ^ (j & 4 ? 3 : 0) and the
// elements 64 i + 8 c + e, i < 4, e < 8: one 16-byte load per i, and 8 lanes
// read 128 consecutive bytes. The Walsh-Hadamard levels over e (and i, for
// g = 256) are in-lane; those over c are exchanges with lane j ^ 1, j ^ 2
// and 7 - j (the half-row mirror, a single DPP step that flips bit 2 of the
// label alone). An exchange level computes
//   own + s * partner, s = +1 / -1 where the label's bit is 0 / 1,
// one fused DPP multiply-add, which leaves a lane with the bit set negated.
// The product of these signs over the levels is (-1)^popcount(c & J), J = the
// label bits transformed; H with its outputs so signed equals H of the input
// shifted by J (H[i][j] (-1)^popcount(i & J) = H[i][j ^ J]), so the lane loads
// the elements of label c ^ J and no sign is left to undo.
#pragma once

#include "common.h"

namespace convrot {

constexpr int kMx4Block = 32;   // elements per scale
constexpr int kMx4Tile = 256;   // elements per K-step of the scale layout

__host__ __device__ constexpr int64_t mx4_pad_rows(int64_t rows) { return (rows + 15) / 16 * 16; }

__device__ __forceinline__ int mx4_label(int lane) {
  const int j = lane & 7;
  return j ^ ((j & 4) ? 3 : 0);
}
// label bits that the rotation transforms across lanes
template <int G>
constexpr int kMx4LaneBits = G >= 64 ? 7 : (G == 16 ? 1 : 0);

template <int CTRL>
__device__ __forceinline__ float mx4_dpp(float v) {
  return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), CTRL, 0xF, 0xF, true));
}
template <int CTRL>
__device__ __forceinline__ double mx4_dpp(double v) {
  const uint64_t b = __double_as_longlong(v);
  const uint32_t lo = __builtin_amdgcn_mov_dpp((int)(uint32_t)b, CTRL, 0xF, 0xF, true);
  const uint32_t hi = __builtin_amdgcn_mov_dpp((int)(uint32_t)(b >> 32), CTRL, 0xF, 0xF, true);
  return __longlong_as_double(((uint64_t)hi << 32) | lo);
}
template <int CTRL>
__device__ __forceinline__ uint32_t mx4_dpp(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, CTRL, 0xF, 0xF, true);
}
constexpr int kDppXor1 = 0xB1;     // quad_perm [1,0,3,2]
constexpr int kDppXor2 = 0x4E;     // quad_perm [2,3,0,1]
constexpr int kDppMirror8 = 0x141;   // row_half_mirror: lane j of 8 <- lane 7 - j
constexpr int kDppMirror16 = 0x140;  // row_mirror: lane j of 16 <- lane 15 - j

// One exchange level: v = v + s * (the partner's v).
template <int CTRL>
__device__ __forceinline__ void mx4_exchange(double (&v)[1][8], double s) {
#pragma unroll
  for (int e = 0; e < 8; ++e) v[0][e] = __builtin_fma(mx4_dpp<CTRL>(v[0][e]), s, v[0][e]);
}

// In fp32 the exchange folds into the multiply-add, which the compiler does
// not do by itself (it takes a move and a multiply-add per element). A DPP operand must not have been written by
// the last two instructions; the compiler does not look into the block for
// that, so both ends wait.
#define CONVROT_FMAC_DPP(CTRL_TEXT, a, b, s)                                                    \
  asm volatile("s_nop 1\n\t"                                                                    \
               "v_fmac_f32_dpp %0, %0, %16 " CTRL_TEXT " row_mask:0xf bank_mask:0xf\n\t"        \
               "v_fmac_f32_dpp %1, %1, %16 " CTRL_TEXT " row_mask:0xf bank_mask:0xf\n\t"        \
               "v_fmac_f32_dpp %2, %2, %16 " CTRL_TEXT " row_mask:0xf bank_mask:0xf\n\t"        \
               "v_fmac_f32_dpp %3, %3, %16 " CTRL_TEXT " row_mask:0xf bank_mask:0xf\n\t"        \
               "v_fmac_f32_dpp %4, %4, %16 " CTRL_TEXT " row_mask:0xf bank_mask:0xf\n\t"        \
               "v_fmac_f32_dpp %5, %5, %16 " CTRL_TEXT " row_mask:0xf bank_mask:0xf\n\t"        \
               "v_fmac_f32_dpp %6, %6, %16 " CTRL_TEXT " row_mask:0xf bank_mask:0xf\n\t"        \
               "v_fmac_f32_dpp %7, %7, %16 " CTRL_TEXT " row_mask:0xf bank_mask:0xf\n\t"        \
               "v_fmac_f32_dpp %8, %8, %16 " CTRL_TEXT " row_mask:0xf bank_mask:0xf\n\t"        \
               "v_fmac_f32_dpp %9, %9, %16 " CTRL_TEXT " row_mask:0xf bank_mask:0xf\n\t"        \
               "v_fmac_f32_dpp %10, %10, %16 " CTRL_TEXT " row_mask:0xf bank_mask:0xf\n\t"      \
               "v_fmac_f32_dpp %11, %11, %16 " CTRL_TEXT " row_mask:0xf bank_mask:0xf\n\t"      \
               "v_fmac_f32_dpp %12, %12, %16 " CTRL_TEXT " row_mask:0xf bank_mask:0xf\n\t"      \
               "v_fmac_f32_dpp %13, %13, %16 " CTRL_TEXT " row_mask:0xf bank_mask:0xf\n\t"      \
               "v_fmac_f32_dpp %14, %14, %16 " CTRL_TEXT " row_mask:0xf bank_mask:0xf\n\t"      \
               "v_fmac_f32_dpp %15, %15, %16 " CTRL_TEXT " row_mask:0xf bank_mask:0xf\n\t"      \
               "s_nop 1"                                                                        \
               : "+v"(a[0]), "+v"(a[1]), "+v"(a[2]), "+v"(a[3]), "+v"(a[4]), "+v"(a[5]),        \
                 "+v"(a[6]), "+v"(a[7]), "+v"(b[0]), "+v"(b[1]), "+v"(b[2]), "+v"(b[3]),        \
                 "+v"(b[4]), "+v"(b[5]), "+v"(b[6]), "+v"(b[7])                                 \
               : "v"(s))

template <int CTRL>
__device__ __forceinline__ void mx4_exchange(float (&v)[4][8], float s) {
#pragma unroll
  for (int i = 0; i < 4; i += 2) {
    if constexpr (CTRL == kDppXor1) CONVROT_FMAC_DPP("quad_perm:[1,0,3,2]", v[i], v[i + 1], s);
    if constexpr (CTRL == kDppXor2) CONVROT_FMAC_DPP("quad_perm:[2,3,0,1]", v[i], v[i + 1], s);
    if constexpr (CTRL == kDppMirror8) CONVROT_FMAC_DPP("row_half_mirror", v[i], v[i + 1], s);
  }
}
#undef CONVROT_FMAC_DPP

// x . blockdiag(H_G) of the tile (or of a chunk i of it, for G <= 64),
// unnormalised, in place; `label` is the lane's own (output) label. Sums in T.
template <int G, typename T, int C>
__device__ __forceinline__ void mx4_hadamard(T (&v)[C][8], int label) {
  static_assert(C == 4 || G <= 64, "a group lies in the chunks at hand");
  constexpr int LE = G < 8 ? G : 8;
#pragma unroll
  for (int i = 0; i < C; ++i) {
#pragma unroll
    for (int h = 1; h < LE; h <<= 1) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if (e & h) continue;
        const T a = v[i][e], b = v[i][e + h];
        v[i][e] = a + b;
        v[i][e + h] = a - b;
      }
    }
  }
  if constexpr (G == 256) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const T a = v[0][e] + v[1][e], b = v[0][e] - v[1][e];
      const T c = v[2][e] + v[3][e], d = v[2][e] - v[3][e];
      v[0][e] = a + c;
      v[1][e] = b + d;
      v[2][e] = a - c;
      v[3][e] = b - d;
    }
  }
  if constexpr (G >= 16) mx4_exchange<kDppXor1>(v, (label & 1) ? T(-1) : T(1));
  if constexpr (G >= 64) {
    mx4_exchange<kDppXor2>(v, (label & 2) ? T(-1) : T(1));
    mx4_exchange<kDppMirror8>(v, (label & 4) ? T(-1) : T(1));
  }
}

// The rotation's signs as masks for packed codes: bit 3 of nibble e of word
// i is set where d = -1 for element 64 i + 8 label + e. `sm` holds the signs
// of a whole 256-element tile.
__device__ __forceinline__ void mx4_sign_masks(const SignMask& sm, int label,
                                               uint32_t (&mask)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t w = (label & 4) ? sm.w[2 * i + 1] : sm.w[2 * i];
    uint32_t b = (w >> (8 * (label & 3))) & 0xFFu;
    b = (b | (b << 12)) & 0x000F000Fu;
    b = (b | (b << 6)) & 0x03030303u;
    b = (b | (b << 3)) & 0x11111111u;
    mask[i] = b << 3;
  }
}

// max over the lane's elements of each i and the 4 lanes that share its block
// (element 64 i + 8 c + e lies in block 2 i + c / 4)
__device__ __forceinline__ uint32_t mx4_block_max(uint32_t m) {
  m = max(m, mx4_dpp<kDppXor1>(m));
  return max(m, mx4_dpp<kDppXor2>(m));
}

// 2^e as a float from the biased exponent b (e = b - 127; b = 0 gives 2^-127,
// a subnormal)
__device__ __forceinline__ float mx4_pow2(uint32_t b) {
  return __uint_as_float(b == 0 ? 0x00400000u : b << 23);
}

// Quantize 8 rotated fp32 values of the lane (one i): the block's biased
// exponent and the codes without the rotation's signs. A block that holds a
// value that is not finite gets exponent 255 and codes 0.
__device__ __forceinline__ void mx4_encode(const float (&v)[8], uint32_t& eb, uint32_t& code) {
  // largest magnitude as an integer: orders finite < inf < NaN
  uint32_t m = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) m = max(m, __float_as_uint(v[e]) & 0x7FFFFFFFu);
  m = mx4_block_max(m);
  const uint32_t field = m >> 23;
  const bool bad = field == 255;
  // floor(log2 max) - 2 from the exponent field; below 2^-125 (subnormals
  // among them) it is clamped to -127
  const uint32_t b = field > 2 ? field - 2 : 0;
  eb = bad ? 255 : b;
  // at 2^-127 the conversion's divisor would be subnormal: both sides are
  // doubled, exactly
  const float up = b == 0 ? 2.0f : 1.0f;
  const float unit = __uint_as_float((b == 0 ? 1u : b) << 23);
  uint32_t w = 0;
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[0] * up, v[1] * up, unit, 0);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[2] * up, v[3] * up, unit, 1);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[4] * up, v[5] * up, unit, 2);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[6] * up, v[7] * up, unit, 3);
  code = bad ? 0 : w;
}

// Two packed 16-bit values -> fp32, exact. Half goes through the mixed-precision
// multiply-add, x * 1 + -0 (which keeps the sign of a zero): the conversion
// instruction runs at a quarter of its rate (gated norm with two layer norms and
// quantized h, 32760 x 5120 half, g = 256: 331 us with conversions, 252 with
// this).
template <bool F16>
__device__ __forceinline__ void mx4_unpack2(uint32_t w, float& lo, float& hi) {
  if constexpr (F16) {
    asm("v_fma_mix_f32 %0, %1, 1.0, neg(0) op_sel:[0,0,0] op_sel_hi:[1,0,0]" : "=v"(lo) : "v"(w));
    asm("v_fma_mix_f32 %0, %1, 1.0, neg(0) op_sel:[1,0,0] op_sel_hi:[1,0,0]" : "=v"(hi) : "v"(w));
  } else {
    lo = bf16lo(w);
    hi = bf16hi(w);
  }
}

template <bool F16>
__device__ __forceinline__ void mx4_unpack8(const u4& w, float (&f)[8]) {
#pragma unroll
  for (int p = 0; p < 4; ++p) mx4_unpack2<F16>(w[p], f[2 * p], f[2 * p + 1]);
}

// The definition, for one i: sums in float64, rounded once to fp32, then the
// codes. With g = 256 the transform over the four chunks comes first and yields
// this i's row of it alone, so that only 8 sums are live.
template <int G, bool F16>
__device__ __forceinline__ void mx4_rotate_encode_f64(const u4 (&raw)[4], int i, int label,
                                                      uint32_t& eb, uint32_t& code) {
  double d[1][8] = {};
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    if (G < 256 && c != i) continue;
    const double s = G == 256 && (__builtin_popcount(c & i) & 1) ? -1.0 : 1.0;
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      uint32_t w = raw[c][p];
      asm volatile("" : "+v"(w));  // keeps the conversions here, off the common path
      d[0][2 * p] = __builtin_fma((double)lo16<F16>(w), s, d[0][2 * p]);
      d[0][2 * p + 1] = __builtin_fma((double)hi16<F16>(w), s, d[0][2 * p + 1]);
    }
  }
  mx4_hadamard<(G < 64 ? G : 64)>(d, label);
  constexpr double norm = 1.0 / (1 << (ilog2(G) / 2));
  float f[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) f[e] = (float)(d[0][e] * norm);
  mx4_encode(f, eb, code);
}

// Rotate and quantize a tile from its packed 16-bit elements (raw[i] = the 8
// elements of label c ^ kMx4LaneBits<G>, i as above): biased exponents and
// codes per i.
//
// Sums in fp32 decide nearly all of it. Such a sum's error is at most delta =
// log2(G) 2^-24 sum|x| over its group (each of the log2(G) additions on its way
// rounds a partial sum of at most sum|x|). Rounding to fp32 and to codes are
// monotone, so where v - delta and v + delta get the same code, and the
// block's largest magnitude +- delta the same exponent, the float64 sum gets
// them too. Where any lane of the wave is left open (or a block lies so low or
// high that fp32 would lose bits of the definition) the wave takes the float64
// sums of that i: one wave in ten or so for normal activations, a quarter of
// the tile at a time. All of it in float64 took 126 us instead of 105 at 32760 x
// 5120, g = 256; inputs that lie on borders throughout (all ones) take 198.
// Sums of four bf16 values hit borders in most waves, and their float64 form
// has no exchanges: g = 4 takes it for bf16 at once (86 us instead of 99; half,
// with finer values, 86 instead of 80).
template <int G, bool F16>
__device__ __forceinline__ void mx4_quantize_tile(const u4 (&raw)[4], int label,
                                                  const uint32_t (&signs)[4], uint32_t (&eb)[4],
                                                  uint32_t (&code)[4]) {
  float v[4][8];
#pragma unroll
  for (int i = 0; i < 4; ++i) mx4_unpack8<F16>(raw[i], v[i]);
  if constexpr (G == 1) {
#pragma unroll
    for (int i = 0; i < 4; ++i) mx4_encode(v[i], eb[i], code[i]);
    return;
  }
  if constexpr (G == 4 && !F16) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      mx4_rotate_encode_f64<G, F16>(raw, i, label, eb[i], code[i]);
      code[i] ^= signs[i];
    }
    return;
  }
  constexpr int lg = ilog2(G) / 2;  // sqrt(G) = 2^lg: the fp32 sums stay unnormalised
  // sum|x| over the group, or over the block where a block holds several
  float mass[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) s += __builtin_fabsf(v[i][e]);
    mass[i] = s;
  }
  if constexpr (G == 256) mass[0] = (mass[0] + mass[1]) + (mass[2] + mass[3]);
#pragma unroll
  for (int i = 0; i < (G == 256 ? 1 : 4); ++i) {
    mass[i] += mx4_dpp<kDppXor1>(mass[i]);
    mass[i] += mx4_dpp<kDppXor2>(mass[i]);
    if constexpr (G >= 64) mass[i] += mx4_dpp<kDppMirror8>(mass[i]);
  }
  if constexpr (G == 256) mass[1] = mass[2] = mass[3] = mass[0];
  mx4_hadamard<G>(v, label);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    // 1 + 2^-9 covers the roundings of the mass itself and of the product
    constexpr float c = ilog2(G) * 0x1p-24f * (1.0f + 0x1p-9f);
    const float delta = mass[i] * c;
    float top = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) top = fmaxf(top, __builtin_fabsf(v[i][e]));
    top = fmaxf(top, mx4_dpp<kDppXor1>(top));
    top = fmaxf(top, mx4_dpp<kDppXor2>(top));
    const uint32_t field = __float_as_uint(top - delta) >> 23;
    const bool zero = mass[i] == 0.f;
    const float unit = __uint_as_float((zero ? 1u : field - 2) << 23);
    uint32_t lo = 0, hi = 0;
    lo = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(lo, v[i][0] - delta, v[i][1] - delta, unit, 0);
    hi = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(hi, v[i][0] + delta, v[i][1] + delta, unit, 0);
    lo = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(lo, v[i][2] - delta, v[i][3] - delta, unit, 1);
    hi = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(hi, v[i][2] + delta, v[i][3] + delta, unit, 1);
    lo = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(lo, v[i][4] - delta, v[i][5] - delta, unit, 2);
    hi = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(hi, v[i][4] + delta, v[i][5] + delta, unit, 2);
    lo = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(lo, v[i][6] - delta, v[i][7] - delta, unit, 3);
    hi = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(hi, v[i][6] + delta, v[i][7] + delta, unit, 3);
    // the comparisons are false for a NaN mass, and |v| <= mass < 2^120; a block
    // of zeros has v = delta = 0, exponent and codes 0
    const bool done = lo == hi && (zero || (field == __float_as_uint(top + delta) >> 23 &&
                                            field >= 40 + lg && mass[i] < 0x1p120f));
    eb[i] = zero ? 0 : field - 2 - lg;
    code[i] = lo;
    if (__any(!done)) mx4_rotate_encode_f64<G, F16>(raw, i, label, eb[i], code[i]);
    code[i] ^= signs[i];
  }
}

// Write a quantized tile: word i of the lane covers elements 64 i + 8 c .. + 7
// (`codes` = the row's tile), lane (c & 3) = i writes the exponent of block
// 2 i + c / 4 (`scales` = the row's 8 bytes of the tile). Blocks at and behind
// `blocks` (the row's end) are not part of the tensor: no codes, exponent 0.
__device__ __forceinline__ void mx4_store_tile(uint8_t* __restrict__ codes,
                                               uint8_t* __restrict__ scales, int label,
                                               int blocks, const uint32_t (&eb)[4],
                                               const uint32_t (&code)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (2 * i + (label >> 2) < blocks)
      *reinterpret_cast<uint32_t*>(codes + 32 * i + 4 * label) = code[i];
  const int q = label & 3;
  const uint32_t lo = q & 1 ? eb[1] : eb[0], hi = q & 1 ? eb[3] : eb[2];
  const int blk = 2 * q + (label >> 2);
  scales[blk] = (uint8_t)(blk < blocks ? (q & 2 ? hi : lo) : 0u);
}

}  // namespace convrot
