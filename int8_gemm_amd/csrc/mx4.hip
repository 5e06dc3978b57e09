// Microscaled 4-bit (MXFP4) tensors: rotate + quantize, and the way back
// (gfx950). Layout and rotation are described in mx4.h.
//
//   quantize: x_r = x . blockdiag(R), R = H_g . diag(d) / sqrt(g) (g = 1: none),
//     each sum rounded once to fp32; per block of 32
//       e = clamp(floor(log2 max|x_r|) - 2, -127, 127),
//       code = x_r / 2^e rounded to a 4-bit float, ties to even, at most 6.
//   dequant:  W_hat = (v 2^e) . blockdiag(R)^T = ((v 2^e) . D) . H / sqrt(g), sums
//     in fp32, rounded once to bf16 / half.
//
// Both move 2 + 17/32 bytes per element, 83 us for 32760 x 5120 at the 5.12 TB/s
// of a large device copy. A wave takes 8 rows of one 256-column tile: its loads
// and stores are 128-byte runs, and the scales of its 8 rows are 64 consecutive
// bytes. Measured at that size in a steady state: quantize 78 us (g = 1), 88 (64),
// 105 (256; 85-93 for a lone launch, whose clock the power limit does not yet hold
// down), read-back 66-76 us. Memory bounds the read-back and g = 1; g = 256 is
// bound by the issue of vector instructions: 22.7 an element are 6.0e7 a launch
// and, at 4 cycles each on 1024 SIMDs, 100 of its 105 us at 2.33 GHz.
// Tried: a grid that fills the card once and walks down the rows, which saves
// the waves' set-up, was no faster (101-109 us at g = 256, 81-88 at g = 1).

#include "internal.h"
#include "mx4.h"

namespace convrot {

namespace {

constexpr int kRowsPerWave = 8;
constexpr int kWaves = 4;

// one unit (8 rows x one 256-column tile) per wave, tiles of the same rows next
// to each other
template <int G, bool F16>
__global__ __launch_bounds__(64 * kWaves) void mx4_quantize_kernel(
    const uint16_t* __restrict__ x, int64_t rows, int K, SignMask sm, int tiles,
    uint8_t* __restrict__ codes, uint8_t* __restrict__ scales) {
  const int lane = threadIdx.x & 63;
  const int label = mx4_label(lane);
  const uint32_t unit = blockIdx.x * kWaves + (threadIdx.x >> 6);  // < 2^26 (checked by the host)
  const int kt = (int)(unit % (uint32_t)tiles);
  const int64_t row = (int64_t)(unit / (uint32_t)tiles) * kRowsPerWave + (lane >> 3);
  const int blocks = min(8, (K - kt * kMx4Tile) / kMx4Block);
  const bool live = row < rows;
  uint32_t signs[4];
  mx4_sign_masks(sm, label, signs);
  const int in = label ^ kMx4LaneBits<G>;
  u4 raw[4];
  // what lies outside the tensor reads its row's (or the last row's) first
  // elements of the tile instead: no branch stands between the loads
  const uint16_t* src = x + min(row, rows - 1) * K + kt * kMx4Tile;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const bool here = 2 * i + (in >> 2) < blocks;
    raw[i] = *reinterpret_cast<const u4*>(src + (here ? 64 * i + 8 * in : 0));
    if (!here || !live) raw[i] = (u4){0, 0, 0, 0};
  }
  uint32_t eb[4], code[4];
  mx4_quantize_tile<G, F16>(raw, label, signs, eb, code);
  if (live)
    mx4_store_tile(codes + row * (K / 2) + kt * (kMx4Tile / 2),
                   scales + ((int64_t)kt * mx4_pad_rows(rows) + row) * 8, label, blocks, eb, code);
}

template <int G, bool F16>
__global__ __launch_bounds__(64 * kWaves) void mx4_dequant_kernel(
    const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales, int64_t rows, int K,
    SignMask sm, int tiles, uint16_t* __restrict__ out) {
  const int lane = threadIdx.x & 63;
  const int label = mx4_label(lane);
  const uint32_t unit = blockIdx.x * kWaves + (threadIdx.x >> 6);
  const int kt = (int)(unit % (uint32_t)tiles);
  const int64_t row = (int64_t)(unit / (uint32_t)tiles) * kRowsPerWave + (lane >> 3);
  const int blocks = min(8, (K - kt * kMx4Tile) / kMx4Block);
  const bool live = row < rows;
  const int in = label ^ kMx4LaneBits<G>;
  uint32_t signs[4];
  mx4_sign_masks(sm, in, signs);  // d multiplies the input of H here
  const uint8_t* src = codes + row * (K / 2) + kt * (kMx4Tile / 2) + 4 * in;
  uint32_t w[4];
  u2 sc = {0, 0};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = live && 2 * i + (in >> 2) < blocks ? *reinterpret_cast<const uint32_t*>(src + 32 * i)
                                              : 0u;
  if (live)
    sc = *reinterpret_cast<const u2*>(scales + ((int64_t)kt * mx4_pad_rows(rows) + row) * 8);
  // the 4 exponents of this lane: bytes 2 i + in / 4
  const uint32_t pick = (in & 4) ? 0x07050301u : 0x06040200u;
  const uint32_t eb = __builtin_amdgcn_perm(sc.y, sc.x, pick);
  constexpr float norm = 1.0f / (1 << (ilog2(G) / 2));
  float v[4][8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t b = (eb >> (8 * i)) & 0xFFu;
    // blocks behind the row's end hold code 0; their exponent byte may be anything
    const bool in_row = 2 * i + (in >> 2) < blocks;
    const float unit_v = !in_row ? 0.0f
                                 : (b == 255 ? __uint_as_float(0x7FC00000u) : mx4_pow2(b) * norm);
    const uint32_t c = G > 1 ? w[i] ^ signs[i] : w[i];
    typedef float f2 __attribute__((ext_vector_type(2)));
    const f2 p0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 0);
    const f2 p1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 1);
    const f2 p2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 2);
    const f2 p3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 3);
    v[i][0] = p0.x * unit_v;
    v[i][1] = p0.y * unit_v;
    v[i][2] = p1.x * unit_v;
    v[i][3] = p1.y * unit_v;
    v[i][4] = p2.x * unit_v;
    v[i][5] = p2.y * unit_v;
    v[i][6] = p3.x * unit_v;
    v[i][7] = p3.y * unit_v;
  }
  if constexpr (G > 1) mx4_hadamard<G>(v, label);
  uint16_t* dst = out + row * K + kt * kMx4Tile + 8 * label;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (!live || 2 * i + (label >> 2) >= blocks) continue;
    *reinterpret_cast<u4*>(dst + 64 * i) =
        (u4){pack16x2<F16>(v[i][0], v[i][1]), pack16x2<F16>(v[i][2], v[i][3]),
             pack16x2<F16>(v[i][4], v[i][5]), pack16x2<F16>(v[i][6], v[i][7])};
  }
}

int64_t wave_units(int64_t rows, int64_t tiles) {
  return (rows + kRowsPerWave - 1) / kRowsPerWave * tiles;
}
int64_t grid_blocks(int64_t rows, int tiles) {
  return (wave_units(rows, tiles) + kWaves - 1) / kWaves;
}

template <int G>
hipError_t quantize_g(const uint16_t* x, int64_t rows, int K, const SignMask& sm, DType dt,
                      uint8_t* codes, uint8_t* scales, hipStream_t st) {
  const int tiles = (K + kMx4Tile - 1) / kMx4Tile;
  const dim3 grid((uint32_t)grid_blocks(rows, tiles)), block(64 * kWaves);
  if (dt == DType::kF16)
    mx4_quantize_kernel<G, true><<<grid, block, 0, st>>>(x, rows, K, sm, tiles, codes, scales);
  else
    mx4_quantize_kernel<G, false><<<grid, block, 0, st>>>(x, rows, K, sm, tiles, codes, scales);
  return hipGetLastError();
}

template <int G>
hipError_t dequant_g(const uint8_t* codes, const uint8_t* scales, int64_t rows, int K,
                     const SignMask& sm, uint16_t* out, DType dt, hipStream_t st) {
  const int tiles = (K + kMx4Tile - 1) / kMx4Tile;
  const dim3 grid((uint32_t)grid_blocks(rows, tiles)), block(64 * kWaves);
  if (dt == DType::kF16)
    mx4_dequant_kernel<G, true><<<grid, block, 0, st>>>(codes, scales, rows, K, sm, tiles, out);
  else
    mx4_dequant_kernel<G, false><<<grid, block, 0, st>>>(codes, scales, rows, K, sm, tiles, out);
  return hipGetLastError();
}

}  // namespace

SignMask mx4_tile_signs(const SignMask& sm, int g) {
  SignMask t{};
  for (int i = 0; i < kMx4Tile; ++i) {
    const int s = i % g;
    t.w[i >> 5] |= ((sm.w[s >> 5] >> (s & 31)) & 1u) << (i & 31);
  }
  return t;
}

bool mx4_grid_fits(int64_t rows, int64_t k) {
  return wave_units(rows, (k + kMx4Tile - 1) / kMx4Tile) <= kMaxLaunchWaves - kWaves;
}

hipError_t launch_mx4_quantize(const uint16_t* x, int64_t rows, int K, int g, const SignMask& sm,
                               DType dt, uint8_t* codes, uint8_t* scales, hipStream_t st) {
  if (rows == 0) return hipSuccess;
  const SignMask t = mx4_tile_signs(sm, g);
  switch (g) {
    case 1: return quantize_g<1>(x, rows, K, t, dt, codes, scales, st);
    case 4: return quantize_g<4>(x, rows, K, t, dt, codes, scales, st);
    case 16: return quantize_g<16>(x, rows, K, t, dt, codes, scales, st);
    case 64: return quantize_g<64>(x, rows, K, t, dt, codes, scales, st);
    default: return quantize_g<256>(x, rows, K, t, dt, codes, scales, st);
  }
}

hipError_t launch_mx4_dequant(const uint8_t* codes, const uint8_t* scales, int64_t rows, int K,
                              int g, const SignMask& sm, uint16_t* out, DType dt,
                              hipStream_t st) {
  if (rows == 0) return hipSuccess;
  const SignMask t = mx4_tile_signs(sm, g);
  switch (g) {
    case 1: return dequant_g<1>(codes, scales, rows, K, t, out, dt, st);
    case 4: return dequant_g<4>(codes, scales, rows, K, t, out, dt, st);
    case 16: return dequant_g<16>(codes, scales, rows, K, t, out, dt, st);
    case 64: return dequant_g<64>(codes, scales, rows, K, t, out, dt, st);
    default: return dequant_g<256>(codes, scales, rows, K, t, out, dt, st);
  }
}

}  // namespace convrot
