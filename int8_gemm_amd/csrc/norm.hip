// Gated residual and norm of a transformer block (gfx950), the step between
// two quantized layers:
//
//   x' = RN16(x + gate * post(o))         (o absent: x' = x, not written)
//   h  = RN16(pre(x') * (1 + scale) + shift)
//   post, pre: RMS   v / sqrt(mean(v^2) + eps) [* weight]
//              layer (v - mean(v)) / sqrt(mean((v - mean(v))^2) + eps) [* weight]
//
// and h goes out in 16 bits, as rotated MXFP4 (the input of the next layer's
// product, the same bits that quantizing the 16-bit h would give), or both.
// pre() reads x' as it was rounded, so that h is a function of the x' that the
// caller gets. Everything else is fp32.
//
// Bound by memory: x and o are read once, x' and h written once (32760 x 5120:
// 1.34 GB, 234-244 us = 5.5-5.7 TB/s, a large device copy reaches 5.1); with h
// quantized 258-263 us, 4.2 TB/s, vector instructions on top (53.9 an element, 0.7
// of the issue slots of the 36 us that 4608 x 3840 take). The row stays in
// registers between the norms (32 elements a lane, in the tile layout of
// mx4.h). A row takes ceil(K / 2048) waves or, up to 1024 elements, 8, 16 or 32
// lanes of one (32760 x 256: 14 us, with a wave per row 39); rows of up to one
// wave share blocks of four waves. Variances are taken in two passes over the
// registers, around the mean.

#include "internal.h"
#include "mx4.h"

namespace convrot {

namespace {

constexpr int kLaneElems = 32;                  // elements of a row per lane
constexpr int kWaveElems = 64 * kLaneElems;     // ... and per wave
constexpr int kBlockWaves = 4;                  // when a row is at most one wave
constexpr int kMaxWaves = 8;                    // K <= 16384

// How a row lies: on `waves` waves of a block, or on 2^shift lanes of one.
struct RowShape {
  int waves, shift;
};

// Sum over 2^shift lanes, the same bits in each: DPP exchanges within 16 lanes,
// then swaps of 16-lane rows and of the wave's halves.
__device__ __forceinline__ float lanes_sum(float v, int shift) {
  typedef uint32_t u2v __attribute__((ext_vector_type(2)));
  v += mx4_dpp<kDppXor1>(v);
  v += mx4_dpp<kDppXor2>(v);
  v += mx4_dpp<kDppMirror8>(v);
  if (shift > 3) v += mx4_dpp<kDppMirror16>(v);
  if (shift > 4) {
    const uint32_t a = __float_as_uint(v);
    const u2v r = __builtin_amdgcn_permlane16_swap(a, a, false, false);
    v = __uint_as_float(r.x) + __uint_as_float(r.y);
  }
  if (shift > 5) {
    const uint32_t a = __float_as_uint(v);
    const u2v r = __builtin_amdgcn_permlane32_swap(a, a, false, false);
    v = __uint_as_float(r.x) + __uint_as_float(r.y);
  }
  return v;
}

// Sum over the row; `part` holds one slot per wave. Two calls in a row use
// different slots, so one barrier each is enough.
__device__ __forceinline__ float row_sum(float v, RowShape rs, float* part) {
  v = lanes_sum(v, rs.shift);
  if (rs.waves == 1) return v;
  const int wave = threadIdx.x >> 6;
  if ((threadIdx.x & 63) == 0) part[wave] = v;
  __syncthreads();
  float s = part[0];
  for (int w = 1; w < rs.waves; ++w) s += part[w];
  return s;
}

template <bool F16>
__device__ __forceinline__ u4 pack(const float (&f)[8]) {
  return (u4){pack16x2<F16>(f[0], f[1]), pack16x2<F16>(f[2], f[3]), pack16x2<F16>(f[4], f[5]),
              pack16x2<F16>(f[6], f[7])};
}

// The largest |v| of a row by its bits (finite < inf < NaN), likewise.
__device__ __forceinline__ uint32_t row_max(uint32_t v, RowShape rs, float* part) {
  typedef uint32_t u2v __attribute__((ext_vector_type(2)));
  v = max(v, mx4_dpp<kDppXor1>(v));
  v = max(v, mx4_dpp<kDppXor2>(v));
  v = max(v, mx4_dpp<kDppMirror8>(v));
  if (rs.shift > 3) v = max(v, mx4_dpp<kDppMirror16>(v));
  if (rs.shift > 4) {
    const u2v r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    v = max(r.x, r.y);
  }
  if (rs.shift > 5) {
    const u2v r = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    v = max(r.x, r.y);
  }
  if (rs.waves == 1) return v;
  const int wave = threadIdx.x >> 6;
  if ((threadIdx.x & 63) == 0) part[wave] = __uint_as_float(v);
  __syncthreads();
  uint32_t m = __float_as_uint(part[0]);
  for (int w = 1; w < rs.waves; ++w) m = max(m, __float_as_uint(part[w]));
  return m;
}

// Normalise v in place (without its weight). `in` marks the lane's chunks that
// lie in the row; the others come in as 0 and go out as anything. `part` has
// kPartSlots slots. reload(i, c): chunk i of v again.
//
// Squares in fp32 reach their range's ends where bf16 values do not: above 2^64
// they overflow, and below 2^-75 they vanish, which counts where eps is as small.
// v / sqrt(mean(v^2) + eps) stays the same when v is divided by 2^by and eps by
// 2^(2 by), exactly, so a row whose mean square lies outside [2^-100, inf) is
// taken once more with the larger of its largest value and sqrt(eps) brought to
// 2^40. All waves of a row see the same sums and go the same way; rows that share
// a wave with such a one repeat their own with by = 0, to the same bits. The
// repetition reads the row from memory chunk by chunk, which leaves the registers
// of the common path as they are.
constexpr int kPartSlots = 5 * kMaxWaves;

template <typename Reload>
__device__ __forceinline__ void normalise(float (&v)[4][8], const bool (&in)[4], NormKind kind,
                                          float k, float eps, RowShape rs, float* part,
                                          Reload reload) {
  const bool layer = kind == NormKind::kLayer;
  if (layer) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) s += v[i][e];  // chunks outside the row hold 0
    const float mean = row_sum(s, rs, part + kMaxWaves) / k;  // a row of one value gives it back
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) v[i][e] -= mean;
  }
  float q = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float c = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) c = __builtin_fmaf(v[i][e], v[i][e], c);
    q += in[i] ? c : 0.f;
  }
  float ms = row_sum(q, rs, part) / k + eps;
  const bool again = !(ms >= 0x1p-100f && ms < __builtin_inff());
  if (__builtin_expect(__any(again), 0)) {
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float c[8];
      reload(i, c);
#pragma unroll
      for (int e = 0; e < 8; ++e) top = max(top, __float_as_uint(c[e]) & 0x7FFFFFFFu);
    }
    top = row_max(top, rs, part + 2 * kMaxWaves) >> 23;
    int by = max((int)top - 127, ((int)(__float_as_uint(eps) >> 23) - 127) >> 1) - 40;
    if (!again || top == 255) by = 0;  // an infinity or a NaN gives what it gave
    float mean = 0.f;
    if (layer) {
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float c[8];
        reload(i, c);
#pragma unroll
        for (int e = 0; e < 8; ++e) s += __builtin_ldexpf(c[e], -by);
      }
      mean = row_sum(s, rs, part + 3 * kMaxWaves) / k;
    }
    q = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      reload(i, v[i]);
      float c = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        v[i][e] = __builtin_ldexpf(v[i][e], -by) - mean;
        c = __builtin_fmaf(v[i][e], v[i][e], c);
      }
      q += in[i] ? c : 0.f;
    }
    ms = row_sum(q, rs, part + 4 * kMaxWaves) / k + __builtin_ldexpf(eps, -2 * by);
  }
  const float r = 1.0f / sqrtf(ms);
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) v[i][e] *= r;
}

// G: 0 = h in 16 bits only, otherwise the rotation group of the quantized h
// (1: none); a 16-bit h goes out as well where its pointer is set.
// EARLY: a phase's vectors are loaded before its sums, so that their latencies
// overlap (77 x 3840: 7.7 -> 6.5 us), otherwise where they are used, with
// fewer registers and so more rows in flight (32760 x 5120: 244 instead of
// 267 us). Five waves a SIMD are asked for where the allocator misses their 96
// registers by one (g = 1, 32760 x 5120: 244 -> 226 us).
template <int G, bool F16, bool EARLY>
__global__ __launch_bounds__(64 * kMaxWaves, G == 1 && !EARLY ? 5 : 1) void norm_residual_kernel(
    NormArgs a, SignMask sm, RowShape rs) {
  __shared__ float part[2 * kPartSlots];
  const int lane = threadIdx.x & 63;
  const int wave = threadIdx.x >> 6;
  const int64_t at = rs.waves == 1 ? (((int64_t)blockIdx.x * kBlockWaves + wave) << (6 - rs.shift)) +
                                         (lane >> rs.shift)
                                   : blockIdx.x;
  const bool live = at < a.m;  // lanes behind the last row go through it and write nothing
  const int64_t row = live ? at : a.m - 1;
  const int label = mx4_label(lane);
  const int lab_in = label ^ kMx4LaneBits<G>;
  const int tile = (rs.waves == 1 ? 0 : wave * 8) + ((lane & ((1 << rs.shift) - 1)) >> 3);
  const int col = tile * kMx4Tile + 8 * lab_in;  // + 64 i
  const int64_t base = row * a.k + col;
  const int64_t mod = (uint32_t)row / (uint32_t)a.rows_per_mod;  // both below 2^31
  bool in[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) in[i] = col + 64 * i < a.k;
  const u4 zero = {0, 0, 0, 0};
  auto load = [&](const uint16_t* p, int i) {
    return in[i] ? *reinterpret_cast<const u4*>(p + 64 * i) : zero;
  };

  auto load4 = [&](u4 (&to)[4], const uint16_t* p) {
#pragma unroll
    for (int i = 0; i < 4; ++i) to[i] = load(p, i);
  };
  // a chunk of the lane's elements of x' or o again, as fp32; the empty asm
  // keeps addresses and values from being held in registers up to there
  auto again_from = [&](const uint16_t* p) {
    return [&, p](int i, float (&c)[8]) {
      int64_t from = base;
      asm volatile("" : "+v"(from));
      mx4_unpack8<F16>(load(p + from, i), c);
    };
  };
  // v = v * by (+ v)
  auto multiply = [](float (&v)[4][8], const u4 (&by)[4], bool plus) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float w[8];
      mx4_unpack8<F16>(by[i], w);
#pragma unroll
      for (int e = 0; e < 8; ++e)
        v[i][e] = plus ? __builtin_fmaf(v[i][e], w[e], v[i][e]) : v[i][e] * w[e];
    }
  };

  u4 xw[4], w1[4], w2[4], w3[4];
  float v[4][8];
  load4(xw, a.x + base);
  if (a.o) {
    load4(w3, a.o + base);
    const uint16_t* gate = a.gate + mod * a.gate_stride + col;
    if (EARLY && a.post_weight) load4(w1, a.post_weight + col);
    if (EARLY && a.gate) load4(w2, gate);
#pragma unroll
    for (int i = 0; i < 4; ++i) mx4_unpack8<F16>(w3[i], v[i]);
    if (a.post_norm != NormKind::kNone)
      normalise(v, in, a.post_norm, (float)a.k, a.eps, rs, part, again_from(a.o));
    if (a.post_weight) {
      if (!EARLY) load4(w1, a.post_weight + col);
      multiply(v, w1, false);
    }
    if (a.gate) {
      if (!EARLY) load4(w2, gate);
      multiply(v, w2, false);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float w[8];
      mx4_unpack8<F16>(xw[i], w);
#pragma unroll
      for (int e = 0; e < 8; ++e) w[e] += v[i][e];
      xw[i] = in[i] ? pack<F16>(w) : zero;
      if (in[i] && live) *reinterpret_cast<u4*>(a.x_out + base + 64 * i) = xw[i];
    }
  }
  const uint16_t* scale = a.scale + mod * a.scale_stride + col;
  const uint16_t* shift = a.shift + mod * a.shift_stride + col;
  if (EARLY && a.weight) load4(w1, a.weight + col);
  if (EARLY && a.scale) load4(w2, scale);
  if (EARLY && a.shift) load4(w3, shift);
#pragma unroll
  for (int i = 0; i < 4; ++i) mx4_unpack8<F16>(xw[i], v[i]);
  normalise(v, in, a.norm, (float)a.k, a.eps, rs, part + kPartSlots,
            again_from(a.o ? a.x_out : a.x));
  if (a.weight) {
    if (!EARLY) load4(w1, a.weight + col);
    multiply(v, w1, false);
  }
  if (a.scale) {
    if (!EARLY) load4(w2, scale);
    multiply(v, w2, true);
  }
  if (!EARLY && a.shift) load4(w3, shift);
  u4 hw[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (a.shift) {
      float w[8];
      mx4_unpack8<F16>(w3[i], w);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[i][e] += w[e];
    }
    hw[i] = pack<F16>(v[i]);
    if (a.h && in[i] && live) *reinterpret_cast<u4*>(a.h + base + 64 * i) = hw[i];
  }
  if constexpr (G > 0) {
    uint32_t signs[4], eb[4], code[4];
    mx4_sign_masks(sm, label, signs);
#pragma unroll
    for (int i = 0; i < 4; ++i) hw[i] = in[i] ? hw[i] : zero;
    mx4_quantize_tile<G, F16>(hw, label, signs, eb, code);
    const int blocks = min(8, (a.k - tile * kMx4Tile) / kMx4Block);
    if (blocks > 0 && live)
      mx4_store_tile(a.h_codes + row * (a.k / 2) + tile * (kMx4Tile / 2),
                     a.h_scales + (tile * mx4_pad_rows(a.m) + row) * 8, label, blocks, eb, code);
  }
}

template <int G>
hipError_t launch_g(const NormArgs& a, const SignMask& sm, DType dt, hipStream_t st) {
  RowShape rs = {(a.k + kWaveElems - 1) / kWaveElems, 6};
  while (rs.shift > 3 && a.k <= kLaneElems << (rs.shift - 1)) --rs.shift;
  const int64_t rows = (int64_t)kBlockWaves << (6 - rs.shift);  // of a block, if it has several
  const dim3 grid((uint32_t)(rs.waves == 1 ? (a.m + rows - 1) / rows : a.m));
  const dim3 block(64 * (rs.waves == 1 ? kBlockWaves : rs.waves));
  // 16 waves a CU is what the EARLY form's registers allow
  const bool early = (int64_t)grid.x * (block.x / 64) <= (int64_t)compute_units() * 16;
  if (dt == DType::kF16) {
    if (early)
      norm_residual_kernel<G, true, true><<<grid, block, 0, st>>>(a, sm, rs);
    else
      norm_residual_kernel<G, true, false><<<grid, block, 0, st>>>(a, sm, rs);
  } else {
    if (early)
      norm_residual_kernel<G, false, true><<<grid, block, 0, st>>>(a, sm, rs);
    else
      norm_residual_kernel<G, false, false><<<grid, block, 0, st>>>(a, sm, rs);
  }
  return hipGetLastError();
}

}  // namespace

bool norm_grid_fits(int64_t m, int64_t k) {
  return m * ((k + kWaveElems - 1) / kWaveElems) <= kMaxLaunchWaves - kBlockWaves;
}

hipError_t launch_norm_residual(const NormArgs& a, int g, const SignMask& sm, DType dt,
                                hipStream_t st) {
  if (a.m == 0) return hipSuccess;
  const SignMask t = g > 0 ? mx4_tile_signs(sm, g) : sm;
  switch (g) {
    case 0: return launch_g<0>(a, t, dt, st);
    case 1: return launch_g<1>(a, t, dt, st);
    case 4: return launch_g<4>(a, t, dt, st);
    case 16: return launch_g<16>(a, t, dt, st);
    case 64: return launch_g<64>(a, t, dt, st);
    default: return launch_g<256>(a, t, dt, st);
  }
}

}  // namespace convrot
