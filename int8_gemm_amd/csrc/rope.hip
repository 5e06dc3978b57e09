// Rotary tables of positions with several axes, and norms of queries and keys
// with the rotation in the same pass (gfx950).
//
// Table: pair p of an axis turns by position * theta^(-2 j / n). Angles are
// formed and reduced in float64 (a position of 10^5 leaves fp32 three digits of
// its angle) and their cos and sin rounded once.
//
// Norm and rotation: v = x / sqrt(mean(x^2) + eps) * weight (or the layer norm)
// over a head, or over all heads of a token, then (a, b) -> (a cos - b sin,
// b cos + a sin) per pair; fp32 between the 16-bit ends. Bound by memory: q and
// k are read once and written once. A lane holds two chunks of eight elements
// of a head so placed that both elements of a pair are its own: chunks 2 t and
// 2 t + 1 for pairs (2 i, 2 i + 1), chunks t and t + pairs / 8 for pairs
// (i, i + pairs).

#include "attention.h"
#include "mx4.h"
#include "wave_sum.h"

namespace convrot {

namespace {

// ---- table -----------------------------------------------------------------

constexpr int kTableThreads = 256;
constexpr int kTableTokens = 16;  // of a block

template <typename P>
__global__ __launch_bounds__(kTableThreads) void rope_table_kernel(RopeTableArgs a) {
  __shared__ double freq[kMaxRopePairs];
  __shared__ int axis_of[kMaxRopePairs];
  for (int p = threadIdx.x; p < a.pairs; p += kTableThreads) {
    int axis = 0;
    while (axis + 1 < a.axes && p >= a.first[axis + 1]) ++axis;
    const int j = a.shared ? p : p - a.first[axis];
    const int n = a.shared ? a.pairs : a.first[axis + 1] - a.first[axis];
    freq[p] = exp2(-a.log2_theta * ((double)j / n));  // 2 j of 2 n elements
    axis_of[p] = axis;
  }
  __syncthreads();
  const int64_t token0 = (int64_t)blockIdx.x * kTableTokens;
  const int tokens = (int)min((int64_t)kTableTokens, a.tokens - token0);
  const P* positions = static_cast<const P*>(a.positions);
  for (int i = threadIdx.x; i < tokens * a.pairs; i += kTableThreads) {
    const int64_t token = token0 + i / a.pairs;
    const int p = i % a.pairs;
    const double angle =
        (double)positions[token * a.token_stride + axis_of[p] * a.axis_stride] * freq[p];
    double s, c;
    sincos(angle, &s, &c);
    reinterpret_cast<float2*>(a.table)[token * a.pairs + p] = make_float2((float)c, (float)s);
  }
}

// ---- norms and rotation ----------------------------------------------------

constexpr int kHeadThreads = 256;

// A lane's place in a head: its chunks, and the pairs behind its entries.
template <bool HALVES>
struct Place {
  int c0, c1;        // chunks of 8 elements
  bool in0, in1;     // ... inside the head
  bool turn0, turn1; // ... rotated
  __device__ Place(int t, int d, int pairs) {
    const int chunks = d / 8, p8 = pairs / 8;
    if (HALVES) {
      const bool turned = t < p8;
      c0 = turned ? t : 2 * p8 + 2 * (t - p8);
      c1 = turned ? t + p8 : c0 + 1;
      turn0 = turn1 = turned;
    } else {
      c0 = 2 * t;
      c1 = c0 + 1;
      turn0 = c0 * 4 < pairs;
      turn1 = c1 * 4 < pairs;
    }
    in0 = c0 < chunks;
    in1 = c1 < chunks;
  }
};

// The lane's 8 (cos, sin), (1, 0) where it turns nothing.
template <bool HALVES>
__device__ __forceinline__ void load_turns(const HeadsArgs& a, const Place<HALVES>& pl, int t,
                                           int64_t token, float (&cs)[8], float (&sn)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) cs[e] = 1.f, sn[e] = 0.f;
  if (!a.table) return;
  const int64_t row = a.table_rows == a.tokens ? token : token % a.table_rows;
  const float4* from = reinterpret_cast<const float4*>(a.table + row * a.pairs * 2 + t * 16);
  if (pl.turn0) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float4 f = from[i];
      cs[2 * i] = f.x, sn[2 * i] = f.y, cs[2 * i + 1] = f.z, sn[2 * i + 1] = f.w;
    }
  }
  if (pl.turn1) {
#pragma unroll
    for (int i = 2; i < 4; ++i) {
      const float4 f = from[i];
      cs[2 * i] = f.x, sn[2 * i] = f.y, cs[2 * i + 1] = f.z, sn[2 * i + 1] = f.w;
    }
  }
}

template <bool HALVES>
__device__ __forceinline__ void turn(float (&v)[2][8], const float (&cs)[8],
                                     const float (&sn)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    float& x = HALVES ? v[0][e] : v[e >> 2][2 * (e & 3)];
    float& y = HALVES ? v[1][e] : v[e >> 2][2 * (e & 3) + 1];
    const float p = x, q = y;
    x = __builtin_fmaf(p, cs[e], -(q * sn[e]));
    y = __builtin_fmaf(q, cs[e], p * sn[e]);
  }
}

template <bool F16>
__device__ __forceinline__ u4 pack8(const float (&f)[8]) {
  return (u4){pack16x2<F16>(f[0], f[1]), pack16x2<F16>(f[2], f[3]), pack16x2<F16>(f[4], f[5]),
              pack16x2<F16>(f[6], f[7])};
}

// Sum over a head's lanes (SHIFT bits), or over all of a row's: `waves` waves of
// the block with one slot each in `part`, or 2^shift lanes of one wave.
struct Span {
  int shift, waves;
};
__device__ __forceinline__ float span_sum(float v, const Span& sp, float* part) {
  if (sp.shift > 2) {
    v = lanes_sum(v, sp.shift);
  } else {
    if (sp.shift > 0) v += mx4_dpp<kDppXor1>(v);
    if (sp.shift > 1) v += mx4_dpp<kDppXor2>(v);
  }
  if (sp.waves == 1) return v;
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
  __syncthreads();
  float s = part[0];
  for (int w = 1; w < sp.waves; ++w) s += part[w];
  return s;
}
__device__ __forceinline__ uint32_t span_max(uint32_t v, const Span& sp, float* part) {
#pragma unroll
  for (int s = 0; s < 6; ++s)
    if (s < sp.shift) v = max(v, (uint32_t)__shfl_xor((int)v, 1 << s));
  if (sp.waves == 1) return v;
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = __uint_as_float(v);
  __syncthreads();
  uint32_t m = __float_as_uint(part[0]);
  for (int w = 1; w < sp.waves; ++w) m = max(m, __float_as_uint(part[w]));
  return m;
}

constexpr int kMaxSpanWaves = 16;
constexpr int kPartSlots = 6 * kMaxSpanWaves;

// Normalise the span's values; absent chunks hold 0 in xw. Squares leave fp32's
// range where bf16 values do not, so a span whose mean square is not in
// [2^-100, inf) is taken again with a power of two out of it and of eps, exactly
// (spans that share a wave repeat theirs with 2^0, to the same bits).
template <int NI, bool F16>
__device__ __forceinline__ void normalise(float (&v)[NI][2][8], const u4 (&xw)[NI][2],
                                          const bool (&in)[NI][2], NormKind kind, float count,
                                          float eps, const Span& sp, float* part) {
  if (kind == NormKind::kNone) return;
  const bool layer = kind == NormKind::kLayer;
  auto each = [&](auto f) {
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e) f(v[i][j][e]);
  };
  auto squares = [&] {
    float q = 0.f;
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float c = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) c = __builtin_fmaf(v[i][j][e], v[i][j][e], c);
        q += in[i][j] ? c : 0.f;
      }
    return q;
  };
  if (layer) {
    float s = 0.f;
    each([&](float& x) { s += x; });
    const float mean = span_sum(s, sp, part) / count;
    each([&](float& x) { x -= mean; });
  }
  float ms = span_sum(squares(), sp, part + kMaxSpanWaves) / count + eps;
  const bool again = !(ms >= 0x1p-100f && ms < __builtin_inff());
  if (__builtin_expect(__any(again), 0)) {
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) mx4_unpack8<F16>(xw[i][j], v[i][j]);
    each([&](float& x) { top = max(top, __float_as_uint(x) & 0x7FFFFFFFu); });
    top = span_max(top, sp, part + 2 * kMaxSpanWaves) >> 23;
    int by = max((int)top - 127, ((int)(__float_as_uint(eps) >> 23) - 127) >> 1) - 40;
    if (!again || top == 255) by = 0;  // an infinity or a NaN gives what it gave
    each([&](float& x) { x = __builtin_ldexpf(x, -by); });
    if (layer) {
      float s = 0.f;
      each([&](float& x) { s += x; });
      const float mean = span_sum(s, sp, part + 3 * kMaxSpanWaves) / count;
      each([&](float& x) { x -= mean; });
    }
    ms = span_sum(squares(), sp, part + 4 * kMaxSpanWaves) / count + __builtin_ldexpf(eps, -2 * by);
  }
  const float r = 1.0f / sqrtf(ms);
  each([&](float& x) { x *= r; });
}

template <bool F16>
__device__ __forceinline__ void weigh(float (&v)[2][8], const uint16_t* w, int c0, int c1,
                                      bool in0, bool in1) {
  float f[8];
  if (in0) {
    mx4_unpack8<F16>(*reinterpret_cast<const u4*>(w + c0 * 8), f);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[0][e] *= f[e];
  }
  if (in1) {
    mx4_unpack8<F16>(*reinterpret_cast<const u4*>(w + c1 * 8), f);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[1][e] *= f[e];
  }
}

// How the heads of one tensor lie on blocks: 2^lanes_shift lanes a head, then
// per-head norms: 2^slot_shift heads of a token at once, in steps over the rest.
struct HeadsShape {
  int lanes_shift;
  int slot_shift[2];
  uint32_t blocks[2];
  int waves;  // row norms: waves of a row (blocks of one row), or 0: 2^row_shift lanes
  int row_shift[2];
};

// Norms of single heads.
template <bool F16, bool HALVES>
__global__ __launch_bounds__(kHeadThreads) void heads_kernel(HeadsArgs a, HeadsShape sh) {
  const bool second = blockIdx.x >= sh.blocks[0];
  const HeadsTensor& x = a.t[second];
  const uint32_t block = blockIdx.x - (second ? sh.blocks[0] : 0);
  const int slot_shift = sh.slot_shift[second];
  const int t = threadIdx.x & ((1 << sh.lanes_shift) - 1);
  const int g = threadIdx.x >> sh.lanes_shift;
  const int slot = g & ((1 << slot_shift) - 1);
  const int per_block = kHeadThreads >> (sh.lanes_shift + slot_shift);
  const int64_t at = (int64_t)block * per_block + (g >> slot_shift);
  const bool live = at < a.tokens;
  const int64_t token = live ? at : a.tokens - 1;
  const Place<HALVES> pl(t, a.d, a.pairs);
  float cs[8], sn[8];
  load_turns<HALVES>(a, pl, t, token, cs, sn);
  const u4 zero = {0, 0, 0, 0};
  const uint16_t* in = x.in + token * x.in_stride;
  uint16_t* out = x.out + token * x.out_stride;
  const Span sp = {sh.lanes_shift, 1};
  // every lane of a wave takes every step: sums are over lanes
  for (int h0 = 0; h0 < x.heads; h0 += 1 << slot_shift) {
    const int h = min(h0 + slot, x.heads - 1);
    const bool write = live && h0 + slot < x.heads;
    const uint16_t* p = in + h * x.in_head_stride;
    u4 xw[1][2];
    xw[0][0] = pl.in0 ? *reinterpret_cast<const u4*>(p + pl.c0 * 8) : zero;
    xw[0][1] = pl.in1 ? *reinterpret_cast<const u4*>(p + pl.c1 * 8) : zero;
    const bool inside[1][2] = {{pl.in0, pl.in1}};
    float v[1][2][8];
    mx4_unpack8<F16>(xw[0][0], v[0][0]);
    mx4_unpack8<F16>(xw[0][1], v[0][1]);
    normalise<1, F16>(v, xw, inside, a.norm, (float)a.d, a.eps, sp, nullptr);
    if (x.weight) weigh<F16>(v[0], x.weight, pl.c0, pl.c1, pl.in0, pl.in1);
    turn<HALVES>(v[0], cs, sn);
    uint16_t* o = out + h * x.out_head_stride;
    if (write && pl.in0) *reinterpret_cast<u4*>(o + pl.c0 * 8) = pack8<F16>(v[0][0]);
    if (write && pl.in1) *reinterpret_cast<u4*>(o + pl.c1 * 8) = pack8<F16>(v[0][1]);
  }
}

// Norms over all heads of a token: NI heads of the row a lane group.
template <int NI, bool F16, bool HALVES>
__global__ __launch_bounds__(64 * kMaxSpanWaves) void rows_kernel(HeadsArgs a, HeadsShape sh) {
  __shared__ float part[kPartSlots];
  const bool second = blockIdx.x >= sh.blocks[0];
  const HeadsTensor& x = a.t[second];
  const uint32_t block = blockIdx.x - (second ? sh.blocks[0] : 0);
  const int t = threadIdx.x & ((1 << sh.lanes_shift) - 1);
  int64_t at;
  int group, groups;
  Span sp;
  if (sh.waves) {
    at = block;
    group = threadIdx.x >> sh.lanes_shift;
    groups = blockDim.x >> sh.lanes_shift;
    sp = {6, sh.waves};
  } else {
    const int shift = sh.row_shift[second];
    at = (int64_t)block * (blockDim.x >> shift) + (threadIdx.x >> shift);
    group = (threadIdx.x & ((1 << shift) - 1)) >> sh.lanes_shift;
    groups = 1 << (shift - sh.lanes_shift);
    sp = {shift, 1};
  }
  const bool live = at < a.tokens;
  const int64_t token = live ? at : a.tokens - 1;
  const Place<HALVES> pl(t, a.d, a.pairs);
  const u4 zero = {0, 0, 0, 0};
  u4 xw[NI][2];
  bool inside[NI][2];
  float v[NI][2][8];
  int head[NI];
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    head[i] = group + i * groups;
    const bool in = head[i] < x.heads;
    inside[i][0] = in && pl.in0;
    inside[i][1] = in && pl.in1;
    const uint16_t* p = x.in + token * x.in_stride + head[i] * x.in_head_stride;
    xw[i][0] = inside[i][0] ? *reinterpret_cast<const u4*>(p + pl.c0 * 8) : zero;
    xw[i][1] = inside[i][1] ? *reinterpret_cast<const u4*>(p + pl.c1 * 8) : zero;
  }
  float cs[8], sn[8];
  load_turns<HALVES>(a, pl, t, token, cs, sn);
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    mx4_unpack8<F16>(xw[i][0], v[i][0]);
    mx4_unpack8<F16>(xw[i][1], v[i][1]);
  }
  normalise<NI, F16>(v, xw, inside, a.norm, (float)(a.d * x.heads), a.eps, sp, part);
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    if (x.weight)
      weigh<F16>(v[i], x.weight + (int64_t)head[i] * a.d, pl.c0, pl.c1, inside[i][0],
                 inside[i][1]);
    turn<HALVES>(v[i], cs, sn);
    uint16_t* o = x.out + token * x.out_stride + head[i] * x.out_head_stride;
    if (live && inside[i][0]) *reinterpret_cast<u4*>(o + pl.c0 * 8) = pack8<F16>(v[i][0]);
    if (live && inside[i][1]) *reinterpret_cast<u4*>(o + pl.c1 * 8) = pack8<F16>(v[i][1]);
  }
}

int log2_up(int64_t n) {
  int s = 0;
  while (((int64_t)1 << s) < n) ++s;
  return s;
}

// lanes of a head: two chunks each
int lanes_shift(int d) { return log2_up((d / 8 + 1) / 2); }

HeadsShape shape(const HeadsArgs& a) {
  HeadsShape sh = {};
  sh.lanes_shift = lanes_shift(a.d);
  for (int i = 0; i < 2; ++i) {
    const HeadsTensor& x = a.t[i];
    if (!x.heads) continue;
    if (!a.row) {
      const int most = log2_up(kHeadThreads) - sh.lanes_shift;
      int s = log2_up(x.heads);
      if (s > most) s = most;
      sh.slot_shift[i] = s;
      const int64_t per = kHeadThreads >> (sh.lanes_shift + s);
      sh.blocks[i] = (uint32_t)((a.tokens + per - 1) / per);
    }
  }
  if (a.row) {
    const int most = a.t[0].heads > a.t[1].heads ? a.t[0].heads : a.t[1].heads;
    const int64_t lanes = (int64_t)most << sh.lanes_shift;
    if (lanes > 64) {
      sh.waves = (int)((lanes + 63) / 64);
      if (sh.waves > kMaxSpanWaves) sh.waves = (sh.waves + 1) / 2;
    }
    for (int i = 0; i < 2; ++i) {
      if (!a.t[i].heads) continue;
      sh.row_shift[i] = log2_up((int64_t)a.t[i].heads << sh.lanes_shift);
      const int64_t per = sh.waves ? 1 : kHeadThreads >> sh.row_shift[i];
      sh.blocks[i] = (uint32_t)((a.tokens + per - 1) / per);
    }
  }
  return sh;
}

template <bool F16, bool HALVES>
hipError_t launch(const HeadsArgs& a, hipStream_t st) {
  const HeadsShape sh = shape(a);
  const dim3 grid(sh.blocks[0] + sh.blocks[1]);
  if (!a.row) {
    heads_kernel<F16, HALVES><<<grid, dim3(kHeadThreads), 0, st>>>(a, sh);
  } else {
    const int most = a.t[0].heads > a.t[1].heads ? a.t[0].heads : a.t[1].heads;
    const dim3 block(sh.waves ? 64 * sh.waves : kHeadThreads);
    if (sh.waves * 64 < (int64_t)most << sh.lanes_shift && sh.waves)
      rows_kernel<2, F16, HALVES><<<grid, block, 0, st>>>(a, sh);
    else
      rows_kernel<1, F16, HALVES><<<grid, block, 0, st>>>(a, sh);
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_rope_table(const RopeTableArgs& a, PosType type, hipStream_t st) {
  if (a.tokens == 0) return hipSuccess;
  const dim3 grid((uint32_t)((a.tokens + kTableTokens - 1) / kTableTokens)), block(kTableThreads);
  switch (type) {
    case PosType::kI32: rope_table_kernel<int32_t><<<grid, block, 0, st>>>(a); break;
    case PosType::kI64: rope_table_kernel<int64_t><<<grid, block, 0, st>>>(a); break;
    default: rope_table_kernel<float><<<grid, block, 0, st>>>(a); break;
  }
  return hipGetLastError();
}

bool heads_row_fits(int64_t heads, int d) {
  return (heads << lanes_shift(d)) <= 2 * 64 * kMaxSpanWaves;
}

bool heads_grid_fits(const HeadsArgs& a) {
  const HeadsShape sh = shape(a);
  const int waves = sh.waves ? sh.waves : kHeadThreads / 64;
  return ((int64_t)sh.blocks[0] + sh.blocks[1]) * waves <= kMaxLaunchWaves;
}

hipError_t launch_qk_norm_rope(const HeadsArgs& a, bool halves, DType dt, hipStream_t st) {
  if (a.tokens == 0) return hipSuccess;
  if (dt == DType::kF16) return halves ? launch<true, true>(a, st) : launch<true, false>(a, st);
  return halves ? launch<false, true>(a, st) : launch<false, false>(a, st);
}

}  // namespace convrot
