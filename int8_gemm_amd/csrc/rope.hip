// Rotary tables of positions with several axes, and norms of queries and keys
// with the rotation in the same pass (gfx950).
//
// Table: pair p of an axis turns by position * theta^(-2 j / n). Angles are formed and
// reduced in float64 (a position of 10^5 leaves fp32 three digits of its angle), in
// quarter turns, whose whole part is exact; cos and sin of the rest, at most an eighth
// of a turn, are their Taylor series to x^12, off by 10^-11, and rounded once. 32760 x 64
// pairs take 8.5 to 9.2 us in a row of launches, 5.1 of which are a launch that writes as much
// and no more (a fill: 4.9); reading the positions and multiplying in float64 adds 1.9, the
// reduction and the series 2.1, each block's frequencies 0.1. 4608 x 64: 4.9 us, 2.6 of them
// such a launch.
//
// Norm and rotation: v = x / sqrt(mean(x^2) + eps) * weight (or the layer norm)
// over a head, or over all heads of a token, then (a, b) -> (a cos - b sin,
// b cos + a sin) per pair; fp32 between the 16-bit ends. Bound by memory: q and
// k are read once and written once. A lane holds two chunks of eight elements
// of a head so placed that both elements of a pair are its own and neighbouring
// lanes read neighbouring chunks, of up to five heads of a token at once: that many
// loads are under way before the first sum, and its cos and sin serve them all. Values
// stay packed; each pass over them unpacks anew. 32760 tokens x 40 heads of 128, q and k:
// 257 us, 5.3 TB/s (a large copy: 4.9); 4608 x 30 heads: 26.5 us.

#include "attention.h"
#include "mx4.h"
#include "wave_sum.h"

namespace convrot {

namespace {

// ---- table -----------------------------------------------------------------

constexpr int kTableThreads = 256;
constexpr int kTableTokens = 32;  // of a block

// (cos, sin) of a quarter turn times `quarters`.
__device__ __forceinline__ float2 cos_sin(double quarters) {
  const double whole = __builtin_rint(quarters);
  const double x = (quarters - whole) * 1.57079632679489661923;
  const double x2 = x * x;
  double c = 1.0 / 479001600;  // 12!
  c = __builtin_fma(c, x2, -1.0 / 3628800);
  c = __builtin_fma(c, x2, 1.0 / 40320);
  c = __builtin_fma(c, x2, -1.0 / 720);
  c = __builtin_fma(c, x2, 1.0 / 24);
  c = __builtin_fma(c, x2, -1.0 / 2);
  c = __builtin_fma(c, x2, 1.0);
  double s = -1.0 / 39916800;  // 11!
  s = __builtin_fma(s, x2, 1.0 / 362880);
  s = __builtin_fma(s, x2, -1.0 / 5040);
  s = __builtin_fma(s, x2, 1.0 / 120);
  s = __builtin_fma(s, x2, -1.0 / 6);
  s = __builtin_fma(s * x2, x, x);
  const float fc = (float)c, fs = (float)s;
  const int turn = (int)(whole - 4.0 * __builtin_floor(whole * 0.25));
  float2 r = turn & 1 ? make_float2(-fs, fc) : make_float2(fc, fs);
  return turn & 2 ? make_float2(-r.x, -r.y) : r;
}

template <typename P>
__global__ __launch_bounds__(kTableThreads) void rope_table_kernel(RopeTableArgs a) {
  __shared__ double freq[kMaxRopePairs];  // quarter turns of a position
  __shared__ int axis_of[kMaxRopePairs];
  for (int p = threadIdx.x; p < a.pairs; p += kTableThreads) {
    int axis = 0;
    while (axis + 1 < a.axes && p >= a.first[axis + 1]) ++axis;
    const int j = a.shared ? p : p - a.first[axis];
    const int n = a.shared ? a.pairs : a.first[axis + 1] - a.first[axis];
    // 2 j of 2 n elements; 2 / pi quarter turns a radian
    freq[p] = exp2(-a.log2_theta * ((double)j / n)) * 0.63661977236758134308;
    axis_of[p] = axis;
  }
  __syncthreads();
  const int64_t token0 = (int64_t)blockIdx.x * kTableTokens;
  const int tokens = (int)min((int64_t)kTableTokens, a.tokens - token0);
  const P* positions = static_cast<const P*>(a.positions) + token0 * a.token_stride;
  float2* table = reinterpret_cast<float2*>(a.table) + token0 * a.pairs;
  const float inv = 1.0f / (float)a.pairs;
  for (int i = threadIdx.x; i < tokens * a.pairs; i += kTableThreads) {
    const int t = (int)(((float)i + 0.5f) * inv);  // i / pairs: i < 2^12, off by less than half
    const int p = i - t * a.pairs;
    table[i] =
        cos_sin((double)positions[t * a.token_stride + axis_of[p] * a.axis_stride] * freq[p]);
  }
}

// ---- norms and rotation ----------------------------------------------------

constexpr int kHeadThreads = 256;
constexpr int kMaxRowWaves = 8;
constexpr int kMaxHeadsOfLane = 5;

// A lane's place in a head of `chunks` chunks, and the pairs behind its entries.
template <bool HALVES>
struct Place {
  int c0, c1;         // chunks of 8 elements
  bool in0, in1;      // ... inside the head
  bool turn0, turn1;  // ... rotated
  int p0, p1;         // first of the four pairs of (HALVES: either half of) them
  __device__ Place(int t, int d, int pairs) {
    const int chunks = d / 8;
    if (HALVES) {
      const int p8 = pairs / 8;
      const bool turned = t < p8;
      c0 = turned ? t : 2 * p8 + 2 * (t - p8);
      c1 = turned ? t + p8 : c0 + 1;
      turn0 = turn1 = turned;
      p0 = 8 * t;
      p1 = p0 + 4;
    } else {
      c0 = t;
      c1 = t + (chunks + 1) / 2;
      p0 = 4 * c0;
      p1 = 4 * c1;
      turn0 = p0 < pairs;
      turn1 = p1 < pairs;
      if (t >= (chunks + 1) / 2) c0 = chunks;  // a lane without a chunk
    }
    in0 = c0 < chunks;
    in1 = c1 < chunks;
    turn0 &= in0;
    turn1 &= in1;
  }
};

// The lane's 8 (cos, sin), anything where it turns nothing.
template <bool HALVES>
__device__ __forceinline__ void load_turns(const HeadsArgs& a, const Place<HALVES>& pl,
                                           int64_t token, float (&cs)[8], float (&sn)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) cs[e] = 1.f, sn[e] = 0.f;
  if (!a.table) return;
  const uint32_t row =
      a.table_rows == a.tokens ? (uint32_t)token : (uint32_t)token % (uint32_t)a.table_rows;
  const float* from = a.table + (int64_t)row * a.pairs * 2;
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    if (!(half ? pl.turn1 : pl.turn0)) continue;
    const float4* f = reinterpret_cast<const float4*>(from + (half ? pl.p1 : pl.p0) * 2);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int at = 4 * half + 2 * i;
      const float4 v = f[i];
      cs[at] = v.x, sn[at] = v.y, cs[at + 1] = v.z, sn[at + 1] = v.w;
    }
  }
}

// Elements that are not rotated stay as they are: (1, 0) would make a NaN of the neighbour of
// an infinity, and lose the sign of a zero.
template <bool HALVES>
__device__ __forceinline__ void turn(float (&v)[2][8], const Place<HALVES>& pl,
                                     const float (&cs)[8], const float (&sn)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const bool turned = HALVES || e < 4 ? pl.turn0 : pl.turn1;
    float& x = HALVES ? v[0][e] : v[e >> 2][2 * (e & 3)];
    float& y = HALVES ? v[1][e] : v[e >> 2][2 * (e & 3) + 1];
    const float p = x, q = y;
    x = turned ? __builtin_fmaf(p, cs[e], -(q * sn[e])) : p;
    y = turned ? __builtin_fmaf(q, cs[e], p * sn[e]) : q;
  }
}

template <bool F16>
__device__ __forceinline__ u4 pack8(const float (&f)[8]) {
  return (u4){pack16x2<F16>(f[0], f[1]), pack16x2<F16>(f[2], f[3]), pack16x2<F16>(f[4], f[5]),
              pack16x2<F16>(f[6], f[7])};
}

// A norm's span: 2^shift lanes of a wave, or `waves` waves of the block, one slot
// each in `part`.
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
constexpr int kPartSlots = 5 * kMaxRowWaves;

// What a norm does to its span: v = (x 2^-by - mean) r.
struct Norm {
  float mean, r;
  int by;
};

// Of N heads' packed values (absent chunks hold 0). Squares leave fp32's range where
// bf16 values do not, so a span whose mean square is not in [2^-100, inf) is taken
// again with a power of two out of it and of eps, exactly (`scaled` is set for the
// wave; spans that share it repeat theirs with 2^0, to the same bits).
template <int N, bool F16>
__device__ __forceinline__ Norm norm_of(u4 (*xw)[2], const bool (*in)[2], NormKind kind,
                                        float count, float eps, const Span& sp, float* part,
                                        bool* scaled) {
  Norm n = {0.f, 1.f, 0};
  if (kind == NormKind::kNone) return n;
  const bool layer = kind == NormKind::kLayer;
  // f over the values, chunk by chunk
  auto sum_of = [&](auto f) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float v[8], c = 0.f;
        mx4_unpack8<F16>(xw[i][j], v);
#pragma unroll
        for (int e = 0; e < 8; ++e) c = f(v[e], c);
        s += in[i][j] ? c : 0.f;
        // the next pass unpacks again: unpacked values are not held over
        asm volatile("" : "+v"(xw[i][j]));
      }
    return s;
  };
  if (layer)
    n.mean = span_sum(sum_of([](float x, float c) { return c + x; }), sp, part) / count;
  const float mean = n.mean;
  float q = layer ? sum_of([=](float x, float c) {
    return __builtin_fmaf(x - mean, x - mean, c);
  })
                  : sum_of([](float x, float c) { return __builtin_fmaf(x, x, c); });
  float ms = span_sum(q, sp, part + kMaxRowWaves) / count + eps;
  const bool again = !(ms >= 0x1p-100f && ms < __builtin_inff());
  if (__builtin_expect(__any(again), 0)) {
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float v[8];
        mx4_unpack8<F16>(xw[i][j], v);
#pragma unroll
        for (int e = 0; e < 8; ++e) top = max(top, __float_as_uint(v[e]) & 0x7FFFFFFFu);
      }
    top = span_max(top, sp, part + 2 * kMaxRowWaves) >> 23;
    int by = max((int)top - 127, ((int)(__float_as_uint(eps) >> 23) - 127) >> 1) - 40;
    if (!again || top == 255) by = 0;  // an infinity or a NaN gives what it gave
    if (layer)
      n.mean = span_sum(sum_of([=](float x, float c) { return c + __builtin_ldexpf(x, -by); }),
                        sp, part + 3 * kMaxRowWaves) /
               count;
    const float m = n.mean;
    q = sum_of([=](float x, float c) {
      const float v = __builtin_ldexpf(x, -by) - m;
      return __builtin_fmaf(v, v, c);
    });
    ms = span_sum(q, sp, part + 4 * kMaxRowWaves) / count + __builtin_ldexpf(eps, -2 * by);
    n.by = by;
    *scaled = true;
  }
  n.r = 1.0f / sqrtf(ms);
  return n;
}

// How the heads of one tensor lie on lanes: 2^lanes_shift lanes a head. A unit is a
// token's heads, or NI per lane group of them for norms of single heads: 2^shift lanes
// of a wave, or a block's `waves`.
struct HeadsShape {
  int lanes_shift;
  struct {
    int shift, segments;
    uint32_t blocks;
  } t[2];
  int waves;
  int64_t grid;  // blocks of both
  int threads() const { return waves > 1 ? 64 * waves : kHeadThreads; }
};

template <int NI, bool F16, bool HALVES, bool ROW>
__global__ __launch_bounds__(ROW ? 64 * kMaxRowWaves : kHeadThreads) void heads_kernel(
    HeadsArgs a, HeadsShape sh) {
  __shared__ float part[kPartSlots];
  const bool second = blockIdx.x >= sh.t[0].blocks;
  const HeadsTensor& x = a.t[second];
  const uint32_t block = blockIdx.x - (second ? sh.t[0].blocks : 0);
  const int ls = sh.lanes_shift;
  const int lane = threadIdx.x & ((1 << ls) - 1);
  int64_t unit;
  int g, groups;
  Span sp;
  if (ROW && sh.waves > 1) {
    unit = block;
    g = threadIdx.x >> ls;
    groups = blockDim.x >> ls;
    sp = {6, sh.waves};
  } else {
    const int shift = sh.t[second].shift;
    unit = (int64_t)block * (kHeadThreads >> shift) + (threadIdx.x >> shift);
    g = (threadIdx.x & ((1 << shift) - 1)) >> ls;
    groups = 1 << (shift - ls);
    sp = {ROW ? shift : ls, 1};
  }
  int64_t token = unit;
  int first = g;
  if (!ROW && sh.t[second].segments > 1) {
    const uint32_t n = sh.t[second].segments;  // units below 2^32
    token = (uint32_t)unit / n;
    first += (int)((uint32_t)unit - (uint32_t)token * n) * groups * NI;
  }
  const bool live = token < a.tokens;  // the others go along and write nothing
  if (!live) token = a.tokens - 1;
  const Place<HALVES> pl(lane, a.d, a.pairs);
  const u4 zero = {0, 0, 0, 0};
  u4 xw[NI][2];
  bool in[NI][2];
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int head = first + i * groups;
    const bool held = head < x.heads;
    in[i][0] = held && pl.in0;
    in[i][1] = held && pl.in1;
    const uint16_t* p = x.in + token * x.in_stride + (int64_t)head * x.in_head_stride;
    xw[i][0] = in[i][0] ? *reinterpret_cast<const u4*>(p + pl.c0 * 8) : zero;
    xw[i][1] = in[i][1] ? *reinterpret_cast<const u4*>(p + pl.c1 * 8) : zero;
  }
  float cs[8], sn[8];
  load_turns<HALVES>(a, pl, token, cs, sn);
  u4 ww[2] = {zero, zero};
  if (!ROW && x.weight) {
    if (pl.in0) ww[0] = *reinterpret_cast<const u4*>(x.weight + pl.c0 * 8);
    if (pl.in1) ww[1] = *reinterpret_cast<const u4*>(x.weight + pl.c1 * 8);
  }
  bool scaled = false;
  Norm all;
  if (ROW)
    all = norm_of<NI, F16>(xw, in, a.norm, (float)(a.d * x.heads), a.eps, sp, part, &scaled);
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int head = first + i * groups;
    if (ROW && x.weight) {
      const uint16_t* w = x.weight + (int64_t)head * a.d;
      if (in[i][0]) ww[0] = *reinterpret_cast<const u4*>(w + pl.c0 * 8);
      if (in[i][1]) ww[1] = *reinterpret_cast<const u4*>(w + pl.c1 * 8);
    }
    const Norm n = ROW ? all
                       : norm_of<1, F16>(&xw[i], &in[i], a.norm, (float)a.d, a.eps, sp, nullptr,
                                         &scaled);
    float v[2][8];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      mx4_unpack8<F16>(xw[i][j], v[j]);
      if (__builtin_expect(scaled, 0)) {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[j][e] = __builtin_ldexpf(v[j][e], -n.by);
      }
      if (a.norm != NormKind::kNone) {
        if (a.norm == NormKind::kLayer) {
#pragma unroll
          for (int e = 0; e < 8; ++e) v[j][e] -= n.mean;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) v[j][e] *= n.r;
      }
      if (x.weight) {
        float w[8];
        mx4_unpack8<F16>(ww[j], w);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[j][e] *= w[e];
      }
    }
    if (a.table) turn<HALVES>(v, pl, cs, sn);
    uint16_t* o = x.out + token * x.out_stride + (int64_t)head * x.out_head_stride;
    if (live && in[i][0]) *reinterpret_cast<u4*>(o + pl.c0 * 8) = pack8<F16>(v[0]);
    if (live && in[i][1]) *reinterpret_cast<u4*>(o + pl.c1 * 8) = pack8<F16>(v[1]);
  }
}

int log2_up(int64_t n) {
  int s = 0;
  while (((int64_t)1 << s) < n) ++s;
  return s;
}

// lanes of a head: two chunks each
int lanes_shift(int d) { return log2_up((d / 8 + 1) / 2); }

// Lanes of a unit that takes `heads` heads, ni per lane group: a power of two within a
// wave, whole waves beyond.
int64_t unit_lanes(int64_t heads, int ls, int ni) {
  const int64_t lanes = ((heads + ni - 1) / ni) << ls;
  return lanes <= 64 ? (int64_t)1 << log2_up(lanes) : (lanes + 63) / 64 * 64;
}

// Heads per lane group. Single heads: two, if that leaves the card filled (4608 tokens x
// 30 heads of 128: one 29.8 us, two 25.9, four 27.3; 32760 x 24 of 64: 95, 82, 84). Rows
// of up to four waves: one (4608 x 30 of 128: 26.9 us, two 27.9, four 30.4; 16384 x 16 of
// 256: 103.5, 102.7, 109). Longer rows: the number that leaves fewest lanes idle, the
// larger of equals, as fewer waves wait for each other (32760 x 40 of 128: one 280 us on
// five waves, two 265, three 263, four 284 with a third of the lanes idle, five 257 on one).
// By sizes alone: how a row's sum is cut decides its last bit.
constexpr int64_t kFilled = 256 * 2048;  // threads of a full card
int heads_of_lane(const HeadsArgs& a, int ls) {
  const int64_t most = a.t[0].heads > a.t[1].heads ? a.t[0].heads : a.t[1].heads;
  const int64_t lanes1 = unit_lanes(most, ls, 1);
  if (!a.row) return most > 1 && a.tokens * lanes1 >= kFilled ? 2 : 1;
  if (lanes1 <= 256) return 1;
  int best = 0;
  double held = 0;
  for (int ni = 1; ni <= kMaxHeadsOfLane; ++ni) {
    const int64_t lanes = unit_lanes(most, ls, ni);
    if (lanes > 64 * kMaxRowWaves) continue;
    // few tokens: as many waves as there are
    if (best && a.tokens * lanes < kFilled) break;
    const double use = (double)(most << ls) / (double)(lanes * ni);
    if (use >= held) {
      best = ni;
      held = use;
    }
  }
  return best;
}

HeadsShape shape(const HeadsArgs& a, int ni) {
  HeadsShape sh = {};
  sh.lanes_shift = lanes_shift(a.d);
  sh.waves = 1;
  if (a.row)
    for (const HeadsTensor& x : a.t) {
      const int64_t waves = (unit_lanes(x.heads, sh.lanes_shift, ni) + 63) / 64;
      if (waves > sh.waves) sh.waves = (int)waves;
    }
  for (int i = 0; i < 2; ++i) {
    if (!a.t[i].heads) continue;
    int64_t lanes = unit_lanes(a.t[i].heads, sh.lanes_shift, ni);
    sh.t[i].segments = a.row || lanes <= 64 ? 1 : (int)(lanes / 64);
    if (lanes > 64) lanes = 64;
    sh.t[i].shift = log2_up(lanes);
    const int64_t per = sh.waves > 1 ? 1 : kHeadThreads / lanes;
    const int64_t blocks = (a.tokens * sh.t[i].segments + per - 1) / per;
    sh.t[i].blocks = (uint32_t)blocks;
    sh.grid += blocks;
  }
  return sh;
}

template <int NI, bool F16, bool HALVES>
hipError_t launch_ni(const HeadsArgs& a, hipStream_t st) {
  const HeadsShape sh = shape(a, NI);
  const dim3 grid((uint32_t)sh.grid), block(sh.threads());
  if (a.row)
    heads_kernel<NI, F16, HALVES, true><<<grid, block, 0, st>>>(a, sh);
  else
    heads_kernel<NI, F16, HALVES, false><<<grid, block, 0, st>>>(a, sh);
  return hipGetLastError();
}

template <bool F16, bool HALVES>
hipError_t launch(const HeadsArgs& a, hipStream_t st) {
  switch (heads_of_lane(a, lanes_shift(a.d))) {
    case 1: return launch_ni<1, F16, HALVES>(a, st);
    case 2: return launch_ni<2, F16, HALVES>(a, st);
    case 3: return launch_ni<3, F16, HALVES>(a, st);
    case 4: return launch_ni<4, F16, HALVES>(a, st);
    default: return launch_ni<5, F16, HALVES>(a, st);
  }
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

bool heads_row_fits(int64_t heads, int d) { return (heads << lanes_shift(d)) <= 2048; }

bool heads_grid_fits(const HeadsArgs& a) {
  const HeadsShape sh = shape(a, heads_of_lane(a, lanes_shift(a.d)));
  return sh.grid * (sh.threads() / 64) <= kMaxLaunchWaves;
}

hipError_t launch_qk_norm_rope(const HeadsArgs& a, bool halves, DType dt, hipStream_t st) {
  if (a.tokens == 0) return hipSuccess;
  if (dt == DType::kF16) return halves ? launch<true, true>(a, st) : launch<true, false>(a, st);
  return halves ? launch<false, true>(a, st) : launch<false, false>(a, st);
}

}  // namespace convrot
