// Attention over packed sequences (gfx950): out = softmax(scale q k^T) v for each
// sequence and head, query heads in groups that share a key head.
//
// One pass over the keys with a running maximum m and sum l of each row's
// softmax: a tile of scores s raises m to m', and l and the accumulated output
// are scaled by 2^(c (m - m')) before the tile's p = 2^(c (s - m')) are added
// (c = scale log2 e). A row is a (query, head of the group) pair, so that a
// group's heads read their keys together.
//
// Scores are formed transposed, S^T = K Q^T, 32 keys x 32 rows an MFMA tile: a
// lane then holds 16 keys of one row, so that maxima and sums are its own but
// for one exchange with the lane 32 away, and P^T, rounded to 16 bits, is in
// the layout of the second product's operand as it is: O^T += V^T P^T, whose
// contraction takes keys in the order in which the first product's result has
// them. V^T comes from LDS through the transposing reads.
//
// That rounding of the weights is half a step of the inputs' type each, as v's own was
// (their sum is taken before, in fp32): the output is off by 0.0023 of its norm in bf16 for
// 0.0017 of one that is rounded once. A second 16-bit part of each weight takes half as many
// products again, which is what bounds these kernels; the one for few rows waits for memory
// and carries it.

#include <type_traits>
#include <utility>

#include "attention.h"
#include "lds_copy.h"

namespace convrot {

namespace {

typedef __bf16 bf8 __attribute__((ext_vector_type(8)));
typedef _Float16 hf8 __attribute__((ext_vector_type(8)));
typedef float v16f __attribute__((ext_vector_type(16)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef short s4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) volatile int* lds_ints;

constexpr int kTileKeys = 64;   // keys of a copied tile
constexpr int kRowsOfTile = 128;
constexpr int kRowsOfWide = 256;
constexpr int kFewUnits = 4;     // least units of a part, few rows
constexpr int kMaxSplits = 512;  // of a row's keys: two rounds of a block per compute unit
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;
// A row's reference m is a largest score of it: it is raised when a score passes it by
// kRoom / c, so weights stay below 2^(kRoom + kLift). Half weights are lifted so that
// those of 2^-18 of the reference's are normal numbers; the sum is lifted with them.
template <bool F16>
constexpr float kRoom = F16 ? 10.f : 32.f;
template <bool F16>
constexpr float kLift = F16 ? 4.f : 0.f;
constexpr float kLowest = -3.402823466e38f;
// Scores start from -m, so those formed below a reference far under zero have only its
// bits. A first pass takes no reference below kDeepest / c, which leaves a weight right to
// 2^-14; scores there get none. Beside a reference above kDeep / c they have none, and a
// row whose reference ends lower, or that has seen nothing above, is gone over again.
constexpr float kDeepest = -256.f;
constexpr float kDeep = -192.f;
// bf16 values may be so large (above 2^96 / keys) that such weights take their sum out of
// fp32 (half ones, below 2^16, are not). A block in whose result something is not finite,
// although the sum of the weights is, goes over its keys again with the reference raised at
// every larger score and 2^32 above it, so that no row's weights sum to more than 1: the
// elements that are finite then replace those that were not, the others stay. Looking costs
// an instruction for two elements of the result and a barrier; 4608 x 4608 x 30 heads take 310
// us, with an infinite value that every row sees 850, with every row formed exactly 710.
constexpr float kOver = 32.f;
constexpr float kMostOver = 1e36f;  // finite where the scale is next to nothing
template <bool F16>
struct Pass {
  static constexpr bool kAgain = !F16;
  float room, over;  // of the first
  __device__ Pass(float c) : room(kRoom<F16> / c), over(0.f) {}
  __device__ void again(float c) {
    over = fminf(kOver / c, kMostOver);
    room = -over;
  }
  __device__ bool first() const { return !kAgain || over == 0.f; }
};

// EXACT: any reference, and the scores that make a row leave one far under zero are formed
// again from zero: whether m is that far under it, the largest of them being `top` above m.
__device__ __forceinline__ bool leaves_far(float below, float top) {
  return below > 2.f * __builtin_fabsf(top - below);
}

// What a row's scores have to pass before it has a reference, and whether it has one by the
// bound that it keeps.
template <bool EXACT>
__device__ __forceinline__ float no_reference(float c) {
  return EXACT ? -__builtin_inff() : kDeepest / c;
}
template <bool EXACT>
__device__ __forceinline__ bool referred(float raise_at) {
  return EXACT ? raise_at > kLowest : raise_at > 0.f;
}

// What a wave finds in its rows' results: elements that are not finite though the sum of
// their weights is, and rows that have to be formed exactly. Those are rows with a reference
// below kDeep or none (m 0) though they see keys, and, where the head is padded, rows whose
// sum is NaN: the chunks behind the head's end repeat its last one in LDS, and an infinity
// there met the query's zeros. An exact pass takes zeros for them.
struct Found {
  bool lost;
  uint64_t inexact;  // rows of the wave
};
// The rows, 32 of which two lanes each hold, of which some lane says so.
__device__ __forceinline__ uint32_t rows_where(bool what) {
  const uint64_t lanes = __ballot(what);
  return (uint32_t)lanes | (uint32_t)(lanes >> 32);
}
template <int DP>
__device__ __forceinline__ bool is_inexact(float mc, float l, bool sees, int d) {
  return mc < kDeep || (l == 0.f && sees) || (d < DP && l != l);
}
// Elements from 8 chunk on of a head of d.
__device__ __forceinline__ u4 inside_head(const u4& w, int chunk, int d) {
  const u4 zero = {0, 0, 0, 0};
  return chunk * 8 < d ? w : zero;
}

template <bool F16>
__device__ __forceinline__ v16f mfma(const u4& a, const u4& b, const v16f& c) {
  if constexpr (F16)
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(hf8, a),
                                                  __builtin_bit_cast(hf8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf8, a),
                                                   __builtin_bit_cast(bf8, b), c, 0, 0, 0);
}

// A head of DP elements (padded) in LDS: rows of DP / 8 chunks of 16 bytes, a row's
// chunks permuted so that neither kind of read meets a bank twice: rows of K are
// read 16 lanes to one chunk of 16 rows, rows of V four lanes to 32 bytes of a row.
template <int DP>
__device__ __forceinline__ int k_slot(int row, int chunk) {
  return DP == 64 ? chunk ^ ((row >> 1) & 7) : chunk ^ (row & 15);
}
template <int DP>
__device__ __forceinline__ int v_slot(int row, int chunk) {
  return DP == 64 ? chunk ^ (((row >> 1) & 1) << 2) : chunk ^ ((row & 3) << 2);
}

template <typename F, int... I>
__device__ __forceinline__ void static_for_each(F& f, std::integer_sequence<int, I...>) {
  (f(std::integral_constant<int, I>{}), ...);
}
// f(0), f(1), .. as constants
template <int N, typename F>
__device__ __forceinline__ void static_for(F f) {
  static_for_each(f, std::make_integer_sequence<int, N>{});
}

__device__ __forceinline__ int wave_number(int tid) {
  return __builtin_amdgcn_readfirstlane(tid >> 6);
}

// The thread's number once more, of which the compiler does not know that it is the same:
// nothing worked out from it is kept in registers from one part of a kernel to the next.
__device__ __forceinline__ int thread_anew() {
  int tid = threadIdx.x;
  asm volatile("" : "+v"(tid));
  return tid;
}

__device__ __forceinline__ float other_half(float v) {
  typedef uint32_t u2v __attribute__((ext_vector_type(2)));
  const uint32_t a = __float_as_uint(v);
  const u2v r = __builtin_amdgcn_permlane32_swap(a, a, false, false);
  return __uint_as_float((threadIdx.x & 32) ? r.x : r.y);
}

// Where a block works: a sequence's rows and keys.
struct Where {
  int q0, k0;  // first query and key
  int lq, lk;
  int tile;    // tile of the sequence's rows
};

// Sequence b of the call. Offsets are held inside the tensors whatever they are.
__device__ __forceinline__ Where sequence(const AttentionArgs& a, int b) {
  Where w;
  int q1, k1;
  if (a.q_offsets) {
    w.q0 = min(max(a.q_offsets[b], 0), (int)a.q_tokens);
    q1 = min(max(a.q_offsets[b + 1], w.q0), (int)a.q_tokens);
  } else {
    w.q0 = b * a.q_each;
    q1 = w.q0 + a.q_each;
  }
  if (a.k_offsets) {
    w.k0 = min(max(a.k_offsets[b], 0), (int)a.k_tokens);
    k1 = min(max(a.k_offsets[b + 1], w.k0), (int)a.k_tokens);
  } else {
    w.k0 = b * a.k_each;
    k1 = w.k0 + a.k_each;
  }
  w.lq = q1 - w.q0;
  w.lk = k1 - w.k0;
  if (a.k_lens) w.lk = min(max(a.k_lens[b], 0), w.lk);
  return w;
}

// The sequence and tile of a slot: tiles of ROWS rows counted through the
// sequences, 64 of them at a time. False behind the last. A slot is below 2^23
// (a grid's blocks), rows (query, head of the group) of all sequences below 2^31.
template <int ROWS>
__device__ bool find(const AttentionArgs& a, uint32_t slot, Where* w) {
  if (!a.q_offsets || a.batch == 1) {  // no counting
    const uint32_t tiles = (uint32_t)(a.q_each * a.group + ROWS - 1) / ROWS;
    const uint32_t b = a.batch == 1 ? 0 : slot / max(tiles, 1u);
    if (b >= (uint32_t)a.batch) return false;
    *w = sequence(a, b);
    w->tile = (int)(slot - b * tiles);
    return w->tile * ROWS < w->lq * a.group;
  }
  const int lane = threadIdx.x & 63;
  uint32_t before = 0;
  for (int base = 0; base < a.batch; base += 64) {
    const int b = base + lane;
    uint32_t upto = 0;
    if (b < a.batch) {
      const int lo = min(max(a.q_offsets[b], 0), (int)a.q_tokens);
      const int hi = min(max(a.q_offsets[b + 1], lo), (int)a.q_tokens);
      upto = (uint32_t)((hi - lo) * a.group + ROWS - 1) / ROWS;  // < 2^26: 64 of them < 2^32
    }
#pragma unroll
    for (int s = 1; s < 64; s <<= 1) {
      const uint32_t below = __shfl_up(upto, s);
      if (lane >= s) upto += below;
    }
    // before <= slot here, so the difference is below 2^23
    const uint64_t past = __ballot(upto > slot - before);
    if (past) {
      const int at = __builtin_ctzll(past);
      const uint32_t first = at ? __builtin_amdgcn_readlane(upto, at - 1) : 0;
      *w = sequence(a, base + at);
      w->tile = (int)(slot - before - first);
      return true;
    }
    before += __builtin_amdgcn_readlane(upto, 63);
  }
  return false;
}

// V^T of 16 keys for the second product, 32 elements of the head: keys 4 half + .. and
// those 8 further, the order in which the first product leaves a row's keys.
template <int DP>
__device__ __forceinline__ u4 values(const uint8_t* vt, int key, int dtile) {
  typedef __attribute__((address_space(3))) s4* lp;
  const int lane = threadIdx.x & 63;
  const int r = key + (lane >> 5) * 4 + ((lane & 15) >> 2);
  const int chunk = dtile * 4 + ((lane >> 4) & 1) * 2 + ((lane & 3) >> 1);
  const int at = r * DP * 2 + v_slot<DP>(r, chunk) * 16 + (lane & 1) * 8;
  uint8_t* p = const_cast<uint8_t*>(vt) + at;
  const u2 w0 = __builtin_bit_cast(u2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lp)p));
  const u2 w1 =
      __builtin_bit_cast(u2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lp)(p + 8 * DP * 2)));
  return (u4){w0.x, w0.y, w1.x, w1.y};
}

template <int DP, int NW>
struct Kernel {
  static constexpr int kRows = 32 * NW;              // rows of a block
  static constexpr int kRowBytes = DP * 2;
  static constexpr int kChunks = DP / 8;
  static constexpr int kTileBytes = kTileKeys * kRowBytes;
  static constexpr int kStages = 2;
  static constexpr int kLds = 2 * kStages * kTileBytes + 16;  // and a flag
  static constexpr int kCopies = kTileBytes / 1024 / NW;  // of a wave, per tile and operand
  static constexpr int kSteps = DP / 16;
  static constexpr int kDTiles = DP / 32;
};

// Values of keys that only some rows of a tile see, and those that fill a tile behind the
// last key. A weight of 0 does not cancel an infinity or a NaN in the product, so a tile
// in which some row's keys end is looked through, infinities and NaN in it are replaced
// by 0 (by every wave that finds one, before its own reads; they all write the same), and
// at the end each row adds those of the keys that it sees.
template <bool F16>
constexpr uint32_t kExp16 = F16 ? 0x7C007C00u : 0x7F807F80u;
template <bool F16>
constexpr uint32_t kExpUnit16 = F16 ? 0x04000400u : 0x00800080u;  // its last bits

template <bool F16>
__device__ __forceinline__ bool nonfinite16(uint32_t h) {
  return (h & kExp16<F16> & 0xFFFFu) == (kExp16<F16> & 0xFFFFu);
}

// True if the tile holds an infinity or a NaN; none is left then.
template <bool F16, int DP, int KEYS>
__device__ __forceinline__ bool clear_nonfinite(uint8_t* vt) {
  int lane = threadIdx.x & 63;
  asm volatile("" : "+v"(lane));  // its addresses are not kept between tiles
  uint32_t found = 0;
#pragma unroll 1
  for (int i = lane; i < KEYS * DP / 8; i += 64) {
    const u4 w = *reinterpret_cast<const u4*>(vt + i * 16);
#pragma unroll
    for (int e = 0; e < 4; ++e)
      found |= ((w[e] & kExp16<F16>) + kExpUnit16<F16>) & 0x80008000u;
  }
  if (__builtin_expect(!__any(found != 0), 1)) return false;
#pragma unroll 1
  for (int i = lane; i < KEYS * DP / 2; i += 64) {
    uint32_t* at = reinterpret_cast<uint32_t*>(vt + i * 4);
    const uint32_t w = *at;
    const uint32_t keep = (nonfinite16<F16>(w & 0xFFFFu) ? 0u : 0xFFFFu) |
                          (nonfinite16<F16>(w >> 16) ? 0u : 0xFFFF0000u);
    if (keep != ~0u) *at = w & keep;
  }
  wait_lgkm0();
  return true;
}

// What key `key` of the tensor has of them, added to a row that sees it.
template <int DTILES, bool F16>
__device__ __forceinline__ void add_nonfinite(const AttentionArgs& a, int64_t key, int hk,
                                              bool sees, v16f (&o)[DTILES]) {
  const int half = (threadIdx.x >> 5) & 1;
  const uint16_t* vr = a.v + key * a.v_stride + (int64_t)hk * a.v_head_stride;
#pragma unroll
  for (int d = 0; d < DTILES; ++d) {
    asm volatile("" ::: "memory");  // one tile's loads at a time
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int e = d * 32 + 8 * (i >> 2) + 4 * half + (i & 3);
      const uint32_t h = e < a.d ? vr[e] : 0;
      if (sees && nonfinite16<F16>(h)) o[d][i] += lo16<F16>(h);
    }
  }
}

// What the kernels for many rows are called with: slots per key head, XCDs, and how many of
// those share a key head.
struct TileCall {
  AttentionArgs a;
  uint32_t slots, xcds, share;
};

// A block's tile of rows and its keys.
struct Tile {
  Where w;
  int hk;           // key head
  int rows, row0;   // of the sequence, first of the tile
  int shift;        // query i sees keys below i + shift (causal)
  int end, full;    // keys that the tile's last query sees, that all of them see
  int t0, tiles;    // key tiles [t0, tiles)
  bool tail;        // a part of a split tile,
  uint32_t piece;   // ... this one
};

// Blocks of an XCD (they are dealt in turn) take neighbouring tiles of the same heads,
// whose keys then meet in its L2. Causal tiles differ in length, so XCDs that share
// heads take a head's tiles in turn. The first a.whole tiles are a block's each, the
// last ones are split. False for a block without a tile.
template <int ROWS, bool CAUSAL>
__device__ __forceinline__ bool locate(const TileCall& call, uint32_t block, Tile* t) {
  const AttentionArgs& a = call.a;
  const uint32_t slots = call.slots, xcds = call.xcds, share = call.share;
  t->tail = a.splits > 1 && block >= a.whole;
  uint32_t id = t->tail ? block - a.whole : block;
  if (CAUSAL && !t->tail) {
    const uint32_t x = id % xcds, heads = (uint32_t)a.k_heads * share / xcds;
    const uint32_t at = id / xcds * share + x % share;
    if (at >= heads * slots) return false;
    id = x / share * heads * slots + at;
  } else {
    const uint32_t total = t->tail ? gridDim.x - a.whole : a.splits > 1 ? a.whole : gridDim.x;
    const uint32_t full = total / xcds, rest = total % xcds;
    const uint32_t x = id % xcds, i = id / xcds;
    id = x * full + min(x, rest) + i;
  }
  t->piece = id;
  uint32_t split = 0;
  if (t->tail) {
    split = id % (uint32_t)a.splits;
    id = a.whole + id / (uint32_t)a.splits;
  }
  uint32_t slot = id % slots;
  t->hk = (int)(id / slots);
  if (CAUSAL) slot = slots - 1 - slot;  // long tiles first
  Where& w = t->w;
  const bool found = find<ROWS>(a, slot, &w);
  t->rows = w.lq * a.group;  // < 2^31 checked
  t->row0 = w.tile * ROWS;
  if (t->tail && split == 0 && threadIdx.x < ROWS) {
    // which row of the output each of the tile's is
    const int r = t->row0 + (int)threadIdx.x;
    int64_t to = -1;
    if (found && r < t->rows)
      to = (int64_t)(w.q0 + r / a.group) * a.q_heads + t->hk * a.group + r % a.group;
    a.part_map[(int64_t)(id - a.whole) * ROWS + threadIdx.x] = to;
  }
  if (!found) return false;
  t->shift = w.lk - w.lq + 1;
  t->end = t->full = w.lk;
  if (CAUSAL) {
    const int last = min(t->rows - 1, t->row0 + ROWS - 1) / a.group, first = t->row0 / a.group;
    t->end = min(w.lk, max(0, last + t->shift));
    t->full = min(w.lk, max(0, first + t->shift));
  }
  t->t0 = 0;
  t->tiles = (t->end + kTileKeys - 1) / kTileKeys;
  if (t->tail) {
    const int per = (t->tiles + a.splits - 1) / a.splits;
    t->t0 = min(t->tiles, (int)split * per);
    t->tiles = min(t->tiles, t->t0 + per);
  }
  return true;
}

// What a second pass leaves of the first one's results and its own.
__device__ __forceinline__ v4f finite_of(v4f before, v4f now) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const bool keep = __builtin_fabsf(before[i]) < __builtin_inff() ||
                      !(__builtin_fabsf(now[i]) < __builtin_inff());
    now[i] = keep ? before[i] : now[i];
  }
  return now;
}
template <bool F16, typename U>
__device__ __forceinline__ U finite_of16(U before, U now) {
#pragma unroll
  for (int i = 0; i < (int)(sizeof(U) / 4); ++i) {
    uint32_t take = 0;
#pragma unroll
    for (int h = 0; h < 32; h += 16)
      if (nonfinite16<F16>(before[i] >> h) && !nonfinite16<F16>(now[i] >> h)) take |= 0xFFFFu << h;
    now[i] = (now[i] & take) | (before[i] & ~take);
  }
  return now;
}

// A row's result, of which this lane holds o, its part l of the sum and the reference m.
// True if something in it is not finite though its sum is.
template <int ROWS, int DTILES, bool F16>
__device__ __forceinline__ bool finish(const AttentionArgs& a, const Tile& t, int row, float l,
                                       float m, float c, const v16f (&o)[DTILES], bool first,
                                       bool write) {
  const int half = (thread_anew() >> 5) & 1;
  const float sum = l + other_half(l);
  const bool some = sum > 0.f || sum != sum;
  const float inv = some ? 1.0f / sum : 0.f;
  const float lse2 = some ? log2f(sum) - kLift<F16> + m * c : -__builtin_inff();
  if (row >= t.rows || !write) return false;
  float most = 0.f;  // infinite or NaN once something is
  if (Pass<F16>::kAgain) {
#pragma unroll
    for (int d = 0; d < DTILES; ++d)
#pragma unroll
      for (int i = 0; i < 16; ++i)
        most = __builtin_elementwise_maximum(most, __builtin_fabsf(o[d][i]));
  }
  const bool lost = !(most < __builtin_inff()) && sum < __builtin_inff();
  if (t.tail) {
    const int64_t at = (int64_t)t.piece * ROWS + row - t.row0;
    if (half == 0 && first) a.part_lse[at] = lse2;
    if (!some) return false;
    float* to = a.part + at * a.d;
#pragma unroll
    for (int d = 0; d < DTILES; ++d)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int e = d * 32 + i * 8 + half * 4;
        v4f f = {o[d][4 * i] * inv, o[d][4 * i + 1] * inv, o[d][4 * i + 2] * inv,
                 o[d][4 * i + 3] * inv};
        if (e >= a.d) continue;
        if (!first) f = finite_of(*reinterpret_cast<const v4f*>(to + e), f);
        *reinterpret_cast<v4f*>(to + e) = f;
      }
    return lost;
  }
  const int token = t.w.q0 + row / a.group, head = t.hk * a.group + row % a.group;
  if (a.lse && half == 0 && first) a.lse[(int64_t)head * a.q_tokens + token] = lse2 * kLn2;
  uint16_t* to = a.out + (int64_t)token * a.out_stride + (int64_t)head * a.out_head_stride;
  // the two lanes of a row hold four elements of each eight: they swap, so that each
  // has every other eight
#pragma unroll
  for (int d = 0; d < DTILES; ++d)
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
      u4 f;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        typedef uint32_t u2v __attribute__((ext_vector_type(2)));
        const int n = 4 * i + 2 * j;
        const u2v x = __builtin_amdgcn_permlane32_swap(
            pack16x2<F16>(o[d][n] * inv, o[d][n + 1] * inv),
            pack16x2<F16>(o[d][n + 4] * inv, o[d][n + 5] * inv), false, false);
        f[j] = x.x;
        f[2 + j] = x.y;
      }
      const int e = d * 32 + (i + half) * 8;
      if (e >= a.d) continue;
      if (!first) f = finite_of16<F16>(*reinterpret_cast<const u4*>(to + e), f);
      *reinterpret_cast<u4*>(to + e) = f;
    }
  return lost;
}

// What some wave of a block finds, noted in a flag for all of them, which come here with
// what they found. What a block then does again is code of its own: as the same code in a
// loop it kept so much from one pass to the next that the first one of 32760 x 512 keys x 40
// heads took 444 us for 427.
__device__ __forceinline__ void note(bool what, lds_ints flag) {
  if (__builtin_expect(__any(what), 0)) *flag = 1;
}
__device__ __forceinline__ void all_noted() {
  wait_lgkm0();
  lds_barrier();
}

// The kernel's arguments (its only parameter) and the block's number once more, as
// thread_anew's.
template <typename C>
__device__ __forceinline__ C call_anew() {
  auto from = (const __attribute__((address_space(4))) C*)__builtin_amdgcn_kernarg_segment_ptr();
  asm volatile("" : "+s"(from));
  C call;
  __builtin_memcpy(&call, from, sizeof(C));
  return call;
}
__device__ __forceinline__ uint32_t block_anew() {
  uint32_t block = blockIdx.x;
  asm volatile("" : "+s"(block));
  return block;
}

// The first key and value of a tile's head, as bytes.
__device__ __forceinline__ const int8_t* head_bytes(const uint16_t* p, const Where& w,
                                                    int64_t stride, int64_t head_stride, int hk) {
  return reinterpret_cast<const int8_t*>(p + (int64_t)w.k0 * stride + (int64_t)hk * head_stride);
}

// A row's query as the first product's operand, and how many keys it sees.
template <int STEPS, bool CAUSAL>
__device__ __forceinline__ void load_query(const AttentionArgs& a, const Where& w, int hk, int row,
                                           u4 (&qf)[STEPS], int* seen) {
  const int half = (thread_anew() >> 5) & 1;
  const int r = min(row, w.lq * a.group - 1);
  const int token = r / a.group, head = hk * a.group + r % a.group;
  *seen = CAUSAL ? min(w.lk, token + w.lk - w.lq + 1) : w.lk;
  const uint16_t* q =
      a.q + (int64_t)(w.q0 + token) * a.q_stride + (int64_t)head * a.q_head_stride;
#pragma unroll
  for (int s = 0; s < STEPS; ++s) {
    const int e = (2 * s + half) * 8;
    const u4 zero = {0, 0, 0, 0};
    qf[s] = e < a.d ? *reinterpret_cast<const u4*>(q + e) : zero;
  }
}

// Scores of keys that a row does not see. The lane's sixteen keys of a unit are those at
// 8 i + 4 half + (0 .. 3).
__device__ __forceinline__ void mask(v16f* s, int key0, int seen) {
  const int left = seen - key0 - 4 * (int)((threadIdx.x >> 5) & 1);
#pragma unroll
  for (int i = 0; i < 16; ++i)
    if (8 * (i >> 2) + (i & 3) >= left) (*s)[i] = -__builtin_inff();
}

// ---- 128 rows a block: a wave's 32, tile after tile ----------------------------
//
// Two 64-key tiles of K and V in LDS, one in use and one on its way. Heads of 65 to 128
// elements run two blocks a compute unit, so that one block's start, softmax and end lie
// under the other's products: the better choice for keys of a few tiles and for rows that
// do not fill the card with 256 (16384 queries x 40 heads of 128 over 256 keys: 143 us, with
// 256 rows a block 180; over 4608: 1410 and 1333). 32760 x 40 heads over 512 keys take 430 us,
// 0.80 PFLOP/s: of a round's 21 us 6.5 are a block's start and end, and the MFMAs are
// busy 0.40 of the cycles at 2.0 GHz (power: fetching the next tile early gains nothing).
// Heads of up to 256: 8192 x 8 heads of 256 in 708 us (0.78 PFLOP/s), one block a compute
// unit, its output a whole 128 registers a lane: a SIMD has one wave, whose products, softmax
// and products follow one another, and the MFMAs are busy 0.32 of the cycles at 2.1 GHz.
// One pass of a wave's 32 rows, from row0 of the block's ROWS on, over the block's keys, U
// units of 32 at a time. Rows that `only` does not name are not written.
template <int DP, int NW, bool F16, bool CAUSAL, int ROWS, int U, bool EXACT>
__device__ __forceinline__ Found walk(const AttentionArgs& a, const Tile& w,
                                      const Pass<F16>& pass, uint8_t* lds, lds_ints flags,
                                      int tid, int row0, uint32_t only) {
  using T = Kernel<DP, NW>;
  const int lane = tid & 63;
  const int wave = wave_number(tid);
  const int half = lane >> 5, col = lane & 31;
  int seen;
  u4 qf[T::kSteps];
  load_query<T::kSteps, CAUSAL>(a, w.w, w.hk, w.row0 + row0 + col, qf, &seen);

  // copies: lane i of a copy fills the 16 bytes behind 16 i
  const int8_t* kbase = head_bytes(a.k, w.w, a.k_stride, a.k_head_stride, w.hk);
  const int8_t* vbase = head_bytes(a.v, w.w, a.v_stride, a.v_head_stride, w.hk);
  const uint32_t kstride = (uint32_t)a.k_stride * 2, vstride = (uint32_t)a.v_stride * 2;
  auto issue = [&](int t, int stage) {
    const int last = w.w.lk - 1 - t * kTileKeys;  // rows behind it repeat it
    const int8_t* kp = kbase + (int64_t)t * kTileKeys * a.k_stride * 2;
    const int8_t* vp = vbase + (int64_t)t * kTileKeys * a.v_stride * 2;
#pragma unroll
    for (int i = 0; i < T::kCopies; ++i) {
      const int at = (wave * T::kCopies + i) * 64;
      const int r = (at + lane) / T::kChunks, c = (at + lane) % T::kChunks;
      const int from = min(r, last);
      const int kc = min(k_slot<DP>(r, c), a.d / 8 - 1), vc = min(v_slot<DP>(r, c), a.d / 8 - 1);
      dma16(kp, from * kstride + kc * 16, stage * T::kTileBytes + at * 16);
      dma16(vp, from * vstride + vc * 16, (T::kStages + stage) * T::kTileBytes + at * 16);
    }
  };

  const float c = a.scale * kLog2e;
  v16f o[T::kDTiles];
  v16f below = (v16f){0};  // -m in every place: the first product starts from it
  float l = 0.f, raise_at = no_reference<EXACT>(c);
#pragma unroll
  for (int d = 0; d < T::kDTiles; ++d) o[d] = (v16f){0};

  if (w.t0 < w.tiles) issue(w.t0, 0);
  for (int t = w.t0; t < w.tiles; ++t) {
    const int stage = (t - w.t0) & 1;
    wait_vmcnt<0>();
    wait_lgkm0();
    lds_barrier();
    if (t + 1 < w.tiles) issue(t + 1, stage ^ 1);
    const uint8_t* kt = lds + stage * T::kTileBytes;
    uint8_t* vt = lds + (T::kStages + stage) * T::kTileBytes;
    const bool masked = (t + 1) * kTileKeys > w.full;
#pragma unroll 1
    for (int u0 = 0; u0 < 2; u0 += U) {
      v16f s[U];
      float top;
      // the units' scores from `from`, and the row's largest
      auto score = [&](const v16f& from) __attribute__((always_inline)) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
          s[u] = from;
#pragma unroll
          for (int st = 0; st < T::kSteps; ++st) {
            const int r = (u0 + u) * 32 + col;
            const u4 kf = *reinterpret_cast<const u4*>(kt + r * T::kRowBytes +
                                                       k_slot<DP>(r, 2 * st + half) * 16);
            s[u] = mfma<F16>(EXACT ? inside_head(kf, 2 * st + half, a.d) : kf, qf[st], s[u]);
          }
          if (masked) mask(&s[u], t * kTileKeys + (u0 + u) * 32, seen);
        }
        top = s[0][0];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int i = 0; i < 16; ++i) top = fmaxf(top, s[u][i]);
        top = fmaxf(top, other_half(top));
      };
      score(below);
      if (__any(top > raise_at)) {
        const bool up = top > raise_at;
        const float left = EXACT && up && leaves_far(below[0], top) ? below[0] : 0.f;
        if (EXACT && __any(left != 0.f)) {
#pragma unroll
          for (int i = 0; i < 16; ++i) below[i] = left != 0.f ? 0.f : below[i];
          score(below);
        }
        const float by = up ? top + pass.over : 0.f;
        // a row without an m has nothing to scale yet (or NaN, which stays)
        const float alpha =
            up && referred<EXACT>(raise_at) ? __builtin_amdgcn_exp2f(-(by + left) * c) : 1.f;
        raise_at = up ? pass.room : raise_at;
        l *= alpha;
#pragma unroll
        for (int i = 0; i < 16; ++i) below[i] -= by;
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int i = 0; i < 16; ++i) s[u][i] -= by;
#pragma unroll
        for (int d = 0; d < T::kDTiles; ++d)
#pragma unroll
          for (int i = 0; i < 16; ++i) o[d][i] *= alpha;
      }
      u4 p[U][2];
#pragma unroll
      for (int u = 0; u < U; ++u) {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          s[u][i] =
              __builtin_amdgcn_exp2f(F16 ? __builtin_fmaf(s[u][i], c, kLift<F16>) : s[u][i] * c);
          l += s[u][i];
        }
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            p[u][h][e] = pack16x2<F16>(s[u][8 * h + 2 * e], s[u][8 * h + 2 * e + 1]);
      }
      if (u0 == 0 && masked && clear_nonfinite<F16, DP, kTileKeys>(vt)) flags[0] = 1;
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int d = 0; d < T::kDTiles; ++d)
            o[d] = mfma<F16>(values<DP>(vt, (u0 + u) * 32 + h * 16, d), p[u][h], o[d]);
    }
  }

  if (CAUSAL || w.full % kTileKeys) {
    wait_lgkm0();
    lds_barrier();
    if (__builtin_expect(flags[0], 0)) {
      const int to = min(w.end, w.tiles * kTileKeys);
#pragma unroll 1
      for (int key = max(w.full / kTileKeys, w.t0) * kTileKeys; key < to; ++key)
        add_nonfinite<T::kDTiles, F16>(a, w.w.k0 + key, w.hk, key < seen, o);
    }
  }
  const int col_anew = thread_anew() & 31, row = w.row0 + row0 + col_anew;
  uint32_t inexact = 0;
  if (!EXACT)
    inexact = rows_where(row < w.rows && is_inexact<DP>(-below[0] * c, l + other_half(l),
                                                        seen > w.t0 * kTileKeys, a.d));
  return {finish<ROWS, T::kDTiles, F16>(a, w, row, l, -below[0], c, o, pass.first(),
                                        only >> col_anew & 1),
          inexact};
}

// What a block goes over again, QT times 32 rows a wave: rows that were inexact, and then,
// or instead, what was lost. The others stay, so that a row's bits do not depend on those
// beside it.
template <int DP, int QT, int NW, bool F16, bool CAUSAL>
__device__ __forceinline__ void walk_anew(bool exact, uint64_t rows, uint8_t* lds,
                                          lds_ints flags) {
  constexpr int kRows = 32 * QT * NW;
  const TileCall call = call_anew<TileCall>();
  const AttentionArgs& a = call.a;
  const int tid = thread_anew();
  Tile w;
  if (!locate<kRows, CAUSAL>(call, block_anew(), &w)) return;
  const float c = a.scale * kLog2e;
  Pass<F16> pass(c);
  bool lost;
  do {
    if (!exact) pass.again(c);
    lost = false;
#pragma unroll 1
    for (int q = 0; q < QT; ++q) {
      if (q > 0) lds_barrier();  // the last tile's reads are done
      const uint32_t only = exact ? (uint32_t)(rows >> (32 * q)) : ~0u;
      lost |= walk<DP, NW, F16, CAUSAL, kRows, 1, true>(a, w, pass, lds, flags, tid,
                                                        (wave_number(tid) * QT + q) * 32, only)
                  .lost;
    }
    if (!Pass<F16>::kAgain || !exact) return;
    exact = false;
    note(lost, flags + 1);
    all_noted();
  } while (flags[1]);
}

template <int DP, int QT, int NW, bool F16, bool CAUSAL>
__device__ __forceinline__ void finish_block(const Found& found, uint8_t* lds, lds_ints flags) {
  note(found.lost, flags + 1);
  note(found.inexact != 0, flags + 2);
  all_noted();
  const int exact = flags[2];
  if (__builtin_expect((exact | flags[1]) != 0, 0))
    walk_anew<DP, QT, NW, F16, CAUSAL>(exact != 0, found.inexact, lds, flags);
}

template <int DP, int NW, bool F16, bool CAUSAL>
__global__ __launch_bounds__(64 * NW, DP > 128 ? 1 : 2) void attention_kernel(TileCall call) {
  const AttentionArgs& a = call.a;
  using T = Kernel<DP, NW>;
  extern __shared__ __align__(1024) uint8_t lds[];
  lds_ints flags = (lds_ints)(lds + 2 * T::kStages * T::kTileBytes);
  if (threadIdx.x == 0) flags[0] = flags[1] = flags[2] = 0;  // a barrier follows in every tile
  Tile w;
  if (!locate<T::kRows, CAUSAL>(call, blockIdx.x, &w)) return;
  const Found found = walk<DP, NW, F16, CAUSAL, T::kRows, 2, false>(
      a, w, Pass<F16>(a.scale * kLog2e), lds, flags, threadIdx.x, wave_number(threadIdx.x) * 32,
      ~0u);
  finish_block<DP, 1, NW, F16, CAUSAL>(found, lds, flags);
}

// MFMAs of the pipeline below, whose accumulators stay where they are put: the output in
// accumulation registers, which no vector instruction but the rare rescaling touches.
// ACC: in accumulation registers. LAST: with the wait before anything else may read what
// it and those before it wrote, which copies that the compiler puts behind it do not
// know of.
template <bool F16, bool ACC, bool LAST = false>
__device__ __forceinline__ void mfma_out(v16f* o, const u4& v, const u4& p) {
#define CONVROT_MFMA_OUT(NAME, CLASS)                                                          \
  if constexpr (LAST)                                                                          \
    asm volatile(NAME " %0, %1, %2, %0\n\ts_nop 15" : CLASS(*o) : "v"(v), "v"(p));             \
  else                                                                                         \
    asm volatile(NAME " %0, %1, %2, %0" : CLASS(*o) : "v"(v), "v"(p))
  if constexpr (F16 && ACC) {
    CONVROT_MFMA_OUT("v_mfma_f32_32x32x16_f16", "+a");
  } else if constexpr (F16) {
    CONVROT_MFMA_OUT("v_mfma_f32_32x32x16_f16", "+v");
  } else if constexpr (ACC) {
    CONVROT_MFMA_OUT("v_mfma_f32_32x32x16_bf16", "+a");
  } else {
    CONVROT_MFMA_OUT("v_mfma_f32_32x32x16_bf16", "+v");
  }
#undef CONVROT_MFMA_OUT
}
template <bool F16>
__device__ __forceinline__ void mfma_first(v16f* s, const u4& k, const u4& q, const v16f& below) {
  if constexpr (F16)
    asm volatile("v_mfma_f32_32x32x16_f16 %0, %1, %2, %3"
                 : "=&v"(*s) : "v"(k), "v"(q), "v"(below));
  else
    asm volatile("v_mfma_f32_32x32x16_bf16 %0, %1, %2, %3"
                 : "=&v"(*s) : "v"(k), "v"(q), "v"(below));
}
template <bool F16>
__device__ __forceinline__ void mfma_score(v16f* s, const u4& k, const u4& q) {
  if constexpr (F16)
    asm volatile("v_mfma_f32_32x32x16_f16 %0, %1, %2, %0" : "+v"(*s) : "v"(k), "v"(q));
  else
    asm volatile("v_mfma_f32_32x32x16_bf16 %0, %1, %2, %0" : "+v"(*s) : "v"(k), "v"(q));
}
// Before a vector instruction reads what such an MFMA wrote, or the other way round.
template <int N>
__device__ __forceinline__ void settle_acc(v16f (&o)[N]) {
  asm volatile("s_nop 15\n\ts_nop 3" : "+a"(o[0]));
#pragma unroll
  for (int i = 1; i < N; ++i) asm volatile("" : "+a"(o[i]));
}
template <int N>
__device__ __forceinline__ void settle_vec(v16f (&s)[N]) {
  asm volatile("s_nop 15\n\ts_nop 3" : "+v"(s[0]));
#pragma unroll
  for (int i = 1; i < N; ++i) asm volatile("" : "+v"(s[i]));
}

// ---- many rows: 64 a wave, one wave a SIMD -----------------------------------
//
// A pipeline over units of 32 keys: a step computes the scores of unit u + 1, the
// weights of unit u and the output of unit u - 1, one MFMA after the other with a few
// vector instructions and an LDS read (three operands ahead) behind each. An operand
// read serves both of a wave's 32-row halves.
//
// Heads of 65 to 128 elements: 256 rows a block, one wave a SIMD with the output in
// accumulation registers. 32760 x 32760 x 40 heads of 128 take 18.1 to 18.9 ms, 1.16 to 1.21
// PFLOP/s, bound by power: the clock falls to 1.86 GHz with the MFMAs busy 0.58 of the
// cycles, and on zeros the same instructions reach 1.51 PFLOP/s. 4.9 vector instructions
// a score; no bank conflicts. Eight waves of 32 rows take twice the LDS reads: 1.53
// PFLOP/s on zeros, 1.14 on random values (this: 1.21 then). Causal, 16384 x 16384 x 16
// heads: 0.93 to 0.96 ms (1.15 to 1.19 PFLOP/s of the scores that count).
//
// Heads of up to 64: 128 rows a block, 32 a wave, the output beside the scores, three waves
// a SIMD; half the products a score, so bound by vector instructions and their latency.
// 16384 x 16384 x 16 heads of 64: 1.12 to 1.17 ms (0.94 to 0.98 PFLOP/s), the kernel above
// 1.18 where this takes 1.12. At 5060 x 5060 x 32 heads, causal, vector instructions issue in
// 0.79 of the busy cycles (the MFMAs 0.47) and the compute units are busy 0.78 of the time.
template <int DP, int QT, int NW>
struct Wide {
  static constexpr int kWaves = NW;
  static constexpr bool kAcc = DP * QT > 64;  // where vector registers do not hold the output
  static constexpr int kRows = 32 * QT * kWaves;
  static constexpr int kRowBytes = DP * 2;
  static constexpr int kChunks = DP / 8;
  static constexpr int kTileBytes = kTileKeys * kRowBytes;
  static constexpr int kUnitBytes = 32 * kRowBytes;
  static constexpr int kStages = 3;
  static constexpr int kV = kStages * kTileBytes;  // values behind the keys
  static constexpr int kLds = 2 * kStages * kTileBytes + 16;
  static constexpr int kCopies = kTileBytes / 1024 / kWaves;
  static constexpr int kSteps = DP / 16;
  static constexpr int kDTiles = DP / 32;
};

template <int DP, int QT, int NW, bool F16, bool CAUSAL>
__global__ __launch_bounds__(64 * NW, DP == 64 ? 3 : 1) void attention_wide_kernel(TileCall call) {
  const AttentionArgs& a = call.a;
  using T = Wide<DP, QT, NW>;
  constexpr int kFrags = 2 * T::kSteps, kSlots = kFrags * QT, kAhead = 3, kRing = 4;
  constexpr int kElems = 16 * QT;  // of a lane and unit
  extern __shared__ __align__(1024) uint8_t lds[];
  lds_ints flags = (lds_ints)(lds + 2 * T::kStages * T::kTileBytes);
  if (threadIdx.x == 0) flags[0] = flags[1] = flags[2] = 0;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int half = lane >> 5, col = lane & 31;
  Tile w;
  if (!locate<T::kRows, CAUSAL>(call, blockIdx.x, &w)) return;

  const int8_t* kbase = head_bytes(a.k, w.w, a.k_stride, a.k_head_stride, w.hk);
  const int8_t* vbase = head_bytes(a.v, w.w, a.v_stride, a.v_head_stride, w.hk);
  const uint32_t kstride = (uint32_t)a.k_stride * 2, vstride = (uint32_t)a.v_stride * 2;
  auto copy = [&](const int8_t* base, uint32_t stride, bool values, int t,
                  int to) __attribute__((always_inline)) {
    const int last = w.w.lk - 1 - t * kTileKeys;  // rows behind it repeat it
    const int8_t* p = base + (int64_t)t * kTileKeys * stride;
#pragma unroll
    for (int i = 0; i < T::kCopies; ++i) {
      const int at = (wave * T::kCopies + i) * 64;
      const int r = (at + lane) / T::kChunks, c = (at + lane) % T::kChunks;
      const int from = values ? v_slot<DP>(r, c) : k_slot<DP>(r, c);
      dma16(p, min(r, last) * stride + min(from, a.d / 8 - 1) * 16, to + at * 16);
    }
  };
  auto copy_k = [&](int t, int stage) __attribute__((always_inline)) {
    if (t < w.tiles) copy(kbase, kstride, false, t, stage * T::kTileBytes);
  };
  auto copy_v = [&](int t, int stage) __attribute__((always_inline)) {
    if (t < w.tiles) copy(vbase, vstride, true, t, T::kV + stage * T::kTileBytes);
  };
  const float c = a.scale * kLog2e;
  const float room = kRoom<F16> / c;
  copy_k(w.t0, 0);
  copy_v(w.t0, 0);
  copy_k(w.t0 + 1, 1);

  int seen[QT];
  u4 qf[QT][T::kSteps];
  const int row0 = w.row0 + wave * QT * 32;
#pragma unroll
  for (int q = 0; q < QT; ++q)
    load_query<T::kSteps, CAUSAL>(a, w.w, w.hk, row0 + q * 32 + col, qf[q], &seen[q]);
  v16f o[QT][T::kDTiles], below[QT], sa[QT], sb[QT];
  u4 pa[QT][2], pb[QT][2];
  float l[QT], raise_at[QT], top[QT];
#pragma unroll
  for (int q = 0; q < QT; ++q) {
    below[q] = (v16f){0};
    raise_at[q] = no_reference<false>(c);
    l[q] = 0.f;
#pragma unroll
    for (int d = 0; d < T::kDTiles; ++d) o[q][d] = (v16f){0};
  }

  // lane's addresses of a unit's operands
  const uint8_t* kat[T::kSteps];
#pragma unroll
  for (int st = 0; st < T::kSteps; ++st)
    kat[st] = lds + col * T::kRowBytes + k_slot<DP>(col, 2 * st + half) * 16;
  const uint8_t* vat[T::kDTiles];
#pragma unroll
  for (int d = 0; d < T::kDTiles; ++d) {
    const int r = half * 4 + ((lane & 15) >> 2);
    const int chunk = d * 4 + ((lane >> 4) & 1) * 2 + ((lane & 3) >> 1);
    vat[d] = lds + T::kV + r * T::kRowBytes + v_slot<DP>(r, chunk) * 16 + (lane & 1) * 8;
  }
  auto read_k = [&](int st, int at) __attribute__((always_inline)) {
    return *reinterpret_cast<const u4*>(kat[st] + at);
  };
  auto read_v = [&](int h, int d, int at) __attribute__((always_inline)) {
    typedef __attribute__((address_space(3))) s4* lp;
    uint8_t* p = const_cast<uint8_t*>(vat[d]) + at + h * 16 * T::kRowBytes;
    const u2 w0 = __builtin_bit_cast(u2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lp)p));
    const u2 w1 = __builtin_bit_cast(
        u2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lp)(p + 8 * T::kRowBytes)));
    return (u4){w0.x, w0.y, w1.x, w1.y};
  };

  u4 ring[kRing];
  // One step. k_at: unit u + 1's keys, v_at: unit u - 1's values, next_at: unit u + 2's
  // keys, all as offsets of LDS. cur: scores, then weights of u; nxt: scores of u + 1.
  auto step = [&](auto pv, v16f(&cur)[QT], v16f(&nxt)[QT], u4(&pin)[QT][2], u4(&pout)[QT][2],
                  int k_at, int v_at, int next_at) __attribute__((always_inline)) {
    constexpr bool kPv = decltype(pv)::value;
    // operand n of this step, or of the next
    auto fetch = [&](auto nn) __attribute__((always_inline)) {
      constexpr int n = decltype(nn)::value;
      if constexpr (n < T::kSteps) {
        ring[n % kRing] = read_k(n, k_at);
      } else if constexpr (n < kFrags) {
        constexpr int i = n - T::kSteps;
        if constexpr (kPv) ring[n % kRing] = read_v(i / T::kDTiles, i % T::kDTiles, v_at);
      } else {
        ring[n % kRing] = read_k(n - kFrags, next_at);
      }
    };
    auto weight = [&](int n) __attribute__((always_inline)) {  // element n: 2^(c s)
      const int q = n / 16, i = n % 16;
      cur[q][i] = __builtin_amdgcn_exp2f(F16 ? __builtin_fmaf(cur[q][i], c, kLift<F16>)
                                             : cur[q][i] * c);
      asm volatile("" : "+v"(cur[q][i]));
    };
    auto gather = [&](int n) __attribute__((always_inline)) {
      const int q = n / 16, i = n % 16;
      l[q] += cur[q][i];
      asm volatile("" : "+v"(l[q]));
      if (i & 1) {
        uint32_t x = pack16x2<F16>(cur[q][i - 1], cur[q][i]);
        asm volatile("" : "+v"(x));
        pout[q][i / 8][i % 8 / 2] = x;
      }
    };
    static_for<kSlots>([&](auto ss) __attribute__((always_inline)) {
      constexpr int slot = decltype(ss)::value, n = slot / QT, q = slot % QT;
      if constexpr (q == 0) fetch(std::integral_constant<int, n + kAhead>{});
      if constexpr (n < T::kSteps) {
        if constexpr (n == 0)
          mfma_first<F16>(&nxt[q], ring[n % kRing], qf[q][n], below[q]);
        else
          mfma_score<F16>(&nxt[q], ring[n % kRing], qf[q][n]);
      } else if constexpr (kPv) {
        constexpr int i = n - T::kSteps, h = i / T::kDTiles, d = i % T::kDTiles;
        mfma_out<F16, T::kAcc>(&o[q][d], ring[n % kRing], pin[q][h]);
      }
      constexpr int e0 = slot * kElems / kSlots, e1 = (slot + 1) * kElems / kSlots;
      constexpr int g0 = slot == 0 ? 0 : (slot - 1) * kElems / kSlots;
      if constexpr (slot > 0) {
#pragma unroll
        for (int e = g0; e < e0; ++e) gather(e);
      }
#pragma unroll
      for (int e = e0; e < e1; ++e) weight(e);
      // the next scores are complete some slots behind their last product
      constexpr int first = QT * T::kSteps + 2, left = kSlots - first;
      if constexpr (slot >= first) {
        constexpr int m0 = (slot - first) * kElems / 2 / left,
                      m1 = (slot - first + 1) * kElems / 2 / left;
#pragma unroll
        for (int e = m0; e < m1; ++e) {
          const int q = e / 8, i = e % 8 * 2;
          if (i == 0) top[q] = -__builtin_inff();
          asm volatile("v_max3_f32 %0, %0, %1, %2"
                       : "+v"(top[q]) : "v"(nxt[q][i]), "v"(nxt[q][i + 1]));
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    });
#pragma unroll
    for (int e = (kSlots - 1) * kElems / kSlots; e < kElems; ++e) gather(e);
  };
  // Scores of a unit before they become weights: its mask, and a new m where one is passed
  auto settle = [&](v16f(&s)[QT], v16f(&before)[QT], u4(&p)[QT][2],
                    int key0) __attribute__((always_inline)) {
    if (key0 + 32 > w.full) {
#pragma unroll
      for (int q = 0; q < QT; ++q) {
        mask(&s[q], key0, seen[q]);
        top[q] = s[q][0];
#pragma unroll
        for (int i = 1; i < 16; ++i) top[q] = fmaxf(top[q], s[q][i]);
      }
    }
    bool raise = false;
#pragma unroll
    for (int q = 0; q < QT; ++q) raise |= top[q] > raise_at[q];
    if (__any(raise)) {
#pragma unroll
      for (int q = 0; q < QT; ++q) {
        if constexpr (T::kAcc)
          settle_acc(o[q]);
        else
          settle_vec(o[q]);
      }
#pragma unroll
      for (int q = 0; q < QT; ++q) {
        const float to = fmaxf(top[q], other_half(top[q]));
        const bool up = to > raise_at[q];
        const float by = up ? to : 0.f;
        // a row without an m has nothing to scale yet (or NaN, which stays)
        const float alpha =
            up && referred<false>(raise_at[q]) ? __builtin_amdgcn_exp2f(-by * c) : 1.f;
        raise_at[q] = up ? room : raise_at[q];
        l[q] *= alpha;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          below[q][i] -= by;
          s[q][i] -= by;
        }
        // weights that the second product has not had yet
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            p[q][h][e] = pack16x2<F16>(before[q][8 * h + 2 * e] * alpha,
                                       before[q][8 * h + 2 * e + 1] * alpha);
#pragma unroll
        for (int d = 0; d < T::kDTiles; ++d)
#pragma unroll
          for (int i = 0; i < 16; ++i) o[q][d][i] *= alpha;
      }
#pragma unroll
      for (int q = 0; q < QT; ++q) {
        if constexpr (T::kAcc)
          settle_acc(o[q]);
        else
          settle_vec(o[q]);
      }
      settle_vec(below);
    }
  };
  using Yes = std::true_type;
  using No = std::false_type;

  if (w.t0 < w.tiles) {
    // keys of the first tile (and of the second, its values) have landed
    wait_vmcnt<0>();
    wait_lgkm0();
    lds_barrier();
    copy_k(w.t0 + 2, 2);
    copy_v(w.t0 + 1, 1);
#pragma unroll
    for (int q = 0; q < QT; ++q) {
      sa[q] = below[q];
      sb[q] = (v16f){0};
#pragma unroll
      for (int h = 0; h < 2; ++h) pa[q][h] = (u4){0, 0, 0, 0};
    }
#pragma unroll
    for (int st = 0; st < T::kSteps; ++st) {
      const u4 kf = read_k(st, 0);
#pragma unroll
      for (int q = 0; q < QT; ++q) mfma_score<F16>(&sa[q], kf, qf[q][st]);
    }
    settle_vec(sa);
#pragma unroll
    for (int q = 0; q < QT; ++q) {
      top[q] = sa[q][0];
#pragma unroll
      for (int i = 1; i < 16; ++i) top[q] = fmaxf(top[q], sa[q][i]);
    }
    settle(sa, sb, pa, w.t0 * kTileKeys);
    // a tile: its first unit's scores are in sa, weights of the unit before in pb
    auto tile = [&](auto pv, auto stage, int t) __attribute__((always_inline)) {
      constexpr int st = decltype(stage)::value, before = (st + 2) % 3, after = (st + 1) % 3;
      const int key0 = t * kTileKeys;
      if (key0 + kTileKeys > w.full &&
          clear_nonfinite<F16, DP, kTileKeys>(lds + T::kV + st * T::kTileBytes))
        flags[0] = 1;
      step(pv, sa, sb, pb, pa, st * T::kTileBytes + T::kUnitBytes,
           before * T::kTileBytes + T::kUnitBytes, after * T::kTileBytes);
      settle(sb, sa, pa, key0 + 32);
      step(Yes{}, sb, sa, pa, pb, after * T::kTileBytes, st * T::kTileBytes,
           after * T::kTileBytes + T::kUnitBytes);
      if (t + 1 < w.tiles) settle(sa, sb, pb, key0 + 64);
    };
    auto turn = [&](auto stage, int t) __attribute__((always_inline)) {
      constexpr int st = decltype(stage)::value;
      wait_vmcnt<0>();
      wait_lgkm0();
      lds_barrier();
      copy_k(t + 2, (st + 2) % 3);
      copy_v(t + 1, (st + 1) % 3);
    };
    using S0 = std::integral_constant<int, 0>;
    using S1 = std::integral_constant<int, 1>;
    using S2 = std::integral_constant<int, 2>;
#pragma unroll
    for (int n = 0; n < kAhead; ++n) ring[n % kRing] = read_k(n, T::kUnitBytes);
    tile(No{}, S0{}, w.t0);
    int t = w.t0 + 1, last = 0;
    while (t < w.tiles) {
      turn(S1{}, t);
      tile(Yes{}, S1{}, t);
      last = 1;
      if (++t >= w.tiles) break;
      turn(S2{}, t);
      tile(Yes{}, S2{}, t);
      last = 2;
      if (++t >= w.tiles) break;
      turn(S0{}, t);
      tile(Yes{}, S0{}, t);
      last = 0;
      ++t;
    }
    // the last unit's output
    constexpr int kLast = 2 * T::kDTiles * QT;
    static_for<kLast>([&](auto ii) __attribute__((always_inline)) {
      constexpr int i = decltype(ii)::value, h = i / QT / T::kDTiles, d = i / QT % T::kDTiles,
                    q = i % QT;
      if constexpr (q == 0) ring[0] = read_v(h, d, last * T::kTileBytes + T::kUnitBytes);
      mfma_out<F16, T::kAcc, i == kLast - 1>(&o[q][d], ring[0], pb[q][h]);
    });
  }
  if (CAUSAL || w.full % kTileKeys) {
    wait_lgkm0();
    lds_barrier();
    if (__builtin_expect(flags[0], 0)) {
      const int to = min(w.end, w.tiles * kTileKeys);
#pragma unroll 1
      for (int key = max(w.full / kTileKeys, w.t0) * kTileKeys; key < to; ++key)
#pragma unroll
        for (int q = 0; q < QT; ++q)
          add_nonfinite<T::kDTiles, F16>(a, w.w.k0 + key, w.hk, key < seen[q], o[q]);
    }
  }
  Found found = {false, 0};
#pragma unroll
  for (int q = 0; q < QT; ++q) {
    const int row = row0 + q * 32 + (thread_anew() & 31);
    const bool sees = seen[q] > w.t0 * kTileKeys;
    const bool inexact =
        row < w.rows && is_inexact<DP>(-below[q][0] * c, l[q] + other_half(l[q]), sees, a.d);
    found.inexact |= (uint64_t)rows_where(inexact) << (32 * q);
    found.lost |=
        finish<T::kRows, T::kDTiles, F16>(a, w, row, l[q], -below[q][0], c, o[q], true, true);
  }
  finish_block<DP, QT, NW, F16, CAUSAL>(found, lds, flags);
}

// ---- few rows: single tokens against a long cache ----------------------------
//
// Up to 32 rows a tile, bound by the bytes of the keys: every wave of a block
// streams its own units of 32 keys, copied two ahead into its own part of LDS, and
// waits for no other wave until the end, where the waves' sums are joined. Weights
// go into the second product in two 16-bit parts, which costs nothing here.
//
// One token of 32 / 4 heads of 128 against 100000 keys streams at 4.5 TB/s, 32 caches of
// 4096 keys at 5.0 (a large copy: 4.9); 12 caches of 1 to 8192 used keys take 48 us, 4.8 of
// them the second launch, which joins the parts; blocks cut by the room of the caches took
// 64.
template <int DP>
struct Few {
  static constexpr int kWaves = DP == 64 ? 4 : 2;
  static constexpr int kUnit = 32;
  static constexpr int kRowBytes = DP * 2;
  static constexpr int kChunks = DP / 8;
  static constexpr int kUnitBytes = kUnit * kRowBytes;
  static constexpr int kRing = 2;
  static constexpr int kWaveBytes = 2 * kRing * kUnitBytes;  // K and V
  static constexpr int kCopies = kUnitBytes / 1024;
  static constexpr int kJoinRow = DP + 4;  // floats of a row of partial sums
  static constexpr int kLds = kWaves * kWaveBytes;
  static constexpr int kFlag = kWaves * (32 * kJoinRow + 64) * 4;  // behind the sums
  static_assert(kFlag + 8 <= kLds, "sums fit the ring");
};

// What a block does: a tile of a sequence's rows with one of the `splits` parts of its
// keys, the sequence's blocks lying `heads` apart from block `first` on. All sequences
// share a.few_blocks blocks by the keys that they use, whatever room their caches have
// (0: a block a tile). False for a block without work.
struct FewWork {
  Where w;
  int split, splits;
  uint32_t first;
};
__device__ __forceinline__ bool locate_few(const AttentionArgs& a, uint32_t at, FewWork* t) {
  const int lane = threadIdx.x & 63;
  auto tiles_of = [&](const Where& w) { return (uint32_t)(w.lq * a.group + 31) / 32; };
  auto units_of = [&](const Where& w) { return (uint32_t)(w.lk + 31) / 32; };
  // rounded up, so that there are no more parts than blocks
  const float share = 1.0001f * (float)a.k_heads / (float)max(a.few_blocks, 1);
  auto units_of_part = [&](float work) {
    return max((uint32_t)kFewUnits, (uint32_t)min(ceilf(work * share), 2147483520.0f));
  };
  auto splits_of = [](uint32_t units, uint32_t chunk) {
    return min(max((units + chunk - 1) / chunk, 1u), (uint32_t)kMaxSplits);
  };
  uint32_t chunk = INT32_MAX, before = 0;  // units of a part
  if (a.batch == 1) {  // no counting
    t->w = sequence(a, 0);
    const uint32_t tiles = tiles_of(t->w), units = units_of(t->w);
    if (a.few_blocks) chunk = units_of_part((float)tiles * (float)units);
    t->splits = (int)splits_of(units, chunk);
    t->w.tile = (int)(at / (uint32_t)t->splits);
    t->split = (int)(at % (uint32_t)t->splits);
    t->first = at - (uint32_t)t->split;
    return (uint32_t)t->w.tile < tiles;
  }
  Where w = {0, 0, 0, 0, 0};
  if (lane < a.batch) w = sequence(a, lane);
  if (a.few_blocks) {
    float work = (float)tiles_of(w) * (float)units_of(w);
    for (int b = 64 + lane; b < a.batch; b += 64) {
      const Where v = sequence(a, b);
      work += (float)tiles_of(v) * (float)units_of(v);
    }
#pragma unroll
    for (int s = 1; s < 64; s <<= 1) work += __shfl_xor(work, s);
    chunk = units_of_part(work);
  }
  for (int base = 0; base < a.batch; base += 64) {
    if (base) {
      w = {0, 0, 0, 0, 0};
      if (base + lane < a.batch) w = sequence(a, base + lane);
    }
    const uint32_t tiles = tiles_of(w), units = units_of(w);  // both below 2^27
    const uint32_t splits = splits_of(units, chunk);
    uint32_t upto = (uint32_t)min((uint64_t)tiles * splits, (uint64_t)1 << 24);
#pragma unroll
    for (int s = 1; s < 64; s <<= 1) {
      const uint32_t below = __shfl_up(upto, s);
      if (lane >= s) upto += below;
    }
    const uint64_t past = __ballot(upto > at - before);  // before <= at
    if (past) {
      const int l = __builtin_ctzll(past);
      const uint32_t begin = l ? __builtin_amdgcn_readlane(upto, l - 1) : 0;
      t->splits = __builtin_amdgcn_readlane(splits, l);
      const uint32_t local = at - before - begin;
      t->w.q0 = __builtin_amdgcn_readlane(w.q0, l);
      t->w.k0 = __builtin_amdgcn_readlane(w.k0, l);
      t->w.lq = __builtin_amdgcn_readlane(w.lq, l);
      t->w.lk = __builtin_amdgcn_readlane(w.lk, l);
      t->w.tile = (int)(local / (uint32_t)t->splits);
      t->split = (int)(local % (uint32_t)t->splits);
      t->first = at - (uint32_t)t->split;
      return true;
    }
    before += __builtin_amdgcn_readlane(upto, 63);
  }
  return false;
}

// One pass over a block's keys; the sums of its waves joined, and the rows that `only`
// names written. True if one of them has an element lost; the second flag takes the rows
// that were inexact.
template <int DP, bool F16, bool EXACT>
__device__ __forceinline__ bool few_pass(const AttentionArgs& a, const FewWork& work,
                                         uint32_t block, const Pass<F16>& pass, uint8_t* lds,
                                         int tid, uint32_t only) {
  using T = Few<DP>;
  constexpr int kSteps = DP / 16, kDTiles = DP / 32;
  const int lane = tid & 63;
  const int wave = wave_number(tid);
  const int half = lane >> 5, col = lane & 31;
  const int group = a.group, hk = (int)(block % (uint32_t)a.k_heads);
  const Where& w = work.w;

  const int rows = w.lq * group, row0 = w.tile * 32;
  const int shift = w.lk - w.lq + 1;
  int end = w.lk, full = w.lk;
  if (a.causal) {
    end = min(w.lk, max(0, min(rows - 1, row0 + 31) / group + shift));
    full = min(w.lk, max(0, row0 / group + shift));
  }
  // units of this part, dealt to the waves
  const int units = (end + T::kUnit - 1) / T::kUnit;
  const int per = (units + work.splits - 1) / work.splits;
  const int first = min(units, work.split * per), last = min(units, first + per);

  u4 qf[kSteps];
  int seen;
  if (a.causal)
    load_query<kSteps, true>(a, w, hk, row0 + col, qf, &seen);
  else
    load_query<kSteps, false>(a, w, hk, row0 + col, qf, &seen);

  const int8_t* kbase = head_bytes(a.k, w, a.k_stride, a.k_head_stride, hk);
  const int8_t* vbase = head_bytes(a.v, w, a.v_stride, a.v_head_stride, hk);
  const uint32_t kstride = (uint32_t)a.k_stride * 2, vstride = (uint32_t)a.v_stride * 2;
  const int ring = wave * T::kWaveBytes;
  auto issue = [&](int u, int stage) {
    const int top = w.lk - 1 - u * T::kUnit;  // rows behind it repeat it
    const int8_t* kp = kbase + (int64_t)u * T::kUnit * a.k_stride * 2;
    const int8_t* vp = vbase + (int64_t)u * T::kUnit * a.v_stride * 2;
    const int to = ring + stage * 2 * T::kUnitBytes;
#pragma unroll
    for (int i = 0; i < T::kCopies; ++i) {
      const int n = i * 64 + lane, from = min(n / T::kChunks, top);
      const int c = min(k_slot<DP>(n / T::kChunks, n % T::kChunks), a.d / 8 - 1);
      dma16(kp, from * kstride + c * 16, to + i * 1024);
    }
#pragma unroll
    for (int i = 0; i < T::kCopies; ++i) {
      const int n = i * 64 + lane, from = min(n / T::kChunks, top);
      const int c = min(v_slot<DP>(n / T::kChunks, n % T::kChunks), a.d / 8 - 1);
      dma16(vp, from * vstride + c * 16, to + T::kUnitBytes + i * 1024);
    }
  };

  const float c = a.scale * kLog2e;
  v16f o[kDTiles], below = (v16f){0};
#pragma unroll
  for (int d = 0; d < kDTiles; ++d) o[d] = (v16f){0};
  float l = 0.f, raise_at = no_reference<EXACT>(c);

  int u = first + wave, stage = 0;
  if (u < last) issue(u, 0);
  for (; u < last; u += T::kWaves, stage ^= 1) {
    const bool more = u + T::kWaves < last;
    wait_lgkm0();  // the other stage's last reads
    asm volatile("" ::: "memory");
    if (more) {
      issue(u + T::kWaves, stage ^ 1);
      wait_vmcnt<3 * T::kCopies>();
    } else {
      wait_vmcnt<T::kCopies>();
    }
    asm volatile("" ::: "memory");
    const uint8_t* kt = lds + ring + stage * 2 * T::kUnitBytes;
    uint8_t* vt = lds + ring + stage * 2 * T::kUnitBytes + T::kUnitBytes;
    v16f s;
    const int key0 = u * T::kUnit;
    float top;
    auto score = [&](const v16f& from) __attribute__((always_inline)) {
      s = from;
#pragma unroll
      for (int st = 0; st < kSteps; ++st) {
        const u4 kf = *reinterpret_cast<const u4*>(kt + col * T::kRowBytes +
                                                   k_slot<DP>(col, 2 * st + half) * 16);
        s = mfma<F16>(EXACT ? inside_head(kf, 2 * st + half, a.d) : kf, qf[st], s);
      }
      if (key0 + T::kUnit > full) mask(&s, key0, seen);
      top = s[0];
#pragma unroll
      for (int i = 1; i < 16; ++i) top = fmaxf(top, s[i]);
      top = fmaxf(top, other_half(top));
    };
    score(below);
    if (__any(top > raise_at)) {
      const bool up = top > raise_at;
      const float left = EXACT && up && leaves_far(below[0], top) ? below[0] : 0.f;
      if (EXACT && __any(left != 0.f)) {
#pragma unroll
        for (int i = 0; i < 16; ++i) below[i] = left != 0.f ? 0.f : below[i];
        score(below);
      }
      const float by = up ? top + pass.over : 0.f;
      const float alpha =
          up && referred<EXACT>(raise_at) ? __builtin_amdgcn_exp2f(-(by + left) * c) : 1.f;
      raise_at = up ? pass.room : raise_at;
      l *= alpha;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        below[i] -= by;
        s[i] -= by;
      }
#pragma unroll
      for (int d = 0; d < kDTiles; ++d)
#pragma unroll
        for (int i = 0; i < 16; ++i) o[d][i] *= alpha;
    }
    u4 hi[2], lo[2];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      s[i] = __builtin_amdgcn_exp2f(F16 ? __builtin_fmaf(s[i], c, kLift<F16>) : s[i] * c);
      l += s[i];
    }
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float p0 = s[8 * h + 2 * e], p1 = s[8 * h + 2 * e + 1];
        const uint32_t p = pack16x2<F16>(p0, p1);
        hi[h][e] = p;
        lo[h][e] = pack16x2<F16>(p0 - lo16<F16>(p), p1 - hi16<F16>(p));
      }
    if (more)
      wait_vmcnt<2 * T::kCopies>();
    else
      wait_vmcnt<0>();
    asm volatile("" ::: "memory");
    // in every unit: the weights' second part would turn an infinity into NaN
    const bool cleared = clear_nonfinite<F16, DP, T::kUnit>(vt);
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int d = 0; d < kDTiles; ++d) {
        const u4 vf = values<DP>(vt, h * 16, d);
        o[d] = mfma<F16>(vf, hi[h], o[d]);
        o[d] = mfma<F16>(vf, lo[h], o[d]);
      }
    if (__builtin_expect(cleared, 0)) {
      const int to = min(end, key0 + T::kUnit);
      for (int key = key0; key < to; ++key)
        add_nonfinite<kDTiles, F16>(a, w.k0 + key, hk, key < seen, o);
    }
  }

  // ---- join the waves: sums of each go to LDS, [row][element], with their m and l ----
  const float sum = l + other_half(l);
  wait_lgkm0();
  lds_barrier();
  constexpr int kPart = 32 * T::kJoinRow;
  float* part = reinterpret_cast<float*>(lds);
  float* stat = part + T::kWaves * kPart;  // [wave][m, l][32]
  lds_ints flags = (lds_ints)(lds + T::kFlag);
  if (tid == 0) flags[0] = flags[1] = 0;
#pragma unroll
  for (int d = 0; d < kDTiles; ++d)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const v4f f = {o[d][4 * i], o[d][4 * i + 1], o[d][4 * i + 2], o[d][4 * i + 3]};
      *reinterpret_cast<v4f*>(part + wave * kPart + col * T::kJoinRow + d * 32 + i * 8 +
                              half * 4) = f;
    }
  if (half == 0) {
    // a row without an m has seen nothing, or only NaN
    stat[wave * 64 + col] = referred<EXACT>(raise_at) ? -below[0] : kLowest;
    stat[wave * 64 + 32 + col] = sum;
  }
  wait_lgkm0();
  lds_barrier();
  const int here = min(32, rows - row0);
  constexpr int kQuads = DP / 4;
  bool lost = false;
  for (int i = tid; i < here * kQuads; i += 64 * T::kWaves) {
    const int jr = i / kQuads, e = i % kQuads * 4;
    if (e >= a.d || (EXACT && !(only >> jr & 1))) continue;
    float m = kLowest;
#pragma unroll
    for (int v = 0; v < T::kWaves; ++v) m = fmaxf(m, stat[v * 64 + jr]);
    float total = 0.f;
    v4f acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int v = 0; v < T::kWaves; ++v) {
      const float lv = stat[v * 64 + 32 + jr];
      if (lv == 0.f) continue;  // saw nothing
      const float f = __builtin_amdgcn_exp2f((stat[v * 64 + jr] - m) * c);
      const v4f x = *reinterpret_cast<const v4f*>(part + v * kPart + jr * T::kJoinRow + e);
      total += f * lv;
#pragma unroll
      for (int q = 0; q < 4; ++q) acc[q] = __builtin_fmaf(f, x[q], acc[q]);
    }
    if (Pass<F16>::kAgain && total < __builtin_inff()) {
#pragma unroll
      for (int q = 0; q < 4; ++q) lost |= !(__builtin_fabsf(acc[q]) < __builtin_inff());
    }
    const bool some = total > 0.f || total != total;
    const float inv = some ? 1.0f / total : 0.f;
    const float lse2 = some ? log2f(total) - kLift<F16> + m * c : -__builtin_inff();
    const int jtoken = (row0 + jr) / group, jhead = hk * group + (row0 + jr) % group;
    if (!EXACT) {
      const bool sees = (a.causal ? min(w.lk, jtoken + shift) : w.lk) > first * T::kUnit;
      if (__builtin_expect(is_inexact<DP>(total == 0.f ? 0.f : m * c, total, sees, a.d), 0))
        atomicOr(reinterpret_cast<int*>(lds + T::kFlag) + 1, 1 << jr);
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) acc[q] *= inv;
    if (a.splits > 1 && e == 0 && work.split == 0) {
      // where the row's parts are; none to join where the row has one
      int2* map = reinterpret_cast<int2*>(a.part_map);
      map[(int64_t)(w.q0 + jtoken) * a.q_heads + jhead] =
          make_int2((int)(work.first * (uint32_t)a.k_heads + (uint32_t)hk) * a.part_step + jr,
                    work.splits > 1 ? work.splits : 0);
    }
    if (work.splits > 1) {
      const int64_t at = (int64_t)block * a.part_step + jr;
      if (e == 0 && pass.first()) a.part_lse[at] = lse2;
      v4f* to = reinterpret_cast<v4f*>(a.part + at * a.d + e);
      if (some) *to = pass.first() ? acc : finite_of(*to, acc);
      continue;
    }
    if (a.lse && e == 0 && pass.first())
      a.lse[(int64_t)jhead * a.q_tokens + w.q0 + jtoken] = lse2 * kLn2;
    const u2 f = {pack16x2<F16>(acc[0], acc[1]), pack16x2<F16>(acc[2], acc[3])};
    u2* to = reinterpret_cast<u2*>(a.out + (int64_t)(w.q0 + jtoken) * a.out_stride +
                                   (int64_t)jhead * a.out_head_stride + e);
    *to = pass.first() ? f : finite_of16<F16>(*to, f);
  }
  return lost;
}

// What a block goes over again, as walk_anew.
template <int DP, bool F16>
__device__ __forceinline__ void few_anew(uint32_t rows, uint8_t* lds, lds_ints flags) {
  const AttentionArgs a = call_anew<AttentionArgs>();
  const uint32_t block = block_anew();
  FewWork work;
  if (!locate_few(a, block / (uint32_t)a.k_heads, &work)) return;
  const float c = a.scale * kLog2e;
  Pass<F16> pass(c);
  bool more = flags[0];
  bool exact = rows != 0;
  do {
    lds_barrier();  // all have read the flags: the ring takes their place
    if (!exact) pass.again(c);
    const bool lost = few_pass<DP, F16, true>(a, work, block, pass, lds, thread_anew(),
                                              exact ? rows : ~0u);
    if (!Pass<F16>::kAgain || !exact) return;
    exact = false;
    note(lost, flags);
    all_noted();
    more |= flags[0] != 0;
  } while (more);
}

template <int DP, bool F16>
__global__ __launch_bounds__(64 * Few<DP>::kWaves, 1) void attention_few_kernel(AttentionArgs a) {
  extern __shared__ __align__(1024) uint8_t lds[];
  FewWork work;
  if (!locate_few(a, blockIdx.x / (uint32_t)a.k_heads, &work)) return;
  const bool lost = few_pass<DP, F16, false>(
      a, work, blockIdx.x, Pass<F16>(a.scale * kLog2e), lds, threadIdx.x, ~0u);
  lds_ints flags = (lds_ints)(lds + Few<DP>::kFlag);
  note(lost, flags);
  all_noted();
  const uint32_t inexact = flags[1];
  if (__builtin_expect((inexact | flags[0]) != 0, 0)) few_anew<DP, F16>(inexact, lds, flags);
}

// Joins the splits of a row: out = sum_s 2^(lse_s - lse) out_s, with a power of two out of
// the factors, so that their sum is below 1 and that of the parts in fp32's range. A block
// takes a row: a thread a split's factor, then groups of lanes, four elements each, the
// splits in turn, all of whose loads are under way together.
constexpr int kJoinThreads = 256;
constexpr float kJoinScale = 1024.f;
static_assert(kMaxSplits < kJoinScale, "the factors' sum");

template <bool F16>
__global__ __launch_bounds__(kJoinThreads) void attention_join_kernel(AttentionArgs a, int lanes) {
  __shared__ float factor[kMaxSplits];
  __shared__ float red[2][kJoinThreads / 64];
  __shared__ __align__(16) float acc[kJoinThreads * 4];
  // few rows: a block a row of the output, which knows its parts; tiles: a block a row of
  // a tile, which knows its row of the output
  int64_t r = blockIdx.x, at, step;
  int splits = a.splits;
  if (a.tile == 32) {
    const int token = (int)(r / a.q_heads);
    if (a.q_offsets && (token < a.q_offsets[0] || token >= a.q_offsets[a.batch])) return;
    const int2 map = reinterpret_cast<const int2*>(a.part_map)[r];
    at = map.x;
    splits = map.y;
    step = (int64_t)a.k_heads * a.part_step;
    // rows that offsets which decrease leave out have no entry: nothing outside is read
    if (splits < 2 || splits > kMaxSplits || at < 0 || at + (splits - 1) * step >= a.parts) return;
  } else {
    step = a.part_step;
    at = r / step * step * splits + r % step;
    r = a.part_map[r];
    if (r < 0) return;
  }
  const int64_t token = r / a.q_heads;
  const int head = (int)(r % a.q_heads);
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int group = tid / lanes, groups = kJoinThreads / lanes, e = tid % lanes * 4;

  float x[kMaxSplits / kJoinThreads];
  float top = kLowest;
#pragma unroll
  for (int i = 0; i < kMaxSplits / kJoinThreads; ++i) {
    const int s = tid + i * kJoinThreads;
    x[i] = s < splits ? a.part_lse[at + s * step] : -__builtin_inff();
    top = fmaxf(top, x[i]);
  }
#pragma unroll
  for (int s = 1; s < 64; s <<= 1) top = fmaxf(top, __shfl_xor(top, s));
  if (lane == 0) red[0][wave] = top;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kJoinThreads / 64; ++i) top = fmaxf(top, red[0][i]);
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < kMaxSplits / kJoinThreads; ++i) {
    const float f = __builtin_amdgcn_exp2f(x[i] - top);  // 0 for a split that saw nothing
    if (tid + i * kJoinThreads < splits) factor[tid + i * kJoinThreads] = f * (1 / kJoinScale);
    sum += f;
  }
#pragma unroll
  for (int s = 1; s < 64; s <<= 1) sum += __shfl_xor(sum, s);
  if (lane == 0) red[1][wave] = sum;
  __syncthreads();
  sum = 0.f;
#pragma unroll
  for (int i = 0; i < kJoinThreads / 64; ++i) sum += red[1][i];

  v4f v = {0.f, 0.f, 0.f, 0.f};
  if (e < a.d) {
    const float* from = a.part + at * a.d + e;
#pragma unroll 8
    for (int s = group; s < splits; s += groups) {
      const float f = factor[s];
      const v4f p = *reinterpret_cast<const v4f*>(from + s * step * a.d);
#pragma unroll
      for (int q = 0; q < 4; ++q)  // what a split that saw nothing holds is not its result
        v[q] = f != 0.f ? __builtin_fmaf(f, p[q], v[q]) : v[q];
    }
  }
  *reinterpret_cast<v4f*>(acc + tid * 4) = v;
  __syncthreads();
  const bool none = sum == 0.f;
  if (a.lse && tid == 0)
    a.lse[head * a.q_tokens + token] = none ? -__builtin_inff() : (top + log2f(sum)) * kLn2;
  if (group == 0 && e < a.d) {
    for (int g = 1; g < groups; ++g) {
      const v4f p = *reinterpret_cast<const v4f*>(acc + (g * lanes) * 4 + e);
#pragma unroll
      for (int q = 0; q < 4; ++q) v[q] += p[q];
    }
    const float inv = none ? 0.f : 1.0f / sum * kJoinScale;
    const u2 f = {pack16x2<F16>(v[0] * inv, v[1] * inv), pack16x2<F16>(v[2] * inv, v[3] * inv)};
    *reinterpret_cast<u2*>(a.out + token * a.out_stride + (int64_t)head * a.out_head_stride + e) =
        f;
  }
}

// The same for the rows of split tiles, of few parts each: `lanes` lanes a row, every
// lane working out the factors.
constexpr int kJoinFew = 12;  // parts; a block a row beyond (31 parts: 4.6 us, so 9.5)

template <bool F16>
__global__ __launch_bounds__(kJoinThreads) void attention_join_rows_kernel(AttentionArgs a,
                                                                           int lanes,
                                                                           uint32_t rows) {
  const uint32_t of_tile =
      blockIdx.x * (uint32_t)(kJoinThreads / lanes) + threadIdx.x / (uint32_t)lanes;
  const int e = (int)(threadIdx.x % (uint32_t)lanes) * 4;
  if (of_tile >= rows) return;
  const int64_t r = a.part_map[of_tile];
  if (r < 0) return;
  const uint32_t step = (uint32_t)a.part_step, splits = (uint32_t)a.splits;
  const int64_t at = (int64_t)(of_tile / step) * step * splits + of_tile % step;
  const float* lse = a.part_lse + at;
  float top = kLowest;
#pragma unroll 4
  for (uint32_t s = 0; s < splits; ++s) top = fmaxf(top, lse[s * step]);
  const float* from = a.part + at * a.d + e;
  float sum = 0.f;
  v4f v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
  for (uint32_t s = 0; s < splits; ++s) {
    const float f = __builtin_amdgcn_exp2f(lse[s * step] - top);
    v4f p = {0.f, 0.f, 0.f, 0.f};
    if (e < a.d) p = *reinterpret_cast<const v4f*>(from + (int64_t)(s * step) * a.d);
    sum += f;
#pragma unroll
    for (int q = 0; q < 4; ++q)  // what a split that saw nothing holds is not its result
      v[q] = f != 0.f ? __builtin_fmaf(f * (1 / kJoinScale), p[q], v[q]) : v[q];
  }
  const bool none = sum == 0.f;
  const int64_t token = r / a.q_heads;
  const int head = (int)(r % a.q_heads);
  if (a.lse && e == 0)
    a.lse[head * a.q_tokens + token] = none ? -__builtin_inff() : (top + log2f(sum)) * kLn2;
  if (e < a.d) {
    const float inv = none ? 0.f : 1.0f / sum * kJoinScale;
    const u2 f = {pack16x2<F16>(v[0] * inv, v[1] * inv), pack16x2<F16>(v[2] * inv, v[3] * inv)};
    *reinterpret_cast<u2*>(a.out + token * a.out_stride + (int64_t)head * a.out_head_stride + e) =
        f;
  }
}

template <typename K>
hipError_t launch_tiles(K kern, int threads, int lds, const AttentionArgs& a,
                        const AttentionPlan& p, hipStream_t st) {
  if (lds > 65536) {
    // per device: the attribute is set on every call (a host-side table write)
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kern),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, lds);
    if (e != hipSuccess) return e;
  }
  const uint32_t xcds = (uint32_t)xcd_count(compute_units());
  uint32_t common = xcds;  // greatest common divisor with the heads
  for (uint32_t y = (uint32_t)a.k_heads; y;) {
    const uint32_t r = common % y;
    common = y;
    y = r;
  }
  const uint32_t share = xcds / common;
  int64_t grid = p.grid;
  if (a.causal && p.splits == 1) {
    const int64_t of_group = p.slots * (a.k_heads / (int)common);
    grid = (of_group + share - 1) / share * xcds;
  }
  const TileCall call = {a, (uint32_t)p.slots, xcds, share};
  kern<<<dim3((uint32_t)grid), dim3(threads), lds, st>>>(call);
  return hipGetLastError();
}

template <int DP, int NW, bool F16>
hipError_t launch_tile(const AttentionArgs& a, const AttentionPlan& p, hipStream_t st) {
  return launch_tiles(a.causal ? attention_kernel<DP, NW, F16, true>
                               : attention_kernel<DP, NW, F16, false>,
                      64 * NW, Kernel<DP, NW>::kLds, a, p, st);
}

template <int DP, int QT, int NW, bool F16>
hipError_t launch_wide(const AttentionArgs& a, const AttentionPlan& p, hipStream_t st) {
  return launch_tiles(a.causal ? attention_wide_kernel<DP, QT, NW, F16, true>
                               : attention_wide_kernel<DP, QT, NW, F16, false>,
                      64 * NW, Wide<DP, QT, NW>::kLds, a, p, st);
}

template <int DP, bool F16>
hipError_t launch_few(const AttentionArgs& a, const AttentionPlan& p, hipStream_t st) {
  using T = Few<DP>;
  auto kern = attention_few_kernel<DP, F16>;
  if (T::kLds > 65536) {
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kern),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, T::kLds);
    if (e != hipSuccess) return e;
  }
  kern<<<dim3((uint32_t)p.grid), dim3(64 * T::kWaves), T::kLds, st>>>(a);
  return hipGetLastError();
}

template <bool F16>
hipError_t launch_dtype(const AttentionArgs& a, const AttentionPlan& p, hipStream_t st) {
  hipError_t e;
  if (p.rows == 32)
    e = a.d <= 64    ? launch_few<64, F16>(a, p, st)
        : a.d <= 128 ? launch_few<128, F16>(a, p, st)
                     : launch_few<256, F16>(a, p, st);
  else if (p.rows == kRowsOfWide)
    e = launch_wide<128, 2, 4, F16>(a, p, st);
  else if (a.d <= 64)
    e = launch_wide<64, 1, 4, F16>(a, p, st);
  else if (a.d <= 128)
    e = launch_tile<128, 4, F16>(a, p, st);
  else
    e = launch_tile<256, 4, F16>(a, p, st);
  if (e != hipSuccess || a.splits == 1) return e;
  int lanes = 1;
  while (lanes * 4 < a.d) lanes *= 2;
  if (p.rows != 32 && p.splits <= kJoinFew) {
    const int64_t per = kJoinThreads / lanes;
    attention_join_rows_kernel<F16>
        <<<dim3((uint32_t)((p.part_rows + per - 1) / per)), dim3(kJoinThreads), 0, st>>>(
            a, lanes, (uint32_t)p.part_rows);
  } else {
    attention_join_kernel<F16>
        <<<dim3((uint32_t)p.part_rows), dim3(kJoinThreads), 0, st>>>(a, lanes);
  }
  return hipGetLastError();
}

size_t workspace_bytes(const AttentionPlan& p, int d) {
  if (p.splits <= 1) return 0;
  if (p.rows == 32)  // parts by block, places by row of the output
    return (size_t)p.grid * p.part_step * (d + 1) * 4 + (size_t)p.part_rows * 8 + 8;
  return (size_t)p.part_rows * ((size_t)p.splits * (d + 1) * 4 + 8);
}

// A kernel's blocks on a full card (256 compute units; a constant, as the split decides
// the order of sums): `room` at a time, a round of which takes `tile` us per key tile and
// `start` us beside. Fitted to 16384 queries x 40 heads of 128 over 256 to 4608 keys
// (10 rounds; measured 143 to 1410 us with 128 rows a block, 180 to 1333 us with 256),
// 48 heads of 64 and 16 of 256 alike.
// In a round of at most half its blocks, those of a kernel that runs two a compute unit
// have one to themselves and take 0.62 of the time.
struct Rounds {
  int rows;
  int64_t room;
  double tile, start, half;
};
constexpr Rounds kRounds64 = {kRowsOfTile, kMaxSplits * 3 / 2, 1.59, 4.3, 0.62};
constexpr Rounds kRounds128 = {kRowsOfTile, kMaxSplits, 1.93, 6.5, 0.62};
constexpr Rounds kRoundsWide = {kRowsOfWide, kMaxSplits / 2, 1.70, 10.6, 1.0};
constexpr Rounds kRounds256 = {kRowsOfTile, kMaxSplits / 2, 2.56, 7.8, 1.0};

// The plan of least estimated time with this kernel; *cost is that time.
AttentionPlan plan_tiles(const AttentionArgs& a, const Rounds& k, size_t workspace,
                         double* cost) {
  AttentionPlan p;
  const int64_t group = a.q_heads / a.k_heads;
  const int64_t rows = a.q_tokens * group, each = a.q_tokens / a.batch;
  p.rows = p.part_step = k.rows;
  int64_t tiles = 0;  // that there are, as far as is known here
  if (a.batch == 1 || !a.q_offsets) {
    p.slots = a.batch * ((each * group + k.rows - 1) / k.rows);
    tiles = p.slots * a.k_heads;
  } else {
    p.slots = (rows + k.rows - 1) / k.rows + a.batch;
    tiles = (rows / k.rows + (a.batch + 1) / 2) * a.k_heads;
  }
  const int64_t blocks = p.slots * a.k_heads;
  p.whole = blocks;
  p.grid = blocks;
  const double keys = (double)(a.k_tokens / a.batch) / kTileKeys;
  // key tiles of a row tile: causal ones differ, come longest first and even out
  double mean = keys;
  if (a.causal) mean = keys > (double)each / 64 ? keys - (double)each / 128 : keys / 2;
  *cost = 1e30;
  // n parts of each of the last `rest` tiles
  auto consider = [&](int64_t whole, int64_t rest, int64_t n) {
    if (n > 1 && n > keys / 4) n = (int64_t)(keys / 4);
    if (n > kMaxSplits) n = kMaxSplits;  // whose factors the join holds
    if (n < 1) return;
    AttentionPlan t = p;
    if (n > 1) {
      t.whole = whole;
      t.splits = (int)n;
      t.part_rows = (blocks - whole) * k.rows;
      t.grid = whole + (blocks - whole) * n;
    }
    const size_t bytes = workspace_bytes(t, a.d);
    if (bytes > workspace) return;
    const int64_t all = rest * n, full = all / k.room, last = all % k.room;
    double rounds = (double)full + (last == 0 ? 0 : 2 * last <= k.room ? k.half : 1.0);
    if (a.causal && full > 0) rounds = (double)all / k.room;
    double us = rounds * (mean / n * k.tile + k.start);
    // the longest block
    if (a.causal && us < keys / n * k.tile * k.half) us = keys / n * k.tile * k.half;
    us += (double)(whole / k.room) * (mean * k.tile + k.start);
    if (n > 1) us += 4 + (double)bytes / 5e6;  // the join: 33 MB 7.4 us, 67 MB 13.2
    if (us < *cost) {
      *cost = us;
      p = t;
    }
  };
  consider(0, tiles, 1);
  if (tiles < k.room) {
    for (int64_t n = 2; n <= 8; ++n) consider(0, tiles, n);
    for (int64_t of = k.room / 2; of <= 2 * k.room; of *= 2)
      if (tiles) consider(0, tiles, of / tiles);
  } else if (!a.causal && tiles == blocks && tiles % k.room) {
    const int64_t rest = tiles % k.room;
    for (int64_t n = 2; n <= 8; ++n) consider(tiles - rest, rest, n);
    for (int64_t of = k.room / 2; of <= 2 * k.room; of *= 2)
      consider(tiles - rest, rest, of / rest);
  }
  return p;
}

AttentionPlan plan_few(const AttentionArgs& a, size_t workspace) {
  AttentionPlan p;
  const int64_t group = a.q_heads / a.k_heads, each = a.q_tokens / a.batch;
  const int64_t rows = a.q_tokens * group;
  p.rows = 32;
  p.slots = a.batch * ((each * group + 31) / 32);
  int64_t longest = a.k_tokens / a.batch, part = each * group;
  if (a.batch > 1 && a.q_offsets) {
    p.slots = (rows + 31) / 32 + a.batch;
    part = rows;
  }
  if (a.batch > 1 && a.k_offsets) longest = a.k_tokens;
  p.part_step = part < 32 ? (int)part : 32;
  p.part_rows = a.q_tokens * a.q_heads;
  // a round of two blocks a compute unit (heads of 256: one), less about half a block a tile
  const int64_t room = a.d > 128 ? kMaxSplits / 2 : kMaxSplits, tiles = p.slots * a.k_heads;
  p.few_blocks = (int)(tiles < room ? room - tiles / 2 : room / 2);
  // nothing to share out: short keys, blocks enough, or too many sequences to read
  p.splits = longest > kFewUnits * 32 && tiles < 2 * room && a.batch <= 1024 ? kMaxSplits : 1;
  p.grid = tiles + p.few_blocks;
  const size_t bytes = workspace_bytes(p, a.d);
  if (p.splits > 1 && bytes > workspace) {  // as many blocks as it holds
    const size_t over = (bytes - workspace + (size_t)p.part_step * (a.d + 1) * 4 - 1) /
                        ((size_t)p.part_step * (a.d + 1) * 4);
    if (over >= (size_t)p.few_blocks) {
      p.splits = 1;
    } else {
      p.few_blocks -= (int)over;
      p.grid -= (int64_t)over;
    }
  }
  if (p.splits == 1) {
    p.few_blocks = 0;
    p.part_rows = 0;
    p.grid = tiles;
  }
  return p;
}

}  // namespace

AttentionPlan plan_attention(const AttentionArgs& a, size_t workspace) {
  const int64_t rows = a.q_tokens * (a.q_heads / a.k_heads);
  if (a.tile == 32 || (a.tile == 0 && rows <= 32 * (int64_t)a.batch))
    return plan_few(a, workspace);
  double cost, wide;
  if (a.d <= 64) return plan_tiles(a, kRounds64, workspace, &cost);
  if (a.d > 128) return plan_tiles(a, kRounds256, workspace, &cost);
  const AttentionPlan p = plan_tiles(a, kRounds128, workspace, &cost);
  const AttentionPlan w = plan_tiles(a, kRoundsWide, workspace, &wide);
  return a.tile ? (a.tile == kRowsOfWide ? w : p) : wide < cost ? w : p;
}

size_t attention_workspace(const AttentionArgs& a, const AttentionPlan& p) {
  return workspace_bytes(p, a.d);
}

void attention_use(AttentionArgs* a, const AttentionPlan& p, void* workspace) {
  a->group = a->q_heads / a->k_heads;
  a->q_each = (int)(a->q_tokens / a->batch);
  a->k_each = (int)(a->k_tokens / a->batch);
  a->splits = p.splits;
  a->whole = (uint32_t)p.whole;
  a->part_step = p.part_step;
  a->few_blocks = p.few_blocks;
  a->tile = p.rows;
  a->parts = p.grid * p.part_step;
  if (p.splits == 1) return;
  char* at = static_cast<char*>(workspace);
  a->part_map = reinterpret_cast<int64_t*>(at);
  at += (p.part_rows * 8 + 15) / 16 * 16;
  a->part = reinterpret_cast<float*>(at);
  const int64_t parts = p.rows == 32 ? a->parts : p.splits * p.part_rows;
  a->part_lse = a->part + (size_t)parts * a->d;
}

hipError_t launch_attention(const AttentionArgs& a, const AttentionPlan& p, DType dt,
                            hipStream_t st) {
  if (p.grid == 0) return hipSuccess;
  return dt == DType::kF16 ? launch_dtype<true>(a, p, st) : launch_dtype<false>(a, p, st);
}

}  // namespace convrot
