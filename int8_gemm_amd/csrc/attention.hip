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

#include "attention.h"
#include "lds_copy.h"

namespace convrot {

namespace {

typedef __bf16 bf8 __attribute__((ext_vector_type(8)));
typedef _Float16 hf8 __attribute__((ext_vector_type(8)));
typedef float v16f __attribute__((ext_vector_type(16)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef short s4 __attribute__((ext_vector_type(4)));

constexpr int kTileKeys = 64;   // keys of a copied tile
constexpr int kRowsOfTile = 128;
constexpr int kMaxSplits = 512;  // two rounds of a block per compute unit
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;
// A row's reference m is a largest score of it: it is raised when a score passes it by
// kRoom / c, so weights stay below 2^(kRoom + kLift). Half weights are lifted so that
// those of 2^-20 of the largest are normal numbers; the sum is lifted with them.
constexpr float kRoom = 8.f;
template <bool F16>
constexpr float kLift = F16 ? 6.f : 0.f;
constexpr float kLowest = -3.402823466e38f;

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

template <int DP, int QT, int NW, bool F16>
struct Kernel {
  static constexpr int kRows = 32 * QT * NW;         // rows of a block
  static constexpr int kRowBytes = DP * 2;
  static constexpr int kChunks = DP / 8;
  static constexpr int kTileBytes = kTileKeys * kRowBytes;
  static constexpr int kStages = 2;
  static constexpr int kLds = 2 * kStages * kTileBytes + 16;  // and a flag
  static constexpr int kCopies = kTileBytes / 1024 / NW;  // of a wave, per tile and operand
  static constexpr int kSteps = DP / 16;
  static constexpr int kDTiles = DP / 32;
};

// Values of keys that only some rows of a tile see. A weight of 0 does not cancel an
// infinity or a NaN in the product, so a tile in which some row's mask ends is looked
// through, infinities and NaN in it are replaced by 0 (by every wave that finds one,
// before its own reads; they all write the same), and at the end each row adds
// those of the keys that it sees.
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
  const int lane = threadIdx.x & 63;
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

template <int DP, int QT, int NW, bool F16, bool CAUSAL>
__global__ __launch_bounds__(64 * NW, DP > 128 ? 1 : 2) void attention_kernel(AttentionArgs a, uint32_t slots,
                                                               uint32_t xcds) {
  using T = Kernel<DP, QT, NW, F16>;
  extern __shared__ __align__(1024) uint8_t lds[];
  volatile int* cleared = reinterpret_cast<int*>(lds + 2 * T::kStages * T::kTileBytes);
  if (CAUSAL && threadIdx.x == 0) *cleared = 0;  // a barrier follows in every tile
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int half = lane >> 5, col = lane & 31;
  const int group = a.group;

  // blocks of an XCD (they are dealt in turn) take neighbouring tiles of the same
  // heads, whose keys then meet in its L2
  // the first a.whole tiles are a block's each, the last ones are split
  const bool tail = blockIdx.x >= a.whole;
  uint32_t id = tail ? blockIdx.x - a.whole : blockIdx.x;
  {
    const uint32_t total = tail ? gridDim.x - a.whole : a.whole;
    const uint32_t full = total / xcds, rest = total % xcds;
    const uint32_t x = id % xcds, i = id / xcds;
    id = x * full + min(x, rest) + i;
  }
  const int splits = tail ? a.splits : 1;
  const int split = tail ? (int)(id % (uint32_t)splits) : 0;
  const uint32_t piece = id;  // of the tail
  if (tail) id = a.whole + id / (uint32_t)splits;
  uint32_t slot = id % slots;
  const int hk = (int)(id / slots);
  if (CAUSAL) slot = slots - 1 - slot;  // long tiles first
  Where w;
  const bool found = find<T::kRows>(a, slot, &w);
  if (tail && split == 0 && threadIdx.x < T::kRows) {
    // which row of the output each of the tile's is
    const int r = w.tile * T::kRows + (int)threadIdx.x;
    int64_t to = -1;
    if (found && r < w.lq * group)
      to = (int64_t)(w.q0 + r / group) * a.q_heads + hk * group + r % group;
    a.part_map[(int64_t)(id - a.whole) * T::kRows + threadIdx.x] = to;
  }
  if (!found) return;

  const int rows = w.lq * group;  // < 2^31 checked
  const int row0 = w.tile * T::kRows;
  // keys that the tile's last and first query see
  const int shift = w.lk - w.lq + 1;
  int end = w.lk, full = w.lk;
  if (CAUSAL) {
    const int last = min(rows - 1, row0 + T::kRows - 1) / group, first = row0 / group;
    end = min(w.lk, max(0, last + shift));
    full = min(w.lk, max(0, first + shift));
  }
  int tiles = (end + kTileKeys - 1) / kTileKeys;
  int t0 = 0;
  if (splits > 1) {
    const int per = (tiles + splits - 1) / splits;
    t0 = min(tiles, split * per);
    tiles = min(tiles, t0 + per);
  }

  // this lane's rows
  int row[QT], seen[QT];
  u4 qf[QT][T::kSteps];
#pragma unroll
  for (int t = 0; t < QT; ++t) {
    row[t] = row0 + (wave * QT + t) * 32 + col;
    const int r = min(row[t], rows - 1);
    const int token = r / group, head = hk * group + r % group;
    seen[t] = CAUSAL ? min(w.lk, token + shift) : w.lk;
    const uint16_t* q = a.q + (int64_t)(w.q0 + token) * a.q_stride + (int64_t)head * a.q_head_stride;
#pragma unroll
    for (int s = 0; s < T::kSteps; ++s) {
      const int c = 2 * s + half;
      const u4 zero = {0, 0, 0, 0};
      qf[t][s] = c * 8 < a.d ? *reinterpret_cast<const u4*>(q + c * 8) : zero;
    }
  }

  // copies: lane i of a copy fills the 16 bytes behind 16 i
  const int8_t* kbase =
      reinterpret_cast<const int8_t*>(a.k + (int64_t)w.k0 * a.k_stride + (int64_t)hk * a.k_head_stride);
  const int8_t* vbase =
      reinterpret_cast<const int8_t*>(a.v + (int64_t)w.k0 * a.v_stride + (int64_t)hk * a.v_head_stride);
  const uint32_t kstride = (uint32_t)a.k_stride * 2, vstride = (uint32_t)a.v_stride * 2;
  auto issue = [&](int t, int stage) {
    const int last = w.lk - 1 - t * kTileKeys;  // rows behind it repeat it
    const int8_t* kp = kbase + (int64_t)t * kTileKeys * a.k_stride * 2;
    const int8_t* vp = vbase + (int64_t)t * kTileKeys * a.v_stride * 2;
#pragma unroll
    for (int i = 0; i < T::kCopies; ++i) {
      const int at = (wave * T::kCopies + i) * 64;
      const int r = (at + lane) / T::kChunks, c = (at + lane) % T::kChunks;
      const int from = min(r, last);
      const int kc = min(k_slot<DP>(r, c), a.d / 8 - 1), vc = min(v_slot<DP>(r, c), a.d / 8 - 1);
      dma16(kp, from * kstride + kc * 16, stage * T::kTileBytes + at * 16);
      dma16(vp, from * vstride + vc * 16,
            (T::kStages + stage) * T::kTileBytes + at * 16);
    }
  };

  v16f o[QT][T::kDTiles];
  v16f below[QT];           // -m in every place: the first product starts from it
  float l[QT], raise_at[QT];
#pragma unroll
  for (int t = 0; t < QT; ++t) {
    below[t] = (v16f){0};
    raise_at[t] = -__builtin_inff();  // no m yet
    l[t] = 0.f;
#pragma unroll
    for (int d = 0; d < T::kDTiles; ++d) o[t][d] = (v16f){0};
  }
  const float c = a.scale * kLog2e;
  const float room = kRoom / c;

  if (t0 < tiles) issue(t0, 0);
  for (int t = t0; t < tiles; ++t) {
    const int stage = (t - t0) & 1;
    wait_vmcnt<0>();
    wait_lgkm0();
    lds_barrier();
    if (t + 1 < tiles) issue(t + 1, stage ^ 1);
    const uint8_t* kt = lds + stage * T::kTileBytes;
    uint8_t* vt = lds + (T::kStages + stage) * T::kTileBytes;
    v16f s[2][QT];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
#pragma unroll
      for (int st = 0; st < T::kSteps; ++st) {
        const int r = u * 32 + col;
        const u4 kf = *reinterpret_cast<const u4*>(kt + r * T::kRowBytes +
                                                   k_slot<DP>(r, 2 * st + half) * 16);
#pragma unroll
        for (int q = 0; q < QT; ++q)
          s[u][q] = mfma<F16>(kf, qf[q][st], st == 0 ? below[q] : s[u][q]);
      }
    }
    const int key0 = t * kTileKeys;
    if (key0 + kTileKeys > full) {
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int q = 0; q < QT; ++q)
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int key = key0 + u * 32 + 8 * (i >> 2) + 4 * half + (i & 3);
            if (key >= seen[q]) s[u][q][i] = -__builtin_inff();
          }
    }
    float top[QT];
    bool raise = false;
#pragma unroll
    for (int q = 0; q < QT; ++q) {
      top[q] = s[0][q][0];
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int i = 0; i < 16; ++i) top[q] = fmaxf(top[q], s[u][q][i]);
      top[q] = fmaxf(top[q], other_half(top[q]));
      raise |= top[q] > raise_at[q];
    }
    if (__any(raise)) {
#pragma unroll
      for (int q = 0; q < QT; ++q) {
        const bool up = top[q] > raise_at[q];
        const float by = up ? top[q] : 0.f;
        // a row without an m has nothing to scale yet (or NaN, which stays)
        const float alpha =
            up && raise_at[q] > kLowest ? __builtin_amdgcn_exp2f(-by * c) : 1.f;
        raise_at[q] = up ? room : raise_at[q];
        l[q] *= alpha;
#pragma unroll
        for (int i = 0; i < 16; ++i) below[q][i] -= by;
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int i = 0; i < 16; ++i) s[u][q][i] -= by;
#pragma unroll
        for (int d = 0; d < T::kDTiles; ++d)
#pragma unroll
          for (int i = 0; i < 16; ++i) o[q][d][i] *= alpha;
      }
    }
    u4 p[2][QT][2];
#pragma unroll
    for (int q = 0; q < QT; ++q) {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          s[u][q][i] = __builtin_amdgcn_exp2f(
              F16 ? __builtin_fmaf(s[u][q][i], c, kLift<F16>) : s[u][q][i] * c);
          l[q] += s[u][q][i];
        }
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            p[u][q][h][e] = pack16x2<F16>(s[u][q][8 * h + 2 * e], s[u][q][8 * h + 2 * e + 1]);
      }
    }
    if (CAUSAL && key0 + kTileKeys > full && clear_nonfinite<F16, DP, kTileKeys>(vt)) *cleared = 1;
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int d = 0; d < T::kDTiles; ++d) {
          const u4 vf = values<DP>(vt, u * 32 + h * 16, d);
#pragma unroll
          for (int q = 0; q < QT; ++q) o[q][d] = mfma<F16>(vf, p[u][q][h], o[q][d]);
        }
  }

  if (CAUSAL) {
    wait_lgkm0();
    lds_barrier();
    if (__builtin_expect(*cleared, 0)) {
      const int to = min(end, tiles * kTileKeys);
#pragma unroll 1
      for (int key = max(full / kTileKeys, t0) * kTileKeys; key < to; ++key)
#pragma unroll
        for (int q = 0; q < QT; ++q)
          add_nonfinite<T::kDTiles, F16>(a, w.k0 + key, hk, key < seen[q], o[q]);
    }
  }

#pragma unroll
  for (int q = 0; q < QT; ++q) {
    const float sum = l[q] + other_half(l[q]);
    const float inv = sum > 0.f || sum != sum ? 1.0f / sum : 0.f;
    const float lse2 = sum > 0.f || sum != sum ? log2f(sum) - kLift<F16> - below[q][0] * c : -__builtin_inff();
    if (row[q] >= rows) continue;
    if (tail) {
      const int64_t at = (int64_t)piece * T::kRows + row[q] - row0;
      if (half == 0) a.part_lse[at] = lse2;
      if (lse2 == -__builtin_inff()) continue;
      float* to = a.part + at * a.d;
#pragma unroll
      for (int d = 0; d < T::kDTiles; ++d)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int e = d * 32 + i * 8 + half * 4;
          const v4f f = {o[q][d][4 * i] * inv, o[q][d][4 * i + 1] * inv, o[q][d][4 * i + 2] * inv,
                         o[q][d][4 * i + 3] * inv};
          if (e < a.d) *reinterpret_cast<v4f*>(to + e) = f;
        }
      continue;
    }
    const int token = row[q] / group, head = hk * group + row[q] % group;
    if (a.lse && half == 0) a.lse[(int64_t)head * a.q_tokens + w.q0 + token] = lse2 * kLn2;
    uint16_t* to = a.out + (int64_t)(w.q0 + token) * a.out_stride + (int64_t)head * a.out_head_stride;
    // the two lanes of a row hold four elements of each eight: they swap, so that each
    // has every other eight
#pragma unroll
    for (int d = 0; d < T::kDTiles; ++d)
#pragma unroll
      for (int i = 0; i < 4; i += 2) {
        u4 f;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          typedef uint32_t u2v __attribute__((ext_vector_type(2)));
          const int n = 4 * i + 2 * j;
          const u2v x = __builtin_amdgcn_permlane32_swap(
              pack16x2<F16>(o[q][d][n] * inv, o[q][d][n + 1] * inv),
              pack16x2<F16>(o[q][d][n + 4] * inv, o[q][d][n + 5] * inv), false, false);
          f[j] = x.x;
          f[2 + j] = x.y;
        }
        const int e = d * 32 + (i + half) * 8;
        if (e < a.d) *reinterpret_cast<u4*>(to + e) = f;
      }
  }
}

// ---- few rows: single tokens against a long cache ----------------------------
//
// Up to 32 rows a tile, bound by the bytes of the keys: every wave of a block
// streams its own units of 32 keys, copied two ahead into its own part of LDS, and
// waits for no other wave until the end, where the waves' sums are joined. Weights
// go into the second product in two 16-bit parts, which costs nothing here.
template <int DP>
struct Few {
  static constexpr int kWaves = DP == 256 ? 2 : 4;
  static constexpr int kUnit = 32;
  static constexpr int kRowBytes = DP * 2;
  static constexpr int kChunks = DP / 8;
  static constexpr int kUnitBytes = kUnit * kRowBytes;
  static constexpr int kRing = 2;
  static constexpr int kWaveBytes = 2 * kRing * kUnitBytes;  // K and V
  static constexpr int kCopies = kUnitBytes / 1024;
  static constexpr int kJoinRow = DP + 4;  // floats of a row of partial sums
  static constexpr int kLds = kWaves * kWaveBytes;
  static_assert(kWaves * (32 * kJoinRow + 64) * 4 <= kLds, "sums fit the ring");
};

template <int DP, bool F16>
__global__ __launch_bounds__(64 * Few<DP>::kWaves, 1) void attention_few_kernel(AttentionArgs a,
                                                                                int chunk) {
  using T = Few<DP>;
  constexpr int kSteps = DP / 16, kDTiles = DP / 32;
  extern __shared__ __align__(1024) uint8_t lds[];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int half = lane >> 5, col = lane & 31;
  const int group = a.group;
  const uint32_t id = blockIdx.x;
  const int split = (int)(id % (uint32_t)a.splits);
  const uint32_t rest = id / (uint32_t)a.splits;
  const int hk = (int)(rest % (uint32_t)a.k_heads);
  Where w;
  if (!find<32>(a, rest / (uint32_t)a.k_heads, &w)) return;

  const int rows = w.lq * group, row0 = w.tile * 32;
  const int shift = w.lk - w.lq + 1;
  int end = w.lk, full = w.lk;
  if (a.causal) {
    end = min(w.lk, max(0, min(rows - 1, row0 + 31) / group + shift));
    full = min(w.lk, max(0, row0 / group + shift));
  }
  // units of this split, dealt to the waves: `chunk`, or more where the sequence is longer
  const int units = (end + T::kUnit - 1) / T::kUnit;
  const int per = max(chunk, (units + a.splits - 1) / a.splits);
  const int first = min(units, split * per), last = min(units, first + per);

  const int row = row0 + col;
  const int r = min(row, rows - 1);
  const int token = r / group, head = hk * group + r % group;
  const int seen = a.causal ? min(w.lk, token + shift) : w.lk;
  u4 qf[kSteps];
  {
    const uint16_t* q = a.q + (int64_t)(w.q0 + token) * a.q_stride + (int64_t)head * a.q_head_stride;
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      const int e = (2 * s + half) * 8;
      const u4 zero = {0, 0, 0, 0};
      qf[s] = e < a.d ? *reinterpret_cast<const u4*>(q + e) : zero;
    }
  }

  const int8_t* kbase =
      reinterpret_cast<const int8_t*>(a.k + (int64_t)w.k0 * a.k_stride + (int64_t)hk * a.k_head_stride);
  const int8_t* vbase =
      reinterpret_cast<const int8_t*>(a.v + (int64_t)w.k0 * a.v_stride + (int64_t)hk * a.v_head_stride);
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

  v16f o[kDTiles], below = (v16f){0};
#pragma unroll
  for (int d = 0; d < kDTiles; ++d) o[d] = (v16f){0};
  float l = 0.f, raise_at = -__builtin_inff();
  const float c = a.scale * kLog2e, room = kRoom / c;

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
    v16f s = below;
#pragma unroll
    for (int st = 0; st < kSteps; ++st) {
      const u4 kf = *reinterpret_cast<const u4*>(kt + col * T::kRowBytes +
                                                 k_slot<DP>(col, 2 * st + half) * 16);
      s = mfma<F16>(kf, qf[st], s);
    }
    const int key0 = u * T::kUnit;
    if (key0 + T::kUnit > full) {
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (key0 + 8 * (i >> 2) + 4 * half + (i & 3) >= seen) s[i] = -__builtin_inff();
    }
    float top = s[0];
#pragma unroll
    for (int i = 1; i < 16; ++i) top = fmaxf(top, s[i]);
    top = fmaxf(top, other_half(top));
    if (__any(top > raise_at)) {
      const bool up = top > raise_at;
      const float by = up ? top : 0.f;
      const float alpha = up && raise_at > kLowest ? __builtin_amdgcn_exp2f(-by * c) : 1.f;
      raise_at = up ? room : raise_at;
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
    const bool cleared =
        a.causal && key0 + T::kUnit > full && clear_nonfinite<F16, DP, T::kUnit>(vt);
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
    stat[wave * 64 + col] = raise_at > kLowest ? -below[0] : kLowest;
    stat[wave * 64 + 32 + col] = sum;
  }
  wait_lgkm0();
  lds_barrier();
  const int here = min(32, rows - row0);
  constexpr int kQuads = DP / 4;
  for (int i = threadIdx.x; i < here * kQuads; i += 64 * T::kWaves) {
    const int jr = i / kQuads, e = i % kQuads * 4;
    if (e >= a.d) continue;
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
    const bool some = total > 0.f || total != total;
    const float inv = some ? 1.0f / total : 0.f;
    const float lse2 = some ? log2f(total) - kLift<F16> + m * c : -__builtin_inff();
    const int jtoken = (row0 + jr) / group, jhead = hk * group + (row0 + jr) % group;
#pragma unroll
    for (int q = 0; q < 4; ++q) acc[q] *= inv;
    if (a.splits > 1) {
      const int64_t at = ((int64_t)split * a.q_tokens + w.q0 + jtoken) * a.q_heads + jhead;
      if (e == 0) a.part_lse[at] = lse2;
      if (some) *reinterpret_cast<v4f*>(a.part + at * a.d + e) = acc;
      continue;
    }
    if (a.lse && e == 0) a.lse[(int64_t)jhead * a.q_tokens + w.q0 + jtoken] = lse2 * kLn2;
    const u2 f = {pack16x2<F16>(acc[0], acc[1]), pack16x2<F16>(acc[2], acc[3])};
    *reinterpret_cast<u2*>(a.out + (int64_t)(w.q0 + jtoken) * a.out_stride + (int64_t)jhead * a.out_head_stride + e) =
        f;
  }
}

// Joins the splits of a row: out = sum_s 2^(lse_s - lse) out_s. A block takes a row: a
// thread a split's factor, then groups of lanes, four elements each, the splits in turn,
// all of whose loads are under way together.
constexpr int kJoinThreads = 256;

template <bool F16>
__global__ __launch_bounds__(kJoinThreads) void attention_join_kernel(AttentionArgs a, int lanes) {
  __shared__ float factor[kMaxSplits];
  __shared__ float red[2][kJoinThreads / 64];
  __shared__ __align__(16) float acc[kJoinThreads * 4];
  // few rows: parts [split][row of the output]; tiles: [tile][split][row of the tile]
  int64_t r = blockIdx.x, at = r, step = a.q_tokens * a.q_heads;
  if (a.part_map) {
    step = kRowsOfTile;
    at = r / step * step * a.splits + r % step;
    r = a.part_map[r];
    if (r < 0) return;
  }
  const int64_t token = r / a.q_heads;
  const int head = (int)(r % a.q_heads);
  if (!a.part_map && a.q_offsets && (token < a.q_offsets[0] || token >= a.q_offsets[a.batch]))
    return;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int group = tid / lanes, groups = kJoinThreads / lanes, e = tid % lanes * 4;

  float x[kMaxSplits / kJoinThreads];
  float top = kLowest;
#pragma unroll
  for (int i = 0; i < kMaxSplits / kJoinThreads; ++i) {
    const int s = tid + i * kJoinThreads;
    x[i] = s < a.splits ? a.part_lse[at + s * step] : -__builtin_inff();
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
    if (tid + i * kJoinThreads < a.splits) factor[tid + i * kJoinThreads] = f;
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
    for (int s = group; s < a.splits; s += groups) {
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
    const float inv = none ? 0.f : 1.0f / sum;
    const u2 f = {pack16x2<F16>(v[0] * inv, v[1] * inv), pack16x2<F16>(v[2] * inv, v[3] * inv)};
    *reinterpret_cast<u2*>(a.out + token * a.out_stride + (int64_t)head * a.out_head_stride + e) = f;
  }
}

template <int DP, int QT, int NW, bool F16>
hipError_t launch_tile(const AttentionArgs& a, const AttentionPlan& p, hipStream_t st) {
  using T = Kernel<DP, QT, NW, F16>;
  auto kern = a.causal ? attention_kernel<DP, QT, NW, F16, true>
                       : attention_kernel<DP, QT, NW, F16, false>;
  if (T::kLds > 65536) {
    // per device: the attribute is set on every call (a host-side table write)
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kern),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, T::kLds);
    if (e != hipSuccess) return e;
  }
  kern<<<dim3((uint32_t)p.grid), dim3(64 * NW), T::kLds, st>>>(a, (uint32_t)p.slots,
                                                               xcd_count(compute_units()));
  return hipGetLastError();
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
  kern<<<dim3((uint32_t)p.grid), dim3(64 * T::kWaves), T::kLds, st>>>(a, p.chunk);
  return hipGetLastError();
}

template <bool F16>
hipError_t launch_dtype(const AttentionArgs& a, const AttentionPlan& p, hipStream_t st) {
  hipError_t e;
  if (p.rows == 32)
    e = a.d <= 64    ? launch_few<64, F16>(a, p, st)
        : a.d <= 128 ? launch_few<128, F16>(a, p, st)
                     : launch_few<256, F16>(a, p, st);
  else if (a.d <= 64)
    e = launch_tile<64, 1, 4, F16>(a, p, st);
  else if (a.d <= 128)
    e = launch_tile<128, 1, 4, F16>(a, p, st);
  else
    e = launch_tile<256, 1, 4, F16>(a, p, st);
  if (e != hipSuccess || a.splits == 1) return e;
  int lanes = 1;
  while (lanes * 4 < a.d) lanes *= 2;
  attention_join_kernel<F16><<<dim3((uint32_t)p.part_rows), dim3(kJoinThreads), 0, st>>>(a, lanes);
  return hipGetLastError();
}

size_t workspace_bytes(const AttentionPlan& p, int d) {
  if (p.splits <= 1) return 0;
  return (size_t)p.part_rows * ((size_t)p.splits * (d + 1) * 4 + (p.rows == 32 ? 0 : 8));
}

}  // namespace

AttentionPlan plan_attention(const AttentionArgs& a, size_t workspace) {
  AttentionPlan p;
  const int64_t group = a.q_heads / a.k_heads;
  const int64_t rows = a.q_tokens * group;  // of a key head
  const int64_t keys = a.k_tokens / a.batch;
  p.rows = rows <= 32 * (int64_t)a.batch ? 32 : kRowsOfTile;
  if (a.q_offsets)
    p.slots = (rows + p.rows - 1) / p.rows + a.batch;
  else
    p.slots = a.batch * ((rows / a.batch + p.rows - 1) / p.rows);
  const int64_t blocks = p.slots * a.k_heads;
  if (p.rows == 32) {
    // sequences may use less of their keys than there is room for: splits of a fixed
    // length, about two rounds of a block per compute unit if all is used
    const int64_t units = (keys + 31) / 32;
    int64_t tiles = (rows + 31) / 32;
    tiles = (tiles > a.batch ? tiles : a.batch) * a.k_heads;
    int64_t chunk = (units * tiles + kMaxSplits - 1) / kMaxSplits;
    if (chunk < 8) chunk = 8;
    int64_t splits = (units + chunk - 1) / chunk;
    if (splits > kMaxSplits) splits = kMaxSplits;
    p.part_rows = a.q_tokens * a.q_heads;
    p.splits = splits < 1 ? 1 : (int)splits;
    while (workspace_bytes(p, a.d) > workspace) --p.splits;
    if (p.splits == 1) p.part_rows = 0;
    p.chunk = (int)((units + p.splits - 1) / p.splits);
    p.grid = blocks * p.splits;
    return p;
  }
  // Blocks run `room` at a time. The tiles behind the last whole round (all, if there
  // are not that many) are split over their keys into as many parts as cost least:
  // rounds of the parts, each with its start and end (about 2.5 key tiles' time), and
  // the join. In a round of at most half its blocks these have a compute unit to
  // themselves and take 0.62 of the time. Causal tiles come longest first and even
  // out by themselves if there is more than one round.
  const int64_t room = a.d > 128 ? kMaxSplits / 2 : kMaxSplits;
  const int64_t tiles = (keys + kTileKeys - 1) / kTileKeys;
  const int64_t whole = blocks / room * room, rest = blocks - whole;
  p.whole = blocks;
  p.grid = blocks;
  if (rest == 0 || (a.causal && whole > 0)) return p;
  double least = 0;
  auto consider = [&](int64_t n) {
    if (n > tiles / 4) n = tiles / 4;
    if (n < 1) return;
    AttentionPlan t = p;
    t.whole = whole;
    t.splits = (int)n;
    t.part_rows = rest * p.rows;
    t.grid = whole + rest * n;
    const int64_t full = rest * n / room, last = rest * n % room;
    const double rounds = full + (last == 0 ? 0 : 2 * last <= room ? 0.62 : 1.0);
    const double cost = rounds * (1.0 / n + 2.5 / tiles) + (n > 1 ? 5.0 / tiles : 0);
    if (least != 0 && (cost >= least || workspace_bytes(t, a.d) > workspace)) return;
    least = cost;
    if (n > 1) p = t;
  };
  for (int64_t n = 1; n <= 8; ++n) consider(n);
  // half a round, one, two
  for (int64_t of = room / 2; of <= 2 * room; of *= 2) consider(of / rest);
  return p;
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
  if (p.splits == 1) return;
  char* at = static_cast<char*>(workspace);
  if (p.rows != 32) {
    a->part_map = reinterpret_cast<int64_t*>(at);
    at += p.part_rows * 8;
  }
  a->part = reinterpret_cast<float*>(at);
  a->part_lse = a->part + (size_t)p.splits * (size_t)p.part_rows * a->d;
}

hipError_t launch_attention(const AttentionArgs& a, const AttentionPlan& p, DType dt,
                            hipStream_t st) {
  if (p.grid == 0) return hipSuccess;
  return dt == DType::kF16 ? launch_dtype<true>(a, p, st) : launch_dtype<false>(a, p, st);
}

}  // namespace convrot
