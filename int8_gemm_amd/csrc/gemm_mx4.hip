// Microscaled 4-bit GEMM (gfx950): y = a . b^T over two MXFP4 tensors.
//
// y[m, n] = RN16(sum_k xa[m, k] wb[n, k] [+ bias[n]]), xa and wb the values that
// codes and scales stand for (layout in mx4.h), products exact, sums in fp32
// inside v_mfma_scale_f32_*_f8f6f4, which takes the two 2^e of each 32-long
// block as operands. Both operands are K-contiguous.
//
// Tiled kernel: the int8 GEMM's pipeline (gemm.hip) with the bytes reread: an
// MFMA of 32 x 32 x 64 4-bit elements takes the same two 1 KB operands as the
// 32 x 32 x 32 int8 one. A K-step is 256 elements: 128 bytes of each row, and
// 8 scale bytes of each row, which the scale layout keeps contiguous over
// rows; every copying wave brings its share of both into the LDS ring with
// global -> LDS copies. The half h of a wave multiplies blocks 4 h .. 4 h + 3 of
// the K-step, one per slice (any order of K serves, if both operands share
// it), so a lane's four scales of a row are one 32-bit LDS read and the
// instruction selects the slice's byte.
//
// Measured: 32760 x 13824 x 5120 1.17-1.18 ms in a steady row, 1.24 (1.18-1.30) as
// the median of the first twelve launches, 3.7-4.0 PFLOP/s, under the power limit:
// the clock falls to 1.63 GHz and the MFMA pipes are busy 0.55 of it (with nearly
// no copies the same loop takes 0.95 ms, without its LDS reads as well 0.90; reads
// from LDS alone cost 2-4%). So are grids of some 240 large tiles (at least 1.63
// GHz, MFMA busy 0.52): a K-step of a 384 x 192 tile takes 0.97 us without its
// copies and 1.16 with them when 20 CUs work, 1.69 and 1.99 when 240 do (4608 x 3840
// x 3840 38-40 us). Smaller grids are bound by their operands' way into the XCDs'
// L2 and by the launch's start and end: 333 x 9216 x K takes 6 us and 0.45 a K-step
// (K = 2048 9.6, 3840 12.4, 5120 14.9 us). Copies without any arithmetic take 0.46 us
// a K-step there, with three stages or four (lines that L2 holds already come at
// 52-62 bytes per cycle and CU, these at 30). Where K / 2 is no multiple of 128 each
// 128-byte piece of a row lies on two lines, which costs that grid 2.4 us more (K
// = 3872 15.2 us against 12.8 at 4096, 4896 17.4 against 14.9 at 5120). Up to 192 rows
// a tile, waves of their own do the copies: issued between the MFMAs of the waves
// that compute, they cost 512 x 5120 x 5120 17.8 instead of 13.3 us. The two large
// tiles' accumulators leave no registers for that. Tried without gain: reading the
// fragments of a whole K-step ahead, a fourth stage for the 128 tile, eight
// computing or eight copying waves, K-steps of half the length with twice the
// stages (copies alone 17.3 -> 21.8 us at 4608 x 3840 x 3840), a wave that touches the
// lines four stages ahead (512 x 5120 x 5120 13.0 -> 16.4), starting the first blocks
// at different times.
//
// The end of K: what stands in the place of columns behind a row's end are
// codes of the next row (the copies stop at the tensor's end) with both
// scales set to 2^-127: every 4-bit value is finite and the products underflow
// to zero.
//
// Few rows: a block takes 16 columns of y; its waves split K and read their
// 16 rows of the weight straight into registers, 128 bytes of a row at a time,
// each weight byte once for all rows; the partial sums are joined in LDS in
// wave order. Bound by the weight's bytes and, with more rows, by each CU's
// loads of x: 13824 x 5120 (37.6 MB) takes 9.5 us with one row, 4.0 TB/s of the
// weight's bytes (8.4 us with weights in the last-level cache). Where the loads of
// x take longer than small tiles would, the tiled kernel is taken (few_rows below).

#include <atomic>
#include <type_traits>

#include "internal.h"
#include "lds_copy.h"
#include "mx4.h"

namespace convrot {

namespace {

typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef float v16f __attribute__((ext_vector_type(16)));

constexpr int kFp4 = 4;  // operand format of the scaled MFMA

// the 4-bit format reads the low half of the operand registers only
__device__ __forceinline__ v8i wide(v4i a) { return __builtin_shufflevector(a, a, 0, 1, 2, 3, -1, -1, -1, -1); }

// global -> LDS copy of 16 bytes per lane (as dma16) from a per-lane address,
// by the lanes of `lanes` only; the mask is set inside the asm block because a
// divergent branch around the copy would split the K-loop's schedule. The two
// moves of the mask stand for the wait state that the copy needs behind M0.
__device__ __forceinline__ void dma16_at(const uint8_t* p, uint32_t lds_base, uint64_t lanes) {
  uint64_t saved;
  asm volatile(
      "s_mov_b32 m0, %2\n\ts_mov_b64 %0, exec\n\ts_mov_b64 exec, %3\n\t"
      "global_load_lds_dwordx4 %1, off\n\ts_mov_b64 exec, %0"
      : "=&s"(saved)
      : "v"(p), "s"(lds_base), "s"(lanes)
      : "memory", "m0");
}

template <int SEL>
__device__ __forceinline__ v16f mfma32(v4i a, uint32_t sa, v4i b, uint32_t sb, v16f c) {
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(wide(a), wide(b), c, kFp4, kFp4, SEL,
                                                         (int)sa, SEL, (int)sb);
}
template <int SEL>
__device__ __forceinline__ v4f mfma16(v4i a, uint32_t sa, v4i b, uint32_t sb, v4f c) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wide(a), wide(b), c, kFp4, kFp4, SEL,
                                                          (int)sa, SEL, (int)sb);
}

// Wait until at most min(p, P) stages of LW copies are outstanding.
template <int P, int LW>
__device__ __forceinline__ void wait_stages(int p) {
  if constexpr (P > 0) {
    if (p < P) {
      wait_stages<P - 1, LW>(p);
      return;
    }
  }
  wait_vmcnt<P * LW>();
}

template <int BM, int BN, int WM, int WN, int NS, int MINB, int NP, bool F16>
__global__ __launch_bounds__(64 * (WM * WN + NP), MINB) void gemm_mx4_kernel(
    const uint8_t* __restrict__ xc, const uint8_t* __restrict__ xs,
    const uint8_t* __restrict__ wc, const uint8_t* __restrict__ ws,
    const uint16_t* __restrict__ bias, int M, int N, int K, int tiles_m, int tiles_n, int nx,
    uint16_t* __restrict__ y) {
  constexpr int BK = 128;                      // bytes of a row per K-step
  constexpr int NW = WM * WN;                  // compute waves: WM along m, WN along n
  constexpr int WTM = BM / WM, WTN = BN / WN;  // wave tile
  constexpr int NJ = WTM / 32, NI = WTN / 32;
  constexpr int DW = NP > 0 ? NP : NW;         // waves that issue copies
  constexpr int RPI = 1024 / BK;               // rows per copy instruction
  constexpr int CPR = BK / 16;
  constexpr int RPB = 2;                       // rows per 256-byte LDS bank line
  constexpr int LC = (BM + BN) / (RPI * DW);   // code copies per copying wave per stage
  constexpr int LW = LC + 1;                   // and one of scales
  constexpr int RW = (BM + BN) / DW;           // rows whose scales a copying wave brings
  constexpr int CODES = (BM + BN) * BK;
  constexpr int STAGE = CODES + (BM + BN) * 8;  // bytes per LDS stage: codes, then scales
  constexpr int H = 4;                         // 64-element slices per K-step
  constexpr int LA = NS;
  static_assert(WTM % 32 == 0 && WTN % 32 == 0 && (BM + BN) % (RPI * DW) == 0, "tile shape");
  static_assert(RW % 2 == 0 && RW / 2 <= 64 && BN % 2 == 0, "two rows' scales per lane");
  static_assert(NS >= 2 && LA * LW < 64, "copies in flight per wave must fit vmcnt");
  extern __shared__ __attribute__((aligned(1024))) uint8_t lds[];

  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wn = wave % WN;
  const int wm = wave / WN;
  const int cw = NP > 0 ? (wave >= NW ? wave - NW : 0) : wave;  // index among the copying waves

  // ---- tile index: XCD-contiguous ranges, grouped rows (as in gemm.hip) ----
  const int ntiles = tiles_m * tiles_n;
  int bid = blockIdx.x;
  {
    const int per = (ntiles + nx - 1) / nx;
    const int xcd = bid % nx;
    const int loc = bid / nx;
    const int full = ntiles - (per - 1) * nx;
    bid = (xcd < full) ? xcd * per + loc : full * per + (xcd - full) * (per - 1) + loc;
  }
  constexpr int GROUP = 8;
  const int group_sz = GROUP * tiles_n;
  const int grp = bid / group_sz;
  const int first_m = grp * GROUP;
  const int gm = min(tiles_m - first_m, GROUP);
  const int in_grp = bid - grp * group_sz;
  const int m0 = (first_m + in_grp % gm) * BM;
  const int n0 = (in_grp / gm) * BN;

  // ---- copies: instruction t of this wave covers the 8 combined rows 8 q ..
  // (weights first, then activations), lane -> row 8 q + lane / 8, 16-byte slot
  // lane % 8. Slot p of a row holds chunk 4 (p' & 1) + p' / 2, p' = p ^ (row / 2) %
  // 8: the two halves of a wave then read neighbouring slots, as the bank
  // swizzle needs. The row groups' addresses are uniform; a lane's offset from
  // them has two forms, for even and odd q. ----
  const int KB = K / 2;
  const int nk = (KB + BK - 1) / BK;
  const int tail = KB - (nk - 1) * BK;  // bytes of the last K-step, a multiple of 16
  uint32_t voff[2];
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int slot = (lane % CPR) ^ ((4 * t + lane / 16) % CPR);
    voff[t] = (uint32_t)(lane / CPR) * (uint32_t)KB + 16u * (4 * (slot & 1) + slot / 2);
  }
  // scales: each of the first RW / 2 lanes brings those of two consecutive
  // rows (pad rows exist up to a multiple of 16)
  const uint8_t* sptr;
  int64_t sstep;
  {
    const int r = cw * RW + 2 * min(lane, RW / 2 - 1);  // a lane's rows are both weights or both not
    const bool w = r < BN;
    const int64_t pad = mx4_pad_rows(w ? N : M);
    const int64_t row = min((int64_t)(w ? n0 + r : m0 + r - BN), pad - 2);
    sptr = (w ? ws : xs) + row * 8;
    sstep = pad * 8;
  }
  const uint32_t lds_u32 = (uint32_t)(uintptr_t)(lds_ptr_t)lds;
  // called once per stage, in order
  auto issue = [&](int s, int slot) {
    dma16_at(sptr, lds_u32 + (uint32_t)(slot * STAGE + CODES + cw * RW * 8),
             RW / 2 == 64 ? ~0ull : (1ull << (RW / 2 % 64)) - 1);
    sptr += sstep;
#pragma unroll
    for (int t = 0; t < LC; ++t) {
      const int q = cw * LC + t;
      const bool w = RPI * q < BN;
      // a group that starts behind the tensor's end reads around its last row;
      // nothing is read behind the end
      const int rows = w ? N : M;
      const int row = min(w ? n0 + RPI * q : m0 + RPI * q - BN, rows - 1);
      const int64_t at = (int64_t)row * KB + (int64_t)s * BK;
      const uint32_t most = (uint32_t)(min(rows - row, RPI) * KB - s * BK - 16);
      const int8_t* base = reinterpret_cast<const int8_t*>(w ? wc : xc) + at;
      dma16(base, min(voff[q & 1], most), lds_u32 + (uint32_t)(slot * STAGE + q * 1024));
    }
  };

  v16f acc[NI][NJ];
#pragma unroll
  for (int i = 0; i < NI; ++i)
#pragma unroll
    for (int j = 0; j < NJ; ++j) acc[i][j] = (v16f){};

  // a stage's copies are complete when at most the copies of the p later
  // stages are outstanding (copies complete in order)
  auto wait_stage = [&](int p) { wait_stages<LA - 1, LW>(p); };

  // The output tile is staged in LDS (the ring is free after the K-loop), then
  // stored as whole rows in 16-byte pieces.
  constexpr int PITCH = BN * 2 + 16;
  static_assert(BM * PITCH <= 160 * 1024, "staged output tile");
  auto store_tile = [&]() {
    wait_lgkm0();
    lds_barrier();
    constexpr int CPR16 = BN * 2 / 16;
#pragma unroll 4
    for (int idx = tid; idx < BM * CPR16; idx += 64 * (NW + NP)) {
      const int r = idx / CPR16;
      const int cc = idx - r * CPR16;
      const int m = m0 + r, n = n0 + 8 * cc;
      if (m < M && n < N)  // N % 16 == 0: a piece is all inside or all outside
        *reinterpret_cast<u4*>(y + (int64_t)m * N + n) =
            *reinterpret_cast<const u4*>(lds + r * PITCH + 16 * cc);
    }
  };

  if constexpr (NP > 0) {
    if (wave >= NW) {
      // ---- producer: same barriers as a consumer ----
#pragma unroll
      for (int s = 0; s < LA; ++s)
        if (s < nk) issue(s, s % NS);
      wait_stage(min(LA - 1, nk - 1));
      lds_barrier();
      for (int s = 0; s + 1 < nk; ++s) {
        wait_stage(min(LA - 2, nk - 2 - s));
        lds_barrier();
        if (s + LA < nk) issue(s + LA, (s + LA) % NS);
      }
      lds_barrier();  // the consumers' last-step barrier
      lds_barrier();  // ... and the one before staging the tile
      store_tile();
      return;
    }
  } else {
#pragma unroll
    for (int s = 0; s < LA; ++s)
      if (s < nk) issue(s, s % NS);
  }

  // MFMA operands: lane -> row lane % 32 of a 32-row block, 16-byte chunk
  // 4 (lane / 32) + h of slice h (one 32-element block of the row)
  const int fr = lane & 31;
  const int fh = lane >> 5;
  const int swz = (fr / RPB) % CPR;
  int dsw[H];
#pragma unroll
  for (int h = 0; h < H; ++h) dsw[h] = 16 * ((2 * h + fh) ^ swz);
  int aoff[NI], boff[NJ];
#pragma unroll
  for (int i = 0; i < NI; ++i) aoff[i] = wn * WTN + i * 32 + fr;
#pragma unroll
  for (int j = 0; j < NJ; ++j) boff[j] = BN + wm * WTM + j * 32 + fr;
  // blocks behind K take scale byte 0
  uint32_t tail_mask = 0;
#pragma unroll
  for (int h = 0; h < H; ++h)
    if (16 * (4 * fh + h) < tail) tail_mask |= 0xFFu << (8 * h);

  // Slices alternate between the register sets X and Y, as in gemm.hip: while
  // the MFMAs of one run, the next one's fragments are read; the barrier of
  // step s comes before its last slice, whose MFMAs overlap the reads of step
  // s + 1 (its scales among them).
  constexpr int NF = NI + NJ;
  v4i xa[NI], xb[NJ], ya[NI], yb[NJ];
  uint32_t sa[NI], sb[NJ], na[NI], nb[NJ];  // scales of this step and the next
  auto read_slice = [&](int s, int h, v4i (&fa)[NI], v4i (&fb)[NJ]) {
    const uint8_t* base = lds + (s % NS) * STAGE + dsw[h];
#pragma unroll
    for (int j = 0; j < NJ; ++j) fb[j] = *reinterpret_cast<const v4i*>(base + boff[j] * BK);
#pragma unroll
    for (int i = 0; i < NI; ++i) fa[i] = *reinterpret_cast<const v4i*>(base + aoff[i] * BK);
  };
  auto read_scales = [&](int s) {
    const uint8_t* base = lds + (s % NS) * STAGE + CODES + 4 * fh;
#pragma unroll
    for (int j = 0; j < NJ; ++j) nb[j] = *reinterpret_cast<const uint32_t*>(base + boff[j] * 8);
#pragma unroll
    for (int i = 0; i < NI; ++i) na[i] = *reinterpret_cast<const uint32_t*>(base + aoff[i] * 8);
  };
  auto take_scales = [&](int s) {
    const uint32_t mask = s == nk - 1 ? tail_mask : 0xFFFFFFFFu;
#pragma unroll
    for (int j = 0; j < NJ; ++j) sb[j] = nb[j] & mask;
#pragma unroll
    for (int i = 0; i < NI; ++i) sa[i] = na[i] & mask;
  };
  auto mfma_slice = [&](auto sel, const v4i (&fa)[NI], const v4i (&fb)[NJ]) {
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
      for (int j = 0; j < NJ; ++j)
        acc[i][j] = mfma32<decltype(sel)::value>(fa[i], sa[i], fb[j], sb[j], acc[i][j]);
  };
  // spread `reads` LDS reads over the NI * NJ MFMAs of a slice
  auto sched_slice = [&](auto reads) {
    constexpr int R = decltype(reads)::value;
    constexpr int NM = NI * NJ;
    constexpr int PER = NM / R > 0 ? NM / R : 1;
    constexpr int NR = NM / PER < R ? NM / PER : R;
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);    // one LDS read
      __builtin_amdgcn_sched_group_barrier(0x008, PER, 0);  // PER MFMAs
    }
    __builtin_amdgcn_sched_group_barrier(0x100, R - NR, 0);
    __builtin_amdgcn_sched_group_barrier(0x008, NM - NR * PER, 0);
  };

  // Without such a use before the branches of the copy issue, the compiler
  // sinks the slices' MFMAs below them, away from the reads they cover.
  auto hold_acc = [&]() {
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
      for (int j = 0; j < NJ; ++j) asm volatile("" : "+v"(acc[i][j]));
  };

  asm volatile("" ::"s"(y), "s"(bias));  // their scalar loads complete before the K-loop
  if constexpr (NP == 0) wait_stage(min(LA - 1, nk - 1));
  lds_barrier();
  read_scales(0);
  read_slice(0, 0, xa, xb);
  take_scales(0);
  for (int s = 0; s < nk; ++s) {
    read_slice(s, 1, ya, yb);
    mfma_slice(std::integral_constant<int, 0>{}, xa, xb);
    sched_slice(std::integral_constant<int, NF>{});
    read_slice(s, 2, xa, xb);
    mfma_slice(std::integral_constant<int, 1>{}, ya, yb);
    sched_slice(std::integral_constant<int, NF>{});
    read_slice(s, 3, ya, yb);
    mfma_slice(std::integral_constant<int, 2>{}, xa, xb);
    sched_slice(std::integral_constant<int, NF>{});
    hold_acc();
    if constexpr (NP == 0) wait_stage(min(LA - 2, nk - 2 - s));  // stage s + 1 landed
    wait_lgkm0();  // this wave's reads of stage s are done
    lds_barrier();
    const bool late = NP == 0 && wave >= 4;
    if constexpr (NP == 0) {
      if (!late && s + LA < nk) issue(s + LA, (s + LA) % NS);
    }
    // the last step reads a stale slot here; those registers are not used
    read_scales(s + 1);
    read_slice(s + 1, 0, xa, xb);
    mfma_slice(std::integral_constant<int, 3>{}, ya, yb);
    sched_slice(std::integral_constant<int, 2 * NF>{});
    hold_acc();
    take_scales(s + 1);
    if constexpr (NP == 0) {
      if (late && s + LA < nk) issue(s + LA, (s + LA) % NS);
    }
  }

  // ---- epilogue: a lane holds row m = lane % 32 of a tile and columns
  // 8 a + 4 (lane / 32) + e for register 4 a + e ----
  wait_lgkm0();  // every wave's last ring reads are done before the tile is staged
  lds_barrier();
#pragma unroll
  for (int i = 0; i < NI; ++i) {
#pragma unroll
    for (int a = 0; a < 4; ++a) {
      const int nl = wn * WTN + i * 32 + 8 * a + 4 * fh;
      u2 bb = {0, 0};
      if (bias && n0 + nl < N) bb = *reinterpret_cast<const u2*>(bias + n0 + nl);
      const float b0 = lo16<F16>(bb.x), b1 = hi16<F16>(bb.x), b2 = lo16<F16>(bb.y),
                  b3 = hi16<F16>(bb.y);
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        const int ml = wm * WTM + j * 32 + fr;
        const v16f& v = acc[i][j];
        const u2 o = {pack16x2<F16>(v[4 * a] + b0, v[4 * a + 1] + b1),
                      pack16x2<F16>(v[4 * a + 2] + b2, v[4 * a + 3] + b3)};
        *reinterpret_cast<u2*>(lds + ml * PITCH + 2 * nl) = o;
      }
    }
  }
  store_tile();
}

// ---- few rows ---------------------------------------------------------------

constexpr int kRowWaves = 8;  // waves that split K; fixed, as it sets the order of the sums

// MF: groups of 16 rows of x, NF: groups of 16 columns of y per block.
template <int MF, int NF, bool F16>
__global__ __launch_bounds__(64 * kRowWaves) void gemm_mx4_rows_kernel(
    const uint8_t* __restrict__ xc, const uint8_t* __restrict__ xs,
    const uint8_t* __restrict__ wc, const uint8_t* __restrict__ ws,
    const uint16_t* __restrict__ bias, int M, int N, int K, uint16_t* __restrict__ y) {
  constexpr int W = kRowWaves;
  // K-steps in flight per wave, as registers allow (8 per operand and step)
  constexpr int U = MF + NF <= 2 ? 4 : (MF + NF <= 5 ? 3 : (MF + NF <= 6 ? 2 : 1));
  constexpr int T = MF * NF;         // 16 x 16 results of the block
  constexpr int TG = T < 4 ? T : 4;  // ... joined at a time
  __shared__ __attribute__((aligned(16))) float part[W][TG][16][20];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15;  // row of a 16-row block
  const int q = lane >> 4;  // 64-element quarter of the 256 elements of a K-step
  const int n0 = blockIdx.x * 16 * NF;
  const int KB = K / 2, nb = K / kMx4Block;
  const int steps = (K + kMx4Tile - 1) / kMx4Tile;
  const int64_t wpad = mx4_pad_rows(N) * 8, xpad = mx4_pad_rows(M) * 8;
  // rows behind the tensors' ends read the last one
  const uint8_t *wrow[NF], *wsr[NF], *xrow[MF], *xsr[MF];
#pragma unroll
  for (int f = 0; f < NF; ++f) {
    const int n = min(n0 + 16 * f + r, N - 1);
    wrow[f] = wc + (int64_t)n * KB;
    wsr[f] = ws + (int64_t)n * 8 + 2 * q;
  }
#pragma unroll
  for (int f = 0; f < MF; ++f) {
    const int m = min(16 * f + r, M - 1);
    xrow[f] = xc + (int64_t)m * KB;
    xsr[f] = xs + (int64_t)m * 8 + 2 * q;
  }
  v4f acc[NF][MF];
#pragma unroll
  for (int f = 0; f < T; ++f) acc[f / MF][f % MF] = (v4f){0.f, 0.f, 0.f, 0.f};

  for (int s0 = wave; s0 < steps; s0 += W * U) {
    v4i wa[U][NF][2], xb[U][MF][2];
    uint32_t sw[U][NF], sx[U][MF];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int s = s0 + u * W;
      if (s >= steps) break;
      // the lane's two blocks; behind the row's end the row's last block with
      // scale 2^-127 on both sides
      const int b0 = 8 * s + 2 * q;
      const uint32_t mask = (b0 < nb ? 0xFFu : 0u) | (b0 + 1 < nb ? 0xFF00u : 0u);
      const int o0 = 16 * min(b0, nb - 1), o1 = 16 * min(b0 + 1, nb - 1);
#pragma unroll
      for (int f = 0; f < NF; ++f) {
        wa[u][f][0] = *reinterpret_cast<const v4i*>(wrow[f] + o0);
        wa[u][f][1] = *reinterpret_cast<const v4i*>(wrow[f] + o1);
        sw[u][f] = *reinterpret_cast<const uint16_t*>(wsr[f] + s * wpad) & mask;
      }
#pragma unroll
      for (int f = 0; f < MF; ++f) {
        xb[u][f][0] = *reinterpret_cast<const v4i*>(xrow[f] + o0);
        xb[u][f][1] = *reinterpret_cast<const v4i*>(xrow[f] + o1);
        sx[u][f] = *reinterpret_cast<const uint16_t*>(xsr[f] + s * xpad) & mask;
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (s0 + u * W >= steps) break;
#pragma unroll
      for (int f = 0; f < NF; ++f)
#pragma unroll
        for (int j = 0; j < MF; ++j) {
          acc[f][j] = mfma16<0>(wa[u][f][0], sw[u][f], xb[u][j][0], sx[u][j], acc[f][j]);
          acc[f][j] = mfma16<1>(wa[u][f][1], sw[u][f], xb[u][j][1], sx[u][j], acc[f][j]);
        }
    }
  }
  // a lane holds columns 4 q .. 4 q + 3 of row r of each result
#pragma unroll
  for (int t0 = 0; t0 < T; t0 += TG) {
    if (t0 > 0) __syncthreads();  // the last group has been read
#pragma unroll
    for (int t = 0; t < TG; ++t)
      *reinterpret_cast<v4f*>(&part[wave][t][r][4 * q]) = acc[(t0 + t) / MF][(t0 + t) % MF];
    __syncthreads();
    const int t = threadIdx.x >> 6, rr = (threadIdx.x >> 2) & 15, c = 4 * (threadIdx.x & 3);
    if (t >= TG) continue;
    const int m = 16 * ((t0 + t) % MF) + rr, n = n0 + 16 * ((t0 + t) / MF) + c;
    if (m >= M || n >= N) continue;
    v4f v = *reinterpret_cast<const v4f*>(&part[0][t][rr][c]);
#pragma unroll
    for (int w = 1; w < W; ++w) v += *reinterpret_cast<const v4f*>(&part[w][t][rr][c]);
    u2 bb = {0, 0};
    if (bias) bb = *reinterpret_cast<const u2*>(bias + n);
    *reinterpret_cast<u2*>(y + (int64_t)m * N + n) =
        (u2){pack16x2<F16>(v[0] + lo16<F16>(bb.x), v[1] + hi16<F16>(bb.x)),
             pack16x2<F16>(v[2] + lo16<F16>(bb.y), v[3] + hi16<F16>(bb.y))};
  }
}

constexpr int64_t kFewRows = 64;  // the most that the few-rows kernel takes

struct Args {
  const uint8_t *xc, *xs, *wc, *ws;
  const uint16_t* bias;
  int m, n, k;
  uint16_t* y;
  int nx;
  hipStream_t st;
};

template <bool F16, int BM, int BN, int WM, int WN, int NS, int MINB, int NP = 0>
hipError_t launch_cfg(const Args& a) {
  constexpr int ring_bytes = NS * (BM + BN) * (128 + 8);
  constexpr int tile_bytes = BM * (BN * 2 + 16);
  constexpr int lds_bytes = ring_bytes > tile_bytes ? ring_bytes : tile_bytes;
  static_assert(lds_bytes <= 160 * 1024, "LDS");
  auto kern = gemm_mx4_kernel<BM, BN, WM, WN, NS, MINB, NP, F16>;
  // once per device (a second thread may repeat it: the call is idempotent)
  static std::atomic<uint64_t> done{0};
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return e;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (!(done.load(std::memory_order_relaxed) & bit)) {
    e = hipFuncSetAttribute(reinterpret_cast<const void*>(kern),
                            hipFuncAttributeMaxDynamicSharedMemorySize, lds_bytes);
    if (e != hipSuccess) return e;
    done.fetch_or(bit, std::memory_order_relaxed);
  }
  const int tiles_m = (a.m + BM - 1) / BM, tiles_n = (a.n + BN - 1) / BN;
  hipLaunchKernelGGL(kern, dim3(tiles_m * tiles_n), dim3(64 * (WM * WN + NP)), lds_bytes, a.st,
                     a.xc, a.xs, a.wc, a.ws, a.bias, a.m, a.n, a.k, tiles_m, tiles_n, a.nx, a.y);
  return hipGetLastError();
}

template <bool F16, int MF, int NF>
hipError_t launch_rows(const Args& a) {
  gemm_mx4_rows_kernel<MF, NF, F16>
      <<<dim3((a.n + 16 * NF - 1) / (16 * NF)), dim3(64 * kRowWaves), 0, a.st>>>(
          a.xc, a.xs, a.wc, a.ws, a.bias, a.m, a.n, a.k, a.y);
  return hipGetLastError();
}

// groups of 16 rows of the few-rows kernel
int row_groups(int64_t m) { return m <= 16 ? 1 : (m <= 32 ? 2 : 4); }

// The few-rows kernel's bytes through the busiest of `cus` CUs, in rows of K: a
// block streams its 16 nf rows of the weight and all of x. *nf: the columns per
// block, in groups of 16, of the least.
int64_t rows_cost(int64_t m, int64_t n, int64_t cus, int* nf) {
  int64_t best = INT64_MAX;
  for (int f = 1; f <= 4; f *= 2) {
    const int64_t blocks = (n + 16 * f - 1) / (16 * f);
    const int64_t cost = (blocks + cus - 1) / cus * (16 * f + m);
    if (cost < best) {
      best = cost;
      *nf = f;
    }
  }
  return best;
}

// The tiled kernel's tiles by the number that names them, and the cost of a round
// of them over the CUs (per_cu to a CU): `start` (first copies, epilogue) and
// `step` for each 256 of K; a last round that leaves one to a CU is cheaper (start1,
// step1). The costs are weights, in us by their scale, fitted so that they rank the
// tiles of a shape; a launch takes some us more than their sum (333 x 9216 x 4096:
// 10.0 by the weights, 12.8 measured).
struct Tile {
  int tile, bm, bn, waves, per_cu;
  double start, step, start1, step1;
};
constexpr Tile kTiles[] = {
    {384, 384, 192, 8, 1, 6.7, 1.24, 6.7, 1.24}, {256, 256, 256, 8, 1, 5.1, 1.14, 5.1, 1.14},
    {192, 192, 192, 8, 1, 5.2, 0.65, 5.2, 0.65}, {160, 128, 192, 8, 1, 2.75, 0.67, 2.75, 0.67},
    {128, 128, 128, 8, 2, 2.3, 0.85, 2.3, 0.48}, {96, 64, 128, 8, 2, 2.0, 0.57, 1.35, 0.38},
    {64, 64, 64, 8, 2, 4.1, 0.40, 1.0, 0.30},   {40, 64, 32, 4, 2, 2.0, 0.34, 1.0, 0.28}};

// The tile of least cost, and that cost. Measured on 620 shapes
// with weights in the last-level cache (m 70 to 20000, n 512 to 14400, k 512 to
// 14400): 0.3% behind each shape's best tile on average, 11% at most; with weights
// from memory 0.4% and 34% (140 x 5504 x 12256, just more 64 tiles than CUs). The
// small tiles earn their places where a few big ones leave CUs idle, best / next
// best of the others: 64 x 32 tiles 64 x 5120 x 13824 12.8 / 14.1 us (weights from
// memory 16.1 / 19.7), 64 x 128 tiles 256 x 5120 x 13824 19.9 / 23.6, 128 tiles
// with one to a CU 512 x 5120 x 13824 26.8 / 30.3, with two 2048 x 9216 x 768 19.3 /
// 21.5, 128 x 192 tiles 1024 x 5120 x 5120 20.2 / 22.2; 384 x 192 tiles 4608 x 3840 x
// 3840 41.7 / 46.4. Bits do not depend on the tile.
double tile_us(int64_t m, int64_t n, int64_t k, int cus, int* tile) {
  const int64_t c = cus > 0 ? cus : 1;
  const double steps = (double)((k + kMx4Tile - 1) / kMx4Tile);
  double best = 1e300;
  for (const Tile& t : kTiles) {
    const int64_t tiles = ((m + t.bm - 1) / t.bm) * ((n + t.bn - 1) / t.bn);
    if (tiles * t.waves > kMaxLaunchWaves) continue;
    const int64_t full = tiles / (c * t.per_cu), rest = tiles % (c * t.per_cu);
    double us = (double)full * (t.start + t.step * steps);
    if (rest > 0) us += rest <= c ? t.start1 + t.step1 * steps : t.start + t.step * steps;
    if (us < best) {
      best = us;
      *tile = t.tile;
    }
  }
  return best;
}

// Whether the few-rows kernel takes m rows: 3 us + 22 KB per us through a CU
// against the tiles' cost and 4 us or, with long weights, 4.2 TB/s of their bytes
// (fitted together: the 4 us stand for what the tiles' weights leave out).
// Measured, few rows / tiles, weights from memory: 13824 x 5120 with 8, 16, 32, 64
// rows 9.5, 10.0, 11.9, 22.5 / 9.6, 9.7, 10.2, 11.7 us; 5120 x 13824 11.6, 13.0, 17.5,
// 24.7 / 15.8, 15.6, 15.6, 16.1; over 302 shapes of up to 256 rows 0.4% behind the best
// kernel on average, over 221 with weights in the last-level cache 0.3%. The two
// add in different orders, so the choice goes by the shape alone and not by the
// device's CUs.
bool few_rows(int64_t m, int64_t n, int64_t k) {
  if (m > kFewRows) return false;
  constexpr int cus = 256;
  int nf, tile;
  const double rows_us = 3.0 + (double)rows_cost(m, n, cus, &nf) * (double)(k / 2) / 22e3;
  const double weight_us = (double)n * (double)k * (17.0 / 32) / 4.2e6;
  return rows_us < fmax(4.0 + tile_us(m, n, k, cus, &tile), weight_us);
}

template <bool F16, int MF>
hipError_t launch_rows_n(int nf, const Args& a) {
  if (nf == 4) return launch_rows<F16, MF, 4>(a);
  if (nf == 2) return launch_rows<F16, MF, 2>(a);
  return launch_rows<F16, MF, 1>(a);
}

template <bool F16>
hipError_t launch_tile(const LaunchPlan& p, int tile, const Args& a) {
  switch (tile) {
    case 16:
      switch (row_groups(a.m)) {
        case 1: return launch_rows_n<F16, 1>(p.tile_n / 16, a);
        case 2: return launch_rows_n<F16, 2>(p.tile_n / 16, a);
        default: return launch_rows_n<F16, 4>(p.tile_n / 16, a);
      }
    case 40: return launch_cfg<F16, 64, 32, 2, 1, 4, 2, 2>(a);
    case 64: return launch_cfg<F16, 64, 64, 2, 2, 4, 2, 4>(a);
    case 96: return launch_cfg<F16, 64, 128, 2, 2, 3, 2, 4>(a);
    case 128:  // one tile to a CU with a longer ring, or two
      if (p.grid <= compute_units()) return launch_cfg<F16, 128, 128, 2, 2, 3, 1, 4>(a);
      return launch_cfg<F16, 128, 128, 2, 2, 2, 2, 4>(a);
    case 160: return launch_cfg<F16, 128, 192, 2, 2, 3, 1, 4>(a);
    case 192: return launch_cfg<F16, 192, 192, 2, 2, 3, 1, 4>(a);
    case 384: return launch_cfg<F16, 384, 192, 4, 2, 2, 1>(a);
    default: return launch_cfg<F16, 256, 256, 2, 4, 2, 1>(a);
  }
}

}  // namespace

bool mx4_gemm_grid_fits(int64_t m, int64_t n, int tile) {
  if (tile == 16) return n / 16 * kRowWaves <= kMaxLaunchWaves;
  for (const Tile& t : kTiles)
    if (t.tile == tile &&
        ((m + t.bm - 1) / t.bm) * ((n + t.bn - 1) / t.bn) * t.waves <= kMaxLaunchWaves)
      return true;
  return false;
}

int mx4_gemm_tile(int64_t m, int64_t n, int64_t k, int64_t call_rows, int cus) {
  if (few_rows(call_rows, n, k)) return 16;
  int tile = 0;
  tile_us(m, n, k, cus, &tile);
  return tile;
}

LaunchPlan plan_mx4_gemm(int64_t m, int64_t n, int64_t k, int tile, int cus) {
  LaunchPlan p;
  if (tile == 0) tile = mx4_gemm_tile(m, n, k, m, cus);
  if (tile == 16) {
    int nf = 1;
    rows_cost(m, n, cus > 0 ? cus : 1, &nf);
    p.tile_m = 16;
    p.tile_n = 16 * nf;
    p.block = 64 * kRowWaves;
    p.grid = (n + p.tile_n - 1) / p.tile_n;
  } else {
    for (const Tile& t : kTiles) {
      if (t.tile != tile) continue;
      p.tile_m = t.bm;
      p.tile_n = t.bn;
      p.block = t.waves * 64;
    }
    p.grid = ((m + p.tile_m - 1) / p.tile_m) * ((n + p.tile_n - 1) / p.tile_n);
    p.xcds = xcd_count(cus);
  }
  p.passes = 1;
  return p;
}

hipError_t launch_mx4_gemm(const uint8_t* xc, const uint8_t* xs, const uint8_t* wc,
                           const uint8_t* ws, const uint16_t* bias, int64_t m, int64_t n,
                           int64_t k, uint16_t* y, int tile, DType dt, hipStream_t st) {
  if (m == 0) return hipSuccess;
  if (tile == 0) tile = mx4_gemm_tile(m, n, k, m, compute_units());
  const LaunchPlan p = plan_mx4_gemm(m, n, k, tile, compute_units());
  const Args a = {xc, xs, wc, ws, bias, (int)m, (int)n, (int)k, y, p.xcds, st};
  return dt == DType::kF16 ? launch_tile<true>(p, tile, a) : launch_tile<false>(p, tile, a);
}

}  // namespace convrot
