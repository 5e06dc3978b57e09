// C ABI of rotary tables, norms of queries and keys, and attention: argument
// checks. Every check runs before any HIP call.

#include <cmath>

#include "api_common.h"
#include "attention.h"

using namespace convrot;

namespace {

constexpr int kMaxHeadDim = 256;
constexpr int64_t kMaxStride = (int64_t)1 << 40;     // elements
constexpr int64_t kMaxKeyStride = (int64_t)1 << 22;  // offsets inside a tile of keys take 32 bits

// tokens x heads x d elements of `size` bytes, a token `stride` and a head
// `head_stride` elements from the next.
struct Box {
  const void* p;
  int64_t tokens, heads, d, stride, head_stride;
  int size;
  uint64_t at() const { return (uint64_t)(uintptr_t)p; }
  bool empty() const { return !p || tokens == 0 || heads == 0; }
  // bytes from the first element to behind the last
  uint64_t extent() const {
    return (uint64_t)(((tokens - 1) * stride + (heads - 1) * head_stride + d) * size);
  }
  // no two of its elements share a place: heads inside a token's stride or tokens inside a head's
  bool apart() const {
    const bool by_token = (heads == 1 || head_stride >= d) &&
                          (tokens == 1 || stride >= (heads - 1) * head_stride + d);
    const bool by_head = (tokens == 1 || stride >= d) &&
                         (heads == 1 || head_stride >= (tokens - 1) * stride + d);
    return by_token || by_head;
  }
  Box turned() const { return {p, heads, tokens, d, head_stride, stride, size}; }
  bool same(const Box& o) const {
    return p == o.p && stride == o.stride && head_stride == o.head_stride && heads == o.heads;
  }
};

// Whether [a, a + na) and [b, b + nb) meet, both repeated every `period` bytes.
bool meet(uint64_t a, uint64_t na, uint64_t b, uint64_t nb, uint64_t period) {
  if (na > period || nb > period) return true;
  const uint64_t gap = (b % period + period - a % period) % period;  // from a up to b
  return gap < na || period - gap < nb;
}

// Whether two boxes may share memory, by their places within a token's stride and a head's.
bool clash_by_token(const Box& a, const Box& b) {
  if (a.empty() || b.empty()) return false;
  if (a.at() + a.extent() <= b.at() || b.at() + b.extent() <= a.at()) return false;
  const uint64_t size = a.size;
  if (a.size != b.size) return true;
  if (a.tokens > 1 || b.tokens > 1) {
    if (a.stride != b.stride || a.stride <= 0) return true;
    const uint64_t wide_a = ((a.heads - 1) * a.head_stride + a.d) * size;
    const uint64_t wide_b = ((b.heads - 1) * b.head_stride + b.d) * size;
    if (!meet(a.at(), wide_a, b.at(), wide_b, (uint64_t)a.stride * size)) return false;
    if (a.head_stride <= 0 || a.stride % a.head_stride) return true;
  }
  if (a.head_stride != b.head_stride || a.head_stride <= 0) return true;
  return meet(a.at(), (uint64_t)a.d * size, b.at(), (uint64_t)b.d * size,
              (uint64_t)a.head_stride * size);
}

// Column ranges of one wider tensor do not clash, nor do interleaved heads, although the
// memory they span does; the same with heads outside of tokens.
bool clash(const Box& a, const Box& b) {
  return clash_by_token(a, b) && clash_by_token(a.turned(), b.turned());
}

// Strides of a tensor whose rows are read or written 16 bytes at a time.
convrot_status check_strides(const char* fn, const char* name, int64_t stride, int64_t head_stride,
                             int64_t tokens, int64_t heads, int64_t most) {
  if (stride < 0 || head_stride < 0 || stride > most || head_stride > kMaxStride)
    return fail(CONVROT_E_INVALID_ARG, "%s: strides of %s: %lld, %lld", fn, name,
                (long long)stride, (long long)head_stride);
  if (tokens > 1 && stride > ((int64_t)1 << 60) / tokens)
    return fail(CONVROT_E_INVALID_ARG, "%s: %s spans too much memory", fn, name);
  if (heads > 1 && head_stride > ((int64_t)1 << 60) / heads)
    return fail(CONVROT_E_INVALID_ARG, "%s: %s spans too much memory", fn, name);
  if (stride % 8 || head_stride % 8)
    return fail(CONVROT_E_MISALIGNED, "%s: strides of %s are not multiples of 8: %lld, %lld", fn,
                name, (long long)stride, (long long)head_stride);
  return CONVROT_OK;
}

// Everything about a call of the attention but its pointers' places.
convrot_status check_attention(const char* fn, const convrot_attention_args& a, DType* dt) {
  if (!dtype_of(a.dtype, dt)) return fail(CONVROT_E_INVALID_ARG, "%s: dtype=%d", fn, (int)a.dtype);
  if (a.q_tokens < 0 || a.k_tokens < 0 || a.batch < 1 || a.q_heads < 1 || a.k_heads < 1 || a.d < 1)
    return fail(CONVROT_E_INVALID_ARG,
                "%s: bad dims q_tokens=%lld k_tokens=%lld batch=%lld heads=%d, %d d=%d", fn,
                (long long)a.q_tokens, (long long)a.k_tokens, (long long)a.batch, a.q_heads,
                a.k_heads, a.d);
  if (a.q_heads % a.k_heads)
    return fail(CONVROT_E_UNSUPPORTED_SHAPE, "%s: %d query heads do not divide into %d groups", fn,
                a.q_heads, a.k_heads);
  if (a.d % 8 || a.d > kMaxHeadDim)
    return fail(CONVROT_E_UNSUPPORTED_SHAPE, "%s: need d %% 8 == 0, d <= %d (d=%d)", fn,
                kMaxHeadDim, a.d);
  // rows (query, head of a group) of a sequence and keys are counted in 32 bits
  const int64_t rows = a.q_tokens * (a.q_heads / a.k_heads);
  if (a.q_tokens >= kMaxDim || a.k_tokens >= kMaxDim - 256 || rows >= kMaxDim - 1024 ||
      a.batch >= ((int64_t)1 << 24))
    return fail(CONVROT_E_UNSUPPORTED_SHAPE, "%s: too large (q_tokens=%lld k_tokens=%lld "
                "batch=%lld)", fn, (long long)a.q_tokens, (long long)a.k_tokens,
                (long long)a.batch);
  if ((!a.q_offsets && a.q_tokens % a.batch) || (!a.k_offsets && a.k_tokens % a.batch))
    return fail(CONVROT_E_INVALID_ARG, "%s: tokens without offsets do not divide into %lld "
                "sequences", fn, (long long)a.batch);
  if (a.tile != 0 && a.tile != 32 && a.tile != 128 && !(a.tile == 256 && a.d > 64 && a.d <= 128))
    return fail(CONVROT_E_INVALID_ARG, "%s: tile=%d not supported (d=%d)", fn, a.tile, a.d);
  if (!(a.scale > 0.0f) || a.scale > 2.0e38f)  // scale log2 e is finite
    return fail(CONVROT_E_INVALID_ARG, "%s: scale=%g", fn, (double)a.scale);
  return CONVROT_OK;
}

AttentionArgs attention_args(const convrot_attention_args& a) {
  AttentionArgs n = {};
  n.q = static_cast<const uint16_t*>(a.q);
  n.k = static_cast<const uint16_t*>(a.k);
  n.v = static_cast<const uint16_t*>(a.v);
  n.out = static_cast<uint16_t*>(a.out);
  n.lse = a.lse;
  n.q_stride = a.q_stride;
  n.q_head_stride = a.q_head_stride;
  n.k_stride = a.k_stride;
  n.k_head_stride = a.k_head_stride;
  n.v_stride = a.v_stride;
  n.v_head_stride = a.v_head_stride;
  n.out_stride = a.out_stride;
  n.out_head_stride = a.out_head_stride;
  n.q_offsets = a.q_offsets;
  n.k_offsets = a.k_offsets;
  n.k_lens = a.k_lens;
  n.q_tokens = a.q_tokens;
  n.k_tokens = a.k_tokens;
  n.batch = (int)a.batch;
  n.q_heads = a.q_heads;
  n.k_heads = a.k_heads;
  n.d = a.d;
  n.causal = a.causal != 0;
  n.scale = a.scale;
  n.tile = a.tile;
  n.splits = 1;
  return n;
}

}  // namespace

extern "C" {

convrot_status convrot_rope_table(const void* positions, convrot_position_type type,
                                  int64_t token_stride, int64_t axis_stride, int64_t tokens,
                                  int axes, const int32_t* dims, double theta, int shared,
                                  float* table, void* stream) {
  const char* fn = "convrot_rope_table";
  if (type != CONVROT_POSITION_I32 && type != CONVROT_POSITION_I64 && type != CONVROT_POSITION_F32)
    return fail(CONVROT_E_INVALID_ARG, "%s: type=%d", fn, (int)type);
  if (tokens < 0 || axes < 1 || axes > kMaxRopeAxes || !dims)
    return fail(CONVROT_E_INVALID_ARG, "%s: tokens=%lld axes=%d", fn, (long long)tokens, axes);
  if (!(theta > 0.0) || !std::isfinite(theta))
    return fail(CONVROT_E_INVALID_ARG, "%s: theta=%g", fn, theta);
  RopeTableArgs a = {};
  for (int i = 0; i < axes; ++i) {
    if (dims[i] < 2 || dims[i] % 2 || dims[i] > 2 * kMaxRopePairs)
      return fail(CONVROT_E_UNSUPPORTED_SHAPE, "%s: axis %d has %d elements", fn, i, dims[i]);
    a.first[i + 1] = a.first[i] + dims[i] / 2;
  }
  a.pairs = a.first[axes];
  if (a.pairs > kMaxRopePairs || tokens > ((int64_t)1 << 28))
    return fail(CONVROT_E_UNSUPPORTED_SHAPE, "%s: %d pairs (at most %d), %lld tokens", fn, a.pairs,
                kMaxRopePairs, (long long)tokens);
  if (token_stride < 0 || axis_stride < 0 || token_stride > kMaxStride || axis_stride > kMaxStride)
    return fail(CONVROT_E_INVALID_ARG, "%s: strides %lld, %lld", fn, (long long)token_stride,
                (long long)axis_stride);
  if (tokens == 0) return ok();
  if (!positions || !table) return fail(CONVROT_E_INVALID_ARG, "%s: null pointer", fn);
  const int size = type == CONVROT_POSITION_I64 ? 8 : 4;
  if (!aligned(positions, size) || !aligned(table, 16))
    return fail(CONVROT_E_MISALIGNED, "%s: misaligned pointer", fn);
  const size_t np =
      (size_t)((tokens - 1) * token_stride + (axes - 1) * axis_stride + 1) * (size_t)size;
  if (overlap(positions, np, table, (size_t)tokens * a.pairs * 8))
    return fail(CONVROT_E_INVALID_ARG, "%s: overlapping buffers", fn);
  a.positions = positions;
  a.token_stride = token_stride;
  a.axis_stride = axis_stride;
  a.tokens = tokens;
  a.axes = axes;
  a.log2_theta = std::log2(theta);
  a.shared = shared != 0;
  a.table = table;
  return hip_status(launch_rope_table(a, (PosType)type, (hipStream_t)stream), fn);
}

convrot_status convrot_qk_norm_rope(const convrot_qk_args* args, void* stream) {
  const char* fn = "convrot_qk_norm_rope";
  if (!args) return fail(CONVROT_E_INVALID_ARG, "%s: null arguments", fn);
  const convrot_qk_args& a = *args;
  DType dt;
  if (!dtype_of(a.dtype, &dt)) return fail(CONVROT_E_INVALID_ARG, "%s: dtype=%d", fn, (int)a.dtype);
  if (a.norm != CONVROT_NORM_NONE && a.norm != CONVROT_NORM_RMS && a.norm != CONVROT_NORM_LAYER)
    return fail(CONVROT_E_INVALID_ARG, "%s: norm=%d", fn, (int)a.norm);
  if (!(a.eps >= 0.0f) || a.eps > 3.0e38f)
    return fail(CONVROT_E_INVALID_ARG, "%s: eps=%g", fn, (double)a.eps);
  if (a.tokens < 0 || a.q_heads < 1 || a.k_heads < 0 || a.d < 1 || a.pairs < 0)
    return fail(CONVROT_E_INVALID_ARG, "%s: bad dims tokens=%lld heads=%d, %d d=%d pairs=%d", fn,
                (long long)a.tokens, a.q_heads, a.k_heads, a.d, a.pairs);
  if (a.d % 8 || a.d > kMaxHeadDim || a.q_heads > 65536 || a.k_heads > 65536)
    return fail(CONVROT_E_UNSUPPORTED_SHAPE,
                "%s: need d %% 8 == 0, d <= %d, at most 65536 heads (d=%d heads=%d, %d)", fn,
                kMaxHeadDim, a.d, a.q_heads, a.k_heads);
  if (2 * (int64_t)a.pairs > a.d || a.pairs % (a.halves ? 8 : 4))
    return fail(CONVROT_E_UNSUPPORTED_SHAPE, "%s: need 2 pairs <= d, pairs %% %d == 0 (pairs=%d)",
                fn, a.halves ? 8 : 4, a.pairs);
  const bool row = a.row != 0 && a.norm != CONVROT_NORM_NONE;
  if (row && (!heads_row_fits(a.q_heads, a.d) || !heads_row_fits(a.k_heads, a.d)))
    return fail(CONVROT_E_UNSUPPORTED_SHAPE, "%s: %d, %d heads of %d are too long a row", fn,
                a.q_heads, a.k_heads, a.d);
  if (a.norm == CONVROT_NORM_NONE && (a.q_weight || a.k_weight))
    return fail(CONVROT_E_INVALID_ARG, "%s: a weight without a norm", fn);
  if (a.pairs > 0 && (a.table_rows < 1 || a.tokens % a.table_rows))
    return fail(CONVROT_E_INVALID_ARG, "%s: a table of %lld rows for %lld tokens", fn,
                (long long)a.table_rows, (long long)a.tokens);
  if (a.tokens >= kMaxDim)
    return fail(CONVROT_E_UNSUPPORTED_SHAPE, "%s: tokens=%lld", fn, (long long)a.tokens);
  HeadsArgs n = {};
  const struct {
    const char* name;
    const void *in, *weight;
    void* out;
    int64_t stride, head_stride, out_stride, out_head_stride;
    int heads;
  } side[] = {{"q", a.q, a.q_weight, a.q_out, a.q_stride, a.q_head_stride, a.q_out_stride,
               a.q_out_head_stride, a.q_heads},
              {"k", a.k, a.k_weight, a.k_out, a.k_stride, a.k_head_stride, a.k_out_stride,
               a.k_out_head_stride, a.k_heads}};
  Box in[2], out[2];
  for (int i = 0; i < 2; ++i) {
    const auto& s = side[i];
    HeadsTensor& t = n.t[i];
    in[i] = {s.in, a.tokens, s.heads, a.d, s.stride, s.head_stride, 2};
    out[i] = {s.out, a.tokens, s.heads, a.d, s.out_stride, s.out_head_stride, 2};
    if (s.heads == 0) continue;
    if (convrot_status e = check_strides(fn, s.name, s.stride, s.head_stride, a.tokens, s.heads,
                                         kMaxStride))
      return e;
    if (convrot_status e = check_strides(fn, s.name, s.out_stride, s.out_head_stride, a.tokens,
                                         s.heads, kMaxStride))
      return e;
    if (a.tokens > 0 && !out[i].apart())
      return fail(CONVROT_E_INVALID_ARG, "%s: %s_out overlaps itself", fn, s.name);
    t.in = static_cast<const uint16_t*>(s.in);
    t.out = static_cast<uint16_t*>(s.out);
    t.weight = static_cast<const uint16_t*>(s.weight);
    t.in_stride = s.stride;
    t.in_head_stride = s.head_stride;
    t.out_stride = s.out_stride;
    t.out_head_stride = s.out_head_stride;
    t.heads = s.heads;
  }
  n.table = a.pairs ? a.table : nullptr;
  n.tokens = a.tokens;
  n.table_rows = a.table_rows;
  n.d = a.d;
  n.pairs = a.pairs;
  n.norm = (NormKind)a.norm;
  n.row = row;
  n.eps = a.eps;
  if (!heads_grid_fits(n))
    return fail(CONVROT_E_UNSUPPORTED_SHAPE, "%s: too many tokens (%lld)", fn,
                (long long)a.tokens);
  if (a.tokens == 0) return ok();
  if (a.pairs && !a.table) return fail(CONVROT_E_INVALID_ARG, "%s: null pointer", fn);
  if (!aligned(a.table, 16)) return fail(CONVROT_E_MISALIGNED, "%s: misaligned pointer", fn);
  for (const auto& s : side) {
    if (s.heads == 0) continue;
    if (!s.in || !s.out) return fail(CONVROT_E_INVALID_ARG, "%s: null pointer", fn);
    if (!aligned(s.in, 16) || !aligned(s.out, 16) || !aligned(s.weight, 16))
      return fail(CONVROT_E_MISALIGNED, "%s: misaligned pointer", fn);
  }
  const size_t ntable = a.pairs ? (size_t)a.table_rows * a.pairs * 8 : 0;
  for (int i = 0; i < 2; ++i) {
    if (out[i].empty()) continue;
    bool bad = clash(out[i], out[1 - i]) && i == 0;
    for (int j = 0; j < 2; ++j)  // a tensor may be updated in place
      bad |= !(i == j && out[i].same(in[i])) && clash(out[i], in[j]);
    bad |= overlap(out[i].p, out[i].extent(), n.table, ntable);
    for (const auto& s : side)
      bad |= overlap(out[i].p, out[i].extent(), s.weight,
                     (size_t)a.d * 2 * (row ? s.heads : 1));
    if (bad) return fail(CONVROT_E_INVALID_ARG, "%s: overlapping buffers", fn);
  }
  return hip_status(launch_qk_norm_rope(n, a.halves != 0, dt, (hipStream_t)stream), fn);
}

size_t convrot_attention_workspace_size(const convrot_attention_args* args) {
  DType dt;
  if (!args || check_attention("convrot_attention_workspace_size", *args, &dt)) return 0;
  const AttentionArgs n = attention_args(*args);
  return attention_workspace(n, plan_attention(n, SIZE_MAX));
}

convrot_status convrot_attention(const convrot_attention_args* args, void* workspace,
                                 size_t workspace_bytes, void* stream) {
  const char* fn = "convrot_attention";
  if (!args) return fail(CONVROT_E_INVALID_ARG, "%s: null arguments", fn);
  const convrot_attention_args& a = *args;
  DType dt;
  if (convrot_status s = check_attention(fn, a, &dt)) return s;
  if (convrot_status s = check_strides(fn, "q", a.q_stride, a.q_head_stride, a.q_tokens, a.q_heads,
                                       kMaxStride))
    return s;
  if (convrot_status s = check_strides(fn, "k", a.k_stride, a.k_head_stride, a.k_tokens, a.k_heads,
                                       kMaxKeyStride))
    return s;
  if (convrot_status s = check_strides(fn, "v", a.v_stride, a.v_head_stride, a.k_tokens, a.k_heads,
                                       kMaxKeyStride))
    return s;
  if (convrot_status s = check_strides(fn, "out", a.out_stride, a.out_head_stride, a.q_tokens,
                                       a.q_heads, kMaxStride))
    return s;
  AttentionArgs n = attention_args(a);
  if (plan_attention(n, SIZE_MAX).grid >= ((int64_t)1 << 23))
    return fail(CONVROT_E_UNSUPPORTED_SHAPE, "%s: too many tiles (q_tokens=%lld heads=%d)", fn,
                (long long)a.q_tokens, a.q_heads);
  if (a.q_tokens == 0) return ok();
  const bool keys = a.k_tokens > 0;
  if (!a.q || !a.out || (keys && (!a.k || !a.v)))
    return fail(CONVROT_E_INVALID_ARG, "%s: null pointer", fn);
  if (!aligned(a.q, 16) || !aligned(a.k, 16) || !aligned(a.v, 16) || !aligned(a.out, 16) ||
      !aligned(a.lse, 4) || !aligned(a.q_offsets, 4) || !aligned(a.k_offsets, 4) ||
      !aligned(a.k_lens, 4) || !aligned(workspace, 256))
    return fail(CONVROT_E_MISALIGNED, "%s: misaligned pointer", fn);
  const Box q = {a.q, a.q_tokens, a.q_heads, a.d, a.q_stride, a.q_head_stride, 2};
  const Box k = {a.k, a.k_tokens, a.k_heads, a.d, a.k_stride, a.k_head_stride, 2};
  const Box v = {a.v, a.k_tokens, a.k_heads, a.d, a.v_stride, a.v_head_stride, 2};
  const Box out = {a.out, a.q_tokens, a.q_heads, a.d, a.out_stride, a.out_head_stride, 2};
  if (!out.apart()) return fail(CONVROT_E_INVALID_ARG, "%s: out overlaps itself", fn);
  if (!workspace) workspace_bytes = 0;
  const size_t noff = (size_t)(a.batch + 1) * 4, nlse = (size_t)(a.q_tokens * a.q_heads) * 4;
  const struct {
    const void* p;
    size_t bytes;
  } flat[] = {{a.lse, nlse}, {workspace, workspace_bytes}};
  const struct {
    const void* p;
    size_t bytes;
  } ints[] = {{a.q_offsets, noff}, {a.k_offsets, noff}, {a.k_lens, noff - 4}};
  bool bad = clash(out, q) || clash(out, k) || clash(out, v);
  for (const auto& i : ints) bad |= overlap(out.p, out.extent(), i.p, i.bytes);
  for (const auto& f : flat) {
    for (const Box* b : {&q, &k, &v, &out})
      if (!b->empty()) bad |= overlap(f.p, f.bytes, b->p, b->extent());
    for (const auto& i : ints) bad |= overlap(f.p, f.bytes, i.p, i.bytes);
  }
  bad |= overlap(a.lse, nlse, workspace, workspace_bytes);
  if (bad) return fail(CONVROT_E_INVALID_ARG, "%s: overlapping buffers", fn);
  const AttentionPlan p = plan_attention(n, workspace_bytes);
  attention_use(&n, p, workspace);
  return hip_status(launch_attention(n, p, dt, (hipStream_t)stream), fn);
}

}  // extern "C"
