// C ABI entry points between the projections of an attention block: argument
// validation and kernel-path dispatch (plain host C++, no device code).  As
// for the matmuls, everything is checked before anything is enqueued, and a
// shape or an alignment outside a fast kernel's predicate takes the generic
// kernel.

#include <stdint.h>

#include <algorithm>

#include "../../include/fp4w.h"
#include "arg_checks.h"
#include "launch.h"

namespace {

using fp4w::Act;
using fp4w::aligned;
using fp4w::AttentionArgs;
using fp4w::KvAppendArgs;
using fp4w::mul_ok;
using fp4w::overlaps;
using fp4w::QkNormRopeArgs;
using fp4w::RopeArgs;
using fp4w::SeqArgs;

constexpr int64_t kMax32 = int64_t(1) << 31;

bool dtype_ok(int dtype) { return dtype == FP4W_F16 || dtype == FP4W_BF16; }

// [M, heads * D] values of T with a stride from row to row.
struct Rows {
  const void* p;
  int64_t stride, width, M;
  int64_t bytes() const { return width <= 0 || M <= 0 ? 0 : ((M - 1) * stride + width) * 2; }
};

bool rows_ok(const Rows& r) {
  if (r.width == 0) return true;
  return r.stride >= r.width && r.stride <= fp4w::kMaxElems && mul_ok(r.stride, r.M);
}

// Two sets of rows may lie side by side in one larger row.
bool rows_overlap(const Rows& a, const Rows& b) {
  if (!overlaps(a.p, a.bytes(), b.p, b.bytes())) return false;
  if (a.stride != b.stride || a.M != b.M) return true;
  const int64_t pitch = a.stride * 2;
  int64_t d = (static_cast<const char*>(b.p) - static_cast<const char*>(a.p)) % pitch;
  if (d < 0) d += pitch;
  return d < a.width * 2 || pitch - d < b.width * 2;
}

bool same_rows(const Rows& a, const Rows& b) { return a.p == b.p && a.stride == b.stride; }

int check_heads(int64_t M, int64_t Hq, int64_t Hk, int64_t D) {
  if (M < 0 || Hq < 0 || Hk < 0 || D < 0 || D > FP8W_MAX_HEAD_SIZE) return FP4W_ERR_SHAPE;
  if (M >= kMax32 || Hq >= (1 << 20) || Hk >= (1 << 20)) return FP4W_ERR_SHAPE;
  return FP4W_OK;
}

int check_rope(const RopeArgs& r, int64_t D) {
  if ((r.cos == nullptr) != (r.sin == nullptr)) return FP4W_ERR_SHAPE;
  if (r.cos == nullptr) return FP4W_OK;
  if (r.rows < 1 || r.dims < 0 || r.dims % 2 != 0 || r.dims > D || !mul_ok(r.rows, r.dims + 1)) return FP4W_ERR_SHAPE;
  return FP4W_OK;
}

int check_seq(const SeqArgs& s, int64_t M) {
  if (s.B < 0 || s.B >= kMax32 || s.max_pages < 0 || s.num_pages < 0 || s.num_pages >= kMax32) return FP4W_ERR_SHAPE;
  if (s.page_size < 1 || s.page_size >= kMax32 || s.max_pages >= kMax32 || s.max_pages * s.page_size >= kMax32) return FP4W_ERR_SHAPE;
  if (!mul_ok(s.B, s.max_pages) || (s.starts == nullptr && s.B != M)) return FP4W_ERR_SHAPE;
  return FP4W_OK;
}

// Bytes of the codes and scales of one cache, or -1.
int64_t cache_codes(const SeqArgs& s, int64_t Hk, int64_t D) {
  if (!mul_ok(s.num_pages, s.page_size) || !mul_ok(s.num_pages * s.page_size, Hk * std::max<int64_t>(D, 1))) return -1;
  return s.num_pages * s.page_size * Hk * D;
}

// Kernels made for heads of 64 and 128.
bool tiled(int64_t D) { return D == 64 || D == 128; }

constexpr int64_t kDecodeRows = 64;  // rows of a sequence and key head that the decode kernel takes

int64_t attention_bytes(int64_t M, int64_t Hq, int64_t Hk, int64_t D, int64_t B, int64_t max_new) {
  if (!tiled(D)) return 0;
  const int64_t G = Hq / Hk;
  return std::max(fp4w::attn_decode_workspace(max_new, Hk, G, D), fp4w::attn_prompt_workspace(M, G, B, Hk, D));
}

bool rope_vec(const RopeArgs& r, int64_t D) {
  const int64_t dims = r.cos ? r.dims : 0;
  return D >= 16 && (D & (D - 1)) == 0 && dims % 16 == 0 && aligned(r.q_weight, 16) && aligned(r.k_weight, 16) &&
         aligned(r.cos, 16) && aligned(r.sin, 16);
}

bool rows_vec(const Rows& r) { return r.width == 0 || (aligned(r.p, 16) && (r.stride % 8 == 0 || r.M == 1)); }

// Rows of int32 and float tables that every call reads.
bool reads_overlap(const Rows& out, const RopeArgs& r, int64_t M, int64_t D) {
  const int64_t table = r.cos ? r.rows * (r.dims / 2) * 4 : 0;
  return overlaps(out.p, out.bytes(), r.q_weight, D * 2) || overlaps(out.p, out.bytes(), r.k_weight, D * 2) ||
         overlaps(out.p, out.bytes(), r.cos, table) || overlaps(out.p, out.bytes(), r.sin, table) ||
         overlaps(out.p, out.bytes(), r.positions, M * 4);
}

}  // namespace

extern "C" {

int fp4w_qk_norm_rope(const void* q, int64_t q_stride, int64_t Hq, const void* k, int64_t k_stride, int64_t Hk,
                      int64_t M, int64_t D, const void* q_weight, const void* k_weight, float weight_offset, float eps,
                      const float* cos, const float* sin, int64_t rope_rows, int64_t rope_dims, int interleaved,
                      const int32_t* positions, void* q_out, int64_t q_out_stride, void* k_out, int64_t k_out_stride,
                      int dtype, void* stream) {
  if (!dtype_ok(dtype)) return FP4W_ERR_DTYPE;
  const RopeArgs rope{q_weight, k_weight, cos, sin, positions, rope_rows, rope_dims, interleaved != 0, weight_offset, eps};
  int st = check_heads(M, Hq, Hk, D);
  if (st == FP4W_OK) st = check_rope(rope, D);
  if (st != FP4W_OK) return st;
  if (M == 0 || D == 0 || Hq + Hk == 0) return FP4W_OK;
  const Rows qi{q, q_stride, Hq * D, M}, ki{k, k_stride, Hk * D, M}, qo{q_out, q_out_stride, Hq * D, M},
      ko{k_out, k_out_stride, Hk * D, M};
  for (const Rows& r : {qi, ki, qo, ko}) {
    if (!rows_ok(r)) return FP4W_ERR_SHAPE;
    if (r.width > 0 && r.p == nullptr) return FP4W_ERR_NULL;
  }
  if (rows_overlap(qo, ko) || (!same_rows(qo, qi) && rows_overlap(qo, qi)) || rows_overlap(qo, ki) ||
      (!same_rows(ko, ki) && rows_overlap(ko, ki)) || rows_overlap(ko, qi) || reads_overlap(qo, rope, M, D) ||
      reads_overlap(ko, rope, M, D))
    return FP4W_ERR_ALIAS;
  const bool vec = rope_vec(rope, D) && rows_vec(qi) && rows_vec(ki) && rows_vec(qo) && rows_vec(ko);
  const QkNormRopeArgs a{q, k, q_out, k_out, q_stride, k_stride, q_out_stride, k_out_stride, M, Hq, Hk, D, rope,
                         static_cast<Act>(dtype), stream};
  return fp4w::launch_qk_norm_rope(a, vec, nullptr) == 0 ? FP4W_OK : FP4W_ERR_LAUNCH;
}

int fp8w_kv_append(const void* k, int64_t k_stride, const void* v, int64_t v_stride, int64_t M, int64_t Hk, int64_t D,
                   const void* q, int64_t q_stride, int64_t Hq, const void* q_weight, const void* k_weight,
                   float weight_offset, float eps, const float* cos, const float* sin, int64_t rope_rows,
                   int64_t rope_dims, int interleaved, const int32_t* positions, void* q_out, int64_t q_out_stride,
                   const int32_t* starts, int64_t B, const int32_t* seq_lens, const int32_t* page_table,
                   int64_t max_pages, uint8_t* k_cache, uint8_t* k_scale, uint8_t* v_cache, uint8_t* v_scale,
                   int64_t num_pages, int64_t page_size, int dtype, void* stream) {
  if (!dtype_ok(dtype)) return FP4W_ERR_DTYPE;
  const RopeArgs rope{q_weight, k_weight, cos, sin, positions, rope_rows, rope_dims, interleaved != 0, weight_offset, eps};
  const SeqArgs seq{starts, seq_lens, page_table, B, max_pages, num_pages, page_size};
  int st = check_heads(M, Hq, Hk, D);
  if (st == FP4W_OK) st = check_rope(rope, D);
  if (st == FP4W_OK) st = check_seq(seq, M);
  if (st != FP4W_OK) return st;
  const int64_t codes = cache_codes(seq, Hk, D), scales = num_pages * Hk;
  if (codes < 0) return FP4W_ERR_SHAPE;
  if (M == 0 || B == 0 || D == 0 || Hq + Hk == 0) return FP4W_OK;
  const Rows ki{k, k_stride, Hk * D, M}, vi{v, v_stride, Hk * D, M}, qi{q, q_stride, Hq * D, M},
      qo{q_out, q_out_stride, Hq * D, M};
  for (const Rows& r : {ki, vi, qi, qo}) {
    if (!rows_ok(r)) return FP4W_ERR_SHAPE;
    if (r.width > 0 && r.p == nullptr) return FP4W_ERR_NULL;
  }
  if (seq_lens == nullptr || (max_pages > 0 && page_table == nullptr)) return FP4W_ERR_NULL;
  if (codes > 0 && (k_cache == nullptr || k_scale == nullptr || v_cache == nullptr || v_scale == nullptr)) return FP4W_ERR_NULL;
  // what is written: q_out and the parts of the cache
  const struct {
    const void* p;
    int64_t bytes;
  } parts[] = {{k_cache, codes}, {k_scale, scales}, {v_cache, codes}, {v_scale, scales}},
    reads[] = {{k, ki.bytes()}, {v, vi.bytes()}, {q, qi.bytes()}, {q_out, qo.bytes()}, {q_weight, D * 2}, {k_weight, D * 2},
               {cos, cos ? rope_rows * (rope_dims / 2) * 4 : 0}, {sin, cos ? rope_rows * (rope_dims / 2) * 4 : 0},
               {positions, M * 4}, {starts, (B + 1) * 4}, {seq_lens, B * 4}, {page_table, B * max_pages * 4}};
  for (int i = 0; i < 4; ++i) {
    for (const auto& r : reads)
      if (overlaps(parts[i].p, parts[i].bytes, r.p, r.bytes)) return FP4W_ERR_ALIAS;
    for (int j = 0; j < i; ++j)
      if (overlaps(parts[i].p, parts[i].bytes, parts[j].p, parts[j].bytes)) return FP4W_ERR_ALIAS;
  }
  if (Hq > 0) {
    if ((!same_rows(qo, qi) && rows_overlap(qo, qi)) || rows_overlap(qo, ki) || rows_overlap(qo, vi) ||
        reads_overlap(qo, rope, M, D) || overlaps(q_out, qo.bytes(), starts, (B + 1) * 4) ||
        overlaps(q_out, qo.bytes(), seq_lens, B * 4) || overlaps(q_out, qo.bytes(), page_table, B * max_pages * 4))
      return FP4W_ERR_ALIAS;
  }
  const bool vec = rope_vec(rope, D) && rows_vec(ki) && rows_vec(vi) && rows_vec(qi) && rows_vec(qo) && page_size % 16 == 0 &&
                   page_size * D <= 16384 && aligned(k_cache, 16) && aligned(v_cache, 16);
  const KvAppendArgs a{k, v, q, q_out, k_stride, v_stride, q_stride, q_out_stride, M, Hk, Hq, D, rope, seq,
                       k_cache, k_scale, v_cache, v_scale, static_cast<Act>(dtype), stream};
  return fp4w::launch_kv_append(a, vec) == 0 ? FP4W_OK : FP4W_ERR_LAUNCH;
}

int64_t fp8w_attention_workspace(int64_t M, int64_t Hq, int64_t Hk, int64_t D, int64_t B, int64_t max_new) {
  const int st = check_heads(M, Hq, Hk, D);
  if (st != FP4W_OK) return st;
  if (B < 0 || B >= kMax32 || max_new < 0) return FP4W_ERR_SHAPE;
  if (Hk == 0 ? Hq != 0 : Hq % Hk != 0) return FP4W_ERR_SHAPE;
  return Hk == 0 || Hq == 0 || M == 0 || B == 0 || max_new == 0 ? 0 : attention_bytes(M, Hq, Hk, D, B, max_new);
}

int fp8w_attention_ex(const void* q, int64_t q_stride, int64_t M, int64_t Hq, int64_t Hk, int64_t D,
                      const int32_t* starts, int64_t B, const int32_t* seq_lens, const int32_t* page_table,
                      int64_t max_pages, int64_t max_new, const uint8_t* k_cache, const uint8_t* k_scale,
                      const uint8_t* v_cache, const uint8_t* v_scale, int64_t num_pages, int64_t page_size, float scale,
                      int causal, int64_t window, void* workspace, int64_t workspace_bytes, void* Y, float* lse,
                      int dtype, void* stream, int path) {
  if (!dtype_ok(dtype)) return FP4W_ERR_DTYPE;
  const SeqArgs seq{starts, seq_lens, page_table, B, max_pages, num_pages, page_size};
  int st = check_seq(seq, M);
  if (st != FP4W_OK) return st;
  if (max_new < 0 || window < 0) return FP4W_ERR_SHAPE;
  if (starts == nullptr) max_new = 1;
  max_new = std::min(max_new, M);
  const int64_t need = fp8w_attention_workspace(M, Hq, Hk, D, B, max_new);
  if (need < 0) return static_cast<int>(need);
  const int64_t codes = cache_codes(seq, Hk, D);
  if (codes < 0) return FP4W_ERR_SHAPE;
  if (path != FP4W_PATH_AUTO && path != FP4W_PATH_ATTN_GENERIC && path != FP4W_PATH_ATTN_DECODE && path != FP4W_PATH_ATTN_PROMPT)
    return FP4W_ERR_PATH;
  if (M == 0 || B == 0 || Hq == 0 || D == 0 || max_new == 0) return FP4W_OK;
  const Rows qi{q, q_stride, Hq * D, M};
  if (!rows_ok(qi)) return FP4W_ERR_SHAPE;
  if (q == nullptr || Y == nullptr || seq_lens == nullptr || (max_pages > 0 && page_table == nullptr)) return FP4W_ERR_NULL;
  if (codes > 0 && (k_cache == nullptr || k_scale == nullptr || v_cache == nullptr || v_scale == nullptr)) return FP4W_ERR_NULL;
  if (need > 0) {
    if (workspace == nullptr) return FP4W_ERR_NULL;
    if (workspace_bytes < need || !aligned(workspace, 16)) return FP4W_ERR_SHAPE;
  }
  const int64_t ybytes = M * Hq * D * 2, lbytes = lse ? M * Hq * 4 : 0, scales = num_pages * Hk;
  const struct {
    const void* p;
    int64_t bytes;
  } outs[] = {{Y, ybytes}, {lse, lbytes}, {workspace, need}},
    reads[] = {{q, qi.bytes()}, {starts, (B + 1) * 4}, {seq_lens, B * 4}, {page_table, B * max_pages * 4},
               {k_cache, codes}, {k_scale, scales}, {v_cache, codes}, {v_scale, scales}};
  for (int i = 0; i < 3; ++i) {
    for (const auto& r : reads)
      if (overlaps(outs[i].p, outs[i].bytes, r.p, r.bytes)) return FP4W_ERR_ALIAS;
    for (int j = 0; j < i; ++j)
      if (overlaps(outs[i].p, outs[i].bytes, outs[j].p, outs[j].bytes)) return FP4W_ERR_ALIAS;
  }
  const bool fast = tiled(D) && page_size % 16 == 0 && rows_vec(qi) && aligned(k_cache, 16) && aligned(v_cache, 16) && aligned(Y, 16);
  // (tokens with some tiles behind them, the tiles of a launch's sequences and a
  // grid's threads are counted in 32 bits)
  const bool counted = max_pages * page_size < kMax32 - 512;
  const bool decode = fast && counted && max_new * (Hq / Hk) <= kDecodeRows && M * Hq < (1 << 25) &&
                      std::min<int64_t>(B, fp4w::kSeqsPerLaunch) * (max_pages * page_size / 64 + 2) < kMax32 / 2;
  const bool prompt = fast && counted && mul_ok(Hk, page_size) && Hk * page_size * D < kMax32 &&
                      (fp4w::attn_row_tiles_most(M, Hq / Hk, B) * Hk + 2 * fp4w::kPromptWork) * 256 < 2 * kMax32;
  if ((path == FP4W_PATH_ATTN_DECODE && !decode) || (path == FP4W_PATH_ATTN_PROMPT && !prompt)) return FP4W_ERR_PATH;
  const AttentionArgs a{q, q_stride, M, Hq, Hk, D, max_new, seq, k_cache, k_scale, v_cache, v_scale, scale, causal != 0,
                        window, workspace, Y, lse, static_cast<Act>(dtype), stream};
  int rc;
  if (decode && (path == FP4W_PATH_AUTO || path == FP4W_PATH_ATTN_DECODE))
    rc = fp4w::launch_attention_decode(a);
  else if (prompt && path != FP4W_PATH_ATTN_GENERIC)
    rc = fp4w::launch_attention_prompt(a);
  else
    rc = fp4w::launch_attention_generic(a);
  return rc == 0 ? FP4W_OK : FP4W_ERR_LAUNCH;
}

int fp8w_attention(const void* q, int64_t q_stride, int64_t M, int64_t Hq, int64_t Hk, int64_t D, const int32_t* starts,
                   int64_t B, const int32_t* seq_lens, const int32_t* page_table, int64_t max_pages, int64_t max_new,
                   const uint8_t* k_cache, const uint8_t* k_scale, const uint8_t* v_cache, const uint8_t* v_scale,
                   int64_t num_pages, int64_t page_size, float scale, int causal, int64_t window, void* workspace,
                   int64_t workspace_bytes, void* Y, float* lse, int dtype, void* stream) {
  return fp8w_attention_ex(q, q_stride, M, Hq, Hk, D, starts, B, seq_lens, page_table, max_pages, max_new, k_cache,
                           k_scale, v_cache, v_scale, num_pages, page_size, scale, causal, window, workspace,
                           workspace_bytes, Y, lse, dtype, stream, FP4W_PATH_AUTO);
}

}  // extern "C"
