// C ABI entry points around a mixture-of-experts block: argument validation
// and kernel-path dispatch (plain host C++, no device code).  As for the
// matmuls, everything is checked before anything is enqueued, and a shape or
// an alignment outside a fast kernel's predicate takes the generic kernel.

#include <stdint.h>

#include <algorithm>

#include "../../include/fp4w.h"
#include "arg_checks.h"
#include "launch.h"

namespace {

using fp4w::Act;
using fp4w::aligned;
using fp4w::BlockNormArgs;
using fp4w::ceil_div;
using fp4w::MoeArgs;
using fp4w::MoeRouteArgs;
using fp4w::mul_ok;
using fp4w::overlaps;

bool dtype_ok(int dtype) { return dtype == FP4W_F16 || dtype == FP4W_BF16; }

// M and M * topk of a call stay below it.
constexpr int64_t kMaxTokens = int64_t(1) << 31;

// A call works through its tokens in parts of equal size with at most this
// many choices: the kernels sort a part's choices in LDS, and the workspace
// does not grow beyond a part's.
constexpr int64_t kPartChoices = 4096;
int64_t part_tokens(int64_t M, int64_t topk) {
  const int64_t most = topk > 0 ? kPartChoices / topk : M;
  return M <= most ? M : ceil_div(M, ceil_div(M, most));
}

int64_t align256(int64_t bytes) { return (bytes + 255) / 256 * 256; }

// Sizes of one layer.  Returns FP4W_OK or an error status.
int check_moe(bool fp8, int64_t M, int64_t K, int64_t topk, int64_t E, int64_t I, int64_t bs) {
  if (M < 0 || K < 0 || topk < 0 || E < 0 || I < 0) return FP4W_ERR_SHAPE;
  if (bs < 1) return FP4W_ERR_BLOCK;
  if (!fp8 && (K % 2 != 0 || I % 2 != 0)) return FP4W_ERR_SHAPE;  // two E2M1 codes per byte
  if (E > FP4W_MOE_MAX_EXPERTS || topk > FP4W_MOE_MAX_TOPK) return FP4W_ERR_SHAPE;
  if (M >= kMaxTokens || M * topk >= kMaxTokens) return FP4W_ERR_SHAPE;
  // byte counts of the weights, the intermediate and the outputs below 2^63
  if (!mul_ok(4 * M, K) || !mul_ok(K, I) || !mul_ok(2 * E, K * I) || K > (int64_t(1) << 40) || I > (int64_t(1) << 40)) return FP4W_ERR_SHAPE;
  return FP4W_OK;
}

int generic_path(bool fp8) { return fp8 ? FP4W_PATH_MOE_FP8_GENERIC : FP4W_PATH_MOE_FP4_GENERIC; }

int stream_path(bool fp8) { return fp8 ? FP4W_PATH_MOE_FP8_STREAM : FP4W_PATH_MOE_FP4_STREAM; }

// The streaming kernels: whole 64-k halves of windows, FP4 blocks of 16, FP8
// blocks of whole 128-k windows, and 32-bit offsets inside A, an expert's
// matrices and the intermediate.
bool stream_ok(bool fp8, const MoeArgs& a) {
  const int64_t n = a.M * a.topk, limit = int64_t(1) << 31;
  return a.K % 64 == 0 && a.I % 64 == 0 && (fp8 ? a.block_size % 128 == 0 : a.block_size == 16) &&
         a.M * a.K * 2 < limit && n * a.I * 4 < limit && (2 * a.I + 16) * (a.K + 128) < limit && aligned(a.A, 16) &&
         aligned(a.w13, 16) && aligned(a.w2, 16) && aligned(a.s13, 4) && aligned(a.s2, 4) && aligned(a.work, 16) &&
         aligned(a.Y, 16);
}

// H (4 bytes a value), then the outputs of the single choices in FP32, once
// for each part of the sum over I.  Sized for a full part wherever there are
// tokens for one: the parts of a larger call may be smaller than the only part
// of a smaller one, and a buffer has to serve every call below its own size.
int64_t workspace_bytes(int64_t tokens, int64_t topk, int64_t K, int64_t I) {
  const int64_t n = std::min(tokens * topk, kPartChoices);
  return align256(n * I * 4) + fp4w::moe_down_splits(tokens, I) * align256(n * K * 4);
}

// The call's arguments for the tokens behind a's.
void next_part(MoeArgs& a) {
  const int64_t row = a.M * a.K * 2, n = a.M * a.topk;
  a.Y = static_cast<unsigned char*>(a.Y) + row;
  if (a.A != nullptr) a.A = static_cast<const unsigned char*>(a.A) + row;
  if (n > 0) {
    a.ids += n;
    a.weights += n;
  }
}

int run_moe(bool fp8, MoeArgs a, int64_t work_bytes, int path) {
  if (!dtype_ok(static_cast<int>(a.act))) return FP4W_ERR_DTYPE;
  if (a.activation != FP4W_ACT_SILU && a.activation != FP4W_ACT_GELU_TANH) return FP4W_ERR_DTYPE;
  const int st = check_moe(fp8, a.M, a.K, a.topk, a.E, a.I, a.block_size);
  if (st != FP4W_OK) return st;
  if (path != FP4W_PATH_AUTO && path != generic_path(fp8) && path != stream_path(fp8)) return FP4W_ERR_PATH;
  if (a.M == 0 || a.K == 0) return FP4W_OK;  // empty output
  // a block longer than either row is one block per row (and column counts cannot overflow)
  a.block_size = std::min(a.block_size, ceil_div(std::max(a.K, a.I), 128) * 128);
  if (a.Y == nullptr) return FP4W_ERR_NULL;
  const int64_t n = a.M * a.topk;
  const int64_t ybytes = a.M * a.K * 2, abytes = ybytes;
  if (n > 0 && (a.ids == nullptr || a.weights == nullptr)) return FP4W_ERR_NULL;
  const bool terms = n > 0 && a.E > 0 && a.I > 0;  // there is something to sum
  const int64_t need = terms ? workspace_bytes(a.M, a.topk, a.K, a.I) : 0;
  if (terms) {
    if (a.A == nullptr || a.w13 == nullptr || a.s13 == nullptr || a.w2 == nullptr || a.s2 == nullptr)
      return FP4W_ERR_NULL;
    if (!fp8 && (a.g13 == nullptr || a.g2 == nullptr)) return FP4W_ERR_NULL;
    if (a.work == nullptr) return FP4W_ERR_NULL;
    if (work_bytes < need) return FP4W_ERR_SHAPE;
    if (!aligned(a.work, 4)) return FP4W_ERR_SHAPE;
  }
  // Y and the workspace are written: neither may overlap an input or the other
  const int64_t per_scale = fp8 ? 4 : 1, half = fp8 ? 1 : 2;
  const struct {
    const void* p;
    int64_t bytes;
  } inputs[] = {{a.A, abytes},
                {a.ids, n * 4},
                {a.weights, n * 4},
                {a.w13, a.E * 2 * a.I * (a.K / half)},
                {a.s13, a.E * 2 * a.I * ceil_div(a.K, a.block_size) * per_scale},
                {a.g13, fp8 ? 0 : a.E * 4},
                {a.w2, a.E * a.K * (a.I / half)},
                {a.s2, a.E * a.K * ceil_div(a.I, a.block_size) * per_scale},
                {a.g2, fp8 ? 0 : a.E * 4}};
  for (const auto& in : inputs)
    if (overlaps(a.Y, ybytes, in.p, in.bytes) || overlaps(a.work, need, in.p, in.bytes)) return FP4W_ERR_ALIAS;
  if (overlaps(a.Y, ybytes, a.work, need)) return FP4W_ERR_ALIAS;
  const int64_t M = a.M, step = part_tokens(M, a.topk);
  a.M = step;  // the first part is a largest one
  const bool fast = terms && stream_ok(fp8, a);
  if (path == stream_path(fp8) && !fast) return FP4W_ERR_PATH;
  for (int64_t m = 0; m < M; m += step) {
    a.M = std::min(step, M - m);
    int rc = 1;  // 1: the streaming kernels do not take the row length
    if (fast && path != generic_path(fp8)) rc = fp8 ? fp4w::launch_moe_fp8(a) : fp4w::launch_moe_fp4(a);
    if (rc == 1 && path == stream_path(fp8)) return FP4W_ERR_PATH;
    if (rc == 1) rc = fp8 ? fp4w::launch_moe_fp8_generic(a) : fp4w::launch_moe_fp4_generic(a);
    if (rc != 0) return FP4W_ERR_LAUNCH;
    if (m + step < M) next_part(a);
  }
  return FP4W_OK;
}

}  // namespace

extern "C" {

int fp4w_block_norm(const void* x, int64_t M, int64_t K, const void* post_weight, const void* gate, int64_t gate_rows,
                    float scale, const void* residual, const void* pre_weight, float weight_offset, float eps,
                    void* residual_out, void* y, int dtype, void* stream) {
  if (!dtype_ok(dtype)) return FP4W_ERR_DTYPE;
  if (M < 0 || K < 0 || !mul_ok(M, K)) return FP4W_ERR_SHAPE;
  if (gate != nullptr && gate_rows != 1 && gate_rows != M) return FP4W_ERR_SHAPE;
  if (M == 0 || K == 0) return FP4W_OK;
  if (x == nullptr || (residual_out == nullptr && y == nullptr)) return FP4W_ERR_NULL;
  if ((y == nullptr) != (pre_weight == nullptr)) return FP4W_ERR_NULL;
  const int64_t bytes = M * K * 2, gate_bytes = gate ? gate_rows * K * 2 : 0;
  if (overlaps(residual_out, bytes, y, bytes)) return FP4W_ERR_ALIAS;
  for (void* out : {residual_out, y}) {
    if ((out != x && overlaps(out, bytes, x, bytes)) || (out != residual && overlaps(out, bytes, residual, bytes)) ||
        overlaps(out, bytes, gate, gate_bytes) || overlaps(out, bytes, post_weight, K * 2) ||
        overlaps(out, bytes, pre_weight, K * 2))
      return FP4W_ERR_ALIAS;
  }
  bool vec = K % 8 == 0;
  for (const void* p : {x, post_weight, gate, residual, pre_weight, static_cast<const void*>(residual_out),
                        static_cast<const void*>(y)})
    vec = vec && aligned(p, 16);
  const BlockNormArgs a{x, post_weight, gate, residual, pre_weight, residual_out, y, M, K, gate ? gate_rows : 1,
                        scale, weight_offset, eps, static_cast<Act>(dtype), stream};
  return fp4w::launch_block_norm(a, vec) == 0 ? FP4W_OK : FP4W_ERR_LAUNCH;
}

int fp4w_moe_route(const void* logits, int64_t M, int64_t E, int64_t topk, int score, const float* select_bias,
                   int renormalize, float scale, int32_t* ids, float* weights, int logits_dtype, void* stream) {
  if (!dtype_ok(logits_dtype) && logits_dtype != FP4W_F32) return FP4W_ERR_DTYPE;
  if (score != FP4W_SCORE_SOFTMAX && score != FP4W_SCORE_SIGMOID) return FP4W_ERR_DTYPE;
  if (M < 0 || E < 0 || topk < 0 || E > FP4W_MOE_MAX_EXPERTS || topk > FP4W_MOE_MAX_TOPK || !mul_ok(M, E) ||
      !mul_ok(M, topk))
    return FP4W_ERR_SHAPE;
  if (M == 0 || topk == 0) return FP4W_OK;
  if ((E > 0 && logits == nullptr) || ids == nullptr || weights == nullptr) return FP4W_ERR_NULL;
  const int64_t obytes = M * topk * 4, lbytes = M * E * (logits_dtype == FP4W_F32 ? 4 : 2);
  if (overlaps(ids, obytes, weights, obytes)) return FP4W_ERR_ALIAS;
  for (const void* out : {static_cast<const void*>(ids), static_cast<const void*>(weights)})
    if (overlaps(out, obytes, logits, lbytes) || overlaps(out, obytes, select_bias, E * 4)) return FP4W_ERR_ALIAS;
  const MoeRouteArgs a{logits, select_bias, ids, weights, M, E, topk, score == FP4W_SCORE_SIGMOID, renormalize != 0,
                       scale, logits_dtype, stream};
  return fp4w::launch_moe_route(a) == 0 ? FP4W_OK : FP4W_ERR_LAUNCH;
}

int64_t fp4w_moe_workspace(int64_t M, int64_t topk, int64_t K, int64_t I) {
  const int st = check_moe(true, M, K, topk, 1, I, 1);
  return st != FP4W_OK ? st : workspace_bytes(M, topk, K, I);
}

int fp4w_moe_ex(const void* A, int64_t M, int64_t K, const int32_t* ids, const float* weights, int64_t topk,
                const uint8_t* w13, const uint8_t* w13_scale, const float* w13_scale_2, const uint8_t* w2,
                const uint8_t* w2_scale, const float* w2_scale_2, int64_t E, int64_t I, int64_t block_size,
                int activation, void* workspace, int64_t workspace_bytes, void* Y, int dtype, void* stream, int path) {
  const MoeArgs a{A, ids, weights, w13, w13_scale, w13_scale_2, w2, w2_scale, w2_scale_2, workspace, Y,
                  M, K, topk, E, I, block_size, activation, static_cast<Act>(dtype), stream};
  return run_moe(false, a, workspace_bytes, path);
}

int fp4w_moe(const void* A, int64_t M, int64_t K, const int32_t* ids, const float* weights, int64_t topk,
             const uint8_t* w13, const uint8_t* w13_scale, const float* w13_scale_2, const uint8_t* w2,
             const uint8_t* w2_scale, const float* w2_scale_2, int64_t E, int64_t I, int64_t block_size,
             int activation, void* workspace, int64_t workspace_bytes, void* Y, int dtype, void* stream) {
  return fp4w_moe_ex(A, M, K, ids, weights, topk, w13, w13_scale, w13_scale_2, w2, w2_scale, w2_scale_2, E, I,
                     block_size, activation, workspace, workspace_bytes, Y, dtype, stream, FP4W_PATH_AUTO);
}

int fp8w_moe_ex(const void* A, int64_t M, int64_t K, const int32_t* ids, const float* weights, int64_t topk,
                const uint8_t* w13, const float* w13_scale, const uint8_t* w2, const float* w2_scale, int64_t E,
                int64_t I, int64_t block_size, int activation, void* workspace, int64_t workspace_bytes, void* Y,
                int dtype, void* stream, int path) {
  const MoeArgs a{A, ids, weights, w13, w13_scale, nullptr, w2, w2_scale, nullptr, workspace, Y,
                  M, K, topk, E, I, block_size, activation, static_cast<Act>(dtype), stream};
  return run_moe(true, a, workspace_bytes, path);
}

int fp8w_moe(const void* A, int64_t M, int64_t K, const int32_t* ids, const float* weights, int64_t topk,
             const uint8_t* w13, const float* w13_scale, const uint8_t* w2, const float* w2_scale, int64_t E,
             int64_t I, int64_t block_size, int activation, void* workspace, int64_t workspace_bytes, void* Y,
             int dtype, void* stream) {
  return fp8w_moe_ex(A, M, K, ids, weights, topk, w13, w13_scale, w2, w2_scale, E, I, block_size, activation,
                     workspace, workspace_bytes, Y, dtype, stream, FP4W_PATH_AUTO);
}

}  // extern "C"
