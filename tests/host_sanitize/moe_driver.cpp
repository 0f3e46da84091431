// Drives the C ABI around a mixture-of-experts block through its validation
// and dispatch with addresses that stand in for device pointers (nothing is
// dereferenced: the launchers here only record the choice).  Prints "ok" and
// exits 0 when every status and every chosen kernel is the expected one.
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include "../../fp8_weight_only_fp4w_amd/csrc/launch.h"
#include "../../include/fp4w.h"

namespace fp4w {
static const char* g_last = "";
int current_device() { return 0; }
int device_cus() { return 256; }
int launch_block_norm(const BlockNormArgs&, bool vec) {
  g_last = vec ? "norm_vec" : "norm";
  return 0;
}
int launch_moe_route(const MoeRouteArgs&) {
  g_last = "route";
  return 0;
}
// what the streaming kernels return: 0 (launched) or 1 (a row does not fit in LDS)
static int g_stream_rc = 0;
int launch_moe_fp4(const MoeArgs&) {
  if (g_stream_rc == 0) g_last = "fp4_stream";
  return g_stream_rc;
}
int launch_moe_fp8(const MoeArgs&) {
  if (g_stream_rc == 0) g_last = "fp8_stream";
  return g_stream_rc;
}
int launch_moe_fp4_generic(const MoeArgs&) {
  g_last = "fp4_generic";
  return 0;
}
int launch_moe_fp8_generic(const MoeArgs&) {
  g_last = "fp8_generic";
  return 0;
}
}  // namespace fp4w

static int failures = 0;
static void expect(bool ok, const char* what, int line) {
  if (!ok) {
    printf("FAIL line %d: %s (last launch: %s)\n", line, what, fp4w::g_last);
    ++failures;
  }
}
#define EXPECT(c) expect((c), #c, __LINE__)
#define LAUNCHED(name) EXPECT(strcmp(fp4w::g_last, name) == 0)

int main() {
  // stand-in device addresses, 64 GiB apart
  auto fake = [](uint64_t i, int off = 0) { return reinterpret_cast<unsigned char*>((i << 36) + off); };
  auto f32 = [&](uint64_t i) { return reinterpret_cast<float*>(fake(i)); };
  auto i32 = [&](uint64_t i) { return reinterpret_cast<int32_t*>(fake(i)); };
  auto norm = [&](int64_t M, int64_t K, int off) {
    fp4w::g_last = "";
    return fp4w_block_norm(fake(1, off), M, K, fake(2), fake(3), M, 0.5f, fake(4), fake(5), 1.0f, 1e-6f, fake(6),
                           fake(7), FP4W_BF16, nullptr);
  };
  EXPECT(norm(5, 64, 0) == FP4W_OK);
  LAUNCHED("norm_vec");
  EXPECT(norm(5, 64, 2) == FP4W_OK);
  LAUNCHED("norm");
  EXPECT(norm(5, 63, 0) == FP4W_OK);
  LAUNCHED("norm");
  EXPECT(norm(int64_t(1) << 40, int64_t(1) << 40, 0) == FP4W_ERR_SHAPE);
  LAUNCHED("");
  EXPECT(norm(INT64_MAX, INT64_MAX, 0) == FP4W_ERR_SHAPE);
  EXPECT(norm(INT64_MIN, 8, 0) == FP4W_ERR_SHAPE);

  auto route = [&](int64_t M, int64_t E, int64_t topk) {
    fp4w::g_last = "";
    return fp4w_moe_route(fake(1), M, E, topk, FP4W_SCORE_SIGMOID, f32(2), 1, 1.0f, i32(3), f32(4), FP4W_F16, nullptr);
  };
  EXPECT(route(7, 5, 9) == FP4W_OK);
  LAUNCHED("route");
  EXPECT(route(7, 0, 2) == FP4W_OK);
  LAUNCHED("route");
  EXPECT(route(INT64_MAX, 8, 2) == FP4W_ERR_SHAPE);
  EXPECT(route(INT64_MAX / 4, 1024, 64) == FP4W_ERR_SHAPE);
  LAUNCHED("");

  const int64_t lots = int64_t(1) << 34;
  auto fp4 = [&](int64_t M, int64_t K, int64_t topk, int64_t E, int64_t I, int64_t bs, int path) {
    fp4w::g_last = "";
    return fp4w_moe_ex(fake(1), M, K, i32(2), f32(3), topk, fake(4), fake(5), f32(6), fake(7), fake(8), f32(9), E, I,
                       bs, FP4W_ACT_SILU, fake(10), lots, fake(11), FP4W_F16, nullptr, path);
  };
  auto fp8 = [&](int64_t M, int64_t K, int64_t topk, int64_t E, int64_t I, int64_t bs, int path) {
    fp4w::g_last = "";
    return fp8w_moe_ex(fake(1), M, K, i32(2), f32(3), topk, fake(4), f32(5), fake(7), f32(8), E, I, bs,
                       FP4W_ACT_GELU_TANH, fake(10), lots, fake(11), FP4W_BF16, nullptr, path);
  };
  EXPECT(fp4(3, 30, 2, 4, 22, 15, FP4W_PATH_AUTO) == FP4W_OK);
  LAUNCHED("fp4_generic");
  EXPECT(fp8(3, 31, 2, 4, 21, 7, FP4W_PATH_AUTO) == FP4W_OK);
  LAUNCHED("fp8_generic");
  EXPECT(fp4(3, 64, 0, 4, 64, 16, FP4W_PATH_AUTO) == FP4W_OK);  // no choices: Y = 0
  LAUNCHED("fp4_generic");
  EXPECT(fp4(3, 64, 2, 0, 64, 16, FP4W_PATH_AUTO) == FP4W_OK);
  LAUNCHED("fp4_generic");
  EXPECT(fp4(3, 64, 2, 4, 64, 16, FP4W_PATH_AUTO) == FP4W_OK);
  LAUNCHED("fp4_stream");
  EXPECT(fp4(3, 64, 2, 4, 64, 16, FP4W_PATH_MOE_FP4_GENERIC) == FP4W_OK);
  LAUNCHED("fp4_generic");
  EXPECT(fp4(3, 96, 2, 4, 64, 16, FP4W_PATH_MOE_FP4_STREAM) == FP4W_ERR_PATH);
  EXPECT(fp4(3, 64, 2, 4, 64, 32, FP4W_PATH_MOE_FP4_STREAM) == FP4W_ERR_PATH);
  EXPECT(fp4(3, 64, 2, 4, 64, 16, FP4W_PATH_MOE_FP8_STREAM) == FP4W_ERR_PATH);
  EXPECT(fp8(3, 64, 2, 4, 64, 128, FP4W_PATH_MOE_FP8_STREAM) == FP4W_OK);
  LAUNCHED("fp8_stream");
  EXPECT(fp8(3, 64, 2, 4, 64, int64_t(1) << 40, FP4W_PATH_AUTO) == FP4W_OK);  // one block per row
  LAUNCHED("fp8_stream");
  EXPECT(fp8(3, 64, 2, 4, 64, 64, FP4W_PATH_AUTO) == FP4W_OK);
  LAUNCHED("fp8_generic");
  EXPECT(fp4(3, 1 << 16, 2, 4, 1 << 16, 16, FP4W_PATH_AUTO) == FP4W_OK);  // past 32-bit offsets
  LAUNCHED("fp4_generic");
  fp4w::g_stream_rc = 1;
  EXPECT(fp4(3, 64, 2, 4, 64, 16, FP4W_PATH_AUTO) == FP4W_OK);
  LAUNCHED("fp4_generic");
  EXPECT(fp8(3, 64, 2, 4, 64, 128, FP4W_PATH_MOE_FP8_STREAM) == FP4W_ERR_PATH);
  fp4w::g_stream_rc = -1;
  EXPECT(fp8(3, 64, 2, 4, 64, 128, FP4W_PATH_AUTO) == FP4W_ERR_LAUNCH);
  fp4w::g_stream_rc = 0;
  for (int64_t big : {INT64_MAX, INT64_MAX / 2 + 1, int64_t(1) << 41}) {
    EXPECT(fp4(big - big % 2, 64, 2, 4, 64, 16, 0) == FP4W_ERR_SHAPE);
    EXPECT(fp4(2, big - big % 2, 2, 4, 64, 16, 0) == FP4W_ERR_SHAPE);
    EXPECT(fp8(2, 64, big, 4, 64, 16, 0) == FP4W_ERR_SHAPE);
    EXPECT(fp8(2, 64, 2, big, 64, 16, 0) == FP4W_ERR_SHAPE);
    EXPECT(fp8(2, 64, 2, 4, big, 16, 0) == FP4W_ERR_SHAPE);
    EXPECT(fp8(2, 64, 2, 4, 64, big, 0) == FP4W_OK);  // one block per row
  }
  EXPECT(fp4w_moe_workspace(INT64_MAX, 1, 1, 1) == FP4W_ERR_SHAPE);
  EXPECT(fp4w_moe_workspace(64, 64, int64_t(1) << 30, int64_t(1) << 28) > 0);
  EXPECT(fp4w_moe_workspace(0, 0, 0, 0) == 0);
  if (failures == 0) printf("ok\n");
  return failures != 0;
}
