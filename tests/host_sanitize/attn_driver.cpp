// Drives the C ABI between the projections of an attention block through its
// validation and dispatch with addresses that stand in for device pointers
// (nothing is dereferenced: the launchers here only record the choice).  Prints
// "ok" and exits 0 when every status and every chosen kernel is the expected one.
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include "../../fp8_weight_only_fp4w_amd/csrc/launch.h"
#include "../../include/fp4w.h"

namespace fp4w {
static const char* g_last = "";
int launch_qk_norm_rope(const QkNormRopeArgs&, bool vec, const SeqArgs*) {
  g_last = vec ? "rope_vec" : "rope";
  return 0;
}
static int g_append_rc = 0;
int launch_kv_append(const KvAppendArgs&, bool vec) {
  g_last = vec ? "append_vec" : "append";
  return g_append_rc;
}
int launch_attention_decode(const AttentionArgs&) {
  g_last = "decode";
  return 0;
}
int launch_attention_prompt(const AttentionArgs&) {
  g_last = "prompt";
  return 0;
}
int launch_attention_generic(const AttentionArgs&) {
  g_last = "generic";
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
  // stand-in device addresses, 16 TiB apart
  auto fake = [](uint64_t i, int off = 0) { return reinterpret_cast<unsigned char*>((i << 44) + off); };
  auto f32 = [&](uint64_t i) { return reinterpret_cast<float*>(fake(i)); };
  auto i32 = [&](uint64_t i) { return reinterpret_cast<int32_t*>(fake(i)); };

  auto rope = [&](int64_t M, int64_t Hq, int64_t Hk, int64_t D, int64_t rows, int64_t dims, int64_t stride, int off) {
    fp4w::g_last = "";
    return fp4w_qk_norm_rope(fake(1, off), stride, Hq, fake(2), stride, Hk, M, D, fake(3), nullptr, 0.0f, 1e-6f, f32(4), f32(5), rows,
                             dims, 0, i32(6), fake(7), stride, fake(8), stride, FP4W_BF16, nullptr);
  };
  EXPECT(rope(5, 4, 2, 128, 100, 128, 512, 0) == FP4W_OK);
  LAUNCHED("rope_vec");
  EXPECT(rope(5, 4, 2, 128, 100, 64, 520, 0) == FP4W_OK);
  LAUNCHED("rope_vec");
  EXPECT(rope(5, 4, 2, 128, 100, 8, 512, 0) == FP4W_OK);  // rotated values in no whole chunks
  LAUNCHED("rope");
  EXPECT(rope(5, 4, 2, 128, 100, 128, 512, 2) == FP4W_OK);
  LAUNCHED("rope");
  EXPECT(rope(5, 4, 2, 128, 100, 128, 515, 0) == FP4W_OK);
  LAUNCHED("rope");
  EXPECT(rope(1, 4, 2, 128, 100, 128, 515, 0) == FP4W_OK);  // one row: its stride is never used
  LAUNCHED("rope_vec");
  EXPECT(rope(5, 4, 2, 80, 100, 80, 512, 0) == FP4W_OK);
  LAUNCHED("rope");
  fp4w::g_last = "";
  for (int64_t big : {INT64_MAX, INT64_MAX / 2 + 1, INT64_MIN, int64_t(1) << 31}) {
    EXPECT(rope(big, 4, 2, 128, 100, 128, 512, 0) == FP4W_ERR_SHAPE);
    EXPECT(rope(5, big, 2, 128, 100, 128, 512, 0) == FP4W_ERR_SHAPE);
    EXPECT(rope(5, 4, big, 128, 100, 128, 512, 0) == FP4W_ERR_SHAPE);
    EXPECT(rope(5, 4, 2, big, 100, 128, 512, 0) == FP4W_ERR_SHAPE);
    EXPECT(rope(5, 4, 2, 128, 100, big, 512, 0) == FP4W_ERR_SHAPE);
    if (big != int64_t(1) << 31) {
      EXPECT(rope(5, 4, 2, 128, big, 128, 512, 0) == FP4W_ERR_SHAPE);
      EXPECT(rope(5, 4, 2, 128, 100, 128, big, 0) == FP4W_ERR_SHAPE);
    }
    LAUNCHED("");
  }

  auto append = [&](int64_t M, int64_t D, int64_t B, int64_t columns, int64_t pages, int64_t page, int off) {
    fp4w::g_last = "";
    return fp8w_kv_append(fake(1, off), 2 * D, fake(2), 2 * D, M, 2, D, fake(3), 4 * D, 4, nullptr, fake(4), 0.0f, 1e-6f, f32(5), f32(6),
                          100, D, 0, nullptr, fake(7), 4 * D, i32(8), B, i32(9), i32(10), columns, fake(11), fake(12), fake(13), fake(14),
                          pages, page, FP4W_F16, nullptr);
  };
  EXPECT(append(9, 128, 3, 5, 20, 16, 0) == FP4W_OK);
  LAUNCHED("append_vec");
  EXPECT(append(9, 128, 3, 5, 20, 128, 0) == FP4W_OK);
  LAUNCHED("append_vec");
  EXPECT(append(9, 128, 3, 5, 20, 144, 0) == FP4W_OK);  // a page past what a workgroup takes
  LAUNCHED("append");
  EXPECT(append(9, 128, 3, 5, 20, 24, 0) == FP4W_OK);
  LAUNCHED("append");
  EXPECT(append(9, 96, 3, 5, 20, 16, 0) == FP4W_OK);
  LAUNCHED("append");
  EXPECT(append(9, 128, 3, 5, 20, 16, 2) == FP4W_OK);
  LAUNCHED("append");
  EXPECT(append(9, 128, 3, 0, 0, 16, 0) == FP4W_OK);  // no pages
  fp4w::g_append_rc = -1;
  EXPECT(append(9, 128, 3, 5, 20, 16, 0) == FP4W_ERR_LAUNCH);
  fp4w::g_append_rc = 0;
  fp4w::g_last = "";
  for (int64_t big : {INT64_MAX, INT64_MAX / 2 + 1, INT64_MIN, int64_t(1) << 31}) {
    EXPECT(append(big, 128, 3, 5, 20, 16, 0) == FP4W_ERR_SHAPE);
    EXPECT(append(9, 128, big, 5, 20, 16, 0) == FP4W_ERR_SHAPE);
    EXPECT(append(9, 128, 3, big, 20, 16, 0) == FP4W_ERR_SHAPE);
    EXPECT(append(9, 128, 3, 5, big, 16, 0) == FP4W_ERR_SHAPE);
    EXPECT(append(9, 128, 3, 5, 20, big, 0) == FP4W_ERR_SHAPE);
    LAUNCHED("");
  }
  const int64_t most = (int64_t(1) << 31) - 1;
  EXPECT(append(9, 128, most, most, 20, 1, 0) == FP4W_ERR_SHAPE);  // a page table past 2^60 entries

  struct Case {
    int64_t M = 9, Hq = 8, Hk = 2, D = 128, B = 3, columns = 5, most = 9, pages = 20, page = 16;
    int off = 0, path = FP4W_PATH_AUTO;
    int64_t window = 0, held = int64_t(1) << 40;
    bool starts = true;
  };
  auto attn = [&](const Case& c) {
    fp4w::g_last = "";
    return fp8w_attention_ex(fake(1, c.off), c.D > 0 && c.D < 4096 && c.Hq > 0 && c.Hq < 4096 ? c.Hq * c.D : 4096, c.M, c.Hq, c.Hk, c.D,
                             c.starts ? i32(2) : nullptr, c.B, i32(3), i32(4), c.columns, c.most, fake(5), fake(6), fake(7), fake(8),
                             c.pages, c.page, 0.1f, 1, c.window, fake(9), c.held, fake(13), f32(14), FP4W_BF16, nullptr, c.path);
  };
  auto with = [](auto set) {
    Case c;
    set(c);
    return c;
  };
#define ATTN(...) attn(with([&](Case& c) { __VA_ARGS__; }))
  EXPECT(ATTN() == FP4W_OK);
  LAUNCHED("decode");  // 9 tokens of 4 heads
  EXPECT(ATTN(c.M = 17; c.most = 16) == FP4W_OK);
  LAUNCHED("decode");
  EXPECT(ATTN(c.M = 17; c.most = 17) == FP4W_OK);
  LAUNCHED("prompt");
  EXPECT(ATTN(c.M = 17; c.most = INT64_MAX) == FP4W_OK);
  LAUNCHED("prompt");
  EXPECT(ATTN(c.M = 3; c.most = 99; c.starts = false) == FP4W_OK);
  LAUNCHED("decode");
  EXPECT(ATTN(c.M = 5000; c.most = 1000; c.path = FP4W_PATH_ATTN_DECODE) == FP4W_ERR_PATH);
  EXPECT(ATTN(c.path = FP4W_PATH_ATTN_PROMPT) == FP4W_OK);
  LAUNCHED("prompt");
  EXPECT(ATTN(c.path = FP4W_PATH_ATTN_GENERIC) == FP4W_OK);
  LAUNCHED("generic");
  for (int path : {FP4W_PATH_ATTN_DECODE, FP4W_PATH_ATTN_PROMPT}) {
    EXPECT(ATTN(c.D = 96; c.path = path) == FP4W_ERR_PATH);
    EXPECT(ATTN(c.page = 24; c.path = path) == FP4W_ERR_PATH);
    EXPECT(ATTN(c.off = 2; c.path = path) == FP4W_ERR_PATH);
  }
  EXPECT(ATTN(c.D = 96; c.held = 0) == FP4W_OK);
  LAUNCHED("generic");
  EXPECT(ATTN(c.page = 8) == FP4W_OK);
  LAUNCHED("generic");
  EXPECT(ATTN(c.columns = (int64_t(1) << 27) - 1) == FP4W_OK);  // tokens with the tiles behind them pass 2^31
  LAUNCHED("generic");
  EXPECT(ATTN(c.columns = (int64_t(1) << 27) - 64) == FP4W_OK);
  LAUNCHED("decode");
  EXPECT(ATTN(c.columns = (int64_t(1) << 27) - 64; c.B = 64) == FP4W_OK);  // 2^30 tiles and more
  LAUNCHED("prompt");
  EXPECT(ATTN(c.M = most; c.most = 1; c.Hq = 2) == FP4W_OK);  // more rows than a grid takes
  LAUNCHED("generic");
  EXPECT(ATTN(c.window = INT64_MAX) == FP4W_OK);
  LAUNCHED("decode");
  EXPECT(ATTN(c.window = -1) == FP4W_ERR_SHAPE);
  EXPECT(ATTN(c.held = 16) == FP4W_ERR_SHAPE);
  EXPECT(ATTN(c.pages = 0; c.columns = 0) == FP4W_OK);
  EXPECT(ATTN(c.B = most; c.columns = most; c.page = 1) == FP4W_ERR_SHAPE);
  for (int64_t big : {INT64_MAX, INT64_MAX / 2 + 1, INT64_MIN, int64_t(1) << 31}) {
    EXPECT(ATTN(c.M = big) == FP4W_ERR_SHAPE);
    EXPECT(ATTN(c.Hq = big) == FP4W_ERR_SHAPE);
    EXPECT(ATTN(c.Hk = big) == FP4W_ERR_SHAPE);
    EXPECT(ATTN(c.D = big) == FP4W_ERR_SHAPE);
    EXPECT(ATTN(c.B = big) == FP4W_ERR_SHAPE);
    EXPECT(ATTN(c.columns = big) == FP4W_ERR_SHAPE);
    EXPECT(ATTN(c.pages = big) == FP4W_ERR_SHAPE);
    EXPECT(ATTN(c.page = big) == FP4W_ERR_SHAPE);
    LAUNCHED("");
  }
  EXPECT(fp8w_attention_workspace(most, (1 << 20) - 1, (1 << 20) - 1, 128, most, INT64_MAX) > 0);
  EXPECT(fp8w_attention_workspace(most, (1 << 20) - 1, 1, 64, most, INT64_MAX) > 0);
  EXPECT(fp8w_attention_workspace(0, 0, 0, 0, 0, 0) == 0);
  EXPECT(fp8w_attention_workspace(1, 1, 1, 128, 1, INT64_MIN) == FP4W_ERR_SHAPE);

  // What the kernels write of the workspace, by the launchers' own arithmetic,
  // is inside what is asked for, for every smaller call too.
  for (int64_t D : {64, 128})
    for (int64_t Hk : {1, 2, 8, 40, 300, 600})
      for (int64_t G : {1, 3, 5, 7, 16, 33, 64, 70})
        for (int64_t asked : {1, 3, 9, 64, 500}) {
          const int64_t held = fp8w_attention_workspace(500, G * Hk, Hk, D, 40, asked);
          for (int64_t n = 1; n <= asked && n * G <= 64; ++n) {
            const int64_t rows = n * G, per_unit = rows <= 16 || D == 64 ? 2 : 1, row_tiles = (rows + 15) / 16;
            const int64_t held_tiles = D == 128 && rows > 16 ? 2 : 1;  // row tiles of a wave
            const int64_t sets = row_tiles <= held_tiles ? 1 : row_tiles <= 2 * held_tiles ? 2 : 4;
            const int64_t shares = fp4w::attn_groups(Hk, static_cast<int>(per_unit)) * (4 / sets);
            EXPECT(shares == fp4w::attn_shares(rows, Hk, D));
            EXPECT(fp4w::kAttnPlanBytes + shares * Hk * 2 * fp4w::attn_part_floats(rows, D) * 4 <= held);
          }
          const int64_t tiles = fp4w::attn_row_tiles_most(500, G, 40) * Hk;
          for (int64_t capacity : {16, 4096, 1 << 20}) {
            const int64_t splits = fp4w::attn_prompt_splits(tiles, capacity);
            EXPECT(splits == 1 || tiles * splits * fp4w::attn_part_floats(fp4w::kPromptRows, D) * 4 <= held);
          }
        }
  if (failures == 0) printf("ok\n");
  return failures != 0;
}
