// Internal interface between the host-side dispatch (dispatch.cpp, plain C++)
// and the HIP launchers (*.hip).  Not part of the public ABI.
#pragma once

#include <stdint.h>

#include <mutex>

namespace fp4w {

constexpr int kMaxHead = 1024;  // FP8W_MAX_HEAD_SIZE of the public header

enum class Act : int { F16 = 0, BF16 = 1 };

// Arguments of one matmul call after validation.  `scales` is uint8 E4M3
// bytes for FP4 and float for FP8; `ws2` is only used by FP4.
struct MatmulArgs {
  const void* A;
  const uint8_t* B;
  const void* scales;
  const float* ws2;
  const void* bias;
  void* Y;
  int64_t M, N, K, block_size, scale_cols;
  Act act;
  void* stream;  // hipStream_t
};

struct DequantArgs {
  const uint8_t* B;
  const uint8_t* scales;
  const float* ws2;
  void* out;
  int64_t N, K, block_size, scale_cols;
  Act act;
  void* stream;
};

struct Fp8DequantArgs {
  const uint8_t* B;
  const float* scales;
  void* out;
  int64_t N, K, block_size, scale_cols;
  Act act;
  void* stream;
};

// Activation quantize/dequantize (W8A8 mode): `count` elements of T.
struct QdqArgs {
  const void* A;
  const float* a_scale;
  void* out;
  int64_t count;
  Act act;
  void* stream;
};

// NVFP4 activation quantization (W4A4 path): `blocks` blocks of 16 elements
// of T.  Packed mode writes `codes` (8 bytes per block) and `scales` (1 byte
// per block); QDQ mode writes `out` (16 elements of T per block).
struct Nvfp4Args {
  const void* A;
  uint8_t* codes;
  uint8_t* scales;
  void* out;
  int64_t blocks;
  Act act;
  void* stream;
};

// Norms around a block with its gate and residual (fp4w_block_norm); absent
// parts are null.  gate_rows is 1 (one row for all) or M.
struct BlockNormArgs {
  const void* x;
  const void* post_weight;
  const void* gate;
  const void* residual;
  const void* pre_weight;
  void* residual_out;
  void* y;
  int64_t M, K, gate_rows;
  float scale, weight_offset, eps;
  Act act;
  void* stream;
};

// Routing of tokens to experts (fp4w_moe_route).  `logits_dtype`: an
// fp4w_dtype, FP4W_F32 included.
struct MoeRouteArgs {
  const void* logits;
  const float* select_bias;
  int32_t* ids;
  float* weights;
  int64_t M, E, topk;
  bool sigmoid, renormalize;
  float scale;
  int logits_dtype;
  void* stream;
};

// One mixture-of-experts layer after validation (fp4w_moe, fp8w_moe).
// s13 / s2: E4M3 bytes (FP4) or floats (FP8); g13 / g2: FP32 per expert (FP4
// only).  `work` holds fp4w_moe_workspace() bytes.
struct MoeArgs {
  const void* A;
  const int32_t* ids;
  const float* weights;
  const uint8_t* w13;
  const void* s13;
  const float* g13;
  const uint8_t* w2;
  const void* s2;
  const float* g2;
  void* work;
  void* Y;
  int64_t M, K, topk, E, I, block_size;
  int activation;
  Act act;
  void* stream;
};

// Norm and rotation of heads (fp4w_qk_norm_rope, and on the way in
// fp8w_kv_append).  Strides in values of T.  cos / sin null: no rotation.
struct RopeArgs {
  const void* q_weight;
  const void* k_weight;
  const float* cos;
  const float* sin;
  const int32_t* positions;
  int64_t rows, dims;
  bool interleaved;
  float weight_offset, eps;
};

// Which rows of a call belong to which sequence, and where its tokens are.
// starts null: row b is sequence b's only new token.
struct SeqArgs {
  const int32_t* starts;
  const int32_t* lens;
  const int32_t* table;
  int64_t B, max_pages, num_pages, page_size;
};

struct QkNormRopeArgs {
  const void* q;
  const void* k;
  void* q_out;
  void* k_out;
  int64_t q_stride, k_stride, q_out_stride, k_out_stride, M, Hq, Hk, D;
  RopeArgs rope;
  Act act;
  void* stream;
};

// q null or Hq 0: keys and values only.
struct KvAppendArgs {
  const void* k;
  const void* v;
  const void* q;
  void* q_out;
  int64_t k_stride, v_stride, q_stride, q_out_stride, M, Hk, Hq, D;
  RopeArgs rope;
  SeqArgs seq;
  uint8_t* k_cache;
  uint8_t* k_scale;
  uint8_t* v_cache;
  uint8_t* v_scale;
  Act act;
  void* stream;
};

// Attention over the cache.  window 0: none.  `work` holds
// fp8w_attention_workspace() bytes.
struct AttentionArgs {
  const void* q;
  int64_t q_stride, M, Hq, Hk, D, max_new;
  SeqArgs seq;
  const uint8_t* k_cache;
  const uint8_t* k_scale;
  const uint8_t* v_cache;
  const uint8_t* v_scale;
  float scale;
  bool causal;
  int64_t window;
  void* work;
  void* Y;
  float* lse;
  Act act;
  void* stream;
};

// Each launcher enqueues its kernel(s) and returns 0, or -1 when HIP reports
// an error at enqueue time.  Preconditions (checked by the dispatcher, never
// by the launcher) are stated next to each.

// Host-side state is per device and initialised once, thread-safely: the
// library keeps no other state between calls.
constexpr int kMaxDevices = 64;

// the calling thread's current HIP device (0 if the query fails)
int current_device();

// compute units of the current device, queried once per device (256 if the
// query fails)
int device_cus();

// Runs f() once per device for the given flag array (device ids beyond
// kMaxDevices run it on every call; f must be idempotent).
template <typename F>
void once_per_device(std::once_flag (&flags)[kMaxDevices], F&& f) {
  const int dev = current_device();
  if (dev < 0 || dev >= kMaxDevices)
    f();
  else
    std::call_once(flags[dev], f);
}

// 1 <= M <= 8, block_size == 16, K % 32 == 0, scale_cols == K / 16,
// A / B 16-byte aligned, scales 4-byte aligned, bias 2-byte aligned.
int launch_fp4_gemv(const MatmulArgs& a);
// The same GEMV with the W4A4 activation step fused: the LDS copy of A is
// NVFP4 quantize-dequantized before use and also written to a_work (M x K,
// 16-byte aligned, disjoint from A); K % 16 == 0.  Returns 1, launching
// nothing, when A does not fit in LDS or M x K / 16 exceeds 1536 blocks.
int launch_fp4_gemv_w4a4(const MatmulArgs& a, void* a_work);
// M >= 1, block_size == 16, K % 64 == 0, scale_cols == K / 16,
// A / B 16-byte aligned, scales 4-byte aligned.
int launch_fp4_gemm(const MatmulArgs& a);
// 1 <= M <= 64, block_size == 16, K % 128 == 0, scale_cols == K / 16,
// A / B 16-byte aligned, scales 4-byte aligned, bias / Y 2-byte aligned.
int launch_fp4_skinny(const MatmulArgs& a);
// any validated FP4 arguments (K may be 0)
int launch_fp4_generic(const MatmulArgs& a);

// 1 <= M <= 8, block_size % 64 == 0, K % 16 == 0, A / B 16-byte aligned,
// scales 4-byte aligned.
int launch_fp8_gemv(const MatmulArgs& a);
// M >= 1, block_size % 64 == 0, K % 64 == 0, A / B 16-byte aligned.
int launch_fp8_gemm(const MatmulArgs& a);
// 1 <= M <= 64, block_size % 128 == 0, K % 128 == 0, A / B 16-byte aligned,
// scales 4-byte aligned.
int launch_fp8_skinny(const MatmulArgs& a);
// any validated FP8 arguments (K may be 0)
int launch_fp8_generic(const MatmulArgs& a);

// K % 8 == 0, block_size % 8 == 0, B 4-byte aligned, out 16-byte aligned,
// N * K / 8 < 2^32.
int launch_dequant_vec(const DequantArgs& a);
// any validated arguments with N, K > 0
int launch_dequant_generic(const DequantArgs& a);

// FP8 dequant: K % 16 == 0, block_size % 16 == 0, B / out 16-byte aligned,
// N * K / 16 < 2^32.
int launch_fp8_dequant_vec(const Fp8DequantArgs& a);
// any validated arguments with N, K > 0
int launch_fp8_dequant_generic(const Fp8DequantArgs& a);

// count % 8 == 0, A and out 16-byte aligned; out == A allowed.
int launch_qdq_vec(const QdqArgs& a);
// any count > 0; out == A allowed.
int launch_qdq_generic(const QdqArgs& a);

// NVFP4 quantization, packed (codes and scales) or QDQ (out; out == A
// allowed).  vec: A 16-byte aligned, and codes 8-byte aligned (packed) or
// out 16-byte aligned (QDQ).  blocks > 0.
int launch_nvfp4_quantize(const Nvfp4Args& a, bool vec);
int launch_nvfp4_qdq(const Nvfp4Args& a, bool vec);

// Library-owned device scratch of the allocation-free entry point (its size
// is FP4W_STATIC_SCRATCH_BYTES of the public header): the address of the
// current device's copy, taken once per device.  0, or -1 when HIP cannot
// provide it.
constexpr int64_t kStaticScratchBytes = int64_t(32) << 20;
int static_scratch(void** out);

// M, K > 0.  vec: K % 8 == 0 and every pointer 16-byte aligned.
int launch_block_norm(const BlockNormArgs& a, bool vec);

// M, topk > 0, topk <= 64, E <= 1024.
int launch_moe_route(const MoeRouteArgs& a);

// Parts that the second product's sum over I may be cut into, at most, for M
// tokens (each part has outputs of its own in the workspace): 32 (or M) token
// rows of two BF16 planes have to fit in LDS.
inline int64_t moe_down_splits(int64_t M, int64_t I) {
  const int64_t rows = M < 32 ? M : 32, bytes = rows * 4 * I, parts = (bytes + (112 << 10) - 1) / (112 << 10);
  return parts < 1 ? 1 : parts < 4 ? parts : 4;
}
// n = M * topk in 1 .. 4096, E in 1 .. 1024, K % 64 == 0, I % 64 == 0 (both >
// 0), block_size 16 (FP4) or a multiple of 128 (FP8); A, w13, w2, work and Y
// 16-byte aligned, scales 4-byte; A, an expert's matrices and n x I x 4 below
// 2^31 bytes.  Return 1, launching nothing, when a token's row does not fit in
// LDS, or the shares of the work cannot be counted in 32 bits.
int launch_moe_fp4(const MoeArgs& a);
int launch_moe_fp8(const MoeArgs& a);
// any validated arguments with M, K > 0 (E, topk and I may be 0)
int launch_moe_fp4_generic(const MoeArgs& a);
int launch_moe_fp8_generic(const MoeArgs& a);

// M, D > 0, Hq + Hk > 0.  seq not null: positions (where rope.positions is
// null) from the sequences, and rows of none left alone.  vec: every pointer (but positions) 16-byte aligned,
// strides multiples of 8, D a power of two from 16 to 1024, and rope.dims and
// D - rope.dims multiples of 16.
int launch_qk_norm_rope(const QkNormRopeArgs& a, bool vec, const SeqArgs* seq);

// M, B, D > 0.  vec: what launch_qk_norm_rope asks for, page_size % 16 == 0
// and page_size * D <= 16384, cache codes 16-byte aligned.
int launch_kv_append(const KvAppendArgs& a, bool vec);

// The decode kernel of attention: workgroups of four waves for each key head,
// one or two for each compute unit in all.  In the workspace, behind the plan of
// a launch's sequences: two partial results for each share of a key head's tiles.
constexpr int kSeqsPerLaunch = 1024;
constexpr int64_t kAttnPlanBytes = 4352;  // (kSeqsPerLaunch + 1) x 4, up to 256
inline int attn_groups(int64_t Hk, int per_unit) {
  const int64_t places = 256 * per_unit;
  return Hk >= places ? 1 : static_cast<int>(places / Hk);
}
// shares of a key head, for up to 64 rows (max_new tokens of G query heads)
inline int64_t attn_shares(int64_t rows, int64_t Hk, int64_t D) {
  if (rows <= 16) return attn_groups(Hk, 2) * 4;
  if (D == 64) return attn_groups(Hk, 2) * (rows <= 32 ? 2 : 1);
  return attn_groups(Hk, 1) * (rows <= 32 ? 4 : 2);
}
// maxima and sums of `rows` rows in whole 16-byte units, then their outputs
constexpr int64_t attn_part_head(int64_t rows) { return (2 * rows + 3) / 4 * 4; }
constexpr int64_t attn_part_floats(int64_t rows, int64_t D) { return attn_part_head(rows) + rows * D; }
// (more rows mean fewer shares: a buffer has to serve fewer new tokens too)
inline int64_t attn_decode_workspace(int64_t max_new, int64_t Hk, int64_t G, int64_t D) {
  int64_t most = 0;
  for (int64_t rows = 16; rows <= 64; rows *= 2) {
    const int64_t n = max_new < rows / G ? max_new : rows / G;
    const int64_t floats = attn_shares(n * G, Hk, D) * Hk * 2 * attn_part_floats(n * G, D);
    most = most > floats ? most : floats;
  }
  return kAttnPlanBytes + most * 4;
}
// D 64 or 128, page_size % 16 == 0, max_new * Hq / Hk <= 64; q, the cache's
// codes, Y and work 16-byte aligned, q_stride % 8 == 0.
int launch_attention_decode(const AttentionArgs& a);
// The prompt kernel: row tiles of kPromptRows rows of a sequence and key head.
// Where there are fewer than kPromptPlaces (heads of 128 have two workgroups a
// compute unit, those of 64 three), their keys are cut into up to 16 parts, whose
// results are in the workspace.  The host knows a row tile's keys only by what the
// page table has room for; the kernel takes fewer parts, so that each has at least
// kPromptPart key tiles: 200 tokens of 40 heads in a table with room for 32768
// take 16 us so, with empty parts 31, and in a table cut to their length 14.  A part costs 133 KB of traffic for D = 128:
// with 784 row tiles, two parts each took 85 us and whole ones 56.  With 272 over
// ragged 5000 to 25000 tokens, 1, 2, 3, 5 and 7 parts took 420, 353, 342, 323 and
// 320 us; with 336 over even 15000, 3, 5 and 6 parts 376, 403 and 395: two full
// rounds of workgroups, and then parts that cost more than they even out.
constexpr int kPromptRows = 128, kPromptPart = 8;
constexpr int64_t kPromptPlaces = 512, kPromptWork = 768;  // workgroups that are wanted where there are too few
inline int64_t attn_row_tiles_most(int64_t M, int64_t G, int64_t B) { return M * G / kPromptRows + B; }
inline int64_t attn_prompt_splits(int64_t tiles, int64_t capacity) {
  if (tiles >= kPromptPlaces) return 1;
  const int64_t want = (kPromptWork + tiles - 1) / tiles, most = capacity / (kPromptPart * 64);
  const int64_t n = want < most ? want : most;
  return n < 1 ? 1 : n < 16 ? n : 16;
}
inline int64_t attn_prompt_workspace(int64_t M, int64_t G, int64_t B, int64_t Hk, int64_t D) {
  const int64_t tiles = attn_row_tiles_most(M, G, B) * Hk;
  const int64_t most = kPromptWork + kPromptPlaces;  // tiles * splits is less where there are several
  return (16 * tiles < most ? 16 * tiles : most) * attn_part_floats(kPromptRows, D) * 4;
}
// as launch_attention_decode, for any max_new; the grid and the row tiles in
// 32 bits.
int launch_attention_prompt(const AttentionArgs& a);
// any validated arguments with M, B, Hq, D > 0
int launch_attention_generic(const AttentionArgs& a);

}  // namespace fp4w
