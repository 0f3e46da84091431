// Mixture-of-experts layer for a few tokens on FP4 or FP8 weights, on MFMA.
//
//   H[a, i] = act(A[m] . W1[e][i]) * (A[m] . W3[e][i])      a = m * topk + j, e = ids[a]
//   Y[m, n] = RNE_T( sum_j weights[a] * (H[a] . W2[e][n]) )
//
// Memory-bound: every chosen expert is read once per pass of up to `rows`
// tokens.  Three kernels: up (H from A), down (each choice's output from H)
// and combine (their weighted sum over a token's choices in the order of j, so
// the result does not depend on scheduling); a single token takes two.
//
// Weights go straight to registers.  A wave owns a tile of 16 weight rows, and
// a unit is 128 bytes of each: lane (li, g) loads chunks g and 4 + g (16 bytes
// each) of row li, its MFMA operand as it stands.  Each of the two loads
// touches half of every line, but back to back they make whole-line requests:
// this pattern alone streams 5.9 TB/s (5.8 where rows start off a line), the
// rate of whole-line loads, with four units in flight on 8 waves a CU, and it
// leaves all of LDS to the token rows.
//
// Plan.  ids live on the device, so which experts are read is only known
// there.  Every workgroup of up and down sorts the assignments by expert in
// LDS (a count, a scan and a scatter over n <= 4096 ids) and cuts each
// expert's tokens into passes of at most `rows`.  The work is the flat list of
// (pass, group of column tiles); workgroup b of the persistent grid takes a
// contiguous share, so it meets few experts.
//
// A pass's token rows are copied to LDS once (zero-padded to whole units) and
// shared by the 8 waves: KS waves split the sum of one column tile, 8 / KS
// tiles run side by side, and each wave's loads run Q units ahead across tiles
// and passes.  Where LDS holds two passes' rows the next ones are fetched
// while this pass is multiplied.  The up kernel's 16 rows are 8 gate rows and
// the 8 up rows that belong to them, so both halves of a product meet in one
// tile.  The down kernel may cut the sum over I into `splits` parts, each a
// pass of its own with its own outputs: its token rows have two planes, and
// rows that do not fit in LDS would mean passes that read the weights again.
//
// Operands (16x16x32 MFMA; lane li = l % 16 is token row for A and weight row
// for B, lane group g = l / 16 selects 8 of a step's 32 k; the result lane
// holds column li, token rows 4g .. 4g + 3).
//  * FP4, more than 4 tokens: E2M1 x E4M3 is exact in FP16 and BF16, so a
//    weight is decoded with its block scale folded in; the expert's FP32
//    scale is applied to the sum.
//  * FP4, up to 4 tokens: the decode GEMV's block-diagonal operand (below).
//  * FP8: E4M3 -> T is exact, a 128-k window (inside one scale block) is summed
//    in a fresh accumulator and added times its FP32 scale.
//
// Measured (us of a layer, GPU time; in brackets the bytes of the experts that
// the ids name, about, at the 4.8 TB/s of a large copy): FP4, 1 token on 8 of 128
// experts of 2048 x 768: 13.5 (4.4); 4 tokens on 24 of 64, 7168 x 2048: 134 (124);
// 32 on 89 of 128, 2048 x 768: 67 (49); 128 on 32 experts of 2880 x 2880: 178 (92).
// FP8, 1 token on 6 experts of 2048 x 1408: 17.4 (11); 16 on 67 of 128, 4096 x
// 1024: 175 (180); 100 on 15 of 16 held, 5120 x 1280: 95.5 (64).  About 7 us of
// each of the two kernels are launch, plan, token rows and first weights, 5 to 8
// the combination; one token saves the plan and the third launch.  Beyond some
// ten tokens an expert the arithmetic takes longer than the bytes: with 16 each,
// of FP4 experts, the first kernel takes 108 of its 118 us when the weights cost
// nothing, and 97 when they are loaded but not multiplied.
//
// H is handed from up to down as two BF16 planes, high part and remainder (16
// significand bits, FP32's exponent range): one BF16 or FP16 rounding of H
// would double the output's error, and in FP16 gate * up may overflow.  The
// down kernel runs both planes through the same decoded weights.  Against 64
// bits the layer's error is then that of its last rounding (128 tokens, BF16:
// 1.663016e-3 of the norm, 1.663014e-3 with FP32 throughout or exactly); 2 to 3
// of 1000 BF16 outputs lie beyond a rounding boundary, 1 to 3 with FP32
// throughout.  A third plane would cost half as many products and LDS again.

#include <hip/hip_runtime.h>

#include <algorithm>
#include <mutex>
#include <type_traits>

#include "device.h"
#include "launch.h"
#include "moe_act.h"

namespace fp4w {
namespace {

constexpr int kWaves = 8;
constexpr int kThreads = 64 * kWaves;
constexpr int Q = 4;          // units a wave has in flight
constexpr int kMaxRows = 32;  // tokens of a pass, at most: two MFMA row tiles

template <int N>
__device__ __forceinline__ void wait_vm() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  __asm__ volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (0x7 << 4) | (0xF << 8));  // vmcnt(N) only
  __asm__ volatile("" ::: "memory");
}

// Barrier for data exchanged by ds_write / ds_read only: loads stay in flight.
__device__ __forceinline__ void lds_barrier() {
  __asm__ volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

struct MoeParams {
  const void* x;        // up: A, T[M, L]; down: H planes, BF16 [2][n][L]
  const uint8_t* w;     // [E, N, L] codes
  const uint8_t* s;     // [E, N, cols] scales
  const float* g;       // FP4: per expert
  const int32_t* ids;   // [n]
  void* out;            // up: H planes, BF16 [2][n][I]; down: FP32 [splits][n][K]
  FastDiv topk, win_per_block, chunks_per_row;  // chunks_per_row: 16-byte chunks of an LDS row
  FastDiv by_rows, by_grid, by_groups, by_splits;
  int n, E, L, N, cols;
  int x_bytes;          // up: M * L * 2; down: 2 * n * L * 2
  int rows;             // tokens per pass
  int tiles, groups;    // column tiles of an expert, and groups of TPW of them
  int splits;           // down: parts of the sum over I (up: 1)
  int fp8;
  int split_units;      // units of a row in a part
  int units;            // of those, per wave and tile
  int buffers;          // 2: LDS holds two passes' rows
  int act;
  int list_max;         // passes at most
};

// Partial sums of the K split, twice: 16 rows a wave, or (FP4, where no pass
// has more than 4 tokens) the block-diagonal form's one value a lane.
__host__ __device__ constexpr uint32_t red_stride_of(bool fp8, int rows) { return !fp8 && rows <= 4 ? 256u : 1024u; }

// What a group of tiles costs in a pass of `tokens` tokens, in sixths of one
// that only waits for memory: the dense forms are bound by their arithmetic
// (measured per unit, 8 waves a CU: FP4 block-diagonal 0.75 us, dense 1.0,
// with a second row tile 1.37).  Shares of equal cost end together, where
// shares of equal bytes let the others wait a quarter of the kernel.
__device__ __forceinline__ uint32_t pass_cost(int fp8, uint32_t tokens) {
  return fp8 ? (tokens > 16 ? 7u : 6u) : tokens > 16 ? 11u : tokens > 4 ? 8u : 6u;
}
constexpr int64_t kMostCost = 11;

struct Plan {
  const uint32_t* list;    // pass: expert | first sorted assignment << 10 | (tokens - 1) << 22
  const uint32_t* before;  // cost of the passes before it
  const uint16_t* sorted;  // assignments, by expert
  int passes;
  uint32_t cost;           // of all passes
};
// list, before and multi [list_max], count [E], part [2 kWaves + 4], sorted and expert [n]
constexpr uint32_t plan_bytes(int n, int E, int list_max) {
  return (12u * list_max + 4u * E + 4u * (2u * kWaves + 4u) + 4u * n + 15u) & ~15u;
}

// Sum over this lane and those below it.
__device__ __forceinline__ uint32_t wave_scan(uint32_t v) {
#define FP4W_SCAN(CTRL, ROWS) \
  v += static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), CTRL, ROWS, 0xF, false))
  FP4W_SCAN(0x111, 0xF);  // row_shr:1
  FP4W_SCAN(0x112, 0xF);  // row_shr:2
  FP4W_SCAN(0x114, 0xF);  // row_shr:4
  FP4W_SCAN(0x118, 0xF);  // row_shr:8
  FP4W_SCAN(0x142, 0xA);  // row_bcast:15 into rows 1 and 3
  FP4W_SCAN(0x143, 0xC);  // row_bcast:31 into rows 2 and 3
#undef FP4W_SCAN
  return v;
}

// The passes of one expert whose assignments are sorted[at ..].
__device__ __forceinline__ void write_passes(const MoeParams& p, uint32_t* list, uint32_t* before, uint32_t slot,
                                             uint32_t cost, uint32_t e, uint32_t at, uint32_t tokens) {
  for (; tokens; ++slot) {
    const uint32_t t = min(tokens, static_cast<uint32_t>(p.rows));
    list[slot] = e | at << 10 | (t - 1) << 22;
    before[slot] = cost;
    cost += pass_cost(p.fp8, t);
    at += t;
    tokens -= t;
  }
}
__device__ __forceinline__ uint32_t passes_cost(const MoeParams& p, uint32_t tokens) {
  const uint32_t rows = static_cast<uint32_t>(p.rows), full = fdiv(tokens, p.by_rows), rest = tokens - full * rows;
  return full * pass_cost(p.fp8, rows) + (rest ? pass_cost(p.fp8, rest) : 0u);
}

// n <= kWavePlan: every wave makes the whole plan by itself, one assignment a
// lane, and writes it to LDS (all the same values), so no barrier is needed.
// Experts come in the order of their first assignment.  The loop over the
// lanes takes about 55 ns an assignment, the other plan 1.0 us up to some
// hundred: they meet at 16.
constexpr int kWavePlan = 16;
__device__ __forceinline__ Plan make_plan_wave(const MoeParams& p, unsigned char* mem) {
  uint32_t* list = reinterpret_cast<uint32_t*>(mem);
  uint32_t* before = list + p.list_max;
  uint16_t* sorted = reinterpret_cast<uint16_t*>(before + p.list_max);
  const int lane = threadIdx.x & 63;
  const int id = lane < p.n ? p.ids[lane] : -1;
  int tokens = 0, rank = 0, first = lane;
  for (int j = p.n - 1; j >= 0; --j) {
    const bool same = __builtin_amdgcn_readlane(id, j) == id;
    tokens += same;
    rank += same && j < lane;
    first = same ? j : first;
  }
  const bool valid = static_cast<uint32_t>(id) < static_cast<uint32_t>(p.E);
  const bool leads = valid && first == lane;
  const uint32_t mine = leads ? static_cast<uint32_t>(tokens) | fdiv(tokens + p.rows - 1, p.by_rows) << 16 : 0u;
  const uint32_t cost = leads ? passes_cost(p, tokens) : 0u;
  const uint32_t upto = wave_scan(mine), cost_upto = wave_scan(cost), at = (upto - mine) & 0xFFFF;
  if (leads) write_passes(p, list, before, (upto - mine) >> 16, cost_upto - cost, static_cast<uint32_t>(id), at, tokens);
  const uint32_t first_at = __shfl(at, first, 64);
  if (valid) sorted[first_at + rank] = static_cast<uint16_t>(lane);
  return Plan{list, before, sorted, static_cast<int>(static_cast<uint32_t>(__builtin_amdgcn_readlane(upto, 63)) >> 16),
              static_cast<uint32_t>(__builtin_amdgcn_readlane(cost_upto, 63))};
}

// All threads of the workgroup; `mem` holds plan_bytes().  Every workgroup
// comes to the same list, and to the same tokens in each pass: an expert with
// several passes has its assignments in rising order.
__device__ __forceinline__ Plan make_plan(const MoeParams& p, unsigned char* mem) {
  uint32_t* list = reinterpret_cast<uint32_t*>(mem);
  uint32_t* before = list + p.list_max;
  uint32_t* multi = before + p.list_max;  // experts of several passes: expert | first sorted assignment << 10
  uint32_t* count = multi + p.list_max;
  uint32_t* part = count + p.E;
  uint16_t* sorted = reinterpret_cast<uint16_t*>(part + 2 * kWaves + 4);
  uint16_t* expert = sorted + p.n;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  for (int e = tid; e < p.E; e += kThreads) count[e] = 0;
  if (tid == 0) part[2 * kWaves] = 0;
  __syncthreads();
  for (int a = tid; a < p.n; a += kThreads) {
    const uint32_t e = static_cast<uint32_t>(p.ids[a]);
    const bool valid = e < static_cast<uint32_t>(p.E);
    expert[a] = static_cast<uint16_t>(valid ? e : 0xFFFFu);
    if (valid) atomicAdd(&count[e], 1u);
  }
  __syncthreads();
  // experts 2 tid and 2 tid + 1 (E <= 1024): tokens in the low half, passes in the high half
  uint32_t c[2], v[2], w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    c[i] = 2 * tid + i < p.E ? count[2 * tid + i] : 0u;
    v[i] = c[i] | fdiv(c[i] + p.rows - 1, p.by_rows) << 16;
    w[i] = passes_cost(p, c[i]);
  }
  const uint32_t sum = wave_scan(v[0] + v[1]), wsum = wave_scan(w[0] + w[1]);
  if (lane == 63) {
    part[wave] = sum;
    part[kWaves + wave] = wsum;
  }
  __syncthreads();
  uint32_t ahead = sum - v[0] - v[1], cost = wsum - w[0] - w[1], total = 0, total_cost = 0;
#pragma unroll
  for (int i = 0; i < kWaves; ++i) {
    const uint32_t t = part[i], tc = part[kWaves + i];
    if (i < wave) {
      ahead += t;
      cost += tc;
    }
    total += t;
    total_cost += tc;
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t e = 2 * tid + i;
    if (c[i]) {
      const uint32_t at = ahead & 0xFFFF;
      count[e] = at;
      if (c[i] > static_cast<uint32_t>(p.rows)) multi[atomicAdd(&part[2 * kWaves], 1u)] = e | at << 10;
      write_passes(p, list, before, ahead >> 16, cost, e, at, c[i]);
    }
    ahead += v[i];
    cost += w[i];
  }
  __syncthreads();
  for (int a = tid; a < p.n; a += kThreads) {
    const uint32_t e = expert[a];
    if (e != 0xFFFFu) sorted[atomicAdd(&count[e], 1u)] = static_cast<uint16_t>(a);
  }
  __syncthreads();
  // Within an expert that order is the atomics'.  With one pass it only
  // decides the MFMA row of a token; with several, which pass a token is in,
  // and there every workgroup has to agree: a wave writes them again in order.
  const int several = __builtin_amdgcn_readfirstlane(part[2 * kWaves]);
  for (int i = wave; i < several; i += kWaves) {
    const uint32_t e = multi[i] & 1023u;
    uint32_t at = multi[i] >> 10;
    for (int a0 = 0; a0 < p.n; a0 += 64) {
      const bool mine = a0 + lane < p.n && expert[a0 + lane] == e;
      const uint64_t m = __ballot(mine);
      if (mine) sorted[at + __popcll(m & ((uint64_t(1) << lane) - 1))] = static_cast<uint16_t>(a0 + lane);
      at += __popcll(m);
    }
  }
  if (several) __syncthreads();
  return Plan{list, before, sorted, static_cast<int>(static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(total)) >> 16),
              static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(total_cost))};
}

// Where share b of the work begins: items (pass, split, group) in order, cut
// at equal cost.
struct Place {
  int pass, item;  // item of the pass
};
__device__ __forceinline__ Place share_begin(const MoeParams& p, const Plan& plan, uint32_t b) {
  const uint32_t per_pass = static_cast<uint32_t>(p.splits * p.groups);
  const uint32_t all = plan.cost * per_pass, each = fdiv(all, p.by_grid), rest = all - each * p.by_grid.d;
  const uint32_t x = b * each + min(b, rest);  // < 2^32: the host sees to it
  if (x >= all) return Place{plan.passes, 0};
  // the last pass whose cost begins at or before x
  const int lane = threadIdx.x & 63;
  int pass = -1;
  for (int i0 = 0; i0 < plan.passes; i0 += 64) {
    const bool at = i0 + lane < plan.passes && plan.before[i0 + lane] * per_pass <= x;
    const int found = __popcll(__ballot(at));
    pass += found;
    if (found < 64) break;
  }
  const uint32_t begin = __builtin_amdgcn_readfirstlane(plan.before[pass]);
  const uint32_t end = pass + 1 < plan.passes ? __builtin_amdgcn_readfirstlane(plan.before[pass + 1]) : plan.cost;
  return Place{pass, static_cast<int>((x - begin * per_pass) / (end - begin))};
}

struct Pass {
  int expert, first, tokens;
};
__device__ __forceinline__ Pass read_pass(const uint32_t* list, int i) {
  const uint32_t v = __builtin_amdgcn_readfirstlane(list[i]);
  return Pass{static_cast<int>(v & 1023), static_cast<int>(v >> 10 & 4095), static_cast<int>(v >> 22) + 1};
}

// value of the lane 8 away in the row of 16
__device__ __forceinline__ float swap8(float v) {
  const int i = __builtin_bit_cast(int, v);
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(i, i, 0x128, 0xF, 0xF, false));  // row_ror:8
}

// H as two BF16 planes, `plane` values apart.  The remainder is exact in FP32;
// where the high part is infinite or NaN it adds nothing.
__device__ __forceinline__ void store_h(__bf16* out, size_t plane, float h) {
  const __bf16 top = static_cast<__bf16>(h);
  const float rest = h - static_cast<float>(top);
  out[0] = top;
  out[plane] = static_cast<__bf16>(__builtin_isfinite(rest) ? rest : 0.0f);
}

// ---- one unit of weights times the token rows

// A unit's scales: FP4 16 E4M3 bytes, FP8 one FP32 value.
template <bool FP8>
using Scale = typename std::conditional<FP8, uint32_t, u32x4>::type;

// A lane's part of one unit: chunks g and 4 + g of its row.  The first of each
// four units of a tile also brings the scales of all four, lane group g those
// of unit g: a load per unit would fetch 16 bytes (FP8: 4) of 16 lines each
// time, and cost as much as half the weights (FP4, K = 2880: 40 of 192 us).
template <bool FP8>
struct Unit {
  u32x4 w[2];
  Scale<FP8> sc;
};
// Loads of any Q = 4 units in a row, at least: two each, and the scales of one
// (they come with every fourth unit of a tile, and with its first).
constexpr int kAheadLoads = 2 * Q + 1;

// RING: the weights travel through a private LDS ring instead, Q + 1 slots of a
// unit, by direct loads of 8 rows x 128 bytes, whose requests are whole lines:
// that streams 6.4 TB/s against 5.9 straight into registers (FP8, 16 tokens on
// 128 experts of 4096 x 1024: 177 against 181 us; FP4, 8 tokens on 32 experts
// of 2880 x 2880: 76.5 against 77.7).  It is taken where the token rows leave
// it 80 KiB of LDS: rows that fit only without it would otherwise become more
// passes, each of which reads the weights again.  A row's chunks are loaded in the order chunk ^ (row & 7), so the
// reads are free of bank conflicts.
constexpr uint32_t kSlotBytes = 2048;
constexpr uint32_t kRingBytes = kWaves * (Q + 1) * kSlotBytes;

template <bool RING>
struct Lane {
  uint32_t at, at8;  // offsets in the tile: REG the lane's first chunk; RING its chunks of rows lr and 8 + lr
};
template <bool RING>
__device__ __forceinline__ Lane<RING> lane_offsets(int lane, uint32_t row_bytes, uint32_t half) {
  if constexpr (RING) {
    const uint32_t lr = lane >> 3, lc = lane & 7, at = lr * row_bytes + 16u * (lc ^ lr);
    return Lane<RING>{at, at + half * row_bytes};
  } else {
    const uint32_t li = lane & 15, row = li < 8 ? li : li - 8 + half;
    return Lane<RING>{row * row_bytes + 16u * (lane >> 4), 0u};
  }
}
// asks for unit u of the tile (zeros without `ok`)
template <bool FP8, bool RING>
__device__ __forceinline__ void load_weights(Unit<FP8>& un, rsrc_t r, const Lane<RING>& l, int u, bool ok,
                                             unsigned char* slot) {
  const uint32_t ub = 128u * static_cast<uint32_t>(u);
  if constexpr (RING) {
    buf_load_lds<16>(r, ok ? l.at + ub : kOutOfRange, slot);
    buf_load_lds<16>(r, ok ? l.at8 + ub : kOutOfRange, slot + 1024);
  } else {
    un.w[0] = buf_load_b128(r, ok ? l.at + ub : kOutOfRange);
    un.w[1] = buf_load_b128(r, ok ? l.at + ub + 64u : kOutOfRange);
  }
}
// RING: the oldest unit's weights to registers, with Q units behind it in
// flight; its slot is asked for again a step later
template <bool FP8>
__device__ __forceinline__ void fetch(Unit<FP8>& un, const unsigned char* slot, int li, int g) {
  const int sw = li & 7;
  wait_vm<kAheadLoads>();
  un.w[0] = *reinterpret_cast<const u32x4*>(slot + 128 * li + 16 * (g ^ sw));
  un.w[1] = *reinterpret_cast<const u32x4*>(slot + 128 * li + 16 * ((4 + g) ^ sw));
}

// The scales change lanes through LDS: a wave's slice has the four units'
// scales of 16 rows, the rows kSlicePitch apart.
template <bool FP8>
constexpr uint32_t kSlicePitch = FP8 ? 20 : 80;
template <bool FP8>
constexpr uint32_t kSliceBytes = 16 * kSlicePitch<FP8>;
template <bool FP8>
__device__ __forceinline__ Scale<FP8> unit_scales(const Unit<FP8>& un, unsigned char* slice, int unit, int li, int g) {
  typedef Scale<FP8> S;
  if ((unit & 3) == 0) *reinterpret_cast<S*>(slice + kSlicePitch<FP8> * li + sizeof(S) * g) = un.sc;
  return *reinterpret_cast<const S*>(slice + kSlicePitch<FP8> * li + sizeof(S) * (unit & 3));
}

// Where a lane reads its token rows: window 0 of its row of the first and of
// the second row tile (high plane), the step per window, the way to the other
// plane (both 0 for a lane that reads the zero block throughout), and the zero
// block, for windows past the row.
struct Rows {
  lds_cbytes a[2];
  lds_cbytes zero;
  uint32_t step, plane;
};

// FP4, dense: lane row li carries token li (and 16 + li in the second row
// tile).  Lane group g holds blocks 2g and 2g + 1 of a window; a weight is
// decoded with its block scale: 67 VALU instructions a window for up to 32
// tokens, where the block-diagonal form below takes 33 for 4.
template <typename Tr, int PLANES, int MT>
__device__ __forceinline__ void fp4_dense(f32x4 (&acc)[2], const Unit<false>& un, const u32x4& sc, const Rows& r, int u,
                                          int NW, int len, int g) {
  typedef typename Tr::vec8 V;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int w = 2 * u + h;
    // E4M3 scales of the window's 8 blocks; blocks past the row (the next
    // row's bytes) count as zero
    const uint32_t s_lo = w < NW ? sc[2 * h] : 0u, s_hi = 128 * w + 64 < len ? sc[2 * h + 1] : 0u;
    const uint32_t s2 = ((g & 2) ? s_hi : s_lo) >> (16 * (g & 1));
    const f32x2 sf = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(s2), false);
    const typename Tr::scale_t sa = Tr::make_scale(sf.x), sb = Tr::make_scale(sf.y);
    V b[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) b[i] = Tr::decode8(un.w[h][i], i < 2 ? sa : sb);
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      const lds_cbytes q = w < NW ? r.a[mt] + r.step * static_cast<uint32_t>(w) : r.zero;
      const uint32_t next = w < NW ? r.plane : 0u;
#pragma unroll
      for (int pl = 0; pl < PLANES; ++pl) {
        u32x4 av[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) av[i] = *reinterpret_cast<const lds_u32x4*>(q + pl * next + 16 * i);
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[mt] = Tr::mfma(__builtin_bit_cast(V, av[i]), b[i], acc[mt]);
      }
    }
  }
}

// FP4, block-diagonal, for up to 4 operand rows: row 4 m + q carries row m in
// the k slots of lane group q only, so the lane (n, g) gets row g's dots with
// single blocks, scaled by one FMA each, and the weights are decoded unscaled.
// The sum is acc[0][0].
template <typename Tr, int PLANES>
__device__ __forceinline__ void fp4_diag(f32x4 (&acc)[2], const Unit<false>& un, const u32x4& sc, const Rows& r, int u,
                                         int NW, int len) {
  typedef typename Tr::vec8 V;
  u32x4 av[2][PLANES][4];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int w = 2 * u + h;
    const lds_cbytes q = w < NW ? r.a[0] + r.step * static_cast<uint32_t>(w) : r.zero;
    const uint32_t next = w < NW ? r.plane : 0u;
#pragma unroll
    for (int pl = 0; pl < PLANES; ++pl)
#pragma unroll
      for (int i = 0; i < 4; ++i) av[h][pl][i] = *reinterpret_cast<const lds_u32x4*>(q + pl * next + 16 * i);
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int w = 2 * u + h;
    const uint32_t s_lo = w < NW ? sc[2 * h] : 0u, s_hi = 128 * w + 64 < len ? sc[2 * h + 1] : 0u;
    const f32x2 s01 = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(s_lo), false);
    const f32x2 s23 = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(s_lo), true);
    const f32x2 s45 = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(s_hi), false);
    const f32x2 s67 = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(s_hi), true);
    const float s8[8] = {s01.x, s01.y, s23.x, s23.y, s45.x, s45.y, s67.x, s67.y};
    f32x4 d[2];
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const V b0 = Tr::decode8_fp4(un.w[h][2 * s]), b1 = Tr::decode8_fp4(un.w[h][2 * s + 1]);
      d[s] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int pl = 0; pl < PLANES; ++pl) {
        d[s] = Tr::mfma(__builtin_bit_cast(V, av[h][pl][2 * s]), b0, d[s]);
        d[s] = Tr::mfma(__builtin_bit_cast(V, av[h][pl][2 * s + 1]), b1, d[s]);
      }
    }
    // result row q of set s is block 2q + s
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
      for (int s = 0; s < 2; ++s) acc[0][0] = fmaf(d[s][q], s8[2 * q + s], acc[0][0]);
  }
}

// FP8: a window's sum in a fresh accumulator, added times its FP32 scale.
template <typename Tr, int PLANES, int MT>
__device__ __forceinline__ void fp8_window(f32x4 (&acc)[2], const Unit<true>& un, uint32_t sc, const Rows& r, int u,
                                           int NW, int len) {
  typedef typename Tr::vec8 V;
  // a last window of 64 k: the bytes past the row are the next row's
  const u32x4 w1 = 128 * u + 64 < len ? un.w[1] : u32x4{0u, 0u, 0u, 0u};
  const V b[4] = {Tr::decode8_fp8(un.w[0].x, un.w[0].y), Tr::decode8_fp8(un.w[0].z, un.w[0].w),
                  Tr::decode8_fp8(w1.x, w1.y), Tr::decode8_fp8(w1.z, w1.w)};
  const float s = u < NW ? __builtin_bit_cast(float, sc) : 0.0f;
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
    const lds_cbytes q = u < NW ? r.a[mt] + r.step * static_cast<uint32_t>(u) : r.zero;
    const uint32_t next = u < NW ? r.plane : 0u;
    f32x4 d = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int pl = 0; pl < PLANES; ++pl) {
      u32x4 av[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        av[i] = *reinterpret_cast<const lds_u32x4*>(q + pl * next + (i & 1) * 16 + (i >> 1) * 128);
#pragma unroll
      for (int i = 0; i < 4; ++i) d = Tr::mfma(__builtin_bit_cast(V, av[i]), b[i], d);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[mt][i] = fmaf(d[i], s, acc[mt][i]);
  }
}

// ---------------------------------------------------------------- several tokens

// UP: the first kernel (A of type T against w13), otherwise the second (H
// planes against w2; its operands are BF16 whatever T is).
template <typename T, bool FP8, bool UP, int KS, bool RING>
__global__ __launch_bounds__(kThreads) void moe_kernel(const MoeParams p) {
  typedef typename std::conditional<UP, T, __bf16>::type X;
  typedef ActTraits<X> Tr;
  constexpr int TPW = kWaves / KS;
  constexpr int UK = FP8 ? 128 : 256;  // k of a unit
  constexpr int PLANES = UP ? 1 : 2;
  extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int li = lane & 15, g = lane >> 4;  // row li, chunk group g
  const int ks = wave % KS, tw = wave / KS;
  unsigned char* slice = smem + static_cast<uint32_t>(wave) * kSliceBytes<FP8>;
  unsigned char* slots = smem + kWaves * kSliceBytes<FP8> + static_cast<uint32_t>(wave) * ((Q + 1) * kSlotBytes);
  unsigned char* red = smem + kWaves * kSliceBytes<FP8> + (RING ? kRingBytes : 0u);
  const uint32_t red_stride = red_stride_of(FP8, p.rows);
  unsigned char* plan_mem = red + (KS > 1 ? 2u * kWaves * red_stride : 0u);
  unsigned char* rows_lds = plan_mem + plan_bytes(p.n, p.E, p.list_max);
  const Plan plan = p.n <= kWavePlan ? make_plan_wave(p, plan_mem) : make_plan(p, plan_mem);

  // This workgroup's share.  (pass, split) pairs are counted through: part v is
  // split v % splits of pass v / splits.
  const Place from = share_begin(p, plan, blockIdx.x), to = share_begin(p, plan, blockIdx.x + 1);
  const int per_pass = p.splits * p.groups;
  const int items = (to.pass - from.pass) * per_pass + to.item - from.item;
  if (items == 0) return;  // the whole workgroup
  const int first_split = static_cast<int>(fdiv(static_cast<uint32_t>(from.item), p.by_groups));
  const int first_part = from.pass * p.splits + first_split, first_group = from.item - first_split * p.groups;
  const int last_part = first_part + static_cast<int>(fdiv(static_cast<uint32_t>(first_group + items - 1), p.by_groups));
  const int total = items * p.units;

  const int split_k = p.split_units * UK;
  const uint32_t row_bytes = FP8 ? static_cast<uint32_t>(p.L) : static_cast<uint32_t>(p.L >> 1);
  const uint32_t srow_bytes = FP8 ? 4u * p.cols : static_cast<uint32_t>(p.cols);
  const uint32_t half = UP ? static_cast<uint32_t>(p.N >> 1) : 8u;  // weight rows from a tile's first 8 to its last 8
  const uint32_t tile_rows = UP ? 8u : 16u;
  const uint32_t pitch = 16u * p.chunks_per_row.d;  // LDS bytes of a token row: whole units and 16
  const uint32_t buffer_bytes = (static_cast<uint32_t>(PLANES * p.rows) * pitch + 256u + 1023u) & ~1023u;
  const rsrc_t x_rsrc = make_rsrc(p.x, static_cast<uint32_t>(p.x_bytes));
  const Lane<RING> lane_at = lane_offsets<RING>(lane, row_bytes, half);
  const uint32_t sl = (li < 8 ? li : li - 8 + half) * srow_bytes;

  // ---- load side
  int l_part = first_part, l_group = first_group, l_unit = 0;
  int l_left = items;  // groups still to load, the current one included
  int l_expert = 0, l_split = 0;
  auto set_part = [&]() {
    const int pass = static_cast<int>(fdiv(static_cast<uint32_t>(l_part), p.by_splits));
    l_expert = read_pass(plan.list, pass).expert;
    l_split = l_part - pass * p.splits;
  };
  set_part();
  rsrc_t br, sr;
  auto set_load_tile = [&]() {
    const int t = l_group * TPW + tw;
    const bool on = l_left > 0 && t < p.tiles;  // past the last tile or the share: every load reads zeros
    const int64_t row = static_cast<int64_t>(l_expert) * p.N + static_cast<int64_t>(on ? t : 0) * tile_rows;
    const uint32_t span = on ? half + 8u : 0u, skip = on ? 128u * p.split_units * l_split : 0u;
    br = make_rsrc(p.w + row * row_bytes + skip, span * row_bytes - skip);
    sr = make_rsrc(p.s + row * srow_bytes, span * srow_bytes);
  };
  set_load_tile();
  auto load = [&](Unit<FP8>& un, unsigned char* slot) {
    const int u = ks * p.units + l_unit, v = u + l_split * p.split_units;  // unit of the part, and of the row
    const bool ok = u < p.split_units && v * UK < p.L;
    if ((l_unit & 3) == 0) {
      // (units past the row: bytes of the next row, or zeros; not used)
      if constexpr (FP8) {
        const uint32_t col = min(fdiv(static_cast<uint32_t>(v + g), p.win_per_block), static_cast<uint32_t>(p.cols - 1));
        un.sc = buf_load_b32(sr, sl + 4u * col);
      } else {
        un.sc = buf_load_b128(sr, sl + 16u * static_cast<uint32_t>(v + g));
      }
    }
    load_weights<FP8, RING>(un, br, lane_at, u, ok, slot);
    if (++l_unit == p.units) {
      l_unit = 0;
      --l_left;
      if (++l_group == p.groups) {
        l_group = 0;
        ++l_part;
        if (l_left > 0) set_part();
      }
      set_load_tile();
    }
  };

  // ---- token rows of a part, by direct loads: LDS chunk q holds row q /
  // chunks_per_row (down: the high parts of all tokens, then the remainders),
  // then 256 bytes of zeros; the zeros, rows' padding and the tail of the last
  // instruction are out-of-range reads, which write zeros
  auto fill = [&](const Pass& ps, int split, int buf) {
    const uint32_t cpr = p.chunks_per_row.d;
    const uint32_t data = static_cast<uint32_t>(PLANES * ps.tokens) * cpr, chunks = data + 16u;
    const uint32_t k0 = static_cast<uint32_t>(split * split_k);
    for (uint32_t q0 = 64u * static_cast<uint32_t>(wave); q0 < chunks; q0 += 64u * kWaves) {
      const uint32_t q = q0 + static_cast<uint32_t>(lane);
      const uint32_t row = fdiv(q, p.chunks_per_row), col = q - row * cpr;
      uint32_t src = kOutOfRange;
      if (q < data && col + 1u < cpr && k0 + col * 8u < static_cast<uint32_t>(p.L)) {
        uint32_t r;
        if constexpr (UP) {
          r = fdiv(plan.sorted[ps.first + row], p.topk);
        } else {
          const bool rest = row >= static_cast<uint32_t>(ps.tokens);
          r = plan.sorted[ps.first + (rest ? row - ps.tokens : row)] + (rest ? static_cast<uint32_t>(p.n) : 0u);
        }
        src = 2u * (r * static_cast<uint32_t>(p.L) + k0) + 16u * col;
      }
      buf_load_lds<16>(x_rsrc, src, rows_lds + buf * buffer_bytes + 16u * q0);
    }
  };

  // ---- the part being multiplied
  f32x4 acc[2] = {f32x4{0.f, 0.f, 0.f, 0.f}, f32x4{0.f, 0.f, 0.f, 0.f}};
  int c_part = first_part, c_group = first_group, c_unit = 0;
  uint32_t turn = 0;
  Pass ps;
  int c_split, len, NW;  // k of the row in this part, and its windows
  int buf = 0, since = 0;
  bool diag;
  Rows rows;
  float gs = 1.0f;  // FP4: the expert's FP32 scale
  auto set_current = [&]() {
    const int pass = static_cast<int>(fdiv(static_cast<uint32_t>(c_part), p.by_splits));
    ps = read_pass(plan.list, pass);
    c_split = c_part - pass * p.splits;
    len = min(split_k, p.L - c_split * split_k);
    NW = (len + 127) >> 7;
    // dense (and FP8) rows past the part's tokens repeat the last one, and
    // their results are dropped
    const lds_cbytes base = (lds_cbytes)(rows_lds + buf * buffer_bytes);
    const uint32_t plane = static_cast<uint32_t>(ps.tokens) * pitch;
    rows.zero = base + PLANES * plane;
    diag = !FP8 && ps.tokens <= 4;
    const bool carries = !diag || ((li & 3) == g && (li >> 2) < ps.tokens);
    const uint32_t off = (FP8 ? 32u : 64u) * g;
    const int m = diag ? li >> 2 : min(li, ps.tokens - 1);
    rows.a[0] = carries ? base + static_cast<uint32_t>(m) * pitch + off : rows.zero;
    rows.a[1] = base + static_cast<uint32_t>(min(16 + li, ps.tokens - 1)) * pitch + off;
    rows.step = carries ? 256u : 0u;
    rows.plane = carries ? plane : 0u;
    // a scalar load: a vector load would wait for the weight loads before it
    if constexpr (!FP8)
      gs = reinterpret_cast<const __attribute__((address_space(4))) float*>(reinterpret_cast<uintptr_t>(p.g))[ps.expert];
  };
  // the rows of the part after this one, into the other buffer
  auto prefetch = [&]() {
    since = 0;
    if (p.buffers == 2 && c_part < last_part) {
      const int pass = static_cast<int>(fdiv(static_cast<uint32_t>(c_part + 1), p.by_splits));
      // the fences keep the unit loads on their side of it: `since` counts those after it
      __asm__ volatile("" ::: "memory");
      fill(read_pass(plan.list, pass), c_part + 1 - pass * p.splits, buf ^ 1);
      __asm__ volatile("" ::: "memory");
    }
  };
  Unit<FP8> ring[Q];
  set_current();
  fill(ps, c_split, 0);
#pragma unroll
  for (int q = 0; q < Q; ++q) load(ring[q], slots + q * kSlotBytes);
  wait_vm<kAheadLoads>();  // the rows are older
  __builtin_amdgcn_s_barrier();
  __asm__ volatile("" ::: "memory");
  prefetch();

  auto multiply = [&](const Unit<FP8>& un, const Scale<FP8>& sc) {
    const int u = ks * p.units + c_unit;
    if constexpr (FP8) {
      if (ps.tokens > 16)
        fp8_window<Tr, PLANES, 2>(acc, un, sc, rows, u, NW, len);
      else
        fp8_window<Tr, PLANES, 1>(acc, un, sc, rows, u, NW, len);
    } else {
      if (diag)
        fp4_diag<Tr, PLANES>(acc, un, sc, rows, u, NW, len);
      else if (ps.tokens > 16)
        fp4_dense<Tr, PLANES, 2>(acc, un, sc, rows, u, NW, len, g);
      else
        fp4_dense<Tr, PLANES, 1>(acc, un, sc, rows, u, NW, len, g);
    }
  };

  // join the K split of a tile and write it
  auto finish = [&]() {
    if (KS > 1) {
      // The two halves of `red` are used in turn, so one barrier is enough: a
      // half is written again after a barrier that its readers reach later.
      // Two row tiles take both halves, between barriers.
      const bool two = ps.tokens > 16;
      unsigned char* part = red + (two ? 0u : turn) * (kWaves * red_stride) + wave * red_stride;
      turn ^= 1;
      if (two) lds_barrier();
      if (diag) {
        reinterpret_cast<float*>(part)[lane] = acc[0][0];
      } else {
        reinterpret_cast<f32x4*>(part)[lane] = acc[0];
        if (two) reinterpret_cast<f32x4*>(part + kWaves * red_stride)[lane] = acc[1];
      }
      lds_barrier();
      if (ks == 0) {
#pragma unroll
        for (int v = 1; v < KS; ++v) {
          const unsigned char* q = part + v * red_stride;
          if (diag) {
            acc[0][0] += reinterpret_cast<const float*>(q)[lane];
          } else {
            acc[0] += reinterpret_cast<const f32x4*>(q)[lane];
            if (two) acc[1] += reinterpret_cast<const f32x4*>(q + kWaves * red_stride)[lane];
          }
        }
      }
      if (two) lds_barrier();
    }
    const int t = c_group * TPW + tw;
    if (ks == 0 && t < p.tiles) {
      auto write = [&](float v, int row) {
        if constexpr (UP) {
          const float up = swap8(v);
          if (row < ps.tokens && li < 8) {
            const size_t at = static_cast<size_t>(plan.sorted[ps.first + row]) * (p.N >> 1) + 8 * t + li;
            store_h(static_cast<__bf16*>(p.out) + at, static_cast<size_t>(p.n) * (p.N >> 1),
                    gated(p.act, v * gs, up * gs));
          }
        } else if (row < ps.tokens) {
          const size_t at = static_cast<size_t>(c_split) * p.n + plan.sorted[ps.first + row];
          static_cast<float*>(p.out)[at * p.N + 16 * t + li] = v * gs;
        }
      };
      if (diag) {
        write(acc[0][0], g);
      } else {
#pragma unroll
        for (int r = 0; r < 4; ++r) write(acc[0][r], 4 * g + r);
        if (ps.tokens > 16) {
#pragma unroll
          for (int r = 0; r < 4; ++r) write(acc[1][r], 16 + 4 * g + r);
        }
      }
    }
    acc[0] = f32x4{0.f, 0.f, 0.f, 0.f};
    acc[1] = f32x4{0.f, 0.f, 0.f, 0.f};
  };

  // the next part's rows take over
  auto next_part = [&]() {
    if (p.buffers == 2) {
      // asked for when this part began; newer are the unit loads since
      if (since >= Q)
        wait_vm<kAheadLoads>();
      else
        wait_vm<0>();
      buf ^= 1;
      set_current();
      lds_barrier();  // every wave's rows have landed, and the other buffer is free
      prefetch();
    } else {
      set_current();
      lds_barrier();  // the last part's rows are read
      fill(ps, c_split, 0);
      wait_vm<0>();
      __builtin_amdgcn_s_barrier();
      __asm__ volatile("" ::: "memory");
    }
  };

  // Units past the end of the share are out-of-range loads, and not
  // multiplied.  No way leaves the loop body before its end: it would merge
  // with the others at the loop head and make every wait there a full one.
  int l_slot = Q, c_slot = 0;  // RING: the slot to ask for next, and the oldest
  for (int f0 = 0; f0 < total; f0 += Q) {
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      const bool on = f0 + q < total;  // uniform across the workgroup
      const Scale<FP8> sc = unit_scales<FP8>(ring[q], slice, c_unit, li, g);
      if constexpr (RING) {
        // the slot that is asked for was read a step ago, and those reads are
        // done: their values have been multiplied
        load(ring[q], slots + l_slot * kSlotBytes);
        Unit<FP8> now;
        fetch<FP8>(now, slots + c_slot * kSlotBytes, li, g);
        l_slot = l_slot == Q ? 0 : l_slot + 1;
        c_slot = c_slot == Q ? 0 : c_slot + 1;
        if (on) multiply(now, sc);
      } else {
        if (on) multiply(ring[q], sc);
        load(ring[q], slots);
      }
      if (on) {
        ++since;
        if (++c_unit == p.units) {
          c_unit = 0;
          finish();
          if (++c_group == p.groups) {
            c_group = 0;
            if (++c_part <= last_part) next_part();
          }
        }
      }
    }
  }
}

// ---------------------------------------------------------------- one token

constexpr uint32_t kTokenRedBytes = 1024;  // 2 x 8 waves x 16 floats

// M = 1: assignment j is choice j of the only token, so no plan is made: a
// pass is a choice, its token row is A for every choice (up) and row j of H
// (down).  What counts is the chain of latencies (launch, ids, first weights,
// join), so up shares out (choice, tile group) pairs to as many workgroups as
// the chip holds, and down gives a workgroup whole column tiles, with the
// choices spread over its waves, and adds them up itself: no third kernel.
//
// In down the two planes of H are two rows of one operand, not two MFMAs.

// up: grid-stride over (choice, group); down: over tiles.
template <typename T, bool FP8, bool UP, int KS, bool RING>
__global__ __launch_bounds__(kThreads) void moe_token_kernel(const MoeParams p, const float* __restrict__ weights) {
  typedef typename std::conditional<UP, T, __bf16>::type X;
  typedef ActTraits<X> Tr;
  constexpr int TPW = kWaves / KS;  // up: tiles side by side; down: choices side by side
  constexpr int UW = FP8 ? 1 : 2;  // windows of a unit
  constexpr int ROWS = UP ? 1 : 2;  // operand rows of a choice
  extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int li = lane & 15, g = lane >> 4;
  const int ks = wave % KS, tw = wave / KS;
  unsigned char* slice = smem + static_cast<uint32_t>(wave) * kSliceBytes<FP8>;
  unsigned char* slots = smem + kWaves * kSliceBytes<FP8> + static_cast<uint32_t>(wave) * ((Q + 1) * kSlotBytes);
  unsigned char* red = smem + kWaves * kSliceBytes<FP8> + (RING ? kRingBytes : 0u);
  unsigned char* rows_lds = red + kTokenRedBytes;
  const int NW = (p.L + 127) >> 7;
  const int NU = (NW + UW - 1) / UW;
  const uint32_t row_bytes = FP8 ? static_cast<uint32_t>(p.L) : static_cast<uint32_t>(p.L >> 1);
  const uint32_t srow_bytes = FP8 ? 4u * p.cols : static_cast<uint32_t>(p.cols);
  const uint32_t half = UP ? static_cast<uint32_t>(p.N >> 1) : 8u;
  const uint32_t tile_rows = UP ? 8u : 16u;
  const uint32_t pitch = static_cast<uint32_t>(NW) * 256u + 16u;  // LDS bytes of a row
  const Lane<RING> lane_at = lane_offsets<RING>(lane, row_bytes, half);
  const uint32_t sl = (li < 8 ? li : li - 8 + half) * srow_bytes;

  // The wave's sequence.  up: items (choice, group) b, b + grid, ..; wave
  // (tw, ks) takes tile group * TPW + tw.  down: tiles b, b + grid, .. and in
  // each the choices tw, tw + TPW, ..
  const int inner = UP ? 1 : (p.n + TPW - 1) / TPW;  // choices of a wave per tile
  const int items = UP ? p.n * p.groups : p.tiles;
  const int mine = items > static_cast<int>(blockIdx.x)
                       ? (items - static_cast<int>(blockIdx.x) + static_cast<int>(gridDim.x) - 1) / static_cast<int>(gridDim.x)
                       : 0;
  const int total = mine * inner * p.units;

  int l_item = blockIdx.x, l_in = 0, l_unit = 0;
  rsrc_t br, sr;
  auto choice_of = [&](int item, int in) { return UP ? item / p.groups : tw + in * TPW; };
  auto tile_of = [&](int item) { return UP ? item % p.groups * TPW + tw : item; };
  // Lane j holds choice j (topk <= 64): its expert, -1 where there is none,
  // the expert's FP32 scale and the choice's weight.  The last two are not
  // waited for here.
  int e_lane = lane < p.n ? p.ids[lane] : -1;
  if (static_cast<uint32_t>(e_lane) >= static_cast<uint32_t>(p.E)) e_lane = -1;
  float g_lane = !FP8 && e_lane >= 0 ? p.g[e_lane] : 1.0f;
  float w_lane = !UP && lane < p.n ? weights[lane] : 0.0f;
  auto expert_of = [&](int j) { return j < p.n ? __builtin_amdgcn_readlane(e_lane, j) : -1; };
  auto value_of = [&](float v, int j) {
    return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), j));
  };
  auto set_load_tile = [&]() {
    const int t = tile_of(l_item);
    const int e = l_item < items ? expert_of(choice_of(l_item, l_in)) : -1;
    const bool on = e >= 0 && t < p.tiles;
    const int64_t row = static_cast<int64_t>(on ? e : 0) * p.N + static_cast<int64_t>(on ? t : 0) * tile_rows;
    const uint32_t span = on ? half + 8u : 0u;
    br = make_rsrc(p.w + row * row_bytes, span * row_bytes);
    sr = make_rsrc(p.s + row * srow_bytes, span * srow_bytes);
  };
  set_load_tile();
  auto load = [&](Unit<FP8>& un, unsigned char* slot) {
    const int u = ks * p.units + l_unit;
    const bool ok = u < NU;
    if ((l_unit & 3) == 0) {
      if constexpr (FP8) {
        const uint32_t col = min(fdiv(static_cast<uint32_t>(u + g), p.win_per_block), static_cast<uint32_t>(p.cols - 1));
        un.sc = buf_load_b32(sr, sl + 4u * col);
      } else {
        un.sc = buf_load_b128(sr, sl + 16u * static_cast<uint32_t>(u + g));
      }
    }
    load_weights<FP8, RING>(un, br, lane_at, u, ok, slot);
    if (++l_unit == p.units) {
      l_unit = 0;
      if (++l_in == inner) {
        l_in = 0;
        l_item += gridDim.x;
      }
      set_load_tile();
    }
  };

  f32x4 acc[2] = {f32x4{0.f, 0.f, 0.f, 0.f}, f32x4{0.f, 0.f, 0.f, 0.f}};
  float sum = 0.0f;  // down: the weighted choices of this wave, lanes g == 0
  Unit<FP8> ring[Q];
  int c_item = blockIdx.x, c_in = 0, c_unit = 0, turn = 0;
  // up: the token's row; down: the high parts of all choices, then the
  // remainders (rows of choices without an expert hold anything: their
  // results are dropped)
  {
    const rsrc_t x_rsrc = make_rsrc(p.x, static_cast<uint32_t>(p.x_bytes));
    const uint32_t cpr = p.chunks_per_row.d;
    const uint32_t data = (UP ? 1u : 2u * p.n) * cpr, chunks = data + 16u;  // and the zero block
    for (uint32_t q0 = 64u * static_cast<uint32_t>(wave); q0 < chunks; q0 += 64u * kWaves) {
      const uint32_t q = q0 + static_cast<uint32_t>(lane);
      const uint32_t row = fdiv(q, p.chunks_per_row), col = q - row * cpr;
      const bool in = q < data && col * 8u < static_cast<uint32_t>(p.L);
      buf_load_lds<16>(x_rsrc, in ? row * (2u * p.L) + 16u * col : kOutOfRange, rows_lds + 16u * q0);
    }
  }
#pragma unroll
  for (int q = 0; q < Q; ++q) load(ring[q], slots + q * kSlotBytes);
  wait_vm<kAheadLoads>();  // the rows, scales and weights are older
  __asm__ volatile("" : "+v"(g_lane), "+v"(w_lane));
  __builtin_amdgcn_s_barrier();
  __asm__ volatile("" ::: "memory");

  auto consume = [&](const Unit<FP8>& un, const Scale<FP8>& sc) {
    const int u = ks * p.units + c_unit;
    const int j = choice_of(c_item, c_in);
    // row m of the operand: up 0: the token; down 0 and 1: the choice's two
    // planes.  FP4: block-diagonal, so lane groups 0 and 1 end with the rows'
    // sums in acc[0]; FP8: lane rows m, group 0 ends with them in acc[0 ..].
    const int m = FP8 ? li & (ROWS - 1) : li >> 2;
    const bool carries = FP8 || ((li & 3) == g && m < ROWS);
    const lds_cbytes base = (lds_cbytes)rows_lds;
    const uint32_t row = UP ? 0u : static_cast<uint32_t>(m * p.n + min(j, p.n - 1));
    Rows rows;
    rows.zero = base + static_cast<uint32_t>(UP ? 1 : 2 * p.n) * pitch;
    rows.a[0] = carries ? base + row * pitch + (FP8 ? 32u : 64u) * g : rows.zero;
    rows.step = carries ? 256u : 0u;
    rows.plane = 0u;
    if constexpr (FP8)
      fp8_window<Tr, 1, 1>(acc, un, sc, rows, u, NW, p.L);
    else
      fp4_diag<Tr, 1>(acc, un, sc, rows, u, NW, p.L);
    if (++c_unit < p.units) return;
    c_unit = 0;
    const int e = expert_of(j);
    float v = acc[0][0];  // lanes g == 0 hold the tile
    if (!UP) v += FP8 ? acc[0][1] : __shfl_xor(acc[0][0], 16, 64);
    acc[0] = f32x4{0.f, 0.f, 0.f, 0.f};
    if constexpr (!UP) {
      if (e >= 0) sum = fmaf(v * value_of(g_lane, j), value_of(w_lane, j), sum);
      if (++c_in < inner) return;
      c_in = 0;
      v = sum;
      sum = 0.0f;
    }
    // join: up the K split of a tile, down the waves' choices (and K splits),
    // each in the order of the waves; the two halves of `red` are used in
    // turn, so one barrier is enough
    float* part = reinterpret_cast<float*>(red) + 128 * turn;
    const int joined = UP ? KS : kWaves;
    if (joined > 1) {
      turn ^= 1;
      if (g == 0) part[16 * wave + li] = v;
      lds_barrier();
    }
    if ((UP ? ks : wave) == 0 && g == 0) {
      if (joined > 1) {
        v = 0.0f;
#pragma unroll
        for (int i = 0; i < (UP ? KS : kWaves); ++i) v += part[16 * (wave + i) + li];
      }
      const int t = tile_of(c_item);
      if (UP) {
        const float up = swap8(v);
        if (e >= 0 && t < p.tiles && li < 8) {
          const float gs = value_of(g_lane, j);
          store_h(static_cast<__bf16*>(p.out) + static_cast<size_t>(j) * (p.N >> 1) + 8 * t + li,
                  static_cast<size_t>(p.n) * (p.N >> 1), gated(p.act, v * gs, up * gs));
        }
      } else {
        static_cast<T*>(p.out)[16 * t + li] = round_to<T>(v);
      }
    }
    c_item += gridDim.x;
  };

  int l_slot = Q, c_slot = 0;  // RING: the slot to ask for next, and the oldest
  for (int f0 = 0; f0 < total; f0 += Q) {
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      const bool on = f0 + q < total;  // uniform across the workgroup
      const Scale<FP8> sc = unit_scales<FP8>(ring[q], slice, c_unit, li, g);
      if constexpr (RING) {
        // the slot that is asked for was read a step ago, and those reads are
        // done: their values have been multiplied
        load(ring[q], slots + l_slot * kSlotBytes);
        Unit<FP8> now;
        fetch<FP8>(now, slots + c_slot * kSlotBytes, li, g);
        l_slot = l_slot == Q ? 0 : l_slot + 1;
        c_slot = c_slot == Q ? 0 : c_slot + 1;
        if (on) consume(now, sc);
      } else {
        if (on) consume(ring[q], sc);
        load(ring[q], slots);
      }
    }
  }
}

// ---------------------------------------------------------------- combine

// Y[m, c .. c + 3] = sum over j of weights[a] * (sum over s of P[s][a, c ..]), a = m * topk + j, in order.
// A few microseconds of latency at these sizes: eight choices' loads at a
// time, none of them behind a branch.  A masked choice reads the token's first
// one instead of its own and does not use it: 100 tokens with three choices in
// four masked take 95.5 us instead of 98.5, where none is masked nothing is lost.
template <typename T>
__global__ __launch_bounds__(256) void moe_combine_kernel(const float* __restrict__ P, const int32_t* __restrict__ ids,
                                                          const float* __restrict__ weights, T* __restrict__ Y, int M,
                                                          int K, int topk, int E, int splits, FastDiv chunks) {
  typedef typename ActTraits<T>::vec8 V;
  const uint32_t all = static_cast<uint32_t>(M) * chunks.d;  // chunks of 4 columns
  const size_t part = static_cast<size_t>(M) * topk * K;     // of one split
  for (uint32_t i = blockIdx.x * 256u + threadIdx.x; i < all; i += 256u * gridDim.x) {
    const uint32_t m = fdiv(i, chunks), c = i - m * chunks.d;
    const float* q = P + static_cast<size_t>(m) * topk * K + 4 * c;
    f32x4 sum = f32x4{0.f, 0.f, 0.f, 0.f};
    for (int j0 = 0; j0 < topk; j0 += 8) {
      f32x4 x[8];
      float w[8];
      bool on[8];
      size_t at[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int k = min(j0 + j, topk - 1);
        w[j] = weights[m * topk + k];
        on[j] = j0 + j < topk && static_cast<uint32_t>(ids[m * topk + k]) < static_cast<uint32_t>(E);
        at[j] = on[j] ? static_cast<size_t>(k) * K : 0;
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = *reinterpret_cast<const f32x4*>(q + at[j]);
      for (int s = 1; s < splits; ++s) {
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] += *reinterpret_cast<const f32x4*>(q + s * part + at[j]);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int k = 0; k < 4; ++k) sum[k] = on[j] ? fmaf(x[j][k], w[j], sum[k]) : sum[k];
    }
    V r;
#pragma unroll
    for (int k = 0; k < 4; ++k) r[k] = round_to<T>(sum[k]);
    const u32x4 bits = __builtin_bit_cast(u32x4, r);
    *reinterpret_cast<u32x2*>(Y + static_cast<size_t>(m) * K + 4 * c) = u32x2{bits.x, bits.y};
  }
}

// --------------------------------------------------------------------- launch

constexpr size_t kMaxLds = 160 * 1024;

// Dynamic LDS above 64 KiB must be allowed per kernel, once per device.
template <auto KERNEL>
void allow_lds() {
  static std::once_flag once[kMaxDevices];
  once_per_device(once, [] {
    (void)hipFuncSetAttribute(reinterpret_cast<const void*>(KERNEL), hipFuncAttributeMaxDynamicSharedMemorySize,
                              static_cast<int>(kMaxLds));
  });
}

struct Shape {
  int rows, buffers, splits, split_units, ks, grid, units, groups, list_max;
  bool ring;
  size_t lds;
};

// Token rows of `planes` planes and the zero block, in whole direct-load
// instructions (the kernel's buffer_bytes).
size_t rows_lds_bytes(int64_t rows, int planes, int windows) {
  return (static_cast<size_t>(rows) * planes * (static_cast<size_t>(windows) * 256 + 16) + 256 + 1023) / 1024 * 1024;
}

// The K split of a tile over KS waves.  The larger it is, the smaller the
// groups of tiles that are shared out and the better the shares' bytes match,
// but every tile then ends with a join.  Measured, us of a layer with the split
// of up at 1, 2, 4 and 8: FP4 K = 7168, 28 units of a row: 142.6, 135.8, 135.4,
// 133.9; FP4 K = 2048, 8 units: 76.4, 75.9, 83.0, 99.3; FP8 K = 4096, 32 units:
// 180.6, 176.7, 175.5, 178.0; FP4 K = 2880, 12 units: 183, 185, 209, 255.  And
// with that of down at 2 and 4: FP8 I = 1024, 8 units: 178.2, 181.9; FP8 I =
// 1280, 10 units: 99.1, 116.4.  So: the largest split that leaves a wave four
// units of a tile, and beyond that only as far as the workgroups would not
// fill the chip.  It is not the best of every row: FP4 K = 2880 gets 2 (1 is 1.1 %
// faster), FP8 K = 4096 gets 8 (4 is 1.4 %), FP4 K = 7168 gets 4 (8 is 1.1 %).
int k_split(int NU, int64_t tiles, int64_t passes, int64_t cus) {
  int ks = 1;
  while (ks < kWaves && NU >= 8 * ks) ks *= 2;
  while (ks < kWaves && NU >= 2 * ks && passes * ((tiles + kWaves / ks - 1) / (kWaves / ks)) < cus) ks *= 2;
  return ks;
}

// The launch of one kernel for several tokens.  False when not even one token
// row fits.
bool plan_shape(const MoeArgs& a, bool fp8, bool up, Shape* out) {
  const int64_t n = a.M * a.topk, L = up ? a.K : a.I;
  const int uk = fp8 ? 128 : 256, NU = static_cast<int>((L + uk - 1) / uk), planes = up ? 1 : 2;
  // Tokens per pass: an expert's tokens beyond `rows` read its weights again;
  // twice the mean and a few more is rarely exceeded.
  const int64_t mean = a.E > 0 ? (n + a.E - 1) / a.E : n;
  const int64_t want = std::max<int64_t>(1, std::min<int64_t>({2 * mean + 4, kMaxRows, a.M}));
  // Rows that fit: first with two buffers, then with one, then (down) with the
  // sum in parts, then fewer rows.
  const int max_splits = up ? 1 : static_cast<int>(moe_down_splits(a.M, a.I));
  const int64_t passes = std::min<int64_t>(n, a.E);
  const size_t slices = kWaves * (fp8 ? kSliceBytes<true> : kSliceBytes<false>);
  auto fits = [&](int64_t rows, int buffers, int splits, bool ring) {
    const int units = (NU + splits - 1) / splits;
    const int64_t list_max = passes + n / rows;
    const size_t lds = slices + (ring ? kRingBytes : 0u) + 2 * kWaves * red_stride_of(fp8, static_cast<int>(rows)) +
                       plan_bytes(static_cast<int>(n), static_cast<int>(a.E), static_cast<int>(list_max)) +
                       buffers * rows_lds_bytes(rows, planes, units * (uk / 128));
    if (lds > kMaxLds) return false;
    *out = Shape{static_cast<int>(rows), buffers, (NU + units - 1) / units, units, 1, 1, 1, 1, static_cast<int>(list_max), ring, lds};
    return true;
  };
  bool ok = fits(want, 2, 1, true) || fits(want, 1, 1, true) || fits(want, 2, 1, false);
  for (int s = 1; !ok && s <= max_splits; ++s) ok = fits(want, 1, s, false);
  for (int64_t rows = want - 1; !ok && rows >= 1; --rows) ok = fits(rows, 1, max_splits, false);
  if (!ok) return false;
  const int64_t tiles = up ? a.I / 8 : a.K / 16, cus = device_cus();
  out->ks = k_split(out->split_units, tiles, passes * out->splits, cus);
  const int64_t groups = (tiles + kWaves / out->ks - 1) / (kWaves / out->ks);
  // the shares are counted in 32 bits
  if (out->list_max * out->splits * groups * kMostCost >= (int64_t(1) << 31)) return false;
  out->groups = static_cast<int>(groups);
  out->units = (out->split_units + out->ks - 1) / out->ks;
  out->grid = static_cast<int>(std::min(passes * out->splits * groups, cus));
  return true;
}

template <typename T, bool FP8, bool UP, int KS, bool RING>
void launch_ring(const MoeParams& p, const Shape& s, hipStream_t st) {
  allow_lds<&moe_kernel<T, FP8, UP, KS, RING>>();
  hipLaunchKernelGGL((moe_kernel<T, FP8, UP, KS, RING>), dim3(s.grid), dim3(kThreads), s.lds, st, p);
}
template <typename T, bool FP8, bool UP, int KS>
void launch_kernel(const MoeParams& p, const Shape& s, hipStream_t st) {
  s.ring ? launch_ring<T, FP8, UP, KS, true>(p, s, st) : launch_ring<T, FP8, UP, KS, false>(p, s, st);
}

template <typename T, bool FP8, bool UP>
void launch_phase(MoeParams p, const Shape& s, hipStream_t st) {
  p.rows = s.rows;
  p.buffers = s.buffers;
  p.splits = s.splits;
  p.split_units = s.split_units;
  p.groups = s.groups;
  p.units = s.units;
  p.list_max = s.list_max;
  p.fp8 = FP8;
  p.by_rows = make_fastdiv(static_cast<uint32_t>(s.rows));
  p.by_grid = make_fastdiv(static_cast<uint32_t>(s.grid));
  p.by_groups = make_fastdiv(static_cast<uint32_t>(s.groups));
  p.by_splits = make_fastdiv(static_cast<uint32_t>(s.splits));
  p.chunks_per_row = make_fastdiv(static_cast<uint32_t>(s.split_units * (FP8 ? 16 : 32) + 1));
  switch (s.ks) {
    case 1: launch_kernel<T, FP8, UP, 1>(p, s, st); break;
    case 2: launch_kernel<T, FP8, UP, 2>(p, s, st); break;
    case 4: launch_kernel<T, FP8, UP, 4>(p, s, st); break;
    default: launch_kernel<T, FP8, UP, 8>(p, s, st); break;
  }
}

template <typename T, bool FP8, bool UP, int KS, bool RING>
void launch_token_ring(const MoeParams& p, const float* weights, int grid, size_t lds, hipStream_t st) {
  allow_lds<&moe_token_kernel<T, FP8, UP, KS, RING>>();
  hipLaunchKernelGGL((moe_token_kernel<T, FP8, UP, KS, RING>), dim3(grid), dim3(kThreads), lds, st, p, weights);
}
template <typename T, bool FP8, bool UP, int KS>
void launch_token_kernel(const MoeParams& p, const float* weights, int grid, size_t lds, hipStream_t st) {
  if (lds + kRingBytes <= kMaxLds)
    launch_token_ring<T, FP8, UP, KS, true>(p, weights, grid, lds + kRingBytes, st);
  else
    launch_token_ring<T, FP8, UP, KS, false>(p, weights, grid, lds, st);
}

template <typename T, bool FP8, bool UP>
void launch_token_ks(const MoeParams& p, const float* weights, int ks, int grid, size_t lds, hipStream_t st) {
  switch (ks) {
    case 1: launch_token_kernel<T, FP8, UP, 1>(p, weights, grid, lds, st); break;
    case 2: launch_token_kernel<T, FP8, UP, 2>(p, weights, grid, lds, st); break;
    case 4: launch_token_kernel<T, FP8, UP, 4>(p, weights, grid, lds, st); break;
    default: launch_token_kernel<T, FP8, UP, 8>(p, weights, grid, lds, st); break;
  }
}

// M = 1.  False where the rows do not fit in LDS.
template <typename T, bool FP8>
bool launch_token(const MoeArgs& a, MoeParams up, MoeParams down, hipStream_t st) {
  const int cus = device_cus();
  const int up_nw = static_cast<int>((a.K + 127) / 128), down_nw = static_cast<int>((a.I + 127) / 128);
  const size_t base = kWaves * kSliceBytes<FP8> + kTokenRedBytes;
  const size_t up_lds = base + rows_lds_bytes(1, 1, up_nw);
  const size_t down_lds = base + rows_lds_bytes(static_cast<int>(a.topk), 2, down_nw);
  if (up_lds > kMaxLds || down_lds > kMaxLds) return false;
  const int up_nu = FP8 ? up_nw : (up_nw + 1) / 2, down_nu = FP8 ? down_nw : (down_nw + 1) / 2;
  const int up_ks = k_split(up_nu, up.tiles, a.topk, cus);
  up.groups = (up.tiles + kWaves / up_ks - 1) / (kWaves / up_ks);
  up.units = (up_nu + up_ks - 1) / up_ks;
  const int up_items = static_cast<int>(a.topk) * up.groups, up_rounds = (up_items + cus - 1) / cus;
  const int up_grid = (up_items + up_rounds - 1) / up_rounds;
  // down: a wave per choice, the waves that this leaves split the sum
  const int down_ks = a.topk > 4 ? 1 : a.topk > 2 ? 2 : a.topk > 1 ? 4 : 8;
  down.units = (down_nu + down_ks - 1) / down_ks;
  const int rounds = (down.tiles + cus - 1) / cus;
  const int down_grid = (down.tiles + rounds - 1) / rounds;
  down.out = a.Y;
  launch_token_ks<T, FP8, true>(up, a.weights, up_ks, up_grid, up_lds, st);
  launch_token_ks<T, FP8, false>(down, a.weights, down_ks, down_grid, down_lds, st);
  return true;
}

template <typename T, bool FP8>
int launch_t(const MoeArgs& a) {
  hipStream_t st = static_cast<hipStream_t>(a.stream);
  const int64_t n = a.M * a.topk;
  __bf16* H = static_cast<__bf16*>(a.work);
  float* P = reinterpret_cast<float*>(static_cast<unsigned char*>(a.work) + (n * a.I * 4 + 255) / 256 * 256);
  MoeParams up{};
  up.ids = a.ids;
  up.topk = make_fastdiv(static_cast<uint32_t>(a.topk));
  up.win_per_block = make_fastdiv(FP8 ? static_cast<uint32_t>(a.block_size / 128) : 1u);
  up.n = static_cast<int>(n);
  up.E = static_cast<int>(a.E);
  up.act = a.activation;
  MoeParams down = up;
  up.x = a.A;
  up.w = a.w13;
  up.s = static_cast<const uint8_t*>(a.s13);
  up.g = a.g13;
  up.out = H;
  up.L = static_cast<int>(a.K);
  up.N = static_cast<int>(2 * a.I);
  up.cols = static_cast<int>((a.K + a.block_size - 1) / a.block_size);
  up.x_bytes = static_cast<int>(a.M * a.K * 2);
  up.tiles = static_cast<int>(a.I / 8);
  up.chunks_per_row = make_fastdiv(static_cast<uint32_t>((a.K + 127) / 128 * 16 + 1));
  down.x = H;
  down.w = a.w2;
  down.s = static_cast<const uint8_t*>(a.s2);
  down.g = a.g2;
  down.out = P;
  down.L = static_cast<int>(a.I);
  down.N = static_cast<int>(a.K);
  down.cols = static_cast<int>((a.I + a.block_size - 1) / a.block_size);
  down.x_bytes = static_cast<int>(n * a.I * 4);
  down.tiles = static_cast<int>(a.K / 16);
  down.chunks_per_row = make_fastdiv(static_cast<uint32_t>((a.I + 127) / 128 * 16 + 1));
  if (a.M == 1 && launch_token<T, FP8>(a, up, down, st)) return hipGetLastError() == hipSuccess ? 0 : -1;
  Shape up_shape, down_shape;
  if (!plan_shape(a, FP8, true, &up_shape) || !plan_shape(a, FP8, false, &down_shape)) return 1;
  launch_phase<T, FP8, true>(up, up_shape, st);
  launch_phase<__bf16, FP8, false>(down, down_shape, st);
  // combine
  const int64_t blocks = (a.M * (a.K / 4) + 255) / 256;
  hipLaunchKernelGGL(moe_combine_kernel<T>, dim3(static_cast<int>(std::min<int64_t>(blocks, 8192))), dim3(256), 0, st, P,
                     a.ids, a.weights, static_cast<T*>(a.Y), static_cast<int>(a.M), static_cast<int>(a.K),
                     static_cast<int>(a.topk), static_cast<int>(a.E), down_shape.splits,
                     make_fastdiv(static_cast<uint32_t>(a.K / 4)));
  return hipGetLastError() == hipSuccess ? 0 : -1;
}

}  // namespace

int launch_moe_fp4(const MoeArgs& a) {
  return a.act == Act::BF16 ? launch_t<__bf16, false>(a) : launch_t<_Float16, false>(a);
}
int launch_moe_fp8(const MoeArgs& a) {
  return a.act == Act::BF16 ? launch_t<__bf16, true>(a) : launch_t<_Float16, true>(a);
}

}  // namespace fp4w
