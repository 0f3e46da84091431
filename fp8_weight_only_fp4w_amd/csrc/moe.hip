// Mixture-of-experts layer for a few tokens on FP4 or FP8 weights, on MFMA.
//
//   H[a, i] = act(A[m] . W1[e][i]) * (A[m] . W3[e][i])      a = m * topk + j, e = ids[a]
//   Y[m, n] = RNE_T( sum_j weights[a] * (H[a] . W2[e][n]) )
//
// Memory-bound: every chosen expert is read once per pass of up to `rows`
// tokens, in whole 128-byte lines, as the decode GEMV reads a single weight
// matrix.  Three kernels: up (H from A), down (each choice's output from H)
// and combine (their weighted sum over a token's choices in the order of j, so
// the result does not depend on scheduling).
//
// Plan.  ids live on the device, so which experts are read is only known
// there.  Every workgroup of up and down sorts the assignments by expert in
// LDS (a count, a scan and a scatter over n <= 4096 ids) and cuts each
// expert's tokens into passes of at most `rows`.  The work is the flat list of
// (pass, group of column tiles); workgroup b of the persistent grid takes a
// contiguous share, so it meets few experts.
//
// A pass's token rows are copied to LDS once (zero-padded to whole 128-k
// windows) and shared by the 8 waves: KS waves split the sum of one column
// tile, 8 / KS tiles run side by side.  A wave streams its weights through a
// private LDS ring of direct loads, D units of 2 KiB ahead of the multiply
// (unit: 128 bytes of 16 rows, loaded as two instructions of 8 rows x 128
// bytes, chunks XOR-swizzled by row), across tiles and passes without a
// break.  The up kernel's 16 rows are 8 gate rows and the 8 up rows that
// belong to them, so both halves of a product meet in one tile.
//
// Operands (16x16x32 MFMA; lane li = l % 16 is token row for A and weight row
// for B, lane group g = l / 16 selects 8 of a step's 32 k; the result lane
// holds column li, token rows 4g .. 4g + 3).
//  * FP4: E2M1 x E4M3 is exact in FP16 and BF16, so a weight is decoded with
//    its block scale folded in; the expert's FP32 scale is applied to the sum.
//  * FP8: E4M3 -> T is exact, a 128-k window (inside one scale block) is summed
//    in a fresh accumulator and added times its FP32 scale.
//
// H is handed from up to down as two BF16 planes, high part and remainder (16
// significand bits, FP32's exponent range): one BF16 or FP16 rounding of H
// would double the output's error, and in FP16 gate * up may overflow.  The
// down kernel runs both planes through the same decoded weights.

#include <hip/hip_runtime.h>

#include <mutex>

#include "device.h"
#include "launch.h"
#include "moe_act.h"

namespace fp4w {
namespace {

constexpr int kWaves = 8;
constexpr int kThreads = 64 * kWaves;
constexpr uint32_t kUnitBytes = 2048;  // 16 rows x 128 bytes

template <int N>
__device__ __forceinline__ void wait_vm() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  __asm__ volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (0x7 << 4) | (0xF << 8));  // vmcnt(N) only
  __asm__ volatile("" ::: "memory");
}

// Barrier for data exchanged by ds_write / ds_read only: direct loads stay in
// flight.
__device__ __forceinline__ void lds_barrier() {
  __asm__ volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

struct MoeParams {
  const void* x;        // up: A, T[M, L]; down: H planes, BF16 [2][n][L]
  const uint8_t* w;     // [E, N, L] codes
  const uint8_t* s;     // [E, N, cols] scales
  const float* g;       // FP4: per expert
  const int32_t* ids;   // [n]
  void* out;            // up: H planes, BF16 [2][n][I]; down: FP32 [n][K]
  FastDiv topk, win_per_block, chunks_per_row;  // chunks_per_row: 16-byte chunks of an LDS row
  int n, E, L, N, cols;
  int x_bytes;          // up: M * L * 2; down: 2 * n * L * 2
  int rows;             // tokens per pass
  int tiles, groups;    // column tiles of an expert, and groups of TPW of them
  int units;            // per wave and tile
  int act;
  int list_max;         // passes at most
};

// LDS: unit rings, partial sums of the K split, then the plan and the token rows.
constexpr uint32_t kRedBytes = 2 * kWaves * 1024;

struct Plan {
  const uint32_t* list;    // pass: expert | first sorted assignment << 10 | (tokens - 1) << 22
  const uint16_t* sorted;  // assignments, by expert
  int passes;
};
// list and multi [list_max], count [E], part [16], sorted and expert [n]
constexpr uint32_t plan_bytes(int n, int E, int list_max) {
  return (8u * list_max + 4u * E + 4u * 16u + 4u * n + 15u) & ~15u;
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
__device__ __forceinline__ void write_passes(uint32_t* list, uint32_t slot, uint32_t e, uint32_t at, uint32_t tokens,
                                             uint32_t rows) {
  for (; tokens; ++slot) {
    const uint32_t t = tokens < rows ? tokens : rows;
    list[slot] = e | at << 10 | (t - 1) << 22;
    at += t;
    tokens -= t;
  }
}

// n <= 64: every wave makes the whole plan by itself, one assignment a lane,
// and writes it to LDS (all the same values), so no barrier is needed.
// Experts come in the order of their first assignment.
__device__ __forceinline__ Plan make_plan_wave(const MoeParams& p, unsigned char* mem) {
  uint32_t* list = reinterpret_cast<uint32_t*>(mem);
  uint16_t* sorted = reinterpret_cast<uint16_t*>(list + p.list_max);
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
  const uint32_t rows = static_cast<uint32_t>(p.rows);
  const uint32_t mine = leads ? static_cast<uint32_t>(tokens) | (tokens + rows - 1) / rows << 16 : 0u;
  const uint32_t upto = wave_scan(mine), before = upto - mine;
  if (leads) write_passes(list, before >> 16, static_cast<uint32_t>(id), before & 0xFFFF, tokens, rows);
  const uint32_t at = __shfl(before, first, 64) & 0xFFFF;
  if (valid) sorted[at + rank] = static_cast<uint16_t>(lane);
  return Plan{list, sorted, static_cast<int>(static_cast<uint32_t>(__builtin_amdgcn_readlane(upto, 63)) >> 16)};
}

// All threads of the workgroup; `mem` holds plan_bytes().  Every workgroup
// comes to the same list, and to the same tokens in each pass: an expert with
// several passes has its assignments in rising order.
__device__ __forceinline__ Plan make_plan(const MoeParams& p, unsigned char* mem) {
  uint32_t* list = reinterpret_cast<uint32_t*>(mem);
  uint32_t* multi = list + p.list_max;  // experts of several passes: expert | first sorted assignment << 10
  uint32_t* count = multi + p.list_max;
  uint32_t* part = count + p.E;
  uint16_t* sorted = reinterpret_cast<uint16_t*>(part + 16);
  uint16_t* expert = sorted + p.n;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  for (int e = tid; e < p.E; e += kThreads) count[e] = 0;
  if (tid == 0) part[8] = 0;
  __syncthreads();
  for (int a = tid; a < p.n; a += kThreads) {
    const uint32_t e = static_cast<uint32_t>(p.ids[a]);
    const bool valid = e < static_cast<uint32_t>(p.E);
    expert[a] = static_cast<uint16_t>(valid ? e : 0xFFFFu);
    if (valid) atomicAdd(&count[e], 1u);
  }
  __syncthreads();
  // experts 2 tid and 2 tid + 1 (E <= 1024): tokens in the low half, passes in the high half
  uint32_t c[2], v[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    c[i] = 2 * tid + i < p.E ? count[2 * tid + i] : 0u;
    v[i] = c[i] | ((c[i] + p.rows - 1) / p.rows) << 16;
  }
  const uint32_t sum = wave_scan(v[0] + v[1]);
  if (lane == 63) part[wave] = sum;
  __syncthreads();
  uint32_t before = sum - v[0] - v[1], total = 0;
#pragma unroll
  for (int i = 0; i < kWaves; ++i) {
    const uint32_t t = part[i];
    if (i < wave) before += t;
    total += t;
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t e = 2 * tid + i;
    if (c[i]) {
      const uint32_t at = before & 0xFFFF;
      count[e] = at;
      if (c[i] > static_cast<uint32_t>(p.rows)) multi[atomicAdd(&part[8], 1u)] = e | at << 10;
      write_passes(list, before >> 16, e, at, c[i], static_cast<uint32_t>(p.rows));
    }
    before += v[i];
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
  const int several = __builtin_amdgcn_readfirstlane(part[8]);
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
  return Plan{list, sorted, static_cast<int>(total >> 16)};
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
//
// a0: the lane's LDS address in window 0 of the high (or only) plane, `step`
// bytes per window and lo_plane to the other plane (both 0 for a lane that
// reads the zero block throughout); `zero`: the zero block, for windows past
// the row.  Every LDS read of the unit is issued before its arithmetic.

// FP4, dense: lane row li carries token li.  A weight is decoded with its
// block scale (lane group g holds blocks 2g and 2g + 1 of a window): about 86
// VALU instructions a window, for up to 16 tokens.
// FP4, DIAG: the decode GEMV's block-diagonal operand, for up to 4 rows.  Row
// 4 m + q carries row m in the k slots of lane group q only, so the lane (n,
// g) gets row g's dots with single blocks, scaled by one FMA each: the
// weights are decoded unscaled, which halves the VALU work.  The sum is
// acc[0].
template <typename Tr, int PLANES, bool DIAG>
__device__ __forceinline__ void fp4_unit(f32x4& acc, const u32x4& sc, const unsigned char* slot, lds_cbytes a0,
                                         uint32_t step, lds_cbytes zero, uint32_t lo_plane, int u, int NW, int L, int li,
                                         int g) {
  typedef typename Tr::vec8 V;
  const int sw = li & 7;
  u32x4 wv[2], av[2][PLANES][4];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int w = 2 * u + h;
    wv[h] = *reinterpret_cast<const u32x4*>(slot + 128 * li + 16 * ((4 * h + g) ^ sw));
    const lds_cbytes q = w < NW ? a0 + step * static_cast<uint32_t>(w) : zero;
    const uint32_t next = w < NW ? lo_plane : 0u;
#pragma unroll
    for (int pl = 0; pl < PLANES; ++pl)
#pragma unroll
      for (int i = 0; i < 4; ++i) av[h][pl][i] = *reinterpret_cast<const lds_u32x4*>(q + pl * next + 16 * i);
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int w = 2 * u + h;
    // E4M3 scales of the window's 8 blocks; blocks past the row (the next
    // row's bytes) count as zero
    const uint32_t s_lo = w < NW ? sc[2 * h] : 0u, s_hi = 128 * w + 64 < L ? sc[2 * h + 1] : 0u;
    if constexpr (DIAG) {
      const f32x2 s01 = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(s_lo), false);
      const f32x2 s23 = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(s_lo), true);
      const f32x2 s45 = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(s_hi), false);
      const f32x2 s67 = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(s_hi), true);
      const float s8[8] = {s01.x, s01.y, s23.x, s23.y, s45.x, s45.y, s67.x, s67.y};
      f32x4 d[2];
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const V b0 = Tr::decode8_fp4(wv[h][2 * s]), b1 = Tr::decode8_fp4(wv[h][2 * s + 1]);
        d[s] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int pl = 0; pl < PLANES; ++pl) {
          d[s] = Tr::mfma(__builtin_bit_cast(V, av[h][pl][2 * s]), b0, d[s]);
          d[s] = Tr::mfma(__builtin_bit_cast(V, av[h][pl][2 * s + 1]), b1, d[s]);
        }
      }
      // result row r of set s is block 2r + s
#pragma unroll
      for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int s = 0; s < 2; ++s) acc[0] = fmaf(d[s][r], s8[2 * r + s], acc[0]);
    } else {
      const uint32_t s2 = ((g & 2) ? s_hi : s_lo) >> (16 * (g & 1));
      const f32x2 sf = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(s2), false);
      const typename Tr::scale_t sa = Tr::make_scale(sf.x), sb = Tr::make_scale(sf.y);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const V b = Tr::decode8(wv[h][i], i < 2 ? sa : sb);
#pragma unroll
        for (int pl = 0; pl < PLANES; ++pl) acc = Tr::mfma(__builtin_bit_cast(V, av[h][pl][i]), b, acc);
      }
    }
  }
}

// FP8: a window's sum in a fresh accumulator, added times its FP32 scale.
// Lane group g takes chunks g and 4 + g (16 k each) of its row's 128 bytes.
template <typename Tr, int PLANES>
__device__ __forceinline__ void fp8_unit(f32x4& acc, uint32_t sc, const unsigned char* slot, lds_cbytes a0,
                                         lds_cbytes zero, uint32_t lo_plane, int u, int NW, int L, int li, int g) {
  typedef typename Tr::vec8 V;
  const int sw = li & 7;
  const u32x4 w0 = *reinterpret_cast<const u32x4*>(slot + 128 * li + 16 * (g ^ sw));
  u32x4 w1 = *reinterpret_cast<const u32x4*>(slot + 128 * li + 16 * ((4 + g) ^ sw));
  const lds_cbytes q = u < NW ? a0 + 256u * static_cast<uint32_t>(u) : zero;
  const uint32_t next = u < NW ? lo_plane : 0u;
  u32x4 av[PLANES][4];
#pragma unroll
  for (int pl = 0; pl < PLANES; ++pl)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      av[pl][i] = *reinterpret_cast<const lds_u32x4*>(q + pl * next + (i & 1) * 16 + (i >> 1) * 128);
  // a last window of 64 k: the bytes past the row are the next row's
  if (128 * u + 64 >= L) w1 = u32x4{0u, 0u, 0u, 0u};
  const V b[4] = {Tr::decode8_fp8(w0.x, w0.y), Tr::decode8_fp8(w0.z, w0.w), Tr::decode8_fp8(w1.x, w1.y),
                  Tr::decode8_fp8(w1.z, w1.w)};
  f32x4 d = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int pl = 0; pl < PLANES; ++pl)
#pragma unroll
    for (int i = 0; i < 4; ++i) d = Tr::mfma(__builtin_bit_cast(V, av[pl][i]), b[i], d);
  const float s = __builtin_bit_cast(float, sc);
#pragma unroll
  for (int i = 0; i < 4; ++i) acc[i] = fmaf(d[i], s, acc[i]);
}

// UP: the first kernel (A of type T against w13), otherwise the second (H
// planes against w2; its operands are BF16 whatever T is).
template <typename T, bool FP8, bool UP, int KS, int D>
__global__ __launch_bounds__(kThreads) void moe_kernel(const MoeParams p) {
  typedef typename std::conditional<UP, T, __bf16>::type X;
  typedef ActTraits<X> Tr;
  typedef typename Tr::vec8 V;
  typedef typename std::conditional<FP8, uint32_t, u32x4>::type Scale;
  constexpr int TPW = kWaves / KS;
  constexpr int S = D + 1;
  constexpr int UW = FP8 ? 1 : 2;  // 128-k windows per unit
  constexpr int PLANES = UP ? 1 : 2;
  constexpr int LPU = 3;  // loads per unit: scales, then two direct weight loads
  extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int li = lane & 15, g = lane >> 4;  // fragment side: row li, chunk group g
  const int lr = lane >> 3, lc = lane & 7;  // load side: row lr of an 8-row half, position lc
  const int ks = wave % KS, tw = wave / KS;
  unsigned char* ring = smem + static_cast<uint32_t>(wave) * (S * kUnitBytes);
  unsigned char* red = smem + kWaves * S * kUnitBytes;
  unsigned char* plan_mem = red + (KS > 1 ? kRedBytes : 0u);
  unsigned char* rows_lds = plan_mem + plan_bytes(p.n, p.E, p.list_max);
  const Plan plan = p.n <= 64 ? make_plan_wave(p, plan_mem) : make_plan(p, plan_mem);

  // this workgroup's share of the flat (pass, group) list
  const uint64_t all = static_cast<uint64_t>(plan.passes) * static_cast<uint64_t>(p.groups);
  const int64_t lo = static_cast<int64_t>(all * blockIdx.x / gridDim.x);
  const int64_t hi = static_cast<int64_t>(all * (blockIdx.x + 1) / gridDim.x);
  if (lo == hi) return;  // the whole workgroup
  const int first_pass = static_cast<int>(lo / p.groups);
  const int first_group = static_cast<int>(lo - static_cast<int64_t>(first_pass) * p.groups);
  const int64_t total = (hi - lo) * p.units;

  const int NW = (p.L + 127) >> 7;
  const int NU = (NW + UW - 1) / UW;
  const uint32_t row_bytes = FP8 ? static_cast<uint32_t>(p.L) : static_cast<uint32_t>(p.L >> 1);
  const uint32_t srow_bytes = FP8 ? 4u * p.cols : static_cast<uint32_t>(p.cols);
  const uint32_t half = UP ? static_cast<uint32_t>(p.N >> 1) : 8u;  // weight rows from a tile's first 8 to its last 8
  const uint32_t tile_rows = UP ? 8u : 16u;
  const uint32_t pitch = static_cast<uint32_t>(NW) * 256u + 16u;  // LDS bytes of a token row
  const rsrc_t x_rsrc = make_rsrc(p.x, static_cast<uint32_t>(p.x_bytes));
  const uint32_t wl = lr * row_bytes + 16u * (lc ^ lr);
  const uint32_t wl8 = wl + half * row_bytes;
  const uint32_t sl = (li < 8 ? li : li - 8 + half) * srow_bytes;

  // ---- load side
  int l_pass = first_pass, l_group = first_group, l_unit = 0;
  int l_expert = read_pass(plan.list, l_pass).expert;
  int64_t l_left = hi - lo;  // groups still to load, the current one included
  rsrc_t br, sr;
  auto set_load_tile = [&]() {
    const int t = l_group * TPW + tw;
    const bool on = l_left > 0 && t < p.tiles;
    const int64_t row = static_cast<int64_t>(l_expert) * p.N + static_cast<int64_t>(on ? t : 0) * tile_rows;
    const uint32_t span = on ? half + 8u : 0u;  // past the last tile or the share: every load reads zeros
    br = make_rsrc(p.w + row * row_bytes, span * row_bytes);
    sr = make_rsrc(p.s + row * srow_bytes, span * srow_bytes);
  };
  set_load_tile();
  auto load = [&](Scale& sc, unsigned char* slot) {
    const int u = ks * p.units + l_unit;
    const bool ok = u < NU;
    if constexpr (FP8) {
      const uint32_t col = min(fdiv(static_cast<uint32_t>(u), p.win_per_block), static_cast<uint32_t>(p.cols - 1));
      sc = buf_load_b32(sr, ok ? sl + 4u * col : kOutOfRange);
    } else {
      sc = buf_load_b128(sr, ok ? sl + 16u * u : kOutOfRange);  // 16 blocks: two windows
    }
    const uint32_t ub = 128u * static_cast<uint32_t>(u);
    buf_load_lds<16>(br, ok ? wl + ub : kOutOfRange, slot);
    buf_load_lds<16>(br, ok ? wl8 + ub : kOutOfRange, slot + 1024);
    if (++l_unit == p.units) {
      l_unit = 0;
      --l_left;
      if (++l_group == p.groups) {
        l_group = 0;
        ++l_pass;
        if (l_left > 0) l_expert = read_pass(plan.list, l_pass).expert;
      }
      set_load_tile();
    }
  };

  // ---- token rows of a pass, by direct loads: LDS chunk q holds row q /
  // chunks_per_row (down: the high parts of all tokens, then the remainders),
  // then 256 bytes of zeros; the zeros, rows' padding and the tail of the last instruction are out-of-range
  // reads, which write zeros
  auto fill = [&](const Pass& ps) {
    const uint32_t cpr = p.chunks_per_row.d;
    const uint32_t data = static_cast<uint32_t>(PLANES * ps.tokens) * cpr, chunks = data + 16u;
    for (uint32_t q0 = 64u * static_cast<uint32_t>(wave); q0 < chunks; q0 += 64u * kWaves) {
      const uint32_t q = q0 + static_cast<uint32_t>(lane);
      const uint32_t row = fdiv(q, p.chunks_per_row), col = q - row * cpr;
      uint32_t src = kOutOfRange;
      if (q < data && col * 8u < static_cast<uint32_t>(p.L)) {
        uint32_t r;
        if constexpr (UP) {
          r = fdiv(plan.sorted[ps.first + row], p.topk);
        } else {
          const bool rest = row >= static_cast<uint32_t>(ps.tokens);
          r = plan.sorted[ps.first + (rest ? row - ps.tokens : row)] + (rest ? static_cast<uint32_t>(p.n) : 0u);
        }
        src = r * (2u * p.L) + 16u * col;
      }
      buf_load_lds<16>(x_rsrc, src, rows_lds + 16u * q0);
    }
  };

  f32x4 acc = f32x4{0.f, 0.f, 0.f, 0.f};
  Scale raw[S];
  int c_pass = first_pass, c_group = first_group, c_unit = 0, turn = 0;
  // FP4: the expert's FP32 scale, read ahead of the pass's rows and waited for
  // with them (a load where a tile ends would wait for every weight load
  // before it)
  Pass ps = read_pass(plan.list, c_pass);
  float gs = FP8 ? 1.0f : p.g[ps.expert];
  fill(ps);
  // where the lane reads its token row: dense (and FP8) rows past the pass's
  // tokens repeat the last one, and their results are dropped
  bool diag;
  lds_cbytes a_lane, zero;
  uint32_t a_step, lo_plane;
  auto place = [&]() {
    const lds_cbytes base = (lds_cbytes)rows_lds;
    lo_plane = static_cast<uint32_t>(ps.tokens) * pitch;  // from a token's high part to its remainder
    zero = base + PLANES * lo_plane;
    diag = !FP8 && ps.tokens <= 4;
    const int m = diag ? li >> 2 : min(li, ps.tokens - 1);
    const bool carries = !diag || ((li & 3) == g && m < ps.tokens);
    a_lane = carries ? base + static_cast<uint32_t>(m) * pitch + (FP8 ? 32u : 64u) * g : zero;
    a_step = carries ? 256u : 0u;
    if (!carries) lo_plane = 0u;
  };
  place();
#pragma unroll
  for (int d = 0; d < D; ++d) load(raw[d], ring + d * kUnitBytes);
  wait_vm<D * LPU>();  // the fill is older
  __asm__ volatile("" : "+v"(gs));
  __builtin_amdgcn_s_barrier();
  __asm__ volatile("" ::: "memory");

  auto consume = [&](const Scale& sc, const unsigned char* slot) {
    const int u = ks * p.units + c_unit;
    wait_vm<D * LPU>();  // this unit's weights have landed
    if constexpr (FP8)
      fp8_unit<Tr, PLANES>(acc, sc, slot, a_lane, zero, lo_plane, u, NW, p.L, li, g);
    else if (diag)
      fp4_unit<Tr, PLANES, true>(acc, sc, slot, a_lane, a_step, zero, lo_plane, u, NW, p.L, li, g);
    else
      fp4_unit<Tr, PLANES, false>(acc, sc, slot, a_lane, a_step, zero, lo_plane, u, NW, p.L, li, g);
    if (++c_unit < p.units) return;
    // end of a tile: join the K split, then the epilogue
    c_unit = 0;
    if (KS > 1) {
      // the two halves of `red` are used in turn, so one barrier is enough: a
      // half is written again after a barrier that its readers reach later
      unsigned char* part = red + turn * (kRedBytes / 2) + wave * 1024 + 16 * lane;
      turn ^= 1;
      *reinterpret_cast<f32x4*>(part) = acc;
      lds_barrier();
      if (ks == 0) {
#pragma unroll
        for (int v = 1; v < KS; ++v) acc += *reinterpret_cast<const f32x4*>(part + v * 1024);
      }
    }
    const int t = c_group * TPW + tw;
    if (ks == 0 && t < p.tiles) {
      auto finish = [&](float v, int row) {
        if constexpr (UP) {
          const float up = swap8(v);
          if (row < ps.tokens && li < 8) {
            const size_t at = static_cast<size_t>(plan.sorted[ps.first + row]) * (p.N >> 1) + 8 * t + li;
            store_h(static_cast<__bf16*>(p.out) + at, static_cast<size_t>(p.n) * (p.N >> 1),
                    gated(p.act, v * gs, up * gs));
          }
        } else if (row < ps.tokens) {
          static_cast<float*>(p.out)[static_cast<size_t>(plan.sorted[ps.first + row]) * p.N + 16 * t + li] = v * gs;
        }
      };
      if (diag) {
        finish(acc[0], g);
      } else {
#pragma unroll
        for (int r = 0; r < 4; ++r) finish(acc[r], 4 * g + r);
      }
    }
    acc = f32x4{0.f, 0.f, 0.f, 0.f};
    if (++c_group == p.groups) {
      c_group = 0;
      ++c_pass;
    }
  };

  int64_t left = total;
  for (int64_t f0 = 0; f0 < total; f0 += S) {
#pragma unroll
    for (int u = 0; u < S; ++u) {
      load(raw[(u + D) % S], ring + ((u + D) % S) * kUnitBytes);
      if (left > 0) {  // uniform across the workgroup
        if (c_unit == 0 && c_group == 0 && c_pass != first_pass) {
          // the next pass's tokens take the place of the last one's
          ps = read_pass(plan.list, c_pass);
          if (!FP8) gs = p.g[ps.expert];
          lds_barrier();
          fill(ps);
          place();
          wait_vm<0>();
          __asm__ volatile("" : "+v"(gs));
          __builtin_amdgcn_s_barrier();
          __asm__ volatile("" ::: "memory");
        }
        consume(raw[u], ring + u * kUnitBytes);
        --left;
      }
    }
  }
  wait_vm<0>();  // loads past the end of the share write zeros to the ring
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
template <typename T, bool FP8, bool UP, int KS, int D>
__global__ __launch_bounds__(kThreads) void moe_token_kernel(const MoeParams p, const float* __restrict__ weights) {
  typedef typename std::conditional<UP, T, __bf16>::type X;
  typedef ActTraits<X> Tr;
  typedef typename Tr::vec8 V;
  typedef typename std::conditional<FP8, uint32_t, u32x4>::type Scale;
  constexpr int TPW = kWaves / KS;  // up: tiles side by side; down: choices side by side
  constexpr int S = D + 1;
  constexpr int UW = FP8 ? 1 : 2;
  constexpr int LPU = 3;
  constexpr int ROWS = UP ? 1 : 2;  // operand rows of a choice
  extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int li = lane & 15, g = lane >> 4;
  const int lr = lane >> 3, lc = lane & 7;
  const int ks = wave % KS, tw = wave / KS;
  unsigned char* ring = smem + static_cast<uint32_t>(wave) * (S * kUnitBytes);
  unsigned char* red = smem + kWaves * S * kUnitBytes;
  unsigned char* rows_lds = red + kTokenRedBytes;
  const int NW = (p.L + 127) >> 7;
  const int NU = (NW + UW - 1) / UW;
  const uint32_t row_bytes = FP8 ? static_cast<uint32_t>(p.L) : static_cast<uint32_t>(p.L >> 1);
  const uint32_t srow_bytes = FP8 ? 4u * p.cols : static_cast<uint32_t>(p.cols);
  const uint32_t half = UP ? static_cast<uint32_t>(p.N >> 1) : 8u;
  const uint32_t tile_rows = UP ? 8u : 16u;
  const uint32_t pitch = static_cast<uint32_t>(NW) * 256u + 16u;  // LDS bytes of a row
  const uint32_t wl = lr * row_bytes + 16u * (lc ^ lr);
  const uint32_t wl8 = wl + half * row_bytes;
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
  auto load = [&](Scale& sc, unsigned char* slot) {
    const int u = ks * p.units + l_unit;
    const bool ok = u < NU;
    if constexpr (FP8) {
      const uint32_t col = min(fdiv(static_cast<uint32_t>(u), p.win_per_block), static_cast<uint32_t>(p.cols - 1));
      sc = buf_load_b32(sr, ok ? sl + 4u * col : kOutOfRange);
    } else {
      sc = buf_load_b128(sr, ok ? sl + 16u * u : kOutOfRange);
    }
    const uint32_t ub = 128u * static_cast<uint32_t>(u);
    buf_load_lds<16>(br, ok ? wl + ub : kOutOfRange, slot);
    buf_load_lds<16>(br, ok ? wl8 + ub : kOutOfRange, slot + 1024);
    if (++l_unit == p.units) {
      l_unit = 0;
      if (++l_in == inner) {
        l_in = 0;
        l_item += gridDim.x;
      }
      set_load_tile();
    }
  };

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
  f32x4 acc = f32x4{0.f, 0.f, 0.f, 0.f};
  float sum = 0.0f;  // down: the weighted choices of this wave, lanes g == 0
  Scale raw[S];
  int c_item = blockIdx.x, c_in = 0, c_unit = 0, turn = 0;
#pragma unroll
  for (int d = 0; d < D; ++d) load(raw[d], ring + d * kUnitBytes);
  wait_vm<D * LPU>();  // the rows, scales and weights are older
  __asm__ volatile("" : "+v"(g_lane), "+v"(w_lane));
  __builtin_amdgcn_s_barrier();
  __asm__ volatile("" ::: "memory");

  auto consume = [&](const Scale& sc, const unsigned char* slot) {
    const int u = ks * p.units + c_unit;
    const int j = choice_of(c_item, c_in);
    wait_vm<D * LPU>();
    // row m of the operand: up 0: the token; down 0 and 1: the choice's two
    // planes.  FP4: block-diagonal, so lane groups 0 and 1 end with the rows'
    // sums in acc[0]; FP8: lane rows m, group 0 ends with them in acc[0 ..].
    const int m = FP8 ? li & (ROWS - 1) : li >> 2;
    const bool carries = FP8 || ((li & 3) == g && m < ROWS);
    const lds_cbytes base = (lds_cbytes)rows_lds;
    const lds_cbytes zero = base + static_cast<uint32_t>(UP ? 1 : 2 * p.n) * pitch;
    const uint32_t row = UP ? 0u : static_cast<uint32_t>(m * p.n + min(j, p.n - 1));
    const lds_cbytes a_lane = carries ? base + row * pitch + (FP8 ? 32u : 64u) * g : zero;
    if constexpr (FP8)
      fp8_unit<Tr, 1>(acc, sc, slot, a_lane, zero, 0u, u, NW, p.L, li, g);
    else
      fp4_unit<Tr, 1, true>(acc, sc, slot, a_lane, carries ? 256u : 0u, zero, 0u, u, NW, p.L, li, g);
    if (++c_unit < p.units) return;
    c_unit = 0;
    const int e = expert_of(j);
    float v = acc[0];  // lanes g == 0 hold the tile
    if (!UP) v += FP8 ? acc[1] : __shfl_xor(acc[0], 16, 64);
    acc = f32x4{0.f, 0.f, 0.f, 0.f};
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

  for (int f0 = 0; f0 < total; f0 += S) {
#pragma unroll
    for (int u = 0; u < S; ++u) {
      load(raw[(u + D) % S], ring + ((u + D) % S) * kUnitBytes);
      if (f0 + u < total) consume(raw[u], ring + u * kUnitBytes);
    }
  }
  wait_vm<0>();
}

// Y[m, c .. c + 7] = sum over j of weights[m * topk + j] * P[m * topk + j, c ..], in the order of j
template <typename T>
__global__ __launch_bounds__(256) void moe_combine_kernel(const float* __restrict__ P, const int32_t* __restrict__ ids,
                                                          const float* __restrict__ weights, T* __restrict__ Y, int M, int K, int topk, int E) {
  const int chunks = K >> 3;
  const int64_t all = static_cast<int64_t>(M) * chunks;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < all; i += 256 * static_cast<int64_t>(gridDim.x)) {
    const int m = static_cast<int>(i / chunks), c = static_cast<int>(i - static_cast<int64_t>(m) * chunks);
    float sum[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) sum[k] = 0.0f;
    for (int j0 = 0; j0 < topk; j0 += 4) {
      // four choices' loads at a time, none of them behind a branch; what a
      // masked choice holds is not used
      f32x4 x[4], y[4];
      float w[4];
      bool on[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int a = m * topk + min(j0 + j, topk - 1);
        const f32x4* q = reinterpret_cast<const f32x4*>(P + static_cast<size_t>(a) * K + 8 * c);
        x[j] = q[0];
        y[j] = q[1];
        w[j] = weights[a];
        on[j] = j0 + j < topk && static_cast<uint32_t>(ids[a]) < static_cast<uint32_t>(E);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          sum[k] = on[j] ? fmaf(x[j][k], w[j], sum[k]) : sum[k];
          sum[4 + k] = on[j] ? fmaf(y[j][k], w[j], sum[4 + k]) : sum[4 + k];
        }
      }
    }
    typename ActTraits<T>::vec8 r;
#pragma unroll
    for (int k = 0; k < 8; ++k) r[k] = round_to<T>(sum[k]);
    *reinterpret_cast<typename ActTraits<T>::vec8*>(Y + static_cast<size_t>(m) * K + 8 * c) = r;
  }
}

// --------------------------------------------------------------------- launch

constexpr size_t kMaxLds = 160 * 1024;

template <typename T, bool FP8, bool UP, int KS, int D>
void allow_lds() {
  static std::once_flag once[kMaxDevices];
  once_per_device(once, [] {
    (void)hipFuncSetAttribute(reinterpret_cast<const void*>(&moe_kernel<T, FP8, UP, KS, D>),
                              hipFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kMaxLds));
  });
}

struct Shape {
  int rows, depth, ks, grid, units, groups, list_max;
  size_t lds;
};

size_t fixed_lds(int depth, int n, int E, int list_max) {
  return static_cast<size_t>(kWaves) * (depth + 1) * kUnitBytes + kRedBytes + plan_bytes(n, E, list_max);
}

// Token rows of `planes` planes and the zero block, in whole direct-load instructions.
size_t rows_lds_bytes(int rows, int planes, int NW) {
  return (static_cast<size_t>(rows) * planes * (static_cast<size_t>(NW) * 256 + 16) + 256 + 1023) / 1024 * 1024;
}

// The K split of a tile over KS waves.  The larger it is, the smaller the
// groups of tiles that are shared out and the better the shares' bytes match,
// but every tile then ends with a join: measured (us of a layer; the split of
// up) FP4 K = 7168, 28 units of a row: 152 at 1, 142 at 2, 139 at 4, 137 at 8;
// FP4 K = 2048, 8 units: 73.6, 73.9, 80.9, 88.5; FP8 K = 4096, 32 units: 185,
// 175, 173, 172; FP8 I = 1024 (down), 8 units: 171.7, 170.2, 173.0, 180.7.  So:
// the largest split that leaves a wave four units of a tile, and beyond that
// only as far as the workgroups would not fill the chip.
int k_split(int NU, int64_t tiles, int64_t passes, int64_t cus) {
  int ks = 1;
  while (ks < kWaves && NU >= 8 * ks) ks *= 2;
  while (ks < kWaves && NU >= 2 * ks && passes * ((tiles + kWaves / ks - 1) / (kWaves / ks)) < cus) ks *= 2;
  return ks;
}

// The launch of one kernel: rows per pass, ring depth and K split.  False
// when not even one token row fits.
bool plan_shape(const MoeArgs& a, bool fp8, bool up, Shape* out) {
  const int64_t n = a.M * a.topk;
  const int64_t L = up ? a.K : a.I;
  const int NW = static_cast<int>((L + 127) / 128), NU = fp8 ? NW : (NW + 1) / 2;
  const int planes = up ? 1 : 2;
  // Tokens per pass: an expert's tokens beyond `rows` read its weights again.
  // Twice the mean and a few more is rarely exceeded, and every row that is
  // not reserved leaves LDS to the ring.
  const int64_t mean = a.E > 0 ? (n + a.E - 1) / a.E : n;
  int64_t want = 2 * mean + 4;
  if (want > 16) want = 16;
  if (want > a.M) want = a.M;  // (a token that names an expert twice may take a second pass)
  if (want < 1) want = 1;
  for (int depth : {4, 2}) {
    for (int64_t rows = want; rows >= 1; --rows) {
      if (depth == 4 && rows < want) break;  // a shallower ring before fewer rows
      const int64_t list_max = (n < a.E ? n : a.E) + n / rows;
      const size_t lds = fixed_lds(depth, static_cast<int>(n), static_cast<int>(a.E), static_cast<int>(list_max)) +
                         rows_lds_bytes(static_cast<int>(rows), planes, NW);
      if (lds > kMaxLds) continue;
      const int64_t tiles = up ? a.I / 8 : a.K / 16;
      const int64_t passes = n < a.E ? n : a.E;
      const int64_t cus = device_cus();
      const int ks = k_split(NU, tiles, passes, cus);
      const int64_t groups = (tiles + kWaves / ks - 1) / (kWaves / ks);
      *out = Shape{static_cast<int>(rows), depth, ks, static_cast<int>(passes * groups < cus ? passes * groups : cus),
                   (NU + ks - 1) / ks, static_cast<int>(groups), static_cast<int>(list_max), lds};
      return true;
    }
  }
  return false;
}

template <typename T, bool FP8, bool UP, int KS, int D>
void launch_kernel(const MoeParams& p, const Shape& s, hipStream_t st) {
  allow_lds<T, FP8, UP, KS, D>();
  hipLaunchKernelGGL((moe_kernel<T, FP8, UP, KS, D>), dim3(s.grid), dim3(kThreads), s.lds, st, p);
}

template <typename T, bool FP8, bool UP>
void launch_phase(MoeParams p, const Shape& s, hipStream_t st) {
  p.rows = s.rows;
  p.groups = s.groups;
  p.units = s.units;
  p.list_max = s.list_max;
#define FP4W_MOE_KS(KS_) \
  s.depth == 4 ? launch_kernel<T, FP8, UP, KS_, 4>(p, s, st) : launch_kernel<T, FP8, UP, KS_, 2>(p, s, st)
  switch (s.ks) {
    case 1: FP4W_MOE_KS(1); break;
    case 2: FP4W_MOE_KS(2); break;
    case 4: FP4W_MOE_KS(4); break;
    default: FP4W_MOE_KS(8); break;
  }
#undef FP4W_MOE_KS
}

template <typename T, bool FP8, bool UP, int KS>
void launch_token_kernel(const MoeParams& p, const float* weights, int grid, size_t lds, hipStream_t st) {
  static std::once_flag once[kMaxDevices];
  once_per_device(once, [] {
    (void)hipFuncSetAttribute(reinterpret_cast<const void*>(&moe_token_kernel<T, FP8, UP, KS, 4>),
                              hipFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kMaxLds));
  });
  hipLaunchKernelGGL((moe_token_kernel<T, FP8, UP, KS, 4>), dim3(grid), dim3(kThreads), lds, st, p, weights);
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

// M = 1.  False where the rows do not fit in LDS beside the rings.
template <typename T, bool FP8>
bool launch_token(const MoeArgs& a, MoeParams up, MoeParams down, hipStream_t st) {
  const size_t base = kWaves * 5 * kUnitBytes + kTokenRedBytes;
  const int cus = device_cus();
  const int up_nw = static_cast<int>((a.K + 127) / 128), down_nw = static_cast<int>((a.I + 127) / 128);
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
  const int64_t blocks = (a.M * (a.K / 8) + 255) / 256;
  hipLaunchKernelGGL(moe_combine_kernel<T>, dim3(static_cast<int>(blocks < 4096 ? blocks : 4096)), dim3(256), 0, st, P,
                     a.ids, a.weights, static_cast<T*>(a.Y), static_cast<int>(a.M), static_cast<int>(a.K),
                     static_cast<int>(a.topk), static_cast<int>(a.E));
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
