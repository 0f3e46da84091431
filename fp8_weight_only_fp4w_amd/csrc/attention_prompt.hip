// Attention over the paged 8-bit cache, head sizes 64 and 128, for many new
// tokens of a sequence (prompts and pieces of them).
//
//   s_t = scale q . K_t    O = sum_t 2^(s_t' - m) V_t / sum_t 2^(s_t' - m),  s' = s log2(e), m the largest s' so far
//
// A workgroup has 128 rows of one sequence and key head (the query heads that
// read this key head, token by token), 32 for each of its four waves, and goes
// through the keys in tiles of 64.  The codes of a tile are converted to T once
// for the workgroup, on their way from registers to LDS, while the tile before
// is worked on; K keeps its codes (its scale is a factor of the scores), V takes
// its scale in the conversion.  Both products run on 32 x 32 x 16 MFMAs, as
// S^T = K Q^T and O^T = V^T P^T, so a lane has one query row: maximum and sum
// need one exchange between two lanes, and P^T is the operand of the second
// product as it leaves the softmax.  For that, key 16 h + 4 a + b of 32 stands
// in row 8 a + 4 h + b of K's tile.
//
// The matrix units, the LDS that feeds them and the vector units are the bound
// together: of 722 us that an earlier form took for a prompt of 8192 tokens with
// 40 query and 8 key heads of 128 (BF16, 687 GFLOP) the products with their LDS
// reads took 461 alone; 509 without the staging, 647 without the loads, 711 without
// the conversions and 650 without the softmax.  It now takes 685 to 718 us on
// different cards, 0.96 to 1.0 PFLOP/s, where a large library product reaches 1.28;
// 28 heads of 64 take 303 to 322.  Rows of 64 a wave (one wave a SIMD) took 1110 us
// and more, 256 rows a workgroup no less than 128.

#include <hip/hip_runtime.h>

#include "attention.h"

namespace fp4w {
namespace {

struct PromptParams {
  AttnParams a;
  float* part;      // splits > 1: partial results
  int32_t splits;   // parts that a row tile's keys are cut into at most
  int64_t units;    // row tiles at most
};

template <typename T>
struct Mfma32;
template <>
struct Mfma32<__bf16> {
  __device__ __forceinline__ static f32x16 run(bf16x8 a, bf16x8 b, f32x16 c) { return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0); }
};
template <>
struct Mfma32<_Float16> {
  __device__ __forceinline__ static f32x16 run(f16x8 a, f16x8 b, f32x16 c) { return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0); }
};

// The larger of a lane's value and that of the lane 32 on.
__device__ __forceinline__ float other_half_max(float x) {
  const auto both = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(both[0]), __uint_as_float(both[1]));
}

// Row tiles are numbered from floor(starts[b] G / R) + b on for sequence b: n
// tokens have at most n G / R + 1 of them, so two sequences never meet.
template <int R>
__device__ __forceinline__ int64_t first_row_tile(const AttnParams& p, int b) {
  return static_cast<int64_t>(seq_start(p.seq, b)) * p.G / R + b;
}

struct RowTile {
  int b, row0, rows, token0, first;  // rows row0 .. of sequence b's rows; its first new row and position
  int held;
  int lo, hi;  // key tiles
};

template <int R>
__device__ __forceinline__ bool row_tile_of(const AttnParams& p, int64_t unit, RowTile& r) {
  r.b = last_not_above(p.seq.B, unit, [&](int i) { return first_row_tile<R>(p, i); });
  const SeqSpan s = seq_span(p.seq, r.b);
  const int n = s.rows < p.max_new ? s.rows : p.max_new;
  const int64_t row0 = (unit - first_row_tile<R>(p, r.b)) * R, all = static_cast<int64_t>(n) * p.G;
  if (row0 < 0 || row0 >= all) return false;
  r.row0 = static_cast<int>(row0);
  r.rows = static_cast<int>(all - row0 < R ? all - row0 : R);
  r.token0 = s.first_row;
  r.first = s.len - s.rows;
  r.held = s.len < p.seq.capacity ? s.len : p.seq.capacity;
  const int low = r.first + r.row0 / p.G, high = r.first + (r.row0 + r.rows - 1) / p.G;  // positions
  const int64_t end = p.causal && static_cast<int64_t>(high) + 1 < r.held ? static_cast<int64_t>(high) + 1 : r.held;
  const int64_t begin = p.window > 0 && low >= p.window ? low - p.window + 1 : 0;
  r.lo = static_cast<int>(begin / kTile);
  r.hi = end > 0 ? static_cast<int>((end + kTile - 1) / kTile) : 0;
  if (r.hi < r.lo) r.hi = r.lo;
  return true;
}

// Parts that a row tile's keys are cut into.
__device__ __forceinline__ int row_parts(const RowTile& r, int splits) {
  const int most = (r.hi - r.lo) / kPromptPart;
  return most < 1 ? 1 : most < splits ? most : splits;
}

template <typename T, int D, int WAVES>
__global__ __launch_bounds__(64 * WAVES, D == 64 ? 3 : 2) void attn_prompt_kernel(const PromptParams pp) {
  constexpr int R = 32 * WAVES, KP = D + 8, VP = kTile + 8, KS = D / 16, DT = D / 32;
  constexpr int THREADS = 64 * WAVES, CHUNKS = kTile * D / 16 / THREADS;  // 16-byte pieces of K (and of V) for each thread
  constexpr int STEP = THREADS / 4;                                       // from one piece of a thread to the next
  typedef typename ActTraits<T>::vec8 vec8;
  __shared__ __attribute__((aligned(16))) T k_lds[2][kTile * KP];
  __shared__ __attribute__((aligned(16))) T v_lds[2][D * VP];
  __shared__ float scale_lds[2][4];
  __shared__ uint16_t nan_lds[2][D][4];  // which of a value's 16 keys of a chunk are NaN; for tiles of nan_tile - 1
  __shared__ int absent_lds[2], nan_tile[2];
  const AttnParams& p = pp.a;
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, col = lane & 31, h = lane >> 5;
  // the last row tiles of a prompt have the most keys: they come first
  const int64_t block = blockIdx.x / p.Hk;
  const int hk = static_cast<int>(blockIdx.x - block * p.Hk);
  const int64_t unit = pp.units - 1 - block / pp.splits;
  const int split = static_cast<int>(block % pp.splits);
  RowTile r;
  if (!row_tile_of<R>(p, unit, r)) return;
  const int parts = row_parts(r, pp.splits), share = (r.hi - r.lo + parts - 1) / parts;
  if (split >= parts) return;
  const int t_begin = r.lo + share * split < r.hi ? r.lo + share * split : r.hi;
  const int t_end = t_begin + share < r.hi ? t_begin + share : r.hi;

  // this lane's row
  const int mine = 32 * wave + col, row = r.row0 + mine;
  const bool valid = mine < r.rows;
  const int token = row / p.G, head = hk * p.G + (row - token * p.G), pos = r.first + token;
  const int k_hi = !valid ? 0 : p.causal && pos + 1 < r.held ? pos + 1 : r.held;
  const int k_lo = p.window > 0 && pos >= p.window ? pos - p.window + 1 : 0;
  vec8 qf[KS];
  {
    const T* q = static_cast<const T*>(p.q) + (static_cast<int64_t>(r.token0) + token) * p.q_stride + static_cast<int64_t>(head) * D + 8 * h;
#pragma unroll
    for (int i = 0; i < KS; ++i) {
      u32x4 v = {0, 0, 0, 0};
      if (valid) v = *reinterpret_cast<const u32x4*>(q + 16 * i);
      v ^= p.flip;
      qf[i] = __builtin_bit_cast(vec8, v);
    }
  }
  // tokens that all of the wave's rows attend; that all of the workgroup's do, and that any does
  const int w_rows = r.rows - 32 * wave < 32 ? r.rows - 32 * wave : 32;
  const int w_low = r.first + (r.row0 + 32 * wave) / p.G, w_high = r.first + (r.row0 + 32 * wave + w_rows - 1) / p.G;
  const int all_lo = p.window > 0 && w_high >= p.window ? w_high - p.window + 1 : 0;
  int all_hi = w_rows <= 0 ? 0 : p.causal && w_low + 1 < r.held ? w_low + 1 : r.held;
  const int g_low = r.first + r.row0 / p.G, g_high = r.first + (r.row0 + r.rows - 1) / p.G;
  const int every_lo = p.window > 0 && g_high >= p.window ? g_high - p.window + 1 : 0;
  const int every_hi = p.causal && g_low + 1 < r.held ? g_low + 1 : r.held;
  const int any_lo = p.window > 0 && g_low >= p.window ? g_low - p.window + 1 : 0;
  const int any_hi = p.causal && g_high + 1 < r.held ? g_high + 1 : r.held;

  // A thread's pieces of a tile are of one chunk of 16 keys (so of one page): of K
  // one key's 16 values each, of V one value's 16 keys.
  const int chunk = (tid >> 4) & 3, piece = (tid & 15) | (wave << 4);
  const uint32_t page_bytes = static_cast<uint32_t>(p.Hk) * p.seq.page * D;
  const uint8_t* k_base = p.k_cache + static_cast<uint32_t>(hk * p.seq.page * D + 16 * piece);
  const uint8_t* v_base = p.v_cache + static_cast<uint32_t>(hk * p.seq.page * D + piece * p.seq.page);
  u32x4 kreg[CHUNKS], vreg[CHUNKS];
  uint32_t k_byte = 0, v_byte = 0;
  struct Place {
    int id;         // page of this thread's chunk in a tile, or -1
    uint32_t slot;  // its first token's
  };
  const int32_t* pages = p.seq.table + r.b * p.seq.max_pages;
  auto place_of = [&](int t) {
    Place at;
    at.id = page_ahead(p.seq, pages, t * kTile + 16 * chunk, t < t_end, &at.slot);
    return at;
  };
  int id = -1;  // of the chunk in the registers
  auto load = [&](Place at) {
    id = at.id;
    const uint32_t known = id < 0 ? 0 : id;
    const uint8_t* k = k_base + static_cast<uint64_t>(known) * page_bytes + at.slot * D;
    const uint8_t* v = v_base + static_cast<uint64_t>(known) * page_bytes + at.slot;
    const uint64_t cell = static_cast<uint64_t>(known) * static_cast<uint32_t>(p.Hk) + hk;
#pragma unroll
    for (int i = 0; i < CHUNKS; ++i) {
      kreg[i] = *reinterpret_cast<const u32x4*>(k + 16 * STEP * i);
      vreg[i] = *reinterpret_cast<const u32x4*>(v + STEP * i * p.seq.page);
    }
    k_byte = p.k_scale[cell];
    v_byte = p.v_scale[cell];
  };
  float power = 1.0f;  // of the values in the registers
  // What the rows of a tile's edge, absent pages and odd scales need, for the
  // tile in the registers, which goes to buffer buf.
  auto prepare = [&](int t, int buf) {
    uint32_t byte = v_byte;
    if (AttnTraits<T>::kLeastV > 0 && __ballot(byte < AttnTraits<T>::kLeastV) != 0) byte = scale_of_zeros<T>(vreg, byte);
    const uint64_t odd = __ballot(id < 0 || !held_scale<T>(byte));  // (every wave has all four chunks)
    if (t * kTile < every_lo || t * kTile + kTile > every_hi || odd != 0) {
      // Not every row attends all of the tile.  Values that none does become 0,
      // whatever they hold; those that T does not hold, and of a page whose scale
      // is no number, become NaN; and NaN is noted apart, with 0 in its place.
      asm volatile("" ::: "memory");
      if (__ballot(!held_scale<T>(byte)) != 0) {
#pragma unroll
        for (int i = 0; i < CHUNKS; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) vreg[i][j] = codes_held<T>(vreg[i][j], byte);
      }
      const int key0 = t * kTile + 16 * chunk;
      uint32_t nans[CHUNKS], any = 0;
#pragma unroll
      for (int i = 0; i < CHUNKS; ++i) nans[i] = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t keep = id < 0 ? 0u : byte_mask(any_lo - (key0 + 4 * j), any_hi - (key0 + 4 * j));
#pragma unroll
        for (int i = 0; i < CHUNKS; ++i) {
          const uint32_t word = vreg[i][j] & keep, n = nan_codes(word) >> 7;
          vreg[i][j] = word & ~(n * 0xffu);
          nans[i] |= ((n & 1) | (n >> 7 & 2) | (n >> 14 & 4) | (n >> 21 & 8)) << (4 * j);
        }
      }
      byte = id < 0 ? 127 : scale_held<T>(byte);
#pragma unroll
      for (int i = 0; i < CHUNKS; ++i) {
        nan_lds[buf][piece + STEP * i][chunk] = static_cast<uint16_t>(nans[i]);
        any |= nans[i];
      }
      if (any != 0) nan_tile[buf] = t + 1;
    }
    power = __uint_as_float((byte > AttnTraits<T>::kDown ? byte - AttnTraits<T>::kDown : 0u) << 23);
    if (wave == 0) {
      if ((lane & 15) == 0) scale_lds[buf][chunk] = id < 0 ? 0.0f : finite_factor(e8m0_to_f32(k_byte) * p.c);
      const uint64_t absent = __ballot(id < 0);
      if (tid == 0) absent_lds[buf] = static_cast<int>((absent & 1) | (absent >> 15 & 2) | (absent >> 30 & 4) | (absent >> 45 & 8));
    }
  };
  auto convert = [&](int buf) {
#pragma unroll
    for (int i = 0; i < CHUNKS; ++i) {
      const int at = piece + STEP * i, key = at / (D / 16), part = at % (D / 16);  // key: of the chunk's 16
      const int row = ((chunk >> 1) << 5) | ((key >> 2) << 3) | ((chunk & 1) << 2) | (key & 3);
      vec8* to = reinterpret_cast<vec8*>(&k_lds[buf][row * KP + 16 * part]);
      to[0] = ActTraits<T>::decode8_fp8(kreg[i].x, kreg[i].y);
      to[1] = ActTraits<T>::decode8_fp8(kreg[i].z, kreg[i].w);
    }
#pragma unroll
    for (int i = 0; i < CHUNKS; ++i) {
      vec8* to = reinterpret_cast<vec8*>(&v_lds[buf][(piece + STEP * i) * VP + 16 * chunk]);
      to[0] = decode8_power<T>(vreg[i].x, vreg[i].y, power);
      to[1] = decode8_power<T>(vreg[i].z, vreg[i].w, power);
    }
  };

  f32x16 acc[DT];
#pragma unroll
  for (int d = 0; d < DT; ++d)
#pragma unroll
    for (int j = 0; j < 16; ++j) acc[d][j] = 0.0f;
  float m = -INFINITY, l = 0.0f;

  if (p.seq.capacity > 0 && t_begin < t_end) {
    if (tid < 2) nan_tile[tid] = 0;
    load(place_of(t_begin));
    Place next = place_of(t_begin + 1);
    uint64_t far_lanes = 0;  // whose queries are held smaller
    if constexpr (AttnTraits<T>::kFarQueries) {
      uint32_t far = 0;
#pragma unroll
      for (int i = 0; i < KS; ++i) {
        const u32x4 v = __builtin_bit_cast(u32x4, qf[i]);
        far |= (far_pair(v.x) | far_pair(v.y)) | (far_pair(v.z) | far_pair(v.w));
      }
      far_lanes = __ballot(far != 0);
      if (far_lanes != 0) {  // (lanes l and l + 32 have a row)
        all_hi = 0;          // no tile goes without the masks, which scale the scores up
        far_lanes |= far_lanes << 32 | far_lanes >> 32;
        if (far_lanes >> lane & 1)
#pragma unroll
          for (int i = 0; i < KS; ++i) {
            const u32x4 v = __builtin_bit_cast(u32x4, qf[i]);
            qf[i] = __builtin_bit_cast(vec8, u32x4{down_pair(v.x), down_pair(v.y), down_pair(v.z), down_pair(v.w)});
          }
      }
    }
    __syncthreads();
    prepare(t_begin, 0);
    convert(0);
    load(next);
    next = place_of(t_begin + 2);
    __syncthreads();
    int buf = 0;
    for (int t = t_begin; t < t_end; ++t, buf ^= 1) {
      if (t + 1 < t_end) prepare(t + 1, buf ^ 1);
      const int key0 = t * kTile;
      const T* ks = k_lds[buf] + col * KP + 8 * h;
      const T* vs = v_lds[buf] + col * VP + 16 * h;
      f32x16 s[2];
      const f32x16 zero = {0.0f};
#pragma unroll
      for (int k = 0; k < KS; ++k)  // (two chains: an MFMA does not wait for the one before)
#pragma unroll
        for (int i = 0; i < 2; ++i)
          s[i] = Mfma32<T>::run(*reinterpret_cast<const vec8*>(ks + 32 * i * KP + 16 * k), qf[k], k == 0 ? zero : s[i]);
      convert(buf ^ 1);  // (behind the last tile: once more what is there already)
      const int absent = absent_lds[buf];
      float factor[2] = {scale_lds[buf][h], scale_lds[buf][2 + h]};
      uint32_t seen = 0xffffffffu;
      if (!(key0 >= all_lo && key0 + kTile <= all_hi && absent == 0)) {
        asm volatile("" ::: "memory");
        seen = 0;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const bool here = ((absent >> (2 * i + h)) & 1) == 0;
          const int my0 = key0 + 32 * i + 16 * h;
          const int from = here ? k_lo - my0 : 16, to = k_hi - my0;  // this lane's 16 keys: [from, to) are attended
          if (far_lanes >> lane & 1) factor[i] = finite_factor(factor[i] * kFarUp);
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const bool on = j >= from && j < to;
            s[i][j] = on ? s[i][j] * factor[i] : -INFINITY;
            seen |= on ? 1u << (16 * i + j) : 0u;
          }
          factor[i] = 1.0f;
        }
      }
      float top = seen != 0 ? kLowest : -INFINITY;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float most = s[i][0];
#pragma unroll
        for (int j = 1; j < 16; ++j) most = fmaxf(most, s[i][j]);
        top = fmaxf(top, most * factor[i]);
      }
      top = other_half_max(top);
      // The maximum that numerators are taken to may lag behind by kLag: they
      // stay in T's range, and the outputs are seldom rescaled.
      if (__ballot(top > m + AttnTraits<T>::kLag) != 0) {
        asm volatile("" ::: "memory");
        const float now = fmaxf(m, top);
        const float shrink = __builtin_amdgcn_exp2f(m - (now > -INFINITY ? now : 0.0f));
        l *= shrink;
#pragma unroll
        for (int d = 0; d < DT; ++d) acc[d] *= shrink;
        m = now;
      }
      const float base = AttnTraits<T>::kLift - (m > -INFINITY ? m : 0.0f);
      vec8 pf[4];
      float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const float e = __builtin_amdgcn_exp2f(fmaf(s[i][j], factor[i], base));
          sum[j & 3] += e;
          pf[2 * i + (j >> 3)][j & 7] = static_cast<T>(e);  // the one rounding between the products
        }
      l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
      if (nan_tile[buf] == t + 1) {
        // 0 x NaN must not reach the rows that do not attend it: the NaN values
        // that each output attends are counted apart (they are 0 in v_lds)
        asm volatile("" ::: "memory");
#pragma unroll
        for (int d = 0; d < DT; ++d) {
          f32x16 hits = {0.0f};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint32_t at = nan_lds[buf][32 * d + col][2 * (k >> 1) + h] >> (8 * (k & 1)), bits = seen >> (8 * k);
            vec8 flag, on;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              flag[j] = static_cast<T>((at >> j) & 1 ? 1.0f : 0.0f);
              on[j] = static_cast<T>((bits >> j) & 1 ? 1.0f : 0.0f);
            }
            hits = Mfma32<T>::run(flag, on, hits);
          }
#pragma unroll
          for (int j = 0; j < 16; ++j) acc[d][j] = hits[j] > 0.0f ? NAN : acc[d][j];
        }
      }
      // D = 64 goes on loading (page 0) behind the last tile: without a branch it
      // takes 320 us for 8192 tokens of 28 heads, with one 335; D = 128 takes 738
      // and 704 for 40 heads.
      if (D == 64 || t + 2 < t_end) load(next);
      next = place_of(t + 3);
#pragma unroll
      for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int d = 0; d < DT; ++d)
          acc[d] = Mfma32<T>::run(*reinterpret_cast<const vec8*>(vs + 32 * d * VP + 32 * (k >> 1) + 8 * (k & 1)), pf[k], acc[d]);
      __syncthreads();
    }
  }
  l += __shfl_xor(l, 32, 64);
  if (!valid) return;
  if (parts == 1) {
    const int64_t at_row = (static_cast<int64_t>(r.token0) + token) * p.Hq + head;
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        store_quad<T>(p, at_row, D, 32 * d + 8 * j + 4 * h, m, l, f32x4{acc[d][4 * j], acc[d][4 * j + 1], acc[d][4 * j + 2], acc[d][4 * j + 3]});
    if (h == 0) store_lse<T>(p, at_row, m, l);
  } else {
    float* part = pp.part + ((unit * p.Hk + hk) * pp.splits + split) * attn_part_floats(R, D);
    float* o = part + attn_part_head(R) + mine * D + 4 * h;
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        *reinterpret_cast<f32x4*>(o + 32 * d + 8 * j) = f32x4{acc[d][4 * j], acc[d][4 * j + 1], acc[d][4 * j + 2], acc[d][4 * j + 3]};
    if (h == 0) {
      part[mine] = m;
      part[R + mine] = l;
    }
  }
}

// Joins the parts of every row that has several: D / 4 lanes for a row, a workgroup for an eighth
// of a row tile and key head.
template <typename T, int D, int R>
__global__ __launch_bounds__(256) void attn_prompt_join_kernel(const PromptParams pp) {
  constexpr int LANES = D / 4, ROWS = 256 / LANES;
  const AttnParams& p = pp.a;
  const int cell = blockIdx.x >> 3, first = (blockIdx.x & 7) * (R / 8), hk = cell % p.Hk, lane = threadIdx.x % LANES;
  const int64_t unit = cell / p.Hk;
  RowTile r;
  if (!row_tile_of<R>(p, unit, r)) return;
  const int parts = row_parts(r, pp.splits);
  if (parts == 1) return;
  const float* part = pp.part + (unit * p.Hk + hk) * pp.splits * attn_part_floats(R, D);
  const int end = first + R / 8 < r.rows ? first + R / 8 : r.rows;
  for (int mine = first + threadIdx.x / LANES; mine < end; mine += ROWS) {
    float m = -INFINITY, l = 0.0f;
    f32x4 o = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
    for (int i = 0; i < parts; ++i) {
      const float* one = part + i * attn_part_floats(R, D);
      join(m, l, o, one[mine], one[R + mine], *reinterpret_cast<const f32x4*>(one + attn_part_head(R) + mine * D + 4 * lane));
    }
    const int row = r.row0 + mine, token = row / p.G;
    const int64_t at_row = (static_cast<int64_t>(r.token0) + token) * p.Hq + hk * p.G + (row - token * p.G);
    store_quad<T>(p, at_row, D, 4 * lane, m, l, o);
    if (lane == 0) store_lse<T>(p, at_row, m, l);
  }
}

template <typename T, int D, int WAVES>
int launch_waves(PromptParams p, int64_t M, int64_t capacity, hipStream_t s) {
  constexpr int R = 32 * WAVES;
  static_assert(R == kPromptRows, "the workspace is sized for these row tiles");
  p.units = attn_row_tiles_most(M, p.a.G, p.a.seq.B);
  p.splits = static_cast<int32_t>(attn_prompt_splits(p.units * p.a.Hk, capacity));
  hipLaunchKernelGGL((attn_prompt_kernel<T, D, WAVES>), dim3(static_cast<uint32_t>(p.units * p.a.Hk * p.splits)), dim3(64 * WAVES), 0, s, p);
  if (p.splits > 1)
    hipLaunchKernelGGL((attn_prompt_join_kernel<T, D, R>), dim3(static_cast<uint32_t>(8 * p.units * p.a.Hk)), dim3(256), 0, s, p);  // (units * Hk < kPromptPlaces)
  return hipGetLastError() == hipSuccess ? 0 : -1;
}

template <typename T>
int launch_t(const PromptParams& p, const AttentionArgs& a, hipStream_t s) {
  const int64_t capacity = a.seq.max_pages * a.seq.page_size;
  if (a.D == 64) return launch_waves<T, 64, 4>(p, a.M, capacity, s);
  return launch_waves<T, 128, 4>(p, a.M, capacity, s);
}

}  // namespace

int launch_attention_prompt(const AttentionArgs& a) {
  PromptParams p;
  p.a = make_attn(a);
  p.part = static_cast<float*>(a.work);
  hipStream_t s = static_cast<hipStream_t>(a.stream);
  return a.act == Act::BF16 ? launch_t<__bf16>(p, a, s) : launch_t<_Float16>(p, a, s);
}

}  // namespace fp4w
