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

#include <hip/hip_runtime.h>

#include "attention.h"

namespace fp4w {
namespace {

struct PromptParams {
  AttnParams a;
  float* part;      // splits > 1: partial results
  int32_t splits;   // parts that a row tile's keys are cut into
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

// Row tiles are numbered from floor(starts[b] G / R) + b on for sequence b: n
// tokens have at most n G / R + 1 of them, so two sequences never meet.
template <int R>
__device__ __forceinline__ int64_t first_row_tile(const AttnParams& p, int b) {
  return static_cast<int64_t>(seq_start(p.seq, b)) * p.G / R + b;
}

struct RowTile {
  int b, row0, rows, token0, first;  // rows row0 .. of sequence b's rows; its first new row and position
  int held;
  int64_t lo, hi;  // key tiles
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
  r.lo = begin / kTile;
  r.hi = end > 0 ? (end + kTile - 1) / kTile : 0;
  if (r.hi < r.lo) r.hi = r.lo;
  return true;
}

template <typename T, int D>
__global__ __launch_bounds__(256, 2) void attn_prompt_kernel(const PromptParams pp) {
  constexpr int R = kPromptRows, KP = D + 8, VP = kTile + 8, KS = D / 16, DT = D / 32;
  constexpr int CHUNKS = kTile * D / 16 / 256;  // 16-byte pieces of K (and of V) for each thread
  typedef typename ActTraits<T>::vec8 vec8;
  __shared__ __attribute__((aligned(16))) T k_lds[2][kTile * KP];
  __shared__ __attribute__((aligned(16))) T v_lds[2][D * VP];
  __shared__ float scale_lds[2][4];
  __shared__ int absent_lds[2], nan_lds[2];
  const AttnParams& p = pp.a;
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, col = lane & 31, h = lane >> 5;
  // the last row tiles of a prompt have the most keys: they come first
  const int64_t block = blockIdx.x / p.Hk;
  const int hk = static_cast<int>(blockIdx.x - block * p.Hk);
  const int64_t unit = pp.units - 1 - block / pp.splits;
  const int split = static_cast<int>(block % pp.splits);
  RowTile r;
  if (!row_tile_of<R>(p, unit, r)) return;
  const int64_t share = (r.hi - r.lo + pp.splits - 1) / pp.splits;
  const int64_t t_begin = r.lo + share * split < r.hi ? r.lo + share * split : r.hi;
  const int64_t t_end = t_begin + share < r.hi ? t_begin + share : r.hi;

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
  // of the wave's rows: tokens that all attend and that any does; of the workgroup's: that any does
  const int w_rows = r.rows - 32 * wave < 32 ? r.rows - 32 * wave : 32;
  const int w_low = r.first + (r.row0 + 32 * wave) / p.G, w_high = r.first + (r.row0 + 32 * wave + w_rows - 1) / p.G;
  const int all_lo = p.window > 0 && w_high >= p.window ? w_high - p.window + 1 : 0;
  const int all_hi = p.causal && w_low + 1 < r.held ? w_low + 1 : r.held;
  const int w_lo = p.window > 0 && w_low >= p.window ? w_low - p.window + 1 : 0;
  const int w_hi = w_rows <= 0 ? 0 : p.causal && w_high + 1 < r.held ? w_high + 1 : r.held;
  const int g_low = r.first + r.row0 / p.G, g_high = r.first + (r.row0 + r.rows - 1) / p.G;
  const int any_lo = p.window > 0 && g_low >= p.window ? g_low - p.window + 1 : 0;
  const int any_hi = p.causal && g_high + 1 < r.held ? g_high + 1 : r.held;

  const int64_t head_bytes = static_cast<int64_t>(p.seq.page) * D;
  // this thread's pieces of a tile: K's key and 16 values, V's value and 16 keys
  u32x4 kreg[CHUNKS], vreg[CHUNKS];
  uint32_t vscale[CHUNKS];
  auto cell_of = [&](int64_t t, int chunk, bool* here) {
    const int id = page_of(p.seq, r.b, static_cast<int>(t * kTile + 16 * chunk));
    *here = id >= 0;
    return static_cast<int64_t>(id < 0 ? 0 : id) * p.Hk + hk;
  };
  auto slot_of = [&](int64_t t, int chunk) {
    const uint32_t token_at = static_cast<uint32_t>(t * kTile + 16 * chunk);
    return static_cast<int>(token_at - fdiv(token_at, p.seq.page_div) * static_cast<uint32_t>(p.seq.page));
  };
  constexpr int KROW = D / 16;  // pieces of a key
  float my_scale = 0.0f;
  int my_absent = 0;
  auto load = [&](int64_t t) {
#pragma unroll
    for (int i = 0; i < CHUNKS; ++i) {
      const int piece = tid + 256 * i, key = piece / KROW, part = piece % KROW;
      bool here;
      const int64_t cell = cell_of(t, key >> 4, &here);
      kreg[i] = *reinterpret_cast<const u32x4*>(p.k_cache + cell * head_bytes + static_cast<int64_t>(slot_of(t, key >> 4) + (key & 15)) * D + 16 * part);
    }
    bool here;
    const int chunk = tid & 3;
    const int64_t cell = cell_of(t, chunk, &here);
    const int slot = slot_of(t, chunk);
    const uint32_t byte = here ? p.v_scale[cell] : 127u;
#pragma unroll
    for (int i = 0; i < CHUNKS; ++i) {
      const int d = (tid >> 2) + 64 * i;
      vreg[i] = *reinterpret_cast<const u32x4*>(p.v_cache + cell * head_bytes + static_cast<int64_t>(d) * p.seq.page + slot);
      vscale[i] = here ? byte : 256u;
    }
    my_scale = here ? e8m0_to_f32(p.k_scale[cell]) * p.c : 0.0f;
    my_absent = here ? 0 : 1;
  };
  auto store = [&](int64_t t, int buf) {
#pragma unroll
    for (int i = 0; i < CHUNKS; ++i) {
      const int piece = tid + 256 * i, key = piece / KROW, part = piece % KROW;
      const int at = (key & 32) | ((key >> 2 & 3) << 3) | ((key >> 4 & 1) << 2) | (key & 3);
      vec8* to = reinterpret_cast<vec8*>(&k_lds[buf][at * KP + 16 * part]);
      to[0] = ActTraits<T>::decode8_fp8(kreg[i].x, kreg[i].y);
      to[1] = ActTraits<T>::decode8_fp8(kreg[i].z, kreg[i].w);
    }
    const int chunk = tid & 3, key0 = static_cast<int>(t * kTile) + 16 * chunk;
    uint32_t byte = vscale[0];
    uint32_t nan_any = 0;
    if (byte > AttnTraits<T>::kMostV || key0 < any_lo || key0 + 16 > any_hi) {
      // values that nobody attends become 0 (whatever they hold), those of a
      // page whose scale is no number (or too large for T) NaN
      const bool here = byte < 256;
      const bool bad = here && byte > AttnTraits<T>::kMostV;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t keep = here ? byte_mask(any_lo - (key0 + 4 * j), any_hi - (key0 + 4 * j)) : 0u;
#pragma unroll
        for (int i = 0; i < CHUNKS; ++i) vreg[i][j] = (bad ? 0x7f7f7f7fu : vreg[i][j]) & keep;
      }
      if (bad || !here) byte = 127;
    }
    const float power = __uint_as_float((byte > AttnTraits<T>::kDown ? byte - AttnTraits<T>::kDown : 0u) << 23);
#pragma unroll
    for (int i = 0; i < CHUNKS; ++i) {
      const int d = (tid >> 2) + 64 * i;
      vec8* to = reinterpret_cast<vec8*>(&v_lds[buf][d * VP + 16 * chunk]);
      to[0] = decode8_power<T>(vreg[i].x, vreg[i].y, power);
      to[1] = decode8_power<T>(vreg[i].z, vreg[i].w, power);
#pragma unroll
      for (int j = 0; j < 4; ++j) nan_any |= nan_codes(vreg[i][j]);
    }
    if (tid < 4) scale_lds[buf][tid] = my_scale;
    const uint64_t absent = __ballot(my_absent != 0);
    if (tid == 0) absent_lds[buf] = static_cast<int>(absent & 15);
    if (nan_any != 0) nan_lds[buf] = static_cast<int>(t) + 1;
  };

  f32x16 acc[DT];
#pragma unroll
  for (int d = 0; d < DT; ++d)
#pragma unroll
    for (int j = 0; j < 16; ++j) acc[d][j] = 0.0f;
  float m = -INFINITY, l = 0.0f;

  if (p.seq.capacity > 0 && t_begin < t_end) {
    if (tid < 2) nan_lds[tid] = 0;
    __syncthreads();
    load(t_begin);
    store(t_begin, 0);
    __syncthreads();
    int buf = 0;
    for (int64_t t = t_begin; t < t_end; ++t, buf ^= 1) {
      if (t + 1 < t_end) load(t + 1);
      const int key0 = static_cast<int>(t * kTile);
      if (key0 < w_hi && key0 + kTile > w_lo) {
        const T* ks = k_lds[buf];
        const T* vs = v_lds[buf];
        f32x16 s[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
#pragma unroll
          for (int j = 0; j < 16; ++j) s[i][j] = 0.0f;
#pragma unroll
          for (int k = 0; k < KS; ++k)
            s[i] = Mfma32<T>::run(*reinterpret_cast<const vec8*>(ks + (32 * i + col) * KP + 16 * k + 8 * h), qf[k], s[i]);
        }
        const int absent = absent_lds[buf];
        const bool whole = key0 >= all_lo && key0 + kTile <= all_hi && absent == 0;
        uint32_t seen = 0xffffffffu;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float factor = scale_lds[buf][2 * i + h];
#pragma unroll
          for (int j = 0; j < 16; ++j) s[i][j] *= factor;
        }
        if (!whole) {
          seen = 0;
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const bool here = ((absent >> (2 * i + h)) & 1) == 0;
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              const int key = key0 + 32 * i + 16 * h + j;
              const bool on = here && key >= k_lo && key < k_hi;
              s[i][j] = on ? s[i][j] : -INFINITY;
              seen |= on ? 1u << (16 * i + j) : 0u;
            }
          }
        }
        float top = -INFINITY;
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int j = 0; j < 16; ++j) top = fmaxf(top, s[i][j]);
        top = fmaxf(top, __shfl_xor(top, 32, 64));
        if (__ballot(top > m) != 0) {
          const float now = fmaxf(m, top);
          const float shrink = __builtin_amdgcn_exp2f(m - (now > -INFINITY ? now : 0.0f));
          l *= shrink;
#pragma unroll
          for (int d = 0; d < DT; ++d) acc[d] *= shrink;
          m = now;
        }
        const float base = (m > -INFINITY ? m : 0.0f) - AttnTraits<T>::kLift;
        vec8 pf[4];
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const float e = __builtin_amdgcn_exp2f(s[i][j] - base);
            sum += e;
            pf[2 * i + (j >> 3)][j & 7] = static_cast<T>(e);  // the one rounding between the products
          }
        l += sum;
        if (nan_lds[buf] == static_cast<int>(t) + 1) {
          // a NaN among the values: 0 x NaN must not reach the rows that do not
          // attend it, so the NaN values that each output attends are counted
          // apart and left out of the product
#pragma unroll
          for (int d = 0; d < DT; ++d) {
            f32x16 hits;
#pragma unroll
            for (int j = 0; j < 16; ++j) hits[j] = 0.0f;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              vec8 v = *reinterpret_cast<const vec8*>(vs + (32 * d + col) * VP + 16 * (2 * (k >> 1) + h) + 8 * (k & 1)), flag, on;
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                const bool nan = !(static_cast<float>(v[j]) == static_cast<float>(v[j]));
                flag[j] = static_cast<T>(nan ? 1.0f : 0.0f);
                v[j] = nan ? static_cast<T>(0.0f) : v[j];
                on[j] = static_cast<T>((seen >> (8 * k + j)) & 1 ? 1.0f : 0.0f);
              }
              hits = Mfma32<T>::run(flag, on, hits);
              acc[d] = Mfma32<T>::run(v, pf[k], acc[d]);
            }
#pragma unroll
            for (int j = 0; j < 16; ++j) acc[d][j] = hits[j] > 0.0f ? NAN : acc[d][j];
          }
        } else {
#pragma unroll
          for (int d = 0; d < DT; ++d)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              acc[d] = Mfma32<T>::run(*reinterpret_cast<const vec8*>(vs + (32 * d + col) * VP + 16 * (2 * (k >> 1) + h) + 8 * (k & 1)), pf[k], acc[d]);
        }
      }
      if (t + 1 < t_end) store(t + 1, buf ^ 1);
      __syncthreads();
    }
  }
  l += __shfl_xor(l, 32, 64);
  if (!valid) return;
  if (pp.splits == 1) {
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

// Joins the parts of every row: D / 4 lanes for a row, a workgroup for a row
// tile and key head.
template <typename T, int D>
__global__ __launch_bounds__(256) void attn_prompt_join_kernel(const PromptParams pp) {
  constexpr int R = kPromptRows, LANES = D / 4, ROWS = 256 / LANES;
  const AttnParams& p = pp.a;
  const int64_t unit = blockIdx.x / p.Hk;
  const int hk = static_cast<int>(blockIdx.x - unit * p.Hk), lane = threadIdx.x % LANES;
  RowTile r;
  if (!row_tile_of<R>(p, unit, r)) return;
  const float* part = pp.part + (unit * p.Hk + hk) * pp.splits * attn_part_floats(R, D);
  for (int mine = threadIdx.x / LANES; mine < r.rows; mine += ROWS) {
    float m = -INFINITY, l = 0.0f;
    f32x4 o = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
    for (int i = 0; i < pp.splits; ++i) {
      const float* one = part + i * attn_part_floats(R, D);
      join(m, l, o, one[mine], one[R + mine], *reinterpret_cast<const f32x4*>(one + attn_part_head(R) + mine * D + 4 * lane));
    }
    const int row = r.row0 + mine, token = row / p.G;
    const int64_t at_row = (static_cast<int64_t>(r.token0) + token) * p.Hq + hk * p.G + (row - token * p.G);
    store_quad<T>(p, at_row, D, 4 * lane, m, l, o);
    if (lane == 0) store_lse<T>(p, at_row, m, l);
  }
}

template <typename T, int D>
int launch_t(const PromptParams& p, hipStream_t s) {
  hipLaunchKernelGGL((attn_prompt_kernel<T, D>), dim3(static_cast<uint32_t>(p.units * p.a.Hk * p.splits)), dim3(256), 0, s, p);
  if (p.splits > 1)
    hipLaunchKernelGGL((attn_prompt_join_kernel<T, D>), dim3(static_cast<uint32_t>(p.units * p.a.Hk)), dim3(256), 0, s, p);
  return hipGetLastError() == hipSuccess ? 0 : -1;
}

}  // namespace

int launch_attention_prompt(const AttentionArgs& a) {
  PromptParams p;
  p.a = make_attn(a);
  p.units = attn_row_tiles_most(a.M, a.Hq / a.Hk, a.seq.B);
  p.splits = static_cast<int32_t>(attn_prompt_splits(p.units * a.Hk, a.seq.max_pages * a.seq.page_size));
  p.part = static_cast<float*>(a.work);
  hipStream_t s = static_cast<hipStream_t>(a.stream);
  if (a.D == 128) return a.act == Act::BF16 ? launch_t<__bf16, 128>(p, s) : launch_t<_Float16, 128>(p, s);
  return a.act == Act::BF16 ? launch_t<__bf16, 64>(p, s) : launch_t<_Float16, 64>(p, s);
}

}  // namespace fp4w
