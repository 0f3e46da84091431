// Attention over the paged 8-bit cache, head sizes 64 and 128, for a few new
// tokens of each sequence (decode, drafted tokens).
//
//   s_t = scale q . K_t    O = sum_t 2^(s_t' - m) V_t / sum_t 2^(s_t' - m),  s' = s log2(e), m the largest s' so far
//
// Every key and value code is read once, and little is computed on it: the
// read of the cache is the bound.  So keys and values go from HBM to registers
// in the operand layout of the MFMAs, with no LDS in between:
//   * S^T = K Q^T by 16 x 16 x 32 MFMAs: a lane's 16 bytes of a key are its K
//     operand of two MFMAs (the sum over d may run in any order as long as Q
//     follows it).
//   * The row that a lane has in the result is one query row, four keys of it
//     a register quad.  Which key stands in which row of the K operand is
//     free, and is chosen so that a lane's 16 scores in a tile of 64 keys are
//     16 keys that lie side by side: those of the 16 bytes that it loads of
//     V^T.  So P^T goes from the softmax into the second MFMA as it is, and V,
//     which the cache holds transposed, needs no exchange either.
//   * Those 16 keys lie in one page (page_size % 16 == 0), so a lane has one
//     scale of K and one of V for a tile: K's is a factor of the scores, V's
//     the exponent operand of the conversion to T.
// The rows of a workgroup are the query heads of one key head, times the new
// tokens: up to 64 of them.
//
// The tiles of all sequences, one after the other, are cut into equal shares,
// one for each wave (or each group of waves with other rows of the same share):
// lengths may differ as they like, the host need not know them, and the
// workspace does not grow with them.  A sequence that lies in several shares is
// joined by a second kernel from the shares' partial results, in order, so a
// row's result does not depend on the order of work.  Short contexts have a
// workgroup for each sequence and key head instead (below).
//
// Measured with BF16, 40 query and 8 key heads of 128, both kernels: a token after
// 131000 (268 MB of cache) 56 us, 4.8 TB/s; 64 sequences of 300 to 8000 tokens
// (533 MB) 105 us, 5.1 TB/s, what a large copy reaches (a read alone: 5.9).  Short
// contexts are bound by loads that wait for each other (lengths, pages, codes): a
// token after 200 takes 7.6 us, after 900 12.  Of the two workgroups of a compute
// unit the older one is served first: after 131000 tokens one ends at 33 us and
// the other at 45.

#include <hip/hip_runtime.h>

#include "attention.h"

namespace fp4w {
namespace {

constexpr int kWaves = 4;
// Up to 16 rows over short contexts (by what the page table has room for), and no
// more workgroups than compute units: a workgroup of eight waves for each sequence
// and key head, in one launch and with nothing left to join.  With 8 key heads of
// 128, 32 sequences of 100 to 1000 tokens take 15 us so and 26 in shares; 1
// sequence of 200, 900 and 2000 tokens 7.6, 12.1 and 21 us against 11.1, 11.4 and
// 12.1 (but a call from the host costs 3 us less in one launch); 128 sequences 51
// against 42.
constexpr int kLocalWaves = 8, kLocalTokens = 1024, kLocalPlaces = 256;
constexpr int64_t kWideJoinRows = 128;  // up to so many rows, the join takes 1024 threads for each

struct DecodeParams {
  AttnParams a;
  int32_t* plan;    // first tile of each sequence among all, kSeqsPerLaunch + 1
  float* part;      // for each share and key head two partial results
  int32_t W;        // shares of a key head
  int32_t rows;     // max_new * G
};

// The tiles that sequence b's rows attend: [lo, lo + count).
struct Tiles {
  int lo, count;
};

__device__ __forceinline__ Tiles tiles_of(const DecodeParams& p, const SeqSpan& s) {
  if (s.rows == 0) return Tiles{0, 0};
  const int first = s.len - s.rows, rows = s.rows < p.a.max_new ? s.rows : p.a.max_new;
  int end = s.len < p.a.seq.capacity ? s.len : p.a.seq.capacity;
  if (p.a.causal && first + rows < end) end = first + rows;
  int begin = 0;
  if (p.a.window > 0 && first >= p.a.window) begin = first - p.a.window + 1;
  const int lo = begin / kTile, hi = end > 0 ? (end + kTile - 1) / kTile : 0;
  return Tiles{lo, hi > lo ? hi - lo : 1};  // rows that attend nothing still need their zeros
}

// A share's partial result of a sequence that it has a part of: the maxima and
// sums of its p.rows rows, then their unnormalised outputs.  A share ends at
// most one sequence that an earlier share began, and begins at most one that a
// later share ends: two places.
__device__ __forceinline__ float* part_of(const DecodeParams& p, int D, int hk, int w, bool begins) {
  return p.part + ((static_cast<int64_t>(w) * p.a.Hk + hk) * 2 + (begins ? 1 : 0)) * attn_part_floats(p.rows, D);
}

// 16 codes.  Those that one wave alone reads bypass what they would evict (about
// 3 % over 530 MB).
template <bool ONCE>
__device__ __forceinline__ u32x4 load_codes(const uint8_t* p) {
  if constexpr (ONCE)
    return __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p));
  else
    return *reinterpret_cast<const u32x4*>(p);
}

// RT x NR tiles of 16 rows: a wave has NR of them and a share of the tiles of
// keys; the RT waves of a workgroup with the same share read the same keys at
// about the same time, from L2.  A wave has the tiles of DEPTH steps ahead in
// registers; with DEPTH 2 it takes a SIMD for itself, and NR 2 converts each
// code once for 32 rows.  (launch_t() has the choice and its figures.)
// What is the same on a wave's lanes goes through readfirstlane, so that it
// stays in scalar registers (3 % with 64 rows).
//
// LOCAL: a workgroup of kLocalWaves waves has one sequence and key head to itself,
// and joins its waves' results in LDS.
template <typename T, int D, int RT, int NR, int DEPTH, bool LOCAL>
__global__ __launch_bounds__(LOCAL ? 64 * kLocalWaves : 256, LOCAL ? 1 : DEPTH == 1 ? 2 : 1) void attn_decode_kernel(const DecodeParams p) {
  constexpr int KL = D / 64, DT = D / 16, SHARES = kWaves / RT;
  typedef typename ActTraits<T>::vec8 vec8;
  __shared__ int prefix[kSeqsPerLaunch + 1];
  __shared__ int wave_total[kWaves];
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63, col = lane & 15, g = lane >> 4;
  const int row_tile = LOCAL ? 0 : wave / SHARES;
  const int group = blockIdx.x / p.a.Hk, hk = blockIdx.x - group * p.a.Hk, w = group * SHARES + wave % SHARES;
  int b = group, at = 0, stop = 1;

  if constexpr (!LOCAL) {
    // first tile of each sequence among all
    int own[kSeqsPerLaunch / 256], sum = 0;
#pragma unroll
    for (int i = 0; i < kSeqsPerLaunch / 256; ++i) {
      const int b = tid * (kSeqsPerLaunch / 256) + i;
      own[i] = b < p.a.seq.B ? tiles_of(p, seq_span(p.a.seq, b)).count : 0;
      sum += own[i];
    }
    int before = sum;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const int o = __shfl_up(before, off, 64);
      if (lane >= off) before += o;
    }
    if (lane == 63) wave_total[wave] = before;
    __syncthreads();
    before -= sum;
    for (int i = 0; i < wave; ++i) before += wave_total[i];
#pragma unroll
    for (int i = 0; i < kSeqsPerLaunch / 256; ++i) {
      const int b = tid * (kSeqsPerLaunch / 256) + i;
      if (b <= p.a.seq.B) prefix[b] = before;
      before += own[i];
    }
    if (tid == 255 && p.a.seq.B == kSeqsPerLaunch) prefix[kSeqsPerLaunch] = before;
    __syncthreads();
    if (blockIdx.x == 0)
      for (int i = tid; i <= p.a.seq.B; i += 256) p.plan[i] = prefix[i];
    const int total = __builtin_amdgcn_readfirstlane(prefix[p.a.seq.B]);
    int share = (total + p.W - 1) / p.W;
    share = share < 1 ? 1 : share;
    at = static_cast<int64_t>(w) * share < total ? w * share : total;
    stop = at + share < total ? at + share : total;
    if (at >= stop) return;
    b = __builtin_amdgcn_readfirstlane(last_not_above(p.a.seq.B, at, [&](int i) { return prefix[i]; }));
  }

  const int64_t head_bytes = static_cast<int64_t>(p.a.seq.page) * D;
  for (; at < stop; ++b) {
    const SeqSpan span = seq_span(p.a.seq, b);
    int t_begin, t_end, count;
    if constexpr (LOCAL) {
      count = tiles_of(p, span).count;
      if (count == 0) return;  // (the whole workgroup)
      const int each = (count + kLocalWaves - 1) / kLocalWaves;
      t_begin = wave * each < count ? wave * each : count;
      t_end = t_begin + each < count ? t_begin + each : count;
      at = stop;
    } else {
      const int from = __builtin_amdgcn_readfirstlane(prefix[b]), to = __builtin_amdgcn_readfirstlane(prefix[b + 1]);
      t_begin = at - from;
      count = to - from;
      if (count <= t_begin) continue;
      t_end = (stop < to ? stop : to) - from;
      at = from + t_end;
    }
    const int lo_tile = tiles_of(p, span).lo;
    const int first = span.len - span.rows, rows_i = span.rows < p.a.max_new ? span.rows : p.a.max_new;
    const int held = span.len < p.a.seq.capacity ? span.len : p.a.seq.capacity;

    // this lane's rows: their queries, and the tokens that they attend
    vec8 qf[NR][KL][2];
    int k_lo[NR], k_hi[NR];
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      const int row = 16 * (NR * row_tile + r) + col, i = row / p.a.G, head = hk * p.a.G + (row - i * p.a.G);
      const bool valid = i < rows_i;
      const int pos = first + i;
      k_hi[r] = !valid ? 0 : p.a.causal && pos + 1 < held ? pos + 1 : held;
      k_lo[r] = p.a.window > 0 && pos >= p.a.window ? pos - p.a.window + 1 : 0;
      const T* q = static_cast<const T*>(p.a.q) + (static_cast<int64_t>(span.first_row) + i) * p.a.q_stride + static_cast<int64_t>(head) * D;
#pragma unroll
      for (int j = 0; j < KL; ++j)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          u32x4 v = {0, 0, 0, 0};
          if (valid) v = *reinterpret_cast<const u32x4*>(q + 64 * j + 16 * g + 8 * e);
          v ^= p.a.flip;
          qf[r][j][e] = __builtin_bit_cast(vec8, v);
        }
    }
    // tokens that every valid row attends, and that any does
    const int last = first + rows_i - 1;
    const int all_lo = p.a.window > 0 && last >= p.a.window ? last - p.a.window + 1 : 0;
    const int all_hi = p.a.causal && first + 1 < held ? first + 1 : held;
    const int any_lo = p.a.window > 0 && first >= p.a.window ? first - p.a.window + 1 : 0;
    const int any_hi = p.a.causal && last + 1 < held ? last + 1 : held;

    f32x4 acc[NR][DT];
    float m[NR], l[NR];
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      m[r] = -INFINITY;
      l[r] = 0.0f;
#pragma unroll
      for (int d = 0; d < DT; ++d) acc[r][d] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }

    float c[NR];  // scale * log2(e), and kFarUp where the row's queries are held smaller
    auto hold_far_rows = [&]() {
#pragma unroll
      for (int r = 0; r < NR; ++r) {
        c[r] = p.a.c;
        if constexpr (AttnTraits<T>::kFarQueries) {
          uint32_t far = 0;
#pragma unroll
          for (int j = 0; j < KL; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const u32x4 v = __builtin_bit_cast(u32x4, qf[r][j][e]);
              far |= (far_pair(v.x) | far_pair(v.y)) | (far_pair(v.z) | far_pair(v.w));
            }
          if (__ballot(far != 0) != 0) {
            far |= __shfl_xor(far, 16, 64);
            far |= __shfl_xor(far, 32, 64);
            if (far != 0) {
              c[r] *= kFarUp;
#pragma unroll
              for (int j = 0; j < KL; ++j)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                  const u32x4 v = __builtin_bit_cast(u32x4, qf[r][j][e]);
                  qf[r][j][e] = __builtin_bit_cast(vec8, u32x4{down_pair(v.x), down_pair(v.y), down_pair(v.z), down_pair(v.w)});
                }
            }
          }
        }
      }
    };

    // pages of this lane's 16 keys as rows of a tile of K (chunk col / 4) and as keys of V (chunk g)
    struct Place {
      int id;         // -1: none
      uint32_t slot;  // of the chunk's first token
    };
    const int32_t* pages = p.a.seq.table + b * p.a.seq.max_pages;
    auto place_of = [&](int t, int chunk) {
      Place at;
      at.id = page_ahead(p.a.seq, pages, (lo_tile + t) * kTile + 16 * chunk, t < t_end, &at.slot);
      return at;
    };
    struct Tile {
      u32x4 k[4][KL], v[DT];
      uint32_t ks, vs;
      int id;  // page of this lane's chunk of V
    };
    auto load_k = [&](Tile& x, Place at_k, Place at_v) {
      const uint8_t* k = p.a.k_cache + (static_cast<int64_t>(at_k.id < 0 ? 0 : at_k.id) * p.a.Hk + hk) * head_bytes +
                         static_cast<int64_t>(at_k.slot + (col & 3)) * D + 16 * g;
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < KL; ++j) x.k[i][j] = load_codes<RT == 1>(k + 4 * i * D + 64 * j);
      const int64_t cell = static_cast<int64_t>(at_v.id < 0 ? 0 : at_v.id) * p.a.Hk + hk;
      x.ks = p.a.k_scale[cell];
      x.vs = p.a.v_scale[cell];
    };
    auto load_v = [&](Tile& x, Place at) {
      const uint8_t* v = p.a.v_cache + (static_cast<int64_t>(at.id < 0 ? 0 : at.id) * p.a.Hk + hk) * head_bytes +
                         static_cast<int64_t>(col) * p.a.seq.page + at.slot;
#pragma unroll
      for (int d = 0; d < DT; ++d) x.v[d] = load_codes<RT == 1>(v + static_cast<int64_t>(16 * d) * p.a.seq.page);
      x.id = at.id;
    };

    // A tile's work; the registers then take the tile at (at_k, at_v).
    auto step = [&](Tile& x, int t, Place at_k, Place at_v) {
      f32x4 s[NR][4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
#pragma unroll
        for (int r = 0; r < NR; ++r) s[r][i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int j = 0; j < KL; ++j) {
          const vec8 a0 = ActTraits<T>::decode8_fp8(x.k[i][j].x, x.k[i][j].y), a1 = ActTraits<T>::decode8_fp8(x.k[i][j].z, x.k[i][j].w);
#pragma unroll
          for (int r = 0; r < NR; ++r) {
            s[r][i] = ActTraits<T>::mfma(a0, qf[r][j][0], s[r][i]);
            s[r][i] = ActTraits<T>::mfma(a1, qf[r][j][1], s[r][i]);
          }
        }
      }
      const float k_scale = e8m0_to_f32(x.ks);
      uint32_t vs_now = x.vs;
      const int id_v = x.id;
      load_k(x, at_k, at_v);

      const int key0 = (lo_tile + t) * kTile;
      const int my0 = key0 + 16 * g;  // this lane's 16 keys
      if (AttnTraits<T>::kLeastV > 0 && __ballot(vs_now < AttnTraits<T>::kLeastV) != 0) vs_now = scale_of_zeros<T>(x.v, vs_now);
      const bool whole = key0 >= all_lo && key0 + kTile <= all_hi && __ballot(id_v < 0 || !held_scale<T>(vs_now)) == 0;
#pragma unroll
      for (int r = 0; r < NR; ++r) {
        const float factor = finite_factor(k_scale * c[r]);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) s[r][i][j] *= factor;
      }
      uint32_t nan_any = 0, seen[NR];
#pragma unroll
      for (int r = 0; r < NR; ++r) seen[r] = 0;
      if (!whole) {
        if (__ballot(!held_scale<T>(vs_now)) != 0) {
#pragma unroll
          for (int d = 0; d < DT; ++d)
#pragma unroll
            for (int j = 0; j < 4; ++j) x.v[d][j] = codes_held<T>(x.v[d][j], vs_now);
        }
#pragma unroll
        for (int r = 0; r < NR; ++r) {
          const int lo = id_v < 0 ? 16 : k_lo[r] - my0, hi = k_hi[r] - my0;  // of this lane's keys, [lo, hi) are attended
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const bool on = 4 * i + j >= lo && 4 * i + j < hi;
              s[r][i][j] = on ? s[r][i][j] : -INFINITY;
              seen[r] |= on ? 1u << (4 * i + j) : 0u;
            }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t keep = id_v < 0 ? 0 : byte_mask(any_lo - (my0 + 4 * j), any_hi - (my0 + 4 * j));
#pragma unroll
          for (int d = 0; d < DT; ++d) {
            const uint32_t word = x.v[d][j] & keep;
            x.v[d][j] = word;
            nan_any |= nan_codes(word);
          }
        }
        vs_now = id_v < 0 ? 127 : scale_held<T>(vs_now);
      }
      float top[NR];
      bool grown = false;
#pragma unroll
      for (int r = 0; r < NR; ++r) {
        top[r] = whole || seen[r] != 0 ? kLowest : -INFINITY;
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) top[r] = fmaxf(top[r], s[r][i][j]);
        top[r] = fmaxf(top[r], __shfl_xor(top[r], 16, 64));
        top[r] = fmaxf(top[r], __shfl_xor(top[r], 32, 64));
        grown = grown || top[r] > m[r];
      }
      if (__ballot(grown) != 0) {
#pragma unroll
        for (int r = 0; r < NR; ++r) {
          const float now = fmaxf(m[r], top[r]);
          const float shrink = __builtin_amdgcn_exp2f(m[r] - (now > -INFINITY ? now : 0.0f));
          l[r] *= shrink;
#pragma unroll
          for (int d = 0; d < DT; ++d) acc[r][d] *= shrink;
          m[r] = now;
        }
      }
      vec8 pf[NR][2];
#pragma unroll
      for (int r = 0; r < NR; ++r) {
        const float base = (m[r] > -INFINITY ? m[r] : 0.0f) - AttnTraits<T>::kLift;
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float e = __builtin_amdgcn_exp2f(s[r][i][j] - base);
            sum += e;
            pf[r][i >> 1][4 * (i & 1) + j] = static_cast<T>(e);  // the one rounding between the products
          }
        l[r] += sum;
      }
      if (!whole && __ballot(nan_any != 0) != 0) {
        // A NaN among the values: 0 x NaN must not reach the rows that do not
        // attend it.  Count for each output the NaN values that it attends,
        // and take them out of the product.
#pragma unroll
        for (int d = 0; d < DT; ++d) {
          f32x4 hits[NR];
#pragma unroll
          for (int r = 0; r < NR; ++r) hits[r] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            vec8 flag;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const uint32_t n = nan_codes(x.v[d][2 * h + (j >> 2)]);
              flag[j] = static_cast<T>((n >> (8 * (j & 3) + 7)) & 1 ? 1.0f : 0.0f);
            }
#pragma unroll
            for (int r = 0; r < NR; ++r) {
              vec8 on;
#pragma unroll
              for (int j = 0; j < 8; ++j) on[j] = static_cast<T>((seen[r] >> (8 * h + j)) & 1 ? 1.0f : 0.0f);
              hits[r] = ActTraits<T>::mfma(flag, on, hits[r]);
            }
          }
#pragma unroll
          for (int j = 0; j < 4; ++j) x.v[d][j] &= ~((nan_codes(x.v[d][j]) >> 7) * 0xffu);
#pragma unroll
          for (int r = 0; r < NR; ++r)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[r][d][j] = hits[r][j] > 0.0f ? NAN : acc[r][d][j];
        }
      }
      const float power = __uint_as_float((vs_now > AttnTraits<T>::kDown ? vs_now - AttnTraits<T>::kDown : 0u) << 23);
#pragma unroll
      for (int d = 0; d < DT; ++d) {
        const vec8 a0 = decode8_power<T>(x.v[d].x, x.v[d].y, power), a1 = decode8_power<T>(x.v[d].z, x.v[d].w, power);
#pragma unroll
        for (int r = 0; r < NR; ++r) {
          acc[r][d] = ActTraits<T>::mfma(a0, pf[r][0], acc[r][d]);
          acc[r][d] = ActTraits<T>::mfma(a1, pf[r][1], acc[r][d]);
        }
      }
      load_v(x, at_v);
    };

    // Loads run ahead by DEPTH tiles, and past the last one they go on at page 0:
    // a branch around them would make the compiler wait for all loads in flight
    // wherever it waits for any.  (Without pages there is nothing to load, and no
    // key to attend.)  No branch belongs there in the LOCAL form either, though it
    // takes 0.8 us of 12 after 900 tokens: this compiler (ROCm 7.2) then loses the
    // live ranges of the last value rows' codes in its scheduler and gives their
    // registers to the softmax, and outputs are wrong (-verify-machineinstrs says
    // so, "no live subrange at use"; without the scheduler the same source is
    // right).  build.py has the verifier on for this file and attention_prompt.hip,
    // whose branch around its loads passes.
    int t = t_begin;
    if (p.a.seq.capacity > 0 && t < t_end) {
      Tile tile[DEPTH];
      Place next_k = place_of(t, col >> 2), next_v = place_of(t, g);
#pragma unroll
      for (int i = 0; i < DEPTH; ++i) {
        load_k(tile[i], next_k, next_v);
        load_v(tile[i], next_v);
        next_k = place_of(t + i + 1, col >> 2);
        next_v = place_of(t + i + 1, g);
      }
      hold_far_rows();  // (behind the first loads: it waits for the queries)
      for (; t < t_end; t += DEPTH) {
#pragma unroll
        for (int i = 0; i < DEPTH; ++i) {
          if (t + i < t_end) {
            const Place after_k = place_of(t + i + DEPTH + 1, col >> 2), after_v = place_of(t + i + DEPTH + 1, g);
            step(tile[i], t + i, next_k, next_v);
            next_k = after_k;
            next_v = after_v;
          }
        }
      }
    }

#pragma unroll
    for (int r = 0; r < NR; ++r) {
      l[r] += __shfl_xor(l[r], 16, 64);
      l[r] += __shfl_xor(l[r], 32, 64);
    }
    if constexpr (LOCAL) {  // pairwise, lane by lane
      static_assert(NR == 1, "one row tile");
      __shared__ f32x4 red_o[kLocalWaves / 2][DT][64];
      __shared__ float red_m[kLocalWaves / 2][64], red_l[kLocalWaves / 2][64];
#pragma unroll
      for (int half = kLocalWaves / 2; half > 0; half >>= 1) {
        if (wave >= half && wave < 2 * half) {
          red_m[wave - half][lane] = m[0];
          red_l[wave - half][lane] = l[0];
#pragma unroll
          for (int d = 0; d < DT; ++d) red_o[wave - half][d][lane] = acc[0][d];
        }
        __syncthreads();
        if (wave < half) {
          const float m0 = m[0], l0 = l[0];
#pragma unroll
          for (int d = 0; d < DT; ++d) {
            m[0] = m0;
            l[0] = l0;
            join(m[0], l[0], acc[0][d], red_m[wave][lane], red_l[wave][lane], red_o[wave][d][lane]);
          }
        }
        __syncthreads();
      }
      if (wave != 0) return;
      t_begin = 0;
      t_end = count;
    }
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      const int out = 16 * (NR * row_tile + r) + col, i = out / p.a.G;
      if (i < rows_i) {
        if (t_begin == 0 && t_end == count) {  // the whole sequence
          const int64_t at_row = (static_cast<int64_t>(span.first_row) + i) * p.a.Hq + hk * p.a.G + (out - i * p.a.G);
#pragma unroll
          for (int d = 0; d < DT; ++d) store_quad<T>(p.a, at_row, D, 16 * d + 4 * g, m[r], l[r], acc[r][d]);
          if (g == 0) store_lse<T>(p.a, at_row, m[r], l[r]);
        } else {
          float* part = part_of(p, D, hk, w, t_begin == 0);
          float* row = part + attn_part_head(p.rows) + out * D + 4 * g;
#pragma unroll
          for (int d = 0; d < DT; ++d) *reinterpret_cast<f32x4*>(row + 16 * d) = acc[r][d];
          if (g == 0) {
            part[out] = m[r];
            part[p.rows + out] = l[r];
          }
        }
      }
    }
  }
}

// Joins the partial results of the sequences that lie in several shares: THREADS
// threads for a row of a head, D / 4 of them for one partial result, AT_ONCE
// results of each loaded together.
template <typename T, int D, int THREADS, int AT_ONCE>
__global__ __launch_bounds__(THREADS) void attn_join_kernel(const DecodeParams p) {
  constexpr int LANES = D / 4, GROUPS = THREADS / LANES;
  __shared__ float red_m[GROUPS], red_l[GROUPS];
  __shared__ f32x4 red_o[GROUPS][LANES];
  const int tid = threadIdx.x, group = tid / LANES, lane = tid % LANES;
  const int64_t row = seq_start(p.a.seq, 0) + blockIdx.x / p.a.Hq;
  const int h = static_cast<int>(blockIdx.x % p.a.Hq);
  if (row >= seq_start(p.a.seq, p.a.seq.B)) return;
  const int b = last_not_above(p.a.seq.B, row, [&](int i) { return seq_start(p.a.seq, i); });
  const int i = static_cast<int>(row) - seq_start(p.a.seq, b);
  const int total = p.plan[p.a.seq.B], from = p.plan[b], to = p.plan[b + 1];
  int share = (total + p.W - 1) / p.W;
  share = share < 1 ? 1 : share;
  const int w0 = from / share, w1 = (to - 1) / share;
  if (i >= p.a.max_new || to <= from || w0 == w1) return;
  const int hk = h / p.a.G, mine = i * p.a.G + (h - hk * p.a.G);
  float m = -INFINITY, l = 0.0f;
  f32x4 o = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int w = w0 + group; w <= w1; w += GROUPS * AT_ONCE) {
    float pm[AT_ONCE], pl[AT_ONCE];
    f32x4 po[AT_ONCE];
#pragma unroll
    for (int j = 0; j < AT_ONCE; ++j) {
      const int v = w + j * GROUPS <= w1 ? w + j * GROUPS : w;
      const float* part = part_of(p, D, hk, v, v == w0);
      pm[j] = part[mine];
      pl[j] = part[p.rows + mine];
      po[j] = *reinterpret_cast<const f32x4*>(part + attn_part_head(p.rows) + mine * D + 4 * lane);
      if (w + j * GROUPS > w1) pm[j] = -INFINITY, pl[j] = 0.0f, po[j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }
#pragma unroll
    for (int j = 0; j < AT_ONCE; ++j) join(m, l, o, pm[j], pl[j], po[j]);
  }
  // pairwise, so that the order does not hang on how many there are
#pragma unroll
  for (int half = GROUPS / 2; half > 0; half >>= 1) {
    if (group >= half && group < 2 * half) {
      if (lane == 0) {
        red_m[group] = m;
        red_l[group] = l;
      }
      red_o[group][lane] = o;
    }
    __syncthreads();
    if (group < half) join(m, l, o, red_m[group + half], red_l[group + half], red_o[group + half][lane]);
  }
  if (group != 0) return;
  store_quad<T>(p.a, row * p.a.Hq + h, D, 4 * lane, m, l, o);
  if (lane == 0) store_lse<T>(p.a, row * p.a.Hq + h, m, l);
}

template <typename T, int D, int RT, int NR, int DEPTH>
int launch_rows(DecodeParams p, int64_t join_rows, hipStream_t s) {
  const int groups = attn_groups(p.a.Hk, DEPTH == 1 ? 2 : 1);
  p.W = groups * (kWaves / RT);
  hipLaunchKernelGGL((attn_decode_kernel<T, D, RT, NR, DEPTH, false>), dim3(groups * p.a.Hk), dim3(256), 0, s, p);
  const dim3 grid(static_cast<uint32_t>(join_rows * p.a.Hq));
  // few rows may have many partial results each, many rows have few
  const int64_t rows = join_rows * p.a.Hq, most = p.a.seq.capacity / kTile;
  if (rows <= kWideJoinRows && most > 64)
    hipLaunchKernelGGL((attn_join_kernel<T, D, 1024, 8>), grid, dim3(1024), 0, s, p);
  else if (rows <= 8 * kWideJoinRows)
    hipLaunchKernelGGL((attn_join_kernel<T, D, 256, 4>), grid, dim3(256), 0, s, p);
  else
    hipLaunchKernelGGL((attn_join_kernel<T, D, 64, 4>), grid, dim3(64), 0, s, p);
  return hipGetLastError() == hipSuccess ? 0 : -1;
}

template <typename T, int D>
int launch_t(const DecodeParams& p, int64_t join_rows, hipStream_t s) {
  // attn_shares() has the same choice.  With two row tiles and two steps a wave,
  // 25 and 50 rows of D = 128 take 71 and 93 us over 8 times 16000 tokens, with
  // one of each 75 and 108.  But 5 rows take 60 us over 131000 tokens with two
  // steps a wave and 56 with one, on two waves a SIMD; and up to 28 rows of D = 64
  // 30 us against 22 over 16 windows of 4096 tokens, where the partial results
  // weigh more.
  const int rows = p.rows;
  if (rows <= 16 && p.a.seq.capacity <= kLocalTokens && p.a.seq.B * p.a.Hk <= kLocalPlaces) {
    hipLaunchKernelGGL((attn_decode_kernel<T, D, 1, 1, 1, true>), dim3(p.a.seq.B * p.a.Hk), dim3(64 * kLocalWaves), 0, s, p);
    return hipGetLastError() == hipSuccess ? 0 : -1;
  }
  if (rows <= 16) return launch_rows<T, D, 1, 1, 1>(p, join_rows, s);
  if constexpr (D == 64)
    return rows <= 32 ? launch_rows<T, D, 2, 1, 1>(p, join_rows, s) : launch_rows<T, D, 4, 1, 1>(p, join_rows, s);
  else
    return rows <= 32 ? launch_rows<T, D, 1, 2, 2>(p, join_rows, s) : launch_rows<T, D, 2, 2, 2>(p, join_rows, s);
}

}  // namespace

int launch_attention_decode(const AttentionArgs& a) {
  DecodeParams p;
  p.a = make_attn(a);
  p.rows = p.a.max_new * p.a.G;
  p.plan = static_cast<int32_t*>(a.work);
  p.part = reinterpret_cast<float*>(static_cast<unsigned char*>(a.work) + kAttnPlanBytes);
  hipStream_t s = static_cast<hipStream_t>(a.stream);
  for (int64_t b = 0; b < a.seq.B; b += kSeqsPerLaunch) {
    SeqArgs seq = a.seq;
    seq.B = a.seq.B - b < kSeqsPerLaunch ? a.seq.B - b : kSeqsPerLaunch;
    seq.lens += b;
    if (seq.starts) seq.starts += b;
    if (seq.table) seq.table += b * seq.max_pages;
    p.a.seq = make_seqs(seq, a.M);
    p.a.seq.row0 = static_cast<int32_t>(b);
    const int64_t rows = seq.starts ? a.M : seq.B;
    int rc;
    if (a.D == 128)
      rc = a.act == Act::BF16 ? launch_t<__bf16, 128>(p, rows, s) : launch_t<_Float16, 128>(p, rows, s);
    else
      rc = a.act == Act::BF16 ? launch_t<__bf16, 64>(p, rows, s) : launch_t<_Float16, 64>(p, rows, s);
    if (rc != 0) return rc;
  }
  return 0;
}

}  // namespace fp4w
