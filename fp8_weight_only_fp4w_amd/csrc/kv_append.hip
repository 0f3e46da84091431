// New keys and values into the paged cache in 8 bits.  For each page that a
// sequence's new tokens reach and each head, for keys and values apart:
//
//   a    = max |x| over the finite new values of the page
//   e    = the smallest exponent with a <= 448 2^e; not below the page's own
//          where earlier tokens of the sequence are in it
//   code = e4m3(x 2^-e)
//
// Where the page's exponent grows, its earlier codes are scaled down with it:
// powers of two make that exact but for codes that leave the normal range.
// Keys are normed and rotated in FP32 on the way and not rounded in between.
//
// A workgroup owns one page and head, so the scale needs no atomics and the
// result does not depend on the order of work.
//
// What is read and written is small; the chain of a workgroup (lengths, page,
// values, maximum, codes) is the time: one token of 8 key and 40 query heads of
// 128 takes 4.9 us with its norms and rotation, 77 of them 5.7 us, 7400 tokens
// without queries 15 to 16 us (3 TB/s; as two launches, with values written token
// by token, 70), with norms, rotation and 40 query heads 45.5 (4.4 TB/s).

#include <hip/hip_runtime.h>

#include "qk_rows.h"

namespace fp4w {
namespace {

struct AppendParams {
  const void* k;
  const void* v;
  int64_t k_stride, v_stride;
  int32_t Hk, D;
  const void* k_weight;
  Rope rope;
  Seqs seq;
  uint8_t* k_cache;
  uint8_t* k_scale;
  uint8_t* v_cache;
  uint8_t* v_scale;
};

// The pages that sequence b's new tokens reach are given numbers from
// starts[b] / page + 2 b on: n tokens reach at most n / page + 2 pages, so the
// numbers of two sequences never meet.
__device__ __forceinline__ int64_t first_unit(const Seqs& s, int b) {
  return static_cast<int64_t>(fdiv(static_cast<uint32_t>(seq_start(s, b)), s.page_div)) + 2 * static_cast<int64_t>(b);
}
inline int64_t most_units(const Seqs& s) { return s.starts ? s.M / s.page + 2 * static_cast<int64_t>(s.B) : s.B; }

// One page's share of a sequence's new tokens: slots [lo, hi) of page `id`
// are rows row .. of the call, at positions position ..; id -1: nothing to do.
struct Run {
  int id, lo, hi, row, position;
};

__device__ __forceinline__ Run run_of(const Seqs& s, int64_t unit) {
  // (without starts a sequence has one page: its units are counted one by one)
  const int b = s.starts ? last_not_above(s.B, unit, [&](int i) { return first_unit(s, i); }) : static_cast<int>(unit);
  const SeqSpan q = seq_span(s, b);
  Run r{-1, 0, 0, 0, 0};
  int first = q.len - q.rows, row = q.first_row;
  if (first < 0) {  // more new rows than tokens: the rows before the first token are absent
    row -= first;
    first = 0;
  }
  const int64_t nth = s.starts ? unit - first_unit(s, b) : 0;  // below 0 only where starts falls
  const int64_t page = static_cast<int64_t>(fdiv(static_cast<uint32_t>(first), s.page_div)) + nth;
  const int64_t from = page * s.page;
  if (nth < 0 || q.rows == 0 || q.len <= first || from >= q.len || from >= s.capacity) return r;
  const int begin = from > first ? static_cast<int>(from) : first;
  const int64_t next = from + s.page;
  const int end = next < q.len ? static_cast<int>(next) : q.len;
  r.id = page_of(s, b, begin);
  r.lo = begin - static_cast<int>(from);
  r.hi = end - static_cast<int>(from);
  r.row = row + (begin - first);
  r.position = begin;
  return r;
}

// Any D, page size, alignment and stride: a wave per token through LDS, twice
// (the page's scale needs every token first).
template <typename T>
__global__ __launch_bounds__(256) void kv_append_generic_kernel(const AppendParams p, int64_t units) {
  __shared__ float buf[4][kMaxHead];
  __shared__ float tops[4];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, tid = threadIdx.x;
  const int D = p.D, page = p.seq.page;
  for (int64_t work = blockIdx.x; work < units * p.Hk * 2; work += gridDim.x) {
    const bool value = work & 1;
    const int64_t pair = work >> 1, unit = pair / p.Hk;
    const int head = static_cast<int>(pair - unit * p.Hk);
    const Run r = run_of(p.seq, unit);
    if (r.id < 0) continue;  // the same on every thread
    const Rope none{nullptr, nullptr, nullptr, 0, 0, false, 0.0f, 0.0f};
    const Rope& rope = value ? none : p.rope;
    const T* weight = value ? nullptr : static_cast<const T*>(p.k_weight);
    const int64_t stride = value ? p.v_stride : p.k_stride;
    const T* x = static_cast<const T*>(value ? p.v : p.k) + r.row * stride + static_cast<int64_t>(head) * D;
    const int64_t at = static_cast<int64_t>(r.id) * p.Hk + head;
    uint8_t* codes = (value ? p.v_cache : p.k_cache) + at * page * D;
    uint8_t* scale = (value ? p.v_scale : p.k_scale) + at;
    const uint32_t before = *scale;
    const int n = r.hi - r.lo;
    const int64_t ts = value ? 1 : D, ds = value ? page : 1;  // steps of a token and of a value in the page
    auto load = [&](int i) {
      const int64_t position = p.rope.positions && i < n ? p.rope.positions[r.row + i] : r.position + i;
      head_to_lds(i < n ? x + i * stride : nullptr, D, weight, rope, position, buf[wave]);
    };
    float top = 0.0f;
    for (int i = 0; i < n; i += 4) {
      load(i + wave);
      if (i + wave < n)
        for (int d = lane; d < D; d += 64) top = fmaxf(top, finite_abs(buf[wave][d]));
      __syncthreads();
    }
    for (int off = 32; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor(top, off, 64));
    if (lane == 0) tops[wave] = top;
    __syncthreads();
    uint32_t e = e8m0_for(fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3])));
    if (r.lo > 0 && before > e) e = before;
    if (r.lo > 0 && e != before) {
      const float down = e8m0_to_f32(before) * e8m0_inverse(e);
      for (int64_t i = tid; i < static_cast<int64_t>(r.lo) * D; i += 256) {
        const int64_t t = value ? i % r.lo : i / D, d = value ? i / r.lo : i - t * D;
        uint8_t* c = codes + t * ts + d * ds;
        const float f = e4m3_to_f32<0>(*c) * down;
        *c = static_cast<uint8_t>(e4m3_pair(f, 0.0f));
      }
    }
    const float inv = e == 255 ? NAN : e8m0_inverse(e);
    for (int i = 0; i < n; i += 4) {
      load(i + wave);
      if (i + wave < n)
        for (int d = lane; d < D; d += 64)
          codes[(r.lo + i + wave) * ts + d * ds] = static_cast<uint8_t>(e4m3_pair(buf[wave][d] * inv, 0.0f));
      __syncthreads();
    }
    if (tid == 0) *scale = static_cast<uint8_t>(e);
    __syncthreads();
  }
}

// Eight values as codes.
__device__ __forceinline__ u32x2 codes8(const float* v, float inv) {
  u32x2 c;
  c.x = e4m3_pair(v[0] * inv, v[1] * inv) | e4m3_pair(v[2] * inv, v[3] * inv) << 16;
  c.y = e4m3_pair(v[4] * inv, v[5] * inv) | e4m3_pair(v[6] * inv, v[7] * inv) << 16;
  return c;
}

// D = 16 LANES, page_size % 16 == 0, at most PASSES * THREADS / LANES tokens of
// a page in the call, everything in 16-byte pieces.  A workgroup has the keys or
// the values of one page and head: LANES lanes a token, whose values stay in
// registers between the maximum and the codes.  Values go through LDS to lie
// along the tokens.  The workgroups behind the pages' have the queries.
template <typename T, int LANES, int THREADS, int PASSES>
__global__ __launch_bounds__(THREADS) void kv_append_kernel(const AppendParams p, const QkParams qp, uint32_t units, FastDiv by_heads, int q_passes) {
  constexpr int D = 16 * LANES, TOKENS = THREADS / LANES, WAVES = THREADS / 64;
  extern __shared__ uint32_t turned[];  // [D][page + 4] bytes
  __shared__ float tops[WAVES];
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, t = tid % LANES, page = p.seq.page;
  const uint32_t cells = units * p.Hk;
  if (blockIdx.x >= 2 * cells) {
    const uint32_t u = (blockIdx.x - 2 * cells) * WAVES + wave, m = u / q_passes;
    if (m < qp.M) qk_row<T, LANES>(qp, m, static_cast<int>(u - m * q_passes));
    return;
  }
  const bool value = blockIdx.x >= cells;
  const uint32_t cell_at = value ? blockIdx.x - cells : blockIdx.x, unit = fdiv(cell_at, by_heads);
  const int head = static_cast<int>(cell_at - unit * p.Hk);
  const Run r = run_of(p.seq, unit);
  if (r.id < 0) return;  // the same on every thread
  const int n = r.hi - r.lo;
  const int64_t at = static_cast<int64_t>(r.id) * p.Hk + head;
  uint8_t* codes = (value ? p.v_cache : p.k_cache) + at * page * D;
  uint8_t* scale = (value ? p.v_scale : p.k_scale) + at;
  const uint32_t before = r.lo > 0 ? *scale : 0;
  const int64_t stride = value ? p.v_stride : p.k_stride;
  const T* x = static_cast<const T*>(value ? p.v : p.k) + r.row * stride + head * D;
  const LaneChunks my = lane_chunks(t, D, value ? 0 : p.rope.dims);
  LaneHead<T> v[PASSES];
#pragma unroll
  for (int i = 0; i < PASSES; ++i) {
    const int token = tid / LANES + i * TOKENS;
    if (token < n) v[i].load(x + token * stride, my);
  }
  float top = 0.0f;
#pragma unroll
  for (int i = 0; i < PASSES; ++i) {
    const int token = tid / LANES + i * TOKENS;
    if (token < n) {
      if (!value) {
        if (p.k_weight) v[i].template norm<LANES>(static_cast<const T*>(p.k_weight), my, p.rope);
        if (p.rope.cos) {
          LaneAngles angles;
          angles.load(p.rope, my, p.rope.positions ? p.rope.positions[r.row + token] : r.position + token);
          v[i].rotate(angles, my, p.rope);
        }
      }
#pragma unroll
      for (int j = 0; j < 16; ++j) top = fmaxf(top, finite_abs(v[i].v[j]));
    }
  }
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor(top, off, 64));
  if (WAVES > 1) {
    if (lane == 0) tops[wave] = top;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < WAVES; ++i) top = fmaxf(top, tops[i]);
  }
  uint32_t e = e8m0_for(top);
  if (before > e) e = before;
  if (r.lo > 0 && e != before) {  // the earlier tokens' codes follow
    const float down = e8m0_to_f32(before) * e8m0_inverse(e);
    if (value) {
      const int words = (r.lo + 3) >> 2;  // of each value's tokens; the last one may hold others' slots too
      for (int i = tid; i < words * D; i += THREADS) {
        const int d = i / words, k = i - d * words;
        uint8_t* c = codes + d * page + 4 * k;
        const uint32_t w = scale_codes(*reinterpret_cast<const uint32_t*>(c), down);
        if (4 * k + 4 <= r.lo) {
          *reinterpret_cast<uint32_t*>(c) = w;
        } else {
          for (int j = 0; j < r.lo - 4 * k; ++j) c[j] = static_cast<uint8_t>(w >> (8 * j));
        }
      }
    } else {
      uint32_t* c = reinterpret_cast<uint32_t*>(codes);
      for (int i = tid; i < r.lo * D / 4; i += THREADS) c[i] = scale_codes(c[i], down);
    }
  }
  const float inv = e == 255 ? NAN : e8m0_inverse(e);
  if (tid == 0) *scale = static_cast<uint8_t>(e);
  if (!value) {
#pragma unroll
    for (int i = 0; i < PASSES; ++i) {
      const int token = tid / LANES + i * TOKENS;
      if (token < n) {
        uint8_t* c = codes + static_cast<int64_t>(r.lo + token) * D;
        *reinterpret_cast<u32x2*>(c + 8 * my.a) = codes8(v[i].v, inv);
        *reinterpret_cast<u32x2*>(c + 8 * my.b) = codes8(v[i].v + 8, inv);
      }
    }
    return;
  }
  if (n == 1) {
    if (tid < LANES) {
      const u32x2 a = codes8(v[0].v, inv), b = codes8(v[0].v + 8, inv);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        codes[(8 * my.a + j) * page + r.lo] = static_cast<uint8_t>(a[j >> 2] >> (8 * (j & 3)));
        codes[(8 * my.b + j) * page + r.lo] = static_cast<uint8_t>(b[j >> 2] >> (8 * (j & 3)));
      }
    }
    return;
  }
  uint8_t* lds = reinterpret_cast<uint8_t*>(turned);
  const int pitch = page + 4;
#pragma unroll
  for (int i = 0; i < PASSES; ++i) {
    const int token = tid / LANES + i * TOKENS;
    if (token < n) {
      const u32x2 a = codes8(v[i].v, inv), b = codes8(v[i].v + 8, inv);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        lds[(8 * my.a + j) * pitch + r.lo + token] = static_cast<uint8_t>(a[j >> 2] >> (8 * (j & 3)));
        lds[(8 * my.b + j) * pitch + r.lo + token] = static_cast<uint8_t>(b[j >> 2] >> (8 * (j & 3)));
      }
    }
  }
  __syncthreads();
  const int words = page >> 2;
  for (int i = tid; i < words * D; i += THREADS) {
    const int d = i / words, k = i - d * words;
    const uint32_t w = turned[d * (pitch >> 2) + k];
    uint8_t* c = codes + d * page + 4 * k;
    if (4 * k >= r.lo && 4 * k + 4 <= r.hi) {
      *reinterpret_cast<uint32_t*>(c) = w;
    } else {
      for (int j = 0; j < 4; ++j)
        if (4 * k + j >= r.lo && 4 * k + j < r.hi) c[j] = static_cast<uint8_t>(w >> (8 * j));
    }
  }
}

template <typename T, int LANES, int THREADS, int PASSES>
int launch_pages(const AppendParams& p, const QkParams& qp, hipStream_t s) {
  const int64_t units = most_units(p.seq);
  const int passes = qp.Hq > 0 ? (qp.Hq + 64 / LANES - 1) / (64 / LANES) : 1;  // waves of a row's queries
  const int64_t q_blocks = qp.Hq > 0 ? (qp.M * passes + THREADS / 64 - 1) / (THREADS / 64) : 0, blocks = 2 * units * p.Hk + q_blocks;
  if (blocks * THREADS >= (int64_t(1) << 32) || qp.M * passes >= (int64_t(1) << 32)) return 1;
  const int lds = p.seq.starts ? 16 * LANES * (p.seq.page + 4) : 0;
  hipLaunchKernelGGL((kv_append_kernel<T, LANES, THREADS, PASSES>), dim3(static_cast<uint32_t>(blocks)), dim3(THREADS), lds, s, p, qp,
                     static_cast<uint32_t>(units), make_fastdiv(static_cast<uint32_t>(p.Hk)), passes);
  return hipGetLastError() == hipSuccess ? 0 : -1;
}

// One token for each sequence: a wave is enough.  Else 256 threads, and as many
// passes as a whole page takes.
template <typename T, int LANES>
int launch_lanes(const AppendParams& p, const QkParams& qp, hipStream_t s) {
  if (!p.seq.starts) return launch_pages<T, LANES, 64, 1>(p, qp, s);
  const int passes = (p.seq.page * LANES + 255) / 256;
  return passes <= 1 ? launch_pages<T, LANES, 256, 1>(p, qp, s)
         : passes <= 2 ? launch_pages<T, LANES, 256, 2>(p, qp, s) : launch_pages<T, LANES, 256, 4>(p, qp, s);
}

// 1: nothing launched, the generic kernels have to take it.
template <typename T>
int launch_vec(const AppendParams& p, const QkParams& qp, hipStream_t s) {
  switch (p.D) {
    case 16: return launch_lanes<T, 1>(p, qp, s);
    case 32: return launch_lanes<T, 2>(p, qp, s);
    case 64: return launch_lanes<T, 4>(p, qp, s);
    case 128: return launch_lanes<T, 8>(p, qp, s);
    case 256: return launch_lanes<T, 16>(p, qp, s);
    case 512: return launch_lanes<T, 32>(p, qp, s);
    case 1024: return launch_lanes<T, 64>(p, qp, s);
  }
  return 1;
}

template <typename T>
int launch_generic(const AppendParams& p, hipStream_t s) {
  const int64_t units = most_units(p.seq), work = units * p.Hk * 2;
  const int grid = static_cast<int>(work < (1 << 20) ? work : 1 << 20);
  if (grid > 0) hipLaunchKernelGGL(kv_append_generic_kernel<T>, dim3(grid), dim3(256), 0, s, p, units);
  return hipGetLastError() == hipSuccess ? 0 : -1;
}

}  // namespace

int launch_kv_append(const KvAppendArgs& a, bool vec) {
  const AppendParams p{a.k, a.v, a.k_stride, a.v_stride, static_cast<int32_t>(a.Hk), static_cast<int32_t>(a.D), a.rope.k_weight,
                       make_rope(a.rope), make_seqs(a.seq, a.M), a.k_cache, a.k_scale, a.v_cache, a.v_scale};
  hipStream_t s = static_cast<hipStream_t>(a.stream);
  if (vec && a.Hk > 0) {
    const QkParams q{a.q, nullptr, a.q_out, nullptr, a.q_stride, 0, a.q_out_stride, 0, a.M, a.q ? static_cast<int32_t>(a.Hq) : 0, 0,
                     static_cast<int32_t>(a.D), a.rope.q_weight, nullptr, p.rope, p.seq};
    const int rc = a.act == Act::BF16 ? launch_vec<__bf16>(p, q, s) : launch_vec<_Float16>(p, q, s);
    if (rc <= 0) return rc;
  }
  if (a.Hq > 0 && a.q != nullptr) {
    const QkNormRopeArgs q{a.q, nullptr, a.q_out, nullptr, a.q_stride, 0, a.q_out_stride, 0, a.M, a.Hq, 0, a.D, a.rope, a.act, a.stream};
    if (launch_qk_norm_rope(q, vec, &a.seq) != 0) return -1;
  }
  return a.act == Act::BF16 ? launch_generic<__bf16>(p, s) : launch_generic<_Float16>(p, s);
}

}  // namespace fp4w
