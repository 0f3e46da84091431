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

#include <hip/hip_runtime.h>

#include "heads.h"

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
inline int64_t most_units(const Seqs& s) { return s.M / s.page + 2 * static_cast<int64_t>(s.B); }

// One page's share of a sequence's new tokens: slots [lo, hi) of page `id`
// are rows row .. of the call, at positions position ..; id -1: nothing to do.
struct Run {
  int id, lo, hi, row, position;
};

__device__ __forceinline__ Run run_of(const Seqs& s, int64_t unit) {
  const int b = last_not_above(s.B, unit, [&](int i) { return first_unit(s, i); });
  const SeqSpan q = seq_span(s, b);
  Run r{-1, 0, 0, 0, 0};
  int first = q.len - q.rows, row = q.first_row;
  if (first < 0) {  // more new rows than tokens: the rows before the first token are absent
    row -= first;
    first = 0;
  }
  const int64_t nth = unit - first_unit(s, b);  // below 0 only where starts falls
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
      for (int i = tid; i < r.lo * D; i += 256) {
        const int t = value ? i % r.lo : i / D, d = value ? i / r.lo : i - t * D;
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

template <typename T>
int launch_t(const AppendParams& p, bool vec, hipStream_t s) {
  const int64_t units = most_units(p.seq), work = units * p.Hk * 2;
  const int grid = static_cast<int>(work < (1 << 20) ? work : 1 << 20);
  if (grid > 0) hipLaunchKernelGGL(kv_append_generic_kernel<T>, dim3(grid), dim3(256), 0, s, p, units);
  return hipGetLastError() == hipSuccess ? 0 : -1;
}

}  // namespace

int launch_kv_append(const KvAppendArgs& a, bool vec) {
  if (a.Hq > 0 && a.q != nullptr) {
    QkNormRopeArgs q{a.q, nullptr, a.q_out, nullptr, a.q_stride, 0, a.q_out_stride, 0, a.M, a.Hq, 0, a.D, a.rope, a.act, a.stream};
    if (launch_qk_norm_rope(q, vec, &a.seq) != 0) return -1;
  }
  const AppendParams p{a.k, a.v, a.k_stride, a.v_stride, static_cast<int32_t>(a.Hk), static_cast<int32_t>(a.D), a.rope.k_weight,
                       make_rope(a.rope), make_seqs(a.seq, a.M), a.k_cache, a.k_scale, a.v_cache, a.v_scale};
  hipStream_t s = static_cast<hipStream_t>(a.stream);
  return a.act == Act::BF16 ? launch_t<__bf16>(p, vec, s) : launch_t<_Float16>(p, vec, s);
}

}  // namespace fp4w
