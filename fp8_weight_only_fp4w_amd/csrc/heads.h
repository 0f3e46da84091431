// Device helpers of the kernels between the projections of an attention block
// (qk_norm_rope.hip, kv_append.hip, attention*.hip): the sequences of a call,
// the page scales, and the norm and rotation of one head.
#pragma once

#include <math.h>

#include "device.h"
#include "launch.h"

namespace fp4w {

// ------------------------------------------------------------------ page scales

// E8M0: 2^(byte - 127), NaN for 255.
__device__ __forceinline__ float e8m0_to_f32(uint32_t b) {
  const uint32_t bits = b == 0 ? 0x00400000u : b == 255 ? 0x7fc00000u : b << 23;
  return __uint_as_float(bits);
}

// The byte of the smallest power of two 2^e >= 2^-126 with a <= 448 * 2^e, for
// a finite a >= 0: 448 is 1.75 * 2^8, so e is a's exponent less 8, plus one
// where a's significand is above 1.75.
__device__ __forceinline__ uint32_t e8m0_for(float a) {
  const uint32_t bits = __float_as_uint(a);
  const int b = static_cast<int>(bits >> 23) - 8 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0);
  return static_cast<uint32_t>(b < 1 ? 1 : b);
}

// 2^-(e) of a byte from 1 to 254, exact (254: 2^-127, a subnormal).
__device__ __forceinline__ float e8m0_inverse(uint32_t b) {
  return b == 254 ? __uint_as_float(0x00400000u) : __uint_as_float((254u - b) << 23);
}

// A page's scale times the call's may pass FP32, but times a key of 0 it has to
// be 0.  NaN stays.
__device__ __forceinline__ float finite_factor(float f) { return f > __FLT_MAX__ ? __FLT_MAX__ : f; }

// ------------------------------------------------------------------ sequences

// SeqArgs for the device, in 32 bits.  capacity: the tokens that a row of the
// page table has room for (0 without pages).
struct Seqs {
  const int32_t* starts;
  const int32_t* lens;
  const int32_t* table;
  int32_t B, M, num_pages, page, capacity, row0;  // row0: sequence 0's row where starts is null
  int64_t max_pages;
  FastDiv page_div;
};

inline Seqs make_seqs(const SeqArgs& s, int64_t M) {
  Seqs d;
  d.starts = s.starts;
  d.lens = s.lens;
  d.table = s.table;
  d.B = static_cast<int32_t>(s.B);
  d.M = static_cast<int32_t>(M);
  d.num_pages = static_cast<int32_t>(s.num_pages);
  d.page = static_cast<int32_t>(s.page_size);
  d.row0 = 0;
  d.capacity = s.num_pages > 0 ? static_cast<int32_t>(s.max_pages * s.page_size) : 0;
  d.max_pages = s.max_pages;
  d.page_div = make_fastdiv(static_cast<uint32_t>(s.page_size));
  return d;
}

// First row of sequence b (b = B: behind the last row), inside [0, M] whatever
// the array holds.
__device__ __forceinline__ int seq_start(const Seqs& s, int b) {
  if (s.starts == nullptr) return s.row0 + b;
  const int v = s.starts[b];
  return v < 0 ? 0 : v > s.M ? s.M : v;
}

// Tokens that sequence b holds, and how many rows of the call are its newest.
struct SeqSpan {
  int first_row, rows, len;  // the first row's position is len - rows
};

__device__ __forceinline__ SeqSpan seq_span(const Seqs& s, int b) {
  const int lo = seq_start(s, b), hi = seq_start(s, b + 1), n = s.lens[b];
  return SeqSpan{lo, hi > lo ? hi - lo : 0, n < 0 ? 0 : n};
}

// Page of token t of sequence b, or -1 where it has none.
__device__ __forceinline__ int page_of(const Seqs& s, int b, int t) {
  if (t < 0 || t >= s.capacity) return -1;
  const int id = s.table[b * s.max_pages + fdiv(static_cast<uint32_t>(t), s.page_div)];
  return id >= 0 && id < s.num_pages ? id : -1;
}

// The same for t >= 0 where there are pages, without a branch: a load under one
// makes the compiler wait for every load in flight where it waits for an older
// one.  *slot: t % page.
__device__ __forceinline__ int page_ahead(const Seqs& s, const int32_t* row, int t, bool wanted, uint32_t* slot) {
  const bool inside = wanted && t < s.capacity;
  const uint32_t at = vgpr(inside ? static_cast<uint32_t>(t) : 0u), index = fdiv(at, s.page_div);
  *slot = at - index * static_cast<uint32_t>(s.page);
  const int id = row[index];
  return inside && id >= 0 && id < s.num_pages ? id : -1;
}

// The largest b in [0, B) with at(b) <= u, for a function that does not fall
// and at(0) <= u; every lane of the wave calls it with the same u.  64 probes
// at a time: two rounds of loads up to B = 4096.
template <typename F>
__device__ __forceinline__ int last_not_above(int B, int64_t u, F&& at) {
  int lo = 0, n = B;
  const int lane = threadIdx.x & 63;
  while (n > 1) {
    const int step = (n + 63) >> 6, i = lane * step;
    const bool ok = i < n && at(lo + (i < n ? i : 0)) <= u;
    const uint64_t hit = __ballot(ok);
    const int last = hit == 0 ? 0 : 63 - __builtin_clzll(hit);
    lo += last * step;
    n = step < n - last * step ? step : n - last * step;
  }
  return lo;
}

// ------------------------------------------------------------------ far queries
//
// Scores are summed over codes of up to 448, and take the page's scale behind the
// sum.  A row with a query of kFar or more (BF16 reaches 2^128) is held times
// 2^-24 for the products, which then stay below 2^104 * 448 * 1024, and its scores
// are scaled up again.
constexpr float kFar = 0x1p104f, kFarUp = 0x1p24f, kFarDown = 0x1p-24f;

// Nonzero if one of a pair of BF16 values is kFar or more (or no number).
__device__ __forceinline__ uint32_t far_pair(uint32_t w) {
  return ((w & 0x7fff7fffu) + 0x0c800c80u) & 0x80008000u;  // 0x7380 is 2^104
}
__device__ __forceinline__ uint32_t down_pair(uint32_t w) {
  const uint32_t lo = __float_as_uint(__uint_as_float(w << 16) * kFarDown), hi = __float_as_uint(__uint_as_float(w & 0xffff0000u) * kFarDown);
  return (hi & 0xffff0000u) | lo >> 16;
}

// ------------------------------------------------------------------ norm and rotation

struct Rope {
  const float* cos;  // null: no rotation
  const float* sin;
  const int32_t* positions;
  int64_t rows;
  int32_t dims;
  bool interleaved;
  float offset, eps;
};

inline Rope make_rope(const RopeArgs& r) {
  return Rope{r.cos, r.sin, r.positions, r.rows, r.cos ? static_cast<int32_t>(r.dims) : 0, r.interleaved, r.weight_offset, r.eps};
}

__device__ __forceinline__ float wave_sum64(float v) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off, 64);
  return v;
}

// One head of any size by one wave: normed (weight not null) and rotated for
// `position`, in FP32, into buf[0 .. D).  x[D] is read before the barriers
// below, so a caller may write over it behind the call.  Every wave of the
// workgroup calls it the same number of times (x null: nothing to do).
template <typename T>
__device__ __forceinline__ void head_to_lds(const T* x, int D, const T* weight, const Rope& r, int64_t position, float* buf) {
  const int lane = threadIdx.x & 63;
  if (x) {
    float sum = 0.0f;
    for (int d = lane; d < D; d += 64) {
      const float v = static_cast<float>(x[d]);
      buf[d] = v;
      sum = fmaf(v, v, sum);
    }
    if (weight) {
      const float inv = 1.0f / sqrtf(wave_sum64(sum) / static_cast<float>(D) + r.eps);
      for (int d = lane; d < D; d += 64) buf[d] *= inv * (r.offset + static_cast<float>(weight[d]));
    }
  }
  __syncthreads();
  if (x && r.cos) {
    const int half = r.dims >> 1;
    const bool known = position >= 0 && position < r.rows;
    const float* c = r.cos + (known ? position : 0) * half;
    const float* s = r.sin + (known ? position : 0) * half;
    for (int i = lane; i < half; i += 64) {  // a pair is read and written by one lane
      const int ia = r.interleaved ? 2 * i : i, ib = r.interleaved ? 2 * i + 1 : i + half;
      const float a = buf[ia], b = buf[ib];
      buf[ia] = known ? fmaf(a, c[i], -(b * s[i])) : NAN;
      buf[ib] = known ? fmaf(b, c[i], a * s[i]) : NAN;
    }
  }
  __syncthreads();
}

// A head by D / 16 lanes (a power of two up to 64), 16 values a lane: two chunks
// of 8, chosen so that both values of a pair are in one lane.  Lane t < dims / 16
// has the rotated chunks t and t + dims / 16, the others two that are not rotated.
struct LaneChunks {
  int a, b;
  bool rotated;
};

__device__ __forceinline__ LaneChunks lane_chunks(int t, int D, int dims) {
  const int half = dims >> 4;
  if (t < half) return LaneChunks{t, t + half, true};
  const int u = (dims >> 3) + t - half;
  return LaneChunks{u, u + ((D - dims) >> 4), false};
}

// cos and sin of a lane's eight pairs at a position (NaN for an unknown one).
struct LaneAngles {
  float c[8], s[8];
  __device__ __forceinline__ void load(const Rope& r, const LaneChunks& at, int64_t position) {
    if (!at.rotated) return;
    const bool known = position >= 0 && position < r.rows;
    const int64_t row = (known ? position : 0) * (r.dims >> 1);
    const int first = r.interleaved ? 4 * at.a : 8 * at.a, second = r.interleaved ? 4 * at.b : first + 4;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const f32x4 cv = *reinterpret_cast<const f32x4*>(r.cos + row + (i ? second : first));
      const f32x4 sv = *reinterpret_cast<const f32x4*>(r.sin + row + (i ? second : first));
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        c[4 * i + j] = known ? cv[j] : NAN;
        s[4 * i + j] = known ? sv[j] : NAN;
      }
    }
  }
};

__device__ __forceinline__ void turn(float& a, float& b, float c, float s) {
  const float x = fmaf(a, c, -(b * s));
  b = fmaf(b, c, a * s);
  a = x;
}

template <typename T>
struct LaneHead {
  float v[16];
  __device__ __forceinline__ void load(const T* x, const LaneChunks& at) {
    typedef typename ActTraits<T>::vec8 vec8;
    const vec8 a = *reinterpret_cast<const vec8*>(x + 8 * at.a), b = *reinterpret_cast<const vec8*>(x + 8 * at.b);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v[i] = static_cast<float>(a[i]);
      v[8 + i] = static_cast<float>(b[i]);
    }
  }
  // every lane of the head's calls it
  template <int LANES>
  __device__ __forceinline__ void norm(const T* weight, const LaneChunks& at, const Rope& r) {
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) sum = fmaf(v[i], v[i], sum);
#pragma unroll
    for (int off = LANES / 2; off > 0; off >>= 1) sum += __shfl_xor(sum, off, 64);
    const float inv = 1.0f / sqrtf(sum / static_cast<float>(16 * LANES) + r.eps);
    LaneHead<T> w;
    w.load(weight, at);
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] *= inv * (r.offset + w.v[i]);
  }
  __device__ __forceinline__ void rotate(const LaneAngles& g, const LaneChunks& at, const Rope& r) {
    if (!at.rotated) return;
    if (r.interleaved) {
#pragma unroll
      for (int i = 0; i < 8; ++i) turn(v[2 * i], v[2 * i + 1], g.c[i], g.s[i]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) turn(v[i], v[8 + i], g.c[i], g.s[i]);
    }
  }
  __device__ __forceinline__ void store(T* y, const LaneChunks& at) const {
    typedef typename ActTraits<T>::vec8 vec8;
    vec8 a, b;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      a[i] = round_to<T>(v[i]);
      b[i] = round_to<T>(v[8 + i]);
    }
    *reinterpret_cast<vec8*>(y + 8 * at.a) = a;
    *reinterpret_cast<vec8*>(y + 8 * at.b) = b;
  }
};

// Two values as E4M3 codes in the low 16 bits, to nearest even; an infinity or
// NaN becomes the NaN code.  Finite values are within +-448.
__device__ __forceinline__ uint32_t e4m3_pair(float a, float b) {
  const uint32_t c = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false) & 0xffffu;
  const uint32_t na = fabsf(a) < INFINITY ? c & 0xffu : 0x7fu, nb = fabsf(b) < INFINITY ? c & 0xff00u : 0x7f00u;
  return na | nb;
}

// Four codes times a power of two of 1 or less.
__device__ __forceinline__ uint32_t scale_codes(uint32_t w, float down) {
  const f32x2 a = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(w), false), b = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(w), true);
  return e4m3_pair(a.x * down, a.y * down) | e4m3_pair(b.x * down, b.y * down) << 16;
}

__device__ __forceinline__ float finite_abs(float x) {
  const float a = fabsf(x);
  return a < INFINITY ? a : 0.0f;
}

}  // namespace fp4w
