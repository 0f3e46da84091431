// What the attention kernels share (attention.hip, attention_prompt.hip): their
// arguments, the types' traits, the join of partial results and the outputs.
#pragma once

#include "heads.h"

namespace fp4w {

constexpr int kTile = 64;  // keys

struct AttnParams {
  const void* q;
  int64_t q_stride;
  int32_t Hq, Hk, G, max_new;
  Seqs seq;
  const uint8_t* k_cache;
  const uint8_t* k_scale;
  const uint8_t* v_cache;
  const uint8_t* v_scale;
  float c;          // |scale| * log2(e)
  uint32_t flip;    // sign bits of a pair of T where scale < 0
  bool causal;
  int32_t window;   // 0: none
  void* Y;
  float* lse;
};

inline AttnParams make_attn(const AttentionArgs& a) {
  AttnParams p;
  p.q = a.q;
  p.q_stride = a.q_stride;
  p.Hq = static_cast<int32_t>(a.Hq);
  p.Hk = static_cast<int32_t>(a.Hk);
  p.G = static_cast<int32_t>(a.Hq / a.Hk);
  p.max_new = static_cast<int32_t>(a.max_new);
  p.seq = make_seqs(a.seq, a.M);
  p.k_cache = a.k_cache;
  p.k_scale = a.k_scale;
  p.v_cache = a.v_cache;
  p.v_scale = a.v_scale;
  p.c = fabsf(a.scale) * 1.44269504088896341f;
  p.flip = a.scale < 0.0f ? 0x80008000u : 0u;
  p.causal = a.causal;
  p.window = static_cast<int32_t>(a.window < 0x7fffffff ? a.window : 0);  // no sequence is longer
  p.Y = a.Y;
  p.lse = a.lse;
  return p;
}

typedef float f32x16 __attribute__((ext_vector_type(16)));

// What differs by the type: P's range and V's exponent.  Numerators are rounded to T
// between the products, as the matrix instructions take both operands in T (at a
// sixteenth of the rate in FP32); their sum is taken before.  With the output's own
// rounding the error against 64 bits, relative and RMS, is 1.9 to 2.1e-3 in BF16 and
// 2.3 to 2.9e-4 in FP16; of the output's rounding alone 1.6 to 1.7e-3 and 2.0 to 2.1e-4.
template <typename T>
struct AttnTraits;
template <>
struct AttnTraits<__bf16> {
  static constexpr float kLift = 0.0f;      // numerators are 2^(s - m + kLift)
  static constexpr float kLag = 8.0f;       // and m may be smaller than the largest s so far by kLag
  // V is held times 2^-kDown.  BF16 values reach FP32's end, and numerators of up to
  // 2^kLag, or a sum over many tokens, would pass it where their average does not.
  // Of that, values below 2^-102 lose bits (down to steps of 2^-109).
  static constexpr uint32_t kDown = 24;
  static constexpr bool kFarQueries = true;
  static constexpr uint32_t kLeastV = 25, kMostV = 254;  // the scales under which T holds every value so
  __device__ __forceinline__ static bf16x2 cvt(uint32_t w, float s, bool hi) {
    return hi ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, s, true) : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, s, false);
  }
};
template <>
struct AttnTraits<_Float16> {
  // FP16 ends at 2^-14: numerators down to 2^-22 keep all their bits so, and
  // the largest value that FP16 data leads to, 2^16, stays finite at half of it
  static constexpr float kLift = 8.0f;
  static constexpr float kLag = 6.0f;
  static constexpr uint32_t kDown = 1;
  static constexpr bool kFarQueries = false;  // 65504 * 448 * 128 is far from FP32's end
  static constexpr uint32_t kLeastV = 0, kMostV = 135;
  __device__ __forceinline__ static f16x2 cvt(uint32_t w, float s, bool hi) {
    return hi ? __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, s, true) : __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, s, false);
  }
};

template <typename T>
__device__ __forceinline__ typename ActTraits<T>::vec8 decode8_power(uint32_t lo, uint32_t hi, float s) {
  const auto a = AttnTraits<T>::cvt(lo, s, false), b = AttnTraits<T>::cvt(lo, s, true);
  const auto c = AttnTraits<T>::cvt(hi, s, false), d = AttnTraits<T>::cvt(hi, s, true);
  typename ActTraits<T>::vec8 r;
  r[0] = a[0]; r[1] = a[1]; r[2] = b[0]; r[3] = b[1];
  r[4] = c[0]; r[5] = c[1]; r[6] = d[0]; r[7] = d[1];
  return r;
}

// Whether T holds every value under scale byte `scale`.
template <typename T>
__device__ __forceinline__ bool held_scale(uint32_t scale) {
  return scale - AttnTraits<T>::kLeastV <= AttnTraits<T>::kMostV - AttnTraits<T>::kLeastV;
}
// Codes of V under a scale byte: those that mean the same under kLeastV where it is
// below that, and the NaN code for what T does not hold.  Under kMostV + x that is
// a code of (16 - x) * 8 or more (for FP16, which holds halves, a value of 2^17),
// from x = 16 on any but 0, and all where the scale is no number.
template <typename T>
__device__ __forceinline__ uint32_t codes_held(uint32_t w, uint32_t scale) {
  constexpr uint32_t kLeast = AttnTraits<T>::kLeastV, kMost = AttnTraits<T>::kMostV;
  if constexpr (kLeast > 0) w = scale_codes(w, __uint_as_float((127 - (scale < kLeast ? kLeast - scale : 0)) << 23));
  const uint32_t x = scale - kMost, step = scale <= kMost ? 0u : scale == 255 ? 0x80808080u : x < 16 ? x * 0x08080808u : 0x7f7f7f7fu;
  return w | ((((w & 0x7f7f7f7fu) + step) & 0x80808080u) >> 7) * 0x7fu;
}
// A page of zeros has the smallest scale: N words of codes that are all 0 go with any.
template <typename T, int N>
__device__ __forceinline__ uint32_t scale_of_zeros(const u32x4 (&v)[N], uint32_t scale) {
  u32x4 any = {0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < N; ++i) any |= v[i];
  return scale < AttnTraits<T>::kLeastV && (((any.x | any.y) | (any.z | any.w)) & 0x7f7f7f7fu) == 0 ? 127 : scale;
}
// The scale that goes with them.
template <typename T>
__device__ __forceinline__ uint32_t scale_held(uint32_t scale) {
  return scale == 255 ? 127 : scale < AttnTraits<T>::kLeastV ? AttnTraits<T>::kLeastV : scale;
}

// 0x80 in each byte of w that is a NaN code.
__device__ __forceinline__ uint32_t nan_codes(uint32_t w) { return ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u; }

// 0xff in the bytes j of a word with lo <= j < hi.
__device__ __forceinline__ uint32_t byte_mask(int lo, int hi) {
  lo = lo < 0 ? 0 : lo > 4 ? 4 : lo;
  hi = hi < 0 ? 0 : hi > 4 ? 4 : hi;
  const uint32_t below_hi = hi == 4 ? 0xffffffffu : (1u << (8 * hi)) - 1, below_lo = lo == 4 ? 0xffffffffu : (1u << (8 * lo)) - 1;
  return below_hi & ~below_lo;
}

// A row's maximum is -inf until it attends a token, and kLowest at least from then
// on.  A row whose every score is -inf has a sum of 0 like one without a token, but
// it is 0 / 0, and only the maximum tells them apart.
constexpr float kLowest = -__FLT_MAX__;

// (m, l, o) and (m2, l2, o2): maximum, sum and output of two sets of tokens.
__device__ __forceinline__ void join(float& m, float& l, f32x4& o, float m2, float l2, f32x4 o2) {
  const float now = fmaxf(m, m2), base = now > -INFINITY ? now : 0.0f;
  const float a = __builtin_amdgcn_exp2f(m - base), c = __builtin_amdgcn_exp2f(m2 - base);
  m = now;
  l = l * a + l2 * c;
  o = o * a + o2 * c;
}

// Four values of a row's output; no token attended: zeros.
template <typename T>
__device__ __forceinline__ void store_quad(const AttnParams& p, int64_t at_row, int D, int d, float m, float l, f32x4 o) {
  typedef T t4 __attribute__((ext_vector_type(4)));
  const bool none = l == 0.0f && m < kLowest;
  const float inv = static_cast<float>(1 << AttnTraits<T>::kDown) / l;
  t4 y;
#pragma unroll
  for (int j = 0; j < 4; ++j) y[j] = round_to<T>(none ? 0.0f : o[j] * inv);  // (0 x inf where all scores are -inf)
  *reinterpret_cast<t4*>(static_cast<T*>(p.Y) + at_row * D + d) = y;
}

template <typename T>
__device__ __forceinline__ void store_lse(const AttnParams& p, int64_t at_row, float m, float l) {
  constexpr float kLn2 = 0.693147180559945309f;
  if (p.lse) p.lse[at_row] = !(l == 0.0f) ? (m + log2f(l) - AttnTraits<T>::kLift) * kLn2 : m < kLowest ? -INFINITY : NAN;
}

}  // namespace fp4w
