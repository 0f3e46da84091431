// Query and key heads of a call's rows, normed and rotated, by waves: the kernel
// of qk_norm_rope.hip, and the queries' part of kv_append.hip's.
#pragma once

#include "heads.h"

namespace fp4w {

struct QkParams {
  const void* q;
  const void* k;
  void* q_out;
  void* k_out;
  int64_t q_stride, k_stride, q_out_stride, k_out_stride, M;
  int32_t Hq, Hk, D;
  const void* q_weight;
  const void* k_weight;
  Rope rope;
  Seqs seq;        // seq.lens not null: positions from the sequences
};

// Position of row m, and whether the row is to be written.
__device__ __forceinline__ bool row_position(const QkParams& p, int64_t m, int64_t* position) {
  if (p.seq.lens != nullptr) {
    if (m >= seq_start(p.seq, p.seq.B)) return false;
    const int b = last_not_above(p.seq.B, m, [&](int i) { return seq_start(p.seq, i); });
    const SeqSpan s = seq_span(p.seq, b);
    *position = static_cast<int64_t>(s.len) - s.rows + (m - s.first_row);
  } else {
    *position = m;
  }
  if (p.rope.positions) *position = p.rope.positions[m];
  return true;
}

// A wave has one row's heads first, first + step, ... (in passes of 64 / LANES
// heads, AT_ONCE passes loaded together), LANES = D / 16 lanes a head.  The
// row's position and angles are looked up once.
template <typename T, int LANES, int AT_ONCE>
__device__ __forceinline__ void qk_row(const QkParams& p, int64_t m, int first, int step) {
  constexpr int PASS = 64 / LANES;
  const int lane = threadIdx.x & 63, t = lane % LANES, sub = lane / LANES, heads = p.Hq + p.Hk;
  int64_t position = 0;
  if (!row_position(p, m, &position)) return;
  const LaneChunks at = lane_chunks(t, 16 * LANES, p.rope.dims);
  LaneAngles angles;
  if (p.rope.cos) angles.load(p.rope, at, position);
  const T* q = static_cast<const T*>(p.q) + m * p.q_stride;
  const T* k = static_cast<const T*>(p.k) + m * p.k_stride;
  T* q_out = static_cast<T*>(p.q_out) + m * p.q_out_stride;
  T* k_out = static_cast<T*>(p.k_out) + m * p.k_out_stride;
  for (int pass = first; pass * PASS < heads; pass += step * AT_ONCE) {
    LaneHead<T> x[AT_ONCE];
#pragma unroll
    for (int i = 0; i < AT_ONCE; ++i) {
      const int h = (pass + i * step) * PASS + sub;
      if (h < heads) x[i].load(h < p.Hq ? q + h * (16 * LANES) : k + (h - p.Hq) * (16 * LANES), at);
    }
#pragma unroll
    for (int i = 0; i < AT_ONCE; ++i) {
      const int h = (pass + i * step) * PASS + sub;
      if (h < heads) {  // the same on every lane of a head
        const T* weight = static_cast<const T*>(h < p.Hq ? p.q_weight : p.k_weight);
        if (weight) x[i].template norm<LANES>(weight, at, p.rope);
        if (p.rope.cos) x[i].rotate(angles, at, p.rope);
        x[i].store(h < p.Hq ? q_out + h * (16 * LANES) : k_out + (h - p.Hq) * (16 * LANES), at);
      }
    }
  }
}

}  // namespace fp4w
