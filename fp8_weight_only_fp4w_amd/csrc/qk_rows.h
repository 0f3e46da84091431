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

// A wave has 64 / LANES heads of one row, LANES = D / 16 lanes a head: those of
// `pass`.  (Several passes a wave, to look up position and angles once, are
// slower: 51 to 59 us against 48 for 8192 rows of 48 heads of 128, for want of
// waves.)
template <typename T, int LANES>
__device__ __forceinline__ void qk_row(const QkParams& p, int64_t m, int pass) {
  const int lane = threadIdx.x & 63, h = pass * (64 / LANES) + lane / LANES;
  int64_t position = 0;
  if (!row_position(p, m, &position) || h >= p.Hq + p.Hk) return;
  const LaneChunks at = lane_chunks(lane % LANES, 16 * LANES, p.rope.dims);
  const bool query = h < p.Hq;
  const int64_t head = static_cast<int64_t>(query ? h : h - p.Hq) * (16 * LANES);
  const T* x = static_cast<const T*>(query ? p.q : p.k) + m * (query ? p.q_stride : p.k_stride) + head;
  const T* weight = static_cast<const T*>(query ? p.q_weight : p.k_weight);
  LaneHead<T> v;
  v.load(x, at);
  LaneAngles angles;
  if (p.rope.cos) angles.load(p.rope, at, position);
  if (weight) v.template norm<LANES>(weight, at, p.rope);  // the same on every lane of a head
  if (p.rope.cos) v.rotate(angles, at, p.rope);
  v.store(static_cast<T*>(query ? p.q_out : p.k_out) + m * (query ? p.q_out_stride : p.k_out_stride) + head, at);
}

}  // namespace fp4w
