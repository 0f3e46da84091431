// Norms of query and key heads with the rotation by position, in one pass:
//
//   n[d] = x[d]                                               without a weight
//        = x[d] * rsqrt(mean(x^2) + eps) * (offset + w[d])    with one
//   (n[i], n[j]) -> (n[i] c - n[j] s, n[j] c + n[i] s)        for the pairs of the first `dims` values
//
// in FP32, rounded once.  Every head is read and written once, so the memory is
// the bound: 8192 rows of 48 heads of 128 in BF16 take 42 to 46 us, 4.5 to 4.9
// TB/s, where a large copy reaches 5.1.  One row takes 3 us: a launch, and a
// chain of position, angles and values.

#include <hip/hip_runtime.h>

#include "qk_rows.h"

namespace fp4w {
namespace {

// Any D, alignment and stride: a wave per head, values through LDS.
template <typename T>
__global__ __launch_bounds__(256) void qk_norm_rope_generic_kernel(const QkParams p) {
  __shared__ float buf[4][kMaxHead];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, heads = p.Hq + p.Hk;
  const int64_t units = p.M * heads;
  for (int64_t base = static_cast<int64_t>(blockIdx.x) * 4; base < units; base += static_cast<int64_t>(gridDim.x) * 4) {
    const int64_t u = base + wave;
    const T* x = nullptr;
    T* y = nullptr;
    const T* w = nullptr;
    int64_t position = 0;
    if (u < units) {
      const int64_t m = u / heads;
      const int h = static_cast<int>(u - m * heads);
      if (row_position(p, m, &position)) {
        if (h < p.Hq) {
          x = static_cast<const T*>(p.q) + m * p.q_stride + static_cast<int64_t>(h) * p.D;
          y = static_cast<T*>(p.q_out) + m * p.q_out_stride + static_cast<int64_t>(h) * p.D;
          w = static_cast<const T*>(p.q_weight);
        } else {
          x = static_cast<const T*>(p.k) + m * p.k_stride + static_cast<int64_t>(h - p.Hq) * p.D;
          y = static_cast<T*>(p.k_out) + m * p.k_out_stride + static_cast<int64_t>(h - p.Hq) * p.D;
          w = static_cast<const T*>(p.k_weight);
        }
      }
    }
    head_to_lds(x, p.D, w, p.rope, position, buf[wave]);
    if (x)
      for (int d = lane; d < p.D; d += 64) y[d] = round_to<T>(buf[wave][d]);
    __syncthreads();
  }
}

// D a power of two from 16 to 1024, everything in 16-byte pieces: `passes` waves
// for a row.
template <typename T, int LANES>
__global__ __launch_bounds__(256) void qk_norm_rope_kernel(const QkParams p, int passes, FastDiv by_passes) {
  const int64_t waves = p.M * passes;
  for (int64_t u = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 6); u < waves; u += static_cast<int64_t>(gridDim.x) * 4) {
    const int64_t m = waves <= 0x7fffffff ? fdiv(static_cast<uint32_t>(u), by_passes) : u / passes;
    qk_row<T, LANES>(p, m, static_cast<int>(u - m * passes));
  }
}

template <typename T, int LANES>
int launch_lanes(const QkParams& p, hipStream_t s) {
  const int passes = (p.Hq + p.Hk + 64 / LANES - 1) / (64 / LANES);
  const int64_t blocks = (p.M * passes + 3) / 4;
  const dim3 grid(static_cast<uint32_t>(blocks < (1 << 20) ? blocks : 1 << 20));
  hipLaunchKernelGGL((qk_norm_rope_kernel<T, LANES>), grid, dim3(256), 0, s, p, passes, make_fastdiv(passes));
  return hipGetLastError() == hipSuccess ? 0 : -1;
}

template <typename T>
int launch_t(const QkParams& p, bool vec, hipStream_t s) {
  if (vec) {
    switch (p.D) {
      case 16: return launch_lanes<T, 1>(p, s);
      case 32: return launch_lanes<T, 2>(p, s);
      case 64: return launch_lanes<T, 4>(p, s);
      case 128: return launch_lanes<T, 8>(p, s);
      case 256: return launch_lanes<T, 16>(p, s);
      case 512: return launch_lanes<T, 32>(p, s);
      case 1024: return launch_lanes<T, 64>(p, s);
    }
  }
  const int64_t blocks = (p.M * (p.Hq + p.Hk) + 3) / 4;
  const int grid = static_cast<int>(blocks < (1 << 20) ? blocks : 1 << 20);
  hipLaunchKernelGGL(qk_norm_rope_generic_kernel<T>, dim3(grid), dim3(256), 0, s, p);
  return hipGetLastError() == hipSuccess ? 0 : -1;
}

}  // namespace

int launch_qk_norm_rope(const QkNormRopeArgs& a, bool vec, const SeqArgs* seq) {
  QkParams p{a.q, a.k, a.q_out, a.k_out, a.q_stride, a.k_stride, a.q_out_stride, a.k_out_stride, a.M,
             static_cast<int32_t>(a.Hq), static_cast<int32_t>(a.Hk), static_cast<int32_t>(a.D),
             a.rope.q_weight, a.rope.k_weight, make_rope(a.rope), Seqs{}};
  if (seq) p.seq = make_seqs(*seq, a.M);
  hipStream_t s = static_cast<hipStream_t>(a.stream);
  return a.act == Act::BF16 ? launch_t<__bf16>(p, vec, s) : launch_t<_Float16>(p, vec, s);
}

}  // namespace fp4w
