// Mixture-of-experts layer for every legal shape (odd sizes, any block size,
// unaligned pointers, empty sums).  Not tuned: the shapes that matter take
// the streaming kernels.
//
//   H[a, i] = act(A[m] . W13[e][i]) * (A[m] . W13[e][I + i])       a = m * topk + j, e = ids[a]
//   Y[m, n] = RNE_T( sum_j weights[a] * (H[a] . W2[e][n]) )
// with W = e2m1 * e4m3 * g[e] (FP4) or e4m3 * scale (FP8).  H is FP32 in the
// workspace.  One wave per output value of each step; lanes stride over the
// sum and the partial sums meet in a wave reduction.  Assignments whose id is
// outside [0, E) contribute nothing, and their H is not written.

#include <hip/hip_runtime.h>

#include "device.h"
#include "launch.h"
#include "moe_act.h"

namespace fp4w {
namespace {

constexpr int kGenWaves = 4;

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off, 64);
  return v;
}

// x[k] . row[k] over this lane's k, the block scale applied to each weight
// (E2M1 x E4M3 is exact; the FP8 product with its FP32 scale rounds once)
template <bool FP4, typename X>
__device__ __forceinline__ float lane_dot(const X* x, const uint8_t* w, const void* scale, int64_t len, int64_t bs,
                                          int lane) {
  float acc = 0.0f;
  for (int64_t k = lane; k < len; k += 64) {
    float v;
    if constexpr (FP4) {
      const f32x2 q = e2m1x2_to_f32<0>(w[k >> 1]);
      v = ((k & 1) ? q.y : q.x) * e4m3_to_f32<0>(static_cast<const uint8_t*>(scale)[k / bs]);
    } else {
      v = e4m3_to_f32<0>(w[k]) * static_cast<const float*>(scale)[k / bs];
    }
    acc = fmaf(static_cast<float>(x[k]), v, acc);
  }
  return acc;
}

template <typename T, bool FP4>
__global__ __launch_bounds__(64 * kGenWaves) void moe_up_generic_kernel(
    const T* __restrict__ A, const int32_t* __restrict__ ids, const uint8_t* __restrict__ w13,
    const uint8_t* __restrict__ s13, const float* __restrict__ g13, float* __restrict__ H, int64_t n, int64_t K,
    int64_t topk, int64_t E, int64_t I, int64_t bs, int act) {
  const int lane = threadIdx.x & 63;
  const int64_t cols = (K + bs - 1) / bs;
  const int64_t wrow = FP4 ? K / 2 : K, srow = FP4 ? cols : 4 * cols;
  const int64_t step = static_cast<int64_t>(gridDim.x) * kGenWaves;
  for (int64_t u = static_cast<int64_t>(blockIdx.x) * kGenWaves + (threadIdx.x >> 6); u < n * I; u += step) {
    const int64_t a = u / I, i = u - a * I;
    const int64_t e = ids[a];
    if (e < 0 || e >= E) continue;
    const T* x = A + a / topk * K;
    const int64_t r0 = e * 2 * I + i, r1 = r0 + I;
    float gate = wave_sum(lane_dot<FP4>(x, w13 + r0 * wrow, s13 + r0 * srow, K, bs, lane));
    float up = wave_sum(lane_dot<FP4>(x, w13 + r1 * wrow, s13 + r1 * srow, K, bs, lane));
    if (FP4) {
      const float g = g13[e];
      gate *= g;
      up *= g;
    }
    if (lane == 0) H[u] = gated(act, gate, up);
  }
}

template <typename T, bool FP4>
__global__ __launch_bounds__(64 * kGenWaves) void moe_down_generic_kernel(
    const float* __restrict__ H, const int32_t* __restrict__ ids, const float* __restrict__ weights,
    const uint8_t* __restrict__ w2, const uint8_t* __restrict__ s2, const float* __restrict__ g2, T* __restrict__ Y,
    int64_t M, int64_t K, int64_t topk, int64_t E, int64_t I, int64_t bs) {
  const int lane = threadIdx.x & 63;
  const int64_t cols = (I + bs - 1) / bs;
  const int64_t wrow = FP4 ? I / 2 : I, srow = FP4 ? cols : 4 * cols;
  const int64_t step = static_cast<int64_t>(gridDim.x) * kGenWaves;
  for (int64_t u = static_cast<int64_t>(blockIdx.x) * kGenWaves + (threadIdx.x >> 6); u < M * K; u += step) {
    const int64_t m = u / K, c = u - m * K;
    float sum = 0.0f;
    for (int64_t j = 0; j < topk; ++j) {
      const int64_t a = m * topk + j, e = ids[a];
      if (e < 0 || e >= E) continue;
      const int64_t r = e * K + c;
      const float d = wave_sum(lane_dot<FP4>(H + a * I, w2 + r * wrow, s2 + r * srow, I, bs, lane));
      sum = fmaf(FP4 ? d * g2[e] : d, weights[a], sum);
    }
    if (lane == 0) Y[u] = round_to<T>(sum);
  }
}

int grid_for(int64_t units) {
  const int64_t g = (units + kGenWaves - 1) / kGenWaves, cap = 256 * 64;
  return static_cast<int>(g < cap ? g : cap);
}

template <typename T, bool FP4>
int launch_t(const MoeArgs& a) {
  hipStream_t s = static_cast<hipStream_t>(a.stream);
  const int64_t n = a.M * a.topk;
  float* H = static_cast<float*>(a.work);
  if (n > 0 && a.I > 0 && a.E > 0)
    hipLaunchKernelGGL((moe_up_generic_kernel<T, FP4>), dim3(grid_for(n * a.I)), dim3(64 * kGenWaves), 0, s,
                       static_cast<const T*>(a.A), a.ids, a.w13, static_cast<const uint8_t*>(a.s13), a.g13, H, n,
                       a.K, a.topk, a.E, a.I, a.block_size, a.activation);
  // with no expert or an empty sum Y is zero: the kernel's loops find nothing
  const int64_t E = a.I > 0 ? a.E : 0;
  hipLaunchKernelGGL((moe_down_generic_kernel<T, FP4>), dim3(grid_for(a.M * a.K)), dim3(64 * kGenWaves), 0, s, H,
                     a.ids, a.weights, a.w2, static_cast<const uint8_t*>(a.s2), a.g2, static_cast<T*>(a.Y), a.M, a.K,
                     a.topk, E, a.I, a.block_size);
  return hipGetLastError() == hipSuccess ? 0 : -1;
}

}  // namespace

int launch_moe_fp4_generic(const MoeArgs& a) {
  return a.act == Act::BF16 ? launch_t<__bf16, true>(a) : launch_t<_Float16, true>(a);
}
int launch_moe_fp8_generic(const MoeArgs& a) {
  return a.act == Act::BF16 ? launch_t<__bf16, false>(a) : launch_t<_Float16, false>(a);
}

}  // namespace fp4w
