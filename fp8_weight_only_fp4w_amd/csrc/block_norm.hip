// Norms after and before a block, with the block's gate and the residual
// scale, in one pass over a row of K values:
//
//   b[k] = x[k]                                                  without a post norm
//        = x[k] * rsqrt(mean(x^2) + eps) * (offset + post[k])    with one
//   r[k] = residual[k] + scale * gate[k] * b[k]
//   y[k] = r[k] * rsqrt(mean(r^2) + eps) * (offset + pre[k])
//
// r is kept in FP32 between the two: y is rounded once, from the unrounded r,
// and so is residual_out.  Sums of squares are FP32.
//
// Memory-bound elementwise work with up to two dependent sums over the row.
// The row lives in registers, so every input is read and every output written
// once; a workgroup owns one row (one wave owns it where a wave's 64 lanes
// hold it), and a sum is a wave reduction, one LDS exchange and one barrier.
// Every value of a row is read before any is written, so the outputs may take
// the place of x and residual.  Rows that the registers of a workgroup do not
// hold take a kernel that reads the row once per sum and once for the result:
// those of more than 32768 values, and of more than 4096 where rows are not
// whole aligned chunks of 8.  With 16 single values a thread (of 1024, so 128
// registers) the compiler keeps 624 bytes a lane in scratch: 4096 rows of 8193
// took 852 us that way and take 229 so, one row 30 and 12.  Four chunks a thread,
// 16385 to 32768 values, spill too (152 bytes a lane), but 1024 rows of 24576 take
// 75 us, and 181 in the other kernel; one row 11 and 28.
// Measured: 8192 rows of 5120 with a residual and a norm before the next block
// (336 MB) take 64.5 us, 5.2 TB/s, above the 4.8 that a large copy reaches.
// 77 rows of 2049 with both norms and a full gate take 5.6 us, one row of 5120
// 3.3: a launch and two dependent sums.

#include <hip/hip_runtime.h>

#include "device.h"
#include "launch.h"

namespace fp4w {
namespace {

struct NormParams {
  const void* x;
  const void* post;
  const void* gate;
  const void* residual;
  const void* pre;
  void* r_out;
  void* y;
  int64_t M, K, gate_pitch;  // gate_pitch: 0 (one row for all) or K
  float scale, offset, eps;
};

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off, 64);
  return v;
}

// Sum over the workgroup's waves (all of them call it), the same bits on
// every lane.  `red`: 2 x 16 floats used in turn, so that one barrier per sum
// is enough: a wave writes a buffer again only after a barrier that every
// wave reaches after it has read that buffer.
__device__ __forceinline__ float block_sum(float v, float* red, int waves, int& turn) {
  v = wave_sum(v);
  if (waves == 1) return v;
  float* buf = red + 16 * turn;
  turn ^= 1;
  if ((threadIdx.x & 63) == 0) buf[threadIdx.x >> 6] = v;
  __syncthreads();
  const int lane = threadIdx.x & 15;
  v = lane < waves ? buf[lane] : 0.0f;
#pragma unroll
  for (int off = 8; off > 0; off >>= 1) v += __shfl_xor(v, off, 64);
  return v;
}

// VEC consecutive values of T as floats, and back (rounded once).
template <typename T, int VEC>
struct Chunk {
  float v[VEC];
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (VEC == 8) {
      const typename ActTraits<T>::vec8 t = *reinterpret_cast<const typename ActTraits<T>::vec8*>(p);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = static_cast<float>(t[i]);
    } else {
      v[0] = static_cast<float>(*p);
    }
  }
  __device__ __forceinline__ void store(T* p) const {
    if constexpr (VEC == 8) {
      typename ActTraits<T>::vec8 t;
#pragma unroll
      for (int i = 0; i < 8; ++i) t[i] = static_cast<T>(v[i]);
      *reinterpret_cast<typename ActTraits<T>::vec8*>(p) = t;
    } else {
      *p = static_cast<T>(v[0]);
    }
  }
};

// WAVE_ROW: a wave per row (4 rows per workgroup), otherwise a workgroup.
// Chunk j of a thread is chunk tid + j * threads of the row.
template <typename T, int VEC, int ITEMS, bool WAVE_ROW>
__global__ __launch_bounds__(WAVE_ROW ? 256 : 1024) void block_norm_kernel(const NormParams p) {
  __shared__ float red[32];
  const int tid = WAVE_ROW ? threadIdx.x & 63 : threadIdx.x;
  const int threads = WAVE_ROW ? 64 : blockDim.x;
  const int waves = WAVE_ROW ? 1 : blockDim.x >> 6;
  const int64_t row0 = WAVE_ROW ? static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 6) : blockIdx.x;
  const int64_t step = static_cast<int64_t>(gridDim.x) * (WAVE_ROW ? 4 : 1);
  const int chunks = static_cast<int>(p.K / VEC);
  const float inv_k = 1.0f / static_cast<float>(p.K);
  int turn = 0;
  for (int64_t row = row0; row < p.M; row += step) {
    const int64_t base = row * p.K;
    Chunk<T, VEC> b[ITEMS], r[ITEMS], g[ITEMS];
    float sum = 0.0f;
#pragma unroll
    for (int j = 0; j < ITEMS; ++j) {
      const int c = tid + j * threads;
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        b[j].v[i] = 0.0f;
        r[j].v[i] = 0.0f;
        g[j].v[i] = 1.0f;
      }
      if (c < chunks) {
        const int64_t k = static_cast<int64_t>(c) * VEC;
        b[j].load(static_cast<const T*>(p.x) + base + k);
        if (p.residual) r[j].load(static_cast<const T*>(p.residual) + base + k);
        if (p.gate) g[j].load(static_cast<const T*>(p.gate) + row * p.gate_pitch + k);
      }
    }
    if (p.post) {
#pragma unroll
      for (int j = 0; j < ITEMS; ++j)
#pragma unroll
        for (int i = 0; i < VEC; ++i) sum = fmaf(b[j].v[i], b[j].v[i], sum);
      sum = block_sum(sum, red, waves, turn);
      const float inv = 1.0f / sqrtf(fmaf(sum, inv_k, p.eps));
#pragma unroll
      for (int j = 0; j < ITEMS; ++j) {
        const int c = tid + j * threads;
        if (c < chunks) {
          Chunk<T, VEC> w;
          w.load(static_cast<const T*>(p.post) + static_cast<int64_t>(c) * VEC);
#pragma unroll
          for (int i = 0; i < VEC; ++i) b[j].v[i] *= inv * (p.offset + w.v[i]);
        }
      }
    }
    sum = 0.0f;
#pragma unroll
    for (int j = 0; j < ITEMS; ++j)
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        r[j].v[i] = fmaf(p.scale * g[j].v[i], b[j].v[i], r[j].v[i]);
        sum = fmaf(r[j].v[i], r[j].v[i], sum);
      }
    if (p.r_out) {
#pragma unroll
      for (int j = 0; j < ITEMS; ++j) {
        const int c = tid + j * threads;
        if (c < chunks) r[j].store(static_cast<T*>(p.r_out) + base + static_cast<int64_t>(c) * VEC);
      }
    }
    if (p.y) {
      sum = block_sum(sum, red, waves, turn);
      const float inv = 1.0f / sqrtf(fmaf(sum, inv_k, p.eps));
#pragma unroll
      for (int j = 0; j < ITEMS; ++j) {
        const int c = tid + j * threads;
        if (c < chunks) {
          Chunk<T, VEC> w;
          w.load(static_cast<const T*>(p.pre) + static_cast<int64_t>(c) * VEC);
#pragma unroll
          for (int i = 0; i < VEC; ++i) w.v[i] = r[j].v[i] * (inv * (p.offset + w.v[i]));
          w.store(static_cast<T*>(p.y) + base + static_cast<int64_t>(c) * VEC);
        }
      }
    }
  }
}

// Any row length: r is computed again for the second sum and for the result.
// The outputs are written in the last pass, each element by the thread that
// has just read it, so they may take the place of x and residual here too.
template <typename T>
__global__ __launch_bounds__(1024) void block_norm_long_kernel(const NormParams p) {
  __shared__ float red[32];
  const int tid = threadIdx.x, threads = blockDim.x, waves = blockDim.x >> 6;
  const float inv_k = 1.0f / static_cast<float>(p.K);
  int turn = 0;
  for (int64_t row = blockIdx.x; row < p.M; row += gridDim.x) {
    const T* x = static_cast<const T*>(p.x) + row * p.K;
    const T* res = p.residual ? static_cast<const T*>(p.residual) + row * p.K : nullptr;
    const T* gate = p.gate ? static_cast<const T*>(p.gate) + row * p.gate_pitch : nullptr;
    const T* post = static_cast<const T*>(p.post);
    const T* pre = static_cast<const T*>(p.pre);
    float inv_post = 1.0f;
    if (post) {
      float sum = 0.0f;
      for (int64_t k = tid; k < p.K; k += threads) {
        const float v = static_cast<float>(x[k]);
        sum = fmaf(v, v, sum);
      }
      inv_post = 1.0f / sqrtf(fmaf(block_sum(sum, red, waves, turn), inv_k, p.eps));
    }
    auto r_at = [&](int64_t k) {
      float b = static_cast<float>(x[k]);
      if (post) b *= inv_post * (p.offset + static_cast<float>(post[k]));
      const float g = gate ? static_cast<float>(gate[k]) : 1.0f;
      return fmaf(p.scale * g, b, res ? static_cast<float>(res[k]) : 0.0f);
    };
    float inv_pre = 1.0f;
    if (p.y) {
      float sum = 0.0f;
      for (int64_t k = tid; k < p.K; k += threads) {
        const float v = r_at(k);
        sum = fmaf(v, v, sum);
      }
      inv_pre = 1.0f / sqrtf(fmaf(block_sum(sum, red, waves, turn), inv_k, p.eps));
    }
    for (int64_t k = tid; k < p.K; k += threads) {
      const float v = r_at(k);
      const float w = p.y ? v * (inv_pre * (p.offset + static_cast<float>(pre[k]))) : 0.0f;
      if (p.r_out) static_cast<T*>(p.r_out)[row * p.K + k] = static_cast<T>(v);
      if (p.y) static_cast<T*>(p.y)[row * p.K + k] = static_cast<T>(w);
    }
  }
}

constexpr int64_t kMaxGrid = int64_t(1) << 20;  // rows beyond it are looped over

template <typename T, int VEC, int ITEMS>
void launch_rows(const NormParams& p, int64_t chunks, hipStream_t s) {
  const int64_t per = (chunks + ITEMS - 1) / ITEMS;
  const int threads = static_cast<int>((per + 63) / 64 * 64);
  const int grid = static_cast<int>(p.M < kMaxGrid ? p.M : kMaxGrid);
  hipLaunchKernelGGL((block_norm_kernel<T, VEC, ITEMS, false>), dim3(grid), dim3(threads), 0, s, p);
}

template <typename T, int VEC>
void launch_t(const NormParams& p, hipStream_t s) {
  const int64_t chunks = p.K / VEC;
  if (chunks <= 64) {
    const int64_t groups = (p.M + 3) / 4;
    const int grid = static_cast<int>(groups < kMaxGrid ? groups : kMaxGrid);
    hipLaunchKernelGGL((block_norm_kernel<T, VEC, 1, true>), dim3(grid), dim3(256), 0, s, p);
  } else if (chunks <= 1024) {
    launch_rows<T, VEC, 1>(p, chunks, s);
  } else if (chunks <= 2048) {
    launch_rows<T, VEC, 2>(p, chunks, s);
  } else if (chunks <= 4096) {
    launch_rows<T, VEC, 4>(p, chunks, s);
  } else {
    const int grid = static_cast<int>(p.M < kMaxGrid ? p.M : kMaxGrid);
    hipLaunchKernelGGL(block_norm_long_kernel<T>, dim3(grid), dim3(1024), 0, s, p);
  }
}

}  // namespace

int launch_block_norm(const BlockNormArgs& a, bool vec) {
  const NormParams p{a.x,     a.post_weight, a.gate, a.residual, a.pre_weight, a.residual_out, a.y, a.M, a.K,
                     a.gate_rows == 1 ? 0 : a.K, a.scale, a.weight_offset, a.eps};
  hipStream_t s = static_cast<hipStream_t>(a.stream);
  if (a.act == Act::BF16)
    vec ? launch_t<__bf16, 8>(p, s) : launch_t<__bf16, 1>(p, s);
  else
    vec ? launch_t<_Float16, 8>(p, s) : launch_t<_Float16, 1>(p, s);
  return hipGetLastError() == hipSuccess ? 0 : -1;
}

}  // namespace fp4w
