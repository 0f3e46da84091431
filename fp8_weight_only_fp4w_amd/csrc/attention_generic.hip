// Attention over the paged 8-bit cache for any head size, page size, alignment
// and number of tokens: a workgroup per row and head, 256 tokens at a time,
// with the running maximum and sum of the softmax in FP32.  Made to be right for
// everything, not fast; attention.hip and attention_prompt.hip have the heads of
// 64 and 128.

#include <hip/hip_runtime.h>

#include "heads.h"

namespace fp4w {
namespace {

struct AttnParams {
  const void* q;
  int64_t q_stride;
  int32_t Hq, Hk, D, max_new;
  Seqs seq;
  const uint8_t* k_cache;
  const uint8_t* k_scale;
  const uint8_t* v_cache;
  const uint8_t* v_scale;
  float scale;
  bool causal;
  int64_t window;
  void* Y;
  float* lse;
};

// Values are summed times 2^-24: BF16 ones reach FP32's end, and their sum passes it.
constexpr float kHoldDown = 0x1p-24f;

__device__ __forceinline__ float block_reduce(float v, float* red, bool sum) {
  for (int off = 32; off > 0; off >>= 1) {
    const float o = __shfl_xor(v, off, 64);
    v = sum ? v + o : fmaxf(v, o);
  }
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  const float r = sum ? (red[0] + red[1]) + (red[2] + red[3]) : fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
  __syncthreads();
  return r;
}

template <typename T>
__global__ __launch_bounds__(256) void attention_generic_kernel(const AttnParams p) {
  __shared__ float qs[kMaxHead], weight[256], v_scale[256], red[4];
  __shared__ int64_t at[256];  // of a token's values in the cache; -1: not attended
  const int tid = threadIdx.x, D = p.D, page = p.seq.page;
  const int64_t units = static_cast<int64_t>(p.seq.M) * p.Hq;
  const int behind = seq_start(p.seq, p.seq.B);
  constexpr int kPer = kMaxHead / 256;
  for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
    const int64_t m = u / p.Hq;
    const int h = static_cast<int>(u - m * p.Hq), hk = h / (p.Hq / p.Hk);
    if (m >= behind) continue;
    const int b = last_not_above(p.seq.B, m, [&](int i) { return seq_start(p.seq, i); });
    const SeqSpan s = seq_span(p.seq, b);
    if (m - s.first_row >= p.max_new) continue;
    const int64_t position = static_cast<int64_t>(s.len) - s.rows + (m - s.first_row);
    int64_t lo = p.window > 0 ? position - p.window + 1 : 0, hi = p.causal ? position + 1 : s.len;
    lo = lo < 0 ? 0 : lo;
    hi = hi < s.len ? hi : s.len;
    hi = hi < p.seq.capacity ? hi : p.seq.capacity;
    const T* q = static_cast<const T*>(p.q) + m * p.q_stride + static_cast<int64_t>(h) * D;
    __syncthreads();
    float most = 0.0f;
    for (int d = tid; d < D; d += 256) most = fmaxf(most, fabsf(static_cast<float>(q[d])));
    const bool far = block_reduce(most, red, false) >= kFar;
    for (int d = tid; d < D; d += 256) qs[d] = static_cast<float>(q[d]) * (far ? kFarDown : 1.0f);
    __syncthreads();
    float top = -INFINITY, sum = 0.0f, acc[kPer] = {};
    for (int64_t t0 = lo; t0 < hi; t0 += 256) {
      const int64_t t = t0 + tid;
      const int id = t < hi ? page_of(p.seq, b, static_cast<int>(t)) : -1;
      float score = -INFINITY, vs = 0.0f;
      at[tid] = -1;
      if (id >= 0) {
        const int64_t cell = static_cast<int64_t>(id) * p.Hk + hk;
        const int slot = static_cast<int>(t - static_cast<int64_t>(fdiv(static_cast<uint32_t>(t), p.seq.page_div)) * page);
        const uint8_t* k = p.k_cache + (cell * page + slot) * D;
        float dot = 0.0f;
        for (int d = 0; d < D; ++d) dot = fmaf(qs[d], e4m3_to_f32<0>(k[d]), dot);
        score = dot * e8m0_to_f32(p.k_scale[cell]) * p.scale * (far ? kFarUp : 1.0f);
        vs = e8m0_to_f32(p.v_scale[cell]);
        at[tid] = cell * D * page + slot;
      }
      // (-inf until a token is attended)
      const float now = fmaxf(top, block_reduce(id >= 0 ? fmaxf(score, -__FLT_MAX__) : -INFINITY, red, false));
      const float base = now > -INFINITY ? now : 0.0f;
      const float w = id >= 0 ? expf(score - base) : 0.0f;
      const float shrink = expf(top - base);
      sum = sum * shrink + block_reduce(w, red, true);
      weight[tid] = w;
      v_scale[tid] = vs * kHoldDown;
      __syncthreads();
      const int n = static_cast<int>(hi - t0 < 256 ? hi - t0 : 256);
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        const int d = tid + j * 256;
        if (d < D) {
          float a = acc[j] * shrink;
          for (int i = 0; i < n; ++i)
            if (at[i] >= 0) {
              const float v = e4m3_to_f32<0>(p.v_cache[at[i] + static_cast<int64_t>(d) * page]) * v_scale[i];
              a = fmaf(weight[i], v, a);
            }
          acc[j] = a;
        }
      }
      top = now;
      __syncthreads();
    }
    // a sum of 0: no token attended, and 0 is stored; or every score is -inf, and 0 / 0
    const bool none = sum == 0.0f && top == -INFINITY;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int d = tid + j * 256;
      if (d < D) static_cast<T*>(p.Y)[u * D + d] = round_to<T>(none ? 0.0f : acc[j] / (sum * kHoldDown));
    }
    if (p.lse != nullptr && tid == 0) p.lse[u] = none ? -INFINITY : sum == 0.0f ? NAN : top + logf(sum);
  }
}

template <typename T>
int launch_t(const AttnParams& p, hipStream_t s) {
  const int64_t units = static_cast<int64_t>(p.seq.M) * p.Hq;
  const int grid = static_cast<int>(units < (1 << 20) ? units : 1 << 20);
  hipLaunchKernelGGL(attention_generic_kernel<T>, dim3(grid), dim3(256), 0, s, p);
  return hipGetLastError() == hipSuccess ? 0 : -1;
}

}  // namespace

int launch_attention_generic(const AttentionArgs& a) {
  const AttnParams p{a.q, a.q_stride, static_cast<int32_t>(a.Hq), static_cast<int32_t>(a.Hk), static_cast<int32_t>(a.D),
                     static_cast<int32_t>(a.max_new), make_seqs(a.seq, a.M), a.k_cache, a.k_scale, a.v_cache, a.v_scale,
                     a.scale, a.causal, a.window, a.Y, a.lse};
  hipStream_t s = static_cast<hipStream_t>(a.stream);
  return a.act == Act::BF16 ? launch_t<__bf16>(p, s) : launch_t<_Float16>(p, s);
}

}  // namespace fp4w
