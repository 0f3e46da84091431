// Routing of tokens to experts: the topk largest keys of each row of logits,
// ties to the lowest index, and the weights of the experts chosen.
//
//   score = softmax(logits) over the row, or sigmoid(logits)
//   key   = logits                 without a selection bias (both scores rise with the logit)
//         = score + select_bias    with one
//   weight = scale * score[chosen]  ( / the chosen scores' sum, renormalised )
//
// A logit of -inf or NaN masks its expert; places that no expert is left for
// get id -1 and weight 0.  A key with a bias is formed in FP64, so that which
// of two nearly equal experts is chosen does not hang on how an FP32 exponential
// rounds; without a bias the comparison is of the logits themselves, exact.
//
// A wave owns a row.  Lane l holds the PER consecutive experts from l * PER
// as integers that order like the keys, 0 for what is masked, and sorts them
// (only as many places as there are choices).  A round is one wave maximum of
// the lanes' first keys (DPP within the rows of 16 lanes, then across them);
// the lowest lane that holds it has the lowest index, and takes its next key
// to the front.  The low half of a 64-bit key is looked at only where several
// lanes share the high half of the maximum.  An expert's weight is computed
// after the rounds by the lane of its place, so a row costs one exponential
// more than its keys need (two for renormalised sigmoids below a half).  One token is bound by latency (a launch and topk
// rounds), a prompt by instructions: about 1150 per row of 256 experts with a
// bias, half of them the 8 rounds and a quarter the FP64 keys.  Measured: 2.7 us
// for one token of 128 experts; 13.3 us for 8192 tokens of 256 with a sigmoid
// and a bias, where a search of all of a lane's keys in every round and both
// halves of each maximum took 15.5.  Weights relative to the largest chosen score
// cost 0.1 us of that, and 0.6 of 14.5 with a softmax whose top the bias passes by.

#include <hip/hip_runtime.h>

#include "device.h"
#include "launch.h"

namespace fp4w {
namespace {

constexpr int kRouteWaves = 4;  // rows per workgroup
// Scores below exp of it (softmax: times the largest) count as 0: FP64, which
// the keys are formed in, ends there.
constexpr float kScoreEnd = -700.0f;

template <int CTRL, int ROW_MASK>
__device__ __forceinline__ uint32_t dpp_max(uint32_t v) {
  // lanes without a source, or outside ROW_MASK, take 0
  const uint32_t o = static_cast<uint32_t>(
      __builtin_amdgcn_update_dpp(0, static_cast<int>(v), CTRL, ROW_MASK, 0xF, false));
  return v > o ? v : o;
}

// maximum over the 64 lanes, on every lane (wave-uniform)
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
  v = dpp_max<0x111, 0xF>(v);  // row_shr:1
  v = dpp_max<0x112, 0xF>(v);  // row_shr:2
  v = dpp_max<0x114, 0xF>(v);  // row_shr:4
  v = dpp_max<0x118, 0xF>(v);  // row_shr:8
  v = dpp_max<0x142, 0xA>(v);  // row_bcast:15 into rows 1 and 3
  v = dpp_max<0x143, 0xC>(v);  // row_bcast:31 into rows 2 and 3
  return __builtin_amdgcn_readlane(v, 63);
}

// The lanes that hold the largest key, 0 where every key is 0 (wave-uniform).
__device__ __forceinline__ uint64_t lanes_of_max(uint32_t key) {
  const uint32_t win = wave_max(key);
  return win ? __ballot(key == win) : 0;
}
__device__ __forceinline__ uint64_t lanes_of_max(uint64_t key) {
  const uint32_t hi = static_cast<uint32_t>(key >> 32), lo = static_cast<uint32_t>(key);
  const uint32_t win = wave_max(hi);
  if (win == 0) return 0;  // every nonzero key has a nonzero high half
  const uint64_t mask = __ballot(hi == win);
  if ((mask & (mask - 1)) == 0) return mask;
  const uint32_t low = wave_max(hi == win ? lo : 0u);
  return __ballot(hi == win && lo == low);
}

template <typename F>
__device__ __forceinline__ F wave_sum(F v) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off, 64);
  return v;
}

// Unsigned integers that order like the values; -inf and NaN give 0, below
// every other value.  -0 and +0 are one value (adding 0 turns -0 into +0).
__device__ __forceinline__ uint32_t order_key(float x) {
  if (!(x > -INFINITY)) return 0u;
  const uint32_t b = __builtin_bit_cast(uint32_t, x + 0.0f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ uint64_t order_key(double x) {
  if (!(x > -INFINITY)) return 0u;
  const uint64_t b = __builtin_bit_cast(uint64_t, x + 0.0);
  return b >> 63 ? ~b : b | (uint64_t(1) << 63);
}
__device__ __forceinline__ float from_order_key(uint32_t k) {
  return __builtin_bit_cast(float, k >> 31 ? k & 0x7FFFFFFFu : ~k);
}
// exp(x - top), 1 where x is the top itself (+inf included)
__device__ __forceinline__ float exp_below(float x, float top) { return x == top ? 1.0f : expf(x - top); }

// PER: experts per lane.  BIAS: FP64 keys of score + bias.
template <typename L, int PER, bool BIAS>
__global__ __launch_bounds__(64 * kRouteWaves) void moe_route_kernel(
    const L* __restrict__ logits, const float* __restrict__ select_bias, int32_t* __restrict__ ids,
    float* __restrict__ weights, int64_t M, int E, int topk, int sigmoid, int renormalize, float scale) {
  typedef typename std::conditional<BIAS, uint64_t, uint32_t>::type key_t;
  const int lane = threadIdx.x & 63;
  const int64_t step = static_cast<int64_t>(gridDim.x) * kRouteWaves;
  for (int64_t m = static_cast<int64_t>(blockIdx.x) * kRouteWaves + (threadIdx.x >> 6); m < M; m += step) {
    const L* row = logits + m * E;
    float x[PER];
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      const int e = lane * PER + j;
      x[j] = e < E ? static_cast<float>(row[e]) : -INFINITY;
    }
    // the largest logit (FP32 order is exact for every logit type)
    float top = -INFINITY;
    uint32_t top_key = 0;
#pragma unroll
    for (int j = 0; j < PER; ++j) top_key = max(top_key, order_key(x[j]));
    top_key = wave_max(top_key);
    if (top_key) top = from_order_key(top_key);
    // the softmax's denominator, where it is needed
    float sum = 1.0f;
    double sum64 = 1.0;
    if (!sigmoid) {
      if constexpr (BIAS) {
        sum64 = 0.0;
#pragma unroll
        for (int j = 0; j < PER; ++j)
          if (x[j] > -INFINITY) sum64 += x[j] == top ? 1.0 : exp(static_cast<double>(x[j]) - static_cast<double>(top));
        sum64 = wave_sum(sum64);
      } else if (!renormalize) {
        sum = 0.0f;
#pragma unroll
        for (int j = 0; j < PER; ++j)
          if (x[j] > -INFINITY) sum += exp_below(x[j], top);
        sum = wave_sum(sum);
      }
    }
    key_t key[PER];
    int slot[PER];
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      const int e = lane * PER + j;
      slot[j] = e;
      if constexpr (BIAS) {
        key[j] = 0;
        if (x[j] > -INFINITY) {
          const double xd = static_cast<double>(x[j]);
          const double s =
              sigmoid ? 1.0 / (1.0 + exp(-xd)) : (x[j] == top ? 1.0 : exp(xd - static_cast<double>(top))) / sum64;
          key[j] = order_key(s + static_cast<double>(select_bias[e]));
        }
      } else {
        key[j] = order_key(x[j]);
      }
    }
    // each pass brings the largest of the rest to place p; equal keys never
    // pass each other, so they stay in the order of their indices
#pragma unroll
    for (int p = 0; p < PER - 1; ++p) {
      if (p >= topk) break;
#pragma unroll
      for (int j = PER - 1; j > p; --j) {
        const bool up = key[j] > key[j - 1];
        const key_t k = key[j];
        const int e = slot[j];
        key[j] = up ? key[j - 1] : k;
        slot[j] = up ? slot[j - 1] : e;
        key[j - 1] = up ? k : key[j - 1];
        slot[j - 1] = up ? e : slot[j - 1];
      }
    }
    // lane i keeps the i-th choice
    int my_id = -1;
    for (int i = 0; i < topk; ++i) {
      const uint64_t mask = lanes_of_max(key[0]);
      if (mask == 0) break;  // nothing is left (wave-uniform)
      const int owner = __builtin_ctzll(mask);
      const int id = __builtin_amdgcn_readlane(slot[0], owner);
      if (lane == i) my_id = id;
      if (lane == owner) {
#pragma unroll
        for (int j = 0; j < PER - 1; ++j) {
          key[j] = key[j + 1];
          slot[j] = slot[j + 1];
        }
        key[PER - 1] = 0;
      }
    }
    // the weight of this lane's choice, up to a factor that renormalising
    // takes out again; its logit is on the lane that holds its expert
    const int from = my_id < 0 ? 0 : my_id;
    float xs = 0.0f;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      const float t = __shfl(x[j], from / PER, 64);
      if (from % PER == j) xs = t;
    }
    // Renormalised scores count in units of exp(ref), where ref is the largest
    // chosen logit: from 87 below 0 (the top) on FP32 would lose the scores,
    // and their quotients with them.  Without a bias ref is the top, and with
    // one it is looked for only where it is below 0 (the top).
    const float most = sigmoid ? 0.0f : top;
    float ref = most;
    if constexpr (BIAS) {
      if (renormalize && __ballot(my_id >= 0 && xs >= most) == 0) {
        const uint32_t k = wave_max(my_id < 0 ? 0u : order_key(xs));
        if (k) ref = from_order_key(k);
      }
    } else if (renormalize) {
      ref = fminf(top, most);
    }
    float w;
    if (sigmoid) {
      const float e = expf(-fabsf(xs));
      w = xs < 0.0f ? e : 1.0f;
      if (ref < 0.0f) w = xs > kScoreEnd ? expf(xs - ref) : 0.0f;
      w = w / (1.0f + e);
    } else {
      w = exp_below(xs, ref);
      if (BIAS && ref < top && xs - top <= kScoreEnd) w = 0.0f;
    }
    if (my_id < 0) w = 0.0f;
    if (renormalize) {
      const float total = wave_sum(w);
      w = total > 0.0f ? w / total : 0.0f;
    } else if (!sigmoid) {
      w = w / (BIAS ? static_cast<float>(sum64) : sum);
    }
    if (lane < topk) {
      ids[m * topk + lane] = my_id;
      weights[m * topk + lane] = my_id < 0 ? 0.0f : w * scale;
    }
  }
}

template <typename L, int PER>
void launch_per(const MoeRouteArgs& a, hipStream_t s) {
  const int64_t groups = (a.M + kRouteWaves - 1) / kRouteWaves;
  const int grid = static_cast<int>(groups < (int64_t(1) << 20) ? groups : int64_t(1) << 20);
#define FP4W_ROUTE(BIAS)                                                                                     \
  hipLaunchKernelGGL((moe_route_kernel<L, PER, BIAS>), dim3(grid), dim3(64 * kRouteWaves), 0, s,             \
                     static_cast<const L*>(a.logits), a.select_bias, a.ids, a.weights, a.M,                  \
                     static_cast<int>(a.E), static_cast<int>(a.topk), static_cast<int>(a.sigmoid),           \
                     static_cast<int>(a.renormalize), a.scale)
  if (a.select_bias)
    FP4W_ROUTE(true);
  else
    FP4W_ROUTE(false);
#undef FP4W_ROUTE
}

template <typename L>
void launch_l(const MoeRouteArgs& a, hipStream_t s) {
  if (a.E <= 64)
    launch_per<L, 1>(a, s);
  else if (a.E <= 128)
    launch_per<L, 2>(a, s);
  else if (a.E <= 256)
    launch_per<L, 4>(a, s);
  else if (a.E <= 512)
    launch_per<L, 8>(a, s);
  else
    launch_per<L, 16>(a, s);
}

}  // namespace

int launch_moe_route(const MoeRouteArgs& a) {
  hipStream_t s = static_cast<hipStream_t>(a.stream);
  switch (a.logits_dtype) {
    case 0: launch_l<_Float16>(a, s); break;
    case 1: launch_l<__bf16>(a, s); break;
    default: launch_l<float>(a, s); break;
  }
  return hipGetLastError() == hipSuccess ? 0 : -1;
}

}  // namespace fp4w
