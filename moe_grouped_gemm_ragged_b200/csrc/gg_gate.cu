// The gate before the routing: each token's k experts and their weights from the router's
// logits, and the gradient of the logits from the gradient of the weights. One warp takes a
// token; its logits stay in registers.
#include <cmath>
#include <cstdint>

#include "gg_ops.cuh"

namespace gg {
namespace gate {

using namespace gg::ops;

constexpr int THREADS = 128;
constexpr int WARPS = THREADS / 32;
constexpr uint32_t ALL = 0xffffffffu;

struct Params {
  const void* logits;
  const float* bias;
  const int32_t* num_tokens;
  int32_t* ids;
  float* weights;
  const float* dweights;
  void* dlogits;
  int32_t* status;
  int64_t T;
  int32_t E;
  int32_t k;
  float scale;
};

__device__ __forceinline__ float load(const float* p) { return *p; }
__device__ __forceinline__ float load(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void store(float* p, float v) { *p = v; }
__device__ __forceinline__ void store(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(ALL, v, d);
  return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v = fmaxf(v, __shfl_xor_sync(ALL, v, d));
  return v;
}

// Unsigned keys that grow with the value; every number's key is above 0, which stands for an
// expert that cannot be chosen. + 0 turns -0 into +0: the two are a tie.
__device__ __forceinline__ uint32_t key_of(float v) {
  const uint32_t u = __float_as_uint(v + 0.f);
  return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ uint64_t key_of(double v) {
  const uint64_t u = (uint64_t)__double_as_longlong(v + 0.0);
  return u ^ ((u >> 63) ? ~0ull : 0x8000000000000000ull);
}
__device__ __forceinline__ uint32_t warp_max_key(uint32_t k) { return __reduce_max_sync(ALL, k); }
__device__ __forceinline__ uint64_t warp_max_key(uint64_t k) {
  const uint32_t hi = __reduce_max_sync(ALL, (uint32_t)(k >> 32));
  const uint32_t lo = __reduce_max_sync(ALL, (uint32_t)(k >> 32) == hi ? (uint32_t)k : 0u);
  return ((uint64_t)hi << 32) | lo;
}
template <bool BIAS> struct KeyOf { using type = uint32_t; };
template <> struct KeyOf<true> { using type = uint64_t; };

// A logit that can be chosen is finite. -inf is the mask; NaN and +inf are reported and then
// treated as masked.
__device__ __forceinline__ float logit_or_mask(float x, bool* bad) {
  if (!(x < INFINITY)) {
    *bad = true;
    return -INFINITY;
  }
  return x;
}

// sigma(x) e^-m for m <= 0: e^(min(x, 0) - m) / (1 + e^-|x|), which stays a normal number for
// the largest of a token's scores however small it is when m is that score's min(x, 0).
__device__ __forceinline__ float sigmoid_over(float x, float m) {
  return expf(fminf(x, 0.f) - m) / (1.f + expf(-fabsf(x)));
}

// Shares of the k chosen (lane s: slot s): softmax or sigmoid scores over their sum.
__device__ __forceinline__ float share(bool live, float x, bool sigmoid) {
  const float at = live ? (sigmoid ? fminf(x, 0.f) : x) : -INFINITY;
  const float m = warp_max(at);
  float v = 0.f;
  if (live) v = sigmoid ? sigmoid_over(x, m) : expf(x - m);
  const float total = warp_sum(v);
  return live ? v / total : 0.f;
}

// Choice by the logit itself without a bias (both scores grow with it, so the choice is
// exact), by sigma(x) + bias in double precision with one: neighbours of 256 scores are often
// closer than fp32 tells apart. Ties go to the lowest index.
template <typename L, int NV, bool BIAS>
__global__ void __launch_bounds__(THREADS) gate_kernel(Params p, bool sigmoid, bool renorm) {
  using Key = typename KeyOf<BIAS>::type;
  const int lane = threadIdx.x & 31;
  const int64_t t = (int64_t)blockIdx.x * WARPS + (threadIdx.x >> 5);
  if (t >= p.T) return;
  bool bad_count = false, bad = false;
  int64_t live_tokens = p.T;
  if (p.num_tokens != nullptr) {
    live_tokens = *p.num_tokens;
    bad_count = live_tokens < 0 || live_tokens > p.T;
  }
  float x[NV];
  Key key[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = lane + 32 * j;
    x[j] = -INFINITY;
    if (c < p.E && t < live_tokens)
      x[j] = logit_or_mask(load(static_cast<const L*>(p.logits) + t * p.E + c), &bad);
    key[j] = 0;
    if (x[j] > -INFINITY) {
      if constexpr (BIAS) {
        const float b = p.bias[c];
        if (!(b < INFINITY)) bad = true;
        else if (b > -INFINITY) key[j] = key_of(1.0 / (1.0 + exp(-(double)x[j])) + (double)b);
      } else {
        key[j] = key_of(x[j]);
      }
    }
  }
  int32_t my_id = -1;
  float my_x = -INFINITY;
  for (int s = 0; s < p.k; ++s) {
    Key best = 0;
    int at = 0;
    float bx = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j)
      if (key[j] > best) {
        best = key[j];
        at = j;
        bx = x[j];
      }
    const Key top = warp_max_key(best);
    if (top == 0) break;  // nothing left to choose
    const uint32_t c = __reduce_min_sync(ALL, best == top ? (uint32_t)(lane + 32 * at) : ALL);
    const float cx = __shfl_sync(ALL, bx, c & 31);
    if (lane == s) {
      my_id = (int32_t)c;
      my_x = cx;
    }
#pragma unroll
    for (int j = 0; j < NV; ++j)
      if (c == (uint32_t)(lane + 32 * j)) key[j] = 0;
  }
  const bool live = my_id >= 0;
  float w;
  if (renorm) {
    w = share(live, my_x, sigmoid);
  } else if (sigmoid) {
    w = live ? sigmoid_over(my_x, 0.f) : 0.f;
  } else {
    const float m = __shfl_sync(ALL, my_x, 0);
    float sum = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j)
      if (x[j] > -INFINITY) sum += expf(x[j] - m);
    sum = warp_sum(sum);
    w = live ? expf(my_x - m) / sum : 0.f;
  }
  if (lane < p.k) {
    p.ids[t * p.k + lane] = my_id;
    p.weights[t * p.k + lane] = live ? p.scale * w : 0.f;
  }
  bad = __any_sync(ALL, bad);
  if (lane == 0 && (bad || (bad_count && t == 0)))
    flag(p.status, (bad ? GG_DEV_BAD_LOGIT : 0u) | (bad_count ? GG_DEV_BAD_COUNT : 0u));
}

// Gradient of the logits. With v the weights before `scale` and g = scale * dweights:
//   softmax over all      dx_j = p_j (g_j - sum_i g_i p_i)   (g_j = 0 for the others)
//   softmax renormalised  dx_i = v_i (g_i - sum g v)
//   sigmoid               dx_i = g_i s_i (1 - s_i)
//   sigmoid renormalised  dx_i = v_i (1 - s_i) (g_i - sum g v)
// The chosen slots' scores are computed again from their logits; dx of a logit that was not
// chosen is 0 but for the first form. A slot of id -1 carries nothing.
template <typename L, int NV>
__global__ void __launch_bounds__(THREADS) gate_backward_kernel(Params p, bool sigmoid,
                                                                bool renorm) {
  const int lane = threadIdx.x & 31;
  const int64_t t = (int64_t)blockIdx.x * WARPS + (threadIdx.x >> 5);
  if (t >= p.T) return;
  const L* row = static_cast<const L*>(p.logits) + t * p.E;
  L* drow = static_cast<L*>(p.dlogits) + t * p.E;
  int32_t id = -1;
  float g = 0.f, x = -INFINITY;
  bool bad = false;
  if (lane < p.k) {
    id = p.ids[t * p.k + lane];
    if (id >= p.E) {
      bad = true;
      id = -1;
    }
    if (id >= 0) {
      bool ignored = false;
      x = logit_or_mask(load(row + id), &ignored);
      if (x > -INFINITY) g = p.scale * p.dweights[t * p.k + lane];
    }
  }
  const bool live = x > -INFINITY;
  const bool any = __any_sync(ALL, live);
  float all[NV];  // softmax over all: the row's logits, then its probabilities
  float mine = 0.f, others = 0.f, m = 0.f, inv = 0.f;
  if (!sigmoid && !renorm) {
    float top = -INFINITY;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = lane + 32 * j;
      bool ignored = false;
      all[j] = c < p.E && any ? logit_or_mask(load(row + c), &ignored) : -INFINITY;
      top = fmaxf(top, all[j]);
    }
    m = any ? warp_max(top) : 0.f;
    float sum = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      all[j] = all[j] > -INFINITY ? expf(all[j] - m) : 0.f;
      sum += all[j];
    }
    sum = warp_sum(sum);
    inv = any ? 1.f / sum : 0.f;
    const float v = live ? expf(x - m) * inv : 0.f;
    others = warp_sum(g * v);
    mine = g * v;
  } else if (renorm) {
    const float v = share(live, x, sigmoid);
    const float mean = warp_sum(g * v);
    mine = live ? v * (g - mean) : 0.f;
    if (sigmoid && live) mine *= sigmoid_over(-x, 0.f);  // 1 - sigma(x) = sigma(-x)
  } else if (live) {
    mine = g * sigmoid_over(x, 0.f) * sigmoid_over(-x, 0.f);
  }
  float d[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) d[j] = !sigmoid && !renorm ? -others * (all[j] * inv) : 0.f;
  for (int s = 0; s < p.k; ++s) {
    const int c = __shfl_sync(ALL, id, s);
    const float v = __shfl_sync(ALL, mine, s);
#pragma unroll
    for (int j = 0; j < NV; ++j)
      if (c == lane + 32 * j) d[j] += v;
  }
#pragma unroll
  for (int j = 0; j < NV; ++j)
    if (lane + 32 * j < p.E) store(drow + lane + 32 * j, d[j]);
  if (bad) flag(p.status, GG_DEV_BAD_ROUTE);
}

template <typename L, bool BIAS>
void launch_gate(const Params& p, bool sigmoid, bool renorm, cudaStream_t stream) {
  const unsigned grid = (unsigned)((p.T + WARPS - 1) / WARPS);
  const int nv = (p.E + 31) / 32;
  if (nv <= 2) gate_kernel<L, 2, BIAS><<<grid, THREADS, 0, stream>>>(p, sigmoid, renorm);
  else if (nv <= 8) gate_kernel<L, 8, BIAS><<<grid, THREADS, 0, stream>>>(p, sigmoid, renorm);
  else gate_kernel<L, 32, BIAS><<<grid, THREADS, 0, stream>>>(p, sigmoid, renorm);
}

template <typename L>
void launch_backward(const Params& p, bool sigmoid, bool renorm, cudaStream_t stream) {
  const unsigned grid = (unsigned)((p.T + WARPS - 1) / WARPS);
  const int nv = (p.E + 31) / 32;
  if (nv <= 2) gate_backward_kernel<L, 2><<<grid, THREADS, 0, stream>>>(p, sigmoid, renorm);
  else if (nv <= 8) gate_backward_kernel<L, 8><<<grid, THREADS, 0, stream>>>(p, sigmoid, renorm);
  else gate_backward_kernel<L, 32><<<grid, THREADS, 0, stream>>>(p, sigmoid, renorm);
}

gg_status check(int64_t T, int32_t E, int32_t k, int32_t score, int32_t flags, float scale,
                const int32_t* dev_status) {
  if (T < 0 || E < 1 || k < 1 || k > E) return GG_ERR_INVALID_ARG;
  if (score != GG_GATE_SOFTMAX && score != GG_GATE_SIGMOID) return GG_ERR_INVALID_ARG;
  if (flags & ~(GG_GATE_RENORM | GG_GATE_LOGITS_F32)) return GG_ERR_INVALID_ARG;
  if (!std::isfinite(scale)) return GG_ERR_INVALID_ARG;
  if (E > GG_MAX_EXPERTS || k > GG_GATE_MAX_K) return GG_ERR_UNSUPPORTED;
  if (T >= (int64_t(1) << 31)) return GG_ERR_UNSUPPORTED;
  if (misaligned(dev_status, 4)) return GG_ERR_UNSUPPORTED;
  return GG_OK;
}

}  // namespace gate
}  // namespace gg

extern "C" {

gg_status gg_gate_topk(const void* logits, int64_t T, int32_t E, int32_t k, const float* bias,
                       int32_t score, int32_t flags, float scale, const int32_t* num_tokens,
                       int32_t* topk_ids, float* weights, int32_t* dev_status,
                       cudaStream_t stream) {
  using namespace gg::gate;
  gg_status s = check(T, E, k, score, flags, scale, dev_status);
  if (s != GG_OK) return s;
  if (bias != nullptr && score != GG_GATE_SIGMOID) return GG_ERR_INVALID_ARG;
  const bool f32 = (flags & GG_GATE_LOGITS_F32) != 0;
  if (misaligned(logits, f32 ? 4 : 2) || misaligned(bias, 4) || misaligned(num_tokens, 4) ||
      misaligned(topk_ids, 4) || misaligned(weights, 4))
    return GG_ERR_UNSUPPORTED;
  if (T > 0 && (logits == nullptr || topk_ids == nullptr || weights == nullptr))
    return GG_ERR_INVALID_ARG;
  int sms = 0;
  if ((s = device_sms(&sms)) != GG_OK) return s;
  if (T == 0) return GG_OK;
  Params p = {};
  p.logits = logits;
  p.bias = bias;
  p.num_tokens = num_tokens;
  p.ids = topk_ids;
  p.weights = weights;
  p.status = dev_status;
  p.T = T;
  p.E = E;
  p.k = k;
  p.scale = scale;
  const bool sig = score == GG_GATE_SIGMOID, renorm = (flags & GG_GATE_RENORM) != 0;
  if (f32 && bias) launch_gate<float, true>(p, sig, renorm, stream);
  else if (f32) launch_gate<float, false>(p, sig, renorm, stream);
  else if (bias) launch_gate<__nv_bfloat16, true>(p, sig, renorm, stream);
  else launch_gate<__nv_bfloat16, false>(p, sig, renorm, stream);
  return launched("gg_gate_topk");
}

gg_status gg_gate_topk_backward(const void* logits, int64_t T, int32_t E, int32_t k,
                                int32_t score, int32_t flags, float scale,
                                const int32_t* topk_ids, const float* dweights, void* dlogits,
                                int32_t* dev_status, cudaStream_t stream) {
  using namespace gg::gate;
  gg_status s = check(T, E, k, score, flags, scale, dev_status);
  if (s != GG_OK) return s;
  const bool f32 = (flags & GG_GATE_LOGITS_F32) != 0;
  if (misaligned(logits, f32 ? 4 : 2) || misaligned(dlogits, f32 ? 4 : 2) ||
      misaligned(topk_ids, 4) || misaligned(dweights, 4))
    return GG_ERR_UNSUPPORTED;
  if (T > 0 && (logits == nullptr || topk_ids == nullptr || dweights == nullptr ||
                dlogits == nullptr))
    return GG_ERR_INVALID_ARG;
  int sms = 0;
  if ((s = device_sms(&sms)) != GG_OK) return s;
  if (T == 0) return GG_OK;
  Params p = {};
  p.logits = logits;
  p.ids = const_cast<int32_t*>(topk_ids);
  p.dweights = dweights;
  p.dlogits = dlogits;
  p.status = dev_status;
  p.T = T;
  p.E = E;
  p.k = k;
  p.scale = scale;
  const bool sig = score == GG_GATE_SIGMOID, renorm = (flags & GG_GATE_RENORM) != 0;
  if (f32) launch_backward<float>(p, sig, renorm, stream);
  else launch_backward<__nv_bfloat16>(p, sig, renorm, stream);
  return launched("gg_gate_topk_backward");
}

}  // extern "C"
