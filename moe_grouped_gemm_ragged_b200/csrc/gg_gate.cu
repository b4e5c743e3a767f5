// The gate before the routing: each token's k experts and their weights from the router's
// logits, and the gradient of the logits from the gradient of the weights. A group of 4 to 32
// lanes takes a token, each lane 2 to 32 neighbouring experts: their logits are a few wide loads
// and stay in registers. What bounds these kernels is instructions, not bytes.
#include <cfloat>
#include <cmath>
#include <cstdint>
#include <type_traits>

#include "gg_ops.cuh"

namespace gg {
namespace gate {

using namespace gg::ops;

constexpr int THREADS = 128;
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

__device__ __forceinline__ float to_float(float v) { return v; }
__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void store(float* p, float v) { *p = v; }
__device__ __forceinline__ void store(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// NV neighbouring logits of a row (first: the lane's first expert, lane * NV); the rest of the
// lane's share, past E, is masked. wide: E is a multiple of 8 and the rows start on 16 bytes, so
// that a lane's share does too when its own size is a multiple of that, and no vector reaches
// past E.
template <int NV>
__device__ __forceinline__ void load_row(const float* row, int first, int E, bool wide,
                                         float (&x)[NV]) {
#pragma unroll
  for (int j = 0; j < NV; j += 4) {
    if ((NV * 4) % 16 == 0 && wide && first + j < E) {
      const float4 v = *reinterpret_cast<const float4*>(row + first + j);
      x[j] = v.x, x[j + 1] = v.y, x[j + 2] = v.z, x[j + 3] = v.w;
    } else {
#pragma unroll
      for (int i = j; i < j + 4 && i < NV; ++i) x[i] = first + i < E ? row[first + i] : -INFINITY;
    }
  }
}
template <int NV>
__device__ __forceinline__ void load_row(const __nv_bfloat16* row, int first, int E, bool wide,
                                         float (&x)[NV]) {
#pragma unroll
  for (int j = 0; j < NV; j += 8) {
    if ((NV * 2) % 16 == 0 && wide && first + j < E) {
      float v[8];
      unpack_bf16(*reinterpret_cast<const uint4*>(row + first + j), v);
#pragma unroll
      for (int i = 0; i < 8; ++i) x[j + i] = v[i];
    } else {
#pragma unroll
      for (int i = j; i < j + 8 && i < NV; ++i)
        x[i] = first + i < E ? __bfloat162float(row[first + i]) : -INFINITY;
    }
  }
}
template <int NV>
__device__ __forceinline__ void store_row(float* row, int first, int E, bool wide,
                                          const float (&x)[NV]) {
#pragma unroll
  for (int j = 0; j < NV; j += 4) {
    if ((NV * 4) % 16 == 0 && wide && first + j < E) {
      *reinterpret_cast<float4*>(row + first + j) =
          make_float4(x[j], x[j + 1], x[j + 2], x[j + 3]);
    } else {
#pragma unroll
      for (int i = j; i < j + 4 && i < NV; ++i)
        if (first + i < E) row[first + i] = x[i];
    }
  }
}
template <int NV>
__device__ __forceinline__ void store_row(__nv_bfloat16* row, int first, int E, bool wide,
                                          const float (&x)[NV]) {
#pragma unroll
  for (int j = 0; j < NV; j += 8) {
    if ((NV * 2) % 16 == 0 && wide && first + j < E) {
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = x[j + i];
      *reinterpret_cast<uint4*>(row + first + j) = pack_bf16(v);
    } else {
#pragma unroll
      for (int i = j; i < j + 8 && i < NV; ++i)
        if (first + i < E) row[first + i] = __float2bfloat16_rn(x[i]);
    }
  }
}

// Reductions over the G lanes of a group (mask: those lanes of the warp).
template <int G>
__device__ __forceinline__ float group_sum(uint32_t mask, float v) {
#pragma unroll
  for (int d = G / 2; d > 0; d >>= 1) v += __shfl_xor_sync(mask, v, d);
  return v;
}
template <int G>
__device__ __forceinline__ float group_max(uint32_t mask, float v) {
#pragma unroll
  for (int d = G / 2; d > 0; d >>= 1) v = fmaxf(v, __shfl_xor_sync(mask, v, d));
  return v;
}
template <int G>
__device__ __forceinline__ uint32_t group_max(uint32_t mask, uint32_t v) {
  if constexpr (G == 32) {
    return __reduce_max_sync(mask, v);
  } else {
#pragma unroll
    for (int d = G / 2; d > 0; d >>= 1) v = max(v, __shfl_xor_sync(mask, v, d));
    return v;
  }
}
template <int G>
__device__ __forceinline__ uint64_t group_max(uint32_t mask, uint64_t v) {
#pragma unroll
  for (int d = G / 2; d > 0; d >>= 1) {
    const uint64_t o = __shfl_xor_sync(mask, v, d);
    v = o > v ? o : v;
  }
  return v;
}

// Unsigned keys that grow with the value; every number's key is above 0, which stands for an
// expert that cannot be chosen. + 0 turns -0 into +0: the two are a tie.
__device__ __forceinline__ uint32_t key_of(float v) {
  const uint32_t u = __float_as_uint(v + 0.f);
  return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t key) {
  return __uint_as_float(key ^ ((key >> 31) ? 0x80000000u : 0xffffffffu));
}
__device__ __forceinline__ uint64_t key_of(double v) {
  const uint64_t u = (uint64_t)__double_as_longlong(v + 0.0);
  return u ^ ((u >> 63) ? ~0ull : 0x8000000000000000ull);
}

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
  return __fdividef(expf(fminf(x, 0.f) - m), 1.f + expf(-fabsf(x)));
}
__device__ __forceinline__ float sigmoid(float x) {
  const float e = expf(-fabsf(x));
  return __fdividef(x < 0.f ? e : 1.f, 1.f + e);
}
// Shares are taken of plain scores where their sum is above this: what a score below the normal
// numbers loses is then under 2^-129 of the sum. Else of scores relative to the largest.
constexpr float PLAIN = 0x1p-20f;

// e^x for x <= 0 by the hardware's power: off by 2 units of 2^-23 of its own and 0.62 |x| of its
// argument's roundings (the product's half unit and log2 e's tenth), which a sum of a token's
// exponentials, the large ones of which have small |x|, hardly shows. 0 of -inf.
__device__ __forceinline__ float fast_exp(float x) {
  float t = x * 1.44269504f;
  asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(t));
  return t;
}

// The score that a biased choice tries first. In units of 2^-23 it is off by at most
// sigma (1 - sigma) (2 + 0.62 |x|) < 0.6 from the fast exponential, 2.5 from the sum and the
// reciprocal and (1 + |bias|) / 2 from the last sum; two scores further apart than CLOSE
// (1 + |bias| + |bias'|) are in the right order, with half of CLOSE to spare.
__device__ __forceinline__ float fast_score(float x, float b) {
  float t = x * -1.44269504f;  // 1 / (1 + 2^(-x log2 e))
  asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(t));
  t += 1.f;
  asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(t));
  return t + b;
}
constexpr float CLOSE = 16.f / 8388608.f;

// fp32 orders are looked up past the k-th until it is seen that no other expert may belong to
// the chosen, one place most often and this many at most. (With a fixed two places about one
// biased token in ten thousand of 256 experts stayed open, and one such token adds 4 us to a
// call.) Where more logits than these are equal at the k-th place, a token goes on to all of its
// experts' doubles: batches of nothing but zeros take 37 us of 32768 x 64 fp32 (10.6 of random
// logits) and 54 of 16411 x 256 (11.9), 65 under a bias (14.5).
constexpr int MORE = 4;

template <int SLOTS>
struct Chosen {  // of one token, in shared memory
  static constexpr int N = SLOTS;
  int32_t id[SLOTS];
  float x[SLOTS];
  float score[SLOTS];
  float bias[SLOTS];
};

// Batcher's odd-even merge sort of a lane's keys, largest first.
template <int NV>
__device__ __forceinline__ void sort_keys(uint32_t (&key)[NV]) {
#pragma unroll
  for (int p = 1; p < NV; p *= 2)
#pragma unroll
    for (int q = p; q >= 1; q /= 2)
#pragma unroll
      for (int j = q % p; j + q < NV; j += 2 * q)
#pragma unroll
        for (int i = j; i < j + q && i + q < NV; ++i)
          if (i / (2 * p) == (i + q) / (2 * p)) {
            const uint32_t hi = max(key[i], key[i + q]), lo = min(key[i], key[i + q]);
            key[i] = hi;
            key[i + q] = lo;
          }
}

// A 32-bit key: the upper 22 bits of a value's unsigned order over the complement of the
// expert's number, so that keys differ, the largest names its expert, and of equal values the
// lowest expert's is the largest. That is the whole of a bf16 value; fp32 values that share
// their 22 bits may come in the wrong order. Keys below LOWEST cannot be chosen.
constexpr uint32_t NUMBER = 0x3ffu;
constexpr uint32_t LOWEST = 0x00800000u;  // of the lowest finite number
static_assert(GG_MAX_EXPERTS <= NUMBER + 1, "an expert's number fits the key");
__device__ __forceinline__ uint32_t packed(float v, int expert) {
  return (key_of(v) & ~NUMBER) | (NUMBER - expert);
}
// A sum of a sigma is never -0.
__device__ __forceinline__ uint32_t packed_score(float v, int expert) {
  const uint32_t u = __float_as_uint(v);
  return ((u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u)) & ~NUMBER) | (NUMBER - expert);
}
__device__ __forceinline__ int expert_of(uint32_t key) { return (int)(NUMBER - (key & NUMBER)); }

// Whether what has the key b, or one below it, is surely under the first k, which have the key a
// or one above it. Under a bias |bias| <= |score| + 1 for the scores' errors.
template <bool BIAS>
__device__ __forceinline__ bool apart(uint32_t a, uint32_t b) {
  if constexpr (!BIAS) return (a ^ b) > NUMBER;
  const float va = value_of(a & ~NUMBER), vb = value_of(b | NUMBER);
  return va - vb > CLOSE * (3.f + fabsf(va) + fabsf(vb) + 2.f);
}

// The k largest keys of the group, in order, into c.id, and with ORDER more until the k-th is
// apart from the last, `most` at most (*open: it is not, and there are others). Each lane has
// sorted its keys; a round compares only the lanes' first keys and moves the winner's up, of
// which only DEPTH (at least `most`, or all of them) can still come first. Returns how many.
enum class Order { WHOLE, LOGITS, SCORES };
template <int G, int DEPTH, Order ORDER, int NV, typename C>
__device__ __forceinline__ int choose(uint32_t mask, int lane, int k, int most,
                                      uint32_t (&key)[NV], C& c, bool* open) {
  uint32_t kth = 0;
  for (int s = 0; s < most; ++s) {
    const uint32_t top = group_max<G>(mask, key[0]);
    if (top < LOWEST) return s;  // nothing left
    const bool won = key[0] == top;
#pragma unroll
    for (int j = 0; j + 1 < DEPTH; ++j) key[j] = won ? key[j + 1] : key[j];
    key[DEPTH - 1] = won ? 0u : key[DEPTH - 1];
    if (lane == 0) c.id[s] = (int32_t)top;
    if constexpr (ORDER != Order::WHOLE) {
      if (s >= k - 1) {
        if (s == k - 1) kth = top;
        else if (apart<ORDER == Order::SCORES>(kth, top)) return s + 1;
      }
    }
  }
  *open = ORDER != Order::WHOLE;
  return most;
}

// What decides the order: sigma(x) + b under a bias, else x.
template <bool BIAS>
__device__ __forceinline__ double double_score(float x, float b) {
  return BIAS ? 1.0 / (1.0 + exp(-(double)x)) + (double)b : (double)x;
}

// Orders n candidates by their doubles, ties to the lowest expert: each finds its place.
template <int G, bool BIAS, typename C>
__device__ __forceinline__ void order_double(uint32_t mask, int lane, int n, const float* bias,
                                             C& c, double* d) {
#pragma unroll 1
  for (int s = lane; s < n; s += G)
    d[s] = double_score<BIAS>(c.x[s], BIAS ? bias[c.id[s]] : 0.f);
  __syncwarp(mask);
  constexpr int PER = (C::N + G - 1) / G;
  int32_t id[PER], place[PER];
  float x[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int s = lane + i * G;
    if (s >= n) continue;
    id[i] = c.id[s];
    x[i] = c.x[s];
    place[i] = 0;
#pragma unroll 1
    for (int q = 0; q < n; ++q)
      place[i] += d[q] > d[s] || (d[q] == d[s] && c.id[q] < id[i]);
  }
  __syncwarp(mask);
#pragma unroll
  for (int i = 0; i < PER; ++i)
    if (lane + i * G < n) {
      c.id[place[i]] = id[i];
      c.x[place[i]] = x[i];
    }
}

// All of the token's experts by doubles, for the very few tokens that need it: a function of its
// own with the keys in local memory, so that it costs the others no registers.
template <typename L, int G, int NV, bool BIAS>
__device__ __noinline__ int choose_double(uint32_t mask, int lane, int want, const L* row,
                                          const float* bias, int E, int32_t* ids) {
  const uint32_t below = (1u << (threadIdx.x & 31)) - 1u;
  uint64_t key[NV];
#pragma unroll 1
  for (int j = 0; j < NV; ++j) {
    const int e = lane * NV + j;
    key[j] = 0;
    if (e >= E) continue;
    bool ignored = false;
    const float x = logit_or_mask(to_float(row[e]), &ignored);
    if constexpr (BIAS) {
      const float b = logit_or_mask(bias[e], &ignored);
      if (x > -INFINITY && b > -INFINITY)
        key[j] = key_of(double_score<BIAS>(x, b));
    } else {
      if (x > -INFINITY) key[j] = key_of(double_score<BIAS>(x, 0.f));
    }
  }
  for (int s = 0; s < want; ++s) {
    uint64_t best = 0;
    int at = 0;
#pragma unroll 1
    for (int j = 0; j < NV; ++j)
      if (key[j] > best) {
        best = key[j];
        at = j;
      }
    const uint64_t top = group_max<G>(mask, best);
    if (top == 0) return s;
    const uint32_t holders = __ballot_sync(mask, best == top);
    if (best == top && (holders & below) == 0) {
      key[at] = 0;
      ids[s] = lane * NV + at;
    }
  }
  return want;
}

// Sorted keys of a lane's bf16 logits, made two at a time, and the logits in fp32. NaN and +inf
// have the largest keys (with their sign set the smallest), so the first and the last of the
// sorted show whether a lane has any.
constexpr uint32_t KEY_INF = 0xff800000u;     // of +inf
constexpr uint32_t KEY_MASKED = 0x007f0000u;  // of -inf

template <int NV>
__device__ __forceinline__ void bf16_keys(uint32_t mask, int first, const __nv_bfloat16* row,
                                          int E, bool wide, uint32_t (&key)[NV], float (&x)[NV],
                                          bool* bad) {
  uint32_t w[NV / 2];  // two logits each
#pragma unroll
  for (int j = 0; j < NV / 2; j += 4) {
    if ((NV * 2) % 16 == 0 && wide && first + 2 * j < E) {
      const uint4 v = *reinterpret_cast<const uint4*>(row + first + 2 * j);
      w[j] = v.x, w[j + 1] = v.y, w[j + 2] = v.z, w[j + 3] = v.w;
    } else {
      const unsigned short* bits = reinterpret_cast<const unsigned short*>(row);
#pragma unroll
      for (int i = j; i < j + 4 && i < NV / 2; ++i) {
        const int e = first + 2 * i;
        w[i] = (e < E ? bits[e] : 0xff80u) | (uint32_t)(e + 1 < E ? bits[e + 1] : 0xff80u) << 16;
      }
    }
  }
  const __nv_bfloat162 zero = __floats2bfloat162_rn(0.f, 0.f);
#pragma unroll
  for (int i = 0; i < NV / 2; ++i) {
    // + 0 turns -0 into +0; a negative number's 16 bits are complemented, a positive one's top
    // bit is set
    const __nv_bfloat162 h = __hadd2(*reinterpret_cast<const __nv_bfloat162*>(&w[i]), zero);
    const uint32_t u = *reinterpret_cast<const uint32_t*>(&h);
    const uint32_t k = u ^ (((u >> 15) & 0x00010001u) * 0xffffu | 0x80008000u);
    const uint32_t number = NUMBER - (first + 2 * i);
    key[2 * i] = (k << 16) | number;
    key[2 * i + 1] = (k & 0xffff0000u) | (number - 1);
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
#pragma unroll 1
  for (int again = 0;; ++again) {
    sort_keys(key);
    const bool odd = key[0] >= KEY_INF || key[NV - 1] < KEY_MASKED;
    if (again || !__any_sync(mask, odd)) break;  // almost always
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if (key[j] >= KEY_INF) key[j] = 0;
      x[j] = logit_or_mask(x[j], bad);
    }
  }
}

template <int G>
__device__ __forceinline__ uint32_t group_mask() {
  return G == 32 ? ALL : ((1u << (G & 31)) - 1u) << ((threadIdx.x & 31) / G * G);
}

// Choice by the logit itself without a bias (both scores grow with it, so the choice is
// exact), by sigma(x) + bias in double precision with one: neighbours of 256 scores are often
// closer than fp32 tells apart. fp32 logits and fp32 scores are looked up a few places further
// than needed, which leaves three cases: each two neighbours are in order for sure (values apart,
// or equal logits under equal biases, a tie in any precision); some are not, but nothing behind
// the last one can belong to the first k: those looked up are put in order by doubles; or the
// k-th and the last are too close for that: all experts are looked through again by doubles.
template <typename L, int G, int NV, bool BIAS>
__global__ void __launch_bounds__(THREADS) gate_kernel(Params p, bool sigmoid, bool renorm,
                                                       bool wide, bool wide_bias) {
  after_previous();
  constexpr bool EXACT = !BIAS && sizeof(L) == 2;  // the keys hold the whole value
  constexpr int SLOTS = GG_GATE_MAX_K + (EXACT ? 0 : MORE);
  __shared__ Chosen<SLOTS> chosen[THREADS / G];
  __shared__ double doubles[EXACT ? 1 : THREADS / G][EXACT ? 1 : SLOTS];
  const int lane = threadIdx.x % G;
  const int64_t t = (int64_t)blockIdx.x * (THREADS / G) + threadIdx.x / G;
  if (t >= p.T) return;  // the whole group
  const uint32_t mask = group_mask<G>();
  Chosen<SLOTS>& c = chosen[threadIdx.x / G];
  const L* row = static_cast<const L*>(p.logits) + t * p.E;
  bool bad_count = false, bad = false;
  int64_t live_tokens = p.T;
  if (p.num_tokens != nullptr) {
    live_tokens = *p.num_tokens;
    bad_count = live_tokens < 0 || live_tokens > p.T;
  }
  float x[NV];
  int got = 0;
  if (t < live_tokens) {
    uint32_t key[NV];
    const int most = EXACT ? p.k : min(p.k + MORE, p.E);
    bool open = false;
    if constexpr (EXACT) {
      bf16_keys<NV>(mask, lane * NV, row, p.E, wide, key, x, &bad);
    } else {
      load_row<NV>(row, lane * NV, p.E, wide, x);
      if constexpr (BIAS) {
        float b[NV];
        load_row<NV>(p.bias, lane * NV, p.E, wide_bias, b);
        // a bias of -inf makes the score and so a key that cannot be chosen
        bool odd = false;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
          odd |= !(x[j] < INFINITY);
          const uint32_t u = packed_score(fast_score(x[j], b[j]), lane * NV + j);
          key[j] = x[j] == -INFINITY ? 0u : u;
          odd |= key[j] >= KEY_INF;
        }
        if (odd) {  // almost never
#pragma unroll
          for (int j = 0; j < NV; ++j) {
            const bool in = fabsf(x[j]) < INFINITY;
            bad |= !(x[j] < INFINITY) || (in && !(b[j] < INFINITY));
            if (!in || !(b[j] < INFINITY)) key[j] = 0;
          }
        }
      } else {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
          const bool in = fabsf(x[j]) < INFINITY;
          bad |= !(x[j] < INFINITY);
          key[j] = in ? packed(x[j], lane * NV + j) : 0u;
          x[j] = in ? x[j] : -INFINITY;
        }
      }
      sort_keys(key);
    }
    constexpr Order ORDER = EXACT ? Order::WHOLE : BIAS ? Order::SCORES : Order::LOGITS;
    if (NV > 8 && most <= 8) got = choose<G, 8, ORDER>(mask, lane, p.k, most, key, c, &open);
    else got = choose<G, NV, ORDER>(mask, lane, p.k, most, key, c, &open);
    open = open && most < p.E;  // the same for the group
    __syncwarp(mask);
#pragma unroll 1
    for (int s = lane; s < got; s += G) {
      const uint32_t k = (uint32_t)c.id[s];
      const int id = expert_of(k);
      c.id[s] = id;
      if constexpr (EXACT)  // the key's value again
        c.x[s] = value_of((k & 0xffff0000u) | ((k >> 31) ? 0u : 0xffffu));
      else c.x[s] = to_float(row[id]);
      if constexpr (BIAS) {
        c.bias[s] = p.bias[id];
        c.score[s] = fast_score(c.x[s], c.bias[s]);
      }
    }
    if constexpr (!EXACT) {
      __syncwarp(mask);
      bool close = false;
#pragma unroll 1
      for (int s = lane; s + 1 < got; s += G) {
        const float x0 = c.x[s], x1 = c.x[s + 1];
        if constexpr (BIAS) {
          const float b0 = c.bias[s], b1 = c.bias[s + 1];
          close |= c.score[s] - c.score[s + 1] <= CLOSE * (1.f + fabsf(b0) + fabsf(b1)) &&
                   !(x0 == x1 && b0 == b1);
        } else {
          close |= !(x0 > x1 || (x0 == x1 && c.id[s] < c.id[s + 1]));
        }
      }
      if (open) {
        got = choose_double<L, G, NV, BIAS>(mask, lane, p.k, row, p.bias, p.E, c.id);
        __syncwarp(mask);
        for (int s = lane; s < got; s += G) c.x[s] = to_float(row[c.id[s]]);
      } else if (__any_sync(mask, close)) {
        order_double<G, BIAS>(mask, lane, got, p.bias, c, doubles[threadIdx.x / G]);
      }
      got = min(got, p.k);
    }
    __syncwarp(mask);
  }
  // shares: each score over the sum of the chosen (renorm) or of all (softmax)
  const bool sig = BIAS || sigmoid;  // a biased gate is a sigmoid
  float m = 0.f, total = 1.f;
  if (got > 0 && (renorm || !sig)) {
    if (!sig) m = c.x[0];  // the largest
    for (bool again = false;; again = true) {
      total = 0.f;
      if (renorm) {
#pragma unroll 1
        for (int s = lane; s < got; s += G) {
          float v;
          if (sig) v = again ? sigmoid_over(c.x[s], m) : gate::sigmoid(c.x[s]);
          else v = expf(c.x[s] - m);
          c.score[s] = v;
          total += v;
        }
      } else if constexpr (!BIAS) {
#pragma unroll
        for (int j = 0; j < NV; ++j) total += fast_exp(x[j] - m);
      }
      total = group_sum<G>(mask, total);
      if (again || !sig || total >= PLAIN) break;
      m = -INFINITY;
#pragma unroll 1
      for (int s = lane; s < got; s += G) m = fmaxf(m, c.x[s]);
      m = fminf(group_max<G>(mask, m), 0.f);
    }
  }
#pragma unroll 1
  for (int s = lane; s < p.k; s += G) {
    float w = 0.f;
    if (s < got) {
      if (renorm) w = c.score[s];
      else w = sig ? gate::sigmoid(c.x[s]) : expf(c.x[s] - m);
      w = p.scale * (w / total);  // a true quotient: the share of an only slot is 1
    }
    p.ids[t * p.k + s] = s < got ? c.id[s] : -1;
    p.weights[t * p.k + s] = w;
  }
  if (bad) flag(p.status, GG_DEV_BAD_LOGIT);
  if (bad_count && t == 0 && lane == 0) flag(p.status, GG_DEV_BAD_COUNT);
}

// Gradient of the logits. With v the weights before `scale` and g = scale * dweights (scaled
// last: differences of dweights are exact):
//   softmax over all      dx_j = p_j (g_j - sum_i g_i p_i)   (g_j = 0 for the others)
//   softmax renormalised  dx_i = v_i (g_i - sum g v)
//   sigmoid               dx_i = g_i s_i (1 - s_i)
//   sigmoid renormalised  dx_i = v_i (1 - s_i) (g_i - sum g v)
// The scores are computed again from the logits; dx of a logit that was not chosen is 0 but for
// the first form, which has a kernel of its own. A slot of id -1 carries nothing; slots of the
// same expert (such ids do not come from gate_topk) add up in their order. What bounds both
// kernels is the chain of their steps: a GPU full of tokens is one wave.
struct Slots {  // of one token, in shared memory
  int32_t id[GG_GATE_MAX_K];
  float g[GG_GATE_MAX_K];
};

// Softmax over all experts. A row in shared memory brings the slots to their experts' lanes.
template <typename L, int G, int NV>
__global__ void __launch_bounds__(THREADS) gate_backward_kernel(Params p, bool wide) {
  after_previous();
  __shared__ Slots slots[THREADS / G];
  // four experts of every lane side by side, then the next four: lanes' vectors are neighbours;
  // 16 floats more put the rows of two 4-lane groups into different banks
  __shared__ __align__(16) float rows[THREADS / G][G * NV + 16];
  const int lane = threadIdx.x % G;
  const int64_t t = (int64_t)blockIdx.x * (THREADS / G) + threadIdx.x / G;
  if (t >= p.T) return;  // the whole group
  const uint32_t mask = group_mask<G>();
  Slots& c = slots[threadIdx.x / G];  // each lane reads only its own
  float* d = rows[threadIdx.x / G];
  float x[NV];
  load_row<NV>(static_cast<const L*>(p.logits) + t * p.E, lane * NV, p.E, wide, x);
#pragma unroll
  for (int j = 0; j < NV / 4; ++j)
    *reinterpret_cast<float4*>(d + (j * G + lane) * 4) = make_float4(0.f, 0.f, 0.f, 0.f);
  bool bad = false;
#pragma unroll 1
  for (int s = lane; s < p.k; s += G) {
    int32_t id = p.ids[t * p.k + s];
    float g = p.dweights[t * p.k + s];
    bad |= id >= p.E;
    if (id < 0 || id >= p.E) id = -1, g = 0.f;
    c.id[s] = id;
    c.g[s] = g;
  }
  __syncwarp(mask);
  for (int s0 = 0; s0 < p.k; s0 += G) {
    const int s = s0 + lane, n = min(p.k - s0, G);
    const int32_t id = s < p.k ? c.id[s] : -1;
    const float v = s < p.k ? c.g[s] : 0.f;
    // expert id is place i of lane id / NV
    const int i = id % NV;
    float* place = d + ((i / 4) * G + id / NV) * 4 + i % 4;
    bool again = false;  // an earlier slot has the same expert
    for (int q = 0; q + 1 < n; ++q) {
      const int32_t other = __shfl_sync(mask, id, q, G);
      again |= q < lane && other == id;
    }
    again = again && id >= 0;
    if (id >= 0 && !again) *place += v;
    if (__any_sync(mask, again)) {  // such ids do not come from gate_topk
      for (int q = 1; q < n; ++q) {
        __syncwarp(mask);
        if (q == lane && again) *place += v;
      }
    }
    __syncwarp(mask);
  }
  float out[NV];
#pragma unroll
  for (int j = 0; j < NV / 4; ++j) {
    const float4 v = *reinterpret_cast<const float4*>(d + (j * G + lane) * 4);
    out[4 * j] = v.x, out[4 * j + 1] = v.y, out[4 * j + 2] = v.z, out[4 * j + 3] = v.w;
  }
  bool ignored = false;
  float top = -INFINITY, total = 0.f, mean = 0.f;
#pragma unroll
  for (int j = 0; j < NV; ++j) top = fmaxf(top, x[j] = logit_or_mask(x[j], &ignored));
  top = fmaxf(group_max<G>(mask, top), -FLT_MAX);  // all of them masked: every share is 0
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    x[j] = fast_exp(x[j] - top);
    total += x[j];
    mean = fmaf(x[j], out[j], mean);
  }
  // the total is 1 or more unless all of them are masked
  const float inv = __fdividef(1.f, fmaxf(group_sum<G>(mask, total), 0.5f));
  mean = group_sum<G>(mask, mean) * inv;
  // Gains of the probable experts that hardly differ (one expert with nearly all of it) cancel
  // against the mean: the mean of what is left takes its rounding off (32768 x 64 bf16 6.2 us for
  // 6.05, 16411 x 256 fp32 7.3 for 6.95).
  float2 pairs = both(0.f);
#pragma unroll
  for (int j = 0; j < NV; j += 2) {
    const float2 d = __fadd2_rn(make_float2(out[j], out[j + 1]), both(-mean));
    pairs = __ffma2_rn(make_float2(x[j], x[j + 1]), d, pairs);
    out[j] = d.x, out[j + 1] = d.y;
  }
  float rest = group_sum<G>(mask, pairs.x + pairs.y) * inv;
  if (rest != rest) rest = 0.f;  // an infinite gain: the plain formula's values
  const float2 share = both(p.scale * inv);
#pragma unroll
  for (int j = 0; j < NV; j += 2) {
    const float2 d = __fadd2_rn(make_float2(out[j], out[j + 1]), both(-rest));
    const float2 dx = __fmul2_rn(__fmul2_rn(make_float2(x[j], x[j + 1]), share), d);
    out[j] = dx.x, out[j + 1] = dx.y;
  }
  store_row<NV>(static_cast<L*>(p.dlogits) + t * p.E, lane * NV, p.E, wide, out);
  if (bad) flag(p.status, GG_DEV_BAD_ROUTE);
}

// The other forms, a lane for each slot (k <= G): zeros first, so that they are on their way to
// memory while the chosen are computed, then those over them. (16411 x 256 fp32, top 6, and
// 131072 x 64 bf16, top 8: 5.0 and 14.4 us, 9.0 and 34 through a row in shared memory as above.)
template <typename L, int G>
__global__ void __launch_bounds__(THREADS) gate_backward_chosen_kernel(Params p, bool sig,
                                                                       bool renorm, bool wide) {
  after_previous();
  const int lane = threadIdx.x % G;
  const int64_t t = (int64_t)blockIdx.x * (THREADS / G) + threadIdx.x / G;
  if (t >= p.T) return;  // the whole group
  const uint32_t mask = group_mask<G>();
  int32_t id = -1;
  float g = 0.f;
  if (lane < p.k) {
    id = p.ids[t * p.k + lane];
    g = p.dweights[t * p.k + lane];
  }
  L* out = static_cast<L*>(p.dlogits) + t * p.E;
  if (wide) {
    constexpr int VEC = 16 / sizeof(L);
    for (int j = lane * VEC; j < p.E; j += G * VEC)
      *reinterpret_cast<uint4*>(out + j) = make_uint4(0, 0, 0, 0);
  } else {
    for (int j = lane; j < p.E; j += G) store(out + j, 0.f);
  }
  if (id >= p.E) {
    flag(p.status, GG_DEV_BAD_ROUTE);
    id = -1;
  }
  float x = -INFINITY;
  bool ignored = false;
  if (id >= 0)
    x = logit_or_mask(to_float(static_cast<const L*>(p.logits)[t * p.E + id]), &ignored);
  const bool live = x > -INFINITY;
  if (!live) id = -1;
  g = live ? g : 0.f;
  float v, mean = 0.f;
  if (renorm) {
    const float m = group_max<G>(mask, sig ? fminf(x, 0.f) : x);
    v = !live ? 0.f : sig ? sigmoid_over(x, m) : expf(x - m);
    const float total = group_sum<G>(mask, v);
    v = live ? v / total : 0.f;  // a true quotient: the share of an only slot is 1, its gradient 0
    mean = group_sum<G>(mask, g * v);
    // The mean of what is left takes the first mean's rounding off: gains that hardly differ
    // keep their differences, whatever the shares.
    g -= mean;
    mean = group_sum<G>(mask, live ? g * v : 0.f);
    if (mean != mean) mean = 0.f;  // an infinite gain: the plain formula's values
  } else {
    v = sigmoid(x);
  }
  if (sig) v *= sigmoid(-x);  // 1 - sigma(x) = sigma(-x)
  float dx = p.scale * (v * (g - mean));  // scaled last: differences of dweights are exact
  bool again = false;  // an earlier slot has the same expert
  for (int q = 0; q + 1 < p.k; ++q) {
    const int32_t other = __shfl_sync(mask, id, q, G);
    again |= q < lane && other == id;
  }
  again = again && live;
  if (__any_sync(mask, again)) {  // the first of them takes the others' in their order
    float sum = dx;
    for (int q = 1; q < p.k; ++q) {
      const int32_t other = __shfl_sync(mask, id, q, G);
      const float more = __shfl_sync(mask, dx, q, G);
      if (q > lane && other == id) sum += more;
    }
    dx = sum;
  }
  __syncwarp(mask);  // the zeros come before
  if (live && !again) store(out + id, dx);
}

template <int N> using Int = std::integral_constant<int, N>;

// Lanes a token and experts a lane: NV, or MORE (half as much again, or three times that) where
// it wastes less. A warp for each token is the quickest for few of them, several tokens a warp the
// cheapest in instructions for many. (32768 tokens of 160 and of 384 experts, top 6 and 8, bf16:
// 12.3 and 21.9 us, 18.4 and 34.6 without MORE.)
template <int NV, int MORE, int LEAST, typename F>
void by_experts(int E, bool few, const F& f) {
  if (few && E <= 32 * LEAST) f(Int<32>(), Int<LEAST>());
  else if (few && E <= 128) f(Int<32>(), Int<4>());
  else if (few && E <= 256) f(Int<32>(), Int<8>());
  else if (E <= 64) f(Int<64 / NV>(), Int<NV>());
  else if (E <= 96) f(Int<96 / MORE>(), Int<MORE>());
  else if (E <= 128) f(Int<128 / NV>(), Int<NV>());
  else if (E <= 192) f(Int<192 / MORE>(), Int<MORE>());
  else if (E <= 256) f(Int<256 / NV>(), Int<NV>());
  else if (E <= 384) f(Int<384 / MORE>(), Int<MORE>());
  else if (E <= 512) f(Int<32>(), Int<16>());
  else if (E <= 768) f(Int<32>(), Int<24>());
  else f(Int<32>(), Int<32>());
}

// 1 x 64 bf16: 1.8 us a call in a graph with a warp a token, 2.6 us with four lanes; 4096 x 64:
// 2.7 and 3.5, 8192 x 64: 4.1 and 3.8, 32768 x 64: 12.6 and 6.7. Backward from all experts
// 512 x 64: 1.8 and with eight lanes 2.5, 4096 x 64 2.5 and 2.7, 8192 x 64 3.7 and 3.0.
constexpr int64_t FEW = 4096;

template <typename L, bool BIAS>
gg_status launch_gate(const Params& p, bool sigmoid, bool renorm, cudaStream_t stream) {
  gg_status s = GG_OK;
  const bool wide = p.E % 8 == 0 && !misaligned(p.logits, 16);
  const bool wide_bias = p.E % 8 == 0 && !misaligned(p.bias, 16);
  const auto go = [&](auto g, auto nv) {
    constexpr int G = decltype(g)::value, NV = decltype(nv)::value, PER = THREADS / G;
    s = launch("gg_gate_topk", gate_kernel<L, G, NV, BIAS>, (unsigned)((p.T + PER - 1) / PER),
               THREADS, stream, p, sigmoid, renorm, wide, wide_bias);
  };
  // eight experts a lane where that fills the GPU better, sixteen and so more tokens a warp for
  // many (bf16 16411 x 64: 4.4 and 4.8 us, 32768 x 64: 7.5 and 6.7; fp32 with a bias 8192 x 256:
  // 8.5 and 9.0, 16411 x 256 14.3 both, 32768 x 256: 25.7 and 23.8)
  constexpr int64_t MANY = sizeof(L) == 2 ? 1 << 21 : 1 << 22;
  if (p.T * p.E < MANY) by_experts<8, 12, 2>(p.E, p.T <= FEW, go);
  else by_experts<16, 24, 2>(p.E, p.T <= FEW, go);
  return s;
}

template <typename L>
gg_status launch_backward(const Params& p, bool sigmoid, bool renorm, cudaStream_t stream) {
  gg_status s = GG_OK;
  if (sigmoid || renorm) {
    const bool wide = p.E * sizeof(L) % 16 == 0 && !misaligned(p.dlogits, 16);
    const auto go = [&](auto g) {
      constexpr int G = decltype(g)::value, PER = THREADS / G;
      return launch("gg_gate_topk_backward", gate_backward_chosen_kernel<L, G>,
                    (unsigned)((p.T + PER - 1) / PER), THREADS, stream, p, sigmoid, renorm, wide);
    };
    // a warp writes few tokens' long rows sooner (512 x 1000 bf16: 2.3 us, 3.1 with eight lanes;
    // 4096 x 1000 4.3 and 4.2, 512 x 64 2.5 and 2.3)
    if (p.k > 16 || (p.T <= 1024 && p.E * sizeof(L) > 1024)) return go(Int<32>());
    return p.k <= 8 ? go(Int<8>()) : go(Int<16>());
  }
  const bool wide = p.E % 8 == 0 && !misaligned(p.logits, 16) && !misaligned(p.dlogits, 16);
  // eight experts a lane: 32768 x 64 bf16 6.2 us, 16411 x 256 fp32 7.3, with sixteen 6.5 and 8.9;
  // twelve are no whole vectors of bf16 (32768 x 160: 15.9 us, 9.7 with 24)
  by_experts<8, 24, 4>(p.E, p.T <= FEW, [&](auto g, auto nv) {
    constexpr int G = decltype(g)::value, NV = decltype(nv)::value, PER = THREADS / G;
    s = launch("gg_gate_topk_backward", gate_backward_kernel<L, G, NV>,
               (unsigned)((p.T + PER - 1) / PER), THREADS, stream, p, wide);
  });
  return s;
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
  if (f32)
    return bias != nullptr ? launch_gate<float, true>(p, sig, renorm, stream)
                           : launch_gate<float, false>(p, sig, renorm, stream);
  return bias != nullptr ? launch_gate<__nv_bfloat16, true>(p, sig, renorm, stream)
                         : launch_gate<__nv_bfloat16, false>(p, sig, renorm, stream);
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
  // zeros are written before the chosen experts' logits are read
  if (overlap(logits, dlogits, T * E * (f32 ? 4 : 2))) return GG_ERR_INVALID_ARG;
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
  return f32 ? launch_backward<float>(p, sig, renorm, stream)
             : launch_backward<__nv_bfloat16>(p, sig, renorm, stream);
}

}  // extern "C"
