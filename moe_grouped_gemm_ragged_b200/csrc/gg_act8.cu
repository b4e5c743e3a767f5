// Between the two expert products: SiLU-and-mul of packed rows, which can keep its input in
// the 8-bit row form, and the backward pass that starts from that form (or from the bf16
// input). And the form itself: packed rows to 8 bits and back.
#include <cstdint>
#include <type_traits>

#include "gg_ops.cuh"

namespace gg {
namespace act8 {

using namespace gg::ops;

constexpr int THREADS = 256;
constexpr int WARPS = THREADS / 32;
constexpr uint32_t ALL = 0xffffffffu;
// Pieces of 32 vectors that a warp takes at once. 64 registers a thread (four blocks an SM) hold
// four of them; the backward pass, with twice the values a piece, two. us for 65536 rows of
// 4096 columns, forward and backward with the 8 bits: 169 and 266 with four, 177 and 213 with two
// (the bytes at the copy rate: 168 and 209); without them 119 and 332, 123 and 250 (125 and 250);
// 262144 x 6144 to 8 bits and back: 729 and 737 with four, 791 and 752 with two (757 each).
constexpr int BLOCKS = 4;
constexpr int MANY = 4, MANY_BACKWARD = 2;

struct Params {
  const uint4* H;           // [rows, N] bf16
  const uint2* H8;          // [rows, N] e4m3
  const uint8_t* H8_scale;  // [rows, 2 ceil(I / 32)] codes
  uint2* H8_out;
  uint8_t* scale_out;
  const uint4* dact;        // [rows, I]
  uint4* act;               // [rows, I]
  uint4* dH;                // [rows, N]
  const int32_t* row_of;
  const float* weights;
  float* dweights;
  const int32_t* used;
  int32_t* status;
  int64_t rows;
  int64_t n;                // assignments (with row_of) or rows
  int64_t tail0;            // first block that only clears rows
  int32_t half;             // I = N / 2
  int32_t concat;
  int32_t zero_tail;
};

// sigma(x) = 1 / (1 + 2^(-x log2 e)) of a pair, by the hardware's powers and reciprocals. In units
// of 2^-23 the power is off by 2 + 0.62 |x| (its own error; its argument's two roundings), the sum
// by 0.5, the reciprocal by 1: 3.5 + 0.62 |x| at most, against half a step of 2^-8 in the bf16
// results.
// Below 2^-126 (x < -87.3) it is 0: such gates are done over (FAR).
__device__ __forceinline__ float2 sigmoid(const float2& x) {
  float2 t = __fmul2_rn(x, both(-1.44269504f));
  asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(t.x));
  asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(t.y));
  t = __fadd2_rn(t, both(1.f));
  asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(t.x));
  asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(t.y));
  return t;
}

// One pair of each direction. h = [g, u] from its 8 bits (or bf16), s the row's weight, q =
// sigma(g):
//   dg = s dact u (q + g q (1 - q)),  du = s dact g q,  act = s g q u,  ds = <dact, g q u>
__device__ __forceinline__ float2 silu_times(const float2& g, const float2& u) {
  return __fmul2_rn(__fmul2_rn(g, sigmoid(g)), u);
}
struct Gradient {
  float2 su, dg, du;  // g q u without the weight, and the two gradients
};
__device__ __forceinline__ Gradient gradient(const float2& g, const float2& u, const float2& sd) {
  const float2 q = sigmoid(g), silu = __fmul2_rn(g, q);
  // 1 - q first, as silu can be past 2^24, where q has no part in their sum
  const float2 slope = __ffma2_rn(silu, __ffma2_rn(both(-1.f), q, both(1.f)), q);
  return {__fmul2_rn(silu, u), __fmul2_rn(__fmul2_rn(sd, u), slope), __fmul2_rn(sd, silu)};
}

// Gates under -87: fp32 holds their sigma (then e^g to the last bit) badly or not at all, while
// bf16 holds g sigma(g) u down to 2^-133. Their products are made with the fourth root of e^g, one
// factor after the other. A vector that has one is told by its bits, one that may by its code.
constexpr float FAR = -87.f;
constexpr uint32_t FAR_BITS = 0xc2af0000u;  // -87.5, the next bf16, in the upper half of a word
constexpr uint32_t FAR_CODE = 125;          // the least with which a block can hold 87: 448 / 4

__device__ __forceinline__ bool any_far(const uint4& v) {  // of eight bf16: -87.5 or further down
  const uint32_t m = __vmaxu2(__vmaxu2(v.x, v.y), __vmaxu2(v.z, v.w));
  return m >= FAR_BITS || (m << 16) >= FAR_BITS;
}
__device__ __forceinline__ float fourth_root(float g) {  // of e^g
  float t = g * 0.36067376f;
  asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(t));
  return t;
}
__device__ __forceinline__ void silu_times_far(float g, float u, float& su) {
  if (!(g < FAR)) return;
  const float e = fourth_root(g);
  su = g * e * u * e * e * e;
}
__device__ __forceinline__ void gradient_far(float g, float u, float sd, float& su, float& dg,
                                             float& du) {
  if (!(g < FAR)) return;
  const float e = fourth_root(g);
  su = g * e * u * e * e * e;
  dg = sd * u * e * (1.f + g) * e * e * e;
  du = g * e * sd * e * e * e;
}

// A row belongs to G lanes of a warp (W 1), or to all W warps of a block (G 32). They take its
// pieces of G vectors in turn, U pieces at once: their loads are in flight together.
template <int G, int W>
__device__ __forceinline__ int64_t my_item() {
  return W == 1 ? (int64_t)blockIdx.x * (THREADS / G) + threadIdx.x / G : blockIdx.x;
}
template <int G, int W, int U>
__device__ __forceinline__ int first_vec() {
  return (W == 1 ? 0 : (threadIdx.x >> 5) * U * G) + threadIdx.x % G;
}
// The lanes that work on the row together, and the first thread of the row's.
template <int G>
__device__ __forceinline__ uint32_t row_mask() {
  return G == 32 ? ALL : ((1u << (G & 31)) - 1u) << ((threadIdx.x & 31) / G * G);
}
template <int G, int W>
__device__ __forceinline__ bool leader() {
  return threadIdx.x % (G * W) == 0;
}

// Packed row of item b (an assignment, or a row), -1 for a dropped assignment. Without row_of the
// row may not be in use; as it is allocated, it can be loaded from while *used is still on its
// way, and what was loaded is then left.
__device__ __forceinline__ int64_t row_of_item(const Params& p, int64_t b, int64_t used,
                                               bool report) {
  if (p.row_of == nullptr) return b;
  const int64_t r = p.row_of[b];
  if (r >= used && report) flag(p.status, GG_DEV_BAD_ROUTE);
  return r >= used ? -1 : r;
}

// The blocks from tail0 on clear the rows of `out` (vecs vectors each) that are not in use.
__device__ __forceinline__ void clear_tail(const Params& p, int64_t used, uint4* out, int vecs) {
  const int64_t warps = (int64_t)(gridDim.x - p.tail0) * WARPS;
  for (int64_t r = used + (blockIdx.x - p.tail0) * WARPS + (threadIdx.x >> 5); r < p.rows;
       r += warps)
    for (int c = threadIdx.x & 31; c < vecs; c += 32) out[r * vecs + c] = make_uint4(0, 0, 0, 0);
}

// Vector index of gate columns [8 c, 8 c + 8) in a row of H, and of the up columns beside
// them; the same for the codes of their blocks.
__device__ __forceinline__ int64_t gate_vec(const Params& p, int c) {
  return p.concat ? c : (c >> 4) * 32 + (c & 15);
}
__device__ __forceinline__ int64_t up_vec(const Params& p, int c) {
  return p.concat ? c + p.half / 8 : gate_vec(p, c) + 16;
}
__device__ __forceinline__ int64_t gate_code(const Params& p, int c) {
  return p.concat ? c >> 2 : (c >> 4) * 8 + ((c >> 2) & 3);
}
__device__ __forceinline__ int64_t up_code(const Params& p, int c) {
  return p.concat ? (c >> 2) + (p.half + kBlock - 1) / kBlock : gate_code(p, c) + 4;
}

// A thread's vectors with far gates, done over when the rest is done. (Beside the rest, as in the
// backward pass, it takes registers that the 8 bits need: 65536 x 4096 231 us, 169 like this. The
// backward pass may have written dH or act over its inputs by then; beside the rest it takes 46.8
// and 50.0 us for 32768 x 1536 from 8 bits and from bf16, 45.6 and 48.6 without it. With far gates
// in every vector it is 53 and 56, forward with the 8 bits 63 instead of 35.)
__device__ __noinline__ void silu_mul_far(const uint4* H, uint4* act, int32_t concat, int vecs,
                                          int c, int step, float scale) {
  for (; c < vecs; c += step) {
    const int64_t at = concat ? c : (c >> 4) * 32 + (c & 15);
    const uint4 gv = H[at];
    if (!any_far(gv)) continue;
    float2 g[4], u[4];
    unpack_bf16(gv, g);
    unpack_bf16(H[at + (concat ? vecs : 16)], u);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float2 a = silu_times(g[j], u[j]);
      silu_times_far(g[j].x, u[j].x, a.x);
      silu_times_far(g[j].y, u[j].y, a.y);
      g[j] = __fmul2_rn(a, both(scale));
    }
    act[c] = pack_bf16(g);
  }
}

template <int G, int W, int U, bool CKPT>
__global__ void __launch_bounds__(THREADS, BLOCKS) silu_mul_kernel(Params p) {
  after_previous();
  const int vecs = p.half / 8;
  const int64_t used =
      rows_in_use(p.used, p.rows, p.status, blockIdx.x == 0 && threadIdx.x == 0);
  if (blockIdx.x >= p.tail0) {
    clear_tail(p, used, p.act, vecs);
    return;
  }
  const int64_t item = my_item<G, W>();
  if (item >= p.n) return;
  const float scale = p.weights != nullptr ? p.weights[item] : 1.f;  // on its way with the row
  const int64_t row = row_of_item(p, item, used, leader<G, W>());
  if (row < 0) return;
  const int64_t base = row * 2 * vecs;
  const int64_t code0 = row * 2 * ((p.half + kBlock - 1) / kBlock);
  bool far = false;
  // a row's lanes go round together: the four lanes of a block exchange their largest values
  for (int c0 = first_vec<G, W, U>(); c0 - (int)(threadIdx.x % G) < vecs; c0 += W * U * G) {
    uint4 gv[U], uv[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int c = c0 + G * i;
      gv[i] = uv[i] = make_uint4(0, 0, 0, 0);
      if (c < vecs) {
        gv[i] = __ldcs(p.H + base + gate_vec(p, c));
        uv[i] = __ldcs(p.H + base + up_vec(p, c));
      }
    }
    if (row >= used) return;  // the row's lanes together
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int c = c0 + G * i;
      if (c - (int)(threadIdx.x % G) >= vecs) break;  // the row's lanes together
      far |= any_far(gv[i]);
      float2 g[4], u[4];
      unpack_bf16(gv[i], g);
      unpack_bf16(uv[i], u);
      if constexpr (CKPT) {
        uint32_t cg, cu;
        bool odd;
        block_codes(row_mask<G>(), gv[i], uv[i], cg, cu, &odd);
        if (c < vecs) {
          p.H8_out[base + gate_vec(p, c)] = to_e4m3(g, cg, odd);
          p.H8_out[base + up_vec(p, c)] = to_e4m3(u, cu, odd);
          if ((c & 3) == 0) {
            p.scale_out[code0 + gate_code(p, c)] = (uint8_t)cg;
            p.scale_out[code0 + up_code(p, c)] = (uint8_t)cu;
          }
        }
      }
      if (c < vecs) {
#pragma unroll
        for (int j = 0; j < 4; ++j) g[j] = __fmul2_rn(silu_times(g[j], u[j]), both(scale));
        p.act[row * vecs + c] = pack_bf16(g);
      }
    }
  }
  if (far)
    silu_mul_far(p.H + base, p.act + row * vecs, p.concat, vecs, first_vec<G, W, U>(), W * G,
                 scale);
}

template <int G, int W, int U, bool FROM8>
__global__ void __launch_bounds__(THREADS, BLOCKS) silu_mul_backward_kernel(Params p) {
  after_previous();
  __shared__ float part[WARPS];
  const int vecs = p.half / 8;
  const int64_t used =
      rows_in_use(p.used, p.rows, p.status, blockIdx.x == 0 && threadIdx.x == 0);
  if (blockIdx.x >= p.tail0) {
    clear_tail(p, used, p.dH, 2 * vecs);
    if (p.act != nullptr) clear_tail(p, used, p.act, vecs);
    return;
  }
  const int64_t item = my_item<G, W>();
  if (item >= p.n) return;
  const float scale = p.weights != nullptr ? p.weights[item] : 1.f;  // on its way with the row
  const int64_t row = row_of_item(p, item, used, leader<G, W>());
  float2 dots = both(0.f);
  if (row >= 0) {
    const int64_t base = row * 2 * vecs;
    const int64_t code0 = row * 2 * ((p.half + kBlock - 1) / kBlock);
    for (int c0 = first_vec<G, W, U>(); c0 < vecs; c0 += W * U * G) {
      uint4 gv[U], uv[U], dv[U];
      uint2 g8[U], u8[U];
      uint8_t cg[U], cu[U];
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int c = c0 + G * i;
        if (c >= vecs) continue;
        if constexpr (FROM8) {
          g8[i] = __ldcs(p.H8 + base + gate_vec(p, c));
          u8[i] = __ldcs(p.H8 + base + up_vec(p, c));
          cg[i] = p.H8_scale[code0 + gate_code(p, c)];
          cu[i] = p.H8_scale[code0 + up_code(p, c)];
        } else {
          gv[i] = __ldcs(p.H + base + gate_vec(p, c));
          uv[i] = __ldcs(p.H + base + up_vec(p, c));
        }
        dv[i] = __ldcs(p.dact + row * vecs + c);
      }
      if (row >= used) return;  // the row's warps together
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int c = c0 + G * i;
        if (c >= vecs) continue;
        float2 g[4], u[4], d[4], a[4];
        bool far;
        if constexpr (FROM8) {
          from_e4m3(g8[i], code_scale(cg[i]), g);
          from_e4m3(u8[i], code_scale(cu[i]), u);
          far = cg[i] >= FAR_CODE;
        } else {
          unpack_bf16(gv[i], g);
          unpack_bf16(uv[i], u);
          far = any_far(gv[i]);
        }
        unpack_bf16(dv[i], d);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 sd = __fmul2_rn(d[j], both(scale));
          Gradient r = gradient(g[j], u[j], sd);
          if (far) {
            gradient_far(g[j].x, u[j].x, sd.x, r.su.x, r.dg.x, r.du.x);
            gradient_far(g[j].y, u[j].y, sd.y, r.su.y, r.dg.y, r.du.y);
          }
          dots = __ffma2_rn(d[j], r.su, dots);
          a[j] = __fmul2_rn(r.su, both(scale));
          g[j] = r.dg;
          u[j] = r.du;
        }
        p.dH[base + gate_vec(p, c)] = pack_bf16(g);
        p.dH[base + up_vec(p, c)] = pack_bf16(u);
        if (p.act != nullptr) p.act[row * vecs + c] = pack_bf16(a);
      }
    }
  }
  // A row that is not in use (only without row_of) keeps its weight's gradient. A warp whose
  // share of such a row is empty has not returned above; it may do so here, as all of its row's
  // warps are past their loops or gone, and none of them reaches the barrier below.
  if (p.dweights == nullptr || row >= used) return;
  float dot = dots.x + dots.y;
#pragma unroll
  for (int d = G / 2; d > 0; d >>= 1) dot += __shfl_xor_sync(row_mask<G>(), dot, d);
  if constexpr (W == 1) {
    if (leader<G, W>()) p.dweights[item] = dot;
  } else {
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = dot;
    __syncthreads();
    if (threadIdx.x == 0) {
      float sum = 0.f;
      for (int i = 0; i < WARPS; ++i) sum += part[i];
      p.dweights[item] = sum;
    }
  }
}

template <int G, int W, int U>
__global__ void __launch_bounds__(THREADS, BLOCKS) pack8_kernel(
    const uint4* X, uint2* X8, uint8_t* scale, int64_t rows, int32_t vecs, const int32_t* used,
    int32_t* status) {
  after_previous();
  const int64_t n = rows_in_use(used, rows, status, blockIdx.x == 0 && threadIdx.x == 0);
  const int64_t r = my_item<G, W>();
  if (r >= rows) return;
  const int64_t codes = (vecs + 3) / 4;
  for (int c0 = first_vec<G, W, U>(); c0 - (int)(threadIdx.x % G) < vecs; c0 += W * U * G) {
    uint4 v[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int c = c0 + G * i;
      v[i] = c < vecs ? __ldcs(X + r * vecs + c) : make_uint4(0, 0, 0, 0);
    }
    if (r >= n) return;
    constexpr int P = U > 1 ? 2 : 1;  // pieces whose codes are found together
#pragma unroll
    for (int i = 0; i < U; i += P) {
      if (c0 + G * i - (int)(threadIdx.x % G) >= vecs) break;  // the row's lanes together
      uint32_t code[2];
      bool odd;
      block_codes(row_mask<G>(), v[i], v[i + P - 1], code[0], code[P - 1], &odd);
#pragma unroll
      for (int k = 0; k < P; ++k) {
        const int c = c0 + G * (i + k);
        if (c >= vecs) continue;
        float2 x[4];
        unpack_bf16(v[i + k], x);
        X8[r * vecs + c] = to_e4m3(x, code[k], odd);
        if ((c & 3) == 0) scale[r * codes + (c >> 2)] = (uint8_t)code[k];
      }
    }
  }
}

template <int G, int W, int U>
__global__ void __launch_bounds__(THREADS, BLOCKS) unpack8_kernel(
    const uint2* X8, const uint8_t* scale, uint4* X, int64_t rows, int32_t vecs,
    const int32_t* used, int32_t zero_tail, int32_t* status) {
  after_previous();
  const int64_t n = rows_in_use(used, rows, status, blockIdx.x == 0 && threadIdx.x == 0);
  const int64_t r = my_item<G, W>();
  if (r >= rows) return;
  const int64_t codes = (vecs + 3) / 4;
  for (int c0 = first_vec<G, W, U>(); c0 < vecs; c0 += W * U * G) {
    uint2 q[U];
    uint8_t s[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int c = c0 + G * i;
      if (c >= vecs) continue;
      q[i] = __ldcs(X8 + r * vecs + c);
      s[i] = scale[r * codes + (c >> 2)];
    }
    if (r >= n && !zero_tail) return;
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int c = c0 + G * i;
      if (c >= vecs) continue;
      float2 x[4] = {};
      if (r < n) from_e4m3(q[i], code_scale(s[i]), x);
      X[r * vecs + c] = pack_bf16(x);
    }
  }
}

// All warps of a block share a row where there are few of them (more than one piece each, or
// there is nothing to share): a warp a row would leave most of the GPU idle. us a call in a
// graph, shared and not, forward with the 8 bits: 8 x 1536 1.8 and 2.9, 8 x 16384 3.9 and 18.4,
// 1001 x 4096 4.0 and 5.8; 2048 x 1536 5.3 and 3.8 (backward 1.8 and 3.4, 4.0 and 20.5, 4.7 and
// 6.5; 6.0 and 4.1).
bool share_row(int64_t items, int64_t vecs, int sms) {
  return vecs > 32 && items <= 8 * (int64_t)sms;
}

// Sizes and indices common to both directions of SiLU-and-mul.
gg_status check(int64_t rows, int64_t N, const int32_t* row_of, const float* weights,
                int64_t n_assign, const int32_t* rows_used, int32_t flags,
                const int32_t* dev_status) {
  if (rows < 0 || N < 1 || n_assign < 0) return GG_ERR_INVALID_ARG;
  if (flags & ~(GG_FLAG_ZERO_TAIL | GG_FLAG_GATE_UP_CONCAT)) return GG_ERR_INVALID_ARG;
  const bool zero = (flags & GG_FLAG_ZERO_TAIL) != 0;
  if (zero && rows_used == nullptr) return GG_ERR_INVALID_ARG;
  if (row_of == nullptr && n_assign != 0) return GG_ERR_INVALID_ARG;
  if (N % ((flags & GG_FLAG_GATE_UP_CONCAT) ? 16 : 256) != 0 || N >= (int64_t(1) << 31) ||
      rows >= (int64_t(1) << 30) || n_assign >= (int64_t(1) << 30))
    return GG_ERR_UNSUPPORTED;
  if (misaligned(row_of, 4) || misaligned(weights, 4) || misaligned(rows_used, 4) ||
      misaligned(dev_status, 4))
    return GG_ERR_UNSUPPORTED;
  return GG_OK;
}

Params params(int64_t rows, int64_t N, const int32_t* row_of, const float* weights,
              int64_t n_assign, const int32_t* rows_used, int32_t flags, int32_t* dev_status) {
  Params p = {};
  p.row_of = row_of;
  p.weights = weights;
  p.used = rows_used;
  p.status = dev_status;
  p.rows = rows;
  p.n = row_of != nullptr ? n_assign : rows;
  p.half = (int32_t)(N / 2);
  p.concat = (flags & GG_FLAG_GATE_UP_CONCAT) ? 1 : 0;
  p.zero_tail = (flags & GG_FLAG_ZERO_TAIL) ? 1 : 0;
  return p;
}

// Calls f with the lanes a row: as many as hold it in U pieces, four (the lanes of a block of 32
// columns) to a warp. 262144 rows of 64 columns to 8 bits take 12 us with four lanes, 56 with a
// warp; SiLU-and-mul of as many rows of 256 columns 55 with four lanes, 112 (backward 69 with
// eight, 135).
template <int N> using Int = std::integral_constant<int, N>;
template <int U, typename F>
void by_length(int64_t vecs, const F& f) {
  if (vecs <= 4 * U) f(Int<4>());
  else if (vecs <= 8 * U) f(Int<8>());
  else if (vecs <= 16 * U) f(Int<16>());
  else f(Int<32>());
}

// Blocks of the launch for `per` items a block; blocks for the tail where rows are cleared.
unsigned blocks_for(Params* p, int64_t per, int sms) {
  p->tail0 = (p->n + per - 1) / per;
  int64_t tail = 0;
  if (p->zero_tail && p->rows > 0) {
    tail = (p->rows + WARPS - 1) / WARPS;
    if (tail > 4 * sms) tail = 4 * sms;
  }
  return (unsigned)(p->tail0 + tail);
}

template <bool CKPT>
gg_status launch_forward(Params p, int sms, cudaStream_t stream) {
  gg_status s = GG_OK;
  const auto go = [&](auto kernel, int64_t per) {
    if (const unsigned grid = blocks_for(&p, per, sms))
      s = launch("gg_silu_mul", kernel, grid, THREADS, stream, p);
  };
  if (share_row(p.n, p.half / 8, sms)) {
    go(silu_mul_kernel<32, WARPS, 1, CKPT>, 1);
  } else {
    by_length<MANY>(p.half / 8, [&](auto g) {
      constexpr int G = decltype(g)::value;
      go(silu_mul_kernel<G, 1, MANY, CKPT>, THREADS / G);
    });
  }
  return s;
}

template <bool FROM8>
gg_status launch_backward(Params p, int sms, cudaStream_t stream) {
  gg_status s = GG_OK;
  const auto go = [&](auto kernel, int64_t per) {
    if (const unsigned grid = blocks_for(&p, per, sms))
      s = launch("gg_silu_mul_backward", kernel, grid, THREADS, stream, p);
  };
  if (share_row(p.n, p.half / 8, sms)) {
    go(silu_mul_backward_kernel<32, WARPS, 1, FROM8>, 1);
  } else {
    by_length<MANY_BACKWARD>(p.half / 8, [&](auto g) {
      constexpr int G = decltype(g)::value;
      go(silu_mul_backward_kernel<G, 1, MANY_BACKWARD, FROM8>, THREADS / G);
    });
  }
  return s;
}

gg_status check_rows8(const void* X, const void* X8, const void* scale, int64_t rows,
                      int64_t cols, const int32_t* rows_used, const int32_t* dev_status) {
  if (rows < 0 || cols < 1) return GG_ERR_INVALID_ARG;
  if (cols % 8 != 0 || cols >= (int64_t(1) << 31) || rows >= (int64_t(1) << 31))
    return GG_ERR_UNSUPPORTED;
  if (misaligned(X, 16) || misaligned(X8, 16) || misaligned(rows_used, 4) ||
      misaligned(dev_status, 4))
    return GG_ERR_UNSUPPORTED;
  if (rows > 0 && (X == nullptr || X8 == nullptr || scale == nullptr)) return GG_ERR_INVALID_ARG;
  return GG_OK;
}

}  // namespace act8
}  // namespace gg

extern "C" {

gg_status gg_silu_mul(const void* H, int64_t rows, int64_t N, const int32_t* rows_used,
                      const int32_t* row_of, int64_t n_assign, const float* weights,
                      int32_t flags, void* act, void* H8, void* H8_scale, int32_t* dev_status,
                      cudaStream_t stream) {
  using namespace gg::act8;
  gg_status s = check(rows, N, row_of, weights, n_assign, rows_used, flags, dev_status);
  if (s != GG_OK) return s;
  if ((H8 == nullptr) != (H8_scale == nullptr)) return GG_ERR_INVALID_ARG;
  if (misaligned(H, 16) || misaligned(act, 16) || misaligned(H8, 16)) return GG_ERR_UNSUPPORTED;
  if (rows > 0 && (H == nullptr || act == nullptr)) return GG_ERR_INVALID_ARG;
  int sms = 0;
  if ((s = device_sms(&sms)) != GG_OK) return s;
  Params p = params(rows, N, row_of, weights, n_assign, rows_used, flags, dev_status);
  p.H = static_cast<const uint4*>(H);
  p.act = static_cast<uint4*>(act);
  p.H8_out = static_cast<uint2*>(H8);
  p.scale_out = static_cast<uint8_t*>(H8_scale);
  return H8 != nullptr ? launch_forward<true>(p, sms, stream)
                       : launch_forward<false>(p, sms, stream);
}

gg_status gg_silu_mul_backward(const void* dact, const void* H, const void* H8,
                               const void* H8_scale, int64_t rows, int64_t N,
                               const int32_t* rows_used, const int32_t* row_of,
                               int64_t n_assign, const float* weights, int32_t flags, void* dH,
                               void* act, float* dweights, int32_t* dev_status,
                               cudaStream_t stream) {
  using namespace gg::act8;
  gg_status s = check(rows, N, row_of, weights, n_assign, rows_used, flags, dev_status);
  if (s != GG_OK) return s;
  if ((H8 == nullptr) != (H8_scale == nullptr)) return GG_ERR_INVALID_ARG;
  if (H != nullptr && H8 != nullptr) return GG_ERR_INVALID_ARG;
  if (misaligned(H, 16) || misaligned(H8, 16) || misaligned(dact, 16) || misaligned(dH, 16) ||
      misaligned(act, 16) || misaligned(dweights, 4))
    return GG_ERR_UNSUPPORTED;
  if (rows > 0 && (dact == nullptr || dH == nullptr || (H == nullptr && H8 == nullptr)))
    return GG_ERR_INVALID_ARG;
  int sms = 0;
  if ((s = device_sms(&sms)) != GG_OK) return s;
  Params p = params(rows, N, row_of, weights, n_assign, rows_used, flags, dev_status);
  p.H = static_cast<const uint4*>(H);
  p.H8 = static_cast<const uint2*>(H8);
  p.H8_scale = static_cast<const uint8_t*>(H8_scale);
  p.dact = static_cast<const uint4*>(dact);
  p.dH = static_cast<uint4*>(dH);
  p.act = static_cast<uint4*>(act);
  p.dweights = dweights;
  return H8 != nullptr ? launch_backward<true>(p, sms, stream)
                       : launch_backward<false>(p, sms, stream);
}

gg_status gg_pack8(const void* X, int64_t rows, int64_t cols, const int32_t* rows_used, void* X8,
                   void* scale, int32_t* dev_status, cudaStream_t stream) {
  using namespace gg::act8;
  gg_status s = check_rows8(X, X8, scale, rows, cols, rows_used, dev_status);
  if (s != GG_OK) return s;
  int sms = 0;
  if ((s = device_sms(&sms)) != GG_OK) return s;
  if (rows == 0) return GG_OK;
  const auto go = [&](auto kernel, int64_t per) {
    s = launch("gg_pack8", kernel, (unsigned)((rows + per - 1) / per), THREADS, stream,
               static_cast<const uint4*>(X), static_cast<uint2*>(X8),
               static_cast<uint8_t*>(scale), rows, (int32_t)(cols / 8), rows_used, dev_status);
  };
  if (share_row(rows, cols / 8, sms)) {
    go(pack8_kernel<32, WARPS, 1>, 1);
  } else {
    by_length<MANY>(cols / 8, [&](auto g) {
      constexpr int G = decltype(g)::value;
      go(pack8_kernel<G, 1, MANY>, THREADS / G);
    });
  }
  return s;
}

gg_status gg_unpack8(const void* X8, const void* scale, int64_t rows, int64_t cols,
                     const int32_t* rows_used, int32_t flags, void* X, int32_t* dev_status,
                     cudaStream_t stream) {
  using namespace gg::act8;
  gg_status s = check_rows8(X, X8, scale, rows, cols, rows_used, dev_status);
  if (s != GG_OK) return s;
  if (flags & ~GG_FLAG_ZERO_TAIL) return GG_ERR_INVALID_ARG;
  if ((flags & GG_FLAG_ZERO_TAIL) && rows_used == nullptr) return GG_ERR_INVALID_ARG;
  int sms = 0;
  if ((s = device_sms(&sms)) != GG_OK) return s;
  if (rows == 0) return GG_OK;
  const auto go = [&](auto kernel, int64_t per) {
    s = launch("gg_unpack8", kernel, (unsigned)((rows + per - 1) / per), THREADS, stream,
               static_cast<const uint2*>(X8), static_cast<const uint8_t*>(scale),
               static_cast<uint4*>(X), rows, (int32_t)(cols / 8), rows_used,
               flags & GG_FLAG_ZERO_TAIL, dev_status);
  };
  if (share_row(rows, cols / 8, sms)) {
    go(unpack8_kernel<32, WARPS, 1>, 1);
  } else {
    by_length<MANY>(cols / 8, [&](auto g) {
      constexpr int G = decltype(g)::value;
      go(unpack8_kernel<G, 1, MANY>, THREADS / G);
    });
  }
  return s;
}

}  // extern "C"
