// Between the two expert products: SiLU-and-mul of packed rows, which can keep its input in
// the 8-bit row form, and the backward pass that starts from that form (or from the bf16
// input). And the form itself: packed rows to 8 bits and back.
#include <cstdint>

#include "gg_ops.cuh"

namespace gg {
namespace act8 {

using namespace gg::ops;

constexpr int THREADS = 128;
constexpr int WARPS = THREADS / 32;

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
  int32_t half;             // I = N / 2
  int32_t concat;
  int32_t zero_tail;
};

__device__ __forceinline__ float sigmoid(float x) { return __fdividef(1.f, 1.f + __expf(-x)); }

// What block b works on: a packed row with the index of its weight, a row to clear (weight
// index -1), or nothing (row -1; the weight's gradient is then 0).
struct Work {
  int64_t row;
  int64_t at;
};
__device__ __forceinline__ Work work_of(const Params& p, int64_t b) {
  const bool report = threadIdx.x == 0;
  if (p.row_of == nullptr) {
    const int64_t used = rows_in_use(p.used, p.rows, p.status, report && b == 0);
    if (b < used) return {b, b};
    return {p.zero_tail ? b : -1, -1};
  }
  const int64_t used = rows_in_use(p.used, p.rows, p.status, report && b == 0);
  if (b < p.n) {
    const int64_t r = p.row_of[b];
    if (r >= used && report) flag(p.status, GG_DEV_BAD_ROUTE);
    return {r >= used || r < 0 ? -1 : r, b};
  }
  const int64_t r = used + (b - p.n);
  return {r < p.rows ? r : -1, -1};
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

__global__ void __launch_bounds__(THREADS) silu_mul_kernel(Params p) {
  const Work w = work_of(p, blockIdx.x);
  if (w.row < 0) return;
  const int vecs = p.half / 8;
  if (w.at < 0) {
    for (int c = threadIdx.x; c < vecs; c += THREADS)
      p.act[w.row * vecs + c] = make_uint4(0, 0, 0, 0);
    return;
  }
  const float scale = p.weights != nullptr ? p.weights[w.at] : 1.f;
  const int64_t base = w.row * 2 * vecs;
  const int64_t code0 = w.row * 2 * ((p.half + kBlock - 1) / kBlock);
  // whole warps go round together: the four lanes of a block exchange their largest values
  for (int c = threadIdx.x; c - (int)(threadIdx.x & 31) < vecs; c += THREADS) {
    float g[8] = {}, u[8] = {};
    const bool in = c < vecs;
    if (in) {
      unpack_bf16(p.H[base + gate_vec(p, c)], g);
      unpack_bf16(p.H[base + up_vec(p, c)], u);
    }
    if (p.H8_out != nullptr) {
      const uint32_t cg = block_code(block_amax(amax_bits(g)));
      const uint32_t cu = block_code(block_amax(amax_bits(u)));
      if (in) {
        p.H8_out[base + gate_vec(p, c)] = to_e4m3(g, cg);
        p.H8_out[base + up_vec(p, c)] = to_e4m3(u, cu);
        if ((c & 3) == 0) {
          p.scale_out[code0 + gate_code(p, c)] = (uint8_t)cg;
          p.scale_out[code0 + up_code(p, c)] = (uint8_t)cu;
        }
      }
    }
    if (in) {
      float a[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) a[i] = scale * (g[i] * sigmoid(g[i]) * u[i]);
      p.act[w.row * vecs + c] = pack_bf16(a);
    }
  }
}

// h = [g, u] from its 8 bits (or bf16), s the row's weight, q = sigma(g):
//   dg = s dact u q (1 + g (1 - q)),  du = s dact g q,  act = s g q u,  ds = <dact, g q u>
__global__ void __launch_bounds__(THREADS) silu_mul_backward_kernel(Params p) {
  __shared__ float part[WARPS];
  const Work w = work_of(p, blockIdx.x);
  const int vecs = p.half / 8;
  float dot = 0.f;
  if (w.row >= 0) {
    const int64_t base = w.row * 2 * vecs;
    if (w.at < 0) {
      for (int c = threadIdx.x; c < vecs; c += THREADS) {
        p.dH[base + c] = p.dH[base + vecs + c] = make_uint4(0, 0, 0, 0);
        if (p.act != nullptr) p.act[w.row * vecs + c] = make_uint4(0, 0, 0, 0);
      }
      return;
    }
    const float scale = p.weights != nullptr ? p.weights[w.at] : 1.f;
    const int64_t code0 = w.row * 2 * ((p.half + kBlock - 1) / kBlock);
    for (int c = threadIdx.x; c < vecs; c += THREADS) {
      float g[8], u[8], d[8], a[8], dg[8], du[8];
      if (p.H8 != nullptr) {
        from_e4m3(p.H8[base + gate_vec(p, c)],
                  code_scale(p.H8_scale[code0 + gate_code(p, c)]), g);
        from_e4m3(p.H8[base + up_vec(p, c)], code_scale(p.H8_scale[code0 + up_code(p, c)]), u);
      } else {
        unpack_bf16(p.H[base + gate_vec(p, c)], g);
        unpack_bf16(p.H[base + up_vec(p, c)], u);
      }
      unpack_bf16(p.dact[w.row * vecs + c], d);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float q = sigmoid(g[i]), silu = g[i] * q, sd = scale * d[i];
        dot = fmaf(d[i], silu * u[i], dot);
        a[i] = scale * (silu * u[i]);
        dg[i] = sd * u[i] * (q * (1.f + g[i] * (1.f - q)));
        du[i] = sd * silu;
      }
      p.dH[base + gate_vec(p, c)] = pack_bf16(dg);
      p.dH[base + up_vec(p, c)] = pack_bf16(du);
      if (p.act != nullptr) p.act[w.row * vecs + c] = pack_bf16(a);
    }
  }
  if (p.dweights == nullptr || w.at < 0) return;  // the same for the whole block
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, d);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = dot;
  __syncthreads();
  if (threadIdx.x == 0) {
    float sum = 0.f;
    for (int i = 0; i < WARPS; ++i) sum += part[i];
    p.dweights[w.at] = sum;
  }
}

__global__ void __launch_bounds__(THREADS) pack8_kernel(const uint4* X, uint2* X8, uint8_t* scale,
                                                        int64_t rows, int32_t vecs,
                                                        const int32_t* used, int32_t* status) {
  const int64_t r = blockIdx.x;
  if (r >= rows_in_use(used, rows, status, r == 0 && threadIdx.x == 0)) return;
  const int64_t codes = (vecs + 3) / 4;
  for (int c = threadIdx.x; c - (int)(threadIdx.x & 31) < vecs; c += THREADS) {
    float x[8] = {};
    if (c < vecs) unpack_bf16(X[r * vecs + c], x);
    const uint32_t code = block_code(block_amax(amax_bits(x)));
    if (c < vecs) {
      X8[r * vecs + c] = to_e4m3(x, code);
      if ((c & 3) == 0) scale[r * codes + (c >> 2)] = (uint8_t)code;
    }
  }
}

__global__ void __launch_bounds__(THREADS) unpack8_kernel(const uint2* X8, const uint8_t* scale,
                                                          uint4* X, int64_t rows, int32_t vecs,
                                                          const int32_t* used, int32_t zero_tail,
                                                          int32_t* status) {
  const int64_t r = blockIdx.x;
  const bool in = r < rows_in_use(used, rows, status, r == 0 && threadIdx.x == 0);
  if (!in && !zero_tail) return;
  const int64_t codes = (vecs + 3) / 4;
  for (int c = threadIdx.x; c < vecs; c += THREADS) {
    float x[8] = {};
    if (in) from_e4m3(X8[r * vecs + c], code_scale(scale[r * codes + (c >> 2)]), x);
    X[r * vecs + c] = pack_bf16(x);
  }
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

unsigned grid_of(const Params& p) {
  return (unsigned)(p.n + (p.row_of != nullptr && p.zero_tail ? p.rows : 0));
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
  if (grid_of(p) == 0) return GG_OK;
  silu_mul_kernel<<<grid_of(p), THREADS, 0, stream>>>(p);
  return launched("gg_silu_mul");
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
  if (grid_of(p) == 0) return GG_OK;
  silu_mul_backward_kernel<<<grid_of(p), THREADS, 0, stream>>>(p);
  return launched("gg_silu_mul_backward");
}

gg_status gg_pack8(const void* X, int64_t rows, int64_t cols, const int32_t* rows_used, void* X8,
                   void* scale, int32_t* dev_status, cudaStream_t stream) {
  using namespace gg::act8;
  gg_status s = check_rows8(X, X8, scale, rows, cols, rows_used, dev_status);
  if (s != GG_OK) return s;
  int sms = 0;
  if ((s = device_sms(&sms)) != GG_OK) return s;
  if (rows == 0) return GG_OK;
  pack8_kernel<<<(unsigned)rows, THREADS, 0, stream>>>(
      static_cast<const uint4*>(X), static_cast<uint2*>(X8), static_cast<uint8_t*>(scale), rows,
      (int32_t)(cols / 8), rows_used, dev_status);
  return launched("gg_pack8");
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
  unpack8_kernel<<<(unsigned)rows, THREADS, 0, stream>>>(
      static_cast<const uint2*>(X8), static_cast<const uint8_t*>(scale), static_cast<uint4*>(X),
      rows, (int32_t)(cols / 8), rows_used, flags & GG_FLAG_ZERO_TAIL, dev_status);
  return launched("gg_unpack8");
}

}  // extern "C"
