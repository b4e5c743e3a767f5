// The way back from the packed layout: each token's rows, weighted and summed in fp32 in the
// order of its slots, and the gradients of the packed rows and of the weights. Without weights
// the sum is the gradient of gg_route.
#include <cstdint>

#include "gg_ops.cuh"

namespace gg {
namespace unroute {

using namespace gg::ops;

constexpr int THREADS = 256;
constexpr int WARPS = THREADS / 32;

struct Params {
  const uint4* Y;           // packed rows [rows, N], 8 bf16 a vector
  const int32_t* row_of;
  const float* weights;
  const uint4* residual;
  uint4* out;
  const uint4* dout;
  uint4* dY;
  float* dweights;
  const int32_t* used;
  int32_t* status;
  int64_t T;
  int64_t rows;
  int64_t vecs;             // vectors of a row
  int32_t k;
};

// Packed row of an assignment: -1 when it was dropped or names no row.
__device__ __forceinline__ int64_t row_at(const Params& p, int64_t i, int64_t rows,
                                          bool report) {
  const int64_t r = p.row_of[i];
  if (r >= rows) {
    if (report) flag(p.status, GG_DEV_BAD_ROUTE);
    return -1;
  }
  return r < 0 ? -1 : r;
}

__global__ void __launch_bounds__(THREADS) unroute_kernel(Params p) {
  const int64_t t = blockIdx.x;
  for (int64_t v = threadIdx.x; v < p.vecs; v += THREADS) {
    float acc[8] = {};
    for (int s = 0; s < p.k; ++s) {
      const int64_t r = row_at(p, t * p.k + s, p.rows, v == 0);
      if (r < 0) continue;
      const float w = p.weights != nullptr ? p.weights[t * p.k + s] : 1.f;
      float y[8];
      unpack_bf16(p.Y[r * p.vecs + v], y);
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i] = fmaf(w, y[i], acc[i]);
    }
    if (p.residual != nullptr) {
      float y[8];
      unpack_bf16(p.residual[t * p.vecs + v], y);
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i] += y[i];
    }
    p.out[t * p.vecs + v] = pack_bf16(acc);
  }
}

// dY[r] = w dout[t] and dw = <dout[t], Y[r]> of every slot; blocks past the tokens write zeros
// to the rows that are not in use.
__global__ void __launch_bounds__(THREADS) unroute_backward_kernel(Params p) {
  __shared__ float part[WARPS];
  const int64_t used =
      rows_in_use(p.used, p.rows, p.status, blockIdx.x == 0 && threadIdx.x == 0);
  if (blockIdx.x >= p.T) {
    const int64_t r = used + (blockIdx.x - p.T);
    if (r >= p.rows) return;
    for (int64_t v = threadIdx.x; v < p.vecs; v += THREADS)
      p.dY[r * p.vecs + v] = make_uint4(0, 0, 0, 0);
    return;
  }
  const int64_t t = blockIdx.x;
  for (int s = 0; s < p.k; ++s) {
    const int64_t r = row_at(p, t * p.k + s, used, threadIdx.x == 0);
    const float w = p.weights != nullptr ? p.weights[t * p.k + s] : 1.f;
    float dot = 0.f;
    if (r >= 0) {
      for (int64_t v = threadIdx.x; v < p.vecs; v += THREADS) {
        float d[8], y[8];
        unpack_bf16(p.dout[t * p.vecs + v], d);
        if (p.dweights != nullptr) {
          unpack_bf16(p.Y[r * p.vecs + v], y);
#pragma unroll
          for (int i = 0; i < 8; ++i) dot = fmaf(d[i], y[i], dot);
        }
        if (p.dY != nullptr) {
#pragma unroll
          for (int i = 0; i < 8; ++i) d[i] *= w;
          p.dY[r * p.vecs + v] = pack_bf16(d);
        }
      }
    }
    if (p.dweights != nullptr) {
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, d);
      if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = dot;
      __syncthreads();
      if (threadIdx.x == 0) {
        float sum = 0.f;
        for (int i = 0; i < WARPS; ++i) sum += part[i];
        p.dweights[t * p.k + s] = sum;
      }
      __syncthreads();
    }
  }
}

gg_status check(int64_t rows, int64_t T, int32_t k, int64_t N, const int32_t* dev_status) {
  if (rows < 0 || T < 0 || k < 1 || N < 1) return GG_ERR_INVALID_ARG;
  if (N % 8 != 0 || N >= (int64_t(1) << 31) || rows >= (int64_t(1) << 31) ||
      T >= (int64_t(1) << 31) || T * k >= (int64_t(1) << 31))
    return GG_ERR_UNSUPPORTED;
  if (misaligned(dev_status, 4)) return GG_ERR_UNSUPPORTED;
  return GG_OK;
}

}  // namespace unroute
}  // namespace gg

extern "C" {

gg_status gg_unroute(const void* Y, int64_t rows, const int32_t* row_of, const float* weights,
                     const void* residual, int64_t T_tok, int32_t k, int64_t N, void* out,
                     int32_t* dev_status, cudaStream_t stream) {
  using namespace gg::unroute;
  gg_status s = check(rows, T_tok, k, N, dev_status);
  if (s != GG_OK) return s;
  if (misaligned(Y, 16) || misaligned(residual, 16) || misaligned(out, 16) ||
      misaligned(row_of, 4) || misaligned(weights, 4))
    return GG_ERR_UNSUPPORTED;
  if (T_tok > 0 && (row_of == nullptr || out == nullptr || (rows > 0 && Y == nullptr)))
    return GG_ERR_INVALID_ARG;
  int sms = 0;
  if ((s = device_sms(&sms)) != GG_OK) return s;
  if (T_tok == 0) return GG_OK;
  Params p = {};
  p.Y = static_cast<const uint4*>(Y);
  p.row_of = row_of;
  p.weights = weights;
  p.residual = static_cast<const uint4*>(residual);
  p.out = static_cast<uint4*>(out);
  p.status = dev_status;
  p.T = T_tok;
  p.rows = rows;
  p.vecs = N / 8;
  p.k = k;
  unroute_kernel<<<(unsigned)T_tok, THREADS, 0, stream>>>(p);
  return launched("gg_unroute");
}

gg_status gg_unroute_backward(const void* dout, const void* Y, int64_t rows,
                              const int32_t* row_of, const float* weights, int64_t T_tok,
                              int32_t k, int64_t N, const int32_t* rows_used, int32_t flags,
                              void* dY, float* dweights, int32_t* dev_status,
                              cudaStream_t stream) {
  using namespace gg::unroute;
  gg_status s = check(rows, T_tok, k, N, dev_status);
  if (s != GG_OK) return s;
  if (flags & ~GG_FLAG_ZERO_TAIL) return GG_ERR_INVALID_ARG;
  const bool zero = (flags & GG_FLAG_ZERO_TAIL) != 0;
  if (zero && (rows_used == nullptr || dY == nullptr)) return GG_ERR_INVALID_ARG;
  if (misaligned(Y, 16) || misaligned(dout, 16) || misaligned(dY, 16) || misaligned(row_of, 4) ||
      misaligned(weights, 4) || misaligned(dweights, 4) || misaligned(rows_used, 4))
    return GG_ERR_UNSUPPORTED;
  if (T_tok > 0 && (dout == nullptr || row_of == nullptr ||
                    (dweights != nullptr && rows > 0 && Y == nullptr)))
    return GG_ERR_INVALID_ARG;
  if (dY == nullptr && dweights == nullptr && rows > 0) return GG_ERR_INVALID_ARG;
  int sms = 0;
  if ((s = device_sms(&sms)) != GG_OK) return s;
  const int64_t grid = T_tok + (zero ? rows : 0);
  if (grid == 0) return GG_OK;
  if (grid >= (int64_t(1) << 31)) return GG_ERR_UNSUPPORTED;
  Params p = {};
  p.Y = static_cast<const uint4*>(Y);
  p.row_of = row_of;
  p.weights = weights;
  p.dout = static_cast<const uint4*>(dout);
  p.dY = static_cast<uint4*>(dY);
  p.dweights = dweights;
  p.used = rows_used;
  p.status = dev_status;
  p.T = T_tok;
  p.rows = rows;
  p.vecs = N / 8;
  p.k = k;
  unroute_backward_kernel<<<(unsigned)grid, THREADS, 0, stream>>>(p);
  return launched("gg_unroute_backward");
}

}  // extern "C"
