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

// Both kernels are held to 64 registers: four blocks an SM keep 128 KB of 16-byte loads in
// flight, which the memory needs. us for 4096 tokens x 8 slots of 2048 columns, and 32768 x 8 of
// 6144: forward 24 and 541 (the bytes at the copy rate: 23 and 562), 28 and 661 with three
// blocks, 33 and 658 with five (spills); backward of the former 48 (44), 51 with three, 63 with
// five.
constexpr int BLOCKS = 4;
constexpr int SLOTS = 8;  // slots taken at once: as many 16-byte loads in flight per thread

// Rows and weights of SLOTS slots of token t, from slot s0 on: negative and 0 for a dropped
// assignment or one past `rows`. Each lane fetches one slot, the warp shares them. Called by
// whole warps.
__device__ __forceinline__ void slots_of(const Params& p, int64_t t, int s0, int64_t rows,
                                         bool report, int32_t (&r)[SLOTS], float (&w)[SLOTS]) {
  const int s = s0 + (threadIdx.x & (SLOTS - 1));
  int32_t row = -1;  // negative: dropped
  float weight = 0.f;
  if (s < p.k) {
    row = p.row_of[t * p.k + s];
    if (row >= rows) {
      if (report && (threadIdx.x & 31) < SLOTS) flag(p.status, GG_DEV_BAD_ROUTE);
      row = -1;
    }
    if (row >= 0) weight = p.weights != nullptr ? p.weights[t * p.k + s] : 1.f;
  }
#pragma unroll
  for (int i = 0; i < SLOTS; ++i) {
    r[i] = __shfl_sync(0xffffffffu, row, i);
    w[i] = __shfl_sync(0xffffffffu, weight, i);
  }
}

// A block takes blockDim.x vectors of a token's columns; a thread's loads of all slots are in
// flight together.
__global__ void __launch_bounds__(THREADS, BLOCKS) unroute_kernel(Params p, int32_t chunks) {
  const int64_t t = blockIdx.x / chunks;
  const int32_t chunk = blockIdx.x % chunks;
  const int64_t v = (int64_t)chunk * blockDim.x + threadIdx.x;
  const bool in = v < p.vecs;
  float acc[8] = {};
  uint4 res = make_uint4(0, 0, 0, 0);
  if (in && p.residual != nullptr) res = p.residual[t * p.vecs + v];
  for (int s0 = 0; s0 < p.k; s0 += SLOTS) {
    int32_t r[SLOTS];
    float w[SLOTS];
    slots_of(p, t, s0, p.rows, chunk == 0 && threadIdx.x < 32, r, w);
    uint4 y[SLOTS];
#pragma unroll
    for (int i = 0; i < SLOTS; ++i)
      if (in && r[i] >= 0) y[i] = __ldcs(p.Y + (int64_t)r[i] * p.vecs + v);  // read once
#pragma unroll
    for (int i = 0; i < SLOTS; ++i) {
      if (r[i] < 0) continue;
      float x[8];
      unpack_bf16(y[i], x);
#pragma unroll
      for (int j = 0; j < 8; ++j) acc[j] = fmaf(w[i], x[j], acc[j]);
    }
  }
  if (!in) return;
  if (p.residual != nullptr) {
    float x[8];
    unpack_bf16(res, x);
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[j] += x[j];
  }
  p.out[t * p.vecs + v] = pack_bf16(acc);
}

// Sums over the warp of eight values at once: each step halves the values a lane holds. Lane l
// ends with the sum of value (l >> 2) & 7, its bits reversed (bit 4 of l is worth 4).
__device__ __forceinline__ float warp_sums(float (&v)[SLOTS]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int n = 4; n >= 1; n /= 2) {
    const bool up = (lane & (4 * n)) != 0;
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const float send = up ? v[i] : v[i + n];
      v[i] = (up ? v[i + n] : v[i]) + __shfl_xor_sync(0xffffffffu, send, 4 * n);
    }
  }
  float x = v[0] + __shfl_xor_sync(0xffffffffu, v[0], 2);
  return x + __shfl_xor_sync(0xffffffffu, x, 1);
}

// dY[r] = w dout[t] and dw = <dout[t], Y[r]> of every slot, one block a token; the blocks past
// the tokens write zeros to the rows that are not in use.
template <bool DY, bool DW>
__global__ void __launch_bounds__(THREADS, BLOCKS) unroute_backward_kernel(Params p) {
  __shared__ float part[WARPS][SLOTS];
  const int64_t used =
      rows_in_use(p.used, p.rows, p.status, blockIdx.x == 0 && threadIdx.x == 0);
  if (blockIdx.x >= p.T) {
    for (int64_t r = used + (blockIdx.x - p.T); r < p.rows; r += gridDim.x - p.T)
      for (int64_t v = threadIdx.x; v < p.vecs; v += blockDim.x)
        p.dY[r * p.vecs + v] = make_uint4(0, 0, 0, 0);
    return;
  }
  const int64_t t = blockIdx.x;
  for (int s0 = 0; s0 < p.k; s0 += SLOTS) {
    int32_t r[SLOTS];
    float w[SLOTS], dot[SLOTS] = {};
    slots_of(p, t, s0, used, threadIdx.x < 32, r, w);
    for (int64_t v = threadIdx.x; v < p.vecs; v += blockDim.x) {
      const uint4 dv = p.dout[t * p.vecs + v];
      uint4 y[SLOTS];
      if constexpr (DW) {
#pragma unroll
        for (int i = 0; i < SLOTS; ++i)
          if (r[i] >= 0) y[i] = __ldcs(p.Y + (int64_t)r[i] * p.vecs + v);
      }
      float d[8];
      unpack_bf16(dv, d);
#pragma unroll
      for (int i = 0; i < SLOTS; ++i) {
        if (r[i] < 0) continue;
        float x[8];
        if constexpr (DW) {
          unpack_bf16(y[i], x);
#pragma unroll
          for (int j = 0; j < 8; ++j) dot[i] = fmaf(d[j], x[j], dot[i]);
        }
        if constexpr (DY) {
#pragma unroll
          for (int j = 0; j < 8; ++j) x[j] = w[i] * d[j];
          p.dY[(int64_t)r[i] * p.vecs + v] = pack_bf16(x);
        }
      }
    }
    if constexpr (DW) {
      const int lane = threadIdx.x & 31;
      const float sum = warp_sums(dot);
      if ((lane & 3) == 0) {
        const int i = ((lane >> 4) & 1) * 4 + ((lane >> 3) & 1) * 2 + ((lane >> 2) & 1);
        part[threadIdx.x >> 5][i] = sum;
      }
      __syncthreads();
      if (threadIdx.x < SLOTS && s0 + threadIdx.x < p.k) {
        float all = 0.f;
        for (int i = 0; i < (int)blockDim.x / 32; ++i) all += part[i][threadIdx.x];
        p.dweights[t * p.k + s0 + threadIdx.x] = all;
      }
      __syncthreads();  // part is written again for the next slots
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
  const int64_t chunks = (p.vecs + THREADS - 1) / THREADS;
  if (T_tok * chunks >= (int64_t(1) << 31)) return GG_ERR_UNSUPPORTED;
  const unsigned threads = 32 * (unsigned)((p.vecs + 32 * chunks - 1) / (32 * chunks));
  unroute_kernel<<<(unsigned)(T_tok * chunks), threads, 0, stream>>>(p, (int32_t)chunks);
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
  if (zero && (rows_used == nullptr || (dY == nullptr && rows > 0))) return GG_ERR_INVALID_ARG;
  if (misaligned(Y, 16) || misaligned(dout, 16) || misaligned(dY, 16) || misaligned(row_of, 4) ||
      misaligned(weights, 4) || misaligned(dweights, 4) || misaligned(rows_used, 4))
    return GG_ERR_UNSUPPORTED;
  if (T_tok > 0 && (dout == nullptr || row_of == nullptr ||
                    (dweights != nullptr && rows > 0 && Y == nullptr)))
    return GG_ERR_INVALID_ARG;
  if (dY == nullptr && dweights == nullptr && rows > 0) return GG_ERR_INVALID_ARG;
  int sms = 0;
  if ((s = device_sms(&sms)) != GG_OK) return s;
  const int64_t tail = !zero ? 0 : rows < 4 * sms ? rows : 4 * sms;  // blocks that clear rows
  const int64_t grid = T_tok + tail;
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
  const int64_t rounds = (p.vecs + THREADS - 1) / THREADS;
  const unsigned threads = 32 * (unsigned)((p.vecs + 32 * rounds - 1) / (32 * rounds));
  if (dweights == nullptr)
    unroute_backward_kernel<true, false><<<(unsigned)grid, threads, 0, stream>>>(p);
  else if (dY == nullptr)
    unroute_backward_kernel<false, true><<<(unsigned)grid, threads, 0, stream>>>(p);
  else
    unroute_backward_kernel<true, true><<<(unsigned)grid, threads, 0, stream>>>(p);
  return launched("gg_unroute_backward");
}

}  // extern "C"
