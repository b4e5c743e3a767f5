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
// five. A thread therefore takes eight or so rows' vectors at once: SLOTS slots each of PER
// tokens. With one token a thread whatever k, 65536 tokens x 1 slot of 4096 columns took 460 us
// forward (now 169, at the copy rate 167), 32768 x 2 253 (131), 16384 x 4 of 2048 70 (57);
// backward of the first two 435 (239) and 265 (205).
constexpr int BLOCKS = 4;

// Rows and weights of SLOTS slots from s0 on of the tokens from t0 on; the row is negative for a
// dropped assignment, one past `rows`, or one that there is not. Each lane fetches one, the warp
// shares them. Called by whole warps.
template <int SLOTS, int PER>
__device__ __forceinline__ void slots_of(const Params& p, int64_t t0, int s0, int64_t rows,
                                         bool report, int32_t (&r)[PER * SLOTS],
                                         float (&w)[PER * SLOTS]) {
  constexpr int N = PER * SLOTS;
  const int e = threadIdx.x % N;
  const int64_t t = t0 + e / SLOTS;
  const int s = s0 + e % SLOTS;
  int32_t row = -1;
  float weight = 0.f;
  if (t < p.T && s < p.k) {
    row = p.row_of[t * p.k + s];
    weight = p.weights != nullptr ? p.weights[t * p.k + s] : 1.f;  // on its way with the row
    if (row >= rows) {
      if (report && threadIdx.x % 32 < N) flag(p.status, GG_DEV_BAD_ROUTE);
      row = -1;
    }
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    r[i] = __shfl_sync(0xffffffffu, row, i);
    w[i] = __shfl_sync(0xffffffffu, weight, i);
  }
}

// blockDim.x threads take a vector each of a piece of a token's columns, blockDim.y such rows of
// threads PER tokens each. More than SLOTS slots (SLOTS 8, PER 1 only) take several rounds.
template <int SLOTS, int PER, bool RESIDUAL>
__global__ void __launch_bounds__(THREADS, BLOCKS) unroute_kernel(Params p, int32_t chunks) {
  after_previous();
  static_assert(PER == 1 || SLOTS < 8, "one round but for SLOTS 8");
  const int32_t chunk = blockIdx.x % chunks;
  const int64_t t0 = ((int64_t)(blockIdx.x / chunks) * blockDim.y + threadIdx.y) * PER;
  const int64_t v = (int64_t)chunk * blockDim.x + threadIdx.x;
  const bool in = v < p.vecs;
  float acc[8] = {};
  for (int s0 = 0; s0 < p.k; s0 += SLOTS) {
    uint4 y[PER * SLOTS], res[PER];
    if constexpr (RESIDUAL) {
#pragma unroll
      for (int i = 0; i < PER; ++i)
        if (in && t0 + i < p.T && s0 + SLOTS >= p.k) res[i] = p.residual[(t0 + i) * p.vecs + v];
    }
    int32_t r[PER * SLOTS];
    float w[PER * SLOTS];
    slots_of<SLOTS, PER>(p, t0, s0, p.rows, chunk == 0 && threadIdx.x < 32, r, w);
#pragma unroll
    for (int i = 0; i < PER * SLOTS; ++i)
      if (in && r[i] >= 0) y[i] = __ldcs(p.Y + (int64_t)r[i] * p.vecs + v);  // read once
#pragma unroll
    for (int i = 0; i < PER; ++i) {
#pragma unroll
      for (int s = 0; s < SLOTS; ++s) {
        if (r[i * SLOTS + s] < 0) continue;
        float x[8];
        unpack_bf16(y[i * SLOTS + s], x);
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[j] = fmaf(w[i * SLOTS + s], x[j], acc[j]);
      }
      if (s0 + SLOTS < p.k) continue;  // more slots to come
      if constexpr (RESIDUAL) {
        float x[8];
        unpack_bf16(res[i], x);
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[j] += x[j];
      }
      if (in && t0 + i < p.T) p.out[(t0 + i) * p.vecs + v] = pack_bf16(acc);
#pragma unroll
      for (int j = 0; j < 8; ++j) acc[j] = 0.f;
    }
  }
}

// Sums over the warp of N values at once, N a power of two: each step halves the values a lane
// holds, then the rest of the lanes add up. Lane l ends with the sum of value number
// sum_index<N>(l).
template <int N>
__device__ __forceinline__ float warp_sums(float (&v)[N]) {
  const int lane = threadIdx.x & 31;
  int d = 16;
#pragma unroll
  for (int n = N / 2; n >= 1; n /= 2, d /= 2) {
    const bool up = (lane & d) != 0;
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const float send = up ? v[i] : v[i + n];
      v[i] = (up ? v[i + n] : v[i]) + __shfl_xor_sync(0xffffffffu, send, d);
    }
  }
  float x = v[0];
#pragma unroll
  for (; d >= 1; d /= 2) x += __shfl_xor_sync(0xffffffffu, x, d);
  return x;
}
template <int N>
__device__ __forceinline__ int sum_index(int lane) {
  int i = 0, d = 16;
#pragma unroll
  for (int n = N / 2; n >= 1; n /= 2, d /= 2) i += (lane & d) != 0 ? n : 0;
  return i;
}

// dY[r] = w dout[t] and dw = <dout[t], Y[r]> of every slot: a row of threads takes PER tokens,
// whole. The blocks past the tokens' write zeros to the rows that are not in use.
template <int SLOTS, int PER, bool DY, bool DW>
__global__ void __launch_bounds__(THREADS, BLOCKS) unroute_backward_kernel(Params p,
                                                                           int32_t blocks) {
  after_previous();
  constexpr int N = PER * SLOTS;
  __shared__ float part[WARPS][N];
  const int64_t used = rows_in_use(p.used, p.rows, p.status,
                                   blockIdx.x == 0 && threadIdx.x == 0 && threadIdx.y == 0);
  if (blockIdx.x >= blocks) {
    const int64_t step = (int64_t)(gridDim.x - blocks) * blockDim.y;
    for (int64_t r = used + (int64_t)(blockIdx.x - blocks) * blockDim.y + threadIdx.y; r < p.rows;
         r += step)
      for (int64_t v = threadIdx.x; v < p.vecs; v += blockDim.x)
        p.dY[r * p.vecs + v] = make_uint4(0, 0, 0, 0);
    return;
  }
  const int64_t t0 = ((int64_t)blockIdx.x * blockDim.y + threadIdx.y) * PER;
  for (int s0 = 0; s0 < p.k; s0 += SLOTS) {
    int32_t r[N];
    float w[N], dot[N] = {};
    slots_of<SLOTS, PER>(p, t0, s0, used, threadIdx.x < 32, r, w);
    for (int64_t v = threadIdx.x; v < p.vecs; v += blockDim.x) {
      uint4 y[N], dv[PER];
#pragma unroll
      for (int i = 0; i < PER; ++i)
        if (t0 + i < p.T) dv[i] = p.dout[(t0 + i) * p.vecs + v];
      if constexpr (DW) {
#pragma unroll
        for (int i = 0; i < N; ++i)
          if (r[i] >= 0) y[i] = __ldcs(p.Y + (int64_t)r[i] * p.vecs + v);
      }
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        float d[8];
        unpack_bf16(dv[i], d);
#pragma unroll
        for (int s = 0; s < SLOTS; ++s) {
          const int e = i * SLOTS + s;
          if (r[e] < 0) continue;
          float x[8];
          if constexpr (DW) {
            unpack_bf16(y[e], x);
#pragma unroll
            for (int j = 0; j < 8; ++j) dot[e] = fmaf(d[j], x[j], dot[e]);
          }
          if constexpr (DY) {
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = w[e] * d[j];
            p.dY[(int64_t)r[e] * p.vecs + v] = pack_bf16(x);
          }
        }
      }
    }
    if constexpr (DW) {
      const int lane = threadIdx.x & 31, warps = blockDim.x / 32;
      const float sum = warp_sums<N>(dot);
      if (lane % (32 / N) == 0)
        part[threadIdx.y * warps + threadIdx.x / 32][sum_index<N>(lane)] = sum;
      __syncthreads();
      const int e = threadIdx.x;
      const int64_t t = t0 + e / SLOTS;
      const int s = s0 + e % SLOTS;
      if (e < N && t < p.T && s < p.k) {
        float all = 0.f;
        for (int i = 0; i < warps; ++i) all += part[threadIdx.y * warps + i][e];
        p.dweights[t * p.k + s] = all;
      }
      __syncthreads();  // part is written again for the next slots
    }
  }
}

// Threads for rows of `vecs` vectors: pieces of at most THREADS, each a whole number of warps;
// short rows several to a block unless there are too few tokens to fill the GPU anyway.
struct Shape {
  int64_t chunks;  // pieces of a row
  dim3 block;
  bool few;
};
Shape shape_of(int64_t T, int64_t vecs, int sms) {
  Shape s;
  s.chunks = (vecs + THREADS - 1) / THREADS;
  const unsigned x = 32 * (unsigned)((vecs + 32 * s.chunks - 1) / (32 * s.chunks));
  s.few = T * s.chunks <= 8 * (int64_t)sms;
  s.block = dim3(x, s.few ? 1 : THREADS / x);
  return s;
}

template <int SLOTS, int PER>
gg_status launch_forward(const Params& p, const Shape& s, cudaStream_t stream) {
  constexpr int LESS = SLOTS <= 2 ? PER / 2 : PER;  // the residual's vectors take registers too
  const int64_t per = (int64_t)s.block.y * (p.residual != nullptr ? LESS : PER);
  const int64_t grid = (p.T + per - 1) / per * s.chunks;
  if (grid >= (int64_t(1) << 31)) return GG_ERR_UNSUPPORTED;
  return launch("gg_unroute",
                p.residual != nullptr ? unroute_kernel<SLOTS, LESS, true>
                                      : unroute_kernel<SLOTS, PER, false>,
                (unsigned)grid, s.block, stream, p, (int32_t)s.chunks);
}

template <int SLOTS, int PER>
gg_status launch_backward(const Params& p, const Shape& s, int64_t tail, cudaStream_t stream) {
  const int64_t per = (int64_t)s.block.y * PER;
  const int64_t blocks = (p.T + per - 1) / per;
  if (blocks + tail >= (int64_t(1) << 31)) return GG_ERR_UNSUPPORTED;
  const auto kernel = p.dweights == nullptr ? unroute_backward_kernel<SLOTS, PER, true, false>
                      : p.dY == nullptr     ? unroute_backward_kernel<SLOTS, PER, false, true>
                                            : unroute_backward_kernel<SLOTS, PER, true, true>;
  return launch("gg_unroute_backward", kernel, (unsigned)(blocks + tail), s.block, stream, p,
                (int32_t)blocks);
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
  const Shape sh = shape_of(T_tok, p.vecs, sms);
  if (sh.few || k > 4) return launch_forward<8, 1>(p, sh, stream);
  if (k > 2) return launch_forward<4, 2>(p, sh, stream);
  if (k > 1) return launch_forward<2, 4>(p, sh, stream);
  return launch_forward<1, 8>(p, sh, stream);
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
  if (T_tok + tail == 0) return GG_OK;
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
  const Shape sh = shape_of(T_tok, p.vecs, sms);
  if (sh.few || k > 4) return launch_backward<8, 1>(p, sh, tail, stream);
  if (k > 2) return launch_backward<4, 2>(p, sh, tail, stream);
  if (k > 1)
    return dweights != nullptr ? launch_backward<2, 2>(p, sh, tail, stream)
                               : launch_backward<2, 4>(p, sh, tail, stream);
  return launch_backward<1, 4>(p, sh, tail, stream);
}

}  // extern "C"
