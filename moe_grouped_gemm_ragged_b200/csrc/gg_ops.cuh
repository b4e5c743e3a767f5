// What the operators around the grouped GEMM share: host checks, and the device pieces of
// 16-byte rows of bf16 and of the 8-bit row form.
#pragma once
#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "gg.h"
#include "ptx.cuh"

namespace gg {
namespace ops {

// gg_api.cu: the current device must be sm_100 (its SM count in *sms); the text of a failure
// goes where gg_last_error finds it.
gg_status device_sms(int* sms);
gg_status cuda_failed(const char* where, cudaError_t e);

inline bool misaligned(const void* p, uintptr_t a) {
  return (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0;
}

// Whether two arrays of n bytes share any.
inline bool overlap(const void* a, const void* b, int64_t n) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return (x < y ? y - x : x - y) < (uintptr_t)n;
}

// Launch with programmatic dependent launch, as the grouped GEMM's kernels: a kernel may be
// scheduled while the one before it on the stream finishes, and waits for that one's completion
// (after_previous, first thing in every thread) before it touches memory. A stream or capture
// that does not take such a launch gets a plain one.
template <typename... Params, typename... Args>
gg_status launch(const char* where, void (*kernel)(Params...), unsigned grid, dim3 block,
                 cudaStream_t stream, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(grid, 1, 1);
  cfg.blockDim = block;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, static_cast<Params>(args)...);
  if (e != cudaSuccess) {
    (void)cudaGetLastError();
    cfg.numAttrs = 0;
    e = cudaLaunchKernelEx(&cfg, kernel, static_cast<Params>(args)...);
  }
  return e == cudaSuccess ? GG_OK : cuda_failed(where, e);
}

// ---------------------------------------------------------------- device
// The end of the kernel before. (No kernel here lets the next one start before its own end:
// 32768 x 64 through the gate and back took 16.8 us instead of 14.2, the next kernel's blocks
// being placed where this one's still ran.)
__device__ __forceinline__ void after_previous() { ptx::griddep_wait(); }

__device__ __forceinline__ void flag(int32_t* status, uint32_t bits) {
  if (status != nullptr) atomicOr(status, (int32_t)bits);
}

// Rows in use: *used clamped to [0, rows] (all of them without a count).
__device__ __forceinline__ int64_t rows_in_use(const int32_t* used, int64_t rows,
                                               int32_t* status, bool report) {
  if (used == nullptr) return rows;
  const int64_t u = *used;
  if (u < 0 || u > rows) {
    if (report) flag(status, GG_DEV_BAD_COUNT);
    return u < 0 ? 0 : rows;
  }
  return u;
}

__device__ __forceinline__ void unpack_bf16(const uint4& v, float (&x)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

__device__ __forceinline__ uint4 pack_bf16(const float (&x)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// The same as pairs, which the two-wide fp32 instructions take.
__device__ __forceinline__ void unpack_bf16(const uint4& v, float2 (&x)[4]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    x[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
}

__device__ __forceinline__ uint4 pack_bf16(const float2 (&x)[4]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x[i].x, x[i].y);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// ---- the 8-bit row form: e4m3 values under one power-of-two scale 2^(c - 127) for 32
// columns, c the least code in [kMinCode, kMaxCode] with amax <= 448 * 2^(c - 127). With a
// power of two the division is exact, so the only rounding is e4m3's own, to nearest even.
// kMinCode keeps every stored value a multiple of bf16's smallest one (2^-133): restoring is
// exact. What bounds these kernels next to the bytes are instructions, so the largest
// magnitudes are found on pairs of bf16 bits, for two blocks at once.
constexpr int kBlock = 32;
constexpr int kMinCode = 9, kMaxCode = 247;

__device__ __forceinline__ float code_scale(uint32_t c) { return __uint_as_float(c << 23); }
__device__ __forceinline__ float code_inverse(uint32_t c) {
  return __uint_as_float((254u - c) << 23);
}

// Magnitudes of the two bf16 in w, those of infinities and NaN as 0.
__device__ __forceinline__ uint32_t finite_bits(uint32_t w) {
  const uint32_t m = w & 0x7fff7fffu;
  return m & ~((((m + 0x00800080u) >> 15) & 0x00010001u) * 0xffffu);
}

// Codes of two blocks: four neighbouring lanes hold the 32 columns of each, eight in `a` and
// eight in `b`. The lanes of `mask` call together; *odd (the same for them): some value is not
// finite.
__device__ __forceinline__ void block_codes(uint32_t mask, const uint4& a, const uint4& b,
                                            uint32_t& ca, uint32_t& cb, bool* odd) {
  constexpr uint32_t M = 0x7fff7fffu;
  const auto over_block = [mask](uint32_t ma, uint32_t mb) {
    // the halves of ma against one another in the low half, those of mb in the high half
    uint32_t m = __vmaxu2(__byte_perm(ma, mb, 0x5410), __byte_perm(ma, mb, 0x7632));
    m = __vmaxu2(m, __shfl_xor_sync(mask, m, 1));
    return __vmaxu2(m, __shfl_xor_sync(mask, m, 2));
  };
  uint32_t m = over_block(__vmaxu2(__vmaxu2(a.x & M, a.y & M), __vmaxu2(a.z & M, a.w & M)),
                          __vmaxu2(__vmaxu2(b.x & M, b.y & M), __vmaxu2(b.z & M, b.w & M)));
  *odd = __any_sync(mask, ((m + 0x00800080u) & 0x80008000u) != 0);
  if (*odd)
    m = over_block(__vmaxu2(__vmaxu2(finite_bits(a.x), finite_bits(a.y)),
                            __vmaxu2(finite_bits(a.z), finite_bits(a.w))),
                   __vmaxu2(__vmaxu2(finite_bits(b.x), finite_bits(b.y)),
                            __vmaxu2(finite_bits(b.z), finite_bits(b.w))));
  // A magnitude 1.m * 2^(x - 127) is above 448 * 2^(x - 135) = 1.75 * 2^(x - 127) when its seven
  // bits m are above 0x60: adding 0x1f then carries into x.
  m += 0x001f001fu;
  ca = (uint32_t)min(max((int)((m & 0xffffu) >> 7) - 8, kMinCode), kMaxCode);
  cb = (uint32_t)min(max((int)(m >> 23) - 8, kMinCode), kMaxCode);
}

// x over the code's scale as e4m3. Where a value is not finite (odd) infinities become NaN (x *
// 0 + ...), which the restored value shows; under the largest code 256 would be restored as
// 2^128, so values end at 240 there.
__device__ __forceinline__ uint2 to_e4m3(const float2 (&x)[4], uint32_t code, bool odd) {
  const float2 inv = both(code_inverse(code));
  float2 v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = __fmul2_rn(x[i], inv);
  if (odd || code == kMaxCode) {
    const float top = code == kMaxCode ? 240.f : 448.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i].x = __fmaf_rn(x[i].x, 0.f, fminf(fmaxf(v[i].x, -top), top));
      v[i].y = __fmaf_rn(x[i].y, 0.f, fminf(fmaxf(v[i].y, -top), top));
    }
  }
  uint16_t h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(h[i]) : "f"(v[i].y), "f"(v[i].x));
  return make_uint2(h[0] | ((uint32_t)h[1] << 16), h[2] | ((uint32_t)h[3] << 16));
}

__device__ __forceinline__ void from_e4m3(const uint2& q, float scale, float2 (&x)[4]) {
  const uint32_t w[2] = {q.x, q.y};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint16_t pair = (uint16_t)(w[i / 2] >> (16 * (i % 2)));
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(pair));
    x[i] = __fmul2_rn(__half22float2(*reinterpret_cast<const __half2*>(&h)), both(scale));
  }
}

}  // namespace ops
}  // namespace gg
