// What the operators around the grouped GEMM share: host checks, and the device pieces of
// 16-byte rows of bf16 and of the 8-bit row form.
#pragma once
#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "gg.h"

namespace gg {
namespace ops {

// gg_api.cu: the current device must be sm_100 (its SM count in *sms); the text of a failure
// goes where gg_last_error finds it.
gg_status device_sms(int* sms);
gg_status cuda_failed(const char* where, cudaError_t e);

inline bool misaligned(const void* p, uintptr_t a) {
  return (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0;
}

inline gg_status launched(const char* where) {
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? GG_OK : cuda_failed(where, e);
}

// ---------------------------------------------------------------- device
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

// ---- the 8-bit row form: e4m3 values under one power-of-two scale 2^(c - 127) for 32
// columns, c the least code in [kMinCode, kMaxCode] with amax <= 448 * 2^(c - 127). With a
// power of two the division is exact, so the only rounding is e4m3's own, to nearest even.
// kMinCode keeps every stored value a multiple of bf16's smallest one (2^-133): restoring is
// exact.
constexpr int kBlock = 32;
constexpr int kMinCode = 9, kMaxCode = 247;

// Code of a block whose largest finite magnitude has the fp32 bits `amax` (a value of
// 1.m * 2^(x - 127) is above 448 * 2^(x - 135) = 1.75 * 2^(x - 127) when m is above 0.75).
__device__ __forceinline__ uint32_t block_code(uint32_t amax) {
  const int c = (int)(amax >> 23) - 8 + ((amax & 0x7fffffu) > 0x600000u ? 1 : 0);
  return (uint32_t)min(max(c, kMinCode), kMaxCode);
}

__device__ __forceinline__ float code_scale(uint32_t c) { return __uint_as_float(c << 23); }
__device__ __forceinline__ float code_inverse(uint32_t c) {
  return __uint_as_float((254u - c) << 23);
}

// Bits of the largest finite |x| of eight values (0 when there is none).
__device__ __forceinline__ uint32_t amax_bits(const float (&x)[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t a = __float_as_uint(x[i]) & 0x7fffffffu;
    m = max(m, a < 0x7f800000u ? a : 0u);
  }
  return m;
}

// The same over the four lanes that hold a block's 32 columns.
__device__ __forceinline__ uint32_t block_amax(uint32_t m) {
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
  return max(m, __shfl_xor_sync(0xffffffffu, m, 2));
}

// x over the code's scale as e4m3; an infinity becomes NaN (x * 0 + ...), which the restored
// value shows. Under the largest code 256 would be restored as 2^128: values end at 240 there.
__device__ __forceinline__ uint2 to_e4m3(const float (&x)[8], uint32_t code) {
  const float inv = code_inverse(code);
  float v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = x[i] * inv;
  if (code == kMaxCode) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = fminf(fmaxf(v[i], -240.f), 240.f);
  }
  uint32_t h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float a = __fmaf_rn(x[2 * i], 0.f, v[2 * i]);
    const float b = __fmaf_rn(x[2 * i + 1], 0.f, v[2 * i + 1]);
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
    h[i] = r;
  }
  return make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
}

__device__ __forceinline__ void from_e4m3(const uint2& q, float scale, float (&x)[8]) {
  const uint32_t w[2] = {q.x, q.y};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint16_t pair = (uint16_t)(w[i / 2] >> (16 * (i % 2)));
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(pair));
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
    x[2 * i] = f.x * scale;
    x[2 * i + 1] = f.y * scale;
  }
}

}  // namespace ops
}  // namespace gg
