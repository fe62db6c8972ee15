// dllm_cache.cuh -- the paged 8-bit key/value cache: its device view, the
// e4m3 conversions and the scale of a block of tokens.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/dllmcommit.h"
#include "dllm_device.cuh"
#include "dllm_launch.cuh"

namespace dllm {

// The pools as the kernels see them.  A page holds page_size tokens of every
// head: codes [page][head][slot][dim], one scale per (page, head).
struct CacheView {
  uint8_t* k;
  uint8_t* v;
  float* k_scale;
  float* v_scale;
  int64_t pages;
  int32_t page_size, heads, dim;
};

inline CacheView cache_view(const dllm_kv_cache& c) {
  CacheView v;
  v.k = static_cast<uint8_t*>(c.k);
  v.v = static_cast<uint8_t*>(c.v);
  v.k_scale = c.k_scale;
  v.v_scale = c.v_scale;
  v.pages = c.num_pages;
  v.page_size = c.page_size;
  v.heads = c.heads;
  v.dim = c.head_dim;
  return v;
}

// Shared validation of a cache and a page table (B, width).
inline dllm_status check_cache(const dllm_kv_cache* c, const int32_t* table, int64_t B, int64_t width) {
  if (!c || !c->k || !c->v || !c->k_scale || !c->v_scale) return DLLM_ERR_INVALID_ARGUMENT;
  if (c->num_pages < 1 || c->num_pages > INT32_MAX || c->heads < 1 || B < 0 || width < 1)
    return DLLM_ERR_INVALID_ARGUMENT;
  if (!aligned16(c->k) || !aligned16(c->v) || !aligned4(c->k_scale) || !aligned4(c->v_scale) || !aligned4(table))
    return DLLM_ERR_INVALID_ARGUMENT;
  if (c->head_dim != 64 && c->head_dim != 128) return DLLM_ERR_UNSUPPORTED;
  if (c->page_size != 16 && c->page_size != 32 && c->page_size != 64 && c->page_size != 128)
    return DLLM_ERR_UNSUPPORTED;
  if (c->heads > 65535) return DLLM_ERR_UNSUPPORTED;
  if (mul_or_neg(mul_or_neg(c->num_pages, c->heads), static_cast<int64_t>(c->page_size) * c->head_dim) < 0)
    return DLLM_ERR_INVALID_ARGUMENT;
  if (mul_or_neg(B, width) < 0 || mul_or_neg(width, c->page_size) < 0) return DLLM_ERR_INVALID_ARGUMENT;
  if (B > 0 && !table) return DLLM_ERR_INVALID_ARGUMENT;
  // positions are int32 in lens and start
  if (width * c->page_size > INT32_MAX || B > 65535) return DLLM_ERR_UNSUPPORTED;
  return DLLM_OK;
}

// Two fp32 values to two e4m3 codes (lo in the low byte): round to nearest
// even, saturating at 448, NaN kept.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t d;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(hi), "f"(lo));
  return d;
}

// Two e4m3 codes (the low 16 bits) to two fp16 values, exactly.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t codes) {
  uint32_t d;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(d) : "h"(static_cast<uint16_t>(codes)));
  return d;
}

__device__ __forceinline__ void f16x2_to_f32(uint32_t h, float& lo, float& hi) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
      : "=f"(lo), "=f"(hi)
      : "r"(h));
}

// The scale of a block whose largest finite magnitude is amax: the smallest
// power of two 2^e, e >= -100, with amax <= 448 2^e.  e4m3 keeps 4
// significant bits at any scale, so a power of two costs no precision, codes
// times scale are exact in bf16, and moving a token into a block of another
// scale (an append that raises it, an eviction) is exact but for underflow.
// 448 = 1.75 2^8: with amax = f 2^x, f in [1, 2), e = x - 8, one more when
// f > 1.75.
__device__ __forceinline__ float block_scale(float amax) {
  const uint32_t b = __float_as_uint(amax);
  int x = static_cast<int>(b >> 23) - 127;               // subnormal amax gives -127: clamped below
  int e = x - 8 + ((b & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  e = e < -100 ? -100 : e;
  return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}

__device__ __forceinline__ bool power_of_two(float s) {
  const uint32_t b = __float_as_uint(s);
  return (b & 0x807FFFFFu) == 0u && b >= 0x0A000000u && b <= 0x75000000u;  // 2^-107 .. 2^107: 1 / s is normal too
}

// The page a table entry names, or -1 (an entry outside the pool names none).
__device__ __forceinline__ int64_t page_at(const int32_t* table, int64_t width, int64_t b, int64_t col, int64_t pages) {
  const int32_t p = table[b * width + col];
  return p >= 0 && p < pages ? p : -1;
}

// The block's largest value in every thread (red: one float per warp).
__device__ __forceinline__ float block_max(float v, float* red) {
  v = warp_max_f32(v);
  const int warp = threadIdx.x >> 5, n = blockDim.x >> 5;
  if (n == 1) return v;
  if ((threadIdx.x & 31) == 0) red[warp] = v;
  __syncthreads();
  v = red[0];
  for (int w = 1; w < n; ++w) v = fmaxf(v, red[w]);
  return v;
}

}  // namespace dllm
