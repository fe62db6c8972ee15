// dllm_attend.cu -- attention of a block of queries over the paged 8-bit
// key/value cache, and the attention weight each cached token draws.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "dllm_cache.cuh"

namespace dllm {

struct AttendParams {
  CacheView c;
  const uint8_t* q;            // bf16
  int64_t qb, ql, qh;          // strides in bytes
  int64_t B, L, Hq;
  const int32_t* table;
  const int32_t* lens;
  const uint8_t* mask;         // nullable
  int64_t mask_stride;
  int64_t width, cap;
  float scale2;                // scale log2 e
  uint16_t* out;               // bf16 (B, L, Hq, D)
  float* lse;                  // (B, L, Hq)
  float* weights;              // (B, heads, cap)
  float decay;
};

// Whether the sequence's token j is attended; its page.
__device__ __forceinline__ bool visible(const AttendParams& p, int64_t b, int64_t j, int n, int64_t& page) {
  page = -1;
  if (j >= n) return false;
  if (p.mask && p.mask[b * p.mask_stride + j] == 0) return false;
  page = page_at(p.table, p.width, b, j / p.c.page_size, p.c.pages);
  return page >= 0;
}

__device__ __forceinline__ int attend_len(const AttendParams& p, int64_t b) {
  const int64_t n = p.lens[b];
  return static_cast<int>(n < 0 ? 0 : (n > p.cap ? p.cap : n));
}

// q . k of one token's codes (D bytes) with a row in shared memory.
template <int D>
__device__ __forceinline__ float dot_codes(const uint8_t* codes, const float* q) {
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < D / 16; ++i) {
    const uint4 x = __ldg(reinterpret_cast<const uint4*>(codes) + i);
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float f0, f1, f2, f3;
      f16x2_to_f32(e4m3x2_to_f16x2(w[e] & 0xFFFFu), f0, f1);
      f16x2_to_f32(e4m3x2_to_f16x2(w[e] >> 16), f2, f3);
      const float* r = q + 16 * i + 4 * e;
      s = fmaf(f0, r[0], s);
      s = fmaf(f1, r[1], s);
      s = fmaf(f2, r[2], s);
      s = fmaf(f3, r[3], s);
    }
  }
  return s;
}

// One warp per query row: 32 keys at a time, one to a lane, with a running
// maximum and sum; the values are then added key by key, D / 32 dims a lane.
template <int D>
__global__ void __launch_bounds__(128) attend_kernel(const __grid_constant__ AttendParams p) {
  __shared__ float q_s[4][D];
  pdl_wait();
  pdl_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * 4 + warp;
  if (row >= p.B * p.L * p.Hq) return;
  const int64_t hq = row % p.Hq, l = row / p.Hq % p.L, b = row / (p.Hq * p.L);
  const int64_t h = hq / (p.Hq / p.c.heads);
  const uint16_t* q = reinterpret_cast<const uint16_t*>(p.q + b * p.qb + l * p.ql + hq * p.qh);
  for (int d = lane; d < D; d += 32) q_s[warp][d] = __uint_as_float(static_cast<uint32_t>(q[d]) << 16);
  __syncwarp();
  const int n = attend_len(p, b);
  const int ps = p.c.page_size;
  float m = -__builtin_huge_valf(), sum = 0.0f;
  float o[D / 32] = {};
  for (int j0 = 0; j0 < n; j0 += 32) {
    const int64_t j = j0 + lane;
    int64_t page;
    const bool ok = visible(p, b, j, n, page);
    float s = -__builtin_huge_valf(), vs = 0.0f;
    if (ok) {
      const int64_t at = page * p.c.heads + h;
      s = dot_codes<D>(p.c.k + (at * ps + j % ps) * D, q_s[warp]) * p.c.k_scale[at] * p.scale2;
      vs = p.c.v_scale[at];
    }
    const unsigned any = __ballot_sync(0xFFFFFFFFu, ok);
    if (any == 0u) continue;
    const float mn = fmaxf(m, warp_max_f32(s));
    const float ref = mn == -__builtin_huge_valf() ? 0.0f : mn;
    const float f = ex2_approx(m - ref);
    const float x = ok ? ex2_approx(s - ref) : 0.0f;
    m = mn;
    float add = x;
#pragma unroll
    for (int o2 = 16; o2 > 0; o2 >>= 1) add += __shfl_xor_sync(0xFFFFFFFFu, add, o2);
    sum = sum * f + add;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) o[i] *= f;
    for (int t = 0; t < 32; ++t) {
      if (!((any >> t) & 1u)) continue;
      const float w = __shfl_sync(0xFFFFFFFFu, x * vs, t);
      const int64_t pg = __shfl_sync(0xFFFFFFFFu, page, t);
      const uint8_t* v = p.c.v + ((pg * p.c.heads + h) * ps + (j0 + t) % ps) * D;
#pragma unroll
      for (int i = 0; i < D / 64; ++i) {
        float f0, f1;
        f16x2_to_f32(e4m3x2_to_f16x2(*reinterpret_cast<const uint16_t*>(v + 64 * i + 2 * lane)), f0, f1);
        o[2 * i] = fmaf(w, f0, o[2 * i]);
        o[2 * i + 1] = fmaf(w, f1, o[2 * i + 1]);
      }
    }
  }
  const float inv = sum != 0.0f ? 1.0f / sum : 0.0f;   // (a NaN sum gives NaN)
#pragma unroll
  for (int i = 0; i < D / 64; ++i) {
    uint32_t d;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(o[2 * i + 1] * inv), "f"(o[2 * i] * inv));
    *reinterpret_cast<uint32_t*>(p.out + row * D + 64 * i + 2 * lane) = d;
  }
  if (lane == 0) p.lse[row] = sum == 0.0f ? -__builtin_huge_valf() : m * kLn2 + logf(sum);
}

// One thread per cached token and key head: the sum over the rows of the head
// group of exp(s - lse).
template <int D>
__global__ void __launch_bounds__(128) attend_weights_kernel(const __grid_constant__ AttendParams p) {
  __shared__ float q_s[D];
  pdl_wait();
  pdl_launch_dependents();
  const int64_t b = blockIdx.z, h = blockIdx.y;
  const int64_t j = static_cast<int64_t>(blockIdx.x) * 128 + threadIdx.x;
  const int n = attend_len(p, b), ps = p.c.page_size;
  int64_t page;
  const bool ok = visible(p, b, j, n, page);
  const int64_t G = p.Hq / p.c.heads;
  const int64_t at = page * p.c.heads + h;
  const float ks = ok ? p.c.k_scale[at] : 0.0f;
  float sum = 0.0f;
  for (int64_t r = 0; r < p.L * G; ++r) {
    const int64_t l = r / G, hq = h * G + r % G;
    const uint16_t* q = reinterpret_cast<const uint16_t*>(p.q + b * p.qb + l * p.ql + hq * p.qh);
    __syncthreads();
    for (int d = threadIdx.x; d < D; d += 128) q_s[d] = __uint_as_float(static_cast<uint32_t>(q[d]) << 16);
    __syncthreads();
    const float lse = p.lse[(b * p.L + l) * p.Hq + hq];
    if (!ok || !(fabsf(lse) < __builtin_huge_valf())) continue;   // a row that attends to nothing gives no weight
    const float s = dot_codes<D>(p.c.k + (at * ps + j % ps) * D, q_s) * ks * p.scale2;
    sum += ex2_approx(s - lse * kLog2e);
  }
  if (j < p.cap) {
    float* w = p.weights + (b * p.c.heads + h) * p.cap + j;
    *w = p.decay == 0.0f ? sum : fmaf(p.decay, *w, sum);
  }
}

}  // namespace dllm

extern "C" {

size_t dllm_cache_attention_workspace_size(int64_t B, int64_t L, int64_t Hq, int64_t heads, int64_t head_dim) {
  (void)B, (void)L, (void)Hq, (void)heads, (void)head_dim;
  return 256;
}

dllm_status dllm_cache_attention(const dllm_kv_cache* cache, const void* q, const int64_t* q_strides, int64_t B,
                                 int64_t L, int64_t Hq, const int32_t* table, int64_t width, const int32_t* lens,
                                 const uint8_t* key_mask, int64_t mask_stride, float scale, void* out, float* lse,
                                 float* weights, float decay, void* workspace, size_t workspace_bytes,
                                 dllm_stream_t stream) {
  using namespace dllm;
  dllm_status st = check_cache(cache, table, B, width);
  if (st != DLLM_OK) return st;
  if (L < 0 || Hq < 1 || Hq % cache->heads != 0) return DLLM_ERR_INVALID_ARGUMENT;
  if (!(scale > 0.0f) || !(scale <= 0x1p+20f) || !(decay >= 0.0f) || !(decay <= 1.0f)) return DLLM_ERR_INVALID_ARGUMENT;
  const int64_t cap = width * cache->page_size;
  if (key_mask && mask_stride < cap) return DLLM_ERR_INVALID_ARGUMENT;
  const int64_t rows = mul_or_neg(mul_or_neg(B, L), Hq);
  if (mul_or_neg(rows, cache->head_dim * 4) < 0 || mul_or_neg(mul_or_neg(B, cache->heads), cap * 4) < 0)
    return DLLM_ERR_INVALID_ARGUMENT;
  if (B == 0 || L == 0) return DLLM_OK;
  if (!q || !q_strides || !lens || !out || !lse) return DLLM_ERR_INVALID_ARGUMENT;
  if (!aligned4(lens) || !aligned4(lse) || !aligned4(weights)) return DLLM_ERR_INVALID_ARGUMENT;
  const int64_t extent[3] = {B, L, Hq};
  for (int i = 0; i < 3; ++i) {
    if (q_strides[i] < 0 || mul_or_neg(mul_or_neg(extent[i], q_strides[i]), 2) < 0) return DLLM_ERR_INVALID_ARGUMENT;
    if (q_strides[i] % 8 != 0) return DLLM_ERR_UNSUPPORTED;
  }
  if (!aligned16(q) || !aligned16(out)) return DLLM_ERR_UNSUPPORTED;
  if (rows > INT32_MAX) return DLLM_ERR_UNSUPPORTED;
  const size_t need = dllm_cache_attention_workspace_size(B, L, Hq, cache->heads, cache->head_dim);
  if (!workspace || workspace_bytes < need) return DLLM_ERR_WORKSPACE;
  if (!aligned16(workspace)) return DLLM_ERR_INVALID_ARGUMENT;
  AttendParams p{};
  p.c = cache_view(*cache);
  p.q = static_cast<const uint8_t*>(q);
  p.qb = q_strides[0] * 2;
  p.ql = q_strides[1] * 2;
  p.qh = q_strides[2] * 2;
  p.B = B;
  p.L = L;
  p.Hq = Hq;
  p.table = table;
  p.lens = lens;
  p.mask = key_mask;
  p.mask_stride = mask_stride;
  p.width = width;
  p.cap = cap;
  p.scale2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634);
  p.out = static_cast<uint16_t*>(out);
  p.lse = lse;
  p.weights = weights;
  p.decay = decay;
  void* args[] = {&p};
  const bool d64 = cache->head_dim == 64;
  st = launch_pdl(d64 ? reinterpret_cast<const void*>(&attend_kernel<64>)
                      : reinterpret_cast<const void*>(&attend_kernel<128>),
                  dim3(static_cast<unsigned>((rows + 3) / 4)), dim3(128), 0, stream, args);
  if (st != DLLM_OK || !weights) return st;
  return launch_pdl(d64 ? reinterpret_cast<const void*>(&attend_weights_kernel<64>)
                        : reinterpret_cast<const void*>(&attend_weights_kernel<128>),
                    dim3(static_cast<unsigned>((cap + 127) / 128), static_cast<unsigned>(cache->heads),
                         static_cast<unsigned>(B)),
                    dim3(128), 0, stream, args);
}

}  // extern "C"
