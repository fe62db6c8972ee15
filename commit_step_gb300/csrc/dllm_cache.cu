// dllm_cache.cu -- writing the paged 8-bit key/value cache: appending tokens
// and evicting the least attended ones.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "dllm_cache.cuh"

namespace dllm {

// ---------------------------------------------------------------------------
// append
// ---------------------------------------------------------------------------
struct AppendParams {
  CacheView c;
  const uint8_t* src[2];       // new keys, new values (bf16)
  int64_t sb[2], sl[2], sh[2];  // their strides in bytes: batch row, token, head
  const int32_t* table;
  const int32_t* start;
  const int32_t* count;        // nullable
  int64_t L, width;
  int32_t cols;                // page columns a call can touch per batch row
};

constexpr int kAppendVec = 8;  // 16-byte vectors (8 dims of one token) a thread holds

// One block per (page column, head, batch row x {keys, values}).  The block
// holds the page's new tokens in registers (one read), finds their largest
// magnitude, fixes the page's scale and writes the codes; tokens the page
// already held are re-expressed when the scale grows.
// Bound: the bf16 read and the e4m3 write, 3 bytes an element.  Measured, 8 x
// 4093 tokens of 8 heads of 128: 36.8 us (5.5 TB/s).
template <int D>
__global__ void __launch_bounds__(256, 4) append_kernel(const __grid_constant__ AppendParams p) {
  __shared__ float red[8];
  pdl_launch_dependents();
  pdl_wait();
  const int64_t b = blockIdx.z >> 1;
  const int kv = blockIdx.z & 1;
  const int h = blockIdx.y;
  const int ps = p.c.page_size;
  const int64_t start = p.start[b];
  int64_t n = p.count ? p.count[b] : p.L;
  n = n < 0 ? 0 : (n > p.L ? p.L : n);
  const int64_t first = start > 0 ? start / ps : 0;
  const int64_t col = first + blockIdx.x;
  const int64_t lo = col * ps;                                   // the page's first position
  const int64_t a = start > lo ? start : lo;
  const int64_t e = start + n < lo + ps ? start + n : lo + ps;   // new positions [a, e) of this page
  if (col >= p.width || a >= e) return;
  const int64_t page = page_at(p.table, p.width, b, col, p.c.pages);
  if (page < 0) return;
  uint8_t* codes = (kv ? p.c.v : p.c.k) + (page * p.c.heads + h) * ps * D;
  float* scale_at = (kv ? p.c.v_scale : p.c.k_scale) + page * p.c.heads + h;
  const uint8_t* src = p.src[kv] + b * p.sb[kv] + h * p.sh[kv];
  constexpr int per_token = D / 8;
  const int from = static_cast<int>(a - lo), to = static_cast<int>(e - lo);  // new slots [from, to)
  uint4 x[kAppendVec];
  // Vector i of this thread: 8 dims of slot slot0 + i step.
  const int slot0 = threadIdx.x / per_token, step = blockDim.x / per_token, d = threadIdx.x % per_token * 8;
  const uint8_t* row = src + (lo + slot0 - start) * p.sl[kv] + d * 2;
  const int64_t row_step = step * p.sl[kv];
#pragma unroll
  for (int i = 0; i < kAppendVec; ++i) {
    const int slot = slot0 + i * step;
    x[i] = make_uint4(0u, 0u, 0u, 0u);
    if (slot >= from && slot < to) x[i] = __ldcs(reinterpret_cast<const uint4*>(row + i * row_step));
  }
  // Largest |bf16| bits (they order as values), two at a time.
  uint32_t top2 = 0;
#pragma unroll
  for (int i = 0; i < kAppendVec; ++i) {
    const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
    for (int q = 0; q < 4; ++q) asm("max.u16x2 %0, %0, %1;" : "+r"(top2) : "r"(w[q] & 0x7FFF7FFFu));
  }
  uint32_t top = max(top2 & 0xFFFFu, top2 >> 16);
  if (top >= 0x7F80u) {                                          // infinities and NaN do not set the scale
    top = 0;
#pragma unroll
    for (int i = 0; i < kAppendVec; ++i) {
      const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const uint32_t u0 = w[q] & 0x7FFFu, u1 = (w[q] >> 16) & 0x7FFFu;
        top = max(top, u0 < 0x7F80u ? u0 : 0u);
        top = max(top, u1 < 0x7F80u ? u1 : 0u);
      }
    }
  }
  const float amax = block_max(__uint_as_float(top << 16), red);
  float s = block_scale(amax);
  if (from > 0) {
    const float old = *scale_at;
    s = fmaxf(s, old);
    if (s != old) {                                              // block-uniform
      for (int v = threadIdx.x; v < from * (D / 4); v += blockDim.x) {
        uint32_t* at = reinterpret_cast<uint32_t*>(codes) + v;
        const uint32_t c = *at;
        float f0, f1, f2, f3;
        f16x2_to_f32(e4m3x2_to_f16x2(c & 0xFFFFu), f0, f1);
        f16x2_to_f32(e4m3x2_to_f16x2(c >> 16), f2, f3);
        *at = e4m3x2(__fdiv_rn(__fmul_rn(f0, old), s), __fdiv_rn(__fmul_rn(f1, old), s)) |
              e4m3x2(__fdiv_rn(__fmul_rn(f2, old), s), __fdiv_rn(__fmul_rn(f3, old), s)) << 16;
      }
    }
    __syncthreads();                                             // every thread has read the old scale
  }
  if (threadIdx.x == 0) *scale_at = s;
  const bool exact = power_of_two(s);
  const float inv = 1.0f / s;
#pragma unroll
  for (int i = 0; i < kAppendVec; ++i) {
    const int slot = slot0 + i * step;
    if (slot < from || slot >= to) continue;
    const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
    uint32_t o[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const float f0 = bf16lo(w[q]), f1 = bf16hi(w[q]);
      // x / s; by a power of two the product with its inverse is the same number
      o[q] = exact ? e4m3x2(f0 * inv, f1 * inv) : e4m3x2(__fdiv_rn(f0, s), __fdiv_rn(f1, s));
    }
    *reinterpret_cast<uint2*>(codes + slot * D + d) = make_uint2(o[0] | o[1] << 16, o[2] | o[3] << 16);
  }
}

// ---------------------------------------------------------------------------
// evict
// ---------------------------------------------------------------------------
struct EvictParams {
  CacheView c;
  const int32_t* table;
  const int32_t* lens;
  const float* weights;        // (B, heads, cap)
  const int32_t* dst_table;
  int32_t* keep;               // (B, heads, budget)
  int32_t* lens_out;           // (B)
  float* weights_out;          // (B, heads, cap)
  int64_t width, dst_width, cap;
  int32_t budget, keep_first, keep_last;
};

constexpr int kSelectThreads = 1024;
constexpr int kSelectBins = 2048;
constexpr int kSelectItems = 4;  // consecutive tokens a thread places at a time
constexpr int kSelectRow = 48 * 1024;  // tokens whose keys a block keeps in shared memory over the passes

__device__ __forceinline__ int seq_len(const int32_t* lens, int64_t b, int64_t cap) {
  const int64_t n = lens[b];
  return static_cast<int>(n < 0 ? 0 : (n > cap ? cap : n));
}

// The order of the weights: NaN lowest, else by value.
__device__ __forceinline__ uint32_t weight_key(float w) { return isnan(w) ? 0u : float_key(w); }

// Sum over the block of (a in the low, b in the high 32 bits) before this
// thread, and the block's total; both below 2^31 in either half.
__device__ __forceinline__ uint64_t block_scan(uint64_t v, uint64_t* warp_sums, uint64_t& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint64_t inc = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint64_t u = __shfl_up_sync(0xFFFFFFFFu, inc, o);
    if (lane >= o) inc += u;
  }
  if (lane == 31) warp_sums[warp] = inc;
  __syncthreads();
  if (warp == 0) {
    uint64_t s = warp_sums[lane];
    uint64_t t = s;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint64_t u = __shfl_up_sync(0xFFFFFFFFu, t, o);
      if (lane >= o) t += u;
    }
    warp_sums[lane] = t;
  }
  __syncthreads();
  total = warp_sums[31];
  const uint64_t before = (warp ? warp_sums[warp - 1] : 0) + inc - v;
  __syncthreads();
  return before;
}

// One block per (head, batch row) picks the tokens that stay: the first
// keep_first, the last keep_last, and among the rest the largest weights (ties
// to the lower slot), by a radix selection of the smallest kept key (11, 11
// and 10 bits) and one ordered pass that numbers the kept tokens.
// Bound: latency of the passes over a row that stays in shared memory (longer
// ones in L2).  Measured, 128 rows of 16384 to 4096: 26 us (30 with the keys
// read again in every pass).
__global__ void __launch_bounds__(kSelectThreads) evict_select_kernel(const __grid_constant__ EvictParams p) {
  __shared__ uint32_t hist[kSelectBins];
  __shared__ uint64_t sums[32];
  __shared__ uint32_t pick_bin, pick_rest;
  extern __shared__ uint32_t row_keys[];                     // the row's keys, when they fit
  pdl_launch_dependents();
  pdl_wait();
  const int h = blockIdx.x;
  const int64_t b = blockIdx.y;
  const int tid = threadIdx.x;
  const int n = seq_len(p.lens, b, p.cap);
  const int m = n < p.budget ? n : p.budget;                 // tokens that stay
  const int f = n < p.keep_first ? n : p.keep_first;
  const int l = n - p.keep_last > f ? n - p.keep_last : f;   // the middle is [f, l)
  const float* w = p.weights + (b * p.c.heads + h) * p.cap;
  uint32_t need = static_cast<uint32_t>(m - (f + n - l));    // of the middle (m >= first + last unless n is small)
  // The need-th largest key of the middle: prefix = its bits found so far.
  uint32_t prefix = 0, mask = 0;
  const bool all = need >= static_cast<uint32_t>(l - f);
  const bool none = need == 0;
  const bool held = n <= kSelectRow;
  if (!all && !none) {
    if (held)
      for (int j = f + tid; j < l; j += kSelectThreads) row_keys[j] = weight_key(w[j]);
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0);
      const uint32_t bins = pass == 2 ? 1024u : 2048u;
      for (uint32_t i = tid; i < bins; i += kSelectThreads) hist[i] = 0;
      __syncthreads();
      for (int j0 = f; j0 < l; j0 += kSelectThreads) {
        const int j = j0 + tid;
        const uint32_t k = j < l ? (held ? row_keys[j] : weight_key(w[j])) : 0u;
        const bool in = j < l && (k & mask) == prefix;
        const uint32_t bin = (k >> shift) & (bins - 1);
        // Weights crowd in a few bins (most tokens draw next to nothing): the
        // bin of the warp's first lane is added once for all its lanes.
        const uint32_t some = __ballot_sync(0xFFFFFFFFu, in);
        if (some == 0u) continue;
        const int lead = __ffs(some) - 1;
        const uint32_t common = __shfl_sync(0xFFFFFFFFu, bin, lead);   // (every lane takes part)
        const bool same = in && bin == common;
        const uint32_t crowd = __ballot_sync(0xFFFFFFFFu, same);
        if ((tid & 31) == lead) atomicAdd(&hist[bin], static_cast<uint32_t>(__popc(crowd)));
        if (in && !same) atomicAdd(&hist[bin], 1u);
      }
      __syncthreads();
      // counts from the top bin down: thread t owns bins 2t and 2t + 1 counted from the top
      const uint32_t c0 = 2u * tid < bins ? hist[bins - 1 - 2 * tid] : 0u;
      const uint32_t c1 = 2u * tid + 1 < bins ? hist[bins - 2 - 2 * tid] : 0u;
      uint64_t total;
      const uint32_t before = static_cast<uint32_t>(block_scan(c0 + c1, sums, total));
      if (before < need && need <= before + c0 + c1) {
        const bool second = need > before + c0;
        pick_bin = bins - 1 - 2 * tid - (second ? 1 : 0);
        pick_rest = need - before - (second ? c0 : 0u);
      }
      __syncthreads();
      prefix |= pick_bin << shift;
      mask |= (bins - 1) << shift;
      need = pick_rest;                                      // still to take among the keys with this prefix
      __syncthreads();
    }
  }
  // Now: keys above `prefix` stay, and the first `need` of those equal to it.
  int32_t* keep = p.keep + (b * p.c.heads + h) * static_cast<int64_t>(p.budget);
  float* wo = p.weights_out + (b * p.c.heads + h) * p.cap;
  uint32_t base_gt = 0, base_eq = 0;
  for (int j0 = 0; j0 < n; j0 += kSelectThreads * kSelectItems) {
    float wj[kSelectItems];
    uint32_t gt = 0, eq = 0;                                 // bits per item
    const int j1 = j0 + tid * kSelectItems;
    if (j1 + kSelectItems <= n) {                            // (rows of cap, a multiple of 16, floats)
#pragma unroll
      for (int i = 0; i < kSelectItems; ++i) wj[i] = w[j1 + i];
    } else {
#pragma unroll
      for (int i = 0; i < kSelectItems; ++i) wj[i] = j1 + i < n ? w[j1 + i] : 0.0f;
    }
#pragma unroll
    for (int i = 0; i < kSelectItems; ++i) {
      const int j = j1 + i;
      const uint32_t k = weight_key(wj[i]);
      const bool middle = j >= f && j < l;
      if (j < n && (!middle || all || (!none && k > prefix))) gt |= 1u << i;
      if (middle && !all && !none && k == prefix) eq |= 1u << i;
    }
    uint64_t total;
    const uint64_t before = block_scan(static_cast<uint64_t>(__popc(gt)) | static_cast<uint64_t>(__popc(eq)) << 32,
                                       sums, total);
    uint32_t g = base_gt + static_cast<uint32_t>(before), q = base_eq + static_cast<uint32_t>(before >> 32);
#pragma unroll
    for (int i = 0; i < kSelectItems; ++i) {
      const bool is_eq = (eq >> i) & 1u;
      const bool stays = ((gt >> i) & 1u) || (is_eq && q < need);
      const uint32_t pos = g + (q < need ? q : need);
      if (stays) {
        keep[pos] = j0 + tid * kSelectItems + i;
        wo[pos] = wj[i];
      }
      g += (gt >> i) & 1u;
      q += is_eq ? 1u : 0u;
    }
    base_gt += static_cast<uint32_t>(total);
    base_eq += static_cast<uint32_t>(total >> 32);
  }
  for (int i = m + tid; i < p.budget; i += kSelectThreads) keep[i] = -1;
  for (int64_t i = m + tid; i < p.cap; i += kSelectThreads) wo[i] = 0.0f;
}

constexpr int kMoveVec = 4;  // 16-byte vectors (16 codes of one token) a thread holds

// One block per (destination page column, head, batch row): gathers the kept
// tokens' keys and values of the page (one read; the chain position -> page ->
// codes is walked once for both, and their bytes are in flight together), finds
// either's largest value, writes them under the page's new scales.
// Bound: one byte read and one written for each element that stays, behind the
// chain.  Measured, 128 x 4096 tokens of 128: 62 us (4.3 TB/s).
template <int D>
__global__ void __launch_bounds__(256, 3) evict_move_kernel(const __grid_constant__ EvictParams p) {
  __shared__ float red[2][8];
  pdl_launch_dependents();
  pdl_wait();
  const int64_t b = blockIdx.z;
  const int h = blockIdx.y;
  const int ps = p.c.page_size;
  const int n = seq_len(p.lens, b, p.cap);
  const int m = n < p.budget ? n : p.budget;
  const int lo = blockIdx.x * ps;
  const int here = m - lo < ps ? m - lo : ps;                    // tokens of this page
  // (lens_out may be lens: the selections have read it, and min(n, budget) comes
  // out the same for a block that reads the new length)
  if (blockIdx.x == 0 && h == 0 && threadIdx.x == 0) p.lens_out[b] = m;
  if (here <= 0) return;
  const int64_t to = page_at(p.dst_table, p.dst_width, b, blockIdx.x, p.c.pages);
  if (to < 0) return;
  const int32_t* keep = p.keep + (b * p.c.heads + h) * static_cast<int64_t>(p.budget) + lo;
  constexpr int per_token = D / 16;
  int64_t at[kMoveVec];                                          // (page, head) and slot of the token, or -1
  int j[kMoveVec];
#pragma unroll
  for (int i = 0; i < kMoveVec; ++i) {
    const int slot = (i * blockDim.x + threadIdx.x) / per_token;
    j[i] = slot < here ? keep[slot] : -1;
  }
#pragma unroll
  for (int i = 0; i < kMoveVec; ++i) {
    at[i] = -1;
    if (j[i] >= 0) {
      const int64_t page = page_at(p.table, p.width, b, j[i] / ps, p.c.pages);
      if (page >= 0) at[i] = page * p.c.heads + h;               // (a token on no page reads as zeros)
    }
  }
  uint4 x[2][kMoveVec];
  float sc[2][kMoveVec];
#pragma unroll
  for (int kv = 0; kv < 2; ++kv)
#pragma unroll
    for (int i = 0; i < kMoveVec; ++i) {
      x[kv][i] = make_uint4(0u, 0u, 0u, 0u);
      sc[kv][i] = 0.0f;
      if (at[i] >= 0) {
        const int d = ((i * blockDim.x + threadIdx.x) % per_token) * 16;
        x[kv][i] = __ldg(reinterpret_cast<const uint4*>((kv ? p.c.v : p.c.k) + (at[i] * ps + j[i] % ps) * D + d));
        sc[kv][i] = (kv ? p.c.v_scale : p.c.k_scale)[at[i]];
      }
    }
  float s[2];
#pragma unroll
  for (int kv = 0; kv < 2; ++kv) {
    float amax = 0.0f;
#pragma unroll
    for (int i = 0; i < kMoveVec; ++i) {
      const uint32_t w[4] = {x[kv][i].x, x[kv][i].y, x[kv][i].z, x[kv][i].w};
      // largest magnitude code (codes order as values), two bytes at a time
      uint32_t top2 = 0;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        asm("max.u16x2 %0, %0, %1;" : "+r"(top2) : "r"(w[q] & 0x007F007Fu));
        asm("max.u16x2 %0, %0, %1;" : "+r"(top2) : "r"((w[q] >> 8) & 0x007F007Fu));
      }
      uint32_t top = max(top2 & 0xFFFFu, top2 >> 16);
      if (top == 0x7Fu) {                                        // NaN does not set the scale
        top = 0;
#pragma unroll 1
        for (int e = 0; e < 16; ++e) {
          const uint32_t c = (w[e >> 2] >> (8 * (e & 3))) & 0x7Fu;
          top = max(top, c < 0x7Fu ? c : 0u);
        }
      }
      float v, unused;
      f16x2_to_f32(e4m3x2_to_f16x2(top), v, unused);
      const float y = __fmul_rn(v, sc[kv][i]);
      if (y < __int_as_float(0x7F800000)) amax = fmaxf(amax, y);
    }
    s[kv] = warp_max_f32(amax);
    if ((threadIdx.x & 31) == 0) red[kv][threadIdx.x >> 5] = s[kv];
  }
  __syncthreads();
  for (int w = 0; w < static_cast<int>(blockDim.x >> 5); ++w) {
    s[0] = fmaxf(s[0], red[0][w]);
    s[1] = fmaxf(s[1], red[1][w]);
  }
#pragma unroll
  for (int kv = 0; kv < 2; ++kv) {
    const float scale = block_scale(s[kv]);
    if (threadIdx.x == 0) (kv ? p.c.v_scale : p.c.k_scale)[to * p.c.heads + h] = scale;
    uint8_t* out = (kv ? p.c.v : p.c.k) + (to * p.c.heads + h) * ps * D;
#pragma unroll
    for (int i = 0; i < kMoveVec; ++i) {
      if (j[i] < 0) continue;
      const int v = i * blockDim.x + threadIdx.x;
      uint32_t w[4] = {x[kv][i].x, x[kv][i].y, x[kv][i].z, x[kv][i].w};
      if (sc[kv][i] != scale) {
        const float ratio = sc[kv][i] / scale;
        if (power_of_two(sc[kv][i]) && power_of_two(scale) && ratio >= 0x1p-14f && ratio <= 0x1p+15f) {
          // Between powers of two the value in units of the new scale is exact
          // in fp16 (a code has 4 bits and is at least 2^-9; fp16 goes to 2^-24).
          const uint32_t r16 = ((__float_as_uint(ratio) >> 23) - 127u + 15u) << 10, r2 = r16 | r16 << 16;
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            uint32_t lo = e4m3x2_to_f16x2(w[q] & 0xFFFFu), hi = e4m3x2_to_f16x2(w[q] >> 16);
            asm("mul.rn.f16x2 %0, %0, %1;" : "+r"(lo) : "r"(r2));
            asm("mul.rn.f16x2 %0, %0, %1;" : "+r"(hi) : "r"(r2));
            uint16_t c0, c1;
            asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(c0) : "r"(lo));
            asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(c1) : "r"(hi));
            w[q] = c0 | static_cast<uint32_t>(c1) << 16;
          }
        } else {
#pragma unroll 1
          for (int q = 0; q < 4; ++q) {
            float f[4];
            f16x2_to_f32(e4m3x2_to_f16x2(w[q] & 0xFFFFu), f[0], f[1]);
            f16x2_to_f32(e4m3x2_to_f16x2(w[q] >> 16), f[2], f[3]);
#pragma unroll
            for (int e = 0; e < 4; ++e) f[e] = __fdiv_rn(__fmul_rn(f[e], sc[kv][i]), scale);
            w[q] = e4m3x2(f[0], f[1]) | e4m3x2(f[2], f[3]) << 16;
          }
        }
      }
      *reinterpret_cast<uint4*>(out + static_cast<int64_t>(v) * 16) = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
}

}  // namespace dllm

extern "C" {

dllm_status dllm_cache_append(const dllm_kv_cache* cache, const void* k, const void* v, const int64_t* k_strides,
                              const int64_t* v_strides, int64_t B, int64_t L, const int32_t* table, int64_t width,
                              const int32_t* start, const int32_t* count, dllm_stream_t stream) {
  using namespace dllm;
  const dllm_status st = check_cache(cache, table, B, width);
  if (st != DLLM_OK) return st;
  if (L < 0 || L > INT32_MAX) return DLLM_ERR_INVALID_ARGUMENT;
  if (B == 0 || L == 0) return DLLM_OK;
  if (!k || !v || !k_strides || !v_strides || !start || !aligned4(start) || !aligned4(count))
    return DLLM_ERR_INVALID_ARGUMENT;
  const int64_t* strides[2] = {k_strides, v_strides};
  const int64_t extent[3] = {B, L, cache->heads};
  for (const int64_t* s : strides)
    for (int i = 0; i < 3; ++i) {
      if (s[i] < 0 || mul_or_neg(mul_or_neg(extent[i], s[i]), 2) < 0) return DLLM_ERR_INVALID_ARGUMENT;
      if (s[i] % 8 != 0) return DLLM_ERR_UNSUPPORTED;
    }
  if (!aligned16(k) || !aligned16(v)) return DLLM_ERR_UNSUPPORTED;
  AppendParams p{};
  p.c = cache_view(*cache);
  p.src[0] = static_cast<const uint8_t*>(k);
  p.src[1] = static_cast<const uint8_t*>(v);
  for (int i = 0; i < 2; ++i) {
    p.sb[i] = strides[i][0] * 2;
    p.sl[i] = strides[i][1] * 2;
    p.sh[i] = strides[i][2] * 2;
  }
  p.table = table;
  p.start = start;
  p.count = count;
  p.L = L;
  p.width = width;
  const int64_t ps = cache->page_size;
  p.cols = static_cast<int32_t>(std::min<int64_t>(width, (L + ps - 1) / ps + 1));
  const unsigned threads = static_cast<unsigned>(std::max<int64_t>(32, ps * cache->head_dim / (8 * kAppendVec)));
  void* args[] = {&p};
  if (2 * B > 65535) return DLLM_ERR_UNSUPPORTED;
  return launch_pdl(cache->head_dim == 64 ? reinterpret_cast<const void*>(&append_kernel<64>)
                                          : reinterpret_cast<const void*>(&append_kernel<128>),
                    dim3(static_cast<unsigned>(p.cols), static_cast<unsigned>(cache->heads),
                         static_cast<unsigned>(2 * B)),
                    dim3(threads), 0, stream, args);
}

dllm_status dllm_cache_evict(const dllm_kv_cache* cache, const int32_t* table, int64_t width, const int32_t* lens,
                             int64_t B, const float* weights, int64_t budget, int64_t keep_first, int64_t keep_last,
                             const int32_t* dst_table, int64_t dst_width, int32_t* keep, int32_t* lens_out,
                             float* weights_out, dllm_stream_t stream) {
  using namespace dllm;
  dllm_status st = check_cache(cache, table, B, width);
  if (st == DLLM_OK) st = check_cache(cache, dst_table, B, dst_width);
  if (st != DLLM_OK) return st;
  if (budget < 1 || keep_first < 0 || keep_last < 0 || keep_first > budget || keep_last > budget - keep_first)
    return DLLM_ERR_INVALID_ARGUMENT;
  const int64_t cap = width * cache->page_size;
  if (budget > dst_width * cache->page_size) return DLLM_ERR_INVALID_ARGUMENT;
  if (mul_or_neg(mul_or_neg(B, cache->heads), mul_or_neg(std::max(cap, budget), 4)) < 0)
    return DLLM_ERR_INVALID_ARGUMENT;
  if (2 * B > 65535) return DLLM_ERR_UNSUPPORTED;
  if (B == 0) return DLLM_OK;
  if (!lens || !weights || !keep || !lens_out || !weights_out) return DLLM_ERR_INVALID_ARGUMENT;
  if (!aligned4(lens) || !aligned4(weights) || !aligned4(keep) || !aligned4(lens_out) || !aligned4(weights_out))
    return DLLM_ERR_INVALID_ARGUMENT;
  // A row's weights are stored while other rows' are still read.
  const uintptr_t w0 = reinterpret_cast<uintptr_t>(weights), w1 = reinterpret_cast<uintptr_t>(weights_out);
  if ((w0 < w1 ? w1 - w0 : w0 - w1) < static_cast<uintptr_t>(B) * cache->heads * cap * 4)
    return DLLM_ERR_INVALID_ARGUMENT;
  EvictParams p{};
  p.c = cache_view(*cache);
  p.table = table;
  p.lens = lens;
  p.weights = weights;
  p.dst_table = dst_table;
  p.keep = keep;
  p.lens_out = lens_out;
  p.weights_out = weights_out;
  p.width = width;
  p.dst_width = dst_width;
  p.cap = cap;
  p.budget = static_cast<int32_t>(budget);
  p.keep_first = static_cast<int32_t>(keep_first);
  p.keep_last = static_cast<int32_t>(keep_last);
  void* args[] = {&p};
  // (set on every call: the current device may be another one)
  if (cap * 4 > 32 * 1024 &&
      cudaFuncSetAttribute(reinterpret_cast<const void*>(&evict_select_kernel),
                           cudaFuncAttributeMaxDynamicSharedMemorySize, kSelectRow * 4) != cudaSuccess)
    return DLLM_ERR_CUDA;
  st = launch_pdl(reinterpret_cast<const void*>(&evict_select_kernel),
                  dim3(static_cast<unsigned>(cache->heads), static_cast<unsigned>(B)), dim3(kSelectThreads),
                  static_cast<size_t>(std::min<int64_t>(cap, kSelectRow)) * 4, stream, args);
  if (st != DLLM_OK) return st;
  const int64_t ps = cache->page_size;
  const unsigned threads = static_cast<unsigned>(std::max<int64_t>(32, ps * cache->head_dim / (16 * kMoveVec)));
  const int64_t cols = (std::min(budget, cap) + ps - 1) / ps;
  return launch_pdl(cache->head_dim == 64 ? reinterpret_cast<const void*>(&evict_move_kernel<64>)
                                          : reinterpret_cast<const void*>(&evict_move_kernel<128>),
                    dim3(static_cast<unsigned>(cols), static_cast<unsigned>(cache->heads), static_cast<unsigned>(B)),
                    dim3(threads), 0, stream, args);
}

}  // extern "C"
