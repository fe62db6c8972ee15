// dllm_embed.cu -- the embedding of a canvas, and its gradient by sorted tokens
// (sm_103a).
//
// Forward: out_i = scale weight[token_i], rows copied in 16-byte vectors.
//
// Backward: grad_weight[v] = scale sum over the positions i of token v of
// grad_i, summed in fp32 in an order that depends on the tokens alone.  The
// positions are sorted by token (a stable radix sort), the sorted list is cut
// into chunks of equal length, and a warp sums the runs of equal tokens in its
// chunk for a slab of columns: however uneven the tokens (half of a noised canvas
// is the mask token), every warp reads the same number of rows.  A run that ends
// inside the chunk it began in is written; the parts of a run that crosses chunks
// go to a workspace and are added in the order of the chunks by a second kernel.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "../../include/dllmcommit.h"
#include "dllm_device.cuh"
#include "dllm_launch.cuh"

namespace dllm {

struct EmbedTokens {
  const int32_t* at;
  int64_t L, stride, T, V;
  // Token i in the order of the rows; V for an id that has no row.
  __device__ __forceinline__ int32_t operator[](int64_t i) const {
    const int32_t v = at[i / L * stride + i % L];
    return v < 0 || v >= V ? static_cast<int32_t>(V) : v;
  }
};

// ---------------------------------------------------------------------------
// forward
// ---------------------------------------------------------------------------
constexpr int kEmThreads = 256;
constexpr int kEmVecs = 4;                              // 16-byte vectors of a lane: a warp copies 2 KB of a row

template <bool BF16>
__device__ __forceinline__ uint4 em_scale(uint4 v, float s) {
  uint4 o;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t w = (&v.x)[i];
    if (BF16)
      asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"((&o.x)[i]) : "f"(bf16hi(w) * s), "f"(bf16lo(w) * s));
    else
      (&o.x)[i] = __float_as_uint(__uint_as_float(w) * s);
  }
  return o;
}

template <bool BF16>
__global__ void __launch_bounds__(kEmThreads) embed_kernel(EmbedTokens tok, const uint8_t* weight, int64_t row_bytes,
                                                           int64_t vecs, float scale, uint8_t* out) {
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int64_t slabs = (vecs + 32 * kEmVecs - 1) / (32 * kEmVecs);
  const int64_t units = tok.T * slabs;
  const int64_t step = static_cast<int64_t>(gridDim.x) * (kEmThreads / 32);
  for (int64_t u = blockIdx.x * static_cast<int64_t>(kEmThreads / 32) + (threadIdx.x >> 5); u < units; u += step) {
    const int64_t i = u / slabs, q0 = (u - i * slabs) * (32 * kEmVecs) + lane;
    const int32_t v = tok[i];
    const uint4* from = reinterpret_cast<const uint4*>(weight + v * row_bytes);
    uint4* to = reinterpret_cast<uint4*>(out) + i * vecs;
    uint4 x[kEmVecs];
#pragma unroll
    for (int e = 0; e < kEmVecs; ++e)
      x[e] = v < tok.V && q0 + 32 * e < vecs ? __ldg(from + q0 + 32 * e) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
    for (int e = 0; e < kEmVecs; ++e)
      if (q0 + 32 * e < vecs) to[q0 + 32 * e] = scale == 1.0f ? x[e] : em_scale<BF16>(x[e], scale);
  }
}

// ---------------------------------------------------------------------------
// the sort
// ---------------------------------------------------------------------------
constexpr int kSortBits = 10;
constexpr int kSortBins = 1 << kSortBits;
constexpr int kSortThreads = 256;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kSortPerWarp = 256;                       // keys of a warp, in their order
constexpr int kSortTile = kSortWarps * kSortPerWarp;    // keys of a block

struct SortKeys {
  EmbedTokens tok;                // the first pass's keys, with their positions
  const int32_t *key, *pos;       // a later pass's (key null: the first pass)
  int32_t* key_out;
  int32_t* pos_out;
  int32_t* table;                 // (bins, blocks)
  int32_t shift, blocks;
  __device__ __forceinline__ int32_t at(int64_t i) const { return key ? key[i] : tok[i]; }
};

// Counts a warp's digits into its row of `count`, in order; with RANK the
// row holds the places its next keys of a digit take.
template <bool RANK>
__device__ __forceinline__ void sort_warp(const SortKeys& p, int64_t first, int32_t* count) {
  const int lane = threadIdx.x & 31;
  for (int64_t i = first; i < first + kSortPerWarp; i += 32) {
    if (i >= p.tok.T) break;                             // warp-uniform
    const bool in = i + lane < p.tok.T;
    const int32_t key = in ? p.at(i + lane) : -1;
    const int digit = in ? (key >> p.shift) & (kSortBins - 1) : kSortBins;
    const uint32_t same = __match_any_sync(0xFFFFFFFFu, digit);
    const int before = __popc(same & ((1u << lane) - 1u));
    if (RANK) {
      const int32_t base = in ? count[digit] : 0;
      __syncwarp();
      if (in) {
        p.key_out[base + before] = key;
        p.pos_out[base + before] = p.key ? p.pos[i + lane] : static_cast<int32_t>(i + lane);
        if (before == 0) count[digit] = base + __popc(same);
      }
    } else if (in && before == 0) {
      count[digit] += __popc(same);
    }
    __syncwarp();
  }
}

__global__ void __launch_bounds__(kSortThreads) embed_sort_count_kernel(SortKeys p) {
  __shared__ int32_t count[kSortWarps][kSortBins];
  for (int i = threadIdx.x; i < kSortWarps * kSortBins; i += kSortThreads) (&count[0][0])[i] = 0;
  __syncthreads();
  pdl_wait();
  pdl_launch_dependents();
  const int warp = threadIdx.x >> 5;
  sort_warp<false>(p, (blockIdx.x * static_cast<int64_t>(kSortWarps) + warp) * kSortPerWarp, count[warp]);
  __syncthreads();
  for (int b = threadIdx.x; b < kSortBins; b += kSortThreads) {
    int32_t s = 0;
    for (int w = 0; w < kSortWarps; ++w) s += count[w][b];
    p.table[static_cast<int64_t>(b) * p.blocks + blockIdx.x] = s;
  }
}

// Exclusive sums over the table, bins outer.
__global__ void __launch_bounds__(1024) embed_sort_scan_kernel(int32_t* table, int64_t n) {
  __shared__ int32_t sums[32];
  pdl_wait();
  pdl_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t per = (n + 1023) / 1024, a = min(n, tid * per), e = min(n, a + per);
  int32_t total = 0;
  for (int64_t i = a; i < e; ++i) total += table[i];
  int32_t scan = total;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int32_t v = __shfl_up_sync(0xFFFFFFFFu, scan, o);
    if (lane >= o) scan += v;
  }
  if (lane == 31) sums[warp] = scan;
  __syncthreads();
  int32_t before = scan - total;
  for (int w = 0; w < warp; ++w) before += sums[w];
  for (int64_t i = a; i < e; ++i) {
    const int32_t v = table[i];
    table[i] = before;
    before += v;
  }
}

__global__ void __launch_bounds__(kSortThreads) embed_sort_place_kernel(SortKeys p) {
  __shared__ int32_t count[kSortWarps][kSortBins];
  for (int i = threadIdx.x; i < kSortWarps * kSortBins; i += kSortThreads) (&count[0][0])[i] = 0;
  __syncthreads();
  pdl_wait();
  pdl_launch_dependents();
  const int warp = threadIdx.x >> 5;
  const int64_t first = (blockIdx.x * static_cast<int64_t>(kSortWarps) + warp) * kSortPerWarp;
  sort_warp<false>(p, first, count[warp]);
  __syncthreads();
  for (int b = threadIdx.x; b < kSortBins; b += kSortThreads) {
    int32_t s = p.table[static_cast<int64_t>(b) * p.blocks + blockIdx.x];
    for (int w = 0; w < kSortWarps; ++w) {
      const int32_t c = count[w][b];
      count[w][b] = s;
      s += c;
    }
  }
  __syncthreads();
  sort_warp<true>(p, first, count[warp]);
}

// ---------------------------------------------------------------------------
// the sums
// ---------------------------------------------------------------------------
constexpr int kRunChunk = 64;                           // sorted positions of a warp
constexpr int kRunWarps = 8;

struct RunParams {
  const int32_t *key, *pos;     // sorted
  int64_t T, V;
  const uint8_t* grad;
  int64_t vecs;                 // 16-byte vectors of a grad row
  float scale;
  void* out;
  int64_t out_stride;
  int32_t accumulate;
  float* part;                  // (chunks, 2, columns)
  int64_t chunks;
  int32_t slabs;                // of 32 vectors
};

// A lane's columns of grad rows: 8 of bf16, 4 of fp32.
template <bool BF16>
struct RunLane {
  static constexpr int kCols = BF16 ? 8 : 4;
  float s[kCols];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int e = 0; e < kCols; ++e) s[e] = 0.0f;
  }
  __device__ __forceinline__ void add(uint4 v) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t w = (&v.x)[i];
      if (BF16) {
        s[2 * i] += bf16lo(w);
        s[2 * i + 1] += bf16hi(w);
      } else {
        s[i % kCols] += __uint_as_float(w);
      }
    }
  }
};

// The sum of a run, scaled, to its row of the gradient.
template <bool OUT16, int COLS>
__device__ __forceinline__ void run_write(const RunParams& p, int64_t row, int64_t col, const float (&s)[COLS]) {
  if (OUT16) {
    uint16_t* at = static_cast<uint16_t*>(p.out) + row * p.out_stride + col;
    uint32_t w[COLS / 2];
    if (COLS == 8) {
      uint4 o = p.accumulate ? *reinterpret_cast<const uint4*>(at) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
      for (int i = 0; i < COLS / 2; ++i) {
        const float lo = fmaf(s[2 * i], p.scale, p.accumulate ? bf16lo((&o.x)[i]) : 0.0f);
        const float hi = fmaf(s[2 * i + 1], p.scale, p.accumulate ? bf16hi((&o.x)[i]) : 0.0f);
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(hi), "f"(lo));
      }
      *reinterpret_cast<uint4*>(at) = make_uint4(w[0], w[1], w[2 % (COLS / 2)], w[3 % (COLS / 2)]);
    } else {
      uint2 o = p.accumulate ? *reinterpret_cast<const uint2*>(at) : make_uint2(0u, 0u);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float lo = fmaf(s[2 * i], p.scale, p.accumulate ? bf16lo((&o.x)[i]) : 0.0f);
        const float hi = fmaf(s[2 * i + 1], p.scale, p.accumulate ? bf16hi((&o.x)[i]) : 0.0f);
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(hi), "f"(lo));
      }
      *reinterpret_cast<uint2*>(at) = make_uint2(w[0], w[1]);
    }
  } else {
    float4* at = reinterpret_cast<float4*>(static_cast<float*>(p.out) + row * p.out_stride + col);
#pragma unroll
    for (int i = 0; i < COLS / 4; ++i) {
      const float4 o = p.accumulate ? at[i] : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      at[i] = make_float4(fmaf(s[4 * i], p.scale, o.x), fmaf(s[4 * i + 1], p.scale, o.y), fmaf(s[4 * i + 2], p.scale, o.z),
                          fmaf(s[4 * i + 3], p.scale, o.w));
    }
  }
}

template <bool BF16, bool OUT16>
__global__ void __launch_bounds__(kRunWarps * 32) embed_sum_kernel(RunParams p) {
  constexpr int kCols = RunLane<BF16>::kCols;
  constexpr int kAhead = 8;
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int64_t u = blockIdx.x * static_cast<int64_t>(kRunWarps) + (threadIdx.x >> 5);
  const int64_t chunk = u / p.slabs;
  if (chunk >= p.chunks) return;
  const int64_t vec = (u - chunk * p.slabs) * 32 + lane;
  const bool live = vec < p.vecs;
  const int64_t a = chunk * kRunChunk, e = min(p.T, a + kRunChunk);
  // The chunk's tokens and positions, two a lane, and its neighbours' tokens.
  const int32_t none = static_cast<int32_t>(p.V);
  int32_t key[2], pos[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const bool in = a + 32 * h + lane < e;
    key[h] = in ? p.key[a + 32 * h + lane] : none;
    pos[h] = in ? p.pos[a + 32 * h + lane] : 0;
  }
  const int32_t left = a > 0 ? p.key[a - 1] : -1, right = e < p.T ? p.key[e] : -1;
  const uint4* grad = reinterpret_cast<const uint4*>(p.grad) + vec;
  RunLane<BF16> sum;
  sum.clear();
  int32_t run = __shfl_sync(0xFFFFFFFFu, key[0], 0);
  bool first = true;
  auto flush = [&](bool last) {
    if (run == none || !live) return;
    const bool crosses = (first && left == run) || (last && right == run);
    if (crosses) {
      float* at = p.part + ((chunk * 2 + (first ? 0 : 1)) * p.vecs + vec) * kCols;
#pragma unroll
      for (int i = 0; i < kCols; i += 4)
        *reinterpret_cast<float4*>(at + i) = make_float4(sum.s[i], sum.s[i + 1], sum.s[i + 2], sum.s[i + 3]);
    } else {
      run_write<OUT16, kCols>(p, run, vec * kCols, sum.s);
    }
  };
#pragma unroll 1
  for (int i = 0; i < kRunChunk; i += kAhead) {
    uint4 x[kAhead];
    int32_t k[kAhead];
#pragma unroll
    for (int q = 0; q < kAhead; ++q) {
      const int j = i + q;
      k[q] = __shfl_sync(0xFFFFFFFFu, j < 32 ? key[0] : key[1], j & 31);
      const int64_t at = __shfl_sync(0xFFFFFFFFu, j < 32 ? pos[0] : pos[1], j & 31);
      x[q] = k[q] != none && live ? __ldcs(grad + at * p.vecs) : make_uint4(0u, 0u, 0u, 0u);
    }
#pragma unroll
    for (int q = 0; q < kAhead; ++q) {
      if (k[q] != run) {                                 // warp-uniform
        flush(false);
        sum.clear();
        run = k[q];
        first = false;
      }
      sum.add(x[q]);
    }
    if (run == none) break;                              // (sorted last)
  }
  flush(true);
}

// Runs that cross chunks: the chunk a run begins in adds its parts.
template <bool BF16, bool OUT16>
__global__ void __launch_bounds__(kRunWarps * 32) embed_join_kernel(RunParams p) {
  constexpr int kCols = RunLane<BF16>::kCols;
  __shared__ float4 share[kRunWarps][kCols / 4][32];
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t chunk = blockIdx.x / p.slabs;
  const int64_t vec = (blockIdx.x - chunk * p.slabs) * 32 + lane;
  const int64_t a = chunk * kRunChunk, e = a + kRunChunk;
  if (e >= p.T) return;
  const int32_t run = p.key[e - 1];
  if (run >= p.V || p.key[e] != run) return;             // the chunk's last run ends with it
  const bool whole = p.key[a] == run;                    // (it is the chunk's first run too)
  if (whole && a > 0 && p.key[a - 1] == run) return;     // and began before it
  // The last chunk the run reaches: keys are sorted, so the first key of a later
  // chunk is `run` exactly while the run goes on.
  int64_t lo = chunk + 1, hi = p.chunks - 1;
  while (lo < hi) {
    const int64_t mid = (lo + hi + 1) / 2;
    if (p.key[mid * kRunChunk] == run) lo = mid; else hi = mid - 1;
  }
  const int64_t parts = lo - chunk + 1;
  const int64_t p0 = parts * warp / kRunWarps, p1 = parts * (warp + 1) / kRunWarps;
  float s[kCols];
#pragma unroll
  for (int i = 0; i < kCols; ++i) s[i] = 0.0f;
  const bool live = vec < p.vecs;
  if (live) {
#pragma unroll 4
    for (int64_t q = p0; q < p1; ++q) {
      const int64_t slot = (chunk + q) * 2 + (q == 0 && !whole ? 1 : 0);
      const float4* at = reinterpret_cast<const float4*>(p.part + (slot * p.vecs + vec) * kCols);
#pragma unroll
      for (int i = 0; i < kCols / 4; ++i) {
        const float4 v = at[i];
        s[4 * i] += v.x, s[4 * i + 1] += v.y, s[4 * i + 2] += v.z, s[4 * i + 3] += v.w;
      }
    }
  }
#pragma unroll
  for (int i = 0; i < kCols / 4; ++i) share[warp][i][lane] = make_float4(s[4 * i], s[4 * i + 1], s[4 * i + 2], s[4 * i + 3]);
  __syncthreads();
  if (warp == 0 && live) {
    for (int w = 1; w < kRunWarps; ++w)
#pragma unroll
      for (int i = 0; i < kCols / 4; ++i) {
        const float4 v = share[w][i][lane];
        s[4 * i] += v.x, s[4 * i + 1] += v.y, s[4 * i + 2] += v.z, s[4 * i + 3] += v.w;
      }
    run_write<OUT16, kCols>(p, run, vec * kCols, s);
  }
}

// Rows of the gradient that no token names: zero.
__global__ void __launch_bounds__(256) embed_zero_kernel(uint8_t* out, int64_t row_bytes, int64_t vecs, int64_t V) {
  pdl_wait();
  pdl_launch_dependents();
  for (int64_t v = blockIdx.x; v < V; v += gridDim.x) {
    uint4* row = reinterpret_cast<uint4*>(out + v * row_bytes);
    for (int64_t q = threadIdx.x; q < vecs; q += 256) row[q] = make_uint4(0u, 0u, 0u, 0u);
  }
}

}  // namespace dllm

namespace {

using namespace dllm;

constexpr int64_t kEmMaxT = int64_t{1} << 30;

int em_sms() {
  static int sms[64] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  if (sms[dev] == 0) {
    int n = 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
      (void)cudaGetLastError();
      return 0;
    }
    sms[dev] = n;
  }
  return sms[dev];
}

struct EmPlan {
  int32_t passes, blocks;
  int64_t chunks;
  size_t key[2], pos[2], table, part, bytes;
};

EmPlan em_plan(int64_t T, int64_t V, int64_t d) {
  EmPlan e{};
  int bits = 0;
  while (bits < 31 && (V >> bits) != 0) ++bits;          // keys 0 .. V
  e.passes = (bits + kSortBits - 1) / kSortBits;
  e.blocks = static_cast<int32_t>((T + kSortTile - 1) / kSortTile);
  e.chunks = (T + kRunChunk - 1) / kRunChunk;
  size_t at = 0;
  auto take = [&at](int64_t bytes) {
    const size_t here = at;
    at += static_cast<size_t>((bytes + 255) / 256 * 256);
    return here;
  };
  for (int i = 0; i < 2; ++i) {
    e.key[i] = take(4 * T);
    e.pos[i] = take(4 * T);
  }
  e.table = take(4 * static_cast<int64_t>(kSortBins) * e.blocks);
  e.part = take(8 * e.chunks * d);
  e.bytes = at;
  return e;
}

// Checks that both directions share.
dllm_status em_check(const int32_t* tokens, int64_t B, int64_t L, int64_t stride, const void* rows, int64_t V, int64_t d,
                     int64_t row_stride, dllm_dtype dt) {
  if (B < 0 || L < 0 || V < 1 || V > INT32_MAX || d < 1 || stride < L || row_stride < d) return DLLM_ERR_INVALID_ARGUMENT;
  if (dt != DLLM_F32 && dt != DLLM_BF16) return DLLM_ERR_INVALID_ARGUMENT;
  const int64_t T = mul_or_neg(B, L);
  if (T < 0 || mul_or_neg(mul_or_neg(B, stride), 4) < 0 || mul_or_neg(mul_or_neg(T, d), 8) < 0 ||
      mul_or_neg(mul_or_neg(V, row_stride), 4) < 0)
    return DLLM_ERR_INVALID_ARGUMENT;
  if (T > 0 && (!tokens || !aligned4(tokens))) return DLLM_ERR_INVALID_ARGUMENT;
  if (!rows && T > 0) return DLLM_ERR_INVALID_ARGUMENT;
  const int64_t group = dt == DLLM_BF16 ? 8 : 4;
  if (!aligned16(rows) || d % group != 0 || row_stride % group != 0) return DLLM_ERR_UNSUPPORTED;
  if (T > kEmMaxT) return DLLM_ERR_UNSUPPORTED;
  return DLLM_OK;
}

}  // namespace

extern "C" {

dllm_status dllm_embed_tokens(const int32_t* tokens, int64_t B, int64_t L, int64_t token_stride, const void* weight,
                              dllm_dtype dt, int64_t V, int64_t d, int64_t weight_stride, float scale, void* out,
                              dllm_stream_t stream) {
  const dllm_status st = em_check(tokens, B, L, token_stride, weight, V, d, weight_stride, dt);
  if (st != DLLM_OK) return st;
  if (!std::isfinite(scale)) return DLLM_ERR_INVALID_ARGUMENT;
  const int64_t T = B * L;
  if (T == 0) return DLLM_OK;
  if (!out) return DLLM_ERR_INVALID_ARGUMENT;
  if (!aligned16(out)) return DLLM_ERR_UNSUPPORTED;
  const int sms = em_sms();
  if (sms == 0) return DLLM_ERR_CUDA;
  const int64_t size = dt == DLLM_BF16 ? 2 : 4;
  EmbedTokens tok{tokens, L, token_stride, T, V};
  const uint8_t* w = static_cast<const uint8_t*>(weight);
  int64_t row_bytes = weight_stride * size, vecs = d * size / 16;
  uint8_t* o = static_cast<uint8_t*>(out);
  const int64_t units = T * ((vecs + 32 * kEmVecs - 1) / (32 * kEmVecs));
  const int64_t blocks = std::min<int64_t>((units + kEmThreads / 32 - 1) / (kEmThreads / 32), sms * 8);
  void* args[] = {&tok, &w, &row_bytes, &vecs, &scale, &o};
  const void* kernel = dt == DLLM_BF16 ? reinterpret_cast<const void*>(&embed_kernel<true>)
                                       : reinterpret_cast<const void*>(&embed_kernel<false>);
  return launch_pdl(kernel, dim3(static_cast<unsigned>(blocks)), dim3(kEmThreads), 0, stream, args);
}

size_t dllm_embed_tokens_backward_workspace_size(int64_t T, int64_t V, int64_t d) {
  if (T <= 0 || V <= 0 || d <= 0 || T > kEmMaxT || V > INT32_MAX || mul_or_neg(T, d) < 0) return 0;
  return em_plan(T, V, d).bytes;
}

dllm_status dllm_embed_tokens_backward(const int32_t* tokens, int64_t B, int64_t L, int64_t token_stride, const void* grad,
                                       dllm_dtype grad_dt, int64_t V, int64_t d, float scale, void* grad_weight,
                                       dllm_dtype grad_weight_dt, int64_t grad_weight_stride, int32_t accumulate,
                                       void* workspace, size_t workspace_bytes, dllm_stream_t stream) {
  if (grad_weight_dt != DLLM_F32 && grad_weight_dt != DLLM_BF16) return DLLM_ERR_INVALID_ARGUMENT;
  const dllm_status st = em_check(tokens, B, L, token_stride, grad, V, d, grad_weight_stride, grad_dt);
  if (st != DLLM_OK) return st;
  if (!std::isfinite(scale) || !grad_weight) return DLLM_ERR_INVALID_ARGUMENT;
  const int64_t T = B * L, size = grad_weight_dt == DLLM_BF16 ? 2 : 4;
  const int64_t group = grad_weight_dt == DLLM_BF16 ? 8 : 4;
  if (!aligned16(grad_weight) || d % group != 0 || grad_weight_stride % group != 0) return DLLM_ERR_UNSUPPORTED;
  if (T > 0 && (!workspace || workspace_bytes < dllm_embed_tokens_backward_workspace_size(T, V, d))) return DLLM_ERR_WORKSPACE;
  if (T > 0 && !aligned16(workspace)) return DLLM_ERR_INVALID_ARGUMENT;
  const int sms = em_sms();
  if (sms == 0) return DLLM_ERR_CUDA;
  dllm_status ok = DLLM_OK;
  if (!accumulate) {
    uint8_t* o = static_cast<uint8_t*>(grad_weight);
    int64_t row_bytes = grad_weight_stride * size, vecs = d * size / 16;
    void* args[] = {&o, &row_bytes, &vecs, &V};
    ok = launch_pdl(reinterpret_cast<const void*>(&embed_zero_kernel), dim3(static_cast<unsigned>(std::min<int64_t>(V, sms * 8))),
                    dim3(256), 0, stream, args);
  }
  if (ok != DLLM_OK || T == 0) return ok;
  const EmPlan e = em_plan(T, V, d);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  SortKeys k{};
  k.tok = EmbedTokens{tokens, L, token_stride, T, V};
  k.table = reinterpret_cast<int32_t*>(ws + e.table);
  k.blocks = e.blocks;
  int64_t cells = static_cast<int64_t>(kSortBins) * e.blocks;
  for (int i = 0; i < e.passes && ok == DLLM_OK; ++i) {
    k.key = i == 0 ? nullptr : reinterpret_cast<int32_t*>(ws + e.key[(i + 1) & 1]);
    k.pos = i == 0 ? nullptr : reinterpret_cast<int32_t*>(ws + e.pos[(i + 1) & 1]);
    k.key_out = reinterpret_cast<int32_t*>(ws + e.key[i & 1]);
    k.pos_out = reinterpret_cast<int32_t*>(ws + e.pos[i & 1]);
    k.shift = i * kSortBits;
    void* args[] = {&k};
    void* sargs[] = {&k.table, &cells};
    const dim3 grid(static_cast<unsigned>(e.blocks));
    ok = launch_pdl(reinterpret_cast<const void*>(&embed_sort_count_kernel), grid, dim3(kSortThreads), 0, stream, args);
    if (ok == DLLM_OK)
      ok = launch_pdl(reinterpret_cast<const void*>(&embed_sort_scan_kernel), dim3(1), dim3(1024), 0, stream, sargs);
    if (ok == DLLM_OK)
      ok = launch_pdl(reinterpret_cast<const void*>(&embed_sort_place_kernel), grid, dim3(kSortThreads), 0, stream, args);
  }
  if (ok != DLLM_OK) return ok;
  RunParams r{};
  r.key = k.key_out;
  r.pos = k.pos_out;
  r.T = T;
  r.V = V;
  r.grad = static_cast<const uint8_t*>(grad);
  r.vecs = d * (grad_dt == DLLM_BF16 ? 2 : 4) / 16;
  r.scale = scale;
  r.out = grad_weight;
  r.out_stride = grad_weight_stride;
  r.accumulate = accumulate != 0 ? 1 : 0;
  r.part = reinterpret_cast<float*>(ws + e.part);
  r.chunks = e.chunks;
  r.slabs = static_cast<int32_t>((r.vecs + 31) / 32);
  const int64_t units = r.chunks * r.slabs;
  if (units > INT32_MAX) return DLLM_ERR_UNSUPPORTED;
  const bool in16 = grad_dt == DLLM_BF16, out16 = grad_weight_dt == DLLM_BF16;
  const void* sum = in16 ? (out16 ? reinterpret_cast<const void*>(&embed_sum_kernel<true, true>)
                                  : reinterpret_cast<const void*>(&embed_sum_kernel<true, false>))
                         : (out16 ? reinterpret_cast<const void*>(&embed_sum_kernel<false, true>)
                                  : reinterpret_cast<const void*>(&embed_sum_kernel<false, false>));
  const void* join = in16 ? (out16 ? reinterpret_cast<const void*>(&embed_join_kernel<true, true>)
                                   : reinterpret_cast<const void*>(&embed_join_kernel<true, false>))
                          : (out16 ? reinterpret_cast<const void*>(&embed_join_kernel<false, true>)
                                   : reinterpret_cast<const void*>(&embed_join_kernel<false, false>));
  void* args[] = {&r};
  ok = launch_pdl(sum, dim3(static_cast<unsigned>((units + kRunWarps - 1) / kRunWarps)), dim3(kRunWarps * 32), 0, stream, args);
  if (ok != DLLM_OK || r.chunks < 2) return ok;
  return launch_pdl(join, dim3(static_cast<unsigned>(units)), dim3(kRunWarps * 32), 0, stream, args);
}

}  // extern "C"
