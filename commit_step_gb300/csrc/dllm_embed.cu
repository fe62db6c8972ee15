// dllm_embed.cu -- the embedding of a canvas, and its gradient by sorted tokens
// (sm_103a).
//
// Forward: out_i = scale weight[token_i], rows copied in 16-byte vectors.
//
// Backward: grad_weight[v] = scale sum over the positions i of token v of
// grad_i, summed in fp32 in an order that depends on the tokens alone.  The
// positions are sorted by token, the sorted list is cut into chunks of equal
// length, and a warp sums the runs of equal tokens in its chunk for a slab of
// columns: however uneven the tokens (half of a noised canvas is the mask token),
// every warp reads the same number of rows.  The parts of a run that crosses
// blocks of 8 chunks go to a workspace and are added in order by a last kernel.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <mutex>

#include "../../include/dllmcommit.h"
#include "dllm_device.cuh"
#include "dllm_launch.cuh"

namespace dllm {

// x / d for x < 2^31 as a multiplication: with 2^(s-1) < d <= 2^s and m = floor(2^32
// (2^s - d) / d) + 1, x / d = (floor(m x / 2^32) + x) >> s (Granlund and Montgomery,
// "Division by invariant integers using multiplication", 1994; the sum stays below
// 2^32 for such x).
struct EmDiv {
  uint32_t d, m, s;
  __device__ __forceinline__ uint32_t operator()(uint32_t x) const { return (__umulhi(x, m) + x) >> s; }
};

inline EmDiv em_div(uint32_t d) {
  EmDiv r{d, 0, 0};
  while ((uint64_t{1} << r.s) < d) ++r.s;
  r.m = static_cast<uint32_t>((((uint64_t{1} << r.s) - d) << 32) / d + 1);
  return r;
}

struct EmbedTokens {
  const int32_t* at;
  EmDiv L;
  int64_t stride, T, V;
  // Token i in the order of the rows; V for an id that has no row.
  __device__ __forceinline__ int32_t operator[](int64_t i) const {
    const uint32_t b = L(static_cast<uint32_t>(i));
    const int32_t v = at[b * stride + (static_cast<uint32_t>(i) - b * L.d)];
    return v < 0 || v >= V ? static_cast<int32_t>(V) : v;
  }
};

// ---------------------------------------------------------------------------
// forward
// ---------------------------------------------------------------------------
constexpr int kEmThreads = 256;
constexpr int kEmVecs = 4;                              // 16-byte vectors of a thread in flight

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

// A block copies `rows` consecutive rows of the output, 16 KB where there are blocks
// enough.  One block a piece, not a grid that fits the GPU: SMs whose memory is further
// away then take fewer pieces (65536 x 2560 bf16: 107 and 97 us, 6.3 TB/s).
template <bool BF16>
__global__ void __launch_bounds__(kEmThreads) embed_kernel(const __grid_constant__ EmbedTokens tok, const uint8_t* weight,
                                                           int64_t row_bytes, EmDiv vecs, int32_t rows, float scale, uint8_t* out) {
  pdl_wait();
  pdl_launch_dependents();
  const int64_t i0 = blockIdx.x * static_cast<int64_t>(rows);
  const int n = static_cast<int>(min(static_cast<int64_t>(rows), tok.T - i0)) * vecs.d;
  uint4* to = reinterpret_cast<uint4*>(out) + i0 * vecs.d;
  for (int j0 = threadIdx.x; j0 < n; j0 += kEmVecs * kEmThreads) {
    uint4 x[kEmVecs];
#pragma unroll
    for (int e = 0; e < kEmVecs; ++e) {
      const int j = j0 + e * kEmThreads;
      x[e] = make_uint4(0u, 0u, 0u, 0u);
      if (j < n) {
        const uint32_t r = vecs(j);
        const int32_t v = tok[i0 + r];
        if (v < tok.V) x[e] = __ldg(reinterpret_cast<const uint4*>(weight + v * row_bytes) + (j - r * vecs.d));
      }
    }
#pragma unroll
    for (int e = 0; e < kEmVecs; ++e) {
      const int j = j0 + e * kEmThreads;
      if (j < n) to[j] = scale == 1.0f ? x[e] : em_scale<BF16>(x[e], scale);
    }
  }
}

// ---------------------------------------------------------------------------
// the sort
// ---------------------------------------------------------------------------
// A stable radix sort of (token, position) by one cluster of 8 CTAs: each CTA
// holds an equal range of the list and each of its warps an equal part of that,
// so that a key's place is the count of smaller digits, of its digit in earlier
// CTAs and warps, and of its digit before it in the warp.  Two passes
// over the digits' counts a pass: one to count, one to place; the counts of the
// CTAs meet through distributed shared memory.
constexpr int kSortBits = 10;                           // of a digit, at most
constexpr int kSortBins = 1 << kSortBits;
constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kSortCtas = 8;
constexpr int kSortAhead = 8;                           // rounds of 32 keys whose loads are in flight together
constexpr int kSortFew = 128;                           // keys that are ranked by comparing all with all
constexpr int kSortSmem = (kSortWarps + 1) * kSortBins * 4;

struct SortParams {
  EmbedTokens tok;
  int32_t* key[2];
  int32_t* pos[2];
  int32_t passes, bits;           // digits, bits of each
};

__device__ __forceinline__ uint32_t em_peer(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ int32_t em_peer_load(uint32_t addr) {
  int32_t v;
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void em_cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// The exclusive sum of v over the block's threads in order.
__device__ __forceinline__ int32_t em_block_scan(int32_t v, int32_t* sums) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int32_t s = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int32_t x = __shfl_up_sync(0xFFFFFFFFu, s, o);
    if (lane >= o) s += x;
  }
  if (lane == 31) sums[warp] = s;
  __syncthreads();
  int32_t before = s - v;
  for (int w = 0; w < warp; ++w) before += sums[w];
  return before;
}

// A warp's keys first .. end - 1 in rounds of 32: with PLACE `count` holds the
// places that the warp's next keys of a digit take, else it counts them.
template <bool PLACE>
__device__ __forceinline__ void sort_warp(const SortParams& p, int pass, int64_t first, int64_t end, int32_t* count) {
  const int lane = threadIdx.x & 31;
  const int32_t* keys = pass == 0 ? nullptr : p.key[(pass + 1) & 1];
  const int32_t* at = pass == 0 ? nullptr : p.pos[(pass + 1) & 1];
  const int32_t mask = (1 << p.bits) - 1;
  const int shift = pass * p.bits;
  for (int64_t i0 = first; i0 < end; i0 += 32 * kSortAhead) {
    int32_t key[kSortAhead], pos[kSortAhead];
#pragma unroll
    for (int q = 0; q < kSortAhead; ++q) {
      const int64_t i = i0 + 32 * q + lane;
      key[q] = i >= end ? -1 : (pass == 0 ? p.tok[i] : __ldcg(keys + i));   // (another CTA may have written it)
      if (PLACE) pos[q] = i >= end ? 0 : (pass == 0 ? static_cast<int32_t>(i) : __ldcg(at + i));
    }
#pragma unroll
    for (int q = 0; q < kSortAhead; ++q) {
      if (i0 + 32 * q >= end) break;                     // warp-uniform
      const bool in = key[q] >= 0;
      const int digit = (key[q] >> shift) & mask;
      if (PLACE) {
        // The lanes with this lane's digit, bit by bit.
        uint32_t same = __ballot_sync(0xFFFFFFFFu, in);
        for (int b = 0; b < p.bits; ++b) {
          const bool set = (digit >> b) & 1;
          const uint32_t with = __ballot_sync(0xFFFFFFFFu, set);
          same &= set ? with : ~with;
        }
        const int before = __popc(same & ((1u << lane) - 1u));
        const int32_t base = in ? count[digit] : 0;
        __syncwarp();
        if (in) {
          p.key[pass & 1][base + before] = key[q];
          p.pos[pass & 1][base + before] = pos[q];
          if (before == 0) count[digit] = base + __popc(same);
        }
        __syncwarp();
      } else if (in) {
        atomicAdd(count + digit, 1);
      }
    }
  }
}

__global__ void __launch_bounds__(kSortThreads, 1) embed_sort_kernel(const __grid_constant__ SortParams p) {
  extern __shared__ __align__(16) int32_t em_smem[];
  __shared__ int32_t sums[kSortWarps];
  int32_t* total = em_smem;                              // per bin, of this CTA
  int32_t* count = em_smem + kSortBins;                  // (warps, bins)
  pdl_wait();
  // The kernel after this one may begin: what it touches before its own wait, no
  // kernel before this one still uses.
  pdl_launch_dependents();
  const int warp = threadIdx.x >> 5;
  if (p.tok.T <= kSortFew) {
    // A thread's place is the count of the keys before its own (a call with 40 keys: 18.5
    // and 12.3 us, with 333: 22.5 and 24.6).
    if (blockIdx.x != 0) return;
    const int n = static_cast<int>(p.tok.T), i = threadIdx.x;
    const int32_t key = i < n ? p.tok[i] : INT32_MAX;
    em_smem[i] = key;
    __syncthreads();
    int place = 0;
    for (int j = 0; j < n; j += 4) {
      const int4 k = *reinterpret_cast<const int4*>(em_smem + j);        // (INT32_MAX behind the last)
      place += (k.x < key || (k.x == key && j < i) ? 1 : 0) + (k.y < key || (k.y == key && j + 1 < i) ? 1 : 0) +
               (k.z < key || (k.z == key && j + 2 < i) ? 1 : 0) + (k.w < key || (k.w == key && j + 3 < i) ? 1 : 0);
    }
    if (i < n) {
      const int last = (p.passes - 1) & 1;
      p.key[last][place] = key;
      p.pos[last][place] = i;
    }
    return;
  }
  const int bins = 1 << p.bits;
  const uint32_t rank = blockIdx.x;
  const int64_t per = (p.tok.T + kSortCtas * kSortWarps - 1) / (kSortCtas * kSortWarps);
  const int64_t first = min(p.tok.T, (rank * static_cast<int64_t>(kSortWarps) + warp) * per), end = min(p.tok.T, first + per);
  for (int pass = 0; pass < p.passes; ++pass) {
    for (int i = threadIdx.x; i < kSortWarps * bins; i += kSortThreads) count[i] = 0;
    __syncthreads();
    sort_warp<false>(p, pass, first, end, count + warp * bins);
    __syncthreads();
    for (int b = threadIdx.x; b < bins; b += kSortThreads) {
      int32_t s = 0;
      for (int w = 0; w < kSortWarps; ++w) {
        const int32_t c = count[w * bins + b];
        count[w * bins + b] = s;
        s += c;
      }
      total[b] = s;
    }
    em_cluster_sync();
    // A bin a thread: its counts in all CTAs, and in the earlier ones.
    static_assert(kSortBins <= kSortThreads);
    const int b = threadIdx.x;
    int32_t all = 0, mine = 0;
    if (b < bins) {
      int32_t v[kSortCtas];
#pragma unroll
      for (uint32_t c = 0; c < kSortCtas; ++c) v[c] = em_peer_load(em_peer(smem_addr(total + b), c));
#pragma unroll
      for (uint32_t c = 0; c < kSortCtas; ++c) {
        all += v[c];
        if (c < rank) mine += v[c];
      }
    }
    const int32_t base = em_block_scan(all, sums) + mine;
    if (b < bins)
      for (int w = 0; w < kSortWarps; ++w) count[w * bins + b] += base;
    __syncthreads();
    sort_warp<true>(p, pass, first, end, count + warp * bins);
    em_cluster_sync();                                   // places written, totals read
  }
}

// Rows of the gradient that no token names become zero.  The grid has a block for
// each group of rows, but a block that runs marks the named ids in shared memory
// (of a window of 2^20 ids) and then takes over the groups of blocks that have not
// begun (clusterlaunchcontrol): an SM marks once, and those whose memory is further
// away take fewer groups (1.09 GB: 143 us, 167 to 172 in equal shares).  It is
// launched behind the sort and runs beside it: it waits for the sort at its end
// only, so that whoever waits for this kernel waits for both.
constexpr int kZeroThreads = 512;
constexpr int kZeroBits = 1 << 20;

struct ZeroParams {
  EmbedTokens tok;
  uint8_t* out;
  int64_t row_bytes;
  EmDiv vecs;                   // 16-byte vectors of a row
  int32_t rows;                 // rows of a group: a power of two
  int32_t *fault, *seen;        // the workspace's word and the device's
};

__global__ void __launch_bounds__(kZeroThreads, 3) embed_zero_kernel(const __grid_constant__ ZeroParams p) {
  extern __shared__ uint32_t em_named[];
  __shared__ __align__(16) uint4 answer;
  __shared__ __align__(8) uint64_t answer_bar;
  pdl_launch_dependents();
  const uint32_t bar = smem_addr(&answer_bar), at = smem_addr(&answer);
  if (threadIdx.x == 0) {
    mbar_init(bar, 1);
    fence_mbar_init();
  }
  const int64_t V = p.tok.V;
  int64_t v0 = -1;                                       // the window
  uint32_t group = blockIdx.x;
  for (uint32_t phase = 0;; phase ^= 1) {
    const int64_t r0 = static_cast<int64_t>(group) * p.rows;
    __syncthreads();
    if (threadIdx.x == 0) {                              // the next group, while this one is written
      mbar_arrive_expect_tx(bar, 16);
      asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(at),
                   "r"(bar)
                   : "memory");
    }
    if (r0 / kZeroBits * kZeroBits != v0) {
      v0 = r0 / kZeroBits * kZeroBits;
      const int64_t v1 = min(V, v0 + kZeroBits);
      for (int i = threadIdx.x; i < (v1 - v0 + 31) / 32; i += kZeroThreads) em_named[i] = 0u;
      __syncthreads();
      // Token i lies at row i / L, column i mod L; a step of the threads' number adds to both.
      const uint32_t L = p.tok.L.d, down = p.tok.L(kZeroThreads), along = kZeroThreads - down * L;
      const uint32_t b0 = p.tok.L(threadIdx.x);
      uint32_t l = threadIdx.x - b0 * L;
      const int32_t* at = p.tok.at + b0 * p.tok.stride + l;
      const int64_t step = down * p.tok.stride + along, wrap = p.tok.stride - L;
      const uint32_t span = static_cast<uint32_t>(v1 - v0), first = static_cast<uint32_t>(v0);
      for (int64_t i0 = threadIdx.x; i0 < p.tok.T; i0 += 8 * kZeroThreads) {
        uint32_t v[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          v[q] = i0 + q * kZeroThreads < p.tok.T ? static_cast<uint32_t>(*at) - first : 0xFFFFFFFFu;
          at += step;
          l += along;
          if (l >= L) {
            l -= L;
            at += wrap;
          }
        }
#pragma unroll
        for (int q = 0; q < 8; ++q)
          if (v[q] < span) {
            // (a frequent token is marked once: atomics on one word take their turns)
            volatile uint32_t* word = &em_named[v[q] >> 5];
            const uint32_t bit = 1u << (v[q] & 31);
            if (!(*word & bit)) atomicOr(&em_named[v[q] >> 5], bit);
          }
      }
      __syncthreads();
    }
    const int n = static_cast<int>(min(static_cast<int64_t>(p.rows), V - r0)) * p.vecs.d;
    for (int j = threadIdx.x; j < n; j += kZeroThreads) {
      const uint32_t r = p.vecs(j);
      const uint32_t bit = static_cast<uint32_t>(r0 - v0) + r;
      if (!((em_named[bit >> 5] >> (bit & 31)) & 1u))
        reinterpret_cast<uint4*>(p.out + (r0 + r) * p.row_bytes)[j - r * p.vecs.d] = make_uint4(0u, 0u, 0u, 0u);
    }
    if (!mbar_wait_bounded(bar, phase)) {
      if (threadIdx.x == 0) {
        atomicExch(p.fault, kFaultFullWait);
        atomicExch(p.seen, kFaultFullWait);
      }
      break;
    }
    uint32_t more;
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b128 a;\n\tld.shared.b128 a, [%2];\n\tmov.u32 %1, 0;\n\t"
        "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, a;\n\t"
        "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, a;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(more), "=r"(group)
        : "r"(at)
        : "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");   // (read before the next answer lands)
    if (!more) break;
  }
  pdl_wait();
}

// ---------------------------------------------------------------------------
// the sums
// ---------------------------------------------------------------------------
constexpr int kRunWarps = 8;
constexpr int kRunMost = 64;                            // sorted positions of a warp, at most

struct RunParams {
  const int32_t *key, *pos;     // sorted
  int64_t T, V;
  const uint8_t* grad;
  int64_t vecs;                 // 16-byte vectors of a grad row
  float scale;
  void* out;
  int64_t out_stride;
  int32_t accumulate;
  int32_t chunk;                // sorted positions of a warp: a multiple of 8
  int64_t blocks;               // of 8 chunks
  float* part;                  // (blocks, 2, columns): a block's first and last run, where they cross its ends
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

// Bound by memory: 65536 rows of 4096 bf16 with half of them one token's, 126464 ids,
// in 125 us (0.54 GB read, some 0.2 written: 5.8 TB/s); four blocks an SM (64
// registers) against three: 134.
//
// A block sums the runs of 8 consecutive chunks in a slab of 32 vectors, a chunk
// a warp.  A run inside a chunk goes to its row; a chunk's first and last runs
// meet those of its neighbours in shared memory, where warp 0 walks the chunks in
// order, and only the runs that reach over the block's ends become parts.
template <bool BF16, bool OUT16>
__global__ void __launch_bounds__(kRunWarps * 32, 4) embed_sum_kernel(const __grid_constant__ RunParams p) {
  constexpr int kCols = RunLane<BF16>::kCols;
  constexpr int kAhead = 8;
  __shared__ float4 edge[kRunWarps][2][kCols / 4][32];
  __shared__ int32_t edge_key[kRunWarps][2];             // of the first and the last run; no row: V
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t block = blockIdx.x / p.slabs;
  const int64_t vec = (blockIdx.x - block * p.slabs) * 32 + lane;
  const bool live = vec < p.vecs;
  const int64_t b0 = block * kRunWarps * p.chunk, b1 = min(p.T, b0 + kRunWarps * p.chunk);
  const int64_t a = min(b1, b0 + warp * p.chunk), e = min(b1, a + p.chunk);
  const int32_t none = static_cast<int32_t>(p.V);
  // The chunk's tokens and positions, two a lane.
  int32_t key[2], pos[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const bool in = a + 32 * h + lane < e;
    key[h] = in ? p.key[a + 32 * h + lane] : none;
    pos[h] = in ? p.pos[a + 32 * h + lane] : 0;
  }
  const uint4* grad = reinterpret_cast<const uint4*>(p.grad) + vec;
  RunLane<BF16> sum;
  sum.clear();
  int32_t run = __shfl_sync(0xFFFFFFFFu, key[0], 0);
  bool first = true;
  auto to_edge = [&](int which) {
    if (lane == 0) edge_key[warp][which] = run;
#pragma unroll
    for (int i = 0; i < kCols / 4; ++i)
      edge[warp][which][i][lane] = make_float4(sum.s[4 * i], sum.s[4 * i + 1], sum.s[4 * i + 2], sum.s[4 * i + 3]);
  };
#pragma unroll 1
  for (int i = 0; i < p.chunk; i += kAhead) {
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
        if (first)
          to_edge(0);
        else if (live && run != none)
          run_write<OUT16, kCols>(p, run, vec * kCols, sum.s);
        sum.clear();
        run = k[q];
        first = false;
      }
      sum.add(x[q]);
    }
    if (run == none) break;                              // (sorted last)
  }
  if (first) {
    to_edge(0);
    run = none;
    sum.clear();
  }
  to_edge(1);                                            // (none: the chunk is one run)
  __syncthreads();
  if (warp != 0 || !live) return;
  const int32_t left = b0 > 0 ? p.key[b0 - 1] : -1, right = b1 < p.T ? p.key[b1] : -1;
  RunLane<BF16> s;
  s.clear();
  int32_t at = edge_key[0][0];
  bool opens = left == at;                               // the run began before the block
  int slot = 0;
  auto flush = [&](bool last) {
    if (at == none) return;
    if (opens || (last && right == at)) {
      float* part = p.part + ((block * 2 + slot) * p.vecs + vec) * kCols;
#pragma unroll
      for (int i = 0; i < kCols; i += 4)
        *reinterpret_cast<float4*>(part + i) = make_float4(s.s[i], s.s[i + 1], s.s[i + 2], s.s[i + 3]);
    } else {
      run_write<OUT16, kCols>(p, at, vec * kCols, s.s);
    }
  };
  for (int w = 0; w < kRunWarps; ++w)
    for (int h = 0; h < 2; ++h) {
      const int32_t k = edge_key[w][h];
      if (k == none) continue;
      if (k != at) {
        flush(false);
        s.clear();
        at = k;
        opens = false;
        slot = 1;
      }
#pragma unroll
      for (int i = 0; i < kCols / 4; ++i) {
        const float4 v = edge[w][h][i][lane];
        s.s[4 * i] += v.x, s.s[4 * i + 1] += v.y, s.s[4 * i + 2] += v.z, s.s[4 * i + 3] += v.w;
      }
    }
  flush(true);
}

// Runs that cross blocks: the block a run begins in adds its parts.
template <bool BF16, bool OUT16>
__global__ void __launch_bounds__(kRunWarps * 32) embed_join_kernel(const __grid_constant__ RunParams p) {
  constexpr int kCols = RunLane<BF16>::kCols;
  __shared__ float4 share[kRunWarps][kCols / 4][32];
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t block = blockIdx.x / p.slabs;
  const int64_t vec = (blockIdx.x - block * p.slabs) * 32 + lane;
  const int64_t span = kRunWarps * p.chunk, a = block * span, e = a + span;
  if (e >= p.T) return;
  const int32_t run = p.key[e - 1];
  if (run >= p.V || p.key[e] != run) return;             // the block's last run ends with it
  const bool whole = p.key[a] == run;                    // (it is the block's first run too)
  if (whole && a > 0 && p.key[a - 1] == run) return;     // and began before it
  // The last block the run reaches: keys are sorted, so the first key of a later
  // block is `run` exactly while the run goes on.
  int64_t lo = block + 1, hi = p.blocks - 1;
  while (lo < hi) {
    const int64_t mid = (lo + hi + 1) / 2;
    if (p.key[mid * span] == run) lo = mid; else hi = mid - 1;
  }
  const int64_t parts = lo - block + 1;
  const int64_t p0 = parts * warp / kRunWarps, p1 = parts * (warp + 1) / kRunWarps;
  float s[kCols];
#pragma unroll
  for (int i = 0; i < kCols; ++i) s[i] = 0.0f;
  const bool live = vec < p.vecs;
  if (live) {
#pragma unroll 8
    for (int64_t q = p0; q < p1; ++q) {
      const int64_t slot = (block + q) * 2 + (q == 0 && !whole ? 1 : 0);
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

}  // namespace dllm

namespace {

using namespace dllm;

constexpr int64_t kEmMaxT = int64_t{1} << 30, kEmMaxD = int64_t{1} << 20;

struct EmDevice {
  int sms = 0;
  cudaError_t err = cudaSuccess;
};
EmDevice g_em[64];
std::once_flag g_em_once[64];

// The current device's SMs, 0 when it cannot be used.
int em_sms() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  std::call_once(g_em_once[dev], [dev]() {
    EmDevice& d = g_em[dev];
    d.err = cudaDeviceGetAttribute(&d.sms, cudaDevAttrMultiProcessorCount, dev);
    if (d.err == cudaSuccess)
      d.err = cudaFuncSetAttribute(reinterpret_cast<const void*>(&embed_sort_kernel), cudaFuncAttributeMaxDynamicSharedMemorySize,
                                   kSortSmem);
    if (d.err == cudaSuccess)
      d.err = cudaFuncSetAttribute(reinterpret_cast<const void*>(&embed_zero_kernel), cudaFuncAttributeMaxDynamicSharedMemorySize,
                                   kZeroBits / 8);
    if (d.err != cudaSuccess) (void)cudaGetLastError();  // report through the status, leave no sticky error
  });
  return g_em[dev].err == cudaSuccess ? g_em[dev].sms : 0;
}

struct EmPlan {
  int32_t passes, bits, chunk;
  int64_t blocks;
  size_t key[2], pos[2], part, bytes;
};

// The least chunk that gives 16 warps to each of 152 SMs (a short list is summed
// by many warps, a long one in whole chunks), for slabs of 256 columns.  The
// size of the workspace depends on it, so it goes by sizes alone.
EmPlan em_plan(int64_t T, int64_t V, int64_t d) {
  EmPlan e{};
  int bits = 0;
  while (bits < 31 && (V >> bits) != 0) ++bits;          // keys 0 .. V
  e.passes = (bits + kSortBits - 1) / kSortBits;
  e.bits = (bits + e.passes - 1) / e.passes;
  e.chunk = 8;
  while (e.chunk < kRunMost && T * ((d + 255) / 256) > static_cast<int64_t>(e.chunk) * 152 * 16) e.chunk *= 2;
  e.blocks = (T + kRunWarps * e.chunk - 1) / (kRunWarps * e.chunk);
  size_t at = 256;                                       // the fault word
  auto take = [&at](int64_t bytes) {
    const size_t here = at;
    at += static_cast<size_t>((bytes + 255) / 256 * 256);
    return here;
  };
  for (int i = 0; i < 2; ++i) {
    e.key[i] = take(4 * T);
    e.pos[i] = take(4 * T);
  }
  e.part = take(8 * e.blocks * d);
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
  if (T > kEmMaxT || d > kEmMaxD) return DLLM_ERR_UNSUPPORTED;
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
  const int64_t size = dt == DLLM_BF16 ? 2 : 4;
  if (overlapping({extent(out, T, d, d, size)}, {extent(weight, V, d, weight_stride, size), extent(tokens, B, L, token_stride, 4)}))
    return DLLM_ERR_INVALID_ARGUMENT;
  const int sms = em_sms();
  if (sms == 0) return DLLM_ERR_CUDA;
  EmbedTokens tok{tokens, em_div(static_cast<uint32_t>(L)), token_stride, T, V};
  const uint8_t* w = static_cast<const uint8_t*>(weight);
  int64_t row_bytes = weight_stride * size;
  EmDiv vecs = em_div(static_cast<uint32_t>(d * size / 16));
  uint8_t* o = static_cast<uint8_t*>(out);
  // 16 KB a block where there are blocks enough for the GPU.
  int32_t rows = static_cast<int32_t>(std::max<int64_t>(1, std::min<int64_t>(kEmThreads * kEmVecs / vecs.d, T / (sms * 4))));
  void* args[] = {&tok, &w, &row_bytes, &vecs, &rows, &scale, &o};
  const void* kernel = dt == DLLM_BF16 ? reinterpret_cast<const void*>(&embed_kernel<true>)
                                       : reinterpret_cast<const void*>(&embed_kernel<false>);
  return launch_pdl(kernel, dim3(static_cast<unsigned>((T + rows - 1) / rows)), dim3(kEmThreads), 0, stream, args);
}

size_t dllm_embed_tokens_backward_workspace_size(int64_t T, int64_t V, int64_t d) {
  if (T <= 0 || V <= 0 || d <= 0 || T > kEmMaxT || V > INT32_MAX || d > kEmMaxD) return 0;
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
  if (overlapping({extent(grad_weight, V, d, grad_weight_stride, size),
                   Extent{workspace, static_cast<int64_t>(dllm_embed_tokens_backward_workspace_size(T, V, d))}},
                  {extent(grad, T, d, d, grad_dt == DLLM_BF16 ? 2 : 4), extent(tokens, B, L, token_stride, 4)}))
    return DLLM_ERR_INVALID_ARGUMENT;
  const int sms = em_sms();
  if (sms == 0) return DLLM_ERR_CUDA;
  if (T == 0) {  // no token: the gradient is zero
    if (accumulate) return DLLM_OK;
    return cudaMemset2DAsync(grad_weight, static_cast<size_t>(grad_weight_stride * size), 0, static_cast<size_t>(d * size),
                             static_cast<size_t>(V), reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
               ? DLLM_OK
               : DLLM_ERR_CUDA;
  }
  const EmPlan e = em_plan(T, V, d);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  SortParams k{};
  k.tok = EmbedTokens{tokens, em_div(static_cast<uint32_t>(L)), token_stride, T, V};
  for (int i = 0; i < 2; ++i) {
    k.key[i] = reinterpret_cast<int32_t*>(ws + e.key[i]);
    k.pos[i] = reinterpret_cast<int32_t*>(ws + e.pos[i]);
  }
  k.passes = e.passes;
  k.bits = e.bits;
  RunParams r{};
  r.key = k.key[(e.passes - 1) & 1];
  r.pos = k.pos[(e.passes - 1) & 1];
  r.T = T;
  r.V = V;
  r.grad = static_cast<const uint8_t*>(grad);
  r.vecs = d * (grad_dt == DLLM_BF16 ? 2 : 4) / 16;
  r.scale = scale;
  r.out = grad_weight;
  r.out_stride = grad_weight_stride;
  r.accumulate = accumulate != 0 ? 1 : 0;
  r.chunk = e.chunk;
  r.blocks = e.blocks;
  r.part = reinterpret_cast<float*>(ws + e.part);
  r.slabs = static_cast<int32_t>((r.vecs + 31) / 32);
  if (r.blocks * r.slabs > INT32_MAX) return DLLM_ERR_UNSUPPORTED;
  const dim3 grid(static_cast<unsigned>(r.blocks * r.slabs)), block(kRunWarps * 32);
  const bool in16 = grad_dt == DLLM_BF16, out16 = grad_weight_dt == DLLM_BF16;
  const void* sum = in16 ? (out16 ? reinterpret_cast<const void*>(&embed_sum_kernel<true, true>)
                                  : reinterpret_cast<const void*>(&embed_sum_kernel<true, false>))
                         : (out16 ? reinterpret_cast<const void*>(&embed_sum_kernel<false, true>)
                                  : reinterpret_cast<const void*>(&embed_sum_kernel<false, false>));
  const void* join = in16 ? (out16 ? reinterpret_cast<const void*>(&embed_join_kernel<true, true>)
                                   : reinterpret_cast<const void*>(&embed_join_kernel<true, false>))
                          : (out16 ? reinterpret_cast<const void*>(&embed_join_kernel<false, true>)
                                   : reinterpret_cast<const void*>(&embed_join_kernel<false, false>));
  ZeroParams z{};
  z.tok = k.tok;
  z.out = static_cast<uint8_t*>(grad_weight);
  z.fault = reinterpret_cast<int32_t*>(ws);
  z.seen = fault_word();
  if (!z.seen) return DLLM_ERR_CUDA;
  z.row_bytes = grad_weight_stride * size;
  z.vecs = em_div(static_cast<uint32_t>(d * size / 16));
  z.rows = 1;
  while (z.rows < 4096 && 2 * z.rows * static_cast<int64_t>(z.vecs.d) <= 4096) z.rows *= 2;   // 64 KB a group
  const size_t zero_smem = static_cast<size_t>((std::min<int64_t>(V, kZeroBits) + 31) / 32 * 4);
  const dim3 zero_grid(static_cast<unsigned>((V + z.rows - 1) / z.rows));
  void *kargs[] = {&k}, *args[] = {&r}, *zargs[] = {&z};
  auto zero = [&] {
    return launch_pdl(reinterpret_cast<const void*>(&embed_zero_kernel), zero_grid, dim3(kZeroThreads), zero_smem, stream, zargs);
  };
  // The zero rows run beside the sort, and beside the sums as well where these fit
  // the GPU at once (each kernel lets the next begin before it waits, so that the
  // sums' blocks only have to have begun).
  const bool sums_first = !accumulate && r.blocks * r.slabs <= 2 * sms;
  dllm_status ok = launch_pdl(reinterpret_cast<const void*>(&embed_sort_kernel), dim3(kSortCtas), dim3(kSortThreads), kSortSmem,
                              stream, kargs, kSortCtas);
  if (ok == DLLM_OK && !accumulate && !sums_first) ok = zero();
  if (ok == DLLM_OK) ok = launch_pdl(sum, grid, block, 0, stream, args);
  if (ok == DLLM_OK && r.blocks > 1) ok = launch_pdl(join, grid, block, 0, stream, args);
  if (ok == DLLM_OK && sums_first) ok = zero();
  return ok;
}

}  // extern "C"
