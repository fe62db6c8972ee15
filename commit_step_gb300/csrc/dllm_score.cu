// dllm_score.cu -- log probabilities of given tokens with the entropy and the
// top alternatives, and the gradient of all three with respect to the logits.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <vector>

#include "dllm_device.cuh"
#include "dllm_launch.cuh"

namespace dllm {

constexpr int kScoreThreads = 256;
constexpr int kScoreWarps = kScoreThreads / 32;
constexpr int kScoreVec = 4;      // 16-byte vectors a thread has in flight
constexpr int kTopCap = 128;      // candidates a warp keeps before it cuts them to the best k
constexpr float kInfF = __builtin_huge_valf();
constexpr float kLow = -0x1p+100f;  // stands for a difference or exponent that carries no mass: 2^kLow = 0, 0 * kLow = 0
constexpr int kEntries = 2048;    // block maxima a CTA keeps

struct ScoreParams {
  const uint8_t* logits;
  int64_t T, V, row_bytes;
  const int32_t* targets;
  float* logprob;
  float* entropy;
  float* lse;
  int32_t* top_ids;
  float* top_logprob;
  int32_t top;
  float ln_veff;              // ln of the number of ids that are not suppressed
  int32_t n_sup;
  int32_t sup[DLLM_MAX_SUPPRESS];  // ascending, distinct
};

// A candidate: value order in the high word, lower ids first in the low word.
// 0 is no candidate (every value's key is above 0).
__device__ __forceinline__ uint64_t candidate(float z, uint32_t id) {
  return static_cast<uint64_t>(float_key(z)) << 32 | (0xFFFFFFFFu - id);
}
__device__ __forceinline__ float candidate_value(uint64_t c) { return key_to_float(static_cast<uint32_t>(c >> 32)); }
__device__ __forceinline__ uint32_t candidate_id(uint64_t c) { return 0xFFFFFFFFu - static_cast<uint32_t>(c); }

__device__ __forceinline__ float no_nan(float z) { return fmaxf(z, -kInfF); }  // NaN -> -inf

// The state of a softmax over some ids: the largest logit m, Z = sum
// 2^((z - m) log2 e), S = sum 2^y y of the same exponents.
struct Soft {
  float m, Z, S;
};

// log2 e (from - to) for from <= to, finite (kLow where the mass vanishes).
__device__ __forceinline__ float shift2(float from, float to) { return fmaxf(from - to, kLow) * kLog2e; }

__device__ __forceinline__ void soft_raise(Soft& a, float m) {
  const float d = shift2(a.m, m), f = ex2_approx(d);
  a.S = f * fmaf(d, a.Z, a.S);
  a.Z *= f;
  a.m = m;
}

__device__ __forceinline__ void soft_join(Soft& a, Soft b) {
  const float m = fmaxf(a.m, b.m);
  soft_raise(a, m);
  soft_raise(b, m);
  a.Z += b.Z;
  a.S += b.S;
}

// Ranks the n candidates in `in` (distinct, in shared memory) against each
// other and stores those with rank < k at out[rank]; `step` threads share the
// work.  in and out do not overlap.
__device__ __forceinline__ void rank_candidates(const uint64_t* in, int n, int k, uint64_t* out, int first, int step) {
  for (int i = first; i < n; i += step) {
    const uint64_t c = in[i];
    int r = 0;
    for (int j = 0; j < n; ++j) r += in[j] > c ? 1 : 0;
    if (r < k) out[r] = c;
  }
}

template <int BYTES>  // of an element
__device__ __forceinline__ float element(const uint4& v, int e) {
  const uint32_t w = (&v.x)[BYTES == 2 ? e >> 1 : e];
  if (BYTES == 4) return __uint_as_float(w);
  return (e & 1) ? bf16hi(w) : bf16lo(w);
}

// One cluster of CTAs per row, each CTA an equal range of the row's 16-byte
// vectors (few rows: up to 8 CTAs a row, so that the whole GPU reads; many
// rows: one CTA a row, several rows to an SM).
//
// One pass over the logits: a warp holds a running maximum and its lanes sums Z
// and S of 2^y and 2^y y, y = (z - m) log2 e, rescaled only when the maximum
// grows.  For the alternatives the pass keeps only the maximum of each block of
// 32 vectors.  The best k elements lie in the best k blocks (by maximum, then
// position: k better blocks would hold k better elements), so afterwards the
// blocks that can be among those are read again, a percent or so of the row,
// and their elements compared one by one.  (Comparing every element with the
// k-th best so far during the pass was six times slower: almost every 1024
// elements of a warp hold one that reaches it.)
// Logits below -2^100 count as -2^100 in the pass; a row whose maximum is not
// within 2^100 of zero is computed from its logits as they are by one CTA.
// Bound: the one read of the logits.  Measured, 4096 x 152064 bf16: 191 us (6.5
// TB/s) without alternatives, 233 us with the top 20; 2048 x 152064 fp32: 186 us
// (6.7 TB/s) and 207 us; 32 x 126464 bf16, top 8: 11 us.
template <int BYTES>
__global__ void __launch_bounds__(kScoreThreads, 4) score_kernel(const __grid_constant__ ScoreParams p) {
  constexpr int EPV = 16 / BYTES;
  __shared__ uint64_t list[kScoreWarps][kTopCap];
  __shared__ uint64_t scratch[kScoreWarps][DLLM_MAX_TOP];
  __shared__ uint64_t best[DLLM_MAX_TOP];                  // this CTA's best k, descending
  __shared__ uint32_t entry[kEntries];                     // float_key of the blocks' maxima (0: none)
  __shared__ uint16_t chosen[kEntries];
  __shared__ uint64_t floor_entry_s;
  __shared__ int32_t n_chosen;
  __shared__ unsigned long long floor_s;                   // no value below this candidate can be among the best k
  __shared__ Soft warp_soft[kScoreWarps];
  __shared__ Soft cta_soft;
  __shared__ int32_t count_s[kScoreWarps];
  __shared__ alignas(16) uint64_t joined[8 * DLLM_MAX_TOP];
  __shared__ uint32_t inf_s;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint32_t rank, size;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
  asm("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(size));
  const int64_t row = blockIdx.x / size;
  const int k = p.top;
  if (threadIdx.x == 0) {
    floor_s = 0;
    floor_entry_s = 0;
    n_chosen = 0;
    inf_s = 0;
  }
  pdl_launch_dependents();
  pdl_wait();

  const uint8_t* base = p.logits + row * p.row_bytes;
  // The row as whole aligned vectors, with up to EPV - 1 elements before and after them.
  const int64_t lead = std::min<int64_t>(p.V, ((16 - (reinterpret_cast<uintptr_t>(base) & 15u)) & 15u) / BYTES);
  const int64_t nvec = (p.V - lead) / EPV;
  const int64_t tail0 = lead + nvec * EPV;
  const uint4* vecs = reinterpret_cast<const uint4*>(base + lead * BYTES);
  const int64_t v0 = nvec * rank / size, v1 = nvec * (rank + 1) / size;
  const int nv = static_cast<int>(v1 - v0);                // this CTA's vectors (V < 2^31)
  const int blocks = (nv + 31) / 32;
  int shift = 0;                                           // 2^shift blocks share an entry
  while (((blocks + (1 << shift) - 1) >> shift) > kEntries) ++shift;
  if (k > 0 && shift > 0)                                  // (else every entry is written once)
    for (int i = threadIdx.x; i < kEntries; i += kScoreThreads) entry[i] = 0;
  __syncthreads();
  Soft a{kLow, 0.0f, 0.0f};

  // The next suppressed id, as an element offset from this CTA's first.
  const int64_t id_base = lead + v0 * EPV;
  int sup_at = 0;
  int64_t next_sup = INT64_MAX;
  auto skip_sup = [&](int64_t upto) {                      // to the first one at or past `upto`
    while (sup_at < p.n_sup && p.sup[sup_at] - id_base < upto) ++sup_at;
    next_sup = sup_at < p.n_sup ? p.sup[sup_at] - id_base : INT64_MAX;
  };
  skip_sup(0);
  const uint4* src = vecs + v0 + lane;
  for (int b0 = warp * (kScoreVec * 32); b0 < nv; b0 += kScoreThreads * kScoreVec) {
    uint4 x[kScoreVec];
    if (b0 + kScoreVec * 32 <= nv) {
#pragma unroll
      for (int u = 0; u < kScoreVec; ++u) x[u] = __ldcs(src + b0 + u * 32);
    } else {
#pragma unroll
      for (int u = 0; u < kScoreVec; ++u) {
        const uint32_t none = BYTES == 2 ? 0xFF80FF80u : 0xFF800000u;   // -inf
        x[u] = make_uint4(none, none, none, none);
        if (b0 + u * 32 + lane < nv) x[u] = __ldcs(src + b0 + u * 32);
      }
    }
    const int64_t end = static_cast<int64_t>(b0 + kScoreVec * 32) * EPV;
    if (next_sup < end) {                                  // rare: a suppressed id among this warp's values
      skip_sup(static_cast<int64_t>(b0) * EPV);
      for (int i = sup_at; i < p.n_sup && p.sup[i] - id_base < end; ++i) {
        const int off = static_cast<int>(p.sup[i] - id_base - static_cast<int64_t>(b0) * EPV);
        const int at = off / EPV % 32 == lane ? off / (32 * EPV) * EPV + off % EPV : -1;
#pragma unroll
        for (int u = 0; u < kScoreVec; ++u)
#pragma unroll
          for (int e = 0; e < EPV; ++e)
            if (u * EPV + e == at) {
              uint32_t& w = (&x[u].x)[BYTES == 2 ? e >> 1 : e];
              w = BYTES == 4 ? 0xFF800000u : ((e & 1) ? (w & 0xFFFFu) | 0xFF800000u : (w & 0xFFFF0000u) | 0xFF80u);
            }
      }
      skip_sup(end);
    }
    // NaN and everything below -2^100 as -2^100; the blocks' maxima.
    float top[kScoreVec];
#pragma unroll
    for (int u = 0; u < kScoreVec; ++u) {
      uint32_t* w = &x[u].x;
#pragma unroll
      for (int q = 0; q < 4; ++q)
        w[q] = BYTES == 2 ? bmax2(w[q], kSentinelBf16x2)
                          : __float_as_uint(fmaxf(__uint_as_float(w[q]), kLow));
      if (BYTES == 2) {
        const uint32_t m2 = bmax2(bmax2(w[0], w[1]), bmax2(w[2], w[3]));
        top[u] = fmaxf(bf16lo(m2), bf16hi(m2));
      } else {
        top[u] = fmaxf(fmaxf(__uint_as_float(w[0]), __uint_as_float(w[1])),
                       fmaxf(__uint_as_float(w[2]), __uint_as_float(w[3])));
      }
    }
    float cm;
    if (k > 0) {
      static_assert(kScoreVec == 4, "");
#pragma unroll
      for (int u = 0; u < kScoreVec; ++u) top[u] = warp_max_f32(top[u]);
      cm = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
      const float mine = lane & 2 ? (lane & 1 ? top[3] : top[2]) : (lane & 1 ? top[1] : top[0]);
      const int block = (b0 >> 5) + lane;
      if (lane < kScoreVec && block < blocks) {
        if (shift == 0) entry[block] = float_key(mine);
        else atomicMax(&entry[block >> shift], float_key(mine));
      }
    } else {
      cm = warp_max_f32(fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])));
    }
    if (cm > a.m) soft_raise(a, cm);                       // warp-uniform
    const uint64_t nm2 = pack2(-a.m, -a.m), l2e2 = pack2(kLog2e, kLog2e);
    uint64_t Z2 = 0, S2 = 0;
#pragma unroll
    for (int u = 0; u < kScoreVec; ++u) {
      const uint32_t* w = &x[u].x;
#pragma unroll
      for (int q = 0; q < EPV / 2; ++q) {
        const uint64_t z = BYTES == 2 ? pack2(bf16lo(w[q]), bf16hi(w[q]))
                                      : pack2(__uint_as_float(w[2 * q]), __uint_as_float(w[2 * q + 1]));
        uint64_t y = add2(z, nm2);
        asm("mul.rn.f32x2 %0, %0, %1;" : "+l"(y) : "l"(l2e2));
        float y0, y1;
        unpack2(y, y0, y1);
        const uint64_t e = pack2(ex2_approx(y0), ex2_approx(y1));
        Z2 = add2(Z2, e);
        S2 = fma2(e, y, S2);
      }
    }
    float z0, z1, s0, s1;
    unpack2(Z2, z0, z1);
    unpack2(S2, s0, s1);
    a.Z += z0 + z1;
    a.S += s0 + s1;
  }

  // The elements outside the whole vectors: the first CTA's first warp holds
  // those before (lanes 0 .. EPV - 1), the last CTA's those after (lanes 16 ..).
  const bool edges = warp == 0 && ((rank == 0 && lead > 0) || (rank == size - 1 && tail0 < p.V));
  const int64_t edge_id = lane < 16 ? lane : tail0 + lane - 16;
  float edge_z = -kInfF;
  bool edge_in = false;
  if (edges) {
    edge_in = lane < 16 ? rank == 0 && edge_id < lead : rank == size - 1 && edge_id < p.V;
    if (edge_in) {
      if (BYTES == 2)
        edge_z = __uint_as_float(static_cast<uint32_t>(reinterpret_cast<const uint16_t*>(base)[edge_id]) << 16);
      else
        edge_z = reinterpret_cast<const float*>(base)[edge_id];
      edge_z = no_nan(edge_z);
      for (int q = 0; q < p.n_sup; ++q)
        if (p.sup[q] == edge_id) edge_in = false;
    }
    const float z = edge_in ? fmaxf(edge_z, kLow) : kLow;
    const float cm = warp_max_f32(z);
    if (cm > a.m) soft_raise(a, cm);
    const float y = (z - a.m) * kLog2e, e = edge_in ? ex2_approx(y) : 0.0f;
    a.Z += e;
    if (edge_in) a.S = fmaf(e, y, a.S);
  }

  int have = 0;                                            // candidates in this warp's list
  if (k > 0) {
    float floor_z = -kInfF;
    uint64_t floor_c = 0;                                  // a candidate below it is not among the best k
    auto cut = [&]() {                                     // keep the best k of the warp's list, raise the floor
      __syncwarp();
      rank_candidates(list[warp], have, k, scratch[warp], lane, 32);
      __syncwarp();
      if (have > k) have = k;
      if (lane < have) list[warp][lane] = scratch[warp][lane];
      __syncwarp();
      if (have == k && lane == 0) atomicMax(&floor_s, static_cast<unsigned long long>(scratch[warp][k - 1]));
      __syncwarp();
    };
    auto offer = [&](float z, uint32_t id, bool in) {      // one value per lane
      const bool near = in && z >= floor_z;
      if (__ballot_sync(0xFFFFFFFFu, near) == 0u) return;
      if (have + 32 > kTopCap) {
        cut();
        const uint64_t g = *const_cast<volatile unsigned long long*>(&floor_s);
        if (g > floor_c) {
          floor_c = g;
          floor_z = candidate_value(g);
        }
      }
      const uint64_t q = candidate(z, id);
      const bool keep = near && q >= floor_c;
      const uint32_t hit = __ballot_sync(0xFFFFFFFFu, keep);
      if (keep) list[warp][have + __popc(hit & ((1u << lane) - 1u))] = q;
      have += __popc(hit);
    };
    if (edges) offer(edge_z, static_cast<uint32_t>(edge_id), edge_in);
    // A floor for the entries: the best entry of each four threads; at least k
    // entries are no worse than the k-th of those 64.
    constexpr int kGroups = kScoreThreads / 4;
    static_assert(kGroups >= DLLM_MAX_TOP, "");
    const int n = (blocks + (1 << shift) - 1) >> shift;
    __syncthreads();
    uint64_t* group_s = joined;
    uint64_t mine = 0;
    for (int e = threadIdx.x; e < n; e += kScoreThreads) {
      const uint64_t c = static_cast<uint64_t>(entry[e]) << 32 | (0xFFFFFFFFu - static_cast<uint32_t>(e));
      mine = c > mine ? c : mine;
    }
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
      const uint64_t c = __shfl_xor_sync(0xFFFFFFFFu, mine, o);
      mine = c > mine ? c : mine;
    }
    if ((threadIdx.x & 3) == 0) group_s[threadIdx.x >> 2] = mine;
    __syncthreads();
    if (threadIdx.x < kGroups) {
      mine = group_s[threadIdx.x];
      int r = 0;
#pragma unroll 4
      for (int j = 0; j < kGroups; j += 2) {
        const ulonglong2 o = *reinterpret_cast<const ulonglong2*>(&group_s[j]);
        r += (o.x > mine ? 1 : 0) + (o.y > mine ? 1 : 0);
      }
      // (among values that only stand for "-2^100 or less" the entries say nothing: then all are taken)
      if (mine != 0 && r == k - 1 && candidate_value(mine) > kLow) floor_entry_s = mine;
    }
    __syncthreads();
    const uint64_t fe = floor_entry_s;
    for (int e = threadIdx.x; e < n; e += kScoreThreads)
      if ((static_cast<uint64_t>(entry[e]) << 32 | (0xFFFFFFFFu - static_cast<uint32_t>(e))) >= fe)
        chosen[atomicAdd(&n_chosen, 1)] = static_cast<uint16_t>(e);
    __syncthreads();
    if (fe != 0) {
      floor_z = candidate_value(fe);
      floor_c = fe & 0xFFFFFFFF00000000ull;                // its value with any id
    }
    const int nb = n_chosen << shift;
    auto load = [&](int c, int& v) {                       // this lane's vector of chosen block c (v: its index, or nv)
      v = nv;
      uint4 x = make_uint4(0u, 0u, 0u, 0u);
      if (c < nb) {
        const int blk = (static_cast<int>(chosen[c >> shift]) << shift) + (c & ((1 << shift) - 1));
        v = min(blk * 32 + lane, nv);
        if (v < nv) x = vecs[v0 + v];
      }
      return x;
    };
    int v, vn;
    uint4 x = load(warp, v);
    for (int c = warp; c < nb; c += kScoreWarps) {
      const uint4 next = load(c + kScoreWarps, vn);        // (its latency passes behind this block's comparisons)
      const int64_t id = id_base + static_cast<int64_t>(v) * EPV;
      uint32_t absent = v < nv ? 0u : 0xFFu;
      for (int q = 0; q < p.n_sup; ++q) {
        const int64_t off = p.sup[q] - id;
        if (off >= 0 && off < EPV) absent |= 1u << off;
      }
#pragma unroll
      for (int e = 0; e < EPV; ++e)
        offer(no_nan(element<BYTES>(x, e)), static_cast<uint32_t>(id) + e, !((absent >> e) & 1u));
      x = next;
      v = vn;
    }
    cut();
  }

  // The warp's state, the CTA's, the row's.
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {                       // one maximum per warp: the sums add up
    a.Z += __shfl_xor_sync(0xFFFFFFFFu, a.Z, o);
    a.S += __shfl_xor_sync(0xFFFFFFFFu, a.S, o);
  }
  if (k > 0 && lane == 0) count_s[warp] = have;
  if (lane == 0) warp_soft[warp] = a;
  __syncthreads();
  if (threadIdx.x == 0) {
    Soft t = warp_soft[0];
    for (int w = 1; w < kScoreWarps; ++w) soft_join(t, warp_soft[w]);
    cta_soft = t;
  }
  int total = 0;
  if (k > 0) {
    // the warps' lists side by side, then the best k of them
    int at = 0;
    for (int w = 0; w < kScoreWarps; ++w) {
      if (w < warp) at += count_s[w];
      total += count_s[w];
    }
    if (lane < have) joined[at + lane] = list[warp][lane];
    if (threadIdx.x < k) best[threadIdx.x] = 0;
    __syncthreads();
    rank_candidates(joined, total, k, best, threadIdx.x, kScoreThreads);
  }
  if (size > 1) {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
    if (rank == 0) {
      auto remote = [&](const void* local, uint32_t r) {
        uint32_t addr;
        asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(addr) : "r"(smem_addr(local)), "r"(r));
        return addr;
      };
      if (threadIdx.x == 0) {
        Soft t = cta_soft;
        for (uint32_t r = 1; r < size; ++r) {
          const uint32_t addr = remote(&cta_soft, r);
          Soft o;
          asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(o.m) : "r"(addr) : "memory");
          asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(o.Z) : "r"(addr + 4) : "memory");
          asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(o.S) : "r"(addr + 8) : "memory");
          soft_join(t, o);
        }
        warp_soft[0] = t;
      }
      if (k > 0) {
        const int n = static_cast<int>(size) * k;
        for (int i = threadIdx.x; i < n; i += kScoreThreads) {
          const uint32_t addr = remote(&best[i % k], static_cast<uint32_t>(i / k));
          uint64_t c;
          asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(c) : "r"(addr) : "memory");
          joined[i] = c;
        }
        __syncthreads();
        if (threadIdx.x < k) best[threadIdx.x] = 0;
        __syncthreads();
        rank_candidates(joined, n, k, best, threadIdx.x, kScoreThreads);   // (zeros rank last: at least k are real)
      }
      __syncthreads();
    }
    // the other CTAs' shared memory has been read
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
    if (rank != 0) return;
  } else {
    if (threadIdx.x == 0) warp_soft[0] = cta_soft;
    __syncthreads();
  }

  Soft t = warp_soft[0];
  if (!(t.m > kLow && t.m < -kLow)) {                      // CTA-uniform, rare: from the logits as they are
    auto logit = [&](int64_t v) {
      for (int q = 0; q < p.n_sup; ++q)
        if (p.sup[q] == v) return -kInfF;
      if (BYTES == 4) return no_nan(reinterpret_cast<const float*>(base)[v]);
      return no_nan(__uint_as_float(static_cast<uint32_t>(reinterpret_cast<const uint16_t*>(base)[v]) << 16));
    };
    float m = -kInfF;
    for (int64_t v = threadIdx.x; v < p.V; v += kScoreThreads) m = fmaxf(m, logit(v));
    m = warp_max_f32(m);
    __syncthreads();
    if (lane == 0) warp_soft[warp].m = m;
    __syncthreads();
    for (int w = 0; w < kScoreWarps; ++w) m = fmaxf(m, warp_soft[w].m);
    t = Soft{m, 0.0f, 0.0f};
    uint32_t infs = 0;                                     // +inf logits share the mass equally
    for (int64_t v = threadIdx.x; v < p.V; v += kScoreThreads) {
      const float z = logit(v);
      infs += z == kInfF ? 1u : 0u;
      const float y = fmaxf(z - m, kLow) * kLog2e, e = ex2_approx(y);
      t.Z += e;
      t.S = fmaf(e, y, t.S);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      t.Z += __shfl_xor_sync(0xFFFFFFFFu, t.Z, o);
      t.S += __shfl_xor_sync(0xFFFFFFFFu, t.S, o);
    }
    if (infs) atomicAdd(&inf_s, infs);
    __syncthreads();
    if (lane == 0) warp_soft[warp] = t;
    __syncthreads();
    t.Z = t.S = 0.0f;
    for (int w = 0; w < kScoreWarps; ++w) {
      t.Z += warp_soft[w].Z;
      t.S += warp_soft[w].S;
    }
  }
  const float ln_z = t.m == kInfF ? logf(static_cast<float>(inf_s)) : logf(t.Z);
  // log p of a logit z (NaN as -inf) under the row's softmax.
  auto log_p = [&](float z) {
    if (t.m == kInfF) return z == kInfF ? -ln_z : -kInfF;
    if (t.m == -kInfF) return -p.ln_veff;                  // no mass anywhere: the uniform limit
    return (z - t.m) - ln_z;
  };
  if (threadIdx.x == 0) {
    float ent = t.m == kInfF ? ln_z : (t.m == -kInfF ? p.ln_veff : ln_z - kLn2 * (t.S / t.Z));
    p.entropy[row] = fminf(fmaxf(ent, 0.0f), p.ln_veff);
    p.lse[row] = fabsf(t.m) == kInfF ? t.m : t.m + ln_z;
    const int32_t id = p.targets[row];
    float lp = 0.0f;                                       // no target
    if (id >= 0 && id < p.V) {
      float z;
      if (BYTES == 2)
        z = __uint_as_float(static_cast<uint32_t>(reinterpret_cast<const uint16_t*>(base)[id]) << 16);
      else
        z = reinterpret_cast<const float*>(base)[id];
      lp = log_p(no_nan(z));
      for (int q = 0; q < p.n_sup; ++q)
        if (p.sup[q] == id) lp = -kInfF;
    }
    p.logprob[row] = lp;
  }
  if (threadIdx.x < k) {
    const uint64_t c = best[threadIdx.x];
    p.top_ids[row * k + threadIdx.x] = static_cast<int32_t>(candidate_id(c));
    p.top_logprob[row * k + threadIdx.x] = log_p(candidate_value(c));
  }
}

// ---------------------------------------------------------------------------
// gradient
// ---------------------------------------------------------------------------
struct ScoreGradParams {
  const uint8_t* logits;
  uint8_t* grad;
  int64_t T, V, row_bytes, grad_row_bytes;
  const int32_t* targets;
  const float* lse;
  const float* entropy;
  const float* g_logprob;     // nullable, as the next
  const float* g_entropy;
  const int32_t* top_ids;     // (T, top), nullable with g_top
  const float* g_top;
  int32_t top;
  int32_t chunks;             // blocks per row
  int32_t n_sup;
  int32_t sup[DLLM_MAX_SUPPRESS];
};

constexpr int kGradThreads = 256;
constexpr int kGradVec = 4;

template <int BYTES>
__device__ __forceinline__ void store_element(uint8_t* row, int64_t v, float f) {
  if (BYTES == 4) {
    reinterpret_cast<float*>(row)[v] = f;
  } else {
    uint16_t h;
    asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(h) : "f"(f));
    reinterpret_cast<uint16_t*>(row)[v] = h;
  }
}

template <int BYTES>
__device__ __forceinline__ float load_element(const uint8_t* row, int64_t v) {
  if (BYTES == 4) return reinterpret_cast<const float*>(row)[v];
  return __uint_as_float(static_cast<uint32_t>(reinterpret_cast<const uint16_t*>(row)[v]) << 16);
}

// With G = g + sum g_top and y = z - lse, p = e^y:
//   dz = -p (G + g_entropy (y + H)) + [v = target] g + sum_j [v = top_j] g_top_j,
// 0 for suppressed ids.  One block per row and chunk of it; every thread
// transforms whole vectors, and the few named ids (target, alternatives,
// suppressed ids), read before anything is written, are stored again after the
// block's vectors, so grad may be the logits' own buffer.
// Bound: one read of the logits and one write of the gradient.  Measured, 4096 x
// 152064 bf16: 354 us (7.0 TB/s).
template <int BYTES>
__global__ void __launch_bounds__(kGradThreads) score_grad_kernel(const __grid_constant__ ScoreGradParams p) {
  constexpr int EPV = 16 / BYTES;
  __shared__ int32_t top_s[DLLM_MAX_TOP];
  __shared__ float gt_s[DLLM_MAX_TOP];
  pdl_wait();
  pdl_launch_dependents();
  const int64_t row = blockIdx.x / p.chunks;
  const int chunk = static_cast<int>(blockIdx.x % p.chunks);
  const uint8_t* in = p.logits + row * p.row_bytes;
  uint8_t* out = p.grad + row * p.grad_row_bytes;
  const float lse = p.lse[row], H = p.entropy[row];
  const float ge = p.g_entropy ? p.g_entropy[row] : 0.0f;
  const int32_t target = p.targets[row];
  if (threadIdx.x < p.top) {
    const int32_t id = p.top_ids[row * p.top + threadIdx.x];
    bool counts = id >= 0 && id < p.V;
    for (int q = 0; q < p.n_sup; ++q) counts = counts && p.sup[q] != id;
    top_s[threadIdx.x] = id;
    gt_s[threadIdx.x] = counts ? p.g_top[row * p.top + threadIdx.x] : 0.0f;
  }
  float g = p.g_logprob ? p.g_logprob[row] : 0.0f;
  if (target < 0 || target >= p.V) g = 0.0f;
  for (int q = 0; q < p.n_sup; ++q)
    if (p.sup[q] == target) g = 0.0f;                      // its log probability is -inf whatever the logits are
  const bool dead = !(fabsf(lse) < kInfF);                 // a row without an ordinary softmax: no gradient
  __syncthreads();
  float G = g;
  for (int j = 0; j < p.top; ++j) G += gt_s[j];
  const float base = dead ? 0.0f : G + ge * H, slope = dead ? 0.0f : ge;
  const float ref = dead ? kInfF : lse;
  auto bulk = [&](float z) {
    const float y = fmaxf(z - ref, kLow);                  // (NaN and -inf: no mass)
    const float x = ex2_approx(y * kLog2e);
    return -x * fmaf(slope, y, base);
  };
  const int64_t lead = std::min<int64_t>(p.V, ((16 - (reinterpret_cast<uintptr_t>(in) & 15u)) & 15u) / BYTES);
  const bool same = ((reinterpret_cast<uintptr_t>(in) ^ reinterpret_cast<uintptr_t>(out)) & 15u) == 0;
  const int64_t nvec = (p.V - lead) / EPV;
  const int64_t c0 = nvec * chunk / p.chunks, c1 = nvec * (chunk + 1) / p.chunks;
  // this block's ids are [e0, e1)
  const int64_t e0 = chunk == 0 ? 0 : lead + c0 * EPV, e1 = chunk == p.chunks - 1 ? p.V : lead + c1 * EPV;

  // The named id of this thread, if it lies here: its gradient, from the logit as it still is.
  int64_t named = -1;
  if (threadIdx.x == 0) named = target;
  else if (threadIdx.x <= p.top) named = top_s[threadIdx.x - 1];
  else if (threadIdx.x >= 128 && threadIdx.x < 128 + p.n_sup) named = p.sup[threadIdx.x - 128];
  float named_grad = 0.0f;
  if (named >= e0 && named < e1) {
    bool sup = false;
    for (int q = 0; q < p.n_sup; ++q) sup = sup || p.sup[q] == named;
    if (!sup && !dead) {
      float hot = named == target ? g : 0.0f;
      for (int j = 0; j < p.top; ++j) hot += top_s[j] == named ? gt_s[j] : 0.0f;
      named_grad = bulk(load_element<BYTES>(in, named)) + hot;
    }
  } else {
    named = -1;
  }
  __syncthreads();

  if (same) {
    const uint4* src = reinterpret_cast<const uint4*>(in + lead * BYTES);
    uint4* dst = reinterpret_cast<uint4*>(out + lead * BYTES);
    for (int64_t v0 = c0; v0 < c1; v0 += kGradThreads * kGradVec) {
      uint4 x[kGradVec];
#pragma unroll
      for (int u = 0; u < kGradVec; ++u) {
        const int64_t v = v0 + u * kGradThreads + threadIdx.x;
        if (v < c1) x[u] = __ldcs(src + v);
      }
#pragma unroll
      for (int u = 0; u < kGradVec; ++u) {
        const int64_t v = v0 + u * kGradThreads + threadIdx.x;
        if (v >= c1) continue;
        uint4 o;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          if (BYTES == 4) {
            (&o.x)[q] = __float_as_uint(bulk(__uint_as_float((&x[u].x)[q])));
          } else {
            const uint32_t w = (&x[u].x)[q];
            uint32_t d;
            asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(bulk(bf16hi(w))), "f"(bulk(bf16lo(w))));
            (&o.x)[q] = d;
          }
        }
        __stcs(dst + v, o);
      }
    }
    const int64_t tail0 = lead + nvec * EPV;
    if (chunk == 0 && threadIdx.x < lead)
      store_element<BYTES>(out, threadIdx.x, bulk(load_element<BYTES>(in, threadIdx.x)));
    if (chunk == p.chunks - 1 && tail0 + threadIdx.x < p.V)
      store_element<BYTES>(out, tail0 + threadIdx.x, bulk(load_element<BYTES>(in, tail0 + threadIdx.x)));
  } else {                                                 // rows whose vectors do not line up: one by one
    for (int64_t v = e0 + threadIdx.x; v < e1; v += kGradThreads)
      store_element<BYTES>(out, v, bulk(load_element<BYTES>(in, v)));
  }
  __syncthreads();
  if (named >= 0) store_element<BYTES>(out, named, named_grad);
}

// Checks shared by both directions; the ascending distinct suppressed ids in `sup`.
static dllm_status check_score(const void* logits, dllm_dtype dt, int64_t T, int64_t V, int64_t row_stride,
                               const int32_t* suppress_ids, int32_t n_suppress, int32_t top,
                               std::vector<int32_t>& sup) {
  if (dt != DLLM_F32 && dt != DLLM_BF16) return DLLM_ERR_INVALID_ARGUMENT;
  if (T < 0 || V < 1 || V > INT32_MAX - 1 || row_stride < V || top < 0) return DLLM_ERR_INVALID_ARGUMENT;
  if (mul_or_neg(T, mul_or_neg(row_stride, 4)) < 0 || mul_or_neg(T, 4 * (static_cast<int64_t>(top) + 1)) < 0)
    return DLLM_ERR_INVALID_ARGUMENT;
  if (n_suppress < 0 || (n_suppress > 0 && !suppress_ids)) return DLLM_ERR_INVALID_ARGUMENT;
  if (n_suppress > DLLM_MAX_SUPPRESS || top > DLLM_MAX_TOP) return DLLM_ERR_UNSUPPORTED;
  sup.assign(suppress_ids, suppress_ids + n_suppress);
  for (int32_t id : sup)
    if (id < 0 || id >= V) return DLLM_ERR_INVALID_ARGUMENT;
  std::sort(sup.begin(), sup.end());
  sup.erase(std::unique(sup.begin(), sup.end()), sup.end());
  if (static_cast<int64_t>(sup.size()) >= V || top > V - static_cast<int64_t>(sup.size()))
    return DLLM_ERR_INVALID_ARGUMENT;
  if (T > 0 && !logits) return DLLM_ERR_INVALID_ARGUMENT;
  if ((reinterpret_cast<uintptr_t>(logits) & (dt == DLLM_BF16 ? 1u : 3u)) != 0) return DLLM_ERR_INVALID_ARGUMENT;
  return DLLM_OK;
}

}  // namespace dllm

extern "C" {

dllm_status dllm_token_logprobs(const void* logits, dllm_dtype dt, int64_t T, int64_t V, int64_t row_stride,
                                const int32_t* targets, const int32_t* suppress_ids, int32_t n_suppress, int32_t top,
                                float* logprob, float* entropy, float* lse, int32_t* top_ids, float* top_logprob,
                                dllm_stream_t stream) {
  using namespace dllm;
  std::vector<int32_t> sup;
  const dllm_status st = check_score(logits, dt, T, V, row_stride, suppress_ids, n_suppress, top, sup);
  if (st != DLLM_OK) return st;
  if (T == 0) return DLLM_OK;
  if (!targets || !logprob || !entropy || !lse || (top > 0 && (!top_ids || !top_logprob)))
    return DLLM_ERR_INVALID_ARGUMENT;
  if (!aligned4(targets) || !aligned4(logprob) || !aligned4(entropy) || !aligned4(lse) || !aligned4(top_ids) ||
      !aligned4(top_logprob))
    return DLLM_ERR_INVALID_ARGUMENT;
  const int64_t bytes = dt == DLLM_BF16 ? 2 : 4;
  // CTAs per row: doubled while the grid would leave SMs without work (304 =
  // two CTAs for each of 152 SMs) and every CTA still gets two passes of its
  // threads' vectors.  Measured, 126464 bf16, top 8, us with 1 / 2 / 4 / 8 CTAs:
  // 32 rows 18.4 / 13.4 / 11.4 / 11.2, 128 rows 23.3 / 19.0 / 14.7 / 22.3, 256
  // rows 28.4 / 20.3 / 26.9 / 41.4, 512 rows 30.3 / 36.7 / 50.0 / 78.9; in fp32 26.7 /
  // 18.8 / 13.6 / 11.8, 31.4 / 23.3 / 17.9 / 24.6, 36.3 / 27.5 / 33.7 / 46.4, 44.9 /
  // 52.5 / 65.3 / 88.9.
  int cluster = 1;
  while (cluster < 8 && T * cluster < 304 && V * bytes >= 2 * cluster * 2 * 16 * kScoreThreads * kScoreVec) cluster *= 2;
  if (T > INT32_MAX / cluster) return DLLM_ERR_UNSUPPORTED;
  ScoreParams p{};
  p.logits = static_cast<const uint8_t*>(logits);
  p.T = T;
  p.V = V;
  p.row_bytes = row_stride * bytes;
  p.targets = targets;
  p.logprob = logprob;
  p.entropy = entropy;
  p.lse = lse;
  p.top_ids = top_ids;
  p.top_logprob = top_logprob;
  p.top = top;
  p.ln_veff = static_cast<float>(std::log(static_cast<double>(V - static_cast<int64_t>(sup.size()))));
  p.n_sup = static_cast<int32_t>(sup.size());
  for (size_t i = 0; i < sup.size(); ++i) p.sup[i] = sup[i];
  void* args[] = {&p};
  const void* kernel = dt == DLLM_BF16 ? reinterpret_cast<const void*>(&score_kernel<2>)
                                       : reinterpret_cast<const void*>(&score_kernel<4>);
  return launch_pdl(kernel, dim3(static_cast<unsigned>(T * cluster)), dim3(kScoreThreads), 0, stream, args, cluster);
}

dllm_status dllm_token_logprobs_backward(const void* logits, dllm_dtype dt, int64_t T, int64_t V, int64_t row_stride,
                                         const int32_t* targets, const int32_t* suppress_ids, int32_t n_suppress,
                                         const float* lse, const float* entropy, const float* grad_logprob,
                                         const float* grad_entropy, int32_t top, const int32_t* top_ids,
                                         const float* grad_top, void* grad, int64_t grad_row_stride,
                                         dllm_stream_t stream) {
  using namespace dllm;
  std::vector<int32_t> sup;
  const dllm_status st = check_score(logits, dt, T, V, row_stride, suppress_ids, n_suppress, top, sup);
  if (st != DLLM_OK) return st;
  if (grad_row_stride < V || mul_or_neg(T, mul_or_neg(grad_row_stride, 4)) < 0) return DLLM_ERR_INVALID_ARGUMENT;
  if (T == 0) return DLLM_OK;
  if (!targets || !lse || !entropy || !grad || (top > 0 && (!top_ids || !grad_top))) return DLLM_ERR_INVALID_ARGUMENT;
  if (!aligned4(targets) || !aligned4(lse) || !aligned4(entropy) || !aligned4(grad_logprob) ||
      !aligned4(grad_entropy) || !aligned4(top_ids) || !aligned4(grad_top))
    return DLLM_ERR_INVALID_ARGUMENT;
  if ((reinterpret_cast<uintptr_t>(grad) & (dt == DLLM_BF16 ? 1u : 3u)) != 0) return DLLM_ERR_INVALID_ARGUMENT;
  const int64_t bytes = dt == DLLM_BF16 ? 2 : 4;
  // A block per 32 KB of a row: two passes of its threads' vectors, so the
  // row's scalars are read once for eight vectors a thread.
  const int64_t chunks = std::max<int64_t>(1, (V * bytes + 32767) / 32768);
  if (mul_or_neg(T, chunks) < 0 || T * chunks > INT32_MAX) return DLLM_ERR_UNSUPPORTED;
  ScoreGradParams p{};
  p.logits = static_cast<const uint8_t*>(logits);
  p.grad = static_cast<uint8_t*>(grad);
  p.T = T;
  p.V = V;
  p.row_bytes = row_stride * bytes;
  p.grad_row_bytes = grad_row_stride * bytes;
  p.targets = targets;
  p.lse = lse;
  p.entropy = entropy;
  p.g_logprob = grad_logprob;
  p.g_entropy = grad_entropy;
  p.top_ids = top_ids;
  p.g_top = grad_top;
  p.top = top;
  p.chunks = static_cast<int32_t>(chunks);
  p.n_sup = static_cast<int32_t>(sup.size());
  for (size_t i = 0; i < sup.size(); ++i) p.sup[i] = sup[i];
  void* args[] = {&p};
  const void* kernel = dt == DLLM_BF16 ? reinterpret_cast<const void*>(&score_grad_kernel<2>)
                                       : reinterpret_cast<const void*>(&score_grad_kernel<4>);
  return launch_pdl(kernel, dim3(static_cast<unsigned>(T * chunks)), dim3(kGradThreads), 0, stream, args);
}

}  // extern "C"
