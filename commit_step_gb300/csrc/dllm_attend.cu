// dllm_attend.cu -- attention of a block of queries over the paged 8-bit
// key/value cache, and the attention weight each cached token draws.
//
// Mathematics.  For the rows r of one key head (the queries of its head group)
// and its tokens j: x = scale log2 e s_k(j) q_r . k_j, p = 2^(x - m_r), l_r =
// sum p, out_r = sum p s_v(j) v_j / l_r, with a running reference m_r.
//
// The transposed products.  A tile is 128 tokens of one head.  S^T = K Q^T and
// O^T += V^T P^T put the tokens (then the head dimension) on the tensor core's
// 128 rows and the queries on its N columns, so a block of 32 queries, or a
// single one, costs N = 32 or 16 columns and not a padded tile of 128 rows;
// and a softmax thread holds one token, so masks, page scales and the weights'
// sums are per-thread values.
//   * K stays in 8 bits: kind::f8f6f4 on the codes as TMA brought them.  The
//     queries are split into two e4m3 parts of one power-of-two scale per row,
//     hi = e4m3(q / s), lo = e4m3(q / s - hi): a bf16 value has 8 significant
//     bits, e4m3 holds 4 of either sign, so hi + lo is exact for elements above
//     2^-9 of the row's largest and off by at most 2^-18 of it below.
//   * V is widened to fp16, which holds e4m3 exactly; P is rounded to fp16 (11
//     bits against bf16's 8) with the tokens' value scales folded in relative
//     to a running reference, so nothing is rescaled per page.  Probabilities
//     are kept at 64 p s_v / v_ref: full precision down to 2^-20 of the row's
//     largest, absolute error 2^-31 of it below.
//   * The reference m_r moves only when a score exceeds it by more than 4 (log2
//     units), so the accumulator in TMEM is rarely rescaled; sums are fp32.
#include <cuda.h>  // CUtensorMap and its enums (types only; the encoder comes from the driver at run time)
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <mutex>

#include "dllm_cache.cuh"

namespace dllm {

constexpr int kTile = 128;             // tokens per tile: the MMA's M
constexpr float kInf = __builtin_huge_valf();

struct AttendParams {
  CUtensorMap tm_k, tm_v;      // the pools as (pages heads page_size) rows of head_dim bytes, box page_size rows
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
  int32_t G;                   // query heads per key head
  int32_t rows;                // L G: the rows of a key head
  int32_t row_tiles;           // tiles of at most N rows
  int32_t tile_rows;           // rows per row tile (the last may hold fewer)
  int32_t ctas;
  float* part_o;               // (2 ctas, N, D): a CTA's unfinished first and last segment
  float* part_ml;              // (2 ctas, N, 2)
  int32_t* fault;
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

// ---------------------------------------------------------------------------
// tensor core and TMEM wrappers
// ---------------------------------------------------------------------------
__device__ __forceinline__ void at_tma_load(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
          dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
      : "memory");
}

__device__ __forceinline__ void at_mma_f8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}

__device__ __forceinline__ void at_mma_f16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}

__device__ __forceinline__ void at_commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void at_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void at_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
// Shared-memory writes of this thread become visible to the tensor core.
__device__ __forceinline__ void at_fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// C consecutive fp32 columns of this warp's 32 TMEM lanes, one lane a thread.
template <int C>
__device__ __forceinline__ void at_ld(uint32_t t, uint32_t (&r)[C]) {
  static_assert(C == 8 || C == 16 || C == 32, "");
  if constexpr (C == 8) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n\t"
                 "tcgen05.wait::ld.sync.aligned;"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(t)
                 : "memory");
  } else if constexpr (C == 16) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(t)
        : "memory");
  } else {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,"
        "%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(t)
        : "memory");
  }
}

// The same columns back; complete when the call returns.
__device__ __forceinline__ void at_st8(uint32_t t, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};\n\t"
      "tcgen05.wait::st.sync.aligned;" ::"r"(t),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
      : "memory");
}

// Shared-memory matrix descriptors: start address / 16 (bits 0-13), leading
// and stride byte offsets / 16 (bits 16-29, 32-45), version 1 (bit 46), swizzle
// (bits 61-63: 2 = 128 bytes, 4 = 64 bytes, 6 = 32 bytes).
//   K-major (K tile and queries, rows of head_dim bytes): the stride offset is
//   the distance of 8-row groups, the leading offset is not used.
//   MN-major (V and P, one row of 64 elements per token, P's of N when that is
//   less): a row is one swizzle span; the leading offset is the distance of
//   groups of 64 elements, the stride offset that of 8-token groups.
__device__ __forceinline__ uint64_t at_desc(uint32_t saddr, uint32_t leading, uint32_t stride, uint32_t swizzle) {
  uint64_t d = static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>(leading >> 4) << 16;
  d |= static_cast<uint64_t>(stride >> 4) << 32;
  d |= static_cast<uint64_t>(1) << 46;
  d |= static_cast<uint64_t>(swizzle) << 61;
  return d;
}

// Instruction descriptor: fp32 accumulator (bits 4-5 = 1), operand types 0
// (e4m3 for kind::f8f6f4, fp16 for kind::f16), A and B MN-major where set (bits
// 15, 16), N / 8 in bits 17-22, M / 16 in bits 24-28.
constexpr uint32_t at_idesc(int n, bool mn_major) {
  return (1u << 4) | (mn_major ? 3u << 15 : 0u) | (static_cast<uint32_t>(n >> 3) << 17) |
         (static_cast<uint32_t>(kTile >> 4) << 24);
}

__device__ __forceinline__ uint32_t f16x2(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}
__device__ __forceinline__ uint64_t at_mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ void sts128(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}
__device__ __forceinline__ void sts64(uint32_t a, uint32_t x, uint32_t y) {
  asm volatile("st.shared.v2.u32 [%0], {%1,%2};" ::"r"(a), "r"(x), "r"(y) : "memory");
}

// Whether any of the 128 threads of named barrier `id` has p set.
__device__ __forceinline__ bool group_any(uint32_t id, bool p) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred a, b;\n\tsetp.ne.u32 a, %2, 0;\n\tbarrier.cta.red.or.pred b, %1, 128, a;\n\t"
      "selp.u32 %0, 1, 0, b;\n\t}"
      : "=r"(r)
      : "r"(id), "r"(p ? 1u : 0u)
      : "memory");
  return r != 0;
}

// ---------------------------------------------------------------------------
// the partition of the work
// ---------------------------------------------------------------------------
// The tiles of all (batch row, key head, row tile) items, in that order, are
// dealt to the CTAs in equal contiguous ranges, so ragged batches and few long
// sequences load every SM alike.  A CTA's range cuts at most its first and its
// last item short; those parts are joined afterwards in CTA order.
__device__ __forceinline__ int tiles_of(const AttendParams& p, int64_t b) {
  const int n = attend_len(p, b);
  return n > 0 ? (n + kTile - 1) / kTile : 1;  // (an empty sequence still has its zeros written)
}

__device__ __forceinline__ int64_t cta_begin(int64_t total, int64_t cta, int64_t ctas) { return total * cta / ctas; }

struct Cursor {
  int64_t w, w1;   // position and end of the CTA's range
  int64_t b;       // batch row at w
  int64_t off;     // position within the batch row's tiles
};

struct Segment {
  int64_t b;
  int32_t h, rt;   // key head, row tile
  int32_t t0, t1;  // tiles [t0, t1) of the sequence
  int32_t T;       // tiles of the sequence
  int32_t len;
  bool starts_range;
};

__device__ __forceinline__ bool next_segment(const AttendParams& p, Cursor& c, int64_t w0, Segment& s) {
  if (c.w >= c.w1) return false;
  s.b = c.b;
  s.len = attend_len(p, c.b);
  s.T = s.len > 0 ? (s.len + kTile - 1) / kTile : 1;
  const int64_t hr = c.off / s.T;
  s.h = static_cast<int32_t>(hr / p.row_tiles);
  s.rt = static_cast<int32_t>(hr % p.row_tiles);
  s.t0 = static_cast<int32_t>(c.off % s.T);
  const int64_t left = c.w1 - c.w;
  s.t1 = s.t0 + left < s.T ? static_cast<int32_t>(s.t0 + left) : s.T;
  s.starts_range = c.w == w0;
  c.w += s.t1 - s.t0;
  c.off += s.t1 - s.t0;
  if (c.off == static_cast<int64_t>(p.c.heads) * p.row_tiles * s.T) {
    ++c.b;
    c.off = 0;
  }
  return true;
}

// One warp: the tiles of batch rows before `upto`, in every lane.
__device__ __forceinline__ int64_t tiles_before(const AttendParams& p, int64_t upto) {
  int64_t sum = 0;
  for (int64_t b = threadIdx.x & 31; b < upto; b += 32) sum += tiles_of(p, b);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
  return sum;
}

// ---------------------------------------------------------------------------
// the attention kernel
// ---------------------------------------------------------------------------
constexpr int kSoftWarps = 8;                          // two groups of 4 warps; a group owns half the columns
constexpr int kWideWarps = 4;                          // widen V
constexpr int kTmaWarp = kSoftWarps + kWideWarps;
constexpr int kMmaWarp = kTmaWarp + 1;
constexpr int kAttendThreads = (kMmaWarp + 1) * 32;
constexpr int kMetaSlots = 8;
constexpr float kSlack = 4.0f;                         // log2: how far a score may exceed the reference
constexpr float kUnset = -1e30f;                       // the reference before the first score
constexpr float kPUnit = 64.0f;                        // P is held at 64 p s_v / v_ref: at most 2^(6 + 4 + 4) in fp16

template <int N>
constexpr int k_stages() { return 3; }
template <int N>
constexpr int v_stages() { return N == 128 ? 2 : 3; }
template <int N>
constexpr int p_buffers() { return N == 128 ? 1 : 2; }  // (a second buffer would cost a ring stage)
template <int N>
constexpr int p_bytes() { return kTile * N * 2; }
constexpr int kWideBytes = 32768;                      // a tile of V in fp16: 2 groups of 64 dims x 128 tokens
template <int D, int N>
constexpr int attend_smem() {
  return 1024 + 2 * kWideBytes + p_buffers<N>() * p_bytes<N>() + 2 * N * D +
         (k_stages<N>() + v_stages<N>()) * kTile * D;
}

struct TileMeta {
  float ks[8], vs[8];   // per page of the tile: scale log2 e s_k, and s_v
  uint32_t valid[4];    // visible tokens
};

// What the MMA and softmax roles share about a tile is in its meta slot; a
// slot is reused after kMetaSlots tiles, which no role lags behind the
// producer (K stages + 2 score buffers + 1).
template <int N>
struct AttendShared {
  uint64_t kfull[4], kempty[4], vfull[4], vempty[4];
  uint64_t mfull[kMetaSlots];
  uint64_t sfull[2], sempty[2], pfull[2], wfull[2], pvdone[2];
  uint64_t qfull;
  TileMeta meta[kMetaSlots];
  alignas(16) float f[N];    // query scales
  alignas(16) float nm[N];   // minus the references
  alignas(16) float fac_o[N];
  alignas(16) float fac_l[N];
  float red[2][4][N / 2];
  int32_t row[N];        // output rows, -1 past the tile's rows
  int64_t w0, w1, b0, off0;
  uint32_t tmem;
  int32_t abort;
};

template <int D, int N>
__global__ void __launch_bounds__(kAttendThreads, 1) attend_kernel(const __grid_constant__ AttendParams p) {
  constexpr int HALF = N / 2;                          // columns of a softmax group
  constexpr int C = HALF < 32 ? HALF : 32;             // columns read from TMEM at a time
  constexpr int KST = k_stages<N>(), VST = v_stages<N>(), PB = p_buffers<N>();
  constexpr int kTileBytes = kTile * D;
  constexpr uint32_t kPRow = N >= 64 ? 128 : 2 * N;    // bytes of a token's row of P (of a group of 64 columns)
  constexpr uint32_t kPSwz = N >= 64 ? 2 : (N == 32 ? 4 : 6);
  constexpr uint32_t kCols = 3 * N <= 64 ? 64 : (3 * N <= 128 ? 128 : (3 * N <= 256 ? 256 : 512));
  extern __shared__ __align__(1024) uint8_t at_smem[];
  __shared__ AttendShared<N> sh;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t base = (smem_addr(at_smem) + 1023u) & ~1023u;
  const uint32_t wide_s = base, p_s = wide_s + 2 * kWideBytes, q_s = p_s + PB * p_bytes<N>();
  const uint32_t k_s = q_s + 2 * N * D, v_s = k_s + KST * kTileBytes;
  volatile int32_t* abort_flag = &sh.abort;

  if (threadIdx.x == 0) {
    for (int i = 0; i < KST; ++i) {
      mbar_init(smem_addr(&sh.kfull[i]), 1);
      mbar_init(smem_addr(&sh.kempty[i]), 1);
    }
    for (int i = 0; i < VST; ++i) {
      mbar_init(smem_addr(&sh.vfull[i]), 1);
      mbar_init(smem_addr(&sh.vempty[i]), kWideWarps);
    }
    for (int i = 0; i < kMetaSlots; ++i) mbar_init(smem_addr(&sh.mfull[i]), 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_addr(&sh.sfull[i]), 1);
      mbar_init(smem_addr(&sh.sempty[i]), kSoftWarps);
      mbar_init(smem_addr(&sh.pfull[i]), kSoftWarps);
      mbar_init(smem_addr(&sh.wfull[i]), kWideWarps);
      mbar_init(smem_addr(&sh.pvdone[i]), 1);
    }
    mbar_init(smem_addr(&sh.qfull), kSoftWarps);
    sh.abort = 0;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&sh.tmem)),
                 "r"(kCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  pdl_wait();
  pdl_launch_dependents();
  if (warp == 0) {   // this CTA's range and the batch row it begins in
    const int64_t hr = static_cast<int64_t>(p.c.heads) * p.row_tiles;
    const int64_t total = tiles_before(p, p.B) * hr;
    const int64_t w0 = cta_begin(total, blockIdx.x, p.ctas), w1 = cta_begin(total, blockIdx.x + 1, p.ctas);
    int64_t before = 0, b = 0;
    while (b < p.B) {                                  // 32 batch rows at a time
      const int64_t t = b + lane < p.B ? tiles_of(p, b + lane) * hr : 0;
      int64_t inc = t;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t u = __shfl_up_sync(0xFFFFFFFFu, inc, o);
        if (lane >= o) inc += u;
      }
      const unsigned in = __ballot_sync(0xFFFFFFFFu, b + lane < p.B && before + inc > w0);
      if (in != 0u) {
        const int l = __ffs(in) - 1;
        before += __shfl_sync(0xFFFFFFFFu, inc - t, l);
        b += l;
        break;
      }
      before += __shfl_sync(0xFFFFFFFFu, inc, 31);
      b += 32;
    }
    if (lane == 0) {
      sh.w0 = w0;
      sh.w1 = w1;
      sh.b0 = b;
      sh.off0 = w0 - before;
    }
  }
  if (D == 64)       // the upper 64 rows of V^T: zeros, once
    for (int i = threadIdx.x; i < 2 * 16384 / 16; i += kAttendThreads)
      sts128(wide_s + static_cast<uint32_t>(i / 1024) * kWideBytes + 16384u + static_cast<uint32_t>(i % 1024) * 16u, 0u,
             0u, 0u, 0u);
  at_fence_async();
  at_fence_before();
  __syncthreads();
  at_fence_after();
  const uint32_t tmem = sh.tmem;

  // Every wait is bounded.  A role whose wait ran out records the fault and
  // raises the abort flag; from then on waits return at once and nothing is
  // issued, so every role reaches the end (with undefined outputs).
  auto wait = [&](uint64_t& bar, uint32_t parity, int32_t code) {
    const uint32_t a = smem_addr(&bar);
    if (mbar_try_wait(a, parity)) return;
    const long long t0 = clock64();
    for (;;) {
      if (*abort_flag) return;
      if (mbar_try_wait_sleep(a, parity, kSleepHintNs)) return;
      if (clock64() - t0 > kWaitLimitCycles) {
        atomicExch(p.fault, code);
        *abort_flag = 1;
        return;
      }
    }
  };

  Cursor cur{sh.w0, sh.w1, sh.b0, sh.off0};
  Segment sg;
  uint32_t g = 0;                                      // tiles this CTA has passed
  const int ps = p.c.page_size;
  const int ppt = kTile / ps;                          // pages per tile

  if (warp == kTmaWarp) {
    // Lane i < ppt follows page i of the tiles.  A page's id is fetched two
    // tiles ahead and its scales one tile ahead of the copies that use them.
    Cursor look = cur;
    Segment ahead;
    int lt = 0;
    bool more = next_segment(p, look, sh.w0, ahead);
    if (more) lt = ahead.t0;
    struct Item {
      int64_t at;      // page heads + head, or -1
      float ks, vs;
      uint32_t nib;    // visible tokens among this lane's four
    };
    struct Raw {
      int32_t id;
      uint32_t nib;
      int32_t h;
      bool on;
    };
    auto fetch = [&](Raw& r) {                         // the next tile's page id and mask bits
      r.on = more;
      r.id = -1;
      r.nib = 0;
      r.h = 0;
      if (!more) return;
      const int64_t col = static_cast<int64_t>(lt) * ppt + lane;
      r.h = ahead.h;
      const int left = ahead.len - lt * kTile;         // tokens from this tile on
      if (lane < ppt && lane * ps < left) r.id = p.table[ahead.b * p.width + col];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int j = lane * 4 + i;
        bool v = j < left;
        if (v && p.mask) v = p.mask[ahead.b * p.mask_stride + static_cast<int64_t>(lt) * kTile + j] != 0;
        r.nib |= (v ? 1u : 0u) << i;
      }
      if (++lt == ahead.t1) {
        more = next_segment(p, look, sh.w0, ahead);
        if (more) lt = ahead.t0;
      }
    };
    auto scales = [&](const Raw& r, Item& it) {
      it.at = r.id >= 0 && r.id < p.c.pages ? static_cast<int64_t>(r.id) * p.c.heads + r.h : -1;
      it.ks = it.vs = 0.0f;
      if (it.at >= 0) {
        it.ks = p.c.k_scale[it.at];
        it.vs = p.c.v_scale[it.at];
      }
      it.nib = r.nib;
    };
    Raw r0, r1;
    Item now, then;
    fetch(r0);
    fetch(r1);
    scales(r0, now);
    bool have = r0.on;
    while (have) {
      const bool next_have = r1.on;
      scales(r1, then);
      fetch(r1);
      const uint32_t ks = g % KST, vs = g % VST, ms = g % kMetaSlots;
      wait(sh.kempty[ks], ((g / KST) & 1u) ^ 1u, kFaultEmptyWait);
      wait(sh.vempty[vs], ((g / VST) & 1u) ^ 1u, kFaultEmptyWait);
      const bool ok = now.at >= 0;
      const unsigned pages = __ballot_sync(0xFFFFFFFFu, ok);
      TileMeta& m = sh.meta[ms];
      if (lane < 8) {
        m.ks[lane] = now.ks * p.scale2;
        m.vs[lane] = now.vs;
      }
      uint32_t bits = (pages >> (lane * 4 / ps)) & 1u ? now.nib << ((lane & 7) * 4) : 0u;
      bits |= __shfl_xor_sync(0xFFFFFFFFu, bits, 1);
      bits |= __shfl_xor_sync(0xFFFFFFFFu, bits, 2);
      bits |= __shfl_xor_sync(0xFFFFFFFFu, bits, 4);
      if ((lane & 7) == 0) m.valid[lane >> 3] = bits;
      __syncwarp();
      if (!*abort_flag) {
        if (lane == 0) {
          const uint32_t bytes = static_cast<uint32_t>(__popc(pages) * ps * D);
          mbar_arrive(smem_addr(&sh.mfull[ms]));
          mbar_arrive_expect_tx(smem_addr(&sh.kfull[ks]), bytes);
          mbar_arrive_expect_tx(smem_addr(&sh.vfull[vs]), bytes);
        }
        __syncwarp();
        if (ok) {
          const int y = static_cast<int>(now.at * ps);
          const uint32_t to = static_cast<uint32_t>(lane * ps * D);
          at_tma_load(k_s + ks * kTileBytes + to, &p.tm_k, 0, y, smem_addr(&sh.kfull[ks]));
          at_tma_load(v_s + vs * kTileBytes + to, &p.tm_v, 0, y, smem_addr(&sh.vfull[vs]));
        }
      }
      __syncwarp();
      now = then;
      have = next_have;
      ++g;
    }
    // On an abort the copies in flight are waited for (bounded) before the CTA ends.
    if (*abort_flag && lane == 0) {
      for (uint32_t i = g > 4 ? g - 4 : 0; i < g; ++i) {
        (void)mbar_wait_bounded(smem_addr(&sh.kfull[i % KST]), (i / KST) & 1u);
        (void)mbar_wait_bounded(smem_addr(&sh.vfull[i % VST]), (i / VST) & 1u);
      }
    }
  } else if (warp == kMmaWarp) {
    if (lane == 0) {
      constexpr uint32_t kSwz = D == 128 ? 2u : 4u;    // K tile and queries: rows of D bytes, swizzled over D bytes
      auto scores = [&](uint32_t t) {                  // S^T of tile t: K (codes) x (hi + lo)
        wait(sh.kfull[t % KST], (t / KST) & 1u, kFaultFullWait);
        wait(sh.sempty[t & 1u], ((t >> 1) & 1u) ^ 1u, kFaultEmptyWait);
        if (*abort_flag) return;
        at_fence_after();
        const uint32_t k = k_s + (t % KST) * kTileBytes, d = tmem + (t & 1u) * N;
#pragma unroll
        for (int part = 0; part < 2; ++part)
#pragma unroll
          for (int kk = 0; kk < D / 32; ++kk)
            at_mma_f8(d, at_desc(k + kk * 32, 16, 8 * D, kSwz),
                      at_desc(q_s + part * N * D + kk * 32, 16, 8 * D, kSwz), at_idesc(N, false),
                      part != 0 || kk != 0 ? 1u : 0u);
        at_commit(smem_addr(&sh.kempty[t % KST]));
        at_commit(smem_addr(&sh.sfull[t & 1u]));
      };
      uint32_t seg = 0;
      while (next_segment(p, cur, sh.w0, sg)) {
        const uint32_t n = static_cast<uint32_t>(sg.t1 - sg.t0);
        wait(sh.qfull, seg & 1u, kFaultFullWait);
        scores(g);
        for (uint32_t i = 0; i < n; ++i) {
          if (i + 1 < n) scores(g + i + 1);
          const uint32_t t = g + i;
          wait(sh.wfull[t & 1u], (t >> 1) & 1u, kFaultFullWait);
          wait(sh.pfull[t & 1u], (t >> 1) & 1u, kFaultFullWait);
          if (*abort_flag) continue;
          at_fence_after();
          const uint32_t v = wide_s + (t & 1u) * kWideBytes, pp = p_s + (t % PB) * p_bytes<N>();
#pragma unroll
          for (int kk = 0; kk < kTile / 16; ++kk)
            at_mma_f16(tmem + 2 * N, at_desc(v + kk * 2048, 16384, 1024, 2), at_desc(pp + kk * 16 * kPRow, 16384, 8 * kPRow, kPSwz),
                       at_idesc(N, true), i != 0 || kk != 0 ? 1u : 0u);
          at_commit(smem_addr(&sh.pvdone[t & 1u]));
        }
        g += n;
        ++seg;
      }
    }
  } else if (warp >= kSoftWarps) {
    // Widen V: 16 codes (one 16-byte piece of a token) at a time, tokens that are not visible as zeros.
    const int tid = threadIdx.x - kSoftWarps * 32;
    constexpr int kPieces = D / 16;                    // of a token
    while (next_segment(p, cur, sh.w0, sg)) {
      for (int i = sg.t0; i < sg.t1; ++i, ++g) {
        wait(sh.mfull[g % kMetaSlots], (g / kMetaSlots) & 1u, kFaultFullWait);
        wait(sh.vfull[g % VST], (g / VST) & 1u, kFaultFullWait);
        if (g >= 2) wait(sh.pvdone[g & 1u], ((g >> 1) & 1u) ^ 1u, kFaultEmptyWait);   // the product that read this buffer
        const TileMeta& m = sh.meta[g % kMetaSlots];
        const uint32_t src = v_s + (g % VST) * kTileBytes, dst = wide_s + (g & 1u) * kWideBytes;
#pragma unroll
        for (int it = 0; it < kPieces; ++it) {
          const int piece = it * 128 + tid, key = piece / kPieces, c = piece % kPieces;
          uint4 x = lds128(src + static_cast<uint32_t>(piece) * 16u);
          if (!((m.valid[key >> 5] >> (key & 31)) & 1u)) x = make_uint4(0u, 0u, 0u, 0u);
          const uint32_t row = dst + (c >= 4 ? 16384u : 0u) + static_cast<uint32_t>(key) * 128u;
          const uint32_t lo = static_cast<uint32_t>(((c & 3) * 2) ^ (key & 7)) * 16u;
          const uint32_t hi = static_cast<uint32_t>(((c & 3) * 2 + 1) ^ (key & 7)) * 16u;
          const uint32_t a0 = e4m3x2_to_f16x2(x.x & 0xFFFFu), a1 = e4m3x2_to_f16x2(x.x >> 16);
          const uint32_t a2 = e4m3x2_to_f16x2(x.y & 0xFFFFu), a3 = e4m3x2_to_f16x2(x.y >> 16);
          const uint32_t b0 = e4m3x2_to_f16x2(x.z & 0xFFFFu), b1 = e4m3x2_to_f16x2(x.z >> 16);
          const uint32_t b2 = e4m3x2_to_f16x2(x.w & 0xFFFFu), b3 = e4m3x2_to_f16x2(x.w >> 16);
          if (c < 4) {                                 // (the order spreads a quarter warp over all banks)
            sts128(row + lo, a0, a1, a2, a3);
            sts128(row + hi, b0, b1, b2, b3);
          } else {
            sts128(row + hi, b0, b1, b2, b3);
            sts128(row + lo, a0, a1, a2, a3);
          }
        }
        at_fence_async();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(smem_addr(&sh.vempty[g % VST]));
          mbar_arrive(smem_addr(&sh.wfull[g & 1u]));
        }
      }
    }
  } else {
    // Softmax: thread (warp % 4, lane) holds token 32 (warp % 4) + lane of the
    // tile; group wg = warp / 4 owns columns [wg HALF, (wg + 1) HALF).
    const int wg = warp >> 2, wq = warp & 3, key = wq * 32 + lane, tid = threadIdx.x & 127;
    const uint32_t bar_id = 1u + static_cast<uint32_t>(wg);
    const uint32_t lanes = static_cast<uint32_t>(wq * 32) << 16;
    const int page_of = key / ps;
    const int c0 = wg * HALF;
    while (next_segment(p, cur, sh.w0, sg)) {
      // The queries: one power-of-two scale per row and two e4m3 parts.
      const int row0 = sg.rt * p.tile_rows;
      const int nrows = min(p.tile_rows, p.rows - row0);
      constexpr int kPer = D / 8;                      // threads per row, 8 elements each
      named_sync(3, kSoftWarps * 32);                  // the previous segment's rows and references are no longer read
      for (int r = threadIdx.x / kPer; r < N; r += kSoftWarps * 32 / kPer) {
        const int e = threadIdx.x % kPer;
        uint4 x = make_uint4(0u, 0u, 0u, 0u);
        const int rr = row0 + r;
        if (r < nrows)
          x = *reinterpret_cast<const uint4*>(p.q + sg.b * p.qb + (rr / p.G) * p.ql +
                                              (static_cast<int64_t>(sg.h) * p.G + rr % p.G) * p.qh + e * 16);
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t u0 = w[i] & 0x7FFFu, u1 = (w[i] >> 16) & 0x7FFFu;
          top = max(top, u0 < 0x7F80u ? u0 : 0u);
          top = max(top, u1 < 0x7F80u ? u1 : 0u);
        }
#pragma unroll
        for (int o = kPer / 2; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
        const float s = block_scale(__uint_as_float(top << 16));
        // (the largest bf16 needs 2^120: its inverse is still normal)
        const float inv = __uint_as_float(0x7F000000u - __float_as_uint(s));
        uint32_t hi[2] = {0u, 0u}, lo[2] = {0u, 0u};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float a = bf16lo(w[i]) * inv, b = bf16hi(w[i]) * inv;
          if (!(fabsf(a) <= 448.0f)) a = __int_as_float(0x7FFFFFFF);   // infinities and NaN: the row's results are NaN
          if (!(fabsf(b) <= 448.0f)) b = __int_as_float(0x7FFFFFFF);
          const uint32_t h = e4m3x2(a, b);
          float ha, hb;
          f16x2_to_f32(e4m3x2_to_f16x2(h), ha, hb);
          const uint32_t l = e4m3x2(a - ha, b - hb);
          hi[i >> 1] |= h << (16 * (i & 1));
          lo[i >> 1] |= l << (16 * (i & 1));
        }
        const int chunk = e >> 1;
        const uint32_t at = static_cast<uint32_t>(r * D + ((D == 128 ? chunk ^ (r & 7) : chunk ^ ((r >> 1) & 3)) << 4) +
                                                  (e & 1) * 8);
        sts64(q_s + at, hi[0], hi[1]);
        sts64(q_s + N * D + at, lo[0], lo[1]);
        if (e == 0) {
          sh.f[r] = s;
          sh.nm[r] = -kUnset;
          sh.row[r] = r < nrows ? static_cast<int32_t>((sg.b * p.L + rr / p.G) * p.Hq + static_cast<int64_t>(sg.h) * p.G +
                                                       rr % p.G)
                                : -1;
        }
      }
      at_fence_async();
      named_sync(3, kSoftWarps * 32);
      if (lane == 0) mbar_arrive(smem_addr(&sh.qfull));

      uint64_t l2[HALF / 2];                           // this token's share of the sums
#pragma unroll
      for (int i = 0; i < HALF / 2; ++i) l2[i] = 0;
      float vref = 0x1p-120f;
      for (int ti = sg.t0; ti < sg.t1; ++ti, ++g) {
        wait(sh.mfull[g % kMetaSlots], (g / kMetaSlots) & 1u, kFaultFullWait);
        const TileMeta& m = sh.meta[g % kMetaSlots];
        const bool valid = (m.valid[wq] >> lane) & 1u;
        const float ck = m.ks[page_of], vs = m.vs[page_of];
        const uint64_t ck2 = pack2(ck, ck);
        wait(sh.sfull[g & 1u], (g >> 1) & 1u, kFaultFullWait);
        at_fence_after();
        const uint32_t s_t = tmem + lanes + (g & 1u) * N + c0;
        // Does any score exceed its reference by more than the slack?
        float over = -kInf;
#pragma unroll
        for (int c = 0; c < HALF; c += C) {
          uint32_t r[C];
          at_ld<C>(s_t + c, r);
#pragma unroll
          for (int i = 0; i < C; i += 4) {
            const float4 f = *reinterpret_cast<const float4*>(&sh.f[c0 + c + i]);
            const float4 n = *reinterpret_cast<const float4*>(&sh.nm[c0 + c + i]);
            float x0, x1, x2, x3;
            unpack2(fma2(at_mul2(pack2(__uint_as_float(r[i]), __uint_as_float(r[i + 1])), ck2), pack2(f.x, f.y),
                         pack2(n.x, n.y)), x0, x1);
            unpack2(fma2(at_mul2(pack2(__uint_as_float(r[i + 2]), __uint_as_float(r[i + 3])), ck2), pack2(f.z, f.w),
                         pack2(n.z, n.w)), x2, x3);
            over = fmaxf(fmaxf(over, fmaxf(x0, x1)), fmaxf(x2, x3));
          }
        }
        const bool raise = valid && (over > kSlack || vs > 16.0f * vref);
        if (group_any(bar_id, raise)) {                // uniform over the group
          // New references: the largest score of each column so far.
#pragma unroll
          for (int c = 0; c < HALF; c += C) {
            uint32_t r[C];
            at_ld<C>(s_t + c, r);
            float mine = -kInf;
#pragma unroll
            for (int i = 0; i < C; ++i) {
              const float x = valid ? __uint_as_float(r[i]) * ck * sh.f[c0 + c + i] : -kInf;
              const float mx = warp_max_f32(x == x ? x : -kInf);
              if (lane == i) mine = mx;
            }
            if (lane < C) sh.red[wg][wq][c + lane] = mine;
          }
          float vmax = warp_max_f32(valid ? vs : 0.0f);
          if (lane == 0) sh.fac_o[c0 + wq] = vmax;
          named_sync(bar_id, 128);
          vmax = fmaxf(fmaxf(sh.fac_o[c0], sh.fac_o[c0 + 1]), fmaxf(sh.fac_o[c0 + 2], sh.fac_o[c0 + 3]));
          const float vnew = fmaxf(vref, vmax);
          named_sync(bar_id, 128);
          if (tid < HALF) {
            const float old = -sh.nm[c0 + tid];
            const float mx = fmaxf(fmaxf(sh.red[wg][0][tid], sh.red[wg][1][tid]),
                                   fmaxf(sh.red[wg][2][tid], sh.red[wg][3][tid]));
            const float now = fmaxf(old, mx);
            const float d = ex2_approx(old - now);
            sh.nm[c0 + tid] = -now;
            sh.fac_l[c0 + tid] = d;
            sh.fac_o[c0 + tid] = d * (vref / vnew);
          }
          vref = vnew;
          named_sync(bar_id, 128);
#pragma unroll
          for (int i = 0; i < HALF / 2; ++i)
            l2[i] = at_mul2(l2[i], *reinterpret_cast<const uint64_t*>(&sh.fac_l[c0 + 2 * i]));
          if (ti > sg.t0) {                            // the accumulator holds earlier tiles
            wait(sh.pvdone[(g - 1) & 1u], ((g - 1) >> 1) & 1u, kFaultFullWait);
            at_fence_after();
#pragma unroll
            for (int c = 0; c < HALF; c += 8) {
              uint32_t r[8];
              const uint32_t o_t = tmem + lanes + 2 * N + c0 + c;
              at_ld<8>(o_t, r);
#pragma unroll
              for (int i = 0; i < 8; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) * sh.fac_o[c0 + c + i]);
              at_st8(o_t, r);
            }
            at_fence_before();
          }
          named_sync(bar_id, 128);                     // (fac_o and red are free again)
        }
        // P of this token, in fp16 for the product and summed in fp32.
        const float vr = valid ? vs * (kPUnit / vref) : 0.0f;
        const uint64_t vr2 = pack2(vr, vr);
        // the product that read this buffer last
        if (g >= PB) wait(sh.pvdone[(g - PB) & 1u], ((g - PB) >> 1) & 1u, kFaultEmptyWait);
        const uint32_t p_row = p_s + (g % PB) * p_bytes<N>() + static_cast<uint32_t>(key) * kPRow;
        const int swz = kPRow == 128 ? key & 7 : (kPRow == 64 ? (key >> 1) & 3 : (key >> 2) & 1);
#pragma unroll
        for (int c = 0; c < HALF; c += C) {
          uint32_t r[C];
          at_ld<C>(s_t + c, r);
          if (c + C == HALF) {                         // the scores have been read
            at_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_addr(&sh.sempty[g & 1u]));
          }
#pragma unroll
          for (int i = 0; i < C; i += 8) {
            uint32_t o[4];
#pragma unroll
            for (int q = 0; q < 8; q += 4) {
              const float4 f = *reinterpret_cast<const float4*>(&sh.f[c0 + c + i + q]);
              const float4 n = *reinterpret_cast<const float4*>(&sh.nm[c0 + c + i + q]);
              float x0, x1, x2, x3;
              unpack2(fma2(at_mul2(pack2(__uint_as_float(r[i + q]), __uint_as_float(r[i + q + 1])), ck2),
                           pack2(f.x, f.y), pack2(n.x, n.y)), x0, x1);
              unpack2(fma2(at_mul2(pack2(__uint_as_float(r[i + q + 2]), __uint_as_float(r[i + q + 3])), ck2),
                           pack2(f.z, f.w), pack2(n.z, n.w)), x2, x3);
              uint64_t e0 = pack2(ex2_approx(x0), ex2_approx(x1)), e1 = pack2(ex2_approx(x2), ex2_approx(x3));
              if (!valid) e0 = e1 = 0;
              l2[(c + i + q) / 2] = add2(l2[(c + i + q) / 2], e0);
              l2[(c + i + q) / 2 + 1] = add2(l2[(c + i + q) / 2 + 1], e1);
              float y0, y1, y2, y3;
              unpack2(at_mul2(e0, vr2), y0, y1);
              unpack2(at_mul2(e1, vr2), y2, y3);
              o[q / 2] = f16x2(y0, y1);
              o[q / 2 + 1] = f16x2(y2, y3);
            }
            const int col = c0 + c + i;
            sts128(p_row + static_cast<uint32_t>(col >> 6) * 16384u +
                       static_cast<uint32_t>(((col & 63) >> 3) ^ swz) * 16u, o[0], o[1], o[2], o[3]);
          }
        }
        at_fence_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(&sh.pfull[g & 1u]));
      }

      // The segment's sums over its tokens, then its rows.
#pragma unroll
      for (int i = 0; i < HALF / 2; ++i) {
        float a, b;
        unpack2(l2[i], a, b);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
          a += __shfl_xor_sync(0xFFFFFFFFu, a, o);
          b += __shfl_xor_sync(0xFFFFFFFFu, b, o);
        }
        if (lane == 0) {
          sh.red[wg][wq][2 * i] = a;
          sh.red[wg][wq][2 * i + 1] = b;
        }
      }
      named_sync(bar_id, 128);
      wait(sh.pvdone[(g - 1) & 1u], ((g - 1) >> 1) & 1u, kFaultFullWait);
      at_fence_after();
      const bool whole = sg.t0 == 0 && sg.t1 == sg.T;
      const int slot = 2 * blockIdx.x + (sg.starts_range ? 0 : 1);
      const int d = key;                               // the accumulator's lane is a dimension
#pragma unroll 1
      for (int c = 0; c < HALF; c += 8) {
        uint32_t r[8];
        at_ld<8>(tmem + lanes + 2 * N + c0 + c, r);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int n = c0 + c + i;
          const int32_t row = sh.row[n];
          if (row < 0) continue;
          const float l = (sh.red[wg][0][c + i] + sh.red[wg][1][c + i]) + (sh.red[wg][2][c + i] + sh.red[wg][3][c + i]);
          const float o = __uint_as_float(r[i]) * (vref * (1.0f / kPUnit));
          if (whole) {
            if (d < D) {
              uint16_t u;
              const float y = l == 0.0f ? 0.0f : o / l;
              asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(u) : "f"(y));
              p.out[static_cast<int64_t>(row) * D + d] = u;
            }
            if (d == 0) p.lse[row] = l == 0.0f ? -kInf : -sh.nm[n] * kLn2 + logf(l);
          } else {
            if (d < D) p.part_o[(static_cast<int64_t>(slot) * N + n) * D + d] = o;
            if (d == 0) {
              p.part_ml[(static_cast<int64_t>(slot) * N + n) * 2] = -sh.nm[n];
              p.part_ml[(static_cast<int64_t>(slot) * N + n) * 2 + 1] = l;
            }
          }
        }
      }
      at_fence_before();
    }
  }
  at_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    at_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kCols) : "memory");
  }
}

// One warp per output row: joins the parts of the items that several CTAs
// share, in CTA order (a part's reference may differ from the others').
template <int D>
__global__ void __launch_bounds__(128) attend_join_kernel(const __grid_constant__ AttendParams p, int N) {
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  if (row >= p.B * p.L * p.Hq) return;
  const int64_t hq = row % p.Hq, l = row / p.Hq % p.L, b = row / (p.Hq * p.L);
  const int64_t h = hq / p.G, rr = l * p.G + hq % p.G;
  const int64_t rt = rr / p.tile_rows;
  const int n = static_cast<int>(rr % p.tile_rows);
  const int64_t hr = static_cast<int64_t>(p.c.heads) * p.row_tiles;
  const int64_t total = tiles_before(p, p.B) * hr;
  const int64_t T = tiles_of(p, b);
  const int64_t i0 = tiles_before(p, b) * hr + (h * p.row_tiles + rt) * T, i1 = i0 + T;   // the item's tiles
  // the CTA that holds tile w: the largest c with total c / ctas <= w
  auto owner = [&](int64_t w) {
    int64_t c = w * p.ctas / total;
    while (c + 1 < p.ctas && cta_begin(total, c + 1, p.ctas) <= w) ++c;
    while (cta_begin(total, c, p.ctas) > w) --c;
    return c;
  };
  const int64_t ca = owner(i0), cb = owner(i1 - 1);
  if (ca == cb) return;                                // written whole
  float m = kUnset, sum = 0.0f;
  float o[D / 32] = {};
  for (int64_t c = ca; c <= cb; ++c) {
    const int64_t begin = cta_begin(total, c, p.ctas);
    if (begin == cta_begin(total, c + 1, p.ctas)) continue;
    const int64_t slot = 2 * c + (begin >= i0 ? 0 : 1);
    const float* ml = p.part_ml + (slot * N + n) * 2;
    const float mc = __ldcg(ml), lc = __ldcg(ml + 1);
    const float now = fmaxf(m, mc);
    const float fa = ex2_approx(m - now), fb = ex2_approx(mc - now);
    sum = sum * fa + lc * fb;
#pragma unroll
    for (int i = 0; i < D / 32; ++i)
      o[i] = o[i] * fa + __ldcg(p.part_o + (slot * N + n) * D + i * 32 + lane) * fb;
    m = now;
  }
#pragma unroll
  for (int i = 0; i < D / 32; ++i) {
    uint16_t u;
    const float y = sum == 0.0f ? 0.0f : o[i] / sum;
    asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(u) : "f"(y));
    p.out[row * D + i * 32 + lane] = u;
  }
  if (lane == 0) p.lse[row] = sum == 0.0f ? -kInf : m * kLn2 + logf(sum);
}

}  // namespace dllm

namespace {

using namespace dllm;

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn at_encode_fn() {
  static EncodeTiledFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, []() {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(f);
  });
  return fn;
}

// One pool as rows of head_dim bytes, a box being the tokens of one page and head.
bool pool_map(CUtensorMap* m, void* base, const CacheView& c, CUtensorMapSwizzle swizzle) {
  EncodeTiledFn fn = at_encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(c.dim), static_cast<cuuint64_t>(c.pages * c.heads * c.page_size)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(c.dim)};
  const cuuint32_t box[2] = {static_cast<cuuint32_t>(c.dim), static_cast<cuuint32_t>(c.page_size)};
  const cuuint32_t estr[2] = {1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, base, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct AttendVariant {
  const void* kernel;
  int smem;
};

template <int N>
AttendVariant attend_variant_n(int dim) {
  if (dim == 64) return {reinterpret_cast<const void*>(&attend_kernel<64, N>), attend_smem<64, N>()};
  return {reinterpret_cast<const void*>(&attend_kernel<128, N>), attend_smem<128, N>()};
}

AttendVariant attend_variant(int dim, int n) {
  switch (n) {
    case 16: return attend_variant_n<16>(dim);
    case 32: return attend_variant_n<32>(dim);
    case 64: return attend_variant_n<64>(dim);
    default: return attend_variant_n<128>(dim);
  }
}

struct AttendDevice {
  int sms = 0;
  cudaError_t err = cudaSuccess;
};
AttendDevice g_at[64];
std::once_flag g_at_once[64];

const AttendDevice* attend_device() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return nullptr;
  std::call_once(g_at_once[dev], [dev]() {
    AttendDevice& d = g_at[dev];
    d.err = cudaDeviceGetAttribute(&d.sms, cudaDevAttrMultiProcessorCount, dev);
    for (int dim = 64; dim <= 128; dim += 64)
      for (int n = 16; n <= 128 && d.err == cudaSuccess; n *= 2) {
        const AttendVariant v = attend_variant(dim, n);
        d.err = cudaFuncSetAttribute(v.kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, v.smem);
      }
    if (d.err != cudaSuccess) (void)cudaGetLastError();  // reported through the status; no sticky error
  });
  return g_at[dev].err == cudaSuccess ? &g_at[dev] : nullptr;
}

// The row tiles of a key head and the columns of a tile: as few tiles as 128
// columns allow, equally filled, then the narrowest built width that holds
// one (a width is the tensor core's N and the softmax's work per token).
struct RowTiles {
  int64_t tiles, rows;
  int n;
};
RowTiles row_tiles(int64_t rows) {
  RowTiles t;
  t.tiles = (rows + 127) / 128;
  t.rows = (rows + t.tiles - 1) / t.tiles;
  t.n = t.rows <= 16 ? 16 : (t.rows <= 32 ? 32 : (t.rows <= 64 ? 64 : 128));
  return t;
}

constexpr size_t kAttendHeader = 256;  // the fault word

size_t attend_workspace(int64_t ctas, int n, int dim) {
  return kAttendHeader + static_cast<size_t>(2 * ctas) * n * (dim + 2) * sizeof(float);
}

}  // namespace

extern "C" {

size_t dllm_cache_attention_workspace_size(int64_t B, int64_t L, int64_t Hq, int64_t heads, int64_t head_dim) {
  using namespace dllm;
  if (B <= 0 || L <= 0 || Hq <= 0 || heads <= 0 || Hq % heads != 0 || head_dim <= 0 || head_dim > 128 ||
      mul_or_neg(L, Hq) < 0)
    return kAttendHeader;
  const AttendDevice* dev = attend_device();
  return attend_workspace(dev ? dev->sms : 1024, row_tiles(L * (Hq / heads)).n, static_cast<int>(head_dim));
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
  // (a TMA coordinate is an int32: the pool's rows of one token and head)
  if (rows > INT32_MAX || cache->num_pages * cache->heads * cache->page_size > INT32_MAX) return DLLM_ERR_UNSUPPORTED;
  if (!workspace) return DLLM_ERR_WORKSPACE;
  if (!aligned16(workspace)) return DLLM_ERR_INVALID_ARGUMENT;
  const RowTiles rt = row_tiles(L * (Hq / cache->heads));
  if (workspace_bytes < attend_workspace(1, rt.n, cache->head_dim)) return DLLM_ERR_WORKSPACE;
  const AttendDevice* dev = attend_device();
  if (!dev) return DLLM_ERR_CUDA;
  // One CTA per SM, fewer when there are fewer tiles than that.
  const int64_t most = mul_or_neg(mul_or_neg(B, cache->heads), rt.tiles * ((cap + kTile - 1) / kTile));
  if (most < 0 || most > (static_cast<int64_t>(1) << 52)) return DLLM_ERR_UNSUPPORTED;
  const int64_t ctas = std::min<int64_t>(dev->sms, most);
  if (workspace_bytes < attend_workspace(ctas, rt.n, cache->head_dim)) return DLLM_ERR_WORKSPACE;
  AttendParams p;
  std::memset(&p, 0, sizeof(p));
  p.c = cache_view(*cache);
  const bool d64 = cache->head_dim == 64;
  if (!pool_map(&p.tm_k, cache->k, p.c, d64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B) ||
      !pool_map(&p.tm_v, cache->v, p.c, CU_TENSOR_MAP_SWIZZLE_NONE))
    return DLLM_ERR_CUDA;
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
  p.G = static_cast<int32_t>(Hq / cache->heads);
  p.rows = static_cast<int32_t>(L * p.G);
  p.row_tiles = static_cast<int32_t>(rt.tiles);
  p.tile_rows = static_cast<int32_t>(rt.rows);
  p.ctas = static_cast<int32_t>(ctas);
  uint8_t* w = static_cast<uint8_t*>(workspace);
  p.fault = reinterpret_cast<int32_t*>(w);
  p.part_o = reinterpret_cast<float*>(w + kAttendHeader);
  p.part_ml = p.part_o + 2 * ctas * rt.n * cache->head_dim;
  void* args[] = {&p};
  const AttendVariant v = attend_variant(cache->head_dim, rt.n);
  st = launch_pdl(v.kernel, dim3(static_cast<unsigned>(ctas)), dim3(kAttendThreads), static_cast<size_t>(v.smem), stream,
                  args);
  if (st != DLLM_OK) return st;
  int n = rt.n;
  void* jargs[] = {&p, &n};
  st = launch_pdl(d64 ? reinterpret_cast<const void*>(&attend_join_kernel<64>)
                      : reinterpret_cast<const void*>(&attend_join_kernel<128>),
                  dim3(static_cast<unsigned>((rows + 3) / 4)), dim3(128), 0, stream, jargs);
  if (st != DLLM_OK || !weights) return st;
  return launch_pdl(d64 ? reinterpret_cast<const void*>(&attend_weights_kernel<64>)
                        : reinterpret_cast<const void*>(&attend_weights_kernel<128>),
                    dim3(static_cast<unsigned>((cap + 127) / 128), static_cast<unsigned>(cache->heads),
                         static_cast<unsigned>(B)),
                    dim3(128), 0, stream, args);
}

}  // extern "C"
