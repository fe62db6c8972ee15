// dllm_attend.cu -- attention of a block of queries over the paged 8-bit
// key/value cache, and the attention weight each cached token draws.
//
// Mathematics.  For the rows r of one key head (the queries of its head group)
// and its tokens j: x = scale log2 e s_k(j) q_r . k_j, y = 2^(x + log2 s_v(j) -
// m_r), out_r = sum y v_j / l_r with l_r = sum y / s_v(j), lse_r = ln 2 (m_r +
// log2 l_r).  The running reference m_r follows a row's largest probability times
// value scale, so what a token adds to the row is held to that and to nothing
// that another row, or a page the row does not attend to, has.
//
// The transposed products.  A tile is 128 tokens of one head.  S^T = K Q^T and
// O^T += V^T P^T put the tokens (then the head dimension) on the tensor core's
// 128 rows and the queries on its N columns, so a block of 32 queries, or a
// single one, costs N = 32 columns and not a padded tile of 128 rows.
//
// K and V stay in 8 bits from HBM to the tensor core (kind::f8f6f4 on the codes
// as TMA brought them): what bounds few rows is the bytes of the cache, and
// then shared memory, which a widened copy of V crosses five times instead of
// two.  The other operand is split into e4m3 parts instead:
//   * a query row into hi = e4m3(q / s) and lo = e4m3(q / s - hi), s a power of
//     two per row: a bf16 value has 8 significant bits and e4m3 holds 4 of
//     either sign, so hi + lo is exact for elements above 2^-9 of the row's
//     largest and off by at most 2^-18 of it below;
//   * P = 64 y <= 256, with fp16's 11 bits (bf16 has 8), into three parts of 4
//     bits, the second and third of 16 and 256 times the remainder, with
//     accumulators of their own: exact but for the rounding to fp16, which is
//     2^-12 of the value, or 2^-22 of the row's largest y where that is more (a
//     new reference lies 1 above its y, in log2; 64 y rounds at 2^-17).
// A reference moves only when a y exceeds it by more than 2 (log2 units), so the
// accumulators in TMEM are rarely rescaled; statistics and sums are fp32.
//
// Measured (head_dim 128, pages of 64 and 128, one GB300, replayed in a graph; with
// one scale on all pages, where references rise in few tiles, and with scales of
// three binades): single tokens, 32 over 8 heads, 4 sequences of 60001 to 131072:
// 123 us both, 6.35 TB/s of cache (95 % of a copy); blocks of 32 queries, 32 heads,
// 8 x 2306 tokens: 39.4 and 42.3 us, 245 and 229 TFLOP/s; 224 rows a head, 16 x
// 5096 tokens, 4 heads: 87.4 and 100.8 us, 428 and 371 TFLOP/s, bound by the softmax
// groups' chain of waits and instructions (of a tile's 3730 clocks in a group, for
// 128 x 56 scores, 720 pass waiting for the scores, 530 reading them, 680 with the
// maxima and the vote, 1270 with three binades, and 1220 with P; tensor pipe 29 %).
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
  int32_t half;                // rows of a softmax group: tile_rows, or half of them when the groups are paired
  int32_t ctas;
  int32_t seg_cost;            // what an item costs besides its tiles, in tiles
  float* part_o;               // (2 ctas, columns, D): a CTA's unfinished first and last segment
  float* part_ml;              // (2 ctas, columns, 2)
  int32_t* fault;
};

__device__ __forceinline__ int attend_len(const AttendParams& p, int64_t b) {
  const int64_t n = __ldcg(p.lens + b);
  return static_cast<int>(n < 0 ? 0 : (n > p.cap ? p.cap : n));
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

// Issued by the one thread of the warp whose `lead` is set; the whole warp
// executes the code around it, so that addresses and descriptors stay in
// uniform registers (computed by a single thread, they cost several times the
// product's own issue time).  Descriptors share their high words.
__device__ __forceinline__ void at_mma_f8(uint32_t lead, uint32_t d, uint32_t a_lo, uint32_t a_hi, uint32_t b_lo,
                                          uint32_t b_hi, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b64 a, b;\n\tsetp.ne.u32 p, %6, 0;\n\tsetp.ne.u32 q, %7, 0;\n\t"
      "mov.b64 a, {%1, %2};\n\tmov.b64 b, {%3, %4};\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %5, p;\n\t}" ::"r"(d),
      "r"(a_lo), "r"(a_hi), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(acc), "r"(lead)
      : "memory");
}

__device__ __forceinline__ void at_commit(uint32_t lead, uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar),
      "r"(lead)
      : "memory");
}

__device__ __forceinline__ uint32_t elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r;
}
__device__ __forceinline__ void at_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void at_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
// Shared-memory writes of this thread become visible to the tensor core.
__device__ __forceinline__ void at_fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// 16 consecutive fp32 columns of this warp's 32 TMEM lanes, one lane a thread.
__device__ __forceinline__ void at_ld16(uint32_t t, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(t)
      : "memory");
}

// Fragments: of 16 TMEM lanes (tokens) by 8 j columns, thread t gets the tokens
// t / 4 and t / 4 + 8 and of each 8 columns the two at 2 (t mod 4): register 4 j +
// 2 s + e is token t / 4 + 8 s, column 8 j + 2 (t mod 4) + e.  A thread then
// meets a quarter of the columns, whose scales and references it can keep in
// registers (read per column from shared memory by every token's thread, they
// cost 512 bytes a warp instruction, more than all else in shared memory).
// 64 columns at each of two places, one wait for both.
__device__ __forceinline__ void at_frag64x2(uint32_t t0, uint32_t t1, uint32_t (&a)[32], uint32_t (&b)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x8.b32 {"
      "%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%64];\n\t"
      "tcgen05.ld.sync.aligned.16x256b.x8.b32 {"
      "%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,"
      "%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63}, [%65];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(a[0]), "=r"(a[1]), "=r"(a[2]), "=r"(a[3]), "=r"(a[4]), "=r"(a[5]), "=r"(a[6]), "=r"(a[7]),
        "=r"(a[8]), "=r"(a[9]), "=r"(a[10]), "=r"(a[11]), "=r"(a[12]), "=r"(a[13]), "=r"(a[14]), "=r"(a[15]),
        "=r"(a[16]), "=r"(a[17]), "=r"(a[18]), "=r"(a[19]), "=r"(a[20]), "=r"(a[21]), "=r"(a[22]), "=r"(a[23]),
        "=r"(a[24]), "=r"(a[25]), "=r"(a[26]), "=r"(a[27]), "=r"(a[28]), "=r"(a[29]), "=r"(a[30]), "=r"(a[31]),
        "=r"(b[0]), "=r"(b[1]), "=r"(b[2]), "=r"(b[3]), "=r"(b[4]), "=r"(b[5]), "=r"(b[6]), "=r"(b[7]),
        "=r"(b[8]), "=r"(b[9]), "=r"(b[10]), "=r"(b[11]), "=r"(b[12]), "=r"(b[13]), "=r"(b[14]), "=r"(b[15]),
        "=r"(b[16]), "=r"(b[17]), "=r"(b[18]), "=r"(b[19]), "=r"(b[20]), "=r"(b[21]), "=r"(b[22]), "=r"(b[23]),
        "=r"(b[24]), "=r"(b[25]), "=r"(b[26]), "=r"(b[27]), "=r"(b[28]), "=r"(b[29]), "=r"(b[30]), "=r"(b[31])
      : "r"(t0), "r"(t1)
      : "memory");
}

// 32 columns at each of two places.
__device__ __forceinline__ void at_frag32x2(uint32_t t0, uint32_t t1, uint32_t (&a)[16], uint32_t (&b)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {"
      "%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%32];\n\t"
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%33];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(a[0]), "=r"(a[1]), "=r"(a[2]), "=r"(a[3]), "=r"(a[4]), "=r"(a[5]), "=r"(a[6]), "=r"(a[7]),
        "=r"(a[8]), "=r"(a[9]), "=r"(a[10]), "=r"(a[11]), "=r"(a[12]), "=r"(a[13]), "=r"(a[14]), "=r"(a[15]),
        "=r"(b[0]), "=r"(b[1]), "=r"(b[2]), "=r"(b[3]), "=r"(b[4]), "=r"(b[5]), "=r"(b[6]), "=r"(b[7]),
        "=r"(b[8]), "=r"(b[9]), "=r"(b[10]), "=r"(b[11]), "=r"(b[12]), "=r"(b[13]), "=r"(b[14]), "=r"(b[15])
      : "r"(t0), "r"(t1)
      : "memory");
}

// 32 columns at each of four places.
__device__ __forceinline__ void at_frag32x4(uint32_t t0, uint32_t t1, uint32_t t2, uint32_t t3, uint32_t (&a)[16],
                                            uint32_t (&b)[16], uint32_t (&c)[16], uint32_t (&d)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {"
      "%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%64];\n\t"
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%65];\n\t"
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {"
      "%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47}, [%66];\n\t"
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {"
      "%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63}, [%67];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(a[0]), "=r"(a[1]), "=r"(a[2]), "=r"(a[3]), "=r"(a[4]), "=r"(a[5]), "=r"(a[6]), "=r"(a[7]),
        "=r"(a[8]), "=r"(a[9]), "=r"(a[10]), "=r"(a[11]), "=r"(a[12]), "=r"(a[13]), "=r"(a[14]), "=r"(a[15]),
        "=r"(b[0]), "=r"(b[1]), "=r"(b[2]), "=r"(b[3]), "=r"(b[4]), "=r"(b[5]), "=r"(b[6]), "=r"(b[7]),
        "=r"(b[8]), "=r"(b[9]), "=r"(b[10]), "=r"(b[11]), "=r"(b[12]), "=r"(b[13]), "=r"(b[14]), "=r"(b[15]),
        "=r"(c[0]), "=r"(c[1]), "=r"(c[2]), "=r"(c[3]), "=r"(c[4]), "=r"(c[5]), "=r"(c[6]), "=r"(c[7]),
        "=r"(c[8]), "=r"(c[9]), "=r"(c[10]), "=r"(c[11]), "=r"(c[12]), "=r"(c[13]), "=r"(c[14]), "=r"(c[15]),
        "=r"(d[0]), "=r"(d[1]), "=r"(d[2]), "=r"(d[3]), "=r"(d[4]), "=r"(d[5]), "=r"(d[6]), "=r"(d[7]),
        "=r"(d[8]), "=r"(d[9]), "=r"(d[10]), "=r"(d[11]), "=r"(d[12]), "=r"(d[13]), "=r"(d[14]), "=r"(d[15])
      : "r"(t0), "r"(t1), "r"(t2), "r"(t3)
      : "memory");
}

// 8 columns of each of an accumulator's three parts.
__device__ __forceinline__ void at_ld3(uint32_t t0, uint32_t t1, uint32_t t2, uint32_t (&r)[24]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%24];\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%8,%9,%10,%11,%12,%13,%14,%15}, [%25];\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%16,%17,%18,%19,%20,%21,%22,%23}, [%26];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23])
      : "r"(t0), "r"(t1), "r"(t2)
      : "memory");
}

// 16 columns back (complete after tcgen05.wait::st).
__device__ __forceinline__ void at_st16(uint32_t t, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(t),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

// Shared-memory matrix descriptors: start address / 16 (bits 0-13), leading
// and stride byte offsets / 16 (bits 16-29, 32-45), version 1 (bit 46), swizzle
// (bits 61-63: 2 = 128 bytes, 4 = 64 bytes, 6 = 32 bytes).
//   K-major (K and queries, a row of head_dim bytes per token or query): the
//   stride offset is the distance of 8-row groups, the leading one is not used.
//   MN-major (V and P, a row per token that is one swizzle span of head_dim or
//   N bytes): the leading offset is the distance of such spans along M or N, the
//   stride offset that of 8-token groups.
__device__ __forceinline__ uint32_t at_desc_lo(uint32_t saddr, uint32_t leading) {
  return ((saddr & 0x3FFFFu) >> 4) | (leading >> 4) << 16;
}
__device__ __forceinline__ constexpr uint32_t at_desc_hi(uint32_t stride, uint32_t swizzle) {
  return (stride >> 4) | 1u << 14 | swizzle << 29;
}

// Instruction descriptor: fp32 accumulator (bits 4-5 = 1), both operands e4m3
// (0), A and B MN-major where set (bits 15, 16), N / 8 in bits 17-22, M / 16 in
// bits 24-28.
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

// One part of P.  Two values of h = 2^-8 P <= 1 in fp16: the fp16 bits 14 .. 7
// (5 bits of exponent, the top one 0, and 3 of mantissa, subnormals alike) are
// the e4m3 code of P rounded toward zero; what is left, exact in fp16, times 16
// is the next part's h.  (Conversions to e4m3 run at a quarter of the rate of
// these integer and half-precision instructions.)
__device__ __forceinline__ uint32_t part_rest16(uint32_t h) {
  uint32_t r;
  asm("{\n\t.reg .b32 t;\n\tsub.rn.f16x2 t, %1, %2;\n\tmul.rn.f16x2 %0, t, %3;\n\t}"
      : "=r"(r)
      : "r"(h), "r"(h & 0xFF80FF80u), "r"(0x4C004C00u));  // 16, 16
  return r;
}
// The codes of four values: bits 14 .. 7 of the halves of a, then of b.
__device__ __forceinline__ uint32_t part_codes(uint32_t a, uint32_t b) { return __byte_perm(a << 1, b << 1, 0x7531); }

// Combines a value over the 8 lanes that hold the same columns.
template <bool MAX>
__device__ __forceinline__ float over_tokens(float v) {
#pragma unroll
  for (int o = 4; o < 32; o <<= 1) {
    const float w = __shfl_xor_sync(0xFFFFFFFFu, v, o);
    v = MAX ? fmaxf(v, w) : v + w;
  }
  return v;
}

// Four 8 x 8 matrices of 16-bit elements, register i's from thread t's row t / 4,
// elements 2 (t mod 4) and the next; thread t gives the address of row t mod 8 of
// matrix t / 8.
__device__ __forceinline__ void stmatrix4(uint32_t addr, uint32_t r0, uint32_t r1, uint32_t r2, uint32_t r3) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(r0), "r"(r1), "r"(r2),
               "r"(r3)
               : "memory");
}

// P's codes are stored as 16-bit pairs, two groups of 8 columns interleaved, so
// column n of the scores becomes column place(n) of P and of the accumulator:
// within 16, bit 3 of n moves below its bits 2 and 1.
__host__ __device__ constexpr int place(int n) { return (n & ~15) | ((n & 6) << 1) | ((n & 8) >> 2) | (n & 1); }

// ln(2^m l), -inf for l = 0: the exponent of l goes to m, which it may all but
// cancel (l is in units of the value scales' inverse).
__device__ __forceinline__ float lse_of(float m, float l) {
  int k;
  const float f = frexpf(l, &k);
  return l == 0.0f ? -kInf : fmaf(m + static_cast<float>(k), kLn2, logf(f));
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
// The work of all (batch row, key head, row tile) items, in that order, is dealt
// to the CTAs in equal contiguous ranges, so ragged batches and few long
// sequences load every SM alike.  It is counted in units: an item is as many
// units as it has tiles, preceded by seg_cost units for what an item costs
// whatever its length (loading its queries, writing its rows).  A CTA's range
// cuts at most its first and its last item short; those parts are joined
// afterwards in CTA order.
__device__ __forceinline__ int tiles_of(const AttendParams& p, int64_t b) {
  const int n = attend_len(p, b);
  return n > 0 ? (n + kTile - 1) / kTile : 1;  // (an empty sequence still has its zeros written)
}
__device__ __forceinline__ uint32_t units_of(const AttendParams& p, int64_t b) {
  return static_cast<uint32_t>(tiles_of(p, b) + p.seg_cost);
}

// CTA c's range begins at unit c q + min(c, r), q = total / ctas, r = total mod
// ctas (the host keeps totals below 2^31).
struct Split {
  uint32_t q, r;
  __device__ __forceinline__ Split(uint32_t total, uint32_t ctas) : q(total / ctas), r(total % ctas) {}
  __device__ __forceinline__ uint32_t begin(uint32_t c) const { return c * q + min(c, r); }
  // The CTA that holds a unit.
  __device__ __forceinline__ uint32_t owner(uint32_t w) const {
    const uint32_t wide = r * (q + 1);
    return w < wide ? w / (q + 1) : r + (w - wide) / max(q, 1u);
  }
};

struct Cursor {
  uint32_t w, w1;  // position and end of the CTA's range, in units
  int32_t b;       // batch row at w
  uint32_t off;    // position within the batch row's units
  int32_t len_of = -1, len = 0;   // a batch row and its length, read once for its items
};

struct Segment {
  int32_t b;
  int32_t h, rt;   // key head, row tile
  int32_t t0, t1;  // tiles [t0, t1) of the sequence
  int32_t T;       // tiles of the sequence
  int32_t len;
  bool starts_range;
};

// The next part of an item that has tiles in the CTA's range.
__device__ __forceinline__ bool next_segment(const AttendParams& p, Cursor& c, uint32_t w0, Segment& s) {
  while (c.w < c.w1) {
    s.b = c.b;
    if (c.len_of != c.b) {
      c.len = attend_len(p, c.b);
      c.len_of = c.b;
    }
    s.len = c.len;
    s.T = s.len > 0 ? (s.len + kTile - 1) / kTile : 1;
    const uint32_t units = static_cast<uint32_t>(s.T + p.seg_cost);
    const uint32_t hr = c.off / units, at = c.off % units;
    s.h = static_cast<int32_t>(hr / static_cast<uint32_t>(p.row_tiles));
    s.rt = static_cast<int32_t>(hr % static_cast<uint32_t>(p.row_tiles));
    const uint32_t end = min(units, at + (c.w1 - c.w));
    s.t0 = max(static_cast<int32_t>(at) - p.seg_cost, 0);
    s.t1 = max(static_cast<int32_t>(end) - p.seg_cost, 0);
    s.starts_range = c.w == w0;
    c.w += end - at;
    c.off += end - at;
    if (c.off == static_cast<uint32_t>(p.c.heads * p.row_tiles) * units) {
      ++c.b;
      c.off = 0;
    }
    if (s.t1 > s.t0) return true;
  }
  return false;
}

// One warp: the units of one head and row tile of all batch rows, in every lane.
__device__ __forceinline__ uint32_t all_units(const AttendParams& p) {
  uint32_t all = 0;
  for (int64_t b = threadIdx.x & 31; b < p.B; b += 32) all += units_of(p, b);
  return __reduce_add_sync(0xFFFFFFFFu, all);
}

// ---------------------------------------------------------------------------
// the attention kernel
// ---------------------------------------------------------------------------
// Warps: two groups of 4 softmax warps, one warp for the copies, one for the
// products.  A group owns a score buffer, a P buffer and an accumulator, and
// works with N columns.  A "job" is one tile for one group:
//   taking turns (at most N rows): the groups take the tiles alternately, each
//   with references and sums of its own, joined at the segment's end (a job is a
//   chain of waits, TMEM reads and barriers longer than the time of a tile, so
//   two are in flight);
//   paired (up to 2 N rows): both groups take every tile, each for its half of
//   the rows, so K and V are read once for up to 128 rows.
// Job J belongs to group J & 1 and is that group's (J >> 1)-th.
template <int N, bool PAIR>
struct AttendShape {
  static constexpr int kRows = PAIR ? 2 * N : N;             // columns of both groups
  static constexpr bool kConcat = N == 32;                   // hi and lo parts as 2 N columns of one product
  static constexpr int kScoreCols = kConcat ? 2 * N : N;     // (with N = 64 TMEM has no room: two products, one sum)
  static constexpr int kStages = N == 32 ? 5 : 4;            // of the K and V rings
  static constexpr int kPBytes = 3 * kTile * N;
  static constexpr int kScore = 0, kAcc = 2 * kScoreCols;    // TMEM columns: scores, then accumulators of 3 N
};
constexpr int kSoftWarps = 8, kCopyWarp = 8, kMmaWarp = 9;
// 384 threads are launched with 168 registers each; the softmax warps (N
// exponents and N sums a thread) take what the last group leaves: 256 x 208 +
// 128 x 88 = 384 x 168.
constexpr int kAttendThreads = 384;
constexpr uint32_t kTmemCols = 512;
constexpr int kMetaSlots = 8;
constexpr float kSlack = 2.0f;                         // log2: how far a score may exceed the reference
constexpr float kHead = 1.0f;                          // log2: how far a new reference lies above its score
constexpr float kUnset = -1e30f;                       // stands for the reference of a part without tokens
constexpr float kPUnit = 64.0f;                        // P = 64 y <= 2^(6 + 2) (e4m3 ends at 448)
constexpr int kPShift = -2;                            // log2 of P / (256 y): exponents are those of P / 256
template <int D, int N, bool PAIR>
constexpr int attend_smem() {
  using S = AttendShape<N, PAIR>;
  return 1024 + 2 * S::kPBytes + 2 * S::kRows * D + 2 * S::kStages * kTile * D + (D == 64 ? kTile * D : 0);
}

struct TileMeta {
  alignas(16) uint8_t mask[kTile];  // the tile's part of the key mask, when there is one
  // Per page of the tile: scale log2 e s_k, log2(s_v / 4), 4 / s_v, and the largest
  // log2(s_v / 4) of the tile's pages (one store: with pages of 16 tokens the copy
  // warp's instructions set the pace).
  float4 page[8];
  uint32_t pages;                   // bits of the pages that exist, and 16 bits up of those without values
  int32_t left;                     // tokens of the sequence in the tile
};

__device__ __forceinline__ bool tile_visible(const TileMeta& m, int key, int page, bool masked) {
  return key < m.left && ((m.pages >> page) & 1u) && (!masked || m.mask[key] != 0);
}

// What the roles share about a tile is in its meta slot; a slot is reused
// after kMetaSlots tiles, and the producer is never that far ahead of a role
// that reads it (kStages tiles ahead of the products, those two jobs ahead of
// the softmax).
template <int N, bool PAIR>
struct AttendShared {
  uint64_t kfull[5], kempty[5], vfull[5], vempty[5];
  uint64_t mfull[kMetaSlots];
  uint64_t sfull[2], sempty[2], pfull[2], pvdone[2];
  uint64_t qfull;
  TileMeta meta[kMetaSlots];
  alignas(16) float f[AttendShape<N, PAIR>::kRows];    // query scales
  alignas(16) float nm[2][N];                          // per group: minus the references,
  alignas(16) float fac_o[2][N];                       // the factors of a rise,
  alignas(16) float fac_l[2][N];
  alignas(16) float delta[2][N];
  alignas(16) float red[2][4][N];                      // maxima or sums per warp
  alignas(16) float fin[2][N];                         // what an accumulator's column is multiplied with at the end
  alignas(16) int32_t row[AttendShape<N, PAIR>::kRows];    // output rows, -1 where a column has none
  uint32_t w0, w1, off0;
  int32_t b0;
  uint32_t tmem;
  int32_t abort;
};

// log2(s / 4) of a value scale s, and 4 / s as the sums use it: exact for powers
// of two, else a page's tokens count by a factor within 2^-18 of s, which the two
// agree on.  A page of no values (2^-100, the least that an append gives) returns
// true and counts by 2^-64, with zeros: its tokens' share of the sums, which may be
// all of them, must stay within fp32's range next to ordinary pages'.
__device__ __forceinline__ bool value_unit(float s, float& lv, float& iv) {
  const bool nothing = !(s > 0x1p-100f);
  const uint32_t b = __float_as_uint(nothing ? 0x1p-64f : fminf(s, 0x1p+120f));
  const int e = static_cast<int>(b >> 23) - 127 + kPShift;
  const float whole = static_cast<float>(e), f = __uint_as_float((b & 0x7FFFFFu) | 0x3F800000u);
  lv = f == 1.0f ? whole : whole + __log2f(f);
  iv = __uint_as_float(static_cast<uint32_t>(127 - e) << 23) * (f == 1.0f ? 1.0f : ex2_approx(whole - lv));
  return nothing;
}

// The copy warp of a CTA: the tiles of its range, K (and V) through the rings
// and what is known of each tile into its meta slot.
template <int D, int ST, bool WITH_V, class SH, class WAIT>
__device__ __forceinline__ void copy_role(const AttendParams& p, SH& sh, const Cursor& cur, uint32_t k_s, uint32_t v_s,
                                          const WAIT& wait) {
  constexpr int kTileBytes = kTile * D, MS = static_cast<int>(sizeof(sh.meta) / sizeof(TileMeta));
  const int lane = threadIdx.x & 31;
  const int ps = p.c.page_size, ppt = kTile / ps;      // pages per tile
  const uint32_t w0 = sh.w0;
  volatile int32_t* abort_flag = &sh.abort;
  uint32_t g = 0;                                      // tiles passed
  // A batch is up to 32 pages of one segment, one to a lane: ids are fetched
  // two batches ahead and scales one batch ahead of the copies that use
  // them, since each can cost a DRAM latency (tile by tile, that latency was
  // the time per tile).
  const int batch_tiles = 32 / ppt;
  struct Batch {
    int32_t b, h, len, t0, n, id;   // batch row, head, length, first tile, tiles; this lane's page id, or -1
  };
  struct Page {
    int32_t at;                     // page heads + head, or -1
    float ks, vs;
  };
  Cursor look = cur;
  Segment ahead;
  bool more = next_segment(p, look, w0, ahead);
  int at_tile = more ? ahead.t0 : 0;
  auto fetch = [&](Batch& t) {                       // the next batch's page ids
    t.n = 0;
    t.id = -1;
    if (!more) return;
    t.b = ahead.b;
    t.h = ahead.h;
    t.len = ahead.len;
    t.t0 = at_tile;
    t.n = min(batch_tiles, ahead.t1 - at_tile);
    const int64_t col = static_cast<int64_t>(at_tile) * ppt + lane;
    if (lane < t.n * ppt && col * ps < t.len) t.id = p.table[static_cast<int64_t>(ahead.b) * p.width + col];
    at_tile += t.n;
    if (at_tile == ahead.t1) {
      more = next_segment(p, look, w0, ahead);
      if (more) at_tile = ahead.t0;
    }
  };
  auto scales = [&](const Batch& t) {
    Page pg{t.id >= 0 && t.id < p.c.pages ? t.id * p.c.heads + t.h : -1, 0.0f, 0.0f};
    if (pg.at >= 0) {
      pg.ks = p.c.k_scale[pg.at];
      if (WITH_V) pg.vs = p.c.v_scale[pg.at];
    }
    return pg;
  };
  Batch now, next;
  fetch(now);
  fetch(next);
  Page page = scales(now);
  while (now.n > 0) {
    Batch later;
    const Page next_page = scales(next);
    fetch(later);
    const unsigned named = __ballot_sync(0xFFFFFFFFu, page.at >= 0);
    float lv = 0.0f, iv = 0.0f, top = kUnset;
    unsigned nothing = 0;
    if (WITH_V) {                                      // (here, a batch after the scales were asked for)
      const bool none = value_unit(page.vs, lv, iv) && page.at >= 0;
      nothing = __ballot_sync(0xFFFFFFFFu, none);
      if (page.at >= 0) top = lv;
      for (int o = 1; o < ppt; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));   // of the tile
    }
    for (int i = 0; i < now.n; ++i, ++g) {
      const uint32_t st = g % ST, ms = g % MS;
      wait(sh.kempty[st], ((g / ST) & 1u) ^ 1u, kFaultEmptyWait);
      if (WITH_V) wait(sh.vempty[st], ((g / ST) & 1u) ^ 1u, kFaultEmptyWait);
      const int slot = lane - i * ppt;               // of this lane's page in the tile
      const bool mine = slot >= 0 && slot < ppt;
      const unsigned tile_pages = 0xFFFFFFFFu >> (32 - ppt), pages = (named >> (i * ppt)) & tile_pages;
      if (__any_sync(0xFFFFFFFFu, *abort_flag != 0)) continue;   // (the whole warp or none)
      if (lane == 0) {
        const uint32_t bytes = static_cast<uint32_t>(__popc(pages) * ps * D);
        mbar_arrive_expect_tx(smem_addr(&sh.kfull[st]), bytes);
        if (WITH_V) mbar_arrive_expect_tx(smem_addr(&sh.vfull[st]), bytes);
      }
      __syncwarp();
      if (mine && page.at >= 0) {
        const int y = page.at * ps;
        const uint32_t to = static_cast<uint32_t>(slot * ps * D);
        at_tma_load(k_s + st * kTileBytes + to, &p.tm_k, 0, y, smem_addr(&sh.kfull[st]));
        if (WITH_V) at_tma_load(v_s + st * kTileBytes + to, &p.tm_v, 0, y, smem_addr(&sh.vfull[st]));
      }
      TileMeta& m = sh.meta[ms];
      const int64_t j0 = static_cast<int64_t>(now.t0 + i) * kTile;
      if (mine) m.page[slot] = make_float4(page.ks * p.scale2, lv, iv, top);
      if (lane == 0) {
        m.pages = pages | ((nothing >> (i * ppt)) & tile_pages) << 16;
        m.left = min(kTile, now.len - static_cast<int32_t>(j0));
      }
      __syncwarp();
      if (lane == 0) {
        if (p.mask) {
          const uint32_t mb = static_cast<uint32_t>(min(static_cast<int64_t>(kTile), p.cap - j0));
          mbar_arrive_expect_tx(smem_addr(&sh.mfull[ms]), mb);
          bulk_copy_g2s(smem_addr(m.mask), p.mask + static_cast<int64_t>(now.b) * p.mask_stride + j0, mb,
                        smem_addr(&sh.mfull[ms]));
        } else {
          mbar_arrive(smem_addr(&sh.mfull[ms]));
        }
      }
      __syncwarp();
    }
    now = next;
    next = later;
    page = next_page;
  }
  // On an abort the copies in flight are waited for (bounded) before the CTA ends.
  if (*abort_flag && lane == 0) {
    for (uint32_t i = g > ST ? g - ST : 0; i < g; ++i) {
      (void)mbar_wait_bounded(smem_addr(&sh.kfull[i % ST]), (i / ST) & 1u);
      if (WITH_V) (void)mbar_wait_bounded(smem_addr(&sh.vfull[i % ST]), (i / ST) & 1u);
      (void)mbar_wait_bounded(smem_addr(&sh.mfull[i % MS]), (i / MS) & 1u);
    }
  }
}

// One row's 8 elements (of the row's D, spread over the D / 8 consecutive
// lanes): the row's power-of-two scale and the elements' two e4m3 parts.
template <int D>
__device__ __forceinline__ float split_query(const uint4& x, uint32_t (&hi)[2], uint32_t (&lo)[2]) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  uint32_t top = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t u0 = w[j] & 0x7FFFu, u1 = (w[j] >> 16) & 0x7FFFu;
    top = max(top, u0 < 0x7F80u ? u0 : 0u);
    top = max(top, u1 < 0x7F80u ? u1 : 0u);
  }
#pragma unroll
  for (int o = D / 16; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
  const float s = block_scale(__uint_as_float(top << 16));
  // (the largest bf16 needs 2^120: its inverse is still normal)
  const float inv = __uint_as_float(0x7F000000u - __float_as_uint(s));
  hi[0] = hi[1] = lo[0] = lo[1] = 0u;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float a = bf16lo(w[j]) * inv, b = bf16hi(w[j]) * inv;
    if (!(fabsf(a) <= 448.0f)) a = __int_as_float(0x7FFFFFFF);   // infinities and NaN: the row's results are NaN
    if (!(fabsf(b) <= 448.0f)) b = __int_as_float(0x7FFFFFFF);
    const uint32_t h = e4m3x2(a, b);
    float ha, hb;
    f16x2_to_f32(e4m3x2_to_f16x2(h), ha, hb);
    const uint32_t l = e4m3x2(a - ha, b - hb);
    hi[j >> 1] |= h << (16 * (j & 1));
    lo[j >> 1] |= l << (16 * (j & 1));
  }
  return s;
}

// Where elements 8 e .. 8 e + 7 of row r lie in a swizzled K-major tile of D-byte rows.
template <int D>
__device__ __forceinline__ uint32_t query_offset(int r, int e) {
  const int chunk = e >> 1;
  return static_cast<uint32_t>(r * D + ((D == 128 ? chunk ^ (r & 7) : chunk ^ ((r >> 1) & 3)) << 4) + (e & 1) * 8);
}

// One warp: the batch row that holds unit w (p.B when there is none), and the
// units before that row; hr = heads times row tiles.
__device__ __forceinline__ void find_row(const AttendParams& p, uint32_t hr, uint32_t w, int32_t& b, uint32_t& before) {
  const int lane = threadIdx.x & 31;
  before = 0;
  b = 0;
  while (b < p.B) {                                    // 32 batch rows at a time
    const uint32_t t = b + lane < p.B ? units_of(p, b + lane) * hr : 0;
    uint32_t inc = t;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t u = __shfl_up_sync(0xFFFFFFFFu, inc, o);
      if (lane >= o) inc += u;
    }
    const unsigned in = __ballot_sync(0xFFFFFFFFu, b + lane < p.B && before + inc > w);
    if (in != 0u) {
      const int l = __ffs(in) - 1;
      before += __shfl_sync(0xFFFFFFFFu, inc - t, l);
      b += l;
      return;
    }
    before += __shfl_sync(0xFFFFFFFFu, inc, 31);
    b += 32;
  }
}

// One warp: the CTA's range and where it begins, into sh.
template <class SH>
__device__ __forceinline__ void plan_range(const AttendParams& p, SH& sh) {
  const uint32_t hr = static_cast<uint32_t>(p.c.heads * p.row_tiles);
  const Split split(all_units(p) * hr, gridDim.x);
  const uint32_t w0 = split.begin(blockIdx.x), w1 = split.begin(blockIdx.x + 1);
  uint32_t before;
  int32_t b;
  find_row(p, hr, w0, b, before);
  if ((threadIdx.x & 31) == 0) {
    sh.w0 = w0;
    sh.w1 = w1;
    sh.b0 = b;
    sh.off0 = w0 - before;
  }
}

template <int D, int N, bool PAIR>
__global__ void __launch_bounds__(kAttendThreads, 1) attend_kernel(const __grid_constant__ AttendParams p) {
  using S = AttendShape<N, PAIR>;
  constexpr int ST = S::kStages;
  constexpr int kTileBytes = kTile * D;
  constexpr uint32_t kSwz = D == 128 ? 2u : 4u;        // K, V and queries: rows of D bytes, swizzled over D bytes
  extern __shared__ __align__(1024) uint8_t at_smem[];
  __shared__ AttendShared<N, PAIR> sh;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t base = (smem_addr(at_smem) + 1023u) & ~1023u;
  const uint32_t p_s = base, q_s = p_s + 2 * S::kPBytes, k_s = q_s + 2 * S::kRows * D;
  const uint32_t v_s = k_s + ST * kTileBytes, zero_s = v_s + ST * kTileBytes;
  volatile int32_t* abort_flag = &sh.abort;

  if (threadIdx.x == 0) {
    for (int i = 0; i < ST; ++i) {
      mbar_init(smem_addr(&sh.kfull[i]), 1);
      mbar_init(smem_addr(&sh.kempty[i]), 1);
      mbar_init(smem_addr(&sh.vfull[i]), 1);
      mbar_init(smem_addr(&sh.vempty[i]), 1);
    }
    for (int i = 0; i < kMetaSlots; ++i) mbar_init(smem_addr(&sh.mfull[i]), 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_addr(&sh.sfull[i]), 1);
      mbar_init(smem_addr(&sh.sempty[i]), 4);
      mbar_init(smem_addr(&sh.pfull[i]), 4);
      mbar_init(smem_addr(&sh.pvdone[i]), 1);
    }
    mbar_init(smem_addr(&sh.qfull), kSoftWarps);
    sh.abort = 0;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&sh.tmem)),
                 "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  // In this order: what the launches behind this one (the join and the weights)
  // read before their own wait, the call's inputs, is then complete.
  pdl_wait();
  pdl_launch_dependents();
  if (warp == 0) plan_range(p, sh);
  if (D == 64)       // the upper 64 rows of V^T: zeros
    for (int i = threadIdx.x; i < kTileBytes / 16; i += kAttendThreads)
      sts128(zero_s + static_cast<uint32_t>(i) * 16u, 0u, 0u, 0u, 0u);
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

  if (warp >= kSoftWarps) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    if (warp == kCopyWarp) {
      copy_role<D, ST, true>(p, sh, cur, k_s, v_s, wait);
    } else if (warp == kMmaWarp) {
      constexpr uint32_t kPerTile = PAIR ? 2 : 1;        // jobs of a tile
      constexpr uint32_t kHiK = at_desc_hi(8 * D, kSwz), kHiP = at_desc_hi(8 * N, N == 64 ? 4u : 6u);
      const uint32_t lead = elect_one();
      const uint32_t kd = at_desc_lo(k_s, 16), qd = at_desc_lo(q_s, 16), pd = at_desc_lo(p_s, kTile * N);
      const uint32_t tm = __shfl_sync(0xFFFFFFFFu, tmem, 0);
      // Stage and phase of the next tile whose scores, and whose output product, are issued.
      uint32_t ss = 0, sp = 0, vs = 0, vp = 0;
      uint32_t js = 0, jv = 0;                           // jobs issued of either
      auto scores = [&]() {                              // S^T of job js: K (codes) x (hi, lo)
        const uint32_t grp = js & 1u;
        wait(sh.kfull[ss], sp, kFaultFullWait);
        wait(sh.sempty[grp], ((js >> 1) & 1u) ^ 1u, kFaultEmptyWait);
        __syncwarp();
        const bool last = kPerTile == 1 || grp == 1;
        if (!*abort_flag) {
          at_fence_after();
          const uint32_t k = kd + ss * (kTileBytes >> 4), q = qd + (PAIR ? grp * (2 * N * D >> 4) : 0u);
          const uint32_t d = tm + S::kScore + grp * S::kScoreCols;
          constexpr int kParts = S::kConcat ? 1 : 2;
  #pragma unroll
          for (int i = 0; i < kParts * (D / 32); ++i) {
            const int part = i / (D / 32), kk = i % (D / 32);
            at_mma_f8(lead, d, k + kk * 2, kHiK, q + part * (N * D / 16) + kk * 2, kHiK,
                      at_idesc(S::kScoreCols, false), i != 0 ? 1u : 0u);
          }
          if (last) at_commit(lead, smem_addr(&sh.kempty[ss]));
          at_commit(lead, smem_addr(&sh.sfull[grp]));
        }
        __syncwarp();
        ++js;
        if (last && ++ss == ST) {
          ss = 0;
          sp ^= 1u;
        }
      };
      uint32_t seg = 0;
      while (next_segment(p, cur, sh.w0, sg)) {
        const uint32_t n = __shfl_sync(0xFFFFFFFFu, static_cast<uint32_t>(sg.t1 - sg.t0) * kPerTile, 0);   // its jobs
        wait(sh.qfull, seg & 1u, kFaultFullWait);
        __syncwarp();
        scores();
        if (n > 1) scores();
        for (uint32_t i = 0; i < n; ++i) {
          const uint32_t grp = jv & 1u;
          if (i + 2 < n) scores();                       // (job i + 2's, as soon as job i's scores have been read)
          wait(sh.vfull[vs], vp, kFaultFullWait);
          wait(sh.pfull[grp], (jv >> 1) & 1u, kFaultFullWait);
          __syncwarp();
          const bool last = kPerTile == 1 || grp == 1;
          if (!*abort_flag) {
            at_fence_after();
            const uint32_t vst = v_s + vs * kTileBytes;
            const uint32_t v = at_desc_lo(vst, zero_s - vst), pp = pd + grp * (S::kPBytes >> 4);
            const uint32_t d = tm + S::kAcc + grp * 3 * N;
  #pragma unroll
            for (int kk = 0; kk < kTile / 32; ++kk)
              at_mma_f8(lead, d, v + kk * (32 * D >> 4), kHiK, pp + kk * (32 * N >> 4), kHiP, at_idesc(3 * N, true),
                        kk != 0 || i >= 2 ? 1u : 0u);
            if (last) at_commit(lead, smem_addr(&sh.vempty[vs]));
            at_commit(lead, smem_addr(&sh.pvdone[grp]));
          }
          __syncwarp();
          ++jv;
          if (last && ++vs == ST) {
            vs = 0;
            vp ^= 1u;
          }
        }
        ++seg;
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    // Softmax: warp w (mod 4) of a group has tokens 32 w .. 32 w + 31 of a tile,
    // a thread tokens 32 w + lane / 4 + 8 q, q = 0 .. 3, and the columns 8 j + 2
    // (lane mod 4) + {0, 1}.  What is stored or cleared by token (P's rows, V's)
    // goes by key = 32 w + lane.
    constexpr int J = N / 8;                           // column pairs of a thread
    const int grp = warp >> 2, wq = warp & 3, key = wq * 32 + lane, tid = threadIdx.x & 127;
    const int col = 2 * (lane & 3);
    const uint32_t bar_id = 1u + static_cast<uint32_t>(grp);
    const uint32_t lanes = static_cast<uint32_t>(wq * 32) << 16;
    const int ps_log = __ffs(ps) - 1, page_of = key >> ps_log;   // (page sizes are powers of two)
    const int c0 = PAIR ? grp * N : 0;                 // the group's first column
    float* nm = sh.nm[grp];
    const uint32_t p_row = p_s + static_cast<uint32_t>(grp) * S::kPBytes + static_cast<uint32_t>(key) * N;
    const int swz = N == 64 ? (key >> 1) & 3 : (key >> 2) & 1;
    const uint32_t s_t = tmem + lanes + S::kScore + static_cast<uint32_t>(grp) * S::kScoreCols;
    const uint32_t o_t = tmem + lanes + S::kAcc + static_cast<uint32_t>(grp) * 3 * N;
    constexpr int kPer = D / 8;                        // threads that load one row of the queries
    constexpr int kStep = kSoftWarps * 32 / kPer;      // rows loaded at a time
    constexpr int kLoads = S::kRows / kStep;
    static_assert(S::kRows % kStep == 0 && N % kStep == 0, "");
    const int step_l = kStep / p.G, step_g = kStep % p.G;
    const int r0 = threadIdx.x / kPer, e = threadIdx.x % kPer;
    uint4 xq[kLoads];
    int32_t at_row[kLoads];
    // This thread's part of a segment's rows.  With 32 columns the next segment's
    // are fetched before this one's sums and epilogue (8 x 2306 tokens, 32 rows of
    // 32 heads: 39.4 us, 40.7 without); with 64 the registers do not reach (107
    // us, 87.4 without, for 224 rows).
    constexpr bool kAhead = N == 32;
    auto fetch_rows = [&](const Segment& s) {
      const int row0 = s.rt * p.tile_rows, nrows = min(p.tile_rows, p.rows - row0);
      // row -> (query l, head of the group), stepped by kStep columns at a time
      int l = (row0 + r0) / p.G, gq = (row0 + r0) % p.G;
      int lw = PAIR ? (row0 + p.half + r0) / p.G : 0, gw = PAIR ? (row0 + p.half + r0) % p.G : 0;
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const int r = r0 + i * kStep;                  // column; its row:
        const int in = PAIR && r >= N ? r - N : r, rr = PAIR && r >= N ? p.half + in : in;
        xq[i] = make_uint4(0u, 0u, 0u, 0u);
        at_row[i] = -1;
        if (PAIR && i == N / kStep) {
          l = lw;
          gq = gw;
        }
        if (rr < nrows && (!PAIR || in < p.half)) {
          const int hq = s.h * p.G + gq;
          xq[i] = *reinterpret_cast<const uint4*>(p.q + s.b * p.qb + l * p.ql + hq * p.qh + e * 16);
          at_row[i] = static_cast<int32_t>((s.b * p.L + l) * p.Hq + hq);
        }
        l += step_l;
        gq += step_g;
        if (gq >= p.G) {
          gq -= p.G;
          ++l;
        }
      }
    };
    Segment ahead;
    bool more = next_segment(p, cur, sh.w0, ahead);
    if (kAhead && more) fetch_rows(ahead);
    while (more) {
      sg = ahead;
      if (!kAhead) fetch_rows(sg);
      // The queries: one power-of-two scale per row and two e4m3 parts.
      // Columns of this group that hold rows, in 16s:
      const int nrows = min(p.tile_rows, p.rows - sg.rt * p.tile_rows);
      const int mine = PAIR ? min(p.half, nrows - grp * p.half) : nrows;
      const int ncols = (mine + 15) & ~15;
      named_sync(3, kSoftWarps * 32);                  // the previous segment's rows and references are no longer read
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const int r = r0 + i * kStep;
        uint32_t hi[2], lo[2];
        const float s = split_query<D>(xq[i], hi, lo);
        const int in = PAIR ? r % N : r;
        const uint32_t at = q_s + static_cast<uint32_t>((PAIR ? r / N : 0) * 2 * N * D) + query_offset<D>(in, e);
        sts64(at, hi[0], hi[1]);
        sts64(at + N * D, lo[0], lo[1]);
        if (e == 0) {
          sh.f[r] = s;
          sh.row[place(r)] = at_row[i];
        }
      }
      if (tid < N) nm[tid] = 0.0f;
      at_fence_async();
      named_sync(3, kSoftWarps * 32);
      if (lane == 0) mbar_arrive(smem_addr(&sh.qfull));

      // Per column pair: the queries' scales, minus the references, and this
      // thread's share of the sums.
      uint64_t f2[J], nm2[J], l2[J];
#pragma unroll
      for (int j = 0; j < J; ++j) {
        f2[j] = *reinterpret_cast<const uint64_t*>(&sh.f[c0 + 8 * j + col]);
        nm2[j] = l2[j] = 0;
      }
      bool begun = false, seen = false;                // the accumulator holds earlier tiles; the references a score
      for (int ti = sg.t0; ti < sg.t1; ++ti, ++g) {
        if (!PAIR && (g & 1u) != static_cast<uint32_t>(grp)) continue;
        const uint32_t nth = PAIR ? g : g >> 1;        // this group's job number
        wait(sh.mfull[g % kMetaSlots], (g / kMetaSlots) & 1u, kFaultFullWait);
        __syncwarp();
        const TileMeta& m = sh.meta[g % kMetaSlots];
        const bool visible = tile_visible(m, key, page_of, p.mask != nullptr);
        const unsigned seen_keys = __ballot_sync(0xFFFFFFFFu, visible);
        // The four tokens' scales (8 consecutive tokens share a page).
        float ck[4], lv[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int page = (wq * 32 + 8 * q) >> ps_log;
          ck[q] = m.page[page].x;
          lv[q] = m.page[page].y;
        }
        const bool nothing = (m.pages >> (16 + page_of)) & 1u;
        if (!visible || nothing) {
          // Codes of tokens that are not visible (any bytes, NaN among them)
          // would meet probabilities of 0: they become zeros.  So do those of
          // pages without values, but NaN.
          wait(sh.vfull[g % ST], (g / ST) & 1u, kFaultFullWait);
          const uint32_t vrow = v_s + (g % ST) * kTileBytes + static_cast<uint32_t>(key) * D;
          if (!visible) {
#pragma unroll
            for (int i = 0; i < D / 16; ++i) sts128(vrow + i * 16, 0u, 0u, 0u, 0u);
          } else {
#pragma unroll 1
            for (int i = 0; i < D / 4; ++i) {
              uint32_t c;
              asm volatile("ld.shared.u32 %0, [%1];" : "=r"(c) : "r"(vrow + i * 4) : "memory");
              c = __vcmpeq4(c & 0x7F7F7F7Fu, 0x7F7F7F7Fu) & c;
              asm volatile("st.shared.u32 [%0], %1;" ::"r"(vrow + i * 4), "r"(c) : "memory");
            }
          }
        }
        __syncwarp();
        if (!seen) {
          // Until a row has a reference of its own: the tile's largest value scale, so
          // that no exponent is rounded for what the reference will take away.
          const float first = -m.page[0].w;
#pragma unroll
          for (int j = 0; j < J; ++j) nm2[j] = pack2(first, first);
          if (tid < N) nm[tid] = first;
        }
        wait(sh.sfull[grp], nth & 1u, kFaultFullWait);
        __syncwarp();
        at_fence_after();
        // Exponents x[q][j] = log2(P / 256) of token q, column pair j; columns past
        // the rows are not looked at (J is cut to what the rows need).
        uint64_t x[4][J];
        {
          uint32_t r[2][N / 2];                        // of tokens 0 .. 15 and 16 .. 31
          if constexpr (S::kConcat) {
            uint32_t lo[2][N / 2];
            at_frag32x4(s_t, s_t + (16u << 16), s_t + N, s_t + N + (16u << 16), r[0], r[1], lo[0], lo[1]);
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
              for (int i = 0; i < N / 2; ++i)
                r[h][i] = __float_as_uint(__uint_as_float(r[h][i]) + __uint_as_float(lo[h][i]));
          } else {
            at_frag64x2(s_t, s_t + (16u << 16), r[0], r[1]);
          }
#pragma unroll
          for (int j = 0; j < J; ++j) {
            if (j % 2 == 0 && 8 * j >= ncols) break;   // (uniform; ncols is a multiple of 16)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const uint32_t* v = &r[q >> 1][4 * j + 2 * (q & 1)];
              // (reference and scale first: they may both be large and next to equal)
              x[q][j] = fma2(at_mul2(pack2(__uint_as_float(v[0]), __uint_as_float(v[1])), pack2(ck[q], ck[q])), f2[j],
                             add2(nm2[j], pack2(lv[q], lv[q])));
            }
          }
        }
        if (seen_keys != 0xFFFFFFFFu) {                // (uniform)
#pragma unroll
          for (int q = 0; q < 4; ++q)
            if (!((seen_keys >> (8 * q + (lane >> 2))) & 1u))
#pragma unroll
              for (int j = 0; j < J; ++j) x[q][j] = pack2(-kInf, -kInf);
        }
        float over = -kInf;
#pragma unroll
        for (int j = 0; j < J; ++j) {
          if (j % 2 == 0 && 8 * j >= ncols) break;
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            float a, b;
            unpack2(x[q][j], a, b);
            over = fmaxf(fmaxf(over, a), b);
          }
        }
        const bool raise = over > kSlack + kPShift || (!seen && seen_keys != 0u);
        if (group_any(bar_id, raise)) {                // uniform over the group
          // New references: the largest y of each column so far, and a bit more
          // (one then has to exceed it eightfold to move it again).
#pragma unroll
          for (int j = 0; j < J; ++j) {
            if (j % 2 == 0 && 8 * j >= ncols) break;
            float ta = -kInf, tb = -kInf;              // (NaN does not set a reference)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              float a, b;
              unpack2(x[q][j], a, b);
              ta = fmaxf(ta, a);
              tb = fmaxf(tb, b);
            }
            ta = over_tokens<true>(ta);
            tb = over_tokens<true>(tb);
            if (lane < 4) *reinterpret_cast<uint64_t*>(&sh.red[grp][wq][8 * j + col]) = pack2(ta, tb);
          }
          named_sync(bar_id, 128);
          if (tid < ncols) {
            const float top = fmaxf(fmaxf(sh.red[grp][0][tid], sh.red[grp][1][tid]),
                                    fmaxf(sh.red[grp][2][tid], sh.red[grp][3][tid])) - kPShift;   // above the old reference
            const float up = top > 0.0f || (!seen && top > -kInf) ? top + kHead : 0.0f;
            const float was = nm[tid], now = was - up, delta = now - was;   // (-up, as the reference is rounded)
            nm[tid] = now;
            sh.delta[grp][tid] = delta;
            const float d = ex2_approx(delta);
            sh.fac_l[grp][tid] = d;
            // (before any score the accumulator is all zeros, and d may be infinite)
            sh.fac_o[grp][place(tid)] = seen ? d : 0.0f;
          }
          named_sync(bar_id, 128);
#pragma unroll
          for (int j = 0; j < J; ++j) {
            if (j % 2 == 0 && 8 * j >= ncols) break;
            const uint64_t delta = *reinterpret_cast<const uint64_t*>(&sh.delta[grp][8 * j + col]);
            nm2[j] = *reinterpret_cast<const uint64_t*>(&nm[8 * j + col]);
            if (seen) l2[j] = at_mul2(l2[j], *reinterpret_cast<const uint64_t*>(&sh.fac_l[grp][8 * j + col]));
#pragma unroll
            for (int q = 0; q < 4; ++q) x[q][j] = add2(x[q][j], delta);
          }
          seen = true;
          if (begun) {
            wait(sh.pvdone[grp], (nth - 1) & 1u, kFaultFullWait);
            __syncwarp();
            at_fence_after();
#pragma unroll 1
            for (int c = 0; c < ncols; c += 16) {
#pragma unroll
              for (int part = 0; part < 3; ++part) {
                uint32_t r[16];
                at_ld16(o_t + part * N + c, r);
#pragma unroll
                for (int i = 0; i < 16; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) * sh.fac_o[grp][c + i]);
                at_st16(o_t + part * N + c, r);
              }
            }
            asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
            at_fence_before();
          }
          // (the next rise writes what is read here only after every warp's vote for it)
        }
        at_fence_before();                             // the scores have been read
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(&sh.sempty[grp]));
        // P: summed in fp32, in three e4m3 parts for the product.
        float iv[4];                                   // (read here: registers are short above)
#pragma unroll
        for (int q = 0; q < 4; ++q) iv[q] = m.page[(wq * 32 + 8 * q) >> ps_log].z;
        if (nth >= 1) wait(sh.pvdone[grp], (nth - 1) & 1u, kFaultEmptyWait);   // the product that read this buffer last
        __syncwarp();
#pragma unroll
        for (int jj = 0; jj < J / 2; ++jj) {           // 16 columns
          if (16 * jj >= ncols) break;
          uint32_t o[3][4];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            uint32_t h[2];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              const int j = 2 * jj + u;
              float a, b;
              unpack2(x[q][j], a, b);
              a = ex2_approx(a);
              b = ex2_approx(b);
              l2[j] = fma2(pack2(a, b), pack2(iv[q], iv[q]), l2[j]);
              h[u] = f16x2(a, b);
            }
            o[0][q] = part_codes(h[0], h[1]);
            h[0] = part_rest16(h[0]);
            h[1] = part_rest16(h[1]);
            o[1][q] = part_codes(h[0], h[1]);
            o[2][q] = part_codes(part_rest16(h[0]), part_rest16(h[1]));
          }
          const uint32_t at = p_row + static_cast<uint32_t>(jj ^ swz) * 16u;
#pragma unroll
          for (int k = 0; k < 3; ++k) stmatrix4(at + k * (kTile * N), o[k][0], o[k][1], o[k][2], o[k][3]);
        }
        begun = true;
        at_fence_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(&sh.pfull[grp]));
      }

      if (kAhead) {
        more = next_segment(p, cur, sh.w0, ahead);
        if (more) fetch_rows(ahead);
      }

      // The segment's sums over its tokens, then its rows.
#pragma unroll
      for (int j = 0; j < J; ++j) {
        float a, b;
        unpack2(l2[j], a, b);
        a = over_tokens<false>(a);
        b = over_tokens<false>(b);
        if (lane < 4) *reinterpret_cast<uint64_t*>(&sh.red[grp][wq][8 * j + col]) = pack2(a, b);
      }
      named_sync(3, kSoftWarps * 32);
      const bool whole = sg.t0 == 0 && sg.t1 == sg.T;
      const int64_t slot = 2 * static_cast<int64_t>(blockIdx.x) + (sg.starts_range ? 0 : 1);
      // Taking turns: the group of the segment's first tile has a part of every
      // row, the other one too when there are two tiles (else its accumulator
      // holds nothing).
      const bool both = !PAIR && sg.t1 - sg.t0 >= 2;
      const int first = PAIR ? 0 : static_cast<int>((g - static_cast<uint32_t>(sg.t1 - sg.t0)) & 1u);
      for (int n = threadIdx.x; n < S::kRows; n += kSoftWarps * 32) {
        const int at = place(n);
        const int32_t row = sh.row[at];
        if (row < 0) continue;
        const int a = PAIR ? n / N : first, c = PAIR ? n % N : n;
        float m = -sh.nm[a][c];
        float l = (sh.red[a][0][c] + sh.red[a][1][c]) + (sh.red[a][2][c] + sh.red[a][3][c]);
        if (l == 0.0f) m = kUnset;                     // (no token: its reference says nothing)
        float fa = 1.0f / kPUnit, fb = 0.0f;
        if (both) {
          const int o = first ^ 1;
          const float lo = (sh.red[o][0][c] + sh.red[o][1][c]) + (sh.red[o][2][c] + sh.red[o][3][c]);
          const float mo = lo == 0.0f ? kUnset : -sh.nm[o][c], top = fmaxf(m, mo);
          const float ea = ex2_approx(m - top), eb = ex2_approx(mo - top);
          l = l * ea + lo * eb;
          fa *= ea;
          fb = 1.0f / kPUnit * eb;
          m = top;
        }
        if (whole) {
          const float inv = l == 0.0f ? 0.0f : 1.0f / l;   // (a NaN sum gives NaN)
          fa *= inv;
          fb *= inv;
          p.lse[row] = lse_of(m, l);
        } else {
          p.part_ml[(slot * S::kRows + at) * 2] = m;
          p.part_ml[(slot * S::kRows + at) * 2 + 1] = l;
        }
        sh.fin[a][place(c)] = fa;
        if (both) sh.fin[first ^ 1][place(c)] = fb;
      }
      // The last product of either group.
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const uint32_t back = PAIR ? 1u : 1u + static_cast<uint32_t>(k);
        if (!PAIR && k == 1 && !both) break;
        const uint32_t j = PAIR ? 2 * (g - 1) + static_cast<uint32_t>(k) : g - back;
        wait(sh.pvdone[j & 1u], (j >> 1) & 1u, kFaultFullWait);
      }
      __syncwarp();
      at_fence_after();
      named_sync(3, kSoftWarps * 32);
      const int d = key;                               // an accumulator's lane is a dimension
      // Taking turns, each group writes half of the columns from both accumulators.
      const int per = PAIR ? N : N / 2;
      const int ca = PAIR ? 0 : grp * per;
#pragma unroll 1
      for (int c = ca; c < ca + per && c < ncols; c += 8) {
        float o[8];
        const int a0 = PAIR ? grp : first;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          if (k == 1 && !both) break;
          const int a = k == 0 ? a0 : a0 ^ 1;
          uint32_t r[24];
          const uint32_t t = tmem + lanes + S::kAcc + static_cast<uint32_t>(a) * 3 * N + c;
          at_ld3(t, t + N, t + 2 * N, r);
          const float4 f0 = *reinterpret_cast<const float4*>(&sh.fin[a][c]);
          const float4 f1 = *reinterpret_cast<const float4*>(&sh.fin[a][c + 4]);
          const float f[8] = {f0.x, f0.y, f0.z, f0.w, f1.x, f1.y, f1.z, f1.w};
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float y = fmaf(fmaf(__uint_as_float(r[16 + i]), 1.0f / 16, __uint_as_float(r[8 + i])), 1.0f / 16,
                                 __uint_as_float(r[i]));
            o[i] = k == 0 ? y * f[i] : fmaf(y, f[i], o[i]);
          }
        }
        if (d >= D) continue;                          // (whole warps)
        const int n = c0 + c;
        const int4 r0 = *reinterpret_cast<const int4*>(&sh.row[n]), r1 = *reinterpret_cast<const int4*>(&sh.row[n + 4]);
        const int32_t rows8[8] = {r0.x, r0.y, r0.z, r0.w, r1.x, r1.y, r1.z, r1.w};
        if (whole) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            uint16_t u;
            asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(u) : "f"(o[i]));
            if (rows8[i] >= 0) p.out[static_cast<int64_t>(rows8[i]) * D + d] = u;
          }
        } else {
          float* part = p.part_o + (slot * S::kRows + n) * D + d;
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (rows8[i] >= 0) part[i * D] = o[i];
        }
      }
      at_fence_before();
      if (!kAhead) more = next_segment(p, cur, sh.w0, ahead);
    }
  }
  at_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    at_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
  }
}

// ---------------------------------------------------------------------------
// the weights
// ---------------------------------------------------------------------------
constexpr int kWeightCols = 64;        // rows (columns of a product) of a job
constexpr int kWeightRows = 256;       // rows of a launch: what the queries' shared memory holds
constexpr int kWeightStages = 8;       // of the K ring
constexpr int kWeightGroups = 4;
constexpr int kWeightSoft = 4 * kWeightGroups, kWeightCopyWarp = kWeightSoft, kWeightMmaWarp = kWeightSoft + 1;
constexpr int kWeightThreads = (kWeightSoft + 2) * 32;
constexpr int kWeightBufs = 2;         // score buffers of a group
// While a group works on tile t the products get to tile t + 7 at most (t + 8
// needs its buffer) and the copies 8 tiles further: a tile's meta slot is free
// again after 16.
constexpr int kWeightMeta = 16;

constexpr int weights_smem(int dim, int chunks) {
  return 1024 + 2 * chunks * kWeightCols * dim + kWeightStages * kTile * dim;
}

struct WeightShared {
  uint64_t kfull[kWeightStages], kempty[kWeightStages];
  uint64_t mfull[kWeightMeta];
  uint64_t sfull[kWeightGroups * kWeightBufs], sempty[kWeightGroups * kWeightBufs];
  uint64_t qfull;
  TileMeta meta[kWeightMeta];
  alignas(16) float f[kWeightRows], nm[kWeightRows];   // query scales, minus the rows' lse (log2 units)
  uint32_t w0, w1, off0;
  int32_t b0;
  uint32_t tmem;
  int32_t abort;
  uint64_t vfull[1], vempty[1];                        // (not used: there is no V)
};

// w[j] = decay w[j] + sum over the rows of exp(s - lse): S^T as in the
// attention; a token's columns lie with four lanes of one warp, so its sum stays
// there and nothing is added atomically.  Four groups of 4 warps take the tiles
// in turn; a job is one tile and up to 64 rows.
// Bound: the softmax's chain of waits and instructions (50 % of the issue slots),
// since each row's scores are computed once more; K's bytes when rows are few.
// The hi and lo parts add up in one buffer of 64 columns, so a group has two (one
// of 128, both parts in one product: 2.7 us more).  Measured, 224 rows a head, 16
// x 5096 tokens, 4 heads: 42 us.
template <int D>
__global__ void __launch_bounds__(kWeightThreads, 1) attend_weights_kernel(const __grid_constant__ AttendParams p,
                                                                           int32_t first_row, int32_t rows) {
  constexpr int ST = kWeightStages, NC = kWeightCols;
  constexpr int kTileBytes = kTile * D;
  constexpr uint32_t kSwz = D == 128 ? 2u : 4u;
  extern __shared__ __align__(1024) uint8_t at_smem[];
  __shared__ WeightShared sh;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int chunks = (rows + NC - 1) / NC;
  const uint32_t base = (smem_addr(at_smem) + 1023u) & ~1023u;
  const uint32_t k_s = base, q_s = k_s + ST * kTileBytes;
  volatile int32_t* abort_flag = &sh.abort;

  if (threadIdx.x == 0) {
    for (int i = 0; i < ST; ++i) {
      mbar_init(smem_addr(&sh.kfull[i]), 1);
      mbar_init(smem_addr(&sh.kempty[i]), 1);
    }
    for (int i = 0; i < kWeightMeta; ++i) mbar_init(smem_addr(&sh.mfull[i]), 1);
    for (int i = 0; i < kWeightGroups * kWeightBufs; ++i) {
      mbar_init(smem_addr(&sh.sfull[i]), 1);
      mbar_init(smem_addr(&sh.sempty[i]), 4);
    }
    mbar_init(smem_addr(&sh.qfull), kWeightSoft);
    sh.abort = 0;
    fence_mbar_init();
  }
  if (warp == kWeightMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&sh.tmem)),
                 "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  pdl_launch_dependents();
  if (warp == 0) plan_range(p, sh);
  at_fence_before();
  __syncthreads();
  at_fence_after();
  const uint32_t tmem = sh.tmem;

  auto wait = [&](uint64_t& bar, uint32_t parity, int32_t code) {   // as in the attention kernel
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
  if (warp == kWeightCopyWarp) {
    copy_role<D, ST, false>(p, sh, cur, k_s, 0, wait);
  } else if (warp == kWeightMmaWarp) {
    constexpr uint32_t kHiK = at_desc_hi(8 * D, kSwz);
    const uint32_t lead = elect_one();
    const uint32_t kd = at_desc_lo(k_s, 16), qd = at_desc_lo(q_s, 16);
    const uint32_t tm = __shfl_sync(0xFFFFFFFFu, tmem, 0);
    uint32_t seg = 0;
    while (next_segment(p, cur, sh.w0, sg)) {
      const uint32_t n = __shfl_sync(0xFFFFFFFFu, static_cast<uint32_t>(sg.t1 - sg.t0), 0);
      wait(sh.qfull, seg & 1u, kFaultFullWait);
      __syncwarp();
      // Four tiles, one to a group, chunk by chunk: so that all groups have work
      // (tile by tile, a group's buffer held the others up).
      for (uint32_t i = 0; i < n; i += kWeightGroups) {
        const uint32_t tiles = min(static_cast<uint32_t>(kWeightGroups), n - i);
        for (int c = 0; c < chunks; ++c) {
          const uint32_t q = qd + static_cast<uint32_t>(c) * (2 * NC * D >> 4);
          for (uint32_t u = 0; u < tiles; ++u) {
            const uint32_t t = g + u, grp = t % kWeightGroups, st = t % ST;
            const uint32_t j = t / kWeightGroups * static_cast<uint32_t>(chunks) + static_cast<uint32_t>(c);
            const uint32_t buf = grp * kWeightBufs + j % kWeightBufs;
            if (c == 0) wait(sh.kfull[st], (t / ST) & 1u, kFaultFullWait);
            wait(sh.sempty[buf], ((j / kWeightBufs) & 1u) ^ 1u, kFaultEmptyWait);
            __syncwarp();
            if (!*abort_flag) {
              at_fence_after();
              const uint32_t k = kd + st * (kTileBytes >> 4);
#pragma unroll
              for (int i = 0; i < 2 * (D / 32); ++i) {   // hi parts, then lo parts
                const int part = i / (D / 32), kk = i % (D / 32);
                at_mma_f8(lead, tm + buf * NC, k + kk * 2, kHiK, q + part * (NC * D / 16) + kk * 2, kHiK,
                          at_idesc(NC, false), i != 0 ? 1u : 0u);
              }
              if (c == chunks - 1) at_commit(lead, smem_addr(&sh.kempty[st]));
              at_commit(lead, smem_addr(&sh.sfull[buf]));
            }
            __syncwarp();
          }
        }
        g += tiles;
      }
      ++seg;
    }
  } else if (warp < kWeightSoft) {
    const int grp = warp >> 2, wq = warp & 3, ps_log = __ffs(p.c.page_size) - 1;
    const uint32_t lanes = static_cast<uint32_t>(wq * 32) << 16;
    constexpr int kPer = D / 8, kStep = kWeightSoft * 32 / kPer;
    uint32_t jobs = 0;                                 // this group's
    pdl_wait();   // the rows' lse (the copies and the plan, which need the call's inputs only, do not wait: 2 us less)
    while (next_segment(p, cur, sh.w0, sg)) {
      named_sync(5, kWeightSoft * 32);                  // (the previous segment's rows are no longer read)
      const int e = threadIdx.x % kPer;
      constexpr int kBatch = kWeightRows / kStep;      // all rows at once
      {
        const int rb = threadIdx.x / kPer;
        uint4 x[kBatch];
        float nm[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          const int r = rb + i * kStep;
          x[i] = make_uint4(0u, 0u, 0u, 0u);
          nm[i] = -kInf;
          if (r < rows) {
            const int l = (first_row + r) / p.G, hq = sg.h * p.G + (first_row + r) - l * p.G;
            x[i] = *reinterpret_cast<const uint4*>(p.q + sg.b * p.qb + l * p.ql + hq * p.qh + e * 16);
            nm[i] = -p.lse[(sg.b * p.L + l) * p.Hq + hq] * kLog2e;
          }
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          const int r = rb + i * kStep;
          if (r >= chunks * NC) break;                 // (whole warps)
          uint32_t hi[2], lo[2];
          const float s = split_query<D>(x[i], hi, lo);
          const uint32_t at = q_s + static_cast<uint32_t>(r / NC * 2 * NC * D) + query_offset<D>(r % NC, e);
          sts64(at, hi[0], hi[1]);
          sts64(at + NC * D, lo[0], lo[1]);
          if (e == 0) {
            sh.f[r] = s;
            sh.nm[r] = fabsf(nm[i]) < kInf ? nm[i] : -kInf;   // (a row whose lse is not finite adds nothing)
          }
        }
      }
      at_fence_async();
      named_sync(5, kWeightSoft * 32);
      if (lane == 0) mbar_arrive(smem_addr(&sh.qfull));
      for (int ti = sg.t0; ti < sg.t1; ++ti, ++g) {
        if (g % kWeightGroups != static_cast<uint32_t>(grp)) continue;
        // This thread's tokens are 32 wq + lane / 4 + 8 q; it writes the weight of
        // the one with q = lane mod 4.
        const int mine = wq * 32 + 8 * (lane & 3) + (lane >> 2);
        const int64_t at = static_cast<int64_t>(ti) * kTile + mine;
        float* wj = p.weights + (static_cast<int64_t>(sg.b) * p.c.heads + sg.h) * p.cap + at;
        const bool in = at < p.cap;
        const float old = in && p.decay != 0.0f ? *wj : 0.0f;
        wait(sh.mfull[g % kWeightMeta], (g / kWeightMeta) & 1u, kFaultFullWait);
        const TileMeta& m = sh.meta[g % kWeightMeta];
        const bool valid = tile_visible(m, mine, mine >> ps_log, p.mask != nullptr);
        float ck[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) ck[q] = m.page[(wq * 32 + 8 * q) >> ps_log].x;
        uint64_t sum2[4] = {0, 0, 0, 0};
        for (int c = 0; c < chunks; ++c, ++jobs) {
          const uint32_t buf = static_cast<uint32_t>(grp) * kWeightBufs + jobs % kWeightBufs;
          wait(sh.sfull[buf], (jobs / kWeightBufs) & 1u, kFaultFullWait);
          __syncwarp();
          at_fence_after();
          const int cols = min(NC, (rows - c * NC + 15) & ~15);
#pragma unroll
          for (int n = 0; n < NC; n += 32) {
            if (n >= cols) break;                      // (uniform)
            uint64_t f2[4], nm2[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              f2[j] = *reinterpret_cast<const uint64_t*>(&sh.f[c * NC + n + 8 * j + 2 * (lane & 3)]);
              nm2[j] = *reinterpret_cast<const uint64_t*>(&sh.nm[c * NC + n + 8 * j + 2 * (lane & 3)]);
            }
            uint32_t r[2][16];                         // tokens 0 .. 15 and 16 .. 31
            const uint32_t s_t = tmem + lanes + buf * NC + n;
            at_frag32x2(s_t, s_t + (16u << 16), r[0], r[1]);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              if (j == 2 && n + 16 >= cols) break;
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                const uint32_t* y = &r[q >> 1][4 * j + 2 * (q & 1)];
                float a, b;
                unpack2(fma2(at_mul2(pack2(__uint_as_float(y[0]), __uint_as_float(y[1])), pack2(ck[q], ck[q])), f2[j],
                             nm2[j]), a, b);
                // (a row that adds nothing has -inf or NaN here)
                sum2[q] = add2(sum2[q], pack2(ex2_approx(fmaxf(a, -1e30f)), ex2_approx(fmaxf(b, -1e30f))));
              }
            }
          }
          at_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_addr(&sh.sempty[buf]));
        }
        // A token's columns lie with four lanes.
        float sum = 0.0f;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          float a, b;
          unpack2(sum2[q], a, b);
          a += b;
          a += __shfl_xor_sync(0xFFFFFFFFu, a, 1);
          a += __shfl_xor_sync(0xFFFFFFFFu, a, 2);
          if ((lane & 3) == q) sum = a;
        }
        if (in) *wj = fmaf(p.decay, old, valid ? sum : 0.0f);
      }
    }
    // Slots past the sequences' last tiles: decayed, or set to 0.
    const int64_t bh = p.B * p.c.heads;
    for (int64_t i = blockIdx.x; i < bh; i += gridDim.x) {
      float* w = p.weights + i * p.cap;
      for (int64_t j = static_cast<int64_t>(tiles_of(p, i / p.c.heads)) * kTile + threadIdx.x; j < p.cap;
           j += kWeightSoft * 32)
        w[j] = p.decay == 0.0f ? 0.0f : p.decay * w[j];
    }
  }
  at_fence_before();
  __syncthreads();
  if (warp == kWeightMmaWarp) {
    at_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
  }
}

// Joins the parts of the items that several CTAs share, in CTA order (a part's
// reference may differ from the others').  Block (x, y) looks at the boundary
// between CTAs x and x + 1: if an item is cut there for the first time, its
// warps join rows 8 y .. 8 y + 7 of it, one each.  Where the item lies takes some
// 500 instructions, which one warp runs for the block, before the attention ends,
// and two parts' rows are asked for before their factors are known.  (What each
// saved when it was built: the one warp 2.1 of 94.9 us at 224 rows a head, the early
// start 1.1 of 12.4 and the early rows 1.4 of 11.3 at a single token over 1999.)
// Rows a block: 8 x 2306 tokens, 32 rows of 32 heads, 39.4
// us, 41.0 and 44.0 with 16 and 32; 224 rows a head, 16 x 5096 tokens, 87.4, 86.0
// and 84.5; a single token the same.
constexpr int kJoinRows = 8;
template <int D>
__global__ void __launch_bounds__(256) attend_join_kernel(const __grid_constant__ AttendParams p, int N, int columns) {
  constexpr int V = D / 32;                            // dimensions of a lane
  struct PartV {
    float v[V];
  };
  __shared__ uint32_t s_ca, s_cb;
  __shared__ int32_t s_b, s_item, s_late;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  pdl_launch_dependents();
  if (warp == 0) {
    const uint32_t hr = static_cast<uint32_t>(p.c.heads * p.row_tiles);
    const uint32_t total = all_units(p) * hr;
    const Split split(total, static_cast<uint32_t>(p.ctas));
    const uint32_t w = split.begin(blockIdx.x + 1);
    uint32_t ca = 0, cb = 0, before, item = 0, i0 = 0;
    int32_t b = 0;
    if (w < total) {
      find_row(p, hr, w, b, before);
      const uint32_t units = units_of(p, b);
      item = (w - before) / units;
      i0 = before + item * units;                      // the item's units: [i0, i0 + units)
      ca = split.owner(i0 + p.seg_cost);               // its first tile's CTA and its last one's
      cb = split.owner(i0 + units - 1);
      if (ca != blockIdx.x) cb = ca;                   // no part before this boundary, or cut before already
    }
    if (lane == 0) {
      s_ca = ca;
      s_cb = cb;
      s_b = b;
      s_item = static_cast<int32_t>(item);
      s_late = split.begin(ca) < i0;
    }
  }
  pdl_wait();                                          // (until here only the lengths were read)
  __syncthreads();
  const uint32_t ca = s_ca, cb = s_cb;
  if (ca == cb) return;
  // CTA ca's part is its last segment unless the item begins its range; the
  // others' is their first.  The statistics of 32 parts are read at a time.
  const int64_t b = s_b;
  const int h = s_item / p.row_tiles, row0 = s_item % p.row_tiles * p.tile_rows;
  const int nrows = min(p.tile_rows, p.rows - row0);
  const uint32_t first = 2 * ca + static_cast<uint32_t>(s_late);
  for (int in = blockIdx.y * kJoinRows + warp; in < min(nrows, static_cast<int>(blockIdx.y + 1) * kJoinRows); in += 8) {
    const int rr = row0 + in, l = rr / p.G;
    const int64_t row = (b * p.L + l) * p.Hq + h * p.G + (rr - l * p.G);
    const int n = place(in >= p.half ? in - p.half + columns : in);   // the row's column (columns: of a softmax group)
    auto slot_of = [&](uint32_t c) { return static_cast<int64_t>(c == ca ? first : 2 * c); };
    float m = kUnset, sum = 0.0f;
    float o[V] = {};
    auto part = [&](uint32_t c) {
      PartV x;
      const float* src = p.part_o + (slot_of(c) * N + n) * D + lane * V;
      if constexpr (V == 4) {
        const float4 y = __ldcg(reinterpret_cast<const float4*>(src));
        x.v[0] = y.x, x.v[1] = y.y, x.v[2] = y.z, x.v[3] = y.w;
      } else {
        const float2 y = __ldcg(reinterpret_cast<const float2*>(src));
        x.v[0] = y.x, x.v[1] = y.y;
      }
      return x;
    };
    const PartV x0 = part(ca), x1 = part(ca + 1);      // (at least two: asked for before their factors are known)
    for (uint32_t c0 = ca; c0 <= cb; c0 += 32) {
      const uint32_t c = c0 + lane;
      float mc = -kInf, lc = 0.0f;
      if (c <= cb) {
        const float2 ml = __ldcg(reinterpret_cast<const float2*>(p.part_ml) + slot_of(c) * N + n);
        mc = ml.x;
        lc = ml.y;
      }
      const float now = fmaxf(m, warp_max_f32(mc));
      const float fa = ex2_approx(m - now), fb = ex2_approx(mc - now);
      float add = lc * fb;
#pragma unroll
      for (int k = 16; k > 0; k >>= 1) add += __shfl_xor_sync(0xFFFFFFFFu, add, k);
      sum = sum * fa + add;
#pragma unroll
      for (int i = 0; i < V; ++i) o[i] *= fa;
      const int parts = static_cast<int>(cb - c0 + 1 < 32 ? cb - c0 + 1 : 32);
      auto add_part = [&](const PartV& x, int k) {
        const float f = __shfl_sync(0xFFFFFFFFu, fb, k);
#pragma unroll
        for (int i = 0; i < V; ++i) o[i] = fmaf(x.v[i], f, o[i]);
      };
      if (c0 == ca) {
        add_part(x0, 0);
        add_part(x1, 1);
      }
#pragma unroll 4
      for (int k = c0 == ca ? 2 : 0; k < parts; ++k) add_part(part(c0 + k), k);
      m = now;
    }
    uint32_t u[V / 2];
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
      const float lo = sum == 0.0f ? 0.0f : o[2 * i] / sum, hi = sum == 0.0f ? 0.0f : o[2 * i + 1] / sum;
      asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(u[i]) : "f"(hi), "f"(lo));
    }
    uint16_t* to = p.out + row * D + lane * V;
    if constexpr (V == 4) *reinterpret_cast<uint2*>(to) = make_uint2(u[0], u[1]);
    else *reinterpret_cast<uint32_t*>(to) = u[0];
    if (lane == 0) p.lse[row] = lse_of(m, sum);
  }
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

template <int N, bool PAIR>
AttendVariant attend_variant_n(int dim) {
  if (dim == 64) return {reinterpret_cast<const void*>(&attend_kernel<64, N, PAIR>), attend_smem<64, N, PAIR>()};
  return {reinterpret_cast<const void*>(&attend_kernel<128, N, PAIR>), attend_smem<128, N, PAIR>()};
}

// By the columns of both groups: 32 and 64 taking turns, 128 paired.
AttendVariant attend_variant(int dim, int columns) {
  if (columns == 32) return attend_variant_n<32, false>(dim);
  if (columns == 64) return attend_variant_n<64, false>(dim);
  return attend_variant_n<64, true>(dim);
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
      for (int n = 32; n <= 128 && d.err == cudaSuccess; n *= 2) {
        const AttendVariant v = attend_variant(dim, n);
        d.err = cudaFuncSetAttribute(v.kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, v.smem);
      }
    for (const void* k : {reinterpret_cast<const void*>(&attend_weights_kernel<64>),
                          reinterpret_cast<const void*>(&attend_weights_kernel<128>)})
      if (d.err == cudaSuccess)
        d.err = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     weights_smem(128, kWeightRows / kWeightCols));
    if (d.err != cudaSuccess) (void)cudaGetLastError();  // reported through the status; no sticky error
  });
  return g_at[dev].err == cudaSuccess ? &g_at[dev] : nullptr;
}

// The row tiles of a key head and the columns of a tile: as few tiles as 128
// columns allow, equally filled, then the narrowest built width that holds one
// (a width is the tensor core's N and the softmax's registers per token).
// Measured: 32 rows 39.4 us with 32 columns, 51.3 with 64 (8 x 2306 tokens, 32
// heads); 64 rows 56.6 us taking turns with 64 columns, 66.0 paired, 65.0 as two
// tiles of 32 (16 x 5096 tokens, 8 heads); 112 rows 54.6 us paired, 54.6 as two
// tiles of 56, 59.7 as four of 28; 224 rows of 2000 to 8192 tokens 88.9 us as two of
// 112, 95.6 as four of 56.
struct RowTiles {
  int64_t tiles, rows, half;
  int columns;
};
RowTiles row_tiles(int64_t rows) {
  RowTiles t;
  t.tiles = (rows + 127) / 128;
  t.rows = (rows + t.tiles - 1) / t.tiles;
  t.columns = t.rows <= 32 ? 32 : (t.rows <= 64 ? 64 : 128);
  t.half = t.columns == 128 ? (t.rows + 1) / 2 : t.rows;
  return t;
}

// What an item costs besides its tiles, in tiles (about 7000 cycles against
// 1500, 2200 and 3700 a tile).  With fewer tiles than SMs there is nothing to
// balance, and each tile is a CTA's.  Measured: 32 sequences of 100 to 4096 tokens,
// 4 rows of 8 heads, 72.7 us without and 33.3 with; 8 of 517 to 4096, 32 rows of 32
// heads, masked, 56.0 and 48.8; 16 of 2000 to 8192, 224 rows of 4 heads, 93.9 and
// 88.9.  One tile more: 33.8, 49.3 and 87.8; one less: 35.8, 48.0 and 90.9.
constexpr int32_t kSegCost32 = 4, kSegCost64 = 3, kSegCost128 = 2;

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
  return attend_workspace(dev ? dev->sms : 1024, row_tiles(L * (Hq / heads)).columns, static_cast<int>(head_dim));
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
  if (key_mask && (!aligned16(key_mask) || mask_stride % 16 != 0)) return DLLM_ERR_UNSUPPORTED;   // (bulk copies)
  // (a TMA coordinate is an int32: the pool's rows of one token and head)
  if (rows > INT32_MAX || cache->num_pages * cache->heads * cache->page_size > INT32_MAX) return DLLM_ERR_UNSUPPORTED;
  if (!workspace) return DLLM_ERR_WORKSPACE;
  if (!aligned16(workspace)) return DLLM_ERR_INVALID_ARGUMENT;
  const RowTiles rt = row_tiles(L * (Hq / cache->heads));
  if (workspace_bytes < attend_workspace(1, rt.columns, cache->head_dim)) return DLLM_ERR_WORKSPACE;
  // Rows are stored while other items' queries are still to be read, and the
  // weights read all of them once more.
  const int64_t D = cache->head_dim, in_place[3] = {L * Hq * D, Hq * D, D};
  int64_t last = D;
  bool same = out == q && !weights;
  for (int i = 0; i < 3; ++i) {
    last += (extent[i] - 1) * q_strides[i];
    same = same && (extent[i] == 1 || q_strides[i] == in_place[i]);
  }
  const uintptr_t q0 = reinterpret_cast<uintptr_t>(q), o0 = reinterpret_cast<uintptr_t>(out);
  if (!same && q0 < o0 + static_cast<uintptr_t>(rows * D) * 2 && o0 < q0 + static_cast<uintptr_t>(last) * 2)
    return DLLM_ERR_INVALID_ARGUMENT;
  const AttendDevice* dev = attend_device();
  if (!dev) return DLLM_ERR_CUDA;
  // One CTA per SM, fewer when there are fewer tiles than that.
  const int64_t most = mul_or_neg(mul_or_neg(B, cache->heads), rt.tiles * ((cap + kTile - 1) / kTile));
  if (mul_or_neg(most, 8) < 0 || most * 8 > INT32_MAX) return DLLM_ERR_UNSUPPORTED;   // (units are 32-bit)
  const int64_t ctas = std::min<int64_t>(dev->sms, most);
  if (workspace_bytes < attend_workspace(ctas, rt.columns, cache->head_dim)) return DLLM_ERR_WORKSPACE;
  AttendParams p;
  std::memset(&p, 0, sizeof(p));
  p.c = cache_view(*cache);
  const bool d64 = cache->head_dim == 64;
  if (!pool_map(&p.tm_k, cache->k, p.c, d64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B) ||
      !pool_map(&p.tm_v, cache->v, p.c, d64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B))
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
  p.half = static_cast<int32_t>(rt.half);
  p.ctas = static_cast<int32_t>(ctas);
  p.seg_cost = ctas < dev->sms ? 0 : (rt.columns == 32 ? kSegCost32 : (rt.columns == 64 ? kSegCost64 : kSegCost128));
  uint8_t* w = static_cast<uint8_t*>(workspace);
  p.fault = reinterpret_cast<int32_t*>(w);
  p.part_o = reinterpret_cast<float*>(w + kAttendHeader);
  p.part_ml = p.part_o + 2 * ctas * rt.columns * cache->head_dim;
  void* args[] = {&p};
  const AttendVariant v = attend_variant(cache->head_dim, rt.columns);
  st = launch_pdl(v.kernel, dim3(static_cast<unsigned>(ctas)), dim3(kAttendThreads), static_cast<size_t>(v.smem),
                  stream, args);
  if (st != DLLM_OK) return st;
  int columns = rt.columns, per_group = rt.columns == 128 ? 64 : rt.columns;
  void* jargs[] = {&p, &columns, &per_group};
  if (ctas > 1)
    st = launch_pdl(d64 ? reinterpret_cast<const void*>(&attend_join_kernel<64>)
                        : reinterpret_cast<const void*>(&attend_join_kernel<128>),
                    dim3(static_cast<unsigned>(ctas - 1), static_cast<unsigned>((rt.rows + kJoinRows - 1) / kJoinRows)),
                    dim3(256), 0, stream, jargs);
  if (st != DLLM_OK || !weights) return st;
  // The weights: kWeightRows rows of a key head at a time, K read once for each.
  p.row_tiles = 1;
  p.seg_cost = p.seg_cost > 0 ? 2 : 0;
  for (int64_t r = 0; r < L * p.G && st == DLLM_OK; r += kWeightRows) {
    int32_t first = static_cast<int32_t>(r), count = static_cast<int32_t>(std::min<int64_t>(kWeightRows, L * p.G - r));
    void* wargs[] = {&p, &first, &count};
    const int chunks = (count + kWeightCols - 1) / kWeightCols;
    st = launch_pdl(d64 ? reinterpret_cast<const void*>(&attend_weights_kernel<64>)
                        : reinterpret_cast<const void*>(&attend_weights_kernel<128>),
                    dim3(static_cast<unsigned>(std::min<int64_t>(
                        dev->sms, B * cache->heads * ((cap + kTile - 1) / kTile)))),
                    dim3(kWeightThreads), static_cast<size_t>(weights_smem(cache->head_dim, chunks)), stream, wargs);
    p.decay = 1.0f;
  }
  return st;
}

}  // extern "C"
