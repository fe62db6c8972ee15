// dllm_head.cu -- scores of given tokens straight from the hidden states, and
// their gradient: logits z = h W^T that are never stored (sm_103a).
//
// Only scored rows (a target in [0, V)) take part: a first kernel numbers them and
// gathers their hidden states (unless all rows are scored), and every later kernel
// reads their count n on the device.
//
// Forward: one matrix product whose epilogue folds a tile's logits into a
// partial softmax (m, sum 2^y, sum 2^y y, y = (z - m) log2 e) per row; a last
// kernel joins a row's partials.
//
// Backward, over pieces of the vocabulary so that only a piece of dz is ever
// held (bf16, as the product's operands have to be; of up to 128 scored rows in two parts,
// whose second takes the half of dH's tiles that is empty then, and for a dW of 32 bits): dz = the product again,
// with p = exp(z - lse) and dz = -p (g + gH (z - lse + H)) + g [v = target] in its
// epilogue; dH += dz W over the piece (K: the piece's ids); dW = dz^T H (K: the
// scored rows).
//
// All products run on the 5th-generation tensor cores, a pair of CTAs a tile of
// 256 x 256 (cta_group::2): each CTA holds 128 rows of A and of the accumulator
// and half of B's columns, so that a slab of K costs a CTA 32 KB of shared memory.
// TMA brings 64-wide slabs of K into a ring (128-byte swizzle), tcgen05.mma (bf16
// in, fp32 accumulate) fills one of two accumulators in TMEM while eight epilogue
// warps of each CTA empty the other.  K-major operands (hidden and weight in the first
// product, dz in the second) lie as rows of 64 k; the others (weight in the
// second, both in the third) are read as they lie in memory, MN-major, as rows
// of 64 m or n.
//
// What bounds it: the weight's stream while there are few rows (32 x 126464 x 4096 in
// 161 to 166 us, 6.2 to 6.5 TB/s), from some 300 rows on the tensor cores, and in a run of
// such calls the card's power: 4096 x 152064 x 3584 in 2.43 to 2.54 ms (1.76 to 1.84
// PFLOP/s), 4506 x 126464 x 4096 backward in 8.4 to 8.7 ms (1.61 to 1.67; a cuBLAS product
// of 8192^3 run for seconds: 1.69).
#include <cuda.h>  // CUtensorMap and its enums (types only; the encoder comes from the driver at run time)
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <mutex>

#include "../../include/dllmcommit.h"
#include "dllm_device.cuh"
#include "dllm_launch.cuh"

namespace dllm {

constexpr int kHdBM = 256;                       // rows of a pair's accumulator tile
constexpr int kHdRows = kHdBM / 2;               // a CTA's
constexpr int kHdBN = 256;                       // its columns at most
constexpr int kHdBK = 64;                        // K of a stage: one 128-byte swizzle row of bf16
constexpr int kHdABytes = kHdRows * kHdBK * 2;   // 16 KB: a CTA's part of a slab of A, whole
constexpr int kHdBBytes = kHdBN / 2 * kHdBK * 2; // 16 KB
constexpr int kHdMaxStages = 16;                 // of the ring: 7 of 32 KB, 6 where tiles are stored by TMA, more of narrow ones
constexpr int kHdEpiWarps = 8;                   // two warpgroups, each reads every other 32-column chunk of a tile
constexpr int kHdTmaWarp = 10;
constexpr int kHdMmaWarp = 11;
constexpr int kHdThreads = 12 * 32;
constexpr int kHdTmemCols = 512;
constexpr int kHdStoreBytes = 32 * 64 * 2;       // a warp's 32 rows of 64 bf16 columns on their way out
constexpr int kHdRing = 7 * (kHdABytes + kHdBBytes);
constexpr int kHdSmem = kHdRing + 1024;
constexpr int kHdBand = 16;                      // row tiles that share a pass over the vocabulary (4096 rows: 32 MB of
                                                 // hidden states of 4096 stay in L2 while the weight streams)
constexpr float kHdCap = 0x1p+125f;              // logits are read within +-2^125 (NaN as the lowest): differences stay finite
constexpr float kHdAbsent = -0x1p+126f;          // suppressed ids and columns past the vocabulary

enum HeadOp { kHdScore, kHdDz, kHdBack };         // the last: dH and dW, tiles of both in one launch
enum HeadOut { kHdBf16, kHdBf16Add, kHdF32 };

// The tensor core adds in fp32 and cuts off what does not fit: summed in one
// accumulator, the logits of d = 4096 were off by 4e-6 of themselves, always toward
// zero, and a confident row's log probability by 2e-5.  So an accumulator takes some
// slabs of K, and these parts are added in registers, rounded.  Entropies of 32 rows of
// d = 4096 and the time of 4096 x 152064 x 3584 in parts of 8, 9, 10, 11 and 12 slabs: off
// by 5.7e-7, 7.1e-7, 7.3e-7, 8.1e-7 and 8.9e-7 of themselves; 2575, 2530, 2478, 2521 and
// 2462 us (16: 2463; 4: some 2760).  dz, which is rounded to bf16, only has to agree with
// a log-sum-exp so formed.
//
// A sum of dW is as long as the rows scored: of 2^21 terms of one sign it was off by
// 1.4 %.  It takes parts of at most 128 slabs, of about one length (backward of 4506 x
// 126464 x 4096, 71 slabs: in one part 8.54 ms, in two 8.58, in three 8.69).  The registers
// that hold them make the epilogue of short tiles slower (61 x 50257 x 768: 65 and 69
// us), so the kernel with parts is another one, taken where there may be as many rows.
// dH's sums are rounded to bf16 and split over the piece's ids already.
__host__ __device__ constexpr int hd_part(int op) { return op == kHdScore ? 10 : (op == kHdDz ? 16 : 128); }

__device__ __forceinline__ int hd_dw_part(int slabs) {
  const int parts = (slabs + hd_part(kHdBack) - 1) / hd_part(kHdBack);
  return (slabs + parts - 1) / parts;
}

// A scored row's constants of the backward pass.
struct HeadRow {
  float lse, entropy, g, gh;
};

struct HeadParams {
  CUtensorMap tm_a, tm_b;        // the operands; where one is the hidden states, the caller's tensor,
  CUtensorMap tm_packed;         // read when every row is scored, and else their gathered copy
  CUtensorMap tm_aw, tm_bw;      // dw's operands, as rows of 64 m or n (tm_packed then for these)
  CUtensorMap tm_out;            // the weight's gradient
  const int32_t* n_rows;         // device: the scored rows; then the splits of the second product (null: all T rows)
  int64_t T, V;
  int64_t v0;                    // the piece's first id
  int64_t cols;                  // its ids
  int64_t d;
  int32_t bn;                    // columns of a tile
  int32_t n_n;                   // tiles along N
  uint32_t idesc, idesc_w;       // (of dw)
  int32_t want_h, want_w;        // dh and dw: wanted
  uint32_t a_bytes;              // what a CTA's load of A brings
  uint32_t stage_bytes;          // of the ring: A, then B's share of a tile
  int32_t stages, clear_a;
  const int32_t* target;         // per scored row
  int32_t n_sup;
  int32_t sup[DLLM_MAX_SUPPRESS];
  float4* part;                  // score: (tiles along N, or pairs where there is one row tile; 2; rows): m, Z, S
  int64_t part_rows;
  float* z_target;               // score: per scored row
  const HeadRow* row;            // dz
  uint16_t* dz;                  // dz: (rows, dz_stride) bf16
  int32_t low;                   // a dw of 32 bits and more than kHdRows rows: dz's second part begins at this row
  int64_t dz_stride;
  float* acc;                    // dh: (splits, row tiles x 256, acc_stride) fp32
  int64_t acc_stride;
  int32_t add;                   // dh: the piece is not the first
  void* grad_w;                  // dw
  int64_t grad_w_stride;
  int32_t grad_w_f32, accumulate;
  int32_t *fault, *seen;         // the workspace's word and the device's
};

// Instruction descriptor of tcgen05.mma.kind::f16: fp32 accumulator (bits 4-5 =
// 1), bf16 A and B (bits 7-9, 10-12 = 1), MN-major A, B (bits 15, 16), N / 8 in
// bits 17-22, M / 16 in bits 24-28.
constexpr uint32_t hd_idesc(bool a_mn, bool b_mn, int bn) {
  return (1u << 4) | (1u << 7) | (1u << 10) | (a_mn ? 1u << 15 : 0u) | (b_mn ? 1u << 16 : 0u) |
         (static_cast<uint32_t>(bn >> 3) << 17) | (static_cast<uint32_t>(kHdBM >> 4) << 24);
}

// Shared-memory descriptor in the 128-byte swizzle: start / 16 in bits 0-13, the
// leading offset / 16 in bits 16-29 (MN-major: the distance of spans of 64 along M
// or N; K-major: unused), the stride offset / 16 in bits 32-45 (1024 bytes, 8
// rows of 128), version 1 at bit 46, swizzle 2 at bits 61-63.
__device__ __forceinline__ uint32_t hd_desc(uint32_t addr) { return ((addr & 0x3FFFFu) >> 4) | (8192u >> 4) << 16; }
constexpr uint32_t kHdDescHigh = (1024u >> 4) | 1u << 14 | 2u << 29;

__device__ __forceinline__ uint32_t hd_elect() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r;
}

// What follows is issued by the one thread of the warp whose `lead` is set; the whole
// warp executes the code around it, so that addresses and descriptors stay in uniform
// registers (formed by a single thread, a product and a load held a slab up by some
// 170 and 190 cycles each: 32 x 126464 x 4096 took 187 us, and 169 so, 4506 x 126464 x 4096
// backward 9.0 and 8.4 ms).

// A load of this CTA's shared memory that counts on the leader's barrier.
__device__ __forceinline__ void hd_load(uint32_t lead, uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %5, 0;\n\t"
      "@q cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];\n\t}" ::
          "r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar), "r"(lead)
      : "memory");
}

__device__ __forceinline__ void hd_expect(uint32_t lead, uint32_t bar, uint32_t bytes) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %2, 0;\n\t"
      "@q mbarrier.arrive.expect_tx.release.cta.shared::cta.b64 _, [%0], %1;\n\t}" ::"r"(bar),
      "r"(bytes), "r"(lead)
      : "memory");
}

__device__ __forceinline__ void hd_mma(uint32_t lead, uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b64 a, b;\n\tsetp.ne.u32 p, %5, 0;\n\tsetp.ne.u32 q, %6, 0;\n\t"
      "mov.b64 a, {%1, %3};\n\tmov.b64 b, {%2, %3};\n\t"
      "@q tcgen05.mma.cta_group::2.kind::f16 [%0], a, b, %4, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "r"(kHdDescHigh), "r"(idesc), "r"(acc), "r"(lead)
      : "memory");
}

// Arrives on the barrier at this place of both CTAs when the products issued so far are done.
__device__ __forceinline__ void hd_commit(uint32_t lead, uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %2, 0;\n\t"
      "@q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n\t}" ::"r"(bar),
      "h"(static_cast<uint16_t>(3)), "r"(lead)
      : "memory");
}

__device__ __forceinline__ uint32_t hd_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// The place of addr in the leader's shared memory.
__device__ __forceinline__ uint32_t hd_leader(uint32_t addr) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(addr));
  return r;
}
// (no memory is passed on, and a release over the cluster took a microsecond)
__device__ __forceinline__ void hd_arrive_leader(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void hd_cluster_sync() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__device__ __forceinline__ void hd_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void hd_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// 32 consecutive fp32 columns of this warp's 32 TMEM lanes, one lane a thread.
__device__ __forceinline__ void hd_ld32(uint32_t taddr, float (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]), "=f"(r[8]),
        "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15]), "=f"(r[16]),
        "=f"(r[17]), "=f"(r[18]), "=f"(r[19]), "=f"(r[20]), "=f"(r[21]), "=f"(r[22]), "=f"(r[23]), "=f"(r[24]),
        "=f"(r[25]), "=f"(r[26]), "=f"(r[27]), "=f"(r[28]), "=f"(r[29]), "=f"(r[30]), "=f"(r[31])
      : "r"(taddr)
      : "memory");
}

// 16 columns.
__device__ __forceinline__ void hd_ld16(uint32_t taddr, float (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]), "=f"(r[8]),
        "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15])
      : "r"(taddr)
      : "memory");
}

// A bounded wait: false after the deadline or once the CTA gave up.
__device__ __forceinline__ bool hd_wait(uint32_t bar, uint32_t parity, volatile int32_t* abort_flag) {
  if (mbar_try_wait(bar, parity)) return true;
  const long long t0 = clock64();
  for (;;) {
    if (mbar_try_wait_sleep(bar, parity, kSleepHintNs)) return true;
    if (*abort_flag) return false;
    if (clock64() - t0 > kWaitLimitCycles) return false;
  }
}

__device__ __forceinline__ void hd_fail(const HeadParams& p, volatile int32_t* abort_flag, int32_t code) {
  if (!*abort_flag) {
    atomicExch(p.fault, code);
    atomicExch(p.seen, code);
    *abort_flag = 1;
  }
}

// bf16 pair, lo in the low half.
__device__ __forceinline__ uint32_t hd_bf16x2(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}

// A tile of dw costs its slabs and, for its output's 128 KB, those of 4 more (512 x
// 126464 x 4096: 1146, 1120 and 1107 us with 2, 3 and 4 more); one of up to 4 slabs 2
// more (61 x 50257 x 768, 2 slabs: 76, 68, 66, 67, 70 and 73 us with 0, 1, 2, 3, 4 and 6
// more; 100 x 126464 x 4096, 4 slabs: 669, 635, 615, 616, 637 and 665).
__host__ __device__ constexpr int hd_dw_cost(int slabs) { return slabs > 4 ? slabs + 4 : slabs + 2; }

// dz in two parts: up to kHdRows scored rows, however many are given, leave half of every
// tile of dh empty, and what bf16 cuts off dz takes it, as the rows from kHdRows on.  For
// a dw of 32 bits dz has its second part whatever the rows (`low`, where it begins, is
// not 0), which meets the same hidden states in as many slabs more: of one part such
// a gradient would be no more exact than one of 16 bits.  (512 x 126464 x 4096 into fp32:
// 1.20 and 1.50 ms, 4506 rows 8.6 and 11.6.)
__device__ __forceinline__ bool hd_two(int64_t n) { return n <= kHdRows; }

// The slabs of a tile of dw.
__device__ __forceinline__ int hd_dw_slabs(int64_t n, int32_t low) {
  return static_cast<int>((n + kHdBK - 1) / kHdBK) * (hd_two(n) || low > 0 ? 2 : 1);
}

// How many ways the second product's K is split: the least of the pairs' time, which
// is their share of all tiles, or the rounds that dh's take where these are more (the
// third product's tiles fill what a last round of dh leaves), and 8 bytes a split of
// every element written and read again (1.5 MB in the time of a slab of 256 x 256 x
// 64).  Called by a whole warp, a lane a number of splits.
__device__ __forceinline__ int hd_splits(int64_t n, int n_n, int bn, int pairs, int slabs, int64_t dw_tiles, int32_t low, int64_t room) {
  const int s = (threadIdx.x & 31) + 1;
  const int tiles = static_cast<int>((n + kHdBM - 1) / kHdBM) * n_n;
  const float size = static_cast<float>(tiles) * static_cast<float>(kHdBM * bn);
  const float share = (static_cast<float>(tiles) * slabs +
                       static_cast<float>(dw_tiles) * hd_dw_cost(hd_dw_slabs(n, low))) / static_cast<float>(pairs);
  const float rounds = ceilf(static_cast<float>(tiles) * s / static_cast<float>(pairs)) * ceilf(static_cast<float>(slabs) / s);
  float cost = fmaxf(share, rounds) * (bn / 256.0f) + s * size * (8.0f / 1.5e6f);
  if (s > 1 && (s > slabs || static_cast<int64_t>(s) * tiles * kHdBM * bn > room)) cost = 3.0e38f;
  const float least = -warp_max_f32(-cost);
  return __ffs(__ballot_sync(0xFFFFFFFFu, cost == least));
}

// A tile of a product.  A split of a short last piece may hold no slab: such a tile
// is passed over (what it adds to, an earlier piece has written).
struct HeadTile {
  int32_t m, n;        // tile coordinates
  int32_t k0, k1;      // slabs
  int32_t split;
  bool dw;
};

// The tiles in the order in which this pair of CTAs takes them: tile i goes to pair i
// mod pairs, dh's before dw's; the pairs that a last round of dh leaves out take as
// many tiles of dw as fit its time first.
template <int OP>
struct HeadWork {
  int64_t pair, pairs;
  int32_t n_n;
  int32_t n_m, slabs, splits;            // of scores, dz or dh
  int64_t total;
  bool two;                              // dz in two parts, for dh and dw
  int32_t low;                           // the second part's first row (0: there is none)
  int32_t slabs_w, rest;                 // dw; dh's tiles in a last round
  int64_t total_w, extra;

  __device__ __forceinline__ HeadWork(const HeadParams& p, int64_t n)
      : pair(blockIdx.x >> 1), pairs(gridDim.x >> 1), n_n(p.n_n), splits(1), two(hd_two(n)), low(two ? kHdRows : p.low), slabs_w(0), rest(0), total_w(0), extra(0) {
    n_m = static_cast<int32_t>((n + kHdBM - 1) / kHdBM);
    if (OP != kHdBack) {
      slabs = static_cast<int32_t>((p.d + kHdBK - 1) / kHdBK);
      total = static_cast<int64_t>(n_m) * n_n;
      return;
    }
    slabs = static_cast<int32_t>((p.cols + kHdBK - 1) / kHdBK);
    splits = p.n_rows[1];
    total = p.want_h ? static_cast<int64_t>(n_m) * n_n * splits : 0;
    slabs_w = hd_dw_slabs(n, low);
    total_w = p.want_w && n > 0 ? (p.cols + kHdBM - 1) / kHdBM * n_n : 0;
    rest = static_cast<int32_t>(total % pairs);
    if (rest > 0) extra = min(static_cast<int64_t>(slabs / splits / hd_dw_cost(slabs_w)), total_w / (pairs - rest));
  }

  // Its tile number `it`; false behind the last.
  __device__ __forceinline__ bool tile(int64_t it, HeadTile& t) const {
    t.split = 0;
    t.k0 = 0;
    t.k1 = slabs;
    t.dw = false;
    int64_t i = it * pairs + pair;
    if (OP != kHdBack) {
      if (i >= total) return false;
      // bands of row tiles, each over the whole vocabulary, its row tiles inner
      const int32_t bands = (n_m + kHdBand - 1) / kHdBand, high = (n_m + bands - 1) / bands;
      const int64_t per_band = static_cast<int64_t>(high) * n_n;
      const int32_t band = static_cast<int32_t>(i / per_band);
      const int32_t in = static_cast<int32_t>(i - band * per_band);
      const int32_t rows = min(high, n_m - band * high);
      t.m = band * high + in % rows;
      t.n = in / rows;
      return true;
    }
    if (i < total) {
      const int64_t tiles = static_cast<int64_t>(n_m) * n_n;
      t.split = static_cast<int32_t>(i / tiles);
      const int32_t in = static_cast<int32_t>(i - t.split * tiles);
      t.m = in / n_n;
      t.n = in % n_n;
      t.k0 = static_cast<int32_t>(static_cast<int64_t>(slabs) * t.split / splits);
      t.k1 = static_cast<int32_t>(static_cast<int64_t>(slabs) * (t.split + 1) / splits);
      return true;
    }
    const bool left_out = pair >= rest;                  // of the last round of dh
    int64_t j = it - total / pairs - (left_out ? 0 : 1);
    if (left_out && j < extra) {
      i = j * (pairs - rest) + pair - rest;
    } else {
      if (left_out) j -= extra;
      i = extra * (pairs - rest) + j * pairs + pair;
    }
    if (i >= total_w) return false;
    t.dw = true;
    t.k1 = slabs_w;
    t.m = static_cast<int32_t>(i / n_n);
    t.n = static_cast<int32_t>(i % n_n);
    return true;
  }
};

// A row's running softmax: m, and sums of 2^y and 2^y y with y = (z - m) log2 e.
struct HeadSoft {
  float m, Z, S;
};

__device__ __forceinline__ void hd_raise(HeadSoft& a, float m) {
  const float d = fmaxf(a.m - m, -1000.0f) * kLog2e, f = ex2_approx(d);
  a.S = f * fmaf(d, a.Z, a.S);
  a.Z *= f;
  a.m = m;
}

__device__ __forceinline__ void hd_join(HeadSoft& a, HeadSoft b) {
  const float m = fmaxf(a.m, b.m);
  hd_raise(a, m);
  hd_raise(b, m);
  a.Z += b.Z;
  a.S += b.S;
}

// The columns of a 32-column chunk at id v0 that hold no id to be counted.
__device__ __forceinline__ uint32_t hd_absent(const int32_t* sup, int n_sup, int64_t v0, int lim) {
  uint32_t absent = lim >= 32 ? 0u : ~((1u << lim) - 1u);
  for (int q = 0; q < n_sup; ++q) {
    const int64_t off = sup[q] - v0;
    if (off >= 0 && off < 32) absent |= 1u << off;
  }
  return absent;
}

// 32 columns of an accumulator row as bf16 to 32-byte aligned memory, whole sectors a
// store; `lim` of them exist.
__device__ __forceinline__ void hd_store_dz(uint16_t* out, const float (&x)[32], int lim) {
#pragma unroll
  for (int j = 0; j < 32; j += 16) {
    if (j >= lim) break;
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(out + j), "r"(hd_bf16x2(x[j], x[j + 1])),
                 "r"(hd_bf16x2(x[j + 2], x[j + 3])), "r"(hd_bf16x2(x[j + 4], x[j + 5])), "r"(hd_bf16x2(x[j + 6], x[j + 7])),
                 "r"(hd_bf16x2(x[j + 8], x[j + 9])), "r"(hd_bf16x2(x[j + 10], x[j + 11])),
                 "r"(hd_bf16x2(x[j + 12], x[j + 13])), "r"(hd_bf16x2(x[j + 14], x[j + 15]))
                 : "memory");
  }
}

// What this warp wrote to its buffer, to column col and row `row` of the tensor.
__device__ __forceinline__ void hd_tile_out(const CUtensorMap* map, int col, int row, uint32_t buf, int lane) {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  __syncwarp();
  if (lane == 0) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];" ::"l"(reinterpret_cast<uint64_t>(map)),
                 "r"(col), "r"(row), "r"(buf)
                 : "memory");
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
  }
}

// This warp's 32 rows of 64 columns (a row a thread, 32 of them in each of x and y), as
// bf16, to column col and row `row` of the tensor: through shared memory in the 128-byte
// swizzle and out by TMA, so that memory sees whole lines (stored from registers, a row a
// thread, the weight's gradient of 512 x 126464 x 4096 took 504 us in a launch of its own,
// and 381 so).
__device__ __forceinline__ void hd_store_tile(const float (&x)[32], const float (&y)[32], uint32_t buf, const CUtensorMap* map, int col,
                                              int row, int lane) {
  if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");   // (the last one has left the buffer)
  __syncwarp();
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float* v = (j < 4 ? x : y) + 8 * (j & 3);
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(buf + lane * 128 + ((j ^ (lane & 7)) << 4)), "r"(hd_bf16x2(v[0], v[1])),
                 "r"(hd_bf16x2(v[2], v[3])), "r"(hd_bf16x2(v[4], v[5])), "r"(hd_bf16x2(v[6], v[7]))
                 : "memory");
  }
  hd_tile_out(map, col, row, buf, lane);
}

// The same, added to what is there, whose 32 x 64 the buffer holds (loaded by TMA while
// the products ran; read from memory a row a thread, 512 x 126464 x 4096 took 9.6 ms
// where it now takes 1.2).
__device__ __forceinline__ void hd_load_old(uint32_t buf, const CUtensorMap* map, int x, int y, uint32_t bar) {
  mbar_arrive_expect_tx(bar, kHdStoreBytes);
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(buf),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
      : "memory");
}

__device__ __forceinline__ void hd_add_tile(const float (&x)[32], const float (&y)[32], uint32_t buf, const CUtensorMap* map, int col,
                                            int row, int lane) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float* v = (j < 4 ? x : y) + 8 * (j & 3);
    const uint32_t at = buf + lane * 128 + ((j ^ (lane & 7)) << 4);
    const uint4 o = lds128(at);
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) w[e] = hd_bf16x2(v[2 * e] + bf16lo((&o.x)[e]), v[2 * e + 1] + bf16hi((&o.x)[e]));
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]) : "memory");
  }
  hd_tile_out(map, col, row, buf, lane);
}

// 32 columns in fp32, stored or added to what is there.
__device__ __forceinline__ void hd_store_tile_f32(const float (&x)[32], uint32_t buf, const CUtensorMap* map, int col, int row, int lane,
                                                  bool add) {
  if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
  __syncwarp();
#pragma unroll
  for (int j = 0; j < 8; ++j)
    asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(buf + lane * 128 + ((j ^ (lane & 7)) << 4)), "f"(x[4 * j]),
                 "f"(x[4 * j + 1]), "f"(x[4 * j + 2]), "f"(x[4 * j + 3])
                 : "memory");
  if (!add) {
    hd_tile_out(map, col, row, buf, lane);
    return;
  }
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  __syncwarp();
  if (lane == 0) {
    asm volatile("cp.reduce.async.bulk.tensor.2d.global.shared::cta.add.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(col), "r"(row), "r"(buf)
                 : "memory");
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
  }
}

__device__ __forceinline__ void hd_store_f32(float* out, const float (&x)[32], int lim, bool add) {
#pragma unroll
  for (int j = 0; j < 32; j += 4) {
    if (j >= lim) break;
    float4* at = reinterpret_cast<float4*>(out + j);
    float4 y = make_float4(x[j], x[j + 1], x[j + 2], x[j + 3]);
    if (add) {
      const float4 o = *at;
      y.x += o.x, y.y += o.y, y.z += o.z, y.w += o.w;
    }
    *at = y;
  }
}

// Of kHdBack, OUT: how dW leaves; LONG: in parts.
template <int OP, int OUT = kHdBf16, bool LONG = false>
__global__ void __launch_bounds__(kHdThreads, 1) head_kernel(const __grid_constant__ HeadParams p) {
  extern __shared__ __align__(1024) uint8_t hd_smem[];
  __shared__ __align__(8) uint64_t full_bar[kHdMaxStages], empty_bar[kHdMaxStages], accf_bar[2], acce_bar[2];
  __shared__ __align__(8) uint64_t old_bar[kHdEpiWarps][2];
  __shared__ uint32_t tmem_slot;
  __shared__ int32_t abort_flag_s;
  __shared__ int32_t sup_s[DLLM_MAX_SUPPRESS];
  volatile int32_t* abort_flag = &abort_flag_s;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = hd_rank();
  const uint32_t ring = (smem_addr(hd_smem) + 1023u) & ~1023u;

  // full (counted in the leader, by the loads of both CTAs) and acce (the epilogue
  // warps of both) are waited for by the leader's products; empty and accf are
  // arrived at in both CTAs by the products.
  if (threadIdx.x == 0) {
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(smem_addr(&full_bar[s]), 1);
      mbar_init(smem_addr(&empty_bar[s]), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(smem_addr(&accf_bar[b]), 1);
      mbar_init(smem_addr(&acce_bar[b]), 2 * kHdEpiWarps);
    }
    for (int b = 0; b < 2 * kHdEpiWarps; ++b) mbar_init(smem_addr(&old_bar[b >> 1][b & 1]), 1);
    abort_flag_s = 0;
    fence_mbar_init();
  }
  for (int q = threadIdx.x; q < p.n_sup; q += blockDim.x) sup_s[q] = p.sup[q];
  // Few rows: what the loads of A leave out of its place reads as zero (the products
  // of rows that do not exist then draw little power, which the weight's stream
  // would pay for in clocks: 32 x 126464 x 4096 183 and 169 us).
  if (p.clear_a) {
    for (uint32_t i = threadIdx.x; i < static_cast<uint32_t>(p.stages) * (kHdABytes / 16); i += kHdThreads)
      asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(ring + i / (kHdABytes / 16) * p.stage_bytes + i % (kHdABytes / 16) * 16),
                   "r"(0)
                   : "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  if (warp == kHdMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&tmem_slot)),
                 "r"(kHdTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  hd_fence_before();
  __syncthreads();
  hd_cluster_sync();
  hd_fence_after();
  const uint32_t tmem = tmem_slot;
  // With one row tile the pair's first tile does not depend on the count: while the
  // rows are numbered, its weight comes to L2.
  if ((OP == kHdScore || OP == kHdDz) && p.T <= kHdBM && warp == kHdTmaWarp && lane == 0 && (blockIdx.x >> 1) < p.n_n)
    for (int x = 0; x < p.d && x < 16 * kHdBK; x += kHdBK)
      asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global [%0, {%1, %2}];" ::"l"(reinterpret_cast<uint64_t>(&p.tm_b)), "r"(x),
                   "r"(static_cast<int>(p.v0) + static_cast<int>(blockIdx.x >> 1) * p.bn + static_cast<int>(rank) * (p.bn / 2))
                   : "memory");
  pdl_wait();
  pdl_launch_dependents();
  const int64_t n = p.n_rows ? *p.n_rows : p.T;
  const HeadWork<OP> work(p, n);
  const bool packed = n != p.T;
  HeadTile t;

  if (warp == kHdTmaWarp) {
    const uint32_t lead = hd_elect(), lead0 = rank == 0 ? lead : 0u;
    const CUtensorMap* ma = OP != kHdBack && packed ? &p.tm_packed : &p.tm_a;
    const CUtensorMap* mw = packed ? &p.tm_packed : &p.tm_bw;
    const int half = p.bn / 2;
    const uint32_t leader_full = hd_leader(smem_addr(&full_bar[0]));
    int s = 0;
    uint32_t ph = 0;
    int64_t issued = 0;
    bool ok = true;
    for (int64_t it = 0; work.tile(it, t) && ok; ++it) {
      const bool dw = OP == kHdBack && t.dw;
      const int m0 = t.m * kHdBM + static_cast<int>(rank) * kHdRows, n0 = t.n * p.bn + static_cast<int>(rank) * half;
      // The second CTA's rows may all be past the end: then its A is not loaded.
      // (Of dz in two parts they are the second part.)
      const bool second = (OP == kHdBack && !dw && work.two) || static_cast<int64_t>(t.m) * kHdBM + kHdRows < (dw ? p.cols : n);
      const uint32_t tx = (second ? 2u : 1u) * (dw ? kHdABytes : p.a_bytes) + static_cast<uint32_t>(p.bn) * kHdBK * 2;
      const uint32_t lead_a = rank == 0 || second ? lead : 0u;
      for (int k = t.k0; k < t.k1; ++k) {
        ok = __all_sync(0xFFFFFFFFu, hd_wait(smem_addr(&empty_bar[s]), ph ^ 1u, abort_flag));
        if (!ok) {
          if (lane == 0) hd_fail(p, abort_flag, kFaultEmptyWait);
          break;
        }
        const uint32_t bar = leader_full + s * 8;
        const uint32_t a = ring + static_cast<uint32_t>(s) * p.stage_bytes, b = a + kHdABytes;
        hd_expect(lead0, smem_addr(&full_bar[s]), tx);
        if (dw) {
          // (dz's second part meets the same hidden states)
          const bool low = work.low > 0 && 2 * k >= t.k1;
          const int y = (low ? k - t.k1 / 2 : k) * kHdBK, yz = low ? y + work.low : y;
          hd_load(lead_a, a, &p.tm_aw, m0, yz, bar);
          hd_load(lead_a, a + 8192, &p.tm_aw, m0 + 64, yz, bar);
          hd_load(lead, b, mw, n0, y, bar);
          if (half > 64) hd_load(lead, b + 8192, mw, n0 + 64, y, bar);
        } else {
          hd_load(lead_a, a, ma, k * kHdBK, m0, bar);
          if (OP == kHdBack) {
            hd_load(lead, b, &p.tm_b, n0, static_cast<int>(p.v0) + k * kHdBK, bar);
            if (half > 64) hd_load(lead, b + 8192, &p.tm_b, n0 + 64, static_cast<int>(p.v0) + k * kHdBK, bar);
          } else {
            hd_load(lead, b, &p.tm_b, k * kHdBK, static_cast<int>(p.v0) + n0, bar);
          }
        }
        ++issued;
        if (++s == p.stages) {
          s = 0;
          ph ^= 1u;
        }
      }
    }
    // The products' last arrivals on this CTA's barriers come before it ends.
    for (int64_t q = issued > p.stages ? issued - p.stages : 0; q < issued && ok; ++q)
      ok = __all_sync(0xFFFFFFFFu, hd_wait(smem_addr(&empty_bar[q % p.stages]), static_cast<uint32_t>((q / p.stages) & 1), abort_flag));
    // Giving up: the copies still in flight land before the CTA ends.
    if (*abort_flag && rank == 0)
      for (int64_t q = issued > p.stages ? issued - p.stages : 0; q < issued; ++q)
        mbar_wait_bounded(smem_addr(&full_bar[q % p.stages]), static_cast<uint32_t>((q / p.stages) & 1));
  } else if (warp == kHdMmaWarp) {
    if (rank == 0) {
      const uint32_t lead = hd_elect();
      int s = 0, j = 0;
      uint32_t ph = 0;
      bool ok = true;
      for (int64_t it = 0; work.tile(it, t) && ok; ++it) {
        if (t.k0 == t.k1) continue;
        const bool dw = OP == kHdBack && t.dw;
        const uint32_t idesc = dw ? p.idesc_w : p.idesc, step_a = (dw ? 2048u : 32u) >> 4;
        const int part = OP != kHdBack ? hd_part(OP) : (LONG && dw ? hd_dw_part(t.k1) : t.k1 - t.k0);
        for (int k0 = t.k0; k0 < t.k1 && ok; k0 += part, ++j) {
          const int buf = j & 1;
          ok = __all_sync(0xFFFFFFFFu, hd_wait(smem_addr(&acce_bar[buf]), static_cast<uint32_t>((j >> 1) & 1) ^ 1u, abort_flag));
          if (!ok) {
            if (lane == 0) hd_fail(p, abort_flag, kFaultEmptyWait);
            break;
          }
          hd_fence_after();
          const uint32_t d_tmem = tmem + static_cast<uint32_t>(buf * kHdBN);
          for (int k = k0; k < t.k1 && k < k0 + part; ++k) {
            ok = __all_sync(0xFFFFFFFFu, hd_wait(smem_addr(&full_bar[s]), ph, abort_flag));
            if (!ok) {
              if (lane == 0) hd_fail(p, abort_flag, kFaultFullWait);
              break;
            }
            hd_fence_after();
            const uint32_t a = ring + static_cast<uint32_t>(s) * p.stage_bytes;
            const uint32_t da = hd_desc(a), db = hd_desc(a + kHdABytes);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)  // 16 k: 32 bytes of a K-major row, 16 rows of 128 bytes MN-major
              hd_mma(lead, d_tmem, da + kk * step_a, db + kk * ((OP == kHdBack ? 2048 : 32) >> 4), idesc, k != k0 || kk != 0 ? 1u : 0u);
            hd_commit(lead, smem_addr(&empty_bar[s]));
            if (++s == p.stages) {
              s = 0;
              ph ^= 1u;
            }
          }
          hd_commit(lead, smem_addr(&accf_bar[buf]));
        }
      }
    }
  } else if (warp < kHdEpiWarps) {
    const int ew = warp & 3, half = warp >> 2;
    const uint32_t lanes = tmem + (static_cast<uint32_t>(ew * 32) << 16);
    constexpr bool add16 = OP == kHdBack && OUT == kHdBf16Add;
    const uint32_t store_buf = ring + kHdRing - (kHdEpiWarps - warp) * (add16 ? 2 : 1) * kHdStoreBytes;   // (back: behind the last stage)
    uint32_t old_phase[2] = {0, 0}, old_asked = 0;
    HeadSoft soft{-kHdCap, 0.0f, 0.0f};
    int j = 0;
    // The next accumulator: warp-uniform, since the TMEM loads are .sync.aligned.
    auto await = [&] {
      const bool ok = __all_sync(0xFFFFFFFFu, hd_wait(smem_addr(&accf_bar[j & 1]), static_cast<uint32_t>((j >> 1) & 1), abort_flag));
      if (!ok && lane == 0) hd_fail(p, abort_flag, kFaultFullWait);
      hd_fence_after();
      return ok;
    };
    // It has been read.
    auto release = [&] {
      hd_fence_before();
      __syncwarp();
      if (lane == 0) hd_arrive_leader(hd_leader(smem_addr(&acce_bar[j & 1])));
      ++j;
    };
    for (int64_t it = 0; work.tile(it, t); ++it) {
      if (t.k0 == t.k1) continue;
      const bool dw = OP == kHdBack && t.dw;
      const int64_t row = static_cast<int64_t>(t.m) * kHdBM + rank * kHdRows + ew * 32 + lane;  // scored row, or (dw) id of the piece
      const int64_t col0 = static_cast<int64_t>(t.n) * p.bn;
      const int64_t width = OP != kHdBack ? p.cols : p.d;
      const int in_tile = static_cast<int>(min(static_cast<int64_t>(p.bn), width - col0));
      // Rows a warp has to visit: those that exist; of dz also the rows up to the
      // end of the third product's last slab, which read as zero.
      const int64_t visit = dw ? p.cols : (OP == kHdDz ? (n + kHdBK - 1) / kHdBK * kHdBK : (work.two ? rank * kHdRows + n : n));
      const bool warp_rows = row - lane < visit;
      if constexpr (OP != kHdBack) {
        HeadRow info{};
        int32_t target = -1;
        if (row < n) target = p.target[row];
        if (OP == kHdDz && row < n) info = p.row[row];
        if (work.n_m > 1) soft = HeadSoft{-kHdCap, 0.0f, 0.0f};
        const int end = !warp_rows ? 0 : (OP == kHdScore ? in_tile : p.bn);
        // What becomes of 32 columns of this thread's row, from column c of the tile.
        auto chunk = [&](float (&z)[32], int c) {
          const int lim = min(32, in_tile - c);
          const int64_t v = p.v0 + col0 + c;
          const uint32_t absent = lim <= 0 ? 0xFFFFFFFFu : hd_absent(sup_s, p.n_sup, v, lim);
          const int64_t hit = target - v;
          if (OP == kHdScore) {
            if (hit >= 0 && hit < 32 && row < n) {
              float zt = 0.0f;
#pragma unroll
              for (int q = 0; q < 32; ++q)
                if (q == hit) zt = z[q];
              if (hit < lim) p.z_target[row] = fminf(fmaxf(zt, -kHdCap), kHdCap);
            }
#pragma unroll
            for (int q = 0; q < 32; ++q) z[q] = fminf(fmaxf(z[q], -kHdCap), kHdCap);
            if (absent != 0u) {
#pragma unroll
              for (int q = 0; q < 32; ++q)
                if ((absent >> q) & 1u) z[q] = kHdAbsent;
            }
            float cm[4] = {-kHdCap, -kHdCap, -kHdCap, -kHdCap};
#pragma unroll
            for (int q = 0; q < 32; ++q) cm[q & 3] = fmaxf(cm[q & 3], z[q]);
            const float m = fmaxf(fmaxf(cm[0], cm[1]), fmaxf(cm[2], cm[3]));
            if (m > soft.m) hd_raise(soft, m);
            float Z[4] = {0.0f, 0.0f, 0.0f, 0.0f}, S[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int q = 0; q < 32; ++q) {
              const float y = (z[q] - soft.m) * kLog2e, e = ex2_approx(y);
              Z[q & 3] += e;
              S[q & 3] = fmaf(e, y, S[q & 3]);
            }
            soft.Z += (Z[0] + Z[1]) + (Z[2] + Z[3]);
            soft.S += (S[0] + S[1]) + (S[2] + S[3]);
          } else {
#pragma unroll
            for (int q = 0; q < 32; ++q) {
              // (a probability that small is 0; times gh the difference itself may pass fp32, and 0 inf is NaN)
              const float y = fmaxf(z[q] - info.lse, -1000.0f);
              const float e = ex2_approx(y * kLog2e);
              z[q] = -e * fmaf(info.gh, y + info.entropy, info.g);
            }
            if (hit >= 0 && hit < 32) {
#pragma unroll
              for (int q = 0; q < 32; ++q)
                if (q == hit) z[q] += info.g;
            }
            if (absent != 0u || row >= n) {
#pragma unroll
              for (int q = 0; q < 32; ++q)
                if (((absent >> q) & 1u) || row >= n) z[q] = 0.0f;
            }
            // (up to the tile's end and the row's; what is there past the piece reads as zero)
            const int room = static_cast<int>(min(static_cast<int64_t>(p.bn - c), p.dz_stride - col0 - c));
            if (row < visit) hd_store_dz(p.dz + row * p.dz_stride + col0 + c, z, room);
            if (row < visit && work.low > 0) {
#pragma unroll
              for (int q = 0; q < 32; ++q) z[q] -= __bfloat162float(__float2bfloat16_rn(z[q]));
              hd_store_dz(p.dz + (row + work.low) * p.dz_stride + col0 + c, z, room);
            }
          }
        };
        if (t.k1 <= hd_part(OP)) {
          // One part: chunk by chunk.
          if (!await()) break;
#pragma unroll 1
          for (int c = 32 * half; c < end; c += 64) {
            float z[32];
            hd_ld32(lanes + static_cast<uint32_t>((j & 1) * kHdBN + c), z);
            chunk(z, c);
          }
          release();
        } else {
          float z[4][32];
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int q = 0; q < 32; ++q) z[i][q] = 0.0f;
          bool ok = true;
          for (int k = 0; k < t.k1 && ok; k += hd_part(OP)) {
            ok = await();
            if (!ok) break;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int c = 64 * i + 32 * half;
              if (warp_rows && c < in_tile) {
#pragma unroll
                for (int h = 0; h < 32; h += 16) {
                  float r[16];
                  hd_ld16(lanes + static_cast<uint32_t>((j & 1) * kHdBN + c + h), r);
#pragma unroll
                  for (int q = 0; q < 16; ++q) z[i][h + q] += r[q];
                }
              }
            }
            release();
          }
          if (!ok) break;
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (64 * i + 32 * half < end) chunk(z[i], 64 * i + 32 * half);
        }
        // With one row tile a thread keeps its row's state from tile to tile.
        if (OP == kHdScore && row < n && (work.n_m > 1 || (it + 1) * work.pairs + work.pair >= work.total))
          p.part[((work.n_m > 1 ? t.n : work.pair) * 2 + half) * p.part_rows + row] = make_float4(soft.m, soft.Z, soft.S, 0.0f);
      } else {
        if (dw && add16 && warp_rows && lane == 0) {
          asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
#pragma unroll
          for (int b = 0; b < 2; ++b)
            if (64 * half + 128 * b < in_tile)
              hd_load_old(store_buf + b * kHdStoreBytes, &p.tm_out, static_cast<int>(col0) + 64 * half + 128 * b,
                          static_cast<int>(p.v0 + row), smem_addr(&old_bar[warp][b]));
          old_asked = 3;
        }
        // This warp's columns: 64 at 64 half, and 64 more 128 further on.
        auto col = [&](int b) { return 64 * half + 128 * b; };
        const int out_row = static_cast<int>(p.v0 + row) - lane;
        bool ok = true;
        // What becomes of 64 columns of this thread's row, 32 of them in x and in y.
        auto put = [&](const float (&x)[32], const float (&y)[32], int b) {
          const int c = col(b), at = static_cast<int>(col0) + c;
          if (dw && add16) {
            ok = ok && __all_sync(0xFFFFFFFFu, hd_wait(smem_addr(&old_bar[warp][b]), old_phase[b], abort_flag));
            if (!ok) return;
            old_phase[b] ^= 1u;
            hd_add_tile(x, y, store_buf + b * kHdStoreBytes, &p.tm_out, at, out_row, lane);
          } else if (dw && OUT == kHdBf16) {
            hd_store_tile(x, y, store_buf, &p.tm_out, at, out_row, lane);
          } else if (dw) {
            hd_store_tile_f32(x, store_buf, &p.tm_out, at, out_row, lane, p.accumulate != 0);
            if (c + 32 < in_tile) hd_store_tile_f32(y, store_buf, &p.tm_out, at + 32, out_row, lane, p.accumulate != 0);
          } else if (row < visit) {
            float* to = p.acc + (static_cast<int64_t>(t.split) * work.n_m * kHdBM + row) * p.acc_stride + col0 + c;
            hd_store_f32(to, x, min(32, in_tile - c), p.add != 0);
            hd_store_f32(to + 32, y, min(32, in_tile - c - 32), p.add != 0);
          }
        };
        const int part = LONG && dw ? hd_dw_part(t.k1) : 0;
        if (!LONG || !dw || part == t.k1) {
          // One part: 64 columns at a time, the accumulator given back before the last are stored.
          if (!await()) break;
          bool released = false;
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            if (!warp_rows || col(b) >= in_tile) break;
            float x[32], y[32];
            const uint32_t from = lanes + static_cast<uint32_t>((j & 1) * kHdBN + col(b));
            hd_ld32(from, x);
            hd_ld32(from + 32, y);
            if (b == 1 || col(1) >= in_tile) {
              release();
              released = true;
            }
            put(x, y, b);
          }
          if (!released) release();
        } else {
          float z[4][32];
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int q = 0; q < 32; ++q) z[i][q] = 0.0f;
          for (int k = t.k0; k < t.k1; k += part) {
            ok = await();
            if (!ok) break;
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (warp_rows && col(i >> 1) < in_tile) {
#pragma unroll
                for (int h = 0; h < 32; h += 16) {
                  float r[16];
                  hd_ld16(lanes + static_cast<uint32_t>((j & 1) * kHdBN + col(i >> 1) + 32 * (i & 1) + h), r);
#pragma unroll
                  for (int q = 0; q < 16; ++q) z[i][h + q] += r[q];
                }
              }
            release();
          }
          if (!ok) break;
#pragma unroll
          for (int b = 0; b < 2; ++b)
            if (warp_rows && col(b) < in_tile) put(z[2 * b], z[2 * b + 1], b);
        }
        if (!ok) {
          if (lane == 0) hd_fail(p, abort_flag, kFaultFullWait);
          break;
        }
        old_asked = 0;
      }
    }
    // Giving up: the old values still in flight land before the CTA ends.
    if (old_asked)
      for (int b = 0; b < 2; ++b) mbar_wait_bounded(smem_addr(&old_bar[warp][b]), old_phase[b]);
    if (OP == kHdBack && lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
  }
  // The third product without a scored row: the gradient is zero.
  if (OP == kHdBack && n == 0 && p.want_w && !p.accumulate) {
    const int64_t chunks = p.d / 8 * (p.grad_w_f32 ? 2 : 1);
    const int64_t stride = p.grad_w_stride * (p.grad_w_f32 ? 4 : 2);
    for (int64_t i = blockIdx.x * static_cast<int64_t>(kHdThreads) + threadIdx.x; i < p.cols * chunks;
         i += static_cast<int64_t>(gridDim.x) * kHdThreads)
      *reinterpret_cast<uint4*>(static_cast<uint8_t*>(p.grad_w) + (p.v0 + i / chunks) * stride + i % chunks * 16) =
          make_uint4(0u, 0u, 0u, 0u);
  }
  // Every product has completed (the epilogue waited for each accumulator) or
  // the CTA gave up; release the TMEM.
  hd_fence_before();
  __syncthreads();
  hd_cluster_sync();                                     // (neither CTA's memory is used by the other any more)
  if (warp == kHdMmaWarp) {
    hd_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kHdTmemCols) : "memory");
  }
}

// ---------------------------------------------------------------------------
// Numbering the scored rows
// ---------------------------------------------------------------------------
constexpr int kHdListThreads = 512;
constexpr int64_t kHdListMost = 16384;           // rows that every block counts for itself

struct HeadListParams {
  const int32_t* targets;
  int64_t T, V;
  int32_t backward;
  const float *lse, *entropy, *g, *gh;     // backward (g, gh nullable)
  int32_t n_sup;
  int32_t sup[DLLM_MAX_SUPPRESS];
  int32_t* n_rows;                         // the count, and the splits of the second product
  int32_t* rows;                           // scored row -> row
  int32_t* place;                          // backward: row -> scored row, or -1
  int32_t* target;                         // per scored row
  HeadRow* row;                            // backward: per scored row
  float *o_logprob, *o_entropy, *o_lse;    // forward: rows that are not scored get 0
  const uint16_t* hidden;
  int64_t stride, d;
  uint16_t* packed;
  int32_t n_d, bn_d, pairs, slabs;         // backward: what decides the splits
  int64_t dw_tiles;
  int32_t low;
  int64_t room;
  int32_t* counts;                         // more than kHdListMost rows: the scored rows of each block
};

// A row of the forward pass is scored when it has a target; in the backward pass
// it counts when a gradient reaches it (and its log-sum-exp is finite).  A
// suppressed target has no gradient.
__device__ __forceinline__ bool hd_row(const HeadListParams& p, int64_t t, HeadRow* out, int32_t* target) {
  const int32_t v = p.targets[t];
  *target = v;
  if (!p.backward) return v >= 0 && v < p.V;
  HeadRow r;
  r.lse = p.lse[t];
  r.entropy = p.entropy[t];
  r.g = p.g ? p.g[t] : 0.0f;
  r.gh = p.gh ? p.gh[t] : 0.0f;
  for (int q = 0; q < p.n_sup; ++q)
    if (p.sup[q] == v) r.g = 0.0f;
  *out = r;
  return v >= 0 && v < p.V && isfinite(r.lse) && (r.g != 0.0f || r.gh != 0.0f);
}

// The rows of a block: at most as many as it has threads.
__device__ __forceinline__ int64_t hd_first(int64_t T, int64_t b) { return min(T, b * ((T + gridDim.x - 1) / gridDim.x)); }

// More than kHdListMost rows: the scored rows of each block of the next kernel.
__global__ void __launch_bounds__(kHdListThreads) head_count_kernel(const __grid_constant__ HeadListParams p) {
  pdl_wait();
  pdl_launch_dependents();
  const int64_t t = hd_first(p.T, blockIdx.x) + threadIdx.x;
  HeadRow r{};
  int32_t v;
  const bool scored = t < hd_first(p.T, blockIdx.x + 1) && hd_row(p, t, &r, &v);
  const int total = __syncthreads_count(scored);
  if (threadIdx.x == 0) p.counts[blockIdx.x] = total;
}

// Numbers the scored rows in order, block by block, and gathers their hidden
// states (with rows of zeros up to the next multiple of 64, the third product's K),
// but for those when every row is scored.  Each block counts the scored rows before
// its own, and all of them, for itself.
__global__ void __launch_bounds__(kHdListThreads) head_rows_kernel(const __grid_constant__ HeadListParams p) {
  __shared__ int32_t warp_sums[kHdListThreads / 32];
  __shared__ int32_t list[kHdListThreads];
  __shared__ int32_t before_s, total_s;
  // (the products' kernel may begin: before its own wait it only sets itself up)
  pdl_launch_dependents();
  if (threadIdx.x == 0) before_s = total_s = 0;
  __syncthreads();
  pdl_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t t0 = hd_first(p.T, blockIdx.x), t1 = hd_first(p.T, blockIdx.x + 1);
  HeadRow r{};
  int32_t v, before = 0, total = 0;
  if (p.counts) {
    for (int64_t b = tid; b < gridDim.x; b += kHdListThreads) {
      const int32_t c = p.counts[b];
      total += c;
      if (b < blockIdx.x) before += c;
    }
  } else {
#pragma unroll 4
    for (int64_t t = tid; t < p.T; t += kHdListThreads) {
      const bool scored = hd_row(p, t, &r, &v);
      total += scored ? 1 : 0;
      before += scored && t < t0 ? 1 : 0;
    }
  }
  total = __reduce_add_sync(0xFFFFFFFFu, total);
  before = __reduce_add_sync(0xFFFFFFFFu, before);
  if (lane == 0) {
    atomicAdd(&total_s, total);
    atomicAdd(&before_s, before);
  }
  const int64_t t = t0 + tid;
  const bool mine = t < t1, scored = mine && hd_row(p, t, &r, &v);
  const uint32_t vote = __ballot_sync(0xFFFFFFFFu, scored);
  if (lane == 0) warp_sums[warp] = __popc(vote);
  __syncthreads();
  int32_t local = __popc(vote & ((1u << lane) - 1u)), count = 0;
  for (int w = 0; w < kHdListThreads / 32; ++w) {
    if (w < warp) local += warp_sums[w];
    count += warp_sums[w];
  }
  const int32_t first = before_s;
  const int64_t n = total_s;
  if (scored) {
    const int32_t at = first + local;
    list[local] = static_cast<int32_t>(t);
    p.rows[at] = static_cast<int32_t>(t);
    p.target[at] = v;
    if (p.backward) p.row[at] = r;
  }
  if (mine && p.backward) p.place[t] = scored ? first + local : -1;
  if (mine && !p.backward && !scored) {
    p.o_logprob[t] = 0.0f;
    p.o_entropy[t] = 0.0f;
    p.o_lse[t] = 0.0f;
  }
  if (blockIdx.x == 0 && warp == 0) {
    const int splits = p.backward ? hd_splits(n, p.n_d, p.bn_d, p.pairs, p.slabs, p.dw_tiles, p.low, p.room) : 1;
    if (lane == 0) {
      p.n_rows[0] = static_cast<int32_t>(n);
      p.n_rows[1] = splits;
    }
  }
  __syncthreads();
  if (n == p.T) return;
  const int64_t vecs = p.d / 8;
  // A unit is a row's 128 vectors, four a lane.
  const int per_row = static_cast<int>((vecs + 127) / 128);
  for (int u = warp; u < count * per_row; u += kHdListThreads / 32) {
    const int i = u / per_row;
    const int64_t q = static_cast<int64_t>(u - i * per_row) * 128 + lane;
    const uint4* from = reinterpret_cast<const uint4*>(p.hidden + list[i] * p.stride);
    uint4* to = reinterpret_cast<uint4*>(p.packed + (first + i) * p.d);
    uint4 x[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (q + 32 * e < vecs) x[e] = __ldcs(from + q + 32 * e);
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (q + 32 * e < vecs) to[q + 32 * e] = x[e];
  }
  if (blockIdx.x == 0) {
    const int64_t end = (n + kHdBK - 1) / kHdBK * kHdBK;
    for (int64_t i = n + warp; i < end; i += kHdListThreads / 32)
      for (int64_t q = lane; q < vecs; q += 32) reinterpret_cast<uint4*>(p.packed + i * p.d)[q] = make_uint4(0u, 0u, 0u, 0u);
  }
}

// ---------------------------------------------------------------------------
// The last kernels
// ---------------------------------------------------------------------------
struct HeadFinishParams {
  const int32_t *n_rows, *rows;  // null: all T rows, scored or not
  const int32_t* target;
  int64_t T, V;
  const float4* part;
  int64_t part_rows;
  int32_t parts, pairs;          // of a row: 2 for each tile along N, or for each pair where there is one row tile
  const float* z_target;
  int32_t n_sup;
  int32_t sup[DLLM_MAX_SUPPRESS];
  float ln_ids;                  // ln |A|
  float *logprob, *entropy, *lse;
};

// 8 rows a block: four lanes of each warp share a row's partials, then half a warp
// joins what they have.  (Of a size that fits an SM beside the products' kernel, so
// that it is there when that ends.)
constexpr int kHdFinishWarps = 16;

__device__ __forceinline__ HeadSoft hd_join_lane(HeadSoft a, int o) {
  hd_join(a, HeadSoft{__shfl_xor_sync(0xFFFFFFFFu, a.m, o), __shfl_xor_sync(0xFFFFFFFFu, a.Z, o), __shfl_xor_sync(0xFFFFFFFFu, a.S, o)});
  return a;
}

__global__ void __launch_bounds__(kHdFinishWarps * 32, 3) head_finish_kernel(const __grid_constant__ HeadFinishParams p) {
  __shared__ HeadSoft share[8][kHdFinishWarps + 1];
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t n = p.n_rows ? *p.n_rows : p.T;
  const int parts = n > kHdBM ? p.parts : min(p.parts, 2 * p.pairs);
  const int64_t base = blockIdx.x * static_cast<int64_t>(8);
  if (base >= n) return;
  HeadSoft a{-kHdCap, 0.0f, 0.0f};
  const int64_t mine = base + (lane & 7);
  if (mine < n)
#pragma unroll 4
    for (int q = 4 * warp + (lane >> 3); q < parts; q += 4 * kHdFinishWarps) {
      const float4 v = __ldcs(p.part + q * p.part_rows + mine);
      hd_join(a, HeadSoft{v.x, v.y, v.z});
    }
  a = hd_join_lane(hd_join_lane(a, 8), 16);
  if (lane < 8) share[lane][warp] = a;
  __syncthreads();
  if (warp >= 4) return;
  const int at = 2 * warp + (lane >> 4);
  const int64_t row = base + at;
  a = share[at][lane & 15];
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) a = hd_join_lane(a, o);
  if ((lane & 15) == 0 && row < n) {
    const float lnZ = logf(a.Z);
    const int32_t t = p.rows ? p.rows[row] : static_cast<int32_t>(row), v = p.target[row];
    if (v < 0 || v >= p.V) {
      p.logprob[t] = p.entropy[t] = p.lse[t] = 0.0f;
      return;
    }
    bool gone = false;
    for (int q = 0; q < p.n_sup; ++q) gone = gone || p.sup[q] == v;
    p.logprob[t] = gone ? -INFINITY : (p.z_target[row] - a.m) - lnZ;
    p.entropy[t] = fminf(fmaxf(fmaf(-kLn2, a.S / a.Z, lnZ), 0.0f), p.ln_ids);
    p.lse[t] = a.m >= kHdCap ? INFINITY : (a.m <= -kHdCap ? -INFINITY : a.m + lnZ);
  }
}

// grad_hidden from the second product's parts, added in a fixed order.  A block
// makes `width` columns of a row: with few splits a thread 8 of them; with many the
// warps share the splits of 256 columns at a time and meet in shared memory.  Width
// 2048, but 256 where rows are few (backward of 61 x 50257 x 768: 69 and 67 us).
constexpr int kHdJoinMany = 4;

__device__ __forceinline__ void hd_add8(float (&y)[8], const float* from) {
  const float4 a = __ldcs(reinterpret_cast<const float4*>(from)), b = __ldcs(reinterpret_cast<const float4*>(from) + 1);
  y[0] += a.x, y[1] += a.y, y[2] += a.z, y[3] += a.w;
  y[4] += b.x, y[5] += b.y, y[6] += b.z, y[7] += b.w;
}

__device__ __forceinline__ void hd_put8(uint16_t* at, const float (&y)[8]) {
  *reinterpret_cast<uint4*>(at) =
      make_uint4(hd_bf16x2(y[0], y[1]), hd_bf16x2(y[2], y[3]), hd_bf16x2(y[4], y[5]), hd_bf16x2(y[6], y[7]));
}

__global__ void __launch_bounds__(256) head_dh_kernel(const int32_t* n_rows, const int32_t* place, const float* acc,
                                                      int64_t acc_stride, int32_t width, int64_t d, uint16_t* out,
                                                      int64_t out_stride) {
  __shared__ float part[8][8][33];
  pdl_wait();
  pdl_launch_dependents();
  const int64_t n = n_rows[0], t = blockIdx.x, c0 = blockIdx.y * static_cast<int64_t>(width);
  const bool two = hd_two(n);
  const int splits = n_rows[1], lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t step = (n + kHdBM - 1) / kHdBM * kHdBM * acc_stride;
  const int32_t row = place[t];
  const float* from = acc + static_cast<int64_t>(row) * acc_stride;
  uint16_t* to = out + t * out_stride;
  if (row < 0 || splits < kHdJoinMany) {
    const int64_t c = c0 + threadIdx.x * 8;
    if (c >= d || c >= c0 + width) return;
    float y[8] = {};
    if (row >= 0)
      for (int s = 0; s < splits; ++s) {
        hd_add8(y, from + s * step + c);
        if (two) hd_add8(y, from + s * step + kHdRows * acc_stride + c);
      }
    hd_put8(to + c, y);
    return;
  }
  for (int64_t b = c0; b < d && b < c0 + width; b += 256) {
    const int64_t c = b + lane * 8;
    float y[8] = {};
    if (c < d)
#pragma unroll 4
      for (int s = warp; s < splits; s += 8) {
        hd_add8(y, from + s * step + c);
        if (two) hd_add8(y, from + s * step + kHdRows * acc_stride + c);
      }
#pragma unroll
    for (int e = 0; e < 8; ++e) part[warp][e][lane] = y[e];
    __syncthreads();
    if (warp == 0 && c < d) {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        for (int w = 1; w < 8; ++w) y[e] += part[w][e][lane];
      hd_put8(to + c, y);
    }
    __syncthreads();
  }
}

// Which wait of any call on this device ran out last.
static __device__ int32_t g_fault_word;

int32_t* fault_word() {
  static int32_t* word[64];
  static std::once_flag once[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return nullptr;
  std::call_once(once[dev], [dev]() {
    void* p = nullptr;
    if (cudaGetSymbolAddress(&p, g_fault_word) == cudaSuccess) word[dev] = static_cast<int32_t*>(p);
    else (void)cudaGetLastError();  // report through the result, leave no sticky error
  });
  return word[dev];
}

}  // namespace dllm

namespace {

using namespace dllm;

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
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

// rows x cols of bf16 or fp32 (cols contiguous) in boxes of box_rows x 128 bytes in
// the 128-byte swizzle; what lies outside reads as 0 and is not written.
bool make_map(CUtensorMap* m, const void* base, int64_t rows, int64_t cols, int64_t stride, uint32_t box_rows, bool f32 = false) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(stride) * (f32 ? 4 : 2)};
  const cuuint32_t box[2] = {f32 ? 32u : static_cast<cuuint32_t>(kHdBK), box_rows};
  const cuuint32_t estr[2] = {1, 1};
  return fn(m, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

const void* hd_back(int out, bool parts) {
  static const void* const k[3][2] = {
      {reinterpret_cast<const void*>(&head_kernel<kHdBack, kHdBf16, false>), reinterpret_cast<const void*>(&head_kernel<kHdBack, kHdBf16, true>)},
      {reinterpret_cast<const void*>(&head_kernel<kHdBack, kHdBf16Add, false>),
       reinterpret_cast<const void*>(&head_kernel<kHdBack, kHdBf16Add, true>)},
      {reinterpret_cast<const void*>(&head_kernel<kHdBack, kHdF32, false>), reinterpret_cast<const void*>(&head_kernel<kHdBack, kHdF32, true>)}};
  return k[out][parts ? 1 : 0];
}

struct HdDevice {
  int sms = 0;
  cudaError_t err = cudaSuccess;
};
HdDevice g_hd[64];
std::once_flag g_hd_once[64];

const HdDevice* hd_device() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return nullptr;
  std::call_once(g_hd_once[dev], [dev]() {
    HdDevice& d = g_hd[dev];
    d.err = cudaDeviceGetAttribute(&d.sms, cudaDevAttrMultiProcessorCount, dev);
    for (const void* k : {reinterpret_cast<const void*>(&head_kernel<kHdScore>), reinterpret_cast<const void*>(&head_kernel<kHdDz>),
                          hd_back(kHdBf16, false), hd_back(kHdBf16, true), hd_back(kHdBf16Add, false), hd_back(kHdBf16Add, true),
                          hd_back(kHdF32, false), hd_back(kHdF32, true)})
      if (d.err == cudaSuccess) d.err = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kHdSmem);
    if (d.err != cudaSuccess) (void)cudaGetLastError();  // report through the status, leave no sticky error
  });
  return g_hd[dev].err == cudaSuccess ? &g_hd[dev] : nullptr;
}

int64_t round_up(int64_t x, int64_t m) { return (x + m - 1) / m * m; }

// How a call uses its workspace, and its tiles.
struct HdPlan {
  int64_t t_pad;        // T to whole tiles
  int32_t bn_v, n_v;    // tiles along the vocabulary (a piece of it in the backward pass)
  int32_t bn_d, n_d;    // along d
  int64_t piece;        // ids of a piece
  int64_t acc;          // floats of the second product's parts
  int64_t list_blocks;  // of the kernel that numbers the rows
  size_t rows, target, place, row, z_target, hidden, part, dz, accs, counts, bytes;   // offsets, size
};

constexpr int64_t kPieceElements = int64_t{1} << 28;  // of dz: 512 MB

// The ids of a piece of dz held in `parts` parts: equal pieces of at most 2^28 elements.
int64_t hd_piece(int64_t t_pad, int64_t V, int64_t parts) {
  const int64_t most = std::max<int64_t>(4096 / parts, kPieceElements / (parts * t_pad) / kHdBN * kHdBN);
  const int64_t pieces = (V + most - 1) / most;
  return round_up((V + pieces - 1) / pieces, kHdBN);
}

// `low`: dz has a second part for every row (the workspace has room for it either way).
HdPlan hd_plan(int64_t T, int64_t V, int64_t d, int64_t sms, bool backward, bool low = false) {
  HdPlan h{};
  h.t_pad = round_up(T, kHdBM);
  const int64_t piece = !backward ? round_up(V, kHdBN) : hd_piece(h.t_pad, V, low ? 2 : 1);
  h.piece = piece;
  // One row tile: the width in [128, 256] with which the busiest pair has the fewest
  // ids (the weight's bytes are what such a call costs); else whole tiles.
  h.bn_v = kHdBN;
  if (h.t_pad == kHdBM) {
    const int64_t pairs = std::max<int64_t>(1, sms / 2);
    int64_t least = INT64_MAX;
    for (int32_t bn = kHdBN; bn >= 128; bn -= 16) {
      const int64_t cost = ((V + bn - 1) / bn + pairs - 1) / pairs * bn;
      if (cost < least) {
        least = cost;
        h.bn_v = bn;
      }
    }
  }
  h.n_v = static_cast<int32_t>((std::min(piece, V) + h.bn_v - 1) / h.bn_v);
  h.n_d = static_cast<int32_t>((d + kHdBN - 1) / kHdBN);
  h.bn_d = static_cast<int32_t>(round_up((d + h.n_d - 1) / h.n_d, 128));
  h.n_d = static_cast<int32_t>((d + h.bn_d - 1) / h.bn_d);
  const int64_t one = h.t_pad * h.n_d * h.bn_d;
  h.acc = std::max<int64_t>({one, std::min<int64_t>(8 * one, int64_t{1} << 25), sms / 2 * kHdBM * kHdBN});
  size_t at = 256;
  auto take = [&at](int64_t bytes) {
    const size_t here = at;
    at += static_cast<size_t>(round_up(bytes, 256));
    return here;
  };
  h.list_blocks = T <= kHdListMost ? std::min<int64_t>((T + 15) / 16, std::max<int64_t>(304, (T + kHdListThreads - 1) / kHdListThreads))
                                   : (T + kHdListThreads - 1) / kHdListThreads;
  h.counts = take(4 * h.list_blocks);
  h.rows = take(4 * T);
  h.target = take(4 * T);
  h.hidden = take(2 * d * round_up(T, kHdBK));
  if (backward) {
    h.place = take(4 * T);
    h.row = take(static_cast<int64_t>(sizeof(HeadRow)) * T);
    const int64_t one_part = h.t_pad * hd_piece(h.t_pad, V, 1), two_parts = T > kHdRows ? 2 * h.t_pad * hd_piece(h.t_pad, V, 2) : 0;
    h.dz = take(2 * std::max(one_part, two_parts));
    h.accs = take(4 * h.acc);
  } else {
    h.z_target = take(4 * T);
    h.part = take(static_cast<int64_t>(sizeof(float4)) * 2 * h.n_v * h.t_pad);
  }
  h.bytes = at + 240;                            // (hd_base leaves out as many at most)
  return h;
}

// Where the offsets of a plan begin: a workspace is 16-byte aligned, and dz is written
// in stores of 32 bytes.  The fault word stays the workspace's own first word.
uint8_t* hd_base(void* workspace) {
  return reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(workspace) + 255) & ~static_cast<uintptr_t>(255));
}

constexpr int64_t kHdMaxT = int64_t{1} << 24, kHdMaxD = int64_t{1} << 20;

struct HdSup {
  int32_t n = 0;
  int32_t id[DLLM_MAX_SUPPRESS];
};

// What forward and backward check alike; `sup` takes the suppressed ids, each once.
dllm_status hd_check(const void* hidden, int64_t T, int64_t d, int64_t hidden_stride, const void* weight, int64_t V,
                     int64_t weight_stride, const int32_t* targets, const int32_t* suppress_ids, int32_t n_suppress,
                     HdSup& sup) {
  if (T < 0 || V < 1 || V > INT32_MAX || d < 1) return DLLM_ERR_INVALID_ARGUMENT;
  if (hidden_stride < d || weight_stride < d) return DLLM_ERR_INVALID_ARGUMENT;
  if (mul_or_neg(mul_or_neg(T, hidden_stride), 2) < 0 || mul_or_neg(mul_or_neg(V, weight_stride), 4) < 0)
    return DLLM_ERR_INVALID_ARGUMENT;
  if (n_suppress < 0 || (n_suppress > 0 && !suppress_ids)) return DLLM_ERR_INVALID_ARGUMENT;
  if (n_suppress > DLLM_MAX_SUPPRESS) return DLLM_ERR_UNSUPPORTED;
  for (int32_t i = 0; i < n_suppress; ++i)
    if (suppress_ids[i] < 0 || suppress_ids[i] >= V) return DLLM_ERR_INVALID_ARGUMENT;
  std::copy(suppress_ids, suppress_ids + n_suppress, sup.id);
  std::sort(sup.id, sup.id + n_suppress);
  sup.n = static_cast<int32_t>(std::unique(sup.id, sup.id + n_suppress) - sup.id);
  if (sup.n >= V) return DLLM_ERR_INVALID_ARGUMENT;
  if (T == 0) return DLLM_OK;
  if (!hidden || !weight || !targets || !aligned4(targets)) return DLLM_ERR_INVALID_ARGUMENT;
  if (d % 8 != 0 || !aligned16(hidden) || !aligned16(weight) || hidden_stride % 8 != 0 || weight_stride % 8 != 0)
    return DLLM_ERR_UNSUPPORTED;
  if (T > kHdMaxT || d > kHdMaxD || hidden_stride > (int64_t{1} << 38) || weight_stride > (int64_t{1} << 38))
    return DLLM_ERR_UNSUPPORTED;
  return DLLM_OK;
}

void hd_ring(HeadParams& p, int op, int32_t a_rows, int64_t pairs) {
  p.a_bytes = static_cast<uint32_t>(a_rows) * kHdBK * 2;
  p.stage_bytes = kHdABytes + static_cast<uint32_t>(round_up(p.bn / 2 * kHdBK * 2, 1024));
  // No more stages than a pair has slabs (what few rows leave empty of each is cleared).
  const int64_t slabs = op == kHdBack ? kHdMaxStages
                                      : (round_up(p.T, kHdBM) / kHdBM * p.n_n + pairs - 1) / pairs * (round_up(p.d, kHdBK) / kHdBK);
  p.stages = std::min<int32_t>(static_cast<int32_t>(std::min<int64_t>(kHdMaxStages, slabs)), (kHdRing - (op == kHdBack ? kHdEpiWarps * kHdStoreBytes * (p.accumulate && !p.grad_w_f32 ? 2 : 1) : 0)) / static_cast<int32_t>(p.stage_bytes));
  p.clear_a = p.T <= kHdRows ? 1 : 0;
}

dllm_status hd_launch(const void* kernel, HeadParams& p, int sms, dllm_stream_t stream) {
  void* args[] = {&p};
  return launch_pdl(kernel, dim3(static_cast<unsigned>(sms / 2 * 2)), dim3(kHdThreads), kHdSmem, stream, args, 2);
}

dllm_status hd_list(HeadListParams& l, const HdPlan& h, uint8_t* ws, dllm_stream_t stream) {
  const dim3 grid(static_cast<unsigned>(h.list_blocks)), block(kHdListThreads);
  void* args[] = {&l};
  if (l.T > kHdListMost) {
    l.counts = reinterpret_cast<int32_t*>(ws + h.counts);
    const dllm_status st = launch_pdl(reinterpret_cast<const void*>(&head_count_kernel), grid, block, 0, stream, args);
    if (st != DLLM_OK) return st;
  }
  return launch_pdl(reinterpret_cast<const void*>(&head_rows_kernel), grid, block, 0, stream, args);
}

}  // namespace

extern "C" {

dllm_status dllm_fault_word(void** word) {
  if (!word) return DLLM_ERR_INVALID_ARGUMENT;
  *word = fault_word();
  return *word ? DLLM_OK : DLLM_ERR_CUDA;
}

size_t dllm_lm_head_logprobs_workspace_size(int64_t T, int64_t V, int64_t d) {
  if (T <= 0 || V <= 0 || d <= 0 || T > kHdMaxT || V > INT32_MAX || d > kHdMaxD) return 256;
  const HdDevice* dev = hd_device();
  return hd_plan(T, V, d, dev ? dev->sms : 152, false).bytes;
}

size_t dllm_lm_head_logprobs_backward_workspace_size(int64_t T, int64_t V, int64_t d) {
  if (T <= 0 || V <= 0 || d <= 0 || T > kHdMaxT || V > INT32_MAX || d > kHdMaxD) return 256;
  const HdDevice* dev = hd_device();
  return hd_plan(T, V, d, dev ? dev->sms : 152, true).bytes;
}

dllm_status dllm_lm_head_logprobs(const void* hidden, int64_t T, int64_t d, int64_t hidden_stride, const void* weight,
                                  int64_t V, int64_t weight_stride, const int32_t* targets, const int32_t* suppress_ids,
                                  int32_t n_suppress, float* logprob, float* entropy, float* lse, void* workspace,
                                  size_t workspace_bytes, dllm_stream_t stream) {
  HdSup sup;
  dllm_status st = hd_check(hidden, T, d, hidden_stride, weight, V, weight_stride, targets, suppress_ids, n_suppress, sup);
  if (st != DLLM_OK || T == 0) return st;
  if (!logprob || !entropy || !lse || !aligned4(logprob) || !aligned4(entropy) || !aligned4(lse)) return DLLM_ERR_INVALID_ARGUMENT;
  const size_t need = dllm_lm_head_logprobs_workspace_size(T, V, d);
  if (!workspace || workspace_bytes < need) return DLLM_ERR_WORKSPACE;
  if (!aligned16(workspace)) return DLLM_ERR_INVALID_ARGUMENT;
  if (overlapping({extent(logprob, 1, T, T, 4), extent(entropy, 1, T, T, 4), extent(lse, 1, T, T, 4),
                   Extent{workspace, static_cast<int64_t>(need)}},
                  {extent(hidden, T, d, hidden_stride, 2), extent(weight, V, d, weight_stride, 2), extent(targets, 1, T, T, 4)}))
    return DLLM_ERR_INVALID_ARGUMENT;
  const HdDevice* dev = hd_device();
  if (!dev) return DLLM_ERR_CUDA;
  const HdPlan h = hd_plan(T, V, d, dev->sms, false);
  uint8_t* ws = hd_base(workspace);
  int32_t* n_rows = reinterpret_cast<int32_t*>(ws + 128);

  HeadListParams l{};
  l.targets = targets;
  l.T = T;
  l.V = V;
  l.n_rows = n_rows;
  l.rows = reinterpret_cast<int32_t*>(ws + h.rows);
  l.target = reinterpret_cast<int32_t*>(ws + h.target);
  l.o_logprob = logprob;
  l.o_entropy = entropy;
  l.o_lse = lse;

  HeadParams p{};
  const uint32_t a_rows = static_cast<uint32_t>(std::min<int64_t>(kHdRows, round_up(T, 8)));
  if (!make_map(&p.tm_a, hidden, T, d, hidden_stride, a_rows) ||
      !make_map(&p.tm_packed, ws + h.hidden, round_up(T, kHdBK), d, d, a_rows) ||
      !make_map(&p.tm_b, weight, V, d, weight_stride, static_cast<uint32_t>(h.bn_v / 2)))
    return DLLM_ERR_CUDA;
  p.n_rows = n_rows;
  p.T = T;
  p.V = V;
  p.cols = V;
  p.d = d;
  p.bn = h.bn_v;
  p.n_n = h.n_v;
  p.idesc = hd_idesc(false, false, h.bn_v);
  hd_ring(p, kHdScore, static_cast<int32_t>(a_rows), dev->sms / 2);
  p.target = l.target;
  p.n_sup = sup.n;
  std::copy(sup.id, sup.id + sup.n, p.sup);
  // One row tile costs the same however many of its rows are scored: they are taken as
  // they are, without the kernel that numbers them (61 x 50257 x 768: 26 and 22 us; 22.5 to
  // 24.5 from box to box).
  const bool direct = T <= kHdBM;
  if (direct) {
    p.n_rows = nullptr;
    p.target = targets;
  }
  p.part = reinterpret_cast<float4*>(ws + h.part);
  p.part_rows = h.t_pad;
  p.z_target = reinterpret_cast<float*>(ws + h.z_target);
  p.fault = static_cast<int32_t*>(workspace);
  p.seen = fault_word();
  if (!p.seen) return DLLM_ERR_CUDA;

  HeadFinishParams f{};
  f.n_rows = p.n_rows;
  f.rows = direct ? nullptr : l.rows;
  f.target = p.target;
  f.T = T;
  f.V = V;
  f.part = p.part;
  f.part_rows = h.t_pad;
  f.parts = 2 * h.n_v;
  f.pairs = dev->sms / 2;
  f.z_target = p.z_target;
  f.n_sup = p.n_sup;
  std::copy(sup.id, sup.id + sup.n, f.sup);
  f.ln_ids = static_cast<float>(std::log(static_cast<double>(V - sup.n)));
  f.logprob = logprob;
  f.entropy = entropy;
  f.lse = lse;

  l.hidden = static_cast<const uint16_t*>(hidden);
  l.stride = hidden_stride;
  l.d = d;
  l.packed = reinterpret_cast<uint16_t*>(ws + h.hidden);
  if (!direct) st = hd_list(l, h, ws, stream);
  if (st != DLLM_OK) return st;
  st = hd_launch(reinterpret_cast<const void*>(&head_kernel<kHdScore>), p, dev->sms, stream);
  if (st != DLLM_OK) return st;
  void* fargs[] = {&f};
  return launch_pdl(reinterpret_cast<const void*>(&head_finish_kernel),
                    dim3(static_cast<unsigned>((T + 7) / 8)), dim3(kHdFinishWarps * 32), 0, stream, fargs);
}

dllm_status dllm_lm_head_logprobs_backward(const void* hidden, int64_t T, int64_t d, int64_t hidden_stride,
                                           const void* weight, int64_t V, int64_t weight_stride, const int32_t* targets,
                                           const int32_t* suppress_ids, int32_t n_suppress, const float* lse,
                                           const float* entropy, const float* grad_logprob, const float* grad_entropy,
                                           void* grad_hidden, int64_t grad_hidden_stride, void* grad_weight,
                                           dllm_dtype grad_weight_dt, int64_t grad_weight_stride, int32_t accumulate,
                                           void* workspace, size_t workspace_bytes, dllm_stream_t stream) {
  HdSup sup;
  dllm_status st = hd_check(hidden, T, d, hidden_stride, weight, V, weight_stride, targets, suppress_ids, n_suppress, sup);
  if (st != DLLM_OK) return st;
  if (grad_weight_dt != DLLM_F32 && grad_weight_dt != DLLM_BF16) return DLLM_ERR_INVALID_ARGUMENT;
  if (grad_hidden && (grad_hidden_stride < d || mul_or_neg(mul_or_neg(T, grad_hidden_stride), 2) < 0)) return DLLM_ERR_INVALID_ARGUMENT;
  if (grad_weight && (grad_weight_stride < d || mul_or_neg(mul_or_neg(V, grad_weight_stride), 4) < 0)) return DLLM_ERR_INVALID_ARGUMENT;
  if ((grad_hidden && (!aligned16(grad_hidden) || grad_hidden_stride % 8 != 0)) ||
      (grad_weight && (!aligned16(grad_weight) || grad_weight_stride % 8 != 0)))
    return DLLM_ERR_UNSUPPORTED;
  if (!grad_hidden && !grad_weight) return DLLM_OK;
  if (T == 0) {  // no row: the weight's gradient is zero
    const size_t size = grad_weight_dt == DLLM_F32 ? 4 : 2;
    if (!grad_weight || accumulate) return DLLM_OK;
    return cudaMemset2DAsync(grad_weight, static_cast<size_t>(grad_weight_stride) * size, 0, static_cast<size_t>(d) * size,
                             static_cast<size_t>(V), reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
               ? DLLM_OK
               : DLLM_ERR_CUDA;
  }
  if (!lse || !entropy || !aligned4(lse) || !aligned4(entropy) || !aligned4(grad_logprob) || !aligned4(grad_entropy))
    return DLLM_ERR_INVALID_ARGUMENT;
  const size_t need = dllm_lm_head_logprobs_backward_workspace_size(T, V, d);
  if (!workspace || workspace_bytes < need) return DLLM_ERR_WORKSPACE;
  if (!aligned16(workspace)) return DLLM_ERR_INVALID_ARGUMENT;
  if (overlapping({extent(grad_hidden, T, d, grad_hidden_stride, 2),
                   extent(grad_weight, V, d, grad_weight_stride, grad_weight_dt == DLLM_F32 ? 4 : 2),
                   Extent{workspace, static_cast<int64_t>(need)}},
                  {extent(hidden, T, d, hidden_stride, 2), extent(weight, V, d, weight_stride, 2), extent(targets, 1, T, T, 4),
                   extent(lse, 1, T, T, 4), extent(entropy, 1, T, T, 4), extent(grad_logprob, 1, T, T, 4),
                   extent(grad_entropy, 1, T, T, 4)}))
    return DLLM_ERR_INVALID_ARGUMENT;
  const HdDevice* dev = hd_device();
  if (!dev) return DLLM_ERR_CUDA;
  const bool low = grad_weight && grad_weight_dt == DLLM_F32 && T > kHdRows;
  const HdPlan h = hd_plan(T, V, d, dev->sms, true, low);
  uint8_t* ws = hd_base(workspace);
  int32_t* n_rows = reinterpret_cast<int32_t*>(ws + 128);

  HeadListParams l{};
  l.targets = targets;
  l.T = T;
  l.V = V;
  l.backward = 1;
  l.lse = lse;
  l.entropy = entropy;
  l.g = grad_logprob;
  l.gh = grad_entropy;
  l.n_sup = sup.n;
  std::copy(sup.id, sup.id + sup.n, l.sup);
  l.n_rows = n_rows;
  l.rows = reinterpret_cast<int32_t*>(ws + h.rows);
  l.place = reinterpret_cast<int32_t*>(ws + h.place);
  l.target = reinterpret_cast<int32_t*>(ws + h.target);
  l.row = reinterpret_cast<HeadRow*>(ws + h.row);

  HeadParams p{};
  const uint32_t a_rows = static_cast<uint32_t>(std::min<int64_t>(kHdRows, round_up(T, 8)));
  p.n_rows = n_rows;
  p.T = T;
  p.V = V;
  p.d = d;
  p.target = l.target;
  p.n_sup = l.n_sup;
  std::copy(sup.id, sup.id + sup.n, p.sup);
  p.row = l.row;
  p.dz = reinterpret_cast<uint16_t*>(ws + h.dz);
  p.low = low ? static_cast<int32_t>(h.t_pad) : 0;
  p.dz_stride = h.piece;
  p.acc = reinterpret_cast<float*>(ws + h.accs);
  p.acc_stride = static_cast<int64_t>(h.n_d) * h.bn_d;
  p.grad_w = grad_weight;
  p.grad_w_stride = grad_weight_stride;
  p.grad_w_f32 = grad_weight_dt == DLLM_F32 ? 1 : 0;
  p.accumulate = accumulate != 0 ? 1 : 0;
  p.fault = static_cast<int32_t*>(workspace);
  p.seen = fault_word();
  if (!p.seen) return DLLM_ERR_CUDA;
  HeadParams pz = p, pb = p;
  const int64_t packed_rows = round_up(T, kHdBK);
  if (!make_map(&pz.tm_a, hidden, T, d, hidden_stride, a_rows) ||
      !make_map(&pz.tm_packed, ws + h.hidden, packed_rows, d, d, a_rows) ||
      !make_map(&pz.tm_b, weight, V, d, weight_stride, static_cast<uint32_t>(h.bn_v / 2)) ||
      !make_map(&pb.tm_a, p.dz, h.t_pad, h.piece, h.piece, a_rows) || !make_map(&pb.tm_b, weight, V, d, weight_stride, 64) ||
      !make_map(&pb.tm_aw, p.dz, h.t_pad + p.low, h.piece, h.piece, 64) || !make_map(&pb.tm_bw, hidden, T, d, hidden_stride, 64) ||
      !make_map(&pb.tm_packed, ws + h.hidden, packed_rows, d, d, 64) ||
      (grad_weight && !make_map(&pb.tm_out, grad_weight, V, d, grad_weight_stride, 32, grad_weight_dt == DLLM_F32)))
    return DLLM_ERR_CUDA;
  pz.bn = h.bn_v;
  pz.idesc = hd_idesc(false, false, h.bn_v);
  pz.n_n = h.n_v;
  hd_ring(pz, kHdDz, static_cast<int32_t>(a_rows), dev->sms / 2);
  pb.bn = h.bn_d;
  pb.n_n = h.n_d;
  pb.idesc = hd_idesc(false, true, h.bn_d);
  pb.idesc_w = hd_idesc(true, true, h.bn_d);
  pb.want_h = grad_hidden ? 1 : 0;
  pb.want_w = grad_weight ? 1 : 0;
  hd_ring(pb, kHdBack, static_cast<int32_t>(a_rows), dev->sms / 2);

  l.hidden = static_cast<const uint16_t*>(hidden);
  l.stride = hidden_stride;
  l.d = d;
  l.packed = reinterpret_cast<uint16_t*>(ws + h.hidden);
  l.n_d = h.n_d;
  l.bn_d = h.bn_d;
  l.pairs = dev->sms / 2;
  l.slabs = static_cast<int32_t>((std::min(h.piece, V) + kHdBK - 1) / kHdBK);
  l.dw_tiles = grad_weight ? (std::min(h.piece, V) + kHdBM - 1) / kHdBM * h.n_d : 0;
  l.low = p.low;
  l.room = h.acc;
  st = hd_list(l, h, ws, stream);
  if (st != DLLM_OK) return st;
  const void* back = hd_back(p.grad_w_f32 ? kHdF32 : (p.accumulate ? kHdBf16Add : kHdBf16), grad_weight && (low ? 2 : 1) * T > hd_part(kHdBack) * kHdBK);
  for (int64_t v0 = 0; v0 < V; v0 += h.piece) {
    const int64_t cols = std::min(h.piece, V - v0);
    for (HeadParams* q : {&pz, &pb}) {
      q->v0 = v0;
      q->cols = cols;
      q->add = v0 > 0 ? 1 : 0;
    }
    // (to the end of the second product's last slab, where dz reads as zero)
    pz.n_n = static_cast<int32_t>((round_up(cols, kHdBK) + h.bn_v - 1) / h.bn_v);
    st = hd_launch(reinterpret_cast<const void*>(&head_kernel<kHdDz>), pz, dev->sms, stream);
    if (st == DLLM_OK) st = hd_launch(back, pb, dev->sms, stream);
    if (st != DLLM_OK) return st;
  }
  if (!grad_hidden) return DLLM_OK;
  const float* acc = p.acc;
  uint16_t* out = static_cast<uint16_t*>(grad_hidden);
  const int32_t* place = l.place;
  int64_t stride = p.acc_stride;
  int32_t width = T <= kHdRows ? 256 : 2048;
  void* args[] = {&n_rows, &place, &acc, &stride, &width, &d, &out, &grad_hidden_stride};
  return launch_pdl(reinterpret_cast<const void*>(&head_dh_kernel), dim3(static_cast<unsigned>(T), static_cast<unsigned>((d + width - 1) / width)),
                    dim3(256), 0, stream, args);
}

}  // extern "C"
