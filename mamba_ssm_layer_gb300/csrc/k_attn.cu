// k_attn.cu -- causal attention of packed sequences on the tensor cores.
//
// A tile is 128 query rows: 128 / PK consecutive tokens x PK query heads that
// share a kv head (PK: the largest power of two that divides H / Hkv, or the
// smallest that covers it, with slots left empty, where that takes fewer tiles), so
// that short prompts fill it and one K/V tile serves all of them.  A CTA takes two
// neighbouring tiles of one sequence through the keys, 128 at a time:
//   S = Q K^T   (tcgen05, 128 x 128 fp32 in tensor memory)
//   P = exp2(c S - c m) as bf16, written over S; l += sum P   (one thread a row)
//   O += P V    (P read from tensor memory, V as an MN-major operand)
// m is the row's reference maximum.  It follows the running maximum only when
// that has grown by more than 2^8 in the exponential: until then P stays below
// 2^8, which bf16 and fp32 hold as well, and O needs no rescaling.  (This and two
// query tiles a CTA are known from the literature.)
// P takes V's type, since both operands of a product have one: a probability is off
// by at most 2^-8 of itself, the sum l is taken before that rounding.  It shows: rms
// error against 64 bits 0.0019 to 0.0023 of the output on the measured prompts, 0.0015
// to 0.0017 with fp32 probabilities, most of which is the output's own rounding.
// Few items over many keys are cut along the keys (SPLIT): a cluster takes an item,
// each of its CTAs a run of the blocks, and they join their maxima, sums and outputs
// through each other's shared memory.
// Otherwise CTAs are persistent: the copies and the first scores of a CTA's next item (a
// tile pair of one head group) run under the last softmax and the output of the
// current one.
// Bound: the tensor cores (8 * 128 * 128 * D operations a tile pair and key block)
// and the exponentials (one a score); while one tile's scores are in the softmax
// warps, the other tile's products run.
// Measured at 32 + 8 heads, as graph replays: one prompt of 8192 tokens, D = 128, 312
// to 356 us by run (1.76 to 1.54 PFLOP/s; the power limit sets the clock; a step of
// both tiles is 2800 cycles for 2048 of products: 1800 of softmax, 950 of them
// exponentials, which a warp alone on its quarter of the SM issues at half the rate of
// two, then the products that the next scores wait for); four chunks of 200..1000
// tokens over up to 6000, D = 64, 107 us (0.8 PFLOP/s); 16 prompts of 64..512 tokens
// 32 us, of which an item's first block and output take as long as its products.  Two
// threads a row (16 softmax warps of 104 registers) took 418 us where one took 371:
// what a warp does once a block (waits, votes, the exchange of maxima) counts twice.
//
// Roles: warps 0-3 softmax and output of tile 0, warps 4-7 of tile 1, warp 8
// issues the products, warp 9 the TMA copies, warps 10 and 11 look through the
// values of blocks that some row sees only in part.  Warps 8-11 hand registers
// to the softmax (a score row is 128 of them).
#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>
#include <type_traits>

#include "m2_common.cuh"
#include "m2_kernels.h"
#include "m2_tc.cuh"

namespace m2 {

constexpr int kAtThreads = 384;
// Registers a thread after the hand-over; launched with 168 (65536 / 384, in
// steps of 8): 2 * 216 + 72 = 3 * 168.
constexpr int kAtRegsSoftmax = 216, kAtRegsOther = 72;
constexpr int kAtRows = 128;      // query rows of a tile, keys of a block
// Up to so many tile pairs are handed out longest first; with more of them, later
// ones first (a sequence's longest) spreads the work as well.  Few pairs, by the
// blocks of the busiest CTA against the mean: four chunks over up to 6000 tokens
// (33 pairs x 8 groups) 95 to 79 sorted, 113 to 79 unsorted; one prompt of 8192
// (128 pairs) 237 to 232 both ways.  Many, sorted and unsorted, us: one prompt of
// 40000 (625 pairs) 7680 and 7670, 128 of 64..512 (666) 188 and 187, 128 of 1..1000
// (1101) 395 and 391, 100 chunks of 200..700 over up to 8000 (751) 1540 and 1540, 128
// of 30, 60 or 3000 (2014) 2200 and 1980.
constexpr int kAtSorted = 512;
constexpr int kAtItems = 4;       // items handed on ahead of their use
// Items whose marks of values are kept apart.  A softmax warp reads item i's marks
// before it takes item i + 2, so that the last item handed on by then is i + 1 +
// kAtItems; a tile that the next items leave empty holds nothing back earlier.
constexpr int kAtMarks = 8;
static_assert(kAtMarks >= kAtItems + 2, "marks are written again only after they have been read");
constexpr int kAtMaskBlocks = 4;  // key blocks that some row of the two tiles sees only in part: at most 3

template <int D>
struct AtCfg {
  static constexpr int kTile = kAtRows * D * 2;            // bytes of a Q, K or V tile
  static constexpr int kStages = D == 128 ? 5 : 10;        // K and V tiles in turn
  static constexpr int kQ = 0;
  static constexpr int kKV = 2 * kTile;
  static constexpr int kBars = kKV + kStages * kTile;
  // Tensor-memory columns: S 2 x 128 (P over it), O 2 x D.  (With D = 64 there is
  // room for P of its own, so that the next scores run under the softmax; scores are
  // then read while products run, which takes twice as long, and four chunks over
  // cached tokens took 119 us instead of 107.)
  static constexpr uint32_t kTmS = 0, kTmO = 256;
};
// What a CTA works on: the copies' thread works it out and hands it on through
// shared memory.
struct __align__(16) AtItem {
  int row_q, left;  // row of tile 0's first token; the sequence's tokens from it on
  int see;          // the last key that this token sees (of the sequence; below 0: none)
  int row_k;        // row of the sequence's first key
  int hg;           // group of PK query heads; below 0: no more items
  int n0, n1;       // key blocks of each tile
  int jm;           // first key block that some row of tile 0 sees only in part
};
struct AtBars {
  uint64_t q_full[2], q_empty[2], s_full[2], p_full[2][2], o_done[2], fin;
  uint64_t full[10], empty[10];
  uint64_t look, clean;  // a masked block's values may be looked through; they are
  uint64_t item_full[kAtItems], item_empty[kAtItems];
  AtItem item[kAtItems];
  // Keys of a masked block whose values are not finite: (item << 32) | bits, by the
  // CTA's item with keys (items without lie between at most); then the last item
  // that has such keys.
  unsigned long long bad[kAtMarks][kAtMaskBlocks * 4 + 1];
  uint32_t tmem;
};
template <int D>
constexpr int at_smem_bytes() {
  static_assert(AtCfg<D>::kBars + (int)sizeof(AtBars) + 1024 <= 232448, "shared memory");
  return AtCfg<D>::kBars + (int)sizeof(AtBars) + 1024;
}

struct AtArgs {
  uint16_t* out;
  const uint16_t* v;
  int32_t ld_o, ld_v;
  int32_t groups;   // H / slots
  int32_t slots;    // heads of a tile: PK or, if that covers H / Hkv, H / Hkv
  int32_t pk_log;
  int32_t gqa;      // H / Hkv
  float scale_log2; // scale * log2(e)
  int32_t nseq;
  int32_t items;    // tile pairs * groups
  int32_t wide;     // output rows start on 32 bytes
  int32_t sorted;   // order[] holds the pairs, most key blocks first
  int32_t split;    // CTAs of an item
  int64_t limit;    // of the pipeline's waits, SM clock cycles
  int32_t cu_q[kSeqs + 1], cu_k[kSeqs + 1];
  int32_t tile[kSeqs + 1];  // first tile pair of each sequence
  uint16_t order[kAtSorted];
};

// 32 columns of this warp's 32 lanes, without waiting.
__device__ __forceinline__ void tmem_ld32_async(uint32_t taddr, float* v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]),
        "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]), "=f"(v[16]),
        "=f"(v[17]), "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]), "=f"(v[24]),
        "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
      : "r"(taddr));
}
// The loads above have arrived; n values may be used after this.
template <int N>
__device__ __forceinline__ void tmem_ld_wait(float* v) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+f"(v[i]));  // no use moves above the wait
}
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float2 fadd2(float2 a, float2 b) {
  uint64_t d;
  asm("{\n\t.reg .b64 ra, rb;\n\tmov.b64 ra, {%1, %2};\n\tmov.b64 rb, {%3, %4};\n\tadd.rn.f32x2 %0, ra, rb;\n\t}"
      : "=l"(d)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(d));
  return r;
}

// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}
// Operands are 128-byte swizzled: Q and K K-major (leading offset unused: 1), V
// MN-major (64 channels a row, rows along the keys; the next 64 channels at the
// leading offset); 8-row atoms 1024 bytes apart (stride offset).
// The products of one tile, operand addresses in units of 16 bytes: the
// descriptors' upper words are constants, steps along K add to the lower ones.
// Every lane comes here and only the leader's product takes place: with a branch
// around them operands pass through vector registers, and a prompt of 8192 tokens
// took 370 us instead of 349.
constexpr uint32_t kDescHi = (1024 >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint64_t at_desc(uint32_t lo) { return ((uint64_t)kDescHi << 32) | lo; }
__device__ __forceinline__ void at_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, int acc, int leader) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc), "r"(leader));
}
__device__ __forceinline__ void at_mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, int acc, int leader) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(acc), "r"(leader));
}
__device__ __forceinline__ void at_commit(uint64_t* bar, int leader) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_addr(bar)),
      "r"(leader)
      : "memory");
}
template <int D>
__device__ __forceinline__ void at_issue_scores(uint32_t d, uint32_t q, uint32_t k, int leader) {
#pragma unroll
  for (int i = 0; i < D / 16; ++i) {
    const uint32_t step = (i >> 2) * (kAtRows * 128 >> 4) + (i & 3) * 2;
    at_mma(d, at_desc((q + step) | (1u << 16)), at_desc((k + step) | (1u << 16)), tc_idesc(kAtRows, kAtRows), i > 0,
           leader);
  }
}
// 64 keys of O += P V; the values' second 64 channels lie kAtRows * 128 bytes on.
template <int D>
__device__ __forceinline__ void at_issue_values(uint32_t d, uint32_t p, uint32_t v, bool acc, int leader) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    at_mma_ts(d, p + 8 * i, at_desc((v + i * (2048 >> 4)) | ((kAtRows * 128 >> 4) << 16)),
              tc_idesc(kAtRows, D) | (1u << 16), acc || i > 0, leader);
}

// 32 bytes, aligned: a whole sector.
__device__ __forceinline__ void store32(uint16_t* p, const uint32_t* w) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
               "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}

// A potentially blocking test, for as long as the hardware likes.  (A time asked for
// becomes sleeping in steps, which took 1 to 2% longer.)
__device__ __forceinline__ bool at_try(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_addr(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}
// mbar_wait without a call (a kernel that hands registers between its warps has to
// be one function), its limit from the launch's parameters.  The hardware may hold a
// suspended wait longer than asked, so that a short limit takes waits that only test
// (TEST), in a kernel of their own: the waits' own instructions matter.  With both
// forms in one kernel and the limit read from global memory, every case took 3 to 4%
// longer.
template <bool TEST>
__device__ __forceinline__ bool at_wait_until(uint64_t* bar, uint32_t parity, long long limit) {
  const long long t0 = clock64();
  while (!(TEST ? mbar_test_wait(bar, parity) : at_try(bar, parity))) {
    if (clock64() - t0 > limit) {
      record_timeout();
      return false;
    }
  }
  return true;
}
template <bool TEST>
__device__ __forceinline__ bool at_wait(uint64_t* bar, uint32_t parity, const AtArgs& a) {
  return mbar_test_wait(bar, parity) || at_wait_until<TEST>(bar, parity, a.limit);
}
// The same for a whole warp, which stays together.
template <bool TEST>
__device__ __forceinline__ bool at_wait_warp(uint64_t* bar, uint32_t parity, const AtArgs& a) {
  if (__all_sync(0xffffffffu, mbar_test_wait(bar, parity))) return true;
  const long long t0 = clock64();
  while (!__all_sync(0xffffffffu, TEST ? mbar_test_wait(bar, parity) : at_try(bar, parity))) {
    if (__any_sync(0xffffffffu, clock64() - t0 > a.limit)) {
      record_timeout();
      return false;
    }
  }
  return true;
}
__device__ __forceinline__ bool at_drain(uint64_t* bar, uint32_t parity) {
  return mbar_test_wait(bar, parity) || at_wait_until<false>(bar, parity, kWaitCycles);
}

// A CTA's k-th item: every other round backwards, so that each CTA gets late
// (long) and early (short) tiles alike.
template <bool SPLIT>
__device__ __forceinline__ int at_pick(int k, const AtArgs& a) {
  if (SPLIT) return k == 0 ? (int)blockIdx.x / a.split : -1;
  const int items = a.items;
  const int g = gridDim.x, id = k * g + (k & 1 ? g - 1 - (int)blockIdx.x : (int)blockIdx.x);
  return id < items ? id : -1;
}

template <bool SPLIT>
__device__ __forceinline__ AtItem at_item(const AtArgs& a, int id) {
  AtItem it;
  const int tokens = kAtRows >> a.pk_log;  // of one tile
  const int k = id / a.groups, p = a.sorted ? a.order[k] : a.tile[a.nseq] - 1 - k;
  it.hg = id % a.groups;
  int lo = 0, hi = a.nseq;  // the last sequence whose first pair is <= p
  while (hi - lo > 1) {
    const int m = (lo + hi) / 2;
    if (a.tile[m] <= p)
      lo = m;
    else
      hi = m;
  }
  const int nq = a.cu_q[lo + 1] - a.cu_q[lo], nk = a.cu_k[lo + 1] - a.cu_k[lo];
  const int q0 = (p - a.tile[lo]) * 2 * tokens;
  it.row_q = a.cu_q[lo] + q0;
  it.left = nq - q0;
  it.see = q0 + nk - nq;
  it.row_k = a.cu_k[lo];
  auto blocks = [&](int first) {
    const int last = it.see + min(first + tokens, it.left) - 1;  // the last key seen
    return first < it.left && last >= 0 ? last / kAtRows + 1 : 0;
  };
  it.n0 = blocks(0);
  it.n1 = blocks(tokens);
  if (SPLIT) {  // this CTA's run of the blocks, as if the sequence began there
    const int run = (max(it.n0, it.n1) + a.split - 1) / a.split, from = (int)blockIdx.x % a.split * run;
    it.n0 = min(max(it.n0 - from, 0), run);
    it.n1 = min(max(it.n1 - from, 0), run);
    it.see -= from * kAtRows;
    it.row_k += from * kAtRows;
  }
  it.jm = max(0, (it.see + 1) >> 7);
  return it;
}

// Two bf16 of the larger magnitudes (their signs mean nothing).
__device__ __forceinline__ void max_abs(uint32_t& a, uint32_t b) {
  asm("max.NaN.xorsign.abs.bf16x2 %0, %0, %1;" : "+r"(a) : "r"(b));
}

// Looks through row r of a value tile for numbers that are not finite: a
// probability of zero does not keep them out of the product.  They are set to
// zero in shared memory and their key is marked; rows that do see the key add
// them at the end.
template <int D>
__device__ __forceinline__ void at_clean_row(uint8_t* tile, int r, unsigned long long* bad,
                                             volatile unsigned long long* marked, uint32_t item) {
  uint32_t top[2] = {0u, 0u};  // largest magnitudes, NaN above all
#pragma unroll
  for (int c = 0; c < D / 8; ++c) {
    const uint4 w = *reinterpret_cast<const uint4*>(tile + sw128_chunk(kAtRows, r, c));
    max_abs(top[0], w.x);
    max_abs(top[1], w.y);
    max_abs(top[0], w.z);
    max_abs(top[1], w.w);
  }
  max_abs(top[0], top[1]);
  if ((top[0] & 0x7F80u) != 0x7F80u && (top[0] & 0x7F800000u) != 0x7F800000u) return;
  *marked = item;
  unsigned long long old = bad[r >> 5];
  for (;;) {
    const unsigned long long want =
        ((unsigned long long)item << 32) | (old >> 32 == item ? (uint32_t)old : 0u) | 1u << (r & 31);
    const unsigned long long seen = atomicCAS(&bad[r >> 5], old, want);
    if (seen == old) break;
    old = seen;
  }
  for (int c = 0; c < D / 8; ++c) {
    uint32_t* p = reinterpret_cast<uint32_t*>(tile + sw128_chunk(kAtRows, r, c));
    for (int i = 0; i < 4; ++i) {
      uint32_t u = p[i];
      if ((u & 0x7F80u) == 0x7F80u) u &= 0xFFFF0000u;
      if ((u & 0x7F800000u) == 0x7F800000u) u &= 0xFFFFu;
      p[i] = u;
    }
  }
}

// A consuming warp's next item; false when there is none (or a wait gave up).
template <bool TEST>
__device__ __forceinline__ bool at_next(const AtArgs& a, AtBars* bars, int pick, int lane, AtItem& it) {
  const int sl = pick % kAtItems;
  if (!at_wait_warp<TEST>(&bars->item_full[sl], (pick / kAtItems) & 1, a)) return false;
  it = bars->item[sl];
  __syncwarp();
  if (lane == 0) mbar_arrive(&bars->item_empty[sl]);
  return it.hg >= 0;
}

// The shared memory of the cluster's CTA `rank`, at this CTA's address.
__device__ __forceinline__ float cluster_ld(const float* p, int rank) {
  float v;
  asm volatile("{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %1, %2;\n\tld.shared::cluster.f32 %0, [a];\n\t}"
               : "=f"(v)
               : "r"(smem_addr(p)), "r"(rank)
               : "memory");
  return v;
}
// Every thread of every CTA of the cluster (each comes here: all waits before it are bounded).
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

template <int D, bool TEST, bool SPLIT>
__global__ void __launch_bounds__(kAtThreads, 1)
    attn_prefill_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                        const __grid_constant__ CUtensorMap tmV, const __grid_constant__ AtArgs a) {
  using C = AtCfg<D>;
  constexpr int NS = C::kStages, HALVES = D / 64, HB = kAtRows * 128;  // 64-channel halves of a tile, bytes of one
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  AtBars* bars = reinterpret_cast<AtBars*>(smem + C::kBars);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int t = 0; t < 2; ++t) {
      mbar_init(&bars->q_full[t], 1);
      mbar_init(&bars->q_empty[t], 1);
      mbar_init(&bars->s_full[t], 1);
      mbar_init(&bars->p_full[t][0], 4);
      mbar_init(&bars->p_full[t][1], 4);
      mbar_init(&bars->o_done[t], 1);
    }
    mbar_init(&bars->fin, 1);
    for (int i = 0; i < kAtItems; ++i) {
      mbar_init(&bars->item_full[i], 1);
      mbar_init(&bars->item_empty[i], 11);  // softmax, products and look-through warps
    }
    mbar_init(&bars->look, 1);
    mbar_init(&bars->clean, 2);
    for (int s = 0; s < NS; ++s) {
      mbar_init(&bars->full[s], 1);
      mbar_init(&bars->empty[s], 1);
    }
    for (int i = 0; i < kAtMarks * (kAtMaskBlocks * 4 + 1); ++i) (&bars->bad[0][0])[i] = ~0ull;
    fence_mbar_init();
  }
  if (warp == 8) tmem_alloc(&bars->tmem, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem;
  const int tokens = kAtRows >> a.pk_log;
  pdl_wait();
  pdl_trigger();
  // SPLIT: the row's maximum, sum, key blocks and output here
  float part_m = -INFINITY, part_l = 0.0f;
  int part_n = 0;
  uint16_t* part_dst = nullptr;

  // Every role walks the same items, which the copies' thread picks; a key block j of an item is copies kv + 2j
  // (K) and kv + 2j + 1 (V) of the CTA, and barrier phases are counted through.
  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kAtRegsOther));
    if (warp == 9 && lane == 0) {
      // ------------------------------------------------------ copies
      const uint64_t keep = policy_evict_normal();
      int kv = 0, nq0 = 0, nq1 = 0;  // copies and Q tiles issued
      bool dead = false;
      for (int pick = 0; !dead; ++pick) {
        const int id = at_pick<SPLIT>(pick, a), sl = pick % kAtItems;
        AtItem it;
        it.hg = -1;
        if (id >= 0) it = at_item<SPLIT>(a, id);
        if (pick >= kAtItems && !at_wait<TEST>(&bars->item_empty[sl], ((pick / kAtItems) - 1) & 1, a)) break;
        bars->item[sl] = it;
        mbar_arrive(&bars->item_full[sl]);
        if (id < 0) break;
        const int n = max(it.n0, it.n1), h0 = it.hg * a.slots, hk = h0 / a.gqa;
        auto load_q = [&](int t) {
          if (!(t ? it.n1 : it.n0) || dead) return;
          int& nq = t ? nq1 : nq0;
          if (nq > 0 && !at_wait<TEST>(&bars->q_empty[t], (nq - 1) & 1, a)) {
            dead = true;
            return;
          }
          mbar_arrive_expect_tx(&bars->q_full[t], C::kTile);
          for (int hf = 0; hf < HALVES; ++hf)
            tma_load_3d(smem + C::kQ + t * C::kTile + hf * HB, &tmQ, hf * 64, h0, it.row_q + t * tokens,
                        &bars->q_full[t], keep);
          ++nq;
        };
        for (int i = 0; i < 2 * n && !dead; ++i, ++kv) {
          const int s = kv % NS;
          if (kv >= NS && !at_wait<TEST>(&bars->empty[s], ((kv / NS) - 1) & 1, a)) {
            dead = true;
            break;
          }
          mbar_arrive_expect_tx(&bars->full[s], C::kTile);
          const CUtensorMap* m = i & 1 ? &tmV : &tmK;
          for (int hf = 0; hf < HALVES; ++hf)
            tma_load_3d(smem + C::kKV + s * C::kTile + hf * HB, m, hf * 64, hk, it.row_k + (i >> 1) * kAtRows,
                        &bars->full[s], keep);
          if (i == 0) {
            load_q(0);
            load_q(1);
          }
        }
      }
      // every copy this thread issued has landed
      if (nq0) at_drain(&bars->q_full[0], (nq0 - 1) & 1);
      if (nq1) at_drain(&bars->q_full[1], (nq1 - 1) & 1);
      for (int i = max(0, kv - NS); i < kv; ++i)
        if (!at_drain(&bars->full[i % NS], (i / NS) & 1)) break;
    } else if (warp == 8) {
      // ------------------------------------------------------ products
      // The whole warp walks the blocks, so that addresses and descriptors stay
      // warp-uniform; one elected lane issues.
      const int leader = elect_one();
      const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
      using T0 = std::integral_constant<int, 0>;
      using T1 = std::integral_constant<int, 1>;
      int nq[2] = {0, 0}, np[2] = {0, 0};  // Q and probability tiles used
      int cleaned = 0;                     // masked blocks looked through
      auto wait = [&](uint64_t* bar, uint32_t parity) { return at_wait_warp<TEST>(bar, parity, a); };
      const uint32_t q0 = (smem_addr(smem + C::kQ) & 0x3FFFFu) >> 4, kv0 = (smem_addr(smem + C::kKV) & 0x3FFFFu) >> 4;
      // S of a tile with the K tile of ring slot `sl`
      auto scores = [&](auto tile, int sl, bool last) {
        constexpr int t = decltype(tile)::value;
        at_issue_scores<D>(tm + C::kTmS + t * kAtRows, q0 + t * (C::kTile >> 4), kv0 + sl * (C::kTile >> 4), leader);
        at_commit(&bars->s_full[t], leader);
        if (last) at_commit(&bars->q_empty[t], leader);  // the tile's last scores
      };
      // O += P V of a tile with the V tile of ring slot `sl`; free: no other tile needs it, last: the tile's last block
      auto values = [&](auto tile, int sl, bool add, bool free, bool last) {
        constexpr int t = decltype(tile)::value;
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {  // the first 64 keys' probabilities come before the others'
          if (!wait(&bars->p_full[t][hf], np[t] & 1)) return false;
          tc_fence_after();
          at_issue_values<D>(tm + C::kTmO + t * D, tm + C::kTmS + t * kAtRows + 32 * hf,
                             kv0 + sl * (C::kTile >> 4) + hf * (8192 >> 4), add || hf > 0, leader);
        }
        ++np[t];
        if (free) at_commit(&bars->empty[sl], leader);
        if (last) at_commit(&bars->o_done[t], leader);
        return true;
      };
      int sl = 0, ph = 0;  // ring slot and phase of the item's next copy
      auto step = [&](int& slot, int& phase, int k) {
        slot += k;
        if (slot >= NS) slot -= NS, phase ^= 1;
      };
      bool dead = false;
      for (int pick = 0; !dead; ++pick) {
        AtItem it;
        if (!at_next<TEST>(a, bars, pick, lane, it)) break;
        // (one value of the warp, for the compiler too)
        const int n0 = __shfl_sync(0xffffffffu, it.n0, 0), n1 = __shfl_sync(0xffffffffu, it.n1, 0);
        const int jm = __shfl_sync(0xffffffffu, it.jm, 0), n = max(n0, n1);
        if (n == 0) continue;
        dead = true;  // until the item is through
        if (!wait(&bars->full[sl], ph)) break;
        if (n0) {
          if (!wait(&bars->q_full[0], nq[0]++ & 1)) break;
          scores(T0(), sl, n0 == 1);
        }
        if (n1) {
          if (!wait(&bars->q_full[1], nq[1]++ & 1)) break;
          scores(T1(), sl, n1 == 1);
        }
        at_commit(&bars->empty[sl], leader);
        if (jm == 0 && leader) mbar_arrive(&bars->look);
        int vs = sl, vph = ph, ks, kph, j = 0;  // slots of V_j and K_j+1
        step(vs, vph, 1);
        for (;; ++j) {
          if (j == n) {
            dead = false;
            break;
          }
          ks = vs, kph = vph;
          step(ks, kph, 1);
          // V_j is there, and looked through if some row must not see all of it
          if (!wait(&bars->full[vs], vph) || (j >= jm && !wait(&bars->clean, cleaned++ & 1))) break;
          const bool more = j + 1 < n, look = leader && more && j + 1 >= jm;
          if (j < n0) {
            if (!values(T0(), vs, j > 0, j >= n1, j + 1 == n0)) break;
            if (j + 1 < n0) {
              if (!wait(&bars->full[ks], kph)) break;
              scores(T0(), ks, j + 2 == n0);
              if (look) mbar_arrive(&bars->look);
            }
          }
          if (j < n1) {
            if (!values(T1(), vs, j > 0, true, j + 1 == n1)) break;
            if (j + 1 < n1) {
              if (j + 1 >= n0) {
                if (!wait(&bars->full[ks], kph)) break;
                if (look) mbar_arrive(&bars->look);
              }
              scores(T1(), ks, j + 2 == n1);
            }
          }
          if (more) at_commit(&bars->empty[ks], leader);
          vs = ks, vph = kph;
          step(vs, vph, 1);
        }
        // past the item's 2 n copies
        const int past = sl + 2 * n;
        ph ^= past / NS & 1;
        sl = past % NS;
      }
      if (leader) {
        tc_commit(&bars->fin);  // everything issued here is done before tensor memory is freed
        at_drain(&bars->fin, 0);
      }
    } else if (warp >= 10) {
      // ------------------------------------------------------ values of masked blocks
      // The products' warp calls for a block once it has issued the block's first
      // scores: only then is the phase of the values' ring slot the block's own or
      // the one before, and it stays so until the block is declared clean.
      int kv = 0, looked = 0;
      uint32_t item = 0;
      bool dead = false;
      for (int pick = 0; !dead; ++pick) {
        AtItem it;
        if (!at_next<TEST>(a, bars, pick, lane, it)) break;
        const int n = max(it.n0, it.n1);
        if (n == 0) continue;
        for (int j = it.jm; j < n; ++j) {
          const int vi = kv + 2 * j + 1;
          if (!at_wait_warp<TEST>(&bars->look, looked++ & 1, a) ||
              !at_wait_warp<TEST>(&bars->full[vi % NS], (vi / NS) & 1, a)) {
            dead = true;
            break;
          }
          for (int r = (warp - 10) * 32 + lane; r < kAtRows; r += 64)
            at_clean_row<D>(smem + C::kKV + (vi % NS) * C::kTile, r, bars->bad[item % kAtMarks] + 4 * (j - it.jm),
                            &bars->bad[item % kAtMarks][kAtMaskBlocks * 4], item);
          fence_proxy_async();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars->clean);
        }
        kv += 2 * n;
        ++item;
      }
    }
    __syncwarp();
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kAtRegsSoftmax));
    // -------------------------------------------------------- softmax and output
    const int t = warp >> 2, r = 32 * (warp & 3) + lane;
    const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
    const uint32_t ts = tmem + lanes + C::kTmS + t * kAtRows, to = tmem + lanes + C::kTmO + t * D;
    const bool pos = a.scale_log2 > 0.0f;
    const float c = pos ? a.scale_log2 : 1.0f;  // a scale <= 0 is applied to the scores first
    int ns = 0, no = 0;                         // score tiles and outputs before this item
    uint32_t item = 0;                          // items with keys before this one
    bool dead = false;
    AtItem it;
    bool more = at_next<TEST>(a, bars, 0, lane, it);
    for (int pick = 0; more; ++pick) {
      const int nt = t ? it.n1 : it.n0;
      const int tok = t * tokens + (r >> a.pk_log);
      const int limit = it.see + tok;  // the last key this row sees
      const int warp_limit = it.see + t * tokens + ((r & ~31) >> a.pk_log);  // the warp's first row
      unsigned long long* bad = bars->bad[item % kAtMarks];
      float m = -INFINITY, l = 0.0f;
      for (int j = 0; j < nt; ++j) {
        if (!at_wait_warp<TEST>(&bars->s_full[t], (ns + j) & 1, a)) {
          dead = true;
          break;
        }
        tc_fence_after();
        float s[kAtRows];
#pragma unroll
        for (int i = 0; i < 4; ++i) tmem_ld32_async(ts + 32 * i, s + 32 * i);
        tmem_ld_wait<kAtRows>(s);
        if (!pos) {
#pragma unroll
          for (int i = 0; i < kAtRows; ++i) s[i] *= a.scale_log2;
        }
        // How many of the block's keys this row sees, and the warp's first row, which sees the fewest.
        const int seen = limit - j * kAtRows + 1, least = warp_limit - j * kAtRows + 1;
        if (least < kAtRows) {
#pragma unroll
          for (int i = 0; i < kAtRows; i += 32) {
            if (least >= i + 32) continue;  // the warp's rows see all 32
            const uint32_t bits = seen >= i + 32 ? ~0u : (1u << max(seen - i, 0)) - 1u;
#pragma unroll
            for (int k = 0; k < 32; ++k) s[i + k] = bits >> k & 1u ? s[i + k] : -INFINITY;
          }
        }
        float mx[4] = {m, s[0], s[1], s[2]};
#pragma unroll
        for (int i = 3; i + 1 < kAtRows; i += 2) mx[(i >> 1) & 3] = max3(mx[(i >> 1) & 3], s[i], s[i + 1]);
        const float mn = max3(fmaxf(mx[0], s[kAtRows - 1]), mx[1], fmaxf(mx[2], mx[3]));
        if (j == 0) {
          m = mn;
        } else {
          const bool grow = (mn - m) * c > 8.0f;
          if (__any_sync(0xffffffffu, grow)) {  // rescale what was summed so far (its products are complete)
            const float f = grow ? ex2((m - mn) * c) : 1.0f;
            if (grow) m = mn;
            l *= f;
            // rolled: unrolled next to 128 scores, it spilled registers of the block loop (16 packed prompts 38 us
            // instead of 33)
#pragma unroll 1
            for (int i = 0; i < D; i += 16) {
              float o[16];
              uint32_t u[16];
              tmem_ld16(to + i, o);
#pragma unroll
              for (int k = 0; k < 16; ++k) u[k] = __float_as_uint(o[k] * f);
              tmem_st16(to + i, u);
            }
          }
        }
        const float b = m == -INFINITY ? 0.0f : -m * c;  // nothing seen yet: every exponential is 0
        const float2 c2 = make_float2(c, c), b2 = make_float2(b, b);
        float2 sum[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
        auto quarter = [&](int i) {  // 32 keys' probabilities
          uint32_t p[16];
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            const float2 z = ffma2(c2, make_float2(s[i + 2 * k], s[i + 2 * k + 1]), b2);
            s[i + 2 * k] = ex2(z.x);
            s[i + 2 * k + 1] = ex2(z.y);
            p[k] = pack_bf16x2(s[i + 2 * k], s[i + 2 * k + 1]);
          }
#pragma unroll
          for (int k = 0; k < 16; ++k) sum[k & 1] = fadd2(sum[k & 1], make_float2(s[i + 2 * k], s[i + 2 * k + 1]));
          tmem_st16(ts + i / 2, p);
        };
        auto half_done = [&](int h) {
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars->p_full[t][h]);
        };
        quarter(0);
        quarter(32);
        half_done(0);
        quarter(64);
        quarter(96);
        half_done(1);
        l += (sum[0].x + sum[1].x) + (sum[0].y + sum[1].y);
      }
      if (dead) break;
      const float inv = l != 0.0f ? 1.0f / l : 0.0f;  // nothing seen: zeros
      const int slot = r & ((1 << a.pk_log) - 1);
      const bool own = tok < it.left && slot < a.slots;  // a row of the output
      uint16_t* dst = a.out + (size_t)(it.row_q + min(tok, it.left - 1)) * a.ld_o + (size_t)(it.hg * a.slots + slot) * D;
      // The next item is taken now: behind the stores, the slot's release would wait for them.
      AtItem next;
      more = at_next<TEST>(a, bars, pick + 1, lane, next);
      if (nt > 0 && !at_wait_warp<TEST>(&bars->o_done[t], no & 1, a)) {
        dead = true;
        break;
      }
      tc_fence_after();
      if (nt > 0 && bad[kAtMaskBlocks * 4] == item) {
        // add the values that were kept out of the products, where they are seen
#pragma unroll 1
        for (int i = 0; i < D; i += 16) {
          float o[16];
          uint32_t u[16];
          tmem_ld16(to + i, o);
          for (int w = 0; w < kAtMaskBlocks * 4; ++w) {
            const int j = it.jm + (w >> 2);
            const unsigned long long e = bad[w];
            for (uint32_t bits = j < nt && (uint32_t)(e >> 32) == item ? (uint32_t)e : 0; bits; bits &= bits - 1) {
              const int key = j * kAtRows + (w & 3) * 32 + __ffs(bits) - 1;
              if (key > limit || !own) continue;
              const uint16_t* vr = a.v + (size_t)(it.row_k + key) * a.ld_v +
                                   (size_t)(it.hg * a.slots / a.gqa) * D + i;
#pragma unroll
              for (int k = 0; k < 16; ++k) {
                const float x = bf16_to_f32(vr[k]);
                if (!(fabsf(x) < INFINITY)) o[k] += x;
              }
            }
          }
          __syncwarp();
#pragma unroll
          for (int k = 0; k < 16; ++k) u[k] = __float_as_uint(o[k]);
          tmem_st16(to + i, u);
        }
        tmem_st_wait();
      }
      if constexpr (SPLIT) {
        part_m = m, part_l = l, part_n = nt;
        part_dst = own ? dst : nullptr;
      } else {
#pragma unroll 1
        for (int i = 0; i < D; i += 32) {
          float o[32];
          if (nt > 0) {
            tmem_ld32_async(to + i, o);
            tmem_ld_wait<32>(o);
          }
          uint32_t w[16];
#pragma unroll
          for (int k = 0; k < 16; ++k) w[k] = l != 0.0f ? pack_bf16x2(o[2 * k] * inv, o[2 * k + 1] * inv) : 0u;
          if (own) {
            if (a.wide) {
              store32(dst + i, w);
              store32(dst + i + 16, w + 8);
            } else {
#pragma unroll
              for (int k = 0; k < 16; k += 4)
                *reinterpret_cast<uint4*>(dst + i + 2 * k) = make_uint4(w[k], w[k + 1], w[k + 2], w[k + 3]);
            }
          }
        }
      }
      tc_fence_before();  // O is read before the next item's products, which wait for this warp's probabilities
      ns += nt;
      no += nt > 0 ? 1 : 0;
      item += max(it.n0, it.n1) > 0 ? 1 : 0;
      it = next;
    }
  }
  tc_fence_before();
  __syncthreads();
  if constexpr (SPLIT) {
    // The tiles' memory is free now: O goes there, [tile][channel][row], then maxima and sums.
    tc_fence_after();
    const int t = warp >> 2, r = 32 * (warp & 3) + lane, n = a.split, d0 = (int)blockIdx.x % n * (D / n);
    float* o_part = reinterpret_cast<float*>(smem) + t * D * kAtRows + r;
    float* m_part = reinterpret_cast<float*>(smem) + 2 * D * kAtRows + t * kAtRows + r;
    float* l_part = m_part + 2 * kAtRows;
    static_assert((2 * D + 4) * kAtRows * 4 <= C::kBars, "shared memory");
    if (warp < 8) {
      *m_part = part_m;
      *l_part = part_l;
      if (part_n > 0) {
        const uint32_t to = tmem + ((uint32_t)(32 * (warp & 3)) << 16) + C::kTmO + t * D;
#pragma unroll 1
        for (int i = 0; i < D; i += 32) {
          float o[32];
          tmem_ld32_async(to + i, o);
          tmem_ld_wait<32>(o);
#pragma unroll
          for (int k = 0; k < 32; ++k) o_part[(i + k) * kAtRows] = o[k];
        }
      }
      tc_fence_before();
    }
    __syncwarp();
    cluster_sync();
    if (warp < 8 && part_dst) {
      const float c = a.scale_log2 > 0.0f ? a.scale_log2 : 1.0f;
      float top = -INFINITY, l = 0.0f, w[8];
      for (int y = 0; y < n; ++y) top = fmaxf(top, cluster_ld(m_part, y));
      uint32_t some = 0;  // parts that saw something
#pragma unroll
      for (int y = 0; y < 8; ++y) {
        w[y] = 0.0f;
        if (y >= n) continue;
        const float m1 = cluster_ld(m_part, y), l1 = cluster_ld(l_part, y);
        if (m1 == -INFINITY && l1 == 0.0f) continue;
        some |= 1u << y;
        w[y] = m1 == -INFINITY ? 1.0f : ex2((m1 - top) * c);  // (a sum of NaN is passed on)
        l = fmaf(l1, w[y], l);
      }
      const float inv = l != 0.0f ? 1.0f / l : 0.0f;
      for (int d = d0; d < d0 + D / n; d += 8) {
        float o[8] = {};
#pragma unroll
        for (int y = 0; y < 8; ++y) {
          if (!(some >> y & 1u)) continue;
#pragma unroll
          for (int k = 0; k < 8; ++k) o[k] = fmaf(cluster_ld(o_part + (d + k) * kAtRows, y), w[y], o[k]);
        }
        *reinterpret_cast<uint4*>(part_dst + d) =
            make_uint4(pack_bf16x2(o[0] * inv, o[1] * inv), pack_bf16x2(o[2] * inv, o[3] * inv),
                       pack_bf16x2(o[4] * inv, o[5] * inv), pack_bf16x2(o[6] * inv, o[7] * inv));
      }
    }
    __syncwarp();
    cluster_sync();  // a CTA's memory stays until all have read it
  }
  if (warp == 8) {
    tc_fence_after();
    tmem_free(tmem, 512);
  }
}

// ------------------------------------------------------------------ host

// Rows of `heads` heads of D channels, as {channel, head, row}; boxes of 64
// channels x box_heads x box_rows land as 128-byte rows, swizzled.
static bool encode_heads(CUtensorMap* map, const uint16_t* base, int D, int heads, int64_t rows, int64_t ld,
                         int box_heads, int box_rows) {
  auto enc = tensor_map_encoder();
  if (!enc) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)heads, (cuuint64_t)rows};
  const cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)ld * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)box_heads, (cuuint32_t)box_rows};
  const cuuint32_t es[3] = {1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<uint16_t*>(base), dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Limit of the pipeline's waits of each device (0: the default), for later launches.
static std::atomic<long long> g_limit[64];

// CTAs of an item: a cut costs a join of about 4 key blocks, and its cluster's CTAs
// have to find room together (in 4 of 5 SMs).  Measured at 32 heads on 8 of 128, one
// sequence, cut and uncut: 16 tokens on 500 keys 10.3 and 8.0 us, 700 10.4 and 10.1,
// 1000 11.3 and 12.4, 4000 15 and 38; 64 tokens on 60000 keys 87 and 581.  (The cut
// kernel spills 124 bytes of stores and 56 of loads a thread, the others none.)
static int at_split(int items, int64_t blocks) {
  int best = 1;
  int64_t cost = blocks;
  for (int n = 2; n <= 8 && items * n <= num_sms() * 4 / 5; n *= 2) {
    const int64_t c = (blocks + n - 1) / n + 4;
    if (c < cost) best = n, cost = c;
  }
  return best;
}

template <int D, bool TEST, bool SPLIT>
static cudaError_t launch_attn_kernel(const AtArgs& a, const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
                                      cudaStream_t s) {
  static int done_mask[64] = {0};
  auto kern = attn_prefill_kernel<D, TEST, SPLIT>;
  constexpr int smem = at_smem_bytes<D>();
  cudaError_t e = set_smem_once((const void*)kern, smem, done_mask);
  if (e != cudaSuccess) return e;
  trace_pre(K_ATTN_PREFILL, s);
  if (SPLIT) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(a.items * a.split);
    cfg.blockDim = dim3(kAtThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = a.split;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    e = cudaLaunchKernelEx(&cfg, kern, q, k, v, a);
  } else {
    e = launch_k(kern, dim3(a.items < num_sms() ? a.items : num_sms()), dim3(kAtThreads), smem, s, true, q, k, v, a);
  }
  trace_post(K_ATTN_PREFILL, s);
  return e;
}

template <int D>
static cudaError_t launch_attn(const AttnArgs& g, int64_t limit, cudaStream_t s) {
  AtArgs a;
  a.limit = limit;
  a.out = g.out;
  a.v = g.v;
  a.ld_o = g.ld_o;
  a.ld_v = g.ld_v;
  a.gqa = g.H / g.Hkv;
  // Heads of a tile: the covering power of two if the dividing one makes more items
  // than there are SMs and the covering one fewer.  Measured, dividing and covering:
  // 59 sequences of 1..2 tokens, 14 heads on 2 (826 and 118 items) 20 and 6.4 us; 16 of
  // 64..512 20.2 and 19.1; but 8 of 20..60 after 500..900, 12 heads on 4 (96 and 32
  // items) 11.8 and 13.4.
  int64_t least = 0;
  for (int cover = 0; cover < 2; ++cover) {
    int log = 0;
    while (log < 7 && (cover ? (1 << log) < a.gqa : a.gqa % (2 << log) == 0)) ++log;
    const int slots = cover ? a.gqa : 1 << log, pair = 2 * (kAtRows >> log);
    if ((1 << log) < slots) continue;  // more heads than rows
    int64_t n = 0;
    for (int i = 0; i < g.nseq; ++i) n += (g.cu_q[i + 1] - g.cu_q[i] + pair - 1) / pair;
    n *= g.H / slots;
    if (cover && (least <= num_sms() || n >= least)) break;
    least = n;
    a.pk_log = log;
    a.slots = slots;
  }
  const int pk = 1 << a.pk_log, tokens = kAtRows / pk;
  a.groups = g.H / a.slots;
  a.scale_log2 = g.scale * 1.4426950408889634f;
  a.nseq = g.nseq;
  a.wide = (reinterpret_cast<uintptr_t>(g.out) & 31) == 0 && g.ld_o % 16 == 0;
  a.tile[0] = 0;
  for (int i = 0; i <= kSeqs; ++i) {
    a.cu_q[i] = g.cu_q[i];
    a.cu_k[i] = g.cu_k[i];
    if (i < kSeqs) a.tile[i + 1] = a.tile[i] + (g.cu_q[i + 1] - g.cu_q[i] + 2 * tokens - 1) / (2 * tokens);
  }
  CUtensorMap q, k, v;
  // without keys no copy of them is issued: any rows do for the maps
  const bool keys = g.Tk > 0;
  if (!encode_heads(&q, g.q, D, g.H, g.Tq, g.ld_q, pk, tokens) ||
      !encode_heads(&k, keys ? g.k : g.q, D, keys ? g.Hkv : 1, keys ? g.Tk : 1, keys ? g.ld_k : g.ld_q, 1, kAtRows) ||
      !encode_heads(&v, keys ? g.v : g.q, D, keys ? g.Hkv : 1, keys ? g.Tk : 1, keys ? g.ld_v : g.ld_q, 1, kAtRows))
    return cudaErrorInvalidValue;
  a.items = a.tile[g.nseq] * a.groups;
  a.sorted = a.tile[g.nseq] <= kAtSorted ? 1 : 0;
  int64_t longest = 0;  // key blocks of a pair
  for (int i = 0; i < g.nseq; ++i) {
    const int nq = a.cu_q[i + 1] - a.cu_q[i], nk = a.cu_k[i + 1] - a.cu_k[i];
    const int64_t n = nq > 0 ? ((int64_t)nk + kAtRows - 1) / kAtRows : 0;
    longest = n > longest ? n : longest;
  }
  const bool test = limit < 1000000;
  a.split = at_split(a.items, longest);
  if (a.sorted) {  // counting sort by key blocks (longer than the last bucket: any order)
    constexpr int kBuckets = 256;
    uint16_t first[kBuckets + 1] = {0}, len[kAtSorted];
    for (int i = 0; i < g.nseq; ++i) {
      const int nq = a.cu_q[i + 1] - a.cu_q[i], nk = a.cu_k[i + 1] - a.cu_k[i];
      for (int t = a.tile[i]; t < a.tile[i + 1]; ++t) {
        const int64_t end = (int64_t)(t - a.tile[i] + 1) * 2 * tokens;
        const int64_t last = (end < nq ? end : nq) - 1 + nk - nq, n = last < 0 ? 0 : last / kAtRows + 1;
        len[t] = (uint16_t)(kBuckets - 1 - (n < kBuckets ? n : kBuckets - 1));
        ++first[len[t] + 1];
      }
    }
    for (int b = 0; b < kBuckets; ++b) first[b + 1] += first[b];
    for (int t = 0; t < a.tile[g.nseq]; ++t) a.order[first[len[t]]++] = (uint16_t)t;
  }
  if (test)
    return a.split > 1 ? launch_attn_kernel<D, true, true>(a, q, k, v, s)
                       : launch_attn_kernel<D, true, false>(a, q, k, v, s);
  return a.split > 1 ? launch_attn_kernel<D, false, true>(a, q, k, v, s) : launch_attn_kernel<D, false, false>(a, q, k, v, s);
}

cudaError_t launch_attn_prefill(const AttnArgs& a, cudaStream_t s) {
  int dev = 0;
  cudaGetDevice(&dev);
  int64_t limit = dev >= 0 && dev < 64 ? g_limit[dev].load(std::memory_order_relaxed) : 0;
  if (limit <= 0) limit = kWaitCycles;
  return a.D == 128 ? launch_attn<128>(a, limit, s) : launch_attn<64>(a, limit, s);
}

int status_attn(int clear) { return tu_status(clear); }
cudaError_t wait_limit_attn(long long cycles) {
  int dev = 0;
  const cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess && dev >= 0 && dev < 64) g_limit[dev].store(cycles, std::memory_order_relaxed);
  return e;
}

}  // namespace m2
