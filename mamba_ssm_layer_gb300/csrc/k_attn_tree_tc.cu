// k_attn_tree_tc.cu -- attention of a tree of drafted tokens over the paged 4-bit cache,
// the tensor-core kernel for trees whose nodes and query heads make many rows.
//
// A tile is T * 128 rows: row m = node m / G with query head m % G of the group.  Units
// (one page of one kv head for one tile) are cut into equal spans, one a CTA.  In a CTA:
//   producer   raw pages (72 * D bytes) by bulk copies into a ring
//   dequant    codes become f16 and take their scale (exactly), stored as the products'
//              128-byte swizzled operands: K [64 tokens][D], V^T [D][64 tokens].  The
//              page's orders are those of 8 x 8 matrix fragments, which stmatrix stores as
//              rows; K's channels stay in the page's order, the queries follow it.
//   products   S = Q K^T and O += P V (tcgen05), Q and P read from tensor memory
//   softmax    a thread a row: S from tensor memory, P as f16 over it, maxima and sums
//              in fp32; the reference follows the maximum once it has grown 2^8 (as in
//              the other attention kernels), so that O is rarely rescaled
// Two chains of S, softmax, P V run side by side, so that one's products run under the
// other's softmax: with T = 2 the chains are the two tiles, for which a page is converted
// once; with T = 1 they are the even and the odd pages of one tile, each with sums and
// outputs of its own, which are joined at the end.  A job is a chain's work on a page.
// A row's node is a 64-bit mask of its path; shifted to a page's tokens it says what the
// row sees there.  Values that are not finite among the nodes' own tokens are kept out of
// the products (0 * Inf) and make NaN of the rows that see them at the end.
// Tiles cut between CTAs are joined by a second kernel.
// Bound: the pipeline's pace, a page every 1400 cycles where rows are few (not the four converting
// warps' instructions alone, as six or eight of them are slower; each chain has one page's scores,
// softmax and P V under way, one after the other) and every 1900 for 256 rows (softmax); a tile's
// start and output some 11000.  16 trees of 9 to 16 nodes over 100 to 4000 tokens 36 us, two of 64 over
// 30000 76 us (0.83 PFLOP/s), a chain of 5 over 700 13.5 us.
#include <cuda_runtime.h>
#include <stdint.h>

#include "m2_attn_tree.cuh"
#include "m2_common.cuh"
#include "m2_kernels.h"
#include "m2_kv4.cuh"
#include "m2_kv4_mma.cuh"
#include "m2_tc.cuh"
#include "m2_tc_attn.cuh"
#include "m2_tree.cuh"

namespace m2 {

constexpr int kTtSoft = 8, kTtDeq = 4, kTtProducts = kTtSoft + kTtDeq, kTtCopies = kTtProducts + 1;  // warps
constexpr int kTtWarps = 14, kTtThreads = kTtWarps * 32;
// What a tile costs beside its pages, in pages (loading queries, storing outputs): the spans
// are cut by the sum.  0, 2, 5, 8: 58.7, 44.6, 37.7, 36.4 us for 16 trees of 9 to 16 nodes,
// 83, 82, 76, 76 for two of 64.
constexpr int kTtSetup = 8;

template <int D, int T>
struct TtCfg {
  static constexpr int kRows = 128 * T;
  static constexpr int kUnit = Kv4Block<D>::kBytes;
  static constexpr int kTile = 64 * D * 2;                // a K or V tile
  static constexpr int kTiles = 4;                        // of each
  static constexpr int kStages = D == 128 ? 9 : 16;       // raw pages
  static constexpr int kK = 0, kV = kTiles * kTile, kRing = 2 * kTiles * kTile;
  static constexpr int kShared = kRing + kStages * kUnit;
  // Tensor-memory columns: S 2 x 64 (P over it), O 2 x D, Q T x D / 2
  static constexpr uint32_t kTmO = 128, kTmQ = 128 + 2 * D;
  static_assert(kTmQ + T * D / 2 <= 512, "tensor memory");
  static constexpr int kRecord = 2 * kRows + kRows * D;   // floats: maxima, sums, outputs
};
struct TtShared {
  uint64_t raw_full[16], raw_empty[16], full[4], empty[4];  // raw pages; K and V tiles of a page
  uint64_t s_full[2], p_full[2];  // by chain
  uint64_t q_full, fin;
  uint64_t merge_full, merge_empty;  // T = 1: the second chain's maxima and sums
  uint64_t bad[8];        // by unit: tokens with values that are not finite
  uint8_t group[8][64];   // and their groups of 16 channels
  int32_t ok[16];         // by raw page: it is one
  int32_t seen[8];        // by unit: likewise
  float m1[128], l1[128];  // T = 1: the second chain's maxima and sums,
  uint32_t odd1[128];      // and its rows' groups that are NaN
  int32_t cta_seg[2], scan[kTtWarps], span[2], run_b, run_base;
  uint32_t tmem;
};
template <int D, int T>
constexpr int tt_smem_bytes() {
  static_assert(TtCfg<D, T>::kShared + (int)sizeof(TtShared) + 1024 <= 232448, "shared memory");
  return TtCfg<D, T>::kShared + (int)sizeof(TtShared) + 1024;
}

// Four 8 x 8 matrices of 16-bit elements from fragments to rows of 16 bytes: lane l gives row l % 8 of matrix l / 8.
__device__ __forceinline__ void stsm4(uint32_t addr, const uint32_t (&x)[4]) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(x[0]), "r"(x[1]),
               "r"(x[2]), "r"(x[3])
               : "memory");
}

__device__ __forceinline__ uint32_t tt_max2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// A run of consecutive pages of one tile: what a CTA's span consists of.
struct TtRun {
  AtrCursor cur;
  int pages, pos, left;  // of the run; the context's length; the span's units after it
  // from the tile's unit `off` on, the first kTtSetup of which are no pages
  __device__ __forceinline__ void set(const AtrArgs& a, int off, int units) {
    const int take = min(units, cur.pages + kTtSetup - off);
    left = units - take;
    cur.page = max(0, off - kTtSetup);
    pages = max(0, off + take - kTtSetup) - cur.page;
    pos = a.g.pos[cur.b];
  }
  __device__ __forceinline__ bool next(const AtrArgs& a, int rows) {
    do {
      if (left == 0) return false;
      cur.page = cur.pages - 1;
      cur.next(a, rows);
      set(a, 0, left);
    } while (pages == 0);
    return true;
  }
};
__device__ __forceinline__ int tt_units(const AtrArgs& a, int b, int rows) {
  const int n = atr_len(a.g, b);
  return n ? ((n + kPage - 1) / kPage + kTtSetup) * a.g.c.Hkv * atr_tiles(a, b, rows) : 0;
}

template <int D, int T>
__global__ void __launch_bounds__(kTtThreads, 1) attn_tree_tc_kernel(const __grid_constant__ AtrArgs a) {
  using C = TtCfg<D, T>;
  using L = Kv4Block<D>;
  constexpr int S = C::kStages, NT = C::kTiles, GW = D / 32;
  extern __shared__ uint8_t raw_smem[];
  uint8_t* smem = raw_smem + (1024 - (smem_addr(raw_smem) & 1023)) % 1024;
  TtShared* sh = reinterpret_cast<TtShared*>(smem + C::kShared);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, cta = blockIdx.x;
  const long long limit = *reinterpret_cast<volatile long long*>(&g_wait_limit);
  auto tt_wait = [&](uint64_t* bar, uint32_t parity) { return mbar_warp_wait(bar, parity, limit); };
  if (tid == 0) {
    for (int i = 0; i < S; ++i) mbar_init(&sh->raw_full[i], 1), mbar_init(&sh->raw_empty[i], kTtDeq);
    for (int i = 0; i < NT; ++i) mbar_init(&sh->full[i], kTtDeq), mbar_init(&sh->empty[i], 1);
    for (int i = 0; i < 2; ++i) mbar_init(&sh->s_full[i], 1), mbar_init(&sh->p_full[i], 4);
    mbar_init(&sh->q_full, T == 2 ? kTtSoft : 4);
    mbar_init(&sh->fin, 1);
    mbar_init(&sh->merge_full, 4), mbar_init(&sh->merge_empty, 4);
    sh->cta_seg[0] = sh->cta_seg[1] = -1;
    fence_mbar_init();
  }
  if (warp == kTtProducts) tmem_alloc(&sh->tmem, 512);
  pdl_wait();
  pdl_trigger();
  const int B = a.g.t.nseq;
  // ---- the span: prefix sums of the sequences' units (one a thread)
  static_assert(kSeqs <= kTtThreads, "a sequence a thread");
  const int mine = tid < B ? tt_units(a, tid, C::kRows) : 0;
  int pre = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, pre, o);
    if (lane >= o) pre += v;
  }
  if (lane == 31) sh->scan[warp] = pre;
  __syncthreads();
  int total = 0;
  pre -= mine;
#pragma unroll
  for (int w = 0; w < kTtWarps; ++w) {
    if (w < warp) pre += sh->scan[w];
    total += sh->scan[w];
  }
  int s0, s1;
  if (a.by_row) {  // tile cta % rows of sequence cta / rows
    const int rows = a.g.c.Hkv * a.most_tiles, b = cta / rows, row = cta - b * rows;
    if (tid == b) {
      const int tiles = atr_tiles(a, b, C::kRows), n = tiles ? mine / (a.g.c.Hkv * tiles) : 0;
      const bool in = row < a.g.c.Hkv * tiles;
      sh->span[0] = pre + (in ? row * n : 0);
      sh->span[1] = sh->span[0] + (in ? n : 0);
    }
    __syncthreads();
    s0 = sh->span[0];
    s1 = sh->span[1];
  } else {
    const int nc = min(a.nc, total), q = nc ? total / nc : 0, extra = total - q * nc;
    s0 = cta < nc ? q * cta + min(cta, extra) : total;
    s1 = cta < nc ? s0 + q + (cta < extra ? 1 : 0) : total;
  }
  if (mine && s0 < s1 && s0 >= pre && s0 < pre + mine) {
    sh->run_b = tid;
    sh->run_base = pre;
  }
  // rows of sequences that take no part
  for (int b = cta; b < B; b += gridDim.x)
    if (atr_len(a.g, b) == 0)
      for (int i = tid; i < atr_nodes(a.g, b) * (a.g.H * D / 8); i += kTtThreads) {
        const int j = i / (a.g.H * D / 8), e = i - j * (a.g.H * D / 8);
        *reinterpret_cast<uint4*>(a.g.out + (size_t)(a.g.t.cu[b] + j) * a.g.ld_o + 8 * e) = make_uint4(0u, 0u, 0u, 0u);
      }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh->tmem;
  const int units = s1 - s0;
  TtRun run;
  bool work = false;
  if (units > 0) {
    run.cur.b = sh->run_b;
    run.cur.load(a, C::kRows);
    const int all = run.cur.pages + kTtSetup;
    int in = s0 - sh->run_base;
    run.cur.hk = in / (run.cur.tiles * all);
    in -= run.cur.hk * (run.cur.tiles * all);
    run.cur.tile = in / all;
    run.set(a, in - run.cur.tile * all, units);
    work = run.pages > 0 || run.next(a, C::kRows);
  }
  if (work) {
    if (warp < kTtSoft) {
      // ------------------------------------------------ softmax and output
      // ch: the chain; x: the row of the CTA's 128 * T
      const int ch = warp >> 2, x = T == 2 ? 32 * warp + lane : 32 * (warp & 3) + lane;
      const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
      const uint32_t ts = tmem + lanes + 64 * ch, to = tmem + lanes + C::kTmO + ch * D;
      const uint32_t tq = tmem + lanes + C::kTmQ + (T == 2 ? ch * (D / 2) : 0);
      uint64_t tree[2];
      int tree_b = -1, u = 0, done = 0;  // units and runs before this one
      bool dead = false, owed = false;  // owed: a hand-over of the second chain that the first may not have taken
      do {
        const int b = run.cur.b, rows = atr_nodes(a.g, b) * a.G, first = a.g.t.cu[b];
        const int xr = run.cur.tile * C::kRows + x, node = min(xr, rows - 1) / a.G, h = min(xr, rows - 1) - node * a.G;
        const bool alive = xr < rows;
        const uint4* q = reinterpret_cast<const uint4*>(a.g.q + (size_t)(first + node) * a.g.ld_q +
                                                        (size_t)(run.cur.hk * a.G + h) * D);
        uint4 v[D / 8];  // the row, on its way while the tree is looked through
#pragma unroll
        for (int i = 0; i < D / 8; ++i) v[i] = alive ? q[i] : make_uint4(0u, 0u, 0u, 0u);
        if (b != tree_b) {
          tree_b = b;
          tree_masks(a.g.t.parent + first, atr_nodes(a.g, b), lane, tree);
        }
        const uint64_t path = tree_mask_of(tree, node);
        const uint64_t mask = alive ? path : 0ull;
        const bool some = __any_sync(0xffffffffu, mask != 0);  // else nothing of this warp is read
        float qs = 1.0f;
        if (some) {
          // magnitudes of bf16 compare as integers (of a NaN too, which makes all of the row NaN either way)
          uint32_t top2 = 0;
#pragma unroll
          for (int i = 0; i < D / 8; ++i) {
            top2 = tt_max2(tt_max2(top2, tt_max2(v[i].x & 0x7FFF7FFFu, v[i].y & 0x7FFF7FFFu)),
                           tt_max2(v[i].z & 0x7FFF7FFFu, v[i].w & 0x7FFF7FFFu));
          }
          float f;
          kv4_query_scale(__uint_as_float(max(top2 << 16, top2 & 0xFFFF0000u)), a.g.scale, f, qs);
          if (T == 2 || ch == 1) {
            // column 8g + 4h + c holds channels 16g + 4c + 2h and the next.  (Rolled, the row from L1: this code runs
            // once a tile, and fetching its instructions took longer than running it.)
#pragma unroll 1
            for (int g = 0; g < D / 32; ++g) {
              uint32_t w[16], y[16];
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const uint4 z = mask ? q[4 * g + i] : make_uint4(0u, 0u, 0u, 0u);
                w[4 * i] = z.x, w[4 * i + 1] = z.y, w[4 * i + 2] = z.z, w[4 * i + 3] = z.w;
              }
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                const uint32_t z = w[(i & 8) + 2 * (i & 3) + (i >> 2 & 1)];
                y[i] = pack_f16x2(bf16lo(z) * f, bf16hi(z) * f);
              }
              tmem_st16(tq + 16 * g, y);
            }
            tmem_st_wait();
          }
        }
        if (T == 2 || ch == 1) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh->q_full);
        }
        float m = -INFINITY, l = 0.0f;
        uint32_t odd = 0;  // groups of channels that are NaN
        const int k0 = T == 2 ? 0 : (u ^ ch) & 1;  // T = 1: the chain's first page of the run
        int last = -1;                             // and its last unit
        for (int k = k0; k < run.pages; k += T == 2 ? 1 : 2) {
          const int un = u + k, nth = T == 2 ? un : un >> 1, base = (run.cur.page + k) * kPage - run.pos;
          if (!tt_wait(&sh->s_full[ch], nth & 1)) {
            dead = true;
            break;
          }
          tc_fence_after();
          if (some) {
            float s[64];
            tmem_ld32_async(ts, s);
            tmem_ld32_async(ts + 32, s + 32);
            const bool there = sh->seen[un & 7] != 0;
            tmem_ld_wait<64>(s);
            if (base > -kPage || !there) {
              uint64_t see = base >= 0 ? mask >> base : base > -kPage ? mask << -base | ((1ull << -base) - 1) : ~0ull;
              if (!there) see = 0;
              const uint32_t lo = (uint32_t)see, hi = (uint32_t)(see >> 32);
#pragma unroll
              for (int i = 0; i < 32; ++i) {
                s[i] = lo >> i & 1u ? s[i] : -INFINITY;
                s[32 + i] = hi >> i & 1u ? s[32 + i] : -INFINITY;
              }
              for (uint64_t e = sh->bad[un & 7] & see; e; e &= e - 1) odd |= sh->group[un & 7][__ffsll((long long)e) - 1];
            }
            float mx[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
            for (int i = 4; i + 1 < 64; i += 2) mx[(i >> 1) & 3] = max3(mx[(i >> 1) & 3], s[i], s[i + 1]);
            const float mn = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * qs;  // qs > 0
            if (last < 0) {
              m = mn;
            } else {
              const bool grow = mn - m > 8.0f;
              if (__any_sync(0xffffffffu, grow)) {  // rescale what was summed so far, its products complete
                if (!tt_wait(&sh->empty[last % NT], (last / NT) & 1)) {
                  dead = true;
                  break;
                }
                tc_fence_after();
                const float f = grow ? ex2(m - mn) : 1.0f;
                if (grow) m = mn;
                l *= f;
#pragma unroll 1
                for (int i = 0; i < D; i += 16) {
                  float o[16];
                  uint32_t y[16];
                  tmem_ld16(to + i, o);
#pragma unroll
                  for (int e = 0; e < 16; ++e) y[e] = __float_as_uint(o[e] * f);
                  tmem_st16(to + i, y);
                }
              }
            }
            // P carries a factor 2^7, which keeps small ones out of f16's subnormals
            const float bias = m == -INFINITY ? 0.0f : 7.0f - m;
            const float2 c2 = make_float2(qs, qs), b2 = make_float2(bias, bias);
            float2 sum[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
#pragma unroll
            for (int i = 0; i < 64; i += 32) {
              uint32_t y[16];
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                const float2 z = ffma2(c2, make_float2(s[i + 2 * e], s[i + 2 * e + 1]), b2);
                const float2 p = make_float2(ex2(z.x), ex2(z.y));
                y[e] = pack_f16x2(p.x, p.y);
                sum[e & 1] = fadd2(sum[e & 1], p);
              }
              tmem_st16(ts + i / 2, y);
            }
            l += (sum[0].x + sum[1].x) + (sum[0].y + sum[1].y);
            tmem_st_wait();
          }
          last = un;
          tc_fence_before();
          // (the first chain has read the second's outputs of the run before, which products write over now)
          if (owed) {
            if (!tt_wait(&sh->merge_empty, (done - 1) & 1)) {
              dead = true;
              break;
            }
            owed = false;
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh->p_full[ch]);
        }
        if (dead) break;
        // ---- the tile leaves this CTA, whole or in part
        u += run.pages;
        const int seg = run.cur.seg(a);
        const bool before = run.cur.page > 0, part = before || run.cur.page + run.pages < run.cur.pages;
        // the last products; of the second chain: the run's last, behind which nothing reads the queries
        const int wait_for = T == 1 && ch == 1 ? u - 1 : last;
        if (wait_for >= 0 && !tt_wait(&sh->empty[wait_for % NT], (wait_for / NT) & 1)) {
          dead = true;
          break;
        }
        tc_fence_after();
        float f0 = 1.0f, f1 = 0.0f;  // the chains' weights
        if (T == 1) {
          if (ch == 1) {
            // The chain goes on to the next run's queries while the first one joins and stores this run.
            if (owed && !tt_wait(&sh->merge_empty, (done - 1) & 1)) {
              dead = true;
              break;
            }
            sh->m1[x] = m, sh->l1[x] = l, sh->odd1[x] = odd;
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh->merge_full);
            ++done;
            owed = true;
            continue;
          }
          if (!tt_wait(&sh->merge_full, done++ & 1)) {
            dead = true;
            break;
          }
          tc_fence_after();
          if (run.pages > 1 || last < 0) {
            const float m1 = sh->m1[x], l1 = sh->l1[x], top = fmaxf(m, m1);
            // (a chain without a page has outputs of an earlier run: they are not looked at)
            f0 = last >= 0 ? ad_weight(m, l, top) : 0.0f, f1 = ad_weight(m1, l1, top);
            l = l * f0 + l1 * f1;
            m = top;
            odd |= sh->odd1[x];
          }
        }
        const bool first_chain = T == 2 || last >= 0, second_chain = T == 1 && (run.pages > 1 || last < 0);
        if (mask == 0) l = 0.0f, m = -INFINITY;
        const float inv = l != 0.0f ? 1.0f / l : 0.0f;  // nothing seen: zeros
        float* rec = a.cta_part + (size_t)(2 * cta + (before ? 0 : 1)) * C::kRecord;
        uint16_t* out = a.g.out + (size_t)(first + node) * a.g.ld_o + (size_t)(run.cur.hk * a.G + h) * D;
        if (part && alive) rec[x] = m, rec[C::kRows + x] = l;
        if (__any_sync(0xffffffffu, alive)) {
#pragma unroll 1
          for (int i = 0; i < D; i += 16) {
            float o[16];
            if (first_chain) {
              tmem_ld16(to + i, o);
            } else {
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] = 0.0f;
            }
            if (second_chain) {
              float p[16];
              tmem_ld16(to + D + i, p);
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] = first_chain ? o[e] * f0 + p[e] * f1 : p[e] * f1;
            }
            if (mask == 0) {
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] = 0.0f;
            } else if (odd >> (i / 16) & 1u) {
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] = __int_as_float(0x7FFFFFFF);
            }
            if (!alive) {
            } else if (part) {
              float* d = rec + 2 * C::kRows + (size_t)x * D + i;
#pragma unroll
              for (int e = 0; e < 16; e += 8) {
                uint32_t y[8];
#pragma unroll
                for (int c = 0; c < 8; ++c) y[c] = __float_as_uint(o[e + c]);
                store32(reinterpret_cast<uint16_t*>(d + e), y);
              }
            } else {
#pragma unroll
              for (int e = 0; e < 16; e += 8)
                *reinterpret_cast<uint4*>(out + i + e) =
                    make_uint4(pack_bf16x2(o[e] * inv, o[e + 1] * inv), pack_bf16x2(o[e + 2] * inv, o[e + 3] * inv),
                               pack_bf16x2(o[e + 4] * inv, o[e + 5] * inv), pack_bf16x2(o[e + 6] * inv, o[e + 7] * inv));
            }
            __syncwarp();  // the next load is the whole warp's
          }
        }
        if (T == 1) {  // the second chain's maxima, sums and outputs are read
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh->merge_empty);
        }
        if (part && tid == 0) sh->cta_seg[before ? 0 : 1] = seg;
      } while (run.next(a, C::kRows));
    } else if (warp < kTtProducts) {
      // ------------------------------------------------ dequant: 16 tokens of K and of V a warp
      const int w0 = warp - kTtSoft, r = lane >> 2, c = lane & 3, mr = lane & 7, mq = lane >> 3;
      int u = 0;
      bool dead = false;
      do {
        for (int k = 0; k < run.pages; ++k, ++u) {
          const int st = u % S, kb = u % NT, page = run.cur.page + k;
          const int base = page * kPage - run.pos, left = run.cur.len - page * kPage;
          const uint8_t* raw = smem + C::kRing + st * C::kUnit;
          if (!tt_wait(&sh->raw_full[st], (u / S) & 1)) {
            dead = true;
            break;
          }
          const bool ok = sh->ok[st] != 0;
          const uint32_t there = ok ? kScaleBits : 0u;  // scales of a page that is none are 0
          uint32_t kc[2][GW], ks[2][GW / 2], vc[2][GW], vs[2][GW];
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            const int blk = w0 + kTtDeq * n;
            lds_words<GW>(raw + L::kK + (8 * blk + r) * (D / 2) + c * (D / 8), kc[n]);
            lds_words<GW / 2>(raw + L::kKs + (8 * blk + r) * (D / 16), ks[n]);
            lds_words<GW>(raw + L::kV + blk * (4 * D) + r * (D / 2) + c * (D / 8), vc[n]);
            lds_words<GW>(raw + L::kVs + (4 * blk + c) * (D / 8), vs[n]);
          }
          if (u >= NT && !tt_wait(&sh->empty[kb], (u / NT - 1) & 1)) {
            dead = true;
            break;
          }
          const bool nodes = base > -kPage;
          const uint32_t ktile = smem_addr(smem + C::kK + kb * C::kTile), vtile = smem_addr(smem + C::kV + kb * C::kTile);
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            const int blk = w0 + kTtDeq * n, t0 = 8 * blk + 2 * c;
#pragma unroll
            for (int w = 0; w < GW; ++w) {
              const uint32_t e = scales02(ks[n][w / 2], there), f = scales13(ks[n][w / 2], there);
              uint32_t x[4];
              codes4(kc[n][w], x);
#pragma unroll
              for (int i = 0; i < 4; ++i) x[i] = w & 1 ? hmul2_hi(x[i], i < 2 ? e : f) : hmul2_lo(x[i], i < 2 ? e : f);
              stsm4(ktile + sw128_chunk(64, 8 * blk + mr, 4 * w + mq), x);
            }
            uint32_t bits = there;  // slots past the last token may hold any scale: theirs become 0
            if (left < kPage) bits &= (t0 < left ? 0x7F80u : 0u) | (t0 + 1 < left ? 0x7F800000u : 0u);
#pragma unroll
            for (int w = 0; w < GW; ++w) {
              uint32_t e = scales02(vs[n][w], bits), f = scales13(vs[n][w], bits);
              if (nodes) e = kv4_finite(e), f = kv4_finite(f);
              uint32_t x[4];
              codes4(vc[n][w], x);
#pragma unroll
              for (int i = 0; i < 4; ++i) x[i] = hmul2(x[i], i < 2 ? e : f);
              stsm4(vtile + mr * 128 + ((blk ^ mr) << 4) + (4 * w + mq) * 1024, x);  // channels 8 (4w + mq) + mr
            }
          }
          if (nodes) {
            // tokens with values that are not finite, of those that hold any
#pragma unroll
            for (int n = 0; n < 2; ++n) {
              const int blk = w0 + kTtDeq * n, t0 = 8 * blk + 2 * c;
              uint32_t g0 = 0, g1 = 0;
#pragma unroll
              for (int w = 0; w < GW; ++w) {
                const uint32_t z = vs[n][w] & 0xF8F8F8F8u;
                g0 |= ((z & 0xFFu) == 0xF8u ? 1u : 0u) << (2 * w) | ((z & 0xFF00u) == 0xF800u ? 2u : 0u) << (2 * w);
                g1 |= ((z & 0xFF0000u) == 0xF80000u ? 1u : 0u) << (2 * w) | ((z & 0xFF000000u) == 0xF8000000u ? 2u : 0u) << (2 * w);
              }
              if (!ok || t0 >= left) g0 = 0;
              if (!ok || t0 + 1 >= left) g1 = 0;
              const uint32_t b0 = __ballot_sync(0xffffffffu, g0 != 0) & 15u, b1 = __ballot_sync(0xffffffffu, g1 != 0) & 15u;
              if (r == 0) sh->group[u & 7][t0] = (uint8_t)g0, sh->group[u & 7][t0 + 1] = (uint8_t)g1;
              uint32_t marks = 0;
#pragma unroll
              for (int i = 0; i < 4; ++i) marks |= (b0 >> i & 1u) << (2 * i) | (b1 >> i & 1u) << (2 * i + 1);
              if (lane == 0) reinterpret_cast<uint8_t*>(&sh->bad[u & 7])[blk] = (uint8_t)marks;
            }
          }
          if (w0 == 0 && lane == 0) sh->seen[u & 7] = ok;
          fence_proxy_async();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&sh->full[kb]);
            mbar_arrive(&sh->raw_empty[st]);
          }
        }
      } while (!dead && run.next(a, C::kRows));
    } else if (warp == kTtProducts) {
      // ------------------------------------------------ products
      // Operand addresses reach the products through uniform registers: what they are made of is
      // broadcast from a lane, which the compiler takes as uniform.
      const int leader = elect_one();
      const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
      const uint32_t k0 = __shfl_sync(0xffffffffu, smem_addr(smem + C::kK) >> 4, 0), v0 = k0 + ((C::kV - C::kK) >> 4);
      int u = 0, runs = 0;
      bool dead = false;
      // scores of job j = (unit, tile); the unit's K is there
      auto scores = [&](int j) {
        const int t = j % T, kb = j / T % NT;
        const uint32_t d = tm + 64 * (j & 1), q = tm + C::kTmQ + t * (D / 2), k = k0 + kb * (C::kTile >> 4);
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
          at_mma_ts(d, q + 8 * i, at_desc((k + (i >> 2) * (64 * 128 >> 4) + (i & 3) * 2) | (1u << 16)), tc_idesc_f16(128, 64),
                    i > 0, leader);
        at_commit(&sh->s_full[j & 1], leader);
      };
      auto there = [&](int un) { return tt_wait(&sh->full[un % NT], (un / NT) & 1); };
      do {
        const int pages = __shfl_sync(0xffffffffu, run.pages, 0), j0 = T * u, j1 = T * (u + pages);
        if (!tt_wait(&sh->q_full, runs++ & 1) || !there(u) || (T == 1 && pages > 1 && !there(u + 1))) {
          dead = true;
          break;
        }
        tc_fence_after();
        scores(j0);
        if (j0 + 1 < j1) scores(j0 + 1);
        for (int j = j0; j < j1; ++j) {
          // P V of this job, then the chain's next scores
          const int un = j / T, t = j % T, vb = un % NT, chain = j & 1;
          const bool more = j + 2 < j1;
          if (!tt_wait(&sh->p_full[chain], (T == 2 ? un : un >> 1) & 1)) {
            dead = true;
            break;
          }
          tc_fence_after();
          const uint32_t d = tm + C::kTmO + chain * D, p = tm + 64 * chain, v = v0 + vb * (C::kTile >> 4);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            at_mma_ts(d, p + 8 * i, at_desc((v + 2 * i) | (1u << 16)), tc_idesc_f16(128, D), j >= j0 + 2 || i > 0, leader);
          if (t == T - 1) at_commit(&sh->empty[vb], leader);
          if (!more) continue;
          if (t == 0) {
            if (!there((j + 2) / T)) {
              dead = true;
              break;
            }
            tc_fence_after();
          }
          scores(j + 2);
        }
        u += pages;
      } while (!dead && run.next(a, C::kRows));
      at_commit(&sh->fin, leader);  // everything issued here is done before tensor memory is freed
      __syncwarp();
      mbar_warp_wait(&sh->fin, 0, kWaitCycles);
    } else if (warp == kTtCopies) {
      // ------------------------------------------------ copies
      const uint64_t pol = a.most_tiles > 1 ? policy_evict_normal() : policy_evict_first();
      int u = 0;
      bool dead = false;
      do {
        const int32_t* table = a.g.c.table + (size_t)run.cur.b * a.g.c.ld_table + run.cur.page;
        for (int k0 = 0; k0 < run.pages && !dead; k0 += 32) {
          const int ids = k0 + lane < run.pages ? table[k0 + lane] : -1, n = min(32, run.pages - k0);
          for (int k = 0; k < n; ++k, ++u) {
            const int st = u % S, page = __shfl_sync(0xffffffffu, ids, k);
            if (u >= S && !tt_wait(&sh->raw_empty[st], (u / S - 1) & 1)) {
              dead = true;
              break;
            }
            if (lane == 0) {
              const bool in = page >= 0 && page < a.g.c.n_pages;
              sh->ok[st] = in;
              if (in) {
                mbar_arrive_expect_tx(&sh->raw_full[st], C::kUnit);
                bulk_g2s(smem + C::kRing + st * C::kUnit, a.g.c.pages + ((size_t)page * a.g.c.Hkv + run.cur.hk) * C::kUnit,
                         C::kUnit, &sh->raw_full[st], pol);
              } else {
                M2_RECORD_ARG(g_status);
                mbar_arrive(&sh->raw_full[st]);
              }
            }
            __syncwarp();
          }
        }
      } while (!dead && run.next(a, C::kRows));
      // every copy has landed before the CTA ends
      for (int i = max(0, u - S); i < u; ++i)
        if (!mbar_warp_wait(&sh->raw_full[i % S], (i / S) & 1, kWaitCycles)) break;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (tid < 2 && !a.by_row) a.cta_seg[2 * cta + tid] = sh->cta_seg[tid];
  if (warp == kTtProducts) tmem_free(tmem, 512);
}

// Tiles cut between CTAs: a warp joins a row of the tile that began in span c and goes on.
constexpr int kTtcWarps = 8;
template <int D, int T>
__global__ void __launch_bounds__(kTtcWarps * 32) attn_tree_tc_combine_kernel(const __grid_constant__ AtrArgs a) {
  using C = TtCfg<D, T>;
  pdl_wait();
  pdl_trigger();
  const int c = blockIdx.x, lane = threadIdx.x & 31, x = blockIdx.y * kTtcWarps + (threadIdx.x >> 5);
  const int seg = a.cta_seg[2 * c + 1];
  if (seg < 0) return;
  uint16_t* out = atr_out(a, seg, x, C::kRows, D);
  if (!out) return;
  int k = 1;  // parts: this span's, then those of the spans that the tile goes on through
  for (int y = c + 1; y < a.nc; y += 32) {
    const uint32_t same = __ballot_sync(0xffffffffu, y + lane < a.nc && a.cta_seg[2 * min(y + lane, a.nc - 1)] == seg);
    k += same == 0xffffffffu ? 32 : __ffs((int)~same) - 1;
    if (same != 0xffffffffu) break;
  }
  auto rec = [&](int y) { return a.cta_part + (size_t)(y == 0 ? 2 * c + 1 : 2 * (c + y)) * C::kRecord; };
  // D / 32 channels a lane
  constexpr int E = D / 32;
  float m = -INFINITY, l = 0.0f, o[E];
#pragma unroll
  for (int e = 0; e < E; ++e) o[e] = 0.0f;
  for (int y = 0; y < k; y += 4) {
    float m1[4], l1[4], v[4][E];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const float* r = rec(min(y + q, k - 1));
      m1[q] = y + q < k ? r[x] : -INFINITY, l1[q] = y + q < k ? r[C::kRows + x] : 0.0f;
      const float* d = r + 2 * C::kRows + (size_t)x * D + lane * E;
      if constexpr (E == 4) {
        const float4 z = *reinterpret_cast<const float4*>(d);
        v[q][0] = z.x, v[q][1] = z.y, v[q][2] = z.z, v[q][3] = z.w;
      } else {
        const float2 z = *reinterpret_cast<const float2*>(d);
        v[q][0] = z.x, v[q][1] = z.y;
      }
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      if (y + q >= k) break;
      const float top = fmaxf(m, m1[q]), f = ad_weight(m, l, top), w = ad_weight(m1[q], l1[q], top);
      m = top;
      l = l * f + l1[q] * w;
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] = o[e] * f + v[q][e] * w;
    }
  }
  const float inv = l != 0.0f ? 1.0f / l : 0.0f;  // nothing seen: zeros
  if constexpr (E == 4)
    *reinterpret_cast<uint2*>(out + 4 * lane) = make_uint2(pack_bf16x2(o[0] * inv, o[1] * inv), pack_bf16x2(o[2] * inv, o[3] * inv));
  else
    *reinterpret_cast<uint32_t*>(out + 2 * lane) = pack_bf16x2(o[0] * inv, o[1] * inv);
}

// ------------------------------------------------------------------ host

template <int D, int T>
static size_t tt_ws_bytes() {
  return (size_t)num_sms() * 2 * TtCfg<D, T>::kRecord * 4 + ((size_t)num_sms() * 2 * 4 + 255) / 256 * 256;
}
size_t attn_tree_tc_ws_bytes(int32_t D) { return D == 128 ? tt_ws_bytes<128, 2>() : tt_ws_bytes<64, 2>(); }

template <int D, int T>
static cudaError_t launch_tt(const AttnTreeArgs& g, cudaStream_t s) {
  using C = TtCfg<D, T>;
  static int done_mask[64] = {0};
  constexpr int smem = tt_smem_bytes<D, T>();
  AtrArgs a;
  a.g = g;
  a.G = g.H / g.c.Hkv;
  a.most_tiles = (g.most * a.G + C::kRows - 1) / C::kRows;
  const int64_t tiles = (int64_t)g.t.nseq * g.c.Hkv * a.most_tiles;
  a.by_row = atr_by_row(tiles, g.c.ld_table);
  a.nc = a.by_row ? (int)tiles : num_sms();
  a.cta_seg = static_cast<int32_t*>(g.ws);
  a.part = nullptr;
  a.cta_part = reinterpret_cast<float*>(static_cast<uint8_t*>(g.ws) + ((size_t)num_sms() * 2 * 4 + 255) / 256 * 256);
  auto kern = attn_tree_tc_kernel<D, T>;
  cudaError_t e = set_smem_once((const void*)kern, smem, done_mask);
  if (e != cudaSuccess) return e;
  trace_pre(K_ATTN_TREE, s);
  e = launch_k(kern, dim3(a.nc), dim3(kTtThreads), smem, s, true, a);
  trace_post(K_ATTN_TREE, s);
  if (e != cudaSuccess || a.by_row) return e;
  const int rows = g.most * a.G < C::kRows ? g.most * a.G : C::kRows;
  trace_pre(K_ATTN_TREE_COMBINE, s);
  e = launch_k(attn_tree_tc_combine_kernel<D, T>, dim3(a.nc, (rows + kTtcWarps - 1) / kTtcWarps), dim3(kTtcWarps * 32), 0, s,
               true, a);
  trace_post(K_ATTN_TREE_COMBINE, s);
  return e;
}

cudaError_t launch_attn_tree_tc(const AttnTreeArgs& a, cudaStream_t s) {
  const int rows = a.most * (a.H / a.c.Hkv);
  // Up to 128 rows as one tile whose pages go to two chains in turn; more as two tiles that
  // share each page.  The other way round: 36 / 42 us (16 trees of up to 64 rows), 91 / 76
  // (two of 256).
  if (a.c.D == 128) return rows <= 128 ? launch_tt<128, 1>(a, s) : launch_tt<128, 2>(a, s);
  return rows <= 128 ? launch_tt<64, 1>(a, s) : launch_tt<64, 2>(a, s);
}

int status_attn_tree_tc(int clear) { return tu_status(clear); }
cudaError_t wait_limit_attn_tree_tc(long long cycles) { return tu_set_wait_limit(cycles); }

}  // namespace m2
