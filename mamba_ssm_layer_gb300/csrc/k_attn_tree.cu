// k_attn_tree.cu -- attention of a tree of drafted tokens over the paged 4-bit cache
// (include/mamba2.h has the rule of what a node sees), for few rows: nodes x query heads
// of a kv head at most 16 (8 have a form of their own).  k_attn_tree_tc.cu serves more.
//
// A unit is half a page (32 tokens) of one kv head; row m is node m / G with query head
// m % G of the group.  The units of all sequences, in the order (sequence, kv head, page),
// are cut into equal spans, one a CTA, and each span into equal runs, one a warp, which
// streams their pages through its own ring.  What a tile costs a warp before its first page
// counts as kAtrSetup units ahead of its own.  On warp MMA:
//   S [16 x 32 tokens] = Q K^T    K codes become f16 and take their scale, exactly
//   O [16 x D] += P V             likewise V; P rounded to f16 (2^-11)
// The pages' orders of codes are those of both products' B operands, P goes from the
// first to the second in registers.  Queries are f16 rows prescaled by an exact power of
// two.  Scores, sums and outputs are fp32.  A row's node is a 64-bit mask of its path;
// shifted to a page's tokens it says what the row sees there.  Rows that a warp, then a
// CTA, holds only in part are joined: warps through shared memory, CTAs by
// attn_tree_combine.
// Bound: latency.  A page takes a warp 6400 cycles, its half pages' scores, softmax and products
// one after the other, and 1000 more pass between pages; with three warps a scheduler nothing is
// full (issue slots 44 %, DRAM 34 %, tensor 27 %).  The start until the first page takes 5 us,
// the joining 5: 64 chains of 4 over 64 to 4096 tokens 62 us (155 MB, 2.5 TB/s).
#include <cuda_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "m2_attn_tree.cuh"
#include "m2_common.cuh"
#include "m2_kernels.h"
#include "m2_kv4.cuh"
#include "m2_kv4_mma.cuh"
#include "m2_tc.cuh"
#include "m2_tree.cuh"

namespace m2 {

constexpr int kAtWarps = 12, kAtrThreads = kAtWarps * 32;

constexpr int kAtrSetup = 2;  // units (even: a page's units stay together); 0, 2, 4: 64.3, 61.7, 61.4 us for 64 sequences
constexpr int kAtrParts = 2 * kAtWarps;  // a warp leaves a first and a last part at most

// ROWS: 8 or 16 a warp.
template <int D, int ROWS>
struct AtrCfg {
  static constexpr int kBytes = Kv4Block<D>::kBytes;
  static constexpr int kStages = D == 128 ? 2 : 4;  // 12 warps * stages * bytes = 216 KB
  static constexpr int kRing = kStages * kBytes;    // of one warp
  static constexpr int kStride = D + 8;             // floats between the rows of a record: no bank conflicts
  static constexpr int kRecord = 2 * ROWS + ROWS * kStride;  // maxima, sums, outputs
};
// Which row tile a partial belongs to, and whether it starts before / ends after the CTA's span.
struct AtrMeta {
  int32_t seg, before, after;
};
template <int ROWS>
struct AtrShared {
  uint16_t* out[kAtrParts][ROWS];  // where a joined row goes: the output, or the CTA's record; null: nowhere
  AtrMeta meta[kAtrParts];
  float part_m[kAtrParts][ROWS], part_l[kAtrParts][ROWS];  // maxima (then weights) and sums
  float row_l[kAtrParts][ROWS];                                // sums of the cut tiles; -1: into a record
  uint32_t row_parts[kAtrParts];
  int32_t cta_seg[2];
  int32_t scan[kAtWarps];
  int32_t run0[kAtWarps + 1], run_b[kAtWarps], run_base[kAtWarps];
};

// Tokens of a page's units h0 to h1 - 1 (of the first `left`) that hold values that are not finite, some group of them.
template <int D>
__device__ __forceinline__ uint64_t atr_bad(const uint8_t* u, int left, int h0, int h1, int lane) {
  constexpr int GW = D / 32;
  uint64_t bad = 0;
  uint32_t vs[GW];  // of token pair `lane`: bytes (even, even, odd, odd)
  lds_words<GW>(u + Kv4Block<D>::kVs + lane * (D / 8), vs);
  uint32_t even = 0, odd = 0;
#pragma unroll
  for (int w = 0; w < GW; ++w) {
    const uint32_t x = vs[w] & 0xF8F8F8F8u;  // exponents
    even |= (x & 0xFFu) == 0xF8u || (x & 0xFF00u) == 0xF800u;
    odd |= (x & 0xFF0000u) == 0xF80000u || (x & 0xFF000000u) == 0xF8000000u;
  }
  const uint32_t be = __ballot_sync(0xffffffffu, even && 2 * lane < left);
  const uint32_t bo = __ballot_sync(0xffffffffu, odd && 2 * lane + 1 < left);
  if (be | bo)
    for (int t = 16 * h0; t < 16 * h1; ++t) bad |= (uint64_t)((be >> t & 1) | (bo >> t & 1) << 1) << (2 * t);
  return bad;
}

// The running softmax of 16 rows in a warp: lane (r, c) = (lane / 4, lane % 4) owns rows r and r + 8.
template <int D>
struct AtrRows {
  uint32_t q[D / 16][4];  // A operand: rows r, r + 8; channels 16g + 4c .. + 3
  float qs[2];            // score factor (log2 units)
  float m[2], l[2];       // reference maximum; this lane's share of the sum
  uint64_t seen[2];       // the rows' paths; 0: no such row
  float o[D / 8][4];      // channels 8i + 2c, + 1 of rows r, r + 8

  // The rows of sequence b for kv head hk.  tree: the sequence's masks, worked out here while the queries are on
  // their way (again: they are another sequence's).
  __device__ __forceinline__ void start(const AtrArgs& a, int b, int hk, uint64_t (&tree)[2], bool again, int lane) {
    const int r = lane >> 2, c = lane & 3, first = a.g.t.cu[b], n = atr_nodes(a.g, b), rows = n * a.G;
    uint2 w[2][D / 16];
    int node[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int x = r + 8 * k;
      node[k] = min(x, rows - 1) / a.G;
      const uint2* q0 = reinterpret_cast<const uint2*>(a.g.q + (size_t)(first + node[k]) * a.g.ld_q +
                                                       (size_t)(hk * a.G + min(x, rows - 1) - node[k] * a.G) * D + 4 * c);
#pragma unroll
      for (int g = 0; g < D / 16; ++g) w[k][g] = x < rows ? q0[4 * g] : make_uint2(0u, 0u);
    }
    if (again) tree_masks(a.g.t.parent + first, n, lane, tree);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const uint64_t path = tree_mask_of(tree, node[k]);
      seen[k] = r + 8 * k < rows ? path : 0ull;
      float top = 0.0f;
#pragma unroll
      for (int g = 0; g < D / 16; ++g)
        top = fmaxf(top, fmaxf(fmaxf(fabsf(bf16lo(w[k][g].x)), fabsf(bf16hi(w[k][g].x))),
                               fmaxf(fabsf(bf16lo(w[k][g].y)), fabsf(bf16hi(w[k][g].y)))));
      float f;
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      kv4_query_scale(top, a.g.scale, f, qs[k]);
#pragma unroll
      for (int g = 0; g < D / 16; ++g) {
        q[g][k] = pack_f16x2(bf16lo(w[k][g].x) * f, bf16hi(w[k][g].x) * f);
        q[g][2 + k] = pack_f16x2(bf16lo(w[k][g].y) * f, bf16hi(w[k][g].y) * f);
      }
      m[k] = -INFINITY, l[k] = 0.0f;
    }
#pragma unroll
    for (int i = 0; i < D / 8; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) o[i][j] = 0.0f;
  }

  // A page in shared memory, its units h0 to h1 - 1.  base: its first token less the
  // context's length (0 or more: only nodes; -64 or less: only context); left: tokens of
  // the sequence from its first on.  (With a whole page's scores registers were spilled.)
  __device__ __forceinline__ void units(const uint8_t* u, int base, int left, int h0, int h1, int lane) {
    using L = Kv4Block<D>;
    constexpr int GW = D / 32;  // words of a lane's codes: 2 groups each
    const int r = lane >> 2, c = lane & 3;
    const bool part = base > -kPage;
    uint64_t bad = part ? atr_bad<D>(u, left, h0, h1, lane) : 0ull;
#pragma unroll 1
    for (int half = h0; half < h1; ++half) {
      float s[4][4];
#pragma unroll
      for (int nt = 0; nt < 4; nt += 2) {  // two tiles of 8 tokens in turn: a product waits for the one before it on its sums
        uint32_t k[2][GW], sc[2][GW / 2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int t = 32 * half + 8 * (nt + h) + r;
          lds_words<GW>(u + L::kK + t * (D / 2) + c * (D / 8), k[h]);
          lds_words<GW / 2>(u + L::kKs + t * (D / 16), sc[h]);
        }
#pragma unroll
        for (int w = 0; w < GW; ++w) {
          uint32_t x[2][4];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t e = scales02(sc[h][w / 2], kScaleBits), f = scales13(sc[h][w / 2], kScaleBits);
            codes4(k[h][w], x[h]);
#pragma unroll
            for (int i = 0; i < 4; ++i) x[h][i] = w & 1 ? hmul2_hi(x[h][i], i < 2 ? e : f) : hmul2_lo(x[h][i], i < 2 ? e : f);
          }
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if (w == 0)
              mma_f16_first(s[nt + h], q[0][0], q[0][1], q[0][2], q[0][3], x[h][0], x[h][1]);
            else
              mma_f16(s[nt + h], q[2 * w][0], q[2 * w][1], q[2 * w][2], q[2 * w][3], x[h][0], x[h][1]);
          }
#pragma unroll
          for (int h = 0; h < 2; ++h)
            mma_f16(s[nt + h], q[2 * w + 1][0], q[2 * w + 1][1], q[2 * w + 1][2], q[2 * w + 1][3], x[h][2], x[h][3]);
        }
      }
      if (part) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const uint64_t see = base >= 0 ? seen[k] >> base : seen[k] << -base | ((1ull << -base) - 1);
          const uint32_t bits = (uint32_t)(see >> (32 * half)) >> (2 * c);
#pragma unroll
          for (int nt = 0; nt < 4; ++nt)
#pragma unroll
            for (int j = 0; j < 2; ++j)
              if (!(bits >> (8 * nt + j) & 1u)) s[nt][2 * k + j] = -INFINITY;
        }
      }
      // softmax: P becomes the second product's A operand.  qs > 0: maxima are taken before it is applied.
      bool grow = false;
      float mx[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        mx[k] = fmaxf(s[0][2 * k], s[0][2 * k + 1]);
#pragma unroll
        for (int nt = 1; nt < 4; ++nt) mx[k] = fmaxf(mx[k], fmaxf(s[nt][2 * k], s[nt][2 * k + 1]));
        mx[k] = fmaxf(mx[k], __shfl_xor_sync(0xffffffffu, mx[k], 1));
        mx[k] = fmaxf(mx[k], __shfl_xor_sync(0xffffffffu, mx[k], 2));
        mx[k] *= qs[k];
        grow |= mx[k] - m[k] > 8.0f;
      }
      // the reference follows the maximum once it has grown 2^8: until then P (with its
      // factor 2^7, which keeps small ones out of f16's subnormals) stays below 2^15
      if (__any_sync(0xffffffffu, grow)) {
        float f[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const bool up = mx[k] - m[k] > 8.0f;
          f[k] = up ? ad_ex2(m[k] - mx[k]) : 1.0f;
          if (up) m[k] = mx[k];
          l[k] *= f[k];
        }
#pragma unroll
        for (int i = 0; i < D / 8; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) o[i][j] *= f[j >> 1];
      }
      uint32_t p[2][4];
      const float b0 = m[0] == -INFINITY ? 0.0f : 7.0f - m[0], b1 = m[1] == -INFINITY ? 0.0f : 7.0f - m[1];
#pragma unroll
      for (int nt = 0; nt < 4; ++nt) {
        const float x0 = ad_ex2(fmaf(s[nt][0], qs[0], b0)), x1 = ad_ex2(fmaf(s[nt][1], qs[0], b0));
        const float x2 = ad_ex2(fmaf(s[nt][2], qs[1], b1)), x3 = ad_ex2(fmaf(s[nt][3], qs[1], b1));
        l[0] += x0 + x1;
        l[1] += x2 + x3;
        p[nt / 2][nt % 2 * 2] = pack_f16x2(x0, x1);
        p[nt / 2][nt % 2 * 2 + 1] = pack_f16x2(x2, x3);
      }
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
        const int blk = 4 * half + 2 * ks;  // 8 tokens; and the next 8
        uint32_t v0[GW], v1[GW], s0[GW], s1[GW];
        lds_words<GW>(u + L::kV + blk * (4 * D) + r * (D / 2) + c * (D / 8), v0);
        lds_words<GW>(u + L::kV + (blk + 1) * (4 * D) + r * (D / 2) + c * (D / 8), v1);
        lds_words<GW>(u + L::kVs + (4 * blk + c) * (D / 8), s0);
        lds_words<GW>(u + L::kVs + (4 * blk + 4 + c) * (D / 8), s1);
        uint32_t k0 = kScaleBits, k1 = kScaleBits;  // slots past the last token may hold any scale: theirs become 0
        if (part) {
          const int t0 = 8 * blk + 2 * c, t1 = t0 + 8;
          k0 = (t0 < left ? 0x7F80u : 0u) | (t0 + 1 < left ? 0x7F800000u : 0u);
          k1 = (t1 < left ? 0x7F80u : 0u) | (t1 + 1 < left ? 0x7F800000u : 0u);
        }
#pragma unroll
        for (int w = 0; w < GW; ++w) {
          uint32_t e0 = scales02(s0[w], k0), f0 = scales13(s0[w], k0), e1 = scales02(s1[w], k1), f1 = scales13(s1[w], k1);
          if (bad) e0 = kv4_finite(e0), f0 = kv4_finite(f0), e1 = kv4_finite(e1), f1 = kv4_finite(f1);
          uint32_t x[4], y[4];
          codes4(v0[w], x);
          codes4(v1[w], y);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            x[i] = hmul2(x[i], i < 2 ? e0 : f0);
            y[i] = hmul2(y[i], i < 2 ? e1 : f1);
            mma_f16(o[4 * w + i], p[ks][0], p[ks][1], p[ks][2], p[ks][3], x[i], y[i]);
          }
        }
      }
    }
    // values that are not finite, kept out of the products: they are NaN to the rows that see them
    for (; bad; bad &= bad - 1) {
      const int t = __ffsll((long long)bad) - 1;
#pragma unroll
      for (int g = 0; g < D / 16; ++g)
        if ((u[L::vs(t, g)] & 0xF8u) == 0xF8u) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint64_t path = seen[j >> 1];
            const bool see = base + t < 0 || path >> (base + t) & 1;
            if (see) o[2 * g][j] = o[2 * g + 1][j] = __int_as_float(0x7FFFFFFF);
          }
        }
    }
  }

  // The sums over the lanes of a row; rows that are none hold nothing.
  __device__ __forceinline__ void finish() {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      l[k] += __shfl_xor_sync(0xffffffffu, l[k], 1);
      l[k] += __shfl_xor_sync(0xffffffffu, l[k], 2);
      if (seen[k] == 0) {
        m[k] = -INFINITY, l[k] = 0.0f;
#pragma unroll
        for (int i = 0; i < D / 8; ++i) o[i][2 * k] = o[i][2 * k + 1] = 0.0f;
      }
    }
  }
  __device__ __forceinline__ void store_part(float* out, float* pm, float* pl, int lane) const {
    const int r = lane >> 2, c = lane & 3;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      if (c == 0) pm[r + 8 * k] = m[k], pl[r + 8 * k] = l[k];
      float* d = out + (r + 8 * k) * AtrCfg<D, 16>::kStride + 2 * c;
#pragma unroll
      for (int i = 0; i < D / 8; ++i) *reinterpret_cast<float2*>(d + 8 * i) = make_float2(o[i][2 * k], o[i][2 * k + 1]);
    }
  }
  __device__ __forceinline__ void store_out(const AtrArgs& a, int b, int hk, int lane) const {
    const int r = lane >> 2, c = lane & 3, rows = atr_nodes(a.g, b) * a.G;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int x = r + 8 * k, node = x / a.G;
      if (x >= rows) continue;
      const float inv = l[k] != 0.0f ? 1.0f / l[k] : 0.0f;  // nothing seen: zeros
      uint16_t* d = a.g.out + (size_t)(a.g.t.cu[b] + node) * a.g.ld_o + (size_t)(hk * a.G + x - node * a.G) * D + 2 * c;
#pragma unroll
      for (int i = 0; i < D / 8; ++i)
        *reinterpret_cast<uint32_t*>(d + 8 * i) = pack_bf16x2(o[i][2 * k] * inv, o[i][2 * k + 1] * inv);
    }
  }
};

// The same for 8 rows, the other way round: tokens (then channels) are the products' rows
// and the queries' rows their 8 columns, so that nothing of a product is empty.  Lane (r, c)
// owns rows 2c and 2c + 1.
template <int D>
struct AtrFewRows {
  uint32_t q[D / 16][2];  // B operand: row r; channels 16g + 4c .. + 3
  float qs[2], m[2], l[2];
  uint64_t seen[2];
  float o[D / 16][4];     // channels 16i + r and 16i + 8 + r of rows 2c, 2c + 1

  __device__ __forceinline__ void start(const AtrArgs& a, int b, int hk, uint64_t (&tree)[2], bool again, int lane) {
    const int r = lane >> 2, c = lane & 3, first = a.g.t.cu[b], n = atr_nodes(a.g, b), rows = n * a.G;
    const int x = min(r, rows - 1), node = x / a.G;
    const uint2* q0 = reinterpret_cast<const uint2*>(a.g.q + (size_t)(first + node) * a.g.ld_q +
                                                     (size_t)(hk * a.G + x - node * a.G) * D + 4 * c);
    uint2 w[D / 16];
#pragma unroll
    for (int g = 0; g < D / 16; ++g) w[g] = r < rows ? q0[4 * g] : make_uint2(0u, 0u);
    if (again) tree_masks(a.g.t.parent + first, n, lane, tree);
    float top = 0.0f;
#pragma unroll
    for (int g = 0; g < D / 16; ++g)
      top = fmaxf(top, fmaxf(fmaxf(fabsf(bf16lo(w[g].x)), fabsf(bf16hi(w[g].x))),
                             fmaxf(fabsf(bf16lo(w[g].y)), fabsf(bf16hi(w[g].y)))));
    float f, scale;
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
    kv4_query_scale(top, a.g.scale, f, scale);
#pragma unroll
    for (int g = 0; g < D / 16; ++g) {
      q[g][0] = pack_f16x2(bf16lo(w[g].x) * f, bf16hi(w[g].x) * f);
      q[g][1] = pack_f16x2(bf16lo(w[g].y) * f, bf16hi(w[g].y) * f);
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      qs[k] = __shfl_sync(0xffffffffu, scale, 8 * c + 4 * k);
      const uint64_t path = tree_mask_of(tree, min(2 * c + k, rows - 1) / a.G);
      seen[k] = 2 * c + k < rows ? path : 0ull;
      m[k] = -INFINITY, l[k] = 0.0f;
    }
#pragma unroll
    for (int i = 0; i < D / 16; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) o[i][j] = 0.0f;
  }

  __device__ __forceinline__ void units(const uint8_t* u, int base, int left, int h0, int h1, int lane) {
    using L = Kv4Block<D>;
    constexpr int GW = D / 32;
    const int r = lane >> 2, c = lane & 3;
    const bool part = base > -kPage;
    const uint64_t bad = part ? atr_bad<D>(u, left, h0, h1, lane) : 0ull;
#pragma unroll 1
    for (int half = h0; half < h1; ++half) {
      float s[2][4];
#pragma unroll
      for (int mt = 0; mt < 2; ++mt) {
        uint32_t k0[GW], k1[GW], c0[GW / 2], c1[GW / 2];
        const int t0 = 32 * half + 16 * mt + r;
        lds_words<GW>(u + L::kK + t0 * (D / 2) + c * (D / 8), k0);
        lds_words<GW>(u + L::kK + (t0 + 8) * (D / 2) + c * (D / 8), k1);
        lds_words<GW / 2>(u + L::kKs + t0 * (D / 16), c0);
        lds_words<GW / 2>(u + L::kKs + (t0 + 8) * (D / 16), c1);
#pragma unroll
        for (int w = 0; w < GW; ++w) {
          const uint32_t e0 = scales02(c0[w / 2], kScaleBits), f0 = scales13(c0[w / 2], kScaleBits);
          const uint32_t e1 = scales02(c1[w / 2], kScaleBits), f1 = scales13(c1[w / 2], kScaleBits);
          uint32_t x[4], y[4];
          codes4(k0[w], x);
          codes4(k1[w], y);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t sx = i < 2 ? e0 : f0, sy = i < 2 ? e1 : f1;
            x[i] = w & 1 ? hmul2_hi(x[i], sx) : hmul2_lo(x[i], sx);
            y[i] = w & 1 ? hmul2_hi(y[i], sy) : hmul2_lo(y[i], sy);
          }
          if (w == 0)
            mma_f16_first(s[mt], x[0], y[0], x[1], y[1], q[0][0], q[0][1]);
          else
            mma_f16(s[mt], x[0], y[0], x[1], y[1], q[2 * w][0], q[2 * w][1]);
          mma_f16(s[mt], x[2], y[2], x[3], y[3], q[2 * w + 1][0], q[2 * w + 1][1]);
        }
      }
      bool grow = false;
      float mx[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        if (part) {
          const uint64_t see = base >= 0 ? seen[k] >> base : seen[k] << -base | ((1ull << -base) - 1);
          const uint32_t bits = (uint32_t)(see >> (32 * half)) >> r;
#pragma unroll
          for (int mt = 0; mt < 2; ++mt)
#pragma unroll
            for (int j = 0; j < 2; ++j)
              if (!(bits >> (16 * mt + 8 * j) & 1u)) s[mt][2 * j + k] = -INFINITY;
        }
        mx[k] = fmaxf(fmaxf(s[0][k], s[0][2 + k]), fmaxf(s[1][k], s[1][2 + k]));
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) mx[k] = fmaxf(mx[k], __shfl_xor_sync(0xffffffffu, mx[k], x));
        mx[k] *= qs[k];
        grow |= mx[k] - m[k] > 8.0f;
      }
      if (__any_sync(0xffffffffu, grow)) {  // (as for 16 rows)
        float f[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const bool up = mx[k] - m[k] > 8.0f;
          f[k] = up ? ad_ex2(m[k] - mx[k]) : 1.0f;
          if (up) m[k] = mx[k];
          l[k] *= f[k];
        }
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) o[i][j] *= f[j & 1];
      }
      uint32_t p[2][2];
      const float b0 = m[0] == -INFINITY ? 0.0f : 7.0f - m[0], b1 = m[1] == -INFINITY ? 0.0f : 7.0f - m[1];
#pragma unroll
      for (int mt = 0; mt < 2; ++mt) {
        const float x0 = ad_ex2(fmaf(s[mt][0], qs[0], b0)), x1 = ad_ex2(fmaf(s[mt][1], qs[1], b1));
        const float x2 = ad_ex2(fmaf(s[mt][2], qs[0], b0)), x3 = ad_ex2(fmaf(s[mt][3], qs[1], b1));
        l[0] += x0 + x2;
        l[1] += x1 + x3;
        p[mt][0] = trans8x8(pack_f16x2(x0, x1));
        p[mt][1] = trans8x8(pack_f16x2(x2, x3));
      }
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
        const int blk = 4 * half + 2 * ks;
        uint32_t v0[GW], v1[GW], s0[GW], s1[GW];
        lds_words<GW>(u + L::kV + blk * (4 * D) + r * (D / 2) + c * (D / 8), v0);
        lds_words<GW>(u + L::kV + (blk + 1) * (4 * D) + r * (D / 2) + c * (D / 8), v1);
        lds_words<GW>(u + L::kVs + (4 * blk + c) * (D / 8), s0);
        lds_words<GW>(u + L::kVs + (4 * blk + 4 + c) * (D / 8), s1);
        uint32_t k0 = kScaleBits, k1 = kScaleBits;  // slots past the last token may hold any scale: theirs become 0
        if (part) {
          const int t0 = 8 * blk + 2 * c, t1 = t0 + 8;
          k0 = (t0 < left ? 0x7F80u : 0u) | (t0 + 1 < left ? 0x7F800000u : 0u);
          k1 = (t1 < left ? 0x7F80u : 0u) | (t1 + 1 < left ? 0x7F800000u : 0u);
        }
#pragma unroll
        for (int w = 0; w < GW; ++w) {
          uint32_t e0 = scales02(s0[w], k0), f0 = scales13(s0[w], k0), e1 = scales02(s1[w], k1), f1 = scales13(s1[w], k1);
          if (bad) e0 = kv4_finite(e0), f0 = kv4_finite(f0), e1 = kv4_finite(e1), f1 = kv4_finite(f1);
          uint32_t x[4], y[4];
          codes4(v0[w], x);
          codes4(v1[w], y);
#pragma unroll
          for (int i = 0; i < 4; ++i) x[i] = hmul2(x[i], i < 2 ? e0 : f0), y[i] = hmul2(y[i], i < 2 ? e1 : f1);
          mma_f16(o[2 * w], x[0], x[1], y[0], y[1], p[ks][0], p[ks][1]);
          mma_f16(o[2 * w + 1], x[2], x[3], y[2], y[3], p[ks][0], p[ks][1]);
        }
      }
    }
    for (uint64_t e = bad; e; e &= e - 1) {
      const int t = __ffsll((long long)e) - 1;
#pragma unroll
      for (int g = 0; g < D / 16; ++g)
        if ((u[L::vs(t, g)] & 0xF8u) == 0xF8u) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const bool see = base + t < 0 || seen[j & 1] >> (base + t) & 1;
            if (see) o[g][j] = __int_as_float(0x7FFFFFFF);
          }
        }
    }
  }

  __device__ __forceinline__ void finish() {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
#pragma unroll
      for (int x = 4; x < 32; x <<= 1) l[k] += __shfl_xor_sync(0xffffffffu, l[k], x);
      if (seen[k] == 0) {
        m[k] = -INFINITY, l[k] = 0.0f;
#pragma unroll
        for (int i = 0; i < D / 16; ++i) o[i][k] = o[i][2 + k] = 0.0f;
      }
    }
  }
  __device__ __forceinline__ void store_part(float* out, float* pm, float* pl, int lane) const {
    const int r = lane >> 2, c = lane & 3;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      if (r == 0) pm[2 * c + k] = m[k], pl[2 * c + k] = l[k];
      float* d = out + (2 * c + k) * AtrCfg<D, 8>::kStride + r;
#pragma unroll
      for (int i = 0; i < D / 16; ++i) d[16 * i] = o[i][k], d[16 * i + 8] = o[i][2 + k];
    }
  }
  __device__ __forceinline__ void store_out(const AtrArgs& a, int b, int hk, int lane) const {
    const int r = lane >> 2, c = lane & 3, rows = atr_nodes(a.g, b) * a.G;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int x = 2 * c + k, node = x / a.G;
      if (x >= rows) continue;
      const float inv = l[k] != 0.0f ? 1.0f / l[k] : 0.0f;  // nothing seen: zeros
      uint16_t* d = a.g.out + (size_t)(a.g.t.cu[b] + node) * a.g.ld_o + (size_t)(hk * a.G + x - node * a.G) * D + r;
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        d[16 * i] = f32_to_bf16(o[i][k] * inv);
        d[16 * i + 8] = f32_to_bf16(o[i][2 + k] * inv);
      }
    }
  }
};

__device__ __forceinline__ void atr_copy16(uint32_t dst, const void* src, uint64_t pol) {
  asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "l"(pol) : "memory");
}

template <int D, int ROWS>
__global__ void __launch_bounds__(kAtrThreads, 1) attn_tree_kernel(const __grid_constant__ AtrArgs a) {
  using C = AtrCfg<D, ROWS>;
  constexpr int S = C::kStages, PARTS = kAtrParts;
  static_assert(PARTS * ROWS <= kAtrThreads && PARTS <= 32, "a thread per part and row");
  static_assert(C::kRecord * 4 <= C::kRing, "a record lies in its warp's ring");
  extern __shared__ __align__(128) uint8_t smem[];
  AtrShared<ROWS>* sh = reinterpret_cast<AtrShared<ROWS>*>(smem + kAtWarps * C::kRing);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, cta = blockIdx.x;
  if (lane == 0) sh->meta[2 * warp].seg = sh->meta[2 * warp + 1].seg = -1;
  if (tid < 2) sh->cta_seg[tid] = -1;
  pdl_wait();
  pdl_trigger();
  const int B = a.g.t.nseq;
  // ---- the span and its runs: prefix sums of the sequences' units (one a thread)
  static_assert(kSeqs <= kAtrThreads, "a sequence a thread");
  const int their = tid < B ? (atr_len(a.g, tid) + kPage - 1) / kPage : 0;
  const int mine = their ? (2 * their + kAtrSetup) * a.g.c.Hkv : 0;
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
  for (int w = 0; w < kAtWarps; ++w) {
    if (w < warp) pre += sh->scan[w];
    total += sh->scan[w];
  }
  int s0, s1;
  if (a.by_row) {  // kv head cta % Hkv of sequence cta / Hkv
    const int b = cta / a.g.c.Hkv;
    if (tid == b) {
      const int n = mine / a.g.c.Hkv;
      sh->run0[0] = pre + (cta - b * a.g.c.Hkv) * n;
      sh->run0[1] = sh->run0[0] + n;
    }
    __syncthreads();
    s0 = sh->run0[0];
    s1 = sh->run0[1];
    __syncthreads();
  } else {
    // at least a unit for every warp: the CTAs without work are the last ones
    const int nc = min(a.nc, (total + kAtWarps - 1) / kAtWarps), q = nc ? total / nc : 0, extra = total - q * nc;
    s0 = cta < nc ? q * cta + min(cta, extra) : total;
    s1 = cta < nc ? s0 + q + (cta < extra ? 1 : 0) : total;
  }
  {
    // run w: its share of the span, the first ones a unit longer
    const int q = (s1 - s0) / kAtWarps, extra = s1 - s0 - q * kAtWarps;
    if (tid <= kAtWarps) sh->run0[tid] = s0 + q * tid + min(tid, extra);
    if (mine && pre < s1 && pre + mine > s0)
      for (int w = 0; w < kAtWarps; ++w) {
        const int u = s0 + q * w + min(w, extra);
        if (u >= pre && u < pre + mine) {
          sh->run_b[w] = tid;
          sh->run_base[w] = pre;
        }
      }
  }
  // rows of sequences that take no part
  for (int b = cta; b < B; b += gridDim.x)
    if (atr_len(a.g, b) == 0)
      for (int i = tid; i < atr_nodes(a.g, b) * (a.g.H * D / 8); i += kAtrThreads) {
        const int j = i / (a.g.H * D / 8), e = i - j * (a.g.H * D / 8);
        *reinterpret_cast<uint4*>(a.g.out + (size_t)(a.g.t.cu[b] + j) * a.g.ld_o + 8 * e) = make_uint4(0u, 0u, 0u, 0u);
      }
  __syncthreads();

  // ---- this warp's run
  uint8_t* ring = smem + warp * C::kRing;
  const int u0 = sh->run0[warp], u1 = sh->run0[warp + 1];
  if (u1 > u0) {
    AtrCursor cur;
    cur.b = sh->run_b[warp];
    cur.load(a, ROWS);
    int at;  // the tile's first unit behind its set-up
    {
      const int each = 2 * cur.pages + kAtrSetup, in = u0 - sh->run_base[warp];
      cur.tile = 0;
      cur.hk = in / each;
      at = u0 - (in - cur.hk * each) + kAtrSetup;
      cur.page = max(u0 - at, 0) / 2;
    }
    // Pages are asked for by all lanes (a bulk copy by one of them held its warp up for
    // 1000 cycles, a page's products take 6500).  Their numbers are loaded ahead, the first two together.
    const uint64_t pol = policy_evict_first();
    AtrCursor ahead = cur;
    int ahead_at = at, id = 0, id_hk = 0, id1 = 0, id1_hk = 0;
    bool more = true, more1 = true;  // id and id1 are pages of the run
    auto look = [&](bool first) {    // id = id1; id1 = the run's next page
      id = id1, id_hk = id1_hk, more = more1;
      if (!more1) return;
      if (!first) {
        if (ahead.page + 1 == ahead.pages) ahead_at += 2 * ahead.pages + kAtrSetup;
        ahead.next(a, ROWS);
      }
      more1 = ahead_at + 2 * ahead.page < u1;
      if (more1) id1 = a.g.c.table[(size_t)ahead.b * a.g.c.ld_table + ahead.page], id1_hk = ahead.hk;
    };
    look(true);
    look(false);
    int fetched = 0;
    uint32_t ok = 0;  // stages that hold a page
    const uint32_t to = smem_addr(ring) + 16 * lane;
    uint64_t tree[2] = {0, 0};
    typename std::conditional<ROWS == 8, AtrFewRows<D>, AtrRows<D>>::type rows;
    int pos = 0, masks_of = -1;
    // Everything stands in this loop once: code that is not in the SM's cache costs some 50 cycles an instruction.
#pragma unroll 1
    for (int i = 0; at + 2 * cur.page < u1; ++i) {
      // the pages up to S - 1 after this one; always a copy group
#pragma unroll 1
      for (; fetched < i + S; ++fetched) {
        if (more) {
          const int st = fetched % S;
          const bool good = id >= 0 && id < a.g.c.n_pages;
          ok = good ? ok | 1u << st : ok & ~(1u << st);
          if (good) {
            const uint8_t* src = a.g.c.pages + ((size_t)id * a.g.c.Hkv + id_hk) * C::kBytes + 16 * lane;
#pragma unroll
            for (int k = 0; k < C::kBytes / 512; ++k) atr_copy16(to + st * C::kBytes + 512 * k, src + 512 * k, pol);
          } else if (lane == 0) {
            M2_RECORD_ARG(g_status);
          }
          look(false);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
      }
      if (i == 0 || cur.page == 0) {
        pos = a.g.pos[cur.b];
        rows.start(a, cur.b, cur.hk, tree, cur.b != masks_of, lane);
        masks_of = cur.b;
      }
      const int st = i % S, left = u1 - at - 2 * cur.page;  // units of the run from this page on
      asm volatile("cp.async.wait_group %0;" ::"n"(S - 1) : "memory");
      __syncwarp();
      if (ok >> st & 1)
        rows.units(ring + st * C::kBytes, cur.page * kPage - pos, cur.len - cur.page * kPage,
                   max(u0 - at - 2 * cur.page, 0), min(left, 2), lane);
      __syncwarp();  // the stage is read
      const bool ends = cur.page + 1 == cur.pages;
      if (ends || left <= 2) {  // the tile leaves this warp
        rows.finish();
        const int end = at + 2 * cur.pages;
        if (at >= u0 && end <= u1) {
          rows.store_out(a, cur.b, cur.hk, lane);
        } else {
          const int slot = end + kAtrSetup >= u1 ? 1 : 0;
          // the last part goes into the ring (free by now), an earlier one through L2
          rows.store_part(slot ? reinterpret_cast<float*>(ring) : a.part + (size_t)(cta * kAtWarps + warp) * C::kRecord,
                          sh->part_m[2 * warp + slot], sh->part_l[2 * warp + slot], lane);
          if (lane == 0) {
            AtrMeta& mt = sh->meta[2 * warp + slot];
            mt.seg = cur.seg(a);
            mt.before = at < s0;
            mt.after = end > s1;
          }
        }
        if (!ends) break;
        at = end + kAtrSetup;
      }
      cur.next(a, ROWS);
      if (cur.b >= B) break;
    }
  }
  __syncthreads();

  // ---- tiles cut between warps
  const int seg_e = lane < PARTS ? sh->meta[lane].seg : -1;
  const uint32_t same = __match_any_sync(0xffffffffu, seg_e);  // entry `lane`: all parts of its tile
  const uint32_t lead = __ballot_sync(0xffffffffu, seg_e >= 0 && (same & ((1u << lane) - 1)) == 0);
  const int ntiles = __popc(lead);
  {
    // a thread per (part, row): those of a tile's first part weigh its parts
    const int e = tid / ROWS, x = tid - e * ROWS;
    const uint32_t parts = __shfl_sync(0xffffffffu, same, e & 31);
    if (e < PARTS && (lead >> e & 1)) {
      float top = -INFINITY, l = 0.0f;
      for (uint32_t y = parts; y; y &= y - 1) top = fmaxf(top, sh->part_m[__ffs(y) - 1][x]);
      for (uint32_t y = parts; y; y &= y - 1) {
        const int k = __ffs(y) - 1;
        const float w = ad_weight(sh->part_m[k][x], sh->part_l[k][x], top);
        l += sh->part_l[k][x] * w;
        sh->part_m[k][x] = w;
      }
      const int k = __popc(lead & ((1u << e) - 1));
      const AtrMeta& mt = sh->meta[e];
      uint16_t* out = atr_out(a, mt.seg, x, ROWS, D);
      if (out && (mt.before || mt.after)) {  // cut between CTAs too
        float* rec = a.cta_part + (size_t)(2 * cta + (mt.before ? 0 : 1)) * C::kRecord;
        rec[x] = top;
        rec[ROWS + x] = l;
        out = reinterpret_cast<uint16_t*>(rec + 2 * ROWS + x * C::kStride);
        l = -1.0f;
      }
      if (x == 0) {
        sh->row_parts[k] = parts;
        if (mt.before || mt.after) sh->cta_seg[mt.before ? 0 : 1] = mt.seg;
      }
      sh->row_l[k][x] = l;
      sh->out[k][x] = out;
    }
  }
  __syncthreads();
  for (int i = tid; i < ntiles * (ROWS * D / 4); i += kAtrThreads) {
    const int k = i / (ROWS * D / 4), x = i / (D / 4) % ROWS, d = i % (D / 4) * 4;
    uint32_t parts = sh->row_parts[k];
    uint16_t* out = sh->out[k][x];
    if (!out) continue;
    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    while (parts) {
      // six parts at a time, their loads together
      float4 v[6];
      float w[6];
#pragma unroll
      for (int j = 0; j < 6; ++j) {
        const int y = parts ? __ffs(parts) - 1 : -1;
        parts &= parts - 1;
        w[j] = 0.0f;
        v[j] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (y >= 0) {
          w[j] = sh->part_m[y][x];
          v[j] = y & 1 ? *reinterpret_cast<const float4*>(smem + (y >> 1) * C::kRing + (x * C::kStride + d) * 4)
                       : *reinterpret_cast<const float4*>(a.part + (size_t)(cta * kAtWarps + (y >> 1)) * C::kRecord +
                                                          x * C::kStride + d);
        }
      }
#pragma unroll
      for (int j = 0; j < 6; ++j)
        o.x = fmaf(v[j].x, w[j], o.x), o.y = fmaf(v[j].y, w[j], o.y), o.z = fmaf(v[j].z, w[j], o.z),
        o.w = fmaf(v[j].w, w[j], o.w);
    }
    const float l = sh->row_l[k][x];
    if (l < 0.0f)
      *reinterpret_cast<float4*>(reinterpret_cast<float*>(out) + d) = o;
    else
      atr_store4(out + d, o, l);
  }
  if (tid < 2 && !a.by_row) a.cta_seg[2 * cta + tid] = sh->cta_seg[tid];
}

// Tiles cut between CTAs: block (c, x) joins row x of the tile that began in span c and
// goes on.  D/4 threads hold four channels each; the parts are dealt out over groups of
// them and joined through shared memory.
constexpr int kAtrcThreads = 128;
template <int D, int ROWS>
__global__ void __launch_bounds__(kAtrcThreads, 16) attn_tree_combine_kernel(const __grid_constant__ AtrArgs a) {
  using C = AtrCfg<D, ROWS>;
  constexpr int P = D / 4, GR = kAtrcThreads / P;
  __shared__ float pm[GR], pl[GR];
  __shared__ float4 po[kAtrcThreads];
  pdl_wait();
  pdl_trigger();
  const int c = blockIdx.x, x = blockIdx.y, tid = threadIdx.x, g = tid / P, d = tid % P * 4;
  const int seg = a.cta_seg[2 * c + 1];
  auto load = [&](int y, float& m, float& l, float4& o) {
    const float* r = a.cta_part + (size_t)(y == 0 ? 2 * c + 1 : 2 * min(c + y, a.nc - 1)) * C::kRecord;
    m = r[x], l = r[ROWS + x];
    o = *reinterpret_cast<const float4*>(r + 2 * ROWS + x * C::kStride + d);
  };
  float m, l;
  float4 o;
  load(g, m, l, o);  // (any span's record may be read; how many there are is known next)
  int k = 1;         // parts: this span's, then those of the spans that the tile goes on through
  for (int y = c + 1; y < a.nc; y += kAtrcThreads) {
    const int n = __syncthreads_count(y + tid < a.nc && a.cta_seg[2 * (y + tid)] == seg);
    k += n;
    if (n < kAtrcThreads) break;
  }
  uint16_t* out = seg < 0 ? nullptr : atr_out(a, seg, x, ROWS, D);
  if (!out) return;
  if (g >= k) m = -INFINITY, l = 0.0f, o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  for (int y = g + GR; y < k; y += GR) {
    float m1, l1;
    float4 v;
    load(y, m1, l1, v);
    const float top = fmaxf(m, m1), f = ad_weight(m, l, top), w = ad_weight(m1, l1, top);
    m = top;
    l = l * f + l1 * w;
    o = make_float4(o.x * f + v.x * w, o.y * f + v.y * w, o.z * f + v.z * w, o.w * f + v.w * w);
  }
  po[tid] = o;
  if (d == 0) pm[g] = m, pl[g] = l;
  __syncthreads();
  if (g == 0) {
    float top = m, sum = 0.0f;
#pragma unroll
    for (int y = 1; y < GR; ++y) top = fmaxf(top, pm[y]);
    float4 t = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
    for (int y = 0; y < GR; ++y) {
      const float w = ad_weight(pm[y], pl[y], top);
      const float4 v = po[y * P + tid];
      sum = fmaf(pl[y], w, sum);
      t = make_float4(fmaf(v.x, w, t.x), fmaf(v.y, w, t.y), fmaf(v.z, w, t.z), fmaf(v.w, w, t.w));
    }
    atr_store4(out + d, t, sum);
  }
}

// ------------------------------------------------------------------ host

template <int D>
static size_t atr_ws_bytes() {
  const size_t n = num_sms();
  return n * (kAtWarps + 2) * AtrCfg<D, 16>::kRecord * 4 + (n * 2 * 4 + 255) / 256 * 256;
}
size_t attn_tree_ws_bytes(int32_t D) {
  const size_t x = D == 128 ? atr_ws_bytes<128>() : atr_ws_bytes<64>(), y = attn_tree_tc_ws_bytes(D);
  return x > y ? x : y;  // whatever the trees
}

template <int D, int ROWS>
static cudaError_t launch_atr(const AttnTreeArgs& g, cudaStream_t s) {
  using C = AtrCfg<D, ROWS>;
  static int done_mask[64] = {0};
  constexpr int smem = kAtWarps * C::kRing + (int)sizeof(AtrShared<ROWS>);
  static_assert(smem <= 232448, "shared memory");
  AtrArgs a;
  a.g = g;
  a.G = g.H / g.c.Hkv;
  a.most_tiles = 1;
  const int64_t tiles = (int64_t)g.t.nseq * g.c.Hkv;
  a.by_row = atr_by_row(tiles, g.c.ld_table);
  a.nc = a.by_row ? (int)tiles : num_sms();
  const size_t n = num_sms();
  a.cta_seg = static_cast<int32_t*>(g.ws);
  a.part = reinterpret_cast<float*>(static_cast<uint8_t*>(g.ws) + (n * 2 * 4 + 255) / 256 * 256);
  a.cta_part = a.part + n * kAtWarps * C::kRecord;
  auto kern = attn_tree_kernel<D, ROWS>;
  cudaError_t e = set_smem_once((const void*)kern, smem, done_mask);
  if (e != cudaSuccess) return e;
  trace_pre(K_ATTN_TREE, s);
  e = launch_k(kern, dim3(a.nc), dim3(kAtrThreads), smem, s, true, a);
  trace_post(K_ATTN_TREE, s);
  if (e != cudaSuccess || a.by_row) return e;
  trace_pre(K_ATTN_TREE_COMBINE, s);
  e = launch_k(attn_tree_combine_kernel<D, ROWS>, dim3(a.nc, g.most * a.G), dim3(kAtrcThreads), 0, s, true, a);
  trace_post(K_ATTN_TREE_COMBINE, s);
  return e;
}

cudaError_t launch_attn_tree(const AttnTreeArgs& a, cudaStream_t s) {
  // 16 rows here / by the tensor-core kernel: 61.9 / 102.9 us for 64 sequences of 64 to
  // 4096 tokens, 14.4 / 15.8 for one of 2000; a second tile of 16 rows would work through
  // every page again.  8 rows by the kernel for 8 / for 16: 46.8 / 56.5 us for the 64, 21.7 /
  // 24.2 for one of 30000; 5 rows of 16 kv heads of 64: 55.4 / 61.8.
  // The launch's largest tree decides for all: 63 chains of 4 and one of 5 take 100 us, 64 of 4 61.
  const int rows = a.most * (a.H / a.c.Hkv);
  if (rows > 16) return launch_attn_tree_tc(a, s);
  if (rows > 8) return a.c.D == 128 ? launch_atr<128, 16>(a, s) : launch_atr<64, 16>(a, s);
  return a.c.D == 128 ? launch_atr<128, 8>(a, s) : launch_atr<64, 8>(a, s);
}

int status_attn_tree(int clear) { return tu_status(clear); }

}  // namespace m2
