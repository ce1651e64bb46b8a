// k_attn_decode.cu -- attention of one query token a sequence over the paged
// 4-bit cache.
//
// A unit is one page (64 tokens) of one kv head: 72 * D contiguous bytes.  The
// units of all sequences, in the order (sequence, head chunk, page), are cut
// into equal spans, one a CTA, and each span into equal runs, one a warp, so
// that ragged lengths, few sequences and single long ones all load every SM
// alike.  A warp streams its units through its own ring of bulk copies and
// keeps the running softmax of up to 16 query heads (HN = 8 or 16) on warp MMA:
//   S^T [64 tokens x HN] = K Q^T    K codes become f16 and take their scale,
//                                   exactly (6 significant bits)
//   O^T [D x HN] += V^T P^T         likewise V; P rounded to f16 (2^-11)
// Queries enter as f16 rows prescaled by an exact power of two (exact but for
// channels more than 2^17 below the head's largest).  f16 is what the codes convert to;
// the rms error against 64 bits is 0.00169 of the output, with fp32 queries and
// probabilities 0.00168.  Scores, sums and outputs are fp32.  Rows that a warp, then a CTA, holds only in part are
// joined: warps through shared memory, CTAs by attn_decode_combine.
// Bound: HBM (4.5 bits a value) once data streams, and the start and the joining of
// rows cut between CTAs.  Measured at 32 + 8 heads of 128, as graph replays: 131000
// tokens of one sequence 35.5 us (4.2 TB/s), 64 sequences of 64..4096 tokens 41 us (4.1
// TB/s); 6 to 7 us of that are the way to the first data, 4 to 5 the joining, and what
// is between runs at 5.6 to 6 TB/s.  A unit is about 1060 instructions of a warp with
// all around it (256 conversions of two codes, 256 multiplications by scales, 64 MMAs
// at HN = 8): 47% of the issue slots over the whole launch.  168 registers a
// thread at D = 128, which spills 24 bytes of stores at HN = 8 and 348 at HN = 16.  8 warps with 3 stages took 48 us
// instead of 37 in the kernel itself, 12 warps with 128 registers the same.
#include <cuda_runtime.h>
#include <stdint.h>

#include "m2_common.cuh"
#include "m2_kernels.h"
#include "m2_kv4.cuh"
#include "m2_tc.cuh"

namespace m2 {

constexpr int kAdWarps = 12;

template <int D>
struct AdCfg {
  static constexpr int kUnit = Kv4Block<D>::kBytes;
  static constexpr int kStages = D == 128 ? 2 : 4;  // 12 warps * stages * unit = 216 KB
  static constexpr int kRing = kStages * kUnit;     // of one warp
  static constexpr int kStride = D + 4;             // floats between the heads of a record: no bank conflicts
};
// A partial result: running maxima and sums of HN heads, then their outputs.
template <int D, int HN>
constexpr int ad_record() {
  return 2 * HN + HN * AdCfg<D>::kStride;
}
constexpr int kAdParts = 2 * kAdWarps;  // a warp leaves a first and a last part at most
// Which row (sequence, head chunk) a partial belongs to, and whether the row
// starts before / ends after the CTA's span.
struct AdMeta {
  int32_t seg, before, after;
};
struct AdShared {
  uint64_t full[kAdWarps][6];
  int32_t ok[kAdWarps][6];
  AdMeta meta[kAdParts];
  float part_m[kAdParts][16], part_l[kAdParts][16];  // the parts' maxima (then their weights) and sums
  float row_l[kAdParts][16];                         // sums of the cut rows
  uint32_t row_parts[kAdParts];                      // their parts, as bits
  int32_t cta_seg[2];
  int32_t scan[kAdWarps];
  int32_t run0[kAdWarps + 1];           // first unit of each warp's run, then the span's end
  int32_t run_b[kAdWarps];              // sequence of the run's first unit
  int32_t run_base[kAdWarps];           // units before that sequence
};

struct AdArgs {
  AttnDecodeArgs g;
  int32_t G, chunks, rows;  // query heads a kv head; chunks of HN heads; rows = Hkv * chunks a sequence
  int32_t nc;               // CTAs
  int32_t by_row;           // one CTA a row: no row is cut
  float* warp_part;         // [nc][kAdWarps] records
  float* cta_part;          // [nc][2] records: a row that began earlier, a row that goes on
  int32_t* cta_seg;         // [nc][2] rows of those, -1 where there is none
};

__device__ __forceinline__ int ad_len(const AttnDecodeArgs& g, int b) {
  const int n = g.len[b], most = g.c.ld_table * kPage;
  if (n > most) M2_RECORD_ARG(g_status);
  return max(0, min(n, most));
}
__device__ __forceinline__ int ad_pages(const AttnDecodeArgs& g, int b) { return (ad_len(g, b) + kPage - 1) / kPage; }

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
      "%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The same from zero.
__device__ __forceinline__ void mma_f16_first(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, "
      "%10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}
// a times one half of s: the instruction broadcasts it.
__device__ __forceinline__ uint32_t hmul2_lo(uint32_t a, uint32_t s) {
  const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&a), __low2half2(*reinterpret_cast<const __half2*>(&s)));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t hmul2_hi(uint32_t a, uint32_t s) {
  const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&a), __high2half2(*reinterpret_cast<const __half2*>(&s)));
  return *reinterpret_cast<const uint32_t*>(&r);
}
// The four bytes of a code word as f16x2.
__device__ __forceinline__ void codes4(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\tcvt.rn.f16x2.e2m1x2 %2, c;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}
__device__ __forceinline__ uint32_t trans8x8(uint32_t a) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(a));
  return r;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float ad_ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// 4-byte words of a lane's codes or scales.
template <int N>
__device__ __forceinline__ void lds_words(const uint8_t* p, uint32_t (&w)[N]) {
  if constexpr (N == 8) {
    const uint4 v = reinterpret_cast<const uint4*>(p)[0], x = reinterpret_cast<const uint4*>(p)[1];
    w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w, w[4] = x.x, w[5] = x.y, w[6] = x.z, w[7] = x.w;
  } else if constexpr (N == 4) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
  } else {
    static_assert(N == 2, "words");
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    w[0] = v.x, w[1] = v.y;
  }
}
// Two scale bytes of a word (0 and 2, or 1 and 3) as f16x2.
constexpr uint32_t kScaleBits = 0x7F807F80u;
__device__ __forceinline__ uint32_t scales02(uint32_t w, uint32_t mask) { return (w << 7) & mask; }
__device__ __forceinline__ uint32_t scales13(uint32_t w, uint32_t mask) { return (w >> 1) & mask; }

// The running softmax of one row (sequence, head chunk) in a warp.  Lane (r, c) =
// (lane / 4, lane % 4) owns heads 2c and 2c + 1 of each tile of 8.
template <int D, int NT>
struct AdRow {
  uint32_t q[NT][D / 16][2];  // B operand: head r, channels 16g + 4c .. + 3
  float qs[NT][2];            // score factor (log2 units) of heads 2c, 2c + 1
  float m[NT][2], l[NT][2];   // reference maximum; this lane's share of the sum
  float o[NT][D / 16][4];     // channels 16i + r and 16i + 8 + r of heads 2c, 2c + 1

  __device__ __forceinline__ void start(const AdArgs& a, int b, int row, int lane) {
    const int r = lane >> 2, c = lane & 3, hk = row / a.chunks, ch = row - hk * a.chunks;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int h = ch * 8 * NT + t * 8 + r;  // within the group
      uint2 w[D / 16];
      float top = 0.0f;
#pragma unroll
      for (int g = 0; g < D / 16; ++g) {
        w[g] = make_uint2(0u, 0u);
        if (h < a.G)
          w[g] = *reinterpret_cast<const uint2*>(a.g.q + (size_t)b * a.g.ld_q + (size_t)(hk * a.G + h) * D + 16 * g + 4 * c);
        top = fmaxf(top, fmaxf(fmaxf(fabsf(bf16lo(w[g].x)), fabsf(bf16hi(w[g].x))),
                               fmaxf(fabsf(bf16lo(w[g].y)), fabsf(bf16hi(w[g].y)))));
      }
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      // 2^-e for a largest magnitude of 2^e ..: exact in f16 except far below the largest
      int e = (int)(__float_as_uint(top) >> 23);
      e = e == 255 ? 127 : max(1, min(e, 253));
      // the factor's sign goes into the queries, and a factor of 0 makes them 0: qs > 0
      const float sc = a.g.scale * 1.4426950408889634f, u = __uint_as_float((uint32_t)e << 23);
      const float f = sc == 0.0f ? 0.0f : copysignf(__uint_as_float((uint32_t)(254 - e) << 23), sc);
#pragma unroll
      for (int g = 0; g < D / 16; ++g) {
        q[t][g][0] = pack_f16x2(bf16lo(w[g].x) * f, bf16hi(w[g].x) * f);
        q[t][g][1] = pack_f16x2(bf16lo(w[g].y) * f, bf16hi(w[g].y) * f);
      }
      const float k = sc == 0.0f ? 1.0f : fmaxf(u * fabsf(sc), 1.17549435e-38f);
      qs[t][0] = __shfl_sync(0xffffffffu, k, 8 * c);
      qs[t][1] = __shfl_sync(0xffffffffu, k, 8 * c + 4);
#pragma unroll
      for (int i = 0; i < 2; ++i) m[t][i] = -INFINITY, l[t][i] = 0.0f;
#pragma unroll
      for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) o[t][i][j] = 0.0f;
    }
  }

  // One unit in shared memory, of which the first `seen` tokens count.  Its scale
  // bytes become f16 once (a token or token pair a lane) in the place where both
  // kinds lay, first K's, after the scores V's: done by every lane for itself, the
  // conversion was an eighth of the unit's instructions.
  __device__ __forceinline__ void unit(uint8_t* u, int seen, int lane) {
    using L = Kv4Block<D>;
    constexpr int GW = D / 32;  // words of a lane's codes: 2 groups each
    const int r = lane >> 2, c = lane & 3;
    uint8_t* sc = u + L::kKs;
    uint32_t vs[GW];  // of token pair `lane`
    {
      uint32_t ks[GW];  // of tokens 2 lane and 2 lane + 1
      lds_words<GW>(sc + lane * (D / 8), ks);
      lds_words<GW>(u + L::kVs + lane * (D / 8), vs);
      __syncwarp();
#pragma unroll
      for (int i = 0; i < GW; i += 2)
        *reinterpret_cast<uint4*>(sc + lane * (D / 4) + 8 * i) =
            make_uint4(scales02(ks[i], kScaleBits), scales13(ks[i], kScaleBits), scales02(ks[i + 1], kScaleBits),
                       scales13(ks[i + 1], kScaleBits));
      __syncwarp();
    }
    float s[4][NT][4];
#pragma unroll
    for (int mt = 0; mt < 4; ++mt) {
      uint32_t k0[GW], k1[GW], s0[GW], s1[GW];
      const int t0 = 16 * mt + r;
      lds_words<GW>(u + L::kK + t0 * (D / 2) + c * (D / 8), k0);
      lds_words<GW>(u + L::kK + (t0 + 8) * (D / 2) + c * (D / 8), k1);
      lds_words<GW>(sc + t0 * (D / 8), s0);
      lds_words<GW>(sc + (t0 + 8) * (D / 8), s1);
#pragma unroll
      for (int w = 0; w < GW; ++w) {
        // scales of groups 4(w/2) .. + 3 lie as (0, 2), (1, 3): this code word's groups are (0, 1) or (2, 3) of them
        const uint32_t e0 = s0[w & ~1], f0 = s0[w | 1], e1 = s1[w & ~1], f1 = s1[w | 1];
        uint32_t x[4], y[4];
        codes4(k0[w], x);
        codes4(k1[w], y);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t sx = i < 2 ? e0 : f0, sy = i < 2 ? e1 : f1;
          x[i] = w & 1 ? hmul2_hi(x[i], sx) : hmul2_lo(x[i], sx);
          y[i] = w & 1 ? hmul2_hi(y[i], sy) : hmul2_lo(y[i], sy);
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          if (w == 0)
            mma_f16_first(s[mt][t], x[0], y[0], x[1], y[1], q[t][0][0], q[t][0][1]);
          else
            mma_f16(s[mt][t], x[0], y[0], x[1], y[1], q[t][2 * w][0], q[t][2 * w][1]);
          mma_f16(s[mt][t], x[2], y[2], x[3], y[3], q[t][2 * w + 1][0], q[t][2 * w + 1][1]);
        }
      }
    }
    // softmax: P as the second product's B operand.  qs > 0: maxima are taken before it is applied.
    if (seen < kPage) {
#pragma unroll
      for (int mt = 0; mt < 4; ++mt)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (16 * mt + r + (j & 2) * 4 >= seen)
#pragma unroll
            for (int t = 0; t < NT; ++t) s[mt][t][j] = -INFINITY;
    }
    uint32_t p[4][NT][2];
    bool grow = false;
    float mx[NT][2];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        mx[t][i] = fmaxf(fmaxf(fmaxf(s[0][t][i], s[0][t][i + 2]), fmaxf(s[1][t][i], s[1][t][i + 2])),
                         fmaxf(fmaxf(s[2][t][i], s[2][t][i + 2]), fmaxf(s[3][t][i], s[3][t][i + 2])));
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) mx[t][i] = fmaxf(mx[t][i], __shfl_xor_sync(0xffffffffu, mx[t][i], x));
        mx[t][i] *= qs[t][i];
        grow |= mx[t][i] - m[t][i] > 8.0f;
      }
    }
    // the reference follows the maximum once it has grown 2^8: until then P (with its
    // factor 2^7, which keeps small ones out of f16's subnormals) stays below 2^15
    if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        float f[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const bool up = mx[t][i] - m[t][i] > 8.0f;
          f[i] = up ? ad_ex2(m[t][i] - mx[t][i]) : 1.0f;
          if (up) m[t][i] = mx[t][i];
          l[t][i] *= f[i];
        }
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) o[t][i][j] *= f[j & 1];
      }
    }
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const float b0 = m[t][0] == -INFINITY ? 0.0f : 7.0f - m[t][0], b1 = m[t][1] == -INFINITY ? 0.0f : 7.0f - m[t][1];
#pragma unroll
      for (int mt = 0; mt < 4; ++mt) {
        const float x0 = ad_ex2(fmaf(s[mt][t][0], qs[t][0], b0)), x1 = ad_ex2(fmaf(s[mt][t][1], qs[t][1], b1));
        const float x2 = ad_ex2(fmaf(s[mt][t][2], qs[t][0], b0)), x3 = ad_ex2(fmaf(s[mt][t][3], qs[t][1], b1));
        l[t][0] += x0 + x2;
        l[t][1] += x1 + x3;
        p[mt][t][0] = trans8x8(pack_f16x2(x0, x1));
        p[mt][t][1] = trans8x8(pack_f16x2(x2, x3));
      }
    }
    {
      // slots past the last token may hold any scale: theirs become 0
      const uint32_t m = (2 * lane < seen ? 0x7F80u : 0u) | (2 * lane + 1 < seen ? 0x7F800000u : 0u);
      __syncwarp();
#pragma unroll
      for (int i = 0; i < GW; i += 2)
        *reinterpret_cast<uint4*>(sc + lane * (D / 4) + 8 * i) =
            make_uint4(scales02(vs[i], m), scales13(vs[i], m), scales02(vs[i + 1], m), scales13(vs[i + 1], m));
      __syncwarp();
    }
#pragma unroll
    for (int ks = 0; ks < 4; ++ks) {
      uint32_t v0[GW], v1[GW], s0[2 * GW], s1[2 * GW];
      lds_words<GW>(u + L::kV + (2 * ks) * (4 * D) + r * (D / 2) + c * (D / 8), v0);
      lds_words<GW>(u + L::kV + (2 * ks + 1) * (4 * D) + r * (D / 2) + c * (D / 8), v1);
      lds_words<2 * GW>(sc + (8 * ks + c) * (D / 4), s0);
      lds_words<2 * GW>(sc + (8 * ks + 4 + c) * (D / 4), s1);
#pragma unroll
      for (int w = 0; w < GW; ++w) {
        const uint32_t e0 = s0[2 * w], f0 = s0[2 * w + 1], e1 = s1[2 * w], f1 = s1[2 * w + 1];
        uint32_t x[4], y[4];
        codes4(v0[w], x);
        codes4(v1[w], y);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          x[i] = hmul2(x[i], i < 2 ? e0 : f0);
          y[i] = hmul2(y[i], i < 2 ? e1 : f1);
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          mma_f16(o[t][2 * w], x[0], x[1], y[0], y[1], p[ks][t][0], p[ks][t][1]);
          mma_f16(o[t][2 * w + 1], x[2], x[3], y[2], y[3], p[ks][t][0], p[ks][t][1]);
        }
      }
    }
  }

  // The sums over the lanes of a head.
  __device__ __forceinline__ void finish() {
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) l[t][i] += __shfl_xor_sync(0xffffffffu, l[t][i], x);
  }
  __device__ __forceinline__ void store_part(float* out, float* pm, float* pl, int lane) const {
    const int r = lane >> 2, c = lane & 3;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int h = 8 * t + 2 * c;
      if (r == 0) {
        pm[h] = m[t][0], pm[h + 1] = m[t][1];
        pl[h] = l[t][0], pl[h + 1] = l[t][1];
      }
      float* d0 = out + h * AdCfg<D>::kStride + r;
      float* d1 = d0 + AdCfg<D>::kStride;
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        d0[16 * i] = o[t][i][0], d1[16 * i] = o[t][i][1];
        d0[16 * i + 8] = o[t][i][2], d1[16 * i + 8] = o[t][i][3];
      }
    }
  }
  __device__ __forceinline__ void store_out(const AdArgs& a, int b, int row, int lane) const {
    const int r = lane >> 2, c = lane & 3, hk = row / a.chunks, ch = row - hk * a.chunks;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int h = ch * 8 * NT + t * 8 + 2 * c + k;
        if (h >= a.G) continue;
        const float inv = l[t][k] != 0.0f ? 1.0f / l[t][k] : 0.0f;  // nothing seen: zeros
        uint16_t* dst = a.g.out + (size_t)b * a.g.ld_o + (size_t)(hk * a.G + h) * D + r;
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          dst[16 * i] = f32_to_bf16(o[t][i][k] * inv);
          dst[16 * i + 8] = f32_to_bf16(o[t][i][2 + k] * inv);
        }
      }
  }
};

// A position in the order of units.
struct AdCursor {
  int b, row, page, pages, len;
  __device__ __forceinline__ void load(const AdArgs& a) {
    len = ad_len(a.g, b);
    pages = (len + kPage - 1) / kPage;
  }
  // to the next unit; b == B past the last one
  __device__ __forceinline__ void next(const AdArgs& a) {
    if (++page < pages) return;
    page = 0;
    if (++row < a.rows) return;
    row = 0;
    do {
      if (++b >= a.g.B) return;
      load(a);
    } while (pages == 0);
  }
};

// A part's weight against the joined maximum; a part that saw nothing has none
// (its sum is 0), and one of NaN scores passes its NaN on.
__device__ __forceinline__ float ad_weight(float m, float l, float top) {
  return m == -INFINITY ? (l == 0.0f ? 0.0f : 1.0f) : ad_ex2(m - top);
}
// Four channels of a row's output.
__device__ __forceinline__ void ad_store4(const AdArgs& a, int seg, int hn, int h, int d, int D, float4 o, float l) {
  const int b = seg / a.rows, row = seg - b * a.rows, hk = row / a.chunks, head = (row - hk * a.chunks) * hn + h;
  const float inv = l != 0.0f ? 1.0f / l : 0.0f;  // nothing seen: zeros
  *reinterpret_cast<uint2*>(a.g.out + (size_t)b * a.g.ld_o + (size_t)(hk * a.G + head) * D + d) =
      make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
}
// Heads of a row that exist.
__device__ __forceinline__ int ad_heads(const AdArgs& a, int seg, int hn) {
  return min(hn, a.G - (seg % a.rows) % a.chunks * hn);
}

template <int D, int NT>
__global__ void __launch_bounds__(kAdWarps * 32, 1) attn_decode_kernel(const AdArgs a) {
  using C = AdCfg<D>;
  constexpr int S = C::kStages, HN = 8 * NT, REC = ad_record<D, HN>();
  static_assert(kAdParts * HN <= kAdWarps * 32 && kAdParts <= 32, "a thread per part and head, a lane per part");
  static_assert(REC * 4 <= C::kRing && S <= 6, "a record lies in its warp's ring");
  extern __shared__ __align__(128) uint8_t smem[];
  AdShared* sh = reinterpret_cast<AdShared*>(smem + kAdWarps * C::kRing);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, cta = blockIdx.x;
  if (lane == 0) {
    for (int s = 0; s < S; ++s) mbar_init(&sh->full[warp][s], 1);
    sh->meta[2 * warp].seg = sh->meta[2 * warp + 1].seg = -1;
    fence_mbar_init();
  }
  if (tid < 2) sh->cta_seg[tid] = -1;
  pdl_wait();
  pdl_trigger();
  const int B = a.g.B;
  // ---- the span and its runs: prefix sums of the sequences' units (the host made sure that 32 bits hold them)
  const int per = (B + kAdWarps * 32 - 1) / (kAdWarps * 32), b0 = min(B, tid * per), b1 = min(B, b0 + per);
  int mine = 0;
  for (int b = b0; b < b1; ++b) mine += ad_pages(a.g, b);
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
  for (int w = 0; w < kAdWarps; ++w) {
    if (w < warp) pre += sh->scan[w];
    total += sh->scan[w];
  }
  pre *= a.rows;
  total *= a.rows;
  int s0, s1;
  if (a.by_row) {  // row cta % rows of sequence cta / rows
    const int b = cta / a.rows;
    if (tid == b / per) {
      int at = pre;
      for (int k = b0; k < b; ++k) at += ad_pages(a.g, k) * a.rows;
      const int n = ad_pages(a.g, b);
      sh->run0[0] = at + (cta - b * a.rows) * n;
      sh->run0[1] = sh->run0[0] + n;
    }
    __syncthreads();
    s0 = sh->run0[0];
    s1 = sh->run0[1];
    __syncthreads();
  } else {
    // at least a unit for every warp: the CTAs without work are the last ones
    const int nc = min(a.nc, (total + kAdWarps - 1) / kAdWarps), q = nc ? total / nc : 0, extra = total - q * nc;
    s0 = cta < nc ? q * cta + min(cta, extra) : total;
    s1 = cta < nc ? s0 + q + (cta < extra ? 1 : 0) : total;
  }
  {
    // run w: its share of the span, the first ones a unit longer
    const int q = (s1 - s0) / kAdWarps, extra = s1 - s0 - q * kAdWarps;
    if (tid <= kAdWarps) sh->run0[tid] = s0 + q * tid + min(tid, extra);
    int at = pre;
    for (int b = b0; b < b1 && at < s1; ++b) {
      const int n = ad_pages(a.g, b) * a.rows;
      if (at + n > s0)
        for (int w = 0; w < kAdWarps; ++w) {
          const int u = s0 + q * w + min(w, extra);
          if (u >= at && u < at + n) {
            sh->run_b[w] = b;
            sh->run_base[w] = at;
          }
        }
      at += n;
    }
  }
  // rows of sequences without tokens
  for (int b = cta; b < B; b += gridDim.x)
    if (ad_len(a.g, b) == 0)
      for (int i = tid; i < a.g.H * D / 8; i += kAdWarps * 32)
        *reinterpret_cast<uint4*>(a.g.out + (size_t)b * a.g.ld_o + 8 * i) = make_uint4(0u, 0u, 0u, 0u);
  __syncthreads();

  // ---- this warp's run
  uint8_t* ring = smem + warp * C::kRing;
  const int u0 = sh->run0[warp], u1 = sh->run0[warp + 1], n = u1 - u0;
  if (n > 0) {
    AdCursor cur;
    cur.b = sh->run_b[warp];
    cur.load(a);
    const int in = u0 - sh->run_base[warp];
    cur.row = in / cur.pages;
    cur.page = in - cur.row * cur.pages;
    AdCursor ahead = cur;
    const uint64_t pol = a.chunks > 1 ? policy_evict_normal() : policy_evict_first();
    auto fetch = [&](int i) {  // unit i of the run into its stage
      const int st = i % S;
      if (lane == 0) {
        const int page = a.g.c.table[(size_t)ahead.b * a.g.c.ld_table + ahead.page];
        const bool ok = page >= 0 && page < a.g.c.n_pages;
        sh->ok[warp][st] = ok;
        if (ok) {
          mbar_arrive_expect_tx(&sh->full[warp][st], C::kUnit);
          bulk_g2s(ring + st * C::kUnit, a.g.c.pages + ((size_t)page * a.g.c.Hkv + ahead.row / a.chunks) * C::kUnit,
                   C::kUnit, &sh->full[warp][st], pol);
        } else {
          M2_RECORD_ARG(g_status);
          mbar_arrive(&sh->full[warp][st]);
        }
      }
      ahead.next(a);
    };
    int fetched = 0;
    for (; fetched < S && fetched < n; ++fetched) fetch(fetched);
    AdRow<D, NT> row;
    row.start(a, cur.b, cur.row, lane);
    int first_page = cur.page;  // of the row's part in this run
    int row_at = u0 - cur.page;      // the row's first unit
    bool dead = false;
    for (int i = 0; i < n; ++i) {
      const int st = i % S;
      if (!__all_sync(0xffffffffu, mbar_wait(&sh->full[warp][st], (i / S) & 1))) {
        dead = true;
        break;
      }
      if (sh->ok[warp][st]) row.unit(ring + st * C::kUnit, min(kPage, cur.len - cur.page * kPage), lane);
      fence_proxy_async();  // the scales' place is written anew by the next copy
      __syncwarp();         // the stage is read
      if (fetched < n) fetch(fetched++);
      const bool ends = cur.page + 1 == cur.pages;
      if (ends || i + 1 == n) {  // the row leaves this warp
        row.finish();
        if (ends && first_page == 0) {
          row.store_out(a, cur.b, cur.row, lane);
        } else {
          const int slot = i + 1 == n ? 1 : 0;
          // the last part goes into the ring (free by now), an earlier one through L2
          row.store_part(slot ? reinterpret_cast<float*>(ring) : a.warp_part + (size_t)(cta * kAdWarps + warp) * REC,
                         sh->part_m[2 * warp + slot], sh->part_l[2 * warp + slot], lane);
          if (lane == 0) {
            AdMeta& mt = sh->meta[2 * warp + slot];
            mt.seg = cur.b * a.rows + cur.row;
            mt.before = row_at < s0;
            mt.after = row_at + cur.pages > s1;
          }
        }
        if (i + 1 < n) {
          cur.next(a);
          first_page = 0;
          row_at = u0 + i + 1;
          row.start(a, cur.b, cur.row, lane);
        }
      } else {
        ++cur.page;
      }
    }
    if (dead) {  // every copy of this warp has landed before the CTA goes on
      for (int i = max(0, fetched - S); i < fetched; ++i)
        if (!mbar_drain(&sh->full[warp][i % S], (i / S) & 1)) break;
    }
  }
  __syncthreads();

  // ---- rows cut between warps
  const int seg_e = lane < kAdParts ? sh->meta[lane].seg : -1;
  const uint32_t same = __match_any_sync(0xffffffffu, seg_e);  // entry `lane`: all parts of its row
  const uint32_t lead = __ballot_sync(0xffffffffu, seg_e >= 0 && (same & ((1u << lane) - 1)) == 0);
  const int nrows = __popc(lead);
  {
    // a thread per (part, head): those of a row's first part weigh its parts
    const int e = tid / HN, h = tid - e * HN;
    const uint32_t parts = __shfl_sync(0xffffffffu, same, e & 31);
    if (e < kAdParts && (lead >> e & 1)) {
      float top = -INFINITY, l = 0.0f;
      for (uint32_t y = parts; y; y &= y - 1) top = fmaxf(top, sh->part_m[__ffs(y) - 1][h]);
      for (uint32_t y = parts; y; y &= y - 1) {
        const int x = __ffs(y) - 1;
        const float w = ad_weight(sh->part_m[x][h], sh->part_l[x][h], top);
        l += sh->part_l[x][h] * w;
        sh->part_m[x][h] = w;
      }
      const int k = __popc(lead & ((1u << e) - 1));
      sh->row_l[k][h] = l;
      sh->row_parts[k] = parts;
      const AdMeta& mt = sh->meta[e];
      if (mt.before || mt.after) {  // cut between CTAs too
        float* rec = a.cta_part + (size_t)(2 * cta + (mt.before ? 0 : 1)) * REC;
        rec[h] = top;
        rec[HN + h] = l;
        if (h == 0) sh->cta_seg[mt.before ? 0 : 1] = mt.seg;
      }
    }
  }
  __syncthreads();
  for (int i = tid; i < nrows * (HN * D / 4); i += kAdWarps * 32) {
    const int k = i / (HN * D / 4), h = i / (D / 4) % HN, d = i % (D / 4) * 4;
    uint32_t parts = sh->row_parts[k];
    const AdMeta& mt = sh->meta[__ffs(parts) - 1];
    if (h >= ad_heads(a, mt.seg, HN)) continue;
    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    while (parts) {
      // four parts at a time, their loads together
      float4 v[4];
      float w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int x = parts ? __ffs(parts) - 1 : -1;
        parts &= parts - 1;
        w[j] = 0.0f;
        v[j] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (x >= 0) {
          w[j] = sh->part_m[x][h];
          v[j] = x & 1 ? *reinterpret_cast<const float4*>(smem + (x >> 1) * C::kRing + (h * C::kStride + d) * 4)
                       : *reinterpret_cast<const float4*>(a.warp_part + (size_t)(cta * kAdWarps + (x >> 1)) * REC +
                                                          h * C::kStride + d);
        }
      }
#pragma unroll
      for (int j = 0; j < 4; ++j)
        o.x = fmaf(v[j].x, w[j], o.x), o.y = fmaf(v[j].y, w[j], o.y), o.z = fmaf(v[j].z, w[j], o.z),
        o.w = fmaf(v[j].w, w[j], o.w);
    }
    if (mt.before || mt.after)
      *reinterpret_cast<float4*>(a.cta_part + (size_t)(2 * cta + (mt.before ? 0 : 1)) * REC + 2 * HN + h * C::kStride +
                                 d) = o;
    else
      ad_store4(a, mt.seg, HN, h, d, D, o, sh->row_l[k][h]);
  }
  if (tid < 2 && !a.by_row) a.cta_seg[2 * cta + tid] = sh->cta_seg[tid];
}

// Rows cut between CTAs: block (c, h) joins head h of the row that began in span
// c and goes on.  D/4 threads hold four channels each; the parts are dealt out
// over groups of them and joined through shared memory.  The first parts are
// loaded before it is known how many there are (any span's record may be read),
// and the blocks are small enough to wait on the SMs for the spans' end.
constexpr int kAcThreads = 128;
template <int D, int NT>
__global__ void __launch_bounds__(kAcThreads, 16) attn_decode_combine_kernel(const AdArgs a) {
  constexpr int HN = 8 * NT, REC = ad_record<D, HN>(), ST = AdCfg<D>::kStride, P = D / 4, GR = kAcThreads / P;
  __shared__ float pm[GR], pl[GR];
  __shared__ float4 po[kAcThreads];
  pdl_wait();
  pdl_trigger();
  const int c = blockIdx.x, h = blockIdx.y, tid = threadIdx.x, g = tid / P, d = tid % P * 4;
  const int seg = a.cta_seg[2 * c + 1];
  auto load = [&](int y, float& m, float& l, float4& o) {
    const float* r = a.cta_part + (size_t)(y == 0 ? 2 * c + 1 : 2 * min(c + y, a.nc - 1)) * REC;
    m = r[h], l = r[HN + h];
    o = *reinterpret_cast<const float4*>(r + 2 * HN + h * ST + d);
  };
  float m, l;
  float4 o;
  load(g, m, l, o);
  int k = 1;  // parts: this span's, then those of the spans that the row goes on through
  for (int x = c + 1; x < a.nc; x += kAcThreads) {
    const int n = __syncthreads_count(x + tid < a.nc && a.cta_seg[2 * (x + tid)] == seg);
    k += n;
    if (n < kAcThreads) break;
  }
  if (seg < 0 || h >= ad_heads(a, seg, HN)) return;
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
    ad_store4(a, seg, HN, h, d, D, t, sum);
  }
}

// ------------------------------------------------------------------ host

static int ad_tiles(int G) { return G <= 8 ? 1 : 2; }
static size_t ad_record_bytes(int D, int nt) { return (size_t)(2 * 8 * nt + 8 * nt * (D + 4)) * 4; }

size_t attn_decode_ws_bytes(int32_t B, int32_t H, int32_t Hkv, int32_t D) {
  (void)B;
  const size_t n = num_sms();
  return n * (kAdWarps + 2) * ad_record_bytes(D, ad_tiles(H / Hkv)) + (n * 2 * 4 + 255) / 256 * 256;
}

template <int D, int NT>
static cudaError_t launch_ad(const AttnDecodeArgs& g, cudaStream_t s) {
  static int done_mask[64] = {0};
  constexpr int smem = kAdWarps * AdCfg<D>::kRing + (int)sizeof(AdShared);
  static_assert(smem <= 232448, "shared memory");
  AdArgs a;
  a.g = g;
  a.G = g.H / g.c.Hkv;
  a.chunks = (a.G + 8 * NT - 1) / (8 * NT);
  a.rows = g.c.Hkv * a.chunks;
  // Few rows in a narrow table: a CTA takes a whole row, and nothing is left to combine.
  // The table's width is what the host knows: lengths are read on the device, and a
  // captured step has to serve while they grow.  Measured, whole rows and spans, us
  // by tokens: 8 rows of 128 (32 query heads) 64: 5.9 and 8.2, 700: 9.3 and 10.7, 1500: 11.9
  // and 11.6, 2048 (32 pages): 13.7 and 11.4; 152 rows 700: 10.0 and 12.7, 2048: 17.2 and
  // 18.5; 16 rows of 64 700: 8.0 and 9.7, 2048: 10.7 and 9.7.
  a.by_row = (int64_t)g.B * a.rows <= num_sms() && g.c.ld_table <= 32;
  a.nc = a.by_row ? g.B * a.rows : num_sms();
  const size_t rec = ad_record<D, 8 * NT>(), n = num_sms();
  a.cta_seg = static_cast<int32_t*>(g.ws);
  a.warp_part = reinterpret_cast<float*>(static_cast<uint8_t*>(g.ws) + (n * 2 * 4 + 255) / 256 * 256);
  a.cta_part = a.warp_part + n * kAdWarps * rec;
  auto kern = attn_decode_kernel<D, NT>;
  cudaError_t e = set_smem_once((const void*)kern, smem, done_mask);
  if (e != cudaSuccess) return e;
  trace_pre(K_ATTN_DECODE, s);
  e = launch_k(kern, dim3(a.nc), dim3(kAdWarps * 32), smem, s, true, a);
  trace_post(K_ATTN_DECODE, s);
  if (e != cudaSuccess || a.by_row) return e;
  trace_pre(K_ATTN_COMBINE, s);
  e = launch_k(attn_decode_combine_kernel<D, NT>, dim3(a.nc, a.G < 8 * NT ? a.G : 8 * NT), dim3(kAcThreads), 0, s,
               true, a);
  trace_post(K_ATTN_COMBINE, s);
  return e;
}

cudaError_t launch_attn_decode(const AttnDecodeArgs& a, cudaStream_t s) {
  const int nt = ad_tiles(a.H / a.c.Hkv);
  if (a.c.D == 128) return nt == 1 ? launch_ad<128, 1>(a, s) : launch_ad<128, 2>(a, s);
  return nt == 1 ? launch_ad<64, 1>(a, s) : launch_ad<64, 2>(a, s);
}

int status_attn_decode(int clear) { return tu_status(clear); }
cudaError_t wait_limit_attn_decode(long long cycles) { return tu_set_wait_limit(cycles); }

}  // namespace m2
