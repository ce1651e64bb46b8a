// k_kv4.cu -- head norm with rotation, and the paged 4-bit cache's writes and
// reads (include/mamba2.h gives the formulas and the page's layout).
#include <cuda_runtime.h>
#include <stdint.h>

#include "m2_common.cuh"
#include "m2_kernels.h"
#include "m2_kv4.cuh"

namespace m2 {

// ------------------------------------------------------------------ head norm and rotation
//
// A warp takes a row, or a part of its heads when there are few rows: a head is
// D/8 lanes of 8 channels, so that the warp holds 256/D heads (a group) at a
// time.  The angles of the row are worked out once, by the warp's lanes, into
// shared memory: p * step mod 2^64 is the angle in turns, exactly, and only its
// top 32 bits (a signed fraction of a half turn) enter the fp32 functions.
// Bound: HBM, one read and one write of every row, and as close the issue rate.
// Measured at 8192 rows of 32 + 8 heads of 128: 31 to 33 us for every form of the
// rotation, 5.1 to 5.5 TB/s.
constexpr int kRopeWarps = 8, kRopeBatch = 4;

// Cosines and sines of the row's angles.
__device__ __forceinline__ void rope_angles(const RopeArgs& a, int64_t row, int lane, float2* cs) {
  const int64_t pos = a.pos[row];
  for (int f = lane; f < a.rot / 2; f += 32) {
    const uint64_t t = (uint64_t)pos * a.step[f];
    float s, c;
    sincospif((float)(int32_t)(t >> 32) * 4.656612873077393e-10f, &s, &c);  // 2^-31
    cs[f] = make_float2(c, s);
  }
  __syncwarp();
}

__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  uint64_t d;
  asm("{\n\t.reg .b64 ra, rb;\n\tmov.b64 ra, {%1, %2};\n\tmov.b64 rb, {%3, %4};\n\tmul.rn.f32x2 %0, ra, rb;\n\t}"
      : "=l"(d)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(d));
  return r;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  uint64_t d;
  asm("{\n\t.reg .b64 ra, rb, rc;\n\tmov.b64 ra, {%1, %2};\n\tmov.b64 rb, {%3, %4};\n\tmov.b64 rc, {%5, %6};\n\t"
      "fma.rn.f32x2 %0, ra, rb, rc;\n\t}"
      : "=l"(d)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(d));
  return r;
}

// A lane's 8 channels are 4 pairs (a, b) of the rotation, so that nothing but the
// sum of squares crosses lanes: channels 4 l .. 4 l + 3 and those rot/2 on (pair i =
// (i, i + rot/2)) or 8 l .. 8 l + 7 (NEXT: pair i = (2 i, 2 i + 1)), as are those of
// the lanes past the rotated channels (PART).  Weights and angles meet once a row:
// with w' = w cos, w" = w sin of the pair,
//   y_a = r (a w'_a - b w"_b),  y_b = r (b w'_b + a w"_a),  r = 1 / sqrt(mean + eps).
template <int D, bool NEXT, bool PART>
__global__ void __launch_bounds__(kRopeWarps * 32, 4) qk_norm_rope_kernel(const RopeArgs a, int parts) {
  constexpr int LH = D / 8, HW = 32 / LH;  // lanes a head, heads a group
  __shared__ float2 turn[kRopeWarps][D / 2];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, l = lane % LH, sub = lane / LH;
  const int64_t id = (int64_t)blockIdx.x * kRopeWarps + warp, row = id / parts;
  pdl_wait();
  pdl_trigger();
  if (row >= a.T) return;
  const bool turns = !PART || 8 * l < a.rot;
  const int ac = NEXT || !turns ? 8 * l : 4 * l;                       // the lane's first channel
  const int bd = NEXT || !turns ? 4 : (PART ? a.rot : D) / 2;  // and its second four's distance
  if (!PART || a.rot) rope_angles(a, row, lane, turn[warp]);
  float2 cs[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) cs[i] = turns ? turn[warp][4 * l + i] : make_float2(1.0f, 0.0f);
  const int gq = (a.H + HW - 1) / HW, groups = gq + (a.Hkv + HW - 1) / HW;
  const int per = (groups + parts - 1) / parts, g0 = (int)(id - row * parts) * per, g1 = min(groups, g0 + per);
  // two words of a lane's channels -> the a and b of two pairs
  auto pairs = [](uint32_t u, uint32_t v, float2& x, float2& y) {
    x = NEXT ? make_float2(bf16lo(u), bf16lo(v)) : make_float2(bf16lo(u), bf16hi(u));
    y = NEXT ? make_float2(bf16hi(u), bf16hi(v)) : make_float2(bf16lo(v), bf16hi(v));
  };
  // the groups from `from` to `to` of n heads at in -> out
  auto run = [&](const uint16_t* in, uint16_t* out, const uint16_t* w, int n, int from, int to) {
    if (from >= to) return;
    float2 ca[2], sb[2], cb[2], sa[2];  // of channel pairs (0, 1), (2, 3): w'_a, -w"_b, w'_b, w"_a
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float2 wa = make_float2(1.0f, 1.0f), wb = wa;
      if (w) {
        const uint32_t u = *reinterpret_cast<const uint32_t*>(w + ac + (NEXT ? 4 * i : 2 * i));
        const uint32_t v = *reinterpret_cast<const uint32_t*>(w + ac + (NEXT ? 4 * i + 2 : bd + 2 * i));
        pairs(u, v, wa, wb);
      }
      const float2 c = make_float2(cs[2 * i].x, cs[2 * i + 1].x), s = make_float2(cs[2 * i].y, cs[2 * i + 1].y);
      ca[i] = mul2(wa, c), cb[i] = mul2(wb, c), sa[i] = mul2(wa, s), sb[i] = mul2(wb, make_float2(-s.x, -s.y));
    }
    const int64_t lane_at = (int64_t)sub * D + ac;
    in += lane_at, out += lane_at;
    for (int gb = from; gb < to; gb += kRopeBatch) {
      uint2 u[kRopeBatch], v[kRopeBatch];
#pragma unroll
      for (int k = 0; k < kRopeBatch; ++k) {
        u[k] = v[k] = make_uint2(0u, 0u);
        if (gb + k < to && (gb + k) * HW + sub < n) {
          const uint16_t* x = in + (gb + k) * (HW * D);
          if (NEXT) {
            const uint4 z = *reinterpret_cast<const uint4*>(x);
            u[k] = make_uint2(z.x, z.z), v[k] = make_uint2(z.y, z.w);
          } else {
            u[k] = *reinterpret_cast<const uint2*>(x);
            v[k] = *reinterpret_cast<const uint2*>(x + bd);
          }
        }
      }
#pragma unroll
      for (int k = 0; k < kRopeBatch; ++k) {
        float2 xa[2], xb[2];
        pairs(u[k].x, v[k].x, xa[0], xb[0]);
        pairs(u[k].y, v[k].y, xa[1], xb[1]);
        float r = 1.0f;
        if (w) {
          const float2 q = fma2(xa[0], xa[0], fma2(xa[1], xa[1], fma2(xb[0], xb[0], mul2(xb[1], xb[1]))));
          float ss = q.x + q.y;
#pragma unroll
          for (int o = LH / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
          r = rsqrtf(ss * (1.0f / D) + a.eps);
        }
        const float2 r2 = make_float2(r, r);
        float2 ya[2], yb[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          // (0 * Inf must not come from one channel into another that it does not turn with)
          const float2 pa = turns ? xa[i] : make_float2(0.0f, 0.0f), pb = turns ? xb[i] : make_float2(0.0f, 0.0f);
          ya[i] = mul2(fma2(xa[i], ca[i], mul2(pb, sb[i])), r2);
          yb[i] = mul2(fma2(xb[i], cb[i], mul2(pa, sa[i])), r2);
        }
        if (gb + k < to && (gb + k) * HW + sub < n) {
          uint16_t* d = out + (gb + k) * (HW * D);
          if (NEXT) {
            *reinterpret_cast<uint4*>(d) = make_uint4(pack_bf16x2(ya[0].x, yb[0].x), pack_bf16x2(ya[0].y, yb[0].y),
                                                      pack_bf16x2(ya[1].x, yb[1].x), pack_bf16x2(ya[1].y, yb[1].y));
          } else {
            *reinterpret_cast<uint2*>(d) = make_uint2(pack_bf16x2(ya[0].x, ya[0].y), pack_bf16x2(ya[1].x, ya[1].y));
            *reinterpret_cast<uint2*>(d + bd) = make_uint2(pack_bf16x2(yb[0].x, yb[0].y), pack_bf16x2(yb[1].x, yb[1].y));
          }
        }
      }
    }
  };
  run(a.q + row * a.ld_q, a.q_out + row * a.ld_qo, a.q_w, a.H, min(g0, gq), min(g1, gq));
  run(a.k + row * a.ld_k, a.k_out + row * a.ld_ko, a.k_w, a.Hkv, max(g0, gq) - gq, max(g1, gq) - gq);
}

cudaError_t launch_qk_norm_rope(const RopeArgs& a, cudaStream_t s) {
  const bool part = a.rot < a.D, next = a.interleaved && a.rot;
  // Few rows: a row's heads are dealt out over several warps, until every SM has
  // 16 (64 rows of 32 + 8 heads of 128: one batch of loads a warp).
  int parts = 1;
  while (parts < 8 && (int64_t)a.T * parts < 16ll * num_sms()) parts *= 2;
  const dim3 grid((unsigned)(((int64_t)a.T * parts + kRopeWarps - 1) / kRopeWarps)), block(kRopeWarps * 32);
  void (*const kernels[2][2][2])(RopeArgs, int) = {
      {{qk_norm_rope_kernel<64, false, false>, qk_norm_rope_kernel<64, false, true>},
       {qk_norm_rope_kernel<64, true, false>, qk_norm_rope_kernel<64, true, true>}},
      {{qk_norm_rope_kernel<128, false, false>, qk_norm_rope_kernel<128, false, true>},
       {qk_norm_rope_kernel<128, true, false>, qk_norm_rope_kernel<128, true, true>}}};
  auto k = kernels[a.D == 128][next][part];
  trace_pre(K_QK_NORM_ROPE, s);
  const cudaError_t e = launch_k(k, grid, block, 0, s, true, a, parts);
  trace_post(K_QK_NORM_ROPE, s);
  return e;
}

// ------------------------------------------------------------------ cache rows
//
// A warp's task is 8 tokens (positions 8b .. 8b+7) of one kv head: there the
// codes of K (8 rows) and of V (one block of the layout), and both kinds of
// scales, are four contiguous runs of a page.  Codes pass through shared memory
// between the layout's order and that of the rows, so that rows and runs are
// both read and written 16 bytes a lane.  Sequence i's tasks start at
// block_base(i): a closed form that leaves room for blocks cut at both ends.
// Bound: HBM (2 bytes a value of the rows, 0.56 of the cache) for the reading.  The
// writing fills no unit (ALU 59%, issue 55%, DRAM 25% at four chunks): its chain of
// loads, quantizing (20 instructions a value) and stores is what it waits for, and
// with few rows both are two launches.  Measured at 8 heads of 128, as graph replays:
// 16 sequences of 64..512 new tokens written and read back in 15 us (21 a call from
// Python), four of 500..2048 after 1000..12000 in 43 us (5.3 TB/s), of it 33 the
// reading; one new token of 1, 16, 64, 256 sequences written in 3.5, 3.8, 4.2, 9.4 us.
__device__ __forceinline__ int64_t block_base(const Kv4RowsArgs& a, int i) { return a.cu[i] / 8 + 2ll * i; }
static int64_t block_count(const Kv4RowsArgs& a) { return a.cu[a.nseq] / 8 + 2ll * a.nseq; }

constexpr int kRowWarps = 8;
struct RowTask {
  int seq, h;
  int64_t first, end;  // positions of the call's tokens of the sequence
  int64_t tok;         // the block's first position
  int page;            // the table's entry: loaded here, looked at when it is needed
  bool any;            // a token of the block belongs to the call
};
__device__ __forceinline__ RowTask row_task(const Kv4RowsArgs& a, int64_t tasks) {
  RowTask t;
  t.any = false;
  const int64_t id = (int64_t)blockIdx.x * kRowWarps + (threadIdx.x >> 5);
  if (id >= tasks) return t;
  // (a division of 64 bits is a good part of a warp's instructions)
  const int64_t p = tasks <= UINT32_MAX ? (int64_t)((uint32_t)id / (uint32_t)a.c.Hkv) : id / a.c.Hkv;
  t.h = (int)(id - p * a.c.Hkv);
  int lo = 0, hi = a.nseq;  // the last i with block_base(i) <= p
  while (hi - lo > 1) {
    const int m = (lo + hi) / 2;
    if (block_base(a, m) <= p)
      lo = m;
    else
      hi = m;
  }
  t.seq = lo;
  t.first = a.pos ? a.pos[lo] : 0;
  t.end = t.first + a.cu[lo + 1] - a.cu[lo];
  const int64_t blk = (t.first >> 3) + (p - block_base(a, lo));  // from the block of `first` (also below zero) on
  t.tok = 8 * blk;
  if (t.tok >= t.end || t.end == t.first || t.first < -(1 << 30)) return t;  // (the last: an idle slot)
  t.any = true;
  const int64_t pg = blk >= 0 ? blk / (kPage / 8) : a.c.ld_table;
  t.page = pg < a.c.ld_table ? a.c.table[(size_t)lo * a.c.ld_table + pg] : -1;
  return t;
}
// The bytes of the task's page and head; null, and the device status, if the table does not give one.
__device__ __forceinline__ uint8_t* row_page(const Kv4RowsArgs& a, const RowTask& t, int unit) {
  if (t.page >= 0 && t.page < a.c.n_pages) return a.c.pages + ((size_t)t.page * a.c.Hkv + t.h) * unit;
  M2_RECORD_ARG(g_status);
  return nullptr;
}

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// Scale byte and codes (8 nibbles, channel order) of this lane's half group;
// the group's other half is on the neighbouring lane.
__device__ __forceinline__ uint32_t quantize8(const uint4& v, uint32_t& byte) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  // bf16 magnitudes compare as integers, and a NaN is above everything
  uint32_t m2 = max_u16x2(max_u16x2(w[0] & 0x7FFF7FFFu, w[1] & 0x7FFF7FFFu),
                          max_u16x2(w[2] & 0x7FFF7FFFu, w[3] & 0x7FFF7FFFu));
  m2 = max_u16x2(m2, __shfl_xor_sync(0xffffffffu, m2, 1));
  const uint32_t m = max(m2 & 0xFFFFu, m2 >> 16);
  const bool nan = m > 0x7F80u;
  byte = nan ? 0xFFu : kv4_scale_byte(__uint_as_float(m << 16));
  float inv;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(kv4_scale(byte)));
  if (nan || byte == 0) inv = 0.0f;
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) c[i] = kv4_codes(make_float2(bf16lo(w[i]), bf16hi(w[i])), inv);
  return __byte_perm(__byte_perm(c[0], c[1], 0x0040), __byte_perm(c[2], c[3], 0x0040), 0x5410);
}

// The low 4 nibbles, one a byte.
__device__ __forceinline__ uint32_t spread4(uint32_t x) {
  x = (x & 0xFFu) | (x & 0xFF00u) << 8;
  return (x | x << 4) & 0x0F0F0F0Fu;
}

template <int D>
__global__ void __launch_bounds__(kRowWarps * 32) kv4_append_kernel(const Kv4RowsArgs a, int64_t tasks) {
  using L = Kv4Block<D>;
  constexpr int LT = D / 8, TI = 32 / LT, RUN = 4 * D;  // lanes a token, tokens at a time, bytes of 8 tokens' codes
  __shared__ __align__(16) uint8_t buf[kRowWarps][2 * RUN + D];  // K codes, V codes, K scales, V scales
  pdl_wait();
  pdl_trigger();
  const RowTask t = row_task(a, tasks);
  if (!t.any) return;
  const int lane = threadIdx.x & 31, l = lane % LT;
  uint8_t* kc = buf[threadIdx.x >> 5];
  uint8_t* vc = kc + RUN;
  uint8_t* ks = vc + RUN;
  uint8_t* vs = ks + D / 2;
  const int t0 = (int)max((int64_t)0, t.first - t.tok), t1 = (int)min((int64_t)8, t.end - t.tok);  // new tokens of the block
  uint4 x[8 / TI], y[8 / TI];
#pragma unroll
  for (int i = 0; i < 8 / TI; ++i) {
    const int n = i * TI + lane / LT;
    x[i] = y[i] = make_uint4(0u, 0u, 0u, 0u);
    if (n >= t0 && n < t1) {
      const size_t row = a.cu[t.seq] + (t.tok + n - t.first);
      x[i] = *reinterpret_cast<const uint4*>(a.k + row * a.ld_k + t.h * D + 8 * l);
      y[i] = *reinterpret_cast<const uint4*>(a.v + row * a.ld_v + t.h * D + 8 * l);
    }
  }
#pragma unroll
  for (int i = 0; i < 8 / TI; ++i) {
    const int n = i * TI + lane / LT, g = l / 2, c = 2 * (l & 1);
    uint32_t kb, vb;
    const uint32_t k8 = quantize8(x[i], kb), v8 = quantize8(y[i], vb);
    *reinterpret_cast<uint16_t*>(kc + L::k(n, g, c) - L::kK) = (uint16_t)k8;
    *reinterpret_cast<uint16_t*>(kc + L::k(n, g, c + 1) - L::kK) = (uint16_t)(k8 >> 16);
    if (l % 2 == 0) {
      ks[L::ks(n, g) - L::kKs] = (uint8_t)kb;
      vs[L::vs(n, g) - L::kVs] = (uint8_t)vb;
    }
    // channel 8l + r is nibble r: the even token's lane writes r = 0..3 of the pair's bytes, the odd one's 4..7
    const uint32_t other = __shfl_xor_sync(0xffffffffu, v8, LT);
    const uint32_t even = n & 1 ? other >> 16 : v8, odd = n & 1 ? v8 >> 16 : other;
    const uint32_t b = spread4(even) | spread4(odd) << 4;
#pragma unroll
    for (int j = 0; j < 4; ++j) vc[L::v(n, l, (n & 1) * 4 + j) - L::kV] = (uint8_t)(b >> (8 * j));
  }
  __syncwarp();
  uint8_t* page = row_page(a, t, L::kBytes);
  if (!page) return;
  const int tk = (int)(t.tok % kPage);
  if (lane < RUN / 16) {
    const uint4 k = *reinterpret_cast<const uint4*>(kc + 16 * lane);
    uint4 v = *reinterpret_cast<const uint4*>(vc + 16 * lane);
    uint8_t* kd = page + L::k(tk, 0, 0) + 16 * lane;
    uint8_t* vd = page + L::v(tk, 0, 0) + 16 * lane;
    const int n = 16 * lane / (D / 2);
    if (n >= t0 && n < t1) *reinterpret_cast<uint4*>(kd) = k;
    // V bytes hold two tokens: the other's nibbles stay when only one is new.  16 bytes are one pair's (D = 128)
    // or two pairs' (D = 64).
    uint32_t keep[2];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int p = (16 * lane + 8 * q) / (D / 8) % 4;
      keep[q] = (2 * p >= t0 && 2 * p < t1 ? 0u : 0x0F0F0F0Fu) | (2 * p + 1 >= t0 && 2 * p + 1 < t1 ? 0u : 0xF0F0F0F0u);
    }
    if ((keep[0] & keep[1]) != 0xFFFFFFFFu) {
      if (keep[0] | keep[1]) {
        const uint4 o = *reinterpret_cast<const uint4*>(vd);
        v.x = (o.x & keep[0]) | (v.x & ~keep[0]);
        v.y = (o.y & keep[0]) | (v.y & ~keep[0]);
        v.z = (o.z & keep[1]) | (v.z & ~keep[1]);
        v.w = (o.w & keep[1]) | (v.w & ~keep[1]);
      }
      *reinterpret_cast<uint4*>(vd) = v;
    }
  }
  // scales, 4 bytes a lane: of one token (K), of a pair (V: bytes 0, 1 of the even token, 2, 3 of the odd one)
  if (lane < D / 8) {
    const int n = 4 * lane / (D / 16), p = 4 * lane / (D / 8);
    if (n >= t0 && n < t1)
      *reinterpret_cast<uint32_t*>(page + L::ks(tk, 0) + 4 * lane) = *reinterpret_cast<const uint32_t*>(ks + 4 * lane);
    const bool e = 2 * p >= t0 && 2 * p < t1, o = 2 * p + 1 >= t0 && 2 * p + 1 < t1;
    uint8_t* d = page + L::vs(tk, 0) + 4 * lane;
    if (e) *reinterpret_cast<uint16_t*>(d) = *reinterpret_cast<const uint16_t*>(vs + 4 * lane);
    if (o) *reinterpret_cast<uint16_t*>(d + 2) = *reinterpret_cast<const uint16_t*>(vs + 4 * lane + 2);
  }
}

// A byte's two codes times their scales (f16): 6 significant bits, exact in f16 and in what is made of it.
__device__ __forceinline__ float2 kv4_value2(uint32_t codes, uint32_t scale2) {
  const uint32_t h = kv4_f16x2(codes);
  return __half22float2(__hmul2(*reinterpret_cast<const __half2*>(&h), *reinterpret_cast<const __half2*>(&scale2)));
}

template <int D>
__global__ void __launch_bounds__(kRowWarps * 32) kv4_gather_kernel(const Kv4RowsArgs a, int64_t tasks) {
  using L = Kv4Block<D>;
  constexpr int LT = D / 8, TI = 32 / LT, RUN = 4 * D;
  __shared__ __align__(16) uint8_t buf[kRowWarps][2 * RUN + D];
  pdl_wait();
  pdl_trigger();
  const RowTask t = row_task(a, tasks);
  uint8_t* page = t.any ? row_page(a, t, L::kBytes) : nullptr;
  if (!page) return;
  const int lane = threadIdx.x & 31, l = lane % LT;
  uint8_t* kc = buf[threadIdx.x >> 5];
  uint8_t* vc = kc + RUN;
  uint8_t* ks = vc + RUN;
  uint8_t* vs = ks + D / 2;
  const int tk = (int)(t.tok % kPage);
  if (lane < RUN / 16) {
    *reinterpret_cast<uint4*>(kc + 16 * lane) = *reinterpret_cast<const uint4*>(page + L::k(tk, 0, 0) + 16 * lane);
    *reinterpret_cast<uint4*>(vc + 16 * lane) = *reinterpret_cast<const uint4*>(page + L::v(tk, 0, 0) + 16 * lane);
  }
  if (lane < D / 8) {
    *reinterpret_cast<uint32_t*>(ks + 4 * lane) = *reinterpret_cast<const uint32_t*>(page + L::ks(tk, 0) + 4 * lane);
    *reinterpret_cast<uint32_t*>(vs + 4 * lane) = *reinterpret_cast<const uint32_t*>(page + L::vs(tk, 0) + 4 * lane);
  }
  __syncwarp();
  // A lane takes 8 channels of a token pair, whose values share bytes.
#pragma unroll
  for (int i = 0; i < 4 / TI; ++i) {
    const int n = 2 * (i * TI + lane / LT), g = l / 2, c = 2 * (l & 1);
    if (t.tok + n >= t.end) continue;
    const bool both = t.tok + n + 1 < t.end;
    const size_t row = a.cu[t.seq] + t.tok + n;
    uint16_t* k = a.k + row * a.ld_k + t.h * D + 8 * l;
    uint16_t* v = a.v + row * a.ld_v + t.h * D + 8 * l;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t sk = (uint32_t)ks[L::ks(n + h, g) - L::kKs] * 0x00800080u;  // f16 bits, twice
      const uint32_t k0 = *reinterpret_cast<const uint16_t*>(kc + L::k(n + h, g, c) - L::kK);
      const uint32_t k1 = *reinterpret_cast<const uint16_t*>(kc + L::k(n + h, g, c + 1) - L::kK);
      uint32_t w[4];
      const float2 x0 = kv4_value2(k0, sk), x1 = kv4_value2(k0 >> 8, sk), x2 = kv4_value2(k1, sk),
                   x3 = kv4_value2(k1 >> 8, sk);
      w[0] = pack_bf16x2(x0.x, x0.y);
      w[1] = pack_bf16x2(x1.x, x1.y);
      w[2] = pack_bf16x2(x2.x, x2.y);
      w[3] = pack_bf16x2(x3.x, x3.y);
      if (h == 0 || both) *reinterpret_cast<uint4*>(k + h * a.ld_k) = make_uint4(w[0], w[1], w[2], w[3]);
    }
    const uint8_t* vsp = vs + L::vs(n, g) - L::kVs;  // the odd token's is 2 bytes on
    const uint32_t sv = (uint32_t)vsp[0] << 7 | (uint32_t)vsp[2] << 23;
    uint32_t w0[4], w1[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 x = kv4_value2(vc[L::v(n, l, 2 * j) - L::kV], sv), y = kv4_value2(vc[L::v(n, l, 2 * j + 1) - L::kV], sv);
      w0[j] = pack_bf16x2(x.x, y.x);
      w1[j] = pack_bf16x2(x.y, y.y);
    }
    *reinterpret_cast<uint4*>(v) = make_uint4(w0[0], w0[1], w0[2], w0[3]);
    if (both) *reinterpret_cast<uint4*>(v + a.ld_v) = make_uint4(w1[0], w1[1], w1[2], w1[3]);
  }
}

static cudaError_t launch_rows(void (*k128)(Kv4RowsArgs, int64_t), void (*k64)(Kv4RowsArgs, int64_t), int id,
                               const Kv4RowsArgs& a, cudaStream_t s) {
  const int64_t tasks = block_count(a) * a.c.Hkv;
  const dim3 grid((unsigned)((tasks + kRowWarps - 1) / kRowWarps)), block(kRowWarps * 32);
  trace_pre(id, s);
  const cudaError_t e = launch_k(a.c.D == 128 ? k128 : k64, grid, block, 0, s, true, a, tasks);
  trace_post(id, s);
  return e;
}
cudaError_t launch_kv4_append(const Kv4RowsArgs& a, cudaStream_t s) {
  return launch_rows(kv4_append_kernel<128>, kv4_append_kernel<64>, K_KV4_APPEND, a, s);
}
cudaError_t launch_kv4_gather(const Kv4RowsArgs& a, cudaStream_t s) {
  return launch_rows(kv4_gather_kernel<128>, kv4_gather_kernel<64>, K_KV4_GATHER, a, s);
}

int status_kv4(int clear) { return tu_status(clear); }

}  // namespace m2
