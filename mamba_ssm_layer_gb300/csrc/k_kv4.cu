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
// A head is D/8 lanes of 8 channels (16-byte loads and stores), so that a
// warp holds 256/D heads of a row.  The angles of a row are shared by all its
// heads: one thread per (row, frequency) evaluates sin and cos into shared
// memory.  p * step mod 2^64 is the angle in turns, exactly; only its top 32
// bits (as a signed fraction of a half turn) enter the fp32 functions.
constexpr int kRopeThreads = 256;

template <int D>
__global__ void __launch_bounds__(kRopeThreads) qk_norm_rope_kernel(const RopeArgs a, int rows_per_cta) {
  constexpr int LH = D / 8, HW = 32 / LH;  // lanes a head, heads a warp
  extern __shared__ float2 cs[];           // [rows][rot / 2] (cos, sin)
  const int r0 = blockIdx.x * rows_per_cta;
  const int rows = min(rows_per_cta, a.T - r0), half = a.rot / 2;
  pdl_wait();
  pdl_trigger();
  for (int i = threadIdx.x; i < rows * half; i += kRopeThreads) {
    const int r = i / half, f = i - r * half;
    const uint64_t turn = (uint64_t)(int64_t)a.pos[r0 + r] * a.step[f];
    float s, c;
    sincospif((float)(int32_t)(turn >> 32) * 4.656612873077393e-10f, &s, &c);  // 2^-31
    cs[i] = make_float2(c, s);
  }
  __syncthreads();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int c0 = (lane % LH) * 8;  // this lane's first channel
  const int heads = a.H + a.Hkv, groups = (heads + HW - 1) / HW;
  for (int t = warp; t < rows * groups; t += kRopeThreads / 32) {
    const int r = t / groups, h = (t - r * groups) * HW + lane / LH;
    const bool on = h < heads, isq = h < a.H;
    const size_t row = r0 + r;
    float x[8];
    if (on) {
      const uint16_t* src = isq ? a.q + row * a.ld_q + (size_t)h * D : a.k + row * a.ld_k + (size_t)(h - a.H) * D;
      const uint4 v = *reinterpret_cast<const uint4*>(src + c0);
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[2 * i] = bf16lo(w[i]);
        x[2 * i + 1] = bf16hi(w[i]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = 0.0f;
    }
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
    for (int o = LH / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    const uint16_t* nw = isq ? a.q_w : a.k_w;
    if (nw) {
      const float rr = rsqrtf(ss * (1.0f / D) + a.eps);
      const uint4 v = *reinterpret_cast<const uint4*>(nw + c0);
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[2 * i] *= rr * bf16lo(w[i]);
        x[2 * i + 1] *= rr * bf16hi(w[i]);
      }
    }
    if (half) {
      const float2* rc = cs + r * half;
      if (a.interleaved) {
        if (c0 < a.rot) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 t2 = rc[c0 / 2 + i];
            const float u = x[2 * i], w = x[2 * i + 1];
            x[2 * i] = u * t2.x - w * t2.y;
            x[2 * i + 1] = w * t2.x + u * t2.y;
          }
        }
      } else {
        // the partner channel is rot/2 away: rot/16 lanes
        const int dl = a.rot / 16, l = lane % LH;
        const bool first = l < dl, in = l < 2 * dl;
        const int src = in ? (first ? lane + dl : lane - dl) : lane;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float o = __shfl_sync(0xffffffffu, x[i], src);
          if (in) {
            const float2 t2 = rc[(first ? c0 : c0 - half) + i];
            x[i] = x[i] * t2.x + (first ? -o : o) * t2.y;
          }
        }
      }
    }
    if (on) {
      uint16_t* dst =
          isq ? a.q_out + row * a.ld_qo + (size_t)h * D : a.k_out + row * a.ld_ko + (size_t)(h - a.H) * D;
      *reinterpret_cast<uint4*>(dst + c0) = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]),
                                                       pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
    }
  }
}

cudaError_t launch_qk_norm_rope(const RopeArgs& a, cudaStream_t s) {
  const int rows = a.T > 4 * num_sms() ? 4 : 1;
  const dim3 grid((a.T + rows - 1) / rows), block(kRopeThreads);
  const size_t smem = (size_t)rows * (a.rot / 2) * sizeof(float2);
  trace_pre(K_QK_NORM_ROPE, s);
  const cudaError_t e = a.D == 128 ? launch_k(qk_norm_rope_kernel<128>, grid, block, smem, s, true, a, rows)
                                   : launch_k(qk_norm_rope_kernel<64>, grid, block, smem, s, true, a, rows);
  trace_post(K_QK_NORM_ROPE, s);
  return e;
}

// ------------------------------------------------------------------ cache rows
//
// A task is one token pair (positions 2p and 2p + 1: they share V's bytes) of
// one kv head, on D/4 lanes: lane l of it holds 8 channels of token l / (D/8).
// The pair's two tokens always lie in one page.  Sequence i's tasks start at
// pair_base(i): a closed form that leaves room for a pair cut at both ends.
__device__ __forceinline__ int64_t pair_base(const Kv4RowsArgs& a, int i) { return a.cu[i] / 2 + 2ll * i; }
static int64_t pair_count(const Kv4RowsArgs& a) { return a.cu[a.nseq] / 2 + 2ll * a.nseq; }

struct PairTask {
  bool any;        // a token of the pair belongs to the call
  int seq, h;
  int64_t tok;     // position of this lane's token
  bool have;       // it belongs to the call
  uint8_t* block;  // its page's block, null if the table does not give one
};

template <int D>
__device__ __forceinline__ PairTask pair_task(const Kv4RowsArgs& a, int64_t tasks) {
  constexpr int LT = D / 4;
  PairTask t;
  const int64_t id = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) / LT;
  t.any = t.have = false;
  t.block = nullptr;
  t.seq = 0;
  t.tok = 0;
  if (id >= tasks) return t;
  const int64_t p = id / a.c.Hkv;
  t.h = (int)(id - p * a.c.Hkv);
  int lo = 0, hi = a.nseq;  // the last i with pair_base(i) <= p
  while (hi - lo > 1) {
    const int m = (lo + hi) / 2;
    if (pair_base(a, m) <= p)
      lo = m;
    else
      hi = m;
  }
  t.seq = lo;
  const int64_t first = a.pos ? a.pos[lo] : 0, end = first + a.cu[lo + 1] - a.cu[lo];
  // pairs from that of `first` (rounded down, also below zero) on
  const int64_t pr = (first >> 1) + (p - pair_base(a, lo));
  t.tok = 2 * pr + (threadIdx.x % LT) / (D / 8);
  t.have = t.tok >= first && t.tok < end;
  t.any = 2 * pr + 1 >= first && 2 * pr < end;
  if (!t.any) return t;
  const int64_t page = pr >= 0 ? pr / (kPage / 2) : a.c.ld_table;
  const int id_page = page < a.c.ld_table ? a.c.table[(size_t)lo * a.c.ld_table + page] : -1;
  if (id_page >= 0 && id_page < a.c.n_pages)
    t.block = a.c.pages + ((size_t)id_page * a.c.Hkv + t.h) * (72 * D);
  else
    M2_RECORD_ARG(g_status);
  t.have = t.have && t.block;
  return t;
}

// 8 channels of a row as fp32.
__device__ __forceinline__ void row8(const uint16_t* p, float (&x)[8]) {
  const uint4 v = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = bf16lo(w[i]);
    x[2 * i + 1] = bf16hi(w[i]);
  }
}

// Scale byte and codes (8 nibbles, channel order) of this lane's half group;
// the group's other half is on the neighbouring lane.
__device__ __forceinline__ uint32_t quantize8(const float (&x)[8], uint32_t& byte) {
  float m = 0.0f;
  bool nan = false;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    m = fmaxf(m, fabsf(x[i]));
    nan |= x[i] != x[i];
  }
  if (nan) m = __int_as_float(0x7fffffff);
  const float o = __shfl_xor_sync(0xffffffffu, m, 1);
  nan = m != m || o != o;
  m = fmaxf(m, o);
  byte = nan ? 0xFFu : kv4_scale_byte(m);
  const float s = nan ? 0.0f : kv4_scale(byte);
  uint32_t c = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) c |= kv4_codes(x[2 * i], x[2 * i + 1], s) << (8 * i);
  return c;
}

template <int D>
__global__ void __launch_bounds__(256) kv4_append_kernel(const Kv4RowsArgs a, int64_t tasks) {
  using L = Kv4Block<D>;
  pdl_wait();
  pdl_trigger();
  const PairTask t = pair_task<D>(a, tasks);
  const int lt = threadIdx.x % (D / 4), l = lt % (D / 8);
  const int c0 = 8 * l, g = c0 / 16, c = (c0 % 16) / 4;
  float x[8] = {}, y[8] = {};
  if (t.have) {
    const size_t row = a.cu[t.seq] + (t.tok - a.pos[t.seq]);
    row8(a.k + row * a.ld_k + t.h * D + c0, x);
    row8(a.v + row * a.ld_v + t.h * D + c0, y);
  }
  uint32_t kb, vb;
  const uint32_t kc = quantize8(x, kb), vc = quantize8(y, vb);
  // the other token's V codes and whether it is new
  const uint32_t vo = __shfl_xor_sync(0xffffffffu, vc, D / 8);
  const bool other = __shfl_xor_sync(0xffffffffu, t.have ? 1 : 0, D / 8) != 0;
  if (!t.block) return;
  const int tk = (int)(t.tok % kPage);
  if (t.have) {
    *reinterpret_cast<uint16_t*>(t.block + L::k(tk, g, c)) = (uint16_t)kc;
    *reinterpret_cast<uint16_t*>(t.block + L::k(tk, g, c + 1)) = (uint16_t)(kc >> 16);
    if (l % 2 == 0) {
      t.block[L::ks(tk, g)] = (uint8_t)kb;
      t.block[L::vs(tk, g)] = (uint8_t)vb;
    }
  }
  // V: channel 8l + r is byte r of the two tokens' codes; the even token's
  // lane writes r = 0..3, the odd one's r = 4..7
  const bool odd = lt >= D / 8;
  const uint32_t ve = odd ? vo : vc, vd = odd ? vc : vo;
  const bool he = odd ? other : t.have, hd = odd ? t.have : other;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = odd ? 4 + i : i;
    uint8_t* p = t.block + L::v(tk, l, r);
    const uint32_t lo = (ve >> (4 * r)) & 15u, hi = (vd >> (4 * r)) & 15u;
    uint32_t b = lo | (hi << 4);
    if (!he)
      b = (*p & 15u) | (hi << 4);  // stored by an earlier call
    else if (!hd)
      b = lo;
    *p = (uint8_t)b;
  }
}

template <int D>
__global__ void __launch_bounds__(256) kv4_gather_kernel(const Kv4RowsArgs a, int64_t tasks) {
  using L = Kv4Block<D>;
  pdl_wait();
  pdl_trigger();
  const PairTask t = pair_task<D>(a, tasks);
  if (!t.have) return;
  const int lt = threadIdx.x % (D / 4), l = lt % (D / 8);
  const int c0 = 8 * l, g = c0 / 16, c = (c0 % 16) / 4, tk = (int)(t.tok % kPage);
  const float sk = kv4_scale(t.block[L::ks(tk, g)]), sv = kv4_scale(t.block[L::vs(tk, g)]);
  uint32_t k[4], v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = kv4_f32x2(t.block[L::k(tk, g, c + i / 2) + i % 2]);
    k[i] = pack_bf16x2(f.x * sk, f.y * sk);
    const uint32_t b0 = t.block[L::v(tk, l, 2 * i)] >> (4 * (tk & 1)),
                   b1 = t.block[L::v(tk, l, 2 * i + 1)] >> (4 * (tk & 1));
    const float2 w = kv4_f32x2((b0 & 15u) | ((b1 & 15u) << 4));
    v[i] = pack_bf16x2(w.x * sv, w.y * sv);
  }
  const size_t row = a.cu[t.seq] + t.tok;
  *reinterpret_cast<uint4*>(a.k + row * a.ld_k + t.h * D + c0) = make_uint4(k[0], k[1], k[2], k[3]);
  *reinterpret_cast<uint4*>(a.v + row * a.ld_v + t.h * D + c0) = make_uint4(v[0], v[1], v[2], v[3]);
}

static cudaError_t launch_rows(void (*k128)(Kv4RowsArgs, int64_t), void (*k64)(Kv4RowsArgs, int64_t), int id,
                               const Kv4RowsArgs& a, cudaStream_t s) {
  const int64_t tasks = pair_count(a) * a.c.Hkv;
  const int per = 256 / (a.c.D / 4);
  const dim3 grid((unsigned)((tasks + per - 1) / per)), block(256);
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
