// k_attn_decode.cu -- attention of one query token a sequence over the paged
// 4-bit cache.
#include <cuda_runtime.h>
#include <stdint.h>

#include "m2_common.cuh"
#include "m2_kernels.h"
#include "m2_kv4.cuh"

namespace m2 {

// One CTA per (sequence, query head): 8 warps take the tokens in turn, lane l
// holding channels 4l .. 4l+3 (D = 128) or 2l, 2l+1; the warps' running
// maxima, sums and outputs are joined at the end.  The simplest form.
template <int D>
__global__ void __launch_bounds__(256) attn_decode_rows_kernel(const AttnDecodeArgs a) {
  using L = Kv4Block<D>;
  constexpr int E = D / 32, W = 8;
  __shared__ float sm[W], sl[W], so[W][D];
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int b = blockIdx.x / a.H, h = blockIdx.x % a.H, hk = h / (a.H / a.c.Hkv);
  int64_t n = a.len[b];
  if (n > (int64_t)a.c.ld_table * kPage) {
    n = (int64_t)a.c.ld_table * kPage;
    M2_RECORD_ARG(g_status);
  }
  float q[E], o[E], m = -INFINITY, l = 0.0f;
  const int d0 = lane * E, g = d0 / 16;
  for (int i = 0; i < E; ++i) {
    q[i] = bf16_to_f32(a.q[(size_t)b * a.ld_q + h * D + d0 + i]) * a.scale;
    o[i] = 0.0f;
  }
  for (int64_t j = warp; j < n; j += W) {
    const int page = a.c.table[(size_t)b * a.c.ld_table + j / kPage], t = (int)(j % kPage);
    if (page < 0 || page >= a.c.n_pages) {
      M2_RECORD_ARG(g_status);
      continue;
    }
    const uint8_t* blk = a.c.pages + ((size_t)page * a.c.Hkv + hk) * L::kBytes;
    const float sk = kv4_scale(blk[L::ks(t, g)]), sv = kv4_scale(blk[L::vs(t, g)]);
    float s = 0.0f;
    for (int i = 0; i < E; i += 2) {
      const int d = d0 + i;
      const float2 f = kv4_f32x2(blk[L::k(t, g, d % 16 / 4) + d % 4 / 2]);
      s += (q[i] * f.x + q[i + 1] * f.y) * sk;
    }
    s = warp_sum(s);
    const float mn = fmaxf(m, s), f = expf(m - mn), p = expf(s - mn);
    m = mn;
    l = l * f + p;
    for (int i = 0; i < E; ++i) {
      const uint32_t c = blk[L::v(t, (d0 + i) / 8, (d0 + i) % 8)] >> (4 * (t & 1));
      o[i] = o[i] * f + p * (kv4_f32x2(c & 15u).x * sv);
    }
  }
  if (lane == 0) {
    sm[warp] = m;
    sl[warp] = l;
  }
  for (int i = 0; i < E; ++i) so[warp][d0 + i] = o[i];
  __syncthreads();
  if (threadIdx.x < D) {
    float top = -INFINITY, sum = 0.0f, acc = 0.0f;
    for (int w = 0; w < W; ++w)
      if (sl[w] != 0.0f) top = fmaxf(top, sm[w]);
    for (int w = 0; w < W; ++w) {
      if (sl[w] == 0.0f) continue;
      const float f = expf(sm[w] - top);
      sum += sl[w] * f;
      acc += so[w][threadIdx.x] * f;
    }
    a.out[(size_t)b * a.ld_o + h * D + threadIdx.x] = f32_to_bf16(sum != 0.0f ? acc / sum : 0.0f);
  }
}

size_t attn_decode_ws_bytes(int32_t B, int32_t H, int32_t Hkv, int32_t D) {
  (void)B;
  (void)H;
  (void)Hkv;
  (void)D;
  return 256;
}

cudaError_t launch_attn_decode(const AttnDecodeArgs& a, cudaStream_t s) {
  trace_pre(K_ATTN_DECODE, s);
  const cudaError_t e = launch_k(a.c.D == 128 ? attn_decode_rows_kernel<128> : attn_decode_rows_kernel<64>,
                                 dim3(a.B * a.H), dim3(256), 0, s, true, a);
  trace_post(K_ATTN_DECODE, s);
  return e;
}

int status_attn_decode(int clear) { return tu_status(clear); }
cudaError_t wait_limit_attn_decode(long long cycles) { return tu_set_wait_limit(cycles); }

}  // namespace m2
