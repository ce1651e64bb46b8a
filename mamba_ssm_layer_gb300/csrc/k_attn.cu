// k_attn.cu -- causal attention of packed sequences.
#include <cuda_runtime.h>
#include <stdint.h>

#include "m2_common.cuh"
#include "m2_kernels.h"

namespace m2 {

// One warp per (query row, head): online softmax over the keys it sees, lane l
// holding channels l * D/32 ..  The simplest form; scores and sums in fp32.
template <int D>
__global__ void __launch_bounds__(256) attn_rows_kernel(const AttnArgs a) {
  constexpr int E = D / 32;
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const int64_t id = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int64_t rows = a.cu_q[a.nseq] - a.cu_q[0];
  if (id >= rows * a.H) return;
  const int row = a.cu_q[0] + (int)(id / a.H), h = (int)(id % a.H), hk = h / (a.H / a.Hkv);
  int seq = 0;
  while (row >= a.cu_q[seq + 1]) ++seq;
  const int nk = a.cu_k[seq + 1] - a.cu_k[seq], nq = a.cu_q[seq + 1] - a.cu_q[seq];
  const int last = row - a.cu_q[seq] + nk - nq;  // the last key seen
  float q[E], o[E], m = -INFINITY, l = 0.0f;
  for (int i = 0; i < E; ++i) {
    q[i] = bf16_to_f32(a.q[(size_t)row * a.ld_q + h * D + lane * E + i]) * a.scale;
    o[i] = 0.0f;
  }
  for (int j = 0; j <= last; ++j) {
    const size_t kr = a.cu_k[seq] + j;
    float s = 0.0f;
    for (int i = 0; i < E; ++i) s = fmaf(q[i], bf16_to_f32(a.k[kr * a.ld_k + hk * D + lane * E + i]), s);
    s = warp_sum(s);
    const float mn = fmaxf(m, s), f = expf(m - mn), p = expf(s - mn);
    m = mn;
    l = l * f + p;
    for (int i = 0; i < E; ++i) o[i] = o[i] * f + p * bf16_to_f32(a.v[kr * a.ld_v + hk * D + lane * E + i]);
  }
  for (int i = 0; i < E; ++i)
    a.out[(size_t)row * a.ld_o + h * D + lane * E + i] = f32_to_bf16(last >= 0 ? o[i] / l : 0.0f);
}

cudaError_t launch_attn_prefill(const AttnArgs& a, cudaStream_t s) {
  const int64_t tasks = (int64_t)(a.cu_q[a.nseq] - a.cu_q[0]) * a.H;
  const dim3 grid((unsigned)((tasks + 7) / 8)), block(256);
  trace_pre(K_ATTN_PREFILL, s);
  const cudaError_t e = launch_k(a.D == 128 ? attn_rows_kernel<128> : attn_rows_kernel<64>, grid, block, 0, s, true, a);
  trace_post(K_ATTN_PREFILL, s);
  return e;
}

int status_attn(int clear) { return tu_status(clear); }
cudaError_t wait_limit_attn(long long cycles) { return tu_set_wait_limit(cycles); }

}  // namespace m2
