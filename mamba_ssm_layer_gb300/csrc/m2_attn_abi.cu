// m2_attn_abi.cu -- the exported entry points of the attention operators
// (include/mamba2.h): host-side checks, and the launches.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include "../../include/mamba2.h"
#include "m2_kernels.h"

namespace m2 {

static inline bool al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

static int status_of(cudaError_t e) {
  if (e != cudaSuccess) {
    cudaGetLastError();
    return M2_ERR_LAUNCH;
  }
  return M2_OK;
}

static bool head_dim_ok(int32_t D) { return D == 64 || D == 128; }

// Head counts of an attention layer.
static int check_heads(int32_t H, int32_t Hkv, int32_t D) {
  if (H <= 0 || Hkv <= 0 || D <= 0 || H % Hkv) return M2_ERR_ARG;
  if (!head_dim_ok(D) || H > 4096) return M2_ERR_UNSUPPORTED;
  return M2_OK;
}

// Rows of `width` elements, `ld` apart, that are read or written 16 bytes at a time.
static int check_rows(const void* p, int32_t ld, int32_t width) {
  if (!p || ld < width) return M2_ERR_ARG;
  if (!al16(p) || ld % 8) return M2_ERR_ALIGN;
  return M2_OK;
}

static int check_offsets(const int32_t* cu, int32_t nseq) {
  if (!cu || nseq <= 0 || cu[0] != 0) return M2_ERR_ARG;
  for (int i = 0; i < nseq; ++i)
    if (cu[i + 1] < cu[i]) return M2_ERR_ARG;
  return M2_OK;
}

static int check_cache(const m2_kv4_cache* c) {
  if (!c || !c->pages || !c->block_table || c->n_pages <= 0 || c->n_kv_heads <= 0 || c->head_dim <= 0 ||
      c->nseq <= 0 || c->ld_table <= 0 || c->ld_table > INT32_MAX / M2_KV4_PAGE)
    return M2_ERR_ARG;
  if (!head_dim_ok(c->head_dim) || c->n_kv_heads > 4096) return M2_ERR_UNSUPPORTED;
  if (!al16(c->pages) || (reinterpret_cast<uintptr_t>(c->block_table) & 3u)) return M2_ERR_ALIGN;
  return M2_OK;
}

static Kv4 kv4_of(const m2_kv4_cache* c) {
  Kv4 k;
  k.pages = static_cast<uint8_t*>(c->pages);
  k.table = c->block_table;
  k.n_pages = c->n_pages;
  k.Hkv = c->n_kv_heads;
  k.D = c->head_dim;
  k.ld_table = c->ld_table;
  return k;
}

// Append (pos set) and gather: checks, then one launch per kSeqs sequences.
static int kv4_rows(const m2_kv4_cache* c, uint16_t* k, int32_t ld_k, uint16_t* v, int32_t ld_v, const int32_t* cu,
                    const int32_t* pos, cudaError_t (*launch)(const Kv4RowsArgs&, cudaStream_t), cudaStream_t s) {
  int st;
  if ((st = check_cache(c))) return st;
  const int32_t w = c->n_kv_heads * c->head_dim;
  if ((st = check_offsets(cu, c->nseq))) return st;
  if (cu[c->nseq] == 0) return M2_OK;  // no rows: their pointers may be null
  if ((st = check_rows(k, ld_k, w)) || (st = check_rows(v, ld_v, w))) return st;
  if (reinterpret_cast<uintptr_t>(pos) & 3u) return M2_ERR_ALIGN;
  for (int32_t i0 = 0; i0 < c->nseq; i0 += kSeqs) {
    const int32_t n = c->nseq - i0 < kSeqs ? c->nseq - i0 : kSeqs;
    if (cu[i0 + n] == cu[i0]) continue;
    Kv4RowsArgs a;
    a.c = kv4_of(c);
    a.c.table += (size_t)i0 * c->ld_table;
    a.k = k + (size_t)cu[i0] * ld_k;
    a.v = v + (size_t)cu[i0] * ld_v;
    a.ld_k = ld_k;
    a.ld_v = ld_v;
    a.pos = pos ? pos + i0 : nullptr;
    a.nseq = n;
    for (int32_t i = 0; i <= kSeqs; ++i) a.cu[i] = cu[i0 + (i < n ? i : n)] - cu[i0];
    const cudaError_t e = launch(a, s);
    if (e != cudaSuccess) return status_of(e);
  }
  return M2_OK;
}

}  // namespace m2

using namespace m2;

extern "C" {

int m2_rope_steps(double theta, int32_t rot_dim, uint64_t* steps) {
  if (!steps || !(theta >= 1.0) || !(theta <= 1e30)) return M2_ERR_ARG;
  if (rot_dim <= 0 || rot_dim > 128 || rot_dim % 16) return M2_ERR_UNSUPPORTED;
  for (int32_t i = 0; i < rot_dim / 2; ++i)
    steps[i] = (uint64_t)ldexp(pow(theta, -2.0 * i / rot_dim) / (2.0 * M_PI), 64);
  return M2_OK;
}

int m2_qk_norm_rope(const uint16_t* q, int32_t ld_q, const uint16_t* k, int32_t ld_k, uint16_t* q_out, int32_t ld_qo,
                    uint16_t* k_out, int32_t ld_ko, const uint16_t* q_w, const uint16_t* k_w, const int32_t* pos,
                    const uint64_t* rope_step, int32_t T, int32_t H, int32_t Hkv, int32_t head_dim, int32_t rot_dim,
                    int32_t interleaved, float eps, cudaStream_t stream) {
  int st;
  if (T < 0 || rot_dim < 0 || !(eps >= 0.0f)) return M2_ERR_ARG;
  if ((st = check_heads(H, Hkv, head_dim))) return st;
  if (rot_dim % 16 || rot_dim > head_dim) return M2_ERR_UNSUPPORTED;
  if (T == 0) return M2_OK;  // no rows: their pointers may be null
  if (rot_dim > 0 && (!pos || !rope_step)) return M2_ERR_ARG;
  const int32_t wq = H * head_dim, wk = Hkv * head_dim;
  if ((st = check_rows(q, ld_q, wq)) || (st = check_rows(k, ld_k, wk)) || (st = check_rows(q_out, ld_qo, wq)) ||
      (st = check_rows(k_out, ld_ko, wk)))
    return st;
  if (!al16(q_w) || !al16(k_w) || (reinterpret_cast<uintptr_t>(pos) & 3u) ||
      (reinterpret_cast<uintptr_t>(rope_step) & 7u))
    return M2_ERR_ALIGN;
  RopeArgs a;
  a.q = q;
  a.k = k;
  a.q_out = q_out;
  a.k_out = k_out;
  a.ld_q = ld_q;
  a.ld_k = ld_k;
  a.ld_qo = ld_qo;
  a.ld_ko = ld_ko;
  a.q_w = q_w;
  a.k_w = k_w;
  a.pos = pos;
  a.step = rope_step;
  a.T = T;
  a.H = H;
  a.Hkv = Hkv;
  a.D = head_dim;
  a.rot = rot_dim;
  a.interleaved = interleaved ? 1 : 0;
  a.eps = eps;
  return status_of(launch_qk_norm_rope(a, stream));
}

size_t m2_kv4_page_bytes(int32_t n_kv_heads, int32_t head_dim) {
  return n_kv_heads > 0 && head_dim_ok(head_dim) ? (size_t)n_kv_heads * 72 * head_dim : 0;
}

int m2_kv4_append(const m2_kv4_cache* cache, const uint16_t* k, int32_t ld_k, const uint16_t* v, int32_t ld_v,
                  const int32_t* cu_rows, const int32_t* kv_pos, cudaStream_t stream) {
  if (!kv_pos) return M2_ERR_ARG;
  return kv4_rows(cache, const_cast<uint16_t*>(k), ld_k, const_cast<uint16_t*>(v), ld_v, cu_rows, kv_pos,
                  launch_kv4_append, stream);
}

int m2_kv4_gather(const m2_kv4_cache* cache, uint16_t* k, int32_t ld_k, uint16_t* v, int32_t ld_v,
                  const int32_t* cu_rows, cudaStream_t stream) {
  return kv4_rows(cache, k, ld_k, v, ld_v, cu_rows, nullptr, launch_kv4_gather, stream);
}

int m2_attn_prefill_varlen(const uint16_t* q, int32_t ld_q, const uint16_t* k, int32_t ld_k, const uint16_t* v,
                           int32_t ld_v, uint16_t* out, int32_t ld_o, int32_t H, int32_t Hkv, int32_t head_dim,
                           int32_t nseq, const int32_t* cu_q, const int32_t* cu_k, float scale, cudaStream_t stream) {
  int st;
  if ((st = check_heads(H, Hkv, head_dim))) return st;
  if (!isfinite(scale)) return M2_ERR_ARG;
  const int32_t wq = H * head_dim, wk = Hkv * head_dim;
  if ((st = check_offsets(cu_q, nseq)) || (st = check_offsets(cu_k, nseq))) return st;
  if (cu_q[nseq] == 0) return M2_OK;  // no rows: their pointers may be null
  if ((st = check_rows(q, ld_q, wq)) || (st = check_rows(out, ld_o, wq))) return st;
  if (cu_k[nseq] > 0 && ((st = check_rows(k, ld_k, wk)) || (st = check_rows(v, ld_v, wk)))) return st;
  AttnArgs a;
  a.q = q;
  a.k = k;
  a.v = v;
  a.out = out;
  a.ld_q = ld_q;
  a.ld_k = ld_k;
  a.ld_v = ld_v;
  a.ld_o = ld_o;
  a.H = H;
  a.Hkv = Hkv;
  a.D = head_dim;
  a.Tq = cu_q[nseq];
  a.Tk = cu_k[nseq];
  a.scale = scale;
  for (int32_t i0 = 0; i0 < nseq; i0 += kSeqs) {
    const int32_t n = nseq - i0 < kSeqs ? nseq - i0 : kSeqs;
    if (cu_q[i0 + n] == cu_q[i0]) continue;
    a.nseq = n;
    for (int32_t i = 0; i <= kSeqs; ++i) {
      a.cu_q[i] = cu_q[i0 + (i < n ? i : n)];
      a.cu_k[i] = cu_k[i0 + (i < n ? i : n)];
    }
    const cudaError_t e = launch_attn_prefill(a, stream);
    if (e != cudaSuccess) return status_of(e);
  }
  return M2_OK;
}

size_t m2_attn_decode_kv4_workspace_bytes(int32_t nseq, int32_t H, int32_t Hkv, int32_t head_dim) {
  if (nseq <= 0 || check_heads(H, Hkv, head_dim)) return 0;
  return attn_decode_ws_bytes(nseq, H, Hkv, head_dim);
}

int m2_attn_decode_kv4(const m2_kv4_cache* cache, const uint16_t* q, int32_t ld_q, uint16_t* out, int32_t ld_o,
                       int32_t H, const int32_t* kv_len, float scale, void* ws, size_t ws_bytes, cudaStream_t stream) {
  int st;
  if ((st = check_cache(cache))) return st;
  if ((st = check_heads(H, cache->n_kv_heads, cache->head_dim))) return st;
  if (!kv_len || !isfinite(scale)) return M2_ERR_ARG;
  if ((int64_t)cache->nseq * cache->ld_table > INT32_MAX / H) return M2_ERR_UNSUPPORTED;  // counted in 32 bits
  const int32_t w = H * cache->head_dim;
  if ((st = check_rows(q, ld_q, w)) || (st = check_rows(out, ld_o, w))) return st;
  if (reinterpret_cast<uintptr_t>(kv_len) & 3u) return M2_ERR_ALIGN;
  if (!ws || (reinterpret_cast<uintptr_t>(ws) & 255u) ||
      ws_bytes < attn_decode_ws_bytes(cache->nseq, H, cache->n_kv_heads, cache->head_dim))
    return M2_ERR_WORKSPACE;
  AttnDecodeArgs a;
  a.c = kv4_of(cache);
  a.q = q;
  a.out = out;
  a.ld_q = ld_q;
  a.ld_o = ld_o;
  a.B = cache->nseq;
  a.H = H;
  a.len = kv_len;
  a.scale = scale;
  a.ws = ws;
  return status_of(launch_attn_decode(a, stream));
}

}  // extern "C"
