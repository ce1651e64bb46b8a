// m2_attn_checks.h -- host-side checks that the entry points of the attention and of
// the tree operators share.
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/mamba2.h"
#include "m2_kernels.h"

namespace m2 {

static inline bool al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

static inline int status_of(cudaError_t e) {
  if (e != cudaSuccess) {
    cudaGetLastError();
    return M2_ERR_LAUNCH;
  }
  return M2_OK;
}

static inline bool head_dim_ok(int32_t D) { return D == 64 || D == 128; }

// Head counts of an attention layer.
static inline int check_heads(int32_t H, int32_t Hkv, int32_t D) {
  if (H <= 0 || Hkv <= 0 || D <= 0 || H % Hkv) return M2_ERR_ARG;
  if (!head_dim_ok(D) || H > 4096) return M2_ERR_UNSUPPORTED;
  return M2_OK;
}

// Rows of `width` elements, `ld` apart, that are read or written 16 bytes at a time.
static inline int check_rows(const void* p, int32_t ld, int32_t width) {
  if (!p || ld < width) return M2_ERR_ARG;
  if (!al16(p) || ld % 8) return M2_ERR_ALIGN;
  return M2_OK;
}

static inline int check_offsets(const int32_t* cu, int32_t nseq) {
  if (!cu || nseq <= 0 || cu[0] != 0) return M2_ERR_ARG;
  for (int i = 0; i < nseq; ++i)
    if (cu[i + 1] < cu[i]) return M2_ERR_ARG;
  return M2_OK;
}

static inline int check_cache(const m2_kv4_cache* c) {
  if (!c || !c->pages || !c->block_table || c->n_pages <= 0 || c->n_kv_heads <= 0 || c->head_dim <= 0 ||
      c->nseq <= 0 || c->ld_table <= 0 || c->ld_table > INT32_MAX / M2_KV4_PAGE)
    return M2_ERR_ARG;
  if (!head_dim_ok(c->head_dim) || c->n_kv_heads > 4096) return M2_ERR_UNSUPPORTED;
  if (!al16(c->pages) || (reinterpret_cast<uintptr_t>(c->block_table) & 3u)) return M2_ERR_ALIGN;
  return M2_OK;
}

static inline Kv4 kv4_of(const m2_kv4_cache* c) {
  Kv4 k;
  k.pages = static_cast<uint8_t*>(c->pages);
  k.table = c->block_table;
  k.n_pages = c->n_pages;
  k.Hkv = c->n_kv_heads;
  k.D = c->head_dim;
  k.ld_table = c->ld_table;
  return k;
}

// Nodes of nseq trees: offsets, and no tree of more than kTreeNodes.
static inline int check_nodes(const int32_t* cu, int32_t nseq) {
  const int st = check_offsets(cu, nseq);
  if (st) return st;
  for (int i = 0; i < nseq; ++i)
    if (cu[i + 1] - cu[i] > kTreeNodes) return M2_ERR_UNSUPPORTED;
  return M2_OK;
}
static inline bool al4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
// The trees of sequences i0 .. (at most kSeqs of them); arrays by node start at their first one.
static inline TreeArgs tree_of(const int32_t* cu, int32_t nseq, int32_t i0, const int32_t* by_node) {
  TreeArgs t;
  t.parent = by_node + cu[i0];
  t.nseq = nseq - i0 < kSeqs ? nseq - i0 : kSeqs;
  for (int32_t i = 0; i <= kSeqs; ++i) t.cu[i] = cu[i0 + (i < t.nseq ? i : t.nseq)] - cu[i0];
  return t;
}

}  // namespace m2
