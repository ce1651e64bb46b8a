// m2_tree_abi.cu -- the exported entry points for trees of drafted tokens
// (include/mamba2.h): host-side checks, and the launches.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "../../include/mamba2.h"
#include "m2_attn_checks.h"
#include "m2_kernels.h"

namespace m2 {

static inline bool al8(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 7u) == 0; }
static inline bool al2(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 1u) == 0; }

// Whether T rows of `width` elements at a and at b share any, both `ld` apart (b may be other columns of a's buffer).
static bool rows_overlap(const uint16_t* a, const uint16_t* b, int32_t ld, int32_t width, int32_t T) {
  const int64_t d = (int64_t)(reinterpret_cast<uintptr_t>(b) - reinterpret_cast<uintptr_t>(a)) / 2;
  const int64_t m = (d % ld + ld) % ld, far = d < 0 ? -d : d;
  return far < (int64_t)(T - 1) * ld + width && (m < width || m > ld - width);
}

static int check_ssm(int32_t H, int32_t P, int32_t N, int32_t G) {
  if (H <= 0 || P <= 0 || N <= 0 || G <= 0 || H % G) return M2_ERR_ARG;
  if (!(N == 16 || N == 32 || N == 64 || N == 128) || P > 256) return M2_ERR_UNSUPPORTED;
  if ((int64_t)H * P + 2ll * G * N > INT32_MAX / 16) return M2_ERR_UNSUPPORTED;
  return M2_OK;
}

}  // namespace m2

using namespace m2;

extern "C" {

int mamba2_tree_conv(const uint16_t* conv_state, const int32_t* conv_pos, const uint16_t* x, int32_t ld_x,
                     const uint16_t* w, const uint16_t* bias, uint16_t* out, int32_t ld_o, int32_t nseq,
                     const int32_t* cu_nodes, const int32_t* parent, int32_t C, int32_t d_conv, int32_t silu,
                     cudaStream_t stream) {
  int st;
  if (C <= 0 || C > INT32_MAX / 16) return M2_ERR_ARG;
  if (d_conv < 2 || d_conv > 8) return M2_ERR_UNSUPPORTED;
  if ((st = check_nodes(cu_nodes, nseq))) return st;
  if (cu_nodes[nseq] == 0) return M2_OK;  // no nodes: their pointers may be null
  if (!conv_state || !conv_pos || !x || !w || !out || !parent || ld_x < C || ld_o < C) return M2_ERR_ARG;
  if (!al4(conv_pos) || !al4(parent) || !al2(conv_state) || !al2(x) || !al2(w) || !al2(bias) || !al2(out))
    return M2_ERR_ALIGN;
  if (ld_x == ld_o && rows_overlap(x, out, ld_x, C, cu_nodes[nseq])) return M2_ERR_ARG;  // nodes read others' rows
  TreeConvArgs a;
  a.w = w;
  a.bias = bias;
  a.ld_x = ld_x;
  a.ld_o = ld_o;
  a.C = C;
  a.dconv = d_conv;
  a.silu = silu ? 1 : 0;
  a.wide = C % 8 == 0 && ld_x % 8 == 0 && ld_o % 8 == 0 && al16(conv_state) && al16(x) && al16(w) && al16(bias) && al16(out);
  for (int32_t i0 = 0; i0 < nseq; i0 += kSeqs) {
    a.t = tree_of(cu_nodes, nseq, i0, parent);
    if (a.t.cu[a.t.nseq] == 0) continue;
    a.ring = conv_state + (size_t)i0 * (d_conv - 1) * C;
    a.pos = conv_pos + i0;
    a.x = x + (size_t)cu_nodes[i0] * ld_x;
    a.out = out + (size_t)cu_nodes[i0] * ld_o;
    if ((st = status_of(launch_tree_conv(a, stream)))) return st;
  }
  return M2_OK;
}

int mamba2_tree_ssm(const float* h, const uint16_t* x, const uint16_t* Bm, const uint16_t* Cm, int32_t ld_in,
                    const uint16_t* dt_raw, int32_t ld_dt, const float* A_log, const float* D, const float* dt_bias,
                    float* y, int32_t nseq, const int32_t* cu_nodes, const int32_t* parent, int32_t H, int32_t P,
                    int32_t N, int32_t G, cudaStream_t stream) {
  int st;
  if ((st = check_ssm(H, P, N, G)) || (st = check_nodes(cu_nodes, nseq))) return st;
  if (cu_nodes[nseq] == 0) return M2_OK;
  if (!h || !x || !Bm || !Cm || !dt_raw || !A_log || !D || !dt_bias || !y || !parent) return M2_ERR_ARG;
  if (ld_in % 4 || ld_in < H * P || ld_in < G * N || ld_dt < H) return M2_ERR_ARG;
  if (!al16(h) || !al8(Bm) || !al8(Cm) || !al8(y) || !al2(x) || !al2(dt_raw) || !al4(A_log) || !al4(D) ||
      !al4(dt_bias) || !al4(parent))
    return M2_ERR_ALIGN;
  TreeSsmArgs a;
  a.A_log = A_log;
  a.D = D;
  a.dt_bias = dt_bias;
  a.ld_in = ld_in;
  a.ld_dt = ld_dt;
  a.H = H;
  a.P = P;
  a.N = N;
  a.G = G;
  a.wide_x = P % 4 == 0 && al8(x);
  for (int32_t i0 = 0; i0 < nseq; i0 += kSeqs) {
    a.t = tree_of(cu_nodes, nseq, i0, parent);
    if (a.t.cu[a.t.nseq] == 0) continue;
    const size_t row = cu_nodes[i0];
    a.h = h + (size_t)i0 * H * P * N;
    a.x = x + row * ld_in;
    a.Bm = Bm + row * ld_in;
    a.Cm = Cm + row * ld_in;
    a.dt = dt_raw + row * ld_dt;
    a.y = y + row * H * P;
    if ((st = status_of(launch_tree_ssm(a, stream)))) return st;
  }
  return M2_OK;
}

int mamba2_tree_commit(const float* h, const uint16_t* conv_state, const int32_t* conv_pos, float* h_out,
                       uint16_t* conv_state_out, int32_t* conv_pos_out, const uint16_t* xbc, int32_t ld_xbc,
                       const uint16_t* u, int32_t ld_u, const uint16_t* dt_raw, int32_t ld_dt, const float* A_log,
                       const float* dt_bias, int32_t nseq, const int32_t* cu_nodes, const int32_t* path,
                       const int32_t* count, int32_t H, int32_t P, int32_t N, int32_t G, int32_t d_conv,
                       cudaStream_t stream) {
  int st;
  if ((st = check_ssm(H, P, N, G))) return st;
  if (d_conv < 2 || d_conv > 8) return M2_ERR_UNSUPPORTED;
  if ((st = check_nodes(cu_nodes, nseq))) return st;
  const int32_t C = H * P + 2 * G * N;
  if (!h || !conv_state || !conv_pos || !h_out || !conv_state_out || !conv_pos_out || !A_log || !dt_bias || !count)
    return M2_ERR_ARG;
  if (!al16(h) || !al16(h_out) || !al2(conv_state) || !al2(conv_state_out) || !al4(conv_pos) || !al4(conv_pos_out) ||
      !al4(A_log) || !al4(dt_bias) || !al4(count))
    return M2_ERR_ALIGN;
  if (cu_nodes[nseq] > 0) {  // else the arrays by node may be missing
    if (!xbc || !u || !dt_raw || !path || ld_xbc < C || ld_u < C || ld_u % 4 || ld_dt < H) return M2_ERR_ARG;
    if (!al8(u + (size_t)H * P) || !al2(xbc) || !al2(dt_raw) || !al4(path)) return M2_ERR_ALIGN;
  } else if (h_out == h && conv_state_out == conv_state && conv_pos_out == conv_pos) {
    return M2_OK;
  }
  TreeCommitArgs a;
  a.A_log = A_log;
  a.dt_bias = dt_bias;
  a.ld_xbc = ld_xbc;
  a.ld_u = ld_u;
  a.ld_dt = ld_dt;
  a.H = H;
  a.P = P;
  a.N = N;
  a.G = G;
  a.dconv = d_conv;
  a.wide = C % 8 == 0 && ld_xbc % 8 == 0 && al16(conv_state) && al16(conv_state_out) && al16(xbc);
  for (int32_t i0 = 0; i0 < nseq; i0 += kSeqs) {
    a.t = tree_of(cu_nodes, nseq, i0, path);
    const size_t row = cu_nodes[i0], state = (size_t)i0 * H * P * N, ring = (size_t)i0 * (d_conv - 1) * C;
    a.count = count + i0;
    a.h = h + state;
    a.h_out = h_out + state;
    a.ring = conv_state + ring;
    a.ring_out = conv_state_out + ring;
    a.pos = conv_pos + i0;
    a.pos_out = conv_pos_out + i0;
    a.xbc = xbc + row * ld_xbc;
    a.u = u + row * ld_u;
    a.dt = dt_raw + row * ld_dt;
    if ((st = status_of(launch_tree_commit(a, stream)))) return st;
  }
  return M2_OK;
}

int m2_verify_tree(const void* p, int64_t ld_p, const void* q, int64_t ld_q, int32_t fmt, int32_t V, int32_t nseq,
                   const int32_t* cu_nodes, const int32_t* parent, const int32_t* token, const float* u,
                   const float* u_next, int32_t* path, int32_t* count, int32_t* next_token, cudaStream_t stream) {
  int st;
  if (fmt != M2_PROB_F32 && fmt != M2_PROB_BF16) return M2_ERR_FORMAT;
  if (V <= 0 || V > (1 << 30)) return M2_ERR_ARG;
  if ((st = check_nodes(cu_nodes, nseq))) return st;
  if (!u_next || !count || !next_token) return M2_ERR_ARG;
  if (!al4(u_next) || !al4(count) || !al4(next_token)) return M2_ERR_ALIGN;
  if (cu_nodes[nseq] > 0) {  // else the arrays by node may be missing
    if (!p || !parent || !token || !u || !path || ld_p < V || (q && ld_q < V)) return M2_ERR_ARG;
    const uintptr_t es = fmt == M2_PROB_BF16 ? 1 : 3;
    if ((reinterpret_cast<uintptr_t>(p) & es) || (reinterpret_cast<uintptr_t>(q) & es) || !al4(parent) || !al4(token) ||
        !al4(u) || !al4(path))
      return M2_ERR_ALIGN;
  }
  VerifyArgs a;
  a.ld_p = ld_p;
  a.ld_q = ld_q;
  a.bf16 = fmt == M2_PROB_BF16;
  a.V = V;
  for (int32_t i0 = 0; i0 < nseq; i0 += kSeqs) {
    a.t = tree_of(cu_nodes, nseq, i0, parent);
    const size_t row = cu_nodes[i0], size = a.bf16 ? 2 : 4;
    a.p = static_cast<const char*>(p) + row * ld_p * size;
    a.q = q ? static_cast<const char*>(q) + row * ld_q * size : nullptr;
    a.token = token + row;
    a.u = u + row;
    a.u_next = u_next + i0;
    a.path = path + row;
    a.count = count + i0;
    a.next = next_token + i0;
    if ((st = status_of(launch_verify_tree(a, stream)))) return st;
  }
  return M2_OK;
}

int m2_kv4_keep(const m2_kv4_cache* cache, const int32_t* cu_nodes, const int32_t* path, const int32_t* count,
                const int32_t* kv_pos, cudaStream_t stream) {
  int st;
  if ((st = check_cache(cache)) || (st = check_nodes(cu_nodes, cache->nseq))) return st;
  if (cu_nodes[cache->nseq] == 0) return M2_OK;
  if (!path || !count || !kv_pos) return M2_ERR_ARG;
  if (!al4(path) || !al4(count) || !al4(kv_pos)) return M2_ERR_ALIGN;
  Kv4KeepArgs a;
  a.c = kv4_of(cache);
  for (int32_t i0 = 0; i0 < cache->nseq; i0 += kSeqs) {
    a.t = tree_of(cu_nodes, cache->nseq, i0, path);
    if (a.t.cu[a.t.nseq] == 0) continue;
    a.c.table = cache->block_table + (size_t)i0 * cache->ld_table;
    a.count = count + i0;
    a.pos = kv_pos + i0;
    if ((st = status_of(launch_kv4_keep(a, stream)))) return st;
  }
  return M2_OK;
}

size_t m2_attn_tree_kv4_workspace_bytes(int32_t H, int32_t Hkv, int32_t head_dim) {
  return check_heads(H, Hkv, head_dim) ? 0 : attn_tree_ws_bytes(head_dim);
}

int m2_attn_tree_kv4(const m2_kv4_cache* cache, const uint16_t* q, int32_t ld_q, uint16_t* out, int32_t ld_o,
                     int32_t H, const int32_t* cu_nodes, const int32_t* parent, const int32_t* kv_pos, float scale,
                     void* ws, size_t ws_bytes, cudaStream_t stream) {
  int st;
  if ((st = check_cache(cache))) return st;
  if ((st = check_heads(H, cache->n_kv_heads, cache->head_dim))) return st;
  if (!isfinite(scale)) return M2_ERR_ARG;
  if ((st = check_nodes(cu_nodes, cache->nseq))) return st;
  if (cu_nodes[cache->nseq] == 0) return M2_OK;
  if (!parent || !kv_pos) return M2_ERR_ARG;
  const int32_t w = H * cache->head_dim;
  if ((st = check_rows(q, ld_q, w)) || (st = check_rows(out, ld_o, w))) return st;
  if (!al4(parent) || !al4(kv_pos)) return M2_ERR_ALIGN;
  if (!ws || (reinterpret_cast<uintptr_t>(ws) & 255u) ||
      ws_bytes < attn_tree_ws_bytes(cache->head_dim))
    return M2_ERR_WORKSPACE;
  AttnTreeArgs a;
  a.c = kv4_of(cache);
  a.ld_q = ld_q;
  a.ld_o = ld_o;
  a.H = H;
  a.scale = scale;
  a.ws = ws;
  // units (pages and what a tile costs beside them, x tiles of at least 16 rows x kv heads) are counted in 32 bits
  if ((cache->nseq < kSeqs ? cache->nseq : kSeqs) * (cache->ld_table + 8ll) > INT32_MAX / (4ll * H + 4 * cache->n_kv_heads))
    return M2_ERR_UNSUPPORTED;
  for (int32_t i0 = 0; i0 < cache->nseq; i0 += kSeqs) {
    a.t = tree_of(cu_nodes, cache->nseq, i0, parent);
    if (a.t.cu[a.t.nseq] == 0) continue;
    a.most = 0;
    for (int32_t i = 0; i < a.t.nseq; ++i) a.most = a.t.cu[i + 1] - a.t.cu[i] > a.most ? a.t.cu[i + 1] - a.t.cu[i] : a.most;
    a.c.table = cache->block_table + (size_t)i0 * cache->ld_table;
    a.q = q + (size_t)cu_nodes[i0] * ld_q;
    a.out = out + (size_t)cu_nodes[i0] * ld_o;
    a.pos = kv_pos + i0;
    if ((st = status_of(launch_attn_tree(a, stream)))) return st;
  }
  return M2_OK;
}

}  // extern "C"
