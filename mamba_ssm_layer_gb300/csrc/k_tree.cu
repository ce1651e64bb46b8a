// k_tree.cu -- the Mamba-2 mixer over trees of drafted tokens: the causal conv, the
// SSM outputs of every node without touching the state, and the move of state, conv
// ring and position along the accepted path (include/mamba2.h has the formulas).
#include <cuda_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "m2_common.cuh"
#include "m2_kernels.h"
#include "m2_tree.cuh"

namespace m2 {

// ------------------------------------------------------------------ conv
//
// A thread takes VEC channels of `piece` consecutive nodes of a sequence, the next node's
// taps on their way under the current one's sums.  A node's window is the last rows of its
// path (the set bits of its mask, from the top), then the ring from the newest token back:
// a lane of the first warp looks up a node's rows for the CTA.
// Sums run as the single-token conv's, oldest tap first; products of two bf16 values are
// exact, so the results are the same bits.
// Bound: latency (masks, rows: 2.6 us for a chain of 5, 10240 channels), also of the loads of
// larger batches, in which a row comes from L2 once for each of its d_conv taps: 16 trees of 16
// nodes 7.1 us (issue slots 40 %, DRAM 7 %), of 64 nodes 20 us (42 MB).
constexpr int kTcThreads = 128, kTcMost = 16, kTcCtas = 5;

// Two fused multiply-adds, each rounded as one.
__device__ __forceinline__ float2 tc_fma2(float2 x, float2 y, float2 z) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(r)
      : "l"(reinterpret_cast<const uint64_t&>(x)), "l"(reinterpret_cast<const uint64_t&>(y)),
        "l"(reinterpret_cast<const uint64_t&>(z)));
  return reinterpret_cast<const float2&>(r);
}
__device__ __forceinline__ float2 tc_pair(uint32_t w) { return make_float2(bf16lo(w), bf16hi(w)); }
__device__ __forceinline__ uint32_t tc_word(const uint4& v, int e) {
  return e == 0 ? v.x : e == 1 ? v.y : e == 2 ? v.z : v.w;
}
__device__ __forceinline__ uint32_t tc_word(const uint2& v, int e) { return e == 0 ? v.x : v.y; }

template <int K, int VEC>
__global__ void __launch_bounds__(kTcThreads) tree_conv_kernel(const __grid_constant__ TreeConvArgs a, int piece) {
  constexpr int L = K - 1, PAIRS = VEC > 1 ? VEC / 2 : 1;
  using T = typename std::conditional<VEC == 8, uint4, typename std::conditional<VEC == 4, uint2, uint16_t>::type>::type;
  __shared__ const uint16_t* tap[kTcMost][K];  // channel 0 of a node's taps, oldest first; null: not part of the tree
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, at_piece = blockIdx.y;
  // sequence i's pieces start at cu[i] / piece + i, which leaves room for a cut last one
  // (pieces of one node need none)
  const int cut = piece > 1;
  int i = 0;
  for (int hi = a.t.nseq; hi - i > 1;) {
    const int m = (i + hi) / 2;
    if (a.t.cu[m] / piece + m * cut <= at_piece)
      i = m;
    else
      hi = m;
  }
  const int first = a.t.cu[i], n = a.t.cu[i + 1] - first, r0 = (at_piece - first / piece - i * cut) * piece;
  if (r0 >= n) return;
  if (threadIdx.x < 32) {
    const int pos = a.pos[i];
    uint64_t m[2];
    tree_masks(a.t.parent + first, n, lane, m);
    uint64_t path = tree_mask_of(m, min(r0 + lane, n - 1));
    if (lane < piece) {
      const bool in = path != 0;
      int slot = (pos % L + L) % L;
#pragma unroll
      for (int j = L; j >= 0; --j) {
        const uint16_t* p;
        if (path) {
          const int at = 63 - __clzll((long long)path);
          path &= ~(1ull << at);
          p = a.x + (size_t)(first + at) * a.ld_x;
        } else {
          slot = slot ? slot - 1 : L - 1;
          p = a.ring + ((size_t)i * L + slot) * a.C;
        }
        tap[lane][j] = in ? p : nullptr;
      }
    }
  }
  const int c = (blockIdx.x * kTcThreads + threadIdx.x) * VEC;
  const bool in = c < a.C;
  float2 w[K][PAIRS], b[PAIRS];  // of two channels
#pragma unroll
  for (int e = 0; e < PAIRS; ++e) {
    b[e] = make_float2(0.0f, 0.0f);
    if (!in) continue;
    if constexpr (VEC > 1) {
      T pack[K];
#pragma unroll
      for (int j = 0; j < K; ++j) pack[j] = reinterpret_cast<const T*>(a.w + (size_t)c * K)[j];
      auto part = [&](int at) {
        const uint32_t u = tc_word(pack[at / VEC], at % VEC / 2);
        return at & 1 ? bf16hi(u) : bf16lo(u);
      };
#pragma unroll
      for (int j = 0; j < K; ++j) w[j][e] = make_float2(part(2 * e * K + j), part((2 * e + 1) * K + j));
      if (a.bias) b[e] = tc_pair(tc_word(*reinterpret_cast<const T*>(a.bias + c), e));
    } else {
#pragma unroll
      for (int j = 0; j < K; ++j) w[j][e] = make_float2(bf16_to_f32(a.w[(size_t)c * K + j]), 0.0f);
      if (a.bias) b[e] = make_float2(bf16_to_f32(a.bias[c]), 0.0f);
    }
  }
  __syncthreads();
  if (!in) return;
  const int count = min(n - r0, piece);
  T next[K] = {};
  auto load = [&](int r) {
    if (!tap[r][0]) return;
#pragma unroll
    for (int j = 0; j < K; ++j) next[j] = *reinterpret_cast<const T*>(tap[r][j] + c);
  };
  load(0);
  uint16_t* out = a.out + (size_t)(first + r0) * a.ld_o + c;
#pragma unroll 1
  for (int r = 0; r < count; ++r, out += a.ld_o) {
    float2 s[PAIRS];
#pragma unroll
    for (int e = 0; e < PAIRS; ++e) {
      s[e] = b[e];
#pragma unroll
      for (int j = 0; j < K; ++j) {
        float2 v;
        if constexpr (VEC > 1)
          v = tc_pair(tc_word(next[j], e));
        else
          v = make_float2(bf16_to_f32(next[j]), 0.0f);
        s[e] = tc_fma2(w[j][e], v, s[e]);
      }
    }
    if (r + 1 < count) load(r + 1);
    if (a.silu) {
#pragma unroll
      for (int e = 0; e < PAIRS; ++e) {
        s[e].x = silu_f(s[e].x);
        if (VEC > 1) s[e].y = silu_f(s[e].y);
      }
    }
    const bool there = tap[r][0] != nullptr;
    if constexpr (VEC == 8)
      *reinterpret_cast<uint4*>(out) = there ? make_uint4(pack_bf16x2(s[0].x, s[0].y), pack_bf16x2(s[1].x, s[1].y),
                                                          pack_bf16x2(s[2].x, s[2].y), pack_bf16x2(s[3].x, s[3].y))
                                             : make_uint4(0u, 0u, 0u, 0u);
    else if constexpr (VEC == 4)
      *reinterpret_cast<uint2*>(out) =
          there ? make_uint2(pack_bf16x2(s[0].x, s[0].y), pack_bf16x2(s[1].x, s[1].y)) : make_uint2(0u, 0u);
    else
      *out = there ? f32_to_bf16(s[0].x) : (uint16_t)0;
  }
}

template <int VEC>
static cudaError_t launch_tree_conv_v(const TreeConvArgs& a, cudaStream_t s) {
  // One node a CTA while all of them run at once; then so many that they do.  For 2, 4, 5, 8,
  // 16 CTAs an SM: 16 x 4 nodes 5.4, 4.9, 4.1, 4.1, 4.1 us, 16 x 16 10.0, 7.1, 7.1, 8.6, 10.3,
  // 64 x 5 8.9, 8.9, 8.9, 11.7, 12.5.
  const int blocks = (a.C + kTcThreads * VEC - 1) / (kTcThreads * VEC), nodes = a.t.cu[a.t.nseq];
  int piece = 1;
  while (piece < kTcMost && (int64_t)blocks * nodes / piece > (int64_t)kTcCtas * num_sms()) piece *= 2;
  const dim3 grid(blocks, nodes / piece + (piece > 1 ? a.t.nseq : 0)), block(kTcThreads);
  switch (a.dconv) {
    case 2: return launch_k(tree_conv_kernel<2, VEC>, grid, block, 0, s, true, a, piece);
    case 3: return launch_k(tree_conv_kernel<3, VEC>, grid, block, 0, s, true, a, piece);
    case 4: return launch_k(tree_conv_kernel<4, VEC>, grid, block, 0, s, true, a, piece);
    case 5: return launch_k(tree_conv_kernel<5, VEC>, grid, block, 0, s, true, a, piece);
    case 6: return launch_k(tree_conv_kernel<6, VEC>, grid, block, 0, s, true, a, piece);
    case 7: return launch_k(tree_conv_kernel<7, VEC>, grid, block, 0, s, true, a, piece);
    default: return launch_k(tree_conv_kernel<8, VEC>, grid, block, 0, s, true, a, piece);
  }
}

cudaError_t launch_tree_conv(const TreeConvArgs& a, cudaStream_t s) {
  trace_pre(K_TREE_CONV, s);
  // Eight channels a thread, or four where eight leave SMs without a block: one chain of 5 nodes
  // and 10240 channels 3.0 / 2.5 us, 16 x 4 nodes 4.1 / 4.4, 16 x 64 20.3 / 22.0.
  const int blocks = (a.C + kTcThreads * 8 - 1) / (kTcThreads * 8);
  cudaError_t e;
  if (!a.wide)
    e = launch_tree_conv_v<1>(a, s);
  else
    e = blocks * a.t.cu[a.t.nseq] < num_sms() ? launch_tree_conv_v<4>(a, s) : launch_tree_conv_v<8>(a, s);
  trace_post(K_TREE_CONV, s);
  return e;
}

// ------------------------------------------------------------------ SSM outputs
//
// With la_j = dt_j A, s_i = the sum of la over node i's path and h the sequence's
// state (which is only read),
//   y_i = e^{s_i} C_i h^T + sum_{j on i's path} e^{s_i - s_j} dt_j (C_i . B_j) x_j + D x_i,
// three products on warp MMA (m16n8k16, bf16, fp32 sums): nodes are the rows,
//   C h^T    k = states, columns = channels p; a warp takes 8 channels (a lane's four
//            consecutive states stand at k = 2c, 2c+1, 2c+8, 2c+9; C is kept in the
//            same order)
//   C B^T    once for the heads of a group
//   L x      L the masked, decayed C B^T times dt
// h and L are fp32 and enter as three bf16 terms each, which hold all 24 bits; the
// smaller two have sums of their own.  s is a pair of floats (64 nodes of a chain
// would cost its differences their last bits).
// Values of x that are not finite would reach nodes beside their path as 0 * Inf: they
// are 0 in the product, and the nodes below them add them when they store.
// Bound: HBM, the state read once (32 KB a head of 64 x 128), up to 16 nodes: 64 chains of
// 5 take 57 us (4.9 TB/s), 16 trees of 16 19 us (of which 3 us pass until the first
// product), one chain 3.5 us; over a whole launch of 16 trees the split and the products take 56 %
// of the issue slots, HBM 42 %.  More nodes: warp MMA and what feeds it (16 x 32 nodes 29 us, 16 x
// 64 65 us).
//
// A CTA takes some heads of one group of a sequence.  Warps of two kinds: products (8 for
// the channels; 16 with 64 nodes, halves of the rows) and helpers, which make L and x of
// the next head under the current head's products; one barrier a head.  A product warp (a
// pair of them with 64 nodes) streams the 8 channels' states it reads through a ring of
// its own, three slots ahead, so that no barrier stands between a slot read and the next
// one asked for.
constexpr int kTsBlock = 64;   // channels of a head at once
constexpr int kTsSlots = 4;
constexpr int kTsSmemMax = 227 * 1024;

template <int N, int MT>
struct TsCfg {
  static constexpr int kNodes = 16 * MT;
  static constexpr int kRow = N + 16;        // bf16 elements between rows of the C and B tiles: no bank conflicts
  static constexpr int kCb = kNodes + 4;     // floats between rows of C B^T
  static constexpr int kL = kNodes + 8;      // bf16 elements between rows of L
  static constexpr int kTerms = 3 * kNodes * kL;  // elements of a head's L
  static constexpr int kK = N < 64 ? N : 64, kHalves = N / kK;  // states of a channel in a slot
  static constexpr int kSlot = 8 * kK;            // floats
  static constexpr int kGroups = MT == 4 ? 2 : 1, kTiles = MT / kGroups;  // product warps for a column, tiles of rows each
  static constexpr int kProd = 8 * kGroups, kHelp = 4 * kGroups, kWarps = kProd + kHelp;
  // the rows of C and B are read once, before the first L is written
  static constexpr int kLs = 2 * kTerms > 2 * kNodes * kRow ? 2 * kTerms : 2 * kNodes * kRow;
};
// Shared memory of a CTA: the rings, masks, C as operands, L's terms twice (and first the
// rows of C and B), x twice, C B^T, the heads' dt, s and e^s.
__host__ __device__ constexpr int ts_x_stride(int P) { return (P + 7) / 8 * 8 + 8; }
template <int N, int MT>
__host__ __device__ inline int ts_smem_bytes(int P, int heads) {
  using C = TsCfg<N, MT>;
  return 8 * kTsSlots * C::kSlot * 4 + C::kNodes * 8 + 32 + C::kNodes * N * 2 + C::kLs * 2 +
         2 * C::kNodes * ts_x_stride(P) * 2 + C::kNodes * C::kCb * 4 + heads * C::kNodes * 16;
}

__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
      "%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], const void* p) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(smem_addr(p))
               : "memory");
}
__device__ __forceinline__ void ldsm2_trans(uint32_t& r0, uint32_t& r1, const void* p) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x2.trans.shared.b16 {%0, %1}, [%2];"
               : "=r"(r0), "=r"(r1)
               : "r"(smem_addr(p))
               : "memory");
}
__device__ __forceinline__ void ts_copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void ts_copy8(void* dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(smem_addr(dst)), "l"(src) : "memory");
}
// Two floats as three pairs of bf16 whose sums they are: each takes the upper 8 bits of
// what is left, which is all 24 (truncation costs fewer instructions than rounding).
__device__ __forceinline__ void split3(float a, float b, uint32_t& hi, uint32_t& mid, uint32_t& lo) {
  const float2 minus = make_float2(-1.0f, -1.0f);
  float2 v = make_float2(a, b);
  auto rest = [&] {
    const float2 u = make_float2(__uint_as_float(__float_as_uint(v.x) & 0xFFFF0000u),
                                 __uint_as_float(__float_as_uint(v.y) & 0xFFFF0000u));
    v = tc_fma2(u, minus, v);
  };
  hi = __byte_perm(__float_as_uint(v.x), __float_as_uint(v.y), 0x7632);
  rest();
  mid = __byte_perm(__float_as_uint(v.x), __float_as_uint(v.y), 0x7632);
  rest();
  lo = __byte_perm(__float_as_uint(v.x), __float_as_uint(v.y), 0x7632);
}

template <int N, int MT>
__global__ void __launch_bounds__(TsCfg<N, MT>::kWarps * 32, MT == 4 ? 1 : 2)
    tree_ssm_kernel(const __grid_constant__ TreeSsmArgs a, int heads, int chunks) {
  using Cf = TsCfg<N, MT>;
  constexpr int KS = N / 16, NODES = Cf::kNodes, MG = Cf::kTiles, SLOTS = MT == 4 ? 2 : 1;
  extern __shared__ __align__(128) uint8_t smem[];
  const int xs = ts_x_stride(a.P);
  uint64_t* mask = reinterpret_cast<uint64_t*>(smem + 8 * kTsSlots * Cf::kSlot * 4);
  // nodes with x that is not finite, three heads in turn
  unsigned long long* bad = reinterpret_cast<unsigned long long*>(mask + NODES);
  uint4* cfrag = reinterpret_cast<uint4*>(bad + 4);  // C as a lane's operands of a tile and 16 states
  uint16_t* lt = reinterpret_cast<uint16_t*>(cfrag + MT * KS * 32);  // L's terms, heads in turn
  uint16_t *ct = lt, *bt = lt + NODES * Cf::kRow;
  uint16_t* xt = lt + Cf::kLs;           // x, heads in turn
  float* cb = reinterpret_cast<float*>(xt + 2 * NODES * xs);
  float* sdt = cb + NODES * Cf::kCb;     // [heads][NODES]
  float* shi = sdt + heads * NODES;
  float* slo = shi + heads * NODES;
  float* ses = slo + heads * NODES;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, r = lane >> 2, c = lane & 3;
  const int help = tid - Cf::kProd * 32;  // below 0: a product warp
  const int i = blockIdx.y, g = blockIdx.x / chunks, per = a.H / a.G;
  const int h0 = g * per + (blockIdx.x - g * chunks) * heads, nh = min(heads, (g + 1) * per - h0);
  const int first = a.t.cu[i], n = a.t.cu[i + 1] - first;
  if (tid < 3) bad[tid] = 0ull;
  __syncthreads();
  pdl_wait();
  pdl_trigger();
  if (n == 0) return;

  // ---- the states.  A slot holds kK states of 8 channels, 16-byte pieces of odd rows
  // with their 64-byte halves exchanged (no bank conflicts).  Every slot has a copy group.
  const int grp = warp / 8 % Cf::kGroups, pw = warp % 8 * 8;
  float* ring = reinterpret_cast<float*>(smem) + (warp & 7) * kTsSlots * Cf::kSlot;
  constexpr int Q = Cf::kK / 4, COPIES = (8 * Q + 31) / 32;  // pieces of a row; copies of a lane
  const int my_row = lane / Q, my_q = Q >= 8 ? lane % Q ^ (my_row & 1) * 4 : lane % Q;  // (rows a copy apart: an even number)
  const uint32_t ring_to = smem_addr(ring) + (my_row * Cf::kK + my_q * 4) * 4;
  const float* ask = a.h + (((size_t)i * a.H + h0) * a.P + pw + my_row) * N + lane % Q * 4;
  int ask_slot = 0, ask_p = pw, ask_head = pw < a.P ? 0 : nh;
  auto ask_state = [&](int half) {
    if (ask_head < nh) {
      const uint32_t to = ring_to + ask_slot * Cf::kSlot * 4;
      const float* from = ask + half * Cf::kK;
#pragma unroll
      for (int k = 0; k < COPIES; ++k) {
        // (with 64 nodes each warp of the pair asks for half)
        if (Cf::kGroups == 2 && (COPIES > 1 ? k % 2 != grp : grp)) continue;
        if (ask_p + my_row + k * (32 / Q) < a.P)
          ts_copy16(to + k * (32 / Q) * Cf::kK * 4, from + (size_t)k * (32 / Q) * N);
      }
      if (half == Cf::kHalves - 1) {
        ask += (size_t)kTsBlock * N;
        ask_p += kTsBlock;
        if (ask_p >= a.P) {
          ask -= (int64_t)(ask_p - pw - a.P) * N;
          ask_p = pw;
          ++ask_head;
        }
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    ask_slot = (ask_slot + 1) % kTsSlots;
  };
  // x of a head, 16 helpers a row: asked for, then looked through by the threads that asked
  // (wide), or both at once.  Columns past P hold anything: they only reach themselves.
  // (halves with all exponent bits set are infinities and NaN)
  auto finite = [](uint32_t w) {
    if ((w & 0x7F80u) == 0x7F80u) w &= 0xFFFF0000u;
    if ((w & 0x7F800000u) == 0x7F800000u) w &= 0xFFFFu;
    return w;
  };
  const int xq = help & 15, xj = help >> 4;
  auto ask_x = [&](int head) {
    uint16_t* d = xt + (head & 1) * NODES * xs;
#pragma unroll 1
    for (int j = xj; j < NODES; j += Cf::kHelp * 2) {
      const uint16_t* src = a.x + (size_t)(first + j) * a.ld_in + (size_t)(h0 + head) * a.P;
#pragma unroll 1
      for (int q = xq; q < (a.wide_x ? a.P / 4 : a.P); q += 16) {
        if (!a.wide_x) {
          const uint32_t v = j < n ? src[q] : 0u;
          const uint32_t f = finite(v);
          if (f != v) atomicOr(&bad[head % 3], 1ull << j);
          d[j * xs + q] = (uint16_t)f;
        } else if (j < n) {
          ts_copy8(d + j * xs + 4 * q, src + 4 * q);
        } else {
          *reinterpret_cast<uint2*>(d + j * xs + 4 * q) = make_uint2(0u, 0u);
        }
      }
    }
  };
  auto look_x = [&](int head) {  // (the copies have landed)
    if (!a.wide_x) return;
    uint16_t* d = xt + (head & 1) * NODES * xs;
#pragma unroll 1
    for (int j = xj; j < NODES; j += Cf::kHelp * 2)
#pragma unroll 1
      for (int q = xq; q < a.P / 4; q += 16) {
        uint2* p = reinterpret_cast<uint2*>(d + j * xs + 4 * q);
        const uint2 v = *p, f = make_uint2(finite(v.x), finite(v.y));
        if (f.x != v.x || f.y != v.y) {
          atomicOr(&bad[head % 3], 1ull << j);
          *p = f;
        }
      }
  };
  // L of a head: a lane keeps two columns (a bf16x2 word), `count` warps take rows in turn.
  // Blocks above the diagonal are never read.
  auto make_l = [&](int head, int w, int count) {
    constexpr int LPR = NODES / 2, RPW = 32 / LPR;
    const int col = lane % LPR * 2;
    const float2 dc = *reinterpret_cast<const float2*>(sdt + head * NODES + col);
    const float2 hc = *reinterpret_cast<const float2*>(shi + head * NODES + col);
    const float2 lc = *reinterpret_cast<const float2*>(slo + head * NODES + col);
    uint16_t* lh = lt + (head & 1) * Cf::kTerms + col;
#pragma unroll(MT == 4 ? 2 : 1)
    for (int row = w * RPW + lane / LPR; row < NODES; row += count * RPW) {
      if (col > (row | 15)) continue;
      const uint64_t m = mask[row] >> col;
      const float hr = shi[head * NODES + row], lr = slo[head * NODES + row];
      const float2 cv = *reinterpret_cast<const float2*>(cb + row * Cf::kCb + col);
      float v0 = expf((hr - hc.x) + (lr - lc.x)) * dc.x * cv.x, v1 = expf((hr - hc.y) + (lr - lc.y)) * dc.y * cv.y;
      v0 = m & 1 ? v0 : 0.0f;
      v1 = m & 2 ? v1 : 0.0f;
      uint32_t w0, w1, w2;
      split3(v0, v1, w0, w1, w2);
      uint32_t* d = reinterpret_cast<uint32_t*>(lh + row * Cf::kL);
      constexpr int T = NODES * Cf::kL / 2;  // words of a term
      d[0] = w0, d[T] = w1, d[2 * T] = w2;
    }
  };

  // ---- the start: dt and the decays' sums, C and B, masks.  What is small is asked for
  // before the states, whose pieces would fill the queues ahead of it.
  int32_t par[SLOTS];
  uint16_t raw[SLOTS];
  float A = 0.0f, bias = 0.0f;
  auto load_head = [&](int head) {  // a lane takes nodes l and l + 32
#pragma unroll
    for (int k = 0; k < SLOTS; ++k) {
      const int j = lane + 32 * k;
      if (j < n) raw[k] = a.dt[(size_t)(first + j) * a.ld_dt + h0 + head];
    }
    A = a.A_log[h0 + head];
    bias = a.dt_bias[h0 + head];
  };
#pragma unroll
  for (int k = 0; k < SLOTS; ++k) {
    par[k] = lane + 32 * k < n ? a.t.parent[first + lane + 32 * k] : -1;
    raw[k] = 0;
  }
  if (warp < nh) load_head(warp);
  if (help >= 0) ask_x(0);
  for (int k = tid; k < NODES * (N / 4); k += Cf::kWarps * 32) {
    const int j = k / (N / 4), e = k % (N / 4) * 4;
    if (j < n) {
      ts_copy8(ct + j * Cf::kRow + e, a.Cm + (size_t)(first + j) * a.ld_in + (size_t)g * N + e);
      ts_copy8(bt + j * Cf::kRow + e, a.Bm + (size_t)(first + j) * a.ld_in + (size_t)g * N + e);
    } else {
      *reinterpret_cast<uint2*>(ct + j * Cf::kRow + e) = make_uint2(0u, 0u);
      *reinterpret_cast<uint2*>(bt + j * Cf::kRow + e) = make_uint2(0u, 0u);
    }
  }
  asm volatile("cp.async.commit_group;" ::: "memory");
  if (help < 0)
    for (int k = 0; k < kTsSlots - 1; ++k) ask_state(k % Cf::kHalves);
  // A warp takes heads in turn: the sums double their reach as the masks do.  (Sums of
  // nodes outside the tree are never used.)
  for (int head = warp; head < nh; head += Cf::kWarps) {
    A = -expf(A);
    float hi[SLOTS], lo[SLOTS];
    int up[SLOTS];
#pragma unroll
    for (int k = 0; k < SLOTS; ++k) {
      const int j = lane + 32 * k;
      up[k] = par[k] < j ? par[k] : -1;
      float dt = softplus_f(bf16_to_f32(raw[k]) + bias);
      dt = j < n ? fminf(fmaxf(dt, 1e-9f), 1e9f) : 0.0f;
      if (j < NODES) sdt[head * NODES + j] = dt;
      hi[k] = dt * A;
      if (hi[k] < -0x1p100f) hi[k] = -0x1p100f;  // nothing is left of either; infinities would differ by NaN
      lo[k] = 0.0f;
    }
#pragma unroll 1
    for (int d = 1; d < n; d *= 2) {
      float nh_[SLOTS], nl[SLOTS];
      int nu[SLOTS];
#pragma unroll
      for (int k = 0; k < SLOTS; ++k) {
        float x = __shfl_sync(0xffffffffu, hi[0], up[k] & 31), y = __shfl_sync(0xffffffffu, lo[0], up[k] & 31);
        int u = __shfl_sync(0xffffffffu, up[0], up[k] & 31);
        if (SLOTS == 2) {
          const float x1 = __shfl_sync(0xffffffffu, hi[SLOTS - 1], up[k] & 31);
          const float y1 = __shfl_sync(0xffffffffu, lo[SLOTS - 1], up[k] & 31);
          const int u1 = __shfl_sync(0xffffffffu, up[SLOTS - 1], up[k] & 31);
          if (up[k] & 32) x = x1, y = y1, u = u1;
        }
        nh_[k] = hi[k], nl[k] = lo[k], nu[k] = up[k];
        if (up[k] >= 0) {
          two_sum_acc(nh_[k], nl[k], x);
          nl[k] += y;
          nu[k] = u < 0 ? -1 : u;
        }
      }
#pragma unroll
      for (int k = 0; k < SLOTS; ++k) hi[k] = nh_[k], lo[k] = nl[k], up[k] = nu[k];
    }
#pragma unroll
    for (int k = 0; k < SLOTS; ++k) {
      const int j = head * NODES + lane + 32 * k;
      if (lane + 32 * k >= NODES) continue;
      shi[j] = hi[k], slo[j] = lo[k];
      ses[j] = expf(hi[k] + lo[k]);
    }
    if (head + Cf::kWarps < nh) load_head(head + Cf::kWarps);
  }
  if (warp == Cf::kWarps - 1) {
    uint64_t m[2];
    tree_masks(a.t.parent + first, n, lane, m);
    if (lane < NODES) mask[lane] = m[0];
    if (MT == 4) mask[lane + 32] = m[1];
  }
  if (help < 0)
    asm volatile("cp.async.wait_group %0;" ::"n"(kTsSlots - 1) : "memory");
  else
    asm volatile("cp.async.wait_group 0;" ::: "memory");
  __syncthreads();
  for (int k = warp; k < MT * KS; k += Cf::kWarps) {
    const uint16_t* cs = ct + (k / KS * 16 + r) * Cf::kRow + k % KS * 16 + 4 * c;
    const uint2 a0 = *reinterpret_cast<const uint2*>(cs), a1 = *reinterpret_cast<const uint2*>(cs + 8 * Cf::kRow);
    cfrag[k * 32 + lane] = make_uint4(a0.x, a1.x, a0.y, a1.y);
  }
  // ---- C B^T
  for (int k = warp; k < MT * 2 * MT; k += Cf::kWarps) {
    const int mt = k / (2 * MT), nt = k % (2 * MT);
    if (nt > 2 * mt + 1) continue;  // above the diagonal: no node stands above one before it
    float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      const uint2 a0 = *reinterpret_cast<const uint2*>(ct + (16 * mt + r) * Cf::kRow + 16 * ks + 4 * c);
      const uint2 a1 = *reinterpret_cast<const uint2*>(ct + (16 * mt + 8 + r) * Cf::kRow + 16 * ks + 4 * c);
      const uint2 b = *reinterpret_cast<const uint2*>(bt + (8 * nt + r) * Cf::kRow + 16 * ks + 4 * c);
      mma_bf16(acc, a0.x, a1.x, a0.y, a1.y, b.x, b.y);
    }
    float* d = cb + (16 * mt + r) * Cf::kCb + 8 * nt + 2 * c;
    *reinterpret_cast<float2*>(d) = make_float2(acc[0], acc[1]);
    *reinterpret_cast<float2*>(d + 8 * Cf::kCb) = make_float2(acc[2], acc[3]);
  }
  if (help >= 0) look_x(0);
  __syncthreads();
  make_l(0, warp, Cf::kWarps);

  if (help >= 0) {
    for (int head = 0; head < nh; ++head) {
      __syncthreads();
      if (help == 0) bad[(head + 2) % 3] = 0ull;  // read by all before, next written behind the next barrier
      if (head + 1 == nh) break;
      ask_x(head + 1);
      asm volatile("cp.async.commit_group;" ::: "memory");
      make_l(head + 1, warp - Cf::kProd, Cf::kHelp);
      asm volatile("cp.async.wait_group 0;" ::: "memory");
      look_x(head + 1);
    }
    return;
  }

  // ---- the products
  auto tile = [&](int q) { return MT == 4 ? (q ? 3 - grp : grp) : q; };  // (L's blocks: 1 + 4 and 2 + 3)
  unsigned live = 0;  // the thread's rows that are part of the tree
#pragma unroll
  for (int q = 0; q < MG; ++q)
#pragma unroll
    for (int e = 0; e < 2; ++e) live |= (mask[16 * tile(q) + r + 8 * e] != 0 ? 1u : 0u) << (2 * q + e);
  const int HP = a.H * a.P;
  float* yr = a.y + (size_t)(first + r) * HP + h0 * a.P + pw + 2 * c;
  int slot = 0;
  for (int head = 0; head < nh; ++head, yr += a.P) {
    const int h = h0 + head;
    const float Dh = a.D[h];
    const uint16_t* lh = lt + (head & 1) * Cf::kTerms;
    const uint16_t* xh = xt + (head & 1) * NODES * xs;
    __syncthreads();  // L and x of this head are there, those of the one before are read
    const uint64_t odd = bad[head % 3];
    for (int p0 = pw; p0 < a.P; p0 += kTsBlock) {
      const int p = p0 + 2 * c;
      // L x
      float t[MG][4];
#pragma unroll
      for (int q = 0; q < MG; ++q) {
        const int mt = tile(q);
        float top[4] = {0.0f, 0.0f, 0.0f, 0.0f}, low[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll(MT == 4 ? 1 : 2)
        for (int ks = 0; ks <= mt; ++ks) {
          uint32_t b0, b1, l[4];
          ldsm2_trans(b0, b1, xh + (16 * ks + (lane & 15)) * xs + p0);
          const uint16_t* ls = lh + (16 * mt + (lane & 15)) * Cf::kL + 16 * ks + (lane >> 4) * 8;
          ldsm4(l, ls);
          mma_bf16(top, l[0], l[1], l[2], l[3], b0, b1);
          ldsm4(l, ls + NODES * Cf::kL);
          mma_bf16(low, l[0], l[1], l[2], l[3], b0, b1);
          ldsm4(l, ls + 2 * NODES * Cf::kL);
          mma_bf16(low, l[0], l[1], l[2], l[3], b0, b1);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) t[q][e] = top[e] + low[e];
      }
      // C h^T, the smaller terms' sums apart
      float acc[MG][4], low[MG][4];
#pragma unroll
      for (int q = 0; q < MG; ++q)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[q][e] = low[q][e] = 0.0f;
#pragma unroll
      for (int half = 0; half < Cf::kHalves; ++half) {
        asm volatile("cp.async.wait_group %0;" ::"n"(kTsSlots - 2) : "memory");
        if (Cf::kGroups == 2)
          named_bar(1 + warp % 8, 64);  // the other warp's part has landed too, and both have read the slot before
        else
          __syncwarp();
        ask_state((half + kTsSlots - 1) % Cf::kHalves);
        const float* hs = ring + slot * Cf::kSlot + r * Cf::kK;
        slot = (slot + 1) % kTsSlots;
#pragma unroll
        for (int kk = 0; kk < Cf::kK / 16; ++kk) {
          const int ks = half * (Cf::kK / 16) + kk;
          const float4 hk = *reinterpret_cast<const float4*>(hs + (Cf::kK >= 32 ? (4 * kk + c) ^ (r & 1) * 4 : c) * 4);
          uint32_t b0[3], b1[3];
          split3(hk.x, hk.y, b0[0], b0[1], b0[2]);
          split3(hk.z, hk.w, b1[0], b1[1], b1[2]);
#pragma unroll
          for (int q = 0; q < MG; ++q) {
            const uint4 f = cfrag[(tile(q) * KS + ks) * 32 + lane];
            mma_bf16(low[q], f.x, f.y, f.z, f.w, b0[2], b1[2]);
            mma_bf16(acc[q], f.x, f.y, f.z, f.w, b0[0], b1[0]);
            mma_bf16(low[q], f.x, f.y, f.z, f.w, b0[1], b1[1]);
          }
        }
      }
#pragma unroll
      for (int q = 0; q < MG; ++q)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int j = 16 * tile(q) + r + 8 * e;
          if (j >= n || p >= a.P) continue;
          const uint32_t xw = *reinterpret_cast<const uint32_t*>(xh + j * xs + p);
          const float es = ses[head * NODES + j];
          float y[2];
#pragma unroll
          for (int f = 0; f < 2; ++f) {
            const int at = 2 * e + f;
            y[f] = fmaf(Dh, f ? bf16hi(xw) : bf16lo(xw), fmaf(acc[q][at] + low[q][at], es, t[q][at]));
            if (!(live >> (2 * q + e) & 1)) y[f] = 0.0f;
          }
          if (odd) {
            for (uint64_t o = mask[j] & odd; o; o &= o - 1) {
              const int at = __ffsll((long long)o) - 1;
              float l = 0.0f;
              for (int k = 2; k >= 0; --k) l += bf16_to_f32(lh[k * NODES * Cf::kL + j * Cf::kL + at]);
              for (int f = 0; f < 2 && p + f < a.P; ++f) {
                const float v = bf16_to_f32(a.x[(size_t)(first + at) * a.ld_in + (size_t)h * a.P + p + f]);
                if (!isfinite(v)) y[f] += (at == j ? l + Dh : l) * v;
              }
            }
          }
          float* d = yr + (size_t)(j - r) * HP + (p0 - pw);  // (past 2^31 elements where H * P is large)
          if (a.P % 2 == 0) {
            *reinterpret_cast<float2*>(d) = make_float2(y[0], y[1]);
          } else {
            d[0] = y[0];
            if (p + 1 < a.P) d[1] = y[1];
          }
        }
    }
  }
}

template <int N, int MT>
static cudaError_t launch_tree_ssm_n(const TreeSsmArgs& a, cudaStream_t s) {
  static int done_mask[64] = {0};
  const int per = a.H / a.G;
  // Heads of a CTA.  Its start (masks, C B^T, the sums) takes as long as 1.5 heads and
  // serves all of them; an SM works through its CTAs, of which two side by side take 0.7
  // of what they take one after the other (64 nodes: one at a time).  Of 16, 8, 4, 2 and 1
  // the one that comes out least; us for 128 heads of 64 x 128 in 8 groups:
  //                          16     8      4      2      1
  //   4 sequences x 16              -      7.4    6.6    8.2
  //   16 x 16                24.2   19.2   20.9   22.8
  //   64 x 5                 61.6   56.8
  //   16 x 64                65.1   69.0   77.1
  int heads = 1;
  double least = 0.0;
  for (int h = per < 16 ? per : 16;; h = (h + 1) / 2) {
    const int64_t ctas = (int64_t)a.t.nseq * a.G * ((per + h - 1) / h), turns = (ctas + num_sms() - 1) / num_sms();
    const double one = h + 1.5, all = MT == 4 || turns == 1 ? turns * one : 0.7 * turns * one;
    if (ts_smem_bytes<N, MT>(a.P, h) <= kTsSmemMax && (least == 0.0 || all < least)) heads = h, least = all;
    if (h == 1) break;
  }
  const int chunks = (per + heads - 1) / heads, smem = ts_smem_bytes<N, MT>(a.P, heads);
  auto k = tree_ssm_kernel<N, MT>;
  // (one limit whatever the call: no call lowers another's)
  cudaError_t e = set_smem_once((const void*)k, kTsSmemMax, done_mask);
  if (e != cudaSuccess) return e;
  return launch_k(k, dim3(a.G * chunks, a.t.nseq), dim3(TsCfg<N, MT>::kWarps * 32), smem, s, true, a, heads, chunks);
}
template <int N>
static cudaError_t launch_tree_ssm_m(const TreeSsmArgs& a, int most, cudaStream_t s) {
  // Rows for 16, 32 or 64 nodes.  us with 16 / 32 / 64, 128 heads as above: 16 sequences x 16
  // nodes 19.2 / 27.5 / 60, 64 x 5 56.8 / 85.5 / 215, one x 5 3.5 / 4.5 / 7.4; 16 x 32 - / 29.4 / 61.4.
  // The launch's largest tree decides for all: conv and outputs of 63 x 5 and one x 64 take 232 us,
  // of 64 x 5 66.
  return most <= 16   ? launch_tree_ssm_n<N, 1>(a, s)
         : most <= 32 ? launch_tree_ssm_n<N, 2>(a, s)
                      : launch_tree_ssm_n<N, 4>(a, s);
}

cudaError_t launch_tree_ssm(const TreeSsmArgs& a, cudaStream_t s) {
  int most = 0;
  for (int i = 0; i < a.t.nseq; ++i) most = a.t.cu[i + 1] - a.t.cu[i] > most ? a.t.cu[i + 1] - a.t.cu[i] : most;
  cudaError_t e;
  trace_pre(K_TREE_SSM, s);
  switch (a.N) {
    case 16: e = launch_tree_ssm_m<16>(a, most, s); break;
    case 32: e = launch_tree_ssm_m<32>(a, most, s); break;
    case 64: e = launch_tree_ssm_m<64>(a, most, s); break;
    default: e = launch_tree_ssm_m<128>(a, most, s); break;
  }
  trace_post(K_TREE_SSM, s);
  return e;
}

// ------------------------------------------------------------------ commit
//
// One launch: the state's blocks, and a block a sequence for ring and position, which it
// stores (perhaps in place) once all of it has read the old one.  It never starts its
// successor early: the conv of a decode step reads ring and position while the launch
// before it may still run.  (With the ring in a launch of its own: one sequence 5.9 us
// instead of 5.5, two 7.0 instead of 5.9, no difference from four on.)
// Channels that cannot be moved 16 bytes at a time take two launches: first the ring's, a
// cluster a sequence, then the state's, which may start its successor early.

// Accepted nodes of sequence i, within its tree.
__device__ __forceinline__ int tree_count(const TreeArgs& t, const int32_t* count, int i) {
  const int n = t.cu[i + 1] - t.cu[i], k = count[i];
  if (k < 0 || k > n) atomicCAS(&g_status, 0, -1);
  return max(0, min(k, n));
}
// Row of the path's entry j, or -1 (reported) if it names no node.
__device__ __forceinline__ int tree_path_row(const TreeArgs& t, int i, int j) {
  const int first = t.cu[i], at = t.parent[first + j];
  if (at >= 0 && at < t.cu[i + 1] - first) return first + at;
  atomicCAS(&g_status, 0, -1);
  return -1;
}

constexpr int kTrThreads = 256, kTrCtas = 8;

// The ring of sequence i, channels from VEC * at on, VEC * step apart; the path's n nodes, position pos.
template <int VEC>
__device__ __forceinline__ void tree_ring(const TreeCommitArgs& a, int i, int n, int pos, int at, int step) {
  using T = typename std::conditional<VEC == 8, uint4, uint16_t>::type;
  const int L = a.dconv - 1, C = a.H * a.P + 2 * a.G * a.N;
  const uint16_t* in = a.ring + (size_t)i * L * C;
  uint16_t* out = a.ring_out + (size_t)i * L * C;
  for (int slot = 0; slot < L; ++slot) {
    // the newest token of the path in this slot: the last j < n with (pos + j) % L == slot
    const int p = ((pos + n - 1 - slot) % L + L) % L, j = n - 1 - p;
    const int row = j >= 0 ? tree_path_row(a.t, i, j) : -1;
    if (row < 0 && in == out) continue;
    const uint16_t* from = row >= 0 ? a.xbc + (size_t)row * a.ld_xbc : in + (size_t)slot * C;
#pragma unroll 4
    for (int c = at * VEC; c < C; c += step * VEC)
      *reinterpret_cast<T*>(out + (size_t)slot * C + c) = *reinterpret_cast<const T*>(from + c);
  }
}

__global__ void __launch_bounds__(kTrThreads) __cluster_dims__(kTrCtas, 1, 1) tree_ring_kernel(const TreeCommitArgs a) {
  pdl_wait();
  pdl_trigger();
  const int i = blockIdx.y, n = tree_count(a.t, a.count, i), pos = a.pos[i];
  tree_ring<1>(a, i, n, pos, blockIdx.x * kTrThreads + threadIdx.x, kTrCtas * kTrThreads);
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
  if (blockIdx.x == 0 && threadIdx.x == 0) a.pos_out[i] = pos + n;
}

__device__ __forceinline__ float4 tc_bf4(const uint16_t* p) {
  const uint2 v = *reinterpret_cast<const uint2*>(p);
  return make_float4(bf16lo(v.x), bf16hi(v.x), bf16lo(v.y), bf16hi(v.y));
}

// The steps of the single-token kernel, in its order and arithmetic, with the state
// in registers: LPR = N/4 lanes a row, ROWS rows a thread.  What the path's nodes bring
// (dt and decay, B, this CTA's channels of x) comes into shared memory in one trip, under
// the state's loads: a CTA's stay is what limits the bytes in flight.
// Bound: HBM, the state read and written once.
template <int LPR, int ROWS>
__global__ void __launch_bounds__(256) tree_state_kernel(const TreeCommitArgs a, int psplit) {
  constexpr int RPW = 32 / LPR, CTA_ROWS = 8 * RPW * ROWS;
  extern __shared__ __align__(128) uint8_t smem[];  // [nodes] of B (N bf16), of x (CTA_ROWS fp32)
  __shared__ float sdt[kTreeNodes], sda[kTreeNodes];
  __shared__ int srow[kTreeNodes];
  const int i = blockIdx.y, block = (int)blockIdx.x - (a.wide ? 1 : 0), tid = threadIdx.x;
  const int h = block / psplit, pc = block % psplit;
  const int warp = tid >> 5, lane = tid & 31, n4 = (lane % LPR) * 4, g = h / (a.H / a.G);
  const size_t base = ((size_t)i * a.H + h) * a.P * a.N;
  const int r0 = warp * RPW + lane / LPR, p0 = pc * CTA_ROWS + r0;
  pdl_wait();
  if (!a.wide) pdl_trigger();
  if (block < 0) {  // the ring's
    const int n = tree_count(a.t, a.count, i), pos = a.pos[i];
    tree_ring<8>(a, i, n, pos, tid, 256);
    __syncthreads();
    if (tid == 0) a.pos_out[i] = pos + n;
    return;
  }
  float4 hv[ROWS];
#pragma unroll
  for (int k = 0; k < ROWS; ++k) {
    const int p = p0 + k * 8 * RPW;
    if (p < a.P) hv[k] = *reinterpret_cast<const float4*>(a.h + base + (size_t)p * a.N + n4);
  }
  const int n = tree_count(a.t, a.count, i);
  float* sx = reinterpret_cast<float*>(smem);
  uint16_t* sb = reinterpret_cast<uint16_t*>(sx + n * CTA_ROWS);
  if (tid < n) {
    const int row = tree_path_row(a.t, i, tid);
    float dt = 0.0f, da = 1.0f;
    if (row >= 0) ssm_dt_dA(bf16_to_f32(a.dt[(size_t)row * a.ld_dt + h]), a.dt_bias[h], a.A_log[h], dt, da);
    srow[tid] = row;
    sdt[tid] = dt;
    sda[tid] = da;
  }
  __syncthreads();
  for (int k = tid; k < n * (LPR + CTA_ROWS); k += 256) {
    const int j = k / (LPR + CTA_ROWS), e = k - j * (LPR + CTA_ROWS), row = srow[j];
    if (row < 0) continue;
    const uint16_t* u = a.u + (size_t)row * a.ld_u;
    if (e < LPR)
      *reinterpret_cast<uint2*>(sb + j * a.N + 4 * e) =
          *reinterpret_cast<const uint2*>(u + (size_t)a.H * a.P + (size_t)g * a.N + 4 * e);
    else if (pc * CTA_ROWS + e - LPR < a.P)
      sx[j * CTA_ROWS + e - LPR] = sdt[j] * bf16_to_f32(u[(size_t)h * a.P + pc * CTA_ROWS + e - LPR]);
  }
  __syncthreads();
  for (int j = 0; j < n; ++j) {
    if (srow[j] < 0) continue;
    const float dA = sda[j];
    const float4 Bv = tc_bf4(sb + j * a.N + n4);
#pragma unroll
    for (int k = 0; k < ROWS; ++k) {
      const float dtx = sx[j * CTA_ROWS + r0 + k * 8 * RPW];  // (of no use past the last channel)
      hv[k].x = fmaf(dA, hv[k].x, dtx * Bv.x);
      hv[k].y = fmaf(dA, hv[k].y, dtx * Bv.y);
      hv[k].z = fmaf(dA, hv[k].z, dtx * Bv.z);
      hv[k].w = fmaf(dA, hv[k].w, dtx * Bv.w);
    }
  }
#pragma unroll
  for (int k = 0; k < ROWS; ++k) {
    const int p = p0 + k * 8 * RPW;
    if (p < a.P) *reinterpret_cast<float4*>(a.h_out + base + (size_t)p * a.N + n4) = hv[k];
  }
}

static cudaError_t launch_tree_ring(const TreeCommitArgs& a, cudaStream_t s) {
  trace_pre(K_TREE_RING, s);
  const cudaError_t e = launch_k(tree_ring_kernel, dim3(kTrCtas, a.t.nseq), dim3(kTrThreads), 0, s, true, a);
  trace_post(K_TREE_RING, s);
  return e;
}

template <int LPR>
static cudaError_t launch_tree_state(const TreeCommitArgs& a, cudaStream_t s) {
  constexpr int RPW = 32 / LPR;
  const int64_t heads = (int64_t)a.t.nseq * a.H;
  const int max_rows = (a.P + 8 * RPW - 1) / (8 * RPW);
  // rows a thread: doubled while the grid has more CTAs than four an SM.  us for 1, 2, 4, 8 rows,
  // 128 heads of 64 x 128: one sequence 6.6, 6.1, 5.9, 6.2, 16 sequences 49.7, 39.1, 33.5, 32.3, 64
  // 174, 132, 106, 98
  int rows = 1;
  while (rows < 8 && rows < max_rows && heads * ((a.P + 8 * RPW * rows - 1) / (8 * RPW * rows)) > 4ll * num_sms()) rows *= 2;
  const int psplit = (a.P + 8 * RPW * rows - 1) / (8 * RPW * rows);
  const dim3 grid(a.H * psplit + (a.wide ? 1 : 0), a.t.nseq), block(256);
  int most = 0;
  for (int i = 0; i < a.t.nseq; ++i) most = a.t.cu[i + 1] - a.t.cu[i] > most ? a.t.cu[i + 1] - a.t.cu[i] : most;
  const int each = a.N * 2 + 8 * RPW * rows * 4, smem = most * each;  // at most 64 * (32 + 2048) bytes: N = 16
  auto go = [&](void (*k)(TreeCommitArgs, int), int* done_mask) {
    // One limit whatever the call's trees (beside it a block has 768 bytes of its own), and asked for before anything
    // is launched: a refusal leaves ring and position as they were.
    cudaError_t e = set_smem_once((const void*)k, kTreeNodes * each, done_mask);
    if (e == cudaSuccess && !a.wide) e = launch_tree_ring(a, s);
    if (e != cudaSuccess) return e;
    trace_pre(K_TREE_STATE, s);
    e = launch_k(k, grid, block, smem, s, true, a, psplit);
    trace_post(K_TREE_STATE, s);
    return e;
  };
  static int done[4][64] = {{0}};
  switch (rows) {
    case 1: return go(tree_state_kernel<LPR, 1>, done[0]);
    case 2: return go(tree_state_kernel<LPR, 2>, done[1]);
    case 4: return go(tree_state_kernel<LPR, 4>, done[2]);
    default: return go(tree_state_kernel<LPR, 8>, done[3]);
  }
}

cudaError_t launch_tree_commit(const TreeCommitArgs& a, cudaStream_t s) {
  switch (a.N / 4) {
    case 4: return launch_tree_state<4>(a, s);
    case 8: return launch_tree_state<8>(a, s);
    case 16: return launch_tree_state<16>(a, s);
    default: return launch_tree_state<32>(a, s);
  }
}

int status_tree(int clear) { return tu_status(clear); }

}  // namespace m2
