// k_verify.cu -- verification of drafted tokens (include/mamba2.h has the rule).
//
// The walk itself is a few comparisons; what takes time is a row of the target (and of
// the draft): one for the token that the walk ends on, one for every sibling that is
// asked after a refusal.  A cluster of 8 CTAs takes a sequence, its CTAs and their warps
// consecutive runs of the vocabulary.  Every CTA gathers the probabilities that the walk
// asks for and walks by itself, the same way, until it needs a sum
//   S = sum_t R(t),  R = max(p - c q, 0)
// whose parts all CTAs give each other: one hand-over a pass.  The last sum's parts, by
// CTA and warp, say which warp's run the random number falls into; that CTA reads it
// again, from L2.
// A refusal takes S q from what remains, so that c grows by S: R never has to be
// stored, whatever the number of refusals.
// R and its sums are pairs of floats (about 2^-46 of the sum; fp64 adds are slow here),
// comparisons fp64: a sum in fp32 would move one drawn token in some thousand.
// Bound: latency, of the passes one after another and of a pass's loads (DRAM 23 %, issue slots
// 28 %): 64 sequences of 5 to 8 nodes over 131072 words 28.4 us (67 MB, 2.4 TB/s; a pass over a
// row 4 to 6 us), from bf16 rows 38, without draft rows 18; over 50256 words 16.3, over 50257
// (rows of fp32 that are not 16-byte aligned) 21.6.  A chain of 5 over 32000 words 6.5 us.
#include <cuda_runtime.h>
#include <stdint.h>

#include "m2_common.cuh"
#include "m2_kernels.h"
#include "m2_tc_attn.cuh"
#include "m2_tree.cuh"

namespace m2 {

constexpr int kVfThreads = 256, kVfWarps = kVfThreads / 32, kVfCtas = 8;

enum { VF_SUM = 0, VF_DRAW = 1 };
struct VfCmd {
  int32_t what, cur;
  float c_hi, c_lo;
  int32_t gone;      // refused tokens, where there is no draft row: their number
};
struct VfShared {
  float tot_hi[2][kVfCtas], tot_lo[2][kVfCtas];  // the CTAs' sums, passes in turn
  VfCmd cmd;
  int32_t gone_tok[kTreeNodes];
  float hi[kVfWarps], lo[kVfWarps];
  int32_t parent[kTreeNodes], token[kTreeNodes], path[kTreeNodes];
  float u[kTreeNodes], p[kTreeNodes], q[kTreeNodes];
  int32_t count;     // accepted nodes so far
  int32_t run;       // drawing: the run that the random number falls into (-1: another CTA's, -2: the row is empty)
  double want;       // and what is left of the number there
  float scan_hi[kVfWarps], scan_lo[kVfWarps];
  int32_t owner, last;
};

// Probabilities that are not positive numbers count as 0.
__device__ __forceinline__ float vf_clean(float x) {  // as integers: 1 .. the largest finite value
  return __float_as_uint(x) - 1u < 0x7F7FFFFFu ? x : 0.0f;
}
template <bool BF>
__device__ __forceinline__ float vf_one(const void* row, int64_t at) {
  return vf_clean(BF ? bf16_to_f32(static_cast<const uint16_t*>(row)[at]) : static_cast<const float*>(row)[at]);
}
// Four of a row from element `at` on as they are; past the end 0.  wide: they can be read at once.
template <bool BF>
__device__ __forceinline__ float4 vf_raw(const void* row, int at, int V, bool wide) {
  float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  if (wide && at + 4 <= V) {
    if (BF) {
      const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(row) + at);
      return make_float4(bf16lo(w.x), bf16hi(w.x), bf16lo(w.y), bf16hi(w.y));
    }
    return *reinterpret_cast<const float4*>(static_cast<const float*>(row) + at);
  }
  auto one = [&](int x) { return BF ? bf16_to_f32(static_cast<const uint16_t*>(row)[x]) : static_cast<const float*>(row)[x]; };
  if (at < V) v.x = one(at);
  if (at + 1 < V) v.y = one(at + 1);
  if (at + 2 < V) v.z = one(at + 2);
  if (at + 3 < V) v.w = one(at + 3);
  return v;
}
template <bool BF>
__device__ __forceinline__ float4 vf_four(const void* row, int at, int V, bool wide) {
  const float4 v = vf_raw<BF>(row, at, V, wide);
  return make_float4(vf_clean(v.x), vf_clean(v.y), vf_clean(v.z), vf_clean(v.w));
}
// (hi, lo) += R of one token; whether there is any.  p - c q in fp32, s, and what its additions and
// the product lost, d: their sum's sign is R's, also where c q is p but for its rounding (s is then 0
// or one place off either way).
__device__ __forceinline__ bool vf_add(float& hi, float& lo, float p, float q, float c_hi, float c_lo) {
  const float t = __fmul_rn(c_hi, q), s = p - t;  // (never one fused step: d needs the product as it was rounded)
  const float d = ((p - s) - t) - fmaf(c_lo, q, fmaf(c_hi, q, -t));
  if (!(s + d > 0.0f)) return false;
  two_sum_acc(hi, lo, s);
  lo += d;
  return true;
}
// The pair with its sum in hi: hi is positive where the sum is.
__device__ __forceinline__ void vf_norm(float& hi, float& lo) {
  const float s = hi + lo;
  lo -= s - hi;
  hi = s;
}
// Two tokens a lane at once.  What is not positive, NaN among it, counts as 0 here;
// infinities are found afterwards (`most` of the draft, the sum of the target).
__device__ __forceinline__ float2 vf_sub2(float2 a, float2 b) { return ffma2(b, make_float2(-1.0f, -1.0f), a); }
__device__ __forceinline__ void vf_sum2(float2& hi, float2& lo, float2 s) {
  const float2 t = fadd2(hi, s), z = vf_sub2(t, hi);
  lo = fadd2(lo, fadd2(vf_sub2(hi, vf_sub2(t, z)), vf_sub2(s, z)));
  hi = t;
}
template <bool ONE>  // c is 1
__device__ __forceinline__ void vf_add2(float2& hi, float2& lo, float2 p, float2 q, float c_hi, float c_lo, float& most) {
  p = make_float2(fmaxf(p.x, 0.0f), fmaxf(p.y, 0.0f));
  q = make_float2(fmaxf(q.x, 0.0f), fmaxf(q.y, 0.0f));
  most = max3(most, q.x, q.y);
  const float2 cq = ONE ? q : make_float2(c_hi * q.x, c_hi * q.y);
  // (c = 1: the product is exact, so that s alone says what is left)
  const float2 t = ONE ? make_float2(fminf(cq.x, p.x), fminf(cq.y, p.y)) : cq;
  float2 s = vf_sub2(p, t), d = vf_sub2(vf_sub2(p, s), t);
  if (!ONE) {
    const float2 e = make_float2(fmaf(c_lo, q.x, fmaf(c_hi, q.x, -t.x)), fmaf(c_lo, q.y, fmaf(c_hi, q.y, -t.y)));
    d = vf_sub2(d, e);
    const bool x = s.x + d.x > 0.0f, y = s.y + d.y > 0.0f;
    s = make_float2(x ? s.x : 0.0f, y ? s.y : 0.0f);
    d = make_float2(x ? d.x : 0.0f, y ? d.y : 0.0f);
  }
  vf_sum2(hi, lo, s);
  lo = fadd2(lo, d);
}

__device__ __forceinline__ void vf_cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void vf_cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void vf_cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
// A word of this CTA's shared memory at the same place in CTA `rank` of the cluster.
__device__ __forceinline__ void vf_put(void* at, int rank, uint32_t v) {
  asm volatile("{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %0, %1;\n\tst.shared::cluster.u32 [a], %2;\n\t}" ::"r"(
                   smem_addr(at)),
               "r"(rank), "r"(v)
               : "memory");
}

// u q S < p - c q (a < b, where b is 0 at least), in fp32 where that decides it: its error is
// below 2^-21 of the three products.  Else in 64 bits, whose latency here is that of a sum.
__device__ __forceinline__ bool vf_less(float u, float q, double S, float p, double c) {
  const float a = u * q * (float)S, t = (float)c * q, b = fmaxf(p - t, 0.0f);
  if (fabsf(a - b) > 9.5367431640625e-7f * (fabsf(a) + p + t)) return a < b;  // 2^-20
  const double left = (double)p - c * q;
  return (double)u * q * S < (left > 0.0 ? left : 0.0);
}

// The walk up to the next sum.  One thread of every CTA holds this.
struct VfWalk {
  int cur, r, count, gone;
  bool known, last;  // S is; the draw was from the untouched row already
  double c, S;
};

template <bool BF>
__global__ void __launch_bounds__(kVfThreads, 4) __cluster_dims__(kVfCtas, 1, 1) verify_tree_kernel(const VerifyArgs a) {
  __shared__ VfShared sh;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, rank = blockIdx.x, i = blockIdx.y;
  const int first = a.t.cu[i], n = a.t.cu[i + 1] - first, V = a.V;
  constexpr int ES = BF ? 2 : 4;
  pdl_wait();
  pdl_trigger();
  vf_cluster_arrive();  // waited for before the first word goes to another CTA, which has to run by then
  auto row_of = [&](const void* m, int64_t ld, int node) {
    return static_cast<const void*>(static_cast<const char*>(m) + (int64_t)(first + node) * ld * ES);
  };
  if (tid < n) {
    const int par = a.t.parent[first + tid], x = a.token[first + tid];
    const bool in = tid > 0 && par >= 0 && par < tid, tok = x >= 0 && x < V;
    sh.parent[tid] = tid == 0 ? par : in ? par : -1;
    sh.token[tid] = tok ? x : -1;
    sh.u[tid] = a.u[first + tid];
    sh.p[tid] = in && tok ? vf_one<BF>(row_of(a.p, a.ld_p, par), x) : 0.0f;
    sh.q[tid] = in && tok && a.q ? vf_one<BF>(row_of(a.q, a.ld_q, par), x) : 0.0f;
  }
  __syncthreads();
  if (n == 0 || a.t.parent[first] != -1) {  // nothing to start from (the same for the whole cluster)
    if (rank == 0) {
      if (tid < n) a.path[first + tid] = -1;
      if (tid == 0) a.count[i] = 0, a.next[i] = -1;
    }
    vf_cluster_wait();
    return;
  }
  VfWalk w;
  w.cur = 0, w.r = 1, w.count = 1, w.gone = 0, w.known = true, w.last = false, w.c = 0.0, w.S = 1.0;
  if (tid == 0) sh.path[0] = 0;
  // runs of the vocabulary, whole rounds of a warp
  const int per = (V + kVfCtas * kVfWarps * 128 - 1) / (kVfCtas * kVfWarps * 128) * 128;
  const int64_t from64 = (int64_t)(rank * kVfWarps + warp) * per;
  const int from = (int)min(from64, (int64_t)V), to = (int)min(from64 + per, (int64_t)V);
  for (int pass = 0;; ++pass) {
    if (tid == 0) {
      VfCmd cmd;
      bool ask = false;  // a sum is needed before the next comparison
      for (; w.r < n && !ask; ) {
        const int r = w.r;
        if (sh.parent[r] != w.cur || sh.token[r] < 0) {
          ++w.r;
          continue;
        }
        if (!w.known) {
          ask = true;
          break;
        }
        bool ok;
        if (a.q) {
          ok = vf_less(sh.u[r], sh.q[r], w.S, sh.p[r], w.c);
        } else {
          bool was = false;
          for (int k = 0; k < w.gone; ++k) was |= sh.gone_tok[k] == sh.token[r];
          ok = !was && vf_less(sh.u[r], 1.0f, w.S, sh.p[r], 0.0);
        }
        ++w.r;
        if (ok) {
          sh.path[w.count++] = r;
          w.cur = r, w.c = 0.0, w.S = 1.0, w.known = true, w.gone = 0;
        } else {
          w.c += w.S;
          w.known = false;
          if (!a.q) sh.gone_tok[w.gone++] = sh.token[r];
        }
      }
      cmd.what = ask ? VF_SUM : VF_DRAW;
      cmd.cur = w.cur;
      cmd.c_hi = a.q ? (float)w.c : 0.0f;
      cmd.c_lo = a.q ? (float)(w.c - (double)cmd.c_hi) : 0.0f;
      cmd.gone = w.gone;
      sh.count = w.count;
      sh.cmd = cmd;
    }
    __syncthreads();
    const VfCmd cmd = sh.cmd;
    const void* p = row_of(a.p, a.ld_p, cmd.cur);
    const bool minus = a.q && cmd.c_hi > 0.0f;  // nothing refused: the draft's row is not read
    const void* q = minus ? row_of(a.q, a.ld_q, cmd.cur) : nullptr;
    const bool wide = ((reinterpret_cast<uintptr_t>(p) | reinterpret_cast<uintptr_t>(q)) & (4 * ES - 1)) == 0;
    float2 hi2[2], lo2[2];
    hi2[0] = hi2[1] = lo2[0] = lo2[1] = make_float2(0.0f, 0.0f);
    float most = 0.0f;
    constexpr int UN = 4, UM = 2;  // loads together (64 registers: four of each were spilled)
    // Refused tokens of a draft without rows are left out of the sums, as out of the search below:
    // taken from them again they would leave roundings where nothing is left.
    auto refused = [&](int x) {
      for (int k = 0; k < cmd.gone; ++k)
        if (sh.gone_tok[k] == x) return true;
      return false;
    };
    bool some_gone = false;  // in this warp's run
    for (int k = 0; k < cmd.gone; ++k) some_gone |= sh.gone_tok[k] >= from && sh.gone_tok[k] < to;
    const bool once = cmd.c_hi == 1.0f && cmd.c_lo == 0.0f;  // one refusal: c is 1
    if (minus) {
      for (int at = from + 4 * lane; at < to; at += 128 * UM) {
        float4 v[UM], m[UM];
#pragma unroll
        for (int k = 0; k < UM; ++k) {
          v[k] = vf_raw<BF>(p, at + 128 * k, to, wide);
          m[k] = vf_raw<BF>(q, at + 128 * k, to, wide);
        }
        if (once) {
#pragma unroll
          for (int k = 0; k < UM; ++k) {
            vf_add2<true>(hi2[0], lo2[0], make_float2(v[k].x, v[k].y), make_float2(m[k].x, m[k].y), 1.0f, 0.0f, most);
            vf_add2<true>(hi2[1], lo2[1], make_float2(v[k].z, v[k].w), make_float2(m[k].z, m[k].w), 1.0f, 0.0f, most);
          }
        } else {
#pragma unroll
          for (int k = 0; k < UM; ++k) {
            vf_add2<false>(hi2[0], lo2[0], make_float2(v[k].x, v[k].y), make_float2(m[k].x, m[k].y), cmd.c_hi, cmd.c_lo, most);
            vf_add2<false>(hi2[1], lo2[1], make_float2(v[k].z, v[k].w), make_float2(m[k].z, m[k].w), cmd.c_hi, cmd.c_lo, most);
          }
        }
      }
    } else {
      for (int at = from + 4 * lane; at < to; at += 128 * UN) {
        float4 v[UN];
#pragma unroll
        for (int k = 0; k < UN; ++k) v[k] = vf_raw<BF>(p, at + 128 * k, to, wide);
        if (some_gone) {
          for (int g = 0; g < cmd.gone; ++g) {
            const int x = sh.gone_tok[g] - at;
#pragma unroll
            for (int k = 0; k < UN; ++k) {
              if (x == 128 * k) v[k].x = 0.0f;
              if (x == 128 * k + 1) v[k].y = 0.0f;
              if (x == 128 * k + 2) v[k].z = 0.0f;
              if (x == 128 * k + 3) v[k].w = 0.0f;
            }
          }
        }
#pragma unroll
        for (int k = 0; k < UN; ++k) {
          vf_sum2(hi2[0], lo2[0], make_float2(fmaxf(v[k].x, 0.0f), fmaxf(v[k].y, 0.0f)));
          vf_sum2(hi2[1], lo2[1], make_float2(fmaxf(v[k].z, 0.0f), fmaxf(v[k].w, 0.0f)));
        }
      }
    }
    float hi = hi2[0].x, lo = lo2[0].x;
    auto more = [&](float h, float l) {
      two_sum_acc(hi, lo, h);
      lo += l;
    };
    more(hi2[0].y, lo2[0].y);
    more(hi2[1].x, lo2[1].x);
    more(hi2[1].y, lo2[1].y);
    if (__any_sync(0xffffffffu, !(hi < INFINITY) || !(lo < INFINITY) || most == INFINITY)) {
      // an infinity among them, which counts as 0: the run once more, value by value
      hi = lo = 0.0f;
      for (int x = from + lane; x < to; x += 32)
        if (!(some_gone && refused(x))) vf_add(hi, lo, vf_one<BF>(p, x), minus ? vf_one<BF>(q, x) : 0.0f, cmd.c_hi, cmd.c_lo);
    }
    two_sum_warp(hi, lo);
    vf_norm(hi, lo);
    if (lane == 0) sh.hi[warp] = hi, sh.lo[warp] = lo;
    if (pass == 0) vf_cluster_wait();
    __syncthreads();
    if (warp == 0) {
      hi = lane < kVfWarps ? sh.hi[lane] : 0.0f, lo = lane < kVfWarps ? sh.lo[lane] : 0.0f;
      two_sum_warp(hi, lo);
      vf_norm(hi, lo);
      if (lane < kVfCtas) {
        vf_put(&sh.tot_hi[pass & 1][rank], lane, __float_as_uint(hi));
        vf_put(&sh.tot_lo[pass & 1][rank], lane, __float_as_uint(lo));
      }
    }
    vf_cluster_sync();
    if (cmd.what == VF_SUM) {
      if (warp == 0) {  // (64-bit additions are slow: three of them, one after the other)
        const int k = lane % kVfCtas;
        double S = (double)sh.tot_hi[pass & 1][k] + (double)sh.tot_lo[pass & 1][k];
#pragma unroll
        for (int o = 1; o < kVfCtas; o <<= 1) S += __shfl_xor_sync(0xffffffffu, S, o);
        w.S = S;
        w.known = true;
      }
      continue;
    }
    // ---- draw: which CTA, which of its warps' runs.  Lane k holds the k-th CTA's sum, then the k-th run's.
    if (warp == 0) {
      auto scan = [&](float& h, float& l) {  // over 8 lanes, inclusive
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) {
          const float oh = __shfl_up_sync(0xffffffffu, h, o), ol = __shfl_up_sync(0xffffffffu, l, o);
          if (lane >= o) {
            two_sum_acc(h, l, oh);
            l += ol;
          }
        }
      };
      static_assert(kVfCtas == 8 && kVfWarps == 8, "eight lanes");
      // the first whose end lies past `want`, else the last with anything in it; -1: there is nothing
      auto pick = [&](bool some, double end, double want) {
        const uint32_t any = __ballot_sync(0xffffffffu, some && lane < 8), past = __ballot_sync(0xffffffffu, some && lane < 8 && end > want);
        return past ? __ffs((int)past) - 1 : 31 - __clz((int)any);
      };
      float h = lane < 8 ? sh.tot_hi[pass & 1][lane] : 0.0f, l = lane < 8 ? sh.tot_lo[pass & 1][lane] : 0.0f;
      const bool some = h > 0.0f;
      scan(h, l);
      const double end = (double)h + (double)l, total = __shfl_sync(0xffffffffu, end, 7);
      double want = (double)a.u_next[i] * total;
      if (!(want > 0.0)) want = 0.0;
      const int cta = pick(some, end, want);
      int run = cta < 0 ? -2 : -1;
      if (cta == rank) {
        const double before = __shfl_sync(0xffffffffu, end, max(cta - 1, 0));
        if (cta > 0) want -= before;
        h = lane < 8 ? sh.hi[lane] : 0.0f, l = lane < 8 ? sh.lo[lane] : 0.0f;
        const bool part = h > 0.0f;
        scan(h, l);
        const double stop = (double)h + (double)l;
        run = pick(part, stop, want);
        const double skip = __shfl_sync(0xffffffffu, stop, max(run - 1, 0));
        if (run > 0) want -= skip;
      }
      if (lane == 0) sh.run = run, sh.want = want, sh.owner = kVfThreads, sh.last = -1;
    }
    __syncthreads();
    const int run = sh.run;
    if (run == -2 && (cmd.c_hi > 0.0f || cmd.gone > 0)) {
      // nothing is left of the row: from the row itself
      if (tid == 0) w.c = 0.0, w.gone = 0, w.r = n;
      __syncthreads();  // sh.run has been read
      continue;
    }
    if (rank == 0) {
      if (tid < n) a.path[first + tid] = tid < sh.count ? sh.path[tid] : -1;
      if (tid == 0) {
        a.count[i] = sh.count;
        if (run == -2) a.next[i] = -1;  // an empty row
      }
    }
    if (run >= 0) {
      // The run again, by the whole CTA: a thread takes consecutive tokens of it.
      const int64_t r0 = min((int64_t)(rank * kVfWarps + run) * per, (int64_t)V);
      const int r1 = (int)min(r0 + per, (int64_t)V), each = (per / kVfThreads + 3) / 4 * 4 + (per % kVfThreads ? 4 : 0);
      const int x0 = (int)min(r0 + (int64_t)tid * each, (int64_t)r1), x1 = (int)min((int64_t)x0 + each, (int64_t)r1);
      auto value = [&](int x, float vp, float vq, float& h, float& l) {
        return !refused(x) && vf_add(h, l, vp, vq, cmd.c_hi, cmd.c_lo);
      };
      float vh = 0.0f, vl = 0.0f;
      bool some = false;
#pragma unroll 2
      for (int x = x0; x < x1; x += 4) {
        const float4 v = vf_four<BF>(p, x, x1, wide), m = minus ? vf_four<BF>(q, x, x1, wide) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        some |= value(x, v.x, m.x, vh, vl);
        some |= value(x + 1, v.y, m.y, vh, vl);
        some |= value(x + 2, v.z, m.z, vh, vl);
        some |= value(x + 3, v.w, m.w, vh, vl);
      }
      float h = vh, l = vl;  // inclusive sums over the threads
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const float oh = __shfl_up_sync(0xffffffffu, h, o), ol = __shfl_up_sync(0xffffffffu, l, o);
        if (lane >= o) {
          two_sum_acc(h, l, oh);
          l += ol;
        }
      }
      if (lane == 31) sh.scan_hi[warp] = h, sh.scan_lo[warp] = l;
      __syncthreads();
      float bh = 0.0f, bl = 0.0f;  // the warps before
      for (int k = 0; k < warp; ++k) {
        two_sum_acc(bh, bl, sh.scan_hi[k]);
        bl += sh.scan_lo[k];
      }
      two_sum_acc(h, l, bh);
      l += bl;
      const double want = sh.want;
      if (some && (double)h + (double)l > want) atomicMin(&sh.owner, tid);
      if (some) atomicMax(&sh.last, tid);
      // what lies before this thread
      const float ph = __shfl_up_sync(0xffffffffu, h, 1), pl = __shfl_up_sync(0xffffffffu, l, 1);
      __syncthreads();
      if (tid == (sh.owner < kVfThreads ? sh.owner : sh.last)) {
        h = lane ? ph : bh, l = lane ? pl : bl;
        int found = -1;
        for (int x = x0; x < x1; ++x) {
          float eh = 0.0f, el = 0.0f;
          if (!value(x, vf_one<BF>(p, x), minus ? vf_one<BF>(q, x) : 0.0f, eh, el)) continue;
          found = x;
          two_sum_acc(h, l, eh);
          l += el;
          if ((double)h + (double)l > want) break;
        }
        a.next[i] = found;
      }
    }
    break;
  }
}

cudaError_t launch_verify_tree(const VerifyArgs& a, cudaStream_t s) {
  const dim3 grid(kVfCtas, a.t.nseq), block(kVfThreads);
  trace_pre(K_VERIFY_TREE, s);
  const cudaError_t e = a.bf16 ? launch_k(verify_tree_kernel<true>, grid, block, 0, s, true, a)
                               : launch_k(verify_tree_kernel<false>, grid, block, 0, s, true, a);
  trace_post(K_VERIFY_TREE, s);
  return e;
}

}  // namespace m2
