// m2_attn_tree.cuh -- what the two kernels of tree attention share: lengths, the order of
// units, and where a row's output goes.
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

#include "m2_common.cuh"
#include "m2_kernels.h"
#include "m2_kv4.cuh"
#include "m2_tree.cuh"

namespace m2 {

struct AtrArgs {
  AttnTreeArgs g;
  int32_t G, most_tiles;    // query heads a kv head; tiles of the launch's largest tree
  int32_t nc, by_row;       // CTAs; one CTA a tile: none is cut
  float* part;              // records within a CTA (warp-MMA kernel)
  float* cta_part;          // [nc][2] records: a tile that began earlier, one that goes on
  int32_t* cta_seg;         // [nc][2] their tiles, -1 where there is none
};

__device__ __forceinline__ int atr_nodes(const AttnTreeArgs& g, int b) { return g.t.cu[b + 1] - g.t.cu[b]; }
// Tokens that the tree's last node could see; 0 for a slot that takes no part.
__device__ __forceinline__ int atr_len(const AttnTreeArgs& g, int b) {
  const int n = atr_nodes(g, b), pos = g.pos[b];
  if (n == 0 || pos < 0) {
    if (n && pos >= -(1 << 30)) M2_RECORD_ARG(g_status);
    return 0;
  }
  const int most = g.c.ld_table * kPage;
  if (pos > most - n) M2_RECORD_ARG(g_status);
  return pos > most - n ? most : pos + n;
}
__device__ __forceinline__ int atr_tiles(const AtrArgs& a, int b, int rows) {
  return (atr_nodes(a.g, b) * a.G + rows - 1) / rows;
}

// A position in the order of units.
struct AtrCursor {
  int b, hk, tile, page, pages, tiles, len;
  __device__ __forceinline__ void load(const AtrArgs& a, int rows) {
    len = atr_len(a.g, b);
    pages = (len + kPage - 1) / kPage;
    tiles = atr_tiles(a, b, rows);
  }
  // to the next unit; b == nseq past the last one
  __device__ __forceinline__ void next(const AtrArgs& a, int rows) {
    if (++page < pages) return;
    page = 0;
    if (++tile < tiles) return;
    tile = 0;
    if (++hk < a.g.c.Hkv) return;
    hk = 0;
    do {
      if (++b >= a.g.t.nseq) return;
      load(a, rows);
    } while (pages == 0);
  }
  __device__ __forceinline__ int seg(const AtrArgs& a) const { return (b * a.g.c.Hkv + hk) * a.most_tiles + tile; }
};

// Row `row` of tile `seg`: where its output goes; null if there is no such row.
__device__ __forceinline__ uint16_t* atr_out(const AtrArgs& a, int seg, int row, int rows, int D) {
  const int tile = seg % a.most_tiles, bh = seg / a.most_tiles, b = bh / a.g.c.Hkv, hk = bh - b * a.g.c.Hkv;
  const int x = tile * rows + row, node = x / a.G;
  if (node >= atr_nodes(a.g, b)) return nullptr;
  return a.g.out + (size_t)(a.g.t.cu[b] + node) * a.g.ld_o + (size_t)(hk * a.G + x - node * a.G) * D;
}
// A CTA a tile, none cut, and nothing to combine, where the tiles are short or enough of
// them to fill the SMs.  (The table's width is what the host knows of the lengths.)  us,
// split / whole, 32 heads over 8 of 128 channels, as many pages as the table is wide:
//                    4 nodes (16 rows)       5 nodes (20 rows)
//   1 x 8 pages      14.3 / 12.0             12.0 / 12.3
//   1 x 16           14.3 / 14.9             15.0 / 17.7
//   1 x 32           14.5 / 20.1             15.9 / 28.1
//   8 x 32           18.6 / 20.5             22.5 / 28.9
//   16 x 32                                  34.0 / 29.4
inline bool atr_by_row(int64_t tiles, int ld_table) {
  return tiles <= num_sms() && ld_table <= (2 * tiles > num_sms() ? 32 : 8);
}
__device__ __forceinline__ void atr_store4(uint16_t* d, float4 o, float l) {
  const float inv = l != 0.0f ? 1.0f / l : 0.0f;  // nothing seen: zeros
  *reinterpret_cast<uint2*>(d) = make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
}

}  // namespace m2
