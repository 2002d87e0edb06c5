// Parts shared by the two kernels that sum the attention weight of cached keys.
#pragma once
#include "cache_common.cuh"
#include "flashmask.h"

namespace fm {

// All rows of a cache head as one tile.
inline Geometry weights_geometry(int H, int Hk, int Hm, int N, int max_pages) {
  Geometry g;
  g.G = H / Hk;
  g.rows = g.G * N;  // below 2^31: B * H * N is
  g.RT = 1;
  g.classes = Hk % Hm == 0 ? Hm : Hk;
  g.words = (max_pages + 31) / 32;
  g.by_G.set(g.G);
  g.by_RT.set(1);
  g.by_Hk.set(Hk);
  g.by_class.set(Hk / g.classes);
  g.by_mask.set(H / Hm);
  return g;
}

// Pages on the line of segment seg: those that some row sees, or all of them (where there
// is no row, keys may still be new).
template <bool kVec>
static __device__ __noinline__ int line_pages(const CacheFwdParams& p, const Geometry& geo, int seg) {
  if constexpr (kVec) return pages_of<true>(p, geo, seg);
  return (row_tile(p, geo, geo.by_Hk.div(seg), 0, blockIdx.x == 0).len + kPage - 1) / kPage;
}

// Position from which on the keys of a sequence are new.
__device__ __forceinline__ int first_new(const WeightsParams& wp, int b, const RowTile& r) {
  return wp.start ? min(max(wp.start[b], 0), r.len) : max(r.shift, 0);
}
// With a column-wise mask: pages that no row sees and whose keys are new have had nothing.
// Warp `warp` of `warps` takes its share of the segments.
template <bool kVec>
__device__ __forceinline__ void clear_unseen(const WeightsParams& wp, const Geometry& geo, int warp, int warps) {
  if constexpr (kVec) {
    const CacheFwdParams& p = wp.f;
    const int lane = threadIdx.x & 31, nseg = p.B * p.c.Hk;
    for (int sg = warp; sg < nseg; sg += warps) {
      const int b = geo.by_Hk.div(sg), hk = sg - b * p.c.Hk;
      const RowTile r = row_tile(p, geo, b, 0, lane == 0);
      const int start = first_new(wp, b, r);
      if (start >= r.len) continue;
      const int first = start / kPage, pages = (r.len + kPage - 1) / kPage;
      const size_t at = static_cast<size_t>(b) * geo.classes + mask_class(p, geo, hk);
      const uint16_t* list = p.list + at * p.max_pages;
      int n = p.listed[at];
      // 32 pages at a time from the last: those of them that are listed are the list's last
      for (int hi = pages; hi > first; hi -= 32) {
        const int lo = max(first, hi - 32);
        const int q = lane < n ? (list[n - 1 - lane] & 0x7fff) - lo : -1;
        const uint32_t seen = __reduce_or_sync(0xffffffffu, q >= 0 && q < 32 ? 1u << q : 0u);
        n -= __popc(seen);
        int page = -1;
        if (lo + lane < hi && !(seen >> lane & 1u)) {
          page = p.table[static_cast<size_t>(b) * p.max_pages + lo + lane];
          if (page < 0 || page >= p.c.pages) {
            record_failure(p.status, kStatusPage, kSiteCachePage);
            page = -1;
          }
        }
        for (uint32_t todo = __ballot_sync(0xffffffffu, page >= 0); todo != 0; todo &= todo - 1) {
          const int i = __ffs(todo) - 1, pg = __shfl_sync(0xffffffffu, page, i);
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const int j = (lo + i) * kPage + lane + 32 * x;
            if (j >= start && j < r.len)
              wp.weights[(static_cast<size_t>(pg) * p.c.Hk + hk) * kPage + lane + 32 * x] = 0.f;
          }
        }
      }
    }
  }
}

}  // namespace fm
