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

constexpr int kUnseenWords = FM_MAX_SEQLEN / kPage / 32;
// Position from which on the keys of a sequence are new.
__device__ __forceinline__ int first_new(const WeightsParams& wp, int b, const RowTile& r) {
  return wp.start ? min(max(wp.start[b], 0), r.len) : max(r.shift, 0);
}
// With a column-wise mask: pages that no row sees and whose keys are new have had nothing.
// Called by all kThreads threads of every CTA; `bits` is shared.
template <int kThreads, bool kVec>
__device__ __forceinline__ void clear_unseen(const WeightsParams& wp, const Geometry& geo, uint32_t* bits) {
  if constexpr (kVec) {
    const CacheFwdParams& p = wp.f;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, nseg = p.B * p.c.Hk;
    for (int sg = blockIdx.x; sg < nseg; sg += gridDim.x) {
      const int b = geo.by_Hk.div(sg), hk = sg - b * p.c.Hk;
      const RowTile rt = row_tile(p, geo, b, 0, tid == 0);
      const int start = first_new(wp, b, rt);
      const int first = start / kPage, pages = (rt.len + kPage - 1) / kPage - first;
      if (start >= rt.len) continue;
      for (int i = tid; i < (pages + 31) / 32; i += kThreads) bits[i] = 0;
      __syncthreads();
      // the list is in order, so the new pages are among its last
      const size_t at = static_cast<size_t>(b) * geo.classes + mask_class(p, geo, hk);
      const int n = p.listed[at];
      for (int i = tid; i < min(pages, n); i += kThreads) {
        const int q = (p.list[at * p.max_pages + n - 1 - i] & 0x7fff) - first;
        if (q >= 0) atomicOr(&bits[q >> 5], 1u << (q & 31));
      }
      __syncthreads();
      for (int i = warp; i < pages; i += kThreads / 32) {
        if (bits[i >> 5] >> (i & 31) & 1u) continue;
        const int page = p.table[static_cast<size_t>(b) * p.max_pages + first + i];
        if (page < 0 || page >= p.c.pages) {
          record_failure(p.status, kStatusPage, kSiteCachePage);
          continue;
        }
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int j = (first + i) * kPage + lane + 32 * x;
          if (j >= start && j < rt.len)
            wp.weights[(static_cast<size_t>(page) * p.c.Hk + hk) * kPage + lane + 32 * x] = 0.f;
        }
      }
      __syncthreads();
    }
  }
}

}  // namespace fm
