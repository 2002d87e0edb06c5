// The pages of each sequence that a column-wise mask leaves visible to a row tile:
// the counterpart of the tile classification for the paged cache.
//
// Latency-bound: 8 or 16 bytes of bounds per cached token, spread over one CTA for
// every 32 pages.
#include "cache_common.cuh"

namespace fm {
namespace {

// Bits of the pages that some row of a row tile sees (vis), of those where an
// interval hides some key from some row (part), and the running count of the
// former per word (prefix; its last entry is the total). A CTA takes one word, 32
// pages; a key hides the positions [lo, hi] of the tile if the union of its
// intervals covers them. The CTA that finishes a row tile last sums its words.
__global__ void __launch_bounds__(256) cache_classify(const CacheFwdParams p, const Geometry geo) {
  __shared__ uint32_t bits[2];
  __shared__ int last;
  const int tile = blockIdx.x / geo.words, w = blockIdx.x - tile * geo.words, b = blockIdx.y;
  const int cls = tile / geo.RT, rt = tile - cls * geo.RT;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const RowTile r = row_tile(p, geo, b, rt, blockIdx.x == 0 && threadIdx.x == 0);
  const int lo = r.shift + r.t_lo, hi = r.shift + r.t_hi;
  int m0 = cls, m1 = cls;  // mask heads of the class
  if (geo.classes != p.mask.Hm) {
    const int each = p.H / p.mask.Hm;
    m0 = cls * geo.G / each;
    m1 = (cls * geo.G + geo.G - 1) / each;
  }
  if (threadIdx.x < 2) bits[threadIdx.x] = 0;
  __syncthreads();
  const int L = p.max_pages * kPage;
  uint32_t vis = 0, part = 0;
  for (int i = 0; i < 4; ++i) {
    const int page = 32 * w + 4 * warp + i;
    bool see = false, cut = false;
    for (int half = 0; half < 2; ++half) {
      const int j = page * kPage + 32 * half + lane;
      if (j >= r.len || hi < lo || (p.mask.causal && j > hi)) continue;
      for (int m = m0; m <= m1; ++m) {
        const size_t at = (static_cast<size_t>(b) * p.mask.Hm + m) * L + j;
        const int s0 = p.mask.lts ? p.mask.lts[at] : 0, e0 = p.mask.lts ? p.mask.lte[at] : 0;
        const int s1 = p.mask.uts ? p.mask.uts[at] : 0, e1 = p.mask.uts ? p.mask.ute[at] : 0;
        cut |= max(s0, lo) < min(e0, hi + 1) || max(s1, lo) < min(e1, hi + 1);
        int reach = p.mask.causal ? max(lo, j) : lo;  // first position not known to be hidden
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          if (s0 <= reach && reach < e0) reach = e0;
          if (s1 <= reach && reach < e1) reach = e1;
        }
        see |= reach <= hi;
      }
    }
    if (__any_sync(0xffffffffu, see)) vis |= 1u << (4 * warp + i);
    if (__any_sync(0xffffffffu, cut)) part |= 1u << (4 * warp + i);
  }
  if (lane == 0) {
    atomicOr(&bits[0], vis);
    atomicOr(&bits[1], part);
  }
  __syncthreads();
  const size_t at = (static_cast<size_t>(b) * geo.classes + cls) * geo.RT + rt;
  if (threadIdx.x == 0) {
    p.vis[at * geo.words + w] = bits[0];
    p.part[at * geo.words + w] = bits[1];
    __threadfence();
    last = atomicAdd(&p.class_done[at], 1) == geo.words - 1;
  }
  __syncthreads();
  if (!last || warp != 0) return;
  __threadfence();
  int sum = 0;
  int32_t* out = p.prefix + at * (geo.words + 1);
  for (int w0 = 0; w0 < geo.words; w0 += 32) {
    const int n = w0 + lane < geo.words ? __popc(__ldcg(&p.vis[at * geo.words + w0 + lane])) : 0;
    int c = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, c, o);
      if (lane >= o) c += x;
    }
    if (w0 + lane < geo.words) out[w0 + lane] = sum + c - n;
    sum += __shfl_sync(0xffffffffu, c, 31);
  }
  if (lane == 0) {
    out[geo.words] = sum;
    p.class_done[at] = 0;
  }
}

}  // namespace

cudaError_t launch_cache_classify(const CacheFwdParams& p, const Geometry& geo, cudaStream_t s) {
  const dim3 grid(static_cast<unsigned>(geo.words) * static_cast<unsigned>(geo.classes * geo.RT),
                  static_cast<unsigned>(p.B));
  cache_classify<<<grid, 256, 0, s>>>(p, geo);
  return cudaGetLastError();
}

}  // namespace fm
