// The pages of each sequence that a column-wise mask leaves visible to a row tile:
// the counterpart of the tile classification for the paged cache. Writes, for every
// row tile, the list of the pages that some row sees, in order, each with a bit that
// says whether intervals hide some of its keys from some row, and their number.
//
// Latency-bound: 8 or 16 bytes of bounds per cached token, spread over one CTA for
// every 32 pages, each thread loading the bounds of 8 keys at once. The CTA that
// finishes a row tile last makes the list from the others' page bits.
#include "cache_common.cuh"

namespace fm {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ void load8(const int32_t* src, int (&v)[8]) {
  const int4 a = reinterpret_cast<const int4*>(src)[0], b = reinterpret_cast<const int4*>(src)[1];
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}

// A key is hidden from the whole tile, positions [lo, hi], if the union of its
// intervals (and of the rows above it, when causal) covers them.
__global__ void __launch_bounds__(kThreads) cache_classify(const CacheFwdParams p, const Geometry geo) {
  __shared__ uint32_t bits[2][kThreads / 32];
  __shared__ int sums[kThreads / 32 + 1];
  __shared__ int last;
  const int tile = blockIdx.x / geo.words, w = blockIdx.x - tile * geo.words, b = blockIdx.y;
  const int cls = tile / geo.RT, rt = tile - cls * geo.RT;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const RowTile r = row_tile(p, geo, b, rt, blockIdx.x == 0 && tid == 0);
  const int lo = r.shift + r.t_lo, hi = r.shift + r.t_hi;
  int m0 = cls, m1 = cls;  // mask heads of the class
  if (geo.classes != p.mask.Hm) {
    const int each = p.H / p.mask.Hm;
    m0 = cls * geo.G / each;
    m1 = (cls * geo.G + geo.G - 1) / each;
  }
  const int L = p.max_pages * kPage;
  const int j0 = (w * kThreads + tid) * 8;  // this thread's keys j0 .. j0 + 7
  const int end = hi < lo ? 0 : p.mask.causal ? min(r.len, hi + 1) : r.len;
  bool see = false, cut = false;
  if (j0 < end) {
    for (int m = m0; m <= m1; ++m) {
      const size_t at = (static_cast<size_t>(b) * p.mask.Hm + m) * L + j0;
      int s0[8] = {}, e0[8] = {}, s1[8] = {}, e1[8] = {};
      if (p.mask.lts) {
        load8(p.mask.lts + at, s0);
        load8(p.mask.lte + at, e0);
      }
      if (p.mask.uts) {
        load8(p.mask.uts + at, s1);
        load8(p.mask.ute + at, e1);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int j = j0 + i;
        if (j >= end) continue;
        cut |= max(s0[i], lo) < min(e0[i], hi + 1) || max(s1[i], lo) < min(e1[i], hi + 1);
        int reach = p.mask.causal ? max(lo, j) : lo;  // first position not known to be hidden
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          if (s0[i] <= reach && reach < e0[i]) reach = e0[i];
          if (s1[i] <= reach && reach < e1[i]) reach = e1[i];
        }
        see |= reach <= hi;
      }
    }
  }
  // a page is eight lanes; a warp has four pages
  const uint32_t sees = __ballot_sync(0xffffffffu, see), cuts = __ballot_sync(0xffffffffu, cut);
  if (lane == 0) {
    uint32_t v = 0, c = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v |= static_cast<uint32_t>((sees >> (8 * i) & 0xffu) != 0) << i;
      c |= static_cast<uint32_t>((cuts >> (8 * i) & 0xffu) != 0) << i;
    }
    bits[0][warp] = v << (4 * warp);
    bits[1][warp] = c << (4 * warp);
  }
  __syncthreads();
  const size_t at = (static_cast<size_t>(b) * geo.classes + cls) * geo.RT + rt;
  if (tid == 0) {
    uint32_t v = 0, c = 0;
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) {
      v |= bits[0][i];
      c |= bits[1][i];
    }
    p.vis[at * geo.words + w] = v;
    p.part[at * geo.words + w] = c;
    __threadfence();
    last = atomicAdd(&p.class_done[at], 1) == geo.words - 1;
  }
  __syncthreads();
  if (!last) return;
  __threadfence();
  uint16_t* list = p.list + at * p.max_pages;
  int total = 0;
  for (int w0 = 0; w0 < geo.words; w0 += kThreads) {
    const bool mine = w0 + tid < geo.words;
    uint32_t v = mine ? __ldcg(&p.vis[at * geo.words + w0 + tid]) : 0;
    const uint32_t c = mine ? __ldcg(&p.part[at * geo.words + w0 + tid]) : 0;
    int sum = __popc(v);
    const int n = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += x;
    }
    if (lane == 31) sums[warp] = sum;
    __syncthreads();
    int before = total + sum - n;
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) {
      if (i < warp) before += sums[i];
      total += sums[i];
    }
    while (v) {
      const int bit = __ffs(v) - 1;
      v &= v - 1;
      list[before++] = static_cast<uint16_t>((32 * (w0 + tid) + bit) | (c >> bit & 1u) << 15);
    }
    __syncthreads();
  }
  if (tid == 0) {
    p.listed[at] = total;
    p.class_done[at] = 0;
  }
}

}  // namespace

cudaError_t launch_cache_classify(const CacheFwdParams& p, const Geometry& geo, cudaStream_t s) {
  const dim3 grid(static_cast<unsigned>(geo.words) * static_cast<unsigned>(geo.classes * geo.RT),
                  static_cast<unsigned>(p.B));
  cache_classify<<<grid, kThreads, 0, s>>>(p, geo);
  return cudaGetLastError();
}

}  // namespace fm
