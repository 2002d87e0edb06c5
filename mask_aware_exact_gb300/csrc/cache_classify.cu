// The pages of each sequence that a column-wise mask leaves visible to a row tile:
// the counterpart of the tile classification for the paged cache. Writes, for every
// row tile, the list of the pages that some row sees, in order, each with a bit that
// says whether intervals hide some of its keys from some row, and their number.
//
// Latency-bound: 8 or 16 bytes of bounds per cached token. A table of up to 32, 64 or
// 128 pages is one pass of a CTA of 256, 512 or 1024 threads (with 1024 threads and a
// cluster of one for all of them, masked calls on up to 64 pages took 1.2 to 1.6 us more,
// of 11 to 16), of more if several mask heads share a class: its warps take the heads side
// by side (16 heads, 10 sequences of up to 2500 tokens: 17 us one head after the other, 12
// so); longer tables are shared by a cluster of up to eight CTAs, whose counts,
// which place a CTA's part of the list, come from the others' shared memory. 8 sequences
// of 131072 tokens: 8.7 us with cold caches.
#include "cache_common.cuh"
#include "flashmask.h"

namespace fm {
namespace {

constexpr int kThreadsMost = 1024;
constexpr int kClusterMost = 8;
constexpr int kWordsMost = FM_MAX_SEQLEN / kPage / 32 / kClusterMost;  // 32-page words of a CTA
// 32-page words that CTAs of kThreads take in one pass
constexpr int words_pass(int threads) { return threads * 8 / (32 * kPage); }

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The int at the same shared-memory address in CTA `rank` of the cluster.
__device__ __forceinline__ int of_cta(const int* at, int rank) {
  uint32_t remote;
  int v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(smem_u32(at)), "r"(rank));
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(remote) : "memory");
  return v;
}

__device__ __forceinline__ void load8(const int32_t* src, int (&v)[8]) {
  const int4 a = reinterpret_cast<const int4*>(src)[0], b = reinterpret_cast<const int4*>(src)[1];
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}

// A key is hidden from the whole tile, positions [lo, hi], if the union of its
// intervals (and of the rows above it, when causal) covers them. A thread takes 8 keys
// at a time, so a page is 8 lanes and a warp takes groups of 4 pages.
// kOne: no cluster; kMany: a class has several mask heads.
template <int kThreads, bool kOne, bool kMany>
__global__ void __launch_bounds__(kThreads) cache_classify(const CacheFwdParams p, const Geometry geo,
                                                            const int cluster) {
  __shared__ uint32_t bits[kWordsMost * 8];  // of groups of 4 pages: visible, and << 4 cut
  __shared__ int before[kWordsMost];  // visible pages of this CTA before a word
  __shared__ int count;               // visible pages of this CTA
  allow_next();
  const int tile = kOne ? blockIdx.x : blockIdx.x / cluster, rank = kOne ? 0 : blockIdx.x - tile * cluster, b = blockIdx.y;
  const int cls = geo.by_RT.div(tile), rt = tile - cls * geo.RT;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int each = (geo.words + cluster - 1) / cluster;
  const int w0 = rank * each, words = max(0, min(each, geo.words - w0));  // words [w0, w0 + words)
  const RowTile r = row_tile(p, geo, b, rt, blockIdx.x == 0 && tid == 0);
  const int lo = r.shift + r.t_lo, hi = r.shift + r.t_hi;
  int m0 = cls, m1 = cls;  // mask heads of the class
  if constexpr (kMany) {
    const int per = p.H / p.mask.Hm;
    m0 = cls * geo.G / per;
    m1 = (cls * geo.G + geo.G - 1) / per;
  }
  const int L = p.max_pages * kPage;
  const int end = hi < lo ? 0 : p.mask.causal ? min(r.len, hi + 1) : r.len;
  // A warp takes a group of pages, and with several mask heads one of them: wm, wm +
  // heads, .., where the other warps of the group have the others.
  constexpr int kWarps = kThreads / 32;
  const int heads = kMany ? min(m1 - m0 + 1, kWarps) : 1, wi = kMany ? warp / heads : warp, wm = warp - wi * heads;
  const int step = kMany ? kWarps / heads : kWarps;
  if constexpr (kMany) {
    for (int i = tid; i < 8 * words; i += kThreads) bits[i] = 0;
    __syncthreads();
  }
#pragma unroll 2
  for (int i = wi < step ? wi : 8 * words; i < 8 * words; i += step) {
    const int j0 = ((8 * w0 + i) * 32 + lane) * 8;  // this thread's keys j0 .. j0 + 7
    bool see = false, cut = false;
    // (the first pass's bounds are on their way before the length is there)
    if (i == wi ? j0 < L : j0 < end) {
#pragma unroll 1
      for (int m = m0 + wm; m <= (kMany ? m1 : m0); m += heads) {
        const size_t at = (static_cast<size_t>(b) * p.mask.Hm + m) * L + j0;
        int s0[8] = {}, e0[8] = {};
        if (p.mask.lts) {
          load8(p.mask.lts + at, s0);
          load8(p.mask.lte + at, e0);
        }
        if (!p.mask.uts) {
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const bool there = j0 + k < end;
            const int from = p.mask.causal ? max(lo, j0 + k) : lo;  // the rows above are hidden anyway
            cut |= there && max(s0[k], lo) < min(e0[k], hi + 1);
            see |= there && !(s0[k] <= from && hi < e0[k]);
          }
        } else {
          int s1[8], e1[8];
          load8(p.mask.uts + at, s1);
          load8(p.mask.ute + at, e1);
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const bool there = j0 + k < end;
            cut |= there && (max(s0[k], lo) < min(e0[k], hi + 1) || max(s1[k], lo) < min(e1[k], hi + 1));
            int reach = p.mask.causal ? max(lo, j0 + k) : lo;  // first position not known to be hidden
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              if (s0[k] <= reach && reach < e0[k]) reach = e0[k];
              if (s1[k] <= reach && reach < e1[k]) reach = e1[k];
            }
            see |= there && reach <= hi;
          }
        }
      }
    }
    const uint32_t sb = __ballot_sync(0xffffffffu, see), cb = __ballot_sync(0xffffffffu, cut);
    if (lane == 0) {
      uint32_t v = 0, c = 0;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        v |= static_cast<uint32_t>((sb >> (8 * k) & 0xffu) != 0) << k;
        c |= static_cast<uint32_t>((cb >> (8 * k) & 0xffu) != 0) << k;
      }
      if (kMany)
        atomicOr(&bits[i], v | c << 4);
      else
        bits[i] = v | c << 4;
    }
  }
  __syncthreads();
  auto word_of = [&](int i) {
    uint32_t v = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) v |= (bits[8 * i + k] & 15u) << (4 * k);
    return v;
  };
  if (warp == 0) {
    int sum = 0;
    for (int i0 = 0; i0 < words; i0 += 32) {
      const int n = i0 + lane < words ? __popc(word_of(i0 + lane)) : 0;
      int c = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, c, o);
        if (lane >= o) c += x;
      }
      if (i0 + lane < words) before[i0 + lane] = sum + c - n;
      sum += __shfl_sync(0xffffffffu, c, 31);
    }
    if (lane == 0) count = sum;
  }
  if (kOne)
    __syncthreads();
  else
    cluster_sync();
  // this CTA's place in the list, and the whole
  int mine = 0, total = 0;
  if (kOne) {
    total = count;
  } else {
    for (int k = 0; k < cluster; ++k) {
      const int x = of_cta(&count, k);
      if (k < rank) mine += x;
      total += x;
    }
  }
  const size_t at = (static_cast<size_t>(b) * geo.classes + cls) * geo.RT + rt;
  uint16_t* list = p.list + at * p.max_pages + mine;
  for (int q = tid; q < 32 * words; q += kThreads) {
    const int i = q >> 5, bit = q & 31;
    const uint32_t v = word_of(i);
    if (v >> bit & 1u)
      list[before[i] + __popc(v & ((1u << bit) - 1u))] =
          static_cast<uint16_t>((32 * (w0 + i) + bit) | (bits[q >> 2] >> (4 + (q & 3)) & 1u) << 15);
  }
  if (rank == 0 && tid == 0) p.listed[at] = total;
  if (!kOne) cluster_sync();  // no CTA leaves while its count may be read
}

template <bool kMany>
cudaError_t launch_t(const CacheFwdParams& p, const Geometry& geo, cudaStream_t s) {
  const dim3 grid(static_cast<unsigned>(geo.classes * geo.RT), static_cast<unsigned>(p.B));
  if (geo.words <= words_pass(kThreadsMost)) {
    // groups of pages, of each head: half as many warps at least
    const int heads = (p.mask.Hm + geo.classes - 1) / geo.classes, warps = 4 * geo.words * heads;
    if (geo.words <= words_pass(256) && warps <= 8)
      cache_classify<256, true, kMany><<<grid, 256, 0, s>>>(p, geo, 1);
    else if (geo.words <= words_pass(512) && warps <= 32)
      cache_classify<512, true, kMany><<<grid, 512, 0, s>>>(p, geo, 1);
    else
      cache_classify<kThreadsMost, true, kMany><<<grid, kThreadsMost, 0, s>>>(p, geo, 1);
    return cudaGetLastError();
  }
  int cluster = 2;
  while (cluster < kClusterMost && cluster * words_pass(kThreadsMost) < geo.words) cluster *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(cluster) * grid.x, grid.y);
  cfg.blockDim = dim3(kThreadsMost);
  cfg.stream = s;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = static_cast<unsigned>(cluster);
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, cache_classify<kThreadsMost, false, kMany>, p, geo, cluster);
}

}  // namespace

cudaError_t launch_cache_classify(const CacheFwdParams& p, const Geometry& geo, cudaStream_t s) {
  return geo.classes != p.mask.Hm ? launch_t<true>(p, geo, s) : launch_t<false>(p, geo, s);
}

}  // namespace fm
