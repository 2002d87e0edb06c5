// Eviction from the 8-bit paged cache: each cache head of a sequence keeps its first
// tokens, its last ones and of the others those of the largest weight, and the kept
// tokens move together, in their order, into fewer pages.
//
// Two kernels. The first finds a segment's (sequence and cache head) kept tokens: the
// weights as ordered 32-bit keys, the m-th largest by three passes over histograms of
// 11, 11 and 10 bits, ties by position, a 64-bit mask for each page and the number kept
// before it. A segment is a CTA's or, if it is long, a cluster's of up to eight, whose
// histograms and counts are added through the others' shared memory. The second writes
// one page of a head at a time: K rows as 16-byte pieces, V columns as bytes (the lanes
// of a warp take the tokens of a row of V, so that the bytes of a source page lie
// together), rounded to the page's new scale.
//
// In place, a page may only be overwritten once the tokens that leave it have been read.
// Kept tokens move towards the front, and the at most 64 of a page go to at most two
// pages, none behind it. Pages are taken in order from a counter, each CTA reads all of
// its page's tokens first and says so; before it writes it waits for the one or two pages
// that read from it, which were taken before and wait for nothing until they have read.
#include <atomic>

#include "cache_common.cuh"
#include "flashmask.h"

namespace fm {
namespace {

// ---------------------------------------------------------------- selection
constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kClusterMost = 8;
constexpr int kBins = 2048;
constexpr int kPagesCached = 256;                                     // of a CTA, with their keys
constexpr int kPagesMost = FM_MAX_SEQLEN / kPage / kClusterMost;      // of a CTA

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ int of_cta(const int* at, int rank) {
  uint32_t remote;
  int v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(smem_u32(at)), "r"(rank));
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(remote) : "memory");
  return v;
}

// Weights in an order of unsigned numbers: NaN below all others, -0 as +0.
__device__ __forceinline__ uint32_t order_key(float w) {
  if (isnan(w)) return 0u;
  const uint32_t u = __float_as_uint(w + 0.f);
  return u >> 31 ? ~u : u | 0x80000000u;
}

// What a sequence has and keeps.
struct Kept {
  int len, n, lo, hi, choose;  // tokens, of them kept; [lo, hi) are chosen from, and how many
};
__device__ __forceinline__ Kept kept_of(const EvictParams& p, int b, bool record) {
  Kept k;
  k.len = p.lens[b];
  const int most = p.max_pages * kPage;
  if (k.len < 0 || k.len > most) {
    if (record) record_failure(p.status, kStatusPage, kSiteEvictLen);
    k.len = min(max(k.len, 0), most);
  }
  k.n = min(k.len, max(p.keep ? p.keep[b] : p.budget, 0));
  const int sink = k.n == k.len ? k.n : min(p.sink, k.n), recent = min(p.recent, k.n - sink);
  k.lo = sink;
  k.hi = k.len - recent;
  k.choose = k.n - sink - recent;
  return k;
}

struct SelectSmem {
  int hist[2][kBins];
  int wsum[kSelWarps + 4];
  int found[2];   // bin, keys wanted of it
  int totals[2];  // keys equal to the last one, tokens kept, of this CTA
};

template <bool kCached>
__global__ void __launch_bounds__(kSelThreads, 1) evict_select_kernel(const EvictParams p, const int cluster) {
  extern __shared__ __align__(16) uint8_t smem[];
  SelectSmem& sh = *reinterpret_cast<SelectSmem*>(smem);
  uint64_t* masks = reinterpret_cast<uint64_t*>(smem + (sizeof(SelectSmem) + 15) / 16 * 16);  // [pages]
  uint64_t* equals = masks + (kCached ? kPagesCached : kPagesMost);
  int* counts = reinterpret_cast<int*>(equals + (kCached ? kPagesCached : kPagesMost));
  uint32_t* keys = reinterpret_cast<uint32_t*>(counts + (kCached ? kPagesCached : kPagesMost));  // kCached
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int seg = blockIdx.x / cluster, rank = blockIdx.x - seg * cluster;
  const int b = seg / p.c.Hk, hk = seg - b * p.c.Hk;
  const Kept kp = kept_of(p, b, tid == 0 && rank == 0 && hk == 0);
  const int pages = (kp.len + kPage - 1) / kPage, each = (pages + cluster - 1) / cluster;
  const int p0 = min(rank * each, pages), np = min(each, pages - p0);
  auto sync_all = [&]() {
    if (cluster == 1)
      __syncthreads();
    else
      cluster_sync();
  };
  if (tid == 0 && rank == 0 && hk == 0) {
    p.info[2 * b] = kp.len;
    p.info[2 * b + 1] = kp.n;
    if (b == 0) *p.ticket = 0;
  }

  // keys of page p0 + i: this lane's tokens lane and lane + 32
  auto load_keys = [&](int i, uint32_t (&k)[2]) {
    const int page = p.table[static_cast<size_t>(b) * p.max_pages + p0 + i];
    k[0] = k[1] = 0u;
    if (page < 0 || page >= p.c.pages) {
      if (lane == 0) record_failure(p.status, kStatusPage, kSiteEvictPage);
    } else {
      const float* at = p.weights + (static_cast<size_t>(page) * p.c.Hk + hk) * kPage + lane;
      k[0] = order_key(at[0]);
      k[1] = order_key(at[32]);
    }
  };
  auto keys_of = [&](int i, uint32_t (&k)[2]) {
    if constexpr (kCached) {
      k[0] = keys[i * kPage + lane];
      k[1] = keys[i * kPage + lane + 32];
    } else {
      load_keys(i, k);
    }
  };
  for (int i = tid; i < 2 * kBins; i += kSelThreads) sh.hist[0][i] = 0;
  if constexpr (kCached) {
#pragma unroll 4
    for (int i = warp; i < np; i += kSelWarps) {
      uint32_t k[2];
      load_keys(i, k);
      keys[i * kPage + lane] = k[0];
      keys[i * kPage + lane + 32] = k[1];
    }
  }
  __syncthreads();

  // the last key that is kept, and how many of those equal to it
  uint32_t last = 0xffffffffu;
  int equal = 0;
  if (kp.choose > 0) {
    uint32_t prefix = 0, known = 0;
    int want = kp.choose;
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bins = pass == 2 ? 1024 : kBins;
      int* hist = sh.hist[pass & 1];
      if (pass == 2) {
        for (int i = tid; i < kBins; i += kSelThreads) hist[i] = 0;
        __syncthreads();
      }
      for (int i = warp; i < np; i += kSelWarps) {
        uint32_t k[2];
        keys_of(i, k);
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int j = (p0 + i) * kPage + lane + 32 * x;
          if (j >= kp.lo && j < kp.hi && (k[x] & known) == prefix) atomicAdd(&hist[k[x] >> shift & (bins - 1)], 1);
        }
      }
      sync_all();
      // this thread's two bins, from the top
      int c[2] = {0, 0};
      const int top = bins - 1 - 2 * tid;
      if (top >= 1) {
        for (int r = 0; r < cluster; ++r) {
          c[0] += cluster == 1 ? hist[top] : of_cta(&hist[top], r);
          c[1] += cluster == 1 ? hist[top - 1] : of_cta(&hist[top - 1], r);
        }
      }
      int all;
      const int above = block_before<kSelWarps>(c[0] + c[1], sh.wsum, all);
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int a = above + (x ? c[0] : 0);
        if (a < want && want <= a + c[x]) {
          sh.found[0] = top - x;
          sh.found[1] = want - a;
        }
      }
      __syncthreads();
      prefix |= static_cast<uint32_t>(sh.found[0]) << shift;
      known |= static_cast<uint32_t>(bins - 1) << shift;
      want = sh.found[1];
      __syncthreads();
    }
    last = prefix;
    equal = want;
  }

  // masks of the pages: what is kept anyway, and what is equal to the last key
  for (int i = warp; i < np; i += kSelWarps) {
    uint32_t k[2], keep[2], same[2];
    keys_of(i, k);
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int j = (p0 + i) * kPage + lane + 32 * x;
      const bool choice = j >= kp.lo && j < kp.hi;
      keep[x] = __ballot_sync(0xffffffffu, choice ? k[x] > last : j < kp.len);
      same[x] = __ballot_sync(0xffffffffu, choice && k[x] == last && equal > 0);
    }
    if (lane == 0) {
      masks[i] = static_cast<uint64_t>(keep[1]) << 32 | keep[0];
      equals[i] = static_cast<uint64_t>(same[1]) << 32 | same[0];
    }
  }
  __syncthreads();
  // a thread's pages in a row: sums before them, of this CTA and of those before it
  const int per = (np + kSelThreads - 1) / kSelThreads, i0 = min(tid * per, np), i1 = min(i0 + per, np);
  auto sums_before = [&](int mine, int which) {
    int all;
    int x = block_before<kSelWarps>(mine, sh.wsum, all);
    if (cluster > 1) {
      if (tid == 0) sh.totals[which] = all;
      cluster_sync();
      for (int r = 0; r < rank; ++r) x += of_cta(&sh.totals[which], r);
    }
    return x;
  };
  int mine = 0;
  for (int i = i0; i < i1; ++i) mine += __popcll(equals[i]);
  int left = equal - sums_before(mine, 0);
  mine = 0;
  for (int i = i0; i < i1; ++i) {
    uint64_t e = equals[i];
    const int n = __popcll(e);
    // the lowest positions first
    for (int drop = n - min(max(left, 0), n); drop > 0; --drop) e &= ~(1ull << (63 - __clzll(static_cast<long long>(e))));
    left -= n;
    masks[i] |= e;
    mine += __popcll(masks[i]);
  }
  int at = sums_before(mine, 1);
  const size_t row = static_cast<size_t>(seg) * p.max_pages;
  int32_t* before = p.before + static_cast<size_t>(seg) * (p.max_pages + 1);
  for (int i = i0; i < i1; ++i) {
    const int n = __popcll(masks[i]), to = (at + kPage - 1) / kPage;
    p.mask[row + p0 + i] = masks[i];
    before[p0 + i] = at;
    p.was_read[row + p0 + i] = 0;
    if (n > 0 && to * kPage < at + n) p.first[row + to] = p0 + i;
    counts[i] = at;
    at += n;
  }
  if (tid == 0 && rank == 0) before[pages] = kp.n;
  if (p.index != nullptr) {
    __syncthreads();
    int32_t* index = p.index + static_cast<size_t>(seg) * p.index_width;
    for (int i = warp; i < np; i += kSelWarps) {
      const uint64_t m = masks[i];
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int bit = lane + 32 * x, r = counts[i] + __popcll(m & ((1ull << bit) - 1ull));
        if ((m >> bit & 1ull) && r < p.index_width) index[r] = (p0 + i) * kPage + bit;
      }
    }
  }
  if (cluster > 1) cluster_sync();  // no CTA leaves while its counts may be read
}

// ---------------------------------------------------------------- pages
constexpr int kMoveThreads = 256;
constexpr int kMoveWarps = kMoveThreads / 32;
constexpr int kWindow = kMoveThreads;  // source pages looked at a time
constexpr int kMinExp = -100;

__device__ __forceinline__ uint32_t codes_times(uint32_t w, float f) {
  uint32_t lo, hi;
  codes_to_f16(w, lo, hi);
  float v[4];
  asm("{.reg .f16 a, b; mov.b32 {a, b}, %2; cvt.f32.f16 %0, a; cvt.f32.f16 %1, b;}" : "=f"(v[0]), "=f"(v[1]) : "r"(lo));
  asm("{.reg .f16 a, b; mov.b32 {a, b}, %2; cvt.f32.f16 %0, a; cvt.f32.f16 %1, b;}" : "=f"(v[2]), "=f"(v[3]) : "r"(hi));
  return pack_e4m3x4(v[0] * f, v[1] * f, v[2] * f, v[3] * f);
}
// Magnitudes of four codes; 0 for a NaN.
__device__ __forceinline__ uint32_t magnitudes(uint32_t w) {
  const uint32_t m = w & 0x7f7f7f7fu;
  return m & ~__vcmpeq4(m, 0x7f7f7f7fu);
}
__device__ __forceinline__ float code_value(uint32_t code) {
  uint32_t lo, hi;
  codes_to_f16(code & 0xffu, lo, hi);
  float v;
  asm("{.reg .f16 a, b; mov.b32 {a, b}, %1; cvt.f32.f16 %0, a;}" : "=f"(v) : "r"(lo));
  return v;
}
// Exponent k of the smallest power of two with 2^9 x <= 448 * 2^k (448 = 1.75 * 2^8), at
// most 127.
__device__ __forceinline__ int scale_exponent9(float x) {
  if (!(x > 0.f)) return kMinExp;
  const uint32_t u = __float_as_uint(x);
  const int e = static_cast<int>(u >> 23) - 127;
  return min(max(((u & 0x7fffffu) <= 0x600000u ? e - 8 : e - 7) + 9, kMinExp), 127);
}

struct MoveSmem {
  int base[kMoveThreads + 1];  // pages to be written before a thread's sequences
  int wsum[kMoveWarps + 4];
  int before[kWindow + 1];
  uint64_t mask[kWindow];
  int token[kPage];            // where each slot's token is now
  int page[kPage];             // its page, -1: none
  float kscale[kPage], vscale[kPage];
  uint32_t vmax[4][kPage];
  float top[2][kPage];         // of each slot, K and V, times 2^-9
  float weight[kPage];
  int exps[2];
  int job;
};

template <int D, bool kInPlace>
__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const EvictParams p) {
  __shared__ MoveSmem sh;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int Hk = p.c.Hk;
  const int32_t* out_table = kInPlace ? p.table : p.out_table;
  const int out_pages = kInPlace ? p.max_pages : p.out_pages;

  // the line of pages to be written: a sequence's pages in order, its heads side by side
  const int per = (p.B + kMoveThreads - 1) / kMoveThreads;
  const int b0 = min(tid * per, p.B), b1 = min(b0 + per, p.B);
  auto pages_of_seq = [&](int b) { return (p.info[2 * b + 1] + kPage - 1) / kPage; };
  int mine = 0;
  for (int b = b0; b < b1; ++b) {
    mine += pages_of_seq(b);
    if (blockIdx.x == 0) {
      p.new_lens[b] = p.info[2 * b + 1];
      if (!kInPlace && pages_of_seq(b) > out_pages) record_failure(p.status, kStatusPage, kSiteEvictRange);
    }
  }
  int total;
  sh.base[tid] = block_before<kMoveWarps>(mine, sh.wsum, total);
  if (tid == 0) sh.base[kMoveThreads] = total;
  const long long jobs = static_cast<long long>(total) * Hk;

  for (long long job = blockIdx.x;; job += gridDim.x) {
    __syncthreads();  // the shared words of the page before have been read
    if constexpr (kInPlace) {
      if (tid == 0) sh.job = atomicAdd(p.ticket, 1);
      __syncthreads();
      job = static_cast<uint32_t>(sh.job);
    }
    if (job >= jobs) break;
    // which page: sequence, page of it, head
    const int unit = static_cast<int>(job / Hk), hk = static_cast<int>(job - static_cast<long long>(unit) * Hk);
    int lo = 0, hi = kMoveThreads;  // base[lo] <= unit < base[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (sh.base[mid] <= unit) lo = mid; else hi = mid;
    }
    int b = lo * per, dp = unit - sh.base[lo];
    for (int n; dp >= (n = pages_of_seq(b)); ++b) dp -= n;
    const int seg = b * Hk + hk, len = p.info[2 * b], kept = p.info[2 * b + 1];
    const int pages = (len + kPage - 1) / kPage, r0 = dp * kPage, cnt = min(kPage, kept - r0);
    const size_t row = static_cast<size_t>(seg) * p.max_pages;
    const int32_t* before = p.before + static_cast<size_t>(seg) * (p.max_pages + 1);
    const int32_t* table = p.table + static_cast<size_t>(b) * p.max_pages;

    // where the slots' tokens are
    for (int s = p.first[row + dp];; s += kWindow) {
      const int n = min(kWindow, pages - s);
      if (tid < n) {
        sh.before[tid] = before[s + tid];
        sh.mask[tid] = p.mask[row + s + tid];
      }
      if (tid == 0) sh.before[n] = before[s + n];
      __syncthreads();
      const int have = sh.before[n];
      if (tid < cnt) {
        const int r = r0 + tid;
        if (r >= sh.before[0] && r < have) {
          int l = 0, h = n;  // before[l] <= r < before[h]
          while (h - l > 1) {
            const int mid = (l + h) >> 1;
            if (sh.before[mid] <= r) l = mid; else h = mid;
          }
          // the k-th token kept of that page
          int k = r - sh.before[l], bit = 0;
          uint64_t m = sh.mask[l];
#pragma unroll
          for (int w = 32; w > 0; w >>= 1) {
            const int c = __popcll(m & ((1ull << w) - 1ull));
            if (k >= c) k -= c, bit += w, m >>= w;
          }
          sh.token[tid] = (s + l) * kPage + bit;
        }
      }
      __syncthreads();
      if (have >= r0 + cnt || s + n >= pages) break;
    }
    bool moved = false;
    if (tid < kPage) {
      int page = -1;
      float ks = 0.f, vs = 0.f;
      if (tid < cnt) {
        moved = !kInPlace || sh.token[tid] != r0 + tid;
        page = table[sh.token[tid] / kPage];
        if (page < 0 || page >= p.c.pages) {
          record_failure(p.status, kStatusPage, kSiteEvictPage);
          page = -1;
        } else {
          const size_t ph = static_cast<size_t>(page) * Hk + hk;
          ks = p.c.kscale[ph];
          vs = p.c.vscale[ph];
        }
      }
      sh.page[tid] = page;
      sh.kscale[tid] = ks;
      sh.vscale[tid] = vs;
    }
    if (!__syncthreads_or(moved)) continue;  // every token stays where it is

    // K: a thread has a quarter of a slot's row; V: a slot's rows q, q + 4, ..
    uint4 kr[D / 64];
    const int ks_slot = tid >> 2, kq = tid & 3;
    const int vslot = lane + 32 * (warp & 1), vq = warp >> 1;
    {
      const int page = sh.page[ks_slot];
      const uint8_t* src = p.c.k8 + (static_cast<size_t>(max(page, 0)) * Hk + hk) * (kPage * D) +
                           (page < 0 ? 0 : sh.token[ks_slot] % kPage) * D + 16 * kq;
#pragma unroll
      for (int i = 0; i < D / 64; ++i)
        kr[i] = page < 0 ? make_uint4(0u, 0u, 0u, 0u) : *reinterpret_cast<const uint4*>(src + 64 * i);
    }
    uint32_t vr[D / 16];
    {
      const int page = sh.page[vslot];
      const uint8_t* src = p.c.v8 + (static_cast<size_t>(max(page, 0)) * Hk + hk) * (kPage * D) +
                           (page < 0 ? 0 : sh.token[vslot] % kPage) + vq * kPage;
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        vr[i] = 0u;
        if (page >= 0) {
#pragma unroll
          for (int j = 0; j < 4; ++j) vr[i] |= static_cast<uint32_t>(src[(16 * i + 4 * j) * kPage]) << (8 * j);
        }
      }
    }
    if (tid < kPage)
      sh.weight[tid] = tid < cnt && sh.page[tid] >= 0
                           ? p.weights[(static_cast<size_t>(sh.page[tid]) * Hk + hk) * kPage + sh.token[tid] % kPage]
                           : 0.f;

    // largest magnitudes
    uint32_t km = 0, vm = 0;
#pragma unroll
    for (int i = 0; i < D / 64; ++i)
      km = __vmaxu4(km, __vmaxu4(__vmaxu4(magnitudes(kr[i].x), magnitudes(kr[i].y)),
                                 __vmaxu4(magnitudes(kr[i].z), magnitudes(kr[i].w))));
    km = __vmaxu4(km, __shfl_xor_sync(0xffffffffu, km, 1));
    km = __vmaxu4(km, __shfl_xor_sync(0xffffffffu, km, 2));
#pragma unroll
    for (int i = 0; i < D / 16; ++i) vm = __vmaxu4(vm, magnitudes(vr[i]));
    auto widest = [](uint32_t m) { return max(max(m & 0xffu, m >> 8 & 0xffu), max(m >> 16 & 0xffu, m >> 24)); };
    const bool kbad = no_scales(sh.kscale[ks_slot], sh.vscale[ks_slot]), vbad = no_scales(sh.kscale[vslot], sh.vscale[vslot]);
    if (kq == 0) sh.top[0][ks_slot] = kbad ? 0.f : code_value(widest(km)) * (sh.kscale[ks_slot] * 0x1p-9f);
    sh.vmax[vq][vslot] = widest(vm);
    __syncthreads();  // all of the page's tokens have been read
    if (kInPlace && tid == 0) {
      asm volatile("fence.acq_rel.gpu;\n\tst.relaxed.gpu.global.s32 [%0], %1;" ::"l"(p.was_read + row + dp), "r"(1)
                   : "memory");
    }
    if (warp < 2) {
      float top = 0.f;
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int s = lane + 32 * x;
        if (warp == 0) {
          top = fmaxf(top, sh.top[0][s]);
        } else if (!no_scales(sh.kscale[s], sh.vscale[s])) {
          const uint32_t m = max(max(sh.vmax[0][s], sh.vmax[1][s]), max(sh.vmax[2][s], sh.vmax[3][s]));
          top = fmaxf(top, code_value(m) * (sh.vscale[s] * 0x1p-9f));
        }
      }
      // (not negative: ordered like their bits)
      const uint32_t bits = __reduce_max_sync(0xffffffffu, __float_as_uint(top));
      if (lane == 0) sh.exps[warp] = scale_exponent9(__uint_as_float(bits));
    }
    bool ok = true;
    if constexpr (kInPlace) {
      // tokens of the page to be overwritten go to at most two pages
      if (tid >= 64 && tid < 66) {
        const int a = before[min(dp, pages)], z = before[min(dp + 1, pages)];
        const int reader = tid == 64 ? a / kPage : (z - 1) / kPage;
        if (z > a && reader != dp) {
          const int32_t* flag = p.was_read + row + reader;
          const uint64_t t0 = global_timer_ns();
          while (true) {
            int v;
            asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(flag) : "memory");
            if (v != 0) break;
            if ((*reinterpret_cast<volatile int32_t*>(p.status) & kStatusTimeout) != 0 ||
                global_timer_ns() - t0 > FM_WAIT_LIMIT_NS) {
              record_failure(p.status, kStatusTimeout, kSiteEvictWait);
              ok = false;
              break;
            }
          }
        }
      }
    }
    ok = __syncthreads_and(ok);
    if (!ok) return;
    if (dp >= out_pages) continue;
    const int to = out_table[static_cast<size_t>(b) * out_pages + dp];
    if (to < 0 || to >= p.c.pages) {
      if (tid == 0) record_failure(p.status, kStatusPage, kSiteEvictPage);
      continue;
    }
    const size_t ph = static_cast<size_t>(to) * Hk + hk;
    const float k_new = __int_as_float((sh.exps[0] + 127) << 23), v_new = __int_as_float((sh.exps[1] + 127) << 23);
    {
      const float f = sh.kscale[ks_slot] / k_new;
      uint8_t* dst = p.c.k8 + ph * (kPage * D) + ks_slot * D + 16 * kq;
#pragma unroll
      for (int i = 0; i < D / 64; ++i) {
        const uint32_t nan = 0x7f7f7f7fu;
        uint4 o = kr[i];
        if (kbad)
          o = make_uint4(nan, nan, nan, nan);
        else if (f != 1.f)
          o = make_uint4(codes_times(o.x, f), codes_times(o.y, f), codes_times(o.z, f), codes_times(o.w, f));
        *reinterpret_cast<uint4*>(dst + 64 * i) = o;
      }
    }
    {
      const float f = sh.vscale[vslot] / v_new;
      uint8_t* dst = p.c.v8 + ph * (kPage * D) + vslot + vq * kPage;
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        uint32_t o = vbad ? 0u : f != 1.f ? codes_times(vr[i], f) : vr[i];
        o &= ~__vcmpeq4(o & 0x7f7f7f7fu, 0x7f7f7f7fu);  // V holds no NaN
#pragma unroll
        for (int j = 0; j < 4; ++j) dst[(16 * i + 4 * j) * kPage] = static_cast<uint8_t>(o >> (8 * j));
      }
    }
    if (tid < kPage) p.weights[ph * kPage + tid] = sh.weight[tid];
    if (tid == 0) {
      p.c.kscale[ph] = k_new;
      p.c.vscale[ph] = v_new;
    }
  }
}

template <typename F>
cudaError_t allow_smem(F* kernel, int bytes, std::atomic<uint64_t>* done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev > 255) return cudaErrorInvalidDevice;
  if (done[dev >> 6].load(std::memory_order_relaxed) >> (dev & 63) & 1) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done[dev >> 6].fetch_or(1ull << (dev & 63), std::memory_order_relaxed);
  return e;
}

template <bool kCached>
cudaError_t launch_select(const EvictParams& p, int cluster, cudaStream_t s) {
  constexpr int kPages = kCached ? kPagesCached : kPagesMost;
  constexpr int kBytes = (sizeof(SelectSmem) + 15) / 16 * 16 + kPages * (8 + 8 + 4) + (kCached ? kPages * kPage * 4 : 0);
  static_assert(kBytes <= 227 * 1024, "shared memory per CTA");
  static std::atomic<uint64_t> done[4];
  const cudaError_t e = allow_smem(evict_select_kernel<kCached>, kBytes, done);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.B) * p.c.Hk * cluster);
  cfg.blockDim = dim3(kSelThreads);
  cfg.dynamicSmemBytes = kBytes;
  cfg.stream = s;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = static_cast<unsigned>(cluster);
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, evict_select_kernel<kCached>, p, cluster);
}

template <int D>
cudaError_t launch_move(const EvictParams& p, int num_sms, cudaStream_t s) {
  const long long most = static_cast<long long>(p.B) * p.c.Hk * (p.out_table ? p.out_pages : p.max_pages);
  const unsigned grid = static_cast<unsigned>(most < 4LL * num_sms ? most : 4LL * num_sms);
  if (p.out_table == nullptr)
    evict_move_kernel<D, true><<<grid, kMoveThreads, 0, s>>>(p);
  else
    evict_move_kernel<D, false><<<grid, kMoveThreads, 0, s>>>(p);
  return cudaGetLastError();
}

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

}  // namespace

EvictWs evict_ws_layout(int B, int Hk, int max_pages) {
  const size_t segs = static_cast<size_t>(B) * Hk;
  EvictWs w;
  size_t off = 256;  // the status word
  w.ticket = off;
  off = up256(off + 4);
  w.info = off;
  off = up256(off + static_cast<size_t>(B) * 8);
  w.mask = off;
  off = up256(off + segs * max_pages * 8);
  w.before = off;
  off = up256(off + segs * (max_pages + 1) * 4);
  w.first = off;
  off = up256(off + segs * max_pages * 4);
  w.was_read = off;
  off = up256(off + segs * max_pages * 4);
  w.total = off;
  return w;
}

cudaError_t launch_cache_evict(int d, const EvictParams& p, int num_sms, cudaStream_t s) {
  int cluster = 1;
  while (cluster < kClusterMost && cluster * kPagesCached < p.max_pages) cluster *= 2;
  const cudaError_t e = cluster * kPagesCached >= p.max_pages ? launch_select<true>(p, cluster, s)
                                                              : launch_select<false>(p, cluster, s);
  if (e != cudaSuccess) return e;
  return d == 64 ? launch_move<64>(p, num_sms, s) : launch_move<128>(p, num_sms, s);
}

}  // namespace fm
