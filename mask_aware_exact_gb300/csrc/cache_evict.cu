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
//
// Measured (whole calls, L2 flushed, into other pages with an index): 64 sequences up to 8192
// of 8 heads of 128 cut to a quarter 184 us: 24 for the first kernel (latency: barriers and the
// weights' way in; its histograms stay in shared memory) and 158 for the second (704 MB, 4.5
// TB/s, 66 % of a copy: the kept bytes of V lie apart, so that its source pages are read
// whole). Two sequences of 131072 cut to an eighth 107 us: 35 and 71 (361 MB, 5.1 TB/s). A page
// to be written is a chain of look-ups, loads, largest codes and stores behind two or three
// barriers; four CTAs an SM hide most of it (three 201 us, five with fewer registers 193, where
// four took 186). In place, caches of 8 heads of 128 that no call has cut before, and their
// floors (the weights, and the kept tokens read and written): 40 sequences of 8192 cut to 2048
// 163 us (52), 64 of them 242 (83); 64 of 2112 that give up 64 tokens 200 (81), of 2049 that give
// up one 157 (81; the pages before its place stay). Equal weights cost no more: with all of
// them zero, 64 sequences of 8192 into other pages take 176 us where spread ones take 210, since
// the tokens that stay lie together.
#include <atomic>

#include "cache_common.cuh"
#include "flashmask.h"

namespace fm {
namespace {

// ---------------------------------------------------------------- selection
constexpr int kClusterMost = 8;
constexpr int kBins = 2048;
constexpr int kPagesShare = 256;                                      // of a CTA while its cluster may grow
// whose keys fit its shared memory (8 segments of 131072 in a table of one page more, whole call:
// 61 us; with the weights read again in each pass 71)
constexpr int kPagesCached = 704;
constexpr int kPagesFew = 64;
constexpr int kPagesMost = FM_MAX_SEQLEN / kPage / kClusterMost;      // of a CTA

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The int at the same shared-memory address in CTA `rank`, written before the last
// cluster_sync. (Several of these are on their way at once: one takes 800 cycles.)
__device__ __forceinline__ int of_cta(const int* at, int rank) {
  uint32_t remote;
  int v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(smem_u32(at)), "r"(rank));
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(remote));
  return v;
}
__device__ __forceinline__ void to_cta(int* at, int rank, int v) {
  uint32_t remote;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(smem_u32(at)), "r"(rank));
  asm volatile("st.shared::cluster.s32 [%0], %1;" ::"r"(remote), "r"(v) : "memory");
}
// Sum of it over the first n CTAs of the cluster.
__device__ __forceinline__ int of_ctas(const int* at, int n) {
  int v[kClusterMost];
#pragma unroll
  for (int r = 0; r < kClusterMost; ++r) v[r] = r < n ? of_cta(at, r) : 0;
  int sum = 0;
#pragma unroll
  for (int r = 0; r < kClusterMost; ++r) sum += v[r];
  return sum;
}

// Four bytes on their way into shared memory.
__device__ __forceinline__ void copy4(void* dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}

// Weights in an order of unsigned numbers: NaN below all others, -0 as +0.
__device__ __forceinline__ uint32_t order_key(float w) {
  const uint32_t u = __float_as_uint(w + 0.f), key = u >> 31 ? ~u : u | 0x80000000u;
  return isnan(w) ? 0u : key;
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
  int wsum[32 + 4];
  int found[2];   // bin, keys wanted of it
  int totals[2];  // of this CTA: keys equal to the last one, tokens kept beside these
  int place;      // of the segment's pages in the list of pages to be written (rank 0)
};

// `most`: pages of a CTA that there is shared memory for.
template <int kThreads, bool kCached>
__global__ void __launch_bounds__(kThreads) evict_select_kernel(const EvictParams p, const int cluster, const int most) {
  constexpr int kWarps = kThreads / 32;
  extern __shared__ __align__(16) uint8_t smem[];
  SelectSmem& sh = *reinterpret_cast<SelectSmem*>(smem);
  uint64_t* masks = reinterpret_cast<uint64_t*>(smem + (sizeof(SelectSmem) + 15) / 16 * 16);  // [pages]
  uint64_t* equals = masks + most;
  int* counts = reinterpret_cast<int*>(equals + most);
  uint32_t* keys = reinterpret_cast<uint32_t*>(counts + most);  // kCached
  int* sums = reinterpret_cast<int*>(keys) + (kCached ? most * kPage : 0);  // of a cluster: the bins of all CTAs
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int seg = blockIdx.x / cluster, rank = blockIdx.x - seg * cluster;
  const int b = seg / p.c.Hk, hk = seg - b * p.c.Hk;
  const Kept kp = kept_of(p, b, tid == 0 && rank == 0 && hk == 0);
  const int pages = (kp.len + kPage - 1) / kPage, each = (pages + cluster - 1) / cluster;
  const int p0 = min(rank * each, pages), np = min(each, pages - p0);
  if (tid == 0 && rank == 0) {
    sh.place = atomicAdd(p.count, (kp.n + kPage - 1) / kPage);
    if (hk == 0) {
      p.info[2 * b] = kp.len;
      p.info[2 * b + 1] = kp.n;
    }
  }

  auto page_of = [&](int i) {
    const int page = p.table[static_cast<size_t>(b) * p.max_pages + p0 + i];
    if (page >= 0 && page < p.c.pages) return page;
    record_failure(p.status, kStatusPage, kSiteEvictPage);
    return -1;
  };
  // keys of a page: this lane's tokens lane and lane + 32
  auto keys_of = [&](int i, uint32_t (&k)[2]) {
    if constexpr (kCached) {
      k[0] = keys[i * kPage + lane];
      k[1] = keys[i * kPage + lane + 32];
    } else {
      const int page = page_of(i);
      const float* at = p.weights + (static_cast<size_t>(max(page, 0)) * p.c.Hk + hk) * kPage + lane;
      const float w0 = at[0], w1 = at[32];
      k[0] = page < 0 ? 0u : order_key(w0);
      k[1] = page < 0 ? 0u : order_key(w1);
    }
  };
  for (int i = tid; i < 2 * kBins; i += kThreads) sh.hist[0][i] = 0;
  if constexpr (kCached) {
    // a warp's pages, each looked up by a lane
    for (int i0 = warp; i0 < np; i0 += 32 * kWarps) {
      const int mine = i0 + lane * kWarps < np ? page_of(i0 + lane * kWarps) : -1;
      const int n = min((np - i0 + kWarps - 1) / kWarps, 32);
      // (all on their way at once: by way of registers they came a few at a time; 2 segments of
      // 300000 tokens, whole call: 162 us, so 140)
      for (int j = 0; j < n; ++j) {
        const int page = __shfl_sync(0xffffffffu, mine, j);
        uint32_t* to = keys + (i0 + j * kWarps) * kPage + lane;
        if (page >= 0) {
          const float* at = p.weights + (static_cast<size_t>(page) * p.c.Hk + hk) * kPage + lane;
          copy4(to, at);
          copy4(to + 32, at + 32);
        } else {
          to[0] = to[32] = 0x7fffffffu;
        }
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    for (int i = warp; i < np; i += kWarps) {
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        uint32_t& k = keys[i * kPage + lane + 32 * x];  // (copied by this thread)
        k = order_key(__uint_as_float(k));
      }
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
        for (int i = tid; i < kBins; i += kThreads) hist[i] = 0;
        __syncthreads();
      }
      for (int i = warp; i < np; i += kWarps) {
        uint32_t k[2];
        keys_of(i, k);
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int j = (p0 + i) * kPage + lane + 32 * x;
          if ((j >= kp.lo) & (j < kp.hi) & ((k[x] & known) == prefix)) atomicAdd(&hist[k[x] >> shift & (bins - 1)], 1);
        }
      }
      const int* bin = hist;
      if (cluster == 1) {
        __syncthreads();
      } else {
        // each CTA adds up its share of the bins for all (a cluster's CTAs that all read all bins
        // of one another took 20000 cycles a pass)
        bin = sums;
        cluster_sync();
        const int share = bins / cluster;
        for (int i = rank * share + tid; i < (rank + 1) * share; i += kThreads) {
          const int v = of_ctas(&hist[i], cluster);
          for (int r = 0; r < cluster; ++r) to_cta(&sums[i], r, v);
        }
        cluster_sync();
      }
      // this thread's bins, from the top
      constexpr int kMine = kBins / kThreads;
      int c[kMine], sum = 0;
      const int top = bins - 1 - kMine * tid;
#pragma unroll
      for (int x = 0; x < kMine; ++x) {
        c[x] = top < x ? 0 : bin[top - x];
        sum += c[x];
      }
      int all;
      int above = block_before<kWarps>(sum, sh.wsum, all);
#pragma unroll
      for (int x = 0; x < kMine; ++x) {
        if (above < want && want <= above + c[x]) {
          sh.found[0] = top - x;
          sh.found[1] = want - above;
        }
        above += c[x];
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
  for (int i = warp; i < np; i += kWarps) {
    uint32_t k[2], keep[2], same[2];
    keys_of(i, k);
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int j = (p0 + i) * kPage + lane + 32 * x;
      const bool choice = (j >= kp.lo) & (j < kp.hi);
      keep[x] = __ballot_sync(0xffffffffu, (choice & (k[x] > last)) | (!choice & (j < kp.len)));
      same[x] = __ballot_sync(0xffffffffu, choice & (k[x] == last) & (equal > 0));
    }
    if (lane == 0) {
      masks[i] = static_cast<uint64_t>(keep[1]) << 32 | keep[0];
      equals[i] = static_cast<uint64_t>(same[1]) << 32 | same[0];
    }
  }
  __syncthreads();
  // a thread's pages in a row: what is equal and what is kept beside it before them, in this
  // CTA and in those before it. Of the equal ones the lowest positions stay.
  const int per = (np + kThreads - 1) / kThreads, i0 = min(tid * per, np), i1 = min(i0 + per, np);
  int same_mine = 0, kept_mine = 0, same_all, kept_all;
  for (int i = i0; i < i1; ++i) same_mine += __popcll(equals[i]), kept_mine += __popcll(masks[i]);
  int same = block_before<kWarps>(same_mine, sh.wsum, same_all), at = block_before<kWarps>(kept_mine, sh.wsum, kept_all);
  if (cluster > 1) {
    if (tid == 0) sh.totals[0] = same_all, sh.totals[1] = kept_all;
    cluster_sync();
    same += of_ctas(&sh.totals[0], rank);
    at += of_ctas(&sh.totals[1], rank);
  }
  at += min(equal, same);
  const size_t row = static_cast<size_t>(seg) * p.max_pages;
  int32_t* before = p.before + static_cast<size_t>(seg) * (p.max_pages + 1);
  const int place = cluster == 1 ? sh.place : of_cta(&sh.place, 0);
  for (int i = i0; i < i1; ++i) {
    uint64_t e = equals[i];
    const int some = __popcll(e);
    for (int drop = some - min(max(equal - same, 0), some); drop > 0; --drop)
      e &= ~(1ull << (63 - __clzll(static_cast<long long>(e))));
    same += some;
    masks[i] |= e;
    const int n = __popcll(masks[i]), to = (at + kPage - 1) / kPage;
    p.mask[row + p0 + i] = masks[i];
    before[p0 + i] = at;
    p.was_read[row + p0 + i] = 0;
    if (n > 0 && to * kPage < at + n) p.list[place + to] = make_int2(seg, to << 16 | (p0 + i));
    counts[i] = at;
    at += n;
  }
  if (tid == 0 && rank == 0) before[pages] = kp.n;
  if (p.index != nullptr) {
    __syncthreads();
    int32_t* index = p.index + static_cast<size_t>(seg) * p.index_width;
    for (int i = warp; i < np; i += kWarps) {
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
constexpr int kWindow = kMoveThreads;  // source pages looked at a time
constexpr int kMinExp = -100;
constexpr int kAheadKept = 4;

__device__ __forceinline__ uint32_t codes_times(uint32_t w, float f) {
  uint32_t lo, hi;
  codes_to_f16(w, lo, hi);
  float v[4];
  asm("{.reg .f16 a, b; mov.b32 {a, b}, %2; cvt.f32.f16 %0, a; cvt.f32.f16 %1, b;}" : "=f"(v[0]), "=f"(v[1]) : "r"(lo));
  asm("{.reg .f16 a, b; mov.b32 {a, b}, %2; cvt.f32.f16 %0, a; cvt.f32.f16 %1, b;}" : "=f"(v[2]), "=f"(v[3]) : "r"(hi));
  return pack_e4m3x4(v[0] * f, v[1] * f, v[2] * f, v[3] * f);
}
// The same for powers of two from 2^-14 to 2^15, as an fp16 pair ff: the products are exact there.
__device__ __forceinline__ uint32_t codes_times_f16(uint32_t w, uint32_t ff) {
  uint32_t lo, hi, r;
  codes_to_f16(w, lo, hi);
  asm("{.reg .b32 x, y; .reg .b16 a, b; mul.rn.f16x2 x, %1, %3; mul.rn.f16x2 y, %2, %3; "
      "cvt.rn.satfinite.e4m3x2.f16x2 a, x; cvt.rn.satfinite.e4m3x2.f16x2 b, y; mov.b32 %0, {a, b};}"
      : "=r"(r)
      : "r"(lo), "r"(hi), "r"(ff));
  return r;
}
// What codes of a page of scale `was` are multiplied by for one of scale `now`. Codes that are
// all zero do not count for `now`, so that the quotient may pass fp32 for them (others leave
// it below 2^19), and zero times infinity would be NaN.
__device__ __forceinline__ float scale_ratio(float was, float now) { return fminf(was / now, 0x1p100f); }
__device__ __forceinline__ bool plain_power(float f) {
  return (__float_as_uint(f) & 0x7fffffu) == 0 && f >= 0x1p-14f && f <= 0x1p15f;
}
// Largest magnitudes of codes, kept as 16-bit pairs: the even bytes of words and the odd ones.
struct Widest {
  uint32_t even = 0, odd = 0;
  __device__ __forceinline__ void add(uint32_t w) {
    even = __vmaxu2(even, w & 0x007f007fu);
    odd = __vmaxu2(odd, w >> 8 & 0x007f007fu);
  }
};
constexpr uint32_t kNan = 0x7f;
// Word without its NaN codes.
__device__ __forceinline__ uint32_t without_nan(uint32_t w) { return w & ~__vcmpeq4(w & 0x7f7f7f7fu, 0x7f7f7f7fu); }
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

// Source pages of a page to be written, from the one of its first token on.
struct Window {
  int before[kWindow + 1];
  int table[kWindow];
  uint64_t mask[kWindow];
};
struct MoveSmem {
  Window window[2];
  int token[kPage];            // where each slot's token is now
  int page[kPage];             // its page, -1: none
  float kscale[kPage], vscale[kPage], weight[kPage];
  uint32_t vmax[4][kPage];     // largest V codes of a slot in a quarter of the rows
  float top[kPage];            // largest K code of each slot
  int exps[2];
  int job;
};

// A page to be written: page dp of sequence b, head hk; its first token is in page s.
struct Move {
  int b, hk, dp, s;
  int pages, cnt;  // pages of the sequence before, tokens of this page
  int seg;
};

template <int D, bool kInPlace>
__global__ void __launch_bounds__(kMoveThreads, 4) evict_move_kernel(const __grid_constant__ EvictParams p) {
  __shared__ MoveSmem sh;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int Hk = p.c.Hk;
  const int32_t* out_table = kInPlace ? p.table : p.out_table;
  const int out_pages = kInPlace ? p.max_pages : p.out_pages;
  const uint32_t jobs = static_cast<uint32_t>(*p.count);  // (written by the kernel before)
  if (blockIdx.x == 0) {
    for (int b = tid; b < p.B; b += kMoveThreads) {
      const int n = p.info[2 * b + 1];
      p.new_lens[b] = n;
      if (!kInPlace && (n + kPage - 1) / kPage > out_pages) record_failure(p.status, kStatusPage, kSiteEvictRange);
    }
  }

  auto locate = [&](const int2& e) {
    Move m;
    m.seg = e.x;
    m.b = p.by_Hk.div(e.x);
    m.hk = e.x - m.b * Hk;
    m.dp = e.y >> 16;
    m.s = e.y & 0xffff;
    const int2 info = reinterpret_cast<const int2*>(p.info)[m.b];
    m.pages = (info.x + kPage - 1) / kPage;
    m.cnt = min(kPage, info.y - m.dp * kPage);
    return m;
  };
  auto row_of = [&](const Move& m) { return static_cast<size_t>(m.seg) * p.max_pages; };
  auto before_of = [&](const Move& m) { return p.before + static_cast<size_t>(m.seg) * (p.max_pages + 1); };
  // this thread's part of the window from page s on
  struct Part {
    int before, end, table;
    uint64_t mask;
  };
  auto load_part = [&](const Move& m, int s) {
    Part x = {};
    const int n = min(kWindow, m.pages - s);
    if (tid < n) {
      x.before = before_of(m)[s + tid];
      x.mask = p.mask[row_of(m) + s + tid];
      x.table = p.table[static_cast<size_t>(m.b) * p.max_pages + s + tid];
    }
    if (tid == 0) x.end = before_of(m)[s + n];
    return x;
  };
  auto store_part = [&](const Move& m, int s, const Part& x, Window& w) {
    const int n = min(kWindow, m.pages - s);
    if (tid < n) {
      w.before[tid] = x.before;
      w.mask[tid] = x.mask;
      w.table[tid] = x.table;
    }
    if (tid == 0) w.before[n] = x.end;
  };

  uint32_t job = blockIdx.x;
  if (kInPlace) {
    if (tid == 0) sh.job = atomicAdd(p.ticket, 1);
    __syncthreads();
    job = static_cast<uint32_t>(sh.job);
  }
  Move m = {};
  int s = 0, cur = 0;
  if (job < jobs) {
    m = locate(p.list[job]);
    s = m.s;
    store_part(m, s, load_part(m, s), sh.window[0]);
  }
  while (job < jobs) {
    __syncthreads();  // the window is there, and the shared words of the page before have been read
    if (kInPlace && tid == 0) sh.job = atomicAdd(p.ticket, 1);
    // where the slots' tokens are
    const int r0 = m.dp * kPage;
    int found = -1, page = -1;
    while (true) {
      const Window& w = sh.window[cur];
      const int n = min(kWindow, m.pages - s), have = w.before[n];
      if (tid < m.cnt && found < 0 && r0 + tid >= w.before[0] && r0 + tid < have) {
        const int r = r0 + tid;
        int l = 0, h = n;  // before[l] <= r < before[h]
        while (h - l > 1) {
          const int mid = (l + h) >> 1;
          if (w.before[mid] <= r) l = mid; else h = mid;
        }
        // the k-th token kept of that page
        int k = r - w.before[l], bit = 0;
        uint64_t x = w.mask[l];
#pragma unroll
        for (int v = 32; v > 0; v >>= 1) {
          const int c = __popcll(x & ((1ull << v) - 1ull));
          if (k >= c) k -= c, bit += v, x >>= v;
        }
        found = (s + l) * kPage + bit;
        page = w.table[l];
        if (page < 0 || page >= p.c.pages) {
          record_failure(p.status, kStatusPage, kSiteEvictPage);
          page = -1;
        }
      }
      if (have >= r0 + m.cnt || s + n >= m.pages) break;
      s += n;  // few are kept: further pages
      __syncthreads();
      store_part(m, s, load_part(m, s), sh.window[cur]);
      __syncthreads();
    }
    float slot_ks = 0.f, slot_vs = 0.f, slot_w = 0.f;
    if (tid < kPage) {
      if (page >= 0) {
        const size_t ph = static_cast<size_t>(page) * Hk + m.hk;
        slot_ks = p.c.kscale[ph];
        slot_vs = p.c.vscale[ph];
        slot_w = p.weights[ph * kPage + (found & (kPage - 1))];
      }
      sh.page[tid] = page;
      sh.token[tid] = found;
    }
    // in place, a page whose tokens all stay is left alone
    const bool moved = __syncthreads_or(tid < m.cnt && (!kInPlace || found != r0 + tid));

    // K: a thread has a quarter of a slot's row. V: the rows vq, vq + 4, .. of a slot, the
    // slots side by side in the lanes, so that the bytes of a source page lie together (with
    // a row's four neighbours in a thread a load touched 10 sectors in place of 4 and the
    // lookups of them bound the kernel).
    const int ks_slot = tid >> 2, kq = tid & 3;
    const int vslot = lane + 32 * (warp & 1), vq = warp >> 1;
    uint4 kr[D / 64];
    uint32_t vr[D / 16];
    if (moved) {
      const int kp = sh.page[ks_slot];
      const uint8_t* src = p.c.k8 + (static_cast<size_t>(max(kp, 0)) * Hk + m.hk) * (kPage * D) +
                           (sh.token[ks_slot] & (kPage - 1)) * D + 16 * kq;
#pragma unroll
      for (int i = 0; i < D / 64; ++i)
        kr[i] = kp < 0 ? make_uint4(0u, 0u, 0u, 0u) : *reinterpret_cast<const uint4*>(src + 64 * i);
      const int vp = sh.page[vslot];
      src = p.c.v8 + (static_cast<size_t>(max(vp, 0)) * Hk + m.hk) * (kPage * D) + (sh.token[vslot] & (kPage - 1)) + vq * kPage;
      uint8_t v[D / 4];
#pragma unroll
      for (int i = 0; i < D / 4; ++i) v[i] = vp < 0 ? 0 : src[4 * i * kPage];
#pragma unroll
      for (int i = 0; i < D / 16; ++i)
        vr[i] = v[4 * i] + (static_cast<uint32_t>(v[4 * i + 1]) << 8) + (static_cast<uint32_t>(v[4 * i + 2]) << 16) +
                (static_cast<uint32_t>(v[4 * i + 3]) << 24);
    }
    // the next page to be written: its first token's page is on its way, then its window
    const uint32_t next = kInPlace ? static_cast<uint32_t>(sh.job) : job + gridDim.x;
    int2 entry = make_int2(0, 0);
    if (next < jobs) entry = p.list[next];
    if (moved) {
      if (tid < kPage) {
        sh.kscale[tid] = slot_ks;
        sh.vscale[tid] = slot_vs;
        sh.weight[tid] = slot_w;
      }
      // largest codes, K's over the slot's four threads
      Widest k, v;
#pragma unroll
      for (int i = 0; i < D / 64; ++i) {
        k.add(kr[i].x);
        k.add(kr[i].y);
        k.add(kr[i].z);
        k.add(kr[i].w);
      }
#pragma unroll
      for (int i = 0; i < D / 16; ++i) v.add(vr[i]);
      uint32_t kw = __vmaxu2(k.even, k.odd);
      kw = max(kw & 0xffffu, kw >> 16);
      // (rare: NaN codes do not count, and V keeps none)
      if (__builtin_expect(__any_sync(0xffffffffu, kw == kNan), 0)) {
        Widest x;
#pragma unroll
        for (int i = 0; i < D / 64; ++i) {
          x.add(without_nan(kr[i].x));
          x.add(without_nan(kr[i].y));
          x.add(without_nan(kr[i].z));
          x.add(without_nan(kr[i].w));
        }
        kw = __vmaxu2(x.even, x.odd);
        kw = max(kw & 0xffffu, kw >> 16);
      }
      uint32_t vw = __vmaxu2(v.even, v.odd);
      vw = max(vw & 0xffffu, vw >> 16);
      if (__builtin_expect(__any_sync(0xffffffffu, vw == kNan), 0)) {
        Widest x;
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          vr[i] = without_nan(vr[i]);
          x.add(vr[i]);
        }
        vw = __vmaxu2(x.even, x.odd);
        vw = max(vw & 0xffffu, vw >> 16);
      }
      kw = max(kw, __shfl_xor_sync(0xffffffffu, kw, 1));
      kw = max(kw, __shfl_xor_sync(0xffffffffu, kw, 2));
      if (kq == 0) sh.top[ks_slot] = code_value(kw);
      sh.vmax[vq][vslot] = vw;
    }
    Move m2 = {};
    Part part = {};
    if (next < jobs) {
      m2 = locate(entry);
      part = load_part(m2, m2.s);
    }
    __syncthreads();  // all of the page's tokens have been read
    if (moved) {
      if (kInPlace && tid == 0)
        asm volatile("fence.acq_rel.gpu;\n\tst.relaxed.gpu.global.s32 [%0], %1;" ::"l"(p.was_read + row_of(m) + m.dp), "r"(1)
                     : "memory");
      if (warp < 2) {
        // the largest magnitudes, times 2^-9, of the slots whose scales are some
        float top = 0.f;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int i = lane + 32 * x;
          if (no_scales(sh.kscale[i], sh.vscale[i])) continue;
          if (warp == 0) {
            top = fmaxf(top, sh.top[i] * (sh.kscale[i] * 0x1p-9f));
          } else {
            const uint32_t c = max(max(sh.vmax[0][i], sh.vmax[1][i]), max(sh.vmax[2][i], sh.vmax[3][i]));
            top = fmaxf(top, code_value(c) * (sh.vscale[i] * 0x1p-9f));
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
          const int a = before_of(m)[min(m.dp, m.pages)], z = before_of(m)[min(m.dp + 1, m.pages)];
          const int reader = tid == 64 ? a / kPage : (z - 1) / kPage;
          if (z > a && reader != m.dp) {
            const int32_t* flag = p.was_read + row_of(m) + reader;
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
      // V of the next page's source pages on its way to L2 (64 x 8192 tokens cut to a quarter:
      // 199 -> 186 us; K's kept rows, or whole pages of K, as well: 236, 198). Where a page
      // keeps fewer than kAheadKept tokens, half of it may be what no slot asks for.
      if (next < jobs && tid < min(kWindow, m2.pages - m2.s)) {
        const int kept = __popcll(part.mask), r2 = m2.dp * kPage;
        if (kept >= kAheadKept && part.before < r2 + m2.cnt && part.before + kept > r2 && part.table >= 0 &&
            part.table < p.c.pages)
          asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(
                           p.c.v8 + (static_cast<size_t>(part.table) * Hk + m2.hk) * (kPage * D)),
                       "r"(kPage * D)
                       : "memory");
      }
      int to = -1;
      if (m.dp < out_pages) {
        to = out_table[static_cast<size_t>(m.b) * out_pages + m.dp];
        if (to < 0 || to >= p.c.pages) {
          if (tid == 0) record_failure(p.status, kStatusPage, kSiteEvictPage);
          to = -1;
        }
      }
      if (to >= 0) {
        const size_t ph = static_cast<size_t>(to) * Hk + m.hk;
        const float k_new = __int_as_float((sh.exps[0] + 127) << 23), v_new = __int_as_float((sh.exps[1] + 127) << 23);
        {
          const float f = scale_ratio(sh.kscale[ks_slot], k_new);
          const bool bad = no_scales(sh.kscale[ks_slot], sh.vscale[ks_slot]);
          uint8_t* dst = p.c.k8 + ph * (kPage * D) + ks_slot * D + 16 * kq;
          if (bad) {
#pragma unroll
            for (int i = 0; i < D / 64; ++i) kr[i] = make_uint4(0x7f7f7f7fu, 0x7f7f7f7fu, 0x7f7f7f7fu, 0x7f7f7f7fu);
          } else if (f != 1.f) {
            if (plain_power(f)) {
              const uint32_t ff = pack_f16x2(f, f);
#pragma unroll
              for (int i = 0; i < D / 64; ++i)
                kr[i] = make_uint4(codes_times_f16(kr[i].x, ff), codes_times_f16(kr[i].y, ff),
                                   codes_times_f16(kr[i].z, ff), codes_times_f16(kr[i].w, ff));
            } else {
#pragma unroll
              for (int i = 0; i < D / 64; ++i)
                kr[i] = make_uint4(codes_times(kr[i].x, f), codes_times(kr[i].y, f), codes_times(kr[i].z, f),
                                   codes_times(kr[i].w, f));
            }
          }
#pragma unroll
          for (int i = 0; i < D / 64; ++i) *reinterpret_cast<uint4*>(dst + 64 * i) = kr[i];
        }
        {
          const float f = scale_ratio(sh.vscale[vslot], v_new);
          const bool bad = no_scales(sh.kscale[vslot], sh.vscale[vslot]);
          if (bad) {
#pragma unroll
            for (int i = 0; i < D / 16; ++i) vr[i] = 0u;
          } else if (f != 1.f) {
            if (plain_power(f)) {
              const uint32_t ff = pack_f16x2(f, f);
#pragma unroll
              for (int i = 0; i < D / 16; ++i) vr[i] = codes_times_f16(vr[i], ff);
            } else {
#pragma unroll
              for (int i = 0; i < D / 16; ++i) vr[i] = codes_times(vr[i], f);
            }
          }
          __syncwarp();
          // four rows of a slot in a thread -> four slots of row 16 i + 4 (lane % 4) + vq
          uint8_t* dst = p.c.v8 + ph * (kPage * D) + (vslot & ~3) + (4 * (lane & 3) + vq) * kPage;
          const uint32_t first = lane & 1 ? 0x3715u : 0x6240u, second = lane & 2 ? 0x3276u : 0x5410u;
#pragma unroll
          for (int i = 0; i < D / 16; ++i) {
            uint32_t x = __byte_perm(vr[i], __shfl_xor_sync(0xffffffffu, vr[i], 1), first);
            x = __byte_perm(x, __shfl_xor_sync(0xffffffffu, x, 2), second);
            *reinterpret_cast<uint32_t*>(dst + 16 * i * kPage) = x;
          }
        }
        if (tid < kPage) p.weights[ph * kPage + tid] = sh.weight[tid];
        if (tid == 0) {
          p.c.kscale[ph] = k_new;
          p.c.vscale[ph] = v_new;
        }
      }
    }
    job = next;
    if (next >= jobs) break;
    cur ^= 1;
    m = m2;
    s = m2.s;
    store_part(m, s, part, sh.window[cur]);
  }
  // the last CTA leaves the counters as the next call wants them
  if (tid == 0 && atomic_add_acq_rel(p.done, 1) == static_cast<int>(gridDim.x) - 1) {
    *p.count = 0;
    *p.ticket = 0;
    *p.done = 0;
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

template <int kThreads, bool kCached>
cudaError_t launch_select(const EvictParams& p, int cluster, cudaStream_t s) {
  // shared memory for the pages that a CTA may have
  const int most = ((p.max_pages + cluster - 1) / cluster + 1) / 2 * 2;
  auto bytes = [](int pages, bool clusters) {
    return static_cast<int>((sizeof(SelectSmem) + 15) / 16 * 16) + pages * (8 + 8 + 4) + (kCached ? pages * kPage * 4 : 0) +
           (clusters ? kBins * 4 : 0);
  };
  static_assert(sizeof(SelectSmem) + 16 + kPagesCached * (20 + kPage * 4) + kBins * 4 <= 227 * 1024 &&
                    sizeof(SelectSmem) + 16 + kPagesMost * 20 + kBins * 4 <= 227 * 1024,
                "shared memory per CTA");
  static std::atomic<uint64_t> done[4];
  const cudaError_t e = allow_smem(evict_select_kernel<kThreads, kCached>, bytes(kCached ? kPagesCached : kPagesMost, true), done);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.B) * p.c.Hk * cluster);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = bytes(most, cluster > 1);
  cfg.stream = s;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = static_cast<unsigned>(cluster);
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, evict_select_kernel<kThreads, kCached>, p, cluster, most);
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
  w.counters = off;  // (at the same place for all sizes: they have to be zero)
  off = up256(off + 12);
  w.info = off;
  off = up256(off + static_cast<size_t>(B) * 8);
  w.mask = off;
  off = up256(off + segs * max_pages * 8);
  w.before = off;
  off = up256(off + segs * (max_pages + 1) * 4);
  w.list = off;
  off = up256(off + segs * max_pages * 8);
  w.was_read = off;
  off = up256(off + segs * max_pages * 4);
  w.total = off;
  return w;
}

cudaError_t launch_cache_evict(int d, EvictParams p, int num_sms, cudaStream_t s) {
  p.by_Hk.set(p.c.Hk);
  // CTAs of a segment: as many as hold its keys, and more down to kPagesFew pages each while
  // they leave SMs free (one segment of 16384 tokens, whole call, measured as below: 29.0 -> 25.6
  // us; shares of 32 pages take 4000 tokens from 17.6 to 22.8)
  int cluster = 1;
  while (cluster < kClusterMost &&
         (cluster * kPagesShare < p.max_pages ||
          (cluster * kPagesFew < p.max_pages && 2LL * p.B * p.c.Hk * cluster <= num_sms)))
    cluster *= 2;
  // CTAs of 256 threads where there are several for each SM, which hide one another's
  // barriers: 64 x 8 segments of 8192, whole calls, 187 us; of 512, 195. Otherwise of 512 (in
  // place, a cache cut the same way again, so that most of it lies in front): 20 x
  // 8 segments 86 us (256: 89, 1024: 97), 8 of 16384 31.6 (34.2, 35.2), 16 of 131072 112 (120,
  // 134: clusters of eight CTAs that fill an SM each do not all find a place at once).
  const bool many = static_cast<long long>(p.B) * p.c.Hk * cluster > 2LL * num_sms;
  cudaError_t e;
  if (cluster * kPagesCached < p.max_pages)
    e = launch_select<1024, false>(p, cluster, s);
  else
    e = many ? launch_select<256, true>(p, cluster, s) : launch_select<512, true>(p, cluster, s);
  if (e != cudaSuccess) return e;
  return d == 64 ? launch_move<64>(p, num_sms, s) : launch_move<128>(p, num_sms, s);
}

}  // namespace fm
