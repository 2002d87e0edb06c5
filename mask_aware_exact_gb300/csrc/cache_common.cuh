// Parts shared by the two kernels of the attention over the paged cache: rows and
// pages, the cut of the line of pages into runs, waits and conversions.
#pragma once
#include "cache.h"
#include "ptx_fp8.cuh"

namespace fm {

// ---------------------------------------------------------------- geometry

// Row tile `rt` of sequence b: its query tokens [t_lo, t_hi] at positions t + shift,
// none when t_hi < t_lo; len is the sequence's length, cut to what the table holds.
struct RowTile {
  int len, live, shift, t_lo, t_hi;
};
__device__ __forceinline__ RowTile row_tile(const CacheFwdParams& p, const Geometry& geo, int b, int rt,
                                            bool record) {
  RowTile r;
  r.live = p.q_lens ? min(max(p.q_lens[b], 0), p.N) : p.N;
  r.len = p.lens[b];
  const int most = p.max_pages * kPage;
  if (r.len < 0 || r.len > most) {
    if (record) record_failure(p.status, kStatusPage, kSiteCacheLen);
    r.len = min(max(r.len, 0), most);
  }
  r.shift = r.len - r.live;
  const int rows = geo.G * r.live, r0 = rt * geo.rows;
  r.t_lo = geo.by_G.div(r0);
  r.t_hi = r0 < rows ? geo.by_G.div(r0 + min(geo.rows, rows - r0) - 1) : r.t_lo - 1;
  return r;
}

__device__ __forceinline__ int mask_class(const CacheFwdParams& p, const Geometry& geo, int hk) {
  return geo.by_class.div(hk);
}

// Pages on a segment's line. (Not inline, like everything here that is not in a hot
// loop: a run that is short spends much of its time on fetching instructions.)
template <bool kVec>
static __device__ __noinline__ int pages_of(const CacheFwdParams& p, const Geometry& geo, int seg) {
  const int bh = geo.by_RT.div(seg), rt = seg - bh * geo.RT;
  const int b = geo.by_Hk.div(bh);
  if constexpr (kVec) {
    const int cls = mask_class(p, geo, bh - b * p.c.Hk);
    const size_t at = (static_cast<size_t>(b) * geo.classes + cls) * geo.RT + rt;
    return p.listed[at];
  } else {
    const RowTile r = row_tile(p, geo, b, rt, false);
    if (r.t_hi < r.t_lo) return 0;
    const int lim = p.mask.causal ? min(r.len, r.shift + r.t_hi + 1) : r.len;
    return lim > 0 ? (lim + kPage - 1) / kPage : 0;
  }
}

// The k-th page on the line of row tile rt of (b, hk), and whether intervals hide
// some of its keys from some row.
template <bool kVec>
__device__ __forceinline__ int page_on_line(const CacheFwdParams& p, const Geometry& geo, int b, int hk, int rt,
                                            int k, int& cut) {
  cut = 0;
  if constexpr (!kVec) return k;
  const size_t at = (static_cast<size_t>(b) * geo.classes + mask_class(p, geo, hk)) * geo.RT + rt;
  const int v = p.list[at * p.max_pages + k];
  cut = v >> 15;
  return v & 0x7fff;
}

__device__ __forceinline__ int atomic_add_acq_rel(int32_t* at, int x) {
  int old;
  asm volatile("atom.add.acq_rel.gpu.global.s32 %0, [%1], %2;" : "=r"(old) : "l"(at), "r"(x) : "memory");
  return old;
}

// A CTA's run on the line of units (pages, or pairs of them) of all segments.
struct Line {
  int run;         // units of a full run
  int lo, hi;      // this CTA's run
  int seg, first;  // segment of its first unit, and that unit's number in it
  bool any_empty;  // some segment has no unit
  bool brief;      // no segment has more than kUncut pages
};
constexpr int kLineWords = 40;  // ints of shared memory for find_run
// Segments of up to this many pages (or an eighth of a run) are not cut: a join takes
// 3 to 4 us, about as long as a CTA takes for 30 pages. 128 segments of up to 32 pages:
// 18.2 us whole, 21.5 cut; 512 of them 45.1, 51.0; of up to 64 pages 65.3 either way.
constexpr int kUncut = 32;
// The same where segments can be cut one by one (see below). One sequence of 1000 tokens,
// 8 cache heads (16 pages): 11.7 us whole, 11.4 cut; 500: 10.1, 11.5; 1500: 13.2, 12.1;
// 2000: 14.4, 12.0.
constexpr int kUncutApart = 16;
// Where there are at least two CTAs for each segment, the segments are cut one by one
// into equal runs if these are not longer than the line's by more than kApart pages:
// a second piece in a run costs a CTA about that much. Cut so / on the line: one
// sequence of 12000 tokens (8 cache heads) 17.1 / 25.3 us, four of up to 4000 14.7 / 17.8,
// 64 segments of 96 visible pages 35.7 / 37.8; with 28, 8 sequences of up to 16000 with 64
// rows would go from 55.8 to 59.2.
constexpr int kApart = 14;

// Sum of x over the threads before this one, and over all of them.
template <int kWarps>
static __device__ __noinline__ int block_before(int x, int* wsum, int& total) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int sum = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, sum, o);
    if (lane >= o) sum += y;
  }
  __syncthreads();  // wsum may still be read
  if (lane == 31) wsum[warp] = sum;
  __syncthreads();
  total = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    const int y = wsum[w];
    if (w < warp) sum += y;
    total += y;
  }
  return sum - x;
}

// Called by all kThreads threads of every CTA; units(s) is the number of units of
// segment s, `pages` the pages of a unit.
template <int kThreads, typename F>
__device__ __forceinline__ Line find_run(int nseg, int min_run, int pages, int* words, F units) {
  constexpr int kWarps = kThreads / 32;
  static_assert(2 * kWarps + 4 <= kLineWords, "shared words");
  int* const wsum = words;
  int* const wmax = words + kWarps;
  int* const found = words + 2 * kWarps;  // lo, hi, segment, first
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int each = (nseg + kThreads - 1) / kThreads;
  const int seg_lo = min(tid * each, nseg), seg_hi = min(seg_lo + each, nseg);
  int mine = 0, longest = 0;
  bool empty = false;
  for (int s = seg_lo; s < seg_hi; ++s) {
    const int n = units(s);
    mine += n;
    longest = max(longest, n);
    empty |= n == 0;
  }
  int before = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, before, o);
    if (lane >= o) before += x;
  }
  longest = __reduce_max_sync(0xffffffffu, longest);
  if (lane == 31) {
    wsum[warp] = before;
    wmax[warp] = longest;
  }
  Line r;
  r.any_empty = __syncthreads_or(empty);
  int total = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    const int x = wsum[w];
    if (w < warp) before += x;
    total += x;
    longest = max(longest, wmax[w]);
  }
  before -= mine;
  const int even = (total + static_cast<int>(gridDim.x) - 1) / static_cast<int>(gridDim.x);
  bool uncut = longest <= max(kUncutApart / pages, even / 8);
  int cut = 0;  // the runs' length if segments are cut one by one
  if (!uncut) {
    const int per = static_cast<int>(gridDim.x) / nseg;  // parts a segment may have
    if (per >= 2) cut = max(min_run, (longest + per - 1) / per);
    if (cut > even + kApart / pages) cut = 0;
    uncut = cut == 0 && longest <= kUncut / pages;
  }
  // the least run only keeps cut segments from falling into many parts
  r.run = max(uncut ? 1 : min_run, even);
  r.brief = longest <= kUncut / pages;
  if (cut > 0) {
    // runs of one segment each: on this line every segment is filled up to whole runs
    r.run = cut;
    const int filled = (mine + cut - 1) / cut * cut;  // a thread has one segment at most
    before = block_before<kWarps>(filled, wsum, total);
    const long long x_wide = static_cast<long long>(cut) * blockIdx.x;
    const int x = static_cast<int>(min(x_wide, static_cast<long long>(total)));
    if (x == total) {
      if (tid == 0) found[0] = found[1] = total, found[2] = nseg, found[3] = 0;
    } else if (before <= x && x < before + filled) {
      found[0] = x;
      found[1] = min(x + cut, before + mine);
      found[2] = seg_lo;
      found[3] = x - before;
    }
  } else {
#pragma unroll
    for (int side = 0; side < 2; ++side) {
      const long long x_wide = static_cast<long long>(r.run) * (blockIdx.x + side);
      const int x = static_cast<int>(min(x_wide, static_cast<long long>(total)));
      if (x == total) {
        if (tid == 0) {
          found[side] = total;
          if (side == 0) found[2] = nseg, found[3] = 0;  // no unit, no segment
        }
      } else if (before <= x && x < before + mine) {
        int s = seg_lo, at = before, n;
        // a thread with one segment knows its units
        while (x >= at + (n = each == 1 ? mine : units(s)) && s + 1 < seg_hi) at += n, ++s;
        const bool next = uncut && x != at;  // on to the segment's end
        found[side] = next ? at + n : x;
        if (side == 0) {
          found[2] = next ? s + 1 : s;
          found[3] = uncut ? 0 : x - at;
        }
      }
    }
  }
  __syncthreads();
  r.lo = found[0];
  r.hi = found[1];
  r.seg = found[2];
  r.first = found[3];
  return r;
}

// Joins. The parts of a cut segment lie in consecutive CTAs from cta0 on. Up to kOnce
// parts are added by the CTA whose part came last. Of more, every kFan are added up
// first, by the last of those, into the place of the group's first, and the last
// group's CTA adds the groups: one CTA alone takes 0.2 us for a part of 8 rows, 0.6 for
// one of 128 (one cache head, 131072 tokens: 47.9 -> 20.8 us, and 152.8 -> 54.4).
struct Join {
  int first, stride, n;  // parts first, first + stride, ..
  bool last;             // the segment's result; else a group's
};
// A part (or group, `group` true) that begins at part `part` of `parts` is written, by
// threads that the caller has met since. True if that was the last of a join.
template <int kOnce, int kFan>
static __device__ __noinline__ bool part_arrives(const CacheFwdParams& p, int cta0, int part, int parts, bool group,
                                                 Join& join) {
  if (parts > kOnce && !group) {
    const int g = part / kFan, n = min(kFan, parts - g * kFan);
    // (the group's first CTA may be the first of another segment's too)
    int32_t* at = p.groups + 2 * (cta0 + g * kFan) + (g == 0 ? 1 : 0);
    if (n > 1) {
      if (atomic_add_acq_rel(at, 1) != n - 1) return false;
      *at = 0;  // ready for the next call
      join = {g * kFan, 1, n, false};
      return true;
    }
  }
  const int n = parts > kOnce ? (parts + kFan - 1) / kFan : parts;
  if (atomic_add_acq_rel(&p.arrived[cta0], 1) != n - 1) return false;
  p.arrived[cta0] = 0;
  join = {0, parts > kOnce ? kFan : 1, n, true};
  return true;
}

// Units run_at .. + 31 of a CTA's run, one per lane: unit k of segment seg is lane
// 0's. Returns how many there are within 32 segments (at most `most`); a lane gets
// its segment, the unit's number in it and the segment's units.
template <typename F>
__device__ __forceinline__ int next_units(int seg, int k, int nseg, int most, F units, int& my_seg, int& my_k,
                                          int& my_n) {
  const int lane = threadIdx.x & 31;
  const int s = seg + lane;
  const int n_all = s < nseg ? units(s) : 0;
  int c = n_all - (lane == 0 ? k : 0);
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, c, o);
    // sums past 2^30 are only compared with lane numbers
    if (lane >= o) c = min(c + x, 1 << 30);
  }
  int j = 0;  // segments that end at or before this lane's unit
#pragma unroll
  for (int i = 16; i > 0; i >>= 1) {
    const int x = __shfl_sync(0xffffffffu, c, j + i - 1);
    if (x <= lane) j += i;
  }
  const int c_j = __shfl_sync(0xffffffffu, c, j);
  my_n = __shfl_sync(0xffffffffu, n_all, j);
  my_seg = seg + j;
  my_k = my_n - (c_j - lane);
  return min(__shfl_sync(0xffffffffu, c, 31), most);
}

// Whether a page's scales are none (negative, infinite or NaN): rows that see a key of
// it get NaN.
__device__ __forceinline__ int no_scales(float k, float v) {
  constexpr float kMost = 3.402823466e38f;
  return !(k >= 0.f && k <= kMost && v >= 0.f && v <= kMost);
}
// The same in three instructions, true for scales of -0 too.
__device__ __forceinline__ int may_be_no_scales(float k, float v) {
  return max(__float_as_uint(k), __float_as_uint(v)) >= 0x7f800000u;
}
// A score is a sum of products of codes and scaled query times c, c = (row's factor) * (K
// scale) kept above 0 so that masked scores stay at -inf. Where c would pass fp32 (a row's
// factor above 1, that is queries of 10^4 and more, and keys near 10^38), 2^110 of it go
// to the sum first: what overflows then is a score that does.
constexpr float kLeast = 1.17549435e-38f;
__device__ __forceinline__ float score_factor(float row, float k_scale) { return fmaxf(row * k_scale, kLeast); }
// What such a row's sums are multiplied by before c; NaN for a page without scales.
__device__ __forceinline__ float score_boost(float row, float k_scale, bool none, float& c) {
  float boost = 1.f;
  if (isinf(c)) {
    boost = __int_as_float((110 + 127) << 23);
    c = score_factor(row * __int_as_float((127 - 110) << 23), k_scale);
  }
  return none ? __int_as_float(0x7fffffff) : boost;
}

// Four codes -> two fp16 pairs.
__device__ __forceinline__ void codes_to_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{.reg .b16 a, b; mov.b32 {a, b}, %2; cvt.rn.f16x2.e4m3x2 %0, a; cvt.rn.f16x2.e4m3x2 %1, b;}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}
__device__ __forceinline__ uint32_t word(const uint4& v, int i) {
  return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
}
__device__ __forceinline__ uint32_t pack_f16x2(float a, float b) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %2, %1;" : "=r"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
      "l"(src), "r"(bytes), "r"(bar)
      : "memory");
}
// Bounded wait: gives up after the library's limit, or when another wait has (a
// page error alone does not end waits). Only the first test is inline: the roles'
// loops have to stay small for the instruction cache.
static __device__ __noinline__ bool cache_wait_slow(uint32_t bar, uint32_t parity, int32_t* status) {
  const uint64_t t0 = global_timer_ns();
  while (!mbar_try_wait(bar, parity)) {
    if ((*reinterpret_cast<volatile int32_t*>(status) & kStatusTimeout) != 0) return false;
    if (global_timer_ns() - t0 > FM_WAIT_LIMIT_NS) {
      record_failure(status, kStatusTimeout, kSiteCacheWait);
      return false;
    }
  }
  return true;
}
__device__ __forceinline__ bool cache_wait(uint32_t bar, uint32_t parity, int32_t* status) {
  return mbar_test_wait(bar, parity) || cache_wait_slow(bar, parity, status);
}
// A CTA that does not find the units of its run, because a caller wrote lens or q_lens
// while the call ran, gives up like a wait that ran out.
static __device__ __noinline__ bool lengths_moved(int32_t* status) {
  if ((threadIdx.x & 31) == 0) record_failure(status, kStatusTimeout, kSiteCacheWait);
  return false;
}
// cache_wait_slow for a counter in shared memory that only grows.
__device__ __forceinline__ bool count_wait(const int* count, int want, int32_t* status) {
  const volatile int* at = count;
  const uint64_t t0 = global_timer_ns();
  while (*at < want) {
    if ((*reinterpret_cast<volatile int32_t*>(status) & kStatusTimeout) != 0) return false;
    if (global_timer_ns() - t0 > FM_WAIT_LIMIT_NS) {
      record_failure(status, kStatusTimeout, kSiteCacheWait);
      return false;
    }
  }
  __threadfence_block();
  return true;
}
// A row's sums: P = 2^(score - m), l = sum P and acc = 2^(shift - mv) sum P V, with m the
// largest score so far and mv the log2 of the largest P * scale of V. mv counts from m: it
// would lose the scale beside a large score. Before the first key they have the lowest
// values, not -inf, so that differences are numbers.
constexpr float kNoScore = -3.402823466e38f, kNoProduct = -1e30f;
// The maxima of two states together. (In one pass: with m's first and then mv's, the sums
// of states took 2 to 3 % of calls whose segments are 20 to 80 pages long.)
__device__ __forceinline__ void join_maxima(float& m, float& mv, float m2, float mv2) {
  const float mm = fmaxf(m, m2);
  mv = fmaxf(mv + (m - mm), mv2 + (m2 - mm));
  m = mm;
}
__device__ __forceinline__ float out_factor(float mv, float l, float shift) {
  return l == 0.f ? 0.f : ex2(mv - shift) / l;
}
// log2 of a page's V scale; of 0, a value so low that nothing is left of its products.
__device__ __forceinline__ float log2_scale(float scale) { return fmaxf(__log2f(scale), -300.f); }
__device__ __forceinline__ float out_lse(float m, float l) {
  return l == 0.f ? -INFINITY : (m + __log2f(l)) * 0.69314718055994531f;
}

}  // namespace fm
