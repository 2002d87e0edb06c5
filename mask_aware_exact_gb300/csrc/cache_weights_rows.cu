// The attention weight of cached keys where a cache head has many query rows (the last
// rows of a prompt, drafted tokens of large groups): products S^T = K Q^T on tcgen05.
//
// Keys stay, rows stream. An item is four pages, 256 keys, as two operands of 128 rows
// in shared memory (fp16, exact for codes), converted once; tiles of 128 query rows pass by
// as the other operand. A first kernel writes those as fp16 tiles in the layout that the tensor
// cores read (128-byte swizzle), each row scaled by a power of two as in the attention,
// with the row's factor and LSE behind them, so that a tile is one bulk copy. With 256 keys
// on a CTA a tile of d = 128 is 32 KB for 1024 cycles of products.
//
// In S^T a thread owns a key (a TMEM lane): the sum over rows is a sum in its registers. x =
// (S * K scale) * factor - LSE, weight 2^x; a row's factor and LSE come from shared memory,
// the factor only where the rows of a tile differ in it (see the row tiles).
//
// K's codes are loaded an item ahead and converted while the products of the item before
// run, into the other of two pairs of operands. The main kernel starts while the row tiles
// are still being written and finds its run meanwhile (238 -> 230 us for the prompt below).
//
// Measured: the last 512 rows of 2 prompts up to 32768, 32 / 8 heads of 128 (2.7e11
// operations, 1.05e9 exponentials): 218 us, 1240 TFLOP/s, 65 % of the measured bf16 rate. The
// tensor cores are busy for 51 % of the cycles and the exponential unit, which gives 26 a
// cycle and SM, would need 145 us; what is left is the two warps a scheduler of the weights,
// each load of a tile, its 64 x 2 exponentials and their sums one chain. Not kept: weights'
// warps with two keys a thread and tiles of 96 rows, 16 of them, keys in TMEM as the
// first operand, units of 64 rows (a product of 128 x 64 takes 45 cycles, ideally 32), half
// tiles loaded ahead of their use 32 columns at a time (254 us).
// 16 sequences of 16384, 4 heads, by rows (us; L2 warm), with the kernel for few rows beside
// it where that takes them:
//   rows            24           32        40     64    128
//   d = 64    29.1 / 22.9  29.2 / 22.9   29.1   29.1   35.5
//   d = 128   37.7 / 29.2  37.7 / 29.2   37.6   38.2   41.5
//
// Items are cut into `parts` ranges of rows where there are few of them, on one line with
// equal runs for the CTAs; the pieces of an item that a run's border cuts leave their
// sums in the workspace, and the last to arrive adds them in order.
//
// Warp roles (480 threads):
//   0-7    weights: warpgroup w has operand w, a key a thread
//   8-11   conversion of K, 32 keys of each operand a warp
//   12     walks the run, looks pages up, brings row tiles in
//   13, 14 issue the products of an operand each: what one thread does between the products
//          of two tiles (waits, commits) takes longer than the tensor cores have work queued
// TMEM: two tiles of S^T for each operand, 128 columns each: a product of 128 keys and 64
// rows would run at 70 % of the rate of one with 128 rows.
#include <atomic>

#include "cache_weights.cuh"

namespace fm {
namespace {

constexpr int kThreads = 480;
constexpr int kMetaRing = 4;
constexpr int kMetaInts = 32;
constexpr int kKeys = 256;
constexpr int kTileRows = 128;
constexpr int kPartsRun = 32;  // (2 prompts up to 32768: 222 us; with 8 229, with 128 224)
constexpr int kHalf = 64;  // rows taken at a time
constexpr int kFactorRing = 8;       // of the row tiles' factors
constexpr int kFactorBytes = 1024;
constexpr uint32_t kNear = 8;  // (factors of their own for all rows: 521 us for the same prompts)
constexpr int kScanWords = kThreads / 32 + 4;

enum MetaWord { kFlags, kSeg, kTile0, kTiles, kCta0, kPieces, kLen, kLive, kPg = 8, kJ0 = 12, kKs = 16, kCutWord = 20 };
enum Flag { kEnd = 1, kWhole = 2, kTail = 4 };

template <int D>
struct Layout {
  static constexpr int kStages = D == 128 ? 2 : 8;  // row tiles in shared memory
  static constexpr int kK = 2;                      // pairs of K operands
  static constexpr int kStageBytes = D * 256;
  static constexpr int kTileBytes = kStageBytes + kFactorBytes;  // in the workspace
  static constexpr int kKOperand = 128 * D * 2;
  static constexpr int kKeysAt = kStages * kStageBytes;
  static constexpr int kFactors = kKeysAt + 2 * kK * kKOperand;
  static constexpr int kMeta = kFactors + kFactorRing * kFactorBytes;
  static constexpr int kWords = kMeta + kMetaRing * kMetaInts * 4;
  static constexpr int kBar = (kWords + (kScanWords + 8) * 4 + 7) / 8 * 8;
  static constexpr int kNumBars = 2 * kStages + 2 * kMetaRing + 2 * kK + 10 + 2 * kFactorRing;
  static constexpr int kTmemSlot = kBar + kNumBars * 8;
  static constexpr int kBytes = kTmemSlot + 16;
};
static_assert(Layout<128>::kBytes <= 227 * 1024 && Layout<64>::kBytes <= 227 * 1024, "shared memory per CTA");

template <int D>
struct Bars {
  using L = Layout<D>;
  uint32_t base;
  __device__ uint32_t at(int i) const { return base + 8 * i; }
  __device__ uint32_t q_full(int s) const { return at(s); }                                   // bytes
  __device__ uint32_t q_empty(int s) const { return at(L::kStages + s); }                     // 2 commits
  __device__ uint32_t meta_full(int s) const { return at(2 * L::kStages + s); }               // 1
  __device__ uint32_t meta_empty(int s) const { return at(2 * L::kStages + kMetaRing + s); }  // 14 warps
  __device__ uint32_t k_full(int s) const { return at(2 * L::kStages + 2 * kMetaRing + s); }  // 4 warps
  __device__ uint32_t k_empty(int s) const { return at(2 * L::kStages + 2 * kMetaRing + L::kK + s); }  // 2 commits
  // of operand w, tile i of S^T
  __device__ uint32_t s_full(int w, int i) const { return at(2 * L::kStages + 2 * kMetaRing + 2 * L::kK + 2 * w + i); }  // commit
  __device__ uint32_t s_empty(int w, int i) const { return s_full(w, i) + 32; }  // 4 warps
  __device__ uint32_t sums(int w) const { return s_full(0, 0) + 64 + 8 * w; }    // 4 warps
  __device__ uint32_t c_full(int i) const { return s_full(0, 0) + 80 + 8 * i; }                       // bytes
  __device__ uint32_t c_empty(int i) const { return s_full(0, 0) + 80 + 8 * (kFactorRing + i); }  // 8 warps
};

__host__ __device__ constexpr uint32_t idesc_f16(int M, int N) {
  return (1u << 4) | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}

// cache_wait whose first tries do not read the clock.
__device__ __forceinline__ bool wait_for(uint32_t bar, uint32_t parity, int32_t* status) {
  return mbar_test_wait(bar, parity) || mbar_try_wait(bar, parity) || cache_wait_slow(bar, parity, status);
}

// ---------------------------------------------------------------- row tiles
// One CTA a tile: 128 rows r = t G + g as fp16 in two (d = 128) or one blocks of 64
// columns, swizzled, then the rows' factors and -LSE in log2 units. Rows behind the last are
// zero with -LSE = -inf, and so are those that saw nothing; a row whose LSE is NaN counts
// as one whose query is.
template <int D>
__global__ void __launch_bounds__(256) weights_tiles_kernel(const __grid_constant__ WeightsParams wp,
                                                            const __grid_constant__ Geometry geo, const int RT) {
  constexpr int kUnits16 = D / 8;               // 16-byte pieces of a row
  constexpr int kPass = 256 / kUnits16;         // rows at a time
  const CacheFwdParams& p = wp.f;
  const int seg = blockIdx.x / RT, tile = blockIdx.x - seg * RT;
  const int b = geo.by_Hk.div(seg), hk = seg - b * p.c.Hk;
  const RowTile r = row_tile(p, geo, b, 0, false);
  const int rows = geo.G * r.live;
  if (tile * kTileRows >= rows) return;
  allow_next();
  const int u = threadIdx.x % kUnits16, r0 = threadIdx.x / kUnits16;
  uint8_t* dst = wp.tiles + static_cast<size_t>(blockIdx.x) * Layout<D>::kTileBytes;
  float* factors = reinterpret_cast<float*>(dst + D * 256);
  uint4 x[kTileRows / kPass];
  float l[kTileRows / kPass];
#pragma unroll
  for (int i = 0; i < kTileRows / kPass; ++i) {
    const int rr = tile * kTileRows + r0 + i * kPass;
    const int tok = geo.by_G.div(rr), h = hk * geo.G + rr - tok * geo.G;
    x[i] = make_uint4(0u, 0u, 0u, 0u);
    l[i] = -INFINITY;
    if (rr < rows) {
      x[i] = *reinterpret_cast<const uint4*>(p.q + b * p.qs[0] + h * p.qs[1] + tok * p.qs[2] + 8 * u);
      l[i] = wp.lse[(static_cast<size_t>(b) * p.H + h) * p.N + tok];
    }
  }
  // exponents of the rows' largest elements; the tile's largest, and its smallest from 255 down
  uint32_t top[kTileRows / kPass];
  __shared__ uint32_t ends[2];
  if (threadIdx.x < 2) ends[threadIdx.x] = 0;
  __syncthreads();
  uint32_t hi = 0, lo = 0;
#pragma unroll
  for (int i = 0; i < kTileRows / kPass; ++i) {
    const uint32_t mk = 0x7fff7fffu;
    const uint32_t a = __vmaxu2(__vmaxu2(x[i].x & mk, x[i].y & mk), __vmaxu2(x[i].z & mk, x[i].w & mk));
    uint32_t t = max(a & 0xffffu, a >> 16);
#pragma unroll
    for (int o = kUnits16 / 2; o > 0; o >>= 1) t = max(t, __shfl_xor_sync(0xffffffffu, t, o));
    top[i] = t;
    if (t != 0 && t < 0x7f80u) hi = max(hi, t >> 7), lo = max(lo, 255u - (t >> 7));
  }
  hi = __reduce_max_sync(0xffffffffu, hi);
  lo = __reduce_max_sync(0xffffffffu, lo);
  if ((threadIdx.x & 31) == 0) {
    atomicMax(&ends[0], hi);
    atomicMax(&ends[1], lo);
  }
  __syncthreads();
  // One power of two for all rows where they are within 2^kNear of the largest: fp16 then
  // holds their elements down to 2^-(30 - kNear) of a row's largest to the bit, and smaller
  // ones to 2^-(39 - kNear) of it.
  const bool near = ends[0] != 0 && ends[0] + ends[1] <= 255u + kNear;
#pragma unroll
  for (int i = 0; i < kTileRows / kPass; ++i) {
    const int row = r0 + i * kPass;
    const bool bad = top[i] >= 0x7f80u || isnan(l[i]);
    // the largest element goes to [2^14, 2^15)
    auto lift = [](uint32_t e) { return min(14 - (static_cast<int>(e) - 127), 126); };
    const int up = near ? lift(ends[0]) : top[i] == 0 || bad ? 0 : lift(top[i] >> 7);
    const float f = bad ? __int_as_float(0x7fffffff) : __int_as_float((up + 127) << 23);
    const uint32_t v[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
    uint32_t y[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      y[j] = pack_f16x2(__uint_as_float(v[j] << 16) * f, __uint_as_float(v[j] & 0xffff0000u) * f);
    *reinterpret_cast<uint4*>(dst + (u >> 3) * 16384 + sw128_offset(row, u & 7)) = make_uint4(y[0], y[1], y[2], y[3]);
    if (u == 0) {
      // (the second is below zero where the first is all rows')
      factors[row] = near && row == 1 ? -1.f : p.scale_log2 * __int_as_float((127 - up) << 23);
      factors[kTileRows + row] = isnan(l[i]) ? 0.f : l[i] == -INFINITY ? -INFINITY : l[i] * -1.4426950408889634f;
    }
  }
}

// ---------------------------------------------------------------- keys
// Bits [lo, hi) of 64, either outside [0, 64] too.
__device__ __forceinline__ uint64_t bit_range(int lo, int hi) {
  lo = min(max(lo, 0), 64);
  hi = min(max(hi, 0), 64);
  const uint64_t below_hi = hi == 64 ? ~0ull : (1ull << hi) - 1ull, below_lo = lo == 64 ? ~0ull : (1ull << lo) - 1ull;
  return below_hi & ~below_lo;
}

// A thread's key: which rows see it.
struct Key {
  int page, j;      // page -1: none
  int lo, hi;       // rows [lo, hi), without
  int a0, b0, a1, b1;  // [a0, b0) and [a1, b1)
  float ks;
  bool special;     // seen row by row, or of a scale beyond 2^90
};

// Rows whose position lies in [s, e), of the sequence's `live` tokens.
__device__ __forceinline__ void row_range(int s, int e, const RowTile& r, int G, int& a, int& b) {
  const long long lo = min(max(static_cast<long long>(s) - r.shift, 0LL), static_cast<long long>(r.live));
  const long long hi = min(max(static_cast<long long>(e) - r.shift, 0LL), static_cast<long long>(r.live));
  a = static_cast<int>(lo) * G;
  b = static_cast<int>(hi) * G;
}

template <bool kVec>
__device__ __forceinline__ Key key_of(const CacheFwdParams& p, const Geometry& geo, const RowTile& r, int b, int hk,
                                      const int* m, int x, int slot) {
  Key k;
  k.page = m[kPg + x];
  k.ks = __int_as_float(m[kKs + x]);
  k.j = m[kJ0 + x] + slot;
  const int cut = m[kCutWord + x];
  const bool there = k.page >= 0 && k.j < r.len;
  k.hi = there ? geo.G * r.live : 0;
  k.lo = p.mask.causal ? max(k.j - r.shift, 0) * geo.G : 0;
  if (k.j - r.shift >= r.live && p.mask.causal) k.lo = k.hi;  // (no product past 32 bits)
  k.a0 = k.b0 = k.a1 = k.b1 = 0;
  k.special = (cut & 2) != 0;
  if constexpr (kVec) {
    if ((cut & 1) && there) {
      if (geo.classes != p.mask.Hm) {
        k.special = true;
      } else {
        const size_t at = (static_cast<size_t>(b) * p.mask.Hm + mask_class(p, geo, hk)) *
                              static_cast<size_t>(p.max_pages * kPage) + k.j;
        if (p.mask.lts) row_range(p.mask.lts[at], p.mask.lte[at], r, geo.G, k.a0, k.b0);
        if (p.mask.uts) row_range(p.mask.uts[at], p.mask.ute[at], r, geo.G, k.a1, k.b1);
      }
    }
  }
  return k;
}
// Row from which on all see the key, as far as causality goes; INT_MAX where that is not all.
__device__ __forceinline__ int seen_from(const Key& k) {
  return k.special || k.b0 > k.a0 || k.b1 > k.a1 ? 0x7fffffff : k.lo;
}
// Whether all rows [u0, u1) see the key (rows behind the last may).
__device__ __forceinline__ bool sees_all(const Key& k, int u0, int u1, int rows) {
  return !k.special && k.lo <= u0 && k.hi >= min(u1, rows) && (k.b0 <= u0 || k.a0 >= u1 || k.a0 >= k.b0) &&
         (k.b1 <= u0 || k.a1 >= u1 || k.a1 >= k.b1);
}
// Bit i: row u0 + i sees the key.
template <bool kVec>
__device__ __noinline__ uint64_t seen_bits(const CacheFwdParams& p, const Geometry& geo, const RowTile& r, int b,
                                           int hk, const Key k, int u0) {
  uint64_t see = bit_range(k.lo - u0, k.hi - u0) & ~bit_range(k.a0 - u0, k.b0 - u0) & ~bit_range(k.a1 - u0, k.b1 - u0);
  if constexpr (kVec) {
    if (k.special && geo.classes != p.mask.Hm && see != 0) {
      // heads of the group have masks of their own
      for (int i = 0; i < kHalf; ++i) {
        if (!(see >> i & 1ull)) continue;
        const int rr = u0 + i, tok = geo.by_G.div(rr), h = hk * geo.G + rr - tok * geo.G, pos = r.shift + tok;
        const size_t at = (static_cast<size_t>(b) * p.mask.Hm + geo.by_mask.div(h)) *
                              static_cast<size_t>(p.max_pages * kPage) + k.j;
        bool hid = false;
        if (p.mask.lts) hid |= p.mask.lts[at] <= pos && pos < p.mask.lte[at];
        if (p.mask.uts) hid |= p.mask.uts[at] <= pos && pos < p.mask.ute[at];
        if (hid) see &= ~(1ull << i);
      }
    }
  }
  return see;
}

template <int D, bool kVec>
__global__ void __launch_bounds__(kThreads, 1) cache_weights_rows_kernel(const __grid_constant__ WeightsParams wp,
                                                                         const __grid_constant__ Geometry geo,
                                                                         const int RT) {
  using L = Layout<D>;
  const CacheFwdParams& p = wp.f;
  extern __shared__ __align__(1024) uint8_t smem[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int nseg = p.B * p.c.Hk;
  if ((smem_u32(smem) & 1023u) != 0) {
    if (tid == 0) record_failure(p.status, kStatusLayout, kSiteCacheWait);
    return;
  }
  const Bars<D> bar{smem_u32(smem + L::kBar)};
  int* words = reinterpret_cast<int*>(smem + L::kWords);
  int* found = words + kScanWords;  // segment, item of it
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kTmemSlot);
  const int* meta = reinterpret_cast<const int*>(smem + L::kMeta);

  if (warp == 13) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  if (tid < L::kNumBars) {
    const int i = tid;
    int n = 1;
    if (i >= L::kStages && i < 2 * L::kStages) n = 2;
    const int m = i - 2 * L::kStages;
    if (m >= kMetaRing && m < 2 * kMetaRing) n = 14;
    const int k = m - 2 * kMetaRing;
    if (k >= 0 && k < 2 * L::kK) n = k < L::kK ? 4 : 2;
    const int x = k - 2 * L::kK;
    if (x >= 4 && x < 10) n = 4;
    if (x >= 10 + kFactorRing) n = 8;
    mbar_init(bar.at(i), n);
    fence_barrier_init();
  }
  // The kernel before (with a mask: the classification) may still run up to here. Its results
  // are the lists of pages with a mask, the row tiles without one.
  if (kVec) wait_for_previous();
  // the line: items of all segments, each `parts` long; this CTA's run
  auto items = [&](int s) { return (line_pages<kVec>(p, geo, s) + 3) >> 2; };
  const int each = (nseg + kThreads - 1) / kThreads;
  const int seg_lo = min(tid * each, nseg), seg_hi = min(seg_lo + each, nseg);
  int mine = 0;
  for (int s = seg_lo; s < seg_hi; ++s) mine += items(s);
  int total;
  const int before = block_before<kThreads / 32>(mine, words, total);
  const int grid = static_cast<int>(gridDim.x);
  // enough parts that a run is 32 of them or more
  const int parts = total == 0 || total >= kPartsRun * grid ? 1 : min(RT, (kPartsRun * grid + total - 1) / total);
  const long long line = static_cast<long long>(total) * parts;
  const int run = static_cast<int>((line + grid - 1) / grid);
  const long long run_lo = min(static_cast<long long>(run) * blockIdx.x, line), run_hi = min(run_lo + run, line);
  const int item_lo = static_cast<int>(run_lo / parts);
  const int item_hi = static_cast<int>((run_hi + parts - 1) / parts);
  if (run_lo < run_hi && before <= item_lo && item_lo < before + mine) {
    int s = seg_lo, at = before, n;
    while (item_lo >= at + (n = items(s)) && s + 1 < seg_hi) at += n, ++s;
    found[0] = s;
    found[1] = item_lo - at;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  auto col_s = [&](int w, int i) { return tmem + 256u * static_cast<uint32_t>(w) + 128u * static_cast<uint32_t>(i); };

  if (warp == 12) {
    // ------------------------------------------------------------ run, pages, row tiles
    int left = run_lo < run_hi ? item_hi - item_lo : 0, item = item_lo;
    int seg = left > 0 ? found[0] : 0, k = left > 0 ? found[1] : 0;
    int piece = 0, tq = 0;
    if (!kVec) wait_for_previous();
    bool ok = true;
    while (ok && left > 0) {
      int my_seg, my_k, my_n;
      const int avail = next_units(seg, k, nseg, min(32, left), items, my_seg, my_k, my_n);
      int m[kMetaInts];
#pragma unroll
      for (int i = 0; i < kMetaInts; ++i) m[i] = 0;
      if (lane < avail) {
        const int b = geo.by_Hk.div(my_seg), hk = my_seg - b * p.c.Hk;
        const RowTile r = row_tile(p, geo, b, 0, true);
        const int pages = line_pages<kVec>(p, geo, my_seg), rows = geo.G * r.live;
        int first = r.len;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          m[kPg + x] = -1;
          if (4 * my_k + x >= pages) continue;
          int cut;
          const int logical = page_on_line<kVec>(p, geo, b, hk, 0, 4 * my_k + x, cut);
          const int pg = p.table[static_cast<size_t>(b) * p.max_pages + logical];
          if (pg < 0 || pg >= p.c.pages) {
            record_failure(p.status, kStatusPage, kSiteCachePage);
            continue;
          }
          const float ks = p.c.kscale[static_cast<size_t>(pg) * p.c.Hk + hk];
          m[kPg + x] = pg;
          m[kJ0 + x] = logical * kPage;
          m[kKs + x] = no_scales(ks, 0.f) ? 0x7fffffff : __float_as_int(ks);
          m[kCutWord + x] = cut | (ks > 0x1p90f ? 2 : 0);
          first = min(first, logical * kPage);
        }
        // row tiles that may see a key, cut into parts
        const int tile_hi = (rows + kTileRows - 1) / kTileRows;
        int tile_lo = 0;
        if (p.mask.causal && first > r.shift) tile_lo = first - r.shift >= r.live ? tile_hi : (first - r.shift) * geo.G / kTileRows;
        const long long lo = static_cast<long long>(item + lane) * parts;
        const int pa = static_cast<int>(max(run_lo, lo) - lo), pb = static_cast<int>(min(run_hi, lo + parts) - lo);
        const int n = tile_hi - tile_lo;
        const int t0 = static_cast<int>(static_cast<long long>(n) * pa / parts), t1 = static_cast<int>(static_cast<long long>(n) * pb / parts);
        m[kFlags] = (pa == 0 && pb == parts ? kWhole : 0) | (pa == 0 ? kTail : 0);
        m[kSeg] = my_seg;
        m[kLen] = r.len;
        m[kLive] = r.live;
        m[kTile0] = tile_lo + t0;
        m[kTiles] = t1 - t0;
        m[kCta0] = static_cast<int>(lo / run);
        m[kPieces] = static_cast<int>((lo + parts - 1) / run) - m[kCta0] + 1;
      }
      for (int t = 0; ok && t < avail; ++t, ++piece) {
        const int ring = piece % kMetaRing;
        if (piece >= kMetaRing) ok = __all_sync(0xffffffffu, wait_for(bar.meta_empty(ring), (piece / kMetaRing - 1) & 1, p.status));
        if (!ok) break;
        if (lane == t) {
          int4* at = reinterpret_cast<int4*>(smem + L::kMeta) + ring * (kMetaInts / 4);
#pragma unroll
          for (int i = 0; i < 6; ++i) at[i] = make_int4(m[4 * i], m[4 * i + 1], m[4 * i + 2], m[4 * i + 3]);
          mbar_arrive(bar.meta_full(ring));
        }
        const int sg = __shfl_sync(0xffffffffu, m[kSeg], t), tile0 = __shfl_sync(0xffffffffu, m[kTile0], t);
        const int tiles = __shfl_sync(0xffffffffu, m[kTiles], t);
        for (int i = 0; ok && i < tiles; ++i, ++tq) {
          const int st = tq % L::kStages;
          const int ci = tq % kFactorRing;
          if (tq >= L::kStages) ok = wait_for(bar.q_empty(st), (tq / L::kStages - 1) & 1, p.status);
          if (ok && tq >= kFactorRing) ok = wait_for(bar.c_empty(ci), (tq / kFactorRing - 1) & 1, p.status);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          if (lane == 0) {
            const uint8_t* src = wp.tiles + (static_cast<size_t>(sg) * RT + tile0 + i) * L::kTileBytes;
            mbar_arrive_expect_tx(bar.q_full(st), L::kStageBytes);
            bulk_load(smem_u32(smem + st * L::kStageBytes), src, L::kStageBytes, bar.q_full(st));
            mbar_arrive_expect_tx(bar.c_full(ci), kFactorBytes);
            bulk_load(smem_u32(smem + L::kFactors + ci * kFactorBytes), src + L::kStageBytes, kFactorBytes, bar.c_full(ci));
          }
        }
      }
      left -= avail;
      item += avail;
      if (avail > 0) {
        seg = __shfl_sync(0xffffffffu, my_seg, avail - 1);
        k = __shfl_sync(0xffffffffu, my_k, avail - 1) + 1;
      } else {
        seg += 32;
        k = 0;
        if (seg >= nseg) ok = lengths_moved(p.status);
      }
    }
    if (ok && piece >= kMetaRing) ok = wait_for(bar.meta_empty(piece % kMetaRing), (piece / kMetaRing - 1) & 1, p.status);
    if (lane == 0) {
      if (ok) {
        (reinterpret_cast<int*>(smem + L::kMeta) + (piece % kMetaRing) * kMetaInts)[kFlags] = kEnd;
        mbar_arrive(bar.meta_full(piece % kMetaRing));
      } else {
        // copies in flight land before the CTA's shared memory is given up
        for (int i = max(0, tq - L::kStages); i < tq; ++i)
          mbar_wait_for(bar.q_full(i % L::kStages), (i / L::kStages) & 1, nullptr, 1000000ull);
        for (int i = max(0, tq - kFactorRing); i < tq; ++i)
          mbar_wait_for(bar.c_full(i % kFactorRing), (i / kFactorRing) & 1, nullptr, 1000000ull);
      }
    }
  } else if (warp >= 13) {
    // ------------------------------------------------------------ products of operand w
    if (lane == 0) {
      const int w = warp - 13;
      const uint64_t dq = sdesc_sw128(smem_u32(smem), 16, 1024);
      const uint64_t dk = sdesc_sw128(smem_u32(smem + L::kKeysAt + w * L::kKOperand), 16, 1024);
      int st = 0, turn = 0, t = 0, kb = 0, kturn = 0;  // stage of the ring and its turns, tile, K
      bool ok = true;
      for (int piece = 0; ok; ++piece) {
        const int ring = piece % kMetaRing;
        if (!wait_for(bar.meta_full(ring), (piece / kMetaRing) & 1, p.status)) break;
        const int* m = meta + ring * kMetaInts;
        if (m[kFlags] & kEnd) break;
        const int tile0 = m[kTile0], tiles = m[kTiles], rows = geo.G * m[kLive];
        mbar_arrive(bar.meta_empty(ring));
        if (tiles == 0) continue;
        ok = wait_for(bar.k_full(kb), kturn & 1, p.status);
        const uint64_t kd = dk + static_cast<uint64_t>((2 * kb * L::kKOperand) >> 4);
        for (int i = 0; ok && i < tiles; ++i, ++t) {
          ok = wait_for(bar.q_full(st), turn & 1, p.status) &&
               (t < 2 || wait_for(bar.s_empty(w, t & 1), ((t >> 1) - 1) & 1, p.status));
          if (!ok) break;
          tc_fence_after();
          const uint32_t idesc = idesc_f16(128, rows - (tile0 + i) * kTileRows > kHalf ? 128 : 64);
          const uint64_t qd = dq + static_cast<uint64_t>((st * L::kStageBytes) >> 4);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint64_t off = static_cast<uint64_t>(((kk >> 2) * 16384 + (kk & 3) * 32) >> 4);
            mma_ss(col_s(w, t & 1), kd + off, qd + off, idesc, kk > 0);
          }
          mma_commit(bar.s_full(w, t & 1));
          mma_commit(bar.q_empty(st));
          if (++st == L::kStages) st = 0, ++turn;
        }
        if (ok) mma_commit(bar.k_empty(kb));
        if (++kb == L::kK) kb = 0, ++kturn;
      }
    }
  } else if (warp >= 8) {
    // ------------------------------------------------------------ conversion
    // A warp has 32 keys of each operand, a thread 16 codes of every kRows-th of them: whole
    // rows side by side (with a key a thread a load touched 32 of them, and the lookups
    // bound calls with few rows: 40 rows at 16 x 16384, 4 heads of 128, took 45.6 us and take 37.6).
    constexpr int kRows = 512 / D, kLanes = 32 / kRows;
    const int key0 = (warp - 8) * 32 + lane / kLanes, chunk = lane % kLanes;
    int piece = 0, kc = 0;
    bool ok = true;
    struct Item {
      int page[2], hk;
      bool some;  // not the end
    };
    // The next piece that has row tiles. `wait` false: if it is there already.
    auto next_item = [&](bool wait) {
      Item x = {};
      while (ok) {
        const int ring = piece % kMetaRing, phase = (piece / kMetaRing) & 1;
        if (!wait && !__all_sync(0xffffffffu, mbar_test_wait(bar.meta_full(ring), phase))) break;
        ok = __all_sync(0xffffffffu, wait_for(bar.meta_full(ring), phase, p.status));
        if (!ok) break;
        const int* m = meta + ring * kMetaInts;
        if (m[kFlags] & kEnd) break;
        const int tiles = m[kTiles], seg = m[kSeg];
        x.page[0] = m[kPg + ((warp - 8) >> 1)];
        x.page[1] = m[kPg + 2 + ((warp - 8) >> 1)];
        __syncwarp();
        if (lane == 0) mbar_arrive(bar.meta_empty(ring));
        ++piece;
        if (tiles == 0) continue;
        x.hk = seg - geo.by_Hk.div(seg) * p.c.Hk;
        x.some = true;
        break;
      }
      return x;
    };
    auto load = [&](const Item& x, int s, uint4 (&w)[D / 16]) {
      const uint8_t* src = p.c.k8 + (static_cast<size_t>(max(x.page[s], 0)) * p.c.Hk + x.hk) * (kPage * D) + (key0 & 63) * D + 16 * chunk;
#pragma unroll
      for (int i = 0; i < D / 16; ++i)
        w[i] = x.page[s] < 0 ? make_uint4(0u, 0u, 0u, 0u) : *reinterpret_cast<const uint4*>(src + i * kRows * D);
    };
    auto convert = [&](int kb, int s, const uint4 (&w)[D / 16]) {
      const uint32_t to = smem_u32(smem + L::kKeysAt + (2 * kb + s) * L::kKOperand) + (chunk >> 2) * 16384;
      // (the upper half's units in another order, for the banks)
      const uint32_t first = (2 * chunk + (chunk >> 2)) & 7, second = first ^ 1;
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        uint32_t h[8];
#pragma unroll
        for (int u = 0; u < 4; ++u) codes_to_f16(word(w[i], u), h[2 * u], h[2 * u + 1]);
        const uint32_t row = key0 + i * kRows;
        const bool up = chunk >= 4;
        st_shared_v4(to + sw128_offset(row, first), up ? h[4] : h[0], up ? h[5] : h[1], up ? h[6] : h[2], up ? h[7] : h[3]);
        st_shared_v4(to + sw128_offset(row, second), up ? h[0] : h[4], up ? h[1] : h[5], up ? h[2] : h[6], up ? h[3] : h[7]);
      }
    };
    uint4 w0[D / 16], w1[D / 16];
    Item now = next_item(true);
    if (now.some) load(now, 0, w0);
    for (; ok && now.some; ++kc) {
      const int kb = kc % L::kK;
      load(now, 1, w1);
      if (kc >= L::kK) ok = __all_sync(0xffffffffu, wait_for(bar.k_empty(kb), (kc / L::kK - 1) & 1, p.status));
      if (!ok) break;
      convert(kb, 0, w0);
      // the next item's codes are on their way while these are converted, if it is known
      Item then = next_item(false);
      if (then.some) load(then, 0, w0);
      convert(kb, 1, w1);
      fence_proxy_async_smem();  // the operands are read by the tensor cores
      __syncwarp();
      if (lane == 0) mbar_arrive(bar.k_full(kb));
      if (!then.some) {
        then = next_item(true);
        if (then.some) load(then, 0, w0);
      }
      now = then;
    }
  } else {
    // ------------------------------------------------------------ weights
    const int w = warp >> 2, key = (warp & 3) * 32 + lane;
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    int ci = 0, cturn = 0, t = 0, syncs = 0;
    bool ok = true;
    for (int piece = 0; ok; ++piece) {
      const int ring = piece % kMetaRing;
      ok = __all_sync(0xffffffffu, wait_for(bar.meta_full(ring), (piece / kMetaRing) & 1, p.status));
      if (!ok) break;
      const int* m = meta + ring * kMetaInts;
      const int flags = m[kFlags];
      if (flags & kEnd) break;
      const int tile0 = m[kTile0], tiles = m[kTiles], seg = m[kSeg], cta0 = m[kCta0], pieces = m[kPieces];
      const int b = geo.by_Hk.div(seg), hk = seg - b * p.c.Hk;
      RowTile r = {};
      r.len = m[kLen], r.live = m[kLive], r.shift = r.len - r.live;
      const int rows = geo.G * r.live;
      const Key k = key_of<kVec>(p, geo, r, b, hk, m, 2 * w + (key >> 6), key & 63);
      __syncwarp();
      if (lane == 0) mbar_arrive(bar.meta_empty(ring));
      const bool there = k.page >= 0 && k.j < r.len;
      float* const at = wp.weights + (static_cast<size_t>(max(k.page, 0)) * p.c.Hk + hk) * kPage + (key & 63);
      float old = 0.f;
      if (there && k.j < first_new(wp, b, r)) old = *at;
      float sum = 0.f;
      // rows from which on nothing of this warp is masked (what keys that are not there get is
      // dropped)
      const int all_from = __reduce_max_sync(0xffffffffu, there ? seen_from(k) : 0);

      for (int i = 0; i < tiles; ++i, ++t) {
        const int row0 = (tile0 + i) * kTileRows, halves = rows - row0 > kHalf ? 2 : 1;
        // (both at once: a test that succeeds takes 100 cycles)
        const bool now = mbar_test_wait(bar.c_full(ci), cturn & 1), done = mbar_test_wait(bar.s_full(w, t & 1), (t >> 1) & 1);
        if (!__all_sync(0xffffffffu, now && done)) {
          ok = __all_sync(0xffffffffu, wait_for(bar.c_full(ci), cturn & 1, p.status) &&
                                           wait_for(bar.s_full(w, t & 1), (t >> 1) & 1, p.status));
          if (!ok) break;
        }
        tc_fence_after();
        const float* fac = reinterpret_cast<const float*>(smem + L::kFactors + ci * kFactorBytes);
        const float2 first = *reinterpret_cast<const float2*>(fac);
        const bool one = first.y < 0.f;
        const float c1 = first.x * k.ks;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (h == halves) break;
          const float4* nl = reinterpret_cast<const float4*>(fac + kTileRows + h * kHalf);
          float4 ahead[4];
#pragma unroll
          for (int q = 0; q < 4; ++q) ahead[q] = nl[q];
          uint32_t sv[64];
          tmem_ld64(col_s(w, t & 1) + lane_base + 64 * h, col_s(w, t & 1) + lane_base + 64 * h + 32, sv);
          if (h + 1 == halves) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar.s_empty(w, t & 1));
          }
          const int u0 = row0 + h * kHalf;
          const bool plain = u0 >= all_from || (kVec && __all_sync(0xffffffffu, !there || sees_all(k, u0, u0 + kHalf, rows)));
          uint64_t acc = f2_make(0.f, 0.f);
          if (plain && one && first.x <= 1.f) {
            const uint64_t c2 = f2_make(c1, c1);
#pragma unroll
            for (int q = 0; q < 16; ++q) {
              const float4 n = q < 4 ? ahead[q] : nl[q];
              const uint32_t* v = sv + 4 * q;
              float x0, x1, x2, x3;
              f2_split(f2_fma(f2_make(__uint_as_float(v[0]), __uint_as_float(v[1])), c2, f2_make(n.x, n.y)), x0, x1);
              f2_split(f2_fma(f2_make(__uint_as_float(v[2]), __uint_as_float(v[3])), c2, f2_make(n.z, n.w)), x2, x3);
              acc = f2_add(acc, f2_add(f2_make(ex2(x0), ex2(x1)), f2_make(ex2(x2), ex2(x3))));
            }
          } else {
            // a row at a time: masked, or with factors of their own
            const uint64_t see = plain ? ~0ull : seen_bits<kVec>(p, geo, r, b, hk, k, u0);
            if (__any_sync(0xffffffffu, see != 0)) {
              float part[2] = {};
#pragma unroll
              for (int q = 0; q < 64; ++q) {
                const float f = one ? first.x : fac[h * kHalf + q], v = __uint_as_float(sv[q]);
                // (a factor past fp32: a product that overflows is a score that does)
                const float cc = f * k.ks;
                const float e = ex2((isinf(cc) ? (v * f) * k.ks : v * cc) + fac[kTileRows + h * kHalf + q]);
                part[q & 1] += ((q < 32 ? static_cast<uint32_t>(see) : static_cast<uint32_t>(see >> 32)) >> (q & 31)) & 1u ? e : 0.f;
              }
              acc = f2_make(part[0], part[1]);
            }
          }
          float x0, x1;
          f2_split(acc, x0, x1);
          sum += x0 + x1;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bar.c_empty(ci));
        if (++ci == kFactorRing) ci = 0, ++cturn;
      }
      if (!ok) break;

      bool store = true;
      if (!(flags & kWhole)) {
        // this warpgroup's keys of the piece
        float* part = wp.partial + (static_cast<size_t>(blockIdx.x) * 2 + (flags & kTail ? 1 : 0)) * kKeys + 128 * w;
        part[key] = sum;
        auto meet = [&]() {  // the four warps
          __syncwarp();
          if (lane == 0) mbar_arrive(bar.sums(w));
          ok = __all_sync(0xffffffffu, wait_for(bar.sums(w), syncs & 1, p.status));
          ++syncs;
          return ok;
        };
        if (!meet()) break;
        if (key == 0) {
          int32_t* count = wp.arrived + 2 * cta0 + w;
          const bool last = atomic_add_acq_rel(count, 1) == pieces - 1;
          if (last) *count = 0;  // ready for the next call
          found[2 + w] = last;
        }
        if (!meet()) break;
        store = found[2 + w];
        if (store) {
          sum = 0.f;
          for (int i = 0; i < pieces; ++i)
            sum += __ldcg(wp.partial + (static_cast<size_t>(cta0 + i) * 2 + (i == 0 ? 1 : 0)) * kKeys + 128 * w + key);
        }
        if (!meet()) break;  // found has been read
      }
      if (store && there) *at = old + sum;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 13) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  clear_unseen<kVec>(wp, geo, static_cast<int>(blockIdx.x) * (kThreads / 32) + warp, grid * (kThreads / 32));
}

template <int D, bool kVec>
cudaError_t launch_t(const WeightsParams& p, const Geometry& geo, int num_sms, cudaStream_t s) {
  static std::atomic<uint64_t> done[4];  // devices whose kernel has its shared memory
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev > 255) return cudaErrorInvalidDevice;
  if (!(done[dev >> 6].load(std::memory_order_relaxed) >> (dev & 63) & 1)) {
    e = cudaFuncSetAttribute(cache_weights_rows_kernel<D, kVec>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             Layout<D>::kBytes);
    if (e != cudaSuccess) return e;
    done[dev >> 6].fetch_or(1ull << (dev & 63), std::memory_order_relaxed);
  }
  const int RT = weights_row_tiles(p.f.H, p.f.c.Hk, p.f.N);
  weights_tiles_kernel<D><<<static_cast<unsigned>(p.f.B) * p.f.c.Hk * RT, 256, 0, s>>>(p, geo, RT);
  e = cudaGetLastError();
  if (e == cudaSuccess && kVec) e = launch_cache_classify(p.f, geo, s);
  if (e != cudaSuccess) return e;
  const int grid = num_sms < kCacheMaxCtas ? num_sms : kCacheMaxCtas;
  return launch_overlapped(cache_weights_rows_kernel<D, kVec>, dim3(static_cast<unsigned>(grid)), kThreads,
                           Layout<D>::kBytes, s, p, geo, RT);
}

}  // namespace

cudaError_t launch_cache_weights_rows(int d, const WeightsParams& p, const Geometry& geo, int num_sms,
                                      cudaStream_t s) {
  const bool vec = p.f.mask.lts != nullptr || p.f.mask.uts != nullptr;
  if (d == 64) return vec ? launch_t<64, true>(p, geo, num_sms, s) : launch_t<64, false>(p, geo, num_sms, s);
  return vec ? launch_t<128, true>(p, geo, num_sms, s) : launch_t<128, false>(p, geo, num_sms, s);
}

}  // namespace fm
