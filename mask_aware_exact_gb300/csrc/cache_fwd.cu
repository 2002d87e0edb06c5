// Attention over the 8-bit paged cache: a few query rows per cache head against
// long sequences (one token of each running sequence, drafted tokens), where
// reading the codes once bounds the call.
//
// Rows. The G = H / Hk query heads that share a cache head and the sequence's
// query tokens form one list of rows, r = t * G + g, here one tile of 8 or 16.
// A segment is one (sequence, cache head, row tile); its work is the list of pages
// that some row of it sees.
//
// Split. All pages of all segments form one line, cut into equal runs, one run per CTA
// (one CTA per SM), whatever the lengths of the sequences; where there are CTAs enough
// each segment is cut by itself instead. A segment cut by a run border leaves partial
// results in the workspace and the CTA that finishes last adds them in order (in groups
// first, if they are many), so results do not depend on timing. Where every segment is
// short the borders move to segment ends: nothing is cut, and the imbalance costs less
// than the joins. find_run has the rules. With a column-wise mask a first kernel lists
// the pages that are visible to a row tile, and only those are on the line.
//
// One producer warp walks the run and loads pages (K codes, V codes: 64 * d bytes
// each, contiguous) with bulk copies into a ring of three slots for each of seven
// consumer warps; tile i of the run goes to warp i mod 7 (or, with many short segments,
// a segment to one warp). The warps keep separate softmax states. When a piece ends each
// leaves its state in shared memory and goes on with the next piece; the last to arrive
// adds them up. The run's last piece and the joins are added up by all warps.
//
// What bounds it. 8 rows: memory, once the cache is long (8 sequences of 131072 tokens,
// 32 / 8 heads of 128: 324 us, 6.6 TB/s, 98 % of a copy; 64 up to 8192: 115 us, 83 %, with
// 12000 of 210000 cycles before the first page and 14000 behind the last). 16 rows: the
// loop's instructions, 900 for a page and tile, of which the seven warps issue 2.2 a
// clock, eleven hardly more (16 sequences up to 16384, 32 / 4 heads of 64, 4 tokens, two
// tiles of 16 rows: 44.8 us, floor 12.4; 50 of 80 thousand cycles in the loop, 9 before
// the first page, the rest joins). Short ones: latency (one sequence of 1000 tokens: 10.9
// us, of which 4 are the way to the first page: where the run begins, page table, page,
// query).
//
// Arithmetic. Codes become fp16 (exact) and enter m16n8k16 instructions with fp32
// accumulators; tcgen05 would need 128 rows. The products are taken transposed,
// S^T = K Q^T and O^T = V^T P^T, so that keys and columns of V fill the 16 rows of
// an instruction and the query rows its 8 columns: with 8 rows nothing is wasted,
// and a code is converted once for all row groups of the tile. A query row is
// scaled by a power of two so that its largest element lies in [2^14, 2^15): fp16
// then holds every bf16 element down to 2^-30 of the largest exactly. P is rounded
// to fp16 (2^-11 relative) after scaling by the page's V scale, relative to the
// row's largest such product: a second running maximum, mv of log2(P * scale),
// beside m of the scores (mv counts from m), so that neither the weights of pages
// with small values (in l) nor the values of pages with small weights are lost. m,
// mv, l and O are fp32.
//
// Layout of a fragment. Lane = 4 g + c. The summed index of S^T is permuted so that
// a lane reads 16 consecutive codes of a key (d = 64 half + 16 c ..), the query laid
// out to match. The keys of an S^T instruction u are ordered so that after the 8x8
// transposes that turn P into the second operand a lane holds the keys 16 c + 4 u ..
// + 3, which are the codes of word u of its 16-byte load of a V column.
#include <atomic>

#include "cache_common.cuh"
#include "flashmask.h"

namespace fm {
namespace {

// With the producer 8 warps, two for each scheduler, 255 registers a thread. Eleven
// consumer warps (two slots each for 8 rows of d = 128) gave the same times for long
// sequences and up to 1.5 us more for short ones.
constexpr int kConsumers = 7;
constexpr int kThreads = 32 * (kConsumers + 1);
constexpr int kSlots = 3;                           // ring slots of a consumer warp
constexpr int kPieceRing = 2 * kConsumers + 2;      // piece descriptors: more than two groups start
constexpr int kBatch = 32 / kConsumers * kConsumers;  // tiles looked up at a time, one per lane
// Pages a run has at least: one for each consumer warp. One sequence of 2500 tokens, 8
// cache heads, at least 4 / 7 / 14 pages: 13.4 / 12.7 / 13.7 us; 6000: 16.1 / 14.4 / 13.9.
constexpr int kMinRun = kConsumers;
// Segments of at most kUncut pages, and at least this many for each CTA: every segment
// is one warp's, without states to add up. 512 sequences up to 512 tokens, 8 cache heads:
// 74 us so, 102 with a segment's pages spread over the warps; 1024 up to 100: 65, 81; 512
// up to 512, 4 tokens: 88, 179. Segments of 62 pages spread better: 225, 209.
constexpr int kAlone = 7;
constexpr float kPShift = 14.f;  // P is stored as 2^14 P
constexpr int kOnce = 4 * kConsumers, kFan = 2 * kConsumers;  // see Join

// ---------------------------------------------------------------- instructions
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_all;" ::: "memory");
}

template <int D, int NT>
struct Smem {
  static constexpr int kRows = 8 * NT;
  static constexpr int kFrags = D / 16 * NT;  // accumulator fragments (four floats a lane) of a warp
  static constexpr int kHalf = kPage * D;  // bytes of a page's K or V
  static constexpr int kRing = 0;          // [consumer][slot]
  static constexpr int kMerge = kRing + kConsumers * kSlots * kHalf;  // float4 [consumer][frag][32]
  static constexpr int kStats = kMerge + kConsumers * kRows * D * 4;  // float [consumer][3][rows]: m, mv, l
  static constexpr int kMeta = kStats + kConsumers * kRows * 3 * 4;   // int4 [consumer][slot]
  static constexpr int kPiece = kMeta + kConsumers * kSlots * 16;    // int [ring][8], see below
  static constexpr int kBars = kPiece + kPieceRing * 32;
  static constexpr int kNumBars = 2 * kConsumers * kSlots + 2 * kPieceRing + 1;
  static constexpr int kScan = kBars + kNumBars * 8;  // int [kLineWords + 20], see the kernel
  static constexpr int kBytes = kScan + (kLineWords + 20) * 4;
};
static_assert(Smem<128, 2>::kBytes <= 227 * 1024 && Smem<64, 2>::kBytes <= 227 * 1024, "shared memory per CTA");

struct Bars {
  uint32_t base;
  __device__ uint32_t full(int w, int s) const { return base + 8 * (w * kSlots + s); }
  __device__ uint32_t empty(int w, int s) const { return base + 8 * ((kConsumers + w) * kSlots + s); }
  __device__ uint32_t piece_full(int s) const { return base + 8 * (2 * kConsumers * kSlots + s); }
  __device__ uint32_t piece_empty(int s) const { return base + 8 * (2 * kConsumers * kSlots + kPieceRing + s); }
  __device__ uint32_t done() const { return base + 8 * (2 * kConsumers * kSlots + 2 * kPieceRing); }
};

// A piece descriptor, int[8]: segment, first tile in the CTA's run, tiles (0: the
// end), whole segment?, slot of its partial result, first CTA and number of the
// segment's parts.

// Floats of one partial result in the workspace: O as its fragments (float4 [frag]
// [lane]), then m, mv, l of the tile's rows.
__host__ __device__ constexpr int part_floats(int D, int rows) { return rows * D + 3 * rows; }

// Transposes an 8 x 8 matrix of 16-bit elements held as a fragment (row g, columns
// 2 c and 2 c + 1 in lane 4 g + c).
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// State of one consumer warp. A lane's rows are 8 t + 2 c + e (m, mv and l are the
// same in all lanes of a row, l once the piece has ended); acc[mt][t]: columns
// 16 mt + g (and + 8) of rows 2 c, 2 c + 1.
template <int D, int NT>
struct State {
  float acc[D / 16][NT][4];
  float m[NT][2], mv[NT][2], l[NT][2];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int n = 0; n < D / 16; ++n)
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[n][t][i] = 0.f;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        m[t][e] = kNoScore, mv[t][e] = kNoProduct;
        l[t][e] = 0.f;
      }
  }
  // Fragments to frags [frag][lane], m, mv, l of the rows to stats [3][8 NT].
  __device__ __forceinline__ void put(float4* frags, float* stats, int lane) const {
#pragma unroll
    for (int n = 0; n < D / 16; ++n)
#pragma unroll
      for (int t = 0; t < NT; ++t)
        frags[(n * NT + t) * 32 + lane] = make_float4(acc[n][t][0], acc[n][t][1], acc[n][t][2], acc[n][t][3]);
    if (lane < 4) {
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float* x = stats + 8 * t + 2 * lane + e;
          x[0] = m[t][e], x[8 * NT] = mv[t][e], x[16 * NT] = l[t][e];
        }
    }
  }
};

// Sums of states, each warp its share of the fragments: warp, warp + kConsumers, ..
// A lane looks after the statistics of row lane % kRows: of all states together in m,
// mv and (a share of) l.
template <int D, int NT>
struct FragmentSums {
  static constexpr int kRows = 8 * NT;
  static constexpr int kFrags = D / 16 * NT, kMine = (kFrags + kConsumers - 1) / kConsumers;
  static constexpr int kAtOnce = 32 / kRows, kSteps = (kConsumers + kAtOnce - 1) / kAtOnce;
  float acc[kMine][4];
  float m, mv, l;
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int q = 0; q < kMine; ++q)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[q][i] = 0.f;
    m = kNoScore, mv = kNoProduct;
    l = 0.f;
  }
  // Row of element e of this lane in the warp's fragment q.
  __device__ __forceinline__ static int row_of(int q, int e, int warp, int lane) {
    return (NT == 2 ? 8 * ((warp + kConsumers * q) & 1) : 0) + 2 * (lane & 3) + e;
  }
  // Adds n states of the merge area in order, from + k modulo kConsumers.
  __device__ __forceinline__ void add(int n, int from, const float4* merge, const float* stats, int warp, int lane) {
    auto place = [&](int k) { return from + k < kConsumers ? from + k : from + k - kConsumers; };
    // states lane / kRows, + kAtOnce, ..
    float xm[kSteps], xv[kSteps], xl[kSteps];
    float mm = m, mmv = mv;
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      const int k = lane / kRows + kAtOnce * i;
      const float* x = stats + 3 * kRows * place(min(k, n - 1)) + lane % kRows;
      xm[i] = x[0], xv[i] = x[kRows], xl[i] = k < n ? x[2 * kRows] : 0.f;
      join_maxima(mm, mmv, xm[i], xv[i]);
    }
#pragma unroll
    for (int o = kRows; o < 32; o <<= 1)
      join_maxima(mm, mmv, __shfl_xor_sync(0xffffffffu, mm, o), __shfl_xor_sync(0xffffffffu, mmv, o));
    l *= ex2(m - mm);
    const float old = ex2(mv + (m - mm) - mmv);
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      const float d = xm[i] - mm;
      l += xl[i] * ex2(d);
      xv[i] = lane / kRows + kAtOnce * i < n ? ex2(xv[i] + d - mmv) : 0.f;
    }
    m = mm;
    mv = mmv;
#pragma unroll
    for (int q = 0; q < kMine; ++q)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[q][i] *= __shfl_sync(0xffffffffu, old, row_of(q, i & 1, warp, lane));
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      if (kAtOnce * i >= n) break;
#pragma unroll
      for (int j = 0; j < kAtOnce; ++j) {
        const float4* fr = merge + place(min(kAtOnce * i + j, n - 1)) * kFrags * 32 + lane;  // times 0 behind the last
#pragma unroll
        for (int q = 0; q < kMine; ++q) {
          const float f0 = __shfl_sync(0xffffffffu, xv[i], kRows * j + row_of(q, 0, warp, lane));
          const float f1 = __shfl_sync(0xffffffffu, xv[i], kRows * j + row_of(q, 1, warp, lane));
          const float4 v = fr[min(warp + kConsumers * q, kFrags - 1) * 32];
          acc[q][0] += v.x * f0;
          acc[q][1] += v.y * f1;
          acc[q][2] += v.z * f0;
          acc[q][3] += v.w * f1;
        }
      }
    }
  }
  // The whole sum of P of the lane's row.
  __device__ __forceinline__ float sum() const {
    float x = l;
#pragma unroll
    for (int o = kRows; o < 32; o <<= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
  }
  // The sums as a state (see State::put).
  __device__ __forceinline__ void put(float4* frags, float* stats, int warp, int lane) const {
#pragma unroll
    for (int q = 0; q < kMine; ++q)
      if (warp + kConsumers * q < kFrags)
        frags[(warp + kConsumers * q) * 32 + lane] = make_float4(acc[q][0], acc[q][1], acc[q][2], acc[q][3]);
    const float x = sum();
    if (warp == 0 && lane < kRows) stats[lane] = m, stats[kRows + lane] = mv, stats[2 * kRows + lane] = x;
  }
  // O and LSE of the row tile that begins at row r0.
  __device__ __forceinline__ void store(const CacheFwdParams& p, const Geometry& geo, int b, int hk, int r0, int rows,
                                        int warp, int lane) const {
    const int g = lane >> 2, c = lane & 3;
    const float x = sum(), f = out_factor(mv, x, kPShift);
#pragma unroll
    for (int q = 0; q < kMine; ++q) {
      const int fr = warp + kConsumers * q;
      const float f0 = __shfl_sync(0xffffffffu, f, row_of(q, 0, warp, lane));
      const float f1 = __shfl_sync(0xffffffffu, f, row_of(q, 1, warp, lane));
      const int rr = r0 + 8 * (fr % NT) + g, tok = geo.by_G.div(rr), h = hk * geo.G + rr - tok * geo.G;
      uint16_t* o = p.o + b * p.os[0] + h * p.os[1] + tok * p.os[2] + 2 * c + fr / NT * 16;
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const uint32_t v = transpose8x8(pack_bf16x2(acc[q][2 * y] * f0, acc[q][2 * y + 1] * f1));
        if (rr < rows && fr < kFrags) *reinterpret_cast<uint32_t*>(o + 8 * y) = v;
      }
    }
    if (warp == 0 && lane < kRows && r0 + lane < rows) {
      const int tok = geo.by_G.div(r0 + lane), h = hk * geo.G + r0 + lane - tok * geo.G;
      p.lse[(static_cast<size_t>(b) * p.H + h) * p.N + tok] = out_lse(m, x);
    }
  }
};

// Bits of the keys at[i], at[i + 2], .. at[i + 14] (i = odd) with s <= pos < e. (Not
// inline: most pages need no look at the mask's words, and the loop stays small.)
static __device__ __noinline__ uint32_t hidden8(const int32_t* s, const int32_t* e, int pos, int odd) {
  uint32_t hid = 0;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int4 a = *reinterpret_cast<const int4*>(s + 4 * q), z = *reinterpret_cast<const int4*>(e + 4 * q);
    const int a0 = odd ? a.y : a.x, z0 = odd ? z.y : z.x, a1 = odd ? a.w : a.z, z1 = odd ? z.w : z.z;
    hid |= (static_cast<uint32_t>(a0 <= pos && pos < z0) | static_cast<uint32_t>(a1 <= pos && pos < z1) << 1) << (2 * q);
  }
  return hid;
}

template <int D, int NT, bool kVec>
__global__ void __launch_bounds__(kThreads, 1) cache_fwd_kernel(const __grid_constant__ CacheFwdParams p,
                                                                 const __grid_constant__ Geometry geo) {
  using S = Smem<D, NT>;
  constexpr int kRows = S::kRows;
  extern __shared__ __align__(1024) uint8_t smem[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int nseg = p.B * p.c.Hk * geo.RT;
  const Bars bar{smem_u32(smem + S::kBars)};
  int* scan = reinterpret_cast<int*>(smem + S::kScan);  // see the words below
  enum { kCount = kLineWords, kJobs, kMerged, kJob0, kJobInts = 8 };

  if (tid < S::kNumBars) {
    // one arrival each, but of piece_empty and done, where every consumer warp arrives
    const bool all = tid >= 2 * kConsumers * kSlots + kPieceRing;
    mbar_init(bar.base + 8 * tid, all ? kConsumers : 1);
    fence_barrier_init();
  }
  if (tid >= kCount && tid <= kMerged) scan[tid] = 0;

  const Line line = find_run<kThreads>(nseg, kMinRun, 1, scan, [&](int seg) { return pages_of<kVec>(p, geo, seg); });
  const int run = line.run, run_lo = line.lo, run_hi = line.hi;
  const bool alone = line.brief && nseg >= kAlone * static_cast<int>(gridDim.x);

  if (warp == kConsumers) {
    // ------------------------------------------------------------ producer
    int seg = line.seg, k = line.first;
    const int tiles = run_hi - run_lo;
    bool ok = true;
    // This lane's page to warp w, at positions q and q + 1 of its ring. K's copy is on its
    // way before the scales are waited for: a barrier counts bytes that land before they
    // are expected.
    auto feed_k = [&](int w, int q, int logical, size_t off) {
      const int slot = q % kSlots;
      if (q >= kSlots && !cache_wait(bar.empty(w, slot), (q / kSlots - 1) & 1, p.status)) return false;
      if (logical >= 0)
        bulk_load(smem_u32(smem + S::kRing + (w * kSlots + slot) * S::kHalf), p.c.k8 + off, S::kHalf, bar.full(w, slot));
      return true;
    };
    auto feed_v = [&](int w, int q, int logical, int cut, size_t off, float k_s, float v_s) {
      const int slot_k = q % kSlots, slot = (q + 1) % kSlots;
      *(reinterpret_cast<int4*>(smem + S::kMeta) + w * kSlots + slot_k) =
          make_int4(logical, cut | may_be_no_scales(k_s, v_s) << 1, __float_as_int(k_s), __float_as_int(v_s));
      mbar_arrive_expect_tx(bar.full(w, slot_k), logical >= 0 ? S::kHalf : 0);
      if (q + 1 >= kSlots && !cache_wait(bar.empty(w, slot), ((q + 1) / kSlots - 1) & 1, p.status)) return false;
      mbar_arrive_expect_tx(bar.full(w, slot), logical >= 0 ? S::kHalf : 0);
      if (logical >= 0)
        bulk_load(smem_u32(smem + S::kRing + (w * kSlots + slot) * S::kHalf), p.c.v8 + off, S::kHalf, bar.full(w, slot));
      return true;
    };
    int pieces = 0;  // published so far
    int done = 0;
    int issued = 0;  // tiles of warp `lane`, if segments are one warp's
    if (alone) {
      // lane w feeds warp w, whose piece entries are 2 w and 2 w + 1; a lane that has
      // issued its segment takes the next of the run
      auto units = [&](int sg) { return sg < nseg ? pages_of<kVec>(p, geo, sg) : 0; };
      int left = tiles, next = 0, my_seg = 0, my_k = 0, my_n = 0;
      int n_all = units(seg + lane);  // of segments seg .. seg + 31 (seg is nseg if the run is empty)
      bool fed = lane < kConsumers;
      while (ok && __any_sync(0xffffffffu, fed)) {
        uint32_t need = __ballot_sync(0xffffffffu, fed && my_k == my_n);
        while (need != 0 && left > 0 && seg < nseg) {
          if (next == 32) {
            seg += 32;
            next = 0;
            n_all = units(seg + lane);
          }
          const int n = __shfl_sync(0xffffffffu, n_all, next);
          if (n > 0) {
            if (lane == __ffs(need) - 1) my_seg = seg + next, my_k = 0, my_n = n;
            need &= need - 1;
            left -= n;
          }
          ++next;
        }
        if (fed) {
          const bool end = (need >> lane) & 1u;  // nothing is left: an empty piece
          if (end || my_k == 0) {
            const int e = 2 * lane + (pieces & 1);
            if (pieces >= 2) ok = cache_wait(bar.piece_empty(e), (pieces / 2 - 1) & 1, p.status);
            if (ok) {
              int* d = reinterpret_cast<int*>(smem + S::kPiece) + 8 * e;
              d[0] = my_seg, d[1] = 0, d[2] = end ? 0 : my_n, d[3] = 1;
              mbar_arrive(bar.piece_full(e));
            }
            ++pieces;
          }
          fed = !end;
        }
        if (ok && fed) {
          const int bh = geo.by_RT.div(my_seg), rt = my_seg - bh * geo.RT, b = geo.by_Hk.div(bh), hk = bh - b * p.c.Hk;
          int cut;
          const int logical = page_on_line<kVec>(p, geo, b, hk, rt, my_k, cut);
          int page = p.table[static_cast<size_t>(b) * p.max_pages + logical];
          if (page < 0 || page >= p.c.pages) {
            record_failure(p.status, kStatusPage, kSiteCachePage);
            page = -1;
          }
          const size_t ph = static_cast<size_t>(max(page, 0)) * p.c.Hk + hk;
          const float ks = p.c.kscale[ph], vs = p.c.vscale[ph];
          const int there = page < 0 ? -1 : logical;
          ok = feed_k(lane, 2 * issued, there, ph * S::kHalf) && feed_v(lane, 2 * issued, there, cut, ph * S::kHalf, ks, vs);
          ++issued;
          ++my_k;
        }
        ok = __all_sync(0xffffffffu, ok);
      }
    }
    while (!alone && ok && done < tiles) {
      // the next tiles of the run, one per lane, over the next 32 segments
      int my_seg, my_k, n_j;
      const int avail = next_units(
          seg, k, nseg, min(kBatch, tiles - done), [&](int sg) { return pages_of<kVec>(p, geo, sg); }, my_seg, my_k, n_j);
      const bool live = lane < avail;
      int page = -1, logical = 0, cut = 0;
      size_t ph = 0;
      if (live) {
        const int bh = geo.by_RT.div(my_seg), rt = my_seg - bh * geo.RT, b = geo.by_Hk.div(bh), hk = bh - b * p.c.Hk;
        logical = page_on_line<kVec>(p, geo, b, hk, rt, my_k, cut);
        page = p.table[static_cast<size_t>(b) * p.max_pages + logical];
        if (page < 0 || page >= p.c.pages) {
          record_failure(p.status, kStatusPage, kSiteCachePage);
          page = -1;
        } else {
          ph = static_cast<size_t>(page) * p.c.Hk + hk;
        }
      }
      const float ks = page >= 0 ? p.c.kscale[ph] : 0.f, vs = page >= 0 ? p.c.vscale[ph] : 1.f;
      // one tile for each consumer warp at a time, issued by as many lanes. A lane
      // waits only for slots that tiles of earlier groups leave, and for piece
      // entries of earlier groups, so the lanes never wait for one another.
      for (int base = 0; ok && base < avail; base += kConsumers) {
        const int in_group = min(kConsumers, avail - base), src = min(base + lane, 31);
        const int sg = __shfl_sync(0xffffffffu, my_seg, src), kk = __shfl_sync(0xffffffffu, my_k, src);
        const int nn = __shfl_sync(0xffffffffu, n_j, src), pg = __shfl_sync(0xffffffffu, page, src);
        const int lg = __shfl_sync(0xffffffffu, logical, src), ct = __shfl_sync(0xffffffffu, cut, src);
        const unsigned long long off =
            __shfl_sync(0xffffffffu, static_cast<unsigned long long>(ph) * S::kHalf, src);
        const int at = done + lane;  // number of the tile in the run
        const bool mine_too = lane < in_group;
        const bool starts = mine_too && (at == 0 || kk == 0);
        const uint32_t who = __ballot_sync(0xffffffffu, starts);
        if (starts) {
          const int n = pieces + __popc(who & ((1u << lane) - 1u)), e = n % kPieceRing;
          if (n >= kPieceRing) ok = cache_wait(bar.piece_empty(e), (n / kPieceRing - 1) & 1, p.status);
          if (ok) {
            const int count = min(nn - kk, tiles - at);
            const int s0 = run_lo + at - kk;  // where the segment begins on the line
            const int cta0 = s0 / run;
            int* d = reinterpret_cast<int*>(smem + S::kPiece) + 8 * e;
            d[0] = sg, d[1] = at, d[2] = count, d[3] = kk == 0 && count == nn;
            d[4] = kk == 0 ? 1 : 0, d[5] = cta0;
            d[6] = (s0 + nn - 1) / run - cta0 + 1;
            mbar_arrive(bar.piece_full(e));
          }
        }
        pieces += __popc(who);
        const int w = at % kConsumers, q = 2 * (at / kConsumers), there = pg < 0 ? -1 : lg;
        if (mine_too && ok) ok = feed_k(w, q, there, off);
        const float k_s = __shfl_sync(0xffffffffu, ks, src), v_s = __shfl_sync(0xffffffffu, vs, src);
        if (mine_too && ok) ok = feed_v(w, q, there, ct, off, k_s, v_s);
        ok = __all_sync(0xffffffffu, ok);
        done += in_group;
      }
      // the tile behind the last one taken
      if (avail > 0) {
        seg = __shfl_sync(0xffffffffu, my_seg, avail - 1);
        k = __shfl_sync(0xffffffffu, my_k, avail - 1) + 1;
      } else {
        seg += 32;
        k = 0;
        // the lengths are not those of the run's search any more
        if (seg >= nseg) ok = lengths_moved(p.status);
      }
    }
    if (!alone && ok && lane == 0) {  // the end: an empty piece
      const int e = pieces % kPieceRing;
      if (pieces >= kPieceRing) ok = cache_wait(bar.piece_empty(e), (pieces / kPieceRing - 1) & 1, p.status);
      if (ok) {
        (reinterpret_cast<int*>(smem + S::kPiece) + 8 * e)[2] = 0;
        mbar_arrive(bar.piece_full(e));
      }
    }
    if (!ok && lane < kConsumers) {
      // copies in flight land before the CTA's shared memory is given up
      const int most = alone ? 2 * issued : (done + kConsumers - 1 - lane) / kConsumers * 2;
      for (int seq = max(0, most - kSlots); seq < most; ++seq)
        mbar_wait_for(bar.full(lane, seq % kSlots), (seq / kSlots) & 1, nullptr, 1000000ull);
    }
    return;
  }

  // -------------------------------------------------------------- consumers
  const int g = lane >> 2, c = lane & 3;
  uint8_t* ring = smem + S::kRing + warp * kSlots * S::kHalf;
  float4* merge = reinterpret_cast<float4*>(smem + S::kMerge);
  float* stats = reinterpret_cast<float*>(smem + S::kStats);
  bool ok = true;
  int syncs = 0;
  // all consumer warps; false when a wait gave up
  auto sync_warps = [&]() {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar.done());
    ok = __all_sync(0xffffffffu, cache_wait(bar.done(), syncs & 1, p.status));
    ++syncs;
    return ok;
  };
  // a partial result is written, by threads that this one has met since: the last of a
  // join notes it for the end of the run, where all warps take part
  auto arrive = [&](int seg, int cta0, int part, int parts, int slot_id, int rows, bool group) {
    Join x;
    if (!part_arrives<kOnce, kFan>(p, cta0, part, parts, group, x)) return;
    int* job = scan + kJob0 + kJobInts * slot_id;
    job[0] = seg, job[1] = cta0, job[2] = parts, job[3] = rows;
    job[4] = x.first, job[5] = x.stride, job[6] = x.n, job[7] = x.last;
    atomicOr(&scan[kJobs], 1 << slot_id);
  };
  int seq = 0;      // ring position of this warp
  int merges = 0;   // pieces so far whose states were merged in shared memory

  int seg = 0, whole = 0, cta0 = 0, parts = 0, rows = 0;  // of the piece; its real rows from the sequence's start
  int last_n = 0, last_from = 0;  // the run's last piece: states in shared memory, place of the first
  for (int piece = 0; ok; ++piece) {
    const int e = alone ? 2 * warp + (piece & 1) : piece % kPieceRing;
    ok = __all_sync(0xffffffffu, cache_wait(bar.piece_full(e), (alone ? piece / 2 : piece / kPieceRing) & 1, p.status));
    if (!ok) break;
    const int* d = reinterpret_cast<const int*>(smem + S::kPiece) + 8 * e;
    const int first = d[1], count = d[2], slot_id = d[4];
    seg = d[0], whole = d[3], cta0 = d[5], parts = d[6];
    __syncwarp();
    if (lane < (alone ? kConsumers : 1)) mbar_arrive(bar.piece_empty(e));  // (one arrival for each warp)
    if (count == 0) break;
    const int writers = alone ? 1 : min(count, kConsumers);  // warps that have tiles, from first % 7 on
    const int mine = alone ? 0 : (warp - first % kConsumers + kConsumers) % kConsumers;
    const bool last = !alone && first + count == run_hi - run_lo;
    if (mine >= writers && !last) {  // on to the next piece, before the others
      merges += writers > 1;
      continue;
    }

    const int bh = geo.by_RT.div(seg), rt = seg - bh * geo.RT, b = geo.by_Hk.div(bh), hk = bh - b * p.c.Hk;
    const RowTile r = row_tile(p, geo, b, rt, lane == 0);
    rows = geo.G * r.live;
    State<D, NT> st;
    st.clear();
    if (mine < writers) {
      uint32_t qf[NT][D / 16][2];
      float crow[NT][2];
      int lim[NT][2], pos[NT][2];
      size_t mrow[NT][2];
      int all_lim = r.len;  // keys that every row of the tile sees as far as causality and length go
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        // the query row that this lane brings in, 16 elements of each half: d = 64 half + 16 c ..
        // (read whether real or not, as long as it exists: the number of real rows is
        // still on its way)
        const int rr = rt * kRows + 8 * t + g;
        const bool there = rr < geo.G * p.N, live = rr < rows;
        const int tok = geo.by_G.div(rr), h = hk * geo.G + rr - tok * geo.G;
        uint4 x[D / 64][2];
        const uint16_t* src = p.q + b * p.qs[0] + h * p.qs[1] + tok * p.qs[2] + 16 * c;
#pragma unroll
        for (int hf = 0; hf < D / 64; ++hf)
#pragma unroll
          for (int u = 0; u < 2; ++u)
            x[hf][u] = there ? *reinterpret_cast<const uint4*>(src + 64 * hf + 8 * u) : make_uint4(0u, 0u, 0u, 0u);
        uint32_t top = 0;
#pragma unroll
        for (int hf = 0; hf < D / 64; ++hf)
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            if (!live) x[hf][u] = make_uint4(0u, 0u, 0u, 0u);
            const uint32_t mk = 0x7fff7fffu;
            const uint32_t a = __vmaxu2(__vmaxu2(x[hf][u].x & mk, x[hf][u].y & mk), __vmaxu2(x[hf][u].z & mk, x[hf][u].w & mk));
            top = max(top, max(a & 0xffffu, a >> 16));
          }
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        // the largest element's exponent becomes 14; rows that are not finite become NaN
        const bool bad = top >= 0x7f80u;
        const int up = top == 0 || bad ? 0 : min(14 - (static_cast<int>(top >> 7) - 127), 126);
        const float f = bad ? __int_as_float(0x7fffffff) : __int_as_float((up + 127) << 23);
        const float back = p.scale_log2 * __int_as_float((127 - up) << 23);
#pragma unroll
        for (int hf = 0; hf < D / 64; ++hf)
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const uint4& v = x[hf][u >> 1];
            const uint32_t w0 = (u & 1) ? v.z : v.x, w1 = (u & 1) ? v.w : v.y;
            qf[t][4 * hf + u][0] = pack_f16x2(__uint_as_float(w0 << 16) * f, __uint_as_float(w0 & 0xffff0000u) * f);
            qf[t][4 * hf + u][1] = pack_f16x2(__uint_as_float(w1 << 16) * f, __uint_as_float(w1 & 0xffff0000u) * f);
          }
        // the rows whose scores this lane holds
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          crow[t][e] = __shfl_sync(0xffffffffu, back, 4 * (2 * c + e));
          const int r2 = rt * kRows + 8 * t + 2 * c + e;
          const int tok2 = geo.by_G.div(r2), h2 = hk * geo.G + r2 - tok2 * geo.G;
          pos[t][e] = r.shift + tok2;
          lim[t][e] = r2 < rows && p.mask.causal ? min(r.len, pos[t][e] + 1) : r.len;
          all_lim = crow[t][e] > 1.f ? 0 : min(all_lim, lim[t][e]);  // (the row may need score_boost)
          mrow[t][e] = kVec ? (static_cast<size_t>(b) * p.mask.Hm + geo.by_mask.div(h2)) *
                                  static_cast<size_t>(p.max_pages * kPage)
                            : 0;
        }
      }
      all_lim = __reduce_min_sync(0xffffffffu, all_lim);

      for (int left = alone ? count : (count - mine + kConsumers - 1) / kConsumers; ok && left > 0; --left) {
        const int sk = seq % kSlots, sv = (seq + 1) % kSlots;
        ok = __all_sync(0xffffffffu, cache_wait(bar.full(warp, sk), (seq / kSlots) & 1, p.status));
        if (!ok) break;
        const int4 meta = *(reinterpret_cast<const int4*>(smem + S::kMeta) + warp * kSlots + sk);
        const float lvs = log2_scale(__int_as_float(meta.w));
        const int j0 = meta.x * kPage;
        // S^T: instruction u holds the keys kb + 4 u and kb + 4 u + 2 of this lane
        const int kb = 16 * (g >> 1) + (g & 1);
        float s[4][NT][4];
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) s[u][t][i] = 0.f;
        const uint8_t* kbase = ring + sk * S::kHalf + kb * D + 16 * c;
#pragma unroll
        for (int hf = 0; hf < D / 64; ++hf) {
          uint4 w[4][2];
#pragma unroll
          for (int u = 0; u < 4; ++u)
#pragma unroll
            for (int x = 0; x < 2; ++x)
              w[u][x] = *reinterpret_cast<const uint4*>(kbase + (4 * u + 2 * x) * D + 64 * hf);
#pragma unroll
          for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              uint32_t a[4];
              codes_to_f16(word(w[u][0], k), a[0], a[2]);
              codes_to_f16(word(w[u][1], k), a[1], a[3]);
#pragma unroll
              for (int t = 0; t < NT; ++t) mma16816(s[u][t], a, qf[t][4 * hf + k][0], qf[t][4 * hf + k][1]);
            }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bar.empty(warp, sk));

        // s[u][t][2 x + e]: key kb + 4 u + 2 x, row 2 c + e; ck times it is the score in
        // log2 units
        const float kscale = __int_as_float(meta.z);
        const bool tail = meta.x < 0 || j0 + kPage > all_lim;
        // Each pass goes over all rows of the lane, so that their chains overlap; a row
        // pair's elements go through packed instructions.
        float ck[NT][2], top[NT][2];
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int e = 0; e < 2; ++e) ck[t][e] = score_factor(crow[t][e], kscale);
        if (__builtin_expect(tail || meta.y, 0)) {
          const bool none = (meta.y & 2) && no_scales(kscale, __int_as_float(meta.w));
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              // bit 2 u + x: key kb + 4 u + 2 x is visible
              const int n = meta.x < 0 ? 0 : min(max(lim[t][e] - (j0 + kb), 0), 16);
              uint32_t see = (1u << ((n + 1) >> 1)) - 1u;
              if constexpr (kVec) {
                if ((meta.y & 1) && meta.x >= 0) {
                  const size_t at = mrow[t][e] + j0 + (kb & ~1);
                  if (p.mask.lts) see &= ~hidden8(p.mask.lts + at, p.mask.lte + at, pos[t][e], g & 1);
                  if (p.mask.uts) see &= ~hidden8(p.mask.uts + at, p.mask.ute + at, pos[t][e], g & 1);
                }
              }
              const float boost = score_boost(crow[t][e], kscale, none, ck[t][e]);
#pragma unroll
              for (int u = 0; u < 4; ++u)
#pragma unroll
                for (int x = 0; x < 2; ++x)
                  s[u][t][2 * x + e] = (see >> (2 * u + x)) & 1u ? s[u][t][2 * x + e] * boost : -INFINITY;
            }
        }
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            top[t][e] = fmax3(fmax3(s[0][t][e], s[0][t][2 + e], s[1][t][e]), fmax3(s[1][t][2 + e], s[2][t][e], s[2][t][2 + e]),
                              fmaxf(s[3][t][e], s[3][t][2 + e])) *
                        ck[t][e];
#pragma unroll
        for (int o = 4; o < 32; o <<= 1)
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < 2; ++e) top[t][e] = fmaxf(top[t][e], __shfl_xor_sync(0xffffffffu, top[t][e], o));
        uint32_t pf[4][NT][2];
        bool moved = false;
        float av[NT][2], fv[NT][2];
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float m_new = fmaxf(st.m[t][e], top[t][e]), d = st.m[t][e] - m_new;
            const float mv_old = st.mv[t][e] + d, mv_new = fmaxf(mv_old, top[t][e] - m_new + lvs);
            st.l[t][e] *= ex2(d);
            av[t][e] = ex2(mv_old - mv_new);
            moved |= av[t][e] != 1.f;
            st.m[t][e] = m_new;
            st.mv[t][e] = mv_new;
            fv[t][e] = ex2(fminf(lvs - mv_new + kPShift, 126.f));
          }
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          const uint64_t c2 = f2_make(ck[t][0], ck[t][1]), nm2 = f2_make(-st.m[t][0], -st.m[t][1]);
          const uint64_t f2 = f2_make(fv[t][0], fv[t][1]);
          uint64_t l2 = f2_make(st.l[t][0], st.l[t][1]);
#pragma unroll
          for (int u = 0; u < 4; ++u)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              float x0, x1, p0, p1;
              f2_split(f2_fma(f2_make(s[u][t][2 * x], s[u][t][2 * x + 1]), c2, nm2), x0, x1);
              const uint64_t pp = f2_make(ex2(x0), ex2(x1));
              l2 = f2_add(l2, pp);
              f2_split(f2_mul(pp, f2), p0, p1);
              pf[u][t][x] = transpose8x8(pack_f16x2(p0, p1));
            }
          f2_split(l2, st.l[t][0], st.l[t][1]);
        }
        if (__builtin_expect(__any_sync(0xffffffffu, moved), 0)) {
#pragma unroll
          for (int n = 0; n < D / 16; ++n)
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
              for (int i = 0; i < 4; ++i) st.acc[n][t][i] *= av[t][i & 1];
        }

        ok = __all_sync(0xffffffffu, cache_wait(bar.full(warp, sv), ((seq + 1) / kSlots) & 1, p.status));
        if (!ok) break;
        uint8_t* vbase = ring + sv * S::kHalf + g * kPage + 16 * c;
        if (__builtin_expect(tail, 0)) {
          // codes behind the sequence's end may be anything, NaN too: they become 0, each
          // lane's where it reads them
          const int n_ok = meta.x < 0 ? 0 : min(max(r.len - (j0 + 16 * c), 0), 16);
          uint32_t keep[4];
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const int nb = min(max(n_ok - 4 * u, 0), 4);
            keep[u] = nb == 4 ? ~0u : (1u << (8 * nb)) - 1u;
          }
#pragma unroll 1
          for (int i0 = 0; i0 < D / 8; i0 += 4) {
            uint4* at = reinterpret_cast<uint4*>(vbase + 8 * i0 * kPage);
            uint4 x[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] = at[8 * i * kPage / 16];
#pragma unroll
            for (int i = 0; i < 4; ++i)
              at[8 * i * kPage / 16] = make_uint4(x[i].x & keep[0], x[i].y & keep[1], x[i].z & keep[2], x[i].w & keep[3]);
          }
          fence_proxy_async_smem();  // the next copy into the slot comes after
        }
#pragma unroll
        for (int n0 = 0; n0 < D / 16; n0 += 4) {
          uint4 w[4][2];
#pragma unroll
          for (int n = 0; n < 4; ++n)
#pragma unroll
            for (int x = 0; x < 2; ++x)
              w[n][x] = *reinterpret_cast<const uint4*>(vbase + (16 * (n0 + n) + 8 * x) * kPage);
#pragma unroll
          for (int u = 0; u < 4; ++u)
#pragma unroll
            for (int n = 0; n < 4; ++n) {
              uint32_t a[4];
              codes_to_f16(word(w[n][0], u) , a[0], a[2]);
              codes_to_f16(word(w[n][1], u) , a[1], a[3]);
#pragma unroll
              for (int t = 0; t < NT; ++t) mma16816(st.acc[n0 + n][t], a, pf[u][t][0], pf[u][t][1]);
            }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bar.empty(warp, sv));
        seq += 2;
      }
      if (!ok) break;
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) st.l[t][e] += __shfl_xor_sync(0xffffffffu, st.l[t][e], o);
    }

    if (last) {
      // the run's last piece is added up below
      ok = __all_sync(0xffffffffu, count_wait(&scan[kMerged], merges, p.status));
      if (mine < writers) st.put(merge + warp * S::kFrags * 32, stats + 3 * kRows * warp, lane);
      last_n = writers;
      last_from = first % kConsumers;
      break;
    }
    if (writers > 1) {
      // leave the state, once the pieces before have been added up
      ok = __all_sync(0xffffffffu, count_wait(&scan[kMerged], merges, p.status));
      ++merges;
      if (!ok) break;
      st.put(merge + warp * S::kFrags * 32, stats + 3 * kRows * warp, lane);
      __threadfence_block();
      __syncwarp();
      int came = 0;
      if (lane == 0) came = atomicAdd(&scan[kCount], 1);
      if (__shfl_sync(0xffffffffu, came, 0) != writers - 1) continue;
      __threadfence_block();
      // the last warp adds the states up, in the order of their first tiles
      st.clear();
      for (int k = 0; k < writers; ++k) {
        const float* x = stats + 3 * kRows * ((first + k) % kConsumers) + 2 * c;
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int e = 0; e < 2; ++e) join_maxima(st.m[t][e], st.mv[t][e], x[8 * t + e], x[kRows + 8 * t + e]);
      }
      for (int k = 0; k < writers; ++k) {
        const int w = (first + k) % kConsumers;
        const float* x = stats + 3 * kRows * w + 2 * c;
        float f[NT][2];
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float d = x[8 * t + e] - st.m[t][e];
            st.l[t][e] += x[2 * kRows + 8 * t + e] * ex2(d);
            f[t][e] = ex2(x[kRows + 8 * t + e] + d - st.mv[t][e]);
          }
#pragma unroll
        for (int n = 0; n < D / 16; ++n)
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            const float4 v = merge[(w * S::kFrags + n * NT + t) * 32 + lane];
            st.acc[n][t][0] += v.x * f[t][0];
            st.acc[n][t][1] += v.y * f[t][1];
            st.acc[n][t][2] += v.z * f[t][0];
            st.acc[n][t][3] += v.w * f[t][1];
          }
      }
      __syncwarp();
      if (lane == 0) {
        scan[kCount] = 0;
        __threadfence_block();
        *reinterpret_cast<volatile int*>(&scan[kMerged]) = merges;
      }
    }
    if (whole) {
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const float f0 = out_factor(st.mv[t][0], st.l[t][0], kPShift);
        const float f1 = out_factor(st.mv[t][1], st.l[t][1], kPShift);
        const int rr = rt * kRows + 8 * t + g;  // the row this lane holds after the transposes
        const int tok = geo.by_G.div(rr), h = hk * geo.G + rr - tok * geo.G;
        uint16_t* o = p.o + b * p.os[0] + h * p.os[1] + tok * p.os[2] + 2 * c;
#pragma unroll
        for (int n = 0; n < D / 16; ++n)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const uint32_t v = transpose8x8(pack_bf16x2(st.acc[n][t][2 * x] * f0, st.acc[n][t][2 * x + 1] * f1));
            if (rr < rows) *reinterpret_cast<uint32_t*>(o + 16 * n + 8 * x) = v;
          }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int r2 = rt * kRows + 8 * t + 2 * c + e;
          if (g == 0 && r2 < rows) {
            const int tok2 = geo.by_G.div(r2), h2 = hk * geo.G + r2 - tok2 * geo.G;
            p.lse[(static_cast<size_t>(b) * p.H + h2) * p.N + tok2] = out_lse(st.m[t][e], st.l[t][e]);
          }
        }
      }
    } else {
      float* out = p.partial + (static_cast<size_t>(blockIdx.x) * 2 + slot_id) * part_floats(D, kRows);
      st.put(reinterpret_cast<float4*>(out), out + kRows * D, lane);
      __syncwarp();
      if (lane == 0) arrive(seg, cta0, blockIdx.x - cta0, parts, slot_id, rows, false);
    }
  }

  // The end of the run. All warps add up the states of the last piece (nothing is left
  // to overlap with), each its fragments, then the parts of the segments of which this
  // CTA's came last. Both go through shared memory and one piece of code, in the order
  // of the keys.
  for (int j = -1; ok && last_n > 0 && j < 2;) {
    Join join = {0, 1, last_n, whole != 0};
    if (j >= 0) {
      if (!((*reinterpret_cast<volatile int*>(&scan[kJobs]) >> j) & 1)) {
        ++j;
        continue;
      }
      const int* job = scan + kJob0 + kJobInts * j;
      seg = job[0], cta0 = job[1], parts = job[2], rows = job[3];
      join = {job[4], job[5], job[6], job[7] != 0};
      last_from = 0;
    }
    const int bh = geo.by_RT.div(seg), rt = seg - bh * geo.RT, b = geo.by_Hk.div(bh), hk = bh - b * p.c.Hk;
    constexpr int kPart = part_floats(D, kRows);
    // part 0 begins in its CTA's run and lies in its second place
    auto place = [&](int part) {
      return p.partial + (static_cast<size_t>(cta0 + part) * 2 + (part == 0 ? 1 : 0)) * kPart;
    };
    FragmentSums<D, NT> f;
    f.clear();
    for (int k0 = 0; ok && k0 < join.n; k0 += kConsumers) {
      const int n = min(join.n - k0, kConsumers);
      if (j >= 0) {
        if (!sync_warps()) break;            // what was there has been read
        constexpr int kUnits = kPart / 4;    // of 16 bytes
#pragma unroll 1
        for (int i = tid; i < n * kUnits; i += 32 * kConsumers) {
          const int k = i / kUnits, u = i - k * kUnits;
          void* dst = u < S::kFrags * 32 ? static_cast<void*>(merge + k * S::kFrags * 32 + u)
                                         : static_cast<void*>(stats + 3 * kRows * k + 4 * (u - S::kFrags * 32));
          cp_async16(smem_u32(dst), place(join.first + (k0 + k) * join.stride) + 4 * u);  // past L1: other CTAs wrote them
        }
        cp_async_wait();
      }
      if (!sync_warps()) break;
      f.add(n, last_from, merge, stats, warp, lane);
    }
    if (!ok) break;
    if (join.last) {
      f.store(p, geo, b, hk, rt * kRows, rows, warp, lane);
      ++j;
    } else {
      if (j >= 0 && tid == 0) atomicAnd(&scan[kJobs], ~(1 << j));
      const int part = j < 0 ? static_cast<int>(blockIdx.x) - cta0 : join.first;
      float* out = place(part);
      f.put(reinterpret_cast<float4*>(out), out + kRows * D, warp, lane);
      if (!sync_warps()) break;
      if (tid == 0) arrive(seg, cta0, part, parts, j < 0 ? (part == 0 ? 1 : 0) : j, rows, j >= 0);
      if (!sync_warps()) break;  // a join that this was the last part of is noted
      if (j < 0) j = 0;
    }
  }

  // segments without a visible page: O = 0, LSE = -inf
  for (int seg = blockIdx.x + gridDim.x * warp; ok && line.any_empty && seg < nseg; seg += gridDim.x * kConsumers) {
    if (pages_of<kVec>(p, geo, seg) != 0) continue;
    const int bh = geo.by_RT.div(seg), rt = seg - bh * geo.RT, b = geo.by_Hk.div(bh), hk = bh - b * p.c.Hk;
    const RowTile r = row_tile(p, geo, b, rt, lane == 0);
    const int row_hi = min(geo.G * r.live, (rt + 1) * kRows);
    for (int rr = rt * kRows; rr < row_hi; ++rr) {
      const int t = geo.by_G.div(rr), h = hk * geo.G + rr - t * geo.G;
      uint16_t* o = p.o + b * p.os[0] + h * p.os[1] + t * p.os[2];
      for (int k = lane; k < D / 2; k += 32) *reinterpret_cast<uint32_t*>(o + 2 * k) = 0u;
      if (lane == 0) p.lse[(static_cast<size_t>(b) * p.H + h) * p.N + t] = -INFINITY;
    }
  }
}

// Lets the kernel have its shared memory, once for each device.
template <int D, int NT, bool kVec>
cudaError_t allow_smem() {
  static std::atomic<uint64_t> done[4];  // devices 0 .. 255
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev > 255) return cudaErrorInvalidDevice;
  if (done[dev >> 6].load(std::memory_order_relaxed) >> (dev & 63) & 1) return cudaSuccess;
  e = cudaFuncSetAttribute(cache_fwd_kernel<D, NT, kVec>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           Smem<D, NT>::kBytes);
  if (e == cudaSuccess) done[dev >> 6].fetch_or(1ull << (dev & 63), std::memory_order_relaxed);
  return e;
}

template <int D, int NT, bool kVec>
cudaError_t launch_t(const CacheFwdParams& p, const Geometry& geo, int num_sms, cudaStream_t s) {
  if (kVec) {
    const cudaError_t c = launch_cache_classify(p, geo, s);
    if (c != cudaSuccess) return c;
  }
  const cudaError_t e = allow_smem<D, NT, kVec>();
  if (e != cudaSuccess) return e;
  const int grid = num_sms < kCacheMaxCtas ? num_sms : kCacheMaxCtas;
  cache_fwd_kernel<D, NT, kVec><<<grid, kThreads, Smem<D, NT>::kBytes, s>>>(p, geo);
  return cudaGetLastError();
}

template <int D, int NT>
cudaError_t launch_nt(const CacheFwdParams& p, const Geometry& geo, int num_sms, cudaStream_t s) {
  return p.mask.lts != nullptr || p.mask.uts != nullptr ? launch_t<D, NT, true>(p, geo, num_sms, s)
                                                        : launch_t<D, NT, false>(p, geo, num_sms, s);
}

// Rows of a tile: 8 or 16 as long as two tiles hold all rows, above that 128 on
// tcgen05. Every tile reads and converts the codes again, which soon costs more than
// rows of a tile that are empty. 16 sequences of 16384 tokens, 4 cache heads, tiles of
// 16 rows / of 128, us:
//   rows       16           24           32           40           64          128
//   d = 64   41.0 / -    58.2 / 68.1  59.0 / 68.1  81.6 / 72.1   104 / 72.8   191 / 76.5
//   d = 128  60.3 / -    83.3 / 86.6  84.9 / 87.0   133 / 91.5   172 / 92.4   325 / 99.5
int rows_of_tile(int rows) { return rows <= 8 ? 8 : rows <= 32 ? 16 : kManyRows; }

Geometry geometry(int H, int Hk, int Hm, int N, int max_pages) {
  Geometry g;
  g.G = H / Hk;
  const int rows = g.G * N;  // below 2^31: B * H * N is
  g.rows = rows_of_tile(rows);
  g.RT = (rows - 1) / g.rows + 1;
  g.classes = Hk % Hm == 0 ? Hm : Hk;
  g.words = (max_pages + 31) / 32;
  g.by_G.set(g.G);
  g.by_RT.set(g.RT);
  g.by_Hk.set(Hk);
  g.by_class.set(Hk / g.classes);
  g.by_mask.set(H / Hm);
  return g;
}

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

}  // namespace

bool cache_line_ok(int B, int H, int Hk, int N, int max_pages) {
  const Geometry g = geometry(H, Hk, Hk, N, max_pages);
  // (rounding up to whole runs adds less than a page for each CTA)
  return static_cast<double>(B) * Hk * g.RT * max_pages < 2147483648.0 - kCacheMaxCtas;
}

CacheWs cache_ws_layout(int B, int H, int Hk, int N, int d, int max_pages) {
  const Geometry g = geometry(H, Hk, Hk, N, max_pages);
  const size_t tiles = static_cast<size_t>(B) * Hk * g.RT;
  CacheWs w;
  // the status word and the counters, which have to be zero, lie at the same place for
  // all sizes, so that one workspace serves them in turn
  size_t off = 256;
  w.arrived = off;
  off = up256(off + kCacheMaxCtas * 4);
  w.groups = off;
  off = up256(off + kCacheMaxCtas * 8);
  w.partial = off;
  off = up256(off + static_cast<size_t>(kCacheMaxCtas) * 2 *
                    (g.rows == kManyRows ? cache_fwd_rows_part_floats(d) : part_floats(d, g.rows)) * 4);
  w.list = off;
  off = up256(off + tiles * max_pages * 2);
  w.listed = off;
  off = up256(off + tiles * 4);
  w.total = off;
  return w;
}

cudaError_t launch_cache_fwd(int d, const CacheFwdParams& p, int num_sms, cudaStream_t s) {
  const Geometry geo = geometry(p.H, p.c.Hk, p.mask.Hm, p.N, p.max_pages);
  if (geo.rows == kManyRows) return launch_cache_fwd_rows(d, p, geo, num_sms, s);
  if (d == 64) return geo.rows == 8 ? launch_nt<64, 1>(p, geo, num_sms, s) : launch_nt<64, 2>(p, geo, num_sms, s);
  return geo.rows == 8 ? launch_nt<128, 1>(p, geo, num_sms, s) : launch_nt<128, 2>(p, geo, num_sms, s);
}

}  // namespace fm
