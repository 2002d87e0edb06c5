// Attention over the 8-bit paged cache for many query rows per cache head (chunks
// of prompts, drafted tokens of large groups): tiles of 128 rows on tcgen05.
//
// The line of pages, its cut into equal runs and the joins are those of the kernel
// for few rows; a unit of the line is a step of two pages, 128 keys. The codes of a
// step arrive by bulk copies and four warps turn them into fp16 operands in shared
// memory (exact), K as [key][d] and V as [d][key], both K-major and 128-byte
// swizzled; S = Q K^T and O += P V then run as kind::f16 with P in TMEM. Taking Q and P
// as sums of e4m3 parts would need no conversion; two parts hold an element of Q down to
// 2^-10 of its row's largest, four what fp16 holds of it (2^-30), three what it holds of
// P. That was not timed.
//
// As in the forward on bf16 tensors two softmax warpgroups split the keys of a step,
// warpgroup w taking page w, with states and accumulators O_w of their own, merged
// when a piece ends. So a warpgroup meets one K scale and one V scale a step: the
// first goes into the exponent, the second into P, relative to the row's largest
// P * scale so far (mv, counted from m of the scores), so that neither the weights of
// pages with small values nor the values of pages with small weights are lost. P is
// stored as fp16(2^7 P * scale / 2^mv) and O_w rescaled only when mv grows by more
// than 2^8.
//
// Warp roles (512 threads):
//   0-7    softmax: thread (w, r) owns row r (= TMEM lane) and the 64 keys of page w;
//          also bring in Q at the start of a piece and write the results at its end.
//   8      S issuer, 9 P V issuer (one thread each).
//   10     walks the run, looks pages up, issues the copies, publishes a step's
//          description to all roles (ring of kMetaRing).
//   12, 13 conversion of K; 14, 15 of V.
// TMEM, d = 128: S (128 columns), two P (64 columns each), O_0 and O_1. P has columns
// of its own, so the next S is computed as soon as this one has been read; with P
// over two regions of S, an S waited for the products of two steps before, 553 us
// where this took 545. With d = 64 there is room for three regions, P over its S:
// 69.5 us for 16 sequences of 16384 with 64 rows; two regions and two P: 77.
//
// Measured: 2 sequences of up to 32768 tokens, 512 query tokens, 32 / 8 heads of 128:
// 554 us, 971 TFLOP/s, 51 % of the bf16 rate (of d = 64: 440 us); 3 sequences up to 109407,
// 64 rows: 172 us, 3.5 TB/s. A step of 128 keys takes 2 180 cycles. (It took 545 us with mv
// as a number of its own; see out_factor. The figures that follow are from then.) Its
// products need 1 024; shared
// memory (d = 128: 32 KB of codes and 64 KB of operands written, 32 KB and 96 KB read)
// 1 750 at 128 bytes a clock; each softmax warp is busy for about 1 900, waits included,
// and the conversion warps for about 1 600. None of them alone is the bound: without
// the conversion the call takes 466 us, without the exponentials 511, without any work
// in the softmax 456. What did not help: Q in TMEM (shared memory reads - 14 %, 556
// us), S and P signalled to each warpgroup by itself (products of 64 keys, 610), the
// next codes loaded while some are converted (567), registers moved from the other
// roles to the softmax (615).
// The row's factor for scores past fp32 has a branch of its own: in the selection of masked
// scores it cost 3 % with d = 64 (455 us). Updating mv behind a branch: 561 us, 446.
#include <atomic>

#include "cache_common.cuh"
#include "flashmask.h"

namespace fm {
namespace {

constexpr int kThreads = 512;
constexpr int kRows = kManyRows;
constexpr int kMetaRing = 16;
constexpr int kMetaInts = 16;
// Steps a run has at least. One sequence of 4000 tokens, 2 cache heads, 128 rows, at
// least 2 / 4 / 8 steps: 29.7 / 26.3 / 27.1 us.
constexpr int kMinRun = 4;
constexpr int kOnce = 16, kFan = 8;  // see Join
constexpr float kPShift = 7.f;
constexpr float kLag = 8.f;  // mv may lag the row's largest product by this much (log2)

// A step's description, int[16]: the step, then four words for each of its two pages
// (first key, or -1 for none; K scale; log2 of the V scale; keys before the end).
enum MetaWord { kFlags, kSeg, kCta0, kParts, kPageWords, kJ0 = 0, kKs, kLvs, kValid };
// kCut and kNoScales << page
enum Flag { kFirstStep = 1, kLastStep = 2, kEnd = 4, kWhole = 8, kTailSlot = 16, kCut = 32, kNoScales = 128 };

template <int D>
struct Layout {
  static constexpr int R = D == 64 ? 3 : 2;   // operand slots of K and of V in shared memory
  static constexpr int kS = D == 64 ? 3 : 1;  // S regions in TMEM
  static constexpr bool kOver = D == 64;      // P lies over its S
  static constexpr int kStages = 2 * R;      // staged code tiles: K and V of R steps
  static constexpr int kTile = 128 * D * 2;  // fp16 operand tile
  static constexpr int kCodes = 128 * D;     // codes of a step, K or V
  static constexpr int kQ = 0;
  static constexpr int kK = kQ + kTile;
  static constexpr int kV = kK + R * kTile;
  static constexpr int kStage = kV + R * kTile;
  static constexpr int kMeta = kStage + kStages * kCodes;
  static constexpr int kWords = kMeta + kMetaRing * kMetaInts * 4;
  static constexpr int kBar = kWords + (kLineWords + 8) * 4;
  static constexpr int kNumBars = 2 * kStages + kMetaRing + 6 * R + 3;
  static constexpr int kTmemSlot = kBar + kNumBars * 8;
  static constexpr int kBytes = kTmemSlot + 16;
};
static_assert(Layout<128>::kBytes <= 227 * 1024 && Layout<64>::kBytes <= 227 * 1024, "shared memory per CTA");
static_assert(kMetaRing > 2 * Layout<64>::R + Layout<64>::kS + 3, "see where an entry is written");
static_assert(Layout<128>::kBar % 8 == 0 && Layout<64>::kBar % 8 == 0, "barriers are 8-byte aligned");

template <int R>
struct Bars {
  static constexpr int kStages = 2 * R, kFirst = 2 * kStages + kMetaRing;
  uint32_t base;
  __device__ uint32_t at(int i) const { return base + 8 * i; }
  __device__ uint32_t stage_full(int s) const { return at(s); }                // bytes
  __device__ uint32_t stage_empty(int s) const { return at(kStages + s); }     // 2 conversion warps
  __device__ uint32_t meta(int s) const { return at(2 * kStages + s); }        // 1
  __device__ uint32_t k_ready(int g) const { return at(kFirst + g); }          // 2
  __device__ uint32_t v_ready(int g) const { return at(kFirst + R + g); }      // 2
  __device__ uint32_t s_full(int g) const { return at(kFirst + 2 * R + g); }   // commit
  __device__ uint32_t p_full(int g) const { return at(kFirst + 3 * R + g); }   // 8
  __device__ uint32_t pv_done(int g) const { return at(kFirst + 4 * R + g); }  // commit
  __device__ uint32_t s_read(int g) const { return at(kFirst + 5 * R + g); }   // 8
  __device__ uint32_t q_full() const { return at(kFirst + 6 * R); }            // 8
  __device__ uint32_t o_free() const { return at(kFirst + 6 * R + 1); }        // 8
  __device__ uint32_t softmax() const { return at(kFirst + 6 * R + 2); }       // 8
};

// TMEM columns: S of step J, P of its page w (64 keys in 32 columns; with places of
// their own two steps in turn), accumulator w.
template <int D>
__device__ __forceinline__ uint32_t col_s(int J) {
  return 128u * static_cast<uint32_t>(J % Layout<D>::kS);
}
template <int D>
__device__ __forceinline__ uint32_t col_p(int J, int w) {
  return Layout<D>::kOver ? col_s<D>(J) + 64u * static_cast<uint32_t>(w)
                          : 128u * Layout<D>::kS + 64u * static_cast<uint32_t>(J & 1) + 32u * static_cast<uint32_t>(w);
}
template <int D>
__device__ __forceinline__ uint32_t col_o(int w) {
  return 128u * Layout<D>::kS + (Layout<D>::kOver ? 0u : 128u) + D * static_cast<uint32_t>(w);
}

// Instruction descriptor, kind::f16 with fp16 A and B (format code 0), both K-major.
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N) {
  return (1u << 4) | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}

// Steps on a segment's line.
template <bool kVec>
__device__ __forceinline__ int steps_of(const CacheFwdParams& p, const Geometry& geo, int seg) {
  return (pages_of<kVec>(p, geo, seg) + 1) >> 1;
}

// Bits of the keys j .. j + 63 with s <= pos < e.
__device__ __forceinline__ uint64_t hidden64(const int32_t* s, const int32_t* e, int pos) {
  uint64_t hid = 0;
#pragma unroll 4
  for (int q = 0; q < 16; ++q) {
    const int4 a = *reinterpret_cast<const int4*>(s + 4 * q), z = *reinterpret_cast<const int4*>(e + 4 * q);
    const uint32_t b = static_cast<uint32_t>(a.x <= pos && pos < z.x) | static_cast<uint32_t>(a.y <= pos && pos < z.y) << 1 |
                       static_cast<uint32_t>(a.z <= pos && pos < z.z) << 2 | static_cast<uint32_t>(a.w <= pos && pos < z.w) << 3;
    hid |= static_cast<uint64_t>(b) << (4 * q);
  }
  return hid;
}

// Scales n (32) TMEM columns of this warp's lanes by f.
__device__ __forceinline__ void tmem_scale32(uint32_t taddr, float f) {
  uint32_t v[32];
  tmem_ld32(taddr, v);
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * f);
  tmem_st32(taddr, v);
}

// Floats of one partial result: O as float4 [D / 4][128 rows], then m, mv, l [128].
constexpr __host__ __device__ int part_floats(int D) { return kRows * D + 3 * kRows; }

template <int D, bool kVec>
__global__ void __launch_bounds__(kThreads, 1) cache_fwd_rows_kernel(const __grid_constant__ CacheFwdParams p,
                                                                     const __grid_constant__ Geometry geo) {
  using L = Layout<D>;
  constexpr int R = L::R, kStages = L::kStages;
  extern __shared__ __align__(1024) uint8_t smem[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int nseg = p.B * p.c.Hk * geo.RT;
  if ((smem_u32(smem) & 1023u) != 0) {
    if (tid == 0) record_failure(p.status, kStatusLayout, kSiteCacheWait);
    return;
  }
  const uint32_t sQ = smem_u32(smem + L::kQ), sK = smem_u32(smem + L::kK), sV = smem_u32(smem + L::kV);
  const Bars<R> bar{smem_u32(smem + L::kBar)};
  int* words = reinterpret_cast<int*>(smem + L::kWords);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kTmemSlot);
  const int* meta_at = reinterpret_cast<const int*>(smem + L::kMeta);

  if (warp == 9) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  if (tid < L::kNumBars) {
    // arrivals: stage_full 1, stage_empty 2, meta 1, k_ready and v_ready 2, s_full 1,
    // p_full 8, pv_done 1, s_read, q_full, o_free and softmax 8
    const int i = tid - 2 * kStages - kMetaRing;
    int n = 1;
    if (tid >= kStages && tid < 2 * kStages) n = 2;
    if (i >= 0 && i < 2 * R) n = 2;
    if ((i >= 3 * R && i < 4 * R) || i >= 5 * R) n = 8;
    mbar_init(bar.at(tid), n);
    fence_barrier_init();
  }
  const Line line = find_run<kThreads>(nseg, kMinRun, 2, words, [&](int s) { return steps_of<kVec>(p, geo, s); });
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  // Waits for the description of step J; its flags, kEnd when the wait gave up.
  auto step_flags = [&](int J) -> int {
    if (!cache_wait(bar.meta(J % kMetaRing), (J / kMetaRing) & 1, p.status)) return kEnd;
    return meta_at[(J % kMetaRing) * kMetaInts + kFlags];
  };
  if (warp == 10) {
    // ------------------------------------------------------------ run, pages, copies
    int seg = line.seg, k = line.first, done = 0;
    const int steps = line.hi - line.lo;
    bool ok = true;
    auto slot_free = [&](int seq) {
      return seq < kStages || cache_wait(bar.stage_empty(seq % kStages), (seq / kStages - 1) & 1, p.status);
    };
    while (ok && done < steps) {
      int my_seg, my_k, my_n;
      const int avail = next_units(
          seg, k, nseg, min(32, steps - done), [&](int s) { return steps_of<kVec>(p, geo, s); }, my_seg, my_k, my_n);
      int page[2] = {-1, -1}, j0[2] = {-1, -1}, valid[2] = {0, 0}, cut[2] = {0, 0}, none[2] = {0, 0};
      float ks[2] = {0.f, 0.f}, lvs[2] = {0.f, 0.f};
      if (lane < avail) {
        const int bh = geo.by_RT.div(my_seg), rt = my_seg - bh * geo.RT, b = geo.by_Hk.div(bh), hk = bh - b * p.c.Hk;
        const int pages = pages_of<kVec>(p, geo, my_seg);
        const RowTile r = row_tile(p, geo, b, rt, true);
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          if (2 * my_k + x >= pages) continue;
          const int logical = page_on_line<kVec>(p, geo, b, hk, rt, 2 * my_k + x, cut[x]);
          const int pg = p.table[static_cast<size_t>(b) * p.max_pages + logical];
          if (pg < 0 || pg >= p.c.pages) {
            record_failure(p.status, kStatusPage, kSiteCachePage);
            continue;
          }
          const size_t ph = static_cast<size_t>(pg) * p.c.Hk + hk;
          page[x] = pg;
          j0[x] = logical * kPage;
          valid[x] = min(r.len - j0[x], kPage);
          const float vs = p.c.vscale[ph];
          ks[x] = p.c.kscale[ph];
          none[x] = no_scales(ks[x], vs);
          lvs[x] = log2_scale(vs);
        }
      }
      for (int t = 0; ok && t < avail; ++t, ++done) {
        const int sg = __shfl_sync(0xffffffffu, my_seg, t), kk = __shfl_sync(0xffffffffu, my_k, t);
        const int nn = __shfl_sync(0xffffffffu, my_n, t);
        int m[kMetaInts] = {};
        int pg[2];
        m[kSeg] = sg;
        const int cuts = __shfl_sync(0xffffffffu, cut[0] | cut[1] << 1 | none[0] << 2 | none[1] << 3, t);
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          pg[x] = __shfl_sync(0xffffffffu, page[x], t);
          int* w = m + kPageWords + 4 * x;
          w[kJ0] = __shfl_sync(0xffffffffu, j0[x], t);
          w[kKs] = __shfl_sync(0xffffffffu, __float_as_int(ks[x]), t);
          w[kLvs] = __shfl_sync(0xffffffffu, __float_as_int(lvs[x]), t);
          w[kValid] = __shfl_sync(0xffffffffu, valid[x], t);
        }
        if (lane == 0) {
          const bool first = done == 0 || kk == 0, last = kk == nn - 1 || done == steps - 1;
          const int s0 = line.lo + done - kk, cta0 = s0 / line.run;  // s0: where the segment begins on the line
          const int parts = (s0 + nn - 1) / line.run - cta0 + 1;
          // a segment that ends and begins in this run is whole: it starts here (its
          // first step does) and ends before the run's end
          const bool starts_here = s0 >= line.lo, ends_here = s0 + nn <= line.hi;
          m[kFlags] = (first ? kFirstStep : 0) | (last ? kLastStep : 0) | (starts_here && ends_here ? kWhole : 0) |
                      (starts_here ? kTailSlot : 0) | kCut * cuts;
          m[kCta0] = cta0;
          m[kParts] = parts;
          ok = slot_free(2 * done);
          if (ok) {
            // the entry was last read for step J - kMetaRing, which every role has left: the K
            // codes of step J - R are converted, so S of step J - 2 R is done, S of step
            // x = J - 2 R - kS is read (or its products are done, if P lay over it), and the
            // products of step x - 3 are done, V with them
            int4* at = reinterpret_cast<int4*>(smem + L::kMeta) + (done % kMetaRing) * (kMetaInts / 4);
#pragma unroll
            for (int i = 0; i < kMetaInts / 4; ++i) at[i] = make_int4(m[4 * i], m[4 * i + 1], m[4 * i + 2], m[4 * i + 3]);
            mbar_arrive(bar.meta(done % kMetaRing));
          }
          const int bh = geo.by_RT.div(sg), hk = bh - geo.by_Hk.div(bh) * p.c.Hk;
          const uint32_t bytes = (pg[0] >= 0 ? L::kCodes / 2 : 0) + (pg[1] >= 0 ? L::kCodes / 2 : 0);
#pragma unroll
          for (int kv = 0; kv < 2; ++kv) {
            const int seq = 2 * done + kv, slot = seq % kStages;
            if (kv == 1 && ok) ok = slot_free(seq);
            if (!ok) break;
            mbar_arrive_expect_tx(bar.stage_full(slot), bytes);
#pragma unroll
            for (int x = 0; x < 2; ++x)
              if (pg[x] >= 0)
                bulk_load(smem_u32(smem + L::kStage + slot * L::kCodes + x * (L::kCodes / 2)),
                          (kv ? p.c.v8 : p.c.k8) + (static_cast<size_t>(pg[x]) * p.c.Hk + hk) * (kPage * D), L::kCodes / 2,
                          bar.stage_full(slot));
          }
        }
        ok = __all_sync(0xffffffffu, ok);
      }
      if (avail > 0) {
        seg = __shfl_sync(0xffffffffu, my_seg, avail - 1);
        k = __shfl_sync(0xffffffffu, my_k, avail - 1) + 1;
      } else {
        seg += 32;
        k = 0;
        if (seg >= nseg) ok = lengths_moved(p.status);
      }
    }
    if (lane == 0) {
      if (ok && slot_free(2 * done)) {
        (reinterpret_cast<int*>(smem + L::kMeta) + (done % kMetaRing) * kMetaInts)[kFlags] = kEnd;
        mbar_arrive(bar.meta(done % kMetaRing));
      } else {
        // copies in flight land before the CTA's shared memory is given up
        for (int seq = max(0, 2 * done - kStages); seq < 2 * done; ++seq)
          mbar_wait_for(bar.stage_full(seq % kStages), (seq / kStages) & 1, nullptr, 1000000ull);
      }
    }
  } else if (warp == 8) {
    // ------------------------------------------------------------ S issuer
    if (lane == 0) {
      constexpr uint32_t idesc = idesc_f16(128, 128);
      const uint64_t dq = sdesc_sw128(sQ, 16, 1024), dk = sdesc_sw128(sK, 16, 1024);
      int pieces = 0;
      for (int J = 0;; ++J) {
        const int flags = step_flags(J);
        if (flags & kEnd) break;
        const int g = J % R;
        // Q of the piece; the region: S of step J - kS has been read, and if P lay over it
        // its products are done; K
        if ((flags & kFirstStep) && !cache_wait(bar.q_full(), pieces++ & 1, p.status)) break;
        if (J >= L::kS) {
          const int x = J - L::kS;
          if (!cache_wait(L::kOver ? bar.pv_done(x % R) : bar.s_read(x % R), (x / R) & 1, p.status)) break;
        }
        if (!cache_wait(bar.k_ready(g), (J / R) & 1, p.status)) break;
        tc_fence_after();
        const uint64_t kd = dk + static_cast<uint64_t>((g * L::kTile) >> 4);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint64_t off = static_cast<uint64_t>(((kk >> 2) * 16384 + (kk & 3) * 32) >> 4);
          mma_ss(tmem + col_s<D>(J), dq + off, kd + off, idesc, kk > 0);
        }
        mma_commit(bar.s_full(g));
      }
    }
  } else if (warp == 9) {
    // ------------------------------------------------------------ P V issuer
    if (lane == 0) {
      constexpr uint32_t idesc = idesc_f16(128, D);
      const uint64_t dv = sdesc_sw128(sV, 16, 1024);
      int pieces = 0;
      for (int J = 0;; ++J) {
        const int flags = step_flags(J);
        if (flags & kEnd) break;
        const int g = J % R;
        const bool first = flags & kFirstStep;
        if (!cache_wait(bar.v_ready(g), (J / R) & 1, p.status)) break;
        // the piece's first products overwrite the accumulators of the piece before
        if (first && pieces > 0 && !cache_wait(bar.o_free(), (pieces - 1) & 1, p.status)) break;
        pieces += first;
        if (!cache_wait(bar.p_full(g), (J / R) & 1, p.status)) break;
        tc_fence_after();
        const uint64_t vd = dv + static_cast<uint64_t>((g * L::kTile) >> 4);
#pragma unroll
        for (int w = 0; w < 2; ++w)
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            mma_ts(tmem + col_o<D>(w), tmem + col_p<D>(J, w) + 8 * kk,
                   vd + static_cast<uint64_t>((w * D * 128 + kk * 32) >> 4), idesc, !first || kk > 0);
        mma_commit(bar.pv_done(g));
      }
    }
  } else if (warp >= 12) {
    // ------------------------------------------------------------ conversion
    // warps 12, 13: K; warps 14, 15: V. Both tiles are blocks of rows of 64 codes: K two
    // halves (d = 128) of 128 keys, V the columns of two pages. A thread's piece of 16
    // codes lies at the same place of every 16th row, so its swizzled units do too. The
    // loop stays short on purpose: with it unrolled the roles' code overflowed the
    // instruction cache, which cost more than anything else here.
    const int kv = (warp - 12) >> 1, ct = tid & 63, pc = ct & 3, row0 = ct >> 2;
    const int blocks = kv ? 2 : D / 64, block_rows = kv ? D : 128, row_bytes = kv ? 64 : D;
    // K, d = 128: odd rows begin with the other half, or the 64 bytes that eight lanes
    // take of two rows would lie in the same banks
    const int swap = !kv && D == 128 ? row0 & 1 : 0;
    const uint32_t u0 = ((2 * pc) ^ (row0 & 7)) << 4, u1 = ((2 * pc + 1) ^ (row0 & 7)) << 4;
    bool ok = true;
    for (int J = 0; ok; ++J) {
      ok = __all_sync(0xffffffffu, cache_wait(bar.meta(J % kMetaRing), (J / kMetaRing) & 1, p.status));
      if (!ok) break;
      const int* m = meta_at + (J % kMetaRing) * kMetaInts;
      if (m[kFlags] & kEnd) break;
      const int valid[2] = {m[kPageWords + kValid], m[kPageWords + 4 + kValid]};
      const int g = J % R, slot = (2 * J + kv) % kStages;
      // the operand slot is free once the products of step J - R have read it
      const uint32_t freed = kv ? bar.pv_done(g) : bar.s_full(g);
      ok = cache_wait(bar.stage_full(slot), ((2 * J + kv) / kStages) & 1, p.status) &&
           (J < R || cache_wait(freed, (J / R - 1) & 1, p.status));
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      uint8_t* codes = smem + L::kStage + slot * L::kCodes + row0 * row_bytes + 16 * pc;
      if (kv && __builtin_expect((valid[0] & valid[1]) != kPage, 0)) {
        // V: codes behind the sequence's end (or of an absent page) become 0, each
        // thread's where it reads them
        for (int x = 0; x < 2; ++x) {
          const int left = valid[x] - 16 * pc;
          uint32_t keep[4];
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const int nb = min(max(left - 4 * u, 0), 4);
            keep[u] = nb == 4 ? ~0u : (1u << (8 * nb)) - 1u;
          }
#pragma unroll 1
          for (int row = 0; row < D; row += 16) {
            uint4* at = reinterpret_cast<uint4*>(codes + (x * D + row) * kPage);
            const uint4 w = *at;
            *at = make_uint4(w.x & keep[0], w.y & keep[1], w.z & keep[2], w.w & keep[3]);
          }
        }
      }
      const uint32_t dst = (kv ? sV : sK) + g * L::kTile + row0 * 128;
      for (int x = 0; x < blocks; ++x) {
        const int y = x ^ swap;
        const uint8_t* src = codes + y * (kv ? kPage * D : 64);
        const uint32_t to = dst + y * block_rows * 128;
#pragma unroll 1
        for (int row = 0; row < block_rows; row += 64) {
          uint4 w[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) w[i] = *reinterpret_cast<const uint4*>(src + (row + 16 * i) * row_bytes);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t h[8];
#pragma unroll
            for (int u = 0; u < 4; ++u) codes_to_f16(word(w[i], u), h[2 * u], h[2 * u + 1]);
            const uint32_t at = to + (row + 16 * i) * 128;
            st_shared_v4(at + u0, h[0], h[1], h[2], h[3]);
            st_shared_v4(at + u1, h[4], h[5], h[6], h[7]);
          }
        }
      }
      fence_proxy_async_smem();  // the operands are read by the tensor cores
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(kv ? bar.v_ready(g) : bar.k_ready(g));
        mbar_arrive(bar.stage_empty(slot));
      }
    }
  } else if (warp < 8) {
    // ------------------------------------------------------------ softmax
    const int w = warp >> 2;
    const int row = (warp & 3) * 32 + lane;
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    float* red = reinterpret_cast<float*>(smem + L::kQ);  // [w][m, mv, l][128], between pieces
    bool ok = true;
    int syncs = 0;
    auto sync_softmax = [&]() {
      __syncwarp();
      if (lane == 0) mbar_arrive(bar.softmax());
      ok = __all_sync(0xffffffffu, cache_wait(bar.softmax(), syncs & 1, p.status));
      ++syncs;
      return ok;
    };
    for (int J = 0; ok;) {
      ok = __all_sync(0xffffffffu, cache_wait(bar.meta(J % kMetaRing), (J / kMetaRing) & 1, p.status));
      if (!ok) break;
      const int* head = meta_at + (J % kMetaRing) * kMetaInts;
      if (head[kFlags] & kEnd) break;
      const int seg = head[kSeg], cta0 = head[kCta0], parts = head[kParts];
      const bool whole = head[kFlags] & kWhole;
      const int slot = head[kFlags] & kTailSlot ? 1 : 0;
      // this thread's row, and Q: columns [w D/2, w D/2 + D/2) of it
      const int bh = geo.by_RT.div(seg), rt = seg - bh * geo.RT, b = geo.by_Hk.div(bh), hk = bh - b * p.c.Hk;
      const RowTile r = row_tile(p, geo, b, rt, tid == 0);
      const int rows = geo.G * r.live;
      const int rr = rt * kRows + row;
      const bool live = rr < rows;
      const bool warp_live = __any_sync(0xffffffffu, live);
      const int tok = geo.by_G.div(rr), h = hk * geo.G + rr - tok * geo.G;
      const int pos = r.shift + tok;
      const int lim = live && p.mask.causal ? min(r.len, pos + 1) : r.len;
      const size_t mrow =
          kVec ? (static_cast<size_t>(b) * p.mask.Hm + geo.by_mask.div(h)) * static_cast<size_t>(p.max_pages * kPage) : 0;
      uint4 x[D / 16];
      const uint16_t* src = p.q + b * p.qs[0] + h * p.qs[1] + tok * p.qs[2] + w * (D / 2);
      uint32_t top = 0;
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        x[i] = live ? *reinterpret_cast<const uint4*>(src + 8 * i) : make_uint4(0u, 0u, 0u, 0u);
        const uint32_t mk = 0x7fff7fffu;
        const uint32_t a = __vmaxu2(__vmaxu2(x[i].x & mk, x[i].y & mk), __vmaxu2(x[i].z & mk, x[i].w & mk));
        top = max(top, max(a & 0xffffu, a >> 16));
      }
      // the last S of the piece before has been read: Q's place is free
      reinterpret_cast<uint32_t*>(red)[w * kRows + row] = top;
      if (!sync_softmax()) break;
      top = max(top, reinterpret_cast<uint32_t*>(red)[(w ^ 1) * kRows + row]);
      if (!sync_softmax()) break;
      const bool bad = top >= 0x7f80u;
      const int up = top == 0 || bad ? 0 : min(14 - (static_cast<int>(top >> 7) - 127), 126);
      const float f = bad ? __int_as_float(0x7fffffff) : __int_as_float((up + 127) << 23);
      const float crow = p.scale_log2 * __int_as_float((127 - up) << 23);
      // keys that every row of the warp sees (none if one may need score_boost)
      const int all_lim = __reduce_min_sync(0xffffffffu, crow > 1.f ? 0 : lim);
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        const uint32_t v[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
        uint32_t y[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          y[j] = pack_f16x2(__uint_as_float(v[j] << 16) * f, __uint_as_float(v[j] & 0xffff0000u) * f);
        const int unit = w * (D / 16) + i;  // 16-byte unit of the row
        st_shared_v4(sQ + (unit >> 3) * 16384 + sw128_offset(row, unit & 7), y[0], y[1], y[2], y[3]);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar.q_full());
      float m_ = kNoScore, mv = kNoProduct, l = 0.f;

      // ---- the piece's steps; what is rare is kept out of the loop's straight line
      int flags;
      for (bool first = true;; first = false, ++J) {
        if (!first) {
          ok = __all_sync(0xffffffffu, cache_wait(bar.meta(J % kMetaRing), (J / kMetaRing) & 1, p.status));
          if (!ok) break;
        }
        const int g = J % R;
        flags = meta_at[(J % kMetaRing) * kMetaInts + kFlags];
        const int4 pw = *reinterpret_cast<const int4*>(meta_at + (J % kMetaRing) * kMetaInts + kPageWords + 4 * w);
        const int j0 = pw.x;
        float c = score_factor(crow, __int_as_float(pw.y));  // a score is S times c
        const float lvs = __int_as_float(pw.z);
        const bool masked = j0 < 0 || j0 + kPage > all_lim || (flags & ((kCut | kNoScales) << w));
        ok = __all_sync(0xffffffffu, cache_wait(bar.s_full(g), (J / R) & 1, p.status));
        if (!ok) break;
        if (!warp_live) {
          if (!L::kOver && lane == 0) mbar_arrive(bar.s_read(g));
        } else {
          tc_fence_after();
          uint32_t sv[64];
          const uint32_t s_addr = tmem + lane_base + col_s<D>(J) + 64 * w;
          tmem_ld64(s_addr, s_addr + 32, sv);
          if constexpr (!L::kOver) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar.s_read(g));
          }
          if (__builtin_expect(masked, 0)) {
            const int n = j0 < 0 ? 0 : min(max(lim - j0, 0), kPage);
            uint64_t hid = n == kPage ? 0ull : ~0ull << n;  // keys this row does not see
            if constexpr (kVec) {
              if ((flags & (kCut << w)) && j0 >= 0) {
                if (p.mask.lts) hid |= hidden64(p.mask.lts + mrow + j0, p.mask.lte + mrow + j0, pos);
                if (p.mask.uts) hid |= hidden64(p.mask.uts + mrow + j0, p.mask.ute + mrow + j0, pos);
              }
            }
            const uint32_t hlo = static_cast<uint32_t>(hid), hhi = static_cast<uint32_t>(hid >> 32);
            const float boost = score_boost(crow, __int_as_float(pw.y), flags & (kNoScales << w), c);
            if (__builtin_expect(__any_sync(0xffffffffu, boost != 1.f), 0)) {
#pragma unroll
              for (int j = 0; j < 64; ++j) sv[j] = __float_as_uint(__uint_as_float(sv[j]) * boost);
            }
#pragma unroll
            for (int j = 0; j < 64; ++j) sv[j] = (((j < 32 ? hlo : hhi) >> (j & 31)) & 1u) ? 0xff800000u : sv[j];
          }
          float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int j = 0; j < 64; j += 8)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              mx[i] = fmax3(mx[i], __uint_as_float(sv[j + 2 * i]), __uint_as_float(sv[j + 2 * i + 1]));
          const float pm = fmax3(fmaxf(mx[0], mx[1]), mx[2], mx[3]) * c;
          const float m_new = fmaxf(m_, pm);
          const float dm = m_ - m_new;
          l *= ex2(dm);
          m_ = m_new;
          const float mv_old = mv + dm, mv_new = fmaxf(mv_old, pm - m_new + lvs);
          const bool rescale = mv_new > mv_old + kLag;
          mv = rescale ? mv_new : mv_old;
          const float f = ex2(fminf(lvs - mv + kPShift, 126.f));
          const uint64_t c2 = f2_make(c, c), nm2 = f2_make(-m_new, -m_new), f2 = f2_make(f, f);
          uint64_t l2 = f2_make(0.f, 0.f);
          uint32_t pk[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            float x0, x1, p0, p1;
            f2_split(f2_fma(f2_make(__uint_as_float(sv[2 * i]), __uint_as_float(sv[2 * i + 1])), c2, nm2), x0, x1);
            const uint64_t pp = f2_make(ex2(x0), ex2(x1));
            l2 = f2_add(l2, pp);
            f2_split(f2_mul(pp, f2), p0, p1);
            pk[i] = pack_f16x2(p0, p1);
          }
          float l0, l1;
          f2_split(l2, l0, l1);
          l += l0 + l1;
          if (!L::kOver && J >= 2) {  // the products that read P of step J - 2 have completed
            ok = __all_sync(0xffffffffu, cache_wait(bar.pv_done((J - 2) % R), ((J - 2) / R) & 1, p.status));
            if (!ok) break;
            tc_fence_after();
          }
          tmem_st32p(tmem + lane_base + col_p<D>(J, w), pk);
          if (__builtin_expect(!first && __any_sync(0xffffffffu, rescale), 0)) {
            // O_w is rescaled once the products of step J - 1 have completed
            ok = __all_sync(0xffffffffu, cache_wait(bar.pv_done((J - 1) % R), ((J - 1) / R) & 1, p.status));
            if (!ok) break;
            tc_fence_after();
            const float alpha = rescale ? ex2(mv_old - mv) : 1.f;
#pragma unroll 1
            for (int ch = 0; ch < D / 32; ++ch) tmem_scale32(tmem + lane_base + col_o<D>(w) + 32 * ch, alpha);
          }
          tmem_st_wait();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar.p_full(g));
        if (flags & kLastStep) break;
      }
      if (!ok) break;

      // ---- the piece's end: the two halves' states are merged
      const int g = J % R;
      ok = __all_sync(0xffffffffu, cache_wait(bar.pv_done(g), (J / R) & 1, p.status));
      ++J;
      if (!ok) break;
      tc_fence_after();
      red[w * 3 * kRows + row] = m_;
      red[(w * 3 + 1) * kRows + row] = mv;
      red[(w * 3 + 2) * kRows + row] = l;
      if (!sync_softmax()) break;
      const float* other = red + (w ^ 1) * 3 * kRows + row;
      const float m = fmaxf(m_, other[0]), da = m_ - m, db = other[0] - m;
      const float mvs = mv + da, mvo = other[kRows] + db, mva = fmaxf(mvs, mvo);
      // the sum in the same order in both warpgroups, so that they agree to the bit
      const float la = l * ex2(da), lb = other[2 * kRows] * ex2(db);
      const float lsum = w == 0 ? la + lb : lb + la;
      const float fs = ex2(mvs - mva), fo = ex2(mvo - mva);
      const float out = whole ? out_factor(mva, lsum, kPShift) : 1.f;
      const float f0 = (w == 0 ? fs : fo) * out, f1 = (w == 0 ? fo : fs) * out;
      float* part = p.partial + (static_cast<size_t>(blockIdx.x) * 2 + slot) * part_floats(D);
      uint16_t* o = p.o + b * p.os[0] + h * p.os[1] + tok * p.os[2] + w * (D / 2);
      if (warp_live) {
#pragma unroll
        for (int ch = 0; ch < D / 64; ++ch) {
          uint32_t va[32], vb[32];
          const uint32_t col = w * (D / 2) + 32 * ch;
          tmem_ld32(tmem + lane_base + col_o<D>(0) + col, va);
          tmem_ld32(tmem + lane_base + col_o<D>(1) + col, vb);
          float y[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) y[i] = __uint_as_float(va[i]) * f0 + __uint_as_float(vb[i]) * f1;
          if (whole) {
            if (live) {
#pragma unroll
              for (int i = 0; i < 4; ++i)
                *reinterpret_cast<uint4*>(o + 32 * ch + 8 * i) =
                    make_uint4(pack_bf16x2(y[8 * i], y[8 * i + 1]), pack_bf16x2(y[8 * i + 2], y[8 * i + 3]),
                               pack_bf16x2(y[8 * i + 4], y[8 * i + 5]), pack_bf16x2(y[8 * i + 6], y[8 * i + 7]));
            }
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
              reinterpret_cast<float4*>(part)[(col / 4 + i) * kRows + row] =
                  make_float4(y[4 * i], y[4 * i + 1], y[4 * i + 2], y[4 * i + 3]);
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar.o_free());
      if (whole) {
        if (live && w == 0) p.lse[(static_cast<size_t>(b) * p.H + h) * p.N + tok] = out_lse(m, lsum);
      } else {
        if (w == 0) {
          float* x = part + kRows * D + row;
          x[0] = m, x[kRows] = mva, x[2 * kRows] = lsum;
        }
        int part_no = static_cast<int>(blockIdx.x) - cta0;
        bool group = false;
        while (true) {
          if (!sync_softmax()) break;  // all of the partial result is written
          int* word = words + kLineWords;
          if (tid == 0) {
            Join x;
            word[0] = part_arrives<kOnce, kFan>(p, cta0, part_no, parts, group, x);
            word[1] = x.first, word[2] = x.stride, word[3] = x.n, word[4] = x.last;
          }
          if (!sync_softmax()) break;
          if (!word[0]) break;
          const int n = word[3], last_join = word[4];
          part_no = word[1];
          group = true;
          float jm = kNoScore, jmv = kNoProduct, jl = 0.f;
          if (warp_live) {
            // the parts in the order of the keys: this thread's row and half of its columns
            const int stride = word[2];
            auto part_at = [&](int i) {
              const int x = part_no + i * stride;
              return p.partial + (static_cast<size_t>(cta0 + x) * 2 + (x == 0 ? 1 : 0)) * part_floats(D);
            };
#pragma unroll 4
            for (int i = 0; i < n; ++i) jm = fmaxf(jm, __ldcg(part_at(i) + kRows * D + row));
#pragma unroll 4
            for (int i = 0; i < n; ++i) {
              const float* x = part_at(i) + kRows * D + row;
              const float dm = __ldcg(x) - jm;
              jmv = fmaxf(jmv, __ldcg(x + kRows) + dm);
              jl += __ldcg(x + 2 * kRows) * ex2(dm);
            }
            const float fin = last_join ? out_factor(jmv, jl, kPShift) : 1.f;
            float* sum = p.partial + (static_cast<size_t>(cta0 + part_no) * 2 + (part_no == 0 ? 1 : 0)) * part_floats(D);
#pragma unroll 1
            for (int ch = 0; ch < D / 32; ++ch) {
              const int col = w * (D / 2) + 16 * ch;
              float y[16];
#pragma unroll
              for (int i = 0; i < 16; ++i) y[i] = 0.f;
#pragma unroll 4
              for (int i = 0; i < n; ++i) {
                const float *x = part_at(i), *st = x + kRows * D + row;
                const float fx = ex2(__ldcg(st + kRows) + (__ldcg(st) - jm) - jmv);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                  const float4 v = __ldcg(reinterpret_cast<const float4*>(x) + (col / 4 + j) * kRows + row);
                  y[4 * j] += v.x * fx;
                  y[4 * j + 1] += v.y * fx;
                  y[4 * j + 2] += v.z * fx;
                  y[4 * j + 3] += v.w * fx;
                }
              }
              if (!last_join) {
                // (only this thread reads these places of the group's first part)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                  reinterpret_cast<float4*>(sum)[(col / 4 + j) * kRows + row] =
                      make_float4(y[4 * j], y[4 * j + 1], y[4 * j + 2], y[4 * j + 3]);
              } else if (live) {
#pragma unroll
                for (int i = 0; i < 2; ++i)
                  *reinterpret_cast<uint4*>(o + 16 * ch + 8 * i) = make_uint4(
                      pack_bf16x2(y[8 * i] * fin, y[8 * i + 1] * fin), pack_bf16x2(y[8 * i + 2] * fin, y[8 * i + 3] * fin),
                      pack_bf16x2(y[8 * i + 4] * fin, y[8 * i + 5] * fin), pack_bf16x2(y[8 * i + 6] * fin, y[8 * i + 7] * fin));
              }
            }
            if (last_join && live && w == 0) p.lse[(static_cast<size_t>(b) * p.H + h) * p.N + tok] = out_lse(jm, jl);
          }
          if (last_join) break;
          if (!sync_softmax()) break;  // the statistics of the group's first part have been read
          if (warp_live && w == 0) {
            float* x = p.partial + (static_cast<size_t>(cta0 + part_no) * 2 + (part_no == 0 ? 1 : 0)) * part_floats(D) +
                       kRows * D + row;
            x[0] = jm, x[kRows] = jmv, x[2 * kRows] = jl;
          }
        }
        if (!ok) break;
      }
      if (!sync_softmax()) break;  // red (Q's place) and the word have been read
    }

    // segments without a visible page: O = 0, LSE = -inf
    for (int sg = blockIdx.x; ok && line.any_empty && sg < nseg; sg += gridDim.x) {
      if (steps_of<kVec>(p, geo, sg) != 0) continue;
      const int bh = geo.by_RT.div(sg), rt2 = sg - bh * geo.RT, b2 = geo.by_Hk.div(bh), hk2 = bh - b2 * p.c.Hk;
      const RowTile r = row_tile(p, geo, b2, rt2, tid == 0);
      const int row_hi = min(geo.G * r.live, (rt2 + 1) * kRows);
      for (int rr = rt2 * kRows + warp; rr < row_hi; rr += 8) {
        const int t = geo.by_G.div(rr), hh = hk2 * geo.G + rr - t * geo.G;
        uint16_t* o = p.o + b2 * p.os[0] + hh * p.os[1] + t * p.os[2];
        for (int i = lane; i < D / 2; i += 32) *reinterpret_cast<uint32_t*>(o + 2 * i) = 0u;
        if (lane == 0) p.lse[(static_cast<size_t>(b2) * p.H + hh) * p.N + t] = -INFINITY;
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int D, bool kVec>
cudaError_t launch_t(const CacheFwdParams& p, const Geometry& geo, int num_sms, cudaStream_t s) {
  static std::atomic<uint64_t> done[4];  // devices whose kernel has its shared memory
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev > 255) return cudaErrorInvalidDevice;
  if (!(done[dev >> 6].load(std::memory_order_relaxed) >> (dev & 63) & 1)) {
    e = cudaFuncSetAttribute(cache_fwd_rows_kernel<D, kVec>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             Layout<D>::kBytes);
    if (e != cudaSuccess) return e;
    done[dev >> 6].fetch_or(1ull << (dev & 63), std::memory_order_relaxed);
  }
  if (kVec) {
    e = launch_cache_classify(p, geo, s);
    if (e != cudaSuccess) return e;
  }
  const int grid = num_sms < kCacheMaxCtas ? num_sms : kCacheMaxCtas;
  cache_fwd_rows_kernel<D, kVec><<<grid, kThreads, Layout<D>::kBytes, s>>>(p, geo);
  return cudaGetLastError();
}

}  // namespace

size_t cache_fwd_rows_part_floats(int d) { return part_floats(d); }

cudaError_t launch_cache_fwd_rows(int d, const CacheFwdParams& p, const Geometry& geo, int num_sms,
                                  cudaStream_t s) {
  const bool vec = p.mask.lts != nullptr || p.mask.uts != nullptr;
  if (d == 64) return vec ? launch_t<64, true>(p, geo, num_sms, s) : launch_t<64, false>(p, geo, num_sms, s);
  return vec ? launch_t<128, true>(p, geo, num_sms, s) : launch_t<128, false>(p, geo, num_sms, s);
}

}  // namespace fm
