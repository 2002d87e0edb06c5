// The attention weight that each cached key is given: for key j of a cache head the sum
// of exp(scale q k_j - LSE) over the query heads that read it and the query rows that see
// it, added to what the key had. Keys are independent of one another, so nothing is
// joined: a warp has a page, takes the products S^T = K Q^T of its 64 keys with 8 rows at
// a time (m16n8k16 with fp16 operands: codes are exact in fp16, queries scaled by a power
// of two as in the attention) and adds each key's exponentials over the rows.
//
// The pages of all (sequence, cache head) segments form one line, cut into equal runs,
// one for each warp. With a column-wise mask the line has only the pages that some row
// sees (the attention's classification, all rows as one tile). A warp brings its pages in
// by bulk copies, kSlots ahead, into slots of its own: no warp waits for another.
//
// Up to 32 rows, as 1, 2 or 4 groups of 8 (kWeightsMany says why not more). K is read
// once: 8 rows are bound by HBM, 32 by instructions (600 a page of d = 64) and their
// latencies, with two warps a scheduler: registers allow no more (9, 10 warps: 33, 31 us for
// the drafted tokens below where 8 took 28). Measured, calls with L2 flushed: 64 sequences up to 8192,
// 32 / 8 heads of 128: 63 us (342 MB, 5.4 TB/s); 8 sequences of 131072, window of 4096 and
// prefix of 2048, 8 / 8 heads: 25 us, 9 of them the classification of 131072 columns; 16
// sequences up to 16384, 4 tokens, 32 / 4 heads of 64: 25 us (42 MB); one sequence of 1000:
// 5.9 us on the GPU. 16 sequences of 16384, 4 heads, by rows (us; L2 warm):
//   rows        4      8     16     24     32
//   d = 64    14.7   14.7   16.8   22.9   22.9
//   d = 128   16.8   16.9   21.1   29.2   29.2
#include <atomic>

#include "cache_weights.cuh"
#include "flashmask.h"

namespace fm {
namespace {

// Warps of a CTA: as many as registers allow, 12 or 8 (16 of 128 registers for 8 rows: 63.0 us
// for the 64 sequences, 63.7 with 12, but 26.8 for the window where 12 take 25.2).
template <int D, int NT>
constexpr int kWarps = NT == 1 || (NT == 2 && D == 64) ? 12 : 8;
// Pages of a warp on their way or being read. (A third less: 64.3 us for the 64 sequences, 63.7
// so; the drafted tokens 27.0, 28.0 so.)
template <int D, int NT>
constexpr int kSlots = (D == 128 ? 24 : 48) / kWarps<D, NT>;
template <int D, int NT>
constexpr int kSmem = kWarps<D, NT> * kSlots<D, NT> * (kPage * D + 8);

// Up to 32 pages of a run, one per lane, and where the run goes on.
struct Batch {
  int n;                         // of all lanes
  int seg, logical, page, cut;   // page -1: there is none
  float kscale;
  int next_seg, next_k;
};

__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Bit i: key at[8 i] has s <= pos < e.
static __device__ __noinline__ uint32_t hidden_step8(const int32_t* s, const int32_t* e, int pos) {
  uint32_t hid = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) hid |= static_cast<uint32_t>(s[8 * i] <= pos && pos < e[8 * i]) << i;
  return hid;
}

// A lane's part of the 8 NT rows: the queries as second operands (row 8 t + lane /
// 4, elements 64 half + 16 (lane % 4) .. + 15), and of the rows 8 t + 2 (lane % 4) + e what
// turns S into weights.
template <int D, int NT>
struct Rows {
  uint32_t q[NT][D / 16][2];
  float crow[NT][2], lse2[NT][2];
  int lim[NT][2], pos[NT][2];
  size_t mrow[NT][2];
  int all_lim;  // keys that every row sees as far as causality and length go (0 if one may need score_boost)
};

template <int D, int NT, bool kVec>
__device__ __forceinline__ void load_rows(const WeightsParams& wp, const Geometry& geo, const RowTile& r, int b,
                                          int hk, Rows<D, NT>& o) {
  const CacheFwdParams& p = wp.f;
  const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  const int rows = geo.G * r.live;
  o.all_lim = r.len;
  // (all loads before the first use: group by group they would wait for one another)
  uint4 x[NT][D / 64][2];
  float lse[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int rr = 8 * t + g;
    const bool live = rr < rows;
    const int tok = geo.by_G.div(rr), h = hk * geo.G + rr - tok * geo.G;
    const uint16_t* src = p.q + b * p.qs[0] + h * p.qs[1] + tok * p.qs[2] + 16 * c;
#pragma unroll
    for (int hf = 0; hf < D / 64; ++hf)
#pragma unroll
      for (int u = 0; u < 2; ++u)
        x[t][hf][u] = live ? *reinterpret_cast<const uint4*>(src + 64 * hf + 8 * u) : make_uint4(0u, 0u, 0u, 0u);
    // rows that saw nothing, and those behind the last, give nothing; one whose LSE is NaN
    // counts as one whose query is (a NaN in S is dropped where the key is masked)
    lse[t] = live ? wp.lse[(static_cast<size_t>(b) * p.H + h) * p.N + tok] : -INFINITY;
  }
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    uint32_t top = 0;
#pragma unroll
    for (int hf = 0; hf < D / 64; ++hf)
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const uint32_t mk = 0x7fff7fffu;
        const uint4 v = x[t][hf][u];
        const uint32_t a = __vmaxu2(__vmaxu2(v.x & mk, v.y & mk), __vmaxu2(v.z & mk, v.w & mk));
        top = max(top, max(a & 0xffffu, a >> 16));
      }
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
    // the row's largest element goes to [2^14, 2^15): fp16 then holds every element down
    // to 2^-30 of it
    float l = lse[t];
    const bool bad = top >= 0x7f80u || isnan(l);
    l = isnan(l) ? 0.f : l == -INFINITY ? INFINITY : l * 1.4426950408889634f;
    const int up = top == 0 || bad ? 0 : min(14 - (static_cast<int>(top >> 7) - 127), 126);
    const float f = bad ? __int_as_float(0x7fffffff) : __int_as_float((up + 127) << 23);
#pragma unroll
    for (int hf = 0; hf < D / 64; ++hf)
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint4 w = x[t][hf][k >> 1];
        const uint32_t lo = k & 1 ? w.z : w.x, hi = k & 1 ? w.w : w.y;
        o.q[t][4 * hf + k][0] = pack_f16x2(__uint_as_float(lo << 16) * f, __uint_as_float(lo & 0xffff0000u) * f);
        o.q[t][4 * hf + k][1] = pack_f16x2(__uint_as_float(hi << 16) * f, __uint_as_float(hi & 0xffff0000u) * f);
      }
    const float crow = p.scale_log2 * __int_as_float((127 - up) << 23);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int rr2 = 8 * t + 2 * c + e;
      const bool live2 = rr2 < rows;
      const int tok2 = geo.by_G.div(rr2), h2 = hk * geo.G + rr2 - tok2 * geo.G;
      o.crow[t][e] = __shfl_sync(0xffffffffu, crow, 4 * (2 * c + e));
      o.pos[t][e] = r.shift + tok2;
      o.lim[t][e] = live2 ? (p.mask.causal ? min(r.len, o.pos[t][e] + 1) : r.len) : 0;
      o.lse2[t][e] = __shfl_sync(0xffffffffu, l, 4 * (2 * c + e));
      o.mrow[t][e] = kVec ? (static_cast<size_t>(b) * p.mask.Hm + geo.by_mask.div(h2)) *
                                static_cast<size_t>(p.max_pages * kPage)
                          : 0;
      // (a row behind the last hides nothing: it adds 0 wherever the others see a key)
      if (live2) o.all_lim = min(o.all_lim, o.crow[t][e] > 1.f ? 0 : o.lim[t][e]);
    }
  }
  o.all_lim = __reduce_min_sync(0xffffffffu, o.all_lim);
}

template <int D, int NT, bool kVec>
__global__ void __launch_bounds__(32 * kWarps<D, NT>, 1)
    cache_weights_kernel(const __grid_constant__ WeightsParams wp, const __grid_constant__ Geometry geo) {
  const CacheFwdParams& p = wp.f;
  constexpr int kW = kWarps<D, NT>, kThreads = 32 * kW, kRing = kSlots<D, NT>;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int wsum[kW], begin[kW][2];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
  const int nseg = p.B * p.c.Hk, grid = static_cast<int>(gridDim.x);
  uint8_t* const ring = smem + warp * kRing * kPage * D;
  const uint32_t bar = smem_u32(smem + kW * kRing * kPage * D) + 8 * kRing * warp;
  if (lane < kRing) {
    mbar_init(bar + 8 * lane, 1);
    fence_barrier_init();
  }
  auto units = [&](int s) { return line_pages<kVec>(p, geo, s); };

  if (kVec) wait_for_previous();  // its results are the lists of pages
  // this warp's run of the line (neighbouring runs go to different CTAs)
  const int each = (nseg + kThreads - 1) / kThreads;
  const int seg_lo = min(tid * each, nseg), seg_hi = min(seg_lo + each, nseg);
  int mine = 0;
  for (int s = seg_lo; s < seg_hi; ++s) mine += units(s);
  int total;
  const int before = block_before<kW>(mine, wsum, total);
  const int runs = grid * kW, run = (total + runs - 1) / runs;
  for (int w = 0; w < kW; ++w) {
    const long long x = static_cast<long long>(run) * (w * grid + static_cast<int>(blockIdx.x));
    if (before <= x && x < before + mine) {
      int s = seg_lo, at = before, n;
      // a thread with one segment knows its units
      while (x >= at + (n = each == 1 ? mine : units(s)) && s + 1 < seg_hi) at += n, ++s;
      begin[w][0] = s;
      begin[w][1] = static_cast<int>(x) - at;
    }
  }
  __syncthreads();
  const long long lo = static_cast<long long>(run) * (warp * grid + static_cast<int>(blockIdx.x));
  int left = static_cast<int>(max(0LL, min(static_cast<long long>(run), total - lo)));  // not in a batch yet

  // the next pages of the run
  auto next_batch = [&](int seg, int k) {
    Batch q = {};
    while (left > 0) {
      int my_k, my_n;
      q.n = next_units(seg, k, nseg, min(32, left), units, q.seg, my_k, my_n);
      if (q.n == 0) {
        seg += 32;
        k = 0;
        if (seg < nseg) continue;
        left = 0;  // the lengths are not those of the run's search any more
        break;
      }
      left -= q.n;
      q.page = -1;
      if (lane < q.n) {
        const int b = geo.by_Hk.div(q.seg), hk = q.seg - b * p.c.Hk;
        q.logical = page_on_line<kVec>(p, geo, b, hk, 0, my_k, q.cut);
        q.page = p.table[static_cast<size_t>(b) * p.max_pages + q.logical];
        if (q.page < 0 || q.page >= p.c.pages) {
          record_failure(p.status, kStatusPage, kSiteCachePage);
          q.page = -1;
        } else {
          q.kscale = p.c.kscale[static_cast<size_t>(q.page) * p.c.Hk + hk];
        }
      }
      q.next_seg = __shfl_sync(0xffffffffu, q.seg, q.n - 1);
      q.next_k = __shfl_sync(0xffffffffu, my_k, q.n - 1) + 1;
      break;
    }
    return q;
  };
  // The page of lane i on its way to slot x (a page that is not there reads another's, and
  // what comes of it is dropped).
  auto fetch = [&](const Batch& q, int i, int x) {
    if (lane == i) {
      const int hk = q.seg - geo.by_Hk.div(q.seg) * p.c.Hk;
      mbar_arrive_expect_tx(bar + 8 * x, kPage * D);
      bulk_load(smem_u32(ring + x * kPage * D), p.c.k8 + (static_cast<size_t>(max(q.page, 0)) * p.c.Hk + hk) * (kPage * D),
                kPage * D, bar + 8 * x);
    }
  };

  Rows<D, NT> rw;
  RowTile r = {};
  int cur = -1, start = 0;
  int slot = 0, turn = 0, ahead = 0;  // of the ring; pages fetched that are not done
  bool ok = true;
  Batch now = left > 0 ? next_batch(begin[warp][0], begin[warp][1]) : Batch{};
  for (; ahead < kRing && ahead < now.n; ++ahead) fetch(now, ahead, ahead);
  while (ok && now.n > 0) {
    // the batch behind this one is looked up while this one's pages are on their way
    const Batch then = next_batch(now.next_seg, now.next_k);
    for (int i = 0; ok && i < now.n; ++i) {
      const int pg = __shfl_sync(0xffffffffu, now.page, i), sg = __shfl_sync(0xffffffffu, now.seg, i);
      const int j0 = __shfl_sync(0xffffffffu, now.logical, i) * kPage, ct = __shfl_sync(0xffffffffu, now.cut, i);
      const float kscale = __shfl_sync(0xffffffffu, now.kscale, i);
      const int b = geo.by_Hk.div(sg), hk = sg - b * p.c.Hk;
      float* const wt = wp.weights + (static_cast<size_t>(max(pg, 0)) * p.c.Hk + hk) * kPage + 16 * c + g;
      const float old[2] = {wt[0], wt[8]};
      if (sg != cur) {
        r = row_tile(p, geo, b, 0, lane == 0);
        start = first_new(wp, b, r);
        load_rows<D, NT, kVec>(wp, geo, r, b, hk, rw);
        cur = sg;
      }
      const bool none = no_scales(kscale, 0.f);
      float sum[4][2] = {};
      ok = __all_sync(0xffffffffu, cache_wait(bar + 8 * slot, turn & 1, p.status));
      if (!ok) break;
      // (keys behind the last row's are seen by none)
      if (r.live > 0 && !(p.mask.causal && r.shift + r.live - 1 < j0)) {
        // instruction u has the keys 16 u + g and 16 u + 8 + g of this lane; halves of a row in
        // another order for odd keys, so that the eight lanes of a phase are in different banks
        const uint8_t* src = ring + slot * kPage * D + g * D + 16 * c;
        float s[4][NT][4] = {};
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          uint4 w[2][D / 64];
#pragma unroll
          for (int x = 0; x < 2; ++x)
#pragma unroll
            for (int hf = 0; hf < D / 64; ++hf)
              w[x][hf] = *reinterpret_cast<const uint4*>(src + (16 * u + 8 * x) * D + (D == 128 ? 64 * (hf ^ (g & 1)) : 0));
          if (D == 128 && (g & 1)) {
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const uint4 t = w[x][0];
              w[x][0] = w[x][D / 64 - 1];
              w[x][D / 64 - 1] = t;
            }
          }
#pragma unroll
          for (int hf = 0; hf < D / 64; ++hf)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              uint32_t a[4];
              codes_to_f16(word(w[0][hf], q), a[0], a[2]);
              codes_to_f16(word(w[1][hf], q), a[1], a[3]);
#pragma unroll
              for (int t = 0; t < NT; ++t) mma16816(s[u][t], a, rw.q[t][4 * hf + q][0], rw.q[t][4 * hf + q][1]);
            }
        }
        // s[u][t][2 x + e]: key 16 u + 8 x + g, row 8 t + 2 c + e
        float ck[NT][2];
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int e = 0; e < 2; ++e) ck[t][e] = score_factor(rw.crow[t][e], kscale);
        if (__builtin_expect(j0 + kPage > rw.all_lim || ct || none, 0)) {
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int n = min(max(rw.lim[t][e] - (j0 + g), 0), kPage);
              uint32_t see = (1u << ((n + 7) >> 3)) - 1u;  // bit i: key 8 i + g
              if constexpr (kVec) {
                if (ct) {
                  const size_t at = rw.mrow[t][e] + j0 + g;
                  if (p.mask.lts) see &= ~hidden_step8(p.mask.lts + at, p.mask.lte + at, rw.pos[t][e]);
                  if (p.mask.uts) see &= ~hidden_step8(p.mask.uts + at, p.mask.ute + at, rw.pos[t][e]);
                }
              }
              const float boost = score_boost(rw.crow[t][e], kscale, none, ck[t][e]);
#pragma unroll
              for (int u = 0; u < 4; ++u)
#pragma unroll
                for (int x = 0; x < 2; ++x)
                  s[u][t][2 * x + e] = (see >> (2 * u + x)) & 1u ? s[u][t][2 * x + e] * boost : -INFINITY;
            }
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          const uint64_t c2 = f2_make(ck[t][0], ck[t][1]), l2 = f2_make(-rw.lse2[t][0], -rw.lse2[t][1]);
#pragma unroll
          for (int u = 0; u < 4; ++u)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              float a, z;
              f2_split(f2_fma(f2_make(s[u][t][2 * x], s[u][t][2 * x + 1]), c2, l2), a, z);
              sum[u][x] += ex2(a) + ex2(z);
            }
        }
      }
      __syncwarp();
      // a page more, of this batch or the next
      for (--ahead; ahead < kRing; ++ahead) {
        const int q = i + 1 + ahead;
        int x = slot + 1 + ahead;
        if (x >= kRing) x -= kRing;
        if (q < now.n)
          fetch(now, q, x);
        else if (q - now.n < then.n)
          fetch(then, q - now.n, x);
        else
          break;
      }
      if (++slot == kRing) slot = 0, ++turn;
#pragma unroll
      for (int u = 0; u < 4; ++u)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          sum[u][x] += __shfl_xor_sync(0xffffffffu, sum[u][x], 1);
          sum[u][x] += __shfl_xor_sync(0xffffffffu, sum[u][x], 2);
        }
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int j = j0 + 16 * c + g + 8 * x;
        const float v = c == 0 ? sum[0][x] : c == 1 ? sum[1][x] : c == 2 ? sum[2][x] : sum[3][x];
        if (pg >= 0 && j < r.len) wt[8 * x] = j < start ? old[x] + v : v;
      }
    }
    now = then;
  }
  if (!ok) {
    // copies in flight land before the CTA's shared memory is given up
    for (int x = 0; x < ahead; ++x)
      mbar_wait_for(bar + 8 * ((slot + x) % kRing), (slot + x >= kRing ? turn + 1 : turn) & 1, nullptr, 1000000ull);
  }
  clear_unseen<kVec>(wp, geo, static_cast<int>(blockIdx.x) * kW + warp, runs);
}

template <int D, int NT, bool kVec>
cudaError_t launch_t(const WeightsParams& p, const Geometry& geo, int num_sms, cudaStream_t s) {
  static std::atomic<uint64_t> done[4];  // devices whose kernel has its shared memory
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev > 255) return cudaErrorInvalidDevice;
  if (!(done[dev >> 6].load(std::memory_order_relaxed) >> (dev & 63) & 1)) {
    e = cudaFuncSetAttribute(cache_weights_kernel<D, NT, kVec>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem<D, NT>);
    if (e != cudaSuccess) return e;
    done[dev >> 6].fetch_or(1ull << (dev & 63), std::memory_order_relaxed);
  }
  if (kVec) {
    e = launch_cache_classify(p.f, geo, s);
    if (e != cudaSuccess) return e;
  }
  if (kVec)
    return launch_overlapped(cache_weights_kernel<D, NT, kVec>, dim3(static_cast<unsigned>(num_sms)),
                             32 * kWarps<D, NT>, kSmem<D, NT>, s, p, geo);
  cache_weights_kernel<D, NT, kVec><<<num_sms, 32 * kWarps<D, NT>, kSmem<D, NT>, s>>>(p, geo);
  return cudaGetLastError();
}

template <int D, int NT>
cudaError_t launch_nt(const WeightsParams& p, const Geometry& geo, int num_sms, cudaStream_t s) {
  return p.f.mask.lts != nullptr || p.f.mask.uts != nullptr ? launch_t<D, NT, true>(p, geo, num_sms, s)
                                                            : launch_t<D, NT, false>(p, geo, num_sms, s);
}

template <int D>
cudaError_t launch_d(const WeightsParams& p, const Geometry& geo, int num_sms, cudaStream_t s) {
  if (geo.rows <= 8) return launch_nt<D, 1>(p, geo, num_sms, s);
  return geo.rows <= 16 ? launch_nt<D, 2>(p, geo, num_sms, s) : launch_nt<D, 4>(p, geo, num_sms, s);
}

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

}  // namespace

WeightsWs weights_ws_layout(int B, int H, int Hk, int N, int d, int max_pages) {
  const size_t segs = static_cast<size_t>(B) * Hk;
  const bool many = H / Hk * N >= kWeightsMany;
  WeightsWs w;
  // the status word and the counters, which have to be zero, lie at the same place for
  // all sizes, so that one workspace serves them in turn
  size_t off = 256;
  w.arrived = off;
  off = up256(off + kCacheMaxCtas * 8);
  w.partial = off;
  off = up256(off + (many ? static_cast<size_t>(kCacheMaxCtas) * 2 * 256 * 4 : 0));
  w.list = off;
  off = up256(off + segs * max_pages * 2);
  w.listed = off;
  off = up256(off + segs * 4);
  w.tiles = off;
  off = up256(off + (many ? segs * weights_row_tiles(H, Hk, N) * weights_tile_bytes(d) : 0));
  w.total = off;
  return w;
}

cudaError_t launch_cache_weights(int d, const WeightsParams& p, int num_sms, cudaStream_t s) {
  const Geometry geo = weights_geometry(p.f.H, p.f.c.Hk, p.f.mask.Hm, p.f.N, p.f.max_pages);
  if (geo.rows >= kWeightsMany) return launch_cache_weights_rows(d, p, geo, num_sms, s);
  return d == 64 ? launch_d<64>(p, geo, num_sms, s) : launch_d<128>(p, geo, num_sms, s);
}

}  // namespace fm
