// Writes new tokens into the 8-bit paged cache. One CTA per (sequence, head,
// page that the call touches): reads the page's new K and V rows once, finds
// the scales, rounds to e4m3 and stores; V is transposed through shared memory
// because its pages hold the tokens of a column together.
//
// The scale of a page and head is the smallest power of two 2^k (k >= -100) with
// absmax <= 448 * 2^k. A power of two costs e4m3 nothing (a code's relative
// error does not depend on the scale while it is normal) and makes the growth
// of a half-filled page exact: its old codes are multiplied by 2^-n, which only
// rounds where they become subnormal.
//
// HBM-bound for prompts: 4 bytes read and 2 written per (K, V) element pair.
// All loads of a thread are issued before the first is used; the page's two barriers
// (its scale needs every row) are covered by the other three CTAs of the SM. 4 x 8192
// tokens, 8 heads of 128: 32.4 us, 5.3 TB/s, 78 % of a copy; with registers held down
// for five CTAs 32.6 us, for six 34.8, for eight 46.9. One token of each of 64
// sequences: 5 us, the trip to the table between two others.
#include "cache.h"
#include "ptx_fp8.cuh"

namespace fm {
namespace {

constexpr int kAppendThreads = 256;
constexpr int kMinExp = -100;

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// Largest magnitude of the 8 bf16 of a chunk, as bf16 bits (ordered like the
// values; infinities and NaN are >= 0x7f80).
__device__ __forceinline__ uint32_t absbits8(const uint4& q) {
  const uint32_t m = 0x7fff7fffu;
  const uint32_t a = __vmaxu2(__vmaxu2(q.x & m, q.y & m), __vmaxu2(q.z & m, q.w & m));
  return max(a & 0xffffu, a >> 16);
}

// Exponent k of the smallest power of two with absmax <= 448 * 2^k (448 = 1.75 *
// 2^8), from bf16 bits of a finite absmax.
__device__ __forceinline__ int scale_exponent(uint32_t absbits) {
  if (absbits == 0) return kMinExp;
  const uint32_t u = absbits << 16;
  const int e = static_cast<int>(u >> 23) - 127;  // denormals: -127, below every kept exponent
  const int k = (u & 0x7fffffu) <= 0x600000u ? e - 8 : e - 7;
  return max(k, kMinExp);
}

__device__ __forceinline__ float pow2(int k) { return __int_as_float((k + 127) << 23); }

// 8 bf16 times inv -> 8 e4m3 codes
__device__ __forceinline__ uint2 codes8(const uint4& q, float inv) {
  return make_uint2(pack_e4m3x4(bf_lo(q.x) * inv, bf_hi(q.x) * inv, bf_lo(q.y) * inv, bf_hi(q.y) * inv),
                    pack_e4m3x4(bf_lo(q.z) * inv, bf_hi(q.z) * inv, bf_lo(q.w) * inv, bf_hi(q.w) * inv));
}

// Four codes times f (a power of two <= 1), rounded again.
__device__ __forceinline__ uint32_t rescale4(uint32_t w, float f) {
  uint32_t lo, hi;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(lo) : "h"(static_cast<uint16_t>(w & 0xffffu)));
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(hi) : "h"(static_cast<uint16_t>(w >> 16)));
  float v[4];
  asm("{.reg .f16 a, b; mov.b32 {a, b}, %2; cvt.f32.f16 %0, a; cvt.f32.f16 %1, b;}" : "=f"(v[0]), "=f"(v[1]) : "r"(lo));
  asm("{.reg .f16 a, b; mov.b32 {a, b}, %2; cvt.f32.f16 %0, a; cvt.f32.f16 %1, b;}" : "=f"(v[2]), "=f"(v[3]) : "r"(hi));
  return pack_e4m3x4(v[0] * f, v[1] * f, v[2] * f, v[3] * f);
}

// A thread holds one 16-byte chunk (8 columns) of kEach consecutive slots of the
// page, for K and for V, so that the codes of a V column leave it as one word.
template <int D>
__global__ void __launch_bounds__(kAppendThreads) append_kernel(const AppendParams p) {
  constexpr int kRowChunks = D / 8;                             // 16-byte chunks of a row
  constexpr int kEach = kPage * kRowChunks / kAppendThreads;    // 4 or 2
  constexpr int kVRow = kPage + 4;  // bytes of a column in shared memory: a word stride of 17
  __shared__ uint32_t kmax[kPage], vmax[kPage];
  __shared__ int exps[2];
  __shared__ __align__(16) uint8_t vt[D * kVRow];

  const int b = blockIdx.x, h = blockIdx.y, tid = threadIdx.x;
  const int start = p.start[b];
  const int cnt = p.count ? min(max(p.count[b], 0), p.N) : p.N;
  if (cnt == 0) return;
  if (start < 0 || static_cast<long long>(start) + cnt > static_cast<long long>(p.max_pages) * kPage) {
    if (tid == 0 && h == 0 && blockIdx.z == 0) record_failure(p.status, kStatusPage, kSiteAppendRange);
    return;
  }
  const int page_i = start / kPage + static_cast<int>(blockIdx.z);
  const int first = page_i * kPage;                // position of slot 0
  const int lo = max(start - first, 0);            // first new slot
  const int hi = min(start + cnt - first, kPage);  // behind the last new slot
  if (lo >= hi) return;

  // the new rows: slot s holds token first + s - start
  uint4 kr[kEach], vr[kEach];
  const int c = tid % kRowChunks, s0 = tid / kRowChunks * kEach;
  const uint16_t* ksrc = p.k + b * p.ks[0] + h * p.ks[1] + 8 * c;
  const uint16_t* vsrc = p.v + b * p.vs[0] + h * p.vs[1] + 8 * c;
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int64_t tok = first + s0 + i - start;
    kr[i] = vr[i] = make_uint4(0u, 0u, 0u, 0u);
    if (s0 + i >= lo && s0 + i < hi) {
      kr[i] = __ldcs(reinterpret_cast<const uint4*>(ksrc + tok * p.ks[2]));
      vr[i] = __ldcs(reinterpret_cast<const uint4*>(vsrc + tok * p.vs[2]));
    }
  }
  const int page = p.table[static_cast<size_t>(b) * p.max_pages + page_i];
  if (page < 0 || page >= p.c.pages) {
    if (tid == 0 && h == 0) record_failure(p.status, kStatusPage, kSiteAppendPage);
    return;
  }
  const size_t ph = static_cast<size_t>(page) * p.c.Hk + h;
  const bool begun = lo > 0;  // the page holds older tokens
  float kold = 0.f, vold = 0.f;
  if (begun) {
    kold = p.c.kscale[ph];
    vold = p.c.vscale[ph];
  }

  // largest magnitude of every new token
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    uint32_t a = absbits8(kr[i]) << 16 | absbits8(vr[i]);
#pragma unroll
    for (int o = kRowChunks / 2; o > 0; o >>= 1) a = __vmaxu2(a, __shfl_xor_sync(0xffffffffu, a, o));
    if (c == 0) {
      kmax[s0 + i] = a >> 16;
      vmax[s0 + i] = a & 0xffffu;
    }
  }
  __syncthreads();
  if (tid < 32) {
    uint32_t a = 0, e = 0;
#pragma unroll
    for (int i = 0; i < kPage / 32; ++i) {
      const uint32_t x = kmax[tid + 32 * i], y = vmax[tid + 32 * i];
      if (x < 0x7f80u && y < 0x7f80u) {  // a token that is not finite does not count
        a = max(a, x);
        e = max(e, y);
      }
    }
    a = __reduce_max_sync(0xffffffffu, a);
    e = __reduce_max_sync(0xffffffffu, e);
    if (tid == 0) {
      exps[0] = scale_exponent(a);
      exps[1] = scale_exponent(e);
    }
  }
  __syncthreads();
  const float kneed = pow2(exps[0]), vneed = pow2(exps[1]);
  const float ks = begun ? fmaxf(kneed, kold) : kneed, vs = begun ? fmaxf(vneed, vold) : vneed;
  const float kinv = 1.f / ks, vinv = 1.f / vs;
  uint8_t* kp = p.c.k8 + ph * (kPage * D);
  uint8_t* vp = p.c.v8 + ph * (kPage * D);
  if (tid == 0) {
    p.c.kscale[ph] = ks;
    p.c.vscale[ph] = vs;
  }

  // K: rows of codes, zeros behind the last token of a page begun here; V: the
  // codes of each column into shared memory
  uint2 vc[kEach];
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int slot = s0 + i;
    const bool bad = kmax[slot] >= 0x7f80u || vmax[slot] >= 0x7f80u;
    vc[i] = bad ? make_uint2(0u, 0u) : codes8(vr[i], vinv);
    if ((slot >= lo && slot < hi) || !begun)
      *reinterpret_cast<uint2*>(kp + slot * D + 8 * c) =
          bad ? make_uint2(0x7f7f7f7fu, 0x7f7f7f7fu) : codes8(kr[i], kinv);
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    // byte j of each slot's codes, slots in order
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < kEach; ++i) w |= ((j < 4 ? vc[i].x : vc[i].y) >> (8 * (j & 3)) & 0xffu) << (8 * i);
    if constexpr (kEach == 4)
      *reinterpret_cast<uint32_t*>(vt + (8 * c + j) * kVRow + s0) = w;
    else
      *reinterpret_cast<uint16_t*>(vt + (8 * c + j) * kVRow + s0) = static_cast<uint16_t>(w);
  }
  // older codes of a page whose scale has grown
  if (begun && ks > kold) {
    const float f = kold * kinv;
    uint32_t* w = reinterpret_cast<uint32_t*>(kp);
    for (int i = tid; i < lo * (D / 4); i += kAppendThreads) w[i] = rescale4(w[i], f);
  }
  __syncthreads();
  if (!begun) {
    // whole columns, 64 bytes each, in 16-byte stores
    for (int i = tid; i < D * 4; i += kAppendThreads) {
      const uint32_t* src = reinterpret_cast<const uint32_t*>(vt + (i >> 2) * kVRow + (i & 3) * 16);
      reinterpret_cast<uint4*>(vp)[i] = make_uint4(src[0], src[1], src[2], src[3]);
    }
  } else {
    const int rows = hi - lo;
    for (int i = tid; i < D * rows; i += kAppendThreads) {
      const int col = i / rows, slot = lo + i - col * rows;
      vp[col * kPage + slot] = vt[col * kVRow + slot];
    }
    if (vs > vold) {
      const float f = vold * vinv;
      for (int i = tid; i < D * lo; i += kAppendThreads) {
        const int at = (i / lo) * kPage + i % lo;
        vp[at] = static_cast<uint8_t>(rescale4(vp[at], f));
      }
    }
  }
}

}  // namespace

cudaError_t launch_append(int d, const AppendParams& p, cudaStream_t s) {
  // pages that N tokens touch at most, wherever they start in a page
  const unsigned pages = static_cast<unsigned>((static_cast<long long>(p.N) + 2 * kPage - 2) / kPage);
  const dim3 grid(static_cast<unsigned>(p.B), static_cast<unsigned>(p.c.Hk), pages);
  if (d == 64)
    append_kernel<64><<<grid, kAppendThreads, 0, s>>>(p);
  else
    append_kernel<128><<<grid, kAppendThreads, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace fm
