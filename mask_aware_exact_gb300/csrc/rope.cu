// Rotary positions of Q and K, and their gradient (the same map with the angle
// negated): pair i of a token at position t turns by t * freqs[i].
//
// The angle only matters modulo a turn, and a far position times an fp32
// frequency has no correct digits left there. So the frequency is held in
// turns per position as a 64-bit fraction, f = freqs[i] / (2 pi) mod 1, and t *
// f is a 64-bit integer product whose overflow is the reduction modulo one
// turn: exact up to |t| * 2^-64 turns, with no fp64 arithmetic (a few results
// per clock and SM on this GPU). The upper 32 bits, read as a signed fraction
// of half turns, go to sincospif.
//
// HBM-bound: every element is read and written once. A thread owns kVec pairs
// of one token and walks over heads of Q and K with the same sine and cosine,
// so their cost (about 25 instructions a pair) is spread over the heads and
// hides behind the loads. It handles kUnroll heads at a time, all loads before
// the first store, which keeps 2 * kUnroll 16-byte loads in flight per thread
// and makes the call correct in place.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "cache.h"
#include "flashmask.h"

namespace fm {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kUnroll = 4;

// f / (2 pi) modulo one turn as a 64-bit fraction, from the bits of the fp64
// f: mantissa times the first 64 bits of 2 / pi, shifted by the exponent. The
// relative error is below 2^-62.
__device__ __forceinline__ uint64_t turns_per_position(double f, bool& finite) {
  const uint64_t u = static_cast<uint64_t>(__double_as_longlong(f));
  const int ex = static_cast<int>((u >> 52) & 0x7ffu);
  finite = ex != 0x7ff;
  if (ex == 0) return 0;  // zero and denormals: less than 2^-1000 turns
  const uint64_t mant = (u & 0xfffffffffffffull) | (1ull << 52);
  constexpr uint64_t kTwoOverPi = 0xA2F9836E4E441529ull;  // floor(2 / pi * 2^64)
  // f = mant * 2^(ex - 1075); f / (2 pi) * 2^64 = hi * 2^(ex - 1024)
  const uint64_t hi = __umul64hi(mant << 11, kTwoOverPi);
  const int sh = ex - 1024;
  uint64_t r;
  if (sh <= 0)
    r = sh > -64 ? hi >> -sh : 0;
  else
    r = sh < 64 ? hi << sh : 0;
  return (u >> 63) ? 0ull - r : r;
}

template <typename T>
__device__ __forceinline__ float to_f(T v);
template <>
__device__ __forceinline__ float to_f<float>(float v) { return v; }
template <>
__device__ __forceinline__ float to_f<__half>(__half v) { return __half2float(v); }
template <>
__device__ __forceinline__ float to_f<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T>
__device__ __forceinline__ T from_f(float v);
template <>
__device__ __forceinline__ float from_f<float>(float v) { return v; }
template <>
__device__ __forceinline__ __half from_f<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// V consecutive elements moved by one access (V * sizeof(T) = 16, or V = 1).
template <typename T, int V>
struct alignas(V * sizeof(T)) Vec {
  T e[V];
};

// kVec elements per access. A chunk of a token's head is kVec pairs: in the half
// layout two accesses, at i and i + n; interleaved, two accesses side by side.
// Chunks behind the rotated ones copy 2 * kVec elements.
template <typename T, int kVec, bool kInterleaved>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const RopeParams p, int heads_each) {
  using V = Vec<T, kVec>;
  const int n = p.rot / 2;
  const int rot_chunks = n / kVec;
  const int chunks = rot_chunks + (p.d - p.rot + 2 * kVec - 1) / (2 * kVec);
  const long long id = static_cast<long long>(blockIdx.x) * kRopeThreads + threadIdx.x;
  const long long token = id / chunks;
  if (token >= static_cast<long long>(p.B) * p.N) return;
  const int chunk = static_cast<int>(id - token * chunks);
  const int b = static_cast<int>(token / p.N), t = static_cast<int>(token - static_cast<long long>(b) * p.N);
  const bool rotated = chunk < rot_chunks;

  // element offsets of the chunk's two accesses within a head
  int e0, e1;
  bool two = true;
  if (rotated) {
    e0 = kInterleaved ? 2 * kVec * chunk : kVec * chunk;
    e1 = kInterleaved ? e0 + kVec : e0 + n;
  } else {
    e0 = p.rot + 2 * kVec * (chunk - rot_chunks);
    e1 = e0 + kVec;
    two = e1 < p.d;
  }

  float cs[kVec], sn[kVec];
#pragma unroll
  for (int i = 0; i < kVec; ++i) cs[i] = 1.f, sn[i] = 0.f;
  if (rotated) {
    const int pos = p.positions ? p.positions[b * p.pos_stride + t] : t;
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      bool finite;
      const uint64_t f = turns_per_position(p.freqs[kVec * chunk + i], finite);
      const uint64_t a = static_cast<uint64_t>(static_cast<int64_t>(pos)) * f;
      // the top 32 bits in units of half turns, in [-1, 1)
      const float half_turns =
          static_cast<float>(static_cast<int32_t>(a >> 32)) * 4.656612873077393e-10f;  // 2^-31
      sincospif(half_turns, &sn[i], &cs[i]);
      const float c = finite ? p.mscale : __int_as_float(0x7fffffff);
      cs[i] *= c;
      sn[i] *= p.inverse ? -c : c;
    }
  }

  const int H = p.t[0].H + p.t[1].H;
  const int h0 = blockIdx.y * heads_each, h1 = min(H, h0 + heads_each);
  for (int h = h0; h < h1; h += kUnroll) {
    V x0[kUnroll], x1[kUnroll];
    T* dst[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int hh = h + u;
      const bool live = hh < h1;
      const RopeTensor& r = p.t[hh < p.t[0].H ? 0 : 1];
      const int hl = hh < p.t[0].H ? hh : hh - p.t[0].H;
      dst[u] = nullptr;
      if (live) {
        const T* src = static_cast<const T*>(r.x) + b * r.xs[0] + hl * r.xs[1] + t * r.xs[2];
        dst[u] = static_cast<T*>(r.y) + b * r.ys[0] + hl * r.ys[1] + t * r.ys[2];
        x0[u] = *reinterpret_cast<const V*>(src + e0);
        if (two) x1[u] = *reinterpret_cast<const V*>(src + e1);
      }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      if (dst[u] == nullptr) continue;
      if (rotated) {
        V y0, y1;
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
          // pair i: elements (i, i + n) or (2i, 2i + 1)
          float a, c;
          if constexpr (!kInterleaved) {
            a = to_f<T>(x0[u].e[i]);
            c = to_f<T>(x1[u].e[i]);
          } else {
            a = to_f<T>(2 * i < kVec ? x0[u].e[(2 * i) % kVec] : x1[u].e[(2 * i) % kVec]);
            c = to_f<T>(2 * i + 1 < kVec ? x0[u].e[(2 * i + 1) % kVec] : x1[u].e[(2 * i + 1) % kVec]);
          }
          const T ya = from_f<T>(a * cs[i] - c * sn[i]);
          const T yc = from_f<T>(c * cs[i] + a * sn[i]);
          if constexpr (!kInterleaved) {
            y0.e[i] = ya;
            y1.e[i] = yc;
          } else {
            if (2 * i < kVec) y0.e[(2 * i) % kVec] = ya; else y1.e[(2 * i) % kVec] = ya;
            if (2 * i + 1 < kVec) y0.e[(2 * i + 1) % kVec] = yc; else y1.e[(2 * i + 1) % kVec] = yc;
          }
        }
        *reinterpret_cast<V*>(dst[u] + e0) = y0;
        *reinterpret_cast<V*>(dst[u] + e1) = y1;
      } else {
        *reinterpret_cast<V*>(dst[u] + e0) = x0[u];
        if (two) *reinterpret_cast<V*>(dst[u] + e1) = x1[u];
      }
    }
  }
}

template <typename T, int kVec>
cudaError_t launch_rope_t(const RopeParams& p, int num_sms, cudaStream_t s) {
  const int chunks = p.rot / 2 / kVec + (p.d - p.rot + 2 * kVec - 1) / (2 * kVec);
  const long long threads = static_cast<long long>(p.B) * p.N * chunks;
  const long long blocks = (threads + kRopeThreads - 1) / kRopeThreads;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
  const int H = p.t[0].H + p.t[1].H;
  // Heads per thread: as many as leave four blocks for every SM, so that long
  // calls share the sines over all heads and short ones spread over the GPU.
  int groups = static_cast<int>((4LL * num_sms + blocks - 1) / blocks);
  const int most = (H + kUnroll - 1) / kUnroll;
  if (groups > most) groups = most;
  int each = (H + groups - 1) / groups;
  each = (each + kUnroll - 1) / kUnroll * kUnroll;
  groups = (H + each - 1) / each;
  if (groups > 65535) return cudaErrorInvalidValue;
  const dim3 grid(static_cast<unsigned>(blocks), static_cast<unsigned>(groups));
  if (p.interleaved)
    rope_kernel<T, kVec, true><<<grid, kRopeThreads, 0, s>>>(p, each);
  else
    rope_kernel<T, kVec, false><<<grid, kRopeThreads, 0, s>>>(p, each);
  return cudaGetLastError();
}

// 16-byte accesses need every row to start on a 16-byte boundary and the rotated
// pairs and the rest to be whole accesses; else one element at a time.
template <typename T>
cudaError_t launch_rope_d(const RopeParams& p, int num_sms, cudaStream_t s) {
  constexpr int kVec = 16 / sizeof(T);
  bool vec = p.d % kVec == 0 && (p.rot / 2) % kVec == 0;
  for (const RopeTensor& t : p.t) {
    if (t.H == 0) continue;
    vec = vec && (reinterpret_cast<uintptr_t>(t.x) & 15u) == 0 &&
          (reinterpret_cast<uintptr_t>(t.y) & 15u) == 0;
    for (int i = 0; i < 3; ++i) vec = vec && t.xs[i] % kVec == 0 && t.ys[i] % kVec == 0;
  }
  return vec ? launch_rope_t<T, kVec>(p, num_sms, s) : launch_rope_t<T, 1>(p, num_sms, s);
}

}  // namespace

cudaError_t launch_rope(const RopeParams& p, int dtype, int num_sms, cudaStream_t s) {
  if (dtype == FM_F32) return launch_rope_d<float>(p, num_sms, s);
  if (dtype == FM_F16) return launch_rope_d<__half>(p, num_sms, s);
  return launch_rope_d<__nv_bfloat16>(p, num_sms, s);
}

}  // namespace fm
