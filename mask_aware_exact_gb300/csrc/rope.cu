// Rotary positions of Q and K, and their gradient (the same map with the angle
// negated): pair i of a token at position t turns by t * freqs[i].
//
// The angle only matters modulo a turn, and a far position times an fp32
// frequency has no correct digits left there. So the frequency is held in
// turns per position as a 64-bit fraction, f = freqs[i] / (2 pi) mod 1, and t *
// f is a 64-bit integer product whose overflow is the reduction modulo one
// turn: right to |t| * 2^-63 turns, whatever f, with no fp64 arithmetic (a few results
// per clock and SM on this GPU). The upper 32 bits, read as a signed fraction
// of half turns, go to sincospif.
//
// HBM-bound: every element is read and written once. A thread owns kVec pairs
// of one token and walks over heads of Q and K with the same sine and cosine,
// so their cost (about 50 instructions a pair) is spread over the heads. Its
// 16-byte pieces of the next kStages heads are always on their way into its own
// slots of shared memory (asynchronous copies, no registers held, no thread waits
// for another). A head's pieces are read before they are written and no other
// thread touches them, so the call is correct in place.
//
// Measured: 32768 tokens, 32 + 32 heads of 128 in bf16, 159 us, 6.7 TB/s, 99 % of a
// copy; the gradient for 2 x 16384 tokens, 32 + 8 heads, half of each turned in
// interleaved pairs, 100 us, 99 %. One token of each of 64 sequences: 2.9 us, which is
// a launch and two trips to memory.
#include <algorithm>

#include "cache.h"
#include "flashmask.h"
#include "rope_common.cuh"

namespace fm {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kBlocksPerSm = 4;  // resident at once
constexpr int kHeadsMost = 16;
constexpr int kStages = 4;  // heads in flight per thread
constexpr int kAtOnce = 8;  // heads loaded at a time when the elements are accessed one by one

// kVec elements per access. A chunk of a token's head is kVec pairs in two accesses
// half the rotated part apart, whatever the layout, so that each access of a warp
// is contiguous (16-byte halves of a sector would each fetch the whole one); one
// pair when kVec is 1. Chunks behind the rotated ones copy two accesses.
template <typename T, int kVec, bool kInterleaved>
__global__ void __launch_bounds__(kRopeThreads, 4) rope_kernel(const RopeParams p, int heads_each) {
  using V = Vec<T, kVec>;
  constexpr bool kAsync = sizeof(V) == 16;
  __shared__ V slots[kAsync ? kStages : 1][2][kAsync ? kRopeThreads : 1];
  const int n = p.rot / 2;
  const int rot_chunks = n / kVec;
  const int copy_chunks = (p.d - p.rot + 2 * kVec - 1) / (2 * kVec);
  const int chunks = rot_chunks + copy_chunks;
  const long long id = static_cast<long long>(blockIdx.x) * kRopeThreads + threadIdx.x;
  const long long token = id / chunks;
  if (token >= static_cast<long long>(p.B) * p.N) return;
  const int chunk = static_cast<int>(id - token * chunks);
  const int b = static_cast<int>(token) / p.N, t = static_cast<int>(token) - b * p.N;
  const bool rotated = chunk < rot_chunks;

  // element offsets of the chunk's two accesses within a head
  int e0, e1;
  bool two = true;
  if (rotated) {
    e0 = kInterleaved && kVec == 1 ? 2 * chunk : kVec * chunk;
    e1 = kInterleaved && kVec == 1 ? e0 + 1 : e0 + n;
  } else {
    e0 = p.rot + kVec * (chunk - rot_chunks);
    e1 = e0 + kVec * copy_chunks;
    two = e1 < p.d;
  }

  const int H = p.t[0].H + p.t[1].H;
  const int h0 = blockIdx.y * heads_each, h1 = min(H, h0 + heads_each);
  auto source = [&](int h) {
    const bool first = h < p.t[0].H;
    const RopeTensor& r = p.t[first ? 0 : 1];
    return static_cast<const T*>(r.x) + b * r.xs[0] + (first ? h : h - p.t[0].H) * r.xs[1] + t * r.xs[2];
  };
  auto fetch = [&](int h, int slot) {
    if constexpr (kAsync) {
      if (h < h1) {
        const T* src = source(h);
        copy16(&slots[slot][0][threadIdx.x], src + e0);
        if (two) copy16(&slots[slot][1][threadIdx.x], src + e1);
      }
      copy_commit();
    }
  };
#pragma unroll
  for (int i = 0; i < kStages; ++i) fetch(h0 + i, i);

  float cs[kVec], sn[kVec];
#pragma unroll
  for (int i = 0; i < kVec; ++i) cs[i] = 1.f, sn[i] = 0.f;
  if (rotated) {
    const int pos = p.positions ? p.positions[b * p.pos_stride + t] : t;
    // interleaved: the first access holds pairs e0 / 2 .., the second pairs e1 / 2 ..
    auto freq = [&](int i) {
      return p.freqs[!kInterleaved || kVec == 1 ? kVec * chunk + i : (i < kVec / 2 ? e0 : e1 - kVec) / 2 + i];
    };
    sines_of(pos, p.mscale, p.inverse, freq, cs, sn);
  }

  auto finish = [&](int h, V x0, V x1) {
    const bool first = h < p.t[0].H;
    const RopeTensor& r = p.t[first ? 0 : 1];
    T* dst = static_cast<T*>(r.y) + b * r.ys[0] + (first ? h : h - p.t[0].H) * r.ys[1] + t * r.ys[2];
    if (rotated) {
      V y0, y1;
#pragma unroll
      for (int i = 0; i < kVec; ++i) {
        // pair i: element i of both accesses, or elements 2 i and 2 i + 1 of the two in a row
        float a, c;
        if constexpr (!kInterleaved) {
          a = to_f<T>(x0.e[i]);
          c = to_f<T>(x1.e[i]);
        } else {
          a = to_f<T>(2 * i < kVec ? x0.e[(2 * i) % kVec] : x1.e[(2 * i) % kVec]);
          c = to_f<T>(2 * i + 1 < kVec ? x0.e[(2 * i + 1) % kVec] : x1.e[(2 * i + 1) % kVec]);
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
      x0 = y0;
      x1 = y1;
    }
    *reinterpret_cast<V*>(dst + e0) = x0;
    if (two) *reinterpret_cast<V*>(dst + e1) = x1;
  };
  if constexpr (kAsync) {
    int slot = 0;
    for (int h = h0; h < h1; ++h) {
      copy_wait<kStages - 1>();
      const V x0 = slots[slot][0][threadIdx.x];
      V x1 = x0;
      if (two) x1 = slots[slot][1][threadIdx.x];
      finish(h, x0, x1);
      fetch(h + kStages, slot);
      slot = slot + 1 == kStages ? 0 : slot + 1;
    }
  } else {
    for (int h = h0; h < h1; h += kAtOnce) {
      V x0[kAtOnce], x1[kAtOnce];
#pragma unroll
      for (int i = 0; i < kAtOnce; ++i) {
        if (h + i >= h1) break;
        const T* src = source(h + i);
        x0[i] = *reinterpret_cast<const V*>(src + e0);
        if (two) x1[i] = *reinterpret_cast<const V*>(src + e1);
      }
#pragma unroll
      for (int i = 0; i < kAtOnce; ++i) {
        if (h + i >= h1) break;
        finish(h + i, x0[i], x1[i]);
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
  // Heads per thread: as many as leave all SMs full, so that short calls spread over the
  // GPU, and at most kHeadsMost: by then the sines cost little, and more blocks even out
  // the end (32768 tokens x 64 heads: 16 heads 171 us, 64 heads 178 us, 4 heads 216 us).
  const long long want = static_cast<long long>(kBlocksPerSm) * num_sms;
  const int each = static_cast<int>(std::min<long long>(kHeadsMost, std::max(1LL, H * blocks / want)));
  const int groups = (H + each - 1) / each;
  if (groups > 65535) return cudaErrorInvalidValue;
  const dim3 grid(static_cast<unsigned>(blocks), static_cast<unsigned>(groups));
  if (p.interleaved)
    rope_kernel<T, kVec, true><<<grid, kRopeThreads, 0, s>>>(p, each);
  else
    rope_kernel<T, kVec, false><<<grid, kRopeThreads, 0, s>>>(p, each);
  return cudaGetLastError();
}

// 16-byte accesses need every row to start on a 16-byte boundary and the rotated
// pairs and the rest to be whole accesses; else one element at a time, which the
// instructions bound: 32768 tokens x 64 heads of 128 in bf16 take 159 us with 16-byte
// accesses, 401 us without.
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
