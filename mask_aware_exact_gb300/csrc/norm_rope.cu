// Norm of every head of Q and K with the rotary positions in the same pass, and its
// gradients.
//
//   forward   y = R(x r w), r = 1 / sqrt(mean(x^2) + eps), R the rotation times mscale
//   backward  g = R^T dy, dw += g x r, dx = r (g w - x r mean(g w x r)); with s1 = sum
//             x^2 and s2 = sum g w x that is dx = r (g w) - x (r^3 s2 / d), so one
//             round of sums over a head gives both, and nothing is kept from the forward
//
// HBM-bound: every element is read and written once (the backward reads two). A head
// is shared by a group of lanes that holds it in registers, each its pairs (or a few of
// them), and adds its sums up by shuffles; a thread walks over heads with the same sines,
// weights and, backward, sums for dw, with 16-byte pieces of the next heads on their way
// into its own slots of shared memory. A thread reads its pieces of a head before it
// writes them and no other thread touches them, so the calls are correct in place.
//
// dw is a sum over tokens and heads: each thread sums what it walks over, a CTA adds its
// threads' sums in a fixed order and leaves them in the workspace, and a second kernel
// adds the CTAs' in order. No atomics: the same call gives the same bits.
//
// The arithmetic runs on pairs of elements (one by one the backward took 182 us where it
// takes 174), and a CTA turns the frequencies into turns a position once for all its tiles,
// in shared memory (174 -> 169 with the slots back at three).
//
// Measured (bf16 forward, 32768 tokens, 32 + 32 heads of 128, 1.07 GB): 160 us, 6.7 TB/s,
// 98 % of a copy. Backward (fp16, 2 x 16384 tokens, 32 + 8 heads of 128, half of each turned,
// interleaved, 1.01 GB): 167 us, 6.0 TB/s, 89 % of a copy; a scheduler issues in 61 % of the
// cycles and the two CTAs that fit an SM hide no more (three CTAs spill: 248 us; rings of 2,
// 3, 4, 5 heads: 174, 169, 171, 174; a ring that runs on into the next tile: 185 against 182
// then). One token of 64 sequences: 3.8 us on the GPU, two trips to memory; a call is the
// host's work for two tensors.
#include <algorithm>
#include <atomic>

#include "cache.h"
#include "flashmask.h"
#include "overlap.cuh"
#include "ptx.cuh"
#include "rope_common.cuh"

namespace fm {
namespace {

constexpr int kThreads = 256;
constexpr int kHeadsMost = 16;
// Heads in flight per thread, and the bytes of their slots.
__host__ __device__ constexpr int stages(bool backward) { return backward ? 3 : 4; }
__host__ __device__ constexpr int slot_bytes(bool backward) { return stages(backward) * (backward ? 4 : 2) * kThreads * 16; }

// The sum of a head's squares, or the magnitude of sum g w x, beyond which they are taken again
// of scaled values.
constexpr float kSumMost = 1e38f;

// Where a thread's chunk c (pairs, or elements that are not turned) lies in a head:
// accesses of kVec elements at e0 and, if `two`, at e1.
struct Chunk {
  int e0, e1;
  bool there, rotated, two;
};
template <int kVec, bool kInterleaved>
__device__ __forceinline__ Chunk chunk_at(int c, int d, int rot) {
  const int n = rot / 2, rot_chunks = n / kVec;
  const int copy_chunks = (d - rot + 2 * kVec - 1) / (2 * kVec);
  Chunk k;
  k.there = c < rot_chunks + copy_chunks;
  k.rotated = c < rot_chunks;
  if (k.rotated) {
    k.e0 = kInterleaved && kVec == 1 ? 2 * c : kVec * c;
    k.e1 = kInterleaved && kVec == 1 ? k.e0 + 1 : k.e0 + n;
    k.two = true;
  } else {
    k.e0 = rot + kVec * (c - rot_chunks);
    k.e1 = k.e0 + kVec * copy_chunks;
    k.two = k.there && k.e1 < d;
  }
  return k;
}

// Turns kVec pairs held as two accesses in a row, v[0 .. kVec) and v[kVec .. 2 kVec).
template <int kVec, bool kInterleaved>
__device__ __forceinline__ void turn(float* v, const float (&cs)[kVec], const float (&sn)[kVec]) {
  if constexpr (!kInterleaved && kVec > 1) {
#pragma unroll
    for (int i = 0; i < kVec; i += 2) {
      const uint64_t x = f2_make(v[i], v[i + 1]), y = f2_make(v[kVec + i], v[kVec + i + 1]);
      const uint64_t c = f2_make(cs[i], cs[i + 1]), s = f2_make(sn[i], sn[i + 1]);
      f2_split(f2_sub(f2_mul(x, c), f2_mul(y, s)), v[i], v[i + 1]);
      f2_split(f2_fma(x, s, f2_mul(y, c)), v[kVec + i], v[kVec + i + 1]);
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < kVec; ++i) {
    const int a = kInterleaved ? 2 * i : i, b = kInterleaved ? 2 * i + 1 : kVec + i;
    const float x = v[a], y = v[b];
    v[a] = x * cs[i] - y * sn[i];
    v[b] = y * cs[i] + x * sn[i];
  }
}

template <typename T, int kVec>
__device__ __forceinline__ void to_floats(const Vec<T, kVec>& v, float* f) {
#pragma unroll
  for (int i = 0; i < kVec; ++i) f[i] = to_f<T>(v.e[i]);
}
template <typename T, int kVec>
__device__ __forceinline__ Vec<T, kVec> from_floats(const float* f) {
  Vec<T, kVec> v;
#pragma unroll
  for (int i = 0; i < kVec; ++i) v.e[i] = from_f<T>(f[i]);
  return v;
}

// Tiles of tokens go to blockIdx.x, groups of heads of one tensor to blockIdx.y: the
// first groups0 are Q's. kPer chunks a thread; 2^lanes_log2 threads a head.
template <typename T, int kVec, int kPer, bool kInterleaved, bool kBackward>
__global__ void __launch_bounds__(kThreads, kBackward ? 2 : 3)
    norm_rope_kernel(const NormParams p, const int heads_each, const int groups0, const int lanes_log2) {
  using V = Vec<T, kVec>;
  constexpr bool kAsync = sizeof(V) == 16;
  constexpr int kIn = kBackward ? 2 : 1;
  constexpr int kStages = stages(kBackward);  // heads in flight per thread
  constexpr int kOwn = 2 * kVec * kPer;       // elements of a head that a thread has
  static_assert(!kAsync || kPer == 1, "one chunk a thread in the slots");
  extern __shared__ __align__(16) uint8_t dynamic_smem[];
  auto& slots = *reinterpret_cast<V(*)[kStages][2 * kIn][kThreads]>(dynamic_smem);  // (without kAsync there are none)

  const int lanes = 1 << lanes_log2, lane = threadIdx.x & (lanes - 1);
  const bool second = static_cast<int>(blockIdx.y) >= groups0;
  const NormTensor& t = p.t[second ? 1 : 0];
  const int h0 = (static_cast<int>(blockIdx.y) - (second ? groups0 : 0)) * heads_each;
  const int h1 = min(t.H, h0 + heads_each);
  const int tokens = p.B * p.N, tile_tokens = kThreads >> lanes_log2;
  const float inv_d = 1.f / static_cast<float>(p.d);

  Chunk ck[kPer];
  float w[kOwn];
#pragma unroll
  for (int c = 0; c < kPer; ++c) {
    ck[c] = chunk_at<kVec, kInterleaved>(lane + c * lanes, p.d, p.rot);
#pragma unroll
    for (int i = 0; i < 2 * kVec; ++i) {
      const int e = i < kVec ? ck[c].e0 + i : ck[c].e1 + i - kVec;
      const bool there = i < kVec ? ck[c].there : ck[c].two;
      float x = 1.f;
      if (t.w != nullptr && there)
        x = p.w_fp32 ? static_cast<const float*>(t.w)[e] : to_f<T>(static_cast<const T*>(t.w)[e]);
      w[c * 2 * kVec + i] = x;
    }
  }
  uint64_t w2[kOwn / 2], dw2[kBackward ? kOwn / 2 : 1];
#pragma unroll
  for (int i = 0; i < kOwn / 2; ++i) {
    w2[i] = f2_make(w[2 * i], w[2 * i + 1]);
    if constexpr (kBackward) dw2[i] = f2_make(0.f, 0.f);
  }

  // what the sines need of each frequency
  __shared__ __align__(16) uint64_t turns[kNormWidest / 2];
  __shared__ __align__(16) float factor[kNormWidest / 2];
  for (int i = threadIdx.x; i < p.rot / 2; i += kThreads) {
    const double f = p.freqs[i];
    bool high = false;
    turns[i] = turns_per_position(f, high);
    if (high && !(fabs(f) < 4.)) turns[i] = turns_of_high(f);
    factor[i] = fabs(f) < kFreqLimit ? p.mscale : __int_as_float(0x7fffffff);
  }
  __syncthreads();

  for (int tile = blockIdx.x; static_cast<long long>(tile) * tile_tokens < tokens; tile += gridDim.x) {
    const long long token_wide = static_cast<long long>(tile) * tile_tokens + (threadIdx.x >> lanes_log2);
    const bool live = token_wide < tokens;
    const int token = live ? static_cast<int>(token_wide) : 0;
    const int b = token / p.N, n = token - b * p.N;
    const T* x_at = static_cast<const T*>(t.x) + b * t.xs[0] + n * t.xs[2];
    const T* g_at = kBackward ? static_cast<const T*>(t.dy) + b * t.ds[0] + n * t.ds[2] : nullptr;
    T* y_at = static_cast<T*>(t.y) + b * t.ys[0] + n * t.ys[2];

    auto fetch = [&](int h, int slot) {
      if constexpr (kAsync) {
        if (h < h1 && live && ck[0].there) {
          const T* x = x_at + h * t.xs[1];
          copy16(&slots[slot][0][threadIdx.x], x + ck[0].e0);
          if (ck[0].two) copy16(&slots[slot][1][threadIdx.x], x + ck[0].e1);
          if constexpr (kBackward) {
            const T* g = g_at + h * t.ds[1];
            copy16(&slots[slot][2][threadIdx.x], g + ck[0].e0);
            if (ck[0].two) copy16(&slots[slot][3][threadIdx.x], g + ck[0].e1);
          }
        }
        copy_commit();
      }
    };
#pragma unroll
    for (int i = 0; i < kStages; ++i) fetch(h0 + i, i);

    float cs[kPer][kVec], sn[kPer][kVec];
    const int pos = p.positions ? p.positions[b * p.pos_stride + n] : n;
#pragma unroll
    for (int c = 0; c < kPer; ++c) {
#pragma unroll
      for (int i = 0; i < kVec; ++i) cs[c][i] = 1.f, sn[c][i] = 0.f;
      if (ck[c].rotated) {
        const int first = lane + c * lanes;
        // interleaved: the first access holds pairs e0 / 2 .., the second pairs e1 / 2 ..
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
          const int pair = !kInterleaved || kVec == 1 ? kVec * first + i
                                                      : (i < kVec / 2 ? ck[c].e0 : ck[c].e1 - kVec) / 2 + i;
          sines_at(pos, turns[pair], factor[pair], kBackward, cs[c][i], sn[c][i]);
        }
      }
    }

    int slot = 0;
    for (int h = h0; h < h1; ++h) {
      float x[kOwn], g[kBackward ? kOwn : 1];
#pragma unroll
      for (int i = 0; i < kOwn; ++i) x[i] = 0.f;
#pragma unroll
      for (int i = 0; i < (kBackward ? kOwn : 1); ++i) g[i] = 0.f;
      if constexpr (kAsync) {
        copy_wait<kStages - 1>();
        if (live && ck[0].there) {
          to_floats<T, kVec>(slots[slot][0][threadIdx.x], x);
          if (ck[0].two) to_floats<T, kVec>(slots[slot][1][threadIdx.x], x + kVec);
          if constexpr (kBackward) {
            to_floats<T, kVec>(slots[slot][2][threadIdx.x], g);
            if (ck[0].two) to_floats<T, kVec>(slots[slot][3][threadIdx.x], g + kVec);
          }
        }
      } else if (live) {
        const T* xh = x_at + h * t.xs[1];
        const T* gh = kBackward ? g_at + h * t.ds[1] : nullptr;
#pragma unroll
        for (int c = 0; c < kPer; ++c) {
          if (!ck[c].there) continue;
          to_floats<T, kVec>(*reinterpret_cast<const V*>(xh + ck[c].e0), x + 2 * kVec * c);
          if (ck[c].two) to_floats<T, kVec>(*reinterpret_cast<const V*>(xh + ck[c].e1), x + 2 * kVec * c + kVec);
          if constexpr (kBackward) {
            to_floats<T, kVec>(*reinterpret_cast<const V*>(gh + ck[c].e0), g + 2 * kVec * c);
            if (ck[c].two) to_floats<T, kVec>(*reinterpret_cast<const V*>(gh + ck[c].e1), g + 2 * kVec * c + kVec);
          }
        }
      }
      if constexpr (kBackward) {
#pragma unroll
        for (int c = 0; c < kPer; ++c)
          if (ck[c].rotated) turn<kVec, kInterleaved>(g + 2 * kVec * c, cs[c], sn[c]);
      }
      // from here on two elements at a time
      uint64_t x2[kOwn / 2], gw[kBackward ? kOwn / 2 : 1];
#pragma unroll
      for (int i = 0; i < kOwn / 2; ++i) {
        x2[i] = f2_make(x[2 * i], x[2 * i + 1]);
        if constexpr (kBackward) gw[i] = f2_mul(f2_make(g[2 * i], g[2 * i + 1]), w2[i]);
      }
      float s1 = 0.f, s2 = 0.f, f = 1.f;
      auto sums = [&]() {
        uint64_t a = f2_make(0.f, 0.f), z = a;
#pragma unroll
        for (int i = 0; i < kOwn / 2; ++i) {
          a = f2_fma(x2[i], x2[i], a);
          if constexpr (kBackward) z = f2_fma(gw[i], x2[i], z);
        }
        s1 = f2_sum(a);
        s2 = f2_sum(z);
        for (int o = 1; o < lanes; o <<= 1) {
          s1 += __shfl_xor_sync(0xffffffffu, s1, o);
          if constexpr (kBackward) s2 += __shfl_xor_sync(0xffffffffu, s2, o);
        }
      };
      sums();
      if (__builtin_expect(__any_sync(0xffffffffu, !(s1 + fabsf(s2) <= kSumMost)), 0)) {
        auto scale = [&](float by) {
          f *= by;
#pragma unroll
          for (int i = 0; i < kOwn / 2; ++i) x2[i] = f2_mul(x2[i], f2_make(by, by));
          sums();
        };
        scale(s1 <= kSumMost ? 1.f : 0x1p-70f);
        if constexpr (kBackward) {
          // a norm of 2^-10 at most: s2 is then below 2^-10 * 2^128 * sqrt(256)
          const int down = max(((__float_as_int(s1) >> 23) - 127) / 2 + 11, 0);
          scale(fabsf(s2) <= kSumMost ? 1.f : __int_as_float((127 - down) << 23));
        }
      }
      // r f of the definition is that of the values as they are
      const float r = rsqrtf(s1 * inv_d + p.eps * f * f);
      float y[kOwn];
      if constexpr (!kBackward) {
        const uint64_t r2 = f2_make(r, r);
#pragma unroll
        for (int i = 0; i < kOwn / 2; ++i) f2_split(f2_mul(f2_mul(x2[i], r2), w2[i]), y[2 * i], y[2 * i + 1]);
#pragma unroll
        for (int c = 0; c < kPer; ++c) {
          if (ck[c].rotated) turn<kVec, kInterleaved>(y + 2 * kVec * c, cs[c], sn[c]);
        }
      } else {
        const float rf = r * f, along = -rf * (r * s2 * inv_d);
        const uint64_t r2 = f2_make(r, r), rf2 = f2_make(rf, rf), along2 = f2_make(along, along);
#pragma unroll
        for (int i = 0; i < kOwn / 2; ++i) {
          const uint64_t u = f2_mul(x2[i], r2);
          dw2[i] = f2_fma(f2_make(g[2 * i], g[2 * i + 1]), u, dw2[i]);
          f2_split(f2_fma(u, along2, f2_mul(gw[i], rf2)), y[2 * i], y[2 * i + 1]);
        }
      }
      if (live) {
        T* yh = y_at + h * t.ys[1];
#pragma unroll
        for (int c = 0; c < kPer; ++c) {
          if (!ck[c].there) continue;
          *reinterpret_cast<V*>(yh + ck[c].e0) = from_floats<T, kVec>(y + 2 * kVec * c);
          if (ck[c].two) *reinterpret_cast<V*>(yh + ck[c].e1) = from_floats<T, kVec>(y + 2 * kVec * c + kVec);
        }
      }
      fetch(h + kStages, slot);
      slot = slot + 1 == kStages ? 0 : slot + 1;
    }
    if constexpr (kAsync) copy_wait<0>();
  }

  if constexpr (kBackward) {
    allow_next();
    if (t.dw == nullptr) return;
    // the CTA's sums: tokens of a warp by shuffles, then the warps in order
    constexpr int kWarps = kThreads / 32;
    __shared__ float sums_small[kAsync ? 1 : kWarps][kAsync ? 1 : kNormWidest];
    float* sums = kAsync ? reinterpret_cast<float*>(dynamic_smem) : &sums_small[0][0];
    static_assert(!kAsync || slot_bytes(true) >= kWarps * kNormWidest * sizeof(float), "sums fit the slots");
    __syncthreads();
    const int warp = threadIdx.x >> 5;
    float dw[kOwn];
#pragma unroll
    for (int i = 0; i < kOwn / 2; ++i) f2_split(dw2[i], dw[2 * i], dw[2 * i + 1]);
#pragma unroll
    for (int c = 0; c < kPer; ++c) {
#pragma unroll
      for (int i = 0; i < 2 * kVec; ++i) {
        float v = dw[c * 2 * kVec + i];
        for (int o = lanes; o < 32; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        const int e = i < kVec ? ck[c].e0 + i : ck[c].e1 + i - kVec;
        if ((i < kVec ? ck[c].there : ck[c].two) && (threadIdx.x & 31) < lanes) sums[warp * kNormWidest + e] = v;
      }
    }
    __syncthreads();
    const int row = blockIdx.y * gridDim.x + blockIdx.x;
    for (int e = threadIdx.x; e < p.d; e += kThreads) {
      float v = 0.f;
#pragma unroll
      for (int k = 0; k < kWarps; ++k) v += sums[k * kNormWidest + e];
      p.partial[static_cast<size_t>(row) * p.d + e] = v;
    }
  }
}

// dw of one tensor (blockIdx.y) and 32 elements: the CTAs' sums in order, 8 rows at a time.
template <typename T>
__global__ void __launch_bounds__(1024) norm_weights_kernel(const NormParams p, const int rows_x, const int groups0,
                                                           const int groups1) {
  __shared__ float sums[32][33];
  wait_for_previous();
  const NormTensor& t = p.t[blockIdx.y];
  if (t.dw == nullptr) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int e = blockIdx.x * 32 + lane;
  const int row0 = blockIdx.y ? groups0 * rows_x : 0, rows = rows_x * (blockIdx.y ? groups1 : groups0);
  float v = 0.f;
  if (e < p.d) {
    const float* at = p.partial + static_cast<size_t>(row0) * p.d + e;
#pragma unroll 8
    for (int r = warp; r < rows; r += 32) v += at[static_cast<size_t>(r) * p.d];
  }
  sums[warp][lane] = v;
  __syncthreads();
  if (warp == 0 && e < p.d) {
    float x = 0.f;
#pragma unroll
    for (int k = 0; k < 32; ++k) x += sums[k][lane];
    if (p.w_fp32)
      static_cast<float*>(t.dw)[e] = x;
    else
      static_cast<T*>(t.dw)[e] = from_f<T>(x);
  }
}

template <typename T, int kVec, int kPer>
cudaError_t allow_smem(int bytes) {
  static std::atomic<uint64_t> done[4];  // devices whose kernels have their shared memory
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev > 255) return cudaErrorInvalidDevice;
  if (done[dev >> 6].load(std::memory_order_relaxed) >> (dev & 63) & 1) return cudaSuccess;
  for (auto* k : {norm_rope_kernel<T, kVec, kPer, true, true>, norm_rope_kernel<T, kVec, kPer, false, true>}) {
    e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
  }
  done[dev >> 6].fetch_or(1ull << (dev & 63), std::memory_order_relaxed);
  return cudaSuccess;
}

// CTAs of a group of heads in the backward pass.
long long backward_blocks(long long tiles, long long want, long long groups) {
  return std::max(1LL, std::min({tiles, want / groups, kNormPartials / groups}));
}

template <typename T, int kVec, int kPer, bool kBackward>
cudaError_t launch_t(const NormParams& p, int num_sms, cudaStream_t s) {
  const int chunks = p.rot / 2 / kVec + (p.d - p.rot + 2 * kVec - 1) / (2 * kVec);
  const int threads = (chunks + kPer - 1) / kPer;
  int lanes_log2 = 0;
  while ((1 << lanes_log2) < threads) ++lanes_log2;
  if (lanes_log2 > 5) return cudaErrorInvalidValue;
  const int tile = kThreads >> lanes_log2;
  const long long tiles = (static_cast<long long>(p.B) * p.N + tile - 1) / tile;
  const int H = p.t[0].H + p.t[1].H;
  const long long want = (kBackward ? 2LL : 3LL) * num_sms;
  int each;  // heads per thread
  if constexpr (kBackward) {
    // All CTAs run at once, each over its share of the tiles: the heads that give the
    // shortest longest share, a tile's sines counted as one head more. (32 + 8 heads of 1024
    // tiles: 16 at a time leave the CTAs of the last 8 waiting, 185 us; 8 at a time 169, 4 at a time 190.)
    const int least = (H + kNormPartials / 2 - 1) / (kNormPartials / 2);
    long long best = 0;
    each = least;
    for (int e = std::max(1, least); e <= std::max(kHeadsMost, least); ++e) {
      const long long g = (p.t[0].H + e - 1) / e + (p.t[1].H + e - 1) / e;
      const long long share = (tiles - 1) / backward_blocks(tiles, want, g) + 1;
      if (best == 0 || share * (e + 1) < best) best = share * (e + 1), each = e;
    }
  } else {
    // as many as leave all SMs full, at most kHeadsMost (32768 tokens, 32 + 32 heads of 128: 163 us;
    // 8 172, 32 168)
    each = static_cast<int>(std::min<long long>(kHeadsMost, std::max(1LL, H * tiles / want)));
  }
  const int groups0 = (p.t[0].H + each - 1) / each, groups1 = (p.t[1].H + each - 1) / each;
  const int groups = groups0 + groups1;
  if (groups > 65535) return cudaErrorInvalidValue;
  long long blocks = tiles;
  if (kBackward) blocks = backward_blocks(tiles, want, groups);
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
  const dim3 grid(static_cast<unsigned>(blocks), static_cast<unsigned>(groups));
  constexpr int kSmem = kVec > 1 ? slot_bytes(kBackward) : 0;
  auto* kernel = p.interleaved ? norm_rope_kernel<T, kVec, kPer, true, kBackward>
                               : norm_rope_kernel<T, kVec, kPer, false, kBackward>;
  if constexpr (kSmem + 2048 > 48 * 1024) {
    const cudaError_t e = allow_smem<T, kVec, kPer>(kSmem);
    if (e != cudaSuccess) return e;
  }
  kernel<<<grid, kThreads, kSmem, s>>>(p, each, groups0, lanes_log2);
  if (kBackward && (p.t[0].dw != nullptr || p.t[1].dw != nullptr)) {
    const cudaError_t st = cudaGetLastError();
    if (st != cudaSuccess) return st;
    return launch_overlapped(norm_weights_kernel<T>, dim3((p.d + 31) / 32, p.t[1].H ? 2 : 1), 1024, 0, s, p,
                             static_cast<int>(blocks), groups0, groups1);
  }
  return cudaGetLastError();
}

// 16-byte accesses need every row to start on a 16-byte boundary and the rotated
// pairs and the rest to be whole accesses; else one element at a time.
template <typename T, bool kBackward>
cudaError_t launch_d(const NormParams& p, int num_sms, cudaStream_t s) {
  constexpr int kVec = 16 / sizeof(T);
  bool vec = p.d % kVec == 0 && (p.rot / 2) % kVec == 0;
  for (const NormTensor& t : p.t) {
    if (t.H == 0) continue;
    vec = vec && ((reinterpret_cast<uintptr_t>(t.x) | reinterpret_cast<uintptr_t>(t.y) |
                   reinterpret_cast<uintptr_t>(t.dy)) & 15u) == 0;
    for (int i = 0; i < 3; ++i) vec = vec && t.xs[i] % kVec == 0 && t.ys[i] % kVec == 0 && t.ds[i] % kVec == 0;
  }
  return vec ? launch_t<T, kVec, 1, kBackward>(p, num_sms, s) : launch_t<T, 1, 4, kBackward>(p, num_sms, s);
}

template <bool kBackward>
cudaError_t launch(const NormParams& p, int dtype, int num_sms, cudaStream_t s) {
  if (dtype == FM_F32) return launch_d<float, kBackward>(p, num_sms, s);
  if (dtype == FM_F16) return launch_d<__half, kBackward>(p, num_sms, s);
  return launch_d<__nv_bfloat16, kBackward>(p, num_sms, s);
}

}  // namespace

cudaError_t launch_norm_rope(const NormParams& p, int dtype, bool backward, int num_sms, cudaStream_t s) {
  return backward ? launch<true>(p, dtype, num_sms, s) : launch<false>(p, dtype, num_sms, s);
}

}  // namespace fm
