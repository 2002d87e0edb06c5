// Parts shared by the rotary kernels: the angle of a position in 64-bit turns,
// conversions, 16-byte accesses and asynchronous copies.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cstdint>

namespace fm {

// The first 192 bits of 2 / pi.
constexpr uint64_t kTwoOverPi0 = 0xa2f9836e4e441529ull, kTwoOverPi1 = 0xfc2757d1f534ddc0ull,
                   kTwoOverPi2 = 0xdb6295993c439041ull;

// f / (2 pi) modulo one turn as a 64-bit fraction, less than two units of it off, from the
// bits of the fp64 f: mantissa times 2 / pi, shifted by the exponent. Up to |f| = 4 the
// first word of 2 / pi has all the bits that stay. `high` is set for a frequency above:
// that one is for turns_of_high.
__device__ __forceinline__ uint64_t turns_per_position(double f, bool& high) {
  const uint64_t u = static_cast<uint64_t>(__double_as_longlong(f));
  const int ex = static_cast<int>((u >> 52) & 0x7ffu), sh = ex - 1024;
  high |= sh > 0;
  // f = m * 2^(ex - 1086); f / (2 pi) * 2^64 = m * (2 / pi) * 2^sh (zero and denormals
  // vanish: sh is -1024)
  const uint64_t m = ((u & 0xfffffffffffffull) | (1ull << 52)) << 11;
  const uint64_t r = sh > -64 ? __umul64hi(m, kTwoOverPi0) >> (-sh & 63) : 0;
  return (u >> 63) ? 0ull - r : r;
}
// The same for |f| >= 4, where the shift moves further bits of 2 / pi up and the first out
// at the top. There are enough of them below kFreqLimit.
constexpr double kFreqLimit = 0x1p129;
static __device__ __noinline__ uint64_t turns_of_high(double f) {
  const uint64_t u = static_cast<uint64_t>(__double_as_longlong(f));
  const int sh = static_cast<int>((u >> 52) & 0x7ffu) - 1024;
  const uint64_t m = ((u & 0xfffffffffffffull) | (1ull << 52)) << 11;
  // m * (2 / pi) * 2^(sh / 64 * 64) as whole and fraction; the whole modulo 2^64
  const bool far = sh >= 64;
  const uint64_t before = far ? kTwoOverPi0 : 0, at = far ? kTwoOverPi1 : kTwoOverPi0;
  const uint64_t low = m * at, fraction = low + __umul64hi(m, far ? kTwoOverPi2 : kTwoOverPi1);
  const uint64_t whole = m * before + __umul64hi(m, at) + (fraction < low);
  const uint64_t r = sh & 63 ? whole << (sh & 63) | fraction >> (64 - (sh & 63)) : whole;
  return (u >> 63) ? 0ull - r : r;
}

// c times cosine and sine (negated for `inverse`) at position pos of `turns` a position.
__device__ __forceinline__ void sines_at(int pos, uint64_t turns, float c, bool inverse, float& cs, float& sn) {
  const uint64_t a = static_cast<uint64_t>(static_cast<int64_t>(pos)) * turns;
  // the top 32 bits in units of half turns, in [-1, 1)
  const float half_turns = static_cast<float>(static_cast<int32_t>(a >> 32)) * 4.656612873077393e-10f;  // 2^-31
  sincospif(half_turns, &sn, &cs);
  cs *= c;
  sn *= inverse ? -c : c;
}

// mscale times cosine and sine (negated for `inverse`) of kVec pairs at position pos;
// freq(i) is the frequency of pair i.
template <int kVec, typename F>
__device__ __forceinline__ void sines_of(int pos, float mscale, bool inverse, F freq, float (&cs)[kVec],
                                         float (&sn)[kVec]) {
  uint64_t turns[kVec];
  bool high = false;
#pragma unroll
  for (int i = 0; i < kVec; ++i) turns[i] = turns_per_position(freq(i), high);
  uint32_t none = 0;  // bit i: no frequency
  if (__builtin_expect(high, 0)) {
    // (one branch behind the loop: one for each pair cost 1 % of the gradient's case)
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      const double f = freq(i);
      if (!(fabs(f) < 4.)) turns[i] = turns_of_high(f);
      if (!(fabs(f) < kFreqLimit)) none |= 1u << i;
    }
  }
#pragma unroll
  for (int i = 0; i < kVec; ++i) {
    sines_at(pos, turns[i], none >> i & 1u ? __int_as_float(0x7fffffff) : mscale, inverse, cs[i], sn[i]);
  }
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

// This thread's copy of 16 bytes into shared memory, in the current group.
__device__ __forceinline__ void copy16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(static_cast<uint32_t>(__cvta_generic_to_shared(dst))),
               "l"(src)
               : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int n>
__device__ __forceinline__ void copy_wait() {  // all but the last n groups have landed
  asm volatile("cp.async.wait_group %0;" ::"n"(n) : "memory");
}

}  // namespace fm
