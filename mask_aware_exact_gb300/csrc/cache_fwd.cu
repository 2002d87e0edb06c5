// Attention over the 8-bit paged cache. Simple form: one warp per query row and
// head, keys one after another, running maximum and sum.
#include "cache.h"
#include "ptx_fp8.cuh"

namespace fm {
namespace {

__device__ __forceinline__ float e4m3_value(uint8_t c) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(c)));
  float f;
  asm("{.reg .f16 a, b; mov.b32 {a, b}, %1; cvt.f32.f16 %0, a;}" : "=f"(f) : "r"(h));
  return f;
}

template <int D>
__global__ void __launch_bounds__(128) cache_fwd_simple(const CacheFwdParams p) {
  const int lane = threadIdx.x & 31;
  const long long row = static_cast<long long>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  if (row >= static_cast<long long>(p.B) * p.H * p.N) return;
  const int t = row % p.N, h = (row / p.N) % p.H, b = row / (static_cast<long long>(p.N) * p.H);
  const int qn = p.q_lens ? min(max(p.q_lens[b], 0), p.N) : p.N;
  if (t >= qn) return;
  int len = p.lens[b];
  const int most = p.max_pages * kPage;
  if (len < 0 || len > most) {
    if (lane == 0) record_failure(p.status, kStatusPage, kSiteCacheLen);
    len = min(max(len, 0), most);
  }
  const int pos = len - qn + t, hk = h / (p.H / p.c.Hk);
  const size_t mrow = (static_cast<size_t>(b) * p.mask.Hm + h / (p.H / p.mask.Hm)) * most;
  float q[D / 32], acc[D / 32];
  for (int i = 0; i < D / 32; ++i) {
    q[i] = __uint_as_float(static_cast<uint32_t>(p.q[b * p.qs[0] + h * p.qs[1] + t * p.qs[2] + lane + 32 * i]) << 16);
    acc[i] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  const int end = p.mask.causal ? min(len, pos + 1) : len;
  for (int j = 0; j < end; ++j) {
    if (p.mask.lts && p.mask.lts[mrow + j] <= pos && pos < p.mask.lte[mrow + j]) continue;
    if (p.mask.uts && p.mask.uts[mrow + j] <= pos && pos < p.mask.ute[mrow + j]) continue;
    const int page = p.table[static_cast<size_t>(b) * p.max_pages + j / kPage];
    if (page < 0 || page >= p.c.pages) {
      if (lane == 0) record_failure(p.status, kStatusPage, kSiteCachePage);
      continue;
    }
    const size_t ph = static_cast<size_t>(page) * p.c.Hk + hk;
    float s = 0.f;
    for (int i = 0; i < D / 32; ++i)
      s += q[i] * e4m3_value(p.c.k8[ph * (kPage * D) + (j % kPage) * D + lane + 32 * i]);
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    s *= p.scale_log2 * p.c.kscale[ph];
    const float mn = fmaxf(m, s);
    const float f = m == -INFINITY ? 0.f : exp2f(m - mn);
    const float w = exp2f(s - (mn == -INFINITY ? 0.f : mn));
    m = mn;
    l = l * f + w;
    const float vs = p.c.vscale[ph];
    for (int i = 0; i < D / 32; ++i)
      acc[i] = acc[i] * f + w * vs * e4m3_value(p.c.v8[ph * (kPage * D) + (lane + 32 * i) * kPage + j % kPage]);
  }
  const bool none = l == 0.f;
  for (int i = 0; i < D / 32; ++i)
    p.o[b * p.os[0] + h * p.os[1] + t * p.os[2] + lane + 32 * i] =
        static_cast<uint16_t>(pack_bf16x2(none ? 0.f : acc[i] / l, 0.f));
  if (lane == 0)
    p.lse[(static_cast<size_t>(b) * p.H + h) * p.N + t] = none ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
}

}  // namespace

cudaError_t launch_cache_fwd(int d, const CacheFwdParams& p, cudaStream_t s) {
  const long long rows = static_cast<long long>(p.B) * p.H * p.N;
  const unsigned grid = static_cast<unsigned>((rows + 3) / 4);
  if (d == 64)
    cache_fwd_simple<64><<<grid, 128, 0, s>>>(p);
  else
    cache_fwd_simple<128><<<grid, 128, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace fm
