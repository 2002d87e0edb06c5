// Launch interface of the rotary and paged-cache kernels.
#pragma once
#include <cuda_runtime.h>
#include <cstddef>
#include <cstdint>

#include "internal.h"

namespace fm {

constexpr int kPage = 64;

struct RopeTensor {
  const void* x;
  void* y;
  int H;
  int64_t xs[3], ys[3];  // batch, head, token
};
struct RopeParams {
  RopeTensor t[2];  // t[1].H = 0 when there is one tensor
  const int32_t* positions;
  int64_t pos_stride;
  const double* freqs;
  int B, N, d, rot, interleaved, inverse;
  float mscale;
};
cudaError_t launch_rope(const RopeParams& p, int dtype, int num_sms, cudaStream_t s);

struct CacheDev {
  uint8_t* k8;
  uint8_t* v8;
  float* kscale;
  float* vscale;
  int pages, Hk;
};
struct AppendParams {
  CacheDev c;
  const int32_t* table;
  int max_pages;
  const uint16_t* k;
  const uint16_t* v;
  int64_t ks[3], vs[3];
  const int32_t* start;
  const int32_t* count;
  int B, N;
  int32_t* status;
};
cudaError_t launch_append(int d, const AppendParams& p, cudaStream_t s);

struct CacheFwdParams {
  const uint16_t* q;
  int64_t qs[3];
  CacheDev c;
  const int32_t* table;
  int max_pages;
  const int32_t* lens;
  const int32_t* q_lens;
  MaskDev mask;  // lts, lte null: no lower interval; uts, ute null: no upper
  int B, H, N;
  float scale_log2;  // scale * log2(e)
  uint16_t* o;
  int64_t os[3];
  float* lse;
  int32_t* status;
  // workspace (see CacheWs)
  int32_t* arrived;     // [CTAs]: partial results that have arrived of the cut segment that begins
                        // in a CTA's run (0 between calls)
  int32_t* groups;      // [CTAs][2]: the same for groups of parts, see Part (also 0 between calls)
  float* partial;       // [CTAs][2] partial results
  uint16_t* list;       // [row tiles][max_pages]: pages that some row sees, in order; bit 15: intervals
                        // hide some key of the page from some row
  int32_t* listed;      // [row tiles]: their number
};
// n / d for 0 <= n < 2^31 by a multiplication: mul = ceil(2^(31 + s) / d) with 2^s >= d,
// n / d = (n * mul) >> (31 + s) (the excess, below n * 2^-31-s, is less than 1 / d).
struct Divisor {
  uint32_t d, mul, shift;
  __host__ void set(int divisor) {
    d = static_cast<uint32_t>(divisor);
    uint32_t s = 0;
    while ((1ull << s) < d) ++s;
    mul = static_cast<uint32_t>(((1ull << (31 + s)) + d - 1) / d);
    shift = s;
  }
  __device__ __forceinline__ int div(int n) const {
    return static_cast<int>((static_cast<uint64_t>(static_cast<uint32_t>(n)) * mul) >> 31 >> shift);
  }
};
// Rows of the attention's work. The G = H / Hk query heads of a cache head and a
// sequence's query tokens form one list of rows, r = t * G + g, cut into RT tiles.
struct Geometry {
  int G, rows, RT;  // query heads per cache head, rows of a tile, row tiles
  int classes;      // mask classes: cache heads whose rows see the same masks share one
  int words;        // 32-bit words of page bits
  Divisor by_G, by_RT, by_Hk, by_class, by_mask;  // G, RT, Hk, Hk / classes, H / Hm
};

// Byte offsets of the workspace regions.
struct CacheWs {
  size_t arrived, groups, partial, list, listed, total;
};
constexpr int kCacheMaxCtas = 256;  // partial results are kept for at most this many CTAs
// Whether the pages of all row tiles can be counted in 32 bits.
bool cache_line_ok(int B, int H, int Hk, int N, int max_pages);
CacheWs cache_ws_layout(int B, int H, int Hk, int N, int d, int max_pages);
cudaError_t launch_cache_classify(const CacheFwdParams& p, const Geometry& geo, cudaStream_t s);
// Many query rows per cache head: tiles of 128 rows on the 5th-generation tensor cores.
constexpr int kManyRows = 128;
size_t cache_fwd_rows_part_floats(int d);  // of one partial result
cudaError_t launch_cache_fwd_rows(int d, const CacheFwdParams& p, const Geometry& geo, int num_sms,
                                  cudaStream_t s);
cudaError_t launch_cache_fwd(int d, const CacheFwdParams& p, int num_sms, cudaStream_t s);

}  // namespace fm
