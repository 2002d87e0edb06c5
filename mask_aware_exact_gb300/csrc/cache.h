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
};
cudaError_t launch_cache_fwd(int d, const CacheFwdParams& p, cudaStream_t s);

}  // namespace fm
