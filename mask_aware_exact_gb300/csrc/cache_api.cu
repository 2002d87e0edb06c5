// Host side of the rotary and paged-cache entry points of include/flashmask.h:
// argument checks, workspace sizes and launches. Nothing here allocates.
#include <atomic>
#include <cmath>

#include "cache.h"
#include "flashmask.h"

static_assert(FM_PAGE == fm::kPage, "page size");

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// SMs of the current device, looked up once per device.
int sm_count() {
  constexpr int kMaxDev = 256;
  static std::atomic<int> cached[kMaxDev];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDev) return 0;
  int n = cached[dev].load(std::memory_order_relaxed);
  if (n == 0) {
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
    cached[dev].store(n, std::memory_order_relaxed);
  }
  return n;
}

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// Whether rows written with these strides lie apart (a dimension of one size may have
// any stride, others not zero).
bool apart(const int64_t* s, int B, int H, int N) {
  return (B == 1 || s[0] != 0) && (H == 1 || s[1] != 0) && (N == 1 || s[2] != 0);
}

// Rows of 8-element (16-byte) pieces need strides that keep them aligned.
bool strides_ok(const int64_t* s) {
  for (int i = 0; i < 3; ++i)
    if (s[i] % 8 != 0) return false;
  return true;
}

// The mask's vectors are read 16 bytes at a time.
bool vectors_ok(const fm_mask* m) {
  return (m->lts == nullptr) == (m->lte == nullptr) && (m->uts == nullptr) == (m->ute == nullptr) &&
         aligned16(m->lts) && aligned16(m->lte) && aligned16(m->uts) && aligned16(m->ute);
}

bool cache_shape_ok(int B, int H, int Hk, int N, int d, int max_pages) {
  if (B <= 0 || H <= 0 || Hk <= 0 || N <= 0 || max_pages <= 0) return false;
  if (d != 64 && d != 128) return false;
  if (H % Hk != 0 || Hk > 65535 || B > 65535) return false;
  if (max_pages > FM_MAX_SEQLEN / FM_PAGE || N > FM_MAX_SEQLEN) return false;
  // rows fit 32 bits, with those that fill a tile up
  if (static_cast<long long>(B) * H > (0x7fffffffLL - 255) / N) return false;
  return fm::cache_line_ok(B, H, Hk, N, max_pages);
}

fm_status cache_ok(const fm_cache* c) {
  if (!c || !c->k8 || !c->v8 || !c->kscale || !c->vscale) return FM_ERR_INVALID_ARG;
  if (!aligned16(c->k8) || !aligned16(c->v8) || !aligned4(c->kscale) || !aligned4(c->vscale))
    return FM_ERR_INVALID_ARG;
  if (c->pages <= 0) return FM_ERR_INVALID_ARG;
  return FM_OK;
}

fm::CacheDev cache_dev(const fm_cache* c) {
  fm::CacheDev r;
  r.k8 = static_cast<uint8_t*>(c->k8);
  r.v8 = static_cast<uint8_t*>(c->v8);
  r.kscale = c->kscale;
  r.vscale = c->vscale;
  r.pages = c->pages;
  r.Hk = c->Hk;
  return r;
}

fm_status check_ws(void* ws, size_t ws_bytes, size_t need) {
  if (!ws || (reinterpret_cast<uintptr_t>(ws) & 255u) != 0 || ws_bytes < need)
    return FM_ERR_WORKSPACE;
  return FM_OK;
}

}  // namespace

extern "C" {

fm_status flashmask_rope(const fm_heads* t, int n_tensors, const int32_t* positions,
                         int64_t pos_stride, const double* freqs, int B, int N, int d, int rot_dim,
                         int interleaved, int dtype, float mscale, int inverse, void* stream) {
  if (!t || n_tensors < 1 || n_tensors > 2) return FM_ERR_INVALID_ARG;
  if (dtype != FM_BF16 && dtype != FM_F16 && dtype != FM_F32) return FM_ERR_INVALID_ARG;
  if (!std::isfinite(mscale)) return FM_ERR_INVALID_ARG;
  if (rot_dim > 0 && !freqs) return FM_ERR_INVALID_ARG;
  if (positions && (reinterpret_cast<uintptr_t>(positions) & 3u) != 0) return FM_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(freqs) & 7u) != 0) return FM_ERR_INVALID_ARG;
  if (B <= 0 || N <= 0 || d <= 0 || rot_dim < 0 || rot_dim > d || rot_dim % 2 != 0)
    return FM_ERR_UNSUPPORTED;
  if (static_cast<long long>(B) * N > 0x7fffffffLL) return FM_ERR_UNSUPPORTED;
  fm::RopeParams p = {};
  long long heads = 0;
  const uintptr_t esize = dtype == FM_F32 ? 4 : 2;
  for (int i = 0; i < n_tensors; ++i) {
    if (!t[i].x || !t[i].y) return FM_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(t[i].x) % esize || reinterpret_cast<uintptr_t>(t[i].y) % esize)
      return FM_ERR_INVALID_ARG;
    if (t[i].H <= 0) return FM_ERR_UNSUPPORTED;
    heads += t[i].H;
    p.t[i].x = t[i].x;
    p.t[i].y = t[i].y;
    p.t[i].H = t[i].H;
    for (int k = 0; k < 3; ++k) {
      p.t[i].xs[k] = t[i].xs[k];
      p.t[i].ys[k] = t[i].ys[k];
    }
  }
  if (heads > 65535 || static_cast<long long>(B) * N * d > (1LL << 38)) return FM_ERR_UNSUPPORTED;
  for (int i = 0; i < n_tensors; ++i)
    if (!apart(t[i].ys, B, t[i].H, N)) return FM_ERR_INVALID_ARG;
  p.positions = positions;
  p.pos_stride = pos_stride;
  p.freqs = freqs;
  p.B = B;
  p.N = N;
  p.d = d;
  p.rot = rot_dim;
  p.interleaved = interleaved ? 1 : 0;
  p.inverse = inverse ? 1 : 0;
  p.mscale = mscale;
  const int sms = sm_count();
  if (sms <= 0) return FM_ERR_CUDA;
  return fm::launch_rope(p, dtype, sms, static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? FM_OK
             : FM_ERR_CUDA;
}

size_t flashmask_cache_workspace_bytes(int B, int H, int Hk, int N, int d, int max_pages) {
  if (!cache_shape_ok(B, H, Hk, N, d, max_pages)) return 0;
  return fm::cache_ws_layout(B, H, Hk, N, d, max_pages).total;
}

fm_status flashmask_cache_append(const fm_cache* cache, const int32_t* page_table, int max_pages,
                                 const void* k, const int64_t ks[3], const void* v,
                                 const int64_t vs[3], const int32_t* start, const int32_t* count,
                                 int B, int N, void* ws, size_t ws_bytes, void* stream) {
  const fm_status cs = cache_ok(cache);
  if (cs != FM_OK) return cs;
  if (!page_table || !k || !v || !ks || !vs || !start) return FM_ERR_INVALID_ARG;
  if (!aligned16(k) || !aligned16(v) || !strides_ok(ks) || !strides_ok(vs)) return FM_ERR_INVALID_ARG;
  if (!aligned4(page_table) || !aligned4(start) || !aligned4(count)) return FM_ERR_INVALID_ARG;
  if (!cache_shape_ok(B, cache->Hk, cache->Hk, N, cache->d, max_pages)) return FM_ERR_UNSUPPORTED;
  const fm_status st = check_ws(ws, ws_bytes, 16);
  if (st != FM_OK) return st;
  fm::AppendParams p;
  p.c = cache_dev(cache);
  p.table = page_table;
  p.max_pages = max_pages;
  p.k = static_cast<const uint16_t*>(k);
  p.v = static_cast<const uint16_t*>(v);
  for (int i = 0; i < 3; ++i) {
    p.ks[i] = ks[i];
    p.vs[i] = vs[i];
  }
  p.start = start;
  p.count = count;
  p.B = B;
  p.N = N;
  p.status = static_cast<int32_t*>(ws);
  return fm::launch_append(cache->d, p, static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? FM_OK
             : FM_ERR_CUDA;
}

fm_status flashmask_fwd_cache(const void* q, const int64_t qs[3], const fm_cache* cache,
                              const int32_t* page_table, int max_pages, const int32_t* lens,
                              const int32_t* q_lens, const fm_mask* mask, int B, int H, int N,
                              float scale, void* o, const int64_t os[3], float* lse, void* ws,
                              size_t ws_bytes, void* stream) {
  const fm_status cs = cache_ok(cache);
  if (cs != FM_OK) return cs;
  if (!q || !qs || !page_table || !lens || !o || !os || !lse) return FM_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(o) || !strides_ok(qs) || !strides_ok(os)) return FM_ERR_INVALID_ARG;
  if (!aligned4(page_table) || !aligned4(lens) || !aligned4(q_lens) || !aligned4(lse))
    return FM_ERR_INVALID_ARG;
  const float scale_log2 = scale * 1.4426950408889634f;
  if (!std::isfinite(scale_log2) || !(scale > 0.f)) return FM_ERR_INVALID_ARG;
  if (mask && !vectors_ok(mask)) return FM_ERR_INVALID_ARG;
  if (!cache_shape_ok(B, H, cache->Hk, N, cache->d, max_pages)) return FM_ERR_UNSUPPORTED;
  if (mask && (mask->Hm <= 0 || H % mask->Hm != 0)) return FM_ERR_UNSUPPORTED;
  const fm::CacheWs L = fm::cache_ws_layout(B, H, cache->Hk, N, cache->d, max_pages);
  const fm_status st = check_ws(ws, ws_bytes, L.total);
  if (st != FM_OK) return st;
  if (!apart(os, B, H, N)) return FM_ERR_INVALID_ARG;
  fm::CacheFwdParams p;
  p.q = static_cast<const uint16_t*>(q);
  p.c = cache_dev(cache);
  p.table = page_table;
  p.max_pages = max_pages;
  p.lens = lens;
  p.q_lens = q_lens;
  p.mask = {};
  p.mask.Hm = 1;
  p.mask.causal = 1;
  if (mask) {
    p.mask.lts = mask->lts;
    p.mask.lte = mask->lte;
    p.mask.uts = mask->uts;
    p.mask.ute = mask->ute;
    p.mask.Hm = mask->Hm;
    p.mask.causal = mask->causal ? 1 : 0;
  }
  p.B = B;
  p.H = H;
  p.N = N;
  p.scale_log2 = scale_log2;
  p.o = static_cast<uint16_t*>(o);
  for (int i = 0; i < 3; ++i) {
    p.qs[i] = qs[i];
    p.os[i] = os[i];
  }
  p.lse = lse;
  char* w = static_cast<char*>(ws);
  p.status = reinterpret_cast<int32_t*>(w);
  p.arrived = reinterpret_cast<int32_t*>(w + L.arrived);
  p.groups = reinterpret_cast<int32_t*>(w + L.groups);
  p.partial = reinterpret_cast<float*>(w + L.partial);
  p.list = reinterpret_cast<uint16_t*>(w + L.list);
  p.listed = reinterpret_cast<int32_t*>(w + L.listed);
  const int sms = sm_count();
  if (sms <= 0) return FM_ERR_CUDA;
  return fm::launch_cache_fwd(cache->d, p, sms, static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? FM_OK
             : FM_ERR_CUDA;
}

}  // extern "C"
