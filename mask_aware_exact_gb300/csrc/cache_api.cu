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

// null: causal, no intervals
fm::MaskDev mask_dev(const fm_mask* m) {
  fm::MaskDev r = {};
  r.Hm = 1;
  r.causal = 1;
  if (m) {
    r.lts = m->lts;
    r.lte = m->lte;
    r.uts = m->uts;
    r.ute = m->ute;
    r.Hm = m->Hm;
    r.causal = m->causal ? 1 : 0;
  }
  return r;
}

fm_status check_ws(void* ws, size_t ws_bytes, size_t need) {
  if (!ws || (reinterpret_cast<uintptr_t>(ws) & 255u) != 0 || ws_bytes < need)
    return FM_ERR_WORKSPACE;
  return FM_OK;
}

// Arguments that the norm with rotary positions and its gradients share.
fm_status norm_params(const fm_norm_heads* t, int n_tensors, const int32_t* positions, int64_t pos_stride,
                      const double* freqs, int B, int N, int d, int rot_dim, int interleaved, int dtype,
                      int weight_dtype, float mscale, float eps, bool backward, fm::NormParams& p) {
  if (!t || n_tensors < 1 || n_tensors > 2) return FM_ERR_INVALID_ARG;
  if (dtype != FM_BF16 && dtype != FM_F16 && dtype != FM_F32) return FM_ERR_INVALID_ARG;
  if (weight_dtype != dtype && weight_dtype != FM_F32) return FM_ERR_INVALID_ARG;
  if (!std::isfinite(mscale) || !std::isfinite(eps) || !(eps >= 1e-30f)) return FM_ERR_INVALID_ARG;
  if (rot_dim > 0 && !freqs) return FM_ERR_INVALID_ARG;
  if (!aligned4(positions) || (reinterpret_cast<uintptr_t>(freqs) & 7u) != 0) return FM_ERR_INVALID_ARG;
  if (B <= 0 || N <= 0 || d <= 0 || d > fm::kNormWidest || rot_dim < 0 || rot_dim > d || rot_dim % 2 != 0)
    return FM_ERR_UNSUPPORTED;
  if (static_cast<long long>(B) * N > 0x7fffffffLL) return FM_ERR_UNSUPPORTED;
  p = {};
  long long heads = 0;
  const uintptr_t esize = dtype == FM_F32 ? 4 : 2, wsize = weight_dtype == FM_F32 ? 4 : 2;
  auto at = [](const void* x) { return reinterpret_cast<uintptr_t>(x); };
  for (int i = 0; i < n_tensors; ++i) {
    const fm_norm_heads& h = t[i];
    if (!h.x || !h.y || (backward && !h.dy)) return FM_ERR_INVALID_ARG;
    if (at(h.x) % esize || at(h.y) % esize || at(h.w) % wsize) return FM_ERR_INVALID_ARG;
    if (backward && (at(h.dy) % esize || at(h.dw) % wsize)) return FM_ERR_INVALID_ARG;
    if (h.H <= 0) return FM_ERR_UNSUPPORTED;
    heads += h.H;
    fm::NormTensor& o = p.t[i];
    o.x = h.x;
    o.y = h.y;
    o.w = h.w;
    o.H = h.H;
    for (int k = 0; k < 3; ++k) {
      o.xs[k] = h.xs[k];
      o.ys[k] = h.ys[k];
    }
    if (backward) {
      o.dy = h.dy;
      o.dw = h.dw;
      for (int k = 0; k < 3; ++k) o.ds[k] = h.ds[k];
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
  p.w_fp32 = weight_dtype == FM_F32 ? 1 : 0;
  p.mscale = mscale;
  p.eps = eps;
  return FM_OK;
}

fm_status launch_norm(const fm::NormParams& p, int dtype, bool backward, void* stream) {
  const int sms = sm_count();
  if (sms <= 0) return FM_ERR_CUDA;
  return fm::launch_norm_rope(p, dtype, backward, sms, static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? FM_OK
             : FM_ERR_CUDA;
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

fm_status flashmask_norm_rope(const fm_norm_heads* t, int n_tensors, const int32_t* positions,
                              int64_t pos_stride, const double* freqs, int B, int N, int d, int rot_dim,
                              int interleaved, int dtype, int weight_dtype, float mscale, float eps,
                              void* stream) {
  fm::NormParams p;
  const fm_status st = norm_params(t, n_tensors, positions, pos_stride, freqs, B, N, d, rot_dim, interleaved,
                                   dtype, weight_dtype, mscale, eps, false, p);
  return st != FM_OK ? st : launch_norm(p, dtype, false, stream);
}

size_t flashmask_norm_workspace_bytes(int d) {
  return d <= 0 || d > fm::kNormWidest ? 0 : static_cast<size_t>(fm::kNormPartials) * d * sizeof(float);
}

fm_status flashmask_norm_rope_bwd(const fm_norm_heads* t, int n_tensors, const int32_t* positions,
                                  int64_t pos_stride, const double* freqs, int B, int N, int d, int rot_dim,
                                  int interleaved, int dtype, int weight_dtype, float mscale, float eps, void* ws,
                                  size_t ws_bytes, void* stream) {
  fm::NormParams p;
  fm_status st = norm_params(t, n_tensors, positions, pos_stride, freqs, B, N, d, rot_dim, interleaved, dtype,
                             weight_dtype, mscale, eps, true, p);
  if (st != FM_OK) return st;
  if (p.t[0].dw || p.t[1].dw) {
    st = check_ws(ws, ws_bytes, flashmask_norm_workspace_bytes(d));
    if (st != FM_OK) return st;
  }
  p.partial = static_cast<float*>(ws);
  return launch_norm(p, dtype, true, stream);
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

size_t flashmask_cache_weights_workspace_bytes(int B, int H, int Hk, int N, int d, int max_pages) {
  if (!cache_shape_ok(B, H, Hk, N, d, max_pages)) return 0;
  return fm::weights_ws_layout(B, H, Hk, N, d, max_pages).total;
}

fm_status flashmask_cache_weights(const void* q, const int64_t qs[3], const fm_cache* cache,
                                  const int32_t* page_table, int max_pages, const int32_t* lens,
                                  const int32_t* q_lens, const fm_mask* mask, int B, int H, int N, float scale,
                                  const float* lse, float* weights, const int32_t* start, void* ws,
                                  size_t ws_bytes, void* stream) {
  const fm_status cs = cache_ok(cache);
  if (cs != FM_OK) return cs;
  if (!q || !qs || !page_table || !lens || !lse || !weights) return FM_ERR_INVALID_ARG;
  if (!aligned16(q) || !strides_ok(qs)) return FM_ERR_INVALID_ARG;
  if (!aligned4(page_table) || !aligned4(lens) || !aligned4(q_lens) || !aligned4(lse) || !aligned4(weights) ||
      !aligned4(start))
    return FM_ERR_INVALID_ARG;
  const float scale_log2 = scale * 1.4426950408889634f;
  if (!std::isfinite(scale_log2) || !(scale > 0.f)) return FM_ERR_INVALID_ARG;
  if (mask && !vectors_ok(mask)) return FM_ERR_INVALID_ARG;
  if (!cache_shape_ok(B, H, cache->Hk, N, cache->d, max_pages)) return FM_ERR_UNSUPPORTED;
  if (mask && (mask->Hm <= 0 || H % mask->Hm != 0)) return FM_ERR_UNSUPPORTED;
  const fm::WeightsWs L = fm::weights_ws_layout(B, H, cache->Hk, N, cache->d, max_pages);
  const fm_status st = check_ws(ws, ws_bytes, L.total);
  if (st != FM_OK) return st;
  fm::WeightsParams p = {};
  p.f.q = static_cast<const uint16_t*>(q);
  for (int i = 0; i < 3; ++i) p.f.qs[i] = qs[i];
  p.f.c = cache_dev(cache);
  p.f.table = page_table;
  p.f.max_pages = max_pages;
  p.f.lens = lens;
  p.f.q_lens = q_lens;
  p.f.mask = mask_dev(mask);
  p.f.B = B;
  p.f.H = H;
  p.f.N = N;
  p.f.scale_log2 = scale_log2;
  p.lse = lse;
  p.weights = weights;
  p.start = start;
  char* w = static_cast<char*>(ws);
  p.f.status = reinterpret_cast<int32_t*>(w);
  p.f.list = reinterpret_cast<uint16_t*>(w + L.list);
  p.f.listed = reinterpret_cast<int32_t*>(w + L.listed);
  p.tiles = reinterpret_cast<uint8_t*>(w + L.tiles);
  p.partial = reinterpret_cast<float*>(w + L.partial);
  p.arrived = reinterpret_cast<int32_t*>(w + L.arrived);
  const int sms = sm_count();
  if (sms <= 0) return FM_ERR_CUDA;
  return fm::launch_cache_weights(cache->d, p, sms, static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? FM_OK
             : FM_ERR_CUDA;
}

size_t flashmask_cache_evict_workspace_bytes(int B, int Hk, int max_pages) {
  if (!cache_shape_ok(B, Hk, Hk, 1, 64, max_pages)) return 0;
  return fm::evict_ws_layout(B, Hk, max_pages).total;
}

fm_status flashmask_cache_evict(const fm_cache* cache, const int32_t* page_table, int max_pages,
                                const int32_t* out_table, int out_pages, const int32_t* lens, float* weights,
                                const int32_t* keep, int budget, int sink, int recent, int32_t* new_lens,
                                int32_t* index, int index_width, int B, void* ws, size_t ws_bytes, void* stream) {
  const fm_status cs = cache_ok(cache);
  if (cs != FM_OK) return cs;
  if (!page_table || !lens || !weights || !new_lens) return FM_ERR_INVALID_ARG;
  if (!aligned4(page_table) || !aligned4(out_table) || !aligned4(lens) || !aligned4(weights) || !aligned4(keep) ||
      !aligned4(new_lens) || !aligned4(index))
    return FM_ERR_INVALID_ARG;
  if (sink < 0 || recent < 0 || (!keep && budget < 0) || (index && index_width < 0)) return FM_ERR_INVALID_ARG;
  if (!cache_shape_ok(B, cache->Hk, cache->Hk, 1, cache->d, max_pages)) return FM_ERR_UNSUPPORTED;
  if (out_table && (out_pages <= 0 || out_pages > FM_MAX_SEQLEN / FM_PAGE)) return FM_ERR_UNSUPPORTED;
  if (out_table == page_table && out_pages != max_pages) return FM_ERR_INVALID_ARG;
  const fm::EvictWs L = fm::evict_ws_layout(B, cache->Hk, max_pages);
  const fm_status st = check_ws(ws, ws_bytes, L.total);
  if (st != FM_OK) return st;
  fm::EvictParams p = {};
  p.c = cache_dev(cache);
  p.table = page_table;
  p.max_pages = max_pages;
  p.out_table = out_table == page_table ? nullptr : out_table;
  p.out_pages = out_pages;
  p.lens = lens;
  p.weights = weights;
  p.keep = keep;
  p.budget = budget;
  p.sink = sink;
  p.recent = recent;
  p.new_lens = new_lens;
  p.index = index;
  p.index_width = index_width;
  p.B = B;
  char* w = static_cast<char*>(ws);
  p.status = reinterpret_cast<int32_t*>(w);
  p.count = reinterpret_cast<int32_t*>(w + L.counters);
  p.ticket = p.count + 1;
  p.done = p.count + 2;
  p.info = reinterpret_cast<int32_t*>(w + L.info);
  p.mask = reinterpret_cast<uint64_t*>(w + L.mask);
  p.before = reinterpret_cast<int32_t*>(w + L.before);
  p.list = reinterpret_cast<int2*>(w + L.list);
  p.was_read = reinterpret_cast<int32_t*>(w + L.was_read);
  const int sms = sm_count();
  if (sms <= 0) return FM_ERR_CUDA;
  return fm::launch_cache_evict(cache->d, p, sms, static_cast<cudaStream_t>(stream)) == cudaSuccess
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
  p.mask = mask_dev(mask);
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
