// C ABI of the windowed attention and the 8-bit cache: argument checks,
// workspace carving and launches. The contract of every entry point is in
// include/sparsepr.h.
#include <math.h>

#include "common.cuh"
#include "internal.h"
#include "visible.cuh"

using namespace spr;

namespace {

bool al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
bool al4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3) == 0; }

sparsepr_status cuda_status(cudaError_t e) {
  return e == cudaSuccess ? SPARSEPR_OK : SPARSEPR_ERR_CUDA;
}

bool known_dtype(sparsepr_dtype dt) { return dt == SPARSEPR_BF16 || dt == SPARSEPR_F32; }

sparsepr_status check_see(const sparsepr_visibility& s) {
  if (s.frame < 1 || s.window < 0 || s.sinks < 0) return SPARSEPR_ERR_INVALID_ARG;
  if (s.causal != 0 && s.causal != 1) return SPARSEPR_ERR_INVALID_ARG;
  return SPARSEPR_OK;
}

// scale log2(e) as the kernels take it: at least the least normal number, since a masked
// logit is -inf times it. (Products below 2^100 give logits of 0 there, to fp32's bits.)
float log2_scale(double scale, int d) {
  const double s = scale > 0.0 ? scale : 1.0 / sqrt(static_cast<double>(d));
  return fmaxf(static_cast<float>(s * 1.4426950408889634074), 1.17549435e-38f);
}
bool good_scale(double scale) { return scale >= 0.0 && isfinite(log2_scale(scale, 64)); }

// sizes that index arithmetic and launch grids hold
constexpr long long kMaxRows = (1ll << 31) - 1;
constexpr long long kMaxHeads = 65535;

sparsepr_status check_window(const sparsepr_window_params* p) {
  if (!p) return SPARSEPR_ERR_INVALID_ARG;
  if (p->B < 1 || p->Hkv < 1 || p->Hq < 1 || p->Hq % p->Hkv != 0) return SPARSEPR_ERR_INVALID_ARG;
  if (p->Nq < 0 || p->Nk < 0) return SPARSEPR_ERR_INVALID_ARG;
  const sparsepr_status s = check_see(p->see);
  if (s != SPARSEPR_OK) return s;
  if (!good_scale(p->scale)) return SPARSEPR_ERR_INVALID_ARG;
  if (p->d != 64 && p->d != 128) return SPARSEPR_ERR_UNSUPPORTED;
  const long long bh = static_cast<long long>(p->B) * p->Hq;
  if (bh > kMaxHeads || bh * p->Nq > kMaxRows ||
      static_cast<long long>(p->B) * p->Hkv * p->Nk > kMaxRows)
    return SPARSEPR_ERR_UNSUPPORTED;
  return SPARSEPR_OK;
}

sparsepr_status check_cache(const sparsepr_cache_params* p) {
  if (!p) return SPARSEPR_ERR_INVALID_ARG;
  if (p->B < 1 || p->B > 1024 || p->Hkv < 1 || p->Hkv > 1024) return SPARSEPR_ERR_INVALID_ARG;
  if (p->n_pages < 1 || p->max_pages < 1) return SPARSEPR_ERR_INVALID_ARG;
  if (p->page != 16 && p->page != 32 && p->page != 64 && p->page != 128)
    return SPARSEPR_ERR_UNSUPPORTED;
  if (p->d != 64 && p->d != 128) return SPARSEPR_ERR_UNSUPPORTED;
  if (static_cast<long long>(p->max_pages) * p->page > kMaxRows) return SPARSEPR_ERR_UNSUPPORTED;
  return SPARSEPR_OK;
}

sparsepr_status check_cache_attention(const sparsepr_cache_params* p,
                                      const sparsepr_cache_attention_params* a) {
  sparsepr_status s = check_cache(p);
  if (s != SPARSEPR_OK) return s;
  if (!a || a->Hq < 1 || a->Hq % p->Hkv != 0 || a->Nq < 0) return SPARSEPR_ERR_INVALID_ARG;
  s = check_see(a->see);
  if (s != SPARSEPR_OK) return s;
  if (!good_scale(a->scale)) return SPARSEPR_ERR_INVALID_ARG;
  const long long bh = static_cast<long long>(p->B) * a->Hq;
  if (bh > kMaxHeads || bh * a->Nq > kMaxRows) return SPARSEPR_ERR_UNSUPPORTED;
  // tiles of all sequences are counted in 32 bits
  if (p->B * (static_cast<long long>(p->max_pages) * p->page / 32 + 4) > kMaxRows)
    return SPARSEPR_ERR_UNSUPPORTED;
  return SPARSEPR_OK;
}

// Workspace regions at 256-byte steps; with base null only sizes are counted.
struct Carver {
  char* base;
  size_t at = 0;
  template <typename T>
  T* take(size_t count) {
    T* p = base ? reinterpret_cast<T*>(base + at) : nullptr;
    at += (count * sizeof(T) + 255) / 256 * 256;
    return p;
  }
};

sparsepr_status check_ws(const void* ws, size_t ws_bytes, size_t need) {
  if (!ws || (reinterpret_cast<uintptr_t>(ws) & 255) != 0 || ws_bytes < need)
    return SPARSEPR_ERR_WORKSPACE;
  return SPARSEPR_OK;
}

int sm_count() {
  int dev = 0, n = 148;
  if (cudaGetDevice(&dev) == cudaSuccess)
    cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
  return n;
}

size_t carve_window(const sparsepr_window_params& p, sparsepr_dtype dt, char* base, WindowArgs* a) {
  Carver w{base};
  a->stats = w.take<DeviceStats>(1);
  const size_t q = static_cast<size_t>(p.B) * p.Hq * p.Nq * p.d;
  const size_t kv = static_cast<size_t>(p.B) * p.Hkv * p.Nk * p.d;
  if (dt == SPARSEPR_F32) {
    a->qb = w.take<__nv_bfloat16>(q);
    a->kb = w.take<__nv_bfloat16>(kv);
    a->vb = w.take<__nv_bfloat16>(kv);
  }
  if (p.Nq > 0) {
    const WindowPlan plan = window_plan(p.B, p.Hq, p.Hkv, p.Nq, p.Nk, p.see);
    a->opart = w.take<float>(plan.part_rows * p.d);
    a->lpart = w.take<float>(plan.part_rows);
  }
  return w.at;
}

size_t carve_cache(const sparsepr_cache_params& p, char* base, CacheArgs* a) {
  Carver w{base};
  a->stats = w.take<DeviceStats>(1);
  a->counts = w.take<int32_t>(16);
  a->pages = w.take<int32_t>(p.n_pages);
  a->targets = w.take<int32_t>(p.n_pages);
  a->remap = w.take<int32_t>(p.n_pages);
  a->copies = w.take<int32_t>(2 * static_cast<size_t>(p.B));
  return w.at;
}

size_t carve_cache_attention(const sparsepr_cache_params& p,
                             const sparsepr_cache_attention_params& q, char* base,
                             CacheAttnArgs* a) {
  Carver w{base};
  w.at = carve_cache(p, base, &a->cache);
  if (q.Nq > 0) {
    const CacheAttnPlan plan = cache_attn_plan(p, q);
    a->pre = w.take<int32_t>(p.B + 2);
    a->opart = w.take<float>(plan.part_rows * p.d);
    a->lpart = w.take<float>(plan.part_rows);
    if (plan.wide) {
      const size_t kv = static_cast<size_t>(plan.group) * p.Hkv * plan.cap * p.d;
      a->kb = w.take<__nv_bfloat16>(kv);
      a->vb = w.take<__nv_bfloat16>(kv);
      // whatever the dtype of q: the size does not know it
      a->qb = w.take<__nv_bfloat16>(static_cast<size_t>(plan.group) * q.Hq * q.Nq * p.d);
    }
  }
  return w.at;
}

// Checks shared by the cache calls; fills the arguments.
sparsepr_status cache_setup(const sparsepr_cache_params* p, const sparsepr_cache* c, void* ws,
                            size_t ws_bytes, CacheArgs* a) {
  const sparsepr_status s = check_cache(p);
  if (s != SPARSEPR_OK) return s;
  if (!c || !c->k8 || !c->v8 || !c->k_scale || !c->v_scale || !c->table || !c->len || !c->ref)
    return SPARSEPR_ERR_INVALID_ARG;
  if (!al16(c->k8) || !al16(c->v8) || !al4(c->k_scale) || !al4(c->v_scale) || !al4(c->table) ||
      !al4(c->len) || !al4(c->ref) || c->k8 == c->v8)
    return SPARSEPR_ERR_INVALID_ARG;
  a->p = *p;
  a->c = *c;
  a->sm_count = sm_count();
  return check_ws(ws, ws_bytes, carve_cache(*p, static_cast<char*>(ws), a));
}

}  // namespace

extern "C" {

size_t sparsepr_window_workspace_bytes(const sparsepr_window_params* p, sparsepr_dtype dt) {
  if (check_window(p) != SPARSEPR_OK || !known_dtype(dt)) return 0;
  WindowArgs a = {};
  return carve_window(*p, dt, nullptr, &a);
}

sparsepr_status sparsepr_window_attention(const void* q, const void* k, const void* v,
                                          sparsepr_dtype dt, const sparsepr_window_params* p,
                                          const int32_t* n_q, const int32_t* n_k, void* out,
                                          float* lse, void* ws, size_t ws_bytes, void* stream) {
  sparsepr_status s = check_window(p);
  if (s != SPARSEPR_OK) return s;
  if (!known_dtype(dt)) return SPARSEPR_ERR_UNSUPPORTED;
  if (p->Nq > 0 && (!q || !out)) return SPARSEPR_ERR_INVALID_ARG;
  if (p->Nk > 0 && (!k || !v)) return SPARSEPR_ERR_INVALID_ARG;
  if (!al16(q) || !al16(k) || !al16(v) || !al16(out) || !al4(lse) || !al4(n_q) || !al4(n_k))
    return SPARSEPR_ERR_INVALID_ARG;
  if (p->Nq > 0 && (out == q || out == k || out == v)) return SPARSEPR_ERR_INVALID_ARG;
  WindowArgs a = {};
  s = check_ws(ws, ws_bytes, carve_window(*p, dt, static_cast<char*>(ws), &a));
  if (s != SPARSEPR_OK) return s;
  if (p->Nq == 0) return SPARSEPR_OK;
  a.q = q;
  a.k = k;
  a.v = v;
  a.out = out;
  a.lse = lse;
  a.n_q = n_q;
  a.n_k = n_k;
  a.B = p->B;
  a.Hq = p->Hq;
  a.Hkv = p->Hkv;
  a.Nq = p->Nq;
  a.Nk = p->Nk;
  a.d = p->d;
  a.see = p->see;
  a.sc = log2_scale(p->scale, p->d);
  a.bf16 = a.kv_bf16 = dt == SPARSEPR_BF16;
  return cuda_status(launch_window_attention(a, static_cast<cudaStream_t>(stream)));
}

size_t sparsepr_cache_workspace_bytes(const sparsepr_cache_params* p,
                                      const sparsepr_cache_attention_params* q) {
  CacheAttnArgs a = {};
  if (!q) return check_cache(p) == SPARSEPR_OK ? carve_cache(*p, nullptr, &a.cache) : 0;
  if (check_cache_attention(p, q) != SPARSEPR_OK) return 0;
  return carve_cache_attention(*p, *q, nullptr, &a);
}

sparsepr_status sparsepr_cache_reserve(const sparsepr_cache_params* p, const sparsepr_cache* c,
                                       const int32_t* n_new, int32_t* start, void* ws,
                                       size_t ws_bytes, void* stream) {
  CacheArgs a = {};
  const sparsepr_status s = cache_setup(p, c, ws, ws_bytes, &a);
  if (s != SPARSEPR_OK) return s;
  if (!n_new || !start || !al4(n_new) || !al4(start) || start == n_new || start == c->len)
    return SPARSEPR_ERR_INVALID_ARG;
  return cuda_status(launch_cache_reserve(a, n_new, start, static_cast<cudaStream_t>(stream)));
}

sparsepr_status sparsepr_cache_append(const void* k, const void* v, sparsepr_dtype dt, int32_t T,
                                      const sparsepr_cache_params* p, const sparsepr_cache* c,
                                      const int32_t* start, const int32_t* n_new, void* ws,
                                      size_t ws_bytes, void* stream) {
  CacheArgs a = {};
  const sparsepr_status s = cache_setup(p, c, ws, ws_bytes, &a);
  if (s != SPARSEPR_OK) return s;
  if (!known_dtype(dt)) return SPARSEPR_ERR_UNSUPPORTED;
  if (T < 0 || !start || !al4(start) || !al4(n_new)) return SPARSEPR_ERR_INVALID_ARG;
  if (T > 0 && (!k || !v || !al16(k) || !al16(v))) return SPARSEPR_ERR_INVALID_ARG;
  if (T / p->page + 2 > kMaxHeads || static_cast<long long>(p->B) * p->Hkv * T > kMaxRows)
    return SPARSEPR_ERR_UNSUPPORTED;
  if (T == 0) return SPARSEPR_OK;
  return cuda_status(launch_cache_append(a, k, v, dt == SPARSEPR_BF16, T, start, n_new,
                                         static_cast<cudaStream_t>(stream)));
}

sparsepr_status sparsepr_cache_attention(const void* q, sparsepr_dtype dt,
                                         const sparsepr_cache_params* p, const sparsepr_cache* c,
                                         const sparsepr_cache_attention_params* qa,
                                         const int32_t* n_q, void* out, float* lse, void* ws,
                                         size_t ws_bytes, void* stream) {
  CacheAttnArgs a = {};
  sparsepr_status s = check_cache_attention(p, qa);
  if (s != SPARSEPR_OK) return s;
  s = cache_setup(p, c, ws, ws_bytes, &a.cache);
  if (s != SPARSEPR_OK) return s;
  if (!known_dtype(dt)) return SPARSEPR_ERR_UNSUPPORTED;
  if (qa->Nq > 0 && (!q || !out || out == q)) return SPARSEPR_ERR_INVALID_ARG;
  if (!al16(q) || !al16(out) || !al4(lse) || !al4(n_q)) return SPARSEPR_ERR_INVALID_ARG;
  s = check_ws(ws, ws_bytes, carve_cache_attention(*p, *qa, static_cast<char*>(ws), &a));
  if (s != SPARSEPR_OK) return s;
  if (qa->Nq == 0) return SPARSEPR_OK;
  a.q = q;
  a.out = out;
  a.lse = lse;
  a.n_q = n_q;
  a.Hq = qa->Hq;
  a.Nq = qa->Nq;
  a.see = qa->see;
  a.sc = log2_scale(qa->scale, p->d);
  a.bf16 = dt == SPARSEPR_BF16;
  return cuda_status(launch_cache_attention(a, static_cast<cudaStream_t>(stream)));
}

sparsepr_status sparsepr_cache_fork(const sparsepr_cache_params* p, const sparsepr_cache* c,
                                    const int32_t* src, const int32_t* dst, int32_t n, void* ws,
                                    size_t ws_bytes, void* stream) {
  CacheArgs a = {};
  const sparsepr_status s = cache_setup(p, c, ws, ws_bytes, &a);
  if (s != SPARSEPR_OK) return s;
  if (n < 0 || (n > 0 && (!src || !dst || !al4(src) || !al4(dst)))) return SPARSEPR_ERR_INVALID_ARG;
  if (n == 0) return SPARSEPR_OK;
  return cuda_status(launch_cache_fork(a, src, dst, n, static_cast<cudaStream_t>(stream)));
}

sparsepr_status sparsepr_cache_free(const sparsepr_cache_params* p, const sparsepr_cache* c,
                                    const int32_t* seq, int32_t n, void* ws, size_t ws_bytes,
                                    void* stream) {
  CacheArgs a = {};
  const sparsepr_status s = cache_setup(p, c, ws, ws_bytes, &a);
  if (s != SPARSEPR_OK) return s;
  if (n < 0 || (n > 0 && (!seq || !al4(seq)))) return SPARSEPR_ERR_INVALID_ARG;
  if (n == 0) return SPARSEPR_OK;
  return cuda_status(launch_cache_free(a, seq, n, static_cast<cudaStream_t>(stream)));
}

sparsepr_status sparsepr_cache_evict(const sparsepr_cache_params* p, const sparsepr_cache* c,
                                     const sparsepr_visibility* see, void* ws, size_t ws_bytes,
                                     void* stream) {
  CacheArgs a = {};
  const sparsepr_status s = cache_setup(p, c, ws, ws_bytes, &a);
  if (s != SPARSEPR_OK) return s;
  if (!see || check_see(*see) != SPARSEPR_OK || !see->causal || see->window < 1)
    return SPARSEPR_ERR_INVALID_ARG;
  return cuda_status(launch_cache_evict(a, *see, static_cast<cudaStream_t>(stream)));
}

sparsepr_status sparsepr_cache_compact(const sparsepr_cache_params* p, const sparsepr_cache* c,
                                       int32_t* n_used, void* ws, size_t ws_bytes, void* stream) {
  CacheArgs a = {};
  const sparsepr_status s = cache_setup(p, c, ws, ws_bytes, &a);
  if (s != SPARSEPR_OK) return s;
  if (!n_used || !al4(n_used)) return SPARSEPR_ERR_INVALID_ARG;
  return cuda_status(launch_cache_compact(a, n_used, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
