// Attention over the paged 8-bit cache.
#include "common.cuh"
#include "e4m3.cuh"
#include "internal.h"
#include "visible.cuh"

namespace spr {
namespace {

constexpr int kRowThreads = 128;

// Keys and values of one sequence and head through its table row.
template <int D>
struct PagedKV {
  const CacheArgs& a;
  const int32_t* row;
  int h;
  __device__ bool ok(int j) const {
    const int id = row[j / a.p.page];
    if (id >= 0 && id < a.p.n_pages) return true;
    raise_status(a.stats, SPARSEPR_ERR_INVALID_ARG);
    return false;
  }
  __device__ size_t slot(int j) const {
    return static_cast<size_t>(row[j / a.p.page]) * a.p.Hkv + h;
  }
  __device__ float dot(int j, const float* q) const {
    const uint8_t* k = static_cast<const uint8_t*>(a.c.k8) +
                       (slot(j) * a.p.page + j % a.p.page) * D;
    float s = 0.f;
    for (int c = 0; c < D; ++c) s += q[c] * from_e4m3(k[c]);
    return s * a.c.k_scale[slot(j)];
  }
  __device__ float v(int j, int c) const {
    const uint8_t* x = static_cast<const uint8_t*>(a.c.v8) +
                       (slot(j) * a.p.page + j % a.p.page) * D;
    return from_e4m3(x[c]) * a.c.v_scale[slot(j)];
  }
};

// One block per query row.
template <typename T, int D>
__global__ void __launch_bounds__(kRowThreads) cache_rows_kernel(const CacheAttnArgs a) {
  __shared__ LiteralScratch<kRowThreads> sm;
  __shared__ float q[D];
  const int i = blockIdx.x, bh = blockIdx.y, b = bh / a.Hq, h = bh % a.Hq;
  const bool report = i == 0 && h == 0 && threadIdx.x == 0;
  const CacheArgs& c = a.cache;
  const int n = clamp_count(a.n_q, b, a.Nq, a.Nq, c.stats, report);
  const int L = clamp_count(c.c.len, b, c.p.max_pages * c.p.page, 0, c.stats, report);
  if (i >= n) return;
  const size_t row = static_cast<size_t>(bh) * a.Nq + i;
  for (int x = threadIdx.x; x < D; x += kRowThreads)
    q[x] = load_f32(static_cast<const T*>(a.q) + row * D + x);
  __syncthreads();
  const PagedKV<D> kv = {c, c.c.table + static_cast<size_t>(b) * c.p.max_pages,
                         h / (a.Hq / c.p.Hkv)};
  float m, l, o;
  literal_row<kRowThreads, D>(kv, q, visible_range(a.see, static_cast<long long>(L) - n + i, L),
                              a.sc, sm, m, l, o);
  const float inv = l == 0.f ? 0.f : 1.f / l;
  for (int x = threadIdx.x; x < D; x += kRowThreads)
    store_f32(static_cast<T*>(a.out) + row * D + x, o * inv);
  if (a.lse && threadIdx.x == 0) a.lse[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2F;
}

}  // namespace

cudaError_t launch_cache_attention(const CacheAttnArgs& a, cudaStream_t st) {
  if (a.Nq == 0) return cudaSuccess;
  const dim3 grid(a.Nq, a.cache.p.B * a.Hq);
  if (a.bf16) {
    if (a.cache.p.d == 128) cache_rows_kernel<__nv_bfloat16, 128><<<grid, kRowThreads, 0, st>>>(a);
    else cache_rows_kernel<__nv_bfloat16, 64><<<grid, kRowThreads, 0, st>>>(a);
  } else {
    if (a.cache.p.d == 128) cache_rows_kernel<float, 128><<<grid, kRowThreads, 0, st>>>(a);
    else cache_rows_kernel<float, 64><<<grid, kRowThreads, 0, st>>>(a);
  }
  return cudaGetLastError();
}

}  // namespace spr
