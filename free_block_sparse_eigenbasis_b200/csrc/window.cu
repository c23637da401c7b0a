// Attention with a sliding window of frames and sink frames.
#include "common.cuh"
#include "internal.h"
#include "visible.cuh"

namespace spr {
namespace {

constexpr int kRowThreads = 128;

template <typename T, int D>
struct DenseKV {
  const T *k, *vals;  // this head's rows
  __device__ bool ok(int) const { return true; }
  __device__ float dot(int j, const float* q) const {
    const T* row = k + static_cast<size_t>(j) * D;
    float s = 0.f;
    for (int c = 0; c < D; ++c) s += q[c] * load_f32(row + c);
    return s;
  }
  __device__ float v(int j, int c) const { return load_f32(vals + static_cast<size_t>(j) * D + c); }
};

// One block per query row.
template <typename T, int D>
__global__ void __launch_bounds__(kRowThreads) window_rows_kernel(const WindowArgs a) {
  __shared__ LiteralScratch<kRowThreads> sm;
  __shared__ float q[D];
  const int i = blockIdx.x, bh = blockIdx.y, b = bh / a.Hq, h = bh % a.Hq;
  const bool report = i == 0 && h == 0 && threadIdx.x == 0;
  const int n = clamp_count(a.n_q, b, a.Nq, a.Nq, a.stats, report);
  const int L = clamp_count(a.n_k, b, a.Nk, a.Nk, a.stats, report);
  if (i >= n) return;
  const size_t row = static_cast<size_t>(bh) * a.Nq + i;
  for (int c = threadIdx.x; c < D; c += kRowThreads)
    q[c] = load_f32(static_cast<const T*>(a.q) + row * D + c);
  __syncthreads();
  const size_t base = (static_cast<size_t>(b) * a.Hkv + h / (a.Hq / a.Hkv)) * a.Nk * D;
  const DenseKV<T, D> kv = {static_cast<const T*>(a.k) + base, static_cast<const T*>(a.v) + base};
  float m, l, o;
  literal_row<kRowThreads, D>(kv, q, visible_range(a.see, static_cast<long long>(L) - n + i, L),
                              a.sc, sm, m, l, o);
  const float inv = l == 0.f ? 0.f : 1.f / l;
  for (int c = threadIdx.x; c < D; c += kRowThreads)
    store_f32(static_cast<T*>(a.out) + row * D + c, o * inv);
  if (a.lse && threadIdx.x == 0) a.lse[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2F;
}

}  // namespace

cudaError_t launch_window_attention(const WindowArgs& a, cudaStream_t st) {
  if (a.Nq == 0) return cudaSuccess;
  const dim3 grid(a.Nq, a.B * a.Hq);
  if (a.bf16) {
    if (a.d == 128) window_rows_kernel<__nv_bfloat16, 128><<<grid, kRowThreads, 0, st>>>(a);
    else window_rows_kernel<__nv_bfloat16, 64><<<grid, kRowThreads, 0, st>>>(a);
  } else {
    if (a.d == 128) window_rows_kernel<float, 128><<<grid, kRowThreads, 0, st>>>(a);
    else window_rows_kernel<float, 64><<<grid, kRowThreads, 0, st>>>(a);
  }
  return cudaGetLastError();
}

}  // namespace spr
