// Visibility by frames (sparsepr_visibility) and the attention of one row
// taken literally, shared by the windowed attention and the attention over
// the cache.
#pragma once

#include "common.cuh"

namespace spr {

constexpr float kLog2eF = 1.4426950408889634f;
constexpr float kLn2F = 0.6931471805599453f;

// Visible keys of a query: [0, s) and [lo, hi), disjoint, s <= lo <= hi <= L.
struct Range {
  int s, lo, hi;
};

// Division of n < 2^31 by an invariant d >= 1, as a product, an addition and a shift
// (Granlund and Montgomery, "Division by invariant integers using multiplication",
// 1994): with l = ceil(log2 d) and m = floor(2^32 (2^l - d) / d) + 1,
// n / d = (floor(m n / 2^32) + n) >> l; the sum stays below 2^32.
struct Divider {
  uint32_t d, mul, shift;
  Divider() = default;
  explicit Divider(int by) : d(static_cast<uint32_t>(by)), shift(0) {
    while ((1ull << shift) < d) ++shift;
    mul = static_cast<uint32_t>(((1ull << 32) * ((1ull << shift) - d)) / d + 1);
  }
  __device__ int div(int n) const {
    return static_cast<int>((__umulhi(mul, static_cast<uint32_t>(n)) + n) >> shift);
  }
  __device__ int mod(int n) const { return n - div(n) * static_cast<int>(d); }
};
struct PlainDivision {
  int d;
  __host__ __device__ int div(int n) const {
    return static_cast<int>(static_cast<uint32_t>(n) / static_cast<uint32_t>(d));
  }
};

// Keys that the query at position p of a sequence of L keys sees. All three
// ends grow with p, so the keys of a run of rows lie in [0, s of the last row)
// and [lo of the first, hi of the last).
// Positions, counts and frames are below 2^31. So is a frame's first position up to that
// of the query, and the end of its frame is below 2^32; only the products of sinks and of
// the window behind the query by the frame need more. by_frame divides by the frame.
template <class Division>
__host__ __device__ inline Range visible_range(const sparsepr_visibility& see, long long pos,
                                               int L, const Division& by_frame) {
  Range r = {0, 0, 0};
  if (pos < 0 || L <= 0) return r;
  const uint32_t p = static_cast<uint32_t>(pos), len = static_cast<uint32_t>(L);
  if (see.window == 0 && see.frame == 1) {  // every key, or every key up to its own
    r.hi = static_cast<int>(see.causal && p + 1 < len ? p + 1 : len);
    return r;
  }
  const uint32_t F = static_cast<uint32_t>(see.frame), W = static_cast<uint32_t>(see.window);
  const uint32_t next = (F == 1 ? p : static_cast<uint32_t>(by_frame.div(static_cast<int>(p)))) + 1;
  uint32_t end = len;  // keys a causal query may look at
  if (see.causal && next * F < len) end = next * F;
  const uint64_t sink = static_cast<uint64_t>(static_cast<uint32_t>(see.sinks)) * F;
  const uint32_t s = sink < end ? static_cast<uint32_t>(sink) : end;
  uint32_t lo = 0, hi = end;
  if (W > 0) {
    if (next > W) lo = (next - W) * F;
    const uint64_t behind = static_cast<uint64_t>(next - 1 + W) * F;
    if (!see.causal && behind < len) hi = static_cast<uint32_t>(behind);
  }
  if (lo < s) lo = s;
  if (hi < lo) hi = lo;
  r.s = static_cast<int>(s);
  r.lo = static_cast<int>(lo < len ? lo : len);
  r.hi = static_cast<int>(hi);
  return r;
}
__host__ __device__ inline Range visible_range(const sparsepr_visibility& see, long long p,
                                               int L) {
  return visible_range(see, p, L, PlainDivision{see.frame});
}

// Of `keys` keys, how many a run of `rows` rows can need at most. (The product of frames
// is formed only where it is at most `keys`.)
inline long long most_visible(const sparsepr_visibility& see, long long rows, long long keys) {
  if (see.window == 0) return keys;
  const long long frames = see.sinks + (see.causal ? 1ll : 2ll) * see.window + 1;
  if (frames > keys / see.frame) return keys;
  const long long span = frames * see.frame + rows;
  return span < keys ? span : keys;
}

// In-use rows of one sequence, clamped to what the buffers hold.
__device__ __forceinline__ int clamp_count(const int32_t* n, int b, int cap, int otherwise,
                                           DeviceStats* stats, bool report) {
  if (!n) return otherwise;
  const int v = n[b];
  if (report && (v < 0 || v > cap)) raise_status(stats, SPARSEPR_ERR_INVALID_ARG);
  return min(max(v, 0), cap);
}

__device__ __forceinline__ float load_f32(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ float load_f32(const float* p) { return *p; }
__device__ __forceinline__ void store_f32(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }
__device__ __forceinline__ void store_f32(float* p, float v) { *p = v; }

// One query row by the definition, by all NT threads of a block: a pass over
// its visible keys with a running maximum and sum, fp32 products, no key
// outside [0, s) and [lo, hi) touched. It is the reading of rows that meet
// NaN or infinities (a product with a hidden NaN is NaN even at weight 0).
//   kv.ok(j)      key j can be read
//   kv.dot(j, q)  q . k_j            kv.v(j, c, x)  x[e] = v_j[c + e], e < D / 32
// Returns the maximum m (log2 units, sc = scale * log2 e), the sum l and, in
// thread c < D, the unnormalised output o of column c; l is NaN for a row whose
// visible logits are all -inf, and 0 for a row that sees nothing.
// Called by the NT threads 0..NT-1 of a block, which `sync` joins. A thread has a key of
// its own in the first product, a warp in the second, every lane D / 32 columns of it.
template <int NT, int D>
struct LiteralScratch {
  float p[NT];
  float o[NT / 32][D];
  float red[32], sum[32];
  int any[32];
};

struct BlockSync {
  __device__ void operator()() const { __syncthreads(); }
};

template <int NT, int D, class KV, class Sync>
__device__ void literal_row(const KV& kv, const float* q, const Range r, float sc,
                            LiteralScratch<NT, D>& sm, const Sync& sync, float& m_out, float& l_out,
                            float& o_out) {
  static_assert(NT % 32 == 0 && NT >= D, "threads");
  constexpr int kWarpsHere = NT / 32, kC = D / 32;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int total = r.s + (r.hi - r.lo);
  float m = -INFINITY, l = 0.f, o[kC] = {};
  bool seen = false;
  for (int base = 0; base < total; base += NT) {
    const int t = base + tid;
    bool on = false;
    float x = -INFINITY;
    if (t < total) {
      const int j = t < r.s ? t : r.lo + (t - r.s);
      on = kv.ok(j);
      if (on) x = sc * kv.dot(j, q);
    }
    float mx = on ? x : -INFINITY;
#pragma unroll
    for (int w = 16; w > 0; w >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
    const bool any = __any_sync(0xffffffffu, on);
    if (lane == 0) {
      sm.red[warp] = mx;
      sm.any[warp] = any;
    }
    sync();
    for (int w = 0; w < kWarpsHere; ++w) {
      mx = fmaxf(mx, sm.red[w]);
      seen = seen || sm.any[w];
    }
    const float mn = fmaxf(m, mx);
    const float corr = (m == -INFINITY) ? 0.f : exp2f(m - mn);
    // weight of this thread's key; -1 marks a key that is not there
    float p = -1.f;
    if (on) p = (mn == -INFINITY) ? (x == x ? 0.f : x) : exp2f(x - mn);
    sm.p[tid] = p;
    float sum = p < 0.f ? 0.f : p;
#pragma unroll
    for (int w = 16; w > 0; w >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, w);
    if (lane == 0) sm.sum[warp] = sum;
    sync();
    sum = 0.f;
    for (int w = 0; w < kWarpsHere; ++w) sum += sm.sum[w];  // the same order in every thread
    l = l * corr + sum;
#pragma unroll
    for (int e = 0; e < kC; ++e) o[e] *= corr;
    const int n = min(NT, total - base);
    constexpr int kAhead = 8;  // keys in flight
    for (int i0 = warp; i0 < n; i0 += kWarpsHere * kAhead) {
      float w[kAhead], v[kAhead][kC];
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const int i = i0 + k * kWarpsHere, u = base + i;
        w[k] = i < n ? sm.p[i] : -1.f;
        if (w[k] < 0.f) {
          w[k] = 0.f;
#pragma unroll
          for (int e = 0; e < kC; ++e) v[k][e] = 0.f;
        } else {
          kv.v(u < r.s ? u : r.lo + (u - r.s), lane * kC, v[k]);
        }
      }
#pragma unroll
      for (int k = 0; k < kAhead; ++k)
#pragma unroll
        for (int e = 0; e < kC; ++e) o[e] += w[k] * v[k][e];
    }
    m = mn;
    sync();
  }
#pragma unroll
  for (int e = 0; e < kC; ++e) sm.o[warp][lane * kC + e] = o[e];
  sync();
  float all = 0.f;
  if (tid < D)
    for (int w = 0; w < kWarpsHere; ++w) all += sm.o[w][tid];
  if (seen && l == 0.f) l = __int_as_float(0x7fc00000);
  sync();
  m_out = m;
  l_out = l;
  o_out = all;
}

}  // namespace spr
