// The paged cache in 8 bits: new tokens written with one power-of-two scale
// for each page and head, and the bookkeeping of pages (reserve, fork, free,
// evict, compact), all on the device so that a step can be captured whole.
#include "common.cuh"
#include "e4m3.cuh"
#include "internal.h"
#include "visible.cuh"

namespace spr {
namespace {

constexpr int kPlanThreads = 1024;  // one block plans; a thread per sequence (B <= 1024)
constexpr int kMinScaleExp = -110;

// Exclusive prefix sum of v over the kPlanThreads threads of the block, the total
// in every thread. Calls alternate between two sets of warp sums, so one barrier
// a call is enough.
template <typename I>
struct PlanScan {
  I sums[2][32];
};
template <typename I>
__device__ __forceinline__ I block_scan(I v, PlanScan<I>& sc, int& turn, I* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  I x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const I y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) sc.sums[turn][warp] = x;
  __syncthreads();
  I w = sc.sums[turn][lane];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const I y = __shfl_up_sync(0xffffffffu, w, o);
    if (lane >= o) w += y;
  }
  turn ^= 1;
  *total = __shfl_sync(0xffffffffu, w, 31);
  const I before = __shfl_sync(0xffffffffu, w, max(warp - 1, 0));
  return (warp ? before : 0) + x - v;
}

constexpr int kPerThread = 4;  // pages of a thread in one round over the pool
constexpr int kRound = kPlanThreads * kPerThread;

// ref of this thread's pages of a round, contiguous; past the pool: -1
__device__ __forceinline__ void load_refs(const int32_t* ref, int n_pages, int base,
                                          int (&r)[kPerThread]) {
#pragma unroll
  for (int e = 0; e < kPerThread; ++e) {
    const int id = base + static_cast<int>(threadIdx.x) * kPerThread + e;
    r[e] = id < n_pages ? ref[id] : -1;
  }
}

__device__ __forceinline__ bool page_ok(const CacheArgs& a, int id) {
  return id >= 0 && id < a.p.n_pages;
}

__global__ void __launch_bounds__(kPlanThreads)
    reserve_kernel(const CacheArgs a, const int32_t* n_new, int32_t* start) {
  __shared__ PlanScan<long long> scan64;
  __shared__ PlanScan<int> scan32;
  __shared__ int first[kPlanThreads + 1];  // first new page of each sequence
  int turn64 = 0, turn32 = 0;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int b = threadIdx.x, page = a.p.page;
  const bool mine = b < a.p.B;
  const long long room = static_cast<long long>(a.p.max_pages) * page;
  int n = 0, len = 0, old = -1;
  long long need = 0;
  bool bad = false, full = false;
  if (mine) {
    n = n_new[b];
    len = a.c.len[b];
    if (n < 0 || len < 0 || len > room) {
      bad = true;
    } else if (len + static_cast<long long>(n) > room) {
      full = true;
    } else if (n > 0) {
      need = (len + static_cast<long long>(n) + page - 1) / page - (len + page - 1) / page;
      if (len % page) {
        const int id = a.c.table[static_cast<size_t>(b) * a.p.max_pages + len / page];
        if (!page_ok(a, id)) {
          bad = true;
        } else if (a.c.ref[id] > 1) {
          old = id;
          ++need;
        }
      }
    }
  }
  bad = __syncthreads_or(bad);
  full = __syncthreads_or(full);
  long long total;
  const long long before = block_scan(need, scan64, turn64, &total);
  if (total > a.p.n_pages) full = true;
  // the first `total` free pages, ascending
  long long found = 0;
  if (!bad && !full)
    for (long long base = 0; base < a.p.n_pages && found < total; base += kRound) {
      int r[kPerThread], mine_free = 0, here;
      load_refs(a.c.ref, a.p.n_pages, static_cast<int>(base), r);
#pragma unroll
      for (int e = 0; e < kPerThread; ++e) mine_free += r[e] == 0;
      long long at = found + block_scan(mine_free, scan32, turn32, &here);
#pragma unroll
      for (int e = 0; e < kPerThread; ++e)
        if (r[e] == 0) {
          if (at < total) a.pages[at] = static_cast<int>(base) + b * kPerThread + e;
          ++at;
        }
      found += here;
    }
  if (found < total) full = true;
  if (mine) a.copies[b] = -1;
  if (bad || full) {  // the same in every thread
    if (mine) start[b] = -1;
    if (b == 0) raise_status(a.stats, bad ? SPARSEPR_ERR_INVALID_ARG : SPARSEPR_ERR_CAPACITY);
    return;
  }
  first[b] = static_cast<int>(mine ? before : total);
  if (b == 0) first[kPlanThreads] = static_cast<int>(total);
  __syncthreads();
  if (mine) {
    start[b] = len;
    a.c.len[b] = len + n;
    if (old >= 0) {
      a.copies[b] = old;
      a.copies[a.p.B + b] = a.pages[before];
      atomicSub(&a.c.ref[old], 1);
    }
  }
  __syncthreads();
  // new page k goes to the sequence b with first[b] <= k < first[b + 1]
  for (int k = b; k < static_cast<int>(total); k += kPlanThreads) {
    int lo = 0, hi = a.p.B;  // first[lo] <= k < first[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (first[mid] <= k) lo = mid;
      else hi = mid;
    }
    const int s = start[lo], id = a.pages[k];
    const bool copied = a.copies[lo] >= 0;
    // a copied last page takes its old column, the others follow the last one
    const int col = copied ? s / page + (k - first[lo]) : (s + page - 1) / page + (k - first[lo]);
    a.c.table[static_cast<size_t>(lo) * a.p.max_pages + col] = id;
    a.c.ref[id] = 1;
  }
}

constexpr int kCopyThreads = 256, kCopyPieces = 1024;  // 16 KB of one page per block

// 16-byte pieces [i0, i0 + kCopyPieces) of page src to page dst, keys or values: four
// loads in flight per thread
__device__ __forceinline__ void copy_pieces(const CacheArgs& a, const void* pool, long long src,
                                            long long dst, int i0) {
  constexpr int kEach = kCopyPieces / kCopyThreads;
  const int pieces = a.p.Hkv * (a.p.page * a.p.d / 16);
  const uint4* from = static_cast<const uint4*>(pool) + src * pieces;
  uint4* to = static_cast<uint4*>(const_cast<void*>(pool)) + dst * pieces;
  uint4 x[kEach];
#pragma unroll
  for (int e = 0; e < kEach; ++e) {
    const int i = i0 + e * kCopyThreads + static_cast<int>(threadIdx.x);
    if (i < pieces) x[e] = __ldcs(from + i);
  }
#pragma unroll
  for (int e = 0; e < kEach; ++e) {
    const int i = i0 + e * kCopyThreads + static_cast<int>(threadIdx.x);
    if (i < pieces) __stcs(to + i, x[e]);
  }
}
__device__ __forceinline__ void copy_scales(const CacheArgs& a, long long src, long long dst) {
  for (int h = threadIdx.x; h < a.p.Hkv; h += blockDim.x) {
    a.c.k_scale[dst * a.p.Hkv + h] = a.c.k_scale[src * a.p.Hkv + h];
    a.c.v_scale[dst * a.p.Hkv + h] = a.c.v_scale[src * a.p.Hkv + h];
  }
}

__global__ void __launch_bounds__(kCopyThreads) copy_last_pages_kernel(const CacheArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the plan
  const int b = blockIdx.y, src = a.copies[b];
  if (src < 0) return;
  const int dst = a.copies[a.p.B + b];
  copy_pieces(a, blockIdx.z ? a.c.v8 : a.c.k8, src, dst, blockIdx.x * kCopyPieces);
  if (blockIdx.x == 0 && blockIdx.z == 0) copy_scales(a, src, dst);
}

__global__ void __launch_bounds__(128)
    fork_kernel(const CacheArgs a, const int32_t* src, const int32_t* dst, int n) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int i = blockIdx.x, s = src[i], t = dst[i];
  bool ok = s >= 0 && s < a.p.B && t >= 0 && t < a.p.B;
  // no valid pair writes a row that another pair reads or writes
  if (ok) {
    ok = a.c.len[t] == 0;
    for (int j = threadIdx.x; j < n; j += blockDim.x)
      if ((j != i && dst[j] == t) || src[j] == t) ok = false;
  }
  if (!__syncthreads_and(ok)) {
    if (threadIdx.x == 0) raise_status(a.stats, SPARSEPR_ERR_INVALID_ARG);
    return;
  }
  const int32_t* from = a.c.table + static_cast<size_t>(s) * a.p.max_pages;
  int32_t* to = a.c.table + static_cast<size_t>(t) * a.p.max_pages;
  for (int j = threadIdx.x; j < a.p.max_pages; j += blockDim.x) {
    const int id = from[j];
    to[j] = id;
    if (page_ok(a, id)) atomicAdd(&a.c.ref[id], 1);
  }
  if (threadIdx.x == 0) a.c.len[t] = a.c.len[s];
}

__device__ __forceinline__ void give_up(const CacheArgs& a, int b, int j0, int j1) {
  int32_t* row = a.c.table + static_cast<size_t>(b) * a.p.max_pages;
  for (int j = j0 + static_cast<int>(threadIdx.x); j < j1; j += static_cast<int>(blockDim.x)) {
    const int id = row[j];
    if (page_ok(a, id)) atomicSub(&a.c.ref[id], 1);
    row[j] = -1;
  }
}

// one block per sequence of the cache; the list says which are emptied
__global__ void __launch_bounds__(128) free_kernel(const CacheArgs a, const int32_t* seq, int n) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int b = blockIdx.x;
  bool named = false, bad = false;
  for (int j = threadIdx.x; j < n; j += blockDim.x) {
    named = named || seq[j] == b;
    bad = bad || seq[j] < 0 || seq[j] >= a.p.B;
  }
  named = __syncthreads_or(named);
  bad = __syncthreads_or(bad);
  if (bad && b == 0 && threadIdx.x == 0) raise_status(a.stats, SPARSEPR_ERR_INVALID_ARG);
  if (!named) return;
  give_up(a, b, 0, a.p.max_pages);
  if (threadIdx.x == 0) a.c.len[b] = 0;
}

__global__ void __launch_bounds__(128) evict_kernel(const CacheArgs a, sparsepr_visibility see) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int b = blockIdx.x;
  const long long len = a.c.len[b], F = see.frame, page = a.p.page;
  const long long room = a.p.max_pages * page;
  if (len < 0 || len > room) {
    if (threadIdx.x == 0) raise_status(a.stats, SPARSEPR_ERR_INVALID_ARG);
    return;
  }
  const long long lo = (len / F - see.window + 1) * F;  // first key of the window at position len
  const long long s = see.sinks * F;
  const long long j0 = (min(s, room) + page - 1) / page, j1 = lo > 0 ? min(lo, len) / page : 0;
  give_up(a, b, static_cast<int>(j0), static_cast<int>(j1));
}

// Plan of the packing: counts[0] moves, pages[i] -> targets[i], remap[pages[i]] = i. One block: the plan is a
// scan over the pool's counts, 4,096 pages a round.
__global__ void __launch_bounds__(kPlanThreads)
    compact_plan_kernel(const CacheArgs a, int32_t* n_used) {
  __shared__ PlanScan<int> scan;
  __shared__ PlanScan<long long> scan64;
  int turn = 0, turn64 = 0;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int n_pages = a.p.n_pages, tid = threadIdx.x;
  int mine = 0;
#pragma unroll 4
  for (int id = tid; id < n_pages; id += kPlanThreads) mine += a.c.ref[id] > 0;
  int used;
  block_scan(mine, scan, turn, &used);
  int holes = 0, moves = 0;
  int r[kPerThread];
  load_refs(a.c.ref, n_pages, 0, r);
  for (long long base = 0; base < n_pages; base += kRound) {
    int next[kPerThread];
    const bool more = base + kRound < n_pages;
    if (more) load_refs(a.c.ref, n_pages, static_cast<int>(base + kRound), next);
    // both counts in one scan, 32 bits each
    long long count = 0, all;
#pragma unroll
    for (int e = 0; e < kPerThread; ++e) {
      const int id = static_cast<int>(base) + tid * kPerThread + e;
      if (r[e] == 0 && id < used) count += 1;
      if (r[e] > 0 && id >= used) count += 1ll << 32;
    }
    const long long at = block_scan(count, scan64, turn64, &all);
    int hole = holes + static_cast<int>(at & 0xffffffffll), move = moves + static_cast<int>(at >> 32);
#pragma unroll
    for (int e = 0; e < kPerThread; ++e) {
      const int id = static_cast<int>(base) + tid * kPerThread + e;
      if (r[e] == 0 && id < used) a.targets[hole++] = id;
      if (r[e] > 0 && id >= used) a.pages[move++] = id;
    }
    holes += static_cast<int>(all & 0xffffffffll);
    moves += static_cast<int>(all >> 32);
    if (more)
#pragma unroll
      for (int e = 0; e < kPerThread; ++e) r[e] = next[e];
  }
  __syncthreads();
  for (int i = tid; i < moves; i += kPlanThreads) a.remap[a.pages[i]] = i;
  if (tid == 0) {
    a.counts[0] = moves;
    a.counts[1] = used;
    *n_used = used;
  }
}

// Bound by memory: 1,176 pages of 196 KB in 76 us (5.9 TB/s read and written).
__global__ void __launch_bounds__(kCopyThreads) compact_move_kernel(const CacheArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the plan
  const int moves = a.counts[0], used = a.counts[1];
  const long long entries = static_cast<long long>(a.p.B) * a.p.max_pages;
  for (long long i = static_cast<long long>(blockIdx.x) * kCopyThreads + threadIdx.x; i < entries;
       i += static_cast<long long>(gridDim.x) * kCopyThreads) {
    const int id = a.c.table[i];
    // (an entry whose page has no count is none of the moves, and remap holds nothing for it)
    if (id >= used && id < a.p.n_pages) {
      const int move = a.remap[id];
      if (move >= 0 && move < moves && a.pages[move] == id) a.c.table[i] = a.targets[move];
    }
  }
  const int pieces = a.p.Hkv * (a.p.page * a.p.d / 16);
  const int parts = (pieces + kCopyPieces - 1) / kCopyPieces;
  for (long long w = blockIdx.x; w < 2ll * moves * parts; w += gridDim.x) {
    const int part = static_cast<int>(w % parts), kv = static_cast<int>(w / parts) & 1;
    const int i = static_cast<int>(w / (2 * parts));
    const int src = a.pages[i], dst = a.targets[i];
    copy_pieces(a, kv ? a.c.v8 : a.c.k8, src, dst, part * kCopyPieces);
    if (part == 0 && kv == 0) {
      copy_scales(a, src, dst);
      if (threadIdx.x == 0) {
        a.c.ref[dst] = a.c.ref[src];
        a.c.ref[src] = 0;
      }
    }
  }
}

// Exponent k of the smallest power of two with amax <= 448 * 2^k, k >= -110:
// amax = m 2^e with m in [0.5, 1) and 448 = 0.875 2^9, so k = e - 9, one more
// when m > 0.875. All of it is read off the bits of amax, with no rounding.
__device__ __forceinline__ int scale_exponent(float amax) {
  const uint32_t u = __float_as_uint(amax);
  const int e = static_cast<int>(u >> 23) - 126;
  const int k = e - 9 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  return u < 0x800000u ? kMinScaleExp : max(k, kMinScaleExp);
}
__device__ __forceinline__ float exp2_int(int k) { return __uint_as_float((k + 127) << 23); }

template <typename T>
__device__ __forceinline__ void load16(const T* p, float (&x)[16]) {
  constexpr int kVec = 16 / sizeof(T);
#pragma unroll
  for (int i = 0; i < 16 / kVec; ++i) {
    const uint4 u = reinterpret_cast<const uint4*>(p)[i];
    const T* e = reinterpret_cast<const T*>(&u);
#pragma unroll
    for (int j = 0; j < kVec; ++j) x[i * kVec + j] = load_f32(e + j);
  }
}

constexpr int kAppendThreads = 128;

// One block per (sequence, head), page that the new tokens reach, and K or V, since
// page and head share a scale. The new tokens of a page and head are contiguous in
// the input and in the page: first their largest magnitude, then, with the values
// still in the first-level cache (32 KB at most), their rounding. Bound by latency at
// the sizes of a step: one token of 8 sequences 2.5 us, a frame of 1,560 tokens and
// 12 heads (14.4 MB) 5.0 us (a sixteenth of a replayed graph of 16 such calls; called one by
// one from Python either takes 12 us, which is the host's time).
template <typename T>
__global__ void __launch_bounds__(kAppendThreads)
    append_kernel(const CacheArgs a, const void* k, const void* v, int T_rows,
                  const int32_t* start_p, const int32_t* n_new) {
  __shared__ float red[kAppendThreads / 32];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int bh = blockIdx.x, b = bh / a.p.Hkv, h = bh % a.p.Hkv;
  const int page = a.p.page, d = a.p.d;
  const bool first = h == 0 && blockIdx.y == 0 && blockIdx.z == 0 && threadIdx.x == 0;
  const int start = start_p[b];
  if (start < 0) return;
  const int n = clamp_count(n_new, b, T_rows, T_rows, a.stats, first);
  const long long room = static_cast<long long>(a.p.max_pages) * page;
  const long long col = start / page + static_cast<long long>(blockIdx.y);
  long long end = static_cast<long long>(start) + n;
  if (end > room) {
    if (first) raise_status(a.stats, SPARSEPR_ERR_INVALID_ARG);
    end = room;
  }
  if (start >= end || col * page >= end) return;  // nothing for this sequence, or not here
  const int id = a.c.table[static_cast<size_t>(b) * a.p.max_pages + col];
  if (!page_ok(a, id) || a.c.ref[id] != 1) {  // no page, or one that other sequences share
    if (threadIdx.x == 0) raise_status(a.stats, SPARSEPR_ERR_INVALID_ARG);
    return;
  }
  const int lo = static_cast<int>(max(static_cast<long long>(start), col * page));
  const int hi = static_cast<int>(min(end, (col + 1) * page));
  const int held = lo - static_cast<int>(col) * page;  // earlier tokens of this page
  const int count = (hi - lo) * d;
  const bool is_v = blockIdx.z == 1;
  const T* src = static_cast<const T*>(is_v ? v : k) +
                 (static_cast<size_t>(bh) * T_rows + (lo - start)) * d;
  uint8_t* page8 = static_cast<uint8_t*>(is_v ? a.c.v8 : a.c.k8) +
                   (static_cast<size_t>(id) * a.p.Hkv + h) * page * d;
  float* scale = (is_v ? a.c.v_scale : a.c.k_scale) + static_cast<size_t>(id) * a.p.Hkv + h;
  const float was = held ? *scale : 0.f;
  float amax = 0.f;
  for (int i = threadIdx.x * 16; i < count; i += kAppendThreads * 16) {
    float x[16];
    load16(src + i, x);
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const float m = fabsf(x[j]);
      if (m < INFINITY) amax = fmaxf(amax, m);
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = amax;
  __syncthreads();
  for (int w = 0; w < kAppendThreads / 32; ++w) amax = fmaxf(amax, red[w]);
  const float need = exp2_int(scale_exponent(amax));
  const float now = fmaxf(was, need);
  const float inv = 1.f / now;  // exact: a power of two
  for (int i = threadIdx.x * 16; i < count; i += kAppendThreads * 16) {
    float x[16];
    load16(src + i, x);
    *reinterpret_cast<uint4*>(page8 + held * d + i) = to_e4m3_16(x, inv);
  }
  if (now != was) {
    if (held) {
      const float ratio = was * inv;  // exact
      for (int i = threadIdx.x * 16; i < held * d; i += kAppendThreads * 16) {
        float x[16];
        from_e4m3_16(*reinterpret_cast<const uint4*>(page8 + i), x);
        *reinterpret_cast<uint4*>(page8 + i) = to_e4m3_16(x, ratio);
      }
    }
    if (threadIdx.x == 0) *scale = now;
  }
}

}  // namespace

namespace {
// A kernel that may be put in place beside the tail of what came before on the stream
// (programmatic dependent launch). Each begins with griddepcontrol.wait, which waits
// for all of that. (Appending a token 3.1 to 2.6 us, packing 95.0 to 91.1 us.)
template <typename... P>
cudaError_t launch_dependent(void (*kernel)(P...), dim3 grid, int threads, cudaStream_t st, P... p) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p...);
}
}  // namespace

cudaError_t launch_cache_reserve(const CacheArgs& a, const int32_t* n_new, int32_t* start,
                                 cudaStream_t st) {
  const cudaError_t e = launch_dependent(reserve_kernel, dim3(1), kPlanThreads, st, a, n_new, start);
  const int pieces = a.p.Hkv * (a.p.page * a.p.d / 16);
  const dim3 grid((pieces + kCopyPieces - 1) / kCopyPieces, a.p.B, 2);
  return e != cudaSuccess ? e : launch_dependent(copy_last_pages_kernel, grid, kCopyThreads, st, a);
}

cudaError_t launch_cache_append(const CacheArgs& a, const void* k, const void* v, bool bf16, int T,
                                const int32_t* start, const int32_t* n_new, cudaStream_t st) {
  const unsigned reach = (static_cast<unsigned>(T) + 2 * a.p.page - 2) / a.p.page;
  const dim3 grid(a.p.B * a.p.Hkv, reach, 2);
  return launch_dependent(bf16 ? append_kernel<__nv_bfloat16> : append_kernel<float>, grid,
                          kAppendThreads, st, a, k, v, T, start, n_new);
}

cudaError_t launch_cache_fork(const CacheArgs& a, const int32_t* src, const int32_t* dst, int n,
                              cudaStream_t st) {
  return launch_dependent(fork_kernel, dim3(n), 128, st, a, src, dst, n);
}

cudaError_t launch_cache_free(const CacheArgs& a, const int32_t* seq, int n, cudaStream_t st) {
  return launch_dependent(free_kernel, dim3(a.p.B), 128, st, a, seq, n);
}

cudaError_t launch_cache_evict(const CacheArgs& a, const sparsepr_visibility& see,
                               cudaStream_t st) {
  return launch_dependent(evict_kernel, dim3(a.p.B), 128, st, a, see);
}

cudaError_t launch_cache_compact(const CacheArgs& a, int32_t* n_used, cudaStream_t st) {
  const cudaError_t e = launch_dependent(compact_plan_kernel, dim3(1), kPlanThreads, st, a, n_used);
  return e != cudaSuccess ? e
                          : launch_dependent(compact_move_kernel, dim3(a.sm_count * 8), kCopyThreads, st, a);
}

}  // namespace spr
