// Attention over the paged 8-bit cache.
//
// A key stands for k8 * ks, a value for v8 * vs, with one power-of-two scale for
// each page and head, so for query row i (x in log2 units)
//   x_ij = (scale log2(e) ks_j) q_i . k8_j,
//   out_i = sum_j 2^(x_ij + log2 vs_j - M_i) v8_j * 2^(M_i - m_i) / l_i,
//   l_i = sum_j 2^(x_ij - m_i),
// m_i = max_j x_ij, M_i = max_j (x_ij + log2 vs_j). With M as the reference of the
// second product its weights are at most 1 whatever the scales are, so they
// fit fp16 (11 bits), and so do all e4m3 values, exactly: both products are
// fp16 MMAs with fp32 sums.
//
// Two kernels. Few query rows per key head (one token, a few speculated
// ones): the cache is read once and the call is bound by that; see
// cache_decode_kernel. Many rows (a whole new frame): the pages are widened to bf16 rows
// (exact) and the windowed attention kernel runs over them.
#include "common.cuh"
#include "e4m3.cuh"
#include "internal.h"
#include "visible.cuh"

namespace spr {
namespace {

constexpr int kTile = 64;            // keys of a tile, at multiples of 64 in the sequence
constexpr int kWarps = 8;            // consumer warps, each takes every 8th tile of the block
constexpr int kConsumers = kWarps * 32;
constexpr int kDecodeThreads = kConsumers + 32;  // and a producer warp
constexpr int kRows = 16;            // query rows of a block: the M of the MMA
constexpr int kDecodeBlocks = 148;   // one per multiprocessor
constexpr int kMinTiles = 4;         // tiles per block at least (they go to different warps)

template <int HD>
struct DecodeSmem {
  static constexpr int kTileBytes = kTile * HD;            // keys or values of a tile
  static constexpr int kStageBytes = 2 * kTileBytes;
  static constexpr int kStages = HD == 128 ? 8 : 16;       // 128 KB in flight
  static constexpr int stage_off = 0;
  static constexpr int merge_off = kStages * kStageBytes;  // [8 warps][HD / 2][32] fp32
  static constexpr int merge_bytes = kWarps * (HD / 2) * 32 * 4;
  static constexpr int pre_off = merge_off + merge_bytes;  // [1025] tiles before each sequence
  static constexpr int misc_off = pre_off + 1032 * 8;
  static constexpr int misc_bytes = 8192;
  static constexpr int bytes = misc_off + misc_bytes + 1024;
};

struct DecodeMisc {
  uint64_t full[16], empty[16];
  float k_scale[16][4], v_log2[16][4];  // per stage and page of the tile; k_scale < 0: no page
  float m[kWarps][kRows], M[kWarps][kRows], l[kWarps][kRows];
  int seen[kWarps][kRows];
  long long warp_sums[16];
  uint32_t flags;
  int abort;
  float q[128];
};
static_assert(sizeof(DecodeMisc) + sizeof(LiteralScratch<kConsumers>) + 64 <= 8192, "misc");

struct DecodeMaps {
  CUtensorMap k, v;  // [n_pages, Hkv * page, HD] bytes, boxes of min(page, 64) rows
};

struct DecodeParams {
  CacheAttnArgs a;
  int group;       // query heads per key head
  int R;           // query rows per key head: group * Nq, contiguous in q
  int row_tiles;   // ceil(R / 16)
  int units_seq;   // Hkv * row_tiles
  int sub_rows;    // min(page, 64): rows of one copy
  int* pre;        // [B + 1] in the workspace: tiles before each sequence (for the combine)
  float* opart;    // [B * units_seq + blocks, 16, HD]
  float* lpart;    // [B * units_seq + blocks, 16]
};

// Tiles that the queries of a sequence need: 0..TA-1, then from TB on.
struct SeqTiles {
  int L, n;        // keys, queries
  int SA, LB, HB;  // keys that some query sees: [0, SA) and [LB, HB)
  int TA, TB, T;
  __device__ int start(int t) const { return (t < TA ? t : TB + (t - TA)) * kTile; }
  // index of the tile that holds a visible key
  __device__ int tile_of(int j) const {
    const int x = j / kTile;
    return x < TA ? x : TA + (x - TB);
  }
};

__device__ __forceinline__ SeqTiles seq_tiles(const CacheAttnArgs& a, int b, bool report) {
  const CacheArgs& c = a.cache;
  SeqTiles s;
  s.n = clamp_count(a.n_q, b, a.Nq, a.Nq, c.stats, report);
  s.L = clamp_count(c.c.len, b, c.p.max_pages * c.p.page, 0, c.stats, report);
  s.SA = s.LB = s.HB = 0;
  if (s.n > 0) {
    const long long p0 = static_cast<long long>(s.L) - s.n;
    const Range first = visible_range(a.see, max(p0, 0ll), s.L);
    const Range last = visible_range(a.see, static_cast<long long>(s.L) - 1, s.L);
    s.SA = last.s;
    s.LB = first.lo;
    s.HB = max(last.hi, s.LB);
  }
  s.TA = (s.SA + kTile - 1) / kTile;
  s.TB = max(s.LB / kTile, s.TA);
  s.T = s.TA + max((s.HB + kTile - 1) / kTile - s.TB, 0);
  return s;
}

// Keys and values of one sequence and head through its table row, limited to
// the tiles [t0, t1) of the sequence.
template <int D>
struct PagedKV {
  const CacheArgs& a;
  const int32_t* row;
  int h;
  SeqTiles s;
  int t0, t1;
  __device__ bool ok(int j) const {
    const int t = s.tile_of(j);
    if (t < t0 || t >= t1) return false;
    const int id = row[j / a.p.page];
    return id >= 0 && id < a.p.n_pages;
  }
  __device__ size_t slot(int j) const {
    return static_cast<size_t>(row[j / a.p.page]) * a.p.Hkv + h;
  }
  __device__ float dot(int j, const float* q) const {
    const uint8_t* k = static_cast<const uint8_t*>(a.c.k8) +
                       (slot(j) * a.p.page + j % a.p.page) * D;
    float s_ = 0.f;
    for (int c = 0; c < D; ++c) s_ = fmaf(q[c], from_e4m3(k[c]), s_);
    return s_ * a.c.k_scale[slot(j)];
  }
  __device__ float v(int j, int c) const {
    const uint8_t* x = static_cast<const uint8_t*>(a.c.v8) +
                       (slot(j) * a.p.page + j % a.p.page) * D;
    return from_e4m3(x[c]) * a.c.v_scale[slot(j)];
  }
};

__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, uint64_t* bar,
                                            int32_t x, int32_t y, int32_t z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z)
      : "memory");
}

// D (16x8, fp32) += A (16x16, fp16) B (16x8, fp16)
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// log2 of a scale; exact for powers of two
__device__ __forceinline__ float log2_of_scale(float s) {
  const uint32_t u = __float_as_uint(s);
  if ((u & 0x7fffffu) == 0 && u >= 0x800000u && u < 0x7f800000u)
    return static_cast<float>(static_cast<int>(u >> 23) - 127);
  return log2f(s);
}

// The block that holds flattened tile x of `total` when block c takes
// [c total / blocks, (c + 1) total / blocks).
__device__ __forceinline__ int owner(long long x, long long total, int blocks) {
  return static_cast<int>(((x + 1) * blocks - 1) / total);
}
__device__ __forceinline__ int blocks_for(long long total) {
  const long long want = (total + kMinTiles - 1) / kMinTiles;
  return static_cast<int>(want < kDecodeBlocks ? (want > 0 ? want : 1) : kDecodeBlocks);
}

struct ConsumerSync {
  __device__ void operator()() const { named_barrier_sync(1, kConsumers); }
};

// Few query rows. The tiles of all (sequence, key head, 16 query rows) units form
// one line that is cut evenly over the blocks, whatever the lengths: a block
// takes a run of it, which may end one unit, hold several and begin another.
// A producer warp looks pages up and streams keys and values by TMA, 128 KB in
// flight; consumer warp w takes every 8th tile and keeps its own running
// maxima, sum and 16 x HD accumulator (in registers, flat over the tile's
// pages); at the end of a unit's run the eight are merged, and runs that do not
// hold the whole unit leave a partial result for cache_combine_kernel.
//
// Fragments of mma m16n8k16 (g = lane / 4, t = lane % 4). The order of d
// within a product and the order of the output columns are free, so a lane takes
// 16 contiguous bytes: of key g (8 keys per product), d = 16 c .. 16 c + 15 at
// chunk c = 2 t + u (HD = 128; c = t for 64), 4 bytes for each step of 16; and of the four
// values 2t, 2t+1, 2t+8, 2t+9 the columns (HD / 8) g .. The tile is swizzled by
// TMA, so that the lanes of a quarter warp meet different banks.
template <int HD, typename T>
__global__ void __launch_bounds__(kDecodeThreads, 1)
    cache_decode_kernel(const __grid_constant__ DecodeMaps maps, const DecodeParams p) {
  using L = DecodeSmem<HD>;
  constexpr int kU = HD / 64;        // 16-byte pieces of a key per lane
  constexpr int kSteps = HD / 16;    // steps of the first product
  constexpr int kNd = HD / 8;        // column tiles of the second product
  const CacheAttnArgs& a = p.a;
  const CacheArgs& c = a.cache;
  const int B = c.p.B, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  float* merge = reinterpret_cast<float*>(smem + L::merge_off);
  long long* pre = reinterpret_cast<long long*>(smem + L::pre_off);
  DecodeMisc& ms = *reinterpret_cast<DecodeMisc*>(smem + L::misc_off);
  LiteralScratch<kConsumers>& scratch = *reinterpret_cast<LiteralScratch<kConsumers>*>(
      smem + L::misc_off + (sizeof(DecodeMisc) + 63) / 64 * 64);

  // tiles before each sequence: a thread counts four sequences, the block scans
  {
    long long mine[4], sum = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int b = tid * 4 + e;
      mine[e] = b < B ? seq_tiles(a, b, blockIdx.x == 0).T : 0;
      sum += mine[e];
    }
    long long x = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) ms.warp_sums[warp] = x;
    if (tid == 0) {
      for (int s = 0; s < L::kStages; ++s) {
        mbar_init(&ms.full[s], 1);
        mbar_init(&ms.empty[s], 1);
      }
      ms.abort = 0;
      ms.flags = 0;
      fence_barrier_init();
    }
    __syncthreads();
    long long before = x - sum;
    for (int w = 0; w < warp; ++w) before += ms.warp_sums[w];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int b = tid * 4 + e;
      if (b <= B) {
        pre[b] = before;
        if (blockIdx.x == 0) p.pre[b] = static_cast<int>(before);
      }
      before += mine[e];
    }
    __syncthreads();
  }
  const long long total = pre[B] * p.units_seq;
  const int blocks = blocks_for(total);
  if (total == 0 || static_cast<int>(blockIdx.x) >= blocks) return;
  const long long begin = total * blockIdx.x / blocks, end = total * (blockIdx.x + 1) / blocks;
  volatile int* abort = &ms.abort;

  // the run of one unit inside [begin, end)
  struct Run {
    int b, x, t0, t1;  // sequence, unit of the sequence, tiles
  };
  auto run_at = [&](long long pos) {
    int lo = 0, hi = B;  // pre[lo] * units <= pos < pre[hi] * units
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (pre[mid] * p.units_seq <= pos) lo = mid;
      else hi = mid;
    }
    const long long tiles = pre[lo + 1] - pre[lo], off = pos - pre[lo] * p.units_seq;
    Run r;
    r.b = lo;
    r.x = static_cast<int>(off / tiles);
    r.t0 = static_cast<int>(off % tiles);
    r.t1 = static_cast<int>(min(tiles, r.t0 + (end - pos)));
    return r;
  };

  if (warp == kWarps) {
    // ------------------------------ producer ---------------------------------
    const int sub = p.sub_rows, spp = kTile / sub;  // copies of a tile (for keys, for values)
    const int page = c.p.page;
    int issued = 0;  // tiles of this block so far
    bool ok = true;
    for (long long pos = begin; pos < end && ok;) {
      const Run r = run_at(pos);
      const SeqTiles s = seq_tiles(a, r.b, false);
      const int h = r.x / p.row_tiles;
      const int32_t* row = c.c.table + static_cast<size_t>(r.b) * c.p.max_pages;
      // 32 pages (or halves of one) are looked up at a time
      const int per_batch = 32 / spp;
      for (int t = r.t0; t < r.t1 && ok; t += per_batch) {
        const int mine = t + lane / spp;  // this lane's tile
        int id = -1, key0 = 0;
        float ks = -1.f, lv = 0.f;
        if (mine < r.t1) {
          key0 = s.start(mine) + (lane % spp) * sub;
          // keys of this copy that some query sees
          const bool wanted = key0 < s.SA || (key0 < s.HB && key0 + sub > s.LB);
          if (wanted) {
            id = row[key0 / page];
            if (id < 0 || id >= c.p.n_pages) {
              raise_status(c.stats, SPARSEPR_ERR_INVALID_ARG);
              id = -1;
            } else {
              const size_t slot = static_cast<size_t>(id) * c.p.Hkv + h;
              ks = fabsf(c.c.k_scale[slot]);
              lv = log2_of_scale(c.c.v_scale[slot]);
            }
          }
        }
        const unsigned have = __ballot_sync(0xffffffffu, id >= 0);
        const int here = min(per_batch, r.t1 - t);
        for (int e = 0; e < here && ok; ++e, ++issued) {
          const int st = issued % L::kStages, round = issued / L::kStages;
          if (lane == 0 && round > 0) ok = mbar_wait(&ms.empty[st], (round + 1) & 1, abort);
          ok = __shfl_sync(0xffffffffu, ok, 0);
          if (!ok) break;
          const bool part = lane / spp == e;  // lanes of this tile
          if (part) {
            ms.k_scale[st][lane % spp] = ks;
            ms.v_log2[st][lane % spp] = lv;
          }
          __syncwarp();
          const unsigned tile_lanes = ((spp == 32 ? 0u : (1u << spp)) - 1u) << (e * spp);
          if (lane == 0)
            mbar_arrive_expect_tx(&ms.full[st], __popc(have & tile_lanes) * 2 * sub * HD);
          __syncwarp();
          if (part && id >= 0) {
            uint8_t* dst = smem + L::stage_off + st * L::kStageBytes + (lane % spp) * sub * HD;
            const int y = h * page + key0 % page;
            tma_load_3d(dst, &maps.k, &ms.full[st], 0, y, id);
            tma_load_3d(dst + L::kTileBytes, &maps.v, &ms.full[st], 0, y, id);
          }
        }
      }
      pos += r.t1 - r.t0;
    }
    // let the copies in flight land before the block goes on
    if (lane == 0) {
      volatile int never = 0;
      for (int n = max(0, issued - L::kStages); n < issued; ++n)
        mbar_wait(&ms.full[n % L::kStages], (n / L::kStages) & 1, &never);
    }
  } else {
    // ------------------------------ consumers --------------------------------
    const int g = lane >> 2, t4 = lane & 3;
    const ConsumerSync sync;
    long long first_tile = 0;  // tiles of this block before the run
    for (long long pos = begin; pos < end;) {
      const Run r = run_at(pos);
      const SeqTiles s = seq_tiles(a, r.b, false);
      const int h = r.x / p.row_tiles, row0 = (r.x % p.row_tiles) * kRows;
      const size_t q_base = (static_cast<size_t>(r.b) * a.Hq + static_cast<size_t>(h) * p.group) *
                                a.Nq + row0;  // of q, out, lse: rows are contiguous
      // the two rows of this lane: their visible keys, their queries in fp16
      // scaled by a power of two to at most 2 in magnitude (exact for bf16
      // unless 2^14 below the row's largest)
      Range rg[2];
      bool live[2];
      float qf[2];  // logits: acc * qf * k_scale
      uint32_t qa[kSteps][4];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int rr = g + 8 * e, i = (row0 + rr) % a.Nq;
        live[e] = row0 + rr < p.R && i < s.n;
        rg[e] = Range{0, 0, 0};
        if (live[e]) rg[e] = visible_range(a.see, static_cast<long long>(s.L) - s.n + i, s.L);
        live[e] = live[e] && (rg[e].s > 0 || rg[e].hi > rg[e].lo);
        float x[kU][16];
        float top = 0.f;
#pragma unroll
        for (int u = 0; u < kU; ++u) {
          if (live[e]) {
            const T* src = static_cast<const T*>(a.q) + (q_base + rr) * HD + 16 * (kU * t4 + u);
            constexpr int kVec = 16 / sizeof(T);
#pragma unroll
            for (int v = 0; v < 16 / kVec; ++v) {
              const uint4 w = reinterpret_cast<const uint4*>(src)[v];
              const T* el = reinterpret_cast<const T*>(&w);
#pragma unroll
              for (int k = 0; k < kVec; ++k) x[u][v * kVec + k] = load_f32(el + k);
            }
          } else {
#pragma unroll
            for (int k = 0; k < 16; ++k) x[u][k] = 0.f;
          }
#pragma unroll
          for (int k = 0; k < 16; ++k) top = fmaxf(top, fabsf(x[u][k]));
        }
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        // 2^-exponent(top), within the normal range both ways
        const int ex = top > 0.f ? min(max(static_cast<int>(__float_as_uint(top) >> 23) - 127, -100), 100) : 0;
        const float down = __uint_as_float((127 - ex) << 23);
        qf[e] = a.sc * __uint_as_float((127 + ex) << 23);
#pragma unroll
        for (int u = 0; u < kU; ++u)
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            qa[4 * u + w][e] = pack_f16x2(x[u][4 * w] * down, x[u][4 * w + 1] * down);
            qa[4 * u + w][2 + e] = pack_f16x2(x[u][4 * w + 2] * down, x[u][4 * w + 3] * down);
          }
      }
      float m[2] = {-INFINITY, -INFINITY}, M[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
      bool seen[2] = {false, false};
      float o[kNd][4];
#pragma unroll
      for (int nd = 0; nd < kNd; ++nd)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[nd][e] = 0.f;

      const int n_tiles = r.t1 - r.t0;
      for (int e0 = (warp + kWarps - static_cast<int>(first_tile % kWarps)) % kWarps; e0 < n_tiles;
           e0 += kWarps) {
        const long long nth = first_tile + e0;
        const int st = static_cast<int>(nth % L::kStages);
        const bool got = mbar_wait(&ms.full[st], static_cast<uint32_t>(nth / L::kStages) & 1u, abort);
        if (!__all_sync(0xffffffffu, got)) continue;  // aborted: the status word says so
        const uint8_t* ks8 = smem + L::stage_off + st * L::kStageBytes;
        const uint8_t* vs8 = ks8 + L::kTileBytes;
        const int k0 = s.start(r.t0 + e0);
        // ---- x = q . k: 8 groups of 8 keys ----
        float acc[8][4];
#pragma unroll
        for (int kn = 0; kn < 8; ++kn) {
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[kn][e] = 0.f;
          const int key = kn * 8 + g;
          uint4 kw[kU];
#pragma unroll
          for (int u = 0; u < kU; ++u) {
            const int chunk = kU == 2 ? ((2 * t4 + u) ^ (key & 7)) : (t4 ^ ((key >> 1) & 3));
            kw[u] = *reinterpret_cast<const uint4*>(ks8 + key * HD + chunk * 16);
          }
#pragma unroll
          for (int u = 0; u < kU; ++u) {
            const uint32_t w[4] = {kw[u].x, kw[u].y, kw[u].z, kw[u].w};
#pragma unroll
            for (int x = 0; x < 4; ++x)
              mma16816(acc[kn], qa[4 * u + x], e4m3x2_to_f16x2(w[x]), e4m3x2_to_f16x2(w[x] >> 16));
          }
        }
        // ---- logits, masks, maxima ----
        bool whole = true, pages = true;
#pragma unroll
        for (int e = 0; e < 2; ++e)
          whole = whole && (!live[e] || (k0 + kTile <= rg[e].s) ||
                            (rg[e].lo <= k0 && k0 + kTile <= rg[e].hi) ||
                            (rg[e].s == rg[e].lo && k0 + kTile <= rg[e].hi));
        const int spp = kTile / p.sub_rows;
        for (int x = 0; x < spp; ++x) pages = pages && !(ms.k_scale[st][x] < 0.f);
        const bool plain = __all_sync(0xffffffffu, whole) && pages;
        float tm[2] = {-INFINITY, -INFINITY}, tM[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int kn = 0; kn < 8; ++kn) {
          const int sp = (kn * 8) / p.sub_rows;
          const float ks = ms.k_scale[st][sp], lv = ms.v_log2[st][sp];
          const float f[2] = {qf[0] * ks, qf[1] * ks};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float x = acc[kn][e] * f[e >> 1];
            if (!plain) {
              const int key = k0 + kn * 8 + 2 * t4 + (e & 1);
              const Range& rr = rg[e >> 1];
              if (ks < 0.f || !(key < rr.s || (key >= rr.lo && key < rr.hi))) x = -INFINITY;
              else seen[e >> 1] = true;
            }
            acc[kn][e] = x;
            tm[e >> 1] = fmaxf(tm[e >> 1], x);
            tM[e >> 1] = fmaxf(tM[e >> 1], x + lv);
          }
        }
        if (plain) seen[0] = seen[1] = true;
        float nm[2], nM[2];  // references, 0 where nothing has been seen
        bool moved = false;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          tm[e] = fmaxf(tm[e], __shfl_xor_sync(0xffffffffu, tm[e], 1));
          tm[e] = fmaxf(tm[e], __shfl_xor_sync(0xffffffffu, tm[e], 2));
          tM[e] = fmaxf(tM[e], __shfl_xor_sync(0xffffffffu, tM[e], 1));
          tM[e] = fmaxf(tM[e], __shfl_xor_sync(0xffffffffu, tM[e], 2));
          const float mn = fmaxf(m[e], tm[e]), Mn = fmaxf(M[e], tM[e]);
          l[e] *= m[e] == -INFINITY ? 0.f : exp2f(m[e] - mn);
          moved = moved || Mn != M[e];
          tM[e] = M[e] == -INFINITY ? 0.f : exp2f(M[e] - Mn);  // factor of the accumulator
          m[e] = mn;
          M[e] = Mn;
          nm[e] = mn == -INFINITY ? 0.f : mn;
          nM[e] = Mn == -INFINITY ? 0.f : Mn;
        }
        if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
          for (int nd = 0; nd < kNd; ++nd) {
            o[nd][0] *= tM[0];
            o[nd][1] *= tM[0];
            o[nd][2] *= tM[1];
            o[nd][3] *= tM[1];
          }
        }
        // ---- weights and the second product, 16 keys at a time ----
#pragma unroll
        for (int kk = 0; kk < kTile / 16; ++kk) {
          const float lv = ms.v_log2[st][(kk * 16) / p.sub_rows];
          const float sh[2] = {lv - nM[0], lv - nM[1]};
          uint32_t pa[4];
#pragma unroll
          for (int half = 0; half < 2; ++half)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float x0 = acc[2 * kk + half][2 * e], x1 = acc[2 * kk + half][2 * e + 1];
              l[e] += ex2_approx(x0 - nm[e]) + ex2_approx(x1 - nm[e]);
              pa[2 * half + e] = pack_f16x2(ex2_approx(x0 + sh[e]), ex2_approx(x1 + sh[e]));
            }
          uint32_t vw[4][kNd / 4];  // keys 2t, 2t+1, 2t+8, 2t+9: HD / 8 bytes of each
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int key = kk * 16 + 2 * t4 + (e & 1) + (e >> 1) * 8;
            if (HD == 128) {
              const uint4 v = *reinterpret_cast<const uint4*>(vs8 + key * HD + (g ^ (key & 7)) * 16);
              vw[e][0] = v.x;
              vw[e][1] = v.y;
              vw[e][kNd / 4 - 2] = v.z;
              vw[e][kNd / 4 - 1] = v.w;
            } else {
              const uint2 v = *reinterpret_cast<const uint2*>(
                  vs8 + key * HD + ((g >> 1) ^ ((key >> 1) & 3)) * 16 + (g & 1) * 8);
              vw[e][0] = v.x;
              vw[e][1] = v.y;
            }
            if (!plain) {
              // a value that no row sees may be anything, also NaN
              const int kx = k0 + key;
              if (ms.k_scale[st][(kk * 16) / p.sub_rows] < 0.f ||
                  !(kx < s.SA || (kx >= s.LB && kx < s.HB)))
#pragma unroll
                for (int w = 0; w < kNd / 4; ++w) vw[e][w] = 0u;
            }
          }
#pragma unroll
          for (int w = 0; w < kNd / 4; ++w) {
            const uint32_t a_lo = __byte_perm(vw[0][w], vw[1][w], 0x5140);
            const uint32_t a_hi = __byte_perm(vw[0][w], vw[1][w], 0x7362);
            const uint32_t b_lo = __byte_perm(vw[2][w], vw[3][w], 0x5140);
            const uint32_t b_hi = __byte_perm(vw[2][w], vw[3][w], 0x7362);
            mma16816(o[4 * w], pa, e4m3x2_to_f16x2(a_lo), e4m3x2_to_f16x2(b_lo));
            mma16816(o[4 * w + 1], pa, e4m3x2_to_f16x2(a_lo >> 16), e4m3x2_to_f16x2(b_lo >> 16));
            mma16816(o[4 * w + 2], pa, e4m3x2_to_f16x2(a_hi), e4m3x2_to_f16x2(b_hi));
            mma16816(o[4 * w + 3], pa, e4m3x2_to_f16x2(a_hi >> 16), e4m3x2_to_f16x2(b_hi >> 16));
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&ms.empty[st]);
      }
      // ---- merge of the warps ----
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        l[e] += __shfl_xor_sync(0xffffffffu, l[e], 1);
        l[e] += __shfl_xor_sync(0xffffffffu, l[e], 2);
        int sn = seen[e];
        sn |= __shfl_xor_sync(0xffffffffu, sn, 1);
        sn |= __shfl_xor_sync(0xffffffffu, sn, 2);
        if (t4 == 0) {
          ms.m[warp][g + 8 * e] = m[e];
          ms.M[warp][g + 8 * e] = M[e];
          ms.l[warp][g + 8 * e] = l[e];
          ms.seen[warp][g + 8 * e] = sn;
        }
      }
      sync();
      float gm[2], gM[2], gl[2];
      bool gs[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        gm[e] = gM[e] = -INFINITY;
        gs[e] = false;
        for (int w = 0; w < kWarps; ++w) {
          gm[e] = fmaxf(gm[e], ms.m[w][g + 8 * e]);
          gM[e] = fmaxf(gM[e], ms.M[w][g + 8 * e]);
          gs[e] = gs[e] || ms.seen[w][g + 8 * e];
        }
        gl[e] = 0.f;
        for (int w = 0; w < kWarps; ++w) {
          const float mw = ms.m[w][g + 8 * e], lw = ms.l[w][g + 8 * e];
          if (mw != -INFINITY) gl[e] += lw * exp2f(mw - gm[e]);
          else if (!(lw == 0.f)) gl[e] = lw;  // NaN
        }
      }
      {
        const float f[2] = {M[0] == -INFINITY ? 0.f : exp2f(M[0] - gM[0]),
                            M[1] == -INFINITY ? 0.f : exp2f(M[1] - gM[1])};
#pragma unroll
        for (int nd = 0; nd < kNd; ++nd)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            merge[(warp * (HD / 2) + nd * 4 + e) * 32 + lane] = o[nd][e] * f[e >> 1];
      }
      sync();
      // this warp sums column tiles kPer warp ..: columns (HD / 8) (2 t) + nd and (HD / 8) (2 t + 1) + nd
      constexpr int kPer = kNd / kWarps;  // 2 or 1
      const bool full_unit = n_tiles == s.T;
      const size_t slot = static_cast<size_t>(r.b) * p.units_seq + r.x + blockIdx.x;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int rr = g + 8 * e, i = (row0 + rr) % a.Nq;
        const bool valid = row0 + rr < p.R && i < s.n;
        const float inv = live[e] && gl[e] > 0.f ? exp2f(gM[e] - gm[e]) / gl[e] : 0.f;
        const float lse = live[e] && gl[e] > 0.f ? gm[e] + log2f(gl[e]) : -INFINITY;
        bool finite = true;
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
          const int nd = warp * kPer + k;
#pragma unroll
          for (int z = 0; z < 2; ++z) {
            float x = 0.f;
            for (int w = 0; w < kWarps; ++w)
              x += merge[(w * (HD / 2) + nd * 4 + 2 * e + z) * 32 + lane];
            x = live[e] ? x * inv : 0.f;
            finite = finite && fabsf(x) < INFINITY;
            const int col = (HD / 8) * (2 * t4 + z) + nd;
            if (full_unit) {
              if (valid) store_f32(static_cast<T*>(a.out) + (q_base + rr) * HD + col, x);
            } else {
              p.opart[(slot * kRows + rr) * HD + col] = x;
            }
          }
        }
        if (warp == 0 && t4 == 0) {
          if (!full_unit) p.lpart[slot * kRows + rr] = lse;
          else if (valid && a.lse) a.lse[q_base + rr] = lse * kLn2F;
        }
        if (live[e] && gs[e] && (!finite || !(gl[e] > 0.f) || !(gl[e] < INFINITY)))
          atomicOr(&ms.flags, 1u << rr);
      }
      sync();
      // Rows whose result is not finite are taken again by the definition (a value
      // or key with NaN that this row, or only another row, sees).
      uint32_t todo = ms.flags;
      while (todo) {
        const int rr = __ffs(todo) - 1, i = (row0 + rr) % a.Nq;
        todo &= todo - 1;
        const PagedKV<HD> kv = {c, c.c.table + static_cast<size_t>(r.b) * c.p.max_pages, h, s, r.t0,
                                r.t1};
        for (int x = tid; x < HD; x += kConsumers)
          ms.q[x] = load_f32(static_cast<const T*>(a.q) + (q_base + rr) * HD + x);
        sync();
        float lm, ll, lo;
        literal_row<kConsumers, HD>(
            kv, ms.q, visible_range(a.see, static_cast<long long>(s.L) - s.n + i, s.L), a.sc,
            scratch, sync, lm, ll, lo);
        const float inv = ll == 0.f ? 0.f : 1.f / ll;
        const float lse = ll == 0.f ? -INFINITY : lm + log2f(ll);
        if (tid < HD) {
          if (full_unit) store_f32(static_cast<T*>(a.out) + (q_base + rr) * HD + tid, lo * inv);
          else p.opart[(slot * kRows + rr) * HD + tid] = lo * inv;
        }
        if (tid == 0) {
          if (!full_unit) p.lpart[slot * kRows + rr] = lse;
          else if (a.lse) a.lse[q_base + rr] = lse * kLn2F;
        }
        sync();
      }
      if (tid == 0) ms.flags = 0;  // read by all before; set again after the next merge's barriers
      first_tile += n_tiles;
      pos += n_tiles;
    }
  }
  __syncthreads();
  if (*abort && tid == 0) raise_status(c.stats, SPARSEPR_ERR_TIMEOUT);
}

// Joins the partial results of units that more than one block worked on, in the
// order of the blocks, and writes the rows that see nothing. One block per
// (sequence, unit); thread = (row, 8 columns).
template <int HD, typename T>
__global__ void __launch_bounds__(kRows* HD / 8) cache_combine_kernel(const DecodeParams p) {
  const CacheAttnArgs& a = p.a;
  const int b = blockIdx.x / p.units_seq, x = blockIdx.x % p.units_seq;
  const long long before = p.pre[b], tiles = p.pre[b + 1] - before;
  const int h = x / p.row_tiles, row0 = (x % p.row_tiles) * kRows;
  const int rr = threadIdx.x / (HD / 8), col = (threadIdx.x % (HD / 8)) * 8;
  const int n = clamp_count(a.n_q, b, a.Nq, a.Nq, a.cache.stats, false);
  const bool valid = row0 + rr < p.R && (row0 + rr) % a.Nq < n;
  const size_t row = (static_cast<size_t>(b) * a.Hq + static_cast<size_t>(h) * p.group) * a.Nq +
                     row0 + rr;
  T* out = static_cast<T*>(a.out) + row * HD + col;
  float num[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  float lse = -INFINITY, inv = 0.f;
  if (tiles > 0) {
    const long long total = static_cast<long long>(p.pre[a.cache.p.B]) * p.units_seq;
    const int blocks = blocks_for(total);
    const long long at = before * p.units_seq + x * tiles;
    const int c0 = owner(at, total, blocks), c1 = owner(at + tiles - 1, total, blocks);
    if (c0 == c1) return;  // written whole
    float M = -INFINITY, den = 0.f;
    bool nan = false;
    for (int c = c0; c <= c1; ++c) {
      const float l = p.lpart[(static_cast<size_t>(blockIdx.x) + c) * kRows + rr];
      M = fmaxf(M, l);
      nan = nan || l != l;
    }
    for (int c = c0; c <= c1; ++c) {
      const size_t slot = (static_cast<size_t>(blockIdx.x) + c) * kRows + rr;
      const float l = p.lpart[slot];
      if (l == -INFINITY) continue;
      const float w = exp2f(l - M);
      den += w;
#pragma unroll
      for (int e = 0; e < 8; e += 4) {
        const float4 o = *reinterpret_cast<const float4*>(p.opart + slot * HD + col + e);
        num[e] = fmaf(w, o.x, num[e]);
        num[e + 1] = fmaf(w, o.y, num[e + 1]);
        num[e + 2] = fmaf(w, o.z, num[e + 2]);
        num[e + 3] = fmaf(w, o.w, num[e + 3]);
      }
    }
    if (den > 0.f || nan) {
      inv = 1.f / den;
      lse = nan ? den : M + log2f(den);
    }
  }
  if (!valid) return;
#pragma unroll
  for (int e = 0; e < 8; ++e) store_f32(out + e, num[e] * inv);
  if (a.lse && col == 0) a.lse[row] = lse * kLn2F;
}

// [n_pages, Hkv * page, HD] bytes, swizzled over the whole row
bool make_page_map(CUtensorMap* m, const void* base, const sparsepr_cache_params& p, int box_rows) {
  EncodeTiledFn enc = encode_tiled_fn();
  if (!enc) return false;
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(p.d), static_cast<cuuint64_t>(p.Hkv) * p.page,
                        static_cast<cuuint64_t>(p.n_pages)};
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(p.d),
                           static_cast<cuuint64_t>(p.Hkv) * p.page * p.d};
  cuuint32_t box[3] = {static_cast<cuuint32_t>(p.d), static_cast<cuuint32_t>(box_rows), 1};
  cuuint32_t es[3] = {1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(base), dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE,
             p.d == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int HD, typename T>
cudaError_t launch_decode(const DecodeParams& p, const DecodeMaps& maps, cudaStream_t st) {
  cudaError_t e = cudaFuncSetAttribute(cache_decode_kernel<HD, T>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       DecodeSmem<HD>::bytes);
  if (e != cudaSuccess) return e;
  cache_decode_kernel<HD, T><<<kDecodeBlocks, kDecodeThreads, DecodeSmem<HD>::bytes, st>>>(maps, p);
  cache_combine_kernel<HD, T><<<p.a.cache.p.B * p.units_seq, kRows * HD / 8, 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace

CacheAttnPlan cache_attn_plan(const sparsepr_cache_params& p, int Hq, int Nq) {
  CacheAttnPlan w = {};
  const int R = Hq / p.Hkv * Nq;
  w.row_tiles = (R + kRows - 1) / kRows;
  w.slots = static_cast<size_t>(p.B) * p.Hkv * w.row_tiles + kDecodeBlocks;
  w.slot_rows = kRows;
  return w;
}

cudaError_t launch_cache_attention(const CacheAttnArgs& a, cudaStream_t st) {
  if (a.Nq == 0) return cudaSuccess;
  const CacheAttnPlan w = cache_attn_plan(a.cache.p, a.Hq, a.Nq);
  DecodeParams p = {};
  p.a = a;
  p.group = a.Hq / a.cache.p.Hkv;
  p.R = p.group * a.Nq;
  p.row_tiles = w.row_tiles;
  p.units_seq = a.cache.p.Hkv * w.row_tiles;
  p.sub_rows = a.cache.p.page < kTile ? a.cache.p.page : kTile;
  p.pre = a.pre;
  p.opart = a.opart;
  p.lpart = a.lpart;
  DecodeMaps maps;
  if (!make_page_map(&maps.k, a.cache.c.k8, a.cache.p, p.sub_rows) ||
      !make_page_map(&maps.v, a.cache.c.v8, a.cache.p, p.sub_rows))
    return cudaErrorInvalidValue;
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  if (a.bf16)
    return a.cache.p.d == 128 ? launch_decode<128, __nv_bfloat16>(p, maps, st)
                              : launch_decode<64, __nv_bfloat16>(p, maps, st);
  return a.cache.p.d == 128 ? launch_decode<128, float>(p, maps, st)
                            : launch_decode<64, float>(p, maps, st);
}

}  // namespace spr
