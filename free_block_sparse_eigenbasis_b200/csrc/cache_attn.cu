// Attention over the paged 8-bit cache.
//
// A key stands for k8 * ks, a value for v8 * vs, with one power-of-two scale for
// each page and head, so for query row i (x in log2 units)
//   x_ij = (scale log2(e) ks_j) q_i . k8_j,
//   out_i = sum_j 2^(x_ij + log2 vs_j - M_i) v8_j * 2^(M_i - m_i) / l_i,
//   l_i = sum_j 2^(x_ij - m_i),
// m_i near max_j x_ij, M_i near max_j (x_ij + log2 vs_j). With M as the reference of the
// second product its weights are below 2^16 whatever the scales are, so they
// fit fp16, and so do all e4m3 values, exactly: both products are fp16 MMAs with fp32
// sums. fp16 holds 11 bits of a weight down to 2^-14 and nothing below 2^-25, and keys that
// far below the largest can still be all of the output, where the values of the largest are
// 0: what fp16 leaves of a tile with such weights is added by a product in tf32, which
// reaches down to 2^-126.
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

constexpr int kWarps = 6;            // 168 registers a thread
constexpr int kDecodeThreads = kWarps * 32;
constexpr int kMaxRows = 16;         // query rows of a block at most: 8 for each NT
constexpr int kDecodeBlocks = 296;   // two per multiprocessor: one streams while the other merges
constexpr int kMinTiles = kWarps;    // tiles per block at least (each goes to another warp)
// Blocks take whole units, or equal runs of tiles that may cut units, whichever is
// estimated shorter: a unit's run costs about 5 us beside its tiles, a tile 2 us of its warp, and
// the combine of cut units 4 us. (48 units of one tile: 49 us when 8 blocks took six tiles
// each, 17 us in 48 blocks; 12 units of 11 tiles: 14.5 us whole, 21.5 us cut; 8 units of
// 24 tiles: 20 us whole, 16.5 us cut.)
constexpr int kWholeTiles = 16;  // units that cannot be longer are never cut
__device__ __forceinline__ bool whole_is_shorter(int longest, long long tiles, long long units) {
  const float b = kDecodeBlocks, u = static_cast<float>(units), t = static_cast<float>(tiles);
  const float cut_blocks = fminf(b, fmaxf(1.f, t / kMinTiles));
  const float whole = ceilf(u / b) * (5.f + 2.f * ceilf(static_cast<float>(longest) / kWarps));
  const float cut = 5.f * (1.f + u / cut_blocks) + 2.f * ceilf(t / (cut_blocks * kWarps)) + 4.f;
  return whole <= cut;
}
// Query rows per key head beyond which pages are widened. In place against widened,
// 4 heads of 20,000 tokens, d = 128: 16 rows 33 and 39 us, 32 rows 34 and 39, 48 rows 49
// and 39; 64 (sequence, head) pairs of 4,000 tokens: 56 and 68, 71 and 70, 81 and 70.
constexpr int kWideRows = 32;
constexpr int kDepth = 2;            // tiles of a warp: one in hand, one on its way

// keys of a tile, at multiples of that in the sequence: 4 KB of keys and of values
__host__ __device__ constexpr int tile_keys(int d) { return 4096 / d; }

template <int HD, int NT>
struct DecodeSmem {
  static constexpr int kTileBytes = 4096;
  static constexpr int kStageBytes = 2 * kTileBytes;
  static constexpr int kStages = kWarps * kDepth;          // 96 KB
  static constexpr int kRegs = HD / 16 * NT * 4;           // accumulators of a lane
  static constexpr int merge_off = kStages * kStageBytes;  // [kMergeWarps][kRegs][32] fp32
  static constexpr int merge_bytes = 8192;
  static constexpr int kMergeWarps = merge_bytes / (kRegs * 128) < kWarps
                                         ? merge_bytes / (kRegs * 128) : kWarps;
  static constexpr int pre_off = merge_off + merge_bytes;  // [1025] tiles before each sequence
  static constexpr int misc_off = pre_off + 1028 * 4;
  static constexpr int misc_bytes = 3 * 1024;
  static constexpr int bytes = misc_off + misc_bytes + 1024;
  // two blocks per multiprocessor (228 KB, 1 KB of it reserved for each block)
  static_assert(2 * (bytes + 1024) <= 228 * 1024, "shared memory");
};

struct DecodeMisc {
  uint64_t full[kWarps][kDepth];
  float m[kWarps][kMaxRows], M[kWarps][kMaxRows], l[kWarps][kMaxRows];
  int seen[kWarps][kMaxRows];
  Range range[kMaxRows];                // of the run's query rows
  float q_scale[kMaxRows];
  int live[kMaxRows], valid[kMaxRows];  // the row sees a key; the row is in use
  int warp_sums[kWarps], warp_max[kWarps];
  uint32_t flags;   // a bit a row: to be taken again by the definition
  uint32_t values;  // a bit a row: a value of the result is not finite
  int abort;
  float q[128];
};
static_assert(sizeof(DecodeMisc) <= DecodeSmem<128, 1>::misc_bytes, "misc");
static_assert(sizeof(LiteralScratch<kDecodeThreads, 128>) <= 8192, "it shares the merge buffer");

struct DecodeMaps {
  CUtensorMap k, v;  // [n_pages, Hkv * page, HD] bytes, boxes of min(page, tile) rows
};

struct DecodeParams {
  CacheAttnArgs a;
  int group;       // query heads per key head
  int R;           // query rows per key head: group * Nq, contiguous in q
  int rows;        // query rows of a unit: 8 or 16
  int row_tiles;   // ceil(R / rows)
  int units_seq;   // Hkv * row_tiles
  int sub_rows;    // min(page, tile): rows of one copy
  int combine_rows;  // query rows of a block of the combine kernel: 1, 2, 4 or 8
  bool always_whole; // blocks take whole units whatever the lengths: nothing to combine
  int* pre;        // [B + 2] in the workspace, for the combine: tiles before each sequence, whole units
  float* opart;    // [B * units_seq + blocks, rows, HD]
  float* lpart;    // [B * units_seq + blocks, rows]
};

// Tiles that the queries of a sequence need: 0..TA-1, then from TB on.
template <int HD>
struct SeqTiles {
  static constexpr int kTile = tile_keys(HD);
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

template <int HD>
__device__ __forceinline__ SeqTiles<HD> seq_tiles(const CacheAttnArgs& a, int b, bool report) {
  constexpr int kTile = tile_keys(HD);
  const CacheArgs& c = a.cache;
  SeqTiles<HD> s;
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
  // (non-negative: shifts, and no division at run time)
  s.TA = static_cast<int>((static_cast<uint32_t>(s.SA) + kTile - 1) / kTile);
  s.TB = max(static_cast<int>(static_cast<uint32_t>(s.LB) / kTile), s.TA);
  s.T = s.TA + max(static_cast<int>((static_cast<uint32_t>(s.HB) + kTile - 1) / kTile) - s.TB, 0);
  return s;
}

// Keys and values of one sequence and head through its table row, limited to
// the tiles [t0, t1) of the sequence.
template <int D>
struct PagedKV {
  const CacheArgs& a;
  const int32_t* row;
  int h;
  SeqTiles<D> s;
  int t0, t1;
  __device__ bool ok(int j) const {
    const int t = s.tile_of(j);
    return t >= t0 && t < t1;
  }
  __device__ bool page_at(int j) const {
    const int id = row[j / a.p.page];
    return id >= 0 && id < a.p.n_pages;
  }
  __device__ size_t slot(int j) const {
    return static_cast<size_t>(row[j / a.p.page]) * a.p.Hkv + h;
  }
  __device__ float dot(int j, const float* q) const {
    if (!page_at(j)) return __int_as_float(0x7fc00000);
    const uint8_t* k = static_cast<const uint8_t*>(a.c.k8) +
                       (slot(j) * a.p.page + j % a.p.page) * D;
    float s_ = 0.f;
#pragma unroll 2
    for (int c = 0; c < D; c += 16) {
      float x[16];
      from_e4m3_16(*reinterpret_cast<const uint4*>(k + c), x);
#pragma unroll
      for (int e = 0; e < 16; ++e) s_ = fmaf(q[c + e], x[e], s_);
    }
    return s_ * a.c.k_scale[slot(j)];
  }
  __device__ void v(int j, int c, float (&x)[D / 32]) const {
    if (!page_at(j)) {
#pragma unroll
      for (int e = 0; e < D / 32; ++e) x[e] = __int_as_float(0x7fc00000);
      return;
    }
    const uint8_t* v8 = static_cast<const uint8_t*>(a.c.v8) +
                        (slot(j) * a.p.page + j % a.p.page) * D + c;
    const float scale = a.c.v_scale[slot(j)];
    uint32_t w;
    if (D == 128) w = *reinterpret_cast<const uint32_t*>(v8);
    else w = *reinterpret_cast<const uint16_t*>(v8);
#pragma unroll
    for (int e = 0; e < D / 32; ++e) x[e] = from_e4m3((w >> (8 * e)) & 0xffu) * scale;
  }
  // the value of key j is there, in the tiles, and not finite
  __device__ bool bad_value(int j) const {
    if (!(j < s.SA || (j >= s.LB && j < s.HB)) || !ok(j) || !page_at(j)) return false;
    const uint4* v8 = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(a.c.v8) +
                                                     (slot(j) * a.p.page + j % a.p.page) * D);
    bool bad = !(fabsf(a.c.v_scale[slot(j)]) < INFINITY);
#pragma unroll 1
    for (int c = 0; c < D / 16; ++c) {
      const uint4 x = v8[c];
      const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
      for (int e = 0; e < 4; ++e)  // NaN is all ones beside the sign
        bad = bad || (((w[e] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) != 0u;
    }
    return bad;
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
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// D (16x8, fp32) += A (16x8, tf32) B (8x8, tf32)
__device__ __forceinline__ void mma1688_tf32(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                             uint32_t b1) {
  asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// rounded to tf32: 11 significant bits
__device__ __forceinline__ uint32_t to_tf32(float x) {
  uint32_t r;
  asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(r) : "f"(x));
  return r;
}

// transpose of an 8x8 matrix of 16-bit values (lane 4 r + c holds row r, columns 2c, 2c + 1)
__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
  uint32_t d;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
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
  if (total < (1 << 22))
    return static_cast<int>((static_cast<uint32_t>(x + 1) * static_cast<uint32_t>(blocks) - 1) /
                            static_cast<uint32_t>(total));
  return static_cast<int>(((x + 1) * blocks - 1) / total);
}
__device__ __forceinline__ int blocks_for(long long total) {
  if (total >= static_cast<long long>(kDecodeBlocks) * kMinTiles) return kDecodeBlocks;
  return max(1, (static_cast<int>(total) + kMinTiles - 1) / kMinTiles);
}

// Few query rows. The tiles of all (sequence, key head, 8 or 16 query rows)
// units form one line that is cut evenly over the blocks, whatever the lengths:
// a block takes a run of it, which may end one unit, hold several and begin
// another; or blocks take whole units, where that is shorter (whole_is_shorter).
// Of a run, warp w takes every 6th tile: it looks the pages up (32 at a time, ahead), fetches keys and values by TMA into its own two stages and keeps
// its own running maxima, sum and accumulator in registers, so that warps do not
// wait for one another (one warp that fetched for all was the bound: 3.3 TB/s).
// The first tiles of the next run are fetched before the warps are merged at
// the end of a run; a run that does not hold its whole unit leaves a partial
// result for cache_combine_kernel.
//
// Both products have the cache as the 16-row operand (keys, then columns of V) and
// the query rows as the 8 columns: x^T = K q^T, o^T = V^T p^T. Fragments of mma
// m16n8k16 (g = lane / 4, t = lane % 4). The order of d within a product and
// the order of the output columns are free, so a lane takes 16 contiguous bytes:
// of keys g and g + 8, d = 16 c .. 16 c + 15 at chunk c = 2 t + u (HD = 128; c = t for
// 64), 4 bytes for each step of 16; and of the values 2t, 2t+1, 2t+8, 2t+9 the
// columns (HD / 8) g .. The tile is swizzled by TMA, so that the lanes of a
// quarter warp meet different banks. The weights are turned into the second
// product's operand by an 8x8 transpose.
//
// Bound by the stream of pages where there is much to read (32 sequences of up to
// 8,192 tokens, 8 key heads: 86.8 us, 4.2 TB/s; 72 us without the arithmetic), else by
// latency: a block's run takes about 7 us around its first tiles (12 heads of 1,000 tokens:
// 17.7 us with the combine). Two blocks of six warps hide one another's ends: one block of
// twelve took 105 us.
template <int HD, int NT, typename T>
__global__ void __launch_bounds__(kDecodeThreads, 2)
    cache_decode_kernel(const __grid_constant__ DecodeMaps maps, const DecodeParams p) {
  using L = DecodeSmem<HD, NT>;
  constexpr int kTile = tile_keys(HD);
  constexpr int kRows = 8 * NT;
  constexpr int kU = HD / 64;        // 16-byte pieces of a key per lane
  constexpr int kSteps = HD / 16;    // steps of the first product, row tiles of the second
  constexpr int kKt = kTile / 16;    // row tiles of the first product, steps of the second
  const CacheAttnArgs& a = p.a;
  const CacheArgs& c = a.cache;
  const int B = c.p.B, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  float* merge = reinterpret_cast<float*>(smem + L::merge_off);
  int* pre = reinterpret_cast<int*>(smem + L::pre_off);
  DecodeMisc& ms = *reinterpret_cast<DecodeMisc*>(smem + L::misc_off);
  LiteralScratch<kDecodeThreads, HD>& scratch =
      *reinterpret_cast<LiteralScratch<kDecodeThreads, HD>*>(smem + L::merge_off);

  // Put in place beside the tail of what came before on the stream, all of which is
  // waited for here; the combine kernel is put in place likewise as blocks end.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (tid == 0) {
    for (int s = 0; s < L::kStages; ++s) mbar_init(&ms.full[0][0] + s, 1);
    ms.abort = 0;
    ms.flags = ms.values = 0;
    fence_barrier_init();
  }
  // tiles before each sequence, and the most tiles of one
  int carry = 0, longest = 0;
  for (int b0 = 0; b0 < B; b0 += kDecodeThreads) {
    const int b = b0 + tid;
    const int mine = b < B ? seq_tiles<HD>(a, b, blockIdx.x == 0).T : 0;
    int x = mine;
    longest = max(longest, mine);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) ms.warp_sums[warp] = x;
    __syncthreads();
    int before = carry + x - mine;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) before += ms.warp_sums[w];
      carry += ms.warp_sums[w];
    }
    if (b < B) {
      pre[b] = before;
      if (blockIdx.x == 0) p.pre[b] = before;
      if (b == B - 1) {
        pre[B] = carry;
        if (blockIdx.x == 0) p.pre[B] = carry;
      }
    }
    __syncthreads();
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) longest = max(longest, __shfl_xor_sync(0xffffffffu, longest, o));
  if (lane == 0) ms.warp_max[warp] = longest;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWarps; ++w) longest = max(longest, ms.warp_max[w]);
  const bool whole_units =
      p.always_whole || whole_is_shorter(longest, static_cast<long long>(carry) * p.units_seq,
                                         static_cast<long long>(B) * p.units_seq);
  if (blockIdx.x == 0 && tid == 0) p.pre[B + 1] = whole_units;
  // positions are units of the sequences in order, or tiles of them
  const long long total = whole_units ? static_cast<long long>(B) * p.units_seq
                                      : static_cast<long long>(carry) * p.units_seq;
  const int blocks = whole_units ? static_cast<int>(min(total, static_cast<long long>(kDecodeBlocks)))
                                 : blocks_for(total);
  if (total == 0 || static_cast<int>(blockIdx.x) >= blocks) return;
  long long begin, end;
  if (total < (1 << 22)) {  // 32-bit divisions; there are under 2^10 blocks
    begin = static_cast<uint32_t>(total) * blockIdx.x / static_cast<uint32_t>(blocks);
    end = static_cast<uint32_t>(total) * (blockIdx.x + 1) / static_cast<uint32_t>(blocks);
  } else {
    begin = total * blockIdx.x / blocks;
    end = total * (blockIdx.x + 1) / blocks;
  }
  volatile int* abort = &ms.abort;

  // the run of one unit inside [begin, end)
  struct Run {
    int b, x, t0, t1;  // sequence, unit of the sequence, tiles
  };
  auto run_at = [&](long long pos) {
    if (whole_units) {
      Run r;
      r.b = static_cast<int>(pos / p.units_seq);
      r.x = static_cast<int>(pos - static_cast<long long>(r.b) * p.units_seq);
      r.t0 = 0;
      r.t1 = pre[r.b + 1] - pre[r.b];
      return r;
    }
    int lo = 0, hi = B;  // pre[lo] * units <= pos < pre[hi] * units
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (static_cast<long long>(pre[mid]) * p.units_seq <= pos) lo = mid;
      else hi = mid;
    }
    const int tiles = pre[lo + 1] - pre[lo];
    const long long off = pos - static_cast<long long>(pre[lo]) * p.units_seq;
    Run r;
    r.b = lo;
    r.x = (off >> 31) == 0 ? static_cast<int>(static_cast<uint32_t>(off) / static_cast<uint32_t>(tiles))
                           : static_cast<int>(off / tiles);
    r.t0 = static_cast<int>(off - static_cast<long long>(r.x) * tiles);
    r.t1 = static_cast<int>(min(static_cast<long long>(tiles), r.t0 + (end - pos)));
    return r;
  };
  // the first position from pos on that has tiles; units without any are written here
  auto with_tiles = [&](long long pos) {
    if (whole_units)
      for (; pos < end; ++pos) {
        const Run r = run_at(pos);
        if (r.t1 > 0) break;
        const int h = r.x / p.row_tiles, row0 = (r.x % p.row_tiles) * kRows;
        const int n = clamp_count(a.n_q, r.b, a.Nq, a.Nq, c.stats, false);
        const size_t base = (static_cast<size_t>(r.b) * a.Hq + static_cast<size_t>(h) * p.group) *
                                a.Nq + row0;
        for (int x = tid; x < kRows * HD; x += kDecodeThreads) {
          const int rr = x / HD;
          if (row0 + rr >= p.R || (row0 + rr) % a.Nq >= n) continue;
          store_f32(static_cast<T*>(a.out) + (base + rr) * HD + x % HD, 0.f);
          if (a.lse && x % HD == 0) a.lse[base + rr] = -INFINITY;
        }
      }
    return pos;
  };
  begin = with_tiles(begin);
  if (begin >= end) return;
  const int sub = p.sub_rows, spp = kTile / sub;  // rows of a copy, copies of a tile: 1, 2, 4
  const int sub_shift = 31 - __clz(sub), page_shift = 31 - __clz(c.p.page);
  const int part = lane & (spp - 1), per_batch = 32 / spp;

  // ---- fetching: tile k of the warp is tile warp + 6 k of its run ----
  struct Look {  // one copy: page (-1: none to fetch), first key, scales
    int id, key0;
    float ks, vs;  // ks < 0: no query sees these keys; NaN: the entry holds no page
  };
  struct Fetch {
    Run r;
    SeqTiles<HD> s;
    int h, count, batch;  // key head, tiles of this warp, first tile of `now`
    Look now, next;
    float ks0, vs0;       // scales of the batch before `now`, whose last tiles are still in use
  } f = {};
  uint32_t fetched = 0;  // tiles of this warp so far
  uint8_t* const my_stages = smem + warp * kDepth * L::kStageBytes;
  auto look_up = [&](int k0) {
    Look x = {-1, 0, -1.f, 1.f};
    const int k = k0 + lane / spp;  // this lane's tile
    if (k < f.count) {
      x.key0 = f.s.start(f.r.t0 + warp + k * kWarps) + part * sub;
      // keys of this copy that some query sees
      if (x.key0 < f.s.SA || (x.key0 < f.s.HB && x.key0 + sub > f.s.LB)) {
        x.id = c.c.table[static_cast<size_t>(f.r.b) * c.p.max_pages + (x.key0 >> page_shift)];
        if (x.id < 0 || x.id >= c.p.n_pages) {
          raise_status(c.stats, SPARSEPR_ERR_INVALID_ARG);
          x.id = -1;
          x.ks = __int_as_float(0x7fc00000);  // logits of keys without a page are NaN
        }
      }
    }
    return x;
  };
  // first needed when a tile is in hand: these loads pass behind its copy
  auto look_up_scales = [&](Look& x) {
    if (x.id >= 0) {
      const size_t slot = static_cast<size_t>(x.id) * c.p.Hkv + f.h;
      x.ks = fabsf(c.c.k_scale[slot]);
      x.vs = c.c.v_scale[slot];
    }
  };
  auto fetch = [&](int k) {
    if (__any_sync(0xffffffffu, *abort != 0)) return;
    if (k == f.batch + per_batch) {
      f.ks0 = f.now.ks;
      f.vs0 = f.now.vs;
      f.now = f.next;
      f.batch = k;
      f.next = look_up(k + per_batch);
      look_up_scales(f.next);
    }
    const int st = fetched % kDepth;
    const bool load = lane / spp == k - f.batch && f.now.id >= 0;  // lanes of this tile
    const unsigned have = __ballot_sync(0xffffffffu, load);
    uint64_t* bar = &ms.full[warp][st];
    if (lane == 0) mbar_arrive_expect_tx(bar, __popc(have) * 2 * sub * HD);
    __syncwarp();
    if (load) {
      uint8_t* dst = my_stages + st * L::kStageBytes + part * sub * HD;
      const int y = f.h * c.p.page + (f.now.key0 & (c.p.page - 1));
      tma_load_3d(dst, &maps.k, bar, 0, y, f.now.id);
      tma_load_3d(dst + L::kTileBytes, &maps.v, bar, 0, y, f.now.id);
    }
    ++fetched;
  };
  auto begin_run = [&](long long pos) {
    f.r = run_at(pos);
    f.s = seq_tiles<HD>(a, f.r.b, false);
    f.h = p.row_tiles == 1 ? f.r.x : f.r.x / p.row_tiles;
    const int n = f.r.t1 - f.r.t0;
    f.count = warp < n ? (n - warp + kWarps - 1) / kWarps : 0;
    f.batch = 0;
    f.now = look_up(0);
    for (int k = 0; k < min(f.count, kDepth); ++k) fetch(k);
    look_up_scales(f.now);
    f.next = look_up(per_batch);
    look_up_scales(f.next);
  };

  {
    const int g = lane >> 2, t4 = lane & 3;
    const BlockSync sync;
    uint32_t taken = 0;  // tiles of this warp so far
    // Queries of a run as the first product's operand, in the merge buffer, which is
    // free then: lane (g, t) holds row g + 8 nt, in fp16, scaled by a power of two so that the
    // row's largest value lies in [2^14, 2^15): values down to 2^-28 of it keep 11 bits (and
    // bf16 values, of 8 bits, are exact down to 2^-31 of it). Thread = (row, 1 / 8 of its columns).
    uint2* const qs = reinterpret_cast<uint2*>(merge);  // [NT][kSteps][32]
    auto put_queries = [&](const Run& r, const SeqTiles<HD>& s, int h) {
      constexpr int kC = HD / 8;  // 16 or 8 columns a thread: a chunk, or half of one
      for (int x0 = tid & ~7; x0 < kRows * 8; x0 += kDecodeThreads) {
        const int rr = x0 >> 3, piece = tid & 7;
        const int row = p.row_tiles == 1 ? rr : (r.x % p.row_tiles) * kRows + rr;
        const int i = a.Nq == 1 ? 0 : row % a.Nq;
        const bool have = row < p.R && i < s.n;
        float x[kC], top = 0.f;
        if (have) {
          const T* src = static_cast<const T*>(a.q) + ((static_cast<size_t>(r.b) * a.Hq +
              static_cast<size_t>(h) * p.group) * a.Nq + row) * HD + kC * piece;
          constexpr int kVec = 16 / sizeof(T);
#pragma unroll
          for (int v = 0; v < kC / kVec; ++v) {
            const uint4 w = reinterpret_cast<const uint4*>(src)[v];
            const T* el = reinterpret_cast<const T*>(&w);
#pragma unroll
            for (int k = 0; k < kVec; ++k) x[v * kVec + k] = load_f32(el + k);
          }
        } else {
#pragma unroll
          for (int k = 0; k < kC; ++k) x[k] = 0.f;
        }
#pragma unroll
        for (int k = 0; k < kC; ++k) top = fmaxf(top, fabsf(x[k]));
        const unsigned eight = 0xffu << (lane & 24);
#pragma unroll
        for (int w = 1; w < 8; w <<= 1) top = fmaxf(top, __shfl_xor_sync(eight, top, w));
        // exponent of the row's largest value, so that its power of two is normal both ways
        const int ex = top > 0.f ? min(max(static_cast<int>(__float_as_uint(top) >> 23) - 127, -112), 127) : 0;
        const float down = __uint_as_float((127 + 14 - ex) << 23);
        const int nt = rr >> 3, to = (rr & 7) * 4;
#pragma unroll
        for (int k = 0; k < kC; k += 4) {
          // columns 16 c + 4 w .. of chunk c = kU t + u are step 4 u + w of lane t
          const int col = kC * piece + k, chunk = col >> 4, w = (col >> 2) & 3;
          const int t = chunk / kU, step = 4 * (chunk % kU) + w;
          qs[(nt * kSteps + step) * 32 + to + t] =
              make_uint2(pack_f16x2(x[k] * down, x[k + 1] * down),
                         pack_f16x2(x[k + 2] * down, x[k + 3] * down));
        }
        if (piece == 0) {
          Range rg = {0, 0, 0};
          if (have) rg = visible_range(a.see, static_cast<long long>(s.L) - s.n + i, s.L);
          const bool on = rg.s > 0 || rg.hi > rg.lo;
          ms.range[rr] = rg;
          ms.live[rr] = on;
          ms.valid[rr] = have;
          ms.q_scale[rr] = a.sc * __uint_as_float((127 - 14 + ex) << 23);
        }
      }
    };
    begin_run(begin);
    put_queries(f.r, f.s, f.h);
    sync();
    for (long long pos = begin; pos < end;) {
      const Run r = f.r;
      const SeqTiles<HD> s = f.s;
      const int h = f.h, row0 = p.row_tiles == 1 ? 0 : (r.x % p.row_tiles) * kRows;
      const size_t q_base = (static_cast<size_t>(r.b) * a.Hq + static_cast<size_t>(h) * p.group) *
                                a.Nq + row0;  // of q, out, lse: rows are contiguous
      float qf[NT][2];   // rows 2 t + e + 8 nt of this lane: logit = accumulator * qf * k_scale
      bool live[NT][2];
      // a tile that starts at key `from` or later and ends by `to` is seen whole by all rows
      int from = 0, to = 0x7fffffff;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int rr = 2 * t4 + e + 8 * nt;
          qf[nt][e] = ms.q_scale[rr];
          live[nt][e] = ms.live[rr];
          const Range rg = ms.range[rr];
          if (live[nt][e]) {
            from = max(from, rg.s == rg.lo ? 0 : rg.lo);
            to = min(to, rg.hi);
          }
        }
#pragma unroll
      for (int w = 1; w < 4; w <<= 1) {
        from = max(from, __shfl_xor_sync(0xffffffffu, from, w));
        to = min(to, __shfl_xor_sync(0xffffffffu, to, w));
      }
      float m[NT][2], M[NT][2], l[NT][2], af[NT][2];
      bool seen[NT][2];
      float o[kSteps][NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          m[nt][e] = M[nt][e] = -INFINITY;
          l[nt][e] = 0.f;
          seen[nt][e] = false;
        }
#pragma unroll
        for (int mt = 0; mt < kSteps; ++mt)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[mt][nt][e] = 0.f;
      }

      const int n_tiles = r.t1 - r.t0, count = f.count;
      for (int kth = 0; kth < count; ++kth, ++taken) {
        const int st = taken % kDepth;
        const bool got = mbar_wait(&ms.full[warp][st], (taken / kDepth) & 1u, abort);
        if (!__all_sync(0xffffffffu, got)) continue;  // aborted: the status word says so
        const uint8_t* ks8 = my_stages + st * L::kStageBytes;
        const uint8_t* vs8 = ks8 + L::kTileBytes;
        const int k0 = s.start(r.t0 + warp + kth * kWarps);
        // ---- x = k . q, 16 keys at a time ----
        float acc[kKt][NT][4];
#pragma unroll
        for (int kt = 0; kt < kKt; ++kt) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[kt][nt][e] = 0.f;
          uint2 qw[NT][kSteps];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int x = 0; x < kSteps; ++x) qw[nt][x] = qs[(nt * kSteps + x) * 32 + lane];
          uint4 kw[2][kU];
#pragma unroll
          for (int x = 0; x < 2; ++x)
#pragma unroll
            for (int u = 0; u < kU; ++u) {
              const int key = kt * 16 + x * 8 + g;
              const int chunk = kU == 2 ? ((2 * t4 + u) ^ (key & 7)) : (t4 ^ ((key >> 1) & 3));
              kw[x][u] = *reinterpret_cast<const uint4*>(ks8 + key * HD + chunk * 16);
            }
#pragma unroll
          for (int u = 0; u < kU; ++u) {
            const uint32_t w0[4] = {kw[0][u].x, kw[0][u].y, kw[0][u].z, kw[0][u].w};
            const uint32_t w1[4] = {kw[1][u].x, kw[1][u].y, kw[1][u].z, kw[1][u].w};
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const uint32_t ka[4] = {e4m3x2_to_f16x2(w0[x]), e4m3x2_to_f16x2(w1[x]),
                                      e4m3x2_to_f16x2(w0[x] >> 16), e4m3x2_to_f16x2(w1[x] >> 16)};
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
                mma16816(acc[kt][nt], ka, qw[nt][4 * u + x].x, qw[nt][4 * u + x].y);
            }
          }
        }
        // ---- logits, masks, maxima ----
        float ks[kKt], lv[kKt];
        bool whole = true;
#pragma unroll
        for (int kt = 0; kt < kKt; ++kt) {
          const int from = (kth - f.batch) * spp + ((kt * 16) >> sub_shift);
          ks[kt] = __shfl_sync(0xffffffffu, from >= 0 ? f.now.ks : f.ks0, from & 31);
          lv[kt] = log2_of_scale(__shfl_sync(0xffffffffu, from >= 0 ? f.now.vs : f.vs0, from & 31));
          whole = whole && ks[kt] >= 0.f;
        }
        // one scale for all values of the tile: the two maxima differ by it
        bool one_scale = true;
#pragma unroll
        for (int kt = 1; kt < kKt; ++kt) one_scale = one_scale && lv[kt] == lv[0];
        const bool plain = whole && k0 >= from && k0 + kTile <= to;  // the same in the whole warp
        // The references m and M of a row (-inf: nothing seen) come from the maxima of an
        // earlier tile; they move only when a value passes them by 2^60 (weights of l, fp32)
        // or 2^15 (weights of the second product, fp16 up to 2^16). M is set 8 below the
        // maximum, so that weights 22 to 29 below the largest are still normal fp16 numbers.
        float tm[NT][2], tM[NT][2];  // this lane's maxima
        bool rise = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            tm[nt][e] = tM[nt][e] = -INFINITY;
#pragma unroll
            for (int kt = 0; kt < kKt; ++kt)
#pragma unroll
              for (int x = 0; x < 2; ++x) {
                float v = acc[kt][nt][2 * x + e] * (qf[nt][e] * ks[kt]);
                if (!plain) {
                  const int key = k0 + kt * 16 + x * 8 + g;
                  const Range rr = ms.range[2 * t4 + e + 8 * nt];
                  if (ks[kt] < 0.f || !(key < rr.s || (key >= rr.lo && key < rr.hi))) v = -INFINITY;
                  else seen[nt][e] = true;
                }
                acc[kt][nt][2 * x + e] = v;
                tm[nt][e] = fmaxf(tm[nt][e], v);
                if (!one_scale) tM[nt][e] = fmaxf(tM[nt][e], v + lv[kt]);
              }
            if (one_scale) tM[nt][e] = tm[nt][e] + lv[0];
            if (plain) seen[nt][e] = true;
            rise = rise || tm[nt][e] > m[nt][e] + 60.f || tM[nt][e] > M[nt][e] + 15.f;
          }
        if (__any_sync(0xffffffffu, rise)) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float x = tm[nt][e], y = tM[nt][e];
#pragma unroll
              for (int w = 4; w < 32; w <<= 1) {
                x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, w));
                y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, w));
              }
              x = fmaxf(m[nt][e], x);
              y = fmaxf(M[nt][e], y - 8.f);
              // -inf only where nothing has been seen: the sums are 0 then
              l[nt][e] *= x == -INFINITY ? 0.f : ex2_approx(m[nt][e] - x);
              af[nt][e] = y == -INFINITY ? 0.f : ex2_approx(M[nt][e] - y);
              m[nt][e] = x;
              M[nt][e] = y;
            }
#pragma unroll
          for (int mt = 0; mt < kSteps; ++mt)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int e = 0; e < 4; ++e) o[mt][nt][e] *= af[nt][e & 1];
        }
        float nm[NT][2], nM[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            nm[nt][e] = m[nt][e] == -INFINITY ? 0.f : m[nt][e];
            nM[nt][e] = M[nt][e] == -INFINITY ? 0.f : M[nt][e];
          }
        // ---- weights and the second product, 16 keys at a time ----
        constexpr int kW = HD / 32;  // words of a value per lane
        // HD / 8 bytes of the value of a key of the tile
        auto load_value = [&](int key, bool unread, uint32_t (&vw)[kW]) {
          if (HD == 128) {
            const uint4 v = *reinterpret_cast<const uint4*>(vs8 + key * HD + (g ^ (key & 7)) * 16);
            vw[0] = v.x;
            vw[1] = v.y;
            vw[kW - 2] = v.z;
            vw[kW - 1] = v.w;
          } else {
            const uint2 v = *reinterpret_cast<const uint2*>(
                vs8 + key * HD + ((g >> 1) ^ ((key >> 1) & 3)) * 16 + (g & 1) * 8);
            vw[0] = v.x;
            vw[1] = v.y;
          }
          if (!plain) {
            // a value that no row sees may be anything, also NaN
            const int kx = k0 + key;
            if (unread || !(kx < s.SA || (kx >= s.LB && kx < s.HB)))
#pragma unroll
              for (int w = 0; w < kW; ++w) vw[w] = 0u;
          }
        };
        __half2 least = __float2half2_rn(1.f);  // of the weights of visible keys
#pragma unroll
        for (int kt = 0; kt < kKt; ++kt) {
          uint32_t pb[NT][2];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const float sh[2] = {lv[kt] - nM[nt][0], lv[kt] - nM[nt][1]};
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const float v0 = acc[kt][nt][2 * x], v1 = acc[kt][nt][2 * x + 1];
              l[nt][0] += ex2_approx(v0 - nm[nt][0]);
              l[nt][1] += ex2_approx(v1 - nm[nt][1]);
              const uint32_t p2 = pack_f16x2(ex2_approx(v0 + sh[0]), ex2_approx(v1 + sh[1]));
              uint32_t p2_seen = p2;
              if (!plain) p2_seen |= (v0 == -INFINITY ? 0x3c00u : 0u) | (v1 == -INFINITY ? 0x3c000000u : 0u);
              least = __hmin2(least, *reinterpret_cast<const __half2*>(&p2_seen));
              pb[nt][x] = transpose8x8(p2);
            }
          }
          uint32_t vw[4][kW];  // keys 2t, 2t+1, 2t+8, 2t+9
#pragma unroll
          for (int e = 0; e < 4; ++e)
            load_value(kt * 16 + 2 * t4 + (e & 1) + (e >> 1) * 8, !(ks[kt] >= 0.f), vw[e]);
#pragma unroll
          for (int w = 0; w < kW; ++w) {
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const uint32_t lo = __byte_perm(vw[0][w], vw[1][w], x ? 0x7362 : 0x5140);
              const uint32_t hi = __byte_perm(vw[2][w], vw[3][w], x ? 0x7362 : 0x5140);
              const uint32_t va[4] = {e4m3x2_to_f16x2(lo), e4m3x2_to_f16x2(lo >> 16),
                                      e4m3x2_to_f16x2(hi), e4m3x2_to_f16x2(hi >> 16)};
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) mma16816(o[2 * w + x][nt], va, pb[nt][0], pb[nt][1]);
            }
          }
        }
        // ---- weights below the normal fp16 numbers: what fp16 left of them, in tf32 ----
        // (By way of shared memory and in a loop of its own: with the products in registers in
        // place of those above the calls that never come here took 1% to 8% longer, not up to 1%.)
        const uint32_t lw = *reinterpret_cast<const uint32_t*>(&least);
        if (__any_sync(0xffffffffu, (lw & 0x7c00u) == 0u || (lw & 0x7c000000u) == 0u)) {
          // [key][row], in place of the keys, which have been read
          float* const left = reinterpret_cast<float*>(my_stages + st * L::kStageBytes);
          uint32_t unread = 0;  // groups of 16 keys that were not fetched
          __syncwarp();
#pragma unroll
          for (int kt = 0; kt < kKt; ++kt) {
            unread |= ks[kt] >= 0.f ? 0u : 1u << kt;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float w = ex2_approx(acc[kt][nt][e] + (lv[kt] - nM[nt][e & 1]));
                left[(kt * 16 + (e >> 1) * 8 + g) * kRows + 8 * nt + 2 * t4 + (e & 1)] =
                    w - __half2float(__float2half_rn(w));
              }
          }
          __syncwarp();
#pragma unroll 1
          for (int j = 0; j < kTile / 8; ++j) {  // 8 keys: 2t and 2t + 1 are rows t and t + 4 of the operand
            const int key = j * 8 + 2 * t4;
            uint32_t vw[2][kW];
#pragma unroll
            for (int e = 0; e < 2; ++e) load_value(key + e, (unread >> (j >> 1)) & 1u, vw[e]);
            uint32_t p2[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int e = 0; e < 2; ++e) p2[nt][e] = to_tf32(left[(key + e) * kRows + 8 * nt + g]);
#pragma unroll
            for (int mt = 0; mt < kSteps; ++mt) {
              const uint32_t v = __byte_perm(vw[0][mt / 2], vw[1][mt / 2], mt & 1 ? 0x7362 : 0x5140);
              const uint32_t v0 = e4m3x2_to_f16x2(v), v1 = e4m3x2_to_f16x2(v >> 16);
              const float2 f0 = __half22float2(*reinterpret_cast<const __half2*>(&v0));
              const float2 f1 = __half22float2(*reinterpret_cast<const __half2*>(&v1));
              const uint32_t va[4] = {__float_as_uint(f0.x), __float_as_uint(f1.x),
                                      __float_as_uint(f0.y), __float_as_uint(f1.y)};
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) mma1688_tf32(o[mt][nt], va, p2[nt][0], p2[nt][1]);
            }
          }
          fence_proxy_async_smem();  // the next copy into this stage comes after these writes
        }
        __syncwarp();
        if (kth + kDepth < count) fetch(kth + kDepth);
      }
      const bool full_unit = n_tiles == s.T;
      const size_t slot = static_cast<size_t>(r.b) * p.units_seq + r.x + blockIdx.x;
      pos = with_tiles(pos + (whole_units ? 1 : n_tiles));
      if (pos < end) begin_run(pos);
      // ---- merge of the warps; those without a tile hold -inf, 0 ----
      const int used = min(n_tiles, kWarps);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          int sn = seen[nt][e];
#pragma unroll
          for (int w = 4; w < 32; w <<= 1) {
            l[nt][e] += __shfl_xor_sync(0xffffffffu, l[nt][e], w);
            sn |= __shfl_xor_sync(0xffffffffu, sn, w);
          }
          if (g == 0) {
            const int rr = 2 * t4 + e + 8 * nt;
            ms.m[warp][rr] = m[nt][e];
            ms.M[warp][rr] = M[nt][e];
            ms.l[warp][rr] = l[nt][e];
            ms.seen[warp][rr] = sn;
          }
        }
      sync();
      float inv[NT][2];
      bool on[NT][2];  // rows that saw a key of this run
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int rr = 2 * t4 + e + 8 * nt;
          float gm = -INFINITY, gM = -INFINITY, gl = 0.f;
          int sn = 0;
#pragma unroll
          for (int w = 0; w < kWarps; ++w) {
            gm = fmaxf(gm, ms.m[w][rr]);
            gM = fmaxf(gM, ms.M[w][rr]);
            sn |= ms.seen[w][rr];
          }
          const float zm = gm == -INFINITY ? 0.f : gm, zM = gM == -INFINITY ? 0.f : gM;
#pragma unroll
          for (int w = 0; w < kWarps; ++w) {
            const float mw = ms.m[w][rr], lw = ms.l[w][rr];
            gl += mw == -INFINITY ? lw : lw * ex2_approx(mw - zm);  // without a maximum: 0 or NaN
          }
          on[nt][e] = live[nt][e] && sn;
          // (NaN: a visible logit is NaN or +inf, and so are the row's softmax and result)
          const bool fine = gl > 0.f && gl < INFINITY, lost = gl != gl;
          inv[nt][e] = on[nt][e] && fine ? exp2f(zM - zm) / gl : on[nt][e] && lost ? gl : 0.f;
          const float lse = on[nt][e] && fine ? gm + log2f(gl) : on[nt][e] && lost ? gl : -INFINITY;
          af[nt][e] = ex2_approx(M[nt][e] - zM);
          if (warp == 0 && g == 0) {
            if (on[nt][e] && !lost && !(fine && inv[nt][e] < INFINITY)) atomicOr(&ms.flags, 1u << rr);
            if (!full_unit) p.lpart[slot * kRows + rr] = lse;
            else if (a.lse && ms.valid[rr]) a.lse[q_base + rr] = lse * kLn2F;
          }
        }
      // the accumulators go through shared memory kMergeWarps warps at a time
      constexpr int kMw = L::kMergeWarps;
#pragma unroll
      for (int mt = 0; mt < kSteps; ++mt)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[mt][nt][e] *= af[nt][e & 1];
      for (int w0 = 0; w0 < used; w0 += kMw) {
        if (w0 > 0) sync();
        if (warp >= w0 && warp < min(w0 + kMw, used)) {
          float* to = merge + (warp - w0) * L::kRegs * 32 + lane;
#pragma unroll
          for (int mt = 0; mt < kSteps; ++mt)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                float& x = to[((mt * NT + nt) * 4 + e) * 32];
                x = w0 > 0 ? x + o[mt][nt][e] : o[mt][nt][e];
              }
        }
      }
      sync();
      // accumulators (mt, nt, e) and (mt, nt, e + 2) of lane (g, t), e < 2, are columns
      // (HD / 8) g + 2 mt and the next of row 2 t + e + 8 nt; the warps share them out
      const int summed = min(used, kMw);
#pragma unroll
      for (int j0 = 0; j0 < L::kRegs / 2; j0 += kWarps) {
        const int j = j0 + warp;
        if (j < L::kRegs / 2) {
          const int e = j & 1, nt = (j >> 1) % NT, mt = j / (2 * NT);
          const float* from = merge + ((mt * NT + nt) * 4 + e) * 32 + lane;
          float x0 = 0.f, x1 = 0.f;
#pragma unroll
          for (int w = 0; w < kMw; ++w)
            if (w < summed) {
              x0 += from[w * L::kRegs * 32];
              x1 += from[w * L::kRegs * 32 + 64];
            }
          const int rr = 2 * t4 + e + 8 * nt, col = (HD / 8) * g + 2 * mt;
          const float iv = NT == 1 ? (e ? inv[0][1] : inv[0][0])
                                   : nt ? (e ? inv[NT - 1][1] : inv[NT - 1][0])
                                        : (e ? inv[0][1] : inv[0][0]);
          const bool here = NT == 1 ? (e ? on[0][1] : on[0][0])
                                    : nt ? (e ? on[NT - 1][1] : on[NT - 1][0])
                                         : (e ? on[0][1] : on[0][0]);
          x0 = here ? x0 * iv : 0.f;
          x1 = here ? x1 * iv : 0.f;
          if (here && iv == iv && !(fabsf(x0) < INFINITY && fabsf(x1) < INFINITY))
            atomicOr(&ms.values, 1u << rr);
          if (!full_unit) {
            *reinterpret_cast<float2*>(p.opart + (slot * kRows + rr) * HD + col) = make_float2(x0, x1);
          } else if (ms.valid[rr]) {
            T* dst = static_cast<T*>(a.out) + (q_base + rr) * HD + col;
            store_f32(dst, x0);
            store_f32(dst + 1, x1);
          }
        }
      }
      sync();
      // A result that is not finite comes from values with NaN. It stands unless one of them is
      // hidden from the row (another query sees it; its weight here is 0, but 0 times NaN is
      // NaN); then the row is taken again by the definition. (32 sequences of 8,192 tokens with
      // a NaN that all see: 0.12 ms for one token and 0.34 for eight, without NaN 0.13 and 0.31;
      // when every such row was taken again 21 and 163.)
      uint32_t todo = ms.flags;
      for (uint32_t doubtful = ms.values & ~todo; doubtful; doubtful &= doubtful - 1) {
        const int rr = __ffs(doubtful) - 1;
        const PagedKV<HD> kv = {c, c.c.table + static_cast<size_t>(r.b) * c.p.max_pages, h, s, r.t0,
                                r.t1};
        const Range rg = ms.range[rr];
        bool bad = false;
#pragma unroll 1
        for (int x = 0; x < 3; ++x) {  // keys that another query may see
          const int from = x == 0 ? rg.s : x == 1 ? max(rg.s, s.LB) : rg.hi;
          const int to = x == 0 ? min(rg.lo, s.SA) : x == 1 ? rg.lo : s.HB;
          for (int j = from + tid; j < to; j += kDecodeThreads) bad = bad || kv.bad_value(j);
        }
        if (__syncthreads_or(bad)) todo |= 1u << rr;
      }
      while (todo) {
        const int rr = __ffs(todo) - 1, i = (row0 + rr) % a.Nq;
        todo &= todo - 1;
        const PagedKV<HD> kv = {c, c.c.table + static_cast<size_t>(r.b) * c.p.max_pages, h, s, r.t0,
                                r.t1};
        for (int x = tid; x < HD; x += kDecodeThreads)
          ms.q[x] = load_f32(static_cast<const T*>(a.q) + (q_base + rr) * HD + x);
        sync();
        float lm, ll, lo;
        literal_row<kDecodeThreads, HD>(
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
      if (tid == 0) ms.flags = ms.values = 0;  // all have read it; set again only behind the next barrier
      if (pos < end) {
        put_queries(f.r, f.s, f.h);
        sync();
      }
    }
    // let the copies in flight land (there are none unless the block aborted)
    if (lane == 0) {
      volatile int never = 0;
      for (uint32_t n = fetched > kDepth ? fetched - kDepth : 0; n < fetched; ++n)
        mbar_wait(&ms.full[warp][n % kDepth], (n / kDepth) & 1u, &never);
    }
  }
  __syncthreads();
  if (*abort && tid == 0) raise_status(c.stats, SPARSEPR_ERR_TIMEOUT);
}

// Joins the partial results of units that more than one block worked on, and
// writes the rows that see nothing. One block per (sequence, unit) and
// combine_rows of its rows; the block's 8 warps share out the rows, and the warps of
// a row share out the parts, then add up in a fixed order; lanes take HD / 32
// columns each. A long history of one sequence is cut into up to 296 parts: with few
// units a block takes one row (8 rows x 74 parts of 4 units: 28 us by one warp a
// row, 17 us by a block a unit).
constexpr int kCombineWarps = 8;

template <int HD, int NT, typename T>
__global__ void __launch_bounds__(kCombineWarps * 32) cache_combine_kernel(const DecodeParams p) {
  constexpr int kRows = 8 * NT, kC = HD / 32;
  __shared__ float sums[kCombineWarps][32][kC + 1];
  const CacheAttnArgs& a = p.a;
  const int b = blockIdx.x / p.units_seq, x = blockIdx.x % p.units_seq;
  const int h = x / p.row_tiles, row0 = (x % p.row_tiles) * kRows;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int per_row = kCombineWarps / p.combine_rows;  // warps of a row
  const int rr = blockIdx.y * p.combine_rows + warp / per_row, sub = warp % per_row;
  asm volatile("griddepcontrol.wait;" ::: "memory");  // all of the decode kernel's writes
  const int before = p.pre[b], tiles = p.pre[b + 1] - before, all = p.pre[a.cache.p.B];
  if (p.pre[a.cache.p.B + 1]) return;  // blocks took whole units
  const int n = clamp_count(a.n_q, b, a.Nq, a.Nq, a.cache.stats, false);
  const bool valid = rr < kRows && row0 + rr < p.R && (row0 + rr) % a.Nq < n;
  const size_t row = (static_cast<size_t>(b) * a.Hq + static_cast<size_t>(h) * p.group) * a.Nq +
                     row0 + rr;
  float num[kC] = {};
  float M = -INFINITY, den = 0.f;
  bool nan = false;
  if (tiles > 0) {
    const long long total = static_cast<long long>(all) * p.units_seq;
    const int blocks = blocks_for(total);
    const long long at = static_cast<long long>(before) * p.units_seq + static_cast<long long>(x) * tiles;
    const int c0 = owner(at, total, blocks), c1 = owner(at + tiles - 1, total, blocks);
    if (c0 == c1) return;  // written whole
    const int count = c1 - c0 + 1;
    const size_t slot0 = (static_cast<size_t>(blockIdx.x) + c0) * kRows + rr;
    if (valid) {
#pragma unroll 4
      for (int i = lane; i < count; i += 32) {
        const float l = p.lpart[slot0 + static_cast<size_t>(i) * kRows];
        M = fmaxf(M, l);
        nan = nan || l != l;
      }
#pragma unroll
      for (int w = 16; w > 0; w >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, w));
      nan = __any_sync(0xffffffffu, nan);
      const float zM = M == -INFINITY ? 0.f : M;
      constexpr int kAhead = 8;  // parts in flight
      for (int i0 = sub; i0 < count; i0 += kAhead * per_row) {
        float w[kAhead], o[kAhead][kC];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
          const int i = i0 + k * per_row;
          const size_t slot = slot0 + static_cast<size_t>(min(i, count - 1)) * kRows;
          w[k] = i < count ? p.lpart[slot] : -INFINITY;
#pragma unroll
          for (int e = 0; e < kC; ++e) o[k][e] = p.opart[slot * HD + lane * kC + e];
        }
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
          const float wk = exp2f(w[k] - zM);  // 0 for a part that holds none of the row's keys
          den += wk;
#pragma unroll
          for (int e = 0; e < kC; ++e) num[e] = fmaf(wk, o[k][e], num[e]);
        }
      }
    }
    if (per_row > 1) {
#pragma unroll
      for (int e = 0; e < kC; ++e) sums[warp][lane][e] = num[e];
      sums[warp][lane][kC] = den;
      __syncthreads();
      if (sub != 0) return;
      for (int w = 1; w < per_row; ++w) {
#pragma unroll
        for (int e = 0; e < kC; ++e) num[e] += sums[warp + w][lane][e];
        den += sums[warp + w][lane][kC];
      }
    }
  }
  if (!valid || sub != 0) return;
  const bool some = den > 0.f || nan;
  const float inv = some ? 1.f / den : 0.f;
  T* out = static_cast<T*>(a.out) + row * HD + lane * kC;
#pragma unroll
  for (int e = 0; e < kC; ++e) store_f32(out + e, num[e] * inv);
  if (a.lse && lane == 0) a.lse[row] = nan ? den : some ? (M + log2f(den)) * kLn2F : -INFINITY;
}

// Many query rows: the tokens that some query sees, widened to bf16 rows
// [sequence - b0, head, position, HD] (exact: 4 significant bits times a power of
// two). One block per tile of a sequence and head. Bound by memory: 21,840 tokens of 12
// heads, 67 MB to 134 MB, in 38 us (5.3 TB/s).
template <int HD>
__global__ void __launch_bounds__(256)
    widen_kernel(const CacheAttnArgs a, int b0, int cap, __nv_bfloat16* kb, __nv_bfloat16* vb) {
  const CacheArgs& c = a.cache;
  const int h = blockIdx.y, b = b0 + blockIdx.z;
  const SeqTiles<HD> s = seq_tiles<HD>(a, b, false);
  if (static_cast<int>(blockIdx.x) >= s.T) return;
  if (static_cast<int>(blockIdx.x) == s.TA - 1) {
    // the attention's tiles of 128 keys read on behind the sinks, with weight 0: no NaN there
    const int from = s.TA * tile_keys(HD);
    const int to = min(min((s.SA + kTileN - 1) / kTileN * kTileN, s.TB * tile_keys(HD)), cap);
    uint4* v = reinterpret_cast<uint4*>(
        vb + ((static_cast<size_t>(blockIdx.z) * c.p.Hkv + h) * cap + from) * HD);
    for (int i = threadIdx.x; i < (to - from) * HD / 8; i += 256) v[i] = make_uint4(0, 0, 0, 0);
  }
  constexpr int kPieces = 4096 / 16;  // 16-byte pieces of the tile's keys, one per thread
  static_assert(kPieces == 256, "threads");
  const int key = s.start(blockIdx.x) + threadIdx.x * 16 / HD, col = threadIdx.x * 16 % HD;
  if (key >= s.L) return;
  const int id = c.c.table[static_cast<size_t>(b) * c.p.max_pages + key / c.p.page];
  const size_t to = ((static_cast<size_t>(blockIdx.z) * c.p.Hkv + h) * cap + key) * HD + col;
  const bool page = id >= 0 && id < c.p.n_pages;
  const bool visible = key < s.SA || (key >= s.LB && key < s.HB);
  if (!page && visible) raise_status(c.stats, SPARSEPR_ERR_INVALID_ARG);
  const size_t slot = static_cast<size_t>(page ? id : 0) * c.p.Hkv + h;
  const size_t from = (slot * c.p.page + key % c.p.page) * HD + col;
#pragma unroll
  for (int kv = 0; kv < 2; ++kv) {
    uint4 u[2];
    if (page) {
      const float scale = (kv ? c.c.v_scale : c.c.k_scale)[slot];
      float x[16];
      from_e4m3_16(*reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(kv ? c.c.v8 : c.c.k8) + from), x);
      uint32_t w[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = pack_bf16x2(x[2 * i] * scale, x[2 * i + 1] * scale);
      u[0] = make_uint4(w[0], w[1], w[2], w[3]);
      u[1] = make_uint4(w[4], w[5], w[6], w[7]);
    } else {  // NaN: a query that needs the token shows it
      const uint32_t w = visible ? 0x7fff7fffu : 0u;
      u[0] = u[1] = make_uint4(w, w, w, w);
    }
    uint4* dst = reinterpret_cast<uint4*>((kv ? vb : kb) + to);
    dst[0] = u[0];
    dst[1] = u[1];
  }
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

template <int HD, int NT, typename T>
cudaError_t launch_decode(const DecodeParams& p, const DecodeMaps& maps, cudaStream_t st) {
  constexpr int kBytes = DecodeSmem<HD, NT>::bytes;
  static std::atomic<uint64_t> allowed{0};
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(cache_decode_kernel<HD, NT, T>), kBytes,
                             allowed);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t first = {};  // programmatic dependent launch
  first.gridDim = dim3(kDecodeBlocks);
  first.blockDim = dim3(kDecodeThreads);
  first.dynamicSmemBytes = kBytes;
  first.stream = st;
  cudaLaunchAttribute early[1];
  early[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early[0].val.programmaticStreamSerializationAllowed = 1;
  first.attrs = early;
  first.numAttrs = 1;
  e = cudaLaunchKernelEx(&first, cache_decode_kernel<HD, NT, T>, maps, p);
  if (e != cudaSuccess || p.always_whole) return e;
  // launched beside the tail of the decode kernel
  cudaLaunchConfig_t cfg = {};
  const int rows = min(p.rows, p.R);
  cfg.gridDim = dim3(p.a.cache.p.B * p.units_seq, (rows + p.combine_rows - 1) / p.combine_rows);
  cfg.blockDim = dim3(kCombineWarps * 32);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, cache_combine_kernel<HD, NT, T>, p);
}
template <int HD, typename T>
cudaError_t launch_decode_rows(const DecodeParams& p, const DecodeMaps& maps, cudaStream_t st) {
  return p.rows == 8 ? launch_decode<HD, 1, T>(p, maps, st) : launch_decode<HD, 2, T>(p, maps, st);
}

}  // namespace

CacheAttnPlan cache_attn_plan(const sparsepr_cache_params& p, const sparsepr_cache_attention_params& q) {
  CacheAttnPlan w = {};
  const long long R = static_cast<long long>(q.Hq / p.Hkv) * q.Nq;
  w.wide = R > kWideRows;
  if (w.wide) {
    // bf16 rows of as many sequences at a time as fit 1 GB
    w.cap = p.max_pages * p.page;
    const long long bytes = 4ll * p.Hkv * w.cap * p.d;
    long long g = (1ll << 30) / bytes;
    w.group = static_cast<int>(g < 1 ? 1 : g < p.B ? g : p.B);
    for (int n : {w.group, p.B % w.group}) {
      if (n == 0) continue;
      const WindowPlan plan = window_plan(n, q.Hq, p.Hkv, q.Nq, w.cap, q.see);
      if (plan.part_rows > w.part_rows) w.part_rows = plan.part_rows;
    }
    return w;
  }
  w.rows = R <= 8 ? 8 : 16;
  w.row_tiles = static_cast<int>((R + w.rows - 1) / w.rows);
  w.part_rows = (static_cast<size_t>(p.B) * p.Hkv * w.row_tiles + kDecodeBlocks) * w.rows;
  return w;
}

namespace {

cudaError_t launch_wide(const CacheAttnArgs& a, const CacheAttnPlan& w, cudaStream_t st) {
  const sparsepr_cache_params& p = a.cache.p;
  WindowArgs x = {};
  x.Hq = a.Hq;
  x.Hkv = p.Hkv;
  x.Nq = a.Nq;
  x.Nk = w.cap;
  x.d = p.d;
  x.see = a.see;
  x.sc = a.sc;
  x.bf16 = a.bf16;
  x.kv_bf16 = true;
  x.k = a.kb;
  x.v = a.vb;
  x.stats = a.cache.stats;
  x.qb = a.qb;
  x.opart = a.opart;
  x.lpart = a.lpart;
  const size_t row = static_cast<size_t>(p.d) * (a.bf16 ? 2 : 4);
  for (int b0 = 0; b0 < p.B; b0 += w.group) {
    const size_t q0 = static_cast<size_t>(b0) * a.Hq * a.Nq;
    x.B = min(w.group, p.B - b0);
    const dim3 grid((w.cap + tile_keys(p.d) - 1) / tile_keys(p.d), p.Hkv, x.B);
    if (p.d == 128) widen_kernel<128><<<grid, 256, 0, st>>>(a, b0, w.cap, a.kb, a.vb);
    else widen_kernel<64><<<grid, 256, 0, st>>>(a, b0, w.cap, a.kb, a.vb);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    x.q = static_cast<const char*>(a.q) + q0 * row;
    x.out = static_cast<char*>(a.out) + q0 * row;
    x.lse = a.lse ? a.lse + q0 : nullptr;
    x.n_q = a.n_q ? a.n_q + b0 : nullptr;
    x.n_k = a.cache.c.len + b0;
    if ((e = launch_window_attention(x, st)) != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace

cudaError_t launch_cache_attention(const CacheAttnArgs& a, cudaStream_t st) {
  if (a.Nq == 0) return cudaSuccess;
  sparsepr_cache_attention_params q = {};
  q.Hq = a.Hq;
  q.Nq = a.Nq;
  q.see = a.see;
  const CacheAttnPlan w = cache_attn_plan(a.cache.p, q);
  if (w.wide) return launch_wide(a, w, st);
  DecodeParams p = {};
  p.a = a;
  p.group = a.Hq / a.cache.p.Hkv;
  p.R = p.group * a.Nq;
  p.rows = w.rows;
  p.row_tiles = w.row_tiles;
  p.units_seq = a.cache.p.Hkv * w.row_tiles;
  p.sub_rows = min(a.cache.p.page, tile_keys(a.cache.p.d));
  // tiles that a sequence can have at most: of its table row, or of what is visible
  const long long keys =
      most_visible(a.see, a.Nq, static_cast<long long>(a.cache.p.max_pages) * a.cache.p.page);
  // (a window may begin and the sinks may end inside a tile)
  p.always_whole = keys / tile_keys(a.cache.p.d) + 4 <= kWholeTiles;
  p.combine_rows = 1;
  if (a.cache.p.B * p.units_seq >= kDecodeBlocks / 2)
    while (p.combine_rows < 8 && p.combine_rows < min(p.rows, p.R)) p.combine_rows *= 2;
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
    return a.cache.p.d == 128 ? launch_decode_rows<128, __nv_bfloat16>(p, maps, st)
                              : launch_decode_rows<64, __nv_bfloat16>(p, maps, st);
  return a.cache.p.d == 128 ? launch_decode_rows<128, float>(p, maps, st)
                            : launch_decode_rows<64, float>(p, maps, st);
}

}  // namespace spr
