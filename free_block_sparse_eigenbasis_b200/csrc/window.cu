// Attention with a sliding window of frames and sink frames on the
// 5th-generation tensor cores.
//
// out_i = sum_j p_ij v_j, p_ij = 2^(x_ij - m_i) / l_i, x_ij = scale log2(e) q_i.k_j
// over the keys that row i sees: [0, s_i) and [lo_i, hi_i), whose ends grow
// with i. A unit of up to 256 rows of one head therefore needs the keys [0, SA)
// and [LB, HB) (SA = s of its last row, LB = lo of its first, HB = hi of its
// last), and nothing between them is read. They are cut into tiles of 128 keys;
// a tile that every row of a warp sees whole takes no mask, one that none of them
// sees weights of 0 at once.
//
// Roles (352 threads) as in the routed attention kernel: two softmax
// warpgroups (thread = query row = TMEM lane), a warp that streams Q and the
// K tiles by TMA, one for the V tiles, one that issues tcgen05.mma. Units of two
// 128-row tiles give tile i to warpgroup i; units of one tile give the even key
// tiles to warpgroup 0 and the odd ones to warpgroup 1, merged at the end. P stays
// in tensor memory.
//
// Bound by the tensor cores with their shared-memory operands: 480p clip (12 heads,
// 32,760 rows, 9,360 keys each at most) 1.45 to 1.70 ms, 1,030 to 1,210 TFLOP/s of
// visible pairs, 60% of the tensor cycles at the 1.7 GHz that the power limit leaves;
// 1.35 ms with no softmax at all, 1.50 ms without the copies of K and V (of 1.55). Tiles of
// 128 x 128, because a product with 64 columns takes as long as one with 128.
#include <type_traits>

#include "common.cuh"
#include "internal.h"
#include "visible.cuh"

namespace spr {
namespace {

constexpr int kStages = 2;  // K and V ring depth
constexpr int kThreads = 352;
constexpr uint32_t kTmemCols = 512;  // S_0, S_1 (128 columns each), O_0, O_1
constexpr float kOverflowSum = 4294967296.0f;  // 2^32: a larger half sum moves the reference
constexpr float kMaxReference = 4194304.0f;
constexpr int kMaxWindowSplits = 16;
constexpr int kPlanSMs = 148;

template <int HD>
struct Smem {
  static constexpr int kAtoms = HD / 64;          // 128-byte swizzle atoms along d
  static constexpr int kSlab = kTileM * 128;      // 64 columns of 128 rows (16 KB)
  static constexpr int kTileBytes = kAtoms * kSlab;
  static constexpr int q_off = 0;                 // two query tiles
  static constexpr int k_off = q_off + 2 * kTileBytes;
  static constexpr int v_off = k_off + kStages * kTileBytes;
  static constexpr int bar_off = v_off + kStages * kTileBytes;
  static constexpr int ml_off = bar_off + 256;    // [2][2][128] row maxima and sums
  static constexpr int flag_off = ml_off + 2048;  // Flags
  static constexpr int bytes = flag_off + 96;
};
// The d = 128 footprint for both head dims, so that one block runs per
// multiprocessor (each takes all 512 columns of tensor memory); the tiles start
// at a 1024-byte boundary.
constexpr int kSmemBytes = Smem<128>::bytes + 1024;
static_assert(kSmemBytes <= static_cast<int>(kMaxDynSmem), "shared memory");

struct Bars {
  uint64_t q_full[2];
  uint64_t kfull[kStages], vfull[kStages], kempty[kStages], vempty[kStages];
  uint64_t vfix[2];
  uint64_t s_full[2], p_full[2][2], pa_done[2], o_done[2];
  uint64_t mma_idle;
  uint32_t tmem_base;
  int abort;
};
static_assert(sizeof(Bars) <= 256, "barrier block");

// Rows whose results need a second look.
struct Flags {
  uint32_t again[8];   // a bit a row: to be taken again by the definition
  uint32_t values[8];  // a bit a row: a value of the result is not finite
  // keys of the block's tiles with values that are not finite:
  int last, first;     // the last one, the first one behind the sinks
  uint32_t nan[4];     // columns that are NaN in a key that all rows of the unit see
};
static_assert(sizeof(Flags) <= 96, "flags");

struct WindowMaps {
  CUtensorMap q, k, v;
};

struct WindowKernelParams {
  WindowArgs a;
  int group;           // query heads per key head
  int R, segs;         // rows per segment, segments (heads, or key heads with packed groups)
  int tiles;           // units per segment
  int unit_rows;       // 256 or 128
  int whole;           // the first units of the grid's order are one block each,
  int splits;          // the others this many, which leave partial results
  int q_box_rows, kv_box_rows;
  // the kernel divides by these: some fifteen divisions at run time took 2,300 cycles
  // at the start of every block
  Divider by_segs, by_group, by_Hq, by_Nq, by_splits, by_frame;
  float* opart;        // [units - whole, splits, unit_rows, d] normalised partial outputs
  float* lpart;        // [units - whole, splits, unit_rows] their log2-sum-exps
};

__device__ __forceinline__ void fma2(float& x0, float& x1, float a0, float a1, float b, float c) {
  asm("{\n\t.reg .b64 ra, rb, rc, rd;\n\t"
      "mov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %4};\n\tmov.b64 rc, {%5, %5};\n\t"
      "fma.rn.f32x2 rd, ra, rb, rc;\n\tmov.b64 {%0, %1}, rd;\n\t}"
      : "=f"(x0), "=f"(x1)
      : "f"(a0), "f"(a1), "f"(b), "f"(c));
}
__device__ __forceinline__ void add2(float2& x, float a, float b) {
  asm("{\n\t.reg .b64 ra, rb, rd;\n\t"
      "mov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\t"
      "add.rn.f32x2 rd, ra, rb;\n\tmov.b64 {%0, %1}, rd;\n\t}"
      : "=f"(x.x), "=f"(x.y)
      : "f"(x.x), "f"(x.y), "f"(a), "f"(b));
}
__device__ __forceinline__ float max3f(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, uint64_t* bar,
                                            int32_t x, int32_t y, int32_t z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z)
      : "memory");
}

__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}

// one lane of the (converged) warp
__device__ __forceinline__ bool elect_one() {
  uint32_t is;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(is));
  return is != 0;
}

// bits [a, b) of a 32-bit word (any a, b)
__device__ __forceinline__ uint32_t bit_range(int a, int b) {
  a = max(a, 0);
  b = min(b, 32);
  if (a >= b) return 0u;
  return (b == 32 ? 0xFFFFFFFFu : ((1u << b) - 1u)) & ~((1u << a) - 1u);
}

// The keys of a unit and this block's share of their tiles.
struct UnitKeys {
  int SA, LB, HB, TA;  // [0, SA) in TA tiles, then [LB, HB)
  int j0, T;           // this block's tiles
  __device__ int start(int j) const { return j < TA ? j * kTileN : LB + (j - TA) * kTileN; }
  __device__ int end(int j) const {
    return min(start(j) + kTileN, j < TA ? SA : HB);
  }
  __device__ int tile_of(int key) const {
    return key < SA ? key / kTileN : TA + (key - LB) / kTileN;
  }
};

// K and V rows of one head for the literal pass, limited to the block's tiles
template <int HD>
struct TileKV {
  const __nv_bfloat16 *k, *vals;
  UnitKeys u;
  __device__ bool ok(int j) const {
    const int t = u.tile_of(j);
    return t >= u.j0 && t < u.j0 + u.T;
  }
  __device__ float dot(int j, const float* q) const {
    const uint4* row = reinterpret_cast<const uint4*>(k + static_cast<size_t>(j) * HD);
    float s = 0.f;
#pragma unroll 4
    for (int c = 0; c < HD / 8; ++c) {
      const uint4 x = row[c];
      const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        s = fmaf(q[c * 8 + 2 * e], __uint_as_float(w[e] << 16), s);
        s = fmaf(q[c * 8 + 2 * e + 1], __uint_as_float(w[e] & 0xFFFF0000u), s);
      }
    }
    return s;
  }
  __device__ void v(int j, int c, float (&x)[HD / 32]) const {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(vals + static_cast<size_t>(j) * HD + c);
#pragma unroll
    for (int e = 0; e < HD / 64; ++e) {
      const uint32_t y = w[e];
      x[2 * e] = __uint_as_float(y << 16);
      x[2 * e + 1] = __uint_as_float(y & 0xFFFF0000u);
    }
  }
};

// The 32 rows of a warp, half a row (HD / 2 columns) at a time, go to memory by
// way of shared memory, so that a store instruction covers whole lines: a thread
// that writes its own row touches 32 lines with each, 4,500 cycles a block at
// d = 128. The 16-byte pieces of a row are swizzled against bank conflicts.
template <typename T, int HD>
struct RowStage {
  static constexpr int kPer = 16 / static_cast<int>(sizeof(T));  // values of a piece
  static constexpr int kPieces = HD / 2 / kPer;                  // of half a row: 4, 8 or 16
  static __device__ __forceinline__ int at(int row, int piece) {
    return row * kPieces + (piece ^ (kPieces >= 8 ? row & 7 : (row >> 1) & 3));
  }
  // 32 columns of the lane's row, the c32-th of its half, times f
  static __device__ __forceinline__ void put(uint4* stage, int lane, int c32, const uint32_t (&o)[32],
                                             float f) {
#pragma unroll
    for (int k = 0; k < 32; k += kPer) {
      uint4 u;
      uint32_t* w = &u.x;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int x = k + e * kPer / 4;
        if constexpr (kPer == 4) w[e] = __float_as_uint(__uint_as_float(o[x]) * f);
        else w[e] = pack_bf16x2(__uint_as_float(o[x]) * f, __uint_as_float(o[x + 1]) * f);
      }
      stage[at(lane, (c32 * 32 + k) / kPer)] = u;
    }
  }
  // dst: the half's first column in the warp's first row; rows: the lanes whose rows are written
  static __device__ __forceinline__ void flush(const uint4* stage, int lane, T* dst, uint32_t rows) {
    __syncwarp();
#pragma unroll
    for (int j = 0; j < kPieces; ++j) {
      const int x = j * 32 + lane, row = x / kPieces, piece = x % kPieces;
      if ((rows >> row) & 1u)
        *reinterpret_cast<uint4*>(dst + static_cast<size_t>(row) * HD + piece * kPer) =
            stage[at(row, piece)];
    }
    __syncwarp();
  }
};

// Segment and tile of the n-th unit of the grid: segments vary fastest, and with a
// causal visibility the last rows of all segments, which see the most, come first.
__device__ __forceinline__ void unit_place(const WindowKernelParams& p, int unit, int& seg,
                                           int& tile) {
  tile = p.by_segs.div(unit);
  seg = unit - tile * p.segs;
  if (p.a.see.causal) tile = p.tiles - 1 - tile;
}

// What the second look at rows needs of a block's unit.
struct Unit {
  UnitKeys keys;
  int r0, i_last, len;
  bool partial;
  long long pos0;
  int kvh;
  size_t row_base, pbase;
};

// Rows whose result is not finite. It comes from values of the block's tiles that are not
// finite. The result stands where the row sees all such keys, and where each of its columns
// that are not finite is NaN in a key that all rows of the unit see. Else a key hidden from the
// row may have done it (its weight is 0, but 0 times NaN is NaN), or a sum that left fp32, and
// the row is taken again by the definition. (480p clip, 1.6 ms: with a NaN in the sink frame or
// all values NaN 3.0 ms, with one in a middle frame, at whose ends units see it in part,
// 70 ms; when every such row was taken again 1,635 and 544 ms.)
template <int HD, typename T>
__device__ __forceinline__ void look_again(const WindowKernelParams& p, const Unit& unit, uint8_t* smem,
                                        Flags& flags) {
  const WindowArgs& a = p.a;
  const UnitKeys& u = unit.keys;
  const size_t kvoff = static_cast<size_t>(unit.kvh) * a.Nk * HD;
  const __nv_bfloat16* const kbase = static_cast<const __nv_bfloat16*>(a.k) + kvoff;
  const __nv_bfloat16* const vbase = static_cast<const __nv_bfloat16*>(a.v) + kvoff;
  auto range_of = [&](int i) { return visible_range(a.see, unit.pos0 + i, unit.len, p.by_frame); };
  uint32_t doubtful = 0;
  for (int w = 0; w < 8; ++w) doubtful |= flags.values[w];
  if (doubtful) {
    if (threadIdx.x == 0) {
      flags.last = -1;
      flags.first = 0x7fffffff;
      for (int c = 0; c < 4; ++c) flags.nan[c] = 0;
    }
    __syncthreads();
    // all rows of the unit see [0, common.s) and [common.lo, common.hi): its first query, or
    // query 0 where rows go on from head to head, ends first, its last begins last
    const Range begin = range_of(p.R != a.Nq ? 0 : unit.r0), end = range_of(unit.i_last);
    const Range common = {begin.s, end.lo, begin.hi};
    int last = -1, first = 0x7fffffff;
    uint32_t nan = 0;  // of this thread's 8 columns
    const int piece = threadIdx.x % (HD / 8);
    static_assert(kThreads % (HD / 8) == 0, "a thread keeps to its columns");
    for (int j = u.j0; j < u.j0 + u.T; ++j) {
      const int k0 = u.start(j), k1 = u.end(j);
      for (int key = k0 + static_cast<int>(threadIdx.x) / (HD / 8); key < k1; key += kThreads / (HD / 8)) {
        const uint4 y = reinterpret_cast<const uint4*>(vbase + static_cast<size_t>(key) * HD)[piece];
        const uint32_t w[4] = {y.x, y.y, y.z, y.w};
        uint32_t here = 0;
        bool bad = false;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const uint32_t x = (w[e >> 1] >> (16 * (e & 1))) & 0x7fffu;
          bad = bad || x >= 0x7f80u;
          here |= x > 0x7f80u ? 1u << e : 0u;
        }
        if (bad) {
          last = max(last, key);
          if (key >= end.s) first = min(first, key);
          if (key < common.s || (key >= common.lo && key < common.hi)) nan |= here;
        }
      }
    }
    if (last >= 0) {
      atomicMax(&flags.last, last);
      atomicMin(&flags.first, first);
      if (nan) atomicOr(&flags.nan[piece >> 2], nan << (8 * (piece & 3)));
    }
    __syncthreads();
    const int ur = threadIdx.x;
    if (ur < 256 && ((flags.values[ur >> 5] >> (ur & 31)) & 1u)) {
      const Range rg = range_of(p.by_Nq.mod(unit.r0 + ur));
      if (flags.last < 0 || flags.last >= rg.hi || (rg.s < rg.lo && flags.first < rg.lo)) {
        bool explained = true;
        for (int c = 0; c < HD; ++c) {
          const float x = unit.partial ? p.opart[(unit.pbase + ur) * HD + c]
                                       : load_f32(static_cast<const T*>(a.out) + (unit.row_base + ur) * HD + c);
          if (!(fabsf(x) < INFINITY)) explained = explained && ((flags.nan[c >> 5] >> (c & 31)) & 1u);
        }
        if (!explained) atomicOr(&flags.again[ur >> 5], 1u << (ur & 31));
      }
    }
    __syncthreads();
  }
  LiteralScratch<kThreads, HD>& scratch = *reinterpret_cast<LiteralScratch<kThreads, HD>*>(smem);
  static_assert(sizeof(scratch) <= 8192, "the query lies behind it");
  float* q = reinterpret_cast<float*>(smem + 8192);
  for (int w = 0; w < 8; ++w) {
    uint32_t todo = flags.again[w];
    while (todo) {
      const int ur = w * 32 + __ffs(todo) - 1;
      todo &= todo - 1;
      const size_t row = unit.row_base + ur;
      const TileKV<HD> kv = {kbase, vbase, u};
      for (int c = threadIdx.x; c < HD; c += kThreads)
        q[c] = load_f32(static_cast<const __nv_bfloat16*>(a.q) + row * HD + c);
      __syncthreads();
      float m, l, o;
      literal_row<kThreads, HD>(kv, q, range_of(p.by_Nq.mod(unit.r0 + ur)), a.sc, scratch, BlockSync{},
                                m, l, o);
      const float inv = l == 0.f ? 0.f : 1.f / l;
      const float lsev = l == 0.f ? -INFINITY : m + log2f(l);
      if (threadIdx.x < HD) {
        if (unit.partial) p.opart[(unit.pbase + ur) * HD + threadIdx.x] = o * inv;
        else store_f32(static_cast<T*>(a.out) + row * HD + threadIdx.x, o * inv);
      }
      if (threadIdx.x == 0) {
        if (unit.partial) p.lpart[unit.pbase + ur] = lsev;
        else if (a.lse) a.lse[row] = lsev * kLn2F;
      }
      __syncthreads();
    }
  }
}

// T: the output type; the inputs are bf16.
template <int HD, typename T>
__global__ void __launch_bounds__(kThreads, 1)
    window_attn_kernel(const __grid_constant__ WindowMaps maps,
                       const __grid_constant__ WindowKernelParams p) {
  using L = Smem<HD>;
  constexpr int kAtoms = HD / 64;
  const WindowArgs& a = p.a;
  if (threadIdx.x >= 8 * 32 && threadIdx.x < 8 * 32 + 3)
    prefetch_map(threadIdx.x == 8 * 32 ? &maps.q : threadIdx.x == 8 * 32 + 1 ? &maps.k : &maps.v);
  // Put in place beside the tail of what came before on the stream, all of which is
  // waited for here, before anything is read. (One token 13.9 to 13.6 us, the ragged
  // prompts 20.1 to 19.7.) The combine kernel, if there is one, is put in place likewise.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  // block = (unit, split)
  const bool partial = static_cast<int>(blockIdx.x) >= p.whole && p.splits > 1;
  const int splits = partial ? p.splits : 1;
  const int cut = static_cast<int>(blockIdx.x) - p.whole;  // block among those of cut units
  const int unit = partial ? p.whole + p.by_splits.div(cut) : static_cast<int>(blockIdx.x);
  const int split = partial ? p.by_splits.mod(cut) : 0;
  int seg, tile;
  unit_place(p, unit, seg, tile);
  const bool packed = p.R != a.Nq;  // the rows of all query heads of a key head
  const int bh0 = packed ? seg * p.group : seg;  // first (sequence, query head) of the segment
  const int b = p.by_Hq.div(bh0), head0 = bh0 - b * a.Hq;
  const int kvh = b * a.Hkv + p.by_group.div(head0);
  const bool report = split == 0 && tile == 0 && head0 == 0 && threadIdx.x == 0;
  const int n = clamp_count(a.n_q, b, a.Nq, a.Nq, a.stats, report);
  const int len = clamp_count(a.n_k, b, a.Nk, a.Nk, a.stats, report);
  const int r0 = tile * p.unit_rows;
  const int rows_unit = min(p.unit_rows, p.R - r0);
  const int nq = rows_unit > kTileM ? 2 : 1;
  const size_t row_base = static_cast<size_t>(bh0) * a.Nq + r0;  // of q, out, lse
  // first and last query of the unit (packed rows wrap from head to head)
  int i_first = p.by_Nq.mod(r0), i_last = p.by_Nq.mod(r0 + rows_unit - 1);
  if (i_last - i_first != rows_unit - 1) {
    i_first = 0;
    i_last = a.Nq - 1;
  }
  if (i_first >= n) return;  // every row lies behind the sequence
  i_last = min(i_last, n - 1);
  const long long pos0 = static_cast<long long>(len) - n;  // position of query 0
  UnitKeys u;
  {
    const Range first = visible_range(a.see, max(pos0 + i_first, 0ll), len, p.by_frame);
    const Range last = visible_range(a.see, pos0 + i_last, len, p.by_frame);
    u.SA = last.s;
    u.LB = first.lo;
    u.HB = last.hi;
    if (u.LB <= u.SA) {  // one range
      u.SA = 0;
      u.LB = 0;
    }
    u.HB = max(u.HB, u.LB);
  }
  u.TA = (u.SA + kTileN - 1) / kTileN;
  const int T_all = u.TA + (u.HB - u.LB + kTileN - 1) / kTileN;
  u.j0 = 0;
  u.T = T_all;
  if (partial) {  // (fewer than 2^24 tiles and 16 splits)
    u.j0 = p.by_splits.div(T_all * split);
    u.T = p.by_splits.div(T_all * (split + 1)) - u.j0;
  }
  const int T_tiles = u.T, j0 = u.j0;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const size_t pbase = partial ? static_cast<size_t>(cut) * p.unit_rows : 0;
  T* const out = static_cast<T*>(a.out);

  if (T_tiles == 0) {
    for (int r = threadIdx.x; r < rows_unit; r += kThreads) {
      if (partial) {
        p.lpart[pbase + r] = -INFINITY;
      } else if ((r0 + r) % a.Nq < n) {
        for (int c = 0; c < HD; c += 16 / static_cast<int>(sizeof(T)))
          *reinterpret_cast<uint4*>(out + (row_base + r) * HD + c) = make_uint4(0, 0, 0, 0);
        if (a.lse) a.lse[row_base + r] = -INFINITY;
      }
    }
    return;
  }
  // tasks of warpgroup i: two query tiles -> every key tile; one -> tiles 2t + i
  const bool two = nq == 2;
  const int ntask[2] = {two ? T_tiles : (T_tiles + 1) / 2, two ? T_tiles : T_tiles / 2};
  // A tile that ends behind its key range holds rows of V that no row of the unit sees. They
  // may be anything, also NaN, and a weight of 0 does not silence them: the V warp clears them.
  // (Rows behind the buffer are zero already: TMA fills them.) At most the last tile of each
  // key range is such a tile. (Both are found here: asked tile by tile the clip took 1.5% longer.)
  const bool short_box = p.kv_box_rows < kTileN;
  const int fix_a = u.TA * kTileN > u.SA && (u.SA < a.Nk || short_box) ? u.TA - 1 : -1;
  const int fix_b =
      u.LB + (T_all - u.TA) * kTileN > u.HB && (u.HB < a.Nk || short_box) ? T_all - 1 : -1;
  auto needs_fix = [&](int j) { return j == fix_a || j == fix_b; };

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* Qs = smem + L::q_off;
  uint8_t* Ks = smem + L::k_off;
  uint8_t* Vs = smem + L::v_off;
  Bars* bars = reinterpret_cast<Bars*>(smem + L::bar_off);
  float* ml = reinterpret_cast<float*>(smem + L::ml_off);
  Flags& flags = *reinterpret_cast<Flags*>(smem + L::flag_off);

  if (threadIdx.x == 9 * 32) {  // while warp 0 takes tensor memory
    mbar_init(&bars->q_full[0], 1);
    mbar_init(&bars->q_full[1], 1);
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&bars->kfull[s], 1);
      mbar_init(&bars->vfull[s], 1);
      mbar_init(&bars->kempty[s], 1);
      mbar_init(&bars->vempty[s], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars->vfix[i], 1);
      mbar_init(&bars->s_full[i], 1);
      mbar_init(&bars->p_full[i][0], kTileM);
      mbar_init(&bars->p_full[i][1], kTileM);
      mbar_init(&bars->pa_done[i], 1);
      mbar_init(&bars->o_done[i], 1);
    }
    mbar_init(&bars->mma_idle, 1);
    bars->abort = 0;
    fence_barrier_init();
  }
  if (threadIdx.x < 8) flags.again[threadIdx.x] = flags.values[threadIdx.x] = 0;
  if (warp == 0) {
    tmem_alloc(&bars->tmem_base, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem_base;
  volatile int* abort = &bars->abort;

  if (warp == 8 || warp == 10) {
    // ------- TMA producers: warp 8 Q and the K tiles, warp 10 the V tiles ------
    const bool is_k = warp == 8;
    uint8_t* ring = is_k ? Ks : Vs;
    uint64_t* full = is_k ? bars->kfull : bars->vfull;
    uint64_t* empty = is_k ? bars->kempty : bars->vempty;
    const CUtensorMap* map = is_k ? &maps.k : &maps.v;
    const uint32_t bytes = kAtoms * p.kv_box_rows * 128;
    auto load_q = [&](int qt) {
      mbar_arrive_expect_tx(&bars->q_full[qt], kAtoms * p.q_box_rows * 128);
      for (int c = 0; c < kAtoms; ++c)
        tma_load_2d(Qs + qt * L::kTileBytes + c * L::kSlab, &maps.q, &bars->q_full[qt], c * 64,
                    static_cast<int32_t>(row_base) + qt * kTileM);
    };
    if (is_k && lane == 0) load_q(0);
    int issued = -1, fixes = 0;
    for (int j = 0; j < T_tiles; ++j) {
      const int st = j % kStages, k0 = u.start(j0 + j);
      bool ok = true;
      if (lane == 0) {
        if (j >= kStages) ok = mbar_wait(&empty[st], ((j / kStages) + 1) & 1, abort);
        if (ok) {
          mbar_arrive_expect_tx(&full[st], bytes);
          for (int c = 0; c < kAtoms; ++c)
            tma_load_3d(ring + st * L::kTileBytes + c * L::kSlab, map, &full[st], c * 64, k0, kvh);
          if (is_k && j == 0 && two) load_q(1);  // needed after the first products of tile 0
        }
      }
      if (!__shfl_sync(0xffffffffu, ok, 0)) break;
      issued = j;
      if (!is_k && needs_fix(j0 + j)) {
        ok = mbar_wait(&full[st], (j / kStages) & 1, abort);
        if (!__all_sync(0xffffffffu, ok)) break;
        for (int c = 0; c < kAtoms; ++c)
          for (int x = (u.end(j0 + j) - k0) * 8 + lane; x < kTileN * 8; x += 32)
            *reinterpret_cast<uint4*>(ring + st * L::kTileBytes + c * L::kSlab + x * 16) =
                make_uint4(0, 0, 0, 0);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->vfix[fixes]);
        ++fixes;
      }
    }
    // let the loads already in flight land before the block goes on
    if (lane == 0) {
      volatile int never = 0;
      for (int j = max(0, issued - kStages + 1); j <= issued; ++j)
        mbar_wait(&full[j % kStages], (j / kStages) & 1, &never);
      if (is_k) {
        mbar_wait(&bars->q_full[0], 0, &never);
        if (two) mbar_wait(&bars->q_full[1], 0, &never);
      }
    }
  } else if (warp == 9) {
    // ------------------------------ MMA issuer --------------------------------
    // The whole warp walks the loop, so that addresses stay in uniform registers,
    // and one elected lane issues; a descriptor is a base plus a constant (with
    // one lane in the loop, each product took 120 cycles to issue, not 64).
    constexpr uint32_t idS = idesc_bf16(kTileM, kTileN, 0);
    constexpr uint32_t idO = idesc_bf16(kTileM, HD, 1);
    const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
    const uint64_t q_desc = smem_desc_sw128(smem_u32(Qs), 16, 1024);
    const uint64_t k_desc = smem_desc_sw128(smem_u32(Ks), 16, 1024);
    const uint64_t v_desc = smem_desc_sw128(smem_u32(Vs), L::kSlab, 1024);
    const bool leader = elect_one();
    bool ok = true;
    auto kv_of = [&](int i, int t) { return two ? t : 2 * t + i; };
    // S_i = Q_(tile of i) K(kv)^T
    auto issue_s = [&](int i, int t) -> bool {
      const int kv = kv_of(i, t), st = kv % kStages;
      if (!__all_sync(0xffffffffu, mbar_wait(&bars->kfull[st], (kv / kStages) & 1, abort))) return false;
      tc_fence_after();
      const uint64_t qd = q_desc + static_cast<uint64_t>((two ? i : 0) * (L::kTileBytes >> 4));
      const uint64_t kd = k_desc + static_cast<uint64_t>(st * (L::kTileBytes >> 4));
      const uint32_t d_tmem = tm + static_cast<uint32_t>(i * kTileN);
      if (leader) {
#pragma unroll
        for (int ks = 0; ks < HD / 16; ++ks) {
          const uint64_t off = ((ks >> 2) * L::kSlab + (ks & 3) * 32) >> 4;
          mma_bf16_ss(d_tmem, qd + off, kd + off, idS, ks > 0 ? 1u : 0u);
        }
        mma_commit(&bars->s_full[i]);
        if (!two || i == 1) mma_commit(&bars->kempty[st]);  // last reader of K(kv)
      }
      __syncwarp();
      return true;
    };
    // O_i += P_i V(kv), P_i from tensor memory, each half as soon as it is stored
    int fixes = 0, fix_of = -1;
    auto issue_pv = [&](int i, int t) -> bool {
      const int kv = kv_of(i, t), st = kv % kStages;
      if (!__all_sync(0xffffffffu, mbar_wait(&bars->vfull[st], (kv / kStages) & 1, abort))) return false;
      if (kv > fix_of && needs_fix(j0 + kv)) {
        if (!__all_sync(0xffffffffu, mbar_wait(&bars->vfix[fixes], 0, abort))) return false;
        fix_of = kv;
        ++fixes;
      }
      const uint64_t vd = v_desc + static_cast<uint64_t>(st * (L::kTileBytes >> 4));
      const uint32_t o_tmem = tm + 2u * kTileN + static_cast<uint32_t>(i * HD);
      const uint32_t p_tmem = tm + static_cast<uint32_t>(i * kTileN);
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        if (!__all_sync(0xffffffffu, mbar_wait(&bars->p_full[i][hf], t & 1, abort))) return false;
        tc_fence_after();
        if (leader) {
#pragma unroll
          for (int k = 0; k < kTileN / 32; ++k) {
            const int ks = hf * (kTileN / 32) + k;
            mma_bf16_ts(o_tmem, p_tmem + static_cast<uint32_t>(ks * 8),
                        vd + static_cast<uint64_t>((ks * 16 * 128) >> 4), idO,
                        (t > 0 || ks > 0) ? 1u : 0u);
          }
          if (hf == 0) {
            mma_commit(&bars->pa_done[i]);
          } else {
            if (!two || i == 1) mma_commit(&bars->vempty[st]);  // last reader of V(kv)
            if (t == ntask[i] - 1) mma_commit(&bars->o_done[i]);
          }
        }
        __syncwarp();
      }
      return true;
    };
    for (int i = 0; i < 2 && ok; ++i) {
      if (i == 0 || two) ok = __all_sync(0xffffffffu, mbar_wait(&bars->q_full[i], 0, abort));
      if (ok && ntask[i] > 0) ok = issue_s(i, 0);
    }
    const int nt = max(ntask[0], ntask[1]);
    for (int t = 0; t < nt && ok; ++t)
      for (int i = 0; i < 2 && ok; ++i) {
        if (t >= ntask[i]) continue;
        ok = issue_pv(i, t);
        if (ok && t + 1 < ntask[i]) ok = issue_s(i, t + 1);
      }
    // all issued MMAs complete before the block releases tensor memory
    if (leader) mma_commit(&bars->mma_idle);
    __syncwarp();
    volatile int never = 0;
    mbar_wait(&bars->mma_idle, 0, &never);
  } else {
    // ------------- softmax: warpgroup i = warp / 4, thread = row -------------
    const int i = warp >> 2;
    const int row = (warp & 3) * 32 + lane;  // 0..127 == TMEM lane
    const int ur = two ? i * kTileM + row : row;  // row of the unit
    const uint32_t lane_base = static_cast<uint32_t>(((warp & 3) * 32) << 16);
    const uint32_t s_tmem = tmem + lane_base + static_cast<uint32_t>(i * kTileN);
    const uint32_t o_base = tmem + lane_base + 2u * kTileN;
    const float sc = a.sc;
    const int qi = p.by_Nq.mod(r0 + ur);
    const bool valid = ur < rows_unit && qi < n;
    Range rg = {0, 0, 0};
    if (valid) rg = visible_range(a.see, pos0 + qi, len, p.by_frame);
    // rows that nobody reads, and rows that see nothing, take every key unmasked
    // against the reference 0 and are dropped at the end
    const bool live = valid && (rg.s > 0 || rg.hi > rg.lo);
    // no live row of the warp sees a key that is neither below s_end nor in [lo_first, hi_end)
    const int s_end = __reduce_max_sync(0xffffffffu, live ? rg.s : 0);
    const int lo_first = __reduce_min_sync(0xffffffffu, live ? rg.lo : 0x7fffffff);
    const int hi_end = __reduce_max_sync(0xffffffffu, live ? rg.hi : 0);
    float m_ref = live ? -INFINITY : 0.f, l_sum = 0.f;
    bool ok = true, seen = false;
    for (int t = 0; t < ntask[i]; ++t) {
      const int kv = two ? t : 2 * t + i;  // local key tile
      const int k0 = u.start(j0 + kv), k1 = u.end(j0 + kv);
      const bool whole = !live || (k1 == k0 + kTileN && (k1 <= rg.s || (rg.lo <= k0 && k1 <= rg.hi) ||
                                                         (rg.s == rg.lo && k1 <= rg.hi)));
      const bool masked = !__all_sync(0xffffffffu, whole);
      uint32_t km[4] = {0xFFFFFFFFu, 0xFFFFFFFFu, 0xFFFFFFFFu, 0xFFFFFFFFu};
      if (masked && !whole) {
        const int e = min(rg.s, k1) - k0, lo = rg.lo - k0, hi = min(rg.hi, k1) - k0;
#pragma unroll
        for (int w = 0; w < 4; ++w)
          km[w] = bit_range(-32 * w, e - 32 * w) | bit_range(lo - 32 * w, hi - 32 * w);
      }
      seen = seen || (km[0] | km[1] | km[2] | km[3]) != 0u;
      // tcgen05.ld / st below are warp-collective: the warp proceeds or stops as one
      if (!__all_sync(0xffffffffu, mbar_wait(&bars->s_full[i], t & 1, abort))) { ok = false; break; }
      tc_fence_after();
      // Only rows of other warps see the tile. (32 heads of 8,192 rows, d = 64, a window of
      // 1,024: 160.5 to 155.6 us. Halves of tiles told apart the same way took 156.5, and 4%
      // more where every tile is seen whole.)
      if (k0 >= s_end && (k0 >= hi_end || k1 <= lo_first)) {
        uint32_t none[32];
#pragma unroll
        for (int c = 0; c < 32; ++c) none[c] = 0u;
        tmem_st32(s_tmem, none);
        tmem_st32(s_tmem + 32, none);
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(&bars->p_full[i][0]);
        mbar_arrive(&bars->p_full[i][1]);
        continue;
      }
      // The row is processed in two halves of 64 key columns: S half hf is
      // loaded, exponentiated and packed, and its P stored over columns
      // [32 hf, 32 hf + 32) of S_i, columns that hold S values already read.
      uint32_t r[kTileN / 2];
      auto load_half = [&](int hf) {
        tmem_ld32(s_tmem + hf * 64, *reinterpret_cast<uint32_t(*)[32]>(r));
        tmem_ld32(s_tmem + hf * 64 + 32, *reinterpret_cast<uint32_t(*)[32]>(r + 32));
        tmem_wait_ld();
        if (masked) {
#pragma unroll
          for (int c = 0; c < kTileN / 2; ++c)
            if (!((km[2 * hf + (c >> 5)] >> (c & 31)) & 1u)) r[c] = __float_as_uint(-INFINITY);
        }
      };
      // scaled maximum of the loaded half: eight chains of three-input maxima
      auto half_max = [&]() -> float {
        float m8[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) m8[k] = __uint_as_float(r[k]);
#pragma unroll
        for (int c = 8; c < kTileN / 2; c += 2)
          m8[(c >> 1) & 7] = max3f(m8[(c >> 1) & 7], __uint_as_float(r[c]), __uint_as_float(r[c + 1]));
        return sc * fmaxf(max3f(m8[0], m8[1], m8[2]),
                          fmaxf(max3f(m8[3], m8[4], m8[5]), fmaxf(m8[6], m8[7])));
      };
      // P = 2^(s sc - m_ref) of the loaded half as bf16 pairs; returns its sum
      uint32_t pk[32];
      auto exp_half = [&](float mref) -> float {
        float2 r4[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f),
                        make_float2(0.f, 0.f)};
        const float nm = (mref == -INFINITY) ? 0.f : -mref;  // no visible key yet: P = 0
#pragma unroll
        for (int c = 0; c < kTileN / 2; c += 2) {
          float xa, xb;
          fma2(xa, xb, __uint_as_float(r[c]), __uint_as_float(r[c + 1]), sc, nm);
          const float ea = ex2_approx(xa), eb = ex2_approx(xb);
          add2(r4[(c >> 1) & 3], ea, eb);
          pk[c >> 1] = pack_bf16x2(ea, eb);
        }
        return (r4[0].x + r4[0].y + r4[1].x + r4[1].y) + (r4[2].x + r4[2].y + r4[3].x + r4[3].y);
      };
      // Reference maximum m_ref: the row maximum of the first tile that holds
      // one of the row's keys, rounded up to a whole number (so that a move by k
      // below is exact; a reference of 2^22 and more goes to the literal pass);
      // later tiles are exponentiated against it with no
      // maximum pass. A half whose sum exceeds 2^32 moves the reference up by
      // the whole number k of log2 units that brings its largest value to at
      // most 1: its values are formed again, and the row sum and O are scaled
      // by 2^-k, exactly. O and the row sum always share one reference, so the
      // result is exact. The sum stays finite, and NaN in it comes from a visible logit that
      // is NaN or +inf: the row's softmax is NaN then.
      if (__any_sync(0xffffffffu, m_ref == -INFINITY)) {
        load_half(0);
        const float m0 = half_max();
        load_half(1);
        const float mt = fmaxf(m0, half_max());
        if (m_ref == -INFINITY) m_ref = ceilf(mt);
      }
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        load_half(hf);
        float rh = exp_half(m_ref);
        const bool over = live && rh > kOverflowSum;
        if (__any_sync(0xffffffffu, over)) {
          load_half(hf);
          float sh = 1.f;  // 2^-k, formed from its bits (0 when k >= 127)
          if (over) {
            const float k = ceilf(half_max() - m_ref);
            sh = (k < 127.f) ? __int_as_float((127 - static_cast<int>(k)) << 23) : 0.f;
            m_ref += k;
          }
          rh = exp_half(m_ref);
          l_sum *= sh;
          // O holds the products of the tiles before (they precede S_i(t)) and, in
          // the second half, those of the first half
          bool there = true;
          if (hf == 1) there = mbar_wait(&bars->pa_done[i], t & 1, abort);
          if (!__all_sync(0xffffffffu, there)) { ok = false; break; }
          tc_fence_after();
          if (t > 0 || hf == 1) {
            const uint32_t o_tmem = o_base + static_cast<uint32_t>(i * HD);
#pragma unroll 1
            for (int c = 0; c < HD / 32; ++c) {
              uint32_t o[32];
              tmem_ld32(o_tmem + c * 32, o);
              tmem_wait_ld();
#pragma unroll
              for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * sh);
              tmem_st32(o_tmem + c * 32, o);
            }
          }
        }
        tmem_st32(s_tmem + hf * 32, pk);
        l_sum += rh;
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(&bars->p_full[i][hf]);
      }
      if (!ok) break;
    }
    // ---------------- epilogue: O / l -> global -------------------------------
    float f0, f1 = 0.f, lsev;  // factors of this thread's O and the other one's, log2-sum-exp
    bool has1 = false, use0 = false, use1 = false;  // one tile: halves that hold keys of the row
    bool lost;  // the row's softmax is NaN
    if (two) {
      lost = live && l_sum != l_sum;
      f0 = lost ? l_sum : live && l_sum > 0.f ? 1.f / l_sum : 0.f;
      lsev = live && l_sum > 0.f ? m_ref + __log2f(l_sum) : -INFINITY;
      if (live && !lost && seen && (l_sum == 0.f || !(l_sum < INFINITY) || !(fabsf(m_ref) < kMaxReference)))
        atomicOr(&flags.again[ur >> 5], 1u << (ur & 31));
      ok = ok && mbar_wait(&bars->o_done[i], 0, abort);
    } else {
      // merge the two halves of the key tiles: each warpgroup writes half of
      // the columns of every row
      ml[i * 2 * kTileM + row] = m_ref;
      ml[i * 2 * kTileM + kTileM + row] = l_sum;
      named_barrier_sync(1, 2 * kTileM);
      const float m0 = ml[row], l0 = ml[kTileM + row];
      const float m1 = ml[2 * kTileM + row], l1 = ml[3 * kTileM + row];
      has1 = ntask[1] > 0;
      lost = live && (l0 != l0 || (has1 && l1 != l1));
      const float mm = has1 ? fmaxf(m0, m1) : m0;
      // a half that holds none of the row's keys has the reference -inf
      use0 = m0 != -INFINITY;
      use1 = has1 && m1 != -INFINITY;
      const float a0 = use0 ? ex2_approx(m0 - mm) : 0.f;
      const float a1 = use1 ? ex2_approx(m1 - mm) : 0.f;
      const float l = l0 * a0 + (has1 ? l1 * a1 : 0.f);
      const bool far = mm != -INFINITY && !(fabsf(mm) < kMaxReference);
      const float inv = lost ? __int_as_float(0x7fc00000) : live && l > 0.f ? 1.f / l : 0.f;
      use0 = use0 || lost;
      f0 = a0 * inv;
      f1 = a1 * inv;
      lsev = live && l > 0.f ? mm + __log2f(l) : -INFINITY;
      if (live && !lost && ((seen && l == 0.f) || !(l < INFINITY) || far))
        atomicOr(&flags.again[ur >> 5], 1u << (ur & 31));
      ok = ok && mbar_wait(&bars->o_done[0], 0, abort);
      if (has1) ok = ok && mbar_wait(&bars->o_done[1], 0, abort);
    }
    if (lost) lsev = __int_as_float(0x7fc00000);
    if (__all_sync(0xffffffffu, ok)) {
      tc_fence_after();
      const bool leads = two || i == 0;
      if (leads && valid) {
        if (partial) p.lpart[pbase + ur] = lsev;
        else if (a.lse) a.lse[row_base + ur] = lsev * kLn2F;
      } else if (leads && partial && ur < rows_unit) {
        p.lpart[pbase + ur] = -INFINITY;
      }
      bool finite = true;
      constexpr int kHalf = HD / 64;  // 32-column pieces of half a row
      const uint32_t rows = __ballot_sync(0xffffffffu, valid);
      const int ur0 = ur - lane;  // the warp's first row
      // the query tile has been read: a quarter of it for each warp
      uint4* stage = reinterpret_cast<uint4*>(Qs + i * L::kTileBytes + (warp & 3) * (L::kTileBytes / 4));
#pragma unroll
      for (int c = 0; c < 2 * kHalf; ++c) {
        if (!two && c / kHalf != i) continue;

        uint32_t o[32];
        tmem_ld32(o_base + (two ? i * HD : 0) + c * 32, o);
        tmem_wait_ld();
        if (!two) {
          uint32_t o1[32];
          if (has1) {
            tmem_ld32(o_base + HD + c * 32, o1);
            tmem_wait_ld();
          }
#pragma unroll
          for (int k = 0; k < 32; ++k)
            o[k] = __float_as_uint((use0 ? __uint_as_float(o[k]) * f0 : 0.f) +
                                   (use1 ? __uint_as_float(o1[k]) * f1 : 0.f));
        }
        const float f = two ? f0 : 1.f;
        float sum = 0.f;  // NaN when a value is not finite
#pragma unroll
        for (int k = 0; k < 32; ++k) sum += __uint_as_float(o[k]) * 0.f;
        finite = finite && sum == 0.f;
        if (!live) {
#pragma unroll
          for (int k = 0; k < 32; ++k) o[k] = 0u;
        }
        if (partial) RowStage<float, HD>::put(stage, lane, c % kHalf, o, f);
        else RowStage<T, HD>::put(stage, lane, c % kHalf, o, f);
        if (c % kHalf == kHalf - 1) {
          const int col = c / kHalf * (HD / 2);
          if (partial) RowStage<float, HD>::flush(stage, lane, p.opart + (pbase + ur0) * HD + col, rows);
          else RowStage<T, HD>::flush(stage, lane, out + (row_base + ur0) * HD + col, rows);
        }
      }
      if (live && !lost && !finite) atomicOr(&flags.values[ur >> 5], 1u << (ur & 31));
    }
  }
  __syncthreads();
  const bool aborted = *abort != 0;
  if (aborted && threadIdx.x == 0) raise_status(a.stats, SPARSEPR_ERR_TIMEOUT);
  if (warp == 0) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
  if (aborted) return;
  uint32_t any = 0;
  for (int w = 0; w < 8; ++w) any |= flags.again[w] | flags.values[w];
  if (any)
    look_again<HD, T>(p, Unit{u, r0, i_last, len, partial, pos0, kvh, row_base, pbase}, smem, flags);
}

// out = sum_s 2^(l_s - M) O_s / sum_s 2^(l_s - M), M = max_s l_s, over the splits'
// normalised partial outputs in a fixed order; a split without any of the
// row's keys has l_s = -inf and is left out (one whose weight is 0 only by underflow is
// not: it may hold NaN or infinities that the row sees). A warp per row: the lanes take one
// split's log-sum-exp each, then HD / 32 columns each.
template <int HD, typename T>
__global__ void __launch_bounds__(256) window_combine_kernel(const WindowKernelParams p) {
  constexpr int kC = HD / 32;
  const WindowArgs& a = p.a;
  asm volatile("griddepcontrol.wait;" ::: "memory");  // all of the attention kernel's writes
  const int lane = threadIdx.x & 31;
  int seg, tile;
  unit_place(p, p.whole + static_cast<int>(blockIdx.y), seg, tile);
  const int r = blockIdx.x * 8 + (threadIdx.x >> 5), r0 = tile * p.unit_rows;
  const int bh0 = p.R != a.Nq ? seg * p.group : seg;
  const int n = clamp_count(a.n_q, bh0 / a.Hq, a.Nq, a.Nq, a.stats, false);
  if (r0 + r >= p.R || r >= p.unit_rows || (r0 + r) % a.Nq >= n) return;
  const size_t base = static_cast<size_t>(blockIdx.y) * p.splits * p.unit_rows + r;
  const size_t row = static_cast<size_t>(bh0) * a.Nq + r0 + r;
  static_assert(kMaxWindowSplits <= 32, "a lane per split");
  // everything is asked for at once: with the parts behind the sums, eight at a time, a call
  // of one token took 16.8 us, not 13.8, and a frame against the cache 230 us, not 221
  const float l = lane < p.splits ? p.lpart[base + static_cast<size_t>(lane) * p.unit_rows] : -INFINITY;
  using Piece = typename std::conditional<kC == 4, float4, float2>::type;
  static_assert(sizeof(Piece) == kC * sizeof(float), "columns of a lane");
  union {
    Piece piece;
    float v[kC];
  } part[kMaxWindowSplits];
#pragma unroll
  for (int s = 0; s < kMaxWindowSplits; ++s)
    if (s < p.splits)
      part[s].piece = *reinterpret_cast<const Piece*>(
          p.opart + (base + static_cast<size_t>(s) * p.unit_rows) * HD + lane * kC);
  float M = l;
#pragma unroll
  for (int w = 16; w > 0; w >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, w));
  const bool nan = __any_sync(0xffffffffu, l != l);
  const uint32_t there = __ballot_sync(0xffffffffu, l != -INFINITY);
  const float weight = l == -INFINITY ? 0.f : exp2f(l - M);
  float num[kC] = {}, den = 0.f;
#pragma unroll
  for (int s = 0; s < kMaxWindowSplits; ++s) {
    const float w = __shfl_sync(0xffffffffu, weight, s);
    if ((there >> s) & 1u) {  // a range without a key of the row may not have written its part
      den += w;
#pragma unroll
      for (int e = 0; e < kC; ++e) num[e] = fmaf(w, part[s].v[e], num[e]);
    }
  }
  const float inv = den > 0.f || nan ? 1.f / den : 0.f;
  T* out = static_cast<T*>(a.out) + row * HD + lane * kC;
#pragma unroll
  for (int e = 0; e < kC; ++e) store_f32(out + e, num[e] * inv);
  if (a.lse && lane == 0)
    a.lse[row] = nan ? den : den > 0.f ? (M + log2f(den)) * kLn2F : -INFINITY;
}

bool make_map2(CUtensorMap* m, const void* base, size_t rows, int d, int box_rows) {
  EncodeTiledFn enc = encode_tiled_fn();
  if (!enc) return false;
  cuuint64_t dims[2] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(rows)};
  cuuint64_t strides[1] = {static_cast<cuuint64_t>(d) * 2};
  cuuint32_t box[2] = {64, static_cast<cuuint32_t>(box_rows)};
  cuuint32_t es[2] = {1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box,
             es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// [heads, rows, d]: rows past a head's end read as zero
bool make_map3(CUtensorMap* m, const void* base, int heads, int rows, int d, int box_rows) {
  EncodeTiledFn enc = encode_tiled_fn();
  if (!enc) return false;
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(rows),
                        static_cast<cuuint64_t>(heads)};
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(d) * 2,
                           static_cast<cuuint64_t>(rows) * d * 2};
  cuuint32_t box[3] = {64, static_cast<cuuint32_t>(box_rows), 1};
  cuuint32_t es[3] = {1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box,
             es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int HD, typename T>
cudaError_t launch_hd(const WindowKernelParams& p, const WindowMaps& maps, int units,
                      cudaStream_t st) {
  static std::atomic<uint64_t> allowed{0};
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(window_attn_kernel<HD, T>), kSmemBytes,
                             allowed);
  if (e != cudaSuccess) return e;
  const unsigned blocks = static_cast<unsigned>(p.whole) +
                          static_cast<unsigned>(units - p.whole) * p.splits;
  cudaLaunchConfig_t first = {};  // programmatic dependent launch
  first.gridDim = dim3(blocks);
  first.blockDim = dim3(kThreads);
  first.dynamicSmemBytes = kSmemBytes;
  first.stream = st;
  cudaLaunchAttribute early[1];
  early[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early[0].val.programmaticStreamSerializationAllowed = 1;
  first.attrs = early;
  first.numAttrs = 1;
  e = cudaLaunchKernelEx(&first, window_attn_kernel<HD, T>, maps, p);
  if (e != cudaSuccess || p.whole == units) return e;
  // launched beside the tail of the attention kernel
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((min(p.unit_rows, p.R) + 7) / 8, units - p.whole);
  cfg.blockDim = dim3(256);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, window_combine_kernel<HD, T>, p);
}

}  // namespace

// How the rows are cut, from the sizes alone.
//   - Short query runs of heads that share a key head are packed into one tile:
//     their rows are contiguous, and the tile's 128 rows are filled.
//   - Units have 256 rows (two tiles, each key tile read once for both) or 128, and
//     the key tiles of the units that do not fill a last round of the multiprocessors,
//     or of all units, may be split over several blocks that are joined afterwards:
//     whichever the estimate below holds for fastest. One block runs per
//     multiprocessor, so blocks take as many rounds as they fill multiprocessors, the
//     last one as long as a full one. A key tile costs 1 for 256 rows and 0.6 for 128
//     (measured 1.7 us and 1.0 us), a block 4 beside its tiles, partial results what
//     their bytes take at 6.5 TB/s, and the combine kernel 2. (A frame of 1,560 rows and
//     12 heads against 21,840 keys: 156 units of 128 rows are two rounds, 357 us; 84 of 256
//     rows in 5 splits three rounds of a fifth, 221 us.)
WindowPlan window_plan(int B, int Hq, int Hkv, int Nq, int Nk, const sparsepr_visibility& see) {
  WindowPlan w = {};
  const int group = Hq / Hkv;
  const bool pack = group > 1 && Nq < kTileM;
  w.R = pack ? group * Nq : Nq;
  w.segs = pack ? B * Hkv : B * Hq;
  double best = -1.0;
  for (int rows = 2 * kTileM; rows >= kTileM; rows -= kTileM) {
    if (rows > kTileM && w.R <= kTileM) continue;
    const long long tiles = (static_cast<long long>(w.R) + rows - 1) / rows, units = tiles * w.segs;
    const long long keys = most_visible(see, rows, Nk);
    const long long key_tiles = (keys + kTileN - 1) / kTileN;
    const double tile_cost = rows > kTileM ? 1.0 : 0.6;
    const auto rounds = [&](long long blocks, long long part) {
      return (blocks + kPlanSMs - 1) / kPlanSMs * (part * tile_cost + 4.0);
    };
    const long long full = units / kPlanSMs * kPlanSMs;  // units of full rounds
    for (const long long whole : {units, full, 0ll}) {
      for (int splits = 1; splits <= kMaxWindowSplits && splits <= key_tiles; ++splits) {
        const long long cut = units - whole;
        if ((cut == 0) != (splits == 1)) continue;  // something to split, or nothing
        if (cut * splits > 16 * kPlanSMs) break;
        double cost = rounds(whole, key_tiles);
        if (cut > 0)
          cost += rounds(cut * splits, (key_tiles + splits - 1) / splits) + 2.0 +
                  static_cast<double>(cut * splits) * rows * 1024 / (6.5e6 * 1.7);
        if (best < 0.0 || cost < best) {
          best = cost;
          w.unit_rows = rows;
          w.tiles = static_cast<int>(tiles);
          w.units = static_cast<int>(units);
          w.whole = static_cast<int>(whole);
          w.splits = splits;
        }
      }
    }
    if (best < 0.0) {  // no keys at all
      w.unit_rows = rows;
      w.tiles = static_cast<int>(tiles);
      w.units = w.whole = static_cast<int>(units);
      w.splits = 1;
    }
  }
  w.part_rows = static_cast<size_t>(w.units - w.whole) * w.splits * w.unit_rows;
  return w;
}

cudaError_t launch_window_attention(const WindowArgs& in, cudaStream_t st) {
  WindowKernelParams p = {};
  p.a = in;
  WindowArgs& a = p.a;
  if (a.Nq == 0) return cudaSuccess;
  const WindowPlan w = window_plan(a.B, a.Hq, a.Hkv, a.Nq, a.Nk, a.see);
  p.group = a.Hq / a.Hkv;
  p.R = w.R;
  p.segs = w.segs;
  p.tiles = w.tiles;
  p.unit_rows = w.unit_rows;
  p.whole = w.whole;
  p.splits = w.splits;
  p.by_segs = Divider(p.segs);
  p.by_group = Divider(p.group);
  p.by_Hq = Divider(a.Hq);
  p.by_Nq = Divider(a.Nq);
  p.by_splits = Divider(p.splits);
  p.by_frame = Divider(a.see.frame);
  p.opart = a.opart;
  p.lpart = a.lpart;
  const size_t q_rows = static_cast<size_t>(a.B) * a.Hq * a.Nq;
  const size_t kv_rows = static_cast<size_t>(a.B) * a.Hkv * a.Nk;
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const bool f32 = !a.bf16;
  if (f32) {  // the MMAs take bf16
    if ((e = launch_cast_bf16(static_cast<const float*>(a.q), a.qb, q_rows * a.d, st)) != cudaSuccess)
      return e;
    a.q = a.qb;
    if (kv_rows > 0 && !a.kv_bf16) {
      if ((e = launch_cast_bf16(static_cast<const float*>(a.k), a.kb, kv_rows * a.d, st)) != cudaSuccess ||
          (e = launch_cast_bf16(static_cast<const float*>(a.v), a.vb, kv_rows * a.d, st)) != cudaSuccess)
        return e;
      a.k = a.kb;
      a.v = a.vb;
    }
  }
  WindowMaps maps;
  p.q_box_rows = q_rows < static_cast<size_t>(kTileM) ? static_cast<int>(q_rows) : kTileM;
  // without keys no tile is read; the maps then describe the queries
  p.kv_box_rows = a.Nk < kTileN ? max(a.Nk, 1) : kTileN;
  if (!make_map2(&maps.q, a.q, q_rows, a.d, p.q_box_rows)) return cudaErrorInvalidValue;
  if (a.Nk > 0) {
    if (!make_map3(&maps.k, a.k, a.B * a.Hkv, a.Nk, a.d, p.kv_box_rows) ||
        !make_map3(&maps.v, a.v, a.B * a.Hkv, a.Nk, a.d, p.kv_box_rows))
      return cudaErrorInvalidValue;
  } else {
    maps.k = maps.q;
    maps.v = maps.q;
  }
  if (a.d == 128)
    return f32 ? launch_hd<128, float>(p, maps, w.units, st)
               : launch_hd<128, __nv_bfloat16>(p, maps, w.units, st);
  return f32 ? launch_hd<64, float>(p, maps, w.units, st)
             : launch_hd<64, __nv_bfloat16>(p, maps, w.units, st);
}

}  // namespace spr
